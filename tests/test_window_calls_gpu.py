"""The windowed operators in the calls that a server makes around the ordinary
ones.  References and bounds are those of window_util."""
import pytest
import torch

from gpu_util import DevDecode, host
from test_window_gpu import decode_case
from window_util import check, decode_reference

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# One workspace for a batch that shrinks
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("H,r,dtype", [(16, 48, torch.bfloat16), (32, 32, torch.bfloat16), (16, 64, torch.float8_e4m3fn)])
def test_workspace_bytes_never_fall_as_a_call_grows(H, r, dtype):
    import rank_kv_attention_gb300 as L
    need = lambda B, longest, window, sinks: L.decode_window_workspace_bytes(B, H, 128, r, longest, window, sinks, dtype)
    grid = [(B, n, w, s) for B in (1, 2, 3, 4, 8, 12, 16, 24, 48, 64, 200) for n in (1, 40, 700, 2100, 60000)
            for w in (1, 30, 600, 2048, 50000) for s in (0, 4, 300)]
    sizes = {c: need(*c) for c in grid}
    for a, x in sizes.items():
        for b, y in sizes.items():
            if all(p <= q for p, q in zip(a, b)):
                assert x <= y, (a, x, b, y)


@pytest.mark.parametrize("H,r,dtype", [(16, 48, "bf16"), (16, 64, "fp8")])
def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones(H, r, dtype):
    import rank_kv_attention_gb300 as L
    lens = [2100, 5, 2099, 700] * 6
    case = decode_case(lens, H, 128, r, dtype, seed=4)
    d = DevDecode(case)
    # the largest of each size: 24 requests need no more states than 4 or 16 do
    ws = L.workspace(L.decode_window_workspace_bytes(24, H, 128, r, 2100, 2048, 4, d.cache.dtype))
    for window, sinks in ((2048, 4), (300, 0)):
        ref, bound = decode_reference(case, window, sinks)
        for B in (24, 16, 12, 8, 5, 4, 2, 1):
            ws.fill_(0xFF)
            longest = max(lens[:B])
            got = L.decode_window(d.q[:B], d.cache, d.B_K, d.B_V, d.seq_lens[:B], d.page_table[:B], longest, window, sinks, ws=ws)
            check(host(got, case.act_dtype), ref[:B], bound[:B], f"B={B} window={window}")
