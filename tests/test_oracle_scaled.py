"""The block-scaled cache's float64 definitions, held to closed forms and worked examples."""
import math

import numpy as np
import pytest

import oracle
import oracle.scaled as S
from oracle.fp8 import e4m3_decode


def one_pool(page_size=16, block=16, heads=1, width=2, pages=2):
    codes = {k: np.zeros((pages, page_size, heads, width), np.uint8) for k in S.POOLS}
    exps = {k: np.zeros((pages, page_size // block, heads), np.uint8) for k in S.POOLS}
    return S.Cache(codes, exps)


def put(cache, x, start, table=((0, 1),)):
    n = len(x)
    rows = {k: np.asarray(x, np.float64).reshape(n, 1, -1) for k in S.POOLS}
    S.write(cache, rows, [0, n], [start], np.array(table))


@pytest.mark.parametrize("a,e", [(448.0, 0), (448.0001, 1), (1.0, -8), (1.75, -8), (1.7500001, -7), (2.0 ** -140, -117),
                                 (0.0, -117), (3e38, 119), (224.0, -1), (256.0, 0)])
def test_needed_exponent(a, e):
    assert S.needed_exp(a) == e
    if S.MIN_EXP < e < S.MAX_EXP:
        assert a <= math.ldexp(448, e) and a > math.ldexp(448, e - 1)


def test_bytes_outside_the_range_read_as_the_nearest_in_it():
    assert list(S.exp_of([0, 9, 10, 127, 246, 247, 255])) == [-117, -117, -117, 0, 119, 119, 119]


def test_values_of_a_full_range_block_are_bf16_values():
    """code * 2^e has at most four significant bits and stays a normal number over the whole range."""
    for e in (S.MIN_EXP, 0, S.MAX_EXP):
        v = e4m3_decode(np.arange(0x7f, dtype=np.uint8)) * 2.0 ** e
        assert v[1] >= 2.0 ** -126 and v[-1] < 2.0 ** 128
        assert np.array_equal(v.astype(np.float32).view(np.uint32) & 0xffff, np.zeros(0x7f, np.uint32))


def test_a_block_grows_and_its_earlier_rows_keep_their_values():
    c = one_pool()
    put(c, [[1.0, -0.5]], 0)
    assert S.exp_of(c.exps["S_K"][0, 0, 0]) == -8 and c.row("S_K", 0, 0)[0].tolist() == [1.0, -0.5]
    put(c, [[100.0, 0.25]], 1)
    assert S.exp_of(c.exps["S_K"][0, 0, 0]) == -2                    # 100 <= 448 / 4
    assert c.row("S_K", 0, 0)[0].tolist() == [1.0, -0.5]         # a power of two apart: exact
    assert abs(c.row("S_K", 0, 1)[0][0] - 100) <= 100 * 2.0 ** -4
    put(c, [[0.001, 0.0]], 2)                                    # a quiet row does not shrink it
    assert S.exp_of(c.exps["S_K"][0, 0, 0]) == -2


def test_growing_rounds_only_what_leaves_the_normal_range():
    c = one_pool(width=8)
    put(c, [[448, 30, 1, 2.0 ** -6, 3 * 2.0 ** -8, 2.0 ** -9, -2.0 ** -9, 0]], 0)
    put(c, [[448 * 8.0] + [0] * 7], 1)                           # three octaves
    v = c.row("S_K", 0, 0)[0]
    assert v[:4].tolist() == [448, 30, 1, 2.0 ** -6]
    # 3 * 2^-11 and 2^-12 in units of the new scale: subnormal steps of 2^-9, ties to even
    assert v[4:7].tolist() == [2.0 ** -6, 0.0, 0.0]


def test_a_first_slot_begins_its_block_anew():
    c = one_pool()
    put(c, [[1e6, 0.0]], 0)
    put(c, [[1.0, 0.0]], 0)
    assert S.exp_of(c.exps["S_K"][0, 0, 0]) == -8 and c.row("S_K", 0, 0)[0][0] == 1.0


def test_blocks_are_apart():
    c = one_pool(page_size=32, block=16)
    put(c, [[1.0, 0.0]] * 16 + [[1000.0, 0.0]] * 3, 0)
    assert (c.exps["R_V"][0, :, 0].astype(int) - 127).tolist() == [-8, 2]


def test_infinities_and_nan_become_nan_and_decide_nothing():
    c = one_pool(width=4)
    put(c, [[np.inf, -np.inf, np.nan, 1.0]], 0)
    v = c.row("S_K", 0, 0)[0]
    assert np.isnan(v[:3]).all() and v[3] == 1.0 and S.exp_of(c.exps["S_K"][0, 0, 0]) == -8


def test_read_is_the_inverse_of_write_to_half_a_step():
    rng = np.random.default_rng(3)
    c = one_pool(page_size=16, block=16, heads=1, width=8, pages=3)
    x = rng.standard_normal((40, 8)) * np.exp(rng.standard_normal((40, 1)) * 3)
    put(c, x, 0, table=[[2, 0, 1]])
    out = S.read(c, "S_K", [0, 40], [0], np.array([[2, 0, 1]]), np.full((40, 1, 8), 7.0))[:, 0]
    for b in range(0, 40, 16):
        blk, got = x[b:b + 16], out[b:b + 16]
        step = 2.0 ** S.needed_exp(np.abs(blk).max())
        assert np.all(np.abs(got - blk) <= np.maximum(2.0 ** -4 * np.abs(blk), 2.0 ** -10 * step))


def test_attention_is_the_materialised_one():
    rng = np.random.default_rng(4)
    H, d_h, r, n = 2, 16, 8, 5
    c = one_pool(heads=1)
    c.codes = {k: S.e4m3_encode(rng.standard_normal((2, 16, 1 if k[0] == "S" else H, d_h if k[0] == "S" else r)) * 50)
               for k in S.POOLS}
    c.exps = {k: np.full((2, 1, c.codes[k].shape[2]), 121, np.uint8) for k in S.POOLS}
    q, B_K, B_V = rng.standard_normal((H, d_h)), rng.standard_normal((H, d_h, r)), rng.standard_normal((H, d_h, r))
    rows = S.history(c, [1, 0], n)
    pools = [np.stack([c.row(k, 1, j) for j in range(n)]) for k in S.POOLS]
    got = S.attend_query(q, rows, B_K, B_V)
    for h in range(H):
        K = pools[0][:, 0] + pools[2][:, h] @ B_K[h].T
        V = pools[1][:, 0] + pools[3][:, h] @ B_V[h].T
        assert np.allclose(got[h], oracle.attend(q[h], K, V), rtol=1e-12, atol=0)
