"""Chunk attention over long contexts and many partial results, against 64 bits."""
import math

import pytest
import torch

import decode_attention_q4kv_b200 as q4
from helpers import cuda
from test_gpu_extend import Case, _attend_close

pytestmark = pytest.mark.gpu

# two row tiles, one row tile on alternate key tiles, few rows, heads of 256
SHAPES = [(64, 4, 1, 128), (16, 4, 1, 128), (4, 4, 1, 128), (16, 4, 1, 256)]


@pytest.mark.parametrize("T,hq,hkv,d", SHAPES)
@pytest.mark.parametrize("n", [33000, 140001, 300000])
def test_sums_over_long_contexts_do_not_drift(T, hq, hkv, d, n):
    # Values of one sign and nearly equal weights: every partial sum grows all the
    # way.  The plan is asked for one split and takes what keeps an accumulator at
    # 32768 tokens, over which the sums fall short by at most 2^-12.  The roundings of
    # keys, values and weights (rms 2^-11 / sqrt(3) each at most) are independent over
    # the tokens; over 33000 and more of about equal weight the three together come to
    # 2^-11 / 180, less than 2^-17; binary32 sums of weights and the merge add less.
    dev = cuda()
    g = torch.Generator(device=dev).manual_seed(n)
    nb = -(-n // 256)
    pool = q4.Q4KVPool(hkv, d, nb, device=dev)
    ids = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    k = (0.3 * torch.randn(n, hkv, d, generator=g, device=dev)).half()
    v = (4.0 + torch.randn(n, hkv, d, generator=g, device=dev)).half()
    pool.quantize(k, v, ids)
    q = torch.randn(1, T, hq, d, generator=g, device=dev).half()
    plan = q4.ExtendPlan(1, T, hq, hkv, d, nb, n_splits=1)
    out = q4.extend_attention(pool, q, ids[None], torch.tensor([n - T], device=dev), torch.tensor([T], device=dev), plan=plan,
                              out_dtype=torch.float32)
    K, V = (x.transpose(0, 1).reshape(hkv, -1, d)[:, :n].double() for x in pool.dequantize(ids, unrotate_k=True))
    for i, h in ((0, 0), (T // 2, 1), (T - 1, hq - 1)):
        seen = n - T + i + 1
        p = torch.softmax(K[0, :seen] @ q[0, i, h].double() / math.sqrt(d), 0)
        want = p @ V[0, :seen]
        off = float((out[0, i, h].double() - want).norm() / want.norm())
        assert off <= 2.0 ** -12 + 2.0 ** -17, (i, h, plan.n_splits, off)
    assert pool.read_device_error() == 0


@pytest.mark.parametrize("T,hq,hkv,d,lens", [(40, 8, 2, 128, [10300, 4000]), (3, 8, 2, 128, [10300, 77]),
                                             (64, 8, 2, 128, [5200, 300]), (9, 4, 2, 256, [2700, 640])])
def test_more_than_a_warp_of_partial_results(T, hq, hkv, d, lens):
    c = Case(lens, T, hq, hkv, d, "fp16", n_new=[T, T - 1], seed=T)
    plan = q4.ExtendPlan(2, T, hq, hkv, d, c.tables.shape[1], n_splits=10000)    # one step of keys each
    assert plan.n_splits > 32
    want, bound = c.want()
    _attend_close(c.run(plan=plan), want, bound)
    one = q4.ExtendPlan(2, T, hq, hkv, d, c.tables.shape[1], n_splits=1)
    assert one.n_splits == 1
    _attend_close(c.run(plan=one), want, bound)


@pytest.mark.parametrize("T,hq,hkv,d", [(70, 8, 2, 128), (300, 4, 2, 128), (70, 8, 2, 256)])
@pytest.mark.parametrize("widths", [(4, 8, 2), (8, 2), (2, 4)])
@pytest.mark.parametrize("window", [0, 333])
def test_mixed_widths_with_more_rows_than_one_tile(T, hq, hkv, d, widths, window):
    evict = [(0, t) for t in range(0, 700, 9)] + [(1, t) for t in range(256, 330)]
    c = Case([900, 350], T, hq, hkv, d, "bf16", n_new=[T, T - 7], widths=widths, seed=T, evict=evict)
    want, bound = c.want(window=window)
    for s in (0, 1, 3):
        plan = q4.ExtendPlan(2, T, hq, hkv, d, c.tables.shape[1], window=window, n_splits=s)
        _attend_close(c.run(plan=plan, window=window), want, bound, what=f"splits {s}")
    assert c.pool.read_device_error() == 0
