"""Calls of the operators that extend a cached prompt as they may be made, each
against the definitions: layouts, strides and arguments at their edges."""
import numpy as np
import pytest
import torch

import decode_attention_q4kv_b200 as q4
from decode_attention_q4kv_b200 import workloads as W
from helpers import cuda, host
from test_gpu_extend import Case, _attend_close

pytestmark = pytest.mark.gpu


def test_output_rows_token_after_token():
    # [T][B][Hq][D] in memory: a sequence's rows lie between those of the others
    dev = cuda()
    c = Case([40, 300, 7], 9, 8, 2, 128, "fp16", n_new=[9, 4, 9], seed=3)
    want, bound = c.want()
    out = torch.full((9, 3, 8, 128), 7.0, device=dev).transpose(0, 1)
    _attend_close(c.run(out=out), want, bound)
    with pytest.raises(q4.Q4KVError):          # neighbours' rows in one place
        c.run(out=torch.zeros(11 * 8 * 128, device=dev).as_strided((3, 9, 8, 128), (1024, 1024, 128, 1)))


@pytest.mark.parametrize("n", [1, 2, 37])
def test_keys_and_values_read_back_into_one_array(n):
    # [n][2][Hkv][D]: rows of keys and of values by turns
    dev = cuda()
    c = Case([300], 0, 2, 2, 128, "fp16", seed=2)
    both = torch.full((n, 2, 2, 128), 9.0, dtype=torch.float16, device=dev)
    args = (c.dev(c.tables), c.dev([200]), c.dev([0, n]), n)
    k, v = c.pool.gather(*args)
    c.pool.gather(*args, k_out=both[:, 0], v_out=both[:, 1])
    assert torch.equal(both[:, 0], k) and torch.equal(both[:, 1], v)
    with pytest.raises(q4.Q4KVError):
        c.pool.gather(*args, k_out=k, v_out=k)


@pytest.mark.parametrize("d,hq,inter", [(128, 7, False), (128, 40, True), (256, 3, False), (256, 16, True)])
@pytest.mark.parametrize("T", [3, 900])
def test_queries_rotated_in_place_inside_a_fused_row(d, hq, inter, T):
    # q, k and v as slices of one row per token; the last group of heads is not full
    dev = cuda()
    g = torch.Generator(device=dev).manual_seed(T)
    qkv = torch.randn(2, T, hq + 4, d, generator=g, device=dev).to(torch.bfloat16)
    ro = q4.Rotary(q4.Rotary.make_table(10000.0 ** (-torch.arange(d // 2) / (d // 2)), T + 50, device=dev), interleaved=inter)
    tab = torch.arange(10, device=dev).view(2, 5)
    lens, n_new = torch.tensor([7, 40], device=dev), torch.tensor([T, T - 2], device=dev)

    def run(x, in_place):
        pool = q4.Q4KVPool(2, d, 10, device=dev)
        q = x[:, :, :hq]
        o = pool.append_rotary(x[:, :, hq:hq + 2], x[:, :, hq + 2:], ro, tab, lens, n_new, q=q, q_out=q if in_place else None)
        assert pool.read_device_error() == 0
        return o, pool

    want, a = run(qkv.clone(), False)
    for _ in range(3):
        x = qkv.clone()
        got, b = run(x, True)
        assert got.data_ptr() == x.data_ptr() and torch.equal(got, want)
        assert torch.equal(x[:, :, hq:], qkv[:, :, hq:])
        assert all(torch.equal(getattr(a, n), getattr(b, n)) for n in ("k_codes4", "k_params4", "v_codes4", "v_params4"))


@pytest.mark.parametrize("width", [4, 8, 2])
@pytest.mark.parametrize("T,d", [(6, 128), (150, 128), (30, 128), (20, 256)])
def test_the_largest_finite_keys(T, d, width):
    # a group of raw keys from -65504 to 65504: its rounded scale may end past fp16
    dev = cuda()
    scale = 1e-6
    c = Case([40], T, 4, 2, d, "fp16", widths=(width,), seed=T, rotated=False)
    k, v = W.random_small(40 + T, 2, d, "fp16", seed=T, scale=1.0)
    k[::3, :, 5], k[::3, :, 9] = 65504.0, -65504.0
    ids = c.tables[0][:1].tolist()
    c.pool.quantize(k.to(dev), v.to(dev), torch.tensor(ids, dtype=torch.int32, device=dev))
    c.ref.quantize_blocks(host(k)[0], host(v)[0], "fp16", ids)
    want, bound = c.want(scale=scale)
    # One step less of the scale moves a key by at most 2^-10 of the group's range,
    # so a logit by x = scale |q|_1 128 and each weight by a factor of e^(+-2x); the
    # output, a mean of values within V, then moves by at most (e^2x - 1) 2 V.
    x = scale * float(c.q.float().abs().sum(-1).max()) * 2.0 ** -10 * 2 * 65504
    _attend_close(c.run(softmax_scale=scale), want, bound + np.expm1(2 * x) * 2 * float(v.float().abs().max()), rel=1.0)


@pytest.mark.parametrize("width,s", [(4, 10000.0), (8, 600.0), (2, 40000.0)])
@pytest.mark.parametrize("T,d", [(6, 128), (150, 128), (30, 128), (20, 256)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_one_key_channel_past_fp16(T, d, width, s, sign):
    # the logits of that token are +Inf or -Inf by the query's sign; the rows that see it are NaN either way
    c = Case([100], T, 4, 2, d, "fp16", widths=(width,), seed=T, rotated=False)
    c.q[..., 8:] = 0.0
    c.q[..., :8] = sign
    clean = c.run()
    t = 100 + T // 2
    blk, slot = int(c.tables[0][0]), t
    codes, params = getattr(c.pool, f"k_codes{width}"), getattr(c.pool, f"k_params{width}")
    codes[blk, 1, slot] = 0
    codes[blk, 1, slot, 0] = (1 << width) - 1      # channel 0 alone
    params[blk, 1, slot, 0, 0], params[blk, 1, slot, 0, 1] = s, 0.0
    got = c.run()
    hit = torch.zeros(1, T, 4, dtype=torch.bool, device=got.device)
    hit[0, T // 2:, 2:] = True
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("T,d", [(6, 128), (150, 128), (30, 128), (20, 256)])
@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_queries_that_are_not_finite_make_their_own_rows_nan(T, d, rotated, bad):
    c = Case([100], T, 4, 2, d, "bf16", seed=T, rotated=rotated)
    c.pool.k_params4[:, :, :, 0, 0] = 0.0          # keys of channel 3's group are positive: with raw keys
    c.pool.k_params4[:, :, :, 0, 1] = 1.0          # every logit has the sign of that channel's query
    clean = c.run()
    c.q[0, T // 2, 1, 3] = bad
    got = c.run()
    hit = torch.zeros(1, T, 4, dtype=torch.bool, device=got.device)
    hit[0, T // 2, 1] = True
    assert bool(torch.isnan(got[hit]).all()) and torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("T,d", [(6, 128), (150, 128), (30, 128), (20, 256)])
@pytest.mark.parametrize("power", [16, 30, 100, 116])
def test_logits_far_below_zero(T, d, power):
    # every key is a constant, every query -2^power: the least key takes all the weight
    dev = cuda()
    c = Case([100], T, 4, 2, d, "bf16", seed=T, rotated=False)
    k, v = W.random_small(100 + T, 2, d, "bf16", seed=T, scale=1.0)
    # whole and half numbers, exact in a group's zero, falling towards the end
    k[:] = (torch.arange(100 + T, 0, -1) / 2.0 + 10.0).view(-1, 1, 1).to(k.dtype)
    ids = c.tables[0][:1].tolist()
    c.pool.quantize(k.to(dev), v.to(dev), torch.tensor(ids, dtype=torch.int32, device=dev))
    c.ref.quantize_blocks(host(k)[0], host(v)[0], "bf16", ids)
    c.q[:] = -2.0 ** power
    want, _ = c.want(scale=2.0 ** -3)
    got = c.run(softmax_scale=2.0 ** -3).cpu().numpy()
    # the values' rounding to fp16 (weights of 1 are exact)
    assert np.all(np.abs(got - want) <= 2.0 ** -11 * np.abs(want) + 2.0 ** -25)


@pytest.mark.parametrize("T,d", [(6, 128), (150, 128), (20, 256)])
@pytest.mark.parametrize("mag,scale", [(2.0 ** -118, 2.0 ** 114.5), (2.0 ** 120, 2.0 ** -123.5), (2.0 ** -110, 1e-20), (1.0, 1e-38)])
def test_the_ends_of_queries_and_scales(T, d, mag, scale):
    # products of scale and query of ordinary size, and next to nothing (the mean of what is live)
    c = Case([100], T, 4, 2, d, "bf16", seed=T, evict=[(0, t) for t in range(0, 100, 7)])
    c.q = (c.q.float() * mag).to(torch.bfloat16)
    want, bound = c.want(scale=scale)
    _attend_close(c.run(softmax_scale=scale), want, bound)


def test_a_workspace_that_is_not_one_piece_is_refused():
    # a byte expanded to the size asked for passes for that many bytes
    dev = cuda()
    c = Case([600], 20, 8, 2, 128, "fp16", seed=1)
    plan = q4.ExtendPlan(1, 20, 8, 2, 128, c.tables.shape[1], n_splits=2)
    n = plan.workspace_bytes
    for ws in (torch.zeros(1, dtype=torch.uint8, device=dev).expand(n), torch.zeros(2 * n, dtype=torch.uint8, device=dev)[::2]):
        with pytest.raises(ValueError):
            c.run(plan=plan, workspace=ws)
    with pytest.raises(q4.Q4KVError):
        c.run(plan=plan, workspace=torch.zeros(n - 1, dtype=torch.uint8, device=dev))
    want, bound = c.want()
    _attend_close(c.run(plan=plan, workspace=torch.zeros(n // 4 + 1, dtype=torch.float32, device=dev)), want, bound)


@pytest.mark.parametrize("T", [1, 6])
def test_one_head_out_of_a_transposed_layout(T):
    # [B][H][T][D] transposed: with one head, rows are in one piece whatever that axis's stride is;
    # keys and values of one sequence or token may differ in the strides of those axes
    dev = cuda()
    g = torch.Generator(device=dev).manual_seed(T)
    q, k, v = (torch.randn(1, 1, T, 128, generator=g, device=dev).half() for _ in "qkv")
    v = torch.cat((v, v), 0)[:1] if T > 1 else torch.cat((v, v), 2)[:, :, :1]
    ro = q4.Rotary(q4.Rotary.make_table(10000.0 ** (-torch.arange(64) / 64), 60, device=dev))
    tab, lens = torch.tensor([[1, 0]], device=dev), torch.tensor([20], device=dev)
    outs = []
    for turn in (lambda x: x.transpose(1, 2), lambda x: x.transpose(1, 2).contiguous()):
        pool = q4.Q4KVPool(1, 128, 2, device=dev)
        qr = pool.append_rotary(turn(k), turn(v), ro, tab, lens, q=turn(q), q_out=turn(torch.empty_like(q)))
        o = q4.extend_attention(pool, qr, tab, lens, out=turn(torch.empty(1, 1, T, 128, device=dev)))
        kv = torch.empty(2, 1, T, 128, dtype=torch.float16, device=dev)
        kk, vv = pool.gather(tab, lens, torch.tensor([0, T], device=dev), T, k_out=kv[0].transpose(0, 1), v_out=kv[1].transpose(0, 1))
        assert pool.read_device_error() == 0 and torch.count_nonzero(vv) > 0
        outs.append((qr, o, kk.clone(), vv.clone(), pool.k_codes4, pool.v_codes4))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


@pytest.mark.parametrize("T,hq,hkv,d,splits", [(70, 8, 2, 128, 0), (20, 8, 2, 128, 3), (4, 8, 2, 128, 0), (33, 4, 2, 256, 2)])
def test_results_repeat_bit_for_bit_beside_other_work(T, hq, hkv, d, splits):
    dev = cuda()
    c = Case([1500, 2900, 40], T, hq, hkv, d, "bf16", n_new=[T, T - 1, T], widths=(4, 8), seed=T, kscale=6.0)
    args = (c.pool, c.q.to(dev), c.dev(c.tables), c.dev(c.lens), c.dev(c.n_new))
    plan = q4.ExtendPlan(3, T, hq, hkv, d, c.tables.shape[1], n_splits=splits)
    first = q4.extend_attention(*args, plan=plan, out_dtype=torch.float32)
    other, big = torch.cuda.Stream(), torch.zeros(1 << 26, device=dev)
    torch.cuda.synchronize()
    for i in range(40):
        if i % 3:
            with torch.cuda.stream(other):
                big.add_(1.0)
        assert torch.equal(q4.extend_attention(*args, plan=plan, out_dtype=torch.float32), first)
    torch.cuda.synchronize()


def test_a_padded_batch_of_prompts_sharing_their_first_blocks():
    # two sequences over the same prefix blocks, an empty one, and one without new tokens
    dev = cuda()
    c = Case([512, 512, 0, 300], 30, 8, 2, 128, "fp16", n_new=[30, 11, 0, 0], seed=7)
    c.tables[1][:2] = c.tables[0][:2]
    want, bound = c.want()
    out = torch.full((4, 30, 8, 128), 3.0, device=dev)
    _attend_close(c.run(out=out), want, bound)
    assert torch.count_nonzero(out[2:]) == 0 and torch.count_nonzero(out[1, 11:]) == 0
    k, v = c.pool.gather(c.dev(c.tables), c.dev([0, 0, 0, 0]), c.dev([0, 512, 1024, 1024, 1324]), 1324)
    assert torch.equal(k[:512], k[512:1024]) and torch.equal(v[:512], v[512:1024])
    assert c.pool.read_device_error() == 0
