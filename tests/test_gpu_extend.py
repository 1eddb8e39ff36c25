"""Extending a cached prompt on the GPU: rotary append, read-back and chunk
attention against the plain definitions (binary32 bit for bit, attention in 64
bits)."""
import numpy as np
import pytest
import torch

import decode_attention_q4kv_b200 as q4
from decode_attention_q4kv_b200 import _lib
from decode_attention_q4kv_b200 import workloads as W
from helpers import assert_pool_equal, cuda, host
from oracle import extend_oracle as E
from oracle import q4kv_oracle as O

pytestmark = pytest.mark.gpu

# Relative L2 error of the attention output in 32 bits.  Rounding to fp16 leaves
# a relative error of rms at most u = 2^-11 / sqrt(3) = 2.8e-4.  For N(0, 1)
# queries and keys a logit has unit variance, and rounding q and K moves it by
# sqrt(2) u, which moves the output by as much relative to its own size; the
# rounded weights and values add u each: sqrt(2 + 1 + 1) u = 5.7e-4.  Twice that.
REL = 1.2e-3


def _attend_close(got, want, bound, rel=REL, what=""):
    a = got.detach().float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(a)), f"{what}: non-finite output"
    eps = {torch.float32: 2.0 ** -20, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[got.dtype]
    err = np.abs(a - want)
    worst = float((err - bound - eps * np.abs(want) - 1e-6).max())
    assert worst <= 0, f"{what}: off by {worst:.2e} more than the roundings explain"
    norm = np.linalg.norm(want)
    off = np.linalg.norm(a - want) / norm if norm else np.linalg.norm(a - want)
    assert off <= rel + eps, f"{what}: relative L2 error {off:.2e}"


class Case:
    """A pool with every sequence's cached and new tokens in place, and its oracle."""

    def __init__(self, lens, T, hq, hkv, d, dtype="fp16", n_new=None, rotated=True, widths=(4,), fp8=False, seed=0,
                 kscale=1.0, evict=(), spare_blocks=1):
        dev = cuda()
        self.lens, self.T, self.hq, self.d, self.dtype, self.n_new = lens, T, hq, d, dtype, n_new
        B = len(lens)
        new = [T] * B if n_new is None else n_new
        mb = max(1, max(-(-(a + t) // 256) for a, t in zip(lens, new))) + spare_blocks
        n = B * mb + 2
        per = [n if w == widths[0] and len(widths) == 1 else -(-n // len(widths)) for w in widths]
        count = {w: c for w, c in zip(widths, per)}
        n4, n8, n2 = count.get(4, 0), count.get(8, 0), count.get(2, 0)
        if fp8:
            n4, n8, n2 = 0, n, 0
        total = n4 + n8 + n2
        rng = np.random.RandomState(seed + 77)
        self.tables = rng.permutation(total)[: B * mb].reshape(B, mb).astype(np.int32)
        rotated = rotated and not fp8
        self.pool = q4.Q4KVPool(hkv, d, n4, n8, k_rotated=rotated, device=dev, n_q2_blocks=n2, fp8=fp8)
        self.ref = O.OraclePool(hkv, d, n4, n8, k_rotated=rotated, n_q2=n2, fp8=fp8)
        for b in range(B):
            m = lens[b] + new[b]
            if m == 0:
                continue
            k, v = W.random_small(m, hkv, d, dtype, seed=seed + 10 * b, scale=1.0)
            k = (k.float() * kscale).to(k.dtype)
            ids = self.tables[b][: -(-m // 256)].tolist()
            self.pool.quantize(k.to(dev), v.to(dev), torch.tensor(ids, dtype=torch.int32, device=dev))
            kh, dt = host(k)
            vh, _ = host(v)
            self.ref.quantize_blocks(kh, vh, dt, ids)
        for b, t in evict:
            sid = int(self.tables[b][t // 256]) * 256 + t % 256
            self.pool.invalidate(torch.tensor([sid], device=dev))
            self.ref.invalidate_slots([sid])
        g = torch.Generator().manual_seed(seed + 5)
        self.q = torch.randn(B, T, hq, d, generator=g).to(W.torch_dtype(dtype))

    def dev(self, x):
        return None if x is None else torch.as_tensor(np.asarray(x), dtype=torch.int32).to(cuda())

    def run(self, q=None, **kw):
        q = self.q.to(cuda()) if q is None else q
        kw.setdefault("out_dtype", torch.float32)
        out = q4.extend_attention(self.pool, q, self.dev(self.tables), self.dev(self.lens), self.dev(self.n_new), **kw)
        torch.cuda.synchronize()
        return out

    def want(self, **kw):
        qh, dt = host(self.q)
        return E.extend_attention(self.ref, qh, dt, self.tables, self.lens, self.n_new, **kw)


SHAPES = [
    # lens, T, Hq, Hkv, D, dtype
    ([0], 1, 8, 8, 128, "fp16"),
    ([255, 0, 256, 700], 1, 8, 2, 128, "bf16"),
    ([0, 1, 300], 5, 12, 3, 128, "fp16"),
    ([130, 511], 33, 20, 4, 128, "fp16"),
    ([64, 1000], 65, 16, 8, 256, "bf16"),
    ([257], 129, 8, 1, 256, "fp16"),
    ([0], 300, 4, 4, 128, "bf16"),
    ([513], 257, 16, 2, 128, "fp16"),
]


@pytest.mark.parametrize("lens,T,hq,hkv,d,dtype", SHAPES)
def test_chunk_attention(lens, T, hq, hkv, d, dtype):
    c = Case(lens, T, hq, hkv, d, dtype, seed=T)
    want, bound = c.want()
    _attend_close(c.run(), want, bound)
    assert c.pool.read_device_error() == 0


@pytest.mark.parametrize("widths,fp8,rotated", [((4,), False, False), ((8,), False, True), ((2,), False, True),
                                                ((4, 8), False, True), ((4, 8, 2), False, True), ((4,), True, False)])
@pytest.mark.parametrize("d", [128, 256])
def test_chunk_attention_block_classes(widths, fp8, rotated, d):
    c = Case([300, 801], 40, 8, 4, d, "fp16", n_new=[40, 17], widths=widths, fp8=fp8, rotated=rotated, seed=d)
    want, bound = c.want()
    _attend_close(c.run(), want, bound, what=f"{widths} fp8={fp8}")
    assert c.pool.read_device_error() == 0


@pytest.mark.parametrize("window", [1, 7, 128, 256, 300, 5000])
@pytest.mark.parametrize("d", [128, 256])
def test_window(window, d):
    c = Case([600, 0, 255], 70, 4, 2, d, "fp16", n_new=[70, 70, 3], seed=window)
    want, bound = c.want(window=window)
    _attend_close(c.run(window=window), want, bound, what=f"window {window}")


@pytest.mark.parametrize("d", [128, 256])
def test_remapped_slots_and_rows_that_see_nothing_live(d):
    # sequence 0: scattered slots gone; sequence 1: every slot gone (rows are 0);
    # sequence 2: everything but the newest tokens gone; sequence 3: the prefix
    # and the first new tokens gone, so the first rows see nothing live
    lens, T = [400, 300, 270, 256], 9
    evict = [(0, t) for t in range(0, 409, 3)] + [(1, t) for t in range(309)] + [(2, t) for t in range(270)] + \
            [(3, t) for t in range(260)]
    c = Case(lens, T, 8, 2, d, "fp16", evict=evict, seed=3)
    want, bound = c.want()
    out = c.run()
    assert torch.count_nonzero(out[1]) == 0 and torch.count_nonzero(out[3, :4]) == 0
    assert np.count_nonzero(want[1]) == 0 and np.abs(want[3, 4]).min() > 0
    _attend_close(out, want, bound)


@pytest.mark.parametrize("T,hq,hkv", [(8, 8, 2), (33, 2, 2), (32, 2, 2), (2, 20, 2), (1, 8, 2)])
@pytest.mark.parametrize("widths,fp8", [((4, 8, 2), False), ((4,), True)])
@pytest.mark.parametrize("window", [0, 1, 13, 300])
def test_few_rows(T, hq, hkv, widths, fp8, window):
    # up to 32 rows of a group share a tile's columns out among copies; 33 do not
    lens = [517, 3, 64]
    evict = [(0, t) for t in range(0, 517, 5)] + [(0, t) for t in range(384, 400)] + [(2, t) for t in range(64)]
    c = Case(lens, T, hq, hkv, 128, "fp16", widths=widths, fp8=fp8, n_new=[T, T, max(1, T - 2)], evict=evict, seed=T)
    want, bound = c.want(window=window)
    for s in (1, 0, 2):
        plan = q4.ExtendPlan(3, T, hq, hkv, 128, c.tables.shape[1], window=window, n_splits=s)
        _attend_close(c.run(window=window, plan=plan), want, bound, what=f"splits {s}")
    assert c.pool.read_device_error() == 0


@pytest.mark.parametrize("d", [128, 256])
def test_garbage_behind_the_mask_and_the_end_stays_out(d):
    # NaN scales in remapped slots, in slots past the end and in blocks past the
    # end; block ids past the end of the sequence are not even valid
    dev = cuda()
    c = Case([290, 20], 6, 8, 2, d, "fp16", evict=[(0, 5), (0, 200), (1, 3)], seed=9)
    want, bound = c.want()
    nan = float("nan")
    for b, n in enumerate([296, 26]):
        for t in ([5, 200] if b == 0 else [3]) + list(range(n, -(-n // 256) * 256)):
            blk, slot = int(c.tables[b][t // 256]), t % 256
            for name in ("k_params4", "v_params4"):
                getattr(c.pool, name)[blk, :, slot] = nan
    for b, n in enumerate([296, 26]):
        c.tables[b][-(-n // 256):] = -1
    out = c.run()
    _attend_close(out, want, bound)
    assert c.pool.read_device_error() == 0
    assert out.device == dev


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("width,fp8", [(4, False), (8, False), (2, False), (8, True)])
@pytest.mark.parametrize("T,d,window,splits", [(5, 128, 0, 0), (40, 128, 50, 3), (300, 128, 0, 1), (70, 256, 0, 2), (70, 256, 33, 1)])
def test_tokens_that_are_not_finite_reach_only_the_rows_that_see_them(which, width, fp8, T, d, window, splits):
    # one token in the cached part, one among the new ones, one of the other
    # sequence remapped: rows that do not see them keep every bit
    c = Case([200, 131], T, 4, 2, d, "fp16", widths=(width,), fp8=fp8, rotated=not fp8, seed=T, evict=[(1, 60)])
    plan = q4.ExtendPlan(2, T, 4, 2, d, c.tables.shape[1], window=window, n_splits=splits)
    clean = c.run(plan=plan, window=window)
    odd = {0: [170, 200 + T // 2], 1: [60]}
    for b, tokens in odd.items():
        for t in tokens:
            blk, slot = int(c.tables[b][t // 256]), t % 256
            if fp8:
                getattr(c.pool, f"{which}_codes8")[blk, 1, slot, 77] = 0x7F
            else:
                getattr(c.pool, f"{which}_params{width}")[blk, 1, slot, 0, slot % 2] = float("inf" if slot % 3 else "nan")
    got = c.run(plan=plan, window=window)
    sees = torch.zeros(2, T, 4, dtype=torch.bool)
    for i in range(T):
        sees[0, i, 2:] = any(t <= 200 + i and (window == 0 or t > 200 + i - window) for t in odd[0])
    assert bool(sees.any()) and not bool(sees.all())
    sees = sees.to(got.device)
    assert bool(torch.isnan(got[sees]).all())
    assert torch.equal(got[~sees], clean[~sees])


@pytest.mark.parametrize("width", [4, 8, 2])
@pytest.mark.parametrize("T,d", [(6, 128), (150, 128), (20, 256)])
def test_the_largest_finite_values(T, d, width):
    # a group from -65504 to 65504: its rounded scale may end past fp16
    dev = cuda()
    lens = [40]
    c = Case(lens, T, 4, 2, d, "fp16", widths=(width,), seed=T, rotated=False)
    m = lens[0] + T
    k, v = W.random_small(m, 2, d, "fp16", seed=T, scale=1.0)
    v[::3, :, 5], v[::3, :, 9] = 65504.0, -65504.0
    ids = c.tables[0][:1].tolist()
    c.pool.quantize(k.to(dev), v.to(dev), torch.tensor(ids, dtype=torch.int32, device=dev))
    c.ref.quantize_blocks(host(k)[0], host(v)[0], "fp16", ids)
    want, bound = c.want()
    # One step less of the scale moves a value by at most 2^-10 of the group's
    # range, 128.  Only the bound per element is asked for: REL supposes values of
    # the output's size, and here values of 65504 cancel to outputs of 1800, which
    # 128 exceeds by 2^-4 of their size.
    _attend_close(c.run(), want, bound + 2.0 ** -10 * 2 * 65504, rel=2.0 ** -3)


@pytest.mark.parametrize("T,d", [(3, 128), (40, 256), (200, 128)])
def test_split_counts_agree(T, d):
    c = Case([1500, 3, 900], T, 8, 2, d, "fp16", n_new=[T, T - 1, 0], seed=T)
    want, bound = c.want()
    mb = c.tables.shape[1]
    for s in (0, 1, 2, 3, mb):
        plan = q4.ExtendPlan(3, T, 8, 2, d, mb, n_splits=s)
        out = c.run(plan=plan)
        _attend_close(out, want, bound, what=f"splits {s} -> {plan.n_splits}")
        assert torch.count_nonzero(out[2]) == 0 and torch.count_nonzero(out[1, T - 1:]) == 0


def test_rows_past_n_new_are_zero_and_neighbours_stay():
    dev = cuda()
    c = Case([100, 40, 0], 7, 8, 2, 128, "bf16", n_new=[0, 7, 2], seed=1)
    want, bound = c.want()
    big = torch.full((5, 9, 8 * 128 + 64), 7.0, dtype=torch.bfloat16, device=dev)
    out = big[1:4, 1:8, : 8 * 128].unflatten(-1, (8, 128))
    got = c.run(out=out)
    assert got.data_ptr() == out.data_ptr()
    _attend_close(got, want, bound)
    assert torch.count_nonzero(got[0]) == 0 and torch.count_nonzero(got[2, 2:]) == 0
    big[1:4, 1:8, : 8 * 128] = 7.0
    assert bool((big == 7.0).all())


def test_strided_queries_and_scale():
    dev = cuda()
    c = Case([77, 300], 10, 6, 2, 128, "fp16", seed=4)
    wide = torch.zeros(2, 10, 10, 128, dtype=torch.float16, device=dev)
    wide[:, :, 1:7] = c.q.to(dev)
    want, bound = c.want(scale=0.03)
    _attend_close(c.run(q=wide[:, :, 1:7], softmax_scale=0.03), want, bound)


def test_large_and_small_queries():
    # magnitudes near the ends of bf16's range that fp16 cannot hold
    c = Case([200], 20, 8, 2, 128, "bf16", seed=6)
    q0 = c.q.clone()
    for mag, scale in ((2.0 ** 60, 2.0 ** -63.5), (2.0 ** -60, 2.0 ** 56.5)):
        c.q = (q0.float() * mag).to(torch.bfloat16)
        want, bound = c.want(scale=scale)
        _attend_close(c.run(softmax_scale=scale), want, bound, what=f"queries x {mag}")


def test_sharp_softmax():
    # keys x 12: one key takes nearly all the weight; logits reach some hundreds,
    # and the rounding of a logit grows with it, so only the bound is checked
    c = Case([700], 30, 8, 2, 128, "fp16", seed=8, kscale=12.0)
    want, bound = c.want()
    _attend_close(c.run(), want, bound, rel=1.0)


@pytest.mark.parametrize("T", [1, 4])
def test_bad_lengths_and_blocks_zero_the_rows_and_raise(T):
    c = Case([300, 310, 290], T, 8, 2, 128, "fp16", seed=2)
    want, bound = c.want()
    mb = c.tables.shape[1]
    good = c.lens
    c.lens = [300, mb * 256 - T + 1, -1]
    out = c.run()
    assert c.pool.read_device_error() & _lib.DEVERR_SEQ_LEN
    assert torch.count_nonzero(out[1:]) == 0
    _attend_close(out[:1], want[:1], bound[:1])
    c.lens = good
    c.tables[1][1] = 10 ** 6
    out = c.run()
    assert c.pool.read_device_error() & _lib.DEVERR_BLOCK_ID
    assert torch.count_nonzero(out[1]) == 0
    _attend_close(out[0], want[0], bound[0])
    _attend_close(out[2], want[2], bound[2])


@pytest.mark.parametrize("widths,fp8,d", [((4,), False, 128), ((4, 8, 2), False, 256), ((4,), True, 128)])
def test_one_token_equals_decode_and_general_path(widths, fp8, d):
    # without counts one token takes the decode kernel, with counts the chunk kernel
    c = Case([900, 17, 256], 1, 8, 2, d, "fp16", seed=12, widths=widths, fp8=fp8)
    lens = c.dev([n + 1 for n in c.lens])
    b = q4.decode_attention(c.pool, c.q.to(cuda())[:, 0].contiguous(), c.dev(c.tables), lens, out_dtype=torch.float32)
    want, bound = c.want()
    a = c.run()
    assert torch.equal(a[:, 0], b)
    _attend_close(a, want, bound)
    c.n_new = [1, 1, 1]
    _attend_close(c.run(), want, bound)
    c.n_new = [1, 0, 1]
    out = c.run()
    assert torch.count_nonzero(out[1]) == 0
    _attend_close(out[0::2], want[0::2], bound[0::2])
    assert c.pool.read_device_error() == 0
    for bad in (-2, 5000):
        c.n_new, c.lens = None, [900, bad, 256]
        out = c.run()
        assert torch.count_nonzero(out[1]) == 0 and c.pool.read_device_error() & _lib.DEVERR_SEQ_LEN


def test_capture_replay_streams_and_repeats():
    dev = cuda()
    c = Case([500, 1200], 12, 8, 2, 128, "fp16", seed=21)
    want, bound = c.want()
    q, tab, lens = c.q.to(dev), c.dev(c.tables), c.dev(c.lens)
    plan = q4.ExtendPlan(2, 12, 8, 2, 128, tab.shape[1], n_splits=2)
    ws = plan.workspace(dev)
    out = torch.zeros(2, 12, 8, 128, device=dev)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        q4.extend_attention(c.pool, q, tab, lens, plan=plan, workspace=ws, out=out)
    s.synchronize()
    first = out.clone()
    _attend_close(first, want, bound)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q4.extend_attention(c.pool, q, tab, lens, plan=plan, workspace=ws, out=out)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)           # no atomics: bit for bit


def test_tables_of_any_alignment_and_two_streams_at_once():
    # a slice of a wider table starts at any int32; two calls with their own
    # scratch run beside each other
    dev = cuda()
    cases = [Case([500, 900, 33], T, 8, 2, 128, "fp16", seed=T) for T in (1, 20)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    args, outs = [], [None, None]
    for c in cases:
        mb = c.tables.shape[1]
        wide = torch.full((3 * mb + 1,), -7, dtype=torch.int32, device=dev)
        wide[1:] = c.dev(c.tables).flatten()
        args.append((c.pool, c.q.to(dev), wide[1:].view(3, mb), c.dev(c.lens)))
    torch.cuda.synchronize()
    for _ in range(5):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                outs[i] = q4.extend_attention(*args[i], out_dtype=torch.float32)
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        want, bound = c.want()
        _attend_close(o, want, bound)


def test_empty_calls():
    dev = cuda()
    c = Case([10], 3, 8, 2, 128, "fp16")
    out = q4.extend_attention(c.pool, c.q.to(dev)[:, :0], c.dev(c.tables), c.dev(c.lens))
    assert out.shape == (1, 0, 8, 128)
    out = q4.extend_attention(c.pool, c.q.to(dev)[:0], c.dev(c.tables)[:0], c.dev(c.lens)[:0])
    assert out.shape == (0, 3, 8, 128)
    assert torch.count_nonzero(c.run(out_dtype=torch.float16)) > 0


@pytest.mark.parametrize("bad", ["dtype", "heads", "plan", "device", "out", "lens", "counts"])
def test_attention_arguments_are_checked(bad):
    dev = cuda()
    c = Case([10], 3, 8, 2, 128, "fp16")
    q, tab, lens = c.q.to(dev), c.dev(c.tables), c.dev(c.lens)
    kw = {}
    if bad == "dtype":
        q = q.float()
    elif bad == "heads":
        q = torch.zeros(1, 3, 9, 128, dtype=torch.float16, device=dev)
    elif bad == "plan":
        kw["plan"] = q4.ExtendPlan(1, 4, 8, 2, 128, tab.shape[1])
    elif bad == "device":
        lens = lens.cpu()
    elif bad == "out":
        kw["out"] = torch.zeros(1, 3, 8, 64, device=dev)
    elif bad == "lens":
        lens = torch.zeros(2, dtype=torch.int32, device=dev)
    else:
        kw["n_new"] = torch.zeros(3, dtype=torch.int32, device=dev)
    with pytest.raises((ValueError, q4.Q4KVError)):
        q4.extend_attention(c.pool, q, tab, lens, **kw)


def test_heads_of_another_size_and_rows_on_top_of_one_another_are_refused():
    dev = cuda()
    c = Case([10, 20], 3, 8, 2, 128, "fp16")
    tab, lens = c.dev(c.tables), c.dev(c.lens)
    plan = q4.ExtendPlan(2, 3, 8, 2, 128, tab.shape[1])
    for d in (64, 256):
        q = torch.zeros(2, 3, 32, d, dtype=torch.float16, device=dev)[:, :, :8]   # rows far enough apart for heads of 128
        with pytest.raises(ValueError):
            q4.extend_attention(c.pool, q, tab, lens, plan=plan)
    one = torch.zeros(1, 3, 8, 128, dtype=torch.float16, device=dev)
    with pytest.raises(q4.Q4KVError):
        q4.extend_attention(c.pool, c.q.to(dev), tab, lens, plan=plan, out=one.expand(2, 3, 8, 128))
    same = c.run(q=c.q[:1].to(dev).expand(2, 3, 8, 128))                             # queries may be shared
    c.q = c.q[:1].expand(2, 3, 8, 128).contiguous()
    assert torch.equal(same, c.run())


# -- rotary append -------------------------------------------------------------

def _table(pairs, n, seed=0):
    inv = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    return q4.Rotary.make_table(inv, n, device="cpu")


def _append_case(lens, T, hq, hkv, d, dtype, rot, axes, inter, given, n_new=None, rotated=True, widths=(4, 0, 0),
                 fp8=False, seed=0, strided=False):
    dev = cuda()
    B = len(lens)
    mb = max(-(-(n + T) // 256) for n in lens)
    n = B * mb
    n4, n8, n2 = (w * n for w in widths) if not fp8 else (0, n, 0)
    n4 = n4 // 4
    pool = q4.Q4KVPool(hkv, d, n4, n8, k_rotated=rotated and not fp8, device=dev, n_q2_blocks=n2, fp8=fp8)
    ref = O.OraclePool(hkv, d, n4, n8, k_rotated=rotated and not fp8, n_q2=n2, fp8=fp8)
    total = n4 + n8 + n2
    tables = np.random.RandomState(seed).permutation(total)[:n].reshape(B, mb).astype(np.int32)
    sids = [int(tables[b][p // 256]) * 256 + p % 256 for b in range(B) for p in range(lens[b], lens[b] + T, 2)]
    pool.invalidate(torch.tensor(sids, device=dev))     # writing a slot makes it live again
    ref.invalidate_slots(sids)
    dt = W.torch_dtype(dtype)
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(B, T, hq + 2 * hkv, d, generator=g).to(dt)
    if not strided:
        q, k, v = (x.contiguous() for x in (qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]))
        dq, dk, dv = q.to(dev), k.to(dev), v.to(dev)
    else:
        q, k, v = qkv[:, :, :hq], qkv[:, :, hq:hq + hkv], qkv[:, :, hq + hkv:]
        dall = qkv.to(dev)
        dq, dk, dv = dall[:, :, :hq], dall[:, :, hq:hq + hkv], dall[:, :, hq + hkv:]
    half, P = rot // 2, max(lens) + T + 5
    table = _table(half, P)
    axis = [(f * axes) // half if axes < 4 else f % axes for f in range(half)]
    if given:
        pos = torch.randint(0, P, (axes, B, T), generator=g, dtype=torch.int32)
        posn = pos.numpy()
    else:
        pos = None
        posn = np.broadcast_to(np.asarray(lens)[:, None] + np.arange(T), (axes, B, T))
    ro = q4.Rotary(table.to(dev), axis_of_pair=axis, interleaved=inter, n_axes=axes)
    nn = None if n_new is None else torch.tensor(n_new, dtype=torch.int32, device=dev)
    got = pool.append_rotary(dk, dv, ro, torch.as_tensor(tables).to(dev), torch.tensor(lens, dtype=torch.int32, device=dev),
                             nn, None if pos is None else pos.to(dev), q=dq)
    torch.cuda.synchronize()
    (qh, name), (kh, _), (vh, _) = host(q.contiguous()), host(k.contiguous()), host(v.contiguous())
    tb = table.numpy()
    wq = E.rotary(qh, name, tb, posn, axis, inter)
    wk = E.rotary(kh, name, tb, posn, axis, inter)
    ref.append_tokens(wk, vh, name, tables, lens, n_new)
    if n_new is not None:
        for b, t in enumerate(n_new):
            wq[b, t:] = 0
    return pool, ref, got, wq, name


@pytest.mark.parametrize("d,hq,hkv,rot,axes,inter,given", [
    (128, 8, 2, 128, 1, False, False), (128, 5, 5, 64, 1, True, False), (128, 9, 3, 96, 3, False, True),
    (128, 40, 8, 128, 3, True, True), (256, 4, 1, 256, 1, False, True), (256, 6, 2, 128, 4, True, True),
    (256, 3, 3, 32, 2, False, False), (256, 16, 8, 224, 4, False, True)])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_rotary_bit_exact(d, hq, hkv, rot, axes, inter, given, dtype):
    lens = [0, 100, 255, 510]
    pool, ref, got, wq, name = _append_case(lens, 5, hq, hkv, d, dtype, rot, axes, inter, given, n_new=[5, 0, 3, 4],
                                            seed=d + rot + axes, strided=axes > 1)
    assert pool.read_device_error() == 0
    assert_pool_equal(pool, ref)
    np.testing.assert_array_equal(host(got)[0].view(np.uint16), wq.view(np.uint16))


@pytest.mark.parametrize("widths,fp8,rotated", [((4, 0, 0), False, False), ((0, 1, 0), False, True), ((0, 0, 1), False, True),
                                                ((4, 1, 1), False, True), ((4, 0, 0), True, False)])
def test_append_rotary_block_classes(widths, fp8, rotated):
    pool, ref, got, wq, _ = _append_case([250, 3], 20, 4, 2, 128, "fp16", 128, 1, False, False, widths=widths, fp8=fp8,
                                         rotated=rotated, seed=5)
    assert pool.read_device_error() == 0
    assert_pool_equal(pool, ref)
    np.testing.assert_array_equal(host(got)[0].view(np.uint16), wq.view(np.uint16))


def test_append_rotary_large_chunk():
    pool, ref, got, wq, _ = _append_case([37], 700, 8, 4, 128, "bf16", 128, 1, False, False, seed=8)
    assert_pool_equal(pool, ref)
    np.testing.assert_array_equal(host(got)[0].view(np.uint16), wq.view(np.uint16))


def test_append_rotary_in_place_and_without_queries():
    dev = cuda()
    outs = []
    for mode in ("new", "same", "none"):
        torch.manual_seed(3)
        pool = q4.Q4KVPool(2, 128, 2, device=dev)
        k, v, q = (torch.randn(1, 6, h, 128, device=dev).half() for h in (2, 2, 4))
        ro = q4.Rotary(_table(64, 64).to(dev))
        tab, lens = torch.tensor([[1, 0]], device=dev), torch.tensor([10], device=dev)
        if mode == "none":
            assert pool.append_rotary(k, v, ro, tab, lens) is None
            o = None
        else:
            o = pool.append_rotary(k, v, ro, tab, lens, q=q, q_out=q if mode == "same" else None)
        outs.append((o, pool.k_codes4.clone(), pool.v_codes4.clone(), pool.k_params4.clone()))
    assert torch.equal(outs[0][0], outs[1][0])
    for x in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0][1:], x[1:]))


@pytest.mark.parametrize("bad", ["heads", "shape", "positions", "q", "q_out", "axis", "table"])
def test_append_rotary_arguments_are_checked(bad):
    dev = cuda()
    pool = q4.Q4KVPool(2, 128, 2, device=dev)
    k, v, q = (torch.zeros(1, 2, h, 128, device=dev).half() for h in (2, 2, 4))
    tab, lens = torch.tensor([[1, 0]], device=dev), torch.tensor([3], device=dev)
    table = _table(64, 64).to(dev)
    kw = {"q": q}
    with pytest.raises((ValueError, q4.Q4KVError)):
        if bad == "heads":
            k = v = torch.zeros(1, 2, 3, 128, device=dev).half()
        elif bad == "shape":
            v = v[:, :1]
        elif bad == "positions":
            kw["positions"] = torch.zeros(2, 1, 2, dtype=torch.int32, device=dev)
        elif bad == "q":
            kw["q"] = q.bfloat16()
        elif bad == "q_out":
            kw = {"q_out": q}
        elif bad == "axis":
            q4.Rotary(table, axis_of_pair=[0] * 63 + [4])
        else:
            table = table[:, :24].contiguous()
        pool.append_rotary(k, v, q4.Rotary(table), tab, lens, **kw)


def test_pool_over_the_callers_arrays():
    dev = cuda()
    a = q4.Q4KVPool(2, 128, 3, 2, device=dev)
    k, v = W.random_small(600, 2, 128, "fp16", seed=4)
    a.quantize(k.to(dev), v.to(dev), torch.tensor([4, 1, 2], dtype=torch.int32, device=dev))
    names = [f"{x}_{p}{w}" for x in "kv" for p in ("codes", "params") for w in "48"]
    b = q4.Q4KVPool.from_tensors(2, 128, a.mask, **{n: getattr(a, n) for n in names})
    assert (b.n_q4_blocks, b.n_q8_blocks, b.n_q2_blocks, b.n_blocks) == (3, 2, 0, 5) and b.nbytes() == a.nbytes()
    ids = torch.tensor([4, 1, 2], dtype=torch.int32, device=dev)
    assert all(torch.equal(x, y) for x, y in zip(a.dequantize(ids), b.dequantize(ids)))
    b.append(k[:1, None].to(dev), v[:1, None].to(dev), ids[1:2, None].contiguous(), torch.zeros(1, dtype=torch.int32, device=dev))
    assert torch.equal(a.k_codes4, b.k_codes4) and a.k_codes4.data_ptr() == b.k_codes4.data_ptr()
    good = {n: getattr(a, n) for n in names}
    for n, t in (("k_codes4", a.k_codes4[:, :, :, :32]), ("v_params8", a.v_params8.float()), ("v_codes8", a.v_codes8[:1])):
        with pytest.raises(ValueError):
            q4.Q4KVPool.from_tensors(2, 128, a.mask, **{**good, n: t})
    with pytest.raises(ValueError):
        q4.Q4KVPool.from_tensors(2, 128, a.mask[:4], **good)
    with pytest.raises(ValueError):
        q4.Q4KVPool.from_tensors(2, 128, a.mask, k_codes16=a.k_codes8, **good)


def test_append_rotary_faults_skip_the_token():
    dev = cuda()
    pool = q4.Q4KVPool(2, 128, 2, device=dev)
    before = pool.k_codes4.clone(), pool.mask.clone()
    k, v, q = (torch.randn(1, 2, h, 128, device=dev).half() for h in (2, 2, 4))
    ro = q4.Rotary(_table(64, 64).to(dev))
    tab = torch.tensor([[1]], dtype=torch.int32, device=dev)

    def call(length, positions, table, bit):
        o = pool.append_rotary(k, v, ro, table, torch.tensor([length], dtype=torch.int32, device=dev), positions=positions, q=q)
        assert pool.read_device_error() & bit
        assert torch.count_nonzero(o) == 0
        assert torch.equal(pool.k_codes4, before[0]) and torch.equal(pool.mask, before[1])

    for bad in (-1, 64):
        call(3, torch.full((1, 1, 2), bad, dtype=torch.int32, device=dev), tab, _lib.DEVERR_POSITION)
    call(64, None, tab, _lib.DEVERR_POSITION)
    ok = torch.zeros((1, 1, 2), dtype=torch.int32, device=dev)
    call(256, ok, tab, _lib.DEVERR_SEQ_LEN)
    call(-1, ok, tab, _lib.DEVERR_SEQ_LEN)
    call(0, ok, torch.tensor([[2]], dtype=torch.int32, device=dev), _lib.DEVERR_BLOCK_ID)


# -- read-back -----------------------------------------------------------------

@pytest.mark.parametrize("d,hkv,widths,fp8,unrotate", [(128, 8, (4,), False, True), (128, 3, (4, 8, 2), False, False),
                                                       (256, 2, (8,), False, True), (256, 5, (4,), False, True),
                                                       (128, 1, (2,), False, True), (256, 2, (4,), True, False)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
def test_gather_bit_exact(d, hkv, widths, fp8, unrotate, dtype):
    dev = cuda()
    c = Case([600, 3, 300, 256], 0, hkv, hkv, d, "fp16", widths=widths, fp8=fp8, seed=d, evict=[(0, 7), (0, 300), (2, 299)])
    starts, counts = [1, 0, 250, 255], [500, 0, 50, 1]
    off = np.concatenate([[0], np.cumsum(counts)]) + 2
    rows = int(off[-1]) + 3
    wide = [torch.full((rows, hkv * d + 8), 5.0, dtype=dtype, device=dev) for _ in "kv"]
    outs = [w[:, : hkv * d].unflatten(1, (hkv, d)) for w in wide]
    c.pool.gather(c.dev(c.tables), c.dev(starts), c.dev(off), rows, out_dtype=dtype, unrotate_k=unrotate, k_out=outs[0],
                  v_out=outs[1])
    assert c.pool.read_device_error() == 0
    want = E.gather(c.ref, c.tables, starts, counts, unrotate)
    for o, w, x in zip(outs, want, wide):
        t = torch.from_numpy(w).to(dtype)
        assert torch.equal(o[2: rows - 3].cpu(), t)
        x[2: rows - 3, : hkv * d] = 5.0
        assert bool((x == 5.0).all())            # rows of no sequence and the gaps between rows


def test_gather_remapped_and_faults():
    dev = cuda()
    c = Case([300], 0, 2, 2, 128, "fp16", seed=2, evict=[(0, 11)])
    off = c.dev([0, 20])
    k, v = c.pool.gather(c.dev(c.tables), None, off, 20)
    assert bool((k[11] == -1e4).all()) and torch.count_nonzero(v[11]) == 0
    mb = c.tables.shape[1]
    k, v = c.pool.gather(c.dev(c.tables), c.dev([mb * 256 - 4]), off, 20)
    assert c.pool.read_device_error() & _lib.DEVERR_SEQ_LEN and torch.count_nonzero(k[4:]) == 0
    k, v = c.pool.gather(c.dev([[99] * mb]), None, off, 20)
    assert c.pool.read_device_error() & _lib.DEVERR_BLOCK_ID and torch.count_nonzero(v) == 0
    k, v = c.pool.gather(c.dev(c.tables), None, c.dev([0, 0]), 0)
    assert k.shape == (0, 2, 128) and v.device == dev


# -- together ------------------------------------------------------------------

def test_extend_step_rotates_writes_attends_and_reads_back():
    """Two turns of an EXTEND path, as a server runs them, against the definitions."""
    dev = cuda()
    B, hq, hkv, d, rot = 2, 8, 2, 128, 128
    pool, ref = q4.Q4KVPool(hkv, d, 8, device=dev), O.OraclePool(hkv, d, 8)
    tables = np.array([[3, 1, 6], [0, 7, 2]], np.int32)
    tab = torch.as_tensor(tables).to(dev)
    table = _table(rot // 2, 2000)
    ro = q4.Rotary(table.to(dev))
    lens = [0, 0]
    g = torch.Generator().manual_seed(0)
    for T, new in ((290, [290, 200]), (6, [5, 6])):
        q, k, v = (torch.randn(B, T, h, d, generator=g).half() for h in (hq, hkv, hkv))
        dl, dn = (torch.tensor(x, dtype=torch.int32, device=dev) for x in (lens, new))
        qr = pool.append_rotary(k.to(dev), v.to(dev), ro, tab, dl, dn, q=q.to(dev))
        out = q4.extend_attention(pool, qr, tab, dl, dn, out_dtype=torch.float32)
        pos = np.asarray(lens)[None, :, None] + np.arange(T)
        axis = [0] * (rot // 2)
        wq = E.rotary(q.numpy(), "fp16", table.numpy(), pos, axis, False)
        ref.append_tokens(E.rotary(k.numpy(), "fp16", table.numpy(), pos, axis, False), v.numpy(), "fp16", tables, lens, new)
        want, bound = E.extend_attention(ref, wq, "fp16", tables, lens, new)
        _attend_close(out, want, bound)
        lens = [a + b for a, b in zip(lens, new)]
    assert_pool_equal(pool, ref, blocks=[3, 1, 0])
    off = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device=dev)
    k, v = pool.gather(tab, None, off, sum(lens), out_dtype=torch.float32, unrotate_k=True)
    wk, wv = E.gather(ref, tables, [0, 0], lens, True)
    assert torch.equal(k.cpu(), torch.from_numpy(wk)) and torch.equal(v.cpu(), torch.from_numpy(wv))
    assert pool.read_device_error() == 0
