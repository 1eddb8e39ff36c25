"""Host-only checks of include/q4kv_extend.h: every function is exported, plans
cover their shapes, and bad arguments are refused before a device is touched;
and the plain definitions against independent forms of them."""
import ctypes

import numpy as np
import pytest
import torch

from decode_attention_q4kv_b200 import _lib
from oracle import extend_oracle as E
from oracle import q4kv_oracle as O
from test_abi import FAKE, _pool

L = _lib.lib()
BAD, UNS = _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED


def test_exports_every_declared_function():
    names = _lib.header_functions(_lib.EXTEND_HEADER)
    assert set(names) == set(_lib._EXTEND_SIGNATURES)
    for n in names:
        assert hasattr(L, n), n


def test_struct_layouts():
    assert ctypes.sizeof(_lib.RotaryDesc) == 16 + 8 + 128
    assert ctypes.sizeof(_lib.ExtendPlan) == 48


def _plan(B=2, T=7, hq=32, hkv=8, d=128, mb=16, window=0, splits=0, sms=148):
    p = _lib.ExtendPlan()
    return L.q4kv_extend_plan_make(B, T, hq, hkv, d, mb, window, splits, sms, ctypes.byref(p)), p


@pytest.mark.parametrize("B,T,hq,hkv,d,mb", [(1, 4, 32, 8, 128, 4), (16, 5, 32, 8, 128, 129), (4, 509, 40, 8, 128, 66),
                                             (5, 256, 16, 8, 256, 33), (1, 2048, 32, 8, 128, 136), (1, 1, 8, 8, 128, 1),
                                             (3, 0, 8, 8, 256, 2), (0, 3, 8, 8, 128, 2), (1, 9, 64, 1, 256, 512)])
@pytest.mark.parametrize("window", [0, 100, 4096])
def test_plan_covers_context(B, T, hq, hkv, d, mb, window):
    st, p = _plan(B, T, hq, hkv, d, mb, window)
    assert st == 0
    assert 1 <= p.n_splits <= mb * 256 // 64 and p.reserved == 0
    if p.n_splits > 1:
        assert p.workspace_bytes >= B * T * hq * p.n_splits * (d + 2) * 4
    # the plan's own split count reproduces it
    st2, p2 = _plan(B, T, hq, hkv, d, mb, window, p.n_splits, 148)
    assert st2 == 0 and (p2.n_splits, p2.workspace_bytes) == (p.n_splits, p.workspace_bytes)


def test_plan_refusals():
    assert _plan(hq=30)[0] == BAD and _plan(B=-1)[0] == BAD and _plan(T=-1)[0] == BAD
    assert _plan(mb=0)[0] == BAD and _plan(window=-1)[0] == BAD and _plan(splits=-1)[0] == BAD
    assert _plan(d=64)[0] == UNS and _plan(hq=130, hkv=2)[0] == UNS
    assert _plan(B=60000, T=60000)[0] == BAD                       # rows past 2^31
    assert _plan(mb=1 << 23)[0] == BAD                             # positions past 2^31
    assert 16 <= _plan(splits=100000)[1].n_splits <= 32            # clamped to the context


def _attend(pool=None, plan=None, q=FAKE, qdt=0, qs=(7 * 4096, 4096), tab=FAKE, lens=FAKE, nn=None, scale=0.0, out=FAKE, odt=1,
            os_=(7 * 4096, 4096), ws=None, ws_bytes=0):
    pool = _pool() if pool is None else pool
    plan = _plan(splits=1)[1] if plan is None else plan
    return L.q4kv_extend_attention(ctypes.byref(pool), ctypes.byref(plan), q, qdt, qs[0], qs[1], tab, lens, nn, scale, out, odt,
                                   os_[0], os_[1], ws, ws_bytes, None)


def test_attention_refusals():
    assert _attend(qdt=2) == BAD and _attend(odt=3) == BAD and _attend(scale=float("nan")) == BAD
    assert _attend(q=None) == BAD and _attend(q=FAKE + 8) == BAD and _attend(out=None) == BAD and _attend(out=FAKE + 2) == BAD
    assert _attend(qs=(7 * 4096, 4095)) == BAD and _attend(qs=(7 * 4096 + 4, 4096)) == BAD and _attend(os_=(7 * 4096, 1024)) == BAD
    assert _attend(os_=(0, 4096)) == BAD and _attend(os_=(4088, 4096)) == BAD     # rows on top of one another
    assert _attend(tab=None) == BAD and _attend(tab=FAKE + 2) == BAD and _attend(lens=None) == BAD and _attend(nn=FAKE + 2) == BAD
    assert _attend(pool=_pool(n_q4_blocks=0)) == BAD
    assert _attend(pool=_pool(n_kv_heads=4)) == BAD                # the plan's heads are not the pool's
    st, p = _plan(splits=4)
    assert st == 0 and p.workspace_bytes > 0
    assert _attend(plan=p) == _lib.ERR_WORKSPACE
    assert _attend(plan=p, ws=FAKE, ws_bytes=p.workspace_bytes - 1) == _lib.ERR_WORKSPACE
    assert _attend(plan=p, ws=FAKE + 16, ws_bytes=p.workspace_bytes) == _lib.ERR_WORKSPACE
    p.n_splits = 100000
    assert _attend(plan=p, ws=FAKE, ws_bytes=1 << 30) == BAD       # not a plan of the library
    assert _attend(plan=_plan(B=0)[1]) == 0 and _attend(plan=_plan(T=0)[1]) == 0


def _rot(**kw):
    d = dict(rot_dim=128, interleaved=0, n_axes=1, max_positions=10, table=FAKE)
    d.update(kw)
    axis = d.pop("axis", 0)
    r = _lib.RotaryDesc()
    for k, v in d.items():
        setattr(r, k, v)
    r.axis[5] = axis
    return r


def _append(pool=None, rot=None, k=FAKE, v=FAKE, dt=0, B=2, T=4, nn=None, ss=4096, ts=1024, q=FAKE, hq=32, qs=(16384, 4096),
            qo=FAKE + 4096, os_=(16384, 4096), tab=FAKE, mb=4, lens=FAKE, pos=None):
    pool = _pool() if pool is None else pool
    rot = _rot() if rot is None else rot
    return L.q4kv_append_rotary(ctypes.byref(pool), ctypes.byref(rot), k, v, dt, B, T, nn, ss, ts, q, hq, qs[0], qs[1], qo, os_[0],
                                os_[1], tab, mb, lens, pos, None)


def test_append_rotary_refusals():
    for r in (_rot(rot_dim=0), _rot(rot_dim=48), _rot(rot_dim=160), _rot(interleaved=2), _rot(n_axes=0), _rot(n_axes=5),
              _rot(max_positions=0), _rot(table=None), _rot(table=FAKE + 8), _rot(axis=1)):
        assert _append(rot=r) == BAD
    assert _append(dt=2) == BAD and _append(k=FAKE + 8) == BAD and _append(ts=1028) == BAD and _append(lens=None) == BAD
    assert _append(hq=0) == BAD and _append(qo=None) == BAD and _append(q=FAKE + 2) == BAD and _append(pos=FAKE + 2) == BAD
    assert _append(qs=(16384, 4092)) == BAD and _append(os_=(16384 + 2, 4096)) == BAD
    assert _append(os_=(4088, 4096)) == BAD and _append(os_=(0, 4096)) == BAD     # rows on top of one another
    assert _append(qo=FAKE, os_=(20480, 4096)) == BAD              # in place with other strides
    assert _append(pool=_pool(n_q4_blocks=0)) == BAD
    assert _append(B=0) == 0 and _append(T=0) == 0


def _gather(pool=None, tab=FAKE, mb=4, B=2, starts=None, off=FAKE, n=10, k=FAKE, v=FAKE, stride=1024, dt=1, un=0):
    pool = _pool() if pool is None else pool
    return L.q4kv_gather_tokens(ctypes.byref(pool), tab, mb, B, starts, off, n, k, v, stride, dt, un, None)


def test_gather_refusals():
    assert _gather(dt=3) == BAD and _gather(un=2) == BAD and _gather(B=-1) == BAD and _gather(n=-1) == BAD and _gather(n=1 << 31) == BAD
    assert _gather(stride=1020) == BAD and _gather(stride=1028) == BAD and _gather(k=None) == BAD and _gather(v=FAKE + 8) == BAD
    assert _gather(tab=None) == BAD and _gather(mb=0) == BAD and _gather(off=None) == BAD and _gather(starts=FAKE + 1) == BAD
    assert _gather(n=0) == 0 and _gather(B=0) == 0


# -- the plain definitions -------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_definition_is_a_complex_product(interleaved):
    rng = np.random.RandomState(0)
    x = rng.randn(2, 3, 2, 128).astype(np.float16)
    ang = rng.rand(50, 32)
    table = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    pos = rng.randint(0, 50, (2, 2, 3))
    axis = [f % 2 for f in range(32)]
    got = E.rotary(x, "fp16", table, pos, axis, interleaved).astype(np.float64)
    for f in range(32):
        ia, ib = (2 * f, 2 * f + 1) if interleaved else (f, f + 32)
        z = (x[..., ia].astype(np.float64) + 1j * x[..., ib]) * (table[..., 0] + 1j * table[..., 1].astype(np.float64))[pos[axis[f]], f][..., None]
        # one rounding to fp16 and two to binary32 per part
        tol = 2.0 ** -11 * 1.01 * np.abs(z) + 2.0 ** -24
        assert np.all(np.abs(got[..., ia] - z.real) <= tol) and np.all(np.abs(got[..., ib] - z.imag) <= tol)
    assert np.array_equal(got[..., 64:], x[..., 64:])


def test_bf16_rounding_of_the_definition_is_torchs():
    x = np.random.RandomState(1).randn(4096).astype(np.float32)
    x[:4] = [1.00390625, 1.01171875, -1.00390625, 0.0]             # ties
    assert np.array_equal(E.from_f32(x, "bf16"), torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16))


def test_chunk_attention_definition_is_decode_of_each_token():
    rng = np.random.RandomState(2)
    pool = O.OraclePool(2, 128, 4)
    k, v = (rng.randn(300, 2, 128).astype(np.float16) for _ in "kv")
    pool.quantize_blocks(k, v, "fp16", [2, 1])
    pool.invalidate_slots([2 * 256 + 7, 1 * 256 + 30])
    q = rng.randn(1, 5, 4, 128).astype(np.float16)
    tables = np.array([[2, 1]])
    out, bound = E.extend_attention(pool, q, "fp16", tables, [290], [4])
    for i in range(4):
        one = O.decode_attention(pool, q[:, i], "fp16", tables, [291 + i])
        assert np.allclose(out[:, i], one, rtol=0, atol=1e-12)
    assert not out[:, 4].any() and (bound[:, :4] > 0).all()
    w, _ = E.extend_attention(pool, q, "fp16", tables, [290], None, window=1)
    kk, vv = E.gather(pool, tables, [290], [5])
    want = vv.transpose(1, 0, 2).repeat(2, 0)                      # a window of one sees itself only
    want = want.transpose(1, 0, 2)[None]
    assert np.allclose(w, want, rtol=0, atol=1e-12)                # (slot 30 of block 1 is position 286)
