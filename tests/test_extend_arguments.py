"""Host-only checks of the calls of include/q4kv_extend.h: strides and arguments
that would make a kernel write one place twice, or read or write past an array, are
refused before a device is touched."""
import copy
import itertools
import pickle

import pytest

import decode_attention_q4kv_b200 as q4

from decode_attention_q4kv_b200 import _lib
from test_abi import FAKE, _pool
from test_extend_abi import _append, _attend, _gather, _plan

BAD = _lib.ERR_INVALID_ARG


def _share(ss, ts, row, B, T):
    at = sorted(b * ss + i * ts for b in range(B) for i in range(T))
    return any(y - x < row for x, y in zip(at, at[1:]))


@pytest.mark.parametrize("B,T", [(2, 2), (2, 7), (3, 2), (5, 3), (4, 1), (1, 5)])
def test_output_rows_that_share_memory_are_refused(B, T):
    # one KV head of 128: rows of 128, strides in eighths of a row
    pool, plan = _pool(n_kv_heads=1), _plan(B=B, T=T, hq=1, hkv=1, mb=4, splits=1)[1]
    assert plan.workspace_bytes > 0            # the check behind that of the rows: a good call ends there
    kinds = set()
    for ss, ts in itertools.product(range(0, 9 * 128, 16), range(128, 9 * 128, 16)):
        shared = _share(ss, ts, 128, B, T)
        kinds.add(shared)
        kw = dict(qs=(128 * T, 128), os_=(ss, ts))
        assert _attend(pool=pool, plan=plan, **kw) == (BAD if shared else _lib.ERR_WORKSPACE), (ss, ts)
        if shared:
            assert _append(pool=pool, B=B, T=T, ss=128 * T, ts=128, hq=1, **kw) == BAD, (ss, ts)
    assert kinds == ({False} if B == 1 else {False, True})


@pytest.mark.parametrize("stride", [128, 192, 256, 400])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_key_and_value_rows_that_share_memory_are_refused(stride, n):
    pool, shared = _pool(n_kv_heads=1), 0
    for apart in range(-6 * stride, 6 * stride + 1, 8):        # elements of 2 bytes
        if any(abs(apart + i * stride) < 128 for i in range(1 - n, n)):
            shared += 1
            assert _gather(pool=pool, n=n, v=FAKE + 2 * apart, stride=stride) == BAD, apart
    assert shared > 0
    assert _gather(pool=pool, n=0, v=FAKE, stride=stride) == 0


@pytest.mark.parametrize("T,hq,hkv,d,tile,streams", [(512, 8, 2, 128, 128, 1), (16, 8, 2, 128, 128, 2), (4, 8, 2, 128, 128, 2),
                                                     (64, 16, 8, 256, 64, 1)])
def test_no_accumulator_takes_more_than_32768_tokens(T, hq, hkv, d, tile, streams):
    for B, mb in itertools.product((1, 7, 300), (1, 127, 128, 129, 257, 1000, 4096, 131072)):
        for splits in (0, 1, 2, 5, 1000):
            st, p = _plan(B=B, T=T, hq=hq, hkv=hkv, d=d, mb=mb, splits=splits)
            assert st == 0
            steps = -(-mb * 256 // (tile * streams))
            assert -(-steps // p.n_splits) * tile <= 32768, (B, mb, splits)
            again = _plan(B=B, T=T, hq=hq, hkv=hkv, d=d, mb=mb, splits=p.n_splits)[1]
            assert (again.n_splits, again.workspace_bytes) == (p.n_splits, p.workspace_bytes)
            if mb <= 128 and splits == 1:
                assert p.n_splits == 1
    p = _plan(B=300, T=T, hq=hq, hkv=hkv, d=d, mb=131072, window=4096)[1]
    assert p.n_splits == 1                     # a window bounds the tokens by itself


@pytest.mark.parametrize("copied", [copy.copy, copy.deepcopy, lambda p: pickle.loads(pickle.dumps(p))])
def test_a_plan_can_be_copied(copied):
    p = q4.ExtendPlan(2, 7, 32, 8, 128, 200, window=5000, n_splits=3, num_sms=148)
    c = copied(p)
    assert (c.n_splits, c.workspace_bytes, c.window, c._shape) == (p.n_splits, p.workspace_bytes, p.window, p._shape)
    assert c._ref._obj is c.c and bytes(c.c) == bytes(p.c)
    with pytest.raises(AttributeError):
        c.nothing
    assert not hasattr(q4.ExtendPlan.__new__(q4.ExtendPlan), "n_splits")
