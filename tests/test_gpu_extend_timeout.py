"""Waits of the chunk-attention kernel that give up: the call ends, the rows of
the blocks concerned are 0, Q4KV_DEVERR_TIMEOUT is raised, and the context stays
usable.  A limit of a few tries stands in for the seconds of the real one: every
block starts with waits for copies that cannot have landed yet."""
import ctypes
import time

import numpy as np
import pytest
import torch

import decode_attention_q4kv_b200 as q4
from decode_attention_q4kv_b200 import _lib
from helpers import cuda
from test_gpu_extend import Case, _attend_close

pytestmark = pytest.mark.gpu


def _limited(c, plan, tries):
    dev = cuda()
    q, tab, lens, nn = c.q.to(dev), c.dev(c.tables), c.dev(c.lens), c.dev(c.n_new)
    out = torch.full(c.q.shape, 7.0, device=dev)
    ws = plan.workspace(dev)
    row = c.hq * c.d
    t0 = time.monotonic()
    _lib.check(_lib.lib().q4kv_selftest_extend_wait(
        ctypes.byref(c.pool.desc), ctypes.byref(plan.c), q.data_ptr(), _lib.F16, c.T * row, row, tab.data_ptr(), lens.data_ptr(),
        nn.data_ptr(), 0.0, out.data_ptr(), _lib.F32, c.T * row, row, None if ws is None else ws.data_ptr(),
        0 if ws is None else ws.numel(), tries, torch.cuda.current_stream(dev).cuda_stream), "selftest")
    torch.cuda.synchronize()
    assert time.monotonic() - t0 < 30.0
    return out


# two row tiles, one row tile on alternate key tiles, few rows, heads of 256
@pytest.mark.parametrize("T,d", [(70, 128), (20, 128), (4, 128), (20, 256)])
@pytest.mark.parametrize("widths,fp8", [((4,), False), ((4, 8, 2), False), ((4,), True)])
@pytest.mark.parametrize("splits", [1, 3])
def test_waits_that_give_up(T, d, widths, fp8, splits):
    c = Case([1500, 700], T, 8, 2, d, "fp16", n_new=[T, T - 1], widths=widths, fp8=fp8, seed=T)
    want, bound = c.want()
    plan = q4.ExtendPlan(2, T, 8, 2, d, c.tables.shape[1], n_splits=splits)
    out = _limited(c, plan, 0)
    assert torch.count_nonzero(out) == 0
    assert c.pool.read_device_error() == _lib.DEVERR_TIMEOUT
    for tries in (1, 2, 3, 5, 9, 20, 50, 200):
        # a row is right or, where its block (any block that has a share of it) gave up, 0
        out = _limited(c, plan, tries).cpu()
        gone = (out == 0).all(-1).numpy()
        lost = bool(c.pool.read_device_error() & _lib.DEVERR_TIMEOUT)
        real = np.ones(gone.shape, bool)
        real[1, T - 1:] = False
        assert gone[~real].all() and (lost or not gone[real].any())
        if not gone.all():
            _attend_close(out[torch.from_numpy(~gone)], want[~gone], bound[~gone], what=f"{tries} tries")
    _attend_close(c.run(plan=plan), want, bound, what="the call after")
    assert c.pool.read_device_error() == 0


def test_the_limit_is_checked():
    c = Case([10], 2, 8, 2, 128, "fp16", n_new=[2])
    plan = q4.ExtendPlan(1, 2, 8, 2, 128, c.tables.shape[1], n_splits=1)
    for bad in (-1, 1 << 24):
        with pytest.raises(q4.Q4KVError):
            _limited(c, plan, bad)
