"""Calls of the operators that extend a cached prompt as they may be made, each
against the definitions: layouts, strides and arguments at their edges."""
import numpy as np
import pytest
import torch

import decode_attention_q4kv_b200 as q4
from helpers import cuda
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
