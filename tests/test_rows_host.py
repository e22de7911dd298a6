"""Refusals of the row operators, on the CPU: every bad argument is turned into an error on the host,
before anything is launched (fake addresses here), and the binding checks tensors before their
addresses reach the library."""
import ctypes

import pytest
import torch

import block_quantized_matmul_quantize_amd as qmm
import rows_util as ref

P = 0x100000       # aligned to every element
OK, ARG, TYPE, SHAPE, WS = 0, -1, -2, -3, -4


def L():
    return qmm.lib()


def test_sort_ids_refusals():
    f = L().qmm_sort_ids
    need = qmm.sort_ids_workspace(100000, 1 << 20)
    assert need > 0 and qmm.sort_ids_workspace(100, 128) == 0
    assert f(P, -1, 4, P, P, P, None, 0, None) == ARG
    assert f(P, 4, 0, P, P, P, None, 0, None) == ARG
    assert f(P, (1 << 30) + 1, 4, P, P, P, None, 0, None) == SHAPE
    assert f(P, 4, (1 << 30) + 1, P, P, P, None, 0, None) == SHAPE
    assert f(None, 4, 4, P, P, P, None, 0, None) == ARG
    assert f(P, 4, 4, None, P, P, None, 0, None) == ARG
    assert f(P, 4, 4, P, P, None, None, 0, None) == ARG
    assert f(P + 2, 4, 4, P, P, P, None, 0, None) == ARG
    assert f(P, 100000, 1 << 20, P, P, P, None, 0, None) == WS
    assert f(P, 100000, 1 << 20, P, P, P, P, need - 1, None) == WS
    assert f(P, 100000, 1 << 20, P, P, P, P + 16, need, None) == ARG
    assert qmm.sort_ids_workspace(-1, 4) == 0 and qmm.sort_ids_workspace(4, 0) == 0


def test_pair_operator_refusals():
    g, c, b = L().qmm_gather_sorted, L().qmm_combine, L().qmm_combine_backward
    Q = P + (1 << 20)
    for call in (lambda t=0, n=4, j=2, k=8, x=P, y=Q: g(t, x, n, j, k, P, P, y, None),
                 lambda t=0, n=4, j=2, k=8, x=P, y=Q: c(t, x, n, j, k, P, P, P, y, None),
                 lambda t=0, n=4, j=2, k=8, x=P, y=Q: b(t, x, P, n, j, k, P, P, P, y, P, None)):
        assert call(t=12) == TYPE
        assert call(n=-1) == ARG
        assert call(j=0) == ARG
        assert call(k=0) == ARG
        assert call(k=(1 << 20) + 1) == SHAPE
        assert call(n=1 << 29, j=4) == SHAPE
        assert call(x=None) == ARG
        assert call(y=None) == ARG
        assert call(y=P) == ARG                # out of place only
        assert call(x=P + 2) == ARG            # fp32 at 2 bytes
        assert call(t=1, x=P + 1) == ARG
        assert call(n=0, x=None, y=None) == OK
    assert g(0, P, 4, 2, 8, None, P, Q, None) == ARG
    assert g(0, P, 4, 2, 8, P, None, Q, None) == ARG
    assert b(0, P, P, 4, 2, 8, P, P, None, Q, P, None) == ARG
    assert b(0, P, P, 4, 2, 8, None, P, None, Q, None, None) == ARG


def test_embed_refusals():
    f = L().qmm_embed
    assert f(3, P, 10, 256, P, 4, 1.0, 0, P, None) == TYPE
    assert f(12, P, 10, 256, P, 4, 1.0, 12, P, None) == TYPE
    assert f(12, P, 10, 255, P, 4, 1.0, 0, P, None) == SHAPE
    assert f(12, P, 0, 256, P, 4, 1.0, 0, P, None) == ARG
    assert f(12, P, 10, 256, P, -1, 1.0, 0, P, None) == ARG
    assert f(12, P + 1, 10, 256, P, 4, 1.0, 0, P, None) == ARG
    assert f(12, P, 10, 256, P, 4, 1.0, 0, P + 4, None) == ARG
    assert f(0, P + 2, 10, 256, P, 4, 1.0, 0, P, None) == ARG
    assert f(0, P, 10, 1 << 21, P, 4, 1.0, 0, P, None) == SHAPE
    assert f(0, None, 10, 256, P, 4, 1.0, 0, P, None) == ARG
    assert f(0, None, 10, 256, None, 0, 1.0, 0, None, None) == OK
    f = L().qmm_embed_backward
    need = qmm.embed_backward_workspace(100, 64, 1000)
    assert need > 0 and qmm.embed_backward_workspace(0, 64, 1000) == 0
    assert f(12, P, 100, 64, P, 1000, 1.0, 0, P, P, need, None) == TYPE
    assert f(0, P, 100, 64, P, 1000, 1.0, 8, P, P, need, None) == TYPE
    assert f(0, P, 100, 64, P, 0, 1.0, 0, P, P, need, None) == ARG
    assert f(0, P, 100, 0, P, 1000, 1.0, 0, P, P, need, None) == ARG
    assert f(0, P, 100, 64, P, 1000, 1.0, 0, None, P, need, None) == ARG
    assert f(0, P, 100, 64, P, 1000, 1.0, 0, P + 2, P, need, None) == ARG
    assert f(0, P, 100, 64, P, 1000, 1.0, 0, P, P, need - 1, None) == WS
    assert f(0, P, 100, 64, P, 1000, 1.0, 0, P, None, need, None) == WS


def test_lora_refusals():
    Q = P + (1 << 20)

    def f(xt=0, wt=0, x=P, n=100, k=64, a=P, rows=32, rank=8, na=3, y=Q, ws=P, nw=1 << 30):
        return L().qmm_lora(xt, wt, x, n, k, a, P, rows, rank, na, P, P, P, y, P, ws, nw, None)

    def g(xt=0, wt=0, x=P, n=100, k=64, a=P, rows=32, rank=8, na=3, y=Q, ws=P, nw=1 << 30):
        return L().qmm_lora_backward(xt, wt, x, P, P, n, k, a, P, rows, rank, na, P, P, P, y, Q, Q, ws, nw, None)

    for call in (f, g):
        assert call(xt=12) == TYPE
        assert call(wt=12) == TYPE
        assert call(xt=30, wt=0) == TYPE
        assert call(xt=1, wt=30) == TYPE
        assert call(n=-1) == ARG
        assert call(k=0) == ARG
        assert call(rows=0) == ARG
        assert call(rank=0) == ARG
        assert call(rank=129) == SHAPE
        assert call(na=0) == ARG
        assert call(na=1 << 21) == SHAPE
        assert call(na=1 << 20, rank=128, k=1 << 20) == SHAPE
        assert call(x=None) == ARG
        assert call(a=None) == ARG
        assert call(x=P + 2) == ARG
        assert call(wt=30, a=P + 1) == ARG
        assert call(y=P) == ARG
        assert call(ws=None) == WS
        assert call(nw=16) == WS
        assert call(ws=P + 8) == ARG
    assert f(n=0, x=None, y=None, ws=None) == OK
    assert L().qmm_lora_backward(0, 0, P, P, P, 10, 64, P, P, 32, 8, 3, P, P, None, None, None, None, None, 0, None) == OK


def test_wrappers_check_tensors_before_addresses():
    x, ids = torch.zeros((4, 16)), torch.zeros((4, 2), dtype=torch.int32)
    bounds, h = torch.zeros(5, dtype=torch.int32), torch.zeros((8, 16))
    with pytest.raises(ValueError, match="device"):
        qmm.sort_ids(ids, 4)
    with pytest.raises(TypeError, match="int32"):
        qmm.sort_ids(ids.long(), 4)
    with pytest.raises(ValueError, match="n_keys"):
        qmm.sort_ids(ids, 0)
    with pytest.raises(ValueError, match="x must be"):
        qmm.gather_sorted(x[:3], ids, bounds)
    with pytest.raises(ValueError, match="contiguous"):
        qmm.gather_sorted(x[:, ::2], ids, bounds)
    with pytest.raises(TypeError, match="float32, float16 or bfloat16"):
        qmm.gather_sorted(x.double(), ids, bounds)
    with pytest.raises(ValueError, match="out must be"):
        qmm.gather_sorted(x, ids, bounds, out=torch.zeros((7, 16)))
    with pytest.raises(ValueError, match="h must be"):
        qmm.combine(h[:7], ids)
    with pytest.raises(ValueError, match="weights must be"):
        qmm.combine(h, ids, torch.zeros((2, 4)))
    with pytest.raises(TypeError, match="base must have"):
        qmm.combine(h, ids, base=x.half())
    with pytest.raises(ValueError, match="3-D"):
        qmm.combine(h)
    with pytest.raises(TypeError, match="bounds"):
        qmm.combine_backward(x, h, ids, None, None)
    with pytest.raises(ValueError, match="dy must be"):
        qmm.combine_backward(x[:3], h, ids, None, bounds)
    with pytest.raises(ValueError, match="table holds"):
        qmm.embed(torch.zeros(143, dtype=torch.uint8), qmm.Q4_K, 1, 256, ids)
    with pytest.raises(ValueError, match="table holds"):
        qmm.embed(x, qmm.F32, 5, 16, ids)
    with pytest.raises(TypeError, match="table must have"):
        qmm.embed(x, qmm.BF16, 4, 16, ids)
    with pytest.raises(TypeError, match="dtype must be"):
        qmm.embed(x, qmm.F32, 4, 16, ids, dtype=torch.float64)
    with pytest.raises(ValueError, match="out must be"):
        qmm.embed(x, qmm.F32, 4, 16, ids, out=torch.zeros((4, 16)))
    with pytest.raises(ValueError, match="dy must be"):
        qmm.embed_backward(x, ids, 4)
    with pytest.raises(ValueError, match="vocab"):
        qmm.embed_backward(torch.zeros((4, 2, 16)), ids, 0)
    a, b, one = torch.zeros((3, 8, 16)), torch.zeros((3, 24, 8)), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="a must be"):
        qmm.lora(x, a[:, :, :8].contiguous(), b, one)
    with pytest.raises(ValueError, match="b must be"):
        qmm.lora(x, a, b[:2], one)
    with pytest.raises(TypeError, match="b must have"):
        qmm.lora(x, a, b.half(), one)
    with pytest.raises(ValueError, match="ids must be"):
        qmm.lora(x, a, b, one[:3])
    with pytest.raises(ValueError, match="scale must be"):
        qmm.lora(x, a, b, one, torch.zeros(2))
    with pytest.raises(ValueError, match="base must be"):
        qmm.lora(x, a, b, one, base=torch.zeros((4, 23)))
    with pytest.raises(ValueError, match="h must be"):
        qmm.lora_backward(x, torch.zeros((4, 24)), torch.zeros((4, 7)), a, b, one)
    with pytest.raises(ValueError, match="device"):
        qmm.lora(x, a, b, one)


def test_tolerance_catches_a_planted_mistake():
    """The oracle's check refuses a result that is off by one rounding step of its type too many, a
    dropped term and a NaN."""
    g = torch.Generator()
    g.manual_seed(1)
    h, pos = torch.randn((8, 32), generator=g), torch.tensor([[0, 3], [5, -1]], dtype=torch.int32)
    h4 = torch.cat([h[:4]])
    want, mag = ref.combine(h4, pos.clamp(max=3), torch.ones((2, 2)), None)
    ref.check(want.float(), want, 2, mag)
    ref.check(want.to(torch.bfloat16), want, 2, mag)
    with pytest.raises(AssertionError):
        ref.check((want * (1 + 2.0 ** -6)).to(torch.bfloat16), want, 2, mag)
    with pytest.raises(AssertionError):
        ref.check((want - h4[3].double() * 1e-3).float(), want, 2, mag)
    bad = want.float()
    bad[0, 0] = float("nan")
    with pytest.raises(AssertionError):
        ref.check(bad, want, 2, mag)


def test_reference_sort():
    ids = torch.tensor([[3, 0], [-1, 3], [2, 0]], dtype=torch.int32)
    order, pos, bounds = ref.sort_ids(ids, 4)
    assert order.tolist() == [1, 5, 4, 0, 3, 2] and pos.tolist() == [[3, 0], [-1, 4], [2, 1]]
    assert bounds.tolist() == [0, 2, 2, 3, 5]


def test_error_message_is_set():
    assert L().qmm_embed(3, P, 10, 256, P, 4, ctypes.c_float(1.0), 0, P, None) == TYPE
    assert b"table type 3" in L().qmm_last_error()
