"""Refusals of the row operators' further forms, on the CPU (fake addresses: every call here ends on the host)."""
import re

import pytest
import torch

import block_quantized_matmul_quantize_amd as qmm
import rows_single
import rows_util as ref

P = 0x100000       # aligned to every element
Q = P + (1 << 20)
OK, ARG, TYPE, SHAPE = 0, -1, -2, -3


def L():
    return qmm.lib()


def test_combine_with_ids_refusals():
    def f(t=0, n=4, j=2, k=8, h=P, ids=P, ne=3, y=Q):
        return L().qmm_combine_ids(t, h, n, j, k, ids, ne, P, P, y, None)

    def b(t=0, n=4, j=2, k=8, h=P, ids=P, ne=3, y=Q):
        return L().qmm_combine_ids_backward(t, P, h, n, j, k, ids, ne, P, y, P, None)

    for call in (f, b):
        assert call(t=12) == TYPE
        assert call(n=-1) == ARG
        assert call(j=0) == ARG
        assert call(k=0) == ARG
        assert call(k=(1 << 20) + 1) == SHAPE
        assert call(n=1 << 29, j=4) == SHAPE
        assert call(ne=0) == ARG
        assert call(ne=-1) == ARG
        assert call(ne=(1 << 30) + 1) == SHAPE
        assert call(ids=None) == ARG
        assert call(ids=P + 2) == ARG
        assert call(h=None) == ARG
        assert call(h=P + 2) == ARG
        assert call(y=None) == ARG
        assert call(y=P) == ARG
        assert call(n=0, h=None, ids=None, y=None) == OK


def test_combine_wrappers_check_ids():
    h, ids = torch.zeros((4, 2, 16)), torch.zeros((4, 2), dtype=torch.int32)
    for call in (lambda **a: qmm.combine(h, **a), lambda **a: qmm.combine_backward(torch.zeros((4, 16)), h, **a)):
        with pytest.raises(ValueError, match="n_exp"):
            call(ids=ids)
        with pytest.raises(ValueError, match="n_exp"):
            call(ids=ids, n_exp=0)
        with pytest.raises(ValueError, match="ids must be"):
            call(ids=ids[:3], n_exp=4)
        with pytest.raises(TypeError, match="ids must have"):
            call(ids=ids.long(), n_exp=4)
        with pytest.raises(ValueError, match="without pos"):
            call(pos=ids, ids=ids, n_exp=4)
        with pytest.raises(ValueError, match="device"):
            call(ids=ids, n_exp=4)


@pytest.mark.parametrize("missing", ["_get_device", "_get_raw_stream"])
def test_stream_without_torchs_private_calls(missing, monkeypatch):
    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(qmm, missing, None)
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    assert qmm._stream() == 1234


class OnDevice:
    """What the binding's last check asks a tensor."""

    def __init__(self, index):
        self.index, self.device = index, f"cuda:{index}"

    def get_device(self):
        return self.index


def test_tensors_on_another_device_than_the_current_one_are_refused(monkeypatch):
    """Their pointers would go to a kernel on the current device's stream."""
    monkeypatch.setattr(qmm, "_get_device", lambda: 0)
    qmm._same_device(OnDevice(0), None, OnDevice(0))
    with pytest.raises(ValueError, match="current device is 0"):
        qmm._same_device(OnDevice(1), OnDevice(1))
    with pytest.raises(ValueError, match="must be on cuda:0"):
        qmm._same_device(OnDevice(0), OnDevice(1))
    monkeypatch.setattr(qmm, "_get_device", None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    qmm._same_device(OnDevice(1))
    with pytest.raises(ValueError, match="current device is 1"):
        qmm._same_device(OnDevice(0))


def test_embed_from_blocks_says_what_alignment_of_y_it_needs():
    """Blocks are decoded into 8 values a store: y at less than 16 bytes is refused, and the contract says so."""
    for y_type, size in ((qmm.F32, 4), (qmm.F16, 2), (qmm.BF16, 2)):
        for off in (size, 8):
            assert L().qmm_embed(qmm.Q4_K, P, 10, 256, P, 4, 1.0, y_type, P + off, None) == ARG
    with open(qmm.HEADER) as f:
        text = re.sub(r"[\s*]+", " ", f.read())
    of_embed = text[text.index("qmm_embed: y[i]"):text.index("qmm_embed_backward: grad[v]")]
    assert "from blocks 16-byte aligned" in of_embed
    assert "from blocks 16 bytes" in text[text.index("Pointers need the alignment"):text.index("Row lengths")]
    assert "16-byte aligned" in qmm.embed.__doc__


@pytest.mark.parametrize("k,rank", [(72, 8), (520, 40), (2048, 128)])
def test_bound_of_single_products_refuses_two_parts_of_three(k, rank):
    """The oracle's bound for one chain of products holds for fp32 products, and refuses one whose operands keep
    16 of their 24 bits, at every size (among sums of k products such a loss would pass)."""
    x, a, b, ids, scale, _ = rows_single.inputs(k, 120, k, 264, rank, 3, torch.float32, torch.float32)
    want = ref.lora(x, a, b, ids, scale, None)[2]
    got = torch.stack([a[int(c)] @ row for c, row in zip(ids, x)])
    ref.check(got, want, rows_single.SINGLE_TERMS, want.abs())

    def cut(t):
        return (t.view(torch.int32) & ~0xff).view(torch.float32)

    for xx, aa in ((cut(x), a), (x, cut(a)), (cut(x), cut(a))):
        got = torch.stack([aa[int(c)].double() @ row.double() for c, row in zip(ids, xx)])
        off = (got - want).abs() > (rows_single.SINGLE_TERMS + 2) * ref.U32 * want.abs()
        assert off.double().mean() > 0.5
        with pytest.raises(AssertionError):
            ref.check(got.float(), want, rows_single.SINGLE_TERMS, want.abs())
