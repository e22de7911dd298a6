"""Forms of the row operators' calls on the GPU: the combine straight on the expert products' results, streams,
single gradients, the precision of single products, the example's gradients."""
import os
import sys

import numpy as np
import pytest
import torch

import block_quantized_matmul_quantize_amd as qmm
import oracle
import rows_single
import rows_util as ref
import synth
from test_gpu_rows import BF16, F16, F32, dev, gen, lora_case, lora_terms, normal, some_ids

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------
# combine on (token, slot) order with ids
# ------------------------------------------------------------------------------------------------
def own_places(ids, n_exp):
    """pos of pairs in (token, slot) order: the pair itself, -1 for an id outside [0, n_exp)."""
    each = torch.arange(ids.numel(), dtype=torch.int32).view(ids.shape)
    return torch.where((ids >= 0) & (ids < n_exp), each, torch.full_like(each, -1))


@pytest.mark.parametrize("n,top_k", [(1, 8), (16, 8), (150, 2)])
@pytest.mark.parametrize("stale", [7.0, float("nan")])
def test_combine_of_matmul_id_without_its_stale_rows(n, top_k, stale):
    """matmul_id leaves the row of a pair without an expert as it was in out; the combine with its ids does
    not read it, and gives it no gradient."""
    n_exp, rows, k = 10, 136, 512
    g, r = gen(n), synth.rngs(40 + n, 2)
    w = torch.from_numpy(np.ascontiguousarray(synth.gen_weights(qmm.Q4_K, n_exp * rows, k, r[0])))
    ids = some_ids(g, n * top_k, n_exp, bad=0.3).view(n, top_k)
    ids[0, 0] = -1
    if n > 1:
        ids[1] = torch.tensor([n_exp, -1] * (top_k // 2), dtype=torch.int32)   # a token without any expert
    pos = own_places(ids, n_exp)
    out = torch.full((n, top_k, rows), stale, device="cuda")
    h, ws = qmm.matmul_id(dev(w), qmm.Q4_K, n_exp, rows, k, dev(normal(g, n, k)), dev(ids), out=out)
    assert qmm.matmul_id_invalid_count(ws) == int((pos < 0).sum())
    weights, base, dy = torch.rand((n, top_k), generator=g), normal(g, n, rows), normal(g, n, rows)
    hc = h.cpu().view(-1, rows)
    for bb in (base, None):
        y = qmm.combine(h, None, dev(weights), base=dev(bb), ids=dev(ids), n_exp=n_exp)
        want, mag = ref.combine(hc, pos, weights, bb)
        ref.check(y, want, top_k + 1, mag, "combine")
    dh, dw = qmm.combine_backward(dev(dy), h, None, dev(weights), ids=dev(ids), n_exp=n_exp)
    wh, ww, mw = ref.combine_backward(dy, hc, pos, weights)
    ref.check(dh, wh.view(dh.shape), 1, wh.view(dh.shape).abs(), "dh")
    ref.check(dw, ww, rows, mw, "dw")
    assert not dh.cpu()[pos < 0].any() and not dw.cpu()[pos < 0].any()


@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n,top_k,k", [(1, 1, 1), (5, 3, 7), (33, 10, 264), (300, 2, 1000)])
@pytest.mark.parametrize("off", [0, 1])
def test_combine_with_ids(n, top_k, k, dtype, off):
    g = gen(n + k)
    n_exp = 12
    ids = some_ids(g, n * top_k, n_exp, bad=0.3).view(n, top_k)
    pos = own_places(ids, n_exp)
    h = normal(g, n * top_k, k, dtype=dtype)
    h[pos.view(-1) < 0] = float("nan")
    w, base, dy = torch.rand((n, top_k), generator=g), normal(g, n, k, dtype=dtype), normal(g, n, k, dtype=dtype)
    hd, idd = dev(h.view(n, top_k, k), off), dev(ids)
    for ww in (w, None):
        based = dev(base, off)
        qmm.combine(hd, None, dev(ww), base=based, out=based, ids=idd, n_exp=n_exp)
        want, mag = ref.combine(h, pos, ww, base)
        ref.check(based, want, top_k + 1, mag, "combine")
        dh, dw = qmm.combine_backward(dev(dy, off), hd, None, dev(ww), ids=idd, n_exp=n_exp)
        wh, wd, mw = ref.combine_backward(dy, h, pos, ww)
        ref.check(dh, wh.view(dh.shape), 1, wh.view(dh.shape).abs(), "dh")
        ref.check(dw, wd, k, mw, "dw")


# ------------------------------------------------------------------------------------------------
# Streams
# ------------------------------------------------------------------------------------------------
def test_stream_is_torchs_current_one():
    """By torch's own calls and by its public one, on the default stream and on another."""
    assert qmm._stream() == torch.cuda.current_stream().cuda_stream
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        assert qmm._stream() == torch.cuda.current_stream().cuda_stream == s.cuda_stream
    assert qmm._stream() == torch.cuda.current_stream().cuda_stream


# ------------------------------------------------------------------------------------------------
# Autograd
# ------------------------------------------------------------------------------------------------
def test_results_require_no_gradient_as_documented():
    """The calls take inputs that require a gradient; autograd records none, and each docstring names the
    call that computes it."""
    g = gen(8)
    t = [dev(normal(g, *s)).requires_grad_() for s in ((12, 32), (24, 32), (3, 8, 32), (3, 32, 8), (12, 2))]
    x, h, a, b, w = t
    ids = dev(torch.randint(0, 3, (12, 2), generator=g, dtype=torch.int32))
    _, pos, bounds = qmm.sort_ids(ids, 3)
    one = ids[:, 0].contiguous()
    for name, y in (("combine", qmm.gather_sorted(x, pos, bounds)), ("combine_backward", qmm.combine(h, pos, w, base=x)),
                    ("embed_backward", qmm.embed(x, qmm.F32, 12, 32, one)), ("lora_backward", qmm.lora(x, a, b, one))):
        assert not y.requires_grad, name
    for call, name in ((qmm.gather_sorted, "combine"), (qmm.combine, "combine_backward"), (qmm.embed, "embed_backward"),
                       (qmm.lora, "lora_backward")):
        assert name in call.__doc__ and "autograd" in call.__doc__


# ------------------------------------------------------------------------------------------------
# Gradient of the gather
# ------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("n,top_k,n_exp,k", [(1, 1, 1, 1), (9, 8, 16, 33), (64, 2, 8, 256)])
def test_gather_gradient(n, top_k, n_exp, k, dtype):
    """combine without weights against the gradient's formula, rows past the valid pairs (which no token owns) NaN;
    and against differences: the gather is linear, so those of any step have no error of their own."""
    g = gen(n + k)
    ids = some_ids(g, n * top_k, n_exp, bad=0.2).view(n, top_k)
    _, pos, bounds = qmm.sort_ids(dev(ids), n_exp)
    d = normal(g, n * top_k, k, dtype=dtype)
    d[int(bounds[-1]):] = float("nan")
    dx = qmm.combine(dev(d), pos)
    want, mag = ref.combine(d, pos.cpu(), None, None)
    ref.check(dx, want, top_k, mag, "dx")
    x, step = normal(g, n, k, dtype=dtype), normal(g, n, k, dtype=dtype)
    valid = int(bounds[-1])

    def loss(v):
        xs = qmm.gather_sorted(dev(v), pos, bounds).cpu().double()
        return float((xs[:valid] * d[:valid].double()).sum())

    slope = loss(x + step) - loss(x)
    moved = (x + step).double() - x.double()   # as the type holds it
    # dx off by the bound of ref.check: top_k + 2 roundings of fp32, then one of the type; 64-bit sums beside it
    rel = (top_k + 2) * ref.U32 + (torch.finfo(dtype).eps if dtype != F32 else 0.0) + 1e-12
    assert abs(slope - float((dx.cpu().double() * moved).sum())) <= rel * float((mag * moved.abs()).sum()) + 1e-9


# ------------------------------------------------------------------------------------------------
# One gradient of the adapters alone
# ------------------------------------------------------------------------------------------------
ELEM = {F32: qmm.F32, F16: qmm.F16, BF16: qmm.BF16}


def backward_of(x, dy, h, a, b, ids, scale, shape, dx=None, da=None, db=None):
    """qmm_lora_backward itself, which takes each gradient or leaves it out; the inputs that the wanted ones do
    not need may be None.  The workspace has its stated size, and what is behind it stays."""
    n, k, rows, rank, na, xt, wt = shape
    size, guard = qmm.lora_backward_workspace(n, k, rows, rank, na), 4096
    ws = torch.full((size + guard,), 77, dtype=torch.uint8, device="cuda")
    p = [None if t is None else t.data_ptr() for t in (x, dy, h, a, b, ids, scale, dx, da, db)]
    st = qmm.lib().qmm_lora_backward(ELEM[xt], ELEM[wt], p[0], p[1], p[2], n, k, p[3], p[4], rows, rank, na, p[5], p[6],
                                     None, p[7], p[8], p[9], ws.data_ptr(), size, qmm._stream())
    assert st == 0, qmm.lib().qmm_last_error()
    assert bool((ws[size:] == 77).all())


# several workgroups an adapter, as many or more for one gradient as for both; none; few rows an adapter; no rows
@pytest.mark.parametrize("n,k,rows,rank,na", [(1300, 130, 72, 16, 1), (2100, 4104, 2000, 40, 1), (513, 256, 512, 12, 2),
                                              (3000, 100, 520, 128, 3), (157, 300, 1000, 33, 57), (0, 64, 40, 8, 2)])
@pytest.mark.parametrize("xt,wt", [(F32, F32), (F32, F16), (BF16, BF16), (F16, F16)])
def test_lora_backward_of_one_gradient(n, k, rows, rank, na, xt, wt):
    x, a, b, ids, scale, _, dy, _ = lora_case(n + k, n, k, rows, rank, na, xt, wt)
    h = ref.lora(x, a, b, ids, scale, None)[2].float()
    none = (ids < 0) | (ids >= na)
    x[none], dy[none], h[none] = float("nan"), float("nan"), float("nan")
    want, mag, most = ref.lora_backward(x, dy, h, a, b, ids, scale, None)
    xd, dyd, hd, ad, bd, idd, sd = (dev(t) for t in (x, dy, h, a, b, ids, scale))
    shape = (n, k, rows, rank, na, xt, wt)
    da = torch.full(a.shape, 5.0, device="cuda")
    backward_of(xd, dyd, None, None, bd, idd, sd, shape, da=da)
    ref.check(da, want[1], lora_terms(rows, 3 * most), mag[1], "da alone")
    db = torch.full(b.shape, 5.0, device="cuda")
    backward_of(None, dyd, hd, None, None, idd, sd, shape, db=db)
    ref.check(db, want[2], 9 * most + 8, mag[2], "db alone")
    dx = torch.full(x.shape, 5.0, dtype=xt, device="cuda")
    backward_of(None, dyd, None, ad, bd, idd, sd, shape, dx=dx)
    ref.check(dx, want[0], lora_terms(rows, rank), mag[0], "dx alone")
    again = torch.full(b.shape, 6.0, device="cuda"), torch.full(x.shape, 6.0, dtype=xt, device="cuda")
    backward_of(None, dyd, hd, ad, bd, idd, sd, shape, dx=again[1], db=again[0])
    assert torch.equal(again[1], dx)
    ref.check(again[0], want[2], 9 * most + 8, mag[2], "db beside dx")


# ------------------------------------------------------------------------------------------------
# Precision of the adapters' products
# ------------------------------------------------------------------------------------------------
# ranks: every width of the first product's tiles and of the second's steps, filled and not
@pytest.mark.parametrize("k,rows,rank", [(72, 264, 8), (2048, 130, 20), (333, 520, 32), (520, 100, 40), (264, 768, 64),
                                         (4104, 72, 100), (200, 1000, 128)])
@pytest.mark.parametrize("xt,wt", [(F32, F32), (F32, F16), (F32, BF16), (F16, F16), (BF16, BF16)])
def test_lora_products_keep_every_bit_of_their_operands(k, rows, rank, xt, wt):
    """Where every result is one chain of products, no sum hides what a product leaves out (SINGLE_TERMS)."""
    na, n = 3, 120
    x, a, b, ids, scale, dy = rows_single.inputs(k + rank, n, k, rows, rank, na, xt, wt)
    wy, _, wh, _ = ref.lora(x, a, b, ids, scale, None)
    y, h = qmm.lora(*(dev(t) for t in (x, a, b, ids, scale)), keep_h=True)
    ref.check(h, wh, rows_single.SINGLE_TERMS, wh.abs(), "h")
    ref.check(y, wy, rows_single.SINGLE_TERMS, wy.abs(), "y")
    h = wh.float()
    want, _, _ = ref.lora_backward(x, dy, h, a, b, ids, scale, None)
    got = qmm.lora_backward(*(dev(t) for t in (x, dy, h, a, b, ids, scale)))
    for u, v, name in zip(got, want, ("dx", "da", "db")):
        ref.check(u, v, rows_single.SINGLE_TERMS, v.abs(), name)


# ------------------------------------------------------------------------------------------------
# The example
# ------------------------------------------------------------------------------------------------
def test_example_moves_along_each_gradient():
    """One step of the example moves each trained tensor along the gradient that 64-bit autograd has for the layer
    without quantized activations.  These are off by at most 1/254 of a block's largest value, 0.9 % of its
    spread where that is 4 times the spread; three products deep and within dz that is below 3 %, and as random
    as dz itself in the sums over rows.  A gradient that lacks a term, a scale or a row's sign is off by its own
    size: the bound, 10 %, is between."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import adapted_layer as ex
    finally:
        sys.path.pop(0)
    layer, n, g = ex.Layer(), 96, gen(21)
    tokens = torch.randint(0, ex.VOCAB, (n,), generator=g, dtype=torch.int32)
    tokens[-2:] = -1
    requests = (torch.arange(n) * ex.REQUESTS // n).to(torch.int32)
    requests[:4] = -1
    top, experts = torch.topk(torch.randn((n, ex.N_EXP), generator=g), ex.TOP_K, dim=1)
    gates, target = torch.softmax(top, 1), normal(g, n, ex.K)
    args = [dev(t) for t in (tokens, requests, experts.to(torch.int32).contiguous(), gates, target)]
    for _ in range(3):   # b begins at zero, where a has no gradient
        layer.step(*args, 0.1)
    trained = [t.cpu().double().requires_grad_() for t in (layer.a, layer.b, layer.extra)]
    layer.step(*args, 0.1)
    moved = [t.detach() - v.cpu().double() for t, v in zip(trained, (layer.a, layer.b, layer.extra))]

    def values(w, qtype, rows):
        return torch.from_numpy(oracle.dequantize(qtype, w.cpu().numpy(), rows, ex.K)).double().view(rows, ex.K)

    a, b, extra = trained
    table, proj = values(layer.table, qmm.Q6_K, ex.VOCAB), values(layer.proj, qmm.Q4_K, ex.K)
    w = torch.stack([values(e, qmm.Q4_K, ex.K) for e in layer.experts])
    tok = tokens.clamp(min=0).long()
    x = (table[tok] * layer.unit + extra[tok]) * (tokens >= 0)[:, None]
    req = requests.clamp(min=0).long()
    low = torch.matmul(b[req], torch.matmul(a[req], x[:, :, None]))[:, :, 0] * (layer.scale.cpu().double()[req])[:, None]
    y = x @ proj.t() / layer.norm + low * (requests >= 0)[:, None]
    z = y
    for j in range(ex.TOP_K):
        z = z + gates[:, j:j + 1].double() * torch.matmul(w[experts[:, j]], y[:, :, None])[:, :, 0] / layer.norm
    want = torch.autograd.grad(((z - target.double()) ** 2).mean(), trained)
    for name, u, v in zip(("a", "b", "extra"), moved, want):
        assert v.norm() > 0 and float((u / u.norm() - v / v.norm()).norm()) <= 0.1, name
