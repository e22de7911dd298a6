"""The row operators at the sizes where they change their launches: sorts of one and two launches a pass,
windows and slices of the adapters' products, adapters sorted beside a product or before it, tables
that are cleared in two launches, and the example that runs everything together."""
import os
import sys

import pytest
import torch

import block_quantized_matmul_quantize_amd as qmm
import rows_util as ref
from test_gpu_rows import BF16, DEV, F16, F32, dev, gen, lora_case, lora_terms, normal, some_ids

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,n_keys,off", [(1023, 100, 1), (1024, 2047, 0), (1025, 2048, 1), (4097, 17, 1), (65536, 200, 0),
                                          (65537, 200, 1), (66000, 70000, 1), (65000, 1 << 22, 1)])
def test_sort_ids_at_launch_borders(n, n_keys, off):
    g = gen(n + n_keys)
    for ids in (some_ids(g, n, n_keys), some_ids(g, n, 3), (torch.arange(n) // 700 % n_keys).to(torch.int32)):
        want = ref.sort_ids(ids, n_keys)
        got = qmm.sort_ids(dev(ids, off), n_keys)
        for w, o, name in zip(want, got, ("order", "pos", "bounds")):
            assert torch.equal(w, o.cpu()), (name, n, n_keys)


# n, k, rows, rank, adapters: more rows than are summed in the second half, sorted beside a product (2048 rows,
# 255 adapters) or before it, tiles spread over workgroups or not, several slices of K and of the columns
LARGE = [(257, 300, 520, 16, 2), (1024, 2056, 40, 4, 7), (2048, 130, 264, 20, 255), (2049, 64, 96, 16, 256),
         (3000, 520, 72, 64, 3), (700, 24, 1040, 100, 1), (64, 8, 2048, 3, 64), (5000, 33, 17, 9, 1000)]


@pytest.mark.parametrize("xt,wt", [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16), (F16, F16)])
@pytest.mark.parametrize("n,k,rows,rank,na", LARGE)
def test_lora_large(n, k, rows, rank, na, xt, wt):
    x, a, b, ids, scale, base, dy, dx_base = lora_case(n + k, n, k, rows, rank, na, xt, wt)
    if na > 100:   # every row its own adapter, as in a step of single tokens
        ids = some_ids(gen(n), n, na)
    none = (ids < 0) | (ids >= na)
    x[none], dy[none] = float("nan"), float("nan")
    xd, ad, bd, idd, sd = dev(x), dev(a), dev(b), dev(ids), dev(scale)
    y, h = qmm.lora(xd, ad, bd, idd, sd, base=dev(base), keep_h=True)
    wy, my, wh, mh = ref.lora(x, a, b, ids, scale, base)
    ref.check(h, wh, 3 * k, mh, "h")
    ref.check(y, wy, lora_terms(k, rank), my, "y")
    assert torch.equal(y, qmm.lora(xd, ad, bd, idd, sd, base=dev(base)))
    h = wh.float()
    h[none] = float("nan")
    got = qmm.lora_backward(xd, dev(dy), dev(h), ad, bd, idd, sd, dx_base=dev(dx_base))
    want, mag, most = ref.lora_backward(x, dy, h, a, b, ids, scale, dx_base)
    ref.check(got[0], want[0], lora_terms(rows, rank), mag[0], "dx")
    ref.check(got[1], want[1], lora_terms(rows, 3 * most), mag[1], "da")
    ref.check(got[2], want[2], 9 * most + 8, mag[2], "db")
    for u, v in zip(got, qmm.lora_backward(xd, dev(dy), dev(h), ad, bd, idd, sd, dx_base=dev(dx_base))):
        assert torch.equal(u, v)


def test_lora_infinity_and_the_largest_values():
    """A value near the largest does not overflow in its parts; an infinity stays itself beside bf16
    matrices, and not finite beside the others, whose parts of zero it meets."""
    x = torch.zeros((3, 64))
    x[1, 3], x[2, 60] = float("inf"), -3.0e38
    a = torch.full((1, 2, 64), 1.0)
    a[0, 1] = -2.0 ** -4
    ids = torch.zeros(3, dtype=torch.int32)
    b = torch.zeros((1, 32, 2))
    b[0, :, 0] = 1.0
    big = x[2, 60]
    for wt in (F32, BF16, F16):
        _, h = qmm.lora(dev(x), dev(a.to(wt)), dev(b.to(wt)), dev(ids), keep_h=True)
        h = h.cpu()
        assert h[0].tolist() == [0.0, 0.0]
        assert torch.equal(h[2], torch.stack([big, big * -2.0 ** -4]))
        assert not torch.isfinite(h[1]).any()
        if wt == BF16:
            assert h[1].tolist() == [float("inf"), float("-inf")]


@pytest.mark.parametrize("dtype,out", [(F32, F32), (BF16, F32)])
def test_embed_backward_table_beyond_the_cache(dtype, out):
    """A table of 280 MB: cleared in two launches, sums that span chunks joined in the second."""
    g = gen(3)
    vocab, n, k = 70000, 500, 1000
    ids = some_ids(g, n, vocab)
    ids = torch.where(torch.rand(n, generator=g) < 0.4, torch.full_like(ids, 60001), ids)
    ids[0] = 17
    dy = normal(g, n, k, dtype=dtype)
    got = qmm.embed_backward(dev(dy), dev(ids), vocab, dtype=out, out=torch.full((vocab, k), 5.0, dtype=out, device=DEV))
    ok = (ids >= 0) & (ids < vocab)
    rows = torch.unique(ids[ok]).long()
    small = torch.searchsorted(rows, ids.clamp(0, vocab - 1).long())
    small = torch.where(ok, small, torch.full_like(small, -1)).to(torch.int32)
    want, mag, most = ref.embed_backward(dy, small, rows.numel(), 1.0)
    ref.check(got[dev(rows)], want, most + 1, mag)
    got[dev(rows)] = 0
    assert not got.any()


def test_example_runs():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    try:
        import adapted_layer
    finally:
        sys.path.pop(0)
    first, last = adapted_layer.main(steps=6, tokens=96, quiet=True)
    assert last < first
