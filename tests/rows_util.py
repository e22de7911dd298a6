"""Plain fp64 forms of the row operators (embedding, expert sort / gather / combine, low-rank adapters)
on CPU tensors, and the tolerance that the library's results are held to.

Tolerance: the library multiplies and adds in fp32 in an order of its own and rounds once at the
store.  A sum of m products taken in fp32 in any order is off by at most (m + 2) * 2^-24 times the sum
of the products' magnitudes (two roundings a term, one of them shared), and the store by half a step
of the output type (and half of the smallest fp16 step).
"""
import torch

U32 = 2.0 ** -24


def check(got, want, terms, magnitude, what=""):
    """got: the library's tensor; want: fp64; terms: products in the longest sum; magnitude: fp64 sum
    of the magnitudes of the terms (want's shape)."""
    assert got.shape == want.shape, (what, got.shape, want.shape)
    g = got.detach().cpu().double()
    err32 = (terms + 2) * U32 * magnitude
    step = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    floor = 2.0 ** -25 if got.dtype == torch.float16 else 1e-38
    bound = err32 + step * (want.abs() + err32) + floor
    bad = ~((g - want).abs() <= bound)
    if bad.any():
        i = tuple(int(v) for v in torch.nonzero(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; at {i} got {g[i]:.9g}, want "
                             f"{want[i]:.9g}, bound {bound[i]:.3g}")


def sort_ids(ids, n_keys):
    flat = [int(v) for v in ids.flatten()]
    valid = [i for i, v in enumerate(flat) if 0 <= v < n_keys]
    order = sorted(valid, key=lambda i: (flat[i], i)) + [i for i, v in enumerate(flat) if not 0 <= v < n_keys]
    pos = [-1] * len(flat)
    for p, i in enumerate(order[:len(valid)]):
        pos[i] = p
    counts = torch.zeros(n_keys, dtype=torch.int64)
    if valid:
        counts.index_add_(0, torch.tensor([flat[i] for i in valid]), torch.ones(len(valid), dtype=torch.int64))
    bounds = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    return (torch.tensor(order, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32).view(ids.shape),
            bounds.to(torch.int32))


def combine(h, pos, weights, base):
    """(fp64 result, magnitude): h [pairs, k], pos [n, top_k]."""
    n, top_k = pos.shape
    y = torch.zeros((n, h.shape[1]), dtype=torch.float64)
    m = torch.zeros_like(y)
    for t in range(n):
        for j in range(top_k):
            p = int(pos[t, j])
            if 0 <= p < n * top_k:
                w = 1.0 if weights is None else float(weights[t, j])
                y[t] += w * h[p].double()
                m[t] += abs(w) * h[p].double().abs()
    if base is not None:
        y += base.double()
        m += base.double().abs()
    return y, m


def combine_backward(dy, h, pos, weights):
    n, top_k = pos.shape
    dh = torch.zeros(h.shape, dtype=torch.float64)
    dw = torch.zeros((n, top_k), dtype=torch.float64)
    mw = torch.zeros_like(dw)
    for t in range(n):
        for j in range(top_k):
            p = int(pos[t, j])
            if 0 <= p < n * top_k:
                dh[p] = (1.0 if weights is None else float(weights[t, j])) * dy[t].double()
                dw[t, j] = (dy[t].double() * h[p].double()).sum()
                mw[t, j] = (dy[t].double() * h[p].double()).abs().sum()
    return dh, dw, mw


def embed_backward(dy, ids, vocab, scale):
    """(fp64 result, magnitude, most rows of one id)."""
    flat, d = ids.flatten().long(), dy.reshape(ids.numel(), dy.shape[-1]).double()
    ok = (flat >= 0) & (flat < vocab)
    g = torch.zeros((vocab, d.shape[1]), dtype=torch.float64)
    m = torch.zeros_like(g)
    g.index_add_(0, flat[ok], d[ok])
    m.index_add_(0, flat[ok], d[ok].abs())
    most = int(torch.bincount(flat[ok], minlength=1).max()) if ok.any() else 0
    return g * scale, m * abs(scale), most


def lora(x, a, b, ids, scale, base):
    """fp64 (y, its magnitude, h, its magnitude)."""
    n, rows, rank = x.shape[0], b.shape[1], a.shape[1]
    y = torch.zeros((n, rows), dtype=torch.float64) if base is None else base.double().clone()
    my, h = y.abs(), torch.zeros((n, rank), dtype=torch.float64)
    mh = torch.zeros_like(h)
    for c in range(a.shape[0]):
        at = torch.nonzero(ids == c)[:, 0]
        if at.numel() == 0:
            continue
        s = 1.0 if scale is None else float(scale[c])
        xa, aa, bb = x[at].double(), a[c].double(), b[c].double()
        h[at], mh[at] = xa @ aa.t(), xa.abs() @ aa.abs().t()
        y[at] += s * (h[at] @ bb.t())
        my[at] += abs(s) * (mh[at] @ bb.abs().t())
    return y, my, h, mh


def lora_backward(x, dy, h, a, b, ids, scale, dx_base):
    """fp64 (dx, da, db) and their magnitudes; most rows of one adapter."""
    dx = torch.zeros(x.shape, dtype=torch.float64) if dx_base is None else dx_base.double().clone()
    mx = dx.abs()
    da, db = torch.zeros(a.shape, dtype=torch.float64), torch.zeros(b.shape, dtype=torch.float64)
    ma, mb, most = torch.zeros_like(da), torch.zeros_like(db), 0
    for c in range(a.shape[0]):
        at = torch.nonzero(ids == c)[:, 0]
        if at.numel() == 0:
            continue
        most = max(most, at.numel())
        s = 1.0 if scale is None else float(scale[c])
        xa, d, aa, bb, hh = x[at].double(), dy[at].double(), a[c].double(), b[c].double(), h[at].double()
        dh, mdh = s * (d @ bb), abs(s) * (d.abs() @ bb.abs())
        dx[at] += dh @ aa
        mx[at] += mdh @ aa.abs()
        da[c], ma[c] = dh.t() @ xa, mdh.t() @ xa.abs()
        db[c], mb[c] = s * (d.t() @ hh), abs(s) * (d.abs().t() @ hh.abs())
    return (dx, da, db), (mx, ma, mb), most
