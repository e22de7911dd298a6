"""Inputs of the adapters for which every element of every result is one chain of products, and the bound that
such a chain is held to.

The library multiplies fp32 operands as sums of three bf16 parts, each the next eight significant bits: up to
eight products of parts, exact in fp32 and of one sign, added one at a time.  Each addition is off by at most a
step, 2^-23 of the product, whichever way the matrix unit rounds; the left-out product of two third parts is below
2^-32 of it.  That makes 17 * 2^-24 a product.  A chain has at most two products and the scale's rounding: 35,
and the last store's one more.  A product that keeps two parts of an operand is off by up to 2^-16, 256 such units.
"""
import torch

SINGLE_TERMS = 34   # rows_util.check adds two to it


def inputs(seed, n, k, rows, rank, na, xt, wt):
    """x, a, b, ids, scale, dy: values of full significands between 1 and 2 (and their negatives), rows of x and dy
    with one value each, in columns of its own among its adapter's rows; an adapter's b has one value in each
    row."""
    g = torch.Generator()
    g.manual_seed(seed)

    def values(*shape):
        v = 1 + torch.rand(shape, generator=g)
        return torch.where(torch.rand(shape, generator=g) < 0.5, v, -v)

    ids = torch.randint(0, na, (n,), generator=g, dtype=torch.int32)
    x, dy = torch.zeros((n, k)), torch.zeros((n, rows))
    for c in range(na):
        at = torch.nonzero(ids == c)[:, 0]
        assert at.numel() <= min(k, rows)
        x[at, torch.randperm(k, generator=g)[:at.numel()]] = values(at.numel())
        dy[at, torch.randperm(rows, generator=g)[:at.numel()]] = values(at.numel())
    a, b = values(na, rank, k), torch.zeros((na, rows, rank))
    own = torch.randint(0, rank, (na, rows, 1), generator=g)
    b.scatter_(2, own, values(na, rows, 1))
    return x.to(xt), a.to(wt), b.to(wt), ids, 1 + torch.rand(na, generator=g), dy.to(xt)
