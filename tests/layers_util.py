"""Helpers for the tests of the layers: guarded device tensors and the
tolerances that their float32 arithmetic allows."""

import torch

DEV = "cuda"
U32 = 2.0 ** -24                                              # unit roundoff of float32
UNIT = {torch.float32: U32, torch.bfloat16: 2.0 ** -8}        # of a stored value: half a unit of its 24 or 8 bits
GUARD = 4096                                                  # elements before and after a guarded tensor


def generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def matrix(gen, rows, cols, dtype, pad=0, offset=0, sigma=1.0, mean=0.0):
    """Normal values in a [rows, cols] view whose rows lie cols + pad apart and
    whose first element lies `offset` elements into an allocation; what lies
    between the rows is NaN, so anything computed from it shows."""
    base = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=dtype, device=DEV)
    v = base[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    v.copy_(torch.randn(rows, cols, generator=gen, device=DEV) * sigma + mean)
    return v


class Out:
    """An output of [rows, cols] inside guard elements, all NaN before the call."""

    def __init__(self, rows, cols, dtype, pad=0, offset=0):
        self.cols, self.lo = cols, GUARD + offset
        self.hi = self.lo + rows * (cols + pad)
        self.all = torch.full((self.hi + GUARD,), float("nan"), dtype=dtype, device=DEV)
        # a payload that no kernel writes
        self.bits = self.all.view(torch.int16 if dtype == torch.bfloat16 else torch.int32)
        self.mark = 0x7FA5 if dtype == torch.bfloat16 else 0x7FA5A5A5
        self.bits.fill_(self.mark)
        self.t = self.all[self.lo:self.hi].view(rows, cols + pad)[:, :cols]

    def vector(self):
        return self.t[0]

    def check(self, what):
        """Every element of the tensor was written, and nothing else was."""
        inside = torch.zeros_like(self.bits, dtype=torch.bool)
        rows, wide = self.t.shape[0], (self.hi - self.lo) // max(1, self.t.shape[0])
        inside[self.lo:self.hi].view(rows, wide)[:, :self.cols] = True
        marked = self.bits == self.mark
        assert bool(marked[~inside].all()), f"{what}: wrote outside the tensor"
        assert not bool(marked[inside].any()), f"{what}: left elements unwritten"


def within(got, want, tol, what):
    """|got - want| <= tol, elementwise; float64 want and tol."""
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: finite in other places"
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    fine = torch.isfinite(want)
    inf = ~fine & ~torch.isnan(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: another infinity"
    over = ((got - want).abs() - tol)[fine]
    if over.numel():
        assert float(over.max()) <= 0, f"{what}: {float(over.max()):.3e} over the tolerance, {int((over > 0).sum())} of {over.numel()}"
