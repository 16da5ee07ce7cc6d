"""Inputs and references shared by the tests of the experts' products, the
gated sum and the gradient calls.

Inputs sit in the middle of a NaN-filled allocation, so a read outside them
shows in the result; outputs sit between guard bytes that must survive."""
import numpy as np

GUARD = 4096  # bytes on each side

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # largest relative error of one rounding


def tdtype(dt):
    import torch
    return torch.float32 if dt == "f32" else torch.bfloat16


def inside_nan(t, offset_elements=0):
    """A copy of t whose allocation continues with NaN on both sides."""
    import torch
    g = GUARD // t.element_size()
    whole = torch.full((2 * g + t.numel() + offset_elements,), float("nan"), dtype=t.dtype, device="cuda")
    body = whole[g + offset_elements:g + offset_elements + t.numel()]
    body.copy_(t.reshape(-1))
    return body.view(t.shape)


class Guarded:
    """An output buffer of `shape`, filled with `fill`, between guards."""

    def __init__(self, shape, dtype, fill=float("nan"), offset_elements=0):
        import torch
        n = int(np.prod(shape))
        es = torch.empty(0, dtype=dtype).element_size()
        self.whole = torch.full((2 * GUARD + (n + offset_elements) * es,), 0xA5, dtype=torch.uint8,
                                device="cuda")
        lo = GUARD + offset_elements * es
        self.lo, self.hi = lo, lo + n * es
        self.t = self.whole[lo:self.hi].view(dtype).view(shape)
        self.t.fill_(fill)

    def intact(self):
        return bool((self.whole[:self.lo] == 0xA5).all()) and bool((self.whole[self.hi:] == 0xA5).all())


def counts_of(rows, R, E, rng):
    """[R, E] counts whose column sums are rows[e], split over the ranks."""
    out = np.zeros((R, E), np.int64)
    for e, n in enumerate(rows):
        out[:, e] = rng.multinomial(int(n), np.full(R, 1.0 / R))
    return out


def experts_ref(op, xs, ws, rows, R, E):
    """fp64 results and, per element, the sum of the products' magnitudes:
    lists per rank.  op "product": xs rows, ws weights; "dgrad": xs = dout;
    "wgrad": xs = dout rows, ws = x rows."""
    import torch
    eloc = E // R
    res, mag = [], []
    for d in range(R):
        at, parts, mags = 0, [], []
        for l in range(eloc):
            n = int(rows[d * eloc + l])
            x = xs[d][at:at + n].double()
            if op == "wgrad":
                y = ws[d][at:at + n].double()
                parts.append((x.t() @ y)[None])
                mags.append((x.abs().t() @ y.abs())[None])
            else:
                w = ws[d][l].double()
                w = w.t() if op == "product" else w
                parts.append(x @ w)
                mags.append(x.abs() @ w.abs())
            at += n
        res.append(torch.cat(parts))
        mag.append(torch.cat(mags))
    return res, mag
