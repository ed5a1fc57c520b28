"""Inputs of the 8-bit product whose results are exact, so that nothing is
within a tolerance by being small: differences of the forward that are the
gradient to the last bit but its own rounding."""
import torch

import rows8_ref as ref


# ----------------------------------------------------------------- differences
def small(t, k, n, device, seed=0):
    """(x8, x scales, w8, w scales, dy): codes of [-3, 3], scales 2^-2 to 2^2 and
    dy in quarters up to 2.  With k up to 227 every y, also with a code one
    larger in each row, is a whole number below 2^11 times a power of two: a
    value of fp16 (with k up to 28 below 2^8: of bf16).  A gradient's products
    are multiples of 2^-4 below 24, so its fp32 sums are exact, and below
    fp16's largest number for up to 2700 of them."""
    g = torch.Generator().manual_seed(seed)

    def held(rows):
        q = torch.zeros(rows, ref.stride(k), dtype=torch.int8)
        q[:, :k] = torch.randint(-3, 4, (rows, k), generator=g)
        return q.to(device), torch.exp2(torch.randint(-2, 3, (rows,), generator=g).float()).to(device)
    x8, xs = held(t)
    w8, ws = held(n)
    return x8, xs, w8, ws, (torch.randint(-8, 9, (t, n), generator=g) / 4.0).to(device)


def differences(forward, x8, xs, w8, ws, dy, k):
    """(d/dx, d/dw) in fp64 of sum(dy y) by what `forward()` says when the codes
    of one column are each one larger: a token's change is its own row's of y,
    a channel's its own column's."""
    dy, base = dy.double(), forward().double()
    out = []
    for codes, scale, along in ((x8, xs, 1), (w8, ws, 0)):
        d = torch.empty(codes.shape[0], k, dtype=torch.float64, device=codes.device)
        for col in range(k):
            codes[:, col] += 1
            d[:, col] = (dy * (forward().double() - base)).sum(along) / scale.double()
            codes[:, col] -= 1
        out.append(d)
    return out
