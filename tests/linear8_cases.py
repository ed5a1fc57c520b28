"""Inputs of the 8-bit product whose results are exact, so that nothing is
within a tolerance by being small: differences of the forward that are the
gradient to the last bit but its own rounding, and whole sums that pass 2^24
on the way to a small odd number, or end next to 2^31."""
import torch

import rows8_ref as ref

LONGEST = 131071


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


# ------------------------------------------------------------------ whole sums
def whole(t, n, device, seed=0):
    """(x8, x scales, w8, w scales, y): rows of LONGEST codes.  But for 81 places
    x is 127 or -127 and w the same, of one sign in the first half and of the
    other in the second, so a sum goes past 10^9 and back; at those places, in
    both halves, both are odd and at most 3, so what is left is odd and at
    most 729, a value of fp16.  The last token and the last channel are -128
    all over: their own sum is 2^31 - 16384, held by a scale of 2^-26."""
    g = torch.Generator().manual_seed(seed)
    half = LONGEST // 2
    few = torch.cat([torch.randperm(half, generator=g)[:40], half + torch.randperm(half, generator=g)[:40],
                     torch.tensor([LONGEST - 1])]).to(device)

    def codes(rows, turned):
        q = torch.zeros(rows, ref.stride(LONGEST), dtype=torch.int8)
        q = q.to(device)
        sign = (torch.randint(0, 2, (rows, 1), generator=g) * 2 - 1).to(device)
        q[:, :half] = (127 * sign).to(torch.int8)
        q[:, half:LONGEST] = ((-127 if turned else 127) * sign).to(torch.int8)
        odd = (torch.randint(-2, 2, (rows, 81), generator=g) * 2 + 1).to(device)
        q[:, few] = odd.to(torch.int8)
        q[-1, :LONGEST] = -128
        return q, odd.double()
    x8, xo = codes(t, False)
    w8, wo = codes(n, True)
    xs, ws = torch.ones(t, device=device), torch.ones(n, device=device)
    ws[-1] = 2.0**-26
    y = xo @ wo.t()
    y[-1, :] = -128 * w8[:, :LONGEST].double().sum(1)
    y[:, -1] = -128 * x8[:, :LONGEST].double().sum(1)
    return x8, xs, w8, ws, y * ws.double()
