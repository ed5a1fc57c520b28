"""The exact cases of the 8-bit product are what they are meant to be: the
definition passes them, and a definition with a mistake planted in it does
not.  On the CPU."""
import pytest
import torch

import linear8_cases as cases
import rows8_ref as ref


def gradients(x8, xs, w8, ws, dy, k):
    return dy.double() @ ref.values(w8, ws, k), dy.double().t() @ ref.values(x8, xs, k)


@pytest.mark.parametrize("size,dtype", [((40, 60, 50), torch.float16), ((20, 227, 30), torch.float16),
                                        ((30, 28, 45), torch.bfloat16)], ids=str)
def test_differences_are_the_gradient_and_no_other(size, dtype):
    t, k, n = size
    x8, xs, w8, ws, dy = cases.small(t, k, n, "cpu")

    def forward():
        y = ref.linear(x8, xs, w8, ws, k, None)[0]
        assert torch.equal(y.to(dtype).double(), y), "y is no value of the type"
        return y.to(dtype)
    far = cases.differences(forward, x8, xs, w8, ws, dy, k)
    for got, want in zip(gradients(x8, xs, w8, ws, dy, k), far):
        assert torch.equal(got, want) and float(want.abs().median()) > 1
        right = got.to(dtype).double()
        ref.within(right, want, ref.half_step(want, dtype))
        later = want.abs().gt(1).nonzero()[-1].tolist()
        wrong = [torch.zeros_like(right), -right, right.roll(1, 1), right.roll(1, 0), right * (1 + 2.0**-6), right.clone()]
        wrong[-1][later[0], later[1]] *= 1.02
        for w in wrong:
            with pytest.raises(AssertionError):
                ref.within(w, want, ref.half_step(want, dtype))


def test_no_fp32_sum_gives_the_whole_sums():
    x8, xs, w8, ws, y = cases.whole(5, 6, "cpu")
    k = cases.LONGEST
    x, w = x8[:, :k].long(), w8[:, :k].long()
    exact = (x.unsqueeze(1) * w).sum(2)
    assert torch.equal(exact.double() * ws.double(), y)
    assert bool((exact[:-1, :-1] % 2 != 0).all()) and int(exact[:-1, :-1].abs().max()) <= 729
    assert torch.equal(y[:-1, :-1].half().double(), y[:-1, :-1])
    assert int(exact[-1, -1]) == 2**31 - 16384
    # sums of 64 products, exact, added up in fp32, front to back and by four
    wide = torch.zeros(5, 6, ref.stride(k), dtype=torch.long)
    wide[:, :, :k] = x.unsqueeze(1) * w
    steps = wide.view(5, 6, -1, 64).sum(3).float()
    assert float(steps.cumsum(2).abs().max()) > 2.0**29
    assert int(torch.iinfo(torch.int32).max) >= int(wide.cumsum(2).abs().max())
    for lanes in (1, 4):
        total = torch.zeros(5, 6)
        for lane in range(lanes):
            own = torch.zeros(5, 6)
            for i in range(lane, steps.shape[2], lanes):
                own = own + steps[:, :, i]
            total = total + own
        wrong = (total.double() * ws.double() != y)[:-1, :-1]
        assert float(wrong.double().mean()) > 0.5
