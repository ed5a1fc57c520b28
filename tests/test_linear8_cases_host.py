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
