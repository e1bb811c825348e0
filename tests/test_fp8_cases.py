"""That the product's inputs tell what they are meant to, on the CPU."""
import pytest
import torch

import fp8_cases


@pytest.mark.parametrize("k", [256, 512, 4224, 5120])
def test_a_cut_product_would_be_seen(k):
    x, w = fp8_cases.cancelling(5, 7, k)
    xv, wv = fp8_cases.values(x), fp8_cases.values(w)
    want = xv @ wv.T
    # multiples of 2^-7 whose sums, run by run, stay below 2^17: exact in fp32
    p = (xv[:, None] * wv[None]).reshape(5, 7, -1, 8)
    assert torch.equal(p * 128, torch.round(p * 128)) and float(p[..., 2:].abs().max()) <= 0.5
    assert float(want.max()) + 2 ** 16 < 2 ** 17
    in_runs = p.float().cumsum(3)
    assert torch.equal(in_runs.double(), p.cumsum(3))
    assert torch.equal(in_runs[..., -1].cumsum(2)[..., -1].double(), want)
    # the cut loses every small product: nothing is left
    assert bool((fp8_cases.cut_product(xv, wv) == 0).all()) and float(want.min()) > 0


def test_the_cut_on_ordinary_products():
    """On random signs it is far below a bf16 result's rounding."""
    g = torch.Generator().manual_seed(2)
    xv, wv = (torch.randint(-15, 16, (4, 4096), generator=g).double() for _ in range(2))
    d = (fp8_cases.cut_product(xv, wv) - xv @ wv.T).abs()
    assert bool((d <= 7 * 2.0 ** -13 * (xv.abs() @ wv.abs().T)).all())
