"""The 8-bit linear layer on the GPU where its kernels and formats end: the largest
grids, exact sums, extreme scales, rounding next to ties."""
import pytest
import torch

import ref64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24           # half a step of fp32
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of the output type
F8, E8 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _bytes(t):
    return t.contiguous().view(torch.uint8).cpu()


@pytest.mark.parametrize("n", [(1 << 26) - 16, (1 << 26) - 15, (1 << 26) - 1])
def test_linear_few_rows_up_to_the_largest_grid(hip, n):
    """The last column count of the kernel for few rows (2^22 - 1 workgroups of 1024
    threads), and the first ones that take tiles. Small whole numbers: the sums are
    exact in either output type."""
    m = 3
    wc = torch.zeros((n, 128), dtype=torch.uint8, device="cuda")
    wc[:, 5] = 0x38 + (torch.arange(n, device="cuda") % 5 * 8).to(torch.uint8)  # 1, 2, 4, 8, 16
    xc = torch.zeros((m, 128), dtype=torch.uint8, device="cuda")
    xc[:, 5] = torch.tensor([0x38, 0x40, 0xC0], dtype=torch.uint8)  # 1, 2, -2
    xs = torch.full((m, 4), 127, dtype=torch.uint8, device="cuda")
    ws = torch.full(((n + 127) // 128, 4), 127, dtype=torch.uint8, device="cuda")
    y = hip.linear_fp8(xc.view(F8), xs.view(E8)[:, :1], wc.view(F8), ws.view(E8)[:, :1], y_dtype=torch.bfloat16)
    want = torch.exp2((torch.arange(n, device="cuda") % 5).float()).to(torch.bfloat16)
    assert torch.equal(y, torch.stack([want, 2 * want, -2 * want]))
