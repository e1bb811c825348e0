"""Size queries of the 8-bit linear layer, on the CPU: 0 bytes for what the calls refuse;
refusals of the norm's eps."""
import pytest


@pytest.fixture(scope="module")
def L():
    import os

    from bit_block_float_amd import build, hif4
    if not os.path.exists(hif4.LIB_PATH):
        build.build()
    return hif4.lib()


@pytest.mark.parametrize("m,n,k", [(100, 100, 64), (300, 300, 1), (300, 300, 64), (300, 300, 127), (300, 300, 4200),
                                   (300, 700, 13825), (1, 1, 64), (5120, 5120, 5119), (1 << 30, 1 << 30, 128),
                                   (1 << 19, 1 << 19, 128), (128, (1 << 31) - 1, 128)])
def test_a_refused_product_needs_no_workspace(L, m, n, k):
    a = 0x100000  # never dereferenced
    assert L.hif4_linear_fp8(a, a, 1 << 16, a, a, 1 << 16, 0, 128, m, n, k, a, 0, a, 1 << 50, None) == 2  # shape
    assert L.hif4_linear_fp8_workspace_bytes(m, n, k) == 0


def test_a_split_product_needs_its_planes(L):
    parts = L.hif4_linear_fp8_workspace_bytes(300, 700, 13824) / (300 * 700 * 4)
    assert parts == int(parts) and 2 <= parts <= 13824 // 128
    assert L.hif4_linear_fp8_workspace_bytes(300, 700, 128) == 0
    assert L.hif4_linear_fp8_workspace_bytes(300, 700, 0) == 0


@pytest.mark.parametrize("eps", [3.5e38, 1e39, 1e300])
def test_norm_refuses_an_eps_beyond_float(L, eps):
    a = 0x100000  # never dereferenced
    assert L.hif4_layer_norm(a, 0, 4, 8, 8, a, a, 0, eps, a, 8, a, a, None) == 8
    assert L.hif4_layer_norm_quantize(a, 0, 4, 64, 64, a, a, 0, eps, None, 0, None, a, a, None) == 8
    assert L.hif4_layer_norm_quantize_fp8(a, 0, 4, 8, 8, a, a, 0, eps, a, a, 4, None) == 8


def test_binding_refuses_a_workspace_that_is_not_contiguous():
    """An expanded tensor has the elements, but not the memory."""
    import torch

    from bit_block_float_amd import hif4
    assert hif4._workspace_bytes(torch.empty(300)) == 1200
    for t in (torch.empty(1, dtype=torch.uint8).expand(1 << 20), torch.empty((8, 8)).T[1:]):
        with pytest.raises(ValueError):
            hif4._workspace_bytes(t)


@pytest.mark.gpu
def test_calls_refuse_a_workspace_that_is_not_contiguous(hip):
    import torch
    wide = torch.empty(1, dtype=torch.uint8, device="cuda").expand(1 << 28)
    x, w = torch.ones((300, 4224), device="cuda"), torch.ones((96, 4224), device="cuda")
    xq, wq = hip.quantize_fp8(x), hip.quantize_fp8(w, block_rows=128)
    assert hip.linear_fp8_workspace_bytes(300, 96, 4224) > 0
    with pytest.raises(ValueError):
        hip.linear_fp8(*xq, *wq, workspace=wide)
    xt, wt = hip.quantize_fp8(x, transposed=True), hip.quantize_fp8(w, block_rows=128, transposed=True)
    with pytest.raises(ValueError):
        hip.linear_fp8_backward(torch.ones((300, 96), device="cuda"), *xt, *wt, workspace=wide)
    _, mean, rstd = hip.layer_norm(x)
    with pytest.raises(ValueError):
        hip.layer_norm_backward(x, x, mean, rstd, workspace=wide)
