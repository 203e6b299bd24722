"""The GEMV's support check counts the LDS of the rows its streaming form
parks beside the staged x: shapes whose staged x alone fills the LDS go to
another kernel instead of failing at the launch."""

import numpy as np
import pytest

import weight_only_int4_quantize_amd as awq


def test_kernel_choice_at_the_lds_limit():
    """Host only (256 CUs, 160 KB): at K = 10240 and M = 7 the staged x of an
    INT4 layer takes 161280 of 163840 bytes, which leaves room for the sums of
    80 rows per block, not of 96."""
    import torch
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are a 256-CU device's")
    assert awq.gemm_kernel(7, 20480, 10240, 512, awq.PATH_GEMV) == "gemv"
    with pytest.raises(awq.AwqError):
        awq.gemm_kernel(7, 24576, 10240, 512, awq.PATH_GEMV)
    assert awq.gemm_kernel(7, 24576, 10240, 512) == "gemm"


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,G", [(8, 513, 8192, 256), (8, 40000, 8192, 64)])
def test_w8_at_the_lds_limit(M, N, K, G):
    """M = 8 at K = 8192: the staged x is the whole LDS."""
    torch = pytest.importorskip("torch")
    g = torch.Generator(device="cuda").manual_seed(5)
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).half()
    x = torch.randn(M, K, generator=g, device="cuda").half()
    q, s, z = awq.awq_quantize_w8(w, G)
    y = awq.awq_gemm_w8(x, q, s, z, G).double().cpu().numpy()
    b = torch.stack([(q >> (8 * j)) & 255 for j in range(4)], -1).flatten(1).double()
    wq = (b - z.double().repeat_interleave(G, 1)) * s.double().repeat_interleave(G, 1)
    ref = (x.double() @ wq.t().contiguous()).cpu().numpy()
    assert np.linalg.norm(y - ref) / np.linalg.norm(ref) <= 1e-3


@pytest.mark.gpu
@pytest.mark.parametrize("N", [20480, 24576])
def test_int4_at_the_lds_limit(N):
    torch = pytest.importorskip("torch")
    M, K, G = 7, 10240, 512
    g = torch.Generator(device="cuda").manual_seed(6)
    w = (torch.randn(N, K, generator=g, device="cuda") * 0.02).half()
    x = torch.randn(M, K, generator=g, device="cuda").half()
    q, s, z = awq.awq_quantize(w, G)
    y = awq.awq_gemm(x, q, s, z, G).double()
    c = torch.stack([(q >> (4 * j)) & 15 for j in range(8)], -1).flatten(1).float()
    wq = (c - z.float().repeat_interleave(G, 1)) * s.float().repeat_interleave(G, 1)
    ref = x.float() @ wq.t().contiguous()
    assert float((y - ref).norm() / ref.norm()) <= 1e-3
