"""Which kernel a fused call runs (awq_gemm_fused_kernel, host only): the
plain call's choice, but the GEMM's small tiles where the plain call takes the
skinny kernel above 32 rows, and for a few hundred rows."""

import pytest

import weight_only_int4_quantize_amd as awq


@pytest.fixture(scope="module", autouse=True)
def cu256():
    import torch
    if torch.cuda.is_available() and torch.cuda.get_device_properties(0).multi_processor_count != 256:
        pytest.skip("the sizes are a 256-CU device's")


@pytest.mark.parametrize("M,N,K,G,bits,path,ws,kernel", [
    (1, 4096, 4096, 128, 4, 0, True, "gemv"),
    (16, 4096, 4096, 128, 4, 0, True, "coltile"),
    (12, 8192, 28672, 128, 4, 0, True, "skinny"),
    (64, 4096, 4096, 128, 4, 0, True, "gemm_small"),       # the plain call: skinny
    (64, 4096, 4096, 128, 4, 3, True, "skinny"),
    (40, 700, 4096, 256, 4, 0, False, "gemm_small"),
    (40, 700, 4096, 32, 4, 0, True, "skinny"),              # groups of 32 have no small tiles
    (200, 512, 4096, 32, 4, 0, True, "gemm"),
    (200, 512, 4096, 128, 4, 2, True, "gemm_small"),
    (2048, 11008, 4096, 128, 4, 0, True, "gemm"),
    (1500, 4000, 2048, 128, 4, 0, True, "gemm_small"),     # 768 tiles of 32 steps
    (1500, 4000, 2048, 128, 4, 0, False, "gemm"),          # without a workspace up to one round of them
    (1, 1000, 4096, 128, 8, 0, False, "gemv"),
    (8, 1000, 4096, 128, 8, 2, False, "gemm_small"),
    (203, 1000, 4096, 64, 8, 0, True, "gemm_small"),
    (2048, 11008, 4096, 64, 8, 0, True, "gemm"),
])
def test_choice(M, N, K, G, bits, path, ws, kernel):
    assert awq.gemm_fused_kernel(M, N, K, G, bits, path, ws) == kernel


def test_invalid():
    for args in ((0, 64, 256, 128), (4, 0, 256, 128), (4, 64, 200, 128), (4, 64, 256, 96), (4, 64, 256, 128, 3),
                 (9, 64, 256, 128, 4, 1), (4, 64, 256, 128, 4, 5), (4, 64, 256, 32, 8), (4, 64, 256, 128, 8, 3),
                 (65, 64, 256, 128, 4, 3), (9, 64, 1 << 23, 128, 8)):
        with pytest.raises(awq.AwqError):
            awq.gemm_fused_kernel(*args)


def test_plain_choice_is_as_it_was():
    assert awq.gemm_kernel(64, 4096, 4096, 128, workspace=True) == "skinny"
    assert awq.gemm_kernel(200, 512, 4096, 128, workspace=True) == "gemm"
