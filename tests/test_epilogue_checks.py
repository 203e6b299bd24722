"""awq_gemm_fused's argument checks, on the host (fake device addresses are
never dereferenced: every call fails before a launch or has nothing to do)."""

import pytest

import weight_only_int4_quantize_amd as awq

OK, NULL, SHAPE, ALIGN, CONFIG, WORKSPACE = 0, 1, 2, 3, 4, 5
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    return awq.load()


def call(L, x=FAKE, qw=FAKE, sc=FAKE, zr=FAKE, M=4, N=16, K=256, G=128, bits=4, bias=FAKE, act=2, mul=FAKE, ms=16,
         res=FAKE, rs=16, y=FAKE, path=0, ws=None, nbytes=0):
    return L.awq_gemm_fused(x, qw, sc, zr, M, N, K, G, bits, bias, act, mul, ms, res, rs, y, path, ws, nbytes, None)


@pytest.mark.parametrize("bits", [4, 8])
def test_fused_checks(L, bits):
    bad = [(dict(bits=3), CONFIG), (dict(bits=16), CONFIG), (dict(act=-1), CONFIG), (dict(act=5), CONFIG),
           (dict(ms=15), SHAPE), (dict(rs=15), SHAPE), (dict(ms=-1), SHAPE), (dict(rs=2 ** 31), SHAPE),
           (dict(bias=FAKE + 1), ALIGN), (dict(mul=FAKE + 1), ALIGN), (dict(res=FAKE + 1), ALIGN),
           (dict(x=None), NULL), (dict(qw=None), NULL), (dict(sc=None), NULL), (dict(zr=None), NULL), (dict(y=None), NULL),
           (dict(x=FAKE + 8), ALIGN), (dict(qw=FAKE + 8), ALIGN), (dict(y=FAKE + 1), ALIGN),
           (dict(G=96), CONFIG), (dict(K=200), SHAPE), (dict(M=-1), SHAPE), (dict(N=-1), SHAPE), (dict(path=9), CONFIG),
           (dict(path=1, M=9), CONFIG), (dict(M=200, ws=FAKE + 64, nbytes=1 << 30), ALIGN),
           (dict(M=200, ws=FAKE, nbytes=256), WORKSPACE)]
    for kw, expect in bad:
        assert call(L, **{"bits": bits, **kw}) == expect, kw
    assert call(L, bits=8, G=32) == CONFIG          # W8 groups are 64 and more
    assert call(L, bits=8, path=3) == CONFIG        # and its kernels two
    assert call(L, bits=bits, M=0) == OK and call(L, bits=bits, N=0) == OK
    # strides of absent operands do not matter
    assert call(L, bits=bits, M=0, mul=None, ms=0, res=None, rs=-4) == OK


def test_binding_checks():
    torch = pytest.importorskip("torch")
    t = torch.zeros(2, 256, dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU tensor"):
        awq.awq_gemm_fused(t, t, t, t)
    with pytest.raises(TypeError):
        awq.awq_gemm_fused([1.0], t, t, t)
