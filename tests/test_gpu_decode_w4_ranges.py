"""4-bit linear layers at the ends of what their arguments may hold: far rows, infinities, large numbers."""
import math

import pytest
import torch

from decode_ref import F

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_decode_w4 import DEV, TYPES, check, weights  # noqa: E402


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


@pytest.mark.parametrize("M, ldx", [(65, 1 << 25), (200000, 11008)])
def test_rows_over_four_gib(d, M, ldx):
    """The same rows far apart and close together give the same bits."""
    w, codes, scales, z, g = weights(32, 256, 64, torch.float16, True, 37)
    x = torch.randn((M, 256), generator=g, device=DEV).half()
    far = torch.empty((M - 1) * ldx + 256, dtype=torch.float16, device=DEV).as_strided((M, 256), (ldx, 1))
    far.copy_(x)
    close = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=32, group=64)
    check(close, x, codes, scales, z, 64)
    assert torch.equal(d.w4_linear(far, w.qweight, w.scales, w.zeros, n=32, group=64), close)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M, K, group", [(1, 256, 64), (5, 200, 32), (20, 256, 128), (40, 1000, 96), (70, 64, 64)])
def test_infinite_inputs_keep_their_sign(d, M, K, group, dtype):
    """What a sum over an infinite x is, by value: infinite where the weight is not 0, NaN where it is."""
    t = TYPES[dtype]
    w, codes, scales, z, g = weights(100, K, group, t, True, 53)
    x = torch.randn((M, K), generator=g, device=DEV).to(t)
    clean = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=100, group=group)
    x[0, K // 3] = math.inf
    x[M - 1, K - 1] = -math.inf
    y = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=100, group=group)
    col = torch.arange(K, device=DEV) // group
    full = ((codes - z[:, col]).to(F) * scales.to(F)[:, col])
    for m in {0, M - 1}:
        want = (x[m].to(F)[None] * full).sum(1)
        assert torch.allclose(y[m].to(F), want, rtol=0, atol=0, equal_nan=True)
    keep = [m for m in range(M) if m not in (0, M - 1)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("M", [1, 12, 33])
def test_large_finite_inputs(d, M):
    """bf16 inputs near the type's end, whose sums fit although 16 times their terms would not."""
    w, codes, scales, z, g = weights(80, 512, 64, torch.bfloat16, True, 59)
    x = torch.randn((M, 512), generator=g, device=DEV)
    x[:, ::64] *= 3e37
    x = x.bfloat16()
    check(d.w4_linear(x, w.qweight, w.scales, w.zeros, n=80, group=64), x, codes, scales, z, 64)
