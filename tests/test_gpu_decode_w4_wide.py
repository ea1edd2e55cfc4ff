"""4-bit linear layers wide enough for the tiles of several weight rows, with any K, and K below a piece."""
import pytest
import torch

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


@pytest.mark.parametrize("zeros", [False, True], ids=["z8", "zeros"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("M, N, K", [(1, 16400, 517), (3, 16400, 1030), (6, 8200, 391), (13, 16391, 645), (20, 8201, 513),
                                     (32, 9000, 2055), (40, 8200, 519), (64, 16400, 1031), (70, 8200, 256)])
def test_wide(d, M, N, K, group, dtype, zeros):
    print(f"w4 wide M={M} N={N} K={K} group={group} {dtype} zeros={zeros}", flush=True)
    t = TYPES[dtype]
    w, codes, scales, z, g = weights(N, K, group, t, zeros, M + N + K + group)
    x = torch.randn((M, K), generator=g, device=DEV).to(t)
    bias = torch.randn(N, generator=g, device=DEV).to(t) if M % 2 else None
    check(d.w4_linear(x, w.qweight, w.scales, w.zeros, n=N, group=group, bias=bias), x, codes, scales, z, group, bias)


@pytest.mark.parametrize("zeros", [False, True], ids=["z8", "zeros"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", range(1, 18))
def test_short_rows(d, K, dtype, zeros):
    """Rows about as long as the 8 columns that are read at a time, beside NaN that is not theirs."""
    t = TYPES[dtype]
    for M, N in ((1, 20), (5, 33), (40, 17)):
        w, codes, scales, z, g = weights(N, K, 32, t, zeros, 100 * K + M)
        big = torch.full((M, K + 24), float("nan"), device=DEV, dtype=t)
        x = big[:, 11:11 + K]
        x.copy_(torch.randn((M, K), generator=g, device=DEV))
        check(d.w4_linear(x, w.qweight, w.scales, w.zeros, n=N, group=32), x, codes, scales, z, 32)


@pytest.mark.parametrize("K", [129, 262, 391, 1021])
def test_nan_past_the_rows_stays_out(d, K):
    """What lies between strided rows, and after the last one, does not reach the result."""
    for M, N in ((1, 50), (7, 20), (16, 16400), (33, 8200), (64, 16400)):
        w, codes, scales, z, g = weights(N, K, 64, torch.float16, True, K + M)
        big = torch.full((M, K + 9), float("nan"), device=DEV).half()
        x = big[:, 1:1 + K]
        x.copy_(torch.randn((M, K), generator=g, device=DEV))
        check(d.w4_linear(x, w.qweight, w.scales, w.zeros, n=N, group=64), x, codes, scales, z, 64)
