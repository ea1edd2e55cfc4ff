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
