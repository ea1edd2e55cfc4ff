"""f8_linear against the product in float64 at sizes that reach each of its kernels (f8_forms)."""
import pytest
import torch

import f8_forms as forms
from drafts_ref import E4M3, check_linear, f8_values

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_f8_linear import DEV, make  # noqa: E402


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M, N, K", forms.SIZES + forms.ODD)
def test_against_the_product(d, M, N, K, dtype):
    x, xs, w, ws, b = make(M, N, K, M + N + K, dtype)
    for bias in (None, b):
        check_linear(d.f8_linear(x, xs, w, ws, bias=bias, dtype=dtype), x, xs, w, ws, bias)


@pytest.mark.parametrize("M, N, K", forms.LONG)
def test_long_rows(d, M, N, K):
    x, xs, w, ws, b = make(M, N, K, K, torch.bfloat16)
    check_linear(d.f8_linear(x, xs, w, ws, bias=b, dtype=torch.bfloat16), x, xs, w, ws, b)


@pytest.mark.parametrize("M, N, K", forms.SIZES + [(16, 400, 9000), (40, 8000, 9000), (64, 500, 9000)])
def test_whole_numbers_are_exact(d, M, N, K):
    """Sums of small whole numbers are exact, and a block, a token or a column in another's place would show."""
    gen = torch.Generator(device=DEV).manual_seed(M + K)
    pick = lambda n: torch.randint(-1, 2, (n, K), device=DEV, generator=gen).float().to(E4M3)  # noqa: E731
    kb, nb = -(-K // 128), -(-N // 128)
    pow2 = lambda *s: torch.exp2(torch.randint(-2, 3, s, device=DEV, generator=gen).float())  # noqa: E731
    x, w, xs, ws = pick(M), pick(N), pow2(M, kb), pow2(nb, kb)
    y = d.f8_linear(x, xs, w, ws, dtype=torch.bfloat16)
    assert torch.equal(y, (f8_values(x, xs) @ f8_values(w, ws).t()).float().bfloat16())


@pytest.mark.parametrize("M, N, K", [(512, 4096, 272), (4096, 4096, 400), (1024, 4096, 272), (2048, 4096, 272)])
def test_rows_apart_with_nan_between(d, M, N, K):
    x, xs, w, ws, b = make(M, N, K, 3)
    want = d.f8_linear(x, xs, w, ws, bias=b)
    room = [torch.full((r, K + 32), 0x7f, dtype=torch.uint8, device=DEV) for r in (M, N)]
    for to, of in zip(room, (x, w)):
        to[:, 16:16 + K] = of.view(torch.uint8)
    out = torch.full((M, N + 8), 3.0, device=DEV).half()
    y = d.f8_linear(room[0].view(E4M3)[:, 16:16 + K], xs, room[1].view(E4M3)[:, 16:16 + K], ws, bias=b, out=out[:, :N])
    assert torch.equal(y, want) and torch.all(out[:, N:] == 3)
