"""f8_linear on the GPU against the product in float64."""
import math

import pytest
import torch

from decode_ref import F
from drafts_ref import E4M3, check_linear, f8_values

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


def codes(shape, gen):
    return (torch.randn(shape, device=DEV, generator=gen) * 120).clamp(-448, 448).to(E4M3)


def make(M, N, K, seed, dtype=torch.float16):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kb = -(-K // 128)
    around = lambda shape, mid: torch.exp(torch.randn(shape, device=DEV, generator=gen) * 0.5) * mid  # noqa: E731
    return (codes((M, K), gen), around((M, kb), 1 / 120), codes((N, K), gen), around((-(-N // 128), kb), max(K, 1) ** -0.5 / 120),
            torch.randn(N, device=DEV, generator=gen).to(dtype))


SIZES = [
    (1, 1, 16), (1, 64, 128), (1, 130, 144), (1, 4096, 4096), (2, 300, 272), (16, 257, 1024), (17, 128, 400), (31, 1000, 640),
    (33, 257, 2048), (64, 500, 1040), (65, 128, 128), (66, 129, 144), (77, 5003, 4072), (100, 300, 4096), (127, 255, 272),
    (128, 128, 256), (129, 260, 384), (200, 1536, 2048), (256, 256, 2048), (257, 700, 4096), (511, 1030, 528), (600, 4096, 256),
    (1025, 520, 1152), (300, 14000, 260), (1100, 4000, 136), (2100, 4100, 400), (10, 9000, 300), (30, 9000, 268), (60, 9000, 1028),
    (70, 8000, 392), (90, 300, 4092), (600, 9000, 140), (1, 300, 17), (3, 40, 33), (20, 200, 1001), (70, 300, 515), (300, 140, 999), (5, 70, 1), (40, 9, 15),
]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M, N, K", SIZES)
def test_against_the_product(d, M, N, K, dtype):
    x, xs, w, ws, b = make(M, N, K, M + N + K, dtype)
    for bias in (None, b):
        y = d.f8_linear(x, xs, w, ws, bias=bias, dtype=dtype)
        assert y.shape == (M, N) and y.dtype == dtype
        check_linear(y, x, xs, w, ws, bias)


@pytest.mark.parametrize("M, N, K", [(2048, 4096, 4096), (3000, 2300, 1104), (4099, 4100, 640)])
def test_large(d, M, N, K):
    x, xs, w, ws, b = make(M, N, K, 5, torch.bfloat16)
    check_linear(d.f8_linear(x, xs, w, ws, bias=b, dtype=torch.bfloat16), x, xs, w, ws, b)


@pytest.mark.parametrize("M", [1, 16, 40, 130, 700])
def test_whole_numbers_are_exact(d, M):
    """Small whole numbers and scales of powers of two: every sum is exact, and so is each result."""
    gen = torch.Generator(device=DEV).manual_seed(M)
    N, K = 520, 896
    pick = lambda n: torch.randint(-4, 5, (n, K), device=DEV, generator=gen).float()  # noqa: E731
    x, w = pick(M), pick(N)
    pow2 = lambda *s: torch.exp2(torch.randint(-2, 3, s, device=DEV, generator=gen).float())  # noqa: E731
    xs, ws = pow2(M, 7), pow2(5, 7)
    y = d.f8_linear(x.to(E4M3), xs, w.to(E4M3), ws, dtype=torch.bfloat16)
    want = (f8_values(x.to(E4M3), xs) @ f8_values(w.to(E4M3), ws).t()).float().bfloat16()
    assert torch.equal(y, want)


@pytest.mark.parametrize("M", [1, 24, 64, 200, 900])
def test_every_column_counts_once(d, M):
    """One column of one token after the other is not zero, and meets its own weight column."""
    K, N = 272, 144
    x = torch.zeros((M, K), device=DEV)
    for i in range(M):
        x[i, (7 * i + 3) % K] = 1
    w = ((torch.arange(K, device=DEV)[None] + torch.arange(N, device=DEV)[:, None]) % 15).float()
    y = d.f8_linear(x.to(E4M3), torch.ones((M, 3), device=DEV), w.to(E4M3), torch.ones((2, 3), device=DEV))
    assert torch.equal(y, (x @ w.t()).half())


@pytest.mark.parametrize("M, N, K", [(3, 200, 300), (40, 300, 256), (150, 260, 272), (600, 300, 384)])
def test_strides_and_places(d, M, N, K):
    """Rows apart, at places that are no multiple of 16 bytes, and what lies between them stays."""
    x, xs, w, ws, b = make(M, N, K, K)
    kb, nb = xs.shape[1], ws.shape[0]

    def within(t, at, more, fill):
        big = torch.full((t.shape[0], t.shape[1] + at + more), fill, device=DEV, dtype=t.dtype if t.dtype != E4M3 else torch.uint8)
        view = big[:, at:at + t.shape[1]]
        view.copy_(t if t.dtype != E4M3 else t.view(torch.uint8))
        return big, view.view(t.dtype) if t.dtype != E4M3 else big.view(E4M3)[:, at:at + t.shape[1]]

    for at, more in ((0, 16), (16, 32), (1, 2), (5, 11)):
        # NaN codes around the rows
        _, xv = within(x, at, more, 0x7f)
        _, wv = within(w, at, more, 0x7f)
        _, sv = within(xs, at, more, math.nan)
        _, tv = within(ws, at, more, math.nan)
        big, out = within(torch.zeros((M, N), device=DEV).half(), at, more, 3.0)
        y = d.f8_linear(xv, sv, wv, tv, bias=b, out=out)
        assert y.data_ptr() == out.data_ptr()
        check_linear(y, x, xs, w, ws, b)
        assert torch.all(big[:, :at] == 3) and torch.all(big[:, at + N:] == 3)


@pytest.mark.parametrize("M", [1, 33, 100, 500])
def test_what_is_not_finite_stays_in_its_rows_and_columns(d, M):
    x, xs, w, ws, _ = make(M, 300, 400, 9)
    want = d.f8_linear(x, xs, w, ws)
    x2, w2, xs2 = x.clone(), w.clone(), xs.clone()
    x2.view(torch.uint8)[M // 2, 399] = 0x7f   # NaN
    w2.view(torch.uint8)[17, 0] = 0xff
    xs2[0, 1] = math.inf
    y = d.f8_linear(x2, xs2, w2, ws)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[M // 2], bad[:, 17], bad[0] = True, True, True
    assert torch.equal(torch.isfinite(y), ~bad)
    assert torch.equal(y[~bad], want[~bad])


def test_scales_of_very_different_sizes(d):
    """Tokens and blocks from 2^-60 to 2^60 whose products are ordinary numbers."""
    for M in (5, 50, 300):
        x, xs, w, ws, _ = make(M, 256, 512, M)
        e = torch.tensor([-60, 60, 20, -30], device=DEV).float()
        check_linear(d.f8_linear(x, xs * torch.exp2(e), w, ws * torch.exp2(-e)), x, xs * torch.exp2(e), w, ws * torch.exp2(-e), None)
        zero = xs.clone()
        zero[:, 2] = 0
        zero[M // 2] = 0
        y = d.f8_linear(x, zero, w, ws)
        assert torch.all(y[M // 2] == 0)
        check_linear(y, x, zero, w, ws, None)


def test_the_same_bits_every_time_and_on_another_stream(d):
    for M, N, K in ((1, 4096, 4096), (40, 1000, 2048), (300, 1000, 2048), (2000, 2048, 1024)):
        x, xs, w, ws, b = make(M, N, K, 4)
        want = d.f8_linear(x, xs, w, ws, bias=b)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        got = d.f8_linear(x, xs, w, ws, bias=b, stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(d.f8_linear(x, xs, w, ws, bias=b), want)


def test_rows_that_lie_far_apart(d):
    """The last rows of x, of the weights and of the output lie past 4 GiB."""
    M, N, K = 80, 70, 256
    x, xs, w, ws, b = make(M, N, K, 8)
    far = 1 << 26
    for rows in (16, 80):
        big = torch.empty(rows * far, dtype=torch.uint8, device=DEV)
        xv = big.as_strided((rows, K), (far, 1)).view(E4M3)
        xv.copy_(x[:rows])
        check_linear(d.f8_linear(xv, xs[:rows], w, ws, bias=b), x[:rows], xs[:rows], w, ws, b)
        del big, xv
    big = torch.empty(N * far, dtype=torch.uint8, device=DEV)
    wv = big.as_strided((N, K), (far, 1)).view(E4M3)
    wv.copy_(w)
    check_linear(d.f8_linear(x, xs, wv, ws, bias=b), x, xs, w, ws, b)
    out = big.view(torch.float16).as_strided((M, N), (far // 2 * N // M // 8 * 8, 1))
    check_linear(d.f8_linear(x, xs, w, ws, bias=b, out=out), x, xs, w, ws, b)


def test_nothing_to_do(d):
    x, xs, w, ws, b = make(3, 200, 256, 1)
    assert d.f8_linear(x[:0], xs[:0], w, ws).shape == (0, 200)
    assert d.f8_linear(x, xs, w[:0], ws[:0]).shape == (3, 0)
    y = d.f8_linear(x[:, :0], xs[:, :0], w[:, :0], ws[:, :0], bias=b)
    assert torch.equal(y, b[None].expand(3, 200))
    assert torch.all(d.f8_linear(x[:, :0], xs[:, :0], w[:, :0], ws[:, :0]) == 0)


@pytest.mark.parametrize("M", [1, 40, 200, 600])
def test_in_a_graph(d, M):
    x, xs, w, ws, b = make(M, 700, 1024, M)
    d.f8_linear(x, xs, w, ws, bias=b)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        y = d.f8_linear(x, xs, w, ws, bias=b)
    for seed in range(3):
        x2, xs2, *_ = make(M, 700, 1024, seed + 50)
        x.view(torch.uint8).copy_(x2.view(torch.uint8))
        xs.copy_(xs2)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, d.f8_linear(x, xs, w, ws, bias=b))


def test_weights_from_quantize(d):
    gen = torch.Generator(device=DEV).manual_seed(2)
    full = torch.randn((300, 700), device=DEV, generator=gen) * 0.03
    q = decode.f8_quantize(full.bfloat16())
    back = decode.f8_values(q.weight, q.scales)
    top = (full.bfloat16().to(F)).abs()
    # half a step of the code, or of the smallest codes', with the quotient's and the product's roundings
    s = q.scales.to(F).repeat_interleave(128, 0)[:300].repeat_interleave(128, 1)[:, :700]
    assert torch.all((back.to(F) - full.bfloat16().to(F)).abs() <= torch.maximum(top * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20))
    x, xs, *_ = make(9, 1, 700, 3)
    check_linear(d.f8_linear(x, xs, q.weight, q.scales), x, xs, q.weight, q.scales, None)


def test_refusals(d):
    x, xs, w, ws, b = make(4, 200, 256, 7)
    for bad in (dict(x=x.view(torch.uint8)), dict(weight=w.float()), dict(x_scales=xs.half()), dict(w_scales=ws.double()),
                dict(bias=b.bfloat16()), dict(dtype=torch.float32), dict(out=torch.empty((4, 200), device=DEV))):
        with pytest.raises(TypeError):
            d.f8_linear(**{**dict(x=x, x_scales=xs, weight=w, w_scales=ws), **bad})
    for bad in (dict(x=x[:, :200]), dict(x=x[0]), dict(x=x.view(torch.uint8).t().contiguous().t().view(E4M3)), dict(weight=w[:100]), dict(x_scales=xs[:3]),
                dict(x_scales=xs[:, :1]), dict(w_scales=ws[:1]), dict(bias=b[:199]), dict(out=torch.empty((4, 199), device=DEV).half()),
                dict(weight=w.cpu()), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            d.f8_linear(**{**dict(x=x, x_scales=xs, weight=w, w_scales=ws), **bad})
    with pytest.raises(decode.DecodeError):  # the output over the scales
        both = torch.zeros(4000, device=DEV)
        d.f8_linear(x, both[:8].view(4, 2), w, ws, out=both.view(torch.float16)[:800].view(4, 200))


@pytest.mark.parametrize("M, N, K", [(1, 5000, 129), (16, 4100, 127), (17, 64, 255), (63, 65, 1153), (64, 64, 18), (65, 130, 131),
                                     (1700, 2000, 143), (800, 5003, 515), (1025, 3100, 257)])
def test_rows_at_odd_bytes(d, M, N, K):
    """Products, places and rows apart, where nothing but single bytes is aligned."""
    for dtype in (torch.float16, torch.bfloat16):
        x, xs, w, ws, b = make(M, N, K, M + N + K, dtype)
        y = d.f8_linear(x, xs, w, ws, bias=b, dtype=dtype)
        check_linear(y, x, xs, w, ws, b)
    room = [torch.full((r, K + 6), 0x7f, dtype=torch.uint8, device=x.device) for r in (M, N)]  # NaN between the rows
    for to, of in zip(room, (x, w)):
        to[:, 3:3 + K] = of.view(torch.uint8)
    cut = [r.view(x.dtype)[:, 3:3 + K] for r in room]
    assert torch.equal(d.f8_linear(cut[0], xs, cut[1], ws, bias=b, dtype=dtype), y)
