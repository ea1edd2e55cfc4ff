"""Linear layers with 4-bit weights against the definition in float64."""
import pytest
import torch

from decode_ref import F, half_step

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
DEV = torch.device("cuda", 0)
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


def weights(N, K, group, t, zeros, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    groups = -(-K // group)
    codes = torch.randint(0, 16, (N, K), generator=g, device=DEV)
    scales = (torch.rand((N, groups), generator=g, device=DEV) * 0.02 + 0.001).to(t)
    z = torch.randint(0, 16, (N, groups), generator=g, device=DEV) if zeros else None
    return decode.w4_pack(codes, scales, z, group), codes, scales, z, g


def check(y, x, codes, scales, z, group, bias=None):
    """Against float64.  Every product that a kernel adds is at most 62 |x| s in size (a code may be
    carried with an offset of 16 that its zero point's term takes back), so binary32 sums of K terms
    are off by at most (K + 64) 2^-24 of their total in the worst case; rounding y adds half a step."""
    col = torch.arange(x.shape[1], device=DEV) // group
    s = scales.to(F)[:, col]
    w = (codes - (8 if z is None else z[:, col])).to(F) * s
    ref = x.to(F) @ w.t()
    size = 62 * x.to(F).abs() @ s.abs().t()
    if bias is not None:
        ref, size = ref + bias.to(F), size + bias.to(F).abs()
    K, u = x.shape[1], half_step(y.dtype)
    fine = torch.finfo(y.dtype)
    err = (y.to(F) - ref).abs()
    assert torch.all(err <= u * ref.abs() + (fine.tiny * fine.eps) / 2 + (1 + u) * (K + 64) * 2.0 ** -24 * size)
    # roundings are independent, so in the 2-norm they add up as a square root
    if ref.numel() > 100:
        norm = ref.norm()
        assert (y.to(F) - ref).norm() <= u * norm + 4 * (K + 64) ** 0.5 * 2.0 ** -24 * size.norm() / max(K, 1) ** 0.5 + 1e-30


SHAPES = [
    (1, 16, 128, 128), (1, 1, 1, 32), (2, 17, 33, 32), (3, 40, 96, 32), (5, 100, 1000, 64), (7, 257, 520, 32),
    (8, 64, 2048, 128), (15, 31, 127, 32), (16, 48, 4096, 256), (17, 130, 384, 96), (31, 33, 640, 128),
    (33, 80, 129, 64), (48, 96, 1024, 128), (63, 65, 776, 64), (64, 128, 2056, 128), (65, 50, 256, 32),
    (130, 200, 512, 128), (1, 4096, 4096, 128), (4, 1024, 11008, 64), (1, 300, 200, 4096), (300, 64, 136, 32),
]


@pytest.mark.parametrize("zeros", [False, True], ids=["z8", "zeros"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M, N, K, group", SHAPES)
def test_shapes(d, M, N, K, group, dtype, zeros):
    print(f"w4 M={M} N={N} K={K} group={group} {dtype} zeros={zeros}", flush=True)
    t = TYPES[dtype]
    w, codes, scales, z, g = weights(N, K, group, t, zeros, M * 7 + N * 3 + K)
    x = torch.randn((M, K), generator=g, device=DEV).to(t)
    bias = torch.randn(N, generator=g, device=DEV).to(t) if (M + N) % 2 else None
    y = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=N, group=group, bias=bias)
    check(y, x, codes, scales, z, group, bias)


@pytest.mark.parametrize("dtype", TYPES)
def test_positive_inputs_do_not_cancel(d, dtype):
    """Activations of one sign, where an offset carried with the codes is largest beside the result."""
    t = TYPES[dtype]
    w, codes, scales, z, g = weights(64, 4096, 128, t, True, 5)
    x = torch.rand((6, 4096), generator=g, device=DEV).to(t)
    check(d.w4_linear(x, w.qweight, w.scales, w.zeros, n=64, group=128), x, codes, scales, z, 128)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 9, 40])
def test_small_integers_are_exact(d, dtype, M):
    t = TYPES[dtype]
    g = torch.Generator(device=DEV).manual_seed(M)
    codes = torch.randint(0, 16, (50, 224), generator=g, device=DEV)
    zeros = torch.randint(0, 16, (50, 7), generator=g, device=DEV)
    w = decode.w4_pack(codes, torch.ones((50, 7), device=DEV, dtype=t), zeros, 32)
    x = torch.zeros((M, 224), device=DEV, dtype=t)  # four terms a row, so that every result fits 8 bits
    x[:, ::56] = torch.randint(-4, 5, (M, 4), generator=g, device=DEV).to(t)
    y = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=50, group=32)
    want = x.to(F) @ (codes - zeros[:, torch.arange(224, device=DEV) // 32]).to(F).t()
    assert torch.equal(y.to(F), want)


@pytest.mark.parametrize("M", [1, 3, 16, 50])
def test_strides_and_odd_alignment(d, M):
    w, codes, scales, z, g = weights(70, 260, 64, torch.float16, True, 11)
    big = torch.randn((M, 301), generator=g, device=DEV).half()
    for x in (big[:, 3:263], big[:, 8:268]):
        out = torch.full((M, 75), 7.0, device=DEV, dtype=torch.float16)
        y = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=70, group=64, out=out[:, 1:71])
        assert y.data_ptr() == out[:, 1:71].data_ptr()
        check(y, x, codes, scales, z, 64)
        assert torch.all(out[:, 0] == 7) and torch.all(out[:, 71:] == 7)


def test_padding_is_not_read_into_results(d):
    """Codes past N and past K, and rows past N of scales, may be anything."""
    w, codes, scales, z, g = weights(21, 130, 32, torch.float16, True, 13)
    x = torch.randn((5, 130), generator=g, device=DEV).half()
    clean = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=21, group=32)
    lane = torch.arange(64, device=DEV)
    past = (lane % 16 >= 5)
    q = w.qweight.clone()
    q[1, :, past] = -1                       # rows 21..31
    word = torch.arange(4, device=DEV)
    q[:, 1, :, 1:] = -1                      # columns 160..255
    q[:, 1, 16:, 0] = -1                     # columns 136..159
    s = w.scales.clone()
    s[:, 21:] = float("nan")
    assert word.numel() == 4 and torch.equal(d.w4_linear(x, q, s, w.zeros, n=21, group=32), clean)


def test_non_finite_inputs_stay_in_their_rows(d):
    w, codes, scales, z, g = weights(40, 256, 64, torch.float16, False, 17)
    x = torch.randn((20, 256), generator=g, device=DEV).half()
    clean = d.w4_linear(x, w.qweight, w.scales, n=40, group=64)
    x[3, 100] = float("nan")
    x[18, 5] = float("inf")
    y = d.w4_linear(x, w.qweight, w.scales, n=40, group=64)
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[18]).any()
    keep = [i for i in range(20) if i not in (3, 18)]
    assert torch.equal(y[keep], clean[keep])


def test_empty_extents(d):
    w, *_ = weights(40, 64, 64, torch.float16, False, 19)
    assert d.w4_linear(torch.empty((0, 64), device=DEV).half(), w.qweight, w.scales, n=40, group=64).shape == (0, 40)
    bias = torch.arange(40, device=DEV).half()
    y = d.w4_linear(torch.empty((3, 0), device=DEV).half(), w.qweight[:, :0], w.scales[:0], n=40, group=64, bias=bias)
    assert torch.equal(y, bias.expand(3, 40))
    y = d.w4_linear(torch.empty((3, 0), device=DEV).half(), w.qweight[:, :0], w.scales[:0], n=40, group=64)
    assert torch.equal(y, torch.zeros_like(y))


def test_same_bits_every_time_on_a_side_stream_and_in_a_graph(d):
    w, codes, scales, z, g = weights(500, 1032, 64, torch.bfloat16, True, 23)
    x = torch.randn((4, 1032), generator=g, device=DEV).bfloat16()
    want = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=500, group=64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(want)
    with torch.cuda.stream(side):
        d.w4_linear(x, w.qweight, w.scales, w.zeros, n=500, group=64, out=out)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.w4_linear(x, w.qweight, w.scales, w.zeros, n=500, group=64, out=out)
    for i in range(3):
        x.copy_(torch.randn((4, 1032), generator=g, device=DEV))
        want = d.w4_linear(x, w.qweight, w.scales, w.zeros, n=500, group=64)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_refusals_on_the_device(d):
    w, *_ = weights(40, 64, 64, torch.float16, True, 29)
    x = torch.zeros((2, 64), device=DEV).half()
    good = dict(x=x, qweight=w.qweight, scales=w.scales, zeros=w.zeros, n=40, group=64)
    d.w4_linear(**good)
    for bad in (dict(n=50), dict(group=32), dict(group=50), dict(scales=w.scales.float()), dict(qweight=w.qweight.cpu()),
                dict(zeros=w.zeros.int()), dict(zeros=w.zeros[:, :16]), dict(bias=torch.zeros(39, device=DEV).half()),
                dict(x=torch.zeros((2, 129), device=DEV).half()), dict(x=x.t()), dict(out=torch.zeros((2, 41), device=DEV).half())):
        with pytest.raises((ValueError, TypeError)):
            d.w4_linear(**{**good, **bad})
