"""rms_norm_f8 on the GPU against its definition in float64."""
import math

import pytest
import torch

from decode_ref import F, values
from drafts_ref import E4M3, blocks, check_norm, norm

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


def make(M, K, dtype, seed, size=2.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    x, r = ((torch.randn((M, K), device=DEV, generator=gen) * s).to(dtype) for s in (size, 1.0))
    return x, r, (1 + torch.randn(K, device=DEV, generator=gen) * 0.3).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M, K", [(1, 1), (3, 7), (1, 128), (5, 129), (4, 512), (7, 520), (2, 1000), (6, 1024), (3, 2048),
                                  (2, 2056), (65, 4096), (3, 4100), (2, 8192), (3, 11008), (2, 16384), (2, 16392), (1, 40001)])
def test_against_the_definition(d, M, K, dtype):
    x, r, g = make(M, K, dtype, M + K)
    for weight, residual in ((g, r), (None, r), (g, None), (None, None)):
        codes, scales, total = d.rms_norm_f8(x, weight, residual, eps=1e-5)
        t, y = norm(x, residual, weight, 1e-5)
        assert codes.shape == (M, K) and codes.dtype == E4M3 and scales.shape == (M, -(-K // 128))
        assert (total is None) == (residual is None)
        assert total is None or torch.equal(total, t)
        check_norm(codes, scales, y, K)


def test_many_rows(d):
    x, r, g = make(70000, 64, torch.bfloat16, 3)
    codes, scales, total = d.rms_norm_f8(x, g, r)
    t, y = norm(x, r, g, 1e-6)
    assert torch.equal(total, t)
    check_norm(codes, scales, y, 64)


@pytest.mark.parametrize("K", [96, 300, 4096, 20000])
def test_strides_and_places(d, K):
    """Rows apart, at odd places, and what lies between them stays."""
    x, r, g = make(5, K, torch.float16, K)
    for at, more in ((0, 8), (3, 5), (1, 16)):
        wide = [torch.full((5, K + more + at), 7.0, dtype=torch.float16, device=DEV) for _ in range(3)]
        wide[0][:, at:at + K], wide[1][:, at:at + K] = x, r
        kb = -(-K // 128)
        codes = torch.full((5, K + more), 9, dtype=torch.uint8, device=DEV)
        scales = torch.full((5, kb + 3), 5.0, device=DEV)
        out = d.rms_norm_f8(wide[0][:, at:at + K], g, wide[1][:, at:at + K], codes=codes[:, at:at + K].view(E4M3) if at <= more else None,
                            scales=scales[:, 1:1 + kb], total=wide[2][:, at:at + K])
        t, y = norm(x, r, g, 1e-6)
        check_norm(out[0].contiguous(), out[1], y, K)
        assert torch.equal(out[2], t)
        assert torch.all(wide[2][:, :at] == 7) and torch.all(wide[2][:, at + K:] == 7)
        assert torch.all(codes[:, :at] == 9) and torch.all(codes[:, at + K:] == 9)
        assert torch.all(scales[:, 0] == 5) and torch.all(scales[:, 1 + kb:] == 5)


@pytest.mark.parametrize("K", [500, 4096, 17000])
@pytest.mark.parametrize("which", ["x", "residual"])
def test_the_total_may_take_an_inputs_place(d, K, which):
    x, r, g = make(9, K, torch.bfloat16, K)
    want = d.rms_norm_f8(x, g, r)
    got = d.rms_norm_f8(x, g, r, total=x if which == "x" else r)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_values_whose_squares_leave_binary32(d):
    """bf16 reaches 2^127: the mean of squares is the formula's all the same, and for tiny rows too where eps is 0."""
    for size, eps in ((1e30, 1e-6), (3e38, 0.0), (1e-30, 0.0), (1e-38, 0.0), (1e-30, 1e-58)):
        for K in (256, 3000, 20000):
            gen = torch.Generator(device=DEV).manual_seed(K)
            x = (torch.rand((3, K), device=DEV, generator=gen) * 2 - 1).mul_(size).to(torch.bfloat16)
            codes, scales, _ = d.rms_norm_f8(x, eps=eps)
            assert torch.isfinite(scales).all()
            # eps is an argument in binary32
            check_norm(codes, scales, norm(x, None, None, float(torch.tensor(eps, dtype=torch.float32)))[1], K)


def test_rows_of_zeros_and_blocks_of_zeros(d):
    x, r, g = make(4, 1000, torch.float16, 5)
    x[1], r[1] = 0, 0
    x[2, 128:256], r[2, 128:256] = 0, 0
    codes, scales, total = d.rms_norm_f8(x, g, r)
    assert torch.all(values(codes)[1] == 0) and torch.all(scales[1] == 0) and torch.all(total[1] == 0)
    assert scales[2, 1] == 0 and torch.all(values(codes)[2, 128:256] == 0)
    check_norm(codes, scales, norm(x, r, g, 1e-6)[1], 1000)


def test_values_that_are_not_finite(d):
    """They stay in their row; a block reads as non-finite where the formula is."""
    x, _, g = make(6, 700, torch.bfloat16, 6)
    x[1, 300] = math.nan
    x[3, 5] = math.inf
    w = g.clone()
    w[600] = math.inf
    for weight in (g, w):
        codes, scales, _ = d.rms_norm_f8(x, weight)
        y = norm(x, None, weight, 1e-6)[1]
        finite = torch.isfinite(blocks(y)).all(-1)
        assert torch.equal(torch.isfinite(scales), finite)
        read = values(codes) * scales.to(F).repeat_interleave(128, 1)[:, :700]
        assert torch.equal(torch.isfinite(blocks(read)).all(-1), finite)
        rows = finite.all(1)
        if rows.any():
            check_norm(codes[rows], scales[rows], y[rows], 700)


def test_nothing_to_do_and_another_stream(d):
    x, r, g = make(0, 300, torch.float16, 1)
    codes, scales, total = d.rms_norm_f8(x, g, r)
    assert codes.shape == (0, 300) and scales.shape == (0, 3) and total.shape == (0, 300)
    codes, scales, _ = d.rms_norm_f8(torch.empty((4, 0), device=DEV).half())
    assert codes.shape == (4, 0) and scales.shape == (4, 0)
    x, r, g = make(300, 4096, torch.float16, 2)
    want = d.rms_norm_f8(x, g, r)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = d.rms_norm_f8(x, g, r, stream=side)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals(d):
    x, r, g = make(4, 256, torch.float16, 7)
    with pytest.raises(TypeError):
        d.rms_norm_f8(x.float())
    with pytest.raises(TypeError):
        d.rms_norm_f8(x, g.bfloat16())
    with pytest.raises(TypeError):
        d.rms_norm_f8(x, g, r.bfloat16())
    for bad in (dict(x=x.t()), dict(x=x[0]), dict(weight=g[:100]), dict(residual=r[:3]), dict(residual=r[:, :100]),
                dict(total=x.clone()), dict(scales=torch.empty((4, 3), device=DEV)), dict(x=x.cpu())):
        with pytest.raises(ValueError):
            d.rms_norm_f8(**{**dict(x=x), **bad})
    both = torch.zeros((5, 256), device=DEV).half()
    for bad in (dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(x=both[:4], residual=r, total=both[1:])):
        with pytest.raises(decode.DecodeError):
            d.rms_norm_f8(**{**dict(x=x), **bad})
