"""rms_norm_f8 of more rows than 512, which fewer threads to a row take, against its definition in float64."""
import pytest
import torch

from drafts_ref import E4M3, check_norm, norm

pytestmark = pytest.mark.gpu
decode = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from test_gpu_rms_norm_f8 import DEV, make  # noqa: E402

# From each number of threads and of groups of columns: full ones, a last one in part, rows at 16 bytes and at 2.
COLUMNS = [8, 200, 512, 520, 513, 1000, 1024, 1030, 2048, 2056, 2050, 4096, 4095, 4100, 6000, 8192, 8190, 11008, 11009, 16384, 16380, 16392, 16385]


@pytest.fixture(scope="module")
def d():
    h = decode.Decode()
    yield h
    h.close()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("K", COLUMNS)
def test_against_the_definition(d, K, dtype):
    for M in (513, 1025):  # one row more than workgroups of four take evenly
        x, r, g = make(M, K, dtype, M + K)
        for weight, residual in ((g, r), (None, None)):
            codes, scales, total = d.rms_norm_f8(x, weight, residual, eps=1e-5)
            t, y = norm(x, residual, weight, 1e-5)
            assert residual is None or torch.equal(total, t)
            check_norm(codes, scales, y, K)


@pytest.mark.parametrize("K", COLUMNS)
@pytest.mark.parametrize("which", ["x", "residual"])
def test_the_total_may_take_an_inputs_place(d, K, which):
    x, r, g = make(771, K, torch.bfloat16, K)
    want = d.rms_norm_f8(x, g, r)
    got = d.rms_norm_f8(x, g, r, total=x if which == "x" else r)
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("K", [300, 1000, 1024, 3000, 4096, 7000, 8192, 12000, 16384, 17000])
def test_values_whose_squares_leave_binary32(d, K):
    """Some of the rows: the others beside them in a workgroup are ordinary."""
    for size, eps in ((1e30, 1e-6), (3e38, 0.0), (1e-30, 0.0), (1e-38, 0.0), (1e-30, 1e-58)):
        gen = torch.Generator(device=DEV).manual_seed(K)
        x = torch.rand((523, K), device=DEV, generator=gen) * 2 - 1
        x[torch.rand(523, device=DEV, generator=gen) < 0.4] *= size
        x = x.to(torch.bfloat16)
        codes, scales, _ = d.rms_norm_f8(x, eps=eps)
        assert torch.isfinite(scales).all()
        check_norm(codes, scales, norm(x, None, None, float(torch.tensor(eps, dtype=torch.float32)))[1], K)


@pytest.mark.parametrize("K", [96, 900, 2000, 4096, 8000, 16000, 20000])
def test_strides_and_places(d, K):
    x, r, g = make(517, K, torch.float16, K)
    for at, more in ((0, 8), (3, 5), (1, 16)):
        wide = [torch.full((517, K + more + at), 7.0, dtype=torch.float16, device=DEV) for _ in range(3)]
        wide[0][:, at:at + K], wide[1][:, at:at + K] = x, r
        kb = -(-K // 128)
        codes = torch.full((517, K + more), 9, dtype=torch.uint8, device=DEV)
        scales = torch.full((517, kb + 3), 5.0, device=DEV)
        cut = slice(at, at + K) if at <= more else slice(0, K)
        out = d.rms_norm_f8(wide[0][:, at:at + K], g, wide[1][:, at:at + K], codes=codes[:, cut].view(E4M3),
                            scales=scales[:, 1:1 + kb], total=wide[2][:, at:at + K])
        t, y = norm(x, r, g, 1e-6)
        check_norm(out[0].contiguous(), out[1], y, K)
        assert torch.equal(out[2], t)
        assert torch.all(wide[2][:, :at] == 7) and torch.all(wide[2][:, at + K:] == 7)
        assert torch.all(codes[:, :cut.start] == 9) and torch.all(codes[:, cut.stop:] == 9)
        assert torch.all(scales[:, 0] == 5) and torch.all(scales[:, 1 + kb:] == 5)


@pytest.mark.parametrize("K", [500, 1000, 4096, 8192, 16384])
def test_zeros_and_values_that_are_not_finite_stay_in_their_rows(d, K):
    x, _, g = make(514, K, torch.bfloat16, 6)
    want = d.rms_norm_f8(x, g)
    bad = [1, 4, 7, 250, 513]
    y = x.clone()
    y[1], y[4, K - 1], y[7, 0], y[250, K // 2], y[513] = 0, float("nan"), float("inf"), float("-inf"), float("nan")
    got = d.rms_norm_f8(y, g)
    keep = torch.ones(514, dtype=torch.bool, device=DEV)
    keep[bad] = False
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a.view(torch.uint8)[keep], b.view(torch.uint8)[keep])
    assert not got[1][1].any() and not got[0].view(torch.uint8)[1].any()
    assert not torch.isfinite(got[1][[4, 513]]).any()
    assert not torch.isfinite(got[1][7, 0]) and not torch.isfinite(got[1][250, K // 2 // 128])
