"""The example's layers on the decode operators against the same layers in float64."""
import pytest
import torch

from decode_ref import F, attend, cached, rotate

pytestmark = pytest.mark.gpu
step = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode_step")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from dense_fp16_gemm_hgemm_amd.decode import w4_unpack  # noqa: E402


def small(**kw):
    return step.Config(**{**dict(hidden=256, heads=8, kv_heads=2, head_dim=64, inner=352, layers=2, page_size=16,
                                 group=32), **kw})


def norm(x):
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt()


def plain(m, x, lens):
    """One token a sequence in float64 over the caches as they are after the step."""
    c = m.config
    freq = 10000.0 ** (-torch.arange(0, c.head_dim, 2, dtype=F, device="cuda") / c.head_dim)
    x = x.to(F)
    for layer in m.layers:
        w = lambda l: w4_unpack(l.w4).to(F).t()  # noqa: E731
        qkv = (norm(x) @ w(layer.qkv)).view(x.shape[0], -1, c.head_dim)
        pos = torch.tensor(lens, device="cuda")
        q = rotate(qkv[:, :c.heads], pos, freq, False)
        k = rotate(qkv[:, c.heads:c.heads + c.kv_heads], pos, freq, False)
        v = qkv[:, c.heads + c.kv_heads:]
        for b, n in enumerate(lens):  # the new token's codes are within a step of its values
            for which, want in (("k", k), ("v", v)):
                have, _ = cached(layer.cache, m.table, b, n + 1, which)
                step = getattr(layer.cache, which + "_scale")[m.table[b, n // c.page_size].long()].to(F)[:, None]
                if layer.cache.k.dtype == torch.float8_e4m3fn:  # half a step is 2^-4 of the value, or 2^-10 codes
                    step = 2.0 ** -4 * want[b].abs() + 2.0 ** -10 * step
                assert torch.all((have[:, n] - want[b]).abs() <= step + 0.02)
        a, _ = attend(q, layer.cache, m.table, [n + 1 for n in lens], list(range(len(lens) + 1)), c.window, c.sinks)
        x = x + a.reshape(x.shape[0], -1) @ w(layer.out)
        g = norm(x) @ w(layer.gate_up)
        x = x + (torch.nn.functional.silu(g[:, :c.inner]) * g[:, c.inner:]) @ w(layer.down)
    return x


@pytest.mark.parametrize("codes", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("window, sinks", [(0, 0), (20, 3)])
def test_steps_follow_the_layers(window, sinks, codes):
    m = step.Model(small(window=window, sinks=sinks), 3, 100, seed=3, codes=codes)
    gen = torch.Generator(device="cuda").manual_seed(4)
    lens = [1, 40, 77]
    cu = torch.tensor([0, 1, 41, 118], dtype=torch.int32, device="cuda")
    x = m.forward(torch.randn((118, 256), device="cuda", generator=gen).half(), cu, 77)
    x = x[cu[1:].long() - 1]
    for _ in range(3):
        got = m.forward(x)
        ref = plain(m, x, lens)
        # A dozen roundings to binary16 on values of a few units lie on the way through two
        # layers (2^-11 each, at most tripled by the products): 12 * 3 * 2^-11 of the largest.
        assert float((got.to(F) - ref).abs().max()) <= 12 * 3 * 2.0 ** -11 * float(ref.abs().max())
        lens = [n + 1 for n in lens]
        assert m.lens.tolist() == lens
        x = got
    m.close()


def test_a_captured_step_equals_an_eager_one():
    runs = []
    for captured in (False, True):
        m = step.Model(small(), 4, 60, seed=5)
        gen = torch.Generator(device="cuda").manual_seed(6)
        cu = torch.tensor([0, 5, 9, 30, 31], dtype=torch.int32, device="cuda")
        x = m.forward(torch.randn((31, 256), device="cuda", generator=gen).half(), cu, 21)[cu[1:].long() - 1]
        outs = []
        if captured:
            g, at, out = m.graph(x)
            at.copy_(x)
            for _ in range(4):
                g.replay()
                torch.cuda.synchronize()
                outs.append(out.clone())
                at.copy_(out)
        else:
            for _ in range(4):
                x = m.forward(x)
                outs.append(x)
        runs.append(outs)
        m.close()
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a, b), i


def test_command_runs(capsys):
    step.main(["--batch", "3", "--prompt", "20", "--steps", "2", "--layers", "1"])
    assert "us a step" in capsys.readouterr().out
