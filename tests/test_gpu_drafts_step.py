"""Trees of drafted tokens through the example's layers: all operators together, against float64."""
import random

import pytest
import torch

from decode_ref import F, cached, rotate
from drafts_ref import attend_tree, check_attend, check_linear, check_norm, norm
from test_gpu_decode_step import small

pytestmark = pytest.mark.gpu
step = pytest.importorskip("dense_fp16_gemm_hgemm_amd.decode_step")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)
from dense_fp16_gemm_hgemm_amd import decode  # noqa: E402


def put(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def drafts(new, seed):
    """seen, depth, cu and parents of random trees."""
    r = random.Random(seed)
    parents = [[r.randint(max(-1, i - 4), i - 1) for i in range(n)] for n in new]
    trees = [decode.tree(p) for p in parents]
    words = max(t[0].shape[1] for t in trees)
    seen = torch.cat([torch.nn.functional.pad(t[0], (0, words - t[0].shape[1])) for t in trees])
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    return seen.cuda(), torch.cat([t[1] for t in trees]).cuda(), cu, parents


def path_of(parents, leaf):
    path = []
    while leaf >= 0:
        path.insert(0, leaf)
        leaf = parents[leaf]
    return path


def follow(m, x, lens, seen, depth, cu):
    """The layers by the operators' calls, each held against its definition on the inputs that it had; the caches
    hold the drafts already, and appending them again changes nothing."""
    c, d = m.config, m.decode
    freq = 10000.0 ** (-torch.arange(0, c.head_dim, 2, dtype=F, device="cuda") / c.head_dim)
    new = [b - a for a, b in zip(cu, cu[1:])]
    pos = depth + torch.repeat_interleave(torch.tensor(lens, device="cuda"), torch.tensor(new, device="cuda")).int()
    total, dcu = [a + b for a, b in zip(lens, new)], put(cu)

    def eight(x, more, w):
        codes, scales, t = d.rms_norm_f8(x, residual=more)
        want, y = norm(x, more, None, 1e-6)
        assert more is None or torch.equal(t, want)
        check_norm(codes, scales, y, x.shape[1])
        out = d.f8_linear(codes, scales, w.f8.weight, w.f8.scales)
        check_linear(out, codes, scales, w.f8.weight, w.f8.scales, None)
        return want, out

    more = None
    for layer in m.layers:
        x, qkv = eight(x, more, layer.qkv)
        qkv = qkv.view(x.shape[0], -1, c.head_dim)
        k, v = qkv[:, c.heads:c.heads + c.kv_heads], qkv[:, c.heads + c.kv_heads:]
        q = d.kv_append(layer.cache, k, v, m.table, put(lens), dcu, max(new), q=qkv[:, :c.heads], rope=m.rope, positions=pos)
        want = rotate(qkv[:, :c.heads], pos, freq, False)
        size = rotate(qkv[:, :c.heads].abs(), pos * 0, freq, False).abs().amax(-1, keepdim=True) * 2
        assert torch.all((q.to(F) - want).abs() <= size * 4 * 2.0 ** -24 + want.abs() * 2.0 ** -11 + 2.0 ** -25)
        for b, n in enumerate(new):
            for which, x64 in (("k", rotate(k, pos, freq, False)), ("v", v.to(F))):
                have, _ = cached(layer.cache, m.table, b, total[b], which)
                pages = m.table[b, torch.arange(lens[b], total[b], device="cuda") // c.page_size].long()
                s = getattr(layer.cache, which + "_scale")[pages].to(F).t()[..., None]
                assert torch.all((have[:, lens[b]:] - x64[cu[b]:cu[b + 1]].transpose(0, 1)).abs() <= s * 0.5 + 2.0 ** -20 * s * 127)
        a = d.kv_attend_tree(q, layer.cache, m.table, put(total), seen, dcu, max(new), window=c.window, sinks=c.sinks)
        check_attend(a, *attend_tree(q, layer.cache, m.table, total, seen, cu, c.window, c.sinks))
        x, g = eight(m.gemm.run(a.view(x.shape[0], -1), layer.out.full), x, layer.gate_up)
        g = torch.nn.functional.silu(g[:, :c.inner].float()) * g[:, c.inner:].float()
        more = m.gemm.run(g.half(), layer.down.full)
    return x + more


def begin(m, prompt, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cu = put([0] + list(torch.tensor(prompt).cumsum(0)))
    m.forward(torch.randn((sum(prompt), 256), device="cuda", generator=gen).half(), cu, max(prompt))
    return gen


@pytest.mark.parametrize("window, sinks", [(0, 0), (20, 3)])
def test_verified_drafts_follow_the_layers(window, sinks):
    m = step.Model(small(window=window, sinks=sinks), 3, 200, seed=3, drafts=True)
    lens, new = [1, 40, 77], [9, 1, 40]
    gen = begin(m, lens, 4)
    for turn in range(3):
        seen, depth, cu, parents = drafts(new, turn)
        x = torch.randn((cu[-1], 256), device="cuda", generator=gen).half()
        got = m.verify(x, seen, depth, put(cu), max(new))
        assert m.lens.tolist() == lens
        assert torch.equal(got, follow(m, x, lens, seen, depth, cu))
        path = [path_of(p, len(p) - 1) for p in parents]
        before = [cached(m.layers[1].cache, m.table, b, lens[b] + new[b], "v")[0] for b in range(3)]
        kept = [0] + list(torch.tensor([len(p) for p in path]).cumsum(0))
        m.accept(put(sum(path, [])), put(kept), max(map(len, path)))
        for b in range(3):
            now, _ = cached(m.layers[1].cache, m.table, b, lens[b] + len(path[b]), "v")
            pages = m.table[b, torch.arange(lens[b], lens[b] + len(path[b]), device="cuda") // 16].long()
            size = m.layers[1].cache.v_scale[pages].to(F).t()[..., None]
            assert torch.all((now[:, lens[b]:] - before[b][:, [lens[b] + i for i in path[b]]]).abs() <= size * 0.51)
        lens = [a + len(p) for a, p in zip(lens, path)]
        assert m.lens.tolist() == lens
    m.close()


def test_a_fork_goes_on_like_its_source():
    m = step.Model(small(), 3, 100, seed=9, drafts=True)
    gen = begin(m, [50, 7, 20], 10)
    m.fork(0, 2)
    assert m.lens.tolist() == [50, 7, 50]
    x = torch.randn((3, 256), device="cuda", generator=gen).half()
    x[2] = x[0]
    y = m.forward(x)
    assert torch.equal(y[0], y[2])
    seen, depth, cu, _ = drafts([6, 6, 6], 11)
    seen[12:], depth[12:] = seen[:6], depth[:6]
    x = torch.randn((18, 256), device="cuda", generator=gen).half()
    x[12:] = x[:6]
    y = m.verify(x, seen, depth, put(cu), 6)
    assert torch.equal(y[:6], y[12:])
    m.close()


def test_drafts_past_the_page_table_are_refused():
    m = step.Model(small(), 2, 32, seed=1, drafts=True)
    gen = begin(m, [10, 25], 2)
    seen, depth, cu, _ = drafts([8, 8], 3)
    x = torch.randn((16, 256), device="cuda", generator=gen).half()
    with pytest.raises(ValueError, match="room for 32"):
        m.verify(x, seen, depth, put(cu), 8)
    m.close()


@pytest.mark.parametrize("code", [torch.int8, torch.float8_e4m3fn])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_with_positions(code, interleaved):
    """Rows of the rotation's table by token: the places' own ones change nothing, others turn by theirs, and ones
    outside the table take its ends."""
    H, D, page, Hq = 2, 64, 16, 6
    table, past, cu, new = put([[3, 1, 5], [0, 4, 2]]), put([5, 20]), put([0, 20, 29]), [20, 9]
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn((29, h, D), device="cuda", generator=gen).half() for h in (Hq, H, H))
    rope = decode.rope_table(48, D)
    places = torch.cat([torch.arange(5, 25), torch.arange(20, 29)]).int().cuda()
    with decode.Decode() as d:
        def run(**kw):
            c = decode.KvCache.empty(6, H, D, page, code)
            return c, d.kv_append(c, k, v, table, past, cu, 20, q=q, interleaved=interleaved, **kw)
        c0, q0 = run(rope=rope)
        c1, q1 = run(rope=rope, positions=places)
        assert torch.equal(q0, q1)
        for n in ("k", "v", "k_scale", "v_scale"):
            assert torch.equal(getattr(c0, n).view(torch.uint8), getattr(c1, n).view(torch.uint8))
        few = rope[:10].contiguous()  # fewer rows than the table has positions
        at = torch.randint(-3, 14, (29,), device="cuda", generator=gen).int()
        c2, q2 = run(rope=few, positions=at)
        freq = 10000.0 ** (-torch.arange(0, D, 2, dtype=F, device="cuda") / D)
        pos = at.clamp(0, 9)
        want = rotate(q, pos, freq, interleaved)
        size = rotate(q.abs(), pos * 0, freq, interleaved).abs().amax(-1, keepdim=True) * 2
        # two products, a sum, the table's own rounding, then binary16
        assert torch.all((q2.to(F) - want).abs() <= size * 4 * 2.0 ** -24 + want.abs() * 2.0 ** -11)
        want = rotate(k, pos, freq, interleaved)
        for b in range(2):
            have, _ = cached(c2, table, b, int(past[b]) + new[b], "k")
            lo, hi = int(cu[b]), int(cu[b + 1])
            pages = table[b, torch.arange(int(past[b]), int(past[b]) + new[b], device="cuda") // page].long()
            s = c2.k_scale[pages].to(F)[..., None]
            x = want[lo:hi]
            near = s * 0.5 if code == torch.int8 else torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)
            assert torch.all((have[:, int(past[b]):].transpose(0, 1) - x).abs() <= near + 2.0 ** -20 * s * 448)
        assert torch.equal(c2.v.view(torch.uint8), c0.v.view(torch.uint8))
        for bad in (at[:28], at.cpu()):
            with pytest.raises(ValueError):
                run(rope=rope, positions=bad)
        with pytest.raises(TypeError):
            run(rope=rope, positions=at.long())
        with pytest.raises(ValueError):
            run(rope=few)


def test_the_whole_step_in_a_graph():
    """verify and accept captured, replayed over other drafts, against the eager ones; the tokens before them stay."""
    runs = []
    seen, depth, cu, parents = drafts([7, 12], 5)
    path = [path_of(p, len(p) - 1) for p in parents]
    kept, cu_kept, most = put(sum(path, [])), put([0, len(path[0]), len(path[0]) + len(path[1])]), max(map(len, path))
    for captured in (False, True):
        m = step.Model(small(), 2, 200, seed=5, drafts=True)
        gen = begin(m, [30, 11], 6)
        x = torch.randn((19, 256), device="cuda", generator=gen).half()
        lens, longest, positions = m.lens.clone(), m.longest, put(cu)
        keep = [[getattr(layer.cache, n).clone() for n in ("k", "v", "k_scale", "v_scale")] for layer in m.layers]

        def one():
            out = m.verify(x, seen, depth, positions, 12)
            m.accept(kept, cu_kept, most)
            return out

        outs = []
        if captured:
            one()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                out = one()
            m.lens.copy_(lens)
            m.longest = longest
            for layer, old in zip(m.layers, keep):
                for n, t in zip(("k", "v", "k_scale", "v_scale"), old):
                    getattr(layer.cache, n).view(torch.uint8).copy_(t.view(torch.uint8))
        for seed in range(3):
            gen.manual_seed(seed)
            x.copy_(torch.randn((19, 256), device="cuda", generator=gen).half())
            if captured:
                g.replay()
                torch.cuda.synchronize()
                outs.append(out.clone())
            else:
                outs.append(one())
        runs.append(outs)
        m.close()
    for i, (a, b) in enumerate(zip(*runs)):
        assert torch.equal(a, b), i


def test_command_runs_with_drafts(capsys):
    step.main(["--batch", "3", "--prompt", "20", "--steps", "2", "--layers", "1", "--drafts", "13"])
    assert "13 drafts each" in capsys.readouterr().out
