"""64-bit references of the operators for drafted tokens, from their definitions, and the tolerances."""
import math

import torch

from decode_ref import F, QMAX, cached, half_step, values

E4M3 = torch.float8_e4m3fn
STEP32 = 2.0 ** -24


def norm(x, residual, weight, eps):
    """(total, y): the sum in x's type, and its norm in float64."""
    t = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    y = t.to(F) / (t.to(F).square().mean(1, keepdim=True) + eps).sqrt()
    return t, y if weight is None else y * weight.to(F)


def norm_slip(K):
    """How far a binary32 norm may be off, relative to each value.  The sum of squares of one sign has at
    most 8 ceil(K / 512) roundings in a thread, 6 over a wave and 16 over waves, and the root halves
    them; mean, eps, root, reciprocal and two products are 6 more."""
    return (4 * -(-K // 512) + 11 + 6) * STEP32


def blocks(y, fill=0.0):
    """[rows, K] as [rows, ceil(K / 128), 128]."""
    kb = -(-y.shape[1] // 128)
    out = torch.full((y.shape[0], kb * 128), fill, dtype=y.dtype, device=y.device)
    out[:, :y.shape[1]] = y
    return out.view(y.shape[0], kb, 128)


def check_norm(codes, scales, y, K):
    """Codes and scales against y [M, K] in float64, which is finite."""
    slip = norm_slip(K)
    want = blocks(y).abs().amax(-1) / 448
    # one rounding more for the division; a scale below binary32's normal numbers is off by its step
    assert torch.all((scales.to(F) - want).abs() <= want * (slip + STEP32) * 1.01 + 2.0 ** -149)
    s = scales.to(F).repeat_interleave(128, 1)[:, :K]
    off = (values(codes) * s - y).abs()
    # half a step of a code is 2^-4 of it, or 2^-10; the quotient has a rounding of its own, which
    # may take it over a border
    near = torch.maximum(half_step(E4M3) * y.abs(), 2.0 ** -10 * s)
    assert torch.all(off <= near * (1 + 2.0 ** -20) + y.abs() * (slip + 2 * STEP32) * 1.01 + 2.0 ** -149)


def f8_values(codes, scales):
    """float64 [rows, K]; scales by row or by 128 rows."""
    s = scales.to(F)
    if scales.shape[0] != codes.shape[0]:
        s = s.repeat_interleave(128, 0)[:codes.shape[0]]
    return values(codes) * s.repeat_interleave(128, 1)[:, :codes.shape[1]]


def check_linear(y, x, xs, w, ws, bias):
    """y against the product in float64.

    The matrix unit adds the products of 8 neighbouring columns in units of 2^-13 of the largest one's power of
    two, cutting off what is below: (256 * 256, 2^e, -256 * 256) among 8 columns gives 2^e for e of 3 and more and
    0 below, and 1.75 * 2^3 gives 2^3.  So each of the 7 other products is off by less than 2^-13 of the largest.
    The sixteen sums of a block, the blocks, the product of two scales, bias and the output are binary32 and
    round as such, at most a step (2^-23) of what is added up."""
    a, b = f8_values(x, xs), f8_values(w, ws)
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    K = x.shape[1]
    tops = [torch.nn.functional.pad(v.abs(), (0, -K % 8)).view(v.shape[0], -1, 8).amax(-1) for v in (a, b)]
    cut = tops[0] @ tops[1].t() * 2.0 ** -13
    if bias is not None:
        want = want + bias.to(F)
        size = size + bias.to(F).abs()
    kb = -(-K // 128)
    bound = 7 * cut + size * (16 + kb + 20) * 2 * STEP32
    tiny = torch.finfo(y.dtype).smallest_normal * half_step(y.dtype)
    off = (y.to(F) - want).abs()
    assert torch.all(off <= bound * 1.01 + want.abs() * half_step(y.dtype) * 1.01 + tiny), (off - bound).max()
    # What is cut off has the signs of the products, and in their sum the size of a random walk: of K parts that
    # are even over 0 .. 2^-13 of a group's largest, sqrt(K / 3) / (K / 8) of `cut`.  Four times that over all results.
    if K >= 64 and y.numel() >= 4096:
        walk = (cut * (K / 3) ** 0.5 / (K / 8)).norm()
        assert off.norm() <= 4 * walk + want.norm() * half_step(y.dtype) + (size * (16 + kb + 20) * 2 * STEP32).norm()


def seen_of(bits, n):
    """bool [n, n] of one sequence's rows of int32 words."""
    a = torch.arange(n, device=bits.device)
    return (bits[:, a // 32] >> (a % 32) & 1).bool()


def attend_tree(q, cache, table, lens, bits, cu, window=0, sinks=0, scale=None):
    """(out, bound) as decode_ref.attend's, with each row's own set of tokens."""
    D = cache.head_dim
    scale = D ** -0.5 if scale is None else scale
    table = table.to(q.device)
    out = torch.zeros(q.shape, dtype=F, device=q.device)
    bound = torch.zeros_like(out)
    G = q.shape[1] // cache.kv_heads
    cap = table.shape[1] * cache.page_size
    for b in range(len(lens)):
        first, n, L = cu[b], cu[b + 1] - cu[b], min(max(lens[b], 0), cap)
        if n == 0 or L == 0:
            continue
        k, ok = cached(cache, table, b, L, "k")
        v, _ = cached(cache, table, b, L, "v")
        mine = seen_of(bits[first:first + n], n)
        c = L - n
        j = torch.arange(L, device=q.device)[None]
        seen = (j < c).expand(n, L).clone()
        if window:
            p = c + (mine & ~torch.eye(n, dtype=torch.bool, device=q.device)).sum(1, keepdim=True)
            seen &= (j > p - window) | (j < sinks)
        at = max(c, 0)
        seen[:, at:] = mine[:, at - c:]
        seen &= ok[None]
        used = seen.any(0)
        for h in range(q.shape[1]):
            kh, vh = (torch.where(used[:, None], x[h // G], torch.zeros_like(x[h // G])) for x in (k, v))
            x = q[first:first + n, h].to(F)
            z = (x @ kh.t()) * scale
            size = (x.abs() @ kh.abs().t()) * abs(scale)
            slip = torch.where(seen, size, torch.zeros_like(size)).amax(1, keepdim=True) * (D + 8) * STEP32
            w = torch.nan_to_num(torch.softmax(z.masked_fill(~seen, -math.inf), -1), nan=0.0)
            out[first:first + n, h] = w @ vh
            tiny = seen.sum(1, keepdim=True) * w.amax(1, keepdim=True) * 2.0 ** -25
            bound[first:first + n, h] = (2.0 ** -11 + 2.0 ** -18 + 2 * slip) * (w @ vh.abs()) + tiny * vh.abs().amax()
    return out, bound


def check_attend(got, ref, bound):
    assert got.shape == ref.shape
    off = (got.to(F) - ref).abs()
    tiny = torch.finfo(got.dtype).smallest_normal
    assert torch.all(off <= bound + half_step(got.dtype) * ref.abs() * 1.01 + tiny), (off - bound).max()


def keep(k, k_scale, table, past, kept, cu):
    """What one of K and V must hold: lists of (page, slot, value rows in units of the page's new scale,
    whether the codes are exactly the old ones), and scales, in float64.  `k` [pages, H, ps, D]."""
    ps, pages, H = k.shape[2], k.shape[0], k.shape[1]
    most = QMAX[k.dtype]
    val, scale = values(k), k_scale.to(F).clone()
    old = k_scale.to(F)
    rows = []
    page_at = lambda b, pos: int(table[b, pos // ps]) if 0 <= pos // ps < table.shape[1] else -1  # noqa: E731
    for b in range(len(past)):
        n = cu[b + 1] - cu[b]
        cap = table.shape[1] * ps
        p0 = min(max(past[b], 0), cap)
        upto = min(p0 + n, cap)
        for lo in range(p0 // ps * ps, upto, ps):
            if max(lo, p0) >= upto:
                continue
            page = page_at(b, lo)
            if not 0 <= page < pages:
                continue
            src = {}
            for pos in range(max(lo, p0), min(lo + ps, upto)):
                i = pos - p0
                of = kept[cu[b] + i]
                e = page_at(b, p0 + of) if of >= i else -1
                src[pos] = (page, pos % ps) if not 0 <= e < pages else (e, (p0 + of) % ps)
            s = old[page].clone()
            for e, slot in src.values():
                if e != page:
                    s = torch.maximum(s, val[e, :, slot].abs().amax(1) * old[e] / most)
            scale[page] = s
            for pos in range(lo, min(lo + ps, upto)):
                e, slot = src.get(pos, (page, pos % ps))
                same = old[e] == s
                ratio = torch.where(s > 0, old[e] / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(s))
                rows.append((page, pos % ps, val[e, :, slot] * ratio[:, None], same & (s > 0)))
    return rows, scale
