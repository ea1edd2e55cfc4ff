"""64-bit references of the decode operators, from their definitions, and the tolerances."""
import math

import torch

F = torch.float64
QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def values(codes):
    """Codes as float64 (float8 through float32, exactly)."""
    return codes.to(F) if codes.dtype == torch.int8 else codes.float().to(F)


def take_pages(buf, pages):
    return buf.view(torch.uint8)[pages].view(buf.dtype)


def random_codes(shape, dtype, gen, device="cuda"):
    if dtype == torch.int8:
        return torch.randint(-127, 128, shape, generator=gen, device=device, dtype=torch.int8)
    x = torch.randn(shape, generator=gen, device=device) * 120
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def cached(cache, table, b, length, which):
    """float64 [kv_heads, length, head_dim] of sequence b, and which positions have a valid page."""
    ps = cache.page_size
    cols = table[b, : -(-length // ps)].long()
    ok = (cols >= 0) & (cols < cache.pages)
    idx = cols.clamp(0, cache.pages - 1)
    buf, sc = getattr(cache, which), getattr(cache, which + "_scale")
    x = values(take_pages(buf, idx)) * sc[idx].to(F)[:, :, None, None]
    x = torch.where(ok[:, None, None, None], x, torch.zeros_like(x))
    return x.transpose(0, 1).reshape(cache.kv_heads, -1, cache.head_dim)[:, :length], ok.repeat_interleave(ps)[:length]


def attend(q, cache, table, lens, cu, window=0, sinks=0, scale=None):
    """(out, bound): float64 attention, and how far a kernel may be from it before its own rounding.

    A kernel rounds each softmax weight to fp16 (half a step, 2^-11 of the weight, or 2^-25 of the
    largest one where the weight is that small), and its logits carry the rounding of a dot
    product of head_dim terms in binary32; 2^-18 covers the exponentials and the sums."""
    D = cache.head_dim
    scale = D ** -0.5 if scale is None else scale
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
        p = torch.arange(n, device=q.device)[:, None] + (L - n)
        j = torch.arange(L, device=q.device)[None]
        seen = (j <= p) & ok[None]
        if window:
            seen &= (j > p - window) | (j < sinks)
        for h in range(q.shape[1]):
            kh, vh = k[h // G], v[h // G]
            used = seen.any(0)
            kh, vh = torch.where(used[:, None], kh, torch.zeros_like(kh)), torch.where(used[:, None], vh, torch.zeros_like(vh))
            x = q[first:first + n, h].to(F)
            z = (x @ kh.t()) * scale
            size = (x.abs() @ kh.abs().t()) * abs(scale)
            slip = torch.where(seen, size, torch.zeros_like(size)).amax(1, keepdim=True) * (D + 8) * 2.0 ** -24
            z = z.masked_fill(~seen, -math.inf)
            w = torch.nan_to_num(torch.softmax(z, -1), nan=0.0)
            out[first:first + n, h] = w @ vh
            tiny = seen.sum(1, keepdim=True) * w.amax(1, keepdim=True) * 2.0 ** -25
            bound[first:first + n, h] = (2.0 ** -11 + 2.0 ** -18 + 2 * slip) * (w @ vh.abs()) + tiny * vh.abs().amax()
    return out, bound


def rotate(x, pos, freq, interleaved):
    """x [T, heads, D] in float64, its first 2 * len(freq) channels turned by pos * freq."""
    half = freq.shape[0]
    angle = pos.to(F)[:, None] * freq
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    r, rest = x[..., :2 * half].to(F), x[..., 2 * half:].to(F)
    if interleaved:
        z = torch.complex(r[..., 0::2].contiguous(), r[..., 1::2].contiguous()) * turn
        r = torch.stack([z.real, z.imag], -1).flatten(-2)
    else:
        z = torch.complex(r[..., :half].contiguous(), r[..., half:].contiguous()) * turn
        r = torch.cat([z.real, z.imag], -1)
    return torch.cat([r, rest], -1)


def layout(lens, page, pages, gen, extra_cols=0, fill=-1):
    """A page table (int32, CPU) for sequences of these lengths over randomly chosen pages."""
    need = [-(-max(n, 0) // page) for n in lens]
    assert sum(need) <= pages
    order = torch.randperm(pages, generator=gen).tolist()
    cols = max(need + [1]) + extra_cols
    table = torch.full((len(lens), cols), fill, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table
