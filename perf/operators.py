"""What the decode operators are measured on: 4-bit linear layers, appending to a paged 8-bit cache, attention over it.

``run`` computes a case in plain torch operations, or, where ``own`` is true,
through the entry points of ``dense_fp16_gemm_hgemm_amd.decode``.

The layouts that both sides take:

* 4-bit weights: ``qweight`` int32 ``[NB, KB, 64, 4]`` with NB = ceil(N / 16) and
  KB = ceil(K / 128).  Word j of entry l = 16 c + r of tile (nb, kb) holds the
  codes 0..15 of row 16 nb + r at k = 128 kb + 32 j + 8 c + e, e = 0..7, at bit
  4 (e // 2) + 16 (e % 2).  ``scales`` ``[ceil(K / group), 16 NB]`` in x's type,
  ``zeros`` uint8 of the same shape, or None for 8 everywhere.
* the cache: ``k`` and ``v`` ``[pages, kv_heads, page_size, head_dim]`` int8 or
  float8_e4m3fn, ``k_scale`` and ``v_scale`` float32 ``[pages, kv_heads]``: a value
  is its code times its page's and head's scale.  Position p of sequence b is
  slot p % page_size of page ``table[b, p // page_size]``.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}


# ---------------------------------------------------------------- cases --

def _w4(name, M, N, K, group, dtype, zeros, bias=False):
    c = dict(op="w4", M=M, N=N, K=K, group=group, dtype=dtype, zeros=zeros, bias=bias)
    return dict(c, name=name) if name else c


def _append(name, B, past, new, Hq, Hkv, D, page, cache, dtype, interleaved=False):
    """`past` tokens at most lie in each sequence's cache, and up to `new` more come to each."""
    c = dict(op="append", B=B, past=past, new=new, Hq=Hq, Hkv=Hkv, D=D, page=page, cache=cache,
             dtype=dtype, interleaved=interleaved)
    return dict(c, name=name) if name else c


def _attend(name, B, L, ragged, tq, Hq, Hkv, D, page, cache, dtype, window=0, sinks=0):
    """Up to `tq` query tokens for each of B sequences of at most L tokens."""
    c = dict(op="attend", B=B, L=L, ragged=ragged, tq=tq, Hq=Hq, Hkv=Hkv, D=D, page=page,
             cache=cache, dtype=dtype, window=window, sinks=sinks)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token through a square projection: the least that a decode step waits for
        _w4("w4_token", 1, 4096, 4096, 128, "fp16", False),
        # a decode batch through the down projection, asymmetric codes
        _w4("w4_batch16_down", 16, 4096, 11008, 64, "bf16", True),
        # sizes that end inside every tile, the finest groups, a bias
        _w4("w4_odd", 7, 5003, 4072, 32, "fp16", True, True),
        # the most tokens that still count as few, through the widest projection
        _w4("w4_batch64_wide", 64, 14336, 4096, 128, "fp16", False),
        # one new token for each of a batch of conversations
        _append("append_token", 64, 1024, 1, 32, 8, 128, 64, "e4m3", "fp16"),
        # prompts of very different lengths, and the cached values read back
        _append("append_prompts", 8, 1000, 4096, 32, 8, 128, 64, "int8", "bf16"),
        # one conversation's next token
        _attend("attend_token", 1, 4096, False, 1, 32, 8, 128, 64, "int8", "fp16"),
        # a batch whose conversations are short and long
        _attend("attend_ragged", 64, 16384, True, 1, 32, 8, 128, 64, "e4m3", "bf16"),
        # the longest contexts: keys and values of over 4 GiB each
        _attend("attend_long", 32, 131072 + 77, False, 1, 32, 8, 128, 64, "int8", "bf16"),
        # a window of recent tokens with the first ones kept, small heads and pages
        _attend("attend_window", 64, 32768, True, 1, 64, 8, 64, 16, "int8", "fp16", 1000, 4),
        # a few drafted tokens are checked at once
        _attend("attend_verify", 24, 8192, True, 6, 64, 8, 128, 32, "e4m3", "fp16"),
        # a long prompt comes in pieces: the next piece attends to the cache so far
        _attend("attend_chunk", 2, 8192, False, 2048, 32, 8, 128, 64, "int8", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("w4", "w4", "append", "attend", "attend", "attend"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "w4":
        return _w4(None, rng.choice((1, 1, 2, 3, 4, 8, _log(rng, 1, 64))), _log(rng, 256, 32768),
                   8 * _log(rng, 32, 1400) if rng.random() < 0.8 else _log(rng, 256, 11200),
                   rng.choice((32, 64, 128, 256)), dtype, rng.random() < 0.5, rng.random() < 0.3)
    Hkv = rng.choice((1, 2, 4, 8))
    Hq = Hkv * rng.choice((1, 2, 4, 5, 7, 8))
    D = rng.choice((64, 128, 128, 256))
    page, cache = rng.choice((16, 32, 64, 128)), rng.choice(("int8", "e4m3"))
    if op == "append":
        if rng.random() < 0.5:
            return _append(None, _log(rng, 1, 128), _log(rng, 1, 1024), rng.choice((1, 1, 1, 3)), Hq,
                           Hkv, D, page, cache, dtype, rng.random() < 0.3)
        return _append(None, _log(rng, 1, 8), _log(rng, 1, 1000), _log(rng, 16, 4096), Hq, Hkv, D,
                       page, cache, dtype, rng.random() < 0.3)
    window, sinks = rng.choice(((0, 0), (0, 0), (_log(rng, 16, 4096), rng.choice((0, 1, 4, 40)))))
    form = rng.random()
    if form < 0.6:
        L = _log(rng, 1, 65536)
        B = _log(rng, 1, max(1, min(128, 2 ** 20 // L)))
        return _attend(None, B, L, rng.random() < 0.5, 1, Hq, Hkv, D, page, cache, dtype, window, sinks)
    if form < 0.8:
        return _attend(None, _log(rng, 1, 32), _log(rng, 8, 16384), rng.random() < 0.7,
                       rng.randint(2, 8), Hq, Hkv, D, page, cache, dtype, window, sinks)
    tq = _log(rng, 16, 1024)
    L = _log(rng, tq, 8192)
    B = rng.choice([b for b in (1, 2, 4) if b == 1 or b * tq * L * Hq * D <= 2 ** 37])
    return _attend(None, B, L, rng.random() < 0.5, tq, Hq, Hkv, D, page, cache, dtype, window, sinks)


def _lengths(case):
    """Cached and new tokens of each sequence: (past, new), by the case alone."""
    B = case["B"]
    r = random.Random(1000003 * B + 31 * case.get("L", case.get("past", 0)) + case.get("tq", case.get("new", 0)))
    if case["op"] == "append":
        if case["new"] <= 8:
            new = [case["new"] if i == 0 else r.randint(1, case["new"]) for i in range(B)]
        else:
            new = [case["new"] if i == 0 else _log(r, 1, case["new"]) for i in range(B)]
        past = [r.randint(0, case["past"]) for _ in range(B)]
        return past, new
    total = [case["L"] if i == 0 or not case["ragged"] else _log(r, 1, case["L"]) for i in range(B)]
    new = [min(t, case["tq"] if i == 0 or not case["ragged"] else r.randint(1, case["tq"]))
           for i, t in enumerate(total)]
    return [t - n for t, n in zip(total, new)], new


# --------------------------------------------------------------- inputs --

def _normal(shape, scale, dtype, gen, clamp=None, rounded=False):
    """Normal values in `dtype`, made in pieces."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat, step = out.view(-1), 1 << 27
    for at in range(0, flat.numel(), step):
        x = torch.randn(min(step, flat.numel() - at), device="cuda", generator=gen).mul_(scale)
        if clamp is not None:
            x.clamp_(-clamp, clamp)
        flat[at:at + step] = (x.round_() if rounded else x).to(dtype)
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = _TYPES[case["dtype"]]
    if case["op"] == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        nb, kb, groups = -(-N // 16), -(-K // 128), -(-K // case["group"])
        s = dict(case=case, x=_normal((M, K), 1.0, t, gen), zeros=None, bias=None)
        s["qweight"] = torch.randint(-2 ** 31, 2 ** 31, (nb, kb, 64, 4), device="cuda", generator=gen,
                                     dtype=torch.int32)
        s["scales"] = (torch.rand((groups, nb * 16), device="cuda", generator=gen) * 0.004 + 0.002).to(t)
        if case["zeros"]:
            s["zeros"] = torch.randint(5, 11, (groups, nb * 16), device="cuda", generator=gen, dtype=torch.uint8)
        if case["bias"]:
            s["bias"] = _normal((N,), 0.5, t, gen)
        return s
    past, new = _lengths(case)
    B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
    codes = _CODES[case["cache"]]
    total = [p + n for p, n in zip(past, new)]
    need = [-(-n // page) for n in total]
    pages = sum(need) + 3
    order = np.random.RandomState(seed % 2 ** 31).permutation(pages)
    table = np.full((B, max(need) + 1), -1, np.int32)  # entries past a sequence's end name no page
    at = 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    put = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(case=case, table=put(table), past=put(past), lens=put(total),
             cu=put([0] + list(np.cumsum(new))), max_new=max(new), max_len=max(total),
             spare=put(int(order[-1])))  # a page that belongs to no sequence
    most = _QMAX[codes]
    s["k"] = _normal((pages, Hkv, page, D), most / 3.6, codes, gen, most, codes == torch.int8)
    s["v"] = _normal((pages, Hkv, page, D), most / 3.6, codes, gen, most, codes == torch.int8)
    for n in ("k_scale", "v_scale"):  # unit-variance keys and values, pages of their own ranges
        s[n] = torch.exp(torch.randn((pages, Hkv), device="cuda", generator=gen) * 0.2) * (3.6 / most)
    if case["op"] == "append":
        T = sum(new)
        s["qkv"] = _normal((T, Hq + 2 * Hkv, D), 1.0, t, gen)  # one fused projection's result
        pos = torch.arange(max(table.shape[1] * page, 1), dtype=torch.float64, device="cuda")
        angle = pos[:, None] * _frequencies(D)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    else:
        s["q"] = _normal((sum(new), Hq, D), 1.0, t, gen)
    return s


def _frequencies(D):
    return 10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D)


# ---------------------------------------------------------- plain forms --

def _w4_plain(s):
    c = s["case"]
    e = torch.arange(8, device="cuda", dtype=torch.int32)
    q = (s["qweight"][..., None] >> (4 * (e // 2) + 16 * (e % 2))) & 15
    nb, kb = q.shape[:2]
    q = q.view(nb, kb, 4, 16, 4, 8).permute(0, 3, 1, 4, 2, 5).reshape(nb * 16, kb * 128)[:c["N"], :c["K"]]
    groups = torch.arange(c["K"], device="cuda") // c["group"]
    w = (q - (8 if s["zeros"] is None else s["zeros"].int().t()[:c["N"], groups])).float()
    w = w * s["scales"].float().t()[:c["N"], groups]
    y = s["x"].float() @ w.t()
    return (y if s["bias"] is None else y + s["bias"].float()).to(s["x"].dtype)


def _rotated(x, rope, pos, interleaved):
    half = x.shape[-1] // 2
    c, n = rope[pos][:, None, :half], rope[pos][:, None, half:]
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * c - b * n, b * c + a * n], -1)


def _to_codes(x, dtype):
    x = x.clamp(-_QMAX[dtype], _QMAX[dtype])
    return (x.round() if dtype == torch.int8 else x).to(dtype)


def _store(x, cache, scale, seq, pos, s):
    """x [T, Hkv, D] in 32 bits goes to position `pos` of sequence `seq`, and its pages' scales grow as they must."""
    ps = cache.shape[2]
    page = s["table"][seq, pos // ps].long()
    amax = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    fill = s["past"] % ps
    first = s["table"].gather(1, (s["past"] // ps).long()[:, None]).squeeze(1)
    first = torch.where(fill > 0, first, s["spare"]).long()  # the pages that hold tokens already
    old = torch.zeros_like(scale).index_copy_(0, first, scale[first])
    grown = torch.where(touched[:, None], torch.maximum(old, amax / _QMAX[cache.dtype]), scale)
    ratio = torch.where(grown > 0, old / grown, torch.ones_like(grown))[first][:, :, None, None]
    raw = cache.view(torch.int8)
    held = raw[first]
    again = _to_codes(held.view(cache.dtype).float() * ratio, cache.dtype).view(torch.int8)
    before = (torch.arange(ps, device="cuda") < fill[:, None])[:, None, :, None]
    raw[first] = torch.where(before & (ratio < 1) & touched[first][:, None, None, None], again, held)
    step = grown[page][:, :, None]
    new = _to_codes(torch.where(step > 0, x / step, torch.zeros_like(x)), cache.dtype)
    raw[page, :, pos % ps] = new.view(torch.int8)
    scale.copy_(grown)


def _places(s, tokens):
    """Each token's sequence, its place among the sequence's new tokens, and its position."""
    at = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    row = at - s["cu"][seq].long()
    return seq, row, row + s["past"][seq].long()


def _append_plain(s):
    c = s["case"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    qkv = s["qkv"]
    seq, _, pos = _places(s, qkv.shape[0])
    q = _rotated(qkv[:, :Hq], s["rope"], pos, c["interleaved"]).to(qkv.dtype)
    _store(_rotated(qkv[:, Hq:Hq + Hkv], s["rope"], pos, c["interleaved"]), s["k"], s["k_scale"], seq, pos, s)
    _store(qkv[:, Hq + Hkv:].float(), s["v"], s["v_scale"], seq, pos, s)
    out = {"q": q, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["cache"] == "e4m3":
        return dict(out, k=s["k"], v=s["v"])
    page = s["table"][seq, pos // c["page"]].long()
    for n in ("k", "v"):
        out[n] = (s[n][page, :, pos % c["page"]].float() * s[n + "_scale"][page][:, :, None]).to(qkv.dtype)
    return out


def _attend_plain(s):
    c = s["case"]
    q, page, ps = s["q"], s["table"].clamp(min=0).long(), c["page"]
    B, P = page.shape
    T, Hq, D = q.shape
    Hkv = c["Hkv"]
    seq, row, _ = _places(s, T)
    rows = torch.zeros((B, s["max_new"], Hq, D), device="cuda")
    rows[seq, row] = q.float()
    rows = rows.view(B, s["max_new"], Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    fetch = lambda n: (s[n].view(torch.int8)[page].view(s[n].dtype).float() * s[n + "_scale"][page][..., None, None]  # noqa: E731
                       ).transpose(1, 2).reshape(B, Hkv, P * ps, D)
    k = fetch("k")
    logits = (rows @ k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, s["max_new"], P * ps).mul_(D ** -0.5)
    del k
    at = torch.arange(P * ps, device="cuda")
    mine = (s["past"].long()[:, None] + torch.arange(s["max_new"], device="cuda"))[:, :, None]
    seen = at <= mine
    if c["window"]:
        seen &= (at > mine - c["window"]) | (at < c["sinks"])
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    p = (logits - logits.amax(-1, keepdim=True)).exp_()
    del logits
    p /= p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, -1, P * ps) @ fetch("v")
    o = o.view(B, Hkv, Hq // Hkv, s["max_new"], D).permute(0, 3, 1, 2, 4).reshape(B, s["max_new"], Hq, D)
    return o[seq, row].to(q.dtype)


# ------------------------------------------------------------------ run --

_kept = {}


def _decode():
    """The module and the handle that a program makes once."""
    if not _kept:
        from dense_fp16_gemm_hgemm_amd import decode
        _kept["module"], _kept["handle"] = decode, decode.Decode()
    return _kept["module"], _kept["handle"]


def run(state):
    c = state["case"]
    if own:
        module, d = _decode()
        if c["op"] == "w4":
            return d.w4_linear(state["x"], state["qweight"], state["scales"], state["zeros"], n=c["N"],
                               group=c["group"], bias=state["bias"])
        if "cache" not in state:  # the cache object that a program keeps beside its buffers
            state["cache"] = module.KvCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        cache = state["cache"]
        if c["op"] == "attend":
            return d.kv_attend(state["q"], cache, state["table"], state["lens"],
                               cu_q=state["cu"], max_q=state["max_new"], max_len=state["max_len"],
                               window=c["window"], sinks=c["sinks"])
        Hq, Hkv, qkv = c["Hq"], c["Hkv"], state["qkv"]
        q = d.kv_append(cache, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], state["table"], state["past"],
                        cu_new=state["cu"], max_new=state["max_new"], q=qkv[:, :Hq], rope=state["rope"],
                        interleaved=c["interleaved"])
        out = {"q": q, "k_scale": state["k_scale"], "v_scale": state["v_scale"]}
        if c["cache"] == "e4m3":
            return dict(out, k=state["k"], v=state["v"])
        k, v = d.kv_read(cache, state["table"], state["past"], state["cu"], tokens=qkv.shape[0],
                         max_tokens=state["max_new"], dtype=qkv.dtype)
        return dict(out, k=k, v=v)
    return {"w4": _w4_plain, "append": _append_plain, "attend": _attend_plain}[c["op"]](state)


def work(case):
    if case["op"] == "w4":
        M, N, K = case["M"], case["N"], case["K"]
        groups = -(-K // case["group"])
        return {"bytes": N * K / 2 + N * groups * (3 if case["zeros"] else 2) + 2 * M * K + 2 * M * N
                + (2 * N if case["bias"] else 0), "flops": 2.0 * M * N * K}
    past, new = _lengths(case)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    T = sum(new)
    if case["op"] == "append":
        # q, k and v come and q goes in 16 bits, codes go in 8; int8 codes are read back as 16-bit values
        return {"bytes": T * D * (4 * Hq + 4 * Hkv + 2 * Hkv + (6 * Hkv if case["cache"] == "int8" else 0))
                + 4 * D * max(p + n for p, n in zip(past, new)), "flops": 3.0 * T * (Hq + Hkv) * D}
    w, sinks = case["window"], case["sinks"]
    seen = read = 0
    for p, n in zip(past, new):
        for i in (range(n) if w else ()):
            at = p + i + 1
            seen += at if at <= w + sinks else w + sinks
        if not w:
            seen += n * p + n * (n + 1) // 2
        read += p + n if not w else min(p + n, w + n - 1 + sinks)
    return {"bytes": read * Hkv * D * 2 + 4 * T * Hq * D, "flops": 4.0 * seen * Hq * D}


# ---------------------------------------------------------------- exact --

def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "w4":
        N, K, g = case["N"], case["K"], case["group"]
        words = s["qweight"].long() & 0xFFFFFFFF
        w = torch.empty((words.shape[0] * 16, words.shape[1] * 128), dtype=f, device="cuda")
        tiles = w.view(words.shape[0], 16, words.shape[1], 4, 4, 8)  # nb, r, kb, j, c, e
        for c in range(4):
            for e in range(8):
                nibble = (words[:, :, 16 * c:16 * c + 16] >> (4 * (e >> 1) + 16 * (e & 1))) % 16
                tiles[:, :, :, :, c, e] = nibble.permute(0, 2, 1, 3).to(f)
        w = w[:N, :K]
        for i in range(0, K, g):
            zero = 8.0 if s["zeros"] is None else s["zeros"][i // g, :N].to(f)[:, None]
            w[:, i:i + g] = (w[:, i:i + g] - zero) * s["scales"][i // g, :N].to(f)[:, None]
        y = s["x"].to(f) @ w.t()
        return y if s["bias"] is None else y + s["bias"].to(f)
    past, new = _lengths(case)
    table, ps, Hq, Hkv, D = s["table"].cpu(), case["page"], case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "append":
        freq, most, T = _frequencies(D), _QMAX[s["k"].dtype], sum(new)
        out = {"q": torch.empty((T, Hq, D), dtype=f, device="cuda")}
        vals = {n: s[n].to(f) for n in ("k", "v")}
        scales = {n: s[n + "_scale"].to(f) for n in ("k", "v")}
        rows = {n: torch.empty((T, Hkv, D), dtype=f, device="cuda") for n in ("k", "v")}

        def coded(x):
            x = x.clamp(-most, most)
            if case["cache"] == "int8":
                return torch.round(x)
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            return torch.round(x / step) * step

        at = 0
        for b in range(case["B"]):
            x = s["qkv"][at:at + new[b]].to(f)
            angle = (past[b] + torch.arange(new[b], dtype=f, device="cuda"))[:, None] * freq
            turn = torch.polar(torch.ones_like(angle), angle)[:, None]
            both = x[:, :Hq + Hkv]
            if case["interleaved"]:
                z = torch.view_as_complex(both.reshape(new[b], Hq + Hkv, D // 2, 2).contiguous()) * turn
                both = torch.view_as_real(z).reshape(new[b], Hq + Hkv, D)
            else:
                z = torch.complex(both[..., :D // 2].contiguous(), both[..., D // 2:].contiguous()) * turn
                both = torch.cat([z.real, z.imag], -1)
            out["q"][at:at + new[b]] = both[:, :Hq]
            for n, y in (("k", both[:, Hq:]), ("v", x[:, Hq + Hkv:])):
                y = y.transpose(0, 1)
                for lo in range(past[b] - past[b] % ps, past[b] + new[b], ps):
                    p = int(table[b, lo // ps])
                    i, j = max(lo, past[b]), min(lo + ps, past[b] + new[b])
                    part = y[:, i - past[b]:j - past[b]]
                    sc = part.abs().amax((1, 2)) / most
                    if i > lo:
                        was = scales[n][p].clone()
                        sc = torch.maximum(sc, was)
                        held = vals[n][p, :, :i - lo]
                        vals[n][p, :, :i - lo] = torch.where((sc > was)[:, None, None],
                                                             coded(held * (was / sc)[:, None, None]), held)
                    scales[n][p] = sc
                    vals[n][p, :, i - lo:j - lo] = coded(part / sc[:, None, None])
                    rows[n][at + i - past[b]:at + j - past[b]] = (
                        vals[n][p, :, i - lo:j - lo] * sc[:, None, None]).transpose(0, 1)
            at += new[b]
        keep = vals if case["cache"] == "e4m3" else rows
        return dict(out, k=keep["k"], v=keep["v"], k_scale=scales["k"], v_scale=scales["v"])
    if sum(new) * Hq * max(p + n for p, n in zip(past, new)) > 2 ** 34:
        return None
    out = torch.empty((sum(new), Hq, D), dtype=f, device="cuda")
    at = 0
    for b in range(case["B"]):
        total = past[b] + new[b]
        pages = table[b, :-(-total // ps)].long().cuda()
        get = lambda n: (s[n].view(torch.int8)[pages].view(s[n].dtype).to(f) * s[n + "_scale"][pages].to(f)[:, :, None, None]  # noqa: E731
                         ).transpose(0, 1).reshape(Hkv, -1, D)[:, :total]
        k, v = get("k"), get("v")
        mine = torch.arange(past[b], total, device="cuda")[:, None]
        at_k = torch.arange(total, device="cuda")[None]
        hidden = at_k > mine
        if case["window"]:
            hidden = hidden | ((at_k + case["window"] <= mine) & (at_k >= case["sinks"]))
        for h in range(Hkv):
            for j in range(h * (Hq // Hkv), (h + 1) * (Hq // Hkv)):
                z = (s["q"][at:at + new[b], j].to(f) @ k[h].t()) / math.sqrt(D)
                out[at:at + new[b], j] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[h]
        at += new[b]
    return out
