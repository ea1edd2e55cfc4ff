"""What the operators of a step that verifies drafted tokens are measured on.

Norms with 8-bit outputs, products of 8-bit floats with block scales, attention for trees of
drafted tokens, and what moves tokens and pages of the cache.  ``run`` computes a case in plain
torch operations, or, where ``own`` is true, through the entry points of
``dense_fp16_gemm_hgemm_amd.decode``.

The layouts that both sides take:

* 8-bit floats: e4m3 codes ``[rows, K]``; activations have a float32 scale for each row and 128
  columns, ``[M, ceil(K / 128)]``, weights one for each 128 rows and 128 columns,
  ``[ceil(N / 128), ceil(K / 128)]``.  A value is its code times its scale.
* the cache: ``k`` and ``v`` ``[pages, kv_heads, page_size, head_dim]`` int8 or
  float8_e4m3fn, ``k_scale`` and ``v_scale`` float32 ``[pages, kv_heads]``.  Position p of
  sequence b is slot p % page_size of page ``table[b, p // page_size]``.
* drafted tokens: the last n of a sequence's tokens in the cache.  Bit a % 32 of word a // 32 of
  ``seen[t]`` (int32) says that token t sees its sequence's drafted token a.
"""
import math
import random

import numpy as np
import torch

own = False

_TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
_CODES = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
_QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
_BLOCK = 128
_EPS = 1e-6


# ---------------------------------------------------------------- cases --

def _named(name, c):
    return dict(c, name=name) if name else c


def _norm(name, M, K, dtype, residual, weight=True):
    return _named(name, dict(op="norm", M=M, K=K, dtype=dtype, residual=residual, weight=weight))


def _linear(name, M, N, K, dtype, bias=False):
    return _named(name, dict(op="linear", M=M, N=N, K=K, dtype=dtype, bias=bias))


def _tree(name, B, L, n, ragged, Hq, Hkv, D, page, cache, dtype, window=0, sinks=0):
    """Up to `n` drafted tokens for each of B sequences of at most L tokens before them."""
    return _named(name, dict(op="tree", B=B, L=L, n=n, ragged=ragged, Hq=Hq, Hkv=Hkv, D=D, page=page, cache=cache,
                             dtype=dtype, window=window, sinks=sinks))


def _keep(name, B, L, n, Hkv, D, page, cache):
    """Of up to `n` drafted tokens of each of B sequences one path is kept."""
    return _named(name, dict(op="keep", B=B, L=L, n=n, Hkv=Hkv, D=D, page=page, cache=cache))


def _copy(name, pages, pairs, Hkv, D, page, cache):
    return _named(name, dict(op="copy", pages=pages, pairs=pairs, Hkv=Hkv, D=D, page=page, cache=cache))


def listed():
    return [
        # one token before a projection: latency
        _norm("norm_token", 1, 4096, "fp16", True),
        # a long prompt's tokens between two layers
        _norm("norm_prompt", 8192, 4096, "bf16", True),
        # one token through a square projection: the least that a step waits for
        _linear("f8_token", 1, 4096, 4096, "fp16"),
        # sizes that end inside every tile, with a bias
        _linear("f8_odd", 77, 5003, 4072, "bf16", True),
        # the drafted tokens of a batch through the widest projection
        _linear("f8_drafts", 512, 14336, 4096, "fp16"),
        # a long prompt through the down projection
        _linear("f8_prompt", 8192, 4096, 11008, "bf16"),
        # one conversation's small tree
        _tree("tree_one", 1, 4096, 12, False, 32, 8, 128, 64, "int8", "fp16"),
        # trees of a batch whose conversations are short and long
        _tree("tree_batch", 32, 12000, 64, True, 32, 8, 128, 64, "e4m3", "bf16"),
        # one conversation's accepted path
        _keep("keep_one", 1, 4096, 12, 8, 128, 64, "e4m3"),
        # the accepted paths of a large batch of deep trees, over small pages
        _keep("keep_batch", 128, 2000, 64, 8, 128, 16, "e4m3"),
        # one conversation is forked: its last page
        _copy("copy_fork", 500, 1, 8, 128, 64, "e4m3"),
        # the pages of a long context move together
        _copy("copy_context", 5000, 2048, 8, 128, 64, "e4m3"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "tree", "tree", "keep", "copy"))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "norm":
        K = 8 * _log(rng, 16, 2048) if rng.random() < 0.8 else _log(rng, 100, 16384)
        return _norm(None, _log(rng, 1, min(8192, 2 ** 25 // K)), K, dtype, rng.random() < 0.7, rng.random() < 0.8)
    if op == "linear":
        N = _log(rng, 256, 16384)
        K = 16 * _log(rng, 16, 768) if rng.random() < 0.85 else _log(rng, 256, 12288)
        M = min(_log(rng, 1, 8192), int(3.5e11 // (N * K)))
        return _linear(None, max(1, M), N, K, dtype, rng.random() < 0.3)
    Hkv = rng.choice((1, 2, 4, 8))
    D = rng.choice((64, 128, 128, 256))
    page, cache = rng.choice((16, 32, 64, 128)), rng.choice(("int8", "e4m3"))
    if op == "tree":
        Hq = Hkv * rng.choice((1, 2, 4, 5, 7, 8))
        window, sinks = rng.choice(((0, 0), (0, 0), (_log(rng, 16, 4096), rng.choice((0, 1, 4, 40)))))
        n, L = _log(rng, 1, 130), _log(rng, 1, 16384)
        B = _log(rng, 1, max(1, min(64, 2 ** 29 // (n * Hq * (L + n)))))
        return _tree(None, B, L, n, rng.random() < 0.6, Hq, Hkv, D, page, cache, dtype, window, sinks)
    if op == "keep":
        return _keep(None, _log(rng, 1, 128), _log(rng, 1, 2000), _log(rng, 2, 130), Hkv, D, page, cache)
    pairs = _log(rng, 1, 1024)
    return _copy(None, pairs * 2 + _log(rng, 1, 1000), pairs, Hkv, D, page, cache)


def _drafts(case):
    """Of each sequence, by the case alone: tokens before the drafts, which drafted token sees which, and one path."""
    r = random.Random(1000003 * case["B"] + 31 * case["L"] + case["n"])
    past, trees, paths = [], [], []
    for b in range(case["B"]):
        whole = b == 0 or not case.get("ragged", True)
        past.append(case["L"] if whole else _log(r, 1, case["L"]))
        n = case["n"] if whole else r.randint(1, case["n"])
        sees, parent = np.eye(n, dtype=bool), [-1] * n
        for i in range(1, n):
            parent[i] = r.randint(max(-1, i - 9), i - 1)
            if parent[i] >= 0:
                sees[i] |= sees[parent[i]]
        trees.append(sees)
        depth = sees.sum(1)
        leaf = int(depth.argmax()) if b % 2 == 0 else r.randrange(n)
        paths.append(np.flatnonzero(sees[leaf]).tolist())
    return past, trees, paths


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


def _around(shape, middle, gen):
    """Positive scales of different sizes."""
    return torch.exp(torch.randn(shape, device="cuda", generator=gen) * 0.3) * middle


def _put(a):
    return torch.tensor(np.asarray(a, dtype=np.int64), device="cuda").to(torch.int32)


def _words(sees, words):
    """A boolean matrix as int32 words, 32 columns each."""
    bits = np.zeros((sees.shape[0], words * 32), dtype=np.uint8)
    bits[:, :sees.shape[1]] = sees
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32).reshape(-1, words)


def _cache(s, case, pages, gen):
    codes = _CODES[case["cache"]]
    most, shape = _QMAX[codes], (pages, case["Hkv"], case["page"], case["D"])
    for n in ("k", "v"):  # unit-variance keys and values, pages of their own ranges
        s[n] = _normal(shape, most / 3.6, codes, gen, most, codes == torch.int8)
        s[n + "_scale"] = _around(shape[:2], 3.6 / most, gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        M, K, t = case["M"], case["K"], _TYPES[case["dtype"]]
        s["x"] = _normal((M, K), 0.3, t, gen)
        s["residual"] = _normal((M, K), 2.0, t, gen) if case["residual"] else None
        s["weight"] = (1 + _normal((K,), 0.2, torch.float32, gen)).to(t) if case["weight"] else None
        return s
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // _BLOCK)
        s["x"] = _normal((M, K), 120.0, torch.float8_e4m3fn, gen, 448.0)
        s["w"] = _normal((N, K), 120.0, torch.float8_e4m3fn, gen, 448.0)
        s["x_scale"] = _around((M, kb), 1 / 120, gen)
        s["w_scale"] = _around((-(-N // _BLOCK), kb), K ** -0.5 / 120, gen)
        s["bias"] = _normal((N,), 0.5, _TYPES[case["dtype"]], gen) if case["bias"] else None
        return s
    order = np.random.RandomState(seed % 2 ** 31)
    if case["op"] == "copy":
        _cache(s, case, case["pages"], gen)
        pages = order.permutation(case["pages"])
        src, dst = pages[:case["pairs"]], pages[case["pairs"]:2 * case["pairs"]]
        src[order.rand(case["pairs"]) < 0.1] = src[0]  # a page that several conversations go on from
        s["src"], s["dst"] = _put(src), _put(dst)
        return s
    past, trees, paths = _drafts(case)
    total = [p + len(t) for p, t in zip(past, trees)]
    need = [-(-n // case["page"]) for n in total]
    pages = sum(need) + 3
    order = order.permutation(pages)
    table = np.full((case["B"], max(need) + 1), -1, np.int32)  # entries past a sequence's end name no page
    at = 0
    for b in range(case["B"]):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    _cache(s, case, pages, gen)
    s.update(table=_put(table), past=_put(past), lens=_put(total))
    if case["op"] == "keep":
        s.update(keep=_put(sum(paths, [])), cu=_put([0] + list(np.cumsum([len(p) for p in paths]))),
                 max_new=max(map(len, paths)), tokens=sum(map(len, paths)))
        return s
    n = max(map(len, trees))
    s.update(cu=_put([0] + list(np.cumsum([len(t) for t in trees]))), max_new=n, max_len=max(total),
             seen=torch.from_numpy(np.concatenate([_words(t, -(-n // 32)) for t in trees])).cuda(),
             q=_normal((sum(map(len, trees)), case["Hq"], case["D"]), 1.0, _TYPES[case["dtype"]], gen))
    return s


# ---------------------------------------------------------- plain forms --

def _norm_plain(s):
    x = s["x"]
    if s["residual"] is not None:
        x = (x.float() + s["residual"].float()).to(x.dtype)
    M, K = x.shape
    h = x.float()
    y = h / (h.square().mean(1, keepdim=True) + _EPS).sqrt()
    if s["weight"] is not None:
        y = y * s["weight"].float()
    kb = -(-K // _BLOCK)
    blocks = torch.zeros((M, kb * _BLOCK), device="cuda")
    blocks[:, :K] = y
    blocks = blocks.view(M, kb, _BLOCK)
    scale = blocks.abs().amax(-1) / 448.0
    codes = torch.where(scale[..., None] > 0, blocks / scale[..., None], torch.zeros_like(blocks)).clamp(-448, 448)
    return {"codes": codes.view(M, -1)[:, :K].to(torch.float8_e4m3fn), "scales": scale,
            "total": None if s["residual"] is None else x}


def _linear_plain(s):
    x, w = s["x"], s["w"]
    k = torch.arange(x.shape[1], device="cuda") // _BLOCK
    n = torch.arange(w.shape[0], device="cuda") // _BLOCK
    y = (x.float() * s["x_scale"][:, k]) @ (w.float() * s["w_scale"][n][:, k]).t()
    if s["bias"] is not None:
        y += s["bias"].float()
    return y.to(_TYPES[s["case"]["dtype"]])


def _places(s, tokens):
    """Each token's sequence, and its place among the sequence's tokens of the call."""
    at = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), at, right=True)
    return seq, at - s["cu"][seq].long()


def _tree_plain(s):
    c = s["case"]
    q, page, ps, Hkv, most = s["q"], s["table"].clamp(min=0).long(), c["page"], c["Hkv"], s["max_new"]
    B, P = page.shape
    T, Hq, D = q.shape
    seq, row = _places(s, T)
    rows = torch.zeros((B, most, Hq, D), device="cuda")
    rows[seq, row] = q.float()
    rows = rows.view(B, most, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    fetch = lambda n: (s[n].view(torch.int8)[page].view(s[n].dtype).float() * s[n + "_scale"][page][..., None, None]  # noqa: E731
                       ).transpose(1, 2).reshape(B, Hkv, P * ps, D)
    k = fetch("k")
    logits = (rows @ k.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, most, P * ps).mul_(D ** -0.5)
    del k
    bit = torch.arange(most, device="cuda")
    sees = torch.zeros((B, most, most), dtype=torch.bool, device="cuda")
    sees[seq, row] = (s["seen"][:, bit // 32] >> (bit % 32) & 1).bool()
    at = torch.arange(P * ps, device="cuda")
    past = s["past"].long()[:, None, None]
    seen = (at < past).expand(B, most, P * ps)
    if c["window"]:  # a token stands as far behind the context as it sees other drafted tokens
        mine = past + (sees & (bit[:, None] != bit)).sum(-1, keepdim=True)
        seen = seen & ((at > mine - c["window"]) | (at < c["sinks"]))
    draft = (at - past).expand(B, most, P * ps)
    seen = seen | ((draft >= 0) & (draft < most) & sees.gather(2, draft.clamp(0, most - 1)))
    logits.masked_fill_(~seen[:, None, None], -math.inf)
    p = (logits - logits.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    del logits
    p /= p.sum(-1, keepdim=True)
    o = p.view(B, Hkv, -1, P * ps) @ fetch("v")
    o = o.view(B, Hkv, Hq // Hkv, most, D).permute(0, 3, 1, 2, 4).reshape(B, most, Hq, D)
    return o[seq, row].to(q.dtype)


def _to_codes(x, dtype):
    x = x.clamp(-_QMAX[dtype], _QMAX[dtype])
    return (x.round() if dtype == torch.int8 else x).to(dtype)


def _keep_plain(s):
    c = s["case"]
    ps, T = c["page"], s["tokens"]
    seq, j = _places(s, T)
    past, table = s["past"].long(), s["table"].long()
    to, of = past[seq] + j, past[seq] + s["keep"].long()
    dp, sp = table[seq, to // ps], table[seq, of // ps]
    comes = (dp != sp)[:, None]  # from another page, with its scale
    kept = past + (s["cu"][1:] - s["cu"][:-1]).long()
    place = torch.arange(table.shape[1] * ps, device="cuda")
    held = (place >= (past // ps * ps)[:, None]) & (place < kept[:, None])  # what the written pages hold afterwards
    hseq, hpos = held.nonzero(as_tuple=True)
    for n in ("k", "v"):
        cache, scale = s[n], s[n + "_scale"]
        raw, old = cache.view(torch.int8), scale.clone()
        moved = raw[sp, :, of % ps].view(cache.dtype).float()
        amax = torch.where(comes, moved.abs().amax(-1) * old[sp], torch.zeros_like(old[sp])) / _QMAX[cache.dtype]
        scale.scatter_reduce_(0, dp[:, None].expand(-1, c["Hkv"]), amax, "amax")
        hp = table[hseq, hpos // ps]
        ratio = torch.where(scale[hp] > 0, old[hp] / scale[hp], torch.ones_like(old[hp]))[..., None]
        now = raw[hp, :, hpos % ps]
        again = _to_codes(now.view(cache.dtype).float() * ratio, cache.dtype).view(torch.int8)
        raw[hp, :, hpos % ps] = torch.where(ratio < 1, again, now)
        ratio = torch.where(scale[dp] > 0, old[sp] / scale[dp], torch.ones_like(old[dp]))[..., None]
        new = _to_codes(moved * ratio, cache.dtype).view(torch.int8)
        raw[dp, :, to % ps] = torch.where(ratio != 1, new, moved.to(cache.dtype).view(torch.int8))
    out = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["cache"] == "e4m3":
        return dict(out, k=s["k"], v=s["v"])
    for n in ("k", "v"):
        out[n] = (s[n][dp, :, to % ps].float() * s[n + "_scale"][dp][:, :, None]).to(torch.float16)
    return out


def _copy_plain(s):
    src, dst = s["src"].long(), s["dst"].long()
    for n in ("k", "v"):
        raw = s[n].view(torch.int8)
        raw[dst] = raw[src]
        s[n + "_scale"][dst] = s[n + "_scale"][src]
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}


# ------------------------------------------------------------------ run --

_kept = {}


def _decode():
    """The module and the handle that a program makes once."""
    if not _kept:
        from dense_fp16_gemm_hgemm_amd import decode
        _kept["module"], _kept["handle"] = decode, decode.Decode()
    return _kept["module"], _kept["handle"]


def _own(s):
    c = s["case"]
    module, d = _decode()
    if c["op"] == "norm":
        codes, scales, total = d.rms_norm_f8(s["x"], s["weight"], s["residual"], eps=_EPS)
        return {"codes": codes, "scales": scales, "total": total}
    if c["op"] == "linear":
        return d.f8_linear(s["x"], s["x_scale"], s["w"], s["w_scale"], bias=s["bias"], dtype=_TYPES[c["dtype"]])
    if "cache" not in s:  # the cache object that a program keeps beside its buffers
        s["cache"] = module.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    cache = s["cache"]
    if c["op"] == "tree":
        return d.kv_attend_tree(s["q"], cache, s["table"], s["lens"], s["seen"], cu_q=s["cu"], max_q=s["max_new"],
                                max_len=s["max_len"], window=c["window"], sinks=c["sinks"])
    if c["op"] == "copy":
        d.kv_copy(cache, s["src"], s["dst"])
        return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}
    d.kv_keep(cache, s["table"], s["past"], s["keep"], s["cu"], max_keep=s["max_new"])
    out = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    if c["cache"] == "e4m3":
        return dict(out, k=s["k"], v=s["v"])
    k, v = d.kv_read(cache, s["table"], s["past"], s["cu"], tokens=s["tokens"], max_tokens=s["max_new"])
    return dict(out, k=k, v=v)


def run(state):
    if own:
        return _own(state)
    return {"norm": _norm_plain, "linear": _linear_plain, "tree": _tree_plain, "keep": _keep_plain,
            "copy": _copy_plain}[state["case"]["op"]](state)


def work(case):
    if case["op"] == "norm":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * (7 if case["residual"] else 3) + 4 * M * -(-K // _BLOCK) + (2 * K if case["weight"] else 0),
                "flops": 8.0 * M * K}
    if case["op"] == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        kb = -(-K // _BLOCK)
        return {"bytes": M * K + N * K + 2 * M * N + 4 * kb * (M + -(-N // _BLOCK)) + (2 * N if case["bias"] else 0),
                "flops": 2.0 * M * N * K}
    row = 2 * case["Hkv"] * case["D"]  # a token's key and value codes
    if case["op"] == "copy":
        return {"bytes": 2.0 * case["pairs"] * (case["page"] * row + 8 * case["Hkv"]), "flops": 0.0}
    past, trees, paths = _drafts(case)
    if case["op"] == "keep":
        moved = sum(k != j for p in paths for j, k in enumerate(p))
        return {"bytes": 2.0 * moved * row + 8.0 * case["B"] * case["Hkv"] + 4.0 * sum(map(len, paths)), "flops": 0.0}
    w, sinks = case["window"], case["sinks"]
    pairs = read = tokens = 0
    for p, t in zip(past, trees):
        tokens += len(t)
        read += len(t) + (min(p, w - 1 + sinks) if w else p)
        before = [p] * len(t) if not w else [min(p, max(0, w - int(d)) + min(sinks, max(0, p - max(0, w - int(d)))))
                                             for d in t.sum(1)]
        pairs += sum(before) + int(t.sum())
    return {"bytes": float(read * row + 4 * tokens * case["Hq"] * case["D"]), "flops": 4.0 * pairs * case["Hq"] * case["D"]}


# ---------------------------------------------------------------- exact --

def _e4m3(x):
    """The nearest numbers of three bits after the leading one, ties to even, down to steps of 2^-9."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(x.clamp(-448, 448) / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(f)
        if case["residual"]:
            h = (h + s["residual"].to(f)).to(s["x"].dtype).to(f)
        y = h * torch.rsqrt((h * h).sum(1, keepdim=True) / case["K"] + _EPS)
        if case["weight"]:
            y = y * s["weight"].to(f)
        codes, scales = torch.empty_like(y), []
        for i in range(0, case["K"], _BLOCK):
            part = y[:, i:i + _BLOCK]
            scales.append(part.abs().amax(1) / 448)
            codes[:, i:i + _BLOCK] = _e4m3(torch.nan_to_num(part / scales[-1][:, None], nan=0.0))
        return {"codes": codes, "scales": torch.stack(scales, 1), "total": h if case["residual"] else None}
    if case["op"] == "linear":
        y = torch.zeros((case["M"], case["N"]), dtype=f, device="cuda")
        ws = s["w_scale"].to(f).repeat_interleave(_BLOCK, 0)[:case["N"]]
        for j, i in enumerate(range(0, case["K"], _BLOCK)):
            a = s["x"][:, i:i + _BLOCK].to(f) * s["x_scale"][:, j:j + 1].to(f)
            y += a @ (s["w"][:, i:i + _BLOCK].to(f) * ws[:, j:j + 1]).t()
        return y if s["bias"] is None else y + s["bias"].to(f)
    if case["op"] == "copy":
        src, dst = s["src"].tolist(), s["dst"].tolist()
        out = {n: s[n].to(f) for n in ("k", "v", "k_scale", "v_scale")}
        for n, x in out.items():
            of = s[n]
            for a, b in zip(src, dst):
                x[b] = of[a].to(f)
        return out
    past, trees, paths = _drafts(case)
    table, ps, Hkv, D = s["table"].cpu(), case["page"], case["Hkv"], case["D"]
    if case["op"] == "keep":
        most = _QMAX[s["k"].dtype]
        coded = (lambda x: torch.round(x.clamp(-127, 127))) if case["cache"] == "int8" else _e4m3
        out = {n + "_scale": s[n + "_scale"].to(f) for n in ("k", "v")}
        for n in ("k", "v"):
            was, scale = s[n].to(f), s[n + "_scale"].to(f)
            now, rows = was.clone(), []
            for b, path in enumerate(paths):
                upto = past[b] + len(path)
                for lo in range(past[b] // ps * ps, upto, ps):
                    p = int(table[b, lo // ps])
                    js = range(max(lo, past[b]) - past[b], min(lo + ps, upto) - past[b])
                    come = {j: (int(table[b, (past[b] + path[j]) // ps]), (past[b] + path[j]) % ps) for j in js}
                    sc = scale[p].clone()
                    for of, slot in come.values():
                        if of != p:
                            sc = torch.maximum(sc, was[of, :, slot].abs().amax(1) * scale[of] / most)
                    out[n + "_scale"][p] = sc
                    for at in range(lo, min(lo + ps, upto)):
                        of, slot = come.get(at - past[b], (p, at % ps))
                        ratio = (scale[of] / sc)[:, None]
                        now[p, :, at % ps] = torch.where(ratio == 1, was[of, :, slot], coded(was[of, :, slot] * ratio))
                if case["cache"] == "int8":
                    rows += [now[int(table[b, at // ps]), :, at % ps] * out[n + "_scale"][int(table[b, at // ps])][:, None]
                             for at in range(past[b], upto)]
            out[n] = torch.stack(rows) if case["cache"] == "int8" else now
        return out
    if sum(map(len, trees)) * case["Hq"] * max(past) > 2 ** 34:
        return None
    Hq = case["Hq"]
    out = torch.empty((sum(map(len, trees)), Hq, D), dtype=f, device="cuda")
    at = 0
    for b, tree in enumerate(trees):
        n, total = len(tree), past[b] + len(tree)
        pages = table[b, :-(-total // ps)].long().cuda()
        get = lambda name: (s[name].view(torch.int8)[pages].view(s[name].dtype).to(f) * s[name + "_scale"][pages].to(f)[:, :, None, None]  # noqa: E731
                            ).transpose(0, 1).reshape(Hkv, -1, D)[:, :total]
        k, v = get("k"), get("v")
        hidden = torch.zeros((n, total), dtype=torch.bool, device="cuda")
        sees = torch.from_numpy(tree).cuda()
        hidden[:, past[b]:] = ~sees
        if case["window"]:
            stands = past[b] + sees.sum(1, keepdim=True) - 1  # each sees itself
            j = torch.arange(past[b], device="cuda")[None]
            hidden[:, :past[b]] = (j + case["window"] <= stands) & (j >= case["sinks"])
        for h in range(Hq):
            z = (s["q"][at:at + n, h].to(f) @ k[h // (Hq // Hkv)].t()) / math.sqrt(D)
            out[at:at + n, h] = torch.softmax(z.masked_fill(hidden, -math.inf), -1) @ v[h // (Hq // Hkv)]
        at += n
    return out
