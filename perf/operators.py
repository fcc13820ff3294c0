"""Cases and plain forms of the paged 8-bit cache operators: append (with the position rotation), select, gather, attention.

The cache: k and v hold e4m3 codes in pages (npages, nkv, page, d); a page has one scale per KV head, a power of two 2^e with
-50 <= e <= 50; a row's value is code * scale. page_table (b, max_pages) names each sequence's pages, seq_len (b) its tokens.
"""
import torch

own = False

FLOAT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn
MIN_EXP, MAX_EXP = -50, 50


def device():
    return torch.device("cuda")


# ------------------------------------------------------------------ cases


def listed():
    return [
        # one new token for each of 64 running sequences: a serving step, all latency
        {"name": "append_decode", "op": "append", "b": 64, "nq": 32, "nkv": 8, "d": 128, "BCP": 1, "page": 64,
         "held": 500, "rot": 128, "pairs": "halves", "padded": False, "dtype": "bf16"},
        # the chunk of the Qwen3-4B-shaped layer behind a prompt that ends inside a page
        {"name": "append_chunk", "op": "append", "b": 1, "nq": 32, "nkv": 8, "d": 128, "BCP": 512, "page": 64,
         "held": 1000, "rot": 128, "pairs": "halves", "padded": False, "dtype": "bf16"},
        # a padded batch in fp32: small heads, small pages, neighbouring pairs, half of the head rotated
        {"name": "append_padded_f32", "op": "append", "b": 3, "nq": 12, "nkv": 4, "d": 64, "BCP": 257, "page": 16,
         "held": 77, "rot": 32, "pairs": "neighbours", "padded": True, "dtype": "f32"},
        # long prompts taken in at once
        {"name": "append_long", "op": "append", "b": 4, "nq": 32, "nkv": 8, "d": 128, "BCP": 2048, "page": 64,
         "held": 1000, "rot": 128, "pairs": "halves", "padded": False, "dtype": "bf16"},
        # the selection of a chunk over the Qwen3-4B-shaped cache
        {"name": "select_chunk", "op": "select", "b": 1, "nq": 32, "nkv": 8, "d": 128, "BCP": 512, "page": 64,
         "L": 32768, "NQ": 4, "BSA": 4096, "ragged": False, "dtype": "bf16"},
        # the selection of a decode step, sequences of all lengths
        {"name": "select_decode", "op": "select", "b": 16, "nq": 32, "nkv": 8, "d": 128, "BCP": 1, "page": 32,
         "L": 8191, "NQ": 1, "BSA": 1024, "ragged": True, "dtype": "bf16"},
        # the selected rows of the Qwen3-4B-shaped cache, for the chunk's attention
        {"name": "gather_selected", "op": "gather", "b": 1, "nkv": 8, "d": 128, "page": 64, "L": 32768, "BSA": 4096,
         "ragged": False, "dtype": "bf16"},
        # every row of a ragged batch, in fp32
        {"name": "gather_all_f32", "op": "gather", "b": 5, "nkv": 4, "d": 64, "page": 16, "L": 2999, "BSA": 0,
         "ragged": True, "dtype": "f32"},
        # a decode step of 32 sequences over their whole caches
        {"name": "attn_decode", "op": "attn", "b": 32, "nq": 32, "nkv": 8, "d": 128, "BCP": 1, "page": 64, "L": 8192,
         "BSA": 0, "chunk": False, "ragged": True, "dtype": "bf16"},
        # a decode step over the selected keys and its own
        {"name": "attn_decode_selected", "op": "attn", "b": 1, "nq": 32, "nkv": 8, "d": 128, "BCP": 1, "page": 64,
         "L": 32768, "BSA": 4096, "chunk": True, "ragged": False, "dtype": "bf16"},
        # a short block of speculative tokens in fp32, one sequence still without a cache
        {"name": "attn_block_f32", "op": "attn", "b": 4, "nq": 12, "nkv": 4, "d": 64, "BCP": 7, "page": 16, "L": 1500,
         "BSA": 0, "chunk": True, "ragged": True, "dtype": "f32"},
        # the chunk of the Qwen3-4B-shaped layer over its selected keys
        {"name": "attn_chunk", "op": "attn", "b": 1, "nq": 32, "nkv": 8, "d": 128, "BCP": 512, "page": 64, "L": 32768,
         "BSA": 4096, "chunk": True, "ragged": False, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, int(lo * (hi / lo) ** rng.random() * (1 + 1e-9)))


def draw(rng):
    op = rng.choice(("append", "select", "gather", "attn"))
    d, page = rng.choice((64, 128)), rng.choice((16, 32, 64, 128))
    nkv, G = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    c = {"op": op, "nkv": nkv, "d": d, "page": page, "dtype": dtype}
    if op == "append":
        BCP = _log(rng, 1, 2048)
        b = _log(rng, 1, max(1, min(64, 4096 // BCP)))
        return {**c, "b": b, "nq": nkv * G, "BCP": BCP, "held": _log(rng, 1, 2000) - 1,
                "rot": rng.choice((0, d // 2, d, d)), "pairs": rng.choice(("halves", "neighbours")),
                "padded": rng.random() < 0.5}
    L = _log(rng, 1, 32768)
    b = _log(rng, 1, max(1, min(32, 65536 // L)))
    BSA = min(L, _log(rng, 1, 4096))
    c.update(b=b, L=L, BSA=BSA, ragged=rng.random() < 0.5)
    if op == "gather":
        return {**c, "BSA": rng.choice((0, BSA)) if b * L <= 32768 else BSA}
    c["nq"] = nkv * G
    if op == "select":
        BCP = _log(rng, 1, max(1, 512 // b))
        return {**c, "BCP": BCP, "NQ": min(_log(rng, 1, 8), max(1, BCP // 10)), "L": L, "BSA": max(1, min(BSA, L // 4))}
    BCP = rng.choice((1, 1, _log(rng, 2, 16), _log(rng, 17, 512) if dtype == "bf16" and b * L <= 16384 else 1))
    return {**c, "BCP": BCP, "BSA": rng.choice((0, BSA)), "chunk": rng.random() < 0.5}


def _lengths(c):
    """Tokens held by each sequence: the first has the most; of a ragged batch of four or more the last has none."""
    top = c["held"] if c["op"] == "append" else c["L"]
    if c["op"] != "append" and not c["ragged"]:
        return [top] * c["b"]
    lens = [max(0, top - (3 * top * i) // (4 * c["b"]) - i % 5) for i in range(c["b"])]
    return lens[:-1] + [0] if len(lens) >= 4 else lens


def _new(c):
    """New tokens of each sequence (append)."""
    return [max(0, c["BCP"] - (c["BCP"] * i) // c["b"] - i % 2) if c["padded"] else c["BCP"] for i in range(c["b"])]


def work(c):
    es = 2 if c["dtype"] == "bf16" else 4
    d, nkv = c["d"], c["nkv"]
    lens = _lengths(c)
    if c["op"] == "append":
        toks = sum(_new(c))
        byts = toks * d * (2 * nkv * (es + 1) + nkv * es + 2 * c["nq"] * es) + toks * c["rot"] * 4
        return {"bytes": byts, "flops": toks * (3 * c["rot"] * (nkv + c["nq"]) + 2 * nkv * d)}
    rows = [min(n, c["BSA"]) if c["BSA"] else n for n in lens]
    if c["op"] == "gather":
        n = c["BSA"] or c["L"]
        return {"bytes": 2 * nkv * d * (sum(rows) + c["b"] * n * es), "flops": 2 * nkv * d * sum(rows)}
    qb = c["b"] * c["nq"] * c["BCP"] * d * es
    if c["op"] == "select":
        byts = qb + nkv * sum(lens) * (d + 4) + 4 * nkv * sum(rows)
        return {"bytes": byts, "flops": 2 * nkv * sum(lens) * d * (c["NQ"] + 1) + 4 * c["b"] * c["nq"] * c["BCP"] * d}
    own_keys = c["b"] * c["BCP"] if c["chunk"] else 0
    pairs = c["nq"] * c["BCP"] * (sum(rows) + (own_keys + 1) // 2)
    return {"bytes": 2 * qb + 2 * nkv * d * (sum(rows) + own_keys * es), "flops": 4 * d * pairs}


# ------------------------------------------------------------------ inputs


def _two_to(e):
    """2^e in fp32 for whole e, from its bits: exact, as a computed power need not be."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=device())


def _paged(g, c, lens, room, keys, values):
    """The paged cache of dense keys and values (b, nkv, n, d): pages in random order, entries past a sequence's pages -1."""
    b, nkv, page, d = c["b"], c["nkv"], c["page"], c["d"]
    P = -(-max(1, room) // page)
    held = torch.tensor([-(-n // page) for n in room_of(lens, c)], device=device())
    used = torch.arange(P, device=device())[None] < held[:, None]
    npages = int(used.sum()) + 3
    table = torch.full((b, P), -1, dtype=torch.int32, device=device())
    table[used] = torch.randperm(npages, generator=g, device=device())[: npages - 3].to(torch.int32)
    pools = []
    for x in (keys, values):
        x = torch.nn.functional.pad(x, (0, 0, 0, P * page - x.shape[2]))
        x = x.view(b, nkv, P, page, d).transpose(1, 2)[used]
        top = x.abs().amax((2, 3))
        m, e = torch.frexp(top)
        scale = _two_to((e - 9 + (m > 0.875)).clamp(MIN_EXP, MAX_EXP))
        pool = torch.zeros(npages, nkv, page, d, dtype=torch.uint8, device=device())
        pool[table[used].long()] = (x / scale[..., None, None]).clamp(-448, 448).to(E4M3).view(torch.uint8)
        scales = torch.ones(npages, nkv, device=device())
        scales[table[used].long()] = scale
        pools += [pool.view(E4M3), scales]
    return {"k": pools[0], "k_scale": pools[1], "v": pools[2], "v_scale": pools[3], "page_table": table,
            "seq_len": torch.tensor(lens, dtype=torch.int32, device=device())}


def room_of(lens, c):
    """Tokens that each sequence's pages have to hold."""
    return [n + m for n, m in zip(lens, _new(c))] if c["op"] == "append" else lens


def _angles(c, n):
    """cos and sin of the first n positions, from 64-bit angles."""
    i = torch.arange(c["rot"] // 2, device=device(), dtype=torch.float64)
    a = torch.arange(n, device=device(), dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / max(1, c["rot"]))
    return a.cos().float(), a.sin().float()


def prepare(c, seed):
    g = torch.Generator(device=device()).manual_seed(seed)
    t = FLOAT[c["dtype"]]
    b, nkv, d = c["b"], c["nkv"], c["d"]
    lens = _lengths(c)
    top = max(1, max(lens))
    keys, values = _randn(g, b, nkv, top, d), _randn(g, b, nkv, top, d)
    s = {"c": c}
    if c["op"] == "append":
        room = top + c["BCP"]
        # a later token may be larger than what its page holds: the page's scale then grows
        s["K"], s["V"] = 2 * _randn(g, b, nkv, c["BCP"], d).to(t), _randn(g, b, nkv, c["BCP"], d).to(t)
        s["Q"] = _randn(g, b, c["nq"], c["BCP"], d).to(t)
        s["cos"], s["sin"] = _angles(c, room) if c["rot"] else (None, None)
        s["new_len"] = torch.tensor(_new(c), dtype=torch.int32, device=device()) if c["padded"] else None
        s["Kr"], s["Qr"] = torch.zeros_like(s["K"]), torch.zeros_like(s["Q"])
        return {**s, **_paged(g, c, lens, room, keys, values)}
    if c["op"] == "select":
        # the keys that the selection is to find lie along a direction that the chunk's outlying queries share
        w = torch.nn.functional.normalize(_randn(g, b, nkv, 1, d), dim=-1)
        n = torch.tensor(lens, device=device())
        r = torch.rand(b, nkv, top, generator=g, device=device())
        r = r.masked_fill(torch.arange(top, device=device()) >= n[:, None, None], -1.0)
        at = r.argsort(-1, descending=True)[..., : c["BSA"]]
        keys = keys.scatter_add(2, at[..., None].expand(-1, -1, -1, d), (24 * w).expand(-1, -1, at.shape[-1], -1).contiguous())
        Q = _randn(g, b, nkv, c["nq"] // nkv, c["BCP"], d)
        out = torch.rand(b, nkv, 1, c["BCP"], generator=g, device=device()).argsort(-1) < max(c["NQ"], c["BCP"] // 10)
        mu = 12 * torch.nn.functional.normalize(_randn(g, b, nkv, 1, 1, d), dim=-1)
        s["Q"] = (Q + torch.where(out[..., None], 24 * w[:, :, None], mu)).reshape(b, c["nq"], c["BCP"], d).to(t)
        s["kv_idx"] = torch.full((b, nkv, min(c["BSA"], c["L"])), -1, dtype=torch.int32, device=device())
        s["s_agg"] = torch.zeros(b, nkv, c["L"], device=device())
        return {**s, **_paged(g, c, lens, c["L"], keys, values)}
    s.update(_paged(g, c, lens, c["L"], keys, values))
    s["kv_idx"] = s["kv_count"] = None
    if c["BSA"]:
        n = torch.tensor(lens, device=device())[:, None, None]
        r = torch.rand(b, nkv, top, generator=g, device=device())
        r = r.masked_fill(torch.arange(top, device=device()) >= n, -1.0)
        at = r.argsort(-1, descending=True)[..., : c["BSA"]].to(torch.int32)
        count = n.clamp(max=c["BSA"]).expand(b, nkv, 1)
        at = torch.where(torch.arange(at.shape[-1], device=device()) < count, at, 2**31 - 1).sort(-1).values
        s["kv_idx"] = torch.nn.functional.pad(at, (0, c["BSA"] - at.shape[-1]), value=2**31 - 1).contiguous()
        s["kv_count"] = count[..., 0].to(torch.int32).contiguous()
    if c["op"] == "attn":
        s["Q"] = (1.5 * _randn(g, b, c["nq"], c["BCP"], d)).to(t)
        s["Kc"] = _randn(g, b, nkv, c["BCP"], d).to(t) if c["chunk"] else None
        s["Vc"] = _randn(g, b, nkv, c["BCP"], d).to(t) if c["chunk"] else None
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    return (_own if own else _plain)(s)


def _own(s):
    import sparse_kv_selection_quoka_b200 as quoka
    c = s["c"]
    if "cache" not in s:  # the handle that a program keeps
        s["cache"] = quoka.QuokaCache(s["k"], s["v"], s["k_scale"], s["v_scale"], s["page_table"], s["seq_len"])
    cache = s["cache"]
    if c["op"] == "append":
        quoka.quoka_cache_append(cache, s["K"], s["V"], s["Q"], s["cos"], s["sin"], interleaved=c["pairs"] == "neighbours",
                                 new_len=s["new_len"], Kr=s["Kr"], Qr=s["Qr"])
        return _state(s)
    if c["op"] == "select":
        idx, count, _, scores = quoka.quoka_cache_select(s["Q"], cache, c["L"], c["NQ"], c["BSA"], kv_idx=s["kv_idx"],
                                                         s_agg=s["s_agg"])
        return {"kv_idx": idx, "kv_count": count, "s_agg": scores}
    if c["op"] == "gather":
        K, V = quoka.quoka_cache_gather(cache, c["L"], s["kv_idx"], s["kv_count"], dtype=FLOAT[c["dtype"]])
        return {"K": K, "V": V}
    O, lse = quoka.quoka_cache_attn(s["Q"], cache, c["L"], s["kv_idx"], s["kv_count"], s["Kc"], s["Vc"], want_lse=True)
    return {"O": O, "lse": lse}


def _state(s):
    return {k: s[k] for k in ("k", "k_scale", "v", "v_scale", "Kr", "Qr")}


def _plain(s):
    return {"append": _plain_append, "select": _plain_select, "gather": _plain_gather, "attn": _plain_attn}[s["c"]["op"]](s)


def _rotated(x, cos, sin, pairs):
    """x (b, h, t, d) in fp32 with its first 2 * cos.shape[-1] columns rotated; cos, sin (b, 1, t, rot / 2)."""
    r = cos.shape[-1]
    if pairs == "halves":
        a, z = x[..., :r], x[..., r:2 * r]
        turned = torch.cat((a * cos - z * sin, z * cos + a * sin), -1)
    else:
        a, z = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        turned = torch.stack((a * cos - z * sin, z * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., 2 * r:]), -1)


def _plain_append(s):
    c = s["c"]
    page, BCP = c["page"], c["BCP"]
    start = s["seq_len"].long()
    fresh = s["new_len"].long() if s["new_len"] is not None else torch.full_like(start, BCP)
    tok = torch.arange(BCP, device=start.device)
    live = (tok < fresh[:, None])[:, None, :, None]
    K, Q = s["K"].float(), s["Q"].float()
    if c["rot"]:
        at = (start[:, None] + tok).clamp(max=s["cos"].shape[0] - 1)
        cos, sin = s["cos"][at][:, None], s["sin"][at][:, None]
        K, Q = _rotated(K, cos, sin, c["pairs"]), _rotated(Q, cos, sin, c["pairs"])
    s["Kr"].copy_(torch.where(live, K.to(s["Kr"].dtype), s["Kr"]))
    s["Qr"].copy_(torch.where(live, Q.to(s["Qr"].dtype), s["Qr"]))
    # the new tokens by the pages they fall in: (b, pages touched, page)
    first = start // page
    P = (BCP + 2 * page - 2) // page
    slot = torch.arange(P * page, device=start.device).view(P, page)
    i = slot - (start % page)[:, None, None]
    new = (i >= 0) & (i < fresh[:, None, None])
    before = (slot < (start % page)[:, None, None])
    touched = new.any(-1)
    col = (first[:, None] + torch.arange(P, device=start.device)).clamp(max=s["page_table"].shape[1] - 1)
    ids = s["page_table"].gather(1, col).long().clamp(min=0)
    row = i.clamp(0, BCP - 1).flatten(1)[:, None, :, None].expand(-1, c["nkv"], -1, c["d"])
    _fill(s["k"], s["k_scale"], K, row, new, before, touched, ids)
    _fill(s["v"], s["v_scale"], s["V"].float(), row, new, before, touched, ids)
    return _state(s)


def _fill(pool, scales, x, row, new, before, touched, ids):
    """Quantises the new rows of x into the pages `ids`, bringing what they hold to the page's scale."""
    b, P, page = new.shape
    x = x.gather(2, row).view(b, x.shape[1], P, page, -1).transpose(1, 2)
    new, before = new[:, :, None, :, None], before[:, :, None, :, None]
    size = torch.where(new & x.isfinite(), x.abs(), 0).amax((3, 4))
    m, k = torch.frexp(size)  # size = m 2^k, 1/2 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(size > 0, k - 9 + (m > 0.875), MIN_EXP).clamp(MIN_EXP, MAX_EXP)
    scale = _two_to(e)
    old_codes, old_scale = pool.view(torch.uint8)[ids], scales[ids]
    scale = torch.where(before.any(-2).squeeze(-1), torch.maximum(scale, old_scale), scale)
    wide = scale[..., None, None]
    codes = (x / wide).clamp(-448, 448).to(E4M3).view(torch.uint8)
    moved = (old_codes.view(E4M3).float() * (old_scale / scale)[..., None, None]).to(E4M3).view(torch.uint8)
    codes = torch.where(new, codes, torch.where(before, moved, old_codes))
    pool.view(torch.uint8)[ids[touched]] = codes[touched]
    scales[ids[touched]] = scale[touched]


def _pages(s, name, wide):
    """All rows of each sequence's table as values (b, nkv, tokens, d): the keys ("k") or the values ("v")."""
    ids = s["page_table"].long().clamp(min=0)
    x = s[name].view(torch.uint8)[ids].view(E4M3).to(wide) * s[name + "_scale"][ids][..., None, None].to(wide)
    return x.transpose(1, 2).flatten(2, 3)[:, :, : s["c"]["L"]]


def _rows(s):
    """The selected (or all) rows and which of them there are: K, V (b, nkv, n, d), there (b, nkv or 1, n)."""
    K, V = _pages(s, "k", torch.float32), _pages(s, "v", torch.float32)
    n = torch.arange(K.shape[2], device=K.device)
    if s["kv_idx"] is None:
        return K, V, (n < s["seq_len"][:, None, None])
    at = s["kv_idx"].long()
    there = torch.arange(at.shape[2], device=K.device) < s["kv_count"][..., None]
    at = torch.where(there, at, 0)[..., None].expand(-1, -1, -1, K.shape[3])
    return K.gather(2, at), V.gather(2, at), there


def _plain_gather(s):
    K, V, there = _rows(s)
    t = FLOAT[s["c"]["dtype"]]
    return {"K": torch.where(there[..., None], K, 0).to(t), "V": torch.where(there[..., None], V, 0).to(t)}


def _plain_select(s):
    # in 64 bits: the scores are compared with one another
    c = s["c"]
    b, nkv, G, d = c["b"], c["nkv"], c["nq"] // c["nkv"], c["d"]
    Q = s["Q"].double()
    mean = Q.mean(2, keepdim=True)
    norm = Q.square().sum(-1).sqrt()
    cos = (Q * mean).sum(-1) / (norm * mean.square().sum(-1).sqrt()).clamp(min=1e-8)
    rank = cos.sort(dim=-1, stable=True).indices[..., : c["NQ"]]
    picked = (Q / norm.clamp(min=1e-12)[..., None]).gather(2, rank[..., None].expand(-1, -1, -1, d))
    group = picked.view(b, nkv, G, c["NQ"], d).mean(2)
    K = _pages(s, "k", torch.float64)
    S = (group @ K.transpose(2, 3)).amax(2) / K.square().sum(-1).sqrt().clamp(min=1e-300)
    here = torch.arange(c["L"], device=K.device) < s["seq_len"][:, None, None]
    n = s["kv_idx"].shape[2]
    count = s["seq_len"][:, None].clamp(max=n).expand(b, nkv)
    order = S.masked_fill(~here, -torch.inf).sort(dim=-1, descending=True, stable=True).indices[..., :n]
    got = torch.arange(n, device=K.device) < count[..., None]
    order = torch.where(got, order, c["L"]).sort(-1).values.to(torch.int32)
    s["kv_idx"].copy_(torch.where(got, order, s["kv_idx"]))
    s["s_agg"].copy_(torch.where(here, S.float(), s["s_agg"]))
    return {"kv_idx": s["kv_idx"], "kv_count": count.contiguous(), "s_agg": s["s_agg"]}


def _plain_attn(s):
    c = s["c"]
    b, nkv, BCP, d = c["b"], c["nkv"], c["BCP"], c["d"]
    K, V, there = _rows(s)
    V = torch.where(there[..., None], V, 0)
    Q = s["Q"].float().view(b, nkv, -1, d)
    S = (Q @ K.transpose(2, 3)).mul_(d ** -0.5)
    S.masked_fill_(~there[:, :, None], -torch.inf)
    if c["chunk"]:
        t = torch.arange(BCP, device=Q.device)
        Sc = (Q @ s["Kc"].float().transpose(2, 3)) * d ** -0.5
        Sc = Sc.view(b, nkv, -1, BCP, BCP).masked_fill(t > t[:, None], -torch.inf).view(b, nkv, -1, BCP)
        S, V = torch.cat((S, Sc), -1), torch.cat((V, s["Vc"].float()), 2)
    top = S.amax(-1, keepdim=True)
    P = S.sub_(top.masked_fill(top == -torch.inf, 0)).exp_()
    total = P.sum(-1, keepdim=True)
    O = torch.where(total > 0, (P @ V) / total, 0)
    lse = (top + total.log()).squeeze(-1)
    return {"O": O.view(b, c["nq"], BCP, d).to(s["Q"].dtype), "lse": lse.reshape(b, c["nq"], BCP)}


# ------------------------------------------------------------------ 64 bits, from the definitions


def _power(e):
    """2^e in 64 bits for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exponent(x):
    """floor(log2 x) of positive 64-bit numbers."""
    return (x.contiguous().view(torch.int64) >> 52) - 1023


def _values(codes):
    """What e4m3 codes stand for: sign, 4 bits of exponent (bias 7), 3 of fraction; exponent 0 is subnormal."""
    u = codes.contiguous().view(torch.uint8).to(torch.int64)
    e, f = (u >> 3) & 15, (u & 7).double()
    v = torch.where(e > 0, (1 + f / 8) * _power(e - 7), f / 8 * 2.0**-6)
    return torch.where((u & 127) == 127, torch.nan, v) * (1 - 2 * (u >> 7))


def _nearest(y):
    """The nearest e4m3 value, ties to an even fraction, nothing beyond 448."""
    y = y.clamp(-448, 448)
    step = _power(_exponent(y.abs().clamp(min=2.0**-6)) - 3)
    return torch.round(y / step) * step


def exact(c, seed):
    s = prepare(c, seed)
    lens, nkv, d, page = _lengths(c), c["nkv"], c["d"], c["page"]
    if c["op"] == "append":
        return _exact_append(c, s, lens)
    out = {"s_agg": None, "kv_idx": None, "kv_count": None} if c["op"] == "select" else {}
    rows = []
    for i, n in enumerate(lens):
        ids = s["page_table"][i, : -(-n // page)].long()
        K = (_values(s["k"].view(torch.uint8)[ids]) * s["k_scale"][ids].double()[..., None, None]).transpose(0, 1).reshape(nkv, -1, d)[:, :n]
        V = (_values(s["v"].view(torch.uint8)[ids]) * s["v_scale"][ids].double()[..., None, None]).transpose(0, 1).reshape(nkv, -1, d)[:, :n]
        if c["op"] != "select" and c["BSA"]:
            m = min(n, c["BSA"])
            at = s["kv_idx"][i, :, :m].long()[..., None].expand(-1, -1, d)
            K, V = K.gather(1, at), V.gather(1, at)
        rows.append(_exact_one(c, s, i, K, V))
    got = {k: torch.stack([r[k] for r in rows]) for k in rows[0]}
    return {**out, **got}


def _exact_one(c, s, i, K, V):
    """Sequence i of a select, gather or attention, given the rows it works on (nkv, n, d)."""
    nkv, G, d = c["nkv"], (c["nq"] // c["nkv"] if "nq" in c else 1), c["d"]
    if c["op"] == "gather":
        pad = (0, 0, 0, (c["BSA"] or c["L"]) - K.shape[1])
        return {"K": torch.nn.functional.pad(K, pad), "V": torch.nn.functional.pad(V, pad)}
    Q = s["Q"][i].double().view(nkv, G, c["BCP"], d)
    if c["op"] == "select":
        unit = Q / Q.norm(dim=-1, keepdim=True)
        mean = Q.mean(2, keepdim=True)
        sq = -(unit * (mean / mean.norm(dim=-1, keepdim=True))).sum(-1)
        best = sq.topk(c["NQ"], -1).indices
        group = torch.stack([unit[:, g].gather(1, best[:, g, :, None].expand(-1, -1, d)) for g in range(G)]).sum(0) / G
        S = (torch.nn.functional.normalize(K, dim=-1, eps=1e-300) @ group.transpose(1, 2)).amax(-1)
        return {"s_agg": torch.nn.functional.pad(S, (0, c["L"] - S.shape[1]))}
    S = torch.einsum("jgtd,jnd->jgtn", Q, K) / d**0.5
    if c["chunk"]:
        Sc = torch.einsum("jgtd,jnd->jgtn", Q, s["Kc"][i].double()) / d**0.5
        Sc = Sc + torch.full((c["BCP"], c["BCP"]), -torch.inf, device=Q.device, dtype=torch.float64).triu(1)
        S, V = torch.cat((S, Sc), -1), torch.cat((V, s["Vc"][i].double()), 1)
    lse = torch.logsumexp(S, -1) if S.shape[-1] else torch.full(S.shape[:-1], -torch.inf, device=Q.device, dtype=torch.float64)
    W = torch.exp(S - lse.masked_fill(lse == -torch.inf, 0)[..., None])
    O = torch.einsum("jgtn,jnd->jgtd", W, V)
    return {"O": O.reshape(c["nq"], c["BCP"], d), "lse": lse.reshape(c["nq"], c["BCP"])}


def _exact_append(c, s, lens):
    page, rot = c["page"], c["rot"]
    out = {"Kr": s["Kr"].double(), "Qr": s["Qr"].double(), "k_scale": s["k_scale"].double(), "v_scale": s["v_scale"].double(),
           "k": _values(s["k"]), "v": _values(s["v"])}
    for i, (n, m) in enumerate(zip(lens, _new(c))):
        if m == 0:
            continue
        turned = {}
        for name in ("K", "Q"):
            x = s[name][i, :, :m].double().clone()
            if rot:
                cos, sin = s["cos"][n : n + m].double(), s["sin"][n : n + m].double()
                lo = slice(0, rot // 2) if c["pairs"] == "halves" else slice(0, rot, 2)
                hi = slice(rot // 2, rot) if c["pairs"] == "halves" else slice(1, rot, 2)
                a, z = x[..., lo].clone(), x[..., hi].clone()
                x[..., lo], x[..., hi] = a * cos - z * sin, a * sin + z * cos
            turned[name] = x
            out[name + "r"][i, :, :m] = x
        for name, x in (("k", turned["K"]), ("v", s["V"][i, :, :m].double())):
            for p in range(n // page, (n + m - 1) // page + 1):
                t0, t1 = max(n, p * page), min(n + m, (p + 1) * page)
                at, rows = int(s["page_table"][i, p]), x[:, t0 - n : t1 - n]
                top = rows.abs().amax((1, 2))
                e = _exponent(top) - 8
                e = (e + (top > 448 * _power(e)).long()).clamp(MIN_EXP, MAX_EXP)
                held = t0 - p * page
                if held:
                    old = _exponent(out[name + "_scale"][at])
                    e = torch.maximum(e, old)
                    out[name][at, :, :held] = _nearest(out[name][at, :, :held] * _power(old - e)[:, None, None])
                out[name + "_scale"][at] = _power(e)
                out[name][at, :, held : held + t1 - t0] = _nearest(rows * _power(-e)[:, None, None])
    return out
