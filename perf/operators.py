"""The operators of the 8-bit paged key/value cache: what is measured, and their plain forms.

A cache holds P pages of ``page`` tokens. Per page, head and block of 32 tokens there are int8 codes of
the keys, ``[D/64][32 tokens][64]``, int8 codes of the values, ``[D][32 positions]`` (token 8j + 2t + e of
the block, with j, t < 4 and e < 2, lies at position 8t + 2j + e), and one fp32 scale each. A page table
names each sequence's pages in order.

Operators:

- append:    new BF16 keys and values go into the pages; a block's scale is the larger of the scale that it
             has for older tokens and amax / 127 of the new ones, and older codes are rounded again when it grows
- read:      a span of tokens back as BF16
- attention: softmax(sm_scale * q k^T) v of T queries for each sequence over its cache, query heads in groups
             that share a key/value head, causal (the queries are the last tokens) or to all keys, with log-sum-exp
- copy:      pages copied to other pages
"""

import math

import torch

own = False

BLOCK = 32


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------- cases --


def listed():
    return [
        # One sequence answering token by token after a short prompt: the smallest call, latency counts.
        dict(name="decode_one", op="attention", B=1, T=1, H=28, Hkv=4, D=128, page=64, L=1000, lo=1.0, causal=True,
             lse=False, ragged_q=False),
        # A serving batch: 64 sequences of different lengths, one token each.
        dict(name="decode_batch", op="attention", B=64, T=1, H=32, Hkv=8, D=128, page=64, L=8192, lo=0.1, causal=True,
             lse=False, ragged_q=False),
        # Two long documents, one token each: few rows, a long axis.
        dict(name="decode_long", op="attention", B=2, T=1, H=28, Hkv=4, D=128, page=128, L=131071, lo=0.7,
             causal=True, lse=True, ragged_q=False),
        # Drafted tokens checked together, another number for each sequence; head dimension 64, small pages.
        dict(name="verify_drafts", op="attention", B=16, T=5, H=16, Hkv=4, D=64, page=32, L=4001, lo=0.3, causal=True,
             lse=True, ragged_q=True),
        # Latents of an odd number of tokens attending to an encoder's states of other lengths, no mask.
        dict(name="cross_encoder", op="attention", B=2, T=4097, H=16, Hkv=16, D=64, page=64, L=1500, lo=0.4,
             causal=False, lse=True, ragged_q=False),
        # A chunk of a long prompt, causal, against all that came before it: the largest product.
        dict(name="prompt_chunk", op="attention", B=1, T=2000, H=32, Hkv=8, D=128, page=128, L=16001, lo=1.0,
             causal=True, lse=False, ragged_q=False),
        # The token that each sequence of a serving batch has just produced goes into its cache.
        dict(name="append_tokens", op="append", B=64, T=1, Hkv=8, D=128, page=64, L=2000),
        # Prompts of different lengths go into the cache, the first block already begun.
        dict(name="append_prompts", op="append", B=16, T=4096, Hkv=8, D=128, page=64, L=700),
        # A few tokens of each of four sequences read back.
        dict(name="read_tail", op="read", B=4, T=33, Hkv=4, D=64, page=32, L=500),
        # Whole prompts handed over in full precision.
        dict(name="read_prompts", op="read", B=8, T=8000, Hkv=8, D=128, page=64, L=8100),
        # Sequences forked for several answers: the last, partly filled page of each is copied.
        dict(name="copy_fork", op="copy", n=16, P=400, Hkv=4, D=128, page=64),
        # Compaction: live pages move into the holes in front of them.
        dict(name="copy_compact", op="copy", n=2000, P=4500, Hkv=8, D=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention"] * 6 + ["append", "append", "read", "copy"])
    D = rng.choice([128, 128, 64])
    page = rng.choice([32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 7, 8])
    if op == "copy":
        return dict(op=op, n=_log_int(rng, 1, 1800), P=4000, Hkv=Hkv, D=D, page=rng.choice([32, 64]))
    if op == "append":
        T = rng.choice([1, _log_int(rng, 2, 4000)])
        return dict(op=op, B=_log_int(rng, 1, 64 if T == 1 else 12), T=T, Hkv=Hkv, D=D, page=page,
                    L=_log_int(rng, 1, 3000))
    if op == "read":
        T = _log_int(rng, 1, 8000)
        return dict(op=op, B=_log_int(rng, 1, 8), T=T, Hkv=Hkv, D=D, page=page, L=T + rng.randrange(0, 100))
    kind = rng.choice(["decode", "decode", "verify", "chunk", "cross"])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    lo = rng.uniform(0.05, 1.0)
    if kind == "decode":
        B = _log_int(rng, 1, 64)
        L, T = _log_int(rng, 1, min(131072, 280000 // B)), 1
    elif kind == "verify":
        B, T = _log_int(rng, 1, 24), rng.randrange(2, 9)
        L = _log_int(rng, T, min(20000, 280000 // B))
    elif kind == "chunk":
        B, T = _log_int(rng, 1, 2), _log_int(rng, 9, 700)
        L = T + _log_int(rng, 1, 10000)
    else:
        B, T, L, G = _log_int(rng, 1, 4), _log_int(rng, 9, 4200), _log_int(rng, 1, 1600), 1
    return dict(op=op, B=B, T=T, H=Hkv * G, Hkv=Hkv, D=D, page=page, L=L, lo=round(lo, 3),
                causal=kind != "cross", lse=rng.random() < 0.5, ragged_q=kind == "verify" and rng.random() < 0.5)


def _lengths(c):
    """The sequences' lengths: from lo * L to L, evenly."""
    B, L = c["B"], c["L"]
    return [max(1, int(round(L * (c["lo"] + (1 - c["lo"]) * (b + 1) / B)))) for b in range(B)]


def _query_lengths(c):
    return [1 + b % c["T"] if c["ragged_q"] else c["T"] for b in range(c["B"])]


def _append_sizes(c):
    """(starts, counts) of the sequences of an append case."""
    starts = [(c["L"] * (b + 1)) // c["B"] for b in range(c["B"])]
    counts = [c["T"] if c["T"] == 1 else max(1, c["T"] - (c["T"] * b) // (2 * c["B"])) for b in range(c["B"])]
    return starts, counts


# ------------------------------------------------------------------ inputs --


def _codes(shape, g, dev):
    out = torch.empty(shape, dtype=torch.int8, device=dev)
    flat = out.view(-1)
    for a in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - a)
        flat[a:a + n] = (torch.randn(n, generator=g, device=dev) * 36.0).round_().clamp_(-127, 127).to(torch.int8)
    return out


def _cache(P, c, g, dev):
    Hkv, D, n = c["Hkv"], c["D"], c["page"] // BLOCK

    def scale():
        return torch.exp(torch.randn((P, Hkv, n), generator=g, device=dev) * 0.25) * (1.0 / 36.0)

    return dict(k_codes=_codes((P, Hkv, n, D // 64, BLOCK, 64), g, dev), v_codes=_codes((P, Hkv, n, D, BLOCK), g, dev),
                k_scale=scale(), v_scale=scale())


def _table(lengths, page, spare, g, dev):
    """A page table whose pages lie in no order, for sequences of up to these lengths, and the number of pages."""
    need = [-(-n // page) for n in lengths]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    table = torch.zeros((len(need), max(need)), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, P


def prepare(case, seed):
    c = dict(case)
    dev = _device()
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = dict(case=c)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def values(*shape):
        return torch.randn(shape, generator=g, device=dev).to(torch.bfloat16)

    if c["op"] == "copy":
        s["cache"] = _cache(c["P"], c, g, dev)
        pages = torch.randperm(c["P"], generator=g, device=dev).to(torch.int32)
        s["src"], s["dst"] = pages[:c["n"]].clone(), pages[c["n"]:2 * c["n"]].clone()
        return s
    if c["op"] == "attention":
        order = torch.randperm(c["B"], generator=g, device=dev).tolist()
        lengths = [_lengths(c)[b] for b in order]
        s["table"], P = _table(lengths, c["page"], 3, g, dev)
        s["lengths"] = ints(lengths)
        s["q_lengths"] = ints(_query_lengths(c)) if c["ragged_q"] else None
        s["q"] = values(c["B"], c["T"], c["H"], c["D"])
    elif c["op"] == "append":
        starts, counts = _append_sizes(c)
        s["table"], P = _table([a + n for a, n in zip(starts, counts)], c["page"], 3, g, dev)
        s["starts"], s["counts"] = ints(starts), None if c["T"] == 1 else ints(counts)
        # read back from the first touched block's beginning: its older tokens' codes may change too
        first = [a // BLOCK * BLOCK for a in starts]
        s["read_starts"], s["read_counts"] = ints(first), ints([a + n - f for a, n, f in zip(starts, counts, first)])
        s["read_T"] = max(a + n - f for a, n, f in zip(starts, counts, first))
        s["k"], s["v"] = values(c["B"], c["T"], c["Hkv"], c["D"]), values(c["B"], c["T"], c["Hkv"], c["D"])
    else:
        s["table"], P = _table([c["L"]] * c["B"], c["page"], 3, g, dev)
        s["starts"] = ints([(c["L"] - c["T"]) * (b + 1) // c["B"] for b in range(c["B"])])
    s["cache"] = _cache(P, c, g, dev)
    return s


# -------------------------------------------------------------- plain forms --


def _keys(cache, pages):
    """Keys of the tokens of ``pages`` [B, N], fp32 [B, Hkv, N * page, D]."""
    c = cache["k_codes"][pages]                                     # [B, N, Hkv, n, D/64, 32, 64]
    x = c.permute(0, 2, 1, 3, 5, 4, 6).float() * cache["k_scale"][pages].permute(0, 2, 1, 3)[..., None, None, None]
    return x.flatten(5, 6).flatten(2, 4)


def _values(cache, pages):
    """Values of the tokens of ``pages`` [B, N], fp32 [B, Hkv, N * page, D]."""
    c = cache["v_codes"][pages]                                     # [B, N, Hkv, n, D, 32]
    x = c.unflatten(5, (4, 4, 2)).permute(0, 2, 1, 3, 6, 5, 7, 4).flatten(4, 6)
    x = x.float() * cache["v_scale"][pages].permute(0, 2, 1, 3)[..., None, None]
    return x.flatten(2, 4)


def _plain_attention(s):
    c, q = s["case"], s["q"]
    B, T, H, D = q.shape
    G = H // c["Hkv"]
    pages = s["table"].long()
    k, v = _keys(s["cache"], pages), _values(s["cache"], pages)
    x = q.float().unflatten(2, (c["Hkv"], G)).permute(0, 2, 3, 1, 4).reshape(B, c["Hkv"], G * T, D)
    z = (x @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    z = z.unflatten(2, (G, T))                                      # [B, Hkv, G, T, L]
    L = z.shape[-1]
    lengths = s["lengths"].long()
    q_len = torch.full_like(lengths, T) if s["q_lengths"] is None else s["q_lengths"].long()
    t, j = torch.arange(T, device=q.device), torch.arange(L, device=q.device)
    last = lengths[:, None] - 1 + (t - q_len[:, None] + 1 if c["causal"] else 0 * t)   # [B, T]: the last key that a row sees
    row = t < q_len[:, None]
    seen = (j <= last[..., None]) & row[..., None]                  # [B, T, L]
    z = z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    p = z.sub_(m.clamp_min(-1e30)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (G, T)) / total.clamp_min(1e-37)
    out = o.permute(0, 3, 1, 2, 4).reshape(B, T, H, D).to(torch.bfloat16)
    if not c["lse"]:
        return out
    return out, (m + total.log()).squeeze(-1).flatten(1, 2)


def _plain_span(table, cache, starts, T, page):
    """(page, block, slot) of tokens starts .. starts + T - 1, each [B, T]."""
    pos = (starts.long()[:, None] + torch.arange(T, device=table.device)).clamp_max(table.shape[1] * page - 1)
    return table.long().gather(1, pos // page), pos % page // BLOCK, pos % BLOCK


def _plain_read(cache, table, starts, counts, T, page):
    pg, blk, slot = _plain_span(table, cache, starts, T, page)
    at = slot % 8 // 2 * 8 + slot // 8 * 2 + slot % 2
    k = cache["k_codes"][pg, :, blk, :, slot].flatten(3, 4)         # [B, T, Hkv, D]
    v = cache["v_codes"][pg, :, blk, :, at]
    k = k.float() * cache["k_scale"][pg, :, blk][..., None]
    v = v.float() * cache["v_scale"][pg, :, blk][..., None]
    if counts is not None:
        there = (torch.arange(T, device=table.device) < counts[:, None])[..., None, None]
        k, v = k * there, v * there
    return k.to(torch.bfloat16), v.to(torch.bfloat16)


def _plain_append(s):
    c, cache, table, x = s["case"], s["cache"], s["table"], None
    B, T, Hkv, D = s["k"].shape
    dev = table.device
    starts = s["starts"].long()
    counts = torch.full_like(starts, T) if s["counts"] is None else s["counts"].long()
    N = (T + BLOCK - 2) // BLOCK + 1                                # blocks that T tokens can touch
    blk = starts[:, None] // BLOCK + torch.arange(N, device=dev)    # [B, N] blocks of the sequences
    t = blk[..., None] * BLOCK + torch.arange(BLOCK, device=dev) - starts[:, None, None]   # [B, N, 32] new token in each slot
    new = (t >= 0) & (t < counts[:, None, None])
    b_at, n_at = torch.nonzero(new.any(-1), as_tuple=True)          # the blocks with a new token
    t, new, blk = t[b_at, n_at], new[b_at, n_at], blk[b_at, n_at]
    older = t < 0                                                   # [M, 32]
    n = c["page"] // BLOCK
    pg, sub = table.long()[b_at, blk // n], blk % n
    limit = torch.full((), 127.0, device=dev)
    slot = torch.arange(BLOCK, device=dev)
    at = slot % 8 // 2 * 8 + slot // 8 * 2 + slot % 2
    for name in ("k", "v"):
        x = s[name][b_at[:, None], t.clamp(0, T - 1)].float() * new[..., None, None]       # [M, 32, Hkv, D]
        amax = x.abs().amax((1, 3))                                 # [M, Hkv]
        before = cache[name + "_scale"][pg, :, sub] * older.any(-1, keepdim=True)
        scale = torch.maximum(amax / limit, before)
        codes = (x / scale.clamp_min(1e-45)[:, None, :, None]).round().clamp(-127, 127)
        if name == "k":
            was = cache["k_codes"][pg, :, sub].permute(0, 3, 1, 2, 4).flatten(3, 4).float()   # [M, 32, Hkv, D]
        else:
            was = cache["v_codes"][pg, :, sub][..., at].permute(0, 3, 1, 2).float()
        was = (was * (before / scale.clamp_min(1e-45))[:, None, :, None]).round()
        codes = torch.where(new[..., None, None], codes, was).to(torch.int8)
        if name == "k":
            cache["k_codes"][pg, :, sub] = codes.unflatten(3, (D // 64, 64)).permute(0, 2, 3, 1, 4)
        else:
            cache["v_codes"][pg, :, sub] = torch.empty((len(pg), Hkv, D, BLOCK), dtype=torch.int8, device=dev).index_copy_(
                3, at, codes.permute(0, 2, 3, 1))
        cache[name + "_scale"][pg, :, sub] = scale


def _plain_copy(s):
    for x in s["cache"].values():
        x[s["dst"].long()] = x[s["src"].long()]


# ---------------------------------------------------------------------- run --


def _handle(s):
    """The cache as the framework's object: what a program makes once and keeps."""
    if "handle" not in s:
        import quantized_attention_fp64_gb300 as sage

        s["sage"], s["handle"] = sage, sage.QuantizedCache(**s["cache"])
    return s["sage"], s["handle"]


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        sage, cache = _handle(s)
        if op == "attention":
            return sage.cache_attention(s["q"], cache, s["table"], s["lengths"], q_lengths=s["q_lengths"],
                                        is_causal=c["causal"], return_lse=c["lse"])
        if op == "append":
            sage.cache_append(cache, s["k"], s["v"], s["table"], s["starts"], counts=s["counts"])
            k, v = sage.cache_read(cache, s["table"], s["read_starts"], s["read_T"], counts=s["read_counts"])
            return k, v, s["cache"]["k_scale"], s["cache"]["v_scale"]
        if op == "read":
            return sage.cache_read(cache, s["table"], s["starts"], c["T"])
        sage.cache_copy_pages(cache, s["src"], s["dst"])
        return s["cache"]
    if op == "attention":
        return _plain_attention(s)
    if op == "append":
        _plain_append(s)
        k, v = _plain_read(s["cache"], s["table"], s["read_starts"], s["read_counts"], s["read_T"], c["page"])
        return k, v, s["cache"]["k_scale"], s["cache"]["v_scale"]
    if op == "read":
        return _plain_read(s["cache"], s["table"], s["starts"], None, c["T"], c["page"])
    _plain_copy(s)
    return s["cache"]  # bytes that were moved: the codes themselves are the outcome


# --------------------------------------------------------------------- work --


def work(case):
    c = case
    Hkv, D = c["Hkv"], c["D"]
    token = 2 * Hkv * (D + 4 / BLOCK)                               # bytes of one cached token, keys and values
    if c["op"] == "copy":
        return dict(bytes=2 * c["n"] * c["page"] * token, flops=0)
    if c["op"] == "append":
        starts, counts = _append_sizes(c)
        back = sum(a % BLOCK + n for a, n in zip(starts, counts))   # tokens read back
        return dict(bytes=sum(counts) * (4 * Hkv * D + token) + back * (token + 4 * Hkv * D), flops=0)
    if c["op"] == "read":
        return dict(bytes=c["B"] * c["T"] * (token + 4 * Hkv * D), flops=0)
    bytes_, flops = 0.0, 0.0
    for n, r in zip(_lengths(c), _query_lengths(c)):
        bytes_ += n * token + r * c["H"] * D * 4 + (r * c["H"] * 4 if c["lse"] else 0)
        seen = sum(max(0, n - r + i + 1) for i in range(r)) if c["causal"] else n * r
        flops += 4.0 * seen * c["H"] * D
    return dict(bytes=bytes_, flops=flops)


# -------------------------------------------------------- the definition, 64 --


def _token(cache, table, b, page, pos):
    """Keys and values of the tokens ``pos`` (a list or range) of sequence b, float64 [n, Hkv, D]."""
    pos = torch.as_tensor(list(pos), dtype=torch.int64, device=table.device)
    pg, blk, i = table[b].long()[pos // page], (pos % page) // BLOCK, pos % BLOCK
    j, r = i // 8, i % 8
    k = cache["k_codes"][pg, :, blk, :, i].double()
    v = cache["v_codes"][pg, :, blk, :, (r // 2) * 8 + j * 2 + r % 2].double()
    k = k.flatten(2) * cache["k_scale"][pg, :, blk].double()[:, :, None]
    return k, v * cache["v_scale"][pg, :, blk].double()[:, :, None]


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    cache, page = s["cache"], c["page"]
    if c["op"] == "copy":
        out = {k: v.clone() for k, v in cache.items()}
        for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
            for k in out:
                out[k][b] = cache[k][a]
        return {k: (v.double() if v.dtype == torch.float32 else None) for k, v in out.items()}
    table = s["table"]
    if c["op"] == "read":
        rows = [_token(cache, table, b, page, range(a, a + c["T"])) for b, a in enumerate(s["starts"].tolist())]
        return torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
    if c["op"] == "append":
        return _exact_append(s)
    B, T, H, D = s["q"].shape
    G = H // c["Hkv"]
    out = torch.zeros((B, T, H, D), dtype=torch.float64, device=table.device)
    lse = torch.full((B, H, T), -math.inf, dtype=torch.float64, device=table.device)
    for b, n in enumerate(s["lengths"].tolist()):
        r = T if s["q_lengths"] is None else int(s["q_lengths"][b])
        k, v = _token(cache, table, b, page, range(n))
        sees = torch.full((r,), n, device=table.device)
        if c["causal"]:
            sees = n - r + 1 + torch.arange(r, device=table.device)
        hidden = torch.arange(n, device=table.device)[None, :] >= sees[:, None]
        for h in range(H):
            z = s["q"][b, :r, h].double() @ k[:, h // G].T / math.sqrt(D)
            z[hidden] = -math.inf
            l = torch.logsumexp(z, 1)
            lse[b, h, :r] = l
            p = torch.exp(z - l[:, None])
            p[torch.isinf(l)] = 0.0
            out[b, :r, h] = p @ v[:, h // G]
    return (out, lse) if c["lse"] else out


def _exact_append(s):
    c, cache, table, page = s["case"], s["cache"], s["table"], s["case"]["page"]
    starts = s["starts"].tolist()
    counts = [c["T"]] * c["B"] if s["counts"] is None else s["counts"].tolist()
    scales = [cache["k_scale"].double(), cache["v_scale"].double()]
    outs = [torch.zeros((c["B"], s["read_T"], c["Hkv"], c["D"]), dtype=torch.float64, device=table.device) for _ in (0, 1)]
    for b, (a, n) in enumerate(zip(starts, counts)):
        first, end = a // BLOCK * BLOCK, a + n
        old = _token(cache, table, b, page, range(first, a))
        pad = -end % BLOCK
        at = torch.arange(first, end + pad, BLOCK, device=table.device)
        pg, blk = table[b].long()[at // page], (at % page) // BLOCK
        for i, name in enumerate(("k", "v")):
            x = s[name][b, :n].double()
            zeros = torch.zeros((pad,) + x.shape[1:], dtype=torch.float64, device=x.device)
            new = torch.cat([torch.zeros_like(old[i]), x, zeros]).reshape(-1, BLOCK, c["Hkv"], c["D"])
            scale = new.abs().amax((1, 3)) / 127.0
            if a > first:
                scale[0] = torch.maximum(scale[0], scales[i][pg[0], :, blk[0]])
            whole = torch.cat([old[i], x, zeros]).reshape(-1, BLOCK, c["Hkv"], c["D"])
            step = scale[:, None, :, None]
            kept = torch.where(step > 0, torch.round(whole / step).clamp(-127, 127) * step, torch.zeros_like(whole))
            outs[i][b, :end - first] = kept.reshape(-1, c["Hkv"], c["D"])[:end - first]
            scales[i][pg, :, blk] = scale
    return outs[0], outs[1], scales[0], scales[1]
