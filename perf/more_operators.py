"""Operators around prompts and long caches: what is measured, and their plain forms.

Operators:

- rotary:  queries and keys turned by their positions (half and interleaved pairs, part of the head,
           frequencies scaled for long contexts)
- prompt:  attention over whole prompts of different lengths, packed one behind the other, query heads in
           groups that share a key/value head, causal or to all keys, keys of earlier tokens in front where a
           prompt goes on, with log-sum-exp
- weights: the attention weights that the tokens of an 8-bit paged cache get from a step's queries, summed
           over the queries and heads of each key/value head, added to running scores
- evict:   each head's tokens with the largest scores, and the latest ones, are kept: selected, moved
           together into other pages and read back

A cache holds P pages of ``page`` tokens. Per page, head and block of 32 tokens there are int8 codes of
the keys, ``[D/64][32 tokens][64]``, int8 codes of the values, ``[D][32 positions]`` (token 8j + 2t + e of
the block, with j, t < 4 and e < 2, lies at position 8t + 2j + e), and one fp32 scale each. A page table
names each sequence's pages in order.
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
        # The token that each sequence of a serving batch has just produced, at far positions.
        dict(name="rotary_token", op="rotary", B=64, T=1, H=32, Hkv=8, D=128, rot=128, pairs="half", base=10000.0,
             scaling="none", factor=1.0, original=0, far=120000),
        # A batch of short texts, a quarter of the head turned, interleaved pairs.
        dict(name="rotary_part", op="rotary", B=4, T=333, H=16, Hkv=4, D=64, rot=16, pairs="interleaved", base=10000.0,
             scaling="linear", factor=4.0, original=0, far=0),
        # A long prompt of a context stretched to four times its length.
        dict(name="rotary_prompt", op="rotary", B=1, T=16001, H=32, Hkv=8, D=128, rot=128, pairs="half",
             base=500000.0, scaling="yarn", factor=4.0, original=32768, far=0),
        # One short question: the smallest call, latency counts.
        dict(name="prompt_one", op="prompt", B=1, L=100, lo=1.0, H=28, Hkv=4, D=128, causal=True, lse=False, past=0,
             spare=0),
        # A serving batch: 16 prompts of different lengths, packed, in a buffer with rows to spare.
        dict(name="prompt_batch", op="prompt", B=16, L=2000, lo=0.05, H=32, Hkv=8, D=128, causal=True, lse=True,
             past=0, spare=77),
        # Packed sequences that see themselves in both directions, head dimension 64, no shared heads.
        dict(name="prompt_both_ways", op="prompt", B=8, L=1500, lo=0.2, H=16, Hkv=16, D=64, causal=False, lse=False,
             past=0, spare=0),
        # One long document, at the benchmark's length and heads.
        dict(name="prompt_long", op="prompt", B=1, L=16384, lo=1.0, H=28, Hkv=4, D=128, causal=True, lse=True, past=0,
             spare=0),
        # One sequence answering token by token: what its token looked at.
        dict(name="weights_one", op="weights", B=1, T=1, H=28, Hkv=4, D=128, page=64, L=1000, lo=1.0),
        # The same for a serving batch of 64 sequences of different lengths.
        dict(name="weights_batch", op="weights", B=64, T=1, H=32, Hkv=8, D=128, page=64, L=8192, lo=0.1),
        # A chunk of a long prompt and all that came before it.
        dict(name="weights_chunk", op="weights", B=1, T=2000, H=32, Hkv=8, D=128, page=128, L=16001, lo=1.0),
        # A few conversations cut back to half, the last tokens always kept.
        dict(name="evict_few", op="evict", B=4, Hkv=4, D=64, page=32, L=1000, lo=0.8, keep=500, recent=64),
        # Sixteen long ones cut back to 4096 tokens each.
        dict(name="evict_batch", op="evict", B=16, Hkv=8, D=128, page=64, L=16001, lo=0.2, keep=4096, recent=512),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "prompt", "prompt", "weights", "weights", "evict"])
    D = rng.choice([128, 128, 64])
    page = rng.choice([32, 64, 64, 128])
    Hkv = rng.choice([1, 2, 4, 7, 8])
    G = rng.choice([1, 2, 4, 5, 7, 8])
    lo = round(rng.uniform(0.02, 1.0), 3)
    if op == "rotary":
        B = _log_int(rng, 1, 64)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, B=B, T=_log_int(rng, 1, max(1, 12000 // B)), H=Hkv * min(G, 4), Hkv=Hkv, D=D,
                    rot=rng.choice([D, D, D // 2, 16, 48]), pairs=rng.choice(["half", "interleaved"]),
                    base=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    original=rng.choice([4096, 8192, 32768]) if scaling == "yarn" else 0, far=rng.choice([0, 1000, 1000000]))
    if op == "prompt":
        B = _log_int(rng, 1, 64)
        L = _log_int(rng, 1, min(8000, 24000 // B))
        return dict(op=op, B=B, L=L, lo=lo, H=Hkv * min(G, 4), Hkv=Hkv, D=D, causal=rng.random() < 0.75,
                    lse=rng.random() < 0.5, past=rng.choice([0, 0, _log_int(rng, 1, max(1, min(4000, 24000 // B)))]),
                    spare=rng.choice([0, rng.randrange(1, 200)]))
    if op == "weights":
        if rng.random() < 0.6:
            B, T = _log_int(rng, 1, 64), rng.choice([1, 1, rng.randrange(2, 9)])
            L = _log_int(rng, T, max(T, min(100000, 250000 // B)))
        else:
            B, T = _log_int(rng, 1, 4), _log_int(rng, 9, 700)
            L = T + _log_int(rng, 1, 8000)
        return dict(op=op, B=B, T=T, H=Hkv * G, Hkv=Hkv, D=D, page=page, L=L, lo=lo)
    B = _log_int(rng, 1, 16)
    L = _log_int(rng, 2, min(60000, 120000 // B))
    keep = max(1, int(L * rng.uniform(0.05, 0.9)))
    return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, L=L, lo=lo, keep=keep, recent=int(keep * rng.choice([0.0, 0.1, 0.5])))


def _lengths(c):
    """The sequences' lengths: from lo * L to L, evenly; one prompt of more than eight is empty."""
    B, L = c["B"], c["L"]
    n = [max(1, int(round(L * (c["lo"] + (1 - c["lo"]) * (b + 1) / B)))) for b in range(B)]
    if c["op"] == "prompt" and B > 8:
        n[1] = 0
    return n


def _past(c):
    """Tokens in front of each prompt's own, whose keys it sees too."""
    return [c["past"] * (b + 1) // c["B"] for b in range(c["B"])]


def _inv_freq(c):
    """The angle that a position adds, for each pair of channels (float64)."""
    rot, base, f = c["rot"], c["base"], c["factor"]
    if c["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2.0))
    w = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if c["scaling"] == "linear":
        return w / f
    if c["scaling"] == "yarn":
        def pair(turns):  # the pair that makes this many turns within the original length
            return rot * math.log(c["original"] / (turns * 2.0 * math.pi)) / (2.0 * math.log(base))

        low, high = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        ramp = ((torch.arange(rot // 2, dtype=torch.float64) - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        return w * (1.0 - ramp) + w / f * ramp
    return w


def _magnitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0


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


def _tables(wants, page, spare, g, dev):
    """Page tables whose pages lie in no order, no page in two of them, and the number of pages."""
    need = [[-(-n // page) for n in lengths] for lengths in wants]
    P = sum(map(sum, need)) + spare
    order = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    tables, at = [], 0
    for rows in need:
        table = torch.zeros((len(rows), max(rows)), dtype=torch.int32, device=dev)
        for b, n in enumerate(rows):
            table[b, :n] = order[at:at + n]
            at += n
        tables.append(table)
    return tables, P


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

    if c["op"] == "rotary":
        s["q"], s["k"] = values(c["B"], c["T"], c["H"], c["D"]), values(c["B"], c["T"], c["Hkv"], c["D"])
        first = torch.randint(0, c["far"] + 1, (c["B"], 1), generator=g, device=dev)
        s["positions"] = (first + torch.arange(c["T"], device=dev)).to(torch.int32)
        s["inv_freq"] = _inv_freq(c).to(dev)
        return s
    order = torch.randperm(c["B"], generator=g, device=dev).tolist()
    lengths = [_lengths(c)[b] for b in order]
    if c["op"] == "prompt":
        past = [_past(c)[b] for b in order]
        s["sizes"] = list(zip(lengths, past))  # a program knows the prompts that it packs
        N, M = sum(lengths), sum(lengths) + sum(past)
        ends, kv_ends = [0], [0]
        for n, p in s["sizes"]:
            ends.append(ends[-1] + n)
            kv_ends.append(kv_ends[-1] + n + p)
        s["offsets"], s["kv_offsets"] = ints(ends), ints(kv_ends) if c["past"] else None
        s["q"] = values(N + c["spare"], c["H"], c["D"])
        more = 0 if c["past"] else c["spare"]
        s["k"], s["v"] = values(M + more, c["Hkv"], c["D"]), values(M + more, c["Hkv"], c["D"])
        return s
    s["lengths"] = ints(lengths)
    if c["op"] == "weights":
        (s["table"],), P = _tables([lengths], c["page"], 3, g, dev)
        s["cache"] = _cache(P, c, g, dev)
        s["q"] = values(c["B"], c["T"], c["H"], c["D"])
        # what some earlier steps have left there
        s["scores"] = torch.rand((c["B"], c["Hkv"], max(lengths)), generator=g, device=dev) * (
            8.0 * c["T"] * c["H"] / c["Hkv"] / c["L"])
        lse = torch.empty((c["B"], c["H"], c["T"]), device=dev)
        for b, n in enumerate(lengths):  # the step's attention has computed it before
            k = _tokens(s["cache"], "k", s["table"][b], n, c["page"])
            z = _logits(s["q"][b], k, c["Hkv"], n)
            lse[b] = torch.logsumexp(z, -1).reshape(c["H"], c["T"])
        s["lse"] = lse
        return s
    (s["table"], s["out_table"]), P = _tables([lengths, [min(n, c["keep"]) for n in lengths]], c["page"], 3, g, dev)
    s["cache"] = _cache(P, c, g, dev)
    # accumulated weights: a few tokens have most of them, and many that nothing looked at have none
    scores = torch.exp(torch.randn((c["B"], c["Hkv"], max(lengths)), generator=g, device=dev) * 2.0)
    scores *= torch.rand(scores.shape, generator=g, device=dev) > 0.1
    s["scores"] = scores
    s["starts"] = torch.zeros_like(s["lengths"])
    return s


# -------------------------------------------------------------- plain forms --


def _plain_rotary(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    angle = s["positions"].double()[..., None] * s["inv_freq"]      # [B, T, rot/2]
    cos, sin = ((f(angle) * _magnitude(c)).float()[:, :, None] for f in (torch.cos, torch.sin))
    out = []
    for x in (s["q"], s["k"]):
        y = x.float()
        if c["pairs"] == "half":
            a, b = y[..., :half], y[..., half:rot]
            turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(3)
        out.append(torch.cat([turned, y[..., rot:]], -1).to(torch.bfloat16))
    return tuple(out)


def _plain_prompt(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    G = H // Hkv
    out = torch.zeros_like(q)
    lse = torch.full((H, q.shape[0]), -math.inf, device=q.device)
    at = kv_at = 0
    for n, past in s["sizes"]:
        m = n + past
        kk, vv = (x[kv_at:kv_at + m].float().permute(1, 0, 2) for x in (k, v))   # [Hkv, m, D]
        step = max(1, (1 << 28) // max(1, H * m))
        for t in range(0, n, step):
            r = min(step, n - t)
            w = min(m, past + t + r) if c["causal"] else m           # keys that some row of these sees
            x = q[at + t:at + t + r].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3).reshape(Hkv, G * r, D)
            z = (x @ kk[:, :w].transpose(1, 2)) * (1.0 / math.sqrt(D))
            z = z.unflatten(1, (G, r))
            if c["causal"]:
                seen = torch.arange(w, device=q.device) <= torch.arange(t, t + r, device=q.device)[:, None] + past
                z = z.masked_fill_(~seen, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = z.sub_(top).exp_()
            total = p.sum(-1, keepdim=True)
            o = (p.flatten(1, 2) @ vv[:, :w]).unflatten(1, (G, r)) / total
            out[at + t:at + t + r] = o.permute(2, 0, 1, 3).reshape(r, H, D).to(torch.bfloat16)
            lse[:, at + t:at + t + r] = (top + total.log()).reshape(H, r)
        at, kv_at = at + n, kv_at + m
    return (out, lse) if c["lse"] else out


def _position(i):
    return i % 8 // 2 * 8 + i // 8 * 2 + i % 2


def _tokens(cache, name, row, n, page):
    """Keys or values of the first n tokens that a row of the table names, fp32 [Hkv, n, D]."""
    x, scale = cache[name + "_codes"][row.long()], cache[name + "_scale"][row.long()]   # [N, Hkv, n, ...]
    if name == "k":
        x = x.permute(1, 0, 2, 4, 3, 5).flatten(4)                  # [Hkv, N, n, 32, D]
    else:
        x = x[..., _position(torch.arange(BLOCK, device=x.device))].permute(1, 0, 2, 4, 3)
    x = x.float() * scale.permute(1, 0, 2)[..., None, None]
    return x.flatten(1, 3)[:, :n]


def _logits(q, k, Hkv, n):
    """Causal logits of a sequence's last tokens q [T, H, D] with its keys k [Hkv, n, D]: [Hkv, G, T, n]."""
    T, H, D = q.shape
    x = q.float().unflatten(1, (Hkv, H // Hkv)).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    z = ((x @ k.transpose(1, 2)) * (1.0 / math.sqrt(D))).unflatten(1, (H // Hkv, T))
    hidden = torch.arange(n, device=q.device) > torch.arange(n - T, n, device=q.device)[:, None]
    return z.masked_fill_(hidden, -math.inf)


def _plain_weights(s):
    c, q, scores = s["case"], s["q"], s["scores"]
    B, T, H, D = q.shape
    Hkv, G, page = c["Hkv"], c["H"] // c["Hkv"], c["page"]
    pages = s["table"].long()
    k = s["cache"]["k_codes"][pages].permute(0, 2, 1, 3, 5, 4, 6).flatten(5, 6)   # [B, Hkv, N, n, 32, D]
    k = k.float() * s["cache"]["k_scale"][pages].permute(0, 2, 1, 3)[..., None, None]
    k = k.flatten(2, 4)[:, :, :scores.shape[2]]                     # [B, Hkv, L, D]
    x = q.float().unflatten(2, (Hkv, G)).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * T, D)
    z = (x @ k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    z = z.unflatten(2, (G, T))                                      # [B, Hkv, G, T, L]
    last = s["lengths"].long()[:, None] - T + torch.arange(T, device=q.device)
    seen = torch.arange(z.shape[-1], device=q.device) <= last[..., None]   # [B, T, L]
    w = z.sub_(s["lse"].unflatten(1, (Hkv, G))[..., None]).exp_()
    w = w.masked_fill_(~seen[:, None, None], 0.0)
    scores += w.sum((2, 3))
    return scores


def _plain_evict(s):
    c, cache, scores = s["case"], s["cache"], s["scores"]
    B, Hkv, S = scores.shape
    D, page, keep = c["D"], c["page"], c["keep"]
    dev = scores.device
    n = s["lengths"].long()
    new = n.clamp_max(keep)                                         # tokens that stay
    recent = n.clamp_max(c["recent"])
    i = torch.arange(S, device=dev)
    first = (n - recent)[:, None, None]                             # tokens that the scores decide on: those before
    x = torch.where(i < first, scores, torch.full((), -math.inf, device=dev))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, i.expand_as(order).contiguous())
    stays = ((i < first) & (rank < (new - recent)[:, None, None])) | ((i >= first) & (i < n[:, None, None]))
    K = min(keep, S)
    at = torch.sort((~stays).to(torch.uint8), dim=-1, stable=True).indices[..., :K]   # [B, Hkv, K], in order
    there = torch.arange(K, device=dev) < new[:, None, None]
    kept = torch.where(there, at, -1).to(torch.int32)
    moved = torch.zeros_like(scores)
    moved[..., :K] = scores.gather(-1, at) * there
    # the tokens' codes and scales
    pad = -K % BLOCK
    at = torch.nn.functional.pad(at, (0, pad))
    there = torch.nn.functional.pad(there.expand_as(kept), (0, pad))
    b = torch.arange(B, device=dev)[:, None, None]
    h = torch.arange(Hkv, device=dev)[:, None]
    pg, blk, slot = s["table"].long()[b, at // page], at % page // BLOCK, at % BLOCK
    M = (K + pad) // BLOCK
    block = torch.arange(M, device=dev)
    to = s["out_table"].long()[:, (block * BLOCK // page).clamp_max(s["out_table"].shape[1] - 1)][:, None].expand(B, Hkv, M)
    to_blk = (block % (page // BLOCK)).expand(B, Hkv, M)
    used = block * BLOCK < new[:, None, None].expand(B, Hkv, 1)     # [B, Hkv, M]
    where = (to[used], h.expand(B, Hkv, M)[used], to_blk[used])
    position = _position(torch.arange(BLOCK, device=dev))
    for name in ("k", "v"):
        scale = (cache[name + "_scale"][pg, h, blk] * there).unflatten(2, (M, BLOCK))
        if name == "k":
            codes = cache["k_codes"][pg, h, blk, :, slot].flatten(3)
        else:
            codes = cache["v_codes"][pg, h, blk, :, _position(slot)]
        most = scale.amax(-1)
        ratio = scale / most.clamp_min(1e-45)[..., None]
        codes = (codes.unflatten(2, (M, BLOCK)).float() * ratio[..., None]).round().to(torch.int8)   # [B, Hkv, M, 32, D]
        if name == "k":
            codes = codes.unflatten(4, (D // 64, 64)).transpose(3, 4)
        else:
            codes = torch.empty((B, Hkv, M, D, BLOCK), dtype=torch.int8, device=dev).index_copy_(4, position, codes.transpose(3, 4))
        cache[name + "_codes"][where] = codes[used]
        cache[name + "_scale"][where] = most[used]
    out = []
    for name in ("k", "v"):
        x = torch.stack([_tokens(cache, name, s["out_table"][b], K, page) for b in range(B)])
        x = torch.nn.functional.pad(x, (0, 0, 0, K - x.shape[2])) * there[..., :K, None]
        out.append(x.transpose(1, 2).to(torch.bfloat16))
    return new.to(torch.int32), kept, moved, out[0], out[1]


# ---------------------------------------------------------------------- run --


def _handles(s):
    """The framework's objects: what a program makes once and keeps."""
    if "sage" not in s:
        import quantized_attention_fp64_gb300 as sage

        c = s["case"]
        s["sage"] = sage
        if c["op"] == "rotary":
            s["angles"] = sage.rotary_table(c["rot"], base=c["base"], scaling=None if c["scaling"] == "none" else c["scaling"],
                                            factor=c["factor"], original_length=c["original"] or None, device=s["q"].device)
        elif c["op"] != "prompt":
            s["handle"] = sage.QuantizedCache(**s["cache"])
    return s["sage"], s.get("handle")


def run(s):
    c = s["case"]
    op = c["op"]
    if own:
        sage, cache = _handles(s)
        if op == "rotary":
            return sage.rotary(s["q"], s["k"], s["positions"], s["angles"], interleaved=c["pairs"] == "interleaved")
        if op == "prompt":
            return sage.prompt_attention(s["q"], s["k"], s["v"], s["offsets"], kv_offsets=s["kv_offsets"],
                                         is_causal=c["causal"], return_lse=c["lse"])
        if op == "weights":
            return sage.cache_add_weights(s["scores"], s["q"], cache, s["table"], s["lengths"], s["lse"], is_causal=True)
        lengths, kept, scores = sage.cache_evict(cache, s["table"], s["lengths"], s["scores"], c["keep"],
                                                 recent=c["recent"], out_table=s["out_table"])
        k, v = sage.cache_read(cache, s["out_table"], s["starts"], kept.shape[2], counts=lengths)
        return lengths, kept, scores, k, v
    return dict(rotary=_plain_rotary, prompt=_plain_prompt, weights=_plain_weights, evict=_plain_evict)[op](s)


# --------------------------------------------------------------------- work --


def work(case):
    c = case
    D, Hkv = c["D"], c["Hkv"]
    if c["op"] == "rotary":
        tokens = c["B"] * c["T"]
        return dict(bytes=tokens * (4.0 * (c["H"] + Hkv) * D + 4), flops=tokens * (c["H"] + Hkv) * c["rot"] * 3.0)
    bytes_, flops = 0.0, 0.0
    if c["op"] == "prompt":
        for n, p in zip(_lengths(c), _past(c)):
            bytes_ += 4.0 * n * c["H"] * D + 4.0 * (n + p) * Hkv * D + (4.0 * n * c["H"] if c["lse"] else 0)
            flops += 4.0 * c["H"] * D * (n * p + n * (n + 1) / 2 if c["causal"] else n * (n + p))
        return dict(bytes=bytes_, flops=flops)
    half = Hkv * (D + 4 / BLOCK)                                    # bytes of a cached token's keys
    for n in _lengths(c):
        if c["op"] == "weights":
            T = c["T"]
            bytes_ += n * (half + 8 * Hkv) + T * c["H"] * (2 * D + 4)
            flops += 2.0 * c["H"] * D * sum(max(0, n - T + t + 1) for t in range(T))
        else:
            m = min(n, c["keep"])
            # selected, moved (read and written), read back (read, and written in BF16)
            bytes_ += 4 * n * Hkv + m * (8 * Hkv + 6 * half + 4 * Hkv * D)
    return dict(bytes=bytes_, flops=flops)


# -------------------------------------------------------- the definition, 64 --


def _cached(cache, row, page, h, ids):
    """Key and value of tokens ids (int64) of head h of a sequence, float64 [n, D] each, and their scales."""
    p, i = row.long()[ids // page], ids % BLOCK
    blk = (ids % page) // BLOCK
    j, r = i // 8, i % 8
    ks, vs = (cache[x + "_scale"][p, h, blk].double() for x in "kv")
    k = cache["k_codes"][p, h, blk, :, i].double().flatten(1) * ks[:, None]
    v = cache["v_codes"][p, h, blk, :, (r // 2) * 8 + 2 * j + r % 2].double() * vs[:, None]
    return k, v, ks, vs


def exact(case, seed):
    s = prepare(case, seed)
    return dict(rotary=_exact_rotary, prompt=_exact_prompt, weights=_exact_weights, evict=_exact_evict)[case["op"]](s)


def _exact_rotary(s):
    c = s["case"]
    turn = torch.polar(torch.full((), _magnitude(c), dtype=torch.float64, device=s["q"].device),
                       s["positions"][:, :, None, None].double() * s["inv_freq"])   # [B, T, 1, rot/2]
    out = []
    for x in (s["q"], s["k"]):
        y = x.double()
        part = y[..., :c["rot"]]
        pair = part.unflatten(3, (2, -1)).transpose(3, 4) if c["pairs"] == "half" else part.unflatten(3, (-1, 2))
        pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
        y[..., :c["rot"]] = (pair.transpose(3, 4) if c["pairs"] == "half" else pair).flatten(3)
        out.append(y)
    return tuple(out)


def _exact_prompt(s):
    c = s["case"]
    H, G, D = c["H"], c["H"] // c["Hkv"], c["D"]
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.full((H, s["q"].shape[0]), -math.inf, dtype=torch.float64, device=dev)
    at = kv_at = 0
    for n, past in s["sizes"]:
        keys = range(kv_at, kv_at + n + past)
        for h in range(H):
            k, v = (s[x][keys.start:keys.stop, h // G].double() for x in "kv")
            for a in range(0, n, 4096):
                b = min(n, a + 4096)
                z = s["q"][at + a:at + b, h].double() @ k.T / math.sqrt(D)
                if c["causal"]:
                    z += torch.full_like(z, -math.inf).triu_(past + a + 1)
                l = torch.logsumexp(z, 1)
                lse[h, at + a:at + b] = l
                out[at + a:at + b, h] = torch.exp(z - l[:, None]) @ v
        at, kv_at = at + n, keys.stop
    return (out, lse) if c["lse"] else out


def _exact_weights(s):
    c = s["case"]
    H, G, T, D = c["H"], c["H"] // c["Hkv"], c["T"], c["D"]
    scores = s["scores"].double()
    for b, n in enumerate(s["lengths"].tolist()):
        ids = torch.arange(n, device=scores.device)
        for h in range(c["Hkv"]):
            k = _cached(s["cache"], s["table"][b], c["page"], h, ids)[0]
            for g in range(h * G, (h + 1) * G):
                z = s["q"][b, :, g].double() @ k.T / math.sqrt(D)
                w = torch.exp(z - s["lse"][b, g].double()[:, None]).tril_(n - T)
                scores[b, h, :n] += w.sum(0)
    return scores


def _exact_evict(s):
    c = s["case"]
    B, Hkv, S = s["scores"].shape
    K, D, page = min(c["keep"], S), c["D"], c["page"]
    dev = s["scores"].device
    kept = torch.full((B, Hkv, K), -1, dtype=torch.int32, device=dev)
    moved = torch.zeros((B, Hkv, S), dtype=torch.float64, device=dev)
    k_out, v_out = (torch.zeros((B, K, Hkv, D), dtype=torch.float64, device=dev) for _ in "kv")
    new = []
    for b, n in enumerate(s["lengths"].tolist()):
        m, last = min(n, K), min(n, c["recent"])
        new.append(m)
        for h in range(Hkv):
            x = s["scores"][b, h, :n - last].double().cpu().numpy()
            best = (-x).argsort(kind="stable")[:m - last].tolist()
            ids = torch.tensor(sorted(best) + list(range(n - last, n)), dtype=torch.int64, device=dev)
            kept[b, h, :m] = ids.to(torch.int32)
            moved[b, h, :m] = s["scores"][b, h][ids].double()
            k, v, ks, vs = _cached(s["cache"], s["table"][b], page, h, ids)
            for x, scale, to in ((k, ks, k_out), (v, vs, v_out)):
                top = torch.stack([p.max() for p in scale.split(BLOCK)]).repeat_interleave(BLOCK)[:m, None]
                to[b, :m, h] = torch.where(top > 0, torch.round(x / top) * top, torch.zeros_like(x))
    return torch.tensor(new, dtype=torch.int32, device=dev), kept, moved, k_out, v_out
