"""Attention weights of cached tokens and eviction by them, on the GPU against the oracle.

A weight w = exp(z - lse) is held to what fp32 can do: the logit's D products (exact in fp32) and their sum err by at
most D 2^-23 sm_scale |q| |k| (Cauchy), its scale and the log-sum-exp in base 2 by 2^-22 (|z| + |lse|), the
exponential by 2^-21 in all. Sums of R weights err by R 2^-24 of the sum at most, adding to the old score by half a
step. Selected tokens, moved codes and scales have to be equal.
"""

import math

import numpy as np
import pytest
import torch

import quantized_attention_fp64_gb300 as sage
from oracle import cache as oc
from quantized_attention_fp64_gb300.api import SageError
from test_cache_gpu import (ATTENTION, DEVICE_PAGE, _library, bf16, dev, f32, ints, make_table, poison_unused,  # noqa: F401
                            random_cache, upload)

pytestmark = pytest.mark.gpu


def weights(c, q, table, lengths, q_lengths, lse, causal, sm, S):
    """(sums, bounds) of the weights, float64 [B, H, S]."""
    B, T, H, D = q.shape
    G = H // c.H
    total, bound = np.zeros((2, B, c.H, S))
    for b in range(B):
        n, r = int(lengths[b]), int(q_lengths[b])
        k, _ = c.tokens(table[b], 0, n)
        sees = np.clip(n - r + 1 + np.arange(r), 0, n) if causal else np.full(r, n)
        for h in range(H):
            z = q[b, :r, h].astype(np.float64) @ k[:, h // G].T * sm
            l = lse[b, h, :r].astype(np.float64)[:, None]
            hidden = (np.arange(n)[None, :] >= sees[:, None]) | np.isinf(l)
            w = np.where(hidden, 0.0, np.exp(np.where(hidden, 0.0, z - np.where(np.isinf(l), 0.0, l))))
            size = np.linalg.norm(q[b, :r, h].astype(np.float64), axis=1)[:, None] * np.linalg.norm(k[:, h // G], axis=1)[None, :]
            err = D * 2.0 ** -23 * sm * size + 2.0 ** -22 * (np.abs(z) + np.where(np.isinf(l), 0.0, np.abs(l))) + 2.0 ** -21
            m = min(n, S)
            total[b, h // G, :m] += w.sum(0)[:m]
            bound[b, h // G, :m] += (w * err).sum(0)[:m] + r * 2.0 ** -24 * w.sum(0)[:m]
    return total, bound * 1.01


def add(rng, H, Hkv, D, page, lengths, q_lengths, T, causal, layout="NHD", sm=None, S=None):
    B = len(lengths)
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    poison_unused(c, table, lengths)
    q = bf16(rng, B, T, H, D)
    scale = 1 / math.sqrt(D) if sm is None else sm
    ql = [T] * B if q_lengths is None else q_lengths
    for b, r in enumerate(ql):
        q[b, r:] = math.nan  # padding may hold anything
    gpu = upload(c)
    S = max(lengths + [1]) + 5 if S is None else S
    wide = torch.from_numpy(rng.random((B, Hkv, S + 3)).astype(np.float32)).cuda()
    scores = wide[:, :, 1:S + 1]
    before = f32(scores).astype(np.float64)
    qq = q if layout == "NHD" else q.transpose(1, 2).contiguous()
    kw = dict(q_lengths=None if q_lengths is None else ints(q_lengths), is_causal=causal, sm_scale=sm, tensor_layout=layout)
    _, lse = sage.cache_attention(qq, gpu, ints(table), ints(lengths), return_lse=True, **kw)
    edges = wide[:, :, 0].clone(), wide[:, :, S + 1:].clone()
    got = sage.cache_add_weights(scores, qq, gpu, ints(table), ints(lengths), lse, **kw)
    assert got is scores and torch.equal(edges[0], wide[:, :, 0]) and torch.equal(edges[1], wide[:, :, S + 1:])
    total, bound = weights(c, f32(q), table, lengths, ql, f32(lse), causal, scale, S)
    after = f32(scores).astype(np.float64)
    tol = bound + 2.0 ** -24 * np.abs(after)
    bad = ~(np.abs(after - before - total) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4].tolist(), float(np.nanmax((np.abs(after - before - total) / (tol + 1e-30)))))
    for b, n in enumerate(lengths):
        assert (after[b, :, min(n, S):] == before[b, :, min(n, S):]).all()
    # the same again, bit for bit
    again = torch.from_numpy(before.astype(np.float32)).cuda()
    sage.cache_add_weights(again, qq, gpu, ints(table), ints(lengths), lse, **kw)
    assert torch.equal(again, scores)


WEIGHTS = ATTENTION + [
    (7, 1, 128, 64, [500], None, 33, True),                   # 7 heads do not divide a tile's 128 rows
    (12, 1, 64, 64, [500, 129, 1], [40, 3, 1], 40, True),
    (130, 1, 64, 64, [200, 40], None, 3, True),               # more heads in a group than a tile has rows
    (4, 4, 128, 128, [129], None, 128, True),
    (2, 1, 128, 64, [128 * 5], None, 640, True),
    (8, 1, 128, 64, [20000], None, 20, True),
]


@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_weights(case):
    add(np.random.default_rng(100 + case), *WEIGHTS[case])


@pytest.mark.parametrize("T", [1, 5, 60])
def test_weights_layout_scale_and_short_scores(T):
    add(np.random.default_rng(7), 8, 2, 128, 64, [300, 77], None, T, True, layout="HND")
    add(np.random.default_rng(8), 8, 2, 64, 64, [300, 77], None, T, False, sm=0.3)
    add(np.random.default_rng(9), 8, 2, 64, 64, [300, 77, 10], None, T, True, S=130)
    add(np.random.default_rng(10), 2, 2, 128, 32, [300, 77, 0], None, T, True, S=1)


@pytest.mark.parametrize("T", [2, 50])
def test_weights_sum_to_the_rows(T):
    """All rows' weights add up to their number: each row's are a softmax."""
    rng = np.random.default_rng(11)
    lengths, H, Hkv, D = [1000, 333], 8, 2, 128
    table, P = make_table(rng, lengths, 64)
    gpu = upload(random_cache(rng, P, Hkv, D, 64))
    q = bf16(rng, 2, T, H, D)
    _, lse = sage.cache_attention(q, gpu, ints(table), ints(lengths), is_causal=True, return_lse=True)
    scores = torch.zeros((2, Hkv, 1000), device="cuda")
    sage.cache_add_weights(scores, q, gpu, ints(table), ints(lengths), lse, is_causal=True)
    want = T * H // Hkv
    assert ((scores.double().sum(-1) - want).abs() <= want * 2.0 ** -11).all()  # the log-sum-exp errs by up to 2^-13


@pytest.mark.parametrize("T", [1, 7, 50])
def test_weights_nan_stays_with_what_it_touches(T):
    rng = np.random.default_rng(12)
    lengths, H, Hkv, D, page = [200, 150], 4, 2, 128, 64
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    c.k_scale[table[0][1], 1, 0] = np.nan  # tokens 64 .. 95 of sequence 0, head 1
    gpu = upload(c)
    q = bf16(rng, 2, T, H, D)
    lse = torch.full((2, H, T), 3.0, device="cuda")
    lse[1, 0, T - 1] = math.nan           # the last row of head 0 (key/value head 0) sees all tokens of sequence 1
    lse[1, 3] = -math.inf                 # rows that saw nothing
    scores = torch.zeros((2, Hkv, 200), device="cuda")
    sage.cache_add_weights(scores, q, gpu, ints(table), ints(lengths), lse, is_causal=True)
    odd = torch.isnan(scores)
    want = torch.zeros_like(odd)
    want[0, 1, 64:96] = True
    want[1, 0, :150] = True
    assert torch.equal(odd, want)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,H", [(128, 4), (64, 10), (64, 2)])
@pytest.mark.parametrize("T", [3, 7, 50, 140])
def test_weights_log_sum_exps_that_are_nan(T, D, H, causal):
    """Rows anywhere whose log-sum-exp is a NaN: the keys that they see become NaN, and all others are as without them."""
    rng = np.random.default_rng(15)
    lengths, q_lengths, Hkv, page = [400, 150, 290], [T, T - 1, T], 2, 64
    table, P = make_table(rng, lengths, page)
    gpu = upload(random_cache(rng, P, Hkv, D, page))
    q = bf16(rng, 3, T, H, D)
    args = dict(cache=gpu, page_table=ints(table), lengths=ints(lengths), q_lengths=ints(q_lengths), is_causal=causal)
    _, lse = sage.cache_attention(q, return_lse=True, **args)
    lse[2, 0, T - 1] = math.inf  # weighs nothing
    start = torch.from_numpy(rng.random((3, Hkv, 400)).astype(np.float32)).cuda()
    rows = [(0, 0, 0), (0, H - 1, T // 2), (1, H // 2, T // 3), (1, 0, T - 1), (2, H - 1, 0), (2, H - 1, T - 1)]  # (1, 0, T - 1) is none
    for some in ([r] for r in rows), [rows]:
        for marks in some:
            without, odd = lse.clone(), lse.clone()
            want_nan = torch.zeros_like(start, dtype=torch.bool)
            for b, h, t in marks:
                without[b, h, t], odd[b, h, t] = -math.inf, math.nan
                if t < q_lengths[b]:
                    want_nan[b, h // (H // Hkv), :lengths[b] - q_lengths[b] + t + 1 if causal else lengths[b]] = True
            want = sage.cache_add_weights(start.clone(), q, lse=without, **args)
            got = sage.cache_add_weights(start.clone(), q, lse=odd, **args)
            assert not torch.isnan(want).any()
            assert torch.equal(torch.isnan(got), want_nan)
            assert torch.equal(got[~want_nan], want[~want_nan])


@pytest.mark.parametrize("lse", [3.0, 500.0, -math.inf])
@pytest.mark.parametrize("T", [3, 50, 140])
def test_weights_keys_whose_scale_is_a_nan(T, lse):
    """A NaN in a key's scale makes its score a NaN if a row sees it, however small the weight, and not otherwise."""
    rng = np.random.default_rng(16)
    lengths, H, Hkv, D, page = [200, 260], 4, 2, 128, 64
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    c.k_scale[table[0][1], 1, 0] = np.nan   # tokens 64 .. 95 of sequence 0
    c.k_scale[table[1][4], 0, 0] = np.nan   # the last four tokens of sequence 1
    gpu = upload(c)
    q = bf16(rng, 2, T, H, D)
    l = torch.full((2, H, T), lse, device="cuda")
    l[1, :2, T - 2:] = -math.inf            # the last two rows of head 0 add nothing: the last two keys have no row
    start = torch.from_numpy(rng.random((2, Hkv, 260)).astype(np.float32)).cuda()
    got = sage.cache_add_weights(start.clone(), q, gpu, ints(table), ints(lengths), l, is_causal=True)
    want = torch.zeros_like(got, dtype=torch.bool)
    if lse > 0:
        want[0, 1, 64:96] = True
        want[1, 0, 256:258] = True
    assert torch.equal(torch.isnan(got), want)
    assert torch.equal(got[1, 0, 258:], start[1, 0, 258:]) and torch.equal(got[0, :, 200:], start[0, :, 200:])


@pytest.mark.parametrize("T", [1, 5, 40])
def test_weights_leave_scores_of_unseen_tokens_as_they_were(T):
    """To the bit: -0 and NaN with a payload, of tokens that no row sees, behind the sequence, and where a row's
    log-sum-exp is minus infinity."""
    rng = np.random.default_rng(17)
    lengths, H, Hkv, D, page = [100, 64, 0], 4, 2, 64, 64
    table, P = make_table(rng, lengths, page)
    gpu = upload(random_cache(rng, P, Hkv, D, page))
    q = bf16(rng, 3, T, H, D)
    start = torch.full((3, Hkv, 130), -0.0, device="cuda")
    start.view(torch.int32)[:, :, ::5] = 0x7FC12345
    lse = torch.full((3, H, T), 3.0, device="cuda")
    lse[1] = -math.inf
    lse[0, :2] = -math.inf
    q_lengths = ints([T, T, T])
    got = sage.cache_add_weights(start.clone(), q, gpu, ints(table), ints(lengths), lse, q_lengths=q_lengths, is_causal=True)
    a, b = start.view(torch.int32), got.view(torch.int32)
    assert torch.equal(a[1:], b[1:]) and torch.equal(a[0, 0], b[0, 0]) and torch.equal(a[0, 1, 100:], b[0, 1, 100:])
    seen = torch.ones(100, dtype=torch.bool, device="cuda")
    seen[::5] = False
    assert (got[0, 1, :100][seen] > 0).all() and torch.isnan(got[0, 1, :100][~seen]).all()


@pytest.mark.parametrize("T", [1, 50])
def test_weights_bad_pages_and_lengths_are_flagged(T):
    rng = np.random.default_rng(13)
    lengths, H, Hkv, D, page = [256, 256], 4, 2, 64, 64
    table, P = make_table(rng, lengths, page)
    gpu = upload(random_cache(rng, P, Hkv, D, page))
    q = bf16(rng, 2, T, H, D)
    lse = torch.full((2, H, T), 5.0, device="cuda")
    ref = sage.cache_add_weights(torch.zeros((2, Hkv, 256), device="cuda"), q, gpu, ints(table), ints(lengths), lse)
    assert sage.device_error() == 0
    broken = table.copy()
    broken[0, 1] = P
    got = sage.cache_add_weights(torch.zeros((2, Hkv, 256), device="cuda"), q, gpu, ints(broken), ints(lengths), lse)
    assert sage.device_error() == DEVICE_PAGE
    want = ref.clone()
    want[0, :, 64:128] = 0
    assert torch.equal(got, want)
    for change in (dict(lengths=ints([300, -1])), dict(q_lengths=ints([T + 1, 0])), dict(q_lengths=ints([-1, 0]))):
        args = {**dict(lengths=ints(lengths)), **change}
        sage.cache_add_weights(torch.zeros((2, Hkv, 256), device="cuda"), q, gpu, ints(table), args["lengths"], lse,
                               q_lengths=args.get("q_lengths"))
        assert sage.device_error() == DEVICE_PAGE


def test_weights_refusals_and_empty_calls():
    rng = np.random.default_rng(14)
    table, P = make_table(rng, [40], 64)
    gpu = upload(random_cache(rng, P, 2, 64, 64))
    q, lse = bf16(rng, 1, 3, 4, 64), torch.zeros((1, 4, 3), device="cuda")
    scores = torch.zeros((1, 2, 40), device="cuda")
    good = dict(scores=scores, q=q, cache=gpu, page_table=ints(table), lengths=ints([40]), lse=lse)
    for change, code in [
        (dict(scores=scores.half()), -3), (dict(scores=scores[0]), -5), (dict(scores=scores[:, :1]), -5),
        (dict(scores=torch.zeros((1, 2, 80), device="cuda")[:, :, ::2]), -6), (dict(q=q.float()), -3), (dict(q=q[:, :, :3]), -5),
        (dict(lse=lse.double()), -3), (dict(lse=lse[:, :, :2]), -5), (dict(lse=lse.transpose(1, 2).contiguous().transpose(1, 2)), -6),
        (dict(lengths=ints([40, 1])), -5), (dict(lengths=torch.tensor([40], device="cuda")), -3), (dict(sm_scale=-1.0), -13),
        (dict(tensor_layout="x"), -6), (dict(q=bf16(rng, 1, 3, 4, 128)), -5)]:
        with pytest.raises(SageError) as err:
            sage.cache_add_weights(**{**good, **change})
        assert err.value.code == code, change
    with pytest.raises(TypeError):
        sage.cache_add_weights(**{**good, "lse": None})
    with pytest.raises(ValueError):
        sage.cache_add_weights(**{**good, "lse": lse.cpu()})
    empty = sage.cache_add_weights(scores[:, :, :0], q, gpu, ints(table), ints([40]), lse)
    assert empty.shape == (1, 2, 0)
    sage.cache_add_weights(scores, q[:, :0], gpu, ints(table), ints([40]), lse[:, :, :0])
    sage.cache_add_weights(scores, q, gpu, ints(table)[:, :0], ints([0]), lse)
    assert (scores == 0).all()


# ------------------------------------------------------------------ eviction --


def select(x, n, keep, recent):
    """The tokens that stay, in order."""
    stay = min(n, keep)
    last = min(recent, stay)
    y = x[:n - last].astype(np.float64)
    y = np.where(np.isnan(y), -np.inf, y)
    nan_last = np.isnan(x[:n - last])
    order = np.lexsort((np.arange(n - last), nan_last, -y))  # by score, NaN behind -inf, then by place
    return sorted(order[:stay - last].tolist()) + list(range(n - last, n))


def evict(c: oc.Cache, table, lengths, scores, keep, recent, out_table):
    """The oracle's eviction: changes c; returns lengths, kept and scores."""
    B, H, S = scores.shape
    new, K = np.zeros(B, np.int64), min(keep, S)
    kept, moved = np.full((B, H, K), -1), np.zeros((B, H, S), np.float32)
    old = [x.copy() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    src = oc.Cache.__new__(oc.Cache)
    src.page_size, src.H, src.D = c.page_size, c.H, c.D
    src.k_codes, src.v_codes, src.k_scale, src.v_scale = old
    for b in range(B):
        n = int(lengths[b])
        for h in range(H):
            ids = select(scores[b, h], n, keep, recent)
            new[b] = m = len(ids)
            kept[b, h, :m], moved[b, h, :m] = ids, scores[b, h, ids]
            for i0 in range(0, m, 32):
                part = ids[i0:i0 + 32]
                at = [src.at(table[b], i) for i in part]
                page, blk = c.at(out_table[b], i0)
                both = [list(x) for x in c.block_codes(page, blk)]
                for which, scales in enumerate((src.k_scale, src.v_scale)):
                    s = np.array([scales[p, h, q] for p, q in at], np.float32)
                    top = np.float32(np.nan) if np.isnan(s).any() else s.max()
                    codes = np.zeros((32, c.D), np.int8)
                    for i, ((p, q), t) in enumerate(zip(at, part)):
                        if top > 0:
                            codes[i] = np.rint(src.block_codes(p, q)[which][t % 32, h].astype(np.float32) * (s[i] / top))
                    whole = np.array(both[which])
                    whole[:, h] = codes
                    both[which] = whole
                    (c.k_scale, c.v_scale)[which][page, h, blk] = top
                c.set_block_codes(page, blk, *[np.array(x) for x in both])
    return new, kept, moved


def same_cache(gpu, c):
    for x, y in ((gpu.k_codes, c.k_codes), (gpu.v_codes, c.v_codes)):
        bad = np.argwhere(x.cpu().numpy() != y)
        assert not len(bad), (len(bad), bad[:3].tolist())
    for x, y in ((gpu.k_scale, c.k_scale), (gpu.v_scale, c.v_scale)):
        x = x.cpu().numpy()
        assert np.array_equal(np.isnan(x), np.isnan(y)) and np.array_equal(x[~np.isnan(x)], y[~np.isnan(y)])


def some_scores(rng, B, H, S):
    """A few large ones, many equal ones (zeros among them), some negative."""
    x = np.exp(rng.standard_normal((B, H, S)) * 2).astype(np.float32)
    x[rng.random(x.shape) < 0.3] = 0.0
    x[rng.random(x.shape) < 0.1] = -0.0
    x[rng.random(x.shape) < 0.2] = 1.5
    x[rng.random(x.shape) < 0.05] *= -1
    return x


EVICTIONS = [
    # H, D, page, lengths, keep, recent
    (1, 128, 32, [40], 20, 5),
    (2, 64, 64, [1], 1, 0),
    (2, 64, 64, [5, 0, 3], 0, 0),
    (2, 128, 64, [100, 31, 64, 65], 64, 64),
    (3, 64, 32, [333, 12, 0, 290], 96, 0),
    (2, 128, 96, [500, 499, 1000], 333, 32),
    (1, 64, 128, [3000], 2999, 1),
    (1, 128, 64, [2500], 100, 0),
    (4, 64, 64, [700, 1500], 800, 799),
    (1, 64, 64, [9000], 1, 0),
    (2, 128, 64, [9000, 40], 4100, 77),
    (1, 64, 32, [(7 * i) % 90 for i in range(200)], 40, 3),
]


@pytest.mark.parametrize("place", ["in place", "other pages"])
@pytest.mark.parametrize("case", range(len(EVICTIONS)))
def test_evict(case, place):
    H, D, page, lengths, keep, recent = EVICTIONS[case]
    rng = np.random.default_rng(200 + case)
    B, S = len(lengths), max(lengths + [1]) + 3
    out_lengths = [min(n, keep) for n in lengths]
    both, P = make_table(rng, lengths + out_lengths, page)
    table, out_table = both[:B], both[B:]
    c = random_cache(rng, P, H, D, page)
    poison_unused(c, both, lengths + out_lengths)
    scores = some_scores(rng, B, H, S)
    scores[:, :, ::7] = np.where(rng.random(scores[:, :, ::7].shape) < 0.1, np.nan, scores[:, :, ::7])
    gpu = upload(c)
    old = dev(scores)
    new, kept, moved = sage.cache_evict(gpu, ints(table), ints(lengths), old, keep, recent=recent,
                                        out_table=None if place == "in place" else ints(out_table))
    want = evict(c, table, lengths, scores, keep, recent, table if place == "in place" else out_table)
    assert np.array_equal(new.cpu().numpy(), want[0])
    assert np.array_equal(kept.cpu().numpy(), want[1])
    assert np.array_equal(moved.cpu().numpy(), want[2], equal_nan=True)
    assert np.array_equal(old.cpu().numpy(), scores, equal_nan=True)
    same_cache(gpu, c)


@pytest.mark.parametrize("D", [64, 128])
def test_evict_one_sequence_in_place_by_another_view(D):
    """A single row of the table may be passed as another view of it, whose distance to a next row is another one."""
    H, page, n, keep, recent = 4, 64, 9000, 5000, 40
    S = n + 3
    for seed in range(3):
        rng = np.random.default_rng(240 + seed)
        table, P = make_table(rng, [n], page)
        c = random_cache(rng, P, H, D, page)
        scores = some_scores(rng, 1, H, S)
        gpu = upload(c)
        row = ints(table)
        first = row[0][:-(-keep // page)][None]      # the columns that the result needs
        assert first.data_ptr() == row.data_ptr() and first.stride(0) != row.stride(0)
        wide = row.as_strided(row.shape, (row.stride(0) + 7, 1))
        for out_table in ((first, wide) if seed % 2 else (wide, first)):
            _, kept, moved = sage.cache_evict(gpu, row, ints([n]), dev(scores), keep, recent=recent, out_table=out_table)
            want = evict(c, table, [n], scores, keep, recent, table)
            assert np.array_equal(kept.cpu().numpy(), want[1]) and np.array_equal(moved.cpu().numpy(), want[2], equal_nan=True)
            same_cache(gpu, c)


def test_evict_scores_of_all_kinds():
    n, keep = 700, 200
    rng = np.random.default_rng(220)
    kinds = [np.zeros(n), np.full(n, -np.inf), np.full(n, np.nan), np.where(np.arange(n) % 3 == 0, np.nan, -np.inf),
             np.arange(n), -np.arange(n), np.where(np.arange(n) % 2, 0.0, -0.0), np.full(n, np.inf),
             rng.standard_normal(n) * 1e-40, rng.integers(0, 3, n), np.float32(1) + rng.integers(0, 4, n) * np.float32(2.0 ** -23),
             np.where(np.arange(n) > 650, 1.0, 0.0)]
    scores = np.stack(kinds).astype(np.float32)[:, None]
    B = len(kinds)
    table, P = make_table(rng, [n] * B, 64)
    for recent in (0, 50):
        gpu = upload(random_cache(rng, P, 1, 64, 64))
        _, kept, moved = sage.cache_evict(gpu, ints(table), ints([n] * B), dev(scores), keep, recent=recent)
        for b in range(B):
            assert kept[b, 0].tolist() == select(scores[b, 0], n, keep, recent), (b, recent)
            assert np.array_equal(moved[b, 0, :keep].cpu().numpy(), scores[b, 0][kept[b, 0].tolist()], equal_nan=True)


def test_evict_long_sequences():
    rng = np.random.default_rng(221)
    n, H, D, page, keep, recent = 70001, 2, 64, 128, 30011, 1000
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, H, D, page)
    scores = some_scores(rng, 1, H, n)
    gpu = upload(c)
    _, kept, _ = sage.cache_evict(gpu, ints(table), ints([n]), dev(scores), keep, recent=recent)
    want = evict(c, table, [n], scores, keep, recent, table)
    assert np.array_equal(kept.cpu().numpy(), want[1])
    same_cache(gpu, c)


def test_evict_scales_of_zero_and_nan():
    rng = np.random.default_rng(222)
    n, H, D, page, keep = 400, 2, 128, 64, 150
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, H, D, page)
    c.k_scale[table[0][0]], c.v_scale[table[0][1]] = 0.0, 0.0
    c.k_scale[table[0][2], 0, 1], c.v_scale[table[0][4], 1, 0] = np.nan, np.nan
    c.k_scale[table[0][5]] = 1e-42
    scores = some_scores(rng, 1, H, n)
    gpu = upload(c)
    sage.cache_evict(gpu, ints(table), ints([n]), dev(scores), keep, recent=10)
    evict(c, table, [n], scores, keep, 10, table)
    same_cache(gpu, c)


def test_evict_bad_pages_and_lengths_are_flagged():
    rng = np.random.default_rng(223)
    H, D, page, keep = 2, 64, 64, 70
    table, P = make_table(rng, [300, 128], page)
    c = random_cache(rng, P, H, D, page)
    scores = some_scores(rng, 2, H, 300)
    gpu = upload(c)
    broken = table.copy()
    broken[1, 1] = P + 7
    out, _ = make_table(rng, [70, 70], page, spare=P)
    out[0, :2], out[1, :2] = (P - 1, P), (P - 2, -1)   # the second page of each is outside the cache
    new, kept, _ = sage.cache_evict(gpu, ints(broken), ints([300, 128]), dev(scores), keep, out_table=ints(out))
    assert sage.device_error() == DEVICE_PAGE
    assert new.tolist() == [70, 70]
    assert kept[0, 0].tolist() == select(scores[0, 0], 300, keep, 0)
    for lengths in ([301, 5], [-3, 5], [2 ** 31 - 1, 5]):
        new, _, _ = sage.cache_evict(upload(c), ints(table), ints(lengths), dev(scores), keep)
        assert sage.device_error() == DEVICE_PAGE
        assert new.tolist() == [0 if lengths[0] < 0 else 70, 5]


def test_evict_refusals_and_empty_calls():
    rng = np.random.default_rng(224)
    table, P = make_table(rng, [40, 10], 64)
    c = random_cache(rng, P, 2, 64, 64)
    gpu = upload(c)
    scores = torch.zeros((2, 2, 40), device="cuda")
    good = dict(cache=gpu, page_table=ints(table), lengths=ints([40, 10]), scores=scores, keep=20, recent=3)
    for change, code in [
        (dict(keep=-1), -5), (dict(recent=-1), -5), (dict(recent=21), -5), (dict(scores=scores[:1]), -5), (dict(scores=scores.int()), -3),
        (dict(lengths=ints([40])), -5), (dict(lengths=ints([[40, 10]])), -5), (dict(lengths=torch.tensor([40, 10], device="cuda")), -3),
        (dict(out_table=ints(table)[:1]), -5), (dict(out_table=ints(table).long()), -3)]:
        with pytest.raises(SageError) as err:
            sage.cache_evict(**{**good, **change})
        assert err.value.code == code, change
    with pytest.raises(TypeError):
        sage.cache_evict(**{**good, "lengths": None})
    same_cache(gpu, c)
    new, kept, moved = sage.cache_evict(**{**good, "keep": 0, "recent": 0})
    assert new.tolist() == [0, 0] and kept.shape == (2, 2, 0) and (moved == 0).all()
    new, kept, moved = sage.cache_evict(gpu, ints(table)[:0], ints([]), scores[:0], 5)
    assert new.shape == (0,) and kept.shape == (0, 2, 5) and moved.shape == (0, 2, 40)
    new, kept, moved = sage.cache_evict(**{**good, "keep": 1000})     # nothing to cut
    assert new.tolist() == [40, 10] and kept.shape == (2, 2, 40) and kept[1, 0].tolist() == list(range(10)) + [-1] * 30


def test_evicted_sequences_go_on():
    """A run of the operators as a program makes it: attention, weights, eviction, new tokens, attention again."""
    rng = np.random.default_rng(225)
    B, H, Hkv, D, page, keep, recent = 2, 4, 2, 128, 64, 160, 16
    lengths = [300, 190]
    table, P = make_table(rng, [n + 40 for n in lengths], page)
    c = random_cache(rng, P, Hkv, D, page)
    gpu = upload(c)
    tab, lens = ints(table), ints(lengths)
    scores = torch.zeros((B, Hkv, 400), device="cuda")
    for step in range(3):
        q = bf16(rng, B, 1, H, D)
        _, lse = sage.cache_attention(q, gpu, tab, lens, is_causal=True, return_lse=True)
        sage.cache_add_weights(scores, q, gpu, tab, lens, lse, is_causal=True)
    lens, kept, scores = sage.cache_evict(gpu, tab, lens, scores, keep, recent=recent)
    before = scores.clone()
    evict_lengths = lens.tolist()
    assert evict_lengths == [keep, keep]
    # the oracle's cache goes the same way, by the kernel's choice
    old = [x.copy() for x in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    src = oc.Cache.__new__(oc.Cache)
    src.page_size, src.H, src.D = page, Hkv, D
    src.k_codes, src.v_codes, src.k_scale, src.v_scale = old
    k, v = bf16(rng, B, 1, Hkv, D), bf16(rng, B, 1, Hkv, D)
    sage.cache_append(gpu, k, v, tab, lens)
    lens += 1
    q = bf16(rng, B, 1, H, D)
    out, lse = sage.cache_attention(q, gpu, tab, lens, is_causal=True, return_lse=True)
    sage.cache_add_weights(scores, q, gpu, tab, lens, lse, is_causal=True)
    # read back, the sequences are the kept tokens (within half a step of their block's scale) and the new one
    kk, vv = sage.cache_read(gpu, tab, torch.zeros_like(lens), keep + 1, counts=lens)
    for b in range(B):
        ks, vs = src.tokens(table[b], 0, lengths[b])
        for h in range(Hkv):
            ids = kept[b, h].cpu().numpy()
            for got, was, scale in ((kk, ks, src.k_scale), (vv, vs, src.v_scale)):
                diff = np.abs(f32(got[b, :keep, h]) - was[ids, h])
                assert diff.max() <= scale.max() * 0.51 + 2.0 ** -8 * np.abs(was).max()
        assert np.abs(f32(kk[b, keep]) - f32(k[b, 0])).max() <= 0.1
    o, l, a = oc.attention_rows(f32(q[0, 0]), f32(kk[0, :, 0]).astype(np.float64), f32(vv[0, :, 0]).astype(np.float64),
                                [keep + 1] * H, 1 / math.sqrt(D))
    # tokens read back are rounded to bf16: 2^-8 of a logit's |q||k|, which is below 50 here with random signs
    assert np.abs(f32(lse[0, :2, 0]) - l[:2]).max() <= 0.05
    grown = (scores - before).sum(-1)
    assert ((grown - H // Hkv).abs() <= 0.01).all()


def test_scores_graph_replay():
    rng = np.random.default_rng(226)
    B, H, Hkv, D, page, keep = 2, 4, 2, 64, 32, 90
    table, P = make_table(rng, [400, 400], page)
    c = random_cache(rng, P, Hkv, D, page)
    gpu = upload(c)
    tab, lens = ints(table), ints([100, 200])
    q = bf16(rng, B, 1, H, D)
    start = torch.from_numpy(some_scores(rng, B, Hkv, 400)).cuda()
    scores = start.clone()
    lse = torch.full((B, H, 1), 4.0, device="cuda")

    def step():
        sage.cache_add_weights(scores, q, gpu, tab, lens, lse, is_causal=True)
        return sage.cache_evict(gpu, tab, lens, scores, keep, recent=7)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            new, kept, moved = step()
    for lengths in ([100, 200], [390, 5], [0, 91]):
        for x, y in zip((gpu.k_codes, gpu.v_codes, gpu.k_scale, gpu.v_scale), (c.k_codes, c.v_codes, c.k_scale, c.v_scale)):
            x.copy_(dev(y))
        lens.copy_(ints(lengths))
        scores.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        x = scores.cpu().numpy()
        cc = oc.Cache.__new__(oc.Cache)
        cc.page_size, cc.H, cc.D = page, Hkv, D
        cc.k_codes, cc.v_codes, cc.k_scale, cc.v_scale = (t.copy() for t in (c.k_codes, c.v_codes, c.k_scale, c.v_scale))
        want = evict(cc, table, lengths, x, keep, 7, table)
        assert np.array_equal(new.cpu().numpy(), want[0]) and np.array_equal(kept.cpu().numpy(), want[1])
        assert np.array_equal(moved.cpu().numpy(), want[2])
        same_cache(gpu, cc)


@pytest.mark.parametrize("T", [1, 50])
def test_weights_refuse_rows_that_overlap(T):
    rng = np.random.default_rng(227)
    table, P = make_table(rng, [100, 90], 64)
    gpu = upload(random_cache(rng, P, 2, 64, 64))
    q, lse = bf16(rng, 2, T, 4, 64), torch.zeros((2, 4, T), device="cuda")
    row = torch.zeros((1, 1, 100), device="cuda")
    args = (ints(table), ints([100, 90]), lse)
    for scores in (row.expand(2, 2, 100), torch.zeros((2, 1, 100), device="cuda").expand(2, 2, 100),
                   torch.zeros(500, device="cuda").as_strided((2, 2, 100), (150, 100, 1))):
        with pytest.raises(SageError) as e:
            sage.cache_add_weights(scores, q, gpu, *args)
        assert e.value.code == -6 and (scores == 0).all()
    scores = torch.zeros((2, 2, 100), device="cuda")
    for x in (q[:1].expand(2, T, 4, 64), q[:, :, :1].expand(2, T, 4, 64)):
        with pytest.raises(SageError) as e:
            sage.cache_add_weights(scores, x, gpu, *args)
        assert e.value.code == -6
    # rows apart in the other order
    turned = torch.zeros((2, 2, 100), device="cuda").transpose(0, 1)
    sage.cache_add_weights(turned, q, gpu, *args)
    sage.cache_add_weights(scores, q, gpu, *args)
    assert torch.equal(turned, scores) and (scores > 0).any()


@pytest.mark.parametrize("T", [1, 40])
def test_scores_graphs_replayed_at_once(T):
    """Two graphs of weights and eviction on caches of their own replay on two streams."""
    rng = np.random.default_rng(228)
    B, H, Hkv, D, page, keep = 3, 8, 2, 128, 64, 700
    runs = []
    for lengths in ([2000, 900, 1500], [800, 3000, 10]):
        table, P = make_table(rng, [n + page for n in lengths], page)
        c = random_cache(rng, P, Hkv, D, page)
        q = bf16(rng, B, T, H, D)
        runs.append((c, upload(c), ints(table), ints(lengths), q, torch.full((B, H, T), 5.0, device="cuda"),
                     torch.zeros((B, Hkv, 3000), device="cuda")))

    def step(r):
        sage.cache_add_weights(r[6], r[4], r[1], r[2], r[3], r[5])
        return sage.cache_evict(r[1], r[2], r[3], r[6], keep, recent=100)

    def restore(r):
        for x, y in zip((r[1].k_codes, r[1].v_codes, r[1].k_scale, r[1].v_scale),
                        (r[0].k_codes, r[0].v_codes, r[0].k_scale, r[0].v_scale)):
            x.copy_(dev(y))
        r[6].zero_()

    want = []
    for r in runs:
        res = step(r)
        want.append([x.clone() for x in res] + [r[6].clone(), r[1].k_codes.clone(), r[1].v_codes.clone()])
        restore(r)
    streams, graphs, got = [torch.cuda.Stream() for _ in runs], [], []
    torch.cuda.synchronize()
    for s, r in zip(streams, runs):
        with torch.cuda.stream(s):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got.append(step(r))
            graphs.append(g)
    for _ in range(4):
        for r in runs:
            restore(r)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for r, res, w in zip(runs, got, want):
            for x, y in zip(list(res) + [r[6], r[1].k_codes, r[1].v_codes], w):
                assert torch.equal(x, y)


def test_a_serving_run():
    """The operators together: packed prompts are turned and attended, go into the cache, are cut back by their
    weights, and tokens are generated behind them at their own positions."""
    from test_cache_gpu import close as close_cached
    from test_prompt_gpu import close as close_prompt, ends, formula

    rng = np.random.default_rng(229)
    rows, H, Hkv, D, page, keep, recent, new = [70, 1, 300, 0, 129], 8, 2, 128, 64, 96, 16, 3
    B, N, T = len(rows), sum(rows), max(rows)
    table, P = make_table(rng, [n + new for n in rows], page)
    gpu = sage.alloc_cache(P, Hkv, "cuda", D, page)
    tab, lens, off = ints(table), ints(rows), ints(ends(rows))
    freqs = sage.rotary_table(D, base=500000.0, scaling="yarn", factor=4.0, original_length=1024, device="cuda")
    q, k, v = bf16(rng, N + 5, H, D), bf16(rng, N + 5, Hkv, D), bf16(rng, N + 5, Hkv, D)
    pos = torch.cat([torch.arange(n) for n in rows + [5]]).to(torch.int32).cuda()
    q, k = sage.rotary(q, k, pos, freqs)
    sm = 1 / math.sqrt(D) / freqs.magnitude ** 2
    out, lse = sage.prompt_attention(q, k, v, off, sm_scale=sm, return_lse=True)
    close_prompt(out[:N], lse[:, :N], formula(q[:N], k[:N], v[:N], rows, rows, True, sm))
    assert (out[N:] == 0).all()

    # into the cache, and what the prompts' rows gave each token
    def padded(x):
        y = torch.zeros((B, T) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        for b in range(B):
            y[b, :rows[b]] = x[ends(rows)[b]:ends(rows)[b + 1]]
        return y

    sage.cache_append(gpu, padded(k), padded(v), tab, torch.zeros_like(lens), counts=lens)
    qp = padded(q)
    _, lse = sage.cache_attention(qp, gpu, tab, lens, q_lengths=lens, is_causal=True, sm_scale=sm, return_lse=True)
    scores = torch.zeros((B, Hkv, T + new), device="cuda")
    sage.cache_add_weights(scores, qp, gpu, tab, lens, lse, q_lengths=lens, is_causal=True, sm_scale=sm)
    total = torch.tensor(rows, device="cuda", dtype=torch.float64)[:, None] * (H // Hkv)
    assert ((scores.double().sum(-1) - total).abs() <= total * 2.0 ** -11).all()
    lens, kept, scores = sage.cache_evict(gpu, tab, lens, scores, keep, recent=recent)
    assert lens.tolist() == [min(n, keep) for n in rows]
    assert kept[2, :, keep - recent:].tolist() == [list(range(rows[2] - recent, rows[2]))] * Hkv

    # new tokens, whose positions go on where the prompts ended
    for t in range(new):
        q, k, v = bf16(rng, B, 1, H, D), bf16(rng, B, 1, Hkv, D), bf16(rng, B, 1, Hkv, D)
        q, k = sage.rotary(q, k, ints([[n + t] for n in rows]), freqs)
        sage.cache_append(gpu, k, v, tab, lens)
        lens = lens + 1
        out, lse = sage.cache_attention(q, gpu, tab, lens, is_causal=True, sm_scale=sm, return_lse=True)
        c = oc.Cache.__new__(oc.Cache)
        c.page_size, c.H, c.D = page, Hkv, D
        c.k_codes, c.v_codes = gpu.k_codes.cpu().numpy(), gpu.v_codes.cpu().numpy()
        c.k_scale, c.v_scale = gpu.k_scale.cpu().numpy(), gpu.v_scale.cpu().numpy()
        close_cached(out, lse, *oc.attention(c, f32(q), table, lens.tolist(), [1] * B, True, sm))
        before = scores.clone()
        sage.cache_add_weights(scores, q, gpu, tab, lens, lse, is_causal=True, sm_scale=sm)
        total, bound = weights(c, f32(q), table, lens.tolist(), [1] * B, f32(lse), True, sm, T + new)
        x = (scores.double() - before.double()).cpu().numpy()
        assert (np.abs(x - total) <= bound + f32(scores).astype(np.float64) * 2.0 ** -24 + 1e-30).all()


def test_evict_again_with_other_tensors():
    """Calls of one signature, whose checks the first one made, take each call's own tensors and sizes."""
    rng = np.random.default_rng(230)
    B, Hkv, D, page, n = 2, 2, 64, 32, 200
    for keep, recent in ((50, 5), (50, 6), (51, 5)):
        for place in ("in place", "other pages"):
            for seed in range(3):
                table, P = make_table(rng, [n, n], page)
                P += 20
                c = random_cache(rng, P, Hkv, D, page)
                gpu = upload(c)
                to = table if place == "in place" else (np.arange(2 * 7).reshape(2, 7) + P - 14).astype(np.int32)
                lengths = [int(x) for x in rng.integers(0, n + 1, B)]
                scores = some_scores(rng, B, Hkv, n)
                got = sage.cache_evict(gpu, ints(table), ints(lengths), dev(scores), keep, recent=recent,
                                       out_table=None if place == "in place" else ints(to))
                want = evict(c, table, lengths, scores, keep, recent, to)
                for x, y in zip(got, want):
                    assert np.array_equal(x.cpu().numpy(), y)
                same_cache(gpu, c)


@pytest.mark.parametrize("T", [1, 40])
def test_scores_and_queries_past_32_bits(T):
    rng = np.random.default_rng(231)
    B, H, Hkv, D, page, n = 3, 4, 2, 64, 64, 150
    table, P = make_table(rng, [n] * B, page)
    c = random_cache(rng, P, Hkv, D, page)
    gpu, tab, lens = upload(c), ints(table), ints([n, 100, 77])
    q, lse = bf16(rng, B, T, H, D), torch.full((B, H, T), 3.0, device="cuda")
    apart = 1 << 30                                             # of sequences
    room = torch.empty(2 * apart + (1 << 16), dtype=torch.float32, device="cuda")
    scores = room.as_strided((B, Hkv, n), (apart, 1 << 12, 1))
    scores.zero_()
    wide = room.view(torch.bfloat16)[1 << 15:].as_strided((B, T, H, D), (apart, H * D, D, 1))
    wide.copy_(q)
    dense = torch.zeros((B, Hkv, n), device="cuda")
    sage.cache_add_weights(dense, q, gpu, tab, lens, lse)
    sage.cache_add_weights(scores, wide, gpu, tab, lens, lse)
    assert torch.equal(scores, dense) and (dense > 0).any()
    got = sage.cache_evict(gpu, tab, lens, scores, 60, recent=9)
    for x, y in zip(got, evict(c, table, [n, 100, 77], dense.cpu().numpy(), 60, 9, table)):
        assert np.array_equal(x.cpu().numpy(), y)
    same_cache(gpu, c)
