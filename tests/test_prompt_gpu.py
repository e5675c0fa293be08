"""Attention over packed prompts on the GPU against the formula in float64.

Outputs are held to a bound that is derived, not fitted. With A = sum_j p_j |v_j| / sum_j p_j (in float64),
an output differs from the formula by at most
  2^-8 |o|    its rounding to bf16 (half a step), where |o| itself may be off by the rest,
  2^-8 A      the rounding of the weights to bf16 (half a step),
  2^-12 A     logits: D products of bf16, exact in fp32, whose sum errs by at most D 2^-23 sum |q k| sm_scale
              < 128 2^-23 12 < 2^-12.4 as an absolute error of the logit here, once in p and once in the sum of p,
              together below 2^-11 A; and exponentials (2^-22) and the fp32 sums of p (at most m 2^-24 < 2^-12),
together below 2^-8 |o| + (2^-8 + 2^-10) A + a little of the product of both, for which 2^-8 |o| becomes
2^-8 (|o| + A / 64). The log-sum-exp errs by the logits' 2^-12.4, the sum's 2^-12 and roundings of numbers below
32 (2^-19 each): 2^-11 in all.
"""

import math

import numpy as np
import pytest
import torch

import quantized_attention_fp64_gb300 as sage
from quantized_attention_fp64_gb300.api import SageError

pytestmark = pytest.mark.gpu

DEVICE_OFFSETS = -17


@pytest.fixture(autouse=True)
def _library(sage_lib):
    torch.cuda.synchronize()
    sage.device_error()
    yield
    torch.cuda.synchronize()
    assert sage.device_error() == 0  # a test that expects one has read and cleared it


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def ends(sizes):
    return [0] + np.cumsum(sizes).tolist()


def formula(q, k, v, rows, keys, causal, sm):
    """(o, lse, A) in float64 of sequences with these rows and keys; rows of no sequence are 0 and -inf."""
    N, H, D = q.shape
    G = H // k.shape[1]
    o = torch.zeros((N, H, D), dtype=torch.float64, device="cuda")
    a = torch.zeros_like(o)
    lse = torch.full((H, N), -math.inf, dtype=torch.float64, device="cuda")
    qd, kd, vd = q.double(), k.double(), v.double()
    at = kv = 0
    for n, m in zip(rows, keys):
        if n and m:
            x = qd[at:at + n].permute(1, 0, 2)
            kk, vv = (t[kv:kv + m].permute(1, 0, 2).repeat_interleave(G, 0) for t in (kd, vd))
            z = x @ kk.transpose(1, 2) * sm
            if causal:
                hidden = torch.arange(m, device="cuda") > torch.arange(n, device="cuda")[:, None] + (m - n)
                z = torch.where(hidden, -math.inf, z)
            top = z.amax(-1, keepdim=True)
            p = torch.where(torch.isinf(top) & (top < 0), 0.0, torch.exp(z - top))
            l = p.sum(-1, keepdim=True)
            # 0 weights times what a row does not see count as 0
            none = l == 0
            pn = p / torch.where(none, 1.0, l)
            o[at:at + n] = (pn @ vv).permute(1, 0, 2)
            a[at:at + n] = (pn @ vv.abs()).permute(1, 0, 2)
            lse[:, at:at + n] = torch.where(none, -math.inf, top + torch.log(l))[..., 0]
        at, kv = at + n, kv + m
    return o, lse, a


def close(out, lse, ref):
    o, l, a = ref
    err = (out.double() - o).abs()
    bound = (o.abs() + a / 64) * 2.0 ** -8 + a * (2.0 ** -8 + 2.0 ** -10) + 1e-30
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert not torch.isnan(out).any() and worst <= 1.0, worst
    if lse is not None:
        there = torch.isfinite(l)
        assert torch.equal(there, torch.isfinite(lse)) and (lse[~there] == -math.inf).all()
        assert not there.any() or (lse.double() - l)[there].abs().max() <= 2.0 ** -11


# rows of each sequence, keys of each (None: the same), query heads, key/value heads, head dimension, causal
CASES = [
    ([1], None, 1, 1, 128, True),
    ([1, 1, 1], None, 4, 2, 64, True),
    ([2, 127, 128, 129], None, 2, 1, 128, True),
    ([255, 256, 257], None, 2, 2, 64, True),
    ([0, 5, 0, 0, 300, 0], None, 4, 4, 128, True),
    ([513, 1, 700], None, 7, 1, 128, True),
    ([1000, 17], None, 5, 5, 64, False),
    ([128, 384, 33], None, 8, 2, 128, False),
    ([1, 7, 130], [400, 7, 131], 4, 1, 128, True),     # a prompt that goes on: more keys than rows
    ([300, 40, 3], [100, 0, 1], 2, 1, 128, True),      # rows that see no key
    ([300, 260], [0, 5], 2, 2, 64, True),
    ([9, 0, 200], [1000, 50, 0], 6, 2, 64, False),
    ([1] * 70 + [129] * 5, None, 3, 1, 128, True),     # more sequences than a warp has lanes
    ([2500], None, 2, 1, 128, True),
    ([1900, 2100], None, 1, 1, 64, True),
    ([40, 4000], [4100, 4001], 2, 1, 128, False),
]


def inputs(seed, rows, keys, H, Hkv, D, spare=0):
    g = gen(seed)
    q, k, v = bf16(g, sum(rows) + spare, H, D), bf16(g, sum(keys) + spare, Hkv, D), bf16(g, sum(keys) + spare, Hkv, D)
    return q, k, v


@pytest.mark.parametrize("case", range(len(CASES)))
def test_prompt_attention(case):
    rows, keys, H, Hkv, D, causal = CASES[case]
    same, keys = keys is None, keys or rows
    q, k, v = inputs(case, rows, keys, H, Hkv, D)
    out, lse = sage.prompt_attention(q, k, v, ints(ends(rows)), kv_offsets=None if same else ints(ends(keys)),
                                     is_causal=causal, return_lse=True)
    close(out, lse, formula(q, k, v, rows, keys, causal, 1 / math.sqrt(D)))
    again = sage.prompt_attention(q, k, v, ints(ends(rows)), kv_offsets=None if same else ints(ends(keys)), is_causal=causal)
    assert torch.equal(again, out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_layouts_strides_and_scale(D, causal):
    rows, H, Hkv = [140, 3, 260], 4, 2
    N = sum(rows)
    g = gen(50)
    fused = bf16(g, N, H + 2 * Hkv, D + 8)          # queries, keys and values of one projection, rows wider than a head
    q, k, v = fused[:, :H, :D], fused[:, H:H + Hkv, :D], fused[:, H + Hkv:, :D]
    ref = formula(q, k, v, rows, rows, causal, 0.2)
    out, lse = sage.prompt_attention(q, k, v, ints(ends(rows)), is_causal=causal, sm_scale=0.2, return_lse=True)
    close(out, lse, ref)
    hnd = [t.transpose(0, 1).contiguous() for t in (q, k, v)]
    out, lse = sage.prompt_attention(*hnd, ints(ends(rows)), is_causal=causal, sm_scale=0.2, return_lse=True, tensor_layout="HND")
    close(out.transpose(0, 1), lse, ref)
    wide = torch.full((N, H, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    sage.prompt_attention(q, k, v, ints(ends(rows)), is_causal=causal, sm_scale=0.2, out=wide[:, :, D:])
    close(wide[:, :, D:], None, ref)
    assert (wide[:, :, :D] == 7.0).all()


def test_one_key_head_shared_without_copies():
    rows = [200, 100]
    g = gen(51)
    q, k, v = bf16(g, 300, 4, 128), bf16(g, 300, 1, 128), bf16(g, 300, 1, 128)
    out = sage.prompt_attention(q, k, v, ints(ends(rows)))
    close(out, None, formula(q, k, v, rows, rows, True, 1 / math.sqrt(128)))


@pytest.mark.parametrize("D", [64, 128])
def test_rest_rows(D):
    rows, spare = [70, 0, 200], 45
    q, k, v = inputs(60, rows, rows, 3, 1, D, spare)
    off = ints([20 + x for x in ends(rows)])        # rows in front of the first sequence, and behind the last
    for t in (q, k, v):
        t[:20] = math.nan
        t[290:] = math.inf
    ref = formula(q[20:290], k[20:290], v[20:290], rows, rows, True, 1 / math.sqrt(D))
    out, lse = sage.prompt_attention(q, k, v, off, return_lse=True)
    close(out[20:290], lse[:, 20:290], ref)
    rest = torch.cat([torch.arange(20), torch.arange(290, 270 + spare)]).cuda()
    assert (out[rest] == 0).all() and (lse[:, rest] == -math.inf).all()
    given = torch.full_like(q, 3.0)
    out, lse = sage.prompt_attention(q, k, v, off, return_lse=True, out=given)
    assert out is given and (given[rest] == 3.0).all() and (lse[:, rest] == -math.inf).all()
    close(given[20:290], lse[:, 20:290], ref)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_what_a_row_does_not_see_does_not_touch_it(what, D):
    rows, H, Hkv = [200, 129, 513], 2, 1
    q, k, v = inputs(70, rows, rows, H, Hkv, D)
    ref = formula(q, k, v, rows, rows, True, 1 / math.sqrt(D))
    # a later token's key and value, in the same key tile as earlier rows and in later tiles
    k2, v2 = k.clone(), v.clone()
    spots = [150, 199, 200 + 128, 329 + 130, 329 + 512]
    for s in spots:
        k2[s], v2[s, 0, 5:9] = what, what
    out, lse = sage.prompt_attention(q, k2, v2, ints(ends(rows)), return_lse=True)
    at = 0
    for n, first in zip(rows, (150, 328, 459)):
        close(out[at:first], lse[:, at:first], [r[at:first] if r.dim() == 3 and r.shape[0] == sum(rows) else r[:, at:first] for r in ref])
        at += n
    if math.isnan(what):
        assert torch.isnan(lse[:, 150:200]).all() and torch.isnan(lse[:, 328]).all() and torch.isnan(lse[:, 459:]).all()
        assert torch.isnan(out[150:200]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,past", [([300, 77], [0, 0]), ([60, 400], [200, 61])])
def test_infinite_values_reach_the_rows_that_see_them(rows, past, D):
    keys = [n + p for n, p in zip(rows, past)]
    H, Hkv = 4, 2
    q, k, v = inputs(71, rows, keys, H, Hkv, D)
    ref = formula(q, k, v, rows, keys, True, 1 / math.sqrt(D))
    v2 = v.clone()
    marks = [(0, 3, 0, math.inf), (0, keys[0] - 30, 1, -math.inf), (0, keys[0] - 1, D - 1, math.nan), (1, keys[1] // 2, 33, math.inf),
             (1, keys[1] - 20, 33, -math.inf), (1, keys[1] - 2, 7, math.inf)]
    start = ends(keys)
    for b, j, c, x in marks:
        v2[start[b] + j, :, c] = x
    out = sage.prompt_attention(q, k, v2, ints(ends(rows)), kv_offsets=ints(ends(keys)))
    want = ref[0].clone()
    at = 0
    for b, n in enumerate(rows):
        for t in range(n):
            for bb, j, c, x in marks:
                if bb == b and j <= past[b] + t:
                    want[at + t, :, c] += x
        at += n
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[odd & ~torch.isnan(want)].double(), want[odd & ~torch.isnan(want)])
    err = (out.double() - ref[0]).abs()
    bound = (ref[0].abs() + ref[2] / 64) * 2.0 ** -8 + ref[2] * (2.0 ** -8 + 2.0 ** -10)
    # the marked value itself is no longer part of the other channels' sums, and theirs are as before
    assert (err[~odd] <= bound[~odd]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("units", ["few", "many"])
def test_infinite_values_of_little_weight(units, causal, D):
    """An infinity that a row sees is in its sum however small the weight, in whichever key tile: the weights here are
    exp(-120) and below, which fp32 does not hold, of keys before and behind those that raise the maximum."""
    rows, past, H, Hkv = [300, 77, 140], [0, 200, 390], 4, 2
    keys = [n + p for n, p in zip(rows, past)]
    q, k, v = inputs(75, rows, keys, H, Hkv, D)
    q[..., 0] = 16.0
    k[..., 0] = 0.0
    start = ends(keys)
    marks = [(0, 3, 0, math.inf), (0, 140, 9, -math.inf), (0, 255, D - 1, math.inf), (0, 290, 33, math.nan), (0, 5, 34, math.inf), (0, 270, 34, -math.inf),
             (1, 2, 1, math.nan), (1, 150, 2, -math.inf), (1, 270, 2, -math.inf), (2, 0, 40, math.inf), (2, 200, 40, -math.inf), (2, 529, 41, math.inf)]
    for b, j, c, x in marks:
        k[start[b] + j, :, 0] = -10.0 * math.sqrt(D)
        v[start[b] + j, :, c] = 0.0
    ref = formula(q, k, v, rows, keys, causal, 1 / math.sqrt(D))
    want = ref[0].clone()
    for b, j, c, x in marks:
        v[start[b] + j, :, c] = x
        at = ends(rows)[b]
        first = max(j - past[b], 0) if causal else 0
        want[at + first:at + rows[b], :, c] += x
    # rows that see none but such keys give them the whole weight
    q = q if units == "few" else q.repeat_interleave(76, 1)
    out = sage.prompt_attention(q, k, v, ints(ends(rows)), kv_offsets=ints(ends(keys)), is_causal=causal)
    out = out if units == "few" else out[:, ::76]
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out[odd & ~torch.isnan(want)].double(), want[odd & ~torch.isnan(want)])
    err = (out.double() - ref[0]).abs()
    bound = (ref[0].abs() + ref[2] / 64) * 2.0 ** -8 + ref[2] * (2.0 ** -8 + 2.0 ** -10)
    assert (err[~odd] <= bound[~odd]).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("share", [0.002, 0.3, 1.0])
def test_many_values_that_are_not_finite(share, causal, D):
    """Any part of the values, in all channels, tiles and sequences: each output is what those that its row sees make of it."""
    rows, past, H, Hkv = [300, 77, 513], [0, 200, 3], 4, 2
    keys = [n + p for n, p in zip(rows, past)]
    q, k, v = inputs(76, rows, keys, H, Hkv, D, spare=30)
    n, m = sum(rows), sum(keys)
    g = gen(77)
    odd = torch.rand(v.shape, generator=g, device="cuda") < share
    kind = torch.tensor([math.inf, -math.inf, math.nan], device="cuda").to(torch.bfloat16)
    kind = kind[torch.randint(0, 3 if share < 1 else 2, v.shape, generator=g, device="cuda")]
    ref = formula(q[:n], k[:m], torch.where(odd, 0.0, v)[:m], rows, keys, causal, 1 / math.sqrt(D))
    v = torch.where(odd, kind, v)
    out = sage.prompt_attention(q, k, v, ints(ends(rows)), kv_offsets=ints(ends(keys)), is_causal=causal)
    x = v.double().repeat_interleave(H // Hkv, 1)
    ups, downs = ((x == s) | x.isnan() for s in (math.inf, -math.inf))
    for b in range(3):
        o, r, a = (t[ends(rows)[b]:ends(rows)[b + 1]] for t in (out, ref[0], ref[2]))
        up, down = (t[ends(keys)[b]:ends(keys)[b + 1]].to(torch.int32).cumsum(0) > 0 for t in (ups, downs))
        at = torch.arange(rows[b], device="cuda") + past[b] if causal else torch.full((rows[b],), keys[b] - 1, device="cuda")
        up, down = up[at], down[at]
        assert torch.equal(torch.isnan(o), up & down)
        assert torch.equal(o == math.inf, up & ~down) and torch.equal(o == -math.inf, down & ~up)
        fine = ~(up | down)
        bound = (r.abs() + a / 64) * 2.0 ** -8 + a * (2.0 ** -8 + 2.0 ** -10) + 1e-30
        assert ((o.double() - r).abs() <= bound)[fine].all()
    assert (out[n:] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_growing_and_falling_logits(D):
    # the running maximum has to follow, early and late, by little and by much
    n = 700
    g = gen(72)
    q, k, v = (bf16(g, n, 2, D) for _ in range(3))
    for shape in (torch.linspace(-3, 3, n), torch.linspace(3, -3, n), torch.sin(torch.arange(n) / 9.0) * 3):
        kk = (k.float() * 0.1 + q.mean(0) + shape.cuda()[:, None, None]).to(torch.bfloat16)
        qq = (q.float() * 0.1 + 1.0).to(torch.bfloat16)
        sm = 1 / math.sqrt(D) / 2
        ref = formula(qq, kk, v, [n], [n], True, sm)
        assert (qq.float().abs().amax() * kk.float().abs().amax() * D * sm) < 120
        out, lse = sage.prompt_attention(qq, kk, v, ints([0, n]), sm_scale=sm, return_lse=True)
        # sum |q k| sm_scale is up to 60 here, five times the bound's: logits err by up to 2^-10
        o, l, a = ref
        assert ((out.double() - o).abs() <= (o.abs() + a / 64) * 2.0 ** -8 + a * (2.0 ** -8 + 2.0 ** -8)).all()
        assert ((lse.double() - l).abs() <= 2.0 ** -9).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("high", [5.375, 2.5])
def test_large_values_whose_sum_is_in_range(high, causal, D):
    """Values of 2^122: a key whose weight is 216 (or 12) times that of those before it leaves the sums finite."""
    n, H = 400, 2
    g = gen(74)
    q = torch.ones((n, H, D), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[[150, 290, 399]] = high
    v = (torch.rand((n, 1, D), generator=g, device="cuda") * 2.0 ** 122).to(torch.bfloat16)
    ref = formula(q, k, v, [n], [n], causal, 1 / D)
    assert torch.isfinite(ref[0]).all()
    out, lse = sage.prompt_attention(q, k, v, ints([0, n]), is_causal=causal, sm_scale=1 / D, return_lse=True)
    close(out, lse, ref)
    out, lse, r = repeated(q, k, v, ints([0, n]), is_causal=causal, sm_scale=1 / D)
    close(out[:, ::r], lse[::r], ref)


def test_peaked_rows_take_one_value():
    n, D = 300, 128
    g = gen(73)
    v = bf16(g, n, 1, D)
    k = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    k[torch.arange(n), 0, torch.arange(n) % D] = 16.0
    q = torch.zeros((n, 1, D), dtype=torch.bfloat16, device="cuda")
    pick = torch.arange(n) // 3
    q[torch.arange(n), 0, pick % D] = 64.0
    out = sage.prompt_attention(q, k, v, ints([0, n]), is_causal=True)
    only = pick < D  # keys pick and pick + D, ... have the same logit; rows that see the first alone copy its value
    rows = torch.nonzero(only & (torch.arange(n) < D))[:, 0]
    assert torch.equal(out[rows], v[pick[rows]])


@pytest.mark.parametrize("off,kv", [
    ([0, 50, 40, 100], None), ([-1, 50, 100], None), ([0, 50, 101], None), ([0, 2 ** 31 - 1, 100], None),
    ([0, 50, 100], [0, 60, 50]), ([0, 50, 100], [0, 50, 90]), ([0, 50, 100], [-5, 50, 80])])
def test_bad_offsets_are_flagged(off, kv):
    g = gen(80)
    q, k, v = bf16(g, 100, 2, 64), bf16(g, 80 if kv else 100, 1, 64), bf16(g, 80 if kv else 100, 1, 64)
    out, lse = sage.prompt_attention(q, k, v, ints(off), kv_offsets=ints(kv) if kv else None, return_lse=True)
    torch.cuda.synchronize()
    assert sage.device_error() == DEVICE_OFFSETS
    assert (out == 0).all() and (lse == -math.inf).all()


def test_empty_calls():
    g = gen(81)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    assert sage.prompt_attention(e, e, e, ints([0])).shape == (0, 2, 64)
    assert sage.prompt_attention(e, e, e, ints([0, 0, 0])).shape == (0, 2, 64)
    q = bf16(g, 5, 2, 64)
    out, lse = sage.prompt_attention(q, e, e, ints([0, 5]), kv_offsets=ints([0, 0]), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = sage.prompt_attention(q, q, q, ints([0]), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_refusals():
    g = gen(82)
    q, k, v = bf16(g, 10, 4, 64), bf16(g, 10, 2, 64), bf16(g, 10, 2, 64)
    off = ints([0, 10])
    bad = [
        (dict(q=q.half()), -3), (dict(offsets=off.long()), -3), (dict(q=q[0]), -5), (dict(k=k[:9]), -5),
        (dict(q=q[:, :3]), -5), (dict(k=k[..., :32], v=v[..., :32]), -5), (dict(offsets=ints([[0, 10]])), -5),
        (dict(offsets=ints([])), -5), (dict(kv_offsets=ints([0, 5, 10])), -5), (dict(tensor_layout="BHND"), -6),
        (dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)), -6), (dict(sm_scale=0.0), -13),
        (dict(sm_scale=math.inf), -13), (dict(offsets=ints([0, 1, 10, 2])[::2]), -6),
        (dict(q=bf16(g, 10, 4, 32), k=bf16(g, 10, 2, 32), v=bf16(g, 10, 2, 32)), -4),
        (dict(q=bf16(g, 10, 4, 65)[..., 1:], k=k), -7), (dict(out=bf16(g, 10, 2, 64)), -5),
        (dict(workspace=torch.empty(10, dtype=torch.uint8, device="cuda")), -9),
    ]
    for change, code in bad:
        with pytest.raises(SageError) as err:
            sage.prompt_attention(**{**dict(q=q, k=k, v=v, offsets=off), **change})
        assert err.value.code == code, (change, err.value)
    with pytest.raises(ValueError):
        sage.prompt_attention(q.cpu(), k, v, off)
    with pytest.raises(ValueError):
        sage.prompt_attention(q, k, v, off.cpu())
    with pytest.raises(TypeError):
        sage.prompt_attention(q, k, None, off)


def test_graph_replay_with_other_offsets():
    N, H, Hkv, D = 600, 4, 2, 128
    q, k, v = inputs(90, [N], [N], H, Hkv, D)
    off = ints([0, 100, 350, 600])
    sage.prompt_attention(q, k, v, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out, lse = sage.prompt_attention(q, k, v, off, return_lse=True)
    for e in ([0, 100, 350, 600], [0, 0, 599, 600], [0, 256, 512, 520]):
        off.copy_(ints(e))
        graph.replay()
        torch.cuda.synchronize()
        rows = np.diff(e).tolist()
        close(out[:e[-1]], lse[:, :e[-1]], formula(q[:e[-1]], k, v, rows, rows, True, 1 / math.sqrt(D)))


def test_two_streams_at_once():
    streams = [torch.cuda.Stream() for _ in range(3)]
    rows = [[900, 30], [100] * 9, [1500]]
    data = [inputs(91 + i, r, r, 4, 1, 128) for i, r in enumerate(rows)]
    refs = [formula(*d, r, r, True, 1 / math.sqrt(128)) for d, r in zip(data, rows)]
    torch.cuda.synchronize()
    outs = [[] for _ in rows]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(sage.prompt_attention(*data[i], ints(ends(rows[i])), return_lse=True))
    torch.cuda.synchronize()
    for got, ref in zip(outs, refs):
        for out, lse in got:
            close(out, lse, ref)


# ------------------------------------------------ calls with a list of units --
# Calls of more units than there are SMs make a list of them first and look the values over. With every query head
# repeated until there are as many, they give the bits of the calls without.


def repeated(q, k, v, off, kv=None, **kw):
    """The same call with each query head `r` times, which has over 300 units; returns it and r."""
    r = -(-304 // q.shape[1])
    out, lse = sage.prompt_attention(q.repeat_interleave(r, 1), k, v, off, kv_offsets=kv, return_lse=True, **kw)
    return out, lse, r


def same_bits(a, b):
    return torch.equal(torch.nan_to_num(a, nan=7.25), torch.nan_to_num(b, nan=7.25)) and torch.equal(a.isnan(), b.isnan())


def check_repeated(q, k, v, off, kv=None, **kw):
    out, lse = sage.prompt_attention(q, k, v, off, kv_offsets=kv, return_lse=True, **kw)
    many, many_lse, r = repeated(q, k, v, off, kv, **kw)
    assert same_bits(many, out.repeat_interleave(r, 1)) and same_bits(many_lse, lse.repeat_interleave(r, 0))
    return out, lse


@pytest.mark.parametrize("case", range(len(CASES)))
def test_many_units(case):
    rows, keys, H, Hkv, D, causal = CASES[case]
    if sum(rows) > 2600:
        rows, keys = [r // 3 for r in rows], [k // 3 for k in keys or rows] if keys else None
    q, k, v = inputs(120 + case, rows, keys or rows, H, Hkv, D, spare=9)
    off = ints(ends(rows))
    out, lse = check_repeated(q, k, v, off, ints(ends(keys)) if keys else None, is_causal=causal)
    n, m = sum(rows), sum(keys or rows)
    close(out[:n], lse[:, :n], formula(q[:n], k[:m], v[:m], rows, keys or rows, causal, 1 / math.sqrt(D)))
    assert (out[n:] == 0).all() and (lse[:, n:] == -math.inf).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("at", [0, 63, 64, 130, 299, 300, 301, 360, 599, 600, 655, 698])
def test_many_units_with_values_that_are_not_finite(at, what, D):
    """One value anywhere: in what a row sees, behind it, in the next sequence's tile, behind the last sequence."""
    rows = [300, 0, 299, 56]
    q, k, v = inputs(140, rows, rows, 4, 2, D, spare=44)
    v[at, 1, 5] = what
    out, lse = check_repeated(q, k, v, ints(ends(rows)))
    bad = ~torch.isfinite(out)
    seen = torch.zeros(out.shape[0], dtype=torch.bool, device="cuda")
    for lo, hi in zip(ends(rows)[:-1], ends(rows)[1:]):
        if lo <= at < hi:
            seen[at:hi] = True
    assert torch.equal(bad[:, 2, 5], seen) and torch.equal(bad[:, 3, 5], seen)
    bad[:, 2:, 5] = False
    assert not bad.any() and not torch.isnan(lse).any()


@pytest.mark.parametrize("D", [64, 128])
def test_many_units_of_longer_keys_with_values_that_are_not_finite(D):
    rows, keys = [60, 400], [261, 461]
    q, k, v = inputs(141, rows, keys, 4, 2, D, spare=20)
    for at in (0, 200, 201, 230, 260, 262, 320, 700, 721):
        w = v.clone()
        w[at, 0, 3] = math.nan
        check_repeated(q[:460], k, w, ints(ends(rows)), ints(ends(keys)))


@pytest.mark.parametrize("off,kv", [
    ([0, 50, 40, 100], None), ([-1, 50, 100], None), ([0, 50, 101], None), ([0, 2 ** 31 - 1, 100], None),
    ([0, 50, 100], [0, 60, 50]), ([0, 50, 100], [0, 50, 90]), ([0, 50, 100], [-5, 50, 80])])
def test_many_units_bad_offsets_are_flagged(off, kv):
    g = gen(142)
    q, k, v = bf16(g, 100, 160, 64), bf16(g, 80 if kv else 100, 1, 64), bf16(g, 80 if kv else 100, 1, 64)
    out, lse = sage.prompt_attention(q, k, v, ints(off), kv_offsets=ints(kv) if kv else None, return_lse=True)
    torch.cuda.synchronize()
    assert sage.device_error() == DEVICE_OFFSETS
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("D", [64, 128])
def test_many_units_leave_rest_rows(D):
    rows = [70, 300]
    q, k, v = inputs(143, rows, rows, 160, 4, D, spare=60)
    off = ints([20, 90, 390])
    out = torch.full_like(q, 7.0)
    sage.prompt_attention(q, k, v, off, out=out)
    assert (out[:20] == 7).all() and (out[390:] == 7).all() and not (out[20:390] == 7).all(-1).any()
    fresh = sage.prompt_attention(q, k, v, off)
    assert (fresh[:20] == 0).all() and (fresh[390:] == 0).all() and torch.equal(fresh[20:390], out[20:390])


def test_units_around_the_number_of_sms():
    """Calls with a unit fewer than SMs, as many, and one more (two tiles of 128 rows for each head)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    q, k, v = inputs(144, [200], [200], sms + 1, 1, 64)
    off = ints([0, 200])
    outs = [sage.prompt_attention(q[:, :h], k, v, off) for h in (sms + 1, sms, sms - 1)]
    assert torch.equal(outs[0][:, :sms], outs[1]) and torch.equal(outs[0][:, :sms - 1], outs[2])
    close(outs[0], None, formula(q, k, v, [200], [200], True, 0.125))


def test_expanded_heads_and_rows_are_refused():
    g = gen(145)
    q, k = bf16(g, 10, 4, 64), bf16(g, 10, 1, 64)
    for change in (dict(k=k.expand(10, 4, 64)), dict(v=k.expand(10, 4, 64)), dict(q=q[:, :1].expand(10, 4, 64)),
                   dict(q=q[:1].expand(10, 4, 64))):
        with pytest.raises(SageError) as err:
            sage.prompt_attention(**{**dict(q=q, k=q, v=q, offsets=ints([0, 10])), **change})
        assert err.value.code == -6


def test_expanded_outputs_are_refused():
    g = gen(149)
    q, k = bf16(g, 10, 4, 64), bf16(g, 10, 1, 64)
    for out in (q[:1].expand(10, 4, 64), q[:, :1].expand(10, 4, 64)):
        with pytest.raises(SageError) as err:
            sage.prompt_attention(k.expand(10, 4, 64).contiguous(), k, k, ints([0, 10]), out=out)
        assert err.value.code == -6
    x = torch.stack([q, q])
    table, pos = sage.rotary_table(64, device="cuda"), torch.arange(10, dtype=torch.int32, device="cuda")
    wide = q[None].expand(2, 10, 4, 64)
    assert torch.equal(sage.rotary(wide, None, pos, table), sage.rotary(x, None, pos, table))  # read, they are fine
    before = q.clone()
    for args, out in (((x, None), wide), ((wide, None), wide), ((x, x[:, :, :1]), (x, wide[:, :, :1]))):
        with pytest.raises(SageError) as err:
            sage.rotary(*args, pos, table, out=out)
        assert err.value.code == -6
    with pytest.raises(SageError) as err:
        sage.rotary(x, x, pos, table, out=(x, x))
    assert err.value.code == -13 and torch.equal(q, before) and torch.equal(x[1], before)


def test_graphs_replayed_at_once():
    """Two captured graphs of calls with a list replay on two streams, each with its own workspace."""
    data = [inputs(146 + i, r, r, 16, 2, 128) for i, r in enumerate(([3000, 500], [100] * 20))]
    offs = [ints(ends(r)) for r in ([3000, 500], [100] * 20)]
    want = [sage.prompt_attention(*d, o, return_lse=True) for d, o in zip(data, offs)]
    streams, graphs, got = [torch.cuda.Stream() for _ in data], [], []
    torch.cuda.synchronize()
    for s, d, o in zip(streams, data, offs):
        with torch.cuda.stream(s):
            sage.prompt_attention(*d, o, return_lse=True)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got.append(sage.prompt_attention(*d, o, return_lse=True))
            graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(5):
        for out, lse in got:
            out.zero_()
            lse.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (out, lse), (o, l) in zip(got, want):
            assert torch.equal(out, o) and torch.equal(lse, l)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H", [2, 160])
def test_outputs_at_half_sectors(H, D):
    """Rows of out that begin 16 bytes into a sector give the same, and nothing beside them is written."""
    rows = [130, 7]
    q, k, v = inputs(150, rows, rows, H, 2, D, spare=3)
    off = ints(ends(rows))
    want = sage.prompt_attention(q, k, v, off)
    for at, width in ((8, D + 16), (0, D + 8), (16, D + 24)):
        wide = torch.full((140, H, width), 3.0, dtype=torch.bfloat16, device="cuda")
        sage.prompt_attention(q, k, v, off, out=wide[:, :, at:at + D])
        assert torch.equal(wide[:137, :, at:at + D], want[:137])
        wide[:137, :, at:at + D] = 3.0
        assert (wide == 3).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("H,Hkv", [(3, 1), (7, 1), (10, 2), (9, 3)])
def test_odd_heads_of_a_key_head(H, Hkv, causal, D):
    """Pairs of query tiles that cross from one row tile to the next, and tiles without a partner, in calls with few
    units and with many (whose heads come several times)."""
    rows, past = [1, 127, 128, 129, 300, 513, 40], [0, 3, 0, 260, 0, 0, 400]
    keys = [n + p for n, p in zip(rows, past)]
    q, k, v = inputs(160, rows, keys, H, Hkv, D)
    off, kv = ints(ends(rows)), ints(ends(keys))
    out, lse = sage.prompt_attention(q, k, v, off, kv_offsets=kv, return_lse=True, is_causal=causal)
    close(out, lse, formula(q, k, v, rows, keys, causal, 1 / math.sqrt(D)))
    many_k, many_v = (x.repeat(1, 31, 1) for x in (k, v))
    many, many_lse = sage.prompt_attention(q.repeat(1, 31, 1), many_k, many_v, off, kv_offsets=kv, return_lse=True, is_causal=causal)
    assert torch.equal(many, out.repeat(1, 31, 1)) and torch.equal(many_lse, lse.repeat(31, 1))
    one, one_lse = sage.prompt_attention(q[128:256], k[130:258], v[130:258], ints([0, 128]), return_lse=True, is_causal=causal)
    close(one, one_lse, formula(q[128:256], k[130:258], v[130:258], [128], [128], causal, 1 / math.sqrt(D)))


@pytest.mark.parametrize("H", [2, 160])
def test_offsets_past_32_bits(H):
    """Rows millions of elements apart: the tensors' last ones lie behind element 2^31."""
    n, D, apart = 300, 128, 1 << 23
    room = torch.empty(n * apart, dtype=torch.bfloat16, device="cuda")
    assert room.numel() > 2 ** 31
    q, k, v = inputs(170, [n], [n], H, 2, D)
    wide = []
    at = 0
    for x in (q, k, v, q):
        wide.append(room[at:].as_strided((n, x.shape[1], D), (apart, D, 1)))
        at += x.shape[1] * D
    for w, x in zip(wide, (q, k, v)):
        w.copy_(x)
    off = ints([0, 40, n])
    want, lse = sage.prompt_attention(q, k, v, off, return_lse=True)
    out, again = sage.prompt_attention(*wide[:3], off, out=wide[3], return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, again)
    # turned in place, and from there to a dense tensor
    table = sage.rotary_table(D, device="cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    tq, tk = sage.rotary(q, k, pos, table)
    sage.rotary(wide[0], wide[1], pos, table, out=(wide[0], wide[1]))
    assert torch.equal(wide[0], tq) and torch.equal(wide[1], tk)


# ------------------------------------------------------------- repeated calls --
# From its second call on a signature goes a shorter way, which has to give outputs laid out like the first one's.


def views(g, N, heads, D, layout):
    """Tensors [N, heads, D] in the layout that are dense views of the other one, without a copy."""
    x = bf16(g, heads, N, D) if layout == "NHD" else bf16(g, N, heads, D)
    return x.transpose(0, 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("layout", ["NHD", "HND"])
def test_repeated_calls_with_dense_views(layout, causal, D):
    rows, H, Hkv = [140, 3, 260], 4, 2
    off = ints(ends(rows))
    for call in range(4):
        g = gen(180 + call)
        q, k, v = (views(g, sum(rows), h, D, layout) for h in (H, Hkv, Hkv))
        assert not q.is_contiguous()
        out, lse = sage.prompt_attention(q, k, v, off, is_causal=causal, return_lse=True, tensor_layout=layout)
        assert out.shape == q.shape
        x, o = ((q, k, v), out) if layout == "NHD" else ([t.transpose(0, 1) for t in (q, k, v)], out.transpose(0, 1))
        close(o, lse, formula(*x, rows, rows, causal, 1 / math.sqrt(D)))


@pytest.mark.parametrize("D", [64, 128])
def test_repeated_calls_with_queries_of_a_projection(D):
    rows, H, Hkv = [140, 3, 260], 4, 2
    for call in range(3):
        g = gen(184 + call)
        fused = bf16(g, sum(rows), H + 2 * Hkv, D)
        q, k, v = fused[:, :H], fused[:, H:H + Hkv], fused[:, H + Hkv:]
        out = sage.prompt_attention(q, k, v, ints(ends(rows)))
        close(out, None, formula(q, k, v, rows, rows, True, 1 / math.sqrt(D)))


def test_a_unit_of_some_seconds():
    """2^28 keys of one sequence, 2.6 s for a unit: who waits for all of it waits longer than for a tile."""
    M, D = 1 << 28, 128
    if torch.cuda.mem_get_info()[0] < 2 * M * D + (8 << 30):
        pytest.skip("not enough free memory")
    ones = torch.ones((M, 1, D), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((3, 1, D), dtype=torch.bfloat16, device="cuda")
    out, lse = sage.prompt_attention(q, ones, ones, ints([0, 3]), kv_offsets=ints([0, M]), is_causal=False, return_lse=True)
    torch.cuda.synchronize()
    assert sage.device_error() == 0
    # all logits are 0: weights of 2^-8, and their sums, are exact
    assert (out == 1).all() and ((lse.double() - 28 * math.log(2)).abs() <= 2.0 ** -18).all()
    del ones
    torch.cuda.empty_cache()


# ------------------------------------------------------------------- long rows --
# The tensor core cuts a product off at 2^-25 of the sum or below, so that a sum of m products of one sign loses up to
# m 2^-26 of itself, 2^-10 for the 65536 keys after which it begins anew; the rest of the bound as above.


def close_long(out, lse, ref):
    o, l, a = ref
    err = (out.double() - o).abs()
    bound = (o.abs() + a / 64) * 2.0 ** -8 + a * (2.0 ** -8 + 2.0 ** -9)
    assert not torch.isnan(out).any() and (err <= bound).all(), (err / bound).max().item()
    assert ((lse.double() - l).abs() <= 2.0 ** -11).all()


def formula_of_row(q, k, v, sm):
    """formula() of one sequence's rows [n, H, D] that see all keys of one key/value head, key by key in parts."""
    n, H, D = q.shape
    x = q.double().permute(1, 0, 2).reshape(H * n, D)
    z = torch.cat([x @ kk.double().T * sm for kk in k[:, 0].split(1 << 20)], 1)
    lse = torch.logsumexp(z, 1)
    o, a = 0.0, 0.0
    for zz, vv in zip(z.split(1 << 20, 1), v[:, 0].split(1 << 20)):
        p = torch.exp(zz - lse[:, None])
        o, a = o + p @ vv.double(), a + p @ vv.double().abs()
    o, a = (t.reshape(H, n, D).permute(1, 0, 2) for t in (o, a))
    return o, lse.reshape(H, n), a


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("M", [(1 << 22) + 77, 65536, 65537, 3 * 65536])
def test_sums_of_long_rows(M, D):
    """Values of one sign, of which a sum in one piece loses 2.6% over 2^22 keys; beside a short sequence."""
    g = gen(190)
    rows, keys, H = [3, 200], [M, 300], 3
    q, k = bf16(g, 203, H, D), bf16(g, M + 300, 1, D)
    v = (1 + torch.rand((M + 300, 1, D), generator=g, device="cuda")).to(torch.bfloat16)
    k[M - 5000:M] *= 1.5  # the maximum follows late, too
    off, kv = ints(ends(rows)), ints(ends(keys))
    for causal in (False, True):
        out, lse = sage.prompt_attention(q, k, v, off, kv_offsets=kv, is_causal=causal, return_lse=True)
        if causal:  # rows one by one, each with the keys that it sees
            ref = [formula_of_row(q[t:t + 1], k[:M - 2 + t], v[:M - 2 + t], 1 / math.sqrt(D)) for t in range(3)]
            ref = torch.cat([r[0] for r in ref]), torch.cat([r[1] for r in ref], 1), torch.cat([r[2] for r in ref])
        else:
            ref = formula_of_row(q[:3], k[:M], v[:M], 1 / math.sqrt(D))
        close_long(out[:3], lse[:, :3], ref)
        close(out[3:], lse[:, 3:], formula(q[3:], k[M:], v[M:], [200], [300], causal, 1 / math.sqrt(D)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads", [2, 200])
def test_prompts_of_many_parts(heads, D):
    """Whole tiles of rows over several parts, in calls with few units and with a list of them; all rows like the last."""
    g = gen(191)
    n, M = 300, 150000
    q = bf16(g, 1, 2, D).expand(n, 2, D).contiguous()
    k = bf16(g, M, 1, D)
    v = (1 + torch.rand((M, 1, D), generator=g, device="cuda")).to(torch.bfloat16)
    v[M - n:] = 0.0
    k[M - n:, :] = -8.0 * q[0, :1].sign()  # what only some rows see has next to no weight with head 0
    sm = 1 / math.sqrt(D)
    x = q.repeat_interleave(heads // 2, 1)
    out, lse = sage.prompt_attention(x, k, v, ints([0, n]), kv_offsets=ints([0, M]), return_lse=True)
    ref = formula_of_row(q[:1], k[:M - n + 1], v[:M - n + 1], sm)
    out, lse = out[:, :heads // 2], lse[:heads // 2]
    close_long(out[:, :1], lse[:1], tuple(r[:, :1].expand(n, 1, D) if r.dim() == 3 else r[:1].expand(1, n) for r in ref))
    assert torch.equal(out, out[:, :1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))


@pytest.mark.parametrize("D", [64, 128])
def test_long_rows_with_values_that_are_not_finite(D):
    g = gen(192)
    n, M = 200, 140000
    q, k = bf16(g, n, 2, D), bf16(g, M, 1, D)
    v = (1 + torch.rand((M, 1, D), generator=g, device="cuda")).to(torch.bfloat16)
    off, kv = ints([0, n]), ints([0, M])
    want, lse = sage.prompt_attention(q, k, v, off, kv_offsets=kv, return_lse=True)
    w = v.clone()
    w[[5, 70000, M - 100], 0, [1, 2, 3]] = torch.tensor([math.inf, -math.inf, math.nan], device="cuda").to(torch.bfloat16)
    w[M - 1, 0, 4] = math.nan
    got, again = sage.prompt_attention(q, k, w, off, kv_offsets=kv, return_lse=True)
    assert torch.equal(again, lse)
    assert (got[:, :, 1] == math.inf).all() and (got[:, :, 2] == -math.inf).all()
    assert torch.isnan(got[100:, :, 3]).all() and torch.isnan(got[199:, :, 4]).all()
    other = torch.ones(D, dtype=torch.bool, device="cuda")
    other[1:4] = False
    assert torch.equal(got[:100, :, 3], want[:100, :, 3]) and torch.equal(got[:199][:, :, other], want[:199][:, :, other])
