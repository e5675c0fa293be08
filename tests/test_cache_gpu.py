"""The 8-bit paged key/value cache on the GPU against the oracle.

Codes, scales and tokens read back match bit for bit. Attention outputs are
held to a bound that is derived, not fitted. With A = sum_j p_j |v_j| / sum_j p_j
(in float64), an output differs from the float64 formula on the same codes by at
most
  2^-8 |o|    the rounding of the output to bf16 (half a step),
  2^-11 A     the rounding of p times the value scale to fp16 for the tensor cores,
  2^-10 A     the value scales: their logarithm and what is raised from it (a bound;
              they err by less),
  2^-12 A     logits: D products accumulated in fp32 err by at most
              (D + 3) 2^-24 sum |q_d k_d| sm_scale < 2^-13.5 here (sum |q k| sm_scale < 10),
              which p and the sum of p each take once,
together below 2^-8 |o| + 2^-9 A. (A channel whose codes are all 0 has no A and comes out as 0; the
test of empty channels allows more.) The log-sum-exp errs by the logits' 2^-13.5 and
some roundings of numbers below 16 (2^-20 each): 2^-13 in all.
"""

import math
import threading

import numpy as np
import pytest
import torch

import quantized_attention_fp64_gb300 as sage
from oracle import cache as oc
from quantized_attention_fp64_gb300.api import SageError

pytestmark = pytest.mark.gpu

DEVICE_PAGE = -16


@pytest.fixture(autouse=True)
def _library(sage_lib):
    torch.cuda.synchronize()
    sage.device_error()
    yield
    torch.cuda.synchronize()
    assert sage.device_error() == 0  # a test that expects one has read and cleared it


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=dtype).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


def f32(t):
    return t.float().cpu().numpy()


def upload(c: oc.Cache):
    return sage.QuantizedCache(dev(c.k_codes), dev(c.v_codes), dev(c.k_scale), dev(c.v_scale))


def random_cache(rng, P, H, D, page):
    """Any codes and scales; blocks that nobody wrote hold NaN scales and the codes -128."""
    c = oc.Cache(P, H, D, page)
    c.k_codes[:] = np.clip(np.rint(rng.standard_normal(c.k_codes.shape) * 40), -127, 127)
    c.v_codes[:] = np.clip(np.rint(rng.standard_normal(c.v_codes.shape) * 40), -127, 127)
    c.k_scale[:] = np.exp(rng.standard_normal(c.k_scale.shape) * 0.3) / 40
    c.v_scale[:] = np.exp(rng.standard_normal(c.v_scale.shape) * 0.3) / 40
    return c


def poison_unused(c: oc.Cache, table, lengths):
    """Blocks behind the sequences' ends get NaN scales; slots behind the end in the last block the code -128."""
    used = np.zeros((c.k_scale.shape[0], c.k_scale.shape[2]), bool)
    for b, n in enumerate(lengths):
        for pos in range(0, n, 32):
            used[c.at(table[b], pos)] = True
        if n % 32:
            page, blk = c.at(table[b], n - 1)
            k, v = (x.copy() for x in c.block_codes(page, blk))
            k[n % 32:], v[n % 32:] = -128, -128
            c.set_block_codes(page, blk, k, v)
    for s in (c.k_scale, c.v_scale):
        s.transpose(0, 2, 1)[~used] = np.nan


def make_table(rng, lengths, page, spare=2, width=None):
    """Pages in no order; entries behind a sequence's last page are far outside the cache."""
    need = [-(-n // page) for n in lengths]
    P = sum(need) + spare
    order = rng.permutation(P)
    table = np.full((len(lengths), width or max(need + [1])), 2 ** 31 - 1, np.int64)
    table[::2][table[::2] == 2 ** 31 - 1] = -5
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table.astype(np.int32), P


def same_tokens(gpu: sage.QuantizedCache, c: oc.Cache, table, lengths):
    """Codes and scales of every token of the sequences, bit for bit."""
    g = oc.Cache.__new__(oc.Cache)
    g.page_size, g.H, g.D = c.page_size, c.H, c.D
    g.k_codes, g.v_codes = gpu.k_codes.cpu().numpy(), gpu.v_codes.cpu().numpy()
    g.k_scale, g.v_scale = gpu.k_scale.cpu().numpy(), gpu.v_scale.cpu().numpy()
    for b, n in enumerate(lengths):
        for pos in range(0, n, 32):
            page, blk = c.at(table[b], pos)
            m = min(32, n - pos)
            for x, y in zip(g.block_codes(page, blk), c.block_codes(page, blk)):
                assert np.array_equal(x[:m], y[:m]), (b, pos)
            for x, y in ((g.k_scale, c.k_scale), (g.v_scale, c.v_scale)):
                assert np.array_equal(x[page, :, blk].view(np.uint32) & 0x7FFFFFFF, y[page, :, blk].view(np.uint32) & 0x7FFFFFFF), (b, pos)


# ------------------------------------------------------------------- append --

APPENDS = [
    # H, D, page, [(starts, counts)] one call after another
    (2, 128, 64, [([0, 0, 0], [1, 1, 1])]),
    (2, 128, 64, [([0, 0, 0], [70, 1, 33]), ([70, 1, 33], [1, 1, 1]), ([71, 2, 34], [1, 0, 30])]),
    (3, 64, 32, [([0, 0], [31, 32]), ([31, 32], [1, 1]), ([32, 33], [64, 65])]),
    (1, 64, 96, [([0], [200]), ([200], [3]), ([203], [53]), ([256], [1])]),
    (2, 128, 128, [([0, 0], [100, 90]), ([40, 90], [5, 2]), ([0, 92], [3, 200])]),  # cut back and written on
    (1, 128, 32, [([0], [5])] + [([5 + i], [1]) for i in range(30)]),
]


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("H,D,page,calls", APPENDS)
def test_append_bit_for_bit(H, D, page, calls, layout):
    rng = np.random.default_rng(11)
    B = len(calls[0][0])
    most = [max(s[b] + n[b] for s, n in calls) for b in range(B)]
    table, P = make_table(rng, most, page)
    c = random_cache(rng, P, H, D, page)  # what lies there before must not matter
    gpu = upload(c)
    lengths = [0] * B
    for i, (starts, counts) in enumerate(calls):
        T = max(counts) + (i % 2)  # a padded token every other call
        k, v = bf16(rng, B, T, H, D), bf16(rng, B, T, H, D)
        k[:, :, :, 3] *= 6
        v[0] *= 0.01 * (i + 1)
        oc.append(c, f32(k), f32(v), table, starts, counts)
        if layout == "HND":
            k, v = (x.transpose(1, 2).contiguous() for x in (k, v))
        sage.cache_append(gpu, k, v, ints(table), ints(starts), counts=ints(counts), tensor_layout=layout)
        lengths = [s + n if n else old for s, n, old in zip(starts, counts, lengths)]
        same_tokens(gpu, c, table, lengths)


def test_append_odd_values():
    # zeros, the smallest and largest numbers, infinities and NaN, one block each, and blocks that had them before
    D, H = 64, 1
    table = np.arange(8, dtype=np.int32)[None]
    c = oc.Cache(8, H, D, 32)
    gpu = upload(c)
    x = np.zeros((1, 256, H, D), np.float32)
    x[0, 32:64] = 2.0 ** -133 * np.arange(32)[:, None, None]       # bf16 denormals
    x[0, 64:96] = 3.3e38 * np.cos(np.arange(32))[:, None, None]
    x[0, 96, 0, 5] = np.inf
    x[0, 128:160] = 1.0
    x[0, 140, 0, 63] = np.nan
    x[0, 160:192] = np.linspace(-1, 1, 32)[:, None, None]
    x[0, 192, 0, 0] = -np.inf
    x[0, 224:256] = np.arange(-127, 129, 8)[:, None, None]         # exact codes, and ties when scaled
    k = torch.from_numpy(x).to(torch.bfloat16).cuda()
    v = k.flip(3).contiguous()
    oc.append(c, f32(k), f32(v), table, [0], [256])
    sage.cache_append(gpu, k, v, ints(table), ints([0]))
    same_tokens(gpu, c, table, [256])
    assert torch.isnan(gpu.k_scale[3:5]).all() and torch.isnan(gpu.k_scale[6]).all() and gpu.k_scale[0] == 0
    # a NaN scale stays while older tokens lie in the block, and goes when it is written from its first slot
    one = torch.ones((1, 1, H, D), dtype=torch.bfloat16, device="cuda")
    for start in (97, 96, 3):
        oc.append(c, f32(one), f32(one), table, [start], [1])
        sage.cache_append(gpu, one, one, ints(table), ints([start]))
        same_tokens(gpu, c, table, [4])
    assert gpu.k_scale[3] == np.float32(1) / np.float32(127)


@pytest.mark.parametrize("D", [64, 128])
def test_append_quotients_at_and_next_to_ties(D):
    """Scales that are powers of two make every half a tie; others put quotients next to one. All sizes of scale."""
    rng = np.random.default_rng(14)
    powers = [-133, -126, -98, -91, -90, -89, -40, -1, 0, 1, 50, 99, 100, 101, 119]
    n = len(powers) * 64
    table, P = make_table(rng, [n], 64)
    c = oc.Cache(P, 2, D, 64)
    gpu = upload(c)
    x = np.empty((1, n, 2, D))
    for i, e in enumerate(powers):
        # a block whose scale is 2^e, halves up to 127; then one whose scale is 2^e times 128..255 / 127 / 128
        halves = rng.integers(-254, 255, (32, 2, D)) / 2.0
        halves[0, :, 0] = 127
        x[0, 64 * i:64 * i + 32] = np.ldexp(halves, e)
        m = np.ldexp(rng.integers(128, 256, (32, 2, D)).astype(float), rng.integers(-9, 0, (32, 2, D)))
        m[0, :, 0] = 255 - i
        x[0, 64 * i + 32:64 * i + 64] = np.ldexp(m * rng.choice([-1, 1], m.shape), e)
    k = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
    v = -k.flip(1).contiguous()
    oc.append(c, f32(k), f32(v), table, [0], [n])
    sage.cache_append(gpu, k, v, ints(table), ints([0]))
    same_tokens(gpu, c, table, [n])
    # scales that a block already has, next to those where quotients come nearest to a turn: older
    # tokens keep the scale, and the new values' quotients by it are halves give or take a step of fp32
    scales = np.array([1 - 2.0 ** -24, 1 + 2.0 ** -23, 3 - 2.0 ** -22, 3 * (1 + 2.0 ** -23), 2 - 2.0 ** -20, 1 + 33 * 2.0 ** -23,
                       5 + 2.0 ** -21, 1 + 2.0 ** -18, 1 - 2.0 ** -19, 7 * (1 - 2.0 ** -22)], np.float32)
    c.k_scale[table[0, :5]] = c.v_scale[table[0, :5]] = scales.reshape(5, 1, 2)
    gpu.k_scale.copy_(torch.from_numpy(c.k_scale))
    gpu.v_scale.copy_(torch.from_numpy(c.v_scale))
    for i in range(10):
        s = float(scales[i])
        x = np.ldexp(rng.integers(1, 256, (1, 31, 2, D)).astype(float), rng.integers(-3, 2, (1, 31, 2, D)))
        x = np.minimum(x, np.floor(100 * s)) * rng.choice([-1, 1], x.shape)
        k = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda()
        v = k.flip(3).contiguous()
        oc.append(c, f32(k), f32(v), table, [32 * i + 1], [31])
        sage.cache_append(gpu, k, v, ints(table), ints([32 * i + 1]))
    same_tokens(gpu, c, table, [320])


def test_append_strided_inputs_and_untouched_rest():
    rng = np.random.default_rng(12)
    H, D, page = 2, 128, 64
    table, P = make_table(rng, [150, 40], page)
    c = random_cache(rng, P, H, D, page)
    gpu = upload(c)
    before = [t.clone() for t in (gpu.k_codes, gpu.v_codes, gpu.k_scale, gpu.v_scale)]
    wide = bf16(rng, 2, 45, 3, H, D)  # keys and values as slices of one tensor
    k, v = wide[:, 3:43, 0], wide[:, 3:43, 2]
    starts, counts = [64, 0], [40, 0]
    oc.append(c, f32(k), f32(v), table, starts, counts)
    sage.cache_append(gpu, k, v, ints(table), ints(starts), counts=ints(counts))
    same_tokens(gpu, c, table, [104, 0])
    touched = int(table[0, 1])
    for t, old in zip((gpu.k_codes, gpu.v_codes, gpu.k_scale, gpu.v_scale), before):
        keep = torch.arange(P, device="cuda") != touched
        assert torch.equal(t[keep].view(torch.uint8), old[keep].view(torch.uint8))


# --------------------------------------------------------------------- read --


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("H,D,page,starts,counts", [
    (2, 128, 64, [0, 0, 5], [1, 64, 90]), (3, 64, 32, [31, 32, 33, 0], [1, 65, 0, 100]), (1, 128, 96, [95], [2]),
])
def test_read_bit_for_bit(H, D, page, starts, counts, layout):
    rng = np.random.default_rng(13)
    B, T = len(starts), max(counts) + 3
    lengths = [s + n for s, n in zip(starts, counts)]
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, H, D, page)
    gpu = upload(c)
    shape = (B, T, H, D) if layout == "NHD" else (B, H, T, D)
    given = [torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
    k, v = sage.cache_read(gpu, ints(table), ints(starts), T, counts=ints(counts), tensor_layout=layout)
    sage.cache_read(gpu, ints(table), ints(starts), T, counts=ints(counts), tensor_layout=layout, out=given)
    for b in range(B):
        ref = c.tokens(table[b], starts[b], starts[b] + counts[b])
        for got, into, r in zip((k, v), given, ref):
            got, into = (x[b] if layout == "NHD" else x[b].transpose(0, 1) for x in (got, into))
            # a code times an fp32 scale, rounded to fp32 and then to bf16
            want = torch.from_numpy(r.astype(np.float32)).to(torch.bfloat16)
            assert torch.equal(got[:counts[b]].cpu(), want)
            assert (got[counts[b]:] == 0).all() and (into[counts[b]:] == 7.0).all()
            assert torch.equal(into[:counts[b]], got[:counts[b]])


# --------------------------------------------------------------------- copy --


@pytest.mark.parametrize("H,D,page,P", [(1, 64, 32, 40), (2, 128, 64, 33), (5, 128, 128, 9)])
def test_copy_pages(H, D, page, P):
    rng = np.random.default_rng(14)
    c = random_cache(rng, P, H, D, page)
    gpu = upload(c)
    order = rng.permutation(P).astype(np.int32)
    n = P // 2
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    src[1] = src[0]              # one page forked twice
    dst[2] = -1                  # no entry
    src[3] = dst[3]              # onto itself: no entry
    sage.cache_copy_pages(gpu, ints(src), ints(dst))
    for t, old in ((gpu.k_codes, c.k_codes), (gpu.v_codes, c.v_codes), (gpu.k_scale, c.k_scale), (gpu.v_scale, c.v_scale)):
        want = old.copy()
        for s, d in zip(src, dst):
            if d >= 0:
                want[d] = old[s]
        assert np.array_equal(t.cpu().numpy(), want)


@pytest.mark.parametrize("H,D,page,P,n", [
    (3, 128, 96, 900, 400),          # chunks that end inside a page, several to a warp
    (7, 64, 32, 6000, 2900), (1, 64, 32, 1 << 20, 5000),
    (8, 128, 4096, 12, 5),
])
def test_copy_many_pages(H, D, page, P, n):
    """Sources and targets in no order; every other page keeps its bytes."""
    gpu = sage.alloc_cache(P, H, "cuda", D=D, page_size=page)
    gen = torch.Generator(device="cuda").manual_seed(15)
    gpu.k_codes.view(torch.int32).random_(generator=gen)
    gpu.v_codes.view(torch.int32).random_(generator=gen)
    gpu.k_scale.uniform_(generator=gen)
    gpu.v_scale.uniform_(generator=gen)
    order = torch.randperm(P, device="cuda", generator=gen).int()
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    src[1::7] = src[0]                 # one page to many
    dst[5::11] = -1                    # and entries that stand for nothing
    src[3], dst[3] = order[-1], order[-1]
    live = (dst >= 0) & (dst != src)
    take = torch.arange(P, device="cuda")
    take[dst[live].long()] = src[live].long()
    arrays = (gpu.k_codes, gpu.v_codes, gpu.k_scale, gpu.v_scale)
    want = [t[take] for t in arrays]
    sage.cache_copy_pages(gpu, src, dst)
    for t, w in zip(arrays, want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("src,dst", [
    ([0, 1], [5, 5]), ([0, 5], [5, 6]), ([0, 99], [5, 6]), ([0, -1], [5, 6]), ([0, 1], [5, 8]),
    ([0, 1], [5, 2 ** 31 - 1]), ([0, -2 ** 31], [5, 7]),
])
def test_copy_refuses_whole_lists(src, dst):
    rng = np.random.default_rng(15)
    c = random_cache(rng, 8, 2, 64, 32)
    gpu = upload(c)
    sage.cache_copy_pages(gpu, ints(src), ints(dst))
    assert sage.device_error() == DEVICE_PAGE
    assert np.array_equal(gpu.k_codes.cpu().numpy(), c.k_codes) and np.array_equal(gpu.v_codes.cpu().numpy(), c.v_codes)
    assert np.array_equal(gpu.k_scale.cpu().numpy(), c.k_scale) and np.array_equal(gpu.v_scale.cpu().numpy(), c.v_scale)


# ---------------------------------------------------------------- attention --


def close(out, lse, ref_o, ref_lse, weight, extra=0.0):
    o = f32(out).astype(np.float64)
    tol = 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -9 * weight + 1e-30 + extra
    bad = ~(np.abs(o - ref_o) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4].tolist(), float(np.nanmax(np.abs(o - ref_o) / tol)))
    if lse is not None:
        l = f32(lse).astype(np.float64)
        assert np.array_equal(np.isinf(l), np.isinf(ref_lse)) and not np.isnan(l).any()
        fin = np.isfinite(ref_lse)
        assert (l[~fin] == -np.inf).all()
        assert np.abs(l[fin] - ref_lse[fin]).max(initial=0.0) <= 2.0 ** -13


def attend(rng, H, Hkv, D, page, lengths, q_lengths, T, causal, layout="NHD", sm=None, **kw):
    B = len(lengths)
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    poison_unused(c, table, lengths)
    q = bf16(rng, B, T, H, D)
    ragged = q_lengths is not None
    ref = oc.attention(c, f32(q), table, lengths, q_lengths if ragged else [T] * B, causal, 1 / math.sqrt(D) if sm is None else sm)
    gpu = upload(c)
    qq = q if layout == "NHD" else q.transpose(1, 2).contiguous()
    out, lse = sage.cache_attention(qq, gpu, ints(table), ints(lengths), q_lengths=ints(q_lengths) if ragged else None,
                                    is_causal=causal, sm_scale=sm, return_lse=True, tensor_layout=layout, **kw)
    close(out if layout == "NHD" else out.transpose(1, 2), lse, *ref)
    # without the log-sum-exp the outputs are the same
    again = sage.cache_attention(qq, gpu, ints(table), ints(lengths), q_lengths=ints(q_lengths) if ragged else None,
                                 is_causal=causal, sm_scale=sm, tensor_layout=layout)
    assert torch.equal(again, out)


ATTENTION = [
    # H, Hkv, D, page, lengths, q_lengths (None: T each), T, causal
    (1, 1, 128, 32, [1], None, 1, True),
    (1, 1, 64, 32, [0], None, 1, False),                                # no key at all
    (7, 1, 128, 64, [1000], None, 1, True),
    (8, 8, 64, 64, [31, 32, 33, 1, 64, 65], None, 1, False),
    (28, 4, 128, 64, [700, 0, 3], None, 1, True),
    (40, 2, 64, 96, [257, 95, 96, 97], None, 1, True),                  # 20 rows of one key/value head
    (64, 1, 128, 128, [300, 129], None, 1, True),                       # 64 rows
    (16, 4, 64, 32, [401, 7, 40], [5, 1, 3], 5, True),
    (4, 2, 128, 64, [5, 2, 1, 0], [4, 4, 3, 2], 4, True),               # rows before the first token see nothing
    (4, 2, 128, 64, [100, 9], [0, 4], 4, True),                         # a sequence without queries
    (6, 2, 128, 64, [150, 33], None, 50, True),
    (2, 2, 64, 64, [77, 130], None, 200, False),
    (4, 4, 128, 32, [140, 200], [130, 129], 131, True),
    (5, 1, 128, 128, [300], None, 129, True),
    (3, 3, 64, 64, [513, 1], None, 257, False),
    (8, 2, 128, 64, [3001], None, 40, True),
    (2, 1, 64, 64, [5000], None, 2, True),
    (4, 4, 128, 64, [20, 300], None, 300, True),                        # more queries than tokens
    (2, 2, 64, 32, [(61 * i) % 500 for i in range(90)], [(37 * i) % 291 for i in range(90)], 290, True),
    (3, 1, 128, 64, [1500, 40, 0, 2300], [190, 10, 190, 0], 190, False),
    # more sequences than threads in a CTA
    (2, 1, 64, 32, [(7 * i) % 90 for i in range(1500)], None, 1, True),
    (5, 1, 64, 32, [(7 * i) % 90 for i in range(1300)], [i % 5 for i in range(1300)], 4, True),
    (4, 1, 64, 32, [(11 * i) % 120 for i in range(700)], [i % 41 for i in range(700)], 40, False),
    (2, 2, 64, 32, [(11 * i) % 120 for i in range(600)], [(3 * i) % 131 for i in range(600)], 130, True),
    # calls whose blocks are cut evenly over the GPU, items shared by CTAs and CTAs by items
    (14, 2, 128, 64, [9001, 10, 0, 4000], None, 1, True),
    (4, 1, 64, 128, [10000, 33], [3, 2], 3, True),
    (40, 2, 128, 64, [8500, 500], None, 1, False),
    (9, 1, 64, 32, [8200, 1, 5], [2, 0, 3], 3, True),
    (8, 4, 128, 64, [(37 * i) % 400 for i in range(130)], None, 1, True),
    (8, 8, 64, 32, [(53 * i) % 300 for i in range(150)], [i % 3 for i in range(150)], 2, True),
    (16, 4, 64, 64, [(91 * i) % 700 for i in range(140)], None, 5, True),
]


@pytest.mark.parametrize("H,Hkv,D,page,lengths,q_lengths,T,causal", ATTENTION)
def test_attention(H, Hkv, D, page, lengths, q_lengths, T, causal):
    attend(np.random.default_rng(21), H, Hkv, D, page, lengths, q_lengths, T, causal)


FOLDED = [
    # 33 to 128 rows of a key/value head over long and short sequences: parts whose key tiles two
    # warpgroups share, whole items and items cut over CTAs, odd numbers of tiles, rows that see none
    (8, 1, 128, 64, [1200, 3000, 1025], None, 8, True),
    (8, 1, 64, 32, [1200, 3000, 1025], None, 8, True),
    (4, 4, 64, 32, [5000, 1100], [100, 33], 100, False),
    (16, 2, 128, 64, [2048] * 40, None, 5, True),
    (4, 1, 128, 32, [9000], [40], 64, True),
    (12, 2, 64, 64, [1500, 20], None, 50, True),
    (5, 1, 128, 128, [511, 512, 513, 575, 577, 0, 1], [25, 24, 0, 1, 25, 25, 25], 25, False),
    (8, 8, 64, 64, [(97 * i) % 1500 for i in range(30)], [(7 * i) % 41 for i in range(30)], 40, True),
    (4, 1, 128, 32, [(61 * i) % 900 for i in range(200)], [(5 * i) % 18 for i in range(200)], 17, True),
]


@pytest.mark.parametrize("H,Hkv,D,page,lengths,q_lengths,T,causal", FOLDED)
def test_attention_one_query_tile(H, Hkv, D, page, lengths, q_lengths, T, causal):
    attend(np.random.default_rng(31), H, Hkv, D, page, lengths, q_lengths, T, causal)


@pytest.mark.parametrize("D", [64, 128])
def test_attention_one_query_tile_nan_and_bad_pages(D):
    """A NaN scale reaches the rows that see it only; a page that is not there counts as one without tokens."""
    rng = np.random.default_rng(32)
    H, Hkv, page, n, T = 8, 1, 64, 2100, 9
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    q = bf16(rng, 1, T, H, D)
    clean = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=True)
    pg, blk = c.at(table[0], n - 1)  # tokens 2080 .. 2099: rows t see up to 2091 + t
    for s in (c.k_scale, c.v_scale):
        was = s[pg, 0, blk]
        s[pg, 0, blk] = np.nan
        out = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=True)
        assert torch.isnan(out.float()).all()
        s[pg, 0, blk] = was
    early = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=True, q_lengths=ints([T]))
    assert torch.equal(early, clean)
    bad = table.copy()
    bad[0, 3] = 2 ** 30
    out, lse = sage.cache_attention(q, upload(c), ints(bad), ints([n]), is_causal=True, return_lse=True)
    assert sage.device_error() == DEVICE_PAGE
    c.k_scale[table[0, 3]] = 0.0  # the definition without these 64 tokens: their weight taken out by hand
    o, l, w = oc.attention(c, f32(q), table, [n], [T], True, 1 / math.sqrt(D))
    c.v_scale[table[0, 3]] = 0.0
    o, _, w = oc.attention(c, f32(q), table, [n], [T], True, 1 / math.sqrt(D))
    part = 1.0 - 64.0 / np.exp(l)  # keys of scale 0 have the logit 0: 64 ones in the sum
    part = np.moveaxis(part, 1, 2)[..., None]
    close(out, lse, o / part, l + np.log(part[..., 0].transpose(0, 2, 1)), w / part)


@pytest.mark.parametrize("case", [2, 7, 10, 11])
def test_attention_hnd_and_scale(case):
    H, Hkv, D, page, lengths, q_lengths, T, causal = ATTENTION[case]
    attend(np.random.default_rng(22), H, Hkv, D, page, lengths, q_lengths, T, causal, layout="HND", sm=0.031)


@pytest.mark.parametrize("T", [1, 3, 20, 150])
def test_attention_peaked_rows(T):
    """Logits far apart: the running maximum moves late and by much; the last tokens hold the largest."""
    rng = np.random.default_rng(23)
    H, Hkv, D, page, n = 4, 2, 128, 64, 900
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    for pos in range(0, n, 32):
        page_, blk = c.at(table[0], pos)
        c.k_scale[page_, :, blk] = (0.2 if pos < 600 else 1.0) * (1 + pos / n) / 40
        c.v_scale[page_, :, blk] = 10.0 ** ((pos // 32) % 5 - 2) / 40
    q = bf16(rng, 1, T, H, D)
    ref = oc.attention(c, f32(q), table, [n], [T], True, 0.088)
    out, lse = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=True, sm_scale=0.088, return_lse=True)
    # sum |q k| sm_scale < 2^4.5 here: four times the logits' error of the bound above
    o, tol = f32(out).astype(np.float64), 2.0 ** -8 * np.abs(ref[0]) + 2.0 ** -9 * ref[2] + 2.0 ** -10 * ref[2]
    assert (np.abs(o - ref[0]) <= tol).all()
    assert np.abs(f32(lse) - ref[1]).max() <= 2.0 ** -11


@pytest.mark.parametrize("T", [1, 6, 13, 40, 140])
def test_attention_nan_stays_with_the_rows_that_see_it(T):
    rng = np.random.default_rng(24)
    H, Hkv, D, page = 4, 2, 64, 64
    lengths = [200 + T, 200 + T]
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    q = bf16(rng, 2, T, H, D)
    clean = sage.cache_attention(q, upload(c), ints(table), ints(lengths), is_causal=True)
    pg, blk = c.at(table[0], 70)
    c.k_scale[pg, 1, blk] = np.nan                      # key/value head 1 of sequence 0
    pg, blk = c.at(table[1], 199 + T)                   # the last block of sequence 1, head 0
    c.v_scale[pg, 0, blk] = np.nan
    out = sage.cache_attention(q, upload(c), ints(table), ints(lengths), is_causal=True)
    assert torch.isnan(out[0, :, 2:].float()).all() and torch.equal(out[0, :, :2], clean[0, :, :2])
    first = (199 + T) // 32 * 32 - 200                  # the first row that sees a token of that block
    assert torch.isnan(out[1, max(first, 0):, :2].float()).all()
    assert torch.equal(out[1, :, 2:], clean[1, :, 2:])
    if first > 0:
        assert torch.equal(out[1, :first, :2], clean[1, :first, :2])


def lost_weights(c, q, table, lengths, q_lengths, sm):
    """What fp16 weights that hold the value scales may lose, [B, T, H, 1] float64. The
    weights p_j s_j are scaled so that the largest is at least 1, and one below 2^-14 is rounded to a
    multiple of 2^-24: by at most 2^-25 of the largest. Codes are at most 127, so over n keys the sum
    errs by at most 127 n 2^-25 max_j p_j s_j / sum_j p_j."""
    B, T, H, _ = q.shape
    lost = np.zeros((B, T, H, 1))
    for b in range(B):
        n = int(lengths[b])
        k, _ = c.tokens(table[b], 0, n)
        s = np.stack([c.v_scale[c.at(table[b], pos)[0], :, c.at(table[b], pos)[1]] for pos in range(n)]).astype(np.float64)
        sees = np.clip(n - q_lengths[b] + 1 + np.arange(T), 0, n)
        for h in range(H):
            z = q[b, :, h].astype(np.float64) @ k[:, h // (H // c.H)].T * sm
            z[np.arange(n)[None, :] >= sees[:, None]] = -np.inf
            p = np.exp(z - z.max(1, keepdims=True))
            lost[b, :, h, 0] = 127 * n * 2.0 ** -25 * (p * s[:, h // (H // c.H)]).max(1) / p.sum(1)
    return lost


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [1, 6, 40, 200])
def test_attention_value_scales_far_apart(T, D):
    """Small values next to huge ones: what a row does not see, or gives no weight, costs it no precision."""
    rng = np.random.default_rng(27)
    H, Hkv, page = 4, 2, 64
    n = 900 + T
    table, P = make_table(rng, [n, n], page)
    c = random_cache(rng, P, Hkv, D, page)
    for pos in range(0, n, 32):
        for b, e in ((0, 1e-6 if pos < 900 else 1e6), (1, 10.0 ** ((pos // 32 * 5) % 13 - 6))):
            pg, blk = c.at(table[b], pos)
            c.v_scale[pg, :, blk] *= e
    q = bf16(rng, 2, T, H, D)
    sm = 1 / math.sqrt(D)
    for lengths in ([n, n], [900, 900]):  # and without the huge tokens of sequence 0
        out, lse = sage.cache_attention(q, upload(c), ints(table), ints(lengths), is_causal=True, return_lse=True)
        extra = lost_weights(c, f32(q), table, lengths, [T, T], sm)
        close(out, lse, *oc.attention(c, f32(q), table, lengths, [T, T], True, sm), extra)


@pytest.mark.parametrize("T", [1, 6, 40])
def test_attention_little_weight_large_values(T):
    """The tokens that the rows give 2^-22 of the weight hold values 2^22 times larger."""
    rng = np.random.default_rng(29)
    H, Hkv, D, page, n = 2, 1, 64, 64, 6144
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    q = np.ones((1, T, H, D), np.float32)
    c.k_codes[:] = np.sign(c.k_codes) + (c.k_codes == 0)
    for pos in range(0, n, 32):
        pg, blk = c.at(table[0], pos)
        k, v = (x.copy() for x in c.block_codes(pg, blk))
        low = pos // 128 % 2 == 1  # every other block of each warp that takes every fourth
        # keys whose product with the queries is 64 s_k or -64 s_k, give or take one channel
        k[:] = -1 if low else 1
        k[np.arange(k.shape[0]), :, np.arange(k.shape[0]) % D] *= -1
        c.set_block_codes(pg, blk, k, v)
        c.k_scale[pg, :, blk] = 15.38 / 124  # logits of 7.69 and -7.69: weights of 3.5 steps of fp16 below its normal numbers
        c.v_scale[pg, :, blk] = 2.0 ** 22 / 40 if low else 1.0 / 40
    out, lse = sage.cache_attention(torch.from_numpy(q).to(torch.bfloat16).cuda(), upload(c), ints(table), ints([n]),
                                    return_lse=True, sm_scale=1.0)
    close(out, lse, *oc.attention(c, q, table, [n], [T], False, 1.0))


@pytest.mark.parametrize("e", [-100, -30, 60, 110])
@pytest.mark.parametrize("T", [1, 20, 150])
def test_attention_queries_of_any_size(T, e):
    """Queries times 2^e and sm_scale times 2^-e: the same logits, and fp16 holds neither."""
    rng = np.random.default_rng(37)
    H, Hkv, D, page, n = 2, 2, 64, 64, 500
    table, P = make_table(rng, [n], page)
    gpu = upload(random_cache(rng, P, Hkv, D, page))
    q = bf16(rng, 1, T, H, D)
    a = sage.cache_attention(q, gpu, ints(table), ints([n]), is_causal=True, sm_scale=0.125, return_lse=True)
    b = sage.cache_attention((q.double() * 2.0 ** e).to(torch.bfloat16), gpu, ints(table), ints([n]), is_causal=True,
                             sm_scale=0.125 * 2.0 ** -e, return_lse=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T", [1, 3, 9, 100])
def test_attention_fresh_cache(T):
    """Tokens of scale 0 (as a cleared cache holds them) are keys and values of 0."""
    gpu = sage.alloc_cache(20, 2, "cuda", D=128, page_size=32)
    q = bf16(np.random.default_rng(38), 1, T, 8, 128)
    out, lse = sage.cache_attention(q, gpu, ints([list(range(20))]), ints([600]), return_lse=True)
    assert (out == 0).all() and (lse - math.log(600)).abs().max().item() <= 2.0 ** -13


@pytest.mark.parametrize("T", [1, 2, 4, 8, 40])
def test_attention_empty_channels(T):
    """Channels whose codes are all 0, as in a padded head dimension."""
    rng = np.random.default_rng(30)
    H, Hkv, D, page, n = 8, 1, 128, 64, 3000
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    c.v_codes[:, :, :, 96:] = 0
    q = bf16(rng, 1, T, H, D)
    out = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=True)
    ref = oc.attention(c, f32(q), table, [n], [T], True, 1 / math.sqrt(D))
    close(out[..., :96], None, *(x[..., :96] if x.ndim == 4 else x for x in ref))
    assert out[..., 96:].abs().max().item() <= 2.0 ** -10 * c.v_scale.max()


def test_attention_unseen_tokens_do_not_matter():
    """Rows of a chunk before a block of huge values, in the same call and the same key tiles."""
    rng = np.random.default_rng(28)
    H, Hkv, D, page, n, T = 4, 1, 128, 64, 640, 300
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    q = bf16(rng, 1, T, H, D)
    as_before = c.v_scale.copy()
    for pos in range(480, n, 32):
        pg, blk = c.at(table[0], pos)
        c.v_scale[pg, :, blk] *= 1e7
    out, lse = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=True, return_lse=True)
    ref = oc.attention(c, f32(q), table, [n], [T], True, 1 / math.sqrt(D))
    # rows t < 140 see the keys up to 339 + t, none of them huge
    close(out, lse, *ref, lost_weights(c, f32(q), table, [n], [T], 1 / math.sqrt(D)))
    c.v_scale[:] = as_before
    small = oc.attention(c, f32(q), table, [n], [T], True, 1 / math.sqrt(D))
    assert np.array_equal(small[0][:, :140], ref[0][:, :140])


@pytest.mark.parametrize("T", [1, 6, 140])
def test_attention_leaves_padding_rows_as_they_were(T):
    rng = np.random.default_rng(25)
    H, Hkv, D, page, lengths = 4, 2, 128, 64, [90, 300, 10]
    q_lengths = [T, max(T - 2, 0), 0]
    table, P = make_table(rng, lengths, page)
    gpu = upload(random_cache(rng, P, Hkv, D, page))
    q = bf16(rng, 3, T, H, D)
    q_bad = q.clone()
    for b, n in enumerate(q_lengths):
        q_bad[b, n:] = float("nan")
    base = torch.full((3, T + 2, H + 1, D), 3.0, dtype=torch.bfloat16, device="cuda")
    view = base[:, 1:-1, :H]
    sage.cache_attention(q_bad, gpu, ints(table), ints(lengths), q_lengths=ints(q_lengths), is_causal=True, out=view)
    ref = sage.cache_attention(q, gpu, ints(table), ints(lengths), q_lengths=ints(q_lengths), is_causal=True)
    for b, n in enumerate(q_lengths):
        assert torch.equal(view[b, :n], ref[b, :n])
        assert (view[b, n:] == 3.0).all() and (ref[b, n:] == 0).all()
    assert (base[:, 0] == 3.0).all() and (base[:, -1] == 3.0).all() and (base[:, :, H] == 3.0).all()


def test_attention_shared_pages_and_same_row_twice():
    rng = np.random.default_rng(26)
    table, P = make_table(rng, [500], 64)
    c = random_cache(rng, P, 2, 128, 64)
    gpu = upload(c)
    both = np.concatenate([table, table, table])
    q = bf16(rng, 1, 1, 8, 128)
    out = sage.cache_attention(q.expand(3, 1, 8, 128).contiguous(), gpu, ints(both), ints([500, 500, 200]))
    one = sage.cache_attention(q, gpu, ints(table), ints([500]))
    assert torch.equal(out[0], out[1])
    # how the work was divided may differ, by roundings of fp32 and one of bf16
    assert (out[0].float() - one[0].float()).abs().max() <= 2.0 ** -7 * one.float().abs().max()
    ref = oc.attention(c, f32(q.expand(3, 1, 8, 128)), both, [500, 500, 200], [1] * 3, False, 1 / math.sqrt(128))
    close(out, None, *ref)


# ------------------------------------------------------------ device checks --


@pytest.mark.parametrize("T", [1, 140])
def test_bad_pages_and_lengths_are_flagged(T):
    rng = np.random.default_rng(27)
    H, D, page = 2, 64, 32
    table, P = make_table(rng, [96, 96], page, spare=0)
    c = random_cache(rng, P, H, D, page)
    gpu = upload(c)
    q = bf16(rng, 2, T, H, D)
    good = sage.cache_attention(q, gpu, ints(table), ints([64, 96]))
    broken = table.copy()
    broken[0, 2] = P            # sequence 0's third page is not there: as if its tokens were none
    broken[1, 1] = -1
    out = sage.cache_attention(q, gpu, ints(broken), ints([96, 96]))
    assert sage.device_error() == DEVICE_PAGE
    assert torch.isfinite(out.float()).all()
    assert (out[0].float() - good[0].float()).abs().max() <= 2.0 ** -7 * good.float().abs().max()
    out = sage.cache_attention(q, gpu, ints(table), ints([2 ** 31 - 1, -3]))   # cut to the table, and to nothing
    assert sage.device_error() == DEVICE_PAGE
    full = sage.cache_attention(q, gpu, ints(table), ints([96, 0]))
    assert torch.equal(out, full) and (out[1] == 0).all()
    before = [t.clone() for t in (gpu.k_codes, gpu.v_codes, gpu.k_scale, gpu.v_scale)]
    k = bf16(rng, 2, 40, H, D)
    for starts, counts in (([96, 200], [40, 1]), ([-1000, 97], [0, 1])):
        sage.cache_append(gpu, k, k, ints(table), ints(starts), counts=ints(counts))
        assert sage.device_error() == DEVICE_PAGE
    wild = np.full_like(table, 2 ** 31 - 1)
    sage.cache_append(gpu, k, k, ints(wild), ints([0, 0]))
    assert sage.device_error() == DEVICE_PAGE
    x = torch.full((2, 40, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    sage.cache_read(gpu, ints(wild), ints([0, 0]), 40, out=(x, x))
    assert sage.device_error() == DEVICE_PAGE and (x == 5.0).all()
    for t, old in zip((gpu.k_codes, gpu.v_codes, gpu.k_scale, gpu.v_scale), before):
        assert torch.equal(t.view(torch.uint8), old.view(torch.uint8))


def test_empty_calls():
    gpu = sage.alloc_cache(4, 2, "cuda", D=64, page_size=32)
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    x = torch.empty((0, 5, 2, 64), dtype=torch.bfloat16, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    sage.cache_append(gpu, x, x, none, e)
    assert sage.cache_read(gpu, none, e, 5)[0].shape == (0, 5, 2, 64)
    assert sage.cache_attention(x, gpu, none, e).shape == (0, 5, 2, 64)
    sage.cache_copy_pages(gpu, e, e)
    y = torch.empty((1, 0, 2, 64), dtype=torch.bfloat16, device="cuda")
    t, z = ints([[0, 1]]), ints([0])
    sage.cache_append(gpu, y, y, t, z)
    assert sage.cache_read(gpu, t, z, 0)[1].shape == (1, 0, 2, 64)
    out, lse = sage.cache_attention(y, gpu, t, z, return_lse=True)
    assert out.shape == (1, 0, 2, 64) and lse.shape == (1, 2, 0)
    # a table without pages: a sequence without tokens
    q = torch.ones((1, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    out, lse = sage.cache_attention(q, gpu, torch.empty((1, 0), dtype=torch.int32, device="cuda"), z, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


# --------------------------------------------------------------- refusals --


def test_refusals():
    gpu = sage.alloc_cache(4, 2, "cuda", D=64, page_size=32)
    x = torch.zeros((1, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    t, n = ints([[0, 1]]), ints([3])

    def refused(code, f, *a, **kw):
        with pytest.raises(SageError) as e:
            f(*a, **kw)
        assert e.value.code == code

    for f in (lambda *a, **kw: sage.cache_append(gpu, a[0], a[0], *a[1:], **kw),
              lambda *a, **kw: sage.cache_attention(a[0], gpu, *a[1:], **kw)):
        refused(-3, f, x.half(), t, n)
        refused(-3, f, x, t.long(), n)
        refused(-3, f, x, t, n.long())
        refused(-5, f, x[0], t, n)
        refused(-5, f, torch.zeros((1, 3, 2, 128), dtype=torch.bfloat16, device="cuda"), t, n)
        refused(-5, f, x, t[0], n)
        refused(-5, f, x, ints([[0], [1]]), n)
        refused(-5, f, x, t, ints([3, 3]))
        refused(-6, f, x, t, n, tensor_layout="BSHD")
        refused(-6, f, x, ints([[0, 0], [1, 1]]).T[:1], n)
        refused(-6, f, x.transpose(2, 3).contiguous().transpose(2, 3), t, n)
        refused(-7, f, torch.zeros((1, 3, 2, 65), dtype=torch.bfloat16, device="cuda")[..., 1:], t, n)
        with pytest.raises(ValueError):
            f(x.cpu(), t, n)
        with pytest.raises(ValueError):
            f(x, t.cpu(), n)
        with pytest.raises(ValueError):
            f(x, t, n.cpu())
        with pytest.raises(TypeError):
            f(x, t, None)
    refused(-5, sage.cache_append, gpu, q, q, t, n)
    refused(-5, sage.cache_append, gpu, x, x[:, :2], t, n)
    refused(-5, sage.cache_attention, torch.zeros((1, 3, 3, 64), dtype=torch.bfloat16, device="cuda"), gpu, t, n)
    refused(-5, sage.cache_attention, q, gpu, t, n, out=x)
    refused(-13, sage.cache_attention, q, gpu, t, n, sm_scale=0.0)
    refused(-13, sage.cache_attention, q, gpu, t, n, sm_scale=math.inf)
    refused(-5, sage.cache_read, gpu, t, n, -1)
    refused(-5, sage.cache_read, gpu, t, n, 3, out=(x, q))
    refused(-3, sage.cache_copy_pages, gpu, n.long(), n)
    refused(-5, sage.cache_copy_pages, gpu, n, ints([1, 2]))
    refused(-5, sage.QuantizedCache, gpu.k_codes, gpu.v_codes, gpu.k_scale[:3], gpu.v_scale)
    refused(-3, sage.QuantizedCache, gpu.k_codes, gpu.v_codes, gpu.k_scale.half(), gpu.v_scale)
    need = sage.cache_attention_workspace_size(1, 3, 4, 2, 64)
    if need:
        refused(-9, sage.cache_attention, q, gpu, t, n, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------ a run of them, as used --


def test_prompt_fork_decode_compact():
    """A prompt in two chunks, a fork that writes on, decoding of both, compaction of the pages: every
    step's attention against the oracle's on the same tokens."""
    rng = np.random.default_rng(31)
    H, Hkv, D, page, P = 8, 2, 128, 64, 16
    sm = 1 / math.sqrt(D)
    c = oc.Cache(P, Hkv, D, page)
    gpu = sage.alloc_cache(P, Hkv, "cuda", D=D, page_size=page)
    table = np.full((2, 4), -1, np.int32)
    table[0] = [9, 4, 13, 2]

    def step(rows, starts, T):
        """New tokens for the given sequences, then their attention."""
        k, v, q = bf16(rng, len(rows), T, Hkv, D), bf16(rng, len(rows), T, Hkv, D), bf16(rng, len(rows), T, H, D)
        lengths = [s + T for s in starts]
        oc.append(c, f32(k), f32(v), table[rows], starts, [T] * len(rows))
        sage.cache_append(gpu, k, v, ints(table[rows]), ints(starts))
        out, lse = sage.cache_attention(q, gpu, ints(table[rows]), ints(lengths), is_causal=True, return_lse=True)
        close(out, lse, *oc.attention(c, f32(q), table[rows], lengths, [T] * len(rows), True, sm))
        same_tokens(gpu, c, table[rows], lengths)

    step([0], [0], 90)
    step([0], [90], 50)                                # 140 tokens: pages 9, 4 and 12 of 13
    table[1] = [9, 4, 7, 11]                           # the fork shares the full pages; its last one is copied
    sage.cache_copy_pages(gpu, ints([13]), ints([7]))
    for a in (c.k_codes, c.v_codes, c.k_scale, c.v_scale):
        a[7] = a[13]
    for i in range(3):
        step([0, 1], [140 + i, 140 + i], 1)
    step([0, 1], [143, 143], 60)                       # into the fourth pages
    moves = [(9, 0), (13, 1), (11, 3), (7, 5)]         # compaction: pages 0..5
    sage.cache_copy_pages(gpu, ints([s for s, _ in moves]), ints([d for _, d in moves]))
    old = [a.copy() for a in (c.k_codes, c.v_codes, c.k_scale, c.v_scale)]
    for s, d in moves:
        for a, o in zip((c.k_codes, c.v_codes, c.k_scale, c.v_scale), old):
            a[d] = o[s]
        table[table == s] = d
    step([0, 1], [203, 203], 1)
    step([1], [204], 7)


def test_cross_attention_to_an_encoder():
    """An encoder's states appended once and attended to by queries of another length, next to the
    framework's attention on full-precision copies: the codes are 8 bits, so the two are near, not equal."""
    rng = np.random.default_rng(32)
    H, D, page, n, T = 4, 128, 64, [77, 150], 260
    gpu = sage.alloc_cache(6, H, "cuda", D=D, page_size=page)
    table = np.array([[0, 2, 4], [1, 3, 5]], np.int32)
    k, v, q = bf16(rng, 2, 150, H, D), bf16(rng, 2, 150, H, D), bf16(rng, 2, T, H, D)
    sage.cache_append(gpu, k, v, ints(table), ints([0, 0]), counts=ints(n))
    out = sage.cache_attention(q, gpu, ints(table), ints(n))
    kk, vv = sage.cache_read(gpu, ints(table), ints([0, 0]), 150, counts=ints(n))
    for b in range(2):
        for x, xx in ((k, kk), (v, vv)):
            # half a code's step of the block's largest value, and the read's rounding to bf16
            assert (x[b, :n[b]].float() - xx[b, :n[b]].float()).abs().max() <= x.float().abs().max() * (0.5 / 127 + 2.0 ** -8)
        z = torch.einsum("thd,jhd->htj", q[b].double(), kk[b, :n[b]].double()) / math.sqrt(D)
        ref = torch.einsum("htj,jhd->thd", z.softmax(-1), vv[b, :n[b]].double())
        # keys and values read back as bf16 differ from the cached ones by 2^-8: logits by at most 2^-8 * 10,
        # weights by twice that, values by 2^-8; and the kernel's own 2^-8 |o| + 2^-9 A, with A < max |v|
        assert (out[b].double() - ref).abs().max() <= (2 * 10 + 3) * 2.0 ** -8 * vv[b].abs().max().double()


def test_graph_replay_with_moving_lengths():
    """One captured step (append, attention) replayed while the program advances lengths and pages."""
    rng = np.random.default_rng(33)
    B, H, Hkv, D, page = 3, 8, 2, 64, 32
    starts0 = [30, 0, 63]
    table, P = make_table(rng, [80, 80, 120], page)
    c = random_cache(rng, P, Hkv, D, page)
    gpu = upload(c)
    t, n0, n1 = ints(table), ints(starts0), ints([s + 1 for s in starts0])
    k, v, q = (torch.zeros((B, 1, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hkv, Hkv, H))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sage.cache_attention(q, gpu, t, n1)  # the first call on a device finds the error word
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sage.cache_append(gpu, k, v, t, n0)
        out, lse = sage.cache_attention(q, gpu, t, n1, is_causal=True, return_lse=True)
    for i in range(5):
        for x, h in ((k, Hkv), (v, Hkv), (q, H)):
            x.copy_(bf16(rng, B, 1, h, D))
        starts = [s + i for s in starts0]
        oc.append(c, f32(k), f32(v), table, starts, [1] * B)
        # an eager call between the replays uses a workspace of its own
        sage.cache_attention(q, gpu, t, n1)
        g.replay()
        close(out, lse, *oc.attention(c, f32(q), table, [s + 1 for s in starts], [1] * B, True, 1 / math.sqrt(D)))
        same_tokens(gpu, c, table, [s + 1 for s in starts])
        n0.add_(1)
        n1.add_(1)


@pytest.mark.parametrize("T", [1, 12, 80])
def test_two_graphs_replayed_at_once(T):
    """Each captured call keeps a workspace of its own: replays on two streams do not disturb one another."""
    rng = np.random.default_rng(35)
    B, H, Hkv, D, page = 2, 8, 2, 128, 64
    lengths = [5000, 3000]
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    gpu, t, n = upload(c), ints(table), ints(lengths)
    qs = [bf16(rng, B, T, H, D) for _ in (0, 1)]
    alone = [sage.cache_attention(q, gpu, t, n, is_causal=True) for q in qs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(sage.cache_attention(q, gpu, t, n, is_causal=True))
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], alone[0]) and torch.equal(outs[1], alone[1])


@pytest.mark.parametrize("T", [1, 12, 80, 300])
def test_page_table_rows_of_a_wider_tensor(T):
    rng = np.random.default_rng(36)
    lengths = [400, 301, 0]
    table, P = make_table(rng, lengths, 32)
    c = random_cache(rng, P, 2, 64, 32)
    gpu = upload(c)
    wide = torch.full((3, table.shape[1] + 9), 2 ** 30, dtype=torch.int32, device="cuda")
    view = wide[:, 4:4 + table.shape[1]]
    view.copy_(ints(table))
    q = bf16(rng, 3, T, 4, 64)
    for a, b in zip(sage.cache_attention(q, gpu, view, ints(lengths), return_lse=True),
                    sage.cache_attention(q, gpu, ints(table), ints(lengths), return_lse=True)):
        assert torch.equal(a, b)
    k, v = sage.cache_read(gpu, view, ints([3, 3, 0]), 290, counts=ints([290, 290, 0]))
    for b in (0, 1):
        for got, want in zip((k, v), c.tokens(table[b], 3, 293)):
            assert torch.equal(got[b].cpu(), torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))
    kk, vv = bf16(rng, 3, 1, 2, 64), bf16(rng, 3, 1, 2, 64)
    oc.append(c, f32(kk), f32(vv), table, [399, 300, 0], [1, 1, 0])
    sage.cache_append(gpu, kk, vv, view, ints([399, 300, 0]), counts=ints([1, 1, 0]))
    same_tokens(gpu, c, table, [400, 301, 0])


def test_threads_with_caches_of_their_own():
    """Caches of different sizes, made and used by threads at the same time, each on a stream of its own."""
    n_threads = 4
    go, found = threading.Barrier(n_threads), [None] * n_threads

    def work(i):
        try:
            rng = np.random.default_rng(50 + i)
            H, D, page, n = 1 + i, (64, 128)[i % 2], 32 * (1 + i // 2), 100 + 40 * i
            table, P = make_table(rng, [n], page)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                k, v, q = bf16(rng, 1, n, H, D), bf16(rng, 1, n, H, D), bf16(rng, 1, 3, 4 * H, D)
                t, zero, lens = ints(table), ints([0]), ints([n])
                go.wait(60)
                for _ in range(20):
                    gpu = sage.alloc_cache(P, H, "cuda", D=D, page_size=page)
                    sage.cache_append(gpu, k, v, t, zero)
                    out, lse = sage.cache_attention(q, gpu, t, lens, is_causal=True, return_lse=True)
                    kk, vv = sage.cache_read(gpu, t, zero, n)
                stream.synchronize()
                c = oc.Cache(P, H, D, page)
                oc.append(c, f32(k), f32(v), table, [0], [n])
                same_tokens(gpu, c, table, [n])
                for got, want in zip((kk, vv), c.tokens(table[0], 0, n)):
                    assert torch.equal(got[0].cpu(), torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16))
                close(out, lse, *oc.attention(c, f32(q), table, [n], [3], True, 1 / math.sqrt(D)))
            found[i] = "right"
        except BaseException as e:  # a thread's failure is the test's
            found[i] = e
            go.abort()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n_threads)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert found == ["right"] * n_threads, found


def test_two_streams_at_once():
    rng = np.random.default_rng(34)
    table, P = make_table(rng, [2000, 1500], 64)
    c = random_cache(rng, P, 2, 128, 64)
    gpu = upload(c)
    t, n = ints(table), ints([2000, 1500])
    qs = [bf16(rng, 2, 1, 8, 128) for _ in range(8)]
    alone = [sage.cache_attention(q, gpu, t, n) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for rep in range(5):
        for i, q in enumerate(qs):
            with torch.cuda.stream(streams[i % 2]):
                outs.append(sage.cache_attention(q, gpu, t, n))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o, alone[i % len(qs)])


# ------------------------------------------- value scales of the whole range --
#
# Scales from 0 and 2^-120 to 2^120 next to one another. The bound is that of the module with two
# parts more: lost_weights() with no scale below 2^-90 (the weights are relative to the largest of
# p_j max(s_j, 2^-90)); and the logarithms, numbers below 2^8 here: six roundings of 2^-17 on the
# way to a weight or to the log-sum-exp, 2^-14 in all, which the 2^-10 A for the value scales holds,
# and with which the log-sum-exp's 2^-13 stays below 2^-12.


def scale_case(rng, Hkv, D, page, n, exponents):
    """A cache of one sequence whose blocks' value scales take the exponents in turn (None: 0)."""
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    for i, pos in enumerate(range(0, n, 32)):
        pg, blk = c.at(table[0], pos)
        e = exponents[i % len(exponents)]
        if e is None:
            k, v = (x.copy() for x in c.block_codes(pg, blk))
            c.set_block_codes(pg, blk, k, np.zeros_like(v))
            c.v_scale[pg, :, blk] = 0.0
        else:
            c.v_scale[pg, :, blk] = np.float32(1.3 * 2.0 ** e)
    return table, c


def check_scales(rng, c, table, n, T, H, D, causal):
    q = bf16(rng, 1, T, H, D)
    sm = 1 / math.sqrt(D)
    out, lse = sage.cache_attention(q, upload(c), ints(table), ints([n]), is_causal=causal, return_lse=True)
    ref_o, ref_lse, weight = oc.attention(c, f32(q), table, [n], [T], causal, sm)
    floor = c.v_scale.copy()
    c.v_scale[:] = np.maximum(c.v_scale, np.float32(2.0 ** -90))
    lost = lost_weights(c, f32(q), table, [n], [T], sm)
    c.v_scale[:] = floor
    o = f32(out).astype(np.float64)
    tol = 2.0 ** -8 * np.abs(ref_o) + 2.0 ** -9 * weight + lost
    bad = ~(np.abs(o - ref_o) <= tol)
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:4].tolist(), o[bad][:4], ref_o[bad][:4])
    err = np.abs(f32(lse).astype(np.float64) - ref_lse)
    assert err.max() <= 2.0 ** -12, err.max()


SCALES = [
    [None, 40],                    # blocks of zeros beside large values
    [100, 40, None],               # the largest seen first
    [-60, 70, -60, -60],
    [-120, 119, 0],
    [-100, -95],                   # small values alone
    [-88, None, 2, 120],
]


@pytest.mark.parametrize("exponents", SCALES)
@pytest.mark.parametrize("n,T,H,Hkv,D", [
    (300, 1, 4, 2, 128), (300, 20, 2, 2, 64), (5000, 2, 4, 1, 128), (9000, 5, 4, 1, 64),
    (700, 40, 2, 2, 64), (3000, 40, 4, 2, 128), (700, 300, 2, 2, 64), (1500, 300, 1, 1, 128),
])
def test_attention_value_scales_of_the_whole_range(n, T, H, Hkv, D, exponents):
    rng = np.random.default_rng(41)
    table, c = scale_case(rng, Hkv, D, 64, n, exponents)
    check_scales(rng, c, table, n, T, H, D, False)
    check_scales(rng, c, table, n, T, H, D, True)


@pytest.mark.parametrize("n,T,H,Hkv,D", [(300, 1, 4, 2, 128), (9000, 5, 4, 1, 64), (3000, 40, 4, 2, 128), (1500, 300, 1, 1, 64)])
def test_attention_large_values_met_last(n, T, H, Hkv, D):
    """All but the last blocks are zeros or small; what they hold of the sum is joined across warps and CTAs."""
    rng = np.random.default_rng(42)
    blocks = -(-n // 32)
    for head, tail in (([None], 110), ([-80], 115), ([-119], 60)):
        table, c = scale_case(rng, Hkv, D, 32, n, head * (blocks - 2) + [tail, tail])
        check_scales(rng, c, table, n, T, H, D, False)


@pytest.mark.parametrize("n,T,H,Hkv,D", [(300, 1, 4, 2, 128), (9000, 5, 4, 1, 64), (6000, 40, 4, 2, 128), (4600, 300, 1, 1, 128),
                                         (4600, 300, 1, 1, 64)])
def test_attention_large_values_met_first(n, T, H, Hkv, D):
    """Ordinary, small and no values behind large ones, over more tiles than are looked up at a time."""
    rng = np.random.default_rng(43)
    blocks = -(-n // 32)
    for head, tail in ((119, [0]), (119, [19]), (30, [-70]), (21, [-31, -32]), (110, [None])):
        table, c = scale_case(rng, Hkv, D, 32, n, [head, head] + tail * blocks)
        check_scales(rng, c, table, n, T, H, D, True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,T,H,Hkv", [(660, 1, 4, 2), (660, 20, 1, 1), (660, 40, 2, 1), (660, 300, 1, 1), (5140, 300, 2, 1)])
def test_attention_large_values_beside_the_last_block(n, T, H, Hkv, D):
    """Every other block's values are large; the last block, alone in its key tile, is none of them."""
    rng = np.random.default_rng(46)
    for exponents in ([-30, 110], [-10, 119], [0, 100]):
        table, c = scale_case(rng, Hkv, D, 64, n, exponents)
        check_scales(rng, c, table, n, T, H, D, False)
        check_scales(rng, c, table, n, T, H, D, True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,T", [(3000, 1), (3000, 2), (3000, 8), (40, 1), (300, 3), (3000, 40)])
def test_attention_empty_and_sparse_channels_exactly(n, T, D):
    """Channels without codes come out as 0, and one code of 1 among many keys as what it is: the bound
    of the module holds for every channel, whatever the others hold."""
    rng = np.random.default_rng(44)
    H, Hkv, page = 4, 1, 64
    table, P = make_table(rng, [n], page)
    c = random_cache(rng, P, Hkv, D, page)
    c.v_codes[:, :, :, D // 2:] = 0
    pg, blk = c.at(table[0], n // 2)
    c.v_codes[pg, 0, blk, D // 2, oc.POSITIONS[n // 2 % 32]] = 1
    q = bf16(rng, 1, T, H, D)
    out, lse = sage.cache_attention(q, upload(c), ints(table), ints([n]), return_lse=True)
    ref = oc.attention(c, f32(q), table, [n], [T], False, 1 / math.sqrt(D))
    # a weight below 2^-14 of the largest is rounded to a multiple of 2^-24, as lost_weights() has it, here once
    one = np.zeros(D)
    one[D // 2] = 1.0 / (127 * n)
    close(out, lse, *ref, lost_weights(c, f32(q), table, [n], [T], 1 / math.sqrt(D)) * one)
    assert (out[..., D // 2 + 1:] == 0).all() and (out[..., D // 2] != 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,Hkv,n", [(1, 1, 20050), (1, 1, 20114), (40, 4, 1100), (40, 4, 1164)])
def test_attention_nan_in_folded_parts(B, Hkv, n, D):
    """33 to 128 rows over parts that both halves of a CTA share: a block of NaN at the end of the
    sequence, in a key tile of the one half or the other, reaches the rows that see it and no others."""
    rng = np.random.default_rng(45)
    G, page, T = 4, 64, 30
    lengths = [n] * B
    table, P = make_table(rng, lengths, page)
    c = random_cache(rng, P, Hkv, D, page)
    gpu = upload(c)
    q, t, lens = bf16(rng, B, T, G * Hkv, D), ints(table), ints(lengths)
    clean, clean_lse = sage.cache_attention(q, gpu, t, lens, is_causal=True, return_lse=True)
    pg, blk = c.at(table[0], n - 1)
    seen = (n - 1) // 32 * 32 - (n - T)          # the first row that sees a token of the last block
    assert 0 < seen < T
    head = Hkv - 1                               # of sequence 0
    mine = slice(head * G, head * G + G)
    for scale in (gpu.k_scale, gpu.v_scale):
        was = scale[pg, head, blk].clone()
        scale[pg, head, blk] = float("nan")
        out, lse = sage.cache_attention(q, gpu, t, lens, is_causal=True, return_lse=True)
        scale[pg, head, blk] = was
        assert torch.isnan(out[0, seen:, mine].float()).all()
        assert torch.equal(out[0, :seen, mine], clean[0, :seen, mine])
        assert torch.equal(lse[0, mine, :seen], clean_lse[0, mine, :seen])
        out[0, :, mine] = clean[0, :, mine]
        assert torch.equal(out, clean)
    # in a block that all rows see, behind a value scale that makes the tiles odd ones
    for pos in (64, 640):
        pg1, blk1 = c.at(table[0], pos)
        pg2, blk2 = c.at(table[0], pos + 64)
        gpu.v_scale[pg1, head, blk1] *= 2.0 ** 30
        for scale in (gpu.k_scale, gpu.v_scale):
            was = scale[pg2, head, blk2].clone()
            scale[pg2, head, blk2] = float("nan")
            out = sage.cache_attention(q, gpu, t, lens, is_causal=True)
            scale[pg2, head, blk2] = was
            assert torch.isnan(out[0, :, mine].float()).all()
            out[0, :, mine] = clean[0, :, mine]
            assert torch.equal(out, clean)
