"""Rotary positions on the GPU against the formula in float64.

An output differs from magnitude (a cos - b sin) by at most half a step of bf16, 2^-8 of itself, and the error of
the sine and cosine, 2^-20 of |a| + |b| (2^-21.4 of the fast functions within half a turn, 2^-24 pi of the angle's
rounding, roundings of the products).
"""

import math

import pytest
import torch

import quantized_attention_fp64_gb300 as sage
from quantized_attention_fp64_gb300.api import SageError

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _library(sage_lib):
    yield
    torch.cuda.synchronize()
    assert sage.device_error() == 0


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def formula(x, positions, table, interleaved, sign=1):
    """(turned, bound) in float64 of x [B, T, H, D] with positions [B, T]."""
    rot, f = table.rotary_dim, table.magnitude
    w = table.inv_freq.cuda()
    # the angle modulo a turn, exactly: positions below 2^31 times 53 bits leave float64, so in two parts
    p = positions.to(torch.int64)
    hi, lo = (p >> 16).double() * 65536.0, (p & 0xFFFF).double()
    angle = (torch.remainder(hi[..., None] * w, 2 * math.pi) + torch.remainder(lo[..., None] * w, 2 * math.pi))[:, :, None]
    c, s = torch.cos(angle) * f, torch.sin(angle) * f * sign
    y = x.double().clone()
    a, b = (y[..., :rot:2].clone(), y[..., 1:rot:2].clone()) if interleaved else (y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone())
    first, second = a * c - b * s, b * c + a * s
    size = torch.zeros_like(y)
    if interleaved:
        y[..., :rot:2], y[..., 1:rot:2] = first, second
        size[..., :rot:2] = size[..., 1:rot:2] = a.abs() + b.abs()
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = first, second
        size[..., :rot // 2] = size[..., rot // 2:rot] = a.abs() + b.abs()
    bound = y.abs() * 2.0 ** -8 + size * abs(f) * 2.0 ** -20
    bound[..., rot:] = 0
    return y, bound


def close(got, ref):
    y, bound = ref
    assert not torch.isnan(got).any()
    assert ((got.double() - y).abs() <= bound).all(), float(((got.double() - y).abs() / (bound + 1e-30)).max())


CASES = [
    # B, T, H, Hkv, D, rotary_dim, interleaved
    (1, 1, 1, 1, 128, 128, False), (1, 1, 1, 1, 64, 64, True), (64, 1, 32, 8, 128, 128, False), (3, 7, 5, 1, 64, 16, False),
    (2, 33, 8, 8, 128, 48, True), (1, 1000, 28, 4, 128, 64, False), (2, 301, 3, 2, 64, 32, True), (5, 2, 40, 40, 128, 128, True),
    (1, 3, 200, 1, 64, 48, False), (1, 2500, 4, 4, 64, 64, False),
]


@pytest.mark.parametrize("far", [0, 1000, 131071, 2 ** 31 - 3000])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_rotary(case, far):
    B, T, H, Hkv, D, rot, interleaved = CASES[case]
    g = gen(case)
    q, k = bf16(g, B, T, H, D), bf16(g, B, T, Hkv, D)
    pos = (far + torch.arange(T, device="cuda") + torch.arange(B, device="cuda")[:, None] * 3).to(torch.int32)
    table = sage.rotary_table(rot, device="cuda")
    before = q.clone(), k.clone()
    qo, ko = sage.rotary(q, k, pos, table, interleaved=interleaved)
    assert torch.equal(q, before[0]) and torch.equal(k, before[1])
    close(qo, formula(q, pos, table, interleaved))
    close(ko, formula(k, pos, table, interleaved))
    assert torch.equal(qo[..., rot:], q[..., rot:])
    # without k; in HND; in place: the same bits
    assert torch.equal(sage.rotary(q, None, pos, table, interleaved=interleaved), qo)
    hq, hk = sage.rotary(q.transpose(1, 2).contiguous(), k.transpose(1, 2).contiguous(), pos, table, interleaved=interleaved,
                         tensor_layout="HND")
    assert torch.equal(hq.transpose(1, 2), qo) and torch.equal(hk.transpose(1, 2), ko)
    got = sage.rotary(q, k, pos, table, interleaved=interleaved, out=(q, k))
    assert got[0] is q and torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("kw", [
    dict(base=500000.0), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
    dict(scaling="yarn", factor=4.0, original_length=4096), dict(scaling="yarn", factor=32.0, original_length=8192, base=1e6),
    dict(inv_freq=[3.0, 0.0, -1.5, 100.25, 1e-9, 2 * math.pi, 0.1, 7.0], magnitude=0.5)])
def test_frequencies(kw):
    g = gen(20)
    table = sage.rotary_table(**({} if "inv_freq" in kw else dict(rotary_dim=64)), device="cuda", **kw)
    q, k = bf16(g, 2, 50, 4, 64), bf16(g, 2, 50, 2, 64)
    pos = torch.randint(-2 ** 20, 2 ** 20, (2, 50), device="cuda").to(torch.int32)
    qo, ko = sage.rotary(q, k, pos, table)
    close(qo, formula(q, pos, table, False))
    close(ko, formula(k, pos, table, False))


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_turns_back_and_is_the_gradient(interleaved):
    g = gen(21)
    table = sage.rotary_table(64, device="cuda", magnitude=1.25)
    x, y = bf16(g, 1, 40, 2, 128), bf16(g, 1, 40, 2, 128)
    pos = torch.arange(100000, 100040, device="cuda").to(torch.int32)
    pb = pos.expand(1, 40)
    forward = sage.rotary(x, None, pos, table, interleaved=interleaved)
    back = sage.rotary(y, None, pos, table, interleaved=interleaved, inverse=True)
    close(back, formula(y, pb, table, interleaved, sign=-1))
    negative = sage.rotary(y, None, -pos, table, interleaved=interleaved)
    assert torch.equal(negative, back)
    # <R x, y> = <x, R^T y>, and differences of the loss sum(R x * y)
    xx = x.double().requires_grad_()
    w = table.inv_freq.cuda()
    angle = pos.double()[:, None, None] * w
    c, s = torch.cos(angle) * 1.25, torch.sin(angle) * 1.25
    a, b = (xx[..., :64:2], xx[..., 1:64:2]) if interleaved else (xx[..., :32], xx[..., 32:64])
    ya, yb = (y[..., :64:2], y[..., 1:64:2]) if interleaved else (y[..., :32], y[..., 32:64])
    loss = ((a * c - b * s) * ya.double() + (b * c + a * s) * yb.double()).sum() + (xx[..., 64:] * y[..., 64:].double()).sum()
    loss.backward()
    assert ((back.double() - xx.grad).abs() <= xx.grad.abs() * 2.0 ** -8 + 2.0 ** -18 * 8).all()
    step = 2.0 ** -6
    for at in ((0, 3, 1, 5), (0, 39, 0, 40), (0, 0, 1, 100)):
        moved = x.double().clone()
        moved[at] += step
        diff = (formula(moved, pb, table, interleaved)[0] - formula(x, pb, table, interleaved)[0]) * y.double()
        assert abs(diff.sum().item() / step - back[at].item()) <= abs(back[at].item()) * 2.0 ** -8 + 1e-4
    assert not torch.isnan(forward).any()


def test_packed_strided_and_shared_positions():
    g = gen(22)
    table = sage.rotary_table(32, device="cuda")
    fused = bf16(g, 90, 12, 64)                       # one projection's queries, keys and values
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    pos = torch.arange(180, device="cuda").to(torch.int32)[::2]
    want = formula(q[None], pos[None], table, False), formula(k[None], pos[None], table, False)
    values = v.clone()
    qo, ko = sage.rotary(q, k, pos, table)
    close(qo[None], want[0])
    close(ko[None], want[1])
    sage.rotary(q, k, pos, table, out=(q, k))
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(v, values)
    # the same positions for every sequence, as a row and as an expanded tensor
    x, y = bf16(g, 3, 30, 4, 64), bf16(g, 3, 30, 1, 64)
    a = sage.rotary(x, y, pos[:30], table)
    b = sage.rotary(x, y, pos[:30].expand(3, 30), table)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    close(a[0], formula(x, pos[:30].expand(3, 30), table, False))


def test_infinities_and_nan_stay_in_their_pair():
    table = sage.rotary_table(64, device="cuda")
    x = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0, 3], x[0, 1, 0, 40] = math.inf, math.nan
    y = sage.rotary(x, None, torch.tensor([5, 9], dtype=torch.int32, device="cuda"), table)
    odd = ~torch.isfinite(y)
    assert sorted(map(tuple, torch.nonzero(odd).tolist())) == [(0, 0, 0, 3), (0, 0, 0, 35), (0, 1, 0, 8), (0, 1, 0, 40)]


def test_refusals_and_empty_calls():
    g = gen(23)
    table = sage.rotary_table(64, device="cuda")
    q, k = bf16(g, 2, 5, 4, 64), bf16(g, 2, 5, 2, 64)
    pos = torch.zeros((2, 5), dtype=torch.int32, device="cuda")
    good = dict(q=q, k=k, positions=pos, table=table)
    for change, code in [
        (dict(q=q.half()), -3), (dict(k=k.float()), -3), (dict(positions=pos.long()), -3), (dict(positions=pos[:1]), -5),
        (dict(positions=pos[:, :4]), -5), (dict(k=k[:, :4]), -5), (dict(k=k[0]), -5), (dict(q=q[0, 0], k=None), -5),
        (dict(tensor_layout="xyz"), -6), (dict(q=q.transpose(2, 3)), -6), (dict(table=sage.rotary_table(128, device="cuda")), -13),
        (dict(out=(q,)), -5), (dict(out=(k, k)), -5), (dict(q=bf16(g, 2, 5, 4, 65)[..., 1:]), -7),
        (dict(q=bf16(g, 2, 5, 4, 32), k=bf16(g, 2, 5, 2, 32), table=sage.rotary_table(32, device="cuda")), -4)]:
        with pytest.raises(SageError) as err:
            sage.rotary(**{**good, **change})
        assert err.value.code == code, (change.keys(), err.value)
    wide = bf16(g, 2, 5, 8, 64)
    with pytest.raises(SageError) as err:  # in its input's place, with other strides
        sage.rotary(wide[:, :, :4], k, pos, table, out=(wide.view(2, 5, 4, 128)[..., :64], torch.empty_like(k)))
    assert err.value.code == -6
    with pytest.raises(TypeError):
        sage.rotary(q, k, None, table)
    with pytest.raises(TypeError):
        sage.rotary(q, k, pos, None)
    with pytest.raises(ValueError):
        sage.rotary(q.cpu(), k, pos, table)
    qo, ko = sage.rotary(q[:, :0], k[:, :0], pos[:, :0], table)
    assert qo.shape == (2, 0, 4, 64) and ko.shape == (2, 0, 2, 64)
    qo, ko = sage.rotary(q[:, :, :0], k, pos, table)
    assert qo.shape == (2, 5, 0, 64) and torch.equal(ko, sage.rotary(k, None, pos, table))


def test_graph_replay_with_moving_positions():
    g = gen(24)
    table = sage.rotary_table(128, device="cuda")
    q, k = bf16(g, 4, 1, 8, 128), bf16(g, 4, 1, 2, 128)
    pos = torch.zeros((4, 1), dtype=torch.int32, device="cuda")
    sage.rotary(q, k, pos, table)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            qo, ko = sage.rotary(q, k, pos, table)
    for step in (0, 77, 100000):
        pos.fill_(step)
        graph.replay()
        torch.cuda.synchronize()
        close(qo, formula(q, pos, table, False))
        close(ko, formula(k, pos, table, False))


@pytest.mark.parametrize("layout", ["NHD", "HND"])
@pytest.mark.parametrize("packed", [False, True])
def test_repeated_calls_with_dense_views(packed, layout):
    """From the second call on a signature goes a shorter way."""
    B, T, H, Hkv, D = 1 if packed else 3, 37, 4, 2, 64
    table = sage.rotary_table(D, device="cuda")
    for call in range(4):
        g = gen(60 + call)
        q, k = ((bf16(g, B, h, T, D) if layout == "NHD" else bf16(g, B, T, h, D)).transpose(1, 2) for h in (H, Hkv))
        pos = torch.randint(0, 5000, (B, T), generator=g, device="cuda").to(torch.int32)
        args = (q[0], k[0], pos[0]) if packed else (q, k, pos)
        got = sage.rotary(*args, table, tensor_layout=layout)
        for x, y in zip((q, k), got):
            y = y[None] if packed else y
            assert y.shape == x.shape
            x, y = (x, y) if layout == "NHD" else (x.transpose(1, 2), y.transpose(1, 2))
            close(y, formula(x, pos, table, False))
