"""Rotary positions, prompt attention, weights of cached tokens and eviction without a GPU: formulas that run on
the host, the C ABI's refusals, none of which launches anything, and the Python binding's."""

import ctypes
import math
import shutil
import subprocess
from fractions import Fraction

import pytest
import torch

import quantized_attention_fp64_gb300 as sage
from quantized_attention_fp64_gb300 import _build, _lib
from quantized_attention_fp64_gb300.api import SageError
from test_cache_host import BAD_CACHES, _addr, _cache, _tab

OK, HEAD_DIM, SHAPE, LAYOUT, ALIGN, NULLPTR, WORKSPACE = 0, -4, -5, -6, -7, -8, -9
ARG, TOO_LARGE = -13, -14
PI = Fraction("3.14159265358979323846264338327950288419716939937510")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


def tensor(ptr=0x70000, sb=1 << 20, ss=512, sh=128):
    return _lib.Bf16Tensor(ptr, sb, ss, sh)


def bad_tensors():
    return [(tensor(0), NULLPTR), (tensor(0x70008), ALIGN), (tensor(sb=4), ALIGN), (tensor(ss=516), ALIGN),
            (tensor(sh=132), ALIGN)]


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    for struct, name in ((_lib.RotaryArgs, "sage_rotary_args"), (_lib.PromptAttentionArgs, "sage_prompt_attention_args"),
                         (_lib.CacheAddWeightsArgs, "sage_cache_add_weights_args"),
                         (_lib.CacheEvictArgs, "sage_cache_evict_args")):
        fields = [f[0] for f in struct._fields_]
        src = tmp_path / f"{name}.c"
        src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "sage.h"\nint main(void) {\n'
                       f'  printf("%zu\\n", sizeof({name}));\n'
                       + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
        exe = tmp_path / name
        subprocess.run([cc, "-std=c99", "-I", str(_build.ROOT) + "/include", str(src), "-o", str(exe)], check=True)
        got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
        assert got == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


# ------------------------------------------------------------------- rotary --


def turns_of(lib, freqs):
    n = len(freqs)
    got = (ctypes.c_uint64 * max(n, 1))()
    assert lib.sage_rotary_turns((ctypes.c_double * max(n, 1))(*freqs), n, got) == OK
    return list(got)[:n]


def test_turns_are_the_part_of_a_turn(lib):
    freqs = [1.0, 0.1, 2.0 ** -40, 1e-12, 0.0, 7.0, 1000.5, -1.0, -1e-6, 6.283185307179586, 3.141592653589793, 1e300, -0.0]
    for f, got in zip(freqs, turns_of(lib, freqs)):
        if abs(f) > 1e16:
            assert 0 <= got < 2 ** 64
            continue
        want = Fraction(f) / (2 * PI)
        # the factor 1 / (2 pi) and the product are off by 2^-53 of the value each, the cut by a unit, and the
        # difference to the whole part below the value by 2^-53 of 1
        bound = abs(want) * Fraction(2, 2 ** 53) + Fraction(1, 2 ** 64) + (Fraction(1, 2 ** 53) if f < 0 else 0)
        off = (Fraction(got, 2 ** 64) - want) % 1
        assert min(off, 1 - off) <= bound, (f, got)


def test_turns_refuse(lib):
    d, u = (ctypes.c_double * 2)(1.0, 2.0), (ctypes.c_uint64 * 2)(7, 7)
    assert lib.sage_rotary_turns(d, -1, u) == SHAPE
    assert lib.sage_rotary_turns(None, 2, u) == NULLPTR and lib.sage_rotary_turns(d, 2, None) == NULLPTR
    assert lib.sage_rotary_turns(None, 0, None) == OK
    for bad in (math.nan, math.inf, -math.inf):
        assert lib.sage_rotary_turns((ctypes.c_double * 2)(1.0, bad), 2, u) == ARG
        assert list(u) == [7, 7]


def test_frequencies_follow_their_formulas():
    for dim, base in ((128, 10000.0), (16, 500000.0), (2, 7.0)):
        w = sage.rotary_inv_freq(dim, base)
        assert w.dtype == torch.float64 and w.tolist() == pytest.approx([base ** (-2 * i / dim) for i in range(dim // 2)],
                                                                        rel=1e-14)
        assert torch.equal(sage.rotary_inv_freq(dim, base, "linear", 4.0), w / 4)
    w = sage.rotary_inv_freq(64)
    n = sage.rotary_inv_freq(64, scaling="ntk", factor=8.0)
    assert n[0] == 1 and n[-1].item() == pytest.approx(w[-1].item() / 8, rel=1e-13) and (n[1:] < w[1:]).all()
    y = sage.rotary_inv_freq(128, scaling="yarn", factor=4.0, original_length=4096)
    w = sage.rotary_inv_freq(128)
    turned = w * 4096 / (2 * math.pi)
    part = w / y
    assert part[turned >= 33].tolist() == pytest.approx([1.0] * int((turned >= 33).sum()), rel=1e-14)
    assert part[turned <= 0.8].tolist() == pytest.approx([4.0] * int((turned <= 0.8).sum()), rel=1e-14)
    assert (part[1:] >= part[:-1] - 1e-14).all() and (part >= 1 - 1e-14).all() and (part <= 4 + 1e-14).all()
    between = (part > 1.001) & (part < 3.999)
    mix = ((w - y) / (w - w / 4))[between]                # the blend is linear in the pair's number
    assert len(mix) > 4 and torch.allclose(mix[1:] - mix[:-1], (mix[1] - mix[0]).expand(len(mix) - 1), rtol=1e-9)


@pytest.mark.parametrize("args", [
    dict(rotary_dim=0), dict(rotary_dim=-2), dict(rotary_dim=7), dict(base=0.0), dict(base=math.nan), dict(factor=0.0),
    dict(scaling="other"), dict(factor=2.0), dict(scaling="ntk", rotary_dim=2), dict(scaling="yarn"),
    dict(scaling="yarn", original_length=0), dict(scaling="yarn", original_length=10, base=1.0),
    dict(scaling="yarn", original_length=10, fast_turns=1.0, slow_turns=2.0)])
def test_frequencies_refuse(args):
    with pytest.raises(SageError) as e:
        sage.rotary_inv_freq(**{**dict(rotary_dim=64), **args})
    assert e.value.code == ARG


@pytest.mark.parametrize("args,code", [
    (dict(), ARG), (dict(rotary_dim=24), ARG), (dict(inv_freq=[1.0] * 8, rotary_dim=8), SHAPE), (dict(inv_freq=[]), ARG),
    (dict(inv_freq=[[1.0] * 8]), SHAPE), (dict(inv_freq=[1.0] * 8, factor=2.0), ARG), (dict(inv_freq=[math.inf] * 8), ARG),
    (dict(rotary_dim=64, magnitude=math.nan), ARG)])
def test_tables_refuse(lib, args, code):
    with pytest.raises(SageError) as e:
        sage.rotary_table(device="cpu", **args)
    assert e.value.code == code


def test_tables_live_on_a_device(lib):
    with pytest.raises(ValueError):
        sage.rotary_table(64, device="cpu")


def _rotary(lib, q=None, k=None, qo=None, ko=None, B=2, T=3, H=4, Hkv=2, D=128, rot=64, turns=0x1000, pos=0x2000, mag=1.0):
    t = tensor()
    return lib.sage_rotary(_lib.RotaryArgs(q or t, k or t, qo or t, ko or t, B, T, H, Hkv, D, rot, turns, pos, 3, 1, mag, 0,
                                           0, None))


def test_rotary_refuses(lib):
    assert lib.sage_rotary(None) == NULLPTR
    for name in ("B", "T", "H", "Hkv", "D"):
        assert _rotary(lib, **{name: -1}) == SHAPE
    assert _rotary(lib, D=96) == HEAD_DIM and _rotary(lib, D=0) == HEAD_DIM
    for rot in (0, -16, 24, 144):
        assert _rotary(lib, rot=rot) == ARG
    assert _rotary(lib, D=64, rot=80) == ARG
    for mag in (math.nan, math.inf):
        assert _rotary(lib, mag=mag) == ARG
    assert _rotary(lib, H=65536) == TOO_LARGE and _rotary(lib, Hkv=65536) == TOO_LARGE
    assert _rotary(lib, T=(1 << 30) + 1) == TOO_LARGE and _rotary(lib, B=1 << 16, T=1 << 15) == TOO_LARGE
    for which in ("q", "k", "qo", "ko"):
        for bad, code in bad_tensors():
            assert _rotary(lib, **{which: bad}) == code, (which, code)
    assert _rotary(lib, turns=None) == NULLPTR and _rotary(lib, pos=None) == NULLPTR
    assert _rotary(lib, turns=0x1008) == ALIGN and _rotary(lib, pos=0x2002) == ALIGN


def test_rotary_refuses_outputs_that_meet(lib):
    """Rows of an output over each other, other rows at an input's address, one output for both."""
    a, b, c = (lambda **kw: tensor(0x70000, **kw)), (lambda **kw: tensor(0x80000, **kw)), (lambda **kw: tensor(0x90000, **kw))  # noqa: E731
    d = lambda **kw: tensor(0xa0000, **kw)  # noqa: E731
    meet = [dict(ss=0), dict(sh=0), dict(sb=0), dict(sh=64), dict(ss=256), dict(sb=512), dict(sb=1024), dict(ss=-256), dict(sh=128, ss=384),
            dict(sh=4096, ss=512, sb=1024), dict(sb=-(1 << 63))]
    for st in meet[:-1]:
        assert _rotary(lib, q=a(), k=b(), qo=c(**st), ko=d()) == LAYOUT, st
    for st in (dict(ss=0), dict(sh=0), dict(sb=0), dict(sh=64), dict(ss=128)):
        assert _rotary(lib, q=a(), k=b(), qo=c(), ko=d(**st)) == LAYOUT, st
        assert _rotary(lib, q=a(**st), k=b(), qo=a(**st), ko=d()) == LAYOUT, st
    for st in (dict(sb=1 << 21), dict(ss=1024), dict(sh=1 << 12)):
        assert _rotary(lib, q=a(), k=b(), qo=a(**st), ko=d()) == LAYOUT, st
        assert _rotary(lib, q=a(), k=b(), qo=c(), ko=b(**st)) == LAYOUT, st
    assert _rotary(lib, q=a(), k=b(), qo=c(), ko=c()) == ARG
    assert _rotary(lib, q=a(), k=b(), qo=b(), ko=d()) == ARG and _rotary(lib, q=a(), k=b(), qo=c(), ko=a()) == ARG
    # what does not meet is taken: the next check that fails is that of the device, or none
    fine = [dict(), dict(ss=1 << 12, sh=128), dict(sh=1 << 12, ss=128, sb=1 << 16), dict(ss=-512), dict(sh=-128, sb=-(1 << 20)), meet[-1]]
    if not torch.cuda.is_available():
        for st in fine:
            assert _rotary(lib, q=a(), k=b(), qo=c(**st), ko=d()) not in (LAYOUT, ARG), st
        assert _rotary(lib, q=a(), k=b(), qo=a(), ko=b()) not in (LAYOUT, ARG)
        assert _rotary(lib, q=a(), k=a(), qo=c(), ko=d()) not in (LAYOUT, ARG)
        assert _rotary(lib, q=a(), k=b(), qo=c(sb=0), ko=d(sb=0), B=1) not in (LAYOUT, ARG)
        assert _rotary(lib, q=a(), k=b(), qo=a(sb=8, ss=0), ko=d(), B=1, T=1) not in (LAYOUT, ARG)


# --------------------------------------------------------- prompt attention --


def _prompt(lib, q=None, k=None, v=None, out=None, N=100, M=100, H=4, Hkv=2, D=128, B=3, off=0x1000, kv=None, sm=0.1, lse=None,
            ws=0x90000, wsn=1 << 40):
    t = tensor()
    return lib.sage_prompt_attention(_lib.PromptAttentionArgs(q or t, k or t, v or t, out or tensor(0x80000), N, M, H, Hkv, D, B, off, kv,
                                                              sm, 1, 1, lse, ws, wsn, None))


def test_prompt_attention_refuses(lib):
    assert lib.sage_prompt_attention(None) == NULLPTR
    n = ctypes.c_size_t(0)
    size = lambda N=100, M=100, H=4, Hkv=2, D=128, B=3: lib.sage_prompt_attention_workspace_size(  # noqa: E731
        N, M, H, Hkv, D, B, ctypes.byref(n))
    assert lib.sage_prompt_attention_workspace_size(100, 100, 4, 2, 128, 3, None) == NULLPTR
    assert size() == OK and n.value > 0
    need = n.value
    for f in (size, lambda **kw: _prompt(lib, **kw)):
        for name in ("N", "M", "H", "Hkv", "D", "B"):
            assert f(**{name: -1}) == SHAPE
        assert f(D=96) == HEAD_DIM and f(H=3) == SHAPE and f(Hkv=0) == SHAPE and f(Hkv=8) == SHAPE
        for name in ("N", "M"):
            assert f(**{name: (1 << 30) + 1}) == TOO_LARGE
        assert f(H=65536) == TOO_LARGE and f(B=65536) == TOO_LARGE
        assert f(N=1 << 30, H=65534) == TOO_LARGE      # blocks of rows of all heads are counted in 32 bits
    assert size(H=0, Hkv=0) == OK and n.value == 0 and size(N=0) == OK and n.value == 0
    for which in ("q", "k", "v", "out"):
        for bad, code in bad_tensors():
            assert _prompt(lib, **{which: bad}) == code, (which, code)
    for which in ("q", "k", "v"):  # expanded rows or heads, and backward ones
        for st in (dict(ss=0), dict(sh=0), dict(ss=-512), dict(sh=-128), dict(ss=1 << 39)):
            assert _prompt(lib, **{which: tensor(**st)}) == LAYOUT
    assert _prompt(lib, out=tensor()) == ARG and _prompt(lib, q=tensor(0x80000)) == ARG and _prompt(lib, v=tensor(0x80000)) == ARG
    assert _prompt(lib, off=None) == NULLPTR and _prompt(lib, off=0x1002) == ALIGN and _prompt(lib, kv=0x1001) == ALIGN
    assert _prompt(lib, lse=0x1002) == ALIGN
    for sm in (0.0, -1.0, math.inf):
        assert _prompt(lib, sm=sm) == ARG
    assert _prompt(lib, ws=None) == NULLPTR and _prompt(lib, ws=0x90010) == ALIGN
    assert _prompt(lib, wsn=need - 1) == WORKSPACE


def test_prompt_attention_refuses_outputs_over_each_other(lib):
    for st in (dict(ss=0), dict(sh=0), dict(ss=384), dict(sh=64), dict(ss=64), dict(ss=-384), dict(sh=512, ss=1024)):
        assert _prompt(lib, out=tensor(0x80000, **st)) == LAYOUT, st
    if not torch.cuda.is_available():
        for st in (dict(), dict(sb=0), dict(ss=-512), dict(ss=128, sh=1 << 14), dict(ss=520), dict(sh=136, ss=544)):
            assert _prompt(lib, out=tensor(0x80000, **st)) not in (LAYOUT, ARG), st
        assert _prompt(lib, out=tensor(0x80000, ss=0), N=1) not in (LAYOUT, ARG)
        assert _prompt(lib, out=tensor(0x80000, sh=0), H=1, Hkv=1) not in (LAYOUT, ARG)


# ------------------------------------------------------ weights and eviction --


def _weights(lib, cache=None, table=None, starts=0x60000, counts=None, q=None, lse=0x80000, scores=0xa0000, sb=4000, sh=1000,
             n=1000, B=2, T=4, H=4, sm=0.1):
    cache = cache or _cache()
    return lib.sage_cache_add_weights(_lib.CacheAddWeightsArgs(_addr(cache), *(table or _tab()), starts, counts, q or tensor(),
                                                               B, T, H, sm, 1, lse, scores, sb, sh, n, None))


def _evict(lib, cache=None, table=None, out=None, starts=0x60000, scores=0xa0000, n=1000, B=2, keep=100, recent=10,
           lens=0xb0000, kept=0xc0000, kept_size=100, moved=0xd0000, ws=0x90000, wsn=1 << 40):
    cache = cache or _cache()
    return lib.sage_cache_evict(_lib.CacheEvictArgs(_addr(cache), *(table or _tab()), *(out or _tab()), starts, scores, 4000,
                                                    1000, n, B, keep, recent, lens, kept, kept_size, moved, ws, wsn, None))


@pytest.mark.parametrize("call", [_weights, _evict])
def test_refusals_shared_with_the_token_entries(lib, call):
    for over, code in BAD_CACHES:
        assert call(lib, cache=_cache(**over)) == code, over
    for which in ("table",) + (("out",) if call is _evict else ()):
        assert call(lib, **{which: _tab(ptr=0)}) == NULLPTR
        assert call(lib, **{which: _tab(ptr=0x50002)}) == ALIGN
        assert call(lib, **{which: _tab(n=-1)}) == SHAPE
        assert call(lib, **{which: _tab(stride=-4)}) == SHAPE
    assert call(lib, starts=None) == NULLPTR and call(lib, starts=0x60002) == ALIGN
    assert call(lib, scores=None) == NULLPTR and call(lib, scores=0xa0002) == ALIGN
    assert call(lib, n=-1) == SHAPE and call(lib, B=-1) == SHAPE and call(lib, B=1 << 16) == TOO_LARGE


def test_weights_refuse(lib):
    assert lib.sage_cache_add_weights(None) == NULLPTR
    assert _weights(lib, counts=0x60001) == ALIGN
    assert _weights(lib, T=-1) == SHAPE and _weights(lib, H=3) == SHAPE and _weights(lib, H=-2) == SHAPE
    assert _weights(lib, T=(1 << 30) + 1) == TOO_LARGE and _weights(lib, H=70000) == TOO_LARGE
    assert _weights(lib, B=60000, table=_tab(n=1 << 20), sb=1 << 30) == TOO_LARGE
    assert _weights(lib, lse=None) == NULLPTR and _weights(lib, lse=0x80001) == ALIGN
    for sm in (0.0, -1.0, math.inf):
        assert _weights(lib, sm=sm) == ARG
    for bad, code in bad_tensors():
        assert _weights(lib, q=bad) == code
    for st in (dict(sb=0), dict(ss=0), dict(sh=0), dict(sb=-1024), dict(ss=-512), dict(sh=-128), dict(sh=1 << 40)):
        assert _weights(lib, q=tensor(**st)) == LAYOUT
    # rows of scores that overlap would be added to by two blocks at once
    for st in (dict(sb=0), dict(sh=0), dict(sh=999), dict(sb=999), dict(sb=1999, sh=1000), dict(sb=1000, sh=1999),
               dict(sb=-1000, sh=1000)):
        assert _weights(lib, **st) == LAYOUT, st


def test_eviction_refuses(lib):
    assert lib.sage_cache_evict(None) == NULLPTR
    n = ctypes.c_size_t(0)
    size = lambda B=2, H=2, D=128, keep=100, S=1000, to=ctypes.byref(n): lib.sage_cache_evict_workspace_size(  # noqa: E731
        B, H, D, keep, S, to)
    assert size() == OK and n.value > 0
    need = n.value
    assert size(to=None) == NULLPTR and size(D=96) == HEAD_DIM and size(B=1 << 16) == TOO_LARGE
    assert size(H=1 << 16) == TOO_LARGE and size(S=(1 << 30) + 1) == TOO_LARGE
    for name in ("B", "H", "keep", "S"):
        assert size(**{name: -1}) == SHAPE
    assert size(keep=1 << 60) == OK
    assert _evict(lib, keep=-1) == SHAPE and _evict(lib, recent=-1) == SHAPE and _evict(lib, recent=101) == SHAPE
    assert _evict(lib, kept_size=99) == SHAPE and _evict(lib, n=(1 << 30) + 1) == TOO_LARGE
    for name in ("lens", "kept", "moved"):
        assert _evict(lib, **{name: None}) == NULLPTR and _evict(lib, **{name: 0xb0002}) == ALIGN
    assert _evict(lib, lens=0x60000) == ARG and _evict(lib, moved=0xa0000) == ARG
    assert _evict(lib, ws=None) == NULLPTR and _evict(lib, ws=0x90010) == ALIGN
    assert _evict(lib, wsn=need - 1) == WORKSPACE


def test_eviction_refuses_other_rows_at_the_table_s_address(lib):
    """Cutting back in place has to be known as that: rows that begin where the table's do are the table's rows."""
    far = lambda stride, n=4: _tab(stride=stride, n=n)  # noqa: E731
    for stride in (0, 4, 6, 16):
        assert _evict(lib, table=far(8), out=far(stride)) == ARG
        assert _evict(lib, table=far(8), out=far(stride, n=2)) == ARG


# ----------------------------------------------------------- Python binding --


def test_host_tensors_are_refused(lib):
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        sage.prompt_attention(x, x, x, off)
    for f in (lambda: sage.rotary(x, x, off, None), lambda: sage.cache_add_weights(x, x, None, off, off, x),
              lambda: sage.cache_evict(None, off, off, x, 5), lambda: sage.prompt_attention(None, x, x, off)):
        with pytest.raises(TypeError):
            f()
    for f in (lambda: sage.prompt_attention_workspace_size(10, 10, 3, 2), lambda: sage.cache_evict_workspace_size(1, 1, 64, -1, 5)):
        with pytest.raises(SageError) as e:
            f()
        assert e.value.code == SHAPE


def test_codes_have_texts(lib):
    texts = [lib.sage_strerror(c) for c in (-16, -17)]
    assert b"page" in texts[0] and b"offsets" in texts[1]
