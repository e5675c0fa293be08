"""The 8-bit paged key/value cache without a GPU: the oracle against plain
formulas, the index arithmetic that the kernels use for lengths and pages from
device memory (compiled for the host), and the C ABI's refusals, none of which
launches anything."""

import ctypes
import math
import shutil
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle.sage_oracle import bf16_round
from quantized_attention_fp64_gb300 import _build, _lib, alloc_cache, cache, cache_append, cache_attention, cache_read
from quantized_attention_fp64_gb300.api import SageError

OK, DTYPE, HEAD_DIM, SHAPE, LAYOUT, ALIGN, NULLPTR, WORKSPACE = 0, -3, -4, -5, -6, -7, -8, -9
ARG, TOO_LARGE = -13, -14


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return _lib.load()


# ------------------------------------------------------------------- oracle --


@pytest.mark.parametrize("D", [64, 128])
def test_oracle_round_trip_is_within_half_a_step(D):
    rng = np.random.default_rng(5)
    c = oc.Cache(6, 2, D, 64)
    table = np.array([[3, 1, 5]])
    k, v = (bf16_round(rng.standard_normal((1, 150, 2, D)).astype(np.float32)) for _ in (0, 1))
    oc.append(c, k, v, table, [0], [150])
    kk, vv = c.tokens(table[0], 0, 150)
    for got, x, scale in ((kk, k, c.k_scale), (vv, v, c.v_scale)):
        for pos in range(150):
            page, blk = c.at(table[0], pos)
            # half a step, and the fp32 rounding of the scale and the quotient (2^-23 of at most 127 steps)
            step = scale[page, :, blk, None] * (0.5 + 127 * 2.0 ** -22)
            assert (np.abs(got[pos] - x[0, pos]) <= step).all()


def test_oracle_scale_grows_and_older_codes_follow():
    c = oc.Cache(1, 1, 64, 32)
    table = np.array([[0]])
    x = np.zeros((1, 3, 1, 64), np.float32)
    x[0, 0], x[0, 1], x[0, 2] = 1.0, 8.0, 2.0
    for t in range(3):
        oc.append(c, x[:, t:t + 1], x[:, t:t + 1], table, [t], [1])
    assert c.k_scale[0, 0, 0] == np.float32(8) / np.float32(127)
    k, v = c.block_codes(0, 0)
    assert k[:3, 0, 0].tolist() == [16, 127, 32] and v[:3, 0, 5].tolist() == [16, 127, 32]


def test_oracle_positions_are_a_permutation():
    assert sorted(oc.POSITIONS.tolist()) == list(range(32))
    for i in range(32):
        j, t, e = i // 8, (i % 8) // 2, i % 2
        assert oc.POSITIONS[8 * j + 2 * t + e] == 8 * t + 2 * j + e


def test_oracle_attention_against_a_direct_sum():
    rng = np.random.default_rng(6)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    o, lse, a = oc.attention_rows(q, k, v, [0, 2, 5], 0.3)
    assert (o[0] == 0).all() and lse[0] == -np.inf
    for r, n in ((1, 2), (2, 5)):
        w = np.exp([0.3 * float(q[r] @ k[j]) for j in range(n)])
        assert np.allclose(o[r], sum(w[j] * v[j] for j in range(n)) / w.sum(), atol=1e-14)
        assert abs(lse[r] - math.log(w.sum())) < 1e-13
        assert (a[r] >= np.abs(o[r]) - 1e-15).all()


# ---------------------------------------------------------- index arithmetic --


@pytest.fixture(scope="module")
def index_host(tmp_path_factory):
    exe = tmp_path_factory.mktemp("cache") / "index"
    src = str(_build.ROOT) + "/tests/helpers/cache_index_host.cu"
    subprocess.run([_build.nvcc_path(), "-std=c++17", src, "-o", str(exe)], check=True, capture_output=True)

    def ask(*lines):
        r = subprocess.run([str(exe)], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return [tuple(int(x) for x in line.split()) for line in r.stdout.splitlines()]

    return ask


def test_lengths_and_pages_from_device_memory_are_cut(index_host):
    assert index_host("length 5 10", "length 10 10", "length 11 10", "length -1 10", "length 0 0", "length 1 0",
                      "length -2147483648 10", "length 2147483647 100") == [
        (5, 0), (10, 0), (10, 1), (0, 1), (0, 0), (0, 1), (0, 1), (100, 1)]
    assert index_host("page 0 4", "page 3 4", "page 4 4", "page -1 4", "page 2147483647 4", "page -2147483648 4",
                      "page 0 0") == [(1,), (1,), (0,), (0,), (0,), (0,), (0,)]


def test_table_capacity_stays_in_32_bits(index_host):
    got = index_host("capacity 0 2", "capacity 10 2", "capacity 1 128", "capacity 67108864 1",
                     "capacity 9223372036854775807 1", "capacity 1099511627776 128")
    assert got[:3] == [(0,), (640,), (4096,)]
    for (n,), per in zip(got[3:], (32, 32, 4096)):
        assert n % per == 0 and 2 ** 31 - 32 - per < n <= 2 ** 31 - 32


def test_every_block_has_its_own_slot(index_host):
    P, H, n = 5, 3, 4
    lines = [f"slot {p} {h} {H} {n} {b}" for p in range(P) for h in range(H) for b in range(n)]
    assert sorted(x for (x,) in index_host(*lines)) == list(range(P * H * n))
    assert index_host("slot 1048575 65534 65535 128 127") == [((1 << 20) * 65535 * 128 - 1,)]


def test_value_positions_match_the_oracle(index_host):
    got = index_host(*[f"position {i}" for i in range(32)])
    assert [p for p, _ in got] == oc.POSITIONS.tolist() and [t for _, t in got] == list(range(32))


# --------------------------------------------------------------------- C ABI --


def _cache(**over):
    c = dict(k=0x10000, v=0x20000, ks=0x30000, vs=0x40000, P=8, page=64, H=2, D=128)
    c.update(over)
    return _lib.Cache(c["k"], c["v"], c["ks"], c["vs"], c["P"], c["page"], c["H"], c["D"])


def _tab(ptr=0x50000, stride=4, n=4):
    return ptr, stride, n


BAD_CACHES = [(dict(D=96), HEAD_DIM), (dict(page=48), SHAPE), (dict(page=0), SHAPE), (dict(H=-1), SHAPE),
              (dict(P=-1), SHAPE), (dict(page=8192), TOO_LARGE), (dict(P=(1 << 20) + 1), TOO_LARGE),
              (dict(H=70000), TOO_LARGE), (dict(k=0), NULLPTR), (dict(v=0x20008), ALIGN), (dict(ks=0x30004), ALIGN),
              (dict(vs=0), NULLPTR)]


def test_cache_size(lib):
    n, c = ctypes.c_size_t(0), _lib.Cache()
    assert lib.sage_cache_size(10, 64, 3, 128, ctypes.byref(n), ctypes.c_void_p(0x100000), ctypes.byref(c)) == OK
    codes = 10 * 3 * 64 * 128
    assert c.k_codes_dev == 0x100000 and c.v_codes_dev == 0x100000 + codes
    assert c.k_scale_dev == 0x100000 + 2 * codes and c.v_scale_dev == c.k_scale_dev + 256
    assert n.value == 2 * codes + 2 * 256 and (c.num_pages, c.page_size, c.H, c.D) == (10, 64, 3, 128)
    assert lib.sage_cache_size(10, 64, 3, 128, None, None, None) == NULLPTR
    assert lib.sage_cache_size(10, 64, 3, 128, ctypes.byref(n), ctypes.c_void_p(0x100000), None) == NULLPTR
    assert lib.sage_cache_size(10, 64, 3, 128, ctypes.byref(n), ctypes.c_void_p(0x100080), ctypes.byref(c)) == ALIGN
    for over, code in BAD_CACHES[:8]:
        a = dict(P=8, page=64, H=2, D=128)
        a.update(over)
        assert lib.sage_cache_size(a["P"], a["page"], a["H"], a["D"], ctypes.byref(n), None, None) == code


def _addr(struct):
    return ctypes.cast(ctypes.pointer(struct), ctypes.c_void_p).value


def _append(lib, cache=None, table=None, starts=0x60000, counts=None, k=None, v=None, B=2, T=4):
    t, cache = _lib.Bf16Tensor(0x70000, 1024, 256, 128), cache or _cache()
    return lib.sage_cache_append(_lib.CacheAppendArgs(_addr(cache), *(table or _tab()), starts, counts, k or t, v or t, B, T,
                                                      None))


def _read(lib, cache=None, table=None, starts=0x60000, counts=None, k=None, v=None, B=2, T=4):
    t, cache = _lib.Bf16Tensor(0x70000, 1024, 256, 128), cache or _cache()
    return lib.sage_cache_read(_lib.CacheReadArgs(_addr(cache), *(table or _tab()), starts, counts, k or t, v or t, B, T, 0,
                                                  None))


def _attend(lib, cache=None, table=None, starts=0x60000, counts=None, k=None, v=None, B=2, T=4, H=4, sm=0.1, lse=None,
            ws=0x90000, wsn=1 << 40):
    t, cache = _lib.Bf16Tensor(0x70000, 2048, 512, 128), cache or _cache()
    return lib.sage_cache_attention(_lib.CacheAttentionArgs(_addr(cache), *(table or _tab()), starts, counts, k or t, v or t,
                                                            B, T, H, sm, 1, 0, lse, ws, wsn, None))


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_refusals_shared_by_the_token_entries(lib, call):
    for over, code in BAD_CACHES:
        assert call(lib, cache=_cache(**over)) == code, over
    assert call(lib, table=_tab(ptr=0)) == NULLPTR
    assert call(lib, table=_tab(ptr=0x50002)) == ALIGN
    assert call(lib, table=_tab(n=-1)) == SHAPE
    assert call(lib, table=_tab(stride=-4)) == SHAPE
    assert call(lib, starts=None) == NULLPTR
    assert call(lib, starts=0x60002) == ALIGN
    assert call(lib, counts=0x60001) == ALIGN
    assert call(lib, B=-1) == SHAPE and call(lib, T=-1) == SHAPE
    assert call(lib, B=1 << 16) == TOO_LARGE and call(lib, T=(1 << 30) + 1) == TOO_LARGE
    for which in ("k", "v"):
        assert call(lib, **{which: _lib.Bf16Tensor(0, 1024, 256, 128)}) == NULLPTR
        assert call(lib, **{which: _lib.Bf16Tensor(0x70008, 1024, 256, 128)}) == ALIGN
        for i in range(3):
            st = [1024, 256, 128]
            st[i] += 4
            assert call(lib, **{which: _lib.Bf16Tensor(0x70000, *st)}) == ALIGN


def test_refusals_of_attention(lib):
    assert _attend(lib, H=3) == SHAPE
    assert _attend(lib, H=-2) == SHAPE
    assert _attend(lib, H=70000) == TOO_LARGE
    for sm in (0.0, -1.0, math.inf):
        assert _attend(lib, sm=sm) == ARG
    assert _attend(lib, lse=0x80002) == ALIGN
    # blocks of all sequences and heads are counted in 32 bits
    assert _attend(lib, B=60000, table=_tab(n=1 << 20)) == TOO_LARGE
    assert lib.sage_cache_attention(None) == NULLPTR and lib.sage_cache_append(None) == NULLPTR
    assert lib.sage_cache_read(None) == NULLPTR
    n = ctypes.c_size_t(0)
    assert lib.sage_cache_attention_workspace_size(2, 4, 4, 2, 128, ctypes.byref(n)) == OK
    if n.value:
        assert _attend(lib, ws=None) == NULLPTR
        assert _attend(lib, ws=0x90010) == ALIGN
        assert _attend(lib, wsn=n.value - 1) == WORKSPACE
    f = lib.sage_cache_attention_workspace_size
    assert f(2, 4, 4, 2, 128, None) == NULLPTR
    assert f(2, 4, 3, 2, 128, ctypes.byref(n)) == SHAPE and f(2, 4, 4, -2, 128, ctypes.byref(n)) == SHAPE
    assert f(2, 4, 4, 2, 96, ctypes.byref(n)) == HEAD_DIM and f(1 << 16, 4, 4, 2, 128, ctypes.byref(n)) == TOO_LARGE
    assert f(0, 4, 4, 2, 128, ctypes.byref(n)) == OK and n.value == 0


def test_refusals_of_copy(lib):
    def copy(cache=None, src=0x50000, dst=0x60000, n=3):
        cache = cache or _cache()
        return lib.sage_cache_copy_pages(_addr(cache), src, dst, n, None)

    for over, code in BAD_CACHES:
        assert copy(cache=_cache(**over)) == code
    assert copy(src=None) == NULLPTR and copy(dst=None) == NULLPTR
    assert copy(src=0x50001) == ALIGN and copy(dst=0x60002) == ALIGN
    assert copy(n=-1) == SHAPE and copy(n=(1 << 20) + 1) == TOO_LARGE
    assert lib.sage_cache_copy_pages(None, 0x50000, 0x60000, 1, None) == NULLPTR


def test_structs_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no host C compiler")
    for struct, name in ((_lib.Cache, "sage_cache"), (_lib.CacheAppendArgs, "sage_cache_append_args"),
                         (_lib.CacheReadArgs, "sage_cache_read_args"),
                         (_lib.CacheAttentionArgs, "sage_cache_attention_args")):
        fields = [f[0] for f in struct._fields_]
        src = tmp_path / f"{name}.c"
        src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "sage.h"\nint main(void) {\n'
                       f'  printf("%zu\\n", sizeof({name}));\n'
                       + "".join(f'  printf("%zu\\n", offsetof({name}, {f}));\n' for f in fields) + "  return 0;\n}\n")
        exe = tmp_path / name
        subprocess.run([cc, "-std=c99", "-I", str(_build.ROOT) + "/include", str(src), "-o", str(exe)], check=True)
        got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
        assert got == [ctypes.sizeof(struct)] + [getattr(struct, f).offset for f in fields]


def test_python_binding_rejects_host_tensors_and_bad_sizes(lib):
    with pytest.raises(ValueError):
        alloc_cache(4, 2, "cpu")
    for args, code in (((4, 2, "cpu", 96), HEAD_DIM), ((4, 2, "cpu", 128, 40), SHAPE), ((1 << 21, 2, "cpu"), TOO_LARGE)):
        with pytest.raises(SageError) as e:
            alloc_cache(*args)
        assert e.value.code == code
    x = torch.zeros(1, 1, 2, 128, dtype=torch.bfloat16)
    for f in (lambda: cache_append(None, x, x, None, None), lambda: cache_read(None, None, None, 1),
              lambda: cache_attention(x, None, None, None)):
        with pytest.raises(TypeError):
            f()


# ------------------------------------------------- the keys of kept calls --


def test_signatures_of_caches_made_in_between():
    """A second cache is made while the first one's signature is being looked up."""
    inner = []

    class Size(int):
        def __hash__(self):
            if not inner:
                inner.append(None)
                inner[0] = cache._signature(8, 2, 2, 64, 0)
            return super().__hash__()

    outer = cache._signature(Size(16), 4, 1, 128, 0)
    hash(outer)
    assert inner[0] is not None and outer != inner[0]


def test_signatures_from_many_threads():
    """One signature for each combination of sizes, whoever asks first."""
    n_threads, rounds = 8, 400
    found = [dict() for _ in range(n_threads)]
    go = threading.Barrier(n_threads)
    was = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)

    def work(i):
        for r in range(rounds):
            go.wait(60)
            for j in range(4):
                sizes = (1000 + r, 1 + (i + j) % 4, 2, 128, 0)
                found[i][sizes] = cache._signature(*sizes)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(n_threads)]
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(was)
    for f in found[1:]:
        assert f == found[0]
    assert len(set(found[0].values())) == len(found[0])


# ----------------------------------------- key tiles of the longest sequences --


@pytest.fixture(scope="module")
def tiles_host(tmp_path_factory):
    exe = tmp_path_factory.mktemp("cache") / "tiles"
    src = str(_build.ROOT) + "/tests/helpers/cache_tiles_host.cu"
    subprocess.run([_build.nvcc_path(), "-std=c++17", src, "-o", str(exe)], check=True, capture_output=True)

    def ask(name, *args):
        lines = "".join(f"{name} {' '.join(map(str, a))}\n" for a in args)
        r = subprocess.run([str(exe)], input=lines, capture_output=True, text=True, check=True)
        return [int(x) for x in r.stdout.split()]

    return ask


LONGEST = 2 ** 31 - 32
LENGTHS = [0, 1, 31, 32, 33, 63, 64, 65, 2 ** 30, LONGEST - 4097, LONGEST - 2048, LONGEST - 64, LONGEST - 33, LONGEST - 32,
           LONGEST - 31, LONGEST - 1, LONGEST]


def test_key_tiles_up_to_the_longest_sequence(tiles_host):
    assert tiles_host("tiles", *[(n,) for n in LENGTHS]) == [-(-n // 64) for n in LENGTHS]


def test_look_ahead_ends_with_the_sequence(tiles_host):
    """Every block that a window of 32 tiles may look up: from any tile of the sequence to 31 tiles behind it."""
    asked = [(2 * t + i, n) for n in LENGTHS for t in {0, max(-(-n // 64) - 1, 0)} for i in range(64)]
    assert tiles_host("tokens", *asked) == [int(32 * blk < n) for blk, n in asked]


def test_tiles_with_hidden_keys(tiles_host):
    """From the first to the last tile, for rows that see all, some and none of it, and for no row at all."""
    asked = [(64 * t, n) for m in LENGTHS for t in {0, max(-(-m // 64) - 1, 0)}
             for n in {max(m - 1, 0), m, 0, 64 * t, 64 * t + 63, 64 * t + 64, 2 ** 31 - 1} if n < 2 ** 31]
    assert tiles_host("hides", *asked) == [int(key0 + 64 > n) for key0, n in asked]
