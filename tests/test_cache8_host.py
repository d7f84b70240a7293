"""The 8-bit cache on the host: declared symbols, refusals, and the arithmetic that its
kernels rely on (rounding without a division, the division of the work among warps),
checked on the CPU.  Every C call below carries an invalid argument, so nothing is launched.
"""
import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest
import torch

import token_level_dynamic_seq_b200 as logo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE, FAKE2 = ctypes.c_void_p(1 << 20), ctypes.c_void_p(2 << 20)
no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="placeholder pointers are only passed where no GPU exists")


def test_header_and_binding_declare_the_same_symbols():
    text = open(os.path.join(ROOT, "include", "logo_cache8.h")).read()
    names = set(re.findall(r"LOGO_API\s+[^;]*?\b(logo_\w+)\s*\(", text))
    assert names == set(logo.EXPORTED_CACHE8)
    lib = logo.load_library()
    for n in names:
        assert hasattr(lib, n), n


def desc(**kw):
    base = dict(B=2, Hkv=2, Lmax=512, d=128, block=64, type=0)
    base.update({n: 1 << 20 for n in ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail")})
    base.update(kw)
    return logo.Cache8Desc(**base)


BAD_CACHES = [
    (None, 1), (desc(d=96), 2), (desc(block=32), 2), (desc(block=0), 2), (desc(type=2), 2), (desc(type=-1), 2),
    (desc(B=0), 1), (desc(Hkv=0), 1), (desc(Lmax=0), 1), (desc(Lmax=(1 << 30) + 1), 2), (desc(B=1 << 20, Hkv=2), 2),
    (desc(k=None), 1), (desc(v=(1 << 20) + 8), 1), (desc(k_scale=None), 1), (desc(v_scale=(1 << 20) + 2), 1),
]


def by(x):
    return None if x is None else ctypes.byref(x)


def rows(B=2, Hq=2, Hkv=2, L=64, d=128, cu=None, nseq=2, max_seqlen=64):
    return logo.Shape(B, Hq, Hkv, L, d, cu, nseq, max_seqlen)


def append(lib, c, sh=None, k=FAKE, v=FAKE, start=FAKE, new_len=FAKE2, ws=FAKE, n=256):
    return lib.logo_cache8_append(by(c), k, v, by(rows() if sh is None else sh), start, new_len, ws, n, None)


def read(lib, c, sh=None, k=FAKE, v=FAKE, start=FAKE, ws=FAKE, n=256):
    return lib.logo_cache8_read(by(c), start, by(rows() if sh is None else sh), k, v, ws, n, None)


def decode(lib, c, Hq=8, n=1, window=16, scale=0.0, q=FAKE, cl=FAKE, gate=FAKE, tau=FAKE, out=FAKE2, sel=None, ws=FAKE,
           nbytes=1 << 30):
    return lib.logo_decode8(q, by(c), cl, gate, tau, Hq, n, window, scale, out, sel, ws, nbytes, None)


@no_gpu_only
@pytest.mark.parametrize("case", range(len(BAD_CACHES)))
def test_every_entry_refuses_a_bad_cache(case):
    lib = logo.load_library()
    c, expect = BAD_CACHES[case]
    for call in (append, read, decode):
        assert call(lib, c) == expect
        assert lib.logo_last_error().decode() != ""


@no_gpu_only
@pytest.mark.parametrize("call", [append, read])
@pytest.mark.parametrize("kw,expect", [
    (dict(sh=rows(B=3)), 1), (dict(sh=rows(Hkv=1)), 1), (dict(sh=rows(d=64)), 1), (dict(sh=rows(L=-1)), 1),
    (dict(sh=rows(B=1, cu=0x1000, nseq=3)), 1), (dict(sh=rows(B=2, cu=0x1000)), 1),
    (dict(sh=rows(B=1, cu=0x1000, max_seqlen=65)), 1), (dict(sh=rows(B=1, cu=0x1002)), 1),
    (dict(ws=None), 3), (dict(n=128), 3), (dict(start=None), 1), (dict(start=ctypes.c_void_p((1 << 20) + 2)), 1),
    (dict(k=None), 1), (dict(v=ctypes.c_void_p((1 << 20) + 16)), 1),   # 16 but not 32 bytes
])
def test_append_and_read_refuse(call, kw, expect):
    assert call(logo.load_library(), desc(), **kw) == expect


@no_gpu_only
def test_append_refuses_tails_and_new_len():
    lib = logo.load_library()
    assert append(lib, desc(k_tail=None)) == 1
    assert append(lib, desc(v_tail=(1 << 20) + 16)) == 1
    assert append(lib, desc(), new_len=FAKE) == 1                    # the same array as start
    assert append(lib, desc(), new_len=ctypes.c_void_p((2 << 20) + 1)) == 1
    assert append(lib, desc(), new_len=ctypes.c_void_p((1 << 20) + 4)) == 1   # one element of the two shared
    assert append(lib, desc(), new_len=ctypes.c_void_p((1 << 20) - 4)) == 1


@no_gpu_only
@pytest.mark.parametrize("kw,expect", [
    (dict(window=0), 1), (dict(Hq=0), 1), (dict(n=0), 1), (dict(Hq=7), 1), (dict(Hq=66), 2), (dict(Hq=8, n=9), 2),
    (dict(n=1 << 30), 2), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(q=None), 1),
    (dict(out=None), 1), (dict(q=ctypes.c_void_p((1 << 20) + 8)), 1), (dict(cl=None), 1), (dict(gate=None), 1),
    (dict(tau=None), 1), (dict(sel=ctypes.c_void_p(3)), 1), (dict(ws=None), 3), (dict(nbytes=256), 3),
    (dict(ws=ctypes.c_void_p((1 << 20) + 8)), 3),
])
def test_decode_refuses(kw, expect):
    assert decode(logo.load_library(), desc(), **kw) == expect


def test_workspace_size():
    lib = logo.load_library()
    size = lambda c, Hq, n: lib.logo_decode8_workspace_size(by(c), Hq, n)  # noqa: E731
    one = size(desc(k=None), 8, 1)      # the buffers need not exist yet
    assert one > 256 and size(desc(), 8, 4) > one and size(desc(), 16, 1) > one
    assert one == 256 + 64 * 4 + (1184 + 4) * 2 * 4 * 130 * 4
    for c, Hq, n in ((None, 8, 1), (desc(d=32), 8, 1), (desc(), 0, 1), (desc(), 8, 0), (desc(), 8, 9), (desc(), 5, 1)):
        assert size(c, Hq, n) == 0


def test_python_refusals():
    c = logo.cache8(2, 2, 200, 64, "cpu", dtype=torch.int8, block=128)
    assert c.k_scale.shape == (2, 2, 2) and c.k_tail.shape == (2, 2, 2, 128, 64) and c.dtype == torch.int8
    parts = [c.k, c.v, c.k_scale, c.v_scale, c.k_tail, c.v_tail]

    def but(i, t):
        return parts[:i] + [t] + parts[i + 1:]

    for bad in (but(0, c.k.view(torch.uint8)), but(1, c.v.view(torch.float8_e4m3fn)), but(2, c.k_scale.double()),
                but(5, c.v_tail.half())):
        with pytest.raises(TypeError):
            logo.Cache8(*bad)
    for bad in (but(1, c.v[:1]), but(3, c.v_scale[..., :1]), but(4, c.k_tail[:, :, :1]), but(2, c.k_scale.new_empty(2, 2, 4)[..., ::2]),
                but(0, c.k.transpose(0, 1))):
        with pytest.raises(ValueError):
            logo.Cache8(*bad)
    x = torch.zeros(2, 2, 1, 64, dtype=torch.bfloat16)
    at = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):   # a cache on the host
        logo.cache8_append(c, x, x, at)
    with pytest.raises(ValueError, match="CUDA"):
        logo.cache8_read(c, at, 1, out=(x, x))
    with pytest.raises(ValueError, match="CUDA"):
        logo.decode8(x, c, at, torch.zeros(2, 1), torch.zeros(1), 16)
    with pytest.raises(ValueError, match="q:"):
        logo.decode8(x[:1], c, at, torch.zeros(2, 1), torch.zeros(1), 16)
    with pytest.raises(logo.LogoError):
        logo.decode8_workspace(c, 2, 64)


# ---------------------------------------------------------------- rounding without a division

def nearest(y, borders, values):
    """Index into `values` (ascending) of the nearest to the Fraction y >= 0, ties to the even index."""
    lo, hi = 0, len(values) - 1
    while lo < hi:
        mid = (lo + hi) // 2
        if y < borders[mid] or (y == borders[mid] and mid % 2 == 0):
            hi = mid
        else:
            lo = mid + 1
    return lo


def grids():
    e4m3 = [Fraction(m, 8) * Fraction(2) ** -6 for m in range(8)]
    e4m3 += [(1 + Fraction(m, 8)) * Fraction(2) ** e for e in range(-6, 9) for m in range(8)][:-1]   # 480 is NaN
    assert e4m3[-1] == 448 and len(e4m3) == 127
    return {448: e4m3, 127: [Fraction(i) for i in range(128)]}


def snap(y):
    """y to 19 significant bits, as the kernel does it in fp32: u = 33 y, then u - (u - y)."""
    u = (y * np.float32(33)).astype(np.float32)
    return (u - (u - y).astype(np.float32)).astype(np.float32)


@pytest.mark.parametrize("top", [448, 127])
def test_snapped_product_rounds_as_the_exact_quotient(top):
    """y = fl(x * fl(Q / a)), rounded to 19 significant bits, lies on the same side of every rounding border as the exact x Q / a,
    borders included, for all 8-bit significands of x and a."""
    values = grids()[top]
    borders = [(a + b) / 2 for a, b in zip(values, values[1:])]
    fine = np.array([float(b) for b in borders])           # borders are exact in fp64
    sig = np.arange(128, 256)
    for shift in range(0, 12):                             # x = X 2^-shift a-units: small x too
        x = (sig[:, None] * 2.0 ** -shift).astype(np.float32)
        a = sig[None, :].astype(np.float32)
        keep = x <= a
        inv = (np.float32(top) / a).astype(np.float32)
        y = (x * inv).astype(np.float32)
        snapped = snap(y).astype(np.float64)
        # exact comparison with the nearest border, in whole numbers
        idx = np.searchsorted(fine, snapped)
        for d in (-1, 0):
            j = np.clip(idx + d, 0, len(fine) - 1)
            scaled = np.vectorize(lambda b: int(b * 4096))(np.array(borders, dtype=object))[j]   # borders are multiples of 2^-10 at least
            num = (sig[:, None].astype(object) * top * 4096) - scaled * (sig[None, :].astype(object) << shift)
            want = np.sign(num.astype(np.float64))
            got = np.sign(snapped - fine[j])
            assert (got == want)[keep].all()
    # a few against the definition itself
    rng = np.random.default_rng(0)
    for _ in range(200):
        X, A = int(rng.integers(128, 256)), int(rng.integers(128, 256))
        s = int(rng.integers(0, 8))
        if X > A << s:
            continue
        inv = np.float32(top) / np.float32(A)
        y = np.float32(np.float32(X * 2.0 ** -s) * inv)
        y = float(snap(np.array([y], np.float32))[0])
        assert nearest(Fraction(y), borders, values) == nearest(Fraction(X * top, A << s), borders, values)


# ---------------------------------------------------------------- division of the decode's work

def plan(length, n, W, any_global, Lmax, STAGE):
    """Units of one sequence as the kernel counts them: (out, in0, in1)."""
    if length <= 0 or length > Lmax:
        return 0, 0, 0
    e0, e1 = length - n - W + 1, length - W
    return (-(-e1 // STAGE) if any_global and e1 > 0 else 0), (e0 // STAGE if e0 > 0 else 0), -(-length // STAGE)


@pytest.mark.parametrize("seed", range(40))
def test_every_unit_of_work_reaches_the_joining_kernel_once(seed):
    """A model of the list of units, of its shares, of the states that warps and CTAs write and of the slots that the
    joining kernel reads: each unit's positions are counted once, and no two states share a slot."""
    rng = np.random.default_rng(seed)
    B, Hkv, n = int(rng.integers(1, 70)), int(rng.integers(1, 9)), int(rng.integers(1, 9))
    Lmax = int(rng.integers(1, 5000))
    W = min(int(rng.integers(1, 6000)), Lmax)
    grid, warps = int(rng.choice([1, 5, 20, 148])), int(rng.choice([1, 3, 6, 8]))
    lens = rng.integers(0, Lmax + 1, B)
    STAGE = int(rng.choice([32, 64]))   # positions of a unit, for d = 128 and 64
    plans = [plan(int(L), n, W, bool(rng.integers(0, 2)), Lmax, STAGE) for L in lens]
    pads = [(b > a) + (o > 0) for o, a, b in plans]      # empty units behind a pair's stages
    units = [o + b - a + e for (o, a, b), e in zip(plans, pads)]
    for L, (o, a, b) in zip(lens, plans):   # stages cover the window of every token, and all before it
        L = int(L)
        for i in range(max(0, n - L), n):
            t = L - n + i
            first = max(0, t - W + 1)
            assert a * STAGE <= first and (t < b * STAGE)
            if o:
                assert first == 0 or first - 1 < o * STAGE
    T = sum(units) * Hkv
    if T == 0:
        return
    cut = lambda u, most: (min(u, most), u)  # noqa: E731

    def first(share, w):
        n, u = share
        return w * (u // n) + min(w, u % n)

    def of(share, x):
        n, u = share
        each, rest = u // n, u % n
        return x // (each + 1) if x < rest * (each + 1) else rest + (x - rest * (each + 1)) // each

    ctas = cut(T, grid)
    run_of, u = [], 0                       # the list: one run after the other
    runs = {}
    for pair in range(B * Hkv):
        o, a, b = plans[pair // Hkv]
        for kind, n_units in ((1, o), (0, b - a)):
            if n_units:
                runs[(pair, kind)] = (u, u + n_units)
                run_of += [(pair, kind)] * n_units
                u += n_units
        run_of += [None] * pads[pair // Hkv]
        u += pads[pair // Hkv]
    assert u == T
    written = {}                            # slot -> units whose states meet there
    for c in range(ctas[0]):
        base = first(ctas, c)
        size = first(ctas, c + 1) - base
        assert size > 0
        inner = cut(size, warps)
        last = [None] * warps
        tails = [None] * warps
        for w in range(inner[0]):
            mine = list(range(base + first(inner, w), base + first(inner, w + 1)))
            assert mine and all(of(ctas, x) == c and of(inner, x - base) == w for x in mine)
            kinds = [run_of[x] for x in mine if run_of[x]]
            if not kinds:
                continue
            last[w] = kinds[-1]
            tails[w] = [x for x in mine if run_of[x] == kinds[-1]]
            for key in dict.fromkeys(kinds[:]):
                if key != kinds[-1]:
                    slot = (c * warps + w + key[0], key[1])
                    assert slot not in written
                    written[slot] = [x for x in mine if run_of[x] == key]
        w = 0
        while w < inner[0]:
            if last[w] is None:
                w += 1
                continue
            v = w
            while v + 1 < inner[0] and last[v + 1] == last[w]:
                v += 1
            slot = (c * warps + w + last[w][0], last[w][1])
            assert slot not in written and slot[0] < 1184 + B * Hkv
            written[slot] = sum(tails[w:v + 1], [])
            w = v + 1
    for (pair, kind), (a, e) in runs.items():   # what the joining kernel reads
        c0, c1 = of(ctas, a), of(ctas, e - 1)
        share = lambda c: cut(first(ctas, c + 1) - first(ctas, c), warps)  # noqa: E731
        v0, v1 = of(share(c0), a - first(ctas, c0)), of(share(c1), e - 1 - first(ctas, c1))
        slots = [c0 * warps + v0] + [c * warps for c in range(c0 + 1, c1 + 1)]
        behind = e + (pads[pair // Hkv] if kind == 0 else 0)
        if first(share(c1), v1 + 1) > behind - first(ctas, c1) and v1 != (v0 if c1 == c0 else 0):
            slots.append(c1 * warps + v1)
        got = sum((written.pop((x + pair, kind)) for x in slots), [])
        assert sorted(got) == list(range(a, e))
    assert not written
