"""The tail cache's host side (no GPU): page layout, tree masks, rotary frequencies and refused arguments."""
import ctypes as C
import math

import numpy as np
import pytest

from long_context_st_b200 import api, _lib
from long_context_st_b200.build import build

BAD, FAKE = -1, 1 << 20  # a refused call never follows its addresses


@pytest.fixture(scope="module", autouse=True)
def built():
    build()


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("d,bk,bv,nkv", [(64, 2, 8, 1), (128, 4, 4, 8), (128, 8, 2, 3)])
def test_layout(ps, d, bk, bv, nkv):
    p = api.make_pages(7, ps, nkv, d, bk, bv)
    off, size = api.pages_layout(p)
    n = nkv * ps
    assert off == (0, n * d * bk // 8, n * (d * bk // 8 + 4), n * (d * (bk + bv) // 8 + 4))
    end = n * (d * (bk + bv) // 8 + 8)
    assert size == (end + 255) // 256 * 256 and api.pages_bytes(p) == 7 * size


@pytest.mark.parametrize("over", [dict(n_pages=0), dict(page_size=8), dict(page_size=48), dict(page_size=256), dict(n_kv=0),
                                  dict(d_h=96), dict(b_k=3), dict(b_v=0), dict(b_k=16)])
def test_bad_pages(over):
    a = dict(n_pages=4, page_size=64, n_kv=2, d_h=128, b_k=4, b_v=4) | over
    with pytest.raises(api.JoltError):
        api.make_pages(**a)


def test_tree_mask():
    rng = np.random.default_rng(0)
    for n in (0, 1, 2, 17, 64):
        parents = [int(rng.integers(-1, i)) for i in range(n)]
        got = api.tree_mask(parents)
        for i in range(n):
            want, j = 0, i
            while j >= 0:
                want |= 1 << j
                j = parents[j]
            assert int(got[i]) == want
    for bad in ([0], [-2], [-1, 1], [-1, 2], [-1] * 65):
        with pytest.raises(api.JoltError):
            api.tree_mask(bad)


def freqs(rot, theta):
    return theta ** (-2.0 * np.arange(rot // 2) / rot)


def close(a, b):
    return np.all(np.abs(a - b) <= 2.0 ** -24 * np.abs(b) * 1.001)


@pytest.mark.parametrize("rot", [2, 4, 64, 128, 130])
def test_rope_freqs(rot):
    theta, factor, orig = 10000.0, 8.0, 8192
    f = freqs(rot, theta)
    got, s = api.rope_freqs(rot, theta)
    assert close(got, f) and s == 1.0
    got, s = api.rope_freqs(rot, theta, "linear", factor)
    assert close(got, f / factor) and s == 1.0
    if rot >= 4:
        got, s = api.rope_freqs(rot, theta, "ntk", factor)
        assert s == 1.0 and abs(got[0] - 1) < 1e-7 and abs(got[-1] / (f[-1] / factor) - 1) < 1e-6
    got, s = api.rope_freqs(rot, theta, "ramp", factor, orig, 1.0, 4.0)
    turns = orig * f / (2 * math.pi)
    w = np.clip((turns - 1.0) / 3.0, 0, 1)
    assert close(got, (1 - w) * f / factor + w * f) and s == 1.0
    got, s = api.rope_freqs(rot, theta, "yarn", factor, orig, 1.0, 32.0)
    at = [rot * math.log(orig / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    hi = hi if hi > lo else lo + 1e-3
    w = 1 - np.clip((np.arange(rot // 2) - lo) / (hi - lo), 0, 1)
    assert close(got, (1 - w) * f / factor + w * f) and abs(s - (0.1 * math.log(factor) + 1)) < 1e-7


@pytest.mark.parametrize("args", [(3, 1e4), (0, 1e4), (514, 1e4), (64, 0.0), (64, math.inf), (64, 1e4, "linear", 0.5),
                                  (2, 1e4, "ntk", 2.0), (64, 1e4, "ramp", 2.0, 0), (64, 1e4, "ramp", 2.0, 64, 4.0, 4.0),
                                  (64, 1e4, "ramp", 2.0, 64, 0.0, 4.0), (64, 1.0, "yarn", 2.0, 64), (64, 1e4, "linear", math.nan)])
def test_rope_freqs_refusals(args):
    with pytest.raises(api.JoltError):
        api.rope_freqs(*args)


def test_rope_refusals():
    ok = dict(q=FAKE, qo=FAKE, nq=4, sq=512, sqo=512, k=FAKE, ko=FAKE, nkv=2, sk=256, sko=256, n=3, d=128, rot=128,
              layout=0, pos=FAKE, freq=FAKE, scaling=1.0, inverse=0, io=1)

    def call(**over):
        a = ok | over
        return _lib.lib().jolt_rope(*a.values(), None)

    assert call(n=0) == 0
    for over in (dict(q=None), dict(ko=None), dict(nq=-1), dict(nq=0, nkv=0), dict(n=-1), dict(d=127), dict(d=0), dict(d=514),
                 dict(rot=130), dict(rot=0), dict(rot=63), dict(layout=2), dict(pos=None), dict(freq=None),
                 dict(scaling=math.nan), dict(scaling=math.inf), dict(inverse=2), dict(io=2), dict(sq=511), dict(sko=0),
                 dict(q=FAKE + 1), dict(qo=FAKE, sqo=1024)):
        assert call(**over) == BAD, over


PAGES = dict(n_pages=4, page_size=64, n_kv=2, d_h=128, b_k=4, b_v=4)


def test_append_and_read_refusals():
    p = api.make_pages(**PAGES)
    ok = dict(p=C.byref(p), pool=FAKE, table=FAKE, mp=4, lens=FAKE, batch=1, n=2, counts=None, src=None, n_src=2, k=FAKE,
              v=FAKE, sb=512, st=256, err=None)

    def append(**over):
        return _lib.lib().jolt_pages_append(*(ok | over).values(), None)

    assert append(batch=0) == 0 and append(n=0) == 0
    for over in (dict(p=None), dict(pool=None), dict(pool=FAKE + 8), dict(table=None), dict(mp=0), dict(mp=1 << 24),
                 dict(lens=None), dict(batch=-1), dict(n=-1), dict(n=3), dict(k=None), dict(v=None), dict(k=FAKE + 2),
                 dict(sb=513), dict(st=4), dict(st=-256), dict(n_src=-1)):
        assert append(**over) == BAD, over
    ok = dict(p=C.byref(p), pool=FAKE, table=FAKE, mp=4, lens=FAKE, batch=1, start=None, n=2, k=FAKE, v=FAKE, sb=512,
              sh=256, err=None)

    def read(**over):
        return _lib.lib().jolt_pages_read(*(ok | over).values(), None)

    assert read(batch=0) == 0 and read(n=0) == 0
    for over in (dict(p=None), dict(pool=None), dict(table=None), dict(lens=None), dict(n=-1), dict(k=None, v=None),
                 dict(v=FAKE + 4), dict(sb=12), dict(sh=-8), dict(mp=0), dict(sh=248), dict(batch=2, sb=128),
                 dict(batch=65536)):
        assert read(**over) == BAD, over


def test_attention_refusals():
    p = api.make_pages(**PAGES)
    ok = dict(p=C.byref(p), pool=FAKE, table=FAKE, mp=4, lens=FAKE, batch=1, n=2, nq=8, counts=None, mask=None, q=FAKE,
              qb=2048, qt=1024, k=FAKE, v=FAKE, kb=512, kt=256, scale=0.1, po=None, pl=None, out=FAKE, lse=None, ws=FAKE,
              wsb=1 << 30)

    def call(**over):
        return _lib.lib().jolt_tree_attn(*(ok | over).values(), None)

    assert call(batch=0) == 0 and call(n=0) == 0
    for over in (dict(p=None), dict(pool=None), dict(pool=FAKE + 4), dict(table=None), dict(mp=0), dict(mp=1 << 20),
                 dict(lens=None), dict(batch=-1), dict(n=65), dict(n=-1), dict(nq=7), dict(nq=0), dict(q=None), dict(q=FAKE + 2),
                 dict(qb=4), dict(qt=1023), dict(k=None), dict(v=None), dict(kt=3), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=math.nan), dict(scale=math.inf), dict(po=FAKE), dict(pl=FAKE), dict(out=None), dict(out=FAKE + 8),
                 dict(ws=None), dict(ws=FAKE + 16), dict(nq=2 * 4097)):
        assert call(**over) == BAD, over
    need = _lib.lib().jolt_tree_attn_workspace(C.byref(p), 1, 2, 8, 4)
    assert need > 256 and call(wsb=need - 1) == -6
    for bad in ((-1, 2, 8, 4), (1, 65, 8, 4), (1, 2, 9, 4), (1, 2, 8, 0)):
        assert _lib.lib().jolt_tree_attn_workspace(C.byref(p), *bad) == 0


def test_quotient_by_reciprocal_gives_the_divisions_codes():
    """jolt_pages_append's quotient: a fl(1/s) rounded, the division only within levels * 2^-21 of a
    half-integer or where it has to be clipped, against clip(rint(a / s)), in float32, near-ties planted one and two ulps either side."""
    f32, rng = np.float32, np.random.default_rng(12)
    for levels in (3, 15, 255):
        s = np.concatenate([rng.uniform(1e-4, 4.0, 300000), 2.0 ** rng.uniform(-24, 15, 100000)]).astype(np.float16)
        s = s[s > 0].astype(f32)
        k = rng.integers(-2, levels + 2, s.size).astype(f32)
        tie = ((k + f32(0.5)) * s).astype(f32)
        up, down = np.nextafter(tie, f32(np.inf)), np.nextafter(tie, f32(-np.inf))
        some = (rng.uniform(-0.7, levels + 0.7, s.size).astype(f32) * s).astype(f32)
        for a in (some, tie, up, down, np.nextafter(up, f32(np.inf)), np.nextafter(down, f32(-np.inf)), (some * f32(1e4)).astype(f32)):
            q = (a * (f32(1) / s).astype(f32)).astype(f32)
            c = np.rint(q)
            near = np.abs((q - c).astype(f32)) >= f32(0.5) - f32(levels) * f32(2.0 ** -21)
            out = (q <= f32(-0.4375)) | (q >= f32(levels) + f32(0.4375))
            want = np.clip(np.rint((a / s).astype(f32)), 0, levels)
            got = np.where(near | out, want, c)
            assert np.array_equal(np.abs(got), want)
            assert near.mean() < 1e-3 or a is not some


@pytest.mark.parametrize("over", [dict(n_kv=8), dict(n_kv=8, io_dtype="f32"), dict(n_kv=1, d_h=64), dict(n_kv=40)])
def test_a_workspace_serves_every_smaller_call(over):
    """One workspace for the largest batch and tree: sequences finish, trees shrink, tables may be narrower. The
    splits a call makes depend on all three (37 and 38 sequences of 8 KV heads, 18 and 19 of larger trees, 8 and 9, 16
    and 17, 128 and 129 query rows fall on different sides of a rule)."""
    p = api.make_pages(**(PAGES | over))

    def size(batch, n_new, g, pages=1024):
        return _lib.lib().jolt_tree_attn_workspace(C.byref(p), batch, n_new, g * p.n_kv, pages)

    batches = [1, 2, 3, 5, 9, 16, 18, 19, 36, 37, 38, 64, 127, 128, 129, 148, 149, 296, 297, 400]
    for g in (1, 4, 8):
        for trees in ([1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64],):
            last = {}
            for b in batches:
                for n in trees:
                    got = size(b, n, g)
                    assert got > 0
                    for key in ((batches[batches.index(b) - 1], n) if b > 1 else None,
                                (b, trees[trees.index(n) - 1]) if n > 1 else None):
                        assert key is None or last[key] <= got, (b, n, g, key)
                    last[b, n] = got
        for pages in (1, 2, 5, 100, 1023):
            assert size(16, 4, g, pages) <= size(16, 4, g, pages + 1)


def test_read_refuses_rows_that_fall_on_one_another():
    """Sequences and heads may be nested either way round, but no two rows may share memory."""
    p = api.make_pages(**PAGES)  # 2 KV heads of 128
    row = 3 * 128

    def read(sb, sh, batch=4):
        return _lib.lib().jolt_pages_read(C.byref(p), FAKE, FAKE, 4, FAKE, batch, None, 3, FAKE, FAKE, sb, sh, None, None)

    for sb, sh in ((row, row), (row, 2 * row), (2 * row - 8, row), (row, 4 * row - 8), (row + 8, row + 16)):
        assert read(sb, sh) == BAD, (sb, sh)


def test_misaligned_arrays_are_refused():
    """int32 and fp32 arrays at multiples of 4 bytes, masks at multiples of 8: as the kernels load them."""
    p = api.make_pages(**PAGES)
    ok = dict(p=C.byref(p), pool=FAKE, table=FAKE, mp=4, lens=FAKE, batch=1, n=2, nq=8, counts=None, mask=None, q=FAKE,
              qb=2048, qt=1024, k=FAKE, v=FAKE, kb=512, kt=256, scale=0.1, po=None, pl=None, out=FAKE, lse=None, ws=FAKE,
              wsb=1 << 30)
    for over in (dict(table=FAKE + 2), dict(lens=FAKE + 1), dict(counts=FAKE + 2), dict(mask=FAKE + 4), dict(lse=FAKE + 2),
                 dict(po=FAKE, pl=FAKE + 2), dict(po=FAKE + 1, pl=FAKE)):
        assert _lib.lib().jolt_tree_attn(*(ok | over).values(), None) == BAD, over
    ok = dict(p=C.byref(p), pool=FAKE, table=FAKE, mp=4, lens=FAKE, batch=1, n=2, counts=None, src=None, n_src=2, k=FAKE,
              v=FAKE, sb=512, st=256, err=None)
    for over in (dict(table=FAKE + 1), dict(lens=FAKE + 2), dict(counts=FAKE + 2), dict(src=FAKE + 2), dict(err=FAKE + 2)):
        assert _lib.lib().jolt_pages_append(*(ok | over).values(), None) == BAD, over
    ok = dict(p=C.byref(p), pool=FAKE, table=FAKE, mp=4, lens=FAKE, batch=1, start=None, n=2, k=FAKE, v=FAKE, sb=512,
              sh=256, err=None)
    for over in (dict(table=FAKE + 2), dict(lens=FAKE + 2), dict(start=FAKE + 2), dict(err=FAKE + 1)):
        assert _lib.lib().jolt_pages_read(*(ok | over).values(), None) == BAD, over
    ok = dict(q=FAKE, qo=FAKE, nq=4, sq=512, sqo=512, k=FAKE, ko=FAKE, nkv=2, sk=256, sko=256, n=3, d=128, rot=128,
              layout=0, pos=FAKE, freq=FAKE, scaling=1.0, inverse=0, io=1)
    for over in (dict(pos=FAKE + 2), dict(freq=FAKE + 2)):
        assert _lib.lib().jolt_rope(*(ok | over).values(), None) == BAD, over


def test_a_description_of_pages_stays_as_it_was_made():
    """The sizes that pools are checked against are formed once: a changed field would let a kernel past the pool."""
    p = api.make_pages(**PAGES)
    for field, value in (("n_pages", 400), ("page_size", 128), ("n_kv", 8), ("io_dtype", 0), ("b_v", 8)):
        with pytest.raises(AttributeError):
            setattr(p, field, value)
    off, size = api.pages_layout(p)
    assert api.pages_bytes(p) == 4 * size and p.n_pages == 4


def test_tree_mask_takes_whole_numbers_alone():
    """A parent that int32 or whole numbers cannot hold is refused, not cut to one that they can."""
    for bad in (np.array([-1, 2 ** 32]), np.array([2 ** 32 - 1]), [-1, 0.5], np.array([-1.5]), [[-1, 0]], [-1, math.nan]):
        with pytest.raises(api.JoltError):
            api.tree_mask(bad)
    for good in (np.array([-1, 0], dtype=np.int64), [-1.0, 0.0], (-1, 0)):
        assert api.tree_mask(good).tolist() == [1, 3]
