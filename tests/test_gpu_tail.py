"""GPU: the tail cache's write, read back and attention, and rotary positions, against 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import oracle
from long_context_st_b200 import api
from tail_ref import (NP, HALF_STEP, rows, f64, make_table, i32, fill_random, stored_rows, attention, check_attention)

pytestmark = pytest.mark.gpu


# ---- rotary positions ------------------------------------------------------------------------------

def rope_ref(x, pos, freq, layout, scaling, inverse):
    y = f64(x).copy()
    rot = 2 * len(freq)
    ang = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None, :]
    c, s = scaling * np.cos(ang)[:, None], scaling * np.sin(ang)[:, None]
    if inverse:
        s = -s
    a, b = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    u, v = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def rope_close(got, ref, io, x):
    # cos and sin are within 2^-22 (float sincospi and the reduced angle's rounding, 2 pi 2^-25), two
    # products and a sum in fp32, one rounding to the type
    size = np.abs(f64(x)).max()
    worst = (np.abs(f64(got) - ref) - HALF_STEP[io] * np.abs(ref)).max()
    assert worst <= 2.0 ** -20 * 2 * size


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,nq,nkv,d,rot", [(1, 8, 2, 64, 64), (5, 32, 8, 128, 128), (257, 4, 1, 128, 32), (3, 3, 0, 6, 6),
                                            (4, 0, 5, 20, 10), (2, 5, 3, 80, 80), (1100, 2, 2, 256, 64)])
def test_rope(cuda_ok, io, layout, n, nq, nkv, d, rot):
    rng = np.random.default_rng(n * 7 + d)
    freq = (500000.0 ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)
    pos = rng.integers(0, 1 << 20, n).astype(np.int32)
    pos[0] = 2 ** 31 - 1
    if n > 2:
        pos[1], pos[2] = -5, 0
    q = rows(rng, (n, nq, d), io) if nq else None
    k = rows(rng, (n, nkv, d), io) if nkv else None
    tp, tf = torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda()
    for inverse in (False, True):
        qo, ko = api.rope(q, k, tp, tf, layout=layout, scaling=1.25, inverse=inverse)
        for x, y in ((q, qo), (k, ko)):
            if x is not None:
                rope_close(y, rope_ref(x, pos, freq, layout, 1.25, inverse), io, x)
                assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_rope_in_place_on_a_fused_projection(cuda_ok, io):
    rng = np.random.default_rng(5)
    n, nq, nkv, d = 33, 8, 2, 128
    qkv = rows(rng, (n, (nq + 2 * nkv) * d), io)
    before = qkv.clone()
    q, k = qkv[:, :nq * d].view(n, nq, d), qkv[:, nq * d:(nq + nkv) * d].view(n, nkv, d)
    freq = (10000.0 ** (-2.0 * np.arange(32) / 64)).astype(np.float32)
    pos = np.arange(n, dtype=np.int32) + 70000
    tp, tf = torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda()
    api.rope(q, k, tp, tf, q_out=q, k_out=k)
    old_q, old_k = before[:, :nq * d].view(n, nq, d), before[:, nq * d:(nq + nkv) * d].view(n, nkv, d)
    rope_close(q, rope_ref(old_q, pos, freq, "half", 1.0, False), io, old_q)
    rope_close(k, rope_ref(old_k, pos, freq, "half", 1.0, False), io, old_k)
    assert torch.equal(qkv[:, (nq + nkv) * d:], before[:, (nq + nkv) * d:])
    api.rope(q, k, tp, tf, q_out=q, k_out=k, inverse=True)
    # there and back: the turned pair (y_a, y_b) was rounded, off by at most h |y_a| and h |y_b|; turned back
    # that is at most h (|y_a c| + |y_b s|) <= h |pair| <= h sqrt(2) max|x|; then the last rounding
    x = f64(old_q)
    h, size = HALF_STEP[io], np.abs(x).max()
    worst = (np.abs(f64(q) - x) - h * np.abs(x)).max()
    assert worst <= h * math.sqrt(2) * size * (1 + h) + 2.0 ** -20 * 4 * size


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_gradient_against_differences(cuda_ok, layout):
    rng = np.random.default_rng(6)
    n, h, d, rot = 4, 2, 16, 12
    freq = rng.uniform(0.01, 1.0, rot // 2).astype(np.float32)
    pos = rng.integers(0, 1000, n).astype(np.int32)
    x, w = rows(rng, (n, h, d), "f32"), rows(rng, (n, h, d), "f32")
    tp, tf = torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda()
    grad, _ = api.rope(w, None, tp, tf, layout=layout, scaling=0.75, inverse=True)
    num = np.zeros(x.shape)
    for at in np.ndindex(*x.shape):
        for sign in (1, -1):
            y = f64(x).copy()
            y[at] += sign
            num[at] += sign * (rope_ref(torch.from_numpy(y), pos, freq, layout, 0.75, False) * f64(w)).sum() / 2
    assert np.abs(f64(grad) - num).max() <= 2.0 ** -20 * 2 * np.abs(f64(w)).max()


def test_python_refusals(cuda_ok):
    """What the tensors themselves give away: types, shapes, strides, devices."""
    f = torch.ones(32, device="cuda")
    q, pos = torch.zeros(3, 4, 64, device="cuda"), i32([0, 1, 2])
    p = api.make_pages(4, 16, 2, 64, 4, 4, io_dtype="f32")
    pool, table, lens = api.new_pool(p), i32([[0, 1], [2, 3]]), i32([0, 0])
    k = torch.zeros(2, 3, 2, 64, device="cuda")
    out, ws = torch.zeros(2, 3, 4, 64, device="cuda"), api.new_tree_workspace(p, 2, 3, 4, 2)
    q4 = out.clone()
    side = torch.cuda.Stream().cuda_stream
    for call in (lambda: api.rope(q.double(), None, pos, f), lambda: api.rope(q.cpu(), None, pos, f),
                 lambda: api.rope(q, None, pos.long(), f), lambda: api.rope(q, None, pos[:2], f),
                 lambda: api.rope(q.transpose(1, 2), None, pos, f), lambda: api.rope(q, None, pos, f, layout="other"),
                 lambda: api.rope(q, None, pos, f, stream=side), lambda: api.rope(q, None, pos, torch.ones(33, device="cuda")),
                 lambda: api.pages_append(p, pool, table, lens, k, k.bfloat16()),
                 lambda: api.pages_append(p, pool[:-1], table, lens, k, k),
                 lambda: api.pages_append(p, pool, table, lens[:1], k, k),
                 lambda: api.pages_append(p, pool, table, lens, k, k.transpose(1, 2).contiguous().transpose(1, 2)),
                 lambda: api.pages_append(p, pool, table, lens, k, k, n_new=4),
                 lambda: api.pages_read(p, pool, table, lens), lambda: api.pages_read(p, pool, table, lens, k, out),
                 lambda: api.tree_attn(p, pool, table, lens, q4, out, ws, k=k),
                 lambda: api.tree_attn(p, pool, table, lens, q4, out[:, :2], ws),
                 lambda: api.tree_attn(p, pool, table, lens, q4, out, ws[:1000]),
                 lambda: api.tree_attn(p, pool, table, lens, q4, out, ws, k=k, v=k, mask=torch.ones(2, 3, device="cuda")),
                 lambda: api.tree_attn(p, pool, table, lens, q4, out, ws, prefix_out=out)):
        with pytest.raises(api.JoltError):
            call()


# ---- write and read back ---------------------------------------------------------------------------

def coded(x, seed, b):
    """The codec's own rotate and quantise of rows [n, d]."""
    codes, sz, err = api.quantize_pack(api.rotate_rows(x.float().contiguous(), seed), b)
    assert int(err) == 0
    return codes, sz


def page_rows(p, pool, which):
    """(codes [page][head][slot][bytes], sz) of keys (0) or values (1), views of the pool."""
    off, size = api.pages_layout(p)
    x = pool.view(p.n_pages, size)
    b = (p.b_k, p.b_v)[which]
    rb = p.d_h * b // 8
    n = p.n_kv * p.page_size
    return (x[:, off[2 * which]:off[2 * which] + n * rb].reshape(p.n_pages, p.n_kv, p.page_size, rb),
            x[:, off[2 * which + 1]:off[2 * which + 1] + 4 * n].contiguous().view(torch.float16)
            .reshape(p.n_pages, p.n_kv, p.page_size, 2))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,bk,bv,ps,nkv", [(128, 4, 4, 64, 8), (128, 8, 2, 16, 3), (64, 2, 8, 32, 2), (64, 4, 2, 128, 1),
                                            (128, 2, 8, 128, 2), (64, 8, 4, 16, 5)])
def test_append_is_the_codec_bit_for_bit(cuda_ok, io, d, bk, bv, ps, nkv):
    rng = np.random.default_rng(d + bk * 3 + ps)
    lens, n = [0, 2 * ps - 1, 37], 19
    counts = [n, 7, 0]
    table, n_pages = make_table(rng, [a + n for a in lens], ps)
    p = api.make_pages(n_pages, ps, nkv, d, bk, bv, io_dtype=io, rot_seed=77)
    pool = api.new_pool(p)
    pool.fill_(0xA5)
    k, v = rows(rng, (3, n, nkv, d), io, True), rows(rng, (3, n, nkv, d), io)
    err = i32([0])
    api.pages_append(p, pool, table, i32(lens), k, v, counts=i32(counts), err=err)
    assert int(err) == 0
    want = torch.full_like(pool, 0xA5)
    tab = table.cpu().numpy()
    off, size = api.pages_layout(p)
    for x, which, b in ((k, 0, bk), (v, 1, bv)):
        rb = d * b // 8
        for s in range(3):
            for i in range(counts[s]):
                t = lens[s] + i
                page, slot = tab[s, t // ps], t % ps
                codes, sz = coded(x[s, i], 77, b)
                for h in range(nkv):
                    at = page * size + off[2 * which] + (h * ps + slot) * rb
                    want[at:at + rb] = codes[h]
                    at = page * size + off[2 * which + 1] + (h * ps + slot) * 4
                    want[at:at + 4] = sz[h].view(torch.uint8)
    assert torch.equal(pool, want)


def test_append_accepted_path_of_a_strided_projection(cuda_ok):
    rng = np.random.default_rng(8)
    d, nkv, ps, n = 128, 2, 16, 9
    p0, n_pages = make_table(rng, [40, 40], ps)
    p = api.make_pages(n_pages, ps, nkv, d, 4, 8, rot_seed=3)
    kv = rows(rng, (2, n, 2 * nkv * d + 64), "bf16")
    k, v = (kv[..., a * nkv * d:(a + 1) * nkv * d].unflatten(-1, (nkv, d)) for a in (0, 1))
    src = i32([[0, 2, 5, 8], [1, 1, 0, 0]])
    pools = [api.new_pool(p) for _ in range(2)]
    lens = i32([15, 30])
    api.pages_append(p, pools[0], p0, lens, k, v, counts=i32([4, 2]), src=src)
    pick = src.long()[:, :, None, None].expand(-1, -1, nkv, d)
    api.pages_append(p, pools[1], p0, lens, k.gather(1, pick).contiguous(), v.gather(1, pick).contiguous(),
                     counts=i32([4, 2]))
    assert torch.equal(pools[0], pools[1]) and int(pools[0].sum()) > 0


def test_append_reports_bad_pages_sources_and_values(cuda_ok):
    rng = np.random.default_rng(9)
    d, nkv, ps = 64, 2, 16
    p = api.make_pages(3, ps, nkv, d, 4, 4, rot_seed=3)
    k = rows(rng, (1, 4, nkv, d), "bf16")
    lens = i32([14])
    for table, src, status in (([[0, 3]], None, -1), ([[0, -1]], None, -1), ([[0, 1]], [[0, 1, 4, -1]], -1),
                               ([[0]], None, -1)):
        pool, err = api.new_pool(p), i32([0])
        pool.fill_(0x11)
        api.pages_append(p, pool, i32(table), lens, k, k, src=None if src is None else i32(src), err=err)
        assert int(err) == status
        codes, _ = page_rows(p, pool, 0)
        assert bool((codes[0, :, 14:] != 0x11).any(-1).all())  # tokens 14, 15 are written all the same
        assert bool((codes[1:] == 0x11).all()) and bool((codes[0, :, :14] == 0x11).all())
    for length in (-1, 29, 33):  # 29: the last of four rows is past the table; -1 and 33: no length at all
        pool, err = api.new_pool(p), i32([0])
        pool.fill_(0x11)
        api.pages_append(p, pool, i32([[0, 1]]), i32([length]), k, k, err=err)
        codes, _ = page_rows(p, pool, 0)
        want = torch.zeros_like(codes, dtype=torch.bool).any(-1)
        if length == 29:
            want[1, :, 13:] = True
        assert int(err) == -1 and torch.equal((codes != 0x11).any(-1), want)
    for bad in (float("nan"), float("inf"), 3e38):
        x = k.clone()
        x[0, 2, 1, 5] = bad
        pool, err = api.new_pool(p), i32([0])
        api.pages_append(p, pool, i32([[0, 1]]), lens, x, k, err=err)
        assert int(err) == -5


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("d,bk,bv,ps,nkv", [(128, 4, 4, 64, 4), (128, 8, 2, 16, 3), (64, 2, 8, 32, 2), (64, 4, 4, 128, 1),
                                            (128, 2, 8, 32, 1), (64, 8, 2, 16, 2)])
def test_read_back(cuda_ok, io, d, bk, bv, ps, nkv):
    rng = np.random.default_rng(d + bk + ps)
    lens, start, n = [0, 3 * ps + 5, 1, ps], [0, ps - 3, 0, 0], 2 * ps + 3
    table, n_pages = make_table(rng, lens, ps)
    p = api.make_pages(n_pages, ps, nkv, d, bk, bv, io_dtype=io, rot_seed=12)
    pool = api.new_pool(p)
    fill_random(rng, p, pool)
    big = torch.full((4, 3, nkv, n + 2, d), 7.0, dtype=NP[io], device="cuda")  # a layer of a bigger tensor
    k_out, v_out = big[:, 0, :, 1:n + 1], big[:, 2, :, 1:n + 1]
    err = i32([0])
    api.pages_read(p, pool, table, i32(lens), k_out, v_out, start=i32(start), err=err)
    assert int(err) == 0
    R = oracle.rotation_matrix(d, 12)
    held = stored_rows(p, pool, table, lens)
    want = np.full((2, 4, nkv, n, d), 7.0)
    for b in range(4):
        for x in range(2):
            y = held[b][x][:, start[b]:start[b] + n] @ R
            want[x, b, :, :y.shape[1]] = y
    # a dequantised value is rounded once, the rotation adds d of them in log2(d) fp32 roundings
    bits = (math.log2(d) + 3) * 2.0 ** -24
    for got, w in ((k_out, want[0]), (v_out, want[1])):
        size = max(np.abs(h).max(initial=0.0) for s in held for h in s) * math.sqrt(d)
        worst = (np.abs(f64(got) - w) - HALF_STEP[io] * np.abs(w)).max()
        assert worst <= bits * size
    assert bool((big[:, 1] == 7).all()) and bool((big[:, :, :, 0] == 7).all()) and bool((big[:, :, :, -1] == 7).all())
    only = torch.full_like(v_out.contiguous(), 7.0)
    api.pages_read(p, pool, table, i32(lens), None, only, start=i32(start))
    assert torch.equal(only, v_out)


def test_read_reports_bad_pages_and_lengths(cuda_ok):
    rng = np.random.default_rng(13)
    p = api.make_pages(3, 16, 1, 64, 4, 4, io_dtype="f32", rot_seed=3)
    pool = api.new_pool(p)
    fill_random(rng, p, pool)
    for table, lens, start, seen in (([[0, 7]], [20], [0], 16), ([[0, -1]], [20], [0], 16), ([[0, 1]], [99], [0], 32),
                                     ([[0, 1]], [-4], [0], 0), ([[0, 1]], [20], [-1], 0)):
        out, err = torch.full((1, 1, 40, 64), 5.0, device="cuda"), i32([0])
        api.pages_read(p, pool, i32(table), i32(lens), out, None, start=i32(start), err=err)
        assert int(err) == -1
        got = (out != 5.0).any(-1)[0, 0]
        assert bool(got[:seen].all()) and not bool(got[seen:].any())


# ---- attention ---------------------------------------------------------------------------------------

def attn_case(seed, lens, n, nq, nkv, d, bk, bv, ps, io, counts=None, tree=True, drafted=True, prefix=False, extra=1):
    rng = np.random.default_rng(seed)
    B = len(lens)
    table, n_pages = make_table(rng, lens, ps, extra_width=extra)
    p = api.make_pages(n_pages, ps, nkv, d, bk, bv, io_dtype=io, rot_seed=31)
    pool = api.new_pool(p)
    fill_random(rng, p, pool)
    q = rows(rng, (B, n, nq, d), io)
    k = v = mask = None
    if drafted:
        k, v = rows(rng, (B, n, nkv, d), io, True), rows(rng, (B, n, nkv, d), io)
        if tree:
            m = np.stack([api.tree_mask([int(rng.integers(-1, i)) for i in range(n)]) for _ in range(B)])
            mask = torch.from_numpy(m.view(np.int64)).cuda()
    pre = None
    if prefix:
        pre = (rows(rng, (B, n, nq, d), io), torch.from_numpy(rng.normal(2.0, 3.0, (B, n, nq)).astype(np.float32)).cuda())
    cnt = i32(counts) if counts is not None else None
    return p, pool, table, lens, q, k, v, mask, cnt, pre


def run_attn(c, out=None, lse=None, ws=None, **over):
    p, pool, table, lens, q, k, v, mask, cnt, pre = c
    out = torch.full_like(q, 9.0, memory_format=torch.contiguous_format) if out is None else out
    lse = torch.full(q.shape[:3], 9.0, device="cuda") if lse is None else lse
    ws = api.new_tree_workspace(p, q.shape[0], q.shape[1], q.shape[2], table.shape[1]) if ws is None else ws
    api.tree_attn(p, pool, table, i32(lens), q, out, ws, k=k, v=v, mask=mask, counts=cnt, lse=lse,
                  prefix_out=pre[0] if pre else None, prefix_lse=pre[1] if pre else None, **over)
    api.check_ws(ws)
    return out, lse


def check_case(c):
    p, pool, table, lens, q, k, v, mask, cnt, pre = c
    out, lse = run_attn(c)
    counts = cnt.cpu().tolist() if cnt is not None else [q.shape[1]] * q.shape[0]
    ref = attention(p, pool, table, lens, q, k, v, mask, cnt, prefix=pre)
    check_attention(p, out, lse, ref, counts)
    for b, n in enumerate(counts):  # rows behind the last drafted token are left as they were
        n = max(n, 0)
        assert bool((out[b, n:] == 9).all()) and bool((lse[b, n:] == 9).all())
    return out, lse


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,nq,nkv", [(1, 8, 2), (1, 4, 4), (1, 8, 1), (3, 4, 2), (5, 12, 4), (16, 8, 2), (64, 4, 2),
                                      (33, 6, 6), (7, 24, 2)])
@pytest.mark.parametrize("d,bk,bv,ps", [(128, 4, 4, 64), (64, 2, 8, 16)])
def test_attention_rows(cuda_ok, io, n, nq, nkv, d, bk, bv, ps):
    check_case(attn_case(n + nq, [3 * ps + 7, 1, 0, 150], n, nq, nkv, d, bk, bv, ps, io, prefix=n == 5))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("bk", [2, 4, 8])
@pytest.mark.parametrize("bv", [2, 4, 8])
@pytest.mark.parametrize("d,n", [(64, 1), (128, 1), (64, 9), (128, 9)])
def test_attention_bits(cuda_ok, io, bk, bv, d, n):
    check_case(attn_case(bk * 10 + bv, [77, 300], n, 4, 2, d, bk, bv, 32, io, prefix=bv == 4))


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("length", [0, 1, 15, 16, 17, 31, 33, 127, 128, 129, 255, 257, 700])
def test_attention_lengths(cuda_ok, ps, length):
    check_case(attn_case(length + ps, [length, 0], 2, 4, 2, 64, 4, 4, ps, "f32", extra=3))


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_attention_long(cuda_ok, io):
    check_case(attn_case(41, [20011], 2, 4, 1, 128, 4, 4, 64, io))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("drafted", [True, False])
def test_attention_padded_batch_and_empty_rows(cuda_ok, io, drafted):
    c = attn_case(43, [0, 40, 0, 9], 6, 4, 2, 64, 8, 4, 16, io, counts=[6, 2, 0, 9], drafted=drafted)
    if drafted:  # row 2 of sequence 0 sees nothing at all
        c[7][0, 2] = 0
    out, lse = check_case(c)
    if drafted:
        assert bool((out[0, 2] == 0).all()) and bool((lse[0, 2] == -math.inf).all())
    else:
        assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_attention_ignores_what_masked_places_hold(cuda_ok, io):
    lens = [21, 50]
    c = attn_case(44, lens, 4, 4, 2, 128, 4, 4, 16, io, counts=[4, 2])
    p, pool, table, _, q, k, v, mask, cnt, _ = c
    mask[0] = torch.tensor([1, 2, 4, 12], device="cuda")  # nobody but row 1 sees token 1
    want = run_attn(c)
    bad = [float("nan"), float("inf"), -torch.finfo(NP[io]).max, float("-inf")]
    for x in bad:
        k[0, 1], v[0, 1] = x, x
        k[1, 2:], v[1, 2:] = x, x
        off, size = api.pages_layout(p)
        pages = pool.view(p.n_pages, size)
        tab = table.cpu().numpy()
        for b, n in enumerate(lens):  # slots behind the last token of the last page
            page = tab[b, (n - 1) // 16]
            for seg in (1, 3):
                sz = pages[page, off[seg]:off[seg] + 2 * 16 * 4].view(torch.float16).view(2, 16, 2)
                sz[:, n % 16:] = x if x == x and abs(x) == math.inf else float("nan")
        got = run_attn(c)
        keep = torch.tensor([0, 2, 3], device="cuda")
        for a, w in zip(got, want):
            assert torch.equal(a[0, keep], w[0, keep]) and torch.equal(a[1], w[1])


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("n,nq", [(4, 4), (40, 2)])
def test_attention_rows_that_see_infinite_values(cuda_ok, io, n, nq):
    c = attn_case(51, [30], n, nq, 1, 64, 4, 4, 16, io)
    v, mask = c[6], c[7]
    want = run_attn(c)
    v[0, 2, 0, 7], v[0, 3, 0, 9] = float("inf"), float("nan")
    out, lse = run_attn(c)
    sees = [(mask[0] >> j) & 1 == 1 for j in (2, 3)]
    assert bool((out[0, sees[0] & ~sees[1], :, 7] == math.inf).all()) and bool(out[0, sees[1], :, 9].isnan().all())
    free = ~sees[0] & ~sees[1]
    assert torch.equal(out[0, free], want[0][0, free]) and torch.equal(lse, want[1])
    keep = [f for f in range(64) if f not in (7, 9)]
    assert torch.equal(out[0][..., keep], want[0][0][..., keep])


def test_attention_strides_no_lse_and_prefix_in_place(cuda_ok):
    rng = np.random.default_rng(46)
    c = attn_case(45, [65, 130], 3, 8, 2, 128, 4, 8, 64, "bf16", prefix=True)
    p, pool, table, lens, q, k, v, mask, cnt, pre = c
    want, want_lse = run_attn(c)
    qkv = rows(rng, (2, 3, (8 + 2 + 2) * 128 + 8), "bf16")
    q2, k2, v2 = (qkv[..., a * 128:b * 128].unflatten(-1, (b - a, 128)) for a, b in ((0, 8), (8, 10), (10, 12)))
    q2.copy_(q), k2.copy_(k), v2.copy_(v)
    out, lse = pre[0].clone(), pre[1].clone()
    got = run_attn((p, pool, table, lens, q2, k2, v2, mask, cnt, (out, lse)), out=out, lse=lse)
    assert torch.equal(got[0], want) and torch.equal(got[1], want_lse)
    ws = api.new_tree_workspace(p, 2, 3, 8, table.shape[1])
    out = torch.empty_like(want)
    api.tree_attn(p, pool, table, i32(lens), q, out, ws, k=k, v=v, mask=mask, prefix_out=pre[0], prefix_lse=pre[1])
    assert torch.equal(out, want)
    nothing = (torch.full_like(pre[0], float("nan")), torch.full_like(pre[1], -math.inf))
    assert torch.equal(run_attn((p, pool, table, lens, q, k, v, mask, cnt, nothing))[0],
                       run_attn((p, pool, table, lens, q, k, v, mask, cnt, None))[0])


def test_attention_reports_bad_pages_and_lengths(cuda_ok):
    c = attn_case(47, [40], 2, 4, 2, 64, 4, 4, 16, "f32")
    p, pool, table, lens, q, k, v, mask, cnt, pre = c
    want = run_attn((p, pool, table, [32], q, k, v, mask, cnt, pre))
    ws = api.new_tree_workspace(p, 1, 2, 4, table.shape[1])
    for bad in (p.n_pages, -1, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = bad
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        api.tree_attn(p, pool, t, i32([40]), q, out, ws, k=k, v=v, mask=mask, lse=lse)
        with pytest.raises(api.JoltError) as e:
            api.check_ws(ws)
        assert e.value.status == -1
        check_attention(p, out, lse, attention(p, pool, table, [32], q, k, v, mask), [2])  # its tokens are not seen
    for length, same in ((-3, 0), (10 ** 6, None)):
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        api.tree_attn(p, pool, table, i32([length]), q, out, ws, k=k, v=v, mask=mask, lse=lse)
        with pytest.raises(api.JoltError):
            api.check_ws(ws)
    del want


@pytest.mark.parametrize("io,n,nq", [("f32", 1, 1), ("bf16", 1, 1), ("bf16", 9, 2), ("f32", 9, 2)])
@pytest.mark.parametrize("batch,nkv", [(24, 16), (100, 1), (130, 1)])
def test_attention_many_sequences(cuda_ok, io, n, nq, batch, nkv):
    """Batches that are divided evenly over the GPU and batches with a block of its own for every sequence,
    some of them empty."""
    lens = [(37 * i) % 300 if i % 5 else 0 for i in range(batch)]
    check_case(attn_case(batch, lens, n, nq * nkv, nkv, 64, 4, 4, 16, io, counts=[n - (i % 3 == 2) for i in range(batch)]))


def test_attention_scales_far_apart(cuda_ok):
    """Value scales over fp16's whole range, constant rows, and rows whose first tile is empty of scale."""
    for io in ("f32", "bf16"):
        c = attn_case(48, [200], 3, 4, 1, 64, 4, 4, 16, io)
        p, pool = c[0], c[1]
        off, size = api.pages_layout(p)
        pages = pool.view(p.n_pages, size)
        rng = np.random.default_rng(3)
        for page in range(p.n_pages):
            for seg in (1, 3):
                sz = pages[page, off[seg]:off[seg] + 16 * 4].view(torch.float16).view(16, 2)
                if seg == 3:
                    sz[:, 0] = torch.from_numpy(2.0 ** rng.integers(-24, 10, 16)).half().cuda()
                sz[::5, 0] = 0.0
        check_case(c)


@pytest.mark.parametrize("d,n,nq", [(128, 40, 2), (64, 40, 2), (128, 2, 2), (64, 9, 2)])
def test_attention_rising_scores(cuda_ok, d, n, nq):
    """Key scales that grow along the sequence: a row's maximum is passed again and again, inside a tile too."""
    c = attn_case(49, [900, 300], n, nq, 1, d, 4, 8, 16, "bf16")
    p, pool, table = c[:3]
    off, size = api.pages_layout(p)
    pages, tab = pool.view(p.n_pages, size), table.cpu().numpy()
    for b, length in enumerate(c[3]):
        for i in range(-(-length // 16)):
            sz = pages[tab[b, i], off[1]:off[1] + 16 * 4].view(torch.float16).view(16, 2)
            sz.copy_((sz.float() * (0.02 * (i * 16 + torch.arange(16, device="cuda")[:, None]) + 0.1)).half())
    check_case(c)


# An MMA step adds 16 products and the sum so far, and drops from each what lies below 24 bits of the largest:
# about sqrt(17 / 3) 2^-24 of it a step, taken as one-sided over the steps below; a row of 128 takes 8 steps, two
# terms each: 16 * 2.4 * 2^-24 = 2^-18.7. Operands keep 22 bits, and the fp32 transforms' seven stages and the joins
# of partial sums add some 2^-22: 2^-18 of the products' size in all, the largest product being counted with a
# factor of two. Codes that entered as subnormals would lose 8 more bits at 2 bits, 6 at 4, 2 at 8.

@pytest.mark.parametrize("io,b", [("f32", 2), ("f32", 4), ("f32", 8), ("bf16", 2)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 12])
def test_scores_keep_their_bits(cuda_ok, io, b, d, n):
    """Sequences of one token: the log-sum-exp is the score itself."""
    c = attn_case(61, [1] * 40, n, 4, 2, d, b, 4, 16, io, drafted=False)
    p, pool, table, lens, q = c[:5]
    _, lse = run_attn(c)
    R = oracle.rotation_matrix(d, p.rot_seed)
    qr = (f64(q) @ R.T) / math.sqrt(d)                                       # [B][n][4][d]
    y = np.stack([s[0][:, 0] for s in stored_rows(p, pool, table, lens)])    # [B][2][d]
    s = np.einsum("bnhgd,bhd->bnhg", qr.reshape(40, n, 2, 2, d), y).reshape(40, n, 4)
    # the codes' part and the offsets' part are formed apart: both count
    size = 2 * np.sqrt(np.mean(qr ** 2) * d) * (np.sqrt(np.mean(y ** 2)) + np.abs(y.mean(-1)).max())
    assert np.sqrt(np.mean((f64(lse) - s) ** 2)) <= 2.0 ** -18 * size


@pytest.mark.parametrize("b", [2, 4, 8])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 4, 12])
def test_outputs_keep_their_bits(cuda_ok, b, d, n):
    """fp32 with q = 0: the output is the values' mean, each partial sum at most the rows' size."""
    c = attn_case(62, [96, 40, 7], n, 4, 2, d, 4, b, 16, "f32", drafted=False)
    p, pool, table, lens, q = c[:5]
    q.zero_()
    out, lse = run_attn(c)
    R = oracle.rotation_matrix(d, p.rot_seed)
    held = [s[1] for s in stored_rows(p, pool, table, lens)]
    size = 2 * np.sqrt(np.mean(np.concatenate([v.reshape(-1) for v in held]) ** 2))
    for i, v in enumerate(held):
        want = np.repeat((v.mean(1) @ R), 2, axis=0)  # [4][d]
        assert np.sqrt(np.mean((f64(out)[i] - want) ** 2)) <= 2.0 ** -18 * size
        assert np.abs(f64(lse)[i] - math.log(lens[i])).max() <= 2.0 ** -21 * max(1.0, math.log(lens[i]))


# ---- streams, graphs, devices ------------------------------------------------------------------------

def test_captured_calls_follow_lengths_and_positions(cuda_ok):
    rng = np.random.default_rng(50)
    B, nq, nkv, d, ps = 2, 8, 2, 128, 32
    cap = 200
    table, n_pages = make_table(rng, [cap, cap], ps, extra_width=0)
    p = api.make_pages(n_pages, ps, nkv, d, 4, 4, rot_seed=9)
    pool, pool2 = api.new_pool(p), api.new_pool(p)
    fill_random(rng, p, pool)
    pool2.copy_(pool)
    freq = torch.from_numpy(api.rope_freqs(d, 500000.0)[0]).cuda()
    lens, pos = i32([60, 0]), i32([60, 0])
    q, k, v = rows(rng, (B, 1, nq, d), "bf16"), rows(rng, (B, 1, nkv, d), "bf16"), rows(rng, (B, 1, nkv, d), "bf16")
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    lse = torch.empty(B, 1, nq, device="cuda")
    ws = api.new_tree_workspace(p, B, 1, nq, table.shape[1])

    def step(pool, lens, pos, out, lse, ws):
        api.rope(q[:, 0], k[:, 0], pos, freq, qr[:, 0], kr[:, 0])
        api.tree_attn(p, pool, table, lens, qr, out, ws, k=kr, v=v, lse=lse)
        api.pages_append(p, pool, table, lens, kr, v)
        lens.add_(1), pos.add_(1)

    want = []
    l2, p2 = lens.clone(), pos.clone()
    xs = [(rows(rng, q.shape, "bf16"), rows(rng, k.shape, "bf16"), rows(rng, k.shape, "bf16")) for _ in range(70)]
    for x in xs:
        q.copy_(x[0]), k.copy_(x[1]), v.copy_(x[2])
        step(pool2, l2, p2, out, lse, ws)
        want.append((out.clone(), lse.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            step(pool, lens, pos, out, lse, ws)
    for x, w in zip(xs, want):
        q.copy_(x[0]), k.copy_(x[1]), v.copy_(x[2])
        graph.replay()
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    assert torch.equal(pool, pool2) and lens.tolist() == [130, 70]
    api.check_ws(ws)


def test_two_streams_with_their_own_workspaces(cuda_ok):
    cs = [attn_case(60 + i, [1500 + 100 * i], 4, 16, 2, 128, 4, 4, 64, "bf16") for i in range(2)]
    want = [run_attn(c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    bufs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]
    wss = [api.new_tree_workspace(c[0], 1, 4, 16, c[2].shape[1]) for c in cs]
    ls = [i32(c[3]) for c in cs]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s, b, ws, l in zip(cs, streams, bufs, wss, ls):
            api.tree_attn(c[0], c[1], c[2], l, c[4], b[0], ws, k=c[5], v=c[6], mask=c[7], lse=b[1], stream=s.cuda_stream)
    torch.cuda.synchronize()
    for b, w in zip(bufs, want):
        assert torch.equal(b[0], w[0]) and torch.equal(b[1], w[1])


# ---- together ------------------------------------------------------------------------------------------

def test_drafted_tree_over_a_compressed_prefill_and_a_tail(cuda_ok):
    """The run as a serving loop makes it: a compressed prefill with pre-RoPE keys, a tail in pages, a
    drafted tree over both; then the accepted path is appended and the next token decoded, and the
    tail is read back, against dense attention over all of it in 64 bits."""
    from synth import get_workload, make_kv, make_inv_freq
    from cache_io import oracle_cells, cells_to_device
    w = get_workload("llama8b_64k_b4", n_layers=4, T=300, batch=1)
    s = api.make_shape(w)
    rng = np.random.default_rng(70)
    K, V = make_kv(w, device="cuda")
    choices = [(64, 64, 4)] * api.n_cells(s)
    cells = oracle_cells(w, K, V, choices, s.rot_seed)
    cache = cells_to_device(s, w, cells, choices)
    inv = make_inv_freq(w.d_h, w.rope_theta)
    inv_t = torch.from_numpy(inv).cuda()
    ws = api.new_workspace(s, api.JOLT_OP_DECODE)
    layer, n, nq, nkv, d = 1, 5, w.n_q, w.n_kv, w.d_h
    table, n_pages = make_table(rng, [90], 16)
    p = api.make_pages(n_pages, 16, nkv, d, 8, 8, rot_seed=s.rot_seed)
    pool = api.new_pool(p)
    tws = api.new_tree_workspace(p, 1, n, nq, table.shape[1])

    # the prefill's dense keys and values as its cells hold them, keys rotated to their positions
    cell_k, cell_v = cells[0], cells[1]
    Kd = oracle.rope(oracle.decompress_cell(cell_k, s.rot_seed)[layer], np.arange(w.T), inv)
    Vd = oracle.decompress_cell(cell_v, s.rot_seed)[layer]
    tail_k, tail_v = rows(rng, (1, 70, nkv, d), "bf16"), rows(rng, (1, 70, nkv, d), "bf16")

    def positions(first, count):
        return torch.arange(first, first + count, dtype=torch.int32, device="cuda")

    _, tk = api.rope(None, tail_k[0], positions(w.T, 70), inv_t)
    api.pages_append(p, pool, table, i32([0]), tk[None], tail_v)
    lens = [70]
    parents = [-1, 0, 0, 1, 3]
    depth = [0, 1, 1, 2, 3]
    for step in range(2):
        m = n if step == 0 else 1
        q, k, v = (rows(rng, (1, m, h, d), "bf16") for h in (nq, nkv, nkv))
        pos = i32([w.T + lens[0] + (depth[i] if step == 0 else 0) for i in range(m)])
        q2, k2 = api.rope(q[0], k[0], pos, inv_t)
        q2, k2 = q2[None], k2[None]
        pre, pre_lse = torch.empty_like(q2), torch.empty(1, m, nq, device="cuda")
        for i in range(m):
            o, l = torch.empty(1, 1, nq, d, dtype=q.dtype, device="cuda"), torch.empty(1, 1, nq, device="cuda")
            api.decode_attn(s, choices, cache, q2[:, i:i + 1].contiguous(), o, ws, lse=l, inv_freq=inv_t,
                            layer_begin=layer, n_layers_call=1)
            pre[:, i], pre_lse[:, i] = o[:, 0], l[:, 0]
        api.check_ws(ws)
        mask = torch.from_numpy(api.tree_mask(parents[:m]).view(np.int64)).cuda()[None] if m > 1 else None
        out, lse = torch.empty_like(q2), torch.empty(1, m, nq, device="cuda")
        api.tree_attn(p, pool, table, i32(lens), q2, out, tws, k=k2, v=v, mask=mask, lse=lse, prefix_out=pre,
                      prefix_lse=pre_lse, attn_scale=s.attn_scale)
        api.check_ws(tws)
        R = oracle.rotation_matrix(d, s.rot_seed)
        (ky, vy), = stored_rows(p, pool, table, lens)
        for i in range(m):
            sees = [j for j in range(m) if (api.tree_mask(parents[:m])[i] >> np.uint64(j)) & np.uint64(1)]
            Ka = np.concatenate([Kd, ky @ R, f64(k2)[0, sees].transpose(1, 0, 2)], axis=1)
            Va = np.concatenate([Vd, vy @ R, f64(v)[0, sees].transpose(1, 0, 2)], axis=1)
            ro, rl = oracle.decode_attention(Ka, Va, f64(q2)[0, i], s.attn_scale)
            got = f64(out)[0, i]
            # decode attention over the compressed prefill is held to 1e-2 of its largest output
            assert np.abs(got - ro).max() <= 1e-2 * np.abs(ro).max()
            assert np.abs(f64(lse)[0, i] - rl).max() <= 1e-3 * np.abs(rl).max()
        if step == 0:
            api.pages_append(p, pool, table, i32(lens), k2, v, counts=i32([3]), src=i32([[0, 1, 3]]), n_new=3)
            lens = [73]
    back = torch.empty(1, nkv, 73, d, dtype=torch.bfloat16, device="cuda")
    api.pages_read(p, pool, table, i32(lens), back, None)
    plain, _ = api.rope(back[0].transpose(0, 1).contiguous(), None, positions(w.T, 73), inv_t, inverse=True)
    # 8 bits of a row: half a step is (max - min) / 510 of the rotated row, at most its norm / 255 / sqrt(2)
    want = f64(tail_k)[0]
    off = np.abs(f64(plain)[:70] - want).max()
    assert off <= np.linalg.norm(want, axis=-1).max() * (1 / 255 + 2 * HALF_STEP["bf16"])
