"""GPU: the tail cache's loops in their steady state (many tiles a block, rows a warp, rounds of barriers), against
64-bit forms with bounds of the errors' own size."""
import math

import numpy as np
import pytest
import torch

import oracle
from long_context_st_b200 import api
from tail_ref import NP, rows, f64, make_table, i32, fill_random
from tail_bounds import HALF, attention64, check64, coded_rows, ratios
from test_gpu_tail import attn_case, run_attn

pytestmark = pytest.mark.gpu


def scale_zero(p, pool, table, b, t, which):
    """(scale, zero) [n_kv][2] of token t of sequence b, keys (0) or values (1): a view of the pool."""
    off, size = api.pages_layout(p)
    page = pool[:p.n_pages * size].view(p.n_pages, size)[int(table[b, t // p.page_size])]
    at = off[2 * which + 1]
    return page[at:at + p.n_kv * p.page_size * 4].view(torch.float16).view(p.n_kv, p.page_size, 2)[:, t % p.page_size]


@pytest.mark.parametrize("n,io", [(3, "bf16"), (8, "bf16"), (16, "bf16"), (17, "bf16"), (40, "bf16"), (3, "f32"), (17, "f32")])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("b", [2, 4, 8])
@pytest.mark.parametrize("at", [(5,), (300,), (130, 599)])
def test_large_values_without_weight_cost_the_others_nothing(cuda_ok, n, io, d, b, at):
    """Value rows 2^12 times the others whose scores are far below theirs: the outputs are as exact as without."""
    c = attn_case(9 + d, [600], n, 1, 1, d, 8, b, 64, io, drafted=False)
    p, pool, table, lens, q = c[:5]
    # a key of codes' scale 0 and zero -40 scores -40 sum(R q), and the queries get a part along R^T 1
    q += (0.6 * torch.ones(d, dtype=torch.float64) @ torch.from_numpy(oracle.rotation_matrix(d, p.rot_seed))).to(q)
    for t in at:
        scale_zero(p, pool, table, 0, t, 0).copy_(torch.tensor([0.0, -40.0]))
        v = scale_zero(p, pool, table, 0, t, 1)
        v.copy_(v.float() * 4096)
    out, lse = run_attn(c)
    ref = attention64(p, pool, table, lens, q)
    check64(out, lse, ref)
    # in the mean of the squares: the output's rounding, and a third of the bound of what comes before it
    err, norm = (out.double() - ref[0]).norm(dim=-1), ref[0].norm(dim=-1)
    own = (ref[0].to(out.dtype).double() - ref[0]).norm(dim=-1)
    before = (ref[2] - HALF[out.dtype] * norm) / 3
    assert float(err.square().mean()) <= float((own.square() + before.square()).mean())


def test_one_workspace_serves_every_smaller_call(cuda_ok):
    """A workspace made once for the largest batch and tree, whatever earlier calls left in it."""
    p0 = api.make_pages(1, 16, 8, 64, 4, 4)
    ws = api.new_tree_workspace(p0, 40, 20, 16, 60)
    ws[256:] = 0xFF
    for batch, n, width in ((40, 20, 60), (38, 1, 60), (37, 1, 60), (19, 9, 31), (18, 9, 60), (16, 2, 60), (5, 20, 60), (1, 1, 1)):
        lens = [(1 + 611 * i) % (16 * width) for i in range(batch)]
        c = attn_case(batch + n, lens, n, 16, 8, 64, 4, 4, 16, "bf16")
        t = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
        t[:, :c[2].shape[1]] = c[2][:, :width]
        c = c[:2] + (t,) + c[3:]
        got, want = run_attn(c, ws=ws), run_attn(c)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- many tiles a block -------------------------------------------------------------------------------
# A batch with more (sequence, KV head) pairs than blocks that fit the GPU at once leaves every sequence one split, so a
# block of the tcgen05 form goes through ceil(length / 128) tiles and a warp of the other through ceil(length / 256).

def hold(c, tight=True, drops=()):
    """Holds a call to its bounds, and sees that a reference without one of these tokens is told apart."""
    p, pool, table, lens, q, k, v, mask, cnt, pre = c
    counts = None if cnt is None else cnt.tolist()
    got = run_attn(c)
    check64(*got, attention64(p, pool, table, lens, q, k, v, mask, counts, prefix=pre), counts, tight)
    for b, t in drops:
        one = [None if x is None else x[b:b + 1] for x in (table, lens, q, k, v, mask, counts)]
        ref = attention64(p, pool, *one, prefix=None if pre is None else [x[b:b + 1] for x in pre], drop=[(0, t)])
        assert max(ratios(got[0][b:b + 1], got[1][b:b + 1], ref, one[-1])) > 1, (b, t)
    return got


@pytest.mark.parametrize("io,n", [("bf16", 1), ("bf16", 4), ("bf16", 5), ("bf16", 9), ("bf16", 17), ("bf16", 40), ("f32", 1),
                                  ("f32", 4), ("f32", 5), ("f32", 9), ("f32", 17), ("f32", 40)])
@pytest.mark.parametrize("d,bk,bv,ps", [(64, 2, 2, 16), (64, 4, 4, 128), (64, 8, 2, 32), (128, 8, 8, 64), (128, 4, 8, 16)])
def test_many_tiles_a_block(cuda_ok, io, n, d, bk, bv, ps):
    lens = [3000 - 149 * i for i in range(20)]
    c = attn_case(n * 3 + bk, lens, n, 16, 16, d, bk, bv, ps, io, counts=[n - (i % 4 == 3) for i in range(20)])
    hold(c, drops=[(0, 2999), (2, lens[2] - 1), (0, 127), (0, 1279), (1, 2303), (1, 0), (4, ps - 1)])  # of sequences that have rows


@pytest.mark.parametrize("n", [1, 5, 9, 17, 40])
@pytest.mark.parametrize("b", [2, 4, 8])
def test_rising_scores_and_changing_value_scales_over_many_tiles(cuda_ok, n, b):
    """Keys whose scales grow to eight times, so that references are raised again and again; values 64 times as
    large from tile 5 to tile 9, so that the unit of the sums changes late and stays above what follows."""
    lens = [2500 - 131 * i for i in range(20)]
    c = attn_case(n + b, lens, n, 16, 16, 64, 8, b, 32, "bf16")
    p, pool, table = c[:3]
    off, size = api.pages_layout(p)
    pages = pool.view(p.n_pages, size)
    for s, length in enumerate(lens):
        for i in range(-(-length // 32)):
            t = i * 32 + torch.arange(32, device="cuda").float()
            page = pages[int(table[s, i])]
            for seg, f in ((1, 1 + 7 * t / 2500), (3, torch.where((t >= 640) & (t < 1280), 64.0, 1.0))):
                sz = page[off[seg]:off[seg] + 16 * 32 * 4].view(torch.float16).view(16, 32, 2)
                sz.copy_((sz.float() * f[None, :, None]).half())
    hold(c, tight=False)


@pytest.mark.parametrize("io,n", [("bf16", 1), ("bf16", 17), ("f32", 17)])
def test_splits_of_two_long_sequences(cuda_ok, io, n):
    c = attn_case(71, [5003, 3001], n, 16, 16, 64, 8, 8, 16, io, prefix=True)
    # splits have 9 tiles of 128 tokens with tcgen05, 14 or 15 of 32 (f32: 28) otherwise
    hold(c, drops=[(0, 5002), (1, 3000)] + [(0, k * 128 - 1) for k in (1, 9, 18, 27)] + [(0, k * 32) for k in (14, 15, 28, 56)])


@pytest.mark.parametrize("io,n,batch", [("bf16", 17, 30), ("bf16", 17, 150), ("bf16", 2, 30), ("f32", 12, 150)])
def test_equal_weights_count_every_token(cuda_ok, io, n, batch):
    """q = 0: the log-sum-exp is the logarithm of the length and the output the values' mean."""
    around = [0, 1, 2] + [k * 128 + x for k in (1, 2, 3, 4, 5, 8, 9, 12) for x in (-1, 0, 1)] + [31, 33, 1800]
    lens = [around[i % len(around)] for i in range(batch)]
    c = attn_case(73, lens, n, 2, 2, 64, 4, 4, 16, io, drafted=False)
    c[4].zero_()
    _, lse = hold(c)
    for b, length in enumerate(lens):
        if length:
            assert float((lse[b].exp().double() - length).abs().max()) < 0.05


def test_captured_tree_follows_lengths_and_counts(cuda_ok):
    """bf16 of 20 rows: one graph over lengths that grow from nothing past many tiles, and counts that change."""
    full = [2100, 900, 1500]
    c = attn_case(75, full, 20, 4, 4, 64, 4, 4, 16, "bf16")
    p, pool, table, _, q, k, v, mask, _, _ = c
    ws = api.new_tree_workspace(p, 3, 20, 4, table.shape[1])
    lens, cnt = i32([0, 0, 0]), i32([20, 20, 20])
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        api.tree_attn(p, pool, table, lens, q, out, ws, k=k, v=v, mask=mask, counts=cnt, lse=lse)
    for now, many in (([0, 0, 0], [20, 20, 20]), ([1, 900, 128], [20, 0, 3]), (full, [20, 19, 1]), ([129, 0, 1500], [1, 20, 20]),
                      ([0, 0, 1], [0, 0, 5])):
        lens.copy_(i32(now)), cnt.copy_(i32(many))
        out.fill_(9), lse.fill_(9)
        graph.replay()
        check64(out, lse, attention64(p, pool, table, now, q, k, v, mask, many), many, tight=False)
        for b, m in enumerate(many):
            assert bool((out[b, m:] == 9).all()) and bool((lse[b, m:] == 9).all())
    api.check_ws(ws)


# ---- pages and lengths that are not there ---------------------------------------------------------------

@pytest.mark.parametrize("io,n", [("f32", 2), ("bf16", 2), ("bf16", 9), ("bf16", 20)])
@pytest.mark.parametrize("ps", [16, 64])
def test_bad_pages_and_lengths_give_what_is_documented(cuda_ok, io, n, ps):
    """Tokens of a page that the table does not name are invisible, a length below 0 holds nothing and one past the
    table all that the table names; each is reported."""
    c = attn_case(77, [1500, 333], n, 4, 2, 64, 4, 8, ps, io, extra=2)
    p, pool, table, lens, q, k, v, mask, _, _ = c
    ws = api.new_tree_workspace(p, 2, n, 4, table.shape[1])

    def call(t, now, same):
        out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:3], 9.0, device="cuda")
        api.tree_attn(p, pool, t, i32(now), q, out, ws, k=k, v=v, mask=mask, lse=lse)
        with pytest.raises(api.JoltError) as e:
            api.check_ws(ws)
        assert e.value.status == -1
        ws[:4] = 0
        check64(out, lse, attention64(p, pool, t, same, q, k, v, mask), tight=False)

    for bad in (p.n_pages, -1, 2 ** 31 - 1, -2 ** 31):
        for entries in ([(0, 0)], [(0, 1)], [(0, 2), (0, 3)], [(1, 0), (0, 1400 // ps), (0, 1499 // ps)]):
            t = table.clone()
            for s, i in entries:
                t[s, i] = bad
            call(t, lens, lens)
    most = table.shape[1] * ps
    for now, same in (([-3, 333], [0, 333]), ([-2 ** 31, -1], [0, 0]), ([1500, 10 ** 6], [1500, most]),
                      ([2 ** 31 - 1, most + 1], [most, most])):
        call(table, now, same)


# ---- many rows a warp -----------------------------------------------------------------------------------

@pytest.mark.parametrize("io,d,bk,bv,ps", [("bf16", 128, 8, 4, 64), ("f32", 64, 2, 8, 16), ("bf16", 64, 4, 2, 128)])
def test_append_of_many_rows_is_the_codec_bit_for_bit(cuda_ok, io, d, bk, bv, ps):
    """45000 rows of each kind, where a round of the grid takes 18944; rows that are not written among them."""
    rng = np.random.default_rng(81)
    n, nkv, lens, counts = 5000, 3, [13, 0, 900], [5000, 4999, 4001]
    table, n_pages = make_table(rng, [a + n for a in lens], ps)
    p = api.make_pages(n_pages, ps, nkv, d, bk, bv, io_dtype=io, rot_seed=7)
    pool = api.new_pool(p)
    pool.fill_(0xA5)
    k, v = rows(rng, (3, n, nkv, d), io, True), rows(rng, (3, n, nkv, d), io)
    bad = table.clone()
    bad[1, 4000 // ps] = n_pages  # sequence 1 has no page there
    err = i32([0])
    api.pages_append(p, pool, bad, i32(lens), k, v, counts=i32(counts), err=err)
    assert int(err) == -1
    want = torch.full_like(pool, 0xA5).view(n_pages, -1)
    off, _ = api.pages_layout(p)
    for x, which, b in ((k, 0, bk), (v, 1, bv)):
        codes, sz, e = api.quantize_pack(api.rotate_rows(x.float().view(-1, d).contiguous(), 7), b)
        assert int(e) == 0
        rb, first = d * b // 8, off[2 * which]
        c = want[:, first:first + nkv * ps * rb].unflatten(-1, (nkv, ps, rb))
        z = want[:, off[2 * which + 1]:off[2 * which + 1] + nkv * ps * 4].unflatten(-1, (nkv, ps, 4))
        for s in range(3):
            t = lens[s] + torch.arange(counts[s], device="cuda")
            page = bad[s].long()[t // ps]
            ok = page < n_pages
            c[page[ok], :, (t % ps)[ok]] = codes.view(3, n, nkv, rb)[s, :counts[s]][ok]
            z[page[ok], :, (t % ps)[ok]] = sz.view(torch.uint8).view(3, n, nkv, 4)[s, :counts[s]][ok]
    assert torch.equal(pool, want.view(-1))


@pytest.mark.parametrize("io,d,bk,bv,ps", [("bf16", 64, 4, 8, 16), ("bf16", 128, 2, 4, 64), ("f32", 64, 8, 2, 32)])
def test_read_of_many_tiles(cuda_ok, io, d, bk, bv, ps):
    """600 tokens of 40 sequences and 32 heads: one block a line, so a warp has five tiles of 16; a page that is not
    there in its fourth."""
    rng = np.random.default_rng(83)
    B, nkv, n = 40, 32, 600
    lens = [700 - 17 * (i % 30) for i in range(B)]
    start = [(5 * i) % 47 for i in range(B)]
    table, n_pages = make_table(rng, lens, ps)
    p = api.make_pages(n_pages, ps, nkv, d, bk, bv, io_dtype=io, rot_seed=12)
    pool = api.new_pool(p)
    fill_random(rng, p, pool)
    gone = 450 // ps
    table[3, gone] = -1
    k_out, v_out = (torch.full((B, nkv, n, d), 7.0, dtype=NP[io], device="cuda") for _ in range(2))
    err = i32([0])
    api.pages_read(p, pool, table, i32(lens), k_out, v_out, start=i32(start), err=err)
    assert int(err) == -1
    R = torch.from_numpy(oracle.rotation_matrix(d, 12)).cuda()
    for b in range(B):
        m = min(n, lens[b] - start[b])
        for o, (c, s, z) in zip((k_out, v_out), coded_rows(p, pool, table, b, lens[b])):
            y = (c * s[..., None] + z[..., None])[:, start[b]:start[b] + m]
            there = torch.isfinite(y[0, :, 0])
            x = y[:, there] @ R
            got = o[b, :, :m].double()
            # a dequantised value is rounded once, the rotation adds d of them in log2(d) fp32 roundings
            size = float(y[:, there].abs().max()) * math.sqrt(d)
            assert float(((got[:, there] - x).abs() - HALF[NP[io]] * x.abs()).max()) <= (math.log2(d) + 3) * 2.0 ** -24 * size
            assert bool((got[:, ~there] == 7).all()) and bool((o[b, :, m:] == 7).all())
            assert bool(there.all()) == (b != 3)


def test_kernel_timing_sees_the_tail_caches_calls(cuda_ok):
    c = attn_case(91, [100, 30], 3, 4, 2, 64, 4, 8, 16, "bf16")
    p, pool, table, lens, q, k, v = c[:7]
    back = torch.empty(2, 2, 100, 64, dtype=torch.bfloat16, device="cuda")
    pos, freq = i32([0, 1, 2]), torch.ones(32, device="cuda")
    api.stats_read(reset=True)
    api.stats_enable(True)
    try:
        api.rope(q[0], k[0], pos, freq)
        run_attn(c)
        api.pages_read(p, pool, table, i32(lens), back, back.clone())
        api.pages_read(p, pool, table, i32(lens), back, None)
        api.pages_append(p, pool, table, i32([0, 0]), k, v)
    finally:
        api.stats_enable(False)
    s = api.stats_read(reset=True)
    assert (s["rope"]["launches"], s["pages"]["launches"], s["tree"]["launches"]) == (1, 3, 1)
    assert all(s[f]["ms"] > 0 for f in ("rope", "pages", "tree"))
    assert s["rope"]["bytes"] == 3 * (2 * 6 * 64 * 2 + 4)
    k_row, v_row = 64 * 4 // 8 + 4 + 64 * 2, 64 * 8 // 8 + 4 + 64 * 2
    assert s["pages"]["bytes"] == 2 * 2 * (100 * (k_row + v_row) + 100 * k_row + 3 * (k_row + v_row))


# ---- what one row or caller does to the others ------------------------------------------------------------

@pytest.mark.parametrize("io,n", [("f32", 3), ("bf16", 3), ("bf16", 7), ("bf16", 12), ("f32", 20), ("bf16", 20), ("bf16", 40)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_not_finite_stays_on_its_own(cuda_ok, io, n, bad):
    c = attn_case(93, [700, 40], n, 4, 4, 128, 4, 4, 32, io, prefix=True)
    p, pool, table, lens, q, k, v, mask, cnt, pre = c
    ref = attention64(p, pool, table, lens, q, k, v, mask, prefix=pre)
    rows_ = ((0, n // 2, 1, 5), (0, 0, 2, 0), (1, n - 1, 0, 127))
    for b, i, h, e in rows_:
        q[b, i, h, e] = bad
    out, lse = run_attn(c)
    for b, i, h, _ in rows_:
        assert bool(out[b, i, h].isnan().all()) and not math.isfinite(float(lse[b, i, h]))
        out[b, i, h], lse[b, i, h] = ref[0][b, i, h].to(out.dtype), ref[1][b, i, h].float()
    check64(out, lse, ref, tight=False)


@pytest.mark.parametrize("n", [1, 20])
def test_broadcast_inputs(cuda_ok, n):
    """One set of queries and drafted rows for all sequences (stride 0)."""
    c = attn_case(95, [300, 0, 77], n, 8, 4, 64, 4, 4, 16, "bf16")
    p, pool, table, lens, q, k, v, mask, _, _ = c
    q1, k1, v1, m1 = (x[:1].expand(3, *x.shape[1:]) for x in (q, k, v, mask))
    want = run_attn(c[:4] + (q1.contiguous(), k1.contiguous(), v1.contiguous(), m1.contiguous(), None, None))
    ws = api.new_tree_workspace(p, 3, n, 8, table.shape[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    api.tree_attn(p, pool, table, i32(lens), q1, out, ws, k=k1, v=v1, mask=m1.contiguous(), lse=lse)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(api.JoltError):
        api.tree_attn(p, pool, table, i32(lens), q1, out, ws, k=k1, v=v1, mask=m1, lse=lse)


def test_calls_at_once_of_both_forms_repeat_bit_for_bit(cuda_ok):
    """Trees of both forms, and a read, on four streams, over and over, with workspaces of their own."""
    cs = [attn_case(96 + i, [2000 + 300 * i, 500], n, 8, 4, 128, 4, 4, 64, io)
          for i, (n, io) in enumerate(((20, "bf16"), (20, "bf16"), (1, "bf16"), (9, "f32")))]
    want = [run_attn(c) for c in cs]
    p, pool, table, lens = cs[0][:4]
    back = torch.empty(2, 4, 1500, 128, dtype=torch.bfloat16, device="cuda")
    api.pages_read(p, pool, table, i32(lens), back, None)
    want_back = back.clone()
    streams = [torch.cuda.Stream() for _ in cs]
    bufs = [(torch.empty_like(w[0]), torch.empty_like(w[1])) for w in want]
    wss = [api.new_tree_workspace(c[0], 2, c[4].shape[1], 8, c[2].shape[1]) for c in cs]
    ls = [i32(c[3]) for c in cs]
    torch.cuda.synchronize()
    for _ in range(30):
        for c, s, b, ws, l in zip(cs, streams, bufs, wss, ls):
            api.tree_attn(c[0], c[1], c[2], l, c[4], b[0], ws, k=c[5], v=c[6], mask=c[7], lse=b[1], stream=s.cuda_stream)
        api.pages_read(p, pool, table, ls[0], back, None, stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    for b, w, ws in zip(bufs, want, wss):
        api.check_ws(ws)
        assert torch.equal(b[0], w[0]) and torch.equal(b[1], w[1])
    assert torch.equal(back[:, :, :500], want_back[:, :, :500])


# ---- offsets past 32 bits -----------------------------------------------------------------------------------

@pytest.mark.parametrize("io,n", [("bf16", 2), ("bf16", 20), ("f32", 9)])
def test_a_pool_past_four_gigabytes(cuda_ok, io, n):
    """The same pages at the end of a 5.4 GB pool and in one of their own: written, attended to and read back alike."""
    rng = np.random.default_rng(97)
    lens, new, nkv, d, ps = [900, 130], 40, 8, 128, 128
    table, few = make_table(rng, [x + new for x in lens], ps)
    small = api.make_pages(few, ps, nkv, d, 8, 8, io_dtype=io, rot_seed=5)
    big = api.make_pages(20000, ps, nkv, d, 8, 8, io_dtype=io, rot_seed=5)
    assert api.pages_bytes(big) > 5 << 30
    far = torch.where(table >= 0, table + (20000 - few), table)
    pools = api.new_pool(small), api.new_pool(big)
    fill_random(rng, small, pools[0])
    size = api.pages_layout(small)[1]
    pools[1].view(20000, size)[20000 - few:] = pools[0].view(few, size)
    k, v, q = rows(rng, (2, new, nkv, d), io), rows(rng, (2, new, nkv, d), io), rows(rng, (2, n, 16, d), io)
    got = []
    for p, pool, t in ((small, pools[0], table), (big, pools[1], far)):
        err = i32([0])
        api.pages_append(p, pool, t, i32(lens), k, v, err=err)
        now = i32([x + new for x in lens])
        out, lse = torch.empty_like(q), torch.empty(2, n, 16, device="cuda")
        ws = api.new_tree_workspace(p, 2, n, 16, t.shape[1])
        api.tree_attn(p, pool, t, now, q, out, ws, k=k[:, :n].contiguous(), v=v[:, :n].contiguous(), lse=lse)
        api.check_ws(ws)
        back = torch.zeros(2, nkv, 940, d, dtype=NP[io], device="cuda")
        api.pages_read(p, pool, t, now, back, None, err=err)
        assert int(err) == 0
        got.append((out, lse, back, pool.view(-1, size)[-few:].clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_rows_past_two_to_the_31_elements(cuda_ok):
    """Sequences of k, v, q, k_out and rotated heads that lie more than 2^31 elements apart."""
    rng = np.random.default_rng(98)
    nkv, d, far = 2, 128, (1 << 31) + 1024
    store = torch.empty(far + (1 << 20), dtype=torch.bfloat16, device="cuda")

    def apart(x, at):
        y = store[at:].as_strided(x.shape, (far,) + x.stride()[1:])
        y.copy_(x)
        return y

    table, n_pages = make_table(rng, [70, 50], 16)
    p = api.make_pages(n_pages, 16, nkv, d, 4, 4, rot_seed=5)
    k, v, q = rows(rng, (2, 30, nkv, d), "bf16"), rows(rng, (2, 30, nkv, d), "bf16"), rows(rng, (2, 30, 4, d), "bf16")
    k2, v2, q2 = apart(k, 0), apart(v, 1 << 16), apart(q, 1 << 17)
    assert k2.stride(0) > 1 << 31
    got = []
    for a, b, c, at in ((k, v, q, None), (k2, v2, q2, 1 << 18)):
        pool = api.new_pool(p)
        api.pages_append(p, pool, table, i32([0, 0]), a, b)
        out, ws = torch.empty_like(q), api.new_tree_workspace(p, 2, 30, 4, table.shape[1])
        api.tree_attn(p, pool, table, i32([30, 30]), c, out, ws, k=a, v=b)
        api.check_ws(ws)
        back = torch.zeros(2, nkv, 30, d, dtype=torch.bfloat16, device="cuda")
        if at is not None:
            back = apart(back, at)
        api.pages_read(p, pool, table, i32([30, 30]), back, None)
        got.append((pool, out, back))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    pos, freq = i32([5, 70000]), torch.from_numpy(api.rope_freqs(d, 10000.0)[0]).cuda()
    want, _ = api.rope(q[:, 0].contiguous(), None, pos, freq)
    turned, _ = api.rope(q2[:, 0], None, pos, freq, q_out=q2[:, 0])
    assert torch.equal(turned, want)
    # one call over more than 2^31 elements, its last tokens as a call of their own
    n = (far // (8 * d)) + 7
    x = store[:n * 8 * d].view(n, 8, d)
    x[-4:] = rows(rng, (4, 8, d), "bf16")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    want, _ = api.rope(x[-4:].clone(), None, pos[-4:].contiguous(), freq)
    api.rope(x, None, pos, freq, q_out=x)
    assert torch.equal(x[-4:], want)


def test_kernel_timing_leaves_captured_launches_out(cuda_ok):
    """Timing is on while a step is captured: the graph runs, and the timing goes on with what is launched outside."""
    c = attn_case(99, [100], 1, 4, 2, 64, 4, 4, 16, "bf16")
    p, pool, table, lens, q = c[:5]
    ws, n = api.new_tree_workspace(p, 1, 1, 4, table.shape[1]), i32(lens)
    out, want = torch.empty_like(q), run_attn(c[:5] + (None, None, None, None, None))[0]
    api.stats_read(reset=True)
    api.stats_enable(True)
    try:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            api.tree_attn(p, pool, table, n, q, out, ws)
        graph.replay()
        assert torch.equal(out, want)
        api.tree_attn(p, pool, table, n, q, out, ws)
        s = api.stats_read(reset=True)
    finally:
        api.stats_enable(False)
    assert s["tree"]["launches"] == 1 and s["tree"]["ms"] > 0


@pytest.mark.parametrize("io,n", [("bf16", 3), ("bf16", 12), ("bf16", 20), ("bf16", 64), ("f32", 20)])
@pytest.mark.parametrize("d,b", [(64, 2), (128, 4), (64, 8)])
def test_value_scales_over_all_of_fp16(cuda_ok, io, n, d, b):
    """Value scales from 2^-24 to 2^10, constant rows of any size and of zeros, tile after tile."""
    c = attn_case(100 + b, [1500, 300], n, 2, 2, d, 8, b, 16, io)
    p, pool = c[0], c[1]
    off, size = api.pages_layout(p)
    sz = pool.view(p.n_pages, size)[:, off[3]:off[3] + 2 * 16 * 4].view(torch.float16).view(p.n_pages, 2, 16, 2)
    rng = np.random.default_rng(b)
    sz[..., 0] = torch.from_numpy(2.0 ** rng.integers(-24, 11, sz.shape[:3])).half().cuda()
    sz[..., 1] = torch.from_numpy(rng.standard_normal(sz.shape[:3]) * 2.0 ** rng.integers(-20, 11, sz.shape[:3])).half().cuda()
    sz[:, :, ::5, 0] = 0.0
    sz[:, :, 3::7] = 0.0
    hold(c, tight=False)
    sz[:] = 0.0  # no value at all
    out, _ = run_attn(c[:5] + (None, None, None, None, None))
    assert bool((out == 0).all())
