"""What is measured of the paged tail cache and the operators around it.

The tail cache keeps the K and V rows of tokens that come after a compressed prefill: every row is
rotated by (1/sqrt(d)) H D (Hadamard times seeded signs), quantised to b bits with an fp16 scale and
zero, and kept in pages. Around it: rotary positions of queries and keys, the write of new rows, the
read back to dense rows, and attention of one or several drafted tokens over the pages, the drafted
tokens themselves (a 64-bit ancestor mask a token) and the partial result of a compressed prefix.

Layout of a page (page_size tokens): K codes [n_kv][page_size][d*b_k/8], K (scale, zero) fp16
[n_kv][page_size][2], V codes, V (scale, zero); pages start at multiples of 256 bytes. Code j of a
row sits at bits [(j*b) mod 8, +b) of byte floor(j*b/8). Position t of sequence s is row
t % page_size of page table[s][t // page_size].
"""
import math

import numpy as np
import torch

own = False

_IO = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoding step of four sequences: latency
        dict(name="rope_step", op="rope", tokens=4, n_q=32, n_kv=8, d=128, rot=128, layout="half", io="bf16",
             inverse=False, far=65536),
        # a prompt chunk of the 70B-shaped workload
        dict(name="rope_prompt", op="rope", tokens=8192, n_q=64, n_kv=8, d=128, rot=128, layout="half", io="bf16",
             inverse=False, far=131072),
        # the backward pass in training precision, half of each head rotated, pairs interleaved, odd length
        dict(name="rope_grad_part", op="rope", tokens=5003, n_q=32, n_kv=8, d=128, rot=64, layout="interleaved",
             io="f32", inverse=True, far=32768),
        # one decoding step writes one token of each sequence, and reads it back
        dict(name="write_step", op="write", batch=4, n_new=1, n_kv=8, d=128, b_k=4, b_v=4, page=64, io="bf16",
             start=1000),
        # a long chunk of a prompt is written, keys at 8 bits and values at 4, from an odd position
        dict(name="write_chunk", op="write", batch=1, n_new=8191, n_kv=8, d=128, b_k=8, b_v=4, page=64, io="bf16",
             start=77),
        # a tail is read back to be folded into a compressed cache
        dict(name="read_fold", op="read", batch=1, tokens=65536, n_kv=8, d=128, b_k=4, b_v=4, page=64, io="bf16"),
        # small heads, two bits, fp32, small pages, odd length
        dict(name="read_small", op="read", batch=3, tokens=259, n_kv=2, d=64, b_k=2, b_v=8, page=16, io="f32"),
        # one token over a short tail, fp32: latency
        dict(name="attn_toy", op="attn", batch=1, tokens=256, n_new=1, n_q=8, n_kv=2, d=64, b_k=4, b_v=4, page=16,
             io="f32", prefix=True),
        # one token of each of four sequences over long ragged tails, joined with the compressed prefix
        dict(name="attn_step_64k", op="attn", batch=4, tokens=65536, n_new=1, n_q=32, n_kv=8, d=128, b_k=4, b_v=4,
             page=64, io="bf16", prefix=True),
        # a tree of 16 drafted tokens a sequence
        dict(name="attn_tree_8k", op="attn", batch=4, tokens=8192, n_new=16, n_q=32, n_kv=8, d=128, b_k=4, b_v=4,
             page=64, io="bf16", prefix=True),
        # a tree of 32 drafted tokens, 64 query heads, the longest context
        dict(name="attn_tree_128k", op="attn", batch=1, tokens=131072, n_new=32, n_q=64, n_kv=8, d=128, b_k=4, b_v=4,
             page=64, io="bf16", prefix=False),
        # odd sizes throughout, mixed bits, fp32, small pages
        dict(name="attn_tree_odd", op="attn", batch=7, tokens=1537, n_new=13, n_q=12, n_kv=4, d=128, b_k=8, b_v=2,
             page=16, io="f32", prefix=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "write", "read", "attn", "attn"])
    heads = rng.choice([(8, 2), (32, 8), (64, 8), (12, 4), (16, 1), (6, 6)])
    d = rng.choice([64, 128])
    io = rng.choice(["bf16", "bf16", "f32"])
    bits = (rng.choice([2, 4, 8]), rng.choice([2, 4, 8]))
    page = rng.choice([16, 32, 64, 128])
    if op == "rope":
        return dict(op=op, tokens=_log(rng, 1, 8000), n_q=heads[0], n_kv=heads[1], d=d,
                    rot=rng.choice([d, d // 2, d // 4]), layout=rng.choice(["half", "interleaved"]), io=io,
                    inverse=rng.random() < 0.5, far=_log(rng, 8192, 1000000))
    if op == "write":
        # what is quantised is compared as the bf16 values it stands for: a value next to a rounding
        # border of the quantiser has no fp32 answer that does not hang on the last bit
        batch = rng.randint(1, 8)
        return dict(op=op, batch=batch, n_new=_log(rng, 1, 8191 // batch), n_kv=heads[1], d=d, b_k=bits[0],
                    b_v=bits[1], page=page, io="bf16", start=rng.randint(0, 3000))
    batch = rng.randint(1, 8)
    if op == "read":
        return dict(op=op, batch=batch, tokens=_log(rng, 1, 65000 // batch), n_kv=heads[1], d=d, b_k=bits[0],
                    b_v=bits[1], page=page, io=io)
    n_new = rng.choice([1, 1, 2, 5, 8, 16, 31, 64])
    most = min(131072, 131072 * 32 * 64 // (n_new * heads[0])) // batch
    return dict(op=op, batch=batch, tokens=_log(rng, 1, min(most, 100000)), n_new=n_new, n_q=heads[0], n_kv=heads[1],
                d=d, b_k=bits[0], b_v=bits[1], page=page, io=io, prefix=rng.random() < 0.5)


# ---- what a case fixes: lengths, counts, sizes ----------------------------------------------------

def _lens(c):
    """Cached tokens of each sequence: ragged, the first the longest."""
    return [max(0, c["tokens"] - (c["tokens"] * i) // (2 * c["batch"]) - (i % 3)) for i in range(c["batch"])]


def _counts(c):
    """Drafted tokens of each sequence: the last sequence of a batch has fewer."""
    n = [c["n_new"]] * c["batch"]
    if c["batch"] > 1 and c["n_new"] > 1:
        n[-1] = c["n_new"] // 2
    return n


def _layout(c):
    """Byte offsets of K codes, K (scale, zero), V codes, V (scale, zero) in a page, and the page's bytes."""
    rows, at, off = c["n_kv"] * c["page"], 0, []
    for size in (rows * c["d"] * c["b_k"] // 8, rows * 4, rows * c["d"] * c["b_v"] // 8, rows * 4):
        off.append(at)
        at += size
    return off, (at + 255) // 256 * 256


def _signs(d, seed):
    """The sign diagonal D: bit 63 of SplitMix64's mix of seed * 2^32 + j."""
    with np.errstate(over="ignore"):
        z = (np.uint64(seed) << np.uint64(32)) + np.arange(d, dtype=np.uint64) + np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    return np.where(z >> np.uint64(63), -1.0, 1.0)


def _rotation(d, seed, device="cuda"):
    """R = (1/sqrt(d)) H D in 64 bits, H[i][j] = (-1)^popcount(i & j)."""
    i = np.arange(d)
    both = i[:, None] & i[None, :]
    odd = ((both[..., None] >> np.arange(8)) & 1).sum(-1) & 1
    return torch.from_numpy((1.0 - 2.0 * odd) * _signs(d, seed)[None, :] / math.sqrt(d)).to(device)


# ---- the plain form -------------------------------------------------------------------------------

def _quantise(x, rot, b):
    """Rows x [..., d] -> (packed codes [..., d*b/8] uint8, (scale, zero) fp16 [..., 2])."""
    y = (x.double() @ rot.T).float()  # in 64 bits: values next to a rounding border
    lo, hi = y.amin(-1), y.amax(-1)
    scale, zero = ((hi - lo) / float(2 ** b - 1)).half(), lo.half()
    s = scale.float()[..., None]
    code = torch.where(s == 0, torch.zeros_like(y), torch.round((y - zero.float()[..., None]) / s))
    code = code.clamp(0, 2 ** b - 1).to(torch.uint8)
    per = 8 // b
    shift = torch.arange(per, device=x.device, dtype=torch.uint8) * b
    packed = (code.unflatten(-1, (-1, per)) << shift).sum(-1, dtype=torch.uint8)
    return packed, torch.stack([scale, zero], -1)


def _dequantise(packed, sz, b):
    """The rotated rows that codes stand for, in 32 bits."""
    shift = torch.arange(8 // b, device=packed.device, dtype=torch.uint8) * b
    code = ((packed[..., None] >> shift) & (2 ** b - 1)).flatten(-2).float()
    sz = sz.float()
    return code * sz[..., :1] + sz[..., 1:]


def _views(c, pool):
    """The pool's K codes, K (scale, zero), V codes, V (scale, zero): [pages][n_kv][page][...], in place."""
    off, size = _layout(c)
    pages = pool.numel() // size
    h, ps, d = c["n_kv"], c["page"], c["d"]
    out = []
    for at, b in ((off[0], c["b_k"]), (off[1], 0), (off[2], c["b_v"]), (off[3], 0)):
        row = d * b // 8 if b else 4
        v = pool.as_strided((pages, h, ps, row), (size, ps * row, row, 1), at)
        out.append(v if b else v.view(torch.float16))
    return out


def _gathered(c, pool, table):
    """Rotated K and V rows of every table position, [batch][n_kv][pages * page][d] in 32 bits."""
    kc, ks, vc, vs = (v[table.clamp(min=0).long()].transpose(1, 2).flatten(2, 3) for v in _views(c, pool))
    return _dequantise(kc, ks, c["b_k"]), _dequantise(vc, vs, c["b_v"])


def _plain_rope(c, s):
    ang = s["pos"].double()[:, None] * s["inv_freq"].double()[None, :]
    cos, sin = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    if c["inverse"]:
        sin = -sin
    rot, out = c["rot"], []
    for x in (s["q"], s["k"]):
        y = x.float().clone()
        if c["layout"] == "half":
            a, b = slice(0, rot // 2), slice(rot // 2, rot)
        else:
            a, b = slice(0, rot, 2), slice(1, rot, 2)
        u, v = x[..., a].float(), x[..., b].float()
        y[..., a], y[..., b] = u * cos - v * sin, v * cos + u * sin
        out.append(y.to(x.dtype))
    return out


def _plain_write(c, s):
    seq, i = s["rows"][:, 0], s["rows"][:, 1]
    at = s["lens"].long()[seq] + i
    page, slot = s["table"].long()[seq, at // c["page"]], at % c["page"]
    kc, ks, vc, vs = _views(c, s["pool"])
    kc[page, :, slot], ks[page, :, slot] = _quantise(s["k"][seq, i], s["rot"], c["b_k"])
    vc[page, :, slot], vs[page, :, slot] = _quantise(s["v"][seq, i], s["rot"], c["b_v"])
    return _plain_read(c, s, s["lens"], s["lens_after"], c["n_new"])


def _plain_read(c, s, start, lens, n):
    k, v = _gathered(c, s["pool"], s["table"])
    at = start.long()[:, None] + torch.arange(n, device=k.device)[None, :]
    there = (at < lens[:, None])[:, None, :, None]
    pick = at.clamp(max=k.shape[2] - 1)[:, None, :, None].expand(-1, c["n_kv"], -1, c["d"])
    rot = s["rot"].float()
    return [torch.where(there, (x.gather(2, pick) @ rot).to(o.dtype), o)
            for x, o in ((k, s["k_out"]), (v, s["v_out"]))]


def _plain_attn(c, s):
    batch, n, h, g, d = c["batch"], c["n_new"], c["n_kv"], c["n_q"] // c["n_kv"], c["d"]
    rot = s["rot"].float()
    q = s["q"].float().view(batch, n, h, g, d).permute(0, 2, 1, 3, 4).reshape(batch, h, n * g, d)
    k, v = _gathered(c, s["pool"], s["table"])
    t = torch.arange(k.shape[2], device=q.device)
    cached = (q @ rot.T) @ k.transpose(-1, -2) * s["scale"]
    cached = cached.masked_fill(t[None, None, None, :] >= s["lens"][:, None, None, None], -math.inf)
    sees = ((s["mask"][:, :, None] >> torch.arange(n, device=q.device)) & 1).bool()  # [batch][n][n]
    sees = sees[:, None, :, None, :].expand(-1, -1, -1, g, -1).reshape(batch, 1, n * g, n)
    new_k, new_v = (x.float().transpose(1, 2) for x in (s["k"], s["v"]))
    drafted = (q @ new_k.transpose(-1, -2) * s["scale"]).masked_fill(~sees, -math.inf)
    scores = torch.cat([cached, drafted], -1)
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(scores - top)
    total = p.sum(-1, keepdim=True)
    acc = (p[..., :-n] @ v) @ rot + p[..., -n:] @ new_v
    lse = top + torch.log(total)
    out = acc / total.clamp(min=1e-37)
    out, lse = (x.view(batch, h, n, g, -1).permute(0, 2, 1, 3, 4).reshape(batch, n, h * g, -1) for x in (out, lse))
    if c["prefix"]:
        joint = torch.logaddexp(lse, s["prefix_lse"][..., None])
        out = out * torch.exp(lse - joint) + s["prefix_out"].float() * torch.exp(s["prefix_lse"][..., None] - joint)
        lse = joint
    there = (torch.arange(n, device=q.device)[None, :] < s["counts"][:, None])[..., None, None]
    return [torch.where(there, out.to(s["out"].dtype), s["out"]), torch.where(there[..., 0], lse[..., 0], s["lse"])]


# ---- the state, one pass --------------------------------------------------------------------------

def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    io, d = _IO[c["io"]], c["d"]

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * sigma

    if c["op"] == "rope":
        i = np.arange(c["rot"] // 2, dtype=np.float64)
        freq = torch.from_numpy((500000.0 ** (-2.0 * i / c["rot"])).astype(np.float32)).cuda()
        pos = torch.randint(0, c["far"], (c["tokens"],), generator=gen, device="cuda", dtype=torch.int32)
        q, k = normal(c["tokens"], c["n_q"], d).to(io), normal(c["tokens"], c["n_kv"], d).to(io)
        return dict(case=c, q=q, k=k, pos=pos, inv_freq=freq, q_out=torch.empty_like(q), k_out=torch.empty_like(k))

    batch, ps, h = c["batch"], c["page"], c["n_kv"]
    write = c["op"] == "write"
    lens = [c["start"] + 3 * i for i in range(batch)] if write else _lens(c)
    held = [n + (c["n_new"] if write else 0) for n in lens]
    width = max(1, max(-(-n // ps) for n in held)) + 1
    used = [-(-n // ps) for n in held]
    pages = sum(used) + 3
    ids = rng.permutation(pages)
    table = np.full((batch, width), -1, dtype=np.int32)
    for b, (n, first) in enumerate(zip(used, np.cumsum([0] + used[:-1]))):
        table[b, :n] = ids[first:first + n]
    size = _layout(c)[1]
    s = dict(case=c, table=torch.from_numpy(table).cuda(), lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
             pool=torch.zeros(pages * size, dtype=torch.uint8, device="cuda"), seed=0x5EED0000 + seed % 1000)
    s["rot"] = _rotation(d, s["seed"])
    # key rows with a few channels larger than the rest, as keys have them
    wide = torch.ones(d, device="cuda")
    wide[torch.arange(4, device="cuda") * (d // 4) + d // 8] = 4.0

    def rows(*shape, key):
        x = normal(*shape, d)
        return (x * wide if key else x).to(io)

    if write:
        n = c["n_new"]
        s["k"], s["v"] = rows(batch, n, h, key=True), rows(batch, n, h, key=False)
        s["lens_after"] = s["lens"] + n
        s["rows"] = torch.cartesian_prod(torch.arange(batch), torch.arange(n)).cuda()
        s["k_out"], s["v_out"] = (torch.zeros(batch, h, n, d, dtype=io, device="cuda") for _ in range(2))
    else:
        for views, b, key in ((_views(c, s["pool"])[:2], c["b_k"], True), (_views(c, s["pool"])[2:], c["b_v"], False)):
            for p in range(0, pages, 512):  # a part at a time: the rotation runs in 64 bits
                codes, sz = _quantise(rows(min(512, pages - p), h, ps, key=key), s["rot"], b)
                views[0][p:p + 512], views[1][p:p + 512] = codes, sz
    if c["op"] == "read":
        s["start"] = torch.zeros_like(s["lens"])
        s["k_out"], s["v_out"] = (torch.zeros(batch, h, c["tokens"], d, dtype=io, device="cuda") for _ in range(2))
    if c["op"] == "attn":
        n = c["n_new"]
        s["q"] = normal(batch, n, c["n_q"], d, sigma=1.5).to(io)
        s["k"], s["v"] = rows(batch, n, h, key=True), rows(batch, n, h, key=False)
        s["counts"] = torch.tensor(_counts(c), dtype=torch.int32, device="cuda")
        s["scale"] = 1.0 / math.sqrt(d)
        mask = np.zeros((batch, n), dtype=np.uint64)
        for b in range(batch):
            for i in range(n):
                parent = int(rng.integers(max(0, i - 4), i)) if i else -1
                mask[b, i] = (mask[b, parent] if i else np.uint64(0)) | (np.uint64(1) << np.uint64(i))
        s["mask"] = torch.from_numpy(mask.view(np.int64)).cuda()
        s["out"] = torch.zeros(batch, n, c["n_q"], d, dtype=io, device="cuda")
        s["lse"] = torch.zeros(batch, n, c["n_q"], device="cuda")
        s["prefix_out"] = normal(batch, n, c["n_q"], d, sigma=0.1).to(io) if c["prefix"] else None
        s["prefix_lse"] = normal(batch, n, c["n_q"]) + math.log(c["tokens"] + 1) if c["prefix"] else None
    return s


def _own_pages(s):
    """The handle a user's program keeps: the pages' description."""
    from long_context_st_b200 import api
    if "pages" not in s:
        c = s["case"]
        size = _layout(c)[1]
        s["pages"] = api.make_pages(s["pool"].numel() // size, c["page"], c["n_kv"], c["d"], c["b_k"], c["b_v"],
                                    io_dtype=c["io"], rot_seed=s["seed"])
        if c["op"] == "attn":
            s["ws"] = api.new_tree_workspace(s["pages"], c["batch"], c["n_new"], c["n_q"], s["table"].shape[1])
    return s["pages"]


def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "rope":
            return _plain_rope(c, s)
        if c["op"] == "write":
            return _plain_write(c, s)
        if c["op"] == "read":
            return _plain_read(c, s, s["start"], s["lens"], c["tokens"])
        return _plain_attn(c, s)
    from long_context_st_b200 import api
    if c["op"] == "rope":
        api.rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_out"], s["k_out"], layout=c["layout"],
                 inverse=c["inverse"])
        return [s["q_out"], s["k_out"]]
    pages = _own_pages(s)
    if c["op"] == "write":
        api.pages_append(pages, s["pool"], s["table"], s["lens"], s["k"], s["v"])
        api.pages_read(pages, s["pool"], s["table"], s["lens_after"], s["k_out"], s["v_out"], start=s["lens"])
        return [s["k_out"], s["v_out"]]
    if c["op"] == "read":
        api.pages_read(pages, s["pool"], s["table"], s["lens"], s["k_out"], s["v_out"])
        return [s["k_out"], s["v_out"]]
    api.tree_attn(pages, s["pool"], s["table"], s["lens"], s["q"], s["out"], s["ws"], k=s["k"], v=s["v"],
                  mask=s["mask"], counts=s["counts"], lse=s["lse"], prefix_out=s["prefix_out"],
                  prefix_lse=s["prefix_lse"], attn_scale=s["scale"])
    return [s["out"], s["lse"]]


def work(c):
    e = 4 if c["io"] == "f32" else 2
    d = c["d"]
    if c["op"] == "rope":
        n = c["tokens"] * (c["n_q"] + c["n_kv"])
        return {"bytes": 2 * n * d * e + 4 * c["tokens"], "flops": 3 * n * c["rot"]}
    row = d * (c["b_k"] + c["b_v"]) // 8 + 8
    if c["op"] == "write":
        n = c["batch"] * c["n_new"] * c["n_kv"]
        # rows in, codes out; codes in again, rows out
        return {"bytes": n * (2 * 2 * d * e + 2 * row), "flops": n * 2 * d * (2 * math.log2(d) + 8)}
    if c["op"] == "read":
        n = sum(_lens(c)) * c["n_kv"]
        return {"bytes": n * (row + 2 * d * e), "flops": n * 2 * d * (math.log2(d) + 3)}
    lens, new = _lens(c), _counts(c)
    seen = sum(n * (m + (n + 1) / 4) for m, n in zip(lens, new))  # a drafted token sees part of its tree
    rows = sum(new) * c["n_q"] * (d * e * (3 if c["prefix"] else 2) + (8 if c["prefix"] else 4))
    return {"bytes": sum(lens) * c["n_kv"] * row + rows + sum(new) * (c["n_kv"] * 2 * d * e + 8),
            "flops": 4 * d * c["n_q"] * seen}


# ---- the definition in 64 bits --------------------------------------------------------------------

def _exact_rows(codes, sz, b, signs):
    """Dense rows of packed codes: each code from its bits, the inverse rotation by butterflies."""
    d = codes.shape[-1] * 8 // b
    j = torch.arange(d, device=codes.device)
    x = (codes.long()[..., j * b // 8] >> (j * b % 8)) & (2 ** b - 1)
    x = x.double() * sz.double()[..., 0:1] + sz.double()[..., 1:2]
    return _exact_hadamard(x) * signs


def _exact_hadamard(x):
    d, step = x.shape[-1], 1
    while step < d:
        y = x.unflatten(-1, (d // (2 * step), 2, step))
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).flatten(-3)
        step *= 2
    return x / math.sqrt(d)


def _exact_sequence(c, s, b, n):
    """K and V rows of the first n positions of sequence b, [n_kv][n][d] in 64 bits."""
    (k0, k1, v0, v1), size = _layout(c)
    ps, h, d = c["page"], c["n_kv"], c["d"]
    used = s["table"][b, :-(-n // ps)].long() if n else s["table"][b, :0].long()
    raw = s["pool"].view(-1, size)[used]
    signs = torch.from_numpy(_signs(d, s["seed"])).cuda()
    got = []
    for at, end, bits in ((k0, k1, c["b_k"]), (v0, v1, c["b_v"])):
        codes = raw[:, at:end].reshape(-1, h, ps, d * bits // 8).transpose(0, 1).flatten(1, 2)[:, :n]
        sz = raw[:, end:end + h * ps * 4].contiguous().view(torch.float16).view(-1, h, ps, 2)
        got.append(_exact_rows(codes, sz.transpose(0, 1).flatten(1, 2)[:, :n], bits, signs))
    return got


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        z = torch.polar(torch.ones_like(s["pos"].double())[:, None].expand(-1, c["rot"] // 2).contiguous(),
                        (-1.0 if c["inverse"] else 1.0) * torch.outer(s["pos"].double(), s["inv_freq"].double()))
        out = []
        for x in (s["q"], s["k"]):
            x = x.double()
            head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
            half = c["layout"] == "half"
            pairs = head.unflatten(-1, (2, -1)).transpose(-1, -2) if half else head.unflatten(-1, (-1, 2))
            turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * z[:, None, :])
            turned = turned.transpose(-1, -2).flatten(-2) if half else turned.flatten(-2)
            out.append(torch.cat([turned, rest], -1))
        return out
    if c["op"] == "write":
        out = []
        signs = torch.from_numpy(_signs(c["d"], s["seed"])).cuda()
        for x, b in ((s["k"], c["b_k"]), (s["v"], c["b_v"])):
            y = _exact_hadamard(x.double() * signs)
            low = y.amin(-1, keepdim=True)
            step = ((y.amax(-1, keepdim=True) - low) / (2 ** b - 1)).half().double()  # held in 16 bits
            low = low.half().double()
            code = torch.round((y - low) / step).clamp(0, 2 ** b - 1)
            out.append((_exact_hadamard(code * step + low) * signs).transpose(1, 2))
        return out
    if c["op"] == "read":
        out = [torch.zeros(c["batch"], c["n_kv"], c["tokens"], c["d"], dtype=torch.float64, device="cuda")
               for _ in range(2)]
        for b, n in enumerate(_lens(c)):
            for o, x in zip(out, _exact_sequence(c, s, b, n)):
                o[b, :, :n] = x
        return out
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device="cuda")
    g = c["n_q"] // c["n_kv"]
    for b, (n, m) in enumerate(zip(_lens(c), _counts(c))):
        keys, values = _exact_sequence(c, s, b, n)
        sees = (s["mask"][b, :m, None] >> torch.arange(m, device="cuda")) & 1
        for h in range(c["n_kv"]):
            q = s["q"][b, :m, h * g:(h + 1) * g].double()  # [m][g][d]
            old = torch.einsum("mgd,td->mgt", q, keys[h])
            new = torch.einsum("mgd,td->mgt", q, s["k"][b, :m, h].double())
            new = torch.where(sees[:, None, :] == 1, new, torch.full_like(new, -math.inf))
            a = torch.cat([old, new], -1) * s["scale"]
            v = torch.cat([values[h], s["v"][b, :m, h].double()])
            if c["prefix"]:  # one more key, whose score is the prefix's log-sum-exp
                a = torch.cat([a, s["prefix_lse"][b, :m, h * g:(h + 1) * g, None].double()], -1)
            w = torch.softmax(a, -1)
            o = torch.einsum("mgt,td->mgd", w[..., :len(v)], v)
            if c["prefix"]:
                o = o + w[..., -1:] * s["prefix_out"][b, :m, h * g:(h + 1) * g].double()
            out[b, :m, h * g:(h + 1) * g] = o
            lse[b, :m, h * g:(h + 1) * g] = torch.logsumexp(a, -1)
    return [out, lse]
