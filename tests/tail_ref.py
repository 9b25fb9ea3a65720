"""Plain 64-bit forms of the tail cache's operators for the tests, and builders of their inputs."""
import math

import numpy as np
import torch

import oracle
from long_context_st_b200 import api

NP = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}  # a rounding to the type, relative


def rows(rng, shape, io, outliers=False):
    x = rng.standard_normal(shape)
    if outliers:
        x[..., shape[-1] // 8] *= 6.0
    return torch.from_numpy(x.astype(np.float32)).to(NP[io]).cuda()


def f64(t):
    return t.detach().cpu().double().numpy()


def make_table(rng, lens, page_size, extra_width=1, spare=2):
    """A table of shuffled page ids wide enough for lens; unused entries are -1. Returns
    (table int32 cuda, n_pages)."""
    used = [-(-n // page_size) for n in lens]
    width = max(used + [0]) + extra_width
    n_pages = sum(used) + spare
    ids = rng.permutation(n_pages)
    t = np.full((len(lens), max(width, 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(used):
        t[b, :n] = ids[at:at + n]
        at += n
    return torch.from_numpy(t).cuda(), max(n_pages, 1)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def fill_random(rng, p, pool):
    """Random codes and plausible (scale, zero) in every row of the pool."""
    off, size = api.pages_layout(p)
    raw = rng.integers(0, 256, (p.n_pages, size), dtype=np.uint8)
    for at, b in ((off[1], p.b_k), (off[3], p.b_v)):
        n = p.n_kv * p.page_size
        sz = np.empty((p.n_pages, n, 2), dtype=np.float16)
        span = rng.uniform(1.0, 5.0, (p.n_pages, n))
        sz[..., 0] = span / (2 ** b - 1)
        sz[..., 1] = -span * rng.uniform(0.4, 0.6, (p.n_pages, n))
        raw[:, at:at + n * 4] = sz.view(np.uint8).reshape(p.n_pages, n * 4)
    pool.copy_(torch.from_numpy(raw.reshape(-1)).cuda()[:pool.numel()])


def stored_rows(p, pool, table, lens):
    """Per sequence (K, V) [n_kv][len][d_h]: what the pages hold, rotated rows in 64 bits."""
    off, size = api.pages_layout(p)
    raw = pool.cpu().numpy()[:p.n_pages * size].reshape(p.n_pages, size)
    tab = table.cpu().numpy()
    out = []
    for b, n in enumerate(lens):
        seq = []
        for x, bits in ((0, p.b_k), (2, p.b_v)):
            rb = p.d_h * bits // 8
            ids = tab[b, :-(-n // p.page_size)] if n else np.zeros(0, dtype=int)
            codes = raw[ids, off[x]:off[x] + p.n_kv * p.page_size * rb].reshape(-1, p.n_kv, p.page_size, rb)
            sz = raw[ids, off[x + 1]:off[x + 1] + p.n_kv * p.page_size * 4].copy().view(np.float16)
            sz = sz.reshape(-1, p.n_kv, p.page_size, 2).astype(np.float64)
            c = oracle.unpack_codes(codes, bits, p.d_h).astype(np.float64)
            y = c * sz[..., :1] + sz[..., 1:]
            seq.append(y.transpose(1, 0, 2, 3).reshape(p.n_kv, -1, p.d_h)[:, :n])
        out.append(tuple(seq))
    return out


def attention(p, pool, table, lens, q, k=None, v=None, mask=None, counts=None, scale=None, prefix=None):
    """out, lse in 64 bits, and a bound on the 2-norm of each out row's error and on each lse's, from
    the kernel's roundings (see tree_attn's comments): R q to 22 bits, fp32 sums, p * scale to 11
    bits (bf16) or 22 (fp32)."""
    B, N, nq, d = q.shape
    g = nq // p.n_kv
    R = oracle.rotation_matrix(d, p.rot_seed)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, lse = np.zeros((B, N, nq, d)), np.full((B, N, nq), -np.inf)
    eo, el = np.zeros((B, N, nq)), np.zeros((B, N, nq))
    io = "f32" if p.io_dtype == 0 else "bf16"
    q, k, v = f64(q), (f64(k) if k is not None else None), (f64(v) if v is not None else None)
    m = mask.cpu().numpy().view(np.uint64) if mask is not None else None
    cnt = counts.cpu().numpy() if counts is not None else [N] * B
    held = stored_rows(p, pool, table, lens)
    for b in range(B):
        ky, vy = held[b]
        for i in range(min(int(cnt[b]), N)):
            if m is not None:
                sees = [j for j in range(min(int(cnt[b]), N)) if (int(m[b, i]) >> j) & 1]
            else:
                sees = list(range(i + 1))
            if k is None:
                sees = []
            for hq in range(nq):
                h = hq // g
                qr = R @ q[b, i, hq]
                keys = np.concatenate([ky[h] @ R, k[b, sees, h]] if sees else [ky[h] @ R])
                vals = np.concatenate([vy[h] @ R, v[b, sees, h]] if sees else [vy[h] @ R])
                s = (keys @ q[b, i, hq]) * scale
                # |score error|: 2 terms of R q, products summed in fp32 (d terms and the centring)
                span = np.abs(ky[h]).max(initial=0.0) + np.abs(keys).max(initial=0.0)
                es = (2.0 ** -21 + (d + 8) * 2.0 ** -24) * scale * 2.0 * span * np.abs(qr).sum()
                if prefix is not None:
                    s = np.append(s, float(prefix[1][b, i, hq]))
                    vals = np.concatenate([vals, f64(prefix[0])[b, i, hq][None]])
                if not len(s) or np.max(s) == -np.inf:
                    continue
                top = np.max(s)
                w = np.exp(s - top)
                lse[b, i, hq] = top + np.log(w.sum())
                out[b, i, hq] = (w / w.sum()) @ np.where(w[:, None] > 0, vals, 0.0)
                es += np.abs(top) * 2.0 ** -22 + len(s) * 2.0 ** -24 + 2.0 ** -21
                el[b, i, hq] = es + np.abs(lse[b, i, hq]) * 2.0 ** -22
                big = np.linalg.norm(vals, axis=-1).max() + np.linalg.norm(vy[h], axis=-1).max(initial=0.0) * 2
                ep = (2.0 ** -12 if io == "bf16" else 2.0 ** -21) + (len(s) + d) * 2.0 ** -24
                eo[b, i, hq] = (2.0 * es + ep) * big + HALF_STEP[io] * np.linalg.norm(out[b, i, hq]) + 1e-30
    return out, lse, eo, el


def check_attention(p, got, got_lse, ref, cnt):
    out, lse, eo, el = ref
    o, l = f64(got), f64(got_lse)
    for b in range(o.shape[0]):
        n = min(int(cnt[b]), o.shape[1])
        off = np.linalg.norm(o[b, :n] - out[b, :n], axis=-1)
        assert np.all(off <= eo[b, :n]), (b, float((off / np.maximum(eo[b, :n], 1e-30)).max()))
        fin = np.isfinite(lse[b, :n])
        assert np.array_equal(fin, np.isfinite(l[b, :n])) and np.all(l[b, :n][~fin] == -np.inf)
        d = np.abs(l[b, :n][fin] - lse[b, :n][fin])
        assert np.all(d <= el[b, :n][fin]), (b, float((d / el[b, :n][fin]).max()))
