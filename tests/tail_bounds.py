"""Attention over the tail cache in 64 bits, with the size that the kernels' roundings should have: for cases
whose outputs are means of many values, where a worst-case bound would pass anything.

Roundings, each half a step of its type, relative to what is rounded:
  R q is carried in 22 bits and its products with the codes are summed in fp32. An MMA step adds 16 products and
  the sum so far, and drops from each what lies below 24 bits of the largest term: over 8 steps (d = 128) of two
  terms each, 17 addends a step, errors uniform and independent, sqrt(16 * 17 / 3) 2^-24 = 2^-20.7 of the
  largest term, at most |R q| times a code row's largest element. bf16 tensors feed codes of 4 and 8 bits as
  subnormals, which costs those sums 6 and 2 more bits. Transforms and the score in fp32: 2^-20 of the score's
  size for the former, |s| 2^-22 for the latter.
  p * scale (or p) is one f16 term for bf16, 2^-11; the tcgen05 form rounds values to f16 too, another 2^-11, and
  2^-(15 + b) of the row's largest element. fp32 has two terms, 2^-21. A bf16 sum over subnormal value codes is
  off by 2^-24 + (10 - b) of its size a step.
Such errors of different tokens are independent, so a sum over tokens is off by the root of the squares; three
times that is the bound. The output's own rounding is counted in full.
"""
import math

import numpy as np
import torch

import oracle
from long_context_st_b200 import api

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def coded_rows(p, pool, table, b, n):
    """((codes, scale, zero) of K, the same of V) of sequence b's first n tokens: [n_kv][n][..] in 64 bits. A
    token without a page has NaN as its scale."""
    off, size = api.pages_layout(p)
    ids = table[b, :-(-n // p.page_size)].long()
    there = (ids >= 0) & (ids < p.n_pages)
    raw = pool[:p.n_pages * size].view(p.n_pages, size)[ids.clamp(0, p.n_pages - 1)]
    out = []
    for x, bits in ((0, p.b_k), (2, p.b_v)):
        rb = p.d_h * bits // 8
        c = raw[:, off[x]:off[x] + p.n_kv * p.page_size * rb].reshape(-1, p.n_kv, p.page_size, rb)
        j = torch.arange(p.d_h, device=c.device) * bits
        c = (c[..., j // 8].long() >> (j % 8)) & (2 ** bits - 1)
        sz = raw[:, off[x + 1]:off[x + 1] + p.n_kv * p.page_size * 4].contiguous().view(torch.float16)
        sz = sz.view(-1, p.n_kv, p.page_size, 2).double()
        sz = torch.where(there[:, None, None, None], sz, math.nan)
        c, sz = (t.transpose(0, 1).flatten(1, 2)[:, :n] for t in (c.double(), sz))
        out.append((c, sz[..., 0], sz[..., 1]))
    return out


def attention64(p, pool, table, lens, q, k=None, v=None, mask=None, counts=None, scale=None, prefix=None, drop=()):
    """(out, lse, bound of an out row's error in the 2-norm, bound of an lse's error); rows behind counts are 0.
    drop: (sequence, token) pairs that are left out, to see that a check would notice."""
    B, N, nq, d = q.shape
    g, dev, io = nq // p.n_kv, q.device, q.dtype
    R = torch.from_numpy(oracle.rotation_matrix(d, p.rot_seed)).to(dev)
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out = torch.zeros(B, N, nq, d, dtype=torch.float64, device=dev)
    lse = torch.full((B, N, nq), -math.inf, dtype=torch.float64, device=dev)
    eo, el = torch.zeros_like(lse), torch.zeros_like(lse)
    bf16 = io == torch.bfloat16
    tc = bf16 and N * g > 16
    lost_k = 10 - p.b_k if bf16 and p.b_k > 2 else 0
    for b in range(B):
        n, m = lens[b], N if counts is None else min(max(int(counts[b]), 0), N)
        if m == 0:
            continue
        (kc, ks, kz), (vc, vs, vz) = coded_rows(p, pool, table, b, n)
        seen = torch.isfinite(ks[0]) if n else torch.zeros(0, dtype=torch.bool, device=dev)
        for s_, t_ in drop:
            if s_ == b:
                seen[t_] = False
        kc, ks, kz, vc, vs, vz = (t[:, seen] for t in (kc, ks, kz, vc, vs, vz))
        for h in range(p.n_kv):
            qr = (q[b, :m, h * g:(h + 1) * g].double() @ R.T).reshape(m * g, d)
            y, x = kc[h] * ks[h, :, None] + kz[h, :, None], vc[h] * vs[h, :, None] + vz[h, :, None]
            s = scale * qr @ y.T
            size = scale * (qr.norm(dim=-1) + qr.sum(-1).abs())[:, None] * (ks[h].abs() * 2 ** p.b_k + kz[h].abs())[None, :]
            ds = (3 * 2.0 ** (lost_k - 20.7) + 2.0 ** -20) * size + 2.0 ** -22 * s.abs()
            vals, rv = x @ R, torch.full_like(x[:, 0], 2.0 ** -11 if bf16 else 2.0 ** -21)
            if tc:
                rv = rv + 2.0 ** -11 + 2.0 ** -(15 + p.b_v) * math.sqrt(d) * x.abs().amax(-1) / x.norm(dim=-1).clamp(min=1e-30)
            if bf16 and not tc:  # products of p * scale with uncentred codes, a step's drop
                rv = rv + 2.0 ** (-24 + 10 - p.b_v) * math.sqrt(d) * vs[h].abs() * 2 ** p.b_v / x.norm(dim=-1).clamp(min=1e-30)
            if k is not None:
                dk, dv = k[b, :m, h].double(), v[b, :m, h].double()
                bits = mask[b, :m] if mask is not None else torch.tensor(
                    [(1 << (i + 1)) - 1 if i < 63 else -1 for i in range(m)], device=dev)
                sees = ((bits[:, None] >> torch.arange(m, device=dev)) & 1).bool().repeat_interleave(g, 0)
                sd = scale * q[b, :m, h * g:(h + 1) * g].double().reshape(m * g, d) @ dk.T
                s = torch.cat([s, sd.masked_fill(~sees, -math.inf)], -1)
                ds = torch.cat([ds, 2.0 ** -20 * scale * q[b, :m, h * g:(h + 1) * g].double().reshape(m * g, d).norm(dim=-1)[:, None]
                                * dk.norm(dim=-1)[None, :]], -1)
                vals, rv = torch.cat([vals, dv]), torch.cat([rv, torch.full_like(dv[:, 0], 2.0 ** -15)])
            pl = None
            if prefix is not None:
                pl = prefix[1][b, :m, h * g:(h + 1) * g].double().reshape(m * g, 1)
                s, ds = torch.cat([s, pl], -1), torch.cat([ds, pl.abs() * 2.0 ** -22], -1)
            l = torch.logsumexp(s, -1) if s.shape[1] else torch.full((m * g,), -math.inf, dtype=torch.float64, device=dev)
            w = torch.nan_to_num(torch.exp(s - l[:, None]), nan=0.0)
            nv = len(vals)
            o = w[:, :nv] @ vals
            norm2 = vals.square().sum(-1)
            if pl is not None:
                po = prefix[0][b, :m, h * g:(h + 1) * g].double().reshape(m * g, d)
                o = o + w[:, -1:] * po
            off2 = (norm2[None, :] - 2 * o @ vals.T + o.square().sum(-1, keepdim=True)).clamp(min=0)  # |v - out|^2
            e_v = (w[:, :nv].square() @ (rv.square() * norm2)).sqrt()
            e_s = (w[:, :nv].square() * ds[:, :nv].square() * off2).sum(-1).sqrt()
            if pl is not None:
                e_s = e_s + w[:, -1] * ds[:, -1] * (po - o).norm(dim=-1)
            e_sum = 2.0 ** -21 * (w[:, :nv] @ norm2.sqrt())
            e_o = HALF[io] * o.norm(dim=-1) + 3 * (e_v + e_s) + e_sum + 1e-30
            e_l = 3 * (w.square() * ds.square()).sum(-1).sqrt() + 2.0 ** -20 + torch.nan_to_num(l.abs(), posinf=0.0) * 2.0 ** -22
            e_l = e_l + (w * ds).sum(-1) / 3  # a drop towards zero is the same for all tokens
            sl = slice(h * g, (h + 1) * g)
            out[b, :m, sl], lse[b, :m, sl] = o.view(m, g, d), l.view(m, g)
            eo[b, :m, sl], el[b, :m, sl] = e_o.view(m, g), e_l.view(m, g)
    return out, lse, eo, el


def ratios(got, got_lse, ref, counts=None):
    """The largest error of an out row and of an lse, in units of their bounds."""
    out, lse, eo, el = ref
    worst = [0.0, 0.0]
    for b in range(out.shape[0]):
        m = out.shape[1] if counts is None else min(max(int(counts[b]), 0), out.shape[1])
        if m == 0:
            continue
        seen = torch.isfinite(lse[b, :m])
        assert torch.equal(seen, torch.isfinite(got_lse[b, :m])) and bool((got_lse[b, :m][~seen] == -math.inf).all())
        assert bool((got[b, :m][~seen] == 0).all()) and bool(torch.isfinite(got[b, :m]).all())
        if bool(seen.any()):
            off = (got[b, :m].double() - out[b, :m]).norm(dim=-1)[seen] / eo[b, :m][seen]
            dl = (got_lse[b, :m].double() - lse[b, :m]).abs()[seen] / el[b, :m][seen]
            worst = [max(worst[0], float(off.max())), max(worst[1], float(dl.max()))]
    return worst


def check64(got, got_lse, ref, counts=None, tight=True):
    """Holds a call to its bounds. tight: the bounds themselves are below a twentieth of the outputs."""
    if tight:
        seen = torch.isfinite(ref[1])
        assert bool((ref[2][seen] <= 0.05 * ref[0].norm(dim=-1)[seen] + 1e-30).all())
    worst = ratios(got, got_lse, ref, counts)
    assert worst[0] <= 1 and worst[1] <= 1, worst
