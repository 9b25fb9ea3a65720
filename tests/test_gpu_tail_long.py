"""GPU: the tail cache's loops in their steady state (many tiles a block, rows a warp, rounds of barriers), against
64-bit forms with bounds of the errors' own size."""
import math

import numpy as np
import pytest
import torch

import oracle
from long_context_st_b200 import api
from tail_ref import NP, rows, f64, make_table, i32, fill_random
from tail_bounds import HALF, attention64, check64, ratios
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
