"""Attention of drafted trees where latent rows hold infinities or NaN: every element of the
output and of lse is what the formula gives, finite or not.

The fp64 oracle follows the formula through them (exp(-inf - lse) * inf is a NaN).  Finite
elements have the tolerances of the tree tests: P and the output are rounded to bf16 (half a
step, 2^-8 relative, each), scores are off by DS at most.
"""

import numpy as np
import pytest
import torch

import paged_head_latent_mla_b200 as M
from oracle import mla_oracle as O
from oracle import spec_oracle as S
from test_tree_host import flat
from workloads import make_custom

pytestmark = pytest.mark.gpu

DS = 3e-4
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_head_latent_mla_b200 import _build

    _build.build()
    return M.load_library()


def tables(d):
    return d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len


def run(d, parents, cache, rope=64, **kw):
    plan = M.mla_plan_tree(*tables(d), np.asarray(parents, dtype=np.int32), num_heads=d.num_heads,
                           page_size=d.page_size, num_pages=d.num_pages, sm_scale=d.sm_scale, rope_dim=rope,
                           wait_timeout_ns=500_000_000, **kw)
    out, lse = M.mla_run(plan, d.q_nope.to(DEV), d.q_pe.to(DEV) if rope else None, cache.to(DEV), return_lse=True)
    assert M.mla_plan_check(plan) == M.MLA_OK
    plan.destroy()
    return out, lse


def check(out, lse, ref):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref_o, ref_l, mass = ref
    assert np.array_equal(np.isnan(out), np.isnan(ref_o)), np.argwhere(np.isnan(out) != np.isnan(ref_o))[:5].tolist()
    assert np.array_equal(np.isnan(lse), np.isnan(ref_l)) and np.array_equal(np.isneginf(lse), np.isneginf(ref_l))
    ok = np.isfinite(ref_o)
    assert (np.abs(out - ref_o)[ok] <= (2.0 ** -8 * (mass + np.abs(ref_o)) + 2 * DS * mass)[ok]).all()
    fin = np.isfinite(ref_l)
    assert np.abs(lse[fin] - ref_l[fin]).max(initial=0) <= DS + 1e-6


def slot(d, b, node):
    n = int(d.qo_indptr[b + 1] - d.qo_indptr[b])
    return O.key_location(d.kv_indptr, d.kv_indices, d.page_size, b, int(d.kv_lens[b]) - n + node)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("column", [3, 300, 500, 520])
@pytest.mark.parametrize("H,split,rope", [(16, 0, 64), (32, 64, 64), (64, -1, 64), (128, 64, 0), (128, 0, 64)])
def test_nodes_that_see_a_row_that_is_not_finite(H, split, rope, column, bad):
    """One element of some nodes' rows.  The tree has every kind of score there (+inf and -inf
    by the sign of the query's element); the chain has query tiles whose rows of one warp see
    a whole key tile, and those of another do not."""
    if column >= 512 + rope:
        pytest.skip("no such column")
    trees = [[-1, 0, 0, 1, 1, 2, 2] + [(i - 1) // 2 for i in range(7, 30)], list(range(-1, 29)), [-1, 0, 0]]
    d = make_custom([30, 30, 3], [30 + 50, 30 + 50, 3 + 64], H, 16, seed=61)
    cache = d.cache[:, :, : 512 + rope].contiguous()
    for b, nodes in ((0, (5, 13, 29)), (1, (10, 20)), (2, (2,))):
        for a in nodes:
            page, at = slot(d, b, a)
            cache[page, at, column] = bad
    out, lse = run(d, flat(trees), cache, rope, split_keys=split)
    with np.errstate(invalid="ignore"):
        ref = S.tree_attention(d.q_nope, d.q_pe if rope else None, cache, *tables(d), flat(trees), 16, d.sm_scale)
    assert np.isnan(ref[0]).any() and not np.isnan(ref[0]).all()
    check(out, lse, ref)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_context_rows_that_are_not_finite(bad):
    """In key tiles that every node sees whole, and in the one that the first node shares."""
    tree = [-1, 0, 0, 1, 2, 2]
    d = make_custom([6, 6], [6 + 130, 6 + 140], 16, 16, seed=62)
    cache = d.cache.clone()
    for b, key in ((0, 20), (0, 129), (1, 139)):
        page, at = O.key_location(d.kv_indptr, d.kv_indices, 16, b, key)
        cache[page, at, 40 + key] = bad
    out, lse = run(d, tree * 2, cache)
    with np.errstate(invalid="ignore"):
        ref = S.tree_attention(d.q_nope, d.q_pe, cache, *tables(d), tree * 2, 16, d.sm_scale)
    check(out, lse, ref)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("H", [16, 128])
def test_slots_behind_a_row_may_hold_anything(H, rope):
    trees = [[-1, 0, 0, 1, 2], [-1], [-1, 0, 1]]
    d = make_custom([5, 1, 3], [5 + 40, 70, 3 + 126], H, 64, seed=63)
    cache = d.cache[:, :, : 512 + rope].contiguous()
    want = run(d, flat(trees), cache, rope)
    used = torch.zeros(cache.shape[:2], dtype=torch.bool)
    for b in range(3):
        for key in range(int(d.kv_lens[b])):
            used[O.key_location(d.kv_indptr, d.kv_indices, 64, b, key)] = True
    assert not used.all()
    cache[~used] = float("nan")
    got = run(d, flat(trees), cache, rope)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_appended_rows_that_are_not_finite():
    """The step's own rows, written by the same enqueue."""
    tree = [-1, 0, 0, 1, 1, 2, 2]
    d = make_custom([7, 7], [7 + 60, 7 + 1], 16, 16, seed=64)
    kv = (torch.randn((14, 576), generator=torch.Generator().manual_seed(65)) * 0.5).to(torch.bfloat16)
    kv[3, 77] = float("-inf")
    kv[11, 400] = float("inf")
    appended = torch.from_numpy(O.append_latent(d.cache, kv, *tables(d), 16)).to(torch.bfloat16)
    plan = M.mla_plan_tree(*tables(d), np.asarray(tree * 2, dtype=np.int32), num_heads=16, page_size=16,
                           num_pages=d.num_pages, sm_scale=d.sm_scale, wait_timeout_ns=500_000_000)
    out, lse = M.mla_run(plan, d.q_nope.to(DEV), d.q_pe.to(DEV), d.cache.to(DEV), return_lse=True, kv_new=kv.to(DEV))
    assert M.mla_plan_check(plan) == M.MLA_OK
    with np.errstate(invalid="ignore"):
        ref = S.tree_attention(d.q_nope, d.q_pe, appended, *tables(d), tree * 2, 16, d.sm_scale)
    assert np.isnan(ref[0]).any()
    check(out, lse, ref)
