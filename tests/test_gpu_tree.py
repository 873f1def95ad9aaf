"""GPU parity of the speculative-decoding operators against the fp64 oracle: attention of
drafted trees, verification, compaction, page copies, and a serving loop of them together.

Attention tolerances: the weights P are rounded to bf16 (half a step, 2^-8 relative) and the
output once more, so
    |out - ref| <= 2^-8 * (mass + |ref|) + 2 * ds * mass,   mass = sum_j w_j |ckv_j|
with ds the error of a score: 576 fp32 products summed in an order of the tensor cores'
choosing, 576 * 2^-24 * sum |q k| * scale, under 3e-4 for inputs of deviation 0.5 (sum |q k|
is about 576 * 0.16 = 92); lse is off by ds plus its own fp32 rounding (|lse| < 16: 1e-6).
Everything else is whole numbers or moved bytes, and exact.
"""

import numpy as np
import pytest
import torch

import paged_head_latent_mla_b200 as M
from oracle import mla_oracle as O
from oracle import spec_oracle as S
from test_tree_host import flat, random_tree
from workloads import make_custom

pytestmark = pytest.mark.gpu

DS = 3e-4
TIMEOUT_NS = 500_000_000
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_head_latent_mla_b200 import _build

    _build.build()
    return M.load_library()


def tables(d):
    return d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len


def tree_plan(d, parents, rope=64, **kw):
    return M.mla_plan_tree(*tables(d), np.asarray(parents, dtype=np.int32), num_heads=d.num_heads,
                           page_size=d.page_size, num_pages=d.num_pages, sm_scale=d.sm_scale, rope_dim=rope,
                           wait_timeout_ns=TIMEOUT_NS, **kw)


def check_attention(out, lse, ref):
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    ref_o, ref_l, mass = ref
    tol = 2.0 ** -8 * (mass + np.abs(ref_o)) + 2 * DS * mass
    bad = ~(np.abs(out - ref_o) <= tol)
    assert not bad.any(), f"{np.argwhere(bad)[:5].tolist()} of {bad.sum()}, {np.nanmax(np.abs(out - ref_o)):.3e}"
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_l))
    fin = np.isfinite(ref_l)
    assert np.abs(lse[fin] - ref_l[fin]).max(initial=0) <= DS + 1e-6


def run_tree(d, parents, rope=64, append=False, seed=0, **kw):
    """Run one tree step on inputs of d; returns (out, lse, cache, oracle's result)."""
    plan = tree_plan(d, parents, rope, **kw)
    cache = d.cache[:, :, : 512 + rope].contiguous()
    q_pe = d.q_pe if rope else None
    kv_new = None
    dev_cache = cache.to(DEV)
    if append:
        g = torch.Generator().manual_seed(seed)
        kv_new = (torch.randn((d.total_tokens, 512 + rope), generator=g) * 0.5).to(torch.bfloat16)
        cache = torch.from_numpy(O.append_latent(cache, kv_new, *tables(d), d.page_size)).to(torch.bfloat16)
    out, lse = M.mla_run(plan, d.q_nope.to(DEV), q_pe.to(DEV) if rope else None, dev_cache, return_lse=True,
                         kv_new=kv_new.to(DEV) if append else None)
    assert M.mla_plan_check(plan) == M.MLA_OK
    if append:
        assert torch.equal(dev_cache.cpu(), cache)
    ref = S.tree_attention(d.q_nope, q_pe, cache, *tables(d), parents, d.page_size, d.sm_scale)
    plan.destroy()
    return out, lse, dev_cache, ref


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("H,P,rope,split,append", [
    (16, 16, 64, 0, True), (32, 32, 64, -1, False), (64, 64, 0, 64, True), (128, 128, 64, 0, False),
    (128, 16, 0, -1, True), (16, 128, 64, 128, False),
])
def test_tree_attention_matches_oracle(H, P, rope, split, append):
    rng = np.random.default_rng(H + P + rope)
    q = [1, 7, 0, 17, 65, 130, 3]
    ctx = [0, 63, 40, 128, 1, 700, 2049]
    trees = [random_tree(rng, n, roots=1 + b % 3) for b, n in enumerate(q)]
    trees[3] = list(range(-1, 16))  # a chain beside trees
    d = make_custom(q, [a + b for a, b in zip(q, ctx)], H, P, seed=11, extra_pool_pages=3)
    out, lse, _, ref = run_tree(d, flat(trees), rope, append, seed=12, split_keys=split)
    check_attention(out, lse, ref)


@pytest.mark.parametrize("n,ctx", [(1, 0), (2, 0), (64, 0), (65, 64), (257, 31), (1024, 0), (1024, 65)])
def test_tree_sizes(n, ctx):
    rng = np.random.default_rng(n)
    d = make_custom([n], [n + ctx], 16, 64, seed=n)
    out, lse, _, ref = run_tree(d, random_tree(rng, n))
    check_attention(out, lse, ref)


def test_many_roots_and_a_star():
    n = 40
    d = make_custom([n, n], [n + 100, n + 5], 64, 32, seed=5)
    out, lse, _, ref = run_tree(d, [-1] * n + [-1] + [0] * (n - 1))
    check_attention(out, lse, ref)


@pytest.mark.parametrize("H", [16, 128])
def test_chain_is_bitwise_the_causal_step(H):
    """(where keys are not split: a tree plan's partial results are fp32)"""
    q, k = [4, 1, 17, 2], [500, 33, 1100, 2]
    d = make_custom(q, k, H, 64, seed=8)
    causal = M.mla_plan(*tables(d), num_heads=H, page_size=64, num_pages=d.num_pages, sm_scale=d.sm_scale,
                        wait_timeout_ns=TIMEOUT_NS, split_keys=-1)
    chain = tree_plan(d, flat([range(-1, n - 1) for n in q]), split_keys=-1)
    args = (d.q_nope.to(DEV), d.q_pe.to(DEV), d.cache.to(DEV))
    a = M.mla_run(causal, *args, return_lse=True)
    b = M.mla_run(chain, *args, return_lse=True)
    assert M.mla_plan_check(causal) == M.MLA_OK and M.mla_plan_check(chain) == M.MLA_OK
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("H", [16, 64, 128])
@pytest.mark.parametrize("where", ["ckv", "kpe", "one"])
def test_masked_rows_may_hold_anything(H, bad, where):
    """Nodes whose latent rows are not finite reach only the nodes that see them; the rest
    is bitwise what it is with finite rows there."""
    n = [30, 9]
    trees = [[-1, 0, 0, 1, 1, 2, 2] + [(i - 1) // 2 for i in range(7, 30)], list(range(-1, 8))]
    d = make_custom(n, [30 + 50, 9 + 64], H, 16, seed=21)
    par = flat(trees)
    odd = {0: [5, 13, 29], 1: [6]}
    clean = d.cache.clone()
    hurt = d.cache.clone()
    sees = []
    for b, nodes in odd.items():
        for i in range(n[b]):
            if set(S.path_of(trees[b], i)) & set(nodes):
                sees.append(int(d.qo_indptr[b]) + i)
        for a in nodes:
            page, slot = O.key_location(d.kv_indptr, d.kv_indices, 16, b, int(d.kv_lens[b]) - n[b] + a)
            part = {"ckv": slice(0, 512), "kpe": slice(512, 576), "one": slice(300, 301)}[where]
            hurt[page, slot, part] = bad
    plan = tree_plan(d, par)
    args = (d.q_nope.to(DEV), d.q_pe.to(DEV))
    a, la = M.mla_run(plan, *args, clean.to(DEV), return_lse=True)
    b, lb = M.mla_run(plan, *args, hurt.to(DEV), return_lse=True)
    assert M.mla_plan_check(plan) == M.MLA_OK
    free = [t for t in range(sum(n)) if t not in sees]
    assert len(free) > 10
    assert torch.equal(a[free], b[free]) and torch.equal(la[free], lb[free])
    if np.isnan(bad):
        assert torch.isnan(lb[sees]).all()


def test_masked_rows_may_hold_anything_with_split_keys():
    """The same where every key tile is an item of its own and the partial results merge."""
    n, ctx = 90, 130
    tree = [-1] + [(i - 1) // 2 for i in range(1, n)]
    d = make_custom([n], [n + ctx], 32, 16, seed=22)
    odd = [7, 40, 88]
    sees = [i for i in range(n) if set(S.path_of(tree, i)) & set(odd)]
    free = [i for i in range(n) if i not in sees]
    hurt = d.cache.clone()
    for a in odd:
        page, slot = O.key_location(d.kv_indptr, d.kv_indices, 16, 0, ctx + a)
        hurt[page, slot] = float("nan")
    plan = tree_plan(d, tree, split_keys=64)
    assert M.mla_plan_get_info(plan)["num_merge"] > 0
    args = (d.q_nope.to(DEV), d.q_pe.to(DEV))
    a, la = M.mla_run(plan, *args, d.cache.to(DEV), return_lse=True)
    b, lb = M.mla_run(plan, *args, hurt.to(DEV), return_lse=True)
    assert M.mla_plan_check(plan) == M.MLA_OK
    assert torch.equal(a[free], b[free]) and torch.equal(la[free], lb[free])
    assert torch.isnan(lb[sees]).all() and torch.isnan(b[sees]).all()


def test_cascade_of_trees_matches_oracle():
    rng = np.random.default_rng(31)
    q = [4, 4, 4, 4, 3, 4]
    trees = [random_tree(rng, n) for n in q]
    d = make_custom(q, [300, 260, 500, 262, 400, 300], 16, 64, seed=31, shared_group=6, shared_pages=4)
    plan = tree_plan(d, flat(trees), cascade=True, host_only=True)
    assert M.mla_plan_get_info(plan)["num_cascade"] > 0
    out, lse, _, ref = run_tree(d, flat(trees), cascade=True)
    check_attention(out, lse, ref)


@pytest.mark.parametrize("first", [0, 2])
def test_tree_graph_replays_updated_steps(first):
    """Captured on one step, replayed on others: more and fewer rows, nodes and keys (the
    step captured second has idle lane quarters only)."""
    rng = np.random.default_rng(41)
    TM, H, P = 40, 32, 32
    specs = [([5, 9, 1], [60, 300, 1]), ([40], [1500]), ([0, 3], [20, 3]), ([8] * 5, [100, 8, 200, 3000, 64])]
    specs = specs[first:] + specs[:first]
    steps = [make_custom(q, k, H, P, seed=43 + i, pool_pages=200) for i, (q, k) in enumerate(specs)]
    trees = [flat([random_tree(rng, n) for n in q]) for q, _ in specs]
    plan = tree_plan(steps[0], trees[0], graph_max_batch=6, graph_max_tokens=TM, graph_max_page_ids=200)
    cache = torch.empty((200, P, 576), dtype=torch.bfloat16, device=DEV)
    qn = torch.zeros((TM, H, 512), dtype=torch.bfloat16, device=DEV)
    qp = torch.zeros((TM, H, 64), dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(qn)
    lse = torch.empty((TM, H), device=DEV)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        cache.copy_(steps[0].cache)
        M.mla_run(plan, qn, qp, cache, out=out, lse=lse)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        M.mla_run(plan, qn, qp, cache, out=out, lse=lse)
    for d, par in list(zip(steps, trees)) + [(steps[0], trees[0])]:
        T = d.total_tokens
        with torch.cuda.stream(s):
            M.mla_plan_tree_update(plan, *tables(d), np.asarray(par, dtype=np.int32), stream=s.cuda_stream)
            cache.copy_(d.cache)
            qn[:T].copy_(d.q_nope)
            qp[:T].copy_(d.q_pe)
            out.fill_(7.0)
            g.replay()
        torch.cuda.synchronize()
        assert M.mla_plan_check(plan) == M.MLA_OK
        check_attention(out[:T], lse[:T],
                        S.tree_attention(d.q_nope, d.q_pe, d.cache, *tables(d), par, P, d.sm_scale))
        assert (out[T:] == 7.0).all()  # rows behind the step's last are left as they were
    del g
    plan.destroy()


@pytest.mark.parametrize("n", [2, 30])
def test_a_wait_that_runs_out_is_reported(n):
    """The first key load is never issued (a planning flag): the waits on it run out, the
    plan reports it, and another plan runs afterwards."""
    d = make_custom([n, n], [n + 300, n + 40], 32, 64, seed=6)
    tree = [-1] + [(i - 1) // 2 for i in range(1, n)]
    args = (d.q_nope.to(DEV), d.q_pe.to(DEV), d.cache.to(DEV))
    plan = M.mla_plan_tree(*tables(d), np.asarray(tree * 2, dtype=np.int32), num_heads=32, page_size=64,
                           num_pages=d.num_pages, sm_scale=d.sm_scale, wait_timeout_ns=100_000_000,
                           debug_flags=M.MLA_DEBUG_DROP_FIRST_KV_LOAD)
    M.mla_run(plan, *args)
    assert M.mla_plan_check(plan) == M.MLA_ERR_DEVICE_TIMEOUT
    plan.destroy()
    out, lse, _, ref = run_tree(d, tree * 2)
    check_attention(out, lse, ref)


# ------------------------------------------------------------------ verification
def verify_plan(q, trees, pool=None, **kw):
    d = make_custom(q, [max(1, n) for n in q], 16, 16, seed=3, tables_only=True, pool_pages=pool)
    return tree_plan(d, flat(trees), **kw), d


def peaked(rng, T, V, dtype):
    z = torch.from_numpy(rng.standard_normal((T, V)) * 3).float()
    p = torch.softmax(z, 1)
    r = torch.softmax(z + torch.from_numpy(rng.standard_normal((T, V)) * 0.7).float(), 1)
    return p.to(dtype), r.to(dtype)


def drafted(rng, d, trees, weights):
    """Tokens drawn from each parent's row of weights."""
    qo = d.qo_indptr.tolist()
    tok = np.zeros(qo[-1], dtype=np.int32)
    for b, tree in enumerate(trees):
        for i, p in enumerate(tree):
            if p >= 0:
                w = weights[qo[b] + p].double().numpy()
                tok[qo[b] + i] = rng.choice(len(w), p=w / w.sum())
    return tok


def check_verify(plan, d, trees, tok, p, r, u, un, rows=None, **kw):
    dev = lambda x: None if x is None else torch.as_tensor(x).to(DEV)  # noqa: E731
    got = M.mla_verify_tree(plan, dev(tok), kw.pop("p_dev", dev(p)), dev(u), dev(un),
                            draft_probs=kw.pop("r_dev", dev(r)), **kw)
    want = S.verify_tree(d.qo_indptr, flat(trees), tok, p.double().numpy(), u, un,
                         None if r is None else r.double().numpy())
    for name, a, b in zip(("accept_index", "num_accepted", "next_token"), got, want):
        a = a.cpu().numpy()
        assert np.array_equal(a, b), (name, np.nonzero(a != b)[0][:5], a[a != b][:5], b[a != b][:5])
    return want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 33, 1000, 8192, 50001])
def test_verify_matches_oracle(dtype, draft, V):
    rng = np.random.default_rng(V + 2 * draft)
    q = [1, 5, 0, 16, 9, 2, 33]
    trees = [random_tree(rng, n, roots=1) for n in q]
    plan, d = verify_plan(q, trees)
    T = d.total_tokens
    p, r = peaked(rng, T, V, dtype)
    tok = drafted(rng, d, trees, r)
    u = rng.random(T, dtype=np.float32)
    un = rng.random(len(q), dtype=np.float32)
    check_verify(plan, d, trees, tok, p, r if draft else None, u, un)


@pytest.mark.parametrize("batch", [1, 40, 80, 160, 400])
def test_verify_batches(batch):
    """Every cluster size (8, 4, 2 and 1 blocks to a row)."""
    rng = np.random.default_rng(batch)
    q = [int(rng.integers(0, 9)) for _ in range(batch - 1)] + [9]
    trees = [random_tree(rng, n, roots=1) for n in q]
    plan, d = verify_plan(q, trees)
    T = d.total_tokens
    p, r = peaked(rng, T, 3001, torch.float32)
    want = check_verify(plan, d, trees, drafted(rng, d, trees, r), p, r, rng.random(T, dtype=np.float32),
                        rng.random(batch, dtype=np.float32))
    if batch > 1:
        assert (want[1] > 1).any() and (want[2][want[1] > 0] >= 0).all()


def test_verify_a_large_vocabulary():
    rng = np.random.default_rng(14)
    q = [9] * 40
    trees = [[-1, 0, 0, 0, 1, 1, 4, 4, 4] for _ in q]
    plan, d = verify_plan(q, trees)
    p, r = peaked(rng, 360, 131071, torch.float32)
    want = check_verify(plan, d, trees, drafted(rng, d, trees, r), p, r, rng.random(360, dtype=np.float32),
                        rng.random(40, dtype=np.float32))
    assert (want[1] > 2).any()


def test_verify_on_two_streams_at_once():
    """Two calls on one plan, each with its own outputs, running side by side."""
    rng = np.random.default_rng(15)
    q = [9] * 30
    trees = [random_tree(rng, 9, roots=1) for _ in q]
    plan, d = verify_plan(q, trees)
    p, r = peaked(rng, 270, 20000, torch.float32)
    tok = drafted(rng, d, trees, r)
    dev = [x.to(DEV) for x in (p, r, torch.from_numpy(tok))]
    u = [rng.random(270, dtype=np.float32) for _ in range(2)]
    un = [rng.random(30, dtype=np.float32) for _ in range(2)]
    ud = [(torch.from_numpy(a).to(DEV), torch.from_numpy(b).to(DEV)) for a, b in zip(u, un)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(M.mla_verify_tree(plan, dev[2], dev[0], *ud[i], draft_probs=dev[1]))
    torch.cuda.synchronize()
    for i in range(2):
        want = S.verify_tree(d.qo_indptr, flat(trees), tok, p.double().numpy(), u[i], un[i], r.double().numpy())
        for g in got[i]:
            for a, b in zip(g, want):
                assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shift_p,shift_r,pitch_p,pitch_r", [(0, 0, 1003, 1003), (1, 1, 1024, 1024), (1, 0, 1024, 1024),
                                                             (0, 0, 1001, 1005), (3, 3, 1007, 1015)])
def test_verify_strides_and_offsets(dtype, shift_p, shift_r, pitch_p, pitch_r):
    rng = np.random.default_rng(9)
    V, q = 1000, [9, 4, 12]
    trees = [random_tree(rng, n, roots=1) for n in q]
    plan, d = verify_plan(q, trees)
    T = d.total_tokens
    p, r = peaked(rng, T, V, dtype)

    def at(x, shift, pitch):
        flat_ = torch.full((T * pitch + shift,), float("nan"), dtype=dtype, device=DEV)
        v = flat_[shift:].view(T, pitch)[:, :V]
        v.copy_(x)
        return v

    for draft in (True, False):
        check_verify(plan, d, trees, drafted(rng, d, trees, r), p, r if draft else None,
                     rng.random(T, dtype=np.float32), rng.random(len(q), dtype=np.float32),
                     p_dev=at(p, shift_p, pitch_p), r_dev=at(r, shift_r, pitch_r) if draft else None)


@pytest.mark.parametrize("draft", [True, False])
def test_verify_borders_are_exact(draft):
    """Weights and random numbers that are sums of powers of two: every sum is exact in any
    order, and the borders are hit exactly."""
    rng = np.random.default_rng(2)
    q = [4] * 200
    trees = [[-1, 0, 0, 0] if b % 2 else [-1, 0, 1, 0] for b in range(200)]
    plan, d = verify_plan(q, trees)
    T, V = d.total_tokens, 16
    p = torch.from_numpy(rng.integers(0, 4, (T, V)) / 16.0).float()
    r = torch.from_numpy(rng.integers(0, 3, (T, V)) / 16.0).float()
    tok = rng.integers(0, V, T).astype(np.int32)
    u = (rng.integers(0, 4, T) / 4).astype(np.float32)
    un = (rng.integers(0, 8, 200) / 8).astype(np.float32)
    check_verify(plan, d, trees, tok, p, r if draft else None, u, un)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** -133, 2.0 ** -120, 2.0, 2.0 ** 100, 2.0 ** 125])
def test_verify_weights_of_any_size(dtype, draft, scale):
    """Weights need not sum to 1: small whole numbers times a power of two, down to the
    types' subnormals (bf16's smallest is 2^-133) and up to near their largest."""
    rng = np.random.default_rng(3)
    q = [5] * 60
    trees = [random_tree(rng, 5, roots=1) for _ in q]
    plan, d = verify_plan(q, trees)
    T, V = d.total_tokens, 37
    p = (torch.from_numpy(rng.integers(0, 4, (T, V))).double() * scale).to(dtype)
    r = (torch.from_numpy(rng.integers(0, 4, (T, V))).double() * scale).to(dtype)
    assert torch.equal(p.double() / scale, (p.double() / scale).round()) and p.any()
    tok = rng.integers(0, V, T).astype(np.int32)
    check_verify(plan, d, trees, tok, p, r if draft else None, rng.random(T, dtype=np.float32),
                 rng.random(60, dtype=np.float32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_odd_weights(dtype, draft):
    """Zero rows, infinities, NaN and negative weights, given tokens, tokens out of range,
    the same token drafted twice."""
    rng = np.random.default_rng(4)
    q = [8] * 24
    trees = [random_tree(rng, 8, roots=1) for _ in q]
    plan, d = verify_plan(q, trees)
    T, V = d.total_tokens, 77
    p, r = peaked(rng, T, V, dtype)
    for x in (p, r):
        x[::5, :40] = 0
        x[::7, 3] = float("nan")
        x[::9, 5] = float("inf")
        x[::4, 11] = -0.25
        x[1::13] = 0
    p[2::11] = float("nan")
    tok = rng.integers(-1, V + 2, T).astype(np.int32)
    tok[::6] = 20
    tok[1::6] = 20
    tok[5] = 2 ** 31 - 1
    tok[6] = -(2 ** 31)
    check_verify(plan, d, trees, tok, p, r if draft else None, rng.random(T, dtype=np.float32),
                 rng.random(len(q), dtype=np.float32))


@pytest.mark.parametrize("shape", ["star", "chain"])
def test_verify_a_thousand_nodes(shape):
    rng = np.random.default_rng(6)
    n, V = 1024, 2000
    trees = [[-1] + [0] * (n - 1) if shape == "star" else list(range(-1, n - 1))]
    plan, d = verify_plan([n], trees)
    p, r = peaked(rng, n, V, torch.float32)
    if shape == "chain":
        r = p.clone()  # always accepted
    else:
        u1 = None
    tok = drafted(rng, d, trees, r)
    u = rng.random(n, dtype=np.float32) * (0.999 if shape == "chain" else 1)
    if shape == "star":  # point masses that the target hardly holds: hundreds of rejections
        p[0, : V // 2] *= 1e-6
        tok = rng.integers(0, V // 2, n).astype(np.int32)
        u = np.maximum(u, np.float32(0.1))
    want = check_verify(plan, d, trees, tok, p, r if shape == "chain" else None, u, rng.random(1, dtype=np.float32))
    assert want[1][0] == (n if shape == "chain" else 1)


def test_verify_long_chain_is_refused_and_left_alone_in_a_graph():
    plan, d = verify_plan([1025], [list(range(-1, 1024))])
    z = torch.zeros((1025, 8), device=DEV)
    i = torch.zeros(1025, dtype=torch.int32, device=DEV)
    f = torch.zeros(1025, device=DEV)
    with pytest.raises(M.MlaError) as e:
        M.mla_verify_tree(plan, i, z, f, f[:1])
    assert e.value.status == M.MLA_ERR_UNSUPPORTED
    # captured on a short step, replayed on the long one
    plan, d = verify_plan([2], [[-1, 0]], pool=100, graph_max_batch=2, graph_max_tokens=1025, graph_max_page_ids=100)
    acc = torch.full((1025,), 9, dtype=torch.int32, device=DEV)
    cnt, nxt = torch.full((2,), 9, dtype=torch.int32, device=DEV), torch.full((2,), 9, dtype=torch.int32, device=DEV)
    args = (plan, i, z, f, torch.zeros(2, device=DEV))
    kw = dict(accept_index=acc, num_accepted=cnt, next_token=nxt)
    M.mla_verify_tree(*args, **kw)
    torch.cuda.synchronize()
    assert acc[:2].tolist() == [0, -1] and acc[2:].eq(9).all() and cnt.tolist() == [1, 9] and nxt.tolist() == [-1, 9]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.mla_verify_tree(*args, **kw)
    long = make_custom([1025], [1025], 16, 16, seed=3, tables_only=True, pool_pages=100)
    M.mla_plan_tree_update(plan, *tables(long), np.arange(-1, 1024, dtype=np.int32))
    g.replay()
    torch.cuda.synchronize()
    assert acc.eq(-1).all() and cnt.tolist() == [0, 9] and nxt.tolist() == [-1, 9]
    del g


def test_verified_tokens_follow_the_target():
    """The first token that a step yields (an accepted child's, else the next token) is
    distributed as the target's row, whatever the drafts: each frequency within five
    standard deviations of its probability."""
    rng = np.random.default_rng(77)
    B, V = 20000, 6
    p = np.array([0.4, 0.05, 0.25, 0.1, 0.2, 0.0])
    r = np.array([0.1, 0.3, 0.1, 0.2, 0.2, 0.1])
    trees = [[-1, 0, 0, 0]] * B
    plan, d = verify_plan([4] * B, trees)
    P = torch.tensor(p, dtype=torch.float32, device=DEV).expand(4 * B, V).contiguous()
    R = torch.tensor(r, dtype=torch.float32, device=DEV).expand(4 * B, V).contiguous()
    u = torch.from_numpy(rng.random(4 * B, dtype=np.float32)).to(DEV)
    un = torch.from_numpy(rng.random(B, dtype=np.float32)).to(DEV)
    for draft in (True, False):
        tok = rng.choice(V, size=(B, 4), p=r).astype(np.int32)
        if not draft:  # point masses: any choice of tokens
            tok[:] = [0, 1, 2, 2]
        t = torch.from_numpy(tok.reshape(-1)).to(DEV)
        acc, cnt, nxt = (x.cpu().numpy() for x in M.mla_verify_tree(plan, t, P, u, un,
                                                                    draft_probs=R if draft else None))
        first = np.where(cnt > 1, tok[np.arange(B), np.maximum(acc.reshape(B, 4)[:, 1], 0)], nxt)
        freq = np.bincount(first, minlength=V) / B
        assert (np.abs(freq - p) <= 5 * np.sqrt(p * (1 - p) / B) + 1e-12).all(), (draft, freq)


def test_verify_refusals():
    plan, d = verify_plan([3], [[-1, 0, 1]])
    p = torch.zeros((3, 8), device=DEV)
    i, f, one = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(3, device=DEV), torch.zeros(1, device=DEV)
    M.mla_verify_tree(plan, i, p, f, one)
    for bad in [dict(target_probs=p.half()), dict(target_probs=p[:2]), dict(target_probs=p.t()),
                dict(target_probs=p[:, ::2]), dict(draft_tokens=i.long()), dict(uniform=f[:2]),
                dict(uniform_next=f), dict(draft_probs=p.bfloat16()), dict(draft_probs=p[:, :7]),
                dict(next_token=i), dict(target_probs=p[:1].expand(3, 8))]:
        kw = dict(draft_tokens=i, target_probs=p, uniform=f, uniform_next=one)
        kw.update(bad)
        with pytest.raises(ValueError):
            M.mla_verify_tree(plan, **kw)
    a = p.data_ptr()
    call = M.load_library().mla_verify_tree
    h = plan.handle
    for args in [(h, a, None, 8, None, 0, 8, 0, a, a, a, a, a, None), (h, a, a, 7, None, 0, 8, 0, a, a, a, a, a, None),
                 (h, a, a, 8, a, 7, 8, 0, a, a, a, a, a, None), (h, a, a, 8, None, 0, 0, 0, a, a, a, a, a, None),
                 (h, a, a, 8, None, 0, 8, 2, a, a, a, a, a, None), (h, a, a + 2, 8, None, 0, 8, 0, a, a, a, a, a, None),
                 (h, a + 1, a, 8, None, 0, 8, 0, a, a, a, a, a, None), (h, a, a, 8, None, 0, 8, 0, a, a, a, None, a, None),
                 (h, a, a, 1 << 29, None, 0, 1 << 29, 0, a, a, a, a, a, None)]:
        assert call(*args) == M.MLA_ERR_INVALID_ARGUMENT
    causal = M.mla_plan(*tables(d), num_heads=16, page_size=16, num_pages=d.num_pages, sm_scale=1.0)
    with pytest.raises(M.MlaError):
        M.mla_verify_tree(causal, i, p, f, one)


# ------------------------------------------------------------------ compaction
def accepted(rng, d, trees):
    """A random path of every row's tree, as mla_verify_tree writes it."""
    qo = d.qo_indptr.tolist()
    acc = np.full(qo[-1], -1, dtype=np.int32)
    cnt = np.zeros(len(trees), dtype=np.int32)
    for b, t in enumerate(trees):
        if t:
            path = S.path_of(t, int(rng.integers(0, len(t))))
            acc[qo[b]: qo[b] + len(path)] = path
            cnt[b] = len(path)
    return acc, cnt


@pytest.mark.parametrize("P,rope,layers", [(16, 64, 1), (32, 0, 3), (64, 64, 5), (128, 64, 130)])
def test_compact_is_bit_exact(P, rope, layers):
    rng = np.random.default_rng(P)
    q = [1, 8, 0, 33, 100, 2]
    trees = [random_tree(rng, n, roots=1) for n in q]
    trees[4] = [i - 1 if i < 1 else (i - 2 if i > 1 else 0) for i in range(100)]  # every other node: a long move
    d = make_custom(q, [n + c for n, c in zip(q, [0, 13, 7, 60, 15, 200])], 16, P, seed=7)
    plan = tree_plan(d, flat(trees), rope)
    acc, cnt = accepted(rng, d, trees)
    g = torch.Generator().manual_seed(5)
    cache = torch.randint(-2 ** 15, 2 ** 15, (layers, d.num_pages, P, 512 + rope), dtype=torch.int16, generator=g)
    dev = cache.to(DEV).view(torch.bfloat16)
    M.mla_compact_kv(plan, torch.from_numpy(acc).to(DEV), torch.from_numpy(cnt).to(DEV), dev)
    got = dev.view(torch.int16).cpu().numpy()
    for i in range(layers):
        want = S.compact_kv(cache[i].numpy(), *tables(d), P, acc, cnt)
        assert np.array_equal(got[i], want)


def test_compact_ignores_entries_out_of_range():
    d = make_custom([4, 4], [20, 30], 16, 16, seed=7)
    plan = tree_plan(d, [-1, 0, 0, 1] * 2)
    acc = np.array([0, -1, 1, 9, 3, 2 ** 31 - 1, -(2 ** 31), 3], dtype=np.int32)
    cnt = np.array([100, 4], dtype=np.int32)
    dev = d.cache.to(DEV)
    M.mla_compact_kv(plan, torch.from_numpy(acc).to(DEV), torch.from_numpy(cnt).to(DEV), [dev])
    want = S.compact_kv(d.cache.view(torch.int16).numpy(), *tables(d), 16, acc, cnt)
    assert np.array_equal(dev.cpu().view(torch.int16).numpy(), want)


def test_compact_refusals():
    d = make_custom([4], [20], 16, 16, seed=7)
    plan = tree_plan(d, [-1, 0, 0, 1])
    cache = d.cache.to(DEV)
    i, n = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    M.mla_compact_kv(plan, i, n, cache)
    with pytest.raises(M.MlaError):
        M.mla_compact_kv(plan, i, n, [cache, cache])
    for bad in [(i[:3], n, cache), (i, i, cache), (i, n, cache.float()), (i, n, cache[:, :, :512]),
                (i, n, cache[:1]), (i.float(), n, cache)]:
        with pytest.raises(ValueError):
            M.mla_compact_kv(plan, *bad)
    # two tokens on one slot: the row's page list repeats a page
    kvi = torch.tensor([1, 1], dtype=torch.int32)
    plan = M.mla_plan_tree([0, 17], [0, 2], kvi, [16], [-1] + [0] * 16, num_heads=16, page_size=16, num_pages=2,
                           sm_scale=1.0)
    with pytest.raises(M.MlaError):
        M.mla_compact_kv(plan, torch.zeros(17, dtype=torch.int32, device=DEV), n, cache)


# ------------------------------------------------------------------ page copies
@pytest.mark.parametrize("P,rope,layers,pairs,part", [(16, 64, 1, 1, False), (32, 0, 3, 40, True),
                                                      (64, 64, 131, 3, False), (128, 64, 2, 9, True),
                                                      (16, 0, 2, 1500, True)])
def test_copy_pages_is_bit_exact(P, rope, layers, pairs, part):
    rng = np.random.default_rng(pairs)
    pool = 2 * pairs + 3
    ids = rng.permutation(pool).astype(np.int32)
    dst = ids[:pairs]
    src = rng.choice(ids[pairs:], pairs).astype(np.int32)  # sources repeat
    n = rng.integers(0, P + 1, pairs).astype(np.int32) if part else None
    g = torch.Generator().manual_seed(5)
    cache = torch.randint(-2 ** 15, 2 ** 15, (layers, pool, P, 512 + rope), dtype=torch.int16, generator=g)
    dev = cache.to(DEV).view(torch.bfloat16)
    M.mla_copy_pages(torch.from_numpy(src), dst.tolist(), list(dev.unbind(0)) if layers == 2 else dev, num_tokens=n)
    M.mla_copy_pages(src, dst, [], num_tokens=n)
    got = dev.view(torch.int16).cpu().numpy()
    for i in range(layers):
        assert np.array_equal(got[i], S.copy_pages(cache[i].numpy(), src, dst, n))


def test_copy_pages_refuses_bad_tables():
    cache = torch.zeros((4, 16, 576), dtype=torch.bfloat16, device=DEV)
    for src, dst, n in [([0], [4], None), ([0, 1], [1, 2], None), ([0, 1], [2, 2], None), ([0], [1], [17]),
                        ([0], [0], None), ([0], [1, 2], None)]:
        with pytest.raises(M.MlaError):
            M.mla_copy_pages(src, dst, cache, num_tokens=n)
    with pytest.raises(ValueError):
        M.mla_copy_pages([0], [1], [cache, cache[:3].contiguous()])
    with pytest.raises(M.MlaError):
        M.mla_copy_pages([0], [1], [cache, cache])
    assert not cache.any()


# ------------------------------------------------------------------ far offsets
def test_offsets_beyond_32_bits():
    """A pool of 4.8 GB: the step's pages lie at its end."""
    P, pages = 128, 33000  # 4.9e9 bytes, 2.4e9 elements
    cache = torch.zeros((pages, P, 576), dtype=torch.bfloat16, device=DEV)
    assert cache.numel() > 2 ** 31
    small = make_custom([6], [6 + 130], 16, P, seed=9)
    far = torch.tensor([pages - 1, pages - 3], dtype=torch.int32)
    for i, pg in enumerate(far.tolist()):
        cache[pg] = small.cache[int(small.kv_indices[i])].to(DEV)
    parents = [-1, 0, 0, 1, 1, 2]
    plan = M.mla_plan_tree(small.qo_indptr, small.kv_indptr, far, small.last_page_len, parents, num_heads=16,
                           page_size=P, num_pages=pages, sm_scale=small.sm_scale, wait_timeout_ns=TIMEOUT_NS)
    out, lse = M.mla_run(plan, small.q_nope.to(DEV), small.q_pe.to(DEV), cache, return_lse=True)
    assert M.mla_plan_check(plan) == M.MLA_OK
    check_attention(out, lse, S.tree_attention(small.q_nope, small.q_pe, small.cache, *tables(small), parents, P,
                                               small.sm_scale))
    acc = torch.tensor([0, 2, 5, -1, -1, -1], dtype=torch.int32, device=DEV)
    M.mla_compact_kv(plan, acc, torch.tensor([3], dtype=torch.int32, device=DEV), cache)
    want = S.compact_kv(small.cache.view(torch.int16).numpy(), *tables(small), P, acc.cpu().numpy(), [3])
    for i, pg in enumerate(far.tolist()):
        assert np.array_equal(cache[pg].cpu().view(torch.int16).numpy(), want[int(small.kv_indices[i])])
    M.mla_copy_pages([pages - 3, pages - 1], [pages - 2, 0], cache, num_tokens=[128, 100])
    assert torch.equal(cache[pages - 2], cache[pages - 3])
    assert torch.equal(cache[0, :100], cache[pages - 1, :100]) and not cache[0, 100:].any()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("graph", [False, True])
def test_serving_loop_of_trees(graph):
    """Steps of draft tree, append and attention per layer, verification, compaction, and a
    fork with a page copy, on a side stream; eagerly and from one captured graph.  After
    every step the outputs match the oracle, and the cache holds the kept tokens' rows in
    order, as if they had been decoded one by one."""
    H, P, V, L, pages = 16, 16, 500, 2, 64
    TM, BM = 24, 3
    rng = np.random.default_rng(123)
    s = torch.cuda.Stream()
    caches = [torch.zeros((pages, P, 576), dtype=torch.bfloat16, device=DEV) for _ in range(L)]
    buf = dict(qn=torch.zeros((TM, H, 512), dtype=torch.bfloat16, device=DEV),
               qp=torch.zeros((TM, H, 64), dtype=torch.bfloat16, device=DEV),
               kv=torch.zeros((L, TM, 576), dtype=torch.bfloat16, device=DEV),
               out=torch.zeros((L, TM, H, 512), dtype=torch.bfloat16, device=DEV), lse=torch.zeros((L, TM, H), device=DEV),
               tok=torch.zeros(TM, dtype=torch.int32, device=DEV), p=torch.zeros((TM, V), device=DEV),
               r=torch.zeros((TM, V), device=DEV), u=torch.zeros(TM, device=DEV), un=torch.zeros(BM, device=DEV),
               acc=torch.zeros(TM, dtype=torch.int32, device=DEV), cnt=torch.zeros(BM, dtype=torch.int32, device=DEV),
               nxt=torch.zeros(BM, dtype=torch.int32, device=DEV))

    def step(plan):
        for i in range(L):
            M.mla_run(plan, buf["qn"], buf["qp"], caches[i], out=buf["out"][i], lse=buf["lse"][i], kv_new=buf["kv"][i])
        M.mla_verify_tree(plan, buf["tok"], buf["p"], buf["u"], buf["un"], draft_probs=buf["r"],
                          accept_index=buf["acc"], num_accepted=buf["cnt"], next_token=buf["nxt"])
        M.mla_compact_kv(plan, buf["acc"], buf["cnt"], caches)

    rows = [dict(pages=[], history=[np.zeros((0, 576)) for _ in range(L)]) for _ in range(2)]
    free = list(rng.permutation(pages))
    plan = g = None
    torch.cuda.synchronize()
    for it in range(5):
        if it == 3:  # fork row 0: full pages are shared, the partly filled one is copied
            a = rows[0]
            n = len(a["history"][0])
            full = n // P
            b = dict(pages=a["pages"][:full], history=[h.copy() for h in a["history"]])
            if n % P:
                b["pages"] = b["pages"] + [free.pop()]
                with torch.cuda.stream(s):
                    M.mla_copy_pages([a["pages"][full]], [b["pages"][full]], caches, num_tokens=[n % P])
            a["pages"] = a["pages"][: -(-n // P)]
            rows.append(b)
        trees = [random_tree(rng, int(rng.integers(1, 9)), roots=1) for _ in rows]
        qo, kvp, kvi, last = [0], [0], [], []
        for row, tree in zip(rows, trees):
            k = len(row["history"][0]) + len(tree)
            while len(row["pages"]) * P < k:
                row["pages"].append(free.pop())
            n_pages = -(-k // P)
            qo.append(qo[-1] + len(tree))
            kvp.append(kvp[-1] + n_pages)
            kvi += row["pages"][:n_pages]
            last.append(k - (n_pages - 1) * P)
        t = [np.asarray(x, dtype=np.int32) for x in (qo, kvp, kvi, last, flat(trees))]
        T = qo[-1]
        new = {k: (rng.standard_normal(tuple(v.shape)) * 0.5) for k, v in buf.items() if k in ("qn", "qp", "kv")}
        p, r = peaked(rng, TM, V, torch.float32)
        d = type("D", (), dict(qo_indptr=torch.from_numpy(t[0])))
        tok = np.zeros(TM, dtype=np.int32)
        tok[:T] = drafted(rng, d, trees, r)
        u, un = rng.random(TM, dtype=np.float32) * 0.5, rng.random(BM, dtype=np.float32)
        with torch.cuda.stream(s):
            for k, v in new.items():
                buf[k].copy_(torch.from_numpy(v))
            for k, v in (("p", p), ("r", r), ("tok", tok), ("u", u), ("un", un)):
                buf[k].copy_(torch.as_tensor(v))
            if plan is None:
                plan = M.mla_plan_tree(*t, num_heads=H, page_size=P, num_pages=pages, sm_scale=192 ** -0.5,
                                       wait_timeout_ns=TIMEOUT_NS, graph_max_batch=BM, graph_max_tokens=TM,
                                       graph_max_page_ids=pages)
            else:
                M.mla_plan_tree_update(plan, *t)
            if graph and g is None:
                s.synchronize()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s):
                    step(plan)
            if graph:
                g.replay()
            else:
                step(plan)
        s.synchronize()
        assert M.mla_plan_check(plan) == M.MLA_OK
        want = S.verify_tree(t[0], t[4], tok, p.double().numpy(), u, un, r.double().numpy())
        got = [buf[k].cpu().numpy() for k in ("acc", "cnt", "nxt")]
        B = len(rows)
        assert np.array_equal(got[0][:T], want[0]) and np.array_equal(got[1][:B], want[1])
        assert np.array_equal(got[2][:B], want[2])
        kv = buf["kv"].double().cpu().numpy()
        for i in range(L):
            # the oracle's cache of this step: each row's history, then its nodes
            o_kvp = np.concatenate([[0], np.cumsum([-(-(len(row["history"][i]) + len(tr)) // P)
                                                    for row, tr in zip(rows, trees)])])
            o_cache = np.zeros((int(o_kvp[-1]), P, 576))
            for b, (row, tr) in enumerate(zip(rows, trees)):
                seq = np.concatenate([row["history"][i], kv[i, qo[b]: qo[b + 1]]])
                o_cache[o_kvp[b]: o_kvp[b + 1]].reshape(-1, 576)[: len(seq)] = seq
                keep = want[0][qo[b]: qo[b] + want[1][b]]
                row["history"][i] = np.concatenate([row["history"][i], kv[i, qo[b]: qo[b + 1]][keep]])
            ref = S.tree_attention(buf["qn"][:T].cpu(), buf["qp"][:T].cpu(), o_cache, t[0], o_kvp,
                                   np.arange(int(o_kvp[-1])), t[3], t[4], P, 192 ** -0.5)
            check_attention(buf["out"][i, :T], buf["lse"][i, :T], ref)
            host = caches[i].double().cpu().numpy()
            for row in rows:
                n = len(row["history"][i])
                stored = host[np.asarray(row["pages"], dtype=np.int64)].reshape(-1, 576)[:n]
                assert np.array_equal(stored, row["history"][i])
    assert max(len(r["history"][0]) for r in rows) > P
    del g
    plan.destroy()
