"""Speculative-tree plans on the host (no GPU): mask words and nodes against the ancestor
relation, the work lists, re-planning, and the refusals of the tree, verification,
compaction and page-copy entry points."""

import ctypes

import numpy as np
import pytest

import paged_head_latent_mla_b200 as M
from oracle import spec_oracle as S
from workloads import make_custom

SCALE = 192 ** -0.5


@pytest.fixture(scope="module", autouse=True)
def built_library():
    from paged_head_latent_mla_b200 import _build

    _build.build()
    return M.load_library()


def random_tree(rng, n, roots=1):
    """Parents of n nodes with up to ``roots`` roots, drawn at random."""
    return [-1 if i < roots and (i == 0 or rng.random() < 0.5) else int(rng.integers(0, i)) for i in range(n)]


def plan_tree(q, k, parents, H=16, P=16, **kw):
    d = make_custom(q, k, H, P, seed=1, tables_only=True)
    kw.setdefault("host_only", True)
    return M.mla_plan_tree(d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len,
                           np.asarray(parents, dtype=np.int32), num_heads=H, page_size=P,
                           num_pages=max(1, d.num_pages), sm_scale=SCALE, **kw), d


def flat(trees):
    return [p for t in trees for p in t]


def visible(desc, tree, H, t):
    """Keys that token t sees, by the plan's records, as {key: times} over all work items."""
    seen = {}
    for w, ti in zip(desc["work"], tree["items"]):
        q_row0, n_rows, _, kv_len, k0, k1, diag, _ = (int(x) for x in w)
        if not q_row0 <= t * H < q_row0 + n_rows:
            continue
        i = (t * H - q_row0) // H
        lim = min(max(0, min(diag + i + 1, kv_len)), k1)
        base, words, first, _ = (int(x) for x in ti)
        for j in range(k0, lim):
            if words and j // 64 >= first:
                if not (int(tree["words"][base + i * words + j // 64 - first]) >> (j % 64)) & 1:
                    continue
            seen[j] = seen.get(j, 0) + 1
    return seen


@pytest.mark.parametrize("split", [0, -1, 64])
@pytest.mark.parametrize("H", [16, 128])
def test_words_are_the_ancestors(H, split):
    rng = np.random.default_rng(3)
    q = [1, 7, 0, 64, 65, 130, 9]
    ctx = [0, 100, 5, 63, 0, 64, 127]
    trees = [random_tree(rng, n, roots=1 + b % 3) for b, n in enumerate(q)]
    trees[6] = list(range(-1, 8))  # a chain among trees
    plan, d = plan_tree(q, [a + b for a, b in zip(q, ctx)], flat(trees), H=H, split_keys=split)
    desc, tree = M.mla_plan_describe(plan), M.mla_plan_describe_tree(plan)
    qo = d.qo_indptr.tolist()
    for b, parents in enumerate(trees):
        for i in range(q[b]):
            want = set(range(ctx[b])) | {ctx[b] + a for a in S.path_of(parents, i)}
            got = visible(desc, tree, H, qo[b] + i)
            assert set(got) == want and all(n == 1 for n in got.values()), (b, i)
    # nodes: parents, children in increasing order, rows
    for b, parents in enumerate(trees):
        nodes = tree["nodes"][qo[b]: qo[b + 1]]
        for i in range(q[b]):
            kids = [c for c in range(q[b]) if parents[c] == i]
            assert nodes[i][0] == parents[i] and nodes[i][3] == b
            assert nodes[i][1] == (kids[0] if kids else -1)
            for a, nxt in zip(kids, kids[1:] + [-1]):
                assert nodes[a][2] == nxt


def test_a_chain_plans_the_causal_step():
    q, k = [4, 1, 9], [300, 77, 1000]
    plan, d = plan_tree(q, k, flat([range(-1, n - 1) for n in q]), H=32, P=32)
    causal = M.mla_plan(d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len, num_heads=32, page_size=32,
                        num_pages=d.num_pages, sm_scale=SCALE, host_only=True)
    a, b = M.mla_plan_describe(plan), M.mla_plan_describe(causal)
    for f in ("kv_len", "work", "merge", "refs"):
        assert np.array_equal(a[f], b[f])
    assert len(M.mla_plan_describe_tree(plan)["words"]) == 0


def test_cascade_prefix_ends_with_the_context():
    """A shared prefix that would reach into the rows' nodes stops before them."""
    P, q = 64, [2, 2, 2]
    # two shared pages = 128 keys; row 1's nodes begin at key 127
    d = make_custom(q, [300, 129, 200], 16, P, seed=2, shared_group=3, shared_pages=2, tables_only=True)
    trees = [[-1, -1]] * 3
    plan = M.mla_plan_tree(d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len, flat(trees), num_heads=16,
                           page_size=P, num_pages=d.num_pages, sm_scale=SCALE, host_only=True, cascade=True)
    desc = M.mla_plan_describe(plan)
    assert desc["info"]["num_cascade"] > 0
    tree = M.mla_plan_describe_tree(plan)
    qo = d.qo_indptr.tolist()
    for w in desc["work"]:
        if w[1] > 2 * 16:  # a tile over several rows
            assert w[5] <= 64
    for b, k in enumerate([300, 129, 200]):
        for i in range(2):
            got = visible(desc, tree, 16, qo[b] + i)
            assert set(got) == set(range(k - 2)) | {k - 2 + i}


def test_update_sees_parents_and_tables():
    plan, d = plan_tree([4], [50], [-1, 0, 0, 1])
    t = (d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len)
    assert M.mla_plan_tree_update(plan, *t, [-1, 0, 0, 1], stream=0)
    assert not M.mla_plan_tree_update(plan, *t, [-1, 0, 1, 1], stream=0)
    assert M.mla_plan_describe_tree(plan)["nodes"][:, 0].tolist() == [-1, 0, 1, 1]
    with pytest.raises(M.MlaError):
        M.mla_plan_tree_update(plan, *t, [-1, 0, 1, 3], stream=0)  # a node cannot continue itself
    assert M.mla_plan_tree_update(plan, *t, [-1, 0, 1, 1], stream=0)  # still the previous step


def test_the_two_updates_are_not_interchangeable():
    plan, d = plan_tree([2], [50], [-1, 0])
    t = (d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len)
    with pytest.raises(M.MlaError):
        M.mla_plan_update(plan, *t, stream=0)
    causal = M.mla_plan(*t, num_heads=16, page_size=16, num_pages=d.num_pages, sm_scale=SCALE, host_only=True)
    with pytest.raises(M.MlaError):
        M.mla_plan_tree_update(causal, *t, [-1, 0], stream=0)
    with pytest.raises(M.MlaError):
        M.mla_plan_describe_tree(causal)


@pytest.mark.parametrize("parents", [[0, -1], [-1, 1], [-1, 2], [-2, 0], [-1], [-1, 0, 1], [-1, 1 << 30]])
def test_bad_parents(parents):
    with pytest.raises(M.MlaError) as e:
        plan_tree([2], [50], parents)
    assert e.value.status == M.MLA_ERR_INVALID_ARGUMENT


def test_refused_steps():
    for kw, q, k, par in [
        (dict(), [4], [3], [-1, 0, 0, 0]),  # a node without a slot
        (dict(context_only=True), [2], [50], [-1, 0]),
        (dict(), [1025], [2000], [-1] + [0] * 1024),  # a tree beyond the bound
    ]:
        with pytest.raises(M.MlaError) as e:
            plan_tree(q, k, par, **kw)
        assert e.value.status == M.MLA_ERR_INVALID_ARGUMENT
    plan_tree([1025], [2000], list(range(-1, 1024)))  # a chain may be any length
    plan_tree([1024], [1024], [-1] + [0] * 1023)
    plan_tree([0, 0], [50, 0], [])
    plan_tree([], [], [])
    with pytest.raises(M.MlaError):
        plan_tree([8], [50], list(range(-1, 7)), graph_max_batch=2, graph_max_tokens=4, graph_max_page_ids=64)


def test_graph_bucket_holds_the_words_of_every_step():
    """The words of any step of a bucket fit the bound that sizes its buffer: a row of q
    nodes spans at most (q + 126) / 64 key tiles."""
    rng = np.random.default_rng(5)
    for _ in range(200):
        q = int(rng.integers(2, 300))
        ctx = int(rng.integers(0, 200))
        plan, _ = plan_tree([q], [q + ctx], [-1] + [0] * (q - 1), H=16, P=16, split_keys=-1)
        words = len(M.mla_plan_describe_tree(plan)["words"])
        if q > 2:
            assert q * ((q + 63) // 64) <= words <= q * ((q + 126) // 64)


# ------------------------------------------------------------------ C ABI refusals
def _caches(n):
    bufs = [ctypes.create_string_buffer(16 * 1152 * 4 + 16) for _ in range(n)]
    at = [(ctypes.addressof(b) + 15) & ~15 for b in bufs]
    return bufs, at


def test_verify_and_compact_need_a_device_tree_plan():
    lib = M.load_library()
    plan, d = plan_tree([2], [50], [-1, 0])  # host only
    causal = M.mla_plan(d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len, num_heads=16, page_size=16,
                        num_pages=d.num_pages, sm_scale=SCALE, host_only=True)
    keep, at = _caches(1)
    a = at[0]
    ptrs = (ctypes.c_void_p * 1)(a)
    for h in (plan.handle, causal.handle, None):
        assert lib.mla_verify_tree(h, a, a, 8, None, 0, 8, 0, a, a, a, a, a, None) == M.MLA_ERR_INVALID_ARGUMENT
        assert lib.mla_compact_kv(h, a, a, ptrs, 1, None) == M.MLA_ERR_INVALID_ARGUMENT
    assert lib.mla_plan_describe_tree(None, None, None, None, None) == M.MLA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("change,status", [
    (dict(src=[4, 1]), 1), (dict(src=[-1, 1]), 1), (dict(dst=[2, 4]), 1), (dict(dst=[-1, 3]), 1),
    (dict(dst=[2, 2]), 1),  # one destination twice
    (dict(dst=[2, 0]), 1),  # a page both read and written
    (dict(src=[2, 0], dst=[2, 3]), 1),  # a page onto itself
    (dict(tokens=[17, 0]), 1), (dict(tokens=[-1, 0]), 1),
    (dict(n=-1), 1), (dict(caches=-1), 1), (dict(width=32), 2), (dict(page=24), 2), (dict(pages=0), 1),
    (dict(null_src=True), 1), (dict(null_cache=True), 1), (dict(odd_cache=True), 1), (dict(same_cache=True), 1),
    (dict(overlap=True), 1), (dict(no_dims=True), 1),
])
def test_copy_pages_refusals(change, status):
    lib = M.load_library()
    keep, at = _caches(2)
    g = dict(src=[0, 1], dst=[2, 3], tokens=None, n=2, caches=2, width=64, page=16, pages=4)
    g.update({k: v for k, v in change.items() if k in g})
    i32 = lambda v: (ctypes.c_int32 * len(v))(*v)  # noqa: E731
    if change.get("null_cache"):
        at[1] = None
    if change.get("odd_cache"):
        at[1] += 8
    if change.get("same_cache"):
        at[1] = at[0]
    if change.get("overlap"):
        at[1] = at[0] + 16
    dims = M._Dims(16, 512, g["width"], g["page"], g["pages"], 1.0)
    st = lib.mla_copy_pages(None if change.get("no_dims") else ctypes.byref(dims),
                            None if change.get("null_src") else i32(g["src"]), i32(g["dst"]),
                            None if g["tokens"] is None else i32(g["tokens"]), g["n"],
                            (ctypes.c_void_p * 2)(*at), g["caches"], None)
    assert st == status


def test_copy_of_nothing_is_ok():
    lib = M.load_library()
    dims = M._Dims(16, 512, 64, 16, 4, 1.0)
    assert lib.mla_copy_pages(ctypes.byref(dims), None, None, None, 0, None, 0, None) == M.MLA_OK
    one = (ctypes.c_int32 * 1)(1)
    zero = (ctypes.c_int32 * 1)(0)
    assert lib.mla_copy_pages(ctypes.byref(dims), zero, one, None, 1, None, 0, None) == M.MLA_OK
    keep, at = _caches(1)
    assert lib.mla_copy_pages(ctypes.byref(dims), zero, one, zero, 1, (ctypes.c_void_p * 1)(at[0]), 1,
                              None) == M.MLA_OK  # no tokens: nothing to launch


def test_python_checks():
    import torch

    plan, _ = plan_tree([2], [50], [-1, 0])
    cpu = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        M.mla_verify_tree(plan, cpu[0], cpu, cpu[0], cpu[0])
    with pytest.raises(ValueError):
        M.mla_compact_kv(plan, cpu, cpu, [torch.zeros(9, 16, 576, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        M.mla_copy_pages([0], [1], [torch.zeros(9, 16, 576, dtype=torch.bfloat16)])
    with pytest.raises(M.MlaError):
        M.mla_copy_pages([0], [1, 2], [torch.zeros(9, 16, 576, dtype=torch.bfloat16)])
    M.mla_copy_pages([], [], [])


def test_python_checks_survive_odd_arguments():
    """Arguments of other kinds raise; a destroyed plan does; nothing is called."""
    import torch

    plan, _ = plan_tree([2], [50], [-1, 0])
    for bad in (None, 3, "x", [1], torch.zeros(2, 0), torch.zeros(2, 8, dtype=torch.float16)):
        with pytest.raises(ValueError):
            M.mla_verify_tree(plan, bad, bad, bad, bad)
    for caches in (None, 5):
        with pytest.raises(TypeError):
            M.mla_compact_kv(plan, torch.zeros(2), torch.zeros(1), caches)
        with pytest.raises(TypeError):
            M.mla_copy_pages([0], [1], caches)
    with pytest.raises(ValueError):
        M.mla_copy_pages([0], [1], [object()])
    with pytest.raises(ValueError):
        M.mla_compact_kv(plan, torch.zeros(2), torch.zeros(1), [object()])
    plan.destroy()
    with pytest.raises(RuntimeError):
        M.mla_compact_kv(plan, torch.zeros(2), torch.zeros(1), [])
