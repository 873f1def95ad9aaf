"""The speculative-decoding operators on the paged latent cache, measured as a serving
loop calls them: attention of a tree of drafted tokens, verification of the tree against
the target's probabilities, compaction of the accepted rows, and copies of cache pages.

Each case is a dict whose "op" names the operator:

  attend   rows of ``nodes`` drafted tokens (a tree) over ``ctx_lo..ctx_hi`` stored keys,
           ``heads`` query heads, pages of ``page`` tokens, kpe width ``rope``; with
           ``append`` the step's latent rows are written into the cache first
  verify   ``batch`` trees against target probabilities over ``vocab`` tokens of type
           ``probs``, drafted from given probabilities (``draft``) or as point masses
  compact  the accepted rows of ``batch`` trees in ``layers`` caches
  copy     ``pairs`` pages (``tokens`` tokens of each; 0: whole pages) in ``layers`` caches

Tree shapes, lengths and page tables follow from the case alone, so that ``work`` counts
them exactly; every value (latent rows, queries, probabilities, random numbers, page
order) follows from the seed.
"""

import math
import random
import zlib

import numpy as np
import torch

own = False

CKV = 512  # latent width; a cache row is [ckv 512 | kpe rope]
SCALE = 192 ** -0.5
PROB_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # two short rows with a small tree each: one decode step of an idle server (latency)
        {"name": "attend_tiny", "op": "attend", "batch": 2, "nodes": 7, "ctx_lo": 37, "ctx_hi": 150, "heads": 16,
         "page": 16, "rope": 64, "append": True},
        # a full decode batch, 16 drafted tokens per row, all 128 heads on this GPU
        {"name": "attend_b64", "op": "attend", "batch": 64, "nodes": 16, "ctx_lo": 512, "ctx_hi": 8192, "heads": 128,
         "page": 64, "rope": 64, "append": False},
        # long contexts with the heads sharded to 16: one query tile per row, keys split
        {"name": "attend_long_h16", "op": "attend", "batch": 16, "nodes": 8, "ctx_lo": 32768, "ctx_hi": 32768,
         "heads": 16, "page": 64, "rope": 64, "append": False},
        # wide trees (many candidate continuations of few prompts), ragged, no rope part
        {"name": "attend_wide", "op": "attend", "batch": 4, "nodes": 257, "ctx_lo": 1000, "ctx_hi": 4096, "heads": 64,
         "page": 32, "rope": 0, "append": True},
        # one chain of four drafted tokens (latency)
        {"name": "verify_one", "op": "verify", "batch": 1, "nodes": 5, "vocab": 32768, "probs": "fp32",
         "draft": True},
        # a full batch of sampled trees over a large vocabulary
        {"name": "verify_b64", "op": "verify", "batch": 64, "nodes": 16, "vocab": 131072, "probs": "fp32",
         "draft": True},
        # top-k drafted trees (point masses), 16-bit probabilities, rows of odd length
        {"name": "verify_point_b128", "op": "verify", "batch": 128, "nodes": 9, "vocab": 65537, "probs": "bf16",
         "draft": False},
        # one row in one layer's cache (latency)
        {"name": "compact_one", "op": "compact", "batch": 1, "nodes": 8, "ctx_lo": 1000, "ctx_hi": 1000, "page": 16,
         "rope": 64, "layers": 1},
        # a decode batch through every layer of a model
        {"name": "compact_b64_layers", "op": "compact", "batch": 64, "nodes": 16, "ctx_lo": 64, "ctx_hi": 128,
         "page": 64, "rope": 64, "layers": 48},
        # fork of one sequence: its partly filled last page in one layer (latency)
        {"name": "fork_one", "op": "copy", "pairs": 1, "tokens": 37, "pool": 64, "page": 64, "rope": 64, "layers": 1},
        # a batch of forks through every layer
        {"name": "fork_b64_layers", "op": "copy", "pairs": 64, "tokens": 0, "pool": 160, "page": 64, "rope": 64,
         "layers": 48},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "verify", "verify", "compact", "copy"])
    if op == "attend":
        heads = rng.choice([16, 32, 64, 128])
        batch, nodes = _log_int(rng, 1, 64), _log_int(rng, 1, 257)
        while batch * nodes > 1028:  # the tokens of a step
            batch = max(1, batch // 2)
        hi = _log_int(rng, 40, 32768)
        while batch * nodes * heads * hi > 64 * 16 * 128 * 4096:
            hi = max(1, hi // 2)
        return {"op": op, "batch": batch, "nodes": nodes, "ctx_lo": rng.randint(0, hi), "ctx_hi": hi, "heads": heads,
                "page": rng.choice([16, 32, 64, 128]), "rope": rng.choice([0, 64, 64]),
                "append": rng.random() < 0.5}
    if op == "verify":
        batch, nodes, vocab = _log_int(rng, 1, 128), _log_int(rng, 1, 33), _log_int(rng, 1000, 131072)
        while batch * nodes * vocab > 64 * 16 * 131072:
            batch = max(1, batch // 2)
        return {"op": op, "batch": batch, "nodes": nodes, "vocab": vocab, "probs": rng.choice(["fp32", "bf16"]),
                "draft": rng.random() < 0.6}
    page = rng.choice([16, 32, 64, 128])
    rope = rng.choice([0, 64, 64])
    if op == "compact":
        batch, nodes, hi = _log_int(rng, 1, 64), _log_int(rng, 2, 33), rng.randint(1, 128)
        return {"op": op, "batch": batch, "nodes": nodes, "ctx_lo": rng.randint(0, hi), "ctx_hi": hi, "page": page,
                "rope": rope, "layers": _log_int(rng, 1, 48)}
    pairs = _log_int(rng, 1, 64)
    return {"op": op, "pairs": pairs, "tokens": rng.choice([0, rng.randint(1, page)]),
            "pool": 2 * pairs + rng.randint(0, 32), "page": page, "rope": rope, "layers": _log_int(rng, 1, 32)}


# ------------------------------------------------------------------ shapes of a case
def _shape_rng(case):
    """A generator of the case's own shapes (the same for every seed)."""
    text = ",".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name")
    return random.Random(zlib.crc32(text.encode()))


def _tree(rng, nodes):
    """Parents of a drafted tree: a main chain of about half the nodes first, then side
    branches hanging from any node that leaves them no deeper than the chain."""
    chain = max(1, (nodes + 1) // 2)
    parents = [i - 1 for i in range(chain)]
    depth = list(range(chain))
    for i in range(chain, nodes):
        fits = [j for j in range(i) if depth[j] + 1 < chain] or [0]
        j = rng.choice(fits)
        parents.append(j)
        depth.append(depth[j] + 1)
    return parents


def _path(parents, node):
    out = []
    while node >= 0:
        out.append(node)
        node = parents[node]
    return out[::-1]


def _rows(case):
    """(context lengths, parents per row, an accepted path per row).  In a batch of
    several rows one in eight drafts fewer nodes, as when a draft ends early."""
    rng = _shape_rng(case)
    batch, nodes = case["batch"], case["nodes"]
    ctx, trees, paths = [], [], []
    for b in range(batch):
        ctx.append(rng.randint(case.get("ctx_lo", 0), case.get("ctx_hi", 0)))
        n = rng.randint(1, nodes) if batch > 1 and b % 8 == 7 else nodes
        trees.append(_tree(rng, n))
        paths.append(_path(trees[-1], rng.randrange(max(0, n // 2), n)))
    return ctx, trees, paths


def _tables(case, ctx, trees, order):
    """Host tables of the step: the rows' pages are ``order``'s first ids."""
    page = case["page"]
    q = [len(t) for t in trees]
    k = [c + n for c, n in zip(ctx, q)]
    n_pages = [-(-x // page) for x in k]
    qo = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    kvp = np.concatenate([[0], np.cumsum(n_pages)]).astype(np.int32)
    last = np.array([x - (n - 1) * page for x, n in zip(k, n_pages)], dtype=np.int32)
    kvi = np.asarray(order[: int(kvp[-1])], dtype=np.int32)
    parents = np.concatenate([np.asarray(t, dtype=np.int32) for t in trees])
    return qo, kvp, kvi, last, parents


def _pool(case, ctx, trees):
    page = case["page"]
    return sum(-(-(c + len(t)) // page) for c, t in zip(ctx, trees)) + 3


def _randn(shape, gen, std=0.5):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for s in range(0, flat.numel(), 1 << 27):
        e = min(flat.numel(), s + (1 << 27))
        flat[s:e] = torch.randn(e - s, generator=gen, device="cuda", dtype=torch.float32) * std
    return out


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(1000003 * (seed % (1 << 40)) + 17)
    host = random.Random(seed)
    st = {"case": case}
    op = case["op"]
    if op == "copy":
        width = CKV + case["rope"]
        st["caches"] = [_randn((case["pool"], case["page"], width), gen) for _ in range(case["layers"])]
        ids = list(range(case["pool"]))
        host.shuffle(ids)
        st["src"] = np.asarray(ids[: case["pairs"]], dtype=np.int32)
        st["dst"] = np.asarray(ids[case["pairs"]: 2 * case["pairs"]], dtype=np.int32)
        st["tokens"] = np.full(case["pairs"], case["tokens"], dtype=np.int32) if case["tokens"] else None
        st["src_dev"] = torch.from_numpy(st["src"].astype(np.int64)).cuda()
        st["dst_dev"] = torch.from_numpy(st["dst"].astype(np.int64)).cuda()
        return st

    ctx, trees, paths = _rows(case)
    page = case.get("page", 64)
    tab = dict(case, page=page)
    pool = _pool(tab, ctx, trees)
    order = list(range(pool))
    host.shuffle(order)
    qo, kvp, kvi, last, parents = _tables(tab, ctx, trees, order)
    T = int(qo[-1])
    st.update(ctx=ctx, trees=trees, qo=qo, kvp=kvp, kvi=kvi, last=last, parents=parents)
    heads, rope = case.get("heads", 16), case.get("rope", 64)
    width = CKV + rope
    if op == "attend":
        st["cache"] = _randn((pool, page, width), gen)
        st["q_nope"] = _randn((T, heads, CKV), gen)
        st["q_pe"] = _randn((T, heads, rope), gen) if rope else None
        st["kv_new"] = _randn((T, width), gen) if case["append"] else None
        # the tree's mask over each row's own nodes, and the rows' key positions
        st["masks"] = [torch.from_numpy(_ancestors(t)).cuda() for t in trees]
        st["pages"] = [torch.from_numpy(kvi[kvp[b]: kvp[b + 1]].astype(np.int64)).cuda() for b in range(len(trees))]
        st["slots"] = torch.cat([_slots(st["pages"][b], ctx[b], len(t), page) for b, t in enumerate(trees)])
    elif op == "compact":
        st["caches"] = [_randn((pool, page, width), gen) for _ in range(case["layers"])]
        acc = np.full(T, -1, dtype=np.int32)
        for b, p in enumerate(paths):
            acc[qo[b]: qo[b] + len(p)] = p
        st["accept_index"] = torch.from_numpy(acc).cuda()
        st["num_accepted"] = torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda")
        pages = [torch.from_numpy(kvi[kvp[b]: kvp[b + 1]].astype(np.int64)).cuda() for b in range(len(trees))]
        st["slots"] = torch.cat([_slots(pages[b], ctx[b], len(t), page) for b, t in enumerate(trees)])
        st["row_of"] = torch.from_numpy(np.repeat(np.arange(len(trees)), np.diff(qo))).cuda()
        st["qo_dev"] = torch.from_numpy(qo.astype(np.int64)).cuda()
        st["paths"] = paths
    else:
        V, kind = case["vocab"], PROB_TYPES[case["probs"]]
        # a peaked target and a draft near it; each drafted token is drawn from the draft's
        # distribution at its parent (sampled) or is one of its most likely ones (point mass)
        par = np.concatenate([np.asarray(t, dtype=np.int64) + qo[b] for b, t in enumerate(trees)])
        first = np.zeros(T, dtype=bool)
        first[qo[:-1]] = True
        rank = np.zeros(T, dtype=np.int64)  # how many earlier siblings a node has
        seen = {}
        for t in range(T):
            if not first[t]:
                rank[t] = seen.get(int(par[t]), 0)
                seen[int(par[t])] = int(rank[t]) + 1
        st["target"] = torch.empty((T, V), dtype=kind, device="cuda")
        st["draft"] = torch.empty((T, V), dtype=kind, device="cuda") if case["draft"] else None
        most = max(seen.values(), default=1)
        picks = torch.empty((T, most), dtype=torch.int64, device="cuda")
        for s in range(0, T, 64):
            n = min(64, T - s)
            z = torch.randn((n, V), generator=gen, device="cuda") * 3.0
            st["target"][s: s + n] = torch.softmax(z, 1)
            z += torch.randn((n, V), generator=gen, device="cuda") * 0.7
            d = torch.softmax(z, 1)
            if case["draft"]:
                st["draft"][s: s + n] = d
                c = d.double().cumsum(1)
                u = torch.rand((n, most), generator=gen, device="cuda", dtype=torch.float64) * c[:, -1:]
                picks[s: s + n] = torch.searchsorted(c, u, right=True).clamp_(max=V - 1)
            else:
                picks[s: s + n] = d.topk(most, dim=1).indices
        par_dev = torch.from_numpy(np.where(first, np.arange(T), par)).cuda()
        st["tokens"] = picks[par_dev, torch.from_numpy(rank).cuda()].to(torch.int32)
        st["uniform"] = torch.rand(T, generator=gen, device="cuda", dtype=torch.float32)
        st["uniform_next"] = torch.rand(len(trees), generator=gen, device="cuda", dtype=torch.float32)
        # children of every token, in order (-1 behind the last), for the plain form
        kids = np.full((T, most), -1, dtype=np.int64)
        for t in range(T):
            if not first[t]:
                kids[par[t], rank[t]] = t
        st["kids"] = torch.from_numpy(kids).cuda()
        st["depth"] = max(len(_path(t, i)) for t in trees for i in range(len(t)))
        st["roots"] = torch.from_numpy(qo[:-1].astype(np.int64)).cuda()
    if own:
        import paged_head_latent_mla_b200 as M

        st["plan"] = M.mla_plan_tree(qo, kvp, kvi, last, parents, num_heads=heads, page_size=page, num_pages=pool,
                                     sm_scale=SCALE, rope_dim=rope)
    return st


def _ancestors(tree):
    """[n, n] truth values: node i sees itself and its ancestors."""
    n = len(tree)
    m = np.zeros((n, n), dtype=bool)
    for i, p in enumerate(tree):
        if p >= 0:
            m[i] = m[p]
        m[i, i] = True
    return m


def _slots(pages, ctx, n, page):
    """Cache rows (over [pool * page]) of a row's n step tokens."""
    pos = torch.arange(ctx, ctx + n, device=pages.device)
    return pages[pos // page] * page + pos % page


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        import paged_head_latent_mla_b200 as M

        if op == "attend":
            out, lse = M.mla_run(st["plan"], st["q_nope"], st["q_pe"], st["cache"], return_lse=True,
                                 kv_new=st["kv_new"])
            return (out, lse, st["cache"]) if st["kv_new"] is not None else (out, lse)
        if op == "verify":
            return M.mla_verify_tree(st["plan"], st["tokens"], st["target"], st["uniform"], st["uniform_next"],
                                     draft_probs=st["draft"])
        if op == "compact":
            M.mla_compact_kv(st["plan"], st["accept_index"], st["num_accepted"], st["caches"])
            return st["caches"]
        M.mla_copy_pages(st["src"], st["dst"], st["caches"], num_tokens=st["tokens"])
        return st["caches"]
    return {"attend": _plain_attend, "verify": _plain_verify, "compact": _plain_compact, "copy": _plain_copy}[op](st)


def _plain_attend(st):
    cache, page = st["cache"], st["case"]["page"]
    width = cache.shape[-1]
    if st["kv_new"] is not None:
        cache.view(-1, width)[st["slots"]] = st["kv_new"]
    out = torch.empty_like(st["q_nope"])
    lse = torch.empty(out.shape[:2], dtype=torch.float32, device=out.device)
    for b, tree in enumerate(st["trees"]):
        t0, n, c = int(st["qo"][b]), len(tree), st["ctx"][b]
        k = cache[st["pages"][b]].view(-1, width)[: c + n].float()
        q = st["q_nope"][t0: t0 + n].float()
        if st["q_pe"] is not None:
            q = torch.cat([q, st["q_pe"][t0: t0 + n].float()], -1)
        s = torch.matmul(q, k.T) * SCALE  # [n, H, keys]
        s[:, :, c:].masked_fill_(~st["masks"][b][:, None, :], -math.inf)
        m = s.amax(-1, keepdim=True)
        s -= m
        s.exp_()
        z = s.sum(-1, keepdim=True)
        out[t0: t0 + n] = torch.matmul(s, k[:, :CKV]) / z
        lse[t0: t0 + n] = (m + z.log())[..., 0]
    return (out, lse, cache) if st["kv_new"] is not None else (out, lse)


def _plain_verify(st):
    """All rows at once, one level of the trees at a time, in 64 bits (acceptance and the
    next token are decided at borders)."""
    p, q, kids = st["target"], st["draft"], st["kids"]
    T, V = p.shape
    B, most = len(st["trees"]), kids.shape[1]
    dev = p.device
    uni, un = st["uniform"].double(), st["uniform_next"].double()
    v = st["roots"].clone()
    alive = torch.ones(B, dtype=torch.bool, device=dev)
    accept = torch.full((T + 1,), -1, dtype=torch.int32, device=dev)
    accept[v] = 0
    count = torch.ones(B, dtype=torch.int64, device=dev)
    final = torch.zeros((B, V), dtype=torch.float64, device=dev)
    rows = torch.arange(B, device=dev)
    for _ in range(st["depth"]):
        w = p[v].double()
        qv = q[v].double() if q is not None else None
        z = torch.ones(B, dtype=torch.float64, device=dev)
        got = torch.full((B,), -1, dtype=torch.int64, device=dev)
        for k in range(most):
            c = kids[v, k]
            test = alive & (c >= 0) & (got < 0)
            at = c.clamp(min=0)
            x = st["tokens"][at].long()
            wx, u = w[rows, x], uni[at]
            limit = u * qv[rows, x] * z if qv is not None else u * z
            ok = test & (limit < wx)
            no = test & ~ok
            if qv is not None:
                w = torch.where(no[:, None], (w - z[:, None] * qv).clamp_(min=0), w)
                z = torch.where(no, w.sum(1), z)
            else:
                z = torch.where(no, (z - wx).clamp(min=0), z)
                w[rows, x] = torch.where(no, torch.zeros_like(wx), wx)
            got = torch.where(ok, c, got)
        ended = alive & (got < 0)
        empty = w.sum(1) == 0
        final = torch.where(ended[:, None], torch.where(empty[:, None], p[v].double(), w), final)
        alive = alive & (got >= 0)
        accept[torch.where(alive, st["roots"] + count, T)] = (got - st["roots"]).int()
        count = count + alive
        v = torch.where(alive, got, v)
    c = final.cumsum(1)
    nxt = torch.searchsorted(c, (un * c[:, -1])[:, None], right=True)[:, 0]
    return accept[:T].contiguous(), count.int(), nxt.int()


def _plain_compact(st):
    page = st["case"]["page"]
    # node k of a row's path goes to the row's k-th step slot
    t = torch.arange(st["slots"].numel(), device="cuda")
    k = t - st["qo_dev"][st["row_of"]]
    keep = k < st["num_accepted"][st["row_of"]]
    src = torch.where(keep, st["qo_dev"][st["row_of"]] + st["accept_index"], t)
    for cache in st["caches"]:
        rows = cache.view(-1, cache.shape[-1])
        rows[st["slots"]] = rows[st["slots"][src]]
    return st["caches"]


def _plain_copy(st):
    n = st["case"]["tokens"] or st["case"]["page"]
    for cache in st["caches"]:
        cache[st["dst_dev"], :n] = cache[st["src_dev"], :n]
    return st["caches"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "copy":
        n = case["tokens"] or case["page"]
        return {"bytes": 2 * case["pairs"] * n * (CKV + case["rope"]) * 2 * case["layers"], "flops": 0}
    ctx, trees, paths = _rows(case)
    T = sum(len(t) for t in trees)
    if op == "attend":
        H, width = case["heads"], CKV + case["rope"]
        keys = sum(c + len(t) for c, t in zip(ctx, trees))
        seen = sum(c + int(a.sum()) for c, t in zip(ctx, trees) for a in _ancestors(t))
        moved = keys * width * 2 + T * H * (width + CKV) * 2 + T * H * 4
        if case["append"]:
            moved += 2 * T * width * 2
        return {"bytes": moved, "flops": 2 * seen * H * (width + CKV)}
    if op == "verify":
        # at least the row that the next token is drawn from, of the target and of the draft
        size = 4 if case["probs"] == "fp32" else 2
        rows = case["batch"] * (2 if case["draft"] else 1)
        return {"bytes": rows * case["vocab"] * size + T * 12 + case["batch"] * 12, "flops": rows * case["vocab"]}
    moved = sum(1 for p in paths for i, a in enumerate(p) if a != i)
    return {"bytes": 2 * moved * (CKV + case["rope"]) * 2 * case["layers"] + 4 * T + 4 * case["batch"], "flops": 0}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return {"attend": _exact_attend, "verify": _exact_verify, "compact": _exact_compact,
            "copy": _exact_copy}[case["op"]](st)


def _exact_attend(st):
    """Key by key positions from the tables; each node's softmax over the list of the keys
    that it sees."""
    cache, page = st["cache"], st["case"]["page"]
    if st["kv_new"] is not None:
        for b, tree in enumerate(st["trees"]):
            for i in range(len(tree)):
                pos = st["ctx"][b] + i
                pg = int(st["kvi"][int(st["kvp"][b]) + pos // page])
                cache[pg, pos % page] = st["kv_new"][int(st["qo"][b]) + i]
    out = torch.zeros(st["q_nope"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    for b, tree in enumerate(st["trees"]):
        c, t0 = st["ctx"][b], int(st["qo"][b])
        stored = torch.cat([cache[int(g)] for g in st["kvi"][st["kvp"][b]: st["kvp"][b + 1]]]).double()
        q = st["q_nope"][t0: t0 + len(tree)].double()
        old = torch.einsum("nhd,kd->nhk", q, stored[:c, :CKV])
        if st["q_pe"] is not None:
            qp = st["q_pe"][t0: t0 + len(tree)].double()
            old = old + torch.einsum("nhd,kd->nhk", qp, stored[:c, CKV:])
        for i in range(len(tree)):
            line = torch.tensor([c + a for a in _path(tree, i)], device="cuda")
            new = q[i] @ stored[line, :CKV].T
            if st["q_pe"] is not None:
                new = new + qp[i] @ stored[line, CKV:].T
            s = torch.cat([old[i], new], 1) * SCALE
            lse[t0 + i] = torch.logsumexp(s, 1)
            w = torch.exp(s - lse[t0 + i][:, None])
            out[t0 + i] = w[:, :c] @ stored[:c, :CKV] + w[:, c:] @ stored[line, :CKV]
    return (out, lse, cache) if st["kv_new"] is not None else (out, lse)


def _exact_verify(st):
    """Row by row and node by node on the host."""
    tok, uni, un = st["tokens"].cpu().numpy(), st["uniform"].cpu().numpy(), st["uniform_next"].cpu().numpy()
    accept = np.full(int(st["qo"][-1]), -1, dtype=np.int32)
    count, nxt = [], []

    def row(m, t):
        return m[t].double().cpu().numpy()

    for b, tree in enumerate(st["trees"]):
        t0, node, path = int(st["qo"][b]), 0, [0]
        while True:
            p = row(st["target"], t0 + node)
            q = row(st["draft"], t0 + node) if st["draft"] is not None else None
            left, mass, chosen = p.copy(), 1.0, None
            for c in [i for i in range(1, len(tree)) if tree[i] == node]:
                x, u = int(tok[t0 + c]), float(uni[t0 + c])
                if u * (q[x] if q is not None else 1.0) * mass < left[x]:
                    chosen = c
                    break
                if q is not None:
                    left = np.maximum(left - mass * q, 0.0)
                    mass = math.fsum(left)
                else:
                    mass = max(mass - left[x], 0.0)
                    left[x] = 0.0
            if chosen is None:
                break
            node = chosen
            path.append(node)
        if not left.any():
            left = p
        c = np.cumsum(left)
        nxt.append(int(np.searchsorted(c, float(un[b]) * c[-1], side="right")))
        accept[t0: t0 + len(path)] = path
        count.append(len(path))
    return (torch.from_numpy(accept), torch.tensor(count, dtype=torch.int32), torch.tensor(nxt, dtype=torch.int32))


def _exact_compact(st):
    page = st["case"]["page"]
    for cache in st["caches"]:
        before = cache.clone()
        for b, path in enumerate(st["paths"]):
            for k, a in enumerate(path):
                if a == k:
                    continue
                to, fr = st["ctx"][b] + k, st["ctx"][b] + a
                base = int(st["kvp"][b])
                cache[int(st["kvi"][base + to // page]), to % page] = \
                    before[int(st["kvi"][base + fr // page]), fr % page]
    return st["caches"]


def _exact_copy(st):
    n = st["case"]["tokens"] or st["case"]["page"]
    for cache in st["caches"]:
        for s, d in zip(st["src"].tolist(), st["dst"].tolist()):
            cache[d, :n] = cache[s, :n].clone()
    return st["caches"]
