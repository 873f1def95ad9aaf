"""fp64 CPU oracle of the speculative-decoding operators (test infrastructure only).

Independent of the CUDA library: every function follows the definitions in
``include/mla.h`` (mla_plan_tree, mla_verify_tree, mla_compact_kv, mla_copy_pages) key by
key and node by node, with no vectorised masks.
"""

import math

import numpy as np

from .mla_oracle import _f64, _i64, gather_row_keys, key_location, kv_lengths


def path_of(parents, node):
    """Node indices from the root of ``node``'s tree to ``node``."""
    out = []
    while node >= 0:
        out.append(int(node))
        node = int(parents[node])
    return out[::-1]


def tree_attention(q_nope, q_pe, cache, qo_indptr, kv_indptr, kv_indices, last_page_len, parents, page_size,
                   sm_scale):
    """(out, lse, mass): mass[t, h, d] = sum_j w_j |ckv_j[d]|, which bounds the effect of
    a relative error of the weights."""
    qn = _f64(q_nope)
    qp = _f64(q_pe) if q_pe is not None else None
    qo, par = _i64(qo_indptr), _i64(parents)
    T, H = qn.shape[:2]
    out = np.zeros((T, H, 512))
    mass = np.zeros((T, H, 512))
    lse = np.full((T, H), -np.inf)
    k_all = kv_lengths(kv_indptr, last_page_len, page_size)
    for b in range(len(qo) - 1):
        n, k_b = int(qo[b + 1] - qo[b]), int(k_all[b])
        if n == 0:
            continue
        keys = gather_row_keys(cache, kv_indptr, kv_indices, page_size, b, k_b)
        c = k_b - n
        for i in range(n):
            t = int(qo[b]) + i
            seen = list(range(c)) + [c + a for a in path_of(par[qo[b]: qo[b + 1]], i)]
            kk = keys[seen]
            s = qn[t] @ kk[:, :512].T
            if qp is not None and qp.shape[-1]:
                s = s + qp[t] @ kk[:, 512:].T
            s = s * sm_scale
            m = s.max(axis=1, keepdims=True)
            e = np.exp(s - m)
            z = e.sum(axis=1, keepdims=True)
            w = e / z
            lse[t] = (m + np.log(z))[:, 0]
            out[t] = w @ kk[:, :512]
            mass[t] = w @ np.abs(kk[:, :512])
    return out, lse, mass


def _weights(row):
    w = np.asarray(row, dtype=np.float64).copy()
    w[~(np.isfinite(w) & (w > 0))] = 0.0
    return w


def verify_tree(qo_indptr, parents, draft_tokens, target, uniform, uniform_next, draft=None):
    """(accept_index [T], num_accepted [B], next_token [B]) of rows of probabilities given
    as arrays of float."""
    qo, par = _i64(qo_indptr), _i64(parents)
    V = target.shape[1]
    B = len(qo) - 1
    accept = np.full(int(qo[-1]), -1, dtype=np.int32)
    count, nxt = np.zeros(B, dtype=np.int32), np.full(B, -1, dtype=np.int32)
    for b in range(B):
        t0, n = int(qo[b]), int(qo[b + 1] - qo[b])
        if n == 0:
            continue
        tree = par[t0: t0 + n]
        v, path = 0, [0]
        while True:
            p = _weights(target[t0 + v])
            q = _weights(draft[t0 + v]) if draft is not None else None
            w, Z, got = p.copy(), 1.0, -1
            for c in np.nonzero(tree == v)[0]:
                x, u = int(draft_tokens[t0 + c]), float(uniform[t0 + c])
                if x < 0:
                    got = int(c)
                    break
                wx = w[x] if x < V else 0.0
                qx = (q[x] if x < V else 0.0) if q is not None else 1.0
                if u * qx * Z < wx:
                    got = int(c)
                    break
                if q is not None:
                    w = np.maximum(w - Z * q, 0.0)
                    Z = math.fsum(w)
                else:
                    Z = max(Z - wx, 0.0)
                    if x < V:
                        w[x] = 0.0
            if got < 0:
                break
            v = got
            path.append(v)
        accept[t0: t0 + len(path)] = path
        count[b] = len(path)
        if not w.any():
            w = p
        total = math.fsum(w)
        if total > 0:
            run = np.cumsum(w)
            hits = np.nonzero((run > float(uniform_next[b]) * total) & (w > 0))[0]
            nxt[b] = hits[0] if len(hits) else np.nonzero(w > 0)[0][-1]
    return accept, count, nxt


def compact_kv(cache, qo_indptr, kv_indptr, kv_indices, last_page_len, page_size, accept_index, num_accepted):
    """The cache (any array of [pages, page_size, width]) after the move."""
    out = cache.copy()
    qo = _i64(qo_indptr)
    k_all = kv_lengths(kv_indptr, last_page_len, page_size)
    for b in range(len(qo) - 1):
        t0, n = int(qo[b]), int(qo[b + 1] - qo[b])
        for k in range(min(int(num_accepted[b]), n)):
            a = int(accept_index[t0 + k])
            if not k <= a < n:
                continue
            c = int(k_all[b]) - n
            out[key_location(kv_indptr, kv_indices, page_size, b, c + k)] = \
                cache[key_location(kv_indptr, kv_indices, page_size, b, c + a)]
    return out


def copy_pages(cache, src, dst, num_tokens=None):
    out = cache.copy()
    for i, (s, d) in enumerate(zip(src, dst)):
        n = cache.shape[1] if num_tokens is None else int(num_tokens[i])
        out[d, :n] = cache[s, :n]
    return out
