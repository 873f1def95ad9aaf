"""What a stream may rely on: the order of the library's launches among the stream's other
work, and how long a plan's buffers stay its own where several streams use it."""

import numpy as np
import pytest
import torch

import paged_head_latent_mla_b200 as M
from workloads import make_custom

pytestmark = pytest.mark.gpu

TIMEOUT_NS = 500_000_000
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_head_latent_mla_b200 import _build

    _build.build()
    return M.load_library()


def tables(d):
    return d.qo_indptr, d.kv_indptr, d.kv_indices, d.last_page_len


def plan_of(d, tree, **kw):
    geometry = dict(num_heads=d.num_heads, page_size=d.page_size, num_pages=d.num_pages, sm_scale=d.sm_scale,
                    wait_timeout_ns=TIMEOUT_NS, **kw)
    if not tree:
        return M.mla_plan(*tables(d), **geometry)
    qo = d.qo_indptr.tolist()
    parents = np.concatenate([np.arange(-1, b - a - 1) for a, b in zip(qo, qo[1:])]).astype(np.int32)
    return M.mla_plan_tree(*tables(d), parents, **geometry)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_what_follows_a_graph_plan_waits_for_its_attention(tree, captured):
    """A graph plan launches the merge of split keys for every step, also for one that
    splits nothing; what the stream holds next starts after the attention all the same."""
    d = make_custom([1] * 60, [2500] * 60, 128, 64, seed=51)
    plan = plan_of(d, tree, split_keys=-1, graph_max_batch=64, graph_max_tokens=64,
                   graph_max_page_ids=len(d.kv_indices))
    assert M.mla_plan_get_info(plan)["num_merge"] == 0
    qn = torch.zeros((64, 128, 512), dtype=torch.bfloat16, device=DEV)
    qp = torch.zeros((64, 128, 64), dtype=torch.bfloat16, device=DEV)
    qn[:60].copy_(d.q_nope)
    qp[:60].copy_(d.q_pe)
    keep = d.cache.to(DEV)
    cache = keep.clone()
    want = M.mla_run(plan, qn, qp, cache)[:60].clone()
    assert M.mla_plan_check(plan) == M.MLA_OK
    out = torch.zeros_like(qn)
    seen = torch.zeros_like(qn)
    s = torch.cuda.Stream()

    def step():
        cache.copy_(keep)
        out.zero_()
        M.mla_run(plan, qn, qp, cache, out=out)
        seen.copy_(out)
        cache.fill_(100.0)

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    if captured:
        with torch.cuda.graph(g, stream=s):
            step()
    for _ in range(5):
        with torch.cuda.stream(s):
            g.replay() if captured else step()
        s.synchronize()
        assert torch.equal(out[:60], want) and torch.equal(seen, out)
    assert M.mla_plan_check(plan) == M.MLA_OK
    del g
    plan.destroy()
