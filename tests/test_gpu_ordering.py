"""What a stream may rely on: the order of the library's launches among the stream's other
work, and how long a plan's buffers stay its own where several streams use it."""

import gc

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


# ------------------------------------------------------------------ several streams, one plan
CALLS = ["append", "run_append", "verify", "compact"]


class Step:
    """A tree plan over eight rows, and calls on it that two streams may make side by side
    (each has outputs of its own, made beforehand: an allocation may wait for the device; a
    compaction of empty paths moves nothing)."""

    def __init__(self, **kw):
        self.d = d = make_custom([4] * 8, [100] * 8, 16, 16, seed=52)
        self.plan = plan_of(d, True, **kw)
        self.q = d.q_nope.to(DEV), d.q_pe.to(DEV)
        self.cache = d.cache.to(DEV)
        self.kv = torch.zeros((32, 576), dtype=torch.bfloat16, device=DEV)
        self.probs = torch.full((32, 64), 1 / 64, device=DEV)
        self.tok = torch.zeros(32, dtype=torch.int32, device=DEV)
        self.u = torch.zeros(32, device=DEV)
        self.acc = torch.full((32,), -1, dtype=torch.int32, device=DEV)
        self.cnt = torch.zeros(8, dtype=torch.int32, device=DEV)
        self.out = torch.zeros_like(self.q[0])
        self.verified = [[torch.zeros(n, dtype=torch.int32, device=DEV) for n in (32, 8, 8)] for _ in range(2)]
        gc.collect()  # (a plan that is collected waits for its own calls)
        torch.cuda.synchronize()

    def call(self, what, i=0):
        if what == "append":
            M.mla_append_kv(self.plan, self.kv, self.cache)
        elif what == "run_append":
            M.mla_run(self.plan, *self.q, self.cache, out=self.out, kv_new=self.kv)
        elif what == "verify":
            M.mla_verify_tree(self.plan, self.tok, self.probs, self.u, self.u[:8], None, *self.verified[i])
        else:
            M.mla_compact_kv(self.plan, self.acc, self.cnt, [self.cache])


@pytest.fixture(scope="module")
def loaded(lib):
    """Every kernel has run once: a kernel's first launch loads it, which may wait for the
    device."""
    step = Step()
    for what in CALLS:
        step.call(what)
    assert M.mla_plan_check(step.plan) == M.MLA_OK


def delayed(stream, f):
    """Enqueue f on the stream behind 0.3 s or so of other work; the event after it."""
    with torch.cuda.stream(stream):
        torch.cuda._sleep(600_000_000)
        f()
        return stream.record_event()


@pytest.mark.parametrize("after", ["destroy", "check", "grow"])
@pytest.mark.parametrize("first", CALLS)
def test_a_plan_waits_for_its_calls_on_every_stream(first, after, loaded):
    """The buffers of a plan that is destroyed go to the next one: not before the last call
    on each stream is done."""
    step = Step()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    done = delayed(a, lambda: step.call(first))
    with torch.cuda.stream(b):
        step.call("verify", 1)
    assert not done.query()
    if after == "destroy":
        step.plan.destroy()
    elif after == "check":
        assert M.mla_plan_check(step.plan) == M.MLA_OK
    else:
        rows = np.arange(4001, dtype=np.int32)  # of one page each, the same page
        M.mla_plan_tree_update(step.plan, 4 * rows, rows, 0 * rows[1:], 4 + 0 * rows[1:],
                               np.tile(np.arange(-1, 3, dtype=np.int32), 4000), stream=b.cuda_stream)
    assert done.query()
    torch.cuda.synchronize()


def test_a_plan_waits_for_many_streams(loaded):
    """More streams than a plan keeps events for."""
    step = Step()
    streams = [torch.cuda.Stream() for _ in range(20)]
    done = [delayed(s, lambda: step.call("compact")) for s in streams[:3]]
    for s in streams[3:]:
        with torch.cuda.stream(s):
            step.call("verify")
            done.append(s.record_event())
    assert not done[0].query()
    step.plan.destroy()
    assert all(e.query() for e in done)
    torch.cuda.synchronize()


def test_calls_on_two_streams_do_not_wait_for_one_another(loaded):
    step = Step()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    late = delayed(a, lambda: step.call("compact"))
    with torch.cuda.stream(b):
        for what in ("verify", "compact", "verify"):
            step.call(what)
        b.synchronize()
    assert not late.query()
    torch.cuda.synchronize()


def test_a_captured_append_is_waited_for(loaded):
    """A graph that captured only an append may replay on any stream."""
    step = Step(graph_max_batch=8, graph_max_tokens=32, graph_max_page_ids=56)
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        step.call("append")
    done = delayed(s, g.replay)
    assert not done.query()
    step.plan.destroy()
    assert done.query()
    torch.cuda.synchronize()
    del g


# ------------------------------------------------------------------ outputs that a call makes
@pytest.mark.parametrize("what", ["run", "verify"])
def test_outputs_belong_to_the_stream_of_the_call(what, loaded):
    """A call on a stream that is not torch's current one writes there: what the current
    stream freed may still be in use on it, and what the call made is not the current
    stream's to hand out once it is freed."""
    step = Step()
    s = torch.cuda.Stream()

    def make(stream):
        if what == "run":
            return M.mla_run(step.plan, *step.q, step.cache, return_lse=True, stream=stream)
        return M.mla_verify_tree(step.plan, step.tok, step.probs, step.u, step.u[:8], stream=stream)

    want = [x.clone() for x in make(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    first = make(None)
    freed = {x.untyped_storage().data_ptr() for x in first}
    torch.cuda.synchronize()
    del first  # (nothing is pending here: only the addresses are looked at)
    got = make(s.cuda_stream)
    s.synchronize()
    there = {x.untyped_storage().data_ptr() for x in got}
    assert not there & freed
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del got
    again = make(None)
    torch.cuda.synchronize()
    assert not {x.untyped_storage().data_ptr() for x in again} & there
    got = make(s.cuda_stream)  # (the stream itself uses its memory again)
    assert {x.untyped_storage().data_ptr() for x in got} == there
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        assert all(torch.equal(a, b) for a, b in zip(make(s.cuda_stream), want))
        assert all(torch.equal(a, b) for a, b in zip(make(None), want))
    with torch.inference_mode():
        assert all(torch.equal(a, b) for a, b in zip(make(None), want))
    torch.cuda.synchronize()


# ------------------------------------------------------------------ replays are not checked
def test_a_replayed_compaction_of_shared_slots_moves_what_the_plan_still_places():
    """A step in which two rows' tokens name the same slots is refused by a call; a graph
    captured on another step of the bucket moves only the rows of the later tokens."""
    P = 16
    apart = make_custom([3, 3], [20, 20], 16, P, seed=55, extra_pool_pages=2)
    qo, kvp, kvi, last = tables(apart)
    shared = kvi.clone()
    shared[2:] = shared[:2]
    kw = dict(num_heads=16, page_size=P, num_pages=apart.num_pages, sm_scale=apart.sm_scale)
    parents = [-1, 0, 0] * 2
    plan = M.mla_plan_tree(qo, kvp, kvi, last, parents, graph_max_batch=2, graph_max_tokens=6, graph_max_page_ids=8,
                           **kw)
    cache = apart.cache.to(DEV)
    acc = torch.tensor([0, 2, -1, 0, 2, -1], dtype=torch.int32, device=DEV)
    cnt = torch.full((2,), 2, dtype=torch.int32, device=DEV)
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        M.mla_compact_kv(plan, acc, cnt, cache)
    with torch.cuda.stream(s):
        M.mla_plan_tree_update(plan, qo, kvp, shared, last, parents)
        with pytest.raises(M.MlaError):
            M.mla_compact_kv(plan, acc, cnt, cache)
        g.replay()
    s.synchronize()
    want = apart.cache.clone()
    page = int(shared[1])  # keys 17, 18 and 19 are its slots 1, 2 and 3
    want[page, 2] = want[page, 3]
    assert torch.equal(cache.cpu(), want)
    del g
    plan.destroy()


def test_the_same_verification_gives_the_same_result():
    """Weights whose sums round, in calls that share a plan's rows and buffers."""
    rng = np.random.default_rng(56)
    T, V = 40 * 9, 5003
    d = make_custom([9] * 40, [9] * 40, 16, 16, seed=56, tables_only=True)
    plan = M.mla_plan_tree(*tables(d), [-1, 0, 0, 0, 1, 1, 4, 4, 4] * 40, num_heads=16, page_size=16,
                           num_pages=d.num_pages, sm_scale=d.sm_scale)
    p, q = (torch.softmax(torch.from_numpy(rng.standard_normal((T, V)) * 2).float(), 1).to(DEV) for _ in range(2))
    tok = torch.multinomial(q, 1).flatten().to(torch.int32)
    u, un = torch.rand(T, device=DEV), torch.rand(40, device=DEV)
    first = M.mla_verify_tree(plan, tok, p, u, un, draft_probs=q)
    for _ in range(20):
        again = M.mla_verify_tree(plan, tok, p, u, un, draft_probs=q)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


# ------------------------------------------------------------------ shared memory
def test_verification_refuses_outputs_in_its_inputs():
    """Outputs are written while inputs are read; rows of weights may be parts of one matrix."""
    d = make_custom([3, 2], [3, 2], 16, 16, seed=57, tables_only=True)
    plan = M.mla_plan_tree(*tables(d), [-1, 0, 0, -1, 0], num_heads=16, page_size=16, num_pages=d.num_pages,
                           sm_scale=d.sm_scale)
    both = torch.full((5, 64), 1 / 32, device=DEV)
    ints = torch.zeros(32, dtype=torch.int32, device=DEV)
    f = torch.zeros(16, device=DEV)
    good = dict(draft_tokens=ints[:5], uniform=f[:5], uniform_next=f[5:7], target_probs=both[:, :32],
                draft_probs=both[:, 32:], accept_index=ints[5:10], num_accepted=ints[10:12], next_token=ints[12:14])
    out = M.mla_verify_tree(plan, **good)
    assert out[0].data_ptr() == ints[5:].data_ptr() and ints[5:14].tolist() == [0, 1, -1, 0, 1, 2, 2, 0, 0]
    as_ints = both.view(torch.int32).view(-1)
    for bad in [dict(accept_index=ints[:5]), dict(accept_index=ints[4:9]), dict(num_accepted=ints[9:11]),
                dict(next_token=ints[11:13]), dict(next_token=f.view(torch.int32)[6:8]),
                dict(num_accepted=f.view(torch.int32)[4:6]), dict(accept_index=as_ints[64 * 4 + 31:][:5]),
                dict(next_token=as_ints[64 * 5 - 2:])]:
        with pytest.raises(M.MlaError) as e:
            M.mla_verify_tree(plan, **{**good, **bad})
        assert e.value.status == M.MLA_ERR_INVALID_ARGUMENT
