"""Calls on another stream than the current one: what they allocate themselves,
results and scratch, is neither memory that the current stream still works on
nor given back to it while the call runs."""
import math

import pytest
import torch

from tests.test_gpu_paged import tq  # noqa: F401

pytestmark = pytest.mark.gpu


def calls(tq):
    """name -> call(stream) that allocates its results and its scratch."""
    d, heads, kv_heads, page, n = 128, 8, 2, 16, 300
    g = torch.Generator(device="cuda").manual_seed(1)

    def rand(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    qk, qv = tq.tq_codebook(d, 4), tq.tq_codebook_mse(d, 4, seed=1)
    x, y = rand(n * kv_heads, d), rand(8, d, dtype=torch.float32)
    kenc, venc = tq.tq_encode(qk, x), tq.tq_encode(qv, x)
    kc, vc = qk.empty_paged(20, kv_heads, page), qv.empty_paged(20, kv_heads, page)
    tq.tq_paged_store(qk, qv, kenc, venc, torch.arange(n, device="cuda"), kc, vc)
    table = torch.arange(20, dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    yq = {m: rand(m, heads * d) for m in (1, 100)}
    start = {m: torch.tensor([0, m], dtype=torch.int32, device="cuda") for m in (1, 100)}
    kv, vv = rand(100, kv_heads * d), rand(100, kv_heads * d)
    logits = tq.tq_score(qk, y, 1, 8, kenc, n * kv_heads)
    rows = n * kv_heads
    cand = torch.arange(48, device="cuda").view(8, 6)

    def flat(r):
        if isinstance(r, tq.Encoded):
            return [r.codes, r.signs, r.norms]
        return list(r) if isinstance(r, tuple) else [r]
    out = {
        "encode": lambda s: tq.tq_encode(qk, x, stream=s),
        "prepare queries": lambda s: tq.tq_prepare_queries(qk, y, stream=s),
        "score": lambda s: tq.tq_score(qk, y, 1, 8, kenc, rows, stream=s),
        "score prepared": lambda s: tq.tq_score_prepared(qk, 1, 8, kenc, rows, tq.tq_score_prepare(qk, y, 1, 8, stream=s),
                                                         stream=s),
        "topk": lambda s: tq.tq_topk(qk, y, kenc, 5, stream=s),
        "attend": lambda s: tq.tq_attend(qv, logits, 1, 8, venc, rows, 0.1, stream=s),
        "prompt": lambda s: tq.tq_attend_prompt(qv, yq[100], kv, vv, start[100], 0.1, stream=s),
        "paged, one token": lambda s: tq.tq_attend_paged(qk, qv, yq[1], start[1], kc, vc, table, lens, 1, 0.1, stream=s),
        "paged, many tokens": lambda s: tq.tq_attend_paged(qk, qv, yq[100], start[100], kc, vc, table, lens, 100, 0.1,
                                                           stream=s),
        "rerank": lambda s: tq.tq_rerank(y, x, cand, 3, stream=s),
        "outlier channels": lambda s: tq.tq_outlier_channels(x, 1, rows, 32, stream=s),
    }
    return {name: (lambda s, f=f: flat(f(s))) for name, f in out.items()}


SIZES = [1 << k for k in range(9, 24)]


def test_memory_of_a_call_on_another_stream(tq):  # noqa: F811
    side = torch.cuda.Stream()
    for name, call in calls(tq).items():
        ref = [t.clone() for t in call(None)]
        torch.cuda.synchronize()
        # what the current stream has let go of but still reads (the copies are made behind a pause)
        old = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
        torch.cuda._sleep(20_000_000)
        copies = [t.clone() for t in old]
        del old
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(bool((c == 7).all()) for c in copies), name
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), name
        del got, copies
        # what the call has let go of while its kernels have yet to run
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = call(side)
        new = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
        torch.cuda.synchronize()
        assert all(bool((c == 9).all()) for c in new), name
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), name
        del got, new
        # a result dropped while the call runs
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        call(side)
        new = [torch.full((n,), 9, dtype=torch.uint8, device="cuda") for n in SIZES for _ in range(3)]
        torch.cuda.synchronize()
        assert all(bool((c == 9).all()) for c in new), name


def test_a_result_is_reused_behind_the_current_stream(tq):  # noqa: F811
    """A result of a call on another stream that the current one reads and lets go
    of is not given to the other stream's next call before it has been read."""
    side = torch.cuda.Stream()
    for name, call in calls(tq).items():
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
        ref = [t.clone() for t in got]
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)
        copies = [t.clone() for t in got]
        shapes = [(t.shape, t.dtype) for t in got]
        del got
        with torch.cuda.stream(side):
            new = [torch.zeros(s, dtype=d, device="cuda") for s, d in shapes]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(copies, ref)), name
        del new


def test_allocation_in_a_captured_call(tq):  # noqa: F811
    """A call on a forked stream of a captured graph that allocates its scratch."""
    some = calls(tq)
    for name in ("paged, many tokens", "prompt", "attend"):
        ref = some[name](None)[0]
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            side.wait_stream(torch.cuda.current_stream())
            got = some[name](side)[0]
            torch.cuda.current_stream().wait_stream(side)
            got = got + 0
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, ref), name
        assert math.isfinite(float(got.float().sum()))
