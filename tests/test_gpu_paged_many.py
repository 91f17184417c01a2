"""Attention of many new tokens over a paged quantized cache (sequences of more
than 64 query rows per KV head take a kernel of their own), against plain fp64
with bounds from the roundings."""
import math

import numpy as np
import pytest
import torch

from tests.paged_reference import attend, unpack
from tests.test_gpu_paged import Batch, check, quantizer, run_case, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,kb,ip,vb", [(128, 4, False, 4), (128, 4, True, 3), (128, 2, True, 2), (128, 5, True, 4),
                                        (128, 3, False, 2), (128, 2, False, 4), (128, 1, False, 3), (64, 4, False, 4),
                                        (64, 3, True, 3), (64, 2, True, 4), (64, 5, True, 2), (64, 1, False, 2)])
def test_every_width(tq, d, kb, ip, vb):  # noqa: F811
    """Chunks with and without a prefix, of one tile of rows and of several,
    tokens that see no key, and a sequence that decodes."""
    seqs = [(40, 40), (33, 300), (1, 200), (90, 1000), (60, 40), (0, 77), (17, 129)]
    worst = run_case(tq, d, kb, ip, vb, 1, 4, 16, seqs, "bf16", seed=kb * 10 + vb + d, many=True)
    print(f"d={d} kb={kb} ip={ip} vb={vb}: worst {worst:.3f} of the bound")


@pytest.mark.parametrize("ip", [False, True])
@pytest.mark.parametrize("group,kv_heads,page,dtype", [(1, 3, 16, "f16"), (3, 2, 48, "bf16"), (7, 1, 64, "bf16"),
                                                       (16, 1, 128, "f16"), (33, 1, 32, "bf16")])
def test_head_layouts(tq, group, kv_heads, page, dtype, ip):  # noqa: F811
    """Blocks of rows that end inside a token's group, pages that do and do not
    divide a tile of 128 keys."""
    n = max(2, 150 // group)
    seqs = [(n, 700), (2 * n + 1, 2 * n + 1), (n, n + 127), (n, n + 128), (n, n + 129)]
    for d in (64, 128):
        run_case(tq, d, 4, ip, 4, kv_heads, group, page, seqs, dtype, seed=group + d, many=True)


@pytest.mark.parametrize("d,ip", [(128, False), (128, True), (64, False), (64, True)])
def test_many_short_and_long_runs(tq, d, ip):  # noqa: F811
    """More blocks of rows than the machine has SMs, and few with a long
    context: blocks that one run has whole, that two share, that many share."""
    run_case(tq, d, 4, ip, 3, 2, 4, 16, [(9 + i % 5, 30 + 41 * (i % 13)) for i in range(90)], "bf16", seed=21, many=True)
    run_case(tq, d, 3, ip, 4, 1, 4, 64, [(70, 9000), (12, 3000)], "bf16", seed=22, many=True)
    run_case(tq, d, 4, ip, 4, 1, 2, 16, [(300, 900)], "f16", seed=23, q_scale=6.0, many=True)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_scales(tq, scale):  # noqa: F811
    for ip in (False, True):
        run_case(tq, 128, 4, ip, 4, 1, 4, 16, [(50, 333), (3, 9)], "bf16", seed=24, many=True, scale=scale)


def test_value_norms_of_any_size(tq):  # noqa: F811
    rng = np.random.default_rng(8)
    (qk, tk), (qv, tv) = quantizer(tq, 128, 4, False), quantizer(tq, 128, 4, False, seed=1)
    n = 40
    for vs, ks in ((1e-6, 1.0), (1e7, 1e-3), (1e20, 1.0)):
        batch = Batch(tq, qk, qv, 1, 16, [300], rng, key_scale=ks)
        ramp = np.where(np.arange(300) < 150, np.float32(vs * 1e-4), np.float32(vs))  # small norms first
        c = batch.caches[1]
        for part in batch.rows[1][0]:
            part[2][:, 0] = part[2][:, 0] * ramp
            for j in range(300):
                c.norms[batch.table[0, j // 16], 0, j % 16, 0] = float(part[2][j, 0])
        y = torch.randn(n, 256, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
        out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                                 batch.table_dev, torch.tensor([300], dtype=torch.int32, device="cuda"), n, 0.1)
        check(out.double().cpu().numpy(), batch, y.double().cpu().numpy(), [0, n], [n], [300], 2, tk, tv, 0.1, "bf16",
              many=True)


def test_bad_pages_hold_no_keys(tq):  # noqa: F811
    rng = np.random.default_rng(9)
    (qk, tk), (qv, tv) = quantizer(tq, 128, 4, True), quantizer(tq, 128, 4, False, seed=1)
    n, kv = 20, 300
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    y = torch.randn(n, 512, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
    for bad in (-1, batch.caches[0].codes.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = batch.table_dev.clone()
        table[0, 0] = bad
        table[0, 3:5] = bad
        out = tq.tq_attend_paged(qk, qv, y, start, *batch.caches, table, lens, n, 0.1).double().cpu().numpy()
        keep = np.r_[16:48, 80:kv]
        rows = [tuple(p[keep] for p in batch.rows[s][0][0]) for s in (0, 1)]
        limits = np.repeat([int((keep < kv - n + 1 + t).sum()) for t in range(n)], 4)
        ref, bound = attend(y.double().cpu().numpy().reshape(4 * n, 128), limits, 0.1, unpack(rows[0], tk), tk,
                            unpack(rows[1], tv), tv, "bf16", True)
        assert np.all(np.abs(out.reshape(4 * n, 128) - ref) <= bound)
    # every page bad: no keys, zeros
    table = torch.full_like(batch.table_dev, -1)
    out = tq.tq_attend_paged(qk, qv, y, start, *batch.caches, table, lens, n, 0.1)
    assert bool((out == 0).all())
    tq.tq_sync_check(qk)


def test_replayed_graph_reads_new_lengths(tq):  # noqa: F811
    """Captured once, replayed after lengths and queries changed in place: as a
    fresh call, bit for bit, also on another stream and behind a second graph
    with a workspace of its own."""
    rng = np.random.default_rng(10)
    (qk, _), (qv, _) = quantizer(tq, 128, 4, True), quantizer(tq, 128, 4, False, seed=1)
    batch = Batch(tq, qk, qv, 2, 16, [900, 400], rng)
    total = 70
    y = torch.randn(total, 2 * 4 * 128, device="cuda").bfloat16()
    start = torch.tensor([0, 40, 70], dtype=torch.int32, device="cuda")
    lens = torch.tensor([900, 400], dtype=torch.int32, device="cuda")
    table = batch.table_dev

    def call(out=None, ws=None, stream=None):
        return tq.tq_attend_paged(qk, qv, y, start, *batch.caches, table, lens, total, 0.09,
                                  out=torch.zeros_like(y) if out is None else out, workspace=ws, stream=stream)

    ws = [tq.attend_paged_workspace(qk, qv, total, 2, 8, 2, total, table.shape[1], 16) for _ in range(2)]
    outs, graphs = [torch.zeros_like(y) for _ in range(2)], []
    call()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(outs[i], ws[i])
        graphs.append(g)
    for cut, end, a, b in ((40, 70, 900, 400), (1, 70, 50, 399), (69, 70, 69, 1), (5, 60, 0, 300), (0, 0, 9, 9)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        start.copy_(torch.tensor([0, cut, end], dtype=torch.int32))
        y.normal_()
        for o in outs:
            o.zero_()
        for g in graphs:
            g.replay()
        ref = call()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
        assert bool((ref[end:] == 0).all())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, call())
    tq.tq_sync_check(qk)


def test_a_prompt_in_chunks(tq):  # noqa: F811
    """A prompt's keys and values encoded, stored and attended chunk by chunk,
    against the same tokens attended at once: each within its bound of the exact
    result."""
    d, hk, group, page, n = 128, 2, 4, 16, 150
    rng = np.random.default_rng(12)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, True), quantizer(tq, d, 4, False, seed=1)
    x = [torch.from_numpy(rng.standard_normal((n * hk, d)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    y = torch.from_numpy(rng.standard_normal((n, hk * group * d)).astype(np.float32)).bfloat16().cuda()
    encs = [tq.tq_encode(qk, x[0]), tq.tq_encode(qv, x[1])]
    kc, vc = qk.empty_paged(12, hk, page), qv.empty_paged(12, hk, page)
    for c in (kc, vc):
        c.norms.fill_(float("nan"))
    pages = rng.permutation(12)[: -(-n // page)]
    slots = torch.from_numpy(np.array([pages[t // page] * page + t % page for t in range(n)], dtype=np.int64)).cuda()
    table = torch.from_numpy(pages.astype(np.int32)[None]).cuda()
    got = torch.empty_like(y)
    for a, b in ((0, 70), (70, 71), (71, 75), (75, n)):
        part = [tq.Encoded(e.codes[a * hk:b * hk], e.signs[a * hk:b * hk], e.norms[a * hk:b * hk]) for e in encs]
        tq.tq_paged_store(qk, qv, *part, slots[a:b], kc, vc)
        tq.tq_attend_paged(qk, qv, y[a:b], torch.tensor([0, b - a], dtype=torch.int32, device="cuda"), kc, vc, table,
                           torch.tensor([b], dtype=torch.int32, device="cuda"), b - a, 1 / math.sqrt(d), out=got[a:b])
    once = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), kc, vc, table,
                              torch.tensor([n], dtype=torch.int32, device="cuda"), n, 1 / math.sqrt(d))
    for h in range(hk):
        ke, ve = (unpack([p.view(n, hk, -1)[:, h].cpu().numpy() for p in (e.codes, e.signs, e.norms)], t)
                  for e, t in zip(encs, (tk, tv)))
        cols = slice(h * group * d, (h + 1) * group * d)
        ref, bound = attend(y[:, cols].double().cpu().numpy().reshape(n * group, d), np.repeat(np.arange(1, n + 1), group),
                            1 / math.sqrt(d), ke, tk, ve, tv, "bf16", True)
        for out in (got, once):
            assert np.all(np.abs(out[:, cols].double().cpu().numpy().reshape(n * group, d) - ref) <= bound)


@pytest.mark.parametrize("n,group", [(3, 4), (3, 5), (40, 4), (200, 2)])
@pytest.mark.parametrize("what", ["key", "value", "value inf"])
def test_what_a_token_does_not_see(tq, n, group, what):  # noqa: F811
    """A norm that is not finite, of a token's key or value, makes NaN of the
    tokens that see it; the tokens before it keep their results, bit for bit."""
    rng = np.random.default_rng(n)
    (qk, _), (qv, _) = quantizer(tq, 128, 4, n != 40), quantizer(tq, 128, 4, False, seed=1)
    kv = n + 150
    batch = Batch(tq, qk, qv, 1, 16, [kv, 60], rng)
    y = torch.randn(n + 1, group * 128, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    start = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([kv, 60], dtype=torch.int32, device="cuda")

    def call():
        return tq.tq_attend_paged(qk, qv, y, start, *batch.caches, batch.table_dev, lens, n, 0.1)
    clean = call()
    for t in (0, 1, n // 2, n - 1):
        at = kv - n + t
        norms = batch.caches[what != "key"].norms[batch.table[0, at // 16], 0, at % 16]
        keep = norms.clone()
        norms[0] = math.inf if what == "value inf" else math.nan
        out = call()
        norms.copy_(keep)
        assert torch.equal(out[:t], clean[:t]) and torch.equal(out[n:], clean[n:])
        assert bool(torch.isnan(out[t:n]).all())
    assert torch.equal(call(), clean)
