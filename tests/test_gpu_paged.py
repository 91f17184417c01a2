"""A quantized KV cache in pages on the GPU: storing rows by slot, and
attention of new tokens over the pages, against plain fp64 (see
paged_reference: the bounds follow from the roundings, not from runs)."""
import math

import numpy as np
import pytest
import torch

import workloads as wl
from oracle import tq_oracle as o
from tests.paged_reference import attend, unpack

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def tq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from online_vector_quantization_tq_b200 import build
    build.build()
    import online_vector_quantization_tq_b200 as pkg
    pkg.lib()
    return pkg


_MADE = {}


def quantizer(tq, d, b, ip, seed=0):
    key = (d, b, ip, seed)
    if key not in _MADE:
        _MADE[key] = (tq.tq_codebook(d, b, seed=seed) if ip else tq.tq_codebook_mse(d, b, seed=seed),
                      o.Tables(d, b, seed=seed) if ip else o.Tables(d, b, seed=seed, mode="mse"))
    return _MADE[key]


def random_rows(q, n, rng, scale=1.0):
    """Packed rows with codes drawn at random (any byte is a valid code) and norms over 2.6 decades."""
    norms = np.stack([rng.uniform(0.05, 20.0, n) * scale, rng.uniform(0.1, 0.6, n)], 1).astype(np.float32)
    return (rng.integers(0, 256, (n, q.code_bytes), dtype=np.uint8),
            rng.integers(0, 256, (n, q.sign_bytes), dtype=np.uint8), norms)


class Batch:
    """A cache in shuffled pages with NaN norms wherever no token is, and the
    sequences' rows in order on the host."""

    def __init__(self, tq, qk, qv, kv_heads, page, kv_lens, rng, spare_pages=3, key_scale=1.0):
        self.page, self.kv_heads, self.kv_lens = page, kv_heads, kv_lens
        need = [-(-n // page) for n in kv_lens]
        npages = sum(need) + spare_pages
        self.width = max(need) + 2
        order = rng.permutation(npages)
        table = np.full((len(kv_lens), self.width), -1, dtype=np.int32)
        table[:, -1] = 1 << 30  # never read
        self.rows, self.caches = [], []
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = order[at:at + n]
            at += n
        self.table = table
        for q, scale in ((qk, key_scale), (qv, 1.0)):
            parts = [rng.integers(0, 256, (npages, kv_heads, page, w), dtype=np.uint8)
                     for w in (q.code_bytes, q.sign_bytes)]
            parts.append(np.full((npages, kv_heads, page, 2), np.nan, dtype=np.float32))
            rows = []
            for i, n in enumerate(kv_lens):
                rows.append([])
                for h in range(kv_heads):
                    new = random_rows(q, n, rng, scale)
                    for j in range(n):
                        for p, x in zip(parts, new):
                            p[table[i, j // page], h, j % page] = x[j]
                    rows[-1].append(new)
            self.rows.append(rows)
            self.caches.append(tq.PagedCache(*(torch.from_numpy(p).cuda() for p in parts)))
        self.table_dev = torch.from_numpy(table).cuda()


def check(out, batch, y, q_start, news, kv_lens, heads, tk, tv, scale, dtype, many=False):
    """Compares every row of every sequence; returns the worst share of the bound."""
    group, d, worst = heads // batch.kv_heads, tk.d, 0.0
    for i, (n, kv) in enumerate(zip(news, kv_lens)):
        if n == 0:
            continue
        rows = slice(q_start[i], q_start[i] + n)
        for h in range(batch.kv_heads):
            cols = slice(h * group * d, (h + 1) * group * d)
            limits = np.repeat(np.clip(kv - n + 1 + np.arange(n), 0, len(batch.rows[0][i][h][2])), group)
            ref, bound = attend(y[rows, cols].reshape(n * group, d), limits, scale, unpack(batch.rows[0][i][h], tk),
                                tk, unpack(batch.rows[1][i][h], tv), tv, dtype, many)
            got = out[rows, cols].reshape(n * group, d)
            assert np.all(np.isfinite(got)), f"sequence {i}, head {h}"
            ratio = np.abs(got - ref) / bound.clip(1e-30)
            assert ratio.max(initial=0.0) <= 1.0, f"sequence {i}, head {h}: {ratio.max():.2f} of the bound"
            assert np.all(got[limits <= 0] == 0.0)
            worst = max(worst, float(ratio.max(initial=0.0)))
    return worst


def run_case(tq, d, kb, ip, vb, kv_heads, group, page, seqs, dtype, seed, gap=2, q_scale=1.0, many=False, scale=None):
    """seqs: (new tokens, keys) of each sequence.  `gap` tokens that belong to
    no sequence stand before the first and behind the last."""
    rng = np.random.default_rng(seed)
    (qk, tk), (qv, tv) = quantizer(tq, d, kb, ip), quantizer(tq, d, vb, False, seed=1)
    news, kv_lens = [s[0] for s in seqs], [s[1] for s in seqs]
    batch = Batch(tq, qk, qv, kv_heads, page, kv_lens, rng)
    heads = kv_heads * group
    starts = [gap + sum(news[:i]) for i in range(len(news) + 1)]
    total = starts[-1] + gap
    wide = torch.from_numpy(rng.standard_normal((total, heads * d + 24)).astype(np.float32) * q_scale)
    y = wide.to(DT[dtype]).cuda()[:, 8: 8 + heads * d]  # a view with a leading dimension of its own
    out = torch.full((total, heads * d + 8), -7.0, dtype=DT[dtype], device="cuda")
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    view = out[:, : heads * d]
    got = tq.tq_attend_paged(qk, qv, y, torch.tensor(starts, dtype=torch.int32, device="cuda"), *batch.caches,
                             batch.table_dev, torch.tensor(kv_lens, dtype=torch.int32, device="cuda"),
                             max(max(news), 1), scale, out=view)
    assert got.data_ptr() == out.data_ptr()
    res = out.float().cpu().numpy().astype(np.float64)
    assert np.all(res[:, heads * d:] == -7.0) and np.all(res[:gap] == -7.0) and np.all(res[starts[-1]:] == -7.0)
    return check(res, batch, y.float().cpu().numpy().astype(np.float64), starts, news, kv_lens, heads, tk, tv, scale,
                 dtype, many)


SMALL = [(1, 1), (1, 17), (1, 0), (0, 40), (1, 300), (1, 63), (1, 64), (1, 65)]


@pytest.mark.parametrize("d,kb,ip,vb", [(128, 4, False, 4), (128, 4, True, 3), (128, 2, True, 2), (128, 5, True, 4),
                                        (128, 3, False, 2), (128, 1, False, 3), (64, 4, False, 4), (64, 3, True, 3),
                                        (64, 2, False, 2), (64, 1, False, 4), (64, 5, True, 2)])
def test_single_tokens_every_width(tq, d, kb, ip, vb):
    """One new token per sequence: lengths of none, one, about a page and a
    tile, with every code width of keys and values."""
    worst = run_case(tq, d, kb, ip, vb, 2, 4, 16, SMALL, "bf16", seed=kb * 100 + vb + d)
    print(f"d={d} kb={kb} ip={ip} vb={vb}: worst {worst:.3f} of the bound")


@pytest.mark.parametrize("group,kv_heads,page,dtype", [(1, 3, 16, "bf16"), (3, 2, 48, "f16"), (7, 1, 32, "f16"),
                                                       (16, 2, 64, "bf16"), (20, 1, 128, "bf16")])
def test_groups_and_pages(tq, group, kv_heads, page, dtype):
    """Head layouts of 1 to 20 query heads per KV head, page sizes that do and
    do not divide a tile, several new tokens per sequence, tokens that see no
    key (more new tokens than keys)."""
    seqs = [(1, 700), (5, 5), (9, 4), (3, 129), (0, 0), (17, 333)]
    run_case(tq, 128, 4, False, 4, kv_heads, group, page, seqs, dtype, seed=group)
    run_case(tq, 64, 4, True, 3, kv_heads, group, page, seqs, dtype, seed=group + 50)


@pytest.mark.parametrize("ip", [False, True])
def test_long_context_is_split_and_joined(tq, ip):
    """A context long enough to be split over many blocks, with a batch of
    ragged lengths, sharp queries (one key has nearly all the weight) among
    them."""
    run_case(tq, 128, 4, ip, 4, 1, 4, 64, [(1, 9000), (2, 257), (1, 3001)], "bf16", seed=3)
    run_case(tq, 64, 3, ip, 3, 1, 8, 16, [(1, 5000)], "f16", seed=4, q_scale=8.0)


def test_chunk_of_a_prompt(tq):
    """Many new tokens at once: 70 and 33 new tokens of sequences with and
    without a prefix."""
    run_case(tq, 128, 4, False, 4, 2, 4, 32, [(70, 200), (33, 33), (1, 90)], "bf16", seed=5)
    run_case(tq, 64, 4, True, 2, 1, 5, 16, [(70, 200), (33, 33)], "f16", seed=6)


def test_value_norms_of_any_size(tq):
    """Value and key norms far outside fp16's range."""
    rng = np.random.default_rng(8)
    (qk, tk), (qv, tv) = quantizer(tq, 128, 4, False), quantizer(tq, 128, 4, False, seed=1)
    for vs, ks in ((1e-6, 1.0), (1e7, 1e-3), (1e20, 1.0)):
        batch = Batch(tq, qk, qv, 1, 16, [100], rng, key_scale=ks)
        c = batch.caches[1]
        c.norms.mul_(vs)
        for part in batch.rows[1][0]:
            part[2][:] = part[2] * np.float32(vs)
        y = torch.randn(1, 256, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
        out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), *batch.caches,
                                 batch.table_dev, torch.tensor([100], dtype=torch.int32, device="cuda"), 1, 0.1)
        check(out.double().cpu().numpy(), batch, y.double().cpu().numpy(), [0, 1], [1], [100], 2, tk, tv, 0.1, "bf16")


def test_bad_pages_hold_no_keys(tq):
    """A table entry outside the cache is skipped: the result is that of the
    other pages' keys alone.  Fewer table columns than kv_len needs: the keys
    beyond are not attended."""
    rng = np.random.default_rng(9)
    (qk, tk), (qv, tv) = quantizer(tq, 128, 4, True), quantizer(tq, 128, 4, False, seed=1)
    batch = Batch(tq, qk, qv, 1, 16, [80], rng)
    y = torch.randn(1, 512, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([80], dtype=torch.int32, device="cuda")
    for bad in (-1, batch.caches[0].codes.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = batch.table_dev.clone()
        table[0, 2] = bad
        out = tq.tq_attend_paged(qk, qv, y, start, *batch.caches, table, lens, 1, 0.1).double().cpu().numpy()
        keep = np.r_[0:32, 48:80]
        rows = [[tuple(p[keep] for p in batch.rows[s][0][0])] for s in (0, 1)]
        ref, bound = attend(y.double().cpu().numpy().reshape(4, 128), [64] * 4, 0.1, unpack(rows[0][0], tk), tk,
                            unpack(rows[1][0], tv), tv, "bf16")
        assert np.all(np.abs(out.reshape(4, 128) - ref) <= bound)
    out = tq.tq_attend_paged(qk, qv, y, start, *batch.caches, batch.table_dev[:, :3], lens, 1, 0.1)
    rows = [tuple(p[:48] for p in batch.rows[s][0][0]) for s in (0, 1)]
    ref, bound = attend(y.double().cpu().numpy().reshape(4, 128), [48] * 4, 0.1, unpack(rows[0], tk), tk,
                        unpack(rows[1], tv), tv, "bf16")
    assert np.all(np.abs(out.double().cpu().numpy().reshape(4, 128) - ref) <= bound)


def test_replayed_graph_reads_new_lengths(tq):
    """Captured once, replayed after lengths, tables and queries changed in
    place: the same as fresh calls, bit for bit; a second graph with a
    workspace of its own interleaved; and the result of another stream."""
    rng = np.random.default_rng(10)
    (qk, _), (qv, _) = quantizer(tq, 128, 4, False), quantizer(tq, 128, 4, False, seed=1)
    batch = Batch(tq, qk, qv, 2, 16, [900, 400], rng)
    y = torch.randn(2, 2 * 4 * 128, device="cuda").bfloat16()
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([900, 400], dtype=torch.int32, device="cuda")
    table = batch.table_dev.clone()

    def call(out=None, ws=None):
        return tq.tq_attend_paged(qk, qv, y, start, *batch.caches, table, lens, 1, 0.09, out=out, workspace=ws)

    ws = [tq.attend_paged_workspace(qk, qv, 2, 2, 8, 2, 1, table.shape[1], 16) for _ in range(2)]
    outs, graphs = [torch.zeros_like(y) for _ in range(2)], []
    call()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(outs[i], ws[i])
        graphs.append(g)
    for a, b in ((900, 400), (16, 399), (0, 1), (555, 2)):
        lens.copy_(torch.tensor([a, b], dtype=torch.int32))
        y.normal_()
        for g in graphs:
            g.replay()
        ref = call()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], ref) and torch.equal(outs[1], ref)
        assert bool((ref[0] == 0).all()) == (a == 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = tq.tq_attend_paged(qk, qv, y, start, *batch.caches, table, lens, 1, 0.09, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, call())


@pytest.mark.parametrize("d,kb,ip,vb,kv_heads,page,tokens", [(128, 4, True, 4, 8, 16, 33), (64, 3, False, 3, 3, 48, 1),
                                                             (128, 2, True, 2, 1, 64, 1000), (96, 4, True, 4, 2, 16, 7)])
def test_store_moves_rows_and_nothing_else(tq, d, kb, ip, vb, kv_heads, page, tokens):
    """Every stored row equals the encoded one; rows without a slot (negative,
    or behind the cache) and all other slots leave the pages as they were."""
    rng = np.random.default_rng(tokens)
    qk = quantizer(tq, d, kb, ip)[0]
    qv = quantizer(tq, d, vb, d == 96, seed=1)[0]  # any quantizer: values with sign bits at d = 96
    npages = -(-tokens // page) + 2
    slots = rng.permutation(npages * page)[:tokens].astype(np.int64)
    slots[::5] = rng.choice([-1, -2 ** 62, npages * page, 2 ** 62], len(slots[::5]))
    encs, caches, befores = [], [], []
    for q in (qk, qv):
        encs.append(tq.Encoded(*(torch.from_numpy(p).cuda() for p in random_rows(q, tokens * kv_heads, rng))))
        c = q.empty_paged(npages, kv_heads, page)
        for t in (c.codes, c.signs):
            t.random_(0, 256)
        c.norms.normal_()
        caches.append(c)
        befores.append([t.clone() for t in (c.codes, c.signs, c.norms)])
    tq.tq_paged_store(qk, qv, *encs, torch.from_numpy(slots).cuda(), *caches)
    for e, c, before in zip(encs, caches, befores):
        for src, dst, ref in zip((e.codes, e.signs, e.norms), (c.codes, c.signs, c.norms), before):
            for t in range(tokens):
                if 0 <= slots[t] < npages * page:
                    ref[slots[t] // page, :, slots[t] % page] = src[t * kv_heads:(t + 1) * kv_heads]
            assert torch.equal(dst, ref)


def test_prompt_encoded_stored_and_decoded(tq):
    """Keys and values of tokens encoded by tq_encode, stored into pages, and
    attended by one new token per sequence: as tq_score and tq_attend over the
    same rows kept contiguously (whose own error is at most 2^-10 of the same
    sum, as its test states), within the two bounds together."""
    d, hk, group, page, n = 128, 2, 4, 16, 203
    rng = np.random.default_rng(12)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, True), quantizer(tq, d, 4, False, seed=1)
    x = [torch.from_numpy(rng.standard_normal((n * hk, d)).astype(np.float32)).bfloat16().cuda() for _ in range(2)]
    kenc, venc = tq.tq_encode(qk, x[0]), tq.tq_encode(qv, x[1])
    npages = 20
    kc, vc = qk.empty_paged(npages, hk, page), qv.empty_paged(npages, hk, page)
    kc.norms.fill_(float("nan"))
    vc.norms.fill_(float("nan"))
    pages = rng.permutation(npages)[: -(-n // page)]
    slots = torch.from_numpy(np.array([pages[t // page] * page + t % page for t in range(n)], dtype=np.int64)).cuda()
    cut = 150  # in two pieces, as a prompt and what follows
    for a, b in ((0, cut), (cut, n)):
        part = [tq.Encoded(e.codes[a * hk:b * hk], e.signs[a * hk:b * hk], e.norms[a * hk:b * hk])
                for e in (kenc, venc)]
        tq.tq_paged_store(qk, qv, *part, slots[a:b], kc, vc)
    y = torch.from_numpy(rng.standard_normal((1, hk * group * d)).astype(np.float32)).bfloat16().cuda()
    table = torch.from_numpy(pages.astype(np.int32)[None]).cuda()
    got = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), kc, vc, table,
                             torch.tensor([n], dtype=torch.int32, device="cuda"), 1, 1 / math.sqrt(d))
    by_head = [[t.view(n, hk, -1).transpose(0, 1).contiguous().view(n * hk, -1) for t in (e.codes, e.signs, e.norms)]
               for e in (kenc, venc)]
    kh, vh = (tq.Encoded(*p) for p in by_head)
    logits = tq.tq_score(qk, y.view(hk * group, d).float(), hk, group, kh, n)
    ref = tq.tq_attend(qv, logits, hk, group, vh, n, 1 / math.sqrt(d)).double().cpu().numpy()
    for h in range(hk):
        ke, ve = (unpack([p[h * n:(h + 1) * n].cpu().numpy() for p in parts], t)
                  for parts, t in zip(by_head, (tk, tv)))
        yy = y.double().cpu().numpy().reshape(hk * group, d)[h * group:(h + 1) * group]
        _, bound = attend(yy, [n] * group, 1 / math.sqrt(d), ke, tk, ve, tv, "bf16")
        err = np.abs(got.double().cpu().numpy().reshape(hk * group, d)[h * group:(h + 1) * group] -
                     ref[h * group:(h + 1) * group])
        assert np.all(err <= bound + 2.0 ** -10 * ve["norm"].max() + 1e-6)


def test_argument_checks(tq):
    """Refused before any launch, with the output left as it was."""
    (qk, _), (qv, _) = quantizer(tq, 128, 4, True), quantizer(tq, 128, 4, False, seed=1)
    kc, vc = qk.empty_paged(4, 2, 16), qv.empty_paged(4, 2, 16)
    y = torch.zeros(1, 1024, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([5], dtype=torch.int32, device="cuda")
    table = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
    out = torch.full_like(y, 3.0)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(tq.TQError):
        tq.tq_attend_paged(qk, qv, y, start, kc, vc, table, lens, 1, float("inf"), out=out)
    with pytest.raises(tq.TQError):
        tq.tq_attend_paged(qk, qv, y, start, kc, vc, table, lens, 1, 0.1, out=out, workspace=small)
    with pytest.raises(tq.TQError):  # values must be TurboQuant-MSE
        tq.tq_attend_paged(qk, qk, y, start, kc, kc, table, lens, 1, 0.1, out=out)
    with pytest.raises(TypeError):
        tq.tq_attend_paged(qk, qv, y.float(), start, kc, vc, table, lens, 1, 0.1, out=out.float())
    with pytest.raises(ValueError):
        tq.tq_attend_paged(qk, qv, y[:, :1000], start, kc, vc, table, lens, 1, 0.1)
    with pytest.raises(ValueError):
        tq.tq_attend_paged(qk, qv, y, start.cpu(), kc, vc, table, lens, 1, 0.1, out=out)
    with pytest.raises(ValueError):
        tq.tq_attend_paged(qk, qv, y, start[:1], kc, vc, table, lens, 1, 0.1, out=out)
    assert bool((out == 3.0).all())
    none = torch.empty(0, 1024, dtype=torch.bfloat16, device="cuda")
    assert tq.tq_attend_paged(qk, qv, none, torch.zeros(1, dtype=torch.int32, device="cuda"), kc, vc, table[:0],
                              lens[:0], 1, 0.1).shape == (0, 1024)


@pytest.mark.parametrize("d,kb,ip,vb", [(128, 4, False, 4), (128, 3, True, 3), (128, 2, True, 4), (128, 1, False, 2),
                                        (64, 4, True, 4), (64, 3, False, 3), (64, 1, False, 2), (64, 2, True, 2)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_block_height(tq, d, kb, ip, vb, dtype):
    """Calls of up to 8, 16, 24 and 32 rows a sequence and KV head, in both
    types (fp16 queries keep their low terms)."""
    for n, group in ((1, 7), (2, 8), (5, 4), (3, 8), (4, 8)):
        run_case(tq, d, kb, ip, vb, 2, group, 16, [(n, 333), (n, n), (1, 70), (0, 5), (n, n + 64)], dtype,
                 seed=d + 7 * n + group, q_scale=3.0)


def test_fp16_results_are_as_good_as_their_type(tq):
    """With sharp heads, where the rounding of the rotated queries to fp16 would
    show: the error against fp64 stays below 2^-11 of the result (its own
    rounding among it), 2-norm over 2-norm."""
    d, n, heads = 128, 2000, 16
    rng = np.random.default_rng(31)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, False), quantizer(tq, d, 4, False, seed=1)
    batch = Batch(tq, qk, qv, 1, 16, [n], rng)
    y = torch.from_numpy(rng.standard_normal((1, heads * d)).astype(np.float32)).half().cuda()
    out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, 1], dtype=torch.int32, device="cuda"), *batch.caches,
                             batch.table_dev, torch.tensor([n], dtype=torch.int32, device="cuda"), 1, 1 / math.sqrt(d))
    ref, _ = attend(y.double().cpu().numpy().reshape(heads, d), [n] * heads, 1 / math.sqrt(d),
                    unpack(batch.rows[0][0][0], tk), tk, unpack(batch.rows[1][0][0], tv), tv, "f16")
    got = out.double().cpu().numpy().reshape(heads, d)
    assert np.linalg.norm(got - ref) <= 2.0 ** -11 * np.linalg.norm(ref)


@pytest.mark.parametrize("kv_heads,shift", [(1, 1), (5, 2), (40, 0), (40, 3)])
def test_store_of_any_alignment(tq, kv_heads, shift):
    """Rows that start at any 4-byte boundary (norms: 8), and more heads than
    one pass of a warp takes."""
    d, page, tokens = 128, 16, 37
    rng = np.random.default_rng(kv_heads + shift)
    qk, qv = quantizer(tq, d, 4, True)[0], quantizer(tq, d, 4, False, seed=1)[0]
    slots = torch.from_numpy(rng.permutation(5 * page)[:tokens].astype(np.int64)).cuda()
    encs, caches = [], []
    for q in (qk, qv):
        parts = []
        for p, step in zip(random_rows(q, tokens * kv_heads, rng), (4, 4, 2)):
            flat = torch.zeros(p.size + 64, dtype=torch.from_numpy(p).dtype, device="cuda")
            at = flat[step * shift: step * shift + p.size]
            at.copy_(torch.from_numpy(p).view(-1))
            parts.append(at.view(p.shape))
        encs.append(tq.Encoded(*parts))
        caches.append(q.empty_paged(5, kv_heads, page))
    tq.tq_paged_store(qk, qv, *encs, slots, *caches)
    for e, c in zip(encs, caches):
        for src, dst in ((e.codes, c.codes), (e.signs, c.signs), (e.norms, c.norms)):
            got = dst[slots // page, :, slots % page].reshape(src.shape)
            assert torch.equal(got, src)


def test_arrays_of_the_wrong_shape_are_refused(tq):
    """Encoded rows that are narrower than the quantizer's, or of another type."""
    qk, qv = quantizer(tq, 128, 4, True)[0], quantizer(tq, 128, 4, False, seed=1)[0]
    kc, vc = qk.empty_paged(2, 1, 16), qv.empty_paged(2, 1, 16)
    ke, ve = qk.empty_encoded(3), qv.empty_encoded(3)
    slots = torch.arange(3, device="cuda")
    tq.tq_paged_store(qk, qv, ke, ve, slots, kc, vc)
    E = tq.Encoded
    for bad in (E(ke.codes, ke.signs[:, :8].contiguous(), ke.norms), E(ke.codes, ke.signs, ke.norms[:, :1].contiguous()),
                E(ke.codes.view(torch.int8), ke.signs, ke.norms), E(ke.codes, ke.signs, ke.norms.half()),
                E(ke.codes[:2], ke.signs, ke.norms)):
        with pytest.raises(ValueError):
            tq.tq_paged_store(qk, qv, bad, ve, slots, kc, vc)
    with pytest.raises(ValueError):
        tq.tq_paged_store(qk, qv, ke, ve, slots.cpu(), kc, vc)


@pytest.mark.parametrize("d,group,most", [(64, 4, 5), (64, 8, 2), (128, 4, 4), (64, 4, 2), (128, 16, 4)])
def test_large_batches_of_unequal_sequences(tq, d, group, most):
    """Enough rows for the join by blocks of rows, where many sequences have
    fewer rows than a block has."""
    seqs = [(most if i % 5 == 0 else i % 2, 20 + 7 * (i % 9)) for i in range(230)]
    run_case(tq, d, 4, False, 4, 4, group, 16, seqs, "bf16", seed=d + group + most)
