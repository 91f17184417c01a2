"""What a token sees of a paged quantized cache, and what reaches it of what it
does not see: batches padded in front, more new tokens than a call takes, norms
of very different sizes, norms that are not finite."""
import math

import numpy as np
import pytest
import torch

from oracle import tq_oracle as o
from tests.paged_reference import attend, unpack
from tests.test_gpu_paged import DT, Batch, check, quantizer, run_case, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,ip", [(64, False), (128, False), (64, True), (128, True)])
def test_fewer_keys_than_new_tokens(tq, d, ip):  # noqa: F811
    """256 new tokens, all in front of the first 128 or so without a key (a batch
    padded in front): whole blocks of rows whose first 128 see nothing, several
    to a run, and such blocks among others."""
    run_case(tq, d, 4, ip, 4, 8, 1, 16, [(256, 128)] * 64, "bf16", seed=d, many=True)
    seqs = [(256, (128, 1, 700, 129, 256, 127)[i % 6]) for i in range(12)] + [(300, 40), (65, 3), (320, 180)]
    run_case(tq, d, 4, ip, 3, 2, 1, 16, seqs, "bf16", seed=d + 1, many=True)
    run_case(tq, d, 3, ip, 4, 1, 4, 48, [(129, 20), (96, 96), (70, 64), (1, 5)], "f16", seed=d + 2, many=True)
    tq.tq_sync_check(quantizer(tq, d, 4, ip)[0])


@pytest.mark.parametrize("d,ip,dtype", [(64, True, "f16"), (128, False, "bf16")])
@pytest.mark.parametrize("max_new,group", [(1, 4), (5, 4), (40, 4), (150, 2)])
def test_more_new_tokens_than_max_new(tq, d, ip, dtype, max_new, group):  # noqa: F811
    """Of a sequence with more than max_new new tokens the first max_new are
    attended, each with the keys that it sees among all of them; the others'
    rows are left as they were."""
    rng = np.random.default_rng(max_new)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, ip), quantizer(tq, d, 4, False, seed=1)
    seqs = [(max_new + 9, 300), (2 * max_new + 300, 2 * max_new + 310), (max_new, 77), (max_new + 1, max_new), (0, 9)]
    news, kv_lens = [s[0] for s in seqs], [s[1] for s in seqs]
    batch = Batch(tq, qk, qv, 2, 16, kv_lens, rng)
    heads, total = 2 * group, sum(news)
    starts = [sum(news[:i]) for i in range(len(news) + 1)]
    y = torch.from_numpy(rng.standard_normal((total, heads * d)).astype(np.float32)).to(DT[dtype]).cuda()
    out = torch.full_like(y, -7.0)
    tq.tq_attend_paged(qk, qv, y, torch.tensor(starts, dtype=torch.int32, device="cuda"), *batch.caches, batch.table_dev,
                       torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), max_new, 1 / math.sqrt(d), out=out)
    tq.tq_sync_check(qk)
    res, yy = out.double().cpu().numpy(), y.double().cpu().numpy()
    for i, (n, kv) in enumerate(seqs):
        m = min(n, max_new)
        rows = slice(starts[i], starts[i] + m)
        assert np.all(res[starts[i] + m: starts[i + 1]] == -7.0)
        for h in range(2):
            cols = slice(h * group * d, (h + 1) * group * d)
            limits = np.repeat(np.clip(kv - n + 1 + np.arange(m), 0, kv), group)
            ref, bound = attend(yy[rows, cols].reshape(m * group, d), limits, 1 / math.sqrt(d),
                                unpack(batch.rows[0][i][h], tk), tk, unpack(batch.rows[1][i][h], tv), tv, dtype,
                                m * group > 64)
            got = res[rows, cols].reshape(m * group, d)
            assert np.all(np.abs(got - ref) <= bound), f"sequence {i}, head {h}"
            assert np.all(got[limits <= 0] == 0.0)


@pytest.mark.parametrize("n,there,group,kv", [(7, 5, 4, 50), (170, 150, 1, 200)])
def test_sequences_that_end_behind_the_queries(tq, n, there, group, kv):  # noqa: F811
    """Fewer rows of queries than q_start counts: those that are there see what
    they would see beside the others."""
    d = 128
    rng = np.random.default_rng(n)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, False), quantizer(tq, d, 4, False, seed=1)
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    y = torch.from_numpy(rng.standard_normal((there, group * d)).astype(np.float32)).bfloat16().cuda()
    out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                             batch.table_dev, torch.tensor([kv], dtype=torch.int32, device="cuda"), n, 0.1)
    limits = np.repeat(kv - n + 1 + np.arange(there), group)
    ref, bound = attend(y.double().cpu().numpy().reshape(there * group, d), limits, 0.1, unpack(batch.rows[0][0][0], tk),
                        tk, unpack(batch.rows[1][0][0], tv), tv, "bf16", there * group > 64)
    assert np.all(np.abs(out.double().cpu().numpy().reshape(there * group, d) - ref) <= bound)


@pytest.mark.parametrize("n,group", [(3, 4), (3, 5), (40, 4), (200, 2)])  # few rows twice, many rows twice
@pytest.mark.parametrize("d,ip", [(128, True), (128, False), (64, True), (64, False)])
@pytest.mark.parametrize("what", [math.inf, -math.inf])
def test_infinite_norms(tq, d, ip, n, group, what):  # noqa: F811
    """An infinite norm of a key, of its residual or of a value makes NaN of the
    tokens that see it, whatever the signs of their products; the tokens before
    it, and the other sequence, keep their results, bit for bit."""
    rng = np.random.default_rng(n + d)
    (qk, _), (qv, _) = quantizer(tq, d, 4, ip), quantizer(tq, d, 4, False, seed=1)
    kv = n + 150
    batch = Batch(tq, qk, qv, 1, 16, [kv, 60], rng)
    y = torch.randn(n + 1, group * d, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    start = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([kv, 60], dtype=torch.int32, device="cuda")

    def call():
        return tq.tq_attend_paged(qk, qv, y, start, *batch.caches, batch.table_dev, lens, n, 0.1)
    clean = call()
    assert bool(torch.isfinite(clean).all())
    for side, which in ((0, 0), (1, 0)) + (((0, 1),) if ip else ()):
        for t in (0, 1, n - 1):
            at = kv - n + t
            norms = batch.caches[side].norms[batch.table[0, at // 16], 0, at % 16]
            keep = norms.clone()
            norms[which] = what
            out = call()
            norms.copy_(keep)
            assert torch.equal(out[:t], clean[:t]) and torch.equal(out[n:], clean[n:])
            assert bool(torch.isnan(out[t:n]).all())
    # residual norms of keys without sign bits, and second entries of values, are not looked at
    for cache in batch.caches[1:] if ip else batch.caches:
        cache.norms[..., 1] = what
    assert torch.equal(call(), clean)


def set_norms(batch, side, norms):
    """Norms of the first sequence's keys (side 0) or values (side 1), for every KV head."""
    cache, n = batch.caches[side], len(norms)
    for h in range(batch.kv_heads):
        batch.rows[side][0][h][2][:, 0] = norms
        for j in range(n):
            cache.norms[batch.table[0, j // batch.page], h, j % batch.page, 0] = float(norms[j])


def documented(got, y, limits, scale, ke, tk, ve, tv, own=2.0 ** -8):
    """Worst share of the precision that include/tq.h states, 2^-9 sum_k softmax_k
    ||v_k|| / sqrt(d) per coordinate beside the output's own rounding, as rows'
    2-norms: 2^-9 sum_k softmax_k ||v_k|| + own ||out||.  (Codes drawn at random
    have ||c|| of about 1.5.  One key with all the weight: its rounding is at most
    2^-11 of 1.5 ||v||.  Two with half each: a logit's error, of 2^-11 0.41 a factor
    and coordinate, has an rms of 1.2e-3 at scale ||k|| = 2, which moves the output
    by a quarter of that times 2.1 ||v||, 2^-10.6 ||v||; more keys, less.)"""
    ref, _ = attend(y, limits, scale, ke, tk, ve, tv, "bf16")
    yt, p = o.prepare_query(y, tk)
    see = np.arange(len(ke["norm"]))[None] < np.asarray(limits)[:, None]
    x = np.where(see, scale * o.score(yt, p, ke, tk), -np.inf)
    assert np.abs(np.where(see, x, 0.0)).max() < 30
    w = np.exp(x - x.max(1, keepdims=True))
    w /= w.sum(1, keepdims=True)
    bound = 2.0 ** -9 * (w @ ve["norm"])
    size = np.linalg.norm(ref, axis=1)
    return float((np.linalg.norm(got - ref, axis=1) / (bound + own * (size + bound))).max())


# (new tokens, query heads of a KV head): few rows, of each block height, and many
ROWS = [(4, 2), (4, 4), (5, 4), (16, 4), (40, 4), (100, 2), (200, 2)]


@pytest.mark.parametrize("n,group", ROWS)
@pytest.mark.parametrize("d,ip", [(128, False), (128, True), (64, False), (64, True)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_norms_that_a_token_does_not_see(tq, d, ip, dtype, n, group):  # noqa: F811
    """The last new token's key or value has a norm 2^16 to 2^60 times the others'
    (of 2.6 decades): the tokens before it keep the documented precision."""
    rng = np.random.default_rng(n)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, ip), quantizer(tq, d, 4, False, seed=1)
    kv = n + 150
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    rows = n * group
    y = torch.from_numpy(rng.standard_normal((n, group * d)).astype(np.float32)).to(DT[dtype]).cuda()
    yy = y.double().cpu().numpy().reshape(rows, d)
    limits = np.repeat(kv - n + 1 + np.arange(n), group)
    before = [batch.rows[s][0][0][2][:, 0].copy() for s in (0, 1)]
    seen = slice(0, rows - group)
    scale = 0.2 / math.sqrt(d)
    for side, up in ((1, 16), (1, 30), (1, 60), (0, 16), (0, 40)):
        for s in (0, 1):
            norms = before[s].copy()
            if s == side:
                norms[-1] = np.float32(10.0 * 2.0 ** up)
            set_norms(batch, s, norms)
        out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                                 batch.table_dev, torch.tensor([kv], dtype=torch.int32, device="cuda"), n, scale)
        got = out.double().cpu().numpy().reshape(rows, d)
        assert np.all(np.isfinite(got if dtype == "bf16" else got[seen]))  # (the last token's may leave fp16)
        ke, ve = unpack(batch.rows[0][0][0], tk), unpack(batch.rows[1][0][0], tv)
        some = {k: v[:-1] for k, v in ke.items()}, {k: v[:-1] for k, v in ve.items()}
        worst = documented(got[seen], yy[seen], limits[seen], scale, some[0], tk, some[1], tv,
                           2.0 ** (-8 if dtype == "bf16" else -11))
        assert worst <= 1.0, (side, up, worst)


@pytest.mark.parametrize("n,group", ROWS)
@pytest.mark.parametrize("d,ip", [(128, False), (64, True)])
def test_norms_of_very_different_sizes(tq, d, ip, n, group):  # noqa: F811
    """Value norms over 2^-60 to 2^60 and key norms over 2^-20 to 2^4, key by key,
    or a few large ones on keys of little weight: the documented precision."""
    rng = np.random.default_rng(n + 1)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, ip), quantizer(tq, d, 4, False, seed=1)
    kv, rows = n + 400, n * group
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    y = torch.from_numpy(rng.standard_normal((n, group * d)).astype(np.float32)).bfloat16().cuda()
    yy = y.double().cpu().numpy().reshape(rows, d)
    limits = np.repeat(kv - n + 1 + np.arange(n), group)
    scale = 1.0 / math.sqrt(d)
    one = rng.uniform(4.0, 16.0, kv)
    few = np.where(rng.random(kv) < 0.02, 2.0 ** 20, 1.0)  # where the logits turn out low, these weigh little
    for knorm, vnorm in ((one, 2.0 ** rng.uniform(-60, 60, kv)), (2.0 ** rng.uniform(-20, 4, kv), one),
                         (one * np.minimum(few, 2.0) ** 0.5, few), (one, np.where(np.arange(kv) < 200, 2.0 ** -50, 1.0)),
                         (one, np.where(np.arange(kv) < 200, 1.0, 2.0 ** -50)), (one, np.full(kv, 2.0 ** -90)),
                         (one, np.full(kv, 2.0 ** 90))):
        set_norms(batch, 0, knorm.astype(np.float32))
        set_norms(batch, 1, vnorm.astype(np.float32))
        out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                                 batch.table_dev, torch.tensor([kv], dtype=torch.int32, device="cuda"), n, scale)
        worst = documented(out.double().cpu().numpy().reshape(rows, d), yy, limits, scale,
                           unpack(batch.rows[0][0][0], tk), tk, unpack(batch.rows[1][0][0], tv), tv)
        assert worst <= 1.0, worst


@pytest.mark.parametrize("n,group", ROWS)
@pytest.mark.parametrize("d,ip,dtype", [(128, False, "bf16"), (128, True, "bf16"), (64, False, "f16"), (64, True, "f16")])
def test_large_logits(tq, d, ip, dtype, n, group):  # noqa: F811
    """Logits up to 2^60 (in fp16, whose queries end at 2^16, by the keys' norms):
    finite results, and a row whose highest logit stands out by more than the
    rounding of the operands (2^-10 of sum |y| |c|, which is below 2^-5 of the
    largest) has that key's value."""
    rng = np.random.default_rng(n + 2)
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, ip), quantizer(tq, d, 4, False, seed=1)
    kv, rows = n + 300, n * group
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    limits = np.repeat(kv - n + 1 + np.arange(n), group)
    keys = rng.uniform(8.0, 16.0, kv).astype(np.float32)
    for up in (12, 18, 24, 30, 60):
        big = 0 if dtype == "f16" else up
        set_norms(batch, 0, keys * np.float32(2.0 ** (up - big)))
        set_norms(batch, 1, rng.uniform(1.0, 64.0, kv).astype(np.float32))
        ke, ve = unpack(batch.rows[0][0][0], tk), unpack(batch.rows[1][0][0], tv)
        y = torch.from_numpy(rng.standard_normal((n, group * d)).astype(np.float32) * np.float32(2.0 ** big))
        y = y.to(DT[dtype]).cuda()
        out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                                 batch.table_dev, torch.tensor([kv], dtype=torch.int32, device="cuda"), n, 1.0)
        got = out.double().cpu().numpy().reshape(rows, d)
        assert np.all(np.isfinite(got)), up
        yt, p = o.prepare_query(y.double().cpu().numpy().reshape(rows, d), tk)
        x = np.where(np.arange(kv)[None] < limits[:, None], o.score(yt, p, ke, tk), -np.inf)
        order = np.sort(x, axis=1)
        most = np.abs(np.where(np.isfinite(x), x, 0.0)).max(1)
        clear = order[:, -1] - order[:, -2] > np.maximum(most * 2.0 ** -5, 40.0)
        assert clear.sum() >= rows / 20
        best = x.argmax(1)[clear]
        ref = (ve["norm"][best][:, None] * tv.centroids[ve["codes"][best]]) @ tv.R
        err = np.linalg.norm(got[clear] - ref, axis=1)
        assert np.all(err <= 2.0 ** -9 * ve["norm"][best] + 2.0 ** -8 * np.linalg.norm(ref, axis=1)), up


@pytest.mark.parametrize("nseq,n,heads", [(700, 1, 8), (3000, 1, 32), (3000, 40, 2), (1 << 18, 1, 2)])
def test_very_many_sequences(tq, nseq, n, heads):  # noqa: F811
    """Every sequence one of 192 kinds (queries, page, up to 48 + n keys), some of them
    without new tokens, a few with more: as the 192 kinds alone, each within the
    documented precision of the exact result."""
    d, kinds, page = 64, 192, 16
    (qk, tk), (qv, tv) = quantizer(tq, d, 4, False), quantizer(tq, d, 4, False, seed=1)
    rng = np.random.default_rng(nseq + n)
    width = (48 + n + page - 1) // page + 1
    caches = []
    for q in (qk, qv):
        c = q.empty_paged(kinds * width, 1, page)
        c.codes.random_(0, 256)
        c.norms.copy_(torch.from_numpy(rng.uniform(0.5, 8.0, c.norms.shape).astype(np.float32)))
        caches.append(c)
    y = torch.from_numpy(rng.standard_normal((kinds, n, heads * d)).astype(np.float32)).bfloat16().cuda()
    lens = torch.from_numpy(rng.integers(n, 48 + n, kinds)).cuda()
    table = torch.arange(kinds * width, device="cuda").view(kinds, width)

    def call(kind, news):
        starts = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), news.cumsum(0)])
        rows = torch.arange(int(starts[-1]), device="cuda")
        seq = torch.searchsorted(starts, rows, right=True) - 1
        at = rows - starts[seq]
        yy = y[kind[seq], at]
        out = tq.tq_attend_paged(qk, qv, yy, starts.to(torch.int32), *caches, table[kind].to(torch.int32),
                                 lens[kind].to(torch.int32), n, 0.1)
        tq.tq_sync_check(qk)
        return out, kind[seq], at
    ref = call(torch.arange(kinds, device="cuda"), torch.full((kinds,), n, device="cuda"))[0].view(kinds, n, heads * d)
    kind = torch.from_numpy(rng.integers(0, kinds, nseq)).cuda()
    news = torch.full((nseq,), n, device="cuda")
    news[::5] = 0
    out, of, at = call(kind, news)
    diff = (out.float() - ref[of, at].float()).view(-1, d).norm(dim=1)
    bound = 2 * (2.0 ** -9 * 8.0 + 2.0 ** -8 * (out.float().view(-1, d).norm(dim=1) + 2.0 ** -9 * 8.0))
    assert bool((diff <= bound).all())
