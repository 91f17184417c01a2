"""A server's steps side by side: prompts on one stream, their keys and values
encoded and stored on a second, other sequences' new tokens on two more, with
one pair of quantizers and a workspace for each call that may run at the same
time.  Results are those of the calls one after the other, bit for bit."""
import pytest
import torch

from tests.test_gpu_paged import quantizer, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,ip,dtype", [(64, False, "bf16"), (64, True, "f16"), (128, False, "f16"), (128, True, "bf16")])
def test_calls_on_four_streams(tq, d, ip, dtype):  # noqa: F811
    heads, kv_heads, page = 8, 2, 16
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    g = torch.Generator(device="cuda").manual_seed(d)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    (qk, _), (qv, _) = quantizer(tq, d, 4, ip), quantizer(tq, d, 4, False, seed=1)
    lens = [3000, 1, 777, 2500, 40]
    total, scale = sum(lens), 0.1
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
    y, k, v = rand(total, heads * d).to(dt), rand(total, kv_heads * d).to(dt), rand(total, kv_heads * d).to(dt)
    rows = [x.view(-1, d).to(torch.bfloat16) for x in (k, v)]
    slots = torch.randperm(total + 500, device="cuda", generator=g)[:total]
    npages = (total + 500 + page - 1) // page
    # the sequences of other steps: a decode batch and a batch with chunks
    kc, vc = (q.empty_paged(800, kv_heads, page) for q in (qk, qv))
    for c in (kc, vc):
        c.codes.random_(0, 256)
        c.norms.uniform_(0.5, 4.0)
        if c.signs.numel():
            c.signs.random_(0, 256)
    batches = []
    for news, kv in (([1] * 16, 5000), ([300, 1, 70, 16], 3000)):
        n = len(news)
        start = torch.tensor([0] + torch.tensor(news).cumsum(0).tolist(), dtype=torch.int32, device="cuda")
        table = torch.randint(0, 800, (n, 320), device="cuda", generator=g, dtype=torch.int32)
        kvs = torch.randint(kv // 2, kv, (n,), device="cuda", generator=g, dtype=torch.int32)
        batches.append((rand(sum(news), heads * d).to(dt), start, kc, vc, table, kvs, max(news), scale))

    def fresh():
        return [q.empty_paged(npages, kv_heads, page) for q in (qk, qv)]

    def store(caches, s):
        encs = [tq.tq_encode(q, x, stream=s) for q, x in zip((qk, qv), rows)]
        tq.tq_paged_store(qk, qv, *encs, slots, *caches, stream=s)
    caches = fresh()
    store(caches, None)
    kept = [[t.view(-1, t.shape[-1]) for t in (c.codes, c.signs, c.norms) if t.shape[-1]] for c in caches]
    at = (slots // page * kv_heads * page + slots % page)[:, None] + torch.arange(kv_heads, device="cuda") * page
    ref = [tq.tq_attend_prompt(qk, y, k, v, cu, scale)] + [tq.tq_attend_paged(qk, qv, *b) for b in batches]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    outs, made = [], []
    for turn in range(6):
        made.append(fresh())
    torch.cuda.synchronize()
    for turn in range(6):
        outs.append([tq.tq_attend_prompt(qk, y, k, v, cu, scale, stream=streams[0])])
        store(made[turn], streams[1])
        outs[-1] += [tq.tq_attend_paged(qk, qv, *b, stream=s) for b, s in zip(batches, streams[2:])]
    torch.cuda.synchronize()
    for q in (qk, qv):
        tq.tq_sync_check(q)
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    for c2 in made:
        for c, want in zip(c2, kept):
            now = [t.view(-1, t.shape[-1]) for t in (c.codes, c.signs, c.norms) if t.shape[-1]]
            assert all(torch.equal(a[at], b[at]) for a, b in zip(now, want))
