"""Prompt attention with logits far beyond what a softmax tells apart, and with
very many sequences."""
import math

import pytest
import torch

from tests.test_gpu_prompt import DT, check, handle, make, run_case, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,dtype,ups", [(128, "bf16", (6, 10, 14, 30, 50)), (64, "bf16", (12, 30)), (128, "f16", (6, 10)),
                                         (64, "f16", (10,))])
def test_large_logits(tq, d, dtype, ups):  # noqa: F811
    """Queries and keys of size 2^up, logits up to about 2^(2 up + 5): finite
    results, and a row whose highest logit stands out by more than fp32's
    rounding of the sums has that key's value."""
    n, group = 400, 2
    y, k, v = make(n, group, 1, d, dtype, 3)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    for up in ups:
        yy, kk = y * 2.0 ** up, k * 2.0 ** up  # (exact)
        out = tq.tq_attend_prompt(handle(tq, d), yy, kk, v, cu, 1.0)
        assert bool(torch.isfinite(out).all()), up
        for h in range(group):
            x = yy[:, h * d:(h + 1) * d].double() @ kk.double().T
            x = x.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
            top = x.topk(2, dim=1)
            # 128 products of fp32 sums: 2^-23 d / 8 of sum |y| |k|; a weight below e^-40 does not show
            size = yy[:, h * d:(h + 1) * d].double().abs().amax(1) * kk.double().abs().amax() * d
            clear = top.values[:, 0] - top.values[:, 1] > (size * d / 8 * 2.0 ** -23).clamp_min(40.0)
            assert int(clear.sum()) > n // 2
            ref = v[top.indices[:, 0]].to(DT[dtype])
            assert torch.equal(out[:, h * d:(h + 1) * d][clear], ref[clear]), up


def test_hundreds_of_sequences(tq):  # noqa: F811
    """More sequences than one look of the search takes, of unequal numbers of work
    items, empty ones among them."""
    lens = [(37 * i) % 5 * ((i * 13) % 29) for i in range(700)]
    lens[5], lens[300], lens[699] = 900, 513, 640
    run_case(tq, 64, 2, 4, lens, "bf16", seed=51)
    run_case(tq, 128, 1, 16, [1 + i % 3 for i in range(257)], "f16", seed=52)


@pytest.mark.parametrize("nseq", [8191, 8193, 100000, 1 << 18])
def test_very_many_sequences(tq, nseq):  # noqa: F811
    """Beyond the sequences whose lengths the kernel keeps; most of one token, a few
    long, some empty.  A token alone in its sequence has its own value."""
    d, q = 64, handle(tq, 64)
    lens = torch.ones(nseq, dtype=torch.int64)
    lens[::7] = 0
    long = {0: 130, 8190: 70, nseq // 2: 300, nseq - 1: 65}
    for i, n in long.items():
        lens[i] = n
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    total = int(starts[-1])
    y, k, v = make(total, 1, 1, d, "bf16", 9)
    cu = starts.to(torch.int32).cuda()
    out = tq.tq_attend_prompt(q, y, k, v, cu, 0.125)
    tq.tq_sync_check(q)
    alone = torch.ones(total, dtype=torch.bool)
    for i, n in long.items():
        alone[int(starts[i]): int(starts[i]) + n] = False
    alone = alone.cuda()
    assert torch.equal(out[alone], v[alone])
    check(out, y, k, v, [int(starts[i]) for i in long], list(long.values()), 1, 1, d, 0.125, "bf16")


def test_one_long_sequence_among_very_many(tq):  # noqa: F811
    """Hundreds of levels that one sequence has alone, a group of many query heads
    and 2^18 sequences: the search passes over the others."""
    d, group, q = 64, 128, handle(tq, 64)
    nseq, at, n = 1 << 18, 200000, 3000
    lens = torch.zeros(nseq, dtype=torch.int64)
    lens[::97] = 1
    lens[at] = n
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    total = int(starts[-1])
    y, k, v = make(total, group, 1, d, "bf16", 10)
    out = tq.tq_attend_prompt(q, y, k, v, starts.to(torch.int32).cuda(), 0.125)
    tq.tq_sync_check(q)
    s = int(starts[at])
    alone = torch.ones(total, dtype=torch.bool, device="cuda")
    alone[s:s + n] = False
    assert torch.equal(out[alone], v[alone].repeat(1, group))
    some = slice(0, 2 * d)  # two of the heads
    check(out[:, some], y[:, some], k, v, [s], [n], 2, 1, d, 0.125, "bf16")
