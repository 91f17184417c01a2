"""Prompt attention: a token's output is made from what it sees alone, bit for
bit, whatever other rows share its warp and its tile."""
import math

import pytest
import torch

from tests.test_gpu_prompt import handle, make, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("group", [1, 3, 4])
def test_neighbours_of_any_size(tq, d, dtype, group):  # noqa: F811
    """Finite queries, keys and values up to 2^12 times larger behind a token, in
    its own sequence or in the next one, change nothing of its output."""
    lens = [700, 301, 90]
    cu = torch.tensor([0, 700, 1001, 1091], dtype=torch.int32, device="cuda")
    y, k, v = make(sum(lens), group, 1, d, dtype, 7, sharp=3.0)
    q = handle(tq, d)
    clean = tq.tq_attend_prompt(q, y, k, v, cu, 1 / math.sqrt(d))
    for at, end in ((700, 1001), (690, 700), (333, 700), (701, 1001), (850, 1001), (1001, 1091)):
        for up in (3, 12):
            y2, k2, v2 = y.clone(), k.clone(), v.clone()
            for x in (y2, k2, v2):
                x[at:end] *= 2.0 ** up
            out = tq.tq_attend_prompt(q, y2, k2, v2, cu, 1 / math.sqrt(d))
            same = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
            same[at:end] = False
            assert torch.equal(out[same], clean[same]), (at, up)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [3, 5, 7, 65])
def test_rows_that_no_query_fills(tq, d, group):  # noqa: F811
    """Groups that do not divide a tile's 128 rows: what an earlier call left in the
    other rows' place does not show."""
    n = 900 if group < 65 else 60
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    y, k, v = make(n, group, 1, d, "bf16", 8, sharp=3.0)
    fill = [x.contiguous() for x in make(128 * 296, 1, 1, d, "bf16", 9)]
    each = torch.arange(0, 128 * 296 + 1, 128, dtype=torch.int32, device="cuda")
    q, outs = handle(tq, d), []
    for up in (-8, 3, 12):  # tiles of 128 whole rows of this size on every SM before the call
        tq.tq_attend_prompt(q, fill[0] * 2.0 ** up, fill[1], fill[2], each, 1 / math.sqrt(d))
        outs.append(tq.tq_attend_prompt(q, y, k, v, cu, 1 / math.sqrt(d)))
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
