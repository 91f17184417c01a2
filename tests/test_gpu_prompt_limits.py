"""Prompt attention with logits far beyond what a softmax tells apart."""
import math

import pytest
import torch

from tests.test_gpu_prompt import DT, handle, make, tq  # noqa: F401

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
