"""Precision of attention over pages with inner-product keys of few bits, whose
sign bits make a large part of the logits, for fp16 queries with many rows."""
import math

import numpy as np
import pytest
import torch

from oracle import tq_oracle as o
from tests.paged_reference import attend, unpack
from tests.test_gpu_paged import Batch, quantizer, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,kb,vb,sharp", [(128, 2, 3, 1.0), (128, 2, 4, 2.0), (128, 3, 3, 2.0), (128, 4, 4, 2.0),
                                           (128, 5, 4, 2.0), (64, 2, 3, 1.0), (64, 2, 2, 2.0), (64, 3, 4, 2.0),
                                           (64, 5, 4, 1.0)])
def test_sign_bits_keep_what_their_operands_hold(tq, d, kb, vb, sharp):  # noqa: F811
    """The error against fp64, as a 2-norm over all rows, is that of the roundings
    that are left.  A value rounded to fp16 is off by half a step at most, evenly: over
    evenly distributed logarithms an rms of R = 2.07e-4 of itself.
      - the result: R ||out||; a weight times norm: R w ||v|| for each key; the
        values' centroids, under one common factor: 2^-13 / sqrt(3) w ||v||;
      - a logit's error e moves the output by w e (v - out), to first order.  e has R
        of each of the d products with projections; of the sign bits' part as a whole
        what the best of 16 common factors leaves of the residual norm's rounding,
        evenly distributed before: sqrt(2 / (17 18)) against sqrt(1 / 3) of the half
        step, 0.14 R; and of the d products with centroids, whose 16 tables are each
        the best of 256, an rms of 2^-13 / sqrt(3) at most.
    Their squares add up; 1.25 times the sum's root allows for 360 rows, few of whose
    keys have weight."""
    rng = np.random.default_rng(77 + d + kb)
    (qk, tk), (qv, tv) = quantizer(tq, d, kb, True), quantizer(tq, d, vb, False, seed=1)
    n, heads, kv = 90, 4, 2000
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    y = torch.from_numpy(sharp * rng.standard_normal((n, heads * d)).astype(np.float32)).half().cuda()
    out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                             batch.table_dev, torch.tensor([kv], dtype=torch.int32, device="cuda"), n, 1 / math.sqrt(d))
    limits = np.repeat(kv - n + 1 + np.arange(n), heads)
    ke, ve = unpack(batch.rows[0][0][0], tk), unpack(batch.rows[1][0][0], tv)
    yd = y.double().cpu().numpy().reshape(n * heads, d)
    ref, bound = attend(yd, limits, 1 / math.sqrt(d), ke, tk, ve, tv, "f16", True)
    got = out.double().cpu().numpy().reshape(n * heads, d)
    assert np.all(np.abs(got - ref) <= bound)
    err = np.linalg.norm(got - ref)
    R, C = 2.07e-4, 2.0 ** -13 / math.sqrt(3)
    yt, p = o.prepare_query(yd, tk)
    x = o.score(yt, p, ke, tk) / math.sqrt(d)
    w = np.where(np.arange(kv)[None] < limits[:, None], np.exp(x - x.max(1, keepdims=True)), 0.0)
    w /= w.sum(1, keepdims=True)
    c = tk.centroids[ke["codes"]]
    scale = ke["norm"][None] / math.sqrt(d)
    part = x - (yt @ c.T) * scale
    each = ke["gamma"][None] * math.sqrt(math.pi / 2) / d * scale
    e2 = C ** 2 * (yt ** 2) @ (c ** 2).T * scale ** 2 + R ** 2 * each ** 2 * (p ** 2).sum(1, keepdims=True)
    e2 += (0.14 * R * part) ** 2
    v = ve["norm"][:, None] * tv.centroids[ve["codes"]] @ tv.R
    far = (ref ** 2).sum(1, keepdims=True) - 2 * ref @ v.T + (v ** 2).sum(1)[None]
    made = R ** 2 * (ref ** 2).sum() + (R ** 2 + C ** 2) * (w ** 2 @ (v ** 2).sum(1)).sum() + (w ** 2 * e2 * far).sum()
    print(f"d={d} kb={kb} vb={vb}: {err / np.linalg.norm(ref):.2e}, {err / math.sqrt(made):.2f} of the roundings")
    assert err <= 1.25 * math.sqrt(made)
