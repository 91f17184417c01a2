"""Precision of attention over pages for fp16 queries with many rows."""
import math

import numpy as np
import pytest
import torch

from oracle import tq_oracle as o
from tests.paged_reference import attend, unpack
from tests.test_gpu_paged import Batch, quantizer, run_case, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,kb,ip,vb", [(128, 4, False, 4), (128, 4, True, 3), (128, 5, True, 4), (128, 2, False, 2),
                                        (128, 1, False, 3), (64, 4, False, 4), (64, 4, True, 4), (64, 2, True, 2),
                                        (64, 3, False, 3)])
def test_fp16_chunks_keep_what_their_operands_hold(tq, d, kb, ip, vb):  # noqa: F811
    """With sharp heads, where the rounding of rotated queries and of centroid times
    norm to fp16 would show (by them alone 1.5e-3 of the result): the error against
    fp64, as a 2-norm over all rows, is that of the roundings that are left.  A value
    rounded to fp16 is off by half a step at most, evenly: an rms of 2^-11 / sqrt(3) of
    its power of two, and over evenly distributed logarithms 0.7355 of that, R = 2.07e-4
    of itself.
      - the result: R ||out||;
      - a weight times norm: R w ||v|| for each key, and the values' centroids, whose
        common factor leaves them within 2^-13: 2^-13 / sqrt(3) w ||v||;
      - a logit's error e moves the output by w e (v - out), to first order.  e has the
        centroids' 2^-13 / sqrt(3) of each of d products, and for inner-product keys R
        of the sign bits' part (residual norm) and R of each of its d products
        (projections).
    These are independent of each other, so their squares add up; 1.25 times the sum's
    root allows for 360 rows, few of whose keys have weight."""
    rng = np.random.default_rng(31 + d + kb)
    (qk, tk), (qv, tv) = quantizer(tq, d, kb, ip), quantizer(tq, d, vb, False, seed=1)
    n, heads, kv = 90, 4, 2000
    batch = Batch(tq, qk, qv, 1, 16, [kv], rng)
    y = torch.from_numpy(rng.standard_normal((n, heads * d)).astype(np.float32)).half().cuda()
    out = tq.tq_attend_paged(qk, qv, y, torch.tensor([0, n], dtype=torch.int32, device="cuda"), *batch.caches,
                             batch.table_dev, torch.tensor([kv], dtype=torch.int32, device="cuda"), n, 1 / math.sqrt(d))
    limits = np.repeat(kv - n + 1 + np.arange(n), heads)
    ke, ve = unpack(batch.rows[0][0][0], tk), unpack(batch.rows[1][0][0], tv)
    yd = y.double().cpu().numpy().reshape(n * heads, d)
    ref, _ = attend(yd, limits, 1 / math.sqrt(d), ke, tk, ve, tv, "f16", True)
    got = out.double().cpu().numpy().reshape(n * heads, d)
    err = np.linalg.norm(got - ref)
    R, C = 2.07e-4, 2.0 ** -13 / math.sqrt(3)
    yt, p = o.prepare_query(yd, tk)
    x = o.score(yt, p, ke, tk) / math.sqrt(d)
    w = np.where(np.arange(kv)[None] < limits[:, None], np.exp(x - x.max(1, keepdims=True)), 0.0)
    w /= w.sum(1, keepdims=True)
    c = tk.centroids[ke["codes"]]
    scale = ke["norm"][None] / math.sqrt(d)
    e2 = C ** 2 * (yt ** 2) @ (c ** 2).T * scale ** 2
    if ip:
        part = x - (yt @ c.T) * scale
        each = ke["gamma"][None] * math.sqrt(math.pi / 2) / d * scale
        e2 += R ** 2 * (part ** 2 + each ** 2 * (p ** 2).sum(1, keepdims=True))
    v = ve["norm"][:, None] * tv.centroids[ve["codes"]] @ tv.R
    far = (ref ** 2).sum(1, keepdims=True) - 2 * ref @ v.T + (v ** 2).sum(1)[None]
    made = R ** 2 * (ref ** 2).sum() + (R ** 2 + C ** 2) * (w ** 2 @ (v ** 2).sum(1)).sum() + (w ** 2 * e2 * far).sum()
    print(f"d={d} kb={kb} ip={ip} vb={vb}: {err / np.linalg.norm(ref):.2e}, {err / math.sqrt(made):.2f} of the roundings")
    assert err <= 1.25 * math.sqrt(made)


@pytest.mark.parametrize("d,kb,ip,vb", [(128, 4, False, 4), (128, 4, True, 3), (128, 2, True, 2), (128, 5, True, 4),
                                        (128, 3, False, 2), (128, 2, False, 4), (128, 1, False, 3), (64, 4, False, 4),
                                        (64, 3, True, 3), (64, 2, True, 4), (64, 5, True, 2), (64, 1, False, 2)])
def test_every_width(tq, d, kb, ip, vb):  # noqa: F811
    """Chunks with and without a prefix, of one tile of rows and of several, tokens
    that see no key, and a sequence that decodes."""
    seqs = [(40, 40), (33, 300), (1, 200), (90, 1000), (60, 40), (0, 77), (17, 129), (300, 280)]
    run_case(tq, d, kb, ip, vb, 1, 4, 16, seqs, "f16", seed=kb * 10 + vb + d, many=True)
    run_case(tq, d, kb, ip, vb, 2, 1, 48, [(256, 128)] * 20 + [(200, 700)], "f16", seed=kb * 10 + vb, many=True)
    tq.tq_sync_check(quantizer(tq, d, kb, ip)[0])
