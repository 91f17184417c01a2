"""A cache of more rows than 31 bits number and more bytes than 32 bits do."""
import numpy as np
import pytest
import torch

from tests.test_gpu_paged import DT, quantizer, random_rows, tq  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kb,ip,vb", [(1, False, 2), (4, True, 4)])
def test_rows_at_the_far_end(tq, kb, ip, vb):  # noqa: F811
    """Tokens stored in the last pages of a large cache (whose other pages are never
    touched) and in a small one: the same rows, and attention the same, bit for bit."""
    d, kv_heads, page = 64, 8, 1024
    npages = 270_000 if kb == 1 else 30_000  # 2.2e9 rows of 8 to 16 bytes; 2.5e8 rows of 32
    rng = np.random.default_rng(kb)
    qk, qv = quantizer(tq, d, kb, ip)[0], quantizer(tq, d, vb, False, seed=1)[0]
    need = npages * kv_heads * page * (qk.code_bytes + qk.sign_bytes + qv.code_bytes + 16)
    if torch.cuda.mem_get_info()[0] < need + (4 << 30):
        pytest.skip("not enough device memory")
    tokens, few = 5000, 6
    encs = [tq.Encoded(*(torch.from_numpy(p).cuda() for p in random_rows(q, tokens * kv_heads, rng))) for q in (qk, qv)]
    pages = torch.tensor([3, 0, 5, 1, 4])
    at = torch.arange(tokens)
    y = torch.from_numpy(rng.standard_normal((40, kv_heads * 4 * d)).astype(np.float32))
    outs = []
    for total in (few, npages):
        kc, vc = qk.empty_paged(total, kv_heads, page), qv.empty_paged(total, kv_heads, page)
        table = total - few + pages
        slots = (table[at // page] * page + at % page).cuda()
        tq.tq_paged_store(qk, qv, *encs, slots, kc, vc)
        got = []
        for c, e in ((kc, encs[0]), (vc, encs[1])):
            for dst, src in ((c.codes, e.codes), (c.norms, e.norms)) + (((c.signs, e.signs),) if c.signs.shape[-1] > 0 else ()):
                back = dst[slots // page, :, slots % page].reshape(src.shape)
                assert torch.equal(back, src)
        for n, dtype in ((1, "bf16"), (8, "f16"), (40, "bf16"), (40, "f16")):
            got.append(tq.tq_attend_paged(
                qk, qv, y[:n].to(DT[dtype]).cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda"), kc, vc,
                table[None].to(torch.int32).cuda(), torch.tensor([tokens], dtype=torch.int32, device="cuda"), n, 0.1))
        tq.tq_sync_check(qk)
        outs.append(got)
        del kc, vc
    for a, b in zip(*outs):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)
    torch.cuda.empty_cache()
