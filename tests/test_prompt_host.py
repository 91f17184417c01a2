"""Argument checks of prompt attention without a GPU: every refusal comes
before a pointer is touched."""
import ctypes

import pytest

fake = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def tq():
    from online_vector_quantization_tq_b200 import build
    build.build()
    import online_vector_quantization_tq_b200 as pkg
    pkg.lib()
    return pkg


def test_refusals(tq):
    L, q = tq.lib(), tq.tq_codebook_mse_host(128, 4)
    names = "q dtype y ldy k ldk v ldv total cu nseq heads kv_heads scale out ldo".split()
    ok = dict(q=q.handle, dtype=1, y=fake, ldy=1536, k=fake, ldk=1536, v=fake, ldv=1536, total=9, cu=fake, nseq=2,
              heads=8, kv_heads=2, scale=0.1, out=fake, ldo=1024)

    def call(**kw):
        a = {**ok, **kw}
        return L.tq_attend_prompt(*(a[n] for n in names), None)

    assert call() == 2 and call(dtype=2) == 2  # a host-only quantizer: everything else was in order
    assert call(total=0) == 0 and call(nseq=0) == 0
    for kw in (dict(q=None), dict(total=-1), dict(nseq=-1), dict(heads=0), dict(kv_heads=0), dict(heads=7),
               dict(y=None), dict(k=None), dict(v=None), dict(cu=None), dict(out=None), dict(scale=float("nan")),
               dict(scale=float("-inf")), dict(ldy=1016), dict(ldk=248), dict(ldv=248), dict(ldo=1016)):
        assert call(**kw) == 1, kw
    for kw in (dict(dtype=0), dict(dtype=9), dict(q=tq.tq_codebook_mse_host(32, 4).handle),
               dict(q=tq.tq_codebook_host(256, 4).handle), dict(heads=129, kv_heads=1, ldy=1 << 16, ldo=1 << 16)):
        assert call(**kw) == 2, kw
    odd = ctypes.c_void_p(0x1008)
    for kw in (dict(y=odd), dict(k=odd), dict(v=odd), dict(out=odd), dict(ldy=1540), dict(ldk=1540), dict(ldv=1540),
               dict(ldo=1028), dict(cu=ctypes.c_void_p(0x1002))):
        assert call(**kw) == 3, kw
    for kw in (dict(total=1 << 31), dict(nseq=1 << 25), dict(heads=1 << 17, kv_heads=1 << 16, ldy=1 << 24, ldo=1 << 24),
               dict(ldk=1 << 40)):
        assert call(**kw) == 7, kw
