"""Argument checks of the paged-cache calls without a GPU: every refusal comes
before a pointer is touched."""
import ctypes

import pytest
import torch

fake = ctypes.c_void_p(0x1000)


@pytest.fixture(scope="module")
def tq():
    from online_vector_quantization_tq_b200 import build
    build.build()
    import online_vector_quantization_tq_b200 as pkg
    pkg.lib()
    return pkg


def rows(tq, codes=0x1000, signs=0x1000, norms=0x1000):
    return tq.binding._Rows(codes, signs, norms)


def test_store_refusals(tq):
    L, qk, qv = tq.lib(), tq.tq_codebook_host(128, 4), tq.tq_codebook_mse_host(128, 4)
    ok = dict(qk=qk.handle, qv=qv.handle, kr=rows(tq), vr=rows(tq, signs=0), slots=fake, tokens=4, heads=2,
              kp=rows(tq), vp=rows(tq, signs=0), npages=3, page=16)

    def call(**kw):
        a = {**ok, **kw}
        return L.tq_paged_store(a["qk"], a["qv"], a["kr"], a["vr"], a["slots"], a["tokens"], a["heads"], a["kp"],
                                a["vp"], a["npages"], a["page"], None)

    assert call() == 2  # host-only quantizers: everything else was in order
    assert call(tokens=0) == 0 and call(npages=0) == 0
    for kw in (dict(qk=None), dict(qv=None), dict(tokens=-1), dict(heads=0), dict(npages=-1), dict(page=0),
               dict(page=24), dict(page=2048), dict(slots=None), dict(kr=None), dict(kp=None), dict(kr=rows(tq, 0)),
               dict(kp=rows(tq, signs=0)), dict(vp=rows(tq, norms=0)), dict(kr=rows(tq, signs=0))):
        assert call(**kw) == 1, kw
    for kw in (dict(kp=rows(tq, codes=0x1008)), dict(vp=rows(tq, norms=0x1008)), dict(kr=rows(tq, codes=0x1002)),
               dict(vr=rows(tq, norms=0x1004)), dict(slots=ctypes.c_void_p(0x1004))):
        assert call(**kw) == 3, kw
    assert call(npages=1 << 31) == 7 and call(heads=1 << 17) == 7


def test_attend_refusals(tq):
    L, qk, qv = tq.lib(), tq.tq_codebook_host(128, 4), tq.tq_codebook_mse_host(128, 4)
    names = ("qk qv dtype y ldy total q_start nseq max_new heads kv_heads kp vp npages page table ldt max_pages "
             "kv_len scale out ldo ws ws_bytes").split()
    ok = dict(qk=qk.handle, qv=qv.handle, dtype=1, y=fake, ldy=1024, total=3, q_start=fake, nseq=3, max_new=1,
              heads=8, kv_heads=2, kp=rows(tq), vp=rows(tq, signs=0), npages=9, page=16, table=fake, ldt=4,
              max_pages=4, kv_len=fake, scale=0.1, out=fake, ldo=1024, ws=fake, ws_bytes=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return L.tq_attend_paged(*(a[n] for n in names), None)

    assert call() == 2  # host-only quantizers: everything else was in order
    assert call(dtype=2) == 2
    assert call(total=0) == 0 and call(nseq=0) == 0 and call(max_new=0) == 0
    for kw in (dict(qk=None), dict(qv=None), dict(total=-1), dict(nseq=-1), dict(heads=7), dict(heads=0),
               dict(kv_heads=0), dict(max_new=-1), dict(page=20), dict(npages=-1), dict(y=None), dict(q_start=None),
               dict(kv_len=None), dict(table=None), dict(out=None), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(ldy=1023), dict(ldo=1020), dict(ldt=3), dict(kp=None),
               dict(kp=rows(tq, norms=0)), dict(max_pages=-1)):
        assert call(**kw) == 1, kw
    for kw in (dict(out=ctypes.c_void_p(0x1002)), dict(ldo=1026), dict(y=ctypes.c_void_p(0x1001)),
               dict(kv_len=ctypes.c_void_p(0x1002)), dict(kp=rows(tq, codes=0x1004))):
        assert call(**kw) == 3, kw
    for kw in (dict(ws=None), dict(ws=ctypes.c_void_p(0x1008))):
        assert call(**kw) == 6, kw
    for kw in (dict(nseq=1 << 25), dict(max_new=1 << 29), dict(max_pages=1 << 28, ldt=1 << 28)):
        assert call(**kw) == 7, kw
    for kw in (dict(dtype=0), dict(dtype=9), dict(qv=qk.handle), dict(qv=tq.tq_codebook_mse_host(64, 4).handle),
               dict(qv=tq.tq_codebook_mse_host(128, 1).handle), dict(qk=tq.tq_codebook_host(96, 4).handle),
               dict(qk=tq.tq_codebook_host(128, 4, rotation="haar").handle)):
        assert call(**kw) == 2, kw
    assert L.tq_attend_paged_workspace_bytes(qk.handle, qv.handle, 3, 3, 7, 2, 1, 4, 16) == 0


def test_cache_shapes_are_checked(tq):
    """The binding refuses arrays that the library would read as something else."""
    q = tq.tq_codebook_host(128, 4)
    good = q.empty_paged(3, 2, 16, device="cpu").check(q)
    P = tq.PagedCache
    for bad in (P(good.codes[:, :, ::2], good.signs, good.norms), P(good.codes, good.signs[:2], good.norms),
                P(good.codes, good.signs, good.norms.double()), P(good.codes[..., :40], good.signs, good.norms),
                P(good.codes.transpose(1, 2), good.signs.transpose(1, 2), good.norms.transpose(1, 2))):
        with pytest.raises(ValueError):
            bad.check(q)
    with pytest.raises(ValueError):
        tq.tq_paged_store(q, q, tq.Encoded(torch.zeros(2, 48, dtype=torch.uint8), torch.zeros(2, 16, dtype=torch.uint8),
                                           torch.zeros(2, 2)), None, torch.zeros(1, dtype=torch.int64), good, good)


def test_host_tensors_are_refused(tq):
    """Before any launch, wherever among the arguments they stand."""
    from online_vector_quantization_tq_b200.binding import _one_device
    q = tq.tq_codebook_host(128, 4)
    none, some = torch.empty(0), torch.empty(3)
    assert _one_device(q, "a b", none, None) == -1
    for tensors in ((some, none), (none, some), (some, some), (None, some)):
        with pytest.raises(ValueError):
            _one_device(q, "a b", *tensors)


def test_attention_of_host_tensors_is_refused(tq):
    q, v = tq.tq_codebook_host(128, 4), tq.tq_codebook_mse_host(128, 4)
    y, cu = torch.zeros(4, 256, dtype=torch.bfloat16), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.tq_attend_prompt(v, y, y, y, cu, 0.1)
    kc, vc = q.empty_paged(3, 2, 16, device="cpu"), v.empty_paged(3, 2, 16, device="cpu")
    table, lens = torch.zeros(1, 2, dtype=torch.int32), torch.tensor([4], dtype=torch.int32)
    with pytest.raises(ValueError):
        tq.tq_attend_paged(q, v, y, cu, kc, vc, table, lens, 4, 0.1, workspace=torch.empty(64, dtype=torch.uint8))
