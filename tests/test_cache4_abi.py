"""Host-side checks of the norms' and the 4-bit cache's entry points: bad arguments are refused before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import cache4_reference as cref


@pytest.fixture(scope="module")
def L():
    from mla_attention_sequence_gb300 import build, laga
    build.build()
    return laga.lib()


P = 4096  # aligned, never dereferenced: every call below fails a check first
BIG = ctypes.c_size_t(1 << 50)


def rope_desc(**kw):
    from mla_attention_sequence_gb300 import laga
    a = dict(tokens=4, n_h=2, d_nope=8, d_rope=8, n_axes=1, sections=[4], theta=1e4, interleaved=1, inverse=0, pos64=0,
             dtype=1)
    a.update(kw)
    return laga.LagaRopeDesc(a["tokens"], a["n_h"], a["d_nope"], a["d_rope"], a["n_axes"],
                             (ctypes.c_int64 * 4)(*a["sections"]), a["theta"], a["interleaved"], a["inverse"], a["pos64"],
                             a["dtype"])


def cache(**kw):
    from mla_attention_sequence_gb300 import laga
    a = dict(codes=P, scales=P, k_rope=P, pages=9, page_size=16, d_c=512, d_rope=8, dtype=1)
    a.update(kw)
    return laga.LagaCache4(*a.values())


def test_norm_rope_refusals(L):
    def call(eps=1e-6, pos=P, q=P, k=P, wq=P, wk=P, qo=P, ko=P, **kw):
        return L.laga_mla_norm_rope(ctypes.byref(rope_desc(**kw)), eps, pos, q, k, wq, wk, qo, ko, None)

    def back(eps=1e-6, pos=P, zq=P, zk=P, q=P, k=P, wq=P, wk=P, dq=P, dk=P, dwq=P, dwk=P, ws=P, size=BIG, **kw):
        return L.laga_mla_norm_rope_bwd(ctypes.byref(rope_desc(**kw)), eps, pos, zq, zk, q, k, wq, wk, dq, dk, dwq, dwk, ws,
                                        size, None)
    both = (dict(tokens=0), dict(d_rope=7), dict(sections=[3]), dict(theta=0.5), dict(inverse=1), dict(pos=None), dict(eps=0.0),
            dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=1e11), dict(q=None), dict(wq=None), dict(k=None), dict(wk=None),
            dict(q=P + 1), dict(wk=P + 1))
    for kw in both:
        assert call(**kw) == 1, kw
        assert back(**kw) == 1, kw
    for kw in (dict(qo=None), dict(ko=None), dict(q=None, wq=None, qo=None, k=None, wk=None, ko=None)):
        assert call(**kw) == 1, kw
    for kw in (dict(zq=None), dict(dq=None), dict(dwq=None), dict(zk=None), dict(dk=None), dict(dwk=P + 1)):
        assert back(**kw) == 1, kw
    assert call(d_nope=1017) == 2 and back(d_nope=1017) == 2 and call(dtype=3) == 2
    assert L.laga_mla_norm_rope(None, 1e-6, P, P, P, P, P, P, P, None) == 1
    n = L.laga_mla_norm_rope_bwd_workspace_size(ctypes.byref(rope_desc()))
    assert n > 0 and L.laga_mla_norm_rope_bwd_workspace_size(ctypes.byref(rope_desc(d_nope=1017))) == 0
    assert back(ws=None) == 3 and back(ws=P + 16) == 3 and back(size=ctypes.c_size_t(64)) == 3


def test_cache_rows_refusals(L):
    ok = dict(batch=2, rows=2, most=3, table=P, starts=P, counts=None, c=P, k=P, w=P, eps=1e-6)

    def append(c=None, rope=rope_desc(), pos=None, **kw):
        a = {**ok, **kw}
        return L.laga_mla_cache4_append(ctypes.byref(c or cache()), *a.values(), ctypes.byref(rope) if rope else None, pos, None)

    def read(c=None, **kw):
        a = {**ok, **kw}
        del a["w"], a["eps"]
        return L.laga_mla_cache4_read(ctypes.byref(c or cache()), *a.values(), None)
    for f in (append, read):
        for kw in (dict(batch=0), dict(rows=0), dict(most=0), dict(table=None), dict(starts=None), dict(table=P + 2),
                   dict(starts=P + 1), dict(counts=P + 2), dict(c=cache(codes=None)), dict(c=cache(scales=P + 8)),
                   dict(c=cache(k_rope=None)), dict(c=cache(pages=0)), dict(c=cache(page_size=0)), dict(c=cache(d_c=0)),
                   dict(c=cache(d_rope=-1)), dict(k=None), dict(k=P + 1)):
            assert f(**kw) == 1, kw
        for kw in (dict(c=cache(d_c=1025)), dict(c=cache(d_rope=258)), dict(c=cache(page_size=65537)), dict(c=cache(dtype=2)),
                   dict(c=cache(pages=1 << 31)), dict(batch=1 << 20, rows=1 << 11)):
            assert f(**kw) == 2, kw
        assert f.__name__ and L.laga_mla_last_error()
    assert append(w=P + 1) == 1 and append(eps=0.0) == 1
    for r in (rope_desc(tokens=5), rope_desc(d_rope=6, sections=[3]), rope_desc(dtype=0), rope_desc(inverse=1), rope_desc(theta=0.0),
              rope_desc(n_axes=2, sections=[2, 2])):
        assert append(rope=r) == 1
    assert append(rope=rope_desc(pos64=1), pos=P + 4) == 1
    assert L.laga_mla_cache4_append(None, 1, 1, 1, P, P, None, P, P, None, 1e-6, None, None, None) == 1


def test_cache_attention_refusals(L):
    from mla_attention_sequence_gb300 import laga

    def call(c=None, mods=None, table=P, lengths=P, q=P, wk=P, wv=P, o=P, l=P, ws=P, size=BIG, **kw):
        a = dict(batch=2, sq=1, n_h=4, d_nope=128, d_v=128, max_pages=8, causal=1, scale=0.0, variant=0)
        a.update(kw)
        d = laga.LagaCache4Desc(*a.values())
        return L.laga_mla_cache4_fwd(ctypes.byref(d), ctypes.byref(c or cache(d_rope=64)), ctypes.byref(mods) if mods else None,
                                     table, lengths, q, wk, wv, o, l, ws, size, None)
    for kw in (dict(batch=0), dict(sq=0), dict(n_h=0), dict(d_nope=0), dict(d_v=0), dict(max_pages=0), dict(table=None),
               dict(lengths=None), dict(lengths=P + 2), dict(q=None), dict(wk=P + 8), dict(o=None), dict(l=None),
               dict(scale=float("nan")), dict(c=cache(codes=P + 8, d_rope=64)), dict(mods=laga.LagaMods(None, None, None, -1.0)),
               dict(mods=laga.LagaMods(P + 2, None, None, 0.0))):
        assert call(**kw) == 1, kw
    for kw in (dict(variant=1), dict(variant=2), dict(d_nope=200), dict(d_v=257), dict(n_h=1 << 16), dict(batch=1 << 31),
               dict(max_pages=1 << 30), dict(batch=1 << 20, sq=1 << 9)):
        assert call(**kw) == 2, kw
    assert call(ws=None) == 3 and call(ws=P + 64) == 3 and call(size=ctypes.c_size_t(1 << 10)) == 3
    d = laga.LagaCache4Desc(2, 1, 4, 128, 128, 8, 1, 0.0, 0)
    n = L.laga_mla_cache4_fwd_workspace_size(ctypes.byref(d), ctypes.byref(cache(codes=None, scales=None, k_rope=None, d_rope=64)))
    assert n > 0 and call(size=ctypes.c_size_t(n - 1)) == 3
    d.variant = 2
    assert L.laga_mla_cache4_fwd_workspace_size(ctypes.byref(d), ctypes.byref(cache(d_rope=64))) == 0


def test_binding_refuses_cpu_tensors():
    from mla_attention_sequence_gb300 import laga
    c = laga.cache4(4, 16, 32, 8, torch.float32, "cpu")
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.cache4_read(c, i[None], i, 1)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.cache4_append(c, torch.zeros(1, 1, 32), torch.zeros(1, 1, 8), i[None], i)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.cache4_fwd(torch.zeros(1, 1, 2, 24), c, torch.zeros(32, 32), torch.zeros(32, 32), i[None], i)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.norm_rope(torch.zeros(1, 1, 2, 24), None, i[None, None], torch.ones(24), sections=[4])
    with pytest.raises(TypeError):
        laga.cache4(4, 16, 32, 8, torch.float16, "cpu")


def test_reference_scales_are_upper_bytes_of_fp16():
    v = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)
    np.testing.assert_array_equal(cref.scale_values()[:248], v[:248])
    assert not np.isfinite(v[248:]).any() and 6 * v[226] == 61440
    # a code times a scale has at most six significant bits: exact in fp16 and bf16
    p = np.multiply.outer(cref.SIZES, v[:227])
    np.testing.assert_array_equal(p.astype(np.float16).astype(np.float64), p)
    np.testing.assert_array_equal(torch.from_numpy(p).bfloat16().double().numpy(), p)


def test_reference_encoding_of_known_blocks():
    x = np.zeros((1, 20))
    x[0, :16] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5, 0.26, 4.99, -0.2, 1, 2, 3]
    x[0, 16:] = [1e6, -1, 0, 61440]
    codes, scales, vals = cref.encode(x)
    assert scales.tolist() == [[15 * 8, 226]]
    np.testing.assert_array_equal(vals[0], [6, -6, 0, 1, 1, 2, 2, 4, 4, -4, 0.5, 4, 0, 1, 2, 3, 61440, 0, 0, 61440])
    np.testing.assert_array_equal(cref.decode(torch.from_numpy(codes), torch.from_numpy(scales), 20)[0].numpy(), vals[0])


def test_append_ignores_what_its_rotation_does_not_use(L):
    """The rows of an append have no heads: its rotation's n_h and d_nope are not looked at, nor is a limit that they
    would pass; without pos neither is pos64. (Another field is wrong in each call: none gets as far as a launch.)"""
    for kw, starts in ((dict(n_h=0, d_nope=0), P), (dict(n_h=-3, d_nope=-1), P), (dict(n_h=1 << 20), P), (dict(d_nope=1 << 20), P),
                       (dict(n_h=60000, d_nope=60000), P), (dict(pos64=1), P + 4)):
        rope = rope_desc(inverse=1, **kw)
        assert L.laga_mla_cache4_append(ctypes.byref(cache()), 2, 2, 3, P, starts, None, P, P, None, 1e-6, ctypes.byref(rope),
                                        None, None) == 1
        assert b"not inverse" in L.laga_mla_last_error(), (kw, L.laga_mla_last_error())
