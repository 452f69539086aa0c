"""Host-side checks of the packed-document entry points: bad arguments are refused before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import masked_reference as ref


@pytest.fixture(scope="module")
def L():
    from mla_attention_sequence_gb300 import build, laga
    build.build()
    return laga.lib()


def desc(**kw):
    from mla_attention_sequence_gb300 import laga
    from mla_attention_sequence_gb300.configs import DSV3_LAST_RANK
    p = DSV3_LAST_RANK.with_(**{k: v for k, v in kw.items() if k in DSV3_LAST_RANK.__dataclass_fields__})
    return laga.make_desc(p, None, kw.get("variant", "auto"), kw.get("flags", 0))


P = 4096  # aligned, never dereferenced: every call below fails a check first
BIG = ctypes.c_size_t(1 << 50)


def fwd(L, d, mods=None, ws=P, size=BIG, **ptr):
    a = dict(q=P, c=P, r=P, wk=P, wv=P, o=P, l=P)
    a.update(ptr)
    return L.laga_mla_masked_fwd(ctypes.byref(d) if d else None, ctypes.byref(mods) if mods else None, *a.values(), ws,
                                 size, None)


def bwd(L, d, mods=None, q8=None, out8=None, ws=P, size=BIG, **ptr):
    a = dict(q=P, c=P, r=P, wk=P, wv=P, o=P, l=P, do=P)
    g = dict(dq=P, dc=P, dr=P, dwk=P, dwv=P)
    for k, v in ptr.items():
        (a if k in a else g)[k] = v
    ref8 = [ctypes.byref(t) if t else None for t in (q8, out8)]
    return L.laga_mla_masked_bwd(ctypes.byref(d), ctypes.byref(mods) if mods else None, *a.values(), *ref8, *g.values(),
                                 ws, size, None)


def mods(**kw):
    from mla_attention_sequence_gb300 import laga
    return laga.LagaMods(kw.get("lo"), kw.get("hi"), kw.get("slopes"), kw.get("cap", 0.0))


def test_forward_refusals(L):
    assert fwd(L, None) == 1
    assert fwd(L, desc(), q=None) == 1
    assert fwd(L, desc(), o=P + 1) == 1
    assert fwd(L, desc(), r=None) == 1
    assert fwd(L, desc(q_offset=15000)) == 1  # a causal shard past the latent
    for cap in (-1.0, float("nan"), float("inf"), 1e-30, 3e38):
        assert fwd(L, desc(), mods(cap=cap)) == 1
        assert b"softcap" in L.laga_mla_last_error()
    assert fwd(L, desc(), mods(lo=P + 2)) == 1
    assert fwd(L, desc(variant="fused_recon")) == 2
    assert fwd(L, desc(flags=2)) == 2  # prebuilt K/V
    assert fwd(L, desc(flags=8)) == 1
    assert fwd(L, desc(dtype="f32", d_nope=200, d_rope=64, Sq=8, S=64, q_offset=0)) == 2
    assert b"256" in L.laga_mla_last_error()
    d = desc()
    n = L.laga_mla_masked_fwd_workspace_size(ctypes.byref(d))
    assert n > L.laga_mla_fwd_workspace_size(ctypes.byref(d)) > 0
    assert fwd(L, d, size=ctypes.c_size_t(n - 1)) == 3
    assert fwd(L, d, ws=None) == 3
    assert fwd(L, d, ws=P + 16) == 3


def test_backward_refusals(L):
    from mla_attention_sequence_gb300 import laga
    d = desc()
    pk = laga.LagaPacked(P, P)
    assert bwd(L, d, dq=None) == 1
    assert bwd(L, d, q=None) == 1
    assert bwd(L, d, q=None, o=None, q8=pk) == 1  # one checkpoint alone
    assert bwd(L, d, q8=pk, out8=pk) == 1  # both a tensor and its checkpoint
    assert bwd(L, d, q=None, o=None, q8=pk, out8=laga.LagaPacked(P, None)) == 1
    assert bwd(L, d, q=None, o=None, q8=laga.LagaPacked(P + 8, P), out8=pk) == 1
    n = L.laga_mla_masked_bwd_workspace_size(ctypes.byref(d))
    assert n > L.laga_mla_masked_fwd_workspace_size(ctypes.byref(d))
    assert bwd(L, d, q=None, o=None, q8=pk, out8=pk, size=ctypes.c_size_t(n - 1)) == 3
    f = desc(variant="fused_recon")
    assert L.laga_mla_masked_bwd_workspace_size(ctypes.byref(f)) == 0


def test_key_bounds_refusals(L):
    ok = dict(B=1, sq=8, skv=8, off=0, split=0, off2=0, starts=P, docs=1, prefix=None, window=0, lo=P, hi=P)

    def call(**kw):
        return L.laga_mla_key_bounds(*{**ok, **kw}.values(), None)
    for kw in (dict(B=0), dict(sq=0), dict(skv=0), dict(docs=0), dict(off=-1), dict(split=8), dict(split=-1),
               dict(split=4, off2=-1), dict(window=-1), dict(starts=None), dict(lo=None), dict(hi=P + 1),
               dict(prefix=P + 2), dict(prefix=P, window=4)):
        assert call(**kw) == 1, kw
    assert call(B=1 << 20) == 2
    assert call(sq=1 << 31) == 2


def test_rope_refusals(L):
    from mla_attention_sequence_gb300 import laga

    def call(pos=P, q=P, k=P, qo=P, ko=P, **kw):
        a = dict(tokens=4, n_h=2, d_nope=8, d_rope=8, n_axes=1, sections=[4], theta=1e4, dtype=1)
        a.update(kw)
        d = laga.LagaRopeDesc(a["tokens"], a["n_h"], a["d_nope"], a["d_rope"], a["n_axes"],
                              (ctypes.c_int64 * 4)(*a["sections"]), a["theta"], 1, 0, kw.get("pos64", 0), a["dtype"])
        return L.laga_mla_rope(ctypes.byref(d), pos, q, k, qo, ko, None)
    assert L.laga_mla_rope(None, P, P, P, P, P, None) == 1
    for kw in (dict(tokens=0), dict(n_h=0), dict(d_rope=7), dict(d_rope=0), dict(n_axes=0), dict(n_axes=5),
               dict(sections=[3]), dict(sections=[5, -1], n_axes=2), dict(theta=0.5), dict(theta=float("inf")),
               dict(theta=float("nan")), dict(pos=None), dict(pos=P + 4, pos64=1), dict(q=None), dict(qo=None),
               dict(q=None, qo=None, k=None, ko=None), dict(q=P + 1)):
        assert call(**kw) == 1, kw
    assert call(dtype=7) == 2
    assert call(d_rope=258, sections=[129]) == 2


def test_pack8_refusals(L):
    for f, args in ((L.laga_mla_pack8, (P, P, P)), (L.laga_mla_unpack8, (P, P, P))):
        assert f(1, 0, 8, *args, None) == 1
        assert f(1, 8, 0, *args, None) == 1
        assert f(5, 8, 8, *args, None) == 2
        assert f(1, 1 << 36, 8, *args, None) == 2
        assert f(1, 8, 1 << 30, *args, None) == 2
        assert f(1, 8, 8, None, P, P, None) == 1
        assert f(1, 8, 8, P, P, None, None) == 1
    assert L.laga_mla_pack8(0, 8, 8, P + 2, P, P, None) == 1
    assert L.laga_mla_unpack8(0, 8, 8, P, P, P + 2, None) == 1


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    from mla_attention_sequence_gb300 import laga
    q, c, r, w = torch.zeros(1, 4, 2, 48), torch.zeros(1, 4, 64), torch.zeros(1, 4, 16), torch.zeros(64, 64)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.masked_fwd(q, c, r, w, w)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.pack8(q)
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.rope(q, r, torch.zeros(1, 1, 4, dtype=torch.int32))
    with pytest.raises(RuntimeError, match="CUDA"):
        laga.key_bounds(torch.zeros(1, 2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        laga.key_bounds(torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(TypeError):
        laga.pack8(torch.zeros(4, dtype=torch.float16))
    with pytest.raises(ValueError, match="both"):
        laga.masked_bwd(laga.Packed8(q, q, torch.float32), c, r, w, w, q, q, q)


def test_reference_checkpoint_table():
    """The tests' own e4m3 table against torch's type, all 256 codes."""
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(ref.e4m3_values(), t)


def test_reference_gradient_by_differences():
    """The 64-bit reference's gradients against central differences of its forward."""
    g = torch.Generator().manual_seed(3)
    x = {k: torch.randn(*s, generator=g, dtype=torch.float64) for k, s in dict(
        q=(1, 6, 2, 7), c_kv=(1, 9, 5), k_rope=(1, 9, 3), W_UK=(5, 8), W_UV=(5, 6)).items()}
    dout = torch.randn(1, 6, 2, 3, generator=g, dtype=torch.float64)
    slopes = torch.tensor([0.1, 0.4])
    seen = torch.rand(1, 6, 9, generator=g) < 0.6
    seen[0, 2] = False
    kw = dict(softcap=1.5, slopes=slopes, pos=torch.arange(6) + 3)
    r = ref.attention(x, seen, dout=dout, **kw)
    for k in x:
        d = torch.randn(x[k].shape, generator=g, dtype=torch.float64)
        h = 1e-5
        up, down = (float((ref.attention({**x, k: x[k] + s * h * d}, seen, **kw)["out"] * dout).sum()) for s in (1, -1))
        name = {"q": "dq", "c_kv": "dc_kv", "k_rope": "dk_rope", "W_UK": "dW_UK", "W_UV": "dW_UV"}[k]
        want = float((r[name] * d).sum())
        assert abs((up - down) / (2 * h) - want) <= 1e-7 * max(1.0, abs(want)), k  # h^2 + 2^-53 / h
