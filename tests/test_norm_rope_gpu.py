"""Norms with rotation, forward and backward, against their definition in 64 bits.

Tolerances (2-norm of the error over that of the result or of its uncancelled size). bf16: one rounding of
the result, at most 2^-8 of it. fp32, in units of 2^-24: a row's sum of at most 32 terms a lane and five
shuffles, halved by the root (20); rsqrt (4); the products with the row's factor and the weight (4); the
turn, its angle's 2^-26 of a turn among it (6); the backward's second sum of as many terms, as a part of the
uncancelled size (40), and its products (6): 80 units, 5e-6."""
import pytest
import torch

import cache4_reference as cref
from mla_attention_sequence_gb300 import build, laga

pytestmark = pytest.mark.gpu
TOL = {torch.bfloat16: 2.0 ** -8, torch.float32: 80 * 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def dev():
    return torch.device("cuda", 0)


def case(B, S, n_h, dn, dr, dtype, axes=1, seed=0, far=5000):
    g = torch.Generator(device=dev()).manual_seed(seed)

    def normal(*s, std=1.0, mean=0.0):
        return (torch.randn(*s, generator=g, device=dev()) * std + mean).to(dtype)
    x = dict(q=normal(B, S, n_h, dn + dr), k=normal(B, S, dr, std=3.0), wq=normal(dn + dr, std=0.3, mean=1.0),
             wk=normal(dr, std=0.3, mean=1.0))
    z = dict(q=normal(B, S, n_h, dn + dr), k=normal(B, S, dr))
    pos = torch.randint(-far, far, (axes, B, S), generator=g, device=dev(), dtype=torch.int32)
    n = dr // 2
    sections = [n // axes] * (axes - 1)
    sections.append(n - sum(sections))
    return x, z, pos, sections


def want_of(x, z, pos, sections, eps, theta, interleaved):
    y = {k: v.double().cpu().requires_grad_(True) for k, v in x.items()}
    q, k = cref.norm_rope(y["q"], y["k"], pos.cpu(), y["wq"], y["wk"], eps, sections, theta, interleaved)
    ((q * z["q"].double().cpu()).sum() + (k * z["k"].double().cpu()).sum()).backward()
    w = dict(q=q.detach(), k_rope=k.detach(), dq=y["q"].grad, dk_rope=y["k"].grad, dw_q=y["wq"].grad, dw_k=y["wk"].grad)
    mag = {}
    for name, v, gr, wt in (("q", y["q"], z["q"], y["wq"]), ("k", y["k"], z["k"], y["wk"])):
        v, gr, wt = v.detach(), gr.double().cpu(), wt.detach()
        r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
        # a turned gradient is as large as the gradient; the second term is no larger than the first
        mag["dq" if name == "q" else "dk_rope"] = 2 * float((r * gr.norm(dim=-1, keepdim=True) * wt.abs().max()).norm())
        mag["dw_" + name] = float((2 ** 0.5 * gr.abs().amax(-1, keepdim=True) * (v * r).abs()).flatten(0, -2).sum(0).norm())
    return w, mag


def check(got, want, mag, dtype):
    for k, a in got.items():
        r = want[k]
        # the rounding is of the result, the arithmetic's error of the uncancelled size
        bound = (2.0 ** -8 * float(r.norm()) if dtype == torch.bfloat16 else 0.0) + TOL[torch.float32] * max(
            float(r.norm()), mag.get(k, 0.0))
        err = float((a.double().cpu() - r).norm())
        assert err <= bound, (k, err, bound)


SHAPES = [(1, 1, 1, 0, 2), (1, 1, 16, 128, 64), (2, 77, 3, 32, 16), (1, 300, 5, 128, 64), (3, 33, 2, 40, 24),
          (1, 50, 3, 7, 10), (2, 9, 2, 0, 64), (1, 40, 2, 190, 66), (1, 21, 3, 192, 64), (1, 19, 2, 448, 64),
          (1, 11, 2, 960, 64), (1, 7, 2, 768, 256), (1, 700, 1, 128, 64), (1, 5, 70, 128, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, interleaved, dtype):
    axes = 1 if shape[4] < 6 else 3
    x, z, pos, sections = case(*shape, dtype, axes)
    kw = dict(eps=1e-6, sections=sections, theta=5e5, interleaved=interleaved)
    q, k = laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    g = laga.norm_rope_bwd(z["q"], z["k"], x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    want, mag = want_of(x, z, pos, sections, 1e-6, 5e5, interleaved)
    check(dict(q=q, k_rope=k, **g), want, mag, dtype)
    # each alone: the sums' order may be another
    q1, none = laga.norm_rope(x["q"], None, pos, x["wq"], **kw)
    none2, k1 = laga.norm_rope(None, x["k"], pos, None, x["wk"], **kw)
    assert none is None and none2 is None
    check(dict(q=q1, k_rope=k1), want, mag, dtype)
    a = laga.norm_rope_bwd(z["q"], None, x["q"], None, pos, x["wq"], **kw)
    b = laga.norm_rope_bwd(None, z["k"], None, x["k"], pos, None, x["wk"], **kw)
    assert set(a) == {"dq", "dw_q"} and set(b) == {"dk_rope", "dw_k"}
    check({**a, **b}, want, mag, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [True, False])
def test_in_place_and_unaligned(interleaved, dtype):
    x, z, pos, sections = case(2, 37, 4, 128, 64, dtype)
    kw = dict(sections=sections, interleaved=interleaved)
    q, k = laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    g = laga.norm_rope_bwd(z["q"], z["k"], x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    for target in (z, x):  # the gradients may be written over those of the results, or over the rows
        xs, zs = {a: v.clone() for a, v in x.items()}, {a: v.clone() for a, v in z.items()}
        t = zs if target is z else xs
        h = laga.norm_rope_bwd(zs["q"], zs["k"], xs["q"], xs["k"], pos, x["wq"], x["wk"],
                               grads=dict(dq=t["q"], dk_rope=t["k"]), **kw)
        assert all(torch.equal(g[n], h[n]) for n in g)

    def shifted(v):
        t = torch.empty(v.numel() + 1, dtype=v.dtype, device=v.device)[1:].view(v.shape)
        return t.copy_(v)
    u, w = shifted(x["q"]), shifted(x["k"])
    want, mag = want_of(x, z, pos, sections, 1e-6, 1e4, interleaved)
    q2, k2 = laga.norm_rope(u, w, pos, shifted(x["wq"]), shifted(x["wk"]), **kw)
    h = laga.norm_rope_bwd(shifted(z["q"]), shifted(z["k"]), u, w, pos, x["wq"], x["wk"], **kw)
    check(dict(q=q2, k_rope=k2, **h), want, mag, dtype)
    qi, ki = laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], q_out=x["q"], k_out=x["k"], **kw)
    assert qi is x["q"] and torch.equal(qi, q) and torch.equal(ki, k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dn", [128, 31])
def test_rows_of_any_size(dtype, dn):
    """Rows whose squares leave fp32 at either end, of zeros, with an infinity or a NaN."""
    x, z, pos, sections = case(1, 16, 1, dn, 64, dtype)
    size = torch.tensor([2.0 ** e for e in range(-120, 120, 15)], device=dev())
    x["q"] = (x["q"].float() * size[:, None, None]).to(dtype)
    x["q"][0, 0] = 0
    kw = dict(eps=1e-12, sections=sections)
    q, k = laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    g = laga.norm_rope_bwd(z["q"], z["k"], x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    want, mag = want_of(x, z, pos, sections, 1e-12, 1e4, True)
    for t in range(16):  # row by row: their gradients' sizes differ by 2^200
        a, r = q[0, t].double().cpu(), want["q"][0, t]
        assert float((a - r).norm()) <= (2.0 ** -8 if dtype == torch.bfloat16 else TOL[dtype]) * float(r.norm()), t
        a, r = g["dq"][0, t].double().cpu(), want["dq"][0, t]
        rms = 1 / torch.sqrt((x["q"][0, t].double().cpu() ** 2).mean() + 1e-12)
        full = 2 * float(rms * z["q"][0, t].double().norm().cpu() * x["wq"].double().abs().max().cpu())
        # half of the type's smallest step counts where the gradient is that small
        floor = (2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -149) * (dn + 64) ** 0.5
        assert float((a - r).norm()) <= TOL[dtype] * max(full, float(r.norm())) + floor, t
    check({n: g[n] for n in ("dw_q", "dw_k", "dk_rope")}, want, mag, dtype)
    x["q"][0, 3, 0, 5] = float("inf")
    x["q"][0, 4, 0, 5] = float("nan")
    q2, _ = laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
    assert torch.isnan(q2[0, 3, 0, 5]) and torch.isnan(q2[0, 4]).all()
    keep = [t for t in range(16) if t not in (3, 4)]
    assert torch.equal(q2[0, keep], q[0, keep])


def test_gradients_by_differences():
    """Central differences of the operator itself in fp32: the step 2^-6 leaves its square, 2.4e-4, times the
    third derivative (some units) and 2^-24 / 2^-6 = 4e-6 of the sum's size; the sum is of 200 values around 1."""
    x, z, pos, sections = case(1, 4, 2, 9, 16, torch.float32, seed=3)
    kw = dict(sections=sections)
    g = laga.norm_rope_bwd(z["q"], z["k"], x["q"], x["k"], pos, x["wq"], x["wk"], **kw)

    def loss(y):
        q, k = laga.norm_rope(y["q"], y["k"], pos, y["wq"], y["wk"], **kw)
        return float((q.double() * z["q"].double()).sum() + (k.double() * z["k"].double()).sum())
    gen = torch.Generator(device=dev()).manual_seed(1)
    for name, grad in (("q", "dq"), ("k", "dk_rope"), ("wq", "dw_q"), ("wk", "dw_k")):
        d = torch.randn(x[name].shape, generator=gen, device=dev())
        d /= d.norm()
        h = 2.0 ** -6
        num = (loss({**x, name: x[name] + h * d}) - loss({**x, name: x[name] - h * d})) / (2 * h)
        assert abs(num - float((g[grad].double() * d.double()).sum())) <= 5e-3 * max(1.0, float(g[grad].norm())), name


def test_same_bits_and_int64_positions():
    x, z, pos, sections = case(2, 700, 9, 128, 64, torch.bfloat16, 3)
    kw = dict(sections=sections)
    g = [laga.norm_rope_bwd(z["q"], z["k"], x["q"], x["k"], p, x["wq"], x["wk"], **kw) for p in (pos, pos, pos.long())]
    for h in g[1:]:
        assert all(torch.equal(g[0][n], h[n]) for n in h)


def test_captured_and_on_another_stream():
    x, z, pos, sections = case(1, 200, 4, 128, 64, torch.bfloat16)
    kw = dict(sections=sections)
    ws = torch.empty(laga._norm_bwd_bytes(bytes(laga._rope_desc((1, 200, 4, 192), 64, tuple(sections), 1e4, True, False,
                                                                False, 1))), dtype=torch.uint8, device=dev())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            q, k = laga.norm_rope(x["q"], x["k"], pos, x["wq"], x["wk"], **kw)
            g = laga.norm_rope_bwd(z["q"], z["k"], x["q"], x["k"], pos, x["wq"], x["wk"], workspace=ws, **kw)
    x["q"].mul_(-3)
    pos.add_(11)
    ws.fill_(255)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    want, mag = want_of(x, z, pos, sections, 1e-6, 1e4, True)
    check(dict(q=q, k_rope=k, **g), want, mag, torch.bfloat16)


def test_of_nothing_and_refusals():
    x, z, pos, sections = case(1, 3, 2, 8, 8, torch.float32)
    q0, k0, p0 = x["q"][:, :0], x["k"][:, :0], pos[:, :, :0]
    q, k = laga.norm_rope(q0.contiguous(), k0.contiguous(), p0.contiguous(), x["wq"], x["wk"])
    assert q.shape == (1, 0, 2, 16) and k.shape == (1, 0, 8)
    g = laga.norm_rope_bwd(q, k, q, k, p0.contiguous(), x["wq"], x["wk"])
    assert not g["dw_q"].any() and not g["dw_k"].any()
    a = (x["q"], x["k"], pos, x["wq"], x["wk"])
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(laga.LagaError, match="eps"):
            laga.norm_rope(*a, eps=bad)
    with pytest.raises(ValueError, match="sections"):
        laga.norm_rope(x["q"], None, pos, x["wq"])
    with pytest.raises(ValueError, match="q_weight"):
        laga.norm_rope(x["q"], x["k"], pos, x["wq"][:4], x["wk"])
    with pytest.raises(ValueError, match="contiguous"):
        laga.norm_rope(x["q"].transpose(1, 2).contiguous().transpose(1, 2), *a[1:])
    with pytest.raises(TypeError):
        laga.norm_rope(x["q"], x["k"], pos, x["wq"].bfloat16(), x["wk"])
    with pytest.raises(ValueError):
        laga.norm_rope(None, None, pos, None)
    with pytest.raises(ValueError, match="k_weight"):
        laga.norm_rope(x["q"], None, pos, x["wq"], x["wk"], sections=[4])
    with pytest.raises(laga.LagaError, match="1024"):
        laga.norm_rope(torch.zeros(1, 1, 1, 1026, device=dev()), None, pos[:, :, :1].contiguous(),
                       torch.ones(1026, device=dev()), sections=[4])
    with pytest.raises(ValueError, match="workspace"):
        laga.norm_rope_bwd(z["q"], z["k"], *a, workspace=torch.empty(8, device=dev()))
