"""The Memory+ backward from activations kept in 8 bits, against 64-bit
definitions over the values that the 8 bits stand for; and a training step of
a small language model through the operators around a memory layer.

Tolerances (U = 2^-24), with the magnitudes of the case's own sums:
* a = x W1 and dz = dout W2^T: e_a, e_z = 2 K U of the sum of magnitudes.
* the gate g = a s(a): |g'| <= 1.1 carries e_a, its own arithmetic (the fast
  exponential, the quotient, two products) 16 U (1 + |a|) of |a|; its slope
  |g''| <= 0.5, 16 U (1 + |a|)^2.
* dy, da, z: those errors through the products, half a step of bf16 each.
* dx, dW1, dW2: the operands' errors through the other operand, 2 n U of the
  sum of magnitudes for n terms, half a step of the output's type.
"""

import pytest
import torch

import plain64 as p64
from plain64 import U32

pytestmark = pytest.mark.gpu

skv = pytest.importorskip("sparse_key_value_b200")
from sparse_key_value_b200.inputs import WORKLOADS, make_inputs  # noqa: E402

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    skv.load()
    assert skv.device_error() == 0
    yield
    assert skv.device_error() == 0


def _case(seed, T, dm, dv, fmt, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rn(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(BF)

    return (*skv.act8_store(rn(T, dm, std=std), fmt), rn(dm, dv, std=dm ** -0.5),
            rn(dv, dm, std=dv ** -0.5), *skv.act8_store(rn(T, dv, std=0.1), fmt), rn(T, dm))


def _within(got, ref, tol, what):
    err = (got.to(F64) - ref).abs()
    assert torch.isfinite(got).all(), what
    bad = err > tol + 1e-30
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {(err / (tol + 1e-30)).max():.3g} of tol"


def _check(x8, xs, W1, W2, y8, ys, dout, grad_dtypes=(F32, BF)):
    T, dm, dv = x8.shape[0], x8.shape[1], y8.shape[1]
    x, y = skv.act8_load(x8, xs, dtype=F32).to(F64), skv.act8_load(y8, ys, dtype=F32).to(F64)
    w1, w2, do = W1.to(F64), W2.to(F64), dout.to(F64)
    a, dz = x @ w1, do @ w2.t()
    ea = 2 * dm * U32 * (x.abs() @ w1.abs())
    ez = 2 * dm * U32 * (do.abs() @ w2.abs().t())
    s = torch.sigmoid(a)
    g, slope = a * s, s * (1 + a * (1 - s))
    eg = 1.1 * ea + 16 * U32 * (1 + a.abs()) * a.abs()
    es = 0.5 * ea + 16 * U32 * (1 + a.abs()) ** 2
    h = p64.half_step(BF)
    dy, da, z = dz * g, dz * y * slope, y * g
    e_dy = dz.abs() * eg + g.abs() * ez + eg * ez + h * dy.abs()
    e_da = y.abs() * (slope.abs() * ez + dz.abs() * es + es * ez) + h * da.abs() + 4 * U32 * da.abs()
    e_z = y.abs() * eg + h * z.abs() + 4 * U32 * z.abs()
    out = None
    for gd in grad_dtypes:
        out = skv.memplus_backward_act8(x8, xs, W1, W2, y8, ys, dout, grad_dtype=gd)
        _within(out["dy"], dy, e_dy + 4 * U32 * dy.abs(), "dy")
        for name, A, B, eA in (("dx", da, w1.t(), e_da), ("dW1", da.t(), x, e_da.t()),
                               ("dW2", z.t(), do, e_z.t())):
            ref = A @ B
            tol = (eA + 2 * A.shape[1] * U32 * A.abs()) @ B.abs()
            if name == "dW1":
                ref, tol = ref.t(), tol.t()
            if gd == BF:
                tol = tol + h * (ref.abs() + tol)
            _within(out[name], ref, tol, f"{name} {gd}")
    return out


@pytest.mark.parametrize("T,dm,dv", [
    (1, 8, 8), (7, 72, 40), (40, 64, 136), (130, 32, 48), (300, 256, 128), (257, 264, 520),
    (1000, 640, 520), (4100, 256, 256), (2000, 1024, 1032)])
def test_matches_64_bits(T, dm, dv):
    for fmt in ("e4m3", "int8"):
        _check(*_case(T + dm + dv, T, dm, dv, fmt))


def test_large_gate_arguments():
    _check(*_case(5, 200, 128, 256, "int8", std=30.0))


def test_agrees_with_the_16_bit_backward():
    """Fed with the same values in bf16 (8-bit values are exact there), the
    library's 16-bit backward gives the same gradients to bf16 rounding."""
    x8, xs, W1, W2, y8, ys, dout = _case(6, 500, 256, 384, "int8")
    a = skv.memplus_backward_act8(x8, xs, W1, W2, y8, ys, dout)
    b = skv.memplus_backward(skv.act8_load(x8, xs), W1, W2, skv.act8_load(y8, ys), dout)
    for k in a:
        ref = b[k].double()
        assert float((a[k].double() - ref).norm()) < 2.0 ** -8 * float(ref.norm()), k


def test_non_finite_group_reads_back_as_nan():
    """A NaN that was stored shows in the gradients of its row, not as a number."""
    x8, xs, W1, W2, y8, ys, dout = _case(7, 70, 64, 128, "int8")
    xs[13] = float("nan")
    out = skv.memplus_backward_act8(x8, xs, W1, W2, y8, ys, dout)
    rows = torch.arange(70, device="cuda") != 13
    assert torch.isnan(out["dy"][13]).all() and torch.isfinite(out["dy"][rows]).all()
    assert torch.isnan(out["dx"][13]).all() and torch.isfinite(out["dx"][rows]).all()
    assert torch.isnan(out["dW1"]).all()


def test_empty_batch():
    x8, xs, W1, W2, y8, ys, dout = _case(8, 4, 64, 128, "e4m3")
    out = skv.memplus_backward_act8(x8[:0], xs[:0], W1, W2, y8[:0], ys[:0], dout[:0])
    assert out["dx"].shape == (0, 64) and (out["dW1"] == 0).all() and (out["dW2"] == 0).all()


def test_reproducible_captured_and_on_another_stream():
    case = _case(9, 700, 256, 264, "int8")
    step = lambda: list(skv.memplus_backward_act8(*case, grad_dtype=BF).values())  # noqa: E731
    ref = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for k in kept:
        k.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, other, kept):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_binding_refuses_mismatched_arguments():
    x8, xs, W1, W2, y8, ys, dout = _case(10, 8, 64, 128, "int8")
    e8, es = skv.act8_store(skv.act8_load(y8, ys), "e4m3")
    with pytest.raises(ValueError):
        skv.memplus_backward_act8(x8, xs, W1, W2, e8, es, dout)        # two formats
    with pytest.raises(ValueError):
        skv.memplus_backward_act8(x8, xs, W2, W1, y8, ys, dout)        # shapes
    with pytest.raises(TypeError):
        skv.memplus_backward_act8(x8, xs, W1.float(), W2, y8, ys, dout)
    with pytest.raises(TypeError):
        skv.memplus_backward_act8(dout, xs, W1, W2, y8, ys, dout)      # not 8 bits
    with pytest.raises(ValueError):
        skv.memplus_backward_act8(x8, xs.t(), W1, W2, y8, ys, dout)


# ------------------------------------------------------- a training step --

def _lm_step(p, ids, targets, dloss, w):
    """Forward and backward of: embedding -> norm -> memory layer (query
    projection, product-key lookup, Memory+ gate) -> residual + norm -> loss
    over the tied table.  Returns (loss, activations, gradients)."""
    T = ids.numel()
    scale = w.d_model ** 0.5
    h0 = skv.embedding_forward(p["E"], ids, scale=scale, pad_id=-100)
    n1 = skv.add_rmsnorm_forward(h0, p["g1"], fmt="int8")  # rows without a token stay zero
    x = n1["y"]
    q = skv.qproj_forward(x, p["Wq"]).view(T, w.H, 2, w.d_half)
    y = torch.empty(T, w.d_v, dtype=BF, device="cuda")
    m, idx, wts = skv.pkm_forward(q, p["K"], p["V"], w.k, x=x, W1=p["W1"], W2=p["W2"], y_out=y)
    y8, ys = skv.act8_store(y, "int8")
    n2 = skv.add_rmsnorm_forward(m, p["g2"], residual=h0)
    loss, lse = skv.linear_xent_forward(n2["y"], p["E"], targets)

    gr = {}
    dn2, gr["E"] = skv.linear_xent_backward(n2["y"], p["E"], targets, lse, dloss)
    b2 = skv.add_rmsnorm_backward(dn2, n2["sum"], p["g2"], n2["rstd"])
    gr["g2"] = b2["dweight"]
    mp = skv.memplus_backward_act8(n1["q8"], n1["scales"], p["W1"], p["W2"], y8, ys, b2["dx"])
    gr["W1"], gr["W2"] = mp["dW1"], mp["dW2"]
    lk = skv.pkm_backward(q, p["K"], p["V"], idx, wts, mp["dy"])
    gr["K"], gr["rows"], gr["V"] = lk["dsubkeys"], lk["uniq_rows"], lk["grad_rows"]
    qp = skv.qproj_backward(x, p["Wq"], lk["dquery"].view(T, -1), dx=mp["dx"])
    gr["Wq"] = qp["dWq"]
    b1 = skv.add_rmsnorm_backward(qp["dx"], n1["sum"], p["g1"], n1["rstd"], dsum=b2["dx"])
    gr["g1"] = b1["dweight"]
    skv.embedding_backward(b1["dx"], ids, p["E"].shape[0], scale=scale, pad_id=-100,
                           grad=gr["E"], accumulate=True)
    return loss, dict(idx=idx), gr


def test_language_model_training_step():
    """The step's loss and every gradient against 64-bit automatic
    differentiation of the same model with the selection held fixed.

    Along any path the values pass at most 16 roundings to bf16 (2^-8 each,
    relative to their norm) and the two int8 copies (half a step of 1/64 of a
    group's maximum, under 2^-5 of the norm of a normal group); to first
    order the gradients are off by at most 16 / 256 + 1 / 32 < 0.1 of their
    norm.  The loss sees the forward's roundings only."""
    V, T = 600, 384
    w = WORKLOADS["memplus"].scaled(name="lm", T=T, H=2, d_half=256, n_sub=256, k=8, d_v=128,
                                    d_model=128)
    inp = make_inputs(w, "cuda")
    g = torch.Generator(device="cuda").manual_seed(12)

    def rn(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(BF)

    p = dict(E=rn(V, 128, std=128 ** -0.5), g1=1 + rn(128, std=0.1), g2=1 + rn(128, std=0.1),
             Wq=rn(128, w.H * 2 * w.d_half, std=128 ** -0.5), K=inp["subkeys"],
             V=(inp["values"].float() * 50).to(BF), W1=inp["W1"], W2=inp["W2"])
    text = torch.randint(0, V, (T + 1,), generator=g, device="cuda", dtype=torch.int32)
    text[-20:] = -100                       # the end is padding: no token, no target
    ids, targets = text[:-1], text[1:]      # slices of one list, the second 4-byte aligned
    n = int((targets != -100).sum())
    dloss = torch.full((T,), 1.0 / n, device="cuda")
    loss, act, gr = _lm_step(p, ids, targets, dloss, w)

    r = {k: v.to(F64).requires_grad_() for k, v in p.items() if k != "V"}
    rows = torch.unique(act["idx"])
    r["V"] = p["V"][rows.long()].to(F64).requires_grad_()
    pos = torch.searchsorted(rows, act["idx"].long())
    norm = lambda h, wt: h * (h.square().mean(1, keepdim=True) + 1e-6) ** -0.5 * wt  # noqa: E731
    h0 = r["E"][ids.long().clamp(min=0)] * 128 ** 0.5 * (ids >= 0)[:, None]
    x = norm(h0, r["g1"])
    q = (x @ r["Wq"]).view(T, w.H, 2, w.d_half)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True).clamp(min=1e-12)  # noqa: E731
    half = w.d_half ** 0.5 * torch.einsum("thcd,hcnd->thcn", unit(q), unit(r["K"]))
    i = act["idx"].long()
    S = half[:, :, 0].gather(2, i // w.n_sub) + half[:, :, 1].gather(2, i % w.n_sub)
    y = torch.einsum("thk,thkd->td", torch.softmax(S, -1), r["V"][pos])
    gate = x @ r["W1"]
    m = (y * gate * torch.sigmoid(gate)) @ r["W2"]
    z = norm(m + h0, r["g2"]) @ r["E"].t()
    keep = torch.nonzero(targets != -100)[:, 0]
    each = torch.logsumexp(z, 1)[keep] - z[keep, targets[keep].long()]
    (each.sum() / n).backward()
    err = (loss[keep].double() - each.detach()).norm() / each.detach().norm()
    assert float(err) < 16 / 256, float(err)
    assert torch.equal(gr["rows"].long(), rows.long())
    for k in r:
        ref = r[k].grad
        rel = float((gr[k].double() - ref).norm() / ref.norm())
        assert rel < 0.1, f"{k}: {rel:.3f} of the gradient's norm"
