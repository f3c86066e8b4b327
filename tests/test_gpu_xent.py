"""Softmax cross entropy over the vocabulary without keeping the logits, and
its gradients, against 64-bit definitions.

Tolerances (U = 2^-24).  The bf16 products are exact and summed in fp32; a
tensor-core sum may truncate where it aligns its terms, so a logit is off by
at most e = 2 d U sum_i |x_i W_i|.
* lse: the largest e of the row; 2^-18 for a term's exponent (its rounding,
  at most 30 U, the one of ex2, 2^-22, and the sum's, under 64 U); 4 U |lse|
  for the reference and the logarithm.
* loss: another e, and the subtraction's rounding.
* d = (p - 1[target]) g: p is off by p (e + 2^-18 + 4 U |lse|), then half a
  step of bf16 on each d; dx and dW: those errors through the products' other
  operand, 2 n U of the sum of magnitudes for n terms, half a step of the
  output's type.
"""

import pytest
import torch

import plain64 as p64
from plain64 import U32

pytestmark = pytest.mark.gpu

skv = pytest.importorskip("sparse_key_value_b200")
BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    skv.load()
    assert skv.device_error() == 0
    yield
    assert skv.device_error() == 0


def _case(seed, T, V, d, std=2.0, ignored=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, W = rn(T, d).to(BF), (rn(V, d) * std * d ** -0.5).to(BF)
    t = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[torch.rand(T, generator=g, device="cuda") < ignored] = IGN
    return x, W, t, rn(T)


def _ref_forward(x, W, t):
    X, Wd = x.to(F64), W.to(F64)
    z = X @ Wd.t()
    e = (2 * x.shape[1] * U32) * (X.abs() @ Wd.abs().t())
    lse = torch.logsumexp(z, 1)
    rows = torch.nonzero((t >= 0) & (t < W.shape[0]))[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - z[rows, t[rows].long()]
    tol = e.amax(1) + 2.0 ** -18 + 4 * U32 * lse.abs()
    return z, e, lse, loss, tol


def _check(x, W, t, dloss, grad_dtypes=(F32, BF), fed_lse=None):
    T, V, d = x.shape[0], W.shape[0], x.shape[1]
    loss, lse = skv.linear_xent_forward(x, W, t, ignore_index=IGN)
    z, e, lse64, loss64, tol = _ref_forward(x, W, t)
    bad = (lse.to(F64) - lse64).abs() > tol
    assert not bad.any(), f"lse: {int(bad.sum())}, {(lse.to(F64) - lse64).abs().max()}"
    bad = (loss.to(F64) - loss64).abs() > tol + e.amax(1) + U32 * loss64.abs()
    assert not bad.any(), f"loss: {int(bad.sum())}"
    assert (loss[t == IGN] == 0).all()
    L = lse.to(F64)
    g = torch.where(t != IGN, dloss.to(F64), torch.zeros((), dtype=F64, device="cuda"))[:, None]
    p = torch.exp(z - L[:, None])
    D = p.clone()
    rows = torch.nonzero(t != IGN)[:, 0]
    D[rows, t[rows].long()] -= 1
    D *= g
    # the reference takes the kernel's lse, so only its use is rounded
    err = g.abs() * p * (e + 2.0 ** -18 + 4 * U32 * L.abs()[:, None]) + p64.half_step(BF) * D.abs()
    X, Wd = x.to(F64), W.to(F64)
    for gd in grad_dtypes:
        dx, dW = skv.linear_xent_backward(x, W, t, lse, dloss, ignore_index=IGN, grad_dtype=gd)
        for got, a, b, ea in ((dx, D, Wd, err), (dW, D.t(), X, err.t())):
            ref = a @ b
            bound = (ea + 2 * a.shape[1] * U32 * a.abs()) @ b.abs() + 1e-30
            if gd == BF:
                bound = bound + p64.half_step(BF) * ref.abs()
            over = (got.to(F64) - ref).abs() > bound
            assert not over.any(), f"{gd} {tuple(got.shape)}: {int(over.sum())} of {over.numel()}"
        assert (dx[t == IGN] == 0).all()
    return loss, lse


@pytest.mark.parametrize("T,V,d", [
    (1, 1, 8), (1, 300, 64), (3, 31, 72), (37, 1000, 136), (130, 257, 128), (256, 256, 64),
    (257, 513, 200), (300, 4100, 520), (1000, 333, 1024), (64, 20011, 256), (700, 5000, 2056)])
def test_matches_64_bits(T, V, d):
    _check(*_case(T + V + d, T, V, d))


def test_several_pieces_of_the_vocabulary():
    """T * V large enough that the backward cuts the vocabulary (about 65536 at most)."""
    _check(*_case(1, 4096, 70001, 64), grad_dtypes=(F32, BF))


def test_peaked_and_wide_logits():
    """Logits of hundreds: one term carries a row's sum, others underflow."""
    x, W, t, dl = _case(2, 200, 700, 64, std=60.0)
    _check(x, W, t, dl)
    z = x.float() @ W.float().t()
    best = z.argmax(1).to(torch.int32)
    loss, _ = skv.linear_xent_forward(x, W, best)
    assert (loss < 1e-3).float().mean() > 0.5


def test_all_ignored_and_ignored_rows_hold_anything():
    x, W, t, dl = _case(3, 65, 500, 64)
    t[:] = IGN
    loss, lse = skv.linear_xent_forward(x, W, t)
    assert (loss == 0).all() and torch.isfinite(lse).all()
    dx, dW = skv.linear_xent_backward(x, W, t, lse, dl)
    assert (dx == 0).all() and (dW == 0).all()
    # NaN in an ignored position's lse and dloss stays out of both gradients
    t[10:] = 7
    lse2, dl2 = lse.clone(), dl.clone()
    lse2[:10], dl2[:10] = float("nan"), float("inf")
    a = skv.linear_xent_backward(x, W, t, lse2, dl2)
    b = skv.linear_xent_backward(x, W, t, lse, dl)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.isfinite(a[0]).all()


def test_another_ignore_index_and_targets_out_of_range():
    x, W, t, dl = _case(4, 40, 90, 64, ignored=0.0)
    t[5], t[6], t[7] = 90, -1, 3
    loss, lse = skv.linear_xent_forward(x, W, t, ignore_index=3)
    assert skv.device_error() == 4  # 90 and -1 are no targets
    assert (loss[5:8] == 0).all() and (loss[:5] != 0).all()
    dx, dW = skv.linear_xent_backward(x, W, t, lse, dl, ignore_index=3)
    assert (dx[5:8] == 0).all() and (dx[8] != 0).any()
    assert skv.device_error() == 0


def test_non_finite_inputs_stay_in_their_rows():
    x, W, t, dl = _case(5, 300, 600, 64, ignored=0.0)
    x[17, 3] = float("nan")
    loss, lse = skv.linear_xent_forward(x, W, t)
    ok = torch.arange(300, device="cuda") != 17
    assert torch.isnan(lse[17]) and torch.isnan(loss[17])
    assert torch.isfinite(lse[ok]).all() and torch.isfinite(loss[ok]).all()
    dx, dW = skv.linear_xent_backward(x, W, t, lse, dl)
    assert torch.isnan(dx[17]).any() and torch.isfinite(dx[ok]).all()


def test_gradient_against_differences():
    """dx and dW against central differences of the 64-bit loss; the bf16
    rounding of d leaves at most 2^-8 of the sum of magnitudes."""
    x, W, t, dl = _case(6, 20, 50, 32)
    X, Wd = x.to(F64), W.to(F64)
    f = lambda a, b: float((_ref_forward(a, b, t)[3] * dl.to(F64)).sum())  # noqa: E731
    _, lse = skv.linear_xent_forward(x, W, t, ignore_index=IGN)
    dx, dW = skv.linear_xent_backward(x, W, t, lse, dl, ignore_index=IGN)
    h = 1e-6
    for i, j in ((0, 0), (7, 31), (19, 12)):
        E = torch.zeros_like(X)
        E[i, j] = h
        diff = (f(X + E, Wd) - f(X - E, Wd)) / (2 * h)
        assert abs(diff - float(dx[i, j])) < 2.0 ** -8 * 2 * float(dl[i].abs() * Wd.abs().max()) + 1e-6
    for i, j in ((0, 0), (int(t[t != IGN][0]), 5), (49, 31)):
        E = torch.zeros_like(Wd)
        E[i, j] = h
        diff = (f(X, Wd + E) - f(X, Wd - E)) / (2 * h)
        assert abs(diff - float(dW[i, j])) < 2.0 ** -8 * float((dl.abs() * X[:, j].abs()).sum()) + 1e-6


def test_empty_batch():
    x, W = torch.empty(0, 64, dtype=BF, device="cuda"), torch.randn(30, 64, device="cuda").to(BF)
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    loss, lse = skv.linear_xent_forward(x, W, t)
    assert loss.numel() == 0 and lse.numel() == 0
    dW = torch.full((30, 64), float("nan"), device="cuda")
    dx, _ = skv.linear_xent_backward(x, W, t, lse, lse, dW=dW)
    assert dx.shape == (0, 64) and (dW == 0).all()


def test_reproducible_captured_and_on_another_stream():
    x, W, t, dl = _case(7, 300, 9000, 128)

    def step():
        loss, lse = skv.linear_xent_forward(x, W, t, ignore_index=IGN)
        return (loss, lse, *skv.linear_xent_backward(x, W, t, lse, dl, ignore_index=IGN,
                                                     grad_dtype=BF))

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
    for a, b, c in zip(ref, other, kept):
        assert torch.equal(a, b) and torch.equal(a, c)
    t.copy_(t.flip(0))
    graph.replay()
    for a, b in zip(kept, step()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,V,d", [(65536, 150, 64), (65536, 70, 8), (40000, 200, 128),
                                   (30000, 650, 64), (5000, 4648, 64), (3001, 9000, 128)])
def test_many_tiles_a_pair_with_warps_out_of_step(T, V, d):
    """Pairs of SMs that go through many tiles, some of whose column warps have
    fewer columns than the others or none: those run ahead of the rest, and
    the join of the four must still take each tile's own maximum and sum."""
    x, W, t, _ = _case(T + V, T, V, d)
    loss, lse = skv.linear_xent_forward(x, W, t, ignore_index=IGN)
    for i in range(0, T, 8192):
        rows = slice(i, i + 8192)
        _, e, lse64, loss64, tol = _ref_forward(x[rows], W, t[rows])
        bad = (lse[rows].to(F64) - lse64).abs() > tol
        assert not bad.any(), f"lse: {int(bad.sum())}"
        bad = (loss[rows].to(F64) - loss64).abs() > tol + e.amax(1) + U32 * loss64.abs()
        assert not bad.any(), f"loss: {int(bad.sum())}"
    for _ in range(20):
        again = skv.linear_xent_forward(x, W, t, ignore_index=IGN)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
