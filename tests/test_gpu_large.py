"""The training operators over tensors of more than 2^31 elements: the ends of
the long tensors against 64-bit forms or against the same call on the end alone."""

import pytest
import torch

import sparse_key_value_b200 as skv

pytestmark = pytest.mark.gpu

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
ROWS, D = 270_000, 8192          # 2.2e9 elements
U16 = 2.0 ** -8


@pytest.fixture(autouse=True)
def _room():
    torch.cuda.empty_cache()
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def _rn(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(shape, dtype=BF, device="cuda")
    for part in out.split(16384):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * scale)
    return out


ENDS = (slice(0, 3), slice(131_071, 131_074), slice(ROWS - 5, ROWS))


def _same(a, b):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_act8_and_norm_forward():
    x, r = _rn(ROWS, D, seed=1), _rn(ROWS, D, seed=2)
    q, s = skv.act8_store(x)
    y = skv.act8_load(q, s)
    for e in ENDS:
        qe, se = skv.act8_store(x[e].clone())
        _same(q[e], qe)
        _same(s[e], se)
        _same(y[e], skv.act8_load(qe, se))
    del q, s, y
    f = skv.add_rmsnorm_forward(x, None, r, fmt="e4m3")
    for e in ENDS:
        g = skv.add_rmsnorm_forward(x[e].clone(), None, r[e].clone(), fmt="e4m3")
        for k in ("sum", "y", "rstd", "q8", "scales"):
            _same(f[k][e], g[k])


def test_norm_backward():
    h, dy = _rn(ROWS, D, seed=3), _rn(ROWS, D, seed=4)
    w = _rn(D, seed=5)
    rstd = torch.cat([(p.float().square().mean(1) + 1e-6).rsqrt() for p in h.split(8192)])
    out = skv.add_rmsnorm_backward(dy, h, w, rstd)
    for e in ENDS:
        n = h[e].double() * rstd[e].double()[:, None]
        g = dy[e].double() * w.double()
        ref = rstd[e].double()[:, None] * (g - n * (g * n).mean(1, keepdim=True))
        tol = U16 * ref.abs() + 1e-5 * ref.abs().max()
        assert ((out["dx"][e].double() - ref).abs() <= tol).all()
    dw, mag = torch.zeros(D, dtype=F64, device="cuda"), torch.zeros(D, dtype=F64, device="cuda")
    for i in range(0, ROWS, 8192):
        p = dy[i:i + 8192].double() * (h[i:i + 8192].double() * rstd[i:i + 8192].double()[:, None])
        dw += p.sum(0)
        mag += p.abs().sum(0)
    # a column's terms pass at most ROWS / 148 additions in a team, 4 and 148 after
    assert ((out["dweight"].double() - dw).abs() <= (ROWS / 148 + 160) * 2.0 ** -24 * mag).all()


def test_embedding():
    E = _rn(ROWS, D, seed=6)
    ids = torch.tensor([0, ROWS - 1, 262_144, ROWS - 1, 5, ROWS - 2, 131_072], device="cuda",
                       dtype=torch.int32)
    _same(skv.embedding_forward(E, ids, scale=2.0), E[ids.long()] * 2)
    del E
    for T in (7, 4000):  # both ways of sorting with their own zeroing
        many = ids.repeat(-(-T // 7))[:T].contiguous()
        dout = _rn(T, D, seed=T)
        grad = skv.embedding_backward(dout, many, ROWS)
        used = torch.zeros(ROWS, dtype=torch.bool, device="cuda")
        used[ids.long()] = True
        for i in ids.unique().tolist():
            rows = dout[many == i].double()
            tol = (len(rows) + 3) * 2.0 ** -24 * rows.abs().sum(0)
            assert ((grad[i].double() - rows.sum(0)).abs() <= tol).all(), i
        for i in range(0, ROWS, 30_000):
            part = grad[i:i + 30_000]
            assert not part[~used[i:i + 30_000]].any()
        del grad


def test_loss():
    T, V = 40, ROWS
    x, W = _rn(T, D, seed=7), _rn(V, D, seed=8, scale=D ** -0.5)
    targets = torch.randint(0, V, (T,), device="cuda", dtype=torch.int32)
    targets[:4] = torch.tensor([V - 1, 0, 262_144, V - 2])
    loss, lse = skv.linear_xent_forward(x, W, targets)
    z = torch.cat([x.double() @ p.double().t() for p in W.split(8192)], 1)
    ref = torch.logsumexp(z, 1)
    pick = z[torch.arange(T), targets.long()]
    assert ((lse.double() - ref).abs() <= 1e-5 * (1 + ref.abs())).all()
    assert ((loss.double() - (ref - pick)).abs() <= 2e-5 * (1 + ref.abs() + pick.abs())).all()
    dl = torch.rand(T, device="cuda")
    dx, dW = skv.linear_xent_backward(x, W, targets, lse, dl)
    d = torch.softmax(z, 1)
    d[torch.arange(T), targets.long()] -= 1
    d *= dl.double()[:, None]
    rows = torch.cat([targets.long(), torch.arange(V - 8, V, device="cuda"),
                      torch.arange(262_140, 262_150, device="cuda")])
    # each d is off by half a bf16 step (eps / 2 = 2^-8 of it), the sums by fp32
    # roundings of T terms
    mag = d[:, rows].abs().t() @ x.double().abs()
    err = (dW[rows].double() - d[:, rows].t() @ x.double()).abs()
    assert (err <= (U16 * 1.02 + 1e-4) * mag + 1e-12).all()
    ref, mag = torch.zeros(T, D, dtype=F64, device="cuda"), torch.zeros(T, D, dtype=F64, device="cuda")
    for i in range(0, V, 8192):
        w = W[i:i + 8192].double()
        ref += d[:, i:i + 8192] @ w
        mag += d[:, i:i + 8192].abs() @ w.abs()
    assert ((dx.double() - ref).abs() <= (U16 * 1.02 + 1e-3) * mag).all()


def test_memplus_backward():
    T, dm, dv = 2_150_000, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(9)
    W1, W2 = _rn(dm, dv, seed=10, scale=dm ** -0.5), _rn(dv, dm, seed=11, scale=dv ** -0.5)
    x8 = torch.randint(-127, 128, (T, dm), generator=g, device="cuda", dtype=torch.int8)
    y8 = torch.randint(-127, 128, (T, dv), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.full((T, dm // 128), 2.0 ** -6, device="cuda")
    ys = torch.full((T, dv // 128), 2.0 ** -6, device="cuda")
    dout = _rn(T, dm, seed=12)
    out = skv.memplus_backward_act8(x8, xs, W1, W2, y8, ys, dout, grad_dtype=BF)
    for e in (slice(0, 256), slice(T - T % 256 - 256, T)):
        part = skv.memplus_backward_act8(x8[e], xs[e], W1, W2, y8[e], ys[e], dout[e], grad_dtype=BF)
        _same(out["dy"][e], part["dy"])
        _same(out["dx"][e], part["dx"])


def test_memplus_weight_gradients_over_many_tokens():
    """dW1 and dW2, whose sums run over the tokens, at 8-bit activations of more
    than 2^31 elements.  Every factor is positive and the last 100 tokens weigh
    about as much as all others, so nothing cancels and no token may be lost.

    Relative to the sums: da and z, half a bf16 step (2^-8) and their fp32
    arithmetic: a and dz sums of 512 positive terms (2 * 512 U = 6e-5 each, U =
    2^-24), the gate and its slope at a > 0 under three times that, the rest
    some 32 U: under 1e-3 in all; the sums over T tokens, 16 products at a time
    and at worst in one slice, T / 16 additions of 2 U, and 64 for the slices."""
    T, dm, dv = 2_150_000, 512, 1024
    g = torch.Generator(device="cuda").manual_seed(21)
    W1 = _rn(dm, dv, seed=22, scale=2.0 / dm).abs()
    W2 = _rn(dv, dm, seed=23, scale=2.0 / dm).abs()
    x8 = torch.randint(1, 128, (T, dm), generator=g, device="cuda", dtype=torch.int8)
    y8 = torch.randint(1, 128, (T, dv), generator=g, device="cuda", dtype=torch.int8)
    xs = torch.full((T, dm // 128), 2.0 ** -6, device="cuda")
    ys = torch.full((T, dv // 128), 2.0 ** -6, device="cuda")
    dout = _rn(T, dm, seed=24).abs_()
    dout[-100:] *= 2.0 ** 14
    out = skv.memplus_backward_act8(x8, xs, W1, W2, y8, ys, dout)
    # a quarter of the columns of each: the 64-bit products then take about a second
    cv, cm = torch.arange(0, dv, 4, device="cuda"), torch.arange(0, dm, 4, device="cuda")
    w1, w2 = W1[:, cv].double(), W2[cv].double()
    dw1 = torch.zeros(dm, len(cv), dtype=F64, device="cuda")
    dw2 = torch.zeros(len(cv), len(cm), dtype=F64, device="cuda")
    for i in range(0, T, 50_000):
        e = slice(i, i + 50_000)
        x, y = x8[e].double() * 2.0 ** -6, y8[e][:, cv].double() * 2.0 ** -6
        do = dout[e].double()
        a, dz = x @ w1, do @ w2.t()
        s = torch.sigmoid(a)
        dw1 += x.t() @ (dz * y * s * (1 + a * (1 - s)))
        dw2 += (y * a * s).t() @ do[:, cm]
    rel = U16 + 1e-3 + 2 * (T / 16 + 64) * 2.0 ** -24
    assert ((out["dW1"][:, cv].double() - dw1).abs() <= rel * dw1).all()
    assert ((out["dW2"][cv][:, cm].double() - dw2).abs() <= rel * dw2).all()
