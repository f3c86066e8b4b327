"""Residual addition + root-mean-square norm with its 16- and 8-bit outputs
and its backward, and activations in 8 bits, against 64-bit definitions.

Tolerances, from the kernels' arithmetic (U = 2^-24, one fp32 rounding):
* h: the same rounding of the same sum, so equal.
* rstd: a lane adds at most 32 squares, then 5 + 16 partial sums, then the
  division, the addition of eps, the root and the quotient; the root halves
  the sum's relative error: at most (32 + 21) / 2 + 4 < 32 U.
* y: two more products and the store's rounding: 34 U + half a step.
* 8-bit values: half a step of the format around a y that is 34 U off.
* dx: rstd (g - n m): n is 1 U off, g 1 U, the mean m a sum like the norm's
  (53 + 4 U of the mean magnitude), then three roundings: at most 64 U of
  rstd (|g| + |n| mean|g n|), one U for adding dsum, half a step.
* dweight: a sum over T rows of products 2 U off: (T + 64) U of the sum of
  magnitudes.
"""

import ctypes
import math

import pytest
import torch

import plain64 as p64
from plain64 import U32

pytestmark = pytest.mark.gpu

skv = pytest.importorskip("sparse_key_value_b200")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    skv.load()
    yield
    assert skv.device_error() == 0


def _rn(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _within(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    assert torch.isfinite(err).all(), what
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {(err / tol).max():.3g} of tol"


# widths: one unit, part of a warp, a short last group, one warp, two, a ragged
# two, four, eight and sixteen warps a row
WIDTHS = [8, 72, 136, 520, 1000, 1024, 2048, 2056, 4096, 8192, 16384]


def _check_fwd(x, r, w, eps, fmt):
    out = skv.add_rmsnorm_forward(x.cuda(), None if w is None else w.cuda(),
                                  residual=None if r is None else r.cuda(), eps=eps, fmt=fmt)
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert torch.equal(out["sum"].cpu(), h)
    y, rstd = p64.norm(h, w, eps)
    _within(out["rstd"], rstd, 32 * U32 * rstd, "rstd")
    _within(out["y"], y, (34 * U32 + p64.half_step(x.dtype)) * y.abs() + 1e-40, "y")
    if fmt is None:
        assert out["q8"] is None and out["scales"] is None
        return
    amax = p64.group_amax(y)
    s = out["scales"].double().cpu()
    assert torch.equal(torch.log2(s), torch.log2(s).round())
    assert (amax <= s * p64.Q8_MAX[fmt] * (1 + 34 * U32)).all()
    assert ((amax > s / 2 * p64.Q8_MAX[fmt] * (1 - 34 * U32)) | (s == 2.0 ** -100)).all()
    v = p64.q8_values(out["q8"].cpu(), out["scales"].cpu())
    _within(v, y, p64.q8_half_step(y, out["scales"].cpu(), fmt) + 34 * U32 * y.abs(), "y8")


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_forward(d, dtype):
    g = torch.Generator().manual_seed(d)
    for T, res, weight, fmt in ((1, True, True, "e4m3"), (13, True, True, "int8"),
                                (9, False, True, None), (5, True, False, "e4m3")):
        x = _rn(g, T, d, dtype=dtype)
        r = _rn(g, T, d, std=2.0, dtype=dtype) if res else None
        w = (1 + _rn(g, d, std=0.1, dtype=F32)).to(dtype) if weight else None
        _check_fwd(x, r, w, 1e-6, fmt)


def test_forward_many_rows():
    g = torch.Generator().manual_seed(3)
    _check_fwd(_rn(g, 4099, 264), _rn(g, 4099, 264), _rn(g, 264), 1e-5, "e4m3")


def test_forward_wide_range_rows():
    """Rows from 1e-18 to 1e15: eps dominates the smallest, every scale holds."""
    g = torch.Generator().manual_seed(4)
    x = _rn(g, 12, 512, dtype=F32) * 10.0 ** torch.linspace(-18, 15, 12)[:, None]
    w = (10.0 ** torch.linspace(-6, 6, 512)).to(F32)
    for fmt in ("e4m3", "int8"):
        _check_fwd(x, None, w, 1e-6, fmt)


def test_zero_rows_and_non_finite_groups():
    x = torch.ones(4, 304)
    x[1] = 0
    x[2, 130] = float("inf")   # the whole row's rms is infinite
    x[3, 5] = float("nan")
    for fmt in ("e4m3", "int8"):
        out = skv.add_rmsnorm_forward(x.cuda(), fmt=fmt)
        v = skv.act8_load(out["q8"], out["scales"]).cpu()
        assert torch.equal(v[1], torch.zeros(304, dtype=BF))
        assert (out["y"][1] == 0).all() and torch.isfinite(v[0]).all()
        assert torch.isnan(v[3]).all() and torch.isnan(out["y"][3]).all()
        assert torch.isnan(v[2, 128:256]).all()  # the group that holds inf / inf


def test_in_place_sum_and_empty():
    g = torch.Generator().manual_seed(6)
    x, r = _rn(g, 33, 1000).cuda(), _rn(g, 33, 1000).cuda()
    ref = skv.add_rmsnorm_forward(x, residual=r, fmt="int8")
    for target in ("x", "r"):
        x2, r2 = x.clone(), r.clone()
        got = skv.add_rmsnorm_forward(x2, residual=r2, fmt="int8",
                                      sum_out=x2 if target == "x" else r2)
        assert got["sum"] is (x2 if target == "x" else r2)
        for k in ("sum", "y", "rstd", "q8", "scales"):
            assert torch.equal(got[k].view(torch.uint8), ref[k].view(torch.uint8)), k
    out = skv.add_rmsnorm_forward(x[:0], residual=r[:0], fmt="e4m3")
    assert out["y"].shape == (0, 1000) and out["scales"].shape == (0, 8)


def _check_bwd(T, d, dtype, dy_dtype, res, weight, fmt, seed):
    g = torch.Generator().manual_seed(seed)
    h = _rn(g, T, d, std=1.5, dtype=dtype)
    w = (1 + _rn(g, d, std=0.2, dtype=F32)).to(dtype) if weight else None
    dy = _rn(g, T, d, dtype=dy_dtype)
    dsum = _rn(g, T, d, dtype=dtype) if res else None
    hd, sc = h.cuda(), None
    if fmt is not None:
        hd, sc = skv.act8_store(h.cuda(), fmt)
        h = skv.act8_load(hd, sc, dtype=F32).cpu()
    rstd = p64.norm(h, None, 1e-6)[1].float()
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    out = skv.add_rmsnorm_backward(dy.cuda(), hd, c(w), rstd.cuda(), dsum=c(dsum), scales=sc)
    h64 = h.double()
    r64, n = rstd.double()[:, None], h64 * rstd.double()[:, None]
    gw = dy.double() * (1.0 if w is None else w.double())
    m = (gw * n).mean(1, keepdim=True)
    dx = r64 * (gw - n * m)
    mag = r64 * (gw.abs() + n.abs() * (gw * n).abs().mean(1, keepdim=True))
    if dsum is not None:
        dx = dx + dsum.double()
    tol = 64 * U32 * mag + U32 * dx.abs()
    if out["dx"].dtype == BF:
        tol = tol + p64.half_step(BF) * dx.abs()
    _within(out["dx"], dx, tol, "dx")
    _within(out["dweight"], (dy.double() * n).sum(0),
            (T + 64) * U32 * (dy.double() * n).abs().sum(0) + 1e-30, "dweight")
    return out


@pytest.mark.parametrize("d", WIDTHS)
def test_backward(d):
    _check_bwd(1, d, BF, BF, True, True, None, d)
    _check_bwd(21, d, BF, F32, False, True, None, d + 1)
    _check_bwd(10, d, F32, F32, True, False, None, d + 2)
    _check_bwd(7, d, F32, BF, True, True, "e4m3", d + 3)
    _check_bwd(12, d, BF, BF, False, True, "int8", d + 4)


def test_backward_many_rows():
    """More rows than blocks x rows in flight: every block makes rounds."""
    for T, d in ((5000, 136), (1301, 2048)):
        _check_bwd(T, d, BF, BF, True, True, None, T)


@pytest.mark.parametrize("T,d,dtype,dy_dtype,res,weight", [
    (11900, 264, BF, BF, True, True), (11841, 512, BF, F32, False, True),
    (5921, 1000, BF, BF, True, False), (2959, 2048, BF, BF, True, True),
    (2963, 2048, BF, BF, False, True), (1300, 4096, BF, BF, True, True),
    (600, 8192, BF, BF, True, True), (11845, 256 + 8, F32, F32, True, True),
    (3001, 1024, F32, BF, True, True), (1201, 2040, F32, F32, False, True),
    (700, 4096, F32, F32, True, True)])
def test_backward_of_long_batches(T, d, dtype, dy_dtype, res, weight):
    """Batches whose rows come through shared memory, and one just below; ends
    that leave some of a block's teams without a row."""
    a = _check_bwd(T, d, dtype, dy_dtype, res, weight, None, T + d)
    b = _check_bwd(T, d, dtype, dy_dtype, res, weight, None, T + d)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])


@pytest.mark.parametrize("T,d,dtype,dy_dtype,fmt", [
    (9500, 272, BF, BF, "int8"), (9475, 512, BF, F32, "e4m3"), (4750, 1000, BF, BF, "int8"),
    (4740, 1008, F32, F32, "e4m3"), (2371, 2048, BF, BF, "int8"), (2371, 2040, BF, BF, "e4m3"),
    (1190, 4096, F32, BF, "int8"), (595, 8192, BF, BF, "e4m3")])
def test_backward_of_long_batches_from_8_bits(T, d, dtype, dy_dtype, fmt):
    """8-bit rows through shared memory where they are multiples of 16 bytes."""
    a = _check_bwd(T, d, dtype, dy_dtype, d % 512 == 0, True, fmt, T + d)
    b = _check_bwd(T, d, dtype, dy_dtype, d % 512 == 0, True, fmt, T + d)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])


@pytest.mark.parametrize("T,d,dtype", [(2367, 2048, BF), (2368, 2048, BF), (9471, 64, BF),
                                       (9472, 64, BF), (9473, 8, F32), (592, 4096, F32),
                                       (593, 16384, BF)])
def test_backward_where_the_path_changes(T, d, dtype):
    _check_bwd(T, d, dtype, dtype, True, True, None, T)


def test_backward_against_differences():
    """dx and dweight against central differences of the 64-bit forward."""
    g = torch.Generator().manual_seed(9)
    T, d, eps = 3, 40, 1e-6
    x, w, dy = (_rn(g, *s, dtype=F32) for s in ((T, d), (d,), (T, d)))
    f = lambda x_, w_: float((p64.norm(x_, w_, eps)[0] * dy.double()).sum())  # noqa: E731
    out = skv.add_rmsnorm_forward(x.cuda(), w.cuda(), eps=eps)
    b = skv.add_rmsnorm_backward(dy.cuda(), out["sum"], w.cuda(), out["rstd"])
    step = 1e-5
    for i, j in ((0, 0), (1, 17), (2, 39)):
        e = torch.zeros(T, d, dtype=torch.float64)
        e[i, j] = step
        diff = (f(x.double() + e, w.double()) - f(x.double() - e, w.double())) / (2 * step)
        assert abs(diff - float(b["dx"][i, j])) < 1e-5 * (1 + abs(diff))
    e = torch.zeros(d, dtype=torch.float64)
    e[11] = step
    diff = (f(x.double(), w.double() + e) - f(x.double(), w.double() - e)) / (2 * step)
    assert abs(diff - float(b["dweight"][11])) < 1e-5 * (1 + abs(diff))


def test_backward_is_reproducible_and_empty():
    a = _check_bwd(700, 1024, BF, BF, True, True, None, 5)
    b = _check_bwd(700, 1024, BF, BF, True, True, None, 5)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
    z = torch.empty(0, 64, device="cuda")
    e = skv.add_rmsnorm_backward(z, z, torch.ones(64, device="cuda"),
                                 torch.empty(0, device="cuda"))
    assert e["dx"].shape == (0, 64) and torch.equal(e["dweight"].cpu(), torch.zeros(64))


def test_captured_and_on_another_stream():
    g = torch.Generator().manual_seed(8)
    x, r, w = _rn(g, 65, 1024).cuda(), _rn(g, 65, 1024).cuda(), _rn(g, 1024).cuda()

    def step():
        f = skv.add_rmsnorm_forward(x, w, residual=r, fmt="e4m3")
        b = skv.add_rmsnorm_backward(f["y"], f["sum"], w, f["rstd"], dsum=f["y"])
        return [f["sum"], f["y"], f["rstd"], f["q8"], f["scales"], b["dx"], b["dweight"]]

    ref = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for t in kept:
        t.view(torch.uint8).zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(ref, other, kept):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


# ------------------------------------------------------------ 8 bits --

@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 120), (5, 128), (2, 136), (17, 1000), (130, 2048)])
def test_act8_round_trip(fmt, dtype, T, d):
    """The stored bytes are the 64-bit quotient rounded once (nearest even),
    the scales the smallest that hold the group, and reading back is exact."""
    g = torch.Generator().manual_seed(T * d)
    x = _rn(g, T, d, dtype=F32) * 10.0 ** (torch.rand(T, 1, generator=g) * 12 - 6)
    x[0, :5] = torch.tensor([448.0, 127.0, -448.0, 2.0 ** -9, 1.75])[: min(5, d)]
    x = x.to(dtype)
    q, s = skv.act8_store(x.cuda(), fmt)
    ref_s = p64.scale_of(p64.group_amax(x.double()), fmt)
    assert torch.equal(s.cpu().double(), ref_s)
    u = x.double() / p64.expand_scales(ref_s, d)
    ref_q = u.float().to(torch.float8_e4m3fn) if fmt == "e4m3" else u.round().to(torch.int8)
    assert torch.equal(q.cpu().view(torch.uint8), ref_q.view(torch.uint8))
    v = p64.q8_values(ref_q, ref_s)
    assert (((v - x.double()).abs()) <= p64.q8_half_step(x.double(), ref_s, fmt)).all()
    for out in (BF, F32):
        got = skv.act8_load(q, s, dtype=out)
        assert torch.equal(got.double().cpu(), v), out


def test_act8_edges():
    for fmt in ("e4m3", "int8"):
        x = torch.zeros(6, 256)
        x[1, 3] = float("nan")
        x[2, 200] = -float("inf")
        x[3] = 2.0 ** -120            # below the smallest scale: reads back as zero
        x[4] = 1.5 * 2.0 ** 126
        x[5, 0], x[5, 1] = 2.0 ** 20, 2.0 ** -20
        q, s = skv.act8_store(x.cuda(), fmt)
        v = skv.act8_load(q, s, dtype=F32).cpu()
        assert (v[0] == 0).all() and (v[3] == 0).all()
        assert torch.isnan(v[1, :128]).all() and (v[1, 128:] == 0).all()
        assert torch.isnan(v[2, 128:]).all() and (v[2, :128] == 0).all()
        assert torch.equal(v[4], x[4])
        assert v[5, 0] == 2.0 ** 20 and v[5, 1] == 0
    q, s = skv.act8_store(torch.empty(0, 64, device="cuda"), "int8")
    assert q.shape == (0, 64) and skv.act8_load(q, s).shape == (0, 64)
    assert math.isfinite(float(s.sum()))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_act8_at_the_largest_values(fmt, dtype):
    """The largest finite value of a type, alone and among others: the largest
    scales that there are (2^120 and 2^122), the stored bytes as everywhere, and
    what reads back is the exact product, infinite where it passes fp32."""
    top = torch.finfo(dtype).max
    x = torch.zeros(3, 136, dtype=torch.float64)
    x[0, 3], x[0, 4], x[0, 130] = top, -top / 2, -top
    x[1] = -top
    x[2, :128] = torch.linspace(-1, 1, 128, dtype=torch.float64) * 2.0 ** 127
    x = x.to(dtype)
    q, s = skv.act8_store(x.cuda(), fmt)
    ref_s = p64.scale_of(p64.group_amax(x.double()), fmt)
    assert torch.equal(s.cpu().double(), ref_s)
    assert float(ref_s.max()) == (2.0 ** 120 if fmt == "e4m3" else 2.0 ** 122)
    u = x.double() / p64.expand_scales(ref_s, 136)
    ref_q = u.float().to(torch.float8_e4m3fn) if fmt == "e4m3" else u.round().to(torch.int8)
    assert torch.equal(q.cpu().view(torch.uint8), ref_q.view(torch.uint8))
    v = p64.q8_values(ref_q, ref_s)
    assert torch.isinf(v.float()).any() and torch.isfinite(v[2].float()).all()
    for out in (BF, F32):
        assert torch.equal(skv.act8_load(q, s, dtype=out).cpu(), v.to(out))


def _forward_through_abi(x, r, w, s, y, fmt):
    """pkm_add_rmsnorm_forward with outputs of the caller's; returns (y8, scales, rstd)."""
    T, d = x.shape
    q = torch.empty(T, d, dtype=torch.int8, device="cuda")
    sc = torch.empty(T, p64.q8_groups(d), device="cuda")
    rstd = torch.empty(T, device="cuda")
    a = skv._lib.NormArgs(T, d, skv._dt(x), 1e-6, fmt, *(skv._ptr(t) for t in (x, r, w, s, y)),
                          *((q.data_ptr(), sc.data_ptr()) if fmt else (None, None)),
                          rstd.data_ptr())
    skv._enqueue("pkm_add_rmsnorm_forward", (ctypes.byref(a),), x.device)
    return (q, sc, rstd) if fmt else (rstd,)


@pytest.mark.parametrize("d", [8, 1000, 2048, 2056, 8192, 16384])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_forward_over_its_own_inputs(d, dtype):
    """y over x or the residual, with the sum elsewhere or over the other one."""
    g = torch.Generator().manual_seed(d)
    x, r, w = (_rn(g, *s, dtype=dtype).cuda() for s in ((37, d), (37, d), (d,)))
    for fmt in (skv.PKM_Q8_NONE, skv.PKM_Q8_INT8):
        s0, y0 = torch.empty_like(x), torch.empty_like(x)
        rest0 = _forward_through_abi(x, r, w, s0, y0, fmt)
        for s_over, y_over in ((None, "x"), (None, "r"), ("x", "r"), ("r", "x"), ("x", None)):
            t = dict(x=x.clone(), r=r.clone())
            s = t[s_over] if s_over else torch.empty_like(x)
            y = t[y_over] if y_over else torch.empty_like(x)
            rest = _forward_through_abi(t["x"], t["r"], w, s, y, fmt)
            for a, b in zip((s, y, *rest), (s0, y0, *rest0)):
                assert torch.equal(a, b), (s_over, y_over)
        alone = torch.empty_like(x)
        _forward_through_abi(x, None, w, None, alone, fmt)
        y = x.clone()
        _forward_through_abi(y, None, w, None, y, fmt)
        assert torch.equal(y, alone)


@pytest.mark.parametrize("T,d", [(33, 72), (61, 1000), (3000, 2048), (610, 8192), (41, 16384)])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", [None, "int8"])
def test_backward_over_its_own_inputs(T, d, dtype, fmt):
    """dx over dsum or dy, on both paths."""
    g = torch.Generator().manual_seed(T)
    h, dy, ds, w = (_rn(g, *s, dtype=dtype).cuda() for s in ((T, d), (T, d), (T, d), (d,)))
    sc, code = None, skv.PKM_Q8_NONE
    if fmt:
        h, sc = skv.act8_store(h, fmt)
        code = skv.PKM_Q8_INT8
    rstd = torch.rand(T, generator=g).cuda() + 0.5
    ref = skv.add_rmsnorm_backward(dy, h, w, rstd, dsum=ds, scales=sc)
    for over in ("dy", "dsum"):
        t = dict(dy=dy.clone(), dsum=ds.clone())
        dw = torch.empty(d, device="cuda")
        a = skv._lib.NormBwdArgs(T, d, skv._dt(dy), skv._dt(dy), code, skv._ptr(t["dy"]), skv._ptr(h),
                                 skv._ptr(sc), skv._ptr(w), skv._ptr(rstd), skv._ptr(t["dsum"]),
                                 skv._ptr(t[over]), skv._ptr(dw), None, 0)
        need = skv.load().pkm_add_rmsnorm_backward_workspace_size(ctypes.byref(a))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        a.workspace, a.workspace_bytes = ws.data_ptr(), need
        skv._enqueue("pkm_add_rmsnorm_backward", (ctypes.byref(a),), dy.device)
        assert torch.equal(t[over], ref["dx"]) and torch.equal(dw, ref["dweight"]), over
