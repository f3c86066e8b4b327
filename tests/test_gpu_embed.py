"""The token embedding with a scale and its gradient by sorted tokens,
against 64-bit definitions (through the C ABI).

Tolerances (U = 2^-24): the forward rounds the product to fp32 and to the
storage type, U + half a step of the value; the gradient of a row with n
tokens adds n terms, scales and stores: (n + 2) U of the sum of magnitudes
plus half a step of the value.  With accumulate one more addition.
"""

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
    assert skv.device_error() == 0
    yield
    assert skv.device_error() == 0


def _ids(g, T, V, kind):
    if kind == "same":
        return torch.full((T,), V // 2, dtype=torch.int32)
    if kind == "uniform":
        return torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    u = torch.rand(T, generator=g, dtype=torch.float64)  # rank-frequency, a few frequent ids
    return ((V + 1.0) ** u - 1).long().clamp(0, V - 1).to(torch.int32)


def _within(got, ref, tol, what):
    err = (got.double().cpu() - ref).abs()
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off by up to {(err - tol).max():.3g}"


@pytest.mark.parametrize("T,V,d,kind", [
    (1, 1, 8, "uniform"), (7, 5, 24, "uniform"), (65, 1000, 136, "zipf"), (509, 317, 520, "zipf"),
    (300, 7, 1024, "uniform"), (33, 90, 2056, "uniform"), (200, 40, 264, "same")])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_forward_and_backward(T, V, d, kind, dtype):
    g = torch.Generator().manual_seed(T + V + d)
    table = torch.randn(V, d, generator=g).to(dtype)
    ids = _ids(g, T, V, kind)
    scale = 1.7
    out = skv.embedding_forward(table.cuda(), ids.cuda(), scale=scale)
    ref = p64.embed(table, ids, scale)
    # the scale itself is an fp32 value: one more U
    _within(out, ref, (2 * U32 + p64.half_step(dtype)) * ref.abs(), "out")
    dout = torch.randn(T, d, generator=g).to(dtype)
    ref, mag, n = p64.embed_grad(dout, ids, V, scale)
    for gdt in (F32, BF):
        grad = skv.embedding_backward(dout.cuda(), ids.cuda(), V, scale=scale, grad_dtype=gdt)
        tol = (n + 3) * U32 * mag + (p64.half_step(BF) * ref.abs() if gdt == BF else 0)
        _within(grad, ref, tol, f"grad {gdt}")


@pytest.mark.parametrize("T,V,kind", [(1024, 131072, "zipf"), (1024, 2, "uniform"),
                                      (1000, 40000, "same"), (1025, 3000, "zipf"),
                                      (1030, 200, "same"), (2049, 7, "uniform"),
                                      (4095, 131072, "zipf"), (4096, 300, "zipf"),
                                      (4097, 65536, "uniform"), (20000, 131071, "zipf"),
                                      (8300, 3, "uniform"), (5000, 70000, "same"),
                                      (131072, 700, "zipf"), (140001, 200000, "zipf")])
def test_backward_many_tokens(T, V, kind):
    """Both sides of the 1024 tokens that are sorted by counting; long lists: several sort blocks, ids over many chunks, up to 18 key bits, and
    more tokens than one cluster sorts."""
    d = 64
    g = torch.Generator().manual_seed(T)
    ids, dout = _ids(g, T, V, kind), torch.randn(T, d, generator=g).to(BF)
    a = skv.embedding_backward(dout.cuda(), ids.cuda(), V, scale=8.0)
    b = skv.embedding_backward(dout.cuda(), ids.cuda(), V, scale=8.0)
    assert torch.equal(a, b)
    ref = torch.zeros(V, d, dtype=torch.float64).index_add_(0, ids.long(), dout.double() * 8)
    mag = torch.zeros(V, d, dtype=torch.float64).index_add_(0, ids.long(), dout.double().abs() * 8)
    n = torch.bincount(ids.long(), minlength=V)[:, None]
    _within(a, ref, (n + 3) * U32 * mag, "grad")
    assert (a.cpu()[n[:, 0] == 0] == 0).all()


@pytest.mark.parametrize("T,d", [(2047, 72), (2048, 72), (2049, 72), (1023, 2056), (1024, 72),
                                 (1025, 2056), (49, 1032), (64, 8)])
@pytest.mark.parametrize("kind", ["zipf", "same", "uniform"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward_at_the_end_of_counting(T, d, kind, accumulate):
    """Both sides of the longest list that is sorted by counting and of the
    longest whose long ids are joined by the sums; several column slices."""
    V = 5000 if T > 1000 else 40
    g = torch.Generator().manual_seed(T)
    ids, dout = _ids(g, T, V, kind), torch.randn(T, d, generator=g).to(BF)
    base = torch.randn(V, d, generator=g) if accumulate else torch.zeros(V, d)
    a = skv.embedding_backward(dout.cuda(), ids.cuda(), V, grad=base.cuda(), accumulate=accumulate)
    ref = base.double().index_add_(0, ids.long(), dout.double())
    mag = base.double().abs().index_add_(0, ids.long(), dout.double().abs())
    n = torch.bincount(ids.long(), minlength=V)[:, None]
    _within(a, ref, (n + 4) * U32 * mag, "grad")
    assert torch.equal(a.cpu()[n[:, 0] == 0], base[n[:, 0] == 0])


def test_padding_and_batch_shape():
    g = torch.Generator().manual_seed(2)
    V, d, pad = 50, 48, 7
    ids = torch.randint(0, V, (4, 33), generator=g, dtype=torch.int32)
    ids[1, 5:] = pad
    ids[3] = pad
    table, dout = torch.randn(V, d, generator=g), torch.randn(4, 33, d, generator=g)
    dout[3] = float("nan")  # whatever stands behind a padding id is never read into a sum
    for p in (pad, -1):
        i = torch.where(ids == pad, torch.tensor(p, dtype=torch.int32), ids)
        out = skv.embedding_forward(table.cuda(), i.cuda(), scale=0.5, pad_id=p).cpu()
        assert out.shape == (4, 33, d) and (out[i == p] == 0).all()
        assert torch.equal(out[i != p], table[i[i != p].long()] * 0.5)
        grad = skv.embedding_backward(dout.cuda(), i.cuda(), V, scale=0.5, pad_id=p)
        ref, mag, n = p64.embed_grad(dout, i, V, 0.5, p)
        _within(grad, ref, (n + 3) * U32 * mag, "grad")
    assert skv.device_error() == 0
    # nothing but padding
    i = torch.full((4, 33), -1, dtype=torch.int32).cuda()
    assert (skv.embedding_backward(dout.cuda(), i, V, pad_id=-1) == 0).all()


def test_accumulate_and_untouched_rows():
    g = torch.Generator().manual_seed(3)
    V, d, T = 60, 72, 300
    ids = torch.randint(0, V // 2, (T,), generator=g, dtype=torch.int32)
    dout = torch.randn(T, d, generator=g)
    ref, mag, n = p64.embed_grad(dout, ids, V, 2.0)
    for dt in (F32, BF):
        base = torch.randn(V, d, generator=g).to(dt)
        got = base.cuda()
        assert skv.embedding_backward(dout.cuda(), ids.cuda(), V, scale=2.0, grad=got,
                                      accumulate=True) is got
        want = ref + base.double()
        tol = (n + 4) * U32 * (mag + base.double().abs())
        if dt == BF:
            tol = tol + p64.half_step(BF) * want.abs()
        _within(got, want, tol, "accumulated")
        assert torch.equal(got.cpu()[V // 2:], base[V // 2:])
        # a gradient buffer full of NaN is overwritten without accumulate
        got.fill_(float("nan"))
        skv.embedding_backward(dout.cuda(), ids.cuda(), V, scale=2.0, grad=got)
        assert torch.isfinite(got.float()).all()


def test_ids_outside_the_table_set_the_status():
    ids = torch.tensor([0, 9, -3, 4, 2 ** 31 - 1], dtype=torch.int32)
    table = torch.randn(5, 16)
    out = skv.embedding_forward(table.cuda(), ids.cuda()).cpu()
    assert skv.device_error() == 4
    assert (out[[1, 2, 4]] == 0).all() and torch.equal(out[[0, 3]], table[[0, 4]])
    grad = skv.embedding_backward(torch.ones(5, 16).cuda(), ids.cuda(), 5).cpu()
    assert skv.device_error() == 4
    assert torch.equal(grad[:, 0], torch.tensor([1.0, 0, 0, 0, 1]))


def test_empty():
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    out = skv.embedding_forward(torch.randn(4, 8).cuda(), ids)
    assert out.shape == (0, 8)
    grad = torch.full((4, 8), float("nan"), device="cuda")
    skv.embedding_backward(torch.empty(0, 8, device="cuda"), ids, 4, grad=grad)
    assert (grad == 0).all()
    one = torch.ones(4, 8, device="cuda")
    skv.embedding_backward(torch.empty(0, 8, device="cuda"), ids, 4, grad=one, accumulate=True)
    assert (one == 1).all()


def test_captured_and_on_another_stream():
    """Replays read the ids of the replay; another stream gives the same bits."""
    g = torch.Generator().manual_seed(5)
    V, d, T = 400, 128, 900
    ids, dout = _ids(g, T, V, "zipf").cuda(), torch.randn(T, d, generator=g).to(BF).cuda()
    ref = skv.embedding_backward(dout, ids, V)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = skv.embedding_backward(dout, ids, V)
    s.synchronize()
    assert torch.equal(ref, other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = skv.embedding_backward(dout, ids, V)
    graph.replay()
    assert torch.equal(kept, ref)
    ids.copy_(_ids(g, T, V, "uniform"))
    graph.replay()
    assert torch.equal(kept, skv.embedding_backward(dout, ids, V))
