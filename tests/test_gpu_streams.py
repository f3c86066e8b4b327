"""The operators around a memory layer called with ``stream=``: a call on a busy
side stream must not have its workspace or outputs handed out to the current
stream before its kernels have run; calls on two streams at once, and longer
batches captured and replayed, give the same bits as one after the other."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _calls():
    import sparse_key_value_b200 as skv
    g = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=g)
    T, V, d = 600, 520, 136
    x, r, dy = (rnd(T, d).to(BF).cuda() for _ in range(3))
    w = rnd(d).to(BF).cuda()
    E = (rnd(V, d) * d ** -0.5).to(BF).cuda()
    W1, W2 = (rnd(d, d) * d ** -0.5).to(BF).cuda(), (rnd(d, d) * d ** -0.5).to(BF).cuda()
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    many = torch.randint(0, V, (5 * T,), generator=g, dtype=torch.int32).cuda()
    many_dy = rnd(5 * T, d).to(BF).cuda()
    dl = torch.rand(T, generator=g).cuda()
    q, s = skv.act8_store(x)
    f = skv.add_rmsnorm_forward(x, w, r)
    _, lse = skv.linear_xent_forward(x, E, ids)
    return {
        "embedding_forward": lambda **k: skv.embedding_forward(E, ids, **k),
        "embedding_backward": lambda **k: skv.embedding_backward(dy, ids, V, **k),
        "embedding_backward_long": lambda **k: skv.embedding_backward(many_dy, many, V, **k),
        "act8_store": lambda **k: skv.act8_store(x, **k),
        "act8_load": lambda **k: skv.act8_load(q, s, **k),
        "add_rmsnorm_forward": lambda **k: skv.add_rmsnorm_forward(x, w, r, fmt="int8", **k),
        "add_rmsnorm_backward": lambda **k: skv.add_rmsnorm_backward(dy, f["sum"], w, f["rstd"], **k),
        "linear_xent_forward": lambda **k: skv.linear_xent_forward(x, E, ids, **k),
        "linear_xent_backward": lambda **k: skv.linear_xent_backward(x, E, ids, lse, dl, **k),
        "memplus_backward_act8": lambda **k: skv.memplus_backward_act8(q, s, W1, W2, q, s, dy, **k),
    }


def _tensors(r):
    if isinstance(r, torch.Tensor):
        return [r]
    return [t for t in (r.values() if isinstance(r, dict) else r) if t is not None]


@pytest.mark.parametrize("name", [
    "embedding_forward", "embedding_backward", "embedding_backward_long", "act8_store", "act8_load",
    "add_rmsnorm_forward", "add_rmsnorm_backward", "linear_xent_forward", "linear_xent_backward",
    "memplus_backward_act8"])
def test_side_stream_keeps_its_memory(name):
    call = _calls()[name]
    want = [t.clone() for t in _tensors(call())]
    side = torch.cuda.Stream()
    sizes = [n for n in (512, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 21, 1 << 22, 1 << 23)
             for _ in range(4)]
    # once before, so that both streams' memory is there and nothing waits for it
    call(stream=side)
    taken = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes]
    del taken
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms: the call below is still waiting
    got = call(stream=side)
    # the current stream takes whatever memory the call gave back, and writes it
    taken = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda") for n in sizes]
    assert not side.query()  # the kernels had not run when the memory was written
    side.synchronize()
    torch.cuda.synchronize()
    del taken
    for a, b in zip(_tensors(got), want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_two_streams_at_once():
    calls = list(_calls().items())
    want = {n: [t.clone() for t in _tensors(f())] for n, f in calls}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for turn in range(6):
        for k, (n, f) in enumerate(calls):
            for j, st in enumerate(streams):  # different operators side by side
                m, h = calls[(k + 3 * j + turn) % len(calls)]
                got.append((m, h(stream=st)))
    torch.cuda.synchronize()
    for n, r in got:
        for a, b in zip(_tensors(r), want[n]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n


@pytest.mark.parametrize("T,V,d,accumulate", [
    (5000, 40000, 520, False), (5000, 40000, 520, True), (40000, 3000, 64, False),
    (140000, 3000, 64, False), (2048, 70000, 256, False)])
def test_embedding_backward_captured(T, V, d, accumulate):
    """Every way of sorting, replayed on other ids and over what earlier
    replays left in the gradient."""
    import sparse_key_value_b200 as skv
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    dout = torch.randn(T, d, generator=g).to(BF).cuda()
    grad = torch.full((V, d), 3.0, device="cuda")
    skv.embedding_backward(dout, ids, V, grad=grad.clone(), accumulate=accumulate)  # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        skv.embedding_backward(dout, ids, V, grad=grad, accumulate=accumulate)
    for turn in range(3):
        ids.copy_((torch.rand(T, generator=g) ** 3 * V).to(torch.int32))
        base = torch.full((V, d), 3.0, device="cuda")
        grad.copy_(base)
        graph.replay()
        want = skv.embedding_backward(dout, ids, V, grad=base, accumulate=accumulate)
        assert torch.equal(grad, want), turn


def test_long_norm_backward_captured():
    import sparse_key_value_b200 as skv
    g = torch.Generator().manual_seed(8)
    T, d = 3000, 2048
    x, dy, ds = (torch.randn(T, d, generator=g).to(BF).cuda() for _ in range(3))
    w = torch.randn(d, generator=g).to(BF).cuda()
    rstd = skv.add_rmsnorm_forward(x, w)["rstd"]
    skv.add_rmsnorm_backward(dy, x, w, rstd, dsum=ds)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = skv.add_rmsnorm_backward(dy, x, w, rstd, dsum=ds)
    for _ in range(2):
        dy.copy_(torch.randn(T, d, generator=g).to(BF))
        graph.replay()
        want = skv.add_rmsnorm_backward(dy, x, w, rstd, dsum=ds)
        assert torch.equal(kept["dx"], want["dx"])
        assert torch.equal(kept["dweight"], want["dweight"])
