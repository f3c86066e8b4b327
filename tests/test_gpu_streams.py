"""The operators around a memory layer called with ``stream=``: a call on a busy
side stream must not have its workspace or outputs handed out to the current
stream before its kernels have run."""

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
    many = torch.randint(0, V, (3 * T,), generator=g, dtype=torch.int32).cuda()
    many_dy = rnd(3 * T, d).to(BF).cuda()
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
