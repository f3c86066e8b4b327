"""Refusals of the operators around a memory layer, on the host: an invalid
call returns its error and launches nothing (no GPU is needed)."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from sparse_key_value_b200 import build
    build.build()
    from sparse_key_value_b200 import _lib
    return _lib.load()


F = ctypes.c_void_p(1 << 20)         # 16-byte aligned, never dereferenced on the host
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD2 = ctypes.c_void_p((1 << 20) + 2)  # for the 4-byte aligned id lists


def _norm(**kw):
    from sparse_key_value_b200 import _lib
    base = dict(T=4, d=64, dtype=1, eps=1e-6, fmt=1, x=F, residual=F, weight=F, sum=F, y=F, y8=F,
                scales=F, rstd=F)
    return _lib.NormArgs(**{**base, **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(d=60), 1), (dict(dtype=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(fmt=0), 1), (dict(fmt=3), 1), (dict(y8=None), 1),
    (dict(x=None), 1), (dict(x=ODD), 1), (dict(residual=ODD), 1), (dict(weight=ODD), 1),
    (dict(sum=ODD), 1), (dict(y=ODD), 1), (dict(y8=ODD), 1), (dict(scales=None), 1),
    (dict(rstd=ODD), 1), (dict(y=None, y8=None, fmt=0), 1), (dict(d=16392), 2),
    (dict(T=2 ** 31), 2)])
def test_norm_forward_refuses(lib, bad, code):
    assert lib.pkm_add_rmsnorm_forward(ctypes.byref(_norm(**bad)), None) == code
    assert lib.pkm_add_rmsnorm_forward(None, None) == 1


def _norm_bwd(**kw):
    from sparse_key_value_b200 import _lib
    base = dict(T=4, d=64, dtype=1, dy_dtype=0, fmt=0, dy=F, sum=F, scales=None, weight=F, rstd=F,
                dsum=F, dx=F, dweight=F, workspace=F, workspace_bytes=1 << 40)
    return _lib.NormBwdArgs(**{**base, **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(d=4), 1), (dict(dtype=5), 1), (dict(dy_dtype=2), 1), (dict(fmt=7), 1),
    (dict(dy=None), 1), (dict(sum=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1),
    (dict(dx=ODD), 1), (dict(dweight=ODD), 1), (dict(fmt=1), 1), (dict(fmt=2, scales=ODD), 1),
    (dict(d=16392), 2), (dict(workspace=None), 6), (dict(workspace_bytes=64 * 4 - 1), 6)])
def test_norm_backward_refuses(lib, bad, code):
    assert lib.pkm_add_rmsnorm_backward(ctypes.byref(_norm_bwd(**bad)), None) == code


def test_norm_workspace_and_empty(lib):
    a = _norm_bwd()
    assert lib.pkm_add_rmsnorm_backward_workspace_size(ctypes.byref(a)) >= 64 * 4
    assert lib.pkm_add_rmsnorm_backward_workspace_size(None) == 0
    assert lib.pkm_add_rmsnorm_forward(ctypes.byref(_norm(T=0, x=None)), None) == 0
    # no weight gradient asked for: an empty call has nothing to do
    assert lib.pkm_add_rmsnorm_backward(ctypes.byref(_norm_bwd(T=0, dweight=None)), None) == 0


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(d=12), 1), (dict(dtype=2), 1), (dict(fmt=0), 1), (dict(fmt=3), 1),
    (dict(x=None), 1), (dict(x=ODD), 1), (dict(q=ODD), 1), (dict(s=ODD), 1), (dict(s=None), 1),
    (dict(T=2 ** 36 + 1), 2), (dict(T=2 ** 36, d=1024), 2)])
def test_act8_refuses(lib, bad, code):
    k = {**dict(x=F, T=4, d=64, dtype=1, fmt=1, q=F, s=F), **bad}
    assert lib.pkm_act8_store(k["x"], k["T"], k["d"], k["dtype"], k["fmt"], k["q"], k["s"],
                              None) == code
    assert lib.pkm_act8_load(k["q"], k["s"], k["T"], k["d"], k["fmt"], k["x"], k["dtype"],
                             None) == code


def _embed(**kw):
    from sparse_key_value_b200 import _lib
    base = dict(T=4, n_rows=10, d=64, dtype=1, grad_dtype=0, scale=1.0, has_pad=0, pad_id=0,
                accumulate=0, ids=F, table=F, out=F, dout=F, grad=F, workspace=F,
                workspace_bytes=1 << 40)
    return _lib.EmbedArgs(**{**base, **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(n_rows=0), 1), (dict(n_rows=2 ** 31), 1), (dict(d=4), 1),
    (dict(d=20), 1), (dict(dtype=9), 1), (dict(scale=float("nan")), 1), (dict(ids=None), 1),
    (dict(ids=ODD2), 1), (dict(T=2 ** 31), 2), (dict(d=65544), 2)])
def test_embed_refuses(lib, bad, code):
    assert lib.pkm_embed_forward(ctypes.byref(_embed(**bad)), None) == code
    assert lib.pkm_embed_backward(ctypes.byref(_embed(**bad)), None) == code


def test_embed_refuses_by_direction(lib):
    fwd = lambda **k: lib.pkm_embed_forward(ctypes.byref(_embed(**k)), None)   # noqa: E731
    bwd = lambda **k: lib.pkm_embed_backward(ctypes.byref(_embed(**k)), None)  # noqa: E731
    assert fwd(table=None) == 1 and fwd(out=ODD) == 1
    assert bwd(dout=None) == 1 and bwd(grad=ODD) == 1 and bwd(grad_dtype=4) == 1
    assert bwd(T=0, grad=None) == 1
    assert bwd(T=2 ** 31 - 64, d=65536) == 2  # more blocks than a grid has
    assert bwd(workspace=None) == 6
    for T in (4, 1024, 1025, 200000):
        need = lib.pkm_embed_workspace_size(ctypes.byref(_embed(T=T)))
        assert need > 0 and bwd(T=T, workspace_bytes=need - 1) == 6
    assert fwd(T=0, ids=None) == 0
    assert fwd(T=0) == 0 and lib.pkm_embed_workspace_size(None) == 0


def test_binding_refuses_bad_tensors():
    """The binding's own checks need no GPU: CPU tensors are refused."""
    import sparse_key_value_b200 as skv
    x = torch.zeros(4, 64)
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: skv.act8_store(x), lambda: skv.add_rmsnorm_forward(x),
                 lambda: skv.embedding_forward(x, ids),
                 lambda: skv.embedding_backward(x, ids, 4)):
        with pytest.raises(ValueError):
            call()


def _xent(**kw):
    from sparse_key_value_b200 import _lib
    base = dict(T=4, V=10, d=64, dtype=1, grad_dtype=0, ignore_index=-100, x=F, W=F, targets=F,
                loss=F, lse=F, dloss=F, dx=F, dW=F, workspace=F, workspace_bytes=1 << 40)
    return _lib.XentArgs(**{**base, **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(V=0), 1), (dict(d=4), 1), (dict(d=60), 1), (dict(dtype=3), 1),
    (dict(dtype=0), 2), (dict(grad_dtype=2), 1), (dict(x=None), 1), (dict(x=ODD), 1),
    (dict(W=ODD), 1), (dict(targets=None), 1), (dict(targets=ODD2), 1), (dict(lse=ODD), 1),
    (dict(d=65544), 2), (dict(V=2 ** 30 + 8), 2),
    (dict(T=2 ** 30 + 1), 2), (dict(T=2 ** 28, V=2 ** 20), 2), (dict(workspace=None), 6)])
def test_xent_refuses(lib, bad, code):
    assert lib.pkm_linear_xent_forward(ctypes.byref(_xent(**bad)), None) == code
    assert lib.pkm_linear_xent_backward(ctypes.byref(_xent(**bad)), None) == code


def test_xent_refuses_by_direction(lib):
    fwd = lambda **k: lib.pkm_linear_xent_forward(ctypes.byref(_xent(**k)), None)   # noqa: E731
    bwd = lambda **k: lib.pkm_linear_xent_backward(ctypes.byref(_xent(**k)), None)  # noqa: E731
    assert fwd(loss=None) == 1 and bwd(dloss=None) == 1 and bwd(dx=ODD) == 1 and bwd(dW=None) == 1
    assert bwd(T=0, dW=None) == 1
    for call, size in ((fwd, lib.pkm_linear_xent_forward_workspace_size),
                       (bwd, lib.pkm_linear_xent_backward_workspace_size)):
        need = size(ctypes.byref(_xent()))
        assert need > 0 and call(workspace_bytes=need - 1) == 6
        assert size(None) == 0 and size(ctypes.byref(_xent(d=60))) == 0
    assert fwd(T=0, x=None) == 0
    # the piece of d stays within 512 MiB (or 1024 columns) however large the vocabulary
    big = _xent(T=16384, V=262144, d=1024)
    need = lib.pkm_linear_xent_backward_workspace_size(ctypes.byref(big))
    assert need <= (512 << 20) + 4 * 16384 * 1024 * 4 + 1024


def _mp8(**kw):
    from sparse_key_value_b200 import _lib
    base = dict(T=4, d_model=64, d_v=32, fmt=2, grad_dtype=0, x8=F, x_scales=F, W1=F, W2=F, y8=F,
                y_scales=F, dout=F, dy=F, dx=F, dW1=F, dW2=F, workspace=F,
                workspace_bytes=1 << 40)
    return _lib.MemplusBwd8Args(**{**base, **kw})


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), 1), (dict(d_model=60), 1), (dict(d_v=0), 1), (dict(fmt=0), 1), (dict(fmt=3), 1),
    (dict(grad_dtype=2), 1), (dict(x8=None), 1), (dict(x_scales=ODD), 1), (dict(W1=ODD), 1),
    (dict(W2=None), 1), (dict(y8=ODD), 1), (dict(y_scales=None), 1), (dict(dout=None), 1),
    (dict(dy=ODD), 1), (dict(dx=None), 1), (dict(dW1=ODD), 1), (dict(dW2=None), 1),
    (dict(T=2 ** 28 + 1), 2), (dict(d_v=65544), 2), (dict(T=2 ** 28, d_model=65536), 2),
    (dict(workspace=None), 6)])
def test_memplus_act8_refuses(lib, bad, code):
    assert lib.pkm_memplus_backward_act8(ctypes.byref(_mp8(**bad)), None) == code


def test_memplus_act8_workspace(lib):
    need = lib.pkm_memplus_backward_act8_workspace_size(ctypes.byref(_mp8()))
    assert need > 0
    a = _mp8(workspace_bytes=need - 1)
    assert lib.pkm_memplus_backward_act8(ctypes.byref(a), None) == 6
    assert lib.pkm_memplus_backward_act8_workspace_size(None) == 0
    for T in (0, 1, 2 ** 28):  # any batch has a size, the empty one too
        lib.pkm_memplus_backward_act8_workspace_size(ctypes.byref(_mp8(T=T)))
        lib.pkm_linear_xent_backward_workspace_size(ctypes.byref(_xent(T=T)))
        lib.pkm_linear_xent_forward_workspace_size(ctypes.byref(_xent(T=T)))
    assert lib.pkm_memplus_backward_act8(ctypes.byref(_mp8(T=0, dW1=None)), None) == 1


def test_binding_refuses_tensors_of_another_device_than_the_stream():
    """``stream`` is a keyword; its device has to be the tensors' one."""
    import inspect

    import sparse_key_value_b200 as skv

    class Stream:
        device = torch.device("cuda", 1)

    x = torch.zeros(4, 64)
    for f in (skv.act8_store, skv.add_rmsnorm_forward):
        assert inspect.signature(f).parameters["stream"].kind is inspect.Parameter.KEYWORD_ONLY
        with pytest.raises(ValueError):
            f(x, stream=Stream())
    # what the check compares: no CPU call can hold a tensor of another GPU
    with pytest.raises(ValueError):
        skv._operands(Stream.device, x)
