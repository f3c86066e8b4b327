"""Product-key memory lookup on B200 (sm_100a): torch-facing binding of
libpkm.so.

Every function here marshals torch tensors into the C ABI declared in
include/pkm.h and calls it on the current CUDA stream; the computation runs
entirely in the library's kernels.  Outputs and workspaces the caller does
not pass are allocated with torch (device memory only); the library itself
never allocates.
"""

from __future__ import annotations

import ctypes
import functools
import inspect
from typing import Optional

import torch

from . import _lib
from ._lib import (PKM_BF16, PKM_F32, PKM_Q8_E4M3, PKM_Q8_INT8, PKM_Q8_NONE, Q8_GROUP, PKMError,
                   BwdArgs, FwdArgs, check, load)

__all__ = ["PKMError", "load", "pkm_forward", "pkm_backward", "embbag_forward",
           "embbag_backward", "forward_workspace_size", "backward_workspace_size",
           "device_error", "fwd_args", "embedding_forward", "embedding_backward",
           "add_rmsnorm_forward", "add_rmsnorm_backward", "act8_store", "act8_load",
           "linear_xent_forward", "linear_xent_backward",
           "memplus_backward_act8"]


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return PKM_BF16
    if t.dtype == torch.float32:
        return PKM_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


def _stream(dev: torch.device, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(dev)
    return ctypes.c_void_p(s.cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libpkm works on CUDA tensors only")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def fwd_args(T, H, d_half, n_sub, k, d_v, dtype=PKM_BF16, d_model=0, memplus=False,
             **ptrs) -> FwdArgs:
    a = FwdArgs()
    a.T, a.H, a.d_half, a.n_sub, a.k, a.d_v, a.dtype = T, H, d_half, n_sub, k, d_v, dtype
    a.d_model = d_model
    if memplus:  # the size query only needs to know Memory+ is on
        a.x = a.W1 = a.W2 = ctypes.c_void_p(16)
    for name, v in ptrs.items():
        setattr(a, name, v)
    return a


def forward_workspace_size(T, H, d_half, n_sub, k, d_v, dtype=PKM_BF16, memplus=False,
                           d_model=0) -> int:
    a = fwd_args(T, H, d_half, n_sub, k, d_v, dtype, d_model, memplus)
    return int(load().pkm_forward_workspace_size(ctypes.byref(a)))


def pkm_forward(query, subkeys, values, k: int, x=None, W1=None, W2=None, out=None, idx=None,
                weights=None, workspace=None, stream=None, phase_events=None, y_out=None):
    """Forward of one memory layer (see pkm_forward in include/pkm.h).

    query [T,H,2,d_half], subkeys [H,2,n_sub,d_half], values [n_sub^2, d_v];
    optional Memory+ gate x [T,d_model], W1 [d_model,d_v], W2 [d_v,d_model].
    ``phase_events``: optional list of 7 torch.cuda.Event recorded at the
    phase boundaries (see pkm_fwd_args.phase_events).
    ``y_out``: Memory+ only, a [T, d_v] tensor receiving the bag output
    before the gate (what memplus_backward needs).
    Returns (out, idx, weights)."""
    _need_cuda(query, subkeys, values, x, W1, W2)
    T, H, two, dh = query.shape
    n = subkeys.shape[2]
    dv = values.shape[1]
    dev = query.device
    memplus = x is not None
    dm = x.shape[1] if memplus else 0
    if out is None:
        out = torch.empty(T, dm if memplus else dv, dtype=query.dtype, device=dev)
    if idx is None:
        idx = torch.empty(T, H, k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(T, H, k, dtype=torch.float32, device=dev)
    a = fwd_args(T, H, dh, n, k, dv, _dt(query), dm, False, query=_p(query), subkeys=_p(subkeys),
                 values=_p(values), x=_p(x), W1=_p(W1), W2=_p(W2), out=_p(out), idx=_p(idx),
                 weights=_p(weights))
    lib = load()
    need = int(lib.pkm_forward_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = _p(workspace), workspace.numel()
    a.y_out = _p(y_out)
    if phase_events is not None:
        if len(phase_events) != 7 or any(e.cuda_event == 0 for e in phase_events):
            raise ValueError("phase_events: 7 events, each recorded once before use")
        arr = (ctypes.c_void_p * len(phase_events))(*[e.cuda_event for e in phase_events])
        a.phase_events = ctypes.cast(arr, ctypes.c_void_p)
    check(lib.pkm_forward(ctypes.byref(a), _stream(dev, stream)), "pkm_forward")
    return out, idx, weights


def _bwd_args(query, subkeys, values, idx, weights, dy, **kw) -> BwdArgs:
    T, H, _, dh = query.shape
    a = BwdArgs()
    a.T, a.H, a.d_half, a.n_sub, a.k, a.d_v = T, H, dh, subkeys.shape[2], idx.shape[2], \
        values.shape[1]
    a.dtype = _dt(query)
    a.query, a.subkeys, a.values = _p(query), _p(subkeys), _p(values)
    a.idx, a.weights, a.dy = _p(idx), _p(weights), _p(dy)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def backward_workspace_size(query, subkeys, values, idx, weights, dy) -> int:
    a = _bwd_args(query, subkeys, values, idx, weights, dy)
    return int(load().pkm_backward_workspace_size(ctypes.byref(a)))


def pkm_backward(query, subkeys, values, idx, weights, dy, sparse: bool = True,
                 dense: Optional[torch.Tensor] = None, want_dscores: bool = False,
                 workspace=None, stream=None, uniq_cap: Optional[int] = None):
    """Backward of the plain lookup (see pkm_backward in include/pkm.h).

    Returns dict(dquery, dsubkeys, uniq_rows, grad_rows, n_uniq, dscores)
    with the sparse value gradient sliced to its n_uniq rows (a host read of
    n_uniq) when ``sparse``; ``dense`` [N, d_v] fp32 receives += if given."""
    _need_cuda(query, subkeys, values, idx, weights, dy, dense)
    T, H, _, dh = query.shape
    dev = query.device
    k = idx.shape[2]
    R = T * H * k
    dq = torch.empty(T, H, 2, dh, dtype=torch.float32, device=dev)
    dK = torch.empty_like(subkeys, dtype=torch.float32)
    cap = R if uniq_cap is None else uniq_cap
    uniq = torch.empty(max(cap, 1), dtype=torch.int32, device=dev) if sparse else None
    grad = torch.empty(max(cap, 1), values.shape[1], dtype=torch.float32, device=dev) \
        if sparse else None
    n_uniq = torch.zeros(1, dtype=torch.int64, device=dev) if sparse else None
    dS = torch.empty(T, H, k, dtype=torch.float32, device=dev) if want_dscores else None
    a = _bwd_args(query, subkeys, values, idx, weights, dy, dquery=_p(dq), dsubkeys=_p(dK),
                  uniq_rows=_p(uniq), grad_rows=_p(grad), n_uniq=_p(n_uniq),
                  uniq_cap=cap if sparse else 0, dvalues_dense=_p(dense), dscores=_p(dS))
    lib = load()
    need = int(lib.pkm_backward_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = _p(workspace), workspace.numel()
    check(lib.pkm_backward(ctypes.byref(a), _stream(dev, stream)), "pkm_backward")
    res = dict(dquery=dq, dsubkeys=dK, dscores=dS, n_uniq=n_uniq)
    if sparse:
        u = int(n_uniq.item())
        res.update(uniq_rows=uniq[:u], grad_rows=grad[:u])
    return res


def embbag_forward(table, idx, w, gate=None, out=None, stream=None):
    """out[t] = (sum_j w[t,j] table[idx[t,j]]) (⊙ gate[t]); idx int32, w fp32 [n_bags, B]."""
    _need_cuda(table, idx, w, gate)
    n_bags, B = idx.shape
    d = table.shape[1]
    if out is None:
        out = torch.empty(n_bags, d, dtype=table.dtype, device=table.device)
    check(load().embbag_forward(_p(table), table.shape[0], d, _dt(table), _p(idx), _p(w),
                                n_bags, B, _p(gate), _p(out), _stream(table.device, stream)),
          "embbag_forward")
    return out


def embbag_backward(dy, idx, w, table=None, n_rows=None, sparse=True, dense=None,
                    want_dw=False, stream=None):
    """Backward of embbag_forward (no gate); see include/pkm.h."""
    _need_cuda(dy, idx, w, table, dense)
    n_bags, B = idx.shape
    d = dy.shape[1]
    dev = dy.device
    n_rows = table.shape[0] if n_rows is None else n_rows
    R = n_bags * B
    dw = torch.empty(n_bags, B, dtype=torch.float32, device=dev) if want_dw else None
    uniq = torch.empty(max(R, 1), dtype=torch.int32, device=dev) if sparse else None
    grad = torch.empty(max(R, 1), d, dtype=torch.float32, device=dev) if sparse else None
    n_uniq = torch.zeros(1, dtype=torch.int64, device=dev) if sparse else None
    lib = load()
    need = int(lib.embbag_backward_workspace_size(n_bags, B, d, n_rows))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    check(lib.embbag_backward(_p(dy), _p(idx), _p(w), n_bags, B, d, _dt(dy), _p(table), n_rows,
                              _p(dw), _p(uniq), _p(grad), _p(n_uniq), R if sparse else 0,
                              _p(dense), _p(ws), ws.numel(), _stream(dev, stream)),
          "embbag_backward")
    res = dict(dw=dw)
    if sparse:
        u = int(n_uniq.item())
        res.update(uniq_rows=uniq[:u], grad_rows=grad[:u])
    return res


def device_error(stream=None, device=None) -> int:
    """Synchronise and read-and-clear the device status word (0 = none)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    code = ctypes.c_int32(0)
    check(load().pkm_get_device_error(_stream(dev, stream), ctypes.byref(code)),
          "pkm_get_device_error")
    return int(code.value)


def memplus_backward(x, W1, W2, y, dout, workspace=None, stream=None):
    """Backward of the Memory+ block (see pkm_memplus_backward in include/pkm.h).

    x [T,d_model], W1 [d_model,d_v], W2 [d_v,d_model], y [T,d_v] (the
    forward's y_out), dout [T,d_model], all bf16.  Returns dict(dy (bf16,
    the dy of pkm_backward), dx, dW1, dW2 (fp32))."""
    _need_cuda(x, W1, W2, y, dout)
    T, dm = x.shape
    dv = W1.shape[1]
    dev = x.device
    dy = torch.empty(T, dv, dtype=x.dtype, device=dev)
    dx = torch.empty(T, dm, dtype=torch.float32, device=dev)
    dW1 = torch.empty(dm, dv, dtype=torch.float32, device=dev)
    dW2 = torch.empty(dv, dm, dtype=torch.float32, device=dev)
    a = _lib.MemplusBwdArgs(T, dm, dv, _p(x), _p(W1), _p(W2), _p(y), _p(dout), _p(dy), _p(dx),
                            _p(dW1), _p(dW2), None, 0)
    lib = load()
    need = int(lib.pkm_memplus_backward_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = _p(workspace), workspace.numel()
    check(lib.pkm_memplus_backward(ctypes.byref(a), _stream(dev, stream)), "pkm_memplus_backward")
    return dict(dy=dy, dx=dx, dW1=dW1, dW2=dW2)


def _qproj_args(x, Wq, q=None, dq=None, dWq=None, dx=None) -> "_lib.QprojArgs":
    T, dm = x.shape
    return _lib.QprojArgs(T, dm, Wq.shape[1], _p(x), _p(Wq), _p(q), _p(dq), _p(dWq), _p(dx),
                          None, 0)


def _qproj_call(fn: str, a, dev, workspace, stream):
    lib = load()
    need = int(lib.pkm_qproj_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = _p(workspace), workspace.numel()
    check(getattr(lib, fn)(ctypes.byref(a), _stream(dev, stream)), fn)


def qproj_forward(x, Wq, out=None, workspace=None, stream=None):
    """q = x Wq (bf16 [T, d_q]; see pkm_qproj_forward in include/pkm.h)."""
    _need_cuda(x, Wq)
    if out is None:
        out = torch.empty(x.shape[0], Wq.shape[1], dtype=x.dtype, device=x.device)
    _qproj_call("pkm_qproj_forward", _qproj_args(x, Wq, q=out), x.device, workspace, stream)
    return out


def qproj_backward(x, Wq, dq, dx=None, workspace=None, stream=None):
    """dWq = x^T dq and dx += dq Wq^T (dq fp32 [T, d_q]; dx fp32 [T, d_model],
    zero-initialised when not given).  Returns dict(dWq, dx)."""
    _need_cuda(x, Wq, dq)
    dev = x.device
    if dx is None:
        dx = torch.zeros(x.shape[0], x.shape[1], dtype=torch.float32, device=dev)
    dWq = torch.empty(x.shape[1], Wq.shape[1], dtype=torch.float32, device=dev)
    dq = dq.reshape(x.shape[0], Wq.shape[1]).contiguous()
    _qproj_call("pkm_qproj_backward", _qproj_args(x, Wq, dq=dq, dWq=dWq, dx=dx), dev, workspace,
                stream)
    return dict(dWq=dWq, dx=dx)


def sparse_optimizer_step(table, rows, grads, count, lr: float, kind: str = "sgd", m=None,
                          v=None, betas=(0.9, 0.999), eps: float = 1e-8, step: int = 1,
                          stream=None):
    """In-place SGD or touched-rows Adam on the rows of a sparse value
    gradient (see pkm_sparse_optimizer_step in include/pkm.h): table
    [n_rows, d], rows int32 [cap], grads fp32 [cap, d], count device int64
    [1] (pkm_backward's uniq_rows, grad_rows, n_uniq); m, v fp32 [n_rows, d]
    for Adam."""
    _need_cuda(table, rows, grads, count, m, v)
    adam = kind == "adam"
    if adam and (m is None or v is None):
        raise ValueError("adam needs the moment tensors m and v")
    a = _lib.SparseOptArgs(1 if adam else 0, lr, betas[0], betas[1], eps, step, table.shape[0],
                           table.shape[1], _dt(table), _p(table), _p(rows), _p(grads), _p(count),
                           rows.shape[0], _p(m), _p(v))
    check(load().pkm_sparse_optimizer_step(ctypes.byref(a), _stream(table.device, stream)),
          "pkm_sparse_optimizer_step")
    return table


def engram_forward(tokens, table, h, orders, K: int, seeds, rows_per_head, alpha=True,
                   rows=False, e=False, out=None, stream=None):
    """Engram lookup (see pkm_engram_forward in include/pkm.h): hashed
    n-gram rows of the stacked table, their sum e and the context gate.

    tokens [n_seq, L] int32, table [sum(rows_per_head), d], h [T, d] CUDA
    tensors (T = n_seq * L); orders, seeds and rows_per_head host sequences
    (head j = o*K + k).  Returns dict(v, alpha, rows, e), the optional ones
    None unless asked for."""
    _need_cuda(tokens, table, h, out)
    if tokens.dtype != torch.int32:
        raise TypeError("tokens must be int32")
    n_seq, L = tokens.shape
    T, d = h.shape
    if T != n_seq * L or table.shape[1] != d or table.dtype != h.dtype:
        raise ValueError("shapes: tokens [n_seq, L], h [n_seq*L, d], table [rows, d], one dtype")
    dev = h.device
    heads = len(orders) * K
    od = (ctypes.c_int32 * len(orders))(*orders)
    sd = (ctypes.c_uint64 * heads)(*[int(x) & (2 ** 64 - 1) for x in seeds])
    md = (ctypes.c_int64 * heads)(*rows_per_head)
    v = torch.empty(T, d, dtype=h.dtype, device=dev) if out is None else out
    a_t = torch.empty(T, dtype=torch.float32, device=dev) if alpha else None
    r_t = torch.empty(T, heads, dtype=torch.int32, device=dev) if rows else None
    e_t = torch.empty(T, d, dtype=h.dtype, device=dev) if e else None
    args = _lib.EngramArgs(n_seq, L, len(orders), K, ctypes.cast(od, ctypes.c_void_p),
                           ctypes.cast(sd, ctypes.c_void_p), ctypes.cast(md, ctypes.c_void_p),
                           d, _dt(h), _p(tokens), _p(table), _p(h), _p(v), _p(a_t), _p(r_t),
                           _p(e_t))
    check(load().pkm_engram_forward(ctypes.byref(args), _stream(dev, stream)),
          "pkm_engram_forward")
    return dict(v=v, alpha=a_t, rows=r_t, e=e_t)


def pkm_select(query, subkeys, k: int, d_v: int = 8, idx=None, weights=None, workspace=None,
               stream=None):
    """The selection alone (see pkm_select in include/pkm.h): returns (idx,
    weights) [T, H, k] as pkm_forward would."""
    _need_cuda(query, subkeys)
    T, H, two, dh = query.shape
    n = subkeys.shape[2]
    dev = query.device
    if idx is None:
        idx = torch.empty(T, H, k, dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty(T, H, k, dtype=torch.float32, device=dev)
    a = fwd_args(T, H, dh, n, k, d_v, _dt(query), 0, False, query=_p(query),
                 subkeys=_p(subkeys), idx=_p(idx), weights=_p(weights))
    lib = load()
    need = int(lib.pkm_forward_workspace_size(ctypes.byref(a)))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    a.workspace, a.workspace_bytes = _p(workspace), workspace.numel()
    check(lib.pkm_select(ctypes.byref(a), _stream(dev, stream)), "pkm_select")
    return idx, weights


def embbag_forward_range(table_shard, row_lo: int, idx, w, out=None, stream=None):
    """Partial bags over one row shard (see embbag_forward_range in
    include/pkm.h): table_shard holds rows [row_lo, row_lo + len) of the full
    table; idx int32 / w fp32 [n_bags, B] hold full-table ids; returns fp32
    [n_bags, d]."""
    _need_cuda(table_shard, idx, w, out)
    n_bags, B = idx.shape
    d = table_shard.shape[1]
    if out is None:
        out = torch.empty(n_bags, d, dtype=torch.float32, device=table_shard.device)
    check(load().embbag_forward_range(_p(table_shard), row_lo, table_shard.shape[0], d,
                                      _dt(table_shard), _p(idx), _p(w), n_bags, B, _p(out),
                                      _stream(table_shard.device, stream)),
          "embbag_forward_range")
    return out


def check_wait_timeout(polls: int = 4096, device=None, stream=None) -> int:
    """Run the bounded-wait failure path (see pkm_check_wait_timeout in
    include/pkm.h) and return the device status it left (PKM_ERR_TIMEOUT = 5
    expected), after checking that the waiting kernel returned."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    done = torch.zeros(1, dtype=torch.int32, device=dev)
    check(load().pkm_check_wait_timeout(polls, _p(done), _stream(dev, stream)),
          "pkm_check_wait_timeout")
    code = device_error(stream, dev)
    if int(done.item()) != 1:
        raise RuntimeError(f"the waiting kernel did not finish as expected ({int(done.item())})")
    return code


def _operands(dev: torch.device, *ts):
    """Contiguous tensors of one GPU (or None)."""
    index = dev.index
    for t in ts:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            _need_cuda(t)
            raise ValueError(f"tensors on different devices: {t.device} and {dev}")


# Small calls take as long as their host side, a third of which is torch.empty
# reading its arguments (1.6 us); the entry that generated code uses takes half.
try:
    from torch._C._dynamo.guards import _empty_strided_cuda
except ImportError:
    _empty_strided_cuda = None


def _new_here(dtype, n, d=None):
    if d is None:
        return _empty_strided_cuda((n,), (1,), dtype)
    return _empty_strided_cuda((n, d), (d, 1), dtype)


def _new(dev: torch.device):
    """new(dtype, n[, d]): an uninitialised tensor on ``dev``."""
    if _empty_strided_cuda is not None and torch.cuda.current_device() == dev.index:
        return _new_here
    return lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=dev)


def _shape(name: str, t: Optional[torch.Tensor], shape, dtype=None):
    if t is None:
        return
    if t.shape != shape:  # shape: a tuple (torch.Size is one)
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")


# The current stream of a device as a plain handle: building a torch Stream
# object for it takes longer than the rest of a call's checks together.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _on_stream(f):
    """Gives ``f`` the keyword ``stream``: the whole call then runs with that
    stream current, so what it allocates comes from the memory that the
    allocator keeps for it.  A workspace taken from another stream's memory
    could be handed out again, when the call returns, before its kernels have
    run."""
    @functools.wraps(f)
    def call(*args, stream: Optional[torch.cuda.Stream] = None, **kw):
        if stream is None:
            return f(*args, **kw)
        _operands(stream.device,
                  *(t for t in (*args, *kw.values()) if isinstance(t, torch.Tensor)))
        with torch.cuda.stream(stream):
            return f(*args, **kw)

    call.__signature__ = inspect.Signature(
        [*inspect.signature(f).parameters.values(),
         inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _enqueue(fn: str, args, dev: torch.device):
    """Call the entry point with ``args`` on the tensors' device and its
    current stream."""
    f = getattr(load(), fn)
    index = dev.index
    s = torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(index)
    if torch.cuda.current_device() == index:
        code = f(*args, s)
    else:
        with torch.cuda.device(dev):
            code = f(*args, s)
    if code:
        check(code, fn)


def _workspace(a, workspace, need: int, dev: torch.device):
    """Puts the workspace into ``a``; returns its tensor, to be kept until the call."""
    if workspace is None:
        a.workspace_bytes = need = max(need, 16)
        workspace = _new(dev)(torch.uint8, need)
    else:
        _operands(dev, workspace)
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.workspace = workspace.data_ptr()
    return workspace


def _embed_args(ids, n_rows, d, dtype, scale, pad_id) -> "_lib.EmbedArgs":
    if ids.dtype != torch.int32:
        raise TypeError("ids must be int32")
    if pad_id is not None and not -2 ** 31 <= pad_id < 2 ** 31:  # ctypes would cut it silently
        raise ValueError(f"pad_id {pad_id} is not an int32")
    return _lib.EmbedArgs(ids.numel(), n_rows, d, dtype, dtype, scale, pad_id is not None,
                          pad_id or 0, 0, ids.data_ptr())


@_on_stream
def embedding_forward(table, ids, scale: float = 1.0, pad_id: Optional[int] = None, out=None):
    """out[t] = scale * table[ids[t]] (see pkm_embed_forward in include/pkm.h).

    table [n_rows, d], ids int32 of any shape; out [*ids.shape, d].
    Positions holding ``pad_id`` give a zero row."""
    dev = table.device
    _operands(dev, table, ids, out)
    n_rows, d = table.shape
    a = _embed_args(ids, n_rows, d, _dt(table), scale, pad_id)
    if out is not None:
        _shape("out", out, (*ids.shape, d), table.dtype)
    elif ids.ndim == 1:
        out = _new(dev)(table.dtype, ids.shape[0], d)
    else:
        out = torch.empty(*ids.shape, d, dtype=table.dtype, device=dev)
    a.table, a.out = table.data_ptr(), out.data_ptr()
    _enqueue("pkm_embed_forward", (ctypes.byref(a),), dev)
    return out


@_on_stream
def embedding_backward(dout, ids, n_rows: int, scale: float = 1.0, pad_id: Optional[int] = None,
                       grad=None, accumulate: bool = False, grad_dtype=torch.float32,
                       workspace=None):
    """Gradient of embedding_forward's table (see pkm_embed_backward in
    include/pkm.h): grad[r] = scale * the sum of dout over the positions of r.

    dout [*ids.shape, d]; returns grad [n_rows, d] (``grad_dtype``, or the
    given tensor), every row written, or added to with ``accumulate``."""
    dev = dout.device
    _operands(dev, dout, ids, grad)
    d = dout.shape[-1]
    _shape("dout", dout, (*ids.shape, d))
    if accumulate and grad is None:
        raise ValueError("accumulate needs grad")
    a = _embed_args(ids, n_rows, d, _dt(dout), scale, pad_id)
    if grad is None:
        grad = _new(dev)(grad_dtype, n_rows, d)
    else:
        _shape("grad", grad, (n_rows, d))
    a.grad_dtype, a.accumulate = _dt(grad), 1 if accumulate else 0
    workspace = _workspace(a, workspace, load().pkm_embed_workspace_size(ctypes.byref(a)), dev)
    a.dout, a.grad = dout.data_ptr(), grad.data_ptr()
    _enqueue("pkm_embed_backward", (ctypes.byref(a),), dev)
    return grad


_Q8 = {"e4m3": (PKM_Q8_E4M3, torch.float8_e4m3fn), "int8": (PKM_Q8_INT8, torch.int8)}


def _q8_fmt(q: torch.Tensor) -> int:
    for fmt, dtype in _Q8.values():
        if q.dtype == dtype:
            return fmt
    raise TypeError(f"8-bit values must be float8_e4m3fn or int8, not {q.dtype}")


def _q8_name(fmt: str):
    if fmt not in _Q8:
        raise ValueError(f"fmt {fmt!r}: 'e4m3' or 'int8'")
    return _Q8[fmt]


def _q8_empty(T: int, d: int, dtype, new):
    return new(dtype, T, d), new(torch.float32, T, (d + Q8_GROUP - 1) // Q8_GROUP)


def _q8_check(name: str, q, scales):
    """Checks an 8-bit activation and its scales, called ``name``; returns (T, d, fmt)."""
    _operands(q.device, q, scales)
    fmt = _q8_fmt(q)
    T, d = q.shape
    _shape(name, scales, (T, (d + Q8_GROUP - 1) // Q8_GROUP), torch.float32)
    return T, d, fmt


@_on_stream
def act8_store(x, fmt: str = "int8"):
    """x [T, d] in 8 bits (see pkm_act8_store in include/pkm.h): returns
    (q [T, d] float8_e4m3fn or int8, scales fp32 [T, ceil(d / 128)])."""
    dev = x.device
    _operands(dev, x)
    code, dtype = _q8_name(fmt)
    T, d = x.shape
    q, scales = _q8_empty(T, d, dtype, _new(dev))
    _enqueue("pkm_act8_store", (x.data_ptr(), T, d, _dt(x), code, q.data_ptr(),
                                scales.data_ptr()), dev)
    return q, scales


@_on_stream
def act8_load(q, scales, dtype=torch.bfloat16, out=None):
    """The values act8_store's (or add_rmsnorm_forward's) 8 bits stand for,
    exact in bf16."""
    T, d, fmt = _q8_check("scales", q, scales)
    dev = q.device
    if out is None:
        out = _new(dev)(dtype, T, d)
    else:
        _operands(dev, out)
        _shape("out", out, (T, d))
    _enqueue("pkm_act8_load", (q.data_ptr(), scales.data_ptr(), T, d, fmt, out.data_ptr(),
                               _dt(out)), dev)
    return out


@_on_stream
def add_rmsnorm_forward(x, weight=None, residual=None, eps: float = 1e-6,
                        fmt: Optional[str] = None, want_y: bool = True, sum_out=None):
    """h = x + residual, y = h / rms(h) * weight (see pkm_add_rmsnorm_forward
    in include/pkm.h).

    x, residual [T, d], weight [d].  Returns dict(sum (x itself without a
    residual), y (None unless ``want_y``), rstd fp32 [T], and with ``fmt``
    ('e4m3' or 'int8') q8, scales: y in 8 bits).  ``sum_out`` may be x or
    residual, to add in place."""
    dev, dt = x.device, x.dtype
    _operands(dev, x, weight, residual, sum_out)
    T, d = shape = x.shape
    _shape("residual", residual, shape, dt)
    _shape("weight", weight, (d,), dt)
    _shape("sum_out", sum_out, shape, dt)
    new = _new(dev)
    h = sum_out
    if h is None and residual is not None:
        h = new(dt, T, d)
    y = new(dt, T, d) if want_y else None
    rstd = new(torch.float32, T)
    q = scales = None
    code = PKM_Q8_NONE
    if fmt is not None:
        code, qdt = _q8_name(fmt)
        q, scales = _q8_empty(T, d, qdt, new)
    a = _lib.NormArgs(T, d, _dt(x), eps, code, _ptr(x), _ptr(residual), _ptr(weight), _ptr(h), _ptr(y),
                      _ptr(q), _ptr(scales), _ptr(rstd))
    _enqueue("pkm_add_rmsnorm_forward", (ctypes.byref(a),), dev)
    return dict(sum=x if h is None else h, y=y, rstd=rstd, q8=q, scales=scales)


@_on_stream
def add_rmsnorm_backward(dy, sum, weight, rstd, dsum=None, scales=None, want_dweight: bool = True,
                         workspace=None):
    """Backward of add_rmsnorm_forward (see pkm_add_rmsnorm_backward in
    include/pkm.h).

    dy [T, d] (bf16 or fp32); ``sum`` the forward's h [T, d], or its 8-bit
    copy together with ``scales`` (act8_store); dsum the gradient that
    reaches the stored sum from elsewhere.  Returns dict(dx: the gradient of
    x and of the residual, in the type of dsum, weight or dy; dweight fp32 [d])."""
    dev = dy.device
    _operands(dev, dy, sum, weight, rstd, dsum)
    T, d = shape = dy.shape
    fmt = PKM_Q8_NONE
    if scales is not None:
        _, _, fmt = _q8_check("scales", sum, scales)
        like = dsum if dsum is not None else weight if weight is not None else dy
        dt = like.dtype
    else:
        dt = sum.dtype
    _shape("sum", sum, shape)
    _shape("weight", weight, (d,), dt)
    _shape("rstd", rstd, (T,), torch.float32)
    _shape("dsum", dsum, shape, dt)
    new = _new(dev)
    dx = new(dt, T, d)
    dweight = new(torch.float32, d) if want_dweight else None
    a = _lib.NormBwdArgs(T, d, _dt(dx), _dt(dy), fmt, _ptr(dy), _ptr(sum), _ptr(scales), _ptr(weight),
                         _ptr(rstd), _ptr(dsum), _ptr(dx), _ptr(dweight), None, 0)
    if want_dweight:
        need = load().pkm_add_rmsnorm_backward_workspace_size(ctypes.byref(a))
        workspace = _workspace(a, workspace, need, dev)
    _enqueue("pkm_add_rmsnorm_backward", (ctypes.byref(a),), dev)
    return dict(dx=dx, dweight=dweight)


def _xent_args(x, W, targets, ignore_index: int) -> "_lib.XentArgs":
    _operands(x.device, x, W, targets)
    T, d = x.shape
    _shape("W", W, (W.shape[0], d), x.dtype)
    _shape("targets", targets, (T,), torch.int32)
    if not -2 ** 31 <= ignore_index < 2 ** 31:
        raise ValueError(f"ignore_index {ignore_index} is not an int32")
    return _lib.XentArgs(T, W.shape[0], d, _dt(x), PKM_F32, ignore_index, x.data_ptr(),
                         W.data_ptr(), targets.data_ptr())


@_on_stream
def linear_xent_forward(x, W, targets, ignore_index: int = -100, workspace=None):
    """Cross entropy of the output layer without keeping the logits (see
    pkm_linear_xent_forward in include/pkm.h).

    x [T, d], W [V, d] bf16, targets int32 [T].  Returns (loss, lse) fp32
    [T]; positions whose target is ``ignore_index`` have loss 0."""
    a = _xent_args(x, W, targets, ignore_index)
    dev = x.device
    new = _new(dev)
    loss, lse = new(torch.float32, a.T), new(torch.float32, a.T)
    a.loss, a.lse = loss.data_ptr(), lse.data_ptr()
    need = load().pkm_linear_xent_forward_workspace_size(ctypes.byref(a))
    workspace = _workspace(a, workspace, need, dev)
    _enqueue("pkm_linear_xent_forward", (ctypes.byref(a),), dev)
    return loss, lse


@_on_stream
def linear_xent_backward(x, W, targets, lse, dloss, ignore_index: int = -100,
                         grad_dtype=torch.float32, dx=None, dW=None, workspace=None):
    """Gradients of linear_xent_forward (see pkm_linear_xent_backward in
    include/pkm.h): lse as the forward gave it, dloss fp32 [T] the upstream
    gradient of each position's loss.  Returns (dx [T, d], dW [V, d]) in
    ``grad_dtype`` (or the given tensors, overwritten)."""
    a = _xent_args(x, W, targets, ignore_index)
    dev = x.device
    _operands(dev, lse, dloss, dx, dW)
    _shape("lse", lse, (a.T,), torch.float32)
    _shape("dloss", dloss, (a.T,), torch.float32)
    if dx is None:
        dx = torch.empty(x.shape, dtype=grad_dtype if dW is None else dW.dtype, device=dev)
    if dW is None:
        dW = torch.empty(W.shape, dtype=dx.dtype, device=dev)
    _shape("dx", dx, x.shape)
    _shape("dW", dW, W.shape, dx.dtype)
    a.grad_dtype = _dt(dx)
    a.lse, a.dloss, a.dx, a.dW = _ptr(lse), _ptr(dloss), _ptr(dx), _ptr(dW)
    need = load().pkm_linear_xent_backward_workspace_size(ctypes.byref(a))
    workspace = _workspace(a, workspace, need, dev)
    _enqueue("pkm_linear_xent_backward", (ctypes.byref(a),), dev)
    return dx, dW


@_on_stream
def memplus_backward_act8(x8, x_scales, W1, W2, y8, y_scales, dout, grad_dtype=torch.float32,
                          workspace=None):
    """Backward of the Memory+ block from 8-bit activations (see
    pkm_memplus_backward_act8 in include/pkm.h).

    x8, x_scales and y8, y_scales: the gate's input [T, d_model] and the bag
    output [T, d_v] as act8_store (or add_rmsnorm_forward) wrote them, in one
    format; W1 [d_model, d_v], W2 [d_v, d_model], dout [T, d_model] bf16.
    Returns dict(dy (bf16), dx, dW1, dW2 (``grad_dtype``))."""
    T, dm, fmt = _q8_check("x_scales", x8, x_scales)
    T2, dv, fmt2 = _q8_check("y_scales", y8, y_scales)
    if T2 != T or fmt2 != fmt:
        raise ValueError("x8 and y8: one number of rows and one format")
    dev = x8.device
    _operands(dev, y8, W1, W2, dout)
    bf = torch.bfloat16
    _shape("W1", W1, (dm, dv), bf)
    _shape("W2", W2, (dv, dm), bf)
    _shape("dout", dout, (T, dm), bf)
    new = _new(dev)
    dy, dx = new(bf, T, dv), new(grad_dtype, T, dm)
    dW1, dW2 = new(grad_dtype, dm, dv), new(grad_dtype, dv, dm)
    a = _lib.MemplusBwd8Args(T, dm, dv, fmt, _dt(dx), _ptr(x8), _ptr(x_scales), _ptr(W1), _ptr(W2),
                             _ptr(y8), _ptr(y_scales), _ptr(dout), _ptr(dy), _ptr(dx), _ptr(dW1), _ptr(dW2),
                             None, 0)
    need = load().pkm_memplus_backward_act8_workspace_size(ctypes.byref(a))
    workspace = _workspace(a, workspace, need, dev)
    _enqueue("pkm_memplus_backward_act8", (ctypes.byref(a),), dev)
    return dict(dy=dy, dx=dx, dW1=dW1, dW2=dW2)
