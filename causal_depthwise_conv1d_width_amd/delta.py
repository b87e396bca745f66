"""Torch binding of include/delta.h: the gated delta rule over packed rows, its step and backward, the layer norm, and
copies between slots of the pools.  As in the package's other entry points, every function only checks tensor metadata,
marshals pointers, sizes and the current stream, and calls the library.

`stream`: the stream the kernels run on (None: the current one).  The caller orders it with the streams that the
arguments come from and go to; results and workspaces that a call makes itself are allocated on it."""
import collections
import ctypes

import torch

from . import _lib
from .ssm import (_BF16, _F32, _flags, _ints, _matrix, _on, _res_dtype, _result, _rows, _seq, _state_array, _stream, _vec,
                  _weight, _work)

DeltaGrads = collections.namedtuple("DeltaGrads", "dq dk dv ddt db dA ddt_bias dinitial_state")
LayerNormGrads = collections.namedtuple("LayerNormGrads", "dx dresidual dweight dbias")


def _shape(q, k, v, dt, b, dt_softplus, qk_norm, scale, beta_max, norm_eps):
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k, v: need [rows, groups, state], [rows, groups, state] and [rows, heads, head_dim] tensors")
    if (dt.dtype is not _F32 and dt.dtype is not _BF16) or b.dtype is not dt.dtype:
        raise ValueError("dt, b: need one dtype, float32 or bfloat16")
    _, H, P = v.shape
    G, N = k.shape[1:]
    if min(H, P, G, N) < 1 or H % G or N > 256:
        raise ValueError("k, v: need heads divisible by groups and 1 <= state <= 256")
    scale = N ** -0.5 if scale is None else float(scale)
    norm_eps = float(norm_eps)
    beta_max = float(beta_max)
    if not 0 <= norm_eps < float("inf"):
        raise ValueError(f"norm_eps: must be finite and not negative (got {norm_eps})")
    if not 0 < beta_max < float("inf"):
        raise ValueError(f"beta_max: must be finite and positive (got {beta_max})")
    if not abs(scale) < float("inf"):
        raise ValueError(f"scale: must be finite (got {scale})")
    return _lib.DeltaShape(H, P, G, N, _lib.F32 if dt.dtype is _F32 else _lib.BF16, int(bool(dt_softplus)),
                           int(bool(qk_norm)), scale, beta_max, norm_eps)


def _inputs(q, k, v, dt, b, A, dt_bias):
    """Pointers and row strides in the order of the C calls."""
    rows, H, P = v.shape
    G, N = k.shape[1:]
    return (*_rows(q, "q", (rows, G, N)), *_rows(k, "k", (rows, G, N)), *_rows(v, "v", (rows, H, P)),
            *_rows(dt, "dt", (rows, H), dt.dtype), *_rows(b, "b", (rows, H), dt.dtype), _vec(A, "A", H, False),
            _vec(dt_bias, "dt_bias", H))


def _plain_shape(v, k, dt):
    return _shape(k, k, v, dt, dt, True, True, None, 1.0, 0.0)


def delta_scan_fwd_workspace_bytes(v, k, dt, nseq):
    """Workspace bytes of delta_scan_fwd for these shapes and nseq sequences."""
    return int(_lib.load_delta().delta_scan_fwd_workspace_bytes(ctypes.byref(_plain_shape(v, k, dt)), v.shape[0], nseq))


def delta_scan_bwd_workspace_bytes(v, k, dt, nseq):
    """Workspace bytes of delta_scan_bwd for these shapes and nseq sequences."""
    return int(_lib.load_delta().delta_scan_bwd_workspace_bytes(ctypes.byref(_plain_shape(v, k, dt)), v.shape[0], nseq))


def delta_scan_fwd(q, k, v, dt, b, A, dt_bias=None, *, scale=None, qk_norm=True, beta_max=1.0, norm_eps=1e-6,
                   dt_softplus=True, cu_seqlens=None, seqlen=None, state_pool=None, cache_indices=None,
                   has_initial_state=None, initial_state=None, final_state=None, out=None, workspace=None, stream=None):
    """y [rows, H, P] of the gated delta rule for q, k [rows, G, N], v [rows, H, P], dt, b [rows, H] (A, dt_bias: [H]).

    decay = exp(A softplus(dt + dt_bias)), rate = beta_max sigmoid(b), scale: N ** -0.5 by default; with qk_norm the rule
    takes q and k of norm one (norm_eps is added to the squared norm).  Sequences and states are those of ssm_scan_fwd: a
    state_pool [slots, H, P, N] fp32 with cache_indices, or initial_state / final_state [nseq, H, P, N]."""
    lib = _lib.load_delta()
    sh = _shape(q, k, v, dt, b, dt_softplus, qk_norm, scale, beta_max, norm_eps)
    rows, H, P = v.shape
    N = k.shape[2]
    seq, nseq = _seq(rows, cu_seqlens, seqlen)
    args = _inputs(q, k, v, dt, b, A, dt_bias)
    st = _lib.SsmStates()
    if state_pool is not None:
        if initial_state is not None or final_state is not None:
            raise ValueError("state_pool: not together with initial_state or final_state")
        if cache_indices is None:
            raise ValueError("cache_indices: required with state_pool")
        st.final, st.slots, st.s_slot = _state_array(state_pool, "state_pool", H, P, N, 1)
        st.cache_indices = _ints(cache_indices, "cache_indices", nseq)
        st.has_initial_state = _flags(has_initial_state, "has_initial_state", nseq)
        st.initial = st.final
    else:
        if cache_indices is not None or has_initial_state is not None:
            raise ValueError("cache_indices, has_initial_state: need a state_pool")
        for t, name in ((initial_state, "initial_state"), (final_state, "final_state")):
            if t is not None:
                p, n, s = _state_array(t, name, H, P, N, nseq)
                if n != nseq or (n > 1 and s != H * P * N):
                    raise ValueError(f"{name}: need a contiguous tensor of {nseq} states")
                st.slots, st.s_slot = max(n, 1), H * P * N
                setattr(st, "initial" if name == "initial_state" else "final", p if n else None)
    dev = _on(v, (q, "q"), (k, "k"), (dt, "dt"), (b, "b"), (A, "A"), (dt_bias, "dt_bias"), (cu_seqlens, "cu_seqlens"),
              (state_pool, "state_pool"), (cache_indices, "cache_indices"), (has_initial_state, "has_initial_state"),
              (initial_state, "initial_state"), (final_state, "final_state"), (out, "out"), (workspace, "workspace"))
    if out is None:
        out = _result(v, (rows, H, P), _BF16, stream)
    yp, yl = _rows(out, "out", (rows, H, P))
    workspace, wp, wb = _work(v, lib.delta_scan_fwd_workspace_bytes(ctypes.byref(sh), rows, nseq), workspace, stream)
    code = lib.delta_scan_fwd(ctypes.byref(sh), rows, *args, ctypes.byref(seq), ctypes.byref(st), yp, yl, wp, wb,
                              _stream(stream, dev))
    _lib.check(lib, code, "delta_scan_fwd")
    return out


def delta_scan_bwd(dy, q, k, v, dt, b, A, dt_bias=None, *, scale=None, qk_norm=True, beta_max=1.0, norm_eps=1e-6,
                   dt_softplus=True, cu_seqlens=None, seqlen=None, initial_state=None, dfinal_state=None, dq=None, dk=None,
                   dv=None, ddt=None, db=None, dA=None, ddt_bias=None, dinitial_state=None, workspace=None, stream=None):
    """Gradients of delta_scan_fwd as a DeltaGrads tuple (ddt_bias: None without dt_bias; dinitial_state: None without
    initial_state or an array for it).  dq, dk, dv, ddt and db may be given as column ranges of wider rows, e.g. one
    gradient array for the convolution's output."""
    lib = _lib.load_delta()
    sh = _shape(q, k, v, dt, b, dt_softplus, qk_norm, scale, beta_max, norm_eps)
    rows, H, P = v.shape
    G, N = k.shape[1:]
    seq, nseq = _seq(rows, cu_seqlens, seqlen)
    args = _inputs(q, k, v, dt, b, A, dt_bias)
    dev = _on(v, (dy, "dy"), (q, "q"), (k, "k"), (dt, "dt"), (b, "b"), (A, "A"), (dt_bias, "dt_bias"),
              (cu_seqlens, "cu_seqlens"), (initial_state, "initial_state"), (dfinal_state, "dfinal_state"), (dq, "dq"),
              (dk, "dk"), (dv, "dv"), (ddt, "ddt"), (db, "db"), (dA, "dA"), (ddt_bias, "ddt_bias"),
              (dinitial_state, "dinitial_state"), (workspace, "workspace"))
    if dinitial_state is None and initial_state is not None:
        dinitial_state = _result(v, (nseq, H, P, N), _F32, stream)
    ptrs = []
    for t, name in ((initial_state, "initial_state"), (dfinal_state, "dfinal_state"), (dinitial_state, "dinitial_state")):
        if t is not None and (tuple(t.shape) != (nseq, H, P, N) or t.dtype != _F32 or not t.is_contiguous()):
            raise ValueError(f"{name}: need a contiguous float32 tensor of shape {(nseq, H, P, N)}")
        ptrs.append(t.data_ptr() if t is not None and nseq else None)

    def new(t, shape, dtype):
        return _result(v, shape, dtype, stream) if t is None else t

    dyr = _rows(dy, "dy", (rows, H, P))
    dq, dk, dv = new(dq, (rows, G, N), _BF16), new(dk, (rows, G, N), _BF16), new(dv, (rows, H, P), _BF16)
    ddt, db, dA = new(ddt, (rows, H), dt.dtype), new(db, (rows, H), dt.dtype), new(dA, (H,), _F32)
    if dt_bias is not None:
        ddt_bias = new(ddt_bias, (H,), _F32)
    workspace, wp, wb = _work(v, lib.delta_scan_bwd_workspace_bytes(ctypes.byref(sh), rows, nseq), workspace, stream)
    code = lib.delta_scan_bwd(ctypes.byref(sh), rows, *dyr, *args, ctypes.byref(seq), ptrs[0], ptrs[1],
                              *_rows(dq, "dq", (rows, G, N)), *_rows(dk, "dk", (rows, G, N)), *_rows(dv, "dv", (rows, H, P)),
                              *_rows(ddt, "ddt", (rows, H), dt.dtype), *_rows(db, "db", (rows, H), dt.dtype),
                              _vec(dA, "dA", H), _vec(ddt_bias, "ddt_bias", H), ptrs[2], wp, wb, _stream(stream, dev))
    _lib.check(lib, code, "delta_scan_bwd")
    return DeltaGrads(dq, dk, dv, ddt, db, dA, ddt_bias, dinitial_state)


def delta_state_update(q, k, v, dt, b, A, dt_bias=None, *, state_pool, cache_indices, scale=None, qk_norm=True,
                       beta_max=1.0, norm_eps=1e-6, dt_softplus=True, out=None, stream=None):
    """One token a sequence: q, k [nseq, G, N], v [nseq, H, P], dt, b [nseq, H]; state_pool slots advance in place."""
    lib = _lib.load_delta()
    sh = _shape(q, k, v, dt, b, dt_softplus, qk_norm, scale, beta_max, norm_eps)
    n, H, P = v.shape
    args = _inputs(q, k, v, dt, b, A, dt_bias)
    if state_pool is None or cache_indices is None:
        raise ValueError("state_pool, cache_indices: required")
    st = _lib.SsmStates()
    st.final, st.slots, st.s_slot = _state_array(state_pool, "state_pool", H, P, k.shape[2], 1)
    st.initial = st.final
    st.cache_indices = _ints(cache_indices, "cache_indices", n)
    dev = _on(v, (q, "q"), (k, "k"), (dt, "dt"), (b, "b"), (A, "A"), (dt_bias, "dt_bias"), (state_pool, "state_pool"),
              (cache_indices, "cache_indices"), (out, "out"))
    if out is None:
        out = _result(v, (n, H, P), _BF16, stream)
    yp, yl = _rows(out, "out", (n, H, P))
    code = lib.delta_state_update(ctypes.byref(sh), n, *args, ctypes.byref(st), yp, yl, _stream(stream, dev))
    _lib.check(lib, code, "delta_state_update")
    return out


# ------------------------------------------------------------------ layer norm
def layer_norm_bwd_workspace_bytes(rows, d):
    return int(_lib.load_delta().layer_norm_bwd_workspace_bytes(rows, d))


def _channels(d):
    if not 1 <= d <= 32768:
        raise ValueError(f"x: needs 1 to 32768 channels (got {d})")


def layer_norm_fwd(x, weight, bias=None, *, residual=None, scale=1.0, eps=1e-5, out=None, residual_out=None, stream=None):
    """(y, residual_out): the layer norm of x, times weight plus bias (None: zero), and None; or, with a residual (float32 or
    bfloat16), that of residual_out = residual + scale x, which may be the residual itself.  x, y: bf16 [rows, d]."""
    lib = _lib.load_delta()
    rows, d = _matrix(x, "x")
    _channels(d)
    xr, (wp, wd) = _rows(x, "x", (rows, d)), _weight(weight, d)
    bp = None
    if bias is not None:
        if bias.dtype is not weight.dtype:
            raise ValueError(f"bias: need weight's dtype {weight.dtype} (got {bias.dtype})")
        bp = _weight(bias, d)[0]
    if residual is None and (residual_out is not None or scale != 1.0):
        raise ValueError("residual_out, scale: need a residual")
    dev = _on(x, (residual, "residual"), (weight, "weight"), (bias, "bias"), (out, "out"), (residual_out, "residual_out"))
    if out is None:
        out = _result(x, (rows, d), _BF16, stream)
    rr, rt, ro = (None, 0), _lib.BF16, (None, 0)
    if residual is not None:
        rt, rr = _res_dtype(residual, "residual"), _rows(residual, "residual", (rows, d), residual.dtype)
        if residual_out is None:
            residual_out = _result(residual, (rows, d), residual.dtype, stream)
        ro = _rows(residual_out, "residual_out", (rows, d), residual.dtype)
        if rows == 0:
            rr = ro = (None, 0)
    code = lib.layer_norm_fwd(rows, d, *xr, *rr, rt, scale, wp, bp, wd, eps, *_rows(out, "out", (rows, d)), *ro,
                              _stream(stream, dev))
    _lib.check(lib, code, "layer_norm_fwd")
    return out, residual_out


def layer_norm_bwd(dy, normed, weight, *, residual=False, dresidual_out=None, scale=1.0, eps=1e-5, dx=None, dresidual=None,
                   dweight=None, dbias=None, workspace=None, stream=None):
    """Gradients of layer_norm_fwd as a LayerNormGrads tuple from what it normed: x, or, with residual=True, its stored
    residual_out (then dresidual in its dtype and dx = scale dresidual; otherwise dresidual is None).  dresidual_out is the
    gradient from normed's other reader (None: none; dresidual may be its buffer)."""
    lib = _lib.load_delta()
    rows, d = _matrix(normed, "normed")
    _channels(d)
    hdt = normed.dtype
    ht = _res_dtype(normed, "normed")
    dyr, hr = _rows(dy, "dy", (rows, d)), _rows(normed, "normed", (rows, d), hdt)
    drr = _rows(dresidual_out, "dresidual_out", (rows, d), hdt) if dresidual_out is not None else (None, 0)
    wp, wd = _weight(weight, d)
    if not residual and (dresidual is not None or scale != 1.0):
        raise ValueError("dresidual, scale: need residual=True")
    dev = _on(normed, (dy, "dy"), (dresidual_out, "dresidual_out"), (weight, "weight"), (dx, "dx"), (dresidual, "dresidual"),
              (dweight, "dweight"), (dbias, "dbias"), (workspace, "workspace"))
    dx = _result(dy, (rows, d), _BF16, stream) if dx is None else dx
    if residual and dresidual is None:
        dresidual = _result(normed, (rows, d), hdt, stream)
    dweight = _result(dy, (d,), _F32, stream) if dweight is None else dweight
    dbias = _result(dy, (d,), _F32, stream) if dbias is None else dbias
    workspace, sp, sb = _work(dy, lib.layer_norm_bwd_workspace_bytes(rows, d), workspace, stream)
    dr = _rows(dresidual, "dresidual", (rows, d), hdt) if residual else (None, 0)
    code = lib.layer_norm_bwd(rows, d, *dyr, *drr, *hr, ht, scale, wp, wd, eps, *_rows(dx, "dx", (rows, d)), *dr,
                              _vec(dweight, "dweight", d), _vec(dbias, "dbias", d), sp, sb, _stream(stream, dev))
    _lib.check(lib, code, "layer_norm_bwd")
    return LayerNormGrads(dx, dresidual, dweight, dbias)


# ------------------------------------------------------------------ slots
def _slots(t, name):
    """The pool's descriptor: any dtype, slots first, each slot's elements without gaps in some order of the dimensions."""
    if t.dim() < 1:
        raise ValueError(f"{name}: need a tensor [slots, ...]")
    size = t.element_size()
    want = 1
    for stride, n in sorted((st, n) for st, n in zip(t.stride()[1:], t.shape[1:]) if n > 1):
        if stride != want:
            raise ValueError(f"{name}: a slot's elements must lie without gaps")
        want *= n
    if 0 in t.shape:
        want = 0
    stride = t.stride(0) if t.shape[0] > 1 else want
    if stride < want:
        raise ValueError(f"{name}: slots overlap")
    return _lib.SlotPool(t.data_ptr() if want else None, t.shape[0], want * size, stride * size)


def state_copy(pools, source, target, *, stream=None):
    """Slot target[i] of every pool becomes what its slot source[i] held before the call, or zeros where source[i] is
    negative: forks, swaps and moves of sequences, and cleared slots.  pools: a tensor [slots, ...] or up to 8 of them (the
    convolution's, the scan's and the delta rule's states), source and target: int32 [n], targets distinct; a target of -1
    leaves the pools as they are."""
    lib = _lib.load_delta()
    pools = [pools] if isinstance(pools, torch.Tensor) else list(pools)
    if not 1 <= len(pools) <= 8:
        raise ValueError(f"pools: need 1 to 8 tensors (got {len(pools)})")
    if source.dim() != 1 or target.shape != source.shape:
        raise ValueError("source, target: need one-dimensional tensors of the same length")
    n = source.numel()
    if n > 8192:
        raise ValueError(f"source: at most 8192 pairs (got {n})")
    sp, tp = _ints(source, "source", n), _ints(target, "target", n)
    names = ["pools"] if len(pools) == 1 else [f"pools[{i}]" for i in range(len(pools))]
    arr = (_lib.SlotPool * len(pools))(*(_slots(t, name) for t, name in zip(pools, names)))
    dev = pools[0].get_device()
    if dev < 0:
        raise ValueError(f"{names[0]}: must be a GPU tensor (got device {pools[0].device})")
    for t, name in (*zip(pools, names), (source, "source"), (target, "target")):
        if t.get_device() != dev:
            raise ValueError(f"{name}: must be on {pools[0].device}, the device of {names[0]} (got {t.device})")
    _lib.check(lib, lib.state_copy(arr, len(pools), n, sp, tp, _stream(stream, dev)), "state_copy")
