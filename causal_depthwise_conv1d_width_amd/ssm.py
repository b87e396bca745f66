"""Torch binding of include/ssm.h: the selective state space scan, its step and backward, and the
norms around a mixer block.  As in the package's other entry points, every function only checks tensor
metadata, marshals pointers, sizes and the current stream, and calls the library.

`stream`: the stream the kernels run on (None: the current one).  The caller orders it with the streams that the
arguments come from and go to; results and workspaces that a call makes itself are allocated on it."""
import collections
import ctypes

import torch

from . import _lib

SsmGrads = collections.namedtuple("SsmGrads", "dx ddt dA dB dC dD ddt_bias dinitial_state")


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(x, *tensors):
    """Every (tensor, name) must live on x's GPU.  Returns its index."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError(f"x: must be a GPU tensor (got device {x.device})")
    for t, name in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{name}: must be on {x.device}, the device of x (got {t.device})")
    return dev


def _stream(stream, dev):
    if stream is not None:
        return stream.cuda_stream
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _empty(like, shape, dtype, stream):
    """A new array for the kernels of `stream`.  Allocated there: memory of the current stream may still be
    used, now or after this call, by work that is not ordered with the kernels."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _result(like, shape, dtype, stream):
    """A new array for the caller, who may drop it while the current stream still uses it."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    t = _empty(like, shape, dtype, stream)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _rows(t, name, shape, dtype=_BF16):
    """(pointer, row stride) of [rows, ...] whose trailing dimensions are contiguous."""
    if t is None or t.shape != shape:
        raise ValueError(f"{name}: need a tensor of shape {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: need dtype {dtype} (got {t.dtype})")
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t.is_contiguous():
        return t.data_ptr(), width
    st = t.stride()
    if t.shape[0] > 0 and (st[-1] != 1 and shape[-1] > 1 or len(shape) == 3 and shape[1] > 1 and st[1] != shape[2]):
        raise ValueError(f"{name}: a row's elements must be contiguous")
    ld = st[0] if t.shape[0] > 1 else width
    if ld < width:
        raise ValueError(f"{name}: rows overlap")
    return t.data_ptr(), ld


def _vec(t, name, n, optional=True):
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name}: required")
    if t.shape != (n,) or t.dtype is not _F32 or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous float32 tensor of shape {(n,)}")
    return t.data_ptr()


def _ints(t, name, n):
    if t is None:
        return None
    if t.dtype is not _I32 or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: need a contiguous int32 tensor of at least {n} entries")
    return t.data_ptr()


def _flags(t, name, n):
    if t is None:
        return None
    if t.dtype not in (torch.bool, torch.uint8) or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name}: need a contiguous bool/uint8 tensor of at least {n} entries")
    return t.data_ptr()


def _seq(rows, cu_seqlens, seqlen):
    s = _lib.Seq()
    if cu_seqlens is not None:
        if seqlen is not None:
            raise ValueError("cu_seqlens and seqlen: give one of them")
        s.cu_seqlens = _ints(cu_seqlens, "cu_seqlens", 1)
        s.nseq = cu_seqlens.numel() - 1
        return s, s.nseq
    s.seqlen = int(seqlen) if seqlen is not None else max(rows, 1)
    if s.seqlen < 1 or rows % s.seqlen:
        raise ValueError(f"seqlen: must divide the {rows} rows")
    return s, rows // s.seqlen


def _shape(x, dt, B, dt_softplus):
    if x.dim() != 3 or B.dim() != 3:
        raise ValueError("x, B: need [rows, heads, head_dim] and [rows, groups, state] tensors")
    if dt.dtype is not _F32 and dt.dtype is not _BF16:
        raise ValueError("dt: dtype must be float32 or bfloat16")
    _, H, P = x.shape
    G, N = B.shape[1:]
    if min(H, P, G, N) < 1 or H % G or N > 256:
        raise ValueError("x, B: need heads divisible by groups and 1 <= state <= 256")
    return _lib.SsmShape(H, P, G, N, _lib.F32 if dt.dtype is _F32 else _lib.BF16, 1 if dt_softplus else 0)


def _state_array(t, name, H, P, N, least):
    """(pointer, slots, slot stride) of FP32 [slots, H, P, N] with contiguous slots."""
    if t.dim() != 4 or t.shape[1:] != (H, P, N) or t.dtype is not _F32:
        raise ValueError(f"{name}: need a float32 tensor [slots, {H}, {P}, {N}]")
    if t.shape[0] < least:
        raise ValueError(f"{name}: needs at least {least} states, has {t.shape[0]}")
    if not t.is_contiguous() and t.numel() and not t[0].is_contiguous():
        raise ValueError(f"{name}: a state must be contiguous")
    return t.data_ptr(), t.shape[0], (t.stride(0) if t.shape[0] > 1 else H * P * N)


def _work(x, need, workspace, stream):
    if workspace is None and need:
        workspace = _empty(x, (need,), torch.uint8, stream)
    if workspace is None:
        return None, None, 0
    if not workspace.is_contiguous():  # its bytes would not be its own
        raise ValueError("workspace: must be contiguous")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def ssm_scan_fwd_workspace_bytes(x, dt, B, nseq):
    """Workspace bytes of ssm_scan_fwd for these shapes and nseq sequences."""
    return int(_lib.load_ssm().ssm_scan_fwd_workspace_bytes(ctypes.byref(_shape(x, dt, B, True)), x.shape[0], nseq))


def ssm_scan_bwd_workspace_bytes(x, dt, B, nseq):
    """Workspace bytes of ssm_scan_bwd for these shapes and nseq sequences."""
    return int(_lib.load_ssm().ssm_scan_bwd_workspace_bytes(ctypes.byref(_shape(x, dt, B, True)), x.shape[0], nseq))


def norm_bwd_workspace_bytes(rows, d, group):
    return int(_lib.load_ssm().norm_bwd_workspace_bytes(rows, d, group))


def ssm_scan_fwd(x, dt, A, B, C, D=None, dt_bias=None, *, cu_seqlens=None, seqlen=None, dt_softplus=True,
                 state_pool=None, cache_indices=None, has_initial_state=None, initial_state=None, final_state=None,
                 out=None, workspace=None, stream=None):
    """y [rows, H, P] of the scan of x [rows, H, P], dt [rows, H], B, C [rows, G, N] (A, D, dt_bias: [H]).

    Sequences: cu_seqlens, or batch rows of seqlen rows (default: one sequence).  States: either a
    state_pool [slots, H, P, N] fp32 with cache_indices, read where has_initial_state is true (None:
    nowhere) and updated in place (as the convolution's conv_state), or initial_state / final_state [nseq, H, P, N]."""
    lib = _lib.load_ssm()
    sh = _shape(x, dt, B, dt_softplus)
    rows, H, P = x.shape
    G, N = B.shape[1:]
    seq, nseq = _seq(rows, cu_seqlens, seqlen)
    xp, xl = _rows(x, "x", (rows, H, P))
    dp, dl = _rows(dt, "dt", (rows, H), dt.dtype)
    Bp, Bl = _rows(B, "B", (rows, G, N))
    Cp, Cl = _rows(C, "C", (rows, G, N))
    Ap, Dp, bp = _vec(A, "A", H, False), _vec(D, "D", H), _vec(dt_bias, "dt_bias", H)
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
    dev = _on(x, (dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"), (dt_bias, "dt_bias"), (cu_seqlens, "cu_seqlens"),
              (state_pool, "state_pool"), (cache_indices, "cache_indices"), (has_initial_state, "has_initial_state"),
              (initial_state, "initial_state"), (final_state, "final_state"), (out, "out"), (workspace, "workspace"))
    if out is None:
        out = _result(x, (rows, H, P), _BF16, stream)
    yp, yl = _rows(out, "out", (rows, H, P))
    need = lib.ssm_scan_fwd_workspace_bytes(ctypes.byref(sh), rows, nseq)
    workspace, wp, wb = _work(x, need, workspace, stream)
    code = lib.ssm_scan_fwd(ctypes.byref(sh), rows, xp, xl, dp, dl, Ap, Bp, Bl, Cp, Cl, Dp, bp, ctypes.byref(seq),
                            ctypes.byref(st), yp, yl, wp, wb, _stream(stream, dev))
    _lib.check(lib, code, "ssm_scan_fwd")
    return out


def ssm_scan_bwd(dy, x, dt, A, B, C, D=None, dt_bias=None, *, cu_seqlens=None, seqlen=None, dt_softplus=True,
                 initial_state=None, dfinal_state=None, dx=None, ddt=None, dA=None, dB=None, dC=None, dD=None,
                 ddt_bias=None, dinitial_state=None, workspace=None, stream=None):
    """Gradients of ssm_scan_fwd as an SsmGrads tuple (dD, ddt_bias: None without D, dt_bias;
    dinitial_state: None without initial_state or an array for it).  dx, ddt, dB and dC may be given as
    column ranges of wider rows, e.g. one gradient array for the convolution's output."""
    lib = _lib.load_ssm()
    sh = _shape(x, dt, B, dt_softplus)
    rows, H, P = x.shape
    G, N = B.shape[1:]
    seq, nseq = _seq(rows, cu_seqlens, seqlen)
    gp, gl = _rows(dy, "dy", (rows, H, P))
    xp, xl = _rows(x, "x", (rows, H, P))
    dp, dl = _rows(dt, "dt", (rows, H), dt.dtype)
    Bp, Bl = _rows(B, "B", (rows, G, N))
    Cp, Cl = _rows(C, "C", (rows, G, N))
    Ap, Dp, bp = _vec(A, "A", H, False), _vec(D, "D", H), _vec(dt_bias, "dt_bias", H)
    dev = _on(x, (dy, "dy"), (dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"), (dt_bias, "dt_bias"),
              (cu_seqlens, "cu_seqlens"), (initial_state, "initial_state"), (dfinal_state, "dfinal_state"), (dx, "dx"),
              (ddt, "ddt"), (dA, "dA"), (dB, "dB"), (dC, "dC"), (dD, "dD"), (ddt_bias, "ddt_bias"),
              (dinitial_state, "dinitial_state"), (workspace, "workspace"))
    if dinitial_state is None and initial_state is not None:
        dinitial_state = _result(x, (nseq, H, P, N), _F32, stream)
    ptrs = []
    for t, name in ((initial_state, "initial_state"), (dfinal_state, "dfinal_state"), (dinitial_state, "dinitial_state")):
        if t is not None and (tuple(t.shape) != (nseq, H, P, N) or t.dtype != torch.float32 or not t.is_contiguous()):
            raise ValueError(f"{name}: need a contiguous float32 tensor of shape {(nseq, H, P, N)}")
        ptrs.append(t.data_ptr() if t is not None and nseq else None)

    def new(t, shape, dtype):
        return _result(x, shape, dtype, stream) if t is None else t

    dx, ddt = new(dx, (rows, H, P), torch.bfloat16), new(ddt, (rows, H), dt.dtype)
    dB, dC = new(dB, (rows, G, N), torch.bfloat16), new(dC, (rows, G, N), torch.bfloat16)
    dA = new(dA, (H,), torch.float32)
    if D is not None:
        dD = new(dD, (H,), torch.float32)
    if dt_bias is not None:
        ddt_bias = new(ddt_bias, (H,), torch.float32)
    need = lib.ssm_scan_bwd_workspace_bytes(ctypes.byref(sh), rows, nseq)
    workspace, wp, wb = _work(x, need, workspace, stream)
    code = lib.ssm_scan_bwd(ctypes.byref(sh), rows, gp, gl, xp, xl, dp, dl, Ap, Bp, Bl, Cp, Cl, Dp, bp, ctypes.byref(seq),
                            ptrs[0], ptrs[1], *_rows(dx, "dx", (rows, H, P)), *_rows(ddt, "ddt", (rows, H), dt.dtype),
                            _vec(dA, "dA", H), *_rows(dB, "dB", (rows, G, N)), *_rows(dC, "dC", (rows, G, N)),
                            _vec(dD, "dD", H), _vec(ddt_bias, "ddt_bias", H), ptrs[2], wp, wb, _stream(stream, dev))
    _lib.check(lib, code, "ssm_scan_bwd")
    return SsmGrads(dx, ddt, dA, dB, dC, dD, ddt_bias, dinitial_state)


def ssm_state_update(x, dt, A, B, C, D=None, dt_bias=None, *, state_pool, cache_indices, dt_softplus=True, out=None,
                     stream=None):
    """One token a sequence: x [nseq, H, P], dt [nseq, H], B, C [nseq, G, N]; state_pool slots advance in place."""
    lib = _lib.load_ssm()
    sh = _shape(x, dt, B, dt_softplus)
    n, H, P = x.shape
    G, N = B.shape[1:]
    xp, xl = _rows(x, "x", (n, H, P))
    dp, dl = _rows(dt, "dt", (n, H), dt.dtype)
    Bp, Bl = _rows(B, "B", (n, G, N))
    Cp, Cl = _rows(C, "C", (n, G, N))
    Ap, Dp, bp = _vec(A, "A", H, False), _vec(D, "D", H), _vec(dt_bias, "dt_bias", H)
    if state_pool is None or cache_indices is None:
        raise ValueError("state_pool, cache_indices: required")
    st = _lib.SsmStates()
    st.final, st.slots, st.s_slot = _state_array(state_pool, "state_pool", H, P, N, 1)
    st.initial = st.final
    st.cache_indices = _ints(cache_indices, "cache_indices", n)
    dev = _on(x, (dt, "dt"), (A, "A"), (B, "B"), (C, "C"), (D, "D"), (dt_bias, "dt_bias"), (state_pool, "state_pool"),
              (cache_indices, "cache_indices"), (out, "out"))
    if out is None:
        out = _result(x, (n, H, P), _BF16, stream)
    yp, yl = _rows(out, "out", (n, H, P))
    code = lib.ssm_state_update(ctypes.byref(sh), n, xp, xl, dp, dl, Ap, Bp, Bl, Cp, Cl, Dp, bp, ctypes.byref(st), yp, yl,
                                _stream(stream, dev))
    _lib.check(lib, code, "ssm_state_update")
    return out


# ------------------------------------------------------------------ norms
def _weight(w, d):
    if w is None or w.shape != (d,) or not w.is_contiguous() or (w.dtype is not _F32 and w.dtype is not _BF16):
        raise ValueError(f"weight: need a contiguous float32 or bfloat16 tensor of shape {(d,)}")
    return w.data_ptr(), _lib.F32 if w.dtype is _F32 else _lib.BF16


def _group(d, group_size):
    g = d if group_size is None else int(group_size)
    if g < 1 or d % g or g > 32768:
        raise ValueError(f"group_size: must divide the {d} channels and be at most 32768")
    return g


def _matrix(x, name):
    if x.dim() != 2:
        raise ValueError(f"{name}: need a 2-D tensor [rows, channels]")
    return x.shape[0], x.shape[1]


def gated_norm_fwd(x, gate, weight, *, group_size=None, norm_before_gate=False, eps=1e-5, out=None, stream=None):
    """RMS norm of x silu(gate) (or the norm of x, times silu(gate), with norm_before_gate) by groups of
    group_size channels (default: all), times weight.  x, gate, y: bf16 [rows, d]."""
    lib = _lib.load_ssm()
    rows, d = _matrix(x, "x")
    g = _group(d, group_size)
    xr, zr, (wp, wd) = _rows(x, "x", (rows, d)), _rows(gate, "gate", (rows, d)), _weight(weight, d)
    dev = _on(x, (gate, "gate"), (weight, "weight"), (out, "out"))
    if out is None:
        out = _result(x, (rows, d), _BF16, stream)
    code = lib.gated_norm_fwd(rows, d, g, *xr, *zr, wp, wd, int(bool(norm_before_gate)), eps, *_rows(out, "out", (rows, d)),
                              _stream(stream, dev))
    _lib.check(lib, code, "gated_norm_fwd")
    return out


def gated_norm_bwd(dy, x, gate, weight, *, group_size=None, norm_before_gate=False, eps=1e-5, dx=None, dgate=None,
                   dweight=None, workspace=None, stream=None):
    """(dx, dgate, dweight [d] fp32) of gated_norm_fwd."""
    lib = _lib.load_ssm()
    rows, d = _matrix(x, "x")
    g = _group(d, group_size)
    dyr, xr, zr = _rows(dy, "dy", (rows, d)), _rows(x, "x", (rows, d)), _rows(gate, "gate", (rows, d))
    wp, wd = _weight(weight, d)
    dev = _on(x, (dy, "dy"), (gate, "gate"), (weight, "weight"), (dx, "dx"), (dgate, "dgate"), (dweight, "dweight"),
              (workspace, "workspace"))
    dx = _result(x, (rows, d), _BF16, stream) if dx is None else dx
    dgate = _result(x, (rows, d), _BF16, stream) if dgate is None else dgate
    dweight = _result(x, (d,), _F32, stream) if dweight is None else dweight
    workspace, sp, sb = _work(x, lib.norm_bwd_workspace_bytes(rows, d, g), workspace, stream)
    code = lib.gated_norm_bwd(rows, d, g, *dyr, *xr, *zr, wp, wd, int(bool(norm_before_gate)), eps,
                              *_rows(dx, "dx", (rows, d)), *_rows(dgate, "dgate", (rows, d)), _vec(dweight, "dweight", d),
                              sp, sb, _stream(stream, dev))
    _lib.check(lib, code, "gated_norm_bwd")
    return dx, dgate, dweight


def _res_dtype(t, name):
    if t.dtype is not _F32 and t.dtype is not _BF16:
        raise ValueError(f"{name}: dtype must be float32 or bfloat16")
    return _lib.F32 if t.dtype is _F32 else _lib.BF16


def residual_norm_fwd(x, residual, weight, *, scale=1.0, eps=1e-5, out=None, residual_out=None, stream=None):
    """(y, residual_out): residual_out = residual + scale x in the residual's type (float32 or bfloat16;
    may be the residual itself), y = its RMS norm times weight.  x, y: bf16 [rows, d]."""
    lib = _lib.load_ssm()
    rows, d = _matrix(x, "x")
    _group(d, None)
    xr, rt = _rows(x, "x", (rows, d)), _res_dtype(residual, "residual")
    rr, (wp, wd) = _rows(residual, "residual", (rows, d), residual.dtype), _weight(weight, d)
    dev = _on(x, (residual, "residual"), (weight, "weight"), (out, "out"), (residual_out, "residual_out"))
    if out is None:
        out = _result(x, (rows, d), _BF16, stream)
    if residual_out is None:
        residual_out = _result(residual, (rows, d), residual.dtype, stream)
    code = lib.residual_norm_fwd(rows, d, *xr, *rr, rt, scale, wp, wd, eps, *_rows(out, "out", (rows, d)),
                                 *_rows(residual_out, "residual_out", (rows, d), residual.dtype), _stream(stream, dev))
    _lib.check(lib, code, "residual_norm_fwd")
    return out, residual_out


def residual_norm_bwd(dy, dresidual_out, residual_out, weight, *, scale=1.0, eps=1e-5, dx=None, dresidual=None,
                      dweight=None, workspace=None, stream=None):
    """(dx, dresidual, dweight [d] fp32) of residual_norm_fwd from its stored residual_out; dresidual_out
    is the gradient from residual_out's other reader (None: none; dresidual may be its buffer)."""
    lib = _lib.load_ssm()
    rows, d = _matrix(residual_out, "residual_out")
    _group(d, None)
    rdt = residual_out.dtype
    rt = _res_dtype(residual_out, "residual_out")
    dyr, ror = _rows(dy, "dy", (rows, d)), _rows(residual_out, "residual_out", (rows, d), rdt)
    drr = _rows(dresidual_out, "dresidual_out", (rows, d), rdt) if dresidual_out is not None else (None, 0)
    wp, wd = _weight(weight, d)
    dev = _on(residual_out, (dy, "dy"), (dresidual_out, "dresidual_out"), (weight, "weight"), (dx, "dx"),
              (dresidual, "dresidual"), (dweight, "dweight"), (workspace, "workspace"))
    dx = _result(dy, (rows, d), _BF16, stream) if dx is None else dx
    dresidual = _result(residual_out, (rows, d), rdt, stream) if dresidual is None else dresidual
    dweight = _result(dy, (d,), _F32, stream) if dweight is None else dweight
    workspace, sp, sb = _work(dy, lib.norm_bwd_workspace_bytes(rows, d, d), workspace, stream)
    code = lib.residual_norm_bwd(rows, d, *dyr, *drr, *ror, rt, scale, wp, wd, eps, *_rows(dx, "dx", (rows, d)),
                                 *_rows(dresidual, "dresidual", (rows, d), rdt), _vec(dweight, "dweight", d), sp, sb,
                                 _stream(stream, dev))
    _lib.check(lib, code, "residual_norm_bwd")
    return dx, dresidual, dweight
