"""Linear attention with one decay per head, and beam search over decode steps:
the Python side of ``include/gdr_ops.h``, in the manner of the package's other
entry points (argument checks and allocation here, everything else in libgdr).

  head_decay_fwd(q, k, v, g, ...)               -> (o, s_final)   prefill, training's forward pass
  head_decay_fwd_varlen(q, k, v, g, cu_seqlens) -> (o, s_final)   packed batch
  head_decay_bwd(q, k, v, g, d_o, ...)          -> dict of gradients
  head_decay_bwd_varlen(q, k, v, g, d_o, cu_seqlens, ...) -> dict of gradients
  head_decay_step(q, k, v, g, state, ...)       -> o              one decode token
  beam_select(logits, scores, ...)              -> (scores, tokens, parents, done)
  beam_reorder(state, parents, ...)             -> state

q, k, v (and d_o) may be views with strides, as slices of one fused projection
are: the last dimension contiguous, every row 16-byte aligned.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import F32, BF16, GdrError, _used_on, load_library

__all__ = ["head_decay_fwd", "head_decay_fwd_varlen", "head_decay_bwd", "head_decay_bwd_varlen", "head_decay_step",
           "head_decay_fwd_workspace_size", "head_decay_bwd_workspace_size", "beam_select",
           "beam_select_workspace_size", "beam_reorder", "HeadDecayDesc", "make_head_decay_desc"]

_CODE = {torch.float32: F32, torch.bfloat16: BF16}
_I64x3 = ctypes.c_int64 * 3


class HeadDecayDesc(ctypes.Structure):
    """Mirror of ``gdr_head_decay_desc`` in include/gdr_ops.h."""
    _fields_ = [("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32), ("Hk", ctypes.c_int32),
                ("Dk", ctypes.c_int32), ("Dv", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q_stride", _I64x3), ("k_stride", _I64x3), ("v_stride", _I64x3), ("do_stride", _I64x3)]


def _code(t: torch.dtype) -> int:
    if t not in _CODE:
        raise TypeError(f"unsupported dtype {t}; use float32 or bfloat16")
    return _CODE[t]


def make_head_decay_desc(B, T, H, Hk, Dk, Dv, *, dtype, scale=1.0, q_stride=None, k_stride=None, v_stride=None,
                         do_stride=None) -> HeadDecayDesc:
    """Strides (sequence, token, head) in elements; None: contiguous [B, T, heads, width]."""
    def of(stride, heads, width):
        return _I64x3(*(stride if stride is not None else (T * heads * width, heads * width, width)))
    return HeadDecayDesc(B, T, H, Hk, Dk, Dv, _code(dtype), scale, of(q_stride, H, Dk), of(k_stride, Hk, Dk),
                         of(v_stride, Hk, Dv), of(do_stride, H, Dv))


def _device(q):
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.device.type != "cuda":
        raise ValueError("q must be a GPU tensor")
    return q.device


def _check_any(name, t, device, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if (t.device, t.dtype, t.shape) == (device, dtype, shape):
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _check_view(name, t, device, dtype, shape):
    """A tensor that may be strided, but for its last dimension."""
    _check_any(name, t, device, dtype, shape)
    if t.stride(-1) != 1 and shape[-1] > 1 and t.numel() > 0:  # (strides of nothing do not matter)
        raise ValueError(f"the last dimension of {name} must be contiguous")


def _check_dev(name, t, device, dtype=None, shape=None):
    _check_any(name, t, device, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# the handle of torch's current stream, without the Stream object around it where torch offers that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _strides(t, dims):
    """(sequence, token, head) strides of a tensor of which ``dims`` are there."""
    st = t.stride()
    return st[:3] if dims == 3 else (0, st[0], st[1]) if dims == 2 else (st[0], 0, st[1])


def _call(dev, name, *args):
    """The library call, on the tensors' device."""
    fn = getattr(load_library(), name)
    if dev.index == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args)
    if rc != 0:
        raise GdrError(rc, name)


def _on(stream, dev, fresh):
    """The handle of the stream the work is enqueued on: ``stream``, or torch's current stream of ``dev``.
    ``fresh``: tensors allocated here, on the current stream."""
    if stream is None:
        return _raw_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    _used_on(stream, dev, *fresh)
    return stream.cuda_stream


def _workspace(workspace, need, dev, fresh):
    if workspace is None:
        if need == 0:
            return None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        fresh.append(workspace)
    else:
        _check_dev("workspace", workspace, dev, torch.uint8)
    return workspace


def _size(name, *args):
    out = ctypes.c_size_t(0)
    rc = getattr(load_library(), name)(*args, ctypes.byref(out))
    if rc != 0:
        raise GdrError(rc, name)
    return int(out.value)


def head_decay_fwd_workspace_size(desc: HeadDecayDesc, packed: bool = False) -> int:
    return _size("gdr_head_decay_fwd_workspace_size", ctypes.byref(desc), int(packed))


def head_decay_bwd_workspace_size(desc: HeadDecayDesc, packed: bool = False, need_dg: bool = True) -> int:
    return _size("gdr_head_decay_bwd_workspace_size", ctypes.byref(desc), int(packed), int(need_dg))


@functools.lru_cache(maxsize=1024)
def _described(kind, need_dg, B, T, H, Hk, Dk, Dv, dtype, scale, *strides):
    """(reference to the descriptor, workspace bytes) of a call: both follow from sizes and strides alone, and a
    program's calls repeat them.  kind: "fwd", "bwd" (a second letter p: packed) or "step"."""
    desc = make_head_decay_desc(B, T, H, Hk, Dk, Dv, dtype=dtype, scale=scale, q_stride=strides[0],
                                k_stride=strides[1], v_stride=strides[2],
                                do_stride=strides[3] if len(strides) > 3 else (0, 0, 0))
    if kind == "step":
        return ctypes.byref(desc), 0
    if kind.startswith("fwd"):
        return ctypes.byref(desc), head_decay_fwd_workspace_size(desc, kind == "fwdp")
    return ctypes.byref(desc), head_decay_bwd_workspace_size(desc, kind == "bwdp", need_dg)


def _tokens(q, k, v, g, cu_seqlens):
    """Checks of a whole-sequence call's inputs: (device, packed, B, T, H, Hk, Dk, Dv, token shape)."""
    dev = _device(q)
    packed = cu_seqlens is not None
    if q.dim() != (3 if packed else 4):
        raise ValueError(f"q must have {3 if packed else 4} dimensions, it has {q.dim()}")
    _code(q.dtype)
    if not isinstance(k, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("k and v must be torch.Tensors")
    if k.dim() != q.dim() or v.dim() != q.dim():
        raise ValueError("q, k and v must have the same number of dimensions")
    if packed:
        _check_dev("cu_seqlens", cu_seqlens, dev, torch.int32)
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be a 1-d int32 tensor of N + 1 entries")
        B, T = cu_seqlens.numel() - 1, q.shape[0]
    else:
        B, T = q.shape[:2]
    H, Dk = q.shape[-2:]
    Hk, Dv = k.shape[-2], v.shape[-1]
    lead = tuple(q.shape[:-2])
    if Hk == 0 and H > 0 or Hk > 0 and H % Hk:
        raise ValueError(f"{H} query heads cannot share {Hk} key/value heads")
    _check_view("q", q, dev, q.dtype, (*lead, H, Dk))
    _check_view("k", k, dev, q.dtype, (*lead, Hk, Dk))
    _check_view("v", v, dev, q.dtype, (*lead, Hk, Dv))
    _check_dev("g", g, dev, torch.float32, (H,))
    return dev, packed, B, T, H, Hk, Dk, Dv, lead


def _fwd(q, k, v, g, cu_seqlens, scale, s0, output_final_state, s_final, o, workspace, stream):
    dev, packed, B, T, H, Hk, Dk, Dv, lead = _tokens(q, k, v, g, cu_seqlens)
    state = (B, H, Dk, Dv)
    if s0 is not None:
        _check_dev("s0", s0, dev, torch.float32, state)
    fresh = []
    if o is None:
        o = torch.empty((*lead, H, Dv), dtype=q.dtype, device=dev)
        fresh.append(o)
    else:
        _check_dev("o", o, dev, q.dtype, (*lead, H, Dv))
    if s_final is not None:
        _check_dev("s_final", s_final, dev, torch.float32, state)
    elif output_final_state:
        s_final = torch.empty(state, dtype=torch.float32, device=dev)
        fresh.append(s_final)
    dims = 2 if packed else 3
    desc, need = _described("fwdp" if packed else "fwd", False, B, T, H, Hk, Dk, Dv, q.dtype, float(scale),
                            _strides(q, dims), _strides(k, dims), _strides(v, dims))
    workspace = _workspace(workspace, need, dev, fresh)
    st = _on(stream, dev, fresh)
    _call(dev, "gdr_head_decay_fwd", desc, _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
          _ptr(s0), _ptr(o), _ptr(s_final), _ptr(workspace), 0 if workspace is None else workspace.numel(),
          st)
    return o, s_final


def head_decay_fwd(q, k, v, g, *, scale: float = 1.0, s0=None, output_final_state: bool = True, s_final=None, o=None,
                   workspace=None, stream=None):
    """Linear attention with a decay per head, S_t = exp(g_h) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.

    q [B,T,H,Dk], k [B,T,Hk,Dk], v [B,T,Hk,Dv] in float32 or bfloat16 (views
    allowed; Hk divides H, query head h reads key/value head h // (H // Hk);
    widths multiples of 8 up to 256); g float32 [H], the log-decays (<= 0);
    s0 float32 [B,H,Dk,Dv] or None.  Returns (o [B,T,H,Dv] in q's dtype,
    s_final float32 [B,H,Dk,Dv] or None); ``s_final`` may be ``s0`` itself.
    """
    return _fwd(q, k, v, g, None, scale, s0, output_final_state, s_final, o, workspace, stream)


def head_decay_fwd_varlen(q, k, v, g, cu_seqlens, *, scale: float = 1.0, s0=None, output_final_state: bool = True,
                          s_final=None, o=None, workspace=None, stream=None):
    """``head_decay_fwd`` of N packed sequences: q [T,H,Dk], k [T,Hk,Dk], v
    [T,Hk,Dv], sequence n being tokens cu_seqlens[n] .. cu_seqlens[n+1]-1
    (int32 [N+1] on the device); s0, s_final [N,H,Dk,Dv].  Rows of o outside
    every sequence are left unwritten."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _fwd(q, k, v, g, cu_seqlens, scale, s0, output_final_state, s_final, o, workspace, stream)


def _bwd(q, k, v, g, d_o, cu_seqlens, scale, s0, ds_final, need_dg, need_ds0, workspace, stream):
    dev, packed, B, T, H, Hk, Dk, Dv, lead = _tokens(q, k, v, g, cu_seqlens)
    _check_view("d_o", d_o, dev, q.dtype, (*lead, H, Dv))
    state = (B, H, Dk, Dv)
    if s0 is not None:
        _check_dev("s0", s0, dev, torch.float32, state)
    if ds_final is not None:
        _check_dev("ds_final", ds_final, dev, torch.float32, state)
    out = {"dq": torch.empty((*lead, H, Dk), dtype=q.dtype, device=dev),
           "dk": torch.empty((*lead, Hk, Dk), dtype=q.dtype, device=dev),
           "dv": torch.empty((*lead, Hk, Dv), dtype=q.dtype, device=dev),
           "dg": torch.zeros((H,), dtype=torch.float32, device=dev) if need_dg and B == 0 else
           torch.empty((H,), dtype=torch.float32, device=dev) if need_dg else None,
           "ds0": torch.empty(state, dtype=torch.float32, device=dev) if need_ds0 else None}
    if B == 0 and T > 0:  # packed tokens of no sequence
        for x in ("dq", "dk", "dv"):
            out[x].zero_()
    fresh = list(out.values())
    dims = 2 if packed else 3
    desc, need = _described("bwdp" if packed else "bwd", bool(need_dg), B, T, H, Hk, Dk, Dv, q.dtype, float(scale),
                            _strides(q, dims), _strides(k, dims), _strides(v, dims), _strides(d_o, dims))
    workspace = _workspace(workspace, need, dev, fresh)
    st = _on(stream, dev, fresh)
    _call(dev, "gdr_head_decay_bwd", desc, _ptr(cu_seqlens), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
          _ptr(s0), _ptr(d_o), _ptr(ds_final), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dg"]),
          _ptr(out["ds0"]), _ptr(workspace), 0 if workspace is None else workspace.numel(),
          st)
    return out


def head_decay_bwd(q, k, v, g, d_o, *, scale: float = 1.0, s0=None, ds_final=None, need_dg: bool = True,
                   need_ds0: bool = True, workspace=None, stream=None):
    """Backward pass of ``head_decay_fwd``: inputs as there, d_o [B,T,H,Dv] in
    q's dtype (a view allowed), ds_final float32 [B,H,Dk,Dv] or None.  Returns a
    dict: dq, dk, dv in q's dtype with the inputs' shapes (dk and dv summed over
    the query heads that share them), dg float32 [H] (None unless ``need_dg``:
    fixed decays need none, and without it no chunk states are kept) and ds0
    float32 (None unless ``need_ds0``)."""
    return _bwd(q, k, v, g, d_o, None, scale, s0, ds_final, need_dg, need_ds0, workspace, stream)


def head_decay_bwd_varlen(q, k, v, g, d_o, cu_seqlens, *, scale: float = 1.0, s0=None, ds_final=None,
                          need_dg: bool = True, need_ds0: bool = True, workspace=None, stream=None):
    """``head_decay_bwd`` of N packed sequences (tensors as for
    ``head_decay_fwd_varlen``).  Rows of dq, dk and dv outside every sequence
    are zero."""
    if cu_seqlens is None:
        raise TypeError("cu_seqlens must be a torch.Tensor")
    return _bwd(q, k, v, g, d_o, cu_seqlens, scale, s0, ds_final, need_dg, need_ds0, workspace, stream)


def head_decay_step(q, k, v, g, state, *, scale: float = 1.0, slots=None, parents=None, state_out=None, o=None,
                    stream=None):
    """One decode token: q [N,H,Dk], k [N,Hk,Dk], v [N,Hk,Dv] (views allowed), g float32 [H].

    state float32 [M,H,Dk,Dv].  In place (no ``state_out``): row n updates
    state[n], or state[slots[n]] (int32 [N]; a slot outside [0, M) is a padded
    row: its output is zero, no state is touched; of rows with the same slot the
    first has it).  With ``state_out`` [N,H,Dk,Dv]: row n continues from
    state[n], or from state[parents[n]] (int32 [N], may repeat; outside [0, M):
    from a zero state), and state is only read.  Returns o [N,H,Dv].
    """
    dev = _device(q)
    if q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q, k and v must have 3 dimensions")
    _code(q.dtype)
    N, H, Dk = q.shape
    Hk, Dv = k.shape[1], v.shape[2]
    if Hk == 0 and H > 0 or Hk > 0 and H % Hk:
        raise ValueError(f"{H} query heads cannot share {Hk} key/value heads")
    _check_view("q", q, dev, q.dtype, (N, H, Dk))
    _check_view("k", k, dev, q.dtype, (N, Hk, Dk))
    _check_view("v", v, dev, q.dtype, (N, Hk, Dv))
    _check_dev("g", g, dev, torch.float32, (H,))
    _check_dev("state", state, dev, torch.float32)
    if state.dim() != 4 or tuple(state.shape[1:]) != (H, Dk, Dv):
        raise ValueError(f"state has shape {tuple(state.shape)}, expected (M, {H}, {Dk}, {Dv})")
    if slots is not None:
        if state_out is not None:
            raise ValueError("slots work in place: pass no state_out (parents go with state_out)")
        _check_dev("slots", slots, dev, torch.int32, (N,))
    if parents is not None:
        if state_out is None:
            raise ValueError("parents need state_out: beams may share a parent")
        _check_dev("parents", parents, dev, torch.int32, (N,))
    if state_out is not None:
        _check_dev("state_out", state_out, dev, torch.float32, (N, H, Dk, Dv))
    fresh = []
    if o is None:
        o = torch.empty((N, H, Dv), dtype=q.dtype, device=dev)
        fresh.append(o)
    else:
        _check_dev("o", o, dev, q.dtype, (N, H, Dv))
    desc, _ = _described("step", False, N, 1, H, Hk, Dk, Dv, q.dtype, float(scale), _strides(q, 1), _strides(k, 1),
                         _strides(v, 1))
    st = _on(stream, dev, fresh)
    _call(dev, "gdr_head_decay_step", desc, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(state),
          state.shape[0], _ptr(slots), _ptr(parents), _ptr(state_out), _ptr(o), st)
    return o


@functools.lru_cache(maxsize=1024)
def beam_select_workspace_size(B: int, K: int, V: int) -> int:
    return _size("gdr_beam_select_workspace_size", B, K, V)


def beam_select(logits, scores, *, done=None, eos_token: int = -1, pad_token: int = 0, workspace=None, stream=None):
    """One step of beam search for B requests of K beams (at most 32).

    logits [B,K,V] in float32 or bfloat16 (rows evenly spaced, as a slice of a
    padded output layer is); scores float32 [B,K], the beams' sums of
    log-probabilities (-inf for beams that do not count yet); done bool [B,K] or
    None.  The candidates of a beam are its score plus the log-softmax of its
    logits; a finished beam offers ``pad_token`` at its own score.  Returns, best
    first: scores float32, tokens int32, parents int32 (the beam that each
    continues) and done bool (the parent was, or the token is ``eos_token``),
    all [B,K].  Equal candidates go to the lower beam, then the lower token;
    what is not a finite number counts as -inf.
    """
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    dev = logits.device
    if dev.type != "cuda":
        raise ValueError("logits must be a GPU tensor")
    if logits.dim() != 3:
        raise ValueError(f"logits must have 3 dimensions, it has {logits.dim()}")
    B, K, V = logits.shape
    row = logits.stride(1) if K > 1 else logits.stride(0)
    if logits.numel() > 0 and ((V > 1 and logits.stride(2) != 1) or (B > 1 and logits.stride(0) != K * row)):
        raise ValueError("logits must have contiguous rows, evenly spaced")
    _check_dev("scores", scores, dev, torch.float32, (B, K))
    if done is not None:
        _check_dev("done", done, dev, torch.bool, (B, K))
    tokens = torch.empty_like(scores, dtype=torch.int32)
    out = (torch.empty_like(scores), tokens, torch.empty_like(tokens), torch.empty_like(scores, dtype=torch.bool))
    fresh = list(out)
    workspace = _workspace(workspace, beam_select_workspace_size(B, K, V), dev, fresh)
    st = _on(stream, dev, fresh)
    _call(dev, "gdr_beam_select", B, K, V, _code(logits.dtype), _ptr(logits), row, _ptr(scores), _ptr(done),
          eos_token, pad_token, *(_ptr(x) for x in out), _ptr(workspace),
          0 if workspace is None else workspace.numel(), st)
    return out


def beam_reorder(state, parents, *, dim: int = 0, out=None, stream=None):
    """The beams' states after a selection: new[.., b, k, ..] = state[.., b, parents[b, k], ..].

    state: any dtype, contiguous, dimensions ``dim`` and ``dim + 1`` of size B and
    K (dim 0: [B,K,..]; dim 1: [L,B,K,..], the layers of a model at once), the
    part behind them a multiple of 16 bytes; parents int32 [B,K] (K at most 32;
    outside [0, K) a beam keeps its state).  In place unless ``out`` (shaped as
    state) is given; returns the reordered tensor.
    """
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a torch.Tensor")
    dev = state.device
    if dev.type != "cuda":
        raise ValueError("state must be a GPU tensor")
    _check_dev("state", state, dev)
    if dim < 0 or state.dim() < dim + 2:
        raise ValueError(f"state of {state.dim()} dimensions has no beams at dimensions {dim}, {dim + 1}")
    B, K = state.shape[dim:dim + 2]
    _check_dev("parents", parents, dev, torch.int32, (B, K))
    if out is None:
        out = state
    else:
        _check_dev("out", out, dev, state.dtype, state.shape)
    L, row = 1, state.element_size()
    for x in state.shape[:dim]:
        L *= x
    for x in state.shape[dim + 2:]:
        row *= x
    st = _on(stream, dev, ())
    _call(dev, "gdr_beam_reorder", L, B, K, row, _ptr(state), _ptr(parents), _ptr(out),
          st)
    return out
