"""Thin ctypes binding of libgdr (include/gdr.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, outputs are allocated with torch (as the operator contract's
loader infers and allocates them, "com.microsoft.GatedDeltaNet" README,
Use section), and the call goes to ``gdr_forward`` on torch's current
stream.  Every step of the computation runs in the library's HIP kernels;
there is no fallback, and a missing library raises ``GDRError``.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import NamedTuple, Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libgdr.so")
_lock = threading.Lock()
_lib = None

ABI_VERSION = 3  # GDR_ABI_VERSION of include/gdr.h the structs below mirror
GDR_OK, GDR_E_INVALID, GDR_E_UNSUPPORTED, GDR_E_ALIAS, GDR_E_WORKSPACE, GDR_E_HIP = range(6)
F32, F16, BF16, E4M3 = 0, 1, 2, 3
RULES = {"linear": 0, "gated": 1, "delta": 2, "gated_delta": 3, "gated_delta_v2": 4}
GATES = {"none": 0, "qwen": 1}
BETAS = {"none": 0, "sigmoid": 1}
ALGOS = {"auto": 0, "recurrent": 1, "decode": 2, "chunked": 3}
ALGO_NAMES = {v: k for k, v in ALGOS.items()}


class GDRError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s: %s" % (status, message))
        self.status = status


class Problem(ctypes.Structure):
    _fields_ = [
        ("total_tokens", ctypes.c_int64),
        ("batch", ctypes.c_int32),
        ("seq_len", ctypes.c_int32),
        ("num_heads_qk", ctypes.c_int32),
        ("num_heads_v", ctypes.c_int32),
        ("head_dim_k", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32),
        ("num_slots", ctypes.c_int32),
        ("act_dtype", ctypes.c_int32),
        ("gate_dtype", ctypes.c_int32),
        ("update_rule", ctypes.c_int32),
        ("gate_activation", ctypes.c_int32),
        ("beta_activation", ctypes.c_int32),
        ("qk_l2_norm", ctypes.c_int32),
        ("decay_per_key", ctypes.c_int32),
        ("rank4", ctypes.c_int32),
        ("chunk_size", ctypes.c_int32),
        ("algo", ctypes.c_int32),
        ("state_update_capacity", ctypes.c_int32),
        ("beta_per_token", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("scan_segments", ctypes.c_int32),
    ]


class Tensors(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "q", "k", "v", "o", "gate", "beta", "erase", "a_log", "dt_bias", "cu_seqlens",
        "slot_ids", "initial_state", "final_state", "gate_scale", "seq_lens")]


class GradientPointers(ctypes.Structure):
    """gdr_gradients"""
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "d_o", "d_final_state", "d_q", "d_k", "d_v", "d_gate", "d_beta", "d_initial_state", "d_a_log",
        "d_dt_bias", "d_gate_scale")] + [("zero_rest", ctypes.c_int32)]


EXPORTS = ("gdr_abi_version", "gdr_status_str", "gdr_last_error", "gdr_validate",
           "gdr_workspace_size", "gdr_select_algo", "gdr_forward", "gdr_forward_noalloc",
           "gdr_backward_workspace_size", "gdr_backward", "gdr_gate", "gdr_gate_backward_workspace_size",
           "gdr_gate_backward", "gdr_rms_norm", "gdr_rms_norm_backward_workspace_size", "gdr_rms_norm_backward",
           "gdr_slab_stream")
NOALLOC_SCRATCH_BYTES = 256 << 20  # GDR_NOALLOC_SCRATCH_BYTES of include/gdr.h


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Open libgdr.so (once).  Raises GDRError when it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise GDRError("GDR_E_HIP", "libgdr.so is not built (python -m gated_delta_rule_token_amd.build)")
        lib = ctypes.CDLL(_LIB_PATH)
        lib.gdr_abi_version.restype = ctypes.c_int
        if lib.gdr_abi_version() != ABI_VERSION:
            raise GDRError("GDR_E_HIP", "libgdr.so has ABI %d, this binding expects %d (rebuild it)"
                           % (lib.gdr_abi_version(), ABI_VERSION))
        lib.gdr_status_str.restype = ctypes.c_char_p
        lib.gdr_status_str.argtypes = [ctypes.c_int]
        lib.gdr_last_error.restype = ctypes.c_char_p
        lib.gdr_validate.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(Tensors)]
        lib.gdr_validate.restype = ctypes.c_int
        lib.gdr_workspace_size.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_size_t)]
        lib.gdr_workspace_size.restype = ctypes.c_int
        lib.gdr_select_algo.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_int32)]
        lib.gdr_select_algo.restype = ctypes.c_int
        lib.gdr_forward.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(Tensors), ctypes.c_void_p,
                                    ctypes.c_size_t, ctypes.c_void_p]
        lib.gdr_forward.restype = ctypes.c_int
        lib.gdr_forward_noalloc.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(Tensors), ctypes.c_void_p]
        lib.gdr_forward_noalloc.restype = ctypes.c_int
        lib.gdr_gate.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_void_p,
                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                 ctypes.c_void_p, ctypes.c_void_p]
        lib.gdr_gate.restype = ctypes.c_int
        lib.gdr_backward_workspace_size.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(ctypes.c_size_t)]
        lib.gdr_backward_workspace_size.restype = ctypes.c_int
        lib.gdr_backward.argtypes = [ctypes.POINTER(Problem), ctypes.POINTER(Tensors),
                                     ctypes.POINTER(GradientPointers), ctypes.c_void_p, ctypes.c_size_t,
                                     ctypes.c_void_p]
        lib.gdr_backward.restype = ctypes.c_int
        lib.gdr_gate_backward_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int32,
                                                         ctypes.POINTER(ctypes.c_size_t)]
        lib.gdr_gate_backward_workspace_size.restype = ctypes.c_int
        lib.gdr_gate_backward.argtypes = ([ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]
                                          + [ctypes.c_void_p] * 11 + [ctypes.c_size_t, ctypes.c_void_p])
        lib.gdr_gate_backward.restype = ctypes.c_int
        lib.gdr_rms_norm.argtypes = ([ctypes.c_int64] + [ctypes.c_int32] * 5 + [ctypes.c_float]
                                     + [ctypes.c_void_p] * 8)
        lib.gdr_rms_norm.restype = ctypes.c_int
        lib.gdr_rms_norm_backward_workspace_size.argtypes = [ctypes.c_int64, ctypes.c_int32,
                                                             ctypes.POINTER(ctypes.c_size_t)]
        lib.gdr_rms_norm_backward_workspace_size.restype = ctypes.c_int
        lib.gdr_rms_norm_backward.argtypes = ([ctypes.c_int64] + [ctypes.c_int32] * 3 + [ctypes.c_void_p] * 8
                                              + [ctypes.c_size_t, ctypes.c_void_p])
        lib.gdr_rms_norm_backward.restype = ctypes.c_int
        lib.gdr_slab_stream.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32,
                                        ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p]
        lib.gdr_slab_stream.restype = ctypes.c_int
        _lib = lib
        return lib


def check(status: int):
    if status != GDR_OK:
        lib = load_library()
        raise GDRError(lib.gdr_status_str(status).decode(), lib.gdr_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _enqueue(fn, dev, *args):
    """Call a library function on torch's current stream of ``dev``, with that
    device current (a launch needs its stream's device to be)."""
    if dev.index == torch.cuda.current_device():
        check(fn(*args, torch.cuda.current_stream(dev).cuda_stream))
    else:
        with torch.cuda.device(dev):
            check(fn(*args, torch.cuda.current_stream(dev).cuda_stream))


def _dtype_code(dt):
    if dt == torch.float32:
        return F32
    if dt == torch.float16:
        return F16
    if dt == torch.bfloat16:
        return BF16
    raise GDRError("GDR_E_INVALID", "unsupported dtype %s (float32, float16 or bfloat16)" % dt)


def _need(t, name, dtype=None, device=None):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise GDRError("GDR_E_INVALID", "%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise GDRError("GDR_E_INVALID", "%s must be on the GPU" % name)
    if device is not None and t.device != device:
        raise GDRError("GDR_E_INVALID", "%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise GDRError("GDR_E_INVALID", "%s must be contiguous" % name)
    if dtype is not None and t.dtype != dtype:
        raise GDRError("GDR_E_INVALID", "%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _int32(value, name):
    """``value`` as the C ABI's int32: ctypes would cut it to its low 32 bits."""
    value = int(value)
    if not -2 ** 31 <= value < 2 ** 31:
        raise GDRError("GDR_E_INVALID", "%s (%d) does not fit in 32 bits" % (name, value))
    return value


def build_problem(q, k, v, *, gate=None, beta=None, erase=None, a_log=None, dt_bias=None,
                  cu_seqlens=None, initial_state=None, slot_ids=None, state=None,
                  update_rule="gated_delta", gate_activation="none", beta_activation="none",
                  qk_l2_norm=False, scale=0.0, chunk_size=64, algo="auto", batch=None,
                  gate_scale=None, seq_lens=None, scan_segments=0):
    """Problem descriptor from tensor shapes (no device access)."""
    rank4 = q.dim() == 4
    if rank4:
        B, L, H, dk = q.shape
        T = B * L
    else:
        T, H, dk = q.shape
        if cu_seqlens is not None:
            B, L = cu_seqlens.shape[0] - 1, 0
        else:
            if batch is None:
                if initial_state is not None:
                    batch = initial_state.shape[0]
                elif slot_ids is not None:
                    batch = slot_ids.shape[0]
                elif seq_lens is not None:
                    batch = seq_lens.shape[0]
                else:
                    batch = 1
            B = int(batch)
            L = T // B if B else 0
    HV, dv = v.shape[-2], v.shape[-1]
    per_key = gate is not None and gate.dim() == q.dim()
    # beta (..., 1): one update rate per token for every value head
    beta_tok = beta is not None and HV > 1 and beta.dim() == q.dim() - 1 and beta.shape[-1] == 1
    p = Problem(
        total_tokens=T, batch=B, seq_len=L, num_heads_qk=H, num_heads_v=HV, head_dim_k=dk,
        head_dim_v=dv, num_slots=0 if state is None else state.shape[0],
        act_dtype=_dtype_code(q.dtype),
        gate_dtype=F32 if gate is None else _dtype_code(gate.dtype),
        update_rule=RULES[update_rule], gate_activation=GATES[gate_activation],
        beta_activation=BETAS[beta_activation], qk_l2_norm=int(bool(qk_l2_norm)),
        decay_per_key=int(per_key), rank4=int(rank4), chunk_size=int(chunk_size),
        algo=ALGOS[algo], state_update_capacity=0, beta_per_token=int(beta_tok), scale=float(scale),
        scan_segments=int(scan_segments))
    return p


def check_shapes(p: Problem, lead, shapes) -> None:
    """Shape check of every tensor of a call against the problem (shapes only,
    no device access).  ``lead`` is q's leading axes ((T,) or (B, L));
    ``shapes`` maps a tensor name to its shape, or None when it is absent.
    Raises GDRError(GDR_E_INVALID) on the first mismatch."""
    lead = tuple(lead)
    H, HV, dk, dv, B = p.num_heads_qk, p.num_heads_v, p.head_dim_k, p.head_dim_v, p.batch
    state = (HV, dv, dk)
    want = {
        "q": [lead + (H, dk)],
        "k": [lead + (H, dk)],
        "v": [lead + (HV, dv)],
        "out": [lead + (HV, dv)],
        "gate": [lead + (HV, dk)] if p.decay_per_key else [lead + (HV,)],
        "beta": [lead + (HV,), lead + (1,)],
        "erase": [lead + (HV, dk)],
        "a_log": [(HV,)],
        "gate_scale": [(HV,)],
        "dt_bias": [(HV, dk)] if p.decay_per_key else [(HV,)],
        "cu_seqlens": [(B + 1,)],
        "seq_lens": [(B,)],
        "slot_ids": [(B,)],
        "initial_state": [(B,) + state],
        "final_state": [(B,) + state],
        "state": [(p.num_slots,) + state],
    }
    for name, shape in shapes.items():
        if shape is None:
            continue
        shape = tuple(shape)
        ok = want.get(name)
        if ok is None:
            raise GDRError("GDR_E_INVALID", "unknown tensor %s" % name)
        if shape not in ok:
            raise GDRError("GDR_E_INVALID", "%s has shape %s, expected %s" % (
                name, shape, " or ".join(str(w) for w in ok)))


def _shapes(**tensors):
    return {k: (None if t is None else tuple(t.shape)) for k, t in tensors.items()}


def workspace_size(problem: Problem) -> int:
    n = ctypes.c_size_t(0)
    check(load_library().gdr_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return int(n.value)


def selected_algo(problem: Problem) -> str:
    a = ctypes.c_int32(0)
    check(load_library().gdr_select_algo(ctypes.byref(problem), ctypes.byref(a)))
    return ALGO_NAMES[a.value]


def _marshal(q, k, v, gate=None, beta=None, erase=None, a_log=None, dt_bias=None,
             cu_seqlens=None, initial_state=None, slot_ids=None, state=None,
             update_rule="gated_delta", gate_activation="none", beta_activation="none",
             qk_l2_norm=False, scale=0.0, chunk_size=64, algo="auto", out=None,
             final_state=None, batch=None, gate_scale=None, seq_lens=None, scan_segments=0):
    """Checked Problem and Tensors structs of one call, with its outputs
    (allocated when not given)."""
    dev = q.device
    _need(q, "q", device=dev)
    _need(k, "k", q.dtype, dev)
    _need(v, "v", q.dtype, dev)
    if gate is not None:
        _need(gate, "gate", device=dev)
    _need(beta, "beta", torch.float32, dev)
    _need(erase, "erase", torch.float32, dev)
    _need(a_log, "a_log", torch.float32, dev)
    _need(dt_bias, "dt_bias", torch.float32, dev)
    _need(gate_scale, "gate_scale", torch.float32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
    _need(slot_ids, "slot_ids", torch.int32, dev)
    _need(initial_state, "initial_state", torch.float32, dev)
    _need(state, "state", torch.float32, dev)
    if k.shape != q.shape:
        raise GDRError("GDR_E_INVALID", "k must have q's shape")
    if v.shape[:-2] != q.shape[:-2]:
        raise GDRError("GDR_E_INVALID", "v must share q's leading axes")
    p = build_problem(q, k, v, gate=gate, beta=beta, erase=erase, a_log=a_log, dt_bias=dt_bias,
                      cu_seqlens=cu_seqlens, initial_state=initial_state, slot_ids=slot_ids,
                      state=state, update_rule=update_rule, gate_activation=gate_activation,
                      beta_activation=beta_activation, qk_l2_norm=qk_l2_norm, scale=scale,
                      chunk_size=chunk_size, algo=algo, batch=batch, gate_scale=gate_scale,
                      seq_lens=seq_lens, scan_segments=scan_segments)
    HV, dv, dk = p.num_heads_v, p.head_dim_v, p.head_dim_k
    lead = tuple(q.shape[:-2])
    if out is None:
        out = torch.empty(lead + (HV, dv), dtype=q.dtype, device=dev)
    else:
        _need(out, "out", q.dtype, dev)
    if state is not None:
        fin = state
    elif final_state is not None:
        fin = _need(final_state, "final_state", torch.float32, dev)
    else:
        fin = torch.empty((p.batch, HV, dv, dk), dtype=torch.float32, device=dev)
    check_shapes(p, lead, _shapes(q=q, k=k, v=v, out=out, gate=gate, beta=beta, erase=erase,
                                  a_log=a_log, gate_scale=gate_scale, dt_bias=dt_bias,
                                  cu_seqlens=cu_seqlens, seq_lens=seq_lens, slot_ids=slot_ids,
                                  initial_state=initial_state,
                                  final_state=None if state is not None else fin, state=state))
    t = Tensors(q=_ptr(q), k=_ptr(k), v=_ptr(v), o=_ptr(out), gate=_ptr(gate), beta=_ptr(beta),
                erase=_ptr(erase), a_log=_ptr(a_log), dt_bias=_ptr(dt_bias),
                cu_seqlens=_ptr(cu_seqlens), slot_ids=_ptr(slot_ids),
                initial_state=_ptr(initial_state), final_state=_ptr(fin),
                gate_scale=_ptr(gate_scale), seq_lens=_ptr(seq_lens))
    return p, t, out, fin


def forward(q, k, v, *, workspace=None, **kw):
    """Run the gated delta rule on the GPU.

    q, k: (T,H,dk) or (B,L,H,dk); v: (T,HV,dv) or (B,L,HV,dv); gate (log
    decay, or the raw projection with gate_activation='qwen'): (...,HV) or
    per key (...,HV,dk); beta: (...,HV) fp32, or (...,1) for one rate per
    token; erase: (...,HV,dk) fp32.
    Raw-gate arm: dt_bias (HV,) or (HV,dk) beside a per-key gate, and either
    a_log (HV,) or the folded gate_scale = -exp(a_log) (HV,).  seq_lens (B,)
    int32 bounds each uniform-packed request to its first seq_lens[b] tokens
    (rows past it in ``o`` are left as they are).  scan_segments: for the
    chunked form, 0 lets the library choose, 1 runs each request's chunks in
    one serial pass, n > 1 splits that chain into n composed segments.
    With ``state`` (a slab (num_slots,HV,dv,dk) fp32) and ``slot_ids``, the
    slab is updated in place and returned as the second result; otherwise a
    final state (B,HV,dv,dk) is allocated (or ``final_state`` is filled).
    ``workspace``: a uint8 device tensor for the chunked form (allocated here
    when not given).  Returns (o, final_state).
    """
    lib = load_library()
    p, t, out, fin = _marshal(q, k, v, **kw)
    ws_bytes = workspace_size(p)
    if ws_bytes and workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=q.device)
    ws_have = 0
    if workspace is not None:
        _need(workspace, "workspace", device=q.device)
        ws_have = workspace.numel() * workspace.element_size()
    stream = torch.cuda.current_stream(q.device).cuda_stream
    # the library checks the real size against what the problem needs
    check(lib.gdr_forward(ctypes.byref(p), ctypes.byref(t), _ptr(workspace), ws_have, stream))
    return out, fin


def forward_noalloc(q, k, v, **kw):
    """``forward`` through gdr_forward_noalloc: the library serves the
    workspace from its own fixed device array (up to NOALLOC_SCRATCH_BYTES);
    nothing is allocated for it.  Same arguments as ``forward`` without
    ``workspace``; outputs are allocated here unless ``out`` / ``final_state``
    / ``state`` are given.  Returns (o, final_state)."""
    lib = load_library()
    p, t, out, fin = _marshal(q, k, v, **kw)
    stream = torch.cuda.current_stream(q.device).cuda_stream
    check(lib.gdr_forward_noalloc(ctypes.byref(p), ctypes.byref(t), stream))
    return out, fin


def gate(a, dt_bias, decay_scale, b=None, want_beta=False, out_decay=None, out_beta=None):
    """Standalone gate fusion ("com.microsoft.LinearAttentionGate"):
    decay = decay_scale * softplus(a + dt_bias), beta = sigmoid(b) if wanted.
    The last axis of ``a`` is the head axis.  Returns (decay, beta-or-None)."""
    lib = load_library()
    dev = a.device
    _need(a, "a", device=dev)
    _need(dt_bias, "dt_bias", torch.float32, dev)
    _need(decay_scale, "decay_scale", torch.float32, dev)
    if b is not None:
        _need(b, "b", a.dtype, dev)
    heads = a.shape[-1]
    decay = out_decay if out_decay is not None else torch.empty_like(a)
    beta = None
    if want_beta:
        beta = out_beta if out_beta is not None else torch.empty_like(a)
    stream = torch.cuda.current_stream(dev).cuda_stream
    check(lib.gdr_gate(a.numel(), heads, _dtype_code(a.dtype), _ptr(a), _ptr(dt_bias),
                       _ptr(decay_scale), _ptr(b), _ptr(decay), _ptr(beta), stream))
    return decay, beta


class Gradients(NamedTuple):
    """Results of ``backward``; None where the call has no such input (or, for
    ``initial_state``, where it was not wanted)."""
    q: torch.Tensor
    k: torch.Tensor
    v: torch.Tensor
    gate: Optional[torch.Tensor]
    beta: Optional[torch.Tensor]
    initial_state: Optional[torch.Tensor]
    a_log: Optional[torch.Tensor]
    dt_bias: Optional[torch.Tensor]
    gate_scale: Optional[torch.Tensor]


_TOKEN_ROWS = ("q", "k", "v", "gate", "beta")


def backward_workspace_size(problem: Problem) -> int:
    n = ctypes.c_size_t(0)
    check(load_library().gdr_backward_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return int(n.value)


def backward(q, k, v, d_o, *, gate=None, beta=None, a_log=None, dt_bias=None, gate_scale=None, cu_seqlens=None,
             seq_lens=None, initial_state=None, d_final_state=None, want_initial_state=None,
             update_rule="gated_delta", gate_activation="none", beta_activation="none", qk_l2_norm=False,
             scale=0.0, batch=None, out=None, workspace=None) -> Gradients:
    """Gradients of ``forward``: the inputs of that call, ``d_o`` (o's shape
    and dtype) and optionally ``d_final_state`` (B,HV,dv,dk) fp32, for the
    rules 'linear', 'gated', 'delta' and 'gated_delta' with one log decay per
    value head.  Nothing of the forward call has to be kept.

    The gradients have their tensors' shapes and dtypes; beta and a raw gate
    get theirs as given (through the sigmoid, the softplus and the L2 norm).
    ``want_initial_state``: whether the initial states' gradient is returned
    (default: when there is an initial state, or ``out`` holds a tensor for
    it; with False such a tensor is left alone).  Rows of tokens that no
    request covers are zero, or left as they are in a gradient passed in
    ``out`` (a ``Gradients`` whose tensors are filled; None entries are
    allocated; a tensor for an input that the call does not have is refused).
    ``workspace``: a uint8 device tensor of ``backward_workspace_size`` bytes
    (allocated here when not given)."""
    lib = load_library()
    dev = q.device
    _need(q, "q", device=dev)
    for name, t, dt in (("k", k, q.dtype), ("v", v, q.dtype), ("d_o", d_o, q.dtype), ("gate", gate, None),
                        ("beta", beta, torch.float32), ("a_log", a_log, torch.float32),
                        ("dt_bias", dt_bias, torch.float32), ("gate_scale", gate_scale, torch.float32),
                        ("cu_seqlens", cu_seqlens, torch.int32), ("seq_lens", seq_lens, torch.int32),
                        ("initial_state", initial_state, torch.float32),
                        ("d_final_state", d_final_state, torch.float32)):
        _need(t, name, dt, dev)
    if k is None or v is None or d_o is None:
        raise GDRError("GDR_E_INVALID", "k, v and d_o are required")
    if batch is None and initial_state is None and d_final_state is not None and d_final_state.dim() == 4:
        batch = d_final_state.shape[0]
    p = build_problem(q, k, v, gate=gate, beta=beta, a_log=a_log, dt_bias=dt_bias, cu_seqlens=cu_seqlens,
                      initial_state=initial_state, update_rule=update_rule, gate_activation=gate_activation,
                      beta_activation=beta_activation, qk_l2_norm=qk_l2_norm, scale=scale, batch=batch,
                      gate_scale=gate_scale, seq_lens=seq_lens)
    need = backward_workspace_size(p)
    lead = tuple(q.shape[:-2])
    states = (p.batch, p.num_heads_v, p.head_dim_v, p.head_dim_k)
    check_shapes(p, lead, _shapes(q=q, k=k, v=v, out=d_o, gate=gate, beta=beta, a_log=a_log, dt_bias=dt_bias,
                                  gate_scale=gate_scale, cu_seqlens=cu_seqlens, seq_lens=seq_lens,
                                  initial_state=initial_state, final_state=d_final_state))
    if want_initial_state is None:
        want_initial_state = initial_state is not None or (out is not None and out.initial_state is not None)
    grads, zero_rest = {}, out is None
    for name, like in (("q", q), ("k", k), ("v", v), ("gate", gate), ("beta", beta), ("initial_state", None),
                       ("a_log", a_log), ("dt_bias", dt_bias), ("gate_scale", gate_scale)):
        if like is None and not (name == "initial_state" and want_initial_state):
            if out is not None and getattr(out, name) is not None and name != "initial_state":
                raise GDRError("GDR_E_INVALID", "out.%s given, but the call has no %s" % (name, name))
            grads[name] = None
            continue
        shape, dtype = (states, torch.float32) if like is None else (tuple(like.shape), like.dtype)
        given = None if out is None else getattr(out, name)
        if given is None:
            # beside gradients of the caller's, whose other rows stay, zeros go into the new ones here
            given = (torch.empty if zero_rest or name not in _TOKEN_ROWS else torch.zeros)(shape, dtype=dtype, device=dev)
        elif tuple(_need(given, "out." + name, dtype, dev).shape) != shape:
            raise GDRError("GDR_E_INVALID", "out.%s has shape %s, expected %s" % (name, tuple(given.shape), shape))
        grads[name] = given
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    t = Tensors(q=_ptr(q), k=_ptr(k), v=_ptr(v), gate=_ptr(gate), beta=_ptr(beta), a_log=_ptr(a_log),
                dt_bias=_ptr(dt_bias), cu_seqlens=_ptr(cu_seqlens), initial_state=_ptr(initial_state),
                gate_scale=_ptr(gate_scale), seq_lens=_ptr(seq_lens))
    g = GradientPointers(d_o=_ptr(d_o), d_final_state=_ptr(d_final_state), zero_rest=int(zero_rest),
                         **{"d_" + name: _ptr(x) for name, x in grads.items()})
    _enqueue(lib.gdr_backward, dev, ctypes.byref(p), ctypes.byref(t), ctypes.byref(g), _ptr(workspace),
             workspace.numel() * workspace.element_size())
    return Gradients(**grads)


class GateGradients(NamedTuple):
    """Results of ``gate_backward``; ``b`` is None without the update rate."""
    a: torch.Tensor
    b: Optional[torch.Tensor]
    dt_bias: torch.Tensor
    decay_scale: torch.Tensor


def gate_backward(a, dt_bias, decay_scale, d_decay, b=None, d_beta=None, workspace=None) -> GateGradients:
    """Gradients of ``gate``: ``d_decay`` (and ``d_beta``, with ``b``) have
    a's shape and dtype; the gradients of dt_bias and decay_scale are sums
    over every row, in fp32.  The last axis of ``a`` is the head axis."""
    lib = load_library()
    dev = a.device
    _need(a, "a", device=dev)
    heads = _int32(a.shape[-1] if a.dim() else 0, "the last axis of a")
    if (b is None) != (d_beta is None):
        raise GDRError("GDR_E_INVALID", "b and d_beta must be given together")
    for name, t in (("d_decay", d_decay), ("b", b), ("d_beta", d_beta)):
        _need(t, name, a.dtype, dev)
        if t is not None and t.shape != a.shape:
            raise GDRError("GDR_E_INVALID", "%s must have a's shape" % name)
    for name, t in (("dt_bias", dt_bias), ("decay_scale", decay_scale)):
        if tuple(_need(t, name, torch.float32, dev).shape) != (heads,):
            raise GDRError("GDR_E_INVALID", "%s must have shape (%d,)" % (name, heads))
    n = ctypes.c_size_t(0)
    check(lib.gdr_gate_backward_workspace_size(a.numel(), heads, ctypes.byref(n)))
    if workspace is None:
        workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    g = GateGradients(torch.empty_like(a), None if b is None else torch.empty_like(b),
                      torch.empty_like(dt_bias), torch.empty_like(decay_scale))
    _enqueue(lib.gdr_gate_backward, dev, a.numel(), heads, _dtype_code(a.dtype), _ptr(a), _ptr(dt_bias),
             _ptr(decay_scale), _ptr(b), _ptr(d_decay), _ptr(d_beta), _ptr(g.a), _ptr(g.b), _ptr(g.dt_bias),
             _ptr(g.decay_scale), _ptr(workspace), workspace.numel() * workspace.element_size())
    return g


class NormOutput(NamedTuple):
    """Results of ``rms_norm``: ``scale`` with an 8-bit output, ``residual``
    with a residual, ``inv_rms`` when wanted; None otherwise."""
    y: torch.Tensor
    scale: Optional[torch.Tensor]
    residual: Optional[torch.Tensor]
    inv_rms: Optional[torch.Tensor]


def _norm_rows(x, weight):
    _need(x, "x", device=x.device)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise GDRError("GDR_E_INVALID", "x needs a last axis of at least one column")
    width = _int32(x.shape[-1], "the last axis of x")
    if weight is not None:
        _need(weight, "weight", device=x.device)
        if tuple(weight.shape) != (width,):
            raise GDRError("GDR_E_INVALID", "weight has shape %s, expected %s" % (tuple(weight.shape), (width,)))
    return x.numel() // width, width


def rms_norm(x, weight=None, *, residual=None, eps=1e-6, out_dtype=None, group=0, want_inv_rms=False,
             residual_out=None) -> NormOutput:
    """Root-mean-square norm over the last axis of ``x`` (fp32, fp16 or bf16):
    y = r / sqrt(mean(r^2) + eps) * weight with r = x + residual, rounded to
    x's dtype and returned as ``residual`` (written into ``residual_out`` when
    given, which may be ``residual`` itself).  ``weight`` has x's dtype or
    fp32.  ``out_dtype=torch.float8_e4m3fn`` gives y in 8 bits with
    ``scale`` = max |y| / 448 over the row (shape (..., 1)), or over each
    ``group`` columns (a power of two from 8 to 512).  ``want_inv_rms``: also
    return 1 / sqrt(mean(r^2) + eps) per row, which ``rms_norm_backward`` takes."""
    lib = load_library()
    dev = x.device
    group = _int32(group, "group")
    rows, width = _norm_rows(x, weight)
    _need(residual, "residual", x.dtype, dev)
    if residual is not None and residual.shape != x.shape:
        raise GDRError("GDR_E_INVALID", "residual must have x's shape")
    if residual_out is not None:
        if residual is None:
            raise GDRError("GDR_E_INVALID", "residual_out given without residual")
        if _need(residual_out, "residual_out", x.dtype, dev).shape != x.shape:
            raise GDRError("GDR_E_INVALID", "residual_out must have x's shape")
    elif residual is not None:
        residual_out = torch.empty_like(x)
    code = _dtype_code(x.dtype)
    if out_dtype is None or out_dtype == x.dtype:
        out_code, y, scale = code, torch.empty_like(x), None
    elif out_dtype == torch.float8_e4m3fn:
        groups = -(-width // group) if group > 0 else 1
        out_code, y = E4M3, torch.empty(x.shape, dtype=out_dtype, device=dev)
        scale = torch.empty(tuple(x.shape[:-1]) + (groups,), dtype=torch.float32, device=dev)
    else:
        raise GDRError("GDR_E_INVALID", "out_dtype must be x's dtype or torch.float8_e4m3fn, got %s" % out_dtype)
    inv = torch.empty(x.shape[:-1], dtype=torch.float32, device=dev) if want_inv_rms else None
    _enqueue(lib.gdr_rms_norm, dev, rows, width, code, code if weight is None else _dtype_code(weight.dtype), out_code,
             group, float(eps), _ptr(x), _ptr(residual), _ptr(weight), _ptr(y), _ptr(scale), _ptr(residual_out),
             _ptr(inv))
    return NormOutput(y, scale, residual_out, inv)


class NormGradients(NamedTuple):
    """Results of ``rms_norm_backward``; ``weight`` (fp32) is None without one."""
    x: torch.Tensor
    weight: Optional[torch.Tensor]


def rms_norm_backward(d_y, x, weight, inv_rms, *, d_residual=None, workspace=None) -> NormGradients:
    """Gradients of ``rms_norm`` (with y in x's dtype).  ``x`` is what was
    normalised: the forward call's ``residual`` result, or its x without one;
    ``inv_rms`` is its result.  ``d_residual`` is the gradient of the
    ``residual`` result, if any.  The returned gradient ``x`` is that of x and
    of the residual alike; ``weight``'s is a sum over every row, in fp32."""
    lib = load_library()
    dev = x.device
    rows, width = _norm_rows(x, weight)
    for name, t in (("d_y", d_y), ("d_residual", d_residual)):
        _need(t, name, x.dtype, dev)
        if t is not None and t.shape != x.shape:
            raise GDRError("GDR_E_INVALID", "%s must have x's shape" % name)
    if d_y is None or inv_rms is None:
        raise GDRError("GDR_E_INVALID", "d_y and inv_rms are required")
    if _need(inv_rms, "inv_rms", torch.float32, dev).shape != x.shape[:-1]:
        raise GDRError("GDR_E_INVALID", "inv_rms must have x's leading axes")
    d_x = torch.empty_like(x)
    d_weight = None
    if weight is not None:
        d_weight = torch.empty(width, dtype=torch.float32, device=dev)
        if workspace is None:
            n = ctypes.c_size_t(0)
            check(lib.gdr_rms_norm_backward_workspace_size(rows, width, ctypes.byref(n)))
            workspace = torch.empty(n.value, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", device=dev)
    code = _dtype_code(x.dtype)
    _enqueue(lib.gdr_rms_norm_backward, dev, rows, width, code, code if weight is None else _dtype_code(weight.dtype),
             _ptr(d_y), _ptr(x), _ptr(weight), _ptr(inv_rms), _ptr(d_residual), _ptr(d_x), _ptr(d_weight),
             _ptr(workspace), 0 if workspace is None else workspace.numel() * workspace.element_size())
    return NormGradients(d_x, d_weight)


def slab_stream(slab, slot_ids, factor=1.0):
    """Multiply in place by ``factor`` the state matrices ``slab[slot_ids[b]]``
    (every head) and nothing else: the state traffic of a decode step over the
    same slot ids, with no compute (a measurement aid).  ``slab`` is fp32
    (num_slots, HV, dv, dk) on the GPU, ``slot_ids`` int32 (B,)."""
    lib = load_library()
    dev = slab.device
    _need(slab, "slab", torch.float32, dev)
    _need(slot_ids, "slot_ids", torch.int32, dev)
    if slab.dim() != 4:
        raise ValueError("slab must be (num_slots, HV, dv, dk)")
    stream = torch.cuda.current_stream(dev).cuda_stream
    check(lib.gdr_slab_stream(_ptr(slab), _ptr(slot_ids), slot_ids.numel(), slab.shape[1],
                              slab.shape[2] * slab.shape[3], slab.shape[0], float(factor), stream))


class Prepared:
    """A gdr_forward call with its argument structs built once (for timing
    loops and replay): ``run()`` only re-issues the C call on the current
    stream.  Holds references to every tensor it points at."""

    def __init__(self, q, k, v, **kw):
        lib = load_library()
        self._lib = lib
        self.o, self.final_state = None, None
        dev = q.device
        p = build_problem(q, k, v, **{key: kw.get(key) for key in (
            "gate", "beta", "erase", "a_log", "dt_bias", "cu_seqlens", "initial_state",
            "slot_ids", "state", "gate_scale", "seq_lens")}, **{key: kw[key] for key in (
                "update_rule", "gate_activation", "beta_activation", "qk_l2_norm", "scale",
                "chunk_size", "algo", "batch", "scan_segments") if key in kw})
        HV, dv, dk = p.num_heads_v, p.head_dim_v, p.head_dim_k
        out = kw.get("out")
        if out is None:
            out = torch.empty(tuple(q.shape[:-2]) + (HV, dv), dtype=q.dtype, device=dev)
        fin = kw.get("state")
        if fin is None:
            fin = kw.get("final_state")
        if fin is None:
            fin = torch.empty((p.batch, HV, dv, dk), dtype=torch.float32, device=dev)
        g = kw.get
        check_shapes(p, tuple(q.shape[:-2]), _shapes(
            q=q, k=k, v=v, out=out, gate=g("gate"), beta=g("beta"), erase=g("erase"),
            a_log=g("a_log"), gate_scale=g("gate_scale"), dt_bias=g("dt_bias"),
            cu_seqlens=g("cu_seqlens"), seq_lens=g("seq_lens"), slot_ids=g("slot_ids"),
            initial_state=g("initial_state"),
            final_state=None if g("state") is not None else fin, state=g("state")))
        ws = workspace_size(p)
        self.workspace = torch.empty(ws, dtype=torch.uint8, device=dev) if ws else None
        self.tensors = dict(kw, q=q, k=k, v=v, out=out, fin=fin)
        self.t = Tensors(q=_ptr(q), k=_ptr(k), v=_ptr(v), o=_ptr(out), gate=_ptr(g("gate")),
                         beta=_ptr(g("beta")), erase=_ptr(g("erase")), a_log=_ptr(g("a_log")),
                         dt_bias=_ptr(g("dt_bias")), cu_seqlens=_ptr(g("cu_seqlens")),
                         slot_ids=_ptr(g("slot_ids")), initial_state=_ptr(g("initial_state")),
                         final_state=_ptr(fin), gate_scale=_ptr(g("gate_scale")),
                         seq_lens=_ptr(g("seq_lens")))
        self.p = p
        self.ws_bytes = ws
        self.algo = selected_algo(p)
        self.o, self.final_state = out, fin
        check(lib.gdr_validate(ctypes.byref(self.p), ctypes.byref(self.t)))

    def run(self, stream=None):
        if stream is None:
            stream = torch.cuda.current_stream(self.o.device).cuda_stream
        check(self._lib.gdr_forward(ctypes.byref(self.p), ctypes.byref(self.t),
                                    _ptr(self.workspace), self.ws_bytes, stream))
        return self.o, self.final_state


def prepare(q, k, v, **kw) -> Prepared:
    return Prepared(q, k, v, **kw)
