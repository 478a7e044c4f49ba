"""Thin ctypes binding of ``libgdn_b200.so`` (argument marshalling only).

Every step of the computation runs in the library's CUDA kernels; torch is
used here only to allocate device tensors and to name the current stream.
There is no CPU fallback: if the library is missing the call raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdn_b200.so")

GDN_DTYPE_BF16 = 0
GDN_DTYPE_F32 = 1

STATUS = {
    0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_UNSUPPORTED",
    4: "GDN_ERR_ALIGNMENT", 5: "GDN_ERR_NO_MEMORY", 6: "GDN_ERR_CUDA", 7: "GDN_ERR_TIMEOUT",
    8: "GDN_ERR_NONFINITE", 9: "GDN_ERR_NOT_IMPLEMENTED",
}

# every symbol include/gdn.h declares
EXPORTS = ("gdn_fwd", "gdn_fwd_f32", "gdn_step", "gdn_step_f32", "gdn_fwd_ex", "gdn_fwd_host",
           "gdn_apply_maps", "gdn_workspace_bytes", "gdn_status_string", "gdn_last_error", "gdn_version",
           "gdn_decode", "gdn_packed", "gdn_bwd", "gdn_seq_workspace_bytes")


class GdnError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, "GDN_ERR_UNKNOWN")
        super().__init__("%s: %s" % (self.name, detail))


class GdnArgs(ctypes.Structure):
    """Mirror of ``gdn_args`` in include/gdn.h (same field order and types)."""
    _fields_ = [
        ("struct_size", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("S_in", ctypes.c_void_p), ("S_out", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("B", ctypes.c_int), ("H", ctypes.c_int), ("T", ctypes.c_longlong),
        ("frame_len", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("reverse", ctypes.c_int), ("accumulate_o", ctypes.c_int),
        ("reset_every", ctypes.c_longlong), ("check_finite", ctypes.c_int),
        ("stream", ctypes.c_void_p), ("stage_ms", ctypes.c_void_p),
        ("mode", ctypes.c_int), ("gamma", ctypes.c_void_p),
        ("qk_norm", ctypes.c_int), ("k_norm_weight", ctypes.c_void_p), ("q_norm_weight", ctypes.c_void_p),
        ("status_dev", ctypes.c_void_p),
        ("phase", ctypes.c_int), ("segment_map", ctypes.c_void_p),
    ]


class GdnSeqArgs(ctypes.Structure):
    """Mirror of ``gdn_seq_args`` in include/gdn.h (same field order and types)."""
    _fields_ = [
        ("struct_size", ctypes.c_int), ("dtype", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("alpha", ctypes.c_void_p), ("beta", ctypes.c_void_p),
        ("q_stride", ctypes.c_longlong), ("k_stride", ctypes.c_longlong), ("v_stride", ctypes.c_longlong),
        ("o", ctypes.c_void_p), ("S_in", ctypes.c_void_p), ("S_out", ctypes.c_void_p),
        ("cu_seqlens", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("fresh", ctypes.c_void_p),
        ("n_seqs", ctypes.c_int), ("n_slots", ctypes.c_int),
        ("seq_len", ctypes.c_longlong), ("n_tokens", ctypes.c_longlong),
        ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("d_k", ctypes.c_int), ("d_v", ctypes.c_int),
        ("d_o", ctypes.c_void_p), ("dS_out", ctypes.c_void_p),
        ("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
        ("dalpha", ctypes.c_void_p), ("dbeta", ctypes.c_void_p), ("dS_in", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("stream", ctypes.c_void_p), ("status_dev", ctypes.c_void_p),
    ]


_SEQ_ARGS_BYTES = ctypes.sizeof(GdnSeqArgs)

GDN_SEQ_BAD_SLOT = 1
GDN_SEQ_SAME_SLOT = 2
GDN_SEQ_BAD_ROWS = 4
GDN_SEQ_TIMEOUT = 8

GDN_MODE_TOKEN = 0
GDN_MODE_FRAME = 1
GDN_QK_NORM_KEYS = 1
GDN_QK_NORM_QUERIES = 2
PHASES = {"all": 0, "prepare": 1, "finish": 2}

NUM_STAGES = 7
STAGES = ("gates", "diag_inverse", "intra", "transition", "scan", "u", "output")


_lib = None


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("CUDA library %s is missing; build it with "
                           "`python -m gated_deltanet_linear_chunkwise_b200.build`" % path)
    lib = ctypes.CDLL(path)
    V, I, LL = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    fwd_sig = [V, V, V, V, V, V, V, V, I, I, LL, I, I, I, V]
    for name in ("gdn_fwd", "gdn_fwd_f32", "gdn_step", "gdn_step_f32"):
        fn = getattr(lib, name)
        fn.argtypes = fwd_sig
        fn.restype = I
    lib.gdn_fwd_host.argtypes = [I] + fwd_sig
    lib.gdn_fwd_host.restype = I
    lib.gdn_fwd_ex.argtypes = [ctypes.POINTER(GdnArgs)]
    lib.gdn_fwd_ex.restype = I
    lib.gdn_apply_maps.argtypes = [V, V, I, I, I, I, I, V]
    lib.gdn_apply_maps.restype = I
    lib.gdn_workspace_bytes.argtypes = [I, I, LL, I, I, I, I]
    lib.gdn_workspace_bytes.restype = ctypes.c_size_t
    for name in ("gdn_decode", "gdn_packed", "gdn_bwd"):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(GdnSeqArgs)]
        fn.restype = I
    lib.gdn_seq_workspace_bytes.argtypes = [ctypes.POINTER(GdnSeqArgs), I]
    lib.gdn_seq_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_status_string.argtypes = [I]
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_last_error.argtypes = []
    lib.gdn_last_error.restype = ctypes.c_char_p
    lib.gdn_version.argtypes = []
    lib.gdn_version.restype = I
    _lib = lib
    return lib


def last_error() -> str:
    return load_library().gdn_last_error().decode()


def check(status: int):
    if status != 0:
        raise GdnError(status, last_error())


def workspace_bytes(B, H, T, frame_len, d_k, d_v, dtype="bf16") -> int:
    dt = GDN_DTYPE_BF16 if dtype in ("bf16", GDN_DTYPE_BF16) else GDN_DTYPE_F32
    return int(load_library().gdn_workspace_bytes(B, H, T, frame_len, d_k, d_v, dt))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _written(*tensors):
    """The caller's tensors that a call has written, told to autograd: a graph that saved one of them
    raises in its backward pass instead of reading the new values."""
    import torch
    torch.autograd.graph.increment_version([t for t in tensors if t is not None])


def gdn_fwd(q, k, v, alpha, beta, frame_len, S_in=None, *, S_out=None, o=None,
            return_state=False, reverse=False, accumulate=False, reset_every=0,
            check_finite=False, workspace=None, stream=None, stage_ms=None, mode="token", gamma=None,
            norm_keys=False, norm_queries=False, k_norm_weight=None, q_norm_weight=None, status=None,
            phase="all", segment_map=None):
    """Chunkwise gated delta rule forward on CUDA tensors.

    q,k [B,T,H,d_k], v [B,T,H,d_v] (bf16 or fp32, all the same), alpha/beta
    [B,T,H] fp32, S_in [B,H,d_v,d_k] fp32 or None.  ``o`` and ``S_out`` may be
    given (written in place; ``o`` is accumulated into when ``accumulate``);
    with ``return_state`` and no ``S_out`` a state tensor is allocated.
    ``stage_ms`` (a ``(ctypes.c_float * NUM_STAGES)()``) receives each kernel
    stage's device time; that call synchronises the stream.
    ``mode="frame"`` runs the frame-wise operator instead (one state update
    per frame of ``frame_len`` tokens); it reads ``gamma`` [B, T/frame_len, H]
    fp32, the per-frame decay, and not ``alpha`` (which may be None).
    ``norm_keys`` / ``norm_queries`` apply the q/k prologue first: keys
    ReLU(RMSNorm(k)) / sqrt(d_k * frame_len), queries ReLU(RMSNorm(q)), with
    optional fp32 [d_k] RMSNorm weights.
    ``status`` (a CUDA int32 tensor of one element) receives, in stream order,
    0 or a nonzero code when a bounded device-side wait gave up.
    ``phase="prepare"`` runs only the stages that do not depend on the entering
    state into ``workspace`` (required), and with ``segment_map`` (fp32
    [B, H, d_k + d_v, d_k]) also writes the call's map S_end = S_begin Phi + Psi;
    ``phase="finish"`` then runs the rest from ``S_in`` on the same workspace.
    Returns (o, S_out or None) (o is None for a prepare call).
    """
    import torch
    B, T, H, d_k = q.shape
    d_v = v.shape[-1]
    if mode not in ("token", "frame"):
        raise GdnError(1, "mode must be 'token' or 'frame'")
    frame = mode == "frame"
    gates = (("beta", beta), ("gamma", gamma)) if frame else (("alpha", alpha), ("beta", beta))
    for name, t in (("q", q), ("k", k), ("v", v)) + gates:
        if t is None:
            raise GdnError(1, "%s is required" % name)
    for name, t in (("q", q), ("k", k), ("v", v)) + gates:
        if not t.is_cuda:
            raise GdnError(1, "%s is not a CUDA tensor" % name)
        if not t.is_contiguous():
            raise GdnError(1, "%s is not contiguous" % name)
    if q.dtype != k.dtype or q.dtype != v.dtype or q.dtype not in (torch.bfloat16, torch.float32):
        raise GdnError(1, "q/k/v must share one dtype, bf16 or fp32")
    if any(t.dtype != torch.float32 for _, t in gates):
        raise GdnError(1, "%s must be fp32" % " and ".join(n for n, _ in gates))
    if frame and tuple(gamma.shape) != (B, T // max(int(frame_len), 1), H):
        raise GdnError(2, "gamma must have shape [B, T / frame_len, H]")
    for name, wt, on in (("k_norm_weight", k_norm_weight, norm_keys), ("q_norm_weight", q_norm_weight, norm_queries)):
        if wt is not None and on and (not wt.is_cuda or not wt.is_contiguous() or wt.dtype != torch.float32
                                      or wt.numel() != d_k):
            raise GdnError(1, "%s must be a contiguous fp32 CUDA tensor of d_k entries" % name)
    for name, t in (("S_in", S_in), ("S_out", S_out), ("o", o)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise GdnError(1, "%s must be a contiguous CUDA tensor" % name)
    if phase not in PHASES:
        raise GdnError(1, "phase must be 'all', 'prepare' or 'finish'")
    prepare = phase == "prepare"
    if segment_map is not None and (not segment_map.is_cuda or not segment_map.is_contiguous()
                                    or segment_map.dtype != torch.float32
                                    or tuple(segment_map.shape) != (B, H, d_k + d_v, d_k)):
        raise GdnError(1, "segment_map must be a contiguous fp32 CUDA tensor [B, H, d_k + d_v, d_k]")
    if o is None and not prepare:
        o = (torch.zeros if accumulate else torch.empty)((B, T, H, d_v), dtype=q.dtype, device=q.device)
    if S_out is None and return_state and not prepare:
        S_out = torch.empty((B, H, d_v, d_k), dtype=torch.float32, device=q.device)
    a = GdnArgs()
    a.phase = PHASES[phase]
    a.segment_map = _ptr(segment_map)
    a.struct_size = ctypes.sizeof(GdnArgs)
    a.dtype = GDN_DTYPE_BF16 if q.dtype == torch.bfloat16 else GDN_DTYPE_F32
    a.q, a.k, a.v = _ptr(q), _ptr(k), _ptr(v)
    a.alpha, a.beta = (None if frame else _ptr(alpha)), _ptr(beta)
    a.S_in, a.S_out, a.o = _ptr(S_in), _ptr(S_out), _ptr(o)
    a.mode = GDN_MODE_FRAME if frame else GDN_MODE_TOKEN
    a.gamma = _ptr(gamma) if frame else None
    if status is not None and (not status.is_cuda or status.dtype != torch.int32 or status.numel() < 1):
        raise GdnError(1, "status must be a CUDA int32 tensor")
    a.status_dev = _ptr(status)
    a.qk_norm = (GDN_QK_NORM_KEYS if norm_keys else 0) | (GDN_QK_NORM_QUERIES if norm_queries else 0)
    a.k_norm_weight = _ptr(k_norm_weight) if norm_keys else None
    a.q_norm_weight = _ptr(q_norm_weight) if norm_queries else None
    a.B, a.H, a.T = B, H, T
    a.frame_len, a.d_k, a.d_v = int(frame_len), d_k, d_v
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()
    a.reverse, a.accumulate_o = int(bool(reverse)), int(bool(accumulate))
    a.reset_every, a.check_finite = int(reset_every), int(bool(check_finite))
    a.stream = _stream_handle(stream, q.device)
    if stage_ms is not None:  # a ctypes float array of NUM_STAGES; the call synchronises
        a.stage_ms = ctypes.cast(stage_ms, ctypes.c_void_p)
    check(load_library().gdn_fwd_ex(ctypes.byref(a)))
    _written(o, S_out, segment_map)
    return o, S_out


def apply_maps(S, maps, *, stream=None):
    """S <- S Phi_j + Psi_j for each segment map in order, in place (``gdn_apply_maps``):
    S fp32 [B, H, d_v, d_k], maps fp32 [n, B, H, d_k + d_v, d_k] (CUDA, contiguous).
    Returns S."""
    import torch
    B, H, d_v, d_k = S.shape
    for name, t in (("S", S), ("maps", maps)):
        if not t.is_cuda or not t.is_contiguous() or t.dtype != torch.float32:
            raise GdnError(1, "%s must be a contiguous fp32 CUDA tensor" % name)
    if maps.dim() != 5 or tuple(maps.shape[1:]) != (B, H, d_k + d_v, d_k):
        raise GdnError(2, "maps must have shape [n, B, H, d_k + d_v, d_k]")
    check(load_library().gdn_apply_maps(_ptr(S), _ptr(maps), maps.shape[0], B, H, d_k, d_v,
                                        _stream_handle(stream, S.device)))
    _written(S)
    return S


def gdn_fwd_host(q, k, v, alpha, beta, frame_len, S_in=None, *, S_out=None, o=None,
                 return_state=False, stream=None, device=None):
    """The whole pass from HOST (CPU) tensors through ``gdn_fwd_host``: the
    library copies the inputs to the GPU, runs the pass, copies o (and the
    state) back and synchronises.  Pinned tensors copy fastest.  Same shapes
    and dtypes as ``gdn_fwd``; returns (o, S_out or None) on the host."""
    import torch
    B, T, H, d_k = q.shape
    d_v = v.shape[-1]
    for name, t in (("q", q), ("k", k), ("v", v), ("alpha", alpha), ("beta", beta), ("S_in", S_in),
                    ("S_out", S_out), ("o", o)):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise GdnError(1, "%s must be a contiguous host tensor" % name)
    if q.dtype != k.dtype or q.dtype != v.dtype or q.dtype not in (torch.bfloat16, torch.float32):
        raise GdnError(1, "q/k/v must share one dtype, bf16 or fp32")
    if alpha.dtype != torch.float32 or beta.dtype != torch.float32:
        raise GdnError(1, "alpha and beta must be fp32")
    if o is None:
        o = torch.empty((B, T, H, d_v), dtype=q.dtype)
    if S_out is None and return_state:
        S_out = torch.empty((B, H, d_v, d_k), dtype=torch.float32)
    dt = GDN_DTYPE_BF16 if q.dtype == torch.bfloat16 else GDN_DTYPE_F32
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    check(load_library().gdn_fwd_host(dt, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S_in),
                                      _ptr(S_out), _ptr(o), B, H, T, int(frame_len), d_k, d_v,
                                      _stream_handle(stream, device)))
    _written(o, S_out)
    return o, S_out


def gdn_step(q, k, v, alpha, beta, frame_len, S_in, *, S_out=None, o=None, workspace=None,
             stream=None):
    """One chunk-causal rollout call: S_in is required; returns (o, S_out).
    ``S_out`` may be ``S_in`` itself (in-place state update)."""
    if S_in is None:
        raise GdnError(1, "gdn_step requires S_in")
    return gdn_fwd(q, k, v, alpha, beta, frame_len, S_in, S_out=S_out, o=o, return_state=True,
                   workspace=workspace, stream=stream)


def bidirectional(q, k, v, alpha, beta, frame_len, *, chunk_len=0, S_in=None, stream=None):
    """Forward scan plus reversed-time scan, outputs summed; ``chunk_len`` > 0
    restarts the reversed scan at every chunk boundary (chunk-causal form).
    Returns (o, S_out of the forward scan)."""
    o, S = gdn_fwd(q, k, v, alpha, beta, frame_len, S_in, return_state=True, stream=stream)
    gdn_fwd(q, k, v, alpha, beta, frame_len, None, o=o, reverse=True, accumulate=True,
            reset_every=chunk_len, stream=stream)
    return o, S


# ---------------------------------------------------------------- sequences of any length
def _need(ok, status, text):
    if not ok:
        raise GdnError(status, text)


def _tokens(name, t, dtype, device, lead, heads, d):
    """A q/k/v-like tensor [*lead, heads, d]: checked; returns the elements between its token rows."""
    if t.dtype is not dtype or t.device != device:
        raise GdnError(1, "%s must have q's device and dtype (%s, %s)" % (name, device, dtype))
    if t.shape != (*lead, heads, d):
        raise GdnError(2, "%s must have shape %s, got %s" % (name, (*lead, heads, d), tuple(t.shape)))
    if t.is_contiguous():  # as any single token with its heads in place is
        return heads * d
    st = t.stride()
    if st[-1] != 1 or (st[-2] != d and heads > 1) or (len(lead) == 2 and min(lead) > 1 and st[0] != lead[1] * st[1]):
        raise GdnError(1, "%s: the heads of a token must be contiguous and the tokens equally far apart" % name)
    # of a single sequence or token a stride says nothing
    step = st[-3] if lead[-1] > 1 or len(lead) == 1 else st[0]
    if step < heads * d:  # an expanded tensor's 0 would read as "contiguous" behind the C interface
        raise GdnError(1, "%s: tokens %d elements apart lie over one another (a token has %d): pass .contiguous()" % (name, step, heads * d))
    return step


def _plain(name, t, dtype, shape, device):
    """The address of a contiguous tensor of one type and shape, or None of None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise GdnError(1, "%s must be a contiguous %s tensor on %s" % (name, str(dtype).replace("torch.", ""), device))
    if t.shape != shape:
        raise GdnError(2, "%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _seq_args(q, k, v, alpha, beta, lead):
    """The arguments that the sequence entries share; `lead` is the tokens' leading shape.  A serving loop pays
    for this at every token, so each attribute is asked for once."""
    import torch
    if q is None or k is None or v is None or alpha is None or beta is None:
        raise GdnError(1, "q, k, v, alpha and beta are required (one is None)")
    if not q.is_cuda:
        raise GdnError(1, "q is not a CUDA tensor")
    dtype, dev, n = q.dtype, q.device, len(lead)
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise GdnError(1, "q/k/v must share one dtype, bf16 or fp32")
    qs, vs = q.shape, v.shape
    if len(qs) != n + 2 or len(vs) != n + 2:
        raise GdnError(2, "q and v must have %d dimensions, got %s and %s" % (n + 2, tuple(qs), tuple(vs)))
    Hk, d_k = qs[n], qs[n + 1]
    H, d_v = vs[n], vs[n + 1]
    a = GdnSeqArgs(_SEQ_ARGS_BYTES, GDN_DTYPE_BF16 if dtype is torch.bfloat16 else GDN_DTYPE_F32,
                   q.data_ptr(), k.data_ptr(), v.data_ptr(),
                   _plain("alpha", alpha, torch.float32, (*lead, H), dev),
                   _plain("beta", beta, torch.float32, (*lead, H), dev),
                   _tokens("q", q, dtype, dev, lead, Hk, d_k), _tokens("k", k, dtype, dev, lead, Hk, d_k),
                   _tokens("v", v, dtype, dev, lead, H, d_v))
    a.H, a.Hk, a.d_k, a.d_v = H, Hk, d_k, d_v
    return a, dtype, dev, H, d_k, d_v


def _lead(q, cu_seqlens):
    """Leading shape of the tokens, and (n_seqs, seq_len, n_tokens)."""
    if cu_seqlens is None:
        if q.dim() != 4:
            raise GdnError(2, "without cu_seqlens q is [B, T, Hk, d_k], got %s" % (tuple(q.shape),))
        B, T = q.shape[:2]
        return (B, T), B, T, B * T
    if q.dim() != 3:
        raise GdnError(2, "with cu_seqlens q is [tokens, Hk, d_k], got %s" % (tuple(q.shape),))
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise GdnError(2, "cu_seqlens must have shape [sequences + 1], got %s" % (tuple(cu_seqlens.shape),))
    return (q.shape[0],), cu_seqlens.numel() - 1, 0, q.shape[0]


class _On:
    """The device of the tensors made current, and `stream` (None: its current one) for the
    call's own allocations, so that their memory is reused in that stream's order."""

    def __init__(self, device, stream):
        import torch
        self.outer = None
        if stream is not None:
            if stream.device != device:
                raise GdnError(1, "stream is on %s, the tensors on %s" % (stream.device, device))
            self.outer = torch.cuda.stream(stream)
            self.handle = stream.cuda_stream
        else:
            if device.index != torch._C._cuda_getDevice():
                self.outer = torch.cuda.device(device)
            self.handle = torch._C._cuda_getCurrentRawStream(device.index)

    def __enter__(self):
        if self.outer is not None:
            self.outer.__enter__()
        return self.handle

    def __exit__(self, *e):
        if self.outer is not None:
            self.outer.__exit__(*e)


def gdn_decode(q, k, v, alpha, beta, S, slots=None, *, o=None, status=None, stream=None):
    """The next one or few tokens of a batch of sequences, in the recurrent form.

    q, k [B, n, Hk, d_k], v [B, n, H, d_v] (bf16 or fp32), alpha, beta [B, n, H] fp32; for n = 1
    the n dimension may be left out of all of them.  H is a multiple of Hk: head h reads q/k head
    h // (H // Hk).  The heads of a token are contiguous; the tokens of q, k, v may be slices of a
    fused projection (equally far apart, a multiple of 16 bytes), but not one row expanded to many.
    S fp32 [n_slots, H, d_v, d_k] holds the states and is updated in place: sequence b's is
    S[slots[b]] (slots int32 [B]; None: S[b]).  A negative slot is a padding entry: its o rows (in an o that
    the call makes they hold nothing) and every state are left alone.  So is a sequence with a slot >= n_slots or the slot of an earlier
    sequence; `status` (a CUDA int32 tensor) then receives GDN_SEQ_BAD_SLOT / GDN_SEQ_SAME_SLOT.
    Returns (o, S).
    """
    import torch
    if q is None or S is None:
        raise GdnError(1, "q and S are required")
    lead = tuple(q.shape[:-2])
    if len(lead) != 1 and len(lead) != 2:
        raise GdnError(2, "q is [B, n, Hk, d_k] or [B, Hk, d_k], got %s" % (tuple(q.shape),))
    a, dtype, dev, H, d_k, d_v = _seq_args(q, k, v, alpha, beta, lead)
    B, n = lead[0], lead[1] if len(lead) == 2 else 1
    n_slots = S.shape[0] if S.dim() else 0
    a.S_in = a.S_out = _plain("S", S, torch.float32, (n_slots, H, d_v, d_k), dev)
    a.n_seqs, a.seq_len, a.n_tokens, a.n_slots = B, n, B * n, n_slots
    if slots is not None:
        a.slots = _plain("slots", slots, torch.int32, (B,), dev)
    if status is not None:
        a.status_dev = _plain("status", status, torch.int32, (1,), dev)
    with _On(dev, stream) as a.stream:
        written = (S,)
        if o is None:
            o = torch.empty(v.shape, dtype=dtype, device=dev)
            a.o = o.data_ptr()
        else:
            a.o = _plain("o", o, dtype, v.shape, dev)
            written = (S, o)
        check((_lib or load_library()).gdn_decode(ctypes.byref(a)))
    torch._C._increment_version(written)  # as _written, in half its time
    return o, S


def gdn_packed(q, k, v, alpha, beta, cu_seqlens=None, S_in=None, *, S_out=None, slots=None, fresh=None, o=None,
               return_state=False, workspace=None, status=None, stream=None):
    """The forward pass over sequences of different lengths packed behind one another.

    q, k [N, Hk, d_k], v [N, H, d_v] (bf16 or fp32), alpha, beta [N, H] fp32; sequence s covers
    the tokens cu_seqlens[s] .. cu_seqlens[s+1] - 1 (int32 [n + 1], on the GPU and read there only).
    Without cu_seqlens: [B, T, heads, d] tensors, B sequences of T tokens.  Heads, strides and slots
    as in ``gdn_decode``; o rows of tokens that no sequence covers are left as they were (in an o that the
    call makes they hold nothing).
    S_in, S_out fp32 [n_slots, H, d_v, d_k] hold the states that enter (None: zeros) and leave
    (None: not stored, unless ``return_state`` makes a tensor of n_slots = n, zeros where a sequence is
    skipped); they may be the same tensor.  ``fresh`` (bool or uint8 [n]) starts the marked sequences from zero without reading S_in.
    ``status`` may also receive GDN_SEQ_BAD_ROWS (a range out of order, out of the tensors or into an
    earlier sequence's).
    Returns (o, S_out or None).
    """
    import torch
    lead, n, T, N = _lead(q, cu_seqlens)
    a, dtype, dev, H, d_k, d_v = _seq_args(q, k, v, alpha, beta, lead)
    a.n_seqs, a.seq_len, a.n_tokens = n, T, N
    a.cu_seqlens = _plain("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), dev)
    a.slots = _plain("slots", slots, torch.int32, (n,), dev)
    if fresh is not None and fresh.dtype == torch.bool:
        fresh = fresh.view(torch.uint8)
    a.fresh = _plain("fresh", fresh, torch.uint8, (n,), dev)
    a.status_dev = _plain("status", status, torch.int32, (1,), dev)
    with _On(dev, stream) as a.stream:
        if o is None:
            o = torch.empty(v.shape, dtype=dtype, device=dev)
        if S_out is None and return_state:
            _need(slots is None, 1, "return_state makes one state a sequence: with slots pass S_out")
            # a skipped sequence's entry is not written
            S_out = (torch.empty if cu_seqlens is None else torch.zeros)((n, H, d_v, d_k), dtype=torch.float32, device=dev)
        a.o = _plain("o", o, dtype, v.shape, dev)
        pool = S_in if S_in is not None else S_out
        a.n_slots = n if pool is None else pool.shape[0] if pool.dim() else 0
        a.S_in = _plain("S_in", S_in, torch.float32, (a.n_slots, H, d_v, d_k), dev)
        a.S_out = _plain("S_out", S_out, torch.float32, (a.n_slots, H, d_v, d_k), dev)
        _seq_workspace(a, workspace, dev, 0)
        check(load_library().gdn_packed(ctypes.byref(a)))
    _written(o, S_out)
    return o, S_out


def _seq_workspace(a, workspace, device, bwd):
    """The caller's workspace, or the library's stream-ordered scratch (the pointer stays NULL);
    a call being captured takes it from torch's allocator, so that the graph keeps its own."""
    import torch
    if workspace is None and torch.cuda.is_current_stream_capturing():
        workspace = torch.empty(seq_workspace_args(a, bwd), dtype=torch.uint8, device=device)
    if workspace is not None and workspace.numel():
        _need(workspace.device == device and workspace.is_contiguous(), 1, "workspace must be a contiguous tensor on %s" % device)
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size()


def seq_workspace_args(a, bwd) -> int:
    return int(load_library().gdn_seq_workspace_bytes(ctypes.byref(a), bwd))


def gdn_bwd(q, k, v, alpha, beta, do, cu_seqlens=None, S_in=None, *, dS_out=None, need_dS_in=None, workspace=None,
            status=None, stream=None):
    """Gradients of ``gdn_packed``: tensors as there, ``do`` the gradient of o and ``dS_out`` that of
    the states that leave (None: zeros); S_in and dS_out are fp32 [n, H, d_v, d_k], one state a
    sequence.  The forward pass is recomputed; nothing of it needs to be kept.
    Returns (dq, dk, dv, dalpha, dbeta, dS_in): the first three in q's dtype, the gates' in fp32, and
    dS_in (fp32) when S_in is given or ``need_dS_in`` asks for it, else None.  Gradients of q/k heads
    that several heads share are summed in fp32; of tokens that no sequence covers they are zeros.
    """
    import torch
    lead, n, T, N = _lead(q, cu_seqlens)
    a, dtype, dev, H, d_k, d_v = _seq_args(q, k, v, alpha, beta, lead)
    a.n_seqs, a.seq_len, a.n_tokens = n, T, N
    a.cu_seqlens = _plain("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), dev)
    state = (n, H, d_v, d_k)
    a.n_slots = n
    a.S_in = _plain("S_in", S_in, torch.float32, state, dev)
    a.dS_out = _plain("dS_out", dS_out, torch.float32, state, dev)
    _need(do is not None, 1, "do is required")
    a.d_o = _plain("do", do, dtype, v.shape, dev)
    a.status_dev = _plain("status", status, torch.int32, (1,), dev)
    with _On(dev, stream) as a.stream:
        dq, dk = (torch.empty(t.shape, dtype=t.dtype, device=dev) for t in (q, k))
        dv = torch.empty(v.shape, dtype=v.dtype, device=dev)
        dalpha, dbeta = (torch.empty(alpha.shape, dtype=torch.float32, device=dev) for _ in range(2))
        dS_in = None
        if need_dS_in or (need_dS_in is None and S_in is not None):
            dS_in = torch.empty(state, dtype=torch.float32, device=dev)
        a.dq, a.dk, a.dv = dq.data_ptr(), dk.data_ptr(), dv.data_ptr()
        a.dalpha, a.dbeta, a.dS_in = dalpha.data_ptr(), dbeta.data_ptr(), _ptr(dS_in)
        _seq_workspace(a, workspace, dev, 1)
        check(load_library().gdn_bwd(ctypes.byref(a)))
    return dq, dk, dv, dalpha, dbeta, dS_in


def seq_workspace_bytes(n_tokens, H, Hk, d_k, d_v, *, n_seqs, packed=True, bwd=False, dtype="bf16") -> int:
    """Scratch of a ``gdn_packed`` (or, with ``bwd``, ``gdn_bwd``) call of these sizes; ``packed``:
    with cu_seqlens, else n_seqs sequences of n_tokens // n_seqs tokens."""
    a = GdnSeqArgs()
    a.dtype = GDN_DTYPE_BF16 if dtype in ("bf16", GDN_DTYPE_BF16) else GDN_DTYPE_F32
    a.n_seqs, a.n_tokens, a.seq_len = n_seqs, n_tokens, 0 if packed or not n_seqs else n_tokens // n_seqs
    a.cu_seqlens = 16 if packed else None  # looked at for NULL only
    a.H, a.Hk, a.d_k, a.d_v = H, Hk, d_k, d_v
    return seq_workspace_args(a, int(bool(bwd)))
