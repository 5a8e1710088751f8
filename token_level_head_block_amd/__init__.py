"""libmhla: the MHLA forward pass on AMD Instinct MI355X (gfx950).

Thin ctypes binding over the C ABI declared in ``include/mhla.h``: the
functions below carry the C names and only marshal arguments (tensor data
pointers, shape structs, the current HIP stream).  Every step of the forward
pass runs in the HIP kernels of ``libmhla.so``; there is no Python or CPU
fallback -- if the library is missing, every call raises.

MHLA (arXiv 2601.07832; paperlayer.ai summary, section 4) splits the tokens of
a 2D/3D grid into M non-overlapping blocks, summarises each block as
S_j = phi(K_j)^T V_j and z_j = sum phi(k), mixes the summaries with a learnable
M x M matrix W, and gives every query o = phi(q) St_i / (phi(q) . zt_i + eps).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmhla.so")

MHLA_OK = 0
MHLA_ERR_INVALID_ARG = 1
MHLA_ERR_UNSUPPORTED = 2
MHLA_ERR_MISALIGNED = 3
MHLA_ERR_ALLOC = 4
MHLA_ERR_HIP = 5

MHLA_F32 = 0
MHLA_BF16 = 1

MHLA_PATH_3KERNEL = 0
MHLA_PATH_FUSED = 1
MHLA_PATH_CAUSAL = 2

MHLA_VARIANT_MIX_RESIDENT = 1 << 8
MHLA_VARIANT_MIX_TILED = 1 << 9
MHLA_VARIANT_NO_PAIR_HEADS = 1 << 10
MHLA_VARIANT_MIX_SPLIT = 1 << 11
MHLA_VARIANT_APPLY_REGS = 1 << 12

MHLA_PHI_ELU1 = 0
MHLA_PHI_RELU_EPS = 1

MHLA_ROPE_HALVES = 0
MHLA_ROPE_INTERLEAVED = 1


class mhla_grid(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("ndim", ctypes.c_int32), ("extent", ctypes.c_int32 * 3),
                ("eps", ctypes.c_float)]


class mhla_block(ctypes.Structure):
    _fields_ = [("extent", ctypes.c_int32 * 3)]


class mhla_layer_params(ctypes.Structure):
    _fields_ = [("ln_w", ctypes.c_void_p), ("ln_b", ctypes.c_void_p), ("w_qkv", ctypes.c_void_p),
                ("b_qkv", ctypes.c_void_p), ("qn_w", ctypes.c_void_p), ("kn_w", ctypes.c_void_p),
                ("lepe_w", ctypes.c_void_p), ("lepe_b", ctypes.c_void_p), ("w_out", ctypes.c_void_p),
                ("b_out", ctypes.c_void_p), ("phi", ctypes.c_int32), ("phi_eps", ctypes.c_float),
                ("ln_eps", ctypes.c_float), ("rms_eps", ctypes.c_float)]


class mhla_seq(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("tokens", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
                ("scale", ctypes.c_float)]


class mhla_rope(ctypes.Structure):
    _fields_ = [("style", ctypes.c_int32), ("axes", ctypes.c_int32), ("section", ctypes.c_int32 * 3),
                ("eps", ctypes.c_float)]


class MhlaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {mhla_status_string(status)}" if what else mhla_status_string(status))


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libmhla.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m token_level_head_block_amd._build`")
        L = ctypes.CDLL(LIB_PATH)
        G, Bk = ctypes.POINTER(mhla_grid), ctypes.POINTER(mhla_block)
        vp = ctypes.c_void_p
        L.mhla_status_string.argtypes = [ctypes.c_int]
        L.mhla_status_string.restype = ctypes.c_char_p
        L.mhla_check_problem.argtypes = [G, Bk, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64)]
        L.mhla_check_problem.restype = ctypes.c_int
        L.mhla_launch_plan.argtypes = [G, Bk, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32),
                                       ctypes.POINTER(ctypes.c_char_p)]
        L.mhla_launch_plan.restype = ctypes.c_int
        L.mhla_backward_workspace_bytes.argtypes = [G, Bk]
        L.mhla_backward_workspace_bytes.restype = ctypes.c_size_t
        L.mhla_backward.argtypes = [vp, vp, vp, vp, vp, G, Bk, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
        L.mhla_backward.restype = ctypes.c_int
        L.mhla_backward_ex.argtypes = [vp, vp, vp, vp, vp, G, Bk, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                       ctypes.c_int32, vp, vp]
        L.mhla_backward_ex.restype = ctypes.c_int
        L.mhla_causal_backward_workspace_bytes.argtypes = [G, Bk]
        L.mhla_causal_backward_workspace_bytes.restype = ctypes.c_size_t
        L.mhla_causal_backward.argtypes = [vp, vp, vp, vp, vp, G, Bk, vp, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
        L.mhla_causal_backward.restype = ctypes.c_int
        L.mhla_causal_state_bytes.argtypes = [G, Bk, ctypes.c_int32]
        L.mhla_causal_state_bytes.restype = ctypes.c_size_t
        L.mhla_causal_stream_workspace_bytes.argtypes = [G, Bk]
        L.mhla_causal_stream_workspace_bytes.restype = ctypes.c_size_t
        L.mhla_causal_stream.argtypes = [vp, vp, vp, vp, ctypes.c_int32, G, Bk, ctypes.c_int32, vp, ctypes.c_int32,
                                         vp, vp, ctypes.c_size_t, vp]
        L.mhla_causal_stream.restype = ctypes.c_int
        L.mhla_workspace_bytes.argtypes = [G, Bk]
        L.mhla_workspace_bytes.restype = ctypes.c_size_t
        L.mhla_forward.argtypes = [vp, vp, vp, vp, G, Bk, vp, vp]
        L.mhla_forward.restype = ctypes.c_int
        L.mhla_forward_ws.argtypes = [vp, vp, vp, vp, G, Bk, vp, vp, ctypes.c_size_t, vp]
        L.mhla_forward_ws.restype = ctypes.c_int
        L.mhla_forward_ex.argtypes = [vp, vp, vp, vp, G, Bk, vp, vp, ctypes.c_size_t, ctypes.c_int32,
                                      vp, vp]
        L.mhla_forward_ex.restype = ctypes.c_int
        L.mhla_forward_noalloc.argtypes = [vp, vp, vp, vp, G, Bk, vp, vp]
        L.mhla_forward_noalloc.restype = ctypes.c_int
        L.mhla_layer_workspace_bytes.argtypes = [G, Bk]
        L.mhla_layer_workspace_bytes.restype = ctypes.c_size_t
        L.mhla_layer_forward.argtypes = [vp, vp, G, Bk, ctypes.POINTER(mhla_layer_params), vp, vp,
                                         ctypes.c_size_t, vp, vp]
        L.mhla_layer_forward.restype = ctypes.c_int
        Sq, Rp = ctypes.POINTER(mhla_seq), ctypes.POINTER(mhla_rope)
        L.mhla_check_seq.argtypes = [Sq]
        L.mhla_check_seq.restype = ctypes.c_int
        for f in (L.mhla_gated_workspace_bytes, L.mhla_gated_backward_workspace_bytes,
                  L.mhla_qk_norm_rope_backward_workspace_bytes):
            f.argtypes = [Sq]
            f.restype = ctypes.c_size_t
        L.mhla_gated_forward.argtypes = [vp] * 6 + [Sq, vp, vp, vp, ctypes.c_size_t, vp]
        L.mhla_gated_forward.restype = ctypes.c_int
        L.mhla_gated_backward.argtypes = [vp] * 8 + [Sq, vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.mhla_gated_backward.restype = ctypes.c_int
        L.mhla_gated_step.argtypes = [vp] * 5 + [Sq, vp, ctypes.c_int32, vp, vp]
        L.mhla_gated_step.restype = ctypes.c_int
        L.mhla_qk_norm_rope.argtypes = [vp] * 6 + [Rp, Sq, vp, vp, vp]
        L.mhla_qk_norm_rope.restype = ctypes.c_int
        L.mhla_qk_norm_rope_backward.argtypes = [vp] * 6 + [Rp, vp, vp, Sq, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.mhla_qk_norm_rope_backward.restype = ctypes.c_int
        _lib = L
    return _lib


# ---------------------------------------------------------------- structs

def make_grid(batch: int, heads: int, head_dim: int, dtype: int, extents, eps: float = 1e-6) -> mhla_grid:
    g = mhla_grid()
    g.batch, g.heads, g.head_dim, g.dtype = batch, heads, head_dim, dtype
    g.ndim = len(extents)
    for a in range(3):
        g.extent[a] = int(extents[a]) if a < len(extents) else 0
    g.eps = eps
    return g


def make_block(extents) -> mhla_block:
    b = mhla_block()
    for a in range(3):
        b.extent[a] = int(extents[a]) if a < len(extents) else 0
    return b


# ---------------------------------------------------------------- C entry points

def mhla_status_string(status: int) -> str:
    return lib().mhla_status_string(int(status)).decode()


def mhla_check_problem(grid: mhla_grid, block: mhla_block):
    """(status, M, T)."""
    m, t = ctypes.c_int64(0), ctypes.c_int64(0)
    st = lib().mhla_check_problem(ctypes.byref(grid), ctypes.byref(block), ctypes.byref(m), ctypes.byref(t))
    return st, m.value, t.value


def mhla_launch_plan(grid: mhla_grid, block: mhla_block, path: int = 0):
    """(status, [kernel names in launch order])."""
    n = ctypes.c_int32(0)
    names = (ctypes.c_char_p * 3)()
    st = lib().mhla_launch_plan(ctypes.byref(grid), ctypes.byref(block), int(path), ctypes.byref(n), names)
    return st, [names[i].decode() for i in range(n.value)]


def mhla_workspace_bytes(grid: mhla_grid, block: mhla_block) -> int:
    return int(lib().mhla_workspace_bytes(ctypes.byref(grid), ctypes.byref(block)))


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check_tensors(q, k, v, W, out, grid: mhla_grid, block: mhla_block):
    """Host-side shape/dtype checks of torch tensors against the grid, so the
    kernels never index past a buffer whose size the C ABI cannot see."""
    import torch
    st, M, _ = mhla_check_problem(grid, block)
    if st != MHLA_OK:
        return
    N = 1
    for a in range(grid.ndim):
        N *= grid.extent[a]
    want = (grid.batch, N, grid.heads, grid.head_dim)
    tdt = torch.bfloat16 if grid.dtype == MHLA_BF16 else torch.float32
    for name, t in (("q", q), ("k", k), ("v", v), ("out", out)):
        if not isinstance(t, torch.Tensor):
            continue
        if tuple(t.shape) != want or t.dtype != tdt or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {tdt} tensor of shape {want}, "
                             f"got {t.dtype} {tuple(t.shape)}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be on a GPU")
    if isinstance(W, torch.Tensor):
        if tuple(W.shape) != (M, M) or W.dtype != torch.float32 or not W.is_contiguous() or not W.is_cuda:
            raise ValueError(f"W must be a contiguous float32 GPU tensor of shape {(M, M)}")


def mhla_forward(q, k, v, W, grid: mhla_grid, block: mhla_block, out, stream=None) -> int:
    _check_tensors(q, k, v, W, out, grid, block)
    return lib().mhla_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(W), ctypes.byref(grid),
                              ctypes.byref(block), _ptr(out), _stream(stream))


def mhla_forward_ws(q, k, v, W, grid: mhla_grid, block: mhla_block, out, ws, ws_bytes: int,
                    stream=None) -> int:
    _check_tensors(q, k, v, W, out, grid, block)
    return lib().mhla_forward_ws(_ptr(q), _ptr(k), _ptr(v), _ptr(W), ctypes.byref(grid),
                                 ctypes.byref(block), _ptr(out), _ptr(ws), int(ws_bytes),
                                 _stream(stream))


MHLA_NOALLOC_SCRATCH_BYTES = 32 << 20


def mhla_forward_noalloc(q, k, v, W, grid: mhla_grid, block: mhla_block, out, stream=None) -> int:
    """mhla_forward with the library's fixed per-GPU scratch as workspace (allocates nothing)."""
    _check_tensors(q, k, v, W, out, grid, block)
    return lib().mhla_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(W), ctypes.byref(grid),
                                      ctypes.byref(block), _ptr(out), _stream(stream))


def mhla_forward_ex(q, k, v, W, grid: mhla_grid, block: mhla_block, out, ws, ws_bytes: int,
                    path: int = MHLA_PATH_3KERNEL, stage_events=None, stream=None) -> int:
    """stage_events: None or 4 events, each a torch.cuda.Event (already
    recorded once, so that its HIP handle exists) or a raw hipEvent_t handle
    (int)."""
    _check_tensors(q, k, v, W, out, grid, block)
    ev = None
    if stage_events is not None:
        if len(stage_events) != 4:
            raise ValueError("stage_events needs 4 events")
        arr = (ctypes.c_void_p * 4)(*[e if isinstance(e, int) else e.cuda_event for e in stage_events])
        if any(a is None or a == 0 for a in arr):
            raise ValueError("stage events have no HIP handle yet; record each once first")
        ev = ctypes.cast(arr, ctypes.c_void_p)
    return lib().mhla_forward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(W), ctypes.byref(grid),
                                 ctypes.byref(block), _ptr(out), _ptr(ws), int(ws_bytes), int(path),
                                 ev, _stream(stream))


def mhla_backward_workspace_bytes(grid: mhla_grid, block: mhla_block) -> int:
    return int(lib().mhla_backward_workspace_bytes(ctypes.byref(grid), ctypes.byref(block)))


def _events(stage_events, n):
    if stage_events is None:
        return None
    if len(stage_events) != n:
        raise ValueError(f"stage_events needs {n} events")
    arr = (ctypes.c_void_p * n)(*[e if isinstance(e, int) else e.cuda_event for e in stage_events])
    if any(a is None or a == 0 for a in arr):
        raise ValueError("stage events have no HIP handle yet; record each once first")
    return ctypes.cast(arr, ctypes.c_void_p)


def mhla_backward(q, k, v, W, dout, grid: mhla_grid, block: mhla_block, dq, dk, dv, dW, ws=None,
                  ws_bytes: int = 0, stage_events=None, stream=None) -> int:
    """Gradients dq, dk, dv (bf16 tensors like q) and dW (fp32 [M, M]) for the
    upstream gradient dout.  stage_events: None or 5 events (torch.cuda.Event
    already recorded once, or raw hipEvent_t handles)."""
    _check_tensors(q, k, v, W, dout, grid, block)
    _check_tensors(dq, dk, dv, dW, None, grid, block)
    return lib().mhla_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(W), _ptr(dout), ctypes.byref(grid),
                               ctypes.byref(block), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dW), _ptr(ws),
                               int(ws_bytes), _events(stage_events, 5), _stream(stream))


def mhla_backward_ex(q, k, v, W, dout, grid: mhla_grid, block: mhla_block, dq, dk, dv, dW, ws=None,
                     ws_bytes: int = 0, variant: int = 0, stage_events=None, stream=None) -> int:
    """As mhla_backward, with MHLA_VARIANT_* flags (MHLA_VARIANT_NO_PAIR_HEADS)."""
    _check_tensors(q, k, v, W, dout, grid, block)
    _check_tensors(dq, dk, dv, dW, None, grid, block)
    return lib().mhla_backward_ex(_ptr(q), _ptr(k), _ptr(v), _ptr(W), _ptr(dout), ctypes.byref(grid),
                                  ctypes.byref(block), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dW), _ptr(ws),
                                  int(ws_bytes), int(variant), _events(stage_events, 5), _stream(stream))


def mhla_causal_backward_workspace_bytes(grid: mhla_grid, block: mhla_block) -> int:
    return int(lib().mhla_causal_backward_workspace_bytes(ctypes.byref(grid), ctypes.byref(block)))


def mhla_causal_backward(q, k, v, W, dout, grid: mhla_grid, block: mhla_block, dq, dk, dv, dW, ws=None,
                         ws_bytes: int = 0, stage_events=None, stream=None) -> int:
    """Gradients through the causal chunkwise form; arguments as mhla_backward."""
    _check_tensors(q, k, v, W, dout, grid, block)
    _check_tensors(dq, dk, dv, dW, None, grid, block)
    return lib().mhla_causal_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(W), _ptr(dout), ctypes.byref(grid),
                                      ctypes.byref(block), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dW), _ptr(ws),
                                      int(ws_bytes), _events(stage_events, 5), _stream(stream))


def mhla_causal_state_bytes(grid: mhla_grid, block: mhla_block, max_chunks: int) -> int:
    return int(lib().mhla_causal_state_bytes(ctypes.byref(grid), ctypes.byref(block), int(max_chunks)))


def mhla_causal_stream_workspace_bytes(grid: mhla_grid, block: mhla_block) -> int:
    return int(lib().mhla_causal_stream_workspace_bytes(ctypes.byref(grid), ctypes.byref(block)))


def mhla_causal_stream(q, k, v, W, grid: mhla_grid, block: mhla_block, n_past: int, state, max_chunks: int, out,
                       ws=None, ws_bytes: int = 0, stream=None) -> int:
    """One call of a causal stream: q, k, v, out [B, N_new, H, d] (the new
    chunks), W fp32 [w_dim, w_dim] (w_dim from W's shape), state fp32 with
    mhla_causal_state_bytes(grid, block, max_chunks) bytes."""
    for t in (q, k, v, out):
        if t is None or not t.is_contiguous():
            raise ValueError("q, k, v and out must be contiguous device tensors")
    if W.dim() != 2 or W.shape[0] != W.shape[1] or not W.is_contiguous():
        raise ValueError("W must be a contiguous square fp32 matrix")
    if not state.is_contiguous() or state.numel() * state.element_size() < mhla_causal_state_bytes(grid, block,
                                                                                                  max_chunks):
        raise ValueError("state is smaller than mhla_causal_state_bytes")
    return lib().mhla_causal_stream(_ptr(q), _ptr(k), _ptr(v), _ptr(W), int(W.shape[0]), ctypes.byref(grid),
                                    ctypes.byref(block), int(n_past), _ptr(state), int(max_chunks), _ptr(out),
                                    _ptr(ws), int(ws_bytes), _stream(stream))


# ---------------------------------------------------------------- convenience

def forward(q, k, v, W, grid_extents, block_extents, eps: float = 1e-6, out=None, ws=None,
            path: int = MHLA_PATH_3KERNEL, stream=None):
    """Allocate `out` if needed, call mhla_forward_ex, raise MhlaError on failure."""
    import torch
    dt = MHLA_BF16 if q.dtype == torch.bfloat16 else MHLA_F32
    B, N, H, d = q.shape
    g = make_grid(B, H, d, dt, grid_extents, eps)
    b = make_block(block_extents)
    if out is None:
        out = torch.empty_like(q)
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    st = mhla_forward_ex(q, k, v, W, g, b, out, ws, nbytes, path, None, stream)
    if st != MHLA_OK:
        raise MhlaError(st, "mhla_forward_ex")
    return out


# ---------------------------------------------------------------- layer

LAYER_PARAM_NAMES = ("ln_w", "ln_b", "w_qkv", "b_qkv", "qn_w", "kn_w", "lepe_w", "lepe_b", "w_out", "b_out")


def mhla_layer_workspace_bytes(grid: mhla_grid, block: mhla_block) -> int:
    return int(lib().mhla_layer_workspace_bytes(ctypes.byref(grid), ctypes.byref(block)))


def _check_layer_tensors(x, W, grid: mhla_grid, block: mhla_block, params: dict, y):
    """Host-side shape/dtype checks of the layer's torch tensors (the C ABI
    cannot see tensor sizes)."""
    import torch
    st, M, _ = mhla_check_problem(grid, block)
    if st != MHLA_OK:
        return
    N = 1
    for a in range(grid.ndim):
        N *= grid.extent[a]
    C = grid.heads * grid.head_dim
    want = {"ln_w": ((C,), torch.float32), "ln_b": ((C,), torch.float32),
            "w_qkv": ((3 * C, C), torch.bfloat16), "b_qkv": ((3 * C,), torch.float32),
            "qn_w": ((C,), torch.float32), "kn_w": ((C,), torch.float32),
            "lepe_w": ((C, 5, 5), torch.float32), "lepe_b": ((C,), torch.float32),
            "w_out": ((C, C), torch.bfloat16), "b_out": ((C,), torch.float32)}
    tensors = [("x", x, ((grid.batch, N, C), torch.bfloat16)), ("y", y, ((grid.batch, N, C), torch.bfloat16)),
               ("W", W, ((M, M), torch.float32))]
    tensors += [(k, params.get(k), want[k]) for k in LAYER_PARAM_NAMES]
    for name, t, (shape, dt) in tensors:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or tuple(t.shape) != shape or t.dtype != dt \
                or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"{name} must be a contiguous {dt} GPU tensor of shape {shape}")


def mhla_layer_forward(x, W, grid: mhla_grid, block: mhla_block, params: dict, y, ws=None, ws_bytes: int = 0,
                       phi: int = MHLA_PHI_ELU1, phi_eps: float = 1e-6, ln_eps: float = 1e-5,
                       rms_eps: float = 1e-6, stage_events=None, stream=None) -> int:
    """The layer forward through the C ABI.  params: dict with the tensors
    named in LAYER_PARAM_NAMES (absent or None for optional ones)."""
    _check_layer_tensors(x, W, grid, block, params, y)
    P = mhla_layer_params()
    for name in LAYER_PARAM_NAMES:
        setattr(P, name, _ptr(params.get(name)))
    P.phi, P.phi_eps, P.ln_eps, P.rms_eps = int(phi), float(phi_eps), float(ln_eps), float(rms_eps)
    return lib().mhla_layer_forward(_ptr(x), _ptr(W), ctypes.byref(grid), ctypes.byref(block), ctypes.byref(P),
                                    _ptr(y), _ptr(ws), int(ws_bytes), _events(stage_events, 5), _stream(stream))


# ---------------------------------------------------------------- gated linear attention, q/k norm and rotation

def make_seq(batch: int, tokens: int, heads: int, kv_heads: int, head_dim: int, dtype: int, scale: float = 1.0,
             q_stride: int = 0, k_stride: int = 0, v_stride: int = 0) -> mhla_seq:
    return mhla_seq(batch, tokens, heads, kv_heads, head_dim, dtype, q_stride, k_stride, v_stride, scale)


def make_rope(sections, style: int = MHLA_ROPE_HALVES, eps: float = 1e-6) -> mhla_rope:
    """sections: the pairs that turn with each axis's position, one entry an axis (1 to 3)."""
    n = len(sections)
    r = mhla_rope(int(style), n, (0, 0, 0), float(eps))
    for a in range(min(n, 3)):
        r.section[a] = int(sections[a])
    return r


def mhla_check_seq(seq: mhla_seq) -> int:
    return lib().mhla_check_seq(ctypes.byref(seq))


def mhla_gated_workspace_bytes(seq: mhla_seq) -> int:
    return int(lib().mhla_gated_workspace_bytes(ctypes.byref(seq)))


def mhla_gated_backward_workspace_bytes(seq: mhla_seq) -> int:
    return int(lib().mhla_gated_backward_workspace_bytes(ctypes.byref(seq)))


def mhla_qk_norm_rope_backward_workspace_bytes(seq: mhla_seq) -> int:
    return int(lib().mhla_qk_norm_rope_backward_workspace_bytes(ctypes.byref(seq)))


def _need(name, t, shape, dtype, device):
    """A contiguous GPU tensor of this shape and type on `device`."""
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _stride_of(name, t, shape, dtype, device):
    """Values between a token of t and the next one, for a tensor [B, T, heads, d] (or rows [B, heads, d])
    whose tokens' values are contiguous and evenly spaced over the whole batch (a slice of a wider row, say)."""
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    h, d = shape[-2:]
    if t.is_contiguous():
        return h * d
    B, T = shape[0], shape[1] if len(shape) == 4 else 1
    sb, st, (sh, sd) = t.stride(0), t.stride(1) if len(shape) == 4 else 0, t.stride()[-2:]
    step = st if T > 1 else sb if B > 1 else h * d
    if sd != 1 or (h > 1 and sh != d) or (T > 1 and B > 1 and sb != T * st) or step < h * d:
        raise ValueError(f"{name}: the values of a token must be contiguous and tokens evenly spaced, "
                         f"got strides {t.stride()} for shape {tuple(shape)}")
    return step


def _check_seq_tensors(q, k, v, seq: mhla_seq, rows: bool = False):
    """The type and device of a sequence problem's tensors, after checking q, k and v (or None) against seq
    (rows: [B, heads, d], one token each).  The C ABI cannot see tensor sizes."""
    import torch
    dt = torch.bfloat16 if seq.dtype == MHLA_BF16 else torch.float32
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be on a GPU")
    B, T, H, Hk, d = seq.batch, seq.tokens, seq.heads, seq.kv_heads, seq.head_dim
    for name, t, h, stride in (("q", q, H, seq.q_stride), ("k", k, Hk, seq.k_stride), ("v", v, Hk, seq.v_stride)):
        if t is None:
            continue
        s = _stride_of(name, t, (B, h, d) if rows else (B, T, h, d), dt, dev)
        if B * T > 1 and s != (stride or h * d):
            raise ValueError(f"{name}: a token stride of {s} where seq has {stride or h * d}")
    return dt, dev


def _check_workspace(ws, ws_bytes, device):
    if hasattr(ws, "numel"):
        if not ws.is_contiguous() or ws.device != device or ws.numel() * ws.element_size() < ws_bytes:
            raise ValueError(f"ws must be a contiguous tensor of at least ws_bytes = {ws_bytes} bytes on {device}")


def _call(fn, device, stream, *args) -> int:
    """fn(*args, stream) with `device` current; stream: None for its current one."""
    import torch
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(device.index)     # current_stream() without its object
    else:
        s = stream if isinstance(stream, int) else stream.cuda_stream
    if device.index == torch.cuda.current_device():
        return fn(*args, s)
    with torch.cuda.device(device):
        return fn(*args, s)


def _check_gated(seq, dt, dev, g, lens, states, **tensors):
    """g [B, T, Hk], lens and states (name: tensor or None) and, by name, tensors with their head counts."""
    import torch
    B, T, Hk, d = seq.batch, seq.tokens, seq.kv_heads, seq.head_dim
    _need("g", g, (B, T, Hk), torch.float32, dev)
    if lens is not None:
        _need("lens", lens, (B,), torch.int32, dev)
    for name, t in states.items():
        if t is not None:
            _need(name, t, (B, Hk, d, d), torch.float32, dev)
    for name, (t, h) in tensors.items():
        _need(name, t, (B, T, h, d), dt, dev)


def mhla_gated_forward(q, k, v, g, seq: mhla_seq, out, lens=None, state=None, state_out=None, ws=None,
                       ws_bytes: int = 0, stream=None) -> int:
    """The C entry point with torch tensors: q, out [B, T, H, d], k, v [B, T, Hk, d], g fp32 [B, T, Hk],
    lens int32 [B] or None, state and state_out fp32 [B, Hk, d, d] or None."""
    dt, dev = _check_seq_tensors(q, k, v, seq)
    _check_gated(seq, dt, dev, g, lens, {"state": state, "state_out": state_out}, out=(out, seq.heads))
    _check_workspace(ws, ws_bytes, dev)
    return _call(lib().mhla_gated_forward, dev, stream, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lens), _ptr(state),
                 ctypes.byref(seq), _ptr(out), _ptr(state_out), _ptr(ws), ws_bytes)


def mhla_gated_backward(q, k, v, g, dout, seq: mhla_seq, dq, dk, dv, dg, lens=None, state=None, dstate_out=None,
                        dstate=None, ws=None, ws_bytes: int = 0, stream=None) -> int:
    """Gradients through mhla_gated_forward: dq, dk, dv like q, k, v (contiguous), dg like g; dstate_out is the
    final state's gradient (or None), dstate receives the initial state's (or None)."""
    import torch
    dt, dev = _check_seq_tensors(q, k, v, seq)
    H, Hk = seq.heads, seq.kv_heads
    _check_gated(seq, dt, dev, g, lens, {"state": state, "dstate_out": dstate_out, "dstate": dstate}, dout=(dout, H),
                 dq=(dq, H), dk=(dk, Hk), dv=(dv, Hk))
    _need("dg", dg, g.shape, torch.float32, dev)
    _check_workspace(ws, ws_bytes, dev)
    return _call(lib().mhla_gated_backward, dev, stream, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lens), _ptr(state),
                 _ptr(dout), _ptr(dstate_out), ctypes.byref(seq), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg),
                 _ptr(dstate), _ptr(ws), ws_bytes)


def _check_step(seq, dev, g, state, slots):
    import torch
    B, Hk, d = seq.batch, seq.kv_heads, seq.head_dim
    n = state.shape[0]
    _need("g", g, (B, Hk), torch.float32, dev)
    _need("state", state, (n, Hk, d, d), torch.float32, dev)
    if slots is not None:
        _need("slots", slots, (B,), torch.int32, dev)
    return n


def mhla_gated_step(q, k, v, g, seq: mhla_seq, state, out, slots=None, stream=None) -> int:
    """One token a row: q, out [B, H, d], k, v [B, Hk, d], g fp32 [B, Hk], state fp32 [num_slots, Hk, d, d]
    (updated in place), slots int32 [B] or None (row b has entry b)."""
    dt, dev = _check_seq_tensors(q, k, v, seq, rows=True)
    n = _check_step(seq, dev, g, state, slots)
    _need("out", out, (seq.batch, seq.heads, seq.head_dim), dt, dev)
    return _call(lib().mhla_gated_step, dev, stream, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(slots),
                 ctypes.byref(seq), _ptr(state), n, _ptr(out))


def _check_rope_tensors(w_q, w_k, positions, freq, rope: mhla_rope, seq: mhla_seq, dev):
    import torch
    _need("positions", positions, (seq.batch, seq.tokens, rope.axes), torch.int32, dev)
    _need("freq", freq, (sum(rope.section),), torch.float32, dev)
    for name, t in (("w_q", w_q), ("w_k", w_k)):
        if t is not None:
            _need(name, t, (seq.head_dim,), torch.float32, dev)


def mhla_qk_norm_rope(q, k, w_q, w_k, positions, freq, rope: mhla_rope, seq: mhla_seq, q_out, k_out,
                      stream=None) -> int:
    """q, q_out [B, T, H, d], k, k_out [B, T, Hk, d], w_q, w_k fp32 [d] or None, positions int32 [B, T, axes],
    freq fp32 [pairs]."""
    dt, dev = _check_seq_tensors(q, k, None, seq)
    _check_rope_tensors(w_q, w_k, positions, freq, rope, seq, dev)
    _need("q_out", q_out, q.shape, dt, dev)
    _need("k_out", k_out, k.shape, dt, dev)
    return _call(lib().mhla_qk_norm_rope, dev, stream, _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k), _ptr(positions),
                 _ptr(freq), ctypes.byref(rope), ctypes.byref(seq), _ptr(q_out), _ptr(k_out))


def mhla_qk_norm_rope_backward(q, k, w_q, w_k, positions, freq, rope: mhla_rope, dq_out, dk_out, seq: mhla_seq, dq,
                               dk, dw_q=None, dw_k=None, ws=None, ws_bytes: int = 0, stream=None) -> int:
    """Gradients through mhla_qk_norm_rope; dw_q, dw_k fp32 [d] or None."""
    import torch
    dt, dev = _check_seq_tensors(q, k, None, seq)
    _check_rope_tensors(w_q, w_k, positions, freq, rope, seq, dev)
    for name, t, like in (("dq_out", dq_out, q), ("dq", dq, q), ("dk_out", dk_out, k), ("dk", dk, k)):
        _need(name, t, like.shape, dt, dev)
    for name, t in (("dw_q", dw_q), ("dw_k", dw_k)):
        if t is not None:
            _need(name, t, (seq.head_dim,), torch.float32, dev)
    _check_workspace(ws, ws_bytes, dev)
    return _call(lib().mhla_qk_norm_rope_backward, dev, stream, _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k),
                 _ptr(positions), _ptr(freq), ctypes.byref(rope), _ptr(dq_out), _ptr(dk_out), ctypes.byref(seq),
                 _ptr(dq), _ptr(dk), _ptr(dw_q), _ptr(dw_k), _ptr(ws), ws_bytes)


def _seq_of(q, k, v, scale=None, rows: bool = False):
    """The sequence problem of tensors q [B, T, H, d], k and v [B, T, Hk, d] (v or None; rows: without T, one
    token each), checked against each other, and their device."""
    import torch
    n = 3 if rows else 4
    if q.dim() != n or k.dim() != n:
        raise ValueError("q, k and v must be [batch, heads, head_dim]" if rows else
                         "q, k and v must be [batch, tokens, heads, head_dim]")
    t, dev = q.dtype, q.device
    dt = MHLA_BF16 if t == torch.bfloat16 else MHLA_F32 if t == torch.float32 else None
    if dt is None:
        raise ValueError(f"q must be bfloat16 or float32, got {t}")
    shape = q.shape
    H, d = shape[-2], shape[-1]
    Hk = k.shape[-2]
    kv = (*shape[:-2], Hk, d)
    qs, ks = _stride_of("q", q, shape, t, dev), _stride_of("k", k, kv, t, dev)
    vs = 0 if v is None else _stride_of("v", v, kv, t, dev)
    if dev.type != "cuda":
        raise ValueError("q must be on a GPU")
    return mhla_seq(shape[0], 1 if rows else shape[1], H, Hk, d, dt, qs, ks, vs,
                    d ** -0.5 if scale is None else scale), dev


def _workspace(n, device):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _raise(st, what):
    if st != MHLA_OK:
        raise MhlaError(st, what)


def gated_forward(q, k, v, g, scale=None, state=None, lens=None, want_state: bool = False):
    """Gated linear attention over a sequence: S_t = exp(g_t) S_{t-1} + k_t v_t^T, out_t = scale S_t^T q_t
    (scale: head_dim ** -0.5 by default).  Returns out, and with want_state (out, the final state).  Runs on the
    current stream of the tensors' device; tensors as for mhla_gated_forward."""
    import torch
    seq, dev = _seq_of(q, k, v, scale)
    _check_gated(seq, q.dtype, dev, g, lens, {"state": state})
    out = q.new_empty(q.shape)
    new = None
    if want_state:
        new = torch.empty(seq.batch, seq.kv_heads, seq.head_dim, seq.head_dim, dtype=torch.float32, device=dev)
    n = mhla_gated_workspace_bytes(seq)
    ws = _workspace(n, dev)
    _raise(_call(lib().mhla_gated_forward, dev, None, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lens), _ptr(state),
                 ctypes.byref(seq), _ptr(out), _ptr(new), _ptr(ws), n), "mhla_gated_forward")
    return (out, new) if want_state else out


def gated_backward(q, k, v, g, dout, scale=None, state=None, dstate=None, lens=None):
    """(dq, dk, dv, dg, gradient of the initial state) of gated_forward, given dout and, if not None, dstate, the
    final state's gradient.  The last one is None where state is."""
    import torch
    seq, dev = _seq_of(q, k, v, scale)
    _check_gated(seq, q.dtype, dev, g, lens, {"state": state, "dstate": dstate}, dout=(dout, seq.heads))
    dq, dk, dv = (t.new_empty(t.shape) for t in (q, k, v))
    dg = torch.empty_like(g)
    dstart = None if state is None else torch.empty_like(state)
    n = mhla_gated_backward_workspace_bytes(seq)
    ws = _workspace(n, dev)
    _raise(_call(lib().mhla_gated_backward, dev, None, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(lens), _ptr(state),
                 _ptr(dout), _ptr(dstate), ctypes.byref(seq), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(dstart),
                 _ptr(ws), n), "mhla_gated_backward")
    return dq, dk, dv, dg, dstart


def gated_step(q, k, v, g, state, scale=None, slots=None):
    """One token for each row: q [B, H, d], k, v [B, Hk, d], g [B, Hk]; state [num_slots, Hk, d, d] is updated in
    place.  Returns out [B, H, d].  slots as for mhla_gated_step."""
    seq, dev = _seq_of(q, k, v, scale, rows=True)
    n = _check_step(seq, dev, g, state, slots)
    out = q.new_empty(q.shape)
    _raise(_call(lib().mhla_gated_step, dev, None, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(slots),
                 ctypes.byref(seq), _ptr(state), n, _ptr(out)), "mhla_gated_step")
    return out


def qk_norm_rope(q, k, w_q, w_k, positions, freq, sections=None, style: int = MHLA_ROPE_HALVES, eps: float = 1e-6):
    """RMSNorm of every head of q and k with weights w_q, w_k (or None), and the rotation by the tokens'
    positions.  sections: pairs of each axis (one axis for all of freq by default).  Returns (q, k)."""
    seq, dev = _seq_of(q, k, None, 1.0)
    rope = make_rope(sections if sections is not None else (freq.numel(),), style, eps)
    _check_rope_tensors(w_q, w_k, positions, freq, rope, seq, dev)
    qo = q.new_empty(q.shape)
    ko = k.new_empty(k.shape)
    _raise(_call(lib().mhla_qk_norm_rope, dev, None, _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k), _ptr(positions),
                 _ptr(freq), ctypes.byref(rope), ctypes.byref(seq), _ptr(qo), _ptr(ko)), "mhla_qk_norm_rope")
    return qo, ko


def qk_norm_rope_backward(q, k, w_q, w_k, positions, freq, sections, dq_out, dk_out, style: int = MHLA_ROPE_HALVES,
                          eps: float = 1e-6):
    """(dq, dk, dw_q, dw_k) of qk_norm_rope; a weight's gradient is None where the weight is."""
    import torch
    seq, dev = _seq_of(q, k, None, 1.0)
    rope = make_rope(sections if sections is not None else (freq.numel(),), style, eps)
    _check_rope_tensors(w_q, w_k, positions, freq, rope, seq, dev)
    _need("dq_out", dq_out, q.shape, q.dtype, dev)
    _need("dk_out", dk_out, k.shape, k.dtype, dev)
    dq = q.new_empty(q.shape)
    dk = k.new_empty(k.shape)
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (w_q, w_k))
    n = mhla_qk_norm_rope_backward_workspace_bytes(seq)
    ws = _workspace(n, dev)
    _raise(_call(lib().mhla_qk_norm_rope_backward, dev, None, _ptr(q), _ptr(k), _ptr(w_q), _ptr(w_k), _ptr(positions),
                 _ptr(freq), ctypes.byref(rope), _ptr(dq_out), _ptr(dk_out), ctypes.byref(seq), _ptr(dq), _ptr(dk),
                 _ptr(dwq), _ptr(dwk), _ptr(ws), n), "mhla_qk_norm_rope_backward")
    return dq, dk, dwq, dwk
