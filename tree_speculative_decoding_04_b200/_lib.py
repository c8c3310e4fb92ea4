"""ctypes binding of libtreeverify.so -- argument marshalling only.

Each function has the name of the C entry point it calls and takes torch tensors
that already live on the GPU; every step of the computation runs in the CUDA
library.  There is no fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtreeverify.so")

TV_OK = 0
SEQ_BAD_PARENT = 1
SEQ_TOO_DEEP = 2
SEQ_TIMEOUT = 4
SEQ_BAD_GEOMETRY = 8
MAX_TREE_ROWS = 256
ATTN_PREFIX_READY = 1
ATTN_ROPE = 2

EXPORTS = (
    "tree_build_mask",
    "tree_attention_workspace_size",
    "tree_attention",
    "tree_attention_noalloc_max_scratch",
    "tree_attention_noalloc",
    "tree_attention_scored_workspace_size",
    "tree_attention_scored",
    "tree_accept",
    "tree_accept_lm_head_workspace_size",
    "tree_accept_lm_head",
    "tree_accept_sample_workspace_size",
    "tree_accept_sample",
    "kv_commit_realign",
    "tree_kv_write",
    "tree_qk_norm_rope",
    "tv_status_string",
    "tv_last_cuda_error",
    "tv_version",
    "tv_set_wait_limit_ns",
)


class TVError(RuntimeError):
    pass


_lib = None


def load(path: str = LIB_PATH):
    """Load the shared library (built by build.py) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise TVError(f"CUDA library not built: {path} (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    P, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    lib.tree_build_mask.argtypes = [P, i32, i32, i32, P, P, P, P]
    lib.tree_attention_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64]
    lib.tree_attention_workspace_size.restype = ctypes.c_size_t
    lib.tree_attention.argtypes = [P, P, P, i64, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P, ctypes.c_size_t,
                                   ctypes.c_uint, P, f32, P, i32, P]
    lib.tree_attention_noalloc_max_scratch.argtypes = []
    lib.tree_attention_noalloc_max_scratch.restype = ctypes.c_size_t
    lib.tree_attention_noalloc.argtypes = [P, P, P, i64, P, P, P, P, i32, i32, i32, i32, i32, f32, P, P]
    lib.tree_attention_noalloc.restype = ctypes.c_int
    lib.tree_accept.argtypes = [P, P, P, P, P, P, i32, i32, i32, i32, P, P, P, P, P]
    lib.tree_accept_lm_head_workspace_size.argtypes = [i32, i32]
    lib.tree_accept_lm_head_workspace_size.restype = ctypes.c_size_t
    lib.tree_accept_lm_head.argtypes = [P, P, P, P, P, P, P, i32, i32, i32, i32, i32, P, P, P, P, P, ctypes.c_size_t,
                                        P]
    lib.kv_commit_realign.argtypes = [P, P, i32, i32, i32, i32, i64, i32, P, P, P, i32, P, P, P, i32, P, P, P, i32, P]
    lib.tree_kv_write.argtypes = [P, P, P, P, i32, i32, i32, i32, i64, i32, P, P, P, f32, P, i32, P]
    lib.tree_attention_scored_workspace_size.argtypes = [i32, i32, i32, i32, i32, i64, i32]
    lib.tree_attention_scored_workspace_size.restype = ctypes.c_size_t
    lib.tree_attention_scored.argtypes = [P, P, P, i64, P, P, P, P, P, i32, i32, i32, i32, i32, f32, f32, i32, P, P,
                                          P, ctypes.c_size_t, P, i32, P]
    lib.tree_accept_sample_workspace_size.argtypes = [i32, i32, i32]
    lib.tree_accept_sample_workspace_size.restype = ctypes.c_size_t
    lib.tree_accept_sample.argtypes = [P, i32, i64, P, P, P, P, P, P, P, P, P, P, i32, i32, i32, i32, P, P, P, P, P,
                                       P, ctypes.c_size_t, P]
    lib.tree_qk_norm_rope.argtypes = [P, i64, P, P, f32, f32, P, P, P, i64, P, P, P, i32, i32, i32, i32, i32, i32,
                                      f32, P, i32, P]
    for name in ("tree_build_mask", "tree_attention", "tree_accept", "tree_accept_lm_head", "kv_commit_realign",
                 "tree_kv_write", "tree_attention_scored", "tree_accept_sample", "tree_qk_norm_rope"):
        getattr(lib, name).restype = ctypes.c_int
    lib.tv_status_string.argtypes = [ctypes.c_int]
    lib.tv_status_string.restype = ctypes.c_char_p
    lib.tv_last_cuda_error.restype = ctypes.c_int
    lib.tv_version.restype = ctypes.c_int
    lib.tv_set_wait_limit_ns.argtypes = [ctypes.c_uint64]
    lib.tv_set_wait_limit_ns.restype = None
    _lib = lib
    return lib


def _check(rc: int, what: str):
    if rc != TV_OK:
        lib = load()
        msg = lib.tv_status_string(rc).decode()
        if msg == "TV_ERR_CUDA":
            msg += f" (cudaError {lib.tv_last_cuda_error()})"
        raise TVError(f"{what}: {msg}")


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise TVError("tensor must live on the GPU")
    if not t.is_contiguous():
        raise TVError("tensor must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


class _on:
    """The device `dev` as the current one for a call, and the call's stream (the
    given one, else that device's current one) as its pointer."""

    __slots__ = ("dev", "stream", "back")

    def __init__(self, stream, dev):
        self.dev, self.stream, self.back = dev, stream, -1

    def __enter__(self):
        current = torch._C._cuda_getDevice()
        if current != self.dev:
            self.back = current
            torch.cuda.set_device(self.dev)
        if self.stream is None:
            return torch._C._cuda_getCurrentRawStream(self.dev)
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.back >= 0:
            torch.cuda.set_device(self.back)
        return False


def _arg(t, dtype, shape, name, dev, rows=False):
    """The address of a checked argument: dtype, shape, the call's GPU, contiguous
    (rows: its strides are checked by _row_stride)."""
    if t.dtype is not dtype:
        raise TVError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise TVError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != dev:
        raise TVError("tensors must live on one GPU" if t.is_cuda else "tensor must live on the GPU")
    if not rows and not t.is_contiguous():
        raise TVError("tensor must be contiguous")
    return t.data_ptr()


def _scratch(t, dev):
    """(address, bytes) of a workspace tensor, or (None, 0)."""
    if t is None:
        return None, 0
    if t.get_device() != dev:
        raise TVError("tensors must live on one GPU" if t.is_cuda else "tensor must live on the GPU")
    if not t.is_contiguous():
        raise TVError("tensor must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


def _gpu_of(t) -> int:
    """The GPU of a call's first tensor; the others must live there too."""
    dev = t.get_device()
    if dev < 0:
        raise TVError("tensor must live on the GPU")
    return dev


def _row_stride(t: torch.Tensor, width: int, name: str) -> int:
    """Elements between the rows of t [B][M+1][...], each row `width` contiguous
    elements and all rows evenly spaced (a dense tensor, or the leading columns of
    one that is wider)."""
    B, n = t.shape[0], t.shape[1]
    inner, want = t.stride()[2:], 1
    for size, st in zip(reversed(t.shape[2:]), reversed(inner)):
        if size != 1 and st != want:
            raise TVError(f"{name}: a row must be contiguous")
        want *= size
    if B * n <= 1:
        return width
    row = t.stride(1) if n > 1 else t.stride(0)
    if row < width or (B > 1 and n > 1 and t.stride(0) != n * row):
        raise TVError(f"{name}: rows must be evenly spaced")
    return row


def _need(t: torch.Tensor, dtype, shape, name):
    if t.dtype != dtype:
        raise TVError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise TVError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")


def tree_build_mask(parent, max_depth, anc_mask, depth, status, stream=None):
    """parent int32 [B][M+1] -> anc_mask uint32-as-int32 [B][M+1][W], depth [B][M+1], status [B]."""
    B, n = parent.shape
    W = (n + 31) // 32
    _need(parent, torch.int32, (B, n), "parent")
    _need(anc_mask, torch.int32, (B, n, W), "anc_mask")
    _need(depth, torch.int32, (B, n), "depth")
    _need(status, torch.int32, (B,), "status")
    rc = load().tree_build_mask(_ptr(parent), B, n - 1, int(max_depth), _ptr(anc_mask), _ptr(depth),
                                _ptr(status), _stream(stream))
    _check(rc, "tree_build_mask")


def tree_attention_workspace_size(B, M, Hq, Hkv, D, S_cap) -> int:
    """Bytes of device scratch tree_attention needs for this shape (0 = none)."""
    return int(load().tree_attention_workspace_size(B, M, Hq, Hkv, D, int(S_cap)))


def attention_workspace(B, M, Hq, Hkv, D, S_cap, device) -> torch.Tensor | None:
    """A device buffer of the workspace size (None when no workspace is needed)."""
    nbytes = tree_attention_workspace_size(B, M, Hq, Hkv, D, S_cap)
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)


def tree_attention(q, k, v, kv_start, kv_len, anc_mask, status, out, workspace=None, scale=None, stream=None,
                   flags=0, depth=None, rope_theta=0.0, slot=None):
    """q [B][M+1][Hq][D] bf16; k, v [B][Hkv][S_cap][D] bf16 (one layer) -> out like q.
    workspace: a uint8 device tensor of at least tree_attention_workspace_size bytes.
    flags: an OR of ATTN_PREFIX_READY (the launch just before this one on the
    stream writes neither the geometry, the slot map nor any prefix K/V column)
    and ATTN_ROPE (q is rotated to kv_len + depth[b][u] with base rope_theta).
    slot: int32 [B] cache slots; k, v are then a pool [n_slots][Hkv][S_cap][D]
    and kv_start / kv_len are [n_slots]."""
    B, n, Hq, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    NS = k.shape[0] if slot is not None else B
    _need(q, torch.bfloat16, (B, n, Hq, D), "q")
    _need(k, torch.bfloat16, (NS, Hkv, S_cap, D), "k")
    _need(v, torch.bfloat16, (NS, Hkv, S_cap, D), "v")
    _need(kv_start, torch.int32, (NS,), "kv_start")
    _need(kv_len, torch.int32, (NS,), "kv_len")
    if slot is not None:
        _need(slot, torch.int32, (B,), "slot")
    if flags & ATTN_ROPE:
        _need(depth, torch.int32, (B, n), "depth")
    _need(anc_mask, torch.int32, (B, n, (n + 31) // 32), "anc_mask")
    _need(status, torch.int32, (B,), "status")
    _need(out, torch.bfloat16, (B, n, Hq, D), "out")
    if scale is None:
        scale = D ** -0.5
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = load().tree_attention(_ptr(q), _ptr(k), _ptr(v), S_cap, _ptr(kv_start), _ptr(kv_len), _ptr(anc_mask),
                               _ptr(status), B, n - 1, Hq, Hkv, D, float(scale), _ptr(out), _ptr(workspace),
                               ws_bytes, int(flags), _ptr(depth) if flags & ATTN_ROPE else None,
                               float(rope_theta), _ptr(slot), NS, _stream(stream))
    _check(rc, "tree_attention")


def tree_accept(logits, draft, parent, depth, anc_mask, status, max_depth, argmax, accept_len, path, bonus,
                stream=None):
    B, n, V = logits.shape
    _need(logits, torch.float32, (B, n, V), "logits")
    for t, name in ((draft, "draft"), (parent, "parent"), (depth, "depth"), (argmax, "argmax")):
        _need(t, torch.int32, (B, n), name)
    _need(anc_mask, torch.int32, (B, n, (n + 31) // 32), "anc_mask")
    _need(status, torch.int32, (B,), "status")
    _need(accept_len, torch.int32, (B,), "accept_len")
    _need(path, torch.int32, (B, int(max_depth) + 1), "path")
    _need(bonus, torch.int32, (B,), "bonus")
    rc = load().tree_accept(_ptr(logits), _ptr(draft), _ptr(parent), _ptr(depth), _ptr(anc_mask), _ptr(status),
                            B, n - 1, V, int(max_depth), _ptr(argmax), _ptr(accept_len), _ptr(path), _ptr(bonus),
                            _stream(stream))
    _check(rc, "tree_accept")


def lm_head_workspace(B, M, device) -> torch.Tensor:
    """A device buffer of tree_accept_lm_head_workspace_size bytes."""
    nbytes = int(load().tree_accept_lm_head_workspace_size(B, M))
    return torch.empty((max(nbytes, 8) + 15) // 16 * 16, dtype=torch.uint8, device=device)


def tree_accept_lm_head(hidden, w_lm, draft, parent, depth, anc_mask, status, max_depth, argmax, accept_len, path,
                        bonus, workspace, stream=None):
    """hidden bf16 [B][M+1][H], w_lm bf16 [V][H] -> argmax of hidden @ w_lm^T per node
    (the logits are never stored), then the acceptance walk (as tree_accept)."""
    B, n, H = hidden.shape
    V = w_lm.shape[0]
    _need(hidden, torch.bfloat16, (B, n, H), "hidden")
    _need(w_lm, torch.bfloat16, (V, H), "w_lm")
    for t, name in ((draft, "draft"), (parent, "parent"), (depth, "depth"), (argmax, "argmax")):
        _need(t, torch.int32, (B, n), name)
    _need(anc_mask, torch.int32, (B, n, (n + 31) // 32), "anc_mask")
    _need(status, torch.int32, (B,), "status")
    _need(accept_len, torch.int32, (B,), "accept_len")
    _need(path, torch.int32, (B, int(max_depth) + 1), "path")
    _need(bonus, torch.int32, (B,), "bonus")
    ws_bytes = workspace.numel() * workspace.element_size()
    rc = load().tree_accept_lm_head(_ptr(hidden), _ptr(w_lm), _ptr(draft), _ptr(parent), _ptr(depth), _ptr(anc_mask),
                                    _ptr(status), B, n - 1, H, V, int(max_depth), _ptr(argmax), _ptr(accept_len),
                                    _ptr(path), _ptr(bonus), _ptr(workspace), ws_bytes, _stream(stream))
    _check(rc, "tree_accept_lm_head")


def attention_scored_workspace_size(B, M, Hq, Hkv, D, S_cap, window) -> int:
    """Bytes of device scratch tree_attention_scored needs for this shape on the
    current device (0 = none: key ranges are not split)."""
    return int(load().tree_attention_scored_workspace_size(B, M, Hq, Hkv, D, int(S_cap), int(window)))


def attention_scored_workspace(B, M, Hq, Hkv, D, S_cap, window, device) -> torch.Tensor | None:
    """A device buffer of tree_attention_scored_workspace_size bytes for this shape
    (None when no workspace is needed).  Calls that may overlap need one each."""
    with torch.cuda.device(device):
        nbytes = attention_scored_workspace_size(B, M, Hq, Hkv, D, S_cap, window)
    if nbytes == 0:
        return None
    return torch.empty((nbytes + 15) // 16 * 16, dtype=torch.uint8, device=device)


def tree_attention_scored(q, k, v, kv_start, kv_len, anc_mask, depth, status, out, workspace=None, scale=None,
                          softcap=0.0, window=0, alibi_slopes=None, stream=None, slot=None):
    """tree_attention with capped, local or distance-biased scores.

    q [B][M+1][Hq][D] bf16; k, v [B][Hkv][S_cap][D] bf16 (one layer; with slot a
    pool [n_slots][Hkv][S_cap][D], kv_start / kv_len [n_slots]) -> out like q.
    softcap: s -> softcap * tanh(s / softcap) (0: off).  window: only keys closer
    than this many positions (0: off).  alibi_slopes fp32 [Hq]: s - slope *
    distance.  workspace: attention_scored_workspace(...)."""
    B, n, Hq, D = q.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    NS = k.shape[0] if slot is not None else B
    bf, i32 = torch.bfloat16, torch.int32
    # (shapes and types first: they are wrong on any device)
    dev = q.get_device()
    a_q, a_k, a_v = (_arg(q, bf, (B, n, Hq, D), "q", dev), _arg(k, bf, (NS, Hkv, S_cap, D), "k", dev),
                     _arg(v, bf, (NS, Hkv, S_cap, D), "v", dev))
    a_ks, a_kl = _arg(kv_start, i32, (NS,), "kv_start", dev), _arg(kv_len, i32, (NS,), "kv_len", dev)
    a_anc, a_dep = _arg(anc_mask, i32, (B, n, (n + 31) // 32), "anc_mask", dev), _arg(depth, i32, (B, n), "depth", dev)
    a_st, a_out = _arg(status, i32, (B,), "status", dev), _arg(out, bf, (B, n, Hq, D), "out", dev)
    a_slot = None if slot is None else _arg(slot, i32, (B,), "slot", dev)
    a_slopes = None if alibi_slopes is None else _arg(alibi_slopes, torch.float32, (Hq,), "alibi_slopes", dev)
    a_ws, ws_bytes = _scratch(workspace, dev)
    if scale is None:
        scale = D ** -0.5
    with _on(stream, _gpu_of(q)) as s:
        rc = load().tree_attention_scored(a_q, a_k, a_v, S_cap, a_ks, a_kl, a_anc, a_dep, a_st, B, n - 1, Hq, Hkv, D,
                                          float(scale), float(softcap), int(window), a_slopes, a_out, a_ws, ws_bytes, a_slot, NS, s)
    _check(rc, "tree_attention_scored")


def accept_sample_workspace(B, M, V, device) -> torch.Tensor:
    """A device buffer of tree_accept_sample_workspace_size bytes for this shape.
    Calls that may overlap need one each."""
    nbytes = int(load().tree_accept_sample_workspace_size(B, M, V))
    return torch.empty((max(nbytes, 8) + 15) // 16 * 16, dtype=torch.uint8, device=device)


def tree_accept_sample(logits, uniform, temperature, draft, parent, depth, anc_mask, status, max_depth, token,
                       accept_len, path, bonus, workspace, top_k=None, top_p=None, min_p=None, logprob=None,
                       stream=None):
    """tree_accept with a token drawn at every node instead of the argmax.

    logits fp32 or bf16 [B][M+1][V] (evenly spaced rows, such as the first V
    columns of a padded vocabulary); uniform fp32 [B][M+1]; temperature fp32 [B]
    (<= 0: greedy); top_k int32 [B], top_p / min_p fp32 [B] or None (off).  Writes
    token int32 [B][M+1], logprob fp32 [B][M+1] (optional), accept_len, path and
    bonus.  workspace: accept_sample_workspace(...)."""
    B, n, V = logits.shape
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise TVError(f"logits: dtype {logits.dtype}, expected torch.float32 or torch.bfloat16")
    i32, f32, md = torch.int32, torch.float32, int(max_depth)
    dev = logits.get_device()
    stride = _row_stride(logits, V, "logits")
    per_node, per_row = (B, n), (B,)
    a_u = _arg(uniform, f32, per_node, "uniform", dev)
    a_T = _arg(temperature, f32, per_row, "temperature", dev)
    a_k = None if top_k is None else _arg(top_k, i32, per_row, "top_k", dev)
    a_p = None if top_p is None else _arg(top_p, f32, per_row, "top_p", dev)
    a_m = None if min_p is None else _arg(min_p, f32, per_row, "min_p", dev)
    a_lp = None if logprob is None else _arg(logprob, f32, per_node, "logprob", dev)
    a_draft, a_par = _arg(draft, i32, per_node, "draft", dev), _arg(parent, i32, per_node, "parent", dev)
    a_dep, a_tok = _arg(depth, i32, per_node, "depth", dev), _arg(token, i32, per_node, "token", dev)
    a_anc, a_st = _arg(anc_mask, i32, (B, n, (n + 31) // 32), "anc_mask", dev), _arg(status, i32, per_row, "status", dev)
    a_al, a_path = _arg(accept_len, i32, per_row, "accept_len", dev), _arg(path, i32, (B, md + 1), "path", dev)
    a_bonus = _arg(bonus, i32, per_row, "bonus", dev)
    a_ws, ws_bytes = _scratch(workspace, dev)
    with _on(stream, _gpu_of(logits)) as s:
        rc = load().tree_accept_sample(logits.data_ptr(), int(logits.dtype is torch.bfloat16), stride, a_u, a_T, a_k,
                                       a_p, a_m, a_draft, a_par, a_dep, a_anc, a_st, B, n - 1, V, md, a_tok, a_lp, a_al,
                                       a_path, a_bonus, a_ws, ws_bytes, s)
    _check(rc, "tree_accept_sample")


def tree_qk_norm_rope(qkv, q_weight, k_weight, q_out, k, v, kv_start, kv_len, depth, eps=1e-6, weight_offset=0.0,
                      rope_theta=10000.0, rotary_dim=None, stream=None, slot=None):
    """The packed projection rows of one layer -> queries and cache rows.

    qkv bf16 [B][M+1][Hq + 2 Hkv][D] (evenly spaced rows): every query and key head
    is RMS-normalised, scaled by weight_offset + its weight (bf16 [D], None: no
    weight) and rotated to kv_len + depth over its first rotary_dim elements
    (default D, 0: no rotation); q goes to q_out [B][M+1][Hq][D], k and v rows to
    columns kv_start + kv_len + r of the layer's cache k, v [B][Hkv][S_cap][D] (a
    pool [n_slots][Hkv][S_cap][D] with slot)."""
    B, n, Hq, D = q_out.shape
    Hkv, S_cap = k.shape[1], k.shape[2]
    NS = k.shape[0] if slot is not None else B
    heads = Hq + 2 * Hkv
    bf, i32 = torch.bfloat16, torch.int32
    dev = q_out.get_device()
    a_qkv = _arg(qkv, bf, (B, n, heads, D), "qkv", dev, rows=True)
    stride = _row_stride(qkv, heads * D, "qkv")
    a_qo = _arg(q_out, bf, (B, n, Hq, D), "q_out", dev)
    a_wq = None if q_weight is None else _arg(q_weight, bf, (D,), "q_weight", dev)
    a_wk = None if k_weight is None else _arg(k_weight, bf, (D,), "k_weight", dev)
    a_k, a_v = _arg(k, bf, (NS, Hkv, S_cap, D), "k", dev), _arg(v, bf, (NS, Hkv, S_cap, D), "v", dev)
    a_ks, a_kl = _arg(kv_start, i32, (NS,), "kv_start", dev), _arg(kv_len, i32, (NS,), "kv_len", dev)
    a_dep = _arg(depth, i32, (B, n), "depth", dev)
    a_slot = None if slot is None else _arg(slot, i32, (B,), "slot", dev)
    with _on(stream, _gpu_of(q_out)) as s:
        rc = load().tree_qk_norm_rope(a_qkv, stride, a_wq, a_wk, float(weight_offset), float(eps), a_qo, a_k, a_v, S_cap, a_ks, a_kl,
                                      a_dep, B, n - 1, Hq, Hkv, D, D if rotary_dim is None else int(rotary_dim),
                                      float(rope_theta), a_slot, NS, s)
    _check(rc, "tree_qk_norm_rope")


def kv_commit_realign(k_layer_ptrs, v_layer_ptrs, B, Hkv, D, S_cap, M, path, accept_len, status, max_depth,
                      kv_start, kv_len, max_len, realign, attn_mask=None, pos_ids=None, stream=None, slot=None):
    """k_layer_ptrs / v_layer_ptrs: int64 CUDA tensors [L] of layer base addresses
    (each layer a bf16 [B][Hkv][S_cap][D] buffer, or a pool [n_slots][Hkv][S_cap][D]
    with slot: int32 [B] cache slots, kv_start / kv_len / mask rows per slot)."""
    L = k_layer_ptrs.numel()
    NS = kv_start.shape[0] if slot is not None else B
    _need(k_layer_ptrs, torch.int64, (L,), "k_layer_ptrs")
    _need(v_layer_ptrs, torch.int64, (L,), "v_layer_ptrs")
    _need(path, torch.int32, (B, int(max_depth) + 1), "path")
    for t, name in ((accept_len, "accept_len"), (status, "status")):
        _need(t, torch.int32, (B,), name)
    for t, name in ((kv_start, "kv_start"), (kv_len, "kv_len")):
        _need(t, torch.int32, (NS,), name)
    if slot is not None:
        _need(slot, torch.int32, (B,), "slot")
    _need(max_len, torch.int32, (1,), "max_len")
    if attn_mask is not None:
        _need(attn_mask, torch.uint8, (NS, S_cap), "attn_mask")
    if pos_ids is not None:
        _need(pos_ids, torch.int32, (NS, S_cap), "pos_ids")
    rc = load().kv_commit_realign(_ptr(k_layer_ptrs), _ptr(v_layer_ptrs), L, B, Hkv, D, int(S_cap), M, _ptr(path),
                                  _ptr(accept_len), _ptr(status), int(max_depth), _ptr(kv_start), _ptr(kv_len),
                                  _ptr(max_len), int(realign), _ptr(attn_mask), _ptr(pos_ids), _ptr(slot), NS,
                                  _stream(stream))
    _check(rc, "kv_commit_realign")


def tree_kv_write(k_layer_ptrs, v_layer_ptrs, tree_k, tree_v, S_cap, kv_start, kv_len, stream=None, depth=None,
                  rope_theta=0.0, slot=None):
    """tree_k / tree_v bf16 [L][B][Hkv][M+1][D] -> the cache of every layer, at
    columns kv_start + kv_len + r (k_layer_ptrs / v_layer_ptrs as for
    kv_commit_realign).  depth int32 [B][M+1]: K rows are rotated to kv_len +
    depth with base rope_theta.  slot: int32 [B] cache slots of a pool (kv_start /
    kv_len then [n_slots])."""
    L, B, Hkv, n, D = tree_k.shape
    NS = kv_start.shape[0] if slot is not None else B
    _need(k_layer_ptrs, torch.int64, (L,), "k_layer_ptrs")
    _need(v_layer_ptrs, torch.int64, (L,), "v_layer_ptrs")
    _need(tree_k, torch.bfloat16, (L, B, Hkv, n, D), "tree_k")
    _need(tree_v, torch.bfloat16, (L, B, Hkv, n, D), "tree_v")
    _need(kv_start, torch.int32, (NS,), "kv_start")
    _need(kv_len, torch.int32, (NS,), "kv_len")
    if depth is not None:
        _need(depth, torch.int32, (B, n), "depth")
    if slot is not None:
        _need(slot, torch.int32, (B,), "slot")
    rc = load().tree_kv_write(_ptr(k_layer_ptrs), _ptr(v_layer_ptrs), _ptr(tree_k), _ptr(tree_v), L, B, Hkv, D,
                              int(S_cap), n - 1, _ptr(kv_start), _ptr(kv_len), _ptr(depth), float(rope_theta),
                              _ptr(slot), NS, _stream(stream))
    _check(rc, "tree_kv_write")


def set_wait_limit_ns(ns: int) -> None:
    """Testing hook: limit (ns) of tree_attention's pipeline waits for later
    launches; 0 restores the default (1 s)."""
    load().tv_set_wait_limit_ns(int(ns))


def layer_pointers(layers, device=None) -> torch.Tensor:
    """Device int64 tensor of the base addresses of a list of layer tensors."""
    dev = device or layers[0].device
    return torch.tensor([t.data_ptr() for t in layers], dtype=torch.int64, device=dev)
