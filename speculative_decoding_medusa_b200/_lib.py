"""ctypes binding of libmedusa_b200.so: one Python function per C entry point,
same names, argument marshalling only (tensor -> pointer and sizes, stream
handle).  Every step of the computation runs in the library's CUDA kernels;
there is no fallback: a missing library or a non-OK status raises.  The prompt
side's calls, the shortest, are marshalled by an extension (csrc/marshal.cpp).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmedusa_b200.so")

MEDUSA_BF16 = 0
MEDUSA_F32 = 1
MEDUSA_ROPE_SCALINGS = {"none": 0, "linear": 1, "llama3": 2, "yarn": 3}
MEDUSA_ACCEPT_GREEDY = 0
MEDUSA_ACCEPT_TYPICAL = 1
MAX_NODES = 256
MAX_KMAX = 32
MAX_HEADS = 16
MAX_BATCH = 128

STATUS_NAMES = {
    0: "MEDUSA_OK", 1: "MEDUSA_ERR_INVALID_ARG", 2: "MEDUSA_ERR_SHAPE",
    3: "MEDUSA_ERR_UNSUPPORTED", 4: "MEDUSA_ERR_CUDA", 5: "MEDUSA_ERR_TIMEOUT",
    6: "MEDUSA_ERR_DEVICE_CHECK", 7: "MEDUSA_ERR_WORKSPACE", 8: "MEDUSA_ERR_ALIGNMENT",
}

# exported symbols declared in include/medusa.h
EXPORTS = (
    "medusa_status_string", "medusa_last_error", "medusa_version",
    "medusa_heads_topk_workspace_size", "medusa_heads_topk",
    "medusa_tree_build",
    "medusa_tree_attention_workspace_size", "medusa_tree_attention",
    "medusa_verify_accept_workspace_size", "medusa_verify_accept",
    "medusa_kv_compact", "medusa_verify_accept_compact", "medusa_heads_topk_tree", "medusa_verify_accept_noalloc",
    "medusa_lmhead_verify_workspace_size", "medusa_lmhead_verify", "medusa_next_step",
    "medusa_tree_from_accuracies", "medusa_sample_bonus", "medusa_topk_merge",
    "medusa_verify_records_workspace_size", "medusa_verify_records", "medusa_verify_from_records",
    "medusa_rope_freqs", "medusa_rope", "medusa_rope_append",
    "medusa_chunk_attention_workspace_size", "medusa_chunk_attention", "medusa_sample_tokens",
    "medusa_wait_flag",
)


class MedusaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class medusa_tree_t(ctypes.Structure):
    _fields_ = [("n_nodes", ctypes.c_int32), ("max_depth", ctypes.c_int32),
                ("n_leaves", ctypes.c_int32), ("parent", ctypes.c_void_p),
                ("depth", ctypes.c_void_p), ("rank", ctypes.c_void_p)]


class medusa_rope_t(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("scale", ctypes.c_float), ("turns", ctypes.c_void_p)]


class medusa_pages_t(ctypes.Structure):
    _fields_ = [("K", ctypes.c_void_p), ("V", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32)]


_lib = None

_V, _I, _Z, _F, _U = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_int


def lib() -> ctypes.CDLL:
    """Load the library (built by ``speculative_decoding_medusa_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: run `python -m speculative_decoding_medusa_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    L.medusa_status_string.restype = ctypes.c_char_p
    L.medusa_status_string.argtypes = [_I]
    L.medusa_last_error.restype = ctypes.c_char_p
    L.medusa_last_error.argtypes = []
    L.medusa_version.restype = _I
    L.medusa_heads_topk_workspace_size.restype = _Z
    L.medusa_heads_topk_workspace_size.argtypes = [_I] * 5 + [_I]
    L.medusa_heads_topk.restype = _I
    L.medusa_heads_topk.argtypes = [_V, _V, _V, _V, _I, _I, _I, _I, _I, _I, _V, _V, _V, _V, _Z, _V, _V]
    L.medusa_heads_topk_tree.restype = _I
    L.medusa_heads_topk_tree.argtypes = [_V, _V, _V, _V, _I, _I, _I, _I, _I, _I, _V, _V, _V, _V, _Z,
                                         ctypes.POINTER(medusa_tree_t), _V, _V, _V, _V, _V, _V, _V,
                                         _V]
    L.medusa_tree_build.restype = _I
    L.medusa_tree_build.argtypes = [ctypes.POINTER(medusa_tree_t), _V, _V, _I, _I, _V, _I,
                                    _V, _V, _V, _V, _V, _V]
    L.medusa_tree_attention_workspace_size.restype = _Z
    L.medusa_tree_attention_workspace_size.argtypes = [_I] * 6 + [_I]
    L.medusa_tree_attention.restype = _I
    L.medusa_tree_attention.argtypes = [_V, _V, _V, _V, _V, _V, _V, _I, _I, _I, _I, _I, _I, _I, _I,
                                        _F, _V, _I, _V, _Z, _V, _V]
    L.medusa_verify_accept_workspace_size.restype = _Z
    L.medusa_verify_accept_workspace_size.argtypes = [_I, _I, _I]
    L.medusa_verify_accept.restype = _I
    L.medusa_verify_accept.argtypes = [_V, _I, _V, ctypes.POINTER(medusa_tree_t), _I, _I, _I, _F, _F,
                                       _F, _V, _V, _V, _V, _V, _Z, _V, _V]
    L.medusa_verify_accept_noalloc.restype = _I
    L.medusa_verify_accept_noalloc.argtypes = [_V, _I, _V, ctypes.POINTER(medusa_tree_t), _I, _I, _I,
                                               _F, _F, _F, _V, _V, _V, _V, _V, _V]
    L.medusa_verify_accept_compact.restype = _I
    L.medusa_verify_accept_compact.argtypes = [_V, _I, _V, ctypes.POINTER(medusa_tree_t), _I, _I, _I,
                                               _F, _F, _F, _V, _V, _V, _V, _V, _V, _I, _V, _I, _I,
                                               _I, _V, _V, _Z, _V, _V]
    L.medusa_kv_compact.restype = _I
    L.medusa_kv_compact.argtypes = [_V, _V, _I, _V, _V, _V, _I, _I, _I, _I, _I, _V, _V, _V]
    L.medusa_lmhead_verify_workspace_size.restype = _Z
    L.medusa_lmhead_verify_workspace_size.argtypes = [_I, _I, _I, _I]
    _LL = ctypes.c_longlong
    L.medusa_topk_merge.restype = _I
    L.medusa_topk_merge.argtypes = [_V, _V, _I, _I, _I, _LL, _LL, _V, _I, _V, _V, _V]
    L.medusa_verify_records_workspace_size.restype = _Z
    L.medusa_verify_records_workspace_size.argtypes = [_I, _I, _I]
    L.medusa_verify_records.restype = _I
    L.medusa_verify_records.argtypes = [_V, _I, _V, ctypes.POINTER(medusa_tree_t), _I, _I, _I, _I,
                                        _F, _V, _V, _V, _Z, _V, _V]
    L.medusa_verify_from_records.restype = _I
    L.medusa_verify_from_records.argtypes = [_V, _I, _V, _V, ctypes.POINTER(medusa_tree_t), _I, _I,
                                             _I, _F, _F, _F, _V, _V, _V, _V, _V, _V]
    L.medusa_sample_bonus.restype = _I
    L.medusa_sample_bonus.argtypes = [_V, _I, _V, _V, _I, _I, _I, _I, _F, ctypes.c_uint64,
                                      ctypes.c_uint64, _V, _V, _V, _V]
    L.medusa_tree_from_accuracies.restype = _I
    L.medusa_tree_from_accuracies.argtypes = [_V, _I, _I, _I, _I, _V, _V, _V, _V]
    L.medusa_next_step.restype = _I
    L.medusa_next_step.argtypes = [_V, _I, _V, _V, _V, _I, _I, _I, _I, _V, _V, _V, _V]
    _D = ctypes.c_double
    L.medusa_rope_freqs.restype = _I
    L.medusa_rope_freqs.argtypes = [_I, _D, _I, _D, _D, _D, _D, _V, _V]
    L.medusa_rope.restype = _I
    L.medusa_rope.argtypes = [_V, _V, _LL, _V, _LL, _I, _V, _I, _I, _I, _I, _I, _V, _LL, _V, _LL,
                              _V]
    L.medusa_rope_append.restype = _I
    L.medusa_rope_append.argtypes = [_V, _V, _LL, _V, _LL, _V, _LL, _I, _V, _V, _V, _I, _I, _I,
                                     _I, _I, _V, _LL, _V, _V, _V]
    L.medusa_chunk_attention_workspace_size.restype = _Z
    L.medusa_chunk_attention_workspace_size.argtypes = [_I] * 4
    L.medusa_chunk_attention.restype = _I
    L.medusa_chunk_attention.argtypes = [_V, _LL, _V, _I, _V, _V, _I, _I, _I, _I, _I, _F, _V, _V,
                                         _Z, _V, _V]
    L.medusa_sample_tokens.restype = _I
    L.medusa_sample_tokens.argtypes = [_V, _I, _LL, _I, _V, _I, _I, _V, _V, _V, _V, _V, _V, _V,
                                       _V, _V]
    L.medusa_wait_flag.restype = _I
    L.medusa_wait_flag.argtypes = [_V, ctypes.c_int32, ctypes.c_longlong, _V, _V]
    L.medusa_lmhead_verify.restype = _I
    L.medusa_lmhead_verify.argtypes = [_V, _V, _I, _V, ctypes.POINTER(medusa_tree_t), _I, _I, _I,
                                       _I, _F, _F, _F, _V, _V, _V, _V, _V, _V, _Z, _V, _V]
    _lib = L
    return L


def _check(st: int) -> None:
    if st != 0:
        raise MedusaError(st, lib().medusa_last_error().decode())


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MEDUSA_BF16
    if t.dtype == torch.float32:
        return MEDUSA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _req(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def new_status(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A 256-byte aligned byte buffer (torch's caching allocator aligns to 512)."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


def _own_workspace(nbytes: int, device, stream) -> torch.Tensor:
    """The workspace of a call that was given none.  It is dropped when the call
    returns, so it comes from the pool of the call's stream: whatever gets the
    memory next then follows the call's kernels."""
    if stream is None:
        return workspace(nbytes, device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    with torch.cuda.stream(stream):
        return workspace(nbytes, device)


class Tree:
    """A candidate tree on the device (parent/depth/rank int32 arrays)."""

    def __init__(self, parent, depth, rank, n_leaves: int, device=None):
        dev = device or "cuda"
        self.parent = torch.as_tensor(parent, dtype=torch.int32).to(dev).contiguous()
        self.depth = torch.as_tensor(depth, dtype=torch.int32).to(dev).contiguous()
        self.rank = torch.as_tensor(rank, dtype=torch.int32).to(dev).contiguous()
        self.n_nodes = int(self.parent.numel())
        self.max_depth = int(torch.as_tensor(depth).max().item()) if self.n_nodes else 0
        self.n_leaves = int(n_leaves)

    @classmethod
    def from_spec(cls, spec, device=None) -> "Tree":
        return cls(spec.parent, spec.depth, spec.rank, spec.n_leaves, device)

    def c(self) -> medusa_tree_t:
        return medusa_tree_t(self.n_nodes, self.max_depth, self.n_leaves,
                             self.parent.data_ptr(), self.depth.data_ptr(), self.rank.data_ptr())


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------


def medusa_heads_topk_workspace_size(B: int, d: int, V: int, K: int, kmax: int, dt: int) -> int:
    return int(lib().medusa_heads_topk_workspace_size(B, d, V, K, kmax, dt))


def medusa_heads_topk(h, W1, b1, W2, kmax: int, topk_ids, topk_vals, logits=None, ws=None,
                      dev_status=None, stream=None) -> None:
    """h [B,d], W1 [K,d,d], b1 [K,d], W2 [K,V,d] -> topk_ids/vals [B,K,kmax]
    (and logits [B,K,V] fp32 when given)."""
    for t, n in ((h, "h"), (W1, "W1"), (b1, "b1"), (W2, "W2"), (topk_ids, "topk_ids"),
                 (topk_vals, "topk_vals")):
        _req(t, n)
    B, d = h.shape
    K, V, _ = W2.shape
    dt = _dt(W2)
    if ws is None:
        ws = _own_workspace(medusa_heads_topk_workspace_size(B, d, V, K, kmax, dt), h.device,
                            stream)
    _check(lib().medusa_heads_topk(_p(h), _p(W1), _p(b1), _p(W2), dt, B, d, V, K, kmax,
                                   _p(topk_ids), _p(topk_vals), _p(logits), _p(ws), ws.numel(),
                                   _p(dev_status), _stream(stream)))


def medusa_heads_topk_tree(h, W1, b1, W2, kmax: int, topk_ids, topk_vals, tree: Tree, root_tok,
                           prefix_len, cand_ids, pos_ids, anc_mask, retrieve, logits=None,
                           ws=None, dev_status=None, stream=None) -> None:
    """medusa_heads_topk, then medusa_tree_build of its lists, in the heads'
    launches."""
    for t, n in ((h, "h"), (W1, "W1"), (b1, "b1"), (W2, "W2"), (topk_ids, "topk_ids"),
                 (topk_vals, "topk_vals")):
        _req(t, n)
    B, d = h.shape
    K, V, _ = W2.shape
    dt = _dt(W2)
    if ws is None:
        ws = _own_workspace(medusa_heads_topk_workspace_size(B, d, V, K, kmax, dt), h.device,
                            stream)
    ct = tree.c()
    _check(lib().medusa_heads_topk_tree(_p(h), _p(W1), _p(b1), _p(W2), dt, B, d, V, K, kmax,
                                        _p(topk_ids), _p(topk_vals), _p(logits), _p(ws),
                                        ws.numel(), ctypes.byref(ct), _p(root_tok),
                                        _p(prefix_len), _p(cand_ids), _p(pos_ids), _p(anc_mask),
                                        _p(retrieve), _p(dev_status), _stream(stream)))


def medusa_tree_build(tree: Tree, root_tok, topk_ids, prefix_len, cand_ids, pos_ids, anc_mask,
                      retrieve, dev_status=None, stream=None) -> None:
    B, K, kmax = topk_ids.shape
    ct = tree.c()
    _check(lib().medusa_tree_build(ctypes.byref(ct), _p(root_tok), _p(topk_ids), K, kmax,
                                   _p(prefix_len), B, _p(cand_ids), _p(pos_ids), _p(anc_mask),
                                   _p(retrieve), _p(dev_status), _stream(stream)))


def medusa_tree_attention_workspace_size(B: int, N: int, Hq: int, Hkv: int, dh: int,
                                         max_prefix: int, dt: int) -> int:
    return int(lib().medusa_tree_attention_workspace_size(B, N, Hq, Hkv, dh, max_prefix, dt))


def medusa_tree_attention(q, k_new, v_new, Kc, Vc, prefix_len, anc_mask, max_prefix: int, out,
                          scale: Optional[float] = None, ws=None, dev_status=None,
                          stream=None) -> None:
    """q [B,N,Hq,dh], k_new/v_new [B,N,Hkv,dh], Kc/Vc [B,Hkv,cap,dh] -> out [B,N,Hq,dh]."""
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (Kc, "Kc"), (Vc, "Vc"),
                 (out, "out")):
        _req(t, n)
    B, N, Hq, dh = q.shape
    Hkv, cap = Kc.shape[1], Kc.shape[2]
    dt = _dt(q)
    if scale is None:
        scale = dh ** -0.5
    if ws is None:
        ws = _own_workspace(medusa_tree_attention_workspace_size(B, N, Hq, Hkv, dh, max_prefix,
                                                                 dt), q.device, stream)
    _check(lib().medusa_tree_attention(_p(q), _p(k_new), _p(v_new), _p(Kc), _p(Vc),
                                       _p(prefix_len), _p(anc_mask), dt, B, N, Hq, Hkv, dh, cap,
                                       max_prefix, float(scale), _p(out), _dt(out), _p(ws),
                                       ws.numel(), _p(dev_status), _stream(stream)))


def medusa_verify_accept_workspace_size(B: int, N: int, V: int) -> int:
    return int(lib().medusa_verify_accept_workspace_size(B, N, V))


def medusa_verify_accept(logits, cand_ids, tree: Tree, accept_len, accepted_nodes,
                         accepted_tokens, bonus, mode: int = MEDUSA_ACCEPT_GREEDY,
                         temperature: float = 1.0, eps: float = 0.09, delta: float = 0.3,
                         ws=None, dev_status=None, stream=None) -> None:
    """logits [B,N,V] -> accept_len [B], accepted_nodes/tokens [B,Dmax+1], bonus [B]."""
    _req(logits, "logits")
    B, N, V = logits.shape
    if ws is None:
        ws = _own_workspace(medusa_verify_accept_workspace_size(B, N, V), logits.device, stream)
    ct = tree.c()
    _check(lib().medusa_verify_accept(_p(logits), _dt(logits), _p(cand_ids), ctypes.byref(ct), B, V,
                                      mode, float(temperature), float(eps), float(delta),
                                      _p(accept_len), _p(accepted_nodes), _p(accepted_tokens),
                                      _p(bonus), _p(ws), ws.numel(), _p(dev_status),
                                      _stream(stream)))


def medusa_kv_compact(Kc, Vc, prefix_len, accepted_nodes, accept_len, compact_src,
                      dev_status=None, stream=None) -> None:
    _req(Kc, "Kc")
    _req(Vc, "Vc")
    B, Hkv, cap, dh = Kc.shape
    max_depth = accepted_nodes.shape[1] - 1
    _check(lib().medusa_kv_compact(_p(Kc), _p(Vc), _dt(Kc), _p(prefix_len), _p(accepted_nodes),
                                   _p(accept_len), B, Hkv, dh, cap, max_depth, _p(compact_src),
                                   _p(dev_status), _stream(stream)))


def medusa_verify_accept_compact(logits, cand_ids, tree: Tree, accept_len, accepted_nodes,
                                 accepted_tokens, bonus, Kc, Vc, prefix_len, compact_src,
                                 mode: int = MEDUSA_ACCEPT_GREEDY, temperature: float = 1.0,
                                 eps: float = 0.09, delta: float = 0.3, ws=None, dev_status=None,
                                 stream=None) -> None:
    """medusa_verify_accept, then medusa_kv_compact of its result, in the
    verification's launches."""
    _req(logits, "logits")
    _req(Kc, "Kc")
    _req(Vc, "Vc")
    B, N, V = logits.shape
    _, Hkv, cap, dh = Kc.shape
    if ws is None:
        ws = _own_workspace(medusa_verify_accept_workspace_size(B, N, V), logits.device, stream)
    ct = tree.c()
    _check(lib().medusa_verify_accept_compact(
        _p(logits), _dt(logits), _p(cand_ids), ctypes.byref(ct), B, V, mode, float(temperature),
        float(eps), float(delta), _p(accept_len), _p(accepted_nodes), _p(accepted_tokens),
        _p(bonus), _p(Kc), _p(Vc), _dt(Kc), _p(prefix_len), Hkv, dh, cap, _p(compact_src),
        _p(ws), ws.numel(), _p(dev_status), _stream(stream)))


def medusa_verify_accept_noalloc(logits, cand_ids, tree: Tree, accept_len, accepted_nodes,
                                 accepted_tokens, bonus, mode: int = MEDUSA_ACCEPT_GREEDY,
                                 temperature: float = 1.0, eps: float = 0.09, delta: float = 0.3,
                                 dev_status=None, stream=None) -> None:
    """medusa_verify_accept without a workspace argument, for callers that
    cannot hand the library device memory per call: the library keeps its
    own fixed 4 MiB scratch on each device.  Calls that overlap on the GPU
    share that scratch and race."""
    _req(logits, "logits")
    B, N, V = logits.shape
    ct = tree.c()
    _check(lib().medusa_verify_accept_noalloc(_p(logits), _dt(logits), _p(cand_ids),
                                              ctypes.byref(ct), B, V, mode, float(temperature),
                                              float(eps), float(delta), _p(accept_len),
                                              _p(accepted_nodes), _p(accepted_tokens), _p(bonus),
                                              _p(dev_status), _stream(stream)))


def medusa_lmhead_verify_workspace_size(B: int, N: int, d: int, V: int) -> int:
    return int(lib().medusa_lmhead_verify_workspace_size(B, N, d, V))


def medusa_lmhead_verify(hidden, lm_head, cand_ids, tree: Tree, accept_len, accepted_nodes,
                         accepted_tokens, bonus, mode: int = MEDUSA_ACCEPT_GREEDY,
                         temperature: float = 1.0, eps: float = 0.09, delta: float = 0.3,
                         logits=None, ws=None, dev_status=None, stream=None) -> None:
    """hidden [B,N,d] bf16, lm_head [V,d] bf16 -> the verify outputs of
    medusa_verify_accept on logits = hidden @ lm_head^T, never materialised
    unless ``logits`` ([B,N,V] fp32) is given."""
    _req(hidden, "hidden")
    _req(lm_head, "lm_head")
    B, N, d = hidden.shape
    V = lm_head.shape[0]
    if ws is None:
        ws = _own_workspace(medusa_lmhead_verify_workspace_size(B, N, d, V), hidden.device, stream)
    ct = tree.c()
    _check(lib().medusa_lmhead_verify(_p(hidden), _p(lm_head), _dt(hidden), _p(cand_ids),
                                      ctypes.byref(ct), B, d, V, mode, float(temperature),
                                      float(eps), float(delta), _p(accept_len),
                                      _p(accepted_nodes), _p(accepted_tokens), _p(bonus),
                                      _p(logits), _p(ws), ws.numel(), _p(dev_status),
                                      _stream(stream)))


def medusa_next_step(node_hidden, accept_len, accepted_nodes, bonus, h_next, root_next,
                     dev_status=None, stream=None) -> None:
    """h_next[b] = node_hidden[b, kept node], root_next[b] = bonus[b]."""
    _req(node_hidden, "node_hidden")
    _req(h_next, "h_next")
    B, N, d = node_hidden.shape
    max_depth = accepted_nodes.shape[1] - 1
    _check(lib().medusa_next_step(_p(node_hidden), _dt(node_hidden), _p(accept_len),
                                  _p(accepted_nodes), _p(bonus), B, N, d, max_depth, _p(h_next),
                                  _p(root_next), _p(dev_status), _stream(stream)))


def medusa_tree_from_accuracies(acc, n_nodes: int, max_depth: int):
    """acc [K, kmax] (array-like, probabilities) -> (parent, depth, rank)
    int32 numpy arrays of the n_nodes-node tree of the most accurate
    combinations, and its expected accept length.  Host only."""
    import numpy as np
    a = np.ascontiguousarray(np.asarray(acc, dtype=np.float32))
    K, kmax = a.shape
    out = [np.zeros(n_nodes, dtype=np.int32) for _ in range(3)]
    e = ctypes.c_double(0.0)
    _check(lib().medusa_tree_from_accuracies(a.ctypes.data, K, kmax, n_nodes, max_depth,
                                             out[0].ctypes.data, out[1].ctypes.data,
                                             out[2].ctypes.data, ctypes.byref(e)))
    return out[0], out[1], out[2], e.value


def medusa_sample_bonus(logits, accept_len, accepted_nodes, bonus, accepted_tokens,
                        temperature: float, seed: int, offset: int = 0, dev_status=None,
                        stream=None) -> None:
    """Redraw the bonus token of each sequence from softmax(logits/T) at the
    kept node (Philox4x32-10, inverse CDF); updates bonus and accepted_tokens."""
    _req(logits, "logits")
    B, N, V = logits.shape
    max_depth = accepted_nodes.shape[1] - 1
    _check(lib().medusa_sample_bonus(_p(logits), _dt(logits), _p(accept_len), _p(accepted_nodes),
                                     B, N, V, max_depth, float(temperature), int(seed),
                                     int(offset), _p(bonus), _p(accepted_tokens), _p(dev_status),
                                     _stream(stream)))


def medusa_topk_merge(vals, ids, rows: int, n_lists: int, list_len: int, row_stride: int,
                      list_stride: int, id_offsets, kmax: int, topk_ids, topk_vals,
                      stream=None) -> None:
    """Best kmax of n_lists candidate lists per row (see include/medusa.h)."""
    _req(vals, "vals")
    _req(ids, "ids")
    _check(lib().medusa_topk_merge(_p(vals), _p(ids), rows, n_lists, list_len, int(row_stride),
                                   int(list_stride), _p(id_offsets), kmax, _p(topk_ids),
                                   _p(topk_vals), _stream(stream)))


def medusa_verify_records_workspace_size(B: int, N: int, V_shard: int) -> int:
    return int(lib().medusa_verify_records_workspace_size(B, N, V_shard))


def medusa_verify_records(logits, cand_ids, tree: Tree, v_offset: int, records, cand_logit,
                          mode: int = MEDUSA_ACCEPT_GREEDY, temperature: float = 1.0, ws=None,
                          dev_status=None, stream=None) -> None:
    """This vocabulary shard's row records ([B*N, 4] float32 view of
    medusa_row_record_t) and candidate logits ([B*N] float32)."""
    _req(logits, "logits")
    B, N, Vs = logits.shape
    if ws is None:
        ws = _own_workspace(medusa_verify_records_workspace_size(B, N, Vs), logits.device, stream)
    ct = tree.c()
    _check(lib().medusa_verify_records(_p(logits), _dt(logits), _p(cand_ids), ctypes.byref(ct), B,
                                       Vs, v_offset, mode, float(temperature), _p(records),
                                       _p(cand_logit), _p(ws), ws.numel(), _p(dev_status),
                                       _stream(stream)))


def medusa_verify_from_records(records, cand_logit, cand_ids, tree: Tree, V: int, accept_len,
                               accepted_nodes, accepted_tokens, bonus,
                               mode: int = MEDUSA_ACCEPT_GREEDY, temperature: float = 1.0,
                               eps: float = 0.09, delta: float = 0.3, dev_status=None,
                               stream=None) -> None:
    """Verification from G shards' records [G, B*N, 4] and the candidate
    logits maximised over the shards [B*N] (typical only)."""
    _req(records, "records")
    G = records.shape[0]
    B = cand_ids.shape[0]
    ct = tree.c()
    _check(lib().medusa_verify_from_records(_p(records), G, _p(cand_logit), _p(cand_ids),
                                            ctypes.byref(ct), B, V, mode, float(temperature),
                                            float(eps), float(delta), _p(accept_len),
                                            _p(accepted_nodes), _p(accepted_tokens), _p(bonus),
                                            _p(dev_status), _stream(stream)))


# ---------------------------------------------------------------------------
# prompt side: rotary positions, paged cache, chunk attention, sampling
# ---------------------------------------------------------------------------


# These calls are short enough for the marshalling to show: on the current
# stream an extension checks the tensors and makes the C call at once.  What it
# does not take (-1), and calls on another stream, go through ctypes below; a
# refusal is told its reason there.

_fast = None


def _marshal():
    """The extension, bound to the library."""
    global _fast
    if _fast is None:
        L = lib()
        path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_marshal.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: run "
                               "`python -m speculative_decoding_medusa_b200.build`")
        loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
        m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
        m.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.medusa_rope, L.medusa_rope_append, L.medusa_chunk_attention,
            L.medusa_sample_tokens)))
        _fast = m
    return _fast


def _dev() -> int:
    """The current device, where a call launches and every tensor must be."""
    return torch.cuda.current_device()


def _raw_stream(stream, dev: int) -> int:
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev)


def _bad_tensor(t, name: str, dev: int, what: str):
    if isinstance(t, torch.Tensor) and t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{name} must be on the current device (cuda:{dev})")
    raise ValueError(f"{name} must be {what}")


def _rows(t: torch.Tensor, name: str, dtype, shape, dev: int):
    """(address, token stride) of a [T, H, dh] tensor whose heads and elements
    are dense (a slice of a packed projection is allowed)."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _bad_tensor(t, name, dev, f"a {dtype} CUDA tensor of shape {tuple(shape)}")
    _, H, dh = shape
    if t.is_contiguous():
        return t.data_ptr(), H * dh
    st = t.stride()
    if (dh > 1 and st[2] != 1) or (H > 1 and st[1] != dh):
        raise ValueError(f"{name}: the heads and elements of a token must be dense")
    return t.data_ptr(), (st[0] if shape[0] > 1 else H * dh)


def _vec(t: Optional[torch.Tensor], name: str, dtype, n: int, dev: int):
    """Address of a dense tensor of n elements (None: NULL)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.numel() != n or t.get_device() != dev or not t.is_contiguous():
        _bad_tensor(t, name, dev, f"a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _3d(t: torch.Tensor, name: str):
    sh = t.shape
    if len(sh) != 3:
        raise ValueError(f"{name} must be a [T, H, dh] CUDA tensor")
    return sh


class _Fixed:
    """The attributes named in _held are set once: the C struct has their
    addresses and sizes, and would not follow a new value."""

    _held = frozenset()

    def __setattr__(self, name, value):
        if name in self._held and name in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed: make a new "
                                 f"{type(self).__name__}")
        object.__setattr__(self, name, value)


class Rope(_Fixed):
    """A rotation of the first ``rot`` elements of each head: the frequencies
    theta^(-2i/rot) under a long-context scaling ("none", "linear", "llama3",
    "yarn"), in pairs (i, i + rot/2), or (2i, 2i + 1) when interleaved.

    ``low_freq_factor`` and ``high_freq_factor`` are full turns over
    ``original_max_position`` (llama3: 1 and 4, yarn: 1 and 32 by default)."""

    _held = frozenset(("rot", "interleaved", "scale", "turns", "_c", "_ref"))

    def __init__(self, rot: int, *, theta: float = 10000.0, interleaved: bool = False,
                 scaling: str = "none", factor: float = 1.0,
                 low_freq_factor: Optional[float] = None,
                 high_freq_factor: Optional[float] = None, original_max_position: int = 8192,
                 device=None):
        import numpy as np
        if scaling not in MEDUSA_ROPE_SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(MEDUSA_ROPE_SCALINGS)}")
        low = 1.0 if low_freq_factor is None else low_freq_factor
        high = (32.0 if scaling == "yarn" else 4.0) if high_freq_factor is None \
            else high_freq_factor
        turns = np.zeros(max(int(rot) // 2, 1), dtype=np.uint64)
        scale = ctypes.c_float(1.0)
        _check(lib().medusa_rope_freqs(rot, theta, MEDUSA_ROPE_SCALINGS[scaling], factor, low, high,
                                       original_max_position, turns.ctypes.data,
                                       ctypes.byref(scale)))
        self.rot, self.interleaved, self.scale = int(rot), bool(interleaved), scale.value
        # full turns per position, in units of 2^-64 (the bits of a uint64)
        self.turns = torch.from_numpy(turns.view(np.int64)).to(device or "cuda")
        self._c = medusa_rope_t(self.rot, int(self.interleaved), self.scale,
                                self.turns.data_ptr())
        self._ref = ctypes.addressof(self._c)


class PagedCache(_Fixed):
    """K and V pools [n_pages, Hkv, page_size, dh] and the page table
    [B, max_pages] int32 of the sequences that use them.  Their contents change
    in place; for other tensors make another PagedCache."""

    _held = frozenset(("K", "V", "table", "dt", "B", "n_pages", "Hkv", "page_size", "dh",
                       "_device", "_c", "_ref"))

    def __init__(self, K: torch.Tensor, V: torch.Tensor, table: torch.Tensor):
        _req(K, "K")
        _req(V, "V")
        _req(table, "table")
        if K.dim() != 4 or V.shape != K.shape or V.dtype is not K.dtype:
            raise ValueError("K and V must be [n_pages, Hkv, page_size, dh] of one dtype")
        if table.dim() != 2 or table.dtype is not torch.int32:
            raise ValueError("table must be [B, max_pages] int32")
        if V.device != K.device or table.device != K.device:
            raise ValueError("K, V and table must be on one device")
        self.K, self.V, self.table = K, V, table
        self._device = K.get_device()
        self.dt = _dt(K)
        self.B = table.shape[0]
        self.n_pages, self.Hkv, self.page_size, self.dh = K.shape
        self._c = medusa_pages_t(K.data_ptr(), V.data_ptr(), table.data_ptr(), self.n_pages,
                                 self.page_size, table.shape[1])
        self._ref = ctypes.addressof(self._c)

    def _on(self, dev: int) -> None:
        if self._device != dev:
            _bad_tensor(self.K, "cache", dev, "on a CUDA device")

    @classmethod
    def dense(cls, Kc: torch.Tensor, Vc: torch.Tensor) -> "PagedCache":
        """The step's dense cache [B, Hkv, cap, dh]: one page of cap slots a sequence."""
        t = torch.arange(Kc.shape[0], dtype=torch.int32, device=Kc.device)
        return cls(Kc, Vc, t.view(-1, 1))


def medusa_rope(rope: Rope, q, k, positions, q_out, k_out, inverse: bool = False,
                stream=None) -> None:
    """q [T,Hq,dh], k [T,Hkv,dh] (or None) rotated at positions [T] int32 into
    q_out, k_out (which may be q and k themselves).  inverse: by the negative
    angle (the gradient of the forward call)."""
    if stream is None:
        st = (_fast or _marshal()).rope(rope._ref, rope.turns, q, k, positions, q_out, k_out,
                                        inverse)
        if st >= 0:
            return _check(st) if st else None
    dev = _dev()
    qsh, dtype = _3d(q, "q"), q.dtype
    T, Hq, dh = qsh
    qp, qs = _rows(q, "q", dtype, qsh, dev)
    op, os_ = _rows(q_out, "q_out", dtype, qsh, dev)
    kp = kop = None
    ks = kos = Hkv = 0
    if k is not None:
        ksh = _3d(k, "k")
        Hkv = ksh[1]
        if ksh[0] != T or ksh[2] != dh:
            raise ValueError("k must have q's tokens and head size")
        kp, ks = _rows(k, "k", dtype, ksh, dev)
        kop, kos = _rows(k_out, "k_out", dtype, ksh, dev)
    pp = _vec(positions, "positions", torch.int32, T, dev)
    if rope.turns.get_device() != dev:
        _bad_tensor(rope.turns, "rope", dev, "on a CUDA device")
    st = lib().medusa_rope(rope._ref, qp, qs, kp, ks, _dt(q), pp, T, Hq, Hkv, dh,
                           1 if inverse else 0, op, os_, kop, kos, _raw_stream(stream, dev))
    if st:
        _check(st)


def medusa_rope_append(rope: Optional[Rope], q, k, v, cu_q, kv_len, q_out, cache: PagedCache,
                       positions=None, dev_status=None, stream=None) -> None:
    """The new tokens q [T,Hq,dh] (or None), k, v [T,Hkv,dh] of cache.B
    sequences: q rotated into q_out, k rotated and v copied into the cache at
    slots kv_len[b] - (cu_q[b+1] - cu_q[b]) .. kv_len[b] - 1."""
    if stream is None:
        ref, turns = (rope._ref, rope.turns) if rope is not None else (None, None)
        st = (_fast or _marshal()).append(ref, turns, q, k, v, cu_q, kv_len, q_out, cache._ref,
                                          cache.K, cache.B, positions, dev_status)
        if st >= 0:
            return _check(st) if st else None
    dev = _dev()
    ksh, dtype = _3d(k, "k"), cache.K.dtype
    T, Hkv, dh = ksh
    if Hkv != cache.Hkv or dh != cache.dh:
        raise ValueError("k must have the cache's heads and head size")
    kp, ks = _rows(k, "k", dtype, ksh, dev)
    vp, vs = _rows(v, "v", dtype, ksh, dev)
    qp = op = ref = None
    qs = os_ = Hq = 0
    if q is not None:
        qsh = _3d(q, "q")
        Hq = qsh[1]
        if qsh[0] != T or qsh[2] != dh:
            raise ValueError("q must have k's tokens and head size")
        qp, qs = _rows(q, "q", dtype, qsh, dev)
        op, os_ = _rows(q_out, "q_out", dtype, qsh, dev)
    if rope is not None:
        ref = rope._ref
        if rope.turns.get_device() != dev:
            _bad_tensor(rope.turns, "rope", dev, "on a CUDA device")
    i32, B = torch.int32, cache.B
    cup = _vec(cu_q, "cu_q", i32, B + 1, dev)
    kvp = _vec(kv_len, "kv_len", i32, B, dev)
    pp = _vec(positions, "positions", i32, T, dev)
    cache._on(dev)
    st = lib().medusa_rope_append(ref, qp, qs, kp, ks, vp, vs, cache.dt, pp, cup, kvp, B, T, Hq,
                                  Hkv, dh, op, os_, cache._ref,
                                  _vec(dev_status, "dev_status", i32, 1, dev),
                                  _raw_stream(stream, dev))
    if st:
        _check(st)


def medusa_chunk_attention_workspace_size(Hq: int, Hkv: int, dh: int, dt: int) -> int:
    return int(lib().medusa_chunk_attention_workspace_size(Hq, Hkv, dh, dt))


def medusa_chunk_attention(q, cache: PagedCache, cu_q, kv_len, out,
                           scale: Optional[float] = None, ws=None, dev_status=None,
                           stream=None) -> None:
    """q [T,Hq,dh] of cache.B sequences' new tokens (their k and v already in
    the cache) -> out [T,Hq,dh], each token over its sequence's slots up to its
    own."""
    if stream is None and ws is not None:
        st = (_fast or _marshal()).attention(q, cache._ref, cache.K, cu_q, kv_len, out, cache.B,
                                             cache.dh ** -0.5 if scale is None else scale, ws,
                                             dev_status)
        if st >= 0:
            return _check(st) if st else None
    dev = _dev()
    qsh, dtype = _3d(q, "q"), cache.K.dtype
    T, Hq, dh = qsh
    if dh != cache.dh:
        raise ValueError("q must have the cache's head size")
    qp, qs = _rows(q, "q", dtype, qsh, dev)
    op, os_ = _rows(out, "out", dtype, qsh, dev)
    if os_ != Hq * dh:
        raise ValueError("out must be dense")
    i32, B = torch.int32, cache.B
    cup = _vec(cu_q, "cu_q", i32, B + 1, dev)
    kvp = _vec(kv_len, "kv_len", i32, B, dev)
    cache._on(dev)
    if ws is None:
        ws = _own_workspace(medusa_chunk_attention_workspace_size(Hq, cache.Hkv, dh, cache.dt),
                            cache.K.device, stream)
    nbytes = ws.numel()
    st = lib().medusa_chunk_attention(qp, qs, cache._ref, cache.dt, cup, kvp, B, T, Hq, cache.Hkv,
                                      dh, dh ** -0.5 if scale is None else scale, op,
                                      _vec(ws, "ws", torch.uint8, nbytes, dev), nbytes,
                                      _vec(dev_status, "dev_status", i32, 1, dev),
                                      _raw_stream(stream, dev))
    if st:
        _check(st)


def medusa_sample_tokens(logits, u, tokens, temperature=None, top_k=None, top_p=None, min_p=None,
                         row_idx=None, kept=None, dev_status=None, stream=None) -> None:
    """tokens [R] int32 drawn from logits [n_rows,V] (rows may be strided) with
    uniform numbers u [R]; temperature, top_p, min_p [R] fp32 and top_k [R]
    int32 are off when None; row_idx [R] picks each draw's row."""
    if stream is None:
        st = (_fast or _marshal()).sample(logits, u, tokens, temperature, top_k, top_p, min_p,
                                          row_idx, kept, dev_status)
        if st >= 0:
            return _check(st) if st else None
    dev = _dev()
    sh = logits.shape
    if len(sh) != 2 or logits.get_device() != dev or (sh[1] > 1 and logits.stride(1) != 1):
        _bad_tensor(logits, "logits", dev, "an [n_rows, V] CUDA tensor with dense rows")
    n, V = sh
    R = u.numel()
    f32, i32 = torch.float32, torch.int32
    st = lib().medusa_sample_tokens(
        logits.data_ptr(), _dt(logits), logits.stride(0) if n > 1 else V, n,
        _vec(row_idx, "row_idx", i32, R, dev), R, V, _vec(u, "u", f32, R, dev),
        _vec(temperature, "temperature", f32, R, dev), _vec(top_k, "top_k", i32, R, dev),
        _vec(top_p, "top_p", f32, R, dev), _vec(min_p, "min_p", f32, R, dev),
        _vec(tokens, "tokens", i32, R, dev), _vec(kept, "kept", i32, R, dev),
        _vec(dev_status, "dev_status", i32, 1, dev), _raw_stream(stream, dev))
    if st:
        _check(st)


def medusa_wait_flag(flag, value: int, budget_cycles: int, dev_status, stream=None) -> None:
    """Run the library's bounded flag wait on ``flag`` (device int32): returns
    once *flag == value, or writes MEDUSA_ERR_TIMEOUT into dev_status after
    budget_cycles SM clock cycles (<= 0: the library's own bound)."""
    _req(flag, "flag")
    _check(lib().medusa_wait_flag(_p(flag), int(value), int(budget_cycles), _p(dev_status),
                                  _stream(stream)))
