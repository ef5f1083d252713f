"""One decode-verify step through the C ABI: buffers plus three calls in order
(heads + top-k with the tree build, tree attention, verify/accept with the KV
compaction; `DecodeLoop` chains the heads with the tree build, the attention, the
lm_head verification, the compaction and the hand-off to the next step).
`PromptPass` fills the cache before the first step: chunks of the prompts
rotated, written and attended, then the root tokens drawn.
Argument marshalling only; all arithmetic runs in libmedusa_b200.so."""
from __future__ import annotations

from typing import Optional

import torch
from torch.cuda import nvtx

from . import _lib as M


class _TreeRotation:
    """The tree's q and k_new rotated at pos_ids, into buffers of their own
    (nothing without a rotation: q and k_new are then taken as positioned)."""

    def __init__(self, rope: Optional[M.Rope], B: int, N: int, Hq: int, Hkv: int, dh: int,
                 dtype: torch.dtype, device):
        self.rope = rope
        if rope is not None:
            self.q = torch.empty(B * N, Hq, dh, dtype=dtype, device=device)
            self.k = torch.empty(B * N, Hkv, dh, dtype=dtype, device=device)

    def __call__(self, q, k_new, pos_ids, stream=None):
        if self.rope is None:
            return q, k_new
        M.medusa_rope(self.rope, q.view(self.q.shape), k_new.view(self.k.shape), pos_ids.view(-1),
                      self.q, self.k, stream=stream)
        return self.q.view(q.shape), self.k.view(k_new.shape)


class PromptPass:
    """Chunks of B prompts on their way into the cache: the new tokens' k
    rotated and written with their v, their q rotated and attended over the
    cache (chunks of any length, one token included), and, where a prompt
    ends, its root token drawn from the logits of its last token.

    ``cache`` is a PagedCache; PagedCache.dense(Kc, Vc) is the decode step's own
    cache, whose prefix_len is then kv_len.  ``max_tokens`` bounds the rows of a
    call.  Nothing synchronises with the host."""

    def __init__(self, *, cache: M.PagedCache, Hq: int, max_tokens: int,
                 rope: Optional[M.Rope] = None, scale: Optional[float] = None):
        dev, dtype = cache.K.device, cache.K.dtype
        self.cache, self.Hq, self.rope, self.scale = cache, Hq, rope, scale
        i32 = dict(dtype=torch.int32, device=dev)
        self.q_rot = torch.empty(max_tokens, Hq, cache.dh, dtype=dtype, device=dev)
        self.attn_out = torch.empty(max_tokens, Hq, cache.dh, dtype=dtype, device=dev)
        self.root_tok = torch.empty(cache.B, **i32)
        self.kept = torch.empty(cache.B, **i32)
        self.status = torch.zeros(1, **i32)
        self.ws = M.workspace(M.medusa_chunk_attention_workspace_size(
            Hq, cache.Hkv, cache.dh, cache.dt), dev)

    def run(self, q, k, v, cu_q, kv_len, positions=None, stream=None) -> torch.Tensor:
        """q [T,Hq,dh], k, v [T,Hkv,dh]: the chunk's rows (unrotated), sequence b's
        at cu_q[b]..cu_q[b+1]; kv_len [B] counts them.  Returns attn_out[:T]."""
        T = q.shape[0]
        if T > self.attn_out.shape[0]:
            raise ValueError("more rows than max_tokens")
        out = self.attn_out[:T]
        with nvtx.range("medusa_rope_append"):
            if self.rope is None:
                M.medusa_rope_append(None, None, k, v, cu_q, kv_len, None, self.cache,
                                     dev_status=self.status, stream=stream)
            else:
                M.medusa_rope_append(self.rope, q, k, v, cu_q, kv_len, self.q_rot[:T], self.cache,
                                     positions, self.status, stream)
                q = self.q_rot[:T]
        with nvtx.range("medusa_chunk_attention"):
            M.medusa_chunk_attention(q, self.cache, cu_q, kv_len, out, self.scale, self.ws,
                                     self.status, stream)
        return out

    def roots(self, logits, u, temperature=None, top_k=None, top_p=None, min_p=None, row_idx=None,
              stream=None) -> torch.Tensor:
        """Root tokens [B] drawn from logits (row b, or row_idx[b])."""
        with nvtx.range("medusa_sample_tokens"):
            M.medusa_sample_tokens(logits, u, self.root_tok, temperature, top_k, top_p, min_p,
                                   row_idx, self.kept, self.status, stream)
        return self.root_tok


class DecodeVerifyStep:
    def __init__(self, *, B: int, d: int, V: int, K: int, kmax: int, tree: M.Tree, Hq: int,
                 Hkv: int, dh: int, cap: int, max_prefix: int, dtype: torch.dtype,
                 accept: str = "greedy", temperature: float = 1.0, eps: float = 0.09,
                 delta: float = 0.3, head_logits: bool = False,
                 attn_out_dtype: Optional[torch.dtype] = None, rope: Optional[M.Rope] = None,
                 device="cuda"):
        self.B, self.d, self.V, self.K, self.kmax = B, d, V, K, kmax
        self.tree, self.Hq, self.Hkv, self.dh, self.cap = tree, Hq, Hkv, dh, cap
        self.max_prefix = max_prefix
        self.mode = M.MEDUSA_ACCEPT_TYPICAL if accept == "typical" else M.MEDUSA_ACCEPT_GREEDY
        self.temperature, self.eps, self.delta = temperature, eps, delta
        dt = M.MEDUSA_BF16 if dtype == torch.bfloat16 else M.MEDUSA_F32
        N, W = tree.n_nodes, tree.max_depth + 1
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_ids = torch.empty(B, K, kmax, **i32)
        self.topk_vals = torch.empty(B, K, kmax, dtype=torch.float32, device=device)
        self.head_logits = (torch.empty(B, K, V, dtype=torch.float32, device=device)
                            if head_logits else None)
        self.cand_ids = torch.empty(B, N, **i32)
        self.pos_ids = torch.empty(B, N, **i32)
        self.anc_mask = torch.empty(N, (N + 31) // 32, **i32)
        self.retrieve = torch.empty(tree.n_leaves, W, **i32)
        self.attn_out = torch.empty(B, N, Hq, dh, dtype=attn_out_dtype or dtype, device=device)
        self.accept_len = torch.empty(B, **i32)
        self.accepted_nodes = torch.empty(B, W, **i32)
        self.accepted_tokens = torch.empty(B, W, **i32)
        self.bonus = torch.empty(B, **i32)
        self.compact_src = torch.empty(B, W, **i32)
        self.status = torch.zeros(1, **i32)
        self.rotation = _TreeRotation(rope, B, N, Hq, Hkv, dh, dtype, device)
        self.ws_heads = M.workspace(M.medusa_heads_topk_workspace_size(B, d, V, K, kmax, dt), device)
        self.ws_attn = M.workspace(M.medusa_tree_attention_workspace_size(
            B, N, Hq, Hkv, dh, max_prefix, dt), device)
        self.ws_verify = M.workspace(M.medusa_verify_accept_workspace_size(B, N, V), device)

    def run(self, h, W1, b1, W2, root_tok, q, k_new, v_new, Kc, Vc, prefix_len, verify_logits,
            stream=None) -> None:
        """Enqueue one step on ``stream``.  Kc/Vc/prefix_len are updated in place
        (tree K/V written, then the kept branch compacted, prefix advanced).
        With a rotation q and k_new come unrotated.  Each call sits in an NVTX
        range of its name (for ncu --nvtx filters)."""
        with nvtx.range("medusa_heads_topk_tree"):
            M.medusa_heads_topk_tree(h, W1, b1, W2, self.kmax, self.topk_ids, self.topk_vals,
                                     self.tree, root_tok, prefix_len, self.cand_ids, self.pos_ids,
                                     self.anc_mask, self.retrieve, self.head_logits,
                                     self.ws_heads, self.status, stream)
        if self.rotation.rope is not None:
            with nvtx.range("medusa_rope"):
                q, k_new = self.rotation(q, k_new, self.pos_ids, stream)
        with nvtx.range("medusa_tree_attention"):
            M.medusa_tree_attention(q, k_new, v_new, Kc, Vc, prefix_len, self.anc_mask,
                                    self.max_prefix, self.attn_out, None, self.ws_attn,
                                    self.status, stream)
        with nvtx.range("medusa_verify_accept_compact"):
            M.medusa_verify_accept_compact(verify_logits, self.cand_ids, self.tree,
                                           self.accept_len, self.accepted_nodes,
                                           self.accepted_tokens, self.bonus, Kc, Vc, prefix_len,
                                           self.compact_src, self.mode, self.temperature,
                                           self.eps, self.delta, self.ws_verify, self.status,
                                           stream)


class DecodeLoop:
    """Decode steps chained on the device (greedy or typical acceptance with
    the verification taken from the tree nodes' hidden states):

        heads + top-k (h) -> tree build (root) -> base model (external; gives
        the nodes' hidden states and tree Q/K/V) -> tree attention ->
        lm_head verify -> KV compaction -> next step (h := kept node's hidden
        state, root := bonus token)

    ``step`` enqueues one step and records its accept_len in ``history``;
    nothing synchronises with the host, so a run of steps can be captured in
    one CUDA graph."""

    def __init__(self, *, B: int, d: int, V: int, K: int, kmax: int, tree: M.Tree, Hq: int,
                 Hkv: int, dh: int, cap: int, max_prefix: int, steps: int,
                 accept: str = "greedy", temperature: float = 1.0, eps: float = 0.09,
                 delta: float = 0.3, rope: Optional[M.Rope] = None, device="cuda"):
        self.B, self.d, self.V, self.K, self.kmax = B, d, V, K, kmax
        self.tree, self.Hq, self.Hkv, self.dh = tree, Hq, Hkv, dh
        self.max_prefix = max_prefix
        self.mode = M.MEDUSA_ACCEPT_TYPICAL if accept == "typical" else M.MEDUSA_ACCEPT_GREEDY
        self.temperature, self.eps, self.delta = temperature, eps, delta
        N, W = tree.n_nodes, tree.max_depth + 1
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_ids = torch.empty(B, K, kmax, **i32)
        self.topk_vals = torch.empty(B, K, kmax, dtype=torch.float32, device=device)
        self.cand_ids = torch.empty(B, N, **i32)
        self.pos_ids = torch.empty(B, N, **i32)
        self.anc_mask = torch.empty(N, (N + 31) // 32, **i32)
        self.retrieve = torch.empty(tree.n_leaves, W, **i32)
        self.attn_out = torch.empty(B, N, Hq, dh, dtype=torch.bfloat16, device=device)
        self.accept_len = torch.empty(B, **i32)
        self.accepted_nodes = torch.empty(B, W, **i32)
        self.accepted_tokens = torch.empty(B, W, **i32)
        self.bonus = torch.empty(B, **i32)
        self.compact_src = torch.empty(B, W, **i32)
        self.history = torch.zeros(steps, B, **i32)
        self.tokens = torch.zeros(steps, B, W, **i32)
        self.status = torch.zeros(1, **i32)
        self.rotation = _TreeRotation(rope, B, N, Hq, Hkv, dh, torch.bfloat16, device)
        bf = M.MEDUSA_BF16
        self.ws_heads = M.workspace(M.medusa_heads_topk_workspace_size(B, d, V, K, kmax, bf), device)
        self.ws_attn = M.workspace(M.medusa_tree_attention_workspace_size(
            B, N, Hq, Hkv, dh, max_prefix, bf), device)
        self.ws_lm = M.workspace(M.medusa_lmhead_verify_workspace_size(B, N, d, V), device)

    def step(self, r: int, h, root, W1, b1, W2, lm_head, base_model, q, k_new, v_new, Kc, Vc,
             prefix_len, stream=None) -> None:
        """Enqueue step ``r``.  h [B, d] bf16 and root [B] int32 are replaced
        by the next step's; Kc/Vc/prefix_len advance by the kept branch.  With a
        rotation q and k_new come unrotated."""
        M.medusa_heads_topk_tree(h, W1, b1, W2, self.kmax, self.topk_ids, self.topk_vals,
                                 self.tree, root, prefix_len, self.cand_ids, self.pos_ids,
                                 self.anc_mask, self.retrieve, None, self.ws_heads, self.status,
                                 stream)
        node_hidden = base_model.forward(self.cand_ids, r)
        q, k_new = self.rotation(q, k_new, self.pos_ids, stream)
        M.medusa_tree_attention(q, k_new, v_new, Kc, Vc, prefix_len, self.anc_mask,
                                self.max_prefix, self.attn_out, None, self.ws_attn, self.status,
                                stream)
        M.medusa_lmhead_verify(node_hidden, lm_head, self.cand_ids, self.tree, self.accept_len,
                               self.accepted_nodes, self.accepted_tokens, self.bonus, self.mode,
                               self.temperature, self.eps, self.delta, None, self.ws_lm,
                               self.status, stream)
        M.medusa_kv_compact(Kc, Vc, prefix_len, self.accepted_nodes, self.accept_len,
                            self.compact_src, self.status, stream)
        M.medusa_next_step(node_hidden, self.accept_len, self.accepted_nodes, self.bonus, h, root,
                           self.status, stream)
        self.history[r].copy_(self.accept_len)
        self.tokens[r].copy_(self.accepted_tokens)
