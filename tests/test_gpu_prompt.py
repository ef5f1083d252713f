"""GPU: the prompt side run together, and handed to the decode step: prompts in
ragged chunks through PromptPass, root tokens drawn, then a decode-verify step
that rotates its tree, on the cache the prompts filled."""
import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from oracle import medusa_oracle as O
from oracle import prompt_oracle as P
from speculative_decoding_medusa_b200 import workloads as W
from speculative_decoding_medusa_b200.step import DecodeVerifyStep, PromptPass
from tests.helpers import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


def _feed(pp, chunks, q, k, v):
    """Run the chunks ([n_b] new tokens each) and collect every token's output."""
    B = len(q)
    done = [0] * B
    out = [[] for _ in range(B)]
    for new in chunks:
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        rows = [torch.cat([x[b][done[b]:done[b] + new[b]] for b in range(B)]).to(DEV)
                for x in (q, k, v)]
        done = [d + n for d, n in zip(done, new)]
        got = pp.run(*rows, torch.tensor(cu, **I32), torch.tensor(done, **I32))
        for b in range(B):
            out[b].append(got[cu[b]:cu[b + 1]].clone())
    torch.cuda.synchronize()
    assert int(pp.status.item()) == 0
    return [torch.cat(o) for o in out], done


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("paged", [False, True])
def test_prompt_then_decode_step(dtype, paged):
    B, Hq, Hkv, dh, cap = 3, 4, 2, 64, 200
    lens = [60, 131, 17]
    chunks = [[20, 100, 0], [39, 1, 16], [1, 30, 1]]
    g = torch.Generator().manual_seed(4)
    q = [torch.randn(n, Hq, dh, generator=g).to(dtype) for n in lens]
    k = [torch.randn(n, Hkv, dh, generator=g).to(dtype) for n in lens]
    v = [torch.randn(n, Hkv, dh, generator=g).to(dtype) for n in lens]
    rope = M.Rope(32, theta=10000.0, scaling="llama3", factor=8.0, original_max_position=64)
    f, s = P.rope_freqs(32, 10000.0, "llama3", 8.0, 1.0, 4.0, 64.0)
    Kc, Vc = torch.zeros(2, B, Hkv, cap, dh, dtype=dtype, device=DEV)
    if paged:
        pool = torch.zeros(2, 20, Hkv, 16, dh, dtype=dtype, device=DEV)
        ids = torch.randperm(20, generator=g).to(torch.int32)
        table = torch.full((3, 9), -1, dtype=torch.int32)
        table[0, :4], table[1], table[2, :2] = ids[:4], ids[4:13], ids[13:15]
        cache = M.PagedCache(pool[0], pool[1], table.to(DEV))
    else:
        cache = M.PagedCache.dense(Kc, Vc)
    pp = PromptPass(cache=cache, Hq=Hq, max_tokens=160, rope=rope)
    out, done = _feed(pp, chunks, q, k, v)
    assert done == lens
    # every token's output, from the definition on the unrotated inputs
    half = torch.finfo(dtype).eps / 2
    for b, n in enumerate(lens):
        pos = np.arange(n)
        qr, kr = P.rope(f64(q[b]), pos, f, s), P.rope(f64(k[b]), pos, f, s)
        K1, V1 = kr.transpose(1, 0, 2)[None], f64(v[b]).transpose(1, 0, 2)[None]
        ref, absv, mag, cnt = P.chunk_attention(qr, K1, V1, np.array([[0]]), [0, n], [n], dh ** -0.5)
        # the kernels' q and k are rounded to the type once (scores move by up to
        # 2 half steps of sum |q k|), then the chunk attention's own bound
        ds = mag * (2 * half * 1.01 + (dh + 2 + 40) * 2.0 ** -23)
        rel = np.expm1(2 * ds) + 2.0 ** -20 + cnt * 2.0 ** -23 + (half if dtype is torch.bfloat16 else 0)
        bound = rel[..., None] * absv
        bound = bound + half * (np.abs(ref) + bound)
        assert (np.abs(f64(out[b]) - ref) <= bound).all()
    # root tokens from the last tokens' logits, each with its own settings
    V = 1000
    logits = torch.randn(7, V, generator=g).to(dtype).to(DEV)
    rows, u, T = [6, 0, 3], [0.2, 0.7, 0.95], [1.0, 0.0, 0.6]
    root = pp.roots(logits, torch.tensor(u, device=DEV), torch.tensor(T, device=DEV),
                    top_p=torch.tensor([0.9, 1.0, 0.5], device=DEV),
                    row_idx=torch.tensor(rows, **I32))
    want = [P.sample_row(f64(logits)[r], float(np.float32(x)), float(np.float32(t)), 0,
                         float(np.float32(tp)))
            for r, x, t, tp in zip(rows, u, T, [0.9, 1.0, 0.5])]
    assert min(w[2] for w in want) > 1e-9
    assert root.tolist() == [w[0] for w in want] and pp.kept.tolist() == [w[1] for w in want]
    if paged:
        return
    # the decode step on the same cache, its tree rotated at pos_ids
    w = W.scaled(W.WORKLOADS["tiny" if dtype is torch.float32 else "llama3_8b"], B=B, d=128, V=V)
    spec = W.tree_for(w)
    N = spec.n_nodes
    hin = W.heads_inputs(w, seed=3)
    step = DecodeVerifyStep(B=B, d=w.d, V=w.V, K=w.K, kmax=w.kmax, tree=M.Tree.from_spec(spec, DEV),
                            Hq=Hq, Hkv=Hkv, dh=dh, cap=cap, max_prefix=max(lens), dtype=dtype,
                            attn_out_dtype=torch.float32, rope=rope, device=DEV)
    tq = torch.randn(B, N, Hq, dh, generator=g).to(dtype)
    tk, tv = (torch.randn(2, B, N, Hkv, dh, generator=g)).to(dtype)
    prefix = torch.tensor(lens, **I32)
    gd = {n: x.to(DEV) for n, x in hin.items()}
    vl = torch.randn(B, N, w.V, generator=g).to(dtype).to(DEV)
    K0, V0 = f64(Kc), f64(Vc)
    step.run(gd["h"], gd["W1"], gd["b1"], gd["W2"], root, tq.to(DEV), tk.to(DEV), tv.to(DEV), Kc,
             Vc, prefix, vl)
    torch.cuda.synchronize()
    assert int(step.status.item()) == 0
    pos = step.pos_ids.cpu().numpy().reshape(-1)
    assert (step.cand_ids[:, 0] == root).all()
    qr = torch.from_numpy(P.rope(f64(tq).reshape(-1, Hq, dh), pos, f, s)).to(dtype)
    kr = torch.from_numpy(P.rope(f64(tk).reshape(-1, Hkv, dh), pos, f, s)).to(dtype)
    ref = O.tree_attention(f64(qr).reshape(B, N, Hq, dh), f64(kr).reshape(B, N, Hkv, dh),
                                 f64(tv), K0, V0, np.array(lens),
                                 step.anc_mask.cpu().numpy().view(np.uint32), dh ** -0.5)["out"]
    # the rounded rotations may differ by a step of the type where the fp32 and
    # fp64 values straddle a border: rare, so the whole is held to a few half
    # steps in norm
    err = np.linalg.norm(f64(step.attn_out) - ref) / np.linalg.norm(ref)
    assert err < 4 * half + 1e-3


def test_captured_prompt_chunk_follows_its_lengths():
    """One graph of a chunk step replayed at growing kv_len (device values):
    the same bits as separate calls."""
    B, Hq, Hkv, dh, n = 2, 8, 2, 128, 24
    g = torch.Generator().manual_seed(9)
    q = torch.randn(4, B * n, Hq, dh, generator=g).bfloat16().to(DEV)
    k, v = torch.randn(2, 4, B * n, Hkv, dh, generator=g).bfloat16().to(DEV)
    rope = M.Rope(128, theta=500000.0, interleaved=True)
    cu = torch.tensor([0, n, 2 * n], **I32)
    res = []
    for captured in (False, True):
        Kc, Vc = torch.zeros(2, B, Hkv, 128, dh, device=DEV).bfloat16()
        pp = PromptPass(cache=M.PagedCache.dense(Kc, Vc), Hq=Hq, max_tokens=B * n, rope=rope)
        kv = torch.tensor([0, 3], **I32)
        bq, bk, bv = q[0].clone(), k[0].clone(), v[0].clone()
        graph = None
        outs = []
        if captured:
            kv.fill_(n)
            pp.run(bq, bk, bv, cu, kv)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                pp.run(bq, bk, bv, cu, kv)
            Kc.zero_()
            Vc.zero_()
            kv.copy_(torch.tensor([0, 3], **I32))
        for r in range(4):
            bq.copy_(q[r])
            bk.copy_(k[r])
            bv.copy_(v[r])
            kv += n
            if captured:
                graph.replay()
            else:
                pp.run(bq, bk, bv, cu, kv)
            outs.append(pp.attn_out.clone())
        torch.cuda.synchronize()
        assert int(pp.status.item()) == 0
        res.append((outs, Kc.clone(), Vc.clone()))
    for a, b in zip(res[0][0], res[1][0]):
        assert torch.equal(a, b)
    assert torch.equal(res[0][1], res[1][1]) and torch.equal(res[0][2], res[1][2])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_calls_on_a_given_stream_and_on_the_current_one(dtype):
    """The two ways a call is marshalled (the extension on the current stream,
    ctypes on a stream that is given): the same launches, packed slices and
    missing operands included, and the same refusals."""
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(5)
    B, T, Hq, Hkv, dh, page = 2, 7, 4, 2, 64, 8
    packed = torch.randn(T, Hq + 2 * Hkv, dh, generator=g, device=dev).to(dtype)
    q, k, v = packed[:, :Hq], packed[:, Hq:Hq + Hkv], packed[:, Hq + Hkv:]
    i32 = dict(dtype=torch.int32, device=dev)
    cu, kv = torch.tensor([0, 3, 7], **i32), torch.tensor([10, 12], **i32)
    rope = M.Rope(32, theta=1e4)
    logits = torch.randn(B, 100, generator=g, device=dev).to(dtype)
    u = torch.rand(B, generator=g, device=dev)
    got = []
    for stream in (None, torch.cuda.current_stream()):
        K, V = torch.zeros(2, 4, Hkv, page, dh, dtype=dtype, device=dev)
        cache = M.PagedCache(K, V, torch.arange(4, **i32).view(2, 2))
        q_rot, out, k_rot = torch.zeros(2, T, Hq, dh, dtype=dtype, device=dev).unbind() + (
            torch.zeros(T, Hkv, dh, dtype=dtype, device=dev),)
        ws = M.workspace(M.medusa_chunk_attention_workspace_size(Hq, Hkv, dh, cache.dt), dev)
        tok, kept = torch.zeros(2, B, **i32).unbind()
        st = M.new_status()
        M.medusa_rope(rope, q, k, torch.arange(T, **i32), q_rot, k_rot, inverse=True,
                      stream=stream)
        first = q_rot.clone()
        M.medusa_rope_append(None, None, k, v, cu, kv, None, cache, dev_status=st, stream=stream)
        M.medusa_rope_append(rope, q, k, v, cu, kv, q_rot, cache, dev_status=st, stream=stream)
        M.medusa_chunk_attention(q_rot, cache, cu, kv, out, None, ws, st, stream)
        M.medusa_sample_tokens(logits, u, tok, top_p=torch.full((B,), 0.9, device=dev), kept=kept,
                               dev_status=st, stream=stream)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        got.append((first, k_rot, K, V, q_rot, out, tok, kept))
        with pytest.raises(ValueError, match="dtype|CUDA"):
            M.medusa_rope(rope, q, k.double(), torch.arange(T, **i32), q_rot, k_rot, stream=stream)
        with pytest.raises(M.MedusaError, match="overlap"):
            M.medusa_chunk_attention(out, cache, cu, kv, out, None, ws, st, stream)
        with pytest.raises(ValueError, match="2 elements"):
            M.medusa_sample_tokens(logits, u, tok[:1], stream=stream)
    for a, b in zip(*got):
        assert torch.equal(a, b) and a.abs().sum() > 0
