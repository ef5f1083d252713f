"""GPU: the prompt side's calls on streams of their own."""
import pytest
import torch

import speculative_decoding_medusa_b200 as M

pytestmark = pytest.mark.gpu

DEV = "cuda"


def test_a_missing_workspace_outlives_its_call_on_another_stream():
    """Two chunk attentions without a workspace queue behind work on streams of
    their own, their ranges split over blocks; what the current stream is given
    and writes meanwhile is none of theirs."""
    Hq, Hkv, dh, page, n = 8, 2, 128, 64, 80
    g = torch.Generator(device=DEV).manual_seed(4)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    K, V = torch.randn(2, n, Hkv, page, dh, generator=g, **bf)
    cache = M.PagedCache(K, V, torch.arange(n, dtype=torch.int32, device=DEV).view(1, n))
    cu = torch.tensor([0, 40], dtype=torch.int32, device=DEV)
    kv = torch.tensor([n * page - 3], dtype=torch.int32, device=DEV)
    qs = [torch.randn(40, Hq, dh, generator=g, **bf) for _ in range(2)]
    nbytes = M.medusa_chunk_attention_workspace_size(Hq, Hkv, dh, M.MEDUSA_BF16)
    ws = M.workspace(nbytes)
    want = [torch.empty_like(q) for q in qs]
    for q, o in zip(qs, want):
        M.medusa_chunk_attention(q, cache, cu, kv, o, ws=ws)
    outs = [torch.zeros_like(q) for q in qs]
    sides = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    # every pool filled and every kernel loaded first, which can wait for the GPU
    for s, q, o in zip(sides, qs, outs):
        M.medusa_chunk_attention(q, cache, cu, kv, o, stream=s)
    taken = [M.workspace(nbytes).fill_(255) for _ in range(4)]
    torch.cuda.synchronize()
    del ws, taken  # free for this stream's next allocations of their size
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for s, q, o in zip(sides, qs, outs):
        with torch.cuda.stream(s):
            torch.cuda._sleep(400_000_000)  # some 200 ms
        M.medusa_chunk_attention(q, cache, cu, kv, o, stream=s)
    taken = [M.workspace(nbytes).fill_(255) for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    assert not sides[0].query()  # its call was still to come
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)
    for t in taken:
        assert bool((t == 255).all())


def test_calls_without_work_between_calls_that_share_a_workspace():
    """A call whose blocks have nothing to do (no new token, or lengths that are
    refused) ends at once; its counters are zeroed before the next call counts."""
    g = torch.Generator(device=DEV).manual_seed(9)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    K, V = torch.randn(2, 40, 2, 64, 128, generator=g, **bf)
    cache = M.PagedCache(K, V, torch.arange(40, **i32).view(1, 40))
    q = torch.randn(9, 8, 128, generator=g, **bf)
    cu, kv = torch.tensor([0, 9], **i32), torch.tensor([2500], **i32)
    none, wrong = torch.tensor([0, 0], **i32), torch.tensor([0, 10], **i32)
    ws = M.workspace(M.medusa_chunk_attention_workspace_size(8, 2, 128, M.MEDUSA_BF16))
    first, st = torch.empty_like(q), M.new_status()
    M.medusa_chunk_attention(q, cache, cu, kv, first, ws=ws)

    def run(out):
        M.medusa_chunk_attention(q, cache, none, kv, out, ws=ws)
        M.medusa_chunk_attention(q, cache, cu, kv, out, ws=ws)
        M.medusa_chunk_attention(q, cache, wrong, kv, out, ws=ws, dev_status=st)

    outs = [torch.zeros_like(q) for _ in range(200)]
    for o in outs:
        run(o)
    graph = torch.cuda.CUDAGraph()
    late = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        run(late)
    for _ in range(50):
        late.zero_()
        graph.replay()
        outs.append(late.clone())
    torch.cuda.synchronize()
    assert int(st.item()) == 6
    for o in outs:
        assert torch.equal(o, first)
