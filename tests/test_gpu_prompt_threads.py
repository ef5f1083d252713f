"""GPU: calls of different sizes from several host threads at once."""
import ctypes
import threading
import time

import pytest
import torch

import speculative_decoding_medusa_b200 as M
from speculative_decoding_medusa_b200 import _lib

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _together(works, turns):
    """Each work turns times in a thread of its own; the errors."""
    errors = []
    start = threading.Barrier(len(works))

    def body(work):
        try:
            torch.cuda.synchronize()  # the device's context, in this thread too
            start.wait()
            for _ in range(turns):
                work()
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))

    threads = [threading.Thread(target=body, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_vocabularies_of_different_sizes(dtype):
    """The shared memory that a draw needs follows its vocabulary: a short one
    must not lower what the kernel is allowed between another thread's
    preparation and its launch."""
    works, checks = [], []
    for V in (300000, 50, 300000, 9000):
        g = torch.Generator(device=DEV).manual_seed(V)
        z = torch.randn(1, V, generator=g, device=DEV).to(dtype)
        u = torch.full((1,), 0.5, device=DEV)
        p = torch.full((1,), 0.9, device=DEV)
        tok, first = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
        M.medusa_sample_tokens(z, u, first, top_p=p)
        s = torch.cuda.Stream()
        works.append(lambda z=z, u=u, p=p, tok=tok, s=s: M.medusa_sample_tokens(
            z, u, tok, top_p=p, stream=s))
        checks.append((tok, first))
    torch.cuda.synchronize()
    assert _together(works, 2000) == []
    for tok, first in checks:
        assert torch.equal(tok, first)


def test_heads_of_different_batches():
    """The same of the heads, whose running lists follow the batch."""
    d, V, K, kmax = 64, 2000, 4, 4
    works, checks = [], []
    g = torch.Generator(device=DEV).manual_seed(3)
    W1 = (torch.randn(K, d, d, generator=g, device=DEV) / 8).bfloat16()
    b1 = torch.randn(K, d, generator=g, device=DEV).bfloat16()
    W2 = torch.randn(K, V, d, generator=g, device=DEV).bfloat16()
    for B in (8, 1, 8, 2):
        h = torch.randn(B, d, generator=g, device=DEV).bfloat16()
        ids, first = torch.zeros(2, B, K, kmax, dtype=torch.int32, device=DEV)
        vals = torch.zeros(B, K, kmax, device=DEV)
        ws = M.workspace(M.medusa_heads_topk_workspace_size(B, d, V, K, kmax, M.MEDUSA_BF16))
        M.medusa_heads_topk(h, W1, b1, W2, kmax, first, vals, ws=ws)
        s = torch.cuda.Stream()
        works.append(lambda h=h, ids=ids, vals=vals, ws=ws, s=s: M.medusa_heads_topk(
            h, W1, b1, W2, kmax, ids, vals, ws=ws, stream=s))
        checks.append((ids, first))
    torch.cuda.synchronize()
    assert _together(works, 1000) == []
    for ids, first in checks:
        assert torch.equal(ids, first)


def test_the_first_call_of_a_thread():
    """A host thread that has made no CUDA call yet."""
    g = torch.Generator(device=DEV).manual_seed(6)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    K, V = torch.randn(2, 3, 2, 64, 128, generator=g, **bf)
    cache = M.PagedCache(K, V, torch.arange(3, dtype=torch.int32, device=DEV).view(1, 3))
    cu = torch.tensor([0, 5], dtype=torch.int32, device=DEV)
    kv = torch.tensor([150], dtype=torch.int32, device=DEV)
    q = torch.randn(5, 4, 128, generator=g, **bf)
    out, first = torch.zeros(2, 5, 4, 128, **bf)
    ws = M.workspace(M.medusa_chunk_attention_workspace_size(4, 2, 128, M.MEDUSA_BF16))
    M.medusa_chunk_attention(q, cache, cu, kv, first, ws=ws)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    errors = []

    def body():
        try:
            M.medusa_chunk_attention(q, cache, cu, kv, out, ws=ws, stream=s)
        except Exception as e:  # noqa: BLE001
            errors.append(repr(e))

    t = threading.Thread(target=body)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert errors == []
    assert torch.equal(out, first)


def test_other_threads_run_during_a_call():
    """The extension's C call with the library's functions replaced by one that
    sleeps (its first argument, the address of the rotation, as microseconds):
    another thread counts meanwhile."""
    m, L = _lib._marshal(), M.lib()
    q = torch.zeros(4, 2, 64, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    own = [ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.medusa_rope, L.medusa_rope_append, L.medusa_chunk_attention, L.medusa_sample_tokens)]
    sleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    count, stop = [0], threading.Event()

    def body():
        while not stop.is_set():
            count[0] += 1
            time.sleep(0.001)

    t = threading.Thread(target=body)
    t.start()
    try:
        m.bind(sleep, *own[1:])
        before = count[0]
        assert m.rope(300000, q, q, None, pos, q, None, False) == 0
        during = count[0] - before
    finally:
        m.bind(*own)
        stop.set()
        t.join()
    assert during > 20
