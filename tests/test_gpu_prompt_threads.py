"""GPU: calls of different sizes from several host threads at once."""
import threading

import pytest
import torch

import speculative_decoding_medusa_b200 as M

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
