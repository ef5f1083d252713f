"""Without a GPU: where a call that is given no workspace takes one from."""
import contextlib
import types

import pytest
import torch

import speculative_decoding_medusa_b200 as M
from speculative_decoding_medusa_b200 import _lib


class _Library:
    """Every entry point succeeds and does nothing."""

    def __getattr__(self, name):
        return lambda *a: 4096 if name.endswith("workspace_size") else 0


@pytest.fixture
def pools(monkeypatch):
    """The stream that is current at each workspace's allocation, with CPU
    tensors in the place of the device's."""
    current, seen = ["ambient"], []

    @contextlib.contextmanager
    def stream(s):
        current.append(s)
        yield
        current.pop()

    def workspace(nbytes, device=None):
        seen.append(current[-1])
        return torch.empty(nbytes, dtype=torch.uint8)

    monkeypatch.setattr(_lib, "lib", lambda: _Library())
    monkeypatch.setattr(_lib, "workspace", workspace)
    monkeypatch.setattr(_lib, "_req", lambda t, name: None)
    monkeypatch.setattr(_lib, "_dev", lambda: -1)
    monkeypatch.setattr(_lib, "_stream", lambda s: None)
    monkeypatch.setattr(_lib, "_raw_stream", lambda s, dev: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    return seen


def _calls():
    B, N, V, d, K, kmax, Hq, Hkv, dh, cap = 2, 4, 50, 8, 3, 2, 4, 2, 64, 16
    i = torch.zeros(B + 1, dtype=torch.int32)
    x = torch.zeros(B, d)
    tree = M.Tree([-1, 0, 0, 1], [0, 1, 1, 2], [0, 0, 1, 0], 2, device="cpu")
    z, kc = torch.zeros(B, N, V), torch.zeros(B, Hkv, cap, dh)
    q, k = torch.zeros(B, N, Hq, dh), torch.zeros(B, N, Hkv, dh)
    W1, b1, W2 = torch.zeros(K, d, d), torch.zeros(K, d), torch.zeros(K, V, d)
    rows = torch.zeros(5, Hq, dh)
    return {
        "heads_topk": lambda s: M.medusa_heads_topk(x, W1, b1, W2, kmax, i, x, stream=s),
        "heads_topk_tree": lambda s: M.medusa_heads_topk_tree(x, W1, b1, W2, kmax, i, x, tree, i,
                                                              i, i, i, i, i, stream=s),
        "tree_attention": lambda s: M.medusa_tree_attention(q, k, k, kc, kc, i, i, cap, q,
                                                            stream=s),
        "verify_accept": lambda s: M.medusa_verify_accept(z, i, tree, i, i, i, i, stream=s),
        "verify_accept_compact": lambda s: M.medusa_verify_accept_compact(
            z, i, tree, i, i, i, i, kc, kc, i, i, stream=s),
        "lmhead_verify": lambda s: M.medusa_lmhead_verify(torch.zeros(B, N, d),
                                                          torch.zeros(V, d), i, tree, i, i, i, i,
                                                          stream=s),
        "verify_records": lambda s: M.medusa_verify_records(z, i, tree, 0, i, x, stream=s),
        "chunk_attention": lambda s: M.medusa_chunk_attention(
            rows, M.PagedCache(kc, kc, torch.zeros(B, 1, dtype=torch.int32)), i, i[:B], rows + 1,
            stream=s),
    }


@pytest.mark.parametrize("name", sorted(_calls()))
def test_a_missing_workspace_comes_from_the_calls_stream(pools, name):
    """It is dropped on return, with the kernels still to run: its memory may go
    to a later user of that stream only."""
    _calls()[name](types.SimpleNamespace(cuda_stream="side"))
    assert pools == ["side"]
    if name != "chunk_attention":  # (its calls on the current stream start in the extension)
        _calls()[name](None)
        assert pools == ["side", "ambient"]
