"""Without a GPU: extreme arguments of the prompt side's C calls, each in a
process of its own, which it may not end."""
import os
import subprocess
import sys

import pytest
import torch

import speculative_decoding_medusa_b200 as M
from speculative_decoding_medusa_b200 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALL = """
import ctypes, sys
import speculative_decoding_medusa_b200 as M
from speculative_decoding_medusa_b200 import _lib
p = _lib.medusa_pages_t(4096, 4096, 4096, {n}, {page}, 8)
# the addresses are never used: every case fails a check of the host
print(M.lib().medusa_chunk_attention(4096, 1 << 20, ctypes.addressof(p), {dt}, 4096, 4096, 2, 4,
                                     {hkv}, {hkv}, {dh}, 0.1, 1 << 30, 4096, 1 << 30, None, None))
"""


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_medusa_b200 import build
    build.build()


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("kw", [dict(dh=0), dict(dh=-128), dict(dh=-2 ** 31),
                                dict(n=2 ** 31 - 1, page=2 ** 31 - 1, hkv=1024)])
def test_chunk_attention_shapes(dt, kw):
    code = CALL.format(**{**dict(n=4, page=16, dt=dt, dh=128, hkv=2), **kw})
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert (r.returncode, r.stdout.strip()) == (0, "2"), r.stderr


def test_a_rotation_and_a_cache_keep_their_tensors(monkeypatch):
    """The C structs hold the tensors' addresses: a new tensor would be taken
    for the old one's memory, so it is refused."""
    r = M.Rope(64, device="cpu")
    for name, value in (("turns", r.turns.clone()), ("scale", 2.0), ("rot", 32),
                        ("interleaved", True)):
        with pytest.raises(AttributeError, match="fixed"):
            setattr(r, name, value)
    monkeypatch.setattr(_lib, "_req", lambda t, name: None)
    cache = M.PagedCache.dense(torch.zeros(2, 1, 8, 64), torch.zeros(2, 1, 8, 64))
    for name in ("K", "V", "table"):
        with pytest.raises(AttributeError, match="make a new PagedCache"):
            setattr(cache, name, getattr(cache, name).clone())
    cache.name = "mine"  # and what the caller adds
    cache.name = "yours"
    cache.table.fill_(1)  # contents are the caller's
    assert cache._c.table == cache.table.data_ptr() and cache._c.K == cache.K.data_ptr()
