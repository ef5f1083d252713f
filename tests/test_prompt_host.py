"""Prompt side without a GPU: the refusals of the C calls, the rotation
frequencies, the binding's argument checks and pins of the oracle."""
import ctypes
import math

import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from oracle import prompt_oracle as P
from speculative_decoding_medusa_b200 import _lib

v = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_medusa_b200 import build
    build.build()
    return M.lib()


def _rope(rot=64, inter=0, turns=4096):
    return _lib.medusa_rope_t(rot, inter, 1.0, turns)


def _pages(K=4096, V=4096, table=4096, n=4, page=16, max_pages=8):
    return _lib.medusa_pages_t(K, V, table, n, page, max_pages)


# the addresses below are never dereferenced: each case fails a host check (or
# asks for no rows) before any launch


def test_rope_refusals(L):
    def call(r=None, q=1 << 20, qs=256, k=1 << 21, ks=128, dt=0, pos=4096, T=4, Hq=4, Hkv=2, dh=64,
             qo=1 << 22, qos=256, ko=1 << 23, kos=128):
        r = _rope() if r is None else r
        return L.medusa_rope(ctypes.addressof(r), q, qs, k, ks, dt, pos, T, Hq, Hkv, dh, 0, qo,
                             qos, ko, kos, None)

    assert L.medusa_rope(None, v(64), 1, None, 0, 0, v(64), 1, 1, 1, 64, 0, v(64), 1, None, 0,
                         None) == 1
    assert call(T=0) == 0                        # nothing to do
    assert call(T=0, q=None, qo=None) == 0
    assert call(T=-1) == 2 and call(Hq=0) == 2 and call(Hkv=0) == 2 and call(dh=2048) == 2
    assert call(dt=3) == 1
    assert call(r=_rope(63)) == 2 and call(r=_rope(66)) == 2 and call(r=_rope(0)) == 2
    assert call(r=_rope(turns=None)) == 1 and call(r=_rope(turns=4100)) == 8
    assert call(q=None) == 1 and call(pos=None) == 1 and call(ko=None) == 1
    assert call(qs=255) == 2 and call(kos=100) == 2
    assert call(q=(1 << 20) + 1) == 8
    assert call(dt=1, q=(1 << 20) + 2) == 8
    # in place needs equal strides; other overlaps are refused
    assert call(qo=1 << 20, qos=512) == 1
    assert call(qo=(1 << 20) + 64) == 1
    assert b"overlap" in L.medusa_last_error()
    assert call(ko=(1 << 21) + 2 * 3 * 128) == 1  # last row against the first
    # slices of one packed buffer (equal strides) may interleave, but not touch
    assert call(qs=512, qo=(1 << 20) + 2 * 200, qos=512) == 1


def test_operands_that_share_memory_are_refused(L):
    """q's and k's operands of one call, among packed slices and apart."""
    r = _rope()
    buf = 1 << 20

    def call(q, k, qo, ko, st, sto=None, T=4):
        sto = sto or st
        return L.medusa_rope(ctypes.addressof(r), q, st, k, st, 0, 4096, T, 4, 2, 64, 0, qo, sto,
                             ko, sto, None)

    n = 4 * 64 * 2  # bytes of q's heads of a token
    # q_out over k, k_out over q, q_out over k_out
    assert call(buf, 2 * buf, 2 * buf, 3 * buf, 512) == 1
    assert call(buf, 2 * buf, 3 * buf, buf + n - 64, 512) == 1
    assert call(buf, 2 * buf, 3 * buf, 3 * buf + 64, 512) == 1
    assert call(buf, buf + n, buf, buf + n - 128, 512) == 1  # k_out a head early, over q
    assert call(buf, buf + n, 3 * buf, 3 * buf + n - 2, 512, T=1) == 1
    assert b"overlap" in L.medusa_last_error()
    pages = _pages()

    def append(q, k, v, qo, st=1024):
        return L.medusa_rope_append(ctypes.addressof(r), q, st, k, st, v, st, 0, None, 4096, 4096,
                                    2, 4, 4, 2, 64, qo, st, ctypes.addressof(pages), None, None)

    assert append(buf, 2 * buf, 3 * buf, 2 * buf + 64) == 1
    assert append(buf, 2 * buf, 3 * buf, 3 * buf - 64) == 1
    assert append(buf, buf + n, buf + n + 256, buf + n) == 1  # packed: q's result over k

    def attend(q, qs, out, T=4):
        return L.medusa_chunk_attention(q, qs, ctypes.addressof(pages), 0, 4096, 4096, 2, T, 4, 2,
                                        128, 0.1, out, None, 0, None, None)

    assert attend(buf, 512, buf) == 1 and attend(buf, 512, buf + 4 * 1024 - 16) == 1
    assert attend(buf, 1024, buf + 1024) == 1     # out dense between q's strided rows
    assert attend(buf, 512, buf + 1008, T=1) == 1


def test_rope_append_refusals(L):
    def call(r=0, q=1 << 20, k=1 << 21, ks=128, vv=1 << 24, vs=128, dt=0, cu=4096, kv=4096, B=2,
             T=4, Hq=4, Hkv=2, dh=64, qo=1 << 22, pages=None):
        r = _rope() if r == 0 else r
        pages = _pages() if pages is None else pages
        return L.medusa_rope_append(ctypes.addressof(r) if r is not None else None, q, 256, k, ks,
                                    vv, vs, dt, None, cu, kv, B, T, Hq, Hkv, dh, qo, 256,
                                    ctypes.addressof(pages), None, None)

    assert call(T=0) == 0
    assert call(pages=_pages(K=None)) == 1 and call(pages=_pages(table=None)) == 1
    assert call(pages=_pages(n=0)) == 2 and call(pages=_pages(page=0)) == 2
    assert call(pages=_pages(max_pages=0)) == 2
    assert call(pages=_pages(V=4097)) == 8
    assert call(B=0) == 2 and call(Hkv=0) == 2 and call(T=-1) == 2
    assert call(r=None) == 1                      # q without a rotation
    assert call(r=_rope(66)) == 2
    assert call(cu=None) == 1 and call(kv=None) == 1 and call(k=None) == 1 and call(vv=None) == 1
    assert call(qo=None) == 1 and call(q=None) == 1
    assert call(ks=64) == 2 and call(vs=64) == 2


def test_chunk_attention_refusals(L):
    def call(q=4096, qs=512, pages=None, dt=0, cu=4096, kv=4096, B=2, T=4, Hq=4, Hkv=2, dh=128,
             scale=0.1, out=4096, ws=4096, ws_bytes=1 << 30):
        pages = _pages() if pages is None else pages
        return L.medusa_chunk_attention(q, qs, ctypes.addressof(pages), dt, cu, kv, B, T, Hq, Hkv,
                                        dh, scale, out, ws, ws_bytes, None, None)

    assert call(T=0) == 0 and call(T=0, q=None, out=None) == 0
    assert call(dt=2) == 1
    assert call(pages=_pages(V=None)) == 1 and call(pages=_pages(K=4104)) == 8
    assert call(B=0) == 2 and call(B=1025) == 2 and call(Hq=3) == 2
    assert call(Hq=258, qs=258 * 128) == 2        # 129 query heads per kv head
    assert call(dh=96) == 2 and call(dt=1, dh=48) == 2 and call(dt=1, dh=288, qs=4 * 288) == 2
    assert call(scale=0.0) == 1 and call(scale=math.inf) == 1 and call(scale=math.nan) == 1
    assert call(q=None) == 1 and call(cu=None) == 1 and call(out=None) == 1
    assert call(qs=504) == 2 and call(qs=516) == 8
    assert call(q=4104) == 8 and call(out=4104) == 8
    assert call(pages=_pages(n=1 << 30, page=1 << 20)) == 2
    assert M.medusa_chunk_attention_workspace_size(0, 1, 128, 0) == 0


def test_sample_tokens_refusals(L):
    def call(lg=4096, dt=0, stride=100, n=2, idx=None, R=2, V=100, u=4096, tok=4096):
        return L.medusa_sample_tokens(lg, dt, stride, n, idx, R, V, u, None, None, None, None, tok,
                                      None, None, None)

    assert call(R=0) == 0 and call(R=0, n=0, lg=None, u=None, tok=None) == 0
    assert call(dt=5) == 1
    assert call(V=0) == 2 and call(V=655361, stride=655361) == 2
    assert call(dt=1, V=327681, stride=327681) == 2
    assert call(R=-1) == 2 and call(R=70000, n=70000) == 2
    assert call(stride=99) == 2
    assert call(R=3) == 2                         # more draws than rows without row_idx
    assert call(lg=None) == 1 and call(u=None) == 1 and call(tok=None) == 1
    assert call(lg=4097) == 8


def test_binding_refuses_wrong_tensors(monkeypatch):
    monkeypatch.setattr(_lib, "_dev", lambda: 0)
    q = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        M.medusa_rope(M.Rope(64, device="cpu"), q, None, torch.zeros(4, dtype=torch.int32), q, None)
    with pytest.raises(ValueError, match="T, H, dh"):
        M.medusa_rope(M.Rope(64, device="cpu"), q[0], None, None, q, None)
    with pytest.raises(ValueError, match="contiguous CUDA"):
        M.PagedCache(torch.zeros(2, 2, 16, 64), torch.zeros(2, 2, 16, 64),
                     torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        M.medusa_sample_tokens(torch.zeros(2, 10), torch.zeros(2), torch.zeros(2))
    with pytest.raises(ValueError, match="scaling"):
        M.Rope(64, scaling="other", device="cpu")


@pytest.mark.parametrize("kw,status", [
    (dict(rot=63), 2), (dict(rot=0), 2), (dict(rot=514), 2), (dict(rot=64, theta=1.0), 1),
    (dict(rot=64, theta=math.inf), 1), (dict(rot=64, scaling="linear", factor=0.5), 1),
    (dict(rot=64, scaling="linear", factor=math.nan), 1),
    (dict(rot=64, scaling="llama3", factor=8.0, low_freq_factor=4.0, high_freq_factor=4.0), 1),
    (dict(rot=64, scaling="yarn", factor=8.0, original_max_position=0), 1)])
def test_rope_freqs_refusals(kw, status):
    with pytest.raises(M.MedusaError) as e:
        M.Rope(device="cpu", **kw)
    assert e.value.status == status


@pytest.mark.parametrize("rot", [2, 6, 34, 64, 128, 512])
@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1.5])
@pytest.mark.parametrize("scaling,kw", [
    ("none", {}), ("linear", dict(factor=4.0)), ("linear", dict(factor=1.0)),
    ("llama3", dict(factor=8.0)),
    ("llama3", dict(factor=32.0, low_freq_factor=0.5, high_freq_factor=16.0,
                    original_max_position=1024)),
    ("yarn", dict(factor=16.0, original_max_position=4096)),
    ("yarn", dict(factor=2.5, low_freq_factor=2.0, high_freq_factor=50.0,
                  original_max_position=32768))])
def test_rope_freqs_match_the_formulas(rot, theta, scaling, kw):
    r = M.Rope(rot, theta=theta, scaling=scaling, device="cpu", **kw)
    high = 32.0 if scaling == "yarn" else 4.0
    f, scale = P.rope_freqs(rot, theta, scaling, kw.get("factor", 1.0),
                            kw.get("low_freq_factor", 1.0), kw.get("high_freq_factor", high),
                            kw.get("original_max_position", 8192.0))
    got = r.turns.numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2.0 * math.pi
    # the oracle's powers and blends run in fp64: a few units of 2^-53 each,
    # times log(theta) for the power; the table itself is exact to 2^-65 turns
    np.testing.assert_allclose(got, f, rtol=2e-14, atol=4e-19)
    assert abs(r.scale - scale) <= 2.0 ** -24 * scale


def test_oracle_rotation_pins():
    """A quarter turn, a norm-preserving rotation, relative positions, and the
    inverse undoing the forward call."""
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    y = P.rope(x, [1], np.array([math.pi / 2, 0.0]))
    np.testing.assert_allclose(y, [[[-3.0, 2.0, 1.0, 4.0, 9.0]]], atol=1e-15)
    y = P.rope(x, [1], np.array([math.pi / 2, 0.0]), interleaved=True)
    np.testing.assert_allclose(y, [[[-2.0, 1.0, 3.0, 4.0, 9.0]]], atol=1e-15)
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 8))
    f, _ = P.rope_freqs(8, 10000.0)
    dots = [float((P.rope(q, [p + 5], f) * P.rope(k, [p], f)).sum()) for p in (0, 7, 100)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-12)
    np.testing.assert_allclose(P.rope(P.rope(q, [77], f), [77], f, inverse=True), q, atol=1e-14)


def test_oracle_attention_pins():
    """Equal keys average the visible values; a page table permutes pages;
    rows before the first slot see nothing."""
    K = np.zeros((3, 1, 2, 4))
    V = np.arange(24, dtype=np.float64).reshape(3, 1, 2, 4)
    q = np.ones((3, 1, 4))
    out, _, _, n = P.chunk_attention(q, K, V, np.array([[2, 0, 1]]), [0, 3], [3], 1.0)
    rows = np.stack([V[2, 0, 0], V[2, 0, 1], V[0, 0, 0]])
    np.testing.assert_allclose(out[2, 0], rows.mean(0))
    np.testing.assert_allclose(out[0, 0], rows[0])
    assert n[:, 0].tolist() == [1, 2, 3]
    out, _, _, n = P.chunk_attention(q, K, V, np.array([[2, 0, 1]]), [0, 3], [1], 1.0)
    assert n[:, 0].tolist() == [0, 0, 1] and (out[:2] == 0).all()


def test_oracle_sampling_pins():
    z = np.log(np.array([0.1, 0.4, 0.1, 0.4]))
    assert P.sample_row(z, 0.0)[:2] == (0, 4)
    assert P.sample_row(z, 0.05)[:2] == (0, 4)
    assert P.sample_row(z, 0.15)[:2] == (1, 4)
    assert P.sample_row(z, 0.999)[:2] == (3, 4)
    assert P.sample_row(z, 0.999, top_k=3)[:2] == (3, 3)   # ties: token 0 before 2
    assert P.sample_row(z, 0.01, top_k=3)[:2] == (0, 3)
    assert P.sample_row(z, 0.01, top_p=0.5)[:2] == (1, 2)
    assert P.sample_row(z, 0.99, top_p=0.3)[:2] == (1, 1)
    assert P.sample_row(z, 0.5, min_p=0.3)[0] == 3
    assert P.sample_row(z, 0.5, temperature=0.0)[:2] == (1, 1)


def test_marshalling_leaves_the_unusual_to_the_binding():
    """The extension makes no call with what it cannot check: -1."""
    m = _lib._marshal()
    q, i = torch.zeros(4, 2, 64), torch.zeros(4, dtype=torch.int32)
    r = M.Rope(64, device="cpu")
    assert m.rope(r._ref, r.turns, q, None, i, q, None, False) == -1        # CPU tensors
    assert m.rope(r._ref, r.turns, None, None, i, q, None, False) == -1
    assert m.rope(r._ref, r.turns, [1.0], None, i, q, None, False) == -1
    assert m.rope(r._ref) == -1
    assert m.append(None, None, None, q, q, i, i, None, 0, q.view(4, 2, 1, 64), 3, None, None) == -1
    assert m.append(None, None, None, q, q, i, i, None, 0, None, 3, None, None) == -1
    assert m.attention(q, 0, q.view(4, 2, 1, 64), i, i, q, 3, 0.1, i, None) == -1
    assert m.attention(q, 0, q, i, i, q, "three", 0.1, i, None) == -1
    assert m.sample(q[0], i, i, None, None, None, None, None, None, None) == -1
    assert m.sample(*[None] * 10) == -1
    with pytest.raises(TypeError):
        m.bind(1, 2)
