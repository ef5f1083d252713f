"""GPU: attention of a chunk of new tokens over a paged cache against the fp64
oracle."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from oracle import prompt_oracle as P
from tests.helpers import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _case(lens, Hq, Hkv, dh, page, dtype, seed=0, dense=False, pad=0, gain=1.0, spare=2):
    """Inputs on the CPU; everything outside the visible slots is NaN."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    kv = [x for _, x in lens]
    T = cu[-1] + pad
    need = [1 if dense else -(-x // page) for x in kv]
    n_pages = B if dense else sum(need) + spare
    ids = list(range(B)) if dense else torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((B, max(max(need), 1)), -77, dtype=torch.int32)
    K = torch.full((n_pages, Hkv, page, dh), math.nan)
    V = torch.full((n_pages, Hkv, page, dh), math.nan)
    at = 0
    for b in range(B):
        for j in range(need[b]):
            table[b, j] = ids[at]
            n = min(page, kv[b] - j * page)
            K[ids[at], :, :n] = torch.randn(Hkv, n, dh, generator=g)
            V[ids[at], :, :n] = torch.randn(Hkv, n, dh, generator=g)
            at += 1
    q = torch.randn(T, Hq, dh, generator=g) * gain
    return q.to(dtype), K.to(dtype), V.to(dtype), table, cu, kv


def _call(q, K, V, table, cu, kv, scale=None, want=0, out=None):
    i32 = dict(dtype=torch.int32, device=DEV)
    qd = q.to(DEV)
    out = torch.full(q.shape, 5.0, dtype=q.dtype, device=DEV) if out is None else out
    st = M.new_status()
    M.medusa_chunk_attention(qd, M.PagedCache(K.to(DEV), V.to(DEV), table.to(DEV)),
                             torch.tensor(cu, **i32), torch.tensor(kv, **i32), out, scale=scale,
                             dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want
    return out


def _check(out, q, K, V, table, cu, kv, scale=None):
    """Error bound per element, with A = sum_j p_j |v_j|:
    - scores: dh products summed in fp32 (2^-23 each, whatever the order), so
      ds <= (dh + 2) 2^-23 max_j sum |q_e k_je| scale; weights then move by a
      factor e^(2 ds) at most;
    - exponentials and the running maximum's rescales: 2^-20 together;
    - weights in bf16 for the value product: half a step, 2^-8 (bf16 only);
    - n values summed in fp32: n 2^-23;
    - the output's rounding: half a step of it."""
    dtype, dh = q.dtype, q.shape[2]
    scale = dh ** -0.5 if scale is None else scale
    n_rows = cu[-1]
    Kz, Vz = torch.nan_to_num(K.float()), torch.nan_to_num(V.float())
    ref, absv, mag, count = P.chunk_attention(f64(q)[:n_rows], f64(Kz), f64(Vz), table.numpy(), cu,
                                              kv, scale)
    got = f64(out)
    ds = (dh + 2) * 2.0 ** -23 * mag
    rel = np.expm1(2 * ds) + 2.0 ** -20 + count * 2.0 ** -23
    half = torch.finfo(dtype).eps / 2
    if dtype is torch.bfloat16:
        rel = rel + half
    bound = rel[..., None] * absv
    bound = bound + half * (np.abs(ref) + bound) + 1e-37
    err = np.abs(got[:n_rows] - ref)
    assert (err <= bound).all(), (float((err / bound).max()), np.argwhere(err > bound)[:4].tolist())
    assert (got[n_rows:] == 5.0).all()


RAGGED = [(3, 40), (0, 9), (1, 130), (17, 17), (5, 3), (1, 1), (0, 0), (40, 300)]
bf16, f32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 48, 64, 96, 128, 130, 200, 256])
def test_page_sizes(dtype, page):
    c = _case(RAGGED, 4, 2, 64, page, dtype, seed=page, pad=3)
    _check(_call(*c), *c)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("Hq,Hkv,dh", [(1, 1, 128), (3, 1, 64), (6, 2, 128), (7, 1, 64), (8, 8, 64),
                                       (16, 1, 128), (48, 1, 64), (128, 1, 64), (5, 1, 128)])
def test_head_layouts(dtype, Hq, Hkv, dh):
    c = _case([(9, 50), (1, 200), (33, 33)], Hq, Hkv, dh, 16, dtype, seed=Hq, pad=1)
    _check(_call(*c), *c)


@pytest.mark.parametrize("dh", [32, 96, 160, 192, 224, 256])
def test_fp32_head_sizes(dh):
    c = _case([(9, 50), (1, 77)], 2, 1, dh, 16, f32, seed=dh)
    _check(_call(*c), *c)


@pytest.mark.parametrize("G", [2, 3, 5, 8])
@pytest.mark.parametrize("dh", [32, 128, 160, 256])
def test_fp32_shared_heads(G, dh):
    c = _case([(5, 40), (1, 9), (3, 3)], 2 * G, 2, dh, 16, f32, seed=dh + G, pad=2)
    _check(_call(*c), *c)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_many_sequences(dtype):
    """More than a warp's lanes, some of them without new tokens."""
    lens = [((b * 7) % 4, 4 + (b * 13) % 60) for b in range(75)]
    c = _case(lens, 4, 2, 64, 8, dtype, seed=3, pad=1)
    _check(_call(*c), *c)


@pytest.mark.parametrize("dtype", [bf16, f32])
@pytest.mark.parametrize("cap", [1, 3, 37, 100, 127, 129, 255, 400])
def test_dense_caches(dtype, cap):
    lens = [(min(3, cap), cap), (1, max(1, cap - 1)), (0, 0), (min(cap, 50), cap)]
    c = _case(lens, 4, 2, 128, cap, dtype, seed=cap, dense=True)
    _check(_call(*c), *c)


@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    ([(1, 5000)], 8, 2, 64), ([(1, 127), (1, 128), (1, 129), (1, 256), (1, 257)], 4, 4, 128),
    ([(300, 700)], 4, 1, 64), ([(129, 129), (256, 256), (257, 300)], 2, 1, 128),
    ([(1, 900)] * 40, 4, 1, 16), ([(2, 2000), (64, 1500), (1, 3000)], 8, 4, 32),
    ([(700, 700)], 2, 2, 16)])
@pytest.mark.parametrize("dh", [64, 128])
def test_long_chunks_and_splits(lens, Hq, Hkv, page, dh):
    """Tiles, query groups and key ranges shared by several blocks."""
    c = _case(lens, Hq, Hkv, dh, page, bf16, seed=len(lens) + dh, pad=2)
    _check(_call(*c), *c)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_large_and_growing_scores(dtype):
    """Scores of hundreds with a maximum that keeps growing along the keys,
    and one key far above all others."""
    c = list(_case([(5, 700), (1, 900), (64, 640)], 4, 2, 64, 64, dtype, seed=5, gain=6.0))
    table, kv = c[3], c[5]
    for b in range(3):
        for j in range(kv[b]):
            c[1][table[b, j // 64], :, j % 64] *= 1.0 + j / 200.0
    c[1][table[0, 2], :, 5] *= 10.0
    _check(_call(*c), *c)
    _check(_call(*c, scale=1e-4), *c, scale=1e-4)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_strided_queries_and_large_values(dtype):
    q, K, V, table, cu, kv = _case([(20, 60), (4, 90)], 4, 2, 64, 16, dtype, seed=1)
    V = V * 1e6
    wide = torch.full((q.shape[0], 8, 64), math.nan, dtype=dtype)
    wide[:, 2:6] = q
    out = torch.full(q.shape, 5.0, dtype=dtype, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    st = M.new_status()
    M.medusa_chunk_attention(wide.to(DEV)[:, 2:6],
                             M.PagedCache(K.to(DEV), V.to(DEV), table.to(DEV)),
                             torch.tensor(cu, **i32), torch.tensor(kv, **i32), out, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    _check(out, q, K, V, table, cu, kv)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_device_checks(dtype):
    """Bad pages and lengths are reported and nothing outside is touched; a
    non-finite value in a visible slot is reported."""
    q, K, V, table, cu, kv = _case([(4, 40), (2, 20)], 2, 1, 64, 16, dtype, pad=2)
    for bad in (-1, K.shape[0], 10 ** 6):
        t2 = table.clone()
        t2[0, 1] = bad
        out = _call(q, K, V, t2, cu, kv, want=6)
        assert (out[6:] == 5.0).all()
    _call(q, K, V, table, cu, [40, 16 * table.shape[1] + 1], want=6)
    _call(q, K, V, table, cu, [-1, 20], want=6)
    _call(q, K, V, table, [0, 9, 6], kv, want=6)
    _call(q, K, V, table, [0, 4, 99], kv, want=6)
    _call(q, K, V, table, [-3, 4, 6], kv, want=6)
    V2 = V.clone()
    V2[table[0, 0], 0, 3, 7] = math.inf
    _call(q, K, V2, table, cu, kv, want=6)


def test_page_offsets_beyond_32_bits():
    """A pool of more than 2^31 elements, the sequence's pages at its end."""
    Hkv, dh, page = 1, 128, 128
    n_pages = (1 << 31) // (Hkv * page * dh) + 40
    K = torch.zeros(n_pages, Hkv, page, dh, dtype=bf16, device=DEV)
    V = torch.zeros(n_pages, Hkv, page, dh, dtype=bf16, device=DEV)
    q, Ks, Vs, table, cu, kv = _case([(3, 300)], 2, 1, dh, page, bf16, spare=0)
    t2 = table + (n_pages - Ks.shape[0])
    K[-Ks.shape[0]:], V[-Ks.shape[0]:] = Ks.to(DEV), Vs.to(DEV)
    _check(_call(q, K, V, t2, cu, kv), q, Ks, Vs, table, cu, kv)


@pytest.mark.parametrize("dtype", [bf16, f32])
def test_capture_streams_and_a_shared_workspace(dtype):
    """Two graphs captured over one workspace replay in turn; a call on a side
    stream gives the same bits; results repeat bit for bit."""
    a = _case([(1, 3000), (60, 900)], 8, 2, 64, 16, dtype, seed=1)
    b = _case([(1, 500)] * 5, 4, 4, 64, 64, dtype, seed=2)
    i32 = dict(dtype=torch.int32, device=DEV)
    dt = M.MEDUSA_BF16 if dtype is bf16 else M.MEDUSA_F32
    ws = M.workspace(max(M.medusa_chunk_attention_workspace_size(8, 2, 64, dt),
                         M.medusa_chunk_attention_workspace_size(4, 4, 64, dt)))
    ws.random_(0, 255)  # its contents on entry do not matter
    work = []
    for q, K, V, table, cu, kv in (a, b):
        cache = M.PagedCache(K.to(DEV), V.to(DEV), table.to(DEV))
        qd, cud, kvd = q.to(DEV), torch.tensor(cu, **i32), torch.tensor(kv, **i32)
        out = torch.empty_like(qd)
        first = torch.empty_like(qd)
        M.medusa_chunk_attention(qd, cache, cud, kvd, first, ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            M.medusa_chunk_attention(qd, cache, cud, kvd, out, ws=ws)
        work.append((g, out, first, qd, cache, cud, kvd))
    for _ in range(3):
        for g, out, first, *_ in work:
            out.fill_(9.0)
            g.replay()
        torch.cuda.synchronize()
        for g, out, first, *_ in work:
            assert torch.equal(out, first)
    g, out, first, qd, cache, cud, kvd = work[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out.fill_(9.0)
    s.wait_stream(torch.cuda.current_stream())
    M.medusa_chunk_attention(qd, cache, cud, kvd, out, ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, first)


def test_no_rows():
    c = _case([(0, 5), (0, 0)], 2, 1, 64, 16, bf16)
    _call(*c)
    c = _case([(0, 5), (0, 0)], 2, 1, 64, 16, bf16, pad=3)
    assert (_call(*c) == 5.0).all()
