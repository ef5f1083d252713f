"""GPU: rotations of so many tokens that resident blocks walk them, alone and
with the write into the cache, against the formulas in 64 bits."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from oracle import prompt_oracle as P

pytestmark = pytest.mark.gpu

DEV = "cuda"
bf16, f32 = torch.bfloat16, torch.float32


def _tokens(work, chunks=0):
    """Tokens of `work` threads' units that take the resident blocks: two for
    each of them and a few more; with chunks, that many times 32 for each."""
    threads = (work + 31) // 32 * 32
    assert work <= 384
    blocks = min(1152 // threads, 32) * torch.cuda.get_device_properties(0).multi_processor_count
    return max(2, 32 * chunks) * blocks + 117


def _kernels(call):
    """Names of the kernels of a call ([] where nothing can be recorded)."""
    try:
        with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CUDA]) as prof:
            call()
            torch.cuda.synchronize()
        return [e.key for e in prof.key_averages()]
    except RuntimeError:
        return []


def _runs_resident(call):
    names = _kernels(call)
    assert not names or any("rope_pipe_kernel" in n for n in names), names


def _rotated(x, pos, freqs, scale, inter):
    """x [T, H, dh] (64 bits) rotated at pos, and the largest rotated magnitude
    of each head."""
    f = torch.from_numpy(np.asarray(freqs)).to(DEV)
    a = pos.double()[:, None] * f
    c, s = (a.cos() * scale)[:, None], (a.sin() * scale)[:, None]
    n = len(freqs)
    i = torch.arange(n, device=DEV)
    e0, e1 = (2 * i, 2 * i + 1) if inter else (i, i + n)
    y = x.clone()
    y[..., e0] = x[..., e0] * c - x[..., e1] * s
    y[..., e1] = x[..., e0] * s + x[..., e1] * c
    return y, x[..., :2 * n].abs().amax(-1, keepdim=True)


def _check(got, x, pos, freqs, scale, inter, dtype):
    """As in test_gpu_rope: half a step of the output, and fp32 arithmetic on a
    pair below 20 * 2^-24 * scale * max|x|; what is not rotated stays."""
    for lo in range(0, x.shape[0], 4096):
        xs = x[lo:lo + 4096].double()
        ref, m = _rotated(xs, pos[lo:lo + 4096], freqs, scale, inter)
        half = torch.finfo(dtype).eps / 2
        err = (got[lo:lo + 4096].double() - ref).abs()
        bound = half * ref.abs() + 20 * 2.0 ** -24 * scale * m * (1 + half) + 1e-37
        n = 2 * len(freqs)
        assert bool((err[..., :n] <= bound[..., :n]).all()), lo
        assert bool((err[..., n:] == 0).all())


def _rope(rot, inter):
    return (M.Rope(rot, theta=10000.0, interleaved=inter, scaling="yarn", factor=4.0,
                   original_max_position=2048),
            *P.rope_freqs(rot, 10000.0, "yarn", 4.0, 1.0, 32.0, 2048.0))


def _normal(g, lead, T, H, dh, dtype):
    """[T, H, dh], `lead` elements into its buffer."""
    flat = torch.empty(lead + T * H * dh, dtype=dtype, device=DEV).normal_(generator=g)
    return flat[lead:].view(T, H, dh)


def _like(x, lead):
    """A copy as far into its buffer as the original, which decides the width of
    the accesses (and so, in fp32, the order of a pair's two products)."""
    flat = torch.empty(lead + x.numel(), dtype=x.dtype, device=DEV)
    return flat[lead:].view(x.shape).copy_(x)


# units of a head: what its rotated halves and the rest fill in vectors of VEC
ROTATIONS = [  # dtype, Hq, Hkv, dh, rot, lead, VEC, chunks
    (bf16, 32, 8, 128, 128, 0, 8, 0),   # 320 units
    (bf16, 32, 8, 128, 64, 0, 8, 0),
    (f32, 16, 4, 128, 128, 0, 4, 0),
    (f32, 5, 1, 64, 48, 0, 4, 0),
    (bf16, 1, 1, 64, 64, 0, 8, 0),      # 8 units: the most blocks
    (f32, 1, 1, 32, 32, 0, 4, 0),
    (bf16, 16, 8, 256, 256, 0, 8, 2),   # 384, and more than 32 tokens a block
    (bf16, 8, 4, 64, 64, 1, 1, 2),      # 384 of single elements, at an odd address
    (f32, 3, 1, 96, 96, 1, 1, 1)]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,dh,rot,lead,VEC,chunks", ROTATIONS)
def test_rotation(dtype, Hq, Hkv, dh, rot, lead, VEC, chunks, inter):
    units = rot // (2 * VEC) + -(-(dh - rot) // (2 * VEC))
    T = _tokens((Hq + Hkv) * units, chunks)
    g = torch.Generator(device=DEV).manual_seed(dh + rot + T)
    q, k = _normal(g, lead, T, Hq, dh, dtype), _normal(g, lead, T, Hkv, dh, dtype)
    pos = torch.randint(-50, 100000, (T,), generator=g, dtype=torch.int32, device=DEV)
    r, f, s = _rope(rot, inter)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    if lead:  # (fresh tensors are aligned; operands share the narrowest)
        qo = _normal(g, lead, T, Hq, dh, dtype)
    _runs_resident(lambda: M.medusa_rope(r, q, k, pos, qo, ko))
    _check(qo, q, pos, f, s, inter, dtype)
    _check(ko, k, pos, f, s, inter, dtype)
    # in place; the inverse undoes it up to the roundings
    q2, k2 = _like(q, lead), _like(k, lead)
    M.medusa_rope(r, q2, k2, pos, q2, k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    back = torch.empty_like(q)
    M.medusa_rope(r, qo, None, pos, back, None, inverse=True)
    n = 2 * len(f)
    # two roundings and two rotations of elements below 6 s, s^2 of the whole
    half = torch.finfo(dtype).eps / 2
    err = (back[..., :n].double() / s ** 2 - q[..., :n].double()).abs()
    assert float(err.max()) <= 6 * (3 * half + 80 * 2.0 ** -24)


def _sequences(kind, T):
    """(new tokens, tokens in the cache with them) of each sequence, T rows."""
    if kind == "one":
        return [(T, T + 1000)]
    if kind == "short":  # leading rows without a slot, nothing in the cache
        n = T // 2
        return [(n, n - 300), (0, 0), (T - n, 5)]
    B = int(kind)
    cuts = sorted(np.random.default_rng(B).integers(0, T + 1, B - 1).tolist())
    if B > 20:
        cuts[3:9] = [cuts[3]] * 6  # sequences without new tokens
        cuts.sort()
    ends = cuts + [T]
    return [(e - b, e - b + (7 * i) % 90) for i, (b, e) in enumerate(zip([0] + cuts, ends))]


APPENDS = [  # dtype, Hq, Hkv, dh, rot, lead, VEC, chunks, page, sequences
    (bf16, 16, 4, 128, 128, 0, 8, 0, 16, "one"),
    (bf16, 16, 4, 128, 64, 0, 8, 0, 16, "256"),
    (bf16, 16, 4, 128, 128, 0, 8, 0, 1, "257"),   # lengths beyond shared memory
    (f32, 8, 2, 64, 64, 0, 4, 0, 7, "300"),
    (f32, 8, 2, 64, 32, 0, 4, 0, 64, "short"),
    (bf16, 1, 1, 64, 64, 0, 8, 0, 48, "5"),
    (bf16, 8, 4, 48, 48, 1, 1, 2, 16, "40"),      # more than 32 tokens a block
    (f32, 8, 4, 48, 48, 1, 1, 1, 200, "short")]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hkv,dh,rot,lead,VEC,chunks,page,kind", APPENDS)
def test_append(dtype, Hq, Hkv, dh, rot, lead, VEC, chunks, page, kind, inter):
    units, v_units = rot // (2 * VEC) + -(-(dh - rot) // (2 * VEC)), -(-dh // (2 * VEC))
    T, pad = _tokens((Hq + Hkv) * units + Hkv * v_units, chunks), 37
    g = torch.Generator(device=DEV).manual_seed(dh + rot + T)
    lens = _sequences(kind, T)
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
    kv = np.array([x for _, x in lens])
    B = len(lens)
    seq = np.repeat(np.arange(B), [n for n, _ in lens])
    slot = kv[seq] - (cu[seq + 1] - np.arange(T))
    per = [-(-x // page) for x in kv]
    n_pages = sum(per) + 2
    ids = torch.randperm(n_pages, generator=g, device=DEV).cpu().numpy()
    table = np.full((B, max(per) + 1), -9)
    at = 0
    for b in range(B):
        table[b, :per[b]] = ids[at:at + per[b]]
        at += per[b]
    q = _normal(g, lead, T + pad, Hq, dh, dtype)
    k, v = _normal(g, lead, T + pad, Hkv, dh, dtype), _normal(g, lead, T + pad, Hkv, dh, dtype)
    K, V = torch.empty(2, n_pages, Hkv, page, dh, dtype=dtype, device=DEV).normal_(generator=g)
    r, f, s = _rope(rot, inter)
    i32 = dict(dtype=torch.int32, device=DEV)
    cud, kvd = torch.tensor(cu, **i32), torch.tensor(kv, **i32)
    tb = torch.tensor(table, **i32)
    slots = torch.from_numpy(slot).to(DEV)
    has = slots >= 0
    rows = torch.from_numpy(np.maximum(slot, 0)).to(DEV)
    page_of = tb.long()[torch.from_numpy(seq).to(DEV), rows // page]

    def check(Kd, Vd, positions, rotate=True):
        left = torch.ones(n_pages, page, dtype=torch.bool, device=DEV)
        left[page_of[has], (rows % page)[has]] = False
        left = left[:, None, :, None].expand(-1, Hkv, -1, dh)
        assert torch.equal(Kd[left], K[left]) and torch.equal(Vd[left], V[left])
        got = Kd[page_of, :, rows % page][has]
        if rotate:
            _check(got, k[:T][has], positions[has], f, s, inter, dtype)
        else:
            assert torch.equal(got, k[:T][has])
        assert torch.equal(Vd[page_of, :, rows % page][has], v[:T][has])

    Kd, Vd, st = K.clone(), V.clone(), M.new_status()
    qo = torch.full_like(q, 3.0)
    cache = M.PagedCache(Kd, Vd, tb)
    _runs_resident(lambda: M.medusa_rope_append(r, q, k, v, cud, kvd, qo, cache, dev_status=st))
    assert int(st.item()) == 0
    _check(qo[:T], q[:T], slots, f, s, inter, dtype)
    assert bool((qo[T:] == 3.0).all())
    check(Kd, Vd, slots)
    # positions of their own, no q; then no rotation
    shifted = (torch.cat([slots, slots[:pad]]) + 100).to(torch.int32)
    K2, V2 = K.clone(), V.clone()
    M.medusa_rope_append(r, None, k, v, cud, kvd, None, M.PagedCache(K2, V2, tb),
                         positions=shifted, dev_status=st)
    check(K2, V2, slots + 100)
    K3, V3 = K.clone(), V.clone()
    M.medusa_rope_append(None, None, k, v, cud, kvd, None, M.PagedCache(K3, V3, tb),
                         dev_status=st)
    check(K3, V3, slots, rotate=False)
    assert int(st.item()) == 0
    # a page out of range: its rows are left and reported, the others written
    bad = tb.clone()
    b = int(seq[T // 3])
    bad[b, 0] = n_pages
    K4, V4 = K.clone(), V.clone()
    M.medusa_rope_append(r, None, k, v, cud, kvd, None, M.PagedCache(K4, V4, bad), dev_status=st)
    mine = (torch.from_numpy(seq).to(DEV) == b) & (slots >= 0) & (slots < page)
    assert int(st.item()) == (6 if bool(mine.any()) else 0)
    ref = K2.clone()
    M.medusa_rope_append(r, None, k, v, cud, kvd, None, M.PagedCache(ref, V2, tb))
    ref[page_of[mine], :, (rows % page)[mine]] = K[page_of[mine], :, (rows % page)[mine]]
    assert torch.equal(K4, ref)
