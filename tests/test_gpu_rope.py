"""GPU: rotary positions, alone and with the write into the cache, against the
fp64 oracle."""
import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from oracle import prompt_oracle as P
from tests.helpers import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _bound(x, y, scale, rot, dtype):
    """Per element: the rounding of the output (half a step of the result),
    and for fp32 arithmetic on a pair (x0, x1): cos and sin within 2 ulp
    (2^-23 relative to 1) of an angle within 2^-28 turns (2.4e-8), their
    product with scale, two products and a sum (2^-24 each) - together below
    10 * 2^-24 * scale * (|x0| + |x1|) <= 20 * 2^-24 * scale * max|x|."""
    half_step = torch.finfo(dtype).eps / 2
    m = np.abs(x[..., :rot]).max(axis=-1, keepdims=True) if rot else 0.0
    return half_step * np.abs(y) + 20 * 2.0 ** -24 * scale * m * (1 + half_step) + 1e-37


def _check(got, x, ref, scale, rot, dtype):
    got = f64(got)
    np.testing.assert_array_equal(got[..., rot:], x[..., rot:])
    err = np.abs(got - ref)
    assert (err <= _bound(x, ref, scale, rot, dtype)).all(), float(err.max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,dh,rot,inter", [
    (1, 1, 1, 64, 64, False), (9, 4, 4, 64, 32, True), (33, 6, 2, 128, 128, False),
    (17, 5, 5, 80, 34, False), (17, 5, 1, 80, 34, True), (3, 2, 1, 7, 2, True),
    (5, 3, 3, 66, 66, False), (2500, 2, 1, 64, 64, True), (2371, 3, 1, 128, 64, False),
    (4, 64, 8, 512, 512, False), (6, 71, 1, 64, 64, False), (300, 8, 2, 128, 34, False),
    (300, 40, 8, 64, 18, True), (5, 200, 8, 128, 34, False)])
def test_rotation(dtype, T, Hq, Hkv, dh, rot, inter):
    g = torch.Generator().manual_seed(T + dh + rot)
    q = torch.randn(T, Hq, dh, generator=g).to(dtype)
    k = (torch.randn(T, Hkv, dh, generator=g) * 3).to(dtype)
    pos = torch.randint(0, 10000, (T,), generator=g, dtype=torch.int32)
    r = M.Rope(rot, theta=10000.0, interleaved=inter, scaling="yarn", factor=4.0,
               original_max_position=2048)
    f, s = P.rope_freqs(rot, 10000.0, "yarn", 4.0, 1.0, 32.0, 2048.0)
    qd, kd = q.to(DEV), k.to(DEV)
    qo, ko = torch.full_like(qd, 7.0), torch.full_like(kd, 7.0)
    M.medusa_rope(r, qd, kd, pos.to(DEV), qo, ko)
    _check(qo, f64(q), P.rope(f64(q), pos.tolist(), f, s, inter), s, rot, dtype)
    _check(ko, f64(k), P.rope(f64(k), pos.tolist(), f, s, inter), s, rot, dtype)
    # in place: the same bits; one tensor alone: the same bits
    q2, k2 = qd.clone(), kd.clone()
    M.medusa_rope(r, q2, k2, pos.to(DEV), q2, k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)
    q3 = torch.empty_like(qd)
    M.medusa_rope(r, qd, None, pos.to(DEV), q3, None)
    assert torch.equal(q3, qo)


def test_far_and_negative_positions():
    """Angles keep their precision at any position (fp32 products would not)."""
    pos = [0, 1, 131071, 1000003, 2 ** 31 - 1, -1, -5000, -2 ** 31]
    q = torch.randn(len(pos), 2, 128, generator=torch.Generator().manual_seed(3))
    r = M.Rope(128, theta=500000.0)
    f, s = P.rope_freqs(128, 500000.0)
    out = torch.empty_like(q, device=DEV)
    M.medusa_rope(r, q.to(DEV), None, torch.tensor(pos, dtype=torch.int32, device=DEV), out, None)
    ref = P.rope(f64(q), pos, f, s)
    # the fp64 oracle's own angle is off by up to |p| f 2^-53 <= 2.4e-7 at 2^31
    err = np.abs(f64(out) - ref)
    x = np.abs(f64(q)).max()
    slack = np.array([abs(p) * 2.0 ** -52 for p in pos])[:, None, None] * 2 * x
    assert (err <= _bound(f64(q), ref, s, 128, torch.float32) + slack).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_gradient(dtype, inter):
    """The inverse call is the transpose: against the formula's gradient, and
    against differences of the forward call (linear, so a large step is exact
    up to roundings)."""
    T, H, dh, rot = 7, 3, 64, 48
    g = torch.Generator().manual_seed(5)
    x, gy = torch.randn(2, T, H, dh, generator=g).to(dtype)
    pos = torch.randint(0, 4000, (T,), generator=g, dtype=torch.int32)
    r = M.Rope(rot, interleaved=inter, scaling="yarn", factor=8.0, original_max_position=4096)
    f, s = P.rope_freqs(rot, 10000.0, "yarn", 8.0, 1.0, 32.0, 4096.0)
    gx = torch.empty_like(gy, device=DEV)
    M.medusa_rope(r, gy.to(DEV), None, pos.to(DEV), gx, None, inverse=True)
    _check(gx, f64(gy), P.rope(f64(gy), pos.tolist(), f, s, inter, inverse=True), s, rot, dtype)
    if dtype is torch.float32:
        d = torch.randn(T, H, dh, generator=g)
        ends = []
        for sign in (1.0, -1.0):
            y = torch.empty(T, H, dh, device=DEV)
            M.medusa_rope(r, (x + sign * d).to(DEV), None, pos.to(DEV), y, None)
            ends.append(f64(y))
        lhs = ((ends[0] - ends[1]) / 2 * f64(gy)).sum()
        rhs = (f64(d) * f64(gx)).sum()
        # three rotations of magnitude <= 6 and T*H*dh products: each element is
        # within 20 * 2^-24 * s * 12, against |gy| <= 6
        assert abs(lhs - rhs) <= 3 * T * H * dh * 20 * 2.0 ** -24 * s * 12 * 6


def test_strided_slices_and_misaligned_starts():
    """q, k as slices of one packed projection, rotated in place inside it and
    out of it; an odd element offset takes narrower accesses."""
    T, Hq, Hkv, dh = 21, 4, 2, 64
    g = torch.Generator().manual_seed(8)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 3
    r = M.Rope(64)
    for lead in (0, 1, 2, 4):
        flat = torch.randn(lead + T * (Hq + 2 * Hkv) * dh, generator=g).to(torch.bfloat16).to(DEV)
        qkv = flat[lead:].view(T, Hq + 2 * Hkv, dh)
        q, k, rest = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:].clone()
        qo = torch.empty(T, Hq, dh, dtype=torch.bfloat16, device=DEV)
        ko = torch.empty(T, Hkv, dh, dtype=torch.bfloat16, device=DEV)
        M.medusa_rope(r, q.contiguous(), k.contiguous(), pos, qo, ko)
        qo2, ko2 = torch.empty_like(qo), torch.empty_like(ko)
        M.medusa_rope(r, q, k, pos, qo2, ko2)
        assert torch.equal(qo2, qo) and torch.equal(ko2, ko)
        M.medusa_rope(r, q, k, pos, q, k)
        assert torch.equal(qkv[:, :Hq], qo) and torch.equal(qkv[:, Hq:Hq + Hkv], ko)
        assert torch.equal(qkv[:, Hq + Hkv:], rest)


def test_refuses_wrong_layouts():
    q = torch.zeros(4, 2, 64, device=DEV)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    r = M.Rope(64)
    with pytest.raises(ValueError, match="dense"):
        M.medusa_rope(r, q.transpose(1, 2).contiguous().transpose(1, 2), None, pos, q, None)
    with pytest.raises(ValueError, match="positions"):
        M.medusa_rope(r, q, None, pos.long(), q, None)
    with pytest.raises(ValueError, match="q_out"):
        M.medusa_rope(r, q, None, pos, torch.zeros(4, 2, 64, device=DEV).bfloat16(), None)
    with pytest.raises(M.MedusaError):
        M.medusa_rope(r, q[1:], None, pos[1:], q[:3], None)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,lens,dense", [
    (16, [(5, 40), (0, 7), (1, 16), (20, 20), (3, 17)], False),
    (1, [(3, 9), (2, 2)], False), (7, [(9, 30), (1, 1)], False),
    (50, [(6, 50), (1, 13), (0, 0)], True)])
@pytest.mark.parametrize("rot", [32, 18])
def test_append(dtype, page, lens, dense, rot):
    Hq, Hkv, dh = 6, 2, 64
    g = torch.Generator().manual_seed(page)
    B, T = len(lens), sum(n for n, _ in lens)
    pad = 4  # rows behind the last sequence
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    kv = [x for _, x in lens]
    n_pages = B if dense else sum(-(-x // page) for x in kv) + 2
    ids = list(range(B)) if dense else torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((B, 1 if dense else max(-(-x // page) for x in kv) + 1), -9,
                       dtype=torch.int32)
    at = 0
    for b, x in enumerate(kv):
        for j in range(1 if dense else -(-x // page)):
            table[b, j] = ids[at]
            at += 1
    K, V = torch.randn(2, n_pages, Hkv, page, dh, generator=g).to(dtype)
    q, = torch.randn(1, T + pad, Hq, dh, generator=g).to(dtype)
    k, v = torch.randn(2, T + pad, Hkv, dh, generator=g).to(dtype)
    r = M.Rope(rot, theta=5000.0)
    f, s = P.rope_freqs(rot, 5000.0)
    Kd, Vd, tb = K.to(DEV), V.to(DEV), table.to(DEV)
    qo = torch.full((T + pad, Hq, dh), 3.0, dtype=dtype, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    st = M.new_status()
    cache = M.PagedCache(Kd, Vd, tb)
    M.medusa_rope_append(r, q.to(DEV), k.to(DEV), v.to(DEV), torch.tensor(cu, **i32),
                         torch.tensor(kv, **i32), qo, cache, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    pos = P.slots(cu, kv, T)[:, 1]
    _check(qo[:T], f64(q)[:T], P.rope(f64(q)[:T], pos, f, s), s, rot, dtype)
    assert (qo[T:] == 3.0).all()
    tn = table.numpy()
    assert torch.equal(Vd.cpu().double(), torch.from_numpy(P.append(f64(V), f64(v)[:T], tn, cu, kv)))
    kr = P.rope(f64(k)[:T], pos, f, s)
    ref = P.append(f64(K), kr, tn, cu, kv)
    written = P.append(np.zeros(K.shape), np.ones((T, Hkv, dh)), tn, cu, kv) > 0
    got = f64(Kd)
    np.testing.assert_array_equal(got[~written], f64(K)[~written])
    back = np.stack([got[tn[b, p // page], :, p % page] for b, p in P.slots(cu, kv, T)])
    _check(torch.from_numpy(back), f64(k)[:T], kr, s, rot, dtype)
    # explicit positions, no q; and no rotation at all
    K2, V2 = K.to(DEV), V.to(DEV)
    shifted = torch.from_numpy(np.concatenate([pos, np.zeros(pad)]).astype(np.int32) + 100).to(DEV)
    M.medusa_rope_append(r, None, k.to(DEV), v.to(DEV), torch.tensor(cu, **i32),
                         torch.tensor(kv, **i32), None, M.PagedCache(K2, V2, tb),
                         positions=shifted)
    kr = P.rope(f64(k)[:T], pos + 100, f, s)
    got = f64(K2)
    back = np.stack([got[tn[b, p // page], :, p % page] for b, p in P.slots(cu, kv, T)])
    _check(torch.from_numpy(back), f64(k)[:T], kr, s, rot, dtype)
    K3, V3 = K.to(DEV), V.to(DEV)
    M.medusa_rope_append(None, None, k.to(DEV), v.to(DEV), torch.tensor(cu, **i32),
                         torch.tensor(kv, **i32), None, M.PagedCache(K3, V3, tb))
    assert torch.equal(K3.cpu().double(), torch.from_numpy(P.append(f64(K), f64(k)[:T], tn, cu, kv)))
    assert torch.equal(V3, Vd)


def test_append_bad_pages_are_reported_and_skipped():
    Hkv, dh, page = 1, 64, 4
    i32 = dict(dtype=torch.int32, device=DEV)
    k = torch.randn(6, Hkv, dh, device=DEV)
    for table, kv in (([[0, 5]], [6]), ([[0, -1]], [6]), ([[0]], [6])):
        K, V = torch.zeros(2, 2, Hkv, page, dh, device=DEV)
        st = M.new_status()
        M.medusa_rope_append(None, None, k, k, torch.tensor([0, 6], **i32), torch.tensor(kv, **i32),
                             None, M.PagedCache(K, V, torch.tensor(table, **i32)), dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 6
        assert torch.equal(K[0, 0], k[:4, 0]) and (K[1] == 0).all()
    # a cache shorter than the chunk: leading rows have no slot, no error
    K, V = torch.zeros(2, 2, Hkv, page, dh, device=DEV)
    st = M.new_status()
    M.medusa_rope_append(None, None, k, k, torch.tensor([0, 6], **i32), torch.tensor([2], **i32),
                         None, M.PagedCache(K, V, torch.tensor([[1]], **i32)), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert torch.equal(K[1, 0, :2], k[4:, 0]) and (K[1, 0, 2:] == 0).all() and (K[0] == 0).all()
