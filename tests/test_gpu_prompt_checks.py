"""GPU: lengths that the prompt side's calls have to refuse on the device."""
import pytest
import torch

import speculative_decoding_medusa_b200 as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
i32 = dict(dtype=torch.int32, device=DEV)


def _attend(dtype, cu, kv, T=8, max_pages=3, page=16):
    """A call over B = len(kv) sequences; the pools hold every page the tables
    name.  Returns out (5.0 on entry) and the status."""
    B = len(kv)
    g = torch.Generator(device=DEV).manual_seed(1)
    K, V = torch.randn(2, 4, 1, page, 64, generator=g, device=DEV).to(dtype)
    table = (torch.arange(B * max_pages, **i32) % 4).view(B, max_pages)
    q = torch.randn(T, 2, 64, generator=g, device=DEV).to(dtype)
    out, st = torch.full_like(q, 5.0), M.new_status()
    M.medusa_chunk_attention(q, M.PagedCache(K, V, table), torch.tensor(cu, **i32),
                             torch.tensor(kv, **i32), out, dev_status=st)
    torch.cuda.synchronize()
    return out, int(st.item())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cu,kv", [
    ([0, 8, 1, 1], [48, 48, 48]),       # rows of the first land in the empty third
    ([0, 8, 1, 1], [20, 20, 20]),
    ([0, 4, 2, 8], [20, 20, 20]),
    ([0, 8, 8, 7], [20, 20, 20]),       # behind every row
    ([0, 8, 9, 8], [20, 20, 20]),
    ([0, 8, 8], [20, 49]),              # a length of a sequence without new tokens
    ([0, 8, 8], [20, -1]),
    ([0] + [8] * 40 + [3], [9] * 41),   # beyond the first 32 sequences
    ([0] * 40 + [8, 8], [9] * 40 + [49]),
    ([0, 2 ** 31 - 1, 8], [9, 9]), ([0, -2 ** 31, 8], [9, 9])])
def test_bad_lengths_leave_every_row(dtype, cu, kv):
    out, status = _attend(dtype, cu, kv)
    assert status == 6
    assert bool((out == 5.0).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_good_lengths_around_them(dtype):
    """The largest lengths that are in range; empty sequences on both sides."""
    out, status = _attend(dtype, [0, 0, 6, 6, 6], [48, 48, 0, 48])
    assert status == 0
    assert bool((out[6:] == 5.0).all()) and bool(torch.isfinite(out[:6]).all())
    assert not bool((out[:6] == 5.0).any())


@pytest.mark.parametrize("T,rot", [(8, 128), (3000, 128), (8, 34)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_append_refuses_lengths_out_of_order(dtype, T, rot):
    """Rows in front of their sequence or behind its end would reach slots of
    older tokens.  A block per row (8), resident blocks (3000) and a rotation
    that vectors do not divide."""
    Hq, Hkv, dh, page = (16, 4, 128, 16) if dtype is torch.bfloat16 else (8, 2, 128, 16)
    g = torch.Generator(device=DEV).manual_seed(T)
    normal = lambda H: torch.randn(T, H, dh, generator=g, device=DEV).to(dtype)
    q, k, v = normal(Hq), normal(Hkv), normal(Hkv)
    r = M.Rope(rot)
    n = T // page + 40

    def append(cu, kv):
        B = len(kv)
        K, V = torch.full((2, n, Hkv, page, dh), 2.5, dtype=dtype, device=DEV)
        table = (torch.arange(B * n, **i32) % n).view(B, n)
        qo, st = torch.full_like(q, 5.0), M.new_status()
        M.medusa_rope_append(r, q, k, v, torch.tensor(cu, **i32), torch.tensor(kv, **i32), qo,
                             M.PagedCache(K, V, table), dev_status=st)
        torch.cuda.synchronize()
        return K, V, qo, int(st.item())

    for cu in ([0, 5, 3, T], [0, T - 2, 0], [0, T, T + 1], [0, -1, T], [0] + [T] * 40 + [T - 1],
               [0] + [T] * 300 + [1]):
        K, V, qo, status = append(cu, [T + 100] * (len(cu) - 1))
        assert status == 6, cu
        assert bool((K == 2.5).all()) and bool((V == 2.5).all()) and bool((qo == 5.0).all()), cu
    # not from 0: the rows in front are reported and left, the others written
    K, V, qo, status = append([2, T], [T + 100])
    assert status == 6
    assert bool((qo[:2] == 5.0).all()) and bool((qo[2:] != 5.0).any(-1).all())
    flat = V.transpose(1, 2).reshape(-1, Hkv, dh)  # slots in order
    first = T + 100 - (T - 2)
    assert bool((flat[:first] == 2.5).all()) and torch.equal(flat[first:T + 100], v[2:])
    assert bool((flat[T + 100:] == 2.5).all())


@pytest.mark.parametrize("T", [8, 3000])
def test_append_with_the_lowest_length(T):
    """Slots below -2^31: none of the rows has one, which is no error."""
    Hkv, dh, page = 8, 128, 16
    k = torch.randn(T, Hkv, dh, generator=torch.Generator(device=DEV).manual_seed(T),
                    device=DEV).bfloat16()
    K, V = torch.full((2, 4, Hkv, page, dh), 2.5, dtype=torch.bfloat16, device=DEV)
    st = M.new_status()
    M.medusa_rope_append(None, None, k, k, torch.tensor([0, T], **i32),
                         torch.tensor([-2 ** 31 + 3], **i32), None,
                         M.PagedCache(K, V, torch.arange(4, **i32).view(1, 4)), dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((K == 2.5).all()) and bool((V == 2.5).all())
