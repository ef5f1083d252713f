"""GPU: chunk attention whose tiles and lengths pass 32 bits."""
import pytest
import torch

import speculative_decoding_medusa_b200 as M

pytestmark = pytest.mark.gpu

DEV = "cuda"
i32 = dict(dtype=torch.int32, device=DEV)


def test_more_tiles_than_an_int_counts():
    """1024 sequences of one new token, 1024 heads, 704 pages of one slot: the
    schedule's axis (3 a tile, 8 a segment) is 2.2e9 long."""
    B, H, dh, n, n_pages = 1024, 1024, 64, 704, 900
    assert B * H * (3 * n + 8) > 2 ** 31
    g = torch.Generator(device=DEV).manual_seed(2)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    K, V = torch.randn(2, n_pages, H, 1, dh, generator=g, **bf)
    q = torch.randn(B, H, dh, generator=g, **bf)
    table = torch.randint(0, n_pages, (B, n), generator=g, **i32)
    kv = torch.randint(n - 9, n + 1, (B,), generator=g, **i32)
    out, st = torch.full_like(q, 5.0), M.new_status()
    M.medusa_chunk_attention(q, M.PagedCache(K, V, table), torch.arange(B + 1, **i32), kv, out,
                             dev_status=st)
    assert int(st.item()) == 0
    half = 2.0 ** -8
    for b in range(0, B, 7):  # and with it every block's share of the axis
        ids = table[b, :int(kv[b])].long()
        k, v = K[ids, :, 0].float(), V[ids, :, 0].float()  # [n, H, dh]
        s = (k * q[b].float()).sum(-1) * dh ** -0.5
        p = torch.softmax(s.double(), 0)[..., None]
        ref, absv = (p * v).sum(0), (p * v.abs()).sum(0)
        # as in test_gpu_chunk_attention: fp32 scores here too (below 2^-15 for
        # sums of |q k| / 8 below 20), exponentials 2^-20, weights in bf16, 704 sums
        rel = 2 * 2.0 ** -15 + 2.0 ** -20 + half + n * 2.0 ** -23
        bound = rel * absv
        bound = bound + half * (ref.abs() + bound)
        err = (out[b].double() - ref).abs()
        assert bool((err <= bound).all()), (b, float((err / bound).max()))


@pytest.mark.parametrize("Hkv,slots", [(1, 2 ** 28 + 1), (1024, 2 ** 27)])
def test_schedules_beyond_the_limits_are_refused(Hkv, slots):
    """A sequence of more than 2^28 tiles, and more tiles than the blocks take:
    reported, nothing written.  (A page of one slot is a tile.)"""
    K, V = torch.zeros(2, 1, Hkv, 1, 64, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(1, slots, **i32)
    q = torch.zeros(1, Hkv, 64, dtype=torch.bfloat16, device=DEV)
    out, st = torch.full_like(q, 5.0), M.new_status()
    M.medusa_chunk_attention(q, M.PagedCache(K, V, table), torch.tensor([0, 1], **i32),
                             torch.tensor([slots], **i32), out, dev_status=st)
    assert int(st.item()) == 6
    assert bool((out == 5.0).all())


def test_a_sequence_that_fills_an_int():
    """kv_len = 2^31 - 1 over one page that the table repeats; the keys are all
    alike, so any row is the page's mean.  bf16, an M tile of 128 rows."""
    page = 1 << 20
    n = 2 ** 31 // page
    g = torch.Generator(device=DEV).manual_seed(3)
    K = torch.zeros(1, 1, page, 64, dtype=torch.bfloat16, device=DEV)
    V = torch.ones(1, 1, page, 64, dtype=torch.bfloat16, device=DEV)
    V[0, 0, :, 1] = (torch.arange(page, device=DEV) % 2 * 2).bfloat16()  # 0, 2, 0, 2, ...
    q = torch.randn(2, 128, 64, generator=g, device=DEV).bfloat16()
    out, st = torch.full_like(q, 5.0), M.new_status()
    M.medusa_chunk_attention(q, M.PagedCache(K, V, torch.zeros(1, n, **i32)),
                             torch.tensor([0, 2], **i32),
                             torch.tensor([2 ** 31 - 1], **i32), out, dev_status=st)
    assert int(st.item()) == 0
    # weights of 1: the sums of a piece, 2^31 / 148 slots, are exact below 2^24;
    # merging them is off by some 2^-20, and the output by a rounding of 2^-8
    err = (out.float() - 1.0).abs()
    assert float(err.max()) <= 2.0 ** -8
