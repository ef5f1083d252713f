"""GPU: tokens sampled from filtered logits against the fp64 oracle.

Decisions are compared wherever the oracle's margin exceeds MARGIN: weights
are within 2^-43 of the largest (rounding) and 2^-40 relative (exponent and
exponential), so masses of a row of V tokens are within V * 2^-43 + 2^-40 of
the oracle's relative to the total: below 2^-25 at V = 2^18, and typically far
less, the roundings being unbiased."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from oracle import prompt_oracle as P
from tests.helpers import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
MARGIN = 1e-9


def _run(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, row_idx=None, want=0):
    R = len(u)
    f = lambda x: None if x is None else torch.tensor(x, dtype=torch.float32, device=DEV)
    i = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)
    tok, kept = torch.full((2, R), -7, dtype=torch.int32, device=DEV)
    st = M.new_status()
    M.medusa_sample_tokens(logits if logits.is_cuda else logits.to(DEV), f(u), tok,
                           temperature=f(temperature), top_k=i(top_k), top_p=f(top_p),
                           min_p=f(min_p), row_idx=i(row_idx), kept=kept, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == want
    return tok.tolist(), kept.tolist()


def _compare(logits, u, temperature=None, top_k=None, top_p=None, min_p=None, least=0.9):
    R = len(u)
    tok, kept = _run(logits, u, temperature, top_k, top_p, min_p)
    z = f64(logits)
    r32 = lambda x, d: float(np.float32(x)) if x is not None else d
    clear = 0
    for r in range(R):
        ref = P.sample_row(z[r], r32(u[r], 0), r32(temperature and temperature[r], 1.0),
                           top_k[r] if top_k else 0, r32(top_p and top_p[r], 1.0),
                           r32(min_p and min_p[r], 0.0))
        if ref[2] > MARGIN:
            clear += 1
            assert (tok[r], kept[r]) == ref[:2], (r, tok[r], kept[r], ref)
    assert clear >= least * R


def _settings(kind, R, rng):
    t = (0.4 + 1.2 * rng.random(R)).tolist()
    k = rng.integers(1, 80, R).tolist() if "k" in kind else None
    p = (0.3 + 0.69 * rng.random(R)).tolist() if "p" in kind else None
    m = (0.001 + 0.2 * rng.random(R)).tolist() if "m" in kind else None
    return dict(temperature=t, top_k=k, top_p=p, min_p=m)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("kind", ["", "k", "p", "m", "kp", "kpm"])
@pytest.mark.parametrize("V", [1, 2, 7, 50, 1000, 4097, 32000])
def test_matches_the_oracle(dtype, kind, V):
    R = 6
    rng = np.random.default_rng(V)
    z = torch.from_numpy(rng.standard_normal((R, V)) * 2.5).to(dtype)
    _compare(z, rng.random(R).tolist(), **_settings(kind, R, rng), least=0.8)


@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, 128256), (torch.float32, 128257),
                                     (torch.float32, 327680), (torch.bfloat16, 655360)])
def test_large_vocabularies(dtype, V):
    R = 3
    rng = np.random.default_rng(V)
    z = torch.from_numpy(rng.standard_normal((R, V)) * 3).to(dtype)
    _compare(z, rng.random(R).tolist(), top_p=[0.5, 0.95, 1.0], top_k=[0, 0, 40], least=0.3)


def test_flat_rows_and_ties():
    """Equal logits: the lowest ids stay, and the draw is uniform over them.
    top_p of n equal tokens keeps ceil(n p)."""
    for dtype in (torch.bfloat16, torch.float32):
        for V in (8, 1000, 20000, 100000):
            z = torch.full((5, V), -3.25).to(dtype)
            u = [0.0, 0.5, 0.75, 1 - 2.0 ** -24, 0.125]
            tok, kept = _run(z, u)
            assert kept == [V] * 5
            assert tok == [int(x * V) for x in u]
            tok, kept = _run(z, u, top_k=[5, 6, 7, 8, 4])
            assert kept == [5, 6, 7, 8 if V > 8 else V, 4]
            assert tok == [int(x * n) for x, n in zip(u, kept)]
            tok, kept = _run(z, u, top_p=[0.5, 0.25, 0.75, 0.0, 2.0 ** -20])
            assert kept == [V // 2, V // 4, 3 * V // 4, 1, 1]
            assert tok == [int(x * n) for x, n in zip(u, kept)]


def test_the_longest_row_of_one_value():
    """Every count of a block in one bin."""
    for dtype, V in ((torch.bfloat16, 655360), (torch.float32, 327680)):
        z = torch.full((3, V), 1.5).to(dtype)
        assert _run(z, [0.5, 0.25, 0.875], top_p=[1.0, 0.5, 0.25]) == (
            [V // 2, V // 8, 7 * V // 32], [V, V // 2, V // 4])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_distinct_values(dtype):
    """Crowded bins: a handful of values over a large vocabulary, cuts inside
    the ties of one value; -0 ties with +0."""
    V, R = 60000, 8
    rng = np.random.default_rng(3)
    vals = np.array([1.0, 0.0, -0.0, 0.5, -2.0])
    z = torch.from_numpy(rng.choice(vals, (R, V))).to(dtype)
    u = rng.random(R).tolist()
    _compare(z, u, top_k=[1, 2, 11000, 13000, 30000, 47000, 59999, 60000], least=0.9)
    _compare(z, u, top_p=[0.05, 0.2, 0.4, 0.6, 0.8, 0.9, 0.99, 0.999], least=0.9)


def test_values_closer_than_a_bin():
    """fp32 logits 1 ulp apart around 1: every level of the key refinement."""
    V, R = 30000, 6
    rng = np.random.default_rng(4)
    z = torch.from_numpy((1.0 + rng.integers(0, 4000, (R, V)) * 2.0 ** -23).astype(np.float32))
    z[:, 17] = 30.0  # and a far leader, so that all of them share one bin
    z[3:, 17] = 1.0
    u = rng.random(R).tolist()
    _compare(z, u, top_k=[2, 100, 15000, 3, 700, 29999], temperature=[9.0] * R, least=0.9)
    _compare(z, u, top_p=[0.1, 0.5, 0.99, 0.3, 0.7, 0.9], temperature=[20.0] * R, least=0.9)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_at_the_end_of_a_stretch(dtype):
    """Zeros (of both signs) as the smallest of the tokens looked at: as the
    lowest of the top tokens, and of a crowded bin."""
    V, R = 20000, 4
    rng = np.random.default_rng(9)
    z = np.where(rng.random((R, V)) < 0.5, 0.0, -0.0)
    z[:, ::200] = 1 + rng.random((R, V // 200))  # a hundred positive tokens
    u = rng.random(R).tolist()
    _compare(torch.from_numpy(z).to(dtype), u, top_k=[90, 101, 200, 256])
    _compare(torch.from_numpy(z).to(dtype), u, top_p=[0.01, 0.03, 0.05, 0.5])
    z[:, ::3] = 1e-3 * rng.random((R, len(z[0, ::3])))  # a third just above zero
    z[:, 5] = 6.0
    _compare(torch.from_numpy(z).to(dtype), u, top_k=[300, 6000, 9000, 15000])
    _compare(torch.from_numpy(z).to(dtype), u, top_p=[0.1, 0.4, 0.6, 0.9])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_magnitudes_far_apart(dtype):
    """Logits from 1e-6 to 8 of both signs, cuts among the smallest; tokens far
    below any weight that a count or a tiny min_p still keeps."""
    V, R = 9000, 6
    rng = np.random.default_rng(10)
    z = 10.0 ** rng.uniform(-6, 0.9, (R, V)) * rng.choice([-1.0, 1.0], (R, V))
    z = torch.from_numpy(z).to(dtype)
    u = [0.0] + rng.random(R - 1).tolist()
    _compare(z, u, top_k=[4500, 4400, 4600, 3900, 8000, 1000])
    _compare(z, u, top_p=[0.9, 0.93, 0.95, 0.97, 0.5, 0.99], temperature=[2.0] * R)
    _compare(z, u, min_p=[0.02, 0.0183, 0.019, 0.3, 1e-30, 1.0], temperature=[2.0] * R, least=0.6)
    _compare(z, u, temperature=[200.0] * R, top_p=[0.3, 0.5, 0.6, 0.7, 0.9, 1.0])
    far = torch.full((R, V), -1000.0).to(dtype)
    far[:, 7:4000:100] = z[:, :40]
    far[:, 9::50] = -60.0
    _compare(far, u, top_k=[20, 40, 41, 100, 2000, 8999])
    _compare(far, u, top_p=[0.5, 0.9, 0.99, 1.0, 1.0, 1.0], min_p=[0.0, 0.0, 0.0, 0.0, 1e-30, 1e-35],
             least=0.5)


def test_masked_and_extreme_logits():
    """-inf and the types' lowest values: never drawn / no mass; temperatures
    far from one; a single finite logit."""
    V = 5000
    rng = np.random.default_rng(5)
    for dtype in (torch.bfloat16, torch.float32):
        z = torch.from_numpy(rng.standard_normal((6, V)) * 4).to(dtype)
        hide = torch.from_numpy(rng.random((6, V)) < 0.7)
        z[:3][hide[:3]] = -math.inf
        z[3:][hide[3:]] = torch.finfo(dtype).min
        u = rng.random(6).tolist()
        _compare(z, u, top_p=[0.9] * 6, top_k=[0, 50, 4000, 0, 50, 4000])
        _compare(z, u, temperature=[1e-3, 100.0, 1e-30, 1e-3, 50.0, 1e30])
        one = torch.full((2, V), -math.inf, dtype=dtype)
        one[0, 4321] = -7.0
        one[1, 0] = torch.finfo(dtype).min
        assert _run(one, [0.3, 0.999], top_p=[0.5, 1.0]) == ([4321, 0], [1, 1])
        top = torch.full((1, V), torch.finfo(dtype).max, dtype=dtype)
        assert _run(top, [0.5]) == ([V // 2], [V])


def test_greedy_and_one_kept():
    z = torch.randn(4, 3000, generator=torch.Generator().manual_seed(1))
    z[1, [5, 900]] = 50.0
    best = [int(x) for x in z.argmax(1)]
    best[1] = 5
    assert _run(z, [0.9] * 4, temperature=[0.0] * 4, top_k=[7] * 4) == (best, [1] * 4)
    assert _run(z, [0.9] * 4, top_k=[1] * 4) == (best, [1] * 4)
    assert _run(z, [0.9] * 4, top_p=[0.0] * 4) == (best, [1] * 4)
    # min_p = 1 keeps the ties of the largest
    tok, kept = _run(z, [0.9] * 4, min_p=[1.0] * 4)
    assert kept == [1, 2, 1, 1] and tok == [best[0], 900, best[2], best[3]]


def test_row_selection_strides_and_alignment():
    """row_idx picks rows (one twice); rows in a wider buffer at every 16-byte
    phase; draws do not depend on the layout."""
    V = 1003
    base = torch.randn(5, V + 40, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    u = [0.1, 0.5, 0.9, 0.5]
    rows = [4, 0, 2, 0]
    base = base.to(DEV)
    for off in range(9):
        view = base[:, off:off + V]
        flat = view.contiguous()[rows]
        want = _run(flat, u, top_p=[0.9] * 4)
        assert _run(view, u, top_p=[0.9] * 4, row_idx=rows) == want
        assert want[0][1] == want[0][3]
    tok, kept = _run(base, u, row_idx=[0, 5, -1, 1], want=6)
    assert tok[1] == tok[2] == -1 and kept[1] == kept[2] == 0 and tok[0] >= 0 and tok[3] >= 0


def test_bad_rows_are_reported():
    z = torch.randn(9, 700, generator=torch.Generator().manual_seed(6))
    z[0, 699] = math.nan
    z[1, 0] = math.inf
    z[2] = -math.inf
    nan = math.nan
    tok, kept = _run(z, [0.5, 0.5, 0.5, 1.0, -0.1, nan, 0.5, 0.5, 0.5],
                     temperature=[1.0] * 6 + [-1.0, 1.0, 1.0], top_p=[1.0] * 7 + [nan, 1.0],
                     min_p=[0.0] * 8 + [1.5], want=6)
    assert tok == [-1] * 9 and kept == [0] * 9


def test_frequencies_follow_the_filtered_distribution():
    z = torch.tensor([0.0, 1.0, 2.0, -1.0, 0.5, 3.0, -2.0, 1.5]).repeat(4000, 1)
    u = ((np.arange(4000) + 0.5) / 4000).tolist()
    tok, kept = _run(z, u, top_k=[4] * 4000)
    assert set(kept) == {4}
    p = np.exp(np.array([1.0, 2.0, 3.0, 1.5]))
    got = np.bincount(tok, minlength=8)[[1, 2, 5, 7]]
    assert np.abs(got - 4000 * p / p.sum()).max() <= 1.0  # a regular grid of u


def test_no_rows_and_repeatable_capture():
    z = torch.randn(3, 40000, device=DEV)
    tok = torch.zeros(3, dtype=torch.int32, device=DEV)
    M.medusa_sample_tokens(z, torch.zeros(0, device=DEV), tok[:0])
    u = torch.rand(3, device=DEV)
    p = torch.full((3,), 0.9, device=DEV)
    M.medusa_sample_tokens(z, u, tok, top_p=p)
    first = tok.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        M.medusa_sample_tokens(z, u, tok, top_p=p)
    for _ in range(3):
        tok.fill_(-1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(tok, first)
