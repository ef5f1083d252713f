"""GPU: shapes that take the prompt side's kernels for many rows: fp32 chunk
attention with few warps or one to a token, and rows sampled by clusters of
every size with two blocks to a multiprocessor."""
import numpy as np
import pytest
import torch

import speculative_decoding_medusa_b200 as M
from tests import test_gpu_chunk_attention as A

pytestmark = pytest.mark.gpu

DEV = "cuda"
MARGIN = 1e-9  # as in test_gpu_sample_tokens


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# a unit is a token and up to R heads of one kv head; its keys are split over as
# many warps as keep units * warps within 48 to a multiprocessor
@pytest.mark.parametrize("warps", [2, 1])
@pytest.mark.parametrize("Hq,Hkv,dh,R", [(14, 2, 64, 4), (7, 1, 128, 4), (3, 3, 32, 1), (4, 2, 64, 2),
                                         (5, 1, 160, 2), (6, 1, 256, 2)])
def test_fp32_chunks_of_many_tokens(warps, Hq, Hkv, dh, R):
    per = Hkv * -(-(Hq // Hkv) // R)  # units of a token
    T = 48 * _sms() // (2 * warps) // per + 3
    assert T * per * 2 * warps > 48 * _sms() >= T * per * warps or warps == 1
    n = T // 3
    lens = [(n, n + 20), (0, 4), (1, 40), (T - n - 4, T - n - 10), (3, 30)]
    c = A._case(lens, Hq, Hkv, dh, 16, torch.float32, seed=T, pad=2)
    A._check(A._call(*c), *c)


def _reference(z, u, temperature, top_k, top_p, min_p):
    """One row in 64 bits on the GPU: (token, kept, margin), the margin as
    oracle.prompt_oracle.sample_row has it."""
    zs, order = torch.sort(z, descending=True, stable=True)  # ties by ascending id
    n = int((zs > -np.inf).sum())
    if temperature == 0.0 or top_k == 1:
        return int(order[0]), 1, np.inf
    w = ((zs[:n] - zs[0]) / temperature).exp()
    if top_k > 0:
        n = min(n, top_k)
    margin, n_p = np.inf, n
    if top_p < 1.0:
        before = w[:n].cumsum(0) - w[:n]
        total = w[:n].sum()
        stay = before < top_p * total
        stay[0] = True
        n_p = int(stay.sum())
        margin = min([margin] + [float(x) for x in (before[max(1, n_p - 1):n_p + 1]
                                                    - top_p * total).abs() / total])
    if min_p > 0.0:
        if n > 1:
            margin = min(margin, float((w[1:n] - min_p).abs().min()) / min_p)
        n = int((w[:n] >= min_p).sum())
    n = max(1, min(n, n_p))
    kept, at = torch.sort(order[:n])
    cum = w[:n][at].cumsum(0)
    total = cum[-1]
    if n > 1:
        margin = min(margin, float((cum[:-1] - u * total).abs().min() / total))
    i = int((cum <= u * total).sum()) if u > 0.0 else 0
    return int(kept[min(i, n - 1)]), n, margin


CASES = [(torch.bfloat16, 32000, 1), (torch.bfloat16, 60001, 2), (torch.bfloat16, 128256, 4),
         (torch.bfloat16, 200000, 8), (torch.float32, 16000, 1), (torch.float32, 32000, 2),
         (torch.float32, 60001, 4), (torch.float32, 128256, 8)]


@pytest.mark.parametrize("kind", ["", "k", "p", "m", "kp", "mixed"])
@pytest.mark.parametrize("dtype,V,cluster", CASES)
def test_many_rows_in_clusters(dtype, V, cluster, kind):
    R = _sms() // 4 + 9  # more than a quarter: clusters as small as hold a row
    size = 2 if dtype is torch.bfloat16 else 4
    assert V * size <= 65536 * cluster and (cluster == 1 or V * size > 32768 * cluster)
    g = torch.Generator(device=DEV).manual_seed(V + len(kind))
    z = torch.randn(R, V, generator=g, device=DEV) * 2.0
    up = torch.randint(0, V, (R, 40), generator=g, device=DEV)
    z.scatter_add_(1, up, torch.rand(R, 40, generator=g, device=DEV) * 10.0)
    z = z.to(dtype)
    rng = np.random.default_rng(V)
    f = lambda x: torch.tensor(x, dtype=torch.float32, device=DEV)
    u = f(rng.random(R).astype(np.float32).clip(0, 1 - 2.0 ** -24))
    t = f(0.5 + rng.random(R))
    mixed = kind == "mixed"
    k = rng.integers(1, 100, R) if "k" in kind or mixed else np.zeros(R, dtype=np.int64)
    p = 0.7 + 0.29 * rng.random(R) if "p" in kind or mixed else np.ones(R)
    m = 0.002 + 0.1 * rng.random(R) if "m" in kind else np.zeros(R)
    if mixed:
        t[rng.random(R) < 0.1] = 0.0
        k[rng.random(R) < 0.5] = 0
        k[3], k[4] = V // 3, V + 5
        p[rng.random(R) < 0.4] = 1.0
        m[rng.random(R) < 0.6] = 0.0
    k = torch.tensor(k, dtype=torch.int32, device=DEV)
    p, m = f(p), f(m)
    tok, kept = torch.full((2, R), -7, dtype=torch.int32, device=DEV)
    st = M.new_status()
    M.medusa_sample_tokens(z, u, tok, temperature=t, top_k=k, top_p=p, min_p=m, kept=kept,
                           dev_status=st)
    assert int(st.item()) == 0
    clear = 0
    for r in range(R):
        token, n, margin = _reference(z[r].double(), float(u[r]), float(t[r]), int(k[r]),
                                      float(p[r]), float(m[r]))
        if margin > MARGIN:
            clear += 1
            assert (int(tok[r]), int(kept[r])) == (token, n), (r, margin)
    assert clear >= 0.8 * R
    # a row's draw does not depend on the others: the same rows again, backwards
    rows = torch.arange(R - 1, -1, -1, dtype=torch.int32, device=DEV)
    flip = lambda x: x.flip(0).contiguous()
    tok2, kept2 = torch.full((2, R), -7, dtype=torch.int32, device=DEV)
    M.medusa_sample_tokens(z, flip(u), tok2, temperature=flip(t), top_k=flip(k), top_p=flip(p),
                           min_p=flip(m), row_idx=rows, kept=kept2)
    assert torch.equal(tok2.flip(0), tok) and torch.equal(kept2.flip(0), kept)
