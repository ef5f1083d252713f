"""Performance cases of the operators around the decode-verify step: rotary positions (alone, and
with the write into the cache), attention of a chunk of new tokens over a paged cache, and sampling
from filtered logits.

With ``own`` false every case runs in plain torch operations; with it true through the library's
entry points.  ``exact`` gives the same results from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

_DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    llama = {"hq": 32, "hkv": 8, "dh": 128}
    rope = {"rot": 128, "theta": 500000.0, "layout": "half", "scaling": "llama3"}
    return [
        # the Tiny workload's nine tree nodes, half of each head rotated: a call that is all latency
        {"name": "rope_tiny_tree", "op": "rope", "dtype": "f32", "tokens": 9, "hq": 4, "hkv": 4,
         "dh": 64, "rot": 32, "theta": 10000.0, "layout": "interleaved", "scaling": "linear",
         "start": 128, "inverse": False},
        # the Llama-3-8B step: 8 sequences of 64 tree nodes at long positions
        {"name": "rope_llama3_tree", "op": "rope", "dtype": "bf16", "tokens": 512, "start": 8192,
         "inverse": False, **llama, **rope},
        # a batch of prompts (8192 tokens) rotated and written into 64-slot pages
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "batch": 8, "q_lo": 700,
         "q_hi": 1348, "kv_lo": 2048, "kv_hi": 4096, "page": 64, "lens": 1, **llama, **rope},
        # 32 single tokens written at the end of long dense caches
        {"name": "append_single_tokens", "op": "append", "dtype": "bf16", "batch": 32, "q_lo": 1,
         "q_hi": 1, "kv_lo": 1000, "kv_hi": 2000, "page": 0, "lens": 2, **llama, **rope},
        # one 8192-token prompt from an empty cache (the largest: tensor-core bound)
        {"name": "attention_prompt_8k", "op": "attention", "dtype": "bf16", "batch": 1,
         "q_lo": 8192, "q_hi": 8192, "kv_lo": 8192, "kv_hi": 8192, "page": 64, "lens": 3, **llama},
        # chunks of ragged length over filled pages of 16, as a serving scheduler mixes them
        {"name": "attention_ragged_chunks", "op": "attention", "dtype": "bf16", "batch": 12,
         "q_lo": 1, "q_hi": 600, "kv_lo": 601, "kv_hi": 6000, "page": 16, "lens": 4, **llama},
        # single tokens of the Llama-3-8B batch over the step's own dense cache
        {"name": "attention_single_tokens", "op": "attention", "dtype": "bf16", "batch": 8,
         "q_lo": 1, "q_hi": 1, "kv_lo": 4096, "kv_hi": 8192, "page": 0, "lens": 5, **llama},
        # the long-context batch, one token each (the most bytes)
        {"name": "attention_single_tokens_32k", "op": "attention", "dtype": "bf16", "batch": 32,
         "q_lo": 1, "q_hi": 1, "kv_lo": 30001, "kv_hi": 32768, "page": 128, "lens": 6, **llama},
        # the Tiny workload's prompt, full precision
        {"name": "attention_tiny_prompt", "op": "attention", "dtype": "f32", "batch": 1,
         "q_lo": 128, "q_hi": 128, "kv_lo": 128, "kv_hi": 128, "page": 0, "lens": 7, "hq": 4,
         "hkv": 4, "dh": 64},
        # one row of a 32000-token vocabulary, top-k and top-p
        {"name": "sample_one_row", "op": "sample", "dtype": "f32", "rows": 1, "vocab": 32000,
         "filters": "top_k_top_p"},
        # the root tokens of the Llama-3-8B batch, nucleus only
        {"name": "sample_roots", "op": "sample", "dtype": "bf16", "rows": 8, "vocab": 128256,
         "filters": "top_p"},
        # every node of the batch's trees, each row with settings of its own
        {"name": "sample_tree_rows", "op": "sample", "dtype": "bf16", "rows": 512,
         "vocab": 128256, "filters": "mixed"},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attention", "attention", "sample"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    heads = {"hkv": hkv, "hq": hkv * rng.choice([1, 2, 3, 4, 7, 8]), "dh": rng.choice([64, 128])}
    rope = {"rot": rng.choice([heads["dh"], heads["dh"] // 2, heads["dh"] // 4 + 2]),
            "theta": rng.choice([10000.0, 500000.0]),
            "layout": rng.choice(["half", "interleaved"]),
            "scaling": rng.choice(["none", "linear", "llama3", "yarn"])}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rope":
        return {"op": op, "dtype": dtype, "tokens": _log_int(rng, 1, 8192),
                "start": _log_int(rng, 1, 1000000), "inverse": rng.random() < 0.3,
                **heads, **rope}
    if op == "append":
        batch = _log_int(rng, 1, 32)
        q_hi = _log_int(rng, 1, 8192 // batch)
        q_lo = rng.randint(1, q_hi)
        kv_lo = q_hi + _log_int(rng, 1, 2000)
        return {"op": op, "dtype": dtype, "batch": batch, "q_lo": q_lo, "q_hi": q_hi,
                "kv_lo": kv_lo, "kv_hi": kv_lo + rng.randint(0, 999),
                "page": rng.choice([0, 8, 16, 48, 64, 128, 200]), "lens": rng.randrange(1 << 20),
                **heads, **rope}
    if op == "attention":
        page = rng.choice([0, 8, 16, 48, 64, 128, 200])
        if dtype == "f32":
            batch, q_hi = _log_int(rng, 1, 4), _log_int(rng, 1, 200)
            kv_lo = q_hi + _log_int(rng, 1, 300)
            kv_hi = kv_lo + rng.randint(0, 99)
        elif rng.random() < 0.5:  # single tokens
            batch, q_hi = _log_int(rng, 1, 64), 1
            kv_lo = _log_int(rng, 1, 16384)
            kv_hi = kv_lo + rng.randint(0, kv_lo // 4)
        else:
            batch = _log_int(rng, 1, 8)
            q_hi = _log_int(rng, 2, 4096 // batch)
            kv_lo = q_hi + _log_int(rng, 1, 4096)
            kv_hi = kv_lo + rng.randint(0, 999)
        return {"op": op, "dtype": dtype, "batch": batch, "q_lo": rng.randint(1, q_hi),
                "q_hi": q_hi, "kv_lo": kv_lo, "kv_hi": kv_hi, "page": page,
                "lens": rng.randrange(1 << 20), **heads}
    vocab = _log_int(rng, 50, 200000)
    rows = _log_int(rng, 1, min(512, 60000000 // vocab))
    return {"op": op, "dtype": dtype, "rows": rows, "vocab": vocab,
            "filters": rng.choice(["none", "top_k", "top_p", "min_p", "top_k_top_p", "mixed"])}


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence."""
    r = random.Random(case["lens"])
    return [(r.randint(case["q_lo"], case["q_hi"]), r.randint(case["kv_lo"], case["kv_hi"]))
            for _ in range(case["batch"])]


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * size + 24),
                "flops": 4 * case["rows"] * case["vocab"]}
    q_row, kv_row = case["hq"] * case["dh"], case["hkv"] * case["dh"]
    if case["op"] == "rope":
        t = case["tokens"]
        return {"bytes": 2 * t * (q_row + kv_row) * size + 4 * t,
                "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    lens = _lengths(case)
    t = sum(n for n, _ in lens)
    if case["op"] == "append":
        return {"bytes": 2 * t * (q_row + 2 * kv_row) * size,
                "flops": 3 * t * (case["hq"] + case["hkv"]) * case["rot"]}
    pairs = sum(n * kv - n * (n - 1) // 2 for n, kv in lens)
    return {"bytes": (2 * t * q_row + 2 * sum(kv for _, kv in lens) * kv_row) * size,
            "flops": 4 * pairs * q_row}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _scaling(case):
    kind = case["scaling"]
    return {"none": {}, "linear": {"factor": 4.0},
            "llama3": {"factor": 8.0, "low_freq_factor": 1.0, "high_freq_factor": 4.0,
                       "original_max_position": 8192},
            "yarn": {"factor": 16.0, "original_max_position": 4096}}[kind]


def prepare(case, seed):
    g = torch.Generator(device=_DEV).manual_seed(int(seed) % (1 << 62))
    dt = _TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=_DEV, dtype=dt)

    def ints(lo, hi, n):
        return torch.randint(lo, hi + 1, (n,), generator=g, device=_DEV, dtype=torch.int32)

    st = {"case": case}
    if case["op"] == "sample":
        R, V = case["rows"], case["vocab"]
        # a bell of scores with a few dozen likely tokens above it
        z = torch.randn(R, V, generator=g, device=_DEV) * 2.0
        n_up = min(V, 40)
        up = torch.randint(0, V, (R, n_up), generator=g, device=_DEV)
        z.scatter_add_(1, up, torch.rand(R, n_up, generator=g, device=_DEV) * 10.0)
        st["logits"] = z.to(dt)
        st["u"] = torch.rand(R, generator=g, device=_DEV)
        pick = torch.rand(4, R, generator=g, device=_DEV)
        f = case["filters"]
        mixed = f == "mixed"
        st["temperature"] = 0.5 + pick[0]
        if mixed:
            st["temperature"] = torch.where(pick[0] < 0.1, 0.0, st["temperature"])
        st["top_k"] = ints(1, 100, R) if "top_k" in f or mixed else None
        st["top_p"] = 0.7 + 0.29 * pick[1] if "top_p" in f or mixed else None
        st["min_p"] = 0.002 + 0.1 * pick[2] if "min_p" in f or mixed else None
        if mixed:  # each filter off in a part of the rows
            st["top_k"] = torch.where(pick[1] < 0.5, 0, st["top_k"])
            st["top_p"] = torch.where(pick[2] < 0.4, 1.0, st["top_p"])
            st["min_p"] = torch.where(pick[3] < 0.6, 0.0, st["min_p"])
        st["tokens"] = torch.empty(R, dtype=torch.int32, device=_DEV)
        st["kept"] = torch.empty(R, dtype=torch.int32, device=_DEV)
        if own:
            import speculative_decoding_medusa_b200 as M
            st["status"] = M.new_status()
        return st

    Hq, Hkv, dh = case["hq"], case["hkv"], case["dh"]
    if case["op"] in ("rope", "append") and own:
        import speculative_decoding_medusa_b200 as M
        st["rope"] = M.Rope(case["rot"], theta=case["theta"],
                            interleaved=case["layout"] == "interleaved",
                            scaling=case["scaling"], **_scaling(case))
        st["status"] = M.new_status()
    if case["op"] == "rope":
        T = case["tokens"]
        st["q"], st["k"] = normal(T, Hq, dh), normal(T, Hkv, dh)
        st["positions"] = case["start"] + ints(0, 64, T)
        st["q_out"], st["k_out"] = torch.empty_like(st["q"]), torch.empty_like(st["k"])
        return st

    lens = _lengths(case)
    B, T = len(lens), sum(n for n, _ in lens)
    page = case["page"] or max(kv for _, kv in lens)
    per = [-(-kv // page) for _, kv in lens]
    n_pages = sum(per) if case["page"] else B
    st["K"], st["V"] = normal(n_pages, Hkv, page, dh), normal(n_pages, Hkv, page, dh)
    order = (torch.randperm(n_pages, generator=g, device=_DEV) if case["page"]
             else torch.arange(B, device=_DEV)).to(torch.int32)
    st["table"] = torch.zeros(B, max(per), dtype=torch.int32, device=_DEV)
    rows = torch.repeat_interleave(torch.arange(B), torch.tensor(per)).to(_DEV)
    cols = torch.cat([torch.arange(n) for n in per]).to(_DEV)
    st["table"][rows, cols] = order
    cu = [0]
    for n, _ in lens:
        cu.append(cu[-1] + n)
    st["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=_DEV)
    st["kv_len"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device=_DEV)
    st["max_q"], st["max_kv"] = max(n for n, _ in lens), max(kv for _, kv in lens)
    if case["op"] == "append":
        # the three are slices of one packed projection, as a model's layer gives them
        qkv = normal(T, Hq + 2 * Hkv, dh)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["q_out"] = torch.empty(T, Hq, dh, dtype=dt, device=_DEV)
    else:
        st["q"] = normal(T, Hq, dh)
        st["out"] = torch.empty_like(st["q"])
    if own:
        import speculative_decoding_medusa_b200 as M
        st["cache"] = M.PagedCache(st["K"], st["V"], st["table"])
        st["status"] = M.new_status()
        if case["op"] == "attention":
            st["ws"] = M.workspace(M.medusa_chunk_attention_workspace_size(
                Hq, Hkv, dh, M.MEDUSA_BF16 if dt == torch.bfloat16 else M.MEDUSA_F32))
    return st


# ---------------------------------------------------------------------------
# the passes
# ---------------------------------------------------------------------------
def _inv_freq(case):
    """Rotation frequencies [rot / 2] (64 bits) and the factor on rotated elements."""
    rot, theta, s = case["rot"], case["theta"], _scaling(case)
    i = torch.arange(rot // 2, device=_DEV, dtype=torch.float64)
    f = theta ** (-2.0 * i / rot)
    if case["scaling"] == "linear":
        return f / s["factor"], 1.0
    if case["scaling"] == "llama3":
        lo, hi, o = s["low_freq_factor"], s["high_freq_factor"], s["original_max_position"]
        turns = o * f / (2.0 * math.pi)  # full turns over the original length
        blend = ((turns - lo) / (hi - lo)).clamp(0.0, 1.0)
        return f * (blend + (1.0 - blend) / s["factor"]), 1.0
    if case["scaling"] == "yarn":
        def index(beta):
            return (rot * math.log(s["original_max_position"] / (2.0 * math.pi * beta))
                    / (2.0 * math.log(theta)))
        low, high = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), rot - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        return f / s["factor"] * ramp + f * (1.0 - ramp), 0.1 * math.log(s["factor"]) + 1.0
    return f, 1.0


def _rotate(case, x, positions, inverse):
    f, scale = _inv_freq(case)
    a = positions.double()[:, None] * f  # far positions need 64-bit angles
    c = (a.cos() * scale).float()[:, None, :]
    s = (a.sin() * (-scale if inverse else scale)).float()[:, None, :]
    rot, half = case["rot"], case["rot"] // 2
    y = x.float()
    if case["layout"] == "half":
        x0, x1 = y[..., :half], y[..., half:rot]
        y = torch.cat([x0 * c - x1 * s, x0 * s + x1 * c, y[..., rot:]], dim=-1)
    else:
        x0, x1 = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([x0 * c - x1 * s, x0 * s + x1 * c], dim=-1).flatten(-2)
        y = torch.cat([z, y[..., rot:]], dim=-1)
    return y.to(x.dtype)


def _slots(st):
    """Sequence and cache slot of every new token."""
    cu, kv = st["cu_q"].long(), st["kv_len"].long()
    n = cu[1:] - cu[:-1]
    t = torch.arange(st["q"].shape[0], device=_DEV)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, kv[seq] - n[seq] + t - cu[seq]


def _plain_append(st):
    case = st["case"]
    seq, slot = _slots(st)
    page = st["K"].shape[2]
    ids = st["table"].long()[seq, slot // page]
    st["K"][ids, :, slot % page] = _rotate(case, st["k"], slot, False)
    st["V"][ids, :, slot % page] = st["v"]
    return _rotate(case, st["q"], slot, False), st["K"], st["V"]


def _plain_attention(st):
    """All sequences padded to the longest: one batched product each way."""
    case = st["case"]
    Hq, Hkv, dh = case["hq"], case["hkv"], case["dh"]
    B, mq, mkv = case["batch"], st["max_q"], st["max_kv"]
    n_cols = st["table"].shape[1]
    ids = st["table"].long().reshape(-1)

    def gather(pool):
        x = pool.index_select(0, ids).view(B, n_cols, Hkv, -1, dh).transpose(1, 2)
        return x.reshape(B, Hkv, -1, dh)[:, :, :mkv].float()

    cu, kv = st["cu_q"].long(), st["kv_len"].long()
    n = cu[1:] - cu[:-1]
    seq, slot = _slots(st)
    i = torch.arange(st["q"].shape[0], device=_DEV) - cu[seq]
    q = torch.zeros(B, mq, Hq, dh, device=_DEV)
    q[seq, i] = st["q"].float()
    q = q.view(B, mq, Hkv, Hq // Hkv, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dh)
    s = torch.matmul(q, gather(st["K"]).transpose(2, 3)).mul_(dh ** -0.5)
    s = s.view(B, Hq, mq, mkv)
    last = (kv - n)[:, None] + torch.arange(mq, device=_DEV)
    hidden = torch.arange(mkv, device=_DEV) > last[..., None]
    s.masked_fill_(hidden[:, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    total = s.sum(-1, keepdim=True)
    o = torch.matmul(s.view(B, Hkv, -1, mkv), gather(st["V"])).view(B, Hq, mq, dh) / total
    return o.transpose(1, 2)[seq, i].to(st["q"].dtype)


def _plain_sample(st):
    z, V = st["logits"], st["logits"].shape[1]
    R = z.shape[0]
    greedy = st["temperature"] == 0
    T = torch.where(greedy, 1.0, st["temperature"]).double()[:, None]
    zs, order = torch.sort(z.float(), dim=1, descending=True, stable=True)
    w = ((zs.double() - zs[:, :1].double()) / T).exp_()
    rank = torch.arange(V, device=_DEV)
    keep = torch.ones(R, V, dtype=torch.bool, device=_DEV)
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        keep &= (k <= 0) | (rank < k)
        w.masked_fill_(~keep, 0.0)
    if st["min_p"] is not None:
        floor = st["min_p"].double()[:, None] > w
    if st["top_p"] is not None:
        p = st["top_p"].double()[:, None]
        total = w.cumsum(1)
        keep &= (p >= 1.0) | (total - w < p * total[:, -1:])
    if st["min_p"] is not None:
        keep &= ~floor
    keep[:, 0] = True
    keep &= ~greedy[:, None] | (rank == 0)
    w.masked_fill_(~keep, 0.0)
    # back to token order
    w = torch.zeros_like(w).scatter_(1, order, w).cumsum(1)
    inside = w > st["u"].double()[:, None] * w[:, -1:]
    return inside.byte().argmax(1).to(torch.int32), keep.sum(1).to(torch.int32)


def run(state):
    st = state
    case = st["case"]
    op = case["op"]
    if own:
        import speculative_decoding_medusa_b200 as M
        if op == "rope":
            M.medusa_rope(st["rope"], st["q"], st["k"], st["positions"], st["q_out"], st["k_out"],
                          inverse=case["inverse"])
            return st["q_out"], st["k_out"]
        if op == "append":
            M.medusa_rope_append(st["rope"], st["q"], st["k"], st["v"], st["cu_q"], st["kv_len"],
                                 st["q_out"], st["cache"], dev_status=st["status"])
            return st["q_out"], st["K"], st["V"]
        if op == "attention":
            M.medusa_chunk_attention(st["q"], st["cache"], st["cu_q"], st["kv_len"], st["out"],
                                     ws=st["ws"], dev_status=st["status"])
            return st["out"]
        M.medusa_sample_tokens(st["logits"], st["u"], st["tokens"],
                               temperature=st["temperature"], top_k=st["top_k"],
                               top_p=st["top_p"], min_p=st["min_p"], kept=st["kept"],
                               dev_status=st["status"])
        return st["tokens"], st["kept"]
    if op == "rope":
        return (_rotate(case, st["q"], st["positions"], case["inverse"]),
                _rotate(case, st["k"], st["positions"], case["inverse"]))
    if op == "append":
        return _plain_append(st)
    if op == "attention":
        return _plain_attention(st)
    return _plain_sample(st)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_rotation(case, x, positions, inverse):
    """Each pair as a complex number times s * e^(+-i a)."""
    rot, s = case["rot"], _scaling(case)
    freqs, scale = [], 1.0
    for j in range(rot // 2):
        f = case["theta"] ** (-(2 * j) / rot)
        if case["scaling"] == "linear":
            f /= s["factor"]
        elif case["scaling"] == "llama3":
            length, o = 2 * math.pi / f, s["original_max_position"]
            if length > o / s["low_freq_factor"]:
                f /= s["factor"]
            elif length >= o / s["high_freq_factor"]:
                mix = ((o / length - s["low_freq_factor"])
                       / (s["high_freq_factor"] - s["low_freq_factor"]))
                f = (1 - mix) * f / s["factor"] + mix * f
        elif case["scaling"] == "yarn":
            o, lt = s["original_max_position"], 2 * math.log(case["theta"])
            lo = max(math.floor(rot * math.log(o / (32 * 2 * math.pi)) / lt), 0)
            hi = min(math.ceil(rot * math.log(o / (2 * math.pi)) / lt), rot - 1)
            up = min(max((j - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
            f = up * f / s["factor"] + (1 - up) * f
            scale = 1.0 + 0.1 * math.log(s["factor"])
        freqs.append(-f if inverse else f)
    a = torch.outer(positions.double(), torch.tensor(freqs, dtype=torch.float64, device=_DEV))
    w = torch.polar(torch.full_like(a, scale), a)[:, None, :]
    y = x.double().clone()
    cols = torch.arange(rot // 2, device=_DEV)
    first, second = ((cols, cols + rot // 2) if case["layout"] == "half"
                     else (2 * cols, 2 * cols + 1))
    z = torch.complex(y[..., first], y[..., second]) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return tuple(_exact_rotation(case, st[n], st["positions"], case["inverse"])
                     for n in ("q", "k"))
    if case["op"] == "append":
        cu, kv = st["cu_q"].tolist(), st["kv_len"].tolist()
        pos = torch.cat([torch.arange(kv[b] - (cu[b + 1] - cu[b]), kv[b], device=_DEV)
                         for b in range(len(kv))])
        k, K, V = _exact_rotation(case, st["k"], pos, False), st["K"].double(), st["V"].double()
        page = K.shape[2]
        for b in range(len(kv)):
            at = pos[cu[b]:cu[b + 1]]
            where = st["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
            K[where, :, at % page] = k[cu[b]:cu[b + 1]]
            V[where, :, at % page] = st["v"][cu[b]:cu[b + 1]].double()
        return _exact_rotation(case, st["q"], pos, False), K, V
    if case["op"] == "attention":
        cu, kv = st["cu_q"].tolist(), st["kv_len"].tolist()
        group = case["hq"] // case["hkv"]
        out = torch.empty(st["q"].shape, dtype=torch.float64, device=_DEV)
        for b, length in enumerate(kv):
            n = cu[b + 1] - cu[b]
            pages = st["table"][b, :-(-length // st["K"].shape[2])].long()
            see = (torch.arange(length, device=_DEV)[None]
                   <= torch.arange(length - n, length, device=_DEV)[:, None])
            for h in range(case["hkv"]):
                k = st["K"][pages, h].flatten(0, 1)[:length].double()
                v = st["V"][pages, h].flatten(0, 1)[:length].double()
                for e in range(h * group, (h + 1) * group):
                    s = st["q"][cu[b]:cu[b + 1], e].double() @ k.T / math.sqrt(case["dh"])
                    s[~see] = -math.inf
                    out[cu[b]:cu[b + 1], e] = torch.softmax(s, 1) @ v
        return out
    # sampling, one row at a time: ranks from the pairs (value, -id), then the filters
    V = case["vocab"]
    ids = torch.arange(V, device=_DEV)
    tokens, kept = [], []
    for r in range(case["rows"]):
        z, T = st["logits"][r].double(), float(st["temperature"][r])
        if T == 0.0:
            tokens.append(int(ids[z == z.max()].min()))
            kept.append(1)
            continue
        by = torch.argsort(-z, stable=True)
        p = torch.softmax(z / T, 0)[by]
        n = V
        if st["top_k"] is not None and int(st["top_k"][r]) > 0:
            n = min(n, int(st["top_k"][r]))
        if st["top_p"] is not None and float(st["top_p"][r]) < 1.0:
            mass = torch.cumsum(p[:n], 0)
            before = torch.cat([mass.new_zeros(1), mass[:-1]])
            by_p = int((before < float(st["top_p"][r]) * mass[-1]).sum())
        else:
            by_p = n
        if st["min_p"] is not None:
            n = min(n, int((p >= float(st["min_p"][r]) * p[0]).sum()))
        n = max(1, min(n, by_p))
        mine = torch.sort(by[:n]).values
        mass = torch.cumsum(torch.softmax(z[mine] / T, 0), 0)
        at = int((mass <= float(st["u"][r]) * mass[-1]).sum())
        tokens.append(int(mine[min(at, n - 1)]))
        kept.append(n)
    return (torch.tensor(tokens, dtype=torch.int32, device=_DEV),
            torch.tensor(kept, dtype=torch.int32, device=_DEV))
