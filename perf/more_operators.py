"""The two forms of latent attention and the ways between them: their cases, plain forms and calls.

A token's keys and values are one latent vector c (512 values) and 64 rotary values that all heads share; a layer's weight
W [H, Dn + Dv, 512] makes a head's Dn key values and Dv values of it. Five operators: reading rows of the paged FP8 cache
back, expanding latents into keys and values, attention over them (the expanded form, for prompts), taking queries into the
latent space and outputs out of it (the absorbed form, for single tokens). ``run`` computes them in plain torch operations,
or with ``own`` through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE, LATENT, ROPE, ROW = 64, 512, 64, 656
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases ------------------
def listed():
    return [
        # the cached prompts of a handful of chats, read back for the expanded form
        {"name": "read few", "op": "read", "B": 8, "kv_lo": 200, "kv_hi": 2000, "skip": False, "dtype": "bf16", "shape": 1},
        # long contexts, a later part of each, kept in 32 bits for a check of the quantisation
        {"name": "read long", "op": "read", "B": 5, "kv_lo": 30000, "kv_hi": 131072, "skip": True, "dtype": "fp32", "shape": 2},
        # queries of a speculative decode step (64 requests x 4 tokens)
        {"name": "absorb decode", "op": "absorb", "T": 256, "H": 64, "Dn": 128, "Dv": 128},
        # the queries of a long prompt's chunks, taken at once
        {"name": "absorb chunk", "op": "absorb", "T": 16384, "H": 64, "Dn": 128, "Dv": 128},
        # outputs of a decode step, one token of each request
        {"name": "project decode", "op": "project", "T": 64, "H": 64, "Dn": 128, "Dv": 128},
        # outputs of an odd number of prompt tokens, wide heads
        {"name": "project chunk", "op": "project", "T": 4099, "H": 128, "Dn": 192, "Dv": 256},
        # a short prompt's keys and values, a tensor-parallel share of the heads, wide heads
        {"name": "expand short", "op": "expand", "N": 1501, "H": 16, "Dn": 192, "Dv": 256},
        # the keys and values of a 32,768-token context
        {"name": "expand long", "op": "expand", "N": 32768, "H": 64, "Dn": 128, "Dv": 128},
        # a handful of chats, one token each, short contexts: latency
        {"name": "attend few", "op": "attend", "B": 8, "q_lo": 1, "q_hi": 1, "kv_lo": 200, "kv_hi": 2000, "H": 64, "Dn": 128, "Dv": 128, "shape": 9},
        # requests of very different lengths in one batch, some without new tokens, wide heads
        {"name": "attend ragged", "op": "attend", "B": 9, "q_lo": 0, "q_hi": 1500, "kv_lo": 1, "kv_hi": 9000, "H": 16, "Dn": 192, "Dv": 256, "shape": 10},
        # a whole prompt attends to itself
        {"name": "attend prompt", "op": "attend", "B": 1, "q_lo": 8192, "q_hi": 8192, "kv_lo": 8192, "kv_hi": 8192, "H": 64, "Dn": 128, "Dv": 128, "shape": 11},
        # a prefill chunk after 30,720 cached tokens
        {"name": "attend chunk", "op": "attend", "B": 1, "q_lo": 2048, "q_hi": 2048, "kv_lo": 32768, "kv_hi": 32768, "H": 64, "Dn": 128, "Dv": 128, "shape": 12},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["read", "absorb", "project", "expand", "attend", "attend", "attend"])
    Dn, Dv = rng.choice([(128, 128), (128, 128), (192, 256)])
    H = rng.choice([1, 5, 8, 16, 24, 64, 64, 128])
    if op == "read":
        hi = _log(rng, 1, 131072)
        return {"op": op, "B": _log(rng, 1, 5 if hi > 20000 else 64), "kv_lo": rng.randint(1, hi), "kv_hi": hi, "skip": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "shape": rng.randrange(10 ** 6)}
    if op in ("absorb", "project"):
        if rng.random() < 0.3:
            Dn, Dv = rng.choice([64, 128, 192, 256]), rng.choice([64, 128, 192, 256])
        return {"op": op, "T": _log(rng, 1, 16384 * 64 * 640 // (H * (LATENT + max(Dn, Dv))) if H >= 64 else 16384), "H": H, "Dn": Dn, "Dv": Dv}
    if op == "expand":
        if rng.random() < 0.3:
            Dn, Dv = rng.choice([64, 128, 192, 256]), rng.choice([64, 128, 192, 256])
        return {"op": op, "N": _log(rng, 1, min(32768, 32768 * 64 * 256 // (H * (Dn + Dv)))), "H": H, "Dn": Dn, "Dv": Dv}
    while True:
        q_hi = rng.choice([1, _log(rng, 2, 16), _log(rng, 17, 8192), _log(rng, 17, 2048)])
        q_lo = q_hi if rng.random() < 0.5 else rng.randint(0, q_hi)
        kv_hi = _log(rng, q_hi, 65536)
        case = {"op": op, "B": _log(rng, 1, 64), "q_lo": q_lo, "q_hi": q_hi, "kv_lo": rng.randint(max(1, min(kv_hi, q_hi // 2)), kv_hi),
                "kv_hi": kv_hi, "H": H, "Dn": Dn, "Dv": Dv, "shape": rng.randrange(10 ** 6)}
        # what the padded plain form holds: logits and rows, in 32 bits
        padded = case["B"] * kv_hi * H * (q_hi + 3 * (Dn + Dv + 2 * ROPE))
        if padded <= 64 * 2048 * 32768 and sum(_lens(case)[0]) > 0 and work(case)["flops"] <= 2.7e12:
            return case


# ------------------------------------------------------------------ sizes ------------------
def _lens(case):
    """New tokens and rows (the new tokens' own among them) of each request."""
    r = random.Random(case["shape"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"])]
    if case["q_lo"] != case["q_hi"] and case["B"] > 2:
        q[0], kv[0] = case["q_hi"], max(kv[0], min(case["kv_hi"], case["q_hi"]))  # the largest chunk is there
    return q, kv


def _read_lens(case):
    """Cached rows of each request and the first of them that is read."""
    r = random.Random(case["shape"])
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"])]
    return kv, [r.randrange(k) // 4 if case["skip"] else 0 for k in kv]


def _visible(q, kv):
    """(token, row) pairs that a request's new tokens see: the last token sees all rows."""
    first = kv - q + 1
    return sum(max(0, first + i) for i in range(q))


def work(case):
    op = case["op"]
    if op == "read":
        n = sum(k - f for k, f in zip(*_read_lens(case)))
        return {"bytes": n * (ROW + (LATENT + ROPE) * (4 if case["dtype"] == "fp32" else 2)), "flops": n * LATENT}
    H, Dn, Dv = case["H"], case["Dn"], case["Dv"]
    if op in ("absorb", "project"):
        D = Dn if op == "absorb" else Dv
        return {"bytes": 2 * H * (case["T"] * (D + LATENT) + D * LATENT), "flops": 2 * case["T"] * H * D * LATENT}
    if op == "expand":
        N, width = case["N"], H * (Dn + Dv)
        return {"bytes": 2 * (N * (LATENT + width) + width * LATENT), "flops": 2 * N * LATENT * width}
    q, kv = _lens(case)
    seen = sum(k for t, k in zip(q, kv) if t)
    return {"bytes": 2 * seen * (H * (Dn + Dv) + ROPE) + 2 * sum(q) * H * (Dn + ROPE + Dv) + 4 * sum(q) * H,
            "flops": 2 * H * (Dn + ROPE + Dv) * sum(_visible(t, k) for t, k in zip(q, kv))}


# ------------------------------------------------------------------ inputs -----------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(shape, g, sigma=1.0):
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    return x.normal_(0.0, sigma, generator=g)


def _latent_rows(n, g):
    """`n` cached rows: 512 e4m3 codes, one fp32 scale per 128 of them, 64 bf16 rotary values."""
    rows = torch.empty((n, ROW), dtype=torch.uint8, device="cuda")
    for at in range(0, n, 1 << 20):
        m = min(1 << 20, n - at)
        x = torch.randn((m, 4, 128), generator=g, device="cuda")
        x *= torch.rand((m, 4, 1), generator=g, device="cuda") + 0.5
        scale = x.abs().amax(-1, keepdim=True).div_(448.0).clamp_(min=2.0 ** -14)
        rows[at:at + m, :LATENT] = (x / scale).to(torch.float8_e4m3fn).view(torch.uint8).view(m, LATENT)
        rows[at:at + m, LATENT:LATENT + 16] = scale.view(m, 4).contiguous().view(torch.uint8)
        rows[at:at + m, LATENT + 16:] = torch.randn((m, ROPE), generator=g, device="cuda").bfloat16().view(torch.uint8)
    return rows


def _starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _prepare_read(case, seed):
    g = _gen(seed)
    kv, first = _read_lens(case)
    pages = [-(-k // PAGE) for k in kv]
    nblk = sum(pages) + 3
    order = torch.randperm(nblk, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((len(kv), max(pages) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    lens = [k - f for k, f in zip(kv, first)]
    return {"pool": _latent_rows(nblk * PAGE, g), "table": table, "first": torch.tensor(first, dtype=torch.int32, device="cuda"),
            "start": _starts(lens), "out": torch.empty((sum(lens), LATENT + ROPE), dtype=DTYPES[case["dtype"]], device="cuda")}


def _weights(case, g):
    """Keys and values of size one from latents of size one."""
    return _normal((case["H"], case["Dn"] + case["Dv"], LATENT), g, LATENT ** -0.5)


def _prepare_absorb(case, seed):
    g = _gen(seed)
    T, H, Dn = case["T"], case["H"], case["Dn"]
    # queries come with their rotary part; their place is the latent part of the 576-wide ones
    return {"q": _normal((T, H, Dn + ROPE), g)[..., :Dn], "w": _weights(case, g),
            "out": torch.empty((T, H, LATENT + ROPE), dtype=torch.bfloat16, device="cuda")[..., :LATENT]}


def _prepare_project(case, seed):
    g = _gen(seed)
    T, H, Dv = case["T"], case["H"], case["Dv"]
    return {"x": _normal((T, H, LATENT), g), "w": _weights(case, g), "out": torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda")}


def _prepare_expand(case, seed):
    g = _gen(seed)
    N, H = case["N"], case["H"]
    return {"latent": _normal((N, LATENT + ROPE), g)[:, :LATENT], "w": _weights(case, g),
            "kv": torch.empty((N, H, case["Dn"] + case["Dv"]), dtype=torch.bfloat16, device="cuda")}


def _prepare_attend(case, seed):
    g = _gen(seed)
    q_len, kv_len = _lens(case)
    T, N, H, Dn, Dv = sum(q_len), sum(kv_len), case["H"], case["Dn"], case["Dv"]
    return {"q": _normal((T, H, Dn + ROPE), g, 1.5), "kv": _normal((N, H, Dn + Dv), g), "rope": _normal((N, LATENT + ROPE), g)[:, LATENT:],
            "req_start": _starts(q_len), "kv_start": _starts(kv_len), "scale": (Dn + ROPE) ** -0.5,
            "longest_q": max(q_len), "longest_kv": max(kv_len),
            "out": torch.empty((T, H, Dv), dtype=torch.bfloat16, device="cuda"), "lse": torch.empty((T, H), device="cuda"), "workspace": None}


def prepare(case, seed):
    s = {"read": _prepare_read, "absorb": _prepare_absorb, "project": _prepare_project, "expand": _prepare_expand,
         "attend": _prepare_attend}[case["op"]](case, seed)
    s["case"], s["err"] = case, torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ the cache read back ----
def _run_read(s):
    out = s["out"]
    if own:
        import dsa_sparse_mla_gb300 as hs
        hs.hs_kv_read(s["pool"], s["table"], s["start"], out, s["err"], first=s["first"])
        return out
    i = torch.arange(out.shape[0], device="cuda")
    start = s["start"].long()
    r = torch.searchsorted(start, i, right=True) - 1
    j = s["first"].long()[r] + i - start[r]
    raw = s["pool"][s["table"][r, j // PAGE].long() * PAGE + j % PAGE]
    codes = raw[:, :LATENT].view(torch.float8_e4m3fn).float().view(-1, 4, 128)
    out[:, :LATENT] = (codes * raw[:, LATENT:LATENT + 16].contiguous().view(torch.float32)[..., None]).view(-1, LATENT)
    out[:, LATENT:] = raw[:, LATENT + 16:].contiguous().view(torch.bfloat16)
    return out


# ------------------------------------------------------------------ a head's products ------
def _run_absorb(s):
    if own:
        import dsa_sparse_mla_gb300 as hs
        hs.hs_mla_absorb(s["q"], s["w"], s["out"], s["err"])
    else:
        key = s["w"][:, :s["case"]["Dn"]].float()
        s["out"].copy_(torch.bmm(s["q"].float().transpose(0, 1), key).transpose(0, 1))
    return s["out"]


def _run_project(s):
    if own:
        import dsa_sparse_mla_gb300 as hs
        hs.hs_mla_project(s["x"], s["w"], s["out"], s["err"])
    else:
        value = s["w"][:, s["case"]["Dn"]:].float()
        s["out"].copy_(torch.bmm(s["x"].float().transpose(0, 1), value.transpose(1, 2)).transpose(0, 1))
    return s["out"]


def _run_expand(s):
    if own:
        import dsa_sparse_mla_gb300 as hs
        hs.hs_mla_expand(s["latent"], s["w"], s["kv"], s["err"])
    else:
        s["kv"].copy_((s["latent"].float() @ s["w"].flatten(0, 1).float().T).view(s["kv"].shape))
    return s["kv"]


# ------------------------------------------------------------------ attention --------------
def _run_attend(s):
    Dn = s["case"]["Dn"]
    if own:
        import dsa_sparse_mla_gb300 as hs
        if s["workspace"] is None:  # kept by the caller from call to call
            s["workspace"] = torch.empty(hs.hs_mla_expanded_workspace_size(s["kv_start"].numel() - 1, s["out"].shape[2]), dtype=torch.uint8,
                                         device="cuda")
        hs.hs_mla_expanded_fwd(s["q"], s["kv"], s["rope"], s["req_start"], s["kv_start"], s["scale"], s["out"], s["err"], s["workspace"],
                               lse=s["lse"])
        return s["out"], s["lse"]
    H, Q, K = s["case"]["H"], s["longest_q"], s["longest_kv"]
    q_start, kv_start = s["req_start"].long(), s["kv_start"].long()
    q_len, kv_len = q_start.diff(), kv_start.diff()
    B = q_len.numel()
    # rows and new tokens of every request, padded to the longest; the padding's values are zeros
    j, i = torch.arange(K, device="cuda"), torch.arange(Q, device="cuda")
    there, real = j < kv_len[:, None], i < q_len[:, None]
    row = torch.where(there, kv_start[:-1, None] + j, 0)
    token = torch.where(real, q_start[:-1, None] + i, 0)
    kv = torch.where(there[..., None, None], s["kv"][row], 0)
    rope = torch.where(there[..., None], s["rope"][row], 0)[:, :, None].expand(B, K, H, ROPE)
    key = torch.cat([kv[..., :Dn], rope], -1).float().permute(0, 2, 3, 1).reshape(B * H, Dn + ROPE, K)
    value = kv[..., Dn:].float().permute(0, 2, 1, 3).reshape(B * H, K, -1)
    q = s["q"][token].float().permute(0, 2, 1, 3).reshape(B * H, Q, Dn + ROPE)
    logit = torch.bmm(q, key).mul_(s["scale"]).view(B, H, Q, K)
    seen = torch.where(real, kv_len[:, None] - q_len[:, None] + 1 + i, 0)
    logit.masked_fill_((j >= seen[..., None])[:, None], -math.inf)
    top = logit.amax(-1, keepdim=True)
    safe = torch.where(top == -math.inf, 0.0, top)
    total = logit.sub_(safe).exp_().sum(-1, keepdim=True)
    out = torch.bmm(logit.view(B * H, Q, K), value).view(B, H, Q, -1) / torch.where(total == 0, 1.0, total)
    s["out"].copy_(out.transpose(1, 2)[real])
    s["lse"].copy_((safe + total.log()).squeeze(-1).transpose(1, 2)[real])
    return s["out"], s["lse"]


def run(state):
    return {"read": _run_read, "absorb": _run_absorb, "project": _run_project, "expand": _run_expand, "attend": _run_attend}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits -------------
def _exact_read(case, s):
    start, first, got = s["start"].tolist(), s["first"].tolist(), []
    pages = s["pool"].view(-1, PAGE, ROW)
    for r in range(case["B"]):
        n = first[r] + start[r + 1] - start[r]
        raw = pages[s["table"][r, :-(-n // PAGE)].long()].view(-1, ROW)[first[r]:n]
        scale = raw[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        latent = raw[:, :LATENT].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double() * scale
        got.append(torch.cat([latent, raw[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1))
    return torch.cat(got)


def _exact_attend(case, s):
    H, Dn, q_start, kv_start = case["H"], case["Dn"], s["req_start"].tolist(), s["kv_start"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    for r in range(case["B"]):
        m, n = q_start[r + 1] - q_start[r], kv_start[r + 1] - kv_start[r]
        rope = s["rope"][kv_start[r]:kv_start[r + 1]].double()
        for h in range(H if m else 0):
            kv = s["kv"][kv_start[r]:kv_start[r + 1], h].double()
            for a in range(max(0, m - n), m, 4096):  # tokens that see at least one row
                b = min(m, a + 4096)
                q = s["q"][q_start[r] + a:q_start[r] + b, h].double()
                z = (q[:, :Dn] @ kv[:, :Dn].T + q[:, Dn:] @ rope.T) * s["scale"]
                sees = torch.arange(a, b, device="cuda") + n - m + 1
                z = z.masked_fill(torch.arange(n, device="cuda") >= sees[:, None], -math.inf)
                at = slice(q_start[r] + a, q_start[r] + b)
                lse[at, h] = torch.logsumexp(z, -1)
                out[at, h] = torch.softmax(z, -1) @ kv[:, Dn:]
    return out, lse


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "read":
        return _exact_read(case, s)
    if case["op"] == "absorb":
        return torch.einsum("thd,hdc->thc", s["q"].double(), s["w"][:, :case["Dn"]].double())
    if case["op"] == "project":
        return torch.einsum("thc,hdc->thd", s["x"].double(), s["w"][:, case["Dn"]:].double())
    if case["op"] == "expand":
        return torch.einsum("nc,hdc->nhd", s["latent"].double(), s["w"].double())
    return _exact_attend(case, s)
