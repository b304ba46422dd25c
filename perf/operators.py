"""The operators around the paged latent cache: their cases, plain forms and calls.

Four operators: rotary positions, attention of new tokens over the paged FP8 cache (MLA in MQA
form), forking and freeing cached requests, and compacting the cache's pages. ``run`` computes
them in plain torch operations, or with ``own`` through the package's entry points.
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
        # rotary: the queries and the shared key of a speculative decode step (64 requests x 4
        # tokens), written into the rotary part of the 576-wide MLA queries
        {"name": "rope decode", "op": "rope", "T": 256, "H": 64, "rot": 64, "x_width": 64, "out_width": 576,
         "interleaved": True, "dtype": "bf16", "far": 65536, "factor": 1.0},
        # a long prefill's chunks taken at once, positions up to a million under a stretched context
        {"name": "rope prefill", "op": "rope", "T": 16384, "H": 64, "rot": 64, "x_width": 192, "out_width": 576,
         "interleaved": True, "dtype": "bf16", "far": 1048576, "factor": 16.0},
        # indexer queries: 64 of 128 dims, half layout, kept in 32 bits for the quantiser that follows
        {"name": "rope indexer", "op": "rope", "T": 2051, "H": 64, "rot": 64, "x_width": 128, "out_width": 128,
         "interleaved": False, "dtype": "fp32", "far": 131072, "factor": 4.0},
        # attention: a handful of chats, one token each, short contexts: latency
        {"name": "attend few short", "op": "attend", "B": 8, "q_lo": 1, "q_hi": 1, "kv_lo": 200, "kv_hi": 2000, "H": 64, "shape": 1},
        # the decode batch of 64 requests with one token and three drafts each
        {"name": "attend drafts", "op": "attend", "B": 64, "q_lo": 4, "q_hi": 4, "kv_lo": 16384, "kv_hi": 65536, "H": 64, "shape": 2},
        # plain decode of 32 requests, one token each, long contexts: the cache is read once
        {"name": "attend decode", "op": "attend", "B": 32, "q_lo": 1, "q_hi": 1, "kv_lo": 30000, "kv_hi": 131072, "H": 64, "shape": 3},
        # requests of very different lengths in one batch, 16 heads, chunks from nothing to hundreds
        {"name": "attend ragged", "op": "attend", "B": 9, "q_lo": 0, "q_hi": 400, "kv_lo": 1, "kv_hi": 9000, "H": 16, "shape": 4},
        # a prefill chunk after 30,720 cached tokens
        {"name": "attend chunk", "op": "attend", "B": 1, "q_lo": 2048, "q_hi": 2048, "kv_lo": 32768, "kv_hi": 32768, "H": 64, "shape": 5},
        # fork: parallel samples of four prompts, their parents released
        {"name": "fork few", "op": "fork", "B": 16, "n": 8, "kv_lo": 100, "kv_hi": 5000, "L": 4, "Li": 1, "Di": 128, "spare": 64, "shape": 6},
        # a wide beam over long contexts and many layers
        {"name": "fork many", "op": "fork", "B": 512, "n": 256, "kv_lo": 1000, "kv_hi": 9000, "L": 24, "Li": 6, "Di": 128, "spare": 700, "shape": 7},
        # compaction after a few requests left
        {"name": "compact some", "op": "compact", "B": 37, "pages": 1500, "used": 1100, "moved": 133, "L": 3, "Li": 1, "Di": 64, "shape": 8},
        # compaction of a badly scattered cache of many layers
        {"name": "compact many", "op": "compact", "B": 300, "pages": 9000, "used": 5000, "moved": 2100, "L": 24, "Li": 6, "Di": 128, "shape": 9},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "attend", "attend", "fork", "compact"])
    if op == "rope":
        rot = rng.choice([16, 32, 64, 64, 64, 96, 128])
        width = rot + rng.choice([0, 0, 32, 64, 128, 130])
        return {"op": op, "T": _log(rng, 1, 8192), "H": rng.choice([1, 3, 8, 16, 32, 64]), "rot": rot, "x_width": width,
                "out_width": rng.choice([rot, rot + 64, rot + 512]), "interleaved": rng.random() < 0.5,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "far": _log(rng, 64, 1048576),
                "factor": rng.choice([1.0, 4.0, 16.0, 40.0])}
    if op == "attend":
        while True:
            q_hi = rng.choice([1, 1, _log(rng, 2, 8), _log(rng, 9, 2048)])
            q_lo = q_hi if rng.random() < 0.5 else rng.randint(0, q_hi)
            kv_hi = _log(rng, max(1, q_hi), 131072)
            case = {"op": op, "B": _log(rng, 1, 64), "q_lo": q_lo, "q_hi": q_hi, "kv_lo": rng.randint(max(1, min(kv_hi, q_hi // 2)), kv_hi),
                    "kv_hi": kv_hi, "H": rng.choice([1, 8, 16, 24, 64, 64, 128]), "shape": rng.randrange(10 ** 6)}
            padded = case["B"] * kv_hi * (2 * q_hi * case["H"] + 1500)
            if case["B"] * kv_hi <= 64 * 65536 and padded <= 8 * 10 ** 9 and sum(_attend_lens(case)[0]) > 0:
                return case
    if op == "fork":
        B = 2 * _log(rng, 1, 128)
        n, hi, L = rng.randint(1, B // 2), _log(rng, 2, 9000), _log(rng, 1, 24)
        return {"op": op, "B": B, "n": n, "kv_lo": rng.randint(1, hi), "kv_hi": hi, "L": L, "Li": rng.randint(0, L), "Di": rng.choice([64, 128]),
                "spare": n + rng.randint(0, 100), "shape": rng.randrange(10 ** 6)}
    pages = _log(rng, 8, 6000)
    used = rng.randint(1, pages)
    return {"op": op, "B": _log(rng, 1, 200), "pages": pages, "used": used, "moved": rng.randint(0, min(used, pages - used)),
            "L": _log(rng, 1, 24), "Li": rng.randint(0, 3), "Di": rng.choice([64, 128]), "shape": rng.randrange(10 ** 6)}


# ------------------------------------------------------------------ sizes ------------------
def _attend_lens(case):
    """New tokens and cached tokens (the new ones among them) of each request."""
    r = random.Random(case["shape"])
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["B"])]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(case["B"])]
    if case["q_lo"] != case["q_hi"] and case["B"] > 2:
        q[0], kv[0] = case["q_hi"], max(kv[0], min(case["kv_hi"], case["q_hi"]))  # the largest chunk is there
    return q, kv


def _fork_lens(case):
    """Cached tokens of the B rows of the table: the second half are the empty rows that children take."""
    r = random.Random(case["shape"])
    half = case["B"] // 2
    lens = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(half)]
    parent = [r.randrange(half) for _ in range(case["n"])]
    return lens, parent


def _visible(q, kv):
    """(token, cached row) pairs that a request's new tokens see: the last token sees all rows."""
    first = kv - q + 1
    return sum(max(0, first + i) for i in range(q))


def work(case):
    if case["op"] == "rope":
        e = 4 if case["dtype"] == "fp32" else 2
        values = case["T"] * (case["H"] + 1) * case["rot"]
        return {"bytes": 2 * values * e + 4 * case["T"] + 4 * case["rot"], "flops": 3 * values}
    if case["op"] == "attend":
        q, kv = _attend_lens(case)
        H = case["H"]
        seen = sum(k for t, k in zip(q, kv) if t)
        return {"bytes": ROW * seen + sum(q) * H * 2 * (LATENT + ROPE + LATENT) + 4 * (seen // PAGE + 2 * case["B"]),
                "flops": 2 * (LATENT + ROPE + LATENT) * H * sum(_visible(t, k) for t, k in zip(q, kv))}
    per_row = ROW * case["L"] + (case["Di"] + 4) * case["Li"]
    if case["op"] == "fork":
        lens, parent = _fork_lens(case)
        tail = sum(lens[p] % PAGE for p in parent)
        pages = sum(-(-lens[p] // PAGE) for p in parent)
        return {"bytes": 2 * tail * per_row + 4 * 6 * pages, "flops": 0}
    return {"bytes": 2 * case["moved"] * PAGE * per_row + 16 * case["pages"] + 8 * case["used"], "flops": 0}


# ------------------------------------------------------------------ inputs -----------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


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


def _inv_freq(rot, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Angle per position of each pair: slow pairs stretched by `factor`, fast ones kept, a ramp between."""
    i = np.arange(rot // 2, dtype=np.float64)
    plain = base ** (-2.0 * i / rot)
    if factor == 1.0:
        return plain, 1.0
    at = [rot * math.log(original / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (fast, slow)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return plain / factor * ramp + plain * (1.0 - ramp), 0.1 * math.log(factor) + 1.0


def _prepare_rope(case, seed):
    g, dt = _gen(seed), DTYPES[case["dtype"]]
    T, H, rot = case["T"], case["H"], case["rot"]
    inv, mscale = _inv_freq(rot, case["factor"])
    return {"x": torch.randn((T, H, case["x_width"]), generator=g, device="cuda").to(dt),
            "key": torch.randn((T, 1, rot), generator=g, device="cuda").to(dt),
            "pos": torch.randint(0, case["far"], (T,), generator=g, device="cuda", dtype=torch.int32),
            "inv_freq": torch.from_numpy(inv).cuda(), "mscale": mscale,
            "out": torch.zeros((T, H, case["out_width"]), dtype=dt, device="cuda"),
            "key_out": torch.zeros((T, 1, rot), dtype=dt, device="cuda")}


def _prepare_attend(case, seed):
    g = _gen(seed)
    q_len, kv_len = _attend_lens(case)
    B, H, T = case["B"], case["H"], sum(q_len)
    pages = [-(-k // PAGE) for k in kv_len]
    nblk = sum(pages) + 3
    order = torch.randperm(nblk, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((B, max(pages) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(pages):
        table[r, :n] = order[at:at + n]
        at += n
    out = torch.empty((T, H, LATENT), dtype=torch.bfloat16, device="cuda")
    return {"q": (2.0 * torch.randn((T, H, LATENT + ROPE), generator=g, device="cuda")).bfloat16(),
            "pool": _latent_rows(nblk * PAGE, g), "table": table, "out": out,
            "req_start": torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device="cuda"),
            "seq_len": torch.tensor(kv_len, dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(LATENT + ROPE),
            "kv_tokens": sum(kv_len), "longest_q": max(q_len), "longest_kv": max(kv_len),
            "err": torch.zeros(1, dtype=torch.int32, device="cuda"), "workspace": None}


def _layers(case, nblk, g):
    """The latent pool of every layer, the indexer keys and their scales, and the layers' addresses."""
    L, Li, Di = case["L"], case["Li"], case["Di"]
    pool = torch.randint(0, 256, (L, nblk * PAGE, ROW), generator=g, device="cuda", dtype=torch.uint8)
    keys = torch.randint(0, 256, (Li, nblk, PAGE, Di), generator=g, device="cuda", dtype=torch.uint8)
    key_scale = torch.rand((Li, nblk, PAGE), generator=g, device="cuda")

    def at(t):
        return torch.tensor([t.data_ptr() + i * t[0].numel() * t.element_size() for i in range(t.shape[0])],
                            dtype=torch.int64, device="cuda")

    return {"pool": pool, "keys": keys, "key_scale": key_scale, "pools_at": at(pool), "keys_at": at(keys),
            "key_scale_at": at(key_scale), "err": torch.zeros(1, dtype=torch.int32, device="cuda")}


def _prepare_fork(case, seed):
    g = _gen(seed)
    lens, parent = _fork_lens(case)
    B, half, n = case["B"], case["B"] // 2, case["n"]
    pages = [-(-k // PAGE) for k in lens]
    nblk = sum(pages) + case["spare"]
    order = torch.randperm(nblk, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((B, max(pages) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, m in enumerate(pages):
        table[r, :m] = order[at:at + m]
        at += m
    refcount = torch.zeros(nblk, dtype=torch.int32, device="cuda")
    refcount[order[:at].long()] = 1
    gone = sorted(set(parent))
    child = (torch.randperm(B - half, generator=g, device="cuda")[:n] + half).to(torch.int32)
    s = _layers(case, nblk, g)
    s.update(table=table, refcount=refcount, child=child, parent=torch.tensor(parent, dtype=torch.int32, device="cuda"),
             gone=torch.tensor(gone, dtype=torch.int32, device="cuda"),
             seq_len=torch.tensor(lens + [0] * (B - half), dtype=torch.int32, device="cuda"),
             src=torch.empty(n, dtype=torch.int32, device="cuda"), dst=torch.empty(n, dtype=torch.int32, device="cuda"))
    return s


def _prepare_compact(case, seed):
    g = _gen(seed)
    N, U, M, B = case["pages"], case["used"], case["moved"], case["B"]
    low = torch.randperm(U, generator=g, device="cuda")[:U - M]
    high = torch.randperm(N - U, generator=g, device="cuda")[:M] + U
    used = torch.cat([low, high])[torch.randperm(U, generator=g, device="cuda")].to(torch.int32)
    width = -(-U // B) + 1
    table = torch.full((B * width,), -1, dtype=torch.int32, device="cuda")
    slot = (torch.arange(U, device="cuda") % B) * width + torch.arange(U, device="cuda") // B
    table[slot] = used
    table[(B - 1) * width + width - 1] = used[0]  # one page is shared by two requests
    refcount = torch.zeros(N, dtype=torch.int32, device="cuda")
    refcount[used.long()] = 1
    refcount[used[0].long()] = 2
    s = _layers(case, N, g)
    s.update(table=table.view(B, width), refcount=refcount, table_out=torch.empty((B, width), dtype=torch.int32, device="cuda"),
             refcount_out=torch.empty(N, dtype=torch.int32, device="cuda"), src=torch.empty(N, dtype=torch.int32, device="cuda"),
             dst=torch.empty(N, dtype=torch.int32, device="cuda"), counts=torch.empty(2, dtype=torch.int32, device="cuda"),
             workspace=torch.empty(4 * (N + N // 1024 + 64), dtype=torch.uint8, device="cuda"))
    return s


def prepare(case, seed):
    s = {"rope": _prepare_rope, "attend": _prepare_attend, "fork": _prepare_fork, "compact": _prepare_compact}[case["op"]](case, seed)
    s["case"] = case
    return s


# ------------------------------------------------------------------ rotary -----------------
def _rotate(x, cos, sin, interleaved):
    x = x.float()
    half = x.shape[-1] // 2
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    pair = (a * cos - b * sin, a * sin + b * cos)
    return torch.stack(pair, -1).flatten(-2) if interleaved else torch.cat(pair, -1)


def _run_rope(s):
    c = s["case"]
    x, out = s["x"][..., c["x_width"] - c["rot"]:], s["out"][..., c["out_width"] - c["rot"]:]
    if own:
        import dsa_sparse_mla_gb300 as hs
        hs.hs_rope(x, s["pos"], s["inv_freq"], out=out, y=s["key"], y_out=s["key_out"], interleaved=c["interleaved"], scale=s["mscale"])
    else:
        angle = (s["pos"].double()[:, None] * s["inv_freq"])[:, None, :]  # far positions: 64 bits
        cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
        out.copy_(_rotate(x, cos, sin, c["interleaved"]))
        s["key_out"].copy_(_rotate(s["key"], cos, sin, c["interleaved"]))
    return out, s["key_out"]


# ------------------------------------------------------------------ attention --------------
def _run_attend(s):
    if own:
        import dsa_sparse_mla_gb300 as hs
        if s["workspace"] is None:  # kept by the caller from call to call
            T, H = s["q"].shape[:2]
            s["workspace"] = torch.empty(hs.hs_paged_mla_workspace_size(T, s["table"].shape[0], H, s["kv_tokens"]),
                                         dtype=torch.uint8, device="cuda")
        hs.hs_paged_mla_fwd(s["q"], s["pool"], s["table"], s["req_start"], s["seq_len"], s["kv_tokens"], s["scale"], s["out"],
                            s["err"], s["workspace"])
        return s["out"]
    H = s["case"]["H"]
    B, Q, K = s["table"].shape[0], s["longest_q"], s["longest_kv"]
    start, kv_len = s["req_start"].long(), s["seq_len"].long()
    q_len = start[1:] - start[:-1]
    # rows of every request, padded to the longest; the padding's values are zeros
    j = torch.arange(K, device="cuda")
    there = j[None, :] < kv_len[:, None]
    row = s["table"].long()[:, j // PAGE].clamp(min=0) * PAGE + j % PAGE
    raw = s["pool"][torch.where(there, row, 0)]
    latent = raw[..., :LATENT].view(torch.float8_e4m3fn).float().view(B, K, 4, 128)
    latent = latent * raw[..., LATENT:LATENT + 16].contiguous().view(torch.float32)[..., None]
    kv = torch.cat([latent.view(B, K, LATENT), raw[..., LATENT + 16:].contiguous().view(torch.bfloat16).float()], -1)
    kv = torch.where(there[..., None], kv, 0.0)
    # new tokens of every request, padded likewise
    i = torch.arange(Q, device="cuda")
    real = i[None, :] < q_len[:, None]
    token = torch.where(real, start[:-1, None] + i, 0)
    seen = torch.where(real, kv_len[:, None] - q_len[:, None] + 1 + i, 0).clamp(min=0)
    q = s["q"][token].float().view(B, Q * H, LATENT + ROPE)
    logit = torch.bmm(q, kv.transpose(1, 2)).mul_(s["scale"]).view(B, Q, H, K)
    logit.masked_fill_((j >= seen[..., None])[:, :, None, :], -math.inf)
    top = logit.amax(-1, keepdim=True)
    logit.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = logit.sum(-1, keepdim=True)
    out = torch.bmm(logit.view(B, Q * H, K), kv[..., :LATENT]).view(B, Q, H, LATENT)
    out = out / torch.where(total == 0, 1.0, total)
    s["out"].copy_(out[real])
    return s["out"]


# ------------------------------------------------------------------ pages ------------------
def _copy_rows(s, src, dst):
    """Rows (page * 64 + place) of every layer's pool and indexer cache."""
    s["pool"][:, dst] = s["pool"][:, src]
    keys, scale = s["keys"].flatten(1, 2), s["key_scale"].flatten(1, 2)
    keys[:, dst] = keys[:, src]
    scale[:, dst] = scale[:, src]


def _run_fork(s):
    table, refcount, seq_len = s["table"].clone(), s["refcount"].clone(), s["seq_len"].clone()
    if own:
        import dsa_sparse_mla_gb300 as hs
        layers = dict(pools=s["pools_at"], k_caches=s["keys_at"], k_scales=s["key_scale_at"], Di=s["case"]["Di"])
        hs.hs_kv_fork(s["parent"], s["child"], table, seq_len, refcount, s["src"], s["dst"], s["err"], **layers)
        hs.hs_kv_free(s["gone"], table, seq_len, refcount, s["err"])
        return table, refcount, seq_len, s["src"], s["dst"], s["pool"], s["keys"], s["key_scale"]
    j = torch.arange(table.shape[1], device="cuda")
    one = torch.ones((), dtype=torch.int32, device="cuda")
    length = seq_len[s["parent"].long()].long()
    full, tail = length // PAGE, length % PAGE
    old = table[s["parent"].long()]
    shared = j[None, :] < full[:, None]
    page_from = old.gather(1, full[:, None])[:, 0]
    free = torch.nonzero(refcount == 0)[:, 0]
    rank = ((tail > 0).cumsum(0) - 1).clamp(min=0)
    page_to = free[rank].to(torch.int32)
    src = torch.where(tail > 0, page_from, -1)
    dst = torch.where(tail > 0, page_to, -1)
    new = torch.where(shared, old, -1)
    new.scatter_(1, full[:, None], dst[:, None])
    table[s["child"].long()] = new
    seq_len[s["child"].long()] = length.to(torch.int32)
    pages = old[shared].long()
    refcount.index_add_(0, pages, one.expand(pages.numel()))
    refcount[dst[dst >= 0].long()] = 1
    place = torch.arange(PAGE, device="cuda")
    copied = place[None, :] < tail[:, None]
    _copy_rows(s, (src[:, None].long() * PAGE + place)[copied], (dst[:, None].long() * PAGE + place)[copied])
    # the parents are released
    gone = s["gone"].long()
    held = (j[None, :] * PAGE) < seq_len[gone].long()[:, None]
    pages = table[gone][held].long()
    refcount.index_add_(0, pages, -one.expand(pages.numel()))
    table[gone] = -1
    seq_len[gone] = 0
    return table, refcount, seq_len, src, dst, s["pool"], s["keys"], s["key_scale"]


def _run_compact(s):
    if own:
        import dsa_sparse_mla_gb300 as hs
        hs.hs_kv_compact(s["table"], s["refcount"], s["table_out"], s["refcount_out"], s["src"], s["dst"], s["counts"], s["err"],
                         s["workspace"], pools=s["pools_at"], k_caches=s["keys_at"], k_scales=s["key_scale_at"], Di=s["case"]["Di"])
        return s["table_out"], s["refcount_out"], s["src"], s["dst"], s["counts"], s["pool"], s["keys"], s["key_scale"]
    refcount, N = s["refcount"], s["refcount"].numel()
    used = refcount > 0
    index = torch.arange(N, device="cuda")
    count = used.sum()
    hole, mover = torch.nonzero(~used & (index < count))[:, 0], torch.nonzero(used & (index >= count))[:, 0]
    to = index.clone()
    to[mover] = hole
    table = s["table"].long()
    table_out = torch.where(table >= 0, to[table.clamp(min=0)], -1).to(torch.int32)
    refcount_out = refcount.clone()
    refcount_out[hole] = refcount[mover]
    refcount_out[mover] = 0
    src, dst = torch.full((2, N), -1, dtype=torch.int32, device="cuda")
    src[:mover.numel()] = mover.to(torch.int32)
    dst[:hole.numel()] = hole.to(torch.int32)
    counts = torch.stack([count, torch.full_like(count, mover.numel())]).to(torch.int32)
    pool = s["pool"].view(s["pool"].shape[0], N, PAGE, ROW)
    pool[:, hole] = pool[:, mover]
    s["keys"][:, hole] = s["keys"][:, mover]
    s["key_scale"][:, hole] = s["key_scale"][:, mover]
    return table_out, refcount_out, src, dst, counts, s["pool"], s["keys"], s["key_scale"]


def run(state):
    return {"rope": _run_rope, "attend": _run_attend, "fork": _run_fork, "compact": _run_compact}[state["case"]["op"]](state)


# ------------------------------------------------------------------ in 64 bits -------------
def exact(case, seed):
    if case["op"] == "rope":
        s = prepare(case, seed)
        turn = torch.exp(1j * s["pos"].double()[:, None, None] * s["inv_freq"]) * s["mscale"]
        got = []
        for v in (s["x"][..., case["x_width"] - case["rot"]:], s["key"]):
            v = v.double()
            if case["interleaved"]:
                z = torch.view_as_complex(v.unflatten(-1, (-1, 2)).contiguous()) * turn
                got.append(torch.view_as_real(z).flatten(-2))
            else:
                z = torch.complex(*v.chunk(2, -1)) * turn
                got.append(torch.cat([z.real, z.imag], -1))
        return tuple(got)
    if case["op"] != "attend" or work(case)["flops"] > 2.5e12:
        return None
    s = prepare(case, seed)
    H, start = case["H"], s["req_start"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    for r, n in enumerate(s["seq_len"].tolist()):
        m = start[r + 1] - start[r]
        pages = s["table"][r, :-(-n // PAGE)].long()
        raw = s["pool"].view(-1, PAGE, ROW)[pages].view(-1, ROW)[:n]
        scale = raw[:, LATENT:LATENT + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
        latent = raw[:, :LATENT].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double() * scale
        rows = torch.cat([latent, raw[:, LATENT + 16:].contiguous().view(torch.bfloat16).double()], 1)
        step = max(1, (1 << 28) // (H * n))
        for a in range(0, m, step):
            b = min(m, a + step)
            q = s["q"][start[r] + a:start[r] + b].double().reshape((b - a) * H, -1)
            z = (q @ rows.T * s["scale"]).view(b - a, H, n)
            sees = torch.arange(a, b, device="cuda") + n - m + 1
            z = z.masked_fill(torch.arange(n, device="cuda") >= sees[:, None, None], -math.inf)
            p = torch.where(sees[:, None, None] > 0, torch.softmax(z, -1), 0.0)
            out[start[r] + a:start[r] + b] = (p.view(-1, n) @ latent).view(b - a, H, LATENT)
    return out
