"""Plain 64-bit implementations that the rotary, paged-attention and page tests compare with, and their
inputs. Written from the definitions, one request (or page) at a time."""
import math

import numpy as np
import torch

PAGE, LATENT, ROPE, ROW = 64, 512, 64, 656


# ------------------------------------------------------------------ rotary -----------------
def rotate(x, positions, inv_freq, interleaved, scale=1.0, inverse=False):
    """x [T, H, rot] (any type) -> float64, and |a| + |b| of each value's pair."""
    v = x.double().cpu().numpy()
    ang = positions.cpu().numpy().astype(np.float64)[:, None] * inv_freq.cpu().numpy()[None, :]
    c, s = np.cos(ang)[:, None, :] * scale, np.sin(ang)[:, None, :] * scale * (-1.0 if inverse else 1.0)
    half = v.shape[-1] // 2
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    out, mag = np.empty_like(v), np.empty_like(v)
    out[..., ia] = v[..., ia] * c - v[..., ib] * s
    out[..., ib] = v[..., ia] * s + v[..., ib] * c
    mag[..., ia] = mag[..., ib] = np.abs(v[..., ia]) + np.abs(v[..., ib])
    return out, mag


# ------------------------------------------------------------------ cached rows ------------
def make_rows(n, g, sigma=1.0):
    """uint8 [n, 656] on the CPU: 512 e4m3 codes, four different group scales, 64 bf16 values."""
    x = torch.randn((n, 4, 128), generator=g) * sigma * (0.25 + 1.5 * torch.rand((n, 4, 1), generator=g))
    scale = (x.abs().amax(-1, keepdim=True) / 448.0).clamp(min=2.0 ** -14)
    rows = torch.empty((n, ROW), dtype=torch.uint8)
    rows[:, :512] = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(n, 512)
    rows[:, 512:528] = scale.view(n, 4).contiguous().view(torch.uint8)
    rows[:, 528:] = (torch.randn((n, 64), generator=g) * sigma).bfloat16().view(torch.uint8)
    return rows


def read_rows(rows):
    """uint8 [n, 656] -> latent float64 [n, 512], rope float64 [n, 64]."""
    codes = rows[:, :512].contiguous().view(torch.float8_e4m3fn).to(torch.float32).double()
    scale = rows[:, 512:528].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    return codes * scale, rows[:, 528:].contiguous().view(torch.bfloat16).double()


def paged_attention(q, pool, table, req_start, seq_len, scale, causal=True):
    """float64 out [T, H, 512], lse [T, H], and two bounds for 16-bit operands: `spread` [T, H, 512] =
    sum_j p_j |v_j|, `delta` [T, H] = the largest possible error of a visible logit when every latent value is
    off by 2^-11 of itself (fp16 rounding) and sums by 2^-18 of their absolute terms."""
    T, H, _ = q.shape
    dev = q.device
    out = torch.zeros((T, H, LATENT), dtype=torch.float64, device=dev)
    spread = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    delta = torch.zeros((T, H), dtype=torch.float64, device=dev)
    start = req_start.tolist()
    for r, n in enumerate(seq_len.tolist()):
        m = start[r + 1] - start[r]
        if m == 0:
            continue
        j = torch.arange(n, device=dev)
        lat, rope = read_rows(pool[table[r].long()[j // PAGE] * PAGE + j % PAGE])
        keys = torch.cat([lat, rope], 1)
        for i in range(m):
            t = start[r] + i
            see = max(0, n - m + 1 + i) if causal else n
            if see == 0:
                continue
            z = q[t].double() @ keys[:see].T * scale
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            s = p.sum(-1, keepdim=True)
            p = p / s
            out[t] = p @ lat[:see]
            spread[t] = p @ lat[:see].abs()
            lse[t] = (top + torch.log(s))[:, 0]
            terms = q[t].double().abs() @ keys[:see].abs().T * abs(scale)
            delta[t] = (terms * (2.0 ** -11 + 2.0 ** -18)).amax(-1)
    return out, lse, spread, delta


def attention_bound(out, spread, delta, lse):
    """Elementwise bounds: the result rounded to bf16 (2^-8 of itself), P and V rounded to fp16 (2^-11 each), each
    softmax weight off by e^(2 delta) - 1, fp32 sums (2^-16), and fp16's smallest step of P (2^-25, next to a
    reference within 2^8 of the largest) for values of the row's size."""
    w = torch.expm1(2 * delta)[..., None] + 2.0 ** -10 + 2.0 ** -16
    tol = out.abs() * 2.0 ** -8 + (spread * w) * (1 + 2.0 ** -8) + spread.amax(-1, keepdim=True) * 2.0 ** -15 + 1e-30
    return tol, delta + 2.0 ** -20 * lse.abs().clamp(min=1.0).nan_to_num(posinf=1.0) + 2.0 ** -16


def make_batch(q_lens, kv_lens, H, seed=0, sigma_q=1.0, extra_pages=3, device="cuda"):
    """A batch over a permuted paged pool; every page slot that holds no token (tails, free pages) is poisoned with NaN
    codes, infinite scales and NaN rotary values, so that a row read past a length shows."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-k // PAGE) for k in kv_lens]
    nblk = sum(pages) + extra_pages
    order = torch.randperm(nblk, generator=g).to(torch.int32)
    pool = torch.full((nblk * PAGE, ROW), 0x7F, dtype=torch.uint8)
    pool[:, 512:528] = torch.full((nblk * PAGE, 4), math.inf).view(torch.uint8)
    pool[:, 528:] = torch.full((nblk * PAGE, 64), math.nan, dtype=torch.bfloat16).view(torch.uint8)
    width = max(pages + [1]) + 1
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    at = 0
    for r, (n, k) in enumerate(zip(pages, kv_lens)):
        table[r, :n] = order[at:at + n]
        j = torch.arange(k)
        if k:
            pool[table[r].long()[j // PAGE] * PAGE + j % PAGE] = make_rows(k, g)
        at += n
    T = sum(q_lens)
    q = (torch.randn((T, H, LATENT + ROPE), generator=g) * sigma_q).bfloat16()
    start = torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)
    return dict(q=q.to(device), pool=pool.to(device), table=table.to(device), req_start=start.to(device),
                seq_len=torch.tensor(kv_lens, dtype=torch.int32).to(device), kv_tokens=sum(kv_lens), scale=1.0 / 24.0)


# ------------------------------------------------------------------ pages ------------------
def copy_rows(layers, src, dst, rows):
    for name in ("pool", "keys", "key_scale"):
        for l in range(layers[name].shape[0]):
            t = layers[name][l].reshape(-1, PAGE, *layers[name][l].shape[(1 if name == "pool" else 2):])
            t[dst, :rows] = t[src, :rows]


def fork(parent, child, table, seq_len, refcount, layers):
    """In place on numpy arrays; returns src, dst, and whether a page was missing."""
    free = [p for p in range(len(refcount)) if refcount[p] <= 0]
    src, dst = np.full(len(parent), -1, np.int32), np.full(len(parent), -1, np.int32)
    short = False
    before = table.copy(), seq_len.copy()
    for i, (pa, ch) in enumerate(zip(parent, child)):
        n = int(before[1][pa])
        full, tail = divmod(n, PAGE)
        table[ch], seq_len[ch] = -1, 0
        if tail:
            if not free:
                short = True
                continue
            src[i], dst[i] = before[0][pa, full], free.pop(0)
            refcount[dst[i]] = 1
            copy_rows(layers, src[i], dst[i], tail)
            table[ch, full] = dst[i]
        for j in range(full):
            table[ch, j] = before[0][pa, j]
            refcount[before[0][pa, j]] += 1
        seq_len[ch] = n
    return src, dst, short


def free(reqs, table, seq_len, refcount):
    bad = False
    for r in reqs:
        if r < 0:
            continue
        for j in range(-(-int(seq_len[r]) // PAGE)):
            if refcount[table[r, j]] > 0:
                refcount[table[r, j]] -= 1
            else:
                bad = True
        table[r], seq_len[r] = -1, 0
    return bad


def compact(table, refcount, layers):
    n = len(refcount)
    used = [p for p in range(n) if refcount[p] > 0]
    U = len(used)
    movers, holes = [p for p in used if p >= U], [p for p in range(U) if refcount[p] <= 0]
    src, dst = np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    to = {}
    for i, (a, b) in enumerate(zip(movers, holes)):
        src[i], dst[i], to[a] = a, b, b
        refcount[b], refcount[a] = refcount[a], 0
        copy_rows(layers, a, b, PAGE)
    for e in np.ndindex(table.shape):
        table[e] = to.get(int(table[e]), table[e])
    return src, dst, np.array([U, len(movers)], np.int32)
