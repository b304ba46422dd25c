"""Plain 64-bit implementations that the tests of the two forms of latent attention compare with, and their bounds. Written from the
definitions, one request and head at a time."""
import math

import numpy as np
import torch

BF16 = 2.0 ** -8  # half a step, relative


def rand(shape, g, sigma=1.0):
    return (torch.randn(shape, generator=g) * sigma).bfloat16()


def weights(H, Dn, Dv, g):
    return rand((H, Dn + Dv, 512), g, 512 ** -0.5)


def starts(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32)


def product(x, w, spec):
    """float64 einsum and its bound: bf16's rounding, and fp32 sums of K products, each off by 2^-23 of the terms so far at most."""
    ref = torch.einsum(spec, x.double(), w.double())
    terms = torch.einsum(spec, x.double().abs(), w.double().abs())
    K = 512 if spec.endswith("->nhd") or spec.endswith("->thd") else x.shape[-1]
    return ref, ref.abs() * BF16 + terms * (K * 2.0 ** -23 * (1 + BF16)) + 1e-38


def attention(q, kv, rope, req_start, kv_start, Dn, scale, causal=True):
    """float64 out [T, H, Dv], lse [T, H] and their bounds. Logits are off by 2^-23 of their absolute terms for each of the Dn + 64
    products, and by 2^-21 of themselves (scale, exponent's argument); a weight by twice that, 2^-8 (bf16) and 2^-21 (exponential); the
    sums over n rows by n 2^-23 of their terms; the result by 2^-8 of itself (bf16). Tokens see only their rows: the others' values,
    whatever they are, are not touched."""
    T, H, D = q.shape
    Dv, dev = kv.shape[2] - Dn, q.device
    out = torch.zeros((T, H, Dv), dtype=torch.float64, device=dev)
    tol, lse = torch.zeros_like(out), torch.full((T, H), -math.inf, dtype=torch.float64, device=dev)
    ltol = torch.zeros_like(lse)
    a, c = req_start.tolist(), kv_start.tolist()
    for r in range(len(a) - 1):
        m, n = a[r + 1] - a[r], c[r + 1] - c[r]
        for i in range(m):
            see = max(0, n - m + 1 + i) if causal else n
            if see == 0:
                continue
            t, rows = a[r] + i, slice(c[r], c[r] + see)
            k = torch.cat([kv[rows, :, :Dn].double(), rope[rows, None].double().expand(see, H, 64)], -1)
            v = kv[rows, :, Dn:].double()
            z = torch.einsum("hd,nhd->hn", q[t].double(), k) * scale
            delta = torch.einsum("hd,nhd->hn", q[t].double().abs(), k.abs()) * abs(scale) * D * 2.0 ** -23 + z.abs() * 2.0 ** -21
            p = torch.softmax(z, -1)
            lse[t] = torch.logsumexp(z, -1)
            out[t] = torch.einsum("hn,nhd->hd", p, v)
            off = torch.expm1(2 * delta.amax(-1, keepdim=True)) + BF16 + 2.0 ** -21 + see * 2.0 ** -22
            tol[t] = out[t].abs() * BF16 + torch.einsum("hn,nhd->hd", p, v.abs()) * off * (1 + BF16) + 1e-30
            ltol[t] = delta.amax(-1) + 2.0 ** -21 + see * 2.0 ** -23 + lse[t].abs() * 2.0 ** -21
    return out, tol, lse, ltol


def holds(got, ref, tol):
    """Everywhere within its bound; infinities and NaN where the reference has them."""
    got = got.double()
    fine = ref.isfinite()
    same = torch.equal(got.isnan(), ref.isnan()) and torch.equal(got[ref.isinf()], ref[ref.isinf()])
    return same and bool(((got - ref).abs()[fine] <= tol.expand_as(ref)[fine]).all())
