"""hs_sparse_mla_fwd with queries whose latent part is far below their rotary part."""
import numpy as np
import pytest

import oracle
from dsa_sparse_mla_gb300 import inputs
from parity import check_mla
from test_gpu_mla import _rows, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("latent", [2.0 ** -60, 2.0 ** -107, 2.0 ** -112, 2.0 ** -130])
def test_latent_part_far_below_the_rotary_part(latent, split):
    """Scaling a head's row until its latent values fit fp16 must not carry its ordinary rotary values out of range."""
    n, T, H, k = 700, 4, 64, 600
    kv = _rows(n, seed=18)
    x = inputs.Stream(19).sub("q").normal((T, H, 576), sigma=2.0)
    x[:, ::3, :512] *= latent
    q = inputs.bf16_bits(x)
    assert (q[:, ::3, :512] & 0x7FFF).any()
    rng = np.random.default_rng(12)
    idx = np.stack([rng.permutation(n)[:k] for _ in range(T)]).astype(np.int32)
    out, lse, flag = _run(q, kv, idx, 0.3, split=split)
    assert flag == 0
    ref, lref = oracle.sparse_mla(q, kv, idx, 0.3)
    check_mla(out, lse, ref, lref)


def test_small_parts_under_a_large_scale():
    n, T, H, k = 700, 4, 64, 600
    kv = _rows(n, seed=20)
    x = inputs.Stream(21).sub("q").normal((T, H, 576))
    x[..., :512] *= 2.0 ** -100
    x[..., 512:] *= 2.0 ** -97
    q = inputs.bf16_bits(x)
    idx = np.stack([np.random.default_rng(13).permutation(n)[:k] for _ in range(T)]).astype(np.int32)
    out, lse, flag = _run(q, kv, idx, 2.0 ** 96)
    assert flag == 0
    ref, lref = oracle.sparse_mla(q, kv, idx, 2.0 ** 96)
    check_mla(out, lse, ref, lref)
