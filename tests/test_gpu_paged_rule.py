"""hs_paged_mla_fwd on either side of the rule that chooses its variants (128 and 768 (token, head) rows per request on average),
and each variant on work that is split over the SMs."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain
from test_gpu_paged_mla import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [127, 128, 129, 767, 768, 769])
def test_either_side(T):
    b = plain.make_batch([T], [T + 500], 1, seed=51)
    check(b)
    # the dequantised copy takes 1,152 bytes for every row of whole tiles, and only past 768 rows
    extra = hs.hs_paged_mla_workspace_size(T, 1, 1, b["kv_tokens"]) - hs.hs_paged_mla_workspace_size(1, 1, 1, b["kv_tokens"])
    assert extra == ((b["kv_tokens"] + 128) * 1152 if T > 768 else 0)


@pytest.mark.parametrize("B", [2, 3])
@pytest.mark.parametrize("rows", [128, 129, 768, 769])
def test_either_side_in_batches(B, rows):
    """The same sums of rows over several requests, most of them in one."""
    q = [rows * B - (B - 1)] + [1] * (B - 1)
    check(plain.make_batch(q, [m + 200 for m in q], 1, seed=52))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("low,high,tokens", [(0, 128, [5, 3]), (128, 768, [20, 16]), (768, 1 << 30, [70, 90])])
def test_split_work_has_the_same_bits_each_time(low, high, tokens, causal):
    """Two requests, and one without new tokens, over many tiles: every block is split into parts, joined in their order."""
    b = plain.make_batch([tokens[0], 0, tokens[1]], [20_000, 50, 7000], 16, seed=53)
    assert low * 3 < sum(tokens) * 16 <= high * 3
    want, lse = check(b, causal)
    for _ in range(10):
        out, l, flag = run(b, causal)
        assert flag == 0 and torch.equal(out, want) and torch.equal(l, lse)


@pytest.mark.parametrize("chunk", [40, 400])
def test_single_tokens_and_a_chunk_in_one_batch(chunk):
    check(plain.make_batch([1] * 9 + [chunk] + [1] * 10, [1 + 97 * i for i in range(9)] + [chunk + 600] + [300 - 7 * i for i in range(10)], 16, seed=54))
