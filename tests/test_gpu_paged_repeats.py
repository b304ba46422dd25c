"""hs_paged_mla_fwd's variants for more than 128 rows per request, many short blocks per SM, many times over: what is not ordered
shows as bits that change."""
import pytest
import torch

import plain_ops as plain
from test_gpu_paged_mla import check, run

pytestmark = pytest.mark.gpu


def again_and_again(b, low, high, times=120):
    T, H, _ = b["q"].shape
    B = b["table"].shape[0]
    assert low * B < T * H <= high * B  # the variant that is meant, by rows per request
    want, lse = check(b)
    for _ in range(times):
        out, l, flag = run(b)
        assert flag == 0 and torch.equal(out, want) and torch.equal(l, lse)


# Blocks have 256 rows, 128 in each of two SMs: with 16 heads, requests of at most 8 tokens leave one SM without rows.
@pytest.mark.parametrize("name,low,high,tokens,requests", [("some", 128, 768, [8, 16, 3, 40, 8, 1, 13, 32], 200),
                                                           ("many", 768, 1 << 30, [8, 100, 3, 150, 8, 1, 77, 60], 96)])
def test_blocks_without_rows_in_one_half(name, low, high, tokens, requests):
    q = [tokens[i % len(tokens)] for i in range(requests)]
    kv = [max(m, 3 + (i * 37) % 300) for i, m in enumerate(q)]
    again_and_again(plain.make_batch(q, kv, 16, seed=41), low, high)


@pytest.mark.parametrize("name,low,high,tokens,requests", [("some", 128, 768, [16, 32, 48, 20], 230), ("many", 768, 1 << 30, [64, 48, 120], 96)])
def test_blocks_of_one_tile(name, low, high, tokens, requests):
    """Blocks that end with the tile they begin with, one after the other: every tile's P buffer also passes an output on."""
    q = [tokens[i % len(tokens)] for i in range(requests)]
    again_and_again(plain.make_batch(q, [max(m, 5 + (i * 29) % 124) for i, m in enumerate(q)], 16, seed=42), low, high)
