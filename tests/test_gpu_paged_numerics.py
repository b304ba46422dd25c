"""hs_paged_mla_fwd where 16-bit operands run out of range: queries whose latent part is far below their rotary part. Every test
runs in all three variants (by rows per request)."""
import pytest
import plain_ops as plain
from test_gpu_paged_mla import check

pytestmark = pytest.mark.gpu

# New tokens of two requests with 16 heads: at most 128 rows per request on average, at most 768, more.
SIZES = {"few": [2, 3], "some": [9, 12], "many": [60, 40]}


def in_size(size, T, B, H):
    rows = T * H
    return {"few": rows <= 128 * B, "some": 128 * B < rows <= 768 * B, "many": rows > 768 * B}[size]


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("latent", [2.0 ** -20, 2.0 ** -60, 2.0 ** -100, 2.0 ** -107, 2.0 ** -112, 2.0 ** -130])
@pytest.mark.parametrize("scale", [1.0 / 24.0, 0.3])
def test_latent_part_far_below_the_rotary_part(size, latent, scale):
    """The power of two that brings a row's latent values into fp16's range scales its rotary values too: ordinary ones must
    neither overflow nor lose their way back. Ordinary rows stand beside the small ones."""
    b = plain.make_batch(SIZES[size], [300, 130], 16, seed=31, sigma_q=2.0)
    assert in_size(size, sum(SIZES[size]), 2, 16)
    b["q"][:, ::3, :512] = (b["q"][:, ::3, :512].double() * latent).bfloat16()
    assert bool(b["q"][:, ::3, :512].any())
    b["scale"] = scale
    check(b)


@pytest.mark.parametrize("size", list(SIZES))
def test_small_parts_under_a_large_scale(size):
    """Both parts tiny, the softmax scale as large: the logits are of order one and either part shows in them."""
    b = plain.make_batch(SIZES[size], [300, 130], 16, seed=32)
    b["q"][..., :512] = (b["q"][..., :512].double() * 2.0 ** -100).bfloat16()
    b["q"][..., 512:] = (b["q"][..., 512:].double() * 2.0 ** -97).bfloat16()
    b["scale"] = 2.0 ** 96
    check(b)
