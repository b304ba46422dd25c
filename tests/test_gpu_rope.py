"""hs_rope against a 64-bit rotation: layouts, types, slices, far positions, in place, two tensors."""
import numpy as np
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain

pytestmark = pytest.mark.gpu

# fp32 angle (rounded to 2^-24 of half a turn: 1.9e-7), sincospi (2 units: 1.2e-7), scale, two products and a
# sum (2^-24 each): 7e-7 of the pair's size, with a margin of less than two
COEF = 1e-6
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}  # half the smallest step


def check(got, x, pos, inv, interleaved, scale=1.0, inverse=False):
    ref, mag = plain.rotate(x, pos, inv, interleaved, scale, inverse)
    err = np.abs(got.double().cpu().numpy() - ref)
    tol = np.abs(ref) * (torch.finfo(x.dtype).eps / 2) + COEF * scale * mag * (1 + torch.finfo(x.dtype).eps) + TINY[x.dtype]
    assert np.all(err <= tol), (err.max(), np.unravel_index(np.argmax(err - tol), err.shape))


def inputs(T, H, rot, dtype, width=None, seed=0, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, H, width or rot), generator=g).to(dtype).cuda()
    pos = torch.randint(0, far, (T,), generator=g, dtype=torch.int32).cuda()
    inv = torch.from_numpy(10000.0 ** (-np.arange(rot // 2) * 2.0 / rot)).cuda()
    return x, pos, inv


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("T,H,rot", [(1, 1, 2), (1, 64, 64), (3, 5, 16), (7, 3, 96), (129, 8, 64), (40, 64, 128), (2, 2, 512), (5, 1, 6),
                                     (2500, 16, 64)])
def test_rotation(T, H, rot, dtype, interleaved):
    x, pos, inv = inputs(T, H, rot, dtype)
    out = torch.empty_like(x)
    hs.hs_rope(x, pos, inv, out=out, interleaved=interleaved, scale=1.25)
    check(out, x, pos, inv, interleaved, 1.25)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("width,off", [(576, 512), (194, 130), (130, 1), (128, 0), (192, 64)])
def test_part_of_a_head_in_place(width, off, interleaved):
    x, pos, inv = inputs(33, 6, 64, torch.bfloat16, width)
    before = x.clone()
    hs.hs_rope(x[..., off:off + 64], pos, inv, interleaved=interleaved)
    check(x[..., off:off + 64], before[..., off:off + 64], pos, inv, interleaved)
    x[..., off:off + 64] = before[..., off:off + 64]
    assert torch.equal(x, before), "values outside the rotary part changed"


def test_queries_and_key_in_one_call_other_strides():
    x, pos, inv = inputs(65, 64, 64, torch.bfloat16)
    xt = x.transpose(0, 1).contiguous().transpose(0, 1)          # heads outermost in memory
    key = inputs(65, 1, 64, torch.bfloat16, seed=3)[0]
    out = torch.zeros((65, 64, 576), dtype=torch.bfloat16, device="cuda")
    key_out = torch.empty_like(key)
    hs.hs_rope(xt, pos, inv, out=out[..., 512:], y=key, y_out=key_out, interleaved=True)
    check(out[..., 512:], x, pos, inv, True)
    check(key_out, key, pos, inv, True)
    assert not out[..., :512].any()


def test_positions_far_and_negative():
    x, _, inv = inputs(6, 2, 64, torch.float32)
    pos = torch.tensor([0, 1, 2 ** 31 - 1, -(2 ** 31), -5, 2 ** 24 + 1], dtype=torch.int32).cuda()
    out = torch.empty_like(x)
    hs.hs_rope(x, pos, inv, out=out)
    # the reference's own product pos * inv_freq is rounded to 2^-53 of up to 2^31
    ref, mag = plain.rotate(x, pos, inv, False)
    err = np.abs(out.double().cpu().numpy() - ref)
    assert np.all(err <= np.abs(ref) * 2.0 ** -24 + (COEF + 2.0 ** -21) * mag)
    assert torch.equal(out[0], x[0])                              # position 0 turns nothing


def test_inverse_undoes_and_matches_the_gradient():
    x, pos, inv = inputs(50, 4, 64, torch.float32)
    y, back = torch.empty_like(x), torch.empty_like(x)
    hs.hs_rope(x, pos, inv, out=y, interleaved=True)
    hs.hs_rope(y, pos, inv, out=back, interleaved=True, inverse=True)
    assert (back - x).abs().max() <= 4 * COEF * x.abs().max() * 2
    # d<y, w>/dx is w turned back: compared with central differences of the 64-bit rotation
    w = torch.randn_like(x)
    grad = torch.empty_like(x)
    hs.hs_rope(w, pos, inv, out=grad, interleaved=True, inverse=True)
    for k in (0, 1, 31, 63):
        e = np.zeros(x.shape)
        e[7, 2, k] = 0.5
        f = [np.sum(plain.rotate(x.double().cpu() + s * torch.from_numpy(e), pos, inv, True)[0] * w.double().cpu().numpy()) for s in (1, -1)]
        assert abs(f[0] - f[1] - float(grad[7, 2, k])) <= 2e-5


def test_stretched_context_matches_its_formula():
    f, s = hs.hs_rope_inv_freq(64, kind="yarn", factor=16.0, original=4096)
    x, pos, _ = inputs(20, 3, 64, torch.bfloat16)
    out = torch.empty_like(x)
    hs.hs_rope(x, pos, f.cuda(), out=out, scale=s)
    check(out, x, pos, f, False, s)


def test_side_stream_graph_and_no_tokens():
    x, pos, inv = inputs(100, 8, 64, torch.bfloat16)
    want, out = torch.empty_like(x), torch.empty_like(x)
    hs.hs_rope(x, pos, inv, out=want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hs.hs_rope(x, pos, inv, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(graph):
        hs.hs_rope(x, pos, inv, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    hs.hs_rope(x[:0], pos[:0], inv, out=out[:0])
