"""How hs_mla_expanded_fwd cuts its work: the number of units that its plan makes (the workspace's first value) against the rule, restated
here for requests of one block each."""
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import latent_ops as plain
from test_gpu_latent import err

pytestmark = pytest.mark.gpu
TURNS, END, LEAST = 5, 6, 8  # turns that splitting may make, tiles' time of a unit's end, tiles of a piece


def pieces(blocks, tiles, workers, slots):
    """Pieces per block: what ends first, a unit's end counted, among the choices whose pieces have room."""
    best, n = -(-blocks // workers) * (tiles + END), 1
    if 2 * blocks > TURNS * workers:
        return 1
    for w in range(1, TURNS + 1):
        k = min(w * workers // blocks, tiles // LEAST)
        if k > 1:
            t = -(-tiles // k)
            if blocks * -(-tiles // t) <= slots and w * (t + END) < best:
                best, n = w * (t + END), -(-tiles // t)
    return n


@pytest.mark.parametrize("B,H,tiles", [(120, 1, 100), (117, 1, 100), (67, 1, 800), (29, 3, 60), (1, 16, 470), (8, 16, 31), (50, 4, 9), (4, 300, 20)])
def test_pieces_have_room_and_end_first(B, H, tiles):
    """(120 blocks of 100 tiles: the least time is that of pieces that do not fit, and what fits takes longer than no pieces at all.)"""
    n, D = 128 * tiles, 128
    kv, rope = torch.empty((B * n, H, 2 * D), dtype=torch.bfloat16, device="cuda").normal_(), torch.empty((B * n, 64), dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.empty((B, H, D + 64), dtype=torch.bfloat16, device="cuda").normal_()
    start, kv_start = plain.starts([1] * B).cuda(), plain.starts([n] * B).cuda()
    out, lse, e = torch.empty((B, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((B, H), device="cuda"), err()
    ws = torch.empty(hs.hs_mla_expanded_workspace_size(B, D), dtype=torch.uint8, device="cuda")
    hs.hs_mla_expanded_fwd(q, kv, rope, start, kv_start, 0.07, out, e, ws, lse=lse)
    assert hs.hs_check_flag(e) == 0
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert int(ws[:4].view(torch.int32)) == B * H * pieces(B * H, tiles, sms, 6 * (sms // 2))
    for r in (0, B - 1):
        one = slice(r, r + 1), slice(r * n, (r + 1) * n)
        ref, tol, rlse, ltol = plain.attention(q[one[0]], kv[one[1]], rope[one[1]], plain.starts([1]), plain.starts([n]), D, 0.07)
        assert plain.holds(out[one[0]], ref, tol) and plain.holds(lse[one[0]], rlse, ltol)
