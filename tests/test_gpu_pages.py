"""Copying, forking, freeing and compacting pages against sequential plain versions: bit-exact."""
import numpy as np
import pytest
import torch

import dsa_sparse_mla_gb300 as hs
import plain_ops as plain

pytestmark = pytest.mark.gpu


class Cache:
    """A cache of L latent and Li indexer layers and B requests, with its copy on the host."""

    def __init__(self, lens, spare, L=2, Li=1, Di=64, empty=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        pages = [-(-n // 64) for n in lens]
        self.nblk, self.B, self.L, self.Li, self.Di = max(1, sum(pages) + spare), len(lens) + empty, L, Li, Di
        order = torch.randperm(self.nblk, generator=g).to(torch.int32)
        table = torch.full((self.B, max(pages + [1]) + 2), -1, dtype=torch.int32)
        ref = torch.zeros(self.nblk, dtype=torch.int32)
        at = 0
        for r, n in enumerate(pages):
            table[r, :n] = order[at:at + n]
            ref[order[at:at + n].long()] = 1
            at += n
        self.host = {"pool": torch.randint(0, 256, (L, self.nblk * 64, 656), generator=g, dtype=torch.uint8),
                     "keys": torch.randint(0, 256, (Li, self.nblk, 64, Di), generator=g, dtype=torch.uint8),
                     "key_scale": torch.rand((Li, self.nblk, 64), generator=g)}
        self.dev = {k: v.cuda() for k, v in self.host.items()}
        self.host = {k: v.numpy() for k, v in self.host.items()}
        self.table, self.ref = table.cuda(), ref.cuda()
        self.seq = torch.tensor(list(lens) + [0] * empty, dtype=torch.int32).cuda()
        self.h_table, self.h_ref, self.h_seq = table.numpy(), ref.numpy(), self.seq.cpu().numpy()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def layers(self):
        def at(t):
            return torch.tensor([t[i].data_ptr() for i in range(t.shape[0])], dtype=torch.int64, device="cuda")
        return dict(pools=at(self.dev["pool"]), k_caches=at(self.dev["keys"]), k_scales=at(self.dev["key_scale"]), Di=self.Di)

    def same(self):
        for a, b in ((self.table, self.h_table), (self.ref, self.h_ref), (self.seq, self.h_seq)):
            np.testing.assert_array_equal(a.cpu().numpy(), b)
        for k in self.dev:
            assert np.array_equal(self.dev[k].cpu().numpy(), self.host[k]), k

    def flag(self):
        return hs.hs_check_flag(self.err)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def do_fork(c, parent, child):
    src, dst = ints([7] * len(parent)), ints([7] * len(parent))
    hs.hs_kv_fork(ints(parent), ints(child), c.table, c.seq, c.ref, src, dst, c.err, **c.layers())
    s, d, short = plain.fork(parent, child, c.h_table, c.h_seq, c.h_ref, c.host)
    np.testing.assert_array_equal(src.cpu().numpy(), s)
    np.testing.assert_array_equal(dst.cpu().numpy(), d)
    return short


@pytest.mark.parametrize("Li,Di", [(0, 128), (1, 64), (2, 128)])
def test_copy_whole_and_partial_pages(Li, Di):
    c = Cache([500, 70], spare=8, L=3, Li=Li, Di=Di)
    free = np.flatnonzero(c.h_ref == 0)
    used = np.flatnonzero(c.h_ref > 0)
    src, dst, rows = [int(used[0]), int(used[1]), -1, int(used[2]), int(used[3]), 3], [int(free[0]), int(free[1]), 2, int(free[2]), int(free[3]), -1], \
        [64, 1, 64, 0, 37, 64]
    hs.hs_kv_copy_pages(ints(src), ints(dst), c.nblk, c.err, rows=ints(rows), **c.layers())
    for s, d, n in zip(src, dst, rows):
        if s >= 0 and d >= 0:
            plain.copy_rows(c.host, s, d, n)
    hs.hs_kv_copy_pages(ints(src[4:5]), ints([int(free[4])]), c.nblk, c.err, **c.layers())
    plain.copy_rows(c.host, src[4], int(free[4]), 64)
    c.same()
    assert c.flag() == 0


def test_copy_refuses_bad_pages_and_rows():
    c = Cache([130], spare=3)
    hs.hs_kv_copy_pages(ints([c.nblk, 0]), ints([0, c.nblk]), c.nblk, c.err, **c.layers())
    assert c.flag() == hs.FLAGS["BAD_BLOCK"]
    c.err.zero_()
    hs.hs_kv_copy_pages(ints([0, 1]), ints([1, 2]), c.nblk, c.err, rows=ints([65, -1]), **c.layers())
    assert c.flag() == hs.FLAGS["BAD_LENGTH"]
    c.err.zero_()
    lay = c.layers()
    lay["pools"] = lay["pools"] + 4
    lay["k_caches"] = lay["k_caches"] + 8
    hs.hs_kv_copy_pages(ints([0]), ints([1]), c.nblk, c.err, **lay)
    assert c.flag() == hs.FLAGS["BAD_INDEX"]
    c.same()                                                       # nothing was written


@pytest.mark.parametrize("lens,forks,spare", [
    ([1], [0], 1), ([64], [0, 0, 0], 0), ([65, 0, 63], [0, 1, 2, 0], 3), ([1000, 64, 777], [2, 0, 1, 2, 2, 0], 9),
    ([5000 + 13 * i for i in range(40)], [i % 40 for i in range(100)], 130)])
def test_fork_shares_pages_and_copies_the_tail(lens, forks, spare):
    c = Cache(lens, spare, empty=len(forks) + 1)
    child = [len(lens) + 1 + i for i in range(len(forks))][::-1]
    assert not do_fork(c, forks, child)
    assert c.flag() == 0
    c.same()
    # the parents leave; every page they alone held is free again
    gone = sorted(set(forks))
    hs.hs_kv_free(ints(gone + [-1]), c.table, c.seq, c.ref, c.err)
    assert not plain.free(gone, c.h_table, c.h_seq, c.h_ref)
    c.same()
    assert c.flag() == 0


def test_fork_many_over_many_pages():
    """More forks and pages than one pass of the planning block takes."""
    c = Cache([33] * 1500, spare=3000, L=1, Li=0, empty=2600)
    order = np.random.default_rng(1).permutation(2600)
    assert not do_fork(c, [int(i) % 1500 for i in range(2600)], [1500 + int(i) for i in order])
    c.same()
    assert c.flag() == 0


def test_fork_without_free_pages():
    c = Cache([70, 64, 10], spare=2, empty=5)
    assert do_fork(c, [0, 1, 2, 0, 1], [3, 4, 5, 6, 7])            # three tails, two free pages
    assert c.flag() == hs.FLAGS["NO_PAGES"]
    c.same()
    assert c.h_seq[6] == 0 and c.h_seq[4] == 64


def test_fork_refuses_bad_requests():
    c = Cache([70, 64], spare=4, empty=4)
    lay = c.layers()
    src, dst = ints([0, 0, 0, 0]), ints([0, 0, 0, 0])
    hs.hs_kv_fork(ints([0, -1, 6, 1]), ints([6, 3, 4, 1]), c.table, c.seq, c.ref, src, dst, c.err, **lay)
    assert c.flag() == hs.FLAGS["BAD_INDEX"]
    assert src.tolist() == [-1] * 4 and dst.tolist() == [-1] * 4
    c.same()
    c.err.zero_()
    c.seq[0] = c.table.shape[1] * 64 + 1
    hs.hs_kv_fork(ints([0]), ints([3]), c.table, c.seq, c.ref, src[:1], dst[:1], c.err, **lay)
    assert c.flag() == hs.FLAGS["BAD_LENGTH"] and int(c.seq[3]) == 0
    c.err.zero_()
    c.seq[0] = 70
    c.table[0, 1] = c.nblk                                         # the tail's page is none
    ref = c.ref.clone()
    hs.hs_kv_fork(ints([0]), ints([3]), c.table, c.seq, c.ref, src[:1], dst[:1], c.err, **lay)
    assert c.flag() == hs.FLAGS["BAD_BLOCK"] and int(c.seq[3]) == 0 and torch.equal(ref, c.ref)


def test_free_refuses_bad_state():
    c = Cache([70, 64, 200], spare=1)
    ref = c.ref.clone()
    c.ref[c.table[0, 0].long()] = 0
    hs.hs_kv_free(ints([0, 3]), c.table, c.seq, c.ref, c.err)
    assert c.flag() == hs.FLAGS["BAD_STATE"] | hs.FLAGS["BAD_INDEX"]
    ref[torch.from_numpy(c.h_table)[0, :2].long().cuda()] = 0
    assert torch.equal(c.ref, ref) and int(c.seq[0]) == 0
    c.err.zero_()
    c.seq[1] = -1
    c.table[2, 1] = c.nblk
    hs.hs_kv_free(ints([1, 2]), c.table, c.seq, c.ref, c.err)
    assert c.flag() == hs.FLAGS["BAD_LENGTH"] | hs.FLAGS["BAD_BLOCK"]


def do_compact(c, alias=False):
    n = c.nblk
    t2 = c.table if alias else torch.full_like(c.table, 5)
    r2 = c.ref if alias else torch.full_like(c.ref, 5)
    src, dst, counts = ints([5] * n), ints([5] * n), ints([9, 9])
    ws = torch.empty(hs.hs_kv_compact_workspace_size(n), dtype=torch.uint8, device="cuda")
    hs.hs_kv_compact(c.table, c.ref, t2, r2, src, dst, counts, c.err, ws, **c.layers())
    s, d, k = plain.compact(c.h_table, c.h_ref, c.host)
    for a, b in ((src, s), (dst, d), (counts, k)):
        np.testing.assert_array_equal(a.cpu().numpy(), b)
    c.table, c.ref = t2, r2
    c.same()
    assert c.flag() == 0


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("lens,spare", [([], 1), ([1], 0), ([64, 640, 100], 0), ([64, 640, 100], 40), ([130] * 700, 900), ([6000, 70000], 2000)])
def test_compact(lens, spare, alias):
    c = Cache(lens, spare, empty=1)
    if len(lens) > 2:                                              # one request shares another's pages
        do_fork(c, [1], [len(lens)]) if int((c.h_ref == 0).sum()) else None
    do_compact(c, alias)
    do_compact(c, alias)                                           # nothing is left to move
    assert plain.compact(c.h_table, c.h_ref, c.host)[2][1] == 0


def test_compact_tells_of_stray_entries():
    c = Cache([100, 100], spare=20)
    U = int((c.h_ref > 0).sum())
    stray = [p for p in range(U, c.nblk) if c.h_ref[p] == 0][0]
    c.table[0, 3], c.h_table[0, 3] = stray, stray
    c.table[1, 3], c.h_table[1, 3] = c.nblk, c.nblk
    n = c.nblk
    t2, r2, src, dst, counts = torch.empty_like(c.table), torch.empty_like(c.ref), ints([0] * n), ints([0] * n), ints([0, 0])
    ws = torch.empty(hs.hs_kv_compact_workspace_size(n), dtype=torch.uint8, device="cuda")
    hs.hs_kv_compact(c.table, c.ref, t2, r2, src, dst, counts, c.err, ws, **c.layers())
    assert c.flag() == hs.FLAGS["BAD_STATE"] | hs.FLAGS["BAD_BLOCK"]
    plain.compact(c.h_table, c.h_ref, c.host)
    np.testing.assert_array_equal(t2.cpu().numpy(), c.h_table)


def test_far_pages_pass_32_bits():
    """Byte offsets past 2^32: the last pages of a 4.4 GB pool."""
    nblk = 105_000
    pool = torch.zeros((nblk * 64, 656), dtype=torch.uint8, device="cuda")
    a = torch.randint(0, 256, (64, 656), dtype=torch.uint8, device="cuda")
    pool[(nblk - 1) * 64:] = a
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.tensor([pool.data_ptr()], dtype=torch.int64, device="cuda")
    hs.hs_kv_copy_pages(ints([nblk - 1]), ints([nblk - 2]), nblk, err, pools=at)
    assert hs.hs_check_flag(err) == 0
    assert torch.equal(pool[(nblk - 2) * 64:(nblk - 1) * 64], a) and not pool[:(nblk - 2) * 64].any()


def test_tables_only_and_graph():
    c = Cache([70, 200], spare=5, empty=2)
    src, dst = ints([0, 0]), ints([0, 0])
    pa, ch = ints([0, 1]), ints([2, 3])
    start = c.table.clone(), c.seq.clone(), c.ref.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_kv_fork(pa, ch, c.table, c.seq, c.ref, src, dst, c.err)
    for t, s in zip((c.table, c.seq, c.ref), start):
        t.copy_(s)
    graph.replay()
    none = {k: v[:0] for k, v in c.host.items()}
    plain.fork([0, 1], [2, 3], c.h_table, c.h_seq, c.h_ref, none)
    c.same()
    assert c.flag() == 0
