"""Device-side driver of the hot path.

``DeviceWorkload`` moves a seeded ``inputs.Workload`` into GPU memory; ``HotPath`` owns the
intermediate and output buffers and runs one step: hs_indexer_scores -> hs_topk ->
hs_sparse_mla_fwd (logical indices through the paged block table), or for decode batches
hs_indexer_topk -> hs_sparse_mla_fwd; ``SharedSetHotPath`` runs the
indexer and top-k for each request's final query token only and lets the request's other query
tokens reuse that set in hs_sparse_mla_fwd (shared index sets); ``LongPrefillPass`` runs every
chunk of a long prefill through the same three calls. ``DeviceHiSparse`` does the
same for the mixed-residency decode (hs_hisparse_resolve -> hs_sparse_mla_fwd on physical rows),
with the older rows in pinned host memory. ``DenseSession`` runs requests that attend densely and may branch
(hs_rope -> hs_kv_append -> hs_paged_mla_fwd; hs_kv_fork, hs_kv_free and hs_kv_compact between steps), from per-head queries to
per-head outputs in either form of latent attention (hs_mla_absorb -> hs_paged_mla_fwd -> hs_mla_project, or hs_kv_read ->
hs_mla_expand -> hs_mla_expanded_fwd).

Only buffer management lives here; all arithmetic runs in libhs.so.
"""
from __future__ import annotations

import dataclasses
import math

import numpy as np
import torch

from . import (hs_hisparse_resolve, hs_hisparse_touch_host, hs_indexer_scores, hs_indexer_topk, hs_kv_append, hs_kv_compact,
               hs_kv_compact_workspace_size, hs_kv_fork, hs_kv_free, hs_kv_read, hs_mla_absorb, hs_mla_expand, hs_mla_expanded_fwd,
               hs_mla_expanded_workspace_size, hs_mla_project, hs_paged_mla_fwd, hs_paged_mla_workspace_size, hs_rope, hs_rope_inv_freq,
               hs_sparse_mla_fwd, hs_sparse_mla_workspace_size, hs_topk)
from .inputs import HiSparseWorkload, Workload


def _t(a: np.ndarray, device, dtype=None) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(a))
    if dtype is not None:
        t = t.view(dtype)
    return t.to(device)


@dataclasses.dataclass
class DeviceWorkload:
    w: Workload
    q_idx: torch.Tensor
    q_scale: torch.Tensor
    weights: torch.Tensor
    k_cache: torch.Tensor
    k_scale: torch.Tensor
    block_table: torch.Tensor
    token_req: torch.Tensor
    token_kvlen: torch.Tensor
    q_mla: torch.Tensor
    kv_pool: torch.Tensor

    @classmethod
    def from_host(cls, w: Workload, device="cuda") -> "DeviceWorkload":
        return cls(w, _t(w.q_idx, device), _t(w.q_scale, device), _t(w.weights, device), _t(w.k_cache, device),
                   _t(w.k_scale, device), _t(w.block_table, device), _t(w.token_req, device),
                   _t(w.token_kvlen, device), _t(w.q_mla.view(np.int16), device).view(torch.bfloat16),
                   _t(w.kv_pool, device))


class HotPath:
    """Buffers and launches for one step of indexer -> top-k -> sparse MLA. With ``fused`` (decode
    batches) the step runs indexer and top-k as the one call hs_indexer_topk, whose scores stay in
    L2 between the two kernels."""

    def __init__(self, dw: DeviceWorkload, fused: bool = False):
        w = dw.w
        dev = dw.q_idx.device
        self.dw = dw
        self.fused = fused
        self.scores = torch.empty((w.T, w.ld), dtype=torch.float32, device=dev)
        self.idx = torch.empty((w.T, w.topk), dtype=torch.int32, device=dev)
        self.out = torch.empty((w.T, w.H, 512), dtype=torch.bfloat16, device=dev)
        self.lse = torch.empty((w.T, w.H), dtype=torch.float32, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        # sparse-MLA scratch: every SM gets an equal share of the (query, tile) work
        self.workspace = torch.empty(hs_sparse_mla_workspace_size(w.H), dtype=torch.uint8, device=dev)

    def step_inputs(self) -> list:
        """The device tensors a step reads that change from step to step (a serving loop copies
        them in); everything else (caches, block tables, pools) stays resident."""
        d = self.dw
        return [d.q_idx, d.q_scale, d.weights, d.q_mla, d.token_req, d.token_kvlen]

    def indexer(self, stream=None):
        d = self.dw
        hs_indexer_scores(d.q_idx, d.q_scale, d.weights, d.k_cache, d.k_scale, d.block_table, d.token_req,
                          d.token_kvlen, self.scores, self.err, num_requests=d.w.B, stream=stream)

    def topk(self, stream=None):
        hs_topk(self.scores, self.dw.token_kvlen, self.dw.w.topk, self.idx, self.err, stream=stream)

    def indexer_topk(self, stream=None):
        d = self.dw
        hs_indexer_topk(d.q_idx, d.q_scale, d.weights, d.k_cache, d.k_scale, d.block_table, d.token_req,
                        d.token_kvlen, self.scores, d.w.topk, self.idx, self.err, num_requests=d.w.B, stream=stream)

    def mla(self, stream=None):
        d = self.dw
        hs_sparse_mla_fwd(d.q_mla, d.kv_pool, self.idx, d.w.softmax_scale, self.out, self.err, lse=self.lse,
                          block_table=d.block_table, token_req=d.token_req, workspace=self.workspace, stream=stream)

    def step(self, stream=None):
        if self.fused:
            self.indexer_topk(stream)
        else:
            self.indexer(stream)
            self.topk(stream)
        self.mla(stream)


class LongPrefillPass:
    """One long-prefill pass: every chunk of one sequence through indexer -> top-k -> sparse MLA,
    chunk after chunk. The sequence's K cache and KV pool and every chunk's query inputs stay
    resident; the scores and top-k buffers are reused by each chunk, and the output holds the
    whole sequence ([chunks, chunk_len, H, 512] bf16 and its LSE)."""

    def __init__(self, chunks: list, device="cuda"):
        w0 = chunks[0]
        self.chunks = chunks
        self.n = len(chunks)
        self.T = w0.T
        self.k_cache = _t(w0.k_cache, device)
        self.k_scale = _t(w0.k_scale, device)
        self.block_table = _t(w0.block_table, device)
        self.token_req = _t(w0.token_req, device)
        self.kv_pool = _t(w0.kv_pool, device)
        self.q_idx = [_t(w.q_idx, device) for w in chunks]
        self.q_scale = [_t(w.q_scale, device) for w in chunks]
        self.weights = [_t(w.weights, device) for w in chunks]
        self.q_mla = [_t(w.q_mla.view(np.int16), device).view(torch.bfloat16) for w in chunks]
        self.token_kvlen = [_t(w.token_kvlen, device) for w in chunks]
        ld = max(w.ld for w in chunks)
        self.scores = torch.empty((w0.T, ld), dtype=torch.float32, device=device)
        self.idx = torch.empty((w0.T, w0.topk), dtype=torch.int32, device=device)
        self.out = torch.empty((self.n, w0.T, w0.H, 512), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((self.n, w0.T, w0.H), dtype=torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = torch.empty(hs_sparse_mla_workspace_size(w0.H), dtype=torch.uint8, device=device)

    def step_inputs(self, c: int) -> list:
        """The device tensors of chunk c that a serving loop would copy in for it."""
        return [self.q_idx[c], self.q_scale[c], self.weights[c], self.q_mla[c], self.token_kvlen[c]]

    def indexer(self, c: int, stream=None, q_idx=None, q_scale=None, weights=None, token_kvlen=None):
        hs_indexer_scores(self.q_idx[c] if q_idx is None else q_idx, self.q_scale[c] if q_scale is None else q_scale,
                          self.weights[c] if weights is None else weights, self.k_cache, self.k_scale,
                          self.block_table, self.token_req,
                          self.token_kvlen[c] if token_kvlen is None else token_kvlen, self.scores, self.err,
                          num_requests=1, stream=stream)

    def topk(self, c: int, stream=None, token_kvlen=None):
        hs_topk(self.scores, self.token_kvlen[c] if token_kvlen is None else token_kvlen, self.chunks[c].topk,
                self.idx, self.err, stream=stream)

    def mla(self, c: int, stream=None, q_mla=None, out=None, lse=None):
        hs_sparse_mla_fwd(self.q_mla[c] if q_mla is None else q_mla, self.kv_pool, self.idx,
                          self.chunks[c].softmax_scale, self.out[c] if out is None else out, self.err,
                          lse=self.lse[c] if lse is None else lse, block_table=self.block_table,
                          token_req=self.token_req, workspace=self.workspace, stream=stream)

    def step(self, stream=None):
        for c in range(self.n):
            self.indexer(c, stream)
            self.topk(c, stream)
            self.mla(c, stream)


class SharedSetHotPath(HotPath):
    """One step with shared index sets: hs_indexer_scores and hs_topk run for the final query token
    of each request only, and hs_sparse_mla_fwd gives every query token its request's set
    (idx_row), limited to the tokens it can see (token_kvlen), so MTP tokens do not re-run the
    indexer."""

    def __init__(self, dw: DeviceWorkload, fused: bool = False):
        super().__init__(dw, fused)
        w = dw.w
        dev = dw.q_idx.device
        req = np.asarray(w.token_req)
        last = np.array([np.flatnonzero(req == r)[np.argmax(w.token_kvlen[req == r])] for r in np.unique(req)])
        row_of_req = np.full(int(req.max()) + 1, -1, np.int32)
        row_of_req[req[last]] = np.arange(len(last), dtype=np.int32)
        li = torch.from_numpy(last).to(dev)
        self.f_q_idx, self.f_q_scale, self.f_weights = (dw.q_idx[li].contiguous(), dw.q_scale[li].contiguous(),
                                                        dw.weights[li].contiguous())
        self.f_req, self.f_kvlen = dw.token_req[li].contiguous(), dw.token_kvlen[li].contiguous()
        self.idx_row = _t(row_of_req[req], dev)
        self.scores = torch.empty((len(last), w.ld), dtype=torch.float32, device=dev)
        self.idx = torch.empty((len(last), w.topk), dtype=torch.int32, device=dev)

    def step_inputs(self) -> list:
        """Only the final tokens' indexer inputs change per step here, with every token's MLA query
        and the token-to-request, visible-length and index-row maps."""
        d = self.dw
        return [self.f_q_idx, self.f_q_scale, self.f_weights, self.f_req, self.f_kvlen, self.idx_row, d.q_mla,
                d.token_req, d.token_kvlen]

    def indexer(self, stream=None):
        d = self.dw
        hs_indexer_scores(self.f_q_idx, self.f_q_scale, self.f_weights, d.k_cache, d.k_scale, d.block_table,
                          self.f_req, self.f_kvlen, self.scores, self.err, num_requests=d.w.B, stream=stream)

    def topk(self, stream=None):
        hs_topk(self.scores, self.f_kvlen, self.dw.w.topk, self.idx, self.err, stream=stream)

    def indexer_topk(self, stream=None):
        d = self.dw
        hs_indexer_topk(self.f_q_idx, self.f_q_scale, self.f_weights, d.k_cache, d.k_scale, d.block_table,
                        self.f_req, self.f_kvlen, self.scores, d.w.topk, self.idx, self.err, num_requests=d.w.B,
                        stream=stream)

    def mla(self, stream=None):
        d = self.dw
        hs_sparse_mla_fwd(d.q_mla, d.kv_pool, self.idx, d.w.softmax_scale, self.out, self.err, lse=self.lse,
                          block_table=d.block_table, token_req=d.token_req, workspace=self.workspace, stream=stream,
                          idx_row=self.idx_row, token_kvlen=d.token_kvlen)


def pinned_uint8(nbytes: int) -> np.ndarray:
    """Page-locked host buffer (device-accessible through unified addressing) as a numpy view.
    The torch tensor owning the memory is kept alive by the returned array's base chain."""
    t = torch.empty(nbytes, dtype=torch.uint8, pin_memory=True)
    a = t.numpy()
    _PINNED_KEEPALIVE.append(t)
    return a


_PINNED_KEEPALIVE: list = []


class DeviceHiSparse:
    """Device state of the mixed-residency decode: pool, block table, LRU state, index stream.
    ``touch_host()`` maps the host tier for the GPU once (hs_hisparse_touch_host); a serving
    system does this when it sets the tier up."""

    def __init__(self, hw: HiSparseWorkload, device="cuda"):
        self.hw = hw
        B, S, k = hw.B, hw.S, hw.k
        self.kv_pool = _t(hw.kv_pool, device)
        self.block_table = _t(hw.block_table, device)
        self.seq_len = _t(hw.seq_len, device)
        self.resident_start = _t(hw.resident_start, device)
        self.slot_row = _t(hw.slot_row, device)
        self.slot_token = torch.full((B, S), -1, dtype=torch.int32, device=device)
        self.slot_stamp = torch.full((B, S), -1, dtype=torch.int32, device=device)
        self.ld_t2s = int(hw.seq_len.max())
        self.tok2slot = torch.full((B, self.ld_t2s), -1, dtype=torch.int32, device=device)
        self.host_rows = torch.tensor([int(h.ctypes.data) for h in hw.host_rows], dtype=torch.int64, device=device)
        self.idx = _t(hw.idx, device)                                     # [steps, B, k]
        self.q = _t(hw.q_mla.view(np.int16), device).view(torch.bfloat16)  # [steps, B, H, 576]
        self.rows = torch.empty((B, k), dtype=torch.int32, device=device)
        self.counters = torch.zeros((B, 3), dtype=torch.int32, device=device)
        self.out = torch.empty((B, hw.H, 512), dtype=torch.bfloat16, device=device)
        self.lse = torch.empty((B, hw.H), dtype=torch.float32, device=device)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = torch.empty(hs_sparse_mla_workspace_size(hw.H), dtype=torch.uint8, device=device)

    def touch_host(self, stream=None):
        hs_hisparse_touch_host(self.host_rows, self.seq_len, self.resident_start, self.err, stream=stream)

    def resolve(self, step: int, stream=None):
        hs_hisparse_resolve(step, self.idx[step], self.seq_len, self.resident_start, self.block_table,
                            self.host_rows, self.kv_pool, self.slot_row, self.slot_token, self.slot_stamp,
                            self.tok2slot, self.rows, self.counters, self.err, stream=stream)

    def mla(self, step: int, stream=None):
        hs_sparse_mla_fwd(self.q[step], self.kv_pool, self.rows, self.hw.softmax_scale, self.out, self.err,
                          lse=self.lse, workspace=self.workspace, stream=stream)

    def step(self, step: int, stream=None):
        self.resolve(step, stream)
        self.mla(step, stream)


def _check_heads(q, latent, rope, w, out, lse, tokens: int, device):
    """What the calls of DenseSession.attend_heads ask of its arguments in either form, all of it before any of them turns or writes
    something: ValueError, or the tensors are as they have to be. Returns (T, H, Dn, Dv)."""
    (T, H, D), Dn, Dv = q.shape, q.shape[2] - 64, out.shape[2]
    given = (q, latent, rope, w, out)
    if T != tokens or (w.shape, out.shape, latent.shape, rope.shape) != ((H, Dn + Dv, 512), (T, H, Dv), (T, 512), (T, 64)) \
            or (lse is not None and lse.shape != (T, H)) or any(x.dtype is not torch.bfloat16 for x in given):
        raise ValueError("q [T,H,Dn+64], latent [T,512], rope [T,64], w [H,Dn+Dv,512] and out [T,H,Dv] must be bf16, lse [T,H], for the "
                         "%d tokens of the last extend" % tokens)
    if Dn not in (64, 128, 192, 256) or Dv not in (64, 128, 192, 256) or not 1 <= H <= 1024:
        raise ValueError("Dn and Dv must be 64, 128, 192 or 256 and H in [1, 1024] (got %d, %d, %d)" % (Dn, Dv, H))
    if lse is not None and lse.dtype is not torch.float32:
        raise ValueError("lse must be float32")
    if any(x.device != device for x in given) or (lse is not None and lse.device != device):
        raise ValueError("tensors must be on the session's device, %s" % device)
    if not (latent.is_contiguous() and rope.is_contiguous() and w.is_contiguous() and (lse is None or lse.is_contiguous())):
        raise ValueError("latent, rope, w and lse must be contiguous")
    for x, name in ((q, "q"), (out, "out")):
        (a, b, c), (t, h, _) = x.stride(), x.shape
        if c != 1 or (t > 1 and (a <= 0 or a % 8)) or (h > 1 and (b <= 0 or b % 8)):
            raise ValueError("%s must have consecutive values in a head, and heads and tokens a multiple of 8 values apart" % name)
    if any(x.data_ptr() % 16 for x in given):
        raise ValueError("q, latent, rope, w and out must be 16-byte aligned")
    return T, H, Dn, Dv


class DenseSession:
    """Requests that attend densely over the paged latent cache and may branch (several samples of one prompt, beams):
    device state for ``B`` request slots and ``L`` layers, and the calls of a step in their order. ``extend`` gives the new
    tokens their positions and pages, then ``attend`` runs once per layer (hs_rope of queries and keys -> hs_kv_append ->
    hs_paged_mla_fwd), or ``attend_heads``, which takes and gives per-head values and picks the form of latent attention. Between
    steps ``fork`` makes slots copies of others (pages shared, the partial one copied), ``free`` empties slots, and ``compact`` moves
    the pages in use to the front. Everything runs on the current stream. The attention's
    workspace is made for steps of ``max_tokens`` and grows with the cached rows, or where a step has more tokens. A captured ``attend`` or
    ``attend_heads`` is one of the tokens of the extend before it, whatever has been extended since; all that it reads stays for as long as
    the session does. Graphs of one session share their buffers: they must not run at the same time."""

    def __init__(self, B: int, H: int, nblk: int, pages: int, L: int = 1, max_tokens: int = 4096, base: float = 10000.0,
                 kind: str = "plain", factor: float = 1.0, device="cuda"):
        i32 = dict(dtype=torch.int32, device=device)
        self.B, self.H, self.nblk, self.L, self.device = B, H, nblk, L, device
        self.pool = torch.zeros((L, nblk * 64, 656), dtype=torch.uint8, device=device)
        self.pools = torch.tensor([p.data_ptr() for p in self.pool], dtype=torch.int64, device=device)
        self.table = torch.full((B, pages), -1, **i32)
        self.seq_len = torch.zeros(B, **i32)
        self.refcount = torch.zeros(nblk, **i32)
        self.src, self.dst = torch.empty(nblk, **i32), torch.empty(nblk, **i32)
        self.counts, self.err = torch.zeros(2, **i32), torch.zeros(1, **i32)
        inv, temperature = hs_rope_inv_freq(64, base, kind, factor)
        self.inv_freq = inv.to(device)
        # YaRN's factor is one of the whole query and key; only 64 of their 576 values are turned, so its square goes with the
        # softmax scale and the rotation takes none
        self.rope_scale, self.softmax_scale = 1.0, temperature ** 2 / 24.0
        self.kv_tokens = 0  # cached rows: shared pages count once per request
        self.workspace = torch.empty(0, dtype=torch.uint8, device=device)
        self._make_room(max_tokens, 0)
        self._kept, self._captured = {}, []  # attend_heads' buffers by name; tensors that captured graphs use
        self.positions, self.read_tokens, self.active, self.pairs = torch.empty(0, **i32), 0, 0, 0  # of the last extend
        self._with_tokens, self._room = None, True  # _requests' offsets; whether the expanded form's buffers could be had
        self.compact_workspace = torch.empty(hs_kv_compact_workspace_size(nblk), dtype=torch.uint8, device=device)

    def _make_room(self, tokens: int, cached: int):
        """A workspace for a step of this many tokens over this many rows. A larger one is made with a quarter to spare, so that a
        growing cache does not make one at every step."""
        need = hs_paged_mla_workspace_size(tokens, self.B, self.H, cached)
        if self.workspace.numel() < need:
            self.workspace = torch.empty(0, dtype=torch.uint8, device=self.device)  # its memory may serve the larger one
            self.workspace = torch.empty(need + need // 4, dtype=torch.uint8, device=self.device)

    def extend(self, new) -> int:
        """``new[r]`` more tokens for slot r: takes free pages where they need some; returns the number of tokens. Tokens are
        ordered by slot. A partial page is a slot's own (fork copied it), so it may be written."""
        new = torch.as_tensor(new, dtype=torch.int32, device=self.device)
        after = self.seq_len + new
        page = torch.arange(self.table.shape[1], device=self.device)[None]
        take = (page >= ((self.seq_len + 63) // 64)[:, None]) & (page < ((after + 63) // 64)[:, None])
        free = (self.refcount <= 0).nonzero()[:, 0][:int(take.sum())].int()
        if int(take.sum()) > free.numel() or int(after.max()) > 64 * self.table.shape[1]:
            raise RuntimeError("the cache has too few pages")
        rows, m = torch.stack([after, new]).cpu().numpy().astype(np.int64)  # of every slot
        self._make_room(int(m.sum()), int(rows.sum()))
        self.kv_tokens = int(rows.sum())
        # rows that the expanded form reads, slots with new tokens, and (token, row) pairs that those see, twice
        self.read_tokens, self.active, self.pairs = int(rows[m > 0].sum()), int((m > 0).sum()), int((m * (2 * rows - m + 1)).sum())
        self.table[take] = free
        self.refcount[free.long()] = 1
        self.token_req = torch.repeat_interleave(torch.arange(self.B, dtype=torch.int32, device=self.device), new)
        self.req_start = torch.cat([new.new_zeros(1), new.cumsum(0).int()])
        T = self.token_req.numel()
        self.positions = (torch.arange(T, dtype=torch.int32, device=self.device)
                          + torch.repeat_interleave(self.seq_len - self.req_start[:-1], new))
        self.seq_len = after
        read = torch.where(new > 0, after, 0)
        self.read_start = torch.cat([read.new_zeros(1), read.cumsum(0).int()])
        self._with_tokens, self._room = None, True
        return T

    def _hold(self, *tensors):
        """Where a graph is being captured, what it uses stays for as long as the session does."""
        if torch.cuda.is_current_stream_capturing():
            self._captured += [x for x in tensors if all(x is not y for y in self._captured)]

    def attend(self, layer: int, q: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor, out: torch.Tensor, lse=None):
        """Layer ``layer`` of the tokens of the last extend: ``q`` bf16 [T, H, 576] and ``rope`` bf16 [T, 64] are rotated in
        place, ``latent`` bf16 [T, 512] and ``rope`` become cache rows, ``out`` bf16 [T, H, 512] receives the attention."""
        self._hold(self.positions, self.token_req, self.req_start, self.seq_len, self.workspace)
        hs_rope(q[..., 512:], self.positions, self.inv_freq, y=rope[:, None], scale=self.rope_scale)
        hs_kv_append(self.token_req, self.positions, self.table, self.err, latent=latent, rope=rope, kv_pool=self.pool[layer])
        hs_paged_mla_fwd(q, self.pool[layer], self.table, self.req_start, self.seq_len, self.kv_tokens, self.softmax_scale, out,
                         self.err, self.workspace, lse=lse)

    #: Heads (Dn, Dv) that the expanded form takes.
    EXPANDED = ((128, 128), (192, 256))
    #: Bytes of expanded keys and values at most (their buffer has a quarter to spare); steps that would need more stay in the absorbed form, as do
    #: those whose buffers cannot be had. A step in the absorbed form gives the rows, keys and values back.
    EXPAND_BYTES = 32 << 30

    def _buffer(self, name: str, *shape, dtype=torch.bfloat16):
        """A buffer that is kept from step to step, made anew with a quarter to spare where it is too small."""
        n, buffer = math.prod(shape), self._kept.get(name)
        if buffer is None or buffer.numel() < n or buffer.dtype != dtype:
            buffer = None
            self._give_back(name)
            self._kept[name] = None
            self._kept[name] = buffer = torch.empty(n + n // 4, dtype=dtype, device=self.device)
        self._hold(buffer)
        return buffer[:n].view(shape)

    def _give_back(self, *names):
        """These buffers' memory may serve other tensors once the calls so far are done. (Not while a graph is captured.)"""
        for name in names if not torch.cuda.is_current_stream_capturing() else ():
            buffer = self._kept.pop(name, None)
            if buffer is not None:
                buffer.record_stream(torch.cuda.current_stream())

    def _expanded_pays(self, T: int, Dn: int, Dv: int) -> bool:
        """Whether the last extend's tokens are faster in the expanded form, by what each form does for a head, in products of the absorbed
        attention: that form makes 1,088 a (token, row) pair and moves 2,176 + Dn + Dv values a token; the other one makes Dn + 64 + Dv a
        pair, at twice the rate, and Dn + Dv values of every row that is read, worth 650 each (512 products, a store and a load). So a long
        prompt among single tokens over long contexts stays absorbed: the rows of those are not worth their expansion.

        Fitted to a layer's step of 418 batches (1 to 64 slots, 16 to 512 tokens each over none to 32,000 rows, and prompts among single tokens;
        16, 64 and 128 heads): in 13 of them the form picked is slower by more than a tenth, by 22 % at most (64 slots x 96 tokens over 300 rows,
        (192, 256)), mostly where both take the host's 100 us. Absorbed / expanded, us, 64 heads of (128, 128): 8 slots over 8,000 rows x 96
        tokens 744 / 1,037, x 192 1,333 / 1,084; one over 32,000 x 128 476 / 614, x 192 656 / 561; 16 over 500 x 64 231 / 219; 8,192
        tokens and 7 slots of one over 60,000 4,154 / 7,757; 1,024 over 16,000 and 32 slots of 4 over 1,000 1,698 / 1,087. (192, 256):
        8 over 8,000 x 192 1,347 / 1,834, x 512 3,456 / 2,457."""
        absorbed = 544 * self.pairs + 400 * (2176 + Dn + Dv) * T
        expanded = (Dn + 64 + Dv) * self.pairs // 4 + 650 * (Dn + Dv) * self.read_tokens
        return T >= 64 and expanded < absorbed

    def _requests(self):
        """req_start and read_start of the slots that have new tokens alone: hs_mla_expanded_fwd picks its variant by the tokens per request
        (a layer's step of 8,192 tokens in one of 64 slots, 64 heads, 991 us with all of them, 900 so; 1,024 over 8,192 rows in one of
        eight 372, 339)."""
        if self.active == self.B:
            return self.req_start, self.read_start
        if self._with_tokens is not None:
            return self._with_tokens
        at = (self.req_start.diff() > 0).cumsum(0).expand(2, -1)  # a slot without tokens writes what the one before it does
        start = torch.zeros((2, self.active + 1), dtype=torch.int32, device=self.device)
        start = start.scatter_(1, at, torch.stack([self.req_start[1:], self.read_start[1:]])).unbind()
        if not torch.cuda.is_current_stream_capturing():  # in a graph it is a part of it
            self._with_tokens = start
        return start

    def attend_heads(self, layer: int, q: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor, w: torch.Tensor, out: torch.Tensor,
                     lse=None, form: str | None = None):
        """Layer ``layer`` of the tokens of the last extend from per-head queries to per-head outputs: ``q`` bf16 [T, H, Dn + 64] (its
        rotary part, the last 64 values, may be rotated in place) and ``rope`` bf16 [T, 64] (rotated in place), ``latent`` bf16 [T, 512],
        the layer's weight ``w`` bf16 [H, Dn + Dv, 512], ``out`` bf16 [T, H, Dv]; logits are scaled by (Dn + 64)^-1/2. ``q`` and ``out`` may be
        slices of wider heads. ``form`` is "absorbed" or "expanded" (heads of 128 and 128, or 192 and 256, alone); None picks it by
        the work of each (_expanded_pays). A call that is refused (ValueError, IndexError), or whose buffers cannot be had, has
        turned and written nothing."""
        if form not in (None, "absorbed", "expanded"):
            raise ValueError("form must be absorbed or expanded")
        pool = self.pool[layer]
        T, H, Dn, Dv = _check_heads(q, latent, rope, w, out, lse, self.positions.numel(), self.pool.device)
        given = form
        if form is None:
            pays = self._room and 2 * self.read_tokens * H * (Dn + Dv) <= self.EXPAND_BYTES and self._expanded_pays(T, Dn, Dv)
            form = "expanded" if (Dn, Dv) in self.EXPANDED and (pays or H > self.H) else "absorbed"
        if form == "expanded" and (Dn, Dv) not in self.EXPANDED:
            raise ValueError("the expanded form takes heads of %s" % " or ".join(map(str, self.EXPANDED)))
        if form == "absorbed" and H > self.H:
            raise ValueError("the session was made for %d heads" % self.H)
        if T == 0:
            return
        if torch.cuda.current_device() != self.pool.device.index:
            raise ValueError("the session's device is not the current one")
        if form == "expanded":
            try:
                rows, kv = self._buffer("rows", self.read_tokens, 576), self._buffer("kv", self.read_tokens, H, Dn + Dv)
                workspace = self._buffer("expanded", hs_mla_expanded_workspace_size(self.active, Dv), dtype=torch.uint8)
                whole = out if out.is_contiguous() else self._buffer("out", T, H, Dv)
            except torch.OutOfMemoryError:
                if given == "expanded" or H > self.H:
                    raise
                form, rows, kv, workspace, self._room = "absorbed", None, None, None, False  # nor is it tried again for the step's other layers
        if form == "absorbed":
            self._give_back("rows", "kv")
            wide, mixed = self._buffer("queries", T, H, 576), self._buffer("mixed", T, H, 512)
        self._hold(self.positions, self.token_req, self.req_start, self.read_start, self.seq_len, self.workspace)
        scale = self.softmax_scale * 24.0 * (Dn + 64) ** -0.5
        if form == "absorbed":
            hs_rope(q[..., Dn:], self.positions, self.inv_freq, out=wide[..., 512:], y=rope[:, None], scale=self.rope_scale)
        else:
            req_start, read_start = self._requests()
            self._hold(req_start, read_start)
            hs_rope(q[..., Dn:], self.positions, self.inv_freq, y=rope[:, None], scale=self.rope_scale)
        hs_kv_append(self.token_req, self.positions, self.table, self.err, latent=latent, rope=rope, kv_pool=pool)
        if form == "absorbed":
            hs_mla_absorb(q[..., :Dn], w, wide[..., :512], self.err)
            hs_paged_mla_fwd(wide, pool, self.table, self.req_start, self.seq_len, self.kv_tokens, scale, mixed, self.err,
                             self.workspace, lse=lse)
            hs_mla_project(mixed, w, out, self.err)
        else:
            hs_kv_read(pool, self.table, self.read_start, rows, self.err)
            hs_mla_expand(rows[:, :512], w, kv, self.err)
            hs_mla_expanded_fwd(q, kv, rows[:, 512:], req_start, read_start, scale, whole, self.err, workspace, lse=lse)
            if whole is not out:
                out.copy_(whole)

    def fork(self, parent, child):
        parent, child = (torch.as_tensor(x, dtype=torch.int32, device=self.device) for x in (parent, child))
        n = parent.numel()
        hs_kv_fork(parent, child, self.table, self.seq_len, self.refcount, self.src[:n], self.dst[:n], self.err, pools=self.pools)

    def free(self, req):
        hs_kv_free(torch.as_tensor(req, dtype=torch.int32, device=self.device), self.table, self.seq_len, self.refcount, self.err)

    def compact(self):
        hs_kv_compact(self.table, self.refcount, self.table, self.refcount, self.src, self.dst, self.counts, self.err,
                      self.compact_workspace, pools=self.pools)
