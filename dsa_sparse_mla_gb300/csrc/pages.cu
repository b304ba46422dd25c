// pages.cu — the pages of a paged cache: copying, forking, freeing and compacting them.
//
// [P3] 「vLLM GLM 5.3 最適化: ハイブリッド HiSparse オフロード」, section 「主要なアーキテクチャ的詳細」: the
// latent pool is a pool of ordinary blocks that requests borrow, one block table for all layers. Here the
// caller's state is that table, the requests' lengths and a use count per page (0: free). A page of a
// request is 64 rows of 656 bytes in each latent layer and 64 keys of Di codes with their fp32 scales in
// each indexer layer, each of them contiguous, so moving it is one contiguous copy per layer.
//
// Which page a fork takes and where a page moves is decided by index alone (the lowest free page, the
// i-th page past the end into the i-th gap), from prefix sums: no result depends on the order in which
// threads run. Use counts are integers, so their atomic sums do not either.
//
// Copies are bound by HBM: a CTA moves one page of one layer at a time, each thread with up to 11
// 16-byte loads in flight before its stores. The planning kernels are bound by their latency; they read
// use counts once, 16 bytes per thread. Measured on a GB300: compaction that moves 2,100 pages of 24 + 6 layers (4.4 GB)
// 687 us, 6,470 GB/s, 0.97 of a plain copy's rate; 256 forks of requests with 24 + 6 layers (255 MB) and their release
// 63 us, of which the copies 34 us, the forks' plan 7.5 us, the release 6 us, and the rest between launches; a compaction of
// 133 pages 13 us (count 2.5, plan 4.5, moves 8.5 one after the other; 15.6 without launching each before the one before it
// ends, which costs the host 1.5 us per launch: small forks, bound by the host, are slower with it, 44 against 41 us).
#include "common.cuh"
#include "launch.cuh"

namespace hs {
namespace pages {

constexpr int kPageBytes = HS_PAGE * HS_KV_ROW_BYTES;  // 41,984
constexpr int kCopyThreads = 256;
constexpr int kVecs = (kPageBytes / 16 + kCopyThreads - 1) / kCopyThreads;  // 11
constexpr int kPlanThreads = 1024;
constexpr int kMaxForks = 8192;  // forks per call: their order is held in shared memory
constexpr int kChunk = 1024;  // pages per CTA of the compaction's planning

struct Layers {
  int32_t L, Li, Di;
  uint8_t* const* pools;
  uint8_t* const* k_caches;
  float* const* k_scales;
};

// One page's first `rows` rows from src to dst in latent layer l < L, or indexer layer l - L.
__device__ __forceinline__ void copy_page(const Layers& y, int l, int64_t src, int64_t dst, int rows, int32_t* err) {
  const int tid = threadIdx.x;
  const uint8_t* s;
  uint8_t* d;
  int n;  // 16-byte pieces
  if (l < y.L) {
    uint8_t* base = y.pools[l];
    if ((uintptr_t)base & 15) {
      if (tid == 0) flag_error(err, HS_FLAG_BAD_INDEX);
      return;
    }
    s = base + src * kPageBytes;
    d = base + dst * kPageBytes;
    n = rows * (HS_KV_ROW_BYTES / 16);
  } else {
    uint8_t* base = y.k_caches[l - y.L];
    float* sc = y.k_scales[l - y.L];
    if (((uintptr_t)base & 15) || ((uintptr_t)sc & 3)) {
      if (tid == 0) flag_error(err, HS_FLAG_BAD_INDEX);
      return;
    }
    s = base + src * (HS_PAGE * y.Di);
    d = base + dst * (HS_PAGE * y.Di);
    n = rows * (y.Di / 16);
    if (tid < rows) sc[dst * HS_PAGE + tid] = sc[src * HS_PAGE + tid];
  }
  uint4 v[kVecs];
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int i = tid + k * kCopyThreads;
    if (i < n) v[k] = *reinterpret_cast<const uint4*>(s + 16 * (int64_t)i);
  }
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int i = tid + k * kCopyThreads;
    if (i < n) *reinterpret_cast<uint4*>(d + 16 * (int64_t)i) = v[k];
  }
}

// Exclusive prefix sum of one value per thread over the block, and the block's sum. `s` holds 33 ints.
__device__ __forceinline__ int block_scan(int v, int* s, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s[warp] = x;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < nw ? s[lane] : 0;
    int z = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, z, o);
      if (lane >= o) z += y;
    }
    if (lane < nw) s[lane] = z - w;
    if (lane == 31) s[32] = z;
  }
  __syncthreads();
  total = s[32];
  return s[warp] + x - v;
}

// ------------------------------------------------------------------ copy -------------------
struct CopyParams {
  int32_t n;
  const int32_t* src;
  const int32_t* dst;
  const int32_t* rows;   // NULL: 64
  int64_t nblk;
  Layers y;
  int32_t* err;
};

__device__ __forceinline__ void copy_entry(const CopyParams& p, int i, int l) {
  const int src = p.src[i], dst = p.dst[i];
  if (src < 0 || dst < 0) return;  // padding
  const int rows = p.rows ? p.rows[i] : HS_PAGE;
  if (src >= p.nblk || dst >= p.nblk || rows < 0 || rows > HS_PAGE) {
    if (threadIdx.x == 0) flag_error(p.err, rows < 0 || rows > HS_PAGE ? HS_FLAG_BAD_LENGTH : HS_FLAG_BAD_BLOCK);
    return;
  }
  if (src != dst) copy_page(p.y, l, src, dst, rows, p.err);
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const CopyParams p) {
  const int layers = p.y.L + p.y.Li;
  const int64_t items = (int64_t)p.n * layers;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) copy_entry(p, (int)(it / layers), (int)(it % layers));
}

// ------------------------------------------------------------------ fork -------------------
struct ForkParams {
  int32_t n, B, bt_stride;
  int64_t nblk;
  const int32_t* parent;
  const int32_t* child;
  int32_t* bt;
  int32_t* seq_len;
  int32_t* ref;
  int32_t* src;
  int32_t* dst;
  Layers y;
  int32_t* err;
};

// The length that fork i copies; -1 (and a flag) where the fork cannot be served.
__device__ __forceinline__ int fork_length(const ForkParams& p, int i, bool tell) {
  const int pa = p.parent[i], ch = p.child[i];
  if (pa < 0 || pa >= p.B || ch < 0 || ch >= p.B || pa == ch) {
    if (tell) flag_error(p.err, HS_FLAG_BAD_INDEX);
    return -1;
  }
  const int len = p.seq_len[pa];
  if (len < 0 || len > (int64_t)p.bt_stride * HS_PAGE) {
    if (tell) flag_error(p.err, HS_FLAG_BAD_LENGTH);
    return -1;
  }
  return len;
}

// One CTA. The forks whose parent ends inside a page take the lowest free pages in fork order:
// src[i] = that page of the parent, dst[i] = the page taken (its use count becomes 1); -1 elsewhere.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(const ForkParams p) {
  __shared__ int s[33];
  __shared__ int fork_of[kMaxForks];  // the fork that takes the r-th free page
  const int tid = threadIdx.x;
  int need = 0;
  for (int base = 0; base < p.n; base += kPlanThreads) {
    const int i = base + tid;
    int page = -1;
    if (i < p.n) {
      const int len = fork_length(p, i, true);
      if (len > 0 && len % HS_PAGE != 0) {
        page = p.bt[(int64_t)p.parent[i] * p.bt_stride + len / HS_PAGE];
        if (page < 0 || page >= p.nblk) {
          flag_error(p.err, HS_FLAG_BAD_BLOCK);
          page = -1;
        }
      }
      p.src[i] = page;
      p.dst[i] = -1;
    }
    int total;
    const int rank = need + block_scan(page >= 0, s, total);
    if (page >= 0) fork_of[rank] = i;
    need += total;
  }
  __syncthreads();
  int found = 0;  // free pages before the current window
  for (int64_t at = 0; at < p.nblk && found < need; at += 4 * kPlanThreads) {
    const int64_t b = at + 4 * tid;
    bool f[4];
    int c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[k] = b + k < p.nblk && p.ref[b + k] <= 0;
      c += f[k];
    }
    int total;
    int r = found + block_scan(c, s, total);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (f[k]) {
        if (r < need) {
          p.dst[fork_of[r]] = (int)(b + k);
          p.ref[b + k] = 1;
        }
        ++r;
      }
    found += total;
  }
  for (int r = found + tid; r < need; r += kPlanThreads) {  // no page left for these forks
    p.src[fork_of[r]] = -1;
    flag_error(p.err, HS_FLAG_NO_PAGES);
  }
}

// After the plan: CTAs of y = 0 write a child's table row and length and count its shared pages; the
// others copy the parent's last, partial page (its rows in use) in one layer each.
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const ForkParams p) {
  const int i = blockIdx.x;
  const int len = fork_length(p, i, false);
  const int full = len < 0 ? 0 : len / HS_PAGE, tail = len < 0 ? 0 : len % HS_PAGE;
  const int dst = p.dst[i];
  if (blockIdx.y > 0) {
    if (dst >= 0) copy_page(p.y, blockIdx.y - 1, p.src[i], dst, tail, p.err);
    return;
  }
  const int ch = p.child[i];
  if (ch < 0 || ch >= p.B || ch == p.parent[i]) return;
  const bool served = len >= 0 && (tail == 0 || dst >= 0);
  int32_t* row = p.bt + (int64_t)ch * p.bt_stride;
  const int32_t* from = p.bt + (int64_t)(served ? p.parent[i] : ch) * p.bt_stride;
  for (int j = threadIdx.x; j < p.bt_stride; j += kCopyThreads) {
    int page = -1;
    if (served && j < full) {
      page = from[j];
      if (page < 0 || page >= p.nblk) {
        flag_error(p.err, HS_FLAG_BAD_BLOCK);
        page = -1;
      } else {
        atomicAdd(p.ref + page, 1);
      }
    } else if (served && j == full && tail) {
      page = dst;
    }
    row[j] = page;
  }
  if (threadIdx.x == 0) p.seq_len[ch] = served ? len : 0;
}

// ------------------------------------------------------------------ free -------------------
struct FreeParams {
  int32_t n, B, bt_stride;
  int64_t nblk;
  const int32_t* req;
  int32_t* bt;
  int32_t* seq_len;
  int32_t* ref;
  int32_t* err;
};

__global__ void __launch_bounds__(kCopyThreads) free_kernel(const FreeParams p) {
  const int r = p.req[blockIdx.x];
  if (r < 0) return;  // padding
  if (r >= p.B) {
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_INDEX);
    return;
  }
  const int len = p.seq_len[r];
  __syncthreads();  // every thread has read the length before it is cleared
  if (len < 0 || len > (int64_t)p.bt_stride * HS_PAGE) {
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_LENGTH);
    return;
  }
  const int held = (len + HS_PAGE - 1) / HS_PAGE;
  int32_t* row = p.bt + (int64_t)r * p.bt_stride;
  for (int j = threadIdx.x; j < p.bt_stride; j += kCopyThreads) {
    const int page = row[j];
    row[j] = -1;
    if (j >= held) continue;
    if (page < 0 || page >= p.nblk) {
      flag_error(p.err, HS_FLAG_BAD_BLOCK);
    } else if (atomicSub(p.ref + page, 1) <= 0) {  // it was free: the count stays as it was
      atomicAdd(p.ref + page, 1);
      flag_error(p.err, HS_FLAG_BAD_STATE);
    }
  }
  if (threadIdx.x == 0) p.seq_len[r] = 0;
}

// ------------------------------------------------------------------ compact ----------------
struct CompactParams {
  int32_t B, bt_stride, N, chunks;
  const int32_t* bt;
  const int32_t* ref;
  int32_t* bt_out;
  int32_t* ref_out;
  int32_t* src;
  int32_t* dst;
  int32_t* counts;      // {pages in use, pages moved}
  int32_t* chunk_used;  // [chunks]: pages in use of each chunk
  int32_t* move;        // [N]: the move that takes a page away, -1 without one
  Layers y;
  int32_t* err;
};

__global__ void __launch_bounds__(kChunk) compact_count_kernel(const CompactParams p) {
  let_next();
  const int i = blockIdx.x * kChunk + threadIdx.x;
  const int n = __syncthreads_count(i < p.N && p.ref[i] > 0);
  if (threadIdx.x == 0) p.chunk_used[blockIdx.x] = n;
}

// With U pages in use, the i-th page in use at or past U moves to the i-th free page before U.
__global__ void __launch_bounds__(kChunk) compact_plan_kernel(const CompactParams p) {
  __shared__ int s[33];
  __shared__ int sums[3];  // in use: in all, before this chunk, before the chunk that holds U
  const int tid = threadIdx.x;
  let_next();
  if (tid < 3) sums[tid] = 0;
  __syncthreads();
  after_previous();
  int all = 0, before = 0;
  for (int c = tid; c < p.chunks; c += kChunk) {
    const int u = p.chunk_used[c];
    all += u;
    before += c < (int)blockIdx.x ? u : 0;
  }
  atomicAdd(&sums[0], all);
  atomicAdd(&sums[1], before);
  __syncthreads();
  const int U = sums[0];
  const int cu = U / kChunk;
  int part = 0;
  for (int c = tid; c < p.chunks && c < cu; c += kChunk) part += p.chunk_used[c];
  atomicAdd(&sums[2], part);
  const int j = cu * kChunk + tid;
  const int mine = __syncthreads_count(j < U && p.ref[j < p.N ? j : 0] > 0);
  const int low = sums[2] + mine;  // pages in use before U
  const int moved = U - low;       // as many as there are free pages before U
  const int i = blockIdx.x * kChunk + tid;
  const bool used = i < p.N && p.ref[i] > 0;
  int total;
  const int rank = sums[1] + block_scan(used, s, total);  // pages in use before i
  if (i < p.N) {
    int m = -1;
    if (i < U && !used) p.dst[i - rank] = i;
    if (i >= U && used) {
      m = rank - low;
      p.src[m] = i;
    }
    p.move[i] = m;
    if (i >= moved) {
      p.src[i] = -1;
      p.dst[i] = -1;
    }
  }
  if (i == 0) {
    p.counts[0] = U;
    p.counts[1] = moved;
  }
}

// Copies every move in every layer, and rewrites the table and the use counts.
__global__ void __launch_bounds__(kCopyThreads) compact_move_kernel(const CompactParams p) {
  after_previous();
  const int moved = p.counts[1], U = p.counts[0];
  const int64_t stride = (int64_t)gridDim.x * kCopyThreads, t0 = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x;
  for (int64_t i = t0; i < (int64_t)p.B * p.bt_stride; i += stride) {
    int e = p.bt[i];
    if (e >= p.N) {
      flag_error(p.err, HS_FLAG_BAD_BLOCK);
    } else if (e >= 0) {
      if (p.move[e] >= 0)
        e = p.dst[p.move[e]];
      else if (e >= U)  // an entry that names a page nobody uses
        flag_error(p.err, HS_FLAG_BAD_STATE);
    }
    p.bt_out[i] = e;
  }
  for (int64_t i = t0; i < p.N; i += stride) {
    const int m = p.move[i], c = p.ref[i];
    if (m >= 0) {
      p.ref_out[p.dst[m]] = c;
      p.ref_out[i] = 0;
    } else if (i >= U || c > 0) {  // the free pages before U get their counts from the moves
      p.ref_out[i] = c;
    }
  }
  const int layers = p.y.L + p.y.Li;
  const int64_t items = (int64_t)moved * layers;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int m = (int)(it / layers);
    copy_page(p.y, (int)(it % layers), p.src[m], p.dst[m], HS_PAGE, p.err);
  }
}

}  // namespace pages

uint64_t compact_workspace_bytes(int64_t nblk) { return 4ull * (nblk + (nblk + pages::kChunk - 1) / pages::kChunk); }

cudaError_t launch_copy_pages(const hs_kv_copy_args* a, int sms, cudaStream_t stream) {
  using namespace pages;
  CopyParams p = {a->n, a->src, a->dst, a->rows, a->nblk, {a->L, a->Li, a->Di, a->pools, a->k_caches, a->k_scales}, a->err_flag};
  int64_t grid = (int64_t)a->n * (a->L + a->Li);
  if (grid > 32LL * sms) grid = 32LL * sms;
  copy_kernel<<<(unsigned)grid, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_fork(const hs_kv_fork_args* a, cudaStream_t stream) {
  using namespace pages;
  ForkParams p = {a->n,       a->B,   a->bt_stride, a->nblk, a->parent, a->child, a->block_table, a->seq_len,
                  a->refcount, a->src, a->dst,       {a->L, a->Li, a->Di, a->pools, a->k_caches, a->k_scales}, a->err_flag};
  fork_plan_kernel<<<1, kPlanThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  fork_kernel<<<dim3((unsigned)a->n, (unsigned)(1 + a->L + a->Li)), kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_free(const hs_kv_free_args* a, cudaStream_t stream) {
  using namespace pages;
  FreeParams p = {a->n, a->B, a->bt_stride, a->nblk, a->req, a->block_table, a->seq_len, a->refcount, a->err_flag};
  free_kernel<<<(unsigned)a->n, kCopyThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_compact(const hs_kv_compact_args* a, int sms, cudaStream_t stream) {
  using namespace pages;
  CompactParams p;
  p.B = a->B;
  p.bt_stride = a->bt_stride;
  p.N = (int32_t)a->nblk;
  p.chunks = (int32_t)((a->nblk + kChunk - 1) / kChunk);
  p.bt = a->block_table;
  p.ref = a->refcount;
  p.bt_out = a->table_out;
  p.ref_out = a->refcount_out;
  p.src = a->src;
  p.dst = a->dst;
  p.counts = a->counts;
  p.move = reinterpret_cast<int32_t*>(a->workspace);
  p.chunk_used = p.move + a->nblk;
  p.y = {a->L, a->Li, a->Di, a->pools, a->k_caches, a->k_scales};
  p.err = a->err_flag;
  compact_count_kernel<<<(unsigned)p.chunks, kChunk, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_next(compact_plan_kernel, dim3((unsigned)p.chunks), kChunk, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_next(compact_move_kernel, dim3((unsigned)(8 * sms)), kCopyThreads, 0, stream, p);
}

}  // namespace hs
