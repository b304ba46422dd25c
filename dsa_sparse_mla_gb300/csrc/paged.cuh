// paged.cuh — what the kernels of the paged attention share: the batch's work as units (block of
// (token, head) rows, 128 cached rows), the dequantisation of a row, and the join of split blocks.
#pragma once

#include "cluster.cuh"
#include "launch.cuh"
#include "query.cuh"

namespace hs {
namespace paged {

constexpr int kKeys = 128;                     // cached rows per tile: two pages
constexpr float kThreshold = 8.0f;             // log2 units
// P is held 2^7 times as large, and so are its sums: up to 2^15 with a reference that lags by the threshold. fp16's smallest step,
// 2^-24, is then 2^-31 of the reference. Without it weights below 2^-25 were lost from P but not from the sum: 262,144 weights
// of 2^-25.25 beside one large one, 0.65 % together, left nothing in the output.
constexpr float kLift = 7.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kScaleMax = 65504.f / 448.f;   // |code * scale| stays finite in fp16
constexpr float kScaleMin = 6.103515625e-05f;  // 2^-14: scales stay fp16 normals
constexpr int kMaxReq = 4096;

struct Desc {  // a block that starts in a cluster and goes on in the next ones
  int32_t row0, nrows, nparts, pad;
};

struct Params {
  int32_t T, B, H, causal, bt_stride, clusters;
  const uint8_t* q;
  const uint8_t* kv;
  int64_t R;
  const int32_t* bt;
  const int32_t* req_start;
  const int32_t* seq_len;
  float scale_log2;  // |softmax_scale| * log2(e)
  uint32_t flip;     // 0x80008000 when softmax_scale < 0: Q changes sign instead
  __nv_bfloat16* out;
  float* lse;
  int32_t* err;
  float* part_out;   // [2 clusters][rows][512]: slot 2c: the part that ends or passes through cluster c, 2c + 1: one that starts there
  float* part_lse;   // [2 clusters][rows]
  Desc* desc;        // [clusters]
  int64_t kv_tokens;
};

struct Req {
  int32_t start, m, seq, nb;  // first token, new tokens, cached rows, row blocks
};

template <int kRows>
__device__ __forceinline__ Req load_req(const Params& p, int r) {
  Req q;
  const int a = p.req_start[r], b = p.req_start[r + 1], s = p.seq_len[r];
  const bool ok = a >= 0 && a <= b && b <= p.T;
  q.start = ok ? a : 0;
  q.m = ok ? b - a : 0;
  q.seq = s >= 0 && s <= (int64_t)p.bt_stride * HS_PAGE ? s : 0;
  q.nb = (int)(((int64_t)q.m * p.H + kRows - 1) / kRows);
  return q;
}
// Cached rows that row g (of the request's (token, head) rows) sees. T * H < 2^31, so the token takes a 32-bit division only. The
// kernels for blocks of 256 rows divide in 64 bits all the same: their raw variant's main loops came out 6 % slower beside the
// shorter code (64 requests x 4 tokens 1,431 us against 1,350), those of the 64-row kernel 9 % faster (decode 514 against 561).
template <int kRows>
__device__ __forceinline__ int sees(const Params& p, const Req& q, int64_t g) {
  if (!p.causal) return q.seq;
  const int token = kRows <= 64 ? (int)((uint32_t)g / (uint32_t)p.H) : (int)(g / p.H);
  const int n = q.seq - q.m + 1 + token;
  return n < 0 ? 0 : n;
}
template <int kRows>
__device__ __forceinline__ int block_rows(const Params& p, const Req& q, int b) {
  const int64_t left = (int64_t)q.m * p.H - (int64_t)b * kRows;
  return left < kRows ? (int)left : kRows;
}
template <int kRows>
__device__ __forceinline__ int block_tiles(const Params& p, const Req& q, int b) {
  const int n = sees<kRows>(p, q, (int64_t)b * kRows + block_rows<kRows>(p, q, b) - 1);
  return n > 0 ? (int)(((uint32_t)n + kKeys - 1) / kKeys) : 1;  // a block that sees nothing still writes its zeros
}

__host__ __device__ __forceinline__ int64_t unit_begin(int64_t c, int64_t U, int64_t C) { return c * U / C; }
__device__ __forceinline__ int64_t unit_cta(int64_t u, int64_t U, int64_t C) { return ((u + 1) * C - 1) / U; }

// A block costs its tiles and what it takes to begin and end it (its queries, its output), in tiles: about four. Measured with
// 1 / 2 / 3 / 4 / 5 / 7 / 10 tiles: 9 ragged requests of up to 400 tokens 331 / 277 / 241 / 217 / 216 / 220 / 230 us; 32 long
// requests of one token 571 / 566 / 561 / 562 / 562 / 565 / 568 us.
constexpr int kBlockCost = 4;

// Splitting costs this many tiles: partial results and their join. A batch of at most one block per cluster is split only where
// its longest block takes longer than an equal share and the join. Measured (us, split / whole): 30 requests x 4 tokens x 64
// heads over 500 / 760 / 1,500 rows 48 / 33, 51 / 38, 66 / 50; 8 x 16 x 16 over 760 / 1,000 38 / 35, 39 / 40; 64 x 1 x 64 over
// 380 / 700 42 / 35, 50 / 46; 16 x 1 x 64 over 700 33 / 44.
template <int kRows>
constexpr int kJoinCost = kRows <= 64 ? 6 : 8;

// Where a cluster's work begins: found by every CTA of it at its start, in shared memory.
struct Start {
  int64_t U;          // cost of all blocks
  int64_t cost;       // cost of the blocks before the first one here
  int64_t base;       // rows before request r in the dequantised copy
  int32_t ntiles;     // tiles of this cluster
  int32_t r, b, ta;   // request, block and tile of the first
};

// Rows that a request takes in the dequantised copy: whole tiles, one at least (zeros), none without new tokens.
__device__ __forceinline__ int64_t copy_rows(const Req& q) {
  return q.m == 0 ? 0 : q.seq == 0 ? kKeys : (int64_t)(((uint32_t)q.seq + kKeys - 1) / kKeys) * kKeys;
}

// A cluster's units as segments: consecutive tiles [ta, tb) of one block.
struct Seg {
  Req q;
  int r, b, ta, tb, tiles, nrows;
  int64_t base;  // the request's first row in the dequantised copy
};
template <int kRows>
struct Walk {
  Req q;
  int r, b, ta;
  int32_t left;
  int64_t base;
  __device__ __forceinline__ Walk(const Params& p, const Start& s) : r(s.r), b(s.b), ta(s.ta), left(s.ntiles), base(s.base) {
    q = load_req<kRows>(p, r);
  }
  __device__ __forceinline__ bool next(const Params& p, Seg& s) {
    if (left <= 0) return false;
    while (b >= q.nb) {
      base += copy_rows(q);
      q = load_req<kRows>(p, ++r);
      b = 0;
    }
    s.q = q;
    s.r = r;
    s.b = b;
    s.ta = ta;
    s.base = base;
    s.tiles = block_tiles<kRows>(p, q, b);
    s.nrows = block_rows<kRows>(p, q, b);
    s.tb = s.tiles < ta + left ? s.tiles : ta + left;
    left -= s.tb - ta;
    ta = 0;
    ++b;
    return true;
  }
};

// Inclusive prefix sum over the lanes of a warp.
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// All threads of the CTA; `pre` is scratch for 2 (B + 1) sums. Prefix sums over the requests' costs and blocks, then the
// request, block and tile where this cluster's share begins and how many tiles it has. A batch whose lengths pass
// kv_tokens has none.
template <int kRows>
__device__ __forceinline__ void find_units(const Params& p, int64_t* pre, Start* st, int c, int threads) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* nblk = reinterpret_cast<int32_t*>(pre + p.B + 1);  // blocks before each request
  for (int r = warp; r < p.B; r += threads / 32) {
    const Req q = load_req<kRows>(p, r);
    int64_t sum = 0;
    for (int b = lane; b < q.nb; b += 32) sum += block_tiles<kRows>(p, q, b) + kBlockCost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) {
      pre[r + 1] = sum;
      nblk[r + 1] = q.nb;
    }
  }
  __syncthreads();
  if (warp == 0) {
    int64_t run = 0, cached = 0, blocks = 0;
    int most = 0;  // tiles of a block: a request's last one has the most
    if (lane == 0) pre[0] = 0, nblk[0] = 0;
    for (int at = 0; at < p.B; at += 32) {
      const bool in = at + lane < p.B;
      const int64_t x = warp_scan(in ? pre[at + lane + 1] : 0, lane), n = warp_scan(in ? nblk[at + lane + 1] : 0, lane);
      if (in) {
        pre[at + lane + 1] = run + x;
        nblk[at + lane + 1] = (int32_t)(blocks + n);
        const Req q = load_req<kRows>(p, at + lane);
        cached += q.seq;
        if (q.nb > 0) most = max(most, block_tiles<kRows>(p, q, q.nb - 1));
      }
      run += __shfl_sync(0xffffffffu, x, 31);
      blocks += __shfl_sync(0xffffffffu, n, 31);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      cached += __shfl_xor_sync(0xffffffffu, cached, o);
      most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
    }
    __syncwarp();
    if (cached > p.kv_tokens) {
      run = 0;
      if (c == 0 && lane == 0) flag_error(p.err, HS_FLAG_BAD_LENGTH);
    }
    const int64_t U = run, C = U < p.clusters ? U : p.clusters;
    auto rows_before = [&](int request) {
      int64_t n = 0;
      for (int r = lane; r < request; r += 32) n += copy_rows(load_req<kRows>(p, r));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
      return n;
    };
    int64_t tiles_before[2] = {0, 0}, cost = 0, base = 0;
    int r0 = 0, b0 = 0, ta0 = 0;
    if (U > 0 && blocks <= p.clusters && (int64_t)(most + kBlockCost - kJoinCost<kRows>) * p.clusters <= U) {
      if (c < blocks) {  // block c
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (nblk[mid] <= c)
            lo = mid;
          else
            hi = mid;
        }
        r0 = lo;
        b0 = c - nblk[lo];
        tiles_before[1] = block_tiles<kRows>(p, load_req<kRows>(p, lo), b0);
        base = rows_before(lo);
      }
    } else if (c < C) {
      for (int end = 0; end < 2; ++end) {  // the share's beginning and its end
        const int64_t u = unit_begin(c + end, U, C);
        int lo = 0, hi = p.B;  // the request with pre[lo] <= u < pre[lo + 1]; the last one with blocks for u = U
        while (hi - lo > 1) {
          const int mid = (lo + hi) >> 1;
          if (pre[mid] <= u && pre[mid] < U)
            lo = mid;
          else
            hi = mid;
        }
        const Req q = load_req<kRows>(p, lo);
        int64_t off = u - pre[lo];  // cost into the request, then into the block
        int b = q.nb, ta = 0;
        for (int at = 0; at < q.nb; at += 32) {
          const int t = at + lane < q.nb ? block_tiles<kRows>(p, q, at + lane) + kBlockCost : 0;
          const int64_t x = warp_scan(t, lane);
          const uint32_t hit = __ballot_sync(0xffffffffu, x > off);
          if (hit) {
            const int l = __ffs(hit) - 1;
            b = at + l;
            off -= __shfl_sync(0xffffffffu, x - t, l);
            ta = off > kBlockCost ? (int)(off - kBlockCost) : 0;
            break;
          }
          off -= __shfl_sync(0xffffffffu, x, 31);
        }
        // where the end lies past the last block, off is 0 and b the number of blocks
        const int64_t at_block = u - off;
        tiles_before[end] = at_block - (int64_t)kBlockCost * (nblk[lo] + b) + ta;
        if (end == 0) {
          r0 = lo;
          b0 = b;
          ta0 = ta;
          cost = at_block;
          base = rows_before(lo);
        }
      }
    }
    if (lane == 0) {
      st->U = U;
      st->cost = cost;
      st->base = base;
      st->ntiles = (int32_t)(tiles_before[1] - tiles_before[0]);
      st->r = r0;
      st->b = b0;
      st->ta = ta0;
    }
  }
  if (c == 0) {  // tell of bad lengths and offsets once
    for (int r = tid; r < p.B; r += threads) {
      const int a = p.req_start[r], e = p.req_start[r + 1], s = p.seq_len[r];
      if (a < 0 || a > e || e > p.T || (r == 0 && a != 0) || (r == p.B - 1 && e != p.T)) flag_error(p.err, HS_FLAG_BAD_INDEX);
      if (s < 0 || s > (int64_t)p.bt_stride * HS_PAGE) flag_error(p.err, HS_FLAG_BAD_LENGTH);
    }
  }
}

// 8 e4m3 codes -> 8 fp16 values code * scale, rounded once: the fp32 scale is split into fp16 hi + lo and
// t = code * lo corrects fma(code, hi, t).
__device__ __forceinline__ uint4 dequant8(uint32_t w0, uint32_t w1, uint32_t hi2, uint32_t lo2) {
  uint4 r;
  asm("{ .reg .b16 a, b, c, d; .reg .b32 x, y, z, u, tx, ty, tz, tu;\n"
      " mov.b32 {a, b}, %4; mov.b32 {c, d}, %5;\n"
      " cvt.rn.f16x2.e4m3x2 x, a; cvt.rn.f16x2.e4m3x2 y, b; cvt.rn.f16x2.e4m3x2 z, c; cvt.rn.f16x2.e4m3x2 u, d;\n"
      " mul.rn.f16x2 tx, x, %7; mul.rn.f16x2 ty, y, %7; mul.rn.f16x2 tz, z, %7; mul.rn.f16x2 tu, u, %7;\n"
      " fma.rn.f16x2 %0, x, %6, tx; fma.rn.f16x2 %1, y, %6, ty; fma.rn.f16x2 %2, z, %6, tz; fma.rn.f16x2 %3, u, %6, tu; }"
      : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
      : "r"(w0), "r"(w1), "r"(hi2), "r"(lo2));
  return r;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// whether one of the eight fp16 values is NaN or infinite (x * 0 is NaN then)
__device__ __forceinline__ bool unsound(const uint4& a, const uint4& b) {
  const __half2 z = __float2half2_rn(0.f);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  __half2 acc = z;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc = __hfma2(*reinterpret_cast<const __half2*>(&w[i]), z, acc);
  return __hisnan(__low2half(acc)) || __hisnan(__high2half(acc));
}

// paged_few.cu: its workspace for partial results (p.part_out is its start), and the launch.
uint64_t few_bytes(int sms);
cudaError_t launch_few(const Params& p, int sms, cudaStream_t stream);

// Joins the parts of split blocks: each part is normalised by its own sum, so out = sum_s e^(lse_s - lse) O_s. A CTA takes
// some rows (a 32nd of a block) of the blocks that start in one or two clusters (many start none), two rows at a time, a float4
// per thread, the parts in two halves. Bound by the latency of the loads (eight in flight per thread). Measured in whole calls:
// one request of 30,000 rows in 152 parts 46 us (133 with a float4 of four rows per thread and all parts in turn); 64 requests
// of 4,000 rows 106 us (112 with eight clusters per CTA).
constexpr int kMergeThreads = 512, kMaxClusters = 160;
template <int kRows>
struct Merge {
  static constexpr int kTake = kRows / 32;             // rows per CTA
  static constexpr int kStarts = kRows <= 64 ? 2 : 1;  // clusters per CTA
  static dim3 grid(int clusters) { return dim3((unsigned)((clusters + kStarts - 1) / kStarts), kRows / kTake); }
};
template <int kRows>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const Params p) {
  constexpr int kTake = Merge<kRows>::kTake, kStarts = Merge<kRows>::kStarts;
  __shared__ float w[kMaxClusters][kTake];
  __shared__ float4 other[256];
  const int tid = threadIdx.x, r0 = blockIdx.y * kTake;
  after_previous();
  Desc desc[kStarts];
#pragma unroll
  for (int k = 0; k < kStarts; ++k) {
    const int c = blockIdx.x * kStarts + k;
    desc[k] = c < p.clusters ? p.desc[c] : Desc{0, 0, 0, 0};
  }
#pragma unroll
  for (int k = 0; k < kStarts; ++k) {
    const Desc d = desc[k];
    if (d.nparts == 0 || r0 >= d.nrows) continue;  // the same for the whole CTA
    const int c = blockIdx.x * kStarts + k;
    auto slot = [&](int s) { return s == 0 ? 2 * c + 1 : 2 * (c + s); };
    // weights of the parts: a warp per row, a lane per part (and 32 further on)
    if (tid / 32 < kTake) {
      const int i = tid / 32, lane = tid % 32, row = r0 + i;
      float m = -INFINITY, z = 0.f;
      for (int s = lane; s < d.nparts; s += 32) {
        const float l = p.part_lse[slot(s) * kRows + row];
        w[s][i] = l;
        m = fmaxf(m, l);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      for (int s = lane; s < d.nparts; s += 32) {
        const float l = w[s][i], e = l == -INFINITY ? 0.f : __expf(l - (m == -INFINITY ? 0.f : m));
        w[s][i] = e;
        z += e;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      for (int s = lane; s < d.nparts; s += 32) w[s][i] = z == 0.f ? 0.f : w[s][i] / z;
      if (lane == 0 && p.lse && row < d.nrows) p.lse[(int64_t)d.row0 + row] = z == 0.f ? -INFINITY : m + __logf(z);
    }
    __syncthreads();
    const int half = tid / 256, col = 4 * (tid % 128);
#pragma unroll 1
    for (int i = tid / 128 % 2; i < kTake; i += 2) {
      float a[4] = {0.f, 0.f, 0.f, 0.f};
      if (r0 + i < d.nrows) {
        const float* from = p.part_out + (int64_t)(r0 + i) * HS_D_LATENT + col;
#pragma unroll 8
        for (int s = half; s < d.nparts; s += 2) {
          const float4 x = *reinterpret_cast<const float4*>(from + (int64_t)slot(s) * kRows * HS_D_LATENT);
          const float ws = w[s][i];
          a[0] += ws * x.x, a[1] += ws * x.y, a[2] += ws * x.z, a[3] += ws * x.w;
        }
      }
      if (half) other[tid - 256] = make_float4(a[0], a[1], a[2], a[3]);
      __syncthreads();
      if (!half && r0 + i < d.nrows) {
        const float4 y = other[tid];
        const __nv_bfloat162 lo = __floats2bfloat162_rn(a[0] + y.x, a[1] + y.y), hi = __floats2bfloat162_rn(a[2] + y.z, a[3] + y.w);
        *reinterpret_cast<uint2*>(p.out + ((int64_t)d.row0 + r0 + i) * HS_D_LATENT + col) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      }
      __syncthreads();
    }
  }
}

}  // namespace paged
}  // namespace hs
