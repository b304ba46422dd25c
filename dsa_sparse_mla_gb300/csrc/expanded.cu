// expanded.cu — hs_mla_expanded_fwd: attention of each request's new tokens over keys and values of every head (the expanded form of
// latent attention; the 64 rotary key values are shared by the heads).
//
//   logit = scale (q[:Dn] . k[j, h] + q[Dn:] . rope[j]),   out = sum_j softmax(logit)_j v[j, h],   one pass over the rows with a
//   running reference and sum: P = 2^(logit log2 e - ref), and where a row's maximum passes ref by 2^8 its reference moves and
//   the accumulator is scaled (so it rarely is).
//
// Work is units of (request, head, block of tokens), a unit's cached rows cut into pieces where there are too few blocks to fill the
// workers' turns. A planning kernel counts units, chooses the pieces and clears a counter; workers take units from the counter, blocks of a head
// one after the other (they share its keys and values in L2), the longest first. A worker is a pair of CTAs with blocks of 256 tokens,
// or, where requests have few tokens, a CTA by itself with blocks of 128 (few_tokens, below).
//
// A pair works with two-SM MMAs: each CTA holds the queries, logits, P and output of its 128 tokens and half of every K and V
// tile (64 of 128 rows of K, half of V's values). Tensor memory: two logit tiles, and with 128 values per head two tiles of P
// and the output; with 256 values P goes through shared memory instead. In each CTA two warpgroups take the tiles in turn, a
// thread to a token: it takes its 128 logits into registers at once, which frees the tile for the product after next, so that a
// tile's softmax has two whole tiles' products to hide under. A token's reference passes from one warpgroup to the other through
// shared memory. The warpgroups also scale and write the output, under the next unit's first products.
//
// Issuing an MMA takes about as long as its execution once a few are under way, and what a warp does between two batches of them
// (barriers, addresses; its code is cold in the instruction caches, which the softmax fills) takes several hundred cycles. So QK and
// PV have a warp each, which work in each other's gaps, and K and V a ring of slots and a copying warp each: 2,048 tokens over 32,768
// rows x 64 heads 2,720 us with one issuing and one copying warp, 1,606 with two. Tried and not kept: the output written by the warpgroup
// that took the last tile alone while the other goes on (prompt of 8,192 tokens 870 -> 955 us), or by a fourth warpgroup (the softmax
// threads have too few registers then: 915).
//
// Bound by the tensor cores for prompts and chunks: 2,048 tokens over 32,768 rows 1,370 to 1,415 us in a few calls (1,880 to 1,940
// TFLOP/s), 1,590 to 1,627 in long runs, under the power limit; 8,192 tokens over themselves 765 to 785, and 871 to 891. There the softmax
// counts by the energy of its instructions: with one for two products and one for two sums instead of one each 1,485 -> 1,380, 1,600 -> 1,520, and
// 845 -> 785, 887 -> 845 (maxima of three by an instruction of their own spilled: 1,420). A unit's end costs about 5,000 cycles (the last
// tile's softmax, PV and output one after the other), a tile 1,280 of MMAs. (192, 256): 9 ragged requests 330 to 338 us, 377 to 387. Bound by HBM for
// single tokens over long rows: 8 requests over 8,000 rows 331 us, 6.3 TB/s; over 200 to 2,000 rows 62 us, 4.8 TB/s, by the last units.
// (Splitting the blocks of a last turn that is not full: 1,024 tokens over 32,768 rows 861 -> 802 us, but 2,048 over 8,192 366 -> 389 to 418,
// by the joins.)
//
// Rows past a request's end are masked as keys and set to zero as values (in shared memory, by a warp that waits for such a tile's copy).
// A row that a token does not see can still reach its output where P = 0 meets a value that is not finite; where an output is not
// finite although the token's logits are, the warp computes it again from the rows that the token sees (rescue).
#include "launch.cuh"
#include "pair.cuh"

namespace hs {
namespace expanded {

constexpr int kTok = 256, kHalf = 128, kKeys = 128;  // tokens of a block (at most), of a CTA; rows of a tile
constexpr int kThreads = 384;                        // Q and K, QK, PV (units in the other CTA), V (and units); 2 x 128 softmax threads
constexpr float kThreshold = 8.0f;                   // log2 units
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kPlanned = 4;                          // requests per thread of the plan
constexpr int kMinPiece = 8;                         // tiles of a piece, at least
constexpr int kPerPair = 6;                          // pieces of split blocks per pair of CTAs, at most
constexpr int kTurns = 5, kEnd = 6;                  // turns that splitting may make; tiles' time that a unit's end and its join take

struct Req {
  int32_t unit0, q0, m, kv0;   // first unit; first token, tokens; first row
  int32_t len, nb, np, slot0;  // rows; blocks; pieces per block; first slot of the pieces
};

struct Unit {
  int32_t tok, nrows, h, kv0;      // first token, tokens, head, first row of the request
  int32_t ta, n, see, len;         // first tile, tiles (0: no more units), rows that the first token sees, rows of the request
  int32_t np, slot, first, pad;    // pieces of the block (1: whole), this piece's slot, the first piece's
};

constexpr int kMaxPlaces = 4;

struct Params {
  int32_t T, B, H, causal, cap;
  int32_t workers, tok;  // pairs of CTAs and 256, or CTAs and 128 tokens of a block
  const uint16_t* q;
  int64_t q_stride_t, q_stride_h;
  const uint16_t* kv;
  int64_t kv_stride, N;
  const uint16_t* rope;
  int64_t rope_stride;
  const int32_t* req_start;
  const int32_t* kv_start;
  float scale_log2;  // |softmax_scale| log2 e
  uint32_t flip;     // 0x80000000 where softmax_scale < 0
  uint16_t* out;
  float* lse;
  int32_t* err;
  int32_t* total;    // [2]: units, the counter
  Req* req;
  int32_t* joined;   // [cap][16]: pieces of a block that are done, for each softmax warp's tokens and columns
  float* part_lse;   // [cap][2][256]
  float* part_out;   // [cap][256][Dv]
};

// ------------------------------------------------------------------------ plan ------------
// Sum over the threads before this one, and of all.
template <int kWarps>
__device__ __forceinline__ int64_t block_before(int64_t v, int64_t* scratch, int64_t* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](int64_t x) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
  const int64_t x = scan(v);
  __syncthreads();
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  const int64_t w = scan(lane < kWarps ? scratch[lane] : 0);  // of the warps up to this lane's
  *all = __shfl_sync(0xffffffffu, w, 31);
  const int64_t before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return x - v + (warp > 0 ? before : 0);
}
// Requests in descending order of their longest block, to a quarter of an octave (within one in any order: no result depends on it).
__device__ __forceinline__ int size_class(int64_t tiles) {
  return tiles <= 0 ? 127 : 126 - (int)((__float_as_uint((float)tiles) >> 21) - (127u << 2));  // 2^24 tiles at most: classes 27 .. 126
}

// One CTA. Thread t plans requests 4 t .. 4 t + 3 (a call has few, as a rule: 128 threads wait less for each other than 1,024). Long
// blocks come first, so that the last units to end are short.
//
// Pieces: U blocks as long as the longest take ceil(U / workers) turns; cut into j pieces each, w turns where j = w workers / U. The least
// of w (longest / j + kEnd) decides, for w up to kTurns. (Instead of these, as many pieces as an even share of all tiles has quarters:
// 256 tokens over 30,000 rows x 16 heads 190 us, 74 so; 300 over 100,000 x 4 heads 341, 104; one token over 60,000 x 16 heads 160, 100, over
// 8,000 x 64 heads 73, 60.) Turns whose pieces do not fit their slots are left out
// (where their pieces were doubled until they did: 120 requests of one token over 12,800 rows 172 us, 149 so; 67 over 102,400 685, 608).
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const Params p) {
  constexpr int kPer = kPlanned, kWarps = kPlanThreads / 32;
  static_assert(kPlanThreads >= 128 && kWarps <= 32, "a thread to a class, a lane to a warp's sum");
  __shared__ int64_t scratch[32];
  __shared__ int32_t classes[128], places[kPer * kPlanThreads];  // requests of a class, and before it; units of a place
  let_next();
  after_previous();
  int start[kPer], m[kPer], kv0[kPer], len[kPer], nb[kPer], np[kPer], place[kPer];
  int64_t most[kPer], tiles[kPer], tokens = 0;
  __shared__ int32_t longest, long_blocks;  // tiles of the longest block; blocks of more than half as many
  __shared__ unsigned long long others;     // tiles of the other blocks
  if (threadIdx.x < 128) classes[threadIdx.x] = 0;
  if (threadIdx.x == 0) longest = 1, long_blocks = 0, others = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kPer * threadIdx.x + k;
    m[k] = start[k] = kv0[k] = len[k] = nb[k] = place[k] = 0;
    most[k] = tiles[k] = 0;
    if (r >= p.B) continue;
    const int64_t a = p.req_start[r], b = p.req_start[r + 1], c = p.kv_start[r], d = p.kv_start[r + 1];
    if (a < 0 || b < a || b > p.T || (r == 0 && a != 0) || (r == p.B - 1 && b != p.T)) flag_error(p.err, HS_FLAG_BAD_INDEX);
    if (a >= 0 && b > a && b <= p.T) {
      start[k] = (int)a, m[k] = (int)(b - a);
      nb[k] = (m[k] + p.tok - 1) / p.tok;
      tokens += m[k];
      if (c < 0 || d < c || d > p.N) {
        flag_error(p.err, HS_FLAG_BAD_LENGTH);
      } else {
        kv0[k] = (int)c, len[k] = (int)(d - c);
      }
      most[k] = (len[k] + kKeys - 1) / kKeys;
      const int64_t least = p.causal ? ((int64_t)len[k] - m[k] + p.tok + kKeys - 1) / kKeys : most[k];  // of the first block
      tiles[k] = nb[k] * (most[k] + (least < 1 ? 1 : least < most[k] ? least : most[k])) / 2 * p.H;
      atomicMax(&longest, (int)most[k]);
    }
    place[k] = atomicAdd(&classes[size_class(nb[k] ? most[k] + 1 : 0)], 1);
  }
  int64_t all = 0;
  block_before<kWarps>(tokens, scratch, &all);
  const bool none = all > p.T;  // requests overlap (offsets out of order, flagged above): no bound on the units would hold
  const int top = longest;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (nb[k] == 0) continue;
    if (2 * most[k] > top)
      atomicAdd(&long_blocks, nb[k] * p.H);
    else
      atomicAdd(&others, (unsigned long long)tiles[k]);
  }
  __syncthreads();
  const int blocks = max(1, long_blocks + (int)((others + top - 1) / top));
  constexpr int64_t kWhole = (int64_t)1 << 32;  // longer than any block
  int64_t piece = kWhole;
  uint32_t full = 0;  // turns whose pieces have no room
  while (2 * blocks <= kTurns * p.workers) {
    int64_t best = (int64_t)((blocks + p.workers - 1) / p.workers) * (top + kEnd);
    int turns = 0;
#pragma unroll 1
    for (int w = 1; w <= kTurns; ++w) {
      const int n = min(w * p.workers / blocks, top / kMinPiece), t = n > 1 ? (top + n - 1) / n : top;
      if (n > 1 && !(full >> w & 1u) && w * (int64_t)(t + kEnd) < best) best = w * (int64_t)(t + kEnd), piece = t, turns = w;
    }
    if (turns == 0) break;
    int64_t slots = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k)
      if (4 * most[k] > 5 * piece) slots += (int64_t)nb[k] * p.H * ((most[k] + piece - 1) / piece);
    block_before<kWarps>(slots, scratch, &all);
    if (all <= p.cap) break;
    full |= 1u << turns, piece = kWhole;
  }
  const bool splits = piece != kWhole;
  int64_t slots = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    np[k] = 4 * most[k] > 5 * piece ? (int)((most[k] + piece - 1) / piece) : 1;
    if (np[k] > 1) slots += (int64_t)nb[k] * p.H * np[k];
  }
  int64_t slot0 = splits ? block_before<kWarps>(slots, scratch, &all) : 0;
  const int split = splits ? (int)all : 0;  // slots in use
  const int64_t before = block_before<kWarps>(threadIdx.x < 128 ? classes[threadIdx.x] : 0, scratch, &all);
  if (threadIdx.x < 128) classes[threadIdx.x] = (int)before;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (kPer * (int)threadIdx.x + k >= p.B) continue;
    place[k] += classes[size_class(nb[k] ? most[k] + 1 : 0)];
    places[place[k]] = none ? 0 : nb[k] * p.H * np[k];
  }
  __syncthreads();
  int64_t units = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kPer * threadIdx.x + k;
    if (r < p.B) units += places[r];
  }
  int64_t unit0 = block_before<kWarps>(units, scratch, &all);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int r = kPer * threadIdx.x + k;
    if (r >= p.B) continue;
    const int n = places[r];
    places[r] = (int32_t)unit0;
    unit0 += n;
  }
  if (threadIdx.x == 0) {
    p.total[0] = (int32_t)all;
    p.total[1] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (kPer * (int)threadIdx.x + k >= p.B) continue;
    p.req[place[k]] = {places[place[k]], start[k], m[k], kv0[k], len[k], nb[k], np[k], (int32_t)slot0};
    if (np[k] > 1) slot0 += (int64_t)nb[k] * p.H * np[k];
  }
  for (int i = threadIdx.x; i < split * 16; i += kPlanThreads) p.joined[i] = 0;
}

// ------------------------------------------------------------------------ attention -------
template <int kDn, int kDv, int kSMs>
struct Shape {
  static constexpr int kQB = kDn / 64 + 1;                    // blocks of 64 values of a query or key
  static constexpr bool kWide = kDv > 128;                    // P through shared memory
  static constexpr int kQBlk = kHalf * 128, kQBytes = kQB * kQBlk;
  static constexpr int kKRows = kKeys / kSMs, kVCols = kDv / kSMs;  // of a tile, in a CTA
  static constexpr int kKBlk = kKRows * 128, kKBytes = kQB * kKBlk;
  static constexpr int kVBlk = kKeys * 128, kVBytes = kVCols / 64 * kVBlk;
  static constexpr int kKSlots = kWide || kSMs == 1 ? 2 : 4, kVSlots = kKSlots;
  static constexpr int kPlaces = kSMs == 1 ? 4 : 2;           // units that the roles can be apart
  static constexpr int kPBlk = kHalf * 128, kPBytes = kWide ? 2 * kPBlk : 0;  // blocks of 64 cached rows
  static constexpr int kOffK = kQBytes, kOffV = kOffK + kKSlots * kKBytes, kOffP = kOffV + kVSlots * kVBytes, kOffRef = kOffP + (kWide ? kPBytes : 8 * 2048);
  static constexpr int kOffOut = kOffP;                       // 2 KB per softmax warp for the output (wide: in P's place, see the unit's end)
  static constexpr int kOffSum = kOffRef + 1024, kOffUnit = kOffSum + 1024, kOffBar = kOffUnit + kMaxPlaces * (int)sizeof(Unit);
  static constexpr int kSmem = kOffBar + 640;
  static constexpr int kColP = 256, kColO = kWide ? 256 : 384;  // tensor-memory columns; logits in 0 .. 255
  static_assert(kDv % 128 == 0 && kDv <= 256 && kSmem <= 232448, "shared and tensor memory");
};

struct Bars {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4], q_full, q_empty, s_full[2], s_empty[2], p_full[2], pv_done[2], o_full, o_free, drain[2];
  uint64_t tail_full, near_end, unit_full[kMaxPlaces], unit_empty[kMaxPlaces];
  uint64_t ref[8], sum[8], over[8];  // [warpgroup][quad]
  uint32_t tmem;
};
static_assert(sizeof(Bars) <= 640, "barriers");

struct Ring {
  int slot;
  uint32_t par;
  __device__ __forceinline__ void next(int n) {
    if (++slot == n) slot = 0, par ^= 1u;
  }
};

// A role's walk over the units: they arrive in kPlaces places of shared memory in turn.
template <int kPlaces, int kSMs>
struct Units {
  const uint8_t* at;
  Bars* br;
  int32_t* err;
  uint32_t back;  // unit_empty[0] of the CTA that hands units out
  bool gives;     // whether this thread gives units back for its role
  // Unit number n (one thread, or every lane of a warp); false after a wait that ran out.
  __device__ __forceinline__ bool take(uint32_t n, Unit& u) const {
    if (!pair::Mma<kSMs>::wait_writes(&br->unit_full[n % kPlaces], (n / kPlaces) & 1u, err)) return false;
    const int4* v = reinterpret_cast<const int4*>(at + n % kPlaces * sizeof(Unit));
    int4* w = reinterpret_cast<int4*>(&u);
#pragma unroll
    for (int i = 0; i < 3; ++i) w[i] = v[i];
    return true;
  }
  __device__ __forceinline__ void give_back(uint32_t n) const {
    if (gives) pair::Mma<kSMs>::arrive(back + 8 * (n % kPlaces));
  }
};

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two fp32 at once: one instruction where two would be, the same bits.
__device__ __forceinline__ uint64_t two(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint64_t two(float a, float b) { return two(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void apart(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }
__device__ __forceinline__ float from_bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// Joins the pieces of a block for a warp's tokens and columns, in the pieces' order. Weights first, a lane to a token; then eight
// lanes to a token, its columns four at a time per lane, the loads of all 32 tokens and two pieces under way at once: the loads' latency is
// what a join takes (16 tokens at a time: 256 tokens over 30,000 rows x 16 heads 235 us, 189 so). Rows past the last token read the first
// one's values instead of none, since loads under a condition wait for each other (489).
template <int kDv>
__device__ __noinline__ void join(const Params& p, const Unit& u, int g, int quad, int rank, int left) {
  constexpr int kCols = kDv / 2, kGroups = 8;
  const int lane = threadIdx.x & 31, sub = lane & 7, rows = kHalf * rank + 32 * quad;
  const float* lse = p.part_lse + ((int64_t)u.first * 2 + g) * kTok + rows;  // [piece][2][256]
  float top = -INFINITY, sum = 0.f;
#pragma unroll 4
  for (int k = 0; k < u.np; ++k) {
    const float y = __ldcg(lse + (int64_t)k * 2 * kTok + lane);
    top = y > top || y != y ? y : top;  // NaN stays
  }
#pragma unroll 4
  for (int k = 0; k < u.np; ++k) {
    const float y = __ldcg(lse + (int64_t)k * 2 * kTok + lane);
    sum += y == -INFINITY ? 0.f : exp2f((y - top) * kLog2e);
  }
  const float scale = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t tok = (int64_t)u.tok + rows;
  if (g == 0 && p.lse && lane < left) p.lse[(tok + lane) * p.H + u.h] = sum == 0.f ? -INFINITY : top + logf(sum);
  uint16_t* out = p.out + (tok * p.H + u.h) * kDv + kCols * g;
  const float* part = p.part_out + ((int64_t)u.first * kTok + rows) * kDv + kCols * g;
#pragma unroll 1
  for (int r0 = 0; r0 < 32; r0 += 4 * kGroups) {
    if (r0 >= left) break;
    float t[kGroups], f[kGroups];
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      t[i] = __shfl_sync(0xffffffffu, top, r0 + 4 * i + (lane >> 3));
      f[i] = __shfl_sync(0xffffffffu, scale, r0 + 4 * i + (lane >> 3));
    }
#pragma unroll 1
    for (int c = 4 * sub; c < kCols; c += 32) {
      float4 acc[kGroups];
#pragma unroll
      for (int i = 0; i < kGroups; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
      for (int k = 0; k < u.np; ++k) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          const int r = r0 + 4 * i + (lane >> 3), rr = r < left ? r : 0;
          const float y = __ldcg(lse + (int64_t)k * 2 * kTok + rr);
          const float4 x = __ldcg(reinterpret_cast<const float4*>(part + ((int64_t)k * kTok + rr) * kDv + c));
          if (y != -INFINITY) {
            const float w = exp2f((y - t[i]) * kLog2e) * f[i];
            acc[i].x = fmaf(w, x.x, acc[i].x);
            acc[i].y = fmaf(w, x.y, acc[i].y);
            acc[i].z = fmaf(w, x.z, acc[i].z);
            acc[i].w = fmaf(w, x.w, acc[i].w);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        const int r = r0 + 4 * i + (lane >> 3);
        if (r < left)
          *reinterpret_cast<uint2*>(out + (int64_t)r * p.H * kDv + c) = make_uint2(pack_bf16(acc[i].x, acc[i].y), pack_bf16(acc[i].z, acc[i].w));
      }
    }
  }
}

// A token's output values col0 .. col0 + kCols - 1 once more, from the rows that it sees alone, where a row of its tiles that it does not
// see holds a value there that is not finite (P = 0 does not silence it). The whole warp works on one token; rare, so plain: a row
// at a time, 32 lanes to a product, the reference and sum (inv) as they are.
template <int kDn, int kDv>
__device__ __noinline__ bool rescue(const Params& p, const Unit& u, int64_t tok, int see, float me, float inv, int col0, float (&acc)[kDv / 64]) {
  constexpr int kCols = kDv / 2, kEach = kCols / 32, kQ = kDn / 32;
  const int lane = threadIdx.x & 31;
  const int lo = u.ta * kKeys, end = min(lo + u.n * kKeys, u.len), seen = min(see, end);
  const uint16_t* kv = p.kv + (int64_t)u.kv0 * p.kv_stride + (int64_t)u.h * (kDn + kDv);
  bool bad = false;
  for (int j = max(seen, lo); j < end; ++j)
#pragma unroll
    for (int e = 0; e < kEach; ++e) bad |= (kv[(int64_t)j * p.kv_stride + kDn + col0 + 32 * e + lane] & 0x7F80u) == 0x7F80u;
  if (!__any_sync(0xffffffffu, bad)) return false;
  const uint16_t* qp = p.q + tok * p.q_stride_t + u.h * p.q_stride_h;
  const uint16_t* rp = p.rope + (int64_t)u.kv0 * p.rope_stride;
  const float coef = __uint_as_float(__float_as_uint(fmaxf(p.scale_log2, 7.5e-37f)) ^ p.flip);
  float q[kQ + 2];
#pragma unroll
  for (int e = 0; e < kQ + 2; ++e) q[e] = from_bf16(qp[32 * e + lane]);
#pragma unroll
  for (int e = 0; e < kEach; ++e) acc[e] = 0.f;
#pragma unroll 1
  for (int j = lo; j < seen; ++j) {
    const uint16_t* k = kv + (int64_t)j * p.kv_stride;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < kQ; ++e) s = fmaf(q[e], from_bf16(k[32 * e + lane]), s);
#pragma unroll
    for (int e = 0; e < 2; ++e) s = fmaf(q[kQ + e], from_bf16(rp[(int64_t)j * p.rope_stride + 32 * e + lane]), s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float w = fast_exp2(fmaf(s, coef, -me)) * inv;
#pragma unroll
    for (int e = 0; e < kEach; ++e) acc[e] = fmaf(w, from_bf16(k[kDn + col0 + 32 * e + lane]), acc[e]);
  }
  return true;
}

// Hands out units: the next one of the plan becomes number n of this pair (CTA).
template <int kPlaces, int kSMs>
struct Giver {
  const Params& p;
  uint64_t* empty;  // of this CTA
  uint8_t* units;
  uint32_t at, full;
  int r0;           // the last unit's request
  // The whole warp; false at the end, and after a wait that ran out.
  __device__ __forceinline__ bool give(uint32_t n, int32_t total, int lane) {
    if (!warp_wait(&empty[n % kPlaces], ((n / kPlaces) & 1u) ^ 1u, p.err, lane)) return false;
    int32_t i = 0;
    if (lane == 0) i = atomicAdd(&p.total[1], 1);
    i = __shfl_sync(0xffffffffu, i, 0);
    Unit u = {};
    if (i < total) {
      // its request: the last that starts at or before it (numbers grow, so the search goes on from the last one)
      for (;;) {
        const int r = r0 + 1 + lane;
        const uint32_t le = __ballot_sync(0xffffffffu, r < p.B && p.req[r < p.B ? r : 0].unit0 <= i);
        r0 += __popc(le);
        if (le != 0xffffffffu) break;
      }
      const Req q = p.req[r0];
      const int per_head = q.nb * q.np, x = i - q.unit0, rest = x % per_head;
      const int b = q.nb - 1 - rest / q.np, piece = rest % q.np;
      u.h = x / per_head;
      u.tok = q.q0 + b * p.tok;
      u.nrows = min(q.m - b * p.tok, p.tok);
      u.kv0 = q.kv0;
      u.len = q.len;
      u.see = p.causal ? q.len - q.m + 1 + b * p.tok : q.len;
      const int64_t last = p.causal ? (int64_t)u.see + u.nrows - 1 : q.len;
      const int64_t tiles = last > 0 ? (last + kKeys - 1) / kKeys : 0;
      const int64_t ta = tiles * piece / q.np, tb = tiles * (piece + 1) / q.np;
      u.ta = (int)ta;
      u.n = tb > ta ? (int)(tb - ta) : 1;
      if (tb == ta) u.len = 0;  // a tile of which no row is there
      u.np = q.np;
      u.first = q.slot0 + (u.h * q.nb + b) * q.np;
      u.slot = u.first + piece;
    }
    if (lane < kSMs) {
      const int4* v = reinterpret_cast<const int4*>(&u);
      const uint32_t place = n % kPlaces;
      if constexpr (kSMs == 2) {
        const uint32_t on = full + 8 * place;
        pair::arrive_expect_tx(on, sizeof(Unit));
#pragma unroll
        for (int k = 0; k < 3; ++k) pair::st_async16(at + place * (uint32_t)sizeof(Unit) + 16 * k, v[k], on);
      } else {
        int4* to = reinterpret_cast<int4*>(units + place * sizeof(Unit));
#pragma unroll
        for (int k = 0; k < 3; ++k) to[k] = v[k];
        pair::Mma<1>::arrive(full + 8 * place);
      }
    }
    __syncwarp();
    return i < total;
  }
};

template <int kDn, int kDv, int kSMs>
__device__ __forceinline__ void attend(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_r, const CUtensorMap& map_v,
                                       const Params& p) {
  using Sh = Shape<kDn, kDv, kSMs>;
  using Mma = pair::Mma<kSMs>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the swizzled blocks need it; the same in both CTAs
    if (threadIdx.x == 0) flag_error(p.err, HS_FLAG_BAD_STATE);
    return;
  }
  Bars& br = *reinterpret_cast<Bars*>(smem + Sh::kOffBar);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = kSMs == 2 ? cluster_ctarank() : 0;
  let_next();
  if (tid < 8) {
    mbar_init(&br.ref[tid], 1);
    mbar_init(&br.sum[tid], 1);
    mbar_init(&br.over[tid], 1);
  } else if (tid >= 32 && tid < 36) {
    mbar_init(&br.k_full[tid - 32], kSMs);
    mbar_init(&br.k_empty[tid - 32], 1);
    mbar_init(&br.v_full[tid - 32], kSMs);
    mbar_init(&br.v_empty[tid - 32], 1);
  } else if (tid >= 64 && tid < 66) {
    const int b = tid - 64;
    mbar_init(&br.s_full[b], 1);
    mbar_init(&br.s_empty[b], 4 * kSMs);
    mbar_init(&br.p_full[b], 4 * kSMs);
    mbar_init(&br.pv_done[b], 1);
    mbar_init(&br.drain[b], 1);
  } else if (tid >= 100 && tid < 100 + kMaxPlaces) {
    mbar_init(&br.unit_full[tid - 100], 1);
    mbar_init(&br.unit_empty[tid - 100], 10 * kSMs + 2);  // copies of K, copies of V and eight softmax warps of a CTA; QK, PV
  } else if (tid == 96) {
    mbar_init(&br.q_full, kSMs);
    mbar_init(&br.q_empty, 1);
    mbar_init(&br.tail_full, 1);
    mbar_init(&br.near_end, 1);
    mbar_init(&br.o_full, 1);
    mbar_init(&br.o_free, 8 * kSMs);
  } else if (tid == 128) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_r);
    prefetch_tensormap(&map_v);
  }
  mbar_fence_init();
  __syncthreads();
  if (kSMs == 2) cluster_sync();  // both CTAs' barriers exist
  if (warp == 0) Mma::alloc(&br.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = br.tmem;
  after_previous();  // the plan
  const Units<Sh::kPlaces, kSMs> us = {smem + Sh::kOffUnit, &br, p.err, Mma::at(br.unit_empty, kSMs - 1), lane == 0};

  if (warp < 4) {
    // 384 threads start with 168 registers (64,512 in all): 128 keep 96, 256 take 200 (63,488)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    Unit u;
    if (warp == 0) {
      // ================================================================ Q and K =================
      if (lane == 0) {
        const uint32_t full = Mma::at(br.k_full, 0), q_full = Mma::at(&br.q_full, 0);
        Ring ring = {0, 1};
        bool ok = true;
#pragma unroll 1
        for (uint32_t n = 0; ok; ++n) {
          ok = us.take(n, u);
          if (!ok || u.n == 0) break;
          int y = u.kv0 + u.ta * kKeys + Sh::kKRows * (int)rank;
          bool asked = false;  // Q: its place is free when the unit before has issued its last QK; until then K goes ahead
#pragma unroll 1
          for (int t = 0; t < u.n; ++t, y += kKeys) {
            if (!asked && (t == Sh::kKSlots - 1 || t == u.n - 1 || pair::test_wait(&br.q_empty, (n & 1u) ^ 1u))) {
              ok = mbar_wait(&br.q_empty, (n & 1u) ^ 1u, p.err);
              if (!ok) break;
              Mma::expect(q_full, Sh::kQBytes);
#pragma unroll 1
              for (int b = 0; b < Sh::kQB; ++b) pair::load_3d<kSMs>(smem + b * Sh::kQBlk, &map_q, q_full, 64 * b, u.h, u.tok + kHalf * (int)rank);
              asked = true;
            }
            ok = mbar_wait(&br.k_empty[ring.slot], ring.par, p.err);
            if (!ok) break;
            uint8_t* s = smem + Sh::kOffK + ring.slot * Sh::kKBytes;
            const uint32_t bar = full + 8 * (uint32_t)ring.slot;
            Mma::expect(bar, Sh::kKBytes);
#pragma unroll 1
            for (int b = 0; b < kDn / 64; ++b) pair::load_3d<kSMs>(s + b * Sh::kKBlk, &map_k, bar, 64 * b, u.h, y);
            pair::load_2d<kSMs>(s + kDn / 64 * Sh::kKBlk, &map_r, bar, 0, y);
            ring.next(Sh::kKSlots);
          }
          us.give_back(n);
        }
        if (!ok) pair::let_copies_land();
      }
    } else if (warp == 1 && rank == 0) {
      // ================================================================ QK ======================
      constexpr uint32_t id = idesc_bf16(kHalf * kSMs, kKeys, 0, 0);
      const uint64_t qd = smem_desc(smem_u32(smem), 16, 1024, 2), kd = smem_desc(smem_u32(smem + Sh::kOffK), 16, 1024, 2);
      Ring ring = {0, 0};
      uint32_t i = 0;
      if (lane == 0) {
        bool ok = true;
#pragma unroll 1
        for (uint32_t n = 0; ok; ++n) {
          ok = us.take(n, u);
          if (!ok || u.n == 0) break;
          ok = mbar_wait(&br.q_full, n & 1u, p.err);
#pragma unroll 1
          for (int t = 0; t < u.n && ok; ++t, ++i) {
            const uint32_t b = i & 1u;
            ok = mbar_wait(&br.k_full[ring.slot], ring.par, p.err) && mbar_wait(&br.s_empty[b], ((i >> 1) & 1u) ^ 1u, p.err);
            if (!ok) break;
            tc_fence_after();
            uint64_t a = qd, k = kd + (uint64_t)((ring.slot * Sh::kKBytes) >> 4);
#pragma unroll 1
            for (int blk = 0; blk < Sh::kQB; ++blk, a += Sh::kQBlk >> 4, k += Sh::kKBlk >> 4)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) Mma::ss(tmem + kKeys * b, a + 2 * kk, k + 2 * kk, id, (blk | kk) != 0 ? 1u : 0u);
            Mma::commit(&br.s_full[b]);
            Mma::commit(&br.k_empty[ring.slot]);
            ring.next(Sh::kKSlots);
          }
          if (!ok) break;
          Mma::commit(&br.q_empty);
          us.give_back(n);
        }
        Mma::commit(&br.drain[0]);
        mbar_wait(&br.drain[0], 0, p.err);
      }
    } else if (warp == 2 && rank == 0) {
      // ================================================================ PV ======================
      constexpr uint32_t id = idesc_bf16(kHalf * kSMs, kDv, 0, 1);
      const uint64_t vd = smem_desc(smem_u32(smem + Sh::kOffV), Sh::kVBlk, 1024, 2), pd = smem_desc(smem_u32(smem + Sh::kOffP), 16, 1024, 2);
      Ring ring = {0, 0};
      uint32_t i = 0;
      if (lane == 0) {
        bool ok = true;
#pragma unroll 1
        for (uint32_t n = 0; ok; ++n) {
          ok = us.take(n, u);
          if (!ok || u.n == 0) break;
          ok = mbar_wait(&br.o_free, (n & 1u) ^ 1u, p.err);
#pragma unroll 1
          for (int t = 0; t < u.n && ok; ++t, ++i) {
            const uint32_t b = i & 1u;
            // What warps of the other CTA wrote to its shared memory: zeros behind a request's last row, and P where it goes through there.
            // With a release and an acquire of every memory at cluster scope 9 ragged requests of (192, 256) take 513 us, 331 so; by a warp
            // of the other CTA that waits for all of its half and hands it on, 343.
            const bool tail = u.len - (u.ta + t) * kKeys < kKeys;
            ok = tail ? Mma::wait_writes(&br.v_full[ring.slot], ring.par, p.err) : mbar_wait(&br.v_full[ring.slot], ring.par, p.err);
            ok = ok && (Sh::kWide ? Mma::wait_writes(&br.p_full[b], (i >> 1) & 1u, p.err) : mbar_wait(&br.p_full[b], (i >> 1) & 1u, p.err));
            if (!ok) break;
            tc_fence_after();
            uint64_t v = vd + (uint64_t)((ring.slot * Sh::kVBytes) >> 4), w = pd;
            uint32_t pt = tmem + Sh::kColP + 64 * b;
#pragma unroll 1
            for (int half = 0; half < 2; ++half, v += 4 * 2048 >> 4, w += Sh::kPBlk >> 4, pt += 32)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t more = (t | half | kk) != 0 ? 1u : 0u;
                if (Sh::kWide)
                  Mma::ss(tmem + Sh::kColO, w + 2 * kk, v + (2048 >> 4) * kk, id, more);
                else
                  Mma::ts(tmem + Sh::kColO, pt + 8 * kk, v + (2048 >> 4) * kk, id, more);
              }
            Mma::commit(&br.pv_done[b]);
            Mma::commit(&br.v_empty[ring.slot]);
            ring.next(Sh::kVSlots);
          }
          if (!ok) break;
          Mma::commit(&br.o_full);
          us.give_back(n);
        }
        Mma::commit(&br.drain[1]);
        mbar_wait(&br.drain[1], 0, p.err);
      }
    } else if (warp == 2) {
      // ================================================================ units ===================
      Giver<Sh::kPlaces, kSMs> giver = {p, br.unit_empty, smem + Sh::kOffUnit, Mma::at(smem + Sh::kOffUnit, lane & 1), Mma::at(br.unit_full, lane & 1), 0};
      const int32_t total = p.total[0];
      // the next one when V is five tiles before the end, so that a pair with much left takes none (9 ragged requests 344 us a unit
      // ahead, 336 so)
#pragma unroll 1
      for (uint32_t n = 0; giver.give(n, total, lane); ++n)
        if (!warp_wait(&br.near_end, n & 1u, p.err, lane)) break;
    } else if (warp == 3) {
      // ================================================================ V =======================
      // A tile that reaches past its request's end is counted on a barrier of this CTA; rows from there on become zeros, then
      // the tile counts as there. Without a pair this warp also hands out the units, the next one three tiles before the end (8
      // requests over 200 to 2,000 rows 62.9 us; at the second tile 67.3, when too many have a long one to come, at the last 67.7).
      Giver<Sh::kPlaces, kSMs> giver = {p, br.unit_empty, smem + Sh::kOffUnit, Mma::at(smem + Sh::kOffUnit, 0), Mma::at(br.unit_full, 0), 0};
      const int32_t total = kSMs == 1 ? p.total[0] : 0;
      bool more = kSMs == 1 && giver.give(0, total, lane);
      const uint32_t full = Mma::at(br.v_full, 0), tail = Mma::at(&br.tail_full, rank);
      Ring ring = {0, 1};
      uint32_t tails = 0;
      bool ok = true;
#pragma unroll 1
      for (uint32_t n = 0; ok; ++n) {
        ok = __all_sync(0xffffffffu, us.take(n, u));
        if (!ok || u.n == 0) break;
        int y = u.kv0 + u.ta * kKeys, left = u.len - u.ta * kKeys;  // rows of the request from the tile's first on
#pragma unroll 1
        for (int t = 0; t < u.n; ++t, y += kKeys, left -= kKeys) {
          ok = warp_wait(&br.v_empty[ring.slot], ring.par, p.err, lane);
          if (!ok) break;
          uint8_t* s = smem + Sh::kOffV + ring.slot * Sh::kVBytes;
          if (lane == 0) {
            const uint32_t bar = left < kKeys ? tail : full + 8 * (uint32_t)ring.slot;
            Mma::expect(bar, Sh::kVBytes);
#pragma unroll 1
            for (int b = 0; b < Sh::kVCols / 64; ++b) pair::load_3d<kSMs>(s + b * Sh::kVBlk, &map_v, bar, kDn + Sh::kVCols * (int)rank + 64 * b, u.h, y);
          }
          if (left < kKeys) {
            ok = warp_wait(&br.tail_full, tails++ & 1u, p.err, lane);
            if (!ok) break;
#pragma unroll 1
            for (int x = 8 * (left < 0 ? 0 : left) + lane; x < 8 * kKeys; x += 32)
#pragma unroll
              for (int b = 0; b < Sh::kVCols / 64; ++b) *reinterpret_cast<uint4*>(s + b * Sh::kVBlk + 16 * x) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) Mma::arrive_writes(full + 8 * (uint32_t)ring.slot);
          }
          ring.next(Sh::kVSlots);
          if (more && t == (u.n > 3 ? u.n - 3 : 0)) more = giver.give(n + 1, total, lane);
          if (kSMs == 2 && rank == 1 && lane == 0 && t == (u.n > 5 ? u.n - 5 : 0)) mbar_arrive(&br.near_end);
        }
        if (ok) us.give_back(n);
      }
      if (!ok) pair::let_copies_land();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ================================================================ softmax, output ===========
    const int quad = warp & 3, g = (warp - 4) >> 2, row = 32 * quad + lane;  // this CTA's token; the tiles whose number has parity g
    const uint32_t lane_base = tmem + ((uint32_t)(32 * quad) << 16);
    const uint32_t s_empty = Mma::at(br.s_empty, 0), p_full = Mma::at(br.p_full, 0), o_free = Mma::at(&br.o_free, 0);
    float* refs = reinterpret_cast<float*>(smem + Sh::kOffRef);  // [2][128]
    float* sums = reinterpret_cast<float*>(smem + Sh::kOffSum);
    const int mine = 4 * g + quad, other = 4 * (g ^ 1) + quad;  // barriers of the two warps that share these tokens
    uint32_t heard = 0;            // references taken
    uint32_t joint = 0;            // units in which this warp had tokens
    const float coef = fmaxf(p.scale_log2, 7.5e-37f);  // not 0, so that a masked column stays -inf
    uint32_t i = 0;                // tiles
    bool ok = true;
#pragma unroll 1
    for (uint32_t n = 0; ok; ++n) {
      Unit u;
      ok = __all_sync(0xffffffffu, us.take(n, u));
      if (!ok || u.n == 0) break;
      const int have = u.nrows - kHalf * (int)rank;  // tokens of this CTA
      const bool idle = 32 * quad >= have, there = row < have;
      int see = p.causal ? u.see + kHalf * (int)rank + row : u.see;
      // a lane without a token computes what nobody reads; it must not be what makes its warp mask a tile
      see = there ? min(see, u.len) : INT32_MAX;
      float ref = -INFINITY, l = 0.f;
      // the other warp with these tokens has read this one's sums and references, and is done with P's place
      if (!idle && joint > 0) ok = warp_wait_all(&br.over[other], (joint - 1) & 1u, p.err);
#pragma unroll 1
      for (int t = 0; t < u.n && ok; ++t, ++i) {
        if ((int)(i & 1) != g) continue;
        const uint32_t ph = (i >> 1) & 1u;
        if (idle) {
          ok = warp_wait_all(&br.s_full[g], ph, p.err);
          if (ok && lane == 0) Mma::arrive_relaxed(s_empty + 8 * (uint32_t)g);
          // This tile's logits may be there before the warps with tokens have handed on P of the tile before last: without the
          // wait, this arrival could count for that one.
          if (ok && i >= 2) ok = warp_wait_all(&br.pv_done[g], ph ^ 1u, p.err);
          __syncwarp();
          if (ok && lane == 0) Mma::arrive(p_full + 8 * (uint32_t)g);
          continue;
        }
        const float before = ref;  // this warpgroup's sum refers to it
        if (t > 0) {               // the other warpgroup's, after the tile before
          ok = warp_wait_all(&br.ref[other], heard & 1u, p.err);
          if (!ok) break;
          ++heard;
          ref = refs[128 * (g ^ 1) + row];
        }
        const float was = ref;  // the accumulator refers to it
        ok = warp_wait_all(&br.s_full[g], ph, p.err);
        if (!ok) break;
        tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + kKeys * g + 32 * c, v[c]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) Mma::arrive_relaxed(s_empty + 8 * (uint32_t)g);
        const int lim = see - (u.ta + t) * kKeys;  // columns that this token sees: all, or as many
        if (p.flip) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[c][j] ^= 0x80000000u;
        }
        if (!__all_sync(0xffffffffu, lim >= kKeys)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[c][j] = 32 * c + j < lim ? v[c][j] : 0xFF800000u;
        }
        float m4[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          m4[c] = fmaxf(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]));
#pragma unroll
          for (int j = 2; j < 32; j += 2) m4[c] = max3(m4[c], __uint_as_float(v[c][j]), __uint_as_float(v[c][j + 1]));
        }
        float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]);
        mx = mx == -INFINITY ? mx : mx * coef;
        if (mx > ref + kThreshold) ref = mx;
        if (t + 1 < u.n) {
          refs[128 * g + row] = ref;
          __syncwarp();
          if (lane == 0) mbar_arrive(&br.ref[mine]);
        }
        // asked early: whether P of the tile before last has been used (with one buffer: of the tile before)
        bool used = i < 2 || pair::test_wait(&br.pv_done[g], ph ^ 1u);
        if (before != ref) l *= fast_exp2(before - ref);
        const float me = ref == -INFINITY ? 0.f : ref;
        uint64_t sum = 0;
        const uint64_t coef2 = two(coef, coef), me2 = two(-me, -me);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float a, b;
            apart(fma2(two(v[c][2 * j], v[c][2 * j + 1]), coef2, me2), a, b);
            a = fast_exp2(a), b = fast_exp2(b);
            // P has V's type, as the product asks: off by 0.16 % in the root mean square, and so is the output, as much as by its own
            // rounding (0.23 % in all, 0.17 with 32-bit weights). The sum is of the weights before. P's remainder in a product of its own
            // would take half as many MMAs again.
            sum = add2(sum, two(a, b));
            v[c][j] = pack_bf16(a, b);
          }
        }
        float s0, s1;
        apart(sum, s0, s1);
        l += s0 + s1;
        if (!__all_sync(0xffffffffu, used)) ok = warp_wait_all(&br.pv_done[g], ph ^ 1u, p.err);
        if (Sh::kWide && ok && i >= 1) ok = warp_wait_all(&br.pv_done[g ^ 1], ((i - 1) >> 1) & 1u, p.err);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (Sh::kWide) {
            uint8_t* blk = smem + Sh::kOffP + (c >> 1) * Sh::kPBlk;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(blk + sw128_offset(row, 64 * (c & 1) + 16 * j)) =
                  make_uint4(v[c][4 * j], v[c][4 * j + 1], v[c][4 * j + 2], v[c][4 * j + 3]);
          } else {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) w[j] = v[c][j];
            tmem_st16(lane_base + Sh::kColP + 64 * g + 16 * c, w);
          }
        }
        if (t > 0) {
          const float al = was == ref ? 1.f : fast_exp2(was - ref);
          // Rare. (A parity tells two tiles apart: PV of the tile three before came before that of two before, which is over.)
          if (__any_sync(0xffffffffu, al != 1.f)) {
            ok = warp_wait_all(&br.pv_done[g ^ 1], ((i - 1) >> 1) & 1u, p.err);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kDv / 32; ++c) {
              uint32_t x[32];
              tmem_ld32(lane_base + Sh::kColO + 32 * c, x);
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(__uint_as_float(x[j]) * al);
              tmem_st32(lane_base + Sh::kColO + 32 * c, x);
            }
          }
        }
        tmem_wait_st();
        if (Sh::kWide) fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (Sh::kWide)
            Mma::arrive_writes(p_full + 8 * (uint32_t)g);
          else
            Mma::arrive(p_full + 8 * (uint32_t)g);
        }
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the unit's end
      if (!idle) {
        // the warpgroups' sums, each with the reference that it refers to; a token's last reference is the larger (it only grows)
        refs[128 * g + row] = ref;
        sums[128 * g + row] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&br.sum[mine]);
        ok = warp_wait_all(&br.sum[other], joint & 1u, p.err);
        if (!ok) break;
        const float ref2 = refs[128 * (g ^ 1) + row], l2 = sums[128 * (g ^ 1) + row];
        const float top = fmaxf(ref, ref2);
        l = (ref == top ? l : l * fast_exp2(ref - top)) + (ref2 == top ? l2 : l2 * fast_exp2(ref2 - top));
        ref = top;
      }
      // A barrier of its own: a parity of pv_done tells two tiles apart, and this warp has not seen the other warpgroup's.
      ok = warp_wait_all(&br.o_full, n & 1u, p.err);
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        const float me = ref == -INFINITY ? 0.f : ref;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const float z = l == 0.f ? -INFINITY : (me + log2f(l)) * kLn2;
        const int64_t tok = (int64_t)u.tok + kHalf * (int)rank + row;
        constexpr int kCols = kDv / 2;  // of this warpgroup
        const bool whole = u.np == 1;
        // 32 columns at a time through 2 KB of shared memory, so that a store covers 64 bytes of each of 8 tokens
        uint8_t* scratch = smem + Sh::kOffOut + (Sh::kWide ? g * Sh::kPBlk + 4096 * quad : 2048 * (warp - 4));
        float* part = p.part_out + ((int64_t)u.slot * kTok + kHalf * (int)rank + row) * kDv + kCols * g;
        const int left = have - 32 * quad;  // tokens of this warp
        const int64_t pitch = (int64_t)p.H * kDv;
        uint16_t* o = p.out + ((tok - lane) * p.H + u.h) * kDv + kCols * g;  // the warp's first token
        bool bad = false;
#pragma unroll 1
        for (int c = 0; c < kCols / 32; ++c) {
          uint32_t x[32];
          tmem_ld32(lane_base + Sh::kColO + kCols * g + 32 * c, x);
          tmem_wait_ld();
          if (l == 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 0u;
          }
          if (whole) {
            uint32_t most = 0;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              x[j] = pack_bf16(__uint_as_float(x[2 * j]) * inv, __uint_as_float(x[2 * j + 1]) * inv);
              most = __vmaxu2(most, x[j] & 0x7FFF7FFFu);
            }
            bad |= (most & 0xFFFFu) >= 0x7F80u || most >= 0x7F800000u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint4*>(scratch + sw64_offset(lane, 16 * j)) = make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = 8 * j + (lane >> 2);
              const uint4 y = *reinterpret_cast<const uint4*>(scratch + sw64_offset(r, 16 * (lane & 3)));
              if (r < left) *reinterpret_cast<uint4*>(o + r * pitch + 32 * c + 8 * (lane & 3)) = y;
            }
            __syncwarp();
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              x[j] = __float_as_uint(__uint_as_float(x[j]) * inv);
              bad |= !(fabsf(__uint_as_float(x[j])) <= 3.4028235e38f);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // 16 columns
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(scratch + sw64_offset(lane, 16 * j)) =
                    make_uint4(x[16 * h + 4 * j], x[16 * h + 4 * j + 1], x[16 * h + 4 * j + 2], x[16 * h + 4 * j + 3]);
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = 8 * j + (lane >> 2);
                const uint4 y = *reinterpret_cast<const uint4*>(scratch + sw64_offset(r, 16 * (lane & 3)));
                if (r < left) *reinterpret_cast<uint4*>(part + (int64_t)(r - lane) * kDv + 32 * c + 16 * h + 4 * (lane & 3)) = y;
              }
              __syncwarp();
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          Mma::arrive(o_free);
          mbar_arrive(&br.over[mine]);
        }
        ++joint;
        for (uint32_t again = __ballot_sync(0xffffffffu, there && bad && l <= 3.4028235e38f); again; again &= again - 1) {
          const int r = __ffs(again) - 1;
          float acc[kCols / 32];
          if (!rescue<kDn, kDv>(p, u, tok - lane + r, __shfl_sync(0xffffffffu, see, r), __shfl_sync(0xffffffffu, me, r),
                                __shfl_sync(0xffffffffu, inv, r), kCols * g, acc))
            continue;
#pragma unroll
          for (int e = 0; e < kCols / 32; ++e) {
            if (whole)
              p.out[((tok - lane + r) * p.H + u.h) * kDv + kCols * g + 32 * e + lane] = (uint16_t)(pack_bf16(acc[e], 0.f) & 0xFFFFu);
            else
              (part + (int64_t)(r - lane) * kDv)[32 * e + lane] = acc[e];
          }
        }
        __syncwarp();
        if (whole) {
          if (g == 0 && there && p.lse) p.lse[tok * p.H + u.h] = z;
        } else {
          const int at = kHalf * (int)rank + row;
          p.part_lse[((int64_t)u.slot * 2 + g) * kTok + at] = z;
          __threadfence();
          __syncwarp();
          int before = 0;
          if (lane == 0) before = atomicAdd(&p.joined[(int64_t)u.first * 16 + 8 * (int)rank + mine], 1);
          before = __shfl_sync(0xffffffffu, before, 0);
          if (before == u.np - 1) {
            __threadfence();  // the last piece to end joins them all
            join<kDv>(p, u, g, quad, (int)rank, left);
          }
        }
      } else {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) Mma::arrive(o_free);
      }
      __syncwarp();
      if (lane == 0) us.give_back(n);
    }
  }
  __syncthreads();
  if (kSMs == 2) cluster_sync();  // no CTA leaves while the other may still signal or read it
  if (warp == 0) {
    tc_fence_after();
    Mma::dealloc(tmem, 512);
  }
}

template <int kDn, int kDv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expanded_pair_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  attend<kDn, kDv, 2>(map_q, map_k, map_r, map_v, p);
}

template <int kDn, int kDv>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Params p) {
  attend<kDn, kDv, 1>(map_q, map_k, map_r, map_v, p);
}

template <int kDn, int kDv, int kSMs>
static cudaError_t launch(Params p, int sms, cudaStream_t stream, const char** why) {
  using Sh = Shape<kDn, kDv, kSMs>;
  void (*kernel)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, const Params);
  if constexpr (kSMs == 2)
    kernel = expanded_pair_kernel<kDn, kDv>;
  else
    kernel = expanded_kernel<kDn, kDv>;
  cudaError_t e = pair::allow_smem(kernel, Sh::kSmem);
  if (e != cudaSuccess) return e;
  p.workers = sms / kSMs, p.tok = kHalf * kSMs;
  CUtensorMap mq, mk, mr, mv;
  if (!pair::encode_heads(&mq, p.q, kDn + HS_D_ROPE, p.H, p.T, p.q_stride_h, p.q_stride_t, kHalf) ||
      !pair::encode_heads(&mk, p.kv, kDn + kDv, p.H, p.N, kDn + kDv, p.kv_stride, Sh::kKRows) ||
      !pair::encode_heads(&mv, p.kv, kDn + kDv, p.H, p.N, kDn + kDv, p.kv_stride, kKeys) ||
      !encode_2d(&mr, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, p.rope, HS_D_ROPE, (uint64_t)p.N, (uint64_t)p.rope_stride * 2, 64, Sh::kKRows,
                 CU_TENSOR_MAP_SWIZZLE_128B)) {
    *why = "cuTensorMapEncodeTiled failed";
    return cudaErrorInvalidValue;
  }
  // 128 threads plan up to 512 requests, 1,024 threads the others
  e = p.B <= 128 * kPlanned ? launch_next(plan_kernel<128>, dim3(1), 128, 0, stream, p) : launch_next(plan_kernel<1024>, dim3(1), 1024, 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_next(kernel, dim3((unsigned)(p.workers * kSMs)), kThreads, Sh::kSmem, stream, mq, mk, mr, mv, p);
}

// Workspace: totals, requests, joins, log-sum-exps and outputs of pieces.
static uint64_t up(uint64_t v) { return (v + 127) / 128 * 128; }
static uint64_t off_req() { return 128; }
static uint64_t off_joined(int B) { return off_req() + up((uint64_t)B * sizeof(Req)); }
static uint64_t off_lse(int B, int cap) { return off_joined(B) + up((uint64_t)cap * 16 * 4); }
static uint64_t off_out(int B, int cap) { return off_lse(B, cap) + up((uint64_t)cap * 2 * kTok * 4); }

// Whether CTAs by themselves are better than pairs: with blocks of at most 128 tokens half of a pair would be idle. Measured (pairs /
// alone, us, 64 heads, 8 requests over 4,000 rows): 16 tokens each 189 / 178, 128 203 / 186, 129 207 / 246, 256 218 / 252; one token
// each over 1,000 rows 70 / 56, one alone over 4,000 38 / 41; 16 heads, 64 requests x 33 tokens over 200 rows 75 / 44. How the tokens spread
// over the requests is on the device: all of them in one of 64, 8,192 over themselves, 783 / 879; 1,024 in one of 8 over 8,192 rows
// 217 / 249; callers leave out requests without tokens. (192, 256) has no room for whole tiles.
static bool few_tokens(int T, int B) { return (int64_t)T <= 128ll * B; }

}  // namespace expanded

uint64_t mla_expanded_workspace_bytes(int B, int Dv, int sms) {
  using namespace expanded;
  const int cap = kPerPair * (sms / 2);
  return off_out(B, cap) + (uint64_t)cap * kTok * Dv * 4;
}

cudaError_t launch_mla_expanded(const hs_mla_expanded_args* a, int sms, cudaStream_t stream, const char** why) {
  using namespace expanded;
  Params p;
  p.T = a->T, p.B = a->B, p.H = a->H, p.causal = a->causal, p.cap = kPerPair * (sms / 2);
  p.q = a->q, p.q_stride_t = a->q_stride_t, p.q_stride_h = a->q_stride_h;
  p.kv = a->kv, p.kv_stride = a->kv_stride, p.N = a->N;
  p.rope = a->rope, p.rope_stride = a->rope_stride;
  p.req_start = a->req_start, p.kv_start = a->kv_start;
  p.scale_log2 = fabsf(a->softmax_scale) * kLog2e;
  p.flip = a->softmax_scale < 0.f ? 0x80000000u : 0u;
  p.out = a->out, p.lse = a->lse, p.err = a->err_flag;
  uint8_t* w = reinterpret_cast<uint8_t*>(a->workspace);
  p.total = reinterpret_cast<int32_t*>(w);
  p.req = reinterpret_cast<Req*>(w + off_req());
  p.joined = reinterpret_cast<int32_t*>(w + off_joined(a->B));
  p.part_lse = reinterpret_cast<float*>(w + off_lse(a->B, p.cap));
  p.part_out = reinterpret_cast<float*>(w + off_out(a->B, p.cap));
  if (a->Dv != 128) return launch<192, 256, 2>(p, sms, stream, why);
  return few_tokens(a->T, a->B) ? launch<128, 128, 1>(p, sms, stream, why) : launch<128, 128, 2>(p, sms, stream, why);
}

}  // namespace hs
