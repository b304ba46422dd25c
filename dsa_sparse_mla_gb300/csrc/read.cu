// read.cu — hs_kv_read: rows of the paged FP8 cache as 16- or 32-bit values.
//
// out[i, c] = e4m3(code[c]) * scale[c / 128] for the 512 latent values (the product rounded to fp32, then to the type), the 64
// rotary values as stored. A warp takes two output rows: it finds the request of the first (32 offsets of out_start at once), asks
// for both cached rows, then converts and stores them; a lane's pieces of codes and of results are such that every access of the warp is
// one run of at least 128 bytes. Bound by HBM: 656 bytes in and 1,152 (2,304) out per row. 214,000 rows to fp32 (634 MB) take 99 us, 6.4
// TB/s, 0.95 of a plain copy. Warps that end and make room for others are better than warps that go on: 110 us with eight blocks of
// 256 threads per SM in a loop (of four rows; one row at a time 109, eight 118), 102 with 16, 99 with a block for every 16 rows.
#include "common.cuh"
#include "launch.cuh"

namespace hs {
namespace read {

constexpr int kThreads = 256, kRows = 2;

struct Params {
  int64_t n, out_stride, R;
  const uint8_t* pool;
  const int32_t* bt;
  const int32_t* first;
  const int32_t* start;
  uint8_t* out;
  int32_t* err;
  int32_t B, bt_stride;
};

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  const __half2 v = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Two e4m3 codes (exact in fp16, so exact here).
__device__ __forceinline__ float2 decode2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes & 0xFFFFu), __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const Params p) {
  constexpr bool k32 = sizeof(T) == 4;
  constexpr int kPieces = k32 ? 4 : 2;            // 16-byte results per lane and row
  constexpr int kCodes = 16 / (int)sizeof(T);     // codes each: 4 or 8
  const int lane = threadIdx.x & 31;
  let_next();
  if (blockIdx.x == 0) {
    for (int r = threadIdx.x; r < p.B; r += kThreads)
      if (p.start[r + 1] < p.start[r] || (r == 0 && p.start[0] != 0) || p.start[r + 1] > p.n) flag_error(p.err, HS_FLAG_BAD_INDEX);
  }
  const int64_t i0 = ((int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * kRows;
  if (i0 >= p.n) return;
  // the last request that starts at or before i0: start[r] <= i0, counted 32 at a time
  int lo = 0, hi = p.B;  // start[lo] <= i0 (else no request has the row), start[hi] > i0 or hi == B
#pragma unroll 1
  while (hi - lo > 1) {
    const int w = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * w;
    const bool le = at < hi && (int64_t)p.start[at] <= i0;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    const int nlo = lo + c * w;
    hi = min(hi, nlo + w);
    lo = nlo;
  }
  const uint8_t* row[kRows];
  int state[kRows];  // 0: left as it is, 1: zeros, 2: read
  int r = lo;
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    const int64_t i = i0 + k;
    while (r + 1 < p.B && (int64_t)p.start[r + 1] <= i) ++r;
    const int64_t off = i - p.start[r];
    state[k] = i < p.n && off >= 0 && i < p.start[r + 1] ? 1 : 0;
    row[k] = p.pool;
    if (state[k]) {
      const int64_t j = off + (p.first ? p.first[r] : 0);
      if (j < 0 || j >= (int64_t)p.bt_stride * HS_PAGE) {
        if (lane == 0) flag_error(p.err, HS_FLAG_BAD_LENGTH);
      } else {
        const int64_t page = p.bt[(int64_t)r * p.bt_stride + j / HS_PAGE];
        if (page < 0 || (page + 1) * HS_PAGE > p.R) {
          if (lane == 0) flag_error(p.err, HS_FLAG_BAD_BLOCK);
        } else {
          state[k] = 2;
          row[k] = p.pool + (page * HS_PAGE + j % HS_PAGE) * HS_KV_ROW_BYTES;
        }
      }
    }
  }
  // lane l's piece q: codes kCodes (l + 32 q) .. ; rotary values 2 l, 2 l + 1
  uint32_t codes[kRows][4], rope[kRows];
  float scale[kRows][kPieces];
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (state[k] == 2) {
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        if (k32) {
          codes[k][q] = __ldg(reinterpret_cast<const uint32_t*>(row[k]) + lane + 32 * q);
        } else {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(row[k]) + lane + 32 * q);
          codes[k][2 * q] = v.x, codes[k][2 * q + 1] = v.y;
        }
        scale[k][q] = __ldg(reinterpret_cast<const float*>(row[k] + HS_D_LATENT) + kCodes * (lane + 32 * q) / 128);
      }
      rope[k] = __ldg(reinterpret_cast<const uint32_t*>(row[k] + HS_D_LATENT + 16) + lane);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) codes[k][q] = 0;
#pragma unroll
      for (int q = 0; q < kPieces; ++q) scale[k][q] = 0.f;
      rope[k] = 0;
    }
  }
#pragma unroll
  for (int k = 0; k < kRows; ++k) {
    if (state[k] == 0) continue;
    uint8_t* out = p.out + (i0 + k) * p.out_stride * (int64_t)sizeof(T);
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const float s = scale[k][q];
      uint4 v;
      if constexpr (k32) {
        const float2 a = decode2(codes[k][q]), b = decode2(codes[k][q] >> 16);
        v = make_uint4(__float_as_uint(a.x * s), __float_as_uint(a.y * s), __float_as_uint(b.x * s), __float_as_uint(b.y * s));
      } else {
        uint32_t w[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float2 a = decode2(codes[k][2 * q + (z >> 1)] >> (16 * (z & 1)));
          w[z] = pack2<T>(a.x * s, a.y * s);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      *reinterpret_cast<uint4*>(out + 16 * (lane + 32 * q)) = v;
    }
    const float a = __uint_as_float(rope[k] << 16), b = __uint_as_float(rope[k] & 0xFFFF0000u);
    uint8_t* o = out + (HS_D_LATENT + 2 * lane) * (int)sizeof(T);
    if constexpr (k32)
      *reinterpret_cast<float2*>(o) = make_float2(a, b);
    else
      *reinterpret_cast<uint32_t*>(o) = pack2<T>(a, b);
  }
}

}  // namespace read

cudaError_t launch_kv_read(const hs_kv_read_args* a, cudaStream_t stream) {
  using namespace read;
  Params p;
  p.n = a->n, p.out_stride = a->out_stride, p.R = a->R;
  p.pool = a->kv_pool, p.bt = a->block_table, p.first = a->first, p.start = a->out_start;
  p.out = reinterpret_cast<uint8_t*>(a->out), p.err = a->err_flag;
  p.B = a->B, p.bt_stride = a->bt_stride;
  const int grid = (int)((a->n + kRows * (kThreads / 32) - 1) / (kRows * (kThreads / 32)));
  auto kernel = a->dtype == HS_BF16 ? read_kernel<__nv_bfloat16> : a->dtype == HS_FP16 ? read_kernel<__half> : read_kernel<float>;
  kernel<<<grid, kThreads, 0, stream>>>(p);  // started early, it waits longer than it gains (8 requests in a graph 4.5 us, 5.7 started early)
  return cudaGetLastError();
}

}  // namespace hs
