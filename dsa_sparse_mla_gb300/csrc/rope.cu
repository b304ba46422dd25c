// rope.cu — rotary positions of queries and keys, any even part of a head, one launch for both.
//
// Token t at position p turns pair i of each head by the angle p * inv_freq[i]:
//   (a, b) -> scale * (a cos - b sin, a sin + b cos)
// where (a, b) are values (2i, 2i + 1) of the rotary part (interleaved) or (i, i + rot / 2) (halves).
// [P1] "vLLM v0.32.0 GLM-5.3 サービング ...", section 「数字がうまくいく理由」: a cached row carries 64
// bf16 RoPE values beside its latent codes; hs_kv_append stores them and the MLA reads them as given.
//
// The angle of a far position. p * inv_freq in fp32 is off by up to p * inv_freq * 2^-24, 0.06 rad
// at a million. Here a pair's frequency is a 64-bit fixed-point fraction of a turn, f = inv_freq /
// (2 pi) * 2^64 (one fp64 multiplication per pair and CTA), and the product p * f mod 2^64 drops whole
// turns exactly, in integers. What is left, read as a signed fraction, is rounded to fp32 once (2^-24
// of half a turn) and goes to sincospif. No table of positions is read or kept.
//
// Bound by HBM: every value is read and written once. A CTA computes the cosines and sines of its
// tokens into shared memory (one thread per (token, pair)), then its threads take units of 8 pairs
// (16-bit types) or 4 pairs (fp32), two 16-byte loads and two 16-byte stores each, over tokens, heads
// and pair groups. Where a base address or a stride is no multiple of 16 bytes, or rot / 2 no multiple
// of the unit's pairs, a unit is one pair (element loads).
#include "common.cuh"

namespace hs {
namespace rope {

constexpr int kThreads = 256;

struct Tensor {
  const uint8_t* x;
  uint8_t* out;
  int64_t xt, xh, ot, oh;  // strides in bytes: token, head
};

struct Params {
  int32_t T, H, H2, half, inverse, per_cta;
  float scale;
  const int32_t* pos;
  const double* inv_freq;
  Tensor a, b;
};

template <typename E>
__device__ __forceinline__ float to_f(E v);
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E>
__device__ __forceinline__ E from_f(float v);
template <>
__device__ __forceinline__ float from_f(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

// Two pieces of a unit: V pairs' values. Interleaved: 2 V consecutive values; halves: V values of the
// first half and the V matching ones of the second.
template <typename E, int V>
union Unit {
  E v[2 * V];
  uint4 w[sizeof(E) * V >= 16 ? 2 : 1];
};

template <typename E, int V, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Params p) {
  extern __shared__ float2 cs[];  // [per_cta][half]: scale * (cos, sin)
  const int t0 = blockIdx.x * p.per_cta;
  const int nt = min(p.per_cta, p.T - t0);
  const int groups = p.half / V;           // units of a head
  const int heads = p.H + p.H2;
  const int items = nt * heads * groups;
  constexpr bool kVec = V > 1;
  constexpr int kAhead = kVec ? 4 : 8;     // units in flight per thread
  Unit<E, V> u[kAhead];

  auto place = [&](int i, int& t, int& g, const E*& src, E*& dst) {
    const int th = i / groups;
    g = i - th * groups;
    t = th / heads;
    const int h = th - t * heads;
    const bool first = h < p.H;
    const Tensor& a = first ? p.a : p.b;
    const int64_t tt = t0 + t, hh = first ? h : h - p.H;
    src = reinterpret_cast<const E*>(a.x + tt * a.xt + hh * a.xh);
    dst = reinterpret_cast<E*>(a.out + tt * a.ot + hh * a.oh);
  };
  auto load = [&](Unit<E, V>& w, const E* src, int g) {
    const E* s0 = src + (kInterleaved ? 2 * V * g : V * g);
    const E* s1 = kInterleaved ? s0 + V : s0 + p.half;
    if constexpr (kVec) {
      w.w[0] = *reinterpret_cast<const uint4*>(s0);
      w.w[1] = *reinterpret_cast<const uint4*>(s1);
    } else {
      w.v[0] = *s0;
      w.v[1] = *s1;
    }
  };
  auto turn_store = [&](Unit<E, V>& w, E* dst, int t, int g) {
    const float2* c = cs + t * p.half + V * g;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int ia = kInterleaved ? 2 * k : k, ib = kInterleaved ? 2 * k + 1 : V + k;
      const float a = to_f(w.v[ia]), b = to_f(w.v[ib]);
      const float2 e = c[k];
      w.v[ia] = from_f<E>(a * e.x - b * e.y);
      w.v[ib] = from_f<E>(a * e.y + b * e.x);
    }
    E* d0 = dst + (kInterleaved ? 2 * V * g : V * g);
    E* d1 = kInterleaved ? d0 + V : d0 + p.half;
    if constexpr (kVec) {
      *reinterpret_cast<uint4*>(d0) = w.w[0];
      *reinterpret_cast<uint4*>(d1) = w.w[1];
    } else {
      *d0 = w.v[0];
      *d1 = w.v[1];
    }
  };

  // the first units' values are on their way while the angles are computed
  E* dst[kAhead];
  int ts[kAhead], gs[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < items) {
      const E* src;
      place(i, ts[k], gs[k], src, dst[k]);
      load(u[k], src, gs[k]);
    }
  }
  for (int i = threadIdx.x; i < nt * p.half; i += kThreads) {
    const int t = i / p.half, k = i - t * p.half;
    double f = p.inv_freq[k] * 0.15915494309189533577;  // turns per position
    f -= floor(f);
    const uint64_t step = (uint64_t)(f * 18446744073709551616.0);
    const int64_t at = (int64_t)((uint64_t)(int64_t)p.pos[t0 + t] * step);  // whole turns drop out
    float s, c;
    sincospif((float)at * 1.0842021724855044e-19f, &s, &c);  // 2^-63: half turns
    cs[i] = make_float2(c * p.scale, (p.inverse ? -s : s) * p.scale);
  }
  __syncthreads();
#pragma unroll 1
  for (int base = 0; base < items; base += kAhead * kThreads) {
    if (base > 0) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = base + threadIdx.x + k * kThreads;
        if (i < items) {
          const E* src;
          place(i, ts[k], gs[k], src, dst[k]);
          load(u[k], src, gs[k]);
        }
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (base + threadIdx.x + k * kThreads < items) turn_store(u[k], dst[k], ts[k], gs[k]);
  }
}

template <typename E, int V>
cudaError_t launch(const Params& p, bool interleaved, unsigned grid, size_t smem, cudaStream_t stream) {
  if (interleaved)
    rope_kernel<E, V, true><<<grid, kThreads, smem, stream>>>(p);
  else
    rope_kernel<E, V, false><<<grid, kThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rope

cudaError_t launch_rope(const hs_rope_args* a, int sms, cudaStream_t stream) {
  using namespace rope;
  const int64_t e = a->dtype == HS_FP32 ? 4 : 2;
  Params p;
  p.T = a->T;
  p.H = a->H;
  p.H2 = a->y ? a->H2 : 0;
  p.half = a->rot / 2;
  p.inverse = a->inverse;
  p.scale = a->scale;
  p.pos = a->positions;
  p.inv_freq = a->inv_freq;
  p.a = {(const uint8_t*)a->x, (uint8_t*)a->out, a->x_stride_t * e, a->x_stride_h * e, a->out_stride_t * e, a->out_stride_h * e};
  p.b = p.a;
  if (a->y)
    p.b = {(const uint8_t*)a->y, (uint8_t*)a->y_out, a->y_stride_t * e, a->y_stride_h * e, a->y_out_stride_t * e,
           a->y_out_stride_h * e};
  uint64_t bits = 0;  // every address and stride; a multiple of 16 bytes only if all are
  for (const Tensor* t : {&p.a, &p.b})
    bits |= (uint64_t)(uintptr_t)t->x | (uint64_t)(uintptr_t)t->out | (uint64_t)t->xt | (uint64_t)t->xh | (uint64_t)t->ot |
            (uint64_t)t->oh;
  const int V = e == 4 ? 4 : 8;
  const bool vec = (bits & 15) == 0 && p.half % V == 0;
  // Tokens per CTA: enough work for the loads in flight, while every SM still gets several CTAs.
  const int64_t units = (int64_t)(p.H + p.H2) * p.half / (vec ? V : 1);
  int per = 1;
  while (per < 8 && (int64_t)2 * per * units <= 4 * kThreads && (int64_t)a->T >= 2LL * per * 4 * sms) per *= 2;
  p.per_cta = per;
  const unsigned grid = (unsigned)((a->T + per - 1) / per);
  const size_t smem = (size_t)per * p.half * sizeof(float2);
  const bool il = a->interleaved != 0;
  switch (a->dtype) {
    case HS_FP32: return vec ? launch<float, 4>(p, il, grid, smem, stream) : launch<float, 1>(p, il, grid, smem, stream);
    case HS_FP16: return vec ? launch<__half, 8>(p, il, grid, smem, stream) : launch<__half, 1>(p, il, grid, smem, stream);
    default:
      return vec ? launch<__nv_bfloat16, 8>(p, il, grid, smem, stream) : launch<__nv_bfloat16, 1>(p, il, grid, smem, stream);
  }
}

}  // namespace hs
