// Rotary positions with several axes: pair (u, v) of channel pair i turns by
// a = pos[axis_i] * inv_freq_i, so that the score of two turned rows depends
// on the difference of their positions along every axis.  The Hilbert table
// may name the source rows (or, in the inverse, the destination rows), which
// saves the permutation pass of its own, and both tensors are strided, so the
// pass from a projection's [B, N, H, d] to the library's [B, H, N, d] is free.
//
// HBM-bound: every row is read once and written once.  A thread owns two
// 16-byte vectors of a row that hold whole pairs (the two halves' vectors, or
// two neighbours when interleaved) and keeps their sines and cosines in
// registers over up to eight heads: the angles do not depend on the head, and at
// one sincospi per pair and row they would cost as much as the copy.  The
// product pos * inv_freq is taken in float64 turns and reduced there; only
// the fraction of a turn goes to float32.  Measured: 32 heads of 128 channels and
// 131,072 tokens in 348 us, 6.2 TB/s, 94 % of what a copy reaches; 64 tokens in 3 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "after.cuh"
#include "sparge_internal.h"

namespace sparge {
namespace {

constexpr int kRopeThreads = 256;
// Three CTAs a SM (80 registers): two left the loads too few (414 us for the
// 1.07 GB of a 128K prompt's queries against 349), four spilled (384 us).
constexpr int kRopeCtas = 3;
constexpr int kBatch = 4;  // heads whose vectors are in flight at once

template <int DT>
struct RopeType;
template <>
struct RopeType<SPARGE_F16> {
  static constexpr int V = 8;  // elements per 16-byte vector
  static __device__ __forceinline__ void load(const uint4& r, float (&f)[8]) {
    const __half2* h = reinterpret_cast<const __half2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = __half22float2(h[i]);
      f[2 * i] = a.x;
      f[2 * i + 1] = a.y;
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint4 r;
    __half2* h = reinterpret_cast<__half2*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    return r;
  }
};
template <>
struct RopeType<SPARGE_BF16> {
  static constexpr int V = 8;
  static __device__ __forceinline__ void load(const uint4& r, float (&f)[8]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(u[i] << 16);
      f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[8]) {
    uint4 r;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return r;
  }
};
template <>
struct RopeType<SPARGE_F32> {
  static constexpr int V = 4;
  static __device__ __forceinline__ void load(const uint4& r, float (&f)[4]) {
    f[0] = __uint_as_float(r.x);
    f[1] = __uint_as_float(r.y);
    f[2] = __uint_as_float(r.z);
    f[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ uint4 store(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

struct RopeArgs {
  const char* src;
  char* dst;
  const int32_t* pos;
  const double* inv_freq;
  const int32_t* axis;
  const int32_t* perm;
  int64_t ss[3], ds[3];  // bytes between batches, heads, tokens
  int64_t pos_stride;
  int32_t B, H, N, vecs;  // vecs: 16-byte vectors of a row
  int32_t rvecs;          // vectors that turn (even)
  int32_t units;          // threads per row: each takes two vectors
  int32_t axes, heads;    // heads per thread
  int32_t groups;         // ceil(H / heads)
  int32_t inverse;
};

// One thread's V pairs in place: rows' vectors a and b, cosines and sines.
template <int DT, bool IL>
__device__ __forceinline__ void turn_pairs(uint4& ra, uint4& rb, const float* cs,
                                           const float* sn) {
  using T = RopeType<DT>;
  constexpr int V = T::V;
  float a[V], c[V];
  T::load(ra, a);
  T::load(rb, c);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    float& u = IL ? (k < V / 2 ? a[2 * k] : c[2 * k - V]) : a[k];
    float& v = IL ? (k < V / 2 ? a[2 * k + 1] : c[2 * k + 1 - V]) : c[k];
    const float u0 = u, v0 = v;
    u = u0 * cs[k] - v0 * sn[k];
    v = u0 * sn[k] + v0 * cs[k];
  }
  ra = T::store(a);
  rb = T::store(c);
}

template <int DT, bool IL>
__global__ void __launch_bounds__(kRopeThreads, kRopeCtas) rope_kernel(const RopeArgs P) {
  using T = RopeType<DT>;
  constexpr int V = T::V;
  begin_after();
  const int64_t item = int64_t(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int32_t p = int32_t(item / P.units);
  const int32_t u = int32_t(item - int64_t(p) * P.units);
  if (p >= P.N) return;
  const int32_t s = P.perm == nullptr ? p : P.perm[p];
  if (uint32_t(s) >= uint32_t(P.N)) return;

  // the two vectors of this thread; vectors behind the turned ones are copied
  const bool turn = 2 * u < P.rvecs;
  int32_t va, vb;
  if (turn) {
    va = IL ? 2 * u : u;
    vb = IL ? 2 * u + 1 : u + P.rvecs / 2;
  } else {
    va = 2 * u;
    vb = 2 * u + 1;
  }
  const bool two = vb < P.vecs;

  for (int32_t bg = blockIdx.y; bg < P.B * P.groups; bg += gridDim.y) {
    const int32_t b = bg / P.groups, g = bg - b * P.groups;
    const int32_t h1 = min(P.H, (g + 1) * P.heads);
    const char* src = P.src + b * P.ss[0] + int64_t(P.inverse ? p : s) * P.ss[2];
    char* dst = P.dst + b * P.ds[0] + int64_t(P.inverse ? s : p) * P.ds[2];
    // kBatch heads' loads before their stores: x and y may be one tensor (each
    // vector is touched by one thread only), so the compiler keeps the order
    uint4 ra[kBatch], rb[kBatch];
    auto load = [&](int32_t h0) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (h0 + i < h1) {
          const uint4* x = reinterpret_cast<const uint4*>(src + (h0 + i) * P.ss[1]);
          ra[i] = x[va];
          if (two) rb[i] = x[vb];
        }
      }
    };
    load(g * P.heads);  // in flight while the angles are computed
    float cs[V], sn[V];
    if (turn) {
      const int32_t* pos = P.pos + b * P.pos_stride;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int32_t pair = u * V + k;
        const int32_t ax = P.axis[pair];
        const double at =
            uint32_t(ax) < uint32_t(P.axes) ? double(pos[int64_t(ax) * P.N + s]) : 0.0;
        // 1 / (2 pi): turns, then the nearest whole turn off
        const double t = at * (P.inv_freq[pair] * 0.15915494309189535);
        const float f = float(2.0 * (t - rint(t)));
        sincospif(f, &sn[k], &cs[k]);
        if (P.inverse) sn[k] = -sn[k];
      }
    }
    for (int32_t h0 = g * P.heads; h0 < h1; h0 += kBatch) {
      if (h0 > g * P.heads) load(h0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (h0 + i >= h1) break;
        if (turn) turn_pairs<DT, IL>(ra[i], rb[i], cs, sn);
        uint4* y = reinterpret_cast<uint4*>(dst + (h0 + i) * P.ds[1]);
        y[va] = ra[i];
        if (two) y[vb] = rb[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const sparge_rope_t& p, const void* src, const int64_t* src_stride,
                        void* dst, const int64_t* dst_stride, const int32_t* pos,
                        const double* inv_freq, const int32_t* axis, const int32_t* perm,
                        bool inverse, cudaStream_t stream) {
  const int32_t es = p.dtype == SPARGE_F32 ? 4 : 2;
  RopeArgs a{};
  a.src = static_cast<const char*>(src);
  a.dst = static_cast<char*>(dst);
  a.pos = pos;
  a.inv_freq = inv_freq;
  a.axis = axis;
  a.perm = perm;
  for (int i = 0; i < 3; ++i) {
    a.ss[i] = src_stride[i];
    a.ds[i] = dst_stride[i];
  }
  a.pos_stride = p.pos_stride;
  a.B = p.B;
  a.H = p.H;
  a.N = p.N;
  a.vecs = p.d * es / 16;
  a.rvecs = p.rot * es / 16;
  a.units = (a.vecs + 1) / 2;
  a.axes = p.axes;
  a.inverse = inverse ? 1 : 0;
  const int64_t gx = cdiv(int64_t(p.N) * a.units, kRopeThreads);
  // Eight heads share a thread's angles where that still leaves every SM
  // eight blocks; small problems spread over the heads instead.
  a.heads = 8;
  while (a.heads > 1 && gx * p.B * cdiv(p.H, a.heads) < 8 * 148) a.heads >>= 1;
  a.groups = int32_t(cdiv(p.H, a.heads));
  const int64_t gy = int64_t(p.B) * a.groups;
  const dim3 grid{unsigned(gx), unsigned(gy < 65535 ? gy : 65535), 1u};
  cudaError_t e;
  if (p.dtype == SPARGE_F16) {
    if (p.interleaved)
      e = launch_after(rope_kernel<SPARGE_F16, true>, grid, kRopeThreads, 0, stream, a);
    else
      e = launch_after(rope_kernel<SPARGE_F16, false>, grid, kRopeThreads, 0, stream, a);
  } else if (p.dtype == SPARGE_BF16) {
    if (p.interleaved)
      e = launch_after(rope_kernel<SPARGE_BF16, true>, grid, kRopeThreads, 0, stream, a);
    else
      e = launch_after(rope_kernel<SPARGE_BF16, false>, grid, kRopeThreads, 0, stream, a);
  } else {
    if (p.interleaved)
      e = launch_after(rope_kernel<SPARGE_F32, true>, grid, kRopeThreads, 0, stream, a);
    else
      e = launch_after(rope_kernel<SPARGE_F32, false>, grid, kRopeThreads, 0, stream, a);
  }
  return e;
}

}  // namespace sparge
