// Writing and reading a paged cache of K and V in 4 bits.
//
// Per group of 32, 64 or 128 channels: s = fp16(absmax / 7), code =
// clamp(rint(x / s), -7, 7) of the IEEE float32 quotient (the rule of the INT8
// predictor's codes, one scale per token and group instead of per block).
// HBM-bound: append reads 4d bytes of K and V per token and head and writes
// d + 4 d/group; read is the other way round.
//
// A row of d channels is held by d/8 lanes, eight channels each, K's row by
// the lower half of 2 d/8 lanes and V's by the upper: a warp holds one (d =
// 128) or two (d = 64) token-heads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kv4_layout.cuh"
#include "sparge_internal.h"

namespace sparge {
namespace {

constexpr int kCacheThreads = 256;

// Largest scale kept: a softmax weight of up to 4 times it stays below 65504.
constexpr float kMaxScale = 16376.0f;

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

struct CacheArgs {
  const char* k;
  const char* v;
  int64_t ks[2], vs[2];  // bytes between tokens and heads
  const int32_t* slots;
  uint8_t* cache;
  int32_t* status;
  int64_t items;  // T * Hkv
  int32_t slots_end;  // num_pages * page_size
  int32_t Hkv, page, tpp, dtype;  // tpp: tiles per page
};

// Where a (token, head) lives: its tile's address and its place in the tile.
__device__ __forceinline__ uint8_t* tile_of(const CacheArgs& A, int32_t slot, int32_t head,
                                            int32_t tile_bytes, int* tok) {
  const int32_t page = slot / A.page, in = slot - page * A.page;
  *tok = in & 15;
  return A.cache + (((int64_t(page) * A.Hkv + head) * A.tpp) + (in >> 4)) * tile_bytes;
}

template <int D, int NG>
__global__ void __launch_bounds__(kCacheThreads) append_kernel(const CacheArgs A) {
  constexpr int LANES = D / 8;        // lanes per row
  constexpr int GL = D / NG / 8;      // lanes per scale group
  constexpr Kv4Tile L{D, NG};
  const int64_t thread = int64_t(blockIdx.x) * kCacheThreads + threadIdx.x;
  const int64_t item = thread / (2 * LANES);
  const bool is_v = (threadIdx.x / LANES) & 1;
  const int lane = threadIdx.x % LANES;
  const int32_t t = int32_t(item / A.Hkv), head = int32_t(item - int64_t(t) * A.Hkv);
  const int32_t slot = item < A.items ? A.slots[t] : -1;
  const bool there = uint32_t(slot) < uint32_t(A.slots_end);

  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (there) {
    const char* src = is_v ? A.v + t * A.vs[0] + head * A.vs[1] : A.k + t * A.ks[0] + head * A.ks[1];
    const uint4 raw = *reinterpret_cast<const uint4*>(src + lane * 16);
    const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (A.dtype == SPARGE_BF16) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
#pragma unroll
  for (int o = 1; o < GL; o <<= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  float sf = __fdiv_rn(m, 7.0f);
  if (sf > kMaxScale) {  // false for a NaN
    sf = kMaxScale;
    if (there && A.status != nullptr) atomicCAS(A.status, 0, int32_t(SPARGE_ERANGE));
  }
  const __half sh = __float2half_rn(sf);
  const float s = __half2float(sh);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // a scale of 0 or NaN has codes 0
    const float q = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x[i], s)), -7.f), 7.f) : 0.f;
    c[i] = uint32_t(int(q) + 8);
  }
  if (!there) return;
  int tok;
  uint8_t* tile = tile_of(A, slot, head, L.bytes(), &tok);
  if (!is_v) {
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) w |= c[e] << (4 * (e / 2) + 16 * (e % 2));
    *reinterpret_cast<uint32_t*>(tile + L.k_word(tok, lane % 4, lane / 4)) = w;
  } else {
    // channels 8 lane .. + 7 of block lane / 2: g = 4 (lane % 2) + 0..3
#pragma unroll
    for (int i = 0; i < 4; ++i)
      tile[L.v_word(tok, lane / 8, 4 * (lane % 2) + i) + (lane / 2) % 4] =
          uint8_t(c[2 * i] | (c[2 * i + 1] << 4));
  }
  if (lane % GL == 0)
    reinterpret_cast<__half*>(tile + (is_v ? L.v_scale(tok) : L.k_scale(tok)))[lane / GL] = sh;
}

template <int D, int NG>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const CacheArgs A) {
  constexpr int LANES = D / 8;
  constexpr int GL = D / NG / 8;
  constexpr Kv4Tile L{D, NG};
  const int64_t thread = int64_t(blockIdx.x) * kCacheThreads + threadIdx.x;
  const int64_t item = thread / (2 * LANES);
  const bool is_v = (threadIdx.x / LANES) & 1;
  const int lane = threadIdx.x % LANES;
  if (item >= A.items) return;
  const int32_t t = int32_t(item / A.Hkv), head = int32_t(item - int64_t(t) * A.Hkv);
  const int32_t slot = A.slots[t];
  const char* base = is_v ? A.v : A.k;
  if (uint32_t(slot) >= uint32_t(A.slots_end) || base == nullptr) return;
  int tok;
  const uint8_t* tile = tile_of(A, slot, head, L.bytes(), &tok);
  uint32_t c[8];
  if (!is_v) {
    const uint32_t w =
        *reinterpret_cast<const uint32_t*>(tile + L.k_word(tok, lane % 4, lane / 4));
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = (w >> (4 * (e / 2) + 16 * (e % 2))) & 15u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = tile[L.v_word(tok, lane / 8, 4 * (lane % 2) + i) + (lane / 2) % 4];
      c[2 * i] = b & 15u;
      c[2 * i + 1] = b >> 4;
    }
  }
  const float s = __half2float(
      reinterpret_cast<const __half*>(tile + (is_v ? L.v_scale(tok) : L.k_scale(tok)))[lane / GL]);
  float x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = float(int(c[i]) - 8) * s;
  const int64_t off = is_v ? t * A.vs[0] + head * A.vs[1] : t * A.ks[0] + head * A.ks[1];
  char* dst = const_cast<char*>(base) + off + lane * (A.dtype == SPARGE_F32 ? 32 : 16);
  if (A.dtype == SPARGE_F32) {
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint4 r;
    uint32_t* u = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (A.dtype == SPARGE_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        u[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(dst) = r;
  }
}

template <bool READ, int D, int NG>
cudaError_t run(const CacheArgs& a, cudaStream_t stream) {
  const int64_t blocks = cdiv(a.items * (2 * D / 8), kCacheThreads);
  if (blocks > INT32_MAX) return cudaErrorNotSupported;
  if (READ)
    read_kernel<D, NG><<<unsigned(blocks), kCacheThreads, 0, stream>>>(a);
  else
    append_kernel<D, NG><<<unsigned(blocks), kCacheThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <bool READ>
cudaError_t pick(const sparge_kv4_t& c, const CacheArgs& a, cudaStream_t s) {
  const int ng = c.d / c.group;
  if (c.d == 64) return ng == 2 ? run<READ, 64, 2>(a, s) : run<READ, 64, 1>(a, s);
  if (ng == 4) return run<READ, 128, 4>(a, s);
  return ng == 2 ? run<READ, 128, 2>(a, s) : run<READ, 128, 1>(a, s);
}

}  // namespace

cudaError_t launch_kv4_cache(const sparge_kv4_t& c, bool read, int32_t T, void* k,
                             const int64_t* ks, void* v, const int64_t* vs,
                             sparge_dtype_t dtype, const int32_t* slots, void* cache,
                             int32_t* status, cudaStream_t stream) {
  CacheArgs a{};
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  for (int i = 0; i < 2; ++i) a.ks[i] = ks[i], a.vs[i] = vs[i];
  a.slots = slots;
  a.cache = static_cast<uint8_t*>(cache);
  a.status = status;
  a.items = int64_t(T) * c.Hkv;
  a.slots_end = c.num_pages * c.page_size;
  a.Hkv = c.Hkv;
  a.page = c.page_size;
  a.tpp = c.page_size / 16;
  a.dtype = dtype;
  return read ? pick<true>(c, a, stream) : pick<false>(c, a, stream);
}

}  // namespace sparge
