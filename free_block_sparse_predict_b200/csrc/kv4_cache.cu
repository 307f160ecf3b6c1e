// Writing and reading a paged cache of K and V in 4 bits.
//
// Per group of 32, 64 or 128 channels: s = fp16(absmax / 7), code =
// clamp(rint(x / s), -7, 7) of the IEEE float32 quotient (the rule of the INT8
// predictor's codes, one scale per token and group instead of per block).
// HBM-bound: append reads 4d bytes of K and V per token and head and writes
// d + 4 d/group; read is the other way round.
//
// A CTA takes 16 rows of two (d = 128) or four heads, usually one tile of each,
// at most parts of 16.  A row of d channels is held by d/8 lanes, eight channels
// each; every second warp takes V's rows, the others K's, and every thread has
// four such pieces in flight.  K's codes of a token lie together and
// are stored as they are; V's lie 64 bytes apart, next to those of the tile's
// other tokens, so append gathers them in shared memory and stores them in the
// cache's order, and read takes them as the words they are, from L1 after the
// first token, and exchanges their bytes among the lanes.
//
// Measured: 33,000 tokens of 8 heads of 128 channels, in groups of 32, in and back
// in 76 us, 344 MB at 4.5 TB/s (69 % of a copy's rate; issue slots are busy for 76
// to 81 % of the cycles); 60 tokens of 12 heads in 5 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "after.cuh"
#include "kv4_layout.cuh"
#include "sm100_ptx.cuh"
#include "sparge_internal.h"

namespace sparge {
namespace {

constexpr int kCacheThreads = 256;

// Largest scale kept: a softmax weight of up to 4 times it stays below 65504.
constexpr float kMaxScale = 16376.0f;

// The larger magnitudes of two pairs, with some sign; a NaN where either is one.
template <int DT>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  if (DT == SPARGE_BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Within 2^-23 of 1 / x, relatively.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

struct CacheArgs {
  const char* k;
  const char* v;
  int64_t ks[2], vs[2];  // bytes between tokens and heads
  const int32_t* slots;
  uint8_t* cache;
  int32_t* status;
  int32_t T, slots_end;  // slots_end: num_pages * page_size
  int32_t Hkv, page, tpp, dtype;  // tpp: tiles per page
  uint32_t low4;  // 15; from a register, a mask and an or are one instruction
};

constexpr int kRows = 16;    // rows per CTA
constexpr int kPasses = 4;   // pieces per thread

template <int D>
struct CacheCfg {
  static constexpr int LANES = D / 8;                          // lanes per row
  static constexpr int PER_PASS = kCacheThreads / (2 * LANES);  // token-heads per pass
  static constexpr int HEADS = kPasses * PER_PASS / kRows;
};

// The CTA's slots: threads 0..15 find each row's tile of KV head 0 (a tile
// number; a head on is tpp tiles on) and its place in it, -1 for rows to skip.
__device__ __forceinline__ int32_t find_slot(const CacheArgs& A, int32_t t, int64_t* tile) {
  int32_t slot = t < A.T ? A.slots[t] : -1;
  if (uint32_t(slot) >= uint32_t(A.slots_end)) return -1;
  const int32_t page = slot / A.page, in = slot - page * A.page;
  *tile = int64_t(page) * A.Hkv * A.tpp + (in >> 4);
  return slot;
}
// A token's place in its tile: pages hold whole tiles.
__device__ __forceinline__ int token_of(int32_t slot) { return slot & 15; }

// Where a thread's piece of pass p stands: rows and heads behind its first.
template <int D>
struct Piece {
  static __device__ __forceinline__ constexpr int row(int p) {
    return p * CacheCfg<D>::PER_PASS % kRows;
  }
  static __device__ __forceinline__ constexpr int head(int p) {
    return p * CacheCfg<D>::PER_PASS / kRows;
  }
};

template <int D, int NG, int DT>
__global__ void __launch_bounds__(kCacheThreads) append_kernel(const CacheArgs A) {
  using C = CacheCfg<D>;
  constexpr int LANES = C::LANES;
  constexpr int GL = D / NG / 8;      // lanes per scale group
  constexpr int WORDS = D / 8;        // 32-bit words of V's codes per token
  constexpr int PITCH = kRows + 1;
  constexpr Kv4Tile L{D, NG};
  __shared__ int32_t s_slot[kRows];
  __shared__ int64_t s_tile[kRows];
  __shared__ int8_t s_order[kRows];   // rows in the order of their words in the cache
  __shared__ uint32_t s_v[C::HEADS][WORDS][PITCH];
  __shared__ __align__(16) __half s_scale[C::HEADS][kRows][2 * NG];

  begin_after();
  const int32_t row0 = int32_t(blockIdx.x) * kRows, head0 = int32_t(blockIdx.y) * C::HEADS;
  const bool is_v = threadIdx.x / 32 & 1;
  const int lane = threadIdx.x % LANES;
  const int at = threadIdx.x / 64 * (32 / LANES) + threadIdx.x % 32 / LANES;
  const char* src = (is_v ? A.v : A.k) + lane * 16;
  const int64_t st = is_v ? A.vs[0] : A.ks[0], sh_ = is_v ? A.vs[1] : A.ks[1];
  src += (row0 + at) * st + head0 * sh_;
  // the rows are asked for whatever their slots are: one latency, not two
  uint4 raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    raw[p] = make_uint4(0, 0, 0, 0);
    if (row0 + at + Piece<D>::row(p) < A.T && head0 + Piece<D>::head(p) < A.Hkv)
      raw[p] = *reinterpret_cast<const uint4*>(src + Piece<D>::row(p) * st + Piece<D>::head(p) * sh_);
  }
  if (threadIdx.x < 32) {
    int64_t tile = 0;
    const int32_t slot = threadIdx.x < kRows ? find_slot(A, row0 + int(threadIdx.x), &tile) : -1;
    const uint32_t key = uint32_t(slot & ~15) | uint32_t(Kv4Tile::v_pos(token_of(slot)));
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint32_t other = __shfl_sync(0xffffffffu, key, i);
      rank += other < key || (other == key && i < int(threadIdx.x));
    }
    if (threadIdx.x < kRows) {
      s_slot[threadIdx.x] = slot;
      s_tile[threadIdx.x] = tile;
      s_order[rank] = int8_t(threadIdx.x);
    }
  }
  __syncthreads();
  auto tile_at = [&](int row, int hd) {
    return A.cache + (s_tile[row] + int64_t(head0 + hd) * A.tpp) * L.bytes();
  };

#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = at + Piece<D>::row(p), hd = Piece<D>::head(p);
    const int32_t slot = s_slot[row];
    const bool there = slot >= 0 && head0 + hd < A.Hkv;
    const uint32_t u[4] = {raw[p].x, raw[p].y, raw[p].z, raw[p].w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (DT == SPARGE_BF16) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
    uint32_t big = max_abs<DT>(max_abs<DT>(u[0], u[1]), max_abs<DT>(u[2], u[3]));
#pragma unroll
    for (int o = 1; o < GL; o <<= 1) big = max_abs<DT>(big, __shfl_xor_sync(0xffffffffu, big, o));
    big = max_abs<DT>(big, big >> 16) & 0x7FFFu;
    float m = DT == SPARGE_BF16 ? __uint_as_float(big << 16)
                                : __half2float(__ushort_as_half(uint16_t(big)));
    // s = fp16(m / 7), the quotient correctly rounded by Markstein's step.
    const bool high = m > 7.0f * kMaxScale;  // as m / 7 > kMaxScale: false for a NaN
    if (high) {
      m = 7.0f * kMaxScale;
      if (there && A.status != nullptr) atomicCAS(A.status, 0, int32_t(SPARGE_ERANGE));
    }
    constexpr float kSeventh = 1.0f / 7.0f;
    const float m0 = m * kSeventh;
    const __half sh = __float2half_rn(fmaf(fmaf(-m0, 7.0f, m), kSeventh, m0));
    const float s = __half2float(sh);
    // Codes pass 7 only where s was saturated or, below fp16's normal range, far
    // from m / 7; a scale of 0 or NaN has codes 0.  Such groups clamp first.
    if (high || !(s >= 6.103515625e-05f)) {
      const float most = 7.25f * s;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = s > 0.f ? fminf(fmaxf(x[i], -most), most) : 0.f;
    }
    // Codes are those of the correctly rounded quotient, without it: x and s have at
    // most 11 bits and |x| < 8 s, so x / s is k + 1/2 or at least 2^-13 away from
    // it.  Rounded to a multiple of 2^-16 (in the sum with 192), x y with a reciprocal good
    // to 2^-22 falls on the halves exactly and on the right side elsewhere.  The
    // next sum's rounding makes it a whole number, plus 8: the low bits.  (Markstein's step
    // for each quotient took twice as many instructions, 80.4 instead of 76.4 us for
    // three prompts in and back; IEEE divisions three times all the others.)
    const float y = s > 0.f ? rcp_approx(s) : 0.f;
    const uint64_t y2 = pack2(y, y), grid = pack2(192.0f, 192.0f);
    uint32_t c[4];  // two codes each, in the two half-words
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t q = add2(fma2(pack2(x[2 * i], x[2 * i + 1]), y2, grid),
                              pack2(12582920.0f - 192.0f, 12582920.0f - 192.0f));
      c[i] = __byte_perm(uint32_t(q), uint32_t(q >> 32), 0x5410);
    }
    if (!is_v) {
      if (there)
        *reinterpret_cast<uint32_t*>(tile_at(row, hd) + L.k_word(token_of(slot), lane % 4, lane / 4)) =
            c[0] + (c[1] << 4) + (c[2] << 8) + (c[3] << 12);
    } else {
      // channels 8 lane .. + 7 lie in block lane / 2: byte (lane / 2) % 4 of the
      // words g = 4 (lane % 2) + 0..3
#pragma unroll
      for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint8_t*>(&s_v[hd][8 * (lane / 8) + 4 * (lane % 2) + i][row])[lane / 2 % 4] =
            uint8_t(c[i] | (c[i] >> 12));
    }
    if (lane % GL == 0) s_scale[hd][row][(is_v ? NG : 0) + lane / GL] = sh;
  }
  __syncthreads();

  // ---- V's words in the order of their addresses, then the scales
  for (int e = threadIdx.x; e < C::HEADS * WORDS * kRows; e += kCacheThreads) {
    const int row = s_order[e % kRows], word = e / kRows % WORDS, hd = e / (kRows * WORDS);
    const int32_t slot = s_slot[row];
    if (slot < 0 || head0 + hd >= A.Hkv) continue;
    *reinterpret_cast<uint32_t*>(tile_at(row, hd) + L.v_word(token_of(slot), word / 8, word % 8)) =
        s_v[hd][word][row];
  }
  for (int e = threadIdx.x; e < C::HEADS * kRows * NG; e += kCacheThreads) {
    const int n = e % NG, row = e / NG % kRows, hd = e / (NG * kRows);
    const int32_t slot = s_slot[row];
    if (slot < 0 || head0 + hd >= A.Hkv) continue;
    reinterpret_cast<uint32_t*>(tile_at(row, hd) + L.k_scale(token_of(slot)))[n] =
        reinterpret_cast<const uint32_t*>(s_scale[hd][row])[n];
  }
}

template <int D, int NG, int DT>
__global__ void __launch_bounds__(kCacheThreads) read_kernel(const CacheArgs A) {
  using C = CacheCfg<D>;
  constexpr int LANES = C::LANES;
  constexpr int GL = D / NG / 8;
  constexpr Kv4Tile L{D, NG};
  __shared__ int32_t s_slot[kRows];
  __shared__ int64_t s_tile[kRows];
  begin_after();
  const int32_t row0 = int32_t(blockIdx.x) * kRows, head0 = int32_t(blockIdx.y) * C::HEADS;
  const bool is_v = threadIdx.x / 32 & 1;
  const int lane = threadIdx.x % LANES;
  const int at = threadIdx.x / 64 * (32 / LANES) + threadIdx.x % 32 / LANES;
  if (threadIdx.x < kRows) {
    int64_t tile = 0;
    s_slot[threadIdx.x] = find_slot(A, row0 + int(threadIdx.x), &tile);
    s_tile[threadIdx.x] = tile;
  }
  __syncthreads();
  constexpr int ES = DT == SPARGE_F32 ? 4 : 2;
  char* dst = const_cast<char*>(is_v ? A.v : A.k);
  const bool wanted = dst != nullptr;
  const int64_t st = is_v ? A.vs[0] : A.ks[0], sh_ = is_v ? A.vs[1] : A.ks[1];
  dst += (row0 + at) * st + head0 * sh_ + lane * 8 * ES;
  // a lane's word: K's (t, j) of its own channels, V's word number `lane`
  uint32_t word[kPasses];
  __half sh[kPasses];
  bool there[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int row = at + Piece<D>::row(p), hd = Piece<D>::head(p);
    const int32_t slot = s_slot[row];
    there[p] = wanted && slot >= 0 && head0 + hd < A.Hkv;
    word[p] = 0;
    sh[p] = __ushort_as_half(0);
    if (there[p]) {
      const int tok = token_of(slot);
      const uint8_t* tile = A.cache + (s_tile[row] + int64_t(head0 + hd) * A.tpp) * L.bytes();
      word[p] = *reinterpret_cast<const uint32_t*>(
          tile + (is_v ? L.v_word(tok, lane / 8, lane % 8) : L.k_word(tok, lane % 4, lane / 4)));
      sh[p] = reinterpret_cast<const __half*>(
          tile + (is_v ? L.v_scale(tok) : L.k_scale(tok)))[lane / GL];
    }
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    // the codes, at the low end of z: V's are the two halves of byte (lane / 2) % 4
    // of the words 8 (lane / 8) + 4 (lane % 2) + 0..3, K's are all its word's
    uint32_t z[8];
    if (is_v) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[2 * i] = __shfl_sync(0xffffffffu, word[p], 8 * (lane / 8) + 4 * (lane % 2) + i, LANES) >>
                   (8 * (lane / 2 % 4));
        z[2 * i + 1] = z[2 * i] >> 4;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = word[p] >> (4 * (e / 2) + 16 * (e % 2));
    }
    if (!there[p]) continue;
    const float s = __half2float(sh[p]);
    const uint64_t s2 = pack2(s, s);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i += 2) {  // 2^23 + u, minus 2^23 + 8
      const uint64_t u = pack2(__uint_as_float((z[i] & A.low4) | 0x4B000000u),
                               __uint_as_float((z[i + 1] & A.low4) | 0x4B000000u));
      unpack2(mul2(add2(u, pack2(-8388616.0f, -8388616.0f)), s2), x[i], x[i + 1]);
    }
    char* to = dst + Piece<D>::row(p) * st + Piece<D>::head(p) * sh_;
    if (DT == SPARGE_F32) {
      reinterpret_cast<float4*>(to)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(to)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      uint32_t r[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (DT == SPARGE_BF16) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
          r[i] = *reinterpret_cast<const uint32_t*>(&h);
        } else {
          const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
          r[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
      }
      *reinterpret_cast<uint4*>(to) = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

template <bool READ, int D, int NG>
cudaError_t run(const CacheArgs& a, cudaStream_t stream) {
  const dim3 grid(unsigned(cdiv(a.T, kRows)), unsigned(cdiv(a.Hkv, CacheCfg<D>::HEADS)));
  const auto go = [&](auto* kernel) {
    return launch_after(kernel, grid, kCacheThreads, 0, stream, a);
  };
  if (a.dtype == SPARGE_F16)
    return READ ? go(read_kernel<D, NG, SPARGE_F16>) : go(append_kernel<D, NG, SPARGE_F16>);
  if (a.dtype == SPARGE_BF16)
    return READ ? go(read_kernel<D, NG, SPARGE_BF16>) : go(append_kernel<D, NG, SPARGE_BF16>);
  return READ ? go(read_kernel<D, NG, SPARGE_F32>) : cudaErrorNotSupported;
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
  a.T = T;
  a.slots_end = c.num_pages * c.page_size;
  a.Hkv = c.Hkv;
  a.page = c.page_size;
  a.tpp = c.page_size / 16;
  a.dtype = dtype;
  a.low4 = 15;
  return read ? pick<true>(c, a, stream) : pick<false>(c, a, stream);
}

}  // namespace sparge
