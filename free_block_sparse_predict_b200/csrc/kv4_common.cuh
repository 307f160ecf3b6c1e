// Shared by the kernels that attend over the 4-bit cache: their arguments, the
// line of work units that is cut over the CTAs, and the codes' way into fp16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "div.cuh"
#include "sm100_ptx.cuh"
#include "sparge_internal.h"

namespace sparge {
namespace kv4 {

constexpr int kSms = 148;
// "No key yet": finite, so that differences stay numbers, and below every finite score
// (scales reach 2^100).
constexpr float kLow = -3.402823466e38f;

struct Masks {
  uint32_t low, high, mixed;  // 0x000F000F, 0x00F000F0, 0x00F0000F
};
struct DecodeArgs {
  const char* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* cu;
  char* o;
  float* lse;
  float* part_o;      // [2 C][rows of a unit][d]: a CTA's first and last unit
  float2* part_ml;    // [2 C][rows of a unit]: maximum (log2) and sum
  uint32_t* arrived;  // [C]: parts of the unit that starts in CTA c; 0 between calls
  int32_t* status;
  int64_t q_stride;  // bytes
  int32_t R, T, Hq, Hkv, max_q, max_pages, len_cap, causal, num_pages, bf16;
  int32_t min_rows, max_rows;  // requests with rows (tokens times G) outside are another kernel's
  Div G, heads, tpp;  // query heads per KV head, KV heads, tiles per page
  Masks masks;
  float scale_log2;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The codes at bits 0-3 and 4-7 of both half-words, as fp16 pairs.
__device__ __forceinline__ uint32_t minus(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
__device__ __forceinline__ uint32_t times(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
// (w & mask) | magic; a LOP3 takes one immediate, so the mask is in a register
// whose value the compiler does not know (it would make two instructions of it)
__device__ __forceinline__ uint32_t pick(uint32_t w, uint32_t mask, uint32_t magic) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
  return d;
}
__device__ __forceinline__ uint32_t codes0(uint32_t w, const Masks& k) {
  return minus(pick(w, k.low, 0x64006400u), 0x64086408u);  // 1024 + u, 1032
}
__device__ __forceinline__ uint32_t codes4(uint32_t w, const Masks& k) {
  return minus(pick(w, k.high, 0x54005400u), 0x54805480u);  // 64 + u, 72
}
__device__ __forceinline__ float2 half2_f(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Request r's rows and keys, as every kernel here takes them.
struct Request {
  int32_t q0, qlen, len, keys;  // first row, rows, length, keys in reach
  bool sound;
};
__device__ __forceinline__ Request request(const DecodeArgs& A, int r) {
  Request x;
  x.q0 = A.cu[r];
  const int32_t q1 = A.cu[r + 1];
  x.len = A.seq_len[r];
  x.sound = x.q0 >= 0 && q1 >= x.q0 && q1 <= A.T && q1 - x.q0 <= A.max_q;
  x.qlen = x.sound ? q1 - x.q0 : 0;
  if (x.len < 0 || x.len > A.len_cap) x.sound = false;
  x.keys = x.len < 0 ? 0 : (x.len > A.len_cap ? A.len_cap : x.len);
  return x;
}

// Length of request r's units in steps of KEYS keys (a unit without keys still
// has its rows to write), and how many there are.
template <int KEYS>
__device__ __forceinline__ int64_t unit_steps(const Request& x) {
  return x.keys > 0 ? (int64_t(x.keys) + KEYS - 1) / KEYS : 1;
}
template <int ROWS>
__device__ __forceinline__ int64_t unit_count(const DecodeArgs& A, const Request& x) {
  const int64_t rows = int64_t(x.qlen) * A.G.d;
  if (rows < A.min_rows || rows > A.max_rows) return 0;
  return int64_t(A.Hkv) * ((rows + ROWS - 1) / ROWS);
}

// a / b, in 32 bits where both fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  return (a | b) >> 32 ? a / b : int64_t(uint32_t(a) / uint32_t(b));
}


// Row `row` (query token times head of the group) of a request and KV head in q and o.
__device__ __forceinline__ int64_t out_row(const DecodeArgs& A, const Request& x, int kvh, int row) {
  const int tok = A.G.quot(row);
  return int64_t(x.q0 + tok) * A.Hq + kvh * int(A.G.d) + (row - tok * int(A.G.d));
}

// One row's final value pair and, from the thread of its first channel, lse.
__device__ __forceinline__ void write_out(const DecodeArgs& A, int64_t at, int D, int ch, float top,
                                          float sum, float x, float y) {
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  if (sum == 0.f) x = y = 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(A.o) + (at * D + ch) / 2;
  if (A.bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x * inv, y * inv);
    *dst = *reinterpret_cast<const uint32_t*>(&h);
  } else {
    *dst = pack_half2(x * inv, y * inv);
  }
  if (ch == 0 && A.lse != nullptr)
    A.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

// Many rows per request, kv4_piece.cu: rows of its units, and its launch.
constexpr int kPieceRows = 256;
cudaError_t launch_kv4_piece(const DecodeArgs& a, int d, int ng, int grid, cudaStream_t s);

}  // namespace kv4
}  // namespace sparge
