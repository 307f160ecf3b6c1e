// Attention of new tokens over the paged 4-bit cache (include/sparge.h,
// sparge_kv4_attn): o = sum_n softmax_n(scale q.k_n) v_n with k_n = s c the
// values that codes c and group scales s stand for.
//
// Few query rows meet many keys, so the cache's bytes bound it: d + 4 d/group
// per token and KV head.  The codes are never turned into a tensor of their
// own: they go from shared memory straight into tensor-core fragments.
//   S^T = K Q^T   m16n8k16, rows = 16 keys, columns = 8 query rows (query
//                 tokens times the heads of the group)
//   O^T = V^T P^T m16n8k16, rows = 16 channels, k = 16 keys
// mma.sync, not tcgen05: the codes have to pass through registers anyway, and
// eight or sixteen query rows leave the tensor pipe idle either way.
//
// A code u = c + 8 becomes an fp16 in two steps, both exact: the four bits are
// masked into the mantissa of 1024 (bits 0-3) or of 64 (bits 4-7), one LOP3 for
// a pair, and the 1024 + 8 or 64 + 8 is subtracted, one HADD2.  (Masking alone
// gives the subnormal u 2^-24, which the tensor cores multiply too, but they
// align sums by the exponent field: measured, that cost seven bits of them.)
//
// Scales: S is summed per group in float32, S = sum_g s_g S_g.  V's scale
// goes into the weights, p s rounded to fp16 once.  Q is fp16 with one power
// of two per row, so bf16 queries lose nothing above 2^-26 of the row's
// largest.  The running maximum is lazy: it is raised (and O rescaled) when a
// score passes it by more than 2 in log2 units, so weights stay below 4 and
// p s below 65504.
//
// A CTA of four warps takes a chunk of one request's keys for one KV head and
// 8 NT query rows; each warp streams its own 16-token tiles through a ring of
// bulk copies.  The warps' results are joined in shared memory, chunks by a
// second kernel, in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "kv4_layout.cuh"
#include "sm100_ptx.cuh"
#include "sparge_internal.h"

namespace sparge {
namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kStages = 4;         // tiles in flight per warp
constexpr int kMaxChunk = 2048;    // tiles per CTA at most
constexpr float kLow = -1e30f;     // "no key yet"; finite, so differences stay numbers
constexpr float kLazy = 2.0f;      // log2 units

struct DecodeArgs {
  const char* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* seq_len;
  const int32_t* cu;
  char* o;
  float* lse;
  float* part_o;   // [T * Hq][splits][d]
  float2* part_ml; // [T * Hq][splits] maximum (log2) and sum
  int32_t* status;
  int64_t q_stride;  // bytes
  int32_t T, Hq, Hkv, G, max_q, max_pages, len_cap, causal, page, tpp, num_pages;
  int32_t splits, chunk;  // chunk: tiles
  int32_t bf16;
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

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The codes at bits 0-3 and 4-7 of both half-words, as fp16 pairs.
__device__ __forceinline__ uint32_t minus(uint32_t x, uint32_t y) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(x), "r"(y));
  return d;
}
__device__ __forceinline__ uint32_t codes0(uint32_t w) {
  return minus((w & 0x000F000Fu) | 0x64006400u, 0x64086408u);  // 1024 + u, 1032
}
__device__ __forceinline__ uint32_t codes4(uint32_t w) {
  return minus((w & 0x00F000F0u) | 0x54005400u, 0x54805480u);  // 64 + u, 72
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

template <int D, int NG, int NT>
struct Cfg {
  static constexpr int TILE = 16 * (D + 4 * NG);
  static constexpr int ROWS = 8 * NT;
  static constexpr int PITCH = D + 4;  // floats per row of the joining buffer
  static constexpr int RING = kStages * TILE;
  static_assert(ROWS * PITCH * 4 <= RING, "a warp's result fits its ring");
  static_assert(TILE % 16 == 0, "bulk copies");
  static int smem(int chunk) { return kWarps * RING + chunk * 4; }
};

template <int D, int NG, int NT>
__global__ void __launch_bounds__(kAttnThreads) kv4_attn_kernel(const DecodeArgs A) {
  using C = Cfg<D, NG, NT>;
  constexpr int J = D / 32;       // words of a token's codes per lane
  constexpr int JG = J / NG;      // of them per scale group
  constexpr int MT = D / 16;      // output row tiles
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kWarps][kStages];
  __shared__ float2 s_ml[kWarps][C::ROWS];
  __shared__ int abort_flag;
  int32_t* s_tile = reinterpret_cast<int32_t*>(smem + kWarps * C::RING);
  volatile int* abort = &abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int split = blockIdx.x, r = blockIdx.z;
  const int kvh = blockIdx.y % A.Hkv, rt = blockIdx.y / A.Hkv;

  const Request req = request(A, r);
  if (!req.sound && split == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    atomicCAS(A.status, 0, int32_t(SPARGE_EINVAL));
  const int rows = req.qlen * A.G, row0 = rt * C::ROWS;
  if (row0 >= rows) return;
  // the last position that any row of this tile sees
  const int last_row = min(row0 + C::ROWS, rows) - 1;
  const int32_t reach =
      A.causal ? min(req.keys, req.len - req.qlen + last_row / A.G + 1) : req.keys;
  const int t_begin = split * A.chunk;
  if (split > 0 && int64_t(t_begin) * 16 >= req.keys) return;
  const int n_tiles = max(0, min(A.chunk, (reach + 15) / 16 - t_begin));

  for (int i = threadIdx.x; i < n_tiles; i += kAttnThreads) {
    const int32_t ti = t_begin + i;
    const int32_t page = A.table[int64_t(r) * A.max_pages + ti / A.tpp];
    const bool ok = uint32_t(page) < uint32_t(A.num_pages);
    s_tile[i] = ok ? (page * A.Hkv + kvh) * A.tpp + ti % A.tpp : -1;
    if (!ok) atomicCAS(A.status, 0, int32_t(SPARGE_EINVAL));
  }
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) mbar_init(&full[w][s], 1);
    fence_mbar_init();
    fence_async_shared();
  }
  __syncthreads();

  uint8_t* ring = smem + warp * C::RING;
  // tile i of this warp is tile warp + kWarps * i of the chunk
  const int mine = n_tiles > warp ? (n_tiles - warp + kWarps - 1) / kWarps : 0;
  auto issue = [&](int i) {
    if (i < mine && lane == 0) {
      uint64_t* bar = &full[warp][i % kStages];
      const int32_t id = s_tile[warp + kWarps * i];
      if (id < 0) {
        mbar_arrive(bar);  // nothing to copy: its keys are left out
      } else {
        mbar_expect_tx(bar, C::TILE);
        bulk_load(ring + (i % kStages) * C::TILE, A.cache + int64_t(id) * C::TILE, C::TILE, bar);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < kStages; ++i) issue(i);

  // ---- Q as B fragments: column g is query row row0 + 8 nt + g; the 32-bit
  // word (t, j) of a token's codes meets channels 32 j + 8 t .. + 7
  uint32_t qf[NT][2 * J][2];
  float f[NT][2];               // score of a column: f * sum_g s_g S_g, in log2 units
  int32_t lim[NT][2];           // the column sees keys below this
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = row0 + 8 * nt + g;
    const bool there = row < rows;
    const int tok = there ? row / A.G : 0, head = kvh * A.G + (there ? row % A.G : 0);
    const char* src = A.q + int64_t(req.q0 + tok) * A.q_stride + int64_t(head) * (D * 2);
    float x[J][8];
    float big = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (there) raw = *reinterpret_cast<const uint4*>(src + (32 * j + 8 * t) * 2);
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (A.bf16) {
          x[j][2 * i] = __uint_as_float(u[i] << 16);
          x[j][2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
          const float2 h = half2_f(u[i]);
          x[j][2 * i] = h.x;
          x[j][2 * i + 1] = h.y;
        }
        big = fmaxf(big, fmaxf(fabsf(x[j][2 * i]), fabsf(x[j][2 * i + 1])));
      }
    }
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
    big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
    // the row's largest goes to [2^12, 2^13): two factors, since one may overflow
    int k = 0;
    if (big > 0.f && big < INFINITY) k = 12 - ilogbf(big);
    const float k1 = ldexpf(1.f, k / 2), k2 = ldexpf(1.f, k - k / 2);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qf[nt][2 * j + i / 2][i & 1] = pack_half2(x[j][2 * i] * k1 * k2, x[j][2 * i + 1] * k1 * k2);
    const float fr = A.scale_log2 * ldexpf(1.f, -k);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int from = (2 * t + c) * 4;  // a lane that holds column 2t + c as its g
      f[nt][c] = __shfl_sync(0xffffffffu, fr, from);
      const int row_c = row0 + 8 * nt + 2 * t + c;
      lim[nt][c] = 0;
      if (row_c < rows)
        lim[nt][c] =
            A.causal ? min(req.keys, req.len - req.qlen + row_c / A.G + 1) : req.keys;
    }
  }
  // tiles below this are seen by every row that is there
  int32_t all_see = req.keys;
  if (A.causal) all_see = min(all_see, req.len - req.qlen + row0 / A.G + 1);

  float m[NT][2], l[NT][2];
  float o[NT][MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) m[nt][c] = kLow, l[nt][c] = 0.f;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
  }

  bool ok = true;
  for (int i = 0; i < mine; ++i) {
    const int stage = i % kStages;
    ok = __all_sync(0xffffffffu,
                    mbar_wait(&full[warp][stage], (i / kStages) & 1, abort, A.status));
    if (!ok) break;
    const uint8_t* tile = ring + stage * C::TILE;
    const int32_t key0 = (t_begin + warp + kWarps * i) * 16;
    const bool copied = s_tile[warp + kWarps * i] >= 0;
    const bool whole = copied && key0 + 16 <= all_see;

    // ---- scales of tokens g and g + 8
    float sk[2][NG], sv[2][NG];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      const __half* s = reinterpret_cast<const __half*>(tile + 16 * D + (g + 8 * a) * NG * 4);
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        sk[a][n] = __half2float(s[n]);
        sv[a][n] = __half2float(s[NG + n]);
      }
    }
    // ---- S^T
    uint32_t ka[J], kb[J];
    if (J == 4) {
      const uint4 wa = *reinterpret_cast<const uint4*>(tile + g * (D / 2) + t * 16);
      const uint4 wb = *reinterpret_cast<const uint4*>(tile + (g + 8) * (D / 2) + t * 16);
      ka[0] = wa.x, ka[1] = wa.y, ka[J - 2] = wa.z, ka[J - 1] = wa.w;
      kb[0] = wb.x, kb[1] = wb.y, kb[J - 2] = wb.z, kb[J - 1] = wb.w;
    } else {
      const uint2 wa = *reinterpret_cast<const uint2*>(tile + g * (D / 2) + t * 8);
      const uint2 wb = *reinterpret_cast<const uint2*>(tile + (g + 8) * (D / 2) + t * 8);
      ka[0] = wa.x, ka[1] = wa.y;
      kb[0] = wb.x, kb[1] = wb.y;
    }
    float s[NT][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float acc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[nt][c] = 0.f;
#pragma unroll
      for (int j = n * JG; j < (n + 1) * JG; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t wa = ka[j] >> (8 * h), wb = kb[j] >> (8 * h);
          const uint32_t a0 = codes0(wa), a1 = codes0(wb), a2 = codes4(wa), a3 = codes4(wb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816(acc[nt], a0, a1, a2, a3, qf[nt][2 * j + h][0], qf[nt][2 * j + h][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          s[nt][c] = n == 0 ? sk[c >> 1][0] * acc[nt][c] : fmaf(sk[c >> 1][n], acc[nt][c], s[nt][c]);
    }
    // in log2 units; rounded before the maximum is taken off, so that the
    // largest weight is exactly 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[nt][c] *= f[nt][c & 1];
    // ---- weights
    uint32_t seen = 0xFu * 0x11111111u;  // bit 4 nt + c: element c of column tile nt
    if (!whole) {
      seen = 0;
      if (copied) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (key0 + g + 8 * (c >> 1) < lim[nt][c & 1]) seen |= 1u << (4 * nt + c);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!(seen >> (4 * nt + c) & 1)) s[nt][c] = -INFINITY;
    }
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 4; ++c) raise |= s[nt][c] > m[nt][c & 1] + kLazy;
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(s[nt][c], s[nt][c + 2]);
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
          const float now = fmaxf(m[nt][c], x);
          const float shrink = ex2_approx(m[nt][c] - now);
          m[nt][c] = now;
          l[nt][c] *= shrink;
#pragma unroll
          for (int k = 0; k < MT; ++k) o[nt][k][c] *= shrink, o[nt][k][c + 2] *= shrink;
        }
      }
    }
    float p[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        p[nt][c] = ex2_approx(s[nt][c] - m[nt][c & 1]);
        if (!whole && !(seen >> (4 * nt + c) & 1)) p[nt][c] = 0.f;
      }
      l[nt][0] += p[nt][0] + p[nt][2];
      l[nt][1] += p[nt][1] + p[nt][3];
    }
    // ---- P^T times V's scales, as B fragments (rows = keys)
    uint32_t pf[NT][NG][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          w[c] = p[nt][c] * sv[c >> 1][n];
          // a key that is not seen counts nothing, whatever its scale is
          if (!whole && !(seen >> (4 * nt + c) & 1)) w[c] = 0.f;
        }
        pf[nt][n][0] = transpose8x8(pack_half2(w[0], w[1]));
        pf[nt][n][1] = transpose8x8(pack_half2(w[2], w[3]));
      }
    }
    // ---- O^T
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      const uint4 v = *reinterpret_cast<const uint4*>(tile + 8 * D + w * 512 + g * 64 + t * 16);
      // tokens 2t, 2t + 1 and 2t + 8, 2t + 9 side by side, the lower and the upper half-words
      const uint32_t a[2] = {__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632)};
      const uint32_t b[2] = {__byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632)};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = a[k >> 1] >> (8 * (k & 1)), y = b[k >> 1] >> (8 * (k & 1));
        const int mt = 4 * w + k;
        const int n = mt * 16 / (D / NG);
        const uint32_t a0 = codes0(x), a1 = codes4(x), a2 = codes0(y), a3 = codes4(y);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          mma16816(o[nt][mt], a0, a1, a2, a3, pf[nt][n][0], pf[nt][n][1]);
      }
    }
    __syncwarp();
    issue(i + kStages);
  }
  if (!ok) {
    *abort = 1;
    if (lane == 0) {
      atomicExch(A.status, int32_t(SPARGE_ETIMEOUT));
      // copies in flight land before the block can end
      for (int s = 0; s < kStages; ++s) {
        mbar_wait_teardown(&full[warp][s], 0);
        mbar_wait_teardown(&full[warp][s], 1);
      }
    }
  }
  __syncwarp();

  // ---- this warp's result: O[row][channel], maximum and sum
  float* so = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], w);
      const int row = 8 * nt + 2 * t + c;
      if (g == 0) s_ml[warp][row] = make_float2(m[nt][c], l[nt][c]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
        *reinterpret_cast<float2*>(so + row * C::PITCH + 16 * mt + 2 * g) =
            make_float2(o[nt][mt][c], o[nt][mt][c + 2]);
    }
  }
  __syncthreads();

  // ---- the warps joined
  for (int e = threadIdx.x; e < C::ROWS * (D / 2); e += kAttnThreads) {
    const int row = e / (D / 2), ch = 2 * (e % (D / 2));
    if (row0 + row >= rows) break;
    float top = kLow;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_ml[w][row].x);
    float sum = 0.f, x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = s_ml[w][row];
      const float a = ex2_approx(ml.x - top);
      const float2 v = *reinterpret_cast<const float2*>(
          reinterpret_cast<const float*>(smem + w * C::RING) + row * C::PITCH + ch);
      sum = fmaf(ml.y, a, sum);
      x = fmaf(v.x, a, x);
      y = fmaf(v.y, a, y);
    }
    const int q = (row0 + row) / A.G, head = kvh * A.G + (row0 + row) % A.G;
    const int64_t at = int64_t(req.q0 + q) * A.Hq + head;
    if (A.splits > 1) {
      const int64_t part = at * A.splits + split;
      *reinterpret_cast<float2*>(A.part_o + part * D + ch) = make_float2(x, y);
      if (ch == 0) A.part_ml[part] = make_float2(top, sum);
    } else {
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
  }
}

// Chunks joined, a warp per row of q and head.
template <int D>
__global__ void __launch_bounds__(kAttnThreads) kv4_join_kernel(const DecodeArgs A) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31;
  const Request req = request(A, blockIdx.y);
  const int64_t e = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t at = int64_t(req.q0) * A.Hq + e;
  if (e >= int64_t(req.qlen) * A.Hq) return;
  const int n = max(1, int((req.keys + int64_t(A.chunk) * 16 - 1) / (int64_t(A.chunk) * 16)));
  const float2* ml = A.part_ml + at * A.splits;
  float top = kLow;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, ml[i].x);
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
  float x[V], sum = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) x[k] = 0.f;
  for (int i = 0; i < n; ++i) {
    const float2 p = ml[i];
    if (p.y == 0.f) continue;  // no key seen: its row was not summed
    const float a = ex2_approx(p.x - top);
    sum = fmaf(p.y, a, sum);
    const float* src = A.part_o + (at * A.splits + i) * D + lane * V;
    float v[V];
    if (V == 4) {
      const float4 q = *reinterpret_cast<const float4*>(src);
      v[0] = q.x, v[1] = q.y, v[V - 2] = q.z, v[V - 1] = q.w;
    } else {
      const float2 q = *reinterpret_cast<const float2*>(src);
      v[0] = q.x, v[1] = q.y;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) x[k] = fmaf(v[k], a, x[k]);
  }
  const float inv = sum == 0.f ? 0.f : 1.0f / sum;
  uint32_t* dst = reinterpret_cast<uint32_t*>(A.o) + (at * D + lane * V) / 2;
#pragma unroll
  for (int k = 0; k < V; k += 2) {
    if (A.bf16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[k] * inv, x[k + 1] * inv);
      dst[k / 2] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      dst[k / 2] = pack_half2(x[k] * inv, x[k + 1] * inv);
    }
  }
  if (lane == 0 && A.lse != nullptr)
    A.lse[at] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

struct Plan {
  int32_t nt, row_tiles, chunk, splits;
};

// How the keys are cut, from the bounds that the host knows (lengths are on
// the device): chunks until every SM has eight CTAs, of eight tiles at least.
Plan make_plan(const sparge_kv4_t& c, const sparge_kv4_attn_t& a) {
  Plan p{};
  const int64_t rows = int64_t(a.max_q) * (a.Hq / c.Hkv);
  p.nt = rows <= 8 ? 1 : 2;
  p.row_tiles = int32_t(cdiv(rows, 8 * p.nt));
  const int64_t tiles = cdiv(kv4_len_cap(c, a), 16);
  const int64_t ctas = int64_t(a.R) * c.Hkv * p.row_tiles;
  const int64_t want = ctas > 0 ? cdiv(148 * 8, ctas) : 1;
  int64_t chunk = cdiv(tiles, want);
  chunk = chunk < 8 ? 8 : (chunk > kMaxChunk ? kMaxChunk : chunk);
  p.chunk = int32_t(chunk);
  const int64_t splits = cdiv(tiles, chunk);
  p.splits = int32_t(splits < 1 ? 1 : splits);
  return p;
}

template <int D, int NG, int NT>
cudaError_t run(const DecodeArgs& a, const Plan& p, int32_t R, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  const int smem = C::smem(p.chunk);
  if (smem > 46 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kv4_attn_kernel<D, NG, NT>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  const dim3 grid(unsigned(p.splits), unsigned(a.Hkv * p.row_tiles), unsigned(R));
  kv4_attn_kernel<D, NG, NT><<<grid, kAttnThreads, smem, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.splits == 1) return e;
  const dim3 join(unsigned(cdiv(int64_t(a.max_q) * a.Hq, kWarps)), unsigned(R));
  kv4_join_kernel<D><<<join, kAttnThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <int D, int NG>
cudaError_t run_nt(const DecodeArgs& a, const Plan& p, int32_t R, cudaStream_t s) {
  return p.nt == 1 ? run<D, NG, 1>(a, p, R, s) : run<D, NG, 2>(a, p, R, s);
}

}  // namespace

bool kv4_attn_fits(const sparge_kv4_t& c, const sparge_kv4_attn_t& a) {
  const Plan p = make_plan(c, a);
  return int64_t(c.Hkv) * p.row_tiles <= 65535;
}

size_t kv4_attn_ws_bytes(const sparge_kv4_t& c, const sparge_kv4_attn_t& a) {
  const Plan p = make_plan(c, a);
  if (p.splits == 1) return 256;
  const size_t rows = size_t(a.T) * a.Hq * p.splits;
  return 256 + align256(rows * sizeof(float2)) + align256(rows * c.d * sizeof(float));
}

cudaError_t launch_kv4_attn(const sparge_kv4_t& c, const sparge_kv4_attn_t& a, const void* q,
                            const void* cache, const int32_t* table, const int32_t* seq_len,
                            const int32_t* cu_q, void* o, float* lse, void* ws,
                            cudaStream_t stream) {
  const Plan p = make_plan(c, a);
  DecodeArgs d{};
  d.q = static_cast<const char*>(q);
  d.cache = static_cast<const uint8_t*>(cache);
  d.table = table;
  d.seq_len = seq_len;
  d.cu = cu_q;
  d.o = static_cast<char*>(o);
  d.lse = lse;
  d.status = static_cast<int32_t*>(ws);
  if (p.splits > 1) {
    const size_t rows = size_t(a.T) * a.Hq * p.splits;
    d.part_ml = ws_ptr<float2>(ws, 256);
    d.part_o = ws_ptr<float>(ws, 256 + align256(rows * sizeof(float2)));
  }
  d.q_stride = a.q_stride * 2;
  d.T = a.T;
  d.Hq = a.Hq;
  d.Hkv = c.Hkv;
  d.G = a.Hq / c.Hkv;
  d.max_q = a.max_q;
  d.max_pages = a.max_pages;
  d.len_cap = int32_t(kv4_len_cap(c, a));
  d.causal = a.causal;
  d.page = c.page_size;
  d.tpp = c.page_size / 16;
  d.num_pages = c.num_pages;
  d.splits = p.splits;
  d.chunk = p.chunk;
  d.bf16 = a.dtype == SPARGE_BF16;
  d.scale_log2 = a.scale * 1.4426950408889634f;
  const int ng = c.d / c.group;
  if (c.d == 64)
    return ng == 2 ? run_nt<64, 2>(d, p, a.R, stream) : run_nt<64, 1>(d, p, a.R, stream);
  if (ng == 4) return run_nt<128, 4>(d, p, a.R, stream);
  return ng == 2 ? run_nt<128, 2>(d, p, a.R, stream) : run_nt<128, 1>(d, p, a.R, stream);
}

}  // namespace sparge
