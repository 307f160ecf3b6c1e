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
// goes into the weights: p is rounded to fp16 and p s once more (the sum of
// weights is of the unrounded p; the two roundings are 2^-10 of p s together, half of a
// bf16 output's own, and save a tenth of the instructions).  Q is fp16 with one power
// of two per row, so bf16 queries lose nothing above 2^-26 of the row's
// largest.  The running maximum is lazy: it is raised (and O rescaled) when a
// score passes it by more than 2 in log2 units, so weights are at most 4.
//
// fp16 ends at 2^-24, and an answer may be carried by very many keys of small
// weight or by small values.  So p is held times 2^10 and s times a power of two
// that brings the largest scale a warp has met to [8, 16), which just keeps 4 p s
// below 65504: a key has all its bits down to p = 2^-24 and p s = 2^-27 of the
// largest, whatever the size of V.  The power falls when a larger scale comes, with O, in
// the branch of the maximum; a step's scales are looked over a lane a token.  All of it
// costs 1 to 2 % (84.7 against 83.2 us for three requests of 115,000 keys).  Without it answers
// that keys 14 nats below the largest carry were off by 58 % of sum p |v| where V was around 0.02,
// with it by 0.2 %, a bf16 output's own rounding.
//
// Work is cut evenly, whatever the lengths: the units (request, KV head, tile
// of 8 NT query rows) stand in one line, each as long as its keys in steps of
// two 16-token tiles and a constant for its start and end, and CTA c of C takes the
// c-th part of the line.  A unit that
// lies within one CTA is finished there; the parts of a cut one go to the
// workspace, and the CTA that arrives last joins them in the order of their
// keys.  The cut depends on the lengths alone, so results are the same bits
// every time.  Inside a CTA the four warps take the steps in turn, each through
// a ring of bulk copies of its own, and are joined in shared memory.
//
// Measured, 32 query heads of 128 channels over 8: one token of 48 requests of 700
// to 8192 keys in 57.5 us (233 MB at 4.1 TB/s), of three of 115,000 in 84.7 us (396 MB
// at 4.7 TB/s, 71 % of a copy's rate), of one of 1009 in 9.2 us.  Issue slots (60 to 65 %)
// and memory share the limit.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "after.cuh"
#include "kv4_common.cuh"
#include "kv4_layout.cuh"
#include "sm100_ptx.cuh"
#include "sparge_internal.h"

namespace sparge {

using namespace kv4;

namespace {

constexpr int kWarps = 4;
constexpr int kAttnThreads = kWarps * 32;
constexpr float kLazy = 2.0f;      // log2 units
constexpr int kLift = 10;          // log2 of what weights are held times
constexpr int kTop = 4;            // V's scales are held below 2^kTop
static_assert(kLazy + kLift + kTop == 16, "4 p s below 65504: 2^12 (16 - 2^-7)");

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A unit's start and end cost a CTA about as much as this many keys: the
// queries, the first copies' latency, the joining (3.5 us against 0.4 us for 32
// keys with every SM full).  Without it, many short requests met one CTA: nine
// requests of 4001 to 1 tokens took 45 us, with it 15.
constexpr int kUnitKeys = 256;

// Resident CTAs per SM, by registers (128 and 255 a thread).
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 4 : 2; }

template <int D, int NG, int NT>
struct Cfg {
  static constexpr int TILE = 16 * (D + 4 * NG);
  static constexpr int ROWS = 8 * NT;
  static constexpr int PITCH = D + 4;  // floats per row of the joining buffer
  // A warp takes TPS tiles (16 TPS keys) per step and has ST steps' copies in
  // flight: with 16 warps a SM some 200 KB (the copy rate times the latency
  // needs about 45 KB).  Four tiles per step, three CTAs a SM: a sixth fewer
  // instructions, 2% slower (84.6 against 83.3 us for three requests of 98K to
  // 128K tokens) and 11.8 against 9.1 us for one of 1009.
  static constexpr int TPS = 2;
  static constexpr int ST = 3 * (128 / D);
  static constexpr int RING = ST * TPS * TILE;
  static constexpr int SMEM = kWarps * RING;
  static constexpr int CTAS = ctas_per_sm(NT);
  static_assert(ROWS * PITCH * 4 <= RING, "a warp's result fits its ring");
  static_assert(CTAS * (SMEM + 2560) <= 228 * 1024, "resident together");
};

// The NG scales of one token's K or V, float32.
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t* at, float (&x)[NG]) {
  if constexpr (NG == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    const float2 a = half2_f(w.x), b = half2_f(w.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else if constexpr (NG == 2) {
    const float2 a = half2_f(*reinterpret_cast<const uint32_t*>(at));
    x[0] = a.x, x[1] = a.y;
  } else {
    x[0] = __half2float(*reinterpret_cast<const __half*>(at));
  }
}

// Those of its V as they lie, two to a word (a single one alone).
template <int NG>
__device__ __forceinline__ void load_words(const uint8_t* at, uint32_t (&v)[(NG + 1) / 2]) {
  if constexpr (NG == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    v[0] = w.x, v[1] = w.y;
  } else if constexpr (NG == 2) {
    v[0] = *reinterpret_cast<const uint32_t*>(at);
  } else {
    v[0] = *reinterpret_cast<const uint16_t*>(at);
  }
}
// A pair of weights times the scale n of such words.
__device__ __forceinline__ uint32_t times_scale(uint32_t p, const uint32_t* v, int n) {
  const __half2 w = *reinterpret_cast<const __half2*>(&v[n / 2]);
  const __half2 x = __hmul2_rn(*reinterpret_cast<const __half2*>(&p),
                               n % 2 ? __high2half2(w) : __low2half2(w));
  return *reinterpret_cast<const uint32_t*>(&x);
}

__device__ __forceinline__ float two_to(int n) { return __uint_as_float(uint32_t(n + 127) << 23); }
// 2^n as fp16, -15 < n < 16, in both halves of a word, and back.
__device__ __forceinline__ uint32_t half_two_to(int n) { return uint32_t(n + 15) * 0x04000400u; }
__device__ __forceinline__ int half_log2(uint32_t x) { return int(x >> 26) - 15; }

template <int D, int NG, int NT>
__global__ void __launch_bounds__(kAttnThreads, Cfg<D, NG, NT>::CTAS)
    kv4_attn_kernel(const DecodeArgs A) {
  using C = Cfg<D, NG, NT>;
  constexpr int J = D / 32;       // words of a token's codes per lane
  constexpr int JG = J / NG;      // of them per scale group
  constexpr int MT = D / 16;      // output row tiles
  constexpr int ST = C::ST, TPS = C::TPS, KEYS = 16 * TPS;
  constexpr int COST = kUnitKeys / KEYS;
  constexpr int BATCH_STEPS = 32 / TPS;  // steps whose tile numbers a warp fetches at once
  static_assert(ST < BATCH_STEPS, "steps in flight lie in two batches");
  static_assert(KEYS == 32, "V's scales of a step: a lane a token");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t full[kWarps][ST];
  __shared__ float2 s_ml[kWarps][C::ROWS];
  __shared__ int64_t s_scan[kWarps + 1];
  __shared__ int64_t s_found[2];
  __shared__ int32_t s_id[kWarps][2][32];  // tile numbers of a warp's next steps, two batches
  __shared__ int s_flag[2];  // a wait gave up; this CTA joins
  volatile int* abort = &s_flag[0];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::RING;
  const Masks masks = A.masks;

  if (threadIdx.x == 0) {
    s_flag[0] = 0;
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < ST; ++s) mbar_init(&full[w][s], 1);
    fence_mbar_init();
    fence_async_shared();
  }

  begin_after();

  // ---- the line of units: its length, and the request where this part starts
  const int per = (A.R + kAttnThreads - 1) / kAttnThreads;
  const int r_lo = min(A.R, int(threadIdx.x) * per), r_hi = min(A.R, r_lo + per);
  int64_t own = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const Request x = request(A, r);
    const int64_t n = unit_count<C::ROWS>(A, x);
    own += n * (unit_steps<KEYS>(x) + COST);
    if (!x.sound && blockIdx.x == 0) atomicCAS(A.status, 0, int32_t(SPARGE_EINVAL));
  }
  int64_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  before += incl - own;
  // parts: a step per warp at least
  int64_t parts = gridDim.x;
  parts = min(parts, (total + kWarps - 1) / kWarps);
  if (total == 0) return;
  const int64_t step = div64(total + parts - 1, parts);
  const int64_t line0 = blockIdx.x * step, line1 = min(line0 + step, total);
  if (line0 >= total) return;
  if (before <= line0 && line0 < before + own) {
    int64_t at = before;
    for (int r = r_lo; r < r_hi; ++r) {
      const Request x = request(A, r);
      const int64_t n = unit_count<C::ROWS>(A, x) * (unit_steps<KEYS>(x) + COST);
      if (line0 < at + n) {
        s_found[0] = r;
        s_found[1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  int r = int(s_found[0]);
  int64_t r_at = s_found[1];  // where request r's units start
  int put = 0, take = 0;      // stages that the next step is copied to and taken from
  uint32_t phase = 0;         // parity of the stage `take`
  bool ok = true;

  for (int64_t line = line0; line < line1;) {
    Request req = request(A, r);
    const int64_t n_steps = unit_steps<KEYS>(req), n_units = unit_count<C::ROWS>(A, req);
    const int64_t length = n_steps + COST;
    if (line >= r_at + n_units * length) {
      r_at += n_units * length;
      ++r;
      continue;
    }
    const int64_t into = line - r_at;
    const int64_t unit = div64(into, length);
    const int64_t steps_at = r_at + unit * length + COST;  // where its first step stands
    const int step0 = int(max(line - steps_at, int64_t(0)));
    const int64_t stop = min(line1, steps_at + n_steps);
    const int step1 = int(max(stop - steps_at, int64_t(0)));
    line = stop;
    if (step1 == step0) continue;  // the next CTA has all of it
    const bool cut = step0 > 0 || step1 < n_steps;
    const int tile_of = A.heads.quot(int(unit)), kvh = int(unit) - tile_of * A.Hkv;
    const int row0 = tile_of * C::ROWS, rows = req.qlen * int(A.G.d);
    // the last key that any row of this tile sees
    const int last_row = min(row0 + C::ROWS, rows) - 1;
    const int32_t reach =
        A.causal ? min(req.keys, req.len - req.qlen + A.G.quot(last_row) + 1) : req.keys;
    const int n_tiles = reach > 0 ? (reach + 15) / 16 : 0;
    const int n_here = min(step1, (n_tiles + TPS - 1) / TPS) - step0;
    // step i of this warp is step step0 + warp + kWarps i of the unit
    const int mine = n_here > warp ? (n_here - warp + kWarps - 1) / kWarps : 0;

    // ---- the ring.  Tile numbers come in batches, a lane to a tile: one batch
    // in shared memory, the next in a register, fetched a batch ahead
    const int32_t* table = A.table + int64_t(r) * A.max_pages;
    auto tile_id = [&](int batch) -> int32_t {
      const int i = BATCH_STEPS * batch + lane / TPS;
      const int ti = TPS * (step0 + warp + kWarps * i) + lane % TPS;
      if (i >= mine || ti >= n_tiles) return -1;
      const int32_t entry = A.tpp.quot(ti), page = table[entry];
      if (uint32_t(page) >= uint32_t(A.num_pages)) {
        atomicCAS(A.status, 0, int32_t(SPARGE_EINVAL));
        return -1;
      }
      return (page * A.Hkv + kvh - entry) * int32_t(A.tpp.d) + ti;
    };
    // where step i's tile numbers are
    auto ids_of = [&](int i) {
      return s_id[warp][i / BATCH_STEPS & 1] + TPS * (i % BATCH_STEPS);
    };
    s_id[warp][0][lane] = tile_id(0);
    int32_t next_id = tile_id(1);
    __syncwarp();
    auto issue = [&](int i) {
      if (i >= mine) return;
      if (i > 0 && i % BATCH_STEPS == 0) {
        // the steps still to be taken lie in the batch before: its place is the other
        ids_of(i)[lane] = next_id;
        next_id = tile_id(i / BATCH_STEPS + 1);
        __syncwarp();
      }
      if (lane == 0) {
        int32_t id[TPS];
        const int32_t* at = ids_of(i);
        bool run = true;  // all there, and one behind the other in memory
        int n = 0;
#pragma unroll
        for (int u = 0; u < TPS; ++u) {
          id[u] = at[u];
          n += id[u] >= 0;
          run = run && id[u] == id[0] + u;
        }
        uint64_t* bar = &full[warp][put];
        uint8_t* dst = ring + put * TPS * C::TILE;
        if (run && id[0] >= 0) {
          mbar_expect_tx(bar, TPS * C::TILE);
          bulk_load(dst, A.cache + int64_t(id[0]) * C::TILE, TPS * C::TILE, bar);
        } else if (n > 0) {
          mbar_expect_tx(bar, n * C::TILE);
#pragma unroll
          for (int u = 0; u < TPS; ++u)
            if (id[u] >= 0)
              bulk_load(dst + u * C::TILE, A.cache + int64_t(id[u]) * C::TILE, C::TILE, bar);
        } else {
          mbar_arrive(bar);  // nothing to copy: these keys are left out
        }
      }
      put = put + 1 == ST ? 0 : put + 1;
    };
    // The queries are asked for before the copies: behind 30 MB of those, at the
    // launch's start, they took 5 us.
    uint4 raw_q[NT][J];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = row0 + 8 * nt + g;
      const bool there = row < rows;
#pragma unroll
      for (int j = 0; j < J; ++j) raw_q[nt][j] = make_uint4(0, 0, 0, 0);
      if (there) {
        const int tok = A.G.quot(row), head = kvh * int(A.G.d) + row - tok * int(A.G.d);
        const char* src =
            A.q + int64_t(req.q0 + tok) * A.q_stride + int64_t(head) * (D * 2) + 16 * t;
#pragma unroll
        for (int j = 0; j < J; ++j)
          raw_q[nt][j] = *reinterpret_cast<const uint4*>(src + 64 * j);
      }
    }
    if (ok) {
#pragma unroll
      for (int i = 0; i < ST; ++i) issue(i);
    }

    // ---- Q as B fragments: column g is query row row0 + 8 nt + g; the 32-bit
    // word (t, j) of a token's codes meets channels 32 j + 8 t .. + 7
    uint32_t qf[NT][2 * J][2];
    float f[NT][2];        // score of a column: f * sum_g s_g S_g, in log2 units
    int32_t lim[NT][2];    // the column sees keys below this
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float x[J][8];
      float big = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint4 raw = raw_q[nt][j];
        const uint32_t u[4] = {raw.x, raw.y, raw.z, raw.w};
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
      // the row's largest goes to [2^12, 2^13) (a subnormal below); two factors,
      // since one may overflow
      const int field = int(__float_as_uint(big) >> 23);
      const int k = field < 255 ? 139 - field : 0, half_k = k >> 1;
      const float k1 = two_to(half_k), k2 = two_to(k - half_k);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          qf[nt][2 * j + i / 2][i & 1] =
              pack_half2(x[j][2 * i] * k1 * k2, x[j][2 * i + 1] * k1 * k2);
      const float fr = A.scale_log2 * two_to(-half_k) * two_to(half_k - k);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f[nt][c] = __shfl_sync(0xffffffffu, fr, (2 * t + c) * 4);  // from a lane of column 2t + c
        const int row_c = row0 + 8 * nt + 2 * t + c;
        lim[nt][c] = 0;
        if (row_c < rows)
          lim[nt][c] =
              A.causal ? min(req.keys, req.len - req.qlen + A.G.quot(row_c) + 1) : req.keys;
      }
    }
    // keys below this are seen by every row that is there
    int32_t all_see = req.keys;
    if (A.causal) all_see = min(all_see, req.len - req.qlen + A.G.quot(row0) + 1);

    float m[NT][2], l[NT][2];
    float o[NT][MT][4];
    uint32_t s_lift = half_two_to(15);  // what V's scales are held times
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) m[nt][c] = kLow, l[nt][c] = 0.f;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
    }

    for (int i = 0; i < mine && ok; ++i) {
      const int stage = take;
      ok = __all_sync(0xffffffffu, mbar_wait(&full[warp][stage], phase, abort, A.status));
      if (!ok) break;
      take = take + 1 == ST ? 0 : take + 1;
      phase ^= take == 0;
      const uint8_t* tiles = ring + stage * TPS * C::TILE;
      const int32_t key0 = (step0 + warp + kWarps * i) * KEYS;
      uint32_t here = 0;  // bit u: tile u was copied
      {
        const int32_t* at = ids_of(i);
#pragma unroll
        for (int u = 0; u < TPS; ++u) here |= uint32_t(at[u] >= 0) << u;
      }

      // One step; MASKED: some row does not see some key of it.
      auto step = [&](auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
        float s[TPS][NT][4];
#pragma unroll
        for (int u = 0; u < TPS; ++u) {
          const uint8_t* tile = tiles + u * C::TILE;
          // ---- S^T
          uint32_t ka[J], kb[J];  // tokens g and g + 8
          if constexpr (J == 4) {
            const uint4 wa = *reinterpret_cast<const uint4*>(tile + g * (D / 2) + t * 16);
            const uint4 wb = *reinterpret_cast<const uint4*>(tile + (g + 8) * (D / 2) + t * 16);
            ka[0] = wa.x, ka[1] = wa.y, ka[2] = wa.z, ka[3] = wa.w;
            kb[0] = wb.x, kb[1] = wb.y, kb[2] = wb.z, kb[3] = wb.w;
          } else {
            const uint2 wa = *reinterpret_cast<const uint2*>(tile + g * (D / 2) + t * 8);
            const uint2 wb = *reinterpret_cast<const uint2*>(tile + (g + 8) * (D / 2) + t * 8);
            ka[0] = wa.x, ka[1] = wa.y;
            kb[0] = wb.x, kb[1] = wb.y;
          }
          float sk[2][NG];
          load_scales<NG>(tile + 16 * D + g * NG * 4, sk[0]);
          load_scales<NG>(tile + 16 * D + (g + 8) * NG * 4, sk[1]);
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
                const uint32_t a0 = codes0(wa, masks), a1 = codes0(wb, masks);
                const uint32_t a2 = codes4(wa, masks), a3 = codes4(wb, masks);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma16816(acc[nt], a0, a1, a2, a3, qf[nt][2 * j + h][0], qf[nt][2 * j + h][1]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                s[u][nt][c] = n == 0 ? sk[c >> 1][0] * acc[nt][c]
                                     : fmaf(sk[c >> 1][n], acc[nt][c], s[u][nt][c]);
          }
          // in log2 units; rounded before the maximum is taken off, so that the
          // largest weight is exactly 1
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; c += 2)
              unpack2(mul2(pack2(s[u][nt][c], s[u][nt][c + 1]), pack2(f[nt][0], f[nt][1])),
                      s[u][nt][c], s[u][nt][c + 1]);
        }
        // ---- keys that a row does not see
        uint32_t seen = ~0u;  // bit 4 (NT u + nt) + c
        if (MASKED) {
          seen = 0;
#pragma unroll
          for (int u = 0; u < TPS; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const bool yes =
                    (here >> u & 1u) && key0 + 16 * u + g + 8 * (c >> 1) < lim[nt][c & 1];
                seen |= uint32_t(yes) << (4 * (NT * u + nt) + c);
                if (!yes) s[u][nt][c] = -INFINITY;
              }
        }
        // ---- V's scales of the step, a lane a token: whether one times s_lift = 2^b is
        // 2^kTop or more, that is, whether its bits reach those of 2^(kTop - b): the
        // sum's top bit (a NaN's too)
        auto scales = [&](uint32_t (&w)[(NG + 1) / 2]) {
          load_words<NG>(tiles + (lane >> 4) * C::TILE + 16 * D + (lane & 15) * NG * 4 + 2 * NG, w);
          // (of a token that does not exist any bytes may stand there)
          if (MASKED && !((here >> (lane >> 4) & 1u) && key0 + lane < req.keys))
            for (uint32_t& x : w) x = 0;
        };
        uint32_t over = 0;
        {
          uint32_t w[(NG + 1) / 2];
          scales(w);
#pragma unroll
          for (uint32_t x : w) over |= x + (s_lift - (kTop - 2) * 0x04000400u);
        }
        // ---- the running maximum
        float high[NT][2];  // this lane's largest of each column
        bool raise = over & 0x80008000u;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
            for (int u = 1; u < TPS; ++u) x = max3(x, s[u][nt][c], s[u][nt][c + 2]);
            high[nt][c] = x;
            raise |= x > m[nt][c] + kLazy;
          }
        if (__any_sync(0xffffffffu, raise)) {
          uint32_t w[(NG + 1) / 2], top = 0;
          scales(w);  // again: seldom, and kept they would cost registers
#pragma unroll
          for (uint32_t x : w) {
            const uint32_t lo = x & 0xFFFFu, hi = x >> 16;
            if (lo < 0x7C00u) top = max(top, lo);  // (a NaN has no size)
            if (hi < 0x7C00u) top = max(top, hi);
          }
          const uint32_t was = s_lift;
          const int e = int(__reduce_max_sync(0xffffffffu, top) >> 10) - 15;
          s_lift = min(s_lift, half_two_to(min(15, kTop - 1 - e)));
          const float o_by = two_to(half_log2(s_lift) - half_log2(was));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x = high[nt][c];
#pragma unroll
              for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
              const float now = fmaxf(m[nt][c], x);
              const float shrink = ex2_approx(m[nt][c] - now);
              m[nt][c] = now;
              l[nt][c] *= shrink;
              const float by = shrink * o_by;
#pragma unroll
              for (int k = 0; k < MT; ++k) o[nt][k][c] *= by, o[nt][k][c + 2] *= by;
            }
          }
        }
#pragma unroll
        for (int u = 0; u < TPS; ++u) {
          const uint8_t* tile = tiles + u * C::TILE;
          uint32_t sv[2][(NG + 1) / 2];  // of tokens g and g + 8, lifted
          load_words<NG>(tile + 16 * D + g * NG * 4 + 2 * NG, sv[0]);
          load_words<NG>(tile + 16 * D + (g + 8) * NG * 4 + 2 * NG, sv[1]);
#pragma unroll
          for (int w = 0; w < (NG + 1) / 2; ++w)
            sv[0][w] = times(sv[0][w], s_lift), sv[1][w] = times(sv[1][w], s_lift);
          // ---- weights, times V's scales, as B fragments (rows = keys)
          uint32_t pf[NT][NG][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            // (two sums: the largest weight is a power of two exactly)
            for (int c = 0; c < 4; c += 2) {
              unpack2(add2(sub2(pack2(s[u][nt][c], s[u][nt][c + 1]), pack2(m[nt][0], m[nt][1])),
                           pack2(kLift, kLift)),
                      p[c], p[c + 1]);
              p[c] = ex2_approx(p[c]);
              p[c + 1] = ex2_approx(p[c + 1]);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (MASKED && !(seen >> (4 * (NT * u + nt) + c) & 1)) p[c] = 0.f;
            l[nt][0] += p[0] + p[2];
            l[nt][1] += p[1] + p[3];
            const uint32_t pa = pack_half2(p[0], p[1]), pb = pack_half2(p[2], p[3]);
#pragma unroll
            for (int n = 0; n < NG; ++n) {
              uint32_t wa = times_scale(pa, sv[0], n), wb = times_scale(pb, sv[1], n);
              if (MASKED) {
                // a key that is not seen counts nothing, whatever its scale is
                const uint32_t bits = seen >> (4 * (NT * u + nt));
                wa &= (bits & 1 ? 0xFFFFu : 0u) | (bits & 2 ? 0xFFFF0000u : 0u);
                wb &= (bits & 4 ? 0xFFFFu : 0u) | (bits & 8 ? 0xFFFF0000u : 0u);
              }
              pf[nt][n][0] = transpose8x8(wa);
              pf[nt][n][1] = transpose8x8(wb);
            }
          }
          // ---- O^T
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            const uint4 v =
                *reinterpret_cast<const uint4*>(tile + 8 * D + w * 512 + g * 64 + t * 16);
            // tokens 2t, 2t + 1 and 2t + 8, 2t + 9 side by side, lower and upper half-words
            const uint32_t a[2] = {__byte_perm(v.x, v.y, 0x5410), __byte_perm(v.x, v.y, 0x7632)};
            const uint32_t b[2] = {__byte_perm(v.z, v.w, 0x5410), __byte_perm(v.z, v.w, 0x7632)};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t x = a[k >> 1] >> (8 * (k & 1)), y = b[k >> 1] >> (8 * (k & 1));
              const int mt = 4 * w + k;
              const int n = mt * 16 / (D / NG);
              const uint32_t a0 = codes0(x, masks), a1 = codes4(x, masks);
              const uint32_t a2 = codes0(y, masks), a3 = codes4(y, masks);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[nt][mt], a0, a1, a2, a3, pf[nt][n][0], pf[nt][n][1]);
            }
          }
        }
      };
      if (here == (1u << TPS) - 1 && key0 + KEYS <= all_see)
        step(std::false_type{});
      else
        step(std::true_type{});
      __syncwarp();
      issue(i + ST);
    }
    if (!ok && *abort == 0) {
      *abort = 1;
      if (lane == 0) atomicExch(A.status, int32_t(SPARGE_ETIMEOUT));
    }
    if (!ok && lane == 0) {
      // copies in flight land (or run out of time) before the ring is used again
      for (int s = 0; s < ST; ++s) {
        mbar_wait_teardown(&full[warp][s], 0);
        mbar_wait_teardown(&full[warp][s], 1);
      }
    }
    __syncwarp();

    // ---- this warp's result: O[row][channel], maximum and sum
    float* so = reinterpret_cast<float*>(ring);
    const float l_by = two_to(-kLift), o_by = two_to(-kLift - half_log2(s_lift));
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], w);
        const int row = 8 * nt + 2 * t + c;
        if (g == 0) s_ml[warp][row] = make_float2(m[nt][c], l[nt][c] * l_by);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          *reinterpret_cast<float2*>(so + row * C::PITCH + 16 * mt + 2 * g) =
              make_float2(o[nt][mt][c] * o_by, o[nt][mt][c + 2] * o_by);
      }
    }
    __syncthreads();

    // ---- the warps joined: finished, or this CTA's part of a cut unit
    const int64_t slot = 2 * int64_t(blockIdx.x) + (step0 > 0 ? 0 : 1);
    const int here_rows = min(C::ROWS, rows - row0);
    auto join_warps = [&](bool finish) {
      for (int e = threadIdx.x; e < here_rows * (D / 2); e += kAttnThreads) {
        const int row = e / (D / 2), ch = 2 * (e % (D / 2));
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
        if (finish) {
          write_out(A, out_row(A, req, kvh, row0 + row), D, ch, top, sum, x, y);
        } else {
          *reinterpret_cast<float2*>(A.part_o + (slot * C::ROWS + row) * D + ch) =
              make_float2(x, y);
          if (ch == 0) A.part_ml[slot * C::ROWS + row] = make_float2(top, sum);
        }
      }
    };
    join_warps(!cut);
    fence_async_shared();  // before the ring's next bulk copies
    if (cut) __threadfence();
    __syncthreads();
    if (!cut) continue;

    // ---- the last of a cut unit's CTAs joins its parts: a warp each fourth of
    // them, in their order, then the warps as above
    const int64_t c0 = step0 == 0 ? int64_t(blockIdx.x) : div64(steps_at, step);
    const int n_parts = int(div64(steps_at + n_steps - 1, step) - c0) + 1;
    if (threadIdx.x == 0)
      s_flag[1] = atomicInc(A.arrived + c0, uint32_t(n_parts - 1)) == uint32_t(n_parts - 1);
    __syncthreads();
    if (!s_flag[1]) continue;
    __threadfence();
    constexpr int V = 4;                   // channels per lane
    constexpr int RPW = 32 * V / D;        // rows that a warp's load covers
    constexpr int ITEMS = C::ROWS / RPW;
    constexpr int EG = ITEMS < 4 ? ITEMS : 4, BATCH = 4;  // rows and parts in flight
    const int ch = V * lane % D, sub = V * lane / D;
#pragma unroll 1
    for (int e0 = 0; e0 < ITEMS && e0 * RPW < here_rows; e0 += EG) {
      float top[EG], sum[EG], x[EG][V];
#pragma unroll
      for (int e = 0; e < EG; ++e) {
        top[e] = kLow, sum[e] = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) x[e][v] = 0.f;
      }
#pragma unroll 1
      for (int k0 = warp; k0 < n_parts; k0 += kWarps * BATCH) {
        float2 ml[BATCH][EG];
        float4 q[BATCH][EG];
        // loads without conditions, so that all are in flight: behind the last
        // part or row they repeat it, and count nothing
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int k = min(k0 + kWarps * i, n_parts - 1);
          // the first part is its CTA's last unit, the others are their CTAs' first
          const int64_t at = (2 * (c0 + k) + (k == 0 ? 1 : 0)) * C::ROWS;
#pragma unroll
          for (int e = 0; e < EG; ++e) {
            const int64_t row = at + min((e0 + e) * RPW + sub, here_rows - 1);
            ml[i][e] = __ldcg(A.part_ml + row);
            q[i][e] = __ldcg(reinterpret_cast<const float4*>(A.part_o + row * D + ch));
          }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
          if (k0 + kWarps * i >= n_parts) {
#pragma unroll
            for (int e = 0; e < EG; ++e) ml[i][e] = make_float2(-INFINITY, 0.f);
          }
#pragma unroll
        for (int e = 0; e < EG; ++e) {
          float now = top[e];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) now = fmaxf(now, ml[i][e].x);
          const float old = ex2_approx(top[e] - now);
          top[e] = now;
          sum[e] *= old;
#pragma unroll
          for (int v = 0; v < V; ++v) x[e][v] *= old;
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const float a = ex2_approx(ml[i][e].x - now);
            sum[e] = fmaf(ml[i][e].y, a, sum[e]);
            x[e][0] = fmaf(q[i][e].x, a, x[e][0]);
            x[e][1] = fmaf(q[i][e].y, a, x[e][1]);
            x[e][2] = fmaf(q[i][e].z, a, x[e][2]);
            x[e][3] = fmaf(q[i][e].w, a, x[e][3]);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < EG; ++e) {
        const int row = (e0 + e) * RPW + sub;
        *reinterpret_cast<float4*>(so + row * C::PITCH + ch) =
            make_float4(x[e][0], x[e][1], x[e][2], x[e][3]);
        if (ch == 0) s_ml[warp][row] = make_float2(top[e], sum[e]);
      }
    }
    __syncthreads();
    join_warps(true);
    fence_async_shared();
    __syncthreads();
  }
}

struct Plan {
  int32_t nt, grid;   // column tiles and CTAs of the kernel above
  int32_t piece_grid;  // CTAs of the other, 0: not needed
};

// More rows than this per request and KV head (tokens times the group's heads)
// are a piece of a prompt, kv4_piece.cu, whose steps cost about the same for up
// to 256 rows, while here every 16 rows read the codes again.  16 requests of 11,000
// to 32,768 keys, 8 KV heads, here and there in us:
//              32 rows      48 rows      64 rows      96 rows
//   128 bf16   225 / 388    328 / 392    432 / 371    637 / 382
//   128 fp16   225 / 415    328 / 420    432 / 411    637 / 418
//    64 bf16   161 / 350    235 / 354    309 / 344    456 / 351
//    64 fp16   161 / 362    235 / 366    309 / 351    456 / 360
// Two requests of up to 8192 keys are latency, and here is faster up to 128 rows (44 / 98).
constexpr int64_t kFewRows = 64;

// CTAs from the bounds that the host knows (lengths are on the device): all
// that are resident at once, fewer when there cannot be a step for each warp.
int32_t grid_of(const sparge_kv4_t& c, const sparge_kv4_attn_t& a, int64_t tiles, int64_t keys,
                int64_t most, int64_t per_cta) {
  const int64_t steps = cdiv(kv4_len_cap(c, a), keys);
  // more than that many CTAs' steps already: no need to multiply on
  int64_t line = steps < 1 ? 1 : steps;
  const int64_t by[] = {tiles, c.Hkv, a.R};
  for (int64_t n : by) line = line > most * per_cta ? line : line * (n < 1 ? 1 : n);
  const int64_t grid = cdiv(line, per_cta);
  return int32_t(grid < most ? grid : most);
}

Plan make_plan(const sparge_kv4_t& c, const sparge_kv4_attn_t& a) {
  Plan p{};
  int64_t rows = int64_t(a.max_q) * (a.Hq / c.Hkv);
  if (rows > kFewRows) {
    // a unit's start costs eight steps, so shorter lines take no more CTAs
    p.piece_grid = grid_of(c, a, cdiv(rows, kPieceRows), 64, kSms, 1);
    if (a.R == 1) return p;
    rows = kFewRows;  // the other requests may bring few
  }
  p.nt = rows <= 8 ? 1 : 2;
  p.grid = grid_of(c, a, cdiv(rows, 8 * p.nt), 32, kSms * ctas_per_sm(p.nt), kWarps);
  return p;
}

// Of one size for every call, so that calls of different shapes may share a
// workspace: no other region ever lies on the counters.
size_t arrived_bytes() { return align256(size_t(kSms) * ctas_per_sm(1) * sizeof(uint32_t)); }
size_t part_rows(const Plan& p) {
  const size_t few = size_t(p.grid) * 2 * 8 * p.nt, piece = size_t(p.piece_grid) * 2 * kPieceRows;
  return few > piece ? few : piece;
}
size_t ml_bytes(const Plan& p) { return align256(part_rows(p) * sizeof(float2)); }

template <int D, int NG, int NT>
cudaError_t run(const DecodeArgs& a, const Plan& p, cudaStream_t stream) {
  using C = Cfg<D, NG, NT>;
  const cudaError_t e = cudaFuncSetAttribute(
      kv4_attn_kernel<D, NG, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_after(kv4_attn_kernel<D, NG, NT>, dim3(unsigned(p.grid)), kAttnThreads, C::SMEM,
                      stream, a);
}

template <int D, int NG>
cudaError_t run_nt(const DecodeArgs& a, const Plan& p, cudaStream_t s) {
  return p.nt == 1 ? run<D, NG, 1>(a, p, s) : run<D, NG, 2>(a, p, s);
}

}  // namespace

size_t kv4_attn_ws_bytes(const sparge_kv4_t& c, const sparge_kv4_attn_t& a) {
  const Plan p = make_plan(c, a);
  return 256 + arrived_bytes() + ml_bytes(p) + part_rows(p) * c.d * sizeof(float);
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
  d.arrived = ws_ptr<uint32_t>(ws, 256);
  d.part_ml = ws_ptr<float2>(ws, 256 + arrived_bytes());
  d.part_o = ws_ptr<float>(ws, 256 + arrived_bytes() + ml_bytes(p));
  d.q_stride = a.q_stride * 2;
  d.R = a.R;
  d.T = a.T;
  d.Hq = a.Hq;
  d.Hkv = c.Hkv;
  d.G = make_div(uint32_t(a.Hq / c.Hkv));
  d.heads = make_div(uint32_t(c.Hkv));
  d.tpp = make_div(uint32_t(c.page_size / 16));
  d.max_q = a.max_q;
  d.max_pages = a.max_pages;
  d.len_cap = int32_t(kv4_len_cap(c, a));
  d.causal = a.causal;
  d.num_pages = c.num_pages;
  d.bf16 = a.dtype == SPARGE_BF16;
  d.masks = Masks{0x000F000Fu, 0x00F000F0u, 0x00F0000Fu};
  d.scale_log2 = a.scale * 1.4426950408889634f;
  const int ng = c.d / c.group;
  d.min_rows = 0;
  d.max_rows = INT32_MAX;
  if (p.piece_grid > 0) {
    if (p.grid > 0) d.min_rows = kFewRows + 1;
    const cudaError_t e = launch_kv4_piece(d, c.d, ng, p.piece_grid, stream);
    if (e != cudaSuccess || p.grid == 0) return e;
    d.min_rows = 0;
    d.max_rows = kFewRows;
  }
  if (c.d == 64) return ng == 2 ? run_nt<64, 2>(d, p, stream) : run_nt<64, 1>(d, p, stream);
  if (ng == 4) return run_nt<128, 4>(d, p, stream);
  return ng == 2 ? run_nt<128, 2>(d, p, stream) : run_nt<128, 1>(d, p, stream);
}

}  // namespace sparge
