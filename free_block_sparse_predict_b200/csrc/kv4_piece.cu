// Attention of many new tokens over the paged 4-bit cache: pieces of prompts,
// where the products bound it and not the cache's bytes.  The same mathematics
// as kv4_attn.cu on tcgen05, with K and V made fp16 tiles in shared memory.
//
// A unit is one KV head of a request and 256 rows of query tokens times heads
// of the group, in two tiles of 128; steps are of 64 keys.  A CTA of 16 warps
// per SM:
//   warp 0       bulk copies of the step's four 16-token tiles of codes
//   warp 1       tensor memory, and one thread that issues every tcgen05.mma:
//                S = Q K^T (128 x 64), a step ahead of the softmax, and O += P V
//   warps 4-7    codes to fp16: K and V rows of 128-byte-swizzled tiles
//   warps 8-15   softmax, a thread per row: mask, running maximum, P in fp16
//                over S, lazy rescale of O, the epilogue
// K and V are made once for both tiles.  Tensor memory holds two S of 64 columns
// and O per tile, so Q stays in shared memory: with Q in tensor memory and one S,
// each step waited for the last one's products (658 us, issued from a lane's number).
//
// Two prompts' last 512 tokens against 52,000 keys together, 32 heads of 128
// channels over 8, take 525 us: 4.4e11 floating-point operations at 0.83 PFLOP/s, 51 % of the
// library's rate for large products.  When it took 541, a step was 2,900 clocks, of which the products
// filled 1,500 (those of S, with half the columns that the pipe can take, are half
// of it); the softmax's 2,700 were the longest chain: 600 to load S and find its
// maximum, 1,600 for weights, of which the 1,024 of the exponential unit are
// shared by both tiles, and 400 from P to the next S.  Without the exponentials
// it took 490 us, without the codes' conversion 517, without either and the
// rest of the softmax's arithmetic 407.  Measured and not kept: the tiles taking turns at the
// exponentials (604), two warps per row with a step each, 24 warps with 88
// registers (720), polling without the barrier unit's suspension (725).
//
// Values: s c has 14 bits.  For bf16 outputs K and V are s c rounded to fp16
// (half of the codes lose nothing).  fp16
// outputs show that (K's rounding alone is two and a half times their own), so
// for them (SPLIT) K and V are each the sum of two tiles, the scale's upper
// eight bits and the rest times c, both exact, with two products.  A token of K or
// of V with a scale of 8192 or more (7 s would pass fp16's end) has its row halved, and its
// scores, or its weight in P, doubled: bits beside those of NaN scales tell the
// softmax warps.  (All rows halved lost the last bit of scales below 2^-13, and 2^-24
// itself.)  Q is fp16
// with one power of two per row, P is fp16 of weights up to 2^8, times 2^6, sums are
// float32.  A token whose scale of V is NaN makes the rows that see it NaN in
// every channel: its row of V must be zeros for those that do not, so it enters
// by its scores.
//
// The line of units is cut evenly over the CTAs and cut units are joined by
// the CTA that comes last, as in kv4_attn.cu.
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "after.cuh"
#include "kv4_common.cuh"
#include "kv4_layout.cuh"

namespace sparge {

using namespace kv4;
static_assert(kPieceRows == 256, "two tiles of 128 rows");

namespace {

constexpr int kPieceThreads = 512;
// Registers per thread at launch and after the warpgroups have split them: the
// shares add up to what the launch has, four times kLaunchRegs.
constexpr int kLaunchRegs = 128, kFeedRegs = 80, kCodeRegs = 96, kRowRegs = 168;
static_assert(kFeedRegs + kCodeRegs + 2 * kRowRegs <= 4 * kLaunchRegs, "register split");
constexpr int kTile = 128;           // rows of an MMA
constexpr int kRows = 2 * kTile;     // rows of a unit
constexpr int kKeys = 64;            // keys of a step
constexpr int kFlags = 16;           // steps whose tiles' validity is remembered
constexpr uint32_t kOdd = 16;        // some token of the step is one that s_odd names
constexpr float kRescale = 8.0f;     // log2 units
// Weights are held times 2^kLift, so that P, which may be doubled, ends at 2^15 and
// keeps its bits down to 2^-20 of the row's largest instead of 2^-14.
constexpr float kLift = 6.0f;
static_assert(kRescale + kLift + 1 <= 15, "P in fp16");
// A unit's start and end in steps: its queries, the pipeline's filling, the
// epilogue (some 12 us against 1.5 us a step; 5 to 10 measured the same).
constexpr int kUnitSteps = 8;

template <int D, int NG, bool SPLIT>
struct PieceCfg {
  static constexpr int CODES = 16 * (D + 4 * NG);      // a 16-token tile of the cache
  static constexpr int RAW = 4 * CODES;
  static constexpr int SLABS = D / 64;                 // 128-byte columns of K and V
  static constexpr int PARTS = SPLIT ? 2 : 1;          // tiles that add up to K, and to V
  static constexpr int ONE = kKeys * D * 2;
  static constexpr int KV = PARTS * ONE;               // K or V of a step
  static constexpr int QT = kTile * D * 2;             // a tile's queries
  static constexpr int Q = 0, K = 2 * QT, V = K + 2 * KV, CODE = V + 2 * KV;
  static constexpr int STAGES = SPLIT && D == 128 ? 3 : 4;  // steps of codes in flight: what fits
  static constexpr int SMEM = CODE + STAGES * RAW;
  // tensor memory per tile: S of even steps, of odd steps, each overwritten by its P | O
  static constexpr int TILE_COLS = 256, O_COL = 128;
  static_assert(SMEM + 4096 <= 227 * 1024, "one CTA per SM");
};

struct PieceBars {
  uint64_t raw_full[4], raw_empty[4];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  // per tile and parity of the step, since either side may be a step ahead of the
  // other's last look
  uint64_t s_full[2][2], p_full[2][2], o_done[2][2];
  uint64_t drain;
};

// What a CTA does next: a unit's steps [step0, step0 + n).
struct Part {
  Request req;
  int64_t steps_at, n_steps;  // of the unit: where its first stands in the line, how many
  int r, kvh, row0, rows, step0, n, n_tiles;
  bool cut, two;
};

struct Line {
  int64_t at, end, step, r_at;
  int r;
};

// The next part of this CTA's stretch of the line, if any.
__device__ __forceinline__ bool next_part(const DecodeArgs& A, Line& line, Part& p) {
  while (line.at < line.end) {
    p.req = request(A, line.r);
    p.n_steps = unit_steps<kKeys>(p.req);
    const int64_t n_units = unit_count<kRows>(A, p.req), length = p.n_steps + kUnitSteps;
    if (line.at >= line.r_at + n_units * length) {
      line.r_at += n_units * length;
      ++line.r;
      continue;
    }
    const int64_t unit = div64(line.at - line.r_at, length);
    p.steps_at = line.r_at + unit * length + kUnitSteps;
    p.step0 = int(max(line.at - p.steps_at, int64_t(0)));
    const int64_t stop = min(line.end, p.steps_at + p.n_steps);
    const int step1 = int(max(stop - p.steps_at, int64_t(0)));
    line.at = stop;
    if (step1 == p.step0) continue;  // the next CTA has all of it
    p.r = line.r;
    p.cut = p.step0 > 0 || step1 < p.n_steps;
    const int tile_of = A.heads.quot(int(unit));
    p.kvh = int(unit) - tile_of * A.Hkv;
    p.row0 = tile_of * kRows;
    p.rows = p.req.qlen * int(A.G.d);
    p.two = p.rows - p.row0 > kTile;
    // the last key that any row of the unit sees
    const int last = min(p.row0 + kRows, p.rows) - 1;
    const int32_t reach =
        A.causal ? min(p.req.keys, p.req.len - p.req.qlen + A.G.quot(last) + 1) : p.req.keys;
    p.n_tiles = reach > 0 ? (reach + 15) / 16 : 0;
    p.n = max(0, min(step1, (p.n_tiles + 3) / 4) - p.step0);
    return true;
  }
  return false;
}

template <int NREG>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(NREG));
}
template <int NREG>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(NREG));
}

constexpr uint32_t kHalves = 0x38003800u;  // 1/2, 1/2

// Eight codes (fp16 pairs) times their scale (in both halves of a word) as 16
// bytes, or, SPLIT, times the scale's upper eight bits and, `rest` bytes on, times
// what is left of it.
template <bool SPLIT>
__device__ __forceinline__ void put_chunk(uint8_t* to, int rest, uint32_t scale, uint32_t a,
                                          uint32_t b, uint32_t c, uint32_t d) {
  if constexpr (SPLIT) {
    const uint32_t u = scale & 0xFFF8FFF8u, r = minus(scale, u);
    *reinterpret_cast<uint4*>(to) = make_uint4(times(a, u), times(b, u), times(c, u), times(d, u));
    *reinterpret_cast<uint4*>(to + rest) =
        make_uint4(times(a, r), times(b, r), times(c, r), times(d, r));
  } else {
    *reinterpret_cast<uint4*>(to) =
        make_uint4(times(a, scale), times(b, scale), times(c, scale), times(d, scale));
  }
}

// The NG scales of one token's K or V, two to a word.
template <int NG>
__device__ __forceinline__ void scale_words(const uint8_t* at, uint32_t (&x)[(NG + 1) / 2]) {
  if constexpr (NG == 4) {
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    x[0] = w.x, x[1] = w.y;
  } else if constexpr (NG == 2) {
    x[0] = *reinterpret_cast<const uint32_t*>(at);
  } else {
    x[0] = *reinterpret_cast<const uint16_t*>(at);
  }
}
// Whether one is 8192 (0x7000) or more, or a NaN.
template <int N>
__device__ __forceinline__ bool any_large(const uint32_t (&x)[N]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) top |= x[i] + 0x10001000u;
  return top & 0x80008000u;
}

// A 16-byte chunk of row `row` (128-byte rows, 128-byte swizzle).
__device__ __forceinline__ uint32_t swizzled(int row, int chunk) {
  return uint32_t(row * 128 + ((chunk ^ (row & 7)) << 4));
}

template <int D, int NG, bool SPLIT>
__global__ void __launch_bounds__(kPieceThreads, 1) kv4_piece_kernel(const __grid_constant__ DecodeArgs A) {
  using C = PieceCfg<D, NG, SPLIT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) PieceBars bars;
  __shared__ int64_t s_scan[kPieceThreads / 32];
  __shared__ int64_t s_found[2];
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort, s_last;
  __shared__ uint32_t s_valid[kFlags];    // bit u: tile u of the step was copied; kOdd: see s_odd
  // keys of the step whose V has a NaN scale, whose K has a large one, whose V has one
  __shared__ uint32_t s_odd[kFlags][3][2];
  begin_after();
  if (smem_u32(smem) & 1023u) {  // the swizzle counts from 1024-byte boundaries
    if (threadIdx.x == 0) atomicCAS(A.status, 0, int32_t(SPARGE_EUNSUPPORTED));
    return;
  }
  volatile int* abort = &s_abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    s_abort = 0;
    for (int i = 0; i < C::STAGES; ++i) mbar_init(&bars.raw_full[i], 1), mbar_init(&bars.raw_empty[i], 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.k_full[i], 4), mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 4), mbar_init(&bars.v_empty[i], 1);
      for (int k = 0; k < 2; ++k)
        mbar_init(&bars.s_full[i][k], 1), mbar_init(&bars.p_full[i][k], 4),
            mbar_init(&bars.o_done[i][k], 1);
    }
    mbar_init(&bars.drain, 1);
    fence_mbar_init();
    fence_async_shared();
  }
  if (warp == 1) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }

  // ---- the line of units: its length, and the request where this part starts
  const int per = (A.R + kPieceThreads - 1) / kPieceThreads;
  const int r_lo = min(A.R, int(threadIdx.x) * per), r_hi = min(A.R, r_lo + per);
  int64_t own = 0;
  for (int r = r_lo; r < r_hi; ++r) {
    const Request x = request(A, r);
    own += unit_count<kRows>(A, x) * (unit_steps<kKeys>(x) + kUnitSteps);
    if (!x.sound && blockIdx.x == 0) atomicCAS(A.status, 0, int32_t(SPARGE_EINVAL));
  }
  int64_t incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) s_scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  int64_t total = 0, before = incl - own;
  for (int w = 0; w < kPieceThreads / 32; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  const int64_t parts = max(int64_t(1), min(int64_t(gridDim.x), total / kUnitSteps));
  Line line;
  line.step = max(int64_t(1), div64(total + parts - 1, parts));
  line.at = blockIdx.x * line.step;
  line.end = min(line.at + line.step, total);
  if (before <= line.at && line.at < before + own) {
    int64_t at = before;
    for (int r = r_lo; r < r_hi; ++r) {
      const Request x = request(A, r);
      const int64_t n = unit_count<kRows>(A, x) * (unit_steps<kKeys>(x) + kUnitSteps);
      if (line.at < at + n) {
        s_found[0] = r;
        s_found[1] = at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  line.r = int(s_found[0]);
  line.r_at = s_found[1];
  if (line.at >= total) line.end = line.at;  // nothing here

  Part p;
  uint32_t g = 0;          // steps of earlier parts
  uint32_t gt[2] = {0, 0};  // steps of earlier parts in which the tile took part
  bool ok = true;
  auto give_up = [&]() {
    *abort = 1;
    atomicExch(A.status, int32_t(SPARGE_ETIMEOUT));
  };

  if (warp < 4) {
    regs_down<kFeedRegs>();
    if (warp == 0) {
      // =================================================== codes
      while (next_part(A, line, p)) {
        __syncthreads();  // the queries are there
        const int32_t* table = A.table + int64_t(p.r) * A.max_pages;
        int32_t id = -1;  // lane: tile lane % 4 of step lane / 4 of the eight at hand
        for (int t = 0; t < p.n && ok; ++t) {
          if ((t & 7) == 0) {
            const int ti = 4 * (p.step0 + t) + lane;
            id = -1;
            if (ti < p.n_tiles) {
              const int32_t entry = A.tpp.quot(ti), page = table[entry];
              if (uint32_t(page) < uint32_t(A.num_pages))
                id = (page * A.Hkv + p.kvh - entry) * int32_t(A.tpp.d) + ti;
              else
                atomicCAS(A.status, 0, int32_t(SPARGE_EINVAL));
            }
          }
          const uint32_t n = g + t, stage = n % C::STAGES;
          if (n >= C::STAGES)
            ok = __all_sync(0xffffffffu,
                            mbar_wait(&bars.raw_empty[stage], (n / C::STAGES - 1) & 1, abort, A.status));
          if (!ok) break;
          const uint32_t there =
              __ballot_sync(0xffffffffu, id >= 0) >> (4 * (t & 7)) & 15u;
          uint8_t* dst = smem + C::CODE + stage * C::RAW;
          if (lane == 0) {
            s_valid[n % kFlags] = there;
#pragma unroll
            for (int i = 0; i < 6; ++i) s_odd[n % kFlags][i / 2][i % 2] = 0;
            if (there)
              mbar_expect_tx(&bars.raw_full[stage], __popc(there) * C::CODES);
            else
              mbar_arrive(&bars.raw_full[stage]);
          }
          __syncwarp();
          if (lane / 4 == (t & 7) && id >= 0)
            bulk_load(dst + (lane & 3) * C::CODES, A.cache + int64_t(id) * C::CODES, C::CODES,
                      &bars.raw_full[stage]);
          __syncwarp();
        }
        if (!ok && lane == 0) give_up();
        g += p.n;
        __syncthreads();  // the part is done
        if (p.cut) __syncthreads(), __syncthreads();
      }
      // copies in flight land before the CTA can end
      if (!ok && lane == 0)
        for (int s = 0; s < C::STAGES; ++s) {
          mbar_wait_teardown(&bars.raw_full[s], 0);
          mbar_wait_teardown(&bars.raw_full[s], 1);
        }
    } else if (warp == 1) {
      // =================================================== products
      bool drained = false;
      const uint32_t idesc_qk = instr_desc(1, 0, 0, 0, kTile, kKeys);
      const uint32_t idesc_pv = instr_desc(1, 0, 0, 1, kTile, D);
      // Descriptors step by their addresses' field, 16 bytes a unit
      const uint64_t dq = smem_desc(smem_u32(smem + C::Q), 16, 1024);
      const uint64_t dk = smem_desc(smem_u32(smem + C::K), 16, 1024);
      const uint64_t dv = smem_desc(smem_u32(smem + C::V), kKeys * 128, 1024);
      while (next_part(A, line, p)) {
        __syncthreads();
        tc_fence_after();
        const int tiles = p.two ? 2 : 1;
        if (elect_one()) {
          auto scores = [&](int i, int t) {  // S of tile i and step t
            const uint32_t m = gt[i] + t, b = (g + t) & 1;
            const uint32_t at = tmem + uint32_t(i * C::TILE_COLS) + (m & 1) * kKeys;
#pragma unroll
            for (int kk = 0; kk < C::PARTS * (D / 16); ++kk) {
              const int slab = kk % (D / 16) / 4, within = (kk % 4) * 32, rest = kk / (D / 16);
              mma_f16_ss(at, dq + (i * C::QT + slab * (kTile * 128) + within) / 16,
                         dk + b * (C::KV / 16) +
                             (rest * C::ONE + slab * (kKeys * 128) + within) / 16,
                         idesc_qk, kk > 0 ? 1u : 0u);
            }
            mma_commit(&bars.s_full[i][m & 1]);
          };
          auto values = [&](int i, int t) {  // O += P V
            const uint32_t m = gt[i] + t, b = (g + t) & 1;
            const uint32_t base = tmem + uint32_t(i * C::TILE_COLS);
#pragma unroll
            for (int kk = 0; kk < C::PARTS * (kKeys / 16); ++kk) {
              const int step = kk % (kKeys / 16), rest = kk / (kKeys / 16);
              mma_f16_ts(base + C::O_COL, base + (m & 1) * kKeys + step * 8,
                         dv + b * (C::KV / 16) + (rest * C::ONE + step * 2048) / 16, idesc_pv,
                         (t > 0 || kk > 0) ? 1u : 0u);
            }
            mma_commit(&bars.o_done[i][m & 1]);
          };
          auto keys_there = [&](int t) {
            const uint32_t n = g + t;
            if (!mbar_wait(&bars.k_full[n & 1], (n >> 1) & 1, abort, A.status)) return false;
            tc_fence_after();
            return true;
          };
          // S of the next step comes before P V of this one, so that the softmax need
          // not wait for it; its columns were those of P two steps back, whose P V has
          // been issued before it.  The order S0, P V0, S1, P V1 of the tiles took 4 %
          // less time than both S before both P V.
          if (ok && p.n > 0 && (ok = keys_there(0))) {
            for (int i = 0; i < tiles; ++i) scores(i, 0);
            mma_commit(&bars.k_empty[g & 1]);
          }
          for (int t = 0; t < p.n && ok; ++t) {
            const uint32_t n = g + t, b = n & 1;
            const bool more = t + 1 < p.n;
            if (more && !(ok = keys_there(t + 1))) break;
            for (int i = 0; i < tiles; ++i) {
              const uint32_t m = gt[i] + t;
              if (more) scores(i, t + 1);
              if (more && i + 1 == tiles) mma_commit(&bars.k_empty[b ^ 1]);
              ok = mbar_wait(&bars.p_full[i][m & 1], (m >> 1) & 1, abort, A.status) &&
                   (i > 0 || mbar_wait(&bars.v_full[b], (n >> 1) & 1, abort, A.status));
              if (!ok) break;
              tc_fence_after();
              values(i, t);
            }
            if (!ok) break;
            mma_commit(&bars.v_empty[b]);
          }
          if (!ok && !drained) {
            give_up();
            // products in flight end before the tensor memory is given back
            mma_commit(&bars.drain);
            mbar_wait_teardown(&bars.drain, 0);
            drained = true;
          }
        }
        __syncwarp();
        g += p.n;
        for (int i = 0; i < tiles; ++i) gt[i] += p.n;
        __syncthreads();
        if (p.cut) __syncthreads(), __syncthreads();
      }
    } else {
      while (next_part(A, line, p)) {
        __syncthreads(), __syncthreads();
        if (p.cut) __syncthreads(), __syncthreads();
      }
    }
  } else if (warp < 8) {
    // =================================================== codes to fp16
    regs_down<kCodeRegs>();
    const int th = threadIdx.x - 128;
    const Masks masks = A.masks;
    while (next_part(A, line, p)) {
      __syncthreads();
      for (int t = 0; t < p.n && ok; ++t) {
        const uint32_t n = g + t, stage = n % C::STAGES, b = n & 1;
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&bars.raw_full[stage], (n / C::STAGES) & 1, abort, A.status) &&
                            (n < 2 || mbar_wait(&bars.k_empty[b], ((n >> 1) - 1) & 1, abort, A.status)));
        if (!ok) break;
        const uint8_t* raw = smem + C::CODE + stage * C::RAW;
        const uint32_t there = s_valid[n % kFlags] & 15u;
        const int left = p.req.keys - (p.step0 + t) * kKeys;  // tokens of the step that exist
        // the scales by which threads 0-63 look at V's tokens, the others at K's (below)
        uint32_t look[(NG + 1) / 2];
        scale_words<NG>(raw + (th % kKeys >> 4) * C::CODES + 16 * D + (th & 15) * NG * 4 +
                            (th < kKeys ? 2 * NG : 0), look);
        // K: word w = t (D / 32) + j of a token's row is its chunk 4 j + t; a thread
        // has the same word of every TOKS-th token
        {
          constexpr int WORDS = D / 8, TOKS = 128 / WORDS;  // 8 (d = 128) or 16 at once
          const int w = th % WORDS, j = w % (D / 32), chunk = 4 * j + w / (D / 32), t0 = th / WORDS;
          uint8_t* to = smem + C::K + b * C::KV + (chunk >> 3) * (kKeys * 128);
          uint32_t word[kKeys / TOKS], scale[kKeys / TOKS];
          const int group = j / (D / 32 / NG);
          const uint32_t own = group & 1 ? 0x3232u : 0x1010u;
#pragma unroll
          for (int k = 0; k < kKeys / TOKS; ++k) {
            const uint8_t* tile = raw + k * TOKS / 16 * C::CODES;
            const int tok = t0 + k * TOKS % 16;
            word[k] = *reinterpret_cast<const uint32_t*>(tile + tok * (D / 2) + w * 4);
            uint32_t x[(NG + 1) / 2];
            scale_words<NG>(tile + 16 * D + tok * NG * 4, x);
            scale[k] = __byte_perm(NG == 4 && group & 2 ? x[(NG - 1) / 2] : x[0], 0u, own);
            if (any_large(x)) scale[k] = times(scale[k], kHalves);
          }
#pragma unroll
          for (int k = 0; k < kKeys / TOKS; ++k) {
            const uint32_t hi = word[k] >> 8;
            put_chunk<SPLIT>(to + swizzled(t0 + k * TOKS, chunk & 7), C::ONE, scale[k],
                             codes0(word[k], masks), codes4(word[k], masks), codes0(hi, masks),
                             codes4(hi, masks));
          }
        }
        // what the softmax warps have to know of a token
        {
          const int tok = th % kKeys;
          if (any_large(look) && tok < left && (there >> (tok >> 4) & 1u)) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < NG; ++i) nan |= (look[i / 2] >> (16 * (i % 2)) & 0x7FFFu) > 0x7C00u;
            atomicOr(&s_odd[n % kFlags][th >= kKeys ? 1 : (nan ? 0 : 2)][tok >> 5], 1u << (tok & 31));
            atomicOr(&s_valid[n % kFlags], kOdd);
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.k_full[b]);
        // V: a thread per token and half h of its words: four chunks of eight
        // channels, byte i of the words 4 h .. 4 h + 3 being chunk 2 i + h
        if (n >= 2)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&bars.v_empty[b], ((n >> 1) - 1) & 1, abort, A.status));
        if (!ok) break;
        {
          const int tok = th % kKeys, h = th / kKeys;
          const uint8_t* tile = raw + (tok >> 4) * C::CODES;
          uint32_t x[(NG + 1) / 2];
          scale_words<NG>(tile + 16 * D + (tok & 15) * NG * 4 + 2 * NG, x);
          const bool large = any_large(x);
          const uint8_t* codes = tile + 8 * D + (4 * h * 16 + Kv4Tile::v_pos(tok & 15)) * 4;
          const bool in = (there >> (tok >> 4) & 1u) && tok < left;
          uint32_t words[C::SLABS][4], scale[NG];
#pragma unroll
          for (int w = 0; w < C::SLABS; ++w)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              words[w][k] = *reinterpret_cast<const uint32_t*>(codes + w * 512 + k * 64);
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            scale[i] = __byte_perm(x[i / 2], 0u, i % 2 ? 0x3232u : 0x1010u);
            if (large) scale[i] = times(scale[i], kHalves);
            if (!in || (scale[i] & 0x7FFFu) > 0x7C00u) scale[i] = 0;  // no row may meet it
          }
#pragma unroll
          for (int w = 0; w < C::SLABS; ++w) {
            uint8_t* to = smem + C::V + b * C::KV + w * (kKeys * 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t c[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // byte i in both half-words: its low half as 1024 + u, its high half
                // (bits 4-7 of the upper) as 64 + u
                const uint32_t two =
                    __byte_perm(words[w][k], 0u, uint32_t(i) | 0x4040u | uint32_t(i) << 8);
                c[k] = minus(pick(two, masks.mixed, 0x54006400u), 0x54806408u);
              }
              put_chunk<SPLIT>(to + swizzled(tok, 2 * i + h), C::ONE,
                               scale[(64 * w + 16 * i) / (D / NG)], c[0], c[1], c[2], c[3]);
            }
          }
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bars.v_full[b]);
          mbar_arrive(&bars.raw_empty[stage]);
        }
      }
      if (!ok && lane == 0) give_up();
      g += p.n;
      __syncthreads();
      if (p.cut) __syncthreads(), __syncthreads();
    }
  } else {
    // =================================================== softmax
    regs_up<kRowRegs>();
    const int tile = (warp - 8) >> 2, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t at = tmem + uint32_t(tile * C::TILE_COLS) + (uint32_t(quad * 32) << 16);
    while (next_part(A, line, p)) {
      const int row = p.row0 + tile * kTile + r;
      const bool row_ok = row < p.rows;
      const bool active = tile == 0 || p.two;
      float f = 0.f;  // log2 units of a unit of S
      int32_t lim = 0;
      uint32_t qw[D / 64][32] = {};
      if (row_ok) {
        const int tok = A.G.quot(row), head = p.kvh * int(A.G.d) + row - tok * int(A.G.d);
        lim = A.causal ? min(p.req.keys, p.req.len - p.req.qlen + tok + 1) : p.req.keys;
        const uint4* src = reinterpret_cast<const uint4*>(
            A.q + int64_t(p.req.q0 + tok) * A.q_stride + int64_t(head) * (D * 2));
        uint4 raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) raw[i] = src[i];
        // the row's largest to [2^12, 2^13) (a subnormal below); two factors, since
        // one may overflow
        float big = 0.f;
        const auto both = [&](uint32_t u) {
          return A.bf16 ? make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u))
                        : half2_f(u);
        };
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = both(u[e]);
            big = fmaxf(big, fmaxf(fabsf(x.x), fabsf(x.y)));
          }
        }
        const int field = int(__float_as_uint(big) >> 23);
        const int k = field < 255 ? 139 - field : 0, half_k = k >> 1;
        const auto two_to = [](int n) { return __uint_as_float(uint32_t(n + 127) << 23); };
        const float k1 = two_to(half_k), k2 = two_to(k - half_k);
        f = A.scale_log2 * two_to(-half_k) * two_to(half_k - k);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t u[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = both(u[e]);
            qw[i / 8][4 * (i % 8) + e] = pack_half2(x.x * k1 * k2, x.y * k1 * k2);
          }
        }
      }
      if (active) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t* w = &qw[i / 8][4 * (i % 8)];
          *reinterpret_cast<uint4*>(smem + C::Q + tile * C::QT + i / 8 * (kTile * 128) +
                                    swizzled(r, i % 8)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_async_shared();
      }
      tc_fence_before();
      __syncthreads();  // the queries are there

      float m = -INFINITY, l = 0.f;  // the maximum P is scaled by, and the sum
      const int steps = active ? p.n : 0;
      for (int t = 0; t < steps; ++t) {
        const uint32_t n = gt[tile] + t, at_s = at + (n & 1) * kKeys;
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&bars.s_full[tile][n & 1], (n >> 1) & 1, abort, A.status));
        if (!ok) break;
        tc_fence_after();
        uint32_t raw[64];
        {
          uint32_t(&r0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&raw[0]);
          uint32_t(&r1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&raw[32]);
          tmem_ld32(at_s, r0);
          tmem_ld32(at_s + 32, r1);
          tmem_wait_ld_fence(r0);
          tmem_wait_ld_fence(r1);
        }
        const int seen = lim - (p.step0 + t) * kKeys;  // keys c < seen
        const uint32_t flags = s_valid[(g + t) % kFlags], there = flags & 15u;
        const uint32_t(&odd)[3][2] = s_odd[(g + t) % kFlags];
        if (flags & kOdd) {
          const uint32_t nan[2] = {odd[0][0], odd[0][1]}, large[2] = {odd[1][0], odd[1][1]};
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            if (large[c >> 5] >> (c & 31) & 1u)
              raw[c] = __float_as_uint(2.0f * __uint_as_float(raw[c]));
            if (nan[c >> 5] >> (c & 31) & 1u) raw[c] = 0x7FFFFFFFu;
          }
        }
        // whether some row of the warp does not see some key of the step
        const bool masked = __any_sync(0xffffffffu, seen < kKeys || there != 15u);
        uint32_t vis[2] = {~0u, ~0u};  // bit c: key c is seen
        if (masked) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const int left = min(max(seen - 32 * w, 0), 32);
            vis[w] = left == 32 ? ~0u : (1u << left) - 1u;
            vis[w] &= (there >> (2 * w) & 1u ? 0xFFFFu : 0u) | (there >> (2 * w + 1) & 1u ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (!(vis[c >> 5] >> (c & 31) & 1u)) raw[c] = 0xFF800000u;  // -inf
        }
        float top[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          top[k] = __uint_as_float(raw[k]);
#pragma unroll
          for (int c = k + 4; c < 64; c += 4) top[k] = fmaxf(top[k], __uint_as_float(raw[c]));
        }
        const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        const float high = most == -INFINITY ? -INFINITY : most * f;
        // O's row is rescaled once the maximum has grown by more than 2^8
        const bool grow = high > m + kRescale;
        const bool rescale = grow && m != -INFINITY;
        if (__any_sync(0xffffffffu, rescale)) {
          // (a maximum that grows is not the part's first: t > 0)
          ok = __all_sync(0xffffffffu, mbar_wait(&bars.o_done[tile][(n - 1) & 1], ((n - 1) >> 1) & 1,
                                                 abort, A.status));
          if (!ok) break;
          tc_fence_after();
          const float shrink = rescale ? ex2_approx(m - high) : 1.f;
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t o[32];
            tmem_ld32(at + C::O_COL + cc * 32, o);
            tmem_wait_ld_fence(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * shrink);
            tmem_st32(at + C::O_COL + cc * 32, o);
          }
          tmem_wait_st();
          if (rescale) l *= shrink;
        }
        if (grow) m = high;
        const float nb = m == -INFINITY ? 0.f : kLift - m;
        const uint64_t f2 = pack2(f, f), nb2 = pack2(nb, nb);
        uint32_t pk[32];
        uint64_t sum[4] = {0, 0, 0, 0};
        // (two copies: with the choice inside, the exponentials of all keys come
        // before the first sum)
        const auto weigh = [&](auto some_masked) {
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float y0, y1;
            unpack2(fma2(pack2(__uint_as_float(raw[c]), __uint_as_float(raw[c + 1])), f2, nb2), y0, y1);
            y0 = ex2_approx(y0);
            y1 = ex2_approx(y1);
            if constexpr (some_masked) {  // (-inf times f is a NaN where f is 0)
              if (!(vis[c >> 5] >> (c & 31) & 1u)) y0 = 0.f;
              if (!(vis[c >> 5] >> ((c & 31) + 1) & 1u)) y1 = 0.f;
            }
            sum[(c >> 1) & 3] = add2(sum[(c >> 1) & 3], pack2(y0, y1));
            pk[c / 2] = pack_half2(y0, y1);
          }
        };
        if (masked) weigh(std::true_type{}); else weigh(std::false_type{});
        float s0, s1;
        unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), s0, s1);
        l += s0 + s1;
        if (flags & kOdd) {
          const uint32_t large[2] = {odd[2][0], odd[2][1]};
#pragma unroll
          for (int c = 0; c < 64; c += 2) {  // 1 or 2 in each half
            const uint32_t two = large[c >> 5] >> (c & 31) & 3u;
            pk[c / 2] = times(pk[c / 2], (two & 1u ? 0x4000u : 0x3C00u) | (two & 2u ? 0x40000000u : 0x3C000000u));
          }
        }
        tmem_st32(at_s, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.p_full[tile][n & 1]);
      }
      if (!ok && lane == 0) give_up();
      // ---- epilogue
      if (ok && steps > 0) {
        const uint32_t n = gt[tile] + steps - 1;
        ok = __all_sync(0xffffffffu,
                        mbar_wait(&bars.o_done[tile][n & 1], (n >> 1) & 1, abort, A.status));
        if (!ok && lane == 0) give_up();
      }
      tc_fence_after();
      const int64_t slot = 2 * int64_t(blockIdx.x) + (p.step0 > 0 ? 0 : 1);
      const int64_t part_row = slot * kRows + tile * kTile + r;
      const float top = m == -INFINITY ? kLow : m;
      const float inv = l == 0.f ? 0.f : 1.0f / l;
      if (active && ok) {
        const int64_t orow = row_ok ? out_row(A, p.req, p.kvh, row) : 0;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32] = {};
          if (steps > 0) {
            tmem_ld32(at + C::O_COL + cc * 32, o);
            tmem_wait_ld_fence(o);
          }
          if (!row_ok) continue;
          if (p.cut) {
            float4* dst = reinterpret_cast<float4*>(A.part_o + part_row * D + cc * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e)
              dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                   __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
          } else {
            uint4* dst = reinterpret_cast<uint4*>(A.o + (orow * D + cc * 32) * 2);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float x = l == 0.f ? 0.f : __uint_as_float(o[8 * e + 2 * k]) * inv;
                const float y = l == 0.f ? 0.f : __uint_as_float(o[8 * e + 2 * k + 1]) * inv;
                if (A.bf16) {
                  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
                  w[k] = *reinterpret_cast<const uint32_t*>(&h);
                } else {
                  w[k] = pack_half2(x, y);
                }
              }
              dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (row_ok) {
          if (p.cut)
            A.part_ml[part_row] = make_float2(top, l);
          else if (A.lse != nullptr)
            A.lse[orow] = l == 0.f ? -INFINITY : (top + (log2f(l) - kLift)) * 0.6931471805599453f;
        }
      }
      tc_fence_before();
      if (p.cut) __threadfence();
      g += p.n;
      gt[0] += p.n;
      if (p.two) gt[1] += p.n;
      __syncthreads();  // the part is done
      if (!p.cut) continue;
      // ---- the last of a cut unit's CTAs joins its parts, in their order, a warp per row
      const int64_t c0 = p.step0 == 0 ? int64_t(blockIdx.x) : div64(p.steps_at, line.step);
      const int n_parts = int(div64(p.steps_at + p.n_steps - 1, line.step) - c0) + 1;
      if (threadIdx.x == 256)
        s_last = atomicInc(A.arrived + c0, uint32_t(n_parts - 1)) == uint32_t(n_parts - 1);
      __syncthreads();
      if (s_last) {
        __threadfence();
        constexpr int V = D / 32;  // channels per lane
        for (int rr = warp - 8; rr < kRows && p.row0 + rr < p.rows; rr += 8) {
          float big = kLow;
          for (int k = 0; k < n_parts; ++k)
            big = fmaxf(big, __ldcg(A.part_ml + (2 * (c0 + k) + (k == 0)) * kRows + rr).x);
          float sum = 0.f, x[V];
#pragma unroll
          for (int v = 0; v < V; ++v) x[v] = 0.f;
#pragma unroll 2
          for (int k = 0; k < n_parts; ++k) {
            const int64_t prow = (2 * (c0 + k) + (k == 0)) * kRows + rr;
            const float2 ml = __ldcg(A.part_ml + prow);
            const float a = ex2_approx(ml.x - big);
            sum = fmaf(ml.y, a, sum);
            const float2* src = reinterpret_cast<const float2*>(A.part_o + prow * D + V * lane);
#pragma unroll
            for (int v = 0; v < V; v += 2) {
              const float2 q = __ldcg(src + v / 2);
              if (ml.y != 0.f) x[v] = fmaf(q.x, a, x[v]), x[v + 1] = fmaf(q.y, a, x[v + 1]);
            }
          }
          const int64_t orow = out_row(A, p.req, p.kvh, p.row0 + rr);
#pragma unroll
          for (int v = 0; v < V; v += 2)
            write_out(A, orow, D, V * lane + v, big - kLift, sum, x[v], x[v + 1]);
        }
      }
      __syncthreads();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int D, int NG, bool SPLIT>
cudaError_t run_one(const DecodeArgs& a, int grid, cudaStream_t stream) {
  using C = PieceCfg<D, NG, SPLIT>;
  const cudaError_t e = cudaFuncSetAttribute(
      kv4_piece_kernel<D, NG, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  // the register split waits for registers that a smaller launch would not have
  cudaFuncAttributes fa;
  const cudaError_t f = cudaFuncGetAttributes(&fa, kv4_piece_kernel<D, NG, SPLIT>);
  if (f != cudaSuccess) return f;
  if (fa.numRegs != kLaunchRegs) return cudaErrorNotSupported;
  return launch_after(kv4_piece_kernel<D, NG, SPLIT>, dim3(unsigned(grid)), kPieceThreads, C::SMEM,
                      stream, a);
}

template <int D, int NG>
cudaError_t run(const DecodeArgs& a, int grid, cudaStream_t s) {
  return a.bf16 ? run_one<D, NG, false>(a, grid, s) : run_one<D, NG, true>(a, grid, s);
}

}  // namespace

cudaError_t kv4::launch_kv4_piece(const DecodeArgs& a, int d, int ng, int grid, cudaStream_t s) {
  if (d == 64) return ng == 2 ? run<64, 2>(a, grid, s) : run<64, 1>(a, grid, s);
  if (ng == 4) return run<128, 4>(a, grid, s);
  return ng == 2 ? run<128, 2>(a, grid, s) : run<128, 1>(a, grid, s);
}

}  // namespace sparge
