// The bookkeeping of one step of a paged cache: pages of ended requests go back
// to the free stack, requests with new tokens get the pages they need from it,
// and every new token gets its slot.
//
// With L the length of request r, n its new tokens and P the page size:
//   have_r = ceil(L / P), need_r = ceil((L + n) / P) - have_r,
//   r is admitted iff its tokens fit and need_r = 0 or sum_{r' <= r} need_r' <= available,
//   its i-th new page is free[available - 1 - sum_{r' < r} need_r' - i],
//   token t of it, at position q = L + t, has slot page(q / P) * P + q % P.
// All sums are prefix sums over the requests, so the result does not depend on
// timing.  Latency-bound: a few KB of metadata, then 4 bytes written per token.
//
// One launch does it, with one barrier over its CTAs.  Every CTA takes the prefix
// sums over all requests for itself (they are in L2 after the first).  Before
// the barrier all inputs that may be outputs too are read, and the pages of
// ended requests are pushed (above the stack's top, where nothing else is read);
// behind it the outputs are written and the new pages are taken.  Measured: 256
// requests with a token each in 5.6 us, 500 with a million together in 10.7.
#include <cooperative_groups.h>

#include <cstdint>

#include "after.cuh"
#include "div.cuh"
#include "sparge_internal.h"

namespace sparge {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 4;  // requests per thread
constexpr int kBatch = 8;    // pages that come back, in flight per thread
constexpr int kPlanMax = kPlanThreads * kPlanPer;
static_assert(kPlanMax == kMaxPlanRequests, "every request has a thread");

// Exclusive prefix sums of N values per thread, in place; total gets the sums.
// sh: 32 values for each of the N.
template <int N>
__device__ __forceinline__ void block_scan(int64_t (&v)[N], int64_t* sh, int64_t (&total)[N]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t incl[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    incl[k] = v[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl[k], o);
      if (lane >= o) incl[k] += up;
    }
    if (lane == 31) sh[32 * k + w] = incl[k];
  }
  __syncthreads();
  if (w < N) {
    int64_t s = sh[32 * w + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    sh[32 * w + lane] = s;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    total[k] = sh[32 * k + 31];
    v[k] = (w > 0 ? sh[32 * k + w - 1] : 0) + incl[k] - v[k];
  }
}

// Pages of that many tokens, 0 <= tokens < 2^31.
__device__ __forceinline__ int32_t pages_of(int32_t tokens, const Div& page) {
  return tokens > 0 ? page.quot(tokens - 1) + 1 : 0;
}

// RUN: consecutive tokens per thread and step.  GRID: the CTAs are the whole
// cooperative grid instead of one cluster.
template <int RUN, bool GRID>
__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const KvPlanArgs A, const Div page,
                                                               const uint32_t id_end) {
  namespace cg = cooperative_groups;
  const int rank = int(blockIdx.x), ctas = int(gridDim.x);
  __shared__ int64_t sh1[64], sh2[32];
  __shared__ unsigned long long s_popped;
  extern __shared__ int32_t s_dyn[];
  int32_t* s_cu = s_dyn;             // [R + 1] start of each request's tokens
  int32_t* s_len = s_cu + A.R + 1;   // [R] L; -1: no tokens or not admitted; -2 - L: ended
  int32_t* s_off = s_len + A.R;      // [R] pages pushed (ended) or popped before it

  begin_after();

  const int32_t P = A.page_size;
  const int64_t cap = int64_t(A.max_pages) * P;
  int64_t count = *A.free_count;
  count = count < 0 ? 0 : (count > A.num_pages ? A.num_pages : count);

  if (threadIdx.x == 0) s_popped = 0;

  // ---- lengths, what comes back, where tokens start; `per` requests a thread
  const int per = (A.R + kPlanThreads - 1) / kPlanThreads, first = threadIdx.x * per;
  int32_t L[kPlanPer], n[kPlanPer];
  int64_t sums[2] = {0, 0};  // tokens, pages that come back
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int r = first + i;
    L[i] = n[i] = 0;
    if (i < per && r < A.R) {
      const int32_t l = A.seq_len[r];
      L[i] = l < 0 ? 0 : int32_t(l > cap ? cap : l);
      n[i] = A.new_len[r];
    }
    if (n[i] > 0) sums[0] += n[i];
    if (n[i] < 0) sums[1] += pages_of(L[i], page);
  }
  int64_t totals[2];
  block_scan(sums, sh1, totals);
  int64_t cu = sums[0], put = sums[1];
  const int64_t tokens = totals[0];
  int64_t avail = count + totals[1];
  if (avail > A.num_pages) avail = A.num_pages;

  // ---- pages needed, admission
  int64_t at = cu, upto[1] = {0}, all[1];
  int32_t want[kPlanPer];
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int64_t after = int64_t(L[i]) + n[i];
    want[i] = -1;  // does not fit (or brings nothing)
    if (n[i] > 0) {
      at += n[i];
      if (after <= cap && at <= A.max_tokens)
        want[i] = pages_of(int32_t(after), page) - pages_of(L[i], page);
    }
    if (want[i] > 0) upto[0] += want[i];
  }
  block_scan(upto, sh2, all);
  int64_t popped = 0;  // pages that went up to this thread's last admitted request
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int r = first + i;
    if (i >= per || r >= A.R) break;
    const int64_t before = upto[0];
    if (want[i] > 0) upto[0] += want[i];
    const bool ok = want[i] == 0 || (want[i] > 0 && upto[0] <= avail);
    if (ok && want[i] > 0) popped = upto[0];
    s_cu[r] = int32_t(cu > INT32_MAX ? INT32_MAX : cu);
    s_len[r] = ok ? L[i] : -1;
    const int64_t off = n[i] < 0 ? put : before;
    s_off[r] = int32_t(off > INT32_MAX ? INT32_MAX : off);
    if (n[i] > 0) cu += n[i];
    if (n[i] < 0) {
      s_len[r] = -2 - L[i];  // ended
      put += pages_of(L[i], page);
    }
  }
  if (threadIdx.x == 0) s_cu[A.R] = int32_t(tokens > INT32_MAX ? INT32_MAX : tokens);
  // needs grow along the requests, so what is taken is the largest sum admitted
  if (popped > 0) atomicMax(&s_popped, (unsigned long long)popped);

  // ---- pages of ended requests, a warp per request
  __syncthreads();
  const int lane = threadIdx.x & 31;
  for (int r = int(threadIdx.x >> 5) * ctas + rank; r < A.R; r += kPlanThreads / 32 * ctas) {
    if (s_len[r] > -2) continue;
    const int pages = pages_of(-2 - s_len[r], page);
    const int32_t* row = A.block_table + int64_t(r) * A.max_pages;
    int32_t* to = A.free_pages + count + s_off[r];
    const int room = int(min(int64_t(pages), A.num_pages - count - s_off[r]));
    for (int j0 = lane; j0 < room; j0 += 32 * kBatch) {
      int32_t id[kBatch];  // loads first: one latency for all
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (j0 + 32 * k < room) id[k] = row[j0 + 32 * k];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (j0 + 32 * k < room) to[j0 + 32 * k] = id[k];
    }
  }

  if (GRID) cg::this_grid().sync(); else cg::this_cluster().sync();

  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = first + i;
      if (i >= per || r >= A.R) break;
      const bool ok = s_len[r] >= 0;
      A.seq_len_out[r] = n[i] < 0 ? 0 : (ok ? L[i] + n[i] : L[i]);
      A.admitted[r] = ok || n[i] <= 0;
      A.cu_new[r] = s_cu[r];
    }
    if (threadIdx.x == 0) {
      A.cu_new[A.R] = s_cu[A.R];
      *A.free_count_out = int32_t(avail - int64_t(s_popped));
    }
  }

  // ---- slots: RUN consecutive tokens per thread and step, so that the search
  // for the request is paid once for them; the first token of a new page writes
  // its table entry
  const int32_t end = s_cu[A.R];
  static_assert(kMaxPlanTokens - 1 <= INT32_MAX - RUN, "t0 + RUN below fits 32 bits");
  const int64_t runs = (int64_t(A.max_tokens) + RUN - 1) / RUN;
  const bool vec = (reinterpret_cast<uintptr_t>(A.slot_map) & 15u) == 0;
  for (int64_t n = int64_t(rank) * kPlanThreads + threadIdx.x; n < runs;
       n += int64_t(ctas) * kPlanThreads) {
    const int32_t t0 = int32_t(n * RUN);
    int32_t slot[RUN];
#pragma unroll
    for (int i = 0; i < RUN; ++i) slot[i] = -1;
    if (t0 < end) {
      int r = 0, hi = A.R;  // the last request that starts at or before t0
      while (hi - r > 1) {
        const int mid = (r + hi) >> 1;
        if (s_cu[mid] <= t0) r = mid; else hi = mid;
      }
      // page p of request r, of which `have` pages were there before; its first
      // token writes the table entry
      auto page_id = [&](int r, int32_t p, int32_t have, bool write) {
        int32_t* entry = A.block_table + int64_t(r) * A.max_pages + p;
        if (p < have) return *entry;
        const int32_t id = A.free_pages[avail - 1 - s_off[r] - (p - have)];
        if (write) *entry = id;
        return id;
      };
      // (a number whose slots pass 32 bits is no page's: slots below 0, not another page's)
      const auto first_slot = [&](int32_t id) {
        const bool fits = uint32_t(id) < id_end || uint32_t(~id) < id_end;
        return fits ? uint32_t(id) * uint32_t(P) : 0x80000000u;
      };
      if (RUN > 1 && t0 + RUN <= s_cu[r + 1] && P >= RUN) {
        // all of one request and of one or two of its pages: nearly every run
        const int32_t len = s_len[r];
        if (len >= 0) {
          const int32_t pos = len + (t0 - s_cu[r]), p = page.quot(pos), have = pages_of(len, page);
          const int32_t in = pos - p * P;
          const uint32_t a = first_slot(page_id(r, p, have, in == 0)) + in;
          uint32_t b = 0;  // so that b + i is token i's slot, if it is in the next page
          if (in + RUN > P) b = first_slot(page_id(r, p + 1, have, true)) + in - P;
#pragma unroll
          for (int i = 0; i < RUN; ++i) slot[i] = int32_t((in + i < P ? a : b) + i);
        }
      } else {
        int32_t next = s_cu[r + 1];    // where the request's tokens end
        int32_t in = P, slot_at = -1;  // offset in the page at hand (P: none), next slot
        for (int i = 0; i < RUN && t0 + i < end; ++i) {
          const int32_t t = t0 + i;
          while (t >= next) next = s_cu[++r + 1], in = P;
          const int32_t len = s_len[r];
          if (len < 0) continue;
          if (in == P) {  // another page
            const int32_t pos = len + (t - s_cu[r]), p = page.quot(pos);
            in = pos - p * P;
            slot_at = int32_t(first_slot(page_id(r, p, pages_of(len, page), in == 0)) + in);
          }
#pragma unroll
          for (int k = 0; k < RUN; ++k)
            if (k == i) slot[k] = slot_at;
          ++slot_at;
          ++in;
        }
      }
    }
    if (RUN % 4 == 0 && vec && t0 + RUN <= A.max_tokens) {
#pragma unroll
      for (int i = 0; i + 3 < RUN; i += 4)
        *reinterpret_cast<int4*>(A.slot_map + t0 + i) =
            make_int4(slot[i], slot[i + 1], slot[i + 2], slot[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < RUN; ++i)
        if (t0 + i < A.max_tokens) A.slot_map[t0 + i] = slot[i];
    }
  }
}

template <int RUN, bool GRID>
cudaError_t run(const KvPlanArgs& a, int max_ctas, cudaStream_t stream) {
  const auto kernel = plan_kernel<RUN, GRID>;
  cudaLaunchConfig_t cfg{};
  // a thread for RUN tokens, up to max_ctas CTAs
  const int64_t ctas = cdiv(a.max_tokens, int64_t(RUN) * kPlanThreads);
  int n = 1;
  if (GRID) n = int(ctas < max_ctas ? ctas : max_ctas);
  while (!GRID && n < max_ctas && n < ctas) n <<= 1;
  cfg.gridDim = dim3(unsigned(n));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (3 * size_t(a.R) + 1) * sizeof(int32_t);
  if (cfg.dynamicSmemBytes > 46 * 1024) {  // 48 KB with the static part need no permission
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               int((3 * kPlanMax + 1) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  if (GRID) {
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
  } else {
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(n);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = attr;
  cfg.numAttrs = GRID ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, kernel, a, make_div(uint32_t(a.page_size)),
                            0x80000000u / uint32_t(a.page_size));
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  // A decode step has about a token per request: a thread each (runs of eight
  // would fetch eight requests' pages one after the other, 9.9 instead of 5.9 us
  // for 256), in a cluster of eight at most.  Prompts' tokens share requests and
  // pages, and writing their slots wants every SM: 10.7 us for 500 prompts of up
  // to 4096 tokens, 29 us in a cluster of sixteen.  The grid's barrier costs
  // about 2 us more than a cluster's: 16,000 tokens take 7.3 us in a cluster and
  // 9.3 us in the grid, 64,000 tokens 13.6 and 8.7 us.
  constexpr int kCluster = 8;
  if (a.max_tokens <= 4 * kCluster * kPlanThreads) return run<1, false>(a, kCluster, stream);
  // a cooperative grid has to be resident at once: a CTA per SM of this device
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? run<4, true>(a, sms, stream) : e;
}

}  // namespace sparge
