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
// One cluster of CTAs does it in one launch.  Every CTA takes the prefix sums
// over all requests for itself (they are in L2 after the first), all inputs
// that may be outputs too are read before the first cluster barrier and
// written behind it, and the pages pushed by the first CTA are read by the
// others behind the second.
#include <cooperative_groups.h>

#include <cstdint>

#include "sparge_internal.h"

namespace sparge {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanPer = 4;  // requests per thread
constexpr int kPlanMax = kPlanThreads * kPlanPer;
static_assert(kPlanMax == kMaxPlanRequests, "every request has a thread");

// Exclusive prefix sum of one value per thread; *total gets the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* sh, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  __syncthreads();  // sh may still be read from the last scan
  if (lane == 31) sh[w] = incl;
  __syncthreads();
  if (w == 0) {
    int64_t s = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += up;
    }
    sh[lane] = s;
  }
  __syncthreads();
  *total = sh[31];
  return (w > 0 ? sh[w - 1] : 0) + incl - v;
}

__global__ void __launch_bounds__(kPlanThreads, 1) plan_kernel(const KvPlanArgs A) {
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = int(cluster.block_rank()), ctas = int(cluster.num_blocks());
  __shared__ int64_t sh[32];
  extern __shared__ int32_t s_dyn[];
  int32_t* s_cu = s_dyn;             // [R + 1] start of each request's tokens
  int32_t* s_len = s_cu + A.R + 1;   // [R] L; -1: no tokens or not admitted; -2 - L: ended
  int32_t* s_off = s_len + A.R;      // [R] pages pushed (ended) or popped before it

  const int32_t P = A.page_size;
  const int64_t cap = int64_t(A.max_pages) * P;
  int64_t count = *A.free_count;
  count = count < 0 ? 0 : (count > A.num_pages ? A.num_pages : count);

  // ---- lengths, what comes back, where tokens start
  int32_t L[kPlanPer], n[kPlanPer];
  int64_t add = 0, back = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int r = threadIdx.x * kPlanPer + i;
    L[i] = n[i] = 0;
    if (r < A.R) {
      const int64_t l = A.seq_len[r];
      L[i] = int32_t(l < 0 ? 0 : (l > cap ? cap : l));
      n[i] = A.new_len[r];
    }
    if (n[i] > 0) add += n[i];
    if (n[i] < 0) back += (L[i] + int64_t(P) - 1) / P;
  }
  int64_t tokens, pushed;
  int64_t cu = block_scan(add, sh, &tokens);
  int64_t put = block_scan(back, sh, &pushed);
  int64_t avail = count + pushed;
  if (avail > A.num_pages) avail = A.num_pages;

  // ---- pages needed, admission
  int64_t at = cu, need = 0;
  int32_t want[kPlanPer];
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int64_t after = int64_t(L[i]) + n[i];
    want[i] = -1;  // does not fit (or brings nothing)
    if (n[i] > 0) {
      at += n[i];
      if (after <= cap && at <= A.max_tokens)
        want[i] = int32_t((after + P - 1) / P - (int64_t(L[i]) + P - 1) / P);
    }
    if (want[i] > 0) need += want[i];
  }
  int64_t all;
  int64_t upto = block_scan(need, sh, &all);
  int64_t taken = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int r = threadIdx.x * kPlanPer + i;
    if (r >= A.R) break;
    const int64_t before = upto;
    if (want[i] > 0) upto += want[i];
    const bool ok = want[i] == 0 || (want[i] > 0 && upto <= avail);
    if (ok) taken += want[i];
    s_cu[r] = int32_t(cu > INT32_MAX ? INT32_MAX : cu);
    s_len[r] = ok ? L[i] : -1;
    const int64_t off = n[i] < 0 ? put : before;
    s_off[r] = int32_t(off > INT32_MAX ? INT32_MAX : off);
    if (n[i] > 0) cu += n[i];
    if (n[i] < 0) {
      s_len[r] = -2 - L[i];  // ended
      put += (L[i] + int64_t(P) - 1) / P;
    }
  }
  if (threadIdx.x == 0) s_cu[A.R] = int32_t(tokens > INT32_MAX ? INT32_MAX : tokens);
  int64_t popped;
  block_scan(taken, sh, &popped);

  cluster.sync();  // every CTA has read what the first one now overwrites
  if (rank == 0) {
#pragma unroll
    for (int i = 0; i < kPlanPer; ++i) {
      const int r = threadIdx.x * kPlanPer + i;
      if (r >= A.R) break;
      const bool ok = s_len[r] >= 0;
      A.seq_len_out[r] = n[i] < 0 ? 0 : (ok ? L[i] + n[i] : L[i]);
      A.admitted[r] = ok || n[i] <= 0;
      A.cu_new[r] = s_cu[r];
    }
    if (threadIdx.x == 0) {
      A.cu_new[A.R] = s_cu[A.R];
      *A.free_count_out = int32_t(avail - popped);
    }
    // pages of ended requests, a warp per request
    const int lane = threadIdx.x & 31;
    for (int r = threadIdx.x >> 5; r < A.R; r += kPlanThreads / 32) {
      if (s_len[r] > -2) continue;
      const int pages = int((int64_t(-2 - s_len[r]) + P - 1) / P);
      for (int j = lane; j < pages; j += 32) {
        const int64_t to = count + s_off[r] + j;
        if (to < A.num_pages) A.free_pages[to] = A.block_table[int64_t(r) * A.max_pages + j];
      }
    }
  }
  cluster.sync();  // the pushed pages are there

  // ---- slots: one token per thread and step; the first token of a new page
  // writes its table entry
  const int32_t end = s_cu[A.R];
  for (int64_t t = int64_t(rank) * kPlanThreads + threadIdx.x; t < A.max_tokens;
       t += int64_t(ctas) * kPlanThreads) {
    int32_t slot = -1;
    if (t < end) {
      int lo = 0, hi = A.R;  // the last request that starts at or before t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid;
      }
      const int32_t len = s_len[lo];
      if (len >= 0) {
        const int64_t pos = int64_t(len) + (t - s_cu[lo]);
        const int32_t page = int32_t(pos / P), in = int32_t(pos - int64_t(page) * P);
        const int32_t have = int32_t((int64_t(len) + P - 1) / P);
        int32_t* entry = A.block_table + int64_t(lo) * A.max_pages + page;
        int32_t id;
        if (page < have) {
          id = *entry;
        } else {
          id = A.free_pages[avail - 1 - s_off[lo] - (page - have)];
          if (in == 0) *entry = id;
        }
        slot = int32_t(int64_t(id) * P + in);
      }
    }
    A.slot_map[t] = slot;
  }
}

}  // namespace

cudaError_t launch_kv_plan(const KvPlanArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  // up to eight CTAs (a portable cluster), one per 4096 tokens
  const int64_t ctas = cdiv(a.max_tokens, 4 * kPlanThreads);
  int n = 1;
  while (n < 8 && n < ctas) n <<= 1;
  cfg.gridDim = dim3(unsigned(n));
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = (3 * size_t(a.R) + 1) * sizeof(int32_t);
  if (cfg.dynamicSmemBytes > 46 * 1024) {  // 48 KB with the static part need no permission
    const cudaError_t e =
        cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int((3 * kPlanMax + 1) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
  }
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(n);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, plan_kernel, a);
}

}  // namespace sparge
