// Page tables, positions and slots of an append, and the return of finished
// sequences' pages, on the GPU (spectra_plan_append, spectra_release_pages).
//
// Both are prefix sums over the sequences (pages taken or given, tokens) and
// then independent writes; the bytes are few, so launch and load latency bound
// them.  One thread-block cluster of 1..8 CTAs per call: every CTA scans all
// sequences by itself (8 bytes each, from L2) and keeps the sums in shared
// memory, so that no sum crosses CTAs; the writes are spread over the cluster's
// warps, each thread finding its sequence by bisection in shared memory.  A cluster
// barrier after the scan stands between the last read of the stack's count and
// of the lengths and the first write to them.  Every CTA reaches the same verdict
// on the checks (same inputs), so a refused call writes nothing.
// Measured, one token for each of 1 / 16 / 256 / 1024 / 4096 sequences behind 16 shared
// pages: 3.7 / 3.8 / 4.8 / 6.8 / 12.6 us in a captured row of calls (launch, scan and a chain of
// three loads); 65536 tokens of 48 prompts 10.2 us.  With sums of 64 bits that every thread added over the
// warps by itself, and whole CTAs instead of warps dealt out, 1024 sequences took 2.9 us more and the
// prompts 1.9 us more.  Releasing 1024 sequences of 64 pages takes 10 us, 16 of 512 pages 14 us.
#include <cuda_runtime.h>

#include <algorithm>

#include "device_common.cuh"
#include "kernels.h"

namespace spectra {

namespace {

constexpr int kPlanThreads = 1024;  // of a CTA at most; a multiple of 32 as small as the call allows
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kMinPlan = 256;      // and at least
constexpr int kPages = 4;       // shared pages that a thread writes at a time

// Counts of tokens and pages.  Sums stay at kMost once they reach it (still associative),
// which the checks refuse.
struct Sums {
  uint32_t tok, pg;
};
constexpr uint32_t kMost = 0x7FFFFFFFu;

__device__ __forceinline__ Sums operator+(Sums a, Sums b) {
  return {min(a.tok + b.tok, kMost), min(a.pg + b.pg, kMost)};
}

// Sums over the lanes below this one, and this one's.
__device__ __forceinline__ Sums warp_scan(Sums v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums a{__shfl_up_sync(0xffffffffu, v.tok, o), __shfl_up_sync(0xffffffffu, v.pg, o)};
    if ((threadIdx.x & 31) >= o) v = v + a;
  }
  return v;
}

// Sums over the threads before this one, started at `carry`; carry: then with the whole CTA.
__device__ __forceinline__ Sums block_scan(Sums v, Sums* warp_s, Sums* carry) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
  const Sums in = warp_scan(v);
  if (lane == 31) warp_s[warp] = in;
  __syncthreads();
  const Sums w = warp_scan(lane < n_warps ? warp_s[lane] : Sums{0, 0});  // (every warp for itself)
  const Sums all{__shfl_sync(0xffffffffu, w.tok, 31), __shfl_sync(0xffffffffu, w.pg, 31)};
  Sums before{__shfl_sync(0xffffffffu, w.tok, (warp - 1) & 31), __shfl_sync(0xffffffffu, w.pg, (warp - 1) & 31)};
  if (warp == 0) before = {0, 0};
  Sums ex{__shfl_up_sync(0xffffffffu, in.tok, 1), __shfl_up_sync(0xffffffffu, in.pg, 1)};
  if (lane == 0) ex = {0, 0};
  __syncthreads();  // warp_s is free again
  const Sums out = *carry + before + ex;
  *carry = *carry + all;
  return out;
}

// Largest b in [0, n) with a[b] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a[m] <= x) lo = m;
    else hi = m;
  }
  return lo;
}

// This thread's number in the cluster: warps are counted across the CTAs, so that few
// items are spread over all SMs.
__device__ __forceinline__ int cluster_thread(int rank, int n_cta) {
  return ((threadIdx.x >> 5) * n_cta + rank) * 32 + (threadIdx.x & 31);
}

struct PlanArgs {
  const int32_t *lengths, *new_tokens, *prefix, *free_pages, *n_free;
  int32_t *n_free_out, *table, *seq_ids, *positions, *offsets, *err;
  int64_t* slots;
  int64_t max_tokens, free_capacity;
  int batch, n_prefix, max_pages, P;
  bool wide;  // the tokens' outputs take 16-byte stores
};

template <int kRun>  // tokens that a thread writes at a time
__global__ void __launch_bounds__(kPlanThreads) plan_append_kernel(const PlanArgs A) {
  extern __shared__ int plan_s[];  // offsets [batch + 1], first page taken [batch + 1]
  __shared__ Sums warp_s[kPlanWarps];
  int* off_s = plan_s;
  int* first_s = plan_s + A.batch + 1;
  const int tid = threadIdx.x, P = A.P, B = A.batch;
  const int rank = blockIdx.x, n_cta = gridDim.x;
  pdl_wait();
  const int n_free = *A.n_free;
  Sums carry{0, 0};
  int bad = 0;  // 1: invalid, 2: capacity
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    const int b = b0 + tid;
    Sums v{0, 0};
    if (b < B) {
      const int len = A.lengths[b], nw = A.new_tokens[b];
      const long long pre = (long long)A.n_prefix * P;
      if (len < 0 || nw < 0 || (len > 0 && len < pre) || (len == 0 && nw > 0 && pre > 0)) {
        bad |= 1;
      } else {
        const long long have = (len + (long long)P - 1) / P, need = ((long long)len + nw + P - 1) / P;
        if (need > A.max_pages || (long long)len + nw > 0x7FFFFFFFll) bad |= 2;
        v.tok = (uint32_t)nw;
        v.pg = (uint32_t)(need - have);
      }
    }
    const Sums at = block_scan(v, warp_s, &carry);
    if (b < B) {
      off_s[b] = (int)at.tok;
      first_s[b] = (int)at.pg;
    }
  }
  if (n_free > A.free_capacity) bad |= 1;  // (its top lies outside the array)
  if (carry.tok > A.max_tokens || n_free < 0 || carry.pg == kMost || carry.pg > (uint32_t)n_free) bad |= 2;
  if (tid == 0) {
    off_s[B] = (int)carry.tok;
    first_s[B] = (int)carry.pg;
  }
  const int any_invalid = __syncthreads_or(bad & 1), any_full = __syncthreads_or(bad & 2);
  cluster_sync_all();  // every CTA has read the stack's count
  if (any_invalid || any_full) {
    if (rank == 0 && tid == 0) device_error(A.err, any_invalid ? SPECTRA_ERR_INVALID : SPECTRA_ERR_CAPACITY);
    return;
  }
  const int n_tok = (int)carry.tok, n_pg = (int)carry.pg;
  const int gt = cluster_thread(rank, n_cta), gn = n_cta * blockDim.x;
  if (gt == 0) *A.n_free_out = n_free - n_pg;
  for (int b = gt; b <= B; b += gn) A.offsets[b] = off_s[b];
  // new pages: the i-th taken is the stack's (n_free - 1 - i)-th
  for (int i = gt; i < n_pg; i += gn) {
    const int b = last_not_above(first_s, B, i);
    const int have = (int)(((long long)A.lengths[b] + P - 1) / P);
    A.table[(size_t)b * A.max_pages + have + (i - first_s[b])] = A.free_pages[n_free - 1 - i];
  }
  // shared pages of every sequence in use
  const int n_runs = (A.n_prefix + kPages - 1) / kPages;
  for (int64_t e = gt; e < (int64_t)B * n_runs; e += gn) {
    const int b = (int)(e / n_runs), k0 = (int)(e - (int64_t)b * n_runs) * kPages;
    int pg[kPages];
#pragma unroll
    for (int u = 0; u < kPages; ++u) pg[u] = A.prefix[min(k0 + u, A.n_prefix - 1)];
    if (A.lengths[b] > 0) {
#pragma unroll
      for (int u = 0; u < kPages; ++u)
        if (k0 + u < A.n_prefix) A.table[(size_t)b * A.max_pages + k0 + u] = pg[u];
    }
  }
  // tokens: a run of them lies in one sequence and one page but for its ends
  for (int64_t i0 = (int64_t)gt * kRun; i0 < A.max_tokens; i0 += (int64_t)gn * kRun) {
    int seq = -1, end = 0, pos = 0, r = 0, k = 0, have = 0, pg = 0;
    int seqs[kRun], poss[kRun];
    int64_t slot[kRun];
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      const int i = (int)i0 + u;
      seqs[u] = poss[u] = -1;
      slot[u] = -1;
      if (i >= n_tok) continue;
      bool page = false;
      if (seq < 0 || i >= end) {
        // the last sequence that starts at or before i has tokens: a sequence
        // without tokens shares its offset with the next one
        seq = last_not_above(off_s, B, i);
        end = off_s[seq + 1];
        const int len = A.lengths[seq];
        pos = len + i - off_s[seq];
        k = pos / P;
        r = pos - k * P;
        have = (int)(((long long)len + P - 1) / P);
        page = true;
      } else {
        ++pos;
        if (++r == P) {
          r = 0;
          ++k;
          page = true;
        }
      }
      if (page && A.slots)
        pg = k >= have ? A.free_pages[n_free - 1 - (first_s[seq] + k - have)]
                       : A.table[(size_t)seq * A.max_pages + k];
      seqs[u] = seq;
      poss[u] = pos;
      slot[u] = (int64_t)pg * P + r;
    }
    if (kRun == 4 && A.wide && i0 + kRun <= A.max_tokens) {
      *reinterpret_cast<int4*>(A.seq_ids + i0) = make_int4(seqs[0], seqs[1 % kRun], seqs[2 % kRun], seqs[3 % kRun]);
      if (A.positions) *reinterpret_cast<int4*>(A.positions + i0) = make_int4(poss[0], poss[1 % kRun], poss[2 % kRun], poss[3 % kRun]);
      if (A.slots) {
        longlong2* p = reinterpret_cast<longlong2*>(A.slots + i0);
        p[0] = make_longlong2(slot[0], slot[1 % kRun]);
        p[1] = make_longlong2(slot[2 % kRun], slot[3 % kRun]);
      }
      continue;
    }
#pragma unroll
    for (int u = 0; u < kRun; ++u) {
      if (i0 + u >= A.max_tokens) break;
      A.seq_ids[i0 + u] = seqs[u];
      if (A.positions) A.positions[i0 + u] = poss[u];
      if (A.slots) A.slots[i0 + u] = slot[u];
    }
  }
}

struct ReleaseArgs {
  const int32_t *finished, *table;
  int32_t *lengths, *free_pages, *n_free, *err;
  int64_t capacity;
  int batch, n_prefix, max_pages, P;
};

__global__ void __launch_bounds__(kPlanThreads) release_pages_kernel(const ReleaseArgs A) {
  extern __shared__ int plan_s[];  // first page given [batch + 1]
  __shared__ Sums warp_s[kPlanWarps];
  int* first_s = plan_s;
  const int tid = threadIdx.x, P = A.P, B = A.batch;
  const int rank = blockIdx.x, n_cta = gridDim.x;
  pdl_wait();
  const int n_free = *A.n_free;
  Sums carry{0, 0};
  int bad = 0;
  for (int b0 = 0; b0 < B; b0 += blockDim.x) {
    const int b = b0 + tid;
    Sums v{0, 0};
    if (b < B && A.finished[b]) {
      const int len = A.lengths[b];
      const long long pre = (long long)A.n_prefix * P;
      if (len < 0 || (len > 0 && len < pre) || len > (long long)A.max_pages * P) bad = 1;
      else if (len > 0) v.pg = (uint32_t)(((long long)len + P - 1) / P - A.n_prefix);
    }
    const Sums at = block_scan(v, warp_s, &carry);
    if (b < B) first_s[b] = (int)at.pg;
  }
  if (tid == 0) first_s[B] = (int)carry.pg;
  const bool full = n_free < 0 || carry.pg == kMost || (int64_t)n_free + carry.pg > A.capacity;
  const int any_invalid = __syncthreads_or(bad);
  cluster_sync_all();  // every CTA has read the lengths and the stack's count
  if (any_invalid || full) {
    if (rank == 0 && tid == 0) device_error(A.err, any_invalid ? SPECTRA_ERR_INVALID : SPECTRA_ERR_CAPACITY);
    return;
  }
  const int n_pg = (int)carry.pg;
  const int gt = cluster_thread(rank, n_cta), gn = n_cta * blockDim.x;
  if (gt == 0) *A.n_free = n_free + n_pg;
  for (int i = gt; i < n_pg; i += gn) {
    const int b = last_not_above(first_s, B, i);
    A.free_pages[n_free + i] = A.table[(size_t)b * A.max_pages + A.n_prefix + (i - first_s[b])];
  }
  for (int b = gt; b < B; b += gn)
    if (A.finished[b]) A.lengths[b] = 0;
}

// One cluster of 1..8 CTAs: a thread for each item up to the cluster's most, and for each
// sequence of the scan up to a CTA's most.  Plain stream order on both sides (what
// follows may read the table and the lengths before its own dependency wait).
template <typename Args>
cudaError_t launch_plan(void (*kern)(const Args), const Args& a, int batch, int64_t items, int smem, cudaStream_t st) {
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  int ctas = 1;
  while (ctas < 8 && items > (int64_t)ctas * kMinPlan) ctas *= 2;
  int threads = kMinPlan;
  while (threads < kPlanThreads && (items > (int64_t)ctas * threads || batch > threads)) threads *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

cudaError_t launch_plan_append(int P, int32_t* err, int batch, const int32_t* lengths, const int32_t* new_tokens,
                               const int32_t* prefix, int n_prefix, const int32_t* free_pages, int64_t free_capacity,
                               const int32_t* n_free, int32_t* n_free_out, int32_t* table, int max_pages, int64_t max_tokens,
                               int32_t* seq_ids, int32_t* positions, int64_t* slots, int32_t* offsets,
                               cudaStream_t st) {
  const PlanArgs a{lengths, new_tokens, prefix,  free_pages, n_free, n_free_out, table, seq_ids, positions,
                   offsets, err,        slots,   max_tokens, free_capacity, batch, n_prefix, max_pages, P,
                   ((reinterpret_cast<uintptr_t>(seq_ids) | reinterpret_cast<uintptr_t>(positions) |
                     reinterpret_cast<uintptr_t>(slots)) & 15) == 0};
  // runs of four tokens only where there are more than threads: a run that spans sequences
  // (decode steps) walks from one to the next
  const int run = max_tokens > 8 * kPlanThreads ? 4 : 1;
  const int64_t items = std::max<int64_t>((max_tokens + run - 1) / run, (int64_t)batch * ((n_prefix + kPages - 1) / kPages));
  return launch_plan(run == 4 ? plan_append_kernel<4> : plan_append_kernel<1>, a, batch, items, 2 * (batch + 1) * 4, st);
}

cudaError_t launch_release_pages(int P, int32_t* err, int batch, const int32_t* finished, int32_t* lengths,
                                 int n_prefix, const int32_t* table, int max_pages, int32_t* free_pages,
                                 int64_t capacity, int32_t* n_free, cudaStream_t st) {
  const ReleaseArgs a{finished, table, lengths, free_pages, n_free, err, capacity, batch, n_prefix, max_pages, P};
  return launch_plan(release_pages_kernel, a, batch, (int64_t)batch * 16, (batch + 1) * 4, st);
}

}  // namespace spectra
