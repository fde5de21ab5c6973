// kvq_page_plan.cu -- block tables and slot maps of a serving step, built on the GPU from
// the requests' lengths, and the return of finished requests' pages.
//
// For request b with kv cached and q new tokens and pages of P tokens,
//   have = ceil(kv / P), want = ceil((kv + q) / P), need = want - have (0 when want does
//   not fit the table), upto = inclusive prefix sum of need,
//   served = want fits, kv + q <= 2^31 - 1 and (need == 0 or upto <= free entries left),
// the pages of a served request come from the free list at upto - need, and token j goes to
// position kv + j, slot = page * P + position % P. Integers only; every output is a
// function of the inputs alone (no atomics), so two calls on the same inputs agree.
//
// The work is a few hundred KB at most, so the time is latency: every CTA scans all requests
// itself (B <= 16384: a block scan of at most 16 requests per thread) into its shared memory,
// and the CTAs share the table entries and the tokens (one per thread,
// the owning request by binary search over the starts in shared memory). Lengths and the
// free-list head may be updated in place: a CTA must not overwrite what another has yet to
// read, so with more than one CTA they are then written by a second launch of one CTA. 2048
// requests with 190 thousand tokens: 39.8 us a pass with one cluster of 8 CTAs and a cluster
// barrier in place of the second launch, 8.8 us with a CTA per 2048 tokens.
#include <algorithm>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanSmall = 256;       // threads of a CTA for steps of up to 256 requests and 1024 tokens (32 requests: 4.15 -> 3.75 us)
constexpr int kPlanPerCta = 2048;     // tokens or requests per CTA before another joins

struct PagePlanParams {
  const int32_t* kv_lens;
  const int32_t* q_lens;
  int32_t* table;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t* free_head_out;
  int32_t* slots;
  int32_t* positions;
  int32_t* q_starts;
  int32_t* kv_out;
  int32_t* info;
  long long table_stride;
  int B, max_pages, n_free, page_shift, n_slots;
  bool fill, move;  // write tables, slots, starts and info; write lengths and the head
};

__device__ __forceinline__ int32_t sat32(long long v) { return v > 0x7fffffffll ? 0x7fffffff : (int32_t)v; }

// Whether a request of kv + q tokens fits its table row, and its length 32 bits.
__device__ __forceinline__ bool fits_table(const PagePlanParams& p, long long kv, long long q) {
  return kv + q <= min((long long)p.max_pages << p.page_shift, 0x7fffffffll);
}

// Inclusive prefix sum of v over the block of NT threads; total in *sum. `part` holds 32 values.
template <int NT>
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  __syncthreads();  // `part` may still be read by the scan before this one
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    long long w = lane < NT / 32 ? part[lane] : 0;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += u;
    }
    part[lane] = w;
  }
  __syncthreads();
  *sum = part[31];
  return v + (warp ? part[warp - 1] : 0);
}

template <int NT>
__global__ void __launch_bounds__(NT) page_plan_kernel(const __grid_constant__ PagePlanParams p) {
  // [B] start (its low 32 bits), [B] first entry of the free list (-1: refused), [B] cached tokens
  extern __shared__ int32_t s_req[];
  __shared__ long long part[32];
  __shared__ long long served_pages;
  __shared__ int refused, past;  // past: the first request whose start is above 2^31 - 1
  int32_t* s_start = s_req;
  int32_t* s_first = s_req + p.B;
  int32_t* s_kv = s_req + 2 * p.B;
  const int tid = threadIdx.x;
  const int P = 1 << p.page_shift;
  if (tid == 0) {
    served_pages = 0;
    refused = 0;
    past = p.B;
  }
  grid_dep_launch();
  grid_dep_wait();
  const int32_t *kv_lens = behind_wait(p.kv_lens), *q_lens = behind_wait(p.q_lens), *free_pages = behind_wait(p.free_pages);
  const int32_t* table = behind_wait(p.table);
  const int head = min(max(ld_fresh(p.free_head), 0), p.n_free);
  const long long room = p.n_free - head;
  const int per = (p.B + NT - 1) / NT;
  const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  long long qs = 0, ns = 0;
  for (int b = b0; b < b1; ++b) {
    const long long kv = max(__ldcg(kv_lens + b), 0), q = max(__ldcg(q_lens + b), 0);
    const long long want = (kv + q + P - 1) >> p.page_shift;
    qs += q;
    ns += fits_table(p, kv, q) ? want - ((kv + P - 1) >> p.page_shift) : 0;
  }
  long long total, wanted;
  long long q_at = block_scan<NT>(qs, part, &total) - qs;
  long long n_at = block_scan<NT>(ns, part, &wanted) - ns;
  long long got = 0;
  int ref = 0;
  for (int b = b0; b < b1; ++b) {
    const long long kv = max(__ldcg(kv_lens + b), 0), q = max(__ldcg(q_lens + b), 0);
    const long long want = (kv + q + P - 1) >> p.page_shift;
    const bool fits = fits_table(p, kv, q);
    const long long need = fits ? want - ((kv + P - 1) >> p.page_shift) : 0;
    const bool served = fits && (need == 0 || n_at + need <= room);
    s_start[b] = (int32_t)(uint32_t)q_at;
    if (q_at > 0x7fffffffll) atomicMin(&past, b);
    s_first[b] = served ? (need ? head + (int)n_at : 0) : -1;
    s_kv[b] = (int32_t)kv;
    if (served) got += need;
    else ++ref;
    q_at += q;
    n_at += need;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    got += __shfl_xor_sync(0xffffffffu, got, off);
    ref += __shfl_xor_sync(0xffffffffu, ref, off);
  }
  if ((tid & 31) == 0) {
    if (got) atomicAdd(reinterpret_cast<unsigned long long*>(&served_pages), (unsigned long long)got);
    if (ref) atomicAdd(&refused, ref);
  }
  __syncthreads();
  const int nthreads = (int)gridDim.x * NT, gt = (int)blockIdx.x * NT + tid;
  if (gt == 0 && p.move) p.free_head_out[0] = head + (int)served_pages;
  if (gt == 0 && p.fill) {
    p.q_starts[p.B] = sat32(total);
    p.info[0] = sat32(total);
    p.info[1] = (int)served_pages;
    p.info[2] = refused;
    p.info[3] = sat32(wanted);
  }
  // starts and lengths; the new tokens of b are the difference of two starts, exact from their
  // low 32 bits however large the sums are
  const int first_past = past;
  auto q_of = [&](int b) {
    return (long long)((b + 1 < p.B ? (uint32_t)s_start[b + 1] : (uint32_t)total) - (uint32_t)s_start[b]);
  };
  for (int b = gt; b < p.B; b += nthreads) {
    if (p.fill) p.q_starts[b] = b < first_past ? s_start[b] : 0x7fffffff;
    if (p.move) p.kv_out[b] = s_first[b] >= 0 ? (int32_t)(s_kv[b] + q_of(b)) : s_kv[b];
  }
  if (!p.fill) return;
  // New table entries. With a warp for every request (many tokens, so many CTAs): a warp each.
  // Else a lane per request writes the first few (a decode step's at most one), the warp
  // together what is left of those with more. (200 requests in one CTA: 6.6 us with warps, 4.2
  // with lanes; 2048 requests with 190 thousand tokens in 103 CTAs: 8.8 and 11.4.)
  constexpr int kFirst = 4;
  const int lane = tid & 31;
  if (nthreads / 32 >= p.B) {
    const int b = gt >> 5;
    if (b < p.B && s_first[b] >= 0) {
      const long long kv = s_kv[b];
      const int first = s_first[b], have = (int)((kv + P - 1) >> p.page_shift);
      const int want = (int)((kv + q_of(b) + P - 1) >> p.page_shift);
      for (int e = have + lane; e < want; e += 32)
        p.table[(long long)b * p.table_stride + e] = free_pages[first + e - have];
    }
  } else for (int b0 = (gt >> 5) * 32; b0 < p.B; b0 += nthreads) {
    const int b = b0 + lane;
    int first = -1, have = 0, want = 0;
    if (b < p.B && s_first[b] >= 0) {
      const long long kv = s_kv[b];
      first = s_first[b];
      have = (int)((kv + P - 1) >> p.page_shift);
      want = (int)((kv + q_of(b) + P - 1) >> p.page_shift);
    }
    for (int e = have; e < min(want, have + kFirst); ++e)
      p.table[(long long)b * p.table_stride + e] = free_pages[first + e - have];
    uint32_t more = __ballot_sync(0xffffffffu, want - have > kFirst);
    while (more) {
      const int l = __ffs(more) - 1;
      more &= more - 1;
      const int f = __shfl_sync(0xffffffffu, first, l), h = __shfl_sync(0xffffffffu, have, l), w = __shfl_sync(0xffffffffu, want, l);
      for (int e = h + kFirst + lane; e < w; e += 32)
        p.table[(long long)(b0 + l) * p.table_stride + e] = free_pages[f + e - h];
    }
  }
  // slots and positions; behind the last token both are -1. Four tokens of a thread at a time, so
  // that their loads overlap: 190 thousand tokens 8.4 us a pass, 12.5 one by one (when, at 32
  // registers a thread, two passes' CTAs also share an SM)
  constexpr int U = NT == kPlanThreads ? 4 : 1;
  for (long long t0 = gt; t0 < p.n_slots; t0 += (long long)U * nthreads) {
    const int32_t* entry[U];
    int slot[U], pos[U], page[U], place[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long t = t0 + (long long)u * nthreads;
      entry[u] = nullptr;
      slot[u] = pos[u] = -1;
      if (t >= min(total, (long long)p.n_slots) || p.B == 0) continue;
      int lo = 0, hi = first_past;  // last request whose start is <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_start[mid] <= t) lo = mid;
        else hi = mid;
      }
      const long long kv = s_kv[lo], at = kv + (t - s_start[lo]);
      pos[u] = sat32(at);
      const int first = s_first[lo];
      if (first < 0) continue;
      const int blk = (int)(at >> p.page_shift), have = (int)((kv + P - 1) >> p.page_shift);
      place[u] = (int)(at & (P - 1));
      entry[u] = blk < have ? table + (long long)lo * p.table_stride + blk : free_pages + first + blk - have;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (entry[u]) page[u] = ld_fresh(entry[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // a page whose slots would not fit 32 bits is no page of a cache
      if (entry[u] && page[u] >= 0 && page[u] <= (0x7fffffff >> p.page_shift)) slot[u] = page[u] * P + place[u];
      const long long t = t0 + (long long)u * nthreads;
      if (t < p.n_slots) {
        p.slots[t] = slot[u];
        p.positions[t] = pos[u];
      }
    }
  }
}

// Finished requests: the pages of every marked row go back in front of the free list's
// head, in row order, and the row's length becomes 0. One CTA: a release is rare and small.
__global__ void __launch_bounds__(kPlanThreads) page_release_kernel(const uint8_t* done, int32_t* kv_lens,
                                                                    const int32_t* table, long long table_stride,
                                                                    int B, int max_pages, int page_shift,
                                                                    int32_t* free_pages, int n_free,
                                                                    int32_t* free_head) {
  __shared__ long long part[32];
  const int tid = threadIdx.x, P = 1 << page_shift;
  grid_dep_launch();
  grid_dep_wait();
  const int head = min(max(ld_fresh(free_head), 0), n_free);
  long long before = 0;  // pages returned by earlier chunks
  for (int c0 = 0; c0 < B; c0 += kPlanThreads) {
    const int b = c0 + tid;
    const bool mine = b < B && done[b] != 0;
    const int n = mine ? (int)min(((long long)max(kv_lens[b], 0) + P - 1) >> page_shift, (long long)max_pages) : 0;
    long long sum;
    const long long at = before + block_scan<kPlanThreads>(n, part, &sum) - n;
    // entry i of the row goes to head - 1 - (at + i): never in front of the list's start
    for (int i = 0; i < n && at + i < head; ++i) free_pages[head - 1 - (at + i)] = table[b * table_stride + i];
    if (mine) kv_lens[b] = 0;
    before += sum;
  }
  __syncthreads();
  if (tid == 0) free_head[0] = head - (int)min(before, (long long)head);
}

}  // namespace

kvq_status launch_page_plan(const int32_t* kv_lens, const int32_t* q_lens, int B, int32_t* table, int max_pages,
                            long long table_stride, const int32_t* free_pages, int n_free, const int32_t* free_head,
                            int32_t* free_head_out, int page_shift, int32_t* slots, int32_t* positions, int n_slots,
                            int32_t* q_starts, int32_t* kv_out, int32_t* info, cudaStream_t s) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e == cudaSuccess) e = allow_smem<page_plan_kernel<kPlanThreads>>(device, kMaxPlanRequests * 12);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, std::string("page_plan: ") + cudaGetErrorString(e));
  PagePlanParams p{kv_lens,  q_lens, table, free_pages, free_head,  free_head_out, slots,   positions, q_starts,
                   kv_out,   info,   table_stride,  B,  max_pages,  n_free,        page_shift, n_slots, true, true};
  const int ctas = std::min(num_sms(device), std::max(1, (std::max(B, n_slots) + kPlanPerCta - 1) / kPlanPerCta));
  auto meet = [](const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
  };
  const size_t lens = (size_t)B * 4;
  const bool in_place = meet(kv_out, lens, kv_lens, lens) || meet(kv_out, lens, q_lens, lens) ||
                        meet(free_head_out, 4, free_head, 4);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  const bool small = B <= kPlanSmall && n_slots <= 4 * kPlanSmall;
  cfg.blockDim = dim3(small ? kPlanSmall : kPlanThreads);
  cfg.dynamicSmemBytes = (size_t)B * 12;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  p.move = ctas == 1 || !in_place;
  e = small ? cudaLaunchKernelEx(&cfg, page_plan_kernel<kPlanSmall>, p) : cudaLaunchKernelEx(&cfg, page_plan_kernel<kPlanThreads>, p);
  if (e == cudaSuccess && !p.move) {
    p.fill = false;
    p.move = true;
    cfg.gridDim = dim3(1);
    e = cudaLaunchKernelEx(&cfg, page_plan_kernel<kPlanThreads>, p);
  }
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, std::string("page_plan launch: ") + cudaGetErrorString(e));
  return KVQ_OK;
}

kvq_status launch_page_release(const uint8_t* done, int32_t* kv_lens, const int32_t* table, long long table_stride,
                               int B, int max_pages, int page_shift, int32_t* free_pages, int n_free,
                               int32_t* free_head, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, page_release_kernel, done, kv_lens, table, table_stride, B, max_pages,
                                           page_shift, free_pages, n_free, free_head);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, std::string("page_release launch: ") + cudaGetErrorString(e));
  return KVQ_OK;
}

}  // namespace kvq
