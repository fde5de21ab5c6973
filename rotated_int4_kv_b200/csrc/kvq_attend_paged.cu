// kvq_attend_paged.cu -- attention of few query tokens per request over a paged int4/int8
// cache for sm_100a, in the rotated domain (the paper describes no read path; it follows
// from the transform being orthonormal, as in the dense decode attention):
//   q~ = Lambda_K^-1 Q diag(s_K) q,   score_t = sigma q~ . (c_K scale_K)_t,
//   o = sum_t softmax(score)_t (c_V scale_V)_t,   out = diag(s_V) Q^T Lambda_V^-1 o.
//
// Work. A unit is (request, KV head, tile of 8 query rows), a query row one (query token,
// head of the KV head's group). Three kernels, each started early by the one in front:
//   rotate  a block per unit prepares its queries (q~ as product fragments);
//   attend  the tiles of all units (128 tokens; 64 where rows are longer) form one line,
//           requests after requests, and every CTA of a persistent grid takes an equal piece
//           of it, however ragged the lengths are: the end of one unit, some whole units, the
//           beginning of another. The lengths live on the GPU, so every CTA adds them up for
//           itself (one block scan). It leaves a partial (m, l, o) per piece of a unit;
//   join    a block per unit adds its partials in CTA order and un-rotates the output.
// One kernel that rotated, merged (last arrival at a counter) and un-rotated inside the
// pieces took 24 us beside the loads instead of 16: 64 ragged requests 88 -> 66 us, 4 x 128K
// tokens 137 -> 125 us, one request of 700 tokens 13.0 -> 11.5 us.
//
// A CTA of attend is one producer warp and four consumer warps; at 128 registers, for three CTAs
// per SM, every form spills some (52 to 180 bytes a thread). The producer streams a tile's
// pages into a ring of stages: per page one TMA box of K codes and one of V codes (swizzled for
// ldmatrix), and the scale rows as plain bulk copies. Consumer warp w takes the w-th quarter of
// a tile's tokens, all channels, and keeps its own softmax state and output; the warps are
// joined when a unit ends, while the producer already loads the next unit's tiles.
//
// Products are mma.m16n8k16 with tokens (scores) or channels (output) as rows and the 8
// query rows as columns. At 4.9 TB/s per further token (75 % of the copy rate) the loop is
// bound by instruction issue and latency (about 280 instructions per 16 tokens of 128
// channels, 130 of them on the integer pipe, 47 % issue), not by HBM (the same with the cache
// in L2) nor by the tensor cores (32 %).
//   * A code enters as a fp16 subnormal (code + 8) 2^-24 (int4: nibble + 8 in the low bits of
//     an fp16 word, or 16 times that in the next four): one logical operation per pair. The
//     offset is taken out by the accumulators' start in the scores and by a product with a
//     constant in the output, the powers of two by the query's fragments and at the end.
//   * The rotation's entries are fp16, one rounding each (none for the SRHT), and q~ is one fp16
//     rounding per element after a power-of-two normalisation per row: 2^-12 relative each on
//     average, so a score's error is about 2^-12 of |q||k|/sqrt(D), as much as the fp16 rounding
//     of the caller's q has put there already. hi + lo pairs would double the score products (8
//     of 24 per 16 tokens) and the 32 or 128 KB of matrix per unit. The output's rotation takes o
//     as hi + lo: a few products more per unit, beside latencies that hide them.
//   * P is fp16 (its sum l is in fp32 of the unrounded values), raised to the top of fp16's
//     range: the largest weight is 2^15, or as much less as V scales from 1 on ask for so that
//     its product with them (one more rounding) stays within fp16 too. A running maximum's
//     headroom takes 2^3 of that at most. Weights down to 2^-26 of the largest so have one
//     rounding of 2^-12 on average (V scales below 1; with scales from 2^15 on: down to 2^-10),
//     smaller ones an error of at most 2^-37 (2^-21) of the largest; a weight times its scale
//     is off by as much again, of the largest weight times a scale of 1 (2^16).
#include <algorithm>
#include <cmath>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

__device__ uint32_t g_paged_err = 0;

namespace {

constexpr int kRows = 8;        // query rows per unit (mma N)
constexpr int kWarps = 4;       // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMaxCtas = 3 * 160;  // partial slots in the workspace: two per CTA

// Warps of a block of the first and the last kernel. At D = 256 a warp per 16 rows of the
// matrix halves the time of a block (drafts on 16K caches 24.9 -> 21.2 us); at D = 128 four
// warps with two such tiles each are better where there are many blocks (64.6 against 68.1 us
// for 512 units).
template <int D>
constexpr int kUnitWarps = D == 128 ? 4 : 16;

template <int D, int G, int BITS>
struct PCfg {
  static constexpr int NC = D / 32;               // 32-channel chunks of a row
  static constexpr int NG = D / G;                // scale groups of a row
  static constexpr int RB = D * BITS / 8;         // code bytes of a row
  static constexpr int MT = D / 16;               // 16-channel tiles (output) and K steps (scores)
  static constexpr int kSub = (D == 128 && BITS == 4) ? 2 : 1;  // 16-token subtiles per warp and tile
  static constexpr int kTile = 16 * kWarps * kSub;         // tokens per tile
  static constexpr int kCtas = D == 128 ? 3 : 2;           // resident CTAs per SM
  static constexpr int kKBytes = kTile * RB;
  static constexpr int kSBytes = kTile * NG * 2;
  static constexpr int kStage = 2 * (kKBytes + kSBytes);
  static constexpr int kObuf = kWarps * (kWarps - 1) * (MT / kWarps) * 32 * 16;  // the warps' outputs, less each one's own quarter
  static constexpr int kOmStride = D + 4;                     // q~, fp32, padded rows
  static constexpr int kQn = BITS == 4 ? NG : NC;             // query fragments: 16 bytes per lane each
  static constexpr int kQf = kQn * 32 * 16;
  static constexpr int kBias = NG * 4 * 16;
  static constexpr int kPrep = kQf + kBias + kRows * 4;       // a unit's prepared query
  static constexpr int kMl = kWarps * 2 * kRows * 4;
  static constexpr int kBars = 256;
  static constexpr int kFixed = kObuf + kPrep + kMl + kBars + 1024;
  static constexpr int kRoom = (kCtas == 3 ? 75 : 113) * 1024 - kFixed;
  static constexpr int kStages = kRoom / kStage < 4 ? kRoom / kStage : 4;
  static constexpr int kSmem = kStages * kStage + kFixed;
  static_assert(kStages >= 2, "shared memory");
  static constexpr int PART = 2 * kRows + kRows * D;          // a partial: m, l, o
};

struct PagedParams {
  CUtensorMap kmap, vmap;  // code pages [num_pages * Hkv][P][RB], box one page of <= 128 bytes a row
  const uint16_t* q;
  const uint16_t* ks;
  const uint16_t* vs;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  const uint4* wq;         // the rotation without signs and factors, as fragments
  const uint4* wo;
  const float* qchan;      // what its channels are multiplied by, K's and V's
  const float* ochan;
  const uint32_t* qsgn;    // sign masks of sample pairs, K's and V's
  const uint4* osgn;
  uint16_t* out;
  uint8_t* qprep;          // [unit] prepared queries
  float* part;             // [2 CTA + (0, 1)] partials of units that are cut
  float* part_unit;        // [unit] partials of whole units
  int2* desc;              // [unit] the first CTA's slot and the number of partials (0: whole)
  long long q_ts, q_hs, table_stride;
  float qfac;              // sigma log2(e)
  int B, n_q, Hq, Hkv, Gq, rt_max, max_q, max_kv, num_pages, page_shift, window, min_tiles;
  bool packed;             // units numbered by where the queries lie (see unit_base)
};

// ---------------------------------------------------------------- small helpers
__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 u2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127

// (a & mask) ^ c where c lies within mask
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t mask, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(mask), "r"(c));
  return d;
}

// Eight int4 codes of a word plus 8, as fp16 pairs: h0 = (n0, n4) 2^-24, h1 = (n1, n5) 2^-20,
// h2 = (n2, n6) 2^-24, h3 = (n3, n7) 2^-20 (subnormals, exact). x1 = 0x00080008 and
// x16 = 0x00800080 come in registers: an instruction holds one constant, the mask.
__device__ __forceinline__ void nib8_plus8(uint32_t w, uint32_t x1, uint32_t x16, uint32_t (&h)[4]) {
  const uint32_t w8 = w >> 8;
  h[0] = and_xor(w, 0x000F000Fu, x1);
  h[1] = and_xor(w, 0x00F000F0u, x16);
  h[2] = and_xor(w8, 0x000F000Fu, x1);
  h[3] = and_xor(w8, 0x00F000F0u, x16);
}
// Four int8 codes of a word plus 128: h0 = (b0, b2) 2^-24, h1 = (b1, b3) 2^-24.
__device__ __forceinline__ void byte4_plus128(uint32_t w, uint32_t (&h)[2]) {
  h[0] = and_xor(w, 0x00FF00FFu, 0x00800080u);
  h[1] = and_xor(w >> 8, 0x00FF00FFu, 0x00800080u);
}
__device__ __forceinline__ void byte4(uint32_t w, uint32_t (&h)[2]) {
  const __half2 o = u2h(0x00800080u);
  byte4_plus128(w, h);
  h[0] = h2u(__hsub2(u2h(h[0]), o));
  h[1] = h2u(__hsub2(u2h(h[1]), o));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

// The power of two 2^-e that brings a row's largest magnitude into [2^14, 2^15); mx is the
// largest of this lane's elements of row g, the row's lanes are c = 0 .. 3. Returns e.
__device__ __forceinline__ int row_exponent(float mx) {
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int e = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 14;
  return mx > 0.0f ? min(max(e, -100), 100) : 0;
}

// Byte offset of 16-byte column cc of token row `row` of a stage's codes: rows of up to 128
// bytes with the TMA swizzle of that width, longer rows as boxes of 128 bytes.
template <int RB, int kTile>
__device__ __forceinline__ int code_off(int row, int cc) {
  if constexpr (RB == 64) return row * 64 + ((cc ^ ((row >> 1) & 3)) << 4);
  return (cc >> 3) * (kTile * 128) + row * 128 + (((cc & 7) ^ (row & 7)) << 4);
}

// Loads from shared memory by 32-bit address (the loop below keeps no 64-bit pointers).
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t a, uint32_t (&v)[N]) {
  if constexpr (N == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[0]) : "r"(a) : "memory");
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(a) : "memory");
  } else {
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const uint4 u = lds128(a + 4 * k);
      v[k] = u.x;
      v[k + 1] = u.y;
      v[k + 2] = u.z;
      v[k + 3] = u.w;
    }
  }
}

// ---------------------------------------------------------------- the requests
struct Request {
  int qs, qn, kv;      // first query token, query tokens, cached tokens
  int t_lo;            // first token that any of its queries attends
  int tile0, nt, rt;   // first tile, tiles, row tiles
};

template <int kTile>
__device__ __forceinline__ Request request_of(const PagedParams& p, int b) {
  Request r;
  r.qs = b;
  r.qn = 1;
  if (p.q_starts) {
    r.qs = min(max(ld_fresh(p.q_starts + b), 0), p.n_q);
    r.qn = min(max(ld_fresh(p.q_starts + b + 1), r.qs), p.n_q) - r.qs;
  }
  r.kv = min(max(ld_fresh(p.kv_lens + b), 0), p.max_kv);
  const long long lo = p.window ? (long long)r.kv - r.qn + 1 - p.window : 0;
  r.t_lo = (int)min(max(lo, 0ll), (long long)r.kv);
  r.tile0 = r.t_lo / kTile;
  r.nt = max(1, (r.kv + kTile - 1) / kTile - r.tile0);
  r.rt = (min(r.qn, p.max_q) * p.Gq + kRows - 1) / kRows;
  return r;
}

// The numbers of units: (row tile of all requests, KV head). A request's row tiles start at
// b rt_max, rt_max being what the longest may have; or packed, where the bound on the longest is
// loose, at floor(first query row / 8) + b: at least ceil(rows / 8) further on for every request,
// as floor(x + y) + 1 >= floor(x) + ceil(y), and n_q Gq / 8 + B of them in all.
__device__ __forceinline__ int unit_base(const PagedParams& p, int b, int qs) {
  return p.packed ? qs * p.Gq / kRows + b : b * p.rt_max;
}

// The request and row tile of row tile x of all requests (rt < 0: none). Packed: the last request
// that starts at or in front of x, by a warp's 32 probes at a time.
__device__ __forceinline__ void request_at(const PagedParams& p, int x, int& b, int& rt) {
  if (!p.packed) {
    b = x / p.rt_max;
    rt = x - b * p.rt_max;
    return;
  }
  const int lane = threadIdx.x & 31;
  auto base = [&](int i) { return unit_base(p, i, min(max(ld_fresh(p.q_starts + i), 0), p.n_q)); };
  int lo = 0, n = p.B;
  while (n > 1) {
    const int step = (n + 31) / 32, i = lo + lane * step;
    const uint32_t at = __ballot_sync(0xffffffffu, lane * step < n && base(i) <= x);
    const int k = at ? 31 - __clz(at) : 0;
    lo += k * step;
    n = min(step, n - k * step);
  }
  b = lo;
  rt = x - base(lo);
}

__device__ __forceinline__ long long tiles_of(const PagedParams& p, const Request& r) {
  return (long long)p.Hkv * r.rt * r.nt;
}

// Inclusive prefix sum over the block's kThreads threads; total in *sum.
__device__ __forceinline__ long long block_scan(long long v, long long* part, long long* sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, off);
    if (lane >= off) v += u;
  }
  __syncthreads();
  if (lane == 31) part[warp] = v;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w <= kWarps; ++w) {
    if (w < warp) before += part[w];
    all += part[w];
  }
  *sum = all;
  return v + before;
}

// A CTA's piece [at, end) of the line of tiles, walked segment by segment (a segment: the
// tiles of one unit). `base` is the place of request b's first tile.
template <int kTile>
struct Walk {
  long long at, end, base;
  int b;
  Request r;
  // the segment: unit u of request b, its tiles [i0, i1)
  int u, i0, i1;

  __device__ __forceinline__ bool next(const PagedParams& p) {
    if (at >= end) return false;
    while (at >= base + tiles_of(p, r)) {
      base += tiles_of(p, r);
      r = request_of<kTile>(p, ++b);
    }
    const long long off = at - base;
    u = (int)(off / r.nt);
    i0 = (int)(off - (long long)u * r.nt);
    i1 = (int)min((long long)r.nt, i0 + (end - at));
    at += i1 - i0;
    return true;
  }
};

// ---------------------------------------------------------------- first kernel: the queries
// Block u: the 8 query rows of unit u, rotated (signs, a product with the rotation's fragments,
// factors) and laid out as the score products' B fragments
// (column = row of the tile), normalised by 2^-e per row, with per group the start of its sum
// (minus what the codes' offset adds to it) and per row the factor back to base-2 scores.
// A block reads the matrix (32 or 128 KB) through L2 before it waits for the kernel in front,
// Done here once per unit, not in every piece of it, and beside the main
// kernel's start.
template <int D, int G, int BITS>
__global__ void __launch_bounds__(kUnitWarps<D> * 32) rotate_paged_kernel(const __grid_constant__ PagedParams p) {
  using C = PCfg<D, G, BITS>;
  constexpr int NC = C::NC, MT = C::MT, NWARP = kUnitWarps<D>, TW = MT / NWARP;
  __shared__ __align__(16) float om[kRows * C::kOmStride];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int unit = blockIdx.x, x = unit / p.Hkv, h = unit - x * p.Hkv;
  uint4 wf[TW][MT];
#pragma unroll
  for (int t = 0; t < TW; ++t)
#pragma unroll
    for (int ks = 0; ks < MT; ++ks) wf[t][ks] = __ldg(p.wq + ((warp + NWARP * t) * MT + ks) * 32 + lane);
  float fac[TW][2];            // of channels g and g + 8 of the warp's tiles
  uint32_t sgn[MT][2];
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    fac[t][0] = __ldg(p.qchan + 16 * (warp + NWARP * t) + g);
    fac[t][1] = __ldg(p.qchan + 16 * (warp + NWARP * t) + g + 8);
  }
#pragma unroll
  for (int ks = 0; ks < MT; ++ks) {
    sgn[ks][0] = __ldg(p.qsgn + 8 * ks + c);
    sgn[ks][1] = __ldg(p.qsgn + 8 * ks + 4 + c);
  }
  grid_dep_wait();
  grid_dep_launch();  // after the wait: what the main kernel reads before its own wait is complete
  int b, rt;
  request_at(p, x, b, rt);
  const Request r = request_of<C::kTile>(p, b);
  const int nrows = min(kRows, min(r.qn, p.max_q) * p.Gq - rt * kRows);
  if (nrows <= 0 || rt < 0) return;
  uint32_t bq[MT][2];
  {
    const int y = rt * kRows + (g < nrows ? g : 0), tok = y / p.Gq, head = h * p.Gq + (y - tok * p.Gq);
    const uint16_t* src = p.q + (long long)(r.qs + tok) * p.q_ts + (long long)head * p.q_hs;
#pragma unroll
    for (int ks = 0; ks < MT; ++ks) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        bq[ks][e] = g < nrows ? ld_fresh(reinterpret_cast<const uint32_t*>(src + 16 * ks + 8 * e + 2 * c)) ^ sgn[ks][e] : 0u;
    }
  }
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    float a0[4] = {0.f, 0.f, 0.f, 0.f}, a1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < MT; ++ks)
      mma_16816((ks & 1) ? a1 : a0, wf[t][ks].x, wf[t][ks].y, wf[t][ks].z, wf[t][ks].w, bq[ks][0], bq[ks][1]);
    float* o0 = om + (2 * c) * C::kOmStride + 16 * (warp + NWARP * t) + g;
    o0[0] = (a0[0] + a1[0]) * fac[t][0];
    o0[C::kOmStride] = (a0[1] + a1[1]) * fac[t][0];
    o0[8] = (a0[2] + a1[2]) * fac[t][1];
    o0[C::kOmStride + 8] = (a0[3] + a1[3]) * fac[t][1];
  }
  __syncthreads();
  uint4* qf = reinterpret_cast<uint4*>(p.qprep + (size_t)unit * C::kPrep);
  float* bias = reinterpret_cast<float*>(qf) + C::kQf / 4;
  float* rowfac = bias + C::kBias / 4;
  const float* qr = om + g * C::kOmStride;
  // K step ks of the codes: int4 chunk ks / 2, channels 8c + (0, 4 | 1, 5) or (2, 6 | 3, 7);
  // int8 channels 16 ks + 4c + (0, 2 | 1, 3)
  auto chan = [&](int ks, int e) {
    if constexpr (BITS == 4) return 32 * (ks >> 1) + 8 * c + ((ks & 1) ? 2 : 0) + (e >> 1) + ((e & 1) ? 4 : 0);
    return 16 * ks + 4 * c + (e >> 1) + ((e & 1) ? 2 : 0);
  };
  float mx = 0.0f;
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    const float4 v = *reinterpret_cast<const float4*>(qr + 16 * k + 4 * c);
    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
  const int ex = row_exponent(mx);
  const float f = pow2f(-ex), fhi = BITS == 4 ? f * 0.0625f : f;  // the odd pairs' codes stand 16 times too high
  if (warp == 0 && c == 0) rowfac[g] = p.qfac * 16777216.0f * pow2f(ex);
  constexpr float kOff = (BITS == 4 ? 8.0f : 128.0f) / 16777216.0f;
  constexpr float kPair = BITS == 4 ? 16.0f : 1.0f;
  static_assert(NC <= NWARP, "a chunk per warp");
  if (warp < NC) {
    const int ch = warp;
    uint32_t h[4];
    float sum[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      h[2 * k] = pack_half2(qr[chan(2 * ch + k, 0)] * f, qr[chan(2 * ch + k, 1)] * f);
      h[2 * k + 1] = pack_half2(qr[chan(2 * ch + k, 2)] * fhi, qr[chan(2 * ch + k, 3)] * fhi);
      const float2 a = __half22float2(u2h(h[2 * k])), b = __half22float2(u2h(h[2 * k + 1]));
      sum[k] = -kOff * ((a.x + a.y) + kPair * (b.x + b.y));
    }
    auto start = [&](int grp, float v) {  // as both token rows of an accumulator of columns 2c', 2c' + 1
      float* d = bias + (grp * 4 + (g >> 1)) * 4 + (g & 1);
      d[0] = v;
      d[2] = v;
    };
    if constexpr (G == 32) {
      qf[ch * 32 + lane] = make_uint4(h[0], h[1], h[2], h[3]);
      float v = sum[0] + sum[1];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      v += __shfl_xor_sync(0xffffffffu, v, 2);
      if (c == 0) start(ch, v);
    } else if constexpr (BITS == 4) {  // lane c's channels lie in half c / 2 of the chunk
      const uint4 z = make_uint4(0, 0, 0, 0), q4 = make_uint4(h[0], h[1], h[2], h[3]);
      qf[(2 * ch) * 32 + lane] = c < 2 ? q4 : z;
      qf[(2 * ch + 1) * 32 + lane] = c < 2 ? z : q4;
      float v = sum[0] + sum[1];
      v += __shfl_xor_sync(0xffffffffu, v, 1);
      if ((c & 1) == 0) start(2 * ch + (c >> 1), v);
    } else {
      qf[ch * 32 + lane] = make_uint4(h[0], h[1], h[2], h[3]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v = sum[k];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (c == 0) start(2 * ch + k, v);
      }
    }
  }
}

// ---------------------------------------------------------------- the kernel
template <int D, int G, int BITS>
__global__ void __launch_bounds__(kThreads, (PCfg<D, G, BITS>::kCtas))
    attend_paged_kernel(const __grid_constant__ PagedParams p) {
  using C = PCfg<D, G, BITS>;
  constexpr int NC = C::NC, NG = C::NG, MT = C::MT, RB = C::RB, kTile = C::kTile;
  constexpr int KS = C::kSub, WT = 16 * KS;  // 16-token subtiles, and tokens, of a warp in a tile
  constexpr int TW = MT / kWarps;            // 16-row tiles per warp in the two rotations
  extern __shared__ uint8_t smem_raw[];
  // an offset, not a rounded pointer: the compiler then knows every access below as shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* ring = smem;
  float4* obuf = reinterpret_cast<float4*>(smem + C::kStages * C::kStage);
  uint4* qf = reinterpret_cast<uint4*>(smem + C::kStages * C::kStage + C::kObuf);  // the unit's prepared query: [fragment][lane],
  float* bias = reinterpret_cast<float*>(qf) + C::kQf / 4;                          // [group][c][4],
  float* rowf = bias + C::kBias / 4;                                                // [8]
  float* wml = rowf + kRows;                                                        // [warp][m, l][8]
  uint64_t* full = reinterpret_cast<uint64_t*>(wml + C::kMl / 4);
  uint64_t* empty = full + C::kStages;
  long long* scan = reinterpret_cast<long long*>(empty + C::kStages);  // [5]
  long long* found = scan + kWarps + 1;                                // base of the first request, its index
  uint4* consts = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(full) + C::kBars - 16);
  static_assert((2 * C::kStages + kWarps + 1 + 2) * 8 <= C::kBars - 24, "barrier region");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWarps);
    }
    fence_mbarrier_init();
    reinterpret_cast<uint32_t*>(consts)[-2] = 0x00080008u;
    reinterpret_cast<uint32_t*>(consts)[-1] = 0x00800080u;
    *consts = make_uint4(0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u);  // -8 2^-24 and -128 2^-24, rows g and g + 8
  }
  grid_dep_launch();
  // Only the prepared queries come from the kernel in front: it started this one when it had
  // itself waited for everything before it.

  // ---- this CTA's piece of the line of tiles
  long long total = 0, mine = 0, upto = 0;
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    mine = b0 + tid < p.B ? tiles_of(p, request_of<kTile>(p, b0 + tid)) : 0;
    long long sum;
    upto = total + block_scan(mine, scan, &sum);
    total += sum;
  }
  const long long per = max((long long)p.min_tiles, (total + gridDim.x - 1) / gridDim.x);
  Walk<kTile> w;
  w.at = min(total, per * blockIdx.x);
  w.end = min(total, w.at + per);
  if (w.at >= w.end) {
    grid_dep_wait();  // the kernel after this one counts on the one in front as well
    return;
  }
  if (p.B <= kThreads) {
    if (mine && w.at >= upto - mine && w.at < upto) {
      found[0] = upto - mine;
      found[1] = tid;
    }
  } else {
    long long before = 0;
    for (int b0 = 0; b0 < p.B && before <= w.at; b0 += kThreads) {
      mine = b0 + tid < p.B ? tiles_of(p, request_of<kTile>(p, b0 + tid)) : 0;
      long long sum;
      upto = before + block_scan(mine, scan, &sum);
      if (mine && w.at >= upto - mine && w.at < upto) {
        found[0] = upto - mine;
        found[1] = b0 + tid;
      }
      before += sum;
    }
  }
  __syncthreads();  // also publishes the barriers' initialisation
  w.base = found[0];
  w.b = (int)found[1];
  w.r = request_of<kTile>(p, w.b);

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    // a tile comes as boxes of min(P, kTile) tokens, at most 8: one lane each
    const int P = 1 << p.page_shift, bt = min(P, kTile), nb = kTile / bt;
    const uint32_t box = (uint32_t)(bt * (RB < 128 ? RB : 128));
    const uint32_t sbytes = (uint32_t)(bt * NG * 2);
    const uint32_t box_bytes = 2 * ((uint32_t)(bt * RB) + sbytes);
    const uint64_t pol = p.rt_max == 1 ? l2_evict_first_policy() : l2_normal_policy();
    int s = 0;               // the stage, and the phase of its barriers
    uint32_t phase = 0;
    bool first = true;       // the ring's first round: its stages are free
    while (w.next(p)) {
      const int h = w.u / w.r.rt;
      const int32_t* row = p.table + (long long)w.b * p.table_stride;
      auto entry = [&](int i) {  // the table entry for this lane's box of tile i; -1: nothing to load
        const long long t = (long long)(w.r.tile0 + i) * kTile + lane * bt;
        int e = -1;
        if (lane < nb && i < w.i1 && t < w.r.kv && t + bt > w.r.t_lo) {
          e = __ldg(row + (t >> p.page_shift));
          if (e < 0 || e >= p.num_pages) {
            atomicOr(&g_paged_err, kErrBadPage);
            e = 0;
          }
        }
        return e;
      };
      int page = entry(w.i0);
      for (int i = w.i0; i < w.i1; ++i) {
        const int coming = entry(i + 1);
        const bool ok = first || mbar_wait_bounded(&empty[s], phase ^ 1);
        if (!__all_sync(0xffffffffu, ok)) {
          if (lane == 0) atomicOr(&g_paged_err, kErrTimeoutLoad);
          return;
        }
        const uint32_t here = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) mbar_arrive_expect_tx(&full[s], (uint32_t)__popc(here) * box_bytes);
        __syncwarp();
        const int t0 = (w.r.tile0 + i) * kTile;
#pragma unroll 1
        for (int x = 0; x < nb; ++x) {
          if (!((here >> x) & 1)) continue;
          const int ph = __shfl_sync(0xffffffffu, page, x) * p.Hkv + h;
          if (elect_one()) {
            uint8_t* st = ring + s * C::kStage;
            const int off = (t0 + x * bt) & (P - 1);  // the box's first row of the page
#pragma unroll
            for (int j = 0; j < (RB + 127) / 128; ++j) {
              uint8_t* kd = st + j * (kTile * 128) + x * box;
              tma_load_3d_hint(kd, &p.kmap, &full[s], 128 * j, off, ph, pol);
              tma_load_3d_hint(kd + C::kKBytes, &p.vmap, &full[s], 128 * j, off, ph, pol);
            }
            uint8_t* sd = st + 2 * C::kKBytes + x * sbytes;
            const size_t srow = ((size_t)ph * P + off) * NG;
            bulk_load(sd, p.ks + srow, sbytes, &full[s]);
            bulk_load(sd + C::kSBytes, p.vs + srow, sbytes, &full[s]);
          }
          __syncwarp();
        }
        page = coming;
        if (++s == C::kStages) {
          s = 0;
          phase ^= 1;
          first = false;
        }
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3, mi = lane >> 3;
  int s = 0;        // the stage, and the phase of its barriers
  uint32_t phase = 0;
  bool ok = true;   // false after a wait ran out: the rest is passed over, every barrier still met
  const uint32_t x1 = reinterpret_cast<volatile uint32_t*>(consts)[-2], x16 = reinterpret_cast<volatile uint32_t*>(consts)[-1];
  // shared-memory addresses of this lane: ring, query fragments, starts, constant, K scales of row
  // g, and the 16-byte columns of its ldmatrix rows (row + 16 leaves the swizzle as it is)
  const uint32_t ring_a = smem_u32(ring), qf_a = smem_u32(qf + lane), bias_a = smem_u32(bias + c * 4), consts_a = smem_u32(consts);
  const uint32_t ks_off = (WT * warp + g) * (NG * 2);
  const int lrow = WT * warp + ((mi & 1) << 3) + (lane & 7);
  uint32_t code_off_[RB == 64 ? 2 : 4];
#pragma unroll
  for (int k = 0; k < (RB == 64 ? 2 : 4); ++k) code_off_[k] = code_off<RB, kTile>(lrow, 2 * k + (mi >> 1));
  auto code_at = [&](int u, int k) {  // columns 2 k, 2 k + 1 of the rows of subtile u
    return code_off_[k % (RB == 64 ? 2 : 4)] + (k / 4) * (kTile * 128) + 16 * u * (RB < 128 ? RB : 128);
  };
  grid_dep_wait();
  while (w.next(p)) {
    const Request& r = w.r;
    const int h = w.u / r.rt, rt = w.u - h * r.rt;
    const int nrows = min(kRows, min(r.qn, p.max_q) * p.Gq - rt * kRows);
    const size_t unit = (size_t)(unit_base(p, w.b, r.qs) + rt) * p.Hkv + h;
    // row x of the tile: query token (rt * 8 + x) / Gq, head of the group the remainder
    auto q_row = [&](int x, int& tok, int& head) {
      const int y = rt * kRows + x;
      tok = y / p.Gq;
      head = h * p.Gq + (y - tok * p.Gq);
    };
    // ---- the unit's prepared query
    {
      constexpr int NV = (C::kPrep / 16 + kWarps * 32 - 1) / (kWarps * 32);
      const uint4* src = reinterpret_cast<const uint4*>(p.qprep + unit * C::kPrep);
      uint4 v[NV];
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int x = tid + k * kWarps * 32;
        if (x < C::kPrep / 16) v[k] = ld_fresh(src + x);
      }
      consumers_sync();  // the segment before has been read to its end
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int x = tid + k * kWarps * 32;
        if (x < C::kPrep / 16) qf[x] = v[k];
      }
    }
    consumers_sync();
    const float rowfac[2] = {rowf[2 * c], rowf[2 * c + 1]};  // of the scores' columns 2c, 2c + 1
    // what rows 2c, 2c + 1 attend: tokens in (lo, hi]
    int hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      int tok, head;
      q_row(min(2 * c + e, nrows - 1), tok, head);
      hi[e] = r.kv - r.qn + tok;
      lo[e] = p.window ? (int)max((long long)hi[e] - p.window, -1ll) : -1;
    }
    int first_hi, last_lo;  // of the tile's first and last row: tokens in between are attended by all rows
    {
      int tok, head;
      q_row(0, tok, head);
      first_hi = r.kv - r.qn + tok;
      q_row(nrows - 1, tok, head);
      last_lo = p.window ? (int)max((long long)r.kv - r.qn + tok - p.window, -1ll) : -1;
    }

    // ---- (3) the tiles. l and o are held divided by 2^(m + ve): weights up to 2^-ve, whose product
    // with a V scale below 2^(ve + 15) stays below 2^15
    constexpr int kVeMin = -15, kVeMax = 1;
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
    float o[MT][4];
#pragma unroll
    for (int i = 0; i < MT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
    int ve = kVeMin;                                  // V scales seen so far are below 2^(ve + 15)
    uint32_t vlim = (uint32_t)(kVeMin + 30) << 10;    // the fp16 bits of 2^(ve + 15); above every scale at kVeMax
    bool bad_row = false;                             // column g attends a V scale that is not finite
    float ms0 = 0.0f, ms1 = 0.0f;                     // m + ve, 0 while nothing has been attended
    auto release = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
      if (++s == C::kStages) {
        s = 0;
        phase ^= 1;
      }
    };
    int t0 = (r.tile0 + w.i0) * kTile + WT * warp;               // the warp's first token of the tile
    for (int i = w.i0; i < w.i1 && ok; ++i, t0 += kTile) {
      if (!__all_sync(0xffffffffu, mbar_wait_bounded(&full[s], phase))) {
        if (lane == 0) atomicOr(&g_paged_err, kErrTimeoutLoad);
        ok = false;
        break;
      }
      const bool edge = t0 + WT > r.kv || t0 < r.t_lo;          // some rows hold no attended token's data
      if (edge && (t0 >= r.kv || t0 + WT <= r.t_lo)) {          // none does
        release();
        continue;
      }
      const uint32_t st = ring_a + s * C::kStage;               // shared-memory address of the stage
      const bool cut = t0 + WT - 1 > first_hi || t0 <= last_lo;  // some (token, row) pairs are masked
      // ---- scores: C layout (tokens g, g + 8; columns 2c, 2c + 1)
      float sc[KS][4];
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        float ska[NG], skb[NG];
        {
          uint32_t sa[NG / 2], sb[NG / 2];
          const uint32_t at = st + ks_off + 2 * C::kKBytes + 16 * u * (NG * 2);
          lds_words(at, sa);
          lds_words(at + 8 * (NG * 2), sb);
#pragma unroll
          for (int j = 0; j < NG / 2; ++j) {
            const float2 fa = __half22float2(u2h(sa[j])), fb = __half22float2(u2h(sb[j]));
            ska[2 * j] = fa.x;
            ska[2 * j + 1] = fa.y;
            skb[2 * j] = fb.x;
            skb[2 * j + 1] = fb.y;
          }
        }
        sc[u][0] = sc[u][1] = sc[u][2] = sc[u][3] = 0.0f;
        auto begin = [&](int grp, float (&a)[4]) {
          const uint4 v = lds128(bias_a + grp * 64);
          a[0] = __uint_as_float(v.x);
          a[1] = __uint_as_float(v.y);
          a[2] = __uint_as_float(v.z);
          a[3] = __uint_as_float(v.w);
        };
        auto add = [&](int grp, const float (&a)[4]) {
          sc[u][0] = fmaf(ska[grp], a[0], sc[u][0]);
          sc[u][1] = fmaf(ska[grp], a[1], sc[u][1]);
          sc[u][2] = fmaf(skb[grp], a[2], sc[u][2]);
          sc[u][3] = fmaf(skb[grp], a[3], sc[u][3]);
        };
        if constexpr (BITS == 4) {
#pragma unroll
          for (int gp = 0; gp < NC / 2; ++gp) {  // two 32-channel chunks per ldmatrix
            uint32_t x[4];                        // (tok g | g + 8) of chunk 2 gp, the same of 2 gp + 1
            ldmatrix_x4(x[0], x[1], x[2], x[3], st + code_at(u, gp));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint32_t a[4], b[4];
              nib8_plus8(x[2 * j], x1, x16, a);
              nib8_plus8(x[2 * j + 1], x1, x16, b);
#pragma unroll
              for (int k = 0; k < 32 / G; ++k) {
                const int grp = (2 * gp + j) * (32 / G) + k;
                const uint4 qv = lds128(qf_a + grp * 512);
                float acc[4];
                begin(grp, acc);
                mma_16816(acc, a[0], b[0], a[1], b[1], qv.x, qv.y);
                mma_16816(acc, a[2], b[2], a[3], b[3], qv.z, qv.w);
                add(grp, acc);
              }
            }
          }
        } else {
#pragma unroll
          for (int ch = 0; ch < NC; ++ch) {  // one 32-channel chunk per ldmatrix
            uint32_t x[4];                   // (tok g | g + 8) of channels 0 - 15, the same of 16 - 31
            ldmatrix_x4(x[0], x[1], x[2], x[3], st + code_at(u, ch));
            uint32_t a[2], b[2], a2[2], b2[2];
            byte4_plus128(x[0], a);
            byte4_plus128(x[1], b);
            byte4_plus128(x[2], a2);
            byte4_plus128(x[3], b2);
            const uint4 qv = lds128(qf_a + ch * 512);
            float acc[4];
            begin(ch * (32 / G), acc);
            mma_16816(acc, a[0], b[0], a[1], b[1], qv.x, qv.y);
            if constexpr (G == 16) {
              add(2 * ch, acc);
              begin(2 * ch + 1, acc);
            }
            mma_16816(acc, a2[0], b2[0], a2[1], b2[1], qv.z, qv.w);
            add(ch * (32 / G) + (32 / G - 1), acc);
          }
        }
      }
      // an infinite K scale can make a score -inf, the mark of a masked place: it becomes NaN (in
      // tiles without masked places only where the smallest score, mn, says so)
      auto unmark = [&] {
#pragma unroll
        for (int u = 0; u < KS; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (sc[u][e] == -INFINITY) sc[u][e] = __int_as_float(0x7fc00000);
      };
      float mn = 0.0f;
      if (cut) {
        unmark();
#pragma unroll
        for (int u = 0; u < KS; ++u) {
          const int ta = t0 + 16 * u + g, tb = ta + 8;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (ta > hi[e] || ta <= lo[e]) sc[u][e] = -INFINITY;
            if (tb > hi[e] || tb <= lo[e]) sc[u][2 + e] = -INFINITY;
          }
        }
      } else {
#pragma unroll
        for (int u = 0; u < KS; ++u) mn = fminf(fminf(mn, fminf(sc[u][0], sc[u][1])), fminf(sc[u][2], sc[u][3]));
      }
      // ---- V scales: a token per lane (two lanes where the warp has 16) for the largest of them.
      // Those of tokens that hold no attended data, and those that are not finite, are made
      // zeros in place (this warp alone reads them)
      const uint32_t vsc = st + 2 * C::kKBytes + C::kSBytes + WT * warp * (NG * 2);
      uint32_t top = 0;
      {
        constexpr int LW = NG / 2 * WT / 32;  // 32-bit words of a lane
        const uint32_t vw = vsc + lane * (LW * 4);
        uint32_t x[LW];
        lds_words(vw, x);
#pragma unroll
        for (int k = 0; k < LW; ++k) top = __vmaxu2(top, x[k]);
        const int t = t0 + lane * WT / 32;
        const bool dead = edge && (t >= r.kv || t < r.t_lo);
        const bool odd = !dead && max(top & 0xFFFFu, top >> 16) >= 0x7C00u;  // not finite, or a sign
        if (__any_sync(0xffffffffu, dead || odd)) {
          bool bad = false;
          top = 0;
#pragma unroll
          for (int k = 0; k < LW; ++k) {
            if (odd && ((x[k] & 0x7C00u) == 0x7C00u || (x[k] & 0x7C000000u) == 0x7C000000u)) bad = true;
            top = __vmaxu2(top, x[k] & 0x7FFF7FFFu);
          }
          if (dead || bad) {
            top = 0;
#pragma unroll
            for (int k = 0; k < LW; ++k) asm volatile("st.shared.u32 [%0], %1;" ::"r"(vw + 4 * k), "r"(0) : "memory");
          }
          uint32_t bads = __ballot_sync(0xffffffffu, bad);
          fence_proxy_async_smem();  // before the producer's next copy into these rows
          __syncwarp();
          while (bads) {
            const int tk = t0 + (__ffs(bads) - 1) * WT / 32;
            bads &= bads - 1;
            int tok, head;
            q_row(min(g, nrows - 1), tok, head);
            const int h1 = r.kv - r.qn + tok;
            if (tk <= h1 && (!p.window || (long long)tk > (long long)h1 - p.window)) bad_row = true;
          }
        }
        top = max(top & 0xFFFFu, top >> 16);
      }
      // ---- online softmax in base 2: m_run is a ceiling of the scores so far; it moves, by
      // some headroom more than needed, only when a score of this stage passes it
      float mx0 = sc[0][0], mx1 = sc[0][1];
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        mx0 = fmaxf(mx0, fmaxf(sc[u][0], sc[u][2]));
        mx1 = fmaxf(mx1, fmaxf(sc[u][1], sc[u][3]));
      }
      mx0 *= rowfac[0];
      mx1 *= rowfac[1];
      if (__any_sync(0xffffffffu, mx0 > m_run[0] || mx1 > m_run[1] || top >= vlim || mn == -INFINITY)) {
        if (mn == -INFINITY) unmark();
        constexpr float kHeadroom = 3.0f;
        float a = mx0, b = mx1;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
          b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, off));
        }
        const uint32_t t = __reduce_max_sync(0xffffffffu, top);
        int nve = ve;
        if (t >= vlim) nve = (int)(t >> 10) - 29;
        const float m0 = a > m_run[0] ? a + kHeadroom : m_run[0];
        const float m1 = b > m_run[1] ? b + kHeadroom : m_run[1];
        const float fv = pow2f(ve - nve);
        const float f0 = (m0 == m_run[0] ? 1.0f : ex2_approx(m_run[0] - m0)) * fv;
        const float f1 = (m1 == m_run[1] ? 1.0f : ex2_approx(m_run[1] - m1)) * fv;
        l_run[0] *= f0;
        l_run[1] *= f1;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          o[mt][0] *= f0;
          o[mt][1] *= f1;
          o[mt][2] *= f0;
          o[mt][3] *= f1;
        }
        m_run[0] = m0;
        m_run[1] = m1;
        ms0 = m0 == -INFINITY ? 0.0f : m0 + (float)nve;
        ms1 = m1 == -INFINITY ? 0.0f : m1 + (float)nve;
        ve = nve;
        vlim = ve < kVeMax ? (uint32_t)(ve + 30) << 10 : 0xFFFFu;
      }
      // P as the B operand of the output product: (tokens 2c, 2c + 1 | + 8; column g)
      uint32_t pb[KS][2];
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        const float p0 = ex2_approx(fmaf(sc[u][0], rowfac[0], -ms0)), p1 = ex2_approx(fmaf(sc[u][1], rowfac[1], -ms1));
        const float p2 = ex2_approx(fmaf(sc[u][2], rowfac[0], -ms0)), p3 = ex2_approx(fmaf(sc[u][3], rowfac[1], -ms1));
        l_run[0] += p0 + p2;
        l_run[1] += p1 + p3;
        pb[u][0] = movmatrix_trans(pack_half2(p0, p1));
        pb[u][1] = movmatrix_trans(pack_half2(p2, p3));
      }
      // ---- output: O[channel][column] += V[channel][token] P[token][column] scale; the codes
      // stand off too high, which a product with a constant takes out again
      const uint4 off = lds128(consts_a);  // read here: four registers in order, not four moves for every product
#pragma unroll
      for (int u = 0; u < KS; ++u) {
        // the scales of tokens 2c, 2c + 1, 2c + 8, 2c + 9
        uint32_t sw[4][NG / 2];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          lds_words(vsc + (2 * c) * (NG * 2) + (16 * u + (e & 1) + ((e & 2) << 2)) * (NG * 2), sw[e]);
        }
        // P times the scale of group grp, as the two B registers
        auto weighted = [&](int grp, uint32_t& b0, uint32_t& b1) {
          const uint32_t sel = (grp & 1) ? 0x7632u : 0x5410u;
          const uint32_t s0 = prmt(sw[0][grp >> 1], sw[1][grp >> 1], sel);
          const uint32_t s1 = prmt(sw[2][grp >> 1], sw[3][grp >> 1], sel);
          b0 = h2u(__hmul2(u2h(s0), u2h(pb[u][0])));
          b1 = h2u(__hmul2(u2h(s1), u2h(pb[u][1])));
        };
        if constexpr (BITS == 4) {
#pragma unroll
          for (int gp = 0; gp < NC / 2; ++gp) {
            uint32_t x[4];  // transposed: (tokens 2c.. | 2c + 8..) of chunk 2 gp, the same of 2 gp + 1
            ldmatrix_x4_trans(x[0], x[1], x[2], x[3], st + C::kKBytes + code_at(u, gp));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int ch = 2 * gp + j;
              uint32_t a[4], b[4];  // channels 4g, 4g + 1 (16 times), 4g + 2, 4g + 3 (16 times) of the chunk
              nib8_plus8(x[2 * j], x1, x16, a);
              nib8_plus8(x[2 * j + 1], x1, x16, b);
              if constexpr (G == 32) {
                uint32_t b0, b1;
                weighted(ch, b0, b1);
                mma_16816(o[2 * ch], a[0], a[1], b[0], b[1], b0, b1);
                mma_16816(o[2 * ch + 1], a[2], a[3], b[2], b[3], b0, b1);
                mma_16816(o[2 * ch], off.x, off.y, off.z, off.w, b0, b1);
                mma_16816(o[2 * ch + 1], off.x, off.y, off.z, off.w, b0, b1);
              } else {
#pragma unroll
                for (int k = 0; k < 2; ++k) {  // lane g's channels lie in half g / 4 of the chunk
                  const uint32_t m = (g >> 2) == k ? 0xffffffffu : 0u;
                  uint32_t b0, b1;
                  weighted(2 * ch + k, b0, b1);
                  mma_16816(o[2 * ch], a[0] & m, a[1] & m, b[0] & m, b[1] & m, b0, b1);
                  mma_16816(o[2 * ch + 1], a[2] & m, a[3] & m, b[2] & m, b[3] & m, b0, b1);
                  mma_16816(o[2 * ch], off.x & m, off.y & m, off.z & m, off.w & m, b0, b1);
                  mma_16816(o[2 * ch + 1], off.x & m, off.y & m, off.z & m, off.w & m, b0, b1);
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int ch = 0; ch < NC; ++ch) {
            uint32_t x[4];  // transposed: (tokens 2c.. | 2c + 8..) of channels 0 - 15, the same of 16 - 31
            ldmatrix_x4_trans(x[0], x[1], x[2], x[3], st + C::kKBytes + code_at(u, ch));
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t a[2], b[2], b0, b1;  // channels 2g, 2g + 1 of the half
              byte4(x[2 * k], a);
              byte4(x[2 * k + 1], b);
              weighted(G == 32 ? ch : 2 * ch + k, b0, b1);
              mma_16816(o[2 * ch + k], a[0], a[1], b[0], b[1], b0, b1);
            }
          }
        }
      }
      release();
    }

    // ---- join the warps: M, L, and O = sum of o 2^(m - M), in true units; a quarter of the
    // channels per warp
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      l_run[0] += __shfl_xor_sync(0xffffffffu, l_run[0], off);
      l_run[1] += __shfl_xor_sync(0xffffffffu, l_run[1], off);
    }
    const uint32_t bad_rows = __ballot_sync(0xffffffffu, bad_row);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m_run[e] += (float)ve;  // from here on with V's power of two
      if ((bad_rows >> (4 * (2 * c + e))) & 15u) l_run[e] = __int_as_float(0x7fc00000);
      if (g == 0) {
        wml[warp * 2 * kRows + 2 * c + e] = m_run[e];
        wml[warp * 2 * kRows + kRows + 2 * c + e] = l_run[e];
      }
    }
    consumers_sync();
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float M = -INFINITY;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) M = fmaxf(M, wml[x * 2 * kRows + 2 * c + e]);
      f[e] = m_run[e] == -INFINITY ? 0.0f : ex2_approx(m_run[e] - M) * pow2f(24);
    }
    float own[TW][4];
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      float4* dst = obuf + ((q * (kWarps - 1) + ((warp - q - 1) & (kWarps - 1))) * TW) * 32 + lane;
#pragma unroll
      for (int t = 0; t < TW; ++t) {
        const float odd = BITS == 4 ? 0.0625f : 1.0f;  // rows g + 8 hold the codes that stood 16 times too high
        float (&v)[4] = o[q * TW + t];
        v[0] *= f[0];
        v[1] *= f[1];
        v[2] *= f[0] * odd;
        v[3] *= f[1] * odd;
        if (q != warp) {
          dst[t * 32] = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) own[t][k] = v[k];
        }
      }
    }
    consumers_sync();
    // ---- the segment's partial: its unit's own when the unit is whole; else a slot of this CTA,
    // the first for the segment that starts its piece, the second for one that ends it. The
    // unit's tiles are [u0, u0 + nt) of the line; CTA x holds [x per, (x + 1) per) of it.
    const bool whole = w.i0 == 0 && w.i1 == r.nt;
    const long long u0 = w.base + (long long)w.u * r.nt, x0 = (long long)blockIdx.x * per;
    const int slot = 2 * (int)blockIdx.x + (x0 >= u0 ? 0 : 1);
    float* dst = whole ? p.part_unit + unit * C::PART : p.part + (size_t)slot * C::PART;
    if (tid < kRows) {
      float M = -INFINITY, L = 0.0f;
#pragma unroll
      for (int x = 0; x < kWarps; ++x) M = fmaxf(M, wml[x * 2 * kRows + tid]);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float mw = wml[x * 2 * kRows + tid], lw = wml[x * 2 * kRows + kRows + tid];
        L += mw != -INFINITY ? lw * ex2_approx(mw - M) : lw;  // nothing attended: 0, or NaN where scores are
      }
      dst[tid] = M;
      dst[kRows + tid] = L;
    }
    if (tid == 0 && w.i0 == 0)
      p.desc[unit] = whole ? make_int2(0, 0) : make_int2(slot, (int)((u0 + r.nt - 1) / per - blockIdx.x) + 1);
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const float4* src = obuf + (warp * (kWarps - 1) * TW + t) * 32 + lane;
#pragma unroll
      for (int k = 0; k < kWarps - 1; ++k) {
        const float4 v = src[k * TW * 32];
        own[t][0] += v.x;
        own[t][1] += v.y;
        own[t][2] += v.z;
        own[t][3] += v.w;
      }
      const int mt = warp * TW + t;  // the channels of tile mt's rows g and g + 8
      const int ch = BITS == 4 ? (mt >> 1) * 32 + 4 * g + ((mt & 1) ? 2 : 0) : 16 * mt + 2 * g;
      float* d0 = dst + 2 * kRows + (2 * c) * D + ch;
      if (2 * c < nrows) *reinterpret_cast<float2*>(d0) = make_float2(own[t][0], own[t][2]);
      if (2 * c + 1 < nrows) *reinterpret_cast<float2*>(d0 + D) = make_float2(own[t][1], own[t][3]);
    }
  }
}

// ---------------------------------------------------------------- last kernel: partials to outputs
// Block u: the partials of unit u in CTA order, then out = Wo (o / l) with o as an fp16 hi + lo
// pair (samples as rows, query rows as columns). A few KB per unit through L2: bound by the
// latency of the chain lengths -> partials -> output; the matrix is loaded before the wait for
// the main kernel.
template <int D, int BITS>
__global__ void __launch_bounds__(kUnitWarps<D> * 32) join_paged_kernel(const __grid_constant__ PagedParams p) {
  constexpr int MT = D / 16, NWARP = kUnitWarps<D>, TW = MT / NWARP, NT = NWARP * 32, ST = D + 4, PART = 2 * kRows + kRows * D;
  __shared__ __align__(16) float om[kRows * ST];
  __shared__ __align__(16) __half xb[kRows * (D + 8)];
  __shared__ float red[2][NT / 8][kRows], wts[kMaxCtas * kRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  const int unit = blockIdx.x, xt = unit / p.Hkv, h = unit - xt * p.Hkv;
  uint4 wf[TW][MT];
#pragma unroll
  for (int t = 0; t < TW; ++t)
#pragma unroll
    for (int ks = 0; ks < MT; ++ks) wf[t][ks] = __ldg(p.wo + ((warp + NWARP * t) * MT + ks) * 32 + lane);
  constexpr int NX = kRows * D / 4 / NT, U = 8;  // float4 values of a thread, partials in flight
  float4 fac[NX];                                // of the channels of each
#pragma unroll
  for (int x = 0; x < NX; ++x) fac[x] = __ldg(reinterpret_cast<const float4*>(p.ochan) + (tid + x * NT) % (D / 4));
  const uint4 sgn = __ldg(p.osgn + tid % (D / 8));  // of this thread's 8 samples of every row
  grid_dep_launch();
  grid_dep_wait();
  // the loads of a step together: request and description; then the first partials' m, l and o
  const int2 d = ld_fresh(p.desc + unit);
  int b, rt;
  request_at(p, xt, b, rt);
  const Request r = request_of<128>(p, b);
  const int nrows = min(kRows, min(r.qn, p.max_q) * p.Gq - rt * kRows);
  if (nrows <= 0 || rt < 0) return;  // no such unit: nothing was written for it
  const int np = max(1, min(d.y, kMaxCtas));
  // the first CTA's slot, then the first slots of the CTAs after it
  auto part = [&](int k) {
    return d.y == 0 ? p.part_unit + (size_t)unit * PART : p.part + (size_t)(k == 0 ? d.x : (d.x & ~1) + 2 * k) * PART;
  };
  float4 v[U][NX];
  auto load_o = [&](int k0) {
#pragma unroll
    for (int k = 0; k < U; ++k)
#pragma unroll
      for (int x = 0; x < NX; ++x)
        if (k0 + k < np) v[k][x] = __ldcg(reinterpret_cast<const float4*>(part(k0 + k) + 2 * kRows) + tid + x * NT);
  };
  {
    const int row = tid & 7, k0 = tid >> 3;
    float m0 = -INFINITY, l0 = 0.0f;  // of partial k0
    if (k0 < np) {
      m0 = __ldcg(part(k0) + row);
      l0 = __ldcg(part(k0) + kRows + row);
    }
    load_o(0);
    float M = m0, L = 0.0f;
    for (int k = k0 + NT / 8; k < np; k += NT / 8) M = fmaxf(M, __ldcg(part(k) + row));
    red[0][k0][row] = M;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NT / 8; ++k) M = fmaxf(M, red[0][k][row]);
    for (int k = k0; k < np; k += NT / 8) {
      const float m = k == k0 ? m0 : __ldcg(part(k) + row), l = k == k0 ? l0 : __ldcg(part(k) + kRows + row);
      const float f = m != -INFINITY ? ex2_approx(m - M) : 0.0f;
      L += m != -INFINITY ? l * f : l;
      wts[k * kRows + row] = f;
    }
    red[1][k0][row] = L;
    __syncthreads();
  }
  {
    float4 acc[NX];
#pragma unroll
    for (int x = 0; x < NX; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < np; k0 += U) {
      if (k0) load_o(k0);
#pragma unroll
      for (int k = 0; k < U; ++k)
#pragma unroll
        for (int x = 0; x < NX; ++x) {
          const float f = k0 + k < np ? wts[(k0 + k) * kRows + (tid + x * NT) / (D / 4)] : 0.0f;
          if (f != 0.0f) {
            acc[x].x = fmaf(f, v[k][x].x, acc[x].x);
            acc[x].y = fmaf(f, v[k][x].y, acc[x].y);
            acc[x].z = fmaf(f, v[k][x].z, acc[x].z);
            acc[x].w = fmaf(f, v[k][x].w, acc[x].w);
          }
        }
    }
#pragma unroll
    for (int x = 0; x < NX; ++x) {
      const int y = tid + x * NT, row = y / (D / 4);
      acc[x] = make_float4(acc[x].x * fac[x].x, acc[x].y * fac[x].y, acc[x].z * fac[x].z, acc[x].w * fac[x].w);
      // rows behind the tile's last were not written
      *reinterpret_cast<float4*>(om + row * ST + 4 * (y - row * (D / 4))) = row < nrows ? acc[x] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __syncthreads();
  float L = 0.0f;
#pragma unroll
  for (int k = 0; k < NT / 8; ++k) L += red[1][k][g];
  const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;  // nothing attended: zeros (NaN stays)
  const float* orow = om + g * ST;
  float mx = 0.0f;
#pragma unroll
  for (int x = 0; x < D / 16; ++x) {
    const float4 v = *reinterpret_cast<const float4*>(orow + 16 * x + 4 * c);
    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
  const int ex = row_exponent(mx * inv);
  const float fx = inv * pow2f(-ex);
  float acc[TW][4] = {};
#pragma unroll
  for (int ks = 0; ks < MT; ++ks) {
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 v = *reinterpret_cast<const float2*>(orow + 16 * ks + 8 * e + 2 * c);
      const __half2 hv = __floats2half2_rn(v.x * fx, v.y * fx);
      const float2 hf = __half22float2(hv);
      hi[e] = h2u(hv);
      lo[e] = pack_half2(v.x * fx - hf.x, v.y * fx - hf.y);
    }
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      mma_16816(acc[t], wf[t][ks].x, wf[t][ks].y, wf[t][ks].z, wf[t][ks].w, hi[0], hi[1]);
      mma_16816(acc[t], wf[t][ks].x, wf[t][ks].y, wf[t][ks].z, wf[t][ks].w, lo[0], lo[1]);
    }
  }
  float fo[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) fo[e] = pow2f(__shfl_sync(0xffffffffu, ex, 4 * (2 * c + e)));
#pragma unroll
  for (int t = 0; t < TW; ++t) {
    __half* x0 = xb + (2 * c) * (D + 8) + 16 * (warp + NWARP * t) + g;
    x0[0] = __float2half_rn(acc[t][0] * fo[0]);
    x0[D + 8] = __float2half_rn(acc[t][1] * fo[1]);
    x0[8] = __float2half_rn(acc[t][2] * fo[0]);
    x0[D + 8 + 8] = __float2half_rn(acc[t][3] * fo[1]);
  }
  __syncthreads();
  for (int x = tid; x < nrows * (D / 8); x += NT) {
    const int row = x / (D / 8), k = x - row * (D / 8);
    const int y = rt * kRows + row, tok = y / p.Gq, head = h * p.Gq + (y - tok * p.Gq);
    const uint4 v = *reinterpret_cast<const uint4*>(xb + row * (D + 8) + 8 * k);
    *(reinterpret_cast<uint4*>(p.out + ((size_t)(r.qs + tok) * p.Hq + head) * D) + k) =
        make_uint4(v.x ^ sgn.x, v.y ^ sgn.y, v.z ^ sgn.z, v.w ^ sgn.w);
  }
}

// ---------------------------------------------------------------- host side
// Workspace: the partials of cut units, then per unit its prepared query, partial and
// description. Nothing in it outlives a call.
constexpr size_t kPartBytes = (size_t)2 * kMaxCtas * (2 * kRows + kRows * kMaxD) * 4;
// of a unit, for every form of a head_dim: fragments, starts and factors; m, l, o; description
constexpr size_t prep_bytes(int D) { return (size_t)(D / 16) * 512 + (D / 16) * 64 + kRows * 4; }
constexpr size_t unit_bytes(int D) { return prep_bytes(D) + (2 * kRows + kRows * D) * 4 + 16; }
constexpr int kFewRows = 32;            // query rows of a request up to which this file's kernels take every call
constexpr long long kFewUnits = 4096;   // units up to which they may take one with more (their workspace: 36 MB, 72 at D = 256)

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
// units of a call with n_q query tokens, at most `rows` query rows of a request: the smaller of
// the two ways to number them (unit_base)
long long units_of(int B, int Hkv, int Gq, int n_q, long long rows) {
  return (long long)Hkv * std::min(B * ceil_div(rows, kRows), (long long)n_q * Gq / kRows + B);
}

template <int D, int G, int BITS>
kvq_status run_paged(const PagedAttendHost& a, cudaStream_t strm) {
  using C = PCfg<D, G, BITS>;
  PagedParams p{};
  const int P = 1 << a.page_shift;
  const uint64_t dims[3] = {(uint64_t)C::RB, (uint64_t)P, (uint64_t)a.num_pages * a.Hkv};
  const uint64_t strides[2] = {(uint64_t)C::RB, (uint64_t)C::RB * P};
  const uint32_t box[3] = {(uint32_t)(C::RB < 128 ? C::RB : 128), (uint32_t)std::min(P, C::kTile), 1u};
  const CUtensorMapSwizzle sw = C::RB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  kvq_status st = encode_tiled_new(&p.kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.kc, dims, strides, box, sw, "K pages");
  if (st == KVQ_OK)
    st = encode_tiled_new(&p.vmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, a.vc, dims, strides, box, sw, "V pages");
  if (st != KVQ_OK) return st;
  p.q = a.q;
  p.ks = a.ks;
  p.vs = a.vs;
  p.table = a.table;
  p.kv_lens = a.kv_lens;
  p.q_starts = a.q_starts;
  p.wq = a.pk->basis->wqf_dev;
  p.wo = a.pv->basis->wof_dev;
  p.qchan = a.pk->dec_dev->chan;
  p.ochan = a.pv->dec_dev->chan;
  p.qsgn = a.pk->dec_dev->sgn;
  p.osgn = reinterpret_cast<const uint4*>(a.pv->dec_dev->sgn);
  p.out = a.out;
  p.q_ts = a.q_token_stride;
  p.q_hs = a.q_head_stride;
  p.table_stride = a.table_stride;
  const float sigma = a.sigma > 0.0f ? a.sigma : 1.0f / sqrtf((float)D);
  p.qfac = sigma * 1.4426950408889634f;
  p.B = a.B;
  p.n_q = a.n_q;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.Gq = a.Hq / a.Hkv;
  p.max_q = a.max_q_len;
  p.rt_max = (int)(((long long)std::min(a.max_q_len, a.n_q) * p.Gq + kRows - 1) / kRows);
  p.max_kv = (int)std::min<long long>(a.max_kv_len, (long long)a.max_pages * P);
  p.num_pages = a.num_pages;
  p.page_shift = a.page_shift;
  p.window = a.window;
  const double attended = a.window ? std::min<double>(p.max_kv, (double)a.window + std::min(a.max_q_len, a.n_q)) : p.max_kv;  // tokens of a unit
  // A piece of t tiles takes about t us, joining a unit's n / t pieces about 0.1 n / t: where
  // there are CTAs to spare, t = sqrt(0.1 n) (one KV head of 256, 16K tokens:
  // 30.6 us with pieces of 2, 24.7 so).
  p.min_tiles = std::max(2, (int)std::sqrt(0.1 * attended / C::kTile));
  const long long rows_max = (long long)std::min(a.max_q_len, a.n_q) * p.Gq;
  const size_t units = (size_t)units_of(a.B, a.Hkv, p.Gq, a.n_q, rows_max);
  p.packed = units < (size_t)a.B * a.Hkv * p.rt_max;  // (then there are q_starts: without, a request has one token)
  static_assert(C::kPrep <= prep_bytes(D), "workspace");
  p.part = reinterpret_cast<float*>(a.ws);
  p.part_unit = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) + kPartBytes);
  p.qprep = reinterpret_cast<uint8_t*>(p.part_unit + units * C::PART);
  p.desc = reinterpret_cast<int2*>(p.qprep + units * C::kPrep);
  // no more CTAs than pieces of min_tiles tiles if every request were as long as it may be
  const long long most = (long long)units * std::max(1, (p.max_kv + C::kTile - 1) / C::kTile);
  const int slots = std::min(kMaxCtas, num_sms(a.pk->device) * C::kCtas);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)units);
  cfg.blockDim = dim3(kUnitWarps<D> * 32);
  cfg.stream = strm;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = allow_smem<attend_paged_kernel<D, G, BITS>>(a.pk->device, C::kSmem);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, rotate_paged_kernel<D, G, BITS>, p);
  if (e == cudaSuccess) {
    cfg.gridDim = dim3((unsigned)std::min<long long>(slots, (most + p.min_tiles - 1) / p.min_tiles));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmem;
    e = cudaLaunchKernelEx(&cfg, attend_paged_kernel<D, G, BITS>, p);
  }
  if (e == cudaSuccess) {
    cfg.gridDim = dim3((unsigned)units);
    cfg.blockDim = dim3(kUnitWarps<D> * 32);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, join_paged_kernel<D, BITS>, p);
  }
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, std::string("attend_paged launch: ") + cudaGetErrorString(e));
  return KVQ_OK;
}

}  // namespace

namespace {

// Whether the prompt kernel takes a call, by what both would take (us, fitted to both kernels
// on 1, 4 and 32 requests of 256, 2048 and 16384 tokens with 1 - 64 query tokens each). Here a
// tile of 8 rows costs little and every row tile converts the cache again; there up to 256 (128)
// rows cost about the same. For example 4 requests of 2048 tokens, 4 query heads per KV head:
// 16 query tokens 29.9 us here and 29.5 there, 32 tokens 47.8 and 30.1; one request of 256
// tokens: 64 query tokens 16.3 and 22.9; 32 requests: 8 tokens 28.6 and 30.7, 12 tokens 39.4
// and 31.0.
bool prefers_prompt(const PagedAttendHost& a) {
  if (a.path) return a.path == 2;
  const int Gq = a.Hq / a.Hkv, q = std::min(a.max_q_len, a.n_q);
  const long long rows = (long long)q * Gq;
  if (rows <= kFewRows) return false;
  const long long units = units_of(a.B, a.Hkv, Gq, a.n_q, rows);
  if (units > kFewUnits) return true;
  const bool d128 = a.pk->D == 128;
  const long long all = (long long)a.n_q * Gq, R = d128 ? 256 : 128;
  const long long cap = std::min<long long>(a.max_kv_len, (long long)a.max_pages << a.page_shift);
  const long long kv = a.window ? std::min<long long>(cap, (long long)a.window + q) : cap;
  const long long tiles = std::max(1ll, ceil_div(kv, d128 ? 128 : 64));
  const double few_tiles = (double)a.Hkv * std::min(a.B * ceil_div(rows, kRows), all / kRows + a.B) * tiles;
  const double prompt_tiles = (double)a.Hkv * std::min(a.B * ceil_div(rows, R), all / R + a.B) * tiles;
  const double few = d128 ? 11.0 + 0.0035 * few_tiles + 0.012 * units : 16.0 + 0.004 * few_tiles + 0.02 * units;
  const double prompt = d128 ? 22.0 + 0.020 * prompt_tiles : 27.0 + 0.035 * prompt_tiles;
  return prompt < few;
}

}  // namespace

size_t paged_workspace_bytes(int B, int Hq, int Hkv, int D, int n_q, int max_q_len, int path) {
  const int Gq = Hq / Hkv;
  const long long rows = (long long)std::min(max_q_len, std::max(n_q, 1)) * Gq;
  if (path == 1) return kPartBytes + (size_t)units_of(B, Hkv, Gq, n_q, rows) * unit_bytes(D);
  if (path == 2) return prompt_part_bytes();
  // whatever kernel a call with these sizes, or smaller ones, goes to
  long long units = units_of(B, Hkv, Gq, n_q, std::min<long long>(rows, kFewRows));
  if (rows > kFewRows) units = std::max(units, std::min(kFewUnits, units_of(B, Hkv, Gq, n_q, rows)));
  const size_t few = kPartBytes + (size_t)units * unit_bytes(D);
  return rows > kFewRows ? std::max(few, prompt_part_bytes()) : few;
}

kvq_status launch_attend_paged(const PagedAttendHost& a, cudaStream_t s) {
  if (prefers_prompt(a)) return launch_attend_prompt(a, a.ws, s);
  return dispatch_dgb(a.pk->D, a.pk->G, a.pk->bits, [&](auto d, auto g, auto b) {
    return run_paged<decltype(d)::value, decltype(g)::value, decltype(b)::value>(a, s);
  });
}

uint32_t paged_error_flags(bool clear) {
  uint32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_paged_err, sizeof(v));
  if (clear && v) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_paged_err, &z, sizeof(z));
  }
  return v;
}

}  // namespace kvq
