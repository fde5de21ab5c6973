// kvq_attend_prompt.cu -- attention of many query tokens per request (prompts, chunks of
// prompts) over a paged int4/int8 cache for sm_100a, on the 5th-generation tensor cores, in
// the rotated domain as the few-token kernel (kvq_attend_paged.cu):
//   q~ = Lambda_K^-1 Q diag(s_K) q,   S = q~ K^T with K = c_K scale_K,
//   O = softmax(sigma S) V with V = c_V scale_V,   out = O (Lambda_V^-1 Q diag(s_V)).
//
// Work. A unit is (request, block of R query rows, KV head), a query row one (query token,
// head of the KV head's group), R = 256 at head_dim 128 and 128 at 256; its tokens are taken
// in tiles of T = 128 (64), of which those that the mask leaves empty for the whole unit are
// not counted. The tiles of all units form one line and every CTA of a persistent grid (one
// per SM) takes an equal piece of it. A unit cut by a piece's border leaves partials (m, l, o)
// in the workspace, which a second kernel joins in CTA order; whole units are written here.
//
// Roles (13 warps):
//   dequantisers  each thread fetches what it converts by async copies, most of a tile ahead; a
//                 word of codes becomes fp16 pairs by masks, times the scale (one rounding per
//                 element), and goes to shared memory as K- or V-rows with a 128-byte swizzle.
//                 Two K and two V tiles are held; every query row of the unit uses them.
//   MMA           a warp issues S = Q K^T (shared, shared -> TMEM) and O += P V (P in TMEM
//                 over S; V as a transposed operand, so one layout serves both).
//   softmax       a thread per query row: the maximum over its S row, exp2, P as fp16 back to
//                 TMEM. O is rescaled only when a row's maximum has grown by more than 2^8
//                 since the last time, which after the first tiles is rare.
// Head_dim 128 has two query blocks of 128 rows that alternate: while one's softmax runs the
// tensor cores work for the other. At head_dim 256 there is room in TMEM for one block and
// two S buffers: the scores of the next tile are made while the softmax of this one runs.
// The query's rotation and the output's un-rotation are products of the same kind: the
// plan's matrix passes through the K tiles' ring, and each row normalises its own result.
//
// Chunks of 2048 tokens on 16K caches (32 / 8 heads of 128): 1.03 ms back to back under the
// power cap (785 TFLOP/s, 57 % of the sustained matrix rate), 8-bit codes 1.08 ms, 4 / 1 heads of
// 256 0.41 ms (495 TFLOP/s); 8 rows at a time with register products the first was 15.2 ms. A
// tile of 256 x 128 takes about 4500 cycles, of which the products 2048; a softmax warp spends
// 1000 on the maxima, 2000 on P (the exponential unit serves two such warps per scheduler). Bound
// by that chain and by the instruction caches: longer (more unrolled) forms of any role slowed
// all of them.
//
// Number formats, each chosen for products of one fp16 tile per operand (a hi + lo pair would
// double their number and the shared memory they wait for):
//   * K and V are fp16 c * scale: exact multiples of 2^-24 below 2^-13 and one rounding (2^-12
//     on average) elsewhere. A tile with a scale from 2^12 (int8: 2^9) on is held divided by 2^8,
//     so that no product leaves fp16, and O is brought to the power of the tile that is added
//     next (beside such a scale, V below 2^-6 in the same tile keeps 2^-17 of 1, not its own 11
//     bits).
//   * The rotation's entries are one fp16 rounding each (none for the SRHT); q~ is one after a
//     power-of-two normalisation per row, as is o before the output's rotation. The join of cut
//     units takes o as hi + lo, which costs nothing beside reading the partials; whole units would
//     pay about 2 us each for it, so a row may be 10 % nearer the formula where its unit is cut.
//   * P is one fp16 rounding, its largest value between 2^7 and 2^15: weights down to 2^-21 of
//     the largest keep 2^-12 on average, smaller ones an error of at most 2^-32 of the largest.
//   * S, O, the maxima and sums are fp32. A token whose V scale is not finite is held as zeros and
//     the rows that attend it (and no others) are set to NaN at the end.
#include <algorithm>
#include <cmath>
#include <string>

#include "kvq_internal.h"
#include "kvq_ptx.cuh"

namespace kvq {

__device__ uint32_t g_prompt_err = 0;

namespace {

constexpr int kPrWarps = 13;
constexpr int kPrThreads = kPrWarps * 32;
constexpr int kPrMaxCtas = 160;
constexpr int kPrPart = 256 * (128 + 2);  // floats of a partial: m, l and o of R rows (R * D = 32768)
constexpr int kFlagRing = 8;              // tiles whose flags are held: softmax is at most three behind

template <int D, int G, int BITS>
struct PrCfg {
  static constexpr int NQ = D == 128 ? 2 : 1;   // blocks of 128 query rows
  static constexpr int SB = D == 128 ? 1 : 2;   // S buffers per block
  static constexpr int R = 128 * NQ;
  static constexpr int T = D == 128 ? 128 : 64;
  static constexpr int ND = kPrWarps - 1 - 4 * NQ;  // dequantiser warps
  static constexpr int NW = D / T;              // ring tiles of a rotation matrix
  static constexpr int NJ = 16 / ND;            // items (a row's 32 channels) of a thread, tile and operand
  static constexpr int CW = BITS;               // 32-bit words of an item's codes
  static constexpr int kQ = NQ * 128 * D * 2;
  static constexpr int kTile = T * D * 2;
  // codes on their way, per dequantiser thread: a ring of half tiles (NJ / 2 items), the next
  // tile's scales (4 bytes per item of K and V), the table entries of the tile after it
  static constexpr int NS = BITS == 4 ? 4 : 3;
  static constexpr int kHalf = NJ / 2 * CW * 4 * ND * 32;
  static constexpr int kRing = NS * kHalf;
  static constexpr int kScales = 2 * NJ * 4 * ND * 32;
  static constexpr int kEnt = NJ * 4 * ND * 32;
  static constexpr int kScan = kPrThreads * 8;
  static constexpr int kFlags = kFlagRing * 5 * 4;
  static constexpr int kBars = 256;
  static_assert(kScan <= kTile, "the scan uses the K tiles");
  static constexpr int kConst = 2 * (D * 4 + D * 2);  // the plans' factors and sign masks
  static constexpr int kSmem = kQ + 4 * kTile + kRing + kScales + kEnt + kConst + kFlags + kBars + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // TMEM columns
  static constexpr int kO = 0;                  // O of block q at q * D
  static constexpr int kS = 256;                // S of block q, buffer s at kS + (q + s) * T
};

struct PromptParams {
  const uint16_t* q;
  const uint8_t* kc;
  const uint16_t* ks;
  const uint8_t* vc;
  const uint16_t* vs;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  const uint16_t* wq;      // [channel][sample], rows in word_channel order
  const uint16_t* wo;      // [sample][channel], columns in word_channel order
  const uint4* wof;        // the same as fragments, natural order (all three without signs and factors)
  const float* qchan;      // what their channels are multiplied by, K's and V's
  const float* ochan;
  const uint4* qsgn;       // sign masks of 8 samples, K's and V's
  const uint4* osgn;
  uint16_t* out;
  float* part;
  int4* desc;              // [CTA]: the cut unit that starts in it (request, row block, head, partials | slot << 16), 0: none
  long long q_ts, q_hs, table_stride;
  float qfac;
  int B, n_q, Hq, Hkv, Gq, max_q, max_kv, num_pages, page_shift, window, min_tiles;
};

__device__ __forceinline__ uint32_t ph2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 pu2h(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ float ppow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
// (a & mask) ^ x where x lies within mask or in bits that are zero in mask
__device__ __forceinline__ uint32_t mask_xor(uint32_t a, uint32_t mask, uint32_t x) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(mask), "r"(x));
  return d;
}
// Eight fp16 values with the signs flipped that the mask names.
__device__ __forceinline__ uint4 flip(uint4 v, uint4 m) { return make_uint4(v.x ^ m.x, v.y ^ m.y, v.z ^ m.z, v.w ^ m.w); }
// 32 channels in word_channel order times their factors (shared memory, natural order).
template <int BITS>
__device__ __forceinline__ void times_channels(float (&v)[32], const float* f) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(f + 4 * k);
    v[word_place(4 * k, BITS)] *= x.x;
    v[word_place(4 * k + 1, BITS)] *= x.y;
    v[word_place(4 * k + 2, BITS)] *= x.z;
    v[word_place(4 * k + 3, BITS)] *= x.w;
  }
}
// The exponent e with mx 2^-e in [2^14, 2^15), 0 for mx = 0.
__device__ __forceinline__ int row_exp(float mx) {
  const int e = (int)((__float_as_uint(mx) >> 23) & 255u) - 127 - 14;
  return mx > 0.0f ? min(max(e, -100), 100) : 0;
}

// ---------------------------------------------------------------- the line of tiles
template <int R, int T>
struct PrRequest {
  int qs, qn, kv, rows, nrt;
  __device__ __forceinline__ void load(const PromptParams& p, int b) {
    qs = b;
    qn = 1;
    if (p.q_starts) {
      qs = min(max(ld_fresh(p.q_starts + b), 0), p.n_q);
      qn = min(max(ld_fresh(p.q_starts + b + 1), qs), p.n_q) - qs;
    }
    kv = min(max(ld_fresh(p.kv_lens + b), 0), p.max_kv);
    rows = min(qn, p.max_q) * p.Gq;
    nrt = (rows + R - 1) / R;
  }
  // tokens [lo, hi) that some row of block rt attends, its first tile and its tiles (at least one)
  __device__ __forceinline__ void span(const PromptParams& p, int rt, int& lo, int& hi, int& tile0, int& nt) const {
    const int first = rt * R / p.Gq, last = (min((rt + 1) * R, rows) - 1) / p.Gq;
    hi = min(max(kv - qn + last + 1, 0), kv);
    lo = p.window ? (int)min((long long)hi, max((long long)kv - qn + first + 1 - p.window, 0ll)) : 0;
    tile0 = lo / T;
    nt = max(1, (hi + T - 1) / T - tile0);
  }
};

// A CTA's piece [at, end) of the line, walked segment by segment.
template <int R, int T>
struct PrWalk {
  long long at, end, base;  // base: the place of block (b, rt)'s first tile
  int b, rt;
  PrRequest<R, T> r;
  int lo, hi, tile0, nt;    // of block (b, rt)
  int h, i0, i1;            // the segment: head h, tiles [i0, i1) of the unit

  __device__ __forceinline__ void start(const PromptParams& p, int b_, long long base_) {
    b = b_;
    base = base_;
    rt = 0;
    r.load(p, b);
    if (r.nrt) r.span(p, 0, lo, hi, tile0, nt);
  }
  __device__ __forceinline__ bool next(const PromptParams& p) {
    if (at >= end) return false;
    while (rt >= r.nrt || at >= base + (long long)p.Hkv * nt) {
      if (rt < r.nrt) {
        base += (long long)p.Hkv * nt;
        ++rt;
      }
      while (rt >= r.nrt) {
        r.load(p, ++b);
        rt = 0;
      }
      r.span(p, rt, lo, hi, tile0, nt);
    }
    const long long off = at - base;
    h = (int)(off / nt);
    i0 = (int)(off - (long long)h * nt);
    i1 = (int)min((long long)nt, i0 + (end - at));
    at += i1 - i0;
    return true;
  }
};

// Sets the CTA's piece and where it starts; false when it is empty. `tot` holds kPrThreads values.
template <int R, int T>
__device__ __forceinline__ bool find_piece(const PromptParams& p, long long* tot, PrWalk<R, T>& w, long long& per) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ long long part[kPrWarps + 1];
  __shared__ long long found[2];
  long long total = 0, upto = 0, mine = 0;
  // the tiles of requests b0 .. b0 + kPrThreads - 1, a warp per request, then a scan over the block
  auto scan = [&](int b0, long long& sum) {
    for (int x = warp; x < kPrThreads; x += kPrWarps) {
      long long n = 0;
      if (b0 + x < p.B) {
        PrRequest<R, T> r;
        r.load(p, b0 + x);
        for (int rt = lane; rt < r.nrt; rt += 32) {
          int lo, hi, t0, nt;
          r.span(p, rt, lo, hi, t0, nt);
          n += nt;
        }
        if (r.nrt > 1) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) n += __shfl_xor_sync(0xffffffffu, n, off);
        }
      } else if (b0 + x >= p.B + kPrWarps) {
        break;
      }
      if (lane == 0) tot[x] = n * p.Hkv;
    }
    __syncthreads();
    mine = b0 + tid < p.B ? tot[tid] : 0;
    long long v = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long u = __shfl_up_sync(0xffffffffu, v, off);
      if (lane >= off) v += u;
    }
    if (lane == 31) part[warp] = v;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int x = 0; x < kPrWarps; ++x) {
      if (x < warp) v += part[x];
      sum += part[x];
    }
    __syncthreads();
    return v;
  };
  for (int b0 = 0; b0 < p.B; b0 += kPrThreads) {
    long long sum;
    upto = total + scan(b0, sum);
    total += sum;
  }
  per = max((long long)p.min_tiles, (total + gridDim.x - 1) / gridDim.x);
  w.at = min(total, per * blockIdx.x);
  w.end = min(total, w.at + per);
  if (w.at >= w.end) return false;
  if (p.B <= kPrThreads) {
    if (mine && w.at >= upto - mine && w.at < upto) {
      found[0] = upto - mine;
      found[1] = tid;
    }
  } else {
    long long before = 0;
    for (int b0 = 0; b0 < p.B && before <= w.at; b0 += kPrThreads) {
      long long sum;
      upto = before + scan(b0, sum);
      if (mine && w.at >= upto - mine && w.at < upto) {
        found[0] = upto - mine;
        found[1] = b0 + tid;
      }
      before += sum;
    }
  }
  __syncthreads();
  w.start(p, (int)found[1], found[0]);
  return true;
}

// ---------------------------------------------------------------- the kernel
template <int D, int G, int BITS>
__global__ void __launch_bounds__(kPrThreads, 1) attend_prompt_kernel(const __grid_constant__ PromptParams p) {
  using C = PrCfg<D, G, BITS>;
  constexpr int NQ = C::NQ, SB = C::SB, R = C::R, T = C::T, ND = C::ND, NW = C::NW, NJ = C::NJ;
  constexpr int NG = D / G, RB = D * BITS / 8;
  constexpr int kBlkQ = 128 * 128, kBlkT = T * 128;  // bytes of a 64-channel block of Q, of a tile
  extern __shared__ uint8_t smem_raw[];
  // an offset, not a rounded pointer: the compiler then knows every access below as shared memory
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* sQ = smem;
  uint8_t* sK = sQ + C::kQ;
  uint8_t* sV = sK + 2 * C::kTile;
  uint8_t* sRing = sV + 2 * C::kTile;
  uint32_t* sScale = reinterpret_cast<uint32_t*>(sRing + C::kRing);
  int32_t* sEnt = reinterpret_cast<int32_t*>(sRing + C::kRing + C::kScales);
  long long* scan = reinterpret_cast<long long*>(sK);  // before the first tile
  float* sQchan = reinterpret_cast<float*>(sRing + C::kRing + C::kScales + C::kEnt);
  float* sOchan = sQchan + D;
  uint4* sQsgn = reinterpret_cast<uint4*>(sOchan + D);
  uint4* sOsgn = sQsgn + D / 8;
  uint32_t* flags = reinterpret_cast<uint32_t*>(sOsgn + D / 8);  // [ring][5]
  uint64_t* kfull = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(flags) + C::kFlags);
  uint64_t* kempty = kfull + 2;
  uint64_t* vfull = kempty + 2;
  uint64_t* vempty = vfull + 2;
  uint64_t* aready = vempty + 2;  // [NQ] an A operand (raw query, q~, o) is in sQ
  uint64_t* sfull = aready + 2;   // [block or buffer] S (or a rotation's result) is in TMEM
  uint64_t* pfull = sfull + 2;    // [block or buffer][half] P is in TMEM
  uint64_t* odone = pfull + 4;    // [NQ] a P V product has been added
  uint64_t* mdone = odone + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  uint32_t* consts = tmem_slot + 1;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&kfull[s], ND);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], ND);
      mbar_init(&vempty[s], 1);
      mbar_init(&aready[s], 4);
      mbar_init(&sfull[s], 1);
      mbar_init(&pfull[2 * s], 4);
      mbar_init(&pfull[2 * s + 1], 4);
      mbar_init(&odone[s], 1);
    }
    mbar_init(mdone, 1);
    consts[0] = BITS == 4 ? 0x64086408u : 0x64806480u;  // 1032 (1152) as fp16 pairs
    consts[1] = 0x64806480u;                            // 1024 + 16 * 8
    fence_mbarrier_init();
  }
  for (int x = tid; x < kFlagRing * 5; x += kPrThreads) flags[x] = 0;
  // factors and signs, used at every unit (read from global memory there, with little L1 left beside
  // this shared memory: chunks of 2048 tokens 1034 us, so 1027)
  for (int x = tid; x < D; x += kPrThreads) {
    sQchan[x] = __ldg(p.qchan + x);
    sOchan[x] = __ldg(p.ochan + x);
    if (x < D / 8) {
      sQsgn[x] = __ldg(p.qsgn + x);
      sOsgn[x] = __ldg(p.osgn + x);
    }
  }
  grid_dep_launch();
  if (warp == kPrWarps - 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dep_wait();  // lengths, table, pages, queries and the workspace may come from the kernel before
  PrWalk<R, T> w;
  long long per;
  const bool any = find_piece<R, T>(p, scan, w, per);
  if (tid == 0) p.desc[blockIdx.x] = make_int4(0, 0, 0, 0);
  __syncthreads();  // the scan's place is free
  bool ok = true;  // false after a wait ran out: the role goes through its loops without work

  if (any && warp < 4 * NQ) {
    // ------------------------------------------------------------ softmax: a thread per query row
    const int qb = NQ == 2 ? warp >> 2 : 0;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = tl + C::kO + qb * D;
    const uint32_t trot = D == 128 ? tl + C::kS + qb * T : tl + C::kO;
    uint8_t* q_row = sQ + qb * (128 * D * 2) + row * 128;
    auto q_unit = [&](int u) {  // 16-byte unit u of this row
      return reinterpret_cast<uint4*>(q_row + (u >> 3) * kBlkQ + (((u & 7) ^ (row & 7)) << 4));
    };
    uint32_t ns[2] = {0, 0}, no = 0;  // phases of sfull, odone so far
    int kt = 0;                       // tiles so far (the flags' ring)
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(bar, ph))) {
        if (lane == 0) atomicOr(&g_prompt_err, kErrTimeoutLoad);
        ok = false;
      }
      tc_fence_after();
    };
    auto announce = [&](uint64_t* bar) {  // this warp's part of an operand in shared memory is written
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    while (w.next(p)) {
      const int n = w.i1 - w.i0;
      if (w.r.rows - w.rt * R <= 128 * qb) {  // no rows for this block
        kt += n;
        continue;
      }
      const int y = w.rt * R + qb * 128 + row;
      const bool valid = y < w.r.rows;
      const int tok = y / p.Gq, head = w.h * p.Gq + (y - tok * p.Gq);
      // ---- the raw query
      {
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(w.r.qs + tok) * p.q_ts + (long long)head * p.q_hs);
#pragma unroll 8
        for (int u = 0; u < D / 8; ++u) *q_unit(u) = valid ? flip(ld_fresh(src + u), sQsgn[u]) : make_uint4(0, 0, 0, 0);
      }
      announce(&aready[qb]);
      // ---- q~, normalised by a power of two per row
      const int s0 = NQ == 2 ? qb : 0;
      wait(&sfull[s0], ns[s0]++ & 1);
      float fac;
      {
        float mx = 0.0f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(trot + c, v);
          tmem_ld_wait();
          tmem_regs_fence(v);
          times_channels<BITS>(v, sQchan + c);
#pragma unroll
          for (int k = 0; k < 32; ++k) mx = fmaxf(mx, fabsf(v[k]));
        }
        const int ex = row_exp(mx);
        const float f = ppow2(-ex);
        fac = p.qfac * ppow2(ex);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(trot + c, v);
          tmem_ld_wait();
          tmem_regs_fence(v);
          times_channels<BITS>(v, sQchan + c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *q_unit(c / 8 + k) = make_uint4(pack_half2(v[8 * k] * f, v[8 * k + 1] * f), pack_half2(v[8 * k + 2] * f, v[8 * k + 3] * f),
                                            pack_half2(v[8 * k + 4] * f, v[8 * k + 5] * f), pack_half2(v[8 * k + 6] * f, v[8 * k + 7] * f));
        }
      }
      announce(&aready[qb]);
      // what this row attends: tokens in (lo, hi]; all rows of the warp attend those in (wlo, whi]
      const int hi = valid ? w.r.kv - w.r.qn + tok : 0x7fffffff;
      const int lo = valid && p.window ? (int)max((long long)hi - p.window, -1ll) : -1;
      const int whi = __reduce_min_sync(0xffffffffu, hi), wlo = __reduce_max_sync(0xffffffffu, lo);
      float m_run = -INFINITY, l_run = 0.0f;
      int ve = 0;          // O is held divided by 2^ve, as V of the tile last added to it
      bool row_nan = false;
      for (int i = 0; i < n; ++i, ++kt) {
        const int idx = NQ == 2 ? qb : (i & 1);
        const uint32_t ts = tl + C::kS + idx * T;
        wait(&sfull[idx], ns[idx]++ & 1);
        if (!ok) continue;
        const int t0 = (w.tile0 + w.i0 + i) * T;
        const bool cut = t0 + T - 1 > whi || t0 <= wlo;
        volatile uint32_t* fl = flags + (kt % kFlagRing) * 5;
        const uint32_t flag = fl[0];
        const float f = (flag & 1) ? fac * 256.0f : fac;
        // The row's maximum. S comes 32 columns at a time, the next ones on their way while these
        // are used; tiles with masked places take a plain loop of their own.
        float mx = -INFINITY;
        auto row_max = [&](const float (&x)[32]) {
#pragma unroll
          for (int k = 0; k < 32; k += 2) mx = fmaxf(mx, fmaxf(x[k], x[k + 1]));
        };
        auto mask = [&](int c, float (&x)[32]) {
#pragma unroll
          for (int k = 0; k < 32; ++k)
            if (t0 + c + k > hi || t0 + c + k <= lo) x[k] = -INFINITY;
        };
        if (cut) {
#pragma unroll 1
          for (int c = 0; c < T; c += 32) {
            float v[32];
            tmem_ld32_now(ts + c, v);
            mask(c, v);
            row_max(v);
          }
        } else {
          float v[T / 32][32];
          tmem_ld32(ts, v[0]);
#pragma unroll
          for (int c = 0; c < T / 32; ++c) {
            tmem_ld_wait();
            tmem_regs_fence(v[c]);
            if (c + 1 < T / 32) tmem_ld32(ts + 32 * (c + 1), v[c + 1 < T / 32 ? c + 1 : c]);
            row_max(v[c]);
          }
        }
        mx *= f;
        // the product before this tile's: every phase of odone is waited for, or a parity could
        // stand for the phase before (with one S buffer, S of this tile came after that product)
        if (SB == 2 && i > 0) wait(&odone[qb], (no + i - 1) & 1);
        const int nve = (flag & 2) ? 8 : 0;
        constexpr float kSlack = 8.0f;
        if (__any_sync(0xffffffffu, mx > m_run + kSlack) || nve != ve) {
          const float m = fmaxf(m_run, mx);
          float g = m == m_run ? 1.0f : ex2_approx(m_run - m);
          l_run *= g;
          if (i > 0) {
            if (nve != ve) g *= nve ? 1.0f / 256.0f : 256.0f;  // exact, and O has fp32's range
            if (SB == 1) wait(&odone[qb], (no + i - 1) & 1);
            if (!ok) continue;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float v[32];
              tmem_ld32(to + c, v);
              tmem_ld_wait();
              tmem_regs_fence(v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] *= g;
              tmem_st32(to + c, v);
            }
          }
          m_run = m;
          ve = nve;
        }
        if (flag & 4) {  // some V scales of the tile are not finite
          for (int t = 0; t < T; ++t)
            if (((fl[1 + (t >> 5)] >> (t & 31)) & 1) && t0 + t <= hi && t0 + t > lo) row_nan = true;
        }
        // P, in two halves: the product starts on the first while the second is made
        // (times 2^kPTop, as l and O then are: with the slack 2^15, within fp16)
        constexpr float kPTop = 15.0f - kSlack;
        const float ms = m_run == -INFINITY ? 0.0f : m_run - kPTop;
        float l0 = 0.0f, l1 = 0.0f;
        auto weights = [&](int c, const float (&x)[32]) {
          uint32_t h[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float a = ex2_approx(fmaf(x[2 * k], f, -ms)), b = ex2_approx(fmaf(x[2 * k + 1], f, -ms));
            l0 += a;
            l1 += b;
            h[k] = pack_half2(a, b);
          }
          tmem_st16(ts + c / 2, h);  // over columns of S that have been read
          if (c + 32 == T / 2 || c + 32 == T) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            // a barrier per half: a warp may be at its second while another is at its first
            if (lane == 0) mbar_arrive(&pfull[2 * idx + (c + 32 == T)]);
          }
        };
        if (cut) {
#pragma unroll 1
          for (int c = 0; c < T; c += 32) {
            float v[32];
            tmem_ld32_now(ts + c, v);
            mask(c, v);
            weights(c, v);
          }
        } else {
          float v[T / 32][32];
          tmem_ld32(ts, v[0]);
#pragma unroll
          for (int c = 0; c < T / 32; ++c) {
            tmem_ld_wait();
            tmem_regs_fence(v[c]);
            if (c + 1 < T / 32) tmem_ld32(ts + 32 * (c + 1), v[c + 1 < T / 32 ? c + 1 : c]);
            weights(32 * c, v[c]);
          }
        }
        l_run += l0 + l1;
      }
      wait(&odone[qb], (no + n - 1) & 1);
      no += n;
      if (row_nan) l_run = __int_as_float(0x7fc00000);
      if (w.i0 == 0 && w.i1 == w.nt) {
        // ---- out = Wo (o / l), o normalised like q~
        const float inv = l_run > 0.0f || l_run != l_run ? 1.0f / l_run : 0.0f;  // nothing attended: zeros (NaN stays)
        float mx = 0.0f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(to + c, v);
          tmem_ld_wait();
          tmem_regs_fence(v);
          times_channels<BITS>(v, sOchan + c);
#pragma unroll
          for (int k = 0; k < 32; ++k) mx = fmaxf(mx, fabsf(v[k]));
        }
        const int ex = row_exp(mx * inv);
        const float f = inv * ppow2(-ex);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(to + c, v);
          tmem_ld_wait();
          tmem_regs_fence(v);
          times_channels<BITS>(v, sOchan + c);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *q_unit(c / 8 + k) = make_uint4(pack_half2(v[8 * k] * f, v[8 * k + 1] * f), pack_half2(v[8 * k + 2] * f, v[8 * k + 3] * f),
                                            pack_half2(v[8 * k + 4] * f, v[8 * k + 5] * f), pack_half2(v[8 * k + 6] * f, v[8 * k + 7] * f));
        }
        announce(&aready[qb]);
        wait(&sfull[s0], ns[s0]++ & 1);
        const float of = ppow2(ex) * ppow2(ve);
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)(w.r.qs + tok) * p.Hq + head) * D);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(trot + c, v);
          tmem_ld_wait();
          tmem_regs_fence(v);
          if (valid && ok) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[c / 8 + k] = flip(make_uint4(pack_half2(v[8 * k] * of, v[8 * k + 1] * of), pack_half2(v[8 * k + 2] * of, v[8 * k + 3] * of),
                                               pack_half2(v[8 * k + 4] * of, v[8 * k + 5] * of), pack_half2(v[8 * k + 6] * of, v[8 * k + 7] * of)),
                                    sOsgn[c / 8 + k]);
          }
        }
      } else {
        // ---- a partial of a unit that other CTAs share: [m][l][4 channels][row]
        const long long u0 = w.base + (long long)w.h * w.nt;
        const long long x0 = (long long)blockIdx.x * per;
        float* dst = p.part + (2 * (long long)blockIdx.x + (x0 >= u0 ? 0 : 1)) * kPrPart;
        const int pr = qb * 128 + row;
        dst[pr] = m_run;
        dst[R + pr] = l_run;
        const float vf = ppow2(ve);
        float4* od = reinterpret_cast<float4*>(dst + 2 * R) + pr;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float v[32];
          tmem_ld32(to + c, v);
          tmem_ld_wait();
          tmem_regs_fence(v);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            od[(size_t)(c / 4 + k) * R] = make_float4(v[4 * k] * vf, v[4 * k + 1] * vf, v[4 * k + 2] * vf, v[4 * k + 3] * vf);
        }
        const long long xa = u0 / per, xb = (u0 + w.nt - 1) / per;
        if (tid == 0 && xa == blockIdx.x) p.desc[blockIdx.x] = make_int4(w.b, w.rt, w.h, (int)(xb - xa + 1) | (x0 >= u0 ? 0 : 1 << 16));
      }
    }
  } else if (any && warp < kPrWarps - 1) {
    // ------------------------------------------------------------ dequantisers
    const int dw = warp - 4 * NQ, dtid = dw * 32 + lane;
    const int P1 = (1 << p.page_shift) - 1;
    int kc = 0, vc = 0, kt = 0;  // ring tiles so far (K with the matrices, V), tiles so far
    auto wait = [&](uint64_t* bar, int count) {  // until ring tile `count` may be written
      if (count >= 2 && ok && !__all_sync(0xffffffffu, mbar_wait_bounded(&bar[count & 1], ((count >> 1) - 1) & 1))) {
        if (lane == 0) atomicOr(&g_prompt_err, kErrTimeoutLoad);
        ok = false;
      }
    };
    auto announce = [&](uint64_t* bar) {
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    auto matrix = [&](const uint16_t* m) {  // a rotation matrix [D][D] through the K ring
#pragma unroll 1
      for (int t = 0; t < NW; ++t, ++kc) {
        wait(kempty, kc);
        uint8_t* dst = sK + (kc & 1) * C::kTile;
        const uint4* src = reinterpret_cast<const uint4*>(m + (size_t)t * T * D);
#pragma unroll 8
        for (int x = dtid; x < T * (D / 8); x += ND * 32) {
          const int r = x / (D / 8), u = x - r * (D / 8);
          *reinterpret_cast<uint4*>(dst + (u >> 3) * kBlkT + r * 128 + (((u & 7) ^ (r & 7)) << 4)) = __ldg(src + x);
        }
        announce(&kfull[kc & 1]);
      }
    };
    // read, not written out: an instruction holds one constant, the mask
    const uint32_t x1 = *reinterpret_cast<volatile uint32_t*>(consts), x16 = *reinterpret_cast<volatile uint32_t*>(consts + 1);
    // item j of this thread: row it_row(j) of a tile, 32 channels from 32 it_chunk(j)
    auto it_row = [&](int j) { return ((dw + ND * j) % (T / 8)) * 8 + (lane & 7); };
    auto it_chunk = [&](int j) { return ((dw + ND * j) / (T / 8)) * 4 + (lane >> 3); };
    struct Item {
      uint32_t c[C::CW];
      uint32_t s;  // the item's scale (G = 32) or two scales
    };
    // item j's codes as fp16 into a tile
    auto convert = [&](uint8_t* tile, int j, const Item& it, bool big) {
      const int r = it_row(j), ch = it_chunk(j);
      uint8_t* dst = tile + (ch >> 1) * kBlkT + r * 128;
      __half2 s0 = pu2h(prmt(it.s, it.s, 0x1010)), s1 = G == 32 ? s0 : pu2h(prmt(it.s, it.s, 0x3232));
      if (big) {
        const __half2 d = __half2half2(__ushort_as_half((unsigned short)0x1c00));  // 2^-8
        s0 = __hmul2(s0, d);
        s1 = __hmul2(s1, d);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 s = k < 2 ? s0 : s1;
        uint4 o;
        if constexpr (BITS == 4) {
          const uint32_t x = it.c[k], x8 = x >> 8;
          const __half2 o1 = pu2h(0x64086408u), o16 = pu2h(0xD480D480u), i16 = pu2h(0x2C002C00u);  // 1032, -72, 1/16
          o.x = ph2u(__hmul2(__hsub2(pu2h(mask_xor(x, 0x000F000Fu, x1)), o1), s));
          o.y = ph2u(__hmul2(__hfma2(pu2h(mask_xor(x, 0x00F000F0u, x16)), i16, o16), s));
          o.z = ph2u(__hmul2(__hsub2(pu2h(mask_xor(x8, 0x000F000Fu, x1)), o1), s));
          o.w = ph2u(__hmul2(__hfma2(pu2h(mask_xor(x8, 0x00F000F0u, x16)), i16, o16), s));
        } else {
          const __half2 o1 = pu2h(0x64806480u);  // 1152
          const uint32_t a = it.c[2 * k], b = it.c[2 * k + 1];
          o.x = ph2u(__hmul2(__hsub2(pu2h(mask_xor(a, 0x00FF00FFu, x1)), o1), s));
          o.y = ph2u(__hmul2(__hsub2(pu2h(mask_xor(a >> 8, 0x00FF00FFu, x1)), o1), s));
          o.z = ph2u(__hmul2(__hsub2(pu2h(mask_xor(b, 0x00FF00FFu, x1)), o1), s));
          o.w = ph2u(__hmul2(__hsub2(pu2h(mask_xor(b >> 8, 0x00FF00FFu, x1)), o1), s));
        }
        *reinterpret_cast<uint4*>(dst + ((((ch & 1) * 4 + k) ^ (r & 7)) << 4)) = o;
      }
    };
    // What a thread converts it fetches itself, by async copies: an arrival at a barrier would
    // wait for loads in flight, not for these. Half h (four per tile: K, K, V, V) goes to ring
    // slot h % NS and is issued NS - 1 halves ahead; the scales of tile i + 1 and the table
    // entries of tile i + 2 go with tile i's first half.
    constexpr int NS = C::NS, HJ = NJ / 2, NT = ND * 32;
    uint8_t* ring = sRing + dtid * 16;
    uint32_t* scale_s = sScale + dtid;
    int32_t* ent_s = sEnt + dtid;
    auto copy16 = [&](uint8_t* dst, const uint8_t* src, bool in) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0) : "memory");
    };
    auto copy4 = [&](void* dst, const void* src, bool in) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 4 : 0) : "memory");
    };
    auto commit = [] { asm volatile("cp.async.commit_group;" ::: "memory"); };
    while (w.next(p)) {
      const int n = w.i1 - w.i0;
      const int32_t* trow = p.table + (long long)w.b * p.table_stride;
      const int t_first = (w.tile0 + w.i0) * T;
      const int t_hi = w.hi, t_lo = w.lo;
      // item j of tile i: its token, and whether the unit attends it
      auto token = [&](int i, int j) { return t_first + i * T + it_row(j); };
      auto live = [&](int i, int j) {
        const int t = token(i, j);
        return i < n && t >= t_lo && t < t_hi;
      };
      auto cache_row = [&](int i, int j, int e) -> long long {  // e: its table entry; -1 where there is no token
        if (!live(i, j)) return -1;
        if (e < 0 || e >= p.num_pages) {
          atomicOr(&g_prompt_err, kErrBadPage);
          e = 0;
        }
        return (((long long)e * p.Hkv + w.h) << p.page_shift) + (token(i, j) & P1);
      };
      long long rows[2][NJ];  // of this tile and the next
      auto fetch_entries = [&](int i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const bool in = live(i, j);
          copy4(ent_s + j * NT, trow + (in ? token(i, j) >> p.page_shift : 0), in);
        }
      };
      auto take_entries = [&](int i, long long (&r)[NJ]) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) r[j] = cache_row(i, j, ent_s[j * NT]);
      };
      auto fetch_scales = [&](const long long (&r)[NJ]) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const long long at = max(r[j], 0ll) * NG + (G == 32 ? it_chunk(j) & ~1 : 2 * it_chunk(j));
          copy4(scale_s + (2 * j) * NT, p.ks + at, r[j] >= 0);
          copy4(scale_s + (2 * j + 1) * NT, p.vs + at, r[j] >= 0);
        }
      };
      auto fetch_half = [&](int isv, int half, bool next, int to) {  // into ring slot `to`
        const uint8_t* base = isv ? p.vc : p.kc;
        uint8_t* dst = ring + to * C::kHalf;
#pragma unroll
        for (int x = 0; x < HJ; ++x) {
          const int j = half * HJ + x;
          const long long row = next ? rows[1][j] : rows[0][j];
#pragma unroll
          for (int y = 0; y < C::CW / 4; ++y)
            copy16(dst + (x * (C::CW / 4) + y) * NT * 16, base + max(row, 0ll) * RB + it_chunk(j) * (4 * BITS) + 16 * y, row >= 0);
        }
      };
      // the start: entries of tiles 0 and 1, scales of tile 0, the first halves
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        rows[0][j] = cache_row(0, j, live(0, j) ? ld_fresh(trow + (token(0, j) >> p.page_shift)) : -1);
        rows[1][j] = -1;
      }
      fetch_entries(1);
      fetch_scales(rows[0]);
      commit();
      matrix(p.wq);
      // halves 0 .. NS - 2, a group each
#pragma unroll
      for (int h = 0; h < NS - 1; ++h) {
        fetch_half(h >> 1, h & 1, false, h);
        commit();
      }
      int slot = 0;  // of the ring
      asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
      for (int i = 0; i < n; ++i, ++kt, ++kc, ++vc) {
        uint32_t ksc[NJ], vsc[NJ];
        // ---- half 4 i: this tile's scales and the next one's entries are here (their group is
        // older than the halves in flight)
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          ksc[j] = scale_s[(2 * j) * NT];
          vsc[j] = scale_s[(2 * j + 1) * NT];
          if (G == 32) {
            ksc[j] = (it_chunk(j) & 1) ? ksc[j] >> 16 : ksc[j] & 0xFFFFu;
            vsc[j] = (it_chunk(j) & 1) ? vsc[j] >> 16 : vsc[j] & 0xFFFFu;
          }
        }
        take_entries(i + 1, rows[1]);
        fetch_scales(rows[1]);
        fetch_entries(i + 2);
        // ---- scales that need care: bit 0 large K, bit 1 large V, bit 2 V not finite
        uint32_t* fl = flags + (kt % kFlagRing) * 5;
        {
          constexpr uint32_t kBig = BITS == 4 ? 0x6C00u : 0x6000u;  // 2^12, 2^9
          uint32_t kx = 0, vx = 0;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const uint32_t a = ksc[j] & 0x7FFF7FFFu, b = vsc[j] & 0x7FFF7FFFu;
            kx = max(kx, max(a & 0xFFFFu, a >> 16));
            vx = max(vx, max(b & 0xFFFFu, b >> 16));
          }
          if (max(kx, vx) >= kBig) {
            uint32_t odd = 0;
            if (max(kx, vx) >= 0x7C00u) {  // scales that are not finite are taken out of the maxima
              auto not_finite = [](uint32_t s) { return (s & 0x7C00u) == 0x7C00u || (s & 0x7C000000u) == 0x7C000000u; };
              kx = vx = 0;
#pragma unroll
              for (int j = 0; j < NJ; ++j) {
                // an infinite K scale becomes NaN: its score may be -inf, the mark of a masked place
                if (not_finite(ksc[j])) ksc[j] = 0x7FFF7FFFu;
                else kx = max(kx, max(ksc[j] & 0x7FFFu, (ksc[j] >> 16) & 0x7FFFu));
                if (not_finite(vsc[j])) {
                  vsc[j] = 0;
                  odd = 4u;
                  atomicOr(&fl[1 + (it_row(j) >> 5)], 1u << (it_row(j) & 31));
                }
                vx = max(vx, max(vsc[j] & 0x7FFFu, (vsc[j] >> 16) & 0x7FFFu));
              }
            }
            atomicOr(&fl[0], (kx >= kBig ? 1u : 0u) | (vx >= kBig ? 2u : 0u) | odd);
          }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(ND * 32) : "memory");
        const uint32_t flag = *reinterpret_cast<volatile uint32_t*>(fl);
        if (dtid < 5) flags[((kt + kFlagRing / 2) % kFlagRing) * 5 + dtid] = 0;  // last read four tiles ago
        // K, then V. Rolled, and softmax' loops as well: the roles' loops together have to stay
        // within the instruction caches.
#pragma unroll 1
        for (int isv = 0; isv < 2; ++isv) {
          uint8_t* tile = isv ? sV + (vc & 1) * C::kTile : sK + (kc & 1) * C::kTile;
          const bool big = flag & (isv ? 2u : 1u);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // this half has landed; the one NS - 1 after it goes to the slot that the half before left
            asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
            Item it[HJ];
#pragma unroll
            for (int x = 0; x < HJ; ++x) {
#pragma unroll
              for (int y = 0; y < C::CW / 4; ++y) {
                const uint4 v = *reinterpret_cast<const uint4*>(ring + slot * C::kHalf + (x * (C::CW / 4) + y) * NT * 16);
                it[x].c[4 * y] = v.x;
                it[x].c[4 * y + 1] = v.y;
                it[x].c[4 * y + 2] = v.z;
                it[x].c[4 * y + 3] = v.w;
              }
              it[x].s = isv ? vsc[half * HJ + x] : ksc[half * HJ + x];
            }
            constexpr int kAhead = NS - 1;
            const int ops = (half + kAhead) / 2;  // operands ahead: 1 or 2, known at compile time
            fetch_half((isv + ops) & 1, (half + kAhead) & 1, ops == 2 || isv, slot == 0 ? NS - 1 : slot - 1);
            commit();
            if (half == 0) wait(isv ? vempty : kempty, isv ? vc : kc);
#pragma unroll
            for (int x = 0; x < HJ; ++x) convert(tile, half * HJ + x, it[x], big);
            if (half == 1) announce(isv ? &vfull[vc & 1] : &kfull[kc & 1]);
            slot = slot + 1 == NS ? 0 : slot + 1;
          }
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j) rows[0][j] = rows[1][j];
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (w.i0 == 0 && w.i1 == w.nt) matrix(p.wo);
    }
  } else if (any) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp walks and waits, an elected lane issues each batch of eight products:
    // the operands' descriptors stay in the warp's uniform registers. (One lane doing all of
    // it took 106 cycles per product, most of them to move descriptors there; a product itself
    // takes 64.)
    constexpr uint32_t id_s = umma_idesc_f16(128, T), id_o = umma_idesc_f16(128, D) | kUmmaTransposeB;
    const uint32_t q_lo = (uint32_t)umma_desc_sw128(smem_u32(sQ)), k_lo = (uint32_t)umma_desc_sw128(smem_u32(sK));
    const uint32_t v_lo = (uint32_t)umma_desc_mn_sw128(smem_u32(sV), kBlkT);
    constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // bits 32 .. 63 of all three
    int kc = 0, vc = 0;
    uint32_t na[2] = {0, 0}, np[2] = {0, 0};
    auto wait = [&](uint64_t* bar, uint32_t ph) {
      if (ok && !__all_sync(0xffffffffu, mbar_wait_bounded(bar, ph))) {
        if (lane == 0) atomicOr(&g_prompt_err, kErrTimeoutLoad);
        ok = false;
      }
      tc_fence_after();
      return ok;
    };
    // columns d = A block q of sQ times the K ring's tile; then arrivals at `done` (and `done2`)
    auto product = [&](uint32_t d, int q, int slot, uint64_t* done, uint64_t* done2) {
      const uint32_t a = q_lo + (uint32_t)(q * (128 * D * 2) >> 4), b = k_lo + (uint32_t)(slot * C::kTile >> 4);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          umma_f16_lo(d, a + (((ks >> 2) * kBlkQ + (ks & 3) * 32) >> 4), b + (((ks >> 2) * kBlkT + (ks & 3) * 32) >> 4), kHi, id_s,
                      ks > 0);
        if (done) umma_commit(done);
        if (done2) umma_commit(done2);
      }
      __syncwarp();
    };
    while (w.next(p)) {
      const int n = w.i1 - w.i0;
      const int nq = NQ == 2 && w.r.rows - w.rt * R > 128 ? 2 : 1;
      auto rotate = [&]() {  // the A operands times a rotation matrix
        for (int q = 0; q < nq; ++q) wait(&aready[q], na[q]++ & 1);
        for (int t = 0; t < NW; ++t, ++kc) {
          if (!wait(&kfull[kc & 1], (kc >> 1) & 1)) continue;
          for (int q = 0; q < nq; ++q)
            product(tmem + (D == 128 ? C::kS + q * T : C::kO + t * T), q, kc & 1, t == NW - 1 ? &sfull[NQ == 2 ? q : 0] : nullptr,
                    q == nq - 1 ? &kempty[kc & 1] : nullptr);
        }
      };
      rotate();
      for (int q = 0; q < nq; ++q) wait(&aready[q], na[q]++ & 1);
      for (int s = 0; s < SB && s < n; ++s, ++kc) {
        if (!wait(&kfull[kc & 1], (kc >> 1) & 1)) continue;
        for (int q = 0; q < nq; ++q)
          product(tmem + C::kS + (NQ == 2 ? q : s) * T, q, kc & 1, &sfull[NQ == 2 ? q : s], q == nq - 1 ? &kempty[kc & 1] : nullptr);
      }
      for (int i = 0; i < n; ++i, ++vc) {
        const bool more = i + SB < n;
        wait(&vfull[vc & 1], (vc >> 1) & 1);
        const uint32_t vb = v_lo + (uint32_t)((vc & 1) * C::kTile >> 4);
        for (int q = 0; q < nq; ++q) {
          const int idx = NQ == 2 ? q : (i & 1);
          const uint32_t ts = tmem + C::kS + idx * T;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!wait(&pfull[2 * idx + half], np[idx] & 1)) continue;
            if (elect_one()) {
#pragma unroll
              for (int kk = half * (T / 32); kk < (half + 1) * (T / 32); ++kk)
                umma_f16_ts_lo(tmem + C::kO + q * D, ts + 8 * kk, vb + (kk * 2048 >> 4), kHi, id_o, i > 0 || kk > 0);
              if (half) umma_commit(&odone[q]);
              if (half && q == nq - 1) umma_commit(&vempty[vc & 1]);
            }
            __syncwarp();
          }
          ++np[idx];
          if (more) {
            if (q == 0) wait(&kfull[kc & 1], (kc >> 1) & 1);
            if (ok) product(ts, q, kc & 1, &sfull[idx], q == nq - 1 ? &kempty[kc & 1] : nullptr);
          }
        }
        if (more) ++kc;
      }
      if (w.i0 == 0 && w.i1 == w.nt) rotate();
    }
    if (elect_one()) umma_commit(mdone);
    if (!mbar_wait_bounded(mdone, 0)) atomicOr(&g_prompt_err, kErrTimeoutLoad);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPrWarps - 1) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- the join
// Block (x, y): rows 8y .. 8y + 7 of the cut unit whose first CTA is x: the partials in CTA
// order, then out = Wo (o / l) with o as an fp16 hi + lo pair. Reading the partials bounds it.
constexpr int kJoinWarps = 4;

template <int D, int BITS>
__global__ void __launch_bounds__(kJoinWarps * 32) join_prompt_kernel(const __grid_constant__ PromptParams p) {
  constexpr int R = 32768 / D, T = D == 128 ? 128 : 64, MT = D / 16, ST = D + 4;
  __shared__ __align__(16) float om[8 * ST];
  __shared__ __align__(16) __half ob[8 * (D + 8)];
  __shared__ float ml[2][8];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint4 sgn = __ldg(p.osgn + tid % (D / 8));  // of this thread's 8 samples of every row
  grid_dep_launch();
  grid_dep_wait();
  const int4 u = ld_fresh(p.desc + blockIdx.x);
  if (u.w == 0) return;
  PrRequest<R, T> r;
  r.load(p, u.x);
  const int r0 = 8 * (int)blockIdx.y, nrows = min(8, min(R, r.rows - u.y * R) - r0);
  if (nrows <= 0) return;
  // the unit's first CTA holds it in slot 1 unless the unit starts its piece; the others in slot 0
  const float* first = p.part + (2 * (long long)blockIdx.x) * kPrPart;
  const int np = u.w & 0xFFFF, first_slot = u.w >> 16;
  auto slot = [&](int k) { return k == 0 ? first + first_slot * kPrPart : first + 2 * (long long)k * kPrPart; };
  if (tid < 8) {
    float M = -INFINITY, L = 0.0f;
    for (int k = 0; k < np; ++k) M = fmaxf(M, __ldcg(slot(k) + r0 + tid));
    for (int k = 0; k < np; ++k) {
      const float m = __ldcg(slot(k) + r0 + tid), l = __ldcg(slot(k) + R + r0 + tid);
      if (m != -INFINITY) L = fmaf(l, ex2_approx(m - M), L);
      else L += l;  // 0, or NaN for a row that attends a value that is no number
    }
    ml[0][tid] = M;
    ml[1][tid] = L;
  }
  __syncthreads();
  for (int x = tid; x < 8 * (D / 4); x += kJoinWarps * 32) {
    const int row = x & 7, k4 = x >> 3;
    const float M = ml[0][row];
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 8;  // partials in flight
    for (int k0 = 0; k0 < np; k0 += U) {
      float4 v[U];
      float m[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (k0 + k < np) {
          m[k] = __ldcg(slot(k0 + k) + r0 + row);
          v[k] = __ldcg(reinterpret_cast<const float4*>(slot(k0 + k) + 2 * R) + (size_t)k4 * R + r0 + row);
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (k0 + k < np && m[k] != -INFINITY) {
          const float f = ex2_approx(m[k] - M);
          acc.x = fmaf(f, v[k].x, acc.x);
          acc.y = fmaf(f, v[k].y, acc.y);
          acc.z = fmaf(f, v[k].z, acc.z);
          acc.w = fmaf(f, v[k].w, acc.w);
        }
      }
    }
    float* o = om + row * ST;
    const float a[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = word_channel(4 * k4 + k, BITS);
      o[ch] = a[k] * __ldg(p.ochan + ch);
    }
  }
  __syncthreads();
  const int g = lane >> 2, c = lane & 3;
  const float L = ml[1][g];
  const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
  const float* orow = om + g * ST;
  float mx = 0.0f;
#pragma unroll
  for (int x = 0; x < D / 16; ++x) {
    const float4 v = *reinterpret_cast<const float4*>(orow + 16 * x + 4 * c);
    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  const int ex = row_exp(mx * inv);
  const float f = inv * ppow2(-ex);
  float acc[MT / kJoinWarps][4] = {};
#pragma unroll
  for (int ks = 0; ks < MT; ++ks) {
    uint32_t bh[2], bl[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 v = *reinterpret_cast<const float2*>(orow + 16 * ks + 8 * e + 2 * c);
      const __half2 hv = __floats2half2_rn(v.x * f, v.y * f);
      const float2 hf = __half22float2(hv);
      bh[e] = ph2u(hv);
      bl[e] = pack_half2(v.x * f - hf.x, v.y * f - hf.y);
    }
#pragma unroll
    for (int t = 0; t < MT / kJoinWarps; ++t) {
      const uint4 a = __ldg(p.wof + ((warp + kJoinWarps * t) * MT + ks) * 32 + lane);
      mma_16816(acc[t], a.x, a.y, a.z, a.w, bh[0], bh[1]);
      mma_16816(acc[t], a.x, a.y, a.z, a.w, bl[0], bl[1]);
    }
  }
  float fo[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) fo[e] = ppow2(__shfl_sync(0xffffffffu, ex, 4 * (2 * c + e)));
#pragma unroll
  for (int t = 0; t < MT / kJoinWarps; ++t) {
    __half* x0 = ob + (2 * c) * (D + 8) + 16 * (warp + kJoinWarps * t) + g;
    x0[0] = __float2half_rn(acc[t][0] * fo[0]);
    x0[D + 8] = __float2half_rn(acc[t][1] * fo[1]);
    x0[8] = __float2half_rn(acc[t][2] * fo[0]);
    x0[D + 8 + 8] = __float2half_rn(acc[t][3] * fo[1]);
  }
  __syncthreads();
  for (int x = tid; x < nrows * (D / 8); x += kJoinWarps * 32) {
    const int row = x / (D / 8), k = x - row * (D / 8);
    const int y = u.y * R + r0 + row, tok = y / p.Gq, head = u.z * p.Gq + (y - tok * p.Gq);
    *(reinterpret_cast<uint4*>(p.out + ((size_t)(r.qs + tok) * p.Hq + head) * D) + k) =
        flip(*reinterpret_cast<const uint4*>(ob + row * (D + 8) + 8 * k), sgn);
  }
}

// ---------------------------------------------------------------- host side
template <int D, int G, int BITS>
kvq_status run_prompt(const PagedAttendHost& a, void* part, cudaStream_t strm) {
  using C = PrCfg<D, G, BITS>;
  PromptParams p{};
  p.q = a.q;
  p.kc = a.kc;
  p.ks = a.ks;
  p.vc = a.vc;
  p.vs = a.vs;
  p.table = a.table ? a.table : a.kv_lens;  // no pages: an address for copies of zero bytes
  p.kv_lens = a.kv_lens;
  p.q_starts = a.q_starts;
  p.wq = a.pk->basis->wq_dev;
  p.wo = a.pv->basis->wo_dev;
  p.wof = a.pv->basis->wof_dev;
  p.qchan = a.pk->dec_dev->chan;
  p.ochan = a.pv->dec_dev->chan;
  p.qsgn = reinterpret_cast<const uint4*>(a.pk->dec_dev->sgn);
  p.osgn = reinterpret_cast<const uint4*>(a.pv->dec_dev->sgn);
  p.out = a.out;
  p.part = reinterpret_cast<float*>(part);
  p.desc = reinterpret_cast<int4*>(p.part + (size_t)2 * kPrMaxCtas * kPrPart);
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
  p.max_kv = (int)std::min<long long>(a.max_kv_len, (long long)a.max_pages << a.page_shift);
  p.num_pages = a.num_pages;
  p.page_shift = a.page_shift;
  p.window = a.window;
  const double attended = a.window ? std::min<double>(p.max_kv, (double)a.window + std::min(a.max_q_len, a.n_q)) : p.max_kv;  // tokens of a unit
  // A piece of t tiles takes about 2.6 t us, joining a unit's n / t pieces about 0.4 n / t:
  // t = sqrt(0.15 n) is best where there are CTAs to spare (one KV head of 256, 16K tokens,
  // at 64 query tokens 90 us with pieces of 2, 60 with 6).
  p.min_tiles = std::max(2, (int)std::sqrt(0.15 * attended / C::T));
  const long long blocks = ((long long)std::min(a.max_q_len, a.n_q) * p.Gq + C::R - 1) / C::R;
  const long long most = (long long)a.B * a.Hkv * blocks * std::max(1, (p.max_kv + C::T - 1) / C::T);
  const int sms = std::min(kPrMaxCtas, num_sms(a.pk->device));
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<long long>(sms, (most + p.min_tiles - 1) / p.min_tiles));
  cfg.blockDim = dim3(kPrThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = strm;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = allow_smem<attend_prompt_kernel<D, G, BITS>>(a.pk->device, C::kSmem);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, attend_prompt_kernel<D, G, BITS>, p);
  if (e == cudaSuccess) {
    const int rows = std::min<long long>(C::R, (long long)std::min(a.max_q_len, a.n_q) * p.Gq);
    cfg.gridDim.y = (unsigned)((rows + 7) / 8);
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, join_prompt_kernel<D, BITS>, p);
  }
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, std::string("attend_paged launch: ") + cudaGetErrorString(e));
  return KVQ_OK;
}

}  // namespace

size_t prompt_part_bytes() {
  return (size_t)2 * kPrMaxCtas * kPrPart * 4 + kPrMaxCtas * sizeof(int4);
}

kvq_status launch_attend_prompt(const PagedAttendHost& a, void* part, cudaStream_t s) {
  return dispatch_dgb(a.pk->D, a.pk->G, a.pk->bits, [&](auto d, auto g, auto b) {
    return run_prompt<decltype(d)::value, decltype(g)::value, decltype(b)::value>(a, part, s);
  });
}

uint32_t prompt_error_flags(bool clear) {
  uint32_t v = 0;
  cudaMemcpyFromSymbol(&v, g_prompt_err, sizeof(v));
  if (clear && v) {
    const uint32_t z = 0;
    cudaMemcpyToSymbol(g_prompt_err, &z, sizeof(z));
  }
  return v;
}

}  // namespace kvq
