// kvq_internal.h -- definitions shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <string>
#include <type_traits>

#include "../../include/kvq.h"

namespace kvq {

constexpr int kMaxD = 256;

// Per-plan constants handed to the codec kernels by value (kernel parameter
// space), so that every per-channel factor is a constant-bank operand.
struct CodecConsts {
  float chan[kMaxD];       // encode: lambda_c * dg_c ; decode: dg_c / lambda_c (rotated channel c)
  uint32_t sgn[kMaxD / 2]; // XOR mask per fp16 pair of the original domain (0x8000 per negative s)
};

// The front of a plan's device block.
struct PlanHeader {
  CodecConsts enc, dec;
  float lambda[kMaxD];
};

// What plans of one device, head_dim, transform and code width share (kvq_plan_basis.cu): the
// rotation without signs and factors.
struct PlanBasis {
  int D, xform, bits;
  const double* q_dev = nullptr;      // Q, row = channel
  const uint16_t* rot_dev = nullptr;  // F128 (see kvq_plan)
  // Paged attention, with E = Q, its rows divided by basis_dg (fp16): E (query rotation) and E^T
  // (output un-rotation), each as row-major [D][D] with the channels in the order of
  // word_channel, and in natural order as mma.m16n8k16 A fragments (16 bytes per (16-row
  // tile, K step, lane)). The kernels multiply channel c by basis_dg / lambda_c (dec.chan) and
  // flip samples by the signs.
  const uint16_t* wq_dev = nullptr;
  const uint16_t* wo_dev = nullptr;
  const uint4* wqf_dev = nullptr;
  const uint4* wof_dev = nullptr;
};

}  // namespace kvq

struct kvq_plan {
  int D = 0;
  int G = 0;
  int device = -1;
  int xform = 0;           // kvq_transform: 0 SRFT, 1 SRHT
  int bits = 4;            // code width: 4 (nibble pairs) or 8 (one byte per channel)
  kvq::CodecConsts enc{};  // lambda_c * dg_c
  kvq::CodecConsts dec{};  // dg_c / lambda_c
  // Device block: copies of `enc` and `dec` for kernels that serve several plans
  // in one launch (grouped encode) or two plans at once (attention: K and V).
  void* dblock = nullptr;
  const kvq::CodecConsts* enc_dev = nullptr;
  const kvq::CodecConsts* dec_dev = nullptr;
  // Tensor-core encode operand in the same block: W = Lambda F_r diag(s) as fp16
  // hi + lo, per 128-channel half 128 hi rows then 128 lo rows, D columns.
  const uint16_t* wt_dev = nullptr;
  // What it shares with other plans, and its F128: the unnormalised 128-point real DFT in
  // slot order, fp16 hi rows [128] then lo rows [128] (the attention kernels apply the
  // plans' signs and per-channel factors around it).
  const kvq::PlanBasis* basis = nullptr;
  const uint16_t* rot_dev = nullptr;
  // Tensor-core decode operand in the same block: W_dec = diag(s) Q^T Lambda^-1 as fp16,
  // D rows (output samples) x D columns (channels, in the dequantiser's pair order).
  const uint16_t* wdec_dev = nullptr;
};

namespace kvq {

// Bytes of one cached vector's codes.
inline int code_row_bytes(const kvq_plan* p) { return p->D * p->bits / 8; }

template <int V>
using IC = std::integral_constant<int, V>;

// Calls f(IC<D>, IC<G>, IC<BITS>) for the quantiser configurations the kernels are
// built for (D 128 | 256, G 32 | 16, BITS 4 | 8); fails with `what` otherwise.
template <typename F>
auto dispatch_dgb(int D, int G, int bits, F&& f) -> decltype(f(IC<128>{}, IC<32>{}, IC<4>{})) {
  if (bits == 4) {
    if (D == 128) return G == 32 ? f(IC<128>{}, IC<32>{}, IC<4>{}) : f(IC<128>{}, IC<16>{}, IC<4>{});
    return G == 32 ? f(IC<256>{}, IC<32>{}, IC<4>{}) : f(IC<256>{}, IC<16>{}, IC<4>{});
  }
  if (D == 128) return G == 32 ? f(IC<128>{}, IC<32>{}, IC<8>{}) : f(IC<128>{}, IC<16>{}, IC<8>{});
  return G == 32 ? f(IC<256>{}, IC<32>{}, IC<8>{}) : f(IC<256>{}, IC<16>{}, IC<8>{});
}

// thread-local last-error text
void set_error(const std::string& msg);
kvq_status fail(kvq_status st, const std::string& msg);

// driver entry point for tensor-map encoding (no link against libcuda)
kvq_status encode_tiled(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                        const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                        CUtensorMapSwizzle swz, const char* what);

// the same without the cache of encoded maps
kvq_status encode_tiled_new(CUtensorMap* map, CUtensorMapDataType dt, int rank, const void* base,
                            const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t* box,
                            CUtensorMapSwizzle swz, const char* what);

int num_sms(int device);

// the shared part of a plan on the current device (kvq_plan_basis.cu)
kvq_status basis_of(int D, int xform, int bits, const PlanBasis** out);
double basis_dg(int c, int D);  // the real DFT's rows' normalisation: 1/sqrt(D), sqrt(2/D) (cos), -sqrt(2/D) (sin)
// a plan's codec operands from its header, both on the device; returns when they are there
kvq_status form_plan(const PlanBasis* b, const PlanHeader* head_dev, uint16_t* wt, uint16_t* wdec);

kvq_status check_plan_device(const kvq_plan* p);

// The channel at place p of a row when every 32-bit word of its codes is converted to fp16
// pairs by masks: int4 pairs (0, 4) (1, 5) (2, 6) (3, 7), int8 pairs (0, 2) (1, 3).
constexpr int word_channel(int p, int bits) {
  return bits == 4 ? (p & ~7) + ((p & 7) >> 1) + 4 * (p & 1) : (p & ~3) + ((p & 3) >> 1) + 2 * (p & 1);
}

// The place of channel c: word_channel(word_place(c)) = c.
constexpr int word_place(int c, int bits) {
  return bits == 4 ? (c & ~7) + 2 * (c & 3) + ((c >> 2) & 1) : (c & ~3) + 2 * (c & 1) + ((c >> 1) & 1);
}

// Lets a kernel use `bytes` of dynamic shared memory on `device` (an attribute of the
// kernel on one device; set once for each).
template <auto Kernel>
cudaError_t allow_smem(int device, int bytes) {
  static std::atomic<uint64_t> done{0};
  const uint64_t bit = 1ull << (device & 63);
  if (device < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// tensor-core encode (kvq_encode_tc.cu)
bool encode_tc_supported(int D, int G);
bool encode_split_supported(const kvq_plan* p);
kvq_status launch_encode_tc(const kvq_encode_job* jobs, int njobs, cudaStream_t s, bool split);
uint32_t encode_tc_error_flags(bool clear);
// encode path: 0 = tensor cores where supported (the radix-2 split kernel for head_dim 256 SRFT
// plans), else the register FFT; 1 = register FFT; 2 = tensor cores, dense product; 3 = tensor
// cores, radix-2 split (head_dim 256 SRFT only)
int encode_path();
kvq_status dispatch_encode(const kvq_encode_job* jobs, int njobs, cudaStream_t s);

// tensor-core decode (kvq_decode_tc.cu)
kvq_status launch_decode_tc(const kvq_plan* p, const uint8_t* codes, const uint16_t* scales, int B, int H,
                            int T_cap, int t0, int n, uint16_t* out, cudaStream_t s);
uint32_t decode_tc_error_flags(bool clear);
// decode path: 0 = tensor cores (default), 1 = register FFT
int decode_path();

// codec launchers (kvq_codec.cu)
kvq_status launch_encode_jobs(const kvq_encode_job* jobs, int njobs, cudaStream_t s);
kvq_status launch_decode(const kvq_plan* p, const uint8_t* codes, const uint16_t* scales, int B, int H,
                         int T_cap, int t0, int n, uint16_t* out, cudaStream_t s);

// attention launchers (kvq_attend.cu)
// One decode-attention problem: plans (quantised caches; none for the fp16 comparator),
// query, caches, output.
struct AttendJobHost {
  const kvq_plan* pk;
  const kvq_plan* pv;
  const uint16_t* q;
  const void* kc;   // K codes (int4) or fp16 K
  const uint16_t* ks;
  const void* vc;   // V codes (int4) or fp16 V
  const uint16_t* vs;
  uint16_t* out;
};
size_t attend_workspace_bytes(int B, int Hq, int Hkv, int D, int T_cap);
kvq_status launch_attend_int4_batch(const AttendJobHost* jobs, int njobs, int B, int Hq, int Hkv, int T_cap,
                                    const int32_t* seq_lens, int T_len, float sigma, void* ws, size_t ws_bytes,
                                    cudaStream_t s);
kvq_status launch_attend_int4(const kvq_plan* pk, const kvq_plan* pv, const uint16_t* q,
                              const uint8_t* kc, const uint16_t* ks, const uint8_t* vc, const uint16_t* vs,
                              int B, int Hq, int Hkv, int T_cap, const int32_t* seq_lens, int T_len,
                              float sigma, uint16_t* out, void* ws, size_t ws_bytes, cudaStream_t s);
kvq_status launch_attend_int4_noalloc(const kvq_plan* pk, const kvq_plan* pv, const uint16_t* q,
                                      const uint8_t* kc, const uint16_t* ks, const uint8_t* vc,
                                      const uint16_t* vs, int B, int Hq, int Hkv, int T_cap,
                                      const int32_t* seq_lens, int T_len, float sigma, uint16_t* out,
                                      cudaStream_t s);
kvq_status launch_attend_int4_append(const kvq_plan* pk, const kvq_plan* pv, const uint16_t* q, const uint16_t* k_new,
                                     const uint16_t* v_new, uint8_t* kc, uint16_t* ks, uint8_t* vc, uint16_t* vs, int B,
                                     int Hq, int Hkv, int T_cap, int pos, float sigma, uint16_t* out, void* ws,
                                     size_t ws_bytes, cudaStream_t s);
kvq_status launch_attend_int4_partial(const kvq_plan* pk, const kvq_plan* pv, const uint16_t* q, const uint8_t* kc,
                                      const uint16_t* ks, const uint8_t* vc, const uint16_t* vs, int B, int Hq,
                                      int Hkv, int T_cap, int t_begin, int t_end, float sigma, float* part, void* ws,
                                      size_t ws_bytes, cudaStream_t s);
kvq_status launch_attend_combine(const kvq_plan* pv, const float* parts, int N, int B, int Hq, uint16_t* out,
                                 cudaStream_t s);
kvq_status launch_attend_fp16(const uint16_t* q, const uint16_t* k, const uint16_t* v, int B, int Hq,
                              int Hkv, int D, int T_cap, const int32_t* seq_lens, int T_len, float sigma,
                              uint16_t* out, void* ws, size_t ws_bytes, cudaStream_t s);

kvq_status attend_split_info(int B, int Hq, int Hkv, int D, int G, int bits, int T, int* splits, int* cluster,
                             int* head_tiles);
// pages (kvq_page_plan.cu, kvq_encode_tc.cu, kvq_decode_tc.cu, kvq_attend_paged.cu)
constexpr int kMaxPlanRequests = 16384;  // requests of one page_plan call (12 bytes of shared memory each)
constexpr int kMaxPageHeads = 128;       // KV heads of a paged encode (a tile holds whole tokens)
kvq_status launch_page_plan(const int32_t* kv_lens, const int32_t* q_lens, int B, int32_t* table, int max_pages,
                            long long table_stride, const int32_t* free_pages, int n_free, const int32_t* free_head,
                            int32_t* free_head_out, int page_shift, int32_t* slots, int32_t* positions, int n_slots,
                            int32_t* q_starts, int32_t* kv_out, int32_t* info, cudaStream_t s);
kvq_status launch_page_release(const uint8_t* done, int32_t* kv_lens, const int32_t* table, long long table_stride,
                               int B, int max_pages, int page_shift, int32_t* free_pages, int n_free,
                               int32_t* free_head, cudaStream_t s);
kvq_status launch_encode_paged(const kvq_paged_encode_job* jobs, int njobs, int n, int H, int page_shift,
                               int num_pages, const int32_t* slots, cudaStream_t s);
kvq_status launch_decode_paged(const kvq_plan* p, const uint8_t* codes, const uint16_t* scales, int num_pages,
                               int page_shift, int H, const int32_t* slots, int n, uint16_t* out, cudaStream_t s);
// One paged attention call (host view of kvq_attend_paged's arguments).
struct PagedAttendHost {
  const kvq_plan* pk;
  const kvq_plan* pv;
  const uint16_t* q;
  long long q_token_stride, q_head_stride;
  const uint8_t* kc;
  const uint16_t* ks;
  const uint8_t* vc;
  const uint16_t* vs;
  int num_pages, page_shift;
  const int32_t* table;
  int max_pages;
  long long table_stride;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  int B, n_q, Hq, Hkv, max_q_len, max_kv_len, window;
  float sigma;
  uint16_t* out;
  void* ws;
  size_t ws_bytes;
  int path;  // 0: either kernel, by what both would take; 1: few query rows; 2: prompts
};
size_t paged_workspace_bytes(int B, int Hq, int Hkv, int D, int n_q, int max_q_len, int path);
kvq_status launch_attend_paged(const PagedAttendHost& a, cudaStream_t s);
uint32_t paged_error_flags(bool clear);
// The kernel for many query rows (kvq_attend_prompt.cu); launch_attend_paged chooses.
size_t prompt_part_bytes();
kvq_status launch_attend_prompt(const PagedAttendHost& a, void* part, cudaStream_t s);
uint32_t prompt_error_flags(bool clear);

kvq_status launch_wait_probe(uint32_t limit_us, cudaStream_t s);

// device error word (bit flags raised by kernels that gave up a bounded wait)
uint32_t* device_error_word();

}  // namespace kvq
