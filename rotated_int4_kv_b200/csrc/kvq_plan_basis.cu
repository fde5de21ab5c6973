// kvq_plan_basis.cu -- what plans of the same head_dim, transform and code width share: the
// rotation without signs and factors, as the attention kernels' operands. Signs and factors
// are a plan's own few KB, which the kernels apply around these (an exact change of sign, one
// fp32 product per element), so a plan holds no matrix of its own for them. And the codec's
// matrices of a plan, formed on the GPU from the shared rotation in 64 bits.
#include <cmath>
#include <map>
#include <memory>
#include <mutex>
#include <tuple>
#include <vector>

#include "kvq_internal.h"

namespace kvq {

// Entry (i, j) of the Sylvester Hadamard matrix in natural order: (-1)^popcount(i & j).
double hadamard_value(int i, int j) { return (__builtin_popcount((unsigned)(i & j)) & 1) ? -1.0 : 1.0; }

double basis_dg(int c, int D) {
  if (c == 0 || c == D - 1) return 1.0 / std::sqrt((double)D);
  return (c & 1) ? std::sqrt(2.0 / D) : -std::sqrt(2.0 / D);
}

namespace {

uint16_t half_bits(float f) { return __half_as_ushort(__float2half_rn(f)); }
float half_value(uint16_t b) { return __half2float(__ushort_as_half(b)); }

// cos and sin of 2 pi r / M for r < M: every angle of an M-point transform, by its residue.
struct Circle {
  std::vector<double> c, s;
  explicit Circle(int M) : c(M), s(M) {
    for (int r = 0; r < M; ++r) {
      const double ang = 6.283185307179586476925286766559 * (double)r / (double)M;
      c[r] = std::cos(ang);
      s[r] = std::sin(ang);
    }
  }
};

// Q, row = channel. The orthonormal real basis in channel order: DC, then (cos_k, +sin_k)
// pairs, then Nyquist; or the normalised Hadamard matrix.
std::vector<double> make_basis(int D, bool hadamard) {
  std::vector<double> q((size_t)D * D);
  const Circle w(D);
  const double one = 1.0 / std::sqrt((double)D), two = std::sqrt(2.0 / D);
  for (int c = 0; c < D; ++c)
    for (int n = 0; n < D; ++n) {
      double& v = q[(size_t)c * D + n];
      const int r = (c + 1) / 2 * n % D;
      if (hadamard) v = hadamard_value(c, n) / std::sqrt((double)D);
      else if (c == 0) v = one;
      else if (c == D - 1) v = (n & 1) ? -one : one;
      else v = two * ((c & 1) ? w.c[r] : w.s[r]);
    }
  return q;
}

constexpr int kF = 128;  // points of the dense attention's transform

// A basis' device block as the host makes it: F128 hi and lo, then four D x D matrices.
size_t rot_halves() { return (size_t)2 * kF * kF; }
size_t block_halves(int D) { return rot_halves() + (size_t)4 * D * D; }

std::vector<uint16_t> make_block(int D, bool hadamard, int bits, const std::vector<double>& basis) {
  std::vector<uint16_t> blk(block_halves(D));
  // dense attention (both head dims): the unnormalised 128-point real DFT in slot order, F128
  // (hi, lo): row 0 = 1, row 1 = (-1)^m, row 2k = cos(2 pi k m / 128), row 2k+1 =
  // -sin(2 pi k m / 128); for the SRHT the 128-point Hadamard matrix (exact in fp16, lo = 0).
  // D = 128 applies it directly, D = 256 to the even and odd samples.
  const Circle w(kF);
  for (int j = 0; j < kF; ++j)
    for (int m = 0; m < kF; ++m) {
      const int r = j / 2 * m % kF;
      double v;
      if (hadamard) v = hadamard_value(j, m);
      else if (j == 0) v = 1.0;
      else if (j == 1) v = (m & 1) ? -1.0 : 1.0;
      else v = (j & 1) ? -w.s[r] : w.c[r];
      const uint16_t hi = half_bits((float)v);
      blk[(size_t)j * kF + m] = hi;
      blk[(size_t)(kF + j) * kF + m] = half_bits((float)(v - (double)half_value(hi)));
    }
  // paged attention: the basis with rows divided by basis_dg (entries cos, -sin, +-1: one fp16
  // rounding each, none for the SRHT), as query rotation (row = channel) and output
  // un-rotation (row = sample). Twice: as row-major matrices with the channels in the order in
  // which the prompt kernel converts a word of codes (word_channel), and in natural order as A
  // fragments: lane (g, c) of K step ks holds (row g | g + 8, columns 16 ks + 2c, + 1 | + 8, + 9)
  std::vector<uint16_t> nat((size_t)D * D);  // row = channel, natural order
  for (int c = 0; c < D; ++c)
    for (int n = 0; n < D; ++n)
      nat[(size_t)c * D + n] =
          half_bits((float)(hadamard ? hadamard_value(c, n) : basis[(size_t)c * D + n] / basis_dg(c, D)));
  for (int which = 0; which < 2; ++which) {
    uint16_t* row = blk.data() + rot_halves() + (size_t)which * D * D;
    uint16_t* frag = row + (size_t)2 * D * D;
    auto entry = [&](int i, int k) { return which ? nat[(size_t)k * D + i] : nat[(size_t)i * D + k]; };
    for (int i = 0; i < D; ++i)
      for (int k = 0; k < D; ++k)
        row[(size_t)i * D + k] = which ? entry(i, word_channel(k, bits)) : entry(word_channel(i, bits), k);
    size_t o = 0;
    for (int mt = 0; mt < D / 16; ++mt)
      for (int ks = 0; ks < D / 16; ++ks)
        for (int lane = 0; lane < 32; ++lane)
          for (int r = 0; r < 4; ++r)
            for (int x = 0; x < 2; ++x) {
              const int i = 16 * mt + (lane >> 2) + 8 * (r & 1), k = 16 * ks + 2 * (lane & 3) + 8 * (r >> 1) + x;
              frag[o++] = entry(i, k);
            }
  }
  return blk;
}

std::mutex g_mu;
// Kept for the process: constants of mathematics, at most eight forms of 0.3 to 1.1 MB a context.
// By the context's number, which no later context has: after a device reset they are made anew.
std::map<std::tuple<unsigned long long, int, int, int>, std::unique_ptr<PlanBasis>> g_bases;

// The number of the current device's context; false where there is none.
bool context_id(unsigned long long* id) {
  using Fn = CUresult (*)(CUcontext, unsigned long long*);
  static const Fn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool ok = cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<Fn>(p) : nullptr;
  }();
  return fn && cudaFree(nullptr) == cudaSuccess && fn(nullptr, id) == CUDA_SUCCESS;  // (cudaFree makes the context)
}

}  // namespace

kvq_status basis_of(int D, int xform, int bits, const PlanBasis** out) {
  unsigned long long id = 0;
  if (!context_id(&id)) return fail(KVQ_ERR_CUDA, "plan_create: no CUDA context");
  std::lock_guard<std::mutex> lk(g_mu);
  auto& slot = g_bases[{id, D, xform, bits}];
  if (!slot) {
    const std::vector<double> q = make_basis(D, xform == 1);
    const std::vector<uint16_t> blk = make_block(D, xform == 1, bits, q);
    const size_t nq = q.size() * 8, nblk = blk.size() * 2;
    void* dev = nullptr;
    if (cudaMalloc(&dev, nq + nblk) != cudaSuccess) return fail(KVQ_ERR_CUDA, "plan_create: cudaMalloc failed");
    if (cudaMemcpy(dev, q.data(), nq, cudaMemcpyHostToDevice) != cudaSuccess ||
        cudaMemcpy(static_cast<char*>(dev) + nq, blk.data(), nblk, cudaMemcpyHostToDevice) != cudaSuccess) {
      cudaFree(dev);
      return fail(KVQ_ERR_CUDA, "plan_create: upload failed");
    }
    slot = std::make_unique<PlanBasis>();
    slot->D = D;
    slot->xform = xform;
    slot->bits = bits;
    slot->q_dev = static_cast<const double*>(dev);
    slot->rot_dev = reinterpret_cast<const uint16_t*>(slot->q_dev + q.size());
    slot->wq_dev = slot->rot_dev + rot_halves();
    slot->wo_dev = slot->wq_dev + (size_t)D * D;
    slot->wqf_dev = reinterpret_cast<const uint4*>(slot->wo_dev + (size_t)D * D);
    slot->wof_dev = reinterpret_cast<const uint4*>(slot->wo_dev + (size_t)2 * D * D);
  }
  *out = slot.get();
  return KVQ_OK;
}

namespace {

// Block c, thread n: the entries of channel c and sample n. Every operation in 64 bits, rounded
// as written, so that the bits are those of the same formulas on a host.
__global__ void __launch_bounds__(kMaxD) form_plan_kernel(const double* q, const PlanHeader* head, int D, bool hadamard,
                                                          int bits, uint16_t* wt, uint16_t* wdec) {
  const int c = blockIdx.x, n = threadIdx.x;
  const double v = q[(size_t)c * D + n], lam = (double)head->lambda[c];
  const double s = (head->enc.sgn[n >> 1] >> (n & 1 ? 31 : 15)) & 1 ? -1.0 : 1.0;
  auto bits16 = [](double x) { return __half_as_ushort(__float2half_rn(__double2float_rn(x))); };
  if (hadamard) {
    wt[(size_t)c * D + n] = bits16(v < 0.0 ? -s : s);
  } else {
    const double w = __dmul_rn(__dmul_rn(lam, v), s);
    const uint16_t hi = bits16(w);
    const size_t row = 256 * (c >> 7) + (c & 127);
    wt[row * D + n] = hi;
    wt[(row + 128) * D + n] = bits16(__dsub_rn(w, (double)__half2float(__ushort_as_half(hi))));
  }
  wdec[(size_t)n * D + word_place(c, bits)] = bits16(__ddiv_rn(__dmul_rn(s, v), lam));
}

}  // namespace

kvq_status form_plan(const PlanBasis* b, const PlanHeader* head_dev, uint16_t* wt, uint16_t* wdec) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(b->D);
  cfg.blockDim = dim3(b->D);
  cudaError_t e = cudaLaunchKernelEx(&cfg, form_plan_kernel, b->q_dev, head_dev, b->D, b->xform == 1, b->bits, wt, wdec);
  if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
  if (e != cudaSuccess) return fail(KVQ_ERR_CUDA, std::string("plan_create: ") + cudaGetErrorString(e));
  return KVQ_OK;
}

}  // namespace kvq
