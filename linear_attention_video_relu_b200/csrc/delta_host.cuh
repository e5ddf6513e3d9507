// delta_host.cuh -- argument checks that the delta rule's entry points share.
#pragma once

#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "delta.cuh"
#include "linattn.h"

namespace la {
namespace delta {

inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p % n) == 0; }
inline bool aligned16(const void* p) { return aligned(p, 16); }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

inline la_status last_error() {
  return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

// Launches a kernel with `smem` bytes of dynamic shared memory. The limit that
// this needs is a property of the kernel on a device, set once. `next`: the
// kernel follows another one of the same call and may be set up while that one
// still runs (programmatic dependent launch); it waits for it by itself.
template <auto kernel>
la_status launch(unsigned grid, int threads, int smem, cudaStream_t stream, const Args& a,
                 bool next) {
  static std::atomic<uint64_t> set{0};   // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return LA_ERR_CUDA;
  }
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(set.load(std::memory_order_relaxed) & bit) || !bit) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess) {
      cudaGetLastError();
      return LA_ERR_UNSUPPORTED;
    }
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = next ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess) return LA_OK;
  cudaGetLastError();
  return LA_ERR_CUDA;
}

inline la_status device_sms(int* sms) {
  int dev = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    return LA_OK;
  cudaGetLastError();
  return LA_ERR_CUDA;
}

// Whether chains take 32 value columns per CTA and not 16 (RT 2 and 1 of the
// chains' kernels). 32 columns cost 1.2 to 1.45 times as long as 16, so they win
// where 16 would leave the device's SMs more than 1.4 times as many rounds of
// CTAs, one per SM. 2048 tokens of D 128, forward: 16 heads 74 us with 16, 107
// with 32; 24 heads 142 and 115; 40 heads (3 rounds and 2) 213 and 220; 64 heads
// 290 and 234; 128 heads 507 and 457. D 64: 32 heads 67 and 90, 40 heads 119 and
// 93, 80 heads 182 and 180, 128 heads 252 and 201. Backward, the CTAs of both
// kernels' chains counted together, since the second kernel's start on what SMs
// the first's leave, D 128: 8 heads 102 and 138, 16 heads 173 and 179, 20 heads (3
// and 2) 244 and 252, 36 heads 344 and 309, 128 heads 1169 and 1060; D 64: 16 heads
// 98 and 117, 40 heads 222 and 215, 128 heads 586 and 524.
inline la_status wide_chains(long long heads, int Dv, bool* wide) {
  int sms = 0;
  const la_status st = device_sms(&sms);
  if (st != LA_OK) return st;
  const long long one = (heads * ((Dv + 15) / 16) + sms - 1) / sms;
  const long long two = (heads * ((Dv + 31) / 32) + sms - 1) / sms;
  *wide = 10 * one > 14 * two;
  return LA_OK;
}

// Planes of what the carried state and the outputs are made from (all bits of
// fp32), and of what only gradients in T are made from.
constexpr int kChainPlanes = 3;
template <typename T>
constexpr int grad_planes() { return sizeof(T) == 2 ? 2 : 3; }

template <typename T, int KD, int PC, int PO>
la_status run_terms(const Args& a, long long heads, cudaStream_t stream) {
  using L = TermsSmem<mm::Io<T>::kPlanes, KD, PC>;
  return launch<terms_kernel<T, KD, PC, PO>>((unsigned)(heads * a.chunks), 128, L::bytes, stream, a,
                                           false);
}

inline la_status check_delta_workspace(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return LA_OK;
  return !ws || (uintptr_t)ws % 256 != 0 || bytes < need ? LA_ERR_WORKSPACE : LA_OK;
}

// The flag word of a workspace that a call is given, whether it needs it or not: of
// one with a control block, which is what lin_attn_device_status reads and clears.
inline int* flag_of(void* ws, size_t bytes) {
  return aligned(ws, sizeof(int)) && bytes >= LA_WORKSPACE_CONTROL_BYTES ? static_cast<int*>(ws)
                                                                         : nullptr;
}

// Sets it to zero on `stream`, for calls whose kernels do not.
inline la_status clear_flag(void* ws, size_t bytes, cudaStream_t stream) {
  int* flag = flag_of(ws, bytes);
  if (!flag || cudaMemsetAsync(flag, 0, sizeof(int), stream) == cudaSuccess) return LA_OK;
  cudaGetLastError();
  return LA_ERR_CUDA;
}

// `to` becomes `from` (or zeros), a call without tokens.
inline la_status copy_state(float* to, const float* from, size_t bytes, void* ws, size_t ws_bytes,
                            cudaStream_t stream) {
  if (!to || to == from) return LA_OK;
  const la_status st = clear_flag(ws, ws_bytes, stream);
  if (st != LA_OK) return st;
  const cudaError_t e = from ? cudaMemcpyAsync(to, from, bytes, cudaMemcpyDeviceToDevice, stream)
                             : cudaMemsetAsync(to, 0, bytes, stream);
  if (e == cudaSuccess) return LA_OK;
  cudaGetLastError();
  return LA_ERR_CUDA;
}

// Checks that need no device.
inline la_status check_delta(const la_delta_params* p) {
  if (!p) return LA_ERR_INVALID_ARG;
  if (p->B < 0 || p->H < 0 || p->N < 0) return LA_ERR_INVALID_ARG;
  if (p->Hk < 1 ? p->H != 0 : p->H % p->Hk != 0) return LA_ERR_INVALID_ARG;
  if (p->D < 8 || p->D > 128 || p->D % 8 || p->Dv < 8 || p->Dv > 128 || p->Dv % 8)
    return LA_ERR_INVALID_ARG;
  if (p->dtype != LA_F32 && p->dtype != LA_BF16) return LA_ERR_INVALID_ARG;
  if (p->layout != LA_LAYOUT_BHND && p->layout != LA_LAYOUT_BNHD) return LA_ERR_INVALID_ARG;
  if (!isfinite(p->scale)) return LA_ERR_INVALID_ARG;
  // tokens are counted in ints, up to whole chunks; a grid has one CTA per head
  // and slice of columns (at most 16 slices), or per head and chunk
  const long long heads = (long long)p->B * p->H;
  if (p->N > INT_MAX - kC) return LA_ERR_UNSUPPORTED;
  if (heads > (1LL << 24) || heads * ((p->N + (long long)kC - 1) / kC) > INT_MAX)
    return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

struct DeltaBytes {
  size_t elt, qk, v, gate;
  explicit DeltaBytes(const la_delta_params& p) {
    elt = p.dtype == LA_BF16 ? 2 : 4;
    const size_t tokens = (size_t)p.B * p.N;
    qk = tokens * p.Hk * p.D * elt;
    v = tokens * p.H * p.Dv * elt;
    gate = tokens * p.H * elt;
  }
};

inline Args delta_args(const la_delta_params& p, const void* q, const void* k, const void* v,
                       const void* g, const void* beta, const float* state, const int* lengths) {
  Args a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.beta = beta;
  a.s0 = state;
  a.lengths = lengths;
  a.B = p.B;
  a.H = p.H;
  a.Hk = p.Hk;
  a.N = p.N;
  a.D = p.D;
  a.Dv = p.Dv;
  a.bnhd = p.layout == LA_LAYOUT_BNHD;
  a.scale = p.scale;
  a.chunks = (p.N + kC - 1) / kC;
  return a;
}

}  // namespace delta
}  // namespace la
