// delta.cu -- the gated delta rule's forward pass (lin_attn_delta_forward in
// include/linattn.h): the kernel for a few tokens, and the choice between it
// and the chunked one (delta_scan.cuh).
#include "linattn.h"

#include <limits.h>
#include <math.h>

#include "delta_host.cuh"
#include "delta_scan.cuh"

namespace la {
namespace delta {
namespace {

// ---- a few tokens -----------------------------------------------------------------
//
// The state is read once into registers, the tokens are applied one after
// another, and it is written once: 8 D Dv bytes per head, which bound a step
// (at one token 6 D Dv flops go with them). A CTA has 32 columns of a head: a
// warp's load covers four rows of them, 128 contiguous bytes each, and its 128
// threads hold 16 rows x 8 column groups of four. Since
//     S_t^T q = a S_{t-1}^T q + beta (k.q) (v - a S_{t-1}^T k),
// one pass over the rows gives S^T k, S^T q and k.q, and a token costs one
// reduction: two shuffles, then four warps' sums through shared memory. 64
// sequences of 32 heads of 128 x 128 (270 MB) take 43 us, 6.2 TB/s; one of 64 x
// 64 takes 4.4 with cold caches and 2.7 in a loop that is replayed, its launch and
// the latency of its loads and of the reduction. (Loading the next
// CTA's rows ahead was slower: fewer CTAs share an SM.)
constexpr int kStepCols = 32, kStepThreads = 128;

template <typename T, int RPT>
__global__ void __launch_bounds__(kStepThreads) step_kernel(const Args a) {
  constexpr int DP = RPT * 16;
  extern __shared__ __align__(16) float kq[];          // [tokens][2][DP]
  __shared__ __align__(16) float red[2][4][2][kStepCols];
  __shared__ float red_kq[2][4];
  const int bh = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int cg = threadIdx.x & 7, rg = threadIdx.x >> 3, warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int col = slice * kStepCols + cg * 4;
  const bool in = col < a.Dv;
  const int len = length_of(a, b);
  const long long s_at = (long long)bh * a.D * a.Dv + col;
  if (a.flag && blockIdx.x == 0 && threadIdx.x == 0) *a.flag = 0;   // nothing waits here

  float4 s[RPT];
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int row = rg + 16 * i;
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (a.s0 && in && row < a.D)
      s[i] = *reinterpret_cast<const float4*>(a.s0 + s_at + (long long)row * a.Dv);
  }
  const Rows rk = rows_of(a, b, hk, a.Hk, a.D), rv = rows_of(a, b, h, a.H, a.Dv);
  const Rows rg1 = rows_of(a, b, h, a.H, 1);
  const T* kp = static_cast<const T*>(a.k) + rk.base;
  const T* qp = static_cast<const T*>(a.q) + rk.base;
  for (int i = threadIdx.x; i < len * DP; i += kStepThreads) {
    const int t = i / DP, d = i % DP;
    const bool live = d < a.D;
    kq[t * 2 * DP + d] = live ? mm::Io<T>::load(kp + t * rk.stride + d) : 0.f;
    kq[t * 2 * DP + DP + d] = live ? mm::Io<T>::load(qp + t * rk.stride + d) : 0.f;
  }
  __syncthreads();

  const T* gp = static_cast<const T*>(a.g) + rg1.base;
  const T* bp = static_cast<const T*>(a.beta) + rg1.base;
  const T* vp = static_cast<const T*>(a.v) + rv.base + col;
  T* op = static_cast<T*>(a.out) + rv.base + col;
  for (int t = 0; t < len; ++t) {
    const float dec = expf(clamp_decay(mm::Io<T>::load(gp + t * rg1.stride)));
    const float bt = mm::Io<T>::load(bp + t * rg1.stride);
    float2 v01 = make_float2(0.f, 0.f), v23 = v01;
    if (in) {
      v01 = mm::Io<T>::load2(vp + t * rv.stride);
      v23 = mm::Io<T>::load2(vp + t * rv.stride + 2);
    }
    const float* kt = kq + t * 2 * DP;
    float x[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) x[i] = 0.f;
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float k = kt[rg + 16 * i], q = kt[DP + rg + 16 * i];
      x[0] = fmaf(k, s[i].x, x[0]);
      x[1] = fmaf(k, s[i].y, x[1]);
      x[2] = fmaf(k, s[i].z, x[2]);
      x[3] = fmaf(k, s[i].w, x[3]);
      x[4] = fmaf(q, s[i].x, x[4]);
      x[5] = fmaf(q, s[i].y, x[5]);
      x[6] = fmaf(q, s[i].z, x[6]);
      x[7] = fmaf(q, s[i].w, x[7]);
      x[8] = fmaf(k, q, x[8]);
    }
#pragma unroll
    for (int i = 0; i < 9; ++i) {
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], 8);
      x[i] += __shfl_xor_sync(0xffffffffu, x[i], 16);
    }
    const int z = t & 1;   // two sets of sums: a warp ahead writes the other one
    if (lane < 8) {
      *reinterpret_cast<float4*>(&red[z][warp][0][cg * 4]) = make_float4(x[0], x[1], x[2], x[3]);
      *reinterpret_cast<float4*>(&red[z][warp][1][cg * 4]) = make_float4(x[4], x[5], x[6], x[7]);
      if (lane == 0) red_kq[z][warp] = x[8];
    }
    __syncthreads();
    float4 ks = make_float4(0.f, 0.f, 0.f, 0.f), qs = ks;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 y = *reinterpret_cast<const float4*>(&red[z][i][0][cg * 4]);
      ks.x += y.x, ks.y += y.y, ks.z += y.z, ks.w += y.w;
      const float4 u = *reinterpret_cast<const float4*>(&red[z][i][1][cg * 4]);
      qs.x += u.x, qs.y += u.y, qs.z += u.z, qs.w += u.w;
      dot += red_kq[z][i];
    }
    const float4 r = make_float4(bt * (v01.x - dec * ks.x), bt * (v01.y - dec * ks.y),
                                 bt * (v23.x - dec * ks.z), bt * (v23.y - dec * ks.w));
    if (rg == 0 && in) {
      T* o = op + t * rv.stride;
      mm::Io<T>::store2(o, a.scale * (dec * qs.x + dot * r.x), a.scale * (dec * qs.y + dot * r.y));
      mm::Io<T>::store2(o + 2, a.scale * (dec * qs.z + dot * r.z),
                        a.scale * (dec * qs.w + dot * r.w));
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const float k = kt[rg + 16 * i];
      s[i].x = fmaf(k, r.x, dec * s[i].x);
      s[i].y = fmaf(k, r.y, dec * s[i].y);
      s[i].z = fmaf(k, r.z, dec * s[i].z);
      s[i].w = fmaf(k, r.w, dec * s[i].w);
    }
  }
  if (a.s1 && in) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int row = rg + 16 * i;
      if (row < a.D) *reinterpret_cast<float4*>(a.s1 + s_at + (long long)row * a.Dv) = s[i];
    }
  }
}

template <typename T, int RPT>
la_status run_step(Args a, int B, cudaStream_t stream) {
  a.slices = (a.Dv + kStepCols - 1) / kStepCols;
  const size_t smem = (size_t)a.N * 2 * RPT * 16 * sizeof(float);
  step_kernel<T, RPT>
      <<<(unsigned)((long long)B * a.H * a.slices), kStepThreads, smem, stream>>>(a);
  return last_error();
}

template <typename T, int KD, int RT, int NBUF>
la_status run_chunks(Args a, int B, cudaStream_t stream) {
  constexpr int PC = kChainPlanes, PO = kChainPlanes;
  const long long heads = (long long)B * a.H;
  const la_status st = run_terms<T, KD, PC, PO>(a, heads, stream);
  if (st != LA_OK) return st;
  using Cfg = ScanCfg<T, KD, RT, PC, PO, NBUF, false>;
  a.slices = (a.Dv + 16 * RT - 1) / (16 * RT);
  return launch<scan_kernel<T, KD, RT, PC, PO, NBUF, false>>(
      (unsigned)(heads * a.slices), Cfg::threads, Cfg::bytes, stream, a, true);
}

// One after another or in chunks: a token takes 0.4 us where its CTAs fit the
// device at once, the two kernels for chunks 10.4 to 12.5 us at few heads whatever
// the tokens, so they are even at 17 (8 heads of D 128) to 20 tokens (D 64, and 32
// heads of D 128). With many heads the chunks' CTAs, one per SM, queue: 256 heads
// of D 128, 24 tokens: 42 against 45 us; 1024 of D 64: 58 against 73.
bool few_tokens(const la_delta_params& p) {
  const long long chains = (long long)p.B * p.H * ((p.Dv + 15) / 16);
  return p.N <= LA_DELTA_STEP_TOKENS || (p.N <= 24 && chains > 512);
}

la_status run_forward(const Args& a, int B, bool is_bf16, bool few, cudaStream_t stream) {
  if (few) {
    if (is_bf16) return a.D <= 64 ? run_step<bf16, 4>(a, B, stream) : run_step<bf16, 8>(a, B, stream);
    return a.D <= 64 ? run_step<float, 4>(a, B, stream) : run_step<float, 8>(a, B, stream);
  }
  if (!is_bf16)
    return a.D <= 64 ? run_chunks<float, 64, 1, 2>(a, B, stream)
                     : run_chunks<float, 128, 1, 1>(a, B, stream);
  bool wide = false;
  const la_status st = wide_chains((long long)B * a.H, a.Dv, &wide);
  if (st != LA_OK) return st;
  if (a.D <= 64)
    return wide ? run_chunks<bf16, 64, 2, 3>(a, B, stream) : run_chunks<bf16, 64, 1, 3>(a, B, stream);
  return wide ? run_chunks<bf16, 128, 2, 2>(a, B, stream) : run_chunks<bf16, 128, 1, 2>(a, B, stream);
}

// Workspace of a forward call that runs in chunks: the control block, a record
// per chunk.
size_t forward_bytes(const la_delta_params& p) {
  if (few_tokens(p)) return 0;
  const size_t chunks = (size_t)p.B * p.H * ((p.N + kC - 1) / kC);
  return LA_WORKSPACE_CONTROL_BYTES + chunks * Record<kChainPlanes, kChainPlanes>::bytes;
}

}  // namespace
}  // namespace delta
}  // namespace la

using namespace la;
using namespace la::delta;

extern "C" {

la_status lin_attn_delta_workspace_size(const la_delta_params* p, size_t* bytes) {
  if (!bytes) return LA_ERR_INVALID_ARG;
  const la_status st = check_delta(p);
  if (st == LA_OK) *bytes = forward_bytes(*p);
  return st;
}

la_status lin_attn_delta_forward(const la_delta_params* p, const void* q, const void* k,
                                 const void* v, const void* log_decay, const void* beta,
                                 const float* state, const int* lengths, void* out,
                                 float* state_out, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  la_status st = check_delta(p);
  if (st != LA_OK) return st;
  const long long heads = (long long)p->B * p->H;
  if (heads == 0) return LA_OK;
  const size_t sbytes = (size_t)heads * p->D * p->Dv * sizeof(float);
  if (!aligned16(state) || !aligned16(state_out)) return LA_ERR_INVALID_ARG;
  if (state_out && state != state_out && overlaps(state, sbytes, state_out, sbytes))
    return LA_ERR_INVALID_ARG;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (p->N == 0) {
    const int* flag = flag_of(workspace, workspace_bytes);
    if (overlaps(flag, sizeof(int), state, sbytes) || overlaps(flag, sizeof(int), state_out, sbytes))
      return LA_ERR_INVALID_ARG;
    return copy_state(state_out, state, sbytes, workspace, workspace_bytes, cs);
  }
  const DeltaBytes n(*p);
  const void* in[6] = {q, k, v, log_decay, beta, lengths};
  const size_t nb[6] = {n.qk, n.qk, n.v, n.gate, n.gate, lengths ? p->B * sizeof(int) : 0};
  for (int i = 0; i < 5; ++i)
    if (!in[i] || !aligned(in[i], i < 3 ? 16 : n.elt)) return LA_ERR_INVALID_ARG;
  if (!aligned(lengths, 4) || !out || !aligned16(out)) return LA_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i)
    if (overlaps(out, n.v, in[i], nb[i]) || overlaps(state_out, sbytes, in[i], nb[i]))
      return LA_ERR_INVALID_ARG;
  if (overlaps(out, n.v, state, sbytes) || overlaps(out, n.v, state_out, sbytes))
    return LA_ERR_INVALID_ARG;
  const size_t need = forward_bytes(*p);
  if ((st = check_delta_workspace(workspace, workspace_bytes, need)) != LA_OK) return st;
  int* const flag = flag_of(workspace, workspace_bytes);
  const size_t used = need ? need : flag ? sizeof(int) : 0;
  for (int i = 0; i < 6; ++i)
    if (overlaps(workspace, used, in[i], nb[i])) return LA_ERR_INVALID_ARG;
  if (overlaps(workspace, used, out, n.v) || overlaps(workspace, used, state, sbytes) ||
      overlaps(workspace, used, state_out, sbytes))
    return LA_ERR_INVALID_ARG;
  Args a = delta_args(*p, q, k, v, log_decay, beta, state, lengths);
  a.out = out;
  a.s1 = state_out;
  a.flag = flag;
  a.rec = static_cast<unsigned char*>(workspace) + LA_WORKSPACE_CONTROL_BYTES;
  return run_forward(a, p->B, p->dtype == LA_BF16, few_tokens(*p), cs);
}

}  // extern "C"
