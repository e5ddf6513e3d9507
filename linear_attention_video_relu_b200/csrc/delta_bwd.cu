// delta_bwd.cu -- the gradients of the gated delta rule
// (lin_attn_delta_backward in include/linattn.h).
//
// With the names of delta.cuh, E_ij = exp(G_i - G_j), the incoming gradient
// dO of the outputs and dS' of the state after a chunk:
//     dX   = P^T dO + z . (K dS')                       z = exp(G_last - G)
//     dR   = T^T dX
//     dS   = exp(G_last) dS' + Q^T (w . dO) - K^T (x . dR)   w = scale e, x = beta e
//     dP   = dO X^T (j <= i),   dA = -dR X^T (j < i)
//     dv_i = beta_i dR_i
//     dq   = w . (dO S^T) + EP K                        EP = scale E . dP
//     dk   = z . (X dS'^T) - x . (dR S^T) + EP^T Q + (F + F^T) K,  F = beta E . dA
//     dbeta_i = dR_i.(v_i - e_i S^T k_i) + sum_j E_ij dA_ij k_i.k_j
//     dg_t = exp(G_last) <S, dS'> + sum_{i >= t} (q_i.(w . dO S^T)_i - k_i.(x . dR S^T)_i)
//            + sum_{j < t} k_j.(z . X dS'^T)_j + sum_{i >= t > j} M_ij,   M = dP.P + dA.A.
// (dg is that of the sums G, summed from t on: of what a pair or a row has in it,
// the terms whose decay does not pass t cancel. They are left out here, so that
// every term of dg_t has exp(g_t) in it, and a decay that forgets nearly all
// has a gradient with digits of its own and not the others' rounding.)
// Nothing is kept from the forward pass: the states before the chunks are made
// again (scan_kernel), then the gradients of the states are carried backwards
// (reverse_kernel), and with both in the workspace all chunks' gradients are
// made at once (gradient_tc_kernel in bf16, gradient_kernel in fp32).
//
// Rounding: sums, and the two states that are carried, are fp32, and fp32 calls
// keep all its bits in every product. In bf16 the operands that only gradients in
// bf16 come from are two bf16 planes, 17 bits: S, dS', X, dR, EP and F, and where
// no gradient of the initial state (fp32) is asked for the chains' T, R, dX too. Of
// such gradients 0.5 to 0.8 % are not the exact value's rounding, where an fp32
// computation has 0.02 to 0.05 %; their distance to the exact values is that of the
// last rounding both ways (1.66e-3). With three planes everywhere the batch of
// 2 x 16 heads of 4096 tokens, D 128, took 1088 us instead of 606: two atoms of
// three planes of S and dS' are more than an SM's shared memory, so that the
// products fell to warp-level instructions, and chains of 32 columns do not fit
// either.
#include "linattn.h"

#include "delta_host.cuh"
#include "delta_scan.cuh"

namespace la {
namespace delta {
namespace {

// ---- the chain of state gradients ----------------------------------------------------
//
// Like scan_kernel, from the last chunk to the first. Per chunk the chain is
//     K dS' -> dX = aux1 + z . (K dS') -> dR = T^T dX
//           -> dS = exp(G_last) dS' + aux2 - K^T (x . dR),
// on warps 0-3; warps 4-7 make aux1 = P^T dO and aux2 = Q^T (w . dO) a chunk
// ahead; warps 8-11 move: dS', dR and dv out, the next chunks' operands in, the
// helpers' a step before the chain's. What bounds it is shared memory, whose pipe
// is 80 % busy (tensor 39 %, issue 38 %): 2.9 us a chunk at D 128 with 32 columns
// (32 heads of 4096 tokens: 186 us), where scan_kernel takes 2.2. (With the
// operands of both in one copy, and all three groups meeting twice a chunk, it
// was 228 us: the helpers waited for the copies and the chain for the helpers.)
// Named barriers: kRevFree.. frees the chain's part of a stage, kRevFreeH.. the
// helpers', who are done with theirs when the chain begins; kRevChain and kRevHelp
// are a group's own; kRevS is the chain's and the helpers', when dS' is stored and
// its aux made; kRevOut tells the copies of dS'; kRevX is the chain's and the
// copies', when dR is stored and dS' has been read; kRevRead tells the chain that
// dR has been read.
enum {
  kRevFree = 1, kRevChain = 4, kRevX = 5, kRevS = 6, kRevHelp = 7, kRevOut = 8, kRevRead = 9,
  kRevFreeH = 10
};

template <typename T, int KD, int RT, int PC, int PO, int NBUF>
struct RevCfg {
  static constexpr int PI = mm::Io<T>::kPlanes, NV = 16 * RT;
  using R = Record<PC, PC>;
  static constexpr int kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  static constexpr int kLN = (NV + 8) * 2, kPlaneS = KD * kLN, kPlaneX = kC * kLN;
  static constexpr int MS = Share<KD, RT>::MS;
  // a stage: what the chain takes from it, Gates, T and K, and what the helpers
  // take, Gates, P, Q and dO
  static constexpr int offK = R::offP, offH = offK + PI * kPlaneK;
  static constexpr int offP = offH + (int)sizeof(Gates), offQ = offP + R::offD - R::offP;
  static constexpr int offO = offQ + PI * kPlaneK;
  static constexpr int stage = offO + PI * kPlaneX;
  static constexpr int offS = NBUF * stage;            // dS', PC planes
  static constexpr int offY = offS + PC * kPlaneS;     // dX, then dR for the helpers
  static constexpr int offX = offY + PC * kPlaneX;     // x . dR
  static constexpr int offW = offX + PC * kPlaneX;     // w . dO
  // per set: aux1 and aux2, each thread's own sums
  static constexpr int aux = 128 * 2 * 16 * (RT + MS);
  static constexpr int offAux = offW + PC * kPlaneX;
  static constexpr int offBar = offAux + 2 * aux;
  static constexpr int bytes = offBar + 2 * NBUF * 8 + 8;
  static constexpr int threads = 256 + kLoadThreads;
};

template <typename T, int KD, int RT, int PC, int PO, int NBUF>
__global__ void __launch_bounds__(256 + kLoadThreads, 1) reverse_kernel(const Args a) {
  using Cfg = RevCfg<T, KD, RT, PC, PO, NBUF>;
  using Rec = typename Cfg::R;
  constexpr int PI = Cfg::PI, NV = Cfg::NV, MS = Cfg::MS, kLN = Cfg::kLN, kLK = Cfg::kLK;
  extern __shared__ __align__(16) unsigned char smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  // an mbarrier per stage and part
  const uint32_t full = sbase + Cfg::offBar, full_h = full + 8 * NBUF;
  volatile int* gave_up = reinterpret_cast<volatile int*>(smem + Cfg::offBar + 2 * NBUF * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * NBUF; ++i) ptx::mbar_init(full + 8 * i, kLoadThreads + 1);
    *gave_up = 0;
    ptx::fence_mbar_init();
  }
  // The kernel before, scan_kernel, starts this one once the records are there,
  // and this one reads nothing of what that one writes.
  ptx::launch_dependents();
  const int head = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  const int b = nth_longest(a, head / a.H, gave_up + 1);   // a barrier
  const int h = head % a.H, bh = b * a.H + h, hk = h / (a.H / a.Hk);
  const int n0 = slice * NV;
  const int len = length_of(a, b), chunks = (len + kC - 1) / kC;
  const Rows rv = rows_of(a, b, h, a.H, a.Dv);
  // step i works on chunk chunks - 1 - i

  if (warp >= 8) {
    // ---- copies, in and out ----
    const int tid = threadIdx.x - 256;
    const Rows rk = rows_of(a, b, hk, a.Hk, a.D);
    const T* kp = static_cast<const T*>(a.k) + rk.base;
    const T* qp = static_cast<const T*>(a.q) + rk.base;
    const T* op = static_cast<const T*>(a.dout) + rv.base + n0;
    T* dvp = static_cast<T*>(a.dv) + rv.base + n0;
    const unsigned char* rec = a.rec + (long long)bh * a.chunks * Rec::bytes;
    auto landed = [&](uint32_t bar) {
      if (sizeof(T) == 2) ptx::cp_async_arrive(bar);
      else ptx::mbar_arrive(bar);
    };
    auto load = [&](int i) {   // the chain's part
      const int buf = i % NBUF, c = chunks - 1 - i;
      const uint32_t at = sbase + buf * Cfg::stage, bar = full + 8 * buf;
      const int rows = min(kC, len - c * kC);
      const long long t = (long long)c * kC;
      load_record<Rec::offP>(at, rec + (long long)c * Rec::bytes, bar, tid);
      mm::load_tile<T, kC, KD, kLoadThreads>(at + Cfg::offK, kLK, Cfg::kPlaneK, kp + t * rk.stride,
                                             rk.stride, rows, a.D, tid);
      landed(bar);
    };
    auto load_h = [&](int i) {   // the helpers'
      const int buf = i % NBUF, c = chunks - 1 - i;
      const uint32_t at = sbase + buf * Cfg::stage, bar = full_h + 8 * buf;
      const int rows = min(kC, len - c * kC);
      const long long t = (long long)c * kC;
      if (tid == 0) {
        const unsigned char* r = rec + (long long)c * Rec::bytes;
        ptx::mbar_expect_tx(bar, (int)sizeof(Gates) + Rec::offD - Rec::offP);
        ptx::bulk_load(at + Cfg::offH, r, sizeof(Gates), bar);
        ptx::bulk_load(at + Cfg::offP, r + Rec::offP, Rec::offD - Rec::offP, bar);
      }
      mm::load_tile<T, kC, KD, kLoadThreads>(at + Cfg::offQ, kLK, Cfg::kPlaneK, qp + t * rk.stride,
                                             rk.stride, rows, a.D, tid);
      mm::load_tile<T, kC, NV, kLoadThreads>(at + Cfg::offO, kLN, Cfg::kPlaneX, op + t * rv.stride,
                                             rv.stride, rows, a.Dv - n0, tid);
      landed(bar);
    };
    using I = Image<KD, PO>;
    const bool end = slice == a.slices - 1;
    const uint32_t sS = sbase + Cfg::offS, sY = sbase + Cfg::offY;
    for (int i = 0; i < NBUF && i < chunks; ++i) {
      load_h(i);
      load(i);
    }
    for (int i = 0; i < chunks; ++i) {
      const int buf = i % NBUF, c = chunks - 1 - i, rows = min(kC, len - c * kC);
      const Gates* gates = reinterpret_cast<const Gates*>(smem + buf * Cfg::stage);
      unsigned char* img = I::at(a, (long long)bh * a.chunks + c);
      if (i + NBUF < chunks) {
        ptx::bar_sync(kRevFreeH + buf, 256);
        load_h(i + NBUF);
      }
      ptx::bar_sync(kRevOut, 256);
      store_image<KD, PO, NV, KD>(img, I::offD, a.atoms, n0, end, sS, kLN, Cfg::kPlaneS, tid);
      ptx::bar_sync(kRevX, 256);
      store_image<KD, PO, NV, kC>(img, I::offR, a.atoms, n0, end, sY, kLN, Cfg::kPlaneX, tid);
      constexpr int V = NV / 8;
      for (int j = tid; j < kC * V; j += kLoadThreads) {
        const int row = j / V, c8 = j % V;
        if (row >= rows || n0 + c8 * 8 >= a.Dv) continue;
        const uint32_t at = sY + row * kLN + c8 * 16;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = 0.f;
#pragma unroll
        for (int p = PO - 1; p >= 0; --p) {
          const uint4 u = ptx::ld_shared_v4(at + p * Cfg::kPlaneX);
          x[0] += ptx::bf16_lo(u.x), x[1] += ptx::bf16_hi(u.x);
          x[2] += ptx::bf16_lo(u.y), x[3] += ptx::bf16_hi(u.y);
          x[4] += ptx::bf16_lo(u.z), x[5] += ptx::bf16_hi(u.z);
          x[6] += ptx::bf16_lo(u.w), x[7] += ptx::bf16_hi(u.w);
        }
        const float bt = gates->tok[row].y;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= bt;
        mm::Io<T>::store8(dvp + ((long long)c * kC + row) * rv.stride + c8 * 8, x);
      }
      if (i + 1 < chunks) ptx::bar_arrive(kRevRead, 256);
      if (i + NBUF < chunks) {
        ptx::bar_sync(kRevFree + buf, 256);
        load(i + NBUF);
      }
    }
    if (sizeof(T) == 2) ptx::cp_async_wait_all();
    if (!*gave_up) return;
    // what this thread has stored is void
    unsigned char* img = I::at(a, (long long)bh * a.chunks);
    void_image<KD, PO, NV, KD>(img, I::offD, a.atoms, n0, chunks, tid);
    void_image<KD, PO, NV, kC>(img, I::offR, a.atoms, n0, chunks, tid);
    constexpr int V = NV / 8;
    for (int c = 0; c < chunks; ++c)
      for (int j = tid; j < kC * V; j += kLoadThreads) {
        const int row = c * kC + j / V, c8 = j % V;
        const float x[8] = {void_value(), void_value(), void_value(), void_value(),
                            void_value(), void_value(), void_value(), void_value()};
        if (row < len && n0 + c8 * 8 < a.Dv)
          mm::Io<T>::store8(dvp + row * rv.stride + c8 * 8, x);
      }
    return;
  }

  const Share<KD, RT> sh(warp & 3);
  const int r = lane >> 2, c2 = (lane & 3) * 2, nw = sh.col;
  const uint32_t lane_at = mm::a_lane<false>(lane, kLN) + nw * 2;
  const uint32_t sS = sbase + Cfg::offS, sY = sbase + Cfg::offY, sX = sbase + Cfg::offX;
  const uint32_t sW = sbase + Cfg::offW;

  if (warp < 4) {
    // ---- the chain: rows sh.state + 16 m + r, r + 8 of dS ----
    float S[MS][2][4];
    const long long s_at = (long long)bh * a.D * a.Dv;
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = sh.state + 16 * m + r + 8 * i, col = n0 + nw + 8 * n + c2;
          float2 x = make_float2(0.f, 0.f);
          if (a.ds1 && row < a.D && col < a.Dv)
            x = *reinterpret_cast<const float2*>(a.ds1 + s_at + (long long)row * a.Dv + col);
          S[m][n][2 * i] = x.x;
          S[m][n][2 * i + 1] = x.y;
        }
    for (int i = 0; i < chunks; ++i) {
      const int buf = i % NBUF;
      const uint32_t sb = sbase + buf * Cfg::stage;
      const Gates* gates = reinterpret_cast<const Gates*>(smem + buf * Cfg::stage);
      const float4* aux =
          reinterpret_cast<const float4*>(smem + Cfg::offAux + (i & 1) * Cfg::aux) + threadIdx.x;
#pragma unroll
      for (int m = 0; m < MS; ++m)
        mm::store_tile<PC>(sS + (sh.state + 16 * m) * kLN + lane_at, Cfg::kPlaneS, S[m]);
      ptx::bar_arrive(kRevOut, 256);
      ptx::bar_sync(kRevS, 256);   // the helpers have seen the stage full and made its aux
      {
        float y[RT][2][4];
        mm::zero(y);
        mm::gemm<RT, 2, PI, PC, PC, false, true, KD / 16>(
            y, sh.rows(sb + Cfg::offK, kLK, Cfg::kPlaneK),
            mm::b_tile<true>(sS + nw * 2, kLN, Cfg::kPlaneS));
        if (i > 0) ptx::bar_sync(kRevRead, 256);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const int row = 16 * sh.tile[j] + r;
          const float z0 = gates->tok[row].z, z1 = gates->tok[row + 8].z;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float4 p = aux[(2 * j + n) * 128];
            y[j][n][0] = fmaf(z0, y[j][n][0], p.x);
            y[j][n][1] = fmaf(z0, y[j][n][1], p.y);
            y[j][n][2] = fmaf(z1, y[j][n][2], p.z);
            y[j][n][3] = fmaf(z1, y[j][n][3], p.w);
          }
          mm::store_tile<PC>(sY + 16 * sh.tile[j] * kLN + lane_at, Cfg::kPlaneX, y[j]);
        }
      }
      {
        float x[RT][1][2][4];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          mm::zero(x[j]);
          mm::gemm<1, 2, PC, PC, PC, true, true, 4>(
              x[j], mm::a_tri<true>(sb + Rec::offT, sh.tile[j]),
              mm::b_tile<true>(sY + 16 * sh.tile[j] * kLN + nw * 2, kLN, Cfg::kPlaneX),
              4 - sh.tile[j], [&] {
                if (j == 0) ptx::bar_sync(kRevChain, 128);
              });
        }
        ptx::bar_sync(kRevChain, 128);   // dX is read: its place takes dR
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const uint32_t at = 16 * sh.tile[j] * kLN + lane_at;
          mm::store_tile<PO>(sY + at, Cfg::kPlaneX, x[j][0]);
          const float be0 = gates->tok[16 * sh.tile[j] + r].x;
          const float be1 = gates->tok[16 * sh.tile[j] + r + 8].x;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][0][n][i] *= i < 2 ? be0 : be1;
          mm::store_tile<PC>(sX + at, Cfg::kPlaneX, x[j][0]);
        }
      }
      const float last = gates->last[0];
      float u[MS][2][4];
      mm::zero(u);
      mm::gemm<MS, 2, PI, PC, PC, true, true, kC / 16>(
          u, mm::a_tile<true>(sb + Cfg::offK + 2 * sh.state, kLK, Cfg::kPlaneK),
          mm::b_tile<true>(sX + nw * 2, kLN, Cfg::kPlaneX), kC / 16,
          [] { ptx::bar_sync(kRevX, 256); });
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const float4 p = aux[((RT + m) * 2 + n) * 128];
          S[m][n][0] = fmaf(last, S[m][n][0], p.x - u[m][n][0]);
          S[m][n][1] = fmaf(last, S[m][n][1], p.y - u[m][n][1]);
          S[m][n][2] = fmaf(last, S[m][n][2], p.z - u[m][n][2]);
          S[m][n][3] = fmaf(last, S[m][n][3], p.w - u[m][n][3]);
        }
      if (i + NBUF < chunks) ptx::bar_arrive(kRevFree + buf, 256);
    }
    if (a.ds0) {
      const bool bad = *gave_up;
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = sh.state + 16 * m + r + 8 * i, col = n0 + nw + 8 * n + c2;
            if (row < a.D && col < a.Dv)
              *reinterpret_cast<float2*>(a.ds0 + s_at + (long long)row * a.Dv + col) =
                  bad ? make_float2(void_value(), void_value())
                      : make_float2(S[m][n][2 * i], S[m][n][2 * i + 1]);
          }
    }
    // what follows takes this kernel's end for scan_kernel's, too
    if (blockIdx.x == 0) ptx::grid_dependency_wait();
    return;
  }

  // ---- the helpers ----
  const int tid = threadIdx.x - 128;
  // aux1 and aux2 of step i
  auto make_aux = [&](int i) {
    const int buf = i % NBUF;
    const uint32_t sb = sbase + buf * Cfg::stage;
    const Gates* gates = reinterpret_cast<const Gates*>(smem + buf * Cfg::stage + Cfg::offH);
    float4* aux = reinterpret_cast<float4*>(smem + Cfg::offAux + (i & 1) * Cfg::aux) + tid;
    wait_phase(full_h + 8 * buf, (i / NBUF) & 1, a.flag, gave_up);
    for (int j = tid; j < kC * NV / 2; j += 128) {
      const int row = j / (NV / 2), col = j % (NV / 2) * 2;
      const uint32_t at = row * kLN + col * 2;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int p = PI - 1; p >= 0; --p) {
        uint32_t u;
        asm volatile("ld.shared.u32 %0, [%1];"
                     : "=r"(u)
                     : "r"(sb + Cfg::offO + p * Cfg::kPlaneX + at));
        x += ptx::bf16_lo(u);
        y += ptx::bf16_hi(u);
      }
      const float wt = gates->tok[row].w;
      mm::store_pair<PC>(sW + at, Cfg::kPlaneX, wt * x, wt * y);
    }
    ptx::bar_sync(kRevHelp, 128);
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      float p[1][2][4];
      mm::zero(p);
      mm::gemm<1, 2, PC, PI, PC, true, true, 4>(
          p, mm::a_tri<true>(sb + Cfg::offP, sh.tile[j]),
          mm::b_tile<true>(sb + Cfg::offO + 16 * sh.tile[j] * kLN + nw * 2, kLN, Cfg::kPlaneX),
          4 - sh.tile[j]);
#pragma unroll
      for (int n = 0; n < 2; ++n)
        aux[(2 * j + n) * 128] = make_float4(p[0][n][0], p[0][n][1], p[0][n][2], p[0][n][3]);
    }
    float u[MS][2][4];
    mm::zero(u);
    mm::gemm<MS, 2, PI, PC, PC, true, true, kC / 16>(
        u, mm::a_tile<true>(sb + Cfg::offQ + 2 * sh.state, kLK, Cfg::kPlaneK),
        mm::b_tile<true>(sW + nw * 2, kLN, Cfg::kPlaneX));
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
      for (int n = 0; n < 2; ++n)
        aux[((RT + m) * 2 + n) * 128] =
            make_float4(u[m][n][0], u[m][n][1], u[m][n][2], u[m][n][3]);
    if (i + NBUF < chunks) ptx::bar_arrive(kRevFreeH + buf, 256);
    ptx::bar_sync(kRevHelp, 128);   // sW may be written again
  };
  if (chunks > 0) make_aux(0);
  for (int i = 0; i < chunks; ++i) {
    wait_phase(full + 8 * (i % NBUF), (i / NBUF) & 1, a.flag, gave_up);   // for the chain
    ptx::bar_sync(kRevS, 256);
    if (i + 1 < chunks) make_aux(i + 1);
  }
}

// ---- a chunk's gradients in fp32 ---------------------------------------------------------
//
// One CTA of sixteen warps per (chunk, head). Warp (m, ch) has rows 16 m of the
// chunk, a quarter of the key columns of dq and dk, and block (m, ch) of the
// products within the chunk. The products with S and dS' run over the value
// columns in slices of NV, one after another (K and Q of three planes leave no
// room for a second slice); then the products within the chunk follow from EP and
// F in shared memory. What it has to read is mostly S and dS' (12 D Dv bytes a
// chunk in three planes each, and 768 Dv of X and dR, where q, k, v, dout and the
// gradients are 4 (4 D + 3 Dv) 64); what it waits for is the latency of its own
// chain of small products, hence the many warps. CTAs go by chunks, then heads:
// the first chunks' dS' and dR were written last and are in the L2 still (of a
// call of three heads of 333 tokens 69 us became 66).
constexpr int kSums = 25 * kC + 16;   // floats: the sums that a chunk's dbeta and dg are made of

template <int KD, int NV, int PO>
struct GradCfg {
  using T = float;
  static constexpr int PI = mm::Io<T>::kPlanes;
  static constexpr int kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  static constexpr int kLN = (NV + 8) * 2, kPlaneS = KD * kLN, kPlaneX = kC * kLN;
  static constexpr int offK = 0, offQ = PI * kPlaneK, offStage = 2 * PI * kPlaneK;
  // a slice: S, dS', dO, X, dR, and V as it is
  static constexpr int offS = 0, offD = PO * kPlaneS, offO = 2 * PO * kPlaneS;
  static constexpr int offX = offO + PI * kPlaneX, offR = offX + PO * kPlaneX;
  static constexpr int offV = offR + PO * kPlaneX;
  static constexpr int stage = offV + kC * NV * (int)sizeof(T);
  // EP and F take its place
  static constexpr int tri = 2 * PO * mm::kTriPlane;
  static constexpr int offGate = offStage + (stage > tri ? stage : tri);
  static constexpr int offDec = offGate + (int)sizeof(Gates);
  static constexpr int offSum = offDec + (int)sizeof(Decays);
  static constexpr int bytes = offSum + kSums * 4;
  static constexpr int threads = 512;
};

// What both kernels below do with a chunk once the sums over the value columns
// are there, by sixteen warps. `smem` offsets: of K and Q (row stride kLK), of
// the tiles EP and F.
struct Within {
  unsigned char* smem;
  uint32_t sbase;
  int offK, offQ, offE;
  const Gates* gates;
  const Decays* dec;
  // sums of rows, by quarter of the columns: [0 ..] q.dq, [4 ..] k.ki, [8 ..]
  // k.ko, [12 ..] M along rows, [20 ..] for dbeta; [16 ..] M along columns, by row
  // tile; [24] dR.v; then <S, dS'> by warp. Of a diagonal block M's row sums give
  // way to what dg takes of it, sum_{i >= t > j} M_ij by t.
  float* sums;
};

// Block (m, ch) of K K^T and Q K^T.
template <int KD, int PI, int PO>
__device__ __forceinline__ void key_products(const Within& x, float (&acc)[2][2][4]) {
  constexpr int kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  constexpr bool kApart = PI == 3;
  const int warp = threadIdx.x >> 5, m = warp & 3, ch = warp >> 2;
  const uint32_t sK = x.sbase + x.offK;
  mm::zero(acc);
  if (ch > m) return;
  mm::Operand ka = mm::a_tile<false>(sK + 16 * m * kLK, kLK, kPlaneK);
  ka.tile = x.offQ - x.offK;
  mm::gemm<2, 2, PI, PI, PO, false, false, KD / 16, 2, kApart>(
      acc, ka, mm::b_tile<false>(sK + 16 * ch * kLK, kLK, kPlaneK));
}

// EP and F from that and the block of dO X^T and dR X^T, and their sums.
template <int PO>
__device__ __forceinline__ void make_within(const Within& x, float scale,
                                            const float (&acc)[2][2][4], const float (&dP)[1][2][4],
                                            const float (&dA)[1][2][4]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m = warp & 3, ch = warp >> 2, r = lane >> 2, c2 = (lane & 3) * 2;
  const uint32_t sE = x.sbase + x.offE, sF = sE + PO * mm::kTriPlane;
  const Gates* gates = x.gates;
  const Decays* dec = x.dec;
  float* sums = x.sums;
  if (ch <= m) {
    float row_sum[2] = {0.f, 0.f}, beta_sum[2] = {0.f, 0.f};
    float M[2][2][2];   // of a diagonal block: column tile, row, column
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int cc = 8 * n + c2, col = 16 * ch + cc;
      float col_sum[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = r + 8 * i, row = 16 * m + rr;
        const float bt = gates->tok[row].y;
        float ep[2], f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const bool in = ch < m || cc + e <= rr, below = ch < m || cc + e < rr;
          float E = 0.f;
          if (ch < m) E = dec->up[row] * dec->down[m - 1][col + e];
          else if (in) E = expf((float)(dec->G[row] - dec->G[col + e]));
          ep[e] = in ? scale * E * dP[0][n][2 * i + e] : 0.f;
          const float ea = below ? -E * dA[0][n][2 * i + e] : 0.f;
          const float kk = acc[0][n][2 * i + e];
          f[e] = bt * ea;
          const float mix = (in ? ep[e] * acc[1][n][2 * i + e] : 0.f) + (below ? f[e] * kk : 0.f);
          M[n][i][e] = mix;
          row_sum[i] += mix;
          col_sum[e] += mix;
          if (below) beta_sum[i] += ea * kk;
        }
        const int o = mm::tri_block(m, ch) + mm::tri_at(rr, cc);
        mm::store_pair<PO>(sE + o, mm::kTriPlane, ep[0], ep[1]);
        mm::store_pair<PO>(sF + o, mm::kTriPlane, f[0], f[1]);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float y = col_sum[e];
        y += __shfl_xor_sync(0xffffffffu, y, 4);
        y += __shfl_xor_sync(0xffffffffu, y, 8);
        y += __shfl_xor_sync(0xffffffffu, y, 16);
        if (r == 0) sums[(16 + m) * kC + col + e] = y;
      }
    }
    if (ch == m) {
      // sum over the rows from t on, then over the columns before t
      row_sum[0] = row_sum[1] = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lo = M[n][0][e], hi = M[n][1][e];   // rows r and r + 8
#pragma unroll
          for (int o = 4; o < 32; o *= 2) {
            const float u = __shfl_down_sync(0xffffffffu, lo, o);
            const float v = __shfl_down_sync(0xffffffffu, hi, o);
            if (lane + o < 32) lo += u, hi += v;
          }
          lo += __shfl_sync(0xffffffffu, hi, lane & 3);
          const int cc = 8 * n + c2 + e;
          if (cc < r) row_sum[0] += lo;
          if (cc < r + 8) row_sum[1] += hi;
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float y = row_sum[i], z = beta_sum[i];
      y += __shfl_xor_sync(0xffffffffu, y, 1);
      y += __shfl_xor_sync(0xffffffffu, y, 2);
      z += __shfl_xor_sync(0xffffffffu, z, 1);
      z += __shfl_xor_sync(0xffffffffu, z, 2);
      if ((lane & 3) == 0) {
        sums[(12 + ch) * kC + 16 * m + r + 8 * i] = y;
        sums[(20 + ch) * kC + 16 * m + r + 8 * i] = z;
      }
    }
  } else if (lane < 16) {
    sums[(12 + ch) * kC + 16 * m + lane] = 0.f;
    sums[(20 + ch) * kC + 16 * m + lane] = 0.f;
    sums[(16 + m) * kC + 16 * ch + lane] = 0.f;
  }
}

// A row of NT 8-column tiles, of whose every tile lane t of the quad has columns
// 2t and 2t + 1, to bf16 memory: the quad's lanes trade words so that each has
// 8 (or 4) columns in a row to store. All lanes take part; `in`: the row exists,
// `cols`: how many of its columns do (a multiple of 8).
template <int NT>
__device__ __forceinline__ void store_row(bf16* p, const float (&x)[NT][4], int half, bool in,
                                          int cols) {
  static_assert(NT == 2 || NT == 4, "the trades below");
  const int t = threadIdx.x & 3;
  uint32_t w[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) w[n] = ptx::pack_bf16x2(x[n][2 * half], x[n][2 * half + 1]);
  auto trade = [&](uint32_t& lo, uint32_t& hi, int bit) {
    const bool up = t & bit;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, up ? lo : hi, bit);
    if (up) lo = y;
    else hi = y;
  };
  trade(w[0], w[1], 1);
  if constexpr (NT == 4) {
    trade(w[2], w[3], 1);
    trade(w[0], w[2], 2);
    trade(w[1], w[3], 2);
    if (in && 8 * t < cols)
      *reinterpret_cast<uint4*>(p + 8 * t) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    const int d = 8 * (t & 1) + 4 * (t >> 1);
    if (in && 8 * (t & 1) < cols) *reinterpret_cast<uint2*>(p + d) = make_uint2(w[0], w[1]);
  }
}

// dq and dk: the products with EP and F on top of what `dq` and `ko` have, and
// their stores; then dbeta and dg from the sums. All of it after a barrier.
template <typename T, int KD, int PO>
__device__ __forceinline__ void finish(const Args& a, const Within& x, int bh, int chunk, int rows,
                                       float (&dq)[1][KD / 32][4], float (&ko)[1][KD / 32][4]) {
  constexpr int PI = mm::Io<T>::kPlanes, NTK = KD / 32, kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  constexpr bool kApart = PI == 3;
  constexpr int kDepth = PI == 1 ? 2 : 1;   // fp32's three planes leave no registers for two
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m = warp & 3, ch = warp >> 2, r = lane >> 2, c2 = (lane & 3) * 2;
  const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const long long t0 = (long long)chunk * kC;
  const Rows rk = rows_of(a, b, hk, a.Hk, a.D);
  const uint32_t sK = x.sbase + x.offK, sQ = x.sbase + x.offQ;
  const uint32_t sE = x.sbase + x.offE, sF = sE + PO * mm::kTriPlane;
  const Gates* gates = x.gates;
  const Decays* dec = x.dec;
  const float* sums = x.sums;
  // dq += EP K;  dk += EP^T Q + F^T K + F K
  {
    const int at = ch * (KD / 4) * 2;
    const mm::Operand bK = mm::b_tile<true>(sK + at, kLK, kPlaneK);
    const mm::Operand bKm = mm::b_tile<true>(sK + 16 * m * kLK + at, kLK, kPlaneK);
    const mm::Operand bQm = mm::b_tile<true>(sQ + 16 * m * kLK + at, kLK, kPlaneK);
    mm::gemm<1, NTK, PO, PI, PO, false, true, 4, kDepth, kApart>(dq, mm::a_tri<false>(sE, m), bK, m + 1);
    mm::gemm<1, NTK, PO, PI, PO, false, true, 4, kDepth, kApart>(ko, mm::a_tri<false>(sF, m), bK, m + 1);
    mm::gemm<1, NTK, PO, PI, PO, true, true, 4, kDepth, kApart>(ko, mm::a_tri<true>(sE, m), bQm, 4 - m);
    mm::gemm<1, NTK, PO, PI, PO, true, true, 4, kDepth, kApart>(ko, mm::a_tri<true>(sF, m), bKm, 4 - m);
  }
  const bool shared = a.Hk != a.H;
  const int d0 = ch * (KD / 4);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * m + r + 8 * i;
    const bool in = row < rows;
    const long long o = shared ? ((long long)bh * a.N + t0 + row) * a.D
                               : rk.base + (t0 + row) * rk.stride;
    if (!shared && sizeof(T) == 2) {
      store_row<NTK>(static_cast<bf16*>(a.dq) + o + d0, dq[0], i, in, a.D - d0);
      store_row<NTK>(static_cast<bf16*>(a.dk) + o + d0, ko[0], i, in, a.D - d0);
      continue;
    }
#pragma unroll
    for (int n = 0; n < NTK; ++n) {
      const int d = d0 + 8 * n + c2;
      if (!in || d >= a.D) continue;
      float* const q = shared ? a.wdq : static_cast<float*>(a.dq);
      float* const k = shared ? a.wdk : static_cast<float*>(a.dk);
      *reinterpret_cast<float2*>(q + o + d) = make_float2(dq[0][n][2 * i], dq[0][n][2 * i + 1]);
      *reinterpret_cast<float2*>(k + o + d) = make_float2(ko[0][n][2 * i], ko[0][n][2 * i + 1]);
    }
  }

  // dbeta and dg: one warp, lane l has tokens 2l and 2l + 1
  if (warp == 0) {
    float in[2], out[2], row[2], col[2];
    const int tile = lane >> 3;
    const Rows rg = rows_of(a, b, h, a.H, 1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      const float4 g = gates->tok[i];
      float y[4];   // four sums of the token, each over four parts
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float* s = sums + (j == 3 ? 20 : 4 * j) * kC + i;
        y[j] = (s[0] + s[kC]) + (s[2 * kC] + s[3 * kC]);
      }
      in[e] = g.w * y[0] - g.x * y[1];
      out[e] = g.z * y[2];
      if (i < rows) {
        const float db = sums[24 * kC + i] - expf((float)dec->G[i]) * y[1] + y[3];
        mm::Io<T>::store(static_cast<T*>(a.dbeta) + rg.base + (t0 + i) * rg.stride, db);
      }
      // of the blocks left of the diagonal one in this row tile, and of those
      // below it in this column tile
      row[e] = col[e] = 0.f;
#pragma unroll
      for (int j = 0; j < 3; ++j) {
        if (j < tile) row[e] += sums[(12 + j) * kC + i];
        if (3 - j > tile) col[e] += sums[(16 + 3 - j) * kC + i];
      }
    }
    // what lies below this tile's row and left of its column: the blocks (2, 0)
    // and (3, 0) for tile 1, (3, 0) and (3, 1) for tile 2
    float part[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      part[j] = sums[(12 + j) * kC + 2 * lane] + sums[(12 + j) * kC + 2 * lane + 1];
#pragma unroll
      for (int o = 1; o < 8; o *= 2) part[j] += __shfl_xor_sync(0xffffffffu, part[j], o);
    }
    const float b20 = __shfl_sync(0xffffffffu, part[0], 16);
    const float b30 = __shfl_sync(0xffffffffu, part[0], 24);
    const float b31 = __shfl_sync(0xffffffffu, part[1], 24);
    float dot = 0.f;
    for (int j = 0; j < 16; ++j) dot += sums[25 * kC + j];
    float end = gates->last[0] * dot;
    if (tile == 1) end += b20 + b30;
    if (tile == 2) end += b30 + b31;
    // sums over the tokens from this lane's on, of `in` to the chunk's end and of
    // `row` to the tile's; and over those before it
    float in_t = in[0] + in[1], row_t = row[0] + row[1];
    float out_t = out[0] + out[1], col_t = col[0] + col[1];
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const float u = __shfl_down_sync(0xffffffffu, in_t, o);
      const float v = __shfl_up_sync(0xffffffffu, out_t, o);
      if (lane + o < 32) in_t += u;
      if (lane >= o) out_t += v;
      if (o < 8) {
        const float w = __shfl_down_sync(0xffffffffu, row_t, o, 8);
        const float z = __shfl_up_sync(0xffffffffu, col_t, o, 8);
        if ((lane & 7) + o < 8) row_t += w;
        if ((lane & 7) >= o) col_t += z;
      }
    }
    // without this lane's own two tokens
    float after = __shfl_down_sync(0xffffffffu, in_t, 1);
    float rest = __shfl_down_sync(0xffffffffu, row_t, 1, 8);
    float before = __shfl_up_sync(0xffffffffu, out_t, 1);
    float left = __shfl_up_sync(0xffffffffu, col_t, 1, 8);
    if (lane == 31) after = 0.f;
    if ((lane & 7) == 7) rest = 0.f;
    if (lane == 0) before = 0.f;
    if ((lane & 7) == 0) left = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 2 * lane + e;
      float dg = e == 0 ? (in_t + before) + (row_t + left)
                        : (after + in[1] + before + out[0]) + (rest + row[1] + left + col[0]);
      dg += end + sums[(12 + tile) * kC + i];
      if (i < rows)
        mm::Io<T>::store(static_cast<T*>(a.dg) + rg.base + (t0 + i) * rg.stride, dg);
    }
  }
}

template <int KD, int NV, int PC, int PO>
__global__ void __launch_bounds__(512, 1) gradient_kernel(const Args a) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  using T = float;
  using Cfg = GradCfg<KD, NV, PO>;
  using Rec = Record<PC, PC>;
  constexpr int kT = Cfg::threads;
  constexpr bool kApart = Cfg::PI == 3;
  constexpr int PI = Cfg::PI, NTK = KD / 32, kLK = Cfg::kLK, kLN = Cfg::kLN;
  extern __shared__ __align__(16) unsigned char smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t sK = sbase + Cfg::offK, sQ = sbase + Cfg::offQ;
  const int heads = gridDim.x / a.chunks, chunk = blockIdx.x / heads, bh = blockIdx.x % heads;
  const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int rows = min(kC, length_of(a, b) - chunk * kC);
  if (rows <= 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int m = warp & 3, ch = warp >> 2, r = lane >> 2, c2 = (lane & 3) * 2;
  const long long t0 = (long long)chunk * kC, at = (long long)bh * a.chunks + chunk;
  const Rows rk = rows_of(a, b, hk, a.Hk, a.D), rv = rows_of(a, b, h, a.H, a.Dv);
  const T* op = static_cast<const T*>(a.dout) + rv.base + t0 * rv.stride;
  const T* vp = static_cast<const T*>(a.v) + rv.base + t0 * rv.stride;

  using I = Image<KD, PO>;
  const unsigned char* img = I::at(a, at);
  auto load_slice = [&](int s) {
    const uint32_t st = sbase + Cfg::offStage;
    const int n0 = s * NV;
    // rows of NV columns out of the image's tiles: all within one atom
    auto load_image = [&](int dst, int plane, int tile, int rows_in_tile) {
      constexpr int V = NV / 8;
      for (int i = tid; i < PO * rows_in_tile * V; i += kT) {
        const int row = i / V, n = n0 / 8 + i % V, p = row / rows_in_tile;
        mm::cp_async16(st + dst + p * plane + (row - p * rows_in_tile) * kLN + i % V * 16,
                       img + n / 8 * I::atom + tile + I::vec(row, n % 8), true);
      }
    };
    load_image(Cfg::offS, Cfg::kPlaneS, I::offS, KD);
    load_image(Cfg::offD, Cfg::kPlaneS, I::offD, KD);
    load_image(Cfg::offX, Cfg::kPlaneX, I::offX, kC);
    load_image(Cfg::offR, Cfg::kPlaneX, I::offR, kC);
    mm::load_tile<T, kC, NV, kT>(st + Cfg::offO, kLN, Cfg::kPlaneX, op + n0, rv.stride, rows,
                                 a.Dv - n0, tid);
    constexpr int E = 16 / (int)sizeof(T), VV = NV / E;
    if (tid < kC * VV) {
      const int row = tid / VV, col = tid % VV * E;
      const bool in = row < rows && n0 + col < a.Dv;
      mm::cp_async16(st + Cfg::offV + tid * 16, in ? vp + row * rv.stride + n0 + col : vp, in);
    }
  };
  static_assert(kC * NV * sizeof(T) / 16 <= kT, "a vector of V per thread");

  const int slices = (a.Dv + NV - 1) / NV;
  const unsigned char* rec = a.rec + at * Rec::bytes;
  mm::copy_bytes<(int)sizeof(Gates), kT>(sbase + Cfg::offGate, rec, tid);
  mm::copy_bytes<(int)sizeof(Decays), kT>(sbase + Cfg::offDec, rec + Rec::offD, tid);
  mm::load_tile<T, kC, KD, kT>(sK, kLK, Cfg::kPlaneK,
                               static_cast<const T*>(a.k) + rk.base + t0 * rk.stride, rk.stride,
                               rows, a.D, tid);
  mm::load_tile<T, kC, KD, kT>(sQ, kLK, Cfg::kPlaneK,
                               static_cast<const T*>(a.q) + rk.base + t0 * rk.stride, rk.stride,
                               rows, a.D, tid);
  load_slice(0);

  float dq[1][NTK][4], ko[1][NTK][4], ki[1][NTK][4];   // dO S^T, X dS'^T, dR S^T
  float dP[1][2][4], dA[1][2][4];                      // block (m, ch) of dO X^T, dR X^T
  mm::zero(dq);
  mm::zero(ko);
  mm::zero(ki);
  mm::zero(dP);
  mm::zero(dA);
  const bool low = ch <= m;       // the block lies on or below the diagonal
  float rv_sum = 0.f, ss = 0.f;   // dR_i . v_i of row tid / 8; <S, dS'>
  for (int s = 0; s < slices; ++s) {
    ptx::cp_async_wait_all();
    __syncthreads();
    const uint32_t st = sbase + Cfg::offStage;
    const unsigned char* stp = smem + Cfg::offStage;
    const mm::Operand aO = mm::a_tile<false>(st + Cfg::offO + 16 * m * kLN, kLN, Cfg::kPlaneX);
    const mm::Operand aX = mm::a_tile<false>(st + Cfg::offX + 16 * m * kLN, kLN, Cfg::kPlaneX);
    const mm::Operand aR = mm::a_tile<false>(st + Cfg::offR + 16 * m * kLN, kLN, Cfg::kPlaneX);
    const int d0 = ch * (KD / 4) * kLN;
    const mm::Operand bS = mm::b_tile<false>(st + Cfg::offS + d0, kLN, Cfg::kPlaneS);
    const mm::Operand bD = mm::b_tile<false>(st + Cfg::offD + d0, kLN, Cfg::kPlaneS);
    mm::gemm<1, NTK, PI, PO, PO, false, false, NV / 16, 1, kApart>(dq, aO, bS);
    mm::gemm<1, NTK, PO, PO, PO, false, false, NV / 16, 1, kApart>(ki, aR, bS);
    mm::gemm<1, NTK, PO, PO, PO, false, false, NV / 16, 1, kApart>(ko, aX, bD);
    if (low) {
      const mm::Operand bX = mm::b_tile<false>(st + Cfg::offX + 16 * ch * kLN, kLN, Cfg::kPlaneX);
      mm::gemm<1, 2, PI, PO, PO, false, false, NV / 16, 1, kApart>(dP, aO, bX);
      mm::gemm<1, 2, PO, PO, PO, false, false, NV / 16, 1, kApart>(dA, aR, bX);
    }
    {   // eight threads to a row, NV / 8 columns each
      const int row = tid >> 3, col = (tid & 7) * (NV / 8);
#pragma unroll
      for (int j = 0; j < NV / 8; j += 2) {
        const float2 v =
            mm::Io<T>::load2s(reinterpret_cast<const T*>(stp + Cfg::offV) + row * NV + col + j);
        float x = 0.f, y = 0.f;
#pragma unroll
        for (int p = PO - 1; p >= 0; --p) {
          const uint32_t u = *reinterpret_cast<const uint32_t*>(
              stp + Cfg::offR + p * Cfg::kPlaneX + row * kLN + (col + j) * 2);
          x += ptx::bf16_lo(u);
          y += ptx::bf16_hi(u);
        }
        rv_sum += x * v.x + y * v.y;
      }
    }
#pragma unroll
    for (int j = tid; j < KD * NV / 2; j += kT) {
      const unsigned char* e = stp + (j / (NV / 2)) * kLN + j % (NV / 2) * 4;
      float x = 0.f, y = 0.f, u = 0.f, v = 0.f;
#pragma unroll
      for (int p = PO - 1; p >= 0; --p) {
        const uint32_t f = *reinterpret_cast<const uint32_t*>(e + Cfg::offS + p * Cfg::kPlaneS);
        const uint32_t g = *reinterpret_cast<const uint32_t*>(e + Cfg::offD + p * Cfg::kPlaneS);
        x += ptx::bf16_lo(f);
        y += ptx::bf16_hi(f);
        u += ptx::bf16_lo(g);
        v += ptx::bf16_hi(g);
      }
      ss += x * u + y * v;
    }
    __syncthreads();   // the slice's place is free
    if (s + 1 < slices) load_slice(s + 1);
  }

  const Gates* gates = reinterpret_cast<const Gates*>(smem + Cfg::offGate);
  const Decays* dec = reinterpret_cast<const Decays*>(smem + Cfg::offDec);
  float* sums = reinterpret_cast<float*>(smem + Cfg::offSum);
  Within x{smem, sbase, Cfg::offK, Cfg::offQ, Cfg::offStage, gates, dec, sums};
  float keys[2][2][4];
  key_products<KD, PI, PO>(x, keys);
  make_within<PO>(x, a.scale, keys, dP, dA);

  // the dots with q and k, then the factors of the rows
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = 16 * m + r + 8 * i;
    const float4 g = gates->tok[row];
    float x = 0.f, y = 0.f, z = 0.f;
#pragma unroll
    for (int n = 0; n < NTK; ++n) {
      const int o = row * kLK + (ch * (KD / 4) + 8 * n + c2) * 2;
      float q0 = 0.f, q1 = 0.f, k0 = 0.f, k1 = 0.f;
#pragma unroll
      for (int p = PI - 1; p >= 0; --p) {
        const uint32_t u = *reinterpret_cast<const uint32_t*>(smem + Cfg::offQ + p * Cfg::kPlaneK + o);
        const uint32_t v = *reinterpret_cast<const uint32_t*>(smem + Cfg::offK + p * Cfg::kPlaneK + o);
        q0 += ptx::bf16_lo(u);
        q1 += ptx::bf16_hi(u);
        k0 += ptx::bf16_lo(v);
        k1 += ptx::bf16_hi(v);
      }
      x += q0 * dq[0][n][2 * i] + q1 * dq[0][n][2 * i + 1];
      y += k0 * ki[0][n][2 * i] + k1 * ki[0][n][2 * i + 1];
      z += k0 * ko[0][n][2 * i] + k1 * ko[0][n][2 * i + 1];
#pragma unroll
      for (int e = 2 * i; e < 2 * i + 2; ++e) {
        dq[0][n][e] *= g.w;
        ko[0][n][e] = g.z * ko[0][n][e] - g.x * ki[0][n][e];   // dk so far
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
      x += __shfl_xor_sync(0xffffffffu, x, o);
      y += __shfl_xor_sync(0xffffffffu, y, o);
      z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    if ((lane & 3) == 0) {
      sums[(0 + ch) * kC + row] = x;
      sums[(4 + ch) * kC + row] = y;
      sums[(8 + ch) * kC + row] = z;
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o *= 2) rv_sum += __shfl_xor_sync(0xffffffffu, rv_sum, o);
  if ((tid & 7) == 0) sums[24 * kC + (tid >> 3)] = rv_sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (lane == 0) sums[25 * kC + warp] = ss;
  __syncthreads();

  finish<T, KD, PO>(a, x, bh, chunk, rows, dq, ko);
}

// ---- the same in bf16, its sums over the value columns on tcgen05 ------------------------
//
// A chunk and head at a time. The operands lie in shared memory as 64-column
// atoms of 128-byte rows (128-byte swizzle), one atom per 64 value columns:
// rows dO, R0, R1, X0, X1 (64 each; dR and X in two planes), then the planes of
// S and of dS' (KD rows each). Tiles that follow one another stack to the 128
// rows of one product, so the planes' products come with few instructions:
//     D1 = [dO; R0] (S0 + S1)^T      dO S^T, and of dR S^T what R0 gives
//     D4 = [R1; .]  S0^T             the rest of dR S^T
//     D2 = [X0; X1] (dS'0 + dS'1)^T  X dS'^T as the sum of the two halves
//     D3 = [dO; R0] (X0 + X1)^T      dP, and of dR X^T what R0 gives
//     D5 = [R1; .]  X0^T             the rest of it
// ("." is whatever follows; its rows are not read.) All accumulators are in
// tensor memory: 3 KD + 128 columns. One thread issues the 32 products of an
// atom while the others sum <S, dS'> and dR.v from the same tiles. Against the
// warp-level products of gradient_kernel (11,000 cycles of the tensor pipes a
// chunk at D = 128) they take about 3,000. What bounds the kernel is that one
// CTA, which fills the SM's shared memory, goes through its stages one by one:
// of 23,000 cycles at D = 128 3,000 wait for the first atom, 7,000 are the two
// atoms' products and copies, 3,000 the way out of tensor memory, 2,000
// make_within and 5,500 finish (32 heads of 4096 tokens: 227 us, of which the
// 256 KB a chunk are 85 at the measured bandwidth; 237 with dlog_decay's rectangles
// of pairs, which came later). A cluster per group of
// shared heads that adds dq and dk up through its shared memory, instead of
// shared_heads_kernel (27 us), was slower: 653 us a call against 646 with two
// heads to a group, 773 against 636 with eight.
template <int KD>
struct GradTcCfg {
  static constexpr int kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  using I = Image<KD, 2>;
  static constexpr int image = 8192;   // dO, then an atom of the image
  static constexpr int tileR0 = image + I::offR, tileR1 = tileR0 + 8192;
  static constexpr int tileX0 = image + I::offX, tileX1 = tileX0 + 8192;
  static constexpr int tileS = image + I::offS, tileD = image + I::offD;
  static constexpr int atom = image + I::atom;
  static_assert(tileX0 == tileR1 + 8192 && tileS == tileX1 + 8192, "tiles that stack");
  // K, Q, EP and F: in the first atom's place once its products are done, or in
  // the second's if there is but one
  static constexpr int offQ = kPlaneK, offE = 2 * kPlaneK;
  static_assert(offE + 4 * mm::kTriPlane <= atom, "they fit");
  // fp32 sums, in the place of the last atom: dq and dk [64][KD + 4], dP and dA
  // [64][68]
  static constexpr int pitch = KD + 4, pitchC = kC + 4;
  static constexpr int offDK = kC * pitch * 4, offP = 2 * offDK, offA = offP + kC * pitchC * 4;
  static_assert(offA + kC * pitchC * 4 <= atom, "they fit");
  static constexpr int offGate = 2 * atom;
  static constexpr int kDecays = (int)(sizeof(Gates) + sizeof(Decays));   // two chunks'
  static constexpr int offSum = offGate + 2 * kDecays;
  static constexpr int offBar = offSum + kSums * 4;
  static constexpr int bytes = 1024 + offBar + 48;   // from a multiple of 1024 on
  static constexpr int threads = 512, columns = 512;   // of tensor memory: a power of two
  // A CTA per SM that goes through the chunks, the next one's first atom on its
  // way during finish; else one per chunk. At D 64 that takes 5 to 7 % off a
  // backward call; at D 128, where a chunk's second atom is waited for all the
  // same and the loop's state is spilled, it adds 7 %.
  static constexpr bool kItems = KD == 64;
};

template <int KD, int PC>
__global__ void __launch_bounds__(512, 1) gradient_tc_kernel(const Args a) {
  ptx::launch_dependents();
  ptx::grid_dependency_wait();
  using Cfg = GradTcCfg<KD>;
  using Rec = Record<PC, PC>;
  constexpr int kLK = Cfg::kLK, PO = 2, NC = KD / 4, NTK = KD / 32;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw), sbase = (raw + 1023u) & ~1023u;
  unsigned char* smem = smem_raw + (sbase - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int heads = a.B * a.H, total = heads * a.chunks;   // items: chunks, then heads
  // the first item from `item` on, by steps of the grid, that has tokens
  auto live = [&](int item) {
    while (item < total && length_of(a, item % heads / a.H) <= item / heads * kC)
      item = total - item > (int)gridDim.x ? item + (int)gridDim.x : total;
    return item;
  };
  int item = live(blockIdx.x);
  if (item >= total) return;
  const int atoms = a.atoms;   // 1 or 2
  // mbarriers per atom: of its copy, and of its products
  const uint32_t landed = sbase + Cfg::offBar, done = landed + 16;
  volatile int* gave_up = reinterpret_cast<volatile int*>(smem + Cfg::offBar + 32);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Cfg::offBar + 40);
  if (tid == 0) {
    for (int t = 0; t < 4; ++t) ptx::mbar_init(landed + 8 * t, 1);
    *gave_up = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async();
  }

  // this thread's place in every tile: row r0 (+ 64 ..), vector c, swizzled
  const int r0 = tid >> 3, c = tid & 7;
  const uint32_t place = r0 * 128 + ((c ^ (r0 & 7)) << 4);
  // atom t of an item to one of the two places
  auto load_atom = [&](int of, int t, int to) {
    const int bh = of % heads, b = bh / a.H;
    const long long t0 = (long long)(of / heads) * kC;
    const Rows rv = rows_of(a, b, bh % a.H, a.H, a.Dv);
    const bf16* op = static_cast<const bf16*>(a.dout) + rv.base + t0 * rv.stride;
    const int n = 64 * t + 8 * c;
    const bool in = r0 < length_of(a, b) - t0 && n < a.Dv;
    mm::cp_async16(sbase + to + place, in ? op + r0 * rv.stride + n : op, in);
    if (tid == 0) {
      const unsigned char* img = Cfg::I::at(a, (long long)bh * a.chunks + of / heads);
      ptx::mbar_expect_tx(landed + 8 * t, Cfg::I::atom);
      ptx::bulk_load(sbase + to + Cfg::image, img + t * Cfg::I::atom, Cfg::I::atom,
                     landed + 8 * t);
    }
  };
  // what an item begins with: its first atom, and its factors
  auto begin = [&](int of, int to, int odd) {
    load_atom(of, 0, to);
    const unsigned char* rec =
        a.rec + ((long long)(of % heads) * a.chunks + of / heads) * Rec::bytes;
    const uint32_t at = sbase + Cfg::offGate + odd * Cfg::kDecays;
    mm::copy_bytes<(int)sizeof(Gates), 512>(at, rec, tid);
    mm::copy_bytes<(int)sizeof(Decays), 512>(at + (int)sizeof(Gates), rec + Rec::offD, tid);
    ptx::cp_async_commit();
  };
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(s_tmem), Cfg::columns);
    ptx::tmem_relinquish();
  }
  __syncthreads();   // the mbarriers are ready for everybody
  uint32_t tmem = 0;
  int first = 0;   // the place of the item's first atom
  begin(item, first, 0);
#pragma unroll 1
  for (int odd = 0; item < total; odd ^= 1) {
    const int chunk = item / heads, bh = item % heads;
    const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
    const int rows = min(kC, length_of(a, b) - chunk * kC);
    const long long t0 = (long long)chunk * kC;
    const Rows rk = rows_of(a, b, hk, a.Hk, a.D), rv = rows_of(a, b, h, a.H, a.Dv);
    const bf16* vp = static_cast<const bf16*>(a.v) + rv.base + t0 * rv.stride;
    const int other = Cfg::atom - first;
    const int within = atoms == 2 ? first : other, last = atoms == 2 ? other : first;
    auto load_within = [&]() {
      mm::load_tile<bf16, kC, KD, 512>(sbase + within, kLK, 0,
                                       static_cast<const bf16*>(a.k) + rk.base + t0 * rk.stride,
                                       rk.stride, rows, a.D, tid);
      mm::load_tile<bf16, kC, KD, 512>(sbase + within + Cfg::offQ, kLK, 0,
                                       static_cast<const bf16*>(a.q) + rk.base + t0 * rk.stride,
                                       rk.stride, rows, a.D, tid);
    };
    if (atoms == 2) load_atom(item, 1, other);
    else load_within();
    ptx::cp_async_commit();
    uint4 v[2];   // row r0's values beside this thread's vectors of dR
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int n = 64 * t + 8 * c;
      v[t] = r0 < rows && n < a.Dv ? *reinterpret_cast<const uint4*>(vp + r0 * rv.stride + n)
                                   : make_uint4(0, 0, 0, 0);
    }

    float rv_sum = 0.f, ss = 0.f;   // dR . v of row r0; <S, dS'>
    for (int t = 0; t < atoms; ++t) {
      if (t == 0) ptx::cp_async_wait<1>();
      else ptx::cp_async_wait<0>();
      wait_phase(landed + 8 * t, odd, a.flag, gave_up);
      ptx::fence_proxy_async();
      ptx::tc_fence_before();
      __syncthreads();
      ptx::tc_fence_after();
      tmem = *s_tmem;
      const uint32_t at0 = sbase + (t == 0 ? first : other);
      if (tid == 0) {
        constexpr uint32_t kBig = ptx::idesc_bf16_f32(128, KD, 0, 0);
        constexpr uint32_t kSmall = ptx::idesc_bf16_f32(128, 64, 0, 0);
        const uint32_t D1 = tmem, D4 = tmem + KD, D2 = tmem + 2 * KD, D3 = tmem + 3 * KD, D5 = D3 + 64;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint32_t k0 = at0 + 32 * kk, more = t > 0 || kk > 0;
          const uint64_t OR = ptx::smem_desc_sw128(k0, 16, 1024);
          const uint64_t R1 = ptx::smem_desc_sw128(k0 + Cfg::tileR1, 16, 1024);
          const uint64_t X0 = ptx::smem_desc_sw128(k0 + Cfg::tileX0, 16, 1024);
          const uint64_t X1 = ptx::smem_desc_sw128(k0 + Cfg::tileX1, 16, 1024);
          const uint64_t S0 = ptx::smem_desc_sw128(k0 + Cfg::tileS, 16, 1024);
          const uint64_t S1 = ptx::smem_desc_sw128(k0 + Cfg::tileS + KD * 128, 16, 1024);
          const uint64_t E0 = ptx::smem_desc_sw128(k0 + Cfg::tileD, 16, 1024);
          const uint64_t E1 = ptx::smem_desc_sw128(k0 + Cfg::tileD + KD * 128, 16, 1024);
          ptx::mma_bf16(D1, OR, S0, kBig, more);
          ptx::mma_bf16(D1, OR, S1, kBig, 1);
          ptx::mma_bf16(D4, R1, S0, kBig, more);
          ptx::mma_bf16(D2, X0, E0, kBig, more);
          ptx::mma_bf16(D2, X0, E1, kBig, 1);
          ptx::mma_bf16(D3, OR, X0, kSmall, more);
          ptx::mma_bf16(D3, OR, X1, kSmall, 1);
          ptx::mma_bf16(D5, R1, X0, kSmall, more);
        }
        ptx::mma_commit(done + 8 * t);
      }
      __syncwarp();
      // meanwhile
      const unsigned char* tile = smem + (t == 0 ? first : other) + place;
      auto add = [](const uint4& p, const uint4& q, float (&f)[8]) {
        const uint32_t u[4] = {p.x, p.y, p.z, p.w}, w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = ptx::bf16_lo(u[i]) + ptx::bf16_lo(w[i]);
          f[2 * i + 1] = ptx::bf16_hi(u[i]) + ptx::bf16_hi(w[i]);
        }
      };
      float x[8], y[8];
      add(*reinterpret_cast<const uint4*>(tile + Cfg::tileR0),
          *reinterpret_cast<const uint4*>(tile + Cfg::tileR1), x);
      add(t == 0 ? v[0] : v[1], make_uint4(0, 0, 0, 0), y);
#pragma unroll
      for (int i = 0; i < 8; ++i) rv_sum = fmaf(x[i], y[i], rv_sum);
#pragma unroll
      for (int p = 0; p < KD / 64; ++p) {
        const unsigned char* S = tile + Cfg::tileS + p * 8192;
        const unsigned char* D = tile + Cfg::tileD + p * 8192;
        add(*reinterpret_cast<const uint4*>(S), *reinterpret_cast<const uint4*>(S + KD * 128), x);
        add(*reinterpret_cast<const uint4*>(D), *reinterpret_cast<const uint4*>(D + KD * 128), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[i], y[i], ss);
      }
    }
    Gates* gates = reinterpret_cast<Gates*>(smem + Cfg::offGate + odd * Cfg::kDecays);
    const Decays* dec = reinterpret_cast<const Decays*>(gates + 1);
    float* sums = reinterpret_cast<float*>(smem + Cfg::offSum);
#pragma unroll
    for (int o = 1; o < 8; o *= 2) rv_sum += __shfl_xor_sync(0xffffffffu, rv_sum, o);
    if (c == 0) sums[24 * kC + r0] = rv_sum;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) sums[25 * kC + warp] = ss;
    if (atoms == 2) {
      wait_phase(done, odd, a.flag, gave_up);
      load_within();   // the first atom's tiles are read: by the products, and (a barrier ago) above
    }
    ptx::cp_async_wait_all();
    __syncthreads();
    const Within x{smem, sbase, within, within + Cfg::offQ, within + Cfg::offE, gates, dec, sums};
    float keys[2][2][4];   // while tcgen05 is at the last atom
    key_products<KD, 1, PO>(x, keys);
    wait_phase(done + 8 * (atoms - 1), odd, a.flag, gave_up);
    ptx::tc_fence_after();

    // out of tensor memory: warp (quad, cq) has lanes 32 quad and a quarter of the
    // columns; token i of this thread is in lanes i (dO, R1, X0) and 64 + i (R0, X1)
    const int quad = warp & 3, cq = warp >> 2, i = (32 * quad + lane) & 63;
    const uint32_t mine = tmem + ((uint32_t)(32 * quad) << 16);
    float* bDQ = reinterpret_cast<float*>(smem + last) + i * Cfg::pitch + cq * NC;
    float* bDK = bDQ + Cfg::offDK / 4;
    float* bP = reinterpret_cast<float*>(smem + last + Cfg::offP) + i * Cfg::pitchC + 16 * cq;
    float* bA = bP + (Cfg::offA - Cfg::offP) / 4;
    float4 g = gates->tok[i];
    const float bad = *gave_up ? void_value() : 0.f;   // a wait was given up
    g.z += bad;   // dk
    g.w += bad;   // dq
    const unsigned char* krow = smem + within + i * kLK + cq * NC * 2;
    float py = bad, pz = 0.f, dk[NC];   // k . (dR S^T), k . (X dS'^T); z . X dS'^T - x . dR S^T
    {
      uint32_t ki[NC], ko[NC];
      ptx::tmem_ld_32x32(mine + (quad < 2 ? KD : 0) + cq * NC, ki);
      ptx::tmem_ld_32x32(mine + 2 * KD + cq * NC, ko);
      ptx::tmem_wait_ld();
      float py1 = 0.f, pz1 = 0.f;
#pragma unroll
      for (int j = 0; j < NC; j += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(krow + 2 * j);
        const uint32_t k[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float k0 = ptx::bf16_lo(k[e / 2]), k1 = ptx::bf16_hi(k[e / 2]);
          const float a0 = __uint_as_float(ki[j + e]), a1 = __uint_as_float(ki[j + e + 1]);
          const float o0 = __uint_as_float(ko[j + e]), o1 = __uint_as_float(ko[j + e + 1]);
          py = fmaf(k0, a0, py);
          py1 = fmaf(k1, a1, py1);
          pz = fmaf(k0, o0, pz);
          pz1 = fmaf(k1, o1, pz1);
          dk[j + e] = g.z * o0 - g.x * a0;
          dk[j + e + 1] = g.z * o1 - g.x * a1;
        }
      }
      py += py1;
      pz += pz1;
    }
    uint32_t small[16];   // quad < 2: of dR X^T what R1 gives, else what R0 gives
    ptx::tmem_ld_32x32(mine + 3 * KD + (quad < 2 ? 64 : 0) + 16 * cq, small);
    ptx::tmem_wait_ld();
    if (quad >= 2) {
#pragma unroll
      for (int j = 0; j < NC; j += 4)
        *reinterpret_cast<float4*>(bDK + j) = make_float4(dk[j], dk[j + 1], dk[j + 2], dk[j + 3]);
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<uint4*>(bA + j) =
            make_uint4(small[j], small[j + 1], small[j + 2], small[j + 3]);
      sums[(12 + cq) * kC + i] = py;   // for the other half's sums
      sums[(20 + cq) * kC + i] = pz;
    }
    __syncthreads();
    if (quad < 2) {
#pragma unroll
      for (int j = 0; j < NC; j += 4) {
        float4 o = *reinterpret_cast<const float4*>(bDK + j);
        o.x += dk[j], o.y += dk[j + 1], o.z += dk[j + 2], o.w += dk[j + 3];
        *reinterpret_cast<float4*>(bDK + j) = o;
      }
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        float4 o = *reinterpret_cast<const float4*>(bA + j);
        o.x += __uint_as_float(small[j]), o.y += __uint_as_float(small[j + 1]);
        o.z += __uint_as_float(small[j + 2]), o.w += __uint_as_float(small[j + 3]);
        *reinterpret_cast<float4*>(bA + j) = o;
      }
      sums[(4 + cq) * kC + i] = py + sums[(12 + cq) * kC + i];
      sums[(8 + cq) * kC + i] = pz + sums[(20 + cq) * kC + i];
      uint32_t q[NC];
      ptx::tmem_ld_32x32(mine + cq * NC, q);
      ptx::tmem_ld_32x32(mine + 3 * KD + 16 * cq, small);
      ptx::tmem_wait_ld();
      float px = 0.f, px1 = 0.f;
#pragma unroll
      for (int j = 0; j < NC; j += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(krow + Cfg::offQ + 2 * j);
        const uint32_t k[4] = {u.x, u.y, u.z, u.w};
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(q[j + e]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          px = fmaf(ptx::bf16_lo(k[e / 2]), f[e], px);
          px1 = fmaf(ptx::bf16_hi(k[e / 2]), f[e + 1], px1);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 4)
          *reinterpret_cast<float4*>(bDQ + j + e) =
              make_float4(g.w * f[e], g.w * f[e + 1], g.w * f[e + 2], g.w * f[e + 3]);
      }
      sums[cq * kC + i] = px + px1;
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<uint4*>(bP + j) =
            make_uint4(small[j], small[j + 1], small[j + 2], small[j + 3]);
    }
    ptx::tc_fence_before();
    __syncthreads();

    // the products within the chunk, by row tiles and quarters of the columns
    const int m = warp & 3, ch = warp >> 2, r = lane >> 2, c2 = (lane & 3) * 2;
    {
      float dP[1][2][4], dA[1][2][4];
      const float* P = reinterpret_cast<const float*>(smem + last + Cfg::offP) +
                       (16 * m + r) * Cfg::pitchC + 16 * ch + c2;
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 p = *reinterpret_cast<const float2*>(P + 8 * e * Cfg::pitchC + 8 * n);
          const float2 q = *reinterpret_cast<const float2*>(P + (Cfg::offA - Cfg::offP) / 4 +
                                                            8 * e * Cfg::pitchC + 8 * n);
          dP[0][n][2 * e] = p.x, dP[0][n][2 * e + 1] = p.y;
          dA[0][n][2 * e] = q.x, dA[0][n][2 * e + 1] = q.y;
        }
      make_within<PO>(x, a.scale, keys, dP, dA);
    }
    float dq[1][NTK][4], ko[1][NTK][4];
    const float* Q = reinterpret_cast<const float*>(smem + last) + (16 * m + r) * Cfg::pitch +
                     ch * NC + c2;
#pragma unroll
    for (int n = 0; n < NTK; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float2 p = *reinterpret_cast<const float2*>(Q + 8 * e * Cfg::pitch + 8 * n);
        const float2 q =
            *reinterpret_cast<const float2*>(Q + Cfg::offDK / 4 + 8 * e * Cfg::pitch + 8 * n);
        dq[0][n][2 * e] = p.x, dq[0][n][2 * e + 1] = p.y;
        ko[0][n][2 * e] = q.x, ko[0][n][2 * e + 1] = q.y;
      }
    if (Cfg::kItems) ptx::fence_proxy_async();
    __syncthreads();
    // the place of the sums is free: the next item's first atom comes in meanwhile
    int next = total;
    if (Cfg::kItems) {
      next = live(total - item > (int)gridDim.x ? item + (int)gridDim.x : total);
      if (next < total) begin(next, last, odd ^ 1);
    }
    finish<bf16, KD, PO>(a, x, bh, chunk, rows, dq, ko);
    if (!Cfg::kItems) break;
    ptx::fence_proxy_async();
    __syncthreads();
    item = next;
    first = last;
  }
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Cfg::columns);
  }
}

// dq and dk of shared heads: the sum over the value heads of a group, in their
// order (a group of none: zeros). Eight columns of a row per thread.
template <typename T>
__global__ void __launch_bounds__(256) shared_heads_kernel(const Args a) {
  ptx::grid_dependency_wait();
  const int V = a.D / 8, group = a.H / a.Hk;
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  const int d = (int)(i % V) * 8, n = (int)(i / V % a.N);
  const long long bk = i / V / a.N;   // b Hk + hk
  const int b = (int)(bk / a.Hk), hk = (int)(bk % a.Hk);
  if (b >= a.B) return;
  if (n >= length_of(a, b)) return;
  const Rows rk = rows_of(a, b, hk, a.Hk, a.D);
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const float* src = (which ? a.wdk : a.wdq) +
                       (((long long)b * a.H + (long long)hk * group) * a.N + n) * a.D + d;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < group; ++g) {
      const float4 u = *reinterpret_cast<const float4*>(src + (long long)g * a.N * a.D);
      const float4 v = *reinterpret_cast<const float4*>(src + (long long)g * a.N * a.D + 4);
      x[0] += u.x, x[1] += u.y, x[2] += u.z, x[3] += u.w;
      x[4] += v.x, x[5] += v.y, x[6] += v.z, x[7] += v.w;
    }
    T* dst = static_cast<T*>(which ? a.dk : a.dq) + rk.base + n * rk.stride + d;
#pragma unroll
    for (int e = 0; e < 8; e += 2) mm::Io<T>::store2(dst + e, x[e], x[e + 1]);
  }
}

// ---- host --------------------------------------------------------------------------------

// (A record has room for three planes of T and of P, which calls that want dstate
// fill: whether one does is not known where the size is asked for.)
struct BwdBytes {
  size_t rec, img, wdq, total;
  int atoms;
  explicit BwdBytes(const la_delta_params& p) {
    const size_t heads = (size_t)p.B * p.H, chunks = heads * ((p.N + kC - 1) / kC);
    const size_t po = p.dtype == LA_BF16 ? grad_planes<bf16>() : grad_planes<float>();
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    atoms = (p.Dv + 63) / 64;
    rec = up(chunks * Record<kChainPlanes, kChainPlanes>::bytes);
    // Image<KD, PO>::atom
    img = chunks * atoms * (2 * po * 128 * (kC + (p.D <= 64 ? 64 : 128)));
    wdq = p.Hk == p.H ? 0 : up(heads * p.N * p.D * sizeof(float));
    total = LA_WORKSPACE_CONTROL_BYTES + rec + img + 2 * wdq;
  }
};

template <typename T>
la_status run_shared_heads(const Args& a, bool next, cudaStream_t stream) {
  const long long count = (long long)a.B * a.Hk * a.N * (a.D / 8);
  return launch<shared_heads_kernel<T>>((unsigned)((count + 255) / 256), 256, 0, stream, a, next);
}

// GNV: value columns to a slice of gradient_kernel (fp32 only).
template <typename T, int KD, int RT, int PC, int NBUF, int GNV = 0>
la_status run_backward(Args a, int B, cudaStream_t stream) {
  constexpr int PO = grad_planes<T>();
  const long long heads = (long long)B * a.H;
  la_status st = run_terms<T, KD, PC, PC>(a, heads, stream);
  if (st != LA_OK) return st;
  a.slices = (a.Dv + 16 * RT - 1) / (16 * RT);
  const unsigned chains = (unsigned)(heads * a.slices);
  constexpr int kStages = 2;   // of scan_kernel
  using Scan = ScanCfg<T, KD, RT, PC, PO, kStages, true>;
  st = launch<scan_kernel<T, KD, RT, PC, PO, kStages, true>>(chains, Scan::threads, Scan::bytes,
                                                             stream, a, true);
  if (st != LA_OK) return st;
  using Rev = RevCfg<T, KD, RT, PC, PO, NBUF>;
  st = launch<reverse_kernel<T, KD, RT, PC, PO, NBUF>>(chains, Rev::threads, Rev::bytes, stream, a,
                                                       true);
  if (st != LA_OK) return st;
  const unsigned each = (unsigned)(heads * a.chunks);
  if constexpr (sizeof(T) == 2) {
    using Grad = GradTcCfg<KD>;
    unsigned grid = each;
    if (Grad::kItems) {
      int sms = 0;
      if ((st = device_sms(&sms)) != LA_OK) return st;
      if (grid > (unsigned)sms) grid = sms;
    }
    st = launch<gradient_tc_kernel<KD, PC>>(grid, Grad::threads, Grad::bytes, stream, a, true);
  } else {
    using Grad = GradCfg<KD, GNV, PO>;
    st = launch<gradient_kernel<KD, GNV, PC, PO>>(each, Grad::threads, Grad::bytes, stream, a, true);
  }
  if (st != LA_OK || a.Hk == a.H) return st;
  return run_shared_heads<T>(a, true, stream);
}

}  // namespace
}  // namespace delta
}  // namespace la

using namespace la;
using namespace la::delta;

extern "C" {

la_status lin_attn_delta_backward_workspace_size(const la_delta_params* p, size_t* bytes) {
  if (!bytes) return LA_ERR_INVALID_ARG;
  const la_status st = check_delta(p);
  if (st == LA_OK) *bytes = BwdBytes(*p).total;
  return st;
}

la_status lin_attn_delta_backward(const la_delta_params* p, const void* dout, const void* q,
                                  const void* k, const void* v, const void* log_decay,
                                  const void* beta, const float* state, const float* dstate_out,
                                  const int* lengths, void* dq, void* dk, void* dv,
                                  void* dlog_decay, void* dbeta, float* dstate, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  la_status st = check_delta(p);
  if (st != LA_OK) return st;
  const long long heads = (long long)p->B * p->H;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (heads == 0) {
    // without value heads, dq and dk are sums over none
    const size_t n = DeltaBytes(*p).qk, nl = p->B * sizeof(int);
    if (n == 0) return LA_OK;
    if (!dq || !dk || !aligned16(dq) || !aligned16(dk) || !aligned(lengths, 4))
      return LA_ERR_INVALID_ARG;
    for (const void* in : {q, k})
      if (overlaps(dq, n, in, n) || overlaps(dk, n, in, n)) return LA_ERR_INVALID_ARG;
    if (overlaps(dq, n, dk, n) || overlaps(dq, n, lengths, nl) || overlaps(dk, n, lengths, nl))
      return LA_ERR_INVALID_ARG;
    int* const flag = flag_of(workspace, workspace_bytes);
    for (const void* x : {(const void*)dq, (const void*)dk, q, k})
      if (overlaps(flag, sizeof(int), x, n)) return LA_ERR_INVALID_ARG;
    if (overlaps(flag, sizeof(int), lengths, nl)) return LA_ERR_INVALID_ARG;
    if ((st = clear_flag(workspace, workspace_bytes, cs)) != LA_OK) return st;
    Args a = delta_args(*p, q, k, v, log_decay, beta, state, lengths);
    a.dq = dq;
    a.dk = dk;
    return p->dtype == LA_F32 ? run_shared_heads<float>(a, false, cs)
                              : run_shared_heads<bf16>(a, false, cs);
  }
  const size_t sbytes = (size_t)heads * p->D * p->Dv * sizeof(float);
  if (!aligned16(state) || !aligned16(dstate_out) || !aligned16(dstate)) return LA_ERR_INVALID_ARG;
  if (dstate && dstate != dstate_out && overlaps(dstate, sbytes, dstate_out, sbytes))
    return LA_ERR_INVALID_ARG;
  if (overlaps(dstate, sbytes, state, sbytes)) return LA_ERR_INVALID_ARG;
  if (p->N == 0) {
    const int* flag = flag_of(workspace, workspace_bytes);
    if (overlaps(flag, sizeof(int), dstate_out, sbytes) || overlaps(flag, sizeof(int), dstate, sbytes))
      return LA_ERR_INVALID_ARG;
    return copy_state(dstate, dstate_out, sbytes, workspace, workspace_bytes, cs);
  }
  const DeltaBytes n(*p);
  const BwdBytes ws(*p);
  const void* in[9] = {dout, q, k, v, log_decay, beta, lengths, state, dstate_out};
  const size_t nin[9] = {n.v, n.qk, n.qk, n.v, n.gate, n.gate, p->B * sizeof(int), sbytes, sbytes};
  void* out[6] = {dq, dk, dv, dlog_decay, dbeta, dstate};
  const size_t nout[6] = {n.qk, n.qk, n.v, n.gate, n.gate, sbytes};
  for (int i = 0; i < 6; ++i)
    if (!in[i] || !aligned(in[i], i < 4 ? 16 : n.elt)) return LA_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)
    if (!out[i] || !aligned(out[i], i < 3 ? 16 : n.elt)) return LA_ERR_INVALID_ARG;
  if (!aligned(lengths, 4)) return LA_ERR_INVALID_ARG;
  if ((st = check_delta_workspace(workspace, workspace_bytes, ws.total)) != LA_OK) return st;
  for (int i = 0; i < 6; ++i) {
    if (overlaps(out[i], nout[i], workspace, ws.total)) return LA_ERR_INVALID_ARG;
    for (int j = 0; j < 9; ++j)
      if (overlaps(out[i], nout[i], in[j], nin[j]) && !(out[i] == dstate && in[j] == dstate_out))
        return LA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], nout[i], out[j], nout[j])) return LA_ERR_INVALID_ARG;
  }
  for (int j = 0; j < 9; ++j)
    if (overlaps(workspace, ws.total, in[j], nin[j])) return LA_ERR_INVALID_ARG;

  Args a = delta_args(*p, q, k, v, log_decay, beta, state, lengths);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  a.flag = reinterpret_cast<int*>(w);
  a.rec = w += LA_WORKSPACE_CONTROL_BYTES;
  a.img = w += ws.rec;
  a.atoms = ws.atoms;
  a.wdq = reinterpret_cast<float*>(w += ws.img);
  a.wdk = reinterpret_cast<float*>(w += ws.wdq);
  a.dout = dout;
  a.ds1 = dstate_out;
  a.ds0 = dstate;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.dg = dlog_decay;
  a.dbeta = dbeta;
  const int B = p->B;
  if (p->dtype == LA_F32)
    return p->D <= 64 ? run_backward<float, 64, 1, 3, 1, 32>(a, B, cs)
                      : run_backward<float, 128, 1, 3, 1, 16>(a, B, cs);
  // the two kernels' chains run side by side
  bool wide = false;
  if ((st = wide_chains(2 * heads, p->Dv, &wide)) != LA_OK) return st;
  // Gradients in bf16 take 17 bits of the chains (see the top); that of the initial
  // state, in fp32, needs all: three planes, which at D 128 leave no room for 32
  // columns (2 x 16 heads of 4096 tokens: 609 us without, 780 with; D 64: 315 and
  // 351).
  if (dstate) {
    if (p->D > 64) return run_backward<bf16, 128, 1, 3, 2>(a, B, cs);
    return wide ? run_backward<bf16, 64, 2, 3, 2>(a, B, cs)
                : run_backward<bf16, 64, 1, 3, 2>(a, B, cs);
  }
  if (p->D <= 64)
    return wide ? run_backward<bf16, 64, 2, 2, 2>(a, B, cs)
                : run_backward<bf16, 64, 1, 2, 2>(a, B, cs);
  return wide ? run_backward<bf16, 128, 2, 2, 2>(a, B, cs)
              : run_backward<bf16, 128, 1, 2, 2>(a, B, cs);
}

}  // extern "C"
