// delta_scan.cuh -- the kernel that carries the delta rule's state from chunk
// to chunk (the formulas are in delta.cuh).
//
// One CTA per (head, slice of 16 RT value columns): the columns of the state do
// not mix, so slices of them are independent chains. Per chunk the chain is
// three dependent products,
//     K S  ->  R  ->  X = T R  ->  S' = exp(G_last) S + K^T (z . X),
// with S kept in fp32 registers; all else is off the chain and runs beside it:
//   warps 0-3    the chain,
//   warps 4-7    out = w . (Q S) + P X and its stores, in the same shares,
//   warps 8-11   copies of the next chunks' K, Q, V and record.
//
// What bounds it is the chain's latency: at D 64 and 16 columns a chunk takes
// 1.53 us (32 heads of 32,760 tokens: 781 us), of which the matrix instructions
// of the busiest warp are 0.4; the rest are three splits into planes, four
// barriers and the operands' way through shared memory, whose pipe is 64 % busy
// (tensor 38 %, instruction issue 30 %). With 32 columns of D 128 (48 heads) it
// is 67 % and the tensor pipe 59 %. The products are warp-level: one takes 21
// cycles from operands to sums in registers, where a tcgen05 product has to be
// committed, waited for and read back from tensor memory before the next step
// of the chain can begin, and its operands, three planes of 128 x 128 state,
// would leave shared memory no room for the next chunk's.
//
// Rounding: the state, T, R and X enter products as PC bf16 planes, and what only
// the outputs or gradients need (S beside Q, X beside P) as PO. Forward both are
// three, all bits of fp32, so neither the carried state nor `out` loses anything
// to the tensor cores: of outputs in bf16 0.012 % are not the rounding of the
// exact value, as of an fp32 computation (four heads of 1024 tokens, D 64). With
// PO = 2, 17 bits, that is 0.76 %, for 5 to 9 % less time (480p clip 930 us
// and 982, ragged batch 577 and 630, D 112 block 171 and 181). The backward pass'
// choice is in delta_bwd.cu.
#pragma once

#include "delta.cuh"

namespace la {
namespace delta {

// Named barriers. Stages: kBarFull.. tells the chain, kBarFullOut.. the outputs'
// warps, kBarFree.. the copies. kBarS, kBarR: the chain's own. kBarOut tells the
// outputs that S is stored; kBarX is the chain's and the outputs', when X is
// stored and S has been read; kBarRead tells the chain that X has been read. So
// the chain waits for the outputs where it has to, not where they begin.
enum {
  kBarFull = 1, kBarFullOut = 4, kBarFree = 7, kBarR = 10, kBarX = 11, kBarS = 12, kBarOut = 13,
  kBarRead = 14
};

template <typename T, int KD, int RT, int PC, int PO, int NBUF, bool BWD>
struct ScanCfg {
  static constexpr int PI = mm::Io<T>::kPlanes, NV = 16 * RT;
  using R = Record<PC, BWD ? PC : PO>;
  // a stage: the record's first part (Gates, T, P), K, Q, V; BWD without P and Q
  static constexpr int kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  static constexpr int kRec = BWD ? R::offP : R::offD;
  static constexpr int offK = kRec, offQ = offK + PI * kPlaneK;
  static constexpr int offV = offQ + (BWD ? 0 : PI * kPlaneK);
  static constexpr int stage = offV + kC * NV * (int)sizeof(T);
  static constexpr int kLN = (NV + 8) * 2;
  static constexpr int kPlaneS = KD * kLN, kPlaneX = kC * kLN;
  static constexpr int offS = NBUF * stage;
  static constexpr int offR = offS + PC * kPlaneS;      // R, then X for the outputs
  static constexpr int offX = offR + PC * kPlaneX;      // z . X
  static constexpr int offBar = offX + PC * kPlaneX;
  static constexpr int bytes = offBar + NBUF * 8 + 8;   // mbarriers, two words
  static constexpr int threads = 256 + kLoadThreads;
};

// NaN for a thread's part of the outputs: the pairs of columns 0 and 8, of `cols`,
// in rows row, row + 8 and so every 64.
template <typename T>
__device__ __noinline__ void void_rows(T* out, long long stride, int row, int rows, int cols) {
  for (; row < rows; row += row & 8 ? kC - 8 : 8)
    for (int n = 0; n < 16 && n < cols; n += 8)
      mm::Io<T>::store2(out + row * stride + n, void_value(), void_value());
}

// BWD: instead of `out`, leave the state before every chunk and X in the
// workspace for the backward pass.
template <typename T, int KD, int RT, int PC, int PO, int NBUF, bool BWD>
__global__ void __launch_bounds__(256 + kLoadThreads, 1) scan_kernel(const Args a) {
  using Cfg = ScanCfg<T, KD, RT, PC, PO, NBUF, BWD>;
  using Rec = typename Cfg::R;
  constexpr int PI = Cfg::PI, NV = Cfg::NV, kLN = Cfg::kLN, kLK = Cfg::kLK;
  constexpr int MS = Share<KD, RT>::MS;
  static_assert(PO <= PC, "X for the outputs lies in R's place");
  extern __shared__ __align__(16) unsigned char smem[];
  const uint32_t sbase = ptx::smem_u32(smem);
  const uint32_t landed = sbase + Cfg::offBar;   // per stage: the record's copy
  volatile int* gave_up = reinterpret_cast<volatile int*>(smem + Cfg::offBar + NBUF * 8);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NBUF; ++i) ptx::mbar_init(landed + 8 * i, 1);
    *gave_up = 0;
    ptx::fence_mbar_init();
  }
  // The kernel after, reverse_kernel, needs the records but nothing from here.
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int head = blockIdx.x / a.slices, slice = blockIdx.x % a.slices;
  const int b = nth_longest(a, head / a.H, gave_up + 1);   // a barrier
  const int h = head % a.H, bh = b * a.H + h, hk = h / (a.H / a.Hk);
  const int n0 = slice * NV;
  const int len = length_of(a, b), chunks = (len + kC - 1) / kC;
  const Rows rv = rows_of(a, b, h, a.H, a.Dv);

  if (warp >= 8) {
    // ---- copies ----
    const int tid = threadIdx.x - 256;
    const Rows rk = rows_of(a, b, hk, a.Hk, a.D);
    const T* kp = static_cast<const T*>(a.k) + rk.base;
    const T* qp = static_cast<const T*>(a.q) + rk.base;
    const T* vp = static_cast<const T*>(a.v) + rv.base + n0;
    const unsigned char* rec = a.rec + (long long)bh * a.chunks * Rec::bytes;
    for (int c = 0; c < chunks; ++c) {
      const int buf = c % NBUF;
      if (c >= NBUF) ptx::bar_sync(kBarFree + buf, 384);
      const uint32_t at = sbase + buf * Cfg::stage;
      const int rows = min(kC, len - c * kC);
      const long long t = (long long)c * kC;
      load_record<Cfg::kRec>(at, rec + (long long)c * Rec::bytes, landed + 8 * buf, tid);
      mm::load_tile<T, kC, KD, kLoadThreads>(at + Cfg::offK, kLK, Cfg::kPlaneK, kp + t * rk.stride,
                                             rk.stride, rows, a.D, tid);
      if (!BWD)
        mm::load_tile<T, kC, KD, kLoadThreads>(at + Cfg::offQ, kLK, Cfg::kPlaneK,
                                               qp + t * rk.stride, rk.stride, rows, a.D, tid);
      // V as it is
      constexpr int E = 16 / (int)sizeof(T), VV = NV / E, STEP = kLoadThreads / VV;
      const int row0 = tid / VV, col = tid % VV * E;
      const int rows_v = n0 + col < a.Dv ? rows : 0;
#pragma unroll
      for (int row = 0; row < kC; row += STEP) {
        const bool in = row0 + row < rows_v;
        mm::cp_async16(at + Cfg::offV + (row0 + row) * NV * (int)sizeof(T) + tid % VV * 16,
                       in ? vp + (t + row0 + row) * rv.stride + col : vp, in);
      }
      ptx::cp_async_wait_all();
      wait_phase(landed + 8 * buf, (c / NBUF) & 1, a.flag, gave_up);
      ptx::bar_arrive(kBarFull + buf, 256);
      ptx::bar_arrive(kBarFullOut + buf, 256);
    }
    return;
  }

  const Share<KD, RT> sh(warp & 3);
  const int r = lane >> 2, c2 = (lane & 3) * 2, nw = sh.col;
  const uint32_t lane_at = mm::a_lane<false>(lane, kLN) + nw * 2;
  const uint32_t sS = sbase + Cfg::offS, sR = sbase + Cfg::offR, sX = sbase + Cfg::offX;

  if (warp < 4) {
    // ---- the chain: rows sh.state + 16 m + r, r + 8 of the state ----
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
          if (a.s0 && row < a.D && col < a.Dv)
            x = *reinterpret_cast<const float2*>(a.s0 + s_at + (long long)row * a.Dv + col);
          S[m][n][2 * i] = x.x;
          S[m][n][2 * i + 1] = x.y;
        }
    const mm::Operand opS = mm::b_tile<true>(sS + nw * 2, kLN, Cfg::kPlaneS);
    const mm::Operand opR = mm::b_tile<true>(sR + nw * 2, kLN, Cfg::kPlaneX);
    const mm::Operand opX = mm::b_tile<true>(sX + nw * 2, kLN, Cfg::kPlaneX);
    for (int c = 0; c < chunks; ++c) {
      const int buf = c % NBUF;
      const unsigned char* cb = smem + buf * Cfg::stage;
      const uint32_t sb = sbase + buf * Cfg::stage;
      const Gates* gates = reinterpret_cast<const Gates*>(cb);
#pragma unroll
      for (int m = 0; m < MS; ++m)
        mm::store_tile<PC>(sS + (sh.state + 16 * m) * kLN + lane_at, Cfg::kPlaneS, S[m]);
      ptx::bar_arrive(kBarOut, 256);
      ptx::bar_sync(kBarFull + buf, 256);
      // what R and X need besides the products, loaded ahead of them
      float4 gt[RT][2];
      float2 vs[RT][2][2];
      const float last = gates->last[0];
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 16 * sh.tile[j] + r + 8 * i;
          gt[j][i] = gates->tok[row];
          const T* v = reinterpret_cast<const T*>(cb + Cfg::offV) + row * NV + nw + c2;
#pragma unroll
          for (int n = 0; n < 2; ++n) vs[j][i][n] = mm::Io<T>::load2s(v + 8 * n);
        }
      {
        float ks[RT][2][4];
        mm::zero(ks);
        mm::gemm<RT, 2, PI, PC, PC, false, true, KD / 16>(
            ks, sh.rows(sb + Cfg::offK, kLK, Cfg::kPlaneK), opS, KD / 16,
            [] { ptx::bar_sync(kBarS, 128); });
        if (c > 0) ptx::bar_sync(kBarRead, 256);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              ks[j][n][2 * i] = gt[j][i].y * vs[j][i][n].x - gt[j][i].x * ks[j][n][2 * i];
              ks[j][n][2 * i + 1] = gt[j][i].y * vs[j][i][n].y - gt[j][i].x * ks[j][n][2 * i + 1];
            }
          mm::store_tile<PC>(sR + 16 * sh.tile[j] * kLN + lane_at, Cfg::kPlaneX, ks[j]);
        }
      }
      {
        float x[RT][1][2][4];
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          mm::zero(x[j]);
          mm::gemm<1, 2, PC, PC, PC, false, true, 4>(
              x[j], mm::a_tri<false>(sb + Rec::offT, sh.tile[j]), opR, sh.tile[j] + 1, [&] {
                if (j == 0) ptx::bar_sync(kBarR, 128);
              });
        }
        ptx::bar_sync(kBarR, 128);   // R is read: its place takes X
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const uint32_t at = 16 * sh.tile[j] * kLN + lane_at;
          mm::store_tile<PO>(sR + at, Cfg::kPlaneX, x[j][0]);
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[j][0][n][i] *= gt[j][i / 2].z;
          mm::store_tile<PC>(sX + at, Cfg::kPlaneX, x[j][0]);
        }
      }
      // summed apart from the state, and added with one rounding to nearest
      float u[MS][2][4];
      mm::zero(u);
      mm::gemm<MS, 2, PI, PC, PC, true, true, kC / 16>(
          u, mm::a_tile<true>(sb + Cfg::offK + 2 * sh.state, kLK, Cfg::kPlaneK), opX,
          kC / 16, [] { ptx::bar_sync(kBarX, 256); });
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) S[m][n][i] = fmaf(last, S[m][n][i], u[m][n][i]);
      if (c + NBUF < chunks) ptx::bar_arrive(kBarFree + buf, 384);
    }
    if (a.s1) {
      const bool bad = *gave_up;
#pragma unroll
      for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int row = sh.state + 16 * m + r + 8 * i, col = n0 + nw + 8 * n + c2;
            if (row < a.D && col < a.Dv)
              *reinterpret_cast<float2*>(a.s1 + s_at + (long long)row * a.Dv + col) =
                  bad ? make_float2(void_value(), void_value())
                      : make_float2(S[m][n][2 * i], S[m][n][2 * i + 1]);
          }
    }
    return;
  }

  // ---- the outputs ----
  T* op = static_cast<T*>(a.out) + rv.base + n0 + nw + c2;
  const int tid = threadIdx.x - 128;
  for (int c = 0; c < chunks; ++c) {
    const int buf = c % NBUF;
    const uint32_t sb = sbase + buf * Cfg::stage;
    const int rows = len - c * kC;
    ptx::bar_sync(kBarFullOut + buf, 256);
    if (BWD) {
      ptx::bar_sync(kBarOut, 256);
      using I = Image<KD, PO>;
      unsigned char* img = I::at(a, (long long)bh * a.chunks + c);
      const bool end = slice == a.slices - 1;
      store_image<KD, PO, NV, KD>(img, I::offS, a.atoms, n0, end, sS, kLN, Cfg::kPlaneS, tid);
      ptx::bar_sync(kBarX, 256);
      store_image<KD, PO, NV, kC>(img, I::offX, a.atoms, n0, end, sR, kLN, Cfg::kPlaneX, tid);
    } else {
      const Gates* gates = reinterpret_cast<const Gates*>(smem + buf * Cfg::stage);
      float o[RT][2][4];
      mm::zero(o);
      mm::gemm<RT, 2, PI, PO, PO, false, true, KD / 16>(
          o, sh.rows(sb + Cfg::offQ, kLK, Cfg::kPlaneK),
          mm::b_tile<true>(sS + nw * 2, kLN, Cfg::kPlaneS), KD / 16,
          [] { ptx::bar_sync(kBarOut, 256); });
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float e = gates->tok[16 * sh.tile[j] + r + 8 * i].w;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            o[j][n][2 * i] *= e;
            o[j][n][2 * i + 1] *= e;
          }
        }
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        float(&oj)[1][2][4] = *reinterpret_cast<float(*)[1][2][4]>(&o[j]);
        mm::gemm<1, 2, PO, PO, PO, false, true, 4>(
            oj, mm::a_tri<false>(sb + Rec::offP, sh.tile[j]),
            mm::b_tile<true>(sR + nw * 2, kLN, Cfg::kPlaneX), sh.tile[j] + 1, [&] {
              if (j == 0) ptx::bar_sync(kBarX, 256);
            });
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 16 * sh.tile[j] + r + 8 * i;
          T* p = op + ((long long)c * kC + row) * rv.stride;
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (row < rows && n0 + nw + 8 * n + c2 < a.Dv)
              mm::Io<T>::store2(p + 8 * n, o[j][n][2 * i], o[j][n][2 * i + 1]);
        }
      }
    }
    if (c + 1 < chunks) ptx::bar_arrive(kBarRead, 256);
    if (c + NBUF < chunks) ptx::bar_arrive(kBarFree + buf, 384);
  }
  if (!*gave_up) return;
  // what this thread has stored is void
  if constexpr (BWD) {
    using I = Image<KD, PO>;
    unsigned char* img = I::at(a, (long long)bh * a.chunks);
    void_image<KD, PO, NV, KD>(img, I::offS, a.atoms, n0, chunks, tid);
    void_image<KD, PO, NV, kC>(img, I::offX, a.atoms, n0, chunks, tid);
  } else {
#pragma unroll
    for (int j = 0; j < RT; ++j)
      void_rows(op, rv.stride, 16 * sh.tile[j] + r, len, a.Dv - (n0 + nw + c2));
  }
}

}  // namespace delta
}  // namespace la
