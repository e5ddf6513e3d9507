// delta.cuh -- the gated delta rule in chunks of 64 tokens: what a chunk has
// of its own tokens.
//
// Per head, with a state S [D, Dv] and a_t = exp(g_t):
//     S_t = a_t S_{t-1} + beta_t k_t (v_t - a_t S_{t-1}^T k_t)^T,
//     out_t = scale S_t^T q_t.
// Over a chunk, with G_i the sum of g over its tokens up to i and S the state
// before it, the recurrence is (Yang et al., "Gated Delta Networks", 2024)
//     A_ij = beta_i exp(G_i - G_j) k_i.k_j  (j < i),     T = (I + A)^-1,
//     R_i  = beta_i (v_i - exp(G_i) S^T k_i),            X = T R,
//     P_ij = scale exp(G_i - G_j) q_i.k_j  (j <= i),
//     out  = scale exp(G) . (Q S) + P X,
//     S'   = exp(G_last) S + K^T (exp(G_last - G) . X).
// T and P need no state: one kernel makes them for all chunks at once and
// leaves them in the workspace, a record per chunk.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mma.cuh"
#include "ptx.cuh"

namespace la {
namespace delta {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;   // tokens per chunk

// Log decays below this count as this: exp(-100) < 4e-44. A decay of zero
// (log decay -inf) would make differences of sums undefined.
constexpr float kMinLogDecay = -100.f;

// Factors of a chunk's decays, in shared memory. The sums G are kept in 64
// bits: what counts are differences of them, and a chunk may hold 64 decays of
// -100. For tokens i > j in different blocks of 16, with m the last token
// before i's block,
//     exp(G_i - G_j) = exp(G_i - G_m) exp(G_m - G_j) = up[i] down[m/16][j],
// two factors of at most 1, so a product underflows only where its value does;
// an exponential of its own is left to the pairs of one block.
struct Gates {
  float4 tok[kC];        // x = beta e, y = beta, z = exp(G_last - G), w = scale e; e = exp(G)
  float last[4];         // exp(G_last)
};
struct Decays {
  double G[kC];
  float up[kC];
  float down[3][kC];
};

// A chunk's record, in the workspace as in shared memory: Gates, T (PC planes),
// P (PO planes), Decays. The first two are all that a chain of states needs.
template <int PC, int PO>
struct Record {
  static constexpr int offT = (int)sizeof(Gates);
  static constexpr int offP = offT + PC * mm::kTriPlane;
  static constexpr int offD = offP + PO * mm::kTriPlane;
  static constexpr int bytes = offD + (int)sizeof(Decays);
  static_assert(offT % 16 == 0 && bytes % 16 == 0, "copied 16 bytes at a time");
};

struct Args {
  const void *q, *k, *v, *g, *beta;
  const float* s0;       // initial state, or null (zeros)
  const int* lengths;    // [B], or null
  void* out;
  float* s1;             // final state, or null
  int B, H, Hk, N, D, Dv, bnhd;
  float scale;
  int slices;            // slices of the value columns
  int chunks;            // chunks of N tokens
  int* flag;             // workspace: its control block's flag word, or null
  unsigned char* rec;    // records [B H][chunks]
  // the backward pass (delta_bwd.cu): per head and chunk an Image, that is planes
  // of the state before it, of the gradient of the state after it, of X and of
  // dR; with shared heads, every head's own part of dq and dk in fp32
  unsigned char* img;
  int atoms;             // of 64 value columns
  float *wdq, *wdk;
  const void* dout;
  const float* ds1;      // gradient of the final state, or null (zeros)
  float* ds0;            // gradient of the initial state, or null
  void *dq, *dk, *dv, *dg, *dbeta;
};

// Where the rows of head (b, h) of a tensor with `heads` heads of `width`
// values start, and how far apart they are.
struct Rows {
  long long base, stride;
};
__device__ __forceinline__ Rows rows_of(const Args& a, int b, int h, int heads, int width) {
  Rows r;
  if (a.bnhd) {
    r.base = ((long long)b * a.N * heads + h) * width;
    r.stride = (long long)heads * width;
  } else {
    r.base = ((long long)b * heads + h) * a.N * width;
    r.stride = width;
  }
  return r;
}

__device__ __forceinline__ int length_of(const Args& a, int b) {
  if (!a.lengths) return a.N;
  const int n = a.lengths[b];
  return n < 0 ? 0 : (n > a.N ? a.N : n);
}

__device__ __forceinline__ float clamp_decay(float g) { return g < kMinLogDecay ? kMinLogDecay : g; }

// A warp's log decays and write strengths: lane l has tokens 2l and 2l + 1.
struct GateRows {
  float g0, g1, b0, b1;
  template <typename T>
  __device__ __forceinline__ void load(const T* g, const T* beta, long long stride, int rows) {
    const int i0 = 2 * (threadIdx.x & 31), i1 = i0 + 1;
    g0 = i0 < rows ? clamp_decay(mm::Io<T>::load(g + i0 * stride)) : 0.f;
    b0 = i0 < rows ? mm::Io<T>::load(beta + i0 * stride) : 0.f;
    g1 = i1 < rows ? clamp_decay(mm::Io<T>::load(g + i1 * stride)) : 0.f;
    b1 = i1 < rows ? mm::Io<T>::load(beta + i1 * stride) : 0.f;
  }
};

// Fills Gates and Decays in: one warp makes the first with G, another one the
// factors up and down.
__device__ __forceinline__ void chunk_gates(const GateRows& x, float scale, bool factors,
                                            Gates* out, Decays* dec) {
  const int lane = threadIdx.x & 31, i0 = 2 * lane, i1 = i0 + 1;
  double t = (double)x.g0 + (double)x.g1;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const double u = __shfl_up_sync(0xffffffffu, t, o);
    if (lane >= o) t += u;
  }
  double before = __shfl_up_sync(0xffffffffu, t, 1);
  if (lane == 0) before = 0.0;
  const double G0 = before + x.g0;
  if (!factors) {
    const double last = __shfl_sync(0xffffffffu, t, 31);
    const float e0 = expf((float)G0), e1 = expf((float)t);
    out->tok[i0] = make_float4(x.b0 * e0, x.b0, expf((float)(last - G0)), scale * e0);
    out->tok[i1] = make_float4(x.b1 * e1, x.b1, expf((float)(last - t)), scale * e1);
    dec->G[i0] = G0;
    dec->G[i1] = t;
    if (lane == 0) out->last[0] = expf((float)last);
    return;
  }
  double edge = 0.0;   // G at the end of the block before this lane's
#pragma unroll
  for (int m = 0; m < 3; ++m) {
    const double Gm = __shfl_sync(0xffffffffu, t, 8 * m + 7);
    if (lane < 8 * m + 8) {
      dec->down[m][i0] = expf((float)(Gm - G0));
      dec->down[m][i1] = expf((float)(Gm - t));
    } else {
      edge = Gm;
    }
  }
  dec->up[i0] = expf((float)(G0 - edge));
  dec->up[i1] = expf((float)(t - edge));
}

// ---- what the backward pass keeps of a chunk ----------------------------------------------
//
// By atoms of 64 value columns; an atom is tiles of 128-byte rows, the planes of
// dR and X (64 rows each) and of S and dS' (KD rows each), whose 16-byte vectors
// lie as the 128-byte swizzle of tensor-core operands wants them (vector c of
// row r at c ^ (r % 8)): an atom is one bulk copy into such operands. Columns
// from Dv on are zero.
template <int KD, int PO>
struct Image {
  static constexpr int offR = 0, offX = PO * kC * 128, offS = 2 * PO * kC * 128;
  static constexpr int offD = offS + PO * KD * 128, atom = offD + PO * KD * 128;
  __device__ static unsigned char* at(const Args& a, long long chunk) {
    return a.img + chunk * a.atoms * atom;
  }
  // vector c (0 .. 7) of a row, from the beginning of a tile
  __device__ __forceinline__ static int vec(int row, int c) {
    return row * 128 + ((c ^ (row & 7)) << 4);
  }
};

// Copies `rows` rows (all planes) of a slice's columns n0 .. n0 + NV from a tile
// in shared memory, whose planes have `tile_rows` rows each, to a tile of the
// image, by 128 threads; the last slice also makes the columns behind it zero.
template <int KD, int PO, int NV, int ROWS>
__device__ __forceinline__ void store_image(unsigned char* img, int tile, int atoms, int n0,
                                            bool last, uint32_t src, int ld, int plane, int tid) {
  using I = Image<KD, PO>;
  constexpr int V = NV / 8;
  for (int i = tid; i < PO * ROWS * V; i += 128) {
    const int row = i / V, n = n0 / 8 + i % V, p = row / ROWS;
    *reinterpret_cast<uint4*>(img + n / 8 * I::atom + tile + I::vec(row, n % 8)) =
        ptx::ld_shared_v4(src + p * plane + (row - p * ROWS) * ld + i % V * 16);
  }
  if (last)
    for (int n = n0 / 8 + V; n < 8 * atoms; ++n)
      for (int row = tid; row < PO * ROWS; row += 128)
        *reinterpret_cast<uint4*>(img + n / 8 * I::atom + tile + I::vec(row, n % 8)) =
            make_uint4(0, 0, 0, 0);
}

// The same places of chunks 0 .. chunks - 1 of a head get NaN instead, each from
// the thread that stored there.
template <int KD, int PO, int NV, int ROWS>
__device__ __noinline__ void void_image(unsigned char* img, int tile, int atoms, int n0, int chunks,
                                        int tid) {
  using I = Image<KD, PO>;
  constexpr int V = NV / 8;
  for (int c = 0; c < chunks; ++c, img += (long long)atoms * I::atom)
    for (int i = tid; i < PO * ROWS * V; i += 128) {
      const int row = i / V, n = n0 / 8 + i % V;
      *reinterpret_cast<uint4*>(img + n / 8 * I::atom + tile + I::vec(row, n % 8)) =
          make_uint4(~0u, ~0u, ~0u, ~0u);
    }
}

// ---- copies into a chain's stages ------------------------------------------------------
//
// Named barriers say when a stage is full and when it is free. Four warps copy:
// a chunk's record in one bulk copy, the rows of K, Q and V in 16-byte ones,
// which also make the rows behind a sequence and the columns behind a head zero
// (in bulk copies of a row each they took 6 us a chunk). fp32 rows are loaded,
// split into planes and stored.
constexpr int kLoadThreads = 128;

constexpr unsigned long long kWaitLimitNs = 2000000000ull;
constexpr int kFlagTimeout = 8;
__device__ __forceinline__ float void_value() { return __int_as_float(0x7fffffff); }

// Waits for a phase, up to kWaitLimitNs; then the workspace's flag says so, and
// `gave_up` (shared by the CTA) lets all later waits through, so that the CTA
// ends: named barriers keep their counts. Its results are void, and it overwrites
// them with NaN, so that this shows where nobody asks for the status (of a
// workspace that the caller never saw). At the end: as a NaN among the factors of
// every chunk it took 2 % of a forward call.
__device__ __forceinline__ void wait_phase(uint32_t bar, uint32_t parity, int* flag,
                                           volatile int* gave_up) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  const unsigned long long t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait_sleep(bar, parity, 1000000)) {
    if (*gave_up) return;
    if (ptx::globaltimer() - t0 > kWaitLimitNs) {
      atomicOr(flag, kFlagTimeout);
      *gave_up = 1;
      return;
    }
  }
}

// The sequence that the chains of rank `n` work on: the n-th longest, so that
// the last CTAs to start are short ones. Batches of random lengths, 16 heads,
// forward, five draws each in the order given and so: 8 sequences of up to 4096
// tokens of D 128: 449 and 426 us on average (526 and 451, 393 and 364 at best, 547
// and 551 at worst); 16 of up to 2048, D 64: 218 and 210; 64 of up to 1024, D 128,
// whose order matters least: 955 and 964. All threads of a CTA call, and meet
// here; `found` is shared by them.
constexpr int kRanked = 128;   // sequences: a thread compares its own with all
__device__ __forceinline__ int nth_longest(const Args& a, int n, volatile int* found) {
  const int t = threadIdx.x;
  if (a.lengths && a.B <= kRanked && t < a.B) {
    const int mine = length_of(a, t);
    int before = 0;
    for (int i = 0; i < a.B; ++i) {
      const int other = length_of(a, i);
      before += other > mine || (other == mine && i < t);
    }
    if (before == n) *found = t;
  }
  __syncthreads();
  return a.lengths && a.B <= kRanked ? *found : n;
}

// A record of BYTES into a stage, by the first of the threads that load.
template <int BYTES>
__device__ __forceinline__ void load_record(uint32_t dst, const unsigned char* src, uint32_t bar,
                                            int tid) {
  if (tid == 0) {
    ptx::mbar_expect_tx(bar, BYTES);
    ptx::bulk_load(dst, src, BYTES, bar);
  }
}

// How the four warps of a chain (and those that work beside it) divide a
// chunk's [64 tokens][16 RT columns] and the state's [KD][16 RT]: RT 1: a row
// tile each; RT 2: two row tiles and half of the columns each, so that the
// operand with the state's columns is loaded by two warps and not by four. Row
// tiles 0 and 3, 1 and 2 go together: a triangular factor has 1 + 4 and 2 + 3
// blocks there.
template <int KD, int RT>
struct Share {
  static constexpr int MS = KD * RT / 64;   // row tiles of the state
  int tile[RT], col, state;                 // row tiles; first column; first row of the state
  __device__ explicit Share(int w) {
    if (RT == 1) {
      tile[0] = w;
      col = 0;
      state = 16 * MS * w;
    } else {
      tile[0] = w & 1;
      tile[RT - 1] = 3 - (w & 1);
      col = 16 * (w >> 1);
      state = 16 * MS * (w & 1);
    }
  }
  // A [m][k] of this warp's row tiles
  __device__ mm::Operand rows(uint32_t at, int ld, int plane) const {
    mm::Operand o = mm::a_tile<false>(at + 16 * tile[0] * ld, ld, plane);
    o.tile = 16 * (tile[RT - 1] - tile[0]) * ld;
    return o;
  }
};

// ---- T and P ------------------------------------------------------------------------
//
// One CTA of four warps per (chunk, head): small, so that several share an SM
// and hide one another's latencies (alone a CTA takes 9,100 cycles at D 64).
// 16,384 chunks of D 64 take 220 us, of which their 814 MB (q and k once, the
// records written) would be 124 at the measured bandwidth. What bounds it is the
// work on single elements, the decays and the splits into planes: instruction issue
// is 52 % busy, shared memory 56 %, the tensor pipe 21 %. With two planes of P, at
// 208 us, P's stores were 8 % of it, the diagonal blocks' inversion 6 %, T's stores
// 4 %.
//
// A long sequence in parts, the next part's T and P made beside the chains of
// the last, gained nothing (1004 and 1005 us a call, with two planes of P): the
// chains slow down by as much.
//
// Warps 1 and 3 make the decays while 0 and 2 begin with the products, and have
// fewer of the ten blocks in turn. T = (I + A)^-1 by 16 x 16 blocks: each warp
// inverts one diagonal block by forward substitution in fp32, a column per lane;
// then warp j makes block column j from the top down,
//     T_ij = -T_ii (A_ij T_jj + ... + A_i,i-1 T_i-1,j),
// as transposed products: the transposed blocks of T that a warp has made
// stay in its registers as the left operands of the next product. A lies in
// T's place until T is written; a diagonal block's fp32 values take two of its
// planes. P goes to the record block by block, through 512 bytes: all of it in
// shared memory would leave room for four CTAs per SM at D = 64, not six.
enum { kTermsLoaded = 1, kTermsGates = 2 };   // named barriers

template <int PI, int KD, int PC>
struct TermsSmem {
  static constexpr int kLK = (KD + 8) * 2, kPlaneK = kC * kLK;
  static constexpr int offQ = PI * kPlaneK;
  static constexpr int offGate = 2 * PI * kPlaneK;   // Gates and T, as in the record
  static constexpr int offT = offGate + (int)sizeof(Gates);
  static constexpr int offD = offT + PC * mm::kTriPlane;
  static constexpr int offP = offD + (int)sizeof(Decays);
  static constexpr int bytes = offP + (PC > 2 ? 0 : 4 * 512);
  static constexpr int ctas = (PI == 1 ? 6 : 3) * 64 / (KD == 64 ? 64 : 96);   // per SM
};

template <typename T, int KD, int PC, int PO>
__global__ void __launch_bounds__(128, TermsSmem<mm::Io<T>::kPlanes, KD, PC>::ctas)
terms_kernel(const Args a) {
  constexpr int PI = mm::Io<T>::kPlanes;
  using L = TermsSmem<PI, KD, PC>;
  using R = Record<PC, PO>;
  static_assert(PC >= 2, "a diagonal block's fp32 values take two planes");
  ptx::launch_dependents();
  extern __shared__ __align__(16) unsigned char smem[];
  const uint32_t sK = ptx::smem_u32(smem), sQ = sK + L::offQ;
  Gates* gates = reinterpret_cast<Gates*>(smem + L::offGate);
  Decays* decays = reinterpret_cast<Decays*>(smem + L::offD);
  const uint32_t sT = sK + L::offT;

  const int chunk = blockIdx.x % a.chunks, bh = blockIdx.x / a.chunks;
  const int b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int rows = min(kC, length_of(a, b) - chunk * kC);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.flag = 0;
  if (rows <= 0) return;
  unsigned char* rec = a.rec + ((long long)bh * a.chunks + chunk) * R::bytes;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, r = lane >> 2, c2 = (lane & 3) * 2;
  {
    const Rows rk = rows_of(a, b, hk, a.Hk, a.D), rg = rows_of(a, b, h, a.H, 1);
    const long long at = (long long)chunk * kC;
    GateRows gr;
    if (w & 1)
      gr.load(static_cast<const T*>(a.g) + rg.base + at * rg.stride,
              static_cast<const T*>(a.beta) + rg.base + at * rg.stride, rg.stride, rows);
    mm::load_tile<T, kC, KD, 128>(sK, L::kLK, L::kPlaneK,
                                  static_cast<const T*>(a.k) + rk.base + at * rk.stride, rk.stride,
                                  rows, a.D, tid);
    mm::load_tile<T, kC, KD, 128>(sQ, L::kLK, L::kPlaneK,
                                  static_cast<const T*>(a.q) + rk.base + at * rk.stride, rk.stride,
                                  rows, a.D, tid);
    ptx::cp_async_wait_all();
    if (w & 1) {   // while the other warps begin
      ptx::bar_arrive(kTermsLoaded, 128);
      chunk_gates(gr, a.scale, w == 3, gates, decays);
      ptx::bar_sync(kTermsGates, 128);
    } else {
      ptx::bar_sync(kTermsLoaded, 128);
    }
  }

  // row r of the diagonal block w: 64 bytes, rows 0-7 in plane 0, 8-15 in plane 1
  unsigned char* diag = smem + L::offT + mm::tri_block(w, w);
  // and 512 bytes of this warp's for a block of P on its way out: the third plane
  // there, if T has one
  const uint32_t sP = PC > 2 ? sT + 2 * mm::kTriPlane + mm::tri_block(w, w) : sK + L::offP + 512 * w;
  // 16 rows x 32 columns at a time, column blocks right of the diagonal left
  // out: warps 1 and 3 the last of their rows, 0 and 2 the first, then the first
  // of rows 3 and the rest of rows 2
#pragma unroll 1
  for (int task = 0; task < 2 - (w & 1); ++task) {
    const int m = task == 0 ? w : (w == 0 ? 3 : 2), half = task == 0 ? w == 3 : w == 2;
    float acc[2][4][4];   // K K^T, Q K^T
    mm::zero(acc);
    mm::Operand ka = mm::a_tile<false>(sK + 16 * m * L::kLK, L::kLK, L::kPlaneK);
    ka.tile = L::offQ;
    mm::gemm<2, 4, PI, PI, PC, false, false, KD / 16, 2, PI == 3>(
        acc, ka, mm::b_tile<false>(sK + 32 * half * L::kLK, L::kLK, L::kPlaneK));
    if (task == 0 && !(w & 1)) ptx::bar_sync(kTermsGates, 128);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      const int j = 2 * half + blk;
      if (j > m) continue;
      float A[2][4], P[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int rr = r + 8 * i, row = 16 * m + rr;
        const float bt = gates->tok[row].y, up = decays->up[row];
        const double Gr = decays->G[row];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          const int cc = 8 * n + c2, col = 16 * j + cc;
          const float* kk = &acc[0][2 * blk + n][2 * i];
          const float* qk = &acc[1][2 * blk + n][2 * i];
          float E0, E1;
          if (j == m) {
            const double2 Gc = *reinterpret_cast<const double2*>(&decays->G[col]);
            E0 = cc <= rr ? expf((float)(Gr - Gc.x)) : 0.f;
            E1 = cc < rr ? expf((float)(Gr - Gc.y)) : 0.f;
            *reinterpret_cast<float2*>(diag + i * mm::kTriPlane + r * 64 + cc * 4) =
                make_float2(cc < rr ? bt * E0 * kk[0] : 0.f, cc + 1 < rr ? bt * E1 * kk[1] : 0.f);
          } else {
            const float2 dn = *reinterpret_cast<const float2*>(&decays->down[m - 1][col]);
            E0 = up * dn.x;
            E1 = up * dn.y;
            A[n][2 * i] = bt * E0 * kk[0];
            A[n][2 * i + 1] = bt * E1 * kk[1];
          }
          // above the diagonal the product could be anything
          P[n][2 * i] = j != m || cc <= rr ? a.scale * E0 * qk[0] : 0.f;
          P[n][2 * i + 1] = j != m || cc < rr ? a.scale * E1 * qk[1] : 0.f;
        }
      }
      const int at = mm::tri_block(m, j);
      if (j < m) mm::store_tile<PC>(sT + at + mm::tri_lane<false>(lane), mm::kTriPlane, A);
      // P goes out in whole rows, a plane at a time
      uint32_t words[4][PO];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        mm::split<PO>(P[u >> 1][(u & 1) * 2], P[u >> 1][(u & 1) * 2 + 1], words[u]);
#pragma unroll
      for (int o = 0; o < PO; ++o) {
        const uint32_t x[4] = {words[0][o], words[1][o], words[2][o], words[3][o]};
        mm::stsm(sP + mm::tri_lane<false>(lane), x);
        __syncwarp();
        *reinterpret_cast<uint4*>(rec + R::offP + o * mm::kTriPlane + at + lane * 16) =
            ptx::ld_shared_v4(sP + lane * 16);
        __syncwarp();
      }
    }
  }
  __syncwarp();

  // the diagonal block: column `cc` of its inverse; the two half warps make
  // the same and store every other row
  {
    const int cc = lane & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == cc ? 1.f : 0.f;
      const float* d = reinterpret_cast<const float*>(diag + (i >> 3) * mm::kTriPlane + (i & 7) * 64);
#pragma unroll
      for (int j = 0; j < i; j += 4) {
        const float4 y = *reinterpret_cast<const float4*>(d + j);
        s -= y.x * x[j];
        if (j + 1 < i) s -= y.y * x[j + 1];
        if (j + 2 < i) s -= y.z * x[j + 2];
        if (j + 3 < i) s -= y.w * x[j + 3];
      }
      x[i] = s;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      // lanes 0-15 store row i, the others row i + 1; even lanes a pair of columns
      const float y = lane < 16 ? x[i] : x[i + 1];
      const float z = __shfl_down_sync(0xffffffffu, y, 1);
      if ((lane & 1) == 0)
        mm::store_pair<PC>(sT + mm::tri_block(w, w) + mm::tri_at(i + (lane >> 4), cc),
                           mm::kTriPlane, y, z);
    }
  }
  __syncthreads();

  // block column w below the diagonal, transposed: t[k] = T_kw^T
  uint32_t t[4][PC][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k == w) {
#pragma unroll
      for (int p = 0; p < PC; ++p)
        mm::ldsm_t(t[k][p], sT + p * mm::kTriPlane + mm::tri_block(k, k) + mm::tri_lane<true>(lane));
    }
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    if (i <= w) continue;
    float m[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) m[n][j] = 0.f;
    uint32_t next[PC][4];
#pragma unroll
    for (int p = 0; p < PC; ++p)
      mm::ldsm(next[p], sT + p * mm::kTriPlane + mm::tri_block(i, w) + mm::tri_lane<true>(lane));
#pragma unroll
    for (int k = 0; k <= i; ++k) {
      if (k < w) continue;
      // k < i: M^T += T_kw^T A_ik^T;  k == i: T_iw^T = -M^T T_ii^T
      uint32_t fb[PC][4];
#pragma unroll
      for (int p = 0; p < PC; ++p) {
#pragma unroll
        for (int u = 0; u < 4; ++u) fb[p][u] = next[p][u];
        if (k < i)
          mm::ldsm(next[p],
                   sT + p * mm::kTriPlane + mm::tri_block(i, k + 1) + mm::tri_lane<true>(lane));
      }
      if (k == i) {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            uint32_t wds[PC];
            mm::split<PC>(-m[n][2 * u], -m[n][2 * u + 1], wds);
#pragma unroll
            for (int p = 0; p < PC; ++p) t[i][p][2 * n + u] = wds[p];
            m[n][2 * u] = m[n][2 * u + 1] = 0.f;
          }
      }
#pragma unroll
      for (int o = PC - 1; o >= 0; --o)
#pragma unroll
        for (int p = 0; p < PC; ++p)
#pragma unroll
          for (int q = 0; q < PC; ++q)
            if (p + q == o) {
#pragma unroll
              for (int n = 0; n < 2; ++n) mm::mma(m[n], t[k][p], fb[q][2 * n], fb[q][2 * n + 1]);
            }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t wds[PC];
        mm::split<PC>(m[n][2 * u], m[n][2 * u + 1], wds);
#pragma unroll
        for (int p = 0; p < PC; ++p) t[i][p][2 * n + u] = wds[p];
      }
  }
  __syncthreads();   // nobody reads A any more
#pragma unroll
  for (int i = 1; i < 4; ++i)
    if (i > w) {
#pragma unroll
      for (int p = 0; p < PC; ++p)
        mm::stsm_t(sT + p * mm::kTriPlane + mm::tri_block(i, w) +
                       mm::tri_at((lane & 7) + (lane >> 4) * 8, ((lane >> 3) & 1) * 8),
                   t[i][p]);
    }
  ptx::fence_proxy_async();
  __syncthreads();
  // Gates and T lie as in the record
  if (tid == 0) {
    mm::bulk_store(rec, sK + L::offGate, R::offP);
    mm::bulk_store(rec + R::offD, sK + L::offD, sizeof(Decays));
    ptx::bulk_commit();
    ptx::bulk_wait_read<0>();
  }
}

}  // namespace delta
}  // namespace la
