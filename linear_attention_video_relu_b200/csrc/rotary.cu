// rotary.cu -- rotary positions of query and key heads (lin_attn_rotary in
// include/linattn.h), and their gradient, which is the transposed rotation.
//
// Every element is read once and written once, so HBM bandwidth bounds it: 537 MB
// in 83 us (D 64, interleaved, a 3D grid, 64 heads), 336 MB in 52 us (half
// layout, half of 128 columns), both at the measured copy's rate. A
// thread has one 16-byte vector of columns of one token (two vectors half a
// segment apart in the half layout) and takes the token's heads one after
// another: the angles are worked out once and kept in registers,
// and several heads' loads are under way at a time. Where there are few tokens
// the heads are split over more threads, which work the same angles out again.
// Rotated vectors and copied ones are different threads' (the grid's first part
// and its second), so that no warp does both. Halves that are no whole number of
// vectors go through shared memory: vectors in, each column's partner from
// wherever it lies, vectors out.
#include "linattn.h"

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;
constexpr int kAhead = 8;   // vectors whose loads a thread issues together
constexpr int kHeads = 4;   // heads are split over threads down to this many each

struct Args {
  const void *q, *k;
  void *q_out, *k_out;
  const int* positions;   // [N] or [B, N], or null: offset + n
  int pos_batch;          // positions of batch entry b start at b * pos_batch
  int offset;
  int B, H, Hk, N, D, dim;
  int bnhd;
  int axes;               // 1, or 3: the latent grid
  int Hg, Wg;
  int start[4];           // first column of each axis' segment, then dim
  int items, rest;        // rotated and copied vectors (or pairs of them) of a row
  int tokens;             // B N
  int per_thread;         // heads per thread
  float amplitude, sign;
  uint64_t freq[kMaxPairs]; // turns per position, less whole ones, in 2^-64
};

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ void unpack(const uint4& r, float (&f)[4]) {
  f[0] = __uint_as_float(r.x);
  f[1] = __uint_as_float(r.y);
  f[2] = __uint_as_float(r.z);
  f[3] = __uint_as_float(r.w);
}
__device__ __forceinline__ void unpack(const uint4& r, float (&f)[8]) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = reinterpret_cast<const uint32_t&>(h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// `y`, but with the words of `x` from column `from` of the vector on (even, as
// dim is): what is not rotated keeps its bits.
template <typename T>
__device__ __forceinline__ uint4 keep(const uint4& x, const uint4& y, int from) {
  constexpr int E = 4 / (int)sizeof(T);   // columns per word
  return make_uint4(from > 0 ? y.x : x.x, from > E ? y.y : x.y, from > 2 * E ? y.z : x.z,
                    from > 3 * E ? y.w : x.w);
}

// A token's heads: where they begin in q and in k, and how far apart they are.
struct Heads {
  long long q, k, step;
};
__device__ __forceinline__ Heads heads_of(const Args& a, int token, int b, int n) {
  Heads r;
  if (a.bnhd) {
    r.q = (long long)token * a.H * a.D;
    r.k = (long long)token * a.Hk * a.D;
    r.step = a.D;
  } else {
    r.q = ((long long)b * a.H * a.N + n) * a.D;
    r.k = ((long long)b * a.Hk * a.N + n) * a.D;
    r.step = (long long)a.N * a.D;
  }
  return r;
}
__device__ __forceinline__ long long head_at(const Args& a, const Heads& t, int h) {
  return h < a.H ? t.q + h * t.step : t.k + (h - a.H) * t.step;
}

// The token's position along the axis.
__device__ __forceinline__ int position(const Args& a, int axis, int b, int n) {
  if (a.axes == 3) {
    const int hw = n / a.Wg;
    return axis == 0 ? a.offset + hw / a.Hg : axis == 1 ? hw % a.Hg : n - hw * a.Wg;
  }
  return a.positions ? a.positions[(long long)b * a.pos_batch + n] : a.offset + n;
}

// cos and sin of pair `m` at position `pos`. The angle is kept in 2^-64 turns,
// where whole turns fall off a 64-bit product by themselves and nothing is rounded:
// what is left is off by the frequency's own error times pos. The frequencies are
// made in 64-bit floating point, up to 2^-55 turns off (theta >= 1), so an angle
// is off by less than 2^-24 turns (3e-7 radians, an fp32 rounding) at every position
// of 32 bits, where an fp32 product would lose whole turns. The upper 32 bits, as a
// signed number of 2^-31 half turns, go to sincospi.
__device__ __forceinline__ void turn(const Args& a, int m, int pos, float* c, float* s) {
  const uint64_t x = (uint64_t)(int64_t)pos * a.freq[m];
  float sn, cs;
  sincospif((float)(int32_t)(x >> 32) * 0x1p-31f, &sn, &cs);
  *c = a.amplitude * cs;
  *s = a.sign * a.amplitude * sn;
}

// Copies what is not rotated of a token's heads: the thread's vector.
template <typename T>
__device__ __forceinline__ void copy_rest(const Args& a, int token, int col) {
  const int b = token / a.N;
  const Heads t = heads_of(a, token, b, token - b * a.N);
  const int h0 = blockIdx.y * a.per_thread, h1 = min(a.H + a.Hk, h0 + a.per_thread);
  for (int h = h0; h < h1; h += kAhead) {
    uint4 x[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (h + j < h1)
        x[j] = *reinterpret_cast<const uint4*>(static_cast<const T*>(h + j >= a.H ? a.k : a.q) +
                                               head_at(a, t, h + j) + col);
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (h + j < h1)
        *reinterpret_cast<uint4*>(static_cast<T*>(h + j >= a.H ? a.k_out : a.q_out) +
                                  head_at(a, t, h + j) + col) = x[j];
  }
}

// HALF: the pair (x, y) is a vector and the one half a segment on; else
// neighbours in a vector.
template <typename T, bool HALF>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ Args a) {
  constexpr int W = kVec<T>, P = HALF ? W : W / 2;   // pairs of a thread
  constexpr int AHEAD = HALF ? kAhead / 2 : kAhead;
  unsigned idx = blockIdx.x * kThreads + threadIdx.x;
  const unsigned rotated = (unsigned)a.tokens * (unsigned)a.items;
  if (idx >= rotated) {
    idx -= rotated;
    const int token = (int)(idx / (unsigned)max(a.rest, 1));
    if (a.rest && token < a.tokens)
      copy_rest<T>(a, token, a.D - a.rest * W + (int)(idx % (unsigned)a.rest) * W);
    return;
  }
  const int item = (int)(idx % (unsigned)a.items), token = (int)(idx / (unsigned)a.items);
  const int b = token / a.N, n = token - b * a.N;

  int col = item * W, second = 0, axis = 0;
  const int pair = HALF ? col : col / 2;
  if (HALF) {
    while (2 * pair >= a.start[axis + 1]) ++axis;
    col = a.start[axis] + pair - a.start[axis] / 2;
    second = (a.start[axis + 1] - a.start[axis]) / 2;
  }
  float c[P], s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
    if (!HALF && 2 * (pair + i) >= a.dim) continue;   // a vector that straddles dim
    if (!HALF && a.axes == 3)
      axis = 2 * (pair + i) >= a.start[1] ? (2 * (pair + i) >= a.start[2] ? 2 : 1) : 0;
    turn(a, pair + i, position(a, axis, b, n), &c[i], &s[i]);
  }

  const Heads t = heads_of(a, token, b, n);
  const int h0 = blockIdx.y * a.per_thread, h1 = min(a.H + a.Hk, h0 + a.per_thread);
  for (int h = h0; h < h1; h += AHEAD) {
    uint4 x[AHEAD], y[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (h + j >= h1) continue;
      const T* src = static_cast<const T*>(h + j >= a.H ? a.k : a.q) + head_at(a, t, h + j) + col;
      x[j] = *reinterpret_cast<const uint4*>(src);
      if (HALF) y[j] = *reinterpret_cast<const uint4*>(src + second);
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (h + j >= h1) continue;
      T* dst = static_cast<T*>(h + j >= a.H ? a.k_out : a.q_out) + head_at(a, t, h + j) + col;
      float f[W], g[W];
      unpack(x[j], f);
      if (HALF) {
        unpack(y[j], g);
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float u = f[i], v = g[i];
          f[i] = u * c[i] - v * s[i];
          g[i] = u * s[i] + v * c[i];
        }
        *reinterpret_cast<uint4*>(dst + second) = pack(g);
      } else {
#pragma unroll
        for (int i = 0; i < W; i += 2) {
          const float u = f[i], v = f[i + 1];
          f[i] = u * c[i / 2] - v * s[i / 2];
          f[i + 1] = u * s[i / 2] + v * c[i / 2];
        }
      }
      *reinterpret_cast<uint4*>(dst) = HALF ? pack(f) : keep<T>(x[j], pack(f), a.dim - 2 * pair);
    }
  }
}

// The half layout with halves of any width: a thread has one vector of columns,
// whose partners it reads from its row in shared memory. A CTA has whole rows
// (their rotated columns), so it may rotate in place: all of a row is read
// before any of it is written. The CTA's angles are worked out once each, by
// all threads alike. (19 MB, 30,030 rows of 80 fp32 columns of which 20 turn:
// 7.0 us with cold caches, 5.6 in a loop that is replayed, of which the bytes are
// 2.9; the rest is the latency of the angles, the loads and the way through shared
// memory, one after another. 64 heads of 32,760 tokens, 20 of 80 bf16 columns, 671
// MB: 286 us, 2.8 times what the bytes take, by the same way.)
template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_rows_kernel(const __grid_constant__ Args a,
                                                               int row_blocks) {
  constexpr int W = kVec<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  if ((int)blockIdx.x >= row_blocks) {
    const unsigned idx = (blockIdx.x - row_blocks) * blockDim.x + threadIdx.x;
    const int token = (int)(idx / (unsigned)max(a.rest, 1));
    if (a.rest && token < a.tokens)
      copy_rest<T>(a, token, a.D - a.rest * W + (int)(idx % (unsigned)a.rest) * W);
    return;
  }
  const int per_block = blockDim.x / a.items, pairs = a.dim / 2, width = a.items * W;
  const int item = threadIdx.x % a.items, local = threadIdx.x / a.items;
  const int token0 = blockIdx.x * per_block, token = token0 + local;
  const bool live = token < a.tokens;
  const int b = live ? token / a.N : 0, n = live ? token - b * a.N : 0;
  const int col = item * W;

  // the angles behind the two sets of rows
  float2* table = reinterpret_cast<float2*>(smem + 2 * kHeads * per_block * width * sizeof(T));
  for (int i = threadIdx.x; i < per_block * pairs; i += blockDim.x) {
    const int t = i / pairs, m = i - t * pairs;
    if (token0 + t >= a.tokens) break;
    const int tb = (token0 + t) / a.N;
    int axis = 0;
    while (2 * m >= a.start[axis + 1]) ++axis;
    float2 cs;
    turn(a, m, position(a, axis, tb, token0 + t - tb * a.N), &cs.x, &cs.y);
    table[i] = cs;
  }
  __syncthreads();
  float c[W], s[W];   // out = c x[own] + s x[partner]
  int partner[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int d = col + i;
    c[i] = 1.f;
    s[i] = 0.f;
    partner[i] = d;
    if (d >= a.dim || !live) continue;
    int axis = 0;
    while (d >= a.start[axis + 1]) ++axis;
    const int half = (a.start[axis + 1] - a.start[axis]) / 2, m = d - a.start[axis];
    const bool low = m < half;
    const float2 cs = table[local * pairs + a.start[axis] / 2 + (low ? m : m - half)];
    c[i] = cs.x;
    s[i] = low ? -cs.y : cs.y;
    partner[i] = low ? d + half : d - half;
  }

  const Heads at = heads_of(a, token, b, n);
  const int h0 = blockIdx.y * a.per_thread, h1 = min(a.H + a.Hk, h0 + a.per_thread);
  T* rows = reinterpret_cast<T*>(smem);
  for (int h = h0, z = 0; h < h1; h += kHeads, z ^= 1) {
    uint4 x[kHeads];
    // two sets of rows: a thread ahead writes the other one
    T* set = rows + z * kHeads * per_block * width;
#pragma unroll
    for (int j = 0; j < kHeads; ++j)
      if (h + j < h1 && live)
        x[j] = *reinterpret_cast<const uint4*>(static_cast<const T*>(h + j >= a.H ? a.k : a.q) +
                                               head_at(a, at, h + j) + col);
#pragma unroll
    for (int j = 0; j < kHeads; ++j)
      if (h + j < h1 && live)
        *reinterpret_cast<uint4*>(set + (j * per_block + local) * width + col) = x[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
      if (h + j >= h1 || !live) continue;
      const T* row = set + (j * per_block + local) * width;
      float f[W];
      unpack(x[j], f);
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i < a.dim) f[i] = f[i] * c[i] + (float)row[partner[i]] * s[i];
      *reinterpret_cast<uint4*>(static_cast<T*>(h + j >= a.H ? a.k_out : a.q_out) +
                                head_at(a, at, h + j) + col) = keep<T>(x[j], pack(f), a.dim - col);
    }
  }
}

// Splits the heads: two full waves of threads, but no fewer than kHeads heads
// each. (32 + 32 heads of 32,760 tokens: 83 us; eight waves, which work every
// angle out four times as often, 110 us.) Returns the grid's y.
unsigned split_heads(Args& a, long long threads, int sms) {
  const int heads = a.H + a.Hk;
  long long groups = (2LL * sms * 2048 + threads - 1) / threads;
  const long long most = (heads + kHeads - 1) / kHeads;
  if (groups > most) groups = most;
  a.per_thread = (int)((heads + groups - 1) / groups + kHeads - 1) / kHeads * kHeads;
  return (unsigned)((heads + a.per_thread - 1) / a.per_thread);
}

template <typename T>
la_status launch(Args& a, bool half, bool in_place, int sms, cudaStream_t stream) {
  constexpr int W = kVec<T>;
  // the half layout by pairs of vectors: every half is whole vectors
  bool whole = true;
  for (int i = 0; i < a.axes; ++i) whole = whole && (a.start[i + 1] - a.start[i]) % (2 * W) == 0;
  const int rotated = (a.dim + W - 1) / W;
  a.items = half && whole ? a.dim / 2 / W : rotated;
  a.rest = in_place ? 0 : a.D / W - rotated;
  const long long threads = (long long)a.tokens * (a.items + a.rest);
  if (threads > (long long)INT_MAX - 2 * kThreads) return LA_ERR_UNSUPPORTED;
  const unsigned y = split_heads(a, threads, sms);
  if (half && !whole) {
    const int per_block = kThreads / a.items, block = per_block * a.items;
    // at most 2 x 4 x 256 vectors of rows, and the pairs of 256
    const size_t smem = (size_t)per_block * (2 * kHeads * a.items * 16 + a.dim / 2 * sizeof(float2));
    const int row_blocks = (a.tokens + per_block - 1) / per_block;
    const long long rest = (long long)a.tokens * a.rest;
    rotary_rows_kernel<T><<<dim3((unsigned)(row_blocks + (rest + block - 1) / block), y), block, smem,
                            stream>>>(a, row_blocks);
  } else {
    const dim3 grid((unsigned)((threads + kThreads - 1) / kThreads), y);
    if (half) rotary_kernel<T, true><<<grid, kThreads, 0, stream>>>(a);
    else rotary_kernel<T, false><<<grid, kThreads, 0, stream>>>(a);
  }
  return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
  return a0 < b0 + nb && b0 < a0 + na;
}

la_status check(const la_rotary_params* p, bool has_k) {
  if (!p) return LA_ERR_INVALID_ARG;
  if (p->B < 0 || p->H < 0 || p->Hk < 0 || p->N < 0) return LA_ERR_INVALID_ARG;
  if (!has_k && p->Hk != 0) return LA_ERR_INVALID_ARG;
  if (p->D < 8 || p->D > 2 * kMaxPairs || p->D % 8) return LA_ERR_INVALID_ARG;
  if (p->dim < 2 || p->dim > p->D || p->dim % 2) return LA_ERR_INVALID_ARG;
  if (p->dtype != LA_F32 && p->dtype != LA_BF16) return LA_ERR_INVALID_ARG;
  if (p->layout != LA_LAYOUT_BHND && p->layout != LA_LAYOUT_BNHD) return LA_ERR_INVALID_ARG;
  if (p->style != LA_ROTARY_INTERLEAVED && p->style != LA_ROTARY_HALF) return LA_ERR_INVALID_ARG;
  if (!(p->theta > 0.0) || isinf(p->theta) || !isfinite(p->amplitude)) return LA_ERR_INVALID_ARG;
  switch (p->scaling) {
    case LA_ROTARY_NO_SCALING: break;
    case LA_ROTARY_NTK:
      if (p->dim == 2) return LA_ERR_INVALID_ARG;   // its exponent is dim / (dim - 2)
    case LA_ROTARY_LINEAR:
    case LA_ROTARY_BY_PARTS:
      if (!(p->factor > 0.0) || isinf(p->factor)) return LA_ERR_INVALID_ARG;
      break;
    default: return LA_ERR_INVALID_ARG;
  }
  if (p->scaling == LA_ROTARY_BY_PARTS &&
      (!(p->original_length > 0.0) || isinf(p->original_length) || !(p->high > p->low) ||
       isinf(p->high) || isinf(p->low)))
    return LA_ERR_INVALID_ARG;
  if (p->grid_t || p->grid_h || p->grid_w) {
    if (p->grid_t < 1 || p->grid_h < 1 || p->grid_w < 1) return LA_ERR_INVALID_ARG;
    if ((long long)p->grid_t * p->grid_h * p->grid_w != p->N) return LA_ERR_INVALID_ARG;
    if (p->rope_dt < 0 || p->rope_dh < 0 || p->rope_dw < 0 ||
        ((p->rope_dt | p->rope_dh | p->rope_dw) & 1) ||
        (long long)p->rope_dt + p->rope_dh + p->rope_dw != p->dim)
      return LA_ERR_INVALID_ARG;
    if (p->scaling != LA_ROTARY_NO_SCALING) return LA_ERR_INVALID_ARG;
  }
  const long long last = (long long)p->offset + (p->grid_t ? p->grid_t : p->N) - 1;
  if (last > INT_MAX) return LA_ERR_UNSUPPORTED;
  if ((long long)p->B * p->N > INT_MAX || (long long)p->H + p->Hk > (1 << 16))
    return LA_ERR_UNSUPPORTED;
  return LA_OK;
}

}  // namespace

extern "C" {

la_status lin_attn_rotary(const la_rotary_params* p, const void* q, const void* k,
                          const int* positions, void* q_out, void* k_out, void* stream) {
  la_status st = check(p, k != nullptr);
  if (st != LA_OK) return st;
  const size_t elt = p->dtype == LA_BF16 ? 2 : 4, tokens = (size_t)p->B * p->N;
  const size_t nq = tokens * p->H * p->D * elt, nk = tokens * p->Hk * p->D * elt;
  if (nq + nk == 0) return LA_OK;
  if ((nq && (!q || !q_out)) || (nk && (!k || !k_out))) return LA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) ||
      ((uintptr_t)positions & 3u))
    return LA_ERR_INVALID_ARG;
  const bool grid = p->grid_t > 0;
  if (grid && positions) return LA_ERR_INVALID_ARG;
  const size_t npos = (p->positions_per_batch ? tokens : (size_t)p->N) * sizeof(int);
  if ((q_out != q && overlaps(q_out, nq, q, nq)) || (k_out != k && overlaps(k_out, nk, k, nk)) ||
      overlaps(q_out, nq, k, nk) || overlaps(k_out, nk, q, nq) || overlaps(q_out, nq, k_out, nk) ||
      overlaps(q_out, nq, positions, npos) || overlaps(k_out, nk, positions, npos))
    return LA_ERR_INVALID_ARG;
  Args a;
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.positions = positions;
  a.pos_batch = p->positions_per_batch ? p->N : 0;
  a.offset = p->offset;
  a.B = p->B;
  a.H = p->H;
  a.Hk = p->Hk;
  a.N = p->N;
  a.D = p->D;
  a.dim = p->dim;
  a.bnhd = p->layout == LA_LAYOUT_BNHD;
  a.axes = grid ? 3 : 1;
  a.Hg = p->grid_h;
  a.Wg = p->grid_w;
  a.start[1] = grid ? p->rope_dt : p->dim;
  a.start[2] = a.start[1] + (grid ? p->rope_dh : 0);
  a.start[3] = p->dim;
  a.tokens = (int)tokens;
  const bool in_place = (nq == 0 || q_out == q) && (nk == 0 || k_out == k);
  a.amplitude = p->amplitude;
  a.sign = p->transpose ? -1.f : 1.f;
  for (int i = 0, m = 0; i < a.axes; ++i) {
    const int width = a.start[i + 1] - a.start[i];
    double theta = p->theta;
    if (p->scaling == LA_ROTARY_NTK) theta *= pow(p->factor, width / (width - 2.0));
    const double octaves = width ? -2.0 * log2(theta) / width : 0.0;
    for (int j = 0; j < width / 2; ++j, ++m) {
      double f = exp2(j * octaves);
      if (p->scaling == LA_ROTARY_LINEAR) f /= p->factor;
      if (p->scaling == LA_ROTARY_BY_PARTS) {
        // whole turns over the original length: `high` and more keep their
        // frequency, `low` and less are stretched
        double keep = (p->original_length * f / (2.0 * M_PI) - p->low) / (p->high - p->low);
        keep = keep < 0.0 ? 0.0 : (keep > 1.0 ? 1.0 : keep);
        f = f * keep + f / p->factor * (1.0 - keep);
      }
      if (!isfinite(f)) return LA_ERR_INVALID_ARG;   // far from 1: theta or factor
      f /= 2.0 * M_PI;
      a.freq[m] = (uint64_t)((f - floor(f)) * 0x1p64);   // below 2^64: f - floor(f) < 1
    }
  }
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return LA_ERR_CUDA;
  }
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool half = p->style == LA_ROTARY_HALF;
  return p->dtype == LA_BF16 ? launch<bf16>(a, half, in_place, sms, cs)
                             : launch<float>(a, half, in_place, sms, cs);
}

}  // extern "C"
