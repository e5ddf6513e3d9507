// The bounded wait of the delta rule's chains (wait_phase in delta.cuh): one that
// nothing ends gives up by itself, says so in the flag and to its CTA, whose later
// waits then end at once; one that ends in time leaves no trace. And what a CTA
// that gave up overwrites: the outputs of its columns and no others, the places of
// its images and no others. Prints "ok" or what differs.
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "delta_scan.cuh"

using namespace la;

// mbarrier 0 never gets its arrival unless `arrive`; mbarrier 1 never does
__global__ void waits(int* flag, float* out, int arrive) {
  __shared__ __align__(8) unsigned long long bars[2];
  __shared__ int gave_up;
  const uint32_t bar = ptx::smem_u32(bars);
  if (threadIdx.x == 0) {
    ptx::mbar_init(bar, 1);
    ptx::mbar_init(bar + 8, 1);
    gave_up = 0;
    ptx::fence_mbar_init();
  }
  __syncthreads();
  if (arrive && threadIdx.x == 0) ptx::mbar_arrive(bar);
  delta::wait_phase(bar, 0, flag, &gave_up);
  if (!arrive) delta::wait_phase(bar + 8, 0, flag, &gave_up);   // at once
  __syncthreads();
  out[threadIdx.x] = gave_up ? delta::void_value() : 1.f;
}

// The outputs' warps of slice `slice` of a head with `len` of N tokens.
template <int RT>
__global__ void void_outputs(delta::bf16* out, int N, int len, int Dv, int slice) {
  const delta::Share<64, RT> sh(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, n0 = 16 * RT * slice + sh.col + (lane & 3) * 2;
  for (int j = 0; j < RT; ++j)
    delta::void_rows(out + n0, (long long)Dv, 16 * sh.tile[j] + (lane >> 2), len, Dv - n0);
}

template <int KD, int PO, int NV, int ROWS>
__global__ void images(unsigned char* img, int tile, int slice, int chunks, bool bad) {
  extern __shared__ __align__(16) unsigned char smem[];
  using I = delta::Image<KD, PO>;
  if (bad)
    return delta::void_image<KD, PO, NV, ROWS>(img, tile, 2, slice * NV, chunks, threadIdx.x);
  for (int i = threadIdx.x; i < PO * ROWS * (NV + 8) * 2; i += 128) smem[i] = 0xff;
  __syncthreads();
  for (int c = 0; c < chunks; ++c)
    delta::store_image<KD, PO, NV, ROWS>(img + c * 2LL * I::atom, tile, 2, slice * NV, false,
                                         ptx::smem_u32(smem), (NV + 8) * 2, ROWS * (NV + 8) * 2,
                                         threadIdx.x);
}

template <int RT>
int check_outputs() {
  const int N = 200, len = 150, Dv = 72;
  delta::bf16* out;
  if (cudaMallocManaged(&out, N * Dv * 2) != cudaSuccess) return printf("no memory\n"), 1;
  for (int slice = 0; slice * 16 * RT < Dv; ++slice) {
    memset(out, 0, N * Dv * 2);
    void_outputs<RT><<<1, 128>>>(out, N, len, Dv, slice);
    if (cudaDeviceSynchronize() != cudaSuccess) return printf("a launch failed\n"), 1;
    for (int i = 0; i < N * Dv; ++i) {
      const bool in = i / Dv < len && i % Dv / (16 * RT) == slice;
      if (isnan(__bfloat162float(out[i])) != in) return printf("output %d, slice %d\n", i, slice), 1;
    }
  }
  return 0;
}

template <int KD, int PO, int NV, int ROWS>
int check_images(int tile) {
  const int chunks = 3, n = chunks * 2 * delta::Image<KD, PO>::atom;
  unsigned char *a, *b;
  if (cudaMallocManaged(&a, n) != cudaSuccess || cudaMallocManaged(&b, n) != cudaSuccess)
    return printf("no memory\n"), 1;
  for (int slice = 0; slice * NV < 128; ++slice) {
    memset(a, 0, n);
    memset(b, 0, n);
    images<KD, PO, NV, ROWS><<<1, 128, PO * ROWS * (NV + 8) * 2>>>(a, tile, slice, chunks, false);
    images<KD, PO, NV, ROWS><<<1, 128>>>(b, tile, slice, chunks, true);
    if (cudaDeviceSynchronize() != cudaSuccess) return printf("a launch failed\n"), 1;
    if (memcmp(a, b, n)) return printf("image %d, slice %d\n", tile, slice), 1;
  }
  return 0;
}

int main() {
  if (check_outputs<1>() || check_outputs<2>()) return 1;
  using I2 = delta::Image<64, 2>;
  using I3 = delta::Image<128, 3>;
  if (check_images<64, 2, 16, 64>(I2::offX) || check_images<64, 2, 32, 64>(I2::offS) ||
      check_images<128, 3, 16, 64>(I3::offR) || check_images<128, 3, 16, 128>(I3::offD))
    return 1;
  constexpr int n = 64;
  int* flag;
  float* out;
  if (cudaMallocManaged(&flag, sizeof(int)) != cudaSuccess ||
      cudaMallocManaged(&out, n * sizeof(float)) != cudaSuccess)
    return printf("no memory\n"), 1;
  for (int arrive = 1; arrive >= 0; --arrive) {
    *flag = 0;
    cudaEvent_t a, b;
    cudaEventCreate(&a);
    cudaEventCreate(&b);
    cudaEventRecord(a);
    waits<<<1, n>>>(flag, out, arrive);
    cudaEventRecord(b);
    if (cudaDeviceSynchronize() != cudaSuccess) return printf("a launch failed\n"), 1;
    float ms = 0.f;
    cudaEventElapsedTime(&ms, a, b);
    const double limit = delta::kWaitLimitNs * 1e-6;
    if (arrive ? ms > limit : ms < limit || ms > 2 * limit) return printf("%g ms\n", ms), 1;
    if (*flag != (arrive ? 0 : delta::kFlagTimeout)) return printf("flag %d\n", *flag), 1;
    for (int i = 0; i < n; ++i)
      if (arrive ? out[i] != 1.f : !isnan(out[i])) return printf("result %g\n", out[i]), 1;
  }
  printf("ok\n");
  return 0;
}
