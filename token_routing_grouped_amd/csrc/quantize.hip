// Rows and weights in 8 bits: e4m3 values with a power-of-two scale per block of 128.
//
// Rows: x [N,H] -> q [N,H], one scale per 128 consecutive values. Bound by memory: 2 (or
// 4) bytes read and 1 written per value. A lane holds eight values, so the 16 lanes of a
// DPP row hold one block and its maximum takes four lane moves; nothing goes through LDS.
// Measured: 8192 x 7168 bf16 (178 MB) 30 us, 5.9 TB/s.
//
// Weights: w [E,K,C] -> q [E,C,K], one scale per 128 x 128. A workgroup takes one block: a
// thread loads an 8 x 8 piece, so it can pack eight k-consecutive bytes of a column, and
// the bytes are transposed through LDS so that both the reads (256-byte runs along C) and
// the writes (128-byte runs along K) are whole cache lines. Measured: 32 x 2048 x 1024 bf16
// (201 MB) 35 us, 5.7 TB/s.
#include "fp8.h"
#include "kernels.h"

namespace moe {
namespace {

constexpr int QT = 256;

template <typename T>
__global__ __launch_bounds__(QT) void quantize_rows_kernel(const T *__restrict__ x, int64_t ngroup,
                                                           int H, int nb, uint8_t *__restrict__ q,
                                                           void *__restrict__ scale, int e8m0) {
  const int64_t gidx = ((int64_t)blockIdx.x * QT + threadIdx.x) >> 4;  // block of 128 values
  const int l = threadIdx.x & 15;
  const bool live = gidx < ngroup;
  const int64_t row = live ? gidx / nb : 0;
  const int b = live ? (int)(gidx - row * nb) : 0;
  const int c = b * kQB + l * 8;
  const bool in = live && c < H;
  typename Vec8<T>::Raw raw = in ? Vec8<T>::load(x + row * H + c) : Vec8<T>::zero();
  float f[8];
  Vec8<T>::get(raw, f);
  u32x2 v;
  const uint32_t e = quantize8(f, &v);
  if (in) *(u32x2 *)(q + row * H + c) = v;
  if (live && l == 0) store_scale(scale, e8m0, gidx, e);
}

template <typename T>
__global__ __launch_bounds__(QT) void quantize_weights_kernel(const T *__restrict__ w, int K, int C,
                                                              int nbk, int nbc,
                                                              uint8_t *__restrict__ q,
                                                              void *__restrict__ scale, int e8m0) {
  constexpr int LD = kQB + 16;
  __shared__ __attribute__((aligned(16))) uint8_t t[kQB * LD];  // [column][k]
  __shared__ uint32_t red[QT / 64];
  const int tid = threadIdx.x;
  const int64_t blk = blockIdx.x;
  const int bk = (int)(blk % nbk);
  const int64_t ec = blk / nbk;
  const int bc = (int)(ec % nbc);
  const int64_t e_ = ec / nbc;
  const int cc = tid & 15, kr = (tid >> 4) * 8;  // this thread's 8 columns and 8 rows
  const int c0 = bc * kQB + cc * 8, k0 = bk * kQB + kr;
  const T *wp = w + (e_ * K) * C;
  typename Vec8<T>::Raw raw[8];
#pragma unroll
  for (int i = 0; i < 8; i++)
    raw[i] = (k0 + i < K && c0 < C) ? Vec8<T>::load(wp + (int64_t)(k0 + i) * C + c0)
                                    : Vec8<T>::zero();
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; i++) {
    float f[8];
    Vec8<T>::get(raw[i], f);
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const uint32_t b = finite_abs_bits(f[j]);
      m = m > b ? m : b;
    }
  }
  m = row16_max(m);
#pragma unroll
  for (int o = 16; o < 64; o <<= 1) {
    const uint32_t v = (uint32_t)__shfl_xor((int)m, o, kWave);
    m = m > v ? m : v;
  }
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < QT / 64; i++) m = m > red[i] ? m : red[i];
  const uint32_t e = scale_exponent(m);
  const float inv = exponent_inverse(e);
  float f[8][8];
#pragma unroll
  for (int i = 0; i < 8; i++) Vec8<T>::get(raw[i], f[i]);
#pragma unroll
  for (int j = 0; j < 8; j++) {
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; i++) g[i] = to_q(f[i][j], inv);
    *(u32x2 *)(t + (cc * 8 + j) * LD + kr) =
        u32x2{pack_e4m3(g[0], g[1], g[2], g[3]), pack_e4m3(g[4], g[5], g[6], g[7])};
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kQB * 8 / QT; i++) {
    const int s = tid + QT * i, col = s >> 3, ch = (s & 7) * 16;
    const int gc = bc * kQB + col, gk = bk * kQB + ch;
    if (gc < C && gk < K)  // K is a multiple of 16
      *(u32x4 *)(q + (e_ * C + gc) * K + gk) = *(const u32x4 *)(t + col * LD + ch);
  }
  if (tid == 0) store_scale(scale, e8m0, (e_ * nbc + bc) * nbk + bk, e);
}

}  // namespace

hipError_t launch_quantize_rows(const void *x, int N, int H, bool bf16, void *q, void *scale,
                                int e8m0, hipStream_t st) {
  const int nb = (H + kQB - 1) / kQB;
  const int64_t ngroup = (int64_t)N * nb, grid = (ngroup * 16 + QT - 1) / QT;
  if (grid == 0) return hipSuccess;
  if (bf16)
    hipLaunchKernelGGL(quantize_rows_kernel<uint16_t>, dim3((uint32_t)grid), dim3(QT), 0, st,
                       (const uint16_t *)x, ngroup, H, nb, (uint8_t *)q, scale, e8m0);
  else
    hipLaunchKernelGGL(quantize_rows_kernel<float>, dim3((uint32_t)grid), dim3(QT), 0, st,
                       (const float *)x, ngroup, H, nb, (uint8_t *)q, scale, e8m0);
  return hipGetLastError();
}

hipError_t launch_quantize_weights(const void *w, int E, int K, int C, bool bf16, void *q,
                                   void *scale, int e8m0, hipStream_t st) {
  const int nbk = (K + kQB - 1) / kQB, nbc = (C + kQB - 1) / kQB;
  const int64_t grid = (int64_t)E * nbk * nbc;
  if (bf16)
    hipLaunchKernelGGL(quantize_weights_kernel<uint16_t>, dim3((uint32_t)grid), dim3(QT), 0, st,
                       (const uint16_t *)w, K, C, nbk, nbc, (uint8_t *)q, scale, e8m0);
  else
    hipLaunchKernelGGL(quantize_weights_kernel<float>, dim3((uint32_t)grid), dim3(QT), 0, st,
                       (const float *)w, K, C, nbk, nbc, (uint8_t *)q, scale, e8m0);
  return hipGetLastError();
}

}  // namespace moe
