// RMS norm with the residual's addition, and its backward.
//
// Forward: r = x + residual (rounded), rstd = 1/sqrt(mean(r^2) + eps), y = r rstd weight,
// as bf16 or fp32, in e4m3 with a power-of-two scale per 128 values, or both. Bound by
// memory. A row is held in the registers of TPR lanes between its one read and its
// writes: eight values per lane and chunk, so the 16 lanes of a DPP row hold one block of
// 128 and its maximum needs no LDS. Rows too long for that are read a second time. Measured:
// 16384 x 2048 bf16 with a residual, to r, y and 8 bits (303 MB): 61 us, 5.0 TB/s, as a large
// copy; one row of 7168: 5.2 us, the launch and one trip to memory and back.
//
// Backward: with g = dy weight and c = mean(g r) rstd^2, dx = rstd (g - r c) + dresidual;
// dweight = sum over rows of dy r rstd. Bound by memory. A workgroup walks rows a grid
// apart with the columns fixed to its threads, so its share of dweight stays in registers;
// the shares are written once and a second launch adds them in a fixed order (no atomics).
// Measured: 16384 x 2048 bf16 with the residual's gradient (269 MB) 55 us, 4.9 TB/s, and 5 us
// for the shares; 333 x 5000 fp32 9 us and 4 us.
#include "fp8.h"
#include "kernels.h"

namespace moe {
namespace {

// sum over the TPR lanes of a row's group, in a fixed order; every lane gets it
template <int TPR>
__device__ __forceinline__ float group_sum(float v, float *red) {
  v = wave_sum_dpp_f32(v);
  if constexpr (TPR > kWave) {
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < TPR / kWave; i++) v += red[i];
  }
  return v;
}

struct NormArgs {
  const void *x, *residual, *weight;
  float eps;
  int N, H, nb;
  void *r, *y;
  uint8_t *q;
  void *scale;
  int e8m0;
  float *rstd;
};

// TPR lanes per row, C chunks of eight values per lane; LOOP: rows longer than TPR * C * 8
// values, in passes over the row
template <typename T, int TPR, int C, bool LOOP>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rmsnorm_kernel(NormArgs a) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  static_assert(TPR == kWave || RPB == 1, "one wave or one workgroup per row");
  using V = Vec8<T>;
  __shared__ float red[2][TPR / kWave];
  const int t = threadIdx.x % TPR, nch = a.H / 8;
  int ph = 0;  // the halves of `red` take turns: one barrier per row
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < a.N;
       row += (int64_t)gridDim.x * RPB, ph ^= 1) {
  const T *x = (const T *)a.x + row * a.H;
  const T *res = a.residual ? (const T *)a.residual + row * a.H : nullptr;
  T *ro = (T *)a.r + row * a.H;
  T *yo = a.y ? (T *)a.y + row * a.H : nullptr;
  const T *w = (const T *)a.weight;

  float f[C][8];
  float ss = 0.0f;
  // r of chunk c, in fp32; written out where there is a residual
  auto take = [&](int c, float *v) {
    V::get(c < nch ? V::load(x + (int64_t)c * 8) : V::zero(), v);
    if (res) {
      float u[8];
      V::get(c < nch ? V::load(res + (int64_t)c * 8) : V::zero(), u);
#pragma unroll
      for (int j = 0; j < 8; j++) v[j] += u[j];
      const typename V::Raw p = V::pack(v);
      V::get(p, v);
      if (c < nch) V::store(ro + (int64_t)c * 8, p);
    }
  };
  if constexpr (!LOOP) {
#pragma unroll
    for (int i = 0; i < C; i++) take(i * TPR + t, f[i]);
#pragma unroll
    for (int i = 0; i < C; i++)
#pragma unroll
      for (int j = 0; j < 8; j++) ss += f[i][j] * f[i][j];
  } else {
    for (int c = t; c < nch; c += TPR) {
      take(c, f[0]);
#pragma unroll
      for (int j = 0; j < 8; j++) ss += f[0][j] * f[0][j];
    }
  }
  ss = group_sum<TPR>(ss, red[ph]);
  const float rstd = 1.0f / sqrtf(ss / (float)a.H + a.eps);
  if (t == 0 && a.rstd) a.rstd[row] = rstd;
  // (r weight) is exact for bf16, so y is rounded once in fp32
  auto give = [&](int c, const float *v) {
    float u[8], y[8];
    V::get(c < nch ? V::load(w + (int64_t)c * 8) : V::zero(), u);
#pragma unroll
    for (int j = 0; j < 8; j++) y[j] = (v[j] * u[j]) * rstd;
    if (yo && c < nch) V::store(yo + (int64_t)c * 8, V::pack(y));
    if (a.q) {
      u32x2 q;
      const uint32_t e = quantize8(y, &q);
      if (c < nch) *(u32x2 *)(a.q + row * a.H + (int64_t)c * 8) = q;
      if (c < nch && (t & 15) == 0) store_scale(a.scale, a.e8m0, row * a.nb + (c >> 4), e);
    }
  };
  if constexpr (!LOOP) {
#pragma unroll
    for (int i = 0; i < C; i++) give(i * TPR + t, f[i]);
  } else {
    // whole passes, so that every lane of a block takes part in its maximum. A lane reads
    // the r that it wrote itself.
    const T *r = res ? (const T *)ro : x;
    for (int c0 = 0; c0 < nch; c0 += TPR) {
      const int c = c0 + t;
      V::get(c < nch ? V::load(r + (int64_t)c * 8) : V::zero(), f[0]);
      give(c, f[0]);
    }
  }
  }  // rows
}

constexpr int kMostGroups = 1 << 20;  // workgroups of a launch; further rows are walked

template <typename T, int TPR, int C, bool LOOP = false>
hipError_t norm_go(const NormArgs &a, hipStream_t st) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  const int grid = a.N / RPB + (a.N % RPB != 0);
  hipLaunchKernelGGL((rmsnorm_kernel<T, TPR, C, LOOP>), dim3(grid < kMostGroups ? grid : kMostGroups),
                     dim3(TPR < 256 ? 256 : TPR), 0, st, a);
  return hipGetLastError();
}
template <typename T>
hipError_t norm_pick(const NormArgs &a, hipStream_t st) {
  const int nch = a.H / 8;
  if (nch <= 64) return norm_go<T, 64, 1>(a, st);
  if (nch <= 128) return norm_go<T, 64, 2>(a, st);
  if (nch <= 256) return norm_go<T, 64, 4>(a, st);
  if (nch <= 512) return norm_go<T, 256, 2>(a, st);
  if (nch <= 1024) return norm_go<T, 256, 4>(a, st);
  if (nch <= 4096) return norm_go<T, 1024, 4>(a, st);
  return norm_go<T, 1024, 1, true>(a, st);
}

struct NormBwdArgs {
  const void *dy, *r, *weight;
  const float *rstd;
  const void *dres;
  int N, H;
  void *dx;
  float *part;  // [gridDim.x][H]
};

// one workgroup of TPR threads per row at a time
template <typename T, int TPR, int C>
__global__ __launch_bounds__(TPR) void rmsnorm_bwd_kernel(NormBwdArgs a) {
  using V = Vec8<T>;
  __shared__ float red[2][TPR / kWave];
  const int t = threadIdx.x, nch = a.H / 8;
  float w[C][8], dw[C][8];
#pragma unroll
  for (int i = 0; i < C; i++) {
    const int c = i * TPR + t;
    V::get(c < nch ? V::load((const T *)a.weight + (int64_t)c * 8) : V::zero(), w[i]);
#pragma unroll
    for (int j = 0; j < 8; j++) dw[i][j] = 0.0f;
  }
  int ph = 0;  // the two halves of `red` take turns, so one barrier per row is enough
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x, ph ^= 1) {
    const float rstd = a.rstd[row];
    typename V::Raw rr[C], rd[C];
#pragma unroll
    for (int i = 0; i < C; i++) {
      const int c = i * TPR + t;
      const int64_t o = row * a.H + (int64_t)c * 8;
      rr[i] = c < nch ? V::load((const T *)a.r + o) : V::zero();
      rd[i] = c < nch ? V::load((const T *)a.dy + o) : V::zero();
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < C; i++) {
      float r[8], d[8];
      V::get(rr[i], r);
      V::get(rd[i], d);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        s += d[j] * w[i][j] * r[j];
        dw[i][j] += d[j] * (r[j] * rstd);
      }
    }
    s = group_sum<TPR>(s, red[ph]);
    const float k = s / (float)a.H * (rstd * rstd);
#pragma unroll
    for (int i = 0; i < C; i++) {
      const int c = i * TPR + t;
      const int64_t o = row * a.H + (int64_t)c * 8;
      float r[8], d[8], z[8];
      V::get(rr[i], r);
      V::get(rd[i], d);
      V::get(a.dres && c < nch ? V::load((const T *)a.dres + o) : V::zero(), z);
#pragma unroll
      for (int j = 0; j < 8; j++) z[j] += rstd * (d[j] * w[i][j] - r[j] * k);
      if (c < nch) V::store((T *)a.dx + o, V::pack(z));
    }
  }
#pragma unroll
  for (int i = 0; i < C; i++) {
    const int c = i * TPR + t;
    if (c < nch) {
      float *p = a.part + (int64_t)blockIdx.x * a.H + (int64_t)c * 8;
      Vec8<float>::store(p, Vec8<float>::pack(dw[i]));
    }
  }
}

// Rows too long for the registers: dweight's shares first (one workgroup per 8 * 256
// columns and share of the rows; it reads dy before dx may overwrite it), then dx.
template <typename T>
__global__ __launch_bounds__(256) void rmsnorm_bwd_cols_kernel(NormBwdArgs a) {
  using V = Vec8<T>;
  const int c = blockIdx.y * 256 + threadIdx.x;
  if (c >= a.H / 8) return;
  float dw[8];
#pragma unroll
  for (int j = 0; j < 8; j++) dw[j] = 0.0f;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x) {
    const float rstd = a.rstd[row];
    float r[8], d[8];
    V::get(V::load((const T *)a.r + row * a.H + (int64_t)c * 8), r);
    V::get(V::load((const T *)a.dy + row * a.H + (int64_t)c * 8), d);
#pragma unroll
    for (int j = 0; j < 8; j++) dw[j] += d[j] * (r[j] * rstd);
  }
  Vec8<float>::store(a.part + (int64_t)blockIdx.x * a.H + (int64_t)c * 8, Vec8<float>::pack(dw));
}
template <typename T>
__global__ __launch_bounds__(1024) void rmsnorm_bwd_long_kernel(NormBwdArgs a) {
  using V = Vec8<T>;
  __shared__ float red[2][16];
  const int t = threadIdx.x, nch = a.H / 8;
  int ph = 0;
  for (int64_t row = blockIdx.x; row < a.N; row += gridDim.x, ph ^= 1) {
    const int64_t base = row * a.H;
    const float rstd = a.rstd[row];
    float s = 0.0f;
    for (int c = t; c < nch; c += 1024) {
      float r[8], d[8], w[8];
      V::get(V::load((const T *)a.r + base + (int64_t)c * 8), r);
      V::get(V::load((const T *)a.dy + base + (int64_t)c * 8), d);
      V::get(V::load((const T *)a.weight + (int64_t)c * 8), w);
#pragma unroll
      for (int j = 0; j < 8; j++) s += d[j] * w[j] * r[j];
    }
    s = group_sum<1024>(s, red[ph]);
    const float k = s / (float)a.H * (rstd * rstd);
    for (int c = t; c < nch; c += 1024) {
      float r[8], d[8], w[8], z[8];
      V::get(V::load((const T *)a.r + base + (int64_t)c * 8), r);
      V::get(V::load((const T *)a.dy + base + (int64_t)c * 8), d);
      V::get(V::load((const T *)a.weight + (int64_t)c * 8), w);
      V::get(a.dres ? V::load((const T *)a.dres + base + (int64_t)c * 8) : V::zero(), z);
#pragma unroll
      for (int j = 0; j < 8; j++) z[j] += rstd * (d[j] * w[j] - r[j] * k);
      V::store((T *)a.dx + base + (int64_t)c * 8, V::pack(z));
    }
  }
}

// dweight[c] = sum of the shares, in a fixed order: 16 lanes hold 64 columns, each of the
// 64 groups of 16 lanes adds every 64th share, then one wave adds the groups
template <typename T>
__global__ __launch_bounds__(1024) void rmsnorm_dw_kernel(const float *__restrict__ part, int G,
                                                          int H, T *__restrict__ dw) {
  __shared__ __attribute__((aligned(16))) float s[64][64];
  const int l = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + l * 4;
  f32x4 v = {0, 0, 0, 0};
  if (c < H)
    for (int g0 = grp; g0 < G; g0 += 512) {  // eight shares' loads at a time
      f32x4 p[8];
#pragma unroll
      for (int i = 0; i < 8; i++) {
        const int g = g0 + 64 * i;
        p[i] = g < G ? *(const f32x4 *)(part + (int64_t)g * H + c) : f32x4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < 8; i++) v += p[i];
    }
  *(f32x4 *)&s[grp][l * 4] = v;
  __syncthreads();
  if (threadIdx.x < 64) {
    const int cc = blockIdx.x * 64 + threadIdx.x;
    float u = 0.0f;
#pragma unroll 8
    for (int g = 0; g < 64; g++) u += s[g][threadIdx.x];
    if (cc < H) {
      if constexpr (sizeof(T) == 2)
        dw[cc] = f32_to_bf16(u);
      else
        dw[cc] = u;
    }
  }
}

template <typename T, int TPR, int C>
hipError_t bwd_go(const NormBwdArgs &a, int G, hipStream_t st) {
  hipLaunchKernelGGL((rmsnorm_bwd_kernel<T, TPR, C>), dim3(G), dim3(TPR), 0, st, a);
  return hipGetLastError();
}
template <typename T>
hipError_t bwd_pick(const NormBwdArgs &a, int G, hipStream_t st) {
  const int nch = a.H / 8;
  if (nch <= 256) return bwd_go<T, 256, 1>(a, G, st);
  if (nch <= 512) return bwd_go<T, 256, 2>(a, G, st);
  if (nch <= 1024) return bwd_go<T, 256, 4>(a, G, st);
  if (nch <= 2048) return bwd_go<T, 512, 4>(a, G, st);
  hipLaunchKernelGGL(rmsnorm_bwd_cols_kernel<T>, dim3(G, (nch + 255) / 256), dim3(256), 0, st, a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  hipLaunchKernelGGL(rmsnorm_bwd_long_kernel<T>, 
                     dim3(a.N < kMostGroups ? a.N : kMostGroups), dim3(1024), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm(const void *x, const void *residual, const void *weight, float eps, int N,
                          int H, bool bf16, void *r, void *y, void *q, void *scale, int e8m0,
                          float *rstd, hipStream_t st) {
  NormArgs a = {x, residual, weight, eps, N, H, (H + kQB - 1) / kQB, r, y, (uint8_t *)q, scale,
                e8m0, rstd};
  return bf16 ? norm_pick<uint16_t>(a, st) : norm_pick<float>(a, st);
}

hipError_t launch_rmsnorm_bwd(const void *dy, const void *r, const void *weight, const float *rstd,
                              const void *dres, int N, int H, bool bf16, void *dx, float *part,
                              hipStream_t st) {
  NormBwdArgs a = {dy, r, weight, rstd, dres, N, H, dx, part};
  const int G = rmsnorm_shares(N, H);
  return bf16 ? bwd_pick<uint16_t>(a, G, st) : bwd_pick<float>(a, G, st);
}

hipError_t launch_rmsnorm_dw(const float *part, int N, int H, bool bf16, void *dw, hipStream_t st) {
  const int G = rmsnorm_shares(N, H), grid = (H + 63) / 64;
  if (bf16)
    hipLaunchKernelGGL(rmsnorm_dw_kernel<uint16_t>, dim3(grid), dim3(1024), 0, st, part, G, H,
                       (uint16_t *)dw);
  else
    hipLaunchKernelGGL(rmsnorm_dw_kernel<float>, dim3(grid), dim3(1024), 0, st, part, G, H,
                       (float *)dw);
  return hipGetLastError();
}

}  // namespace moe
