// Grouped products over e4m3 operands for few rows per expert (decoding, small batches).
//
// Bound by streaming the weights: each byte is used for the few rows of its expert. The
// weights go straight from memory into registers as matrix operands, two blocks of 128 ahead,
// without LDS or barriers on the way; a workgroup's four waves hold 32 output columns each and
// share the rows' operands through the L1 cache. Latency is hidden by the number of
// workgroups, five (32-row tiles: three) on a CU; more blocks ahead in fewer workgroups were
// slower (64 rows, 8 experts, K 4096, 1024 columns: 30 us with eight blocks against 26), as
// were 64-row tiles against the 256 x 256 kernel. Measured: the up projection of eight decoded
// tokens (24 live experts, H 7168, I 2048; 705 MB of weights) 125 us, 5.6 TB/s; the down
// projection (352 MB) 71 us, 5.0 TB/s. A large copy reads and writes 5.1 TB/s on this card.
//
// The matrix cores have time to spare here, so the operands are widened to bf16, exactly, and
// multiplied by bf16 instructions, which sum the products in fp32 without cutting them off
// (the 8-bit instructions keep 13 bits below the largest of eight). Each block's sum is
// multiplied by its row's and its weight's scale in fp32.
//
//   v_mfma_f32_16x16x32_bf16, four to a block: lane l holds row l % 16 of its operand, and of
//   the block's 128 values the 16-byte chunks l / 16 and l / 16 + 4, eight values at a time;
//   both operands alike, so the order along K does not matter.
#include "../../include/moe.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// eight e4m3 values as bf16, exactly
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
  bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

constexpr int kSB = 48;  // blocks of K whose scales LDS holds at a time

// TT: 16-row pieces of a tile; NW: waves, TN 16-column pieces each; U: blocks in flight (of
// both operands: loads are waited for in the order of their issue, so rows fetched later than
// the weights ahead of them would hold those back); OCC: waves per SIMD
template <bool SWI, int TT, int TN, int NW, int U, int OCC>
__global__ __launch_bounds__(64 * NW, OCC) void skinny_kernel(Fp8Args g) {
  constexpr int NT = 64 * NW, BT = 16 * TT, BN = 16 * TN * NW;
  __shared__ float s_sa[kSB][BT];           // row scales
  __shared__ f32x2 s_sw[kSB][BN / 16];      // weight scales of a 16-column piece's even and odd rows
  __shared__ int s_tab[2 * (MOE_MAX_EXPERTS + 1)];
  int *s_pref = s_tab, *s_off = s_tab + MOE_MAX_EXPERTS + 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  for (int i = tid; i <= g.E; i += NT) {
    const int o = g.foff[i];
    s_off[i] = o;
    if (i < g.E) s_pref[i] = (g.foff[i + 1] - o + BT - 1) / BT;
  }
  __syncthreads();
  if (s_off[g.E] > g.cap) return;
  wave0_exclusive_scan(s_pref, g.E);
  __syncthreads();
  // XCD x (= blockIdx % 8) takes one contiguous run of the tiles; an expert's row tiles of one
  // column tile are neighbours, so they share its weights in one L2
  const int ntn = (g.C + BN - 1) / BN;
  const int64_t G = (int64_t)s_pref[g.E] * ntn;
  int64_t L;
  {
    const int x = blockIdx.x % kNumXcd;
    const int64_t i = blockIdx.x / kNumXcd, q = G / kNumXcd;
    const int r = (int)(G % kNumXcd);
    if (i >= q + (x < r ? 1 : 0)) return;
    L = x * q + (x < r ? x : r) + i;
  }
  int lo = 0, hi = g.E - 1;  // largest e with s_pref[e] <= mtile
  {
    const int mtile = (int)(L / ntn);
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_pref[mid] <= mtile) lo = mid; else hi = mid - 1;
    }
  }
  const int mte = s_pref[lo + 1] - s_pref[lo], l = (int)(L - (int64_t)s_pref[lo] * ntn);
  const int e = __builtin_amdgcn_readfirstlane(lo);
  const int nt = __builtin_amdgcn_readfirstlane(l / mte);
  const int row0 = __builtin_amdgcn_readfirstlane(s_off[lo] + (l - l / mte * mte) * BT);
  const int rows = __builtin_amdgcn_readfirstlane(min(BT, s_off[lo + 1] - row0));
  const int I = g.C >> 1, nk = g.nbk;

  auto w_row = [&](int n) {  // memory row of tile column n
    int c = nt * BN + n;
    c = c < g.C ? c : g.C - 1;
    return SWI && g.concat ? (c & 1 ? I : 0) + (c >> 1) : c;
  };
  auto a_row = [&](int r) {  // memory row of tile row r (past the segment: its first)
    const int s = row0 + (r < rows ? r : 0);
    return (int64_t)(g.a_rows ? g.a_rows[s] : s);
  };
  const int fr = lane & 15, fg = lane >> 4;
  const uint8_t *pw[TN], *pa[TT];
#pragma unroll
  for (int n = 0; n < TN; n++)
    pw[n] = g.w + ((int64_t)e * g.C + w_row((wave * TN + n) * 16 + fr)) * g.K;

  // a block's two chunks of a row; past K (in the last block) the row's last chunk again,
  // which the rows' operand then cancels
  auto at = [&](const uint8_t *p, int kb, u32x4 *v) {
    const int k = min(kb, nk - 1) * kQB + fg * 16;
    v[0] = *(const u32x4 *)(p + min(k, g.K - 16));
    v[1] = *(const u32x4 *)(p + min(k + 64, g.K - 16));
  };
  u32x4 w[U][TN][2], a[U][TT][2];
  // the weights first: their addresses need no row map
#pragma unroll
  for (int u = 0; u < U; u++)
#pragma unroll
    for (int n = 0; n < TN; n++) at(pw[n], u, w[u][n]);
#pragma unroll
  for (int t = 0; t < TT; t++) pa[t] = g.a + a_row(t * 16 + fr) * g.K;
#pragma unroll
  for (int u = 0; u < U; u++)
#pragma unroll
    for (int t = 0; t < TT; t++) at(pa[t], u, a[u][t]);

  f32x4 acc[TN][TT];
#pragma unroll
  for (int n = 0; n < TN; n++)
#pragma unroll
    for (int t = 0; t < TT; t++) acc[n][t] = f32x4{0, 0, 0, 0};

  static_assert(kSB % U == 0, "the sets' order holds over the scales' chunks");
  for (int kc = 0; kc < nk; kc += kSB) {
    if (kc > 0) __syncthreads();
    for (int i = tid; i < kSB * BT; i += NT) {
      const int r = i / kSB, k = i % kSB;
      if (kc + k < nk)
        s_sa[k][r] = scale_value(g.a_scale, g.a_e8m0, a_row(r) * nk + kc + k);
    }
    for (int i = tid; i < kSB * (BN / 16) * 2; i += NT) {
      const int f = i / (kSB * 2), odd = (i / kSB) & 1, k = i % kSB;
      if (kc + k < nk)
        s_sw[k][f][odd] = scale_value(g.w_scale, g.w_e8m0,
                                      ((int64_t)e * g.nbc + w_row(f * 16 + odd) / kQB) * nk + kc + k);
    }
    __syncthreads();
    const int end = min(nk, kc + kSB);
    for (int k0 = kc; k0 < end; k0 += U) {
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int kb = k0 + u;
        if (kb >= end) break;  // uniform
        if ((kb + 1) * kQB > g.K) {  // chunks past K
          const int k = kb * kQB + fg * 16;
#pragma unroll
          for (int t = 0; t < TT; t++) {
            if (k >= g.K) a[u][t][0] = u32x4{0, 0, 0, 0};
            if (k + 64 >= g.K) a[u][t][1] = u32x4{0, 0, 0, 0};
          }
        }
        f32x4 d[TN][TT];
#pragma unroll
        for (int q = 0; q < 4; q++) {
          bf16x8 bt[TT];
#pragma unroll
          for (int t = 0; t < TT; t++) {
            const u32x4 v = a[u][t][q >> 1];
            bt[t] = (q & 1) ? widen(v[2], v[3]) : widen(v[0], v[1]);
          }
#pragma unroll
          for (int n = 0; n < TN; n++) {
            const u32x4 v = w[u][n][q >> 1];
            const bf16x8 an = (q & 1) ? widen(v[2], v[3]) : widen(v[0], v[1]);
#pragma unroll
            for (int t = 0; t < TT; t++)
              d[n][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  an, bt[t], q ? d[n][t] : f32x4{0, 0, 0, 0}, 0, 0, 0);
          }
        }
#pragma unroll
        for (int t = 0; t < TT; t++) at(pa[t], kb + U, a[u][t]);
#pragma unroll
        for (int n = 0; n < TN; n++) at(pw[n], kb + U, w[u][n]);
        const int k = kb - kc;
#pragma unroll
        for (int t = 0; t < TT; t++) {
          const float sa = s_sa[k][t * 16 + fr];
#pragma unroll
          for (int n = 0; n < TN; n++) {
            const f32x2 sw = s_sw[k][wave * TN + n];
            const float x0 = sa * sw[0], x1 = sa * sw[1];
            acc[n][t][0] += d[n][t][0] * x0;
            acc[n][t][1] += d[n][t][1] * x1;
            acc[n][t][2] += d[n][t][2] * x0;
            acc[n][t][3] += d[n][t][3] * x1;
          }
        }
      }
    }
  }
  // The sums are pinned here: a matrix instruction moved under a later per-lane condition
  // would take its operands from loads that only the condition's lanes make.
#pragma unroll
  for (int n = 0; n < TN; n++)
#pragma unroll
    for (int t = 0; t < TT; t++) asm volatile("" : "+v"(acc[n][t]));

  // ---- epilogue: acc[n][t] of lane l holds columns 16 n + 4 (l / 16) .. + 3 of the wave's and
  // row 16 t + l % 16. SwiGLU: a in fp32, which a pass of its own puts in 8 bits (a tile of
  // one block of 128 pairs would be twice as wide, too few tiles for the chip to share evenly).
#pragma unroll
  for (int t = 0; t < TT; t++) {
    const int tok = t * 16 + fr;
    if (tok >= rows) continue;
    const int64_t s = row0 + tok;
#pragma unroll
    for (int n = 0; n < TN; n++) {
      const int c = nt * BN + (wave * TN + n) * 16 + fg * 4;
      if (c >= g.C) continue;
      const f32x4 v = acc[n][t];
      if (g.out)
        *(u32x2 *)(g.out + s * g.C + c) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
      if constexpr (SWI)
        *(f32x2 *)(g.f32 + s * I + (c >> 1)) = f32x2{silu_fast(v[0]) * v[1], silu_fast(v[2]) * v[3]};
      else if (g.f32)
        *(f32x4 *)(g.f32 + s * g.C + c) = v;
    }
  }
}

template <bool SWI, int TT, int TN, int NW, int U, int OCC>
hipError_t go(const Fp8Args &g, int64_t grid, hipStream_t st) {
  hipLaunchKernelGGL((skinny_kernel<SWI, TT, TN, NW, U, OCC>), dim3((uint32_t)grid), dim3(64 * NW), 0,
                     st, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp8_skinny(bool swiglu, const Fp8Args &g, int bt, int64_t grid,
                                  hipStream_t st) {
  if (swiglu) return bt == 16 ? go<true, 1, 2, 4, 2, 5>(g, grid, st) : go<true, 2, 2, 4, 2, 3>(g, grid, st);
  return bt == 16 ? go<false, 1, 2, 4, 2, 5>(g, grid, st) : go<false, 2, 2, 4, 2, 3>(g, grid, st);
}

}  // namespace moe
