// Host-side check of the 8-bit operators' C entries (csrc/api_fp8.hip, csrc/schedule.hip) on
// the CPU, built with AddressSanitizer and UndefinedBehaviorSanitizer against stub launchers.
//
// Every "device" buffer is a host allocation of exactly the size include/moe.h documents
// (workspaces: exactly what the queries return); the stubs read or write every byte of every
// extent that the kernels use, so that a wrong layout, a short query or a wrong extent is an
// access that the sanitizer reports. `plant` makes the combine write one element too many.
#include <hip/hip_runtime.h>

#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "../token_routing_grouped_amd/csrc/api_common.h"

static bool g_plant = false, g_dry = false;
static int g_launches = 0, g_checks = 0;
hipError_t hipEventRecord(hipEvent_t, hipStream_t) { return hipSuccess; }
hipError_t hipGetDevice(int *d) { return *d = 0, hipSuccess; }

static volatile unsigned char g_sink;
static void rd(const void *p, size_t bytes) {
  if (g_dry || !bytes) return;
  if (!p) abort();
  unsigned char s = 0;
  for (size_t i = 0; i < bytes; i++) s ^= ((const unsigned char *)p)[i];
  g_sink = s;
}
static void wr(void *p, size_t bytes) {
  if (g_dry || !bytes) return;
  if (!p) abort();
  memset(p, 0x5a, bytes);
}
static size_t nb(int64_t l) { return (size_t)((l + 127) / 128); }
static size_t sz(int e8m0) { return e8m0 ? 1 : 4; }

namespace moe {

thread_local TimingHook g_hook;

hipError_t launch_quantize_rows(const void *x, int N, int H, bool bf16, void *q, void *scale, int e8m0,
                                hipStream_t) {
  g_launches++;
  rd(x, (size_t)N * H * (bf16 ? 2 : 4));
  wr(q, (size_t)N * H);
  wr(scale, N * nb(H) * sz(e8m0));
  return hipSuccess;
}
hipError_t launch_quantize_weights(const void *w, int E, int K, int C, bool bf16, void *q, void *scale,
                                   int e8m0, hipStream_t) {
  g_launches++;
  rd(w, (size_t)E * K * C * (bf16 ? 2 : 4));
  wr(q, (size_t)E * K * C);
  wr(scale, E * nb(K) * nb(C) * sz(e8m0));
  return hipSuccess;
}
hipError_t launch_rmsnorm(const void *x, const void *residual, const void *weight, float, int N, int H,
                          bool bf16, void *r, void *y, void *q, void *scale, int e8m0, float *rstd,
                          hipStream_t) {
  g_launches++;
  const size_t es = bf16 ? 2 : 4, n = (size_t)N * H * es;
  rd(x, n);
  rd(weight, H * es);
  if (residual) rd(residual, n), wr(r, n);
  if (y) wr(y, n);
  if (q) wr(q, (size_t)N * H), wr(scale, N * nb(H) * sz(e8m0));
  if (rstd) wr(rstd, (size_t)N * 4);
  return hipSuccess;
}
hipError_t launch_rmsnorm_bwd(const void *dy, const void *r, const void *weight, const float *rstd,
                              const void *dres, int N, int H, bool bf16, void *dx, float *part,
                              hipStream_t) {
  g_launches++;
  const size_t es = bf16 ? 2 : 4, n = (size_t)N * H * es;
  rd(dy, n), rd(r, n), rd(weight, H * es), rd(rstd, (size_t)N * 4);
  if (dres) rd(dres, n);
  wr(dx, n);
  wr(part, (size_t)rmsnorm_shares(N, H) * H * 4);
  return hipSuccess;
}
hipError_t launch_rmsnorm_dw(const float *part, int N, int H, bool bf16, void *dw, hipStream_t) {
  g_launches++;
  if (N > 0) rd(part, (size_t)rmsnorm_shares(N, H) * H * 4);
  wr(dw, (size_t)H * (bf16 ? 2 : 4));
  return hipSuccess;
}
hipError_t launch_gemm_fp8(bool swiglu, const Fp8Args &g, hipStream_t) {
  g_launches++;
  if (fp8_grid(g) <= 0) return hipErrorInvalidValue;
  const size_t cap = (size_t)g.cap;
  rd(g.foff, (size_t)(g.E + 1) * 4);
  if (g.a_rows) rd(g.a_rows, cap * 4);
  rd(g.a, (size_t)g.a_span * g.K);
  rd(g.a_scale, g.a_span * nb(g.K) * sz(g.a_e8m0));
  rd(g.w, (size_t)g.E * g.C * g.K);
  rd(g.w_scale, g.E * nb(g.C) * nb(g.K) * sz(g.w_e8m0));
  if (g.nbk != (int)nb(g.K) || g.nbc != (int)nb(g.C)) return hipErrorInvalidValue;
  if (g.out) wr(g.out, cap * g.C * 2);
  if (!swiglu) {
    if (!g.out != (g.f32 != nullptr) || (g.f32 && !fp8_skinny(g))) return hipErrorInvalidValue;
    if (g.f32) wr(g.f32, cap * g.C * 4);
    if (g.ys) wr(g.ys, cap * ((g.C + kYCols - 1) / kYCols));
  } else if (fp8_skinny(g)) {
    wr(g.f32, cap * (g.C / 2) * 4);
  } else {
    wr(g.aq, cap * (g.C / 2));
    wr(g.aq_scale, cap * nb(g.C / 2));
  }
  return hipSuccess;
}
hipError_t launch_combine_to_bf16(const void *y, const uint8_t *ys, const int32_t *tok_off,
                                  const int32_t *s_rev, const float *scores, int N, int H, int cap, void *out,
                                  hipStream_t) {
  g_launches++;
  rd(y, (size_t)cap * H * (ys ? 2 : 4));
  if (ys) rd(ys, (size_t)cap * ((H + kYCols - 1) / kYCols));
  rd(tok_off, (size_t)(N + 1) * 4);
  rd(s_rev, (size_t)cap * 4);
  rd(scores, (size_t)cap * 4);
  wr(out, (size_t)N * H * 2 + (g_plant ? 2 : 0));
  return hipSuccess;
}

}  // namespace moe

#define EXPECT(call, want)                                                                        \
  do {                                                                                            \
    const int got_ = (int)(call);                                                                 \
    g_checks++;                                                                                   \
    if (got_ != (int)(want)) {                                                                    \
      fprintf(stderr, "%s:%d: %s returned %d\n", __FILE__, __LINE__, #call, got_);                \
      exit(3);                                                                                    \
    }                                                                                             \
  } while (0)

struct Buf {
  std::vector<unsigned char> v;
  void *p;
  explicit Buf(size_t bytes) : v(bytes), p(bytes ? v.data() : nullptr) {}
  Buf(const Buf &) = delete;
};
struct Meta {
  Buf freq, foff, xg, ss, sr, toff, rs, st;
  moe_metadata m;
  Meta(int N, int K, int E, int cap)
      : freq((size_t)E * 4), foff((size_t)(E + 1) * 4), xg((size_t)cap * 4), ss((size_t)cap * 4),
        sr((size_t)cap * 4), toff((size_t)(N + 1) * 4), rs((size_t)cap * 4), st(4) {
    m = {N, K, E, cap, (int32_t *)freq.p, (int32_t *)foff.p, (int32_t *)xg.p, (int32_t *)ss.p,
         (int32_t *)sr.p, (int32_t *)toff.p, (float *)rs.p, (uint32_t *)st.p};
  }
};

static void rows_case(int N, int H, moe_dtype dt, moe_scale_type st) {
  const size_t es = dt == MOE_BF16 ? 2 : 4, s = sz(st == MOE_SCALE_E8M0), n = (size_t)N * H;
  Buf x(n * es), z(n * es), w(H * es), r(n * es), y(n * es), q(n), sc(N * nb(H) * s), rstd((size_t)N * 4);
  EXPECT(moe_quantize_rows(x.p, N, H, dt, q.p, sc.p, st, nullptr), MOE_OK);
  EXPECT(moe_rmsnorm_forward(x.p, z.p, w.p, 1e-6f, N, H, dt, r.p, y.p, q.p, sc.p, st, (float *)rstd.p, nullptr),
         MOE_OK);
  EXPECT(moe_rmsnorm_forward(x.p, nullptr, w.p, 0.0f, N, H, dt, nullptr, nullptr, q.p, sc.p, st, nullptr, nullptr),
         MOE_OK);
  const size_t need = moe_rmsnorm_backward_workspace(N, H);
  Buf ws(need), dw(H * es);
  for (void *dres : {z.p, (void *)nullptr})
    EXPECT(moe_rmsnorm_backward(y.p, r.p, w.p, (float *)rstd.p, dres, N, H, dt, x.p, dw.p, ws.p, need, nullptr),
           MOE_OK);
}

static void expert_case(int N, int K, int E, int cap, int H, int I, moe_scale_type xs, moe_scale_type wt) {
  Meta M(N, K, E, cap);
  const size_t sx = sz(xs == MOE_SCALE_E8M0), sw = sz(wt == MOE_SCALE_E8M0);
  Buf x((size_t)N * H), xsc(N * nb(H) * sx), u((size_t)E * 2 * I * H), usc(E * nb(2 * I) * nb(H) * sw);
  Buf d((size_t)E * H * I), dsc(E * nb(H) * nb(I) * sw), out((size_t)N * H * 2), h((size_t)cap * 2 * I * 2);
  for (void *hs : {h.p, (void *)nullptr})
    for (int lay = 0; lay < 2; lay++) {
      const size_t need = moe_expert_forward_fp8_workspace(&M.m, H, I);
      Buf ws(need);
      EXPECT(moe_expert_forward_fp8(&M.m, x.p, xsc.p, xs, u.p, usc.p, d.p, dsc.p, wt, H, I, (moe_gateup_layout)lay,
                                    hs, out.p, ws.p, need, nullptr),
             MOE_OK);
      if (need)
        EXPECT(moe_expert_forward_fp8(&M.m, x.p, xsc.p, xs, u.p, usc.p, d.p, dsc.p, wt, H, I, (moe_gateup_layout)lay,
                                      hs, out.p, ws.p, need - 1, nullptr),
               MOE_ENOSPC);
    }
  EXPECT(moe_grouped_gemm_fp8(&M.m, x.p, xsc.p, xs, u.p, usc.p, wt, H, 2 * I, 1, h.p, nullptr), MOE_OK);
  Buf a((size_t)cap * H), asc(cap * nb(H) * sx);
  EXPECT(moe_grouped_gemm_fp8(&M.m, a.p, asc.p, xs, u.p, usc.p, wt, H, 2 * I, 0, h.p, nullptr), MOE_OK);
}

static void weights_case(int E, int K, int C, moe_dtype dt, moe_scale_type st) {
  const size_t n = (size_t)E * K * C;
  Buf w(n * (dt == MOE_BF16 ? 2 : 4)), q(n), s(E * nb(K) * nb(C) * sz(st == MOE_SCALE_E8M0));
  EXPECT(moe_quantize_weights(w.p, E, K, C, dt, q.p, s.p, st, nullptr), MOE_OK);
}

// sizes at the limits, with the stubs touching nothing
static void limits() {
  g_dry = true;
  void *A = (void *)4096;
  Meta B(1 << 12, 8, 256, 1 << 15);
  const int L = 1 << 20;
  const size_t need = moe_expert_forward_fp8_workspace(&B.m, L, L);
  if (need < (size_t)(1 << 15) * L * 3) exit(5);
  EXPECT(moe_expert_forward_fp8(&B.m, A, A, MOE_SCALE_E8M0, A, A, A, A, MOE_SCALE_FP32, L, L, MOE_GATEUP_CONCAT, A, A,
                                A, need, nullptr),
         MOE_OK);
  Meta T(1 << 12, 8, 1024, 1 << 15);  // more tiles than are counted
  EXPECT(moe_expert_forward_fp8(&T.m, A, A, MOE_SCALE_E8M0, A, A, A, A, MOE_SCALE_FP32, L, L, MOE_GATEUP_CONCAT, A, A,
                                A, need, nullptr),
         MOE_EUNSUPPORTED);
  Meta F(1 << 11, 8, 1024, 1 << 14);  // 16 rows per expert on average: a in fp32 first
  if (moe_expert_forward_fp8_workspace(&F.m, L, L) < (size_t)(1 << 14) * L * 7) exit(5);
  Meta N(0, 64, 1024, 0);
  N.m.N = (1 << 25) - 1;
  N.m.capacity = (1 << 30);
  EXPECT(moe_grouped_gemm_fp8(&N.m, A, A, MOE_SCALE_E8M0, A, A, MOE_SCALE_E8M0, 16, 2 * L, 1, A, nullptr),
         MOE_EINVAL);  // capacity without its arrays
  if (moe_rmsnorm_backward_workspace(0x7fffffff, L) != (size_t)64 * L * 4) exit(5);
  EXPECT(moe_rmsnorm_backward(A, A, A, (float *)A, A, 0x7fffffff, L, MOE_BF16, A, A, A, (size_t)64 * L * 4, nullptr),
         MOE_OK);
  EXPECT(moe_quantize_rows(A, 0x7fffffff, 128, MOE_BF16, A, A, MOE_SCALE_FP32, nullptr), MOE_EUNSUPPORTED);
  EXPECT(moe_quantize_weights(A, 1024, L, 2 * L, MOE_BF16, A, A, MOE_SCALE_FP32, nullptr), MOE_EUNSUPPORTED);
  g_dry = false;
}

int main(int argc, char **argv) {
  g_plant = argc > 1 && !strcmp(argv[1], "plant");
  if (g_plant) {
    expert_case(16, 2, 4, 32, 128, 128, MOE_SCALE_E8M0, MOE_SCALE_E8M0);
    return 0;
  }
  for (moe_dtype dt : {MOE_BF16, MOE_FP32})
    for (moe_scale_type a : {MOE_SCALE_E8M0, MOE_SCALE_FP32}) {
      for (int N : {0, 1, 5, 600})
        for (int H : {8, 128, 136, 20000 / 8 * (N > 5 ? 0 : 8) + 8}) rows_case(N, H, dt, a);
      weights_case(1, 16, 16, dt, a);
      weights_case(3, 144, 272, dt, a);
    }
  for (moe_scale_type a : {MOE_SCALE_E8M0, MOE_SCALE_FP32})
    for (moe_scale_type w : {MOE_SCALE_E8M0, MOE_SCALE_FP32}) {
      expert_case(0, 2, 4, 0, 128, 128, a, w);
      expert_case(16, 2, 4, 0, 128, 128, a, w);
      expert_case(1, 1, 1, 1, 16, 16, a, w);
      expert_case(9, 2, 3, 18, 144, 48, a, w);     // few rows
      expert_case(300, 2, 2, 600, 272, 80, a, w);  // few tiles
      expert_case(2000, 1, 2, 1900, 64, 592, a, w);   // the up projection in large tiles
      expert_case(2000, 1, 2, 1900, 1040, 48, a, w);  // the down projection
      expert_case(3000, 1, 2, 3000, 272, 144, a, w);  // both
      expert_case(4, 64, 1024, 256, 128, 16, a, w);
    }
  limits();
  printf("abi ok: %d checks, %d stub launches\n", g_checks, g_launches);
  return 0;
}
