// C ABI of the 8-bit operators: argument checks, workspace layout, and the ordered launches
// on the caller's stream. Nothing here allocates, frees, synchronises or reads device memory.
#include "api_common.h"

using namespace moe;

namespace {

inline bool dtype_ok(moe_dtype dt) { return dt == MOE_BF16 || dt == MOE_FP32; }
inline bool scale_ok(moe_scale_type s) { return s == MOE_SCALE_FP32 || s == MOE_SCALE_E8M0; }
// row lengths of the norm and of rows in 8 bits: whole chunks of eight values
inline bool row_ok(int32_t H) { return H > 0 && H % 8 == 0 && H <= (1 << 20); }
// sides of an 8-bit product: whole 16-byte chunks
inline bool side_ok(int32_t L, int32_t most) { return L > 0 && L % 16 == 0 && L <= most; }
// Addresses that the kernels read and write 16 (q: 8) bytes at a time, and fp32 scales. (Null
// passes: whether a tensor may be missing is checked where it is taken.)
template <typename... P>
inline bool at16(const P *...p) {
  return ((((uintptr_t)p | ...) & 15) == 0);
}
inline bool scale_at(const void *p, moe_scale_type t) {
  return t == MOE_SCALE_E8M0 || ((uintptr_t)p & 3) == 0;
}
inline int32_t blocks(int32_t L) { return (L + MOE_QBLOCK - 1) / MOE_QBLOCK; }
inline moe_status status_of(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

Fp8Args fp8_args(const moe_metadata *m, int32_t K, int32_t C) {
  Fp8Args g = {};
  g.foff = m->expert_frequency_offset;
  g.E = m->E;
  g.cap = m->capacity;
  g.C = C;
  g.K = K;
  g.nbk = blocks(K);
  g.nbc = blocks(C);
  return g;
}

struct Fp8Ws {
  size_t aq, as, y, ys, a32, total;
};
Fp8Ws fp8_layout(const moe_metadata *m, int32_t H, int32_t I) {
  const size_t cap = (size_t)m->capacity;
  Fp8Ws w;
  w.aq = 0;
  w.as = w.aq + align_up(cap * (size_t)I);
  w.y = w.as + align_up(cap * (size_t)blocks(I));
  // the kernel for few rows: a in fp32 first; y in fp32, else in fp16 with scales
  const bool up = fp8_skinny(fp8_args(m, H, 2 * I)), down = fp8_skinny(fp8_args(m, I, H));
  w.ys = w.y + align_up(cap * (size_t)H * (down ? sizeof(float) : 2));
  w.a32 = w.ys + (down ? 0 : align_up(cap * (size_t)((H + kYCols - 1) / kYCols)));
  w.total = w.a32 + (up ? align_up(cap * (size_t)I * sizeof(float)) : 0);
  return w;
}

}  // namespace

extern "C" {

moe_status moe_quantize_rows(const void *x, int32_t N, int32_t H, moe_dtype dt, void *q,
                             void *scale, moe_scale_type scale_type, void *stream) {
  if (N < 0) return MOE_EINVAL;
  if (!dtype_ok(dt) || !scale_ok(scale_type) || !row_ok(H)) return MOE_EUNSUPPORTED;
  if (N > 0 && (!x || !q || !scale)) return MOE_EINVAL;
  if (!at16(x) || (uintptr_t)q % 8 || !scale_at(scale, scale_type)) return MOE_EINVAL;
  // 16 lanes per block of 128, fewer than 2^32 in a launch
  if ((int64_t)N * blocks(H) >= (1 << 28) - 16) return MOE_EUNSUPPORTED;
  if (N == 0) return MOE_OK;
  hipStream_t st = (hipStream_t)stream;
  Bracket b(MOE_KERNEL_QUANT_ROWS, st);
  return status_of(launch_quantize_rows(x, N, H, dt == MOE_BF16, q, scale,
                                        scale_type == MOE_SCALE_E8M0, st));
}

moe_status moe_quantize_weights(const void *w, int32_t E, int32_t K, int32_t C, moe_dtype dt,
                                void *q, void *scale, moe_scale_type scale_type,
                                void *stream) {
  if (E < 1 || E > MOE_MAX_EXPERTS) return MOE_EINVAL;
  if (!dtype_ok(dt) || !scale_ok(scale_type)) return MOE_EUNSUPPORTED;
  if (!side_ok(K, 1 << 20) || !side_ok(C, 1 << 21)) return MOE_EUNSUPPORTED;
  if (!w || !q || !scale || !at16(w, q) || !scale_at(scale, scale_type)) return MOE_EINVAL;
  // a workgroup of 256 lanes per block, fewer than 2^32 lanes in a launch
  if ((int64_t)E * blocks(K) * blocks(C) >= 1 << 24) return MOE_EUNSUPPORTED;
  hipStream_t st = (hipStream_t)stream;
  Bracket b(MOE_KERNEL_QUANT_WEIGHTS, st);
  return status_of(launch_quantize_weights(w, E, K, C, dt == MOE_BF16, q, scale,
                                           scale_type == MOE_SCALE_E8M0, st));
}

moe_status moe_rmsnorm_forward(const void *x, const void *residual, const void *weight,
                               float eps, int32_t N, int32_t H, moe_dtype dt,
                               void *residual_out, void *y, void *q, void *scale,
                               moe_scale_type scale_type, float *rstd, void *stream) {
  if (N < 0 || !(eps >= 0.0f)) return MOE_EINVAL;
  if (!dtype_ok(dt) || !row_ok(H)) return MOE_EUNSUPPORTED;
  if (q && !scale_ok(scale_type)) return MOE_EUNSUPPORTED;
  if (N > 0) {
    if (!x || !weight || (!y && !q) || (!q != !scale) || (!residual != !residual_out))
      return MOE_EINVAL;
  }
  if (!at16(x, residual, weight, residual_out, y) || (uintptr_t)q % 8 || (uintptr_t)rstd % 4 ||
      !scale_at(scale, scale_type))
    return MOE_EINVAL;
  if (N == 0) return MOE_OK;
  hipStream_t st = (hipStream_t)stream;
  Bracket b(MOE_KERNEL_RMSNORM, st);
  return status_of(launch_rmsnorm(x, residual, weight, eps, N, H, dt == MOE_BF16, residual_out, y,
                                  q, scale, scale_type == MOE_SCALE_E8M0, rstd, st));
}

size_t moe_rmsnorm_backward_workspace(int32_t N, int32_t H) {
  if (N <= 0 || H <= 0) return 0;
  return (size_t)rmsnorm_shares(N, H) * (size_t)H * sizeof(float);
}

moe_status moe_rmsnorm_backward(const void *dy, const void *r, const void *weight,
                                const float *rstd, const void *dresidual, int32_t N, int32_t H,
                                moe_dtype dt, void *dx, void *dweight, void *workspace,
                                size_t workspace_bytes, void *stream) {
  if (N < 0) return MOE_EINVAL;
  if (!dtype_ok(dt) || !row_ok(H)) return MOE_EUNSUPPORTED;
  if (!dweight || (N > 0 && (!dy || !r || !weight || !rstd || !dx))) return MOE_EINVAL;
  if (!at16(dy, r, weight, dresidual, dx, dweight, workspace) || (uintptr_t)rstd % 4)
    return MOE_EINVAL;
  const size_t need = moe_rmsnorm_backward_workspace(N, H);
  if (workspace_bytes < need || (need > 0 && !workspace)) return MOE_ENOSPC;
  hipStream_t st = (hipStream_t)stream;
  if (N > 0) {
    Bracket b(MOE_KERNEL_RMSNORM_BWD, st);
    if (launch_rmsnorm_bwd(dy, r, weight, rstd, dresidual, N, H, dt == MOE_BF16, dx,
                           (float *)workspace, st) != hipSuccess)
      return MOE_EHIP;
  }
  Bracket b(MOE_KERNEL_RMSNORM_DW, st);
  return status_of(launch_rmsnorm_dw((const float *)workspace, N, H, dt == MOE_BF16, dweight, st));
}

moe_status moe_grouped_gemm_fp8(const moe_metadata *meta, const void *a, const void *a_scale,
                                moe_scale_type a_scale_type, const void *w,
                                const void *w_scale, moe_scale_type w_scale_type, int32_t K,
                                int32_t C, int32_t gather, void *out, void *stream) {
  if (!meta_ok(meta)) return MOE_EINVAL;
  if (!scale_ok(a_scale_type) || !scale_ok(w_scale_type)) return MOE_EUNSUPPORTED;
  if (!side_ok(K, 1 << 20) || !side_ok(C, 1 << 21)) return MOE_EUNSUPPORTED;
  const bool any = meta->N > 0 && meta->capacity > 0;
  if (any && (!a || !a_scale || !w || !w_scale || !out)) return MOE_EINVAL;
  if (!at16(a, w, out) || !scale_at(a_scale, a_scale_type) || !scale_at(w_scale, w_scale_type))
    return MOE_EINVAL;
  if (!any) return MOE_OK;
  Fp8Args g = fp8_args(meta, K, C);
  g.a = (const uint8_t *)a;
  g.a_rows = gather ? meta->x_gather_idx : nullptr;
  g.a_span = gather ? meta->N : meta->capacity;
  g.a_scale = a_scale;
  g.a_e8m0 = a_scale_type == MOE_SCALE_E8M0;
  g.w = (const uint8_t *)w;
  g.w_scale = w_scale;
  g.w_e8m0 = w_scale_type == MOE_SCALE_E8M0;
  g.out = (uint16_t *)out;
  if (fp8_grid(g) < 0) return MOE_EUNSUPPORTED;
  hipStream_t st = (hipStream_t)stream;
  Bracket b(MOE_KERNEL_GROUPED_FP8, st);
  return status_of(launch_gemm_fp8(false, g, st));
}

size_t moe_expert_forward_fp8_workspace(const moe_metadata *meta, int32_t H, int32_t I) {
  if (!meta || H <= 0 || I <= 0 || meta->capacity < 0) return 0;
  return fp8_layout(meta, H, I).total;
}

moe_status moe_expert_forward_fp8(const moe_metadata *meta, const void *x, const void *x_scale,
                                  moe_scale_type x_scale_type, const void *w_up,
                                  const void *w_up_scale, const void *w_down,
                                  const void *w_down_scale, moe_scale_type w_scale_type,
                                  int32_t H, int32_t I, moe_gateup_layout layout,
                                  void *h_save, void *out, void *workspace,
                                  size_t workspace_bytes, void *stream) {
  if (!meta_ok(meta)) return MOE_EINVAL;
  if (!scale_ok(x_scale_type) || !scale_ok(w_scale_type)) return MOE_EUNSUPPORTED;
  if (layout != MOE_GATEUP_INTERLEAVED && layout != MOE_GATEUP_CONCAT) return MOE_EUNSUPPORTED;
  if (!side_ok(H, 1 << 20) || !side_ok(I, 1 << 20)) return MOE_EUNSUPPORTED;
  if (meta->N > 0 &&
      (!x || !x_scale || !w_up || !w_up_scale || !w_down || !w_down_scale || !out))
    return MOE_EINVAL;
  if (!at16(x, w_up, w_down, h_save, out, workspace) || !scale_at(x_scale, x_scale_type) ||
      !scale_at(w_up_scale, w_scale_type) || !scale_at(w_down_scale, w_scale_type))
    return MOE_EINVAL;
  const Fp8Ws L = fp8_layout(meta, H, I);
  if (workspace_bytes < L.total || (L.total > 0 && !workspace)) return MOE_ENOSPC;
  if (meta->N == 0) return MOE_OK;
  hipStream_t st = (hipStream_t)stream;
  uint8_t *ws = (uint8_t *)workspace;

  Fp8Args up = fp8_args(meta, H, 2 * I);
  up.a = (const uint8_t *)x;
  up.a_rows = meta->x_gather_idx;
  up.a_span = meta->N;
  up.a_scale = x_scale;
  up.a_e8m0 = x_scale_type == MOE_SCALE_E8M0;
  up.w = (const uint8_t *)w_up;
  up.w_scale = w_up_scale;
  up.w_e8m0 = w_scale_type == MOE_SCALE_E8M0;
  up.out = (uint16_t *)h_save;
  up.aq = ws + L.aq;
  up.aq_scale = ws + L.as;
  up.f32 = (float *)(ws + L.a32);
  up.concat = layout == MOE_GATEUP_CONCAT;
  Fp8Args dn = fp8_args(meta, I, H);
  dn.a = up.aq;
  dn.a_span = meta->capacity;
  dn.a_scale = up.aq_scale;
  dn.a_e8m0 = 1;
  dn.w = (const uint8_t *)w_down;
  dn.w_scale = w_down_scale;
  dn.w_e8m0 = up.w_e8m0;
  if (fp8_skinny(dn)) {
    dn.f32 = (float *)(ws + L.y);
  } else {
    dn.out = (uint16_t *)(ws + L.y);
    dn.ys = ws + L.ys;
  }
  if (fp8_grid(up) < 0 || fp8_grid(dn) < 0) return MOE_EUNSUPPORTED;
  if (meta->capacity > 0) {
    Bracket b(MOE_KERNEL_UP_SWIGLU_FP8, st);
    if (launch_gemm_fp8(true, up, st) != hipSuccess) return MOE_EHIP;
  }
  if (meta->capacity > 0 && fp8_skinny(up)) {  // rows past the last pair: never read
    Bracket b(MOE_KERNEL_QUANT_ROWS, st);
    if (launch_quantize_rows(up.f32, meta->capacity, I, false, up.aq, up.aq_scale, 1, st) !=
        hipSuccess)
      return MOE_EHIP;
  }
  if (meta->capacity > 0) {
    Bracket b(MOE_KERNEL_DOWN_FP8, st);
    if (launch_gemm_fp8(false, dn, st) != hipSuccess) return MOE_EHIP;
  }
  Bracket b(MOE_KERNEL_COMBINE, st);
  const int32_t *off = meta->num_activated_expert_per_token_offset;
  const int32_t *rev = meta->s_reverse_scatter_idx;
  return status_of(launch_combine_to_bf16(ws + L.y, dn.ys, off, rev, meta->router_scores, meta->N, H,
                                          meta->capacity, out, st));
}

}  // extern "C"
