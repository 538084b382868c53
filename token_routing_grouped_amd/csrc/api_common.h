// What the C ABI's host code shares: argument checks, alignment, and the timing hook.
#pragma once
#include <limits.h>

#include "../../include/moe.h"
#include "kernels.h"

namespace moe {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
inline size_t elem_size(moe_dtype dt) { return dt == MOE_BF16 ? 2 : 4; }

inline bool meta_ok(const moe_metadata *m) {
  if (!m) return false;
  if (m->N < 0 || m->K < 1 || m->K > MOE_MAX_TOPK || m->E < 1 || m->E > MOE_MAX_EXPERTS)
    return false;
  const int64_t NK = (int64_t)m->N * m->K;
  if (NK >= INT32_MAX) return false;
  if (m->capacity < 0) return false;
  if (!m->expert_frequency || !m->expert_frequency_offset ||
      !m->num_activated_expert_per_token_offset || !m->status)
    return false;
  if (m->capacity > 0 &&
      (!m->x_gather_idx || !m->s_scatter_idx || !m->s_reverse_scatter_idx || !m->router_scores))
    return false;
  if ((int64_t)meta_blocks(NK) * (m->E + 1) >= INT32_MAX) return false;
  return true;
}

// H and I in whole 16-byte bf16 chunks; the GEMM tiles at their edges may be partial
inline bool dims_ok(int32_t H, int32_t I) {
  return H > 0 && I > 0 && H % 8 == 0 && I % 8 == 0 && H <= (1 << 20) && I <= (1 << 20);
}

// ---- diagnostics: events around the launches of one kernel. The hook belongs to the
// host thread that armed it (thread-local): launches made by other threads never read
// or advance it, so arming it in one thread cannot race with another thread's calls.
struct TimingHook {
  int kernel = -1;
  hipEvent_t const *events = nullptr;
  int n = 0, i = 0;
};
extern thread_local TimingHook g_hook;

struct Bracket {  // records the start event on construction, the end event on destruction
  hipStream_t st;
  bool on;
  int slot;
  Bracket(moe_kernel_id k, hipStream_t s) : st(s), on(false), slot(0) {
    if (g_hook.events && g_hook.kernel == (int)k && g_hook.i < g_hook.n) {
      on = true;
      slot = g_hook.i++;
      (void)hipEventRecord(g_hook.events[2 * slot], st);
    }
  }
  ~Bracket() {
    if (on) (void)hipEventRecord(g_hook.events[2 * slot + 1], st);
  }
};

}  // namespace moe
