// Grouped products over e4m3 operands with a scale per block of 128, on gfx950 matrix cores.
//
//   out[s,:] = sum over the blocks b of K of  (a_s,b . w_n,b) sa[s,b] sw[n/128,b]
//
// for the sorted positions s of each expert's segment. Sums are fp32, but that the matrix
// cores cut each of eight products next to each other along K off 2^13 below the largest
// one's power of two (measured, in-bounds, at every position of a block; the 32-wide fp8
// instructions of the same rate as bf16's do the same): about 1.6e-5 of a result of rounded
// normal values, against 1.7e-3 for the outputs' bf16. Taken for twice the rate of bf16
// products, the only exact way. One v_mfma_f32_16x16x128_f8f6f4 covers exactly one block of
// the reduction. The weights are its first operand, so a lane holds four consecutive output
// columns of one token: one token scale per lane, and (gate, up) pairs side by side.
//
// Scales that are powers of two (e8m0) go into the matrix instruction, which multiplies each
// operand row's products by them for nothing; fp32 scales multiply the block's sums (K 7168,
// 4096 columns, 12800 uneven rows: 602 us against 538 for the same product with e8m0 scales).
//
// Tiles are up to 256 tokens x 256 columns, eight waves of 128 x 64 (2 x 4 of them): the most
// sums that the registers hold, so that a block's operands, 64 KB, serve 1024 clocks of each
// SIMD's two waves. One workgroup per CU stays for the whole launch and takes its tiles in
// turn, so that a tile's first blocks are loaded under the epilogue of the one before. An
// expert's rows are shared out evenly over its tiles, and 16-row pieces without rows are not
// multiplied (uneven experts: 538 us against 575 with tiles of 256 rows and a rest). Where a
// few rounds of tiles leave many CUs idle in the last one, the shares are smaller (kStepRows).
//
// LDS holds two stages of 256 + 256 rows of 128 bytes, filled by direct global-to-LDS loads one
// block ahead of the products, in eighths between them. The 16-byte chunk c of row r lies at
// chunk c ^ ((r / 2) % 8), so the 16 rows that a fragment read takes at one chunk cover all 64
// banks once. Chunks past K, whole in both operands, come from a page of zeros; rows past the
// segment repeat its first row, and store its results again where that saves a branch.
//
// Bounds: the largest product (196k rows, K 4096, 4096 columns; 3.46 ms, 2.22 PFLOP/s) by the
// power of the matrix cores and by what a step does beside them: its matrix instructions alone
// take 56 % of the cycles, without any loads 78 %, with all loads answered by the L2 85 %. A
// library's product of that rate on one matrix of 8192^3, one scale in all, reaches 2.92.
// Short reductions (K 512: 48 us for 24k rows, 2048 columns) by the stores' bandwidth and the
// time from a launch to its first products.
#include "../../include/moe.h"
#include "fp8.h"
#include "kernels.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __attribute__((aligned(128))) uint32_t g_zeros[32];  // starts zeroed, never written

// 16 bytes per lane from global memory to LDS: lane l's go to lds + 16 l. Written as asm so
// that the compiler does not make every later LDS read wait for it (it cannot tell the two
// stages apart); nothing is returned in registers, and the wait is wait_loads(), ahead of
// the barrier that hands the stage over.
__device__ __forceinline__ void load_to_lds(const void *p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds), "v"(p)
               : "memory");
}
// the same from a uniform address plus a lane's 32-bit offset
__device__ __forceinline__ void load_to_lds(const void *base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// all but the last N memory operations of this wave (they count down in order of issue)
template <int N>
__device__ __forceinline__ void wait_loads_before() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p);
}

// The choice of a tile's rows, 256 down to 128: fewer where the rounds of tiles that the
// workgroups make are then better filled. A step costs as much for its weights as for
// kStepRows of its rows (measured: with 128 rows 74 % of its time with 256); rows are counted as
// the mean of the most and of the average, and what is not 6 % better is not worth it. 24k
// rows (763 an expert), K 2048, 1024 columns: 63 us with 256, 57.5 with 224 (chosen), 75 with
// 192; K 512, 2048 columns: 48.6, 45.1 (chosen), 51. 33k rows (1024 an expert), K 2048: 85.6,
// 80.8, 78.8 (chosen); K 512: 59.8 (chosen), 63.9, 60.9. 9k rows: 35.1, 32.1, 31.9 (chosen).
constexpr float kStepRows = 236.0f, kWorth = 0.94f;
// row tiles of n rows, at most `most` each (n < 2^31, most of 128 to 256)
__device__ __forceinline__ int tiles_of(int n, int most) {
  return (int)(((uint32_t)n + (uint32_t)most - 1) / (uint32_t)most);
}
constexpr int kKC = 8;  // blocks of K whose scales LDS holds at a time (two such sets)

// Four lanes that share a token (16 apart) hold four consecutive bf16 columns each of pieces
// n and n + 1: a[0..1] and b[0..1]. They exchange them, so that lane r of the four has the
// eight columns 8 r .. 8 r + 7 of the 32 and a store takes 64 bytes of every row (stores as
// the lanes hold them, 8 bytes each, cost 18 % of the largest product's time).
__device__ __forceinline__ u32x4 columns8(u32x2 a, u32x2 b) {
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 2; j++) {
    const auto h = __builtin_amdgcn_permlane32_swap(a[j], b[j], false, false);
    const auto q = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
    v[j] = q[0];
    v[2 + j] = q[1];
  }
  return v;
}
// maximum over the four lanes that share a token
__device__ __forceinline__ uint32_t max4(uint32_t m) {
  const auto h = __builtin_amdgcn_permlane32_swap(m, m, false, false);
  m = h[0] > h[1] ? h[0] : h[1];
  const auto q = __builtin_amdgcn_permlane16_swap(m, m, false, false);
  return q[0] > q[1] ? q[0] : q[1];
}
constexpr uint32_t kInf = 0x7f800000u;
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ u32x2 to_bf16(const f32x4 &v) {
  return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}
__device__ __forceinline__ u32x2 to_f16(const f32x4 &v, float by) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(u32x2, f16x4{(_Float16)(v[0] * by), (_Float16)(v[1] * by),
                                         (_Float16)(v[2] * by), (_Float16)(v[3] * by)});
}

// WT x WN waves. HW: both scales are e8m0. FAR: rows are found by 64-bit addresses per lane,
// chunks past K come from a page of zeros, and every column piece has scales of its own; else
// (K in whole blocks, each operand's bytes counted in 32 bits) by a uniform address that moves
// along K and a fixed offset per lane.
template <bool HW, bool SWI, bool FAR, int BT, int BN, int WT, int WN>
__global__ __launch_bounds__(64 * WT * WN, 2) void gemm_fp8_kernel(Fp8Args g) {
  constexpr int NT = 64 * WT * WN, NW = WT * WN;
  constexpr int TT = BT / WT / 16, TN = BN / WN / 16;  // 16 x 16 pieces of a wave
  constexpr int ROWS = BT + BN, STAGE = ROWS * kQB;
  constexpr int LA = BT / 8 / NW, LB = BN / 8 / NW;  // 1 KB loads per wave and block
  static_assert(BT % (8 * NW) == 0 && BN % (8 * NW) == 0, "a load is of one operand");
  static_assert(!SWI || BN == 256, "a SwiGLU tile holds one block of 128 pairs");
  constexpr int F = BN / 16;  // column pieces of the tile
  // The rows of a tile in pieces of 16, to the waves in turn. The first two and the last two
  // pieces that a wave multiplies in a step are always there (they carry the step's loads and
  // the next one's reads); those between are left out where the tile has no rows for them.
  auto order = [](int t) constexpr { return t < 2 ? t : t < TT - 2 ? t + 2 : t - (TT - 4); };
  constexpr int SIZES = 5;  // of a tile's rows
  constexpr int SA = kKC * BT / NT, SW = (kKC * F * 2 + NT - 1) / NT;  // scales per thread
  static_assert(kKC * BT % NT == 0 && NT % BT == 0, "whole rounds");
  __shared__ __attribute__((aligned(128))) uint8_t smem[2 * STAGE];
  __shared__ uint32_t s_sa[2][kKC][BT];    // token scales (bits: e8m0 byte or fp32)
  __shared__ uint32_t s_sw[2][kKC][F][2];  // weight scales of a piece's even and odd rows
  __shared__ uint32_t s_max[SWI ? WN : 1][SWI ? BT : 1];  // a token's largest |a|, per wave
  __shared__ int s_num[SIZES];
  __shared__ int s_tab[2 * (MOE_MAX_EXPERTS + 1)];
  int *s_pref = s_tab, *s_off = s_tab + MOE_MAX_EXPERTS + 1;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WN, wn = wave % WN;
  const int ntn = (g.C + BN - 1) / BN;
  const int stride = gridDim.x / kNumXcd;
  for (int i = tid; i <= g.E; i += NT) {
    const int o = g.foff[i];
    s_off[i] = o;
  }
  __syncthreads();
  if (s_off[g.E] > g.cap) return;
  // Rows of a tile at most: wave j counts the tiles of at most BT - 32 j rows.
  static_assert(SIZES <= NW, "a wave for each");
  if (wave < SIZES) {
    const int most = BT - 32 * wave;
    int n = 0;
    for (int i = lane; i < g.E; i += 64) n += tiles_of(s_off[i + 1] - s_off[i], most);
    n = wave_inclusive_scan_dpp(n);
    if (lane == 63) s_num[wave] = n;
  }
  __syncthreads();
  int most = BT;
  {
    const float per = (float)ntn / (float)(kNumXcd * stride), total = (float)s_off[g.E];
    float best = 0.0f;
#pragma unroll
    for (int j = 0; j < SIZES; j++) {
      const int rows = BT - 32 * j;
      const float n = (float)s_num[j];  // (no tiles: any choice)
      const float cost = ceilf(n * per - 1e-3f) * (kStepRows + 0.5f * ((float)rows + total / n));
      if (j == 0 || cost < best) {
        best = j == 0 ? cost * kWorth : cost;
        most = rows;
      }
    }
  }
  most = __builtin_amdgcn_readfirstlane(most);
  for (int i = tid; i < g.E; i += NT) s_pref[i] = tiles_of(s_off[i + 1] - s_off[i], most);
  __syncthreads();
  wave0_exclusive_scan(s_pref, g.E);
  __syncthreads();
  // Persistent workgroups: XCD x (= blockIdx % 8) owns one contiguous run of the tiles, which
  // its workgroups take in turn
  const int64_t G = (int64_t)s_pref[g.E] * ntn;
  const int x = blockIdx.x % kNumXcd;
  const int64_t gq = G / kNumXcd;
  const int gr = (int)(G % kNumXcd);
  const int64_t tend = (x + 1) * gq + min(x + 1, gr);
  int64_t L = x * gq + min(x, gr) + blockIdx.x / kNumXcd;
  if (L >= tend) return;
  // two blocks at least: a tile is entered by its first two (FAR: what is past K is zeros)
  const int nk = FAR ? max(g.nbk, 2) : g.nbk, I = g.C >> 1;
  const uint32_t lds0 = lds_address(smem);

  // ---- a tile: its expert, first row, rows and column tile
  struct Tile {
    int e, nt, row0, rows;
  };
  auto find_tile = [&](int64_t l_, int lo) {
    // within an expert, groups of four row tiles, column tiles outer: the tiles that an XCD
    // works on at a time then share their rows as well as their weights. The expert is the
    // last e with s_pref[e] <= mtile, from lo on: a workgroup's tiles ascend.
    const int mtile = (int)(l_ / ntn);
    while (s_pref[lo + 1] <= mtile) lo++;
    const int mte = s_pref[lo + 1] - s_pref[lo];
    const int l = (int)(l_ - (int64_t)s_pref[lo] * ntn);
    constexpr int GM = 4;
    const int gi = l / (GM * ntn), rem = l - gi * GM * ntn, gm = min(GM, mte - gi * GM);
    const int nt = rem / gm, mt = gi * GM + rem - nt * gm;
    // an expert's rows in even shares, of whole pieces
    const int each = ((s_off[lo + 1] - s_off[lo] + mte - 1) / mte + 15) & ~15;
    const int row0 = s_off[lo] + mt * each;
    Tile t;
    t.e = __builtin_amdgcn_readfirstlane(lo);
    t.nt = __builtin_amdgcn_readfirstlane(nt);
    t.row0 = __builtin_amdgcn_readfirstlane(row0);
    t.rows = __builtin_amdgcn_readfirstlane(min(each, s_off[lo + 1] - row0));
    return t;
  };
  // An opaque copy: what is derived from it is computed where it is used and not kept in
  // registers across the loops, where the sums need them.
  auto here = [](uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
  };
  // Rows of a stage that this lane loads: (wave + NW i) * 8 + lane / 8, all of them at the
  // same chunk. Their memory rows (FAR) or offsets; last, the row whose scales this thread
  // fetches.
  const int ck = ((lane & 7) ^ ((lane >> 4) | ((wave & 1) << 2))) * 16;
  uint32_t arow[LA], wrow[LB], srow;
  uint32_t nrow[LA + 1];  // the next tile's token rows
  auto token_rows = [&](const Tile &t) {
    const int tid_ = (int)here(tid);
#pragma unroll
    for (int i = 0; i <= LA; i++) {
      const int r = i < LA ? (wave + NW * i) * 8 + ((tid_ & 63) >> 3) : tid_ % BT;
      const int s = t.row0 + (r < t.rows ? r : 0);
      nrow[i] = (uint32_t)(g.a_rows ? g.a_rows[s] : s);
    }
  };
  // memory row of tile column n: SwiGLU tiles hold (gate, up) pairs
  auto w_row = [&](const Tile &t, int n) {
    int c = t.nt * BN + n;
    c = c < g.C ? c : g.C - 1;
    return SWI && g.concat ? (c & 1 ? I : 0) + (c >> 1) : c;
  };
  const uint8_t *pa, *pw;  // block to be loaded, of both operands
  int kl;                  // its number
  auto load_tile = [&](const Tile &t) {  // the loads' rows, from nrow
    const int lane_ = (int)here(lane), c_ = (int)here(ck);
#pragma unroll
    for (int i = 0; i < LA; i++) arow[i] = FAR ? nrow[i] : nrow[i] * (uint32_t)g.K + c_;
#pragma unroll
    for (int i = 0; i < LB; i++) {
      const uint32_t r = (uint32_t)w_row(t, (wave + NW * i) * 8 + (lane_ >> 3));
      wrow[i] = FAR ? r : r * (uint32_t)g.K + c_;
    }
    pa = g.a;
    pw = g.w + (int64_t)t.e * g.C * g.K;
    kl = 0;
  };
  auto advance = [&] {
    kl++;
    pa += kQB;
    pw += kQB;
  };
  auto load = [&](uint32_t stage, int i) {
    const uint32_t st = stage + wave * 1024 + NW * i * 1024;
    if constexpr (!FAR) {
      if (i < LA) load_to_lds(pa, arow[i], st);
      else load_to_lds(pw, wrow[i - LA], st);
    } else {
      const uint32_t c = here(ck);
      const uint8_t *p = (i < LA ? pa : pw) +
                         ((uint64_t)here(i < LA ? arow[i] : wrow[i - LA]) * (uint32_t)g.K + c);
      load_to_lds(kl * kQB + (int)c < g.K ? p : (const uint8_t *)g_zeros + c, st);
    }
  };
  // ---- scales of kKC blocks from kb: fetched into registers, put into LDS later
  uint32_t ra[SA], rw[SW];
  auto get_scales = [&](const Tile &t, uint32_t row, int kb) {
    const int tid_ = (int)here(tid);
    const int64_t base = (int64_t)here(row) * g.nbk;
#pragma unroll
    for (int i = 0; i < SA; i++) {
      const int64_t at = base + min(kb + tid_ / BT + i * (NT / BT), g.nbk - 1);
      ra[i] = HW ? (uint32_t)((const uint8_t *)g.a_scale)[at]
                 : __float_as_uint(scale_value(g.a_scale, g.a_e8m0, at));
    }
#pragma unroll
    for (int i = 0; i < SW; i++) {
      const int j = min(tid_ + NT * i, kKC * F * 2 - 1);
      const int k = j / (F * 2), f = (j >> 1) % F, odd = j & 1;
      const int64_t at =
          ((int64_t)t.e * g.nbc + w_row(t, f * 16 + odd) / kQB) * g.nbk + min(kb + k, g.nbk - 1);
      rw[i] = HW ? (uint32_t)((const uint8_t *)g.w_scale)[at]
                 : __float_as_uint(scale_value(g.w_scale, g.w_e8m0, at));
    }
  };
  auto put_scales = [&](int set) {
    const int tid_ = (int)here(tid);
#pragma unroll
    for (int i = 0; i < SA; i++) s_sa[set][tid_ / BT + i * (NT / BT)][tid_ % BT] = ra[i];
#pragma unroll
    for (int i = 0; i < SW; i++) {
      const int j = tid_ + NT * i;
      if (j < kKC * F * 2) (&s_sw[set][0][0][0])[j] = rw[i];
    }
  };

  // ---- LDS reads of a step. The operand of 16 rows: lane l takes 32 bytes of row l % 16, the
  // chunks l / 16 and l / 16 + 4 (both operands alike, so any choice gives the same sums; this
  // one reads at 250 B/clk per CU, chunks 2 (l / 16) and the next at 127, measured). Addresses
  // of this wave's first rows (tokens, weights; first and second chunk) in the stage to be
  // read next, and of its scales; pieces are constant offsets away.
  const int fr = lane & 15, fg = lane >> 4;
  const uint32_t fo0 = lds0 + fr * kQB + ((fg ^ (fr >> 1)) << 4);
  uint32_t ta0 = fo0 + wt * 16 * kQB, wa0 = fo0 + (BT + wn * (BN / WN)) * kQB;
  uint32_t ta1 = ta0 ^ 64, wa1 = wa0 ^ 64;
  const uint32_t la = lds_address(s_sa) + (wt * 16 + fr) * 4;
  const uint32_t lw = lds_address(s_sw) + wn * (TN * 8) + (HW ? (fr & 1) * 4 : 0);
  auto pair = [&](uint32_t a0, uint32_t a1, int off) {
    typedef const __attribute__((address_space(3))) i32x4 *P;
    const i32x4 a = *(P)(uintptr_t)(a0 + off), b = *(P)(uintptr_t)(a1 + off);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto word = [&](uint32_t a) {
    return *(const __attribute__((address_space(3))) uint32_t *)(uintptr_t)a;
  };
  i32x8 an[TN], bt[3];  // tokens' pieces: t in bt[t % 3]
  // Scales of the weights' pieces: of a lane's row (HW), or of even and odd rows. All pieces of
  // a wave lie in the same blocks of 128 rows, but for gates and ups one after the other where
  // I is no multiple of 128 (FAR).
  constexpr int NS = FAR ? TN : 1;
  uint32_t sn[NS][2], sx[NS][2], sa[3];  // sx: the next block's
  auto weights_piece = [&](int si, int n) {  // si: the block's place among the scales in LDS
    an[n] = pair(wa0, wa1, n * 16 * kQB);
    if (n < NS) {
      const uint32_t p = lw + si * (F * 8) + n * 8;
      sx[n][0] = word(p);
      if constexpr (!HW) sx[n][1] = word(p + 4);
    }
  };
  auto next_scales = [&] {
#pragma unroll
    for (int n = 0; n < NS; n++) {
      sn[n][0] = sx[n][0];
      sn[n][1] = sx[n][1];
    }
  };
  auto tokens_piece = [&](int si, int t) {
    bt[t % 3] = pair(ta0, ta1, order(t) * WT * 16 * kQB);
    sa[t % 3] = word(la + si * (BT * 4) + order(t) * WT * 64);
  };
  auto tokens_next = [&](int si) {  // the next block's first piece
    bt[TT % 3] = pair(ta0, ta1, 0);
    sa[TT % 3] = word(la + si * (BT * 4));
  };

  // One step of the reduction multiplies the operands of one block. The weights' pieces are in
  // registers when it begins, and the tokens' pieces are read ahead of their products. With
  // two pieces left, their operands in registers, every wave has read all of the stage, and
  // its loads into the other one, made a step ago, are awaited: one barrier hands both over.
  // The last two pieces' products then cover the loads of the block after next into the free
  // stage and the reads of the next block's weights, each piece as soon as its registers are
  // free. A tile's last two steps load the next tile's first blocks, so these are under way
  // during the epilogue.
  Tile tile = find_tile(L, 0);
  token_rows(tile);
  load_tile(tile);
  srow = nrow[LA];
#pragma unroll
  for (int i = 0; i < LA + LB; i++) load(lds0, i);
  get_scales(tile, srow, 0);
  advance();
#pragma unroll
  for (int i = 0; i < LA + LB; i++) load(lds0 + STAGE, i);
  put_scales(0);
  wait_loads();
  __syncthreads();
#pragma unroll
  for (int n = 0; n < TN; n++) weights_piece(0, n);
  next_scales();
  tokens_piece(0, 0);
  auto other_of = [&](uint32_t s) { return s ^ (lds0 ^ (lds0 + STAGE)); };
  // Loads made in a step's last pieces, of tokens; those of weights in the first pieces of the
  // next. (The largest product: 3430 us; none early 3710, two 3545, six 3470, all 3450 and the
  // uneven experts 970 us against 876; both operands in turn 3560; weights first 3385, but the
  // other cases 1 to 2 % slower.)
  constexpr int EARLY = (LA + LB) / 2;
  static_assert(LA + LB - EARLY == 4, "two in each of two pieces");
  uint32_t stage = lds0;  // of the block being multiplied
  int set = 0;            // its scales' set
  // Tokens past the segment repeat its first row, operands and scales, so they may store its
  // results again; where the columns fill whole tiles every store can then be issued.
  const bool even = g.C % BN == 0;
  constexpr int STORES = 4 * (SWI ? 1 : TN / 2);  // of four pieces of rows
  bool stored = false;
  for (;;) {
  const bool more = L + stride < tend;
  const Tile next = find_tile(more ? L + stride : L, tile.e);  // the last tile: itself, unused
  token_rows(next);
  f32x4 acc[TN][TT];
#pragma unroll
  for (int n = 0; n < TN; n++)
#pragma unroll
    for (int t = 0; t < TT; t++) acc[n][t] = f32x4{0, 0, 0, 0};
  // The products of pieces n and t. fp32 scales: a block's sums d are multiplied and added one
  // product later, when the matrix instruction is done.
  f32x4 d;
  float x0 = 0.0f, x1 = 0.0f;
  auto add = [&](int n, int t) {
    if constexpr (!HW) {
      acc[n][t][0] += d[0] * x0;
      acc[n][t][1] += d[1] * x1;
      acc[n][t][2] += d[2] * x0;
      acc[n][t][3] += d[3] * x1;
      asm volatile("" : "+v"(acc[n][t]));
    }
  };
  auto multiply = [&](int n, int t, int pn, int pt) {  // pn, pt: the product before, if >= 0
    const int m = FAR ? n : 0;
    if constexpr (HW) {
      acc[n][t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          an[n], bt[t % 3], acc[n][t], 0, 0, 0, (int)sn[m][0], 0, (int)sa[t % 3]);
      // pinned to this place: the compiler would gather the products behind the barrier, and
      // hold all their operands until then
      asm volatile("" : "+v"(acc[n][t]));
    } else {
      const f32x4 z = {0, 0, 0, 0};
      f32x4 e_ = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          an[n], bt[t % 3], z, 0, 0, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
      asm volatile("" : "+v"(e_));
      if (pn >= 0) add(pn, pt);
      d = e_;
      x0 = __uint_as_float(sa[t % 3]) * __uint_as_float(sn[m][0]);
      x1 = SWI || FAR ? __uint_as_float(sa[t % 3]) * __uint_as_float(sn[m][1]) : x0;
    }
  };
  const int live = (tile.rows + WT * 16 - 1) / (WT * 16);  // pieces with rows
  for (int kb = 0; kb < nk; kb++) {
    const int k = kb % kKC, len = min(kKC, nk - (kb - k));
    const bool last = k == len - 1;  // of the blocks whose scales are in this set
    if (k == len / 2) {
      if (kb - k + kKC < nk) get_scales(tile, srow, kb - k + kKC);
      else get_scales(next, nrow[LA], 0);
    }
    const int si = set * kKC + k;
#pragma unroll
    for (int t = 0; t < TT - 2; t++) {
      if (t + 1 < TT - 2) tokens_piece(si, t + 1);
      if (t + 1 == TT - 3) tokens_piece(si, TT - 2);
      if (t == TT - 3) tokens_piece(si, TT - 1);
      if (t < 2 || order(t) < live) {
#pragma unroll
        for (int n = 0; n < TN; n++) {
          multiply(n, t, n ? n - 1 : t ? TN - 1 : -1, n ? t : t - 1);
          if (t < 2 && n % 2 == 1 && kb > 0) load(other_of(stage), EARLY + t * 2 + n / 2);
        }
      } else if (order(t) == live || t == 2) {
        add(TN - 1, t - 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    if (order(TT - 3) < live) add(TN - 1, TT - 3);
    // after an epilogue whose stores are all issued: not for those, only for the loads ahead
    // of them
    if (stored && kb == 0) wait_loads_before<STORES>();
    else wait_loads();
    if (last) put_scales(set ^ 1);
    __syncthreads();
    const uint32_t other = other_of(stage), d = other - stage;
    ta0 += d;
    ta1 += d;
    wa0 += d;
    wa1 += d;
    if (kb + 2 == nk) load_tile(next);
    else advance();
    const int sj = last ? (set ^ 1) * kKC : si + 1;
    static_assert((TT - 3) % 3 == TT % 3, "the piece after the last takes the free operand");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < TN; n++) {
      multiply(n, TT - 2, n ? n - 1 : -1, TT - 1);
      multiply(n, TT - 1, n, TT - 2);
      weights_piece(sj, n);
      if (n == 0) tokens_next(sj);
#pragma unroll
      for (int i = n * EARLY / TN; i < (n + 1) * EARLY / TN; i++) load(stage, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    add(TN - 1, TT - 1);
    next_scales();
    if (kb + 1 == nk) {  // before the epilogue's stores
#pragma unroll
      for (int i = EARLY; i < LA + LB; i++) load(stage, i);
    }
    stage = other;
    if (last) set ^= 1;
    bt[0] = bt[TT % 3];
    sa[0] = sa[TT % 3];
  }
  srow = nrow[LA];

  const int nt = tile.nt, row0 = tile.row0, rows = tile.rows;
  // ---- epilogues: acc[n][t] of lane l holds columns 16 n + 4 (l / 16) .. + 3 of token
  // 16 t + l % 16 of its wave
  // Rows of piece t in 16 bits, two column pieces at a time: bf16; or, for the combine, fp16
  // with a power of two for the wave's 64 columns of a row, which puts their largest at
  // 2^14 .. 2^15. fp16 keeps three bits more, so that the sum's one rounding to bf16 counts.
  static_assert(SWI || BN / WN == kYCols, "one scale per wave and row");
  auto store_rows = [&](int t) {
    const int tok = (order(t) * WT + wt) * 16 + fr;
    const int64_t s = row0 + (tok < rows ? tok : 0);
    uint16_t *o = g.out + s * g.C;
    float by = 1.0f;
    if (!SWI && g.ys) {
      // the largest of the bits of |y|; where that is no finite value's (rare), of the finite ones
      uint32_t m = 0;
      auto largest = [&](auto bits) {
        m = 0;
#pragma unroll
        for (int n = 0; n < TN; n++) {
          if (nt * BN + wn * (BN / WN) + n * 16 >= g.C) continue;  // whole pieces, uniform
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const uint32_t b = bits(acc[n][t][i]);
            m = b > m ? b : m;
          }
        }
      };
      largest(abs_bits);
      if (ballot64(m >= kInf)) largest(finite_abs_bits);
      m = max4(m);
      const uint32_t ex = y_exponent(m);
      by = __uint_as_float((268u - ex) << 23);
      const int c0 = nt * BN + wn * (BN / WN);
      if (fg == 0 && c0 < g.C) g.ys[s * ((g.C + kYCols - 1) / kYCols) + c0 / kYCols] = (uint8_t)ex;
    }
#pragma unroll
    for (int n = 0; n < TN; n += 2) {
      const u32x4 v = !SWI && g.ys ? columns8(to_f16(acc[n][t], by), to_f16(acc[n + 1][t], by))
                                   : columns8(to_bf16(acc[n][t]), to_bf16(acc[n + 1][t]));
      const int c = nt * BN + wn * (BN / WN) + n * 16 + fg * 8;
      if (even || (tok < rows && c < g.C)) *(u32x4 *)(o + c) = v;
    }
  };
  if constexpr (!SWI) {
#pragma unroll
    for (int t = 0; t < TT; t++)
      if (order(t) < live) store_rows(t);
  } else {
    // a = silu(gate) up; the block of 128 is the whole tile, so a token's maximum is taken
    // over the four lanes that share it and over the WN waves
    float av[TN][TT][2];
#pragma unroll
    for (int t = 0; t < TT; t++) {
      const int tok = (order(t) * WT + wt) * 16 + fr;
      if (g.out && order(t) < live) store_rows(t);
      uint32_t m = 0;
#pragma unroll
      for (int n = 0; n < TN; n++) {
        const bool in = nt * BN + wn * (BN / WN) + n * 16 < g.C;  // whole pieces, uniform
        const f32x4 v = acc[n][t];
#pragma unroll
        for (int p = 0; p < 2; p++) {
          const float a = silu_fast(v[2 * p]) * v[2 * p + 1];  // a few 2^-24, far below h's error
          av[n][t][p] = a;
          const uint32_t b = in ? abs_bits(a) : 0;
          m = b > m ? b : m;
        }
      }
      if (ballot64(m >= kInf)) {  // rare: what is not finite becomes NaN and sets no scale
        m = 0;
#pragma unroll
        for (int n = 0; n < TN; n++) {
          const bool in = nt * BN + wn * (BN / WN) + n * 16 < g.C;
#pragma unroll
          for (int p = 0; p < 2; p++) {
            const uint32_t b = abs_bits(av[n][t][p]);
            if (b >= kInf) av[n][t][p] = __uint_as_float(0x7fc00000u);
            m = in && b < kInf && b > m ? b : m;
          }
        }
      }
      m = max4(m);
      if (fg == 0) s_max[wn][tok] = m;
    }
    __syncthreads();
    static_assert(TN == 4, "four pieces, one for each lane that shares a token");
#pragma unroll
    for (int t = 0; t < TT; t++) {
      const int tok = (order(t) * WT + wt) * 16 + fr;
      uint32_t m = s_max[0][tok];
#pragma unroll
      for (int w = 1; w < WN; w++) m = m > s_max[w][tok] ? m : s_max[w][tok];
      const uint32_t ex = scale_exponent(m);
      const float inv = exponent_inverse(ex);
      // The lane's two bytes of each piece; the four lanes of a token then exchange them, so
      // that lane fg has the eight bytes of piece fg.
      uint32_t b[TN];
#pragma unroll
      for (int n = 0; n < TN; n++)
        b[n] = pack_e4m3(av[n][t][0] * inv, av[n][t][1] * inv, 0.0f, 0.0f);
      // a 4 x 4 exchange of 16 bits: rows of 32 lanes, then of 16
      const auto h0 = __builtin_amdgcn_permlane32_swap(b[0], b[2], false, false);
      const auto h1 = __builtin_amdgcn_permlane32_swap(b[1], b[3], false, false);
      const auto q0 = __builtin_amdgcn_permlane16_swap(h0[0], h1[0], false, false);
      const auto q1 = __builtin_amdgcn_permlane16_swap(h0[1], h1[1], false, false);
      const u32x2 q = {q0[0] | (q0[1] << 16), q1[0] | (q1[1] << 16)};
      const int j = nt * kQB + wn * (BN / WN / 2) + fg * 8;
      if (even ? order(t) < live : tok < rows && j < I)
        *(u32x2 *)(g.aq + (int64_t)(row0 + (tok < rows ? tok : 0)) * I + j) = q;
      if (wn == 0 && fg == 0 && tok < rows)
        g.aq_scale[(int64_t)(row0 + tok) * ((I + kQB - 1) / kQB) + nt] = (uint8_t)ex;
    }
  }
  if (!more) break;
  L += stride;
  stored = even && live >= 4;  // STORES of them at least, behind the loads
  tile = next;
  }  // tiles
}

template <bool HW, bool SWI, bool FAR>
hipError_t go(const Fp8Args &g, int64_t grid, hipStream_t st) {
  auto kern = gemm_fp8_kernel<HW, SWI, FAR, 256, 256, 2, 4>;
  int dev = 0, ncu = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&ncu, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
    return hipErrorInvalidValue;
  const int64_t most = (int64_t)(ncu + kNumXcd - 1) / kNumXcd * kNumXcd;
  hipLaunchKernelGGL(kern, dim3((uint32_t)(grid < most ? grid : most)), dim3(512), 0, st, g);
  return hipGetLastError();
}
template <bool HW, bool SWI>
hipError_t go(const Fp8Args &g, int64_t grid, hipStream_t st) {
  const bool near = g.K % kQB == 0 && g.nbk > 1 && !(g.concat && g.C / 2 % kQB) && (int64_t)g.a_span * g.K <= 0xffffffffll &&
                    (int64_t)g.C * g.K <= 0xffffffffll;
  return near ? go<HW, SWI, false>(g, grid, st) : go<HW, SWI, true>(g, grid, st);
}

}  // namespace

hipError_t launch_gemm_fp8(bool swiglu, const Fp8Args &g, hipStream_t st) {
  const int64_t grid = fp8_grid(g);
  if (grid < 0) return hipErrorInvalidValue;
  if (grid == 0) return hipSuccess;
  int bt, bn;
  fp8_tile(g, &bt, &bn);
  if (fp8_skinny(g)) return launch_gemm_fp8_skinny(swiglu, g, bt, grid, st);
  const bool hw = g.a_e8m0 && g.w_e8m0;
  if (swiglu) return hw ? go<true, true>(g, grid, st) : go<false, true>(g, grid, st);
  return hw ? go<true, false>(g, grid, st) : go<false, false>(g, grid, st);
}

}  // namespace moe
