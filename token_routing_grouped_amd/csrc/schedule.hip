// Host-side size arithmetic of the kernels: tile shapes and grid sizes of the grouped
// GEMMs and the router's workspace. Host code only (no kernels), so it can also be
// built for the CPU alone and checked there under sanitizers.
#include "kernels.h"

namespace moe {

// router workspace, in floats: per-chunk softmax sums [E][nblk], then their totals [E]
size_t route_ws_floats(int64_t NK, int E) { return (size_t)(meta_blocks(NK) + 1) * (size_t)E; }

// bf16 tiles: 256x256x32 with eight waves where the fixed dimensions allow it (half
// the bytes per flop of 128x128), else 128x128; 32x128x64 with two waves when the
// capacity averages at most 16 rows per expert (decode), so the matrix work per
// streamed weight byte matches the rows there are and more workgroups stream weights.
// At few tokens the 128x128 tiles also replace the 256x256 ones where those would
// number fewer than the CUs (grouped-M) or where the experts average fewer than 128
// rows (weight gradients).
// Shapes whose output columns (and, grouped-M, reduction; varlen-K, output rows) do
// not fill whole 128-wide tiles take the 128x128x32 tiles with edge handling; H and I
// are multiples of 8 (one 16-byte chunk) there.
bool gemm_ragged(GemmKind kind, const GemmArgs &g) {
  if (kind == kWeightGrad) return g.M % 128 != 0 || g.N % 128 != 0;
  return g.N % 128 != 0 || g.K % 32 != 0;
}

void gemm_tile(GemmKind kind, const GemmArgs &g, int *bm, int *bn, int *bk) {
  if (gemm_ragged(kind, g)) {
    *bm = *bn = 128;
    *bk = 32;
  } else if (kind == kWeightGrad) {
    // few rows per expert: each tile is a short reduction and then a store burst, and the
    // 128x128 tiles (several workgroups per CU) overlap one tile's stores with another's
    // loads
    const bool big = g.M % 256 == 0 && g.N % 256 == 0 &&
                     (int64_t)g.cap >= kWgradFewRows * (int64_t)g.E;
    *bm = big ? 256 : 128;
    *bn = big ? 256 : 128;
    *bk = 32;
  } else {
    const bool skinny = (int64_t)g.cap <= 16LL * g.E && g.N % 128 == 0 && g.K % 64 == 0;
    bool big = g.N % 256 == 0 && g.K % 32 == 0;
    if (big && !skinny) {
      // fewer 256x256 tiles than the chip has CUs (bounded from the capacity): the
      // 128x128 tiles, four times as many, keep more of the chip busy
      const int64_t mt = ((int64_t)g.cap + (int64_t)g.E * 255) / 256;
      if (mt * (g.N / 256) < kGemmFewTiles) big = false;
    }
    *bm = skinny ? 32 : big ? 256 : 128;
    *bn = skinny ? 128 : big ? 256 : 128;
    *bk = skinny ? 64 : big ? 32 : (g.K % 64 == 0 ? 64 : 32);
  }
}

// Launch size: varlen-K launches one workgroup per output tile of every expert (-1
// when that exceeds the grid limit); grouped-M returns an upper bound of its tiles
// (row tiles of every expert segment, bounded from the capacity, times column tiles,
// capped at INT_MAX), and the launch caps its persistent grid at what the chip holds.
// Partial edge tiles count as tiles.
int gemm_grid(GemmKind kind, const GemmArgs &g) {
  int bm, bn, bk;
  gemm_tile(kind, g, &bm, &bn, &bk);
  const int64_t ntn = ((int64_t)g.N + bn - 1) / bn;
  if (kind == kWeightGrad) {
    const int64_t grid = (int64_t)g.E * (((int64_t)g.M + bm - 1) / bm) * ntn;
    return grid > 0x7fffffff ? -1 : (int)grid;
  }
  const int64_t mt = ((int64_t)g.cap + (int64_t)g.E * (bm - 1)) / bm;
  const int64_t tiles = mt * ntn;
  return tiles > 0x7fffffff ? 0x7fffffff : (int)tiles;
}

// fp32 checking mode: one workgroup per 128x128 tile (grouped-M: row tiles of every
// expert segment, bounded from the capacity; varlen-K: every expert's output tiles);
// -1 when that exceeds the grid limit.
int gemm_grid_f32(GemmKind kind, const GemmArgs &g) {
  int64_t grid;
  const int64_t ntn = ((int64_t)g.N + kGemmBN - 1) / kGemmBN;
  if (kind == kWeightGrad) {
    grid = (int64_t)g.E * (((int64_t)g.M + kGemmBM - 1) / kGemmBM) * ntn;
  } else {
    const int64_t mt = ((int64_t)g.cap + (int64_t)g.E * (kGemmBM - 1)) / kGemmBM;
    grid = mt * ntn;
  }
  return grid > 0x7fffffff ? -1 : (int)grid;
}

// Row tiles of every segment, bounded from the capacity, times column tiles.
static int64_t fp8_tiles(const Fp8Args &g, int bt, int bn) {
  int64_t mt = ((int64_t)g.cap + (int64_t)g.E * (bt - 1)) / bt;
  if (mt > g.cap) mt = g.cap;  // no segment of a tile is empty
  return mt * (((int64_t)g.C + bn - 1) / bn);
}

// 8-bit products. The weight-streaming kernel's tiles of 16 or 32 x 128 where there are few
// rows per expert on average (from the capacity), and where those tiles number no more than
// the CUs: there 256 x 256 tiles would leave most of the chip idle. Else 256 x 256. Measured:
// the expert layer at H 7168, I 2048, 32 experts: 8 rows per expert 278 us with 16-row tiles
// against 371 with 256; 16 rows 318 with 32-row tiles against 366; 24 rows 406 against 395.
// At H 2048, I 512: 16 rows 58 against 64, 24 rows 69 against 63. One product by few tiles:
// 12 experts, 270 rows, K 1040, 592 columns 12 us against 26; 4 experts, 200 rows, K and
// columns 2048 23 against 26, but 600 rows (352 tiles by 32, K 2048, 2048 columns) 48
// against 38.
constexpr int kFp8Cus = 256;
bool fp8_skinny(const Fp8Args &g) {
  return (int64_t)g.cap <= 20 * (int64_t)g.E || fp8_tiles(g, 32, 128) <= kFp8Cus;
}
void fp8_tile(const Fp8Args &g, int *bt, int *bn) {
  const bool skinny = fp8_skinny(g);
  *bt = !skinny ? 128 : (int64_t)g.cap <= 8 * (int64_t)g.E ? 16 : 32;
  *bn = skinny ? 128 : 256;
}

// In whole rounds of the XCDs; fewer than 2^32 lanes in a launch.
int64_t fp8_grid(const Fp8Args &g) {
  int bt, bn;
  fp8_tile(g, &bt, &bn);
  const int64_t grid = (fp8_tiles(g, bt, bn) + 7) / 8 * 8;
  return grid >= (1 << 23) ? -1 : grid;
}

}  // namespace moe
