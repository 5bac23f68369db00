// tiles_dev.h -- rows of experts as the row-tiled products find them: offsets
// [E + 1] (null: every row is expert 0's) as device values that the host cannot
// check, clamped so that no list leads out of a buffer; a block of an expert's
// rows by its number; row tiles and the order in which workgroups take them; and the rows of
// no expert, which are cleared.
#pragma once

#include "device.h"
#include "plan_block.h"

namespace e4b {

__device__ __forceinline__ int32_t clamped_offset(const int32_t *offsets, int i, int E, int32_t rows) {
  if (!offsets) return i < E ? 0 : rows;
  return min(max(offsets[i], 0), rows);
}

// Zeros to bytes from .. to of p (p 16-byte aligned, from and to even), the work of
// `threads` threads: 16 bytes a store but for the ends.
__device__ __forceinline__ void clear_bytes(char *p, int64_t from, int64_t to, int64_t thread, int64_t threads) {
  const int64_t a = min((from + 15) / 16 * 16, to), b = max(to / 16 * 16, a);
  if (thread < (a - from) / 2) reinterpret_cast<uint16_t *>(p + from)[thread] = 0;
  if (thread < (to - b) / 2) reinterpret_cast<uint16_t *>(p + b)[thread] = 0;
  for (int64_t i = a + thread * 16; i < b; i += threads * 16) *reinterpret_cast<u32x4 *>(p + i) = u32x4{0u, 0u, 0u, 0u};
}

// Workgroups that clear the rows of no expert, of `bytes` at most (the host does not
// know how many of the rows those are).
constexpr int64_t kClearBytes = 1 << 16;  // a workgroup's share
inline int64_t clear_groups(int64_t bytes, int64_t most) {
  const int64_t n = (bytes + kClearBytes - 1) / kClearBytes;
  return n < most ? n : most;
}

// inclusive sums over the wave's lanes: shifts by 1, 2, 4, 8 within a row of 16, then
// the rows' last lanes to the rows behind
__device__ __forceinline__ int32_t wave_scan(int32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// Block `block` of the experts' blocks of `height` rows: its expert, first row and the
// end of the expert's rows; false where the experts have fewer blocks. Uniform over a wave.
__device__ __forceinline__ bool block_of(const int32_t *__restrict__ offsets, int E, int32_t rows, int height,
                                         int32_t block, int lane, int &e, int32_t &r0, int32_t &hi) {
  e = 0;
  r0 = block * height;
  hi = rows;
  if (!offsets) return true;
  int32_t skip = block;  // blocks before this one
  // (where most rows are no expert's, most workgroups have no block: they do not look through all experts)
  const int32_t live = clamped_offset(offsets, E, E, rows);
  const int32_t most = (live + (height - 1) * min(E, live)) / height;
  for (int e0 = 0; e0 < E; e0 += 64) {
    const int i = min(e0 + lane, E - 1);
    int32_t a = offsets[i], b = offsets[i + 1];
    a = min(max(a, 0), rows);
    b = min(max(b, 0), rows);
    const int32_t n = e0 + lane < E && b > a ? (b - a + height - 1) / height : 0, incl = wave_scan(n);
    const int32_t total = __builtin_amdgcn_readlane(incl, 63);
    if (skip < total) {
      const int at = __ffsll(static_cast<unsigned long long>(__ballot(incl > skip))) - 1;
      e = e0 + at;
      r0 = __builtin_amdgcn_readlane(a + (skip - incl + n) * height, at);
      hi = __builtin_amdgcn_readlane(b, at);
      return true;
    }
    skip -= total;
    if (block >= most) return false;
  }
  return false;
}

// The tiles of a call: the map's, or without offsets simply the rows in turn
// (no map is made then: its launch took 4.7 us of a 2048 x 2048 -> 4096 product's 61).
__device__ __forceinline__ int tile_count(const LinearArgs &g, int bm) {
  return g.tile_map ? g.tile_offsets[g.E] : int((g.rows + bm - 1) / bm);
}
__device__ __forceinline__ int4 tile_of(const LinearArgs &g, int t, int bm) {
  if (g.tile_map) return g.tile_map[t];
  return int4{0, 0, t * bm, int(min(int64_t(bm), g.rows - int64_t(t) * bm))};
}

// Tile L of n_mt row tiles by n_nt column tiles, in groups of `group` row tiles so that tiles near each
// other share both operands.
__device__ __forceinline__ void tile_at(uint32_t L, int n_mt, int n_nt, int group, int &mt, int &nt) {
  const uint32_t grp = L / uint32_t(group * n_nt), rem = L % uint32_t(group * n_nt), m0 = grp * group;
  const uint32_t gm = min(uint32_t(group), uint32_t(n_mt) - m0);
  mt = int(m0 + rem % gm);
  nt = int(rem / gm);
}

// The row tile, column tile and share of k of this workgroup: the real tiles, one share of k
// after the other, split evenly over the 8 XCDs (block b runs on XCD b % 8) so that an XCD's L2 sees
// both operands again. False for the workgroups without a tile, which come last.
__device__ __forceinline__ bool place_of(int n_mt, int n_nt, int splits, int group, int &mt, int &nt, int &share) {
  const uint32_t W = uint32_t(n_mt) * uint32_t(n_nt), per = (W * splits + 7) / 8, xi = blockIdx.x / 8;
  uint32_t L = (blockIdx.x % 8) * per + xi;
  if (xi >= per || L >= W * splits) return false;
  share = int(L / W);
  L -= share * W;
  tile_at(L, n_mt, n_nt, group, mt, nt);
  return true;
}

}  // namespace e4b
