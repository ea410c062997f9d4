// Token groups of the expert-grouped calls: the rows of X (or dY) are sorted
// by expert, expert e's being offsets[e] .. offsets[e + 1] - 1, and the
// offsets live on the device (a router wrote them; the host never reads
// them). Every CTA of a grouped kernel builds the same small table in its
// own shared memory and derives its work from it.
#pragma once

#include "ptx.cuh"

namespace qlora {

constexpr unsigned int kErrBadOffsets = 2u;  // device error word, bit 1
constexpr int kMaxGroups = 1024;

struct GroupArgs {
  const int *offsets;  // device int32 [groups + 1], or NULL: one group of all the tokens
  int groups;
  int tokens;          // rows of the token operand
};

// first[e]: first token of group e (first[groups]: one past the last group);
// cum[e]: token tiles of the groups before e (cum[groups]: all of them).
struct GroupTable {
  int *first;
  int *cum;
};
constexpr int kGroupTableBytes = 2 * (kMaxGroups + 1) * 4 + 8;  // a multiple of 16

__device__ __forceinline__ GroupTable group_table(uint8_t *smem) {
  int *p = reinterpret_cast<int *>(smem);
  return GroupTable{p, p + kMaxGroups + 1};
}

// Build the table with one warp (all 32 lanes). Offsets are data: each is
// clamped to [0, tokens] and the sequence is made ascending by a running
// maximum, so whatever they hold, the groups are disjoint ranges of rows and
// no index derived from them leaves the buffers. If that changed any of
// them, bit 1 of the device error word is set.
__device__ __forceinline__ void build_group_table(const GroupArgs &a, int tile, const GroupTable &t) {
  const int lane = threadIdx.x & 31;
  // all the loads first: a scan that waited for each 32 offsets in turn would
  // cost a trip to L2 per 32 experts
#pragma unroll 8
  for (int i = lane; i <= a.groups; i += 32)
    t.first[i] = a.offsets != nullptr ? __ldg(a.offsets + i) : (i == 0 ? 0 : a.tokens);
  __syncwarp();
  int carry = 0;
  bool bad = false;
  for (int base = 0; base <= a.groups; base += 32) {
    const int i = base + lane;
    int v = 0;
    if (i <= a.groups) {
      const int raw = t.first[i];
      v = raw < 0 ? 0 : (raw > a.tokens ? a.tokens : raw);
      bad |= v != raw;
    }
    int m = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, m, d);
      if (lane >= d && o > m) m = o;
    }
    if (carry > m) m = carry;
    if (i <= a.groups) {
      bad |= m != v;
      t.first[i] = m;
    }
    carry = __shfl_sync(0xFFFFFFFFu, m, 31);
  }
  __syncwarp();
  int sum = 0;
  if (lane == 0) t.cum[0] = 0;
  for (int base = 0; base < a.groups; base += 32) {
    const int i = base + lane;
    int c = 0;
    if (i < a.groups) c = (t.first[i + 1] - t.first[i] + tile - 1) / tile;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, c, d);
      if (lane >= d) c += o;
    }
    c += sum;
    if (i < a.groups) t.cum[i + 1] = c;
    sum = __shfl_sync(0xFFFFFFFFu, c, 31);
  }
  if (bad) atomicOr(&g_error_word, kErrBadOffsets);
}

// The group that token tile `tt` (0 <= tt < cum[groups]) belongs to: the last
// e with cum[e] <= tt.
__device__ __forceinline__ int group_of_tile(const GroupTable &t, int groups, int tt) {
  int lo = 0, hi = groups;  // cum[lo] <= tt < cum[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.cum[mid] <= tt) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace qlora
