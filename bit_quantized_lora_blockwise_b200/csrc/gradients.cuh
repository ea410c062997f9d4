// Adapter gradients of many experts in one persistent launch:
//   dA_e = f (M o X_e)^T Gs_e   [K, r],    dB_e = s (XA_e^T dY_e)   [r, N]
// (M, f: the dropout mask and factor, 1 without dropout), each the product over
// the expert's tokens alone. skinny_kernel computes the same sums with one
// cluster per tile, split over the tokens; with more tiles than resident CTAs
// its cost is the CTA itself (tables, TMEM, first copies, shared-memory
// reduction: some 10 us), not the sums. Here two CTAs per SM (one for more than
// 64 ranks) run over the (product, expert, 128-row tile) units with the ring
// running on from one unit to the next and two TMEM accumulators, so that a
// unit's readout overlaps the next one's products. Bound by reading X and dY
// once.
//
// The token rows are the MMA's K: MN-major operands, 64 tokens a stage, from
// the expert's first row on (a row coordinate, aligned to nothing). The last
// block may reach into the next expert's rows: warp 2 sets those rows of both
// operands to zero in shared memory before the MMAs read them, so not even a
// NaN there can enter. An expert without tokens has no units: its gradients
// are set to zero by warp 3 of all CTAs.
//
// Gs is s dY B^T in two 16-bit parts (ptx.cuh), so that dA carries its own
// rounding and none of G's: in one part dA's error was 1.4 times what its
// rounding alone makes, and in fp16 a G below 2^-14 (B starts at zero) lost its
// bits though dA, summed over the tokens, was in range. The parts lie side by
// side in a stage and in TMEM: one MMA of twice the columns, joined at the
// readout. (Backward of 8192 rows over 8 experts of 4096 x 11008 with dropout:
// 807-828 us, 797-818 with G in one part.) A unit has at most BN ranks of dA or
// 2 BN of dB; of more, a row tile's units follow one another, so that the
// second finds its tokens in L2.
//
// Dropout: dX, the launch before this one, evaluates the same mask and leaves
// its keep bits in the workspace (T K / 8 bytes). The units of dB come first:
// they need nothing from dX and fill the SMs that its last round leaves idle;
// every role waits for dX before its first unit of dA. (8192 rows, 8 experts of
// 4096 x 11008: with the generator evaluated here once more this launch ended
// 100 us after dX, with the bits and the units handed out as below 53; without
// dropout 30.)
//
// Experts are uneven and a CTA has only a few units, so the units are handed
// out as CTAs become free, the expert with the most tokens first, from a counter
// in the workspace (with a fixed stride the SMs were active 69 % of the time).
// Warp 0 takes them and passes them on through a small ring. Every unit's sums
// are its own, so who computes it changes nothing.
//
// Roles: warp 0 TMA, warp 1 TMEM + MMA, warp 2 tails, warp 3 zeros, warps 4-7
// readout and stores, warps 8-15 (DROP) take each landed stage of X through the
// mask.
#pragma once

#include "groups.cuh"
#include "ptx.cuh"

namespace qlora {

struct GradientArgs {
  CUtensorMap tm_x, tm_gs, tm_gs2;  // X [T, K], Gs [T, r] and its second part: 64 x 64 boxes
  CUtensorMap tm_dy, tm_xa;  // dY [T, N], XA [T, r]
  void *dA, *dB;             // [E, K, r], [E, r, N], 16-bit
  float a_scale, b_scale;    // f, s
  int K, N, r;
  int f16;
  GroupArgs groups;
  const uint32_t *keep;   // DROP: keep bits of X, [T][K / 32], written by the kernel before this one
  unsigned int *counter;  // units taken beyond each CTA's first; zero when the launch starts
};

// The experts with tokens, by their number (to a quarter of a power of two),
// the most first; then the others. One warp; `start`: kSizeClasses ints. Returns
// how many have tokens. Every CTA gets the same order: within a class and a
// step, by lane.
constexpr int kSizeClasses = 128;
__device__ __forceinline__ int order_by_size(const GroupTable &gt, int groups, int *start, uint16_t *order) {
  const int lane = threadIdx.x & 31;
  auto size_class = [&](int e) {  // 0: the most tokens, kSizeClasses - 1: none
    if (e >= groups) return kSizeClasses;
    const int n = gt.first[e + 1] - gt.first[e];
    if (n == 0) return kSizeClasses - 1;
    const int log = 31 - __clz(n), quarter = log >= 2 ? (n >> (log - 2)) & 3 : (n << (2 - log)) & 3;
    return kSizeClasses - 2 - (4 * log + quarter);  // n < 2^31: at most 123
  };
  // experts of each class, then (place) where it starts
  for (int i = lane; i < kSizeClasses; i += 32) start[i] = 0;
  __syncwarp();
  auto each = [&](bool place) {
    for (int base = 0; base < groups; base += 32) {
      const int cls = size_class(base + lane);
      const uint32_t peers = __match_any_sync(0xFFFFFFFFu, cls);
      const int before = __popc(peers & ((1u << lane) - 1u));
      const int at = cls < kSizeClasses ? start[cls] + before : 0;
      if (place && cls < kSizeClasses) order[at] = static_cast<uint16_t>(base + lane);
      __syncwarp();
      if (before == 0 && cls < kSizeClasses) start[cls] += __popc(peers);
      __syncwarp();
    }
  };
  each(false);
  int carry = 0;
  for (int base = 0; base < kSizeClasses; base += 32) {
    const int n = start[base + lane];
    int sum = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, sum, d);
      if (lane >= d) sum += o;
    }
    start[base + lane] = carry + sum - n;
    carry += __shfl_sync(0xFFFFFFFFu, sum, 31);
  }
  __syncwarp();
  const int some = start[kSizeClasses - 1];
  __syncwarp();
  each(true);
  return some;
}

// Units of a 128-row tile of dA and of dB.
template <int BN>
struct GradientUnits {
  __host__ __device__ static constexpr int of_dA(int r) { return (r + BN - 1) / BN; }
  __host__ __device__ static constexpr int of_dB(int r) { return (r + 2 * BN - 1) / (2 * BN); }
};

template <int BN_, int STAGES_, bool DROP_>
struct GradientCfg {
  static constexpr int BN = BN_, STAGES = STAGES_;
  static constexpr bool DROP = DROP_;
  static constexpr int A_BYTES = 128 * 64 * 2, PART = BN_ * 64 * 2, STAGE = A_BYTES + 2 * PART;
  static constexpr int OFF_BAR = STAGES_ * STAGE;
  static constexpr int UNITS = 4;  // ring of the CTA's units
  // full[S] empty[S] ready[S] tmem_full[2] tmem_empty[2] landed tail drain unit_full[U] unit_empty[U]
  static constexpr int NBARS = 3 * STAGES_ + 7 + 2 * UNITS;
  // misc: tmem base, abort flag, experts with tokens; the unit ring, the group
  // table, the experts by size and the classes' starts
  static constexpr int OFF_MISC = (OFF_BAR + NBARS * 8 + 15) & ~15;
  static constexpr int OFF_UNITS = OFF_MISC + 16;
  static constexpr int OFF_GROUPS = OFF_UNITS + UNITS * 4;
  static constexpr int OFF_ORDER = OFF_GROUPS + kGroupTableBytes;
  static constexpr int OFF_CLASSES = OFF_ORDER + kMaxGroups * 2;
  static constexpr int SMEM_BYTES = OFF_CLASSES + kSizeClasses * 4;
  static constexpr int UNIT_READERS = DROP_ ? 14 : 6;  // MMA, tails, readout (4), mask (8)
  static constexpr int THREADS = DROP_ ? 512 : 256;
  static constexpr uint32_t TMEM_COLS = 4 * BN_;  // two accumulators of two parts
  static constexpr int PER_SM = SMEM_BYTES <= 113 * 1024 ? 2 : 1;
  static_assert(BN_ == 64 || BN_ == 128, "ranks of a unit of dA");
  static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::PER_SM) gradient_kernel(const __grid_constant__ GradientArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  auto ready_bar = [&](int s) { return bar0 + 8u * (2 * C::STAGES + s); };
  auto tmem_full = [&](int b) { return bar0 + 8u * (3 * C::STAGES + b); };
  auto tmem_empty = [&](int b) { return bar0 + 8u * (3 * C::STAGES + 2 + b); };
  const uint32_t landed_bar = bar0 + 8u * (3 * C::STAGES + 4), tail_bar = landed_bar + 8u, drain_bar = tail_bar + 8u;
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);
  volatile int *s_unit = reinterpret_cast<volatile int *>(smem + C::OFF_UNITS);
  uint16_t *s_order = reinterpret_cast<uint16_t *>(smem + C::OFF_ORDER);
  auto unit_full = [&](uint32_t k) { return drain_bar + 8u + 8u * (k % C::UNITS); };
  auto unit_empty = [&](uint32_t k) { return drain_bar + 8u + 8u * (C::UNITS + k % C::UNITS); };
  const GroupTable gt = group_table(smem + C::OFF_GROUPS);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
      mbar_init(ready_bar(s), 8);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tmem_full(b), 1);
      mbar_init(tmem_empty(b), 4);
    }
    mbar_init(landed_bar, 1);
    mbar_init(tail_bar, 1);
    mbar_init(drain_bar, 1);
    for (int k = 0; k < C::UNITS; ++k) {
      mbar_init(unit_full(k), 1);
      mbar_init(unit_empty(k), C::UNIT_READERS);
    }
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  // Late, like the dense backward's last launch: every operand is complete
  // when this launch starts, and nothing it writes is touched by the kernel
  // before it, for which each thread waits only before exiting.
  grid_dep_launch();
  int *s_some = reinterpret_cast<int *>(smem + C::OFF_MISC + 8);
  if (warp == 3) {
    build_group_table(a.groups, 64, gt);
    __syncwarp();
    const int some = order_by_size(gt, a.groups.groups, reinterpret_cast<int *>(smem + C::OFF_CLASSES), s_order);
    if (lane == 0) *s_some = some;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;

  const int na = GradientUnits<C::BN>::of_dA(a.r), nb1 = GradientUnits<C::BN>::of_dB(a.r);
  const int ta = (a.K + 127) / 128 * na, tb = (a.N + 127) / 128 * nb1;
  const int some = *s_some, nb = some * tb, units = nb + some * ta;
  struct Unit {
    bool second;  // dB
    int group, row0, rank0, tok0, ntok, nk;  // nk > 0
    bool wide;    // both halves of the stage's B operand: two parts of BN ranks, or 2 BN ranks
  };
  auto unit_at = [&](int u) {
    Unit t;
    t.second = u < nb;
    const int v = t.second ? u : u - nb, per = t.second ? tb : ta;
    const int at = v / per;
    t.group = s_order[at];
    const int w = v - at * per, n = t.second ? nb1 : na, tile = w / n;
    t.row0 = tile * 128;
    t.rank0 = (w - tile * n) * (t.second ? 2 * C::BN : C::BN);
    t.wide = !t.second || a.r - t.rank0 > C::BN;
    t.tok0 = gt.first[t.group];
    t.ntok = gt.first[t.group + 1] - t.tok0;
    t.nk = (t.ntok + 63) / 64;
    return t;
  };

  // (each thread of a role, unit by unit; the bounded waits start after it)
  bool dx_done = !C::DROP;
  auto wait_dx = [&](const Unit &t) {
    if (!dx_done && !t.second) {
      grid_dep_wait();
      dx_done = true;
    }
  };

  // the CTA's k-th unit (a warp, or the one thread of a role); false: there are no more
  auto take_warp = [&](uint32_t k, Unit &t) -> bool {
    if (!warp_wait_all(unit_full(k), (k / C::UNITS) & 1u, s_abort)) return false;
    const int u = s_unit[k % C::UNITS];
    __syncwarp();
    if (lane == 0) mbar_arrive(unit_empty(k));
    if (u < units) t = unit_at(u);
    return u < units;
  };
  auto take_thread = [&](uint32_t k, Unit &t) -> bool {
    if (!mbar_wait(unit_full(k), (k / C::UNITS) & 1u, s_abort)) return false;
    const int u = s_unit[k % C::UNITS];
    mbar_arrive(unit_empty(k));
    if (u < units) t = unit_at(u);
    return u < units;
  };

  Unit t;
  if (warp == 0) {
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      int u = blockIdx.x;
      for (uint32_t k = 0; ok; ++k) {
        if (!mbar_wait(unit_empty(k), ((k / C::UNITS) & 1u) ^ 1u, s_abort)) break;
        s_unit[k % C::UNITS] = u;
        mbar_arrive(unit_full(k));
        if (u >= units) break;
        t = unit_at(u);
        wait_dx(t);
        const CUtensorMap *ma = t.second ? &a.tm_dy : &a.tm_x, *mb = t.second ? &a.tm_xa : &a.tm_gs;
        const CUtensorMap *mb2 = t.second ? &a.tm_xa : &a.tm_gs2;
        const int rank2 = t.second ? t.rank0 + C::BN : t.rank0;
        for (int j = 0; j < t.nk; ++j, ++it) {
          const int s = it % C::STAGES, tok = t.tok0 + j * 64;
          if (!mbar_wait(empty_bar(s), ((it / C::STAGES) & 1u) ^ 1u, s_abort)) { ok = false; break; }
          const uint32_t dst = sbase + s * C::STAGE;
          mbar_arrive_expect_tx(full_bar(s), t.wide ? C::STAGE : C::STAGE - C::PART);
          tma_load_2d(dst, ma, full_bar(s), t.row0, tok);
          tma_load_2d(dst + 8192, ma, full_bar(s), t.row0 + 64, tok);
#pragma unroll
          for (int c = 0; c < C::BN / 64; ++c)
            tma_load_2d(dst + C::A_BYTES + c * 8192, mb, full_bar(s), t.rank0 + c * 64, tok);
          if (t.wide) {
#pragma unroll
            for (int c = 0; c < C::BN / 64; ++c)
              tma_load_2d(dst + C::A_BYTES + C::PART + c * 8192, mb2, full_bar(s), rank2 + c * 64, tok);
          }
        }
        u = static_cast<int>(gridDim.x + atomicAdd(a.counter, 1u));
      }
      // wait (bounded) for the copies still in flight
      const uint32_t inflight = it < static_cast<uint32_t>(C::STAGES) ? it : C::STAGES;
      for (uint32_t i = 0; i < inflight; ++i) {
        const uint32_t jb = it - 1 - i;
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(full_bar(jb % C::STAGES), (jb / C::STAGES) & 1u)) {
          if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t id_one = idesc_dtype(make_idesc_bf16(128, C::BN, 1, 1), a.f16);
      const uint32_t id_two = idesc_dtype(make_idesc_bf16(128, 2 * C::BN, 1, 1), a.f16);
      uint32_t it = 0, tails = 0;
      bool ok = true;
      for (uint32_t k = 0; ok && take_thread(k, t); ++k) {
        wait_dx(t);
        const int b = k & 1u;
        const uint32_t idesc = t.wide ? id_two : id_one;
        if (!mbar_wait(tmem_empty(b), ((k >> 1) & 1u) ^ 1u, s_abort)) { ok = false; break; }
        tc_fence_after();
        for (int j = 0; j < t.nk; ++j, ++it) {
          const int s = it % C::STAGES;
          if (!mbar_wait(C::DROP ? ready_bar(s) : full_bar(s), (it / C::STAGES) & 1u, s_abort)) { ok = false; break; }
          if (j == t.nk - 1 && (t.ntok & 63)) {  // (only this thread follows the ring's phases)
            mbar_arrive(landed_bar);
            if (!mbar_wait(tail_bar, tails & 1u, s_abort)) { ok = false; break; }
            ++tails;
          }
          tc_fence_after();
          const uint32_t ad = sbase + s * C::STAGE, bd = ad + C::A_BYTES;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_ss(tmem_base + b * 2 * C::BN, smem_desc_sw128(ad + kk * 2048, 8192, 1024),
                      smem_desc_sw128(bd + kk * 2048, 8192, 1024), idesc, (j > 0 || kk > 0) ? 1u : 0u);
          tc_commit(empty_bar(s));
        }
        if (!ok) break;
        tc_commit(tmem_full(b));
      }
      if (it > 0) {
        tc_commit(drain_bar);
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(drain_bar, 0)) {
          if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
        }
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    uint32_t it = 0, tails = 0;
    for (uint32_t k = 0; take_warp(k, t); ++k) {
      wait_dx(t);
      it += t.nk;
      const int rows = t.ntok & 63;
      if (rows == 0) continue;
      // once the last block has landed (and X is masked): its rows past the
      // expert's last token (a row is 128 consecutive bytes of each 64 x 64
      // chunk, whatever the swizzle)
      if (!warp_wait_all(landed_bar, tails & 1u, s_abort)) break;
      ++tails;
      uint8_t *stage = smem + (it - 1) % C::STAGES * C::STAGE;
      const int first = rows * 8, per = 512 - first;  // 16-byte pieces of a chunk
      for (int i = lane; i < per * (2 + C::BN / 64 * (t.wide ? 2 : 1)); i += 32) {
        const int c = i / per, o = first + i - c * per;
        *reinterpret_cast<uint4 *>(stage + c * 8192 + o * 16) = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(tail_bar);
    }
  } else if (warp >= 4 && warp < 8) {
    const int q = warp - 4;
    const bool f16 = a.f16 != 0;
    const float inv = 1.0f / part_scale(f16);  // (a power of two)
    for (uint32_t k = 0; take_warp(k, t); ++k) {
      const int b = k & 1u;
      const float scale = t.second ? a.b_scale : a.a_scale;
      wait_dx(t);
      if (!warp_wait_all(tmem_full(b), (k >> 1) & 1u, s_abort)) break;
      tc_fence_after();
      const int base = t.row0 + q * 32;  // K and N are multiples of 64: 32 rows or none
#pragma unroll 1
      for (int ch = 0; ch < (t.second ? 2 : 1) * C::BN && t.rank0 + ch < a.r && base < (t.second ? a.N : a.K); ch += 32) {
        const int c0 = t.rank0 + ch;
        const uint32_t tcol = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * 2 * C::BN + ch;
        if (!t.second) {  // a row of dA per lane, 16 columns of both parts at a time
          uint16_t *dst = reinterpret_cast<uint16_t *>(a.dA) +
                          (static_cast<int64_t>(t.group) * a.K + base + lane) * a.r + c0;
#pragma unroll 1
          for (int h = 0; h < 32 && c0 + h < a.r; h += 16) {
            uint32_t w[16], w2[16];
            tmem_ld_32x32b_x16(tcol + h, w);
            tmem_ld_32x32b_x16(tcol + C::BN + h, w2);
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = join_parts(w[j], w2[j], inv) * scale;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (c0 + h + 8 * i < a.r)
                *reinterpret_cast<uint4 *>(dst + h + 8 * i) =
                    make_uint4(pack_16x2(v[8 * i], v[8 * i + 1], f16), pack_16x2(v[8 * i + 2], v[8 * i + 3], f16),
                               pack_16x2(v[8 * i + 4], v[8 * i + 5], f16), pack_16x2(v[8 * i + 6], v[8 * i + 7], f16));
          }
        } else {  // dB is stored along N
          uint32_t w[32];
          tmem_ld_32x32b_x32(tcol, w);
          float v[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(w[j]) * scale;
          uint4 out[4];
          rows_to_columns(v, lane, f16, out);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int col = c0 + 8 * i + (lane & 7);
            if (col < a.r)
              *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(a.dB) +
                                         (static_cast<int64_t>(t.group) * a.r + col) * a.N + base + (lane >> 3) * 8) =
                  out[i];
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(tmem_empty(b));
    }
  } else if (warp == 3) {
    // the gradients of the experts without tokens, consecutive bytes each
    auto zero = [&](void *grad, int e, int64_t elements) {
      uint8_t *dst = static_cast<uint8_t *>(grad) + e * elements * 2;
      for (int64_t i = (blockIdx.x * 32 + lane) * 16; i < elements * 2; i += gridDim.x * 512)
        *reinterpret_cast<uint4 *>(dst + i) = make_uint4(0u, 0u, 0u, 0u);
    };
    for (int at = some; at < a.groups.groups; ++at) {
      zero(a.dA, s_order[at], static_cast<int64_t>(a.K) * a.r);
      zero(a.dB, s_order[at], static_cast<int64_t>(a.N) * a.r);
    }
  } else if (C::DROP && warp >= 8) {
    // M o X. 16-byte piece c of row r of a 64-wide chunk lies at c ^ (r & 7)
    // in the row's 128 bytes. A thread takes 32 columns of a token row, one
    // word of keep bits and four pieces of one chunk; 8 lanes' rows differ, so
    // the pieces they touch at a time lie in different banks. Bit 8 i + 7 - k
    // of the word shifted left by k is the sign of byte i, which prmt spreads
    // over a 16-bit element. (Rows past the expert's last token are not
    // masked: warp 2 zeroes them.)
    const int r = (warp - 8) * 8 + (lane & 7), word = lane >> 3;
    const int64_t ld = a.K / 32;
    uint32_t it = 0;
    bool ok = true;
    for (uint32_t k = 0; ok && take_warp(k, t); ++k) {
      wait_dx(t);
      const uint32_t *bits = a.keep + static_cast<int64_t>(t.tok0 + r) * ld + t.row0 / 32 + word;
      const bool in_row = t.row0 / 32 + word < ld;
      for (int j = 0; j < t.nk; ++j, ++it) {
        const int s = it % C::STAGES;
        const uint32_t w = !t.second && in_row && j * 64 + r < t.ntok ? __ldcg(bits + j * 64 * ld) : 0u;
        if (!warp_wait_all(full_bar(s), (it / C::STAGES) & 1u, s_abort)) { ok = false; break; }
        if (!t.second) {
          uint8_t *row = smem + s * C::STAGE + (word >> 1) * 8192 + r * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 *at = reinterpret_cast<uint4 *>(row + ((((word & 1) * 4 + i) ^ (r & 7)) << 4));
            const uint32_t sel = 0x0101u * (0x88u + 0x11u * i) + 0x4400u;  // byte i of both sources, signs only
            const uint4 v = *at;
            *at = make_uint4(v.x & prmt(w << 7, w << 6, sel), v.y & prmt(w << 5, w << 4, sel),
                             v.z & prmt(w << 3, w << 2, sel), v.w & prmt(w << 1, w, sel));
          }
          fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(ready_bar(s));
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  grid_dep_wait();
}

}  // namespace qlora
