// Rank-r adapter products of the QLoRA layer on tcgen05 (sm_100a):
//   X A (forward, before the fused GEMM), dY B^T, X^T G and dY^T (X A)
//   (backward) — out[rows, r] = scale * sum_k Aop[row, k] Bop[j, k].
// The adapters are trainable and only they receive gradients (intvml.com
// "DL0087 QLoRA", component 4; Figure 1, dashed path).
//
// The reduction dimension is long (K, N or M tokens) and the output thin
// (r columns), so K is split across the CTAs of a thread-block cluster (one
// cluster per 128-row tile, up to 8 CTAs). Each CTA streams its K range
// through a TMA ring into a TMEM accumulator, parks its fp32 partial in its
// own shared memory, and after a cluster barrier every CTA sums one slice of
// rows over all the cluster's partials through distributed shared memory,
// in rank order (deterministic), and writes the bf16 result (optionally a
// second copy with another scale, optionally transposed). No global
// partials, no counters, one launch.
//
// Roles: warp 0 TMA, warp 1 TMEM + MMA issue, warps 4-7 TMEM readout (lane
// quadrant = warp - 4); all 8 warps take part in the cluster reduction.
//
// Expert groups (GROUPED = true; groups.cuh). Products over token rows (X A,
// dY B^T): a tile is 128 rows of one expert, clusters past the last tile
// leave at once (the host sizes the grid for the worst split of the tokens).
// Products over the tokens (X^T G, dY^T XA; A_MN): a tile is (expert, 128
// output rows), reduced over that expert's tokens alone. Its first token
// need not be a multiple of anything (it is a row coordinate), but the last
// 64-token block may reach into the next expert's rows: warp 2 sets those
// rows of both operands to zero in shared memory before the MMAs read them,
// so that not even a NaN there can enter this expert's gradient. An expert
// without tokens gets zeros. dA takes G in two 16-bit parts, which the dY B^T
// launch writes (ptx.cuh; the reasons are in gradients.cuh): the second part's
// columns follow the first's in a stage and in TMEM, and the readout joins
// them. (Backward of 2048 rows, 11008 x 4096 with dropout: 187 us, 184 with G
// in one part.)
//
// Adapter dropout (DROP = true): the product reads M o X in place of X (kept
// elements as they are; the factor is in the output's scale). X never makes
// a pass of its own: warps 4-11, idle until the readout, take each landed
// 16 KB stage of X through the mask in shared memory before the MMAs read
// it, 16 bytes (8 elements, one Philox counter) at a time. (A dropout launch
// ahead of the product wrote and re-read X: 840 us against 777 for the whole
// backward of 8192 rows through 4096 x 11008; with four masking warps, whose
// latency a stage then waits for, that last launch trailed dX by 130 us,
// with eight by 97.)
#pragma once

#include "codec.cuh"
#include "dropout.cuh"
#include "groups.cuh"
#include "ptx.cuh"

namespace qlora {

// One product of the launch.
struct SkinnyProblem {
  CUtensorMap tm_a;  // A operand: K-major box {64, 128} or MN-major 64x64 chunks
  CUtensorMap tm_b;  // B operand: K-major box {64, BN} or MN-major 64x64 chunks
  CUtensorMap tm_b2;  // TWO_PART, parts == 2: the B operand's second part
  void *out;         // bf16 [rows, cols] (ld out_ld) or transposed [cols, rows]
  void *out2;        // optional second output, same layout
  int64_t out_ld, out2_ld;
  float out_scale, out2_scale;
  int transpose;
  int rows;     // extent of the 128-row MMA dimension
  int cols;     // r
  int kblocks;  // 64-deep K blocks in total
  int masked;   // DROP: the A operand is taken through the mask (X; not dY)
  int parts;    // TWO_PART: 16-bit parts of the B operand (2: Gs; else XA, in one)
  int rest;     // GROUPED: out2 (same scale) holds the second part of what out rounds: G, for dA
};

struct SkinnyArgs {
  // Up to two independent products of the same operand layouts in one
  // launch: CTAs [0, prob0_ctas) take prob[0], the next ones prob[1].
  SkinnyProblem prob[2];
  int prob0_ctas;
  int splits;   // CTAs per cluster (1, 2, 4 or 8), each taking a K range
  unsigned int *zero_words;  // optional: words CTA 0 sets to zero (tile counters of the next kernel)
  int nzero;
  int early;  // 1: neither operand is written by the kernel just before this one in the stream, so the
              // first ring stages may be loaded before waiting for that kernel (programmatic launch)
  int late;   // 1: every operand is complete when this launch starts and nothing it writes is touched by
              // the kernel before it, so the whole product runs without waiting for that kernel; each
              // thread waits for it only before exiting, so this grid still completes after it
  int f16;   // operands and outputs are fp16 (else bf16)
  GroupArgs groups;  // GROUPED only; prob[i].rows is then per expert for products over the tokens
  DropoutArgs drop;  // DROP only
  int64_t drop_ld;   // row length of the masked operand X
};

template <int BN_, bool A_MN_, bool B_MN_, int STAGES_, bool GROUPED_ = false, bool DROP_ = false>
struct SkinnyCfg {
  static constexpr bool GROUPED = GROUPED_, DROP = DROP_;
  static_assert(!DROP_ || GROUPED_, "dropout comes with groups");
  static constexpr int BN = BN_, STAGES = STAGES_;
  static constexpr bool A_MN = A_MN_, B_MN = B_MN_;
  static_assert(BN_ % 64 == 0 && BN_ <= 256, "rank tile");
  static constexpr int A_BYTES = 128 * 64 * 2;
  // dA's G comes in two 16-bit parts (ptx.cuh), side by side in a stage and in TMEM
  static constexpr bool TWO_PART = GROUPED_ && A_MN_;
  static constexpr int PART_BYTES = BN_ * 64 * 2;
  static constexpr int B_BYTES = PART_BYTES * (TWO_PART ? 2 : 1);
  static constexpr int OFF_A = 0;
  static constexpr int OFF_B = STAGES_ * A_BYTES;
  static constexpr int OFF_BAR = OFF_B + STAGES_ * B_BYTES;
  // full[S], empty[S], tmem_full, drain, (GROUPED: landed, tail), (DROP: ready[S])
  static constexpr int NBARS = 2 * STAGES_ + (GROUPED_ ? 4 : 2) + (DROP_ ? STAGES_ : 0);
  static constexpr int OFF_MISC = (OFF_BAR + NBARS * 8 + 15) & ~15;
  static constexpr int OFF_GROUPS = OFF_MISC + 16;
  static constexpr int SMEM_BYTES = OFF_GROUPS + (GROUPED_ ? kGroupTableBytes : 0);
  static constexpr int THREADS = DROP_ ? 384 : 256;  // DROP: warps 8-11 mask beside warps 4-7
  static constexpr uint32_t TMEM_COLS = (BN_ <= 64 ? 64 : (BN_ <= 128 ? 128 : 256)) * (TWO_PART ? 2 : 1);
  static constexpr int PART_LD = BN_ + 4;  // fp32 per partial row (16-byte pad against bank conflicts)
  static_assert(128 * PART_LD * 4 <= OFF_BAR, "the partial reuses the ring");
  static_assert(SMEM_BYTES <= (BN_ <= 128 ? 113 * 1024 : 232448), "shared memory per CTA: two on an SM up to rank 128");
  static constexpr uint32_t TX = A_BYTES + PART_BYTES;  // (and another PART_BYTES for a second part)
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) skinny_kernel(const __grid_constant__ SkinnyArgs args) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw;  // 1024-byte aligned: the 128-byte swizzle atoms need it
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (C::STAGES + s); };
  const uint32_t tmem_full = bar0 + 8u * (2 * C::STAGES);
  const uint32_t drain_bar = bar0 + 8u * (2 * C::STAGES + 1);
  uint32_t *s_tmem = reinterpret_cast<uint32_t *>(smem + C::OFF_MISC);
  volatile int *s_abort = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 4);

  const int splits = args.splits;
  const int pi = static_cast<int>(blockIdx.x) >= args.prob0_ctas ? 1 : 0;
  const SkinnyProblem &P = args.prob[pi];
  const int local_block = static_cast<int>(blockIdx.x) - (pi ? args.prob0_ctas : 0);
  const uint32_t rank = splits > 1 ? cluster_ctarank() : 0u;
  const int tile = local_block / splits;
  const uint32_t landed_bar = bar0 + 8u * (2 * C::STAGES + 2), tail_bar = landed_bar + 8u;
  auto ready_bar = [&](int s) { return bar0 + 8u * (2 * C::STAGES + 4 + s); };
  int row0 = tile * 128;
  int row_end = P.rows;    // one past the tile's last row
  int kblocks = P.kblocks;
  int group = 0;           // expert
  int tok0 = 0, ntok = 0;  // products over the tokens: the expert's first token and count
  const GroupTable gt = group_table(smem + C::OFF_GROUPS);
  if (warp == 3 && lane == 0) {
    tma_prefetch_desc(&P.tm_a);
    tma_prefetch_desc(&P.tm_b);
    if (C::TWO_PART && P.parts == 2) tma_prefetch_desc(&P.tm_b2);
  }
  if constexpr (C::GROUPED) {
    // late launches run on inputs that are complete when they start
    if (!args.late) grid_dep_wait();
    if (blockIdx.x == 0)  // (before a launch without tokens leaves)
      for (int i = threadIdx.x; i < args.nzero; i += blockDim.x) args.zero_words[i] = 0u;
    if (warp == 2) build_group_table(args.groups, 128, gt);  // beside the barriers and TMEM below
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    mbar_init(tmem_full, 1);
    mbar_init(drain_bar, 1);
    if (C::GROUPED) {
      mbar_init(landed_bar, 1);
      mbar_init(tail_bar, 1);
    }
    for (int s = 0; s < C::STAGES && C::DROP; ++s) mbar_init(ready_bar(s), 8);
    *s_abort = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmem), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *s_tmem;
  if constexpr (C::GROUPED) {
    if constexpr (C::A_MN) {
      const int row_tiles = (P.rows + 127) / 128;
      group = tile / row_tiles;
      row0 = (tile - group * row_tiles) * 128;
      tok0 = gt.first[group];
      ntok = gt.first[group + 1] - tok0;
      kblocks = (ntok + 63) / 64;
    } else {
      if (tile >= gt.cum[args.groups.groups]) {  // the whole cluster leaves
        if (warp == 1) tmem_dealloc(tmem_base, C::TMEM_COLS);
        grid_dep_launch();
        return;
      }
      group = group_of_tile(gt, args.groups.groups, tile);
      row0 = gt.first[group] + (tile - gt.cum[group]) * 128;
      row_end = gt.first[group + 1];
    }
  }
  const int kb_begin = static_cast<int>((static_cast<int64_t>(rank) * kblocks) / splits);
  const int kb_end = static_cast<int>((static_cast<int64_t>(rank + 1) * kblocks) / splits);
  const int nk = kb_end - kb_begin;
  // this CTA's last block ends inside: its rows past the expert's last token are zeroed
  const int tail_rows = C::GROUPED && C::A_MN && nk > 0 && kb_end == kblocks ? ntok & 63 : 0;

  // producer state: stages issued so far (the first ring's worth may go out
  // ahead of the wait for the previous kernel, see SkinnyArgs::early)
  int issued = 0;
  auto issue = [&](int j) {
    const int s = j % C::STAGES;
    const int kb = kb_begin + j;
    const uint32_t a_dst = sbase + C::OFF_A + s * C::A_BYTES;
    const uint32_t b_dst = sbase + C::OFF_B + s * C::B_BYTES;
    mbar_arrive_expect_tx(full_bar(s), C::TX + (C::TWO_PART && P.parts == 2 ? C::PART_BYTES : 0));
    if constexpr (C::GROUPED) {
      if (C::A_MN) {  // token rows of both operands from the expert's first one on
        const int tok = tok0 + kb * 64;
        tma_load_2d(a_dst, &P.tm_a, full_bar(s), row0, tok);
        tma_load_2d(a_dst + 8192, &P.tm_a, full_bar(s), row0 + 64, tok);
#pragma unroll
        for (int c = 0; c < C::BN / 64; ++c) tma_load_2d(b_dst + c * 8192, &P.tm_b, full_bar(s), c * 64, tok);
        if (P.parts == 2) {
#pragma unroll
          for (int c = 0; c < C::BN / 64; ++c)
            tma_load_2d(b_dst + C::PART_BYTES + c * 8192, &P.tm_b2, full_bar(s), c * 64, tok);
        }
      } else {  // the expert's adapter: a slice of a 3-D map
        tma_load_2d(a_dst, &P.tm_a, full_bar(s), kb * 64, row0);
        if (C::B_MN) {
#pragma unroll
          for (int c = 0; c < C::BN / 64; ++c)
            tma_load_3d(b_dst + c * 8192, &P.tm_b, full_bar(s), c * 64, kb * 64, group);
        } else {
          tma_load_3d(b_dst, &P.tm_b, full_bar(s), kb * 64, 0, group);
        }
      }
      return;
    }
    if (C::A_MN) {
      tma_load_2d(a_dst, &P.tm_a, full_bar(s), row0, kb * 64);
      tma_load_2d(a_dst + 8192, &P.tm_a, full_bar(s), row0 + 64, kb * 64);
    } else {
      tma_load_2d(a_dst, &P.tm_a, full_bar(s), kb * 64, row0);
    }
    if (C::B_MN) {
#pragma unroll
      for (int c = 0; c < C::BN / 64; ++c) tma_load_2d(b_dst + c * 8192, &P.tm_b, full_bar(s), c * 64, kb * 64);
    } else {
      tma_load_2d(b_dst, &P.tm_b, full_bar(s), kb * 64, 0);
    }
  };
  if (!C::GROUPED && args.early && !args.late && warp == 0 && lane == 0)
    for (; issued < nk && issued < C::STAGES; ++issued) issue(issued);
  if (!C::GROUPED && !args.late) grid_dep_wait();
  grid_dep_launch();
  if (!C::GROUPED && blockIdx.x == 0)
    for (int i = threadIdx.x; i < args.nzero; i += blockDim.x) args.zero_words[i] = 0u;

  if (warp == 0) {
    if (lane == 0) {
      for (; issued < nk; ++issued) {
        const int s = issued % C::STAGES;
        if (!mbar_wait(empty_bar(s), ((issued / C::STAGES) & 1u) ^ 1u, s_abort)) break;
        issue(issued);
      }
      // wait (bounded) for this thread's copies still in flight
      const int inflight = issued < C::STAGES ? issued : C::STAGES;
      for (int i = 0; i < inflight; ++i) {
        const int jb = issued - 1 - i;
        const unsigned long long t0 = globaltimer_ns();
        while (!mbar_try_wait(full_bar(jb % C::STAGES), (jb / C::STAGES) & 1u)) {
          if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if ((!C::GROUPED || nk > 0) && elect_one()) {
      const uint32_t idesc = idesc_dtype(make_idesc_bf16(128, C::BN, C::A_MN ? 1 : 0, C::B_MN ? 1 : 0), args.f16);
      bool ok = true;
      for (int j = 0; j < nk; ++j) {
        const int s = j % C::STAGES;
        const uint32_t landed = C::DROP && P.masked ? ready_bar(s) : full_bar(s);
        if (!mbar_wait(landed, (j / C::STAGES) & 1u, s_abort)) { ok = false; break; }
        if (C::GROUPED && tail_rows > 0 && j == nk - 1) {
          mbar_arrive(landed_bar);  // (only this thread follows the ring's phases)
          if (!mbar_wait(tail_bar, 0, s_abort)) { ok = false; break; }
        }
        tc_fence_after();
        const uint32_t a_addr = sbase + C::OFF_A + s * C::A_BYTES;
        const uint32_t b_addr = sbase + C::OFF_B + s * C::B_BYTES;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const uint64_t ad = C::A_MN ? smem_desc_sw128(a_addr + kk * 2048, 8192, 1024)
                                      : smem_desc_sw128(a_addr + kk * 32, 16, 1024);
          const uint64_t bd = C::B_MN ? smem_desc_sw128(b_addr + kk * 2048, 8192, 1024)
                                      : smem_desc_sw128(b_addr + kk * 32, 16, 1024);
          tc_mma_ss(tmem_base, ad, bd, idesc, (j > 0 || kk > 0) ? 1u : 0u);
          if (C::TWO_PART && P.parts == 2)
            tc_mma_ss(tmem_base + C::BN, ad, smem_desc_sw128(b_addr + C::PART_BYTES + kk * 2048, 8192, 1024), idesc,
                      (j > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(empty_bar(s));
      }
      if (ok) tc_commit(tmem_full);
      tc_commit(drain_bar);
      const unsigned long long t0 = globaltimer_ns();
      while (!mbar_try_wait(drain_bar, 0)) {
        if (globaltimer_ns() - t0 > kWaitTimeoutNs) break;
      }
    }
    __syncwarp();
  } else if (C::GROUPED && warp == 2) {
    if (tail_rows > 0) {
      // once the last block has landed, zero its rows past the expert's last
      // token (a row is 128 consecutive bytes of each 64 x 64 chunk, whatever
      // the swizzle), then let the MMA thread read it
      const int s = (nk - 1) % C::STAGES;
      if (warp_wait_all(landed_bar, 0, s_abort)) {
        const int first = tail_rows * 8, per = 512 - first;  // 16-byte pieces of a chunk
        const int nch = 2 + C::BN / 64 * (P.parts == 2 ? 2 : 1);
        for (int i = lane; i < per * nch; i += 32) {
          const int c = i / per, o = first + i - c * per;
          uint8_t *chunk = c < 2 ? smem + C::OFF_A + s * C::A_BYTES + c * 8192
                                 : smem + C::OFF_B + s * C::B_BYTES + (c - 2) * 8192;
          *reinterpret_cast<uint4 *>(chunk + o * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(tail_bar);
      }
    }
  } else if (warp >= 4) {
    const int q = warp - 4;
    if constexpr (C::DROP) {
      // M o X, stage by stage. 16-byte piece c of row r of a 64-wide K-major
      // (or MN-major) chunk lies at c ^ (r & 7) in the row's 128 bytes. A
      // thread's four pieces are 32 rows apart; their masks are formed side by
      // side, two before and two after the stage before theirs is masked, so
      // that the shared-memory accesses (256 clocks a stage, beside some 1000
      // for the generator, whose instructions fill the issue slots) and the
      // fence pass meanwhile. Rows
      // of no token of this expert are masked too: never stored (K-major) or
      // zeroed by warp 2.
      const int tid = q * 32 + lane, c = tid & 7, r0 = tid >> 3;
      const uint32_t swz = static_cast<uint32_t>(c ^ (r0 & 7)) << 4;  // (the same for rows 32 apart)
      const uint64_t ld8 = static_cast<uint64_t>(args.drop_ld) / 8;
      uint4 mask[4];  // of the stage at hand
      // masks i0 and i0 + 1 of stage j. Counter of the piece in row r0:
      // K-major 128 token rows of one chunk, MN-major 64 token rows of two
      auto masks = [&](int j, int i0, uint4 (&m)[4]) {
        const int kb = kb_begin + j;
        const uint64_t first = C::A_MN ? static_cast<uint64_t>(tok0 + kb * 64 + r0) * ld8 + (row0 / 8 + c)
                                       : static_cast<uint64_t>(row0 + r0) * ld8 + (kb * 8 + c);
#pragma unroll
        for (int i = i0; i < i0 + 2; ++i)
          m[i] = dropout_mask8(args.drop, first + (C::A_MN ? (i & 1) * 32 * ld8 + (i >> 1) * 8 : i * 32 * ld8));
      };
      if (P.masked && nk > 0) {
        masks(0, 0, mask);
        masks(0, 2, mask);
      }
      for (int j = 0; P.masked && j < nk; ++j) {
        const int s = j % C::STAGES;
        if (!warp_wait_all(full_bar(s), (j / C::STAGES) & 1u, s_abort)) break;
        uint8_t *piece = smem + C::OFF_A + s * C::A_BYTES + r0 * 128 + swz;
        uint4 v[4], next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const uint4 *>(piece + i * 4096);
        if (j + 1 < nk) masks(j + 1, 0, next);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4 *>(piece + i * 4096) =
              make_uint4(v[i].x & mask[i].x, v[i].y & mask[i].y, v[i].z & mask[i].z, v[i].w & mask[i].w);
        if (j + 1 < nk) {
          masks(j + 1, 2, next);
#pragma unroll
          for (int i = 0; i < 4; ++i) mask[i] = next[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(ready_bar(s));
      }
    }
    // TMEM -> this CTA's fp32 partial in shared memory (the ring is idle now)
    const bool ok = (!C::GROUPED || nk > 0) && warp_wait_all(tmem_full, 0, s_abort);
    tc_fence_after();
    float *part = reinterpret_cast<float *>(smem);
    const int lrow = (q & 3) * 32 + lane;
#pragma unroll 1
    for (int ch = q >> 2; ch < C::BN / 32; ch += C::THREADS / 128 - 1) {
      uint32_t u[32];
      if (ok && nk > 0) {
        tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>((q & 3) * 32) << 16) + ch * 32, u);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] = 0u;
      }
      if (C::TWO_PART && P.parts == 2 && ok && nk > 0) {
        uint32_t w[32];
        tmem_ld_32x32b_x32(tmem_base + (static_cast<uint32_t>((q & 3) * 32) << 16) + C::BN + ch * 32, w);
        const float inv = 1.0f / part_scale(args.f16 != 0);  // (a power of two)
#pragma unroll
        for (int j = 0; j < 32; ++j) u[j] = __float_as_uint(join_parts(u[j], w[j], inv));
      }
      float4 *dst = reinterpret_cast<float4 *>(part + lrow * C::PART_LD + ch * 32);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dst[j] = make_float4(__uint_as_float(u[4 * j]), __uint_as_float(u[4 * j + 1]),
                             __uint_as_float(u[4 * j + 2]), __uint_as_float(u[4 * j + 3]));
    }
    tc_fence_before();
  }

  __syncthreads();
  if (splits > 1) cluster_sync();  // every partial of the cluster is in place

  // Reduce this CTA's slice of rows over the cluster's partials, rank order.
  {
    const int R = 128 / splits;
    const int c4n = C::BN / 4;  // float4 per row
    const int units = R * c4n;
    const uint32_t part_addr = sbase;
    for (int u = threadIdx.x; u < units; u += C::THREADS) {
      int lr, c4;
      if (P.transpose) {  // consecutive threads -> consecutive rows (coalesced transposed store)
        c4 = u / R;
        lr = u - c4 * R;
      } else {  // consecutive threads -> consecutive columns
        lr = u / c4n;
        c4 = u - lr * c4n;
      }
      if (c4 * 4 >= P.cols) continue;  // (a multiple of 8: four columns or none)
      const int lrow = static_cast<int>(rank) * R + lr;
      const uint32_t off = static_cast<uint32_t>((lrow * C::PART_LD + c4 * 4) * 4);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (splits > 1) {
        // all peers' loads in flight at once, then summed in rank order
        float4 x[8];
#pragma unroll
        for (int sp = 0; sp < 8; ++sp)
          if (sp < splits) x[sp] = ld_cluster_f4(map_cluster(part_addr + off, sp));
#pragma unroll
        for (int sp = 0; sp < 8; ++sp)
          if (sp < splits) {
            v.x += x[sp].x;
            v.y += x[sp].y;
            v.z += x[sp].z;
            v.w += x[sp].w;
          }
      } else {
        v = *reinterpret_cast<const float4 *>(smem + off);
      }
      const int row = row0 + lrow;
      if (row >= row_end) continue;
      const float vv[4] = {v.x, v.y, v.z, v.w};
      for (int o = 0; o < 2; ++o) {
        uint16_t *dst = reinterpret_cast<uint16_t *>(o ? P.out2 : P.out);
        if (dst == nullptr) continue;
        if constexpr (C::GROUPED && C::A_MN) dst += static_cast<int64_t>(group) * P.rows * P.cols;  // this expert's
        const float sc = o ? P.out2_scale : P.out_scale;
        const int64_t ld = o ? P.out2_ld : P.out_ld;
        const bool f16 = args.f16 != 0;
        if (P.transpose) {
#pragma unroll
          for (int e = 0; e < 4; ++e) dst[static_cast<int64_t>(c4 * 4 + e) * ld + row] = to_16(vv[e] * sc, f16);
        } else {
          uint2 w = make_uint2(pack_16x2(vv[0] * sc, vv[1] * sc, f16), pack_16x2(vv[2] * sc, vv[3] * sc, f16));
          if (C::GROUPED && o && P.rest) {  // out2_scale is out_scale: what `out` rounded away
            auto rest = [&](int e, uint32_t pair) {
              return static_cast<uint32_t>(
                  second_part(vv[e] * sc, static_cast<uint16_t>(e & 1 ? pair >> 16 : pair), f16));
            };
            w = make_uint2(rest(0, w.x) | rest(1, w.x) << 16, rest(2, w.y) | rest(3, w.y) << 16);
          }
          *reinterpret_cast<uint2 *>(dst + static_cast<int64_t>(row) * ld + c4 * 4) = w;
        }
      }
    }
  }
  if (splits > 1) cluster_sync();  // peers are done reading this CTA's partial

  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if (args.late) grid_dep_wait();
}

}  // namespace qlora
