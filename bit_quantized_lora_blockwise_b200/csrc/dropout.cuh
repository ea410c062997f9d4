// Dropout from a counter-based generator: whether element i is kept is a
// pure function of (seed, offset, i), so no mask is ever stored; the forward
// and the backward (and a recomputed forward) evaluate the same function.
//
// Generator: Philox4x32 with 10 rounds (J. Salmon, M. Moraes, R. Dror,
// D. Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11), 64-bit key
// = seed, 128-bit counter = offset + i / 8 in its low 64 bits. One counter
// gives four words = eight 16-bit halves; element i takes half i % 8 (low
// half of word 0 first) and is kept where half >= threshold, threshold =
// round(p 2^16). Kept elements are scaled by 2^16 / (2^16 - threshold), the
// exact inverse of the keep probability at that resolution, so the mean is
// preserved exactly.
#pragma once

#include "ptx.cuh"

namespace qlora {

struct DropoutArgs {
  uint32_t key[10][2];  // the rounds' keys, formed once on the host: constant operands of the rounds' xors
  uint64_t offset;
  uint32_t threshold;  // 0: nothing is dropped
  uint32_t both;       // the threshold in both halves
  uint32_t low15;      // and its lower 15 bits
  float factor;        // 2^16 / (2^16 - threshold)
};

inline DropoutArgs dropout_args(uint64_t seed, uint64_t offset, uint32_t threshold) {
  DropoutArgs d;
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
  for (int round = 0; round < 10; ++round, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
    d.key[round][0] = k0;
    d.key[round][1] = k1;
  }
  d.offset = offset;
  d.threshold = threshold;
  d.both = threshold << 16 | threshold;
  d.low15 = d.both & 0x7FFF7FFFu;
  d.factor = static_cast<float>(65536.0 / (65536.0 - threshold));
  return d;
}

// The eight halves of one counter, two per word.
__device__ __forceinline__ uint4 philox4x32_10(const DropoutArgs &d, uint64_t counter) {
  uint32_t c0 = static_cast<uint32_t>(counter), c1 = static_cast<uint32_t>(counter >> 32), c2 = 0u, c3 = 0u;
#pragma unroll
  for (int round = 0; round < 10; ++round) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    const uint32_t n0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ d.key[round][0];
    const uint32_t n2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ d.key[round][1];
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    c0 = n0;
    c2 = n2;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Both halves of a word against the threshold at once: bit 15 and bit 31 tell
// whether the low and the high half are kept (the other bits are of no use).
// With the top bit forced, a subtraction compares the 15 bits below it without
// a borrow between the halves; the top bits themselves decide where they
// differ. Three integer operations where two compares of shifted halves, with
// their selects, take six.
__device__ __forceinline__ uint32_t keep_signs(const DropoutArgs &d, uint32_t word) {
  const uint32_t z = (word | 0x80008000u) - d.low15;
  return (word & ~d.both) | (~(word ^ d.both) & z);
}

// Keep bits of the eight elements of one counter (bit j: element j).
__device__ __forceinline__ uint32_t dropout_keep8(const DropoutArgs &d, uint64_t group) {
  const uint4 w = philox4x32_10(d, d.offset + group);
  // four elements a word, a byte of ones or zeros each (the signs of bytes 1
  // and 3), a bit of each byte kept, the four bytes added up
  const uint32_t lo = prmt(keep_signs(d, w.x), keep_signs(d, w.y), 0xFDB9u);
  const uint32_t hi = prmt(keep_signs(d, w.z), keep_signs(d, w.w), 0xFDB9u);
  return (((lo & 0x08040201u) | (hi & 0x80402010u)) * 0x01010101u) >> 24;
}

// The same as masks of the four words of eight 16-bit elements.
__device__ __forceinline__ uint4 dropout_mask8(const DropoutArgs &d, uint64_t group) {
  const uint4 w = philox4x32_10(d, d.offset + group);
  auto mask = [&](uint32_t word) {
    const uint32_t s = keep_signs(d, word);
    return prmt(s, s, 0xBB99u);
  };
  return make_uint4(mask(w.x), mask(w.y), mask(w.z), mask(w.w));
}

enum DropoutType : int { DROP_BF16 = 0, DROP_F16 = 1, DROP_F32 = 2 };

// Two elements of a word's halves, masked: times the factor (fp32 product, one
// rounding). A dropped element is +0, whatever it held (NaN and infinity too).
template <int TYPE>
__device__ __forceinline__ uint32_t dropout_pair(uint32_t v, uint32_t mask, float factor) {
  v &= mask;
  float lo, hi;
  if constexpr (TYPE == DROP_F16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&v));
    lo = f.x;
    hi = f.y;
  } else {
    lo = __uint_as_float(v << 16);
    hi = __uint_as_float(v & 0xFFFF0000u);
  }
  return pack_16x2(lo * factor, hi * factor, TYPE == DROP_F16);
}

// y[i] = keep(i) ? x[i] * factor : 0 over n elements; x and y 16-byte
// aligned, y == x allowed. One thread per counter (8 elements: one 16-byte
// load and store for 16-bit types, two for fp32).
template <int TYPE>
__global__ void __launch_bounds__(256) dropout_kernel(const void *x, void *y, int64_t n,
                                                      const __grid_constant__ DropoutArgs d) {
  const float factor = d.factor;
  grid_dep_wait();
  grid_dep_launch();
  const int64_t full = n / 8;
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t g0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t g = g0; g < full; g += step) {
    if constexpr (TYPE == DROP_F32) {
      const float4 a = reinterpret_cast<const float4 *>(x)[2 * g], b = reinterpret_cast<const float4 *>(x)[2 * g + 1];
      const uint32_t k = dropout_keep8(d, static_cast<uint64_t>(g));
      reinterpret_cast<float4 *>(y)[2 * g] =
          make_float4(k & 1u ? a.x * factor : 0.0f, k & 2u ? a.y * factor : 0.0f, k & 4u ? a.z * factor : 0.0f,
                      k & 8u ? a.w * factor : 0.0f);
      reinterpret_cast<float4 *>(y)[2 * g + 1] =
          make_float4(k & 16u ? b.x * factor : 0.0f, k & 32u ? b.y * factor : 0.0f, k & 64u ? b.z * factor : 0.0f,
                      k & 128u ? b.w * factor : 0.0f);
    } else {
      const uint4 v = reinterpret_cast<const uint4 *>(x)[g];
      const uint4 m = dropout_mask8(d, static_cast<uint64_t>(g));
      reinterpret_cast<uint4 *>(y)[g] =
          make_uint4(dropout_pair<TYPE>(v.x, m.x, factor), dropout_pair<TYPE>(v.y, m.y, factor),
                     dropout_pair<TYPE>(v.z, m.z, factor), dropout_pair<TYPE>(v.w, m.w, factor));
    }
  }
  // the last, partial counter: one thread, element by element
  const int rest = static_cast<int>(n - full * 8);
  if (rest > 0 && g0 == 0) {
    const uint32_t k = dropout_keep8(d, static_cast<uint64_t>(full));
    for (int j = 0; j < rest; ++j) {
      const int64_t i = full * 8 + j;
      if constexpr (TYPE == DROP_F32) {
        const float v = reinterpret_cast<const float *>(x)[i];
        reinterpret_cast<float *>(y)[i] = (k >> j) & 1u ? v * factor : 0.0f;
      } else {
        const uint32_t v = reinterpret_cast<const uint16_t *>(x)[i];
        reinterpret_cast<uint16_t *>(y)[i] = static_cast<uint16_t>(dropout_pair<TYPE>(v, (k >> j) & 1u ? 0xFFFFu : 0u, factor));
      }
    }
  }
}

}  // namespace qlora
