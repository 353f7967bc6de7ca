// Dropout from a counter: which elements are dropped is a function of the seed, the step, the site (which
// dropout of the model) and the element's row and column, so no mask is ever stored.
//
// Philox's key is the seed, its counter (column / 8, row, site, step): 128 bits for eight columns of a row,
// 16 for each (word j / 2's lower, then upper half).  An element is dropped where its 16 bits are below
// P = round(65536 p).  Sixteen bits resolve p to 2^-17, and half the calls of 32 bits an element are left: at
// 16384 x 1536 BF16 the rounds of one call per four elements would take as long as the memory traffic.
#pragma once

#include "act.cuh"
#include "philox.cuh"

namespace gift {

struct Dropout {
  const unsigned long long *rng;   // device: seed, step
  uint32_t below;                  // P; 0: nothing is dropped and rng is not read
  uint32_t site;
  float scale;                     // 65536 / (65536 - P)
};

// What a thread draws with: loaded once per kernel.
struct Draw {
  uint32_t k0 = 0, k1 = 0, site, step = 0, below;
  float scale;
  __device__ __forceinline__ explicit Draw(const Dropout &d) : site(d.site), below(d.below), scale(d.scale) {
    if (below) {
      const unsigned long long seed = d.rng[0];
      k0 = (uint32_t)seed;
      k1 = (uint32_t)(seed >> 32);
      step = (uint32_t)d.rng[1];
    }
  }
  // the bits of the eight columns from 8 group
  __device__ __forceinline__ U4 bits(uint32_t row, uint32_t group) const {
    return philox4x32_10(U4{group, row, site, step}, k0, k1);
  }
  // bit j: column 8 group + j of the row is kept.  A half is at least P where, in the upper half of a word, it is
  // at least P 2^16.
  __device__ __forceinline__ uint32_t keep8(uint32_t row, uint32_t group) const {
    const U4 r = bits(row, group);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w}, least = below << 16;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m |= (w[j] << 16 >= least ? 1u << (2 * j) : 0u) | (w[j] >= least ? 2u << (2 * j) : 0u);
    return m;
  }
  // dropped to 0, or scaled: v[k] holds columns 2 k and 2 k + 1 of a group
  __device__ __forceinline__ void apply8(float2 *v, uint32_t row, uint32_t group) const {
    const U4 r = bits(row, group);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w}, least = below << 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j].x = w[j] << 16 >= least ? v[j].x * scale : 0.0f;
      v[j].y = w[j] >= least ? v[j].y * scale : 0.0f;
    }
  }
  // of the 16 columns from 8 group
  __device__ __forceinline__ uint32_t keep16(uint32_t row, uint32_t group) const {
    return keep8(row, group) | keep8(row, group + 1) << 8;
  }
};

}  // namespace gift
