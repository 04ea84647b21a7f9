// Dropout masks from a counter-based generator: Philox4x32 (Salmon, Moraes,
// Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", 2011), with 7
// rounds, the fewest that the paper finds to pass its whole test battery; a mask is
// drawn again wherever it is needed and never stored.
//
// Of one draw's 128 bits every element takes 15: piece e is the low 15 bits
// of half (e % 2) of word e / 2, so one draw serves 8 consecutive keys of a row
// and a probability is met to 2^-16.  (About 4
// instructions an element; 7 bits each would halve that and meet a probability to 2^-8 only.)
#pragma once

#include <cstdint>

namespace cpattn {

struct Draw {
  uint32_t w[4];
};

// What a call's masks are drawn with: the seed, and the counter's last word.
struct DropKey {
  uint32_t k0, k1, c3;
  uint32_t add;  // (2^15 - threshold) in both halves: see keep_halves
};

__device__ __forceinline__ DropKey drop_key(const uint64_t* rng, uint32_t threshold) {
  const uint64_t seed = rng[0], offset = rng[1];
  return DropKey{uint32_t(seed), uint32_t(seed >> 32), uint32_t(offset), (0x8000u - threshold) * 0x10001u};
}

// The same with the keys of all rounds formed beforehand, where there are registers for them: the adds are a fifth
// of a draw's instructions (forward under dropout, 8 x 2048, 16 heads of 64: 447 -> 408 us).
struct DropKeys {
  uint32_t k0[7], k1[7], c3, add;
};
__device__ __forceinline__ DropKeys drop_keys(const DropKey& key) {
  DropKeys x;
  x.c3 = key.c3;
  x.add = key.add;
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    x.k0[r] = key.k0 + uint32_t(r) * 0x9E3779B9u;
    x.k1[r] = key.k1 + uint32_t(r) * 0xBB67AE85u;
    asm volatile("" : "+r"(x.k0[r]), "+r"(x.k1[r]));  // not to be formed again
  }
  return x;
}
__device__ __forceinline__ uint32_t round_key0(const DropKey& key, int r) { return key.k0 + uint32_t(r) * 0x9E3779B9u; }
__device__ __forceinline__ uint32_t round_key1(const DropKey& key, int r) { return key.k1 + uint32_t(r) * 0xBB67AE85u; }
__device__ __forceinline__ uint32_t round_key0(const DropKeys& key, int r) { return key.k0[r]; }
__device__ __forceinline__ uint32_t round_key1(const DropKeys& key, int r) { return key.k1[r]; }

// Counter: keys 8 block .. 8 block + 7 of query i (counted in its sequence), and
// sequence * heads + head.
template <class K>
__device__ __forceinline__ Draw draw(const K& key, uint32_t block, uint32_t i, uint32_t seq_head) {
  uint32_t c0 = block, c1 = i, c2 = seq_head, c3 = key.c3;
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t a = uint64_t(c0) * 0xD2511F53u, b = uint64_t(c2) * 0xCD9E8D57u;
    c0 = uint32_t(b >> 32) ^ c1 ^ round_key0(key, r);
    c1 = uint32_t(b);
    c2 = uint32_t(a >> 32) ^ c3 ^ round_key1(key, r);
    c3 = uint32_t(a);
  }
  return Draw{{c0, c1, c2, c3}};
}

// Bits 15 and 31: whether the two pieces of a word reach the threshold.
__device__ __forceinline__ uint32_t keep_halves(uint32_t word, uint32_t add) { return (word & 0x7fff7fffu) + add; }

// The same as a mask of a pair of 16-bit values: each half all ones or zeros.
__device__ __forceinline__ uint32_t keep_mask(uint32_t word, uint32_t add) {
  uint32_t m;
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(m) : "r"(keep_halves(word, add)));
  return m;
}

// One bit for each of a draw's 8 keys, the first key's lowest.
__device__ __forceinline__ uint32_t keep_bits(const Draw& d, uint32_t add) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = keep_halves(d.w[i], add) & 0x80008000u;
    bits |= (t >> (15 - 2 * i)) | (t >> (30 - 2 * i));
  }
  return bits & 0xffu;
}

}  // namespace cpattn
