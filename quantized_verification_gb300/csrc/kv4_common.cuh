// kv4_common.cuh -- the 4-bit paged KV cache, shared by the kernels that
// write it, read it back and attend over it.
//
// The cache is a pool of blocks of 32 positions. Block `page` of key/value
// head h is a record of 34 D bytes at (page * Hkv + h) * 34 D:
//   [0, 16 D)      key codes    [32][D/2]   (even element in the low nibble)
//   [16 D, 32 D)   value codes  [32][D/2]
//   [32 D, 33 D)   key scales   [32][D/32]
//   [33 D, 34 D)   value scales [32][D/32]
// One record holds all that 32 positions of a head need, so that attention
// fetches it with a single bulk copy (4352 bytes at D = 128).
//
// A code is a two's-complement nibble q in [-7, 7]; a scale byte b, shared by
// 32 elements, stands for s = (1 + (b & 7) / 8) 2^((b >> 3) - 15): 5 exponent
// and 3 mantissa bits without sign, zero, infinity or NaN, so that any byte
// is a finite scale. q has 3 significant bits and s has 4, so q * s is exact
// in bf16. That is why the scale has 8 bits and not 16 or 32: the tensor
// cores take the cache's values without any rounding, and the values read
// back as bf16 are the very values attention uses.
#pragma once

#include <cstdint>

#include "qv_ptx.cuh"

namespace qv {

constexpr int kKv4Block = 32;    // positions per record
constexpr int kKv4Group = 32;    // elements per scale

template <int D>
struct Kv4Rec {
    static constexpr int RowBytes = D / 2;            // codes of one position
    static constexpr int RowScales = D / kKv4Group;   // scale bytes of one position
    static constexpr int KC = 0;
    static constexpr int VC = 16 * D;
    static constexpr int KS = 32 * D;
    static constexpr int VS = 33 * D;
    static constexpr int Bytes = 34 * D;
};

// The binary32 value of a scale byte: its 8 bits are the low exponent and the
// high mantissa bits of a binary32 number with the exponent offset by 112.
__device__ __forceinline__ float kv4_scale(uint32_t b) { return __uint_as_float((b << 20) + (112u << 23)); }

// Page of block `blk` of sequence b, or -1 when the table's entry is outside
// [0, pages). Without a table sequence b's blocks are pages b * NB + blk.
__device__ __forceinline__ int kv4_page(const int32_t* table, int b, int NB, int pages, int blk) {
    if (!table) return b * NB + blk;
    const int p = table[(size_t)b * NB + blk];
    return (unsigned)p < (unsigned)pages ? p : -1;
}

}  // namespace qv
