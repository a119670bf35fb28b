// k_kv4.cu -- key/value rows quantized to 4 bits as they are written into the
// paged cache, and cached positions read back as values.
//
//   Lower bit widths are the next step the Quasar summaries name
//   (gist.science/it, gist.science/de and gist.science/ja summaries, section
//   5); the cache keeps the a0 rule (symmetric, round half to even) with 7
//   for 127 and one scale for every 32 elements of a head's row, so that an
//   outlier channel costs its own 32 neighbours precision and no others.
//
// A CTA takes the positions of one sequence in one block, for one head or a
// few, so that the chain start -> block table -> record is walked once for all
// of them. A thread moves 8 elements (16 bytes of bf16), four threads a scale
// group, consecutive threads on consecutive elements: the wide side moves in
// runs of 256 bytes (a head's row at D = 128), the codes in whole sectors, and
// the four rows of a thread are requested before the first is worked on. Bound
// by launch latency at a step's few rows (2.4 us), by memory and its latency at
// prompt lengths: 85 MB in 15.6 us (5.4 TB/s) for the two prompts below, 113 MB
// in 19.4 us (5.8 TB/s) for the four caches; a plain copy runs at 6.8.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4_common.cuh"
#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace qv {
namespace {

constexpr int kKv4Threads = 256;

struct Kv4Args {
    const uint8_t* x;          // write: rows [B*T][(Hq + 2 Hkv) D] fp32 or bf16
    uint8_t* k_out;            // read: [B*T][Hkv D] fp32 or bf16
    uint8_t* v_out;
    uint8_t* cache;
    const int32_t* table;
    const int32_t* start;
    const int32_t* count;
    int T, Hq, Hkv, NB, pages;
    int heads;                 // heads of a CTA
};

// What a CTA works on: sequence b's rows in one block. Rows past the count,
// positions outside the block table and pages outside the pool have none.
struct Block {
    int first;                 // the sequence's row (j) at the block's slot 0; may be negative
    int rows;                  // rows j in [0, rows) exist
    const uint8_t* page;       // the block's records, or null
};
__device__ __forceinline__ Block find_block(const Kv4Args& a, int b, int nth, size_t rec_bytes) {
    const int start = a.start[b], cnt = a.count ? a.count[b] : a.T;
    const long long blk = (long long)(start >> 5) + nth;         // (>> rounds down)
    Block k;
    k.rows = cnt < a.T ? cnt : a.T;
    k.page = nullptr;
    k.first = (int)(blk * kKv4Block - start);
    if (blk < 0 || blk >= a.NB || k.first >= k.rows) return k;
    const int page = kv4_page(a.table, b, a.NB, a.pages, (int)blk);
    if (page >= 0) k.page = a.cache + (size_t)page * a.Hkv * rec_bytes;
    return k;
}

// The larger magnitude, NaN if either is NaN.
__device__ __forceinline__ float max_abs_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(fabsf(b)));
    return y;
}

template <bool BF16>
struct Raw {                   // 8 elements as they are in memory
    uint4 u[BF16 ? 1 : 2];
    __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) u[i] = reinterpret_cast<const uint4*>(p)[i];
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) {
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (BF16) {
                    v[2 * k] = __uint_as_float(w[k] << 16);
                    v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
                } else {
                    v[4 * i + k] = __uint_as_float(w[k]);
                }
            }
        }
    }
};

// The largest magnitude of three, NaN if one is NaN.
__device__ __forceinline__ float max_abs_nan3(float a, float b, float c) {
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// The scale byte of a group whose largest magnitude is amax: the nearest scale
// to fl32(amax / 7), ties to the even byte. Rounding adds half of the last
// kept bit (and the kept bit itself, for ties) to the binary32 pattern.
//
// A bf16 amax has 8 significant bits, and its seventh is either halfway between
// two scales or further than 2^-11 of itself from there: the product with
// fl32(1/7), within 2 units of the last place, decides as the quotient does
// once its last 4 bits are rounded away (checked for every bf16 number).
template <bool BF16>
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    uint32_t u;
    if (BF16) u = (__float_as_uint(__fmul_rn(amax, 1.0f / 7.0f)) + 8u) & ~15u;
    else u = __float_as_uint(__fdiv_rn(amax, 7.0f));
    const int b = (int)((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - 896;
    return (uint32_t)(b < 0 ? 0 : (b > 255 ? 255 : b));
}

// The codes of 8 elements, four neighbouring threads (of `mask`) a group.
//
// The code is the integer nearest fl32(x / s). With r = fl32(1 / s) and
// q0 = fl32(x r), the residual x - q0 s is exact in a fused multiply-add, and
// q0 + r * residual is the correctly rounded quotient (one correction step of
// Markstein, IBM J. Res. Dev. 34, 1990; checked against the quotient for every
// binary32 significand and all 8 significands of s). Adding 1.5 * 2^23 + 8
// rounds it half to even and leaves q + 8 in the low bits; the eight sums are
// weighted by 16^i, and one subtraction takes the constant parts off.
// |x / s| < 7.5 by the choice of s, but for scales cut off at the largest one.
//
// A bf16 x has 8 significant bits and s has 4, so that x / s is either halfway
// between two integers or further than 2^-11 from there. x r with an r within 2
// units of the last place of 1 / s, rounded to a multiple of 2^-11 by adding
// 1.5 * 2^12, is then on the quotient's side of every halfway point, or on it
// (checked for every such x and s and five r). That takes two operations an
// element in place of four; with the reciprocal and the product with 1/7 in
// place of two divisions the prompt-length write is no longer bound by
// instruction issue.
template <bool BF16>
__device__ __forceinline__ uint32_t encode8(float (&v)[8], unsigned mask, uint32_t& sb) {
    float am = max_abs_nan3(max_abs_nan3(v[0], v[1], v[2]), max_abs_nan3(v[3], v[4], v[5]), max_abs_nan(fabsf(v[6]), v[7]));
    am = max_abs_nan(am, __shfl_xor_sync(mask, am, 1));
    am = max_abs_nan(am, __shfl_xor_sync(mask, am, 2));
    if (!(am <= 7.f * 122880.f)) {                             // rare: NaN counts as 0, large magnitudes saturate
        am = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = v[i] == v[i] ? fminf(fmaxf(v[i], -7.f * 122880.f), 7.f * 122880.f) : 0.f;
            am = fmaxf(am, fabsf(v[i]));
        }
        am = fmaxf(am, __shfl_xor_sync(mask, am, 1));
        am = fmaxf(am, __shfl_xor_sync(mask, am, 2));
    }
    sb = scale_byte<BF16>(am);
    const float s = kv4_scale(sb);
    float r;
    if (BF16) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    else r = __fdiv_rn(1.0f, s);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float q;
        if (BF16) {
            q = __fadd_rn(__fmaf_rn(v[i], r, 6144.0f), 12582920.0f - 6144.0f);
        } else {
            const float q0 = __fmul_rn(v[i], r);
            q = __fadd_rn(__fmaf_rn(__fmaf_rn(-q0, s, v[i]), r, q0), 12582920.0f);
        }
        w += __float_as_uint(q) * (1u << (4 * i));
    }
    constexpr uint32_t ones = 0x11111111u;
    return (w - 0x4B400000u * ones) ^ 0x88888888u;             // q + 8, then two's complement
}

// Five CTAs an SM for bf16 rows (48 registers): two prompts of 8190 tokens, 8
// heads, D = 128, in 15.6 us (17.2 with four CTAs, 16.7 with six, which spill).
template <int D, bool BF16>
__global__ void __launch_bounds__(kKv4Threads, BF16 ? 5 : 3) kv4_write_kernel(const Kv4Args a) {
    using Rec = Kv4Rec<D>;
    constexpr int Chunks = D / 8;                              // threads of a row
    constexpr int Rows = kKv4Threads / Chunks;                 // rows the CTA takes at once
    constexpr int Steps = 2 * kKv4Block / Rows;                // keys, then values
    allow_dependent_launch();
    grid_dependency_wait();
    const int b = blockIdx.z, h0 = blockIdx.y * a.heads;
    const Block k = find_block(a, b, blockIdx.x, Rec::Bytes);
    if (!k.page) return;
    const int c = threadIdx.x % Chunks, r = threadIdx.x / Chunks;
    const unsigned mask = 0xFu << (threadIdx.x & 28);
    constexpr int E = BF16 ? 2 : 4;
    const size_t rowlen = (size_t)(a.Hq + 2 * a.Hkv) * D;
    for (int h = h0; h < min(a.Hkv, h0 + a.heads); ++h) {
        uint8_t* rec = const_cast<uint8_t*>(k.page) + (size_t)h * Rec::Bytes;
        const uint8_t* x = a.x + ((size_t)b * a.T * rowlen + (size_t)(a.Hq + h) * D + c * 8) * E;
        Raw<BF16> raw[Steps];
#pragma unroll
        for (int i = 0; i < Steps; ++i) {
            const int kv = i / (Steps / 2), slot = (i % (Steps / 2)) * Rows + r, j = k.first + slot;
            if (j >= 0 && j < k.rows) raw[i].load(x + ((size_t)j * rowlen + (size_t)kv * a.Hkv * D) * E);
        }
#pragma unroll
        for (int i = 0; i < Steps; ++i) {
            const int kv = i / (Steps / 2), slot = (i % (Steps / 2)) * Rows + r, j = k.first + slot;
            if (j < 0 || j >= k.rows) continue;                // (whole rows: groups of 4 threads stay together)
            float v[8];
            raw[i].values(v);
            uint32_t sb;
            const uint32_t w = encode8<BF16>(v, mask, sb);
            *reinterpret_cast<uint32_t*>(rec + (kv ? Rec::VC : Rec::KC) + slot * Rec::RowBytes + c * 4) = w;
            if ((c & 3) == 0) rec[(kv ? Rec::VS : Rec::KS) + slot * Rec::RowScales + (c >> 2)] = (uint8_t)sb;
        }
    }
}

// The values of 8 codes as four bf16 pairs: a nibble shifted to bits 3..6 with
// its sign bit flipped, under the bf16 pattern of 16.0, is 24 + q; one fused
// multiply-add gives (24 + q) s - 24 s = q s exactly. That yields the pairs
// (j, j + 4), which byte permutations put in order.
__device__ __forceinline__ uint4 decode8(uint32_t w, uint32_t sb) {
    const uint32_t s = sb * 0x00100010u + 0x38003800u;
    uint32_t off, p[4];
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(off) : "r"(s), "r"(0xC1C0C1C0u));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t y = ((j == 0 ? w << 3 : w >> (4 * j - 3)) & 0x00780078u) ^ 0x41C041C0u;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(p[j]) : "r"(y), "r"(s), "r"(off));
    }
    return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410), __byte_perm(p[0], p[1], 0x7632),
                      __byte_perm(p[2], p[3], 0x7632));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Args a) {
    using Rec = Kv4Rec<D>;
    constexpr int Chunks = D / 8, Rows = kKv4Threads / Chunks, Steps = 2 * kKv4Block / Rows;
    allow_dependent_launch();
    grid_dependency_wait();
    const int b = blockIdx.z, h0 = blockIdx.y * a.heads;
    const Block k = find_block(a, b, blockIdx.x, Rec::Bytes);
    if (!k.page) return;
    const int c = threadIdx.x % Chunks, r = threadIdx.x / Chunks;
    constexpr int E = BF16 ? 2 : 4;
    for (int h = h0; h < min(a.Hkv, h0 + a.heads); ++h) {
        const uint8_t* rec = k.page + (size_t)h * Rec::Bytes;
        uint32_t w[Steps], sb[Steps];
#pragma unroll
        for (int i = 0; i < Steps; ++i) {                      // (every slot of the record can be read)
            const int kv = i / (Steps / 2), slot = (i % (Steps / 2)) * Rows + r;
            w[i] = *reinterpret_cast<const uint32_t*>(rec + (kv ? Rec::VC : Rec::KC) + slot * Rec::RowBytes + c * 4);
            sb[i] = rec[(kv ? Rec::VS : Rec::KS) + slot * Rec::RowScales + (c >> 2)];
        }
#pragma unroll
        for (int i = 0; i < Steps; ++i) {
            const int kv = i / (Steps / 2), slot = (i % (Steps / 2)) * Rows + r, j = k.first + slot;
            if (j < 0 || j >= k.rows) continue;
            const uint4 y = decode8(w[i], sb[i]);
            uint8_t* o = (kv ? a.v_out : a.k_out) + (((size_t)b * a.T + j) * (size_t)a.Hkv * D + (size_t)h * D + c * 8) * E;
            if (BF16) {
                *reinterpret_cast<uint4*>(o) = y;
            } else {
                *reinterpret_cast<uint4*>(o) = make_uint4(y.x << 16, y.x & 0xFFFF0000u, y.y << 16, y.y & 0xFFFF0000u);
                *reinterpret_cast<uint4*>(o + 16) = make_uint4(y.z << 16, y.z & 0xFFFF0000u, y.w << 16, y.w & 0xFFFF0000u);
            }
        }
    }
}

// One CTA per sequence, block that its T rows can touch, and group of heads:
// as many heads as leave `ctas_per_sm` CTAs an SM (or one head each). Writing
// takes 8: with 16 the two prompts above take 18.7 us for 17.2. Reading takes 32,
// since with ragged counts many CTAs find nothing to do: four caches of up to
// 16384 positions 19.4 us, 22.5 with 8, 25.6 with one head a CTA.
template <class Kernel>
cudaError_t launch_rows(Kernel kernel, Kv4Args& a, int B, int sms, int ctas_per_sm, cudaStream_t s) {
    const int blocks = (a.T + kKv4Block - 2) / kKv4Block + 1;
    a.heads = 1;
    while (a.heads * 2 <= a.Hkv && (long long)blocks * B * ceil_div(a.Hkv, a.heads * 2) >= (long long)ctas_per_sm * sms)
        a.heads *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)ceil_div(a.Hkv, a.heads), (unsigned)B);
    cfg.blockDim = dim3(kKv4Threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

cudaError_t launch_kv4_write(const void* x, bool bf16, const int32_t* start, const int32_t* count,
                             const int32_t* table, int B, int T, int Hq, int Hkv, int D, int NB, int pages,
                             uint8_t* cache, int sms, cudaStream_t s) {
    Kv4Args a = {};
    a.x = static_cast<const uint8_t*>(x);
    a.cache = cache; a.table = table; a.start = start; a.count = count;
    a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.NB = NB; a.pages = pages;
    if (D == 128) return bf16 ? launch_rows(kv4_write_kernel<128, true>, a, B, sms, 8, s) : launch_rows(kv4_write_kernel<128, false>, a, B, sms, 8, s);
    return bf16 ? launch_rows(kv4_write_kernel<64, true>, a, B, sms, 8, s) : launch_rows(kv4_write_kernel<64, false>, a, B, sms, 8, s);
}

cudaError_t launch_kv4_read(const uint8_t* cache, const int32_t* start, const int32_t* count, const int32_t* table,
                            int B, int T, int Hkv, int D, int NB, int pages, void* k_out, void* v_out, bool bf16,
                            int sms, cudaStream_t s) {
    Kv4Args a = {};
    a.k_out = static_cast<uint8_t*>(k_out); a.v_out = static_cast<uint8_t*>(v_out);
    a.cache = const_cast<uint8_t*>(cache); a.table = table; a.start = start; a.count = count;
    a.T = T; a.Hkv = Hkv; a.NB = NB; a.pages = pages;
    if (D == 128) return bf16 ? launch_rows(kv4_read_kernel<128, true>, a, B, sms, 32, s) : launch_rows(kv4_read_kernel<128, false>, a, B, sms, 32, s);
    return bf16 ? launch_rows(kv4_read_kernel<64, true>, a, B, sms, 32, s) : launch_rows(kv4_read_kernel<64, false>, a, B, sms, 32, s);
}

}  // namespace qv
