// attn_kv4_common.cuh -- what the two kernels of attention over the 4-bit cache
// share (k_attn_kv4.cu on mma.sync; k_attn_kv4_tc.cu on tcgen05, for heads of 128
// values and long contexts): the arguments, the cut of the work into places,
// the unpacking of codes, and the waits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kv4_common.cuh"
#include "qv.h"
#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace qv {
namespace kv4attn {

constexpr int kRowTile = 32;                    // query rows of a tile
constexpr int kMinUnits = 16;                   // places of a CTA's range at least: two units a warp
constexpr int kAttnMaxT = QV_MAX_M;             // tokens of a step
constexpr size_t kCounterBytes = 4096;         // at the workspace's start, whatever the shape
constexpr int kJoinSlots = (int)(kCounterBytes / 12);   // three arrays of counters; also the most CTAs
constexpr unsigned kJoinAll = 32;               // parts of a tile that are joined at once (Join)
constexpr unsigned kJoinFan = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTileCost = 20;                   // units' worth of a tile's own costs
constexpr int kMaxCluster = 8;                  // CTAs of a cluster that share a tile
constexpr int kClusterUnits = 6;                // a larger cluster while its CTAs have more units than this
constexpr int kClusterMost = 48;                // no clusters above so many units a CTA
constexpr int kAloneMost = 40;                  // units of a tile that has a CTA to itself, though not all fit at once
constexpr int kTcMinUnits = 8;                  // the same for the tcgen05 kernel: two steps of 128 positions,
constexpr int kTcTileCost = 18;                 // and a tile's costs
constexpr float kLazy = 8.f;                    // log2 of the growth a running maximum may lag behind
constexpr float kBias = 7.f;                    // log2 of p at the running maximum: 2^(kBias + kLazy + 0.5) < 65504

// A row's running maximum moves to product v: c, with p = 2^(sl2 x + c) for a
// product x, and the product at which it moves next. Up to |m| = 2^20 the
// roundings of sl2 x + c and of the limit stay below 2^-1, and p in f16's
// range (65504). Above, the last bit of sl2 x nears 1 and more: no lag, no bias (-m is
// exact), and p <= 2^8 as long as m's last bit is 16 at most. From 2^27 on the
// scores hold no information that fp32 keeps: the row becomes NaN. m stays above
// -2^27: scores below that have p = 0 next to any others, and a row with no
// others ends as 0 / 0.
struct RowMax {
    float c, limit;
    __device__ __forceinline__ RowMax(float v, float sl2) {
        const float m = fmaxf(rintf(v * sl2), -134217728.f);
        if (fabsf(m) < 1048576.f) {
            c = kBias - m;
            // (2 ulp: p < 2^15.5 all the same; by quarters, since __fdividef is 0 for
            // divisors above 2^126, and sl2 may be up to 2^127.8)
            limit = __fdividef(0.25f * (m + kLazy), 0.25f * sl2);
        } else {
            c = m < 134217728.f ? -m : __uint_as_float(0x7FC00000u);
            limit = v;
        }
    }
};

struct Args {
    const uint16_t* qkv;       // [B*T][(Hq + 2 Hkv) D] bf16
    const uint8_t* cache;
    const int32_t* table;      // [B][NB] or null
    const int32_t* len;        // [B]
    int B, T, Hq, Hkv, G, NB, pages;
    int RT, rows;              // row tiles per head group, query rows per row tile
    int C;                     // CTAs of the cluster that takes a tile, or 0: the line of units
    float scale;
    void* out;                 // [B*T][Hq D] fp32 or bf16
    unsigned* counters;        // arrivals (Join), zero between calls
    float* partials;           // [grid][2][slot]
    int hold;                  // test hook: request no record
    unsigned long long wait_ns;
};

__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// {lo, hi} rounded to bf16.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// (a & b) ^ c
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0x6A;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hfma2_f16(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2_f16(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// {lo, hi} rounded to f16.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float2 unpack_f16x2(uint32_t x) {
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(lo), "=f"(hi) : "r"(x));
    return make_float2(lo, hi);
}

// A key scale as a bf16 pair, and -24 and -136 times it (exact: 2 + 4 and 4 + 4 bits).
struct KeyScale {
    uint32_t s, off;
    __device__ __forceinline__ KeyScale() {}
    __device__ __forceinline__ explicit KeyScale(uint32_t b) {
        s = b * 0x00100010u + 0x38003800u;
        off = hmul2_bf16(s, 0xC1C0C1C0u);                 // -24.0
    }
};
// Nibbles J of the two 16-bit halves of x as bf16 values q * s: shifted to bits
// 3..6 with the sign bit flipped, under 16.0 (0x4180), a nibble is 24 + q.
// Left shifts are multiplications by a register (the FMA pipe has room, the
// ALU, which does the masking and the right shifts, is the busiest pipe). Low:
// the lowest nibble stays where it is, under 128.0 (0x4300), as 136 + q; one
// instruction less for one register more a scale.
template <int J, bool Low>
__device__ __forceinline__ uint32_t key_pair(uint32_t x, const KeyScale& sc, uint32_t eight) {
    if constexpr (Low && J == 0)
        return hfma2_bf16(and_xor(x, 0x000F000Fu, 0x43084308u), sc.s, hmul2_bf16(sc.s, 0xC308C308u));   // -136.0
    const uint32_t y = J == 0 ? x * eight : x >> (J == 0 ? 0 : 4 * J - 3);
    return hfma2_bf16(and_xor(y, 0x00780078u, 0x41C041C0u), sc.s, sc.off);
}
// The value scales of two positions times 2^-6 as an f16 pair, and -24 times them.
struct ValScale {
    uint32_t s, off;
    __device__ __forceinline__ ValScale() {}
    __device__ __forceinline__ ValScale(uint32_t b_lo, uint32_t b_hi) {
        s = pack_f16x2(__uint_as_float((b_lo << 20) + (106u << 23)), __uint_as_float((b_hi << 20) + (106u << 23)));
        off = hmul2_f16(s, 0xCE00CE00u);                  // -24.0
    }
};
// The same in f16: bits 6..9 under 16.0 (0x4C00).
template <int J>
__device__ __forceinline__ uint32_t val_pair(uint32_t x, const ValScale& sc, uint32_t four, uint32_t sixty4) {
    const uint32_t y = J == 0 ? x * sixty4 : (J == 1 ? x * four : x >> (J < 2 ? 0 : 4 * J - 6));
    return hfma2_f16(and_xor(y, 0x03C003C0u, 0x4E004E00u), sc.s, sc.off);
}

// A thread's code words and scales of two key rows.
template <int W>
struct Keys {
    uint32_t x[2][W];
    KeyScale sc[2];
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, unsigned bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ bool bar_wait(uint64_t* bar, unsigned parity, volatile int* abort,
                                         unsigned long long limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (*abort) return false;
        if (mbar_try_wait(bar, parity)) return true;
        if (global_timer_ns() - t0 > limit_ns) {
            *abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}
__device__ __forceinline__ uint32_t lds_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

// How the parts of a tile, those of CTAs c0 .. c0 + n - 1, are joined: by the
// last CTA to arrive, or, above kJoinAll, in groups of about kJoinFan by the
// last of each group, which leaves the sum in its first part's place, and the
// groups by the last of those. Groups follow from n alone: the same sums from
// call to call. GB300, one sequence of 131071 positions, 1 key/value head, 5
// tokens of 4 heads: 304 parts in one go 149 us, in groups 37 us;
// one token 36 and 18 us. Up to 32 parts one join is as fast as two.
// In shared memory, kept by one thread: registers are dear.
struct Join {
    unsigned c0, groups, size;
    unsigned first, count, step;                // the present join's parts: first, first + step, ..
    unsigned last;                              // this CTA is the last of them to arrive
    __device__ __forceinline__ void begin(unsigned c0_, unsigned c1) {
        const unsigned n = c1 - c0_ + 1;
        c0 = c0_;
        groups = n <= kJoinAll ? 1 : (n + kJoinFan - 1) / kJoinFan;
        size = (n + groups - 1) / groups;
        groups = (n + size - 1) / size;
        const unsigned g = (blockIdx.x - c0) / size;
        first = c0 + g * size;
        count = min(size, n - g * size);
        step = 1;
    }
    // This CTA's part is written. A tile's first group may begin where another
    // tile's later group does, hence three arrays of counters.
    __device__ __forceinline__ void arrive(unsigned* counters) {
        unsigned* counter = counters + (step != 1 ? 2 * kJoinSlots + c0 : (first == c0 ? c0 : kJoinSlots + first));
        __threadfence();
        last = atomicAdd(counter, 1u) == count - 1;
        if (last) {
            *counter = 0;
            __threadfence();
        }
    }
    __device__ __forceinline__ bool final() const { return groups == 1 || step != 1; }
    __device__ __forceinline__ void next() {
        first = c0;
        count = groups;
        step = size;
    }
};

// The cached positions of sequence b.
__device__ __forceinline__ int seq_len(const Args& a, int b) {
    const long long cap = (long long)a.NB * kKv4Block;
    const int n = a.len[b];
    return n < 0 ? 0 : ((long long)n > cap ? (int)cap : n);
}

// A CTA's range of the line of places: every tile (b, kh, rt) takes its units
// and `cost` more, sequence by sequence.
struct Range {
    unsigned u0, u1;           // this CTA's places
    unsigned per;              // places of a CTA
    unsigned seq_at;           // where the places of sequence b, the first of the range, begin
    int b;
};
// All threads of the CTA call it; s_scan holds 16 words. False: nothing to do.
template <int Threads>
__device__ __forceinline__ bool find_range(const Args& a, int own_units, int cost, int min_units, unsigned* s_scan,
                                           Range& g) {
    static_assert(Threads / 32 <= 14, "s_scan");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tps = a.Hkv * a.RT;                              // tiles of a sequence
    if (a.B <= 32) {                                           // each warp for itself: nothing to wait for
        unsigned mine = 0;
        if (lane < a.B) mine = (unsigned)(((seq_len(a, lane) + kKv4Block - 1) / kKv4Block + own_units + cost) * tps);
        unsigned incl = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const unsigned v = __shfl_up_sync(0xffffffffu, incl, off);
            if (lane >= off) incl += v;
        }
        const unsigned total = __shfl_sync(0xffffffffu, incl, 31);
        g.per = max((total + gridDim.x - 1) / gridDim.x, (unsigned)min_units);
        g.u0 = g.per * blockIdx.x;
        g.u1 = min(total, g.u0 + g.per);
        if (g.u0 >= g.u1) return false;
        g.b = __ffs(__ballot_sync(0xffffffffu, incl > g.u0)) - 1;   // the first sequence that ends behind u0
        g.seq_at = __shfl_sync(0xffffffffu, incl - mine, g.b);
        return true;
    }
    const int seg = (a.B + Threads - 1) / Threads;             // sequences per thread
    unsigned mine = 0;
    for (int b = tid * seg; b < min(a.B, (tid + 1) * seg); ++b)
        mine += (unsigned)(((seq_len(a, b) + kKv4Block - 1) / kKv4Block + own_units + cost) * tps);
    unsigned incl = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const unsigned v = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += v;
    }
    if (lane == 31) s_scan[warp] = incl;
    __syncthreads();
    unsigned before = incl - mine, total = 0;
#pragma unroll
    for (int w = 0; w < Threads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    g.per = max((total + gridDim.x - 1) / gridDim.x, (unsigned)min_units);
    g.u0 = g.per * blockIdx.x;
    g.u1 = min(total, g.u0 + g.per);
    if (g.u0 >= g.u1) return false;                            // (the whole CTA)
    if (g.u0 >= before && g.u0 < before + mine) {              // exactly one thread
        unsigned at = before;
        int b = tid * seg;
        while (true) {
            const unsigned n = (unsigned)(((seq_len(a, b) + kKv4Block - 1) / kKv4Block + own_units + cost) * tps);
            if (g.u0 < at + n) break;
            at += n;
            ++b;
        }
        s_scan[14] = at;
        s_scan[15] = (unsigned)b;
    }
    __syncthreads();
    g.seq_at = s_scan[14];
    g.b = (int)s_scan[15];
    return true;
}

}  // namespace kv4attn

// k_attn_kv4_tc.cu
cudaError_t launch_attn_kv4_tc(const kv4attn::Args& a, int NR, bool out_bf16, int grid, int tile_cost, int min_units,
                               cudaStream_t s);
cudaError_t read_and_clear_attn_kv4_tc_error(unsigned* code);

}  // namespace qv
