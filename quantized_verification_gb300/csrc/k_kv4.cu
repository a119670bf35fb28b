// k_kv4.cu -- key/value rows quantized to 4 bits as they are written into the
// paged cache, and cached positions read back as values.
//
//   Lower bit widths are the next step the Quasar summaries name
//   (gist.science/it, gist.science/de and gist.science/ja summaries, section
//   5); the cache keeps the a0 rule (symmetric, round half to even) with 7
//   for 127 and one scale for every 32 elements of a head's row, so that an
//   outlier channel costs its own 32 neighbours precision and no others.
//
// Both kernels move 8 elements a thread (16 bytes of bf16), four threads a
// scale group, consecutive threads on consecutive elements of a row: reads and
// writes of the wide side are whole lines, those of the code side whole
// sectors (64 bytes a head's row at D = 128). They are bound by memory at
// prompt lengths and by launch latency at a step's few rows.

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
    int T, rows, Hq, Hkv, NB, pages;
};

// The record position a (sequence, row) maps to, or false: rows past the
// sequence's count, positions outside the block table and pages outside the
// pool have none.
__device__ __forceinline__ bool locate(const Kv4Args& a, int row, int& page, int& slot) {
    const int b = row / a.T, j = row - b * a.T;
    if (a.count && j >= a.count[b]) return false;
    const long long pos = (long long)a.start[b] + j;
    if (pos < 0 || pos >= (long long)a.NB * kKv4Block) return false;
    page = kv4_page(a.table, b, a.NB, a.pages, (int)(pos / kKv4Block));
    slot = (int)(pos % kKv4Block);
    return page >= 0;
}

template <bool BF16>
__device__ __forceinline__ void load8(const uint8_t* p, float (&v)[8]) {
    if (BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 16);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
}

// The scale byte of a group whose largest magnitude is amax: the nearest scale
// to fl32(amax / 7), ties to the even byte. Rounding adds half of the last
// kept bit (and the kept bit itself, for ties) to the binary32 pattern.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
    const uint32_t u = __float_as_uint(__fdiv_rn(amax, 7.0f));
    const int b = (int)((u + 0x7FFFFu + ((u >> 20) & 1u)) >> 20) - 896;
    return (uint32_t)(b < 0 ? 0 : (b > 255 ? 255 : b));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kKv4Threads) kv4_write_kernel(const Kv4Args a) {
    using Rec = Kv4Rec<D>;
    allow_dependent_launch();
    grid_dependency_wait();
    const int ipr = 2 * a.Hkv * D / 8;                         // items of 8 elements per row
    const int item = blockIdx.y * blockDim.x + threadIdx.x;
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (item >= ipr || row >= a.rows) return;                  // whole groups of 4 threads
    float v[8];
    const size_t e0 = (size_t)row * (size_t)(a.Hq + 2 * a.Hkv) * D + (size_t)a.Hq * D + (size_t)item * 8;
    load8<BF16>(a.x + e0 * (BF16 ? 2 : 4), v);
    int page, slot;
    if (!locate(a, row, page, slot)) return;
    const int lane = (threadIdx.y * blockDim.x + threadIdx.x) & 31;
    const unsigned mask = 0xFu << (lane & ~3);
    // magnitudes are compared as bit patterns: infinities and NaN sort last
    uint32_t am = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    am = max(am, __shfl_xor_sync(mask, am, 1));
    am = max(am, __shfl_xor_sync(mask, am, 2));
    if (am >= 0x7F800000u) {                                   // rare: NaN counts as 0, infinities saturate
        am = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (isnan(v[i])) v[i] = 0.f;
            v[i] = fminf(fmaxf(v[i], -3.402823466e38f), 3.402823466e38f);
            am = max(am, __float_as_uint(v[i]) & 0x7FFFFFFFu);
        }
        am = max(am, __shfl_xor_sync(mask, am, 1));
        am = max(am, __shfl_xor_sync(mask, am, 2));
    }
    const uint32_t sb = scale_byte(__uint_as_float(am));
    const float s = kv4_scale(sb);
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(rintf(__fdiv_rn(v[i], s)), -7.f), 7.f);
        w |= ((uint32_t)(int)q & 15u) << (4 * i);
    }
    const int kv = item >= ipr / 2, rem = item - kv * (ipr / 2);
    const int h = rem / (D / 8), c = rem - h * (D / 8);
    uint8_t* rec = a.cache + ((size_t)page * a.Hkv + h) * Rec::Bytes;
    *reinterpret_cast<uint32_t*>(rec + (kv ? Rec::VC : Rec::KC) + slot * Rec::RowBytes + c * 4) = w;
    if ((c & 3) == 0) rec[(kv ? Rec::VS : Rec::KS) + slot * Rec::RowScales + (c >> 2)] = (uint8_t)sb;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kKv4Threads) kv4_read_kernel(const Kv4Args a) {
    using Rec = Kv4Rec<D>;
    allow_dependent_launch();
    grid_dependency_wait();
    const int ipr = 2 * a.Hkv * D / 8;
    const int item = blockIdx.y * blockDim.x + threadIdx.x;
    const int row = blockIdx.x * blockDim.y + threadIdx.y;
    if (item >= ipr || row >= a.rows) return;
    int page, slot;
    if (!locate(a, row, page, slot)) return;
    const int kv = item >= ipr / 2, rem = item - kv * (ipr / 2);
    const int h = rem / (D / 8), c = rem - h * (D / 8);
    const uint8_t* rec = a.cache + ((size_t)page * a.Hkv + h) * Rec::Bytes;
    const uint32_t w = *reinterpret_cast<const uint32_t*>(rec + (kv ? Rec::VC : Rec::KC) + slot * Rec::RowBytes + c * 4);
    const float s = kv4_scale(rec[(kv ? Rec::VS : Rec::KS) + slot * Rec::RowScales + (c >> 2)]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((int)(w << (28 - 4 * i)) >> 28) * s;   // exact: 7 significant bits
    const size_t e = (size_t)row * a.Hkv * D + (size_t)rem * 8;
    uint8_t* o = (kv ? a.v_out : a.k_out) + e * (BF16 ? 2 : 4);
    if (BF16) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __byte_perm(__float_as_uint(v[2 * i]), __float_as_uint(v[2 * i + 1]), 0x7632);
        *reinterpret_cast<uint4*>(o) = make_uint4(p[0], p[1], p[2], p[3]);
    } else {
        *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(o + 16) = make_float4(v[4], v[5], v[6], v[7]);
    }
}

template <class Kernel>
cudaError_t launch_rows(Kernel kernel, const Kv4Args& a, int D, cudaStream_t s) {
    const int ipr = 2 * a.Hkv * D / 8;                         // a multiple of 16
    const int bx = ipr < kKv4Threads ? ipr : kKv4Threads;
    const int by = kKv4Threads / bx;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ceil_div(a.rows, by), (unsigned)ceil_div(ipr, bx));
    cfg.blockDim = dim3((unsigned)bx, (unsigned)by);
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
                             uint8_t* cache, cudaStream_t s) {
    Kv4Args a = {};
    a.x = static_cast<const uint8_t*>(x);
    a.cache = cache; a.table = table; a.start = start; a.count = count;
    a.T = T; a.rows = B * T; a.Hq = Hq; a.Hkv = Hkv; a.NB = NB; a.pages = pages;
    if (D == 128) return bf16 ? launch_rows(kv4_write_kernel<128, true>, a, D, s) : launch_rows(kv4_write_kernel<128, false>, a, D, s);
    return bf16 ? launch_rows(kv4_write_kernel<64, true>, a, D, s) : launch_rows(kv4_write_kernel<64, false>, a, D, s);
}

cudaError_t launch_kv4_read(const uint8_t* cache, const int32_t* start, const int32_t* count, const int32_t* table,
                            int B, int T, int Hkv, int D, int NB, int pages, void* k_out, void* v_out, bool bf16,
                            cudaStream_t s) {
    Kv4Args a = {};
    a.k_out = static_cast<uint8_t*>(k_out); a.v_out = static_cast<uint8_t*>(v_out);
    a.cache = const_cast<uint8_t*>(cache); a.table = table; a.start = start; a.count = count;
    a.T = T; a.rows = B * T; a.Hkv = Hkv; a.NB = NB; a.pages = pages;
    if (D == 128) return bf16 ? launch_rows(kv4_read_kernel<128, true>, a, D, s) : launch_rows(kv4_read_kernel<128, false>, a, D, s);
    return bf16 ? launch_rows(kv4_read_kernel<64, true>, a, D, s) : launch_rows(kv4_read_kernel<64, false>, a, D, s);
}

}  // namespace qv
