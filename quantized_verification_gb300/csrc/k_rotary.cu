// k_rotary.cu -- rotary positions of the query and key heads of qkv rows.
//
//   For a head x of row t (after an optional RMS norm, x gamma / sqrt(mean x^2
//   + eps)) and each rotated pair i of its values (a, b):
//     (a, b) -> (a c - b s, b c + a s),
//     c, s = magnitude * cos, sin of pos[t] * freq[i],
//   with the angle's product not rounded: in binary32 it would be off by 2^-24 of
//   itself, 0.004 at position 65536. Here a frequency becomes a 64-bit fraction
//   of a turn, the position multiplies it modulo 2^64 (whole turns fall off by
//   themselves), and only the result's top 32 bits are converted (half a step of
//   binary32, 2^-26 turns). The fraction is off by 2^-62 of the frequency in turns
//   at most: by 2^-26 turns at the farthest int32 position for frequencies up to 32,
//   in proportion above.
//
// Bound by memory: a row is read and written once. A warp takes a row (or, of few
// rows, some of its heads): it forms the row's cosines and sines once, two or so a
// lane, then a group of lanes takes a head at a time: a lane holds two vectors whose
// values pair up (i and i + rot / 2, or neighbours), so that the rotation needs no
// exchange and the norm a few shuffles; what a lane needs of the row stays in its
// registers from head to head. Several heads are requested ahead. GB300: 16001 rows
// of 32/8 heads of 128, bf16, normed, copied to another buffer, 70 us = 5.6 TB/s
// (0.83 of the measured copy bandwidth; a block for four rows with a shared table 78
// us); 2043 rows of 12/4 heads of 64, fp32, 6.5 us; 5 rows 2.7 us.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace qv {
namespace {

constexpr int kWarps = 4;                  // of a block
constexpr int kMaxRot = 256;

// freq / (2 pi) as a fraction of 2^64, whole turns dropped.
__device__ __forceinline__ uint64_t turns_of(float freq) {
    constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;     // 2^64 / (2 pi)
    const uint32_t b = __float_as_uint(freq);
    const int e = (int)(b >> 23 & 255u);
    const uint64_t mant = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
    const int shift = (e ? e : 1) - 126;                      // freq = mant * 2^-24 * 2^shift
    uint64_t t = __umul64hi(mant << 40, kInvTwoPi);
    t = shift <= -64 || shift >= 64 ? 0 : shift < 0 ? t >> -shift : t << shift;
    return b >> 31 ? 0 - t : t;
}

template <typename V>
__device__ __forceinline__ void unpack(const V& v, float* x);
template <>
__device__ __forceinline__ void unpack<uint4>(const uint4& v, float* x) {       // 8 bf16
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void unpack<uint2>(const uint2& v, float* x) {       // 4 bf16
    const uint32_t w[2] = {v.x, v.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
template <>
__device__ __forceinline__ void unpack<float4>(const float4& v, float* x) {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void pack(const float* x, uint4& v) {
    v = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void pack(const float* x, uint2& v) { v = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3])); }
__device__ __forceinline__ void pack(const float* x, float4& v) { v = make_float4(x[0], x[1], x[2], x[3]); }

// V: a lane's vector of VEC values. GS: lanes of a head (a power of two), of
// which D / (2 VEC) have values. parts: pieces a row's heads are cut into.
template <typename V, int VEC, int kAhead>
__global__ void __launch_bounds__(kWarps * 32) rotary_kernel(const RotaryArgs a, int GS, int heads, int parts) {
    __shared__ float2 tables[kWarps][kMaxRot / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long job = (long long)blockIdx.x * kWarps + warp;
    const int row = (int)(job / parts), part = (int)(job - (long long)row * parts), half = a.rot / 2;
    allow_dependent_launch();
    if (row >= a.M) return;
    const int group = lane / GS, u = lane & (GS - 1), wide = 32 / GS;      // heads a warp takes at a time
    const int nr = a.rot / (2 * VEC), units = a.D / (2 * VEC);
    const bool rotated = u < nr, there = u < units;
    int oa, ob;                                               // the lane's two vectors
    if (rotated && !a.interleaved) {
        oa = VEC * u;
        ob = half + VEC * u;
    } else {                                                  // neighbours, rotated or not
        oa = 2 * VEC * u;
        ob = oa + VEC;
    }
    grid_dependency_wait();
    float2* cs = tables[warp];
    {
        const uint64_t pos = (uint64_t)(int64_t)a.pos[row];
        for (int i = lane; i < half; i += 32) {
            float s, c;
            sincospif((float)(int32_t)((turns_of(a.freq[i]) * pos) >> 32) * 0x1p-31f, &s, &c);
            cs[i] = make_float2(c * a.magnitude, s * a.magnitude);
        }
        __syncwarp();
    }
    uint64_t c2[VEC / 2], s2[VEC / 2];                        // cosines and sines of the lane's pairs, two by two
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
        const float2 v0 = rotated ? cs[VEC * u + 2 * i] : make_float2(1.f, 0.f);
        const float2 v1 = rotated ? cs[VEC * u + 2 * i + 1] : make_float2(1.f, 0.f);
        c2[i] = pair(v0.x, v1.x);
        s2[i] = pair(v0.y, v1.y);
    }
    const float inv_d = 1.f / (float)a.D;
    const V* x = static_cast<const V*>(a.x) + (size_t)row * (a.Hq + 2 * a.Hkv) * (a.D / VEC);
    V* out = static_cast<V*>(a.out) + (size_t)row * (a.Hq + 2 * a.Hkv) * (a.D / VEC);
    const int last = (heads + wide - 1) / wide * wide, stride = parts * wide;
    for (int h0 = part * wide + group; h0 < last; h0 += kAhead * stride) {
        V va[kAhead], vb[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + k * stride;
            va[k] = V{};
            vb[k] = V{};
            if (there && h < heads) {
                va[k] = x[(h * a.D + oa) / VEC];
                vb[k] = x[(h * a.D + ob) / VEC];
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int h = h0 + k * stride;
            if (h - group >= last) break;                     // (the warp's heads run together)
            const bool in = there && h < heads, value = h >= a.Hq + a.Hkv;   // value heads: copied
            float px[VEC], qx[VEC];
            unpack(va[k], px);
            unpack(vb[k], qx);
            uint64_t p[VEC / 2], q[VEC / 2];
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i) {
                p[i] = pair(px[2 * i], px[2 * i + 1]);
                q[i] = pair(qx[2 * i], qx[2 * i + 1]);
            }
            if (a.q_gamma) {
                uint64_t ss = mul2(p[0], p[0]);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    if (i > 0) ss = fma2(p[i], p[i], ss);
                    ss = fma2(q[i], q[i], ss);
                }
                float sum, odd;
                unpair(ss, sum, odd);
                sum += odd;
                for (int o = GS / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                const float r = rsqrtf(sum * inv_d + a.eps);
                const uint64_t r2 = pair(r, r);
                const uint16_t* g = h < a.Hq ? a.q_gamma : a.k_gamma;
                if (in && !value) {
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        const uint32_t ga = reinterpret_cast<const uint32_t*>(g + oa)[i];
                        const uint32_t gb = reinterpret_cast<const uint32_t*>(g + ob)[i];
                        p[i] = mul2(p[i], mul2(r2, pair(__uint_as_float(ga << 16), __uint_as_float(ga & 0xFFFF0000u))));
                        q[i] = mul2(q[i], mul2(r2, pair(__uint_as_float(gb << 16), __uint_as_float(gb & 0xFFFF0000u))));
                    }
                }
            }
            if (!in) continue;
            if (!value) {
                float y[VEC], z[VEC];
                if (a.interleaved) {
                    float c[VEC], s[VEC], pv[VEC], qv[VEC];
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        unpair(c2[i], c[2 * i], c[2 * i + 1]);
                        unpair(s2[i], s[2 * i], s[2 * i + 1]);
                        unpair(p[i], pv[2 * i], pv[2 * i + 1]);
                        unpair(q[i], qv[2 * i], qv[2 * i + 1]);
                    }
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        y[2 * i] = pv[2 * i] * c[i] - pv[2 * i + 1] * s[i];
                        y[2 * i + 1] = pv[2 * i + 1] * c[i] + pv[2 * i] * s[i];
                        z[2 * i] = qv[2 * i] * c[VEC / 2 + i] - qv[2 * i + 1] * s[VEC / 2 + i];
                        z[2 * i + 1] = qv[2 * i + 1] * c[VEC / 2 + i] + qv[2 * i] * s[VEC / 2 + i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < VEC / 2; ++i) {
                        // (the sign goes into a product's operand: a packed subtraction is an addition)
                        const uint64_t minus = q[i] ^ 0x8000000080000000ull;
                        unpair(fma2(minus, s2[i], mul2(p[i], c2[i])), y[2 * i], y[2 * i + 1]);
                        unpair(fma2(p[i], s2[i], mul2(q[i], c2[i])), z[2 * i], z[2 * i + 1]);
                    }
                }
                pack(y, va[k]);
                pack(z, vb[k]);
            }
            out[(h * a.D + oa) / VEC] = va[k];
            out[(h * a.D + ob) / VEC] = vb[k];
        }
    }
}

template <typename V, int VEC, int kAhead>
cudaError_t launch(const RotaryArgs& a, int GS, int heads, int parts, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ceil_div((long long)a.M * parts, kWarps));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotary_kernel<V, VEC, kAhead>, a, GS, heads, parts);
}

template <typename V, int VEC>
cudaError_t by_rows(const RotaryArgs& a, int sms, cudaStream_t s) {
    int GS = 1;
    while (GS < a.D / (2 * VEC)) GS *= 2;
    const int heads = a.Hq + (a.out == a.x ? 1 : 2) * a.Hkv;
    // few rows: a warp for every 32 / GS heads, so that all heads of a row are in flight at once. 32/8 heads of
    // 128, normed, so against a warp a row: 5 rows 2.7 and 7.5 us, 300 rows 4.2 and 7.6, 1000 rows 9.0 and 10.1,
    // 2043 rows 17.6 and 12.9
    if (a.M < 8 * sms) return launch<V, VEC, 1>(a, GS, heads, ceil_div(heads, 32 / GS), s);
    return launch<V, VEC, 4>(a, GS, heads, 1, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, int sms, cudaStream_t s) {
    if (!bf16) return by_rows<float4, 4>(a, sms, s);
    if (a.rot % 16 == 0 && a.D % 16 == 0) return by_rows<uint4, 8>(a, sms, s);
    return by_rows<uint2, 4>(a, sms, s);
}

}  // namespace qv
