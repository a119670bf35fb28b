// k_rotary.cu -- rotary positions of the query and key heads of qkv rows.
//
//   For a head x of row t (after an optional RMS norm, x gamma / sqrt(mean x^2
//   + eps)) and each rotated pair i of its values (a, b):
//     (a, b) -> (a c - b s, b c + a s),
//     c, s = magnitude * cos, sin of pos[t] * freq[i],
//   with the angle's product not rounded: in binary32 it would be off by 2^-24 of
//   itself, 0.004 at position 65536. Here a frequency becomes a 64-bit fraction
//   of a turn, the position multiplies it modulo 2^64 (whole turns fall off by
//   themselves), and only the result's top 32 bits are converted, so that an
//   angle is off by 2^-25 turns at most at any int32 position.
//
// Bound by memory: a row is read and written once. A block takes one or
// kTokens tokens, forms their cosines and sines once for all heads in shared
// memory, then a group of lanes takes a head: a lane holds two vectors whose
// values pair up (i and i + rot / 2, or neighbours), so that the rotation needs no
// exchange and the norm a few shuffles.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace qv {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxRot = 256;
constexpr int kTokens = 4;

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
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void pack(const float* x, uint4& v) {
    v = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
}
__device__ __forceinline__ void pack(const float* x, uint2& v) { v = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3])); }
__device__ __forceinline__ void pack(const float* x, float4& v) { v = make_float4(x[0], x[1], x[2], x[3]); }

// V: a lane's vector of VEC values. GS: lanes of a head (a power of two), of
// which D / (2 VEC) have values. TB: tokens of a block.
template <typename V, int VEC, int TB>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int GS, int heads) {
    __shared__ float2 cs[TB][kMaxRot / 2];
    const int t0 = blockIdx.x * TB, nt = min(TB, a.M - t0), half = a.rot / 2;
    allow_dependent_launch();
    grid_dependency_wait();
    for (int e = threadIdx.x; e < nt * half; e += kThreads) {
        const int t = e / half, i = e - t * half;
        const int64_t turn = (int64_t)(turns_of(a.freq[i]) * (uint64_t)(int64_t)a.pos[t0 + t]);
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);
        cs[t][i] = make_float2(c * a.magnitude, s * a.magnitude);
    }
    __syncthreads();

    const int group = threadIdx.x / GS, u = threadIdx.x & (GS - 1);
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
    const size_t W = (size_t)(a.Hq + 2 * a.Hkv) * a.D;
    const int wh = 32 / GS, last = (heads + wh - 1) / wh * wh;  // a warp's heads run together
    for (int t = 0; t < nt; ++t) {
        float c[VEC], s[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float2 v = rotated ? cs[t][VEC * u + i] : make_float2(1.f, 0.f);
            c[i] = v.x;
            s[i] = v.y;
        }
        const V* x = static_cast<const V*>(a.x);
        V* out = static_cast<V*>(a.out);
        const size_t row = (size_t)(t0 + t) * W;
        for (int h = blockIdx.y * (kThreads / GS) + group; h < last; h += gridDim.y * (kThreads / GS)) {
            const bool in = there && h < heads;
            const size_t pa = (row + (size_t)h * a.D + oa) / VEC, pb = (row + (size_t)h * a.D + ob) / VEC;
            V va{}, vb{};
            if (in) {
                va = x[pa];
                vb = x[pb];
            }
            if (h >= a.Hq + a.Hkv) {                          // a value head: copied
                if (in) {
                    out[pa] = va;
                    out[pb] = vb;
                }
                if (a.q_gamma == nullptr) continue;
            }
            float p[VEC], q[VEC];
            unpack(va, p);
            unpack(vb, q);
            if (a.q_gamma) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < VEC; ++i) ss += p[i] * p[i] + q[i] * q[i];
                for (int o = GS / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                const float r = __frcp_rn(__fsqrt_rn(ss / (float)a.D + a.eps));
                const uint16_t* g = h < a.Hq ? a.q_gamma : a.k_gamma;
                if (in) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        p[i] = p[i] * r * __uint_as_float((uint32_t)g[oa + i] << 16);
                        q[i] = q[i] * r * __uint_as_float((uint32_t)g[ob + i] << 16);
                    }
                }
            }
            if (!in || h >= a.Hq + a.Hkv) continue;
            float y[VEC], z[VEC];
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    y[2 * i] = p[2 * i] * c[i] - p[2 * i + 1] * s[i];
                    y[2 * i + 1] = p[2 * i + 1] * c[i] + p[2 * i] * s[i];
                    z[2 * i] = q[2 * i] * c[VEC / 2 + i] - q[2 * i + 1] * s[VEC / 2 + i];
                    z[2 * i + 1] = q[2 * i + 1] * c[VEC / 2 + i] + q[2 * i] * s[VEC / 2 + i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    y[i] = p[i] * c[i] - q[i] * s[i];
                    z[i] = q[i] * c[i] + p[i] * s[i];
                }
            }
            pack(y, va);
            pack(z, vb);
            out[pa] = va;
            out[pb] = vb;
        }
    }
}

template <typename V, int VEC, int TB>
cudaError_t launch(const RotaryArgs& a, int GS, int heads, int parts, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ceil_div(a.M, TB), parts);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotary_kernel<V, VEC, TB>, a, GS, heads);
}

template <typename V, int VEC>
cudaError_t by_tokens(const RotaryArgs& a, int sms, cudaStream_t s) {
    int GS = 1;
    while (GS < a.D / (2 * VEC)) GS *= 2;
    const int heads = a.Hq + (a.out == a.x ? 1 : 2) * a.Hkv;
    // few rows: a head per group, so that the heads of a row are in flight at once
    if (a.M < 4 * sms) return launch<V, VEC, 1>(a, GS, heads, ceil_div(heads, kThreads / GS), s);
    return launch<V, VEC, kTokens>(a, GS, heads, 1, s);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool bf16, int sms, cudaStream_t s) {
    if (!bf16) return by_tokens<float4, 4>(a, sms, s);
    if (a.rot % 16 == 0 && a.D % 16 == 0) return by_tokens<uint4, 8>(a, sms, s);
    return by_tokens<uint2, 4>(a, sms, s);
}

}  // namespace qv
