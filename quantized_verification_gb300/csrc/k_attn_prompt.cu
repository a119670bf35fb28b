// k_attn_prompt.cu -- attention of many query rows on the tcgen05 tensor cores:
// whole prompts, packed one behind the other (causal), and the rows of a batch
// over a prefix that all its sequences share (partial results, merged by
// k_attn.cu's kernel with each sequence's own cache).
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = 2^(c s_rj - m_r),  s = q_r . k_j,
//   c = scale * log2 e, over the keys that row r sees.
//
// Rows. A query tile is 128 rows of one key/value head: the G query heads of
// each of 128 / G consecutive tokens (one TMA box of the qkv rows, heads inside
// tokens), so that any G fills it and a causal tile's diagonal is short. A CTA
// takes two neighbouring tiles over the same keys, or one where two would leave
// SMs idle.
// Packed prompts need no list of tiles: a tile of tokens that reaches over the end
// of a sequence runs over both sequences' keys, each row between its own limits.
//
// Roles: warps 0-3 and 4-7 form the softmax of a tile each (thread = row, the
// whole row of 128 scores in registers: no shuffles), the next warp's elected
// thread issues the products, the last one the TMA loads of keys and values,
// 128 positions each, into one ring. Per tile and 128 keys:
//   S = Q K^T      8 tcgen05.mma (D = 128), M = N = 128, both operands K-major
//                  in shared memory, the accumulator in tensor memory
//   P = 2^(cS-m)   rounded to bf16 over S's columns in tensor memory; the
//                  maximum m lags (up to 2^8), so that O is rarely rescaled; the
//                  rescaling is done by the softmax threads themselves, at a time
//                  when no product writes O
//   O += P V       8 tcgen05.mma, P from tensor memory, V as stored (M/N-major)
// With two tiles one's softmax runs under the other's products; with one tile S
// has two buffers.
// fp32 outputs: P as two bf16 parts (residue 2^-18), twice the second product;
// the tensor cores cut the accumulator off at every product (1.6e-8 of it, all
// one way), so every kFlush steps O is added in binary32 to the row's sums, which
// lie where the output goes.
//
// Masked tiles. A key that some row of the CTA does not see may hold anything;
// its score is replaced before use, and its value must not be multiplied by
// that row's 0. In tiles with such keys the values that are not finite are
// replaced by 0 in shared memory and noted; a row that does see one gets NaN.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace qv {

__device__ unsigned int g_attn_prompt_error;

namespace {

constexpr int kKeys = 128;                 // key positions per step
constexpr int kTileRows = 128;             // query rows per tile
constexpr int kFlush = 8;                  // steps O accumulates for fp32 outputs
constexpr float kLag = 8.0f;               // how far (log2) scores may rise above m
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT>
struct Layout {
    static constexpr int H = D / 64;                        // 128-byte halves of a row
    static constexpr int Tile = 128 * D * 2;                // bytes of 128 rows
    static constexpr int Stages = D == 128 ? (NT == 2 ? 5 : 6) : 8;
    static constexpr int Q = 0;
    static constexpr int Ring = NT * Tile;
    static constexpr int Bar = Ring + Stages * Tile;
    // barriers: full, empty [Stages], Q, S full [2], P full [2], PV done [2], scan joint, scan alone [2], drain
    static constexpr int bEmpty = Stages, bQ = 2 * Stages, bS = bQ + 1, bP = bS + 2, bPV = bP + 2, bJoint = bPV + 2,
                         bAlone = bJoint + 1, bDrain = bAlone + 2, kBars = bDrain + 1;
    static constexpr int Bad = Bar + (kBars + 1) / 2 * 16;             // keys with values that are not finite [3][4] words
    static constexpr int Misc = Bad + 3 * 16;               // tensor memory base, abort word
    static constexpr int Bytes = Misc + 16;
    static constexpr int Alloc = Bytes + 1024;              // slack to align the base to 1024 B
    // with two tiles the other warps fill a warpgroup, which hands registers over:
    // 384 threads of 168 become 256 of 208 and 128 of 88
    static constexpr int Threads = NT == 2 ? 384 : 192;
    // tensor memory columns: S (P over it) of both tiles or buffers, then O
    static constexpr int kO = 256;
    static constexpr int Cols = 512;
    static_assert(Bar % 8 == 0 && Bad % 16 == 0, "alignment");
    static_assert(Alloc <= (int)kMaxDynSmem, "shared memory budget");
};

struct Maps {
    CUtensorMap q, k, v;      // [rows][heads][D] bf16, boxes 64 x G x TM and 64 x 1 x 128
};

struct Args {
    const int32_t* cu;        // prompts: [B + 1] first rows; prefix: [1] its length
    int B;
    int M;                    // qkv rows
    int G, TM;                // query heads per key/value head, tokens per tile
    int Hkv, Hq;
    int k_head, v_head;       // head index of key/value head 0 in the k and v maps
    int P;                    // prefix: positions there is room for
    int blocks;               // prompts: groups of NT tiles; prefix: the same
    int splits;               // prefix: parts its positions are cut into
    float c;                  // scale * log2 e
    void* out;                // prompts: [M][Hq * D]
    float* part_o;            // prefix: [splits][M][Hq][D]
    float2* part_ml;          // prefix: [splits][M][Hq] (m, l)
    int hold;                 // test hook: request no load
    unsigned long long wait_ns;
};

__device__ __forceinline__ void umma_bf16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id,
                                             uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate) : "memory");
}
// Instruction descriptor of kind::f16 with bf16 operands, M = 128, f32
// accumulator; b_mn: B stored N-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
// Descriptor of V as the N-major B operand: atoms of 64 dims x 8 positions
// (128-byte swizzle), the next 8 positions 1024 bytes on, the next 64 dims
// `half` bytes on.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr, uint32_t half) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(half >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int head, int row,
                                            uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
                 :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
                    "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Two bf16 values, lo in the low half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

// A wait of at most limit_ns; false (and *abort set, the error noted) when it
// runs out, false at once when another wait has.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, unsigned parity, volatile int* abort,
                                          unsigned long long limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
        if (global_timer_ns() - t0 > limit_ns) {
            *abort = 1;
            atomicOr(&g_attn_prompt_error, kErrFullWait);
            return false;
        }
    }
}
// The same for a whole warp, which goes on or gives up as one.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, unsigned parity, volatile int* abort,
                                          unsigned long long limit_ns) {
    return __all_sync(0xffffffffu, lane_wait(bar, parity, abort, limit_ns));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The first row of the sequence that holds row tok (cu[0] <= tok < cu[B]), one
// per lane; the lanes' rows do not fall and span few sequences. The whole warp
// calls. Any values of cu stay in bounds: the result lies in [0, tok].
__device__ __forceinline__ int sequence_start(const int32_t* __restrict__ cu, int B, int tok) {
    const int lane = threadIdx.x & 31;
    const int tmin = __shfl_sync(0xffffffffu, tok, 0), tmax = __shfl_sync(0xffffffffu, tok, 31);
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int v = at < hi ? cu[at] : INT_MAX;
        const int n = __popc(__ballot_sync(0xffffffffu, v <= tmin));
        lo += (n > 0 ? n - 1 : 0) * step;
        hi = min(hi, lo + step);
    }
    int start = cu[lo];
    for (int base = lo + 1; tmax > tmin && base < B; base += 32) {
        const int v = base + lane < B ? cu[base + lane] : INT_MAX;
        for (int k = 0; k < 32; ++k) {
            const int b = __shfl_sync(0xffffffffu, v, k);
            if (b <= tok && b > start) start = b;
        }
        if (__shfl_sync(0xffffffffu, v, 31) > tmax) break;
    }
    return min(max(start, 0), tok);
}

// What a CTA does: tiles' first tokens and the key positions they run over.
struct Item {
    int kh, t0, split;
    int first, end;           // tokens [first, end) are rows to compute
    int k0, k1;               // prefix: the part's positions; prompts: k0 only
    int nt[2];                // steps of each tile
};

// The whole warp calls.
template <int NT, bool PREFIX>
__device__ __forceinline__ Item item_of(const Args& a, int item) {
    Item it;
    it.kh = item % a.Hkv;
    item /= a.Hkv;
    const int blk = item % a.blocks;
    it.split = item / a.blocks;
    // prompts: the last rows, which see most, first
    it.t0 = (PREFIX ? blk : a.blocks - 1 - blk) * (NT * a.TM);
    it.nt[0] = it.nt[1] = 0;
    if (PREFIX) {
        it.first = it.t0;
        it.end = min(it.t0 + NT * a.TM, a.M);
        const int len = min(max(a.cu[0], 0), a.P);
        const int tiles = (len + kKeys - 1) / kKeys, per = (tiles + a.splits - 1) / a.splits;
        it.k0 = min(it.split * per, tiles) * kKeys;
        it.k1 = min(len, it.k0 + per * kKeys);
        const int n = it.k1 > it.k0 ? (it.k1 - it.k0 + kKeys - 1) / kKeys : 0;
        it.nt[0] = n;
        if (NT == 2) it.nt[1] = it.t0 + a.TM < a.M ? n : 0;
    } else {
        const int c0 = min(max(a.cu[0], 0), a.M), cB = min(max(a.cu[a.B], 0), a.M);
        it.first = max(it.t0, c0);
        it.end = min(it.t0 + NT * a.TM, cB);
        it.k0 = it.k1 = 0;
        if (it.first < it.end) {
            it.k0 = sequence_start(a.cu, a.B, it.first);
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int e = min(it.t0 + (i + 1) * a.TM, it.end);
                if (e > max(it.t0 + i * a.TM, it.first)) it.nt[i] = (e - it.k0 + kKeys - 1) / kKeys;
            }
        }
    }
    return it;
}

template <int D, int NT, int PARTS, bool PREFIX>
__global__ void __launch_bounds__(Layout<D, NT>::Threads, 1)
attn_prompt_kernel(const __grid_constant__ Maps maps, const Args a) {
    using Ly = Layout<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Ly::Bar);
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + Ly::Bad);
    uint32_t* tmem_ptr = reinterpret_cast<uint32_t*>(smem + Ly::Misc);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + Ly::Misc + 4);
    constexpr int kMmaWarp = NT * 4, kLoadWarp = kMmaWarp + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < Ly::Stages; ++s) {
            mbar_init(&bar[s], 1);
            mbar_init(&bar[Ly::bEmpty + s], 1);
        }
        mbar_init(&bar[Ly::bQ], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar[Ly::bS + i], 1);
            mbar_init(&bar[Ly::bP + i], 4);
            mbar_init(&bar[Ly::bPV + i], 1);
            mbar_init(&bar[Ly::bAlone + i], 4);
        }
        mbar_init(&bar[Ly::bJoint], 8);
        mbar_init(&bar[Ly::bDrain], 1);
        for (int i = 0; i < 12; ++i) bad[i] = 0;
        *abort = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(tmem_ptr, Ly::Cols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tmem_ptr;
    allow_dependent_launch();
    grid_dependency_wait();
    const Item it = item_of<NT, PREFIX>(a, blockIdx.x);
    const int nmax = NT == 2 ? max(it.nt[0], it.nt[1]) : it.nt[0];

    if (warp >= kMmaWarp) {
    if (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kLoadWarp) {
        // -------------------------------------------------------------- loads
        if (lane == 0 && nmax > 0 && !a.hold) {
            prefetch_tensormap(&maps.q);
            prefetch_tensormap(&maps.k);
            prefetch_tensormap(&maps.v);
            mbar_arrive_expect_tx(&bar[Ly::bQ], (unsigned)(NT * Ly::H * 128 * a.G * a.TM));
            for (int i = 0; i < NT; ++i)
                for (int h = 0; h < Ly::H; ++h)
                    tma_load_3d(sbase + Ly::Q + i * Ly::Tile + h * 16384, &maps.q, 64 * h, it.kh * a.G, it.t0 + i * a.TM,
                                &bar[Ly::bQ]);
            int n = 0;                                       // loads requested: keys 0, values 0, keys 1, ...
            for (; n < 2 * nmax; ++n) {
                const int s = n % Ly::Stages, use = n / Ly::Stages;
                if (use > 0 && !lane_wait(&bar[Ly::bEmpty + s], (use - 1) & 1, abort, a.wait_ns)) break;
                mbar_arrive_expect_tx(&bar[s], Ly::Tile);
                const CUtensorMap* m = n & 1 ? &maps.v : &maps.k;
                const int head = (n & 1 ? a.v_head : a.k_head) + it.kh;
                for (int h = 0; h < Ly::H; ++h)
                    tma_load_3d(sbase + Ly::Ring + s * Ly::Tile + h * 16384, m, 64 * h, head, it.k0 + (n >> 1) * kKeys,
                                &bar[s]);
            }
            // no copy is in flight when the block ends
            const unsigned long long t0 = global_timer_ns();
            while (!mbar_try_wait(&bar[Ly::bQ], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
            for (int j = max(0, n - Ly::Stages); j < n; ++j)
                while (!mbar_try_wait(&bar[j % Ly::Stages], (j / Ly::Stages) & 1) && global_timer_ns() - t0 < 2 * kWaitLimitNs) {
                }
        }
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------- products
        if (lane == 0 && nmax > 0) {
            constexpr uint32_t id_s = idesc_bf16(kKeys, false), id_o = idesc_bf16(D, true);
            auto full = [&](int load) { return lane_wait(&bar[load % Ly::Stages], (load / Ly::Stages) & 1, abort, a.wait_ns); };
            auto scores = [&](int i, int load, int col) {
                const uint32_t q = sbase + Ly::Q + i * Ly::Tile, k = sbase + Ly::Ring + (load % Ly::Stages) * Ly::Tile;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_bf16_ss(tm + col, sw128_kmajor_desc(q + (kk >> 2) * 16384 + (kk & 3) * 32),
                                 sw128_kmajor_desc(k + (kk >> 2) * 16384 + (kk & 3) * 32), id_s, kk > 0);
            };
            auto outputs = [&](int i, int load, int col, bool add) {
                const uint32_t v = sbase + Ly::Ring + (load % Ly::Stages) * Ly::Tile;
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int kk = 0; kk < kKeys / 16; ++kk)
                        umma_f16_ta(tm + Ly::kO + i * D, tm + col + part * 64 + kk * 8, v_desc(v + kk * 2048, 16384), id_o,
                                    add || part > 0 || kk > 0);
            };
            auto release = [&](int load) { umma_commit(&bar[Ly::bEmpty + load % Ly::Stages]); };
            bool ok = lane_wait(&bar[Ly::bQ], 0, abort, a.wait_ns) && full(0);
            tc_fence_after();
            if (NT == 2) {
                if (ok) {
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        if (it.nt[i] > 0) {
                            scores(i, 0, i * 128);
                            umma_commit(&bar[Ly::bS + i]);
                        }
                    release(0);
                }
                for (int n = 0; ok && n < nmax; ++n) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        if (!ok || n >= it.nt[i]) continue;
                        const bool last = i == 1 || n >= it.nt[1];       // the last tile to use values n
                        ok = lane_wait(&bar[Ly::bP + i], n & 1, abort, a.wait_ns) && full(2 * n + 1);
                        if (!ok) break;
                        tc_fence_after();
                        outputs(i, 2 * n + 1, i * 128, PARTS == 2 ? n % kFlush != 0 : n > 0);
                        if (n == it.nt[i] - 1) umma_commit(&bar[Ly::bPV + i]);
                        if (last) release(2 * n + 1);
                        if (n + 1 < it.nt[i]) {
                            ok = full(2 * n + 2);
                            if (!ok) break;
                            scores(i, 2 * n + 2, i * 128);
                            umma_commit(&bar[Ly::bS + i]);
                            if (i == 1 || n + 1 >= it.nt[1]) release(2 * n + 2);
                        }
                    }
                }
            } else {
                if (ok) {
                    scores(0, 0, 0);
                    umma_commit(&bar[Ly::bS]);
                    release(0);
                }
                for (int n = 0; ok && n < nmax; ++n) {
                    if (n + 1 < nmax) {
                        ok = full(2 * n + 2);
                        if (!ok) break;
                        scores(0, 2 * n + 2, ((n + 1) & 1) * 128);
                        umma_commit(&bar[Ly::bS + ((n + 1) & 1)]);
                        release(2 * n + 2);
                    }
                    ok = lane_wait(&bar[Ly::bP], n & 1, abort, a.wait_ns) && full(2 * n + 1);
                    if (!ok) break;
                    tc_fence_after();
                    outputs(0, 2 * n + 1, (n & 1) * 128, PARTS == 2 ? n % kFlush != 0 : n > 0);
                    umma_commit(&bar[Ly::bPV]);
                    release(2 * n + 1);
                }
            }
            // nothing reads operands or writes tensor memory when the block ends
            umma_commit(&bar[Ly::bDrain]);
            const unsigned long long t0 = global_timer_ns();
            while (!mbar_try_wait(&bar[Ly::bDrain], 0) && global_timer_ns() - t0 < kWaitLimitNs) {
            }
        }
    }
    } else {
        // ------------------------------------------------------------ softmax
        if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        const int i = NT == 2 ? warp >> 2 : 0, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int tile_t0 = it.t0 + i * a.TM;
        const int tok = tile_t0 + r / a.G, head = it.kh * a.G + r % a.G;
        const bool valid = r < a.TM * a.G && tok >= it.first && tok < it.end;
        const int nt = NT == 2 && i == 1 ? it.nt[1] : it.nt[0];
        const int other = NT == 2 ? (i == 1 ? it.nt[0] : it.nt[1]) : 0;
        // keys [lo, hi] are seen by this row; tiles inside [all_lo, all_hi] by every row of the CTA
        int lo, hi, all_lo, all_hi;
        if (PREFIX) {
            lo = all_lo = it.k0;
            hi = all_hi = it.k1 - 1;
        } else if (nmax > 0) {
            lo = sequence_start(a.cu, a.B, min(max(tok, it.first), it.end - 1));
            hi = min(max(tok, it.first), it.end - 1);
            all_lo = sequence_start(a.cu, a.B, it.end - 1);
            all_hi = it.first;
        } else {
            lo = all_lo = 0;
            hi = all_hi = -1;
        }
        const size_t row = (size_t)tok * a.Hq + head;        // of the outputs
        float* acc = nullptr;                                // where the sums of fp32 outputs lie
        if (PREFIX)
            acc = a.part_o + ((size_t)it.split * a.M * a.Hq + row) * D;
        else if (PARTS == 2)
            acc = reinterpret_cast<float*>(a.out) + row * D;
        const uint32_t o_col = tm + lanes + Ly::kO + i * D;

        float m = neg_inf(), m_acc = neg_inf(), l = 0.f;
        bool ok = true;
        int masked = 0;                                      // tiles scanned
        unsigned joint = 0, alone = 0;
        // O added to the sums: o 1 (and what was there times 2^(m_acc - m), unless it is the first)
        auto flush = [&](bool fresh, float mul) {
            const float f = m_acc == neg_inf() ? 0.f : ex2(m_acc - m);
#pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
                uint32_t o[32];
                tmem_ld<32>(o_col + c0, o);
                tmem_ld_wait();
                if (valid) {
                    float4* p = reinterpret_cast<float4*>(acc + c0);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                        if (!fresh) w = p[j];
                        w.x = (w.x * f + __uint_as_float(o[4 * j])) * mul;
                        w.y = (w.y * f + __uint_as_float(o[4 * j + 1])) * mul;
                        w.z = (w.z * f + __uint_as_float(o[4 * j + 2])) * mul;
                        w.w = (w.w * f + __uint_as_float(o[4 * j + 3])) * mul;
                        p[j] = w;
                    }
                }
                __syncwarp();
            }
            m_acc = m;
        };

        for (int n = 0; n < nt; ++n) {
            const int buf = NT == 2 ? i : n & 1;
            ok = warp_wait(&bar[Ly::bS + buf], (NT == 2 ? n : n >> 1) & 1, abort, a.wait_ns);
            if (!ok) break;
            tc_fence_after();
            const uint32_t s_col = tm + lanes + buf * 128;
            uint32_t s[4][32];
#pragma unroll
            for (int q = 0; q < 4; ++q) tmem_ld<32>(s_col + 32 * q, s[q]);
            const int kb = it.k0 + n * kKeys;
            const bool part = kb < all_lo || kb + kKeys - 1 > all_hi;
            tmem_ld_wait();
            float poison = 0.f;
            if (part) {
                const int from = lo - kb, to = hi - kb;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (32 * q + j < from || 32 * q + j > to) s[q][j] = 0xFF800000u;
                // values that are not finite: 0 in shared memory, their keys noted
                const int load = 2 * n + 1;
                ok = warp_wait(&bar[load % Ly::Stages], (load / Ly::Stages) & 1, abort, a.wait_ns);
                if (!ok) break;
                const bool both = NT == 2 && n < other;
                uint32_t* mark = bad + (masked % 3) * 4;
                const uint32_t v = sbase + Ly::Ring + (load % Ly::Stages) * Ly::Tile;
                const int step = both ? 256 : 128;
                for (int e = both ? threadIdx.x : r; e < Ly::Tile / 16; e += step) {
                    uint32_t w[4];
                    lds_v4_u32(v + e * 16, w[0], w[1], w[2], w[3]);
                    bool any = false;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t h0 = w[j] & 0x7F80u, h1 = w[j] & 0x7F800000u;
                        if (h0 == 0x7F80u) w[j] &= 0xFFFF0000u, any = true;
                        if (h1 == 0x7F800000u) w[j] &= 0x0000FFFFu, any = true;
                    }
                    if (any) {
                        const int key = (e >> 3) & 127;      // 8 chunks a row; the halves one behind the other
                        sts_v4_u32(v + e * 16, w[0], w[1], w[2], w[3]);
                        atomicOr(&mark[key >> 5], 1u << (key & 31));
                    }
                }
                fence_proxy_async_smem();
                if (both) {
                    warp_arrive(&bar[Ly::bJoint]);
                    ok = warp_wait(&bar[Ly::bJoint], joint++ & 1, abort, a.wait_ns);
                } else {
                    warp_arrive(&bar[Ly::bAlone + i]);
                    ok = warp_wait(&bar[Ly::bAlone + i], alone++ & 1, abort, a.wait_ns);
                }
                if (!ok) break;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t b = mark[w];
                    if (b == 0) continue;
                    // the row's keys among these 32
                    const int f0 = max(from - 32 * w, 0), t0 = min(to - 32 * w, 31);
                    if (f0 <= t0 && f0 < 32 && (b >> f0 << f0 << (31 - t0)) != 0) poison = __uint_as_float(0x7FC00000u);
                }
                // the marks of the tile after the next: the tiles' larger count of steps clears them
                if (r == 0 && (nt > other || (nt == other && i == 0))) {
                    uint32_t* next = bad + ((masked + 2) % 3) * 4;
                    next[0] = next[1] = next[2] = next[3] = 0;
                }
                ++masked;
            }
            if (PARTS == 2 && n > 0 && n % kFlush == 0) {
                if (NT == 1) {                               // with two tiles S's barrier stands for it
                    ok = warp_wait(&bar[Ly::bPV], (n - 1) & 1, abort, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                }
                flush(n == kFlush, 1.f);
            }

            float mx0 = neg_inf(), mx1 = mx0, mx2 = mx0, mx3 = mx0;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                mx0 = fmaxf(mx0, __uint_as_float(s[0][j]));
                mx1 = fmaxf(mx1, __uint_as_float(s[1][j]));
                mx2 = fmaxf(mx2, __uint_as_float(s[2][j]));
                mx3 = fmaxf(mx3, __uint_as_float(s[3][j]));
            }
            const float top = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * a.c;
            const bool move = top > m + kLag || (m == neg_inf() && top > m);
            const float f = !move ? 1.f : (m == neg_inf() ? 0.f : ex2(m - top));
            if (move) m = top;
            l = l * f + poison;
            if (__any_sync(0xffffffffu, move) && n > 0 && !(PARTS == 2 && n % kFlush == 0)) {
                if (NT == 1) {
                    ok = warp_wait(&bar[Ly::bPV], (n - 1) & 1, abort, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                }
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld<32>(o_col + c0, o);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                    tmem_st_x32(o_col + c0, o);
                }
            }
            const float ms = m == neg_inf() ? 0.f : m;       // a row that has seen no key yet
            float l0 = 0.f, l1 = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint32_t hi2[16];
                uint32_t lo2[PARTS == 2 ? 16 : 1];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float p0 = ex2(fmaf(__uint_as_float(s[q][2 * j]), a.c, -ms));
                    const float p1 = ex2(fmaf(__uint_as_float(s[q][2 * j + 1]), a.c, -ms));
                    hi2[j] = pack2(p0, p1);
                    if (PARTS == 2) {
                        // the sum takes what the product takes
                        const float h0 = __uint_as_float(hi2[j] << 16), h1 = __uint_as_float(hi2[j] & 0xFFFF0000u);
                        lo2[j] = pack2(p0 - h0, p1 - h1);
                        l0 += h0 + __uint_as_float(lo2[j] << 16);
                        l1 += h1 + __uint_as_float(lo2[j] & 0xFFFF0000u);
                    } else {
                        l0 += p0;
                        l1 += p1;
                    }
                }
                tmem_st_x16(s_col + 16 * q, hi2);
                if constexpr (PARTS == 2) tmem_st_x16(s_col + 64 + 16 * q, lo2);
            }
            l += l0 + l1;
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&bar[Ly::bP + i]);
        }

        // ------------------------------------------------------------ outputs
        if (ok && nt > 0) {
            // (one tile: its last product but one may not have completed either)
            if (NT == 1 && nt > 1) ok = warp_wait(&bar[Ly::bPV], nt & 1, abort, a.wait_ns);
            ok = ok && warp_wait(&bar[Ly::bPV + i], NT == 2 ? 0 : (nt - 1) & 1, abort, a.wait_ns);
            tc_fence_after();
        }
        if (ok && nt > 0) {
            const float inv = PREFIX ? 1.f : 1.f / l;
            if (PREFIX || PARTS == 2) {
                flush(PARTS == 1 || nt <= kFlush, inv);
                if (PREFIX && valid) a.part_ml[(size_t)it.split * a.M * a.Hq + row] = make_float2(m, l);
            } else {
                uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + row * D);
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 32) {
                    uint32_t o[32];
                    tmem_ld<32>(o_col + c0, o);
                    tmem_ld_wait();
                    if (valid) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            uint4 w;
                            w.x = pack2(__uint_as_float(o[8 * j]) * inv, __uint_as_float(o[8 * j + 1]) * inv);
                            w.y = pack2(__uint_as_float(o[8 * j + 2]) * inv, __uint_as_float(o[8 * j + 3]) * inv);
                            w.z = pack2(__uint_as_float(o[8 * j + 4]) * inv, __uint_as_float(o[8 * j + 5]) * inv);
                            w.w = pack2(__uint_as_float(o[8 * j + 6]) * inv, __uint_as_float(o[8 * j + 7]) * inv);
                            p[c0 / 8 + j] = w;
                        }
                    }
                    __syncwarp();
                }
            }
        } else if (PREFIX && valid && nt == 0) {
            a.part_ml[(size_t)it.split * a.M * a.Hq + row] = make_float2(neg_inf(), 0.f);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tm, Ly::Cols);
    }
}

template <int D, int NT, int PARTS, bool PREFIX>
cudaError_t launch(const Maps& maps, const Args& a, int grid, cudaStream_t s) {
    using Ly = Layout<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(attn_prompt_kernel<D, NT, PARTS, PREFIX>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::Alloc);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(Ly::Threads);
    cfg.dynamicSmemBytes = Ly::Alloc;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_prompt_kernel<D, NT, PARTS, PREFIX>, maps, a);
}

template <bool PREFIX>
cudaError_t dispatch(const Maps& maps, const Args& a, int D, int nt, int parts, int grid, cudaStream_t s) {
#define QV_CASE(DV, NTV, PV) \
    if (D == DV && nt == NTV && parts == PV) return launch<DV, NTV, PV, PREFIX>(maps, a, grid, s);
    QV_CASE(128, 1, 1) QV_CASE(128, 1, 2) QV_CASE(128, 2, 1) QV_CASE(128, 2, 2)
    QV_CASE(64, 1, 1) QV_CASE(64, 1, 2) QV_CASE(64, 2, 1) QV_CASE(64, 2, 2)
#undef QV_CASE
    return cudaErrorInvalidValue;
}

// Tiles a CTA takes: two share every key tile they read and hide each other's
// softmax, one where two would leave SMs without work.
int tiles_per_cta(long long tiles, int Hkv, int sms) { return tiles * Hkv > sms ? 2 : 1; }

}  // namespace

int attention_prompt_tokens(int G) { return kTileRows / G; }

cudaError_t launch_attention_prompt(const CUtensorMap& q, const CUtensorMap& kv, const int32_t* cu, int B, int M, int Hq,
                                    int Hkv, int D, float scale, void* out, bool out_bf16, int sms, int hold,
                                    unsigned long long wait_ns, cudaStream_t s) {
    Maps maps;
    maps.q = q;
    maps.k = maps.v = kv;
    Args a = {};
    a.cu = cu; a.B = B; a.M = M;
    a.G = Hq / Hkv; a.TM = attention_prompt_tokens(a.G);
    a.Hkv = Hkv; a.Hq = Hq; a.k_head = Hq; a.v_head = Hq + Hkv;
    a.c = scale * kLog2e;
    a.out = out;
    a.hold = hold; a.wait_ns = wait_ns ? wait_ns : kWaitLimitNs;
    const int tiles = ceil_div(M, a.TM), nt = tiles_per_cta(tiles, Hkv, sms);
    a.blocks = ceil_div(tiles, nt);
    a.splits = 1;
    return dispatch<false>(maps, a, D, nt, out_bf16 ? 1 : 2, a.blocks * Hkv, s);
}

// The cut of a prefix of P positions under M rows: enough parts that every SM
// has one, of at least 4 steps where that leaves enough.
static void prefix_cut(int M, int Hq, int Hkv, int P, int sms, int* nt, int* blocks, int* splits) {
    const int TM = attention_prompt_tokens(Hq / Hkv), tiles = ceil_div(M, TM);
    *nt = tiles >= 2 ? 2 : 1;
    *blocks = ceil_div(tiles, *nt);
    const long long items = (long long)*blocks * Hkv;
    const int steps = ceil_div(P, kKeys);
    long long n = items >= sms ? 1 : sms / items;
    if (n > kPrefixMaxSplits) n = kPrefixMaxSplits;
    if (n > steps) n = steps;
    *splits = n < 1 ? 1 : (int)n;
}

size_t attention_prefix_workspace_bytes(int M, int Hq, int Hkv, int D, int P, int sms) {
    int nt, blocks, splits;
    prefix_cut(M, Hq, Hkv, P, sms, &nt, &blocks, &splits);
    return (size_t)splits * M * Hq * (D * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attention_prefix(const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v, const int32_t* len,
                                    int M, int Hq, int Hkv, int D, int P, float scale, bool exact, void* ws, int sms,
                                    int hold, unsigned long long wait_ns, PrefixParts* parts, cudaStream_t s) {
    Maps maps;
    maps.q = q;
    maps.k = k;
    maps.v = v;
    Args a = {};
    a.cu = len; a.B = 0; a.M = M;
    a.G = Hq / Hkv; a.TM = attention_prompt_tokens(a.G);
    a.Hkv = Hkv; a.Hq = Hq; a.P = P;
    a.c = scale * kLog2e;
    a.hold = hold; a.wait_ns = wait_ns ? wait_ns : kWaitLimitNs;
    int nt;
    prefix_cut(M, Hq, Hkv, P, sms, &nt, &a.blocks, &a.splits);
    a.part_o = static_cast<float*>(ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)a.splits * M * Hq * D);
    parts->o = a.part_o;
    parts->ml = reinterpret_cast<const float*>(a.part_ml);
    parts->splits = a.splits;
    return dispatch<true>(maps, a, D, nt, exact ? 2 : 1, a.blocks * Hkv * a.splits, s);
}

cudaError_t read_and_clear_attn_prompt_error(unsigned* code) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_prompt_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_prompt_error, &zero, sizeof(unsigned));
}

}  // namespace qv
