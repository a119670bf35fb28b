// k_attn_kv4.cu -- attention of the verify tokens over a 4-bit paged KV cache.
//
//   The attention of k_attn.cu (causal grouped-query scaled dot-product
//   attention; the non-GEMM computation of the layer stays in high precision:
//   Quasar, gist.science/ja summary, section 2.2 item 3) with the cache of
//   kv4_common.cuh in place of the bf16 one: 4.25 bits per cached element
//   instead of 16. The step's own keys and values are the bf16 rows of the
//   qkv projection, unrounded.
//
// Work split. A tile is one (sequence, key/value head, group of at most 32 of
// its T * Hq/Hkv query rows); a unit is one record of 32 cached positions, or
// 32 of the step's own rows. Two ways to share the units, by plan():
//   Clusters, where every tile can have CTAs of its own: up to 8 CTAs take
//     equal parts of one tile and add their results through each other's shared
//     memory (each owns a part of the outputs), one barrier. Short contexts.
//   One line: the units of all tiles, sequence by sequence, form one line that
//     the CTAs cut into equal ranges, so that ragged lengths leave no SM idle.
//     A tile that lies in one range is written by its CTA; one that is cut
//     leaves partial results (running maximum, running sum, weighted values) in
//     the workspace, and the last of its CTAs to arrive adds them in range
//     order (many of them in groups first, Join). Nobody waits for anybody, and
//     the order of arrival changes nothing. Every tile takes kTileCost places more
//     than its units (its start and its end; GB300, 24 sequences of 33 to 16001
//     positions, 5 tokens, 32/8 heads of 64, bf16 out: 41 us with 10, 37 with 20,
//     39 with 34).
//
// Inside a CTA each of the W warps (8 or 12) takes every W-th unit of the range
// and keeps its own online softmax; the step's first 32 own rows are warp 0's,
// which gets one unit less (10 % on the same batch), and a longer step's next
// ones those of warps 1, 2, .. A record comes in
// one bulk copy into the warp's own ring. Both products run on the tensor cores
// (mma.sync m16n8k16, fp32 accumulation) with the keys, or the value dims, on
// the M side and the query rows on the N side in tiles of 8: few rows do not
// fill a tcgen05 tile's 128 (k_attn_kv4_tc.cu takes over from 9 or 17 rows, tc_rows).
//   S^T = K Q^T:  in bf16. Codes become bf16 values exactly (kv4_common.cuh): a nibble
//     shifted to bits 3..6 under the pattern of 16.0 is the number 24 + q, and
//     one fused multiply-add gives (24 + q) s - 24 s = q s without rounding.
//     A thread's 4 * W code words are one 16-byte read (W = D / 32) and all
//     belong to one scale group; which k index of the product each nibble
//     takes is free, so the query fragments are permuted to match.
//   P in base 2, kept unnormalised: p = 2^(7 + s - m). m is a whole number (so
//     that every rescaling factor is an exact power of two) that follows the
//     row's maximum lazily: it moves only when a score exceeds it by more than
//     8 (p is below 2^15.6 then; RowMax), so the usual step needs no reduction across
//     lanes and no rescaling. P is split into two f16 parts (an error of 2^-22 P, and
//     2^-32 of the largest P below f16's normal range) for fp32 outputs; for
//     bf16 outputs one part is enough (2^-11 P, an eighth of the output's own
//     rounding).
//   O^T += V^T P^T:  in f16, whose 11 bits make P's parts. The value scales
//     are taken times 2^-6, where every product q s is exact in f16 (2^-21 to
//     7 * 1920, and 24 s below 65504), and the output is multiplied by 2^6.
//     V's pairs run along keys: the 16-bit halves of two keys' words
//     interleave (prmt), after which the nibble step, with the pattern of 16.0
//     in f16, gives the A fragments of the dims a thread owns.
// What bounds it (GB300). Long contexts: the ALUs, which unpack 256 codes a
// position (55 % busy, with 61 % of the issue slots; DRAM 47 %): one token over
// 131071 and 120000 positions, 8 key/value heads, bf16 out, 72 us, 3.9 TB/s of
// cache. Short ones: the chain launch, lengths, table, record, products, merge:
// one token over 517 positions 5.9 us, 5 tokens over 2043 8.7 us.
//
// Every byte of a record is a finite value, so positions at and past a
// sequence's length may hold anything: their probability is 0 and 0 * v = 0.
// The step's own value rows can hold infinities or NaN in rows that some
// query rows must not see (padding): they are taken as 0 in the product and
// added afterwards to the rows that do see them.

#include <cooperative_groups.h>

#include "attn_kv4_common.cuh"

namespace cg = cooperative_groups;

namespace qv {

__device__ unsigned int g_attn_kv4_error;

namespace {

using namespace kv4attn;

template <int D, int NR>
struct Layout {
    using Rec = Kv4Rec<D>;
    static constexpr int W = D / 32;                      // 32-bit code words of a thread per key row
    static constexpr int KS = D / 16;                     // k steps of Q K^T = dim tiles of P V
    // What a warp's outputs take of its registers decides how many warps an SM
    // holds: 16 (two CTAs, 128 registers a thread), 12 (168) or 8 (255). The
    // tensor and ALU work of a step comes in dependent runs, so warps are what
    // keeps the pipes busy.
    static constexpr int ORegs = KS * NR * 4;
    static constexpr int Ctas = ORegs <= 64 ? 2 : 1;
    static constexpr int Warps = ORegs <= 64 ? 8 : (ORegs <= 96 ? 12 : 8);
    static constexpr int Threads = Warps * 32;
    static constexpr int Stages = D == 64 ? 4 : (NR == 2 ? 2 : (Warps * Ctas >= 12 ? 3 : 4));
    // With 8 warps on an SM the products of the next 16 positions are formed
    // between those of P and V of the present ones.
    static constexpr bool Pipe = Warps * Ctas == 8;
    static constexpr bool QRegs = ORegs <= 32;            // the query fragments stay in registers
    static constexpr int RW = NR * 8;
    static constexpr int Ring = 0;
    static constexpr int RingBytes = Warps * Stages * Rec::Bytes;
    static constexpr int AreaBytes = Warps * RW * D * 4; // the warps' outputs [Warps][NR*4*KS][32], in the drained ring
    static constexpr int Q = Ring + RingBytes;            // query fragments [NR][KS][32] uint2
    static constexpr int ML = Q + NR * KS * 32 * 8;       // m [Warps][RW], l [Warps][RW]
    static constexpr int Recv = ML + 2 * Warps * RW * 4;  // from the cluster's CTAs: items [C][RW*D/4/C], m [C][RW], l [C][RW]
    static constexpr int Bar = Recv + RW * D * 4 + 2 * kMaxCluster * RW * 4;
    static constexpr int Valid = Bar + Warps * Stages * 8;
    static constexpr int Scan = Valid + Warps * Stages * 4;    // unsigned [Warps], then [14], [15]: the first sequence's place and number
    static constexpr int Misc = Scan + 16 * 4;
    static constexpr int Tok = Misc + 64;                 // int [RW]: the step's last row that a query row sees
    static constexpr int Bytes = Tok + RW * 4;
    static constexpr int Items = RW * D / 4;              // groups of 4 dims of one row
    static constexpr int Slot = RW * D + 2 * RW;          // floats of a partial result: items, m, l
    static_assert(AreaBytes <= RingBytes, "the warps' outputs fit the ring");
    static_assert(Q % 16 == 0 && Recv % 16 == 0 && Bar % 8 == 0 && Scan % 4 == 0, "alignment");
};

template <int D, int NR, bool OUTBF>
__global__ void __launch_bounds__(Layout<D, NR>::Threads, Layout<D, NR>::Ctas) attn_kv4_kernel(const Args a) {
    using Ly = Layout<D, NR>;
    using Rec = Kv4Rec<D>;
    constexpr int W = Ly::W, KS = Ly::KS, S = Ly::Stages, RW = Ly::RW, kWarps = Ly::Warps, kThreads = Ly::Threads;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Ly::Bar) + warp * S;
    volatile int* valid = reinterpret_cast<volatile int*>(smem + Ly::Valid) + warp * S;
    float* s_area = reinterpret_cast<float*>(smem + Ly::Ring);
    float* s_wm = reinterpret_cast<float*>(smem + Ly::ML);
    float* s_wl = s_wm + kWarps * RW;
    unsigned* s_scan = reinterpret_cast<unsigned*>(smem + Ly::Scan);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + Ly::Misc);
    int* s_flag = reinterpret_cast<int*>(smem + Ly::Misc) + 1;       // an own value row is not finite
    Join* s_join = reinterpret_cast<Join*>(smem + Ly::Misc + 16);
    int* s_tok = reinterpret_cast<int*>(smem + Ly::Tok);
    const float NEG_INF = -__uint_as_float(0x7F800000u);
    const uint32_t ring = sbase + (uint32_t)(Ly::Ring + warp * S * Rec::Bytes);

    if (lane == 0)
        for (int s = 0; s < S; ++s) mbar_init(&bars[s], 1);
    if (tid == 0) {
        *abort = 0;
        s_flag[0] = 0;
    }
    fence_barrier_init();
    if (a.C > 1) cluster_arrive_relaxed();                       // waited for before the first store into another CTA
    allow_dependent_launch();
    grid_dependency_wait();

    const int own_units = (a.T + 31) / 32, tps = a.Hkv * a.RT;   // own units of a tile, tiles of a sequence
    const int C = a.C;                                           // CTAs of a cluster that share one tile, or 0
    const int rank = C > 0 ? (int)(blockIdx.x % (unsigned)C) : 0;
    Range rg = {0, 0, 1, 0, 0};
    if (C == 0 && !find_range<kThreads>(a, own_units, kTileCost, kMinUnits, s_scan, rg)) return;
    const unsigned per = rg.per, u1 = C > 0 ? 1 : rg.u1;
    unsigned seq_at = rg.seq_at, u = rg.u0;
    int b_next = C > 0 ? (int)(blockIdx.x / (unsigned)C) / tps : rg.b;
    unsigned issued = 0, used = 0;                               // this warp's records so far
    bool dead = false;                                           // a wait of this warp ran out: it takes no more units
    const size_t rowlen = (size_t)(a.Hq + 2 * a.Hkv) * D;
    const float sl2 = a.scale * kLog2e;
    const int key_g = g ^ ((g >> 1) & 1);                        // position in its 8 of S^T row g (see below)
    uint32_t c4 = 4u, c8 = 8u, c64 = 64u;                        // multipliers the compiler may not turn into shifts
    asm volatile("" : "+r"(c4), "+r"(c8), "+r"(c64));

    while (u < u1) {
        // ---- the tile that place u belongs to, and this CTA's part [ua, ub) of it
        const int b = b_next;
        const int L = seq_len(a, b);
        const int nc = (L + kKv4Block - 1) / kKv4Block, nu = nc + own_units;
        unsigned tile_at = 0;
        int ti, ua, ub;
        if (C > 0) {                                             // the one tile, its units cut into C equal parts
            ti = (int)(blockIdx.x / (unsigned)C) - b * tps;
            const int part = (nu + C - 1) / C;
            ua = min(nu, rank * part);
            ub = min(nu, ua + part);
            u = u1;
        } else {
            const unsigned places = (unsigned)(nu + kTileCost);
            ti = (int)((u - seq_at) / places);
            tile_at = seq_at + (unsigned)ti * places;
            ua = (int)(u - tile_at);
            ub = (int)min((unsigned)nu, u1 - tile_at);
            u = tile_at + places;                                // where this CTA goes on
            if (ti == tps - 1) {
                seq_at = u;
                ++b_next;
            }
            if (ua >= nu) continue;                              // (only empty places of the tile)
        }
        const int kh = ti / a.RT, rt = ti - kh * a.RT;
        const int r0 = rt * a.rows, R = min(a.rows, a.T * a.G - r0);   // query rows of this tile

        // ---- the queries (word w of a row's 16-byte piece at dims t4 * D/4 + 8 w
        // holds the pairs (d, d + 4) of two k steps), requested before anything waits
        constexpr int QLoads = (NR * W * 32 + kThreads - 1) / kThreads;
        uint4 qraw[QLoads];
#pragma unroll
        for (int i = 0; i < QLoads; ++i) {
            const int e = tid + i * kThreads, ln = e & 31, w = (e >> 5) % W, r = 8 * ((e >> 5) / W) + (ln >> 2);
            qraw[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < R) {
                const int j = (r0 + r) / a.G, h = kh * a.G + (r0 + r) - j * a.G;
                qraw[i] = *reinterpret_cast<const uint4*>(a.qkv + ((size_t)b * a.T + j) * rowlen + (size_t)h * D + (ln & 3) * (D / 4) + 8 * w);
            }
        }

        // The cached units go round the warps; the step's first 32 own rows, which
        // take about as long as one, are warp 0's, which sits out the first round.
        const int last = min(ub, nc);
        const bool own = ub > nc;
        auto unit_of = [&](int round) {
            const int slot = (round + (own && warp == 0 ? 1 : 0)) * kWarps + warp;
            return ua + slot - (own ? 1 : 0);
        };
        int round_issue = 0;
        int next = unit_of(0);                                   // next unit to request, and its page
        // (the table's entry is looked at only when it is used, a unit later)
        auto page_of = [&](int unit) {
            return unit >= last ? -1 : (a.table ? a.table[(size_t)b * a.NB + unit] : b * a.NB + unit);
        };
        int page = page_of(next);
        auto issue = [&]() {                                     // request the next unit's record, if there is one
            if (next >= last || dead) return;
            if (lane == 0) {
                const int s = issued % S;
                const bool there = (unsigned)page < (unsigned)a.pages;
                valid[s] = there;
                if (!a.hold) {
                    if (there) {
                        mbar_arrive_expect_tx(&bars[s], Rec::Bytes);
                        bulk_load(ring + (uint32_t)(s * Rec::Bytes), a.cache + ((size_t)page * a.Hkv + kh) * Rec::Bytes,
                                  Rec::Bytes, &bars[s]);
                    } else {
                        mbar_arrive(&bars[s]);
                    }
                }
            }
            ++issued;
            next = unit_of(++round_issue);
            page = page_of(next);
        };
#pragma unroll 1
        for (int s = 0; s < S; ++s) issue();

        // ---- the query fragments, permuted to match
#pragma unroll
        for (int i = 0; i < QLoads; ++i) {
            const int e = tid + i * kThreads;
            if (e < NR * W * 32) {
                const int ln = e & 31, w = (e >> 5) % W, nt = (e >> 5) / W;
                const uint4 q = qraw[i];
                uint2* dst = reinterpret_cast<uint2*>(smem + Ly::Q) + (nt * KS + 2 * w) * 32 + ln;
                dst[0] = make_uint2(__byte_perm(q.x, q.z, 0x5410), __byte_perm(q.x, q.z, 0x7632));
                dst[32] = make_uint2(__byte_perm(q.y, q.w, 0x5410), __byte_perm(q.y, q.w, 0x7632));
            }
        }
        if (tid < RW) s_tok[tid] = tid < R ? (r0 + tid) / a.G : -1;
        __syncthreads();
        uint2 qf[Ly::QRegs ? NR : 1][Ly::QRegs ? KS : 1];
        if constexpr (Ly::QRegs) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
                    lds_v2_u32(sbase + (uint32_t)(Ly::Q + ((nt * KS + kk) * 32 + lane) * 8), qf[nt][kk].x, qf[nt][kk].y);
        }
        float o[KS][NR][4];                                      // O^T: dims x rows
        // rows 8 nt + 2 t4 + e: p = 2^(sl2 x + c) of the product x (RowMax);
        // limit: the product at which m moves (-inf before the first key)
        float c[NR][2], limit[NR][2], l_run[NR][2];
#pragma unroll
        for (int nt = 0; nt < NR; ++nt) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.f;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                c[nt][e] = 0.f;
                limit[nt][e] = NEG_INF;
                l_run[nt][e] = 0.f;
            }
        }

        // The products of 16 positions into the running softmax: products in,
        // probabilities out.
        auto softmax = [&](float (&acc)[NR][4]) {
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) grow = grow || fmaxf(acc[nt][e], acc[nt][2 + e]) > limit[nt][e];
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float v = fmaxf(acc[nt][e], acc[nt][2 + e]);
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        if (v > limit[nt][e]) {                  // (the same in the row's 8 lanes)
                            const RowMax to(v, sl2);
                            const float f = limit[nt][e] == NEG_INF ? 0.f : ex2(to.c - c[nt][e]);
                            c[nt][e] = to.c;
                            limit[nt][e] = to.limit;
                            l_run[nt][e] *= f;
#pragma unroll
                            for (int i = 0; i < KS; ++i) {
                                o[i][nt][e] *= f;
                                o[i][nt][2 + e] *= f;
                            }
                        }
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float p0 = ex2(acc[nt][e] * sl2 + c[nt][e]), p1 = ex2(acc[nt][2 + e] * sl2 + c[nt][e]);
                    acc[nt][e] = p0;
                    acc[nt][2 + e] = p1;
                    l_run[nt][e] += p0 + p1;
                }
        };
        // P^T of 16 positions as the B operand (rows g; keys 2 t4, 2 t4 + 1 and
        // + 8) in parts of 16 bits: f16 ones for the cache's values, bf16 ones of
        // p 2^-6 for the step's own
        constexpr int Parts = OUTBF ? 1 : 2, OwnParts = OUTBF ? 2 : 3;
        auto p_frag = [&](const float (&p)[NR][4], uint32_t (&f)[Parts][NR][2]) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t h = pack_f16x2(p[nt][2 * k], p[nt][2 * k + 1]);
                    f[0][nt][k] = movmatrix_trans(h);
                    if constexpr (Parts == 2) {
                        const float2 hv = unpack_f16x2(h);
                        f[1][nt][k] = movmatrix_trans(pack_f16x2(p[nt][2 * k] - hv.x, p[nt][2 * k + 1] - hv.y));
                    }
                }
        };
        auto own_p_frag = [&](const float (&p)[NR][4], uint32_t (&f)[OwnParts][NR][2]) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float x = p[nt][2 * k] * 0x1p-6f, y = p[nt][2 * k + 1] * 0x1p-6f;
#pragma unroll
                    for (int q = 0; q < OwnParts; ++q) {
                        const uint32_t h = pack_bf16x2(x, y);
                        f[q][nt][k] = movmatrix_trans(h);
                        x -= __uint_as_float(h << 16);
                        y -= __uint_as_float(h & 0xFFFF0000u);
                    }
                }
        };
        // fp32 outputs: the products of 16 positions are formed from zero and added
        // with a rounded addition. The tensor cores cut an accumulator off below its
        // last bit, and a long run of products drifts towards zero: 2e-6 for one
        // token over 131071 positions, 3e-7 this way, for 5 % of the time.
        auto pv = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, const uint32_t (&f)[Parts][NR][2]) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
                if constexpr (OUTBF) {
                    mma_f16_16816(o[i][nt], a0, a1, a2, a3, f[0][nt][0], f[0][nt][1]);
                } else {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16_16816(d, a0, a1, a2, a3, f[Parts - 1][nt][0], f[Parts - 1][nt][1]);
                    mma_f16_16816(d, a0, a1, a2, a3, f[0][nt][0], f[0][nt][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[i][nt][e] += d[e];
                }
            }
        };
        auto own_pv = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                          const uint32_t (&f)[OwnParts][NR][2]) {
#pragma unroll
            for (int q = 0; q < OwnParts; ++q)
#pragma unroll
                for (int nt = 0; nt < NR; ++nt) mma_bf16_16816(o[i][nt], a0, a1, a2, a3, f[q][nt][0], f[q][nt][1]);
        };
        auto qk = [&](float (&acc)[NR][4], int kk, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt) {
                uint2 q;
                if constexpr (Ly::QRegs) q = qf[nt][kk];
                else lds_v2_u32(sbase + (uint32_t)(Ly::Q + ((nt * KS + kk) * 32 + lane) * 8), q.x, q.y);
                mma_bf16_16816(acc[nt], a0, a1, a2, a3, q.x, q.y);
            }
        };
        auto zero = [&](float (&acc)[NR][4]) {
#pragma unroll
            for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
        };

        // ---- the step's own rows, straight from the qkv rows (bf16), while the
        // first records are on their way: unit nc + i holds rows 32 i .. 32 i + 31
#pragma unroll 1
        for (int un = max(ua, nc) + warp; un < ub; un += kWarps) {
            const uint16_t* base = a.qkv + (size_t)b * a.T * rowlen + (size_t)(a.Hq + kh) * D;
            bool bad = false;
#pragma unroll 1
            for (int j0 = (un - nc) * 32; j0 < min(a.T, (un - nc) * 32 + 32); j0 += 16) {
                float acc[NR][4];
                zero(acc);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    uint4 x[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int j = j0 + 8 * k + key_g;
                        x[k] = make_uint4(0u, 0u, 0u, 0u);
                        if (j < a.T) x[k] = *reinterpret_cast<const uint4*>(base + (size_t)j * rowlen + t4 * (D / 4) + 8 * w);
                    }
                    qk(acc, 2 * w, __byte_perm(x[0].x, x[0].z, 0x5410), __byte_perm(x[1].x, x[1].z, 0x5410),
                       __byte_perm(x[0].x, x[0].z, 0x7632), __byte_perm(x[1].x, x[1].z, 0x7632));
                    qk(acc, 2 * w + 1, __byte_perm(x[0].y, x[0].w, 0x5410), __byte_perm(x[1].y, x[1].w, 0x5410),
                       __byte_perm(x[0].y, x[0].w, 0x7632), __byte_perm(x[1].y, x[1].w, 0x7632));
                }
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int tok = s_tok[8 * nt + 2 * t4 + e];      // rows 0..tok are visible
                        if (j0 + key_g > tok) acc[nt][e] = NEG_INF;
                        if (j0 + 8 + key_g > tok) acc[nt][2 + e] = NEG_INF;
                    }
                softmax(acc);
                uint32_t f[OwnParts][NR][2];
                own_p_frag(acc, f);
#pragma unroll
                for (int w = 0; w < W / 2; ++w) {
                    uint32_t y[2][2][4];
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int j = j0 + 8 * k + 2 * t4 + (e ^ (t4 & 1));
                            uint4 v = make_uint4(0u, 0u, 0u, 0u);
                            if (j < a.T) v = *reinterpret_cast<const uint4*>(base + (size_t)j * rowlen + (size_t)a.Hkv * D + g * (D / 8) + 8 * w);
                            y[k][e][0] = v.x; y[k][e][1] = v.y; y[k][e][2] = v.z; y[k][e][3] = v.w;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {        // infinities and NaN: 0 here, added below
                                if ((y[k][e][i] & 0x7F80u) == 0x7F80u) { y[k][e][i] &= 0xFFFF0000u; bad = true; }
                                if ((y[k][e][i] & 0x7F800000u) == 0x7F800000u) { y[k][e][i] &= 0xFFFFu; bad = true; }
                            }
                        }
                    // tile 4 w + j: rows g are dims 8 w + j, rows g + 8 dims 8 w + 4 + j
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int sel = j & 1 ? 0x7632 : 0x5410, i0 = j >> 1;
                        own_pv(4 * w + j, __byte_perm(y[0][0][i0], y[0][1][i0], sel), __byte_perm(y[0][0][2 + i0], y[0][1][2 + i0], sel),
                               __byte_perm(y[1][0][i0], y[1][1][i0], sel), __byte_perm(y[1][0][2 + i0], y[1][1][2 + i0], sel), f);
                    }
                }
            }
            if (bad) s_flag[0] = 1;
        }

        // ---- the cached units of this warp, 16 positions at a time. Row i of S^T
        // (and k index i of P V) is position i ^ ((i >> 1) & 1) of its 8:
        // neighbouring rows g of a 16-byte read, and the four t4 of an 8-byte one,
        // then alternate between the two halves of the banks
        auto load_keys = [&](Keys<W>& k2, uint32_t rec, int p0) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int key = p0 + 8 * k + key_g;
                const uint32_t at = rec + (uint32_t)(Rec::KC + key * Rec::RowBytes + t4 * (D / 8));
                if constexpr (W == 4) lds_v4_u32(at, k2.x[k][0], k2.x[k][1], k2.x[k][2], k2.x[k][3]);
                else lds_v2_u32(at, k2.x[k][0], k2.x[k][1]);
                k2.sc[k] = KeyScale(lds_u8(rec + (uint32_t)(Rec::KS + key * Rec::RowScales + (D == 128 ? t4 : t4 >> 1))));
            }
        };
        constexpr bool kLow = NR == 1;                           // (larger tiles have no registers to spare)
        auto qk_word = [&](float (&acc)[NR][4], const Keys<W>& k2, int w) {
            qk(acc, 2 * w, key_pair<0, kLow>(k2.x[0][w], k2.sc[0], c8), key_pair<0, kLow>(k2.x[1][w], k2.sc[1], c8),
               key_pair<1, kLow>(k2.x[0][w], k2.sc[0], c8), key_pair<1, kLow>(k2.x[1][w], k2.sc[1], c8));
            qk(acc, 2 * w + 1, key_pair<2, kLow>(k2.x[0][w], k2.sc[0], c8), key_pair<2, kLow>(k2.x[1][w], k2.sc[1], c8),
               key_pair<3, kLow>(k2.x[0][w], k2.sc[0], c8), key_pair<3, kLow>(k2.x[1][w], k2.sc[1], c8));
        };
        auto mask = [&](float (&acc)[NR][4], int p0, int left) {
            if (p0 + 16 > left) {
#pragma unroll
                for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (p0 + 8 * (e >> 1) + key_g >= left) acc[nt][e] = NEG_INF;
            }
        };
        // P V of 16 positions; with Pipe the following step's products are formed in
        // between, two k steps after every second dim tile
        auto values = [&](uint32_t rec, int p0, const uint32_t (&f)[Parts][NR][2], float (&nxt)[NR][4], const Keys<W>& k2) {
            uint32_t y[2][2][W / 2];                             // [k index + 8][even, odd key][word]
            ValScale sc[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t sb[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = p0 + 8 * k + 2 * t4 + (e ^ (t4 & 1));
                    const uint32_t at = rec + (uint32_t)(Rec::VC + key * Rec::RowBytes + g * (D / 16));
                    if constexpr (W == 4) lds_v2_u32(at, y[k][e][0], y[k][e][1]);
                    else y[k][e][0] = lds_u32(at);
                    sb[e] = lds_u8(rec + (uint32_t)(Rec::VS + key * Rec::RowScales + (D == 128 ? g >> 1 : g >> 2)));
                }
                sc[k] = ValScale(sb[0], sb[1]);
            }
#pragma unroll
            for (int w = 0; w < W / 2; ++w) {
                const uint32_t a0 = __byte_perm(y[0][0][w], y[0][1][w], 0x5410), a1 = __byte_perm(y[0][0][w], y[0][1][w], 0x7632);
                const uint32_t a2 = __byte_perm(y[1][0][w], y[1][1][w], 0x5410), a3 = __byte_perm(y[1][0][w], y[1][1][w], 0x7632);
                pv(4 * w, val_pair<0>(a0, sc[0], c4, c64), val_pair<0>(a1, sc[0], c4, c64), val_pair<0>(a2, sc[1], c4, c64), val_pair<0>(a3, sc[1], c4, c64), f);
                pv(4 * w + 1, val_pair<1>(a0, sc[0], c4, c64), val_pair<1>(a1, sc[0], c4, c64), val_pair<1>(a2, sc[1], c4, c64), val_pair<1>(a3, sc[1], c4, c64), f);
                if (Ly::Pipe) qk_word(nxt, k2, 2 * w);
                pv(4 * w + 2, val_pair<2>(a0, sc[0], c4, c64), val_pair<2>(a1, sc[0], c4, c64), val_pair<2>(a2, sc[1], c4, c64), val_pair<2>(a3, sc[1], c4, c64), f);
                pv(4 * w + 3, val_pair<3>(a0, sc[0], c4, c64), val_pair<3>(a1, sc[0], c4, c64), val_pair<3>(a2, sc[1], c4, c64), val_pair<3>(a3, sc[1], c4, c64), f);
                if (Ly::Pipe) qk_word(nxt, k2, 2 * w + 1);
            }
        };
        // Waits for the record of unit `un`, the i-th this warp takes; its cached
        // positions (0: no page), or -1 when the wait ran out.
        auto take = [&](int un, unsigned i) {
            const bool ok = bar_wait(&bars[i % S], (i / S) & 1u, abort, a.wait_ns);
            if (!__all_sync(0xffffffffu, ok)) {
                atomicOr(&g_attn_kv4_error, kErrFullWait);
                dead = true;
                return -1;
            }
            return valid[i % S] ? min(kKv4Block, L - un * kKv4Block) : 0;
        };
        auto done = [&]() {                                      // with the oldest record
            ++used;
            __syncwarp();                                        // every lane has read the stage
            issue();
        };
        if constexpr (!Ly::Pipe) {
#pragma unroll 1
            for (int round = 0, un = unit_of(0); un < last && !dead; un = unit_of(++round)) {
                const int left = take(un, used);
                if (left < 0) break;
                const uint32_t rec = ring + (uint32_t)((used % S) * Rec::Bytes);
#pragma unroll 1
                for (int p0 = 0; p0 < left; p0 += 16) {
                    Keys<W> k2;
                    load_keys(k2, rec, p0);
                    float acc[NR][4];
                    zero(acc);
#pragma unroll
                    for (int w = 0; w < W; ++w) qk_word(acc, k2, w);
                    mask(acc, p0, left);
                    softmax(acc);
                    uint32_t f[Parts][NR][2];
                    p_frag(acc, f);
                    values(rec, p0, f, acc, k2);
                }
                done();
            }
        } else {
            // acc: the products of the present step (record, p0); nxt: those of
            // the following one, formed between the present one's tiles of P V
            int round = 0, un = unit_of(0);
            int left = 0;                                        // of the present record
            while (un < last && !dead) {                         // the first record with a page
                left = take(un, used);
                if (left != 0) break;
                done();
                un = unit_of(++round);
            }
            if (left > 0) {
                uint32_t rec = ring + (uint32_t)((used % S) * Rec::Bytes);
                int p0 = 0;
                float acc[NR][4];
                {
                    Keys<W> k2;
                    load_keys(k2, rec, 0);
                    zero(acc);
#pragma unroll
                    for (int w = 0; w < W; ++w) qk_word(acc, k2, w);
                }
#pragma unroll 1
                while (true) {
                    // the following step: in this record, or in the next one
                    const int left_now = left;
                    const uint32_t rec_now = rec;
                    const int p_now = p0;
                    bool fresh = false, more = true;
                    p0 += 16;
                    if (p0 >= left) {
                        fresh = true;
                        p0 = 0;
                        un = unit_of(++round);
                        if (un < last) {
                            left = take(un, used + 1);
                            if (left < 0) break;
                            rec = ring + (uint32_t)(((used + 1) % S) * Rec::Bytes);
                        } else {
                            more = false;                        // (the last step's products are formed again, in vain)
                            rec = rec_now;
                        }
                    }
                    Keys<W> k2;
                    load_keys(k2, rec, p0);
                    mask(acc, p_now, left_now);
                    softmax(acc);
                    uint32_t f[Parts][NR][2];
                    p_frag(acc, f);
                    float nxt[NR][4];
                    zero(nxt);
                    values(rec_now, p_now, f, nxt, k2);
#pragma unroll
                    for (int nt = 0; nt < NR; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[nt][e] = nxt[nt][e];
                    if (fresh) done();
                    if (!more) break;
                }
            }
        }

        // ---- the warps' results side by side in shared memory (the ring has been
        // read: every record requested has been waited for)
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float l = l_run[nt][e];
                l += __shfl_xor_sync(0xffffffffu, l, 4);
                l += __shfl_xor_sync(0xffffffffu, l, 8);
                l += __shfl_xor_sync(0xffffffffu, l, 16);
                if (g == 0) {
                    s_wm[warp * RW + 8 * nt + 2 * t4 + e] = limit[nt][e] == NEG_INF ? NEG_INF : -c[nt][e];
                    s_wl[warp * RW + 8 * nt + 2 * t4 + e] = l;
                }
            }
        __syncthreads();
        constexpr int Plane = NR * 4 * (W / 2) * 32;             // float4: [warp][(nt, c, word)][lane], the word's 4 tiles
        float4* s_area4 = reinterpret_cast<float4*>(s_area);
#pragma unroll
        for (int nt = 0; nt < NR; ++nt)
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int w = 0; w < W / 2; ++w)
                    s_area4[warp * Plane + ((nt * 4 + q) * (W / 2) + w) * 32 + lane] =
                        make_float4(o[4 * w][nt][q], o[4 * w + 1][nt][q], o[4 * w + 2][nt][q], o[4 * w + 3][nt][q]);
        // each warp's weight for a row, the row's maximum and sum (m and l in place)
        if (tid < RW) {
            float M = s_wm[tid], l = 0.f;
            for (int x = 1; x < kWarps; ++x) M = fmaxf(M, s_wm[x * RW + tid]);
            for (int x = 0; x < kWarps; ++x) {
                const float m = s_wm[x * RW + tid], f = m == NEG_INF ? 0.f : ex2(m - M);
                l += f * s_wl[x * RW + tid];
                s_wm[x * RW + tid] = f;
            }
            s_wl[tid] = M;
            s_wl[RW + tid] = l;
        }
        __syncthreads();

        // ---- items of 4 dims of one row: (nt, e, word, half, lane); the warps'
        // parts added at the row's common maximum. Whole tiles go out, parts of
        // tiles to the workspace
        auto item_at = [&](int it, int& r, int& d0) {
            const int ln = it & 31, q = it >> 5, hf = q & 1, w = (q >> 1) % (W / 2), ne = (q >> 1) / (W / 2);
            r = 8 * (ne >> 1) + 2 * (ln & 3) + (ne & 1);
            d0 = (ln >> 2) * (D / 8) + 8 * w + 4 * hf;
        };
        auto item_sum = [&](int it, int r, int d0, float (&v)[4], float& M, float& l) {
            const int ln = it & 31, q = it >> 5, hf = q & 1, w = (q >> 1) % (W / 2), ne = (q >> 1) / (W / 2);
            M = s_wl[r];
            l = s_wl[RW + r];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = 0.f;
#pragma unroll
            for (int x = 0; x < kWarps; ++x) {
                const float f = s_wm[x * RW + r];
                const float4 y = s_area4[x * Plane + (((ne >> 1) * 4 + 2 * hf + (ne & 1)) * (W / 2) + w) * 32 + ln];
                v[0] += f * y.x; v[1] += f * y.y; v[2] += f * y.z; v[3] += f * y.w;
            }
            if (s_flag[0] && r < R) {                            // rare: own value rows that are not finite
                const int tk = (r0 + r) / a.G;
                const int jb = max(0, (ua - nc) * 32), je = min(tk + 1, (ub - nc) * 32);
                const uint16_t* vb = a.qkv + (size_t)b * a.T * rowlen + (size_t)(a.Hq + a.Hkv + kh) * D + d0;
                for (int j = jb; j < je; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t y = vb[(size_t)j * rowlen + i];
                        if ((y & 0x7F80u) == 0x7F80u) v[i] += __uint_as_float(y << 16);
                    }
            }
        };
        auto store = [&](int r, int d0, const float (&v)[4], float l) {
            if (r >= R) return;
            const int j = (r0 + r) / a.G, h = kh * a.G + (r0 + r) - j * a.G;
            const size_t at = ((size_t)b * a.T + j) * (size_t)a.Hq * D + (size_t)h * D + d0;
            const float inv = 64.f / l;                          // (the values were taken times 2^-6)
            if (OUTBF)
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) =
                    make_uint2(pack_bf16x2(v[0] * inv, v[1] * inv), pack_bf16x2(v[2] * inv, v[3] * inv));
            else
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) =
                    make_float4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
        };
        if (C > 1) {
            // into the CTAs that own the items, then the sum of this CTA's
            cg::cluster_group cluster = cg::this_cluster();
            float4* r_v = reinterpret_cast<float4*>(smem + Ly::Recv);
            float* r_m = reinterpret_cast<float*>(smem + Ly::Recv) + RW * D;
            float* r_l = r_m + kMaxCluster * RW;
            const int mine = Ly::Items / C;
            cluster_wait();                                      // every CTA of the cluster has started
            for (int it = tid; it < Ly::Items; it += kThreads) {
                int r, d0;
                float v[4], M, l;
                item_at(it, r, d0);
                item_sum(it, r, d0, v, M, l);
                const int k = it / mine;
                *cluster.map_shared_rank(r_v + rank * mine + (it - k * mine), k) = make_float4(v[0], v[1], v[2], v[3]);
                if (d0 == 0)
                    for (int q = 0; q < C; ++q) {
                        *cluster.map_shared_rank(r_m + rank * RW + r, q) = M;
                        *cluster.map_shared_rank(r_l + rank * RW + r, q) = l;
                    }
            }
            cluster.sync();                                      // every push has landed
            for (int i = tid; i < mine; i += kThreads) {
                int r, d0;
                item_at(rank * mine + i, r, d0);
                float M = NEG_INF, l = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
                for (int q = 0; q < C; ++q) M = fmaxf(M, r_m[q * RW + r]);
                for (int q = 0; q < C; ++q) {
                    const float m = r_m[q * RW + r], f = m == NEG_INF ? 0.f : ex2(m - M);
                    const float4 x = r_v[q * mine + i];
                    l += f * r_l[q * RW + r];
                    v[0] += f * x.x; v[1] += f * x.y; v[2] += f * x.z; v[3] += f * x.w;
                }
                store(r, d0, v, l);
            }
        } else if (ua == 0 && ub == nu) {
            for (int it = tid; it < Ly::Items; it += kThreads) {
                int r, d0;
                float v[4], M, l;
                item_at(it, r, d0);
                item_sum(it, r, d0, v, M, l);
                store(r, d0, v, l);
            }
        } else {
            float* slot = a.partials + ((size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0)) * Ly::Slot;
            for (int it = tid; it < Ly::Items; it += kThreads) {
                int r, d0;
                float v[4], M, l;
                item_at(it, r, d0);
                item_sum(it, r, d0, v, M, l);
                *reinterpret_cast<float4*>(slot + it * 4) = make_float4(v[0], v[1], v[2], v[3]);
                if (d0 == 0) {
                    slot[RW * D + r] = M;
                    slot[RW * D + RW + r] = l;
                }
            }
            const unsigned c0 = tile_at / per, c1 = (tile_at + (unsigned)nu - 1) / per;   // the tile's CTAs
            if (tid == 0) s_join->begin(c0, c1);
            // (called twice below: as a loop it cost the main loop registers, 74 us
            // against 72 for one token over 131071 and 120000 positions)
            auto join_once = [&]() {                             // true: nothing left to do
                __syncthreads();                                 // (the parts are written before thread 0's fence)
                if (tid == 0) s_join->arrive(a.counters);
                __syncthreads();
                if (!s_join->last) return true;
                // The parts, added in range order at the rows' maxima, kParts
                // of them at a time: first their weights (in the ring), then their
                // items, kAhead parts' loads in flight.
                constexpr int kParts = 64;
                constexpr int Own = (Ly::Items + kThreads - 1) / kThreads;    // items of a thread
                constexpr int kAhead = Own >= 3 ? 3 : (Own == 2 ? 4 : 8);
                static_assert((2 * kParts + 3) * RW * 4 <= Ly::RingBytes, "the parts' weights fit the ring");
                float* w_f = s_area;                             // [kParts][RW] maxima, then weights
                float* w_l = w_f + kParts * RW;
                float* w_M = w_l + kParts * RW;                  // [RW] so far: maximum, sum, the last rescaling
                float* w_L = w_M + RW;
                float* w_r = w_L + RW;
                const unsigned n = s_join->count, first = s_join->first, step = s_join->step, begin = s_join->c0;
                auto part = [&](unsigned i) {
                    const unsigned ci = first + i * step;
                    return a.partials + ((size_t)ci * 2 + (ci == begin ? 1 : 0)) * Ly::Slot;
                };
                float v[Own][4];
#pragma unroll
                for (int k = 0; k < Own; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[k][j] = 0.f;
                if (tid < RW) {
                    w_M[tid] = NEG_INF;
                    w_L[tid] = 0.f;
                }
#pragma unroll 1
                for (unsigned n0 = 0; n0 < n; n0 += kParts) {
                    const unsigned nn = min(n - n0, (unsigned)kParts);
                    for (unsigned e = tid; e < nn * RW; e += kThreads) {
                        const float* pp = part(n0 + e / RW) + RW * D + e % RW;
                        w_f[e] = __ldcg(pp);
                        w_l[e] = __ldcg(pp + RW);
                    }
                    __syncthreads();
                    if (tid < RW) {
                        const float old = w_M[tid];
                        float M = old, sum = 0.f;
                        for (unsigned i = 0; i < nn; ++i) M = fmaxf(M, w_f[i * RW + tid]);
                        for (unsigned i = 0; i < nn; ++i) {
                            const float m = w_f[i * RW + tid], f = m == NEG_INF ? 0.f : ex2(m - M);
                            w_f[i * RW + tid] = f;
                            sum += f * w_l[i * RW + tid];
                        }
                        const float fo = old == NEG_INF ? 0.f : ex2(old - M);
                        w_r[tid] = fo;
                        w_M[tid] = M;
                        w_L[tid] = w_L[tid] * fo + sum;
                    }
                    __syncthreads();
                    int r[Own];
#pragma unroll
                    for (int k = 0; k < Own; ++k) {
                        int d0;
                        item_at(min(tid + k * kThreads, Ly::Items - 1), r[k], d0);
                        const float fo = w_r[r[k]];
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[k][j] *= fo;
                    }
#pragma unroll 1
                    for (unsigned i0 = 0; i0 < nn; i0 += kAhead) {
                        float4 x[kAhead][Own];
#pragma unroll
                        for (int i = 0; i < kAhead; ++i) {
                            const float* pp = part(n0 + min(i0 + i, nn - 1));
#pragma unroll
                            for (int k = 0; k < Own; ++k)
                                x[i][k] = __ldcg(reinterpret_cast<const float4*>(pp) + min(tid + k * kThreads, Ly::Items - 1));
                        }
#pragma unroll
                        for (int i = 0; i < kAhead; ++i)
                            if (i0 + i < nn) {
#pragma unroll
                                for (int k = 0; k < Own; ++k) {
                                    const float f = w_f[(i0 + i) * RW + r[k]];
                                    v[k][0] += f * x[i][k].x; v[k][1] += f * x[i][k].y;
                                    v[k][2] += f * x[i][k].z; v[k][3] += f * x[i][k].w;
                                }
                            }
                    }
                    __syncthreads();
                }
                const bool final = s_join->final();
                float* sum = part(0);
#pragma unroll
                for (int k = 0; k < Own; ++k) {
                    const int it = tid + k * kThreads;
                    if (it < Ly::Items) {
                        int r, d0;
                        item_at(it, r, d0);
                        if (final) store(r, d0, v[k], w_L[r]);
                        else *reinterpret_cast<float4*>(sum + it * 4) = make_float4(v[k][0], v[k][1], v[k][2], v[k][3]);
                    }
                }
                if (final) return true;
                if (tid < RW) {
                    sum[RW * D + tid] = w_M[tid];
                    sum[RW * D + RW + tid] = w_L[tid];
                }
                __syncthreads();                                 // (everyone has read the join's state)
                if (tid == 0) s_join->next();
                return false;
            };
            if (!join_once()) join_once();
        }
        fence_proxy_async_smem();                                // before the ring's next copies
        __syncthreads();                                         // the ring, Q and the flags are free again
        if (tid == 0) s_flag[0] = 0;
    }
    // after a wait that ran out: no copy may be in flight when the CTA ends
    if (dead && !a.hold) {
        volatile int none = 0;
        for (; used < issued; ++used) bar_wait(&bars[used % S], (used / S) & 1u, &none, kWaitLimitNs);
    }
}

template <int D, int NR, bool OUTBF>
cudaError_t launch(const Args& a, int grid, cudaStream_t s) {                  // a.C > 1: clusters of a.C CTAs
    using Ly = Layout<D, NR>;
    static_assert(Ly::Bytes <= (int)(Ly::Ctas == 2 ? kMaxDynSmem / 2 - 1024 : kMaxDynSmem), "shared memory budget");
    cudaError_t e = cudaFuncSetAttribute(attn_kv4_kernel<D, NR, OUTBF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::Bytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(Ly::Threads);
    cfg.dynamicSmemBytes = Ly::Bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = a.C > 1 ? a.C : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, attn_kv4_kernel<D, NR, OUTBF>, a);
}

// Tiles of so many groups of 8 rows, heads of 128, go to the tcgen05 kernel:
// its time hardly depends on the rows of a tile or on P's parts, this kernel's
// grows with them. GB300, here / there in us for 8, 16, 24, 32 rows, 24
// sequences of 8000 positions: fp32 out 67/83, 94/89, 127/105, 170/109; bf16 out
// 59/80, 76/84, 100/99, 126/102. 2 of 131071, fp32, from 16 rows: 116/113,
// 151/136, 203/137.
constexpr int tc_rows(bool out_bf16) { return out_bf16 ? 3 : 2; }

struct Plan {
    int RT, rows, NR;
    int C;                       // CTAs of the cluster that takes a tile, or 0: one line of units cut into equal ranges
    bool tc;                     // the tcgen05 kernel
    int grid, cost, min_units;
    size_t total;                // workspace bytes; 0: more units than the kernel's 32-bit places can count
};
Plan plan(int B, int T, int Hq, int Hkv, int D, int NB, int sms, bool out_bf16) {
    const int rows = T * (Hq / Hkv);
    const long long units = (long long)NB + (T + 31) / 32;     // of a tile at most
    Plan p;
    long long tiles = 0;
    int slots = 0;
    // The head group's rows in as few tiles of at most `most` rows as there can
    // be, of equal size.
    auto cut = [&](int most) {
        p.RT = (rows + most - 1) / most;
        p.rows = (rows + p.RT - 1) / p.RT;
        p.NR = (p.rows + 7) / 8;
        tiles = (long long)B * Hkv * p.RT;
        slots = sms * (D / 64 * p.NR <= 4 ? 2 : 1);            // CTAs the GPU holds
    };
    // Short contexts: tiles of 8 rows (each reads the cache, from L2) while they
    // and their clusters all fit the GPU at once. GB300, 5 tokens over 2043
    // positions: 24 tiles of 7 rows 8.5 us, 8 tiles of 20 rows 10.9 us; where
    // they do not fit it is the other way round (5 tokens, 16 sequences of 300:
    // 17.3 us against 11.2).
    cut(8);
    p.C = 1;
    while (p.C < kMaxCluster && units > (long long)kClusterUnits * p.C) p.C *= 2;
    if (tiles * p.C > slots || units > (long long)kClusterMost * p.C) {
        cut(kRowTile);
        p.C = 1;
        while (p.C < kMaxCluster && tiles * p.C * 2 <= slots && units > (long long)kClusterUnits * p.C) p.C *= 2;
        // More tiles than CTAs fit at once: still a CTA each, one after the other,
        // where contexts are short and two CTAs share an SM. GB300, one line / a
        // CTA each: 64 sequences of 100 to 300 positions, 8 key/value heads, 1 token
        // of 4 heads 16.7/13.6 us, 5 tokens with heads of 64 21.3/18.2; up to 1200
        // positions 28.1/25.3. With one CTA an SM (5 tokens, heads of 128) 32/39.
        const bool alone = p.C == 1 && slots == 2 * sms && units <= kAloneMost;
        if ((tiles * p.C > slots && !alone) || units > (long long)kClusterMost * p.C) p.C = 0;
    }
    p.tc = p.C == 0 && D == 128 && p.NR >= tc_rows(out_bf16);
    p.cost = p.tc ? kTcTileCost : kTileCost;
    p.min_units = p.tc ? kTcMinUnits : kMinUnits;
    const long long most = tiles * (units + p.cost);           // places at most
    long long ctas = p.tc ? 2LL * sms : slots;
    ctas = ctas < kJoinSlots ? ctas : kJoinSlots;
    const long long want = (most + p.min_units - 1) / p.min_units;
    p.grid = p.C > 0 ? (int)(tiles * p.C) : (int)(want < ctas ? want : ctas);
    p.total = kCounterBytes + (p.C > 0 ? 0 : (size_t)p.grid * 2 * (p.NR * 8 * D + 2 * p.NR * 8) * 4);
    if (most >= (1ll << 31)) p.total = 0;
    return p;
}

}  // namespace

size_t attention_kv4_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int NB, int sms) {
    const size_t f = plan(B, T, Hq, Hkv, D, NB, sms, false).total, h = plan(B, T, Hq, Hkv, D, NB, sms, true).total;
    return f == 0 || h == 0 ? 0 : (f > h ? f : h);             // enough for both output types
}

cudaError_t launch_attention_kv4(const uint16_t* qkv, const uint8_t* cache, const int32_t* table, const int32_t* len,
                                 int B, int T, int Hq, int Hkv, int D, int NB, int pages, float scale, void* out,
                                 bool out_bf16, void* ws, int sms, int hold, unsigned long long wait_ns,
                                 cudaStream_t s) {
    const Plan p = plan(B, T, Hq, Hkv, D, NB, sms, out_bf16);
    Args a;
    a.qkv = qkv; a.cache = cache; a.table = table; a.len = len;
    a.B = B; a.T = T; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.NB = NB; a.pages = pages;
    a.RT = p.RT; a.rows = p.rows; a.C = p.C;
    a.scale = scale; a.out = out;
    a.counters = static_cast<unsigned*>(ws);
    a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
    a.hold = hold; a.wait_ns = wait_ns ? wait_ns : kWaitLimitNs;
    if (p.tc) return launch_attn_kv4_tc(a, p.NR, out_bf16, p.grid, p.cost, p.min_units, s);
#define QV_KV4_CASE(DV, NRV) \
    if (D == DV && p.NR == NRV) return out_bf16 ? launch<DV, NRV, true>(a, p.grid, s) : launch<DV, NRV, false>(a, p.grid, s);
    QV_KV4_CASE(128, 1) QV_KV4_CASE(128, 2) QV_KV4_CASE(128, 3) QV_KV4_CASE(128, 4)
    QV_KV4_CASE(64, 1) QV_KV4_CASE(64, 2) QV_KV4_CASE(64, 3) QV_KV4_CASE(64, 4)
#undef QV_KV4_CASE
    return cudaErrorInvalidValue;
}

cudaError_t read_and_clear_attn_kv4_error(unsigned* code) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_kv4_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    unsigned tc = 0;
    e = read_and_clear_attn_kv4_tc_error(&tc);
    if (e != cudaSuccess) return e;
    *code |= tc;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_kv4_error, &zero, sizeof(unsigned));
}

}  // namespace qv
