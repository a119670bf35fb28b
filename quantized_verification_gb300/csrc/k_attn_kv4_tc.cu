// k_attn_kv4_tc.cu -- attention over the 4-bit paged KV cache for heads of 128
// values, tiles of 9 (bf16 outputs: 17) to 32 query rows and long contexts, on
// the tcgen05 tensor cores.
//
//   What is computed, the cut of the work into tiles, units and places, and the
//   arithmetic (exact unpacking, base-2 probabilities with a lazy whole-number
//   maximum, two f16 parts of P for fp32 outputs) are k_attn_kv4.cu's; only the
//   products are formed elsewhere. On mma.sync many query rows keep the legacy
//   tensor pipe busy about as long as the unpacking the ALUs, with too few warps
//   to overlap the two. GB300, fp32 out, 24 sequences of 8000 positions, 8
//   key/value heads: 24 rows 105 us against 127, 32 rows 109 us against 170 (31
//   us to read the cache). What is left is the ALUs' and the issue slots' (49 and
//   54 % busy) and the waits of 4 unpacking warps a scheduler.
//
// A CTA takes 128 positions (4 records) a step. 8 warps work on them, a ninth
// requests records and issues the products; they meet at mbarriers, and the
// order is such that nothing is waited for that was not begun long before:
//   1. the keys of the NEXT step (thread = position, half the dims) become bf16
//      pairs in tensor memory, the A operand of S^T = K Q^T: 8 tcgen05.mma, M =
//      128 positions, N = the query rows padded to 16 or 32, B = Q in shared
//      memory, two S buffers;
//   2. this step's products are read (thread = position, the rows of every other
//      n8 tile) and compared with the rows' limits: does a maximum have to move?
//   3. the values become f16 (times 2^-6) in shared memory, the M-major A
//      operand of the second product (rows of positions, 128-byte swizzle; the
//      unpacked order of 8 dims is just an order of output rows);
//   4. with every warp's answer to 2 there by now, the probabilities go to
//      shared memory, and O^T += V^T P^T: 8 tcgen05.mma, M = 128 dims, N = the
//      rows' first parts side by side with their second parts, accumulated in
//      tensor memory while the next step begins.
// Two CTAs share an SM. The step's own keys and values are few and are not of
// the cache's format: they are attended to with plain fp32 arithmetic while the
// first records load; their outputs wait in tensor memory and are merged at the
// end. A tile's start, own rows and end take as long as about kTcTileCost units:
// 24 sequences of 33 to 16001 positions, 20 rows, 61 us with 18, 63 with 22, 64
// with 14.

#include "attn_kv4_common.cuh"

namespace qv {

__device__ unsigned int g_attn_kv4_tc_error;

namespace {

using namespace kv4attn;

constexpr int kTcWorkers = 256;                 // threads that unpack and form the softmax
constexpr int kTcThreads = kTcWorkers + 32;     // and the ninth warp
constexpr int kTcKeys = 128;                    // positions per step: 4 records
constexpr int kTcStages = 3;
constexpr int kTcMaxParts = 128;                // parts of a tile merged at once (their weights fill the value buffer)
// Steps that O accumulates before it is added to the sums, for fp32 outputs. The
// tensor cores cut the accumulator off below its last bit at every product, so
// that a long run drifts towards zero, 1.6e-8 of its result a product: 8e-6 for
// 7000 positions without these sums, 7e-7 with 4 steps (32 products), 4e-7 with
// 2, for 2 % more of the time.
constexpr int kTcFlush = 4;
constexpr int kTcOwnStride = 36;                // floats from one own row's scores to the next one's
constexpr int D = 128;

template <int NR, bool OUTBF>
struct TcLayout {
    using Rec = Kv4Rec<D>;
    static constexpr int RW = NR * 8;
    static constexpr int NS = (RW + 15) / 16 * 16;        // columns of S
    static constexpr int NO = OUTBF ? NS : 2 * RW;        // columns of O: first parts, then second parts
    static constexpr int V = 0;                           // [2 halves][128 positions][128 B], and the own scores
    static constexpr int P = V + 2 * kTcKeys * 128;       // [128 positions][128 B]
    static constexpr int Q = P + kTcKeys * 128;           // [2 halves][NS rows][128 B]
    static constexpr int Ring = Q + 2 * 32 * 128;
    static constexpr int Bar = Ring + kTcStages * 4 * Rec::Bytes;   // full [stages], then the kBar ones
    static constexpr int Cnt = Bar + (kTcStages + 9) * 8; // cached positions per record [stages][4]
    static constexpr int Row = Cnt + kTcStages * 16;      // floats per row: c, limit, f, own m, own l, w1, w2, M, l
    static constexpr int Red = Row + 9 * 32 * 4;          // [4][32]
    static constexpr int Scan = Red + 4 * 32 * 4;
    static constexpr int Misc = Scan + 16 * 4;
    static constexpr int Bytes = Misc + 64;
    static constexpr int Alloc = Bytes + 1024;            // slack to align the base to 1024 B
    static constexpr int Slot = RW * D + 2 * RW;          // floats of a partial result: [row][lane], m, l
    static constexpr int kK = 0, kS = 64, kO = 128, kOwn = 192, kSum = 224;   // tensor memory columns (S twice 32)
    static constexpr int Cols = 256;
    static_assert(Bar % 8 == 0 && Row % 16 == 0 && Ring % 16 == 0, "alignment");
    static_assert(2 * kTcMaxParts * 32 * 4 <= 2 * kTcKeys * 128, "the parts' weights fit the value buffer");
    static_assert(kTcOwnStride * kAttnMaxT * 4 <= 3 * kTcKeys * 128, "the own scores fit the buffers of V and P");
};

// Shared-memory descriptor of an operand stored with the M (or N) dimension
// contiguous: atoms of 64 16-bit elements x 8 k rows (128-byte swizzle), the
// next 8 k rows 1024 bytes on, the next 64 elements `mn_stride` bytes on.
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t saddr, uint32_t mn_stride) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(mn_stride >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}
// Instruction descriptor of kind::f16, M = 128, f32 accumulator. fmt: 0 f16, 1
// bf16 (both operands); mn: both operands M/N-major instead of K-major.
__host__ __device__ constexpr uint32_t idesc(int fmt, int N, bool mn) {
    return (1u << 4) | ((uint32_t)fmt << 7) | ((uint32_t)fmt << 10) | (mn ? (1u << 15) | (1u << 16) : 0u) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D[tmem] (+)= A[smem] * B[smem], one K = 16 step, issued by one thread.
__device__ __forceinline__ void umma_f16_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t id,
                                            uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(id), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// The 8 values of a row array for an n8 tile.
__device__ __forceinline__ void row8(const float* p, int tile, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[2 * tile], b = reinterpret_cast<const float4*>(p)[2 * tile + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
// bar_wait that reports the error `bit` if this wait is the one that ran out.
__device__ __forceinline__ bool wait_for(uint64_t* bar, unsigned parity, volatile int* abort, unsigned long long limit_ns,
                                         unsigned bit) {
    if (mbar_try_wait(bar, parity)) return true;
    const unsigned long long t0 = global_timer_ns();
    while (true) {
        if (*abort) return false;
        if (mbar_try_wait(bar, parity)) return true;
        if (global_timer_ns() - t0 > limit_ns) {
            *abort = 1;
            atomicOr(&g_attn_kv4_tc_error, bit);
            return false;
        }
    }
}
// One arrival per warp, for all its lanes.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

template <int NR, bool OUTBF>
__global__ void __launch_bounds__(kTcThreads, 2) attn_kv4_tc_kernel(const Args a, int tile_cost, int min_units) {
    using Ly = TcLayout<NR, OUTBF>;
    using Rec = Kv4Rec<D>;
    constexpr int RW = Ly::RW, NT = (NR + 1) / 2;                // n8 tiles of a thread: hf, hf + 2
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const bool worker = warp < kTcWorkers / 32;
    const int q4 = warp & 3, hf = (warp >> 2) & 1;                     // record (tensor memory lanes 32 q4 ..), half
    const int key = 32 * q4 + lane;                              // this thread's position, and its lane of O
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + Ly::Bar);
    uint64_t* bar_s = full + kTcStages;                          // S of a step is formed
    uint64_t* bar_o = bar_s + 1;                                 // O has taken a step's values
    uint64_t* bar_k = bar_s + 2;                                 // the keys of a step are in tensor memory (8 warps)
    uint64_t* bar_g = bar_s + 3;                                 // every warp has compared a step's products (8 warps)
    uint64_t* bar_p = bar_s + 4;                                 // the values and probabilities are in place (8 warps)
    uint64_t* bar_end = bar_s + 5;
    uint64_t* bar_r = bar_s + 6;                                 // the products' maxima are in place (8 warps)
    uint64_t* bar_m = bar_s + 7;                                 // the rows' maxima have moved (8 warps)
    volatile int* cnt = reinterpret_cast<volatile int*>(smem + Ly::Cnt);
    float* s_c = reinterpret_cast<float*>(smem + Ly::Row);       // p = 2^(sl2 x + c) of the product x (RowMax)
    float* s_lim = s_c + 32;                                     // the product at which m moves
    float* s_f = s_c + 64;
    float* s_m2 = s_c + 96;
    float* s_l2 = s_c + 128;
    float* s_w1 = s_c + 160;
    float* s_w2 = s_c + 192;
    float* s_M = s_c + 224;
    float* s_L = s_c + 256;
    float* s_red = reinterpret_cast<float*>(smem + Ly::Red);
    unsigned* s_scan = reinterpret_cast<unsigned*>(smem + Ly::Scan);
    volatile int* abort = reinterpret_cast<volatile int*>(smem + Ly::Misc);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + Ly::Misc) + 1;
    Join* s_join = reinterpret_cast<Join*>(smem + Ly::Misc + 32);
    volatile unsigned* s_grow = reinterpret_cast<volatile unsigned*>(smem + Ly::Misc) + 4;   // [2] the step whose maxima move, + 1
    float* s_own = reinterpret_cast<float*>(smem + Ly::V);       // [T][kTcOwnStride] own scores, before the first values
    const float NEG_INF = -__uint_as_float(0x7F800000u);

    // Tensor memory before dependents may start: one of theirs that held it
    // while it waited for this grid would never let it go.
    if (!worker) {
        tmem_alloc(s_tmem, Ly::Cols);
        tmem_relinquish();
    }
    if (tid == 32) {
        for (int s = 0; s < kTcStages + 2; ++s) mbar_init(&full[s], 1);
        mbar_init(bar_k, kTcWorkers / 32);
        mbar_init(bar_g, kTcWorkers / 32);
        mbar_init(bar_p, kTcWorkers / 32);
        mbar_init(bar_end, 1);
        mbar_init(bar_r, kTcWorkers / 32);
        mbar_init(bar_m, kTcWorkers / 32);
        *abort = 0;
        s_grow[0] = s_grow[1] = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *s_tmem;
    const uint32_t tlane = tmem + ((uint32_t)(32 * q4) << 16);   // this warp's lanes
    allow_dependent_launch();
    grid_dependency_wait();

    const int own_units = (a.T + 31) / 32, tps = a.Hkv * a.RT;
    const float sl2 = a.scale * kLog2e;
    const size_t rowlen = (size_t)(a.Hq + 2 * a.Hkv) * D;
    const uint64_t q_desc = sw128_kmajor_desc(sbase + (uint32_t)Ly::Q);
    const uint64_t v_desc = sw128_mnmajor_desc(sbase + (uint32_t)Ly::V, kTcKeys * 128);
    const uint64_t p_desc = sw128_mnmajor_desc(sbase + (uint32_t)Ly::P, kTcKeys * 128);
    uint32_t c4 = 4u, c8 = 8u, c64 = 64u;                        // multipliers the compiler may not turn into shifts
    asm volatile("" : "+r"(c4), "+r"(c8), "+r"(c64));
    unsigned steps_issued = 0, steps = 0;                        // 128-position steps requested / begun so far
    unsigned moves = 0;                                          // steps in which some row's maximum moved
    Range rg;
    bool work = find_range<kTcThreads>(a, own_units, tile_cost, min_units, s_scan, rg);
    const unsigned per = rg.per, u1 = work ? rg.u1 : 0;
    unsigned seq_at = rg.seq_at, u = work ? rg.u0 : 0;
    int b_next = rg.b;

    while (u < u1) {
        // ---- the tile that place u belongs to, and this CTA's part [ua, ub) of it
        const int b = b_next;
        const int L = seq_len(a, b);
        const int nc = (L + kKv4Block - 1) / kKv4Block, nu = nc + own_units;
        const unsigned places = (unsigned)(nu + tile_cost);
        const int ti = (int)((u - seq_at) / places);
        const unsigned tile_at = seq_at + (unsigned)ti * places;
        const int kh = ti / a.RT, rt = ti - kh * a.RT;
        const int ua = (int)(u - tile_at), ub = (int)min((unsigned)(nc + 1), u1 - tile_at);   // (the own rows are one piece)
        u = tile_at + places;                                    // where this CTA goes on
        if (ti == tps - 1) {
            seq_at = u;
            ++b_next;
        }
        if (ua > nc) continue;                                   // (nothing but empty places)
        const int r0 = rt * a.rows, R = min(a.rows, a.T * a.G - r0);   // query rows of this tile
        const bool own = ub > nc;
        const int last = min(ub, nc), nsteps = ua < last ? (last - ua + 3) / 4 : 0;

        // ---- records: lane i of the ninth warp requests record i of a step
        int unit = ua + lane;                                    // its next unit, and that unit's page
        auto page_of = [&](int x) {
            return x >= last ? -1 : (a.table ? a.table[(size_t)b * a.NB + x] : b * a.NB + x);
        };
        int page = !worker && lane < 4 ? page_of(unit) : -1;
        int to_issue = nsteps;
        auto issue = [&]() {
            if (to_issue == 0 || __any_sync(0xffffffffu, *abort)) return;
            --to_issue;
            const int s = steps_issued % kTcStages;
            const bool there = lane < 4 && unit < last && (unsigned)page < (unsigned)a.pages;
            if (lane < 4) cnt[4 * s + lane] = there ? min(kKv4Block, L - unit * kKv4Block) : 0;
            const unsigned who = __ballot_sync(0xffffffffu, there);
            __syncwarp();                                        // the counts, before lane 0 arrives (a ballot orders no memory)
            if (lane == 0 && !a.hold) {
                if (who) mbar_arrive_expect_tx(&full[s], (unsigned)__popc(who) * Rec::Bytes);
                else mbar_arrive(&full[s]);
            }
            __syncwarp();
            if (there && !a.hold)
                bulk_load(sbase + (uint32_t)(Ly::Ring + (4 * s + lane) * Rec::Bytes),
                          a.cache + ((size_t)page * a.Hkv + kh) * Rec::Bytes, Rec::Bytes, &full[s]);
            ++steps_issued;
            unit += 4;
            if (lane < 4) page = page_of(unit);
        };
        if (!worker)
            for (int s = 0; s < kTcStages; ++s) issue();

        // ---- Q, rows of 128-byte halves; 8 dims in the order 0 4 1 5 2 6 3 7
        for (int e = tid; e < Ly::NS * 16; e += kTcThreads) {
            const int n = e >> 4, ch = e & 15;
            uint4 x = make_uint4(0u, 0u, 0u, 0u);
            if (n < R) {
                const int j = (r0 + n) / a.G, h = kh * a.G + (r0 + n) - j * a.G;
                x = *reinterpret_cast<const uint4*>(a.qkv + ((size_t)b * a.T + j) * rowlen + (size_t)h * D + 8 * ch);
            }
            sts_v4_u32(sbase + (uint32_t)(Ly::Q + (ch >> 3) * Ly::NS * 128 + n * 128 + (((ch & 7) ^ (n & 7)) << 4)),
                       __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                       __byte_perm(x.y, x.w, 0x7632));
        }
        if (tid < 32) {
            s_c[tid] = 0.f;
            s_lim[tid] = NEG_INF;
            s_m2[tid] = NEG_INF;
            s_l2[tid] = 0.f;
        }
        float l[NT][8];                                          // this position's sums
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 8; ++i) l[t][i] = 0.f;
        const int dim = (key & 0x78) + ((key & 1) << 2) + ((key & 7) >> 1);   // the dim of O's lane `key`

        // ---- the step's own rows, in fp32
        if (own) {
            const uint16_t* kb = a.qkv + (size_t)b * a.T * rowlen + (size_t)(a.Hq + kh) * D;
            const uint16_t* vb = kb + (size_t)a.Hkv * D + dim;
            const int tmax = (r0 + R - 1) / a.G;                 // the last row seen here
            uint32_t v[8];                                       // 8 rows' values; the first 8 arrive during the scores
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = vb[(size_t)min(k, tmax) * rowlen];
            for (int e = tid >> 1; e < R * a.T; e += kTcThreads / 2) {   // two lanes a score, half the dims each
                const int r = e / a.T, j = e - r * a.T, tk = (r0 + r) / a.G;
                float x = NEG_INF;
                if (j <= tk) {
                    const int h = kh * a.G + (r0 + r) - tk * a.G;
                    const int d0 = (tid & 1) * (D / 2);
                    const uint4* qp = reinterpret_cast<const uint4*>(a.qkv + ((size_t)b * a.T + tk) * rowlen + (size_t)h * D + d0);
                    const uint4* kp = reinterpret_cast<const uint4*>(kb + (size_t)j * rowlen + d0);
                    float s0 = 0.f, s1 = 0.f;
#pragma unroll 4
                    for (int i = 0; i < D / 16; ++i) {
                        const uint4 x4 = qp[i], y4 = kp[i];
                        const uint32_t xs[4] = {x4.x, x4.y, x4.z, x4.w}, ys[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            s0 += __uint_as_float(xs[k] << 16) * __uint_as_float(ys[k] << 16);
                            s1 += __uint_as_float(xs[k] & 0xFFFF0000u) * __uint_as_float(ys[k] & 0xFFFF0000u);
                        }
                    }
                    s0 += s1;
                    x = (s0 + __shfl_xor_sync(3u << (lane & 30), s0, 1)) * sl2;
                }
                s_own[j * kTcOwnStride + r] = x;
            }
            __syncthreads();
            // each row's maximum, probabilities and sum: 2^lg lanes a row
            const int lg = a.T <= 8 ? 3 : 5, sub = lane >> lg, l0 = lane & ((1 << lg) - 1);
            for (int rw = warp << (5 - lg); rw < R; rw += (kTcThreads / 32) << (5 - lg)) {
                const int r = rw + sub;
                float m = NEG_INF, sum = 0.f;
                if (r < R)
                    for (int j = l0; j < a.T; j += 1 << lg) m = fmaxf(m, s_own[j * kTcOwnStride + r]);
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    if (off < 1 << lg) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                const float mm = m == NEG_INF ? 0.f : m;         // (no score above -inf)
                if (r < R)
                    for (int j = l0; j < a.T; j += 1 << lg) {
                        const float p = ex2(s_own[j * kTcOwnStride + r] - mm);
                        s_own[j * kTcOwnStride + r] = p;
                        sum += p;
                    }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1)
                    if (off < 1 << lg) sum += __shfl_xor_sync(0xffffffffu, sum, off);
                if (l0 == 0 && r < R) {
                    s_m2[r] = sum == 0.f ? NEG_INF : mm;         // (a NaN goes on)
                    s_l2[r] = sum;
                }
            }
            __syncthreads();
            if (worker) {
                float o2[NT][8];
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 8; ++i) o2[t][i] = 0.f;
#pragma unroll 1
                for (int j0 = 0; j0 <= tmax; j0 += 8) {
                    if (j0 > 0) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = vb[(size_t)min(j0 + k, tmax) * rowlen];
                    }
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        if (j0 + k > tmax) continue;             // (the same in all threads)
                        const int j = j0 + k, rmin = j * a.G - r0;   // rows from rmin on see row j
                        const float y = __uint_as_float(v[k] << 16);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (hf + 2 * t < NR) {
                                float p8[8];
                                row8(s_own + j * kTcOwnStride, hf + 2 * t, p8);
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const float sum = o2[t][i] + p8[i] * y;
                                    o2[t][i] = 8 * (hf + 2 * t) + i >= rmin ? sum : o2[t][i];
                                }
                            }
                    }
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (hf + 2 * t < NR) {
                        uint32_t ov[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(o2[t][i]);
                        tmem_st_x8(tlane + Ly::kOwn + 8 * (hf + 2 * t), ov);
                    }
                tmem_st_wait();
            }
        }
        fence_proxy_async_smem();                                // Q, before the products read it
        __syncthreads();

        // ---- 128 positions at a time. `steps` counts them over all tiles: the
        // parity of every barrier follows from it. Between here and the barrier
        // behind the steps every wait has a limit, and warps whose waits ran out
        // may be at different places: they decide as whole warps (votes), and no
        // barrier without a limit stands on a way that some of them may not take.
        if (!worker) {
            auto s_product = [&](int t0) {                       // S of step t0 of the tile
                const bool ok = wait_for(bar_k, (steps + t0) & 1u, abort, kWaitLimitNs, kErrTcWait);
                if (__all_sync(0xffffffffu, ok) && elect_one()) {
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_f16_ta(tmem + Ly::kS + 32 * ((steps + t0) & 1u), tmem + Ly::kK + 8 * ks,
                                    q_desc + (uint64_t)(((ks >> 2) * Ly::NS * 128 + (ks & 3) * 32) >> 4),
                                    idesc(1, Ly::NS, false), ks != 0);
                    umma_commit(bar_s);
                }
                __syncwarp();
            };
            if (nsteps > 0) s_product(0);
#pragma unroll 1
            for (int t0 = 0; t0 < nsteps; ++t0) {
                if (t0 + 1 < nsteps) s_product(t0 + 1);
                const bool ok = wait_for(bar_p, (steps + t0) & 1u, abort, kWaitLimitNs, kErrTcWait);
                if (__all_sync(0xffffffffu, ok) && elect_one()) {
                    tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        umma_f16_ss(tmem + Ly::kO, v_desc + (uint64_t)(ks * 2048 >> 4), p_desc + (uint64_t)(ks * 2048 >> 4),
                                    idesc(0, Ly::NO, true), ks != 0 || (OUTBF ? t0 != 0 : t0 % kTcFlush != 0) ? 1u : 0u);
                    umma_commit(bar_o);
                }
                __syncwarp();
                issue();                                         // (the stage's codes have all been read)
            }
        } else {
            auto unpack_keys = [&](int t0) {                     // of step t0 -> tensor memory, columns 32 hf ..
                const unsigned st = steps + t0;
                const int s = st % kTcStages;
                wait_for(&full[s], (st / kTcStages) & 1u, abort, a.wait_ns, kErrFullWait);
                const uint32_t rec = sbase + (uint32_t)(Ly::Ring + (4 * s + q4) * Rec::Bytes);
                const uint32_t at = rec + (uint32_t)(Rec::KC + lane * Rec::RowBytes + hf * 32);
                const int sw = (lane >> 1) & 1;                  // neighbours start with different 16 bytes
                uint32_t x[2][4];
                lds_v4_u32(at + 16 * sw, x[0][0], x[0][1], x[0][2], x[0][3]);
                lds_v4_u32(at + 16 * (1 - sw), x[1][0], x[1][1], x[1][2], x[1][3]);
                const uint32_t sb = lds_u32(rec + (uint32_t)(Rec::KS + lane * 4)) >> (16 * hf);
                uint32_t k32[32];
#pragma unroll
                for (int gr = 0; gr < 2; ++gr) {
                    const KeyScale sc((sb >> (8 * gr)) & 255u);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t y = sw == gr ? x[0][w] : x[1][w];
                        k32[16 * gr + 4 * w] = key_pair<0, true>(y, sc, c8);
                        k32[16 * gr + 4 * w + 1] = key_pair<1, true>(y, sc, c8);
                        k32[16 * gr + 4 * w + 2] = key_pair<2, true>(y, sc, c8);
                        k32[16 * gr + 4 * w + 3] = key_pair<3, true>(y, sc, c8);
                    }
                }
                tmem_st_x32(tlane + Ly::kK + 32 * hf, k32);
                tmem_st_wait();
                tc_fence_before();
                warp_arrive(bar_k);
            };
            if (nsteps > 0) unpack_keys(0);
#pragma unroll 1
            for (int t0 = 0; t0 < nsteps; ++t0) {
                const unsigned st = steps + t0;
                const int s = st % kTcStages;
                wait_for(bar_s, st & 1u, abort, kWaitLimitNs, kErrTcWait);   // (S is formed and the keys' columns are free)
                tc_fence_after();
                if (t0 + 1 < nsteps) unpack_keys(t0 + 1);
                // this position's products with the rows of tiles hf, hf + 2
                const bool there = lane < cnt[4 * s + q4];
                uint32_t x[NT][8];
                bool grow = false;
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (hf + 2 * t < NR) tmem_ld<8>(tlane + Ly::kS + 32 * (st & 1u) + 8 * (hf + 2 * t), x[t]);
                tmem_ld_wait();
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (hf + 2 * t < NR) {
                        float lim[8];
                        row8(s_lim, hf + 2 * t, lim);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (!there) x[t][i] = __float_as_uint(NEG_INF);
                            grow |= __uint_as_float(x[t][i]) > lim[i];
                        }
                    }
                if (grow) s_grow[st & 1u] = st + 1;
                tc_fence_before();
                warp_arrive(bar_g);
                // values: the previous step's product has read the buffer
                if (t0 > 0) wait_for(bar_o, (st - 1) & 1u, abort, kWaitLimitNs, kErrTcWait);
                const uint32_t stage = sbase + (uint32_t)(Ly::Ring + 4 * s * Rec::Bytes);
#pragma unroll
                for (int it = 0; it < 2; ++it) {
                    const int ch = tid & 3, pos = (tid >> 2) + 64 * it;   // 16 bytes of codes: 32 dims of one position
                    const uint32_t rec = stage + (uint32_t)((pos >> 5) * Rec::Bytes);
                    uint32_t y4[4];
                    lds_v4_u32(rec + (uint32_t)(Rec::VC + (pos & 31) * Rec::RowBytes + ch * 16), y4[0], y4[1], y4[2], y4[3]);
                    const uint32_t sb = lds_u8(rec + (uint32_t)(Rec::VS + (pos & 31) * 4 + ch));
                    const ValScale sc(sb, sb);
                    // chunks 2, 3 (dims 64 ..) store their words in pairs the other
                    // way round: the four chunks then fall on different banks
                    const bool odd = (ch & 2) != 0;
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t y = odd ? y4[w ^ 1] : y4[w];
                        const int c16 = (ch & 1) * 4 + (odd ? w ^ 1 : w);
                        sts_v4_u32(sbase + (uint32_t)(Ly::V + (ch >> 1) * kTcKeys * 128 + pos * 128 + ((c16 ^ (pos & 7)) << 4)),
                                   val_pair<0>(y, sc, c4, c64), val_pair<1>(y, sc, c4, c64), val_pair<2>(y, sc, c4, c64),
                                   val_pair<3>(y, sc, c4, c64));
                    }
                }
                wait_for(bar_g, st & 1u, abort, kWaitLimitNs, kErrTcWait);
                if (__any_sync(0xffffffffu, s_grow[st & 1u] == st + 1)) {   // rare: some row's maximum moves
                    tc_fence_after();
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (hf + 2 * t < NR) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float v = __uint_as_float(x[t][i]);
#pragma unroll
                                for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
                                if (lane == 0) s_red[q4 * 32 + 8 * (hf + 2 * t) + i] = v;
                            }
                        }
                    warp_arrive(bar_r);
                    wait_for(bar_r, moves & 1u, abort, kWaitLimitNs, kErrTcWait);
                    if (tid < RW) {
                        const float v = fmaxf(fmaxf(s_red[tid], s_red[32 + tid]), fmaxf(s_red[64 + tid], s_red[96 + tid]));
                        float f = 1.f;
                        if (v > s_lim[tid]) {
                            const RowMax to(v, sl2);
                            f = s_lim[tid] == NEG_INF ? 0.f : ex2(to.c - s_c[tid]);
                            s_c[tid] = to.c;
                            s_lim[tid] = to.limit;
                        }
                        s_f[tid] = f;
                    }
                    warp_arrive(bar_m);
                    wait_for(bar_m, moves & 1u, abort, kWaitLimitNs, kErrTcWait);
                    ++moves;
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (hf + 2 * t < NR) {
                            float f8[8];
                            row8(s_f, hf + 2 * t, f8);
#pragma unroll
                            for (int i = 0; i < 8; ++i) l[t][i] *= f8[i];
                            if (t0 > 0) {
#pragma unroll
                                for (int part = 0; part < (OUTBF ? 1 : 2); ++part) {
                                    uint32_t ov[8];
                                    tmem_ld<8>(tlane + Ly::kO + part * RW + 8 * (hf + 2 * t), ov);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f8[i]);
                                    tmem_st_x8(tlane + Ly::kO + part * RW + 8 * (hf + 2 * t), ov);
                                }
                                if (!OUTBF && t0 > kTcFlush) {
                                    uint32_t ov[8];
                                    tmem_ld<8>(tlane + Ly::kSum + 8 * (hf + 2 * t), ov);
                                    tmem_ld_wait();
#pragma unroll
                                    for (int i = 0; i < 8; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * f8[i]);
                                    tmem_st_x8(tlane + Ly::kSum + 8 * (hf + 2 * t), ov);
                                }
                                tmem_st_wait();
                            }
                        }
                }
                if (!OUTBF && t0 > 0 && t0 % kTcFlush == 0) {    // the next product begins O afresh
                    tc_fence_after();
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (hf + 2 * t < NR) {
                            uint32_t h8[8], l8[8], s8[8];
                            tmem_ld<8>(tlane + Ly::kO + 8 * (hf + 2 * t), h8);
                            tmem_ld<8>(tlane + Ly::kO + RW + 8 * (hf + 2 * t), l8);
                            if (t0 > kTcFlush) tmem_ld<8>(tlane + Ly::kSum + 8 * (hf + 2 * t), s8);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float y = __uint_as_float(h8[i]) + __uint_as_float(l8[i]);
                                s8[i] = __float_as_uint(t0 > kTcFlush ? __uint_as_float(s8[i]) + y : y);
                            }
                            tmem_st_x8(tlane + Ly::kSum + 8 * (hf + 2 * t), s8);
                        }
                    tmem_st_wait();
                }
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (hf + 2 * t < NR) {
                        const int tile = hf + 2 * t;
                        uint32_t hi[4], lo[4];
                        float c[8];
                        row8(s_c, tile, c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float p0 = ex2(__uint_as_float(x[t][2 * i]) * sl2 + c[2 * i]);
                            const float p1 = ex2(__uint_as_float(x[t][2 * i + 1]) * sl2 + c[2 * i + 1]);
                            l[t][2 * i] += p0;
                            l[t][2 * i + 1] += p1;
                            hi[i] = pack_f16x2(p0, p1);
                            const float2 h = unpack_f16x2(hi[i]);
                            lo[i] = pack_f16x2(p0 - h.x, p1 - h.y);
                        }
                        const uint32_t prow = sbase + (uint32_t)(Ly::P + key * 128);
                        sts_v4_u32(prow + (uint32_t)((tile ^ (key & 7)) << 4), hi[0], hi[1], hi[2], hi[3]);
                        if (!OUTBF) sts_v4_u32(prow + (uint32_t)(((NR + tile) ^ (key & 7)) << 4), lo[0], lo[1], lo[2], lo[3]);
                    }
                fence_proxy_async_smem();
                tc_fence_before();
                warp_arrive(bar_p);
            }
        }
        steps += (unsigned)nsteps;

        // ---- the rows' sums, and the weights of the cache's and the own part
        if (nsteps > 0) {
            wait_for(bar_o, (steps - 1) & 1u, abort, kWaitLimitNs, kErrTcWait);
            tc_fence_after();
            if (worker)
#pragma unroll
            for (int t = 0; t < NT; ++t)
                if (hf + 2 * t < NR) {
#pragma unroll
                    for (int w = 4; w > 0; w >>= 1)              // half the values stay, the other lane has the rest
#pragma unroll
                        for (int i = 0; i < w; ++i) {
                            const bool up = (lane & (4 * w)) != 0;
                            const float give = up ? l[t][i] : l[t][i + w];
                            l[t][i] = (up ? l[t][i + w] : l[t][i]) + __shfl_xor_sync(0xffffffffu, give, 4 * w);
                        }
                    float y = l[t][0];
                    y += __shfl_xor_sync(0xffffffffu, y, 2);
                    y += __shfl_xor_sync(0xffffffffu, y, 1);
                    if ((lane & 3) == 0) s_red[q4 * 32 + 8 * (hf + 2 * t) + (lane >> 2)] = y;
                }
        }
        __syncthreads();
        if (tid < RW) {
            const float lc = nsteps > 0 ? (s_red[tid] + s_red[32 + tid]) + (s_red[64 + tid] + s_red[96 + tid]) : 0.f;
            const float e1 = s_lim[tid] == NEG_INF ? NEG_INF : -s_c[tid], e2 = s_m2[tid];
            const float M = fmaxf(e1, e2);
            const float w1 = e1 == NEG_INF ? 0.f : ex2(e1 - M), w2 = e2 == NEG_INF ? 0.f : ex2(e2 - M);
            s_w1[tid] = 64.f * w1;                               // (the values were taken times 2^-6)
            s_w2[tid] = w2;
            s_M[tid] = M;
            s_L[tid] = lc * w1 + s_l2[tid] * w2;
            s_f[tid] = 1.f / s_L[tid];
        }
        __syncthreads();
        float v[NT][8];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            uint32_t h8[8], l8[8], o8[8], s8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h8[i] = l8[i] = o8[i] = s8[i] = 0u;
            if (worker && hf + 2 * t < NR) {
                if (nsteps > 0) {
                    tmem_ld<8>(tlane + Ly::kO + 8 * (hf + 2 * t), h8);
                    if (!OUTBF) tmem_ld<8>(tlane + Ly::kO + RW + 8 * (hf + 2 * t), l8);
                    if (!OUTBF && nsteps > kTcFlush) tmem_ld<8>(tlane + Ly::kSum + 8 * (hf + 2 * t), s8);
                }
                if (own) tmem_ld<8>(tlane + Ly::kOwn + 8 * (hf + 2 * t), o8);
                tmem_ld_wait();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = min(8 * (hf + 2 * t) + i, RW - 1);
                v[t][i] = (__uint_as_float(s8[i]) + (__uint_as_float(h8[i]) + __uint_as_float(l8[i]))) * s_w1[r] + __uint_as_float(o8[i]) * s_w2[r];
            }
        }
        // this lane's dim of the rows; inv holds one over their sums
        auto store = [&](const float (&x)[NT][8], const float* inv) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int ra = r0 + 8 * (hf + 2 * t);
                int j = ra / a.G, hg = ra - j * a.G;             // token, head of the group
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 8 * (hf + 2 * t) + i;
                    if (worker && r < R) {
                        const size_t at = ((size_t)b * a.T + j) * (size_t)a.Hq * D + (size_t)(kh * a.G + hg) * D + dim;
                        if (OUTBF) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(x[t][i] * inv[r]);
                        else static_cast<float*>(a.out)[at] = x[t][i] * inv[r];
                    }
                    if (++hg == a.G) {
                        hg = 0;
                        ++j;
                    }
                }
            }
        };
        if (ua == 0 && own) {
            store(v, s_f);
        } else {
            float* slot = a.partials + ((size_t)blockIdx.x * 2 + (ua == 0 ? 1 : 0)) * Ly::Slot;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 8 * (hf + 2 * t) + i;
                    if (worker && r < RW) slot[r * D + key] = v[t][i];   // (rows past R too: they are read, not used)
                }
            if (tid < RW) {
                slot[RW * D + tid] = s_M[tid];
                slot[RW * D + RW + tid] = s_L[tid];
            }
            const unsigned c0 = tile_at / per, c1 = (tile_at + (unsigned)nc) / per;   // the tile's CTAs
            if (tid == 0) s_join->begin(c0, c1);
#pragma unroll 1
            while (true) {
                __syncthreads();                                 // (the part is written before thread 0's fence)
                if (tid == 0) s_join->arrive(a.counters);
                __syncthreads();
                if (!s_join->last) break;
                // The parts, added in range order at the rows' common maxima:
                // the weights first (in the value buffer, [part][32]), then four
                // parts' rows at a time.
                const unsigned n = s_join->count, first = s_join->first, step = s_join->step, begin = s_join->c0;
                auto part = [&](unsigned i) {
                    const unsigned ci = first + i * step;
                    return a.partials + ((size_t)ci * 2 + (ci == begin ? 1 : 0)) * Ly::Slot;
                };
                float* s_f2 = reinterpret_cast<float*>(smem + Ly::V);
                float* s_l3 = s_f2 + kTcMaxParts * 32;
                float run[NT][8];                                // this dim's sums so far, at the maxima s_M
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 8; ++i) run[t][i] = 0.f;
                if (tid < 32) {
                    s_M[tid] = NEG_INF;
                    s_L[tid] = 0.f;
                }
#pragma unroll 1
                for (unsigned n0 = 0; n0 < n; n0 += kTcMaxParts) {
                    const unsigned nn = min(n - n0, (unsigned)kTcMaxParts);
                    for (unsigned e = tid; e < nn * 32; e += kTcThreads) {
                        const float* pp = part(n0 + (e >> 5));
                        const int r = min((int)(e & 31), RW - 1);
                        s_f2[e] = __ldcg(pp + RW * D + r);
                        s_l3[e] = __ldcg(pp + RW * D + RW + r);
                    }
                    __syncthreads();
                    if (tid < 32) {
                        const float old = s_M[tid];
                        float M = old, sum = 0.f;
                        for (unsigned i = 0; i < nn; ++i) M = fmaxf(M, s_f2[i * 32 + tid]);
                        for (unsigned i = 0; i < nn; ++i) {
                            const float m = s_f2[i * 32 + tid], f = m == NEG_INF ? 0.f : ex2(m - M);
                            s_f2[i * 32 + tid] = f;
                            sum += f * s_l3[i * 32 + tid];
                        }
                        const float fo = old == NEG_INF ? 0.f : ex2(old - M);
                        s_f[tid] = fo;
                        s_M[tid] = M;
                        s_L[tid] = s_L[tid] * fo + sum;
                        s_w1[tid] = 1.f / s_L[tid];
                    }
                    __syncthreads();
#pragma unroll
                    for (int t = 0; t < NT; ++t)
                        if (worker && hf + 2 * t < NR) {
                            float f8[8];
                            row8(s_f, hf + 2 * t, f8);
#pragma unroll
                            for (int i = 0; i < 8; ++i) run[t][i] *= f8[i];
#pragma unroll 1
                            for (unsigned i0 = 0; i0 < nn; i0 += 4) {
                                float x[4][8];
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const float* pp = part(n0 + min(i0 + k, nn - 1)) + 8 * (hf + 2 * t) * D + key;
#pragma unroll
                                    for (int i = 0; i < 8; ++i) x[k][i] = __ldcg(pp + i * D);
                                }
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (i0 + k < nn) {
                                        row8(s_f2 + (i0 + k) * 32, hf + 2 * t, f8);
#pragma unroll
                                        for (int i = 0; i < 8; ++i) run[t][i] += x[k][i] * f8[i];
                                    }
                            }
                        }
                    __syncthreads();
                }
                if (s_join->final()) {
                    store(run, s_w1);
                    break;
                }
                float* sum = part(0);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 8 * (hf + 2 * t) + i;
                        if (worker && r < RW) sum[r * D + key] = run[t][i];
                    }
                if (tid < RW) {
                    sum[RW * D + tid] = s_M[tid];
                    sum[RW * D + RW + tid] = s_L[tid];
                }
                __syncthreads();                                 // (everyone has read the join's state)
                if (tid == 0) s_join->next();
            }
        }
        tc_fence_before();                                       // O has been read
        __syncthreads();
        tc_fence_after();
    }
    // after a wait that ran out: no copy and no product may be in flight when the CTA ends
    if (work && *abort && !worker) {
        volatile int none = 0;
        if (!a.hold)
            for (unsigned s = steps_issued > kTcStages ? steps_issued - kTcStages : 0; s < steps_issued; ++s)
                bar_wait(&full[s % kTcStages], (s / kTcStages) & 1u, &none, kWaitLimitNs);
        if (elect_one()) umma_commit(bar_end);
        __syncwarp();
        bar_wait(bar_end, 0u, &none, kWaitLimitNs);
    }
    tc_fence_before();
    __syncthreads();
    if (!worker) {
        tc_fence_after();
        tmem_dealloc(tmem, Ly::Cols);
    }
}

template <int NR, bool OUTBF>
cudaError_t launch(const Args& a, int grid, int tile_cost, int min_units, cudaStream_t s) {
    using Ly = TcLayout<NR, OUTBF>;
    static_assert(Ly::Alloc <= (int)(kMaxDynSmem / 2 - 1024), "two CTAs per SM");
    cudaError_t e = cudaFuncSetAttribute(attn_kv4_tc_kernel<NR, OUTBF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::Alloc);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = Ly::Alloc;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv4_tc_kernel<NR, OUTBF>, a, tile_cost, min_units);
}

}  // namespace

cudaError_t launch_attn_kv4_tc(const kv4attn::Args& a, int NR, bool out_bf16, int grid, int tile_cost, int min_units,
                               cudaStream_t s) {
    if (NR == 2 && !out_bf16) return launch<2, false>(a, grid, tile_cost, min_units, s);
#define QV_KV4_TC_CASE(NRV) \
    if (NR == NRV) return out_bf16 ? launch<NRV, true>(a, grid, tile_cost, min_units, s) : launch<NRV, false>(a, grid, tile_cost, min_units, s);
    QV_KV4_TC_CASE(3) QV_KV4_TC_CASE(4)
#undef QV_KV4_TC_CASE
    return cudaErrorInvalidValue;
}

cudaError_t read_and_clear_attn_kv4_tc_error(unsigned* code) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_kv4_tc_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_kv4_tc_error, &zero, sizeof(unsigned));
}

}  // namespace qv
