// k_attn_prompt.cu -- attention of many query rows on the tcgen05 tensor cores:
// whole prompts, packed one behind the other (causal), and the rows of a batch
// over a prefix that all its sequences share (partial results over its parts and
// over parts of each sequence's cache, merged with the step's own keys by a second
// kernel).
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
// Roles: 4 warps form the softmax of a tile (thread = row, its 128 scores in
// registers: no shuffles), one warp issues the products, one the TMA loads of keys
// and values, 128 positions each, into one ring. Per tile and 128 keys:
//   S = Q K^T      8 tcgen05.mma (D = 128), M = N = 128, both operands K-major
//                  in shared memory, the accumulator in tensor memory
//   P = 2^(cS-m)   rounded to bf16 over S's columns in tensor memory. The reference
//                  m lies 8 above a row's first maximum and moves only when a score
//                  passes it, to 8 above that: no P is above 1, and O is hardly
//                  ever rescaled. When it is, the softmax threads do it
//                  themselves, at a time when no product writes it
//   O += P V       8 tcgen05.mma, P from tensor memory, V as stored (M/N-major)
// With two tiles one's softmax runs under the other's products; with one tile S
// has two buffers.
// Rounding of P. The product takes operands of one type, V's bf16. For bf16 outputs P
// is one part: half a step (2^-8) of each probability makes them 2.0e-3 off in the
// 2-norm, where their own rounding alone makes 1.6e-3 (with the rounded P in l as well
// the same to 2 %). fp32 outputs take two parts (residue 2^-17), twice the second
// product, and are 1.5 to 3.4e-6 off, at 1.8 times the time (6000 tokens 0.34 ms, 0.19
// for bf16). A third part has room in tensor memory with one tile a CTA only (heads of
// 128) and was still 0.3 to 3.6e-6 off by the cuts that follow: 6000 tokens 0.57 ms,
// five prompts of up to 1500 tokens 39 us instead of 31.
// Sums. The tensor cores cut the accumulator off at every product (1.6e-8 of it, all
// one way, more as it outgrows what is added). For fp32 outputs O is added in binary32
// every kFlush steps to the row's sums, which lie where the output goes (every 4 steps
// 1.5 to 2.7e-6 off, 8 to 20 % slower); for bf16 ones every kFlushLong steps to a
// prefix's partial results. A prompt's bf16 outputs have no room for sums: there O's
// high part is kept and O goes on with the rest (carry).
//
// Bound by the tensor cores from about 1000 rows on, where S, P and O pass through
// tensor memory in time. GB300, causal, bf16 outputs: one prompt of 16001 tokens, 64/8
// heads of 128, 2.45 ms (1710 TFLOP/s, 0.90 of a measured cuBLAS product; 2.7 ms
// = 0.81 of it where the power limit is reached); 6000 tokens, 32/8 heads, 0.19 ms
// (heads of 64 0.160, fp32 outputs 0.344); 2043 tokens 31 us; 24 prompts of 33 to
// 4001 tokens 322 to 325 us (1190 TFLOP/s; 339 to 344 in a stream of calls). A step of two
// tiles takes about 2500 cycles of the 2080 that its 32 products need; a block's first
// and last steps, whose code and data are cold, 2 to 4 thousand more. 97 tokens: 6 us,
// of which 2.4 are start and first loads.
// Prefixes: 64 tokens, 64/8 heads behind 100001 positions 163 us (1290 TFLOP/s with
// the caches' parts and the merge; 176 in a stream of calls), 24 sequences of 5 tokens
// behind 8190, fp32, 50 us.
//
// Masked tiles. A key that some row of the CTA does not see may hold anything;
// its score is replaced before use, and its value must not be multiplied by
// that row's 0. In a prompt's steps with such keys two more warps replace the values
// that are not finite by 0 in shared memory and note them; a row that does see one
// gets NaN. (In the softmax warps the same took 6 % longer over packed prompts.) Behind
// the end of a prefix or cache lies what no row sees: the softmax warps write 0 over it.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace qv {

__device__ unsigned int g_attn_prompt_error;

namespace {

constexpr int kPrefixMaxSplits = 64;       // parts of a prefix, and of a cache
constexpr int kKeys = 128;                 // key positions per step
constexpr int kTileRows = 128;             // query rows per tile
constexpr int kFlush = 8;                  // steps O accumulates for fp32 outputs
// The same for bf16 ones, whose rounding hides more: the cuts of 2^20 positions of one sign made them 4.3e-3 too small,
// those of 2^15 are below 1e-4.
constexpr int kFlushLong = 256;
// How far (log2) m lies above the maximum that set it. P is a floating-point number
// and keeps its relative precision; with m above every score the sums overflow no
// earlier than those with a running maximum (a reference that lagged 2^40 behind
// gave infinities for values from 3e26 on), and 2^-8 costs nothing: weights below
// 2^-118 of a row's largest are 0.
constexpr float kRoom = 8.0f;
constexpr int kPolls = 32;                 // of a barrier, before a wait looks at the timer
constexpr float kLog2e = 1.4426950408889634f;

// l of a part without positions, which writes no outputs. (A part whose scores are all -inf has l = 0, and outputs of 0,
// or NaN where a value is not finite.)
constexpr float kNoPositions = -1.0f;

constexpr int kItemBytes = 64;

template <int D, int NT>
struct Layout {
    static constexpr int H = D / 64;                        // 128-byte halves of a row
    static constexpr int Tile = 128 * D * 2;                // bytes of 128 rows
    static constexpr int Stages = D == 128 ? (NT == 2 ? 5 : 6) : 8;
    static constexpr int Q = 0;
    static constexpr int Ring = NT * Tile;
    static constexpr int Bar = Ring + Stages * Tile;
    // barriers: full, empty [Stages], Q full, empty, S full [2], halves of P [2][2], PV done [2], values looked at [8],
    // items full, empty [2], next item, drain
    static constexpr int bEmpty = Stages, bQ = 2 * Stages, bQEmpty = bQ + 1, bS = bQEmpty + 1, bP = bS + 2, bPV = bP + 4,
                         bScan = bPV + 2, bItem = bScan + 8, bItemEmpty = bItem + 2, bNext = bItemEmpty + 2,
                         bDrain = bNext + 1, kBars = bDrain + 1;
    static constexpr int Bad = Bar + (kBars + 1) / 2 * 16;  // keys with values that are not finite [16][4] words
    static constexpr int Items = Bad + 16 * 16;              // what the CTA works on and what comes next
    static constexpr int Next = Items + 2 * kItemBytes;     // the answer to a request for another block's item
    static constexpr int Misc = Next + 16;                  // tensor memory base, abort word
    static constexpr int Bytes = Misc + 16;
    static constexpr int Alloc = Bytes + 1024;              // slack to align the base to 1024 B
    // softmax warps, then a warpgroup with the products', the loads' and two values'
    // warps. With two tiles it hands registers over: 384 threads of 168 become 256 of
    // 216 and 128 of 72
    static constexpr int Warps = NT * 4;
    static constexpr int Threads = Warps * 32 + 128;
    // tensor memory columns: S (P over it) of both tiles or buffers, then O
    static constexpr int kO = 256;
    static constexpr int Cols = 512;
    static_assert(Bar % 8 == 0 && Bad % 16 == 0, "alignment");
    static_assert(Alloc <= (int)kMaxDynSmem, "shared memory budget");
};

struct Maps {
    CUtensorMap q, k, v;      // [rows][heads][D] bf16, boxes 64 x G x TM and 64 x 1 x 128
    CUtensorMap kc, vc;       // [B][Lmax][Hkv][D] bf16, boxes 64 x 1 x 128 x 1
};

struct Args {
    const int32_t* cu;        // prompts: [B + 1] first rows; prefix: [1] its length
    const int32_t* len;       // prefix: [B] cached positions behind it
    int B, T;
    int M;                    // qkv rows
    int G, TM;                // query heads per key/value head, tokens per tile
    int Hkv, Hq;
    int k_head, v_head;       // head index of key/value head 0 in the k and v maps
    int P, Lmax;              // prefix, caches: positions there is room for
    int blocks;               // groups of NT tiles
    int splits, own_splits;   // parts the prefix and a cache are cut into
    float c;                  // scale * log2 e
    void* out;                // prompts: [M][Hq * D]
    float* part_o;            // prefix: [parts][M][Hq][D]
    float2* part_ml;          // prefix: [parts][M][Hq] (m, l)
    int hold;                 // test hook: request no load
    unsigned long long wait_ns;
};

// Shared-memory descriptors, 128-byte swizzle: the high word is the same for all
// (8-row groups 1024 bytes apart, the format's version, the swizzle); the low
// word is the address / 16 and, for V as the N-major B operand (atoms of 64 dims x
// 8 positions), the distance of the next 64 dims, a half of the tile.
constexpr uint32_t kDescHigh = (1024u >> 4) | 1u << 14 | 2u << 29;
constexpr uint32_t kDescK = 1u << 16, kDescV = (16384u >> 4) << 16;
// One K = 16 step of D[tmem] (+)= A B^T, A from shared memory or from tensor
// memory. The whole warp calls, one lane (`lead`) issues: control flow and
// descriptors stay uniform, which a branch on the lane would not leave them.
__device__ __forceinline__ void umma_ss(uint32_t lead, uint32_t d_tmem, uint32_t a_desc, uint32_t b_desc, uint32_t id,
                                        uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "mov.b64 a, {%1, %6};\n\tmov.b64 b, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_desc), "r"(b_desc), "r"(id), "r"(accumulate), "r"(lead), "n"(kDescHigh) : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint32_t b_desc, uint32_t id,
                                        uint32_t accumulate) {
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
                 "mov.b64 b, {%2, %6};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
                 :: "r"(d_tmem), "r"(a_tmem), "r"(b_desc), "r"(id), "r"(accumulate), "r"(lead), "n"(kDescHigh) : "memory");
}
__device__ __forceinline__ void commit(uint32_t lead, uint32_t bar) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
                 :: "r"(bar), "r"(lead) : "memory");
}
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p;
}
// Instruction descriptor of kind::f16 with bf16 operands, M = 128, f32
// accumulator; b_mn: B stored N-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int head, int row,
                                            uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(row), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int head, int pos, int seq,
                                            uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];"
                 :: "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(head), "r"(pos), "r"(seq),
                    "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[16]) {
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
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
// tcgen05.wait::ld that the loaded values pass through, so that no use of them is moved before it.
__device__ __forceinline__ void tmem_ld_done(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                   "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29])
                 :: "memory");
    asm volatile("" : "+r"(v[30]), "+r"(v[31]) :: "memory");
}
__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }

// A wait of at most limit_ns; false (and *abort set, the error noted) when it
// runs out, false at once when another wait has.
__device__ __forceinline__ bool lane_wait(uint64_t* bar, unsigned parity, volatile int* abort,
                                          unsigned long long limit_ns) {
    // reading the timer takes longer than most waits: not before a wait has been a long one
    for (int k = 0; k < kPolls; ++k)
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

// The stage that holds a load, and the parity of its being filled.
struct Slot {
    int s;
    uint32_t parity;
    template <int STAGES>
    __device__ __forceinline__ void advance(int by) {
        s += by;
        if (s >= STAGES) {
            s -= STAGES;
            parity ^= 1;
        }
    }
};

// One piece of work: the tiles' first tokens and the key positions they run over.
struct Item {
    int kh;                   // key/value head, -1: no more work
    int t0;
    int seq;                  // prefix: the sequence whose cache this is, or -1 for the prefix itself
    int part;                 // prefix: the index of the partial results
    int first, end;           // tokens [first, end) are rows to compute
    int k0, k1;               // prefix: the part's positions; prompts: k0 only
    int all_lo;               // where the last row's sequence begins
    int whole, rest;          // in steps [whole, rest) every row sees every key
    int nt[2];                // steps of each tile
};
static_assert(sizeof(Item) <= kItemBytes, "items fit their slots");

// Whether some row of the item does not see some key of step n.
__device__ __forceinline__ bool partly(const Item& it, int n) { return n < it.whole || n >= it.rest; }

// The whole warp calls.
template <int NT, bool PREFIX>
__device__ __forceinline__ Item item_of(const Args& a, int item) {
    Item it;
    it.kh = item % a.Hkv;
    item /= a.Hkv;
    it.seq = -1;
    it.nt[0] = it.nt[1] = 0;
    if (PREFIX) {
        int len, parts, at;
        if (item < a.blocks * a.splits) {
            it.t0 = item % a.blocks * (NT * a.TM);
            it.end = min(it.t0 + NT * a.TM, a.M);
            it.part = at = item / a.blocks;
            len = min(max(a.cu[0], 0), a.P);
            parts = a.splits;
        } else {
            item -= a.blocks * a.splits;
            it.seq = item % a.B;
            it.t0 = it.seq * a.T;
            it.end = it.t0 + a.T;
            at = item / a.B;
            it.part = a.splits + at;
            len = min(max(a.len[it.seq], 0), a.Lmax);
            parts = a.own_splits;
        }
        it.first = it.t0;
        const int tiles = (len + kKeys - 1) / kKeys, per = (tiles + parts - 1) / parts;
        it.k0 = min(at * per, tiles) * kKeys;
        it.k1 = min(len, it.k0 + per * kKeys);
        it.nt[0] = it.k1 > it.k0 ? (it.k1 - it.k0 + kKeys - 1) / kKeys : 0;
        if (NT == 2) it.nt[1] = it.t0 + a.TM < it.end ? it.nt[0] : 0;
        it.all_lo = it.k0;
        it.whole = 0;
        it.rest = (it.k1 - it.k0) / kKeys;
    } else {
        it.part = 0;
        it.t0 = (a.blocks - 1 - item) * (NT * a.TM);          // the last rows, which see most, first
        const int c0 = min(max(a.cu[0], 0), a.M), cB = min(max(a.cu[a.B], 0), a.M);
        it.first = max(it.t0, c0);
        it.end = min(it.t0 + NT * a.TM, cB);
        it.k0 = it.k1 = it.all_lo = it.whole = it.rest = 0;
        if (it.first < it.end) {
            // (the lanes' rows do not fall: the first row in the lower half of the warp, the last in the upper)
            const int start = sequence_start(a.cu, a.B, (threadIdx.x & 16) ? it.end - 1 : it.first);
            it.k0 = __shfl_sync(0xffffffffu, start, 0);
            it.all_lo = __shfl_sync(0xffffffffu, start, 31);
            it.whole = (it.all_lo - it.k0 + kKeys - 1) / kKeys;
            it.rest = (it.first - it.k0 + 1) / kKeys;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int e = min(it.t0 + (i + 1) * a.TM, it.end);
                if (e > max(it.t0 + i * a.TM, it.first)) it.nt[i] = (e - it.k0 + kKeys - 1) / kKeys;
            }
        }
    }
    return it;
}

// Asks for the item of a block of this launch that has not started yet: such a
// block then never starts. The answer arrives at `next` (16 bytes) and `bar`.
__device__ __forceinline__ void request_item(uint32_t next, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 :: "r"(next), "r"(smem_u32(bar)) : "memory");
}
// The block's index, or -1 if none was left.
__device__ __forceinline__ int requested_item(uint32_t next) {
    int item;
    asm volatile("{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 x;\n\tld.shared.b128 h, [%1];\n\t"
                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\tmov.b32 x, -1;\n\t"
                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 x, h;\n\tmov.b32 %0, x;\n\t}"
                 : "=r"(item) : "r"(next) : "memory");
    return item;
}

// Four pieces of 16 bytes of a row in each lane become one piece (lane % 4) of
// the rows of each of four neighbouring lanes: 64 bytes of a row side by side.
__device__ __forceinline__ void transpose4(uint32_t (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int d = 1; d <= 2; d *= 2) {
        const bool up = lane & d;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c & d) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t &x = v[4 * c + j], &y = v[4 * (c + d) + j];
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? x : y, d);
                if (up) x = got; else y = got;
            }
        }
    }
}

// bf16 outputs of long sequences: where a row's outputs go lies the high part of its sums (kept), O has the rest, so
// that the products' cuts are those of a small sum. f: what the row's reference has moved by since `kept` was written,
// 0 before that. The sum of both goes apart again, or, to end with, whole into O. The whole warp calls (kept is null
// in rows that are not computed); out of line, so that the steps' code stays together.
template <int D>
__device__ __noinline__ void carry(uint32_t o_col, uint16_t* kept, float f, bool whole) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        uint32_t o[32], rest[2][16];
        tmem_ld<32>(o_col + c, o);
        tmem_ld_done(o);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint32_t w[4] = {};
            uint4* p = reinterpret_cast<uint4*>(kept + c) + j;
            if (kept && f != 0.f) {
                const uint4 x = *p;
                w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int e = 8 * j + 2 * k;
                float a = __uint_as_float(w[k] << 16) * f + __uint_as_float(o[e]);
                float b = __uint_as_float(w[k] & 0xFFFF0000u) * f + __uint_as_float(o[e + 1]);
                if (!whole) {
                    w[k] = __float_as_uint(a) >> 16 | (__float_as_uint(b) & 0xFFFF0000u);
                    a -= __uint_as_float(w[k] << 16);
                    b -= __uint_as_float(w[k] & 0xFFFF0000u);
                }
                rest[e / 16][e % 16] = __float_as_uint(a);
                rest[e / 16][e % 16 + 1] = __float_as_uint(b);
            }
            if (kept && !whole) *p = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        tmem_st(o_col + c, rest[0]);
        tmem_st(o_col + c + 16, rest[1]);
    }
    tmem_st_wait();
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
    // steps O accumulates, and whether it then starts anew (fp32 sums elsewhere) or goes on with what its high part,
    // kept where the outputs go, leaves
    constexpr int kSteps = PARTS == 2 ? kFlush : kFlushLong;
    constexpr bool kAnew = PREFIX || PARTS == 2;
    constexpr int kMmaWarp = Ly::Warps, kLoadWarp = kMmaWarp + 1, kScanWarp = kMmaWarp + 2;   // two of those

    if (threadIdx.x == 0) {
        for (int s = 0; s < Ly::kBars; ++s) {
            const bool halves = s >= Ly::bP && s < Ly::bP + 4, scan = s >= Ly::bScan && s < Ly::bScan + 8;
            const bool taken = s >= Ly::bItemEmpty && s < Ly::bItemEmpty + 2;
            mbar_init(&bar[s], halves ? 4 : scan ? 2 : taken ? Ly::Warps + (PREFIX ? 1 : 3) : 1);
        }
        for (int i = 0; i < 64; ++i) bad[i] = 0;
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

    // Item k of the CTA, as the loading warp has left it.
    auto take = [&](int k, Item& it) {
        if (!warp_wait(&bar[Ly::bItem + (k & 1)], (k >> 1) & 1, abort, a.wait_ns)) return false;
        it = *reinterpret_cast<const Item*>(smem + Ly::Items + (k & 1) * kItemBytes);
        warp_arrive(&bar[Ly::bItemEmpty + (k & 1)]);
        return it.kh >= 0;
    };

    if (warp >= kMmaWarp) {
    if (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kLoadWarp) {
        // ------------------------------------------------------ items and loads
        if (lane == 0) {
            prefetch_tensormap(&maps.q);
            prefetch_tensormap(&maps.k);
            prefetch_tensormap(&maps.v);
        }
        int cur = blockIdx.x, published = 0, asked = 0;
        int queries = 0, s = 0;                              // s: the next load's stage
        uint32_t round = 0;                                  // times round the ring, as far as they matter: 0, then 1, 2, 1, ...
        bool ok = true;
        while (ok) {
            Item it;
            it.kh = -1;
            it.nt[0] = it.nt[1] = 0;
            if (cur >= 0) it = item_of<NT, PREFIX>(a, cur);
            const int nmax = max(it.nt[0], it.nt[1]);
            if (PREFIX || nmax > 0 || cur < 0) {             // (rows of no sequence: nothing to do)
                if (published >= 2)
                    ok = warp_wait(&bar[Ly::bItemEmpty + (published & 1)], ((published >> 1) - 1) & 1, abort, a.wait_ns);
                if (!ok) break;
                if (lane == 0) {
                    *reinterpret_cast<Item*>(smem + Ly::Items + (published & 1) * kItemBytes) = it;
                    mbar_arrive(&bar[Ly::bItem + (published & 1)]);
                }
                ++published;
            }
            if (cur < 0) break;
            if (lane == 0 && nmax > 0 && !a.hold) {
                if (queries > 0) ok = lane_wait(&bar[Ly::bQEmpty], (queries - 1) & 1, abort, a.wait_ns);
                if (ok) {
                    mbar_arrive_expect_tx(&bar[Ly::bQ], (unsigned)(NT * Ly::H * 128 * a.G * a.TM));
                    for (int i = 0; i < NT; ++i)
                        for (int h = 0; h < Ly::H; ++h)
                            tma_load_3d(sbase + Ly::Q + i * Ly::Tile + h * 16384, &maps.q, 64 * h, it.kh * a.G,
                                        it.t0 + i * a.TM, &bar[Ly::bQ]);
                    ++queries;
                }
                for (int n = 0; ok && n < 2 * nmax; ++n) {   // keys 0, values 0, keys 1, ...
                    if (round > 0) ok = lane_wait(&bar[Ly::bEmpty + s], (round - 1) & 1, abort, a.wait_ns);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&bar[s], Ly::Tile);
                    const uint32_t dst = sbase + Ly::Ring + s * Ly::Tile;
                    const int pos = it.k0 + (n >> 1) * kKeys;
                    if (PREFIX && it.seq >= 0) {
                        for (int h = 0; h < Ly::H; ++h)
                            tma_load_4d(dst + h * 16384, n & 1 ? &maps.vc : &maps.kc, 64 * h, it.kh, pos, it.seq, &bar[s]);
                    } else {
                        for (int h = 0; h < Ly::H; ++h)
                            tma_load_3d(dst + h * 16384, n & 1 ? &maps.v : &maps.k, 64 * h,
                                        (n & 1 ? a.v_head : a.k_head) + it.kh, pos, &bar[s]);
                    }
                    if (++s == Ly::Stages) {
                        s = 0;
                        round = round == 1 ? 2 : 1;
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            // the next item, once all of this one's loads are under way: asked for earlier, the first blocks would
            // take the long items of a short launch for themselves
            if (lane == 0) {
                fence_proxy_async_smem();                    // the last answer has been read
                mbar_arrive_expect_tx(&bar[Ly::bNext], 16);
                request_item(sbase + Ly::Next, &bar[Ly::bNext]);
            }
            ++asked;
            ok = warp_wait(&bar[Ly::bNext], (asked - 1) & 1, abort, a.wait_ns);
            if (ok) cur = requested_item(sbase + Ly::Next);
        }
        // no copy and no answer is in flight when the block ends
        if (lane == 0) {
            const unsigned long long t0 = global_timer_ns();
            auto drain = [&](uint64_t* b, unsigned parity) {
                while (!mbar_try_wait(b, parity) && global_timer_ns() - t0 < 2 * kWaitLimitNs) {
                }
            };
            if (asked > 0) drain(&bar[Ly::bNext], (asked - 1) & 1);
            if (queries > 0) drain(&bar[Ly::bQ], (queries - 1) & 1);
            for (int j = 0; j < Ly::Stages; ++j)             // stages from s on were last filled the time before
                if (j < s || round > 0) drain(&bar[j], (j < s ? round : round - 1) & 1);
        }
    } else if (warp == kMmaWarp) {
        // ----------------------------------------------------------- products
        const uint32_t lead = elect_lane();
        constexpr uint32_t id_s = idesc_bf16(kKeys, false), id_o = idesc_bf16(D, true);
        const uint32_t t0 = __shfl_sync(0xffffffffu, tm, 0);            // uniform, and known to be
        const uint32_t bars = sbase + Ly::Bar, ring = (sbase + Ly::Ring) >> 4;
        auto at = [&](int b) { return bars + 8 * b; };
        Slot next = {0, 0};                                  // the item's first load
        auto wait = [&](int b, uint32_t parity) { return lane_wait(&bar[b], parity, abort, a.wait_ns); };
        auto test = [&](int b, uint32_t parity) { return mbar_test_wait(&bar[b], parity); };
        uint32_t c0 = 0, c1 = 0;                             // steps of the tiles so far
        uint32_t looks = 0;                                  // steps so far: whose values have been looked at
        bool ok = true;
        Item it;
        for (int k_item = 0, q_item = 0; ok && take(k_item, it); ++k_item) {
            const int n0 = __shfl_sync(0xffffffffu, it.nt[0], 0), n1 = NT == 2 ? __shfl_sync(0xffffffffu, it.nt[1], 0) : 0;
            const int nmax = max(n0, n1);
            if (nmax == 0) continue;
            Slot k = next, v = next;
            v.template advance<Ly::Stages>(1);
            // that step looks' values are there, and have been looked at
            auto there = [&](const Slot& v) {
                return PREFIX ? wait(v.s, v.parity) : wait(Ly::bScan + (looks & 7), (looks >> 3) & 1);
            };
            auto scores = [&](int i, int col) {
                const uint32_t q = ((sbase + Ly::Q + i * Ly::Tile) >> 4) | kDescK, kd = (ring + k.s * (Ly::Tile >> 4)) | kDescK;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    umma_ss(lead, t0 + col, q + (kk >> 2) * 1024 + (kk & 3) * 2, kd + (kk >> 2) * 1024 + (kk & 3) * 2, id_s,
                            kk > 0);
            };
            auto outputs = [&](int i, int col, int half, uint32_t add) {
                const uint32_t vd = (ring + v.s * (Ly::Tile >> 4)) | kDescV;
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
#pragma unroll
                    for (int kk = 0; kk < kKeys / 32; ++kk)  // each half of P lies over its half of S
                        umma_ts(lead, t0 + Ly::kO + i * D, t0 + col + half * 64 + part * 32 + kk * 8,
                                vd + (half * 4 + kk) * 128, id_o, half > 0 || part > 0 || kk > 0 ? 1u : add);
            };
            ok = __all_sync(0xffffffffu, wait(Ly::bQ, q_item & 1) && wait(k.s, k.parity));
            ++q_item;
            if (!ok) break;
            tc_fence_after();
            if (NT == 2) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    if ((i ? n1 : n0) > 0) {
                        scores(i, i * 128);
                        commit(lead, at(Ly::bS + i));
                    }
                commit(lead, at(Ly::bEmpty + k.s));
                if (nmax == 1) commit(lead, at(Ly::bQEmpty));
                k.template advance<Ly::Stages>(2);
                bool filled = false;                         // whether values n and keys n + 1 are known to be there
                for (int n = 0; ok && n < nmax; ++n) {
                    if (!filled) {
                        ok = __all_sync(0xffffffffu, there(v) && (n + 1 >= nmax || wait(k.s, k.parity)));
                        if (!ok) break;
                    }
                    ++looks;
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const int ni = i ? n1 : n0;
                        if (!ok || n >= ni) continue;
                        const uint32_t c = (i ? c1 : c0) + n;
                        ok = __all_sync(0xffffffffu, wait(Ly::bP + 2 * i, c & 1));
                        if (!ok) break;
                        tc_fence_after();
                        outputs(i, i * 128, 0, kAnew ? n % kSteps != 0 : n > 0);
                        ok = __all_sync(0xffffffffu, wait(Ly::bP + 2 * i + 1, c & 1));
                        if (!ok) break;
                        tc_fence_after();
                        outputs(i, i * 128, 1, 1);
                        if (n + 1 < ni) scores(i, i * 128);
                        if (i == 1 || n >= n1) {             // the last tile to use these keys and values
                            // a look at the next step's, before the commits wait for the queue of products
                            Slot kn = k, vn = v;
                            kn.template advance<Ly::Stages>(2);
                            vn.template advance<Ly::Stages>(2);
                            const bool vt = PREFIX ? test(vn.s, vn.parity) : test(Ly::bScan + (looks & 7), (looks >> 3) & 1);
                            filled = __all_sync(0xffffffffu, (n + 1 >= nmax || vt) & (n + 2 >= nmax || test(kn.s, kn.parity)));
                        }
                        commit(lead, at(n + 1 < ni ? Ly::bS + i : Ly::bPV + i));
                        if (n + 1 < ni && (i == 1 || n + 1 >= n1)) {
                            commit(lead, at(Ly::bEmpty + k.s));
                            if (n + 2 == nmax) commit(lead, at(Ly::bQEmpty));
                        }
                        if (i == 1 || n >= n1) commit(lead, at(Ly::bEmpty + v.s));
                    }
                    k.template advance<Ly::Stages>(2);
                    v.template advance<Ly::Stages>(2);
                    next.template advance<Ly::Stages>(2);
                }
                c0 += n0;
                c1 += n1;
            } else {
                scores(0, (c0 & 1) * 128);
                commit(lead, at(Ly::bS + (c0 & 1)));
                commit(lead, at(Ly::bEmpty + k.s));
                if (nmax == 1) commit(lead, at(Ly::bQEmpty));
                k.template advance<Ly::Stages>(2);
                for (int n = 0; n < n0; ++n, ++c0) {
                    const int buf = c0 & 1;
                    if (n + 1 < n0) {
                        ok = __all_sync(0xffffffffu, wait(k.s, k.parity));
                        if (!ok) break;
                        scores(0, (buf ^ 1) * 128);
                        commit(lead, at(Ly::bS + (buf ^ 1)));
                        commit(lead, at(Ly::bEmpty + k.s));
                        if (n + 2 == n0) commit(lead, at(Ly::bQEmpty));
                    }
                    // (a barrier for each buffer: a warp may be a step ahead of another)
                    ok = __all_sync(0xffffffffu, there(v) && wait(Ly::bP + 2 * buf, (c0 >> 1) & 1));
                    ++looks;
                    if (!ok) break;
                    tc_fence_after();
                    outputs(0, buf * 128, 0, kAnew ? n % kSteps != 0 : n > 0);
                    ok = __all_sync(0xffffffffu, wait(Ly::bP + 2 * buf + 1, (c0 >> 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    outputs(0, buf * 128, 1, 1);
                    commit(lead, at(Ly::bPV + buf));
                    commit(lead, at(Ly::bEmpty + v.s));
                    k.template advance<Ly::Stages>(2);
                    v.template advance<Ly::Stages>(2);
                    next.template advance<Ly::Stages>(2);
                }
            }
        }
        // nothing reads operands or writes tensor memory when the block ends
        commit(lead, at(Ly::bDrain));
        const unsigned long long now = global_timer_ns();
        while (!mbar_try_wait(&bar[Ly::bDrain], 0) && global_timer_ns() - now < kWaitLimitNs) {
        }
    } else if (!PREFIX) {
        // ---------------------------------------------- values that are not finite
        // In steps with keys that some row does not see: noted by key, then 0 in shared memory. The products wait for
        // these warps in every step, so that the ring is never ahead of them.
        Slot values = {1, 0};                                // the stage of the step's values
        uint32_t looks = 0;
        bool ok = true;
        Item it;
        for (int k_item = 0; ok && take(k_item, it); ++k_item) {
            const int nmax = max(it.nt[0], it.nt[1]);
            for (int n = 0; n < nmax; ++n, ++looks, values.template advance<Ly::Stages>(2)) {
                ok = warp_wait(&bar[values.s], values.parity, abort, a.wait_ns);
                if (!ok) break;
                if (partly(it, n)) {
                    uint32_t* mark = bad + (looks & 15) * 4;
                    const uint32_t at = (warp - kScanWarp) * 32 + lane, v = sbase + Ly::Ring + values.s * Ly::Tile + at * 16;
#pragma unroll 1
                    for (int e0 = 0; e0 < Ly::Tile / 1024; e0 += 8) {
                        uint32_t inf = 0;
#pragma unroll
                        for (int e = e0; e < e0 + 8; ++e) {
                            uint32_t w[4];
                            lds_v4_u32(v + e * 1024, w[0], w[1], w[2], w[3]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) inf |= (w[j] & 0x7F807F80u) + 0x00800080u;   // carries out of all ones
                        }
                        if (!(inf & 0x80008000u)) continue;
#pragma unroll 1
                        for (int e = e0; e < e0 + 8; ++e) {
                            uint32_t w[4];
                            lds_v4_u32(v + e * 1024, w[0], w[1], w[2], w[3]);
                            bool any = false;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                if ((w[j] & 0x7F80u) == 0x7F80u) w[j] &= 0xFFFF0000u, any = true;
                                if ((w[j] & 0x7F800000u) == 0x7F800000u) w[j] &= 0x0000FFFFu, any = true;
                            }
                            if (!any) continue;
                            const int key = (e * 64 + at) >> 3 & 127;        // 8 chunks a row; the halves one behind the other
                            sts_v4_u32(v + e * 1024, w[0], w[1], w[2], w[3]);
                            atomicOr(&mark[key >> 5], 1u << (key & 31));
                        }
                    }
                }
                fence_proxy_async_smem();
                // the marks of eight steps on: those of eight steps ago, whose products, which wait for every row's look at
                // the marks, are done (the ring holds four steps at most)
                if (warp == kScanWarp && lane < 4) bad[((looks + 8) & 15) * 4 + lane] = 0;
                warp_arrive(&bar[Ly::bScan + (looks & 7)]);
            }
        }
    }
    } else {
        // ------------------------------------------------------------ softmax
        if (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int i = NT == 2 ? warp >> 2 : 0, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t o_col = tm + lanes + Ly::kO + i * D;
        const int row_token = r / a.G, row_head = r - row_token * a.G;
        unsigned steps = 0;                                  // of this tile, in the items before
        unsigned looks = 0, ends = 0;                        // steps of both tiles so far; items with steps of this one
        Slot values = {1, 0};                                // prefix: the stage of the item's first values
        bool ok = true;
        Item it;
        for (int k_item = 0; ok && take(k_item, it); ++k_item) {
            const int tok = it.t0 + i * a.TM + row_token, head = it.kh * a.G + row_head;
            const bool valid = r < a.TM * a.G && tok >= it.first && tok < it.end;
            const int nt = NT == 2 && i == 1 ? it.nt[1] : it.nt[0];
            // keys [lo, hi] are seen by this row
            int lo = it.k0, hi = it.k1 - 1;
            if (!PREFIX) {
                hi = min(max(tok, it.first), it.end - 1);
                if (it.all_lo != it.k0) lo = sequence_start(a.cu, a.B, hi);
            }
            const long long row = valid ? (long long)tok * a.Hq + head : -1;         // of the outputs
            float m = neg_inf(), m_acc = neg_inf(), l = 0.f;

            // O, 32 columns at a time, to where fp32 sums or partial results lie: what is there times 2^(m_acc - m)
            // (unless this is the first time) plus O, times mul
            auto flush = [&](bool fresh, float mul) {
                float* acc = PREFIX ? a.part_o + (size_t)it.part * a.M * a.Hq * D : reinterpret_cast<float*>(a.out);
                const float f = (m_acc == neg_inf() ? 0.f : ex2(m_acc - m)) * mul;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t o[2][16];
                    tmem_ld<16>(o_col + c, o[0]);
                    tmem_ld<16>(o_col + c + 16, o[1]);
                    tmem_ld_wait();
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[q][j] = __float_as_uint(__uint_as_float(o[q][j]) * mul);
                        transpose4(o[q]);
                    }
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const int src = (lane & ~3) + t;
                        const long long to = __shfl_sync(0xffffffffu, row, src);
                        const float g = __shfl_sync(0xffffffffu, f, src);
                        if (to < 0) continue;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            float4* p = reinterpret_cast<float4*>(acc + to * D + c + 16 * q) + (lane & 3);
                            float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (!fresh) w = *p;
                            w.x = w.x * g + __uint_as_float(o[q][4 * t]);
                            w.y = w.y * g + __uint_as_float(o[q][4 * t + 1]);
                            w.z = w.z * g + __uint_as_float(o[q][4 * t + 2]);
                            w.w = w.w * g + __uint_as_float(o[q][4 * t + 3]);
                            *p = w;
                        }
                    }
                    __syncwarp();
                }
                m_acc = m;
            };

            // all products of this item's steps before n are done
            auto products_done = [&](int n) {
                const unsigned before = steps + n - 1;
                const bool done = NT == 1  ? warp_wait(&bar[Ly::bPV + (before & 1)], (before >> 1) & 1, abort, a.wait_ns)
                                  : n < nt ? warp_wait(&bar[Ly::bS + i], (before + 1) & 1, abort, a.wait_ns)
                                           : warp_wait(&bar[Ly::bPV + i], ends & 1, abort, a.wait_ns);
                tc_fence_after();
                return done;
            };

            auto carry_on = [&](bool whole) {
                carry<D>(o_col, row < 0 ? nullptr : reinterpret_cast<uint16_t*>(a.out) + row * D,
                         m_acc == neg_inf() ? 0.f : ex2(m_acc - m), whole);
                m_acc = m;
            };

            // (fp32 outputs: one stretch, and a flush every kFlush steps within it)
            for (int n0 = 0; n0 < nt; n0 = PARTS == 2 ? nt : n0 + kFlushLong) {
            if (PARTS == 1 && n0 > 0) {
                ok = products_done(n0);
                if (!ok) break;
                if constexpr (PREFIX)
                    flush(n0 == kFlushLong, 1.f);
                else
                    carry_on(false);
            }
            const int n1 = PARTS == 2 ? nt : min(nt, n0 + kFlushLong);
            for (int n = n0; n < n1; ++n) {
                const unsigned step = steps + n;
                const int buf = NT == 2 ? i : step & 1;
                const uint32_t s_col = tm + lanes + buf * 128;
                const int kb = it.k0 + n * kKeys;
                const bool part = partly(it, n);
                const bool flushed = PARTS == 2 ? n > 0 && n % kFlush == 0 : kAnew && n == n0;
                uint32_t see[4];                             // which of the keys the row sees
                ok = warp_wait(&bar[Ly::bS + buf], (NT == 2 ? step : step >> 1) & 1, abort, a.wait_ns);
                if (!ok) break;
                if (part) {
                    const int from = lo - kb, to = hi - kb;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int f0 = max(from - 32 * q, 0), t0 = min(to - 32 * q, 31);
                        see[q] = f0 <= t0 && f0 < 32 ? 0xFFFFFFFFu >> (31 - t0) >> f0 << f0 : 0u;
                    }
                }
                if (PARTS == 2 && flushed) {
                    if (NT == 1) ok = warp_wait(&bar[Ly::bPV + (buf ^ 1)], ((step - 1) >> 1) & 1, abort, a.wait_ns);
                    if (!ok) break;
                    tc_fence_after();
                    flush(n == kFlush, 1.f);
                }

                // P with the reference so far, or, in rows where a score passes it, with a new one
                bool raise = n == 0;
#pragma unroll 1
                while (true) {
                    uint32_t s[4][32];
                    tc_fence_after();
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld<32>(s_col + 32 * q, s[q]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld_done(s[q]);
                    if (part) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(see[q] >> j & 1u)) s[q][j] = 0xFF800000u;
                    }
                    float mx[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) mx[q] = neg_inf();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            mx[q] = max3(mx[q], __uint_as_float(s[q][2 * j]), __uint_as_float(s[q][2 * j + 1]));
                    const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * a.c;
                    // a row's reference goes by its own scores alone, whatever the rows beside it hold (the shared memory
                    // of a tile that 128 / G tokens do not fill is never written); rows that are not computed have no say
                    const bool above = top > m;
                    if (raise) {
                        const float f = !above ? 1.f : m == neg_inf() ? 0.f : ex2(m - (top + kRoom));
                        if (above) m = top + kRoom;
                        l *= f;
                        if (n > 0 && !flushed) {
                            if (NT == 1) ok = warp_wait(&bar[Ly::bPV + (buf ^ 1)], ((step - 1) >> 1) & 1, abort, a.wait_ns);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c0 = 0; c0 < D; c0 += 8) {
                                uint32_t o[8];
                                tmem_ld<8>(o_col + c0, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                                tmem_st(o_col + c0, o);
                            }
                        }
                    }
                    const float ms = m == neg_inf() ? 0.f : m;   // a row that has seen no key yet
                    const uint64_t c2 = pair(a.c, a.c), m2 = pair(-ms, -ms);
                    const uint64_t minus = pair(-1.f, -1.f);
                    uint64_t l2 = pair(0.f, 0.f), l3 = l2;
                    bool again = false;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t hi2[2][16], lo2[2][16];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float p0, p1;
                                unpair(fma2(pair(__uint_as_float(s[2 * h + q][2 * j]), __uint_as_float(s[2 * h + q][2 * j + 1])),
                                            c2, m2), p0, p1);
                                p0 = ex2(p0);
                                p1 = ex2(p1);
                                const uint32_t x = pack2(p0, p1);
                                hi2[q][j] = x;
                                const uint64_t p = pair(p0, p1);
                                if (PARTS == 2) {
                                    float d0, d1;
                                    unpair(fma2(pair(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)), minus, p),
                                           d0, d1);
                                    lo2[q][j] = pack2(d0, d1);
                                }
                                if (j & 1) l3 = add2(l3, p); else l2 = add2(l2, p);
                            }
                        // (only now, so that the maximum is taken while the exponentials are)
                        if (h == 0 && !raise && __any_sync(0xffffffffu, valid && above)) {
                            again = true;
                            break;
                        }
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            tmem_st(s_col + 64 * h + 16 * q, hi2[q]);
                            if constexpr (PARTS == 2) tmem_st(s_col + 64 * h + 32 + 16 * q, lo2[q]);
                        }
                        if (PREFIX && h == 0 && part) {      // values behind the end, which may be anything, are 0
                            const int at = values.s + 2 * n, turns = at / Ly::Stages, stage = at - turns * Ly::Stages;
                            ok = warp_wait(&bar[stage], (values.parity + turns) & 1, abort, a.wait_ns);
                            if (!ok) break;
#pragma unroll 4
                            for (int e = r; e < Ly::Tile / 16; e += 128)     // 8 chunks a row; the halves one behind the other
                                if ((e >> 3 & 127) >= it.k1 - kb)
                                    sts_v4_u32(sbase + Ly::Ring + stage * Ly::Tile + e * 16, 0u, 0u, 0u, 0u);
                            fence_proxy_async_smem();
                        }
                        if (!PREFIX && h == 1 && part) {     // a row that sees a key whose value is not finite is NaN
                            const unsigned look = looks + n;
                            ok = warp_wait(&bar[Ly::bScan + (look & 7)], (look >> 3) & 1, abort, a.wait_ns);
                            if (!ok) break;
                            const volatile uint32_t* mark = bad + (look & 15) * 4;
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if (mark[w] & see[w]) l = __uint_as_float(0x7FC00000u);
                        }
                        tmem_st_wait();
                        tc_fence_before();
                        warp_arrive(&bar[Ly::bP + 2 * buf + h]);
                    }
                    if (again) {
                        raise = true;
                        continue;
                    }
                    float x0, x1;
                    unpair(add2(l2, l3), x0, x1);
                    l += x0 + x1;
                    break;
                }
                if (!ok) break;
            }
            if (!ok) break;
            }

            // -------------------------------------------------------- outputs
            if (ok && nt > 0) {
                ok = products_done(nt);
                ++ends;
                if (!kAnew && nt > kFlushLong && ok) carry_on(true);
            }
            if (ok && nt > 0) {
                const float inv = PREFIX ? 1.f : 1.f / l;
                if constexpr (kAnew) {
                    flush(nt <= kSteps, inv);
                    if (PREFIX && valid) a.part_ml[(size_t)it.part * a.M * a.Hq + row] = make_float2(m, l);
                } else {
#pragma unroll 1
                    for (int c = 0; c < D; c += 32) {
                        uint32_t o[32], w[16];
                        tmem_ld<32>(o_col + c, o);
                        tmem_ld_done(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            w[j] = pack2(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
                        transpose4(w);
#pragma unroll
                        for (int t = 0; t < 4; ++t) {
                            const long long to = __shfl_sync(0xffffffffu, row, (lane & ~3) + t);
                            if (to >= 0)
                                *(reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + to * D + c) + (lane & 3)) =
                                    make_uint4(w[4 * t], w[4 * t + 1], w[4 * t + 2], w[4 * t + 3]);
                        }
                        __syncwarp();
                    }
                }
            } else if (PREFIX && valid && nt == 0) {
                a.part_ml[(size_t)it.part * a.M * a.Hq + row] = make_float2(neg_inf(), kNoPositions);
            }
            tc_fence_before();
            steps += nt;
            const int nmax = max(it.nt[0], it.nt[1]);
            looks += nmax;
            const int at = values.s + 2 * nmax, turns = at / Ly::Stages;
            values.s = at - turns * Ly::Stages;
            values.parity = (values.parity + turns) & 1;
        }
    }
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tm, Ly::Cols);
    }
}

// The parts' results over the prefix and the caches, and the step's own keys, of
// which there are few, become a row's outputs. Of few rows a block takes one: its
// first warp the own keys, the others every third part, so that the chain is two
// loads deep however many parts there are. Of many rows a warp takes one, with
// less to do in all. One pass of qv_attention_verify_prefix, block against warp: 252 rows
// of 27 parts 11.4 and 14.8 us, 1024 rows of 21 33.0 and 34.9, 3840 rows of 11 59
// and 54, 4096 rows of 10 163 and 160.
constexpr int kMergeWarps = 4;
constexpr int kMergeFewRows = 2048;
struct MergeArgs {
    const uint16_t* qkv;
    const float* part_o;
    const float2* part_ml;
    int parts, rows;          // rows: B * T * Hq
    int T, Hq, Hkv;
    float c;
    void* out;
    int out_bf16;
};
// Sums with a reference of their own: outputs (N values a lane) and l (a lane's
// share), times 2^-top; top is -inf where nothing lies above it (o and l then 0 or
// NaN as they are).
template <int N>
struct Sums {
    float o[N], l, top;
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int x = 0; x < N; ++x) o[x] = 0.f;
        l = 0.f;
        top = neg_inf();
    }
    // The lanes' highest, and the reference it gives.
    __device__ __forceinline__ float reference() {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        return top == neg_inf() ? 0.f : top;
    }
};
__device__ __forceinline__ float weight(float top, float of) { return top == neg_inf() ? 1.f : ex2(top - of); }

// Row w over the step's own keys: scores and products in binary32.
template <int D>
__device__ __forceinline__ void merge_own(const MergeArgs& a, int w, Sums<D / 32>& r) {
    constexpr int N = D / 32;
    constexpr int kOwn = kTileRows / 32;                      // own scores of a lane: up to 128 tokens
    const int lane = threadIdx.x & 31;
    const int tok = w / a.Hq, head = w - tok * a.Hq, first = tok / a.T * a.T, own = tok - first + 1;
    const size_t W = (size_t)(a.Hq + 2 * a.Hkv) * D;
    const uint16_t* key = a.qkv + (size_t)first * W + (size_t)(a.Hq + head / (a.Hq / a.Hkv)) * D + lane * N;
    const uint16_t* val = key + (size_t)a.Hkv * D;
    auto load = [&](const uint16_t* p, float (&x)[N]) {
        uint32_t v[N / 2];
        if constexpr (N == 4) {
            const uint2 t = *reinterpret_cast<const uint2*>(p);
            v[0] = t.x;
            v[1] = t.y;
        } else {
            v[0] = *reinterpret_cast<const uint32_t*>(p);
        }
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            x[2 * j] = __uint_as_float(v[j] << 16);
            x[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
    };
    r.clear();
    float q[N], s[kOwn];
    load(a.qkv + (size_t)tok * W + (size_t)head * D + lane * N, q);
#pragma unroll
    for (int u = 0; u < kOwn; ++u) {
        s[u] = neg_inf();
#pragma unroll 4
        for (int j = 32 * u; j < min(own, 32 * u + 32); ++j) {
            float k[N], d = 0.f;
            load(key + (size_t)j * W, k);
#pragma unroll
            for (int x = 0; x < N; ++x) d += q[x] * k[x];
#pragma unroll
            for (int x = 16; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
            if (j - 32 * u == lane) s[u] = d * a.c;
        }
        r.top = fmaxf(r.top, s[u]);
    }
    const float ref = r.reference();
#pragma unroll
    for (int u = 0; u < kOwn; ++u) {
        if (32 * u >= own) break;
        const float f = 32 * u + lane < own ? ex2(s[u] - ref) : 0.f;
        r.l += f;
#pragma unroll 4
        for (int j = 32 * u; j < min(own, 32 * u + 32); ++j) {
            const float g = __shfl_sync(0xffffffffu, f, j - 32 * u);
            float v[N];
            load(val + (size_t)j * W, v);
#pragma unroll
            for (int x = 0; x < N; ++x) r.o[x] += g * v[x];
        }
    }
}

// Row w over the parts at, at + STEP, ...
template <int D, int STEP>
__device__ __forceinline__ void merge_parts(const MergeArgs& a, int w, int at, Sums<D / 32>& r) {
    constexpr int N = D / 32;
    constexpr int kParts = (2 * kPrefixMaxSplits + STEP * 32 - 1) / (STEP * 32);
    constexpr int kAhead = 8;
    const int lane = threadIdx.x & 31, count = (a.parts - at + STEP - 1) / STEP;
    r.clear();
    float2 ml[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
        const int j = 32 * u + lane;
        ml[u] = make_float2(neg_inf(), kNoPositions);
        if (j < count) ml[u] = a.part_ml[(size_t)(at + j * STEP) * a.rows + w];
        r.top = fmaxf(r.top, ml[u].x);
    }
    const float ref = r.reference();
#pragma unroll
    for (int u = 0; u < kParts; ++u) {
        if (32 * u >= count) break;
        const bool none = ml[u].y == kNoPositions;
        const float f = none ? 0.f : ex2(ml[u].x - ref);
        if (!none) r.l += f * ml[u].y;
        const unsigned there = __ballot_sync(0xffffffffu, !none);
        // kAhead parts' values are requested before the first is used
        for (int j0 = 0; j0 < min(count - 32 * u, 32); j0 += kAhead) {
            float v[kAhead][N];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
#pragma unroll
                for (int x = 0; x < N; ++x) v[j][x] = 0.f;
                if (!(there >> (j0 + j) & 1u)) continue;
                const float* p = a.part_o + ((size_t)(at + (32 * u + j0 + j) * STEP) * a.rows + w) * D + lane * N;
                if constexpr (N == 4) {
                    const float4 t = *reinterpret_cast<const float4*>(p);
                    v[j][0] = t.x, v[j][1] = t.y, v[j][2] = t.z, v[j][3] = t.w;
                } else {
                    const float2 t = *reinterpret_cast<const float2*>(p);
                    v[j][0] = t.x, v[j][1] = t.y;
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const float g = __shfl_sync(0xffffffffu, f, j0 + j);
#pragma unroll
                for (int x = 0; x < N; ++x) r.o[x] += g * v[j][x];
            }
        }
    }
}

template <int D, bool FEW>
__global__ void __launch_bounds__(kMergeWarps * 32) prefix_merge_kernel(const MergeArgs a) {
    constexpr int N = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    allow_dependent_launch();
    grid_dependency_wait();
    auto sum = [](float l) {
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
        return l;
    };
    Sums<N> r;
    if constexpr (FEW) {
        __shared__ float s_o[kMergeWarps][D];
        __shared__ float2 s_ml[kMergeWarps];
        const int w = blockIdx.x;
        if (warp == 0)
            merge_own<D>(a, w, r);
        else
            merge_parts<D, kMergeWarps - 1>(a, w, warp - 1, r);
        r.l = sum(r.l);
        if (lane == 0) s_ml[warp] = make_float2(r.top, r.l);
#pragma unroll
        for (int x = 0; x < N; ++x) s_o[warp][lane * N + x] = r.o[x];
        __syncthreads();
        const int d = threadIdx.x;
        if (d >= D) return;
        float m = neg_inf(), num = 0.f, den = 0.f;
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) m = fmaxf(m, s_ml[k].x);
#pragma unroll
        for (int k = 0; k < kMergeWarps; ++k) {
            const float f = weight(s_ml[k].x, m);
            num += f * s_o[k][d];
            den += f * s_ml[k].y;
        }
        if (a.out_bf16)
            static_cast<__nv_bfloat16*>(a.out)[(size_t)w * D + d] = __float2bfloat16_rn(num / den);
        else
            static_cast<float*>(a.out)[(size_t)w * D + d] = num / den;
    } else {
        const long long w = (long long)blockIdx.x * kMergeWarps + warp;
        if (w >= a.rows) return;
        Sums<N> own;
        merge_own<D>(a, (int)w, own);
        merge_parts<D, 1>(a, (int)w, 0, r);
        const float m = fmaxf(r.top, own.top), f = weight(r.top, m), g = weight(own.top, m);
        const float inv = 1.f / (sum(r.l) * f + sum(own.l) * g);
#pragma unroll
        for (int x = 0; x < N; ++x) r.o[x] = (r.o[x] * f + own.o[x] * g) * inv;
        if (a.out_bf16) {
            uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) + (size_t)w * D + lane * N);
#pragma unroll
            for (int x = 0; x < N / 2; ++x) p[x] = pack2(r.o[2 * x], r.o[2 * x + 1]);
        } else {
            float* p = static_cast<float*>(a.out) + (size_t)w * D + lane * N;
#pragma unroll
            for (int x = 0; x < N; ++x) p[x] = r.o[x];
        }
    }
}

template <int D, bool FEW>
cudaError_t launch_merge(const MergeArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(FEW ? a.rows : ceil_div(a.rows, kMergeWarps));
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, prefix_merge_kernel<D, FEW>, a);
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

// Tiles a CTA takes. Two share every key tile they read and hide each other's
// softmax, one has twice the items to spread: better while every SM has two at
// most. Heads of 128, 32/8 heads, bf16 outputs, one tile against two: 1000 rows
// 17.9 and 20.9 us, 1200 rows (304 tiles) 20.9 and 23.9, 1500 rows 28.3 and 27.5,
// 2043 rows 42.0 and 34.6; heads of 64, 12/4 heads, 2500 rows (240 tiles) 25.2 and 32.8.
int tiles_per_cta(long long tiles, int Hkv, int sms) { return tiles * Hkv > 2 * sms ? 2 : 1; }

}  // namespace

int attention_prompt_tokens(int G) { return kTileRows / G; }

cudaError_t launch_attention_prompt(const CUtensorMap& q, const CUtensorMap& kv, const int32_t* cu, int B, int M, int Hq,
                                    int Hkv, int D, float scale, void* out, bool out_bf16, int sms, int hold,
                                    unsigned long long wait_ns, cudaStream_t s) {
    Maps maps;
    maps.q = q;
    maps.k = maps.v = maps.kc = maps.vc = kv;
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

// How the work of a batch behind a prefix is cut: enough parts of the prefix that
// every SM has one; enough of each cache that every SM has one, or up to four of
// at least three steps, so that a long cache among short ones does not end last.
struct PrefixCut {
    int nt, blocks, splits, own_max;
};
static PrefixCut prefix_cut(int B, int T, int Hq, int Hkv, int P, int sms) {
    PrefixCut c;
    const int M = B * T, TM = attention_prompt_tokens(Hq / Hkv), tiles = ceil_div(M, TM);
    c.nt = tiles >= 2 ? 2 : 1;
    c.blocks = ceil_div(tiles, c.nt);
    const long long items = (long long)c.blocks * Hkv, own = (long long)B * Hkv;
    auto clamp = [](long long n, long long hi) { return (int)(n < 1 ? 1 : n > hi ? hi : n); };
    c.splits = clamp(sms / items, P < kKeys * kPrefixMaxSplits ? ceil_div(P, kKeys) : kPrefixMaxSplits);
    const long long even = 4ll * sms / own < 4 ? 4ll * sms / own : 4;
    c.own_max = clamp(sms / own > even ? sms / own : even, kPrefixMaxSplits);
    return c;
}

size_t attention_prefix_workspace_bytes(int B, int T, int Hq, int Hkv, int D, int P, int sms) {
    const PrefixCut c = prefix_cut(B, T, Hq, Hkv, P, sms);
    return (size_t)(c.splits + c.own_max) * B * T * Hq * (D * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attention_prefix(const PrefixCall& c, int sms, int hold, unsigned long long wait_ns, cudaStream_t s) {
    const PrefixCut cut = prefix_cut(c.B, c.T, c.Hq, c.Hkv, c.P, sms);
    Maps maps;
    maps.q = c.q;
    maps.k = c.pk;
    maps.v = c.pv;
    maps.kc = c.kc;
    maps.vc = c.vc;
    Args a = {};
    a.cu = c.prefix_len; a.len = c.cache_len;
    a.B = c.B; a.T = c.T; a.M = c.B * c.T;
    a.G = c.Hq / c.Hkv; a.TM = attention_prompt_tokens(a.G);
    a.Hkv = c.Hkv; a.Hq = c.Hq; a.P = c.P; a.Lmax = c.Lmax;
    a.blocks = cut.blocks; a.splits = cut.splits;
    // parts of one step where there are SMs for them, else of three
    const int steps = ceil_div(c.Lmax, kKeys), parts = sms >= (long long)c.B * c.Hkv * steps ? steps : ceil_div(steps, 3);
    a.own_splits = parts < cut.own_max ? parts : cut.own_max;
    a.c = c.scale * kLog2e;
    a.hold = hold; a.wait_ns = wait_ns ? wait_ns : kWaitLimitNs;
    a.part_o = static_cast<float*>(c.ws);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)(a.splits + a.own_splits) * a.M * a.Hq * c.D);
    const long long grid = ((long long)a.blocks * a.splits + (long long)c.B * a.own_splits) * c.Hkv;
    cudaError_t e = dispatch<true>(maps, a, c.D, cut.nt, c.out_bf16 ? 1 : 2, (int)grid, s);
    if (e != cudaSuccess) return e;
    MergeArgs m;
    m.qkv = c.qkv; m.part_o = a.part_o; m.part_ml = a.part_ml;
    m.parts = a.splits + a.own_splits; m.rows = a.M * c.Hq;
    m.T = c.T; m.Hq = c.Hq; m.Hkv = c.Hkv;
    m.c = a.c; m.out = c.out; m.out_bf16 = c.out_bf16 ? 1 : 0;
    if (m.rows <= kMergeFewRows) return c.D == 128 ? launch_merge<128, true>(m, s) : launch_merge<64, true>(m, s);
    return c.D == 128 ? launch_merge<128, false>(m, s) : launch_merge<64, false>(m, s);
}

cudaError_t read_and_clear_attn_prompt_error(unsigned* code) {
    cudaError_t e = cudaMemcpyFromSymbol(code, g_attn_prompt_error, sizeof(unsigned));
    if (e != cudaSuccess) return e;
    const unsigned zero = 0;
    return cudaMemcpyToSymbol(g_attn_prompt_error, &zero, sizeof(unsigned));
}

}  // namespace qv
