// k_logprobs.cu -- log probability of one given token per row of logits, the
// row's entropy, and its K most probable tokens.
//
//   The verifier's logits stay in high precision for the acceptance test
//   (gist.science/it summary, section 2 item 3); a server reports the emitted
//   tokens' log probabilities from the same logits.
//
// With m = max_v x_v, z_v = (x_v - m) log2 e, S = sum 2^z_v, T = sum z_v 2^z_v:
//   log p_v = (x_v - m) - ln S,   H = ln S - ln 2 * T / S.
// One pass over the row: each thread keeps its own running m, S and T and
// rescales the sums when m has grown by d (Run): S *= 2^-d, T = 2^-d (T - d S).
// The alternatives cost the pass nothing more: m is also the thread's largest
// logit. Of 32 of these maxima (the two largest of each of 16 warps; with 4 warps
// the largest of every 4 lanes) the K-th largest, tau, is a lower bound of the
// K-th largest logit, and few more than K threads reach it. Only those threads'
// entries (1/512 or 1/128 of the slice each) are read again, from L2, and the
// entries at or above tau are ordered by counting, for each, those before it (by
// value, then by the lower index). Where ties or masks leave too many of them,
// warps keep sorted lists of 32 instead.
//
// A row is the work of one CTA (of 512 threads, or 128 for many short rows), or
// of a cluster of C that split it (launch_token_logprobs): each sends its
// statistics, its entries at or above its own tau and its largest maxima to the
// first, which takes a tau of the whole row from the latter before it counts. One
// cluster barrier in all.
//
// Bound by memory when there are many rows (GB300: 2000 rows of 151936 fp32
// logits with their 5 most probable tokens 194 us, 6.3 TB/s; a plain copy runs
// at 6.8) and by the chain of loads, reductions and barriers when there are few
// (5 such rows with 20 tokens each 7.0 us).

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "qv_internal.h"
#include "qv_ptx.cuh"

namespace cg = cooperative_groups;

namespace qv {
namespace {

constexpr int kLpThreads = 512;                 // of a CTA that has a long row, or a part of it
constexpr int kLpSmall = 128;                   // of a CTA that has a short one (launch_token_logprobs)
constexpr int kLpMaxCluster = 16;
constexpr int kLpUnroll = 4;                    // vectors in flight per thread
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kLpTops = 64;                     // maxima of a row that the CTAs of a cluster send, kLpTops / C each
// Entries of a row ordered by counting (of a CTA of a cluster: 1 / kLpMaxCluster of that).
__host__ __device__ constexpr int lp_cand(int threads) { return threads == kLpThreads ? 1024 : 256; }
static_assert(lp_cand(kLpThreads) / kLpMaxCluster >= 32 && lp_cand(kLpThreads) >= kLpThreads &&
              lp_cand(kLpSmall) >= kLpSmall, "a CTA's K entries and its warps' lists of 32 fit");

struct LpArgs {
    const uint8_t* x;          // logits [M][V]
    const int32_t* tok;        // [M]
    int V, K;
    float* logprob;            // [M]
    float* entropy;            // [M] or null
    int32_t* top_tok;          // [M][K]
    float* top_lp;             // [M][K]
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The larger of the two, NaN if either is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Running statistics of some entries: their maximum (-inf for none), and the
// sums S and T relative to it.
struct Stat {
    float m, S, T;
};
__device__ __forceinline__ Stat combine(Stat a, Stat b) {
    const float m = fmaxf(a.m, b.m);
    // a part with no probability (S == 0: nothing above -inf) adds nothing
    const float da = a.S == 0.f ? 0.f : (a.m - m) * kLog2e, db = b.S == 0.f ? 0.f : (b.m - m) * kLog2e;
    const float fa = ex2(max_nan(da, -150.f)), fb = ex2(max_nan(db, -150.f));
    Stat r;
    r.m = m;
    r.S = a.S * fa + b.S * fb;
    r.T = (fa == 0.f ? 0.f : fa * (a.T + da * a.S)) + (fb == 0.f ? 0.f : fb * (b.T + db * b.S));
    return r;
}

// A thread's running statistics: as Stat, but S and T relative to `ref`, which
// lags up to kLpLag behind the maximum m. A ref that followed every new maximum
// would rescale S up to once every group of entries of a rising row, 2^-22 off
// each time. Where a maximum lies more than kLpLag above the rest, ref is the
// maximum itself: S is 1 and a certain token's log probability 0, never above.
//
// Entries are added group by group (16 or 32 of them). A plain sum of n groups is
// off by up to n 2^-24; Exact keeps what the additions lost (Kahan) for rows of
// more than kLpPlain entries. With one running sum and no lag log probabilities
// of 2^22 logits a row were off by up to 8e-5, now by 1e-6. GB300, us without /
// with the second sums: 2000 rows of 151936 bf16 logits 129/131, of 60000 71/73,
// fp32 194/196, 1 row of 32003 bf16 6.1/6.4.
constexpr float kLpLag = 8.f;
constexpr int kLpPlain = 1 << 19;               // 68 groups of a thread at most
template <bool Exact>
struct Run {
    float m, ref, S, T, cS, cT;                                // (-inf and -inf before the first entry, then zeros)
    // S and T relative to `to`, ref or more.
    __device__ __forceinline__ void move(float to) {
        const float d = (ref - to) * kLog2e;                   // -inf on the first entries (S = T = 0)
        const float f = ex2(d);
        T = f == 0.f ? 0.f : f * (T + d * S);
        S *= f;
        if (Exact) {
            cT = f == 0.f ? 0.f : f * (cT + d * cS);
            cS *= f;
        }
        ref = to;
    }
    static __device__ __forceinline__ void add(float& sum, float& lost, float x) {
        if (Exact) {
            const float y = x - lost, t = sum + y;
            lost = (t - sum) - y;
            sum = t;
        } else {
            sum += x;
        }
    }
    template <int N>
    __device__ __forceinline__ void entries(const float (&v)[N]) {
        float mx = v[0];
#pragma unroll
        for (int i = 1; i < N; ++i) mx = fmaxf(mx, v[i]);
        m = fmaxf(m, mx);
        if (mx > ref + kLpLag) move(mx);
        // nothing above -inf yet: subtract 0, so that -inf entries count 0
        const float r = ref < -3.4028235e38f ? 0.f : ref;
        constexpr int P = N < 4 ? N : 4;                       // the group's own sums, in P parts
        float s[P], t[P];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float z = max_nan((v[i] - r) * kLog2e, -150.f);   // 2^-150 is 0 in binary32; keeps 0 * z finite
            const float e = ex2(z);
            s[i % P] = i < P ? e : s[i % P] + e;
            t[i % P] = i < P ? z * e : t[i % P] + z * e;
        }
#pragma unroll
        for (int n = P / 2; n > 0; n >>= 1)
#pragma unroll
            for (int i = 0; i < n; ++i) {
                s[i] += s[i + n];
                t[i] += t[i + n];
            }
        add(S, cS, s[0]);
        add(T, cT, t[0]);
    }
    __device__ __forceinline__ Stat stat() {                   // relative to m
        if (m > ref) move(m);
        return Exact ? Stat{m, S - cS, T - cT} : Stat{m, S, T};
    }
};

// A key that orders entries by value, then by the lower index; 0 is below all.
// -0 counts as +0. (A NaN's key is 1: below every number's.)
__device__ __forceinline__ unsigned long long entry_key(float v, int idx) {
    if (v != v) return 1ull;
    const uint32_t u = __float_as_uint(v + 0.f);
    const uint32_t o = u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
    return ((unsigned long long)o << 32) | (uint32_t)~(uint32_t)idx;
}
__device__ __forceinline__ float key_value(unsigned long long k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

// The 32 largest of two descending lists, descending; `o` is the other list
// reversed (lane i holds its entry 31 - i).
template <class T>
__device__ __forceinline__ T warp_merge_desc(T v, T o) {
    const int lane = threadIdx.x & 31;
    v = o > v ? o : v;                                         // bitonic, and the 32 largest of both
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const T p = __shfl_xor_sync(0xffffffffu, v, j);
        v = (lane & j) == 0 ? (p > v ? p : v) : (p < v ? p : v);
    }
    return v;
}
// Merges the descending lists of warps 0..n-1 (n a power of two) into warp
// 0's. All threads of the CTA call it.
template <class T>
__device__ __forceinline__ T block_merge_desc(T v, T* sm /* [n][32] */, int n) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int h = n >> 1; h > 0; h >>= 1) {
        if (warp >= h && warp < 2 * h) sm[warp * 32 + lane] = v;
        __syncthreads();
        if (warp < h) v = warp_merge_desc(v, sm[(warp + h) * 32 + 31 - lane]);
    }
    return v;
}

template <bool BF16>
struct Row {
    static constexpr int E = BF16 ? 8 : 4;      // entries of a 16-byte vector
    const uint8_t* p;
    int head, nvec, tail;                       // leading single entries, vectors, trailing single entries

    __device__ Row(const uint8_t* x, size_t row, int V) {
        p = x + row * (size_t)V * (BF16 ? 2 : 4);
        const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15u);
        head = min(V, ((16 - off) & 15) / (BF16 ? 2 : 4));
        nvec = (V - head) / E;
        tail = V - head - nvec * E;
    }
    __device__ __forceinline__ float at(int i) const {
        if (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
        return reinterpret_cast<const float*>(p)[i];
    }
    __device__ __forceinline__ uint4 vec(int n) const {
        return reinterpret_cast<const uint4*>(p + (size_t)head * (BF16 ? 2 : 4))[n];
    }
    static __device__ __forceinline__ void unpack(const uint4& u, float* v) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (BF16) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
                v[i] = __uint_as_float(w[i]);
            }
        }
    }
    // The single entry thread t of the row's first CTA owns, or -1.
    __device__ __forceinline__ int single(int t) const {
        if (t < head) return t;
        if (t >= 16 && t < 16 + tail) return head + nvec * E + (t - 16);
        return -1;
    }
};

__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }

// Inserts the keys of the lanes where `want` holds into the warp's descending
// list (lane i holds the i-th).
__device__ __forceinline__ void warp_insert(unsigned long long& list, unsigned long long key, bool want) {
    const int lane = threadIdx.x & 31;
    unsigned who = __ballot_sync(0xffffffffu, want);
    while (who) {
        const unsigned long long k = __shfl_sync(0xffffffffu, key, __ffs(who) - 1);
        who &= who - 1;
        const int pos = __popc(__ballot_sync(0xffffffffu, list > k));
        const unsigned long long up = __shfl_up_sync(0xffffffffu, list, 1);
        list = lane < pos ? list : (lane == pos ? k : up);
    }
}

// Visits the entries that thread t of the CTA owns, 32 vectors at a time (the
// whole warp calls it): fn(value, index, there).
template <int Threads, bool BF16, class F>
__device__ __forceinline__ void for_thread(const Row<BF16>& r, int t, bool first_cta, int v0, int v1, F&& fn) {
    constexpr int E = Row<BF16>::E;
    const int lane = threadIdx.x & 31;
    const int one = first_cta ? r.single(t) : -1;
    if (one >= 0) fn(r.at(one), one, lane == 0);
    for (int base = v0 + t; base < v1; base += 32 * Threads) {
        const int vn = base + lane * Threads;
        float v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) v[e] = 0.f;
        if (vn < v1) Row<BF16>::unpack(r.vec(vn), v);
#pragma unroll
        for (int e = 0; e < E; ++e) fn(v[e], r.head + vn * E + e, vn < v1);
    }
}

template <bool BF16, int Threads, bool Exact>
__global__ void __launch_bounds__(Threads, Threads == kLpThreads ? 2 : 10) token_logprobs_kernel(const LpArgs a) {
    constexpr int Warps = Threads / 32, Cand = lp_cand(Threads);
    constexpr bool Clusters = Threads == kLpThreads;           // CTAs of short rows have theirs to themselves
    constexpr int E = Row<BF16>::E;
    __shared__ Stat s_stat[Warps];
    // written by every CTA of the row (in its first CTA)
    __shared__ Stat c_stat[kLpMaxCluster];
    __shared__ float c_top[kLpTops];
    __shared__ unsigned long long c_keys[Clusters ? Cand : 1];
    __shared__ int c_n[kLpMaxCluster];
    __shared__ unsigned long long s_keys[Cand];             // entries, or the warps' lists
    __shared__ float s_top[32], s_sorted[32];
    __shared__ int s_who[Threads];
    __shared__ int s_n, s_m;
    __shared__ float s_tau, s_max, s_ls;
    cg::cluster_group cluster = cg::this_cluster();
    const int C = Clusters ? (int)cluster.num_blocks() : 1, rank = Clusters ? (int)cluster.block_rank() : 0;
    if (C > 1) cluster_arrive_relaxed();                       // waited for before the first store into another CTA
    allow_dependent_launch();
    grid_dependency_wait();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float NEG_INF = -__uint_as_float(0x7F800000u);
    const size_t row = blockIdx.x / C;
    const Row<BF16> r(a.x, row, a.V);
    const int per = (r.nvec + C - 1) / C;
    const int v0 = min(r.nvec, rank * per), v1 = min(r.nvec, v0 + per);
    if (tid == 0) s_n = s_m = 0;
    // the given token's logit, early: its two loads hide behind the pass
    const int tok = rank == 0 && tid == Threads - 32 ? a.tok[row] : -1;
    const bool in_range = tok >= 0 && tok < a.V;
    const float x_tok = in_range ? r.at(tok) : 0.f;

    // ---- the pass
    Run<Exact> run = {NEG_INF, NEG_INF, 0.f, 0.f, 0.f, 0.f};
    const int own1 = rank == 0 ? r.single(tid) : -1;
    const float x_own = own1 >= 0 ? r.at(own1) : 0.f;
    if (own1 >= 0) {
        const float v[1] = {x_own};
        run.entries(v);
    }
    int n = v0 + tid;
    for (; n + (kLpUnroll - 1) * Threads < v1; n += kLpUnroll * Threads) {
        uint4 u[kLpUnroll];
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) u[i] = r.vec(n + i * Threads);
        float v[kLpUnroll * E];
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) Row<BF16>::unpack(u[i], v + i * E);
        run.entries(v);
    }
    for (; n < v1; n += Threads) {
        float v[E];
        Row<BF16>::unpack(r.vec(n), v);
        run.entries(v);
    }
    Stat st = run.stat();
    const float mine = st.m;

    // ---- each warp's statistics and two largest maxima, then the CTA's
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        Stat o;
        o.m = __shfl_xor_sync(0xffffffffu, st.m, off);
        o.S = __shfl_xor_sync(0xffffffffu, st.S, off);
        o.T = __shfl_xor_sync(0xffffffffu, st.T, off);
        st = combine(st, o);
    }
    if (a.K > 0) {
        if constexpr (Warps == 16) {                           // the two largest of a warp
            const unsigned at = __ballot_sync(0xffffffffu, mine == st.m);
            float second = lane == __ffs(at) - 1 ? NEG_INF : mine;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) second = fmaxf(second, __shfl_xor_sync(0xffffffffu, second, off));
            if (lane == 0) {
                s_top[warp] = st.m;
                s_top[16 + warp] = second;
            }
        } else {                                               // the largest of every Warps lanes
            float top = mine;
#pragma unroll
            for (int off = 1; off < Warps; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            if (lane % Warps == 0) s_top[(warp * 32 + lane) / Warps] = top;
        }
    }
    if (lane == 0) s_stat[warp] = st;
    __syncthreads();
    auto reduce16 = [&](const Stat* p, int count) {            // in a fixed order; the same in every lane
        Stat c = lane < count ? p[lane] : Stat{NEG_INF, 0.f, 0.f};
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
            Stat o;
            o.m = __shfl_xor_sync(0xffffffffu, c.m, off);
            o.S = __shfl_xor_sync(0xffffffffu, c.S, off);
            o.T = __shfl_xor_sync(0xffffffffu, c.T, off);
            c = combine(c, o);
        }
        return c;
    };
    // The place of p[i] among N numbers (Threads / N threads a number, all of
    // which get it); ties by the index.
    auto place_of = [&](const float* p, int N, int& i) {
        const int G = Threads / N;                          // threads a number
        i = tid / G;
        const float v = p[i];
        int before = 0;
        for (int j = tid % G; j < N; j += G) before += (p[j] > v || (p[j] == v && j < i)) ? 1 : 0;
        for (int off = 1; off < G; off <<= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
        return before;
    };
    Stat c = {NEG_INF, 0.f, 0.f};
    if (warp == Warps - 1) c = reduce16(s_stat, Warps);     // (the last warp's lane 0 finishes a row of one CTA)
    int total = 0;
    if (a.K > 0) {
        {
            int i;
            const int place = place_of(s_top, 32, i);
            if (tid % (Threads / 32) == 0) s_sorted[place] = s_top[i];
        }
        __syncthreads();
        const float tau = s_sorted[a.K - 1];

        // ---- the entries at or above tau
        const int cap = C > 1 ? Cand / kLpMaxCluster : Cand;
        if (mine >= tau) {
            s_who[atomicAdd(&s_m, 1)] = tid;                   // (the order of the list does not matter)
            if (own1 >= 0 && x_own >= tau) {
                const int p = atomicAdd(&s_n, 1);
                if (p < cap) s_keys[p] = entry_key(x_own, own1);
            }
        }
        __syncthreads();
        const int who = s_m, each = (v1 - v0 + Threads - 1) / Threads;   // vectors of a thread
        for (int i = tid; i < who * each; i += Threads) {
            const int f = i / each, vn = v0 + s_who[f] + (i - f * each) * Threads;
            if (vn >= v1) continue;
            float v[E];
            Row<BF16>::unpack(r.vec(vn), v);
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (v[e] >= tau) {
                    const int p = atomicAdd(&s_n, 1);
                    if (p < cap) s_keys[p] = entry_key(v[e], r.head + vn * E + e);
                }
        }
        __syncthreads();
        total = s_n;
        if (total > cap) {                                     // ties or masks: the K first by sorted lists
            unsigned long long list = 0;
            for (int i = warp; i < who; i += Warps)
                for_thread<Threads>(r, s_who[i], rank == 0, v0, v1, [&](float v, int idx, bool there) {
                    const bool in = there && v >= tau;
                    if (!__any_sync(0xffffffffu, in)) return;
                    const unsigned long long k = in ? entry_key(v, idx) : 0ull;
                    const unsigned long long least = __shfl_sync(0xffffffffu, list, a.K - 1);
                    warp_insert(list, k, in && k > least);
                });
            list = block_merge_desc(list, s_keys, Warps);
            __syncthreads();
            if (warp == 0) s_keys[lane] = list;
            total = a.K;                                       // (cap >= 32 entries were there)
            __syncthreads();
        }
    }
    if (C > 1) {                                               // into the first CTA
        cluster_wait();                                        // every CTA of the cluster has started
        const int part = Cand / kLpMaxCluster, tops = kLpTops / C;
        if (tid == Threads - 32) *cluster.map_shared_rank(c_stat + rank, 0) = c;
        if (a.K > 0) {
            if (tid < total) *cluster.map_shared_rank(c_keys + rank * part + tid, 0) = s_keys[tid];
            if (tid >= 64 && tid < 64 + tops) *cluster.map_shared_rank(c_top + rank * tops + tid - 64, 0) = s_sorted[tid - 64];
            if (tid == 0) *cluster.map_shared_rank(c_n + rank, 0) = total;
        }
        cluster.sync();                                        // every push has landed
        if (rank != 0) return;
        if (warp == Warps - 1) c = reduce16(c_stat, C);
        if (a.K > 0) {
            int i;
            const int place = place_of(c_top, kLpTops, i);
            if (place == a.K - 1 && tid % (Threads / kLpTops) == 0) s_tau = c_top[i];
            if (tid == 0) s_n = 0;
            __syncthreads();
            const unsigned long long least = entry_key(s_tau, 0x7FFFFFFF);
            for (int e = tid; e < C * part; e += Threads)
                if (e % part < c_n[e / part] && c_keys[e] >= least) s_keys[atomicAdd(&s_n, 1)] = c_keys[e];
        }
    }
    if (tid == Threads - 32) {
        const bool none = c.m == NEG_INF;                      // every entry is -inf (or NaN, and then S is NaN)
        s_max = none ? 0.f : c.m;
        s_ls = none ? c.S : logf(c.S);
        a.logprob[row] = in_range ? (x_tok - s_max) - s_ls : 0.f;   // tokens outside the vocabulary (padding) count 0
        if (a.entropy) {
            const float h = none ? s_ls : s_ls - kLn2 * (c.T / c.S);
            a.entropy[row] = h < 0.f ? 0.f : h;                // (rounding below 0)
        }
    }
    if (a.K == 0) return;
    __syncthreads();
    if (C > 1) total = s_n;
    // ---- an entry's place is the number of entries before it
    const size_t o = row * (size_t)a.K;
    for (int e = tid; e < total; e += Threads) {
        const unsigned long long key = s_keys[e];
        int place = 0;
#pragma unroll 8
        for (int i = 0; i < total; ++i) place += s_keys[i] > key ? 1 : 0;
        if (place < a.K) {
            a.top_tok[o + place] = (int32_t)~(uint32_t)key;
            a.top_lp[o + place] = (key_value(key) - s_max) - s_ls;
        }
    }
    if (tid >= total && tid < a.K) {                           // a row with fewer numbers than K
        a.top_tok[o + tid] = -1;
        a.top_lp[o + tid] = __uint_as_float(0x7FC00000u);
    }
}

}  // namespace

cudaError_t launch_token_logprobs(const void* x, bool bf16, const int32_t* tok, int M, int V, int K, float* logprob,
                                  float* entropy, int32_t* top_tok, float* top_lp, int sms, cudaStream_t s) {
    LpArgs a;
    a.x = static_cast<const uint8_t*>(x);
    a.tok = tok; a.V = V; a.K = K; a.logprob = logprob; a.entropy = entropy; a.top_tok = top_tok; a.top_lp = top_lp;
    // Many short rows: CTAs of 128 threads, ten an SM. A row's reductions and
    // barriers are then most of its time, and overlap. GB300, 20 tokens, us with
    // 512 / 128 threads: fp32: 600 rows of 3245 9.6/6.2 (300: 5.3/5.5), 2000 of 8000
    // 32/18, of 16000 44/33, 1200 of 32003 37.8/39.6 (600: 15.3/21.5), 2000 of 65000
    // 102/152, of 151936 221/349; bf16: 3859 of 3245 57/24, 600 10.2/6.8 (300:
    // 5.6/6.0), 2000 of 8000 34/17, of 16000 39/24, of 32003 53/41, 1200 of 32003
    // 27.6/24.4 (600: 14.3/17.5), 2000 of 60000 71/77, of 151936 129/193.
    const bool small = V <= (1 << 15) && M > 2 * sms * (V >> 13 > 1 ? V >> 13 : 1);
    int C = 1;
    while (!small && C < kLpMaxCluster && (long long)M * C * 2 <= 2 * sms && V / (C * 2) >= 2 * kLpThreads * (bf16 ? 8 : 4)) C *= 2;
    auto kernel = small ? (bf16 ? token_logprobs_kernel<true, kLpSmall, false> : token_logprobs_kernel<false, kLpSmall, false>)
                : V <= kLpPlain ? (bf16 ? token_logprobs_kernel<true, kLpThreads, false> : token_logprobs_kernel<false, kLpThreads, false>)
                                : (bf16 ? token_logprobs_kernel<true, kLpThreads, true> : token_logprobs_kernel<false, kLpThreads, true>);
    if (C > 8) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(M * C));
    cfg.blockDim = dim3(small ? kLpSmall : kLpThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace qv
