// kda_logprobs.cu -- log probabilities of given tokens, with rank, entropy and the most likely tokens.
//
// Of a row of logits x and z = scale * x:   lse = log sum exp z,   logprob = z_t - lse,
//     entropy = lse - sum p z,   rank = place of t in the order (x descending, lowest index first),
// and the first `top` tokens of that order.
//
// One pass over the row.  Each thread takes its exponents relative to a reference, its warp's first step's maximum m (a
// later one where a term would pass 2^6: a rescaling whenever one lane of a warp meets a larger maximum took nearly half of
// the instructions, and terms up to 2^60, which fp32 has the room for, left the entropy of a sharp row up to 2^-18 off: it is
// the difference of two numbers as large as the exponent), and keeps the sum of e^(z - z_m), the same sum weighted by the
// exponents, and the count of elements ahead of the given token; they are joined by the usual rescaling.
// Exponents are in powers of two, y = x c - r with c = scale * log2 e and the reference r = m c rounded: r is a number
// like any other, so its rounding is no error.  Where that rounding is no longer small, from 2^20 on (rows of a type's
// lowest value alone), y = (x - m) c.
// An element costs about five instructions (maxima and clamps of bf16 two at a time, sums two at a time); the count of
// those ahead only where a step's maximum reaches the given token.
//
// The most likely tokens cost the pass little: each thread leaves the maximum of every step of its own.  The `top` pairs of
// threads with the largest maxima hold all of the `top` largest elements (an element of another pair has `top` maxima above
// it), so the smallest of those maxima bounds them, and only the steps that reach it are read again.
//
// A cluster of C CTAs serves a row, each a contiguous slice of it: its sums and its sorted list go into the shared memory
// of the first, which joins them.
//
// Measured in a graph: 2048 rows of 131072 bf16, 1 alternative: 112 us, 4.8 TB/s; 256 rows of 100003, 8: 22.4 us; 4 rows of
// 131072 fp32, 20: 9.3 us.  The pass alone runs at 6.2 TB/s; the rest is what follows it in each CTA, a chain of steps of a
// few thousand clocks (sums, order of the maxima, the steps read again, order of what they hold).
#include <cfloat>
#include <cuda_bf16.h>
#include "common.cuh"
#include "tc.cuh"

namespace kda {

constexpr int kLogThreads = 256, kLogWarps = kLogThreads / 32, kLogGroups = kLogThreads / 2, kLogMaxTop = 32, kLogSteps = 24;
constexpr int kLogFew = 64, kLogKeep = 1024, kLogHits = 1024, kLogMaxCluster = 8;
constexpr float kLogAbove = 6.f;                 // powers of two that a term may be above its reference
constexpr int kStatusToken = -1;                 // KDA_ERR_INVALID_ARG, recorded on the device
using LogKey = unsigned long long;               // a value's order bits, then its index negated; 0: none

__device__ __forceinline__ float log_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {    // NaN if either is
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
}
// Bits that order like the values (-0 like 0), and back.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t o) { return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu)); }
__device__ __forceinline__ LogKey log_key(uint32_t order, int i) { return static_cast<LogKey>(order) << 32 | static_cast<uint32_t>(~i); }

// Sums of a part of a row relative to the reference of one of its elements, m (NaN or infinite where the part holds such
// a one): sum 2^y, sum 2^y y.
struct LogSums { float m, s, w; };
// m times c as the reference that exponents are taken from; from 2^20 on m itself is, and c multiplies differences.
__device__ __forceinline__ bool log_wide(float m, float c) { return fabsf(m * c) >= 0x1p20f && fabsf(m) < INFINITY; }
__device__ __forceinline__ float log_gap(float m, float to, float c) {         // reference of m less the reference of `to`
    if (log_wide(m, c) || log_wide(to, c)) return (m - to) * c;
    return __fmul_rn(m, c) - __fmul_rn(to, c);
}
__device__ __forceinline__ LogSums log_move(LogSums a, float m, float c) {     // the same relative to a larger maximum
    if (!(a.s > 0.f)) return LogSums{m, 0.f, 0.f};
    const float d = fmaxf(log_gap(a.m, m, c), -200.f), f = log_ex2(d);
    return LogSums{m, a.s * f, f * fmaf(d, a.s, a.w)};
}
// The sums of the lanes of a warp, joined: relative to the largest maximum, each moved there once.
__device__ __forceinline__ LogSums log_warp(LogSums a, float c) {
    const bool bad = __any_sync(0xffffffffu, a.m != a.m);
    const float m = from_order(__reduce_max_sync(0xffffffffu, order_bits(a.m)));
    LogSums x = log_move(a, m, c);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        x.s += __shfl_xor_sync(0xffffffffu, x.s, off);
        x.w += __shfl_xor_sync(0xffffffffu, x.w, off);
    }
    if (bad) x.m = __int_as_float(0x7fffffff);
    return x;
}

template <typename T> struct LogVec;             // a chunk of 16 bytes
template <> struct LogVec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    __device__ static __forceinline__ float one(const float* p) { return __ldg(p); }
    __device__ static __forceinline__ void unpack(uint4 v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
    template <int U> __device__ static __forceinline__ float top(const uint4 (&v)[U]) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[4];
            unpack(v[u], x);
            m = max_nan(max_nan(max_nan(m, x[0]), x[1]), max_nan(x[2], x[3]));
        }
        return m;
    }
    // how many of them are above x0, or not below it
    template <bool EQ, int U> __device__ static __forceinline__ int ahead(const uint4 (&v)[U], float x0) {
        int n = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[4];
            unpack(v[u], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) n += EQ ? x[i] >= x0 : x[i] > x0;
        }
        return n;
    }
    // the elements, none below `low`
    __device__ static __forceinline__ void above(uint4 v, float low, float (&x)[4]) {
        unpack(v, x);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = fmaxf(x[i], low);
    }
};
template <> struct LogVec<uint16_t> {
    static constexpr int N = 8;
    __device__ static __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ static __forceinline__ float one(const uint16_t* p) { return bf16_bits_to_f32(__ldg(p)); }
    __device__ static __forceinline__ void unpack(uint4 v, float (&x)[8]) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = bf16x2_bits_to_f32(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
    template <int U> __device__ static __forceinline__ float top(const uint4 (&v)[U]) {
        uint32_t m = max_nan2(max_nan2(v[0].x, v[0].y), max_nan2(v[0].z, v[0].w));
#pragma unroll
        for (int u = 1; u < U; ++u) m = max_nan2(m, max_nan2(max_nan2(v[u].x, v[u].y), max_nan2(v[u].z, v[u].w)));
        const float2 f = bf16x2_bits_to_f32(m);
        return max_nan(f.x, f.y);
    }
    template <bool EQ, int U> __device__ static __forceinline__ int ahead(const uint4 (&v)[U], float x0) {
        const __nv_bfloat162 l = __float2bfloat162_rn(x0);      // (x0 is one of them)
        __nv_bfloat162 n = __float2bfloat162_rn(0.f);           // (counts up to 256 are exact)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
                n = __hadd2(n, EQ ? __hge2(x, l) : __hgt2(x, l));
            }
        }
        return static_cast<int>(__low2float(n) + __high2float(n));
    }
    __device__ static __forceinline__ void above(uint4 v, float low, float (&x)[8]) {
        const uint32_t h = __bfloat16_as_ushort(__float2bfloat16_rd(low)), l = h | h << 16;      // (down: it must not reach m)
        unpack(make_uint4(max2(v.x, l), max2(v.y, l), max2(v.z, l), max2(v.w, l)), x);
    }
};

struct LogArgs {
    const void* x; long long ld;
    const int32_t* tok;
    int V, top, C;
    float scale, c;                              // c = scale * log2 e
    float* logprob; int32_t* rank; float* entropy;
    float* top_lp; int32_t* top_tok;
    int* status;
};

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, LogKey v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" :: "r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, float a, float b, float c, int d) {
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};"
                 :: "r"(addr), "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(d) : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kLogThreads, 4)
kda_logprobs_kernel(const LogArgs a)
{
    using Vec = LogVec<T>;
    constexpr int N = Vec::N, U = 4;             // U chunks a thread and step, loaded together
    __shared__ __align__(16) float4 s_part[kLogMaxCluster];             // of the row's slices: m, s, w, count
    __shared__ LogKey s_lists[kLogMaxCluster][kLogMaxTop];
    __shared__ LogSums s_sum[kLogWarps];
    __shared__ int s_cnt[kLogWarps];
    __shared__ __align__(16) LogKey s_key[kLogGroups];
    __shared__ __align__(16) uint32_t s_val[kLogGroups];
    __shared__ int s_rank[kLogGroups];
    __shared__ float s_step[kLogSteps][kLogThreads];                    // maxima of each thread's steps, or of several
    __shared__ LogKey s_keep[kLogKeep];
    __shared__ int s_hit[kLogHits];                                     // steps to read again: a thread's first chunk of each
    __shared__ LogKey s_list[kLogMaxTop];
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ LogKey s_least, s_next;
    __shared__ LogSums s_all;
    __shared__ int s_count, s_hits, s_ok;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int C = a.C, rank = C > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    const long long rw = blockIdx.x / static_cast<unsigned>(C);
    const T* row = static_cast<const T*>(a.x) + rw * a.ld;
    const int top = a.top;
    const int t = a.tok ? a.tok[rw] : 0;
    if (a.tok && (t < 0 || t >= a.V)) {          // padding, or a token that is none (the same in every CTA of the cluster)
        if (rank != 0) return;
        if (tid == 0) {
            if (t >= a.V) set_status(a.status, kStatusToken);
            a.logprob[rw] = 0.f;
            if (a.rank) a.rank[rw] = 0;
            if (a.entropy) a.entropy[rw] = 0.f;
        }
        if (tid < top) {
            a.top_lp[rw * top + tid] = -INFINITY;
            a.top_tok[rw * top + tid] = -1;
        }
        return;
    }
    if (C > 1) {                                 // the first CTA's barrier is up before the others arrive on it
        if (tid == 0) {
            tc::mbar_init(&s_bar, 32 * C);
            tc::mbar_fence_init();
        }
        __syncthreads();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }
    const float xt = Vec::one(row + t), c = a.c;
    // the row's whole chunks of 16 bytes, `per` of them in this CTA; and its ends, a few single elements, in the first
    const int head = min(a.V, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(row) & 15u)) % 16u / sizeof(T)));
    const int all_chunks = (a.V - head) / N, per = (all_chunks + C - 1) / C;
    const int begin = min(rank * per, all_chunks), chunks = min(per, all_chunks - begin);
    const int first = head + begin * N;                                    // element of this CTA's chunk 0
    const uint4* body = reinterpret_cast<const uint4*>(row + first);
    const int tail = head + all_chunks * N, singles = rank == 0 ? head + a.V - tail : 0;
    auto single = [&](int i) { return i < head ? i : tail + i - head; };   // element of single i

    // 1. the pass: thread t takes chunks t, t + 256, ..
    float m = -INFINITY, r = 0.f, low = -1e30f;          // reference m c; what is below `low` counts as that much (2^-150 is 0)
    float lim = -INFINITY;                               // another reference from here on
    bool wide = false;
    float2 s2 = make_float2(0.f, 0.f), w2 = s2;
    int cnt = 0, at = 0;                         // at: step of U chunks where the largest element was met first
    float largest = -INFINITY;
    const float inv = 1.f / c;
    auto raise = [&](float b) {
        const float old = m;
        m = max_nan(m, b);
        const LogSums x = log_move(LogSums{old, s2.x, w2.x}, m, c), y = log_move(LogSums{old, s2.y, w2.y}, m, c);
        s2 = make_float2(x.s, y.s);
        w2 = make_float2(x.w, y.w);
        wide = log_wide(m, c);
        r = fabsf(m) < INFINITY && !wide ? __fmul_rn(m, c) : 0.f;
        low = fabsf(m) < INFINITY ? __fsub_rd(m, 160.f * inv) : -1e30f;
        lim = fmaf(kLogAbove, inv, m);
    };
    constexpr int kStep = U * kLogThreads;       // chunks a step
    const int fold = ((chunks + kStep - 1) / kStep + kLogSteps - 1) / kLogSteps;         // steps that share a place of s_step
    int slot = 0, left = fold;
    float held = -INFINITY;
#pragma unroll 1
    for (int k0 = 0; k0 < chunks; k0 += kStep) {
        uint4 v[U];
        const int k = k0 + tid;
        if (k0 + kStep <= chunks) {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = __ldg(body + k + u * kLogThreads);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = k + u * kLogThreads < chunks ? __ldg(body + k + u * kLogThreads) : Vec::nothing();
        }
        const float b = Vec::template top<U>(v);
        held = fmaxf(held, b);
        s_step[slot][tid] = held;
        if (--left == 0) {
            left = fold;
            ++slot;
            held = -INFINITY;
        }
        if (b > largest) {
            largest = b;
            at = k0;
        }
        const float top = k0 > 0 ? b : from_order(__reduce_max_sync(0xffffffffu, order_bits(b)));
        if (!(top <= lim)) raise(top);           // (a NaN is above everything, and stays)
        if (!wide) {
            const float2 c2 = make_float2(c, c), r2 = make_float2(-r, -r);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[N];
                Vec::above(v[u], low, x);
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float2 y = ffma2(make_float2(x[i], x[i + 1]), c2, r2), e = make_float2(log_ex2(y.x), log_ex2(y.y));
                    s2 = fadd2(s2, e);
                    w2 = ffma2(e, y, w2);
                }
            }
        } else {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                float x[N];
                Vec::unpack(k + u * kLogThreads < chunks ? __ldg(body + k + u * kLogThreads) : Vec::nothing(), x);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float y = fmaxf((x[i] - m) * c, -150.f), e = log_ex2(y);
                    s2.x += e;
                    w2.x = fmaf(e, y, w2.x);
                }
            }
        }
        if (b >= xt) {
            if (k0 + kStep <= chunks && first + (k0 + kStep) * N <= t) {
                cnt += Vec::template ahead<true, U>(v, xt);
            } else if (first + k0 * N > t) {
                cnt += Vec::template ahead<false, U>(v, xt);
            } else {
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    if (k + u * kLogThreads >= chunks) break;
                    float x[N];
                    Vec::unpack(__ldg(body + k + u * kLogThreads), x);
                    const int i0 = first + (k + u * kLogThreads) * N;
#pragma unroll
                    for (int i = 0; i < N; ++i) cnt += x[i] > xt || (x[i] == xt && i0 + i < t);
                }
            }
        }
    }
    const uint32_t mv = tid < chunks ? order_bits(largest) : 0u;           // of the chunks alone
    if (tid < singles) {
        const int i = single(tid);
        const float x = Vec::one(row + i);
        if (!(x <= lim)) raise(x);
        const float y = wide ? fmaxf((x - m) * c, -150.f) : fmaf(fmaxf(x, low), c, -r), e = log_ex2(y);
        s2.x += e;
        w2.x = fmaf(e, y, w2.x);
        cnt += x > xt || (x == xt && i < t);
    }

    // 2. the slice's sums; the groups' maxima (a group without elements has 0, below every value)
    {
        // (a thread that saw -inf alone has taken those for 2^y at y = low c: no sum)
        LogSums part{m, m == -INFINITY ? 0.f : s2.x + s2.y, m == -INFINITY ? 0.f : w2.x + w2.y};
        part = log_warp(part, c);
        const int wcnt = __reduce_add_sync(0xffffffffu, cnt);
        if (lane == 0) { s_sum[warp] = part; s_cnt[warp] = wcnt; }
    }
    const uint32_t gv = max(mv, __shfl_xor_sync(0xffffffffu, mv, 1));
    if ((tid & 1) == 0) { s_val[tid >> 1] = gv; s_rank[tid >> 1] = 0; }
    if (tid == 0) s_count = s_hits = 0;
    if (tid < kLogMaxTop) s_list[tid] = 0;
    __syncthreads();
    if (warp == 0) {
        const LogSums part = log_warp(lane < kLogWarps ? s_sum[lane] : LogSums{-INFINITY, 0.f, 0.f}, c);
        const int ahead = __reduce_add_sync(0xffffffffu, lane < kLogWarps ? s_cnt[lane] : 0);
        if (lane == 0) {
            s_all = part;
            s_part[0] = make_float4(part.m, part.s, part.w, __int_as_float(ahead));
        }
    }

    if (top > 0) {
        // 3. the groups in the order of their maxima (equal ones by number): a thread compares one with half of them
        const int g = tid & (kLogGroups - 1), q0 = tid / kLogGroups * (kLogGroups / 2);
        {
            const uint32_t v = s_val[g];
            int above = 0;
#pragma unroll
            for (int i = 0; i < kLogGroups / 2; i += 4) {
                const uint4 o = *reinterpret_cast<const uint4*>(s_val + q0 + i);
                above += (o.x > v || (o.x == v && q0 + i < g)) + (o.y > v || (o.y == v && q0 + i + 1 < g)) +
                         (o.z > v || (o.z == v && q0 + i + 2 < g)) + (o.w > v || (o.w == v && q0 + i + 3 < g));
            }
            atomicAdd(&s_rank[g], above);
        }
        __syncthreads();
        if (tid < kLogGroups && s_rank[tid] == top - 1) s_least = s_val[tid];
        __syncthreads();
        // the groups at or above the `top`-th hold what is looked for; where many share its value, they are taken by key:
        // value, then lowest index
        const uint32_t least = static_cast<uint32_t>(s_least);
        const bool on = tid < kLogGroups && s_val[tid] >= least && s_val[tid] != 0;
        const int many = __syncthreads_count(on);
        if (many <= kLogFew) {
            if (tid == 0) s_least = log_key(least, 0x7fffffff);          // (below every key of that value)
        } else {
            LogKey key = 0;
            if (mv != 0 && mv == gv && gv >= least) {                    // this thread's first element of that value
#pragma unroll 1
                for (int u = 0; u < U && key == 0; ++u) {
                    const int k = at + tid + u * kLogThreads;
                    if (k >= chunks) break;
                    float x[N];
                    Vec::unpack(__ldg(body + k), x);
#pragma unroll
                    for (int i = N - 1; i >= 0; --i)
                        if (order_bits(x[i]) == mv) key = log_key(mv, first + k * N + i);
                }
            }
            __syncwarp();
            const LogKey o = __shfl_xor_sync(0xffffffffu, key, 1);
            key = key > o ? key : o;
            if ((tid & 1) == 0) { s_key[tid >> 1] = key; s_rank[tid >> 1] = 0; }
            __syncthreads();
            const LogKey v = s_key[g];
            int above = 0;
            if (v) {
#pragma unroll
                for (int i = 0; i < kLogGroups / 2; ++i) above += s_key[q0 + i] > v;
                atomicAdd(&s_rank[g], above);
            }
            if (tid == 0) s_least = 0;
            __syncthreads();
            if (tid < kLogGroups && s_key[tid] && s_rank[tid] == top - 1) s_least = s_key[tid];
        }
        __syncthreads();

        // 4. the elements at or above that, put in order by counting.  Only elements beside each other in a few threads can make
        // them many; then one after another is looked for instead
        const LogKey bound = s_least;
        const float reach = from_order(static_cast<uint32_t>(bound >> 32));
        auto scan = [&](auto&& use) {
#pragma unroll 1
            for (int z = 0; z * fold * kStep + tid < chunks; ++z) {
                if (s_step[z][tid] < reach) continue;
#pragma unroll 1
                for (int k0 = z * fold * kStep + tid; k0 < min((z + 1) * fold * kStep, chunks); k0 += kStep) {
                    uint4 v[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) v[u] = k0 + u * kLogThreads < chunks ? __ldg(body + k0 + u * kLogThreads) : Vec::nothing();
#pragma unroll 1
                    for (int u = 0; u < U; ++u) {
                        const uint4 one[1] = {u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3]};
                        const int k = k0 + u * kLogThreads;
                        if (k >= chunks || Vec::template top<1>(one) < reach) continue;
                        float e[N];
                        Vec::unpack(one[0], e);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            const LogKey y = log_key(order_bits(e[i]), first + k * N + i);
                            if (y >= bound) use(y);
                        }
                    }
                }
            }
            if (tid < singles) {
                const LogKey y = log_key(order_bits(Vec::one(row + single(tid))), single(tid));
                if (y >= bound) use(y);
            }
        };
        auto keep = [&](LogKey e) {
            const int i = atomicAdd(&s_count, 1);
            if (i < kLogKeep) s_keep[i] = e;
        };
        // the steps that reach it, first, then their chunks a thread each: one latency for all of them (each thread its own, one
        // after another, 2048 rows of 131072, 20 alternatives: 163 us to 137, caches flushed)
#pragma unroll 4
        for (int z = 0; z * fold * kStep + tid < chunks; ++z) {
            if (s_step[z][tid] < reach) continue;
            for (int k0 = z * fold * kStep + tid; k0 < min((z + 1) * fold * kStep, chunks); k0 += kStep) {
                const int i = atomicAdd(&s_hits, 1);
                if (i < kLogHits) s_hit[i] = k0;
            }
        }
        __syncthreads();
        const int hits = s_hits;
        if (hits <= kLogHits) {
            for (int i = tid; i < hits * U; i += kLogThreads) {
                const int k = s_hit[i / U] + i % U * kLogThreads;
                if (k >= chunks) continue;
                const uint4 one[1] = {__ldg(body + k)};
                if (Vec::template top<1>(one) < reach) continue;
                float e[N];
                Vec::unpack(one[0], e);
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    const LogKey y = log_key(order_bits(e[j]), first + k * N + j);
                    if (y >= bound) keep(y);
                }
            }
            if (tid < singles) {
                const LogKey y = log_key(order_bits(Vec::one(row + single(tid))), single(tid));
                if (y >= bound) keep(y);
            }
        } else {
            scan(keep);
        }
        __syncthreads();
        const int n = s_count;
        if (n <= kLogKeep) {
            for (int i = tid; i < n; i += kLogThreads) {
                const LogKey e = s_keep[i];
                int above = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) above += s_keep[j] > e;
                if (above < top) s_list[above] = e;
            }
        } else {
            LogKey last = ~0ull;
            for (int i = 0; i < top; ++i) {
                if (tid == 0) s_next = 0;
                __syncthreads();
                LogKey best = 0;
                scan([&](LogKey e) { if (e < last && e > best) best = e; });
                if (best) atomicMax(&s_next, best);
                __syncthreads();
                last = s_next;
                if (tid == 0) s_list[i] = last;
                __syncthreads();
            }
        }
    }
    __syncthreads();

    // 5. the slices' sums and lists, joined by the first CTA
    if (C > 1) {
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (warp == 0) {
            const LogKey e = lane < top ? s_list[lane] : 0;
            const float4 p = s_part[0];
            if (rank != 0) {
                st_cluster_u64(tc::mapa(tc::smem_u32(&s_lists[rank][lane]), 0), e);
                if (lane == 0) st_cluster_v4(tc::mapa(tc::smem_u32(&s_part[rank]), 0), p.x, p.y, p.z, __float_as_int(p.w));
            } else {
                s_lists[0][lane] = e;
            }
            tc::mbar_arrive_remote(tc::mapa(tc::smem_u32(&s_bar), 0));
        }
        if (rank != 0) return;
        if (warp == 0) {
            bool came = tc::mbar_wait_cluster_bounded(&s_bar, 0, kWaitLimitNs);
            came = __all_sync(0xffffffffu, came);
            const float4 p = came && lane < C ? s_part[lane] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
            const LogSums part = log_warp(LogSums{p.x, p.y, p.z}, c);
            const int ahead = __reduce_add_sync(0xffffffffu, __float_as_int(p.w));
            // at least `top` elements are not below the smallest of the slices' `few`-th largest: only those are put in order
            const int few = (top + C - 1) / C;
            const uint32_t v = top > 0 && came && lane < C ? static_cast<uint32_t>(s_lists[lane][few - 1] >> 32) : 0xffffffffu;
            const uint32_t least = __reduce_min_sync(0xffffffffu, v);
            if (lane == 0) {
                s_all = part;
                s_part[0].w = __int_as_float(ahead);
                s_least = static_cast<LogKey>(least) << 32;
                s_count = 0;
                s_ok = came;
                if (!came) set_status(a.status, kStatusTimeout);
            }
        }
        __syncthreads();
        if (!s_ok) {                             // (the others may still write here: not before they have left)
            tc::cluster_sync();
            return;
        }
        if (top > 0) {
            const LogKey bound = s_least;
            for (int i = tid; i < C * kLogMaxTop; i += kLogThreads) {
                const LogKey e = s_lists[i / kLogMaxTop][i % kLogMaxTop];
                if (e != 0 && e >= bound) s_keep[atomicAdd(&s_count, 1)] = e;
            }
            __syncthreads();
            const int n = s_count;
            if (tid < kLogMaxTop) s_list[tid] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += kLogThreads) {
                const LogKey e = s_keep[i];
                int above = 0;
#pragma unroll 4
                for (int j = 0; j < n; ++j) above += s_keep[j] > e;
                if (above < top) s_list[above] = e;
            }
            __syncthreads();
        }
    }

    // 6. the row's answers
    const LogSums all = s_all;
    const bool none = !(all.m < INFINITY);       // a NaN or +inf in the row
    const float nan = __int_as_float(0x7fffffff), ln2 = 0.69314718055994531f;
    const bool far = log_wide(all.m, c);
    const float l2 = log2f(all.s), ref = far || !(fabsf(all.m) < INFINITY) ? 0.f : __fmul_rn(all.m, c);
    auto log_prob = [&](float x) {               // (a row of -inf alone: no token has a probability; a difference may pass 2^128)
        return x == -INFINITY ? -INFINITY : far || log_wide(x, c) ? fmaf(2.f * a.scale, 0.5f * x - 0.5f * all.m, -l2 * ln2)
                                          : (fmaf(x, c, -ref) - l2) * ln2;
    };
    if (tid == 0) {
        if (a.tok) {
            a.logprob[rw] = none ? nan : log_prob(xt);
            if (a.rank) a.rank[rw] = none ? 0 : 1 + __float_as_int(s_part[0].w);
        }
        if (a.entropy) a.entropy[rw] = none ? nan : all.s > 0.f ? (l2 - all.w / all.s) * ln2 : 0.f;
    }
    if (tid < top) {
        const LogKey e = s_list[tid];
        a.top_lp[rw * top + tid] = none ? nan : e == 0 ? -INFINITY : log_prob(from_order(static_cast<uint32_t>(e >> 32)));
        a.top_tok[rw * top + tid] = none || e == 0 ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(e));
    }
}

// CTAs a row: as many as run at once, of slices that a step or more of every thread takes.  (2048 rows of 131072 bf16, 1, 2, 4
// CTAs a row: 112, 134, 176 us; 256 of 100003: 23.1, 22.4, 30.1; 4 of 131072 fp32, 1, 2, 4, 8: 21.0, 15.2, 11.3, 9.3)
int logprobs_cluster(int R, int V, int sms, int bytes) {
    int C = 1;
    while (C < kLogMaxCluster && static_cast<long long>(R) * 2 * C <= 4 * sms && V / (2 * C) * bytes >= 16384) C *= 2;
    return C;
}

int launch_token_logprobs(const void* x, int f32, long long ld, const int32_t* tok, int R, int V, int top, float scale,
                          float* logprob, int32_t* rank, float* entropy, float* top_lp, int32_t* top_tok, int* status,
                          cudaStream_t stream)
{
    if (R == 0) return 0;
    static int sms[kMaxDevicesAttr] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return -3;
    if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -3;
    const int C = logprobs_cluster(R, V, sms[dev], f32 ? 4 : 2);
    const LogArgs a{x, ld, tok, V, top, C, scale, scale * 1.4426950408889634f, logprob, rank, entropy, top_lp, top_tok, status};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(R) * C);
    cfg.blockDim = dim3(kLogThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return (f32 ? cudaLaunchKernelEx(&cfg, kda_logprobs_kernel<float>, a) : cudaLaunchKernelEx(&cfg, kda_logprobs_kernel<uint16_t>, a)) ==
           cudaSuccess ? 0 : -3;
}

}  // namespace kda
