// kda_logprobs.cu -- log probabilities of given tokens, with rank, entropy and the most likely tokens.
//
// Of a row of logits x and z = scale * x:   lse = log sum exp z,   logprob = z_t - lse,
//     entropy = lse - sum p z,   rank = place of t in the order (x descending, lowest index first),
// and the first `top` tokens of that order.
//
// One pass over the row: each thread keeps a running maximum m of its elements, the sum of e^(z - z_m), the same sum
// weighted by the exponents, and the count of elements ahead of the given token; they are joined by the usual rescaling.
// Exponents are y = (x - m) c with c = scale * log2 e: the difference first, so that rows of a type's lowest value alone
// do not overflow, and the largest terms have the smallest errors.
//
// The most likely tokens cost the pass nothing: a thread's maximum is known.  The `top` threads (groups of 4) with the
// largest maxima hold all of the `top` largest elements (an element of another group has `top` maxima above it), so
// only their elements are read again, and what is at least the smallest of those maxima is put in order.
#include <cfloat>
#include "common.cuh"
#include "tc.cuh"

namespace kda {

constexpr int kLogThreads = 512, kLogGroups = kLogThreads / 4, kLogMaxTop = 32, kLogKeep = 1024;
constexpr int kStatusToken = -1;                 // KDA_ERR_INVALID_ARG, recorded on the device

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
// Bits that order like the values (-0 like 0), and back.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);
    return b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t o) { return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu)); }

// Sums of a part of a row relative to its maximum m (NaN where the part holds one): sum 2^y, sum 2^y y.
struct LogSums { float m, s, w; };
__device__ __forceinline__ LogSums log_move(LogSums a, float m, float c) {     // the same relative to a larger maximum
    if (!(a.s > 0.f)) return LogSums{m, 0.f, 0.f};
    const float d = fmaxf((a.m - m) * c, -200.f), f = log_ex2(d);
    return LogSums{m, a.s * f, f * fmaf(d, a.s, a.w)};
}
__device__ __forceinline__ LogSums log_join(LogSums a, LogSums b, float c) {
    const float m = max_nan(a.m, b.m);
    a = log_move(a, m, c);
    b = log_move(b, m, c);
    return LogSums{m, a.s + b.s, a.w + b.w};
}

template <typename T> struct LogVec;             // a chunk of 16 bytes
template <> struct LogVec<float> {
    static constexpr int N = 4;
    __device__ static __forceinline__ float one(const float* p) { return __ldg(p); }
    __device__ static __forceinline__ void unpack(uint4 v, float (&x)[4]) {
        x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y); x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    }
};
template <> struct LogVec<uint16_t> {
    static constexpr int N = 8;
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
};

struct LogArgs {
    const void* x; long long ld;
    const int32_t* tok;
    int R, V, top;
    float scale, c;                              // c = scale * log2 e
    float* logprob; int32_t* rank; float* entropy;
    float* top_lp; int32_t* top_tok;
    int* status;
};

// Elements [i, i + N) of a row whose 16-byte chunks begin at i: whole, or those inside [0, V) (others -inf).
template <typename T>
__device__ __forceinline__ uint4 log_load(const T* row, int i, int V) {
    constexpr int N = LogVec<T>::N;
    if (i >= 0 && i + N <= V) return __ldcs(reinterpret_cast<const uint4*>(row + i));
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (N == 4) {
            w[k] = i + k >= 0 && i + k < V ? __float_as_uint(__ldg(row + i + k)) : 0xff800000u;
        } else {
            const uint32_t lo = i + 2 * k >= 0 && i + 2 * k < V ? __ldg(row + i + 2 * k) : 0xff80u;
            const uint32_t hi = i + 2 * k + 1 >= 0 && i + 2 * k + 1 < V ? __ldg(row + i + 2 * k + 1) : 0xff80u;
            w[k] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__global__ void __launch_bounds__(kLogThreads, 2)
kda_logprobs_kernel(const LogArgs a)
{
    using Vec = LogVec<T>;
    constexpr int N = Vec::N, U = 4;             // U chunks a thread and step, loaded together
    constexpr int kStep = kLogThreads * N;       // elements of a chunk of every thread
    __shared__ LogSums s_sum[kLogThreads / 32];
    __shared__ int s_cnt[kLogThreads / 32];
    __shared__ __align__(16) unsigned long long s_key[kLogGroups];
    __shared__ __align__(16) uint32_t s_val[kLogGroups];
    __shared__ int s_rank[kLogGroups];
    __shared__ int s_own[kLogMaxTop];
    __shared__ unsigned long long s_keep[kLogKeep];
    __shared__ unsigned long long s_list[kLogMaxTop];
    __shared__ unsigned long long s_least, s_next;
    __shared__ int s_count;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const long long rw = blockIdx.x;
    const T* row = static_cast<const T*>(a.x) + rw * a.ld;
    const int top = a.top, V = a.V;
    const int t = a.tok ? a.tok[rw] : 0;
    if (a.tok && (t < 0 || t >= V)) {            // padding, or a token that is none
        if (tid == 0) {
            if (t >= V) set_status(a.status, kStatusToken);
            a.logprob[rw] = 0.f;
            if (a.rank) a.rank[rw] = 0;
            if (a.entropy) a.entropy[rw] = 0.f;
        }
        for (int i = tid; i < top; i += kLogThreads) {
            a.top_lp[rw * top + i] = -INFINITY;
            a.top_tok[rw * top + i] = -1;
        }
        return;
    }
    const float xt = Vec::one(row + t);
    // chunks begin on 16 bytes: the first one may begin before the row
    const int first = -static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    const int steps = (V - first + kStep - 1) / kStep;                     // chunks a thread, at most
    const int mine = first + tid * N;                                      // this thread's chunks: mine + k * kStep

    // 1. the pass
    LogSums acc{-INFINITY, 0.f, 0.f};
    int cnt = 0, at = 0;                         // at: step of U chunks where the maximum was met first
    const float c = a.c;
    for (int k0 = 0; k0 < steps; k0 += U) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = log_load(row, min(mine + (k0 + u) * kStep, V), V);
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[N];
            Vec::unpack(v[u], x);
#pragma unroll
            for (int i = 0; i < N; ++i) m = max_nan(m, x[i]);
        }
        if (!(m <= acc.m)) {                     // (a NaN is above everything, and stays)
            at = acc.m != acc.m ? at : k0;
            acc = log_move(acc, max_nan(m, acc.m), c);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float x[N];
            Vec::unpack(v[u], x);
            const int i0 = mine + (k0 + u) * kStep;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float y = fmaxf((x[i] - acc.m) * c, -150.f), e = log_ex2(y);      // (2^-150 is 0)
                acc.s += e;
                acc.w = fmaf(e, y, acc.w);
            }
            if (i0 + N <= t && i0 >= 0) {
#pragma unroll
                for (int i = 0; i < N; ++i) cnt += x[i] >= xt;
            } else if (i0 > t) {
#pragma unroll
                for (int i = 0; i < N; ++i) cnt += x[i] > xt;
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) cnt += i0 + i >= 0 && (x[i] > xt || (x[i] == xt && i0 + i < t));
            }
        }
    }

    // 2. the row's sums
    LogSums all = acc;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        const LogSums o{__shfl_xor_sync(0xffffffffu, all.m, off), __shfl_xor_sync(0xffffffffu, all.s, off),
                        __shfl_xor_sync(0xffffffffu, all.w, off)};
        all = log_join(all, o, c);
    }
    const int wcnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) { s_sum[warp] = all; s_cnt[warp] = wcnt; }
    // the groups' maxima; a group without elements has 0, below every value
    const bool has = mine < V;
    const uint32_t mv = has ? order_bits(acc.m) : 0u;
    uint32_t gv = max(mv, __shfl_xor_sync(0xffffffffu, mv, 1));
    gv = max(gv, __shfl_xor_sync(0xffffffffu, gv, 2));
    if ((tid & 3) == 0) { s_val[tid >> 2] = gv; s_rank[tid >> 2] = 0; }
    if (tid == 0) s_count = 0;
    __syncthreads();
    all = s_sum[0];
    int ahead = s_cnt[0];
    for (int i = 1; i < kLogThreads / 32; ++i) {
        all = log_join(all, s_sum[i], c);
        ahead += s_cnt[i];
    }
    const bool none = !(all.m < INFINITY);       // a NaN or +inf in the row
    const float ls = logf(all.s);                // lse = scale * m + ls
    if (tid == 0) {
        const float nan = __int_as_float(0x7fffffff);
        if (a.tok) {
            // (a row of -inf alone: no token has a probability)
            a.logprob[rw] = none ? nan : xt == -INFINITY ? -INFINITY : fmaf(a.scale, xt - all.m, -ls);
            if (a.rank) a.rank[rw] = none ? 0 : 1 + ahead;
        }
        if (a.entropy) a.entropy[rw] = none ? nan : all.s > 0.f ? fmaf(-0.69314718055994531f, all.w / all.s, ls) : 0.f;
    }
    if (top == 0) return;
    if (none) {
        for (int i = tid; i < top; i += kLogThreads) {
            a.top_lp[rw * top + i] = __int_as_float(0x7fffffff);
            a.top_tok[rw * top + i] = -1;
        }
        return;
    }

    // 3. the groups in the order of their maxima (equal ones by number): a thread compares a quarter
    {
        const int g = tid & (kLogGroups - 1), q0 = tid / kLogGroups * (kLogGroups / 4);
        const uint32_t v = s_val[g];
        int above = 0;
#pragma unroll
        for (int i = 0; i < kLogGroups / 4; i += 4) {
            const uint4 o = *reinterpret_cast<const uint4*>(s_val + q0 + i);
            above += (o.x > v || (o.x == v && q0 + i < g)) + (o.y > v || (o.y == v && q0 + i + 1 < g)) +
                     (o.z > v || (o.z == v && q0 + i + 2 < g)) + (o.w > v || (o.w == v && q0 + i + 3 < g));
        }
        atomicAdd(&s_rank[g], above);
    }
    __syncthreads();
    if (tid < kLogGroups && s_rank[tid] == min(top, kLogGroups) - 1) s_least = s_val[tid];
    __syncthreads();
    // the groups at or above the `top`-th, by key now: value, then lowest index
    const uint32_t least = static_cast<uint32_t>(s_least);
    unsigned long long key = 0;
    if (has && mv == gv && gv >= least) {        // this thread's first element of that value
        const int k1 = min(at + U, steps);
        for (int k = at; k < k1 && key == 0; ++k) {
            float x[N];
            Vec::unpack(log_load(row, min(mine + k * kStep, V), V), x);
#pragma unroll
            for (int i = N - 1; i >= 0; --i) {
                const int idx = mine + k * kStep + i;
                if (idx >= 0 && idx < V && order_bits(x[i]) == mv)
                    key = static_cast<unsigned long long>(mv) << 32 | static_cast<uint32_t>(~idx);
            }
        }
    }
    __syncwarp();
    unsigned long long o = __shfl_xor_sync(0xffffffffu, key, 1);
    key = key > o ? key : o;
    o = __shfl_xor_sync(0xffffffffu, key, 2);
    key = key > o ? key : o;
    if ((tid & 3) == 0) { s_key[tid >> 2] = key; s_rank[tid >> 2] = 0; }
    __syncthreads();
    {
        const int g = tid & (kLogGroups - 1), q0 = tid / kLogGroups * (kLogGroups / 4);
        const unsigned long long v = s_key[g];
        int above = 0;
        if (v) {
#pragma unroll 8
            for (int i = 0; i < kLogGroups / 4; ++i) above += s_key[q0 + i] > v;
            atomicAdd(&s_rank[g], above);
        }
    }
    if (tid < kLogMaxTop) s_own[tid] = -1;
    if (tid == 0) s_least = 0;
    __syncthreads();
    if (tid < kLogGroups && s_key[tid]) {
        const int r = s_rank[tid];
        if (r < top) s_own[r] = tid;
        if (r == top - 1) s_least = s_key[tid];
    }
    __syncthreads();

    // 4. their elements at or above the smallest of their maxima: a warp a group, put in order by counting.  Only
    // elements beside each other in one group can make them many; then one after another is looked for instead
    const unsigned long long bound = s_least;
    auto scan = [&](auto&& use) {
        for (int r = warp; r < top; r += kLogThreads / 32) {
            const int g = s_own[r];
            if (g < 0) continue;
            for (int k = lane >> 2; k < steps; k += 8) {
                const int i0 = first + (4 * g + (lane & 3)) * N + k * kStep;
                if (i0 >= V) continue;
                float x[N];
                Vec::unpack(log_load(row, i0, V), x);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const unsigned long long e = static_cast<unsigned long long>(order_bits(x[i])) << 32 | static_cast<uint32_t>(~(i0 + i));
                    if (i0 + i >= 0 && i0 + i < V && e >= bound) use(e);
                }
            }
        }
    };
    scan([&](unsigned long long e) {
        const int i = atomicAdd(&s_count, 1);
        if (i < kLogKeep) s_keep[i] = e;
    });
    __syncthreads();
    const int n = s_count;
    if (tid < kLogMaxTop) s_list[tid] = 0;
    __syncthreads();
    if (n <= kLogKeep) {
        for (int i = tid; i < n; i += kLogThreads) {
            const unsigned long long e = s_keep[i];
            int above = 0;
            for (int j = 0; j < n; ++j) above += s_keep[j] > e;
            if (above < top) s_list[above] = e;
        }
        __syncthreads();
    } else {
        unsigned long long last = ~0ull;
        for (int i = 0; i < top; ++i) {
            if (tid == 0) s_next = 0;
            __syncthreads();
            unsigned long long best = 0;
            scan([&](unsigned long long e) { if (e < last && e > best) best = e; });
            if (best) atomicMax(&s_next, best);
            __syncthreads();
            last = s_next;
            if (tid == 0) s_list[i] = last;
            __syncthreads();
        }
    }
    if (tid < top) {
        const unsigned long long e = s_list[tid];
        const float x = from_order(static_cast<uint32_t>(e >> 32));
        a.top_lp[rw * top + tid] = e == 0 || x == -INFINITY ? -INFINITY : fmaf(a.scale, x - all.m, -ls);
        a.top_tok[rw * top + tid] = e == 0 ? -1 : static_cast<int32_t>(~static_cast<uint32_t>(e));
    }
}

int launch_token_logprobs(const void* x, int f32, long long ld, const int32_t* tok, int R, int V, int top, float scale,
                          float* logprob, int32_t* rank, float* entropy, float* top_lp, int32_t* top_tok, int* status,
                          cudaStream_t stream)
{
    if (R == 0) return 0;
    const LogArgs a{x, ld, tok, R, V, top, scale, scale * 1.4426950408889634f, logprob, rank, entropy, top_lp, top_tok, status};
    if (f32) kda_logprobs_kernel<float><<<static_cast<unsigned>(R), kLogThreads, 0, stream>>>(a);
    else kda_logprobs_kernel<uint16_t><<<static_cast<unsigned>(R), kLogThreads, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace kda
