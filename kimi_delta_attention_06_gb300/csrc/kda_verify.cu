// kda_verify.cu -- verification of drafted tokens (speculative sampling).
//
// Draft j of a sequence is accepted while u_j q_j(x_j) < p_j(x_j).  At the first rejected
// position i the next token is drawn from w = max(0, p_i - q_i) (from p_i when w is all zero),
// after a whole accepted draft from w = p at the position after it: the smallest t with
// sum_{s <= t} w_s > u sum w.
//
// Only two rows of V values are read (one when nothing was rejected), so the kernel is a single
// pass over them.  One cluster of C CTAs serves a sequence, each CTA a contiguous slice of the
// vocabulary and each warp a contiguous part of it; the slice sums are exchanged through
// distributed shared memory, the CTA whose slice crosses the threshold narrows it to a warp's
// part, then to one warp's share of that, then walks it.
//
// Which token is drawn depends on sums of up to V terms compared with a threshold, so they carry
// about 45 bits: a lane's sum is an unevaluated pair of floats (Knuth's two-sum, 1969; the
// difference p - q by Dekker's fast form, 1971, exact for p > q >= 0), and so are the lanes joined;
// fp64 only joins the warps' sums.  fp64 throughout would be bound by its rate (2 operations a
// clock and SM): joining a CTA's 512 lanes in fp64 alone took longer than reading its slice.
#include "common.cuh"
#include "tc.cuh"

namespace kda {

constexpr int kVerMaxWarps = 16;

struct VerRows {
    const float* p;
    const float* q;          // nullptr: no draft row (or a certain draft: `hot`)
    int hot;                 // certain draft's token (weight 0), -1 = none
};

__device__ __forceinline__ float ver_clean(float x) {      // negative, NaN, infinite -> 0
    return x < __int_as_float(0x7f800000) ? fmaxf(x, 0.f) : 0.f;
}
// Weight of a token as a pair hi + lo (exact).
__device__ __forceinline__ float ver_weight(float p, float q, float& lo) {
    p = ver_clean(p);
    q = ver_clean(q);
    const float d = fmaxf(p - q, 0.f);
    lo = d > 0.f ? (p - d) - q : 0.f;
    return d;
}
__device__ __forceinline__ double ver_one(const VerRows& w, int t) {
    float lo;
    const float hi = ver_weight(t == w.hot ? 0.f : __ldg(w.p + t), w.q ? __ldg(w.q + t) : 0.f, lo);
    return static_cast<double>(hi) + static_cast<double>(lo);
}

// Sum of the weights of tokens [a, b), over the lanes of a warp.
template <bool Q>
__device__ __forceinline__ double ver_sum(const VerRows& w, int a, int b, int lane) {
    constexpr int U = 16;                      // loads in flight per row and lane
    float hi = 0.f, lo = 0.f;
    for (int t0 = a + lane; t0 < b; t0 += 32 * U) {
        float p[U], q[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int t = t0 + 32 * i;
            p[i] = t < b ? __ldg(w.p + t) : 0.f;
            q[i] = Q && t < b ? __ldg(w.q + t) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float e;
            const float d = ver_weight(t0 + 32 * i == w.hot ? 0.f : p[i], q[i], e);
            const float s = hi + d, z = s - hi;
            lo += ((hi - (s - z)) + (d - z)) + e;
            hi = s;
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {              // (still pairs of floats: fp64 adds of a whole warp are slow)
        const float h = __shfl_xor_sync(0xffffffffu, hi, off), e = __shfl_xor_sync(0xffffffffu, lo, off);
        const float s = hi + h, z = s - hi;
        lo = (lo + e) + ((hi - (s - z)) + (h - z));
        hi = s;
    }
    return static_cast<double>(hi) + static_cast<double>(lo);
}
__device__ __forceinline__ double ver_sum(const VerRows& w, int a, int b, int lane) {
    return w.q ? ver_sum<true>(w, a, b, lane) : ver_sum<false>(w, a, b, lane);
}

// Lane i of a warp holds the sum of part i.  The first part with weight whose running sum exceeds x
// (else the last with weight: rounding left x at the total); `base` grows by the parts before it.
__device__ __forceinline__ int ver_find(double part, double x, double& base) {
    const int lane = threadIdx.x & 31;
    double c = part;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double o = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) c += o;
    }
    const unsigned has = __ballot_sync(0xffffffffu, part > 0.);
    const unsigned over = __ballot_sync(0xffffffffu, part > 0. && base + c > x);
    const int at = over ? __ffs(over) - 1 : has ? 31 - __clz(has) : 0;
    const double before = __shfl_sync(0xffffffffu, c, at > 0 ? at - 1 : 0);
    if (at > 0) base += before;
    return at;
}
__device__ __forceinline__ double warp_total(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

__global__ void __launch_bounds__(kVerMaxWarps * 32, 2)
kda_verify_kernel(const float* __restrict__ tp, long long ldp, const float* __restrict__ dp, long long ldq,
                  const int32_t* __restrict__ toks, const int32_t* __restrict__ num_draft,
                  const float* __restrict__ ua, const float* __restrict__ us, int K, int V, int C,
                  int32_t* __restrict__ out, int32_t* __restrict__ num_out, int* status)
{
    __shared__ double s_part[kVerMaxWarps];
    __shared__ double s_total, s_want, s_base;
    __shared__ int s_first, s_bad, s_owner;

    const int rank = C > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    const long long n = blockIdx.x / static_cast<unsigned>(C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int threads = blockDim.x, warps = threads >> 5;

    // 1. the accepted count (every CTA of the cluster on its own)
    const int nd = num_draft ? num_draft[n] : K;
    if (tid == 0) { s_first = nd; s_bad = nd < 0 || nd > K; }
    __syncthreads();
    int x = -1;
    if (tid < K && !s_bad && tid < nd) {
        x = toks[n * K + tid];
        if (x < 0 || x >= V) {
            s_bad = 1;
        } else {
            const float p = tp[(n * (K + 1) + tid) * ldp + x];
            const float q = dp ? dp[(n * K + tid) * ldq + x] : 1.f;
            // fp64 holds the product of two floats exactly
            const bool ok = static_cast<double>(ua[n * K + tid]) * static_cast<double>(q) < static_cast<double>(p);
            if (!ok) atomicMin(&s_first, tid);
        }
    }
    __syncthreads();
    if (s_bad) {                                            // the same in every CTA of the cluster
        if (rank == 0) {
            for (int i = tid; i <= K; i += threads) out[n * (K + 1) + i] = -1;
            if (tid == 0) { num_out[n] = 0; set_status(status, -1); }
        }
        return;
    }
    const int a = s_first;
    if (rank == 0) {
        if (tid < a) out[n * (K + 1) + tid] = x;
        for (int i = a + 1 + tid; i <= K; i += threads) out[n * (K + 1) + i] = -1;
        if (tid == 0) num_out[n] = a + 1;
    }

    // 2. slice sums; a residual without weight falls back to p itself
    VerRows w;
    w.p = tp + (n * (K + 1) + a) * ldp;
    w.q = a < nd && dp ? dp + (n * K + a) * ldq : nullptr;
    w.hot = a < nd && !dp ? toks[n * K + a] : -1;
    const int S = (V + C - 1) / C;
    const int c0 = min(V, rank * S), c1 = min(V, c0 + S);
    const int sub = (c1 - c0 + warps - 1) / warps;
    while (true) {
        const int a0 = min(c1, c0 + warp * sub), a1 = min(c1, a0 + sub);
        const double s = ver_sum(w, a0, a1, lane);
        if (lane == 0) s_part[warp] = s;
        __syncthreads();
        if (warp == 0) {
            const double t = warp_total(lane < warps ? s_part[lane] : 0.);
            if (lane == 0) s_total = t;
        }
        if (C > 1) tc::cluster_sync();
        if (warp == 0) {
            __syncwarp();
            double part = 0.;
            if (C > 1) { if (lane < C) part = ld_cluster_f64(tc::mapa(tc::smem_u32(&s_total), lane)); }
            else if (lane == 0) part = s_total;
            const double total = warp_total(part), want = static_cast<double>(us[n]) * total;
            double base = 0.;
            const int owner = ver_find(part, want, base);
            if (lane == 0) { s_owner = total > 0. ? owner : -1; s_want = want; s_base = base; }
        }
        __syncthreads();
        if (C > 1) tc::cluster_sync();                      // s_total may change or go away after this
        if (s_owner >= 0 || (!w.q && w.hot < 0)) break;
        w.q = nullptr;
        w.hot = -1;
        __syncthreads();                                    // everyone has read s_owner
    }
    if (s_owner < 0) {
        if (rank == 0 && tid == 0) out[n * (K + 1) + a] = -1;
        return;
    }
    if (rank != s_owner) return;

    // 3. narrow: this CTA's warp part, then one warp's share of that, then walk
    const double want = s_want;
    if (warp == 0) {
        double base = s_base;
        const int f = ver_find(lane < warps ? s_part[lane] : 0., want, base);
        if (lane == 0) { s_first = f; s_base = base; }
    }
    __syncthreads();
    const int b0 = min(c1, c0 + s_first * sub), b1 = min(c1, b0 + sub);
    const int sub2 = (b1 - b0 + warps - 1) / warps;
    const double s2 = ver_sum(w, min(b1, b0 + warp * sub2), min(b1, b0 + (warp + 1) * sub2), lane);
    if (lane == 0) s_part[warp] = s2;
    __syncthreads();
    if (warp != 0) return;
    double base = s_base;
    const int g = ver_find(lane < warps ? s_part[lane] : 0., want, base);
    const int d0 = min(b1, b0 + g * sub2), d1 = min(b1, d0 + sub2);
    int pick = -1;
    for (int t0 = d0; t0 < d1; t0 += 32) {
        const int t = t0 + lane;
        const double wt = t < d1 ? ver_one(w, t) : 0.;
        double c = wt;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, c, off);
            if (lane >= off) c += o;
        }
        const unsigned has = __ballot_sync(0xffffffffu, wt > 0.);
        const unsigned over = __ballot_sync(0xffffffffu, wt > 0. && base + c > want);
        if (over) { pick = t0 + __ffs(over) - 1; break; }
        if (has) pick = t0 + 31 - __clz(has);               // rounding left the threshold above the sum: the last one
        base += __shfl_sync(0xffffffffu, c, 31);
    }
    if (lane == 0) out[n * (K + 1) + a] = pick;
}

int launch_verify(const float* tp, long long ldp, const float* dp, long long ldq, const int32_t* toks,
                  const int32_t* num_draft, const float* ua, const float* us, int N, int K, int V, int32_t* out,
                  int32_t* num_out, int* status, cudaStream_t stream)
{
    // Few sequences: 16 CTAs of 16 warps each (16 is past the portable cluster size), so that a row
    // of 131072 is one round of loads.  Many: up to 8 CTAs of 8 warps, in slices of 2048 tokens
    // at least, several per SM so that one's reads cover another's acceptance and narrowing.
    const bool few = static_cast<long long>(N) * 16 <= 152 && V > 8 * 4096;
    const int most = few ? 16 : 8, warps = few ? 16 : 8;
    int C = 1;
    while (C < most && static_cast<long long>(N) * C < 8 * 152 && V / (2 * C) >= 2048) C *= 2;
    static bool wide_done[kMaxDevicesAttr] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return -3;
    if (C > 8 && !wide_done[dev]) {
        if (cudaFuncSetAttribute(kda_verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return -3;
        wide_done[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(N) * C);
    cfg.blockDim = dim3(static_cast<unsigned>(warps) * 32);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kda_verify_kernel, tp, ldp, dp, ldq, toks, num_draft, ua, us, K, V, C, out, num_out,
                              status) == cudaSuccess ? 0 : -3;
}

}  // namespace kda
