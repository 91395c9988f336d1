// kda_verify.cu -- verification of drafted tokens (speculative sampling).
//
// Draft j of a sequence is accepted while u_j q_j(x_j) < p_j(x_j).  At the first rejected
// position i the next token is drawn from w = max(0, p_i - q_i) (from p_i when w is all zero),
// after a whole accepted draft from w = p at the position after it: the smallest t with
// sum_{s <= t} w_s > u sum w.
//
// Only two rows of V values are read (one when nothing was rejected), so the kernel is a single
// pass over them.  One cluster of C CTAs serves a sequence, each CTA a contiguous slice of the
// vocabulary and each warp a contiguous part of it.  Every CTA writes its slice's sum into the
// shared memory of all the others and waits for theirs (no cluster barrier after the reads); the
// one whose slice crosses the threshold narrows it to a warp's part, that to one warp's share of it,
// and that to a lane's.
//
// Which token is drawn depends on sums of up to V terms compared with a threshold, so they carry
// about 45 bits, as unevaluated pairs of floats: Knuth's two-sum (1969) adds, the difference p - q
// is Dekker's fast form (1971, exact for p > q >= 0), and the threshold u * total is a product with
// its rounding error from one fma.  fp64 runs at 2 operations a clock and SM here: joining a CTA's
// 512 lanes in it took longer than reading its slice, and the few joins after the reads 5 us.
//
// Measured: one sequence of 3 drafts, V = 131072, 8.6 us (latency: drafts, their odds, rows, exchange,
// the crossing part); 256 sequences of 4 drafts, V = 100003, 48.4 us (205 MB: 4.2 TB/s).
#include "common.cuh"
#include "tc.cuh"

namespace kda {

constexpr int kVerMaxWarps = 16, kVerMaxCluster = 16;

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
// A sum as a pair: |lo| at most half a step of hi.
struct Pair { float hi, lo; };
__device__ __forceinline__ Pair pair_add(Pair a, Pair b) {
    const float s = a.hi + b.hi, z = s - a.hi;
    const float e = ((a.hi - (s - z)) + (b.hi - z)) + (a.lo + b.lo);
    const float h = s + e;                                 // (|s| >= |e|)
    return Pair{h, e - (h - s)};
}
__device__ __forceinline__ Pair pair_times(float u, Pair a) {
    const float p = __fmul_rn(u, a.hi), e = fmaf(u, a.hi, -p) + u * a.lo;      // (p stays a product of its own)
    const float h = p + e;
    return Pair{h, e - (h - p)};
}
__device__ __forceinline__ bool pair_above(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Pair pair_xor(Pair a, int off) {
    return Pair{__shfl_xor_sync(0xffffffffu, a.hi, off), __shfl_xor_sync(0xffffffffu, a.lo, off)};
}
__device__ __forceinline__ Pair pair_from(Pair a, int lane) {
    return Pair{__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
__device__ __forceinline__ Pair warp_total(Pair v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v = pair_add(v, pair_xor(v, off));
    return v;
}
__device__ __forceinline__ Pair ver_one(const VerRows& w, int t) {
    float lo;
    const float hi = ver_weight(t == w.hot ? 0.f : __ldg(w.p + t), w.q ? __ldg(w.q + t) : 0.f, lo);
    return Pair{hi, lo};
}

// Sum of the weights of tokens [a, b), over the lanes of a warp.
template <bool Q>
__device__ __forceinline__ Pair ver_sum(const VerRows& w, int a, int b, int lane) {
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
    return warp_total(pair_add(Pair{hi, 0.f}, Pair{lo, 0.f}));
}
__device__ __forceinline__ Pair ver_sum(const VerRows& w, int a, int b, int lane) {
    return w.q ? ver_sum<true>(w, a, b, lane) : ver_sum<false>(w, a, b, lane);
}

// Lane i of a warp holds the sum of part i.  The first part with weight whose running sum exceeds x
// (else the last with weight: rounding left x at the total); `base` grows by the parts before it.
__device__ __forceinline__ int ver_find(Pair part, Pair x, Pair& base) {
    const int lane = threadIdx.x & 31;
    Pair c = part;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Pair o{__shfl_up_sync(0xffffffffu, c.hi, off), __shfl_up_sync(0xffffffffu, c.lo, off)};
        if (lane >= off) c = pair_add(c, o);
    }
    const unsigned has = __ballot_sync(0xffffffffu, part.hi > 0.f);
    const unsigned over = __ballot_sync(0xffffffffu, part.hi > 0.f && pair_above(pair_add(base, c), x));
    const int at = over ? __ffs(over) - 1 : has ? 31 - __clz(has) : 0;
    const Pair before = pair_from(c, at > 0 ? at - 1 : 0);
    if (at > 0) base = pair_add(base, before);
    return at;
}

__device__ __forceinline__ void st_cluster_pair(uint32_t addr, Pair v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" :: "r"(addr), "f"(v.hi), "f"(v.lo) : "memory");
}

__global__ void __launch_bounds__(kVerMaxWarps * 32, 2)
kda_verify_kernel(const float* __restrict__ tp, long long ldp, const float* __restrict__ dp, long long ldq,
                  const int32_t* __restrict__ toks, const int32_t* __restrict__ num_draft,
                  const float* __restrict__ ua, const float* __restrict__ us, int K, int V, int C,
                  int32_t* __restrict__ out, int32_t* __restrict__ num_out, int* status)
{
    __shared__ Pair s_part[kVerMaxWarps], s_share[kVerMaxWarps];
    __shared__ __align__(8) Pair s_slice[2][kVerMaxCluster];          // sums of the cluster's slices, of each pass
    __shared__ __align__(8) uint64_t s_bar;
    __shared__ Pair s_want, s_base;
    __shared__ int s_owner;

    const int rank = C > 1 ? static_cast<int>(tc::cluster_ctarank()) : 0;
    const long long n = blockIdx.x / static_cast<unsigned>(C);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int warps = blockDim.x >> 5;
    if (C > 1) {                                            // the others' barriers are up before this CTA writes to them
        if (tid == 0) {
            tc::mbar_init(&s_bar, C);
            tc::mbar_fence_init();
        }
        __syncthreads();
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    }

    // 1. the accepted count: every warp on its own, a draft a lane (two for more than 32)
    const int nd = num_draft ? num_draft[n] : K;
    bool bad = nd < 0 || nd > K;
    int a = nd, hot = -1;
    for (int j0 = 0; j0 < K && !bad; j0 += 32) {
        const int j = j0 + lane;
        int x = 0;
        bool ok = true, in = true;
        if (j < nd) {
            x = toks[n * K + j];
            in = x >= 0 && x < V;
            if (in) {
                const float p = __ldg(tp + (n * (K + 1) + j) * ldp + x);
                const float q = dp ? __ldg(dp + (n * K + j) * ldq + x) : 1.f;
                // fp64 holds the product of two floats exactly
                ok = static_cast<double>(ua[n * K + j]) * static_cast<double>(q) < static_cast<double>(p);
            }
        }
        bad = __any_sync(0xffffffffu, !in);
        const unsigned no = __ballot_sync(0xffffffffu, !ok);
        if (no && a == nd) {                                // the first rejected draft
            a = j0 + __ffs(no) - 1;
            hot = __shfl_sync(0xffffffffu, x, a - j0);
        }
        if (rank == 0 && warp == 0 && j < min(nd, a)) out[n * (K + 1) + j] = x;
    }
    if (bad) {                                              // the same in every CTA of the cluster
        if (C > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (rank == 0 && warp == 0) {
            for (int i = lane; i <= K; i += 32) out[n * (K + 1) + i] = -1;
            if (lane == 0) { num_out[n] = 0; set_status(status, -1); }
        }
        return;
    }
    if (rank == 0 && warp == 0) {
        for (int i = a + 1 + lane; i <= K; i += 32) out[n * (K + 1) + i] = -1;
        if (lane == 0) num_out[n] = a + 1;
    }

    // 2. slice sums; a residual without weight falls back to p itself
    VerRows w;
    w.p = tp + (n * (K + 1) + a) * ldp;
    w.q = a < nd && dp ? dp + (n * K + a) * ldq : nullptr;
    w.hot = a < nd && !dp ? hot : -1;
    const int S = (V + C - 1) / C;
    const int c0 = min(V, rank * S), c1 = min(V, c0 + S);
    const int sub = (c1 - c0 + warps - 1) / warps;
    for (int pass = 0;; ++pass) {
        const int a0 = min(c1, c0 + warp * sub), a1 = min(c1, a0 + sub);
        const Pair s = ver_sum(w, a0, a1, lane);
        if (lane == 0) s_part[warp] = s;
        if (C > 1 && pass == 0) {
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        }
        __syncthreads();
        if (warp == 0) {
            const Pair mine = warp_total(lane < warps ? s_part[lane] : Pair{0.f, 0.f});
            Pair part = lane == 0 ? mine : Pair{0.f, 0.f};
            bool came = true;
            if (C > 1) {
                if (lane < C) {
                    st_cluster_pair(tc::mapa(tc::smem_u32(&s_slice[pass][rank]), lane), mine);
                    tc::mbar_arrive_remote(tc::mapa(tc::smem_u32(&s_bar), lane));
                }
                came = tc::mbar_wait_cluster_bounded(&s_bar, pass, kWaitLimitNs);
                came = __all_sync(0xffffffffu, came);
                part = came && lane < C ? s_slice[pass][lane] : Pair{0.f, 0.f};
            }
            const Pair total = warp_total(part), want = pair_times(us[n], total);
            Pair base{0.f, 0.f};
            const int owner = ver_find(part, want, base);
            if (lane == 0) {
                s_owner = !came ? -2 : total.hi > 0.f ? owner : -1;
                s_want = want;
                s_base = base;
                if (!came) set_status(status, kStatusTimeout);
            }
        }
        __syncthreads();
        if (s_owner != -1 || (!w.q && w.hot < 0)) break;
        w.q = nullptr;                                      // (once: a second pass has neither)
        w.hot = -1;
    }
    if (s_owner < 0) {
        if (s_owner == -1 && rank == 0 && tid == 0) out[n * (K + 1) + a] = -1;
        return;
    }
    if (rank != s_owner) return;

    // 3. the crossing warp's part over all warps again, then the crossing share of that over the
    // lanes of one: E neighbours a lane, and the crossing lane walks its own
    const Pair want = s_want;
    Pair base = s_base;
    const int f = ver_find(lane < warps ? s_part[lane] : Pair{0.f, 0.f}, want, base);
    const int b0 = min(c1, c0 + f * sub), b1 = min(c1, b0 + sub), sub2 = (b1 - b0 + warps - 1) / warps;
    const Pair s2 = ver_sum(w, min(b1, b0 + warp * sub2), min(b1, b0 + (warp + 1) * sub2), lane);
    if (lane == 0) s_share[warp] = s2;
    __syncthreads();
    if (warp != 0) return;
    const int g = ver_find(lane < warps ? s_share[lane] : Pair{0.f, 0.f}, want, base);
    const int d0 = min(b1, b0 + g * sub2), d1 = min(b1, d0 + sub2);
    const int E = (d1 - d0 + 31) / 32, m0 = min(d1, d0 + lane * E), m1 = min(d1, m0 + E);
    float hi = 0.f, lo = 0.f;
#pragma unroll 8
    for (int t = m0; t < m1; ++t) {
        float e;
        const float d = ver_weight(t == w.hot ? 0.f : __ldg(w.p + t), w.q ? __ldg(w.q + t) : 0.f, e);
        const float s = hi + d, z = s - hi;
        lo += ((hi - (s - z)) + (d - z)) + e;
        hi = s;
    }
    const int at = ver_find(pair_add(Pair{hi, 0.f}, Pair{lo, 0.f}), want, base);
    if (lane != at) return;
    int pick = -1;                                          // (rounding may leave the threshold past the end: the last weight)
    for (int t = m0; t < m1; ++t) {
        const Pair wt = ver_one(w, t);
        base = pair_add(base, wt);
        if (wt.hi > 0.f) {
            pick = t;
            if (pair_above(base, want)) break;
        }
    }
    out[n * (K + 1) + a] = pick;
}

// CTAs of 16 warps a row: as many as leave each an SM of its own, as each one's acceptance, exchange and narrowing are
// latency that more of them only repeat (152 SMs: 256 rows of 100003 48.6 us at one CTA a row, 55 at two; of 8 warps 54 at
// two, 52 at four, 59 at eight; with two on some SMs 24 rows of 90511 took 15.1 instead of 12.1, 100 of 50000 20.3 instead of
// 16.5, 78 of 37080 14.8 instead of 11.7).  Clusters of 8 do not find room on all SMs (19 rows: 15.0 with 8, 13.4 with 4), on
// nine tenths of them they do.  Few sequences take up to 16, past the portable cluster size, where the device holds that
// many such clusters, so that a row of 131072 is one round of loads; slices of 2048 tokens at least.
int verify_cluster(int N, int V, int sms, int clusters16) {
    const int most = static_cast<long long>(N) * 16 <= sms && N <= clusters16 && V > 8 * 4096 ? 16 : 8;
    int C = 1;
    while (C < most && static_cast<long long>(N) * 2 * C <= (C == 4 ? sms * 9 / 10 : sms) && V / (2 * C) >= 2048) C *= 2;
    return C;
}

namespace {
cudaLaunchConfig_t verify_config(unsigned rows, int C, cudaLaunchAttribute (&at)[1]) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(rows * C);
    cfg.blockDim = dim3(kVerMaxWarps * 32);
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cfg;
}
// Clusters of 16 that the device holds at once: 0 where it refuses them.
int clusters_of_16() {
    cudaLaunchAttribute at[1];
    const cudaLaunchConfig_t cfg = verify_config(1, 16, at);
    int n = 0;
    if (cudaFuncSetAttribute(kda_verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kda_verify_kernel, &cfg) != cudaSuccess) {
        cudaGetLastError();                                 // (the smaller clusters do without)
        return 0;
    }
    return n;
}
}  // namespace

int launch_verify(const float* tp, long long ldp, const float* dp, long long ldq, const int32_t* toks,
                  const int32_t* num_draft, const float* ua, const float* us, int N, int K, int V, int32_t* out,
                  int32_t* num_out, int* status, cudaStream_t stream)
{
    static int sms[kMaxDevicesAttr] = {}, held[kMaxDevicesAttr] = {};       // of each device; held: clusters of 16, + 1
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return -3;
    if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -3;
    if (!held[dev]) held[dev] = clusters_of_16() + 1;
    const int C = verify_cluster(N, V, sms[dev], held[dev] - 1);
    cudaLaunchAttribute at[1];
    cudaLaunchConfig_t cfg = verify_config(static_cast<unsigned>(N), C, at);
    cfg.stream = stream;
    return cudaLaunchKernelEx(&cfg, kda_verify_kernel, tp, ldp, dp, ldq, toks, num_draft, ua, us, K, V, C, out, num_out,
                              status) == cudaSuccess ? 0 : -3;
}

}  // namespace kda
