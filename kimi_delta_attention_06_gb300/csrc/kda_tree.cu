// kda_tree.cu -- the KDA recurrence along the branches of a tree of drafted tokens.
//
// Node i continues the state of its parent (the sequence's own state for a child of the last token):
//     S_i = (I - beta_i k_i k_i^T) Diag(alpha_i) S_parent(i) + beta_i k_i v_i^T,    o_i = S_i^T q_i.
// Written out along the path from the root to i, with A(i, a) the product of the alphas of the nodes after a on it
// (all of them for a = 0, the state before the tree), and u_i = beta_i (v_i - (alpha_i S_parent(i))^T k_i):
//     u_i = beta_i (v_i - S_0^T (A(i, 0) k_i) - sum_a [k_i . A(i, a) k_a] u_a)      a: the nodes before i on its path
//     o_i =              S_0^T (A(i, 0) q_i) + sum_a [q_i . A(i, a) k_a] u_a        and i itself (A = 1)
// So no node's state is formed: S_0 is read once, for one product with the 2 K decayed keys and queries, and what is left
// are K x K numbers a head and a triangular solve that each column of the state does for itself.  The decays along a
// path are products of alphas, which neither overflow nor cancel.
#include "common.cuh"
#include "tree.cuh"

namespace kda {

constexpr int kStatusTree = -1;                  // KDA_ERR_INVALID_ARG, recorded on the device

struct TreeArgs {
    const uint16_t *q, *k, *v;
    const float* la;
    const uint16_t* beta;
    const float* pool;
    const int32_t *slots, *parents;
    void* out;
    int num_slots, out_f32, N, K, H, decay;
    int* status;
};

template <int D, int KP>
struct TreeShape {
    static constexpr int kThreads = 2 * D, kPitch = KP + 4;
    static constexpr int oAlpha = 0, oKey = oAlpha + KP * D, oQuery = oKey + KP * D;        // floats: [node][channel]
    static constexpr int oKd = oQuery + KP * D, oQd = oKd + D * kPitch;                     // [channel][node]
    static constexpr int oM = oQd + D * kPitch, oN = oM + KP * KP;                          // [node][node]
    static constexpr int oU = oAlpha;                                                       // (once the decays are done with)
    static constexpr int kBytes = (oN + KP * KP) * 4 + KP * 8 + KP * 4;
};

template <int D, int KP>
__global__ void __launch_bounds__(2 * D)
kda_tree_kernel(const TreeArgs a)
{
    using Sh = TreeShape<D, KP>;
    extern __shared__ __align__(16) float sm[];
    uint64_t* s_set = reinterpret_cast<uint64_t*>(sm + Sh::oN + KP * KP);
    float* s_beta = reinterpret_cast<float*>(s_set + KP);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int n = blockIdx.x / a.H, h = blockIdx.x - n * a.H;
    const int slot = a.slots ? a.slots[n] : n;
    if (slot < 0 || slot >= a.num_slots) {
        if (tid == 0) set_status(a.status, kStatusTree);
        return;
    }
    if (warp == 0) {
        uint64_t set[2];
        if (tree_sets(a.parents + static_cast<long long>(n) * a.K, a.K, lane, set) && lane == 0) set_status(a.status, kStatusTree);
        if (lane < KP) s_set[lane] = set[0];
        if (lane + 32 < KP) s_set[lane + 32] = set[1];
    }
    __syncthreads();
    const size_t tok0 = static_cast<size_t>(n) * a.K * a.H + h;                             // [node][h] rows a.H apart
    for (int i = tid; i < KP * D; i += Sh::kThreads) {
        const int j = i / D, ch = i % D;
        const bool on = j < a.K && s_set[j];
        const size_t at = (tok0 + static_cast<size_t>(j) * a.H) * D + ch;
        sm[Sh::oKey + i] = on ? bf16_bits_to_f32(a.k[at]) : 0.f;
        sm[Sh::oQuery + i] = on ? bf16_bits_to_f32(a.q[at]) : 0.f;
        sm[Sh::oAlpha + i] = !on || a.decay == 2 ? 1.f : expf(a.decay == 0 ? a.la[at] : a.la[tok0 + static_cast<size_t>(j) * a.H]);
    }
    if (tid < KP) s_beta[tid] = tid < a.K ? bf16_bits_to_f32(a.beta[tok0 + static_cast<size_t>(tid) * a.H]) : 0.f;
    __syncthreads();
    // a warp a node, up its path
    for (int i = warp; i < KP; i += Sh::kThreads / 32) {
        constexpr int C = D / 32;
        float key[C], query[C], p[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            key[c] = sm[Sh::oKey + i * D + lane + 32 * c];
            query[c] = sm[Sh::oQuery + i * D + lane + 32 * c];
            p[c] = 1.f;
        }
        uint64_t left = s_set[i];
        while (left) {
            const int b = 63 - __clzll(left);
            left &= ~(1ull << b);
            float m = 0.f, w = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float kb = p[c] * sm[Sh::oKey + b * D + lane + 32 * c];
                m = fmaf(key[c], kb, m);
                w = fmaf(query[c], kb, w);
                p[c] *= sm[Sh::oAlpha + b * D + lane + 32 * c];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                m += __shfl_xor_sync(0xffffffffu, m, off);
                w += __shfl_xor_sync(0xffffffffu, w, off);
            }
            if (lane == 0) {
                sm[Sh::oM + i * KP + b] = m;
                sm[Sh::oN + i * KP + b] = w;
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            sm[Sh::oKd + (lane + 32 * c) * Sh::kPitch + i] = p[c] * key[c];
            sm[Sh::oQd + (lane + 32 * c) * Sh::kPitch + i] = p[c] * query[c];
        }
    }
    __syncthreads();
    // the product with the state: a column a thread, the keys' rows in the first half of the CTA, the queries' in the other
    const int col = tid % D, half = tid / D;
    const float* S = a.pool + (static_cast<size_t>(slot) * a.H + h) * D * D + col;
    const float* rows = sm + (half ? Sh::oQd : Sh::oKd);
    float acc[KP];
#pragma unroll
    for (int i = 0; i < KP; ++i) acc[i] = 0.f;
#pragma unroll 1
    for (int k0 = 0; k0 < D; k0 += 8) {
        float s[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) s[k] = __ldg(S + (k0 + k) * D);
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int i = 0; i < KP; i += 4) {
                const float4 r = *reinterpret_cast<const float4*>(rows + (k0 + k) * Sh::kPitch + i);
                acc[i] = fmaf(r.x, s[k], acc[i]);
                acc[i + 1] = fmaf(r.y, s[k], acc[i + 1]);
                acc[i + 2] = fmaf(r.z, s[k], acc[i + 2]);
                acc[i + 3] = fmaf(r.w, s[k], acc[i + 3]);
            }
    }
    float* u = sm + Sh::oU;
    if (half == 0) {
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            const uint64_t set = s_set[i];
            if (set == 0) continue;
            float x = bf16_bits_to_f32(a.v[(tok0 + static_cast<size_t>(i) * a.H) * D + col]) - acc[i];
            for (uint64_t left = set & ~(1ull << i); left;) {
                const int b = 63 - __clzll(left);
                left &= ~(1ull << b);
                x = fmaf(-sm[Sh::oM + i * KP + b], u[b * D + col], x);
            }
            u[i * D + col] = s_beta[i] * x;
        }
    }
    __syncthreads();
    if (half == 1) {
#pragma unroll
        for (int i = 0; i < KP; ++i) {
            if (i >= a.K) break;
            float o = 0.f;
            if (s_set[i]) {
                o = acc[i];
                for (uint64_t left = s_set[i]; left;) {
                    const int b = 63 - __clzll(left);
                    left &= ~(1ull << b);
                    o = fmaf(sm[Sh::oN + i * KP + b], u[b * D + col], o);
                }
            }
            const size_t at = (tok0 + static_cast<size_t>(i) * a.H) * D + col;
            if (a.out_f32) reinterpret_cast<float*>(a.out)[at] = o;
            else reinterpret_cast<uint16_t*>(a.out)[at] = f32_to_bf16_bits(o);
        }
    }
}

namespace {
template <int D, int KP>
int launch_tree_shape(const TreeArgs& a, cudaStream_t stream) {
    using Sh = TreeShape<D, KP>;
    static bool attr_done[kMaxDevicesAttr] = {};
    if (!raise_smem_limit(reinterpret_cast<const void*>(kda_tree_kernel<D, KP>), Sh::kBytes, attr_done)) return -3;
    kda_tree_kernel<D, KP><<<static_cast<unsigned>(a.N) * a.H, Sh::kThreads, Sh::kBytes, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}
template <int D>
int launch_tree_dim(const TreeArgs& a, cudaStream_t stream) {
    return a.K <= 8 ? launch_tree_shape<D, 8>(a, stream) : a.K <= 16 ? launch_tree_shape<D, 16>(a, stream)
         : a.K <= 32 ? launch_tree_shape<D, 32>(a, stream) : launch_tree_shape<D, 64>(a, stream);
}
}  // namespace

int launch_decode_tree(const uint16_t* q, const uint16_t* k, const uint16_t* v, const float* la, const uint16_t* beta,
                       const float* pool, int num_slots, const int32_t* slots, const int32_t* parents, void* out, int out_f32,
                       int N, int K, int H, int D, int decay, int* status, cudaStream_t stream)
{
    const TreeArgs a{q, k, v, la, beta, pool, slots, parents, out, num_slots, out_f32, N, K, H, decay, status};
    return D == 128 ? launch_tree_dim<128>(a, stream) : launch_tree_dim<64>(a, stream);
}

}  // namespace kda
