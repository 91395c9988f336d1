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
//
// The product P^T [128 columns x 2 K] = S_0^T [128 x D] rows^T [D x 2 K] runs on the tensor cores with S_0^T in TMEM (its
// lanes are the state's columns, so a warp's loads of a state's row are 128 contiguous bytes and nothing passes through
// shared memory), as three tf32 products of the operands' leading 11 bits and what is left of them: 22 bits, an fp32
// product but for 2^-21.  A thread of the epilogue then has one column of all rows.
#include "common.cuh"
#include "tc.cuh"
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

// A CTA takes 128 columns: one head's state of 128 x 128, or two of 64 x 64 (items).  Nodes go through the product
// in chunks of at most 32, so that their rows fit beside the rest.
template <int D, int KP>
struct TreeShape {
    static constexpr int kThreads = 256, kItems = 128 / D;
    static constexpr int KC = KP < 32 ? KP : 32, kChunks = KP / KC;
    static constexpr int kRows = kItems * 2 * KC;                       // N of a product: per item the keys, then the queries
    static constexpr int kSlabs = D / 32;                               // 32 channels: 128 bytes of a row of fp32
    static constexpr uint32_t kTile = kRows * 128u * kSlabs;            // one term of the rows
    static constexpr bool kWhole = kChunks > 1 || D == 64;              // S_0 stays in TMEM (else a quarter at a time, in turns)
    static constexpr int kBufs = kWhole ? kSlabs : 2;                   // buffers of 32 channels (leading bits, the rest)
    static constexpr uint32_t kD = kBufs * 64u;                         // TMEM column of the accumulators
    static constexpr uint32_t kUsed = kD + kChunks * kRows;
    static constexpr uint32_t kCols = kUsed <= 256u ? 256u : 512u;
    static_assert(kUsed <= 512u, "TMEM");
    static constexpr int kNodes = kItems * KP;
    // bytes of shared memory
    static constexpr uint32_t oRows = 0, oAlpha = 2 * kTile;            // rows: leading bits, the rest
    static constexpr uint32_t oKey = oAlpha + kNodes * D * 4u, oQuery = oKey + kNodes * D * 2u, oValue = oQuery + kNodes * D * 2u;
    static constexpr uint32_t oM = oValue + kNodes * D * 2u, oN = oM + kItems * KP * KP * 4u;
    static constexpr uint32_t oU = oAlpha;                              // [node][column] (once the decays are done with)
    static constexpr uint32_t oSet = oN + kItems * KP * KP * 4u, oBeta = oSet + kNodes * 8u, oBar = oBeta + kNodes * 4u;
    static constexpr uint32_t kBytes = oBar + 64u + 1024u;              // (the base is moved up to 1024 bytes)
    static_assert(kBytes <= 232448u, "227 KB of shared memory");
};

__device__ __forceinline__ void tree_tmem_ld8(uint32_t ta, float (&r)[8]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(ta));
    tc::tmem_wait_ld();
}
// D += A B, A (tf32) in TMEM.
__device__ __forceinline__ void tree_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], %2, %3, p;\n\t}\n"
        :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(acc));
}
template <int V> struct TreeInt { static constexpr int value = V; };
// The leading 11 bits of x; x less these is exact.
__device__ __forceinline__ float tree_lead(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

template <int D, int KP>
__global__ void __launch_bounds__(256, TreeShape<D, KP>::kCols <= 256u ? 2 : 1)
kda_tree_kernel(const TreeArgs a)
{
    using Sh = TreeShape<D, KP>;
    constexpr int KC = Sh::KC, kItems = Sh::kItems, C = D / 32;         // C: channels a lane
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (1024u - (tc::smem_u32(smem_raw) & 1023u)) % 1024u;
    float* s_alpha = reinterpret_cast<float*>(sm + Sh::oAlpha);
    const uint16_t* s_key = reinterpret_cast<uint16_t*>(sm + Sh::oKey);
    const uint16_t* s_query = reinterpret_cast<uint16_t*>(sm + Sh::oQuery);
    const uint16_t* s_value = reinterpret_cast<uint16_t*>(sm + Sh::oValue);
    float* s_m = reinterpret_cast<float*>(sm + Sh::oM);
    float* s_n = reinterpret_cast<float*>(sm + Sh::oN);
    float* s_u = reinterpret_cast<float*>(sm + Sh::oU);
    uint64_t* s_set = reinterpret_cast<uint64_t*>(sm + Sh::oSet);
    float* s_beta = reinterpret_cast<float*>(sm + Sh::oBeta);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::oBar);        // [0..1] a buffer's products are done, [2] all are, [3..4] a buffer is written
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 6);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2;
    const long long heads = static_cast<long long>(a.N) * a.H, first = static_cast<long long>(blockIdx.x) * kItems;
    if (tid == 0) {
        tc::mbar_init(&bars[0], 1);
        tc::mbar_init(&bars[1], 1);
        tc::mbar_init(&bars[2], 1);
        tc::mbar_init(&bars[3], 128);
        tc::mbar_init(&bars[4], 128);
        tc::mbar_fence_init();
    }
    if (warp == 7) tc::tmem_alloc(s_tmem, Sh::kCols);

    // 1. this thread's column of the state, half of the channels a group
    const int column = 32 * (warp & 3) + lane, item = column / D, col = column % D;
    const bool there = first + item < heads;
    const long long at = there ? first + item : heads - 1;              // n * H + h
    const int n = static_cast<int>(at / a.H), h = static_cast<int>(at - static_cast<long long>(n) * a.H);
    const int slot = a.slots ? a.slots[n] : n;
    const bool good = there && slot >= 0 && slot < a.num_slots;
    if (there && !good && col == 0 && group == 0) set_status(a.status, kStatusTree);
    constexpr int kHalf = D / 2;
    float s[kHalf];
    {
        const float* S = a.pool + ((good ? static_cast<size_t>(slot) : 0) * a.H + h) * D * D + group * kHalf * D + col;
#pragma unroll
        for (int k = 0; k < kHalf; ++k) s[k] = __ldcs(S + k * D);
    }

    // 2. the trees and the nodes' inputs
    if (warp < kItems && first + warp < heads) {
        const int seq = static_cast<int>((first + warp) / a.H);
        uint64_t set[2];
        if (tree_sets(a.parents + static_cast<long long>(seq) * a.K, a.K, lane, set) && lane == 0) set_status(a.status, kStatusTree);
        if (lane < KP) s_set[warp * KP + lane] = set[0];
        if (lane + 32 < KP) s_set[warp * KP + lane + 32] = set[1];
    } else if (warp < kItems) {
        for (int i = lane; i < KP; i += 32) s_set[warp * KP + i] = 0;
    }
    for (int e = warp; e < Sh::kNodes; e += 8) {                        // a warp a node
        const int it = e / KP, j = e % KP;
        if (j >= a.K || first + it >= heads) continue;
        const long long nh = first + it;
        const long long sq = nh / a.H;
        const size_t tok = static_cast<size_t>(sq * a.K + j) * a.H + static_cast<size_t>(nh - sq * a.H);
        const size_t from = tok * D + lane * C;
        uint8_t* key = sm + Sh::oKey + (e * D + lane * C) * 2;
        float al[C];
        if constexpr (C == 4) {
            *reinterpret_cast<uint2*>(key) = *reinterpret_cast<const uint2*>(a.k + from);
            *reinterpret_cast<uint2*>(key + (Sh::oQuery - Sh::oKey)) = *reinterpret_cast<const uint2*>(a.q + from);
            *reinterpret_cast<uint2*>(key + (Sh::oValue - Sh::oKey)) = *reinterpret_cast<const uint2*>(a.v + from);
        } else {
            *reinterpret_cast<uint32_t*>(key) = *reinterpret_cast<const uint32_t*>(a.k + from);
            *reinterpret_cast<uint32_t*>(key + (Sh::oQuery - Sh::oKey)) = *reinterpret_cast<const uint32_t*>(a.q + from);
            *reinterpret_cast<uint32_t*>(key + (Sh::oValue - Sh::oKey)) = *reinterpret_cast<const uint32_t*>(a.v + from);
        }
        if (a.decay == 0) {
#pragma unroll
            for (int c = 0; c < C; ++c) al[c] = a.la[from + c];
        } else {
            const float one = a.decay == 1 ? a.la[tok] : 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) al[c] = one;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) s_alpha[e * D + lane * C + c] = expf(al[c]);
        if (lane == 0) s_beta[e] = bf16_bits_to_f32(a.beta[tok]);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *s_tmem, lane_tm = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    bool ok = true;

    // S_0^T into TMEM: buffer b, channels `c0` .. + 31 of this thread's (its half of them)
    auto put = [&](int b, auto c0) {
        uint32_t lead[32], rest[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float x = s[c0() + i], y = tree_lead(x);
            lead[i] = __float_as_uint(y);
            rest[i] = __float_as_uint(x - y);
        }
        tc::tmem_st32x(lane_tm + b * 64, lead);
        tc::tmem_st32x(lane_tm + b * 64 + 32, rest);
        tc::tmem_wait_st();
        tc::fence_before_sync();
    };
    auto zero = [] { return 0; };
    auto second = [] { return kHalf > 32 ? 32 : 0; };
    // slab of the rows that a buffer of this turn stands for
    constexpr uint32_t id = tc::idesc(128, Sh::kRows, tc::kFmtTF32, false, false);
    auto product = [&](int b, int slab, int chunk, bool start) {        // one thread
        const uint32_t d = tm + Sh::kD + chunk * Sh::kRows, ta = tm + b * 64;
        const uint32_t lead = tc::smem_u32(sm) + Sh::oRows + slab * (Sh::kRows * 128u);
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            const uint64_t bl = tc::sdesc(lead + k * 32u, 16, 1024, tc::kSwizzle128B);
            const uint64_t br = tc::sdesc(lead + Sh::kTile + k * 32u, 16, 1024, tc::kSwizzle128B);
            tree_mma(d, ta + k * 8u, bl, id, start && k == 0 ? 0u : 1u);
            tree_mma(d, ta + k * 8u, br, id, 1u);
            tree_mma(d, ta + 32u + k * 8u, bl, id, 1u);
        }
    };

#pragma unroll 1
    for (int chunk = 0; chunk < Sh::kChunks; ++chunk) {
        // 3. a warp a node, up its path: M, N and the decayed rows, in their two terms
        for (int f = warp; f < kItems * KC; f += 8) {
            const int it = f / KC, r = f % KC, i = chunk * KC + r, e = it * KP + i;
            uint64_t left = s_set[e];
            float key[C], query[C], p[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const bool on = left != 0;
                key[c] = on ? bf16_bits_to_f32(s_key[e * D + lane * C + c]) : 0.f;
                query[c] = on ? bf16_bits_to_f32(s_query[e * D + lane * C + c]) : 0.f;
                p[c] = 1.f;
            }
            while (left) {                                      // 4 nodes of the path at a time
                float v[8];                                     // their products with the key, then with the query
                int b4[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const bool on = left != 0;
                    const int b = on ? 63 - __clzll(left) : 0, eb = it * KP + b;
                    left &= ~(1ull << b);
                    b4[z] = on ? b : -1;
                    v[z] = v[z + 4] = 0.f;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        const float kb = p[c] * bf16_bits_to_f32(s_key[eb * D + lane * C + c]);
                        v[z] = fmaf(key[c], kb, v[z]);
                        v[z + 4] = fmaf(query[c], kb, v[z + 4]);
                        const float al = s_alpha[eb * D + lane * C + c];
                        p[c] = on ? p[c] * al : p[c];
                    }
                }
                // 8 sums over the lanes, halved from step to step: lane l has sum l / 4 in the end
                auto halve = [&](int off, int count) {
                    const bool up = (lane & off) != 0;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (z < count) {
                            const float give = up ? v[z] : v[z + count];
                            v[z] = (up ? v[z + count] : v[z]) + __shfl_xor_sync(0xffffffffu, give, off);
                        }
                };
                halve(16, 4);
                halve(8, 2);
                halve(4, 1);
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
                const int z = lane >> 2 & 3;
                const int b = z == 0 ? b4[0] : z == 1 ? b4[1] : z == 2 ? b4[2] : b4[3];
                if ((lane & 3) == 0 && b >= 0) (lane < 16 ? s_m : s_n)[(it * KP + i) * KP + b] = v[0];
            }
            const uint32_t rk = it * 2 * KC + r, rq = rk + KC;
            float kl[C], kr[C], ql[C], qr[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float x = p[c] * key[c], y = p[c] * query[c];
                kl[c] = tree_lead(x); kr[c] = x - kl[c];
                ql[c] = tree_lead(y); qr[c] = y - ql[c];
            }
            uint8_t* dk = sm + Sh::oRows + tc::sw128_off32(rk, lane * C, Sh::kRows);
            uint8_t* dq = sm + Sh::oRows + tc::sw128_off32(rq, lane * C, Sh::kRows);
            if constexpr (C == 4) {
                *reinterpret_cast<float4*>(dk) = make_float4(kl[0], kl[1], kl[2], kl[3]);
                *reinterpret_cast<float4*>(dk + Sh::kTile) = make_float4(kr[0], kr[1], kr[2], kr[3]);
                *reinterpret_cast<float4*>(dq) = make_float4(ql[0], ql[1], ql[2], ql[3]);
                *reinterpret_cast<float4*>(dq + Sh::kTile) = make_float4(qr[0], qr[1], qr[2], qr[3]);
            } else {
                *reinterpret_cast<float2*>(dk) = make_float2(kl[0], kl[1]);
                *reinterpret_cast<float2*>(dk + Sh::kTile) = make_float2(kr[0], kr[1]);
                *reinterpret_cast<float2*>(dq) = make_float2(ql[0], ql[1]);
                *reinterpret_cast<float2*>(dq + Sh::kTile) = make_float2(qr[0], qr[1]);
            }
        }
        tc::fence_smem_to_async();
        // 4. the product
        if (chunk == 0) {
            if constexpr (Sh::kWhole) {
                put(group * (Sh::kSlabs / 2), zero);
                if constexpr (kHalf > 32) put(group * (Sh::kSlabs / 2) + 1, second);
            } else {
                put(group, zero);
            }
        }
        __syncthreads();
        if (warp == 0) {
            tc::fence_after_sync();
            if (tc::elect_one()) {
                if constexpr (Sh::kWhole) {
                    for (int b = 0; b < Sh::kBufs; ++b) product(b, b, chunk, b == 0);
                    tc::mma_commit(&bars[2]);
                } else {
                    product(0, 0, 0, true);
                    tc::mma_commit(&bars[0]);
                    product(1, 2, 0, false);
                    tc::mma_commit(&bars[1]);
                }
            }
            __syncwarp();
        }
        if constexpr (!Sh::kWhole) {
            // the second quarters follow where the first have been read
            ok = tc::mbar_wait_bounded(&bars[group], 0, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
                tc::fence_after_sync();
                put(group, second);
            }
            tc::mbar_arrive(&bars[3 + group]);
            if (warp == 0) {
                for (int b = 0; b < 2; ++b) {
                    ok = tc::mbar_wait_bounded(&bars[3 + b], 0, kWaitLimitNs) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
                    if (tc::elect_one()) {
                        product(b, 1 + 2 * b, 0, false);
                        if (b == 1) tc::mma_commit(&bars[2]);
                    }
                    __syncwarp();
                }
            }
        }
        ok = tc::mbar_wait_bounded(&bars[2], chunk & 1, kWaitLimitNs) && ok;
        ok = __all_sync(0xffffffffu, ok);
        tc::fence_after_sync();
        if (Sh::kChunks > 1) __syncthreads();
    }

    // 5. a column a thread: u by the first group, up to KP of them
    const uint64_t* set = s_set + item * KP;
    const float* beta = s_beta + item * KP;
    const float* M = s_m + item * KP * KP;
    const float* Nn = s_n + item * KP * KP;
    float* u = s_u + item * KP * D + col;                               // [node] D apart
    auto rows_at = [&](int i, int query) {                              // TMEM columns of nodes i .. i + 7
        return lane_tm + Sh::kD + (i / KC) * Sh::kRows + item * 2 * KC + query * KC + i % KC;
    };
    // x - sum of row[b] u[b] over the nodes of `on`: up to 16 places from registers, whose u do not wait for shared memory
    // (a place that is not on the path is left out, not multiplied by zero: it may hold anything); else 4 of the path at
    // a time, their loads together
    constexpr bool kRegs = KP <= 16;
    float ur[kRegs ? KP : 1];
    auto along = [&](float x, const float* row, uint64_t on, auto upto, float sign) {
        if constexpr (kRegs) {
            constexpr int n4 = (decltype(upto)::value + 3) / 4;
            const uint32_t bits = static_cast<uint32_t>(on);
            float4 m[n4 > 0 ? n4 : 1];
#pragma unroll
            for (int q = 0; q < n4; ++q) m[q] = reinterpret_cast<const float4*>(row)[q];
            float y = 0.f;
#pragma unroll
            for (int q = 0; q < n4; ++q) {
                if (bits >> (4 * q) & 1) x = fmaf(sign * m[q].x, ur[4 * q], x);
                if (bits >> (4 * q + 1) & 1) y = fmaf(sign * m[q].y, ur[4 * q + 1], y);
                if (bits >> (4 * q + 2) & 1) x = fmaf(sign * m[q].z, ur[4 * q + 2], x);
                if (bits >> (4 * q + 3) & 1) y = fmaf(sign * m[q].w, ur[4 * q + 3], y);
            }
            return x + y;
        } else {
            while (on) {
                int b4[4];
                float m[4], w[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    b4[z] = on ? 63 - __clzll(on) : -1;
                    if (on) on &= ~(1ull << b4[z]);
                }
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    m[z] = row[max(b4[z], 0)];
                    w[z] = u[max(b4[z], 0) * D];
                }
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (b4[z] >= 0) x = fmaf(sign * m[z], w[z], x);
            }
            return x;
        }
    };
    // a step for every place 0 .. KP - 1, unrolled where u is in registers
    auto nodes8 = [&](auto i0, auto&& use) {
        constexpr int z = decltype(i0)::value;
        use(TreeInt<z>{}, 0); use(TreeInt<z + 1>{}, 1); use(TreeInt<z + 2>{}, 2); use(TreeInt<z + 3>{}, 3);
        use(TreeInt<z + 4>{}, 4); use(TreeInt<z + 5>{}, 5); use(TreeInt<z + 6>{}, 6); use(TreeInt<z + 7>{}, 7);
    };
    auto solve = [&](auto z0, int i0) {                                 // u of places i0 .. i0 + 7 (z0: the same, if unrolled)
        float P[8];
        tree_tmem_ld8(rows_at(i0, 0), P);
        nodes8(z0, [&](auto z, int r) {
            const int i = i0 + r;
            const uint64_t on = set[i];
            float x = 0.f;
            if (on) {
                x = bf16_bits_to_f32(s_value[(item * KP + i) * D + col]) - P[r];
                x = beta[i] * along(x, M + i * KP, on & ~(1ull << i), z, -1.f);
                u[i * D] = x;
            }
            if constexpr (kRegs) ur[decltype(z)::value] = x;
        });
    };
    auto answer = [&](auto z0, int i0) {                                // outputs of places i0 .. i0 + 7
        float P[8];
        tree_tmem_ld8(rows_at(i0, 1), P);
        nodes8(z0, [&](auto z, int r) {
            const int i = i0 + r;
            const uint64_t on = set[i];
            float o = 0.f;
            if (on) o = along(P[r], Nn + i * KP, on, TreeInt<decltype(z)::value + 1>{}, 1.f);
            if (good && ok && i < a.K) {
                const size_t to = ((static_cast<size_t>(n) * a.K + i) * a.H + h) * D + col;
                if (a.out_f32) reinterpret_cast<float*>(a.out)[to] = o;
                else reinterpret_cast<uint16_t*>(a.out)[to] = f32_to_bf16_bits(o);
            }
        });
    };
    if (group == 0) {
        if constexpr (kRegs) {
            solve(TreeInt<0>{}, 0);
            if constexpr (KP > 8) solve(TreeInt<8>{}, 8);
        } else {
#pragma unroll 1
            for (int i0 = 0; i0 < a.K; i0 += 8) solve(TreeInt<0>{}, i0);
        }
    }
    __syncthreads();
    // 6. the outputs: the first places (whose paths are short) by the group that has u at hand
    if constexpr (kRegs) {
        if (group == 0) {
            answer(TreeInt<0>{}, 0);
        } else if constexpr (KP > 8) {
#pragma unroll
            for (int i = 0; i < KP; ++i) ur[i] = u[i * D];              // (unset where there is no node: not used)
            answer(TreeInt<8>{}, 8);
        }
    } else {
#pragma unroll 1
        for (int i0 = 8 * group; i0 < a.K; i0 += 16) answer(TreeInt<0>{}, i0);
    }
    if (!ok) set_status(a.status, kStatusTimeout);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 7) tc::tmem_dealloc(tm, Sh::kCols);
}

namespace {
template <int D, int KP>
int launch_tree_shape(const TreeArgs& a, cudaStream_t stream) {
    using Sh = TreeShape<D, KP>;
    static bool attr_done[kMaxDevicesAttr] = {};
    if (!raise_smem_limit(reinterpret_cast<const void*>(kda_tree_kernel<D, KP>), Sh::kBytes, attr_done)) return -3;
    const long long heads = static_cast<long long>(a.N) * a.H;
    kda_tree_kernel<D, KP><<<static_cast<unsigned>((heads + Sh::kItems - 1) / Sh::kItems), Sh::kThreads, Sh::kBytes, stream>>>(a);
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
