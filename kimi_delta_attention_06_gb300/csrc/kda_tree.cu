// kda_tree.cu -- the KDA recurrence along the branches of a tree of drafted tokens.
//
// Node i continues the state of its parent (the sequence's own state for a child of the last token):
//     S_i = (I - beta_i k_i k_i^T) Diag(alpha_i) S_parent(i) + beta_i k_i v_i^T,    o_i = S_i^T q_i.
// Written out along the path from the root to i, with A(i, a) the product of the alphas of the nodes after a on it
// (all of them for a = 0, the state before the tree), and u_i = beta_i (v_i - (alpha_i S_parent(i))^T k_i):
//     u_i = beta_i (v_i - S_0^T (A(i, 0) k_i) - sum_a [k_i . A(i, a) k_a] u_a)      a: the nodes before i on its path
//     o_i =              S_0^T (A(i, 0) q_i) + sum_a [q_i . A(i, a) k_a] u_a        and i itself (A = 1)
// So no node's state is formed: S_0 is read once, for one product with the 2 K decayed keys and queries.  The decays along
// a path are products of alphas, which neither overflow nor cancel.  With L_ab = beta_a [k_a . A(a, b) k_b] and N the
// second bracket, both on paths alone, and V, P, Q the rows v, S_0^T (A k), S_0^T (A q), that is
//     O = Q + W (V - P),      W = N (I + L)^-1 Diag(beta),
// where W is K x K numbers a head, a row of which a warp finds by substitution along the node's path; every column of
// the state then only takes the sum over a path.
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

template <bool WIDE> struct TreeBits { using type = uint32_t; };
template <> struct TreeBits<true> { using type = uint64_t; };
__device__ __forceinline__ int tree_top(uint32_t x) { return 31 - __clz(x); }
__device__ __forceinline__ int tree_top(uint64_t x) { return 63 - __clzll(x); }

template <int D, int KP>
__global__ void __launch_bounds__(256, TreeShape<D, KP>::kCols <= 256u ? 2 : 1)
kda_tree_kernel(const TreeArgs a)
{
    using Sh = TreeShape<D, KP>;
    using Set = typename TreeBits<(KP > 32)>::type;                     // a path: bit b is place b
    constexpr int KC = Sh::KC, kItems = Sh::kItems, C = D / 32, G = D / 64;
    constexpr Set kOne = 1;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = smem_raw + (1024u - (tc::smem_u32(smem_raw) & 1023u)) % 1024u;
    float* s_alpha = reinterpret_cast<float*>(sm + Sh::oAlpha);
    const uint16_t* s_value = reinterpret_cast<uint16_t*>(sm + Sh::oValue);
    float* s_m = reinterpret_cast<float*>(sm + Sh::oM);
    float* s_n = reinterpret_cast<float*>(sm + Sh::oN);                 // N, then W
    float* s_e = reinterpret_cast<float*>(sm + Sh::oU);                 // V - P (more than 32 places)
    uint64_t* s_set = reinterpret_cast<uint64_t*>(sm + Sh::oSet);
    float* s_beta = reinterpret_cast<float*>(sm + Sh::oBeta);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::oBar);        // [0..1] a buffer's products are done, [2] all are, [3..4] a buffer is written
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 6);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2;
    const uint32_t heads = static_cast<uint32_t>(a.N) * a.H, first = blockIdx.x * static_cast<uint32_t>(kItems);
    if (tid == 0) {
        tc::mbar_init(&bars[0], 1);
        tc::mbar_init(&bars[1], 1);
        tc::mbar_init(&bars[2], 1);
        tc::mbar_init(&bars[3], 128);
        tc::mbar_init(&bars[4], 128);
        tc::mbar_fence_init();
    }
    if (warp == 7) tc::tmem_alloc(s_tmem, Sh::kCols);
    // the items' sequence and head (past the last: the last again)
    int seq[kItems], head[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t x = min(first + i, heads - 1);
        seq[i] = static_cast<int>(x / static_cast<uint32_t>(a.H));
        head[i] = static_cast<int>(x - static_cast<uint32_t>(seq[i]) * a.H);
    }

    // 1. this thread's column of the state, half of the channels a group
    const int column = 32 * (warp & 3) + lane, item = kItems == 1 ? 0 : column / D, col = column % D;
    const bool there = first + item < heads;
    const int n = kItems == 1 || item == 0 ? seq[0] : seq[kItems - 1], h = kItems == 1 || item == 0 ? head[0] : head[kItems - 1];
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
    if (warp < kItems) {
        uint64_t set[2] = {0, 0};
        if (first + warp < heads &&
            tree_sets(a.parents + static_cast<long long>(warp == 0 ? seq[0] : seq[kItems - 1]) * a.K, a.K, lane, set) && lane == 0)
            set_status(a.status, kStatusTree);
        if (lane < KP) s_set[warp * KP + lane] = set[0];
        if (lane + 32 < KP) s_set[warp * KP + lane + 32] = set[1];
    }
    for (int e = warp; e < Sh::kNodes; e += 8) {                        // a warp a node
        const int it = e / KP, j = e % KP;
        if (j >= a.K) continue;
        const size_t tok = (static_cast<size_t>(it == 0 ? seq[0] : seq[kItems - 1]) * a.K + j) * a.H + (it == 0 ? head[0] : head[kItems - 1]);
        const size_t from = tok * D + lane * C;
        uint8_t* key = sm + Sh::oKey + (e * D + lane * C) * 2;
        float4 al;
        if constexpr (C == 4) {
            *reinterpret_cast<uint2*>(key) = *reinterpret_cast<const uint2*>(a.k + from);
            *reinterpret_cast<uint2*>(key + (Sh::oQuery - Sh::oKey)) = *reinterpret_cast<const uint2*>(a.q + from);
            *reinterpret_cast<uint2*>(key + (Sh::oValue - Sh::oKey)) = *reinterpret_cast<const uint2*>(a.v + from);
            if (a.decay == 0) al = *reinterpret_cast<const float4*>(a.la + from);
        } else {
            *reinterpret_cast<uint32_t*>(key) = *reinterpret_cast<const uint32_t*>(a.k + from);
            *reinterpret_cast<uint32_t*>(key + (Sh::oQuery - Sh::oKey)) = *reinterpret_cast<const uint32_t*>(a.q + from);
            *reinterpret_cast<uint32_t*>(key + (Sh::oValue - Sh::oKey)) = *reinterpret_cast<const uint32_t*>(a.v + from);
            if (a.decay == 0) {
                const float2 x = *reinterpret_cast<const float2*>(a.la + from);
                al.x = x.x; al.y = x.y;
            }
        }
        if (a.decay == 0) {
            al.x = expf(al.x);
            al.y = expf(al.y);
            if (C == 4) { al.z = expf(al.z); al.w = expf(al.w); }
        } else {
            al.x = a.decay == 1 ? expf(a.la[tok]) : 1.f;
            al.y = al.z = al.w = al.x;
        }
        if constexpr (C == 4) *reinterpret_cast<float4*>(s_alpha + e * D + lane * C) = al;
        else *reinterpret_cast<float2*>(s_alpha + e * D + lane * C) = make_float2(al.x, al.y);
        if (lane == 0) s_beta[e] = bf16_bits_to_f32(a.beta[tok]);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *s_tmem, lane_tm = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    bool ok = true;

    // S_0^T into TMEM: buffer b, 32 channels of this thread's half
    auto put = [&](int b, auto from) {
        uint32_t lead[32], rest[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float x = s[decltype(from)::value + i], y = tree_lead(x);
            lead[i] = __float_as_uint(y);
            rest[i] = __float_as_uint(x - y);
        }
        tc::tmem_st32x(lane_tm + b * 64, lead);
        tc::tmem_st32x(lane_tm + b * 64 + 32, rest);
        tc::tmem_wait_st();
        tc::fence_before_sync();
    };
    using Low = TreeInt<0>;
    using High = TreeInt<(kHalf > 32 ? 32 : 0)>;
    constexpr uint32_t id = tc::idesc(128, Sh::kRows, tc::kFmtTF32, false, false);
    auto product = [&](int b, int slab, int chunk, bool start) {        // buffer b times the slab of its channels (one thread)
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
        // 3. half a warp a node, up its path: L (less beta), N and the decayed rows, in their two terms.  Lane l of the 16:
        // channels 4 l .. + 3 of each 64
        const int hl = lane & 15;
        for (int f = 2 * warp + (lane >> 4); f < kItems * KC; f += 16) {
            const int it = f / KC, r = f % KC, i = chunk * KC + r, e = it * KP + i;
            const uint8_t* keys = sm + Sh::oKey + (it * KP * D + 4 * hl) * 2;
            const float* alphas = s_alpha + it * KP * D + 4 * hl;
            Set left = static_cast<Set>(s_set[e]);
            const bool node = left != 0;
            float2 key[2 * G], query[2 * G], p[2 * G];
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const uint2 x = *reinterpret_cast<const uint2*>(keys + (i * D + 64 * g) * 2);
                const uint2 y = *reinterpret_cast<const uint2*>(keys + (i * D + 64 * g) * 2 + (Sh::oQuery - Sh::oKey));
                key[2 * g] = bf16x2_bits_to_f32(node ? x.x : 0u);
                key[2 * g + 1] = bf16x2_bits_to_f32(node ? x.y : 0u);
                query[2 * g] = bf16x2_bits_to_f32(node ? y.x : 0u);
                query[2 * g + 1] = bf16x2_bits_to_f32(node ? y.y : 0u);
                p[2 * g] = p[2 * g + 1] = make_float2(1.f, 1.f);
            }
            while (__any_sync(0xffffffffu, left != 0)) {                // 4 nodes of the path at a time
                float v[8];                                             // their products with the key, then with the query
                int b4[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) {
                    const bool on = left != 0;
                    const int b = on ? tree_top(left) : 0;
                    left &= ~(kOne << b);
                    b4[z] = on ? b : -1;
                    float2 m, w;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const uint2 x = *reinterpret_cast<const uint2*>(keys + (b * D + 64 * g) * 2);
                        const float4 al = *reinterpret_cast<const float4*>(alphas + b * D + 64 * g);
                        const float2 k0 = fmul2(p[2 * g], bf16x2_bits_to_f32(x.x)), k1 = fmul2(p[2 * g + 1], bf16x2_bits_to_f32(x.y));
                        m = g == 0 ? fmul2(key[0], k0) : ffma2(key[2 * g], k0, m);
                        w = g == 0 ? fmul2(query[0], k0) : ffma2(query[2 * g], k0, w);
                        m = ffma2(key[2 * g + 1], k1, m);
                        w = ffma2(query[2 * g + 1], k1, w);
                        if (on) {
                            p[2 * g] = fmul2(p[2 * g], make_float2(al.x, al.y));
                            p[2 * g + 1] = fmul2(p[2 * g + 1], make_float2(al.z, al.w));
                        }
                    }
                    v[z] = m.x + m.y;
                    v[z + 4] = w.x + w.y;
                }
                // 8 sums over the 16 lanes, halved from step to step: lane l has sum l / 2 in the end
                auto halve = [&](int off, int count) {
                    const bool up = (lane & off) != 0;
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (z < count) {
                            const float give = up ? v[z] : v[z + count];
                            v[z] = (up ? v[z + count] : v[z]) + __shfl_xor_sync(0xffffffffu, give, off);
                        }
                };
                halve(8, 4);
                halve(4, 2);
                halve(2, 1);
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
                const int b = lane & 4 ? (lane & 2 ? b4[3] : b4[2]) : (lane & 2 ? b4[1] : b4[0]);
                if ((lane & 1) == 0 && b >= 0) (lane & 8 ? s_n : s_m)[(it * KP + i) * KP + b] = v[0];
            }
            const uint32_t rk = it * 2 * KC + r;
#pragma unroll
            for (int g = 0; g < G; ++g) {
                auto split = [&](uint32_t row, float2 x, float2 y) {
                    uint8_t* d = sm + Sh::oRows + tc::sw128_off32(row, 64 * g + 4 * hl, Sh::kRows);
                    const float4 lead = make_float4(tree_lead(x.x), tree_lead(x.y), tree_lead(y.x), tree_lead(y.y));
                    *reinterpret_cast<float4*>(d) = lead;
                    *reinterpret_cast<float4*>(d + Sh::kTile) = make_float4(x.x - lead.x, x.y - lead.y, y.x - lead.z, y.y - lead.w);
                };
                split(rk, fmul2(p[2 * g], key[2 * g]), fmul2(p[2 * g + 1], key[2 * g + 1]));
                split(rk + KC, fmul2(p[2 * g], query[2 * g]), fmul2(p[2 * g + 1], query[2 * g + 1]));
            }
        }
        tc::fence_smem_to_async();
        // 4. the product
        if (chunk == 0) {
            if constexpr (Sh::kWhole) {
                put(group * (Sh::kSlabs / 2), Low{});
                if constexpr (kHalf > 32) put(group * (Sh::kSlabs / 2) + 1, High{});
            } else {
                put(group, Low{});
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
                put(group, High{});
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
        if (chunk + 1 < Sh::kChunks) {                                  // the rows are written again
            ok = tc::mbar_wait_bounded(&bars[2], chunk & 1, kWaitLimitNs) && ok;
            ok = __all_sync(0xffffffffu, ok);
            __syncthreads();
        }
    }

    // 5. W while the products run: a warp a row, lane b place b (and b + 32): w_c is final once the places above c are done
    for (int e = warp; e < Sh::kNodes; e += 8) {
        const int it = e / KP, i = e % KP;
        const Set on = static_cast<Set>(s_set[e]);
        if (on == 0) continue;
        constexpr int P = KP > 32 ? 2 : 1;
        float w[P];
        float* row = s_n + (it * KP + i) * KP;
#pragma unroll
        for (int z = 0; z < P; ++z) w[z] = on >> (lane & (KP - 1)) + 32 * z & 1 ? row[(lane & (KP - 1)) + 32 * z] : 0.f;
        for (Set left = on; left & (left - 1);) {                       // (nothing is below the path's first node)
            const int c = tree_top(left);
            left &= ~(kOne << c);
            float wc = __shfl_sync(0xffffffffu, w[0], c & 31);
            if constexpr (P == 2) {
                const float hi = __shfl_sync(0xffffffffu, w[1], c & 31);
                wc = c >= 32 ? hi : wc;
            }
            wc *= s_beta[it * KP + c];
#pragma unroll
            for (int z = 0; z < P; ++z) {
                const int b = (lane & (KP - 1)) + 32 * z;
                if (left >> b & 1) w[z] = fmaf(-wc, s_m[(it * KP + c) * KP + b], w[z]);
            }
        }
#pragma unroll
        for (int z = 0; z < P; ++z) {
            const int b = lane + 32 * z;
            if (b < KP && (on >> b & 1)) row[b] = w[z] * s_beta[it * KP + b];
        }
    }
    ok = tc::mbar_wait_bounded(&bars[2], (Sh::kChunks - 1) & 1, kWaitLimitNs) && ok;
    ok = __all_sync(0xffffffffu, ok);
    __syncthreads();
    tc::fence_after_sync();

    // 6. a column a thread, 8 places a group in turn
    const uint64_t* set = s_set + item * KP;
    const float* W = s_n + item * KP * KP;
    auto rows_at = [&](int i, int query) {                              // TMEM columns of places i .. i + 7
        return lane_tm + Sh::kD + (i / KC) * Sh::kRows + item * 2 * KC + query * KC + i % KC;
    };
    auto value = [&](int i) { return bf16_bits_to_f32(s_value[(item * KP + i) * D + col]); };
    const size_t step = static_cast<size_t>(a.H) * D;
    const size_t to = (static_cast<size_t>(n) * a.K * a.H + h) * D + col;
    auto give = [&](int i, float o) {
        if (!good || !ok || i >= a.K) return;
        if (a.out_f32) reinterpret_cast<float*>(a.out)[to + i * step] = o;
        else reinterpret_cast<uint16_t*>(a.out)[to + i * step] = f32_to_bf16_bits(o);
    };
    if constexpr (KP <= 32) {
        float e[KP];                                                    // V - P (of places without a node: anything, not used)
#pragma unroll
        for (int i0 = 0; i0 < KP; i0 += 8) {
            if (i0 >= a.K) break;
            float P[8];
            tree_tmem_ld8(rows_at(i0, 0), P);
#pragma unroll
            for (int r = 0; r < 8; ++r) e[i0 + r] = value(i0 + r) - P[r];
        }
#pragma unroll
        for (int i0 = 0; i0 < KP; i0 += 8) {
            if (i0 >= a.K) break;
            if ((KP == 8 ? 0 : i0 / 8 & 1) != group) continue;
            float o[8];
            tree_tmem_ld8(rows_at(i0, 1), o);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int i = i0 + r;
                const uint32_t on = static_cast<uint32_t>(set[i]);
                float x = o[r], y = 0.f;
                // (what is not on the path is left out, not multiplied by zero: it may hold anything)
#pragma unroll
                for (int b = 0; b <= i; b += 4) {
                    if ((on >> b & 15) == 0) continue;
                    const float4 w = *reinterpret_cast<const float4*>(W + i * KP + b);
                    if (on >> b & 1) x = fmaf(w.x, e[b], x);
                    if (b + 1 < KP && (on >> (b + 1) & 1)) y = fmaf(w.y, e[b + 1], y);
                    if (b + 2 < KP && (on >> (b + 2) & 1)) x = fmaf(w.z, e[b + 2], x);
                    if (b + 3 < KP && (on >> (b + 3) & 1)) y = fmaf(w.w, e[b + 3], y);
                }
                give(i, on ? x + y : 0.f);
            }
        }
    } else {
        float* e = s_e + item * KP * D + col;
#pragma unroll 1
        for (int i0 = 8 * group; i0 < a.K; i0 += 16) {
            float P[8];
            tree_tmem_ld8(rows_at(i0, 0), P);
#pragma unroll
            for (int r = 0; r < 8; ++r) e[(i0 + r) * D] = value(i0 + r) - P[r];
        }
        __syncthreads();
#pragma unroll 1
        for (int i0 = 8 * group; i0 < a.K; i0 += 16) {
            float o[8];
            tree_tmem_ld8(rows_at(i0, 1), o);
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const Set on = static_cast<Set>(set[i0 + r]);
                float x = o[r];
                for (Set left = on; left;) {                            // 4 of the path at a time, their loads together
                    int b4[4];
                    float m[4], w[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        b4[z] = left ? tree_top(left) : -1;
                        if (left) left &= ~(kOne << b4[z]);
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        m[z] = W[(i0 + r) * KP + max(b4[z], 0)];
                        w[z] = e[max(b4[z], 0) * D];
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        if (b4[z] >= 0) x = fmaf(m[z], w[z], x);
                }
                give(i0 + r, on ? x : 0.f);
            }
        }
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
