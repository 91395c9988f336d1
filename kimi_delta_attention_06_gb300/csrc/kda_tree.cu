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
// where W is K x K numbers a head, a row of which a warp finds by substitution along the node's path.
//
// The product P^T [128 columns x 2 K] = S_0^T [128 x D] rows^T [D x 2 K] runs on the tensor cores with S_0^T in TMEM (its
// lanes are the state's columns, so a warp's loads of a state's row are 128 contiguous bytes and nothing passes through
// shared memory), as three tf32 products of the operands' leading 11 bits and what is left of them: 22 bits, an fp32
// product but for 2^-21.  So do L and N, as products of the decayed rows with the keys over their decays (CTAs in which a
// decay leaves 2^-100 .. 2^100 walk their paths instead), and W (V - P), with V - P in TMEM in S_0^T's place (a NaN
// or an infinity in it enters as 0, and is put back for the nodes whose paths hold it: 0 * NaN is none).
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
    // L and N have accumulators of their own where there is room, else those of the product, before it
    static constexpr uint32_t kProduct = kD + kChunks * kRows;
    static constexpr bool kApart = kProduct + kChunks * kRows <= (kProduct <= 256u ? 256u : 512u);
    static constexpr uint32_t kL = kApart ? kProduct : kD;
    static constexpr uint32_t kUsed = kL + kChunks * kRows;
    static constexpr uint32_t kCols = kUsed <= 256u ? 256u : 512u;
    static_assert(kUsed <= 512u && 2 * KP <= kD, "TMEM");
    static constexpr int kNodes = kItems * KP;
    static constexpr uint32_t kSide = kNodes * 128u * kSlabs;           // one term of the keys over their decays
    // bytes of shared memory.  (The side's products read 64 rows from each item's first: what follows it, beyond KP)
    static constexpr uint32_t oSide = 0, oRows = oSide + 2 * kSide, oDecay = oRows + 2 * kTile;
    static constexpr uint32_t oM = kChunks > 1 ? oDecay + kNodes * D * 4u : oDecay;        // (one chunk: the decays are done with)
    static constexpr uint32_t kMN = kItems * KP * KP * 4u, oN = oM + kMN;
    static constexpr uint32_t oLog = oRows;                             // log alphas as they arrive
    // W [place][32 places a slab] in two terms, in the side's place; V in the decays'
    static constexpr int kWRows = KP < 16 ? 16 : KP, kWSlabs = KP > 32 ? 2 : 1;
    static constexpr uint32_t kW = kItems * kWRows * 128u * kWSlabs, oW = oSide;
    static constexpr bool kVSide = oM == oDecay && 2 * kMN + kNodes * D * 2u > kNodes * D * 4u;
    static constexpr uint32_t oV = kVSide ? oW + 2 * kW : oM == oDecay ? oDecay + 2 * kMN : oDecay;
    static_assert(2 * kW + (kVSide ? kNodes * D * 2u : 0u) <= 2 * kSide, "W in the side's place");
    static_assert(kNodes * D * 4u <= 2 * kTile, "log alphas in the rows' place");
    static constexpr uint32_t kPast = oN + kMN > oDecay + kNodes * D * 4u ? oN + kMN : oDecay + kNodes * D * 4u;
    static constexpr uint32_t oSet = kPast, oBeta = oSet + kNodes * 8u, oBar = oBeta + kNodes * 4u;
    static constexpr uint32_t kBytes = oBar + 64u;
    static_assert(kBytes <= 232448u && (kCols > 256u || kBytes <= 115712u), "227 KB of shared memory, or 113");
    static_assert(oRows + 2 * kTile >= oSide + 2 * kSide + 8192u, "the side's last products stay within");
};

__device__ __forceinline__ void tree_tmem_ld8(uint32_t ta, float (&r)[8]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                 : "r"(ta));
    tc::tmem_wait_ld();
}
__device__ __forceinline__ void tree_tmem_st8(uint32_t ta, const float (&r)[8]) {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(r);
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 :: "r"(ta), "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7]) : "memory");
}
// D += A B in tf32, A in TMEM or shared memory; descriptors by their low words (the addresses; kTreeDesc: the high word).
constexpr uint32_t kTreeDesc = 1024u >> 4 | 1u << 14 | tc::kSwizzle128B << 29;
__device__ __forceinline__ uint32_t tree_desc(uint32_t saddr) { return (saddr >> 4 & 0x3fffu) | (16u >> 4) << 16; }
__device__ __forceinline__ void tree_mma(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], [%1], b, %4, p;\n\t}\n"
        :: "r"(d), "r"(a), "r"(b), "r"(kTreeDesc), "r"(id), "r"(acc));
}
__device__ __forceinline__ void tree_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::tf32 [%0], a, b, %4, p;\n\t}\n"
        :: "r"(d), "r"(a), "r"(b), "r"(kTreeDesc), "r"(id), "r"(acc));
}
__device__ __forceinline__ void tree_copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void tree_copy4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void tree_copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
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
    constexpr int KC = Sh::KC, kItems = Sh::kItems, G = D / 64;
    constexpr Set kOne = 1;
    extern __shared__ __align__(1024) uint8_t sm[];
    float* s_decay = reinterpret_cast<float*>(sm + Sh::oDecay);         // [place][channel]: products of alphas from the root
    float* s_m = reinterpret_cast<float*>(sm + Sh::oM);
    float* s_n = reinterpret_cast<float*>(sm + Sh::oN);                 // N, then W
    uint64_t* s_set = reinterpret_cast<uint64_t*>(sm + Sh::oSet);
    float* s_beta = reinterpret_cast<float*>(sm + Sh::oBeta);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::oBar);        // [0..1] a buffer's products are done, [2] all are, [3..4] a buffer is written, [5] L's and N's, [6] W's
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 7);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, group = warp >> 2;
    const uint32_t heads = static_cast<uint32_t>(a.N) * a.H, first = blockIdx.x * static_cast<uint32_t>(kItems);
    if (tid == 0) {
        tc::mbar_init(&bars[0], 1);
        tc::mbar_init(&bars[1], 1);
        tc::mbar_init(&bars[2], 1);
        tc::mbar_init(&bars[3], 128);
        tc::mbar_init(&bars[4], 128);
        tc::mbar_init(&bars[5], 1);
        tc::mbar_init(&bars[6], 1);
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

    const int column = 32 * (warp & 3) + lane, item = kItems == 1 ? 0 : column / D, col = column % D;
    const bool there = first + item < heads;
    const int n = kItems == 1 || item == 0 ? seq[0] : seq[kItems - 1], h = kItems == 1 || item == 0 ? head[0] : head[kItems - 1];
    const int slot = a.slots ? a.slots[n] : n;
    const bool good = there && slot >= 0 && slot < a.num_slots;
    if (there && !good && col == 0 && group == 0) set_status(a.status, kStatusTree);
    constexpr int kUnits = KC / 8, kPer = D / 4;                        // units a thread, units a node
    uint2 kx[kUnits], qx[kUnits];
    auto token = [&](int it, int j) {                                   // row of place j of an item in the inputs
        return (static_cast<size_t>(it == 0 ? seq[0] : seq[kItems - 1]) * a.K + j) * a.H + (it == 0 ? head[0] : head[kItems - 1]);
    };
    auto fetch = [&](int chunk) {
#pragma unroll
        for (int z = 0; z < kUnits; ++z) {
            const int f = (tid + 256 * z) / kPer, c = (tid + 256 * z) % kPer * 4, it = f / KC, j = chunk * KC + f % KC;
            kx[z] = qx[z] = make_uint2(0u, 0u);
            if (j < a.K) {
                const size_t at = token(it, j) * D + c;
                kx[z] = *reinterpret_cast<const uint2*>(a.k + at);
                qx[z] = *reinterpret_cast<const uint2*>(a.q + at);
            }
        }
    };
    // 1. on their way, in this order, as what comes later waits for what came before: log alphas, keys and queries of the
    // first chunk (units of 4 channels), the state (a column a thread, half of the channels a group)
    for (int f = tid; f < (a.decay == 0 ? Sh::kNodes * kPer : a.decay == 1 ? Sh::kNodes : 0); f += 256) {
        const int e = a.decay == 0 ? f / kPer : f, j = e % KP;
        if (j >= a.K) continue;
        if (a.decay == 0) tree_copy16(tc::smem_u32(sm) + Sh::oLog + f * 16, a.la + token(e / KP, j) * D + f % kPer * 4);
        else tree_copy4(tc::smem_u32(sm) + Sh::oLog + f * 4, a.la + token(e / KP, j));
    }
    fetch(0);
    const size_t tok0 = static_cast<size_t>(n) * a.K * a.H + h;         // this item's place 0 in the inputs
    constexpr int kHalf = D / 2;
    float s[kHalf];
    {
        const float* S = a.pool + ((good ? static_cast<size_t>(slot) : 0) * a.H + h) * D * D + group * kHalf * D + col;
#pragma unroll
        for (int k = 0; k < kHalf; ++k) s[k] = __ldcs(S + k * D);
    }

    // 2. the trees
    if (warp < kItems) {
        uint64_t set[2] = {0, 0};
        if (first + warp < heads &&
            tree_sets(a.parents + static_cast<long long>(warp == 0 ? seq[0] : seq[kItems - 1]) * a.K, a.K, lane, set) && lane == 0)
            set_status(a.status, kStatusTree);
        if (lane < KP) s_set[warp * KP + lane] = set[0];
        if (lane + 32 < KP) s_set[warp * KP + lane + 32] = set[1];
    } else if (warp >= 4 && tid - 128 < Sh::kNodes) {
        const int e = tid - 128, j = e % KP;
        s_beta[e] = j < a.K ? bf16_bits_to_f32(a.beta[token(e / KP, j)]) : 0.f;
    }
    tree_copies_done();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *s_tmem, lane_tm = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    bool ok = true;
    // decays along the paths: a channel a thread, a node's its parent's times its alpha
    bool far = false;                                                   // one has left the range whose inverse is at hand
    if (group == 0) {
        float* dec = s_decay + item * KP * D + col;
        const float* la = reinterpret_cast<const float*>(sm + Sh::oLog);
#pragma unroll 1
        for (int j0 = 0; j0 < a.K; j0 += 8) {                           // (what does not depend on other nodes first)
            float al[8];
            int up[8];
            bool on[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const int e = item * KP + j0 + r;
                const Set set = static_cast<Set>(s_set[e]);
                const Set above = set & ~(kOne << (j0 + r));
                up[r] = above ? tree_top(above) : -1;
                on[r] = set != 0;
                al[r] = a.decay == 2 ? 1.f : expf(a.decay == 0 ? la[e * D + col] : la[e]);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                const float x = up[r] >= 0 ? al[r] * dec[up[r] * D] : al[r];
                dec[(j0 + r) * D] = x;
                far |= on[r] && (x < 0x1p-100f || (x > 0x1p100f && x < INFINITY));
            }
        }
    }
    // (a key over such a decay would overflow: those CTAs walk their paths)
    const bool walk = __syncthreads_or(far) != 0;

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
        const uint32_t rows = tree_desc(tc::smem_u32(sm) + Sh::oRows + slab * (Sh::kRows * 128u));
#pragma unroll
        for (uint32_t k = 0; k < 4; ++k) {
            tree_mma(d, ta + k * 8u, rows + k * 2u, id, start && k == 0 ? 0u : 1u);
            tree_mma(d, ta + k * 8u, rows + Sh::kTile / 16u + k * 2u, id, 1u);
            tree_mma(d, ta + 32u + k * 8u, rows + k * 2u, id, 1u);
        }
    };

    // the keys over their decays (64 rows from an item's first) times the item's rows: L and N, transposed
    constexpr uint32_t id_side = tc::idesc(64, 2 * KC, tc::kFmtTF32, false, false);
    auto side = [&](int it, int chunk) {                                // (one thread; into the columns of the chunk's rows)
        const uint32_t d = tm + Sh::kL + chunk * Sh::kRows + it * 2 * KC;
        const uint32_t sa = tree_desc(tc::smem_u32(sm) + Sh::oSide + it * KP * 128u);
        const uint32_t sb = tree_desc(tc::smem_u32(sm) + Sh::oRows + it * 2 * KC * 128u);
#pragma unroll
        for (uint32_t k = 0; k < Sh::kSlabs * 4u; ++k) {
            const uint32_t pa = sa + (k >> 2) * (Sh::kNodes * 8u) + (k & 3) * 2u, pb = sb + (k >> 2) * (Sh::kRows * 8u) + (k & 3) * 2u;
            tree_mma_ss(d, pa, pb, id_side, k > 0 ? 1u : 0u);
            tree_mma_ss(d, pa, pb + Sh::kTile / 16u, id_side, 1u);
            tree_mma_ss(d, pa + Sh::kSide / 16u, pb, id_side, 1u);
        }
    };
    auto split = [&](uint32_t off, uint32_t term, float4 x) {           // four channels of a row in their two terms
        const float4 lead = make_float4(tree_lead(x.x), tree_lead(x.y), tree_lead(x.z), tree_lead(x.w));
        *reinterpret_cast<float4*>(sm + off) = lead;
        *reinterpret_cast<float4*>(sm + off + term) = make_float4(x.x - lead.x, x.y - lead.y, x.z - lead.z, x.w - lead.w);
    };

    auto fetch_v = [&] {                                                // V, as the first operand's columns go: [place][column of the item]
        for (int f = tid; f < Sh::kNodes * D / 8; f += 256) {
            const int e = f / (D / 8), j = e % KP;
            if (j < a.K) tree_copy16(tc::smem_u32(sm) + Sh::oV + f * 16, a.v + token(e / KP, j) * D + f % (D / 8) * 8);
        }
    };

#pragma unroll 1
    for (int chunk = 0; chunk < Sh::kChunks; ++chunk) {
        // 3. the rows: keys and queries times their decays, keys over them
        if (chunk > 0) fetch(chunk);
#pragma unroll
        for (int z = 0; z < kUnits; ++z) {
            const int f = (tid + 256 * z) / kPer, c = (tid + 256 * z) % kPer * 4, it = f / KC, r = f % KC, e = it * KP + chunk * KC + r;
            const bool node = s_set[e] != 0;
            const float2 k0 = bf16x2_bits_to_f32(kx[z].x), k1 = bf16x2_bits_to_f32(kx[z].y);
            const float2 q0 = bf16x2_bits_to_f32(qx[z].x), q1 = bf16x2_bits_to_f32(qx[z].y);
            const float4 p = *reinterpret_cast<const float4*>(s_decay + e * D + c);
            const float4 none = make_float4(0.f, 0.f, 0.f, 0.f);
            const uint32_t row = it * 2 * KC + r;
            split(Sh::oRows + tc::sw128_off32(row, c, Sh::kRows), Sh::kTile,
                  node ? make_float4(p.x * k0.x, p.y * k0.y, p.z * k1.x, p.w * k1.y) : none);
            split(Sh::oRows + tc::sw128_off32(row + KC, c, Sh::kRows), Sh::kTile,
                  node ? make_float4(p.x * q0.x, p.y * q0.y, p.z * q1.x, p.w * q1.y) : none);
            split(Sh::oSide + tc::sw128_off32(e, c, Sh::kNodes), Sh::kSide,
                  node ? make_float4(k0.x * __frcp_rn(p.x), k0.y * __frcp_rn(p.y), k1.x * __frcp_rn(p.z), k1.y * __frcp_rn(p.w)) : none);
        }
        tc::fence_smem_to_async();
        if (chunk == 0) {
            if constexpr (Sh::kWhole) {
                put(group * (Sh::kSlabs / 2), Low{});
                if constexpr (kHalf > 32) put(group * (Sh::kSlabs / 2) + 1, High{});
            } else {
                put(group, Low{});
            }
        }
        __syncthreads();
        if (chunk + 1 == Sh::kChunks && !Sh::kVSide) fetch_v();         // (the decays are done with)
        // 4. the products, L's and N's first where they share accumulators
        auto sides = [&] {
            if (!walk && warp == 4) {                                   // (beside warp 0, which issues the others)
                tc::fence_after_sync();
                if (tc::elect_one()) {
                    for (int it = 0; it < kItems; ++it) side(it, chunk);
                    tc::mma_commit(&bars[5]);
                }
                __syncwarp();
            }
        };
        auto paths = [&] {                                              // L and N into shared memory
        if (!walk) {
            if (group == 0) {
                // row a of the product is lane a % 16 of warp a / 16
                if (16 * warp < KP) {
                    ok = tc::mbar_wait_bounded(&bars[5], chunk & 1, kWaitLimitNs) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
                    const int b = 16 * warp + lane;
#pragma unroll
                    for (int it = 0; it < kItems; ++it)
#pragma unroll
                        for (int c0 = 0; c0 < 2 * KC; c0 += 8) {
                            float x[8];
                            tree_tmem_ld8(lane_tm + Sh::kL + chunk * Sh::kRows + it * 2 * KC + c0, x);
                            float* to = (c0 < KC ? s_m : s_n) + (it * KP + chunk * KC + c0 % KC) * KP + b;
                            if (lane < 16 && b < KP) {
#pragma unroll
                                for (int r = 0; r < 8; ++r) to[r * KP] = x[r];
                            }
                        }
                    tc::fence_before_sync();
                }
                tc::named_sync(1, 128);
            }
        } else {
            // half a warp a node, up its path; lane l of the 16: channels 4 l .. + 3 of each 64
            const int hl = lane & 15;
#pragma unroll 1
            for (int f = 2 * warp + (lane >> 4); f < kItems * KC; f += 16) {
                const int it = f / KC, i = chunk * KC + f % KC, e = it * KP + i;
                Set left = static_cast<Set>(s_set[e]);
                float key[4 * G], query[4 * G], p[4 * G];
#pragma unroll
                for (int c = 0; c < 4 * G; ++c) {
                    const size_t at = token(it, left ? i : 0) * D + c / 4 * 64 + 4 * hl + c % 4;
                    key[c] = bf16_bits_to_f32(a.k[at]);
                    query[c] = bf16_bits_to_f32(a.q[at]);
                    p[c] = 1.f;
                }
                while (__any_sync(0xffffffffu, left != 0)) {
                    const bool on = left != 0;
                    const int b = on ? tree_top(left) : 0;
                    left &= ~(kOne << b);
                    const size_t tok = token(it, b);
                    float m = 0.f, w = 0.f;
#pragma unroll
                    for (int c = 0; c < 4 * G; ++c) {
                        const size_t at = tok * D + c / 4 * 64 + 4 * hl + c % 4;
                        const float kb = p[c] * bf16_bits_to_f32(a.k[at]);
                        m = fmaf(key[c], kb, m);
                        w = fmaf(query[c], kb, w);
                        p[c] *= a.decay == 2 ? 1.f : expf(a.la[a.decay == 0 ? at : tok]);
                    }
#pragma unroll
                    for (int off = 8; off > 0; off >>= 1) {
                        m += __shfl_xor_sync(0xffffffffu, m, off);
                        w += __shfl_xor_sync(0xffffffffu, w, off);
                    }
                    if (hl == 0 && on) {
                        s_m[(it * KP + i) * KP + b] = m;
                        s_n[(it * KP + i) * KP + b] = w;
                    }
                }
            }
        }
        };
        if (warp == 0) tc::fence_after_sync();
        sides();
        if constexpr (!Sh::kApart) {
            paths();
            if (warp == 0) tc::fence_after_sync();
        }
        if (warp == 0) {
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
        if constexpr (Sh::kApart) paths();
        if (chunk + 1 < Sh::kChunks) {                                  // the rows are written again
            ok = tc::mbar_wait_bounded(&bars[2], chunk & 1, kWaitLimitNs) && ok;
            ok = __all_sync(0xffffffffu, ok);
            __syncthreads();
        }
    }

    if constexpr (Sh::kVSide) {                                         // (the side is done with)
        if (!walk) {
            ok = tc::mbar_wait_bounded(&bars[5], (Sh::kChunks - 1) & 1, kWaitLimitNs) && ok;
            ok = __all_sync(0xffffffffu, ok);
        }
        fetch_v();
    }
    __syncthreads();
    // 5. W while the products run: a warp a row, lane b place b (and b + 32): w_c is final once the places above c are done.
    // Zeros where the path does not lead
    constexpr int kLanes = KP < 32 ? KP : 32, kP = KP > 32 ? 2 : 1;     // lanes a row, places a lane
#pragma unroll 1
    for (int e = warp * (32 / kLanes) + lane / kLanes; e < Sh::kNodes; e += 8 * (32 / kLanes)) {
        const int it = e / KP, i = e % KP, mine = lane % kLanes;
        const Set on = static_cast<Set>(s_set[e]);
        float w[kP];
        float* row = s_n + (it * KP + i) * KP;
        const float* L = s_m + it * KP * KP + mine;
        const float* beta = s_beta + it * KP;
#pragma unroll
        for (int z = 0; z < kP; ++z) w[z] = on >> (mine + 32 * z) & 1 ? row[mine + 32 * z] : 0.f;
        // (nothing is below a path's first node)
        for (Set left = on; __any_sync(0xffffffffu, (left & (left - 1)) != 0);) {
            int c4[4];
            Set below[4];
            float b4[4], m4[4][kP];
#pragma unroll
            for (int y = 0; y < 4; ++y) {                               // 4 places of the path, their loads together
                c4[y] = left ? tree_top(left) : 0;
                left &= ~(kOne << c4[y]);
                below[y] = left;
                b4[y] = beta[c4[y]];
#pragma unroll
                for (int z = 0; z < kP; ++z) m4[y][z] = L[c4[y] * KP + 32 * z];
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                float wc = __shfl_sync(0xffffffffu, w[0], c4[y] & 31, kLanes);
                if constexpr (kP == 2) {
                    const float hi = __shfl_sync(0xffffffffu, w[1], c4[y] & 31);
                    wc = c4[y] >= 32 ? hi : wc;
                }
                wc *= b4[y];
#pragma unroll
                for (int z = 0; z < kP; ++z)
                    if (below[y] >> (mine + 32 * z) & 1) w[z] = fmaf(-wc, m4[y][z], w[z]);
            }
        }
#pragma unroll
        for (int z = 0; z < kP; ++z) {
            const int b = mine + 32 * z;
            const float x = on >> b & 1 ? w[z] * beta[b] : 0.f, y = tree_lead(x);
            float* to = reinterpret_cast<float*>(sm + Sh::oW + z * (kItems * Sh::kWRows * 128) +
                                                 tc::sw128_off32(it * Sh::kWRows + i, mine, kItems * Sh::kWRows));
            to[0] = y;
            to[Sh::kW / 4] = x - y;
        }
    }
    tc::fence_smem_to_async();
    tree_copies_done();
    ok = tc::mbar_wait_bounded(&bars[2], (Sh::kChunks - 1) & 1, kWaitLimitNs) && ok;
    ok = __all_sync(0xffffffffu, ok);
    __syncthreads();
    tc::fence_after_sync();

    // 6. V - P, a column a thread and every other 8 places a group, into S_0^T's place
    const uint64_t* set = s_set + item * KP;
    const uint16_t* v = reinterpret_cast<const uint16_t*>(sm + Sh::oV) + item * KP * D + col;
    auto rows_at = [&](int i, int query) {                              // TMEM columns of places i .. i + 7
        return lane_tm + Sh::kD + (i / KC) * Sh::kRows + item * 2 * KC + query * KC + i % KC;
    };
    Set none = 0;                                                       // places where it is no number (0 goes in: 0 * NaN is none)
#pragma unroll 2
    for (int i0 = 8 * group; i0 < KP; i0 += 16) {
        float x[8], y[8];
        tree_tmem_ld8(rows_at(i0, 0), x);
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            float d = set[i0 + r] != 0 ? bf16_bits_to_f32(v[(i0 + r) * D]) - x[r] : 0.f;
            if (!(fabsf(d) < INFINITY)) {
                none |= kOne << (i0 + r);
                d = 0.f;
            }
            x[r] = tree_lead(d);
            y[r] = d - x[r];
        }
        tree_tmem_st8(lane_tm + i0, x);
        tree_tmem_st8(lane_tm + KP + i0, y);
    }
    tc::tmem_wait_st();
    tc::fence_before_sync();
    const bool some = __syncthreads_or(none != 0) != 0;
    if (warp == 0) {
        tc::fence_after_sync();
        if (tc::elect_one()) {
            // Q += W (V - P), per item and chunk (N at least 16: what follows 8 places' columns is not read again)
            constexpr int kN = KC < 16 ? 16 : KC;
            constexpr uint32_t id_w = tc::idesc(128, kN, tc::kFmtTF32, false, false);
            for (int chunk = 0; chunk < Sh::kChunks; ++chunk)
                for (int it = 0; it < kItems; ++it) {
                    const uint32_t d = tm + Sh::kD + chunk * Sh::kRows + it * 2 * KC + KC;
                    const uint32_t sw = tree_desc(tc::smem_u32(sm) + Sh::oW + (it * Sh::kWRows + chunk * KC) * 128u);
#pragma unroll
                    for (uint32_t k = 0; k < KP / 8; ++k) {
                        const uint32_t at = sw + (k >> 2) * (kItems * Sh::kWRows * 8u) + (k & 3) * 2u;
                        tree_mma(d, tm + k * 8u, at, id_w, 1u);
                        tree_mma(d, tm + k * 8u, at + Sh::kW / 16u, id_w, 1u);
                        tree_mma(d, tm + KP + k * 8u, at, id_w, 1u);
                    }
                }
            tc::mma_commit(&bars[6]);
        }
        __syncwarp();
    }
    if (some) {                                                         // the other group's places of this column too
        Set* s_none = reinterpret_cast<Set*>(sm + Sh::oRows);           // (the rows are done with)
        s_none[group * 128 + column] = none;
        __syncthreads();
        none |= s_none[(1 - group) * 128 + column];
    }
    ok = tc::mbar_wait_bounded(&bars[6], 0, kWaitLimitNs) && ok;
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after_sync();

    // 7. the outputs, every other 8 places a group
    const size_t step = static_cast<size_t>(a.H) * D;
    const size_t to = tok0 * D + col;
#pragma unroll 1
    for (int i0 = 8 * group; i0 < a.K; i0 += 16) {
        float o[8];
        tree_tmem_ld8(rows_at(i0, 1), o);
        if (!good || !ok) continue;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            if (i0 + r >= a.K) break;
            const Set on = static_cast<Set>(set[i0 + r]);
            float x = on ? o[r] : 0.f;
            if (on & none) x = __int_as_float(0x7fffffff);
            if (a.out_f32) reinterpret_cast<float*>(a.out)[to + (i0 + r) * step] = x;
            else reinterpret_cast<uint16_t*>(a.out)[to + (i0 + r) * step] = f32_to_bf16_bits(x);
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
