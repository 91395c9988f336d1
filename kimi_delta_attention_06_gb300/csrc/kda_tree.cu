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
// where W is K x K numbers a head, found by substitution: by lanes of a warp a row, along the node's path or over all places.
//
// The product P^T [128 columns x 2 K] = S_0^T [128 x D] rows^T [D x 2 K] runs on the tensor cores with S_0^T in TMEM (its
// lanes are the state's columns, a thread's a column), as three tf32 products of the operands' leading 11 bits and what is left of them: 22 bits, an fp32
// product but for 2^-21.  The tensor cores round sums towards zero: the two small products have an accumulator of their own, or
// go first, and W (V - P) is not added to Q there (errors of 64 x 8 heads of 64 x 64, 48 nodes, against 64 bits:
// 1.4e-6 -> 2.5e-7).  So do L and N, as products of the decayed rows with the keys over their decays (nodes on whose paths
// a decay leaves 2^-100 .. 2^100 walk them instead: a node's arithmetic follows from its own path alone), and W (V - P), with
// V - P in TMEM in S_0^T's place (a NaN or an infinity in it enters as 0, and is put back for the nodes whose paths hold it:
// 0 * NaN is none).
//
// Measured in a graph: 256 sequences x 32 heads of 128 x 128, trees of 16 nodes: 185 us for 0.70 GB that cannot be done without
// (103 us of HBM); 64 x 8 of 64 x 64, 48 nodes: 46 us; one sequence, 32 heads, 8 nodes: 6.4 us.  Bound by a turn's chain (decays,
// rows, product, V - P, product, outputs; 13 thousand clocks at 16 nodes) with two CTAs an SM to fill it, one from 17
// nodes on, where TMEM and shared memory hold no more.  Decays outside the range from
// the fourth node on, or everywhere: 262 and 292 us at 16 nodes, 125 and 116 at 48.
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
    int num_slots, out_f32, N, K, H, decay, sms;
    int* status;
};

// A turn of a CTA is 128 columns: one head's state of 128 x 128, or two of 64 x 64 (items).  Nodes go through the product
// in chunks of at most 32, so that their rows fit beside the rest.
template <int D, int KP>
struct TreeShape {
    static constexpr int kItems = 128 / D, kNodes = kItems * KP;
    static constexpr int KC = KP < 32 ? KP : KP == 64 && D == 64 ? 16 : 32, kChunks = KP / KC;
    static constexpr int kSlabs = D / 32;                               // 32 channels: 128 bytes of a row of fp32, a quarter or half of S_0
    // The rows' two terms lie one after the other per item, so that one product serves both, up to 32 places; beyond,
    // a tile a term.  kRows: rows of a slab; kItem: rows (and accumulators) of an item; kRest: from a row to its second term
    static constexpr bool kStack = KP <= 32;
    static constexpr int kItem = (kStack ? 4 : 2) * KC, kRows = kItems * kItem;
    static constexpr uint32_t kTile = kRows * 128u * kSlabs, kRest = kStack ? 2 * KC * 128u : kTile, kTiles = kStack ? kTile : 2 * kTile;
    // the keys over their decays: 8 rows and their second terms in turn, or a tile a term
    static constexpr int kSideItem = (kStack ? 2 : 1) * KP, kSideRows = kItems * kSideItem;
    static constexpr uint32_t kSide = kSideRows * 128u * kSlabs, kSides = kStack ? kSide : 2 * kSide;
    // CTAs an SM, slabs of S_0 that are on their way in shared memory (each group its own), and in TMEM (all of them
    // where it is used twice)
    static constexpr int kCtas = KP <= 16 ? 2 : 1, kRing = KP == 32 ? 4 : 2;
    static constexpr bool kWhole = kChunks > 1;
    static constexpr int kBufs = kWhole ? kSlabs : 2;
    static constexpr uint32_t kD = kBufs * 64u;                         // TMEM column of the accumulators
    // L and N have accumulators of their own where there is room, else those of the product, before it
    static constexpr uint32_t kProduct = kD + kChunks * kRows, kMost = 512u / kCtas;
    static constexpr bool kApart = kProduct + kChunks * kRows <= kMost;
    static constexpr uint32_t kL = kApart ? kProduct : kD, kUsed = kL + kChunks * kRows;
    static constexpr uint32_t kCols = kUsed <= 128u ? 128u : kUsed <= 256u ? 256u : 512u;
    static_assert(kCols <= kMost && 2 * KP <= kD, "TMEM");
    static_assert(KC >= 16 || kApart, "16 columns of W (V - P) in L's place");
    static_assert(kStack || kWhole, "the small products first: the state is there twice");
    static_assert(kApart || kBufs == kSlabs, "the first products do not wait for what follows the last slab");
    // bytes of shared memory.  (The side's products read 64 rows from each item's first: what follows it, beyond KP)
    static constexpr uint32_t oSide = 0, oRows = oSide + kSides, oState = oRows + kTiles;
    static constexpr uint32_t oM = oState + kRing * 16384u, kMN = kItems * KP * KP * 4u, oN = oM + kMN, oV = oN + kMN;
    // W [place][32 places a slab] in two terms, in the side's place
    static constexpr int kWRows = KP < 16 ? 16 : KP, kWSlabs = KP > 32 ? 2 : 1;
    static constexpr uint32_t kW = kItems * kWRows * 128u * kWSlabs, oW = oSide;
    static_assert(2 * kW <= kSides, "W in the side's place");
    // a thread's share of the rows: CH channels of one place, or of two; lanes of a warp go over places
    static constexpr int kLanes = KP < 32 ? KP : 32, kPlaces = KP / kLanes, kG = 32 / kLanes, CH = 16 / kG;
    static constexpr uint32_t kBit = KP > 32 ? 8u : 4u;                 // bytes of a set
    static constexpr uint32_t oNone = oRows;                            // of 256 threads: places that are no number
    static constexpr int kRounds = KP == 8 ? 3 : KP == 16 ? 4 : KP == 32 ? 5 : 6;      // of the decays' products, doubling their reach
    static constexpr uint32_t oSet = oV + kNodes * D * 2u, oBeta = oSet + 2 * kNodes * kBit;
    static constexpr uint32_t oFar = oBeta + 2 * kNodes * 2u, oDesc = oFar + 2 * kRounds * kNodes, oBar = oDesc + 2 * kNodes * kBit;
    static constexpr uint32_t kBytes = oBar + 288u;
    // W by whole rows of L (else along the paths), where a row has so many lanes, and a lane so many quads of places
    static constexpr bool kDense = KP > 16;
    static constexpr int kWLanes = KP / 4 < 256 / kNodes ? KP / 4 : 256 / kNodes, kQuads = KP / 4 / kWLanes;
    static_assert(kBytes <= (kCtas == 1 ? 232448u : 115712u), "shared memory");
    static_assert(oState >= oSide + kSides + 8192u, "the side's last products stay within");
    static_assert(256u * kBit <= kTiles && D % CH == 0, "none; channels");
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
__device__ __forceinline__ void tree_copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// x rounded to its leading 11 bits (to the nearest: what is left is then as often negative, and so are the products that are
// left out); x less these is exact.  (A NaN that turns into a number here is still one in x less it.)
__device__ __forceinline__ float tree_lead(float x) { return __uint_as_float((__float_as_uint(x) + 0x1000u) & 0xffffe000u); }
constexpr float kTreeMost = 0x1.ffep127f;        // from here on it would be infinite

template <bool WIDE> struct TreeBits { using type = uint32_t; };
template <> struct TreeBits<true> { using type = uint64_t; };
__device__ __forceinline__ int tree_top(uint32_t x) { return 31 - __clz(x); }
__device__ __forceinline__ int tree_top(uint64_t x) { return 63 - __clzll(x); }
__device__ __forceinline__ float tree_rcp(float x) {                    // to within a step, of a normal number
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

constexpr int kTreeThreads = 320;                // 8 warps that work, one that issues products, one that brings the state
constexpr uint32_t kTreeAll = 1;                 // named barrier of the 8 warps

// 8 warps in two groups of 4, each a whole set of TMEM's lanes (a thread a column of the state).
//   1  the state's first slabs into TMEM      2  decays along the paths, rows into shared memory      3  the other slabs, as they come
//   4  L and N out of TMEM                    5  W                                  6  V - P into TMEM            7  outputs
// The inputs of the next turn are on their way from 3 on; the state's next slabs, and the rest of it into L2, always.
template <int D, int KP>
__global__ void __launch_bounds__(kTreeThreads, TreeShape<D, KP>::kCtas)
kda_tree_kernel(const TreeArgs a)
{
    using Sh = TreeShape<D, KP>;
    using Set = typename TreeBits<(KP > 32)>::type;                     // a path: bit b is place b
    constexpr int KC = Sh::KC, kItems = Sh::kItems, G = D / 64, kSlabs = Sh::kSlabs, kRing = Sh::kRing, kBufs = Sh::kBufs;
    constexpr int kChunks = Sh::kChunks;
    constexpr Set kOne = 1;
    extern __shared__ __align__(1024) uint8_t sm[];
    float* s_m = reinterpret_cast<float*>(sm + Sh::oM);
    float* s_n = reinterpret_cast<float*>(sm + Sh::oN);
    Set* s_sets = reinterpret_cast<Set*>(sm + Sh::oSet);                // [2][place]: of this turn and the next
    uint16_t* s_betas = reinterpret_cast<uint16_t*>(sm + Sh::oBeta);    // [2][place]
    int8_t* s_fars = reinterpret_cast<int8_t*>(sm + Sh::oFar);          // [2][round][place]: the ancestor 2^round up, -1 without one
    Set* s_descs = reinterpret_cast<Set*>(sm + Sh::oDesc);              // [2][place]: the places whose paths it is on
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Sh::oBar);
    uint64_t *b_full = bars, *b_empty = bars + 4;                       // a slab is in shared memory; has been read
    uint64_t *b_put = bars + 8, *b_free = bars + 12;                    // is in TMEM; its products are done
    uint64_t *b_rows = bars + 16, *b_side = bars + 17, *b_read = bars + 18;    // the rows are written; L and N are done; have been read
    uint64_t *b_prod = bars + 19, *b_e = bars + 20, *b_w = bars + 21;   // the product is done; V - P is in TMEM; W (V - P) is done
    // everything is; the trees of even and odd turns are there; such a turn is done.  (Of each barrier, the side that completes
    // a phase waits for the side that waits on it before it can complete the next)
    uint64_t *b_last = bars + 22, *b_tree = bars + 14, *b_done = bars + 24;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 23);
    Set* s_bad = reinterpret_cast<Set*>(bars + 26);                     // [2][item]: places whose row of L holds no number, ..
    Set* s_far = s_bad + 2 * kItems;                                    // .. whose decays leave the products' range

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kRing; ++i) {
            tc::mbar_init(&b_full[i], 1);
            tc::mbar_init(&b_empty[i], 128);
        }
        for (int i = 0; i < kBufs; ++i) {
            tc::mbar_init(&b_put[i], 128);
            if (!Sh::kWhole) tc::mbar_init(&b_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&b_tree[i], 32);
            tc::mbar_init(&b_done[i], 1);
        }
        tc::mbar_init(b_rows, 256);
        tc::mbar_init(b_side, 1);
        tc::mbar_init(b_read, 256);
        tc::mbar_init(b_prod, 1);
        tc::mbar_init(b_e, 256);
        tc::mbar_init(b_w, 1);
        tc::mbar_init(b_last, 1);
        tc::mbar_fence_init();
        for (int i = 0; i < 2 * kItems; ++i) s_bad[i] = s_far[i] = 0;
    }
    if (warp == 8) tc::tmem_alloc(s_tmem, Sh::kCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *s_tmem, sm0 = tc::smem_u32(sm);
    const uint32_t heads = static_cast<uint32_t>(a.N) * a.H, stride = gridDim.x * static_cast<uint32_t>(kItems);
    // what a turn works on: the items' sequence and head (past the last: the last again)
    struct Turn {
        uint32_t first;
        int seq[kItems], head[kItems];
        __device__ __forceinline__ Turn(uint32_t f, uint32_t heads, int H) : first(f) {
#pragma unroll
            for (int i = 0; i < kItems; ++i) {
                const uint32_t x = min(first + i, heads - 1);
                seq[i] = static_cast<int>(x / static_cast<uint32_t>(H));
                head[i] = static_cast<int>(x - static_cast<uint32_t>(seq[i]) * H);
            }
        }
        __device__ __forceinline__ int n(int it) const { return kItems == 1 || it == 0 ? seq[0] : seq[kItems - 1]; }
        __device__ __forceinline__ int h(int it) const { return kItems == 1 || it == 0 ? head[0] : head[kItems - 1]; }
        // row of place j of an item in the inputs
        __device__ __forceinline__ size_t token(int it, int j, int K, int H) const { return (static_cast<size_t>(n(it)) * K + j) * H + h(it); }
    };
    auto slot_of = [&](const Turn& w, int it) {                         // -1: none to read
        const int slot = a.slots ? a.slots[w.n(it)] : w.n(it);
        return w.first + it < heads && slot >= 0 && slot < a.num_slots ? slot : -1;
    };
    bool ok = true;
    const uint32_t begin = blockIdx.x * static_cast<uint32_t>(kItems);
    const int chunks = kChunks == 1 ? 1 : (a.K + KC - 1) / KC;          // (of the places that there are)

    if (warp == 9) {
        // ---- the trees; the state: slabs of 32 channels through the ring; all inputs a turn ahead into L2 ----
        uint32_t c = 0, turn = 0;                                       // slabs and turns so far
        for (uint32_t first = begin; first < heads && ok; first += stride, ++turn) {
            const Turn w(first, heads, a.H);
            const float* S[kItems];
#pragma unroll
            for (int it = 0; it < kItems; ++it) {
                const int slot = slot_of(w, it);
                S[it] = a.pool + ((slot >= 0 ? static_cast<size_t>(slot) : 0) * a.H + w.h(it)) * D * D;
            }
            if (first + stride < heads) {
                const Turn z(first + stride, heads, a.H);
#pragma unroll
                for (int it = 0; it < kItems; ++it) {
                    if (const int slot = slot_of(z, it); slot >= 0 && lane == 0)
                        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                                     :: "l"(a.pool + (static_cast<size_t>(slot) * a.H + z.h(it)) * D * D), "r"(D * D * 4) : "memory");
                    for (int j = lane; j < a.K; j += 32) {
                        const size_t at = z.token(it, j, a.K, a.H) * D;
#pragma unroll
                        for (int x = 0; x < D * 2; x += 128) {
                            asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const uint8_t*>(a.k + at) + x));
                            asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const uint8_t*>(a.q + at) + x));
                            asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const uint8_t*>(a.v + at) + x));
                        }
                        if (a.decay == 0)
#pragma unroll
                            for (int x = 0; x < D * 4; x += 128)
                                asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const uint8_t*>(a.la + at) + x));
                    }
                }
            }
            // the trees, where the last turn's but one have been read
            const uint32_t odd = turn & 1;
            if (turn >= 2) ok = tc::mbar_wait_bounded(&b_done[odd], (turn / 2 - 1) & 1, kWaitLimitNs);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            for (int i = lane; i < Sh::kNodes; i += 32) {
                const int j = i % KP;
                s_betas[odd * Sh::kNodes + i] = j < a.K ? a.beta[w.token(i / KP, j, a.K, a.H)] : 0;
            }
#pragma unroll 1
            for (int it = 0; it < kItems; ++it) {
                uint64_t set[2] = {0, 0};
                if (first + it < heads && tree_sets(a.parents + static_cast<long long>(w.n(it)) * a.K, a.K, lane, set) && lane == 0)
                    set_status(a.status, kStatusTree);
                Set desc[2] = {0, 0};
#pragma unroll 4
                for (int c = 0; c < (Sh::kDense ? KP : 0); ++c) {
                    const Set path = static_cast<Set>(__shfl_sync(0xffffffffu, KP > 32 && c >= 32 ? set[1] : set[0], c & 31));
                    desc[0] |= (path >> lane & 1) << c;
                    if constexpr (KP > 32) desc[1] |= (path >> (lane + 32) & 1) << c;
                }
                int far[2];                                             // the parent at first
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                    const int j = lane + 32 * z;
                    const uint64_t above = set[z] & ~(1ull << j);
                    far[z] = above ? tree_top(above) : -1;
                    if (j >= KP) continue;
                    s_sets[(odd * kItems + it) * KP + j] = static_cast<Set>(set[z]);
                    if (Sh::kDense) s_descs[(odd * kItems + it) * KP + j] = desc[z];
                }
#pragma unroll 1
                for (int r = 0; r < Sh::kRounds; ++r) {
                    int8_t* to = s_fars + ((odd * Sh::kRounds + r) * kItems + it) * KP;
                    if (lane < KP) to[lane] = static_cast<int8_t>(far[0]);
                    if (lane + 32 < KP) to[lane + 32] = static_cast<int8_t>(far[1]);
                    int next[2];
#pragma unroll
                    for (int z = 0; z < 2; ++z) {
                        const int n0 = __shfl_sync(0xffffffffu, far[0], far[z] & 31), n1 = __shfl_sync(0xffffffffu, far[1], far[z] & 31);
                        next[z] = far[z] >= 32 ? n1 : n0;
                    }
#pragma unroll
                    for (int z = 0; z < 2; ++z) far[z] = far[z] >= 0 ? next[z] : -1;
                }
            }
            tc::mbar_arrive(&b_tree[odd]);
            for (int q = 0; q < kSlabs && ok; ++q, ++c) {
                const uint32_t at = c % kRing;
                if (c >= kRing) ok = tc::mbar_wait_bounded(&b_empty[at], (c / kRing - 1) & 1, kWaitLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) {
                    tc::mbar_arrive_expect_tx(&b_full[at], 16384u);
#pragma unroll
                    for (int it = 0; it < kItems; ++it)
                        tc::bulk_load_g2s(sm0 + Sh::oState + at * 16384u + it * (16384u / kItems), S[it] + q * 32 * D, 16384u / kItems, &b_full[at]);
                }
                __syncwarp();
            }
        }
        // (copies in flight land before the shared memory is given back)
        if (!ok)
            for (uint32_t i = c > kRing ? c - kRing : 0; i < c; ++i) tc::mbar_wait_bounded(&b_full[i % kRing], i / kRing & 1, kWaitLimitNs);
        __syncwarp();
    } else if (warp == 8) {
        // ---- the products ----
        if (tc::elect_one()) {
            constexpr uint32_t id = tc::idesc(128, Sh::kRows, tc::kFmtTF32, false, false);
            constexpr uint32_t id_rest = tc::idesc(128, 2 * KC, tc::kFmtTF32, false, false);
            constexpr uint32_t id_side = tc::idesc(64, Sh::kItem, tc::kFmtTF32, false, false);
            // (N at least 16: what follows 8 places' columns is not read again)
            constexpr int kN = KC < 16 ? 16 : KC;
            constexpr uint32_t id_w = tc::idesc(128, kN, tc::kFmtTF32, false, false);
            uint32_t turn = 0, run = 0, puts = 0;
            for (uint32_t first = begin; first < heads && ok; first += stride, ++turn) {
                for (int chunk = 0; chunk < chunks && ok; ++chunk, ++run) {
                    ok = tc::mbar_wait_bounded(b_rows, run & 1, kWaitLimitNs);
                    if (!ok) break;
                    tc::fence_after_sync();
                    auto side = [&] {
                        // the keys over their decays (64 rows from an item's first) times the item's rows: L and N, transposed
#pragma unroll 1
                        for (int it = 0; it < kItems; ++it) {
                            const uint32_t d = tm + Sh::kL + chunk * Sh::kRows + it * Sh::kItem;
                            const uint32_t sa = tree_desc(sm0 + Sh::oSide + it * Sh::kSideItem * 128u);
                            const uint32_t sb = tree_desc(sm0 + Sh::oRows + it * Sh::kItem * 128u);
#pragma unroll
                            for (uint32_t x = 0; x < (Sh::kStack ? 1u : 2u) * kSlabs * 4u; ++x) {
                                const uint32_t k = x % (kSlabs * 4u);
                                const uint32_t pa = sa + (k >> 2) * (Sh::kSideRows * 8u) + (k & 3) * 2u, pb = sb + (k >> 2) * (Sh::kRows * 8u) + (k & 3) * 2u;
                                if (Sh::kStack || x >= kSlabs * 4u) {
                                    tree_mma_ss(d, pa, pb, id_side, x > 0 ? 1u : 0u);
                                } else {
                                    tree_mma_ss(d, pa, pb + Sh::kRest / 16u, id_side, x > 0 ? 1u : 0u);
                                    tree_mma_ss(d, pa + Sh::kSide / 16u, pb, id_side, 1u);
                                }
                            }
                        }
                        tc::mma_commit(b_side);
                    };
                    if (!Sh::kApart) {
                        side();
                        ok = tc::mbar_wait_bounded(b_read, run & 1, kWaitLimitNs);
                        if (!ok) break;
                        tc::fence_after_sync();
                    }
                    const uint32_t d = tm + Sh::kD + chunk * Sh::kRows;
                    for (int q = 0; q < kSlabs; ++q) {
                        // (beside the slabs that wait for the first ones' place)
                        if (Sh::kApart && q == kBufs % kSlabs) side();
                        const int b = q % kBufs;
                        if (chunk == 0) {
                            ok = tc::mbar_wait_bounded(&b_put[b], puts / kBufs & 1, kWaitLimitNs);
                            if (!ok) break;
                            tc::fence_after_sync();
                            ++puts;
                        }
                        const uint32_t ta = tm + b * 64, rows = tree_desc(sm0 + Sh::oRows + q * (Sh::kRows * 128u));
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k) {
                            // (stacked: both terms of the rows, their accumulators side by side, the small ones' second)
                            if constexpr (Sh::kStack) {
                                tree_mma(d, ta + k * 8u, rows + k * 2u, id, q == 0 && k == 0 ? 0u : 1u);
#pragma unroll
                                for (uint32_t it = 0; it < kItems; ++it)
                                    tree_mma(d + it * Sh::kItem + 2 * KC, ta + 32u + k * 8u, rows + it * Sh::kItem * 8u + k * 2u, id_rest, 1u);
                            } else {
                                tree_mma(d, ta + k * 8u, rows + Sh::kRest / 16u + k * 2u, id, q == 0 && k == 0 ? 0u : 1u);
                                tree_mma(d, ta + 32u + k * 8u, rows + k * 2u, id, 1u);
                            }
                        }
                        if (!Sh::kWhole) tc::mma_commit(&b_free[b]);
                    }
                    if (!Sh::kStack && ok)
#pragma unroll
                        for (uint32_t x = 0; x < kSlabs * 4u; ++x)
                            tree_mma(d, tm + (x >> 2) * 64 + (x & 3) * 8u,
                                     tree_desc(sm0 + Sh::oRows + (x >> 2) * (Sh::kRows * 128u)) + (x & 3) * 2u, id, 1u);
                    if (ok) tc::mma_commit(b_prod);
                }
                if (!ok) break;
                ok = tc::mbar_wait_bounded(b_e, turn & 1, kWaitLimitNs);
                if (!ok) break;
                tc::fence_after_sync();
                // W (V - P), per item and chunk, where L was
                for (int chunk = 0; chunk < chunks; ++chunk)
#pragma unroll 1
                    for (int it = 0; it < kItems; ++it) {
                        const uint32_t d = tm + Sh::kL + chunk * Sh::kRows + it * Sh::kItem;
                        const uint32_t sw = tree_desc(sm0 + Sh::oW + (it * Sh::kWRows + chunk * KC) * 128u);
#pragma unroll
                        for (uint32_t x = 0; x < KP / 4; ++x) {
                            const uint32_t k = x % (KP / 8), at = sw + (k >> 2) * (kItems * Sh::kWRows * 8u) + (k & 3) * 2u;
                            if (x >= KP / 8) {
                                tree_mma(d, tm + k * 8u, at, id_w, 1u);
                            } else {
                                tree_mma(d, tm + k * 8u, at + Sh::kW / 16u, id_w, x > 0 ? 1u : 0u);
                                tree_mma(d, tm + KP + k * 8u, at, id_w, 1u);
                            }
                        }
                    }
                tc::mma_commit(b_w);
            }
            // nothing of this CTA's is left running when it returns its TMEM
            tc::mma_commit(b_last);
            if (!tc::mbar_wait_bounded(b_last, 0, kWaitLimitNs)) ok = false;
        }
        __syncwarp();
    } else {
        const int group = warp >> 2, column = 32 * (warp & 3) + lane, item = kItems == 1 ? 0 : column / D, col = column % D;
        const uint32_t lane_tm = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        // this thread's share of the rows
        constexpr int CH = Sh::CH, kPlaces = Sh::kPlaces, kWords = CH / 2;
        const int place = lane % Sh::kLanes, block = (warp * Sh::kG + lane / Sh::kLanes) * CH, part = block / D, chan = block % D;
        // the inputs on their way: log alphas, keys and queries
        float la[kPlaces][CH];
        uint32_t kx[kPlaces][kWords], qx[kPlaces][kWords];
        auto fetch = [&](const Turn& w) {
#pragma unroll
            for (int z = 0; z < kPlaces; ++z) {
                const int j = min(place + 32 * z, a.K - 1);
                const size_t tok = w.token(part, j, a.K, a.H), at = tok * D + chan;
                if (a.decay == 0) {
#pragma unroll
                    for (int c = 0; c < CH; c += 4) {
                        const float4 x = *reinterpret_cast<const float4*>(a.la + at + c);
                        la[z][c] = x.x; la[z][c + 1] = x.y; la[z][c + 2] = x.z; la[z][c + 3] = x.w;
                    }
                } else {
                    const float x = a.decay == 1 ? a.la[tok] : 0.f;
#pragma unroll
                    for (int c = 0; c < CH; ++c) la[z][c] = x;
                }
                auto words = [&](const uint16_t* from, uint32_t (&to)[kWords]) {
                    if constexpr (kWords == 2) {
                        const uint2 x = *reinterpret_cast<const uint2*>(from);
                        to[0] = x.x; to[1] = x.y;
                    } else {
#pragma unroll
                        for (int c = 0; c < kWords; c += 4) {
                            const uint4 x = *reinterpret_cast<const uint4*>(from + 2 * c);
                            to[c] = x.x; to[c + 1] = x.y; to[c + 2] = x.z; to[c + 3] = x.w;
                        }
                    }
                };
                words(a.k + at, kx[z]);
                words(a.q + at, qx[z]);
            }
        };
        auto fetch_v = [&](const Turn& w) {                             // [place][column of the item]
            for (int f = tid; f < Sh::kNodes * D / 8; f += 256) {
                const int e = f / (D / 8), j = e % KP;
                if (j < a.K) tree_copy16(sm0 + Sh::oV + f * 16, a.v + w.token(e / KP, j, a.K, a.H) * D + f % (D / 8) * 8);
            }
        };
        auto split = [&](uint32_t off, uint32_t term, float4 x) {       // four channels of a row in their two terms
            const float4 lead = make_float4(tree_lead(x.x), tree_lead(x.y), tree_lead(x.z), tree_lead(x.w));
            *reinterpret_cast<float4*>(sm + off) = lead;
            *reinterpret_cast<float4*>(sm + off + term) = make_float4(x.x - lead.x, x.y - lead.y, x.z - lead.z, x.w - lead.w);
        };
        Turn next(begin, heads, a.H);
        fetch(next);
        uint32_t turn = 0, run = 0, slab = 0;
#pragma unroll 1
        for (; next.first < heads; ++turn) {
            const Turn now = next;
            const uint32_t odd = turn & 1;                              // of what completes once a turn
            const Set* s_set = s_sets + odd * Sh::kNodes;
            const uint16_t* s_beta = s_betas + odd * Sh::kNodes;
            const int slot = slot_of(now, item);
            if (slot < 0 && now.first + item < heads && col == 0 && group == 0) set_status(a.status, kStatusTree);
            fetch_v(now);
            // 1, 3. slab q of the state into TMEM (a group each in turn)
            auto put = [&](int q) {
                const uint32_t c = slab + q, b = q % kBufs;
                ok = tc::mbar_wait_bounded(&b_full[c % kRing], c / kRing & 1, kWaitLimitNs) && ok;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                const float* S = reinterpret_cast<const float*>(sm + Sh::oState + c % kRing * 16384u) + item * 32 * D + col;
                uint32_t lead[32], rest[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = S[i * D], y = tree_lead(x);
                    lead[i] = __float_as_uint(y);
                    rest[i] = __float_as_uint(x - y);
                }
                tc::fence_smem_to_async();                              // (the copy that follows the arrival must not overtake a load)
                tc::mbar_arrive(&b_empty[c % kRing]);
                // (the first of a turn follow on its last turn's end)
                if (q >= kBufs) {
                    ok = tc::mbar_wait_bounded(&b_free[b], (turn * (kSlabs / kBufs) + q / kBufs - 1) & 1, kWaitLimitNs);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) return;
                    tc::fence_after_sync();
                }
                tc::tmem_st32x(lane_tm + b * 64, lead);
                tc::tmem_st32x(lane_tm + b * 64 + 32, rest);
                tc::tmem_wait_st();
                tc::fence_before_sync();
                tc::mbar_arrive(&b_put[b]);
            };
#pragma unroll 1
            for (int q = group; q < kBufs && ok; q += 2) put(q);
            // 2. decays along the paths: a node's product reaches 1, 2, 4 .. nodes up, a lane a node
            ok = tc::mbar_wait_bounded(&b_tree[odd], turn / 2 & 1, kWaitLimitNs) && ok;
            ok = __all_sync(0xffffffffu, ok);
            float p[kPlaces][CH];
#pragma unroll
            for (int z = 0; z < kPlaces; ++z)
#pragma unroll
                for (int c = 0; c < CH; ++c) p[z][c] = expf(la[z][c]);
            const int8_t* fars = s_fars + (odd * Sh::kRounds * kItems + part) * KP + place;
#pragma unroll 1
            for (int r = 0; r < Sh::kRounds; ++r) {
                int up[kPlaces];
                bool more = false;
#pragma unroll
                for (int z = 0; z < kPlaces; ++z) {
                    up[z] = fars[r * kItems * KP + 32 * z];
                    more |= up[z] >= 0;
                }
                if (!__any_sync(0xffffffffu, more)) break;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    float y[kPlaces];
#pragma unroll
                    for (int z = 0; z < kPlaces; ++z) {
                        y[z] = __shfl_sync(0xffffffffu, p[0][c], up[z], Sh::kLanes);
                        if constexpr (kPlaces == 2) {
                            const float hi = __shfl_sync(0xffffffffu, p[1][c], up[z]);
                            y[z] = up[z] >= 32 ? hi : y[z];
                        }
                    }
#pragma unroll
                    for (int z = 0; z < kPlaces; ++z) p[z][c] *= up[z] >= 0 ? y[z] : 1.f;
                }
            }
            auto add = [&](Set* to, Set places) {
                if constexpr (KP > 32) atomicOr(reinterpret_cast<unsigned long long*>(to), static_cast<unsigned long long>(places));
                else atomicOr(to, places);
            };
            // (a key over a decay outside this range would overflow: nodes with such a one on their paths walk them, and they alone.
            // NaN and infinities do not count)
            Set mine[kPlaces];
#pragma unroll
            for (int z = 0; z < kPlaces; ++z) {
                mine[z] = s_set[part * KP + place + 32 * z];
                float least = INFINITY, most = 0.f;
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    least = fminf(least, p[z][c]);
                    most = fmaxf(most, p[z][c] < INFINITY ? p[z][c] : 0.f);
                }
                if ((least < 0x1p-100f || most > 0x1p100f) && mine[z] != 0) add(s_far + odd * kItems + part, kOne << (place + 32 * z));
            }
            // the next turn's inputs, into what is done with: before the other slabs, or behind them where registers are short
            // (16 nodes: 196 us before them, 189 behind; 32: 445, 475)
            auto ahead = [&](int chunk) {
                if (chunk + 1 < chunks) return;
                next = Turn(now.first + stride, heads, a.H);
                if (next.first < heads) fetch(next);
            };

#pragma unroll 1
            for (int chunk = 0; chunk < chunks; ++chunk, ++run) {
                // the rows: keys and queries times their decays, keys over them
#pragma unroll
                for (int z = 0; z < kPlaces; ++z) {
                    const int i = place + 32 * z;
                    if (kChunks > 1 && i / KC != chunk) continue;
                    const uint32_t row = part * Sh::kItem + i % KC;
                    const uint32_t beside = part * Sh::kSideItem + (Sh::kStack ? i / 8 * 16 + i % 8 : i);
#pragma unroll
                    for (int c = 0; c < CH; c += 4) {
                        float k[4], q[4], d[4];
#pragma unroll
                        for (int w = 0; w < 2; ++w) {
                            const float2 x = bf16x2_bits_to_f32(mine[z] ? kx[z][c / 2 + w] : 0u), y = bf16x2_bits_to_f32(mine[z] ? qx[z][c / 2 + w] : 0u);
                            k[2 * w] = x.x; k[2 * w + 1] = x.y;
                            q[2 * w] = y.x; q[2 * w + 1] = y.y;
                        }
#pragma unroll
                        for (int w = 0; w < 4; ++w) d[w] = mine[z] ? p[z][c + w] : 1.f;
                        split(Sh::oRows + tc::sw128_off32(row, chan + c, Sh::kRows), Sh::kRest,
                              make_float4(d[0] * k[0], d[1] * k[1], d[2] * k[2], d[3] * k[3]));
                        split(Sh::oRows + tc::sw128_off32(row + KC, chan + c, Sh::kRows), Sh::kRest,
                              make_float4(d[0] * q[0], d[1] * q[1], d[2] * q[2], d[3] * q[3]));
                        split(Sh::oSide + tc::sw128_off32(beside, chan + c, Sh::kSideRows), Sh::kStack ? 1024u : Sh::kSide,
                              make_float4(k[0] * tree_rcp(d[0]), k[1] * tree_rcp(d[1]), k[2] * tree_rcp(d[2]), k[3] * tree_rcp(d[3])));
                    }
                }
                tc::fence_smem_to_async();
                tc::mbar_arrive(b_rows);
                if (Sh::kCtas == 1) ahead(chunk);
                // 3. the other slabs
                if (chunk == 0) {
#pragma unroll 1
                    for (int q = kBufs + group; q < kSlabs && ok; q += 2) put(q);
                    slab += kSlabs;
                }
                if (Sh::kCtas > 1) ahead(chunk);
                tc::named_sync(kTreeAll, 256);                          // (of all threads: what is far)
                if (tid == 0)
                    for (int it = 0; it < kItems; ++it) s_bad[(1 - odd) * kItems + it] = s_far[(1 - odd) * kItems + it] = 0;
                bool walk = false;
#pragma unroll
                for (int it = 0; it < kItems; ++it) walk |= s_far[odd * kItems + it] != 0;
                // 4. L and N of the chunk's nodes.  Dense: beta L, and zeros where the path does not lead (L: nor to the node itself);
                // what is no number in L enters as 0, and the node is marked: its own and its descendants' outputs are none
                auto walks = [&](int it, int i) { return (s_set[it * KP + i] & s_far[odd * kItems + it]) != 0; };
                // row x of the product is lane x % 16 of warp x / 16
                constexpr int kOwn = Sh::kStack ? 8 : 16;           // places a warp (stacked: lanes 8 .. 15 their second terms)
                if (const int b = kOwn * (warp & 3) + lane; b - lane < KP && (Sh::kDense || group == 0)) {     // dense: one group L, the other N
                    ok = tc::mbar_wait_bounded(b_side, run & 1, kWaitLimitNs) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                    tc::fence_after_sync();
#pragma unroll 1
                    for (int it = 0; it < kItems; ++it) {
                        // (nothing of it is wanted where all nodes walk)
                        if (Sh::kDense && walk && !__any_sync(0xffffffffu, lane < KC && s_set[it * KP + chunk * KC + lane] != 0 && !walks(it, chunk * KC + lane))) continue;
                        const Set below = Sh::kDense && b < KP ? s_descs[(odd * kItems + it) * KP + b] : 0;
                        float* to = (group == 0 ? s_m : s_n) + (it * KP + chunk * KC) * KP + b;
                        static_assert(Sh::kDense || kChunks == 1);
                        float any = 0.f;                            // NaN where one is none
#pragma unroll
                        for (int c0 = 0; c0 < (Sh::kDense ? 1 : 2) * KC; c0 += 8) {
                            float x[8];
                            const uint32_t from = lane_tm + Sh::kL + chunk * Sh::kRows + it * Sh::kItem + group * KC + c0;
                            tree_tmem_ld8(from, x);
                            if constexpr (Sh::kStack) {
                                float y[8];
                                tree_tmem_ld8(from + 2 * KC, y);
#pragma unroll
                                for (int r = 0; r < 8; ++r) x[r] += __shfl_xor_sync(0xffffffffu, x[r], 8) + y[r];
                            }
                            const int first = chunk * KC + c0;
                            if (!Sh::kDense) {
                                if (c0 == KC) to = s_n + (it * KP - KC) * KP + b;
                            } else if (group == 0) {
                                const uint4 beta = *reinterpret_cast<const uint4*>(s_beta + it * KP + first);
                                const uint32_t beta2[4] = {beta.x, beta.y, beta.z, beta.w};
#pragma unroll
                                for (int r = 0; r < 8; r += 2) {
                                    const float2 f = bf16x2_bits_to_f32(beta2[r / 2]);
                                    x[r] = (below >> (first + r) & 1) && b != first + r ? x[r] * f.x : 0.f;
                                    x[r + 1] = (below >> (first + r + 1) & 1) && b != first + r + 1 ? x[r + 1] * f.y : 0.f;
                                    any = fmaf(x[r + 1], 0.f, fmaf(x[r], 0.f, any));
                                }
                            } else {
#pragma unroll
                                for (int r = 0; r < 8; ++r) x[r] = below >> (first + r) & 1 ? x[r] : 0.f;
                            }
                            if (lane < kOwn && b < KP) {
#pragma unroll
                                for (int r = 0; r < 8; ++r) to[(c0 + r) * KP] = x[r];
                            }
                        }
                        if (any != 0.f && lane < kOwn && b < KP) {
#pragma unroll 1
                            for (int r = 0; r < KC; ++r)
                                if (!walks(it, chunk * KC + r) && !(fabsf(to[r * KP]) < INFINITY)) {
                                    to[r * KP] = 0.f;
                                    add(s_bad + odd * kItems + it, kOne << (chunk * KC + r));
                                }
                        }
                    }
                    tc::fence_before_sync();
                }
                if (walk) {
                    // those of the nodes below a far decay again: half a warp a node, up its path; lane l of the 16: channels
                    // 4 l .. + 3 of each 64
                    const int hl = lane & 15;
                    tc::named_sync(kTreeAll, 256);
#pragma unroll 1
                    for (int f = 2 * warp + (lane >> 4); f < kItems * KC; f += 16) {
                        const int it = f / KC, i = chunk * KC + f % KC, e = it * KP + i;
                        Set left = walks(it, i) ? s_set[e] : 0;
                        if (Sh::kDense) {
                            if (left || s_set[e] == 0)
#pragma unroll
                                for (int b = hl; b < KP; b += 16) s_m[e * KP + b] = s_n[e * KP + b] = 0.f;
                            __syncwarp();
                        }
                        if (Sh::kDense && !__any_sync(0xffffffffu, left != 0)) continue;
                        float key[4 * G], query[4 * G], p[4 * G];
#pragma unroll
                        for (int c = 0; c < 4 * G; ++c) {
                            const size_t at = now.token(it, left ? i : 0, a.K, a.H) * D + c / 4 * 64 + 4 * hl + c % 4;
                            key[c] = bf16_bits_to_f32(a.k[at]);
                            query[c] = bf16_bits_to_f32(a.q[at]);
                            p[c] = 1.f;
                        }
                        while (__any_sync(0xffffffffu, left != 0)) {
                            const bool on = left != 0;
                            const int b = on ? tree_top(left) : 0;
                            left &= ~(kOne << b);
                            const size_t tok = now.token(it, b, a.K, a.H);
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
                                if (Sh::kDense) {
                                    m *= b < i ? bf16_bits_to_f32(s_beta[e]) : 0.f;
                                    if (!(fabsf(m) < INFINITY) && b < i) add(s_bad + odd * kItems + it, kOne << i);
                                    m = fabsf(m) < INFINITY ? m : 0.f;
                                }
                                s_m[e * KP + b] = m;
                                s_n[e * KP + b] = w;
                            }
                        }
                    }
                }
                if (!Sh::kApart) tc::mbar_arrive(b_read);
                if (chunk + 1 < chunks) {                               // the rows are written again
                    ok = tc::mbar_wait_bounded(b_prod, run & 1, kWaitLimitNs) && ok;
                    ok = __all_sync(0xffffffffu, ok);
                }
            }
            tc::named_sync(kTreeAll, 256);
            // 5. W while the products run.  Dense: kWLanes lanes a row, each every kWLanes-th quad of its places: from the last quad of
            // places up, whose four numbers are solved for by every lane, then taken out of the places above them (zeros where a
            // path does not lead).  Else 32 / kLanes rows a warp along their paths, lane b place b: w_c is final once the places
            // above c are done.  (256 x 32 heads, dense to paths: 8 nodes 177 to 162 us, 16: 231 to 214, 32: 445 to 487, 64: 1240
            // to 1530; the dense one is given what two CTAs an SM have no registers for.)
            if constexpr (Sh::kDense) {
                constexpr int kL = Sh::kWLanes, kQ = Sh::kQuads;
                const int e = min(tid / kL, Sh::kNodes - 1), it = e / KP, i = e % KP, s = tid % kL;
                if (32 * warp < Sh::kNodes * kL) {
                    const float* L = s_m + it * KP * KP;
                    float w[kQ][4];
#pragma unroll
                    for (int j = 0; j < kQ; ++j) {
                        const float4 n = *reinterpret_cast<const float4*>(s_n + e * KP + (j * kL + s) * 4);
                        w[j][0] = n.x; w[j][1] = n.y; w[j][2] = n.z; w[j][3] = n.w;
                    }
#pragma unroll
                    for (int b = KP / 4 - 1; b >= 0; --b) {
                        if (4 * b >= a.K) continue;                     // (no rows of L there)
                        float x[4];
#pragma unroll
                        for (int r = 0; r < 4; ++r) x[r] = __shfl_sync(0xffffffffu, w[b / kL][r], b % kL, kL);
                        const float* at = L + 4 * b * KP;
                        const float4 l1 = *reinterpret_cast<const float4*>(at + KP + 4 * b), l2 = *reinterpret_cast<const float4*>(at + 2 * KP + 4 * b),
                                     l3 = *reinterpret_cast<const float4*>(at + 3 * KP + 4 * b);
                        x[2] = fmaf(-x[3], l3.z, x[2]);
                        x[1] = fmaf(-x[2], l2.y, fmaf(-x[3], l3.y, x[1]));
                        x[0] = fmaf(-x[1], l1.x, fmaf(-x[2], l2.x, fmaf(-x[3], l3.x, x[0])));
#pragma unroll
                        for (int j = 0; j <= b / kL; ++j)
#pragma unroll
                            for (int r = 3; r >= 0; --r) {
                                const float4 l = *reinterpret_cast<const float4*>(at + r * KP + (j * kL + s) * 4);
                                w[j][0] = fmaf(-x[r], l.x, w[j][0]);
                                w[j][1] = fmaf(-x[r], l.y, w[j][1]);
                                w[j][2] = fmaf(-x[r], l.z, w[j][2]);
                                w[j][3] = fmaf(-x[r], l.w, w[j][3]);
                            }
                    }
                    const Set on = s_set[e];
                    if (tid / kL < Sh::kNodes)
#pragma unroll
                        for (int j = 0; j < kQ; ++j) {
                            const int b = (j * kL + s) * 4;
                            const uint2 beta = *reinterpret_cast<const uint2*>(s_beta + it * KP + b);
                            const float2 lo = bf16x2_bits_to_f32(beta.x), hi = bf16x2_bits_to_f32(beta.y);
                            split(Sh::oW + tc::sw128_off32(it * Sh::kWRows + i, b, kItems * Sh::kWRows), Sh::kW,
                                  make_float4(on >> b & 1 ? w[j][0] * lo.x : 0.f, on >> (b + 1) & 1 ? w[j][1] * lo.y : 0.f,
                                              on >> (b + 2) & 1 ? w[j][2] * hi.x : 0.f, on >> (b + 3) & 1 ? w[j][3] * hi.y : 0.f));
                        }
                }
            } else {
                constexpr int kLanes = Sh::kLanes;
#pragma unroll 1
                for (int e = warp * (32 / kLanes) + lane / kLanes; e < Sh::kNodes; e += 8 * (32 / kLanes)) {
                    const int it = e / KP, i = e % KP, mine = lane % kLanes;
                    const Set on = s_set[e];
                    const float* L = s_m + it * KP * KP + mine;
                    const uint16_t* beta = s_beta + it * KP;
                    float w = on >> mine & 1 ? s_n[(it * KP + i) * KP + mine] : 0.f;
                    // (nothing is below a path's first node)
                    for (Set left = on; __any_sync(0xffffffffu, (left & (left - 1)) != 0);) {
                        int c4[4];
                        Set below[4];
                        float b4[4], m4[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {                   // 4 places of the path, their loads together
                            c4[y] = left ? tree_top(left) : 0;
                            left &= ~(kOne << c4[y]);
                            below[y] = left;
                            b4[y] = bf16_bits_to_f32(beta[c4[y]]);
                            m4[y] = L[c4[y] * KP];
                        }
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float wc = __shfl_sync(0xffffffffu, w, c4[y] & 31, kLanes) * b4[y];
                            if (below[y] >> mine & 1) w = fmaf(-wc, m4[y], w);
                        }
                    }
                    const float x = on >> mine & 1 ? w * bf16_bits_to_f32(beta[mine]) : 0.f, y = tree_lead(x);
                    float* to = reinterpret_cast<float*>(sm + Sh::oW + tc::sw128_off32(it * Sh::kWRows + i, mine, kItems * Sh::kWRows));
                    to[0] = y;
                    to[Sh::kW / 4] = x - y;
                }
            }
            tc::fence_smem_to_async();
            tree_copies_done();
            ok = tc::mbar_wait_bounded(b_prod, (run - 1) & 1, kWaitLimitNs) && ok;
            ok = __all_sync(0xffffffffu, ok);
            tc::named_sync(kTreeAll, 256);
            tc::fence_after_sync();
            // 6. V - P, a column a thread and every other 8 places a group, into S_0^T's place
            const Set* set = s_set + item * KP;
            const uint16_t* v = reinterpret_cast<const uint16_t*>(sm + Sh::oV) + item * KP * D + col;
            auto rows_at = [&](int i, int query, float (&x)[8]) {       // places i .. i + 7 of P, or of Q
                const uint32_t from = lane_tm + Sh::kD + (i / KC) * Sh::kRows + item * Sh::kItem + query * KC + i % KC;
                tree_tmem_ld8(from, x);
                if constexpr (Sh::kStack) {
                    float y[8];
                    tree_tmem_ld8(from + 2 * KC, y);
#pragma unroll
                    for (int r = 0; r < 8; ++r) x[r] += y[r];
                }
            };
            Set none = Sh::kDense ? s_bad[odd * kItems + item] : 0;     // places where it is no number (0 goes in: 0 * NaN is none)
#pragma unroll 2
            for (int i0 = 8 * group; i0 < KP; i0 += 16) {
                float x[8], y[8];
                rows_at(i0, 0, x);
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    float d = set[i0 + r] != 0 ? bf16_bits_to_f32(v[(i0 + r) * D]) - x[r] : 0.f;
                    if (!(fabsf(d) < kTreeMost)) {
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
            tc::mbar_arrive(b_e);
            if (!tc::named_sync_and(kTreeAll, 256, none == 0)) {        // the other group's places of this column too
                Set* s_none = reinterpret_cast<Set*>(sm + Sh::oNone);   // (the rows are done with)
                s_none[group * 128 + column] = none;
                tc::named_sync(kTreeAll, 256);
                none |= s_none[(1 - group) * 128 + column];
                tc::named_sync(kTreeAll, 256);
            }
            ok = tc::mbar_wait_bounded(b_w, odd, kWaitLimitNs) && ok;
            ok = __all_sync(0xffffffffu, ok);
            tc::fence_after_sync();

            // 7. the outputs, every other 8 places a group
            const size_t step = static_cast<size_t>(a.H) * D;
            const size_t to = now.token(item, 0, a.K, a.H) * D + col;
#pragma unroll 1
            for (int i0 = 8 * group; i0 < a.K; i0 += 16) {
                float o[8], x8[8];
                rows_at(i0, 1, o);
                tree_tmem_ld8(lane_tm + Sh::kL + (i0 / KC) * Sh::kRows + item * Sh::kItem + i0 % KC, x8);
                if (slot < 0 || !ok) continue;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    if (i0 + r >= a.K) break;
                    const Set on = set[i0 + r];
                    float x = on ? o[r] + x8[r] : 0.f;
                    if (on & none) x = __int_as_float(0x7fffffff);
                    if (a.out_f32) reinterpret_cast<float*>(a.out)[to + (i0 + r) * step] = x;
                    else reinterpret_cast<uint16_t*>(a.out)[to + (i0 + r) * step] = f32_to_bf16_bits(x);
                }
            }
            tc::fence_before_sync();
            // (a wait that ran out: nothing more is begun)
            if (!tc::named_sync_and(kTreeAll, 256, ok)) { ok = false; break; }
            tc::fence_after_sync();
            if (tid == 0) tc::mbar_arrive(&b_done[odd]);
        }
        tree_copies_done();
    }
    if (!ok) set_status(a.status, kStatusTimeout);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 8) tc::tmem_dealloc(tm, Sh::kCols);
}

namespace {
template <int D, int KP>
int launch_tree_shape(const TreeArgs& a, cudaStream_t stream) {
    using Sh = TreeShape<D, KP>;
    static bool attr_done[kMaxDevicesAttr] = {};
    if (!raise_smem_limit(reinterpret_cast<const void*>(kda_tree_kernel<D, KP>), Sh::kBytes, attr_done)) return -3;
    const long long heads = static_cast<long long>(a.N) * a.H;
    const long long turns = (heads + Sh::kItems - 1) / Sh::kItems, at_once = static_cast<long long>(a.sms) * Sh::kCtas;
    kda_tree_kernel<D, KP><<<static_cast<unsigned>(turns < at_once ? turns : at_once), kTreeThreads, Sh::kBytes, stream>>>(a);
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
    static int sms[kMaxDevicesAttr] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return -3;
    if (!sms[dev] && cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -3;
    const TreeArgs a{q, k, v, la, beta, pool, slots, parents, out, num_slots, out_f32, N, K, H, decay, sms[dev], status};
    return D == 128 ? launch_tree_dim<128>(a, stream) : launch_tree_dim<64>(a, stream);
}

}  // namespace kda
