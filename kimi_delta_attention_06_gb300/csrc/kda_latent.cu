// kda_latent.cu -- absorbed latent attention over the paged cache.
//
// Row (n, j, h) of the output: x_t = scale * (q[:512] . c_t + q[512:] . r_t) over the tokens the
// query sees, out = sum_t softmax(x)_t c_t, with one pass over the tokens: the running maximum m,
// the sum l of exp(x - m) and the weighted sum of c are rescaled when m grows.
//
// All K * H rows of a sequence read the same cached vectors, so both products run on the tensor
// cores with the cached tokens on the M side: per tile of 64 tokens
//     S^T [64 tokens x R rows]      = C [64 x 576] Q^T                 (M = 64, N = R)
//     O^T [512 channels x R rows]  += C[:, :512]^T P^T [64 x R]        (4 blocks of M = 128, N = R)
// with R = 16, 32 or 64 rows a CTA, so few rows do not leave the tensor cores' M side empty.  One
// shared-memory tile of C (128-byte swizzle) serves both: K-major for S, MN-major for O.
//
// An e4m3 cache enters both products as it is, without being expanded:
//   - q / 2^k (2^k a row: the largest magnitude in (224, 448]) is the sum of two e4m3 values, exactly
//     where |q| is above 1/900 of the row's largest (8 bits of bf16 in 4 + 4), within 2^-17 of it
//     below.  The position part is bf16 and has its own accumulator, as the scale s of a token
//     belongs to its latent only: x = scale * (2^k s S_c + S_r).
//   - s moves from the latents to the weights: O = sum (p s) codes.  p s is the sum of three e5m2
//     values (3 bits each: a relative 2^-9, less than a rounding to bf16), scaled so that the
//     largest lies in 2^10 .. 2^15, which leaves 26 binades or more below it.
// Measured, 32 heads: 64 sequences (970k tokens), bf16, K = 1, 185 us, 6.0 TB/s (HBM); e4m3 133 us
// (4.8 TB/s; 16 heads 112 us; the softmax warps' chain through each tile); 16 sequences (214k tokens), K = 4,
// e4m3 100 us, bf16 93 us (64 rows a CTA: over e4m3 58 us are tiles, of 2750 clocks each, 2364 of them products
// whose operands shared memory feeds at 128 bytes a clock, 28 us segments' starts and ends, 13 us the join); one
// sequence of 145408, bf16, 42 us, 6 of them the join.
// Expanding the tile to bf16 instead (exact too) took 4800 clocks a tile of 64 rows: loads into
// registers hold too little in flight beside 227 KB of shared memory, and the tile is written and
// read once more.
#include <cuda.h>
#include "latent.cuh"
#include "tc.cuh"
#include "tree.cuh"

namespace kda {

struct LatentCache {
    const uint8_t* rows;
    const int32_t* table;        // [N, max_pages]
    int num_pages, page_size, max_pages;
};

// ---- work split ------------------------------------------------------------------------------
// The sequences' 64-token tiles, one after another, are cut into G equal runs, one per CTA
// (x the row tiles, which run side by side over the same tokens so that the second reader finds
// them in L2).  A CTA's run covers parts of one or several sequences (segments).  A segment that
// is a whole sequence is finished by its CTA; the others leave partial (m, l, O) in scratch, at
// most two per CTA (its first and its last), which the combine kernel joins.  A segment costs
// its start (Q, the first copies) and its end (O) besides its tiles, so each sequence counts
// `lead` tiles more before its first one; a run's share of them is no work.
//
// Trees have places without a node, mostly their last ones, and with them whole row tiles to leave out.  So a tree's row
// tiles are sequences of their own (all sequences' first row tiles, all their second ones, .. `each` times), of length 0
// where no row of theirs is a node, and a run is a CTA's alone.  In this order the readers of a sequence's tokens still
// run side by side where most trees are full (16 sequences of 341k tokens in all, trees of 4 to 8 nodes x 32 heads, e4m3:
// 233 -> 204 us; a sequence's row tiles one after another: 203, and 64 x 8000 tokens, 4 nodes x 64 heads, bf16: 395 us
// for 352).
constexpr int kTile = 64;                       // tokens per tile
constexpr int kMinTiles = 2;                    // shortest run of tiles worth a CTA of its own

struct LatWork {
    const int32_t* seq_lens;
    int N, G;                                   // G: most runs
    int lead;
    int least;                                  // shortest length of a sequence that is not empty (a tree's K nodes)
    long long max_len;
    int each;                                   // row tiles that are sequences of their own (1: none are), ..
    int most;                                   // (kMaxNeed)
    const uint8_t* need;                        // .. and how many of them a sequence needs (nullptr: all), ..
    const int32_t* lens;                        // .. beside its length (0: of an empty one)
};
// Up to so many sequences are looked at for it (shared memory; of more, all row tiles are worked through).
template <bool E4M3> constexpr int kMaxNeed = E4M3 ? 512 : 128;

// (What only trees have is a constant for chains: with it looked up, one sequence of 145408 x 32 heads took 43.4 us for 42.2,
// 64 of 1k to 64k 189.2 for 187.2, 3 of up to 200 x 4 heads 8.5 for 8.1.)
template <bool TREE> __device__ __forceinline__ int lat_each(const LatWork& w) { return TREE ? w.each : 1; }
template <bool TREE>
__device__ __forceinline__ int lat_seq(const LatWork& w, int n) {
    const int len = w.seq_lens[n];
    return len < (TREE ? w.least : 0) || len > w.max_len ? 0 : len;
}
template <bool TREE>
__device__ __forceinline__ int lat_len(const LatWork& w, int n) {
    if (lat_each<TREE>(w) <= 1) return lat_seq<TREE>(w, n);
    const int seqs = w.N / w.each, tile = n / seqs, s = n - tile * seqs;
    return !w.need ? lat_seq<TREE>(w, s) : tile < w.need[s] ? w.lens[s] : 0;
}
// Row tiles that a tree needs, as one warp finds it: R rows each, H of a node, up to its last place with a node.
__device__ __forceinline__ int lat_need(const int32_t* parents, int K, int H, int R, int lane) {
    const unsigned lo = __ballot_sync(0xffffffffu, lane < K && __ldg(parents + lane) >= -1);
    const unsigned hi = K > 32 ? __ballot_sync(0xffffffffu, lane + 32 < K && __ldg(parents + lane + 32) >= -1) : 0u;
    const int last = hi ? 64 - __clz(hi) : 32 - __clz(lo);
    return (last * H + R - 1) / R;
}
__device__ __forceinline__ int lat_tiles(int len) { return (len + kTile - 1) / kTile; }
__device__ __forceinline__ int lat_count(const LatWork& w, int len) { return len > 0 ? lat_tiles(len) + w.lead : 0; }   // with the lead
// Runs in use for T tiles, and the bounds of run c.
__device__ __forceinline__ long long lat_runs(long long T, int G) {
    const long long r = (T + kMinTiles - 1) / kMinTiles;
    return r < G ? r : G;
}
__device__ __forceinline__ long long run_div(long long x, long long y) {      // x / y of non-negative numbers
    return x >> 32 ? x / y : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
}
__device__ __forceinline__ long long run_begin(long long T, long long runs, long long c) { return run_div(c * T, runs); }
// The run that holds tile t: the largest c with c T / runs (rounded down) <= t.
__device__ __forceinline__ long long run_of(long long T, long long runs, long long t) { return run_div((t + 1) * runs - 1, T); }

// Walks the segments of one run; every warp keeps its own copy (init is warp-collective).
template <bool TREE>
struct SegWalk {
    long long pos, end, base;                   // next tile, end of the run, first (counted) tile of sequence n
    int n, len, count;                          // count: its tiles and its lead
    int t0, t1;                                 // current segment: tiles [t0, t1) of sequence n
    long long total;                            // tiles of all sequences, counted with their leads
    bool first;

    __device__ __forceinline__ void init(const LatWork& w, int c) {
        const int lane = threadIdx.x & 31;
        const int len0 = lane < w.N ? lat_len<TREE>(w, lane) : 0;     // the first 32 stay in registers
        long long T = lat_count(w, len0);
        for (int i = lane + 32; i < w.N; i += 32) T += lat_count(w, lat_len<TREE>(w, i));
        if (w.N <= 32 && __reduce_max_sync(0xffffffffu, static_cast<unsigned>(T)) < (1u << 26)) {
            T = __reduce_add_sync(0xffffffffu, static_cast<unsigned>(T));
        } else {
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) T += __shfl_xor_sync(0xffffffffu, T, off);
        }
        pos = end = base = 0;
        total = T;
        n = len = count = t0 = t1 = 0;
        first = true;
        if (T == 0) return;
        const long long runs = lat_runs(T, w.G);
        if (c >= runs) return;
        pos = run_begin(T, runs, c);
        end = run_begin(T, runs, c + 1);
        for (int i0 = 0; i0 < w.N; i0 += 32) {
            const int lane_len = i0 == 0 ? len0 : i0 + lane < w.N ? lat_len<TREE>(w, i0 + lane) : 0;
            const int mine = lat_count(w, lane_len);
            int incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + incl > pos);
            if (hit) {
                const int at = __ffs(hit) - 1;
                n = i0 + at;
                base += __shfl_sync(0xffffffffu, incl - mine, at);
                len = __shfl_sync(0xffffffffu, lane_len, at);
                count = lat_count(w, len);
                return;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    // The next segment; false when the run is done.
    __device__ bool next(const LatWork& w) {
        while (pos < end) {
            while (pos >= base + count) {
                base += count;
                ++n;
                len = lat_len<TREE>(w, n);
                count = lat_count(w, len);
            }
            const long long stop = end - base < count ? end - base : count;
            t0 = max(0, static_cast<int>(pos - base) - w.lead);
            t1 = max(0, static_cast<int>(stop) - w.lead);
            pos = base + stop;
            if (t1 > t0) return true;           // (else the run ends within the lead)
        }
        return false;
    }
    __device__ bool whole() const { return t0 == 0 && t1 == lat_tiles(len); }
};

// ---- the tensor-core kernel --------------------------------------------------------------------
// q [rows, 576] in boxes of 64 columns; the cache in boxes of whole rows, as slabs of 128 bytes (64 bf16
// values; 128 codes, or the position key); the scales of an e4m3 cache in boxes of 16 bytes.  (A box a
// slab instead is 36 copies a tile with pages of 16 tokens: 64 sequences 191 -> 208 us, e4m3 134 -> 185,
// K = 4 94 -> 145.)
struct LatMaps { CUtensorMap q, c, s; };

// The sequence that a run begins and leaves to the next one (n; -1: none), the counted tiles before it and of all.
struct LatCut { long long before, T; int n; };

struct LatArgs {
    LatWork w;
    LatentCache ch;
    const uint16_t* q;
    const int32_t* parents;                      // of a tree's nodes [N, K], else nullptr
    int K, H, rows, RT;                          // rows = K * H, RT row tiles
    int box;                                     // cache rows per TMA box (divides the page and the tile)
    float scale_log2;
    uint16_t* out;
    float* lse;
    float *part_o, *part_ml;                     // partials: [run][row tile][2][R][512], [..][R][2]
    LatCut* cuts;                                // [G]: of each run; nullptr where sequences are few
    int* status;
};

// Row tiles of sequence n that are sequences of their own and not left out (a warp together).
template <int R, bool TREE>
__device__ __forceinline__ int lat_needed(const LatArgs& a, int n, int lane) {
    return lat_each<TREE>(a.w) <= 1 || a.w.N / a.w.each > a.w.most ? a.w.each
                                                        : lat_need(a.parents + static_cast<long long>(n) * a.K, a.K, a.H, R, lane);
}
// Of few sequences: the counted tiles of all, and of those before row tile `tile` of sequence n; its own length and row tiles.
struct LatCount { long long T, before; int len, need; };
template <int R, bool TREE>
__device__ __forceinline__ LatCount lat_counted(const LatArgs& a, int n, int tile, int lane) {
    const int each = lat_each<TREE>(a.w), seqs = a.w.N / each;
    LatCount c{0, 0, 0, 0};
    for (int i0 = 0; i0 < seqs; i0 += 32) {
        const int i = i0 + lane, v = i < seqs ? lat_seq<TREE>(a.w, i) : 0;
        int mine = each;
        if (each > 1)
#pragma unroll 4
            for (int k = i0; k < min(i0 + 32, seqs); ++k) {
                const int need = lat_needed<R, TREE>(a, k, lane);
                mine = i == k ? need : mine;
            }
        const long long count = lat_count(a.w, v);
        c.T += mine * count;
        c.before += (min(mine, tile) + (i < n && mine > tile ? 1 : 0)) * count;
        if (n >= i0 && n < i0 + 32) {
            c.len = __shfl_sync(0xffffffffu, v, n - i0);
            c.need = __shfl_sync(0xffffffffu, mine, n - i0);
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        c.T += __shfl_xor_sync(0xffffffffu, c.T, off);
        c.before += __shfl_xor_sync(0xffffffffu, c.before, off);
    }
    return c;
}

template <int R, bool E4M3>
struct LatShape {
    // softmax, rescale, epilogue: groups of 4 warps, each RW rows of a tile (64 rows, one group of 4 warps to two: 16 trees of
    // 4 to 8 nodes x 32 heads over 341k tokens, e4m3, 204 -> 184 us; 3 of 12 nodes x 4 heads over 200 tokens at most, bf16, 17.6 -> 14.4;
    // 16 chains of 8 x 32 over the same, e4m3, 229 -> 223)
    static constexpr int kGroups = R == 64 ? 2 : 1, RW = R / kGroups;
    static constexpr int kSoft = 128 * kGroups;
    static constexpr int kMmaWarp = 4 * kGroups, kTmaWarp = kMmaWarp + 1;
    static constexpr int kThreads = kSoft + 64;
    // as many as fit: a stage is taken for a copy's latency (about 3000 clocks) and both products
    static constexpr int kStages = E4M3 ? (R <= 32 ? 4 : 3) : 2;
    static constexpr uint32_t kSlabQ = R * 128u;
    // bf16: 9 slabs of 64 values; e4m3: 4 slabs of 128 codes, the position key's, 64 scales of 16 bytes
    // (a slab: 128 bytes of a row; a tile: 8 groups of 8 rows, each of kSlabs slabs of 8 x 128 bytes, which is
    // what one copy of whole rows lays down)
    static constexpr uint32_t kSlabs = E4M3 ? 5u : 9u, kSlabC = 1024u, kGroup = kSlabs * kSlabC, kRows = 8u * kGroup;
    static constexpr uint32_t kStage = kRows + (E4M3 ? 1024u : 0u);
    // Q: 9 slabs of 64 bf16; e4m3: 2 terms x 4 slabs of 128 codes, then the position part's
    // e4m3: the three terms of P lie side by side along N where TMEM holds three accumulators for them
    // (R <= 32: the codes are then read once for all three; 64 sequences, R = 32: 170 -> 149 us), else
    // in tiles of their own that share one accumulator
    static constexpr bool kSide = E4M3 && R <= 32;
    static constexpr uint32_t kO = kSide ? 3u * R : R;                                // TMEM columns of a block of O
    static constexpr uint32_t kP = E4M3 && !kSide ? 3u : 1u;                          // tiles of P
    static constexpr uint32_t oQ = 0, oC = 9u * kSlabQ, oP = oC + kStages * kStage, oBar = oP + kP * kTile * 128u;
    static constexpr uint32_t kBytes = oBar + 112u + 7u * R * 4u;
    static constexpr uint32_t kS = E4M3 ? 2u * R : R;                                 // TMEM columns of one S buffer
    static constexpr uint32_t kUsed = 4u * kO + 2u * kS;
    static constexpr uint32_t kTmemCols = kUsed <= 128u ? 128u : kUsed <= 256u ? 256u : 512u;
    static_assert(kUsed <= 512u, "TMEM");
};
static_assert(LatShape<64, false>::kBytes + 64 * 8 + 5 * kMaxNeed<false> <= 232448 && LatShape<64, true>::kBytes + 64 * 8 + 5 * kMaxNeed<true> <= 232448,
              "227 KB of shared memory");

// A row's weights are exp2(x - m).  m follows the row's maximum M lazily: bf16, m <= M <= m + 8 (the
// sums have the range for it); e4m3, m + 10 <= M <= m + 15, so that the weights times s fill e5m2's
// range and stay below its 57344.
template <bool E4M3> constexpr float kAbove = E4M3 ? 10.f : 0.f;
template <bool E4M3> constexpr float kMost = E4M3 ? 15.f : 8.f;
constexpr uint32_t kBarSoft = 1;                 // named barrier of the softmax warps

// Columns of S^T in the 16 x 256-bit shape: thread T holds tokens T / 4 and T / 4 + 8 of its warp's
// 16, rows 8 b + 2 (T % 4) + {0, 1}: registers 4 b + {0, 1} (token T / 4) and 4 b + {2, 3}.
template <int R>
__device__ __forceinline__ void tmem_ld_s(uint32_t ta, float (&r)[R / 2]) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    if constexpr (R == 16) {
        asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
                     : "r"(ta));
    } else {
#pragma unroll
        for (int i = 0; i < R / 32; ++i)
            asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                         "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                         : "=r"(u[16 * i + 0]), "=r"(u[16 * i + 1]), "=r"(u[16 * i + 2]), "=r"(u[16 * i + 3]),
                           "=r"(u[16 * i + 4]), "=r"(u[16 * i + 5]), "=r"(u[16 * i + 6]), "=r"(u[16 * i + 7]),
                           "=r"(u[16 * i + 8]), "=r"(u[16 * i + 9]), "=r"(u[16 * i + 10]), "=r"(u[16 * i + 11]),
                           "=r"(u[16 * i + 12]), "=r"(u[16 * i + 13]), "=r"(u[16 * i + 14]), "=r"(u[16 * i + 15])
                         : "r"(ta + 32u * i));
    }
    tc::tmem_wait_ld();
}

// 16 rows of a block of O (the sum of its three accumulators where P's terms lie side by side).
template <int R, bool SIDE>
__device__ __forceinline__ void load_o(uint32_t ta, float (&o)[16]) {
    tc::tmem_ld16(ta, o);
    if constexpr (SIDE) {
        float p[16], q[16];
        tc::tmem_ld16(ta + R, p);
        tc::tmem_ld16(ta + 2 * R, q);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] += p[i] + q[i];
    } else {
        tc::tmem_wait_ld();
    }
}

// The last K - 1 tokens of a sequence are seen by some of its queries and not by others.  In P the others
// have zeros there, but 0 * NaN is none in the product: latents that are NaN or infinite leave rows
// [lo, hi) of the tile before it.  For the queries that see such a token, an e4m3 one's score is NaN, and
// so is their sum; a bf16 one may score -inf and leave the sum alone, so mark_nonfinite puts it back.
template <int R, bool E4M3>
__device__ __forceinline__ bool drop_nonfinite(uint8_t* c, int lo, int hi, int tid) {
    using Sh = LatShape<R, E4M3>;
    constexpr int W = E4M3 ? 4 : 8;                              // slabs of latents
    auto kept = [](uint32_t w) {                                 // NaN codes, or an exponent of ones: zeroed
        return w & ~(E4M3 ? __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u));
    };
    bool found = false;
    for (int i = tid; i < W * (hi - lo) * 8; i += Sh::kSoft) {
        const int ch = i & 7, slab = i / 8 % W, r = lo + i / (8 * W);
        uint4* p = reinterpret_cast<uint4*>(c + (r >> 3) * Sh::kGroup + slab * Sh::kSlabC + (r & 7) * 128 + ch * 16);
        const uint4 v = *p, k = make_uint4(kept(v.x), kept(v.y), kept(v.z), kept(v.w));
        if (k.x != v.x || k.y != v.y || k.z != v.z || k.w != v.w) {
            *p = k;
            found = true;
        }
    }
    return found;
}

// In O, the results of rows that see a NaN or infinite bf16 latent among the segment's tokens from `clear` on: NaN in
// that channel (weight 0: 0 * inf; any other weight has made the sum NaN already).
// (Of a tree's nodes, the rows that see one of them: `seen`, else the rows that see past the first.)
template <int R, bool TREE>
__device__ __noinline__ void mark_nonfinite(const LatentCache& ch, int n, int clear, int from, int to, const int* s_j,
                                            const uint64_t* seen, uint32_t ta, int channel, int row_g) {
#pragma unroll 1
    for (int b = 0; b < 4; ++b) {
        int first = 0x7fffffff;                                  // the first such token: rows that see past it
        uint64_t nodes = 0;                                      // or all of them, as a tree's nodes
        for (int t = max(from, max(clear, 0)); t < to && first == 0x7fffffff; ++t) {
            int page = ch.table[static_cast<size_t>(n) * ch.max_pages + t / ch.page_size];
            if (page < 0 || page >= ch.num_pages) page = 0;     // (as it was copied)
            const uint8_t* row = ch.rows + (static_cast<size_t>(page) * ch.page_size + t % ch.page_size) * kLatRowBf16;
            if ((reinterpret_cast<const uint16_t*>(row)[128 * b + channel] & 0x7f80u) == 0x7f80u) {
                if constexpr (TREE) nodes |= 1ull << (t - clear);
                else first = t;
            }
        }
        if (!__any_sync(0xffffffffu, TREE ? nodes != 0 : first != 0x7fffffff)) continue;
#pragma unroll 1
        for (int c0 = row_g; c0 < row_g + LatShape<R, false>::RW; c0 += 16) {
            float o[16];
            tc::tmem_ld16(ta + b * R + c0, o);
            tc::tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (TREE ? (seen[c0 + i] & nodes) != 0 : clear + s_j[c0 + i] > first) o[i] = __int_as_float(0x7fffffff);
            tc::tmem_st16(ta + b * R + c0, o);
        }
        tc::tmem_wait_st();
    }
}

template <int R, bool E4M3, bool TREE>
__global__ void __launch_bounds__(LatShape<R, E4M3>::kThreads, 1)
kda_latent_decode_kernel(const __grid_constant__ LatMaps maps, const LatArgs a)
{
    using Sh = LatShape<R, E4M3>;
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* sQ = smem + Sh::oQ;
    uint8_t* sC = smem + Sh::oC;
    uint8_t* sP = smem + Sh::oP;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sh::oBar);
    uint64_t *full = bars, *empty = bars + 4, *s_full = bars + 8, *p_full = bars + 10, *q_full = bars + 11;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 12);
    float* s_red = reinterpret_cast<float*>(bars + 14);         // [4][R]
    float* s_f = s_red + 4 * R;                                 // [R]
    int* s_j = reinterpret_cast<int*>(s_f + R);                 // [R]: query token of each row
    float* s_a = s_f + 2 * R;                                   // [R]: e4m3: 2^k * scale of each row
    uint64_t* s_set = reinterpret_cast<uint64_t*>(s_a + R);     // [R]: TREE: the nodes that each row sees (none: no node itself)
    int32_t* s_lens = reinterpret_cast<int32_t*>(s_set + R);    // [kMaxNeed]: TREE: each sequence's length, ..
    uint8_t* s_need = reinterpret_cast<uint8_t*>(s_lens + kMaxNeed<E4M3>);    // .. and its row tiles
    constexpr int NS = Sh::kStages;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rt = blockIdx.x % a.RT, run = blockIdx.x / a.RT;
    LatWork work = a.w;
    // of a segment: its sequence, its first row there and how many follow
    const int each = lat_each<TREE>(a.w);
    auto seq_of = [&](int n) { return each > 1 ? n % (a.w.N / each) : n; };
    auto row_of = [&](int n) { return each > 1 ? n / (a.w.N / each) * R : rt * R; };
    auto rows_of = [&](int n) { return min(R, a.rows - row_of(n)); };

    if (tid == 0) {
        for (int i = 0; i < NS; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], 1);
        }
        tc::mbar_init(&s_full[0], 1);
        tc::mbar_init(&s_full[1], 1);
        tc::mbar_init(p_full, Sh::kSoft);
        tc::mbar_init(q_full, E4M3 ? Sh::kSoft : 1);
        tc::mbar_fence_init();
    }
    {   // the page table goes to L2 while the lengths that say where to read it are on their way: a line a thread
        const size_t lines = (static_cast<size_t>(a.w.N / each) * a.ch.max_pages * 4 + 127) / 128;
        const size_t mine = static_cast<size_t>(blockIdx.x) * Sh::kThreads + tid;
        if (mine < lines) asm volatile("prefetch.global.L2 [%0];" :: "l"(reinterpret_cast<const uint8_t*>(a.ch.table) + mine * 128));
    }
    if (tid == 0) {
        tc::tma_prefetch_map(&maps.c);
        if (E4M3) tc::tma_prefetch_map(&maps.s);
        else tc::tma_prefetch_map(&maps.q);
    }
    if (tid < R) s_j[tid] = min((rt * R + tid) / a.H, a.K - 1);
    if (each > 1 && work.N / each <= kMaxNeed<E4M3>) {
        const int seqs = work.N / each;
#pragma unroll 4
        for (int i = warp; i < seqs; i += Sh::kThreads / 32) {
            const int need = lat_need(a.parents + static_cast<long long>(i) * a.K, a.K, a.H, R, lane);
            if (lane == 0) s_need[i] = static_cast<uint8_t>(need);
        }
        for (int i = tid; i < seqs; i += Sh::kThreads) s_lens[i] = lat_seq<TREE>(a.w, i);
        work.need = s_need;
        work.lens = s_lens;
    }
    if (warp == Sh::kMmaWarp) tc::tmem_alloc(s_tmem, Sh::kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the combine kernel waits for this grid's end
    const uint32_t tm = *s_tmem, tmO = tm, tmS = tm + 4 * Sh::kO;
    SegWalk<TREE> sw;
    sw.init(work, run);
    bool ok = true;

    if (warp < Sh::kMmaWarp) {
        // ---- softmax: rows row_g .. + RW, a thread's tokens and rows of them as tmem_ld_s gives them ----
        constexpr int RW = Sh::RW;
        const int wq = Sh::kGroups > 1 ? warp & 3 : warp, row_g = Sh::kGroups > 1 ? (warp >> 2) * RW : 0;
        const int tq = lane >> 2, rq = row_g + 2 * (lane & 3);
        const uint32_t lane_tm = static_cast<uint32_t>(wq * 32) << 16;
        float m[RW / 4], l[RW / 4];
        int g = 0;                                              // tiles done by this CTA
        while (ok && sw.next(work)) {
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) { m[i] = -INFINITY; l[i] = 0.f; }
            const int clear = sw.len - (TREE ? a.K : a.K - 1);  // tokens that every row sees
            const int seq = seq_of(sw.n), row0 = row_of(sw.n), nrows = rows_of(sw.n);
            bool spoilt = false;                                // a later one held a NaN or infinity
            if constexpr (TREE) {                               // (the last readers of the sets before are past a barrier)
                if (warp == 0) {
                    uint64_t set[2];
                    if (tree_sets(a.parents + static_cast<long long>(seq) * a.K, a.K, lane, set) && lane == 0)
                        set_status(a.status, kStatusIndex);
#pragma unroll
                    for (int r = lane; r < (R < 32 ? 32 : R); r += 32) {
                        const uint64_t mine = tree_set_of(set, min((row0 + min(r, R - 1)) / a.H, a.K - 1));
                        if (r < R) s_set[r] = mine;
                    }
                }
                if (!E4M3) tc::named_sync(kBarSoft, Sh::kSoft);  // (e4m3: the one after Q)
            }
            if constexpr (E4M3) {
                // Q of the segment (the last S product of the segment before has run): a warp a row, the
                // loads of 4 rows in flight
#pragma unroll 1
                for (int rb = warp; rb < R; rb += 4 * Sh::kMmaWarp) {
                    uint4 w0[4], w1[4];
                    uint32_t rope[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint16_t* src = a.q + (static_cast<long long>(seq) * a.rows + row0 + min(rb + Sh::kMmaWarp * k, nrows - 1)) * kLatQ;
                        w0[k] = reinterpret_cast<const uint4*>(src)[2 * lane];
                        w1[k] = reinterpret_cast<const uint4*>(src)[2 * lane + 1];
                        rope[k] = reinterpret_cast<const uint32_t*>(src + kLatDim)[lane];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = rb + Sh::kMmaWarp * k;
                        const uint32_t wv[8] = {w0[k].x, w0[k].y, w0[k].z, w0[k].w, w1[k].x, w1[k].y, w1[k].z, w1[k].w};
                        uint32_t top2 = 0u;                     // largest magnitudes by their bits, two at a time
#pragma unroll
                        for (int i = 0; i < 8; ++i) top2 = __vmaxu2(top2, wv[i] & 0x7fff7fffu);
                        uint32_t top = __reduce_max_sync(0xffffffffu, max(top2 & 0xffffu, top2 >> 16));
                        // (a row with a NaN or an infinity gets codes of NaN, as its scores are none)
                        const bool none = top >= 0x7f80u;
                        const int e = none ? 0 : lat_scale_exponent(top << 16, 120);
                        // 2^-(8 + e): a denormal from e = 119 on (products with it are exact, as with the others)
                        const float inv = __uint_as_float(e < 119 ? static_cast<uint32_t>(119 - e) << 23 : 0x400000u >> (e - 119));
                        uint32_t t1[4], t2[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t c1[2], c2[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {       // x = q / 2^k: 8 bits, at most 448; fp16 holds x / 2^8
                                const float2 f = bf16x2_bits_to_f32(wv[2 * i + h]);
                                const uint32_t x = f32x2_to_f16x2(f.x * inv, f.y * inv), y = f16x2_round_e4m3(x);
                                c1[h] = e4m3_codes(y);
                                c2[h] = e4m3_codes(f16x2_round_e4m3(f16x2_sub(x, y)));
                            }
                            t1[i] = none ? 0x7f7f7f7fu : __byte_perm(c1[0], c1[1], 0x6420);
                            t2[i] = none ? 0u : __byte_perm(c2[0], c2[1], 0x6420);
                        }
                        uint8_t* d = sQ + (lane >> 3) * Sh::kSlabQ + r * 128 + (((lane & 7) ^ (r & 7)) << 4);
                        *reinterpret_cast<uint4*>(d) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
                        *reinterpret_cast<uint4*>(d + 4 * Sh::kSlabQ) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
                        *reinterpret_cast<uint32_t*>(sQ + 8 * Sh::kSlabQ + tc::sw128_off16(r, 2 * lane, R)) = rope[k];
                        if (lane == 0) s_a[r] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
                    }
                }
                tc::fence_smem_to_async();
                tc::mbar_arrive(q_full);
                tc::named_sync(kBarSoft, Sh::kSoft);             // s_a is read by all
            }
            for (int t = sw.t0; t < sw.t1; ++t, ++g) {
                ok = __all_sync(0xffffffffu, ok && tc::mbar_wait_bounded(&s_full[g & 1], (g >> 1) & 1, kWaitLimitNs));
                float x[RW / 2];
                float s0 = 1.f, s1 = 1.f, e0 = 0.f, e1 = 0.f;   // e4m3: scales of the thread's two tokens, their exponents
                if (ok) {
                    tc::fence_after_sync();
                    tmem_ld_s<RW>(tmS + (g & 1) * Sh::kS + row_g + lane_tm, x);
                    if constexpr (E4M3) {
                        const float* sc = reinterpret_cast<const float*>(sC + g % NS * Sh::kStage + Sh::kRows);
                        s0 = sc[(16 * wq + tq) * 4];
                        s1 = sc[(16 * wq + tq + 8) * 4];
                        // (held above -90, so that the sums of 2^(x - m) stay within fp32; see f0, f1)
                        e0 = static_cast<float>(max(static_cast<int>(__float_as_uint(s0) >> 23) - 127, -90));
                        e1 = static_cast<float>(max(static_cast<int>(__float_as_uint(s1) >> 23) - 127, -90));
                        // a scale that is NaN or infinite: the token's scores are NaN, for the rows that see it, and
                        // it enters P as if it were 1, where the others have zeros
                        float a0 = e0, a1 = e1;
                        if (!(fabsf(s0) < INFINITY)) { a0 = __int_as_float(0x7fffffff); s0 = 1.f; e0 = 0.f; }
                        if (!(fabsf(s1) < INFINITY)) { a1 = __int_as_float(0x7fffffff); s1 = 1.f; e1 = 0.f; }
                        float xr[RW / 2];
                        tmem_ld_s<RW>(tmS + (g & 1) * Sh::kS + R + row_g + lane_tm, xr);
                        // x: scores in powers of two, plus the scale's exponent (the weights carry s)
#pragma unroll
                        for (int i = 0; i < RW / 2; ++i) {
                            const float sa = s_a[8 * (i >> 2) + rq + (i & 1)] * (i & 2 ? s1 : s0);
                            x[i] = fmaf(x[i], sa, fmaf(xr[i], a.scale_log2, i & 2 ? a1 : a0));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < RW / 2; ++i) x[i] *= a.scale_log2;
                    }
                }
                const int tok = t * kTile + 16 * wq + tq;     // and tok + 8
                const bool edge = (t + 1) * kTile > clear;
                if (edge) {
#pragma unroll
                    for (int i = 0; i < RW / 2; ++i) {
                        const int r = 8 * (i >> 2) + rq + (i & 1);
                        if constexpr (TREE) {
                            const int node = tok + 4 * (i & 2) - clear;
                            x[i] = node < 0 || (node < a.K && s_set[r] >> node & 1) ? x[i] : -INFINITY;
                        } else {
                            const int see = clear + s_j[r];
                            x[i] = tok + 4 * (i & 2) < see ? x[i] : -INFINITY;
                        }
                    }
                    // rows past the end of the sequence hold anything: they enter the second product as zeros
                    const int valid = sw.len - t * kTile;
                    if (ok && valid < kTile) {
                        uint8_t* c = sC + g % NS * Sh::kStage;
                        constexpr int W = E4M3 ? 4 : 8;         // slabs of latents
                        for (int i = tid; i < W * (kTile - valid) * 8; i += Sh::kSoft) {
                            const int ch = i & 7, slab = i / 8 % W, r = valid + i / (8 * W);
                            *reinterpret_cast<uint4*>(c + (r >> 3) * Sh::kGroup + slab * Sh::kSlabC + (r & 7) * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
                        }
                        if (E4M3) {                             // and their scales are not to be used
                            if (16 * wq + tq >= valid) { s0 = 1.f; e0 = 0.f; }
                            if (16 * wq + tq + 8 >= valid) { s1 = 1.f; e1 = 0.f; }
                        }
                    }
                    if (ok && (TREE || a.K > 1))
                        spoilt |= drop_nonfinite<R, E4M3>(sC + g % NS * Sh::kStage, max(0, clear - t * kTile), min(kTile, valid), tid);
                }
                bool grow = !ok;
#pragma unroll
                for (int i = 0; i < RW / 2; ++i) grow |= x[i] > m[2 * (i >> 2) + (i & 1)] + kMost<E4M3>;
                bool waited = g == 0;                           // for the previous tile's product: it has read P and is in O
                if (!tc::named_sync_and(kBarSoft, Sh::kSoft, !grow)) {
                    if (ok && !waited) ok = tc::mbar_wait_bounded(&empty[(g - 1) % NS], (g - 1) / NS & 1, kWaitLimitNs);
                    waited = true;
                    ok = tc::named_sync_and(kBarSoft, Sh::kSoft, ok);
                    if (!ok) break;
                    tc::fence_after_sync();
#pragma unroll
                    for (int i = 0; i < RW / 4; ++i) {           // maxima of the tile, per row
                        float v = fmaxf(x[4 * (i >> 1) + (i & 1)], x[4 * (i >> 1) + 2 + (i & 1)]);
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                        if (lane < 4) s_red[wq * R + 8 * (i >> 1) + rq + (i & 1)] = v;
                    }
                    tc::named_sync(kBarSoft, Sh::kSoft);
#pragma unroll
                    for (int i = 0; i < RW / 4; ++i) {
                        const int r = 8 * (i >> 1) + rq + (i & 1);
                        const float mx = fmaxf(fmaxf(s_red[r], s_red[R + r]), fmaxf(s_red[2 * R + r], s_red[3 * R + r]));
                        const float mn = fmaxf(m[i], mx - kAbove<E4M3>);
                        const float f = mn == m[i] ? 1.f : lat_ex2(m[i] - mn);
                        m[i] = mn;
                        l[i] *= f;
                        if (wq == 0 && lane < 4) s_f[r] = f;
                    }
                    tc::named_sync(kBarSoft, Sh::kSoft);
                    if (t > sw.t0) {                            // O *= f, 16 columns (rows) at a time
#pragma unroll 1
                        for (int c0 = row_g; c0 < (Sh::kGroups > 1 ? row_g + RW : static_cast<int>(Sh::kO)); c0 += 16) {
                            const float* f = s_f + c0 % R;
                            bool one = true;
#pragma unroll
                            for (int i = 0; i < 16; ++i) one = one && f[i] == 1.f;
                            if (one) continue;
#pragma unroll 1
                            for (int b = 0; b < 4; ++b) {
                                float o[16];
                                tc::tmem_ld16(tmO + b * Sh::kO + c0 + lane_tm, o);
                                tc::tmem_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) o[i] *= f[i];
                                tc::tmem_st16(tmO + b * Sh::kO + c0 + lane_tm, o);
                            }
                        }
                        tc::tmem_wait_st();
                    }
                }
                // P = exp2(x - m), rounded for the product (see above); the sums keep fp32.  It is made in
                // registers while the previous tile's product still reads P
                const int tr = 16 * wq + tq;
                // e4m3: exp2(x - m) carries 2^e; the sums take it out (r0, r1), and a scale below 2^-90 puts the
                // rest of it in (f0, f1, else 1).  A NaN score leaves no NaN in P, but one in the sums
                const float r0 = lat_ex2(-e0), r1 = lat_ex2(-e1), f0 = s0 * r0, f1 = s1 * r1;
                uint32_t pk[E4M3 ? 3 * (RW / 8) : RW / 4];
#pragma unroll
                for (int b = 0; b < RW / 8; ++b) {
                    const float m0 = m[2 * b] == -INFINITY ? 0.f : m[2 * b], m1 = m[2 * b + 1] == -INFINITY ? 0.f : m[2 * b + 1];
                    const float p0 = lat_ex2(x[4 * b] - m0), p1 = lat_ex2(x[4 * b + 1] - m1);
                    const float p2 = lat_ex2(x[4 * b + 2] - m0), p3 = lat_ex2(x[4 * b + 3] - m1);
                    if constexpr (!E4M3) {
                        l[2 * b] += p0 + p2;
                        l[2 * b + 1] += p1 + p3;
                        pk[2 * b] = f32x2_to_bf16x2_bits(p0, p1);
                        pk[2 * b + 1] = f32x2_to_bf16x2_bits(p2, p3);
                    } else {
                        l[2 * b] += fmaf(p0, r0, p2 * r1);
                        l[2 * b + 1] += fmaf(p1, r0, p3 * r1);
                        uint32_t u = f32x2_to_f16x2(p0 * f0, p1 * f0), v = f32x2_to_f16x2(p2 * f1, p3 * f1);
#pragma unroll
                        for (int k = 0; k < 3; ++k) {           // three terms, each the rounding of what is left
                            const uint32_t ru = f16x2_round_e5m2(u), rv = f16x2_round_e5m2(v);
                            pk[3 * b + k] = __byte_perm(ru, rv, 0x7531);
                            u = f16x2_sub(u, ru);
                            v = f16x2_sub(v, rv);
                        }
                    }
                }
                // (a wait that ran out is agreed on at the next vote, so that no warp leaves the others there)
                if (ok && !waited) ok = tc::mbar_wait_bounded(&empty[(g - 1) % NS], (g - 1) / NS & 1, kWaitLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) continue;
#pragma unroll
                for (int b = 0; b < RW / 8; ++b) {
                    if constexpr (!E4M3) {
                        const uint32_t off = tc::sw128_off16(tr, 8 * b + rq, kTile);
                        *reinterpret_cast<uint32_t*>(sP + off) = pk[2 * b];
                        *reinterpret_cast<uint32_t*>(sP + off + 8 * 128) = pk[2 * b + 1];    // token + 8: same swizzle
                    } else {
#pragma unroll
                        for (int k = 0; k < 3; ++k) {
                            const uint32_t n = 8 * b + rq + (Sh::kSide ? k * R : 0);
                            uint8_t* d = sP + (Sh::kSide ? 0 : k * kTile * 128) + tr * 128 + (((n >> 4) ^ (tr & 7)) << 4) + (n & 15);
                            *reinterpret_cast<uint16_t*>(d) = static_cast<uint16_t>(pk[3 * b + k]);
                            *reinterpret_cast<uint16_t*>(d + 8 * 128) = static_cast<uint16_t>(pk[3 * b + k] >> 16);
                        }
                    }
                }
                tc::fence_smem_to_async();
                tc::fence_before_sync();
                tc::mbar_arrive(p_full);
            }
            // ---- epilogue of the segment: O^T is complete once the last product is ----
            ok = ok && tc::mbar_wait_bounded(&empty[(g - 1) % NS], (g - 1) / NS & 1, kWaitLimitNs);
            ok = tc::named_sync_and(kBarSoft, Sh::kSoft, ok);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll
            for (int i = 0; i < RW / 4; ++i) {
                float v = l[i];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                const int r = 8 * (i >> 1) + rq + (i & 1);
                if (lane < 4) s_red[wq * R + r] = v;
                if (wq == 0 && lane < 4) s_f[r] = m[i];
            }
            if (!tc::named_sync_and(kBarSoft, Sh::kSoft, !spoilt) && !E4M3)
                mark_nonfinite<R, TREE>(a.ch, seq, clear, sw.t0 * kTile, min(sw.len, sw.t1 * kTile), s_j, s_set, tmO + lane_tm,
                                        32 * wq + lane, row_g);
            const bool whole = sw.whole();
            const long long row_at = static_cast<long long>(seq) * a.rows + row0;
            const size_t part = (static_cast<size_t>(run) * a.RT + rt) * 2 + (sw.first ? 0 : 1);
            if (tid < R) {                                       // a thread a row
                float mr = s_f[tid], sum = (s_red[tid] + s_red[R + tid]) + (s_red[2 * R + tid] + s_red[3 * R + tid]);
                if (TREE && s_set[tid] == 0) {                   // no node: it has seen nothing
                    mr = -INFINITY;
                    sum = 0.f;
                }
                if (!whole) *reinterpret_cast<float2*>(a.part_ml + (part * R + tid) * 2) = make_float2(mr, sum);
                else if (a.lse && tid < nrows) a.lse[row_at + tid] = (mr + log2f(sum)) * 0.69314718055994531f;
                s_f[tid] = sum == 0.f ? 0.f : 1.f / sum;
            }
            tc::named_sync(kBarSoft, Sh::kSoft);
            const int ch = 32 * wq + lane;
            if (!whole) {
                float* d32 = a.part_o + part * R * kLatDim + ch;
#pragma unroll 1
                for (int c = row_g / 4; c < (row_g + RW) / 4; ++c) {     // 16 rows x 128 channels a step
                    float o[16];
                    load_o<R, Sh::kSide>(tmO + (c & 3) * Sh::kO + (c >> 2) * 16 + lane_tm, o);
                    float* d = d32 + (c >> 2) * 16 * kLatDim + (c & 3) * 128;
#pragma unroll
                    for (int i = 0; i < 16; ++i) d[i * kLatDim] = o[i];
                }
            } else {
                // two rows a store: packed as (row i, row i + 1) of one channel, then the even lane of a pair
                // takes both channels of row i, the odd lane those of row i + 1
                const int odd = lane & 1;
                const uint32_t sel = odd ? 0x3276u : 0x5410u;
                uint16_t* d16 = a.out + (row_at + odd) * kLatDim + (ch - odd);
#pragma unroll 1
                for (int c = row_g / 4; c < (row_g + RW) / 4; ++c) {
                    const int c0 = (c >> 2) * 16;
                    if (c0 >= nrows) break;
                    float o[16];
                    load_o<R, Sh::kSide>(tmO + (c & 3) * Sh::kO + c0 + lane_tm, o);
                    uint16_t* d = d16 + c0 * kLatDim + (c & 3) * 128;
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float2 f = *reinterpret_cast<const float2*>(s_f + c0 + i);
                        float y0 = o[i] * f.x, y1 = o[i + 1] * f.y;
                        if constexpr (TREE) {                    // (a place without a node may hold anything)
                            y0 = f.x == 0.f ? 0.f : y0;
                            y1 = f.y == 0.f ? 0.f : y1;
                        }
                        const uint32_t w = f32x2_to_bf16x2_bits(y0, y1);
                        const uint32_t got = __shfl_xor_sync(0xffffffffu, w, 1);
                        if (c0 + i + odd < nrows) *reinterpret_cast<uint32_t*>(d + i * kLatDim) = __byte_perm(w, got, sel);
                    }
                }
            }
            tc::fence_before_sync();                             // the next segment's product overwrites O
            sw.first = false;
        }
        // sequences that hold nothing, where the kernel that joins sees those alone that are cut
        if (a.cuts && ok)
            for (int n = run; n < a.w.N; n += a.w.G) {
                if (lat_len<TREE>(work, n) != 0) continue;
                const int seq = seq_of(n), row0 = row_of(n), nrows = rows_of(n);
                const long long at = static_cast<long long>(seq) * a.rows + row0;
                for (int i = tid; i < nrows * (kLatDim / 8); i += Sh::kSoft) reinterpret_cast<uint4*>(a.out + at * kLatDim)[i] = make_uint4(0, 0, 0, 0);
                if (a.lse && tid < nrows) a.lse[at + tid] = -INFINITY;
                if (tid == 0 && row0 == 0 && lat_seq<TREE>(a.w, seq) != a.w.seq_lens[seq]) set_status(a.status, kStatusIndex);
            }
    } else if (warp == Sh::kMmaWarp) {
        // ---- both products; whichever has its inputs goes first ----
        // One thread runs it all: the tensor cores queue only about two products, so what stands between
        // two groups of them (a vote, an election) is lost
        constexpr uint32_t id_s = tc::idesc(64, R, tc::kFmtBF16, false, false);
        constexpr uint32_t id_o = E4M3 ? tc::idesc8(128, Sh::kO, tc::kFmtE4M3, tc::kFmtE5M2, true, true)
                                       : tc::idesc(128, R, tc::kFmtBF16, true, true);
        constexpr uint32_t id_c = tc::idesc8(64, R, tc::kFmtE4M3, tc::kFmtE4M3, false, false);
        // descriptors: constant high words, low words = address / 16 and the leading offset
        const uint64_t d0 = tc::sdesc(0, 16, 1024, tc::kSwizzle128B), dC = tc::sdesc(0, Sh::kSlabC, Sh::kGroup, tc::kSwizzle128B);
        const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
        const uint32_t q_lo = static_cast<uint32_t>(d0) | (tc::smem_u32(sQ) >> 4);
        const uint32_t hi_c = static_cast<uint32_t>(dC >> 32);
        const uint32_t c_lo = static_cast<uint32_t>(dC) | (tc::smem_u32(sC) >> 4);
        const uint32_t p_lo = static_cast<uint32_t>(d0) | (tc::smem_u32(sP) >> 4);
        SegWalk<TREE> sv = sw;                                  // the O product's walk follows the S product's
        bool more_s = sw.next(work), more_o = sv.next(work);
        int gs = 0, go = 0, qs = 0;                             // S and O tiles issued, segments whose Q is in
        int ts = sw.t0, to = sv.t0;
        uint64_t since = 0;
        uint32_t idle = 0;
        const bool leader = tc::elect_one();
        while (more_o && leader) {
            bool moved = false;
            // O of a tile before S of the next but one; S at most one tile ahead of O (its S buffer is
            // read before P is written)
            if (go < gs && tc::mbar_test_wait(p_full, go & 1)) {
                tc::fence_after_sync();
                const uint32_t c = c_lo + go % NS * (Sh::kStage >> 4);
                const uint32_t acc = to > sv.t0 ? 1u : 0u;
#pragma unroll
                for (uint32_t b = 0; b < 4; ++b) {
                    if constexpr (!E4M3) {
#pragma unroll
                        for (uint32_t k = 0; k < 4; ++k)
                            tc::mma_f16_lo(tmO + b * R, c + ((b * 2u * Sh::kSlabC + k * 2u * Sh::kGroup) >> 4), hi_c,
                                           p_lo + (k * 2048u >> 4), hi, id_o, k > 0 ? 1u : acc);
                    } else if constexpr (Sh::kSide) {
#pragma unroll
                        for (uint32_t k = 0; k < 2; ++k)     // 2 steps of 32 tokens, all terms at once
                            tc::mma_f8_lo(tmO + b * Sh::kO, c + ((b * Sh::kSlabC + k * 4u * Sh::kGroup) >> 4), hi_c,
                                          p_lo + (k * 4096u >> 4), hi, id_o, k > 0 ? 1u : acc);
                    } else {
#pragma unroll
                        for (uint32_t k = 0; k < 6; ++k)     // 2 steps of 32 tokens x 3 terms
                            tc::mma_f8_lo(tmO + b * R, c + ((b * Sh::kSlabC + k / 3u * 4u * Sh::kGroup) >> 4), hi_c,
                                          p_lo + ((k % 3u * kTile * 128u + k / 3u * 4096u) >> 4), hi, id_o, k > 0 ? 1u : acc);
                    }
                }
                tc::mma_commit(&empty[go % NS]);
                ++go;
                if (++to == sv.t1) {
                    more_o = sv.next(work);
                    to = sv.t0;
                }
                moved = true;
            }
            if (more_s && gs <= go + 1 && (ts > sw.t0 || tc::mbar_test_wait(q_full, qs & 1)) &&
                tc::mbar_test_wait(&full[gs % NS], gs / NS & 1)) {
                tc::fence_after_sync();
                const uint32_t c = c_lo + gs % NS * (Sh::kStage >> 4), d = tmS + (gs & 1) * Sh::kS;
                if constexpr (!E4M3) {
#pragma unroll
                    for (uint32_t k = 0; k < 36; ++k)
                        tc::mma_f16_lo(d, c + (((k >> 2) * Sh::kSlabC + (k & 3) * 32u) >> 4), hi_c,
                                       q_lo + (((k >> 2) * Sh::kSlabQ + (k & 3) * 32u) >> 4), hi, id_s, k > 0 ? 1u : 0u);
                } else {
#pragma unroll
                    for (uint32_t k = 0; k < 32; ++k)        // 16 steps of 32 codes x 2 terms of q
                        tc::mma_f8_lo(d, c + (((k >> 3) * Sh::kSlabC + (k >> 1 & 3) * 32u) >> 4), hi_c,
                                      q_lo + (((k & 1) * 4u * Sh::kSlabQ + (k >> 3) * Sh::kSlabQ + (k >> 1 & 3) * 32u) >> 4), hi,
                                      id_c, k > 0 ? 1u : 0u);
#pragma unroll
                    for (uint32_t k = 0; k < 4; ++k)         // the position part, bf16
                        tc::mma_f16_lo(d + R, c + ((4u * Sh::kSlabC + k * 32u) >> 4), hi_c,
                                       q_lo + ((8u * Sh::kSlabQ + k * 32u) >> 4), hi, id_s, k > 0 ? 1u : 0u);
                }
                tc::mma_commit(&s_full[gs & 1]);
                ++gs;
                if (++ts == sw.t1) {
                    ++qs;
                    more_s = sw.next(work);
                    ts = sw.t0;
                }
                moved = true;
            }
            if (moved) {
                idle = 0;
            } else if ((++idle & 255u) == 0) {                  // the clock is read every 256 idle rounds
                const uint64_t now = tc::globaltimer_ns();
                if (idle == 256u) since = now;
                else if (now - since > kWaitLimitNs) { ok = false; break; }
            }
        }
        // nothing of this CTA's is left running when it returns its TMEM
        if (leader && gs > 0 && !tc::mbar_wait_bounded(&s_full[(gs - 1) & 1], ((gs - 1) >> 1) & 1, kWaitLimitNs)) ok = false;
        if (leader && go > 0 && !tc::mbar_wait_bounded(&empty[(go - 1) % NS], (go - 1) / NS & 1, kWaitLimitNs)) ok = false;
        __syncwarp();
    } else {
        // ---- TMA: C tiles in boxes of `box` whole rows (one page or a part of one); bf16: Q of each segment ----
        const int nbox = kTile / a.box;
        int g = 0, seg = 0;
        LatCut cut{0, 0, -1};
        while (ok && sw.next(work)) {
            auto pages = [&](int t) {                           // lane i: first cache row of box i of tile t, -1 = past the end
                const int tok = t * kTile + lane * a.box;
                if (t >= sw.t1 || lane >= nbox || tok >= sw.len) return -1;
                int page = a.ch.table[static_cast<size_t>(seq_of(sw.n)) * a.ch.max_pages + tok / a.ch.page_size];
                if (page < 0 || page >= a.ch.num_pages) { set_status(a.status, kStatusIndex); page = 0; }
                return page * a.ch.page_size + tok % a.ch.page_size;
            };
            int at = pages(sw.t0);
            if constexpr (!E4M3) {
                // Q is free once the last S product of the segment before has run
                if (g > 0) ok = tc::mbar_wait_bounded(&s_full[(g - 1) & 1], ((g - 1) >> 1) & 1, kWaitLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (lane == 0) tc::mbar_arrive_expect_tx(q_full, 9u * Sh::kSlabQ);
                __syncwarp();
                if (lane < 9)
                    tc::tma_load_2d(tc::smem_u32(sQ) + lane * Sh::kSlabQ, &maps.q, 64 * lane,
                                    static_cast<int>(static_cast<long long>(seq_of(sw.n)) * a.rows + row_of(sw.n)), q_full);
                ++seg;
            }
            for (int t = sw.t0; t < sw.t1; ++t, ++g) {
                const int next = pages(t + 1);
                if (g >= NS) ok = tc::mbar_wait_bounded(&empty[g % NS], (g / NS - 1) & 1, kWaitLimitNs);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const int boxes = __popc(__ballot_sync(0xffffffffu, at >= 0));
                const uint32_t dst = tc::smem_u32(sC) + g % NS * Sh::kStage;
                // rows that softmax threads zeroed are overwritten by the copy: order the two
                tc::fence_smem_to_async();
                if (lane == 0)
                    tc::mbar_arrive_expect_tx(&full[g % NS], static_cast<uint32_t>(boxes * a.box) * (Sh::kSlabs * 128u + (E4M3 ? 16u : 0u)));
                __syncwarp();
                if (at >= 0) {                                   // a box a lane: all of its rows in one copy
                    tc::tma_load_4d(dst + lane * (a.box >> 3) * Sh::kGroup, &maps.c, 0, 0, 0, at >> 3, &full[g % NS]);
                    if (E4M3) tc::tma_load_2d(dst + Sh::kRows + lane * a.box * 16, &maps.s, kLatScaleAt, at, &full[g % NS]);
                }
                if constexpr (R == 64 && !E4M3) {
                    // the next tile is fetched into L2 meanwhile, as two stages do not cover a copy from HBM: 64
                    // sequences x 64 heads 209 -> 194 us, 16 x K = 4 x 32 heads 105 -> 97, one of 145408 x 64
                    // heads 55.6 -> 53.3.  (With 32 rows HBM is the bound: 189 -> 205.  Three stages of an e4m3
                    // cache cover it: no change.  Two tiles ahead: 196, 99, 53.7.)
                    if ((each > 1 || rt == 0) && next >= 0) tc::tma_prefetch_4d(&maps.c, 0, 0, 0, next >> 3);
                }
                at = next;
            }
            if (sw.t0 == 0 && !sw.whole()) cut = LatCut{sw.base, sw.total, sw.n};
        }
        if (a.cuts && rt == 0 && lane == 0) a.cuts[run] = ok ? cut : LatCut{0, 0, -1};      // for the kernel that joins
        // copies in flight land before the CTA's shared memory is given back
        if (!ok) {
            if (seg > 0) tc::mbar_wait_bounded(q_full, (seg - 1) & 1, kWaitLimitNs);
            for (int i = max(0, g - NS); i < g; ++i) tc::mbar_wait_bounded(&full[i % NS], i / NS & 1, kWaitLimitNs);
        }
    }
    if (!ok) set_status(a.status, kStatusTimeout);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == Sh::kMmaWarp) tc::tmem_dealloc(tm, Sh::kTmemCols);
}

// Joins the partials of sequences that several CTAs worked on, and writes empty sequences.  A block
// takes one row (x 1 / Q of its channels when there are few rows): NG groups of 128 / Q threads, 4
// channels a thread, group i every NG-th partial, in one pass with the running maximum and 8 partials'
// loads in flight; then the groups are joined.
constexpr int kMaxRuns = 1024;                  // partials of a row (at most one a run)

template <int R, bool TREE>
__global__ void __launch_bounds__(512)
kda_latent_combine_kernel(const LatArgs a, int Q, int NG)
{
    __shared__ float4 s_acc[512];
    __shared__ float2 s_ml[16];                                 // (m, l) of each group
    const int lanes = 128 / Q;
    const int unit = blockIdx.x / Q, n = unit / a.rows, row = unit % a.rows;
    const int tid = threadIdx.x, grp = tid / lanes, ch = (blockIdx.x % Q * lanes + tid % lanes) * 4;
    const int each = lat_each<TREE>(a.w), tile = each > 1 ? row / R : 0;     // (of those that are sequences of their own)
    const LatCount c = lat_counted<R, TREE>(a, n, tile, tid & 31);
    if (tid == 0 && row == 0 && a.w.seq_lens[n] != c.len) set_status(a.status, kStatusIndex);    // out of range: counted as 0
    const long long T = c.T, before = c.before;
    const int tiles = tile < c.need ? lat_tiles(c.len) : 0;
    const long long at = static_cast<long long>(n) * a.rows + row;
    int c0 = 0, parts = 1, late = 0;
    if (tiles > 0) {
        const long long runs = lat_runs(T, a.w.G);
        c0 = static_cast<int>(run_of(T, runs, before + a.w.lead));
        parts = static_cast<int>(run_of(T, runs, before + a.w.lead + tiles - 1)) - c0 + 1;
        // a run's partial is its first segment's, unless it began with an earlier sequence's tiles
        // (the one before a sequence's lead is work)
        late = run_begin(T, runs, c0) < before ? 1 : 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");          // every block: this grid ends after the one before it
    if (tiles == 0) {
        if (grp == 0) *reinterpret_cast<uint2*>(a.out + at * kLatDim + ch) = make_uint2(0u, 0u);
        if (tid == 0 && ch == 0 && a.lse) a.lse[at] = -INFINITY;
        return;
    }
    if (parts == 1) return;                                      // its CTA finished it
    const int r = row % R;
    const size_t stride = static_cast<size_t>(a.RT) * 2 * R;     // rows of partials between runs
    const size_t base = (static_cast<size_t>(c0) * a.RT + (each > 1 ? 0 : row / R)) * 2 * R + r;
    auto slot = [&](int i) { return base + i * stride + (i == 0 && late ? R : 0); };
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    // joins B partials (m, l, O) with it; one that saw nothing (m = -inf, l = 0) has no part in it
    auto join = [&](const auto& v, const auto& x) {
        constexpr int B = sizeof(v) / sizeof(float2);
        float mx = M;
#pragma unroll
        for (int i = 0; i < B; ++i) mx = fmaxf(mx, v[i].x);
        const float f = mx == M ? 1.f : lat_ex2(M - mx);
        M = mx;
        L *= f;
        acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (v[i].x == -INFINITY && v[i].y == 0.f) continue;
            const float w = v[i].x == M ? 1.f : lat_ex2(v[i].x - M);
            L += w * v[i].y;
            acc.x += w * x[i].x; acc.y += w * x[i].y; acc.z += w * x[i].z; acc.w += w * x[i].w;
        }
    };
    for (int i0 = grp; i0 < parts; i0 += 8 * NG) {
        float2 v[8];
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * NG;
            v[k] = i < parts ? *reinterpret_cast<const float2*>(a.part_ml + slot(i) * 2) : make_float2(-INFINITY, 0.f);
            x[k] = i < parts ? *reinterpret_cast<const float4*>(a.part_o + slot(i) * kLatDim + ch) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
        join(v, x);
    }
    if (NG > 1) {
        s_acc[tid] = acc;
        if (tid % lanes == 0) s_ml[grp] = make_float2(M, L);
        __syncthreads();
    }
    if (grp == 0) {
        for (int i = 1; i < NG; ++i) {
            const float2 v[1] = {s_ml[i]};
            const float4 x[1] = {s_acc[tid + i * lanes]};
            join(v, x);
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2*>(a.out + at * kLatDim + ch) = make_uint2(f32x2_to_bf16x2_bits(acc.x * inv, acc.y * inv),
                                                                          f32x2_to_bf16x2_bits(acc.z * inv, acc.w * inv));
        if (ch == 0 && a.lse) a.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
    }
}

// The same for many rows of few partials: a warp a row, 16 channels a lane, no block-wide step.
// (Four blocks an SM are enough: for more, the compiler spills into 48 registers.)
// MANY: of the runs' cut sequences alone.
template <int R, bool MANY, bool TREE>
__global__ void __launch_bounds__(128, 4)
kda_latent_combine_rows_kernel(const LatArgs a)
{
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int each = lat_each<TREE>(a.w), seqs = a.w.N / each;
    int n, row, tiles;
    long long T, before;
    if constexpr (MANY) {                                        // unit: row of a run's cut sequence
        const int per = each > 1 ? R : a.rows, run = static_cast<int>(unit / per);
        asm volatile("griddepcontrol.wait;" ::: "memory");
        const LatCut cut = run < a.w.G ? a.cuts[run] : LatCut{0, 0, -1};
        if (cut.n < 0) return;
        n = each > 1 ? cut.n % seqs : cut.n;
        row = static_cast<int>(unit - static_cast<long long>(run) * per) + (each > 1 ? cut.n / seqs * R : 0);
        tiles = lat_tiles(lat_seq<TREE>(a.w, n));
        T = cut.T;
        before = cut.before;
    } else {                                                     // unit: n * rows + row
        n = static_cast<int>(min(unit, static_cast<long long>(seqs) * a.rows - 1) / a.rows);
        row = static_cast<int>(unit - static_cast<long long>(n) * a.rows);
        const int tile = each > 1 ? min(row, a.rows - 1) / R : 0;        // (of those that are sequences of their own)
        const LatCount c = lat_counted<R, TREE>(a, n, tile, lane);
        if (lane == 0 && row == 0 && a.w.seq_lens[n] != c.len) set_status(a.status, kStatusIndex);   // out of range: counted as 0
        tiles = tile < c.need ? lat_tiles(c.len) : 0;
        T = c.T;
        before = c.before;
    }
    const long long at = static_cast<long long>(n) * a.rows + row;
    int c0 = 0, parts = 1, late = 0;
    if (tiles > 0) {
        const long long runs = lat_runs(T, a.w.G);
        c0 = static_cast<int>(run_of(T, runs, before + a.w.lead));
        parts = static_cast<int>(run_of(T, runs, before + a.w.lead + tiles - 1)) - c0 + 1;
        late = run_begin(T, runs, c0) < before ? 1 : 0;
    }
    if (!MANY) asm volatile("griddepcontrol.wait;" ::: "memory");            // every block: this grid ends after the one before it
    if (row >= a.rows) return;                                   // (past the last row)
    uint2* out = reinterpret_cast<uint2*>(a.out + at * kLatDim) + lane;
    if (tiles == 0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) out[32 * k] = make_uint2(0u, 0u);
        if (lane == 0 && a.lse) a.lse[at] = -INFINITY;
        return;
    }
    if (parts == 1) return;                                      // its CTA finished it
    const size_t stride = static_cast<size_t>(a.RT) * 2 * R;
    const size_t base = (static_cast<size_t>(c0) * a.RT + (each > 1 ? 0 : row / R)) * 2 * R + row % R;
    float M = -INFINITY, L = 0.f;
    float4 acc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += 32) {                     // 32 partials at a time, one pass
        const size_t mine = base + (i0 + lane) * stride + (i0 + lane == 0 && late ? R : 0);
        const float2 ml = i0 + lane < parts ? *reinterpret_cast<const float2*>(a.part_ml + mine * 2) : make_float2(-INFINITY, 0.f);
        float mx = ml.x;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float Mn = fmaxf(M, mx), f = Mn == M ? 1.f : lat_ex2(M - Mn);
        M = Mn;
        const bool none = ml.x == -INFINITY && ml.y == 0.f;      // saw nothing there
        const float w = none ? -1.f : ml.x == M ? 1.f : lat_ex2(ml.x - M);
        float sum = none ? 0.f : w * ml.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        L = L * f + sum;
#pragma unroll
        for (int k = 0; k < 4; ++k) { acc[k].x *= f; acc[k].y *= f; acc[k].z *= f; acc[k].w *= f; }
        const int some = min(32, parts - i0);
#pragma unroll 2
        for (int i = 0; i < some; ++i) {
            const float wi = __shfl_sync(0xffffffffu, w, i);
            const size_t sl = base + (i0 + i) * stride + (i0 + i == 0 && late ? R : 0);
            const float4* o = reinterpret_cast<const float4*>(a.part_o + sl * kLatDim) + lane;
            float4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = o[32 * k];
            if (wi >= 0.f)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    acc[k].x += wi * v[k].x; acc[k].y += wi * v[k].y; acc[k].z += wi * v[k].z; acc[k].w += wi * v[k].w;
                }
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        out[32 * k] = make_uint2(f32x2_to_bf16x2_bits(acc[k].x * inv, acc[k].y * inv),
                                 f32x2_to_bf16x2_bits(acc[k].z * inv, acc[k].w * inv));
    if (lane == 0 && a.lse) a.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
}

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    if (!fn) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &qr) == cudaSuccess &&
            qr == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    }
    return fn;
}
// [rows, cols], rows `pitch` bytes apart, boxes of box_cols x box_rows, zeros past the end
bool map_2d(CUtensorMap* m, CUtensorMapDataType dt, const void* base, long long rows, int cols, int pitch, int box_cols,
            int box_rows, CUtensorMapSwizzle swz) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(m, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swz,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A cache [slots, pitch bytes] as [slots / 8][slabs][8 rows][128 bytes]: boxes of `rows` rows, all slabs
bool map_rows(CUtensorMap* m, CUtensorMapDataType dt, const void* base, long long slots, int pitch, int slab, int slabs, int rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[4] = {static_cast<cuuint64_t>(slab), 8u, static_cast<cuuint64_t>(slabs), static_cast<cuuint64_t>(slots / 8)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(pitch), 128u, static_cast<cuuint64_t>(pitch) * 8};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(slab), 8u, static_cast<cuuint32_t>(slabs), static_cast<cuuint32_t>(rows / 8)};
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    return fn(m, dt, 4, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sm_count() {
    static int count[kMaxDevicesAttr] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return 0;
    if (!count[dev] && cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return count[dev];
}

template <int R, bool E4M3, bool TREE>
int launch_decode_shape(const LatMaps& maps, const LatArgs& a, cudaStream_t stream) {
    using Sh = LatShape<R, E4M3>;
    constexpr uint32_t bytes = Sh::kBytes + (TREE ? R * 8u + 5u * kMaxNeed<E4M3> : 0u);
    static bool attr_done[kMaxDevicesAttr] = {};
    if (!raise_smem_limit(reinterpret_cast<const void*>(kda_latent_decode_kernel<R, E4M3, TREE>), static_cast<int>(bytes), attr_done))
        return -3;
    kda_latent_decode_kernel<R, E4M3, TREE><<<static_cast<unsigned>(a.w.G) * a.RT, Sh::kThreads, bytes, stream>>>(maps, a);
    if (cudaGetLastError() != cudaSuccess) return -3;
    cudaLaunchConfig_t cfg = {};
    // a row's partials number about G / N + 1: few of them (many sequences), a warp a row; else
    // groups of threads with 8 of them each (4: 1 to 10 us more), a row's channels over 4 blocks where
    // rows are too few for a block on each SM (20 tokens of 48 rows each, 192 rows: 16.5 us with 4, 15.3
    // with 1; 24 rows over 33851 tokens: 19.8 with 4, 27.4 with 1 and a pass each for maxima, sums and O)
    const int seqs = a.w.N / a.w.each, about = a.w.G / a.w.N + 1;
    const bool by_warp = about <= 16 || a.cuts;
    // (of the cut sequences, where those are what is joined: G at most)
    const long long warps = a.cuts ? static_cast<long long>(a.w.G) * (a.w.each > 1 ? R : a.rows) : static_cast<long long>(seqs) * a.rows;
    const int Q = static_cast<long long>(seqs) * a.rows < sm_count() ? 4 : 1;
    int NG = 1;
    while (NG < 4 * Q && NG * 8 < about) NG *= 2;
    cfg.gridDim = dim3(by_warp ? static_cast<unsigned>((warps + 3) / 4) : static_cast<unsigned>(seqs) * a.rows * Q);
    cfg.blockDim = dim3(by_warp ? 128 : 128 / Q * NG);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    if (a.cuts) return cudaLaunchKernelEx(&cfg, kda_latent_combine_rows_kernel<R, true, TREE>, a) == cudaSuccess ? 0 : -3;
    if (by_warp) return cudaLaunchKernelEx(&cfg, kda_latent_combine_rows_kernel<R, false, TREE>, a) == cudaSuccess ? 0 : -3;
    return cudaLaunchKernelEx(&cfg, kda_latent_combine_kernel<R, TREE>, a, Q, NG) == cudaSuccess ? 0 : -3;
}

template <bool TREE>
int launch_decode_rows(int R, int e4m3, const LatMaps& maps, const LatArgs& a, cudaStream_t stream) {
    if (e4m3) return R == 16 ? launch_decode_shape<16, true, TREE>(maps, a, stream)
                   : R == 32 ? launch_decode_shape<32, true, TREE>(maps, a, stream) : launch_decode_shape<64, true, TREE>(maps, a, stream);
    return R == 16 ? launch_decode_shape<16, false, TREE>(maps, a, stream)
         : R == 32 ? launch_decode_shape<32, false, TREE>(maps, a, stream) : launch_decode_shape<64, false, TREE>(maps, a, stream);
}

// Rows a CTA takes: 16, 32 or 64.
int rows_per_cta(int rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
}  // namespace

// Runs of tiles (times row tiles: one CTA per SM) and the scratch bytes of their partials.
int latent_decode_runs(int rows) {
    const int R = rows_per_cta(rows), RT = (rows + R - 1) / R, sms = sm_count();
    const int G = sms / RT > 0 ? sms / RT : (sms > 0 ? 1 : 0);
    return G < kMaxRuns ? G : kMaxRuns;
}
// A tree's row tiles as sequences of their own: one run a CTA (see the work split).  Two of a bf16 cache stay together: where
// some of the second are left out, what the first have read has left L2 (16 trees of 2 to 4 nodes x 32 heads over 341k
// tokens: apart 141 us, together 128; e4m3, apart: 122, chains of 4, all of whose rows are there: 127).
static bool tree_split(int rows, bool tree, int e4m3) { return tree && rows > (e4m3 ? 64 : 128); }
// Few sequences every warp of the joining kernel counts itself, while the attention runs; of many sequences and rows it is told
// which are cut, and looks at those alone (512 chains of 8 x 32 rows over 200 tokens, e4m3: 345 -> 216 us; 64 of 16 x 32 over
// 2000: 211 -> 204; but 64 of 1 x 32 over 1k to 64k, bf16: 188.3 -> 189.0).
static bool join_cuts(int N, int rows, bool apart) {
    return N > 32 && (apart || N > 128 || static_cast<long long>(N) * rows > 8192);
}
size_t latent_decode_scratch(int rows, int N, bool tree, int e4m3) {
    const size_t R = rows_per_cta(rows), RT = (rows + R - 1) / R;
    const bool apart = tree_split(rows, tree, e4m3);
    const size_t runs = apart ? latent_decode_runs(64) : latent_decode_runs(rows) * RT;
    return runs * 2 * R * (kLatDim + 2) * sizeof(float) + (join_cuts(N, rows, apart) ? latent_decode_runs(apart ? 64 : rows) * sizeof(LatCut) : 0);
}

int launch_latent_decode(const uint16_t* q, const void* cache, int e4m3, int num_pages, int page_size,
                         const int32_t* table, int max_pages, const int32_t* seq_lens, const int32_t* parents, int N, int K,
                         int H, float sm_scale, uint16_t* out, float* lse, void* scratch, int* status, cudaStream_t stream)
{
    LatArgs a = {};
    const int rows = K * H, R = rows_per_cta(rows);
    // (a segment's start and end in tiles: the best of 1, 2, 3, 4, 6 and of 4, 6, 8, 10, where Q is split too)
    const bool apart = tree_split(rows, parents != nullptr, e4m3);
    const int each = apart ? (rows + R - 1) / R : 1;
    a.w = LatWork{seq_lens, N * each, latent_decode_runs(apart ? 64 : rows), N * each == 1 ? 0 : e4m3 && R == 64 ? 8 : 2, parents ? K : 0,
                  static_cast<long long>(max_pages) * page_size, each, e4m3 ? kMaxNeed<true> : kMaxNeed<false>, nullptr, nullptr};
    if (a.w.G <= 0) return -3;
    a.ch = LatentCache{static_cast<const uint8_t*>(cache), table, num_pages, page_size, max_pages};
    a.q = q;
    a.parents = parents;
    a.K = K;
    a.H = H;
    a.rows = rows;
    a.RT = apart ? 1 : (rows + R - 1) / R;
    a.box = page_size % 64 == 0 ? 64 : page_size % 32 == 0 ? 32 : 16;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.lse = lse;
    a.part_o = static_cast<float*>(scratch);
    a.part_ml = a.part_o + static_cast<size_t>(a.w.G) * a.RT * 2 * R * kLatDim;
    if (join_cuts(N, rows, apart)) a.cuts = reinterpret_cast<LatCut*>(a.part_ml + static_cast<size_t>(a.w.G) * a.RT * 2 * R * 2);
    a.status = status;
    LatMaps maps;
    const CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B;
    const long long slots = static_cast<long long>(num_pages) * page_size;
    if (!map_2d(&maps.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, static_cast<long long>(N) * rows, kLatQ, kLatQ * 2, 64, R, swz))
        return -3;
    // (an empty cache holds no token to read; the map then only has to be valid)
    if (num_pages == 0) a.w.max_len = 0;
    maps.c = maps.s = maps.q;
    if (num_pages > 0 && !e4m3 &&
        !map_rows(&maps.c, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cache, slots, kLatRowBf16, 64, 9, a.box))
        return -3;
    if (num_pages > 0 && e4m3 &&
        (!map_rows(&maps.c, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, slots, kLatRowE4m3, 128, 5, a.box) ||
         !map_2d(&maps.s, CU_TENSOR_MAP_DATA_TYPE_UINT8, cache, slots, kLatRowE4m3, kLatRowE4m3, 16, a.box,
                 CU_TENSOR_MAP_SWIZZLE_NONE)))
        return -3;
    return parents ? launch_decode_rows<true>(R, e4m3, maps, a, stream) : launch_decode_rows<false>(R, e4m3, maps, a, stream);
}

}  // namespace kda
