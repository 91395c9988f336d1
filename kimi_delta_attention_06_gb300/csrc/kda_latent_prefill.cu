// kda_latent_prefill.cu -- expanded latent attention over packed prompts: per head keys
// [k (128), r (64, shared by the heads)] and values v (128).
//
// Row (i, h): x_t = scale * (q[:128] . k_t + q[128:] . r_t) over the keys the query sees,
// out = sum_t softmax(x)_t v_t, with the running maximum and sum of one pass.
//
// A CTA takes one head and 256 query rows, as two tiles of 128 that take turns: while the tensor
// cores work for one tile, the other's softmax runs.  Per tile of 128 keys
//     S [128 x 128]  = Q [128 x 192] [K, r]^T          (M = N = 128; Q, K, r from shared memory)
//     O [128 x 128] += P [128 x 128] V                 (P from TMEM, where it replaces S)
// S, P and O stay in TMEM (2 x 128 + 2 x 128 columns: all of it); a softmax thread owns one row.
// Keys and values pass through a ring of eight 16 KB slabs (64 channels x 128 keys), K's two, r's
// one and V's two a tile, in the order in which the products use and free them.
//
// Bound by the tensor cores and, in long runs, by the power limit of the card: 32 heads, causal, 8192
// tokens take 393 us in a graph (1750 TFLOP/s; a plain matrix product reaches 1900 for moments and holds
// 1730 for seconds), 2048 tokens after 32768 cached ones 852 us (1660 TFLOP/s: 256 CTAs on 152 SMs).  One
// thread issues all products: with one warp a query tile the two tiles' products interleaved instead of
// taking turns (518 -> 586 us, against 451 with one thread).
//
// Few queries over many keys: the keys are split over CTAs, whose partial (m, l, O) a second kernel joins
// (see expanded_span).
#include <cuda.h>
#include "latent.cuh"
#include "tc.cuh"

namespace kda {

constexpr int kExpK = 128, kExpV = 128, kExpQ = kExpK + kLatRope;

// Rows that see nothing (no keys at all): zeros and -inf.
__global__ void __launch_bounds__(256)
kda_expanded_empty_kernel(long long rows, uint16_t* __restrict__ out, float* __restrict__ lse)
{
    const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;       // 16 bytes each
    if (i >= rows * (kExpV / 8)) return;
    reinterpret_cast<uint4*>(out)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (lse && i < rows) lse[i] = -INFINITY;
}

struct ExpMaps { CUtensorMap q, k, v, r; };      // 64-channel x 128-row boxes, 128-byte swizzle

struct ExpArgs {
    const uint16_t* v;                           // values, as for the maps
    long long ldv, hdv;
    int total_k;
    const int32_t *cu_q, *cu_k;
    int num_seqs, H, causal, hg;                 // hg: heads that go side by side
    float scale_log2;
    uint16_t* out;
    float* lse;
    int* status;
    // split keys: part z takes key tiles [z span, (z + 1) span); partials [part][head][32 x 4 channels][query] of O
    // and [part][head][query] of (m, l), so that a warp's rows are next to each other
    int span, parts, total_q;
    float4* part_o;
    float2* part_ml;
};

constexpr int kExpTile = 128;                    // rows of a query tile, keys of a key tile
constexpr int kExpRows = 2 * kExpTile;           // query rows a CTA
constexpr uint32_t kSlab = kExpTile * 128u;      // 64 channels x 128 rows of bf16
constexpr uint32_t kRing = 8;
constexpr int kExpCopyWarp = 9;
constexpr int kExpThreads = 320;                 // warps 0-3, 4-7: softmax of tile 0, 1; 8: products; 9: copies
constexpr uint32_t kExpBars = 20;                // barriers of a pass
constexpr uint32_t oExpQ = 0, oExpRing = 6 * kSlab, oExpBar = oExpRing + kRing * kSlab, oExpFirst = oExpBar + 2 * kExpBars * 8 + 16;
constexpr uint32_t kExpSmem = oExpFirst + 3 * kExpV * 4 + 16;
static_assert(kExpSmem <= 232448, "227 KB of shared memory");
// Key tiles that query rows [r0, r0 + 128) of a sequence see.
__device__ __forceinline__ int exp_tiles(int r0, int Lq, int Lk, int causal) {
    const int r1 = min(r0 + kExpTile, Lq) - 1;
    const int see = r0 >= Lq ? 0 : causal ? r1 + 1 + Lk - Lq : Lk;
    return see > 0 ? (see + kExpTile - 1) / kExpTile : 0;
}
constexpr float kExpTau = 8.f;                   // scores may exceed the running maximum by 2^8 before a rescale

// A row has zeros in P for the keys that it does not see, but 0 * NaN is none: in a tile of keys that some rows see and
// others do not (the diagonal, and a sequence's last tile, which the next one's keys share), a value that is NaN or
// infinite spoils the rows that do not see it.  So such values leave these tiles before the product; for each channel the
// first key with a NaN, an infinity and a negative infinity is kept, and the rows that see past it get it into their
// results (CAREFUL below).  Looking the tiles over costs the kernel with split keys nothing (2048 queries x 8 heads over 18432
// keys 127 us, as without); the one with whole keys, whose softmax loop is out of registers, 4 to 10 % (8192 tokens x 32
// heads 389 -> 412 us, behind a call; by two warps more, as the values come too late for them, 430).  That one looks where a
// row's results are no numbers beside a sum of weights that is one, and where there are such values in those tiles, the CTA
// takes its rows a second time.  (A row computed again by a warp over its keys, as was done at first, took 0.3 us a key.)
__device__ __noinline__ void drop_nonfinite(uint4* p, uint4 v, int key, int* first, volatile int* any) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t at = 16 * (i & 1), bits = w[i >> 1] >> at & 0xffffu;
        if ((bits & 0x7f80u) != 0x7f80u) continue;
        atomicMin(first + (bits & 0x7fu ? 0 : bits >> 15 ? 2 * kExpV : kExpV) + i, key);
        w[i >> 1] &= ~(0xffffu << at);
    }
    *any = 1;
    __threadfence_block();                       // the other query tile's threads see the marks once they see the zeros
    *p = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ bool any_nonfinite(uint4 v) {         // of eight bf16 values
    const uint32_t top = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                  __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return top >= 0x7f800000u || (top & 0xffffu) >= 0x7f80u;
}
// Keys [from, 128) of a tile of values in slabs lo (channels 0 .. 63) and hi, by the 128 threads of a query tile.
__device__ __noinline__ void clean_tile(uint8_t* lo, uint8_t* hi, int from, int key0, int* first) {
    volatile int* any = first + 3 * kExpV;
    bool found = false;
    for (int x = threadIdx.x & 127; x < (kExpTile - from) * 16; x += kExpTile) {
        const int r = from + (x >> 4), c = x & 7;                // 16 bytes: 8 channels of a key
        uint4* p = reinterpret_cast<uint4*>((x & 8 ? hi : lo) + r * 128 + c * 16);
        const uint4 v = *p;
        if (any_nonfinite(v)) {
            drop_nonfinite(p, v, key0 + r, first + (x & 8) * 8 + ((c ^ (r & 7)) << 3), any);
            found = true;
        }
    }
    if (found || *any) tc::fence_smem_to_async();
}
// What the keys that a thread's row sees put into its results (O in TMEM): NaN, infinities or nothing.
__device__ __noinline__ void put_back(uint32_t tO, const int* first, int see) {
#pragma unroll 1
    for (int c = 0; c < kExpV; c += 16) {
        float o[16];
        tc::tmem_ld16(tO + c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int* f = first + c + i;
            const bool none = see > f[0], pos = see > f[kExpV], neg = see > f[2 * kExpV];
            o[i] += none || (pos && neg) ? __int_as_float(0x7fffffff) : pos ? INFINITY : neg ? -INFINITY : 0.f;
        }
        tc::tmem_st16(tO + c, o);
    }
    tc::tmem_wait_st();
}

__device__ __forceinline__ void clear_marks(uint8_t* smem) {     // [3][channels] and a flag, by the whole CTA
    int* first = reinterpret_cast<int*>(smem + oExpFirst);
    for (int i = threadIdx.x; i < 3 * kExpV + 1; i += kExpThreads) first[i] = i < 3 * kExpV ? 0x7fffffff : 0;
}

// What a CTA works on: rows [q0, q0 + 256) of head h of a sequence (its queries from cq on, its keys from ck on) over the
// key tiles from j0 on, nt[w] for query tile w; cut[w]: tile w has more parts than this one.
struct ExpUnit {
    int h, cq, q0, Lq, Lk, ck, more, part, j0, nmax;
    int nt[2];
    bool cut[2];
};

// The barriers of a pass and its copies (by one thread).
struct ExpCopies {
    const ExpMaps& maps;
    const ExpUnit& u;
    uint64_t *full, *q_full;
    uint32_t ring, sq;
    __device__ __forceinline__ ExpCopies(const ExpMaps& m, const ExpUnit& unit, uint8_t* smem, uint64_t* bars)
        : maps(m), u(unit), full(bars), q_full(bars + 18), ring(tc::smem_u32(smem + oExpRing)), sq(tc::smem_u32(smem + oExpQ)) {}
    __device__ __forceinline__ void q(int w) const {
        if (u.nt[w] == 0) return;
        tc::mbar_arrive_expect_tx(&q_full[w], 3u * kSlab);
        for (int s = 0; s < 3; ++s)
            tc::tma_load_3d(sq + (w * 3u + s) * kSlab, &maps.q, 64 * s, u.h, u.cq + u.q0 + w * kExpTile, &q_full[w]);
    }
    __device__ __forceinline__ void kv(uint32_t i, int j, int s) const {   // slab s of key tile j, the i-th of all, to slot i % 8
        const uint32_t slot = i & (kRing - 1), dst = ring + slot * kSlab;
        const int key = u.ck + (u.j0 + j) * kExpTile;
        tc::mbar_arrive_expect_tx(&full[slot], kSlab);
        if (s < 2) tc::tma_load_3d(dst, &maps.k, 64 * s, u.h, key, &full[slot]);
        else if (s == 2) tc::tma_load_2d(dst, &maps.r, 0, key, &full[slot]);
        else tc::tma_load_3d(dst, &maps.v, 64 * (s - 3), u.h, key, &full[slot]);
    }
    __device__ __forceinline__ void start() const {
        uint64_t* bars = full;
        for (uint32_t i = 0; i < kRing; ++i) tc::mbar_init(&full[i], 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bars[8 + i], 1);                      // kfree, vfree, s_full
            tc::mbar_init(&bars[10 + i], 1);
            tc::mbar_init(&bars[12 + i], 1);
            tc::mbar_init(&bars[14 + 2 * i], kExpTile);          // p_full
            tc::mbar_init(&bars[15 + 2 * i], kExpTile);
            tc::mbar_init(&q_full[i], 1);
        }
        tc::mbar_fence_init();
        // the first copies go out before the CTA meets, in the order in which they are used
        if (u.nmax > 0) {
            q(0);
            for (int s = 0; s < 3; ++s) kv(s, 0, s);
            q(1);
            for (int s = 3; s < 5; ++s) kv(s, 0, s);
        }
    }
};

// One pass over the unit by all warps.  `bad`: a row of this thread has results that are no numbers beside a sum that is one.
// CAREFUL: see drop_nonfinite.
template <bool SPLIT, bool CAREFUL>
__device__ __forceinline__ void run_unit(const ExpMaps& maps, const ExpArgs& a, const ExpUnit& u, uint8_t* smem, uint64_t* bars,
                                         uint32_t tm, bool& ok, bool& bad)
{
    uint64_t *full = bars, *kfree = bars + 8, *vfree = bars + 10, *s_full = bars + 12, *p_full = bars + 14, *q_full = bars + 18;
    int* s_first = reinterpret_cast<int*>(smem + oExpFirst);     // [3][channels], then a flag
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = u.h, cq = u.cq, q0 = u.q0, Lq = u.Lq, Lk = u.Lk, more = u.more, part = u.part, j0 = u.j0, nmax = u.nmax;
    const int nt[2] = {u.nt[0], u.nt[1]};
    const bool cut[2] = {u.cut[0], u.cut[1]};
    const ExpCopies copies(maps, u, smem, bars);

    if (warp < 8) {
        // ---- softmax: one row a thread ----
        const int w = warp >> 2, row = q0 + w * kExpTile + (tid & 127);
        const uint32_t lane_tm = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tm + w * 128u + lane_tm, tO = tm + 256u + w * 128u + lane_tm;
        const int see = (a.causal ? row + more : Lk) - j0 * kExpTile;
        const int all = (a.causal ? q0 + w * kExpTile + more : Lk) - j0 * kExpTile;   // keys that every row sees
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < nt[w]; ++j) {
            if (CAREFUL && all < (j + 1) * kExpTile) {
                const uint32_t i = 5u * j + 3u, s0 = i & (kRing - 1), s1 = (i + 1u) & (kRing - 1);
                ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&full[s0], (i / kRing) & 1, kWaitLimitNs) &&
                                                 tc::mbar_wait_bounded(&full[s1], ((i + 1u) / kRing) & 1, kWaitLimitNs));
                if (!ok) break;
                clean_tile(smem + oExpRing + s0 * kSlab, smem + oExpRing + s1 * kSlab, max(all - j * kExpTile, 0),
                           (j0 + j) * kExpTile, s_first);
            }
            ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&s_full[w], j & 1, kWaitLimitNs));
            if (!ok) break;
            tc::fence_after_sync();
            uint32_t u[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc::tmem_ld32x(tS + 32u * c, u[c]);
            tc::tmem_wait_ld();
            const int vis = see - j * kExpTile;                  // columns of this tile that the row sees
            // mx = the largest score; p = exp2(u * by - ref) below
            float mx = -INFINITY, by = a.scale_log2;
            if (__any_sync(0xffffffffu, vis < kExpTile)) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float x = 32 * c + i < vis ? __uint_as_float(u[c][i]) * a.scale_log2 : -INFINITY;
                        u[c][i] = __float_as_uint(x);
                        mx = fmaxf(mx, x);
                    }
                by = 1.f;
            } else if (a.scale_log2 >= 0.f) {
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx = fmaxf(mx, fmaxf(__uint_as_float(u[c][i]), __uint_as_float(u[c][i + 1])));
                mx *= by;
            } else {
                mx = INFINITY;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) mx = fminf(mx, fminf(__uint_as_float(u[c][i]), __uint_as_float(u[c][i + 1])));
                mx *= by;
            }
            if (__any_sync(0xffffffffu, mx > m + kExpTau)) {     // (the product before this tile's scores is in O)
                const float mn = fmaxf(m, mx);
                const float f = mn == m ? 1.f : lat_ex2(m - mn);
                m = mn;
                l *= f;
                if (j > 0) {
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) {
                        float o[16];
                        tc::tmem_ld16(tO + 16u * c, o);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] *= f;
                        tc::tmem_st16(tO + 16u * c, o);
                    }
                }
            }
            const float2 neg = make_float2(m == -INFINITY ? 0.f : -m, m == -INFINITY ? 0.f : -m), by2 = make_float2(by, by);
            float2 sum = make_float2(0.f, 0.f);
            uint32_t pk[32];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 x = ffma2(make_float2(__uint_as_float(u[c][2 * i]), __uint_as_float(u[c][2 * i + 1])), by2, neg);
                    const float2 p = make_float2(lat_ex2(x.x), lat_ex2(x.y));
                    sum = fadd2(sum, p);
                    pk[(c & 1) * 16 + i] = f32x2_to_bf16x2_bits(p.x, p.y);   // the sums keep fp32; the product takes bf16
                }
                if (c & 1) {                                     // 64 keys: the product takes each half as it comes
                    tc::tmem_st32x(tS + 16u * (c - 1), pk);
                    tc::tmem_wait_st();
                    tc::fence_before_sync();
                    tc::mbar_arrive(&p_full[2 * w + (c >> 1)]);
                }
            }
            l += sum.x + sum.y;
        }
        // ---- the tile's result: the last product is complete once s_full's next phase is ----
        if (ok && nt[w] > 0) {
            ok = __all_sync(0xffffffffu, tc::mbar_wait_bounded(&s_full[w], nt[w] & 1, kWaitLimitNs));
            tc::fence_after_sync();
        }
        if (CAREFUL && ok && nt[w] > 0 && *const_cast<volatile int*>(s_first + 3 * kExpV)) put_back(tO, s_first, see + j0 * kExpTile);
        float check = 0.f;                                       // NaN once a result is none or infinite
        if (SPLIT && cut[w]) {                                   // a part of the keys: to the joining kernel
            if (ok && nt[w] > 0) {
                const size_t ph = static_cast<size_t>(part) * a.H + h;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    uint32_t o[32];
                    tc::tmem_ld32x(tO + 32u * c, o);
                    tc::tmem_wait_ld();
                    if (row < Lq) {
                        float4* d = a.part_o + (ph * 32 + 8 * c) * a.total_q + cq + row;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            d[static_cast<size_t>(i) * a.total_q] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                                                __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    }
                }
                if (row < Lq) a.part_ml[ph * a.total_q + cq + row] = make_float2(m, l);
            }
        } else if (ok && part == 0 && q0 + w * kExpTile < Lq) {
            const bool mine = row < Lq;
            const long long at = (static_cast<long long>(cq) + row) * a.H + h;
            const bool some = nt[w] > 0 && l != 0.f;            // (else the row sees nothing: zeros)
            const float inv = 1.f / l;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t o[32];
                tc::tmem_ld32x(tO + 32u * c, o);
                tc::tmem_wait_ld();
                uint32_t pk[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x0 = __uint_as_float(o[2 * i]) * inv, x1 = __uint_as_float(o[2 * i + 1]) * inv;
                    check = fmaf(x1, 0.f, fmaf(x0, 0.f, check));
                    pk[i] = some ? f32x2_to_bf16x2_bits(x0, x1) : 0u;
                }
                if (mine) {
                    uint4* d = reinterpret_cast<uint4*>(a.out + at * kExpV + 32 * c);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[i] = make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
                }
            }
            if (mine && a.lse) a.lse[at] = (m + log2f(l)) * 0.69314718055994531f;     // nothing seen: -inf
        }
        // (where the sum is none the row saw a NaN itself, in a key or in q)
        bad = !CAREFUL && row < Lq && l > 0.f && !(check == 0.f);
    } else if (warp == 8) {
        // ---- products, in the order PV 0, QK 0, PV 1, QK 1 of consecutive key tiles ----
        constexpr uint32_t id_s = tc::idesc(128, 128, tc::kFmtBF16, false, false);
        constexpr uint32_t id_o = tc::idesc(128, 64, tc::kFmtBF16, false, true), id_o2 = tc::idesc(128, 128, tc::kFmtBF16, false, true);
        const uint64_t d0 = tc::sdesc(0, 16, 1024, tc::kSwizzle128B), dV = tc::sdesc(0, kSlab, 1024, tc::kSwizzle128B);
        const uint32_t hi = static_cast<uint32_t>(d0 >> 32);
        const uint32_t q_lo = static_cast<uint32_t>(d0) | (tc::smem_u32(smem + oExpQ) >> 4);
        const uint32_t k_lo = static_cast<uint32_t>(d0) | (tc::smem_u32(smem + oExpRing) >> 4);
        const uint32_t v_lo = static_cast<uint32_t>(dV) | (tc::smem_u32(smem + oExpRing) >> 4);
        // One thread runs it all: what stands between two products is then a barrier look or two (the
        // tensor cores queue only about two products, so every clock more is lost)
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            if (!tc::mbar_test_wait(bar, parity)) ok = tc::mbar_wait_bounded(bar, parity, kWaitLimitNs);
            return ok;
        };
        auto qk = [&](int w, int j) {                            // S_w = Q_w K_j^T
            const uint32_t q = q_lo + w * (3u * kSlab >> 4), d = tm + w * 128u;
#pragma unroll
            for (uint32_t s = 0; s < 3; ++s) {
                const uint32_t i = 5u * j + s, slot = i & (kRing - 1);
                if (!wait(&full[slot], (i / kRing) & 1)) return;
                const uint32_t b = k_lo + slot * (kSlab >> 4);
#pragma unroll
                for (uint32_t k = 0; k < 4; ++k)
                    tc::mma_f16_lo(d, q + (s * kSlab >> 4) + k * 2u, hi, b + k * 2u, hi, id_s, s > 0 || k > 0 ? 1u : 0u);
            }
            tc::mma_commit(&s_full[w]);
        };
        auto pv = [&](int w, int j) {                            // O_w += P_w V_j, half the keys at a time
            const uint32_t i = 5u * j + 3u, s0 = i & (kRing - 1), s1 = (i + 1u) & (kRing - 1);
            const uint32_t b0 = v_lo + s0 * (kSlab >> 4), b1 = v_lo + s1 * (kSlab >> 4);
            const uint32_t d = tm + 256u + w * 128u, p = tm + w * 128u, acc = j > 0 ? 1u : 0u;
            if (!wait(&full[s0], (i / kRing) & 1) || !wait(&full[s1], ((i + 1u) / kRing) & 1)) return;
#pragma unroll
            for (uint32_t half = 0; half < 2; ++half) {
                if (!wait(&p_full[2 * w + half], j & 1)) return;
                tc::fence_after_sync();
                if (s0 + 1u == s1) {                             // V's two slabs adjacent: all channels at once
#pragma unroll
                    for (uint32_t k = 4 * half; k < 4 * half + 4; ++k)
                        tc::mma_f16_ta(d, p + k * 8u, b0 + k * 128u, hi, id_o2, k > 0 ? 1u : acc);
                } else {                                         // (every eighth tile: the ring wraps between them)
#pragma unroll
                    for (uint32_t k = 4 * half; k < 4 * half + 4; ++k) {
                        tc::mma_f16_ta(d, p + k * 8u, b0 + k * 128u, hi, id_o, k > 0 ? 1u : acc);
                        tc::mma_f16_ta(d + 64u, p + k * 8u, b1 + k * 128u, hi, id_o, k > 0 ? 1u : acc);
                    }
                }
            }
        };
        if (tc::elect_one()) {
            for (int w = 0; w < 2; ++w)
                if (nt[w] > 0 && wait(&q_full[w], 0)) {
                    tc::fence_after_sync();
                    qk(w, 0);
                }
            if (ok && nmax > 0) tc::mma_commit(&kfree[0]);
            for (int j = 0; j < nmax && ok; ++j) {
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    if (j < nt[w] && ok) {
                        pv(w, j);
                        if (ok && j + 1 == nt[w]) tc::mma_commit(&s_full[w]);        // the tile's result
                    }
                    if (w == 1 && ok) tc::mma_commit(&vfree[j & 1]);
                    if (j + 1 < nt[w] && ok) qk(w, j + 1);
                }
                if (ok && j + 1 < nmax) tc::mma_commit(&kfree[(j + 1) & 1]);
            }
            // nothing is left running when the TMEM goes back
            if (ok && nmax > 0) wait(&vfree[(nmax - 1) & 1], ((nmax - 1) >> 1) & 1);
        }
        __syncwarp();
    } else {
        // ---- copies ----
        if (lane == 0) {
            uint32_t i = nmax > 0 ? 5u : 0u;                     // slabs issued: 5 j + s goes to slot (5 j + s) % 8
            for (int j = 1; j < nmax && ok; ++j) {
#pragma unroll
                for (int s = 0; s < 5; ++s) {
                    // slab i - 8 leaves its slot first: V of tile j - 2 from s = 1 on, K and r of tile j - 1 from
                    // s = 3 on (s = 0 takes the last slab of K j - 2, waited for with the first)
                    if (s == 1 && j >= 2) ok = tc::mbar_wait_bounded(&vfree[j & 1], ((j - 2) >> 1) & 1, kWaitLimitNs);
                    if (s == 3) ok = tc::mbar_wait_bounded(&kfree[(j - 1) & 1], ((j - 1) >> 1) & 1, kWaitLimitNs);
                    if (!ok) break;
                    copies.kv(i++, j, s);
                }
            }
            if (!ok) {                                           // copies in flight land before the CTA ends
                for (int w = 0; w < 2; ++w)
                    if (nt[w] > 0) tc::mbar_wait_bounded(&q_full[w], 0, kWaitLimitNs);
                for (uint32_t x = i > kRing ? i - kRing : 0; x < i; ++x)
                    tc::mbar_wait_bounded(&full[x & (kRing - 1)], (x / kRing) & 1, kWaitLimitNs);
            }
        }
        __syncwarp();
    }
}

// A second pass of a CTA that had its rows' keys whole: its own barriers.
__device__ __noinline__ void run_unit_again(const ExpMaps& maps, const ExpArgs& a, const ExpUnit& u, uint8_t* smem, uint32_t tm) {
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + oExpBar) + kExpBars;
    // values that are NaN or infinite among the keys from the first that some row does not see to the end of the last tile
    // (what lies past all keys is copied as zeros)
    const int all = max(a.causal ? u.q0 + u.more : u.Lk, 0), end = min(u.nmax * kExpTile, a.total_k - u.ck);
    const uint16_t* v = a.v + static_cast<long long>(u.ck) * a.ldv + u.h * a.hdv;
    bool found = false;
    for (long long x = all * 16LL + threadIdx.x; x < end * 16LL; x += kExpThreads)
        found = found || any_nonfinite(*reinterpret_cast<const uint4*>(v + (x >> 4) * a.ldv + (x & 15) * 8));
    if (!__syncthreads_or(found)) return;
    clear_marks(smem);
    if (threadIdx.x == 32 * kExpCopyWarp) ExpCopies(maps, u, smem, bars).start();
    __syncthreads();
    tc::fence_after_sync();
    bool ok = true, bad;
    run_unit<false, true>(maps, a, u, smem, bars, tm, ok, bad);
    if (!ok) set_status(a.status, kStatusTimeout);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
}

template <bool SPLIT>
__global__ void __launch_bounds__(kExpThreads, 1)
kda_expanded_kernel(const __grid_constant__ ExpMaps maps, const __grid_constant__ ExpArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + oExpBar);
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 2 * kExpBars);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y * a.hg + blockIdx.x % a.hg;
    if (h >= a.H) return;                                        // (the last group's)
    // the unit (sequence n, 256 rows from q0): the last rows of a sequence, the longest, come first
    int n = 0, q0 = 0, cq = 0, Lq = 0;
    {
        int base = 0;
        const int want = static_cast<int>(blockIdx.x / a.hg);
        for (int i0 = 0; i0 < a.num_seqs; i0 += 32) {
            const int i = i0 + lane;
            const int c = i < a.num_seqs ? a.cu_q[i] : 0, len = i < a.num_seqs ? a.cu_q[i + 1] - c : 0;
            const int units = (len + kExpRows - 1) / kExpRows;
            int incl = units;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int o = __shfl_up_sync(0xffffffffu, incl, off);
                if (lane >= off) incl += o;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, base + incl > want);
            if (hit) {
                const int at = __ffs(hit) - 1;
                n = i0 + at;
                cq = __shfl_sync(0xffffffffu, c, at);
                Lq = __shfl_sync(0xffffffffu, len, at);
                q0 = (base + __shfl_sync(0xffffffffu, incl, at) - 1 - want) * kExpRows;
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    const int ck = a.cu_k[n], Lk = a.cu_k[n + 1] - ck;
    // keys that row i sees: i + more (causal), else all; key tiles of query tile w: nt[w]
    const int more = a.causal ? 1 + Lk - Lq : Lk;
    int nt[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) nt[w] = exp_tiles(q0 + w * kExpTile, Lq, Lk, a.causal);
    const int part = SPLIT ? static_cast<int>(blockIdx.z) : 0, j0 = SPLIT ? part * a.span : 0;
    bool cut[2] = {false, false};                                // tile w has more parts than one
    if constexpr (SPLIT) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel waits for this grid's end
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            cut[w] = nt[w] > a.span;
            nt[w] = max(0, min(nt[w] - j0, a.span));
        }
    }
    const int nmax = max(nt[0], nt[1]);
    if (SPLIT && part > 0 && nmax == 0) return;                  // no such part
    const ExpUnit u{h, cq, q0, Lq, Lk, ck, more, part, j0, nmax, {nt[0], nt[1]}, {cut[0], cut[1]}};
    if (tid == 32 * kExpCopyWarp) ExpCopies(maps, u, smem, bars).start();
    if (SPLIT) clear_marks(smem);
    __syncwarp();
    if (warp == 8) tc::tmem_alloc(s_tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *s_tmem;
    bool ok = true, bad = false;

    run_unit<SPLIT, SPLIT>(maps, a, u, smem, bars, tm, ok, bad);
    if (!ok) set_status(a.status, kStatusTimeout);
    __syncwarp();
    tc::fence_before_sync();
    const bool again = __syncthreads_or(bad);
    tc::fence_after_sync();
    if (!SPLIT && again && __syncthreads_and(ok)) run_unit_again(maps, a, u, smem, tm);
    if (warp == 8) tc::tmem_dealloc(tm, 512);
}

// Joins the parts of rows whose keys were split: 8 rows a block, 4 channels a thread, one pass over the
// parts with the running maximum, B parts' loads in flight.
template <int B>
__global__ void __launch_bounds__(256)
kda_expanded_join_kernel(const ExpArgs a)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
    const int row = blockIdx.x * 8 + (lane & 7), c4 = warp * 4 + (lane >> 3);     // query of all sequences, channels 4 c4 ..
    int parts = 0;
    if (row < a.total_q) {
        int lo = 0, hi = a.num_seqs;                             // cu_q[lo] <= row < cu_q[lo + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.cu_q[mid] <= row) lo = mid; else hi = mid;
        }
        const int cq = a.cu_q[lo], Lq = a.cu_q[lo + 1] - cq, Lk = a.cu_k[lo + 1] - a.cu_k[lo], in = row - cq;
        const int nt = exp_tiles(in / kExpTile * kExpTile, Lq, Lk, a.causal);
        parts = nt > a.span ? min((nt + a.span - 1) / a.span, a.parts) : 0;
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");          // every block: this grid ends after the one before it
    const size_t step = static_cast<size_t>(a.H) * a.total_q;
    const float2* ml = a.part_ml + static_cast<size_t>(h) * a.total_q + row;
    const float4* o = a.part_o + (static_cast<size_t>(h) * 32 + c4) * a.total_q + row;
    float M = -INFINITY, L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p0 = 0; p0 < parts; p0 += B) {
        float2 v[B];
        float4 x[B];
        float mx = M;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const bool in = p0 + i < parts;
            v[i] = in ? ml[(p0 + i) * step] : make_float2(-INFINITY, 0.f);
            x[i] = in ? o[(p0 + i) * 32 * step] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int i = 0; i < B; ++i) mx = fmaxf(mx, v[i].x);
        const float f = mx == M ? 1.f : lat_ex2(M - mx);
        M = mx;
        L *= f;
        acc.x *= f; acc.y *= f; acc.z *= f; acc.w *= f;
#pragma unroll
        for (int i = 0; i < B; ++i) {
            if (v[i].x == -INFINITY && v[i].y == 0.f) continue;  // sees nothing there
            const float w = v[i].x == M ? 1.f : lat_ex2(v[i].x - M);
            L += w * v[i].y;
            acc.x += w * x[i].x; acc.y += w * x[i].y; acc.z += w * x[i].z; acc.w += w * x[i].w;
        }
    }
    if (parts > 0) {
        const size_t at = static_cast<size_t>(row) * a.H + h;
        const float inv = L == 0.f ? 0.f : 1.f / L;
        *reinterpret_cast<uint2*>(a.out + at * kExpV + 4 * c4) = make_uint2(f32x2_to_bf16x2_bits(acc.x * inv, acc.y * inv),
                                                                            f32x2_to_bf16x2_bits(acc.z * inv, acc.w * inv));
        if (c4 == 0 && a.lse) a.lse[at] = (M + log2f(L)) * 0.69314718055994531f;
    }
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
// bf16 [tokens][heads][channels] (heads = 0: [tokens][channels]), strides in elements; boxes of 64
// channels x 1 head x 128 tokens, 128-byte swizzle, zeros past the end
bool map_tokens(CUtensorMap* m, const void* base, long long tokens, int heads, int channels, long long token_stride,
                long long head_stride) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const bool three = heads > 0;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(three ? heads : tokens),
                                static_cast<cuuint64_t>(tokens)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(three ? head_stride : token_stride) * 2,
                                   static_cast<cuuint64_t>(token_stride) * 2};
    const cuuint32_t box[3] = {64u, three ? 1u : static_cast<cuuint32_t>(kExpTile), static_cast<cuuint32_t>(kExpTile)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, three ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int exp_sm_count() {
    static int count[kMaxDevicesAttr] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return 0;
    if (!count[dev] && cudaDeviceGetAttribute(&count[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return count[dev];
}
constexpr int kExpMinSpan = 4, kExpWorth = 8, kExpMaxSms = 256;
}  // namespace

// Scratch of `parts` parts of every row.
size_t expanded_scratch(long long parts, int H, int total_q) {
    return static_cast<size_t>(parts) * H * total_q * (kExpV + 2) * sizeof(float);
}

// Key tiles a part, 0 = whole.  The CTAs (256 queries of one head each) of a few queries over many
// keys leave most SMs idle, and each takes its keys in series, 1.5 us a tile of 128.  So where they
// are fewer than two for each SM, the keys are split so that all parts together are about one for each SM:
// 256 queries x 4 heads over 33024 keys 393 -> 31 us, 16 x 1 over 12016 134 -> 13.5, 2048 x 8 over 18432
// 223 -> 131, one prompt of 4000 x 4 heads 54 -> 29.
// A split costs a scratch allocation and a second launch: called from Python, 2000 queries x 4 heads (16
// tiles) go from 31 to 22 us, 1300 (11) stay at 22, 1000 (8) go from 18 to 22.  So it is made where it
// takes 8 tiles or more out of the longest series.
int expanded_span(const int32_t* cu_q, const int32_t* cu_k, int num_seqs, int H, int causal, int total_q, int units,
                  int* parts) {
    const int sms = exp_sm_count();
    *parts = 1;
    if (sms == 0 || sms > kExpMaxSms || static_cast<long long>(units) * H >= 2LL * sms) return 0;
    int nt[2 * kExpMaxSms], used = 0, longest = 0;               // key tiles of the units
    long long sum = 0;
    for (int n = 0; n < num_seqs; ++n) {
        const int Lq = cu_q[n + 1] - cu_q[n], Lk = cu_k[n + 1] - cu_k[n];
        for (int r = 0; r < Lq; r += kExpRows) {
            const int see = causal ? (r + kExpRows < Lq ? r + kExpRows : Lq) + Lk - Lq : Lk;
            nt[used] = see > 0 ? (see + kExpTile - 1) / kExpTile : 0;
            sum += nt[used];
            longest = nt[used] > longest ? nt[used] : longest;
            ++used;
        }
    }
    const long long most = units * static_cast<long long>(H) <= sms ? sms : 2LL * sms;
    long long span = (sum * H + sms - 1) / sms;
    if (span < kExpMinSpan) span = kExpMinSpan;
    for (; span < longest; span += span / 8 + 1) {               // the parts all run at once, in 256 MB of partials at most
        long long ctas = 0;
        for (int i = 0; i < used; ++i) ctas += nt[i] > span ? (nt[i] + span - 1) / span : 1;
        if (ctas * H <= most && expanded_scratch((longest + span - 1) / span, H, total_q) <= (size_t{256} << 20)) break;
    }
    if (longest - span < kExpWorth) return 0;
    *parts = static_cast<int>((longest + span - 1) / span);
    return static_cast<int>(span);
}

// units: sum over sequences of ceil(queries / 256); span: see above, with its scratch
int launch_latent_prefill(const uint16_t* q, const uint16_t* k, long long ldk, long long hdk, const uint16_t* v,
                          long long ldv, long long hdv, const uint16_t* r, long long ldr, const int32_t* cu_q,
                          const int32_t* cu_k, int num_seqs, int total_q, int total_k, int units, int H, int causal,
                          float sm_scale, uint16_t* out, float* lse, int span, int parts, void* scratch, int* status,
                          cudaStream_t stream)
{
    if (total_k == 0) {
        const long long rows = static_cast<long long>(total_q) * H;
        kda_expanded_empty_kernel<<<static_cast<unsigned>((rows * (kExpV / 8) + 255) / 256), 256, 0, stream>>>(rows, out, lse);
        return cudaGetLastError() == cudaSuccess ? 0 : -3;
    }
    ExpMaps maps;
    if (!map_tokens(&maps.q, q, total_q, H, kExpQ, static_cast<long long>(H) * kExpQ, kExpQ) ||
        !map_tokens(&maps.k, k, total_k, H, kExpK, ldk, hdk) || !map_tokens(&maps.v, v, total_k, H, kExpV, ldv, hdv) ||
        !map_tokens(&maps.r, r, total_k, 0, kLatRope, ldr, 0))
        return -3;
    ExpArgs a = {};
    a.v = v;
    a.ldv = ldv;
    a.hdv = hdv;
    a.total_k = total_k;
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.num_seqs = num_seqs;
    a.H = H;
    a.causal = causal;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.lse = lse;
    a.status = status;
    // A prompt's last queries have the most keys and come first, of some heads side by side, so that short
    // units fill the end: 8192 tokens x 32 heads 441 -> 393 us with 8 heads (401 with 16), 2000 x 32 54.7 ->
    // 41.2 with 16 (49.9 with 8), 16384 x 32 1550 -> 1479 with 4 or 8 (1516 with 16).  The heads' keys and
    // values are to stay in L2: less than 64 MB.  Behind long prefixes the units are much alike, and a head's
    // go together (2048 queries over 18432 keys, 8 heads: 128 us so, 148 side by side).
    a.hg = 1;
    if (causal && total_k < 2LL * total_q)
        while (a.hg < 16 && 2 * a.hg <= H && total_k * 2LL * a.hg * (kExpK + kExpV) * 2 < (64 << 20)) a.hg *= 2;
    const dim3 grid(static_cast<unsigned>(units) * a.hg, static_cast<unsigned>((H + a.hg - 1) / a.hg), static_cast<unsigned>(parts));
    if (span == 0) {
        static bool attr_done[kMaxDevicesAttr] = {};
        if (!raise_smem_limit(reinterpret_cast<const void*>(kda_expanded_kernel<false>), static_cast<int>(kExpSmem), attr_done)) return -3;
        kda_expanded_kernel<false><<<grid, kExpThreads, kExpSmem, stream>>>(maps, a);
        return cudaGetLastError() == cudaSuccess ? 0 : -3;
    }
    a.span = span;
    a.parts = parts;
    a.total_q = total_q;
    a.part_o = static_cast<float4*>(scratch);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(parts) * H * 32 * total_q);
    static bool attr_done[kMaxDevicesAttr] = {};
    if (!raise_smem_limit(reinterpret_cast<const void*>(kda_expanded_kernel<true>), static_cast<int>(kExpSmem), attr_done)) return -3;
    kda_expanded_kernel<true><<<grid, kExpThreads, kExpSmem, stream>>>(maps, a);
    if (cudaGetLastError() != cudaSuccess) return -3;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((static_cast<unsigned>(total_q) + 7) / 8, static_cast<unsigned>(H));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    // (4 parts' loads at a time where there are no more: 2048 queries x 8 heads 131 -> 128 us)
    return cudaLaunchKernelEx(&cfg, parts <= 4 ? kda_expanded_join_kernel<4> : kda_expanded_join_kernel<8>, a) == cudaSuccess
               ? 0 : -3;
}

}  // namespace kda
