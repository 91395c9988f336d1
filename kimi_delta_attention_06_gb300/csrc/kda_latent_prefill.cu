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
// Bound by the power limit of the card: 32 heads, causal, 8192 tokens take 443 us (1550 TFLOP/s at
// 1370 W), 2048 tokens after 32768 cached ones 840 us (1690 TFLOP/s); a seconds-long plain matrix
// product holds 1727.  One thread issues all products: with one warp a query tile the two tiles'
// products interleaved instead of taking turns (518 -> 586 us, against 451 with one thread).
#include <cuda.h>
#include "latent.cuh"
#include "tc.cuh"

namespace kda {

constexpr int kExpK = 128, kExpV = 128, kExpQ = kExpK + kLatRope;

struct ExpKv {
    const uint16_t *k, *v, *r;
    long long ldk, hdk, ldv, hdv, ldr;
};

// One warp computes one row in fp32, straight from the formula, over keys [k0, k0 + see).  Lane i
// owns key and value channels 4 i .. 4 i + 3 and position values 2 i, 2 i + 1.
__device__ __noinline__ void expanded_row(const uint16_t* __restrict__ q, const ExpKv& kv, int h, long long k0, int see,
                             float scale_log2, uint16_t* __restrict__ out, float* __restrict__ lse)
{
    const int lane = threadIdx.x & 31;
    const uint2 qw = reinterpret_cast<const uint2*>(q)[lane];
    const float2 q0 = bf16x2_bits_to_f32(qw.x), q1 = bf16x2_bits_to_f32(qw.y);
    const float2 qr = bf16x2_bits_to_f32(reinterpret_cast<const uint32_t*>(q + kExpK)[lane]);
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int t = 0; t < see; ++t) {
        const long long at = k0 + t;
        const uint2 kw = reinterpret_cast<const uint2*>(kv.k + at * kv.ldk + h * kv.hdk)[lane];
        const float2 a = bf16x2_bits_to_f32(kw.x), b = bf16x2_bits_to_f32(kw.y);
        const float2 r = bf16x2_bits_to_f32(reinterpret_cast<const uint32_t*>(kv.r + at * kv.ldr)[lane]);
        float x = q0.x * a.x + q0.y * a.y + q1.x * b.x + q1.y * b.y + qr.x * r.x + qr.y * r.y;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        x *= scale_log2;
        if (x > m) {
            const float f = lat_ex2(m - x);
            m = x;
            l *= f;
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] *= f;
        }
        const float p = x == -INFINITY ? 0.f : lat_ex2(x - m);
        l += p;
        const uint2 vw = reinterpret_cast<const uint2*>(kv.v + at * kv.ldv + h * kv.hdv)[lane];
        const float2 c = bf16x2_bits_to_f32(vw.x), d = bf16x2_bits_to_f32(vw.y);
        acc[0] += p * c.x; acc[1] += p * c.y; acc[2] += p * d.x; acc[3] += p * d.y;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;      // (a NaN sum stays NaN)
    reinterpret_cast<uint2*>(out)[lane] = make_uint2(f32x2_to_bf16x2_bits(acc[0] * inv, acc[1] * inv),
                                                     f32x2_to_bf16x2_bits(acc[2] * inv, acc[3] * inv));
    if (lse && lane == 0) *lse = (m + log2f(l)) * 0.69314718055994531f;     // l = 0: -inf
}


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
    const uint16_t* q;
    ExpKv kv;
    const int32_t *cu_q, *cu_k;
    int num_seqs, H, causal;
    float scale_log2;
    uint16_t* out;
    float* lse;
    int* status;
};

constexpr int kExpTile = 128;                    // rows of a query tile, keys of a key tile
constexpr int kExpRows = 2 * kExpTile;           // query rows a CTA
constexpr uint32_t kSlab = kExpTile * 128u;      // 64 channels x 128 rows of bf16
constexpr uint32_t kRing = 8;
constexpr int kExpCopyWarp = 9;
constexpr int kExpThreads = 320;                 // warps 0-3, 4-7: softmax of tile 0, 1; 8: products; 9: copies
constexpr uint32_t oExpQ = 0, oExpRing = 6 * kSlab, oExpBar = oExpRing + kRing * kSlab;
constexpr uint32_t kExpSmem = oExpBar + 32 * 8 + 16;
constexpr float kExpTau = 8.f;                   // scores may exceed the running maximum by 2^8 before a rescale

__global__ void __launch_bounds__(kExpThreads, 1)
kda_expanded_kernel(const __grid_constant__ ExpMaps maps, const ExpArgs a)
{
    extern __shared__ __align__(1024) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + oExpBar);
    uint64_t *full = bars, *kfree = bars + 8, *vfree = bars + 10, *s_full = bars + 12, *p_full = bars + 14, *q_full = bars + 18;
    uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 20);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int h = blockIdx.y;
    // the unit (sequence n, 256 rows from q0): the last rows of a sequence, the longest, come first
    int n = 0, q0 = 0, cq = 0, Lq = 0;
    {
        int base = 0;
        const int want = static_cast<int>(blockIdx.x);
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
    for (int w = 0; w < 2; ++w) {
        const int r0 = q0 + w * kExpTile, r1 = min(r0 + kExpTile, Lq) - 1;        // its rows r0 .. r1
        const int see = r0 >= Lq ? 0 : a.causal ? r1 + more : Lk;
        nt[w] = see > 0 ? (see + kExpTile - 1) / kExpTile : 0;
    }
    const int nmax = max(nt[0], nt[1]);
    const uint32_t ring = tc::smem_u32(smem + oExpRing), sq = tc::smem_u32(smem + oExpQ);
    auto copy_q = [&](int w) {
        if (nt[w] == 0) return;
        tc::mbar_arrive_expect_tx(&q_full[w], 3u * kSlab);
        for (int s = 0; s < 3; ++s)
            tc::tma_load_3d(sq + (w * 3u + s) * kSlab, &maps.q, 64 * s, h, cq + q0 + w * kExpTile, &q_full[w]);
    };
    auto copy_kv = [&](uint32_t i, int j, int s) {               // slab s of key tile j, the i-th of all, to slot i % 8
        const uint32_t slot = i & (kRing - 1), dst = ring + slot * kSlab;
        const int key = ck + j * kExpTile;
        tc::mbar_arrive_expect_tx(&full[slot], kSlab);
        if (s < 2) tc::tma_load_3d(dst, &maps.k, 64 * s, h, key, &full[slot]);
        else if (s == 2) tc::tma_load_2d(dst, &maps.r, 0, key, &full[slot]);
        else tc::tma_load_3d(dst, &maps.v, 64 * (s - 3), h, key, &full[slot]);
    };

    if (tid == 32 * kExpCopyWarp) {
        for (uint32_t i = 0; i < kRing; ++i) tc::mbar_init(&full[i], 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&kfree[i], 1);
            tc::mbar_init(&vfree[i], 1);
            tc::mbar_init(&s_full[i], 1);
            tc::mbar_init(&p_full[2 * i], kExpTile);
            tc::mbar_init(&p_full[2 * i + 1], kExpTile);
            tc::mbar_init(&q_full[i], 1);
        }
        tc::mbar_fence_init();
        // the first copies go out before the CTA meets, in the order in which they are used
        if (nmax > 0) {
            copy_q(0);
            for (int s = 0; s < 3; ++s) copy_kv(s, 0, s);
            copy_q(1);
            for (int s = 3; s < 5; ++s) copy_kv(s, 0, s);
        }
    }
    __syncwarp();
    if (warp == 8) tc::tmem_alloc(s_tmem, 512);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tm = *s_tmem;
    bool ok = true;

    if (warp < 8) {
        // ---- softmax: one row a thread ----
        const int w = warp >> 2, row = q0 + w * kExpTile + (tid & 127);
        const uint32_t lane_tm = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tm + w * 128u + lane_tm, tO = tm + 256u + w * 128u + lane_tm;
        const int see = a.causal ? row + more : Lk;
        float m = -INFINITY, l = 0.f;
        for (int j = 0; j < nt[w]; ++j) {
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
        if (ok && q0 + w * kExpTile < Lq) {
            const bool mine = row < Lq;
            const long long at = (static_cast<long long>(cq) + row) * a.H + h;
            const bool some = nt[w] > 0 && l != 0.f;            // (else the row sees nothing: zeros)
            const float inv = 1.f / l;
            float check = 0.f;                                   // NaN once a value is none or infinite
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
            const bool bad = some && !(check == 0.f);
            if (mine && a.lse) a.lse[at] = (m + log2f(l)) * 0.69314718055994531f;     // nothing seen: -inf
            // a NaN or infinity in a key or value that other rows of the tile see spoils this row's sum
            // (0 * NaN): such a row is computed again over exactly its own keys
            unsigned again = __ballot_sync(0xffffffffu, mine && bad);
            while (again) {
                const int r = row - lane + __ffs(again) - 1;
                again &= again - 1;
                const long long ra = (static_cast<long long>(cq) + r) * a.H + h;
                expanded_row(a.q + ra * kExpQ, a.kv, h, ck, a.causal ? r + more : Lk, a.scale_log2, a.out + ra * kExpV,
                             a.lse ? a.lse + ra : nullptr);
            }
        }
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
                    copy_kv(i++, j, s);
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
    if (!ok) set_status(a.status, kStatusTimeout);
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 8) tc::tmem_dealloc(tm, 512);
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
}  // namespace

// units: sum over sequences of ceil(queries / 256)
int launch_latent_prefill(const uint16_t* q, const uint16_t* k, long long ldk, long long hdk, const uint16_t* v,
                          long long ldv, long long hdv, const uint16_t* r, long long ldr, const int32_t* cu_q,
                          const int32_t* cu_k, int num_seqs, int total_q, int total_k, int units, int H, int causal,
                          float sm_scale, uint16_t* out, float* lse, int* status, cudaStream_t stream)
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
    a.q = q;
    a.kv = ExpKv{k, v, r, ldk, hdk, ldv, hdv, ldr};
    a.cu_q = cu_q;
    a.cu_k = cu_k;
    a.num_seqs = num_seqs;
    a.H = H;
    a.causal = causal;
    a.scale_log2 = sm_scale * 1.4426950408889634f;
    a.out = out;
    a.lse = lse;
    a.status = status;
    static bool attr_done[kMaxDevicesAttr] = {};
    if (!raise_smem_limit(reinterpret_cast<const void*>(kda_expanded_kernel), static_cast<int>(kExpSmem), attr_done)) return -3;
    kda_expanded_kernel<<<dim3(static_cast<unsigned>(units), static_cast<unsigned>(H)), kExpThreads, kExpSmem, stream>>>(maps, a);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace kda
