// kda_cache.cu -- the latent cache as it is written (bf16, or e4m3 with one power-of-two scale a
// token) and read back.  Both kernels move bytes: one warp per token, 16-byte accesses, the
// token's row in registers once, so they are bound by HBM for long runs and by the launch for a
// decode step's few rows.  Measured, e4m3: 145408 tokens written in 42 us (6.2 TB/s of 6.7), 214k
// tokens in pages of 48 read back in 60 us (6.4 TB/s); 512 tokens written and read back 5.4 us.
#include "latent.cuh"

namespace kda {

constexpr int kCacheThreads = 256;

// A token's latents at src (32 lanes x 32 bytes) into its cache row.  Lane: 16 latents.  Returns the exponent of an e4m3 row's
// scale, which put_scale writes after the position part, so that a row is written from its first byte to its last (the scale
// before the position part: 145408 tokens with their read-back 85.8 us for 84.3).
template <bool E4M3>
__device__ __forceinline__ int put_latents(uint8_t* row, const uint4* src, int lane) {
    if constexpr (!E4M3) {
        uint4* dst = reinterpret_cast<uint4*>(row);
        const uint4 a = src[lane], b = src[lane + 32];
        dst[lane] = a;
        dst[lane + 32] = b;
        return 0;
    } else {
        // 16 latents of this lane: one 16-byte store of codes
        const uint4 a = src[2 * lane], b = src[2 * lane + 1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        float x[16];
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = bf16x2_bits_to_f32(w[i]);
            x[2 * i] = f.x; x[2 * i + 1] = f.y;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float m = fabsf(x[i]);
            const bool fin = m < __int_as_float(0x7f800000);          // false for NaN and infinities
            amax = fmaxf(amax, fin ? m : 0.f);
            x[i] = fin ? x[i] : __int_as_float(0x7fffffff);
        }
        amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));   // non-negative: bits order
        const int e = lat_scale_exponent(__float_as_uint(amax));
        const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);          // 2^-e: products are exact
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            o[i] = f32x2_to_e4m3x2(x[4 * i] * inv, x[4 * i + 1] * inv) |
                   (f32x2_to_e4m3x2(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
        reinterpret_cast<uint4*>(row)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
        return e;
    }
}
template <bool E4M3>
__device__ __forceinline__ void put_scale(uint8_t* row, int e, int lane) {
    if (E4M3 && lane < 4)
        reinterpret_cast<uint32_t*>(row + kLatScaleAt)[lane] = lane == 0 ? static_cast<uint32_t>(127 + e) << 23 : 0u;
}

// 16 consecutive latents per lane (32 bytes), 2 position values per lane.
template <bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
kda_latent_append_kernel(const uint16_t* __restrict__ c, long long ldc, const uint16_t* __restrict__ r, long long ldr,
                         uint8_t* __restrict__ cache, long long num_rows, const int32_t* __restrict__ slots, int T,
                         int* status)
{
    const int lane = threadIdx.x & 31;
    const long long t = static_cast<long long>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5);
    if (t >= T) return;
    const int slot = slots[t];
    const uint4* src = reinterpret_cast<const uint4*>(c + t * ldc);
    const uint32_t rope = reinterpret_cast<const uint32_t*>(r + t * ldr)[lane];
    if (slot < 0) return;
    if (slot >= num_rows) {
        if (lane == 0) set_status(status, kStatusIndex);
        return;
    }
    uint8_t* row = cache + static_cast<size_t>(slot) * lat_row_bytes(E4M3);
    const int e = put_latents<E4M3>(row, src, lane);
    reinterpret_cast<uint32_t*>(row + (E4M3 ? kLatDim : 2 * kLatDim))[lane] = rope;
    put_scale<E4M3>(row, e, lane);
}

// The same with the position parts rotated on the way: pair i of a key or query turns by pos * f_i,
//     (x, y) -> (x cos - y sin, x sin + y cos),
// with pairs of neighbours (2 i, 2 i + 1) or of the two halves (i, i + 32).  The angle matters modulo a turn, and
// pos * f rounded to 32 bits is off by 0.03 rad at pos = 10^6, so it is taken in fixed point: f / 2 pi as a 64-bit
// fraction of a turn (its whole turns vanish at whole positions), times pos modulo 2^64, is exact but for the
// fraction's own rounding, at most pos * 2^-63.
//
// A warp takes a token: lane i the angle of pair i, once; then 8 lanes a head, 4 pairs a lane, 16 heads in flight, the first
// of them on their way before the slot is known.  Bound by HBM: 32768 tokens of 32 heads, bf16, 55 us (6.2 TB/s; in another
// session 52, over e4m3 50); 768 of them, e4m3, 3.4 us, most of it the launch and two loads one after the other.  (Heads of a token over 2 warps: 56 and
// 3.2 us, over 4: 74 and 3.3.  The loads after the angle: 59 and 4.1.)
constexpr int kRopeThreads = 128;

// f / 2 pi modulo a turn, in units of 2^-64: 24 bits of f times 96 bits of 1 / 2 pi, moved to its place.  (|f| < 2^32.)
__device__ __forceinline__ uint64_t rope_turns(float f) {
    constexpr uint64_t hi = 0x28be60dbull, lo = 0x9391054a7f09d5f4ull;      // floor(2^96 / 2 pi)
    const uint32_t b = __float_as_uint(f), e = b >> 23 & 0xffu;
    const uint64_t m = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
    const uint64_t p0 = m * lo, p1 = __umul64hi(m, lo) + m * hi;
    const int s = max(182 - static_cast<int>(e ? e : 1), 1);               // f = m 2^(e - 150); 96 - 64 + 150 - e
    const uint64_t t = s >= 128 ? 0 : s >= 64 ? p1 >> (s - 64) : (p1 << (64 - s)) | (p0 >> s);
    return b >> 31 ? ~t + 1 : t;
}

struct RopeArgs {
    const uint16_t* c; long long ldc;
    const uint16_t* r; long long ldr;
    uint8_t* cache; long long num_rows;
    const int32_t* slots;
    const int32_t* pos;
    const float* freq;
    const uint16_t* q; long long ldq, hdq;
    uint16_t* q_out; long long ldo, hdo;
    int T, H;
    int* status;
};

// 4 pairs of a lane: loaded, turned, stored.  INTER: 8 neighbours (16 bytes); else 4 of each half (8 bytes each).
template <bool INTER>
struct RopePairs {
    uint32_t w[4];
    __device__ __forceinline__ void load(const uint16_t* p, int g) {
        if constexpr (INTER) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + 8 * g);
            w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
        } else {
            const uint2 a = *reinterpret_cast<const uint2*>(p + 4 * g), b = *reinterpret_cast<const uint2*>(p + 32 + 4 * g);
            w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
        }
    }
    __device__ __forceinline__ void turn(const float (&cs)[4], const float (&sn)[4]) {
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 x = bf16x2_bits_to_f32(w[i]);
                w[i] = f32x2_to_bf16x2_bits(x.x * cs[i] - x.y * sn[i], x.x * sn[i] + x.y * cs[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 x = bf16x2_bits_to_f32(w[i]), y = bf16x2_bits_to_f32(w[i + 2]);
                w[i] = f32x2_to_bf16x2_bits(x.x * cs[2 * i] - y.x * sn[2 * i], x.y * cs[2 * i + 1] - y.y * sn[2 * i + 1]);
                w[i + 2] = f32x2_to_bf16x2_bits(x.x * sn[2 * i] + y.x * cs[2 * i], x.y * sn[2 * i + 1] + y.y * cs[2 * i + 1]);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t* p, int g) const {
        if constexpr (INTER) {
            *reinterpret_cast<uint4*>(p + 8 * g) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<uint2*>(p + 4 * g) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2*>(p + 32 + 4 * g) = make_uint2(w[2], w[3]);
        }
    }
};

template <bool E4M3, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
kda_latent_append_rope_kernel(const RopeArgs a)
{
    const int lane = threadIdx.x & 31, g = lane & 7, sub = lane >> 3;
    const long long t = static_cast<long long>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
    if (t >= a.T) return;
    const int slot = a.slots[t], pos = a.pos[t];
    const float f = a.freq[lane];
    // (the first heads' loads, and the key's, beside those)
    constexpr int U = 4;                         // heads in flight, a lane
    RopePairs<INTER> x[U], key;
    const uint16_t* q = a.q + t * a.ldq;
    auto load = [&](int h0) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (const int h = h0 + 4 * i; h < a.H) x[i].load(q + h * a.hdq, g);
    };
    load(sub);                                   // (none without queries: H is 0 then)
    if (sub == 0) key.load(a.r + t * a.ldr, g);
    if (slot < 0) return;
    if (slot >= a.num_rows) {
        if (lane == 0) set_status(a.status, kStatusIndex);
        return;
    }
    const uint64_t turns = rope_turns(f) * static_cast<uint64_t>(static_cast<long long>(pos));
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f, &s, &c);
    if (!(fabsf(f) < 0x1p32f)) s = c = __int_as_float(0x7fffffff);
    float cs[4], sn[4];                          // of pairs 4 g .. 4 g + 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        cs[i] = __shfl_sync(0xffffffffu, c, 4 * g + i);
        sn[i] = __shfl_sync(0xffffffffu, s, 4 * g + i);
    }
    uint8_t* row = a.cache + static_cast<size_t>(slot) * lat_row_bytes(E4M3);
    const int e = put_latents<E4M3>(row, reinterpret_cast<const uint4*>(a.c + t * a.ldc), lane);
    if (sub == 0) {
        key.turn(cs, sn);
        key.store(reinterpret_cast<uint16_t*>(row + (E4M3 ? kLatDim : 2 * kLatDim)), g);
    }
    put_scale<E4M3>(row, e, lane);
    uint16_t* out = a.q_out + t * a.ldo;
    for (int h0 = sub; h0 < a.H;) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (const int h = h0 + 4 * i; h < a.H) {
                x[i].turn(cs, sn);
                x[i].store(out + h * a.hdo, g);
            }
        h0 += 4 * U;
        load(h0);
    }
}

// A warp reads kGatherTok consecutive packed tokens, their loads in flight together.
constexpr int kGatherTok = 4;

template <bool E4M3>
__global__ void __launch_bounds__(kCacheThreads)
kda_latent_gather_kernel(const uint8_t* __restrict__ cache, int num_pages, int page_size,
                         const int32_t* __restrict__ table, int max_pages, const int32_t* __restrict__ start,
                         const int32_t* __restrict__ cu, int num_seqs, int T,
                         uint16_t* __restrict__ c, long long ldc, uint16_t* __restrict__ r, long long ldr, int* status)
{
    const int lane = threadIdx.x & 31;
    const long long tb = (static_cast<long long>(blockIdx.x) * (kCacheThreads / 32) + (threadIdx.x >> 5)) * kGatherTok;
    if (tb >= T) return;
    // lane i < kGatherTok finds token tb + i: its sequence (cu[n] <= t < cu[n + 1]), page and row
    long long mine = -1;
    const long long t_mine = tb + lane;
    if (lane < kGatherTok && t_mine < T) {
        int lo = 0, hi = num_seqs;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cu[mid] <= t_mine) lo = mid; else hi = mid;
        }
        const long long pos = t_mine - cu[lo] + (start ? start[lo] : 0);
        const long long pg = pos / page_size;
        if (pos >= 0 && pg < max_pages) {
            const int page = table[static_cast<size_t>(lo) * max_pages + pg];
            if (page >= 0 && page < num_pages) mine = static_cast<long long>(page) * page_size + (pos - pg * page_size);
        }
        if (mine < 0) set_status(status, kStatusIndex);
    }
    long long slot[kGatherTok];
#pragma unroll
    for (int i = 0; i < kGatherTok; ++i) slot[i] = __shfl_sync(0xffffffffu, mine, i);
    if constexpr (!E4M3) {
        uint4 a[kGatherTok], b[kGatherTok];
        uint32_t p[kGatherTok];
#pragma unroll
        for (int i = 0; i < kGatherTok; ++i)
            if (slot[i] >= 0) {
                const uint8_t* row = cache + static_cast<size_t>(slot[i]) * kLatRowBf16;
                a[i] = __ldg(reinterpret_cast<const uint4*>(row) + lane);
                b[i] = __ldg(reinterpret_cast<const uint4*>(row) + lane + 32);
                p[i] = __ldg(reinterpret_cast<const uint32_t*>(row + 2 * kLatDim) + lane);
            }
#pragma unroll
        for (int i = 0; i < kGatherTok; ++i)
            if (slot[i] >= 0) {
                uint4* dst = reinterpret_cast<uint4*>(c + (tb + i) * ldc);
                dst[lane] = a[i];
                dst[lane + 32] = b[i];
                reinterpret_cast<uint32_t*>(r + (tb + i) * ldr)[lane] = p[i];
            }
    } else {
        // lane: codes 8 * lane .. + 7 of each half of the row, so that both 16-byte stores of a
        // warp cover whole 512-byte runs
        uint2 a[kGatherTok], b[kGatherTok];
        uint32_t p[kGatherTok];
        float s[kGatherTok];
#pragma unroll
        for (int i = 0; i < kGatherTok; ++i)
            if (slot[i] >= 0) {
                const uint8_t* row = cache + static_cast<size_t>(slot[i]) * kLatRowE4m3;
                a[i] = __ldg(reinterpret_cast<const uint2*>(row) + lane);
                b[i] = __ldg(reinterpret_cast<const uint2*>(row) + lane + 32);
                p[i] = __ldg(reinterpret_cast<const uint32_t*>(row + kLatDim) + lane);
                s[i] = __ldg(reinterpret_cast<const float*>(row + kLatScaleAt));
            }
#pragma unroll
        for (int i = 0; i < kGatherTok; ++i)
            if (slot[i] >= 0) {
                auto expand = [&](uint2 w) {           // code * s is a bf16 value: no rounding here
                    const float2 f0 = e4m3x2_to_f32(w.x), f1 = e4m3x2_to_f32(w.x >> 16);
                    const float2 f2 = e4m3x2_to_f32(w.y), f3 = e4m3x2_to_f32(w.y >> 16);
                    return make_uint4(f32x2_to_bf16x2_bits(f0.x * s[i], f0.y * s[i]), f32x2_to_bf16x2_bits(f1.x * s[i], f1.y * s[i]),
                                      f32x2_to_bf16x2_bits(f2.x * s[i], f2.y * s[i]), f32x2_to_bf16x2_bits(f3.x * s[i], f3.y * s[i]));
                };
                uint4* dst = reinterpret_cast<uint4*>(c + (tb + i) * ldc);
                dst[lane] = expand(a[i]);
                dst[lane + 32] = expand(b[i]);
                reinterpret_cast<uint32_t*>(r + (tb + i) * ldr)[lane] = p[i];
            }
    }
}

int launch_latent_append(const uint16_t* c, long long ldc, const uint16_t* r, long long ldr, void* cache, int e4m3,
                         long long num_rows, const int32_t* slots, int T, int* status, cudaStream_t stream)
{
    if (T == 0) return 0;
    const unsigned blocks = (static_cast<unsigned>(T) + kCacheThreads / 32 - 1) / (kCacheThreads / 32);
    uint8_t* p = static_cast<uint8_t*>(cache);
    if (e4m3) kda_latent_append_kernel<true><<<blocks, kCacheThreads, 0, stream>>>(c, ldc, r, ldr, p, num_rows, slots, T, status);
    else kda_latent_append_kernel<false><<<blocks, kCacheThreads, 0, stream>>>(c, ldc, r, ldr, p, num_rows, slots, T, status);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

int launch_latent_gather(const void* cache, int e4m3, int num_pages, int page_size, const int32_t* table, int max_pages,
                         const int32_t* start, const int32_t* cu, int num_seqs, int T, uint16_t* c, long long ldc,
                         uint16_t* r, long long ldr, int* status, cudaStream_t stream)
{
    if (T == 0) return 0;
    constexpr unsigned per = kCacheThreads / 32 * kGatherTok;
    const unsigned blocks = (static_cast<unsigned>(T) + per - 1) / per;
    const uint8_t* p = static_cast<const uint8_t*>(cache);
    if (e4m3)
        kda_latent_gather_kernel<true><<<blocks, kCacheThreads, 0, stream>>>(p, num_pages, page_size, table, max_pages, start,
                                                                          cu, num_seqs, T, c, ldc, r, ldr, status);
    else
        kda_latent_gather_kernel<false><<<blocks, kCacheThreads, 0, stream>>>(p, num_pages, page_size, table, max_pages, start,
                                                                           cu, num_seqs, T, c, ldc, r, ldr, status);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

int launch_latent_append_rope(const uint16_t* c, long long ldc, const uint16_t* r, long long ldr, void* cache, int e4m3,
                              long long num_rows, const int32_t* slots, const int32_t* pos, const float* freq, int inter,
                              const uint16_t* q, long long ldq, long long hdq, uint16_t* q_out, long long ldo, long long hdo,
                              int T, int H, int* status, cudaStream_t stream)
{
    if (T == 0) return 0;
    const RopeArgs a{c, ldc, r, ldr, static_cast<uint8_t*>(cache), num_rows, slots, pos, freq, q, ldq, hdq, q_out, ldo, hdo,
                     T, q ? H : 0, status};
    constexpr unsigned per = kRopeThreads / 32;
    const unsigned blocks = static_cast<unsigned>((static_cast<long long>(T) + per - 1) / per);
    if (e4m3) {
        if (inter) kda_latent_append_rope_kernel<true, true><<<blocks, kRopeThreads, 0, stream>>>(a);
        else kda_latent_append_rope_kernel<true, false><<<blocks, kRopeThreads, 0, stream>>>(a);
    } else {
        if (inter) kda_latent_append_rope_kernel<false, true><<<blocks, kRopeThreads, 0, stream>>>(a);
        else kda_latent_append_rope_kernel<false, false><<<blocks, kRopeThreads, 0, stream>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace kda
