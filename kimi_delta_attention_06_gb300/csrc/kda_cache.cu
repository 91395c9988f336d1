// kda_cache.cu -- the latent cache as it is written (bf16, or e4m3 with one power-of-two scale a
// token) and read back.  Both kernels move bytes: one warp per token, 16-byte accesses, the
// token's row in registers once, so they are bound by HBM for long runs and by the launch for a
// decode step's few rows.  Measured, e4m3: 145408 tokens written in 42 us (6.2 TB/s of 6.7), 214k
// tokens in pages of 48 read back in 60 us (6.4 TB/s); 512 tokens written and read back 5.4 us.
#include "latent.cuh"

namespace kda {

constexpr int kCacheThreads = 256;

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
    if constexpr (!E4M3) {
        uint4* dst = reinterpret_cast<uint4*>(row);
        const uint4 a = src[lane], b = src[lane + 32];
        dst[lane] = a;
        dst[lane + 32] = b;
        reinterpret_cast<uint32_t*>(row + 2 * kLatDim)[lane] = rope;
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
        reinterpret_cast<uint32_t*>(row + kLatDim)[lane] = rope;
        if (lane < 4)
            reinterpret_cast<uint32_t*>(row + kLatScaleAt)[lane] =
                lane == 0 ? static_cast<uint32_t>(127 + e) << 23 : 0u;
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

}  // namespace kda
