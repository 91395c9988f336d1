// kda_latent.cu -- absorbed latent attention over the paged cache.
//
// Row (n, j, h) of the output: x_t = scale * (q[:512] . c_t + q[512:] . r_t) over the tokens the
// query sees, out = sum_t softmax(x)_t c_t, with one pass over the tokens: the running maximum m,
// the sum l of exp(x - m) and the weighted sum of c are rescaled when m grows.
#include "latent.cuh"

namespace kda {

struct LatentCache {
    const uint8_t* rows;
    const int32_t* table;        // [N, max_pages]
    int num_pages, page_size, max_pages;
};

// One warp computes one row in fp32, straight from the formula.  Lane i owns latents
// 16 i .. 16 i + 15 and position values 2 i, 2 i + 1.
template <bool E4M3>
__device__ void latent_row(const uint16_t* __restrict__ q, const LatentCache& ch, int n, int see, float scale_log2,
                           uint16_t* __restrict__ out, float* __restrict__ lse, int* status)
{
    const int lane = threadIdx.x & 31;
    float qc[16], acc[16];
    {
        const uint4* p = reinterpret_cast<const uint4*>(q) + 2 * lane;
        const uint4 a = p[0], b = p[1];
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 f = bf16x2_bits_to_f32(w[i]);
            qc[2 * i] = f.x; qc[2 * i + 1] = f.y;
        }
    }
    const float2 qr = bf16x2_bits_to_f32(reinterpret_cast<const uint32_t*>(q + kLatDim)[lane]);
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    float m = -INFINITY, l = 0.f;
    int page = 0;
    for (int t = 0; t < see; ++t) {
        const int in = t % ch.page_size;
        if (in == 0 || t == 0) {
            page = ch.table[static_cast<size_t>(n) * ch.max_pages + t / ch.page_size];
            if (page < 0 || page >= ch.num_pages) {
                if (lane == 0) set_status(status, kStatusIndex);
                page = 0;
            }
        }
        const uint8_t* row = ch.rows + (static_cast<size_t>(page) * ch.page_size + in) * lat_row_bytes(E4M3);
        float c[16];
        float2 r;
        if constexpr (E4M3) {
            const uint4 a = reinterpret_cast<const uint4*>(row)[lane];
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
            const float s = *reinterpret_cast<const float*>(row + kLatScaleAt);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = e4m3x2_to_f32(w[i]), g = e4m3x2_to_f32(w[i] >> 16);
                c[4 * i] = f.x * s; c[4 * i + 1] = f.y * s; c[4 * i + 2] = g.x * s; c[4 * i + 3] = g.y * s;
            }
            r = bf16x2_bits_to_f32(reinterpret_cast<const uint32_t*>(row + kLatDim)[lane]);
        } else {
            const uint4* p = reinterpret_cast<const uint4*>(row) + 2 * lane;
            const uint4 a = p[0], b = p[1];
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float2 f = bf16x2_bits_to_f32(w[i]);
                c[2 * i] = f.x; c[2 * i + 1] = f.y;
            }
            r = bf16x2_bits_to_f32(reinterpret_cast<const uint32_t*>(row + 2 * kLatDim)[lane]);
        }
        float x = qr.x * r.x + qr.y * r.y;
#pragma unroll
        for (int i = 0; i < 16; ++i) x += qc[i] * c[i];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
        x *= scale_log2;
        if (x > m) {
            const float f = lat_ex2(m - x);
            m = x;
            l *= f;
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] *= f;
        }
        const float p = x == -INFINITY ? 0.f : lat_ex2(x - m);
        l += p;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] += p * c[i];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;      // (a NaN sum stays NaN)
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = f32x2_to_bf16x2_bits(acc[2 * i] * inv, acc[2 * i + 1] * inv);
    uint4* d = reinterpret_cast<uint4*>(out) + 2 * lane;
    d[0] = make_uint4(o[0], o[1], o[2], o[3]);
    d[1] = make_uint4(o[4], o[5], o[6], o[7]);
    if (lse && lane == 0) *lse = (m + log2f(l)) * 0.69314718055994531f;     // l = 0: -inf
}

template <bool E4M3>
__global__ void __launch_bounds__(128)
kda_latent_rows_kernel(const uint16_t* __restrict__ q, LatentCache ch, const int32_t* __restrict__ seq_lens, int K, int H,
                       long long rows, float scale_log2, uint16_t* __restrict__ out, float* __restrict__ lse, int* status)
{
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= rows) return;
    const int n = static_cast<int>(row / (static_cast<long long>(K) * H));
    const int j = static_cast<int>(row / H % K);
    int len = seq_lens[n];
    if (len < 0 || len > static_cast<long long>(ch.max_pages) * ch.page_size) {
        if ((threadIdx.x & 31) == 0) set_status(status, kStatusIndex);
        len = 0;
    }
    latent_row<E4M3>(q + row * kLatQ, ch, n, len - (K - 1 - j), scale_log2, out + row * kLatDim, lse ? lse + row : nullptr,
                     status);
}

int launch_latent_decode(const uint16_t* q, const void* cache, int e4m3, int num_pages, int page_size,
                         const int32_t* table, int max_pages, const int32_t* seq_lens, int N, int K, int H,
                         float sm_scale, uint16_t* out, float* lse, int* status, cudaStream_t stream)
{
    const long long rows = static_cast<long long>(N) * K * H;
    const LatentCache ch{static_cast<const uint8_t*>(cache), table, num_pages, page_size, max_pages};
    const float sl2 = sm_scale * 1.4426950408889634f;
    const unsigned blocks = static_cast<unsigned>((rows + 3) / 4);
    if (e4m3) kda_latent_rows_kernel<true><<<blocks, 128, 0, stream>>>(q, ch, seq_lens, K, H, rows, sl2, out, lse, status);
    else kda_latent_rows_kernel<false><<<blocks, 128, 0, stream>>>(q, ch, seq_lens, K, H, rows, sl2, out, lse, status);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace kda
