// kda_latent_prefill.cu -- expanded latent attention over packed prompts: per head keys
// [k (128), r (64, shared by the heads)] and values v (128).
//
// Row (i, h): x_t = scale * (q[:128] . k_t + q[128:] . r_t) over the keys the query sees,
// out = sum_t softmax(x)_t v_t, with the running maximum and sum of one pass.
#include "latent.cuh"

namespace kda {

constexpr int kExpK = 128, kExpV = 128, kExpQ = kExpK + kLatRope;

struct ExpKv {
    const uint16_t *k, *v, *r;
    long long ldk, hdk, ldv, hdv, ldr;
};

// One warp computes one row in fp32, straight from the formula, over keys [k0, k0 + see).  Lane i
// owns key and value channels 4 i .. 4 i + 3 and position values 2 i, 2 i + 1.
__device__ void expanded_row(const uint16_t* __restrict__ q, const ExpKv& kv, int h, long long k0, int see,
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

__global__ void __launch_bounds__(128)
kda_expanded_rows_kernel(const uint16_t* __restrict__ q, ExpKv kv, const int32_t* __restrict__ cu_q,
                         const int32_t* __restrict__ cu_k, int num_seqs, int total_q, int H, int causal, float scale_log2,
                         uint16_t* __restrict__ out, float* __restrict__ lse)
{
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (row >= static_cast<long long>(total_q) * H) return;
    const int t = static_cast<int>(row / H), h = static_cast<int>(row % H);
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_q[mid] <= t) lo = mid; else hi = mid;
    }
    const int Lq = cu_q[lo + 1] - cu_q[lo], Lk = cu_k[lo + 1] - cu_k[lo];
    const int see = causal ? t - cu_q[lo] + 1 + Lk - Lq : Lk;
    expanded_row(q + row * kExpQ, kv, h, cu_k[lo], see, scale_log2, out + row * kExpV, lse ? lse + row : nullptr);
}

int launch_latent_prefill(const uint16_t* q, const uint16_t* k, long long ldk, long long hdk, const uint16_t* v,
                          long long ldv, long long hdv, const uint16_t* r, long long ldr, const int32_t* cu_q,
                          const int32_t* cu_k, int num_seqs, int total_q, int total_k, int max_q, int H, int causal,
                          float sm_scale, uint16_t* out, float* lse, int* status, cudaStream_t stream)
{
    const ExpKv kv{k, v, r, ldk, hdk, ldv, hdv, ldr};
    const long long rows = static_cast<long long>(total_q) * H;
    kda_expanded_rows_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(
        q, kv, cu_q, cu_k, num_seqs, total_q, H, causal, sm_scale * 1.4426950408889634f, out, lse);
    return cudaGetLastError() == cudaSuccess ? 0 : -3;
}

}  // namespace kda
