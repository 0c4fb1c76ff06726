// decode_fp8.cu -- split-free decode over the 8-bit cache (mlra_decode_fp8):
// mlra_decode with c_b[t] = sigma[t / 16][b] e[t][b].  One CTA per (sequence,
// head, branch); a lane owns d_c / 32 latent columns, the warps take every
// eighth token each with a running maximum and sum, and meet at the end.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace mlra {
namespace {

constexpr int kWarps = 8;

template <int DC, int DR>
__global__ void __launch_bounds__(kWarps * 32) decode_fp8_kernel(const DecodeArgs a, const float* latent_scale) {
    constexpr int E = DC / 32, ER = DR / 32;
    __shared__ float ms[kWarps], ls[kWarps], os[kWarps][DC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = a.branches, H = a.heads, P = a.page_size;
    const int b = blockIdx.x % B, h = blockIdx.x / B % H, n = blockIdx.x / B / H;
    const uint8_t* cache = reinterpret_cast<const uint8_t*>(a.latent);
    const int L = a.seqlens[n];
    int bad = seqlen_valid(L, P, a.max_pages) ? 0 : MLRA_ERR_DEVICE_BAD_SEQLEN;
    const int32_t* bt = a.block_table + (size_t)n * a.max_pages;
    if (!bad) {
        bool out = false;
        for (int i = lane; i < ceil_div(L, P); i += 32) out |= bt[i] < 0 || bt[i] >= a.num_pages;
        if (__any_sync(0xffffffffu, out)) bad = MLRA_ERR_DEVICE_BAD_INDEX;
    }
    float ql[E], qr[ER], o[E];
    for (int j = 0; j < E; ++j) ql[j] = __bfloat162float(a.q_lat[(((size_t)n * H + h) * B + b) * DC + lane + 32 * j]), o[j] = 0.f;
    for (int j = 0; j < ER; ++j) qr[j] = __bfloat162float(a.q_rope[((size_t)n * H + h) * DR + lane + 32 * j]);
    float m = -INFINITY, l = 0.f;
    for (int t = warp; !bad && t < L; t += kWarps) {
        const size_t r = (size_t)bt[t / P] * P + t % P;
        const float sigma = latent_scale[r / kFp8Block * B + b];
        float c[E], s = 0.f;
        for (int j = 0; j < E; ++j) {
            __nv_fp8_e4m3 e;
            e.__x = cache[(r * B + b) * DC + lane + 32 * j];
            c[j] = sigma * static_cast<float>(e), s = fmaf(ql[j], c[j], s);
        }
        for (int j = 0; j < ER; ++j) s = fmaf(qr[j], __bfloat162float(a.rope[r * DR + lane + 32 * j]), s);
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s), alpha = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = fmaf(l, alpha, p);
        for (int j = 0; j < E; ++j) o[j] = fmaf(o[j], alpha, p * c[j]);
    }
    if (lane == 0) ms[warp] = m, ls[warp] = l;
    for (int j = 0; j < E; ++j) os[warp][lane + 32 * j] = o[j];
    __syncthreads();
    float mx = -INFINITY, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, ms[w]);
    for (int w = 0; w < kWarps; ++w) sum += ls[w] * exp2f(ms[w] - mx);
    if (bad && threadIdx.x == 0) record_error(a.err, bad);
    for (int k = threadIdx.x; k < DC; k += kWarps * 32) {
        float v = 0.f;
        for (int w = 0; w < kWarps; ++w) v += os[w][k] * exp2f(ms[w] - mx);
        a.out[(((size_t)n * H + h) * B + b) * DC + k] = to_bf16(bad ? 0.f : v * a.out_scale / sum);
    }
}

template <int DC>
cudaError_t launch_dc(const DecodeArgs& a, const float* s, cudaStream_t stream) {
    const unsigned grid = (unsigned)a.batch * a.heads * a.branches;
    if (a.d_r == 64) decode_fp8_kernel<DC, 64><<<grid, kWarps * 32, 0, stream>>>(a, s);
    else decode_fp8_kernel<DC, 32><<<grid, kWarps * 32, 0, stream>>>(a, s);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeArgs& a, const float* latent_scale, cudaStream_t stream) {
    switch (a.d_c) {
        case 64: return launch_dc<64>(a, latent_scale, stream);
        case 128: return launch_dc<128>(a, latent_scale, stream);
        case 256: return launch_dc<256>(a, latent_scale, stream);
        case 512: return launch_dc<512>(a, latent_scale, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace mlra
