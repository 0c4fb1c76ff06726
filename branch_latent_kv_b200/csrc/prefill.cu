// prefill.cu -- causal attention of packed prompt tokens over the paged
// latent cache (mlra_prefill): out = out_scale softmax(scale (q_lat . c_b +
// q_rope . k_r)) c_b over the tokens up to the query's own, every branch on
// its own.  One warp per (query row, head, branch): a lane owns d_c / 32
// latent columns and d_r / 32 key columns, and the warp walks the tokens with
// a running maximum and sum.
#include "common.cuh"
#include "kernels.h"

namespace mlra {
namespace {

constexpr int kWarps = 4;

template <int DC, int DR>
__global__ void __launch_bounds__(kWarps * 32) prefill_kernel(const PrefillArgs a) {
    constexpr int E = DC / 32, ER = DR / 32;
    const int lane = threadIdx.x & 31;
    const long long item = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int B = a.branches, H = a.heads, P = a.page_size;
    if (item >= (long long)a.tokens * H * B) return;
    const int row = (int)(item / (H * B)), h = (int)(item / B) % H, b = (int)(item % B);
    // the sequence whose run holds this row
    int n = -1, c0 = 0, q = 0;
    for (int m = 0; m < a.batch; ++m) {
        const int lo = a.cu_seqlens[m], hi = a.cu_seqlens[m + 1];
        if (lo >= 0 && hi >= lo && hi <= a.tokens) {
            if (row >= lo && row < hi) n = m, c0 = lo, q = hi - lo;
        } else if (lane == 0 && a.status != nullptr) {
            record_error(a.status, MLRA_ERR_DEVICE_BAD_SEQLEN);
        }
    }
    if (n < 0) return;
    const int L = a.seqlens[n];
    int bad = 0;
    if (L < q || !seqlen_valid(L, P, a.max_pages)) bad = MLRA_ERR_DEVICE_BAD_SEQLEN;
    const int32_t* bt = a.block_table + (size_t)n * a.max_pages;
    if (!bad) {
        bool out = false;
        for (int i = lane; i < ceil_div(L, P); i += 32) out |= bt[i] < 0 || bt[i] >= a.num_pages;
        if (__any_sync(0xffffffffu, out)) bad = MLRA_ERR_DEVICE_BAD_INDEX;
    }
    __nv_bfloat16* dst = a.out + (((size_t)row * H + h) * B + b) * DC;
    if (bad) {
        if (lane == 0 && a.status != nullptr) record_error(a.status, bad);
        for (int j = 0; j < E; ++j) dst[lane + 32 * j] = to_bf16(0.f);
        return;
    }
    float ql[E], qr[ER], o[E];
    for (int j = 0; j < E; ++j) ql[j] = __bfloat162float(a.q_lat[(((size_t)row * H + h) * B + b) * DC + lane + 32 * j]), o[j] = 0.f;
    for (int j = 0; j < ER; ++j) qr[j] = __bfloat162float(a.q_rope[((size_t)row * H + h) * DR + lane + 32 * j]);
    float m = -INFINITY, l = 0.f;
    const int last = L - q + (row - c0);
    for (int t = 0; t <= last; ++t) {
        const size_t r = (size_t)bt[t / P] * P + t % P;
        float c[E], s = 0.f;
        for (int j = 0; j < E; ++j) c[j] = __bfloat162float(a.latent[(r * B + b) * DC + lane + 32 * j]), s = fmaf(ql[j], c[j], s);
        for (int j = 0; j < ER; ++j) s = fmaf(qr[j], __bfloat162float(a.rope[r * DR + lane + 32 * j]), s);
        for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
        s *= a.scale_log2;
        const float mn = fmaxf(m, s), alpha = exp2f(m - mn), p = exp2f(s - mn);
        m = mn;
        l = fmaf(l, alpha, p);
        for (int j = 0; j < E; ++j) o[j] = fmaf(o[j], alpha, p * c[j]);
    }
    for (int j = 0; j < E; ++j) dst[lane + 32 * j] = to_bf16(o[j] * a.out_scale / l);
}

template <int DC>
cudaError_t launch_dc(const PrefillArgs& a, cudaStream_t stream) {
    const long long items = (long long)a.tokens * a.heads * a.branches;
    const unsigned grid = (unsigned)((items + kWarps - 1) / kWarps);
    if (a.d_r == 64) prefill_kernel<DC, 64><<<grid, kWarps * 32, 0, stream>>>(a);
    else prefill_kernel<DC, 32><<<grid, kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill(const PrefillArgs& a, cudaStream_t stream) {
    if (a.status != nullptr) {
        const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(int), stream);
        if (e != cudaSuccess) return e;
    }
    if (a.tokens == 0) return cudaSuccess;
    switch (a.d_c) {
        case 64: return launch_dc<64>(a, stream);
        case 128: return launch_dc<128>(a, stream);
        case 256: return launch_dc<256>(a, stream);
        case 512: return launch_dc<512>(a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace mlra
