// append_fp8.cu -- new tokens written into the 8-bit paged cache.
//
// The cache keeps each branch's latents as e4m3 values with one fp32 scale
// for every 16 tokens of a page:  c_b[t] = sigma[t / 16][b] * e[t][b].  For a
// block of 16 tokens and a branch
//   sigma = the smallest power of two with amax <= 448 sigma, not below 2^-40
// (448 is the largest e4m3 value; amax over the finite new values), and a
// block that holds earlier tokens of the sequence keeps the larger of its
// scale and the new one, its earlier rows rounded again where it grew.  A
// power of two costs e4m3 no precision (the quotient x / sigma is exact, so a
// value is rounded once, to half a step, 2^-4 of it) and makes that second
// rounding exact too, except for values that fall below the normal range.
// RoPE keys are turned to their positions as mlra_prepare turns them and stay
// bf16.
//
// One warp per (16-token block, branch): its 16 rows of d_c bf16 values fit a
// lane's registers (d_c / 16 16-byte loads each, all in flight at once), so
// the maximum, the scale and the rounded rows need one pass over the data and
// no shared memory; one more warp per block turns the keys.  The blocks a
// sequence touches are not known on the host, so the grid has T / 16 + 2 N
// places, of which sequence n owns those from cu[n] / 16 + 2 n on (q new
// tokens touch at most q / 16 + 2 blocks); a warp finds its sequence by a
// 32-way search.  Bound by the chain search -> table -> rows for single tokens
// (the rows are requested before the table answers): 2.8 us for 16 sequences.
// 23,449 prompt tokens of four 128-wide branches, 42 MB, take 12.1 us (3.5 TB/s),
// with 60 % of the issue slots used, by conversions and rotations.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace mlra {
namespace {

using namespace sm100;

constexpr int kAppendWarps = 2;
constexpr unsigned kFull = 0xffffffffu;

// A sequence's new tokens: rows [row0, row0 + q) of c_new, positions
// [begin, begin + q).
struct Run {
    int row0, q, begin;
};

// The run of offsets c0, c1 and length L; false when one is out of range.
__device__ __forceinline__ bool run_of(const AppendFp8Args& a, int c0, int c1, int L, Run& r) {
    r.row0 = c0;
    r.q = c1 - c0;
    r.begin = L - r.q;
    if (c0 < 0 || c1 < c0 || c1 > a.tokens) return false;
    return r.q == 0 || (L >= r.q && (long long)L <= (long long)a.max_pages * a.page_size);
}

// First place of sequence n, whose offset is c0 (in 64 bits: it may be anything).
__device__ __forceinline__ long long place_of(int c0, int n) { return ((long long)c0 >> 4) + 2ll * n; }

// Whole warp: the last sequence whose first place is at or before v, its
// offsets and length (the last round loads them with what it searches).
__device__ __forceinline__ int find_seq(const AppendFp8Args& a, long long v, int lane, int& c0, int& c1, int& L) {
    int lo = 0, len = a.batch;  // the answer lies in [lo, lo + len)
    while (len > 32) {
        const int step = (len + 31) / 32, n = lo + lane * step, end = lo + len;
        const unsigned hit = __ballot_sync(kFull, n < end && place_of(__ldg(a.cu_seqlens + n), n) <= v);
        lo += (hit ? 31 - __clz(hit) : 0) * step;
        len = min(step, end - lo);
    }
    const int n = lo + min(lane, len - 1);
    c0 = __ldg(a.cu_seqlens + n);
    c1 = __ldg(a.cu_seqlens + n + 1);
    L = __ldg(a.seqlens + n);
    const unsigned hit = __ballot_sync(kFull, lane < len && place_of(c0, n) <= v);
    const int k = hit ? 31 - __clz(hit) : 0;
    c0 = __shfl_sync(kFull, c0, k);
    c1 = __shfl_sync(kFull, c1, k);
    L = __shfl_sync(kFull, L, k);
    return lo + k;
}

// Exponent of the smallest power of two s with amax <= 448 s (448 = 1.75 2^8),
// amax a finite non-negative float.
__device__ __forceinline__ int scale_exponent(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u);
    return max(e, kFp8MinScaleExp);
}

__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3)));
}

// The bf16 pair of a 32-bit word as floats.
__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <int DC>
// (16 CTAs of two warps an SM for rows up to 128 wide, 64 registers: a prompt
// batch of 23,449 tokens 12.1 us; 12 CTAs 12.5 us, 20 with 48 registers 12.7 us)
__global__ void __launch_bounds__(kAppendWarps * 32, DC <= 128 ? 16 : DC == 256 ? 8 : 4)
append_fp8_kernel(const AppendFp8Args a) {
    constexpr int ROW = DC / 8;        // 16-byte units of a row
    constexpr int U = DC / 16;         // units per lane: 16 rows over 32 lanes
    const int lane = threadIdx.x & 31;
    const int B = a.branches, P = a.page_size;
    launch_dependents();
    wait_prerequisite_grid();

    if (blockIdx.x == 0 && a.status != nullptr) {  // runs out of range, whichever places they claim
        for (int n = threadIdx.x; n < a.batch; n += blockDim.x) {
            Run r;
            if (!run_of(a, __ldg(a.cu_seqlens + n), __ldg(a.cu_seqlens + n + 1), __ldg(a.seqlens + n), r))
                record_error(a.status, MLRA_ERR_DEVICE_BAD_SEQLEN);
        }
    }
    // (at most (2^27 + 2^17) 9 warps: 32 bits)
    const uint32_t item = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const uint32_t v = item / (uint32_t)(B + 1);
    const int b = (int)(item - v * (uint32_t)(B + 1));  // branch, or B for the keys
    if (v >= (uint32_t)a.places) return;
    int c0, c1, L;
    const int n = find_seq(a, v, lane, c0, c1, L);
    Run r;
    if (!run_of(a, c0, c1, L, r)) return;
    const long long j = v - place_of(c0, n);
    if (j < 0 || r.q == 0 || (r.begin & ~15) + 16 * j >= (long long)r.begin + r.q) return;
    const int p0 = (r.begin & ~15) + 16 * (int)j;  // first position of the block
    const int lo = max(r.begin, p0) - p0, hi = min(r.begin + r.q - p0, 16);  // new slots of the block
    const int page = __ldg(a.block_table + (size_t)n * a.max_pages + p0 / P);
    // the row of c_new that slot 0 of the block would have (lo rows further is the first)
    const long long src0 = (long long)r.row0 + (p0 - r.begin);
    const bool page_ok = page >= 0 && page < a.num_pages;
    const size_t block = page_ok ? ((size_t)page * P + p0 % P) / 16 : 0;

    if (b == B) {
        // ------------------------------------------------------------ RoPE keys
        if (!page_ok) {
            if (lane == 0 && a.status != nullptr) record_error(a.status, MLRA_ERR_DEVICE_BAD_INDEX);
            return;
        }
        const int half = a.d_r / 2;
        if (lane >= half) return;
        // Angles in turns.  Position p0 + i turns by frac(p0 turns) + i turns: the
        // first reduced to [0, 1) in fp64 once, and i times the upper 19 bits of
        // `turns` exact in fp32, so that its fraction is too; 2^-23 of a turn in all.
        const double turns = a.rope_turns[lane], base = (double)p0 * turns;
        const float f0 = (float)(base - floor(base));
        const float t_hi = __uint_as_float(__float_as_uint((float)turns) & ~31u), t_lo = (float)(turns - (double)t_hi);
        __nv_bfloat162 x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i >= lo && i < hi)
                x[i] = __ldg(reinterpret_cast<const __nv_bfloat162*>(a.kr_new + (src0 + i) * a.d_r) + lane);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if (i < lo || i >= hi) continue;
            const float whole = (float)i * t_hi;
            float s, c;
            sincospif(2.f * fmaf((float)i, t_lo, f0 + (whole - floorf(whole))), &s, &c);
            const float x0 = __low2float(x[i]), x1 = __high2float(x[i]);
            reinterpret_cast<__nv_bfloat162*>(a.rope_cache + (block * 16 + i) * a.d_r)[lane] =
                __floats2bfloat162_rn(x0 * c - x1 * s, x0 * s + x1 * c);
        }
        return;
    }

    // ---------------------------------------------------------------- one branch
    const size_t W = (size_t)B * DC;
    uint4 x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = lane + 32 * i, slot = u / ROW, col = u % ROW;
        x[i] = make_uint4(0u, 0u, 0u, 0u);
        if (slot >= lo && slot < hi)
            x[i] = __ldg(reinterpret_cast<const uint4*>(a.c_new + (src0 + slot) * W + (size_t)b * DC) + col);
    }
    if (!page_ok) return;
    float* scale = a.latent_scale + block * B + b;
    const float old = lo > 0 ? *scale : 0.f;
    // largest magnitude, as 16-bit integers (|bf16| is ordered like its bits), two
    // at a time; again over the finite values where one is not
    uint32_t mx2 = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        mx2 = __vimax3_u16x2(mx2, x[i].x & 0x7fff7fffu, x[i].y & 0x7fff7fffu);
        mx2 = __vimax3_u16x2(mx2, x[i].z & 0x7fff7fffu, x[i].w & 0x7fff7fffu);
    }
    uint32_t mx = __reduce_max_sync(kFull, max(mx2 & 0xffffu, mx2 >> 16));
    if (mx >= 0x7f80u) {
        mx = 0;
#pragma unroll 1
        for (int i = 0; i < U; ++i) {
            uint4 y = x[0];
#pragma unroll
            for (int k = 1; k < U; ++k) y = k == i ? x[k] : y;
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t h0 = w[k] & 0x7fffu, h1 = (w[k] >> 16) & 0x7fffu;
                mx = max(mx, h0 < 0x7f80u ? h0 : 0u);
                mx = max(mx, h1 < 0x7f80u ? h1 : 0u);
            }
        }
        mx = __reduce_max_sync(kFull, mx);
    }
    const float fresh = __uint_as_float((uint32_t)(scale_exponent(__uint_as_float(mx << 16)) + 127) << 23);
    const float sigma = fmaxf(fresh, old), inv = 1.f / sigma;
    uint8_t* codes = a.latent_cache + block * 16 * W + (size_t)b * DC;
    if (lo > 0 && sigma != old) {
        // the block's scale grew: its earlier rows at the new one
        const float ratio = old * inv;
        for (int u = lane; u < lo * ROW; u += 32) {
            uint2* at = reinterpret_cast<uint2*>(codes + (u / ROW) * W) + u % ROW;
            uint2 e = *at;
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = from_e4m3x2(((k < 2 ? e.x : e.y) >> (16 * (k & 1))) & 0xffffu);
                o[k] = e4m3x2(f.x * ratio, f.y * ratio);
            }
            *at = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
        }
    }
    if (lane == 0) *scale = sigma;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = lane + 32 * i, slot = u / ROW, col = u % ROW;
        if (slot < lo || slot >= hi) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = bf16_pair(w[k]);
            o[k] = e4m3x2(f.x * inv, f.y * inv);
        }
        reinterpret_cast<uint2*>(codes + slot * W)[col] = make_uint2(o[0] | o[1] << 16, o[2] | o[3] << 16);
    }
}

template <int DC>
cudaError_t launch_dc(const AppendFp8Args& a, cudaStream_t stream) {
    const long long warps = a.places * (a.branches + 1);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((warps + kAppendWarps - 1) / kAppendWarps));
    cfg.blockDim = dim3(kAppendWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, append_fp8_kernel<DC>, a);
}

}  // namespace

cudaError_t launch_append_fp8(const AppendFp8Args& a, cudaStream_t stream) {
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
