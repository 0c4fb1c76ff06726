// decode_split.cuh -- what the tensor-core decode kernels share: head groups,
// the walk over a CTA's ranges of the split plan, the softmax warps'
// reductions, and the in-kernel merge of split sequences.
#pragma once

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"

namespace mlra {

using namespace sm100;

constexpr int kT = kTileTokens;     // tokens per tile = MMA M
constexpr int kThreads = 352;      // of a decode_tc.cu CTA
constexpr float kRescaleLog2 = 8.0f;
constexpr int kSmemLimit = 232448;  // max dynamic shared memory per CTA on sm_100

// Head groups.  The MMAs take one tile of HP heads (N = 16, or 32 when there
// are more than 16 heads); more heads run as ceil(H / HP) groups side by
// side.  CTA g * cpg + i (cpg = grid / groups) runs window i of one cost plan
// over cpg windows for heads [HP g, HP g + HP), so the groups stream the same
// tokens at about the same time and every read of a cache line after the
// first hits L2 (the latents are shared by all heads).  Each group has its own
// partial slots (a block of cpg + batch) and split counters (a block of
// batch); CTAs past groups * cpg only take part in the fused up-projection.
struct HeadGroup {
    int ci, cpg;   // window of this CTA, windows (CTAs) per group
    int h0, hn;    // first head of the group, heads in it
    int slot0;     // first partial slot of the group
    int cnt0;      // first split counter of the group
    bool idle;     // no group: beyond groups * cpg
};

template <int HP>
__device__ __forceinline__ HeadGroup head_group(const DecodeArgs& a) {
    constexpr int kHP = HP;
    HeadGroup hg;
    const int groups = (a.heads + HP - 1) / HP;
    hg.cpg = a.num_ctas / groups;
    const int g = (int)blockIdx.x / hg.cpg;
    hg.ci = (int)blockIdx.x - g * hg.cpg;
    hg.idle = g >= groups;
    hg.h0 = g * kHP;
    hg.hn = hg.idle ? 0 : min(kHP, a.heads - hg.h0);
    hg.slot0 = g * (hg.cpg + a.batch);
    hg.cnt0 = g * a.batch;
    return hg;
}

// 2^x on the special-function unit (ex2.approx, flush-to-zero: results below
// 2^-126 become 0, which only affects probabilities that are negligible).
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Max over the 32 lanes of a warp of each of 16 values, reduce-scattered:
// the result for column c ends up in lanes 2c and 2c+1.  16 shuffles.
__device__ __forceinline__ float warp_colmax16(const float (&v)[16], int lane) {
    float a8[8], a4[4], a2[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // lanes with bit 4 keep columns 8..15
        const bool hi = lane & 16;
        const float keep = hi ? v[i + 8] : v[i], send = hi ? v[i] : v[i + 8];
        a8[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool hi = lane & 8;
        const float keep = hi ? a8[i + 4] : a8[i], send = hi ? a8[i] : a8[i + 4];
        a4[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 8));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool hi = lane & 4;
        const float keep = hi ? a4[i + 2] : a4[i], send = hi ? a4[i] : a4[i + 2];
        a2[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 4));
    }
    const bool hi = lane & 2;
    const float keep = hi ? a2[1] : a2[0], send = hi ? a2[0] : a2[1];
    const float a1 = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 2));
    return fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
}

// Max over the 32 lanes of a warp of each of 8 values, reduce-scattered:
// the result for column c ends up in lanes 4c..4c+3.  9 shuffles.
__device__ __forceinline__ float warp_colmax8(const float (&v)[8], int lane) {
    float a4[4], a2[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // lanes with bit 4 keep columns 4..7
        const bool hi = lane & 16;
        const float keep = hi ? v[i + 4] : v[i], send = hi ? v[i] : v[i + 4];
        a4[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const bool hi = lane & 8;
        const float keep = hi ? a4[i + 2] : a4[i], send = hi ? a4[i] : a4[i + 2];
        a2[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 8));
    }
    const bool hi = lane & 4;
    const float keep = hi ? a2[1] : a2[0], send = hi ? a2[0] : a2[1];
    float a1 = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 4));
    a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 2));
    return fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, 1));
}

// And of 4 values: column c in lanes 8c..8c+7.  6 shuffles.
__device__ __forceinline__ float warp_colmax4(const float (&v)[4], int lane) {
    float a2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {  // lanes with bit 4 keep columns 2..3
        const bool hi = lane & 16;
        const float keep = hi ? v[i + 2] : v[i], send = hi ? v[i] : v[i + 2];
        a2[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 16));
    }
    const bool hi = lane & 8;
    const float keep = hi ? a2[1] : a2[0], send = hi ? a2[0] : a2[1];
    float a1 = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, 8));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, o));
    return a1;
}

// The same for a softmax group's N = 4, 8 or 16 heads: column c in lanes
// [c 32 / N, (c + 1) 32 / N).
template <int N>
__device__ __forceinline__ float warp_colmax(const float (&v)[N], int lane) {
    if constexpr (N == 4) return warp_colmax4(v, lane);
    else if constexpr (N == 8) return warp_colmax8(v, lane);
    else return warp_colmax16(v, lane);
}

// TMEM loads and stores of a softmax group's N = 4, 8 or 16 columns.
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[N]) {
    if constexpr (N == 4) tmem_ld4(taddr, v);
    else if constexpr (N == 8) tmem_ld8(taddr, v);
    else tmem_ld16(taddr, v);
}
template <int N>
__device__ __forceinline__ void tmem_st_cols(uint32_t taddr, const float (&v)[N]) {
    if constexpr (N == 4) tmem_st4(taddr, v);
    else if constexpr (N == 8) tmem_st8(taddr, v);
    else tmem_st16(taddr, v);
}

// Sum over the 32 lanes of a warp of each of N values (N = 16, 32, 64, 128),
// reduce-scattered: afterwards, for N >= 32, lane L holds in v[r]
// (r < N/32) the warp total of value N/32*L + r; for N = 16, lanes 2c and
// 2c+1 hold in v[0] the total of value c.  N - 1 + (N < 32) shuffles.
template <int LIVE, int O, int N>
__device__ __forceinline__ void warp_sum_scatter(float (&v)[N], int lane) {
    if constexpr (O >= 1) {
        if constexpr (LIVE >= 2) {
            constexpr int H = LIVE / 2;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const bool hi = lane & O;
                const float keep = hi ? v[i + H] : v[i], send = hi ? v[i] : v[i + H];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, O);
            }
            warp_sum_scatter<H, O / 2, N>(v, lane);
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
            warp_sum_scatter<1, O / 2, N>(v, lane);
        }
    }
}

template <int DR>
__device__ __forceinline__ uint64_t rope_desc(uint32_t addr) {
    return DR == 64 ? smem_desc(addr, 16, 1024, kLayoutSw128) : smem_desc(addr, 16, 512, kLayoutSw64);
}

// The sequence walk every role performs identically: the next sequence n
// (cost start cum) with tiles [tb, te) in this CTA's cost window [A0, A1).
// next_len holds seqlens[n], loaded one range ahead (first_len starts it).
// The caller advances past the range with finish_segment.
__device__ __forceinline__ int first_len(const DecodeArgs& a, int n) {
    return n < a.batch ? __ldg(a.seqlens + n) : 0;
}

template <int SEQ = kSeqCost>
__device__ __forceinline__ bool next_segment(const DecodeArgs& a, int& n, int& cum, int A0, int A1,
                                             int& L, int& tiles, int& tb, int& te, int& next_len, int end) {
    while (n < end && cum < A1) {
        L = next_len;
        next_len = n + 1 < end ? __ldg(a.seqlens + n + 1) : 0;
        tiles = seq_tiles(L, a.page_size, a.max_pages);
        if (tiles > 0) {
            tb = first_tile_at(cum, tiles, A0);
            te = first_tile_at(cum, tiles, A1);
            if (tb < te) return true;
            cum += tiles * kTileCost + SEQ;
        }
        ++n;
    }
    return false;
}
__device__ __forceinline__ bool next_segment(const DecodeArgs& a, int& n, int& cum, int A0, int A1,
                                             int& L, int& tiles, int& tb, int& te, int& next_len) {
    return next_segment<kSeqCost>(a, n, cum, A0, A1, L, tiles, tb, te, next_len, a.batch);
}

template <int SEQ = kSeqCost>
__device__ __forceinline__ void finish_segment(int& n, int& cum, int tiles) {
    cum += tiles * kTileCost + SEQ;
    ++n;
}

// The sequence of the CTA's next range after sequence n (cost start cum,
// `tiles` tiles) in its window [A0, A1), or -1 if n is its last.
__device__ __forceinline__ int next_range_seq(const DecodeArgs& a, int n, int cum, int tiles, int A0, int A1) {
    int c = cum + tiles * kTileCost + kSeqCost;
    for (int m = n + 1; m < a.batch && c < A1; ++m) {
        const int t = seq_tiles(__ldg(a.seqlens + m), a.page_size, a.max_pages);
        if (t > 0) {
            if (first_tile_at(c, t, A0) < first_tile_at(c, t, A1)) return m;
            c += t * kTileCost + kSeqCost;
        }
    }
    return -1;
}

// End of the kernel, all threads: the merge of split sequences.
//
// Sequence n with S > 1 splits (CTAs c0..c1) is merged by the CTAs whose
// range ends in it: c0..c1-1 always, c1 when n is also its last sequence.
// Each such CTA waits until all S splits have counted their partials into
// seq_cnt[n], then combines rows [i R / G, (i+1) R / G) of the R = NB * DC
// (branch, latent column) rows, i = c - c0, G the group size:
//   o = out_scale * sum_s w_s o_s / sum_s w_s,  w_s = 2^(lse_s - max_s lse_s)
// per (branch, head) -- the log-sum-exp merge of independent softmax
// partitions, summed in split order.  The S log-sum-exp rows (consecutive
// slots) and each split's slice of partial rows (contiguous) arrive by bulk
// copies.  A CTA leaves the count as soon as its wait is over (the count
// guards only the wait; the partials stay in place until the next launch),
// and the last of the S + G counts returns seq_cnt[n] to zero.  The arithmetic
// is laid out for latency: every thread loads its values for up to 8 splits
// at once before combining them.
template <int NB, int DC, int HP, int THREADS = kThreads>
__device__ __forceinline__ void merge_tail(const DecodeArgs& a, const HeadGroup& grp, int n, int cum, int tiles,
                                           bool c1_member, int chunk, float* w_s, int* flag, uint64_t* bar) {
    constexpr int kHP = HP;
    constexpr int QD = HP / 4;    // head quads of a row
    constexpr int HB = NB * kHP;  // (branch, head) columns of a split's log-sum-exp row
    constexpr int R = NB * DC;    // (branch, latent column) rows
    const int tid = threadIdx.x;
    const int H = a.heads;

    if (n < 0) return;
    int c0, c1;
    seq_owners(cum, tiles, chunk, &c0, &c1);
    const int S = c1 - c0 + 1;
    if (S == 1) return;  // written by the epilogue
    // c1 belongs to the group when no later tile is its own (the next valid
    // sequence starts in a later window); worked out at the range's start
    const int G = c1_member ? S : S - 1;
    const int gi = grp.ci - c0;  // 0 <= gi < G: n is this CTA's last sequence
    const int r0 = (int)((long long)gi * R / G), r1 = (int)((long long)(gi + 1) * R / G);
    const int rows = r1 - r0;
    const size_t slot_c0 = (size_t)grp.slot0 + c0 + n;  // the partial slot of split 0
    int* cnt = a.seq_cnt + grp.cnt0 + n;
    float* part_s = w_s + S * HB;  // [S][rows][16 heads]
    // wait until every split of n has counted its partials
    if (tid == 0) {
        const uint64_t t0 = globaltimer_ns();
        bool ok = true;
        while (ld_acquire_gpu(cnt) < S) {
            if (globaltimer_ns() - t0 > 2000000000ull) {
                ok = false;
                break;
            }
            __nanosleep(32);
        }
        if (!ok) {
            *flag = 2;
            record_error(a.err, MLRA_ERR_DEVICE_TIMEOUT);
        }
    }
    __syncthreads();
    if (*flag & 2) return;
    int departed = 0;
    if (tid < 32) {
        // the partials were published by generic stores and acquired by
        // thread 0 (ordered before this warp by the barrier); the copies read
        // them through the async proxy
        fence_proxy_async_global();
        if (tid == 0) {
            mbar_arrive_expect_tx(bar, (uint32_t)(S * HB + S * rows * kHP) * 4u);
            bulk_load(w_s, a.lse_part + slot_c0 * HB, (uint32_t)(S * HB) * 4u, bar);
        }
        __syncwarp();
        if (rows > 0)
            for (int sp = tid; sp < S; sp += 32)
                bulk_load(part_s + (size_t)sp * rows * kHP, a.o_part + ((slot_c0 + sp) * R + r0) * kHP,
                          (uint32_t)rows * kHP * 4u, bar);
        // this CTA leaves the count (its result is needed only at the end)
        if (tid == 0) departed = atomicAdd(cnt, 1);
    }
    if (!mbar_wait(bar, 0)) {
        // never expected: report it, and give the copies a last bounded
        // chance to land before this CTA's shared memory goes away
        if (tid == 0) record_error(a.err, MLRA_ERR_DEVICE_TIMEOUT);
        mbar_wait(bar, 0, 200000000ull);
        return;
    }
    // weights out_scale * 2^(lse - max) / sum, two threads per (branch, head)
    // column, each over every other split, eight splits' values in flight
    static_assert(2 * HB <= THREADS && HB % 16 == 0, "two threads per column in whole warps");
    if (tid < 2 * HB) {
        const int col = tid >> 1, half = tid & 1;
        float mx = -INFINITY;
        bool bad = false;
        for (int s0 = half; s0 < S; s0 += 16) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s0 + 2 * j < S ? w_s[(s0 + 2 * j) * HB + col] : -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                bad |= v[j] == bad_split_marker();
                if (v[j] != bad_split_marker()) mx = fmaxf(mx, v[j]);
            }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        bad = __shfl_xor_sync(0xffffffffu, (int)bad, 1) != 0 || bad;
        float sum = 0.f;
        for (int s0 = half; s0 < S; s0 += 16) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = s0 + 2 * j < S ? w_s[(s0 + 2 * j) * HB + col] : -INFINITY;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = bad ? 0.f : fast_exp2(v[j] - mx);
                sum += v[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s0 + 2 * j < S) w_s[(s0 + 2 * j) * HB + col] = v[j];
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        const float norm = bad ? 0.f : a.out_scale / sum;
        for (int s0 = half; s0 < S; s0 += 16) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (s0 + 2 * j < S) w_s[(s0 + 2 * j) * HB + col] *= norm;
        }
        if (bad && half == 0 && col % kHP < grp.hn) atomicOr(flag, 1);
    }
    __syncthreads();
    const bool bad = *flag & 1;
    if (bad && tid == 0) record_error(a.err, MLRA_ERR_DEVICE_BAD_INDEX);

    // items (row, head quad), quads fastest: conflict-free 16-byte reads; the
    // weighted sum over the splits in split order, eight splits' loads at once
    for (int e = tid; e < rows * QD; e += THREADS) {
        const int lr = e / QD, q = e % QD, row = r0 + lr;
        const int b = row / DC, k = row % DC;
        const float* w = w_s + b * kHP + 4 * q;
        const float* src = part_s + lr * kHP + 4 * q;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = 0; s0 < S; s0 += 8) {
            float4 v[8], wv[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const bool in = s0 + j < S;
                v[j] = in ? *reinterpret_cast<const float4*>(src + (size_t)(s0 + j) * rows * kHP)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
                wv[j] = in ? *reinterpret_cast<const float4*>(w + (s0 + j) * HB) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                acc.x = fmaf(wv[j].x, v[j].x, acc.x);
                acc.y = fmaf(wv[j].y, v[j].y, acc.y);
                acc.z = fmaf(wv[j].z, v[j].z, acc.z);
                acc.w = fmaf(wv[j].w, v[j].w, acc.w);
            }
        }
        if (bad) acc = make_float4(0.f, 0.f, 0.f, 0.f);
        __nv_bfloat16* dst = a.out + (((size_t)n * H + grp.h0) * NB + b) * DC + k;
        const float v4[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (4 * q + j < grp.hn) dst[(size_t)(4 * q + j) * NB * DC] = to_bf16(v4[j]);
    }
    if (tid == 0 && departed == S + G - 1) *cnt = 0;
}

}  // namespace mlra
