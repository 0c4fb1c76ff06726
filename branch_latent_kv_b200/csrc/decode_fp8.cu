// decode_fp8.cu -- split-KV decode over the 8-bit cache on the sm_100a tensor
// cores (mlra_decode_fp8): mlra_decode with c_b[t] = sigma_b[t / 16] e_b[t],
// e an e4m3 value.
//
// The split plan, the merge and the pipeline are those of decode_tc.cu: one
// persistent CTA per SM walks its tiles of 128 tokens; warp 0 copies, warp 1
// issues the score MMAs, warp 2 the output MMAs, warp 3 looks ahead for
// sequences that need no tile and for the range that ends the CTA's window,
// warps 4 to 19 are the softmax.  What the 8-bit cache changes:
//
// The latents go to the tensor cores as they lie in memory (kind::f8f6f4),
// so a token costs half the shared-memory reads that bound the MMAs here
// (M = 128 and few heads: the latents, operand A, are the traffic) and no
// conversion.  B has to be 8 bits then too, which a query or a probability is
// not; but N is free until the columns cost as much as A does (N = 64 at
// M = 128), so each is split into parts that stand side by side in N:
//  - a query value, scaled so that the largest of its head and branch is at
//    most 448, into hi + lo, both e4m3: 4 + 4 significant bits carry bf16's 8;
//    what the smallest values lose is 2^-10 of a unit of which the largest has
//    224 or more, 2^-17.8 of it.  S = S_hi + S_lo, added when the scores are
//    read; the units are factors of the columns, so that a head's accuracy
//    depends on no other head or branch.
//  - a probability into three e5m2 parts: each takes the leading 3 bits of
//    what is left (the upper byte of a half is an e5m2 value), the last one
//    rounded: 9 significant bits, 2^-9 of it.  e5m2 because its exponent is
//    fp16's; the second and third part are scaled up by 2^2 and 2^5 (their
//    columns are summed apart), so that nothing above 2^-22 is lost.  The largest
//    weight lies at 2^2 .. 2^15; in long ranges, whose flat tails are made of small
//    ones, it is kept higher.
// The value scales go into the probabilities:
//   z_t = log2(e) scale s_t + log2 sigma_t,  w_t = 2^(z_t - M) = p_t sigma_t,
//   o = sum w_t e_t / l,  l = sum w_t / sigma_t,
// with M the running reference of the products p sigma, which are what is
// rounded (a token row's sigma, its logarithm and reciprocal are per-thread
// scalars).  Sums, references and outputs are fp32.
//
// Softmax: four groups of four warps, each the owner of one branch's 16 heads
// (of half of them with two branches, a quarter with one), a thread having
// one token of the tile.  A branch of a tile is one step of the pipeline
// (score MMA, softmax, output MMA), so a chunk of latents leaves its place in
// the ring as soon as its own branch is done.  With half the bytes a tile lasts 1.9 us at HBM's
// rate, less than one group takes for two branches (2.1 us, the two-group
// layout of decode_tc.cu), so the branches are worked on side by side.
// The four warps of a group share the reference M of each head, which a warp
// that meets a score past it has to raise; they vote on that through an
// mbarrier: a warp casts its vote when it has its scores, goes on as if nobody
// needed a raise, and looks at the votes before it hands its weights over (a
// barrier in this place cost a quarter of the step).
//
// Bound by memory in the middle and by latency at both ends.  16 x 8192 tokens
// of four branches, 84.6 MB: 32.6 us back to back (2.6 TB/s): 6.2 us to the
// first references (lengths, plan, table, queries, first tile), then 2.05 us
// per tile of each SM (5.4 TB/s), 4 us for the epilogue and 4 for the merge.
// Longer batches keep more of the rate: 373 MB of ragged lengths 92 us (4.1 TB/s),
// 337 MB of one 512-wide branch 72 us (4.7 TB/s); tensor pipe at 8 and 14 %.
#include <cuda_fp8.h>

#include <cstddef>

#include "common.cuh"
#include "decode_split.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace mlra {
namespace {

constexpr int kHP = 16;       // heads per tile
constexpr int kSN = 2 * kHP;  // score columns of a branch: hi and lo query parts
constexpr int kPN = 3 * kHP;  // output columns of a block: three probability parts
constexpr int kMaxStages = 9;
constexpr int kMaxSteps = 5;
// The reference M sits 2^base below the largest weight when it is set, and is
// raised when a weight passes 2^kTop (e5m2 holds 1.75 2^15).  What is left of a
// weight ends at 2^-22, so a range of n tokens leaves out n 2^-(22 + base) of its
// largest weight at most: base is log2 n - 11, from 2 (n = 2^13) to kBaseMost.
// It is no higher than that asks for, since raises cost: 16 x 8192 tokens 32.7 us
// with 2, 33.9 with 5, 34.6 with 8, the ragged batch 94.9, 96.6, 99.5.  With 2
// throughout, 2^18 tokens 2^24.5 below one of no value came out as zero.
// (kBaseMost is no 8: where fp32's step is 16, a largest score less 8 can round to
// 16 below it, a weight of 2^16.)
constexpr float kTop = 15.0f;
constexpr int kBaseMost = 7;
// Contexts of up to this many tiles are not split: 64 x 500 tokens of four
// branches 17.5 us against 24.3 us split, 1 x 256 of the tiny shape 10.0 against
// 14.4; at eight tiles 4 x 1000 tokens take 26.2 us against 17.4 us split.
constexpr int kWholeTiles = 4;
constexpr int kGroups = 4;                      // softmax groups of four warps
constexpr int kSoft = kGroups * 128;            // softmax threads
constexpr int kFp8Threads = 128 + kSoft;        // and the copy, MMA and helper warps

template <int NB, int DC, int DR>
struct Cfg {
    static constexpr int W = NB * DC;                            // latent bytes per token
    static constexpr int NCH = W / 128;                          // 128-byte chunks of a token row
    static constexpr int BPC = DC >= 128 ? 1 : 128 / DC;         // branches per chunk
    static constexpr int SBR = BPC;                              // branches per step (a chunk is not divided)
    // a range change in cost units of the split plan (a tile is 8): new queries,
    // the first tile's references and an epilogue take about two tiles' time.
    // us at 4, 12, 20 of 16 x 8192 tokens, 64 ragged sequences and 32 x 16384 tokens:
    //   4 x 128  33.3 33.1 32.8   96.8 94.6 92.0   85.8 84.0 85.8
    //   4 x 64   30.2 29.6 28.1   73.9 71.9 71.2   66.5 65.3 65.3
    //   2 x 256  29.7 30.0 29.8   86.7 85.8 85.6   77.0 76.4 78.3
    //   2 x 128  23.1 23.4 23.0   60.1 59.9 59.3   54.2 53.0 54.9
    //   2 x 64   22.0 22.4 22.3   52.0 51.4 49.8   47.6 45.8 45.8
    //   1 x 512  28.4 28.5 28.8   82.7 82.1 81.4   73.0 72.0 73.9
    //   1 x 256  21.7 21.8 22.1   57.0 56.6 56.6   50.8 50.2 51.6
    //   1 x 128  18.5 19.0 18.4   45.4 45.3 45.4   41.4 40.1 41.3
    static constexpr int RANGE_COST = NB == 1 ? 12 : 20;
    static constexpr int HG = kHP * NB / kGroups;                // heads of a softmax group: 16, 8 or 4
    static constexpr int GPB = kGroups / NB;                     // groups per branch
    static constexpr int GPS = GPB * SBR;                        // groups per step
    static constexpr int CPS = SBR * DC / 128;                   // chunks per step
    static constexpr int NSTEP = NB / SBR;                       // steps per tile
    static constexpr int CHUNK_BYTES = kT * 128;
    static constexpr int ROPE_ROW = DR * 2;
    static constexpr int ROPE_BYTES = kT * ROPE_ROW;
    static constexpr int Q_CHUNK_BYTES = kSN * 128;
    static constexpr int Q_BYTES = NCH * Q_CHUNK_BYTES;
    static constexpr int QR_SPAN = (kHP * ROPE_ROW + 1023) / 1024 * 1024;
    static constexpr int P_PART_BYTES = kT * kHP;                // one part of one branch
    static constexpr int P_BRANCH_BYTES = 3 * P_PART_BYTES;
    static constexpr int P_BYTES = SBR * P_BRANCH_BYTES;
    static constexpr int MISC_BYTES = 2560;
    // steps between their score MMA and their output MMA (a tile's and one
    // more); RoPE tiles in flight (more where a tile is a chunk or two); RoPE
    // score slots (one is written again when the steps that read it are over)
    static constexpr int NSP = NSTEP == 4 ? 5 : SBR == 2 ? 3 : 4;
    static constexpr int NROPE = NCH >= 4 ? 2 : NCH == 2 ? 3 : 4;
    static constexpr int NRS = (NSP + 2 * NSTEP - 2) / NSTEP > 2 ? (NSP + 2 * NSTEP - 2) / NSTEP : 2;
    static constexpr int FIXED = NROPE * ROPE_BYTES + Q_BYTES + QR_SPAN + NSP * P_BYTES + MISC_BYTES;
    static constexpr int NSTAGE_FIT = (kSmemLimit - FIXED) / CHUNK_BYTES;
    static constexpr int NSTAGE = NSTAGE_FIT > kMaxStages ? kMaxStages : NSTAGE_FIT;
    static constexpr int OFF_CHUNK = 0;
    static constexpr int OFF_ROPE = OFF_CHUNK + NSTAGE * CHUNK_BYTES;
    static constexpr int OFF_Q = OFF_ROPE + NROPE * ROPE_BYTES;
    static constexpr int OFF_QR = OFF_Q + Q_BYTES;
    static constexpr int OFF_P = OFF_QR + QR_SPAN;
    static constexpr int OFF_MISC = OFF_P + NSP * P_BYTES;
    static constexpr int SMEM_BYTES = OFF_MISC + MISC_BYTES;
    // TMEM columns: output blocks, score slots, RoPE score slots
    static constexpr int O_BLOCKS = NCH * BPC;
    static constexpr int S_COL0 = O_BLOCKS * kPN;
    static constexpr int S_SLOT_COLS = SBR * kSN;
    static constexpr int R_COL0 = S_COL0 + NSP * S_SLOT_COLS;
    static constexpr int COLS = R_COL0 + NRS * kHP;
    static constexpr int TMEM_COLS = COLS <= 128 ? 128 : COLS <= 256 ? 256 : 512;
    static_assert(NRS * NSTEP >= NSP + NSTEP - 1, "a RoPE score is read before its slot is written again");
    static_assert(NB % SBR == 0 && SBR * DC % 128 == 0 && NSTEP * CPS == NCH, "steps fill whole chunks");
    static_assert(CPS >= 1 && NSTAGE >= 2 * CPS && NROPE <= 4 && NSP <= kMaxSteps, "rings");
    static_assert(COLS <= 512 && SMEM_BYTES <= kSmemLimit, "TMEM and shared memory");
    static_assert(Q_BYTES % 1024 == 0 && ROPE_BYTES % 1024 == 0 && P_BYTES % 1024 == 0, "regions stay aligned");
};

struct Misc {
    uint64_t chunk_full[kMaxStages];
    uint64_t chunk_empty[kMaxStages];
    uint64_t rope_full[4];
    uint64_t rope_empty[4];
    uint64_t s_full[kMaxSteps];   // step g in slot g % NSP: its scores are in TMEM
    uint64_t p_full[kMaxSteps];   // its probabilities are in shared memory
    uint64_t p_empty[kMaxSteps];  // its output MMA finished
    uint64_t vote[kGroups];  // a group's four warps have voted on a tile
    uint64_t q_full;      // a range's queries are in shared memory (written by the softmax warps)
    uint64_t drain[2];
    uint64_t merge_full;
    uint32_t tmem_base;
    int abort_flag;
    int plan[4];
    int last_seg[4];
    int merge_flag;
    uint8_t raise[kGroups][2];    // tile t (t & 1): some warp of the group needs a higher reference
    float red[kGroups][4][kHP];       // [group][quadrant][head]: maxima of a raise, at the end sums
    alignas(16) float m_run[kGroups][kHP];  // references M; read as float4
    alignas(16) float q_unit[2][4 * kHP];   // range k in place k % 2: unit of the queries of each [branch][head]
    float factor[kGroups][kHP];       // a raise: what O and l shrink by; at the end 1 / l
};
static_assert(offsetof(Misc, m_run) % 16 == 0 && offsetof(Misc, q_unit) % 16 == 0, "float4 access");

struct Maps {
    CUtensorMap lat;   // latent bytes [pages * P][W]
    CUtensorMap rope;  // RoPE keys [pages * P][d_r]
};

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t e4m3x2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t v) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)v, __NV_E4M3)));
}

// Keeps the uses of loaded TMEM columns below the wait before it.
template <int N>
__device__ __forceinline__ void tie(float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// Two fp32 values as a pair of halves.
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// What a pair of halves has beyond its upper bytes (exact).
__device__ __forceinline__ uint32_t half_rest(uint32_t h) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(h & 0xff00ff00u));
    return r;
}
__device__ __forceinline__ uint32_t half_times(uint32_t h, uint32_t k2) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(k2));
    return r;
}
// The upper bytes of four halves.
__device__ __forceinline__ uint32_t upper_bytes(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7531); }

template <int NB, int DC, int DR>
__global__ void __launch_bounds__(kFp8Threads, 1)
decode_fp8_kernel(const __grid_constant__ Maps maps, const __grid_constant__ DecodeArgs a,
                  const float* __restrict__ latent_scale, const int whole) {
    using C = Cfg<NB, DC, DR>;
    static_assert(sizeof(Misc) <= C::MISC_BYTES, "barriers and scratch fit the MISC region");
    extern __shared__ __align__(1024) uint8_t sm[];  // (the swizzle atoms start at 1024 bytes)
    Misc& misc = *reinterpret_cast<Misc*>(sm + C::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = a.page_size;
    const HeadGroup grp = head_group<kHP>(a);

    if (warp == 0 && lane < 2) prefetch_tensormap(lane == 0 ? &maps.lat : &maps.rope);
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NSTAGE; ++i) mbar_init(&misc.chunk_full[i], 1), mbar_init(&misc.chunk_empty[i], 1);
        for (int i = 0; i < C::NROPE; ++i) mbar_init(&misc.rope_full[i], 1), mbar_init(&misc.rope_empty[i], 1);
        for (int i = 0; i < C::NSP; ++i) {
            mbar_init(&misc.s_full[i], 1);
            mbar_init(&misc.p_full[i], 4 * C::GPS);
            mbar_init(&misc.p_empty[i], 1);
        }
        for (int g = 0; g < kGroups; ++g) {
            mbar_init(&misc.vote[g], 4);
            misc.raise[g][0] = misc.raise[g][1] = 0;
        }
        mbar_init(&misc.q_full, 4 * kGroups);
        mbar_init(&misc.drain[0], 1);
        mbar_init(&misc.drain[1], 1);
        mbar_init(&misc.merge_full, 1);
        misc.abort_flag = 0;
        misc.last_seg[0] = -1;
        misc.merge_flag = 0;
        fence_barrier_init();
    }
    launch_dependents();
    // warp 0 computes the plan and goes on to its copies; the others meet it
    int n_first, cum_first;
    if (warp == 0) {
        wait_prerequisite_grid();
        if (whole) {
            n_first = grp.ci;
            cum_first = 0;
            if (lane == 0) misc.plan[1] = 1 << 28, misc.plan[2] = n_first, misc.plan[3] = 0;
            __syncwarp();
            named_bar_arrive<2, kFp8Threads>();
        } else {
        const int total = warp_cost_prefix<C::RANGE_COST>(a.seqlens, a.batch, P, a.max_pages);
        const int chunk = plan_chunk(total, grp.cpg);
        n_first = a.batch;
        cum_first = total;
        if (!grp.idle && (long long)grp.ci * chunk < total)
            warp_find_seq<C::RANGE_COST>(a.seqlens, a.batch, P, a.max_pages, grp.ci * chunk, &n_first, &cum_first);
        if (lane == 0) {
            misc.plan[1] = chunk;
            misc.plan[2] = n_first;
            misc.plan[3] = cum_first;
        }
        __syncwarp();
        named_bar_arrive<2, kFp8Threads>();
        }
    } else {
        if (warp == 1) {
            tmem_alloc(&misc.tmem_base, C::TMEM_COLS);
            tmem_relinquish();
        }
        tc_fence_before();
        named_bar_sync<2, kFp8Threads>();
        tc_fence_after();
        wait_prerequisite_grid();
        n_first = misc.plan[2];
        cum_first = misc.plan[3];
        if (warp == 3) {
            // sequences with an invalid length: zeros and an error code
            for (int m = blockIdx.x; m < a.batch; m += a.num_ctas) {
                if (seq_tiles(__ldg(a.seqlens + m), P, a.max_pages) > 0) continue;
                uint4* dst = reinterpret_cast<uint4*>(a.out + (size_t)m * a.heads * C::W);
                for (int e = lane; e < a.heads * C::W / 8; e += 32) dst[e] = make_uint4(0u, 0u, 0u, 0u);
                if (lane == 0) record_error(a.err, MLRA_ERR_DEVICE_BAD_SEQLEN);
            }
        }
    }
    const int chunk = misc.plan[1];
    const int A0 = whole ? 0 : grp.ci * chunk, A1 = A0 + chunk;  // this CTA's cost window
    const int seq_end = whole ? n_first + 1 : a.batch;           // and the sequences it may reach
    const uint32_t tmem = misc.tmem_base;            // (warp 0 never uses it)
    volatile int* abort_flag = &misc.abort_flag;

    if (n_first < a.batch) {
        int n = n_first, cum = cum_first, next_len = first_len(a, n);
        int L, tiles, tb, te;
        if (warp == 0) {
            // ------------------------------------------------------------ producer
            uint32_t cc = 0, tc = 0;  // chunks and tiles issued
            const uint64_t policy = grp.cpg == a.num_ctas ? l2_policy_evict_first() : l2_policy_evict_normal();
            bool ok = true;
            while (ok && next_segment<C::RANGE_COST>(a, n, cum, A0, A1, L, tiles, tb, te, next_len, seq_end)) {
                const int32_t* bt = a.block_table + (size_t)n * a.max_pages;
                int win_base = tb * kT / P, win_val = 0;  // 32 block-table entries, one per lane
                if (win_base + lane < a.max_pages) win_val = __ldg(bt + win_base + lane);
                win_val = (win_val >= 0 && win_val < a.num_pages) ? win_val : 0;  // (the softmax warps report bad ones)
                for (int j = tb; j < te && ok; ++j) {
                    const int tok0 = j * kT;
                    const int npages = ceil_div(min(kT, L - tok0), P);
                    const int page0 = tok0 / P;
                    if (page0 + npages > win_base + 32) {
                        win_base = page0;
                        const int v = page0 + lane < a.max_pages ? __ldg(bt + page0 + lane) : 0;
                        win_val = (v >= 0 && v < a.num_pages) ? v : 0;
                    }
                    const int rs = tc % C::NROPE;
                    if (lane == 0) {
                        if (tc >= (uint32_t)C::NROPE) ok = mbar_wait(&misc.rope_empty[rs], ((tc / C::NROPE) - 1) & 1);
                        if (ok) mbar_arrive_expect_tx(&misc.rope_full[rs], npages * P * C::ROPE_ROW);
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    for (int q = 0; q < npages; ++q) {
                        const int page = __shfl_sync(0xffffffffu, win_val, page0 + q - win_base);
                        if (lane == 0)
                            tma_load_2d_hint(sm + C::OFF_ROPE + rs * C::ROPE_BYTES + q * P * C::ROPE_ROW, &maps.rope, 0,
                                             page * P, &misc.rope_full[rs], policy);
                    }
                    ++tc;
                    for (int c = 0; c < C::NCH && ok; ++c) {
                        const int stage = cc % C::NSTAGE;
                        if (lane == 0) {
                            ok = mbar_wait(&misc.chunk_empty[stage], ((cc / C::NSTAGE) & 1) ^ 1);
                            if (ok) mbar_arrive_expect_tx(&misc.chunk_full[stage], npages * P * 128);
                        }
                        ok = __shfl_sync(0xffffffffu, ok, 0);
                        if (!ok) break;
                        for (int q = 0; q < npages; ++q) {
                            const int page = __shfl_sync(0xffffffffu, win_val, page0 + q - win_base);
                            if (lane == 0)
                                tma_load_2d_hint(sm + C::OFF_CHUNK + stage * C::CHUNK_BYTES + q * P * 128, &maps.lat, c * 128,
                                                 page * P, &misc.chunk_full[stage], policy);
                        }
                        ++cc;
                    }
                    ok = __shfl_sync(0xffffffffu, ok && !*abort_flag, 0);
                }
                finish_segment<C::RANGE_COST>(n, cum, tiles);
            }
            if (lane == 0) {
                if (!ok) {
                    record_error(a.err, MLRA_ERR_DEVICE_TIMEOUT);
                    *abort_flag = 1;
                }
                // no copy may land after this CTA has exited
                for (uint32_t i = 0; i < (uint32_t)C::NSTAGE && i < cc; ++i) {
                    const uint32_t k = cc - 1 - i;
                    mbar_wait(&misc.chunk_full[k % C::NSTAGE], (k / C::NSTAGE) & 1, 200000000ull);
                }
                for (uint32_t i = 0; i < (uint32_t)C::NROPE && i < tc; ++i) {
                    const uint32_t k = tc - 1 - i;
                    mbar_wait(&misc.rope_full[k % C::NROPE], (k / C::NROPE) & 1, 200000000ull);
                }
            }
        } else if (warp == 1) {
            // ------------------------------------------------------------ score MMAs
            constexpr uint32_t ID_S = idesc_f8_f32(128, kSN, kE4M3, kE4M3, false, false);
            constexpr uint32_t ID_R = idesc_bf16_f32(128, kHP, false, false);
            const uint32_t base = smem_u32(sm);
            const uint64_t dA = smem_desc(base + C::OFF_CHUNK, 16, 1024, kLayoutSw128);  // K-major
            const uint64_t dQ = smem_desc(base + C::OFF_Q, 16, 1024, kLayoutSw128);
            const uint64_t dQR = rope_desc<DR>(base + C::OFF_QR);
            const uint64_t dR = rope_desc<DR>(base + C::OFF_ROPE);
            uint32_t gs = 0, tc = 0, sc = 0, stage = 0, phase = 0;
            bool ok = true;
            while (ok && next_segment<C::RANGE_COST>(a, n, cum, A0, A1, L, tiles, tb, te, next_len, seq_end)) {
                ok = mbar_wait_warp(&misc.q_full, sc & 1);
                tc_fence_after();
                for (int j = tb; j < te && ok; ++j) {
                    const uint32_t rs = tc % C::NROPE;
                    ok = mbar_wait_warp(&misc.rope_full[rs], (tc / C::NROPE) & 1);
#pragma unroll 1
                    for (int st = 0; st < C::NSTEP && ok; ++st) {
                        ok = mbar_wait_warp(&misc.chunk_full[stage], phase);
                        const uint32_t slot = gs % C::NSP;
                        if (ok && gs >= (uint32_t)C::NSP) ok = mbar_wait_warp(&misc.p_empty[slot], ((gs / C::NSP) - 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        if (st == 0) {
                            // RoPE score of the tile, shared by every branch
                            const uint32_t d = tmem + C::R_COL0 + (tc % C::NRS) * kHP;
                            const uint64_t k0 = dR + ((rs * C::ROPE_BYTES) >> 4);
#pragma unroll
                            for (int kk = 0; kk < DR / 16; ++kk)
                                if (elect_one()) mma_bf16(d, k0 + kk * 2, dQR + kk * 2, ID_R, kk ? 1u : 0u);
                            if (elect_one()) mma_commit(&misc.rope_empty[rs]);
                            __syncwarp();
                        }
                        const uint32_t dS = tmem + C::S_COL0 + slot * C::S_SLOT_COLS;
#pragma unroll 1
                        for (int c = 0; c < C::CPS && ok; ++c) {
                            if (c > 0) {
                                ok = mbar_wait_warp(&misc.chunk_full[stage], phase);
                                if (!ok) break;
                                tc_fence_after();
                            }
                            const uint64_t a0 = dA + ((stage * C::CHUNK_BYTES) >> 4);
                            const uint64_t q0 = dQ + (((st * C::CPS + c) * C::Q_CHUNK_BYTES) >> 4);
                            // 32 bytes (K) at a time; the chunk's branch (or, of two, the one of its half)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const int g = DC == 64 ? kk / 2 : c * 128 / DC;
                                const bool first = DC == 64 ? kk % 2 == 0 : c * 128 % DC == 0 && kk == 0;
                                if (elect_one()) mma_f8(dS + g * kSN, a0 + kk * 2, q0 + kk * 2, ID_S, first ? 0u : 1u);
                            }
                            if (++stage == (uint32_t)C::NSTAGE) stage = 0, phase ^= 1;
                        }
                        if (!ok) break;
                        if (elect_one()) mma_commit(&misc.s_full[slot]);
                        __syncwarp();
                        ++gs;
                    }
                    ++tc;
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) ok = false;
                }
                ++sc;
                finish_segment<C::RANGE_COST>(n, cum, tiles);
            }
            if (!ok && lane == 0) {
                record_error(a.err, MLRA_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
            }
            if (elect_one()) mma_commit(&misc.drain[0]);
            __syncwarp();
            mbar_wait(&misc.drain[0], 0, 200000000ull);
            __syncwarp();
        } else if (warp == 2) {
            // ------------------------------------------------------------ output MMAs
            constexpr uint32_t ID_O = idesc_f8_f32(128, kPN, kE4M3, kE5M2, true, true);
            const uint32_t base = smem_u32(sm);
            // A: the chunk as [128 latent columns][tokens], MN-major (a token row is one
            // 128-byte swizzle row); B: 16 heads x 8 tokens core matrices, MN-major
            const uint64_t dA = smem_desc(base + C::OFF_CHUNK, C::CHUNK_BYTES, 1024, kLayoutSw128);
            const uint64_t dP = smem_desc(base + C::OFF_P, 128, C::P_PART_BYTES, kLayoutNone);
            uint32_t gs = 0, stage = 0;
            bool ok = true;
            while (ok && next_segment<C::RANGE_COST>(a, n, cum, A0, A1, L, tiles, tb, te, next_len, seq_end)) {
                for (int j = tb; j < te && ok; ++j) {
#pragma unroll 1
                    for (int st = 0; st < C::NSTEP; ++st) {
                        const uint32_t slot = gs % C::NSP;
                        ok = mbar_wait_warp(&misc.p_full[slot], (gs / C::NSP) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t b0 = dP + ((slot * C::P_BYTES) >> 4);
#pragma unroll
                        for (int c = 0; c < C::CPS; ++c) {
                            const uint64_t a0 = dA + ((stage * C::CHUNK_BYTES) >> 4);
#pragma unroll
                            for (int g2 = 0; g2 < C::BPC; ++g2) {
                                // branch of the step whose P multiplies this chunk (the rows of a
                                // shared chunk's other branch are left out later)
                                const int g = DC == 64 ? g2 : c * 128 / DC;
                                const uint32_t d = tmem + ((st * C::CPS + c) * C::BPC + g2) * kPN;
#pragma unroll
                                for (int kt = 0; kt < kT / 32; ++kt)
                                    if (elect_one())
                                        mma_f8(d, a0 + (kt * 4096 >> 4), b0 + ((g * C::P_BRANCH_BYTES + kt * 512) >> 4), ID_O,
                                               (j == tb && kt == 0) ? 0u : 1u);
                            }
                            if (elect_one()) mma_commit(&misc.chunk_empty[stage]);
                            if (++stage == (uint32_t)C::NSTAGE) stage = 0;
                        }
                        if (elect_one()) mma_commit(&misc.p_empty[slot]);
                        __syncwarp();
                        ++gs;
                    }
                    if (__shfl_sync(0xffffffffu, *abort_flag, 0)) ok = false;
                }
                finish_segment<C::RANGE_COST>(n, cum, tiles);
            }
            if (!ok && lane == 0) {
                record_error(a.err, MLRA_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
            }
            if (elect_one()) mma_commit(&misc.drain[1]);
            __syncwarp();
            mbar_wait(&misc.drain[1], 0, 200000000ull);
            __syncwarp();
        } else if (warp == 3) {
            // ------------------------------------------------------------ the merge's sequence
            // this CTA's last range, and whether the owner of its last tile merges it
            // (as in decode_tc.cu: no later sequence starts in that window)
            int last_n = -1, last_cum = 0, last_tiles = 0;
            while (next_segment<C::RANGE_COST>(a, n, cum, A0, A1, L, tiles, tb, te, next_len, seq_end)) {
                last_n = n, last_cum = cum, last_tiles = tiles;
                finish_segment<C::RANGE_COST>(n, cum, tiles);
            }
            if (lane == 0 && last_n >= 0) {
                int c1_member = 1;
                const int c1 = (last_cum + (last_tiles - 1) * kTileCost) / chunk;
                for (int m = last_n + 1; m < a.batch; ++m) {
                    if (seq_tiles(__ldg(a.seqlens + m), P, a.max_pages) == 0) continue;
                    c1_member = (last_cum + last_tiles * kTileCost + C::RANGE_COST) / chunk != c1;
                    break;
                }
                misc.last_seg[0] = last_n;
                misc.last_seg[1] = last_cum;
                misc.last_seg[2] = last_tiles;
                misc.last_seg[3] = c1_member;
            }
        } else if (warp >= 4) {
            // ------------------------------------------------------------ queries, softmax, epilogue
            constexpr int HG = C::HG;
            const int sg = (warp - 4) >> 2;                  // softmax group
            const int br = sg / C::GPB;                      // its branch
            const int hoff = HG * (sg % C::GPB);             // its first head
            const int st = br / C::SBR, bsel = br % C::SBR;  // the branch's step in a tile, its place in the step
            const uint32_t gbar = 8 + sg;                    // its named barrier (128 threads)
            const int quad = warp & 3;                       // TMEM lane quadrant
            const int row = quad * 32 + lane;                // token (S) / latent column (O); also the thread's number in the group
            const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
            const int H = a.heads, log_p = __ffs(P) - 1;     // (P is a power of two)
            uint32_t tcnt = 0, ranges = 0;
            bool dead = false;
            int pend_a = -1, pend_b = -1;

            // A range: its tiles, and what this thread has in hand when they begin:
            // its token's page one tile ahead, its scale, and its heads' query units.
            struct Range {
                int n, cum, L, tiles, tb, te;
                int page_next;
                float sig;
                const float* unit;
                bool bad;
            };
            auto page_of = [&](const Range& r, int j) {
                return j < r.te && j * kT + row < r.L ? __ldg(a.block_table + (size_t)r.n * a.max_pages + ((j * kT + row) >> log_p)) : 0;
            };
            auto scale_of = [&](Range& r, int page, int j) {
                const bool real = page >= 0 && page < a.num_pages;
                r.bad |= !real;
                return __ldg(latent_scale + (((size_t)(real ? page : 0) << log_p) + ((j * kT + row) & (P - 1))) / kFp8Block * NB + br);
            };
            // The next range, its queries split and written to shared memory (all
            // groups; their score MMAs of the range before are over).  False: none is
            // left, or a group has given up.
            auto begin_range = [&](Range& r) {
                if (!next_segment<C::RANGE_COST>(a, n, cum, A0, A1, L, tiles, tb, te, next_len, seq_end)) return false;
                r.n = n, r.cum = cum, r.L = L, r.tiles = tiles, r.tb = tb, r.te = te, r.bad = false;
                finish_segment<C::RANGE_COST>(n, cum, tiles);
                const int page = page_of(r, r.tb);
                r.page_next = page_of(r, r.tb + 1);
                // 16 head rows; heads past the last are zero
                constexpr int UPR = C::W / 8;               // 8-value units per head row
                constexpr int UNITS = kHP * UPR;
                constexpr int U = (UNITS + kSoft - 1) / kSoft;  // units of a thread, side by side
                constexpr int SEG = DC / 8 / U;             // threads of one head and branch
                static_assert(SEG <= 32 && SEG * U * 8 == DC, "a warp has whole heads of a branch");
                const int sid = threadIdx.x - 128, h = sid * U / UPR, u0 = sid * U % UPR;
                const bool some = sid * U < UNITS && h < grp.hn;
                const uint4* q = reinterpret_cast<const uint4*>(a.q_lat + ((size_t)r.n * H + grp.h0 + h) * C::W) + u0;
                uint4 v[U];
#pragma unroll
                for (int i = 0; i < U; ++i) v[i] = some ? __ldg(q + i) : make_uint4(0u, 0u, 0u, 0u);
                constexpr int RU = DR / 8;                  // 16-byte units of a RoPE row
                uint4 rv = make_uint4(0u, 0u, 0u, 0u);
                if (sid < kHP * RU && sid / RU < grp.hn)
                    rv = __ldg(reinterpret_cast<const uint4*>(a.q_rope + ((size_t)r.n * H + grp.h0 + sid / RU) * DR) + sid % RU);
                // the largest finite magnitude of the head and branch, as 16-bit integers
                uint32_t mx = 0;
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
                        mx = max(mx, lo < 0x7f80u ? lo : 0u);
                        mx = max(mx, hi < 0x7f80u ? hi : 0u);
                    }
                }
                if constexpr (SEG == 32) mx = __reduce_max_sync(0xffffffffu, mx);
                else
#pragma unroll
                for (int o = SEG / 2; o > 0; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                // their unit: the smallest power of two tau with mx <= 448 tau (2^-100 at
                // least: both it and its reciprocal are normal numbers)
                const int e = max((int)(mx >> 7) - 135 + ((mx & 0x7fu) > 0x60u), -100);
                const float inv_tau = __uint_as_float((uint32_t)(127 - e) << 23);
                // (the other place holds the units of the range that slower groups are in)
                float* unit = misc.q_unit[ranges++ & 1];
                if (sid * U < UNITS && sid % SEG == 0) unit[u0 * 8 / DC * kHP + h] = __uint_as_float((uint32_t)(127 + e) << 23);
                r.unit = unit + br * kHP + hoff;
                // (every group comes here for every range, also one that has given up:
                // then all stop)
                if (named_bar_or<5, kSoft>(dead)) {
                    dead = true;
                    return false;
                }
                r.sig = scale_of(r, page, r.tb);
                if (sid < kHP * RU) {
                    const int h = sid / RU, u = sid % RU;
                    *reinterpret_cast<uint4*>(sm + C::OFF_QR + (DR == 64 ? h * 128 + ((u ^ (h & 7)) << 4) : h * 64 + ((u ^ ((h >> 1) & 3)) << 4))) = rv;
                }
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const int col = (u0 + i) * 8;
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x = __uint_as_float(w[k] << 16) * inv_tau, y = __uint_as_float(w[k] & 0xffff0000u) * inv_tau;
                        x = fmaf(x, 0.f, x);  // infinities become NaN: the head's scores are NaN as in full precision
                        y = fmaf(y, 0.f, y);
                        hi[k] = e4m3x2(x, y);
                        const float2 f = from_e4m3x2(hi[k]);
                        lo[k] = e4m3x2(x - f.x, y - f.y);
                    }
                    if (sid * U < UNITS) {
                        uint8_t* dst = sm + C::OFF_Q + col / 128 * C::Q_CHUNK_BYTES + h * 128 +
                                       (((col % 128 / 16) ^ (h & 7)) << 4) + col % 16;
                        *reinterpret_cast<uint2*>(dst) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                        *reinterpret_cast<uint2*>(dst + kHP * 128) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&misc.q_full);
                return true;
            };

            Range rg;
            bool more = begin_range(rg);
            while (more) {  // (a group that has given up goes on to the barrier in begin_range)
                const int tb = rg.tb, te = rg.te;
                const float* unit = rg.unit;
                // (four units stay in registers: one 512-wide branch 72.4 us against 74.0; with
                // eight or sixteen heads they cost more there: 16 x 8192 tokens 35.0 us from 32.8)
                float tau4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) tau4[i] = unit[i];
                int page_next = rg.page_next;
                float sig = rg.sig, sig_next = 0.f;
                float l[HG];  // this thread's share of sum w / sigma
#pragma unroll
                for (int i = 0; i < HG; ++i) l[i] = 0.f;

                for (int j = tb; j < te && !dead; ++j, ++tcnt) {
                    const uint32_t gs = tcnt * C::NSTEP + st, slot = gs % C::NSP, parity = (gs / C::NSP) & 1;
                    const bool masked = j * kT + row >= rg.L;
                    const int page_after = page_of(rg, j + 2);
                    if (j + 1 < te) sig_next = scale_of(rg, page_next, j + 1);
                    page_next = page_after;
                    const float ls = fast_log2(sig), k = sig * a.scale_log2;  // a score of the MMAs times k and its unit is in log2 units
                    const float rs = masked ? 0.f : __frcp_rn(sig);
                    // z: log2 of p sigma per head
                    float z[HG];
                    auto read_scores = [&]() {
                        constexpr int N = HG < 8 ? HG : 8;  // heads at a time (registers)
                        const uint32_t s_at = lanes + C::S_COL0 + slot * C::S_SLOT_COLS + bsel * kSN + hoff;
                        const uint32_t r_at = lanes + C::R_COL0 + (tcnt % C::NRS) * kHP + hoff;
#pragma unroll
                        for (int i0 = 0; i0 < HG; i0 += N) {
                            float tau[N], hi[N], low[N], r[N];
#pragma unroll
                            for (int i = 0; i < N; ++i) tau[i] = HG == 4 ? tau4[i] : unit[i0 + i];
                            tmem_ld_cols<N>(r_at + i0, r);
                            tmem_ld_cols<N>(s_at + i0, hi);
                            tmem_ld_cols<N>(s_at + kHP + i0, low);
                            tmem_wait_ld();
                            tie(r), tie(hi), tie(low);
#pragma unroll
                            for (int i = 0; i < N; ++i) z[i0 + i] = fmaf(hi[i] + low[i], k * tau[i], fmaf(r[i], a.scale_log2, ls));
                        }
                        if (masked) {
#pragma unroll
                            for (int i = 0; i < HG; ++i) z[i] = -INFINITY;
                        }
                    };
                    auto less_references = [&]() {
#pragma unroll
                        for (int i = 0; i < HG; i += 4) {
                            const float4 m = *reinterpret_cast<const float4*>(&misc.m_run[sg][i]);
                            z[i] -= m.x;
                            z[i + 1] -= m.y;
                            z[i + 2] -= m.z;
                            z[i + 3] -= m.w;
                        }
                    };
                    // w = 2^z (z less its reference) and its three parts into shared
                    // memory (core matrices of 16 heads x 8 tokens)
                    auto write_weights = [&]() {
                        uint32_t h[HG / 2];
#pragma unroll
                        for (int i = 0; i < HG; i += 2) {
                            z[i] = fast_exp2(z[i]);
                            z[i + 1] = fast_exp2(z[i + 1]);
                            h[i / 2] = pack_half(z[i], z[i + 1]);
                        }
                        uint8_t* dst = sm + C::OFF_P + slot * C::P_BYTES + bsel * C::P_BRANCH_BYTES + (row >> 3) * 128 + (row & 7) * 16 + hoff;
#pragma unroll
                        for (int part = 0; part < 3; ++part) {
                            if (part > 0) {
#pragma unroll
                                for (int i = 0; i < HG / 2; ++i) {
                                    // (exact: times 4, times 8; the last part is rounded, not cut)
                                    h[i] = half_times(half_rest(h[i]), part == 1 ? 0x44004400u : 0x48004800u);
                                    if (part == 2) h[i] += 0x00800080u;
                                }
                            }
                            if constexpr (HG == 16)
                                *reinterpret_cast<uint4*>(dst + part * C::P_PART_BYTES) =
                                    make_uint4(upper_bytes(h[0], h[1]), upper_bytes(h[2], h[3]), upper_bytes(h[4], h[5]), upper_bytes(h[6], h[7]));
                            else if constexpr (HG == 8)
                                *reinterpret_cast<uint2*>(dst + part * C::P_PART_BYTES) =
                                    make_uint2(upper_bytes(h[0], h[1]), upper_bytes(h[2], h[3]));
                            else
                                *reinterpret_cast<uint32_t*>(dst + part * C::P_PART_BYTES) = upper_bytes(h[0], h[1]);
                        }
                    };

                    const bool ok = mbar_wait(&misc.s_full[slot], parity);
                    tc_fence_after();
                    read_scores();
                    bool raise = j == tb;  // the first tile sets the references
                    if (!raise) {
                        less_references();
                        float top = z[0];
#pragma unroll
                        for (int i = 1; i < HG; ++i) top = fmaxf(top, z[i]);
                        const bool need = __any_sync(0xffffffffu, top > kTop || !ok);
                        if (lane == 0) {
                            if (need) *reinterpret_cast<volatile uint8_t*>(&misc.raise[sg][tcnt & 1]) = 1;
                            mbar_arrive(&misc.vote[sg]);
                        }
                        write_weights();
                    } else if (lane == 0) {
                        mbar_arrive(&misc.vote[sg]);
                    }
                    // (every warp votes: what it waits for before is bounded well below this)
                    const bool ok1 = mbar_wait(&misc.vote[sg], tcnt & 1, 8000000000ull);
                    raise |= *reinterpret_cast<volatile uint8_t*>(&misc.raise[sg][tcnt & 1]) != 0;
                    if (!ok1 || raise) {
                        // all four warps: exact column maxima, new references, O and l at
                        // them, the weights again
                        if (!ok1 || named_bar_or_id<128>(gbar, !ok)) {
                            dead = true;
                            break;
                        }
                        if (j > tb) read_scores();
                        constexpr int SPAN = 32 / HG;
                        const float v = warp_colmax<HG>(z, lane);
                        if ((lane & (SPAN - 1)) == 0) misc.red[sg][quad][lane / SPAN] = v;
                        if (row == 0) misc.raise[sg][tcnt & 1] = 0;  // (all have read it before the barrier above)
                        named_bar_sync_id<128>(gbar);
                        if (row < HG) {
                            const int base = min(max(28 - __clz(te - tb - 1), 2), kBaseMost);  // log2 of the range's tokens less 11
                            const float t = fmaxf(fmaxf(misc.red[sg][0][row], misc.red[sg][1][row]),
                                                  fmaxf(misc.red[sg][2][row], misc.red[sg][3][row])) - (float)base;
                            const float m = misc.m_run[sg][row], mnew = j == tb ? t : fmaxf(m, t);
                            misc.factor[sg][row] = j == tb ? 1.f : fast_exp2(m - mnew);
                            misc.m_run[sg][row] = mnew;  // (all have read the old one before the barrier above)
                        }
                        named_bar_sync_id<128>(gbar);
                        if (j > tb) {
                            // O holds earlier tiles of the range: rescaled once their output MMAs are
                            // done (the last one of this branch is a tile back)
                            const uint32_t before = gs - C::NSTEP;
                            const bool ok2 = mbar_wait(&misc.p_empty[before % C::NSP], (before / C::NSP) & 1);
                            if (named_bar_or_id<128>(gbar, !ok2)) {
                                dead = true;
                                break;
                            }
                            tc_fence_after();
#pragma unroll
                            for (int i = 0; i < HG; ++i) l[i] *= misc.factor[sg][i];
#pragma unroll 1
                            for (int e = 0; e < C::CPS * C::BPC; ++e) {
                                const int c = e / C::BPC, g2 = e % C::BPC;
                                if ((DC == 64 ? g2 : c * 128 / DC) != bsel) continue;
#pragma unroll
                                for (int part = 0; part < 3; ++part) {
                                    const uint32_t at = lanes + ((st * C::CPS + c) * C::BPC + g2) * kPN + part * kHP + hoff;
                                    float o[HG];
                                    tmem_ld_cols<HG>(at, o);
                                    tmem_wait_ld();
                                    tie(o);
#pragma unroll
                                    for (int i = 0; i < HG; ++i) o[i] *= misc.factor[sg][i];
                                    tmem_st_cols<HG>(at, o);
                                }
                            }
                            tmem_wait_st();
                        }
                        read_scores();
                        less_references();
                        write_weights();
                    }
#pragma unroll
                    for (int i = 0; i < HG; ++i) l[i] = fmaf(z[i], rs, l[i]);
                    // rows past the end of the sequence become zero before the output MMA
                    // reads them: each group of the step clears its share of each row
                    if (masked) {
                        constexpr int BYTES = 128 / C::GPS;
#pragma unroll
                        for (int c = 0; c < C::CPS; ++c) {
                            uint8_t* p = sm + C::OFF_CHUNK + ((gs * C::CPS + c) % C::NSTAGE) * C::CHUNK_BYTES + row * 128 + sg % C::GPS * BYTES;
#pragma unroll
                            for (int u = 0; u < BYTES / 16; ++u) *reinterpret_cast<uint4*>(p + u * 16) = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&misc.p_full[slot]);
                    sig = sig_next;
                }
                // the next range's queries now: its scores are made during the epilogue
                const Range rd = rg;
                more = begin_range(rg);
                if (dead) break;

                // ---------------------------------------------------- epilogue
                const int n = rd.n, cum = rd.cum, tiles = rd.tiles;
                {
                    float f[HG];
#pragma unroll
                    for (int i = 0; i < HG; ++i) f[i] = l[i];
                    warp_sum_scatter<HG, 16, HG>(f, lane);
                    constexpr int SPAN = 32 / HG;
                    if ((lane & (SPAN - 1)) == 0) misc.red[sg][quad][lane / SPAN] = f[0];
                }
                const bool bad = named_bar_or_id<128>(gbar, rd.bad);  // also publishes red
                const bool single = cum >= A0 && cum + (tiles - 1) * kTileCost < A1;
                const size_t slot = (size_t)grp.slot0 + grp.ci + n;
                if (row < HG) {
                    const float lt = misc.red[sg][0][row] + misc.red[sg][1][row] + misc.red[sg][2][row] + misc.red[sg][3][row];
                    misc.factor[sg][row] = 1.0f / lt;
                    if (!single)
                        a.lse_part[(slot * NB + br) * kHP + hoff + row] = bad ? bad_split_marker() : misc.m_run[sg][row] + __log2f(lt);
                }
                {
                    const uint32_t last = (tcnt - 1) * C::NSTEP + st;
                    const bool ok = mbar_wait(&misc.p_empty[last % C::NSP], (last / C::NSP) & 1);
                    if (named_bar_or_id<128>(gbar, !ok)) {
                        dead = true;
                        continue;
                    }
                }
                tc_fence_after();
                constexpr int WIDTH = DC >= 128 ? 128 : DC;  // valid rows of an output block
#pragma unroll 1
                for (int e = 0; e < C::CPS * C::BPC; ++e) {
                    const int c = e / C::BPC, g2 = e % C::BPC;
                    if ((DC == 64 ? g2 : c * 128 / DC) != bsel) continue;
                    const uint32_t at = lanes + ((st * C::CPS + c) * C::BPC + g2) * kPN + hoff;
                    const int first = g2 * WIDTH;  // valid rows: this branch's of a shared chunk
                    const bool mine = row >= first && row < first + WIDTH;
                    const int col = DC >= 128 ? c * 128 % DC + row : row - first;  // latent column
                    constexpr int N = HG < 8 ? HG : 8;
#pragma unroll
                    for (int i0 = 0; i0 < HG; i0 += N) {
                        float o[N], o1[N], o2[N];
                        tmem_ld_cols<N>(at + i0, o);
                        tmem_ld_cols<N>(at + kHP + i0, o1);
                        tmem_ld_cols<N>(at + 2 * kHP + i0, o2);
                        tmem_wait_ld();
                        tie(o), tie(o1), tie(o2);
                        if (!mine) continue;
#pragma unroll
                        for (int i = 0; i < N; ++i) o[i] = bad ? 0.f : fmaf(o2[i], 1.f / 32, fmaf(o1[i], 0.25f, o[i])) * misc.factor[sg][i0 + i];
                        if (single) {
                            const int h0 = hoff + i0;
                            __nv_bfloat16* dst = a.out + (((size_t)n * H + grp.h0 + h0) * NB + br) * DC + col;
#pragma unroll
                            for (int i = 0; i < N; ++i)
                                if (h0 + i < grp.hn) dst[(size_t)i * C::W] = to_bf16(o[i] * a.out_scale);
                        } else {
                            float* dst = a.o_part + ((slot * NB + br) * DC + col) * kHP + hoff + i0;
                            if constexpr (N == 4)
                                *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
                            else
                                st_global_v8(dst, o[0], o[1], o[2], o[3], o[4], o[5], o[6], o[7]);
                        }
                    }
                }
                if (bad && row == 0) record_error(a.err, MLRA_ERR_DEVICE_BAD_INDEX);
                tc_fence_before();
                named_bar_sync_id<128>(gbar);  // factor and red are reused by the next range
                if (threadIdx.x == 128 && !single) {
                    if (pend_a < 0) pend_a = n; else pend_b = n;
                }
            }
            if (dead && row == 0) {
                record_error(a.err, MLRA_ERR_DEVICE_TIMEOUT);
                *abort_flag = 1;
            }
            // every group's partial stores, then one release fence, then the counts
            const bool any_dead = named_bar_or<6, kSoft>(dead);
            if (!any_dead && threadIdx.x == 128 && pend_a >= 0) {
                fence_acq_rel_gpu();
                red_add_relaxed_gpu(a.seq_cnt + grp.cnt0 + pend_a, 1);
                if (pend_b >= 0) red_add_relaxed_gpu(a.seq_cnt + grp.cnt0 + pend_b, 1);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
    if (*abort_flag) return;
    merge_tail<NB, DC, kHP, kFp8Threads>(a, grp, misc.last_seg[0], misc.last_seg[1], misc.last_seg[2], misc.last_seg[3] != 0, chunk,
                            reinterpret_cast<float*>(sm + C::OFF_CHUNK), &misc.merge_flag, &misc.merge_full);
}

template <int NB, int DC, int DR>
cudaError_t launch_cfg(const DecodeArgs& a, const float* latent_scale, int whole, cudaStream_t stream) {
    using C = Cfg<NB, DC, DR>;
    Maps maps;
    const uint64_t rows = (uint64_t)a.num_pages * a.page_size;
    if (!encode_rows(&maps.lat, a.latent, 1, C::W, rows, 128, a.page_size, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_rows(&maps.rope, a.rope, 2, DR, rows, DR, a.page_size, rope_swizzle(DR)))
        return cudaErrorInvalidValue;
    auto kernel = decode_fp8_kernel<NB, DC, DR>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
    if (e != cudaSuccess) return e;
    // the merge stages below MISC (the bound of decode_tc.cu)
    for (int S = 2; S <= a.num_ctas; ++S) {
        const size_t share = ((size_t)C::W + S - 2) / (S - 1);
        if (sizeof(float) * ((size_t)S * NB * kHP + S * share * kHP) > (size_t)C::OFF_MISC) return cudaErrorInvalidConfiguration;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.num_ctas);
    cfg.blockDim = dim3(kFp8Threads);
    cfg.dynamicSmemBytes = C::SMEM_BYTES;
    cfg.stream = stream;
    // cooperative where sequences are split: every CTA is resident, so the merge's
    // waits end
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeCooperative;
    attr[1].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = whole ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a, latent_scale, whole);
}

template <int NB, int DC>
cudaError_t launch_shape(const DecodeArgs& a, const float* latent_scale, int whole, cudaStream_t stream) {
    return a.d_r == 64 ? launch_cfg<NB, DC, 64>(a, latent_scale, whole, stream)
                       : launch_cfg<NB, DC, 32>(a, latent_scale, whole, stream);
}

}  // namespace

cudaError_t launch_decode_fp8(const DecodeArgs& args, const float* latent_scale, cudaStream_t stream) {
    DecodeArgs a = args;
    const int groups = ceil_div(a.heads, kHP);
    const long long tiles = ((long long)a.max_pages * a.page_size + kT - 1) / kT;
    // short contexts (by the block table): a CTA takes whole sequences, one each,
    // where there are CTAs for all; nothing is split, so nothing is merged or waited for
    const int whole = tiles <= kWholeTiles && a.batch * (long long)groups <= a.num_ctas;
    if (whole) a.num_ctas = a.batch * groups;
#define MLRA_FP8_CASE(NB_, DC_) \
    if (a.branches == NB_ && a.d_c == DC_) return launch_shape<NB_, DC_>(a, latent_scale, whole, stream);
    MLRA_FP8_CASE(2, 64)
    MLRA_FP8_CASE(4, 64)
    MLRA_FP8_CASE(1, 128)
    MLRA_FP8_CASE(2, 128)
    MLRA_FP8_CASE(4, 128)
    MLRA_FP8_CASE(1, 256)
    MLRA_FP8_CASE(2, 256)
    MLRA_FP8_CASE(1, 512)
#undef MLRA_FP8_CASE
    return cudaErrorInvalidValue;
}

}  // namespace mlra
