// prefill.cu -- causal attention of packed prompt tokens over the paged
// latent cache, on the sm_100a tensor cores (mlra_prefill).
//
// For new token i of a sequence, at position p, head h and branch b
//   s_t = scale * (q_lat[i,h,b] . c_b[t] + q_rope[i,h] . k_r[t]),  t <= p,
//   out[i,h,b] = out_scale * sum_t softmax_t(s)_t c_b[t]
// ("MLRA: Breaking the Sharding Bottleneck in Latent Attention", wispaper.ai
// blog, section "The Core Insight": every branch is attended independently).
// All heads of a branch read the same latents, which are keys and values at
// once, so a branch is one problem with the (token, head) pairs as rows:
//   S = [Q | Qr] [C | Kr]^T,  O += P C,
// rows r = i H + h lying in memory at a constant stride whatever H is.
//
// One CTA per (128 MT rows of a sequence, branch), or, for d_c = 512, a pair:
//   warp 0     finds the CTA's row blocks, one after the other, and copies: Q
//              once a block, then per tile of KT tokens the latents and the
//              keys (one TMA box per page, or part of one) into two rings
//   warp 1     MMAs (tcgen05, one elected thread) and TMEM:
//                S[slot] = Q C^T + Qr Kr^T   K = d_c + d_r, N = KT
//                O += P[slot] C              P from TMEM, the same tile of C as
//                                            MN-major operand, N = VN
//   warp 2     the sequence's pages: all in the pool?
//   warps 4..  softmax, one thread per row (a TMEM lane): one pass with a
//              running maximum and sum; P goes to TMEM as bf16 over the
//              scores it came from; at the end O / sum is written
// Two score slots keep the tensor pipe busy while a softmax runs: the two
// 128-row tiles of a CTA (MT = 2, d_c <= 128) or, where one tile's output
// fills half of TMEM (MT = 1), two consecutive token tiles.  Work item w uses
// slot w % 2; PV(w) and then QK(w + 2) are issued when softmax w is done, and
// because MMAs run in issue order the slot needs no further barrier.
// The running maximum is raised only when a score exceeds it by 2^8 (a row's
// O is rescaled then, by the row's own warp, without a barrier between warps).
//
// The grid has a CTA for each row block, but one that has issued its last copy
// takes the place of one that has not started (cluster launch control): the
// next block's queries, first tiles and first scores come while this one's
// last softmax and its output are under way.  Prompts of 1 to 1024 tokens, 612
// blocks: 49 us, where a new CTA for every block cost 12 us more.  (Where a block's
// tokens are split, each CTA has one block.)
//
// What the widths ask for, with what it measured:
//  - d_c <= 128: tiles of 128 x 128 scores, a row of them in one thread's
//    registers: the softmax warpgroups take registers from the first one.
//  - d_c >= 256: the latent queries live in TMEM (operand A of the score MMA),
//    so shared memory holds latents only, up to four tiles of 64 tokens in flight.
//  - d_c = 512: a row's output does not fit TMEM beside the scores, and two CTAs
//    that each compute all scores for half of the output do 1.5 times the
//    products, out of smaller tiles.  A pair divides the columns for both instead:
//    each CTA has the partial scores of its 256 columns and sends them to the
//    other (st.async to its shared memory), the softmax adds the two.  Two
//    prompts of 3937 tokens together, 16 heads: 603 us with all scores computed
//    twice, 319 as a pair, 252 with the queries in TMEM and the scores sent by
//    warps of their own (8 to 11), 241 with blocks one after the other, 234 with
//    the next block's queries written before this one's output.
//  - few row blocks: a cluster of up to 8 CTAs divides a block's tokens, and
//    joins outputs, maxima and sums over distributed shared memory (one new
//    token after 8191 of four 128-wide branches: 28 us against 129).
//
// Bound by (a rate counts the masked half of the diagonal tiles as nothing):
//  - d_c = 128, 8192 tokens of 16 heads and four branches: 1.09 PFLOP/s in short
//    runs (1073 us), 0.93 under the power cap.  An item's softmax (128 scores a
//    thread, their exponentials on the special-function units) takes 1900 to
//    2600 cycles, its MMAs 1280 and a pair of items 4550: each row tile is a
//    chain, its softmax, its output product, its next scores, of which only the
//    other tile's fills the gaps.  No unit is full: tensor pipe 59 % of the cycles,
//    special functions 48, issue slots 34.
//  - d_c = 512: 2900 cycles per 64 tokens, of which the products are 1500: the
//    exchange of the partial scores is a chain of TMEM read, store, add.
//  - short prompts: 6 us of dependent reads before an SM's first product, its
//    blocks' outputs, and the spread of the SMs' last blocks.
//
// P is rounded to bf16 (the output MMA takes P and C in one type, and C is
// bf16): half a step, 2^-8 of each probability, averaged over the row; the
// sum is of the unrounded ones.  Scores, maxima, sums and O are fp32.
#include <array>

#include "common.cuh"
#include "kernels.h"
#include "sm100.cuh"
#include "tensor_map.cuh"

namespace mlra {
namespace {

using namespace sm100;

constexpr int kSmemMax = 232448;
constexpr float kRescale = 8.0f;  // log2 of how far a score may pass the running maximum

template <int DC, int DR>
struct Cfg {
    static constexpr bool PAIR = DC == 512;             // two CTAs share the columns of a row block
    static constexpr int NV = PAIR ? 2 : 1;             // CTAs per row block and branch
    static constexpr int DL = DC / NV;                  // latent columns of this CTA
    static constexpr int RL = PAIR ? 32 : DR;           // RoPE columns of this CTA
    static constexpr int MT = DL <= 128 ? 2 : 1;        // 128-row tiles per CTA
    static constexpr int KT = DL <= 128 ? 128 : 64;     // tokens per tile
    static constexpr int VN = DL;                       // value columns
    static constexpr int BM = 128 * MT;
    static constexpr int NCH = DL / 64;                 // 64-column (128-byte) chunks of a latent row
    static constexpr int Q_CHUNK = 128 * 128;
    static constexpr int QR_BYTES = 128 * RL * 2;
    static constexpr bool QT = MT == 1;                 // the latent queries live in TMEM, else in shared memory
    static constexpr int Q_LAT = QT ? 0 : NCH * Q_CHUNK;
    static constexpr int Q_TILE = Q_LAT + QR_BYTES;
    static constexpr int C_CHUNK = KT * 128;
    static constexpr int C_BYTES = NCH * C_CHUNK;
    static constexpr int K_BYTES = KT * RL * 2;
    static constexpr int X_BYTES = PAIR ? 128 * KT * 4 : 0;  // the other CTA's share of an item's scores (two slots)
    static constexpr int MISC = 1024;
    // ring depths: the tile a PV reads, the one the next QK reads, and what
    // fits beyond
    static constexpr int NK = DC == 64 ? 4 : DC >= 256 ? 3 : 2;
    static constexpr int NC_FIT = (kSmemMax - 1024 - MISC - MT * Q_TILE - NK * K_BYTES - 2 * X_BYTES) / C_BYTES;
    static constexpr int NC = NC_FIT > 4 ? 4 : NC_FIT;
    static constexpr int OFF_Q = 0;  // Q tile m: chunks, then its RoPE part
    static constexpr int OFF_C = MT * Q_TILE;
    static constexpr int OFF_K = OFF_C + NC * C_BYTES;
    static constexpr int OFF_X = OFF_K + NK * K_BYTES;
    static constexpr int OFF_MISC = OFF_X + 2 * X_BYTES;
    static constexpr int SMEM = OFF_MISC + MISC + 1024;
    // TMEM columns: two score slots, then the output tiles
    static constexpr int S_COLS = KT;
    static constexpr int O_COL = 2 * S_COLS;
    static constexpr int Q_COL = O_COL + MT * VN;       // QT: [rows][d_c / 2], pairs of bf16
    static constexpr int COLS = Q_COL + (QT ? DL / 2 : 0);
    static constexpr int TMEM_COLS = COLS <= 256 ? 256 : 512;
    static constexpr int SOFT_WARPS = 4 * MT;
    static constexpr int THREADS = 128 + 32 * SOFT_WARPS + (PAIR ? 128 : 0);
    // (the next scores' tile is waited for ahead of the PV before it, whose tile
    // must not be the one that makes room for it)
    static_assert((MT == 2 || NC >= 3) && NC >= 2 && SMEM <= kSmemMax, "shared memory");
    static_assert(COLS <= 512, "TMEM");
    static_assert(Q_TILE % 1024 == 0 && C_CHUNK % 1024 == 0 && K_BYTES % 1024 == 0, "swizzle atoms stay aligned");
};

// Registers of the two softmax warpgroups (a row of 128 scores each thread)
// and of the first warpgroup, out of what the block was launched with: 3 x 128
// threads of at most 168.
constexpr int kSoftRegs = 200, kOtherRegs = 104;
static_assert(128 * (2 * kSoftRegs + kOtherRegs) <= 3 * 128 * 168, "the split fits the launch");

// A row block: sequence (-1: no more), first row in it, rows, first packed row,
// tokens before the new ones (-1: zeros), branch, tokens that some row sees; the
// tiles and the row blocks with queries that this CTA had before it.
struct Job {
    int n, row0, rows, out0, past, b, kv_end;
    uint32_t tiles, asked;
};

struct Misc {
    uint64_t c_full[4], c_empty[4];
    uint64_t k_full[4], k_empty[4];
    uint64_t s_full[2];   // item w in slot w % 2: its scores are in TMEM
    uint64_t p_full[2];   // its probabilities are in TMEM
    uint64_t o_done[2];   // its output MMA has finished (MT = 2: the last item's only, as s_full of
                          // item w + 2 says so of the others: its MMAs come after PV(w))
    // a pair, per item: the other CTA's scores are here; they are read here; they
    // are read there; this CTA's are read out of TMEM for sending
    uint64_t x_full[2], x_read[2], x_empty[2], x_taken[2];
    uint64_t q_tmem;  // QT: the latent queries are in TMEM
    uint64_t q_full, q_empty;  // the queries in shared memory; every score MMA of the row block has read them
    // row block k of this CTA in place k % 2: it is known; its pages are checked; every reader is done with it
    uint64_t job_full[2], checked[2], job_empty[2];
    // answers to requests for another CTA's place are here; a pair, whose second CTA
    // hears them from the first: they have been read there
    uint64_t next_full[2], next_read[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
    int bad[2];  // a page of the sequence lies outside the pool
    Job job[2];
    alignas(16) uint32_t next[2][4];
};

struct Maps {
    CUtensorMap q, qr, lat, rope;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// Pairs of fp32 in one 64-bit register, for the packed FMA and add.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
    return r;
}
__device__ __forceinline__ uint64_t pack2(float lo, float hi) { return pack2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    uint32_t a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(v));
    lo = __uint_as_float(a);
    hi = __uint_as_float(b);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One step of a 4 x 4 transpose of 16-byte pieces o[4 k ..] between the lanes of
// a group of four: lanes BIT apart exchange the pieces whose index differs in BIT.
template <int BIT>
__device__ __forceinline__ void swap_quarters(uint32_t* o, int lane) {
    const bool hi = lane & BIT;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (k & BIT) continue;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint32_t &x = o[4 * k + u], &y = o[4 * (k | BIT) + u];
            const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? x : y, BIT);
            if (hi) x = got;
            else y = got;
        }
    }
}

// Row blocks ("places") of sequence n, whose offset is c0, start at c0 H / BM +
// n: room for ceil(q H / BM) of them.  In 64 bits, since c0 may be anything.
__device__ __forceinline__ long long place_of(int c0, int n, int heads, int BM) {
    const long long rows = (long long)c0 * heads;
    return (rows >= 0 ? rows / BM : -((BM - 1 - rows) / BM)) + n;
}

// Whole warp: the last sequence whose first place is at or before v, its
// offsets and length (the last round loads them with what it searches).
__device__ __forceinline__ int find_seq(const PrefillArgs& a, long long v, int BM, int& c0, int& c1, int& L) {
    const int lane = threadIdx.x & 31;
    int lo = 0, len = a.batch;  // the answer lies in [lo, lo + len)
    while (len > 32) {
        const int step = (len + 31) / 32, n = lo + lane * step, end = lo + len;
        const unsigned hit = __ballot_sync(0xffffffffu, n < end && place_of(__ldg(a.cu_seqlens + n), n, a.heads, BM) <= v);
        lo += (hit ? 31 - __clz(hit) : 0) * step;
        len = min(step, end - lo);
    }
    const int n = lo + min(lane, len - 1);
    c0 = __ldg(a.cu_seqlens + n);
    c1 = __ldg(a.cu_seqlens + n + 1);
    L = __ldg(a.seqlens + n);
    const unsigned hit = __ballot_sync(0xffffffffu, lane < len && place_of(c0, n, a.heads, BM) <= v);
    const int k = hit ? 31 - __clz(hit) : 0;
    c0 = __shfl_sync(0xffffffffu, c0, k);
    c1 = __shfl_sync(0xffffffffu, c1, k);
    L = __shfl_sync(0xffffffffu, L, k);
    return lo + k;
}

// Takes the place of a CTA that has not started: its index, or -1 when none is
// left (then no other request may follow).
__device__ __forceinline__ void request_place(uint32_t* answer, uint64_t* bar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                 ::"r"(smem_u32(answer)), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ int place_taken(const uint32_t* answer) {
    uint32_t got, x;
    asm volatile(
        "{\n.reg .pred p;\n.reg .b128 h;\n"
        "ld.shared.b128 h, [%2];\n"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n"
        "selp.u32 %0, 1, 0, p;\n"
        "mov.u32 %1, 0;\n"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, _, _, _}, h;\n}"
        : "=r"(got), "=r"(x) : "r"(smem_u32(answer)) : "memory");
    return got ? (int)x : -1;
}

template <int DR>
__device__ __forceinline__ uint64_t rope_desc(uint32_t addr) {
    return DR == 64 ? smem_desc(addr, 16, 1024, kLayoutSw128) : smem_desc(addr, 16, 512, kLayoutSw64);
}

template <int DC, int DR>
__global__ void __launch_bounds__(Cfg<DC, DR>::THREADS, 1)
prefill_kernel(const __grid_constant__ Maps maps, const __grid_constant__ PrefillArgs a, const long long places,
               const int log_splits) {
    using C = Cfg<DC, DR>;
    static_assert(sizeof(Misc) <= C::MISC, "barriers fit");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Misc& misc = *reinterpret_cast<Misc*>(sm + C::OFF_MISC);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int H = a.heads, B = a.branches, P = a.page_size;
    // a cluster: the `splits` parts of a row block's tokens, each a CTA or a pair
    const int splits = 1 << log_splits, cluster = splits * C::NV;
    const int crank = blockIdx.x & (cluster - 1), split = crank / C::NV, rank = crank % C::NV;
    const bool has_rope = !C::PAIR || DR == 64 || rank == 0;
    const int rope0 = C::PAIR && DR == 64 ? rank * C::RL : 0;  // its first RoPE column
    const size_t W = (size_t)B * DC;
    volatile int* abort_flag = &misc.abort_flag;
    // this CTA's tiles of a row block: [t0, t0 + ntiles) of all (none where there
    // are fewer than parts)
    auto span = [&](const Job& job, int& t0, int& ntiles) {
        const int all_tiles = ceil_div(job.kv_end, C::KT);
        t0 = all_tiles * split >> log_splits;  // (at most 2^25 tiles, 8 parts)
        ntiles = (all_tiles * (split + 1) >> log_splits) - t0;
    };
    // row block k of this CTA, once it is known
    auto job_at = [&](uint32_t k, Job& job) {
        const bool ok = mbar_wait_warp(&misc.job_full[k & 1], (k >> 1) & 1);
        job = misc.job[k & 1];
        return ok;
    };
    auto job_done = [&](uint32_t k) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&misc.job_empty[k & 1]);
    };
    // warp 0: the row block of place `id` becomes row block k, its queries are
    // requested; false: the place has none
    Job mine;
    bool ok0 = true;
    auto take = [&](uint32_t id, uint32_t k, uint32_t tiles, uint32_t asked) {
        const int b = id % B;
        const long long place = places - 1 - id / B;  // a sequence's later row blocks see more tokens: they start first
        int c0, c1, L;
        const int n = find_seq(a, place, C::BM, c0, c1, L);
        const bool run = c0 >= 0 && c1 >= c0 && c1 <= a.tokens;
        const long long row0 = (place - place_of(c0, n, H, C::BM)) * C::BM;
        if (!run || row0 < 0 || row0 >= (long long)(c1 - c0) * H) return false;
        const bool good = L >= c1 - c0 && seqlen_valid(L, P, a.max_pages);
        const int rows = (c1 - c0) * H, past = L - (c1 - c0);
        mine = Job{n, (int)row0, rows, c0 * H, good ? past : -1, b, past + (min((int)row0 + C::BM, rows) - 1) / H + 1, tiles, asked};
        if (lane == 0) {
            misc.job[k & 1] = mine;
            mbar_arrive(&misc.job_full[k & 1]);
            if (!good && a.status != nullptr) record_error(a.status, MLRA_ERR_DEVICE_BAD_SEQLEN);
        }
        if (!good) return true;
        if (asked > 0) ok0 = mbar_wait_warp(&misc.q_empty, (asked - 1) & 1);
        if (ok0 && lane == 0) {
            mbar_arrive_expect_tx(&misc.q_full, C::MT * (C::Q_LAT + (has_rope ? C::QR_BYTES : 0)));
            for (int m = 0; m < C::MT; ++m) {
                uint8_t* dst = sm + C::OFF_Q + m * C::Q_TILE;
                const int y = c0 * H + (int)row0 + m * 128;
                for (int c = 0; !C::QT && c < C::NCH; ++c)
                    tma_load_2d(dst + c * C::Q_CHUNK, &maps.q, b * DC + rank * C::DL + c * 64, y, &misc.q_full);
                if (has_rope) tma_load_2d(dst + C::Q_LAT, &maps.qr, rope0, y, &misc.q_full);
            }
        }
        return true;
    };

    launch_dependents();
    // warp 0 sets up the barriers, finds the first row block and requests its
    // queries; the others meet it then
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NC; ++i) mbar_init(&misc.c_full[i], 1), mbar_init(&misc.c_empty[i], 1);
        for (int i = 0; i < C::NK; ++i) mbar_init(&misc.k_full[i], 1), mbar_init(&misc.k_empty[i], 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&misc.s_full[i], 1);
            mbar_init(&misc.p_full[i], 4);
            mbar_init(&misc.o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&misc.x_full[i], 1);
            mbar_init(&misc.x_read[i], 4);
            mbar_init(&misc.x_empty[i], 1);
            mbar_init(&misc.x_taken[i], 4);
        }
        mbar_init(&misc.q_tmem, 4);
        mbar_init(&misc.q_full, 1);
        mbar_init(&misc.q_empty, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&misc.job_full[i], 1);
            mbar_init(&misc.checked[i], 1);
            mbar_init(&misc.job_empty[i], 2 + C::SOFT_WARPS + (C::PAIR ? 5 : 0));  // the warps that read it
        }
        for (int i = 0; i < 2; ++i) mbar_init(&misc.next_full[i], 1), mbar_init(&misc.next_read[i], 1);
        mbar_init(&misc.drain, 1);
        misc.abort_flag = 0;
        misc.job[0].n = -1;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&misc.tmem_base, C::TMEM_COLS);
        tmem_relinquish();
    }
    wait_prerequisite_grid();
    const uint32_t first = blockIdx.x / C::NV >> log_splits;
    bool have = false;
    if (warp == 0) have = take(first, 0, 0, 0);
    tc_fence_before();
    if (cluster > 1) cluster_sync();  // (the other CTAs' barriers are set up too)
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc.tmem_base;
    if constexpr (C::MT == 2) {
        if (warp < 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    }
    if (warp == 0) {
        // ------------------------------------------------------------ copies
        const int box = min(P, C::KT);
        uint32_t blocks = 0, asked = 0, done = 0, requests = 0;  // row blocks, of them with queries; tiles whose copies were issued
        bool ok = true;
        for (uint32_t id = first;;) {
            if (have) ++blocks;
            if (have && mine.past >= 0) {
                ++asked;
                ok = ok0;
                int t0, ntiles;
                span(mine, t0, ntiles);
                const int col0 = mine.b * DC + rank * C::DL;
                const int32_t* bt = a.block_table + (size_t)mine.n * a.max_pages;
                int win = t0 * C::KT / P, page_of_lane = 0;  // 32 block-table entries from `win` on
                if (win + lane < a.max_pages) page_of_lane = __ldg(bt + win + lane);
                for (int i = 0; i < ntiles && ok; ++i) {
                    const int tok0 = (t0 + i) * C::KT, nbox = ceil_div(min(C::KT, mine.kv_end - tok0), box);
                    const int page0 = tok0 / P;
                    if (page0 + (nbox * box + P - 1) / P > win + 32) {
                        win = page0;
                        page_of_lane = win + lane < a.max_pages ? __ldg(bt + win + lane) : 0;
                    }
                    const uint32_t cs = done % C::NC, ks = done % C::NK;
                    if (lane == 0) {
                        if (done >= C::NK) ok = mbar_wait(&misc.k_empty[ks], (done / C::NK - 1) & 1);
                        if (ok && done >= C::NC) ok = mbar_wait(&misc.c_empty[cs], (done / C::NC - 1) & 1);
                        ok = ok && !*abort_flag;
                        if (ok) {
                            mbar_arrive_expect_tx(&misc.k_full[ks], has_rope ? nbox * box * C::RL * 2 : 0);
                            mbar_arrive_expect_tx(&misc.c_full[cs], nbox * box * C::NCH * 128);
                        }
                    }
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (!ok) break;
                    for (int q = 0; q < nbox; ++q) {
                        const int tok = tok0 + q * box;
                        int page = __shfl_sync(0xffffffffu, page_of_lane, tok / P - win);
                        page = page >= 0 && page < a.num_pages ? page : 0;  // (the page check reports it)
                        const int y = page * P + tok % P;
                        if (lane == 0) {
                            if (has_rope)
                                tma_load_2d(sm + C::OFF_K + ks * C::K_BYTES + q * box * C::RL * 2, &maps.rope, rope0, y, &misc.k_full[ks]);
                            for (int c = 0; c < C::NCH; ++c)
                                tma_load_2d(sm + C::OFF_C + cs * C::C_BYTES + c * C::C_CHUNK + q * box * 128, &maps.lat,
                                            col0 + c * 64, y, &misc.c_full[cs]);
                        }
                    }
                    ++done;
                }
            }
            if (id == 0 && a.status != nullptr) {  // offsets out of range, whichever places they claim
                bool bad = false;
#pragma unroll 4
                for (int m = lane; m < a.batch; m += 32) {
                    const int c0 = __ldg(a.cu_seqlens + m), c1 = __ldg(a.cu_seqlens + m + 1);
                    bad |= c0 < 0 || c1 < c0 || c1 > a.tokens;
                }
                if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(a.status, MLRA_ERR_DEVICE_BAD_SEQLEN);
            }
            if (!ok || log_splits > 0) break;
            // the place of a CTA (or pair) that has not started, asked for when this row
            // block's last copy is under way (packed prompts 48.9 us; four tiles earlier
            // 51.4: the CTAs end further apart)
            const uint32_t at = requests & 1, phase = (requests >> 1) & 1;
            if (C::PAIR && rank == 0 && requests >= 2) ok = mbar_wait_warp(&misc.next_read[at], phase ^ 1);
            if (!ok) break;
            ++requests;
            if (lane == 0) {
                fence_proxy_async_smem();  // (the answer that was here has been read)
                mbar_arrive_expect_tx(&misc.next_full[at], 16);
                if (rank == 0) request_place(misc.next[at], &misc.next_full[at]);
            }
            ok = mbar_wait_warp(&misc.next_full[at], phase);
            if (!ok) break;
            int next;
            if (rank == 0) {
                next = place_taken(misc.next[at]);
                if (C::PAIR && lane == 0)
                    st_async_v4(map_shared_rank(smem_u32(misc.next[at]), 1), map_shared_rank(smem_u32(&misc.next_full[at]), 1), (uint32_t)next, 0u, 0u, 0u);
            } else {
                next = (int)*reinterpret_cast<volatile uint32_t*>(misc.next[at]);
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_shared_rank(smem_u32(&misc.next_read[at]), 0));
            }
            __syncwarp();
            if (next < 0) break;
            id = next / C::NV;
            if (blocks >= 2) ok = mbar_wait_warp(&misc.job_empty[blocks & 1], ((blocks >> 1) - 1) & 1);
            if (!ok) break;
            have = take(id, blocks, done, asked);
        }
        if (ok && blocks >= 2) ok = mbar_wait_warp(&misc.job_empty[blocks & 1], ((blocks >> 1) - 1) & 1);
        if (lane == 0) {
            if (ok) {
                misc.job[blocks & 1].n = -1;  // no more
                mbar_arrive(&misc.job_full[blocks & 1]);
            } else {
                *abort_flag = 1;
            }
            // no copy or answer may land after this CTA has gone
            constexpr uint64_t kLong = 200000000ull;
            if (asked > 0 && ok0) mbar_wait(&misc.q_full, (asked - 1) & 1, kLong);
            if (requests > 0) mbar_wait(&misc.next_full[(requests - 1) & 1], ((requests - 1) >> 1) & 1, kLong);
            for (uint32_t i = done > C::NK ? done - C::NK : 0; i < done; ++i) mbar_wait(&misc.k_full[i % C::NK], (i / C::NK) & 1, kLong);
            for (uint32_t i = done > C::NC ? done - C::NC : 0; i < done; ++i) mbar_wait(&misc.c_full[i % C::NC], (i / C::NC) & 1, kLong);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMAs
        constexpr uint32_t ID_S = idesc_bf16_f32(128, C::KT, false, false);
        constexpr uint32_t ID_O = idesc_bf16_f32(128, C::VN, false, true);
        const uint32_t at0 = smem_u32(sm);
        const uint64_t dQ = smem_desc(at0 + C::OFF_Q, 16, 1024, kLayoutSw128);
        const uint64_t dQr = rope_desc<C::RL>(at0 + C::OFF_Q + C::Q_LAT);
        const uint64_t dC = smem_desc(at0 + C::OFF_C, 16, 1024, kLayoutSw128);           // K-major
        const uint64_t dV = smem_desc(at0 + C::OFF_C, C::C_CHUNK, 1024, kLayoutSw128);  // MN-major
        const uint64_t dK = rope_desc<C::RL>(at0 + C::OFF_K);
        // (one warp's dependent instructions take four cycles and more each:
        // ring positions are counted, not divided, and the two tiles unrolled)
        struct Ring {
            uint32_t at = 0, phase = 0;
            __device__ __forceinline__ void next(uint32_t depth) {
                if (++at == depth) at = 0, phase ^= 1;
            }
        };
        Ring c_new, k_new, c_old;  // the tile of the next scores (latents, keys); the tile of the next PV
        auto landed = [&]() { return mbar_wait_warp(&misc.k_full[k_new.at], k_new.phase) && mbar_wait_warp(&misc.c_full[c_new.at], c_new.phase); };
        auto scores = [&](int m, int slot) {  // the elected thread: S[slot] = Q C^T + Qr Kr^T of the new tile
            const uint32_t d = tmem + slot * C::S_COLS;
            const uint64_t qr = dQr + ((m * C::Q_TILE) >> 4), k0 = dK + ((k_new.at * C::K_BYTES) >> 4);
            const uint64_t q = dQ + ((m * C::Q_TILE) >> 4), c = dC + ((c_new.at * C::C_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < C::RL / 16; ++k)
                if (has_rope) mma_bf16(d, qr + 2 * k, k0 + 2 * k, ID_S, k ? 1u : 0u);
#pragma unroll
            for (int k = 0; k < C::DL / 16; ++k) {
                const uint64_t ck = c + ((k / 4 * C::C_CHUNK) >> 4) + k % 4 * 2;
                if constexpr (C::QT) mma_bf16_ts(d, tmem + C::Q_COL + 8 * k, ck, ID_S, k || has_rope ? 1u : 0u);
                else mma_bf16(d, q + ((k / 4 * C::Q_CHUNK) >> 4) + k % 4 * 2, ck, ID_S, k || has_rope ? 1u : 0u);
            }
            mma_commit(&misc.s_full[slot]);
            if (m == C::MT - 1) mma_commit(&misc.k_empty[k_new.at]);
        };
        auto values = [&](int m, int slot, bool first, bool last) {  // the elected thread: O[m] += P[slot] C of the old tile
            const uint32_t d = tmem + C::O_COL + m * C::VN, p = tmem + slot * C::S_COLS;
            const uint64_t v = dV + ((c_old.at * C::C_BYTES) >> 4);
#pragma unroll
            for (int k = 0; k < C::KT / 16; ++k) mma_bf16_ts(d, p + 8 * k, v + (k * 2048 >> 4), ID_O, k == 0 && first ? 0u : 1u);
            if (C::MT == 1 || last) mma_commit(&misc.o_done[slot]);
            if (m == C::MT - 1) mma_commit(&misc.c_empty[c_old.at]);
        };
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            Job job;
            ok = job_at(k, job);
            if (!ok || job.n < 0) break;
            job_done(k);
            if (job.past < 0) continue;
            int t0, ntiles;
            span(job, t0, ntiles);
            ok = ntiles == 0 || mbar_wait_warp(&misc.q_full, job.asked & 1);
            if constexpr (C::QT) ok = ok && mbar_wait_warp(&misc.q_tmem, job.asked & 1);
            // the first scores: of both row tiles, or of the first two token tiles
#pragma unroll
            for (int s = 0; s < 2 && ntiles > 0; ++s) {
                const int slot = C::MT == 2 ? s : (job.tiles + s) & 1;
                if (C::MT == 1 && s >= ntiles) continue;  // (one tile only)
                if (s == 0 || C::MT == 1) ok = ok && landed();
                if (ok) {
                    tc_fence_after();
                    if (elect_one()) scores(C::MT == 2 ? s : 0, slot);
                    __syncwarp();
                    if (s == C::MT - 1 || C::MT == 1) c_new.next(C::NC), k_new.next(C::NK);
                }
            }
            if (ntiles <= (C::MT == 2 ? 1 : 2) && elect_one()) mma_commit(&misc.q_empty);
            __syncwarp();
            for (int i = 0; i < ntiles && ok; ++i) {
                constexpr int AHEAD = C::MT == 2 ? 1 : 2;
                const bool more = i + AHEAD < ntiles;
                if (more) ok = landed();
#pragma unroll
                for (int m = 0; m < C::MT; ++m) {
                    const uint32_t at = job.tiles + i;
                    const int slot = C::MT == 2 ? m : at & 1;
                    ok = ok && mbar_wait_warp(&misc.p_full[slot], (C::MT == 2 ? at : at >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
                        values(m, slot, i == 0, i == ntiles - 1);
                        if (more) scores(m, slot);
                    }
                    __syncwarp();
                }
                if (i + AHEAD + 1 == ntiles && elect_one()) mma_commit(&misc.q_empty);
                __syncwarp();
                c_old.next(C::NC);
                if (more) c_new.next(C::NC), k_new.next(C::NK);
                if ((i & 7) == 7 && __shfl_sync(0xffffffffu, *abort_flag, 0)) ok = false;
            }
        }
        if (!ok && lane == 0) *abort_flag = 1;
        // every MMA has finished before TMEM is freed
        if (elect_one()) mma_commit(&misc.drain);
        __syncwarp();
        mbar_wait(&misc.drain, 0, 200000000ull);
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ page checks
        // every page of a row block's sequence has to lie in the pool
        for (uint32_t k = 0;; ++k) {
            Job job;
            if (!job_at(k, job) || job.n < 0) break;
            bool bad = false;
            if (job.past >= 0) {
                const int32_t* bt = a.block_table + (size_t)job.n * a.max_pages;
                const int pages = ceil_div(job.past + job.rows / H, P);
#pragma unroll 4
                for (int e = lane; e < pages; e += 32) {
                    const int page = __ldg(bt + e);
                    bad |= page < 0 || page >= a.num_pages;
                }
            }
            bad = __any_sync(0xffffffffu, bad);
            if (lane == 0) {
                misc.bad[k & 1] = bad;
                mbar_arrive(&misc.checked[k & 1]);
                if (bad && a.status != nullptr) record_error(a.status, MLRA_ERR_DEVICE_BAD_INDEX);
            }
            job_done(k);
        }
    } else if (C::PAIR && warp == 3) {
        // ------------------------------------------------------------ pair: room for the other CTA's scores
        // (a warp of its own: the arrival over there releases what its thread
        // wrote, and a thread that has just sent scores waits 1000 cycles for that)
        bool ok = true;
        if (lane == 0) {
            mbar_arrive_expect_tx(&misc.x_full[0], C::X_BYTES);
            mbar_arrive_expect_tx(&misc.x_full[1], C::X_BYTES);
        }
        for (uint32_t k = 0; ok; ++k) {
            Job job;
            ok = job_at(k, job);
            if (!ok || job.n < 0) break;
            int t0, ntiles = 0;
            if (job.past >= 0) span(job, t0, ntiles);
            for (uint32_t at = job.tiles; at < job.tiles + ntiles && ok; ++at) {
                ok = mbar_wait_warp(&misc.x_read[at & 1], (at >> 1) & 1);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&misc.x_full[at & 1], C::X_BYTES);
                    mbar_arrive_cluster(map_shared_rank(smem_u32(&misc.x_empty[at & 1]), crank ^ 1));
                }
                __syncwarp();
            }
            job_done(k);
        }
        if (!ok && lane == 0) *abort_flag = 1;
    } else if (C::PAIR && warp >= 8) {
        // ------------------------------------------------------------ pair: this CTA's share of the scores
        // each thread sends its row to the same thread of the other CTA, as
        // [four tokens][row] of 16 bytes, while the softmax is an item behind
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t there = map_shared_rank(smem_u32(sm + C::OFF_X) + r * 16, crank ^ 1);
        const uint32_t full = map_shared_rank(smem_u32(&misc.x_full[0]), crank ^ 1);
        bool ok = true;
        for (uint32_t k = 0; ok; ++k) {
            Job job;
            ok = job_at(k, job);
            if (!ok || job.n < 0) break;
            int t0, ntiles = 0;
            if (job.past >= 0) span(job, t0, ntiles);
            const uint32_t end = job.tiles + ntiles;
            for (uint32_t at = job.tiles; at < end && ok; ++at) {
                const uint32_t slot = at & 1;
                ok = mbar_wait_warp(&misc.s_full[slot], (at >> 1) & 1);
                if (!ok) break;
                tc_fence_after();
                uint32_t x[C::KT];
#pragma unroll
                for (int c = 0; c < C::KT / 32; ++c) tmem_ld32(lanes + slot * C::S_COLS + 32 * c, x + 32 * c);
                tmem_wait_ld();
                reg_tie<C::KT>(x);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&misc.x_taken[slot]);
                if (at >= 2) ok = mbar_wait_warp(&misc.x_empty[slot], ((at >> 1) - 1) & 1);
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < C::KT / 4; ++c)
                    st_async_v4(there + slot * C::X_BYTES + c * 2048, full + slot * 8, x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            }
            job_done(k);
        }
        if (!ok && lane == 0) *abort_flag = 1;
    } else if (warp >= 4) {
        // ------------------------------------------------------------ softmax
        if constexpr (C::MT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
        // (a scale of 0 as 1e-30: every finite score still weighs the same, and a
        // masked score, infinite, stays so)
        const float sc = a.scale_log2 == 0.f ? 1e-30f : a.scale_log2;
        const int g = (warp - 4) / 4, quad = warp & 3, r = quad * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
        const uint32_t o_addr = lanes + C::O_COL + g * C::VN;
        // One loop over the items of all row blocks, a block's end and the next one's
        // start a branch of it (8192 tokens 1076 us; with a loop over the blocks
        // around a loop over their items 1120).  Item `at`, of all of this CTA's,
        // covers the tokens from tok0 on.
        uint32_t nth = 0, at = 0, end = 0;
        int tok0 = 0, pos_first = 0;
        float mx = 0.f, l = 0.f;  // running maximum (log2 units) and sum
        bool ok = true, open = false, asked = false;
        // QT: this row's latent queries of a row block into TMEM (rows past the last: zeros)
        auto put_queries = [&](const Job& job) {
            const size_t y = (size_t)job.out0 + job.row0 + r;
            const bool real = y < (size_t)a.tokens * H;
            const uint4* src = reinterpret_cast<const uint4*>(a.q_lat + y * W + job.b * DC + rank * C::DL);
#pragma unroll
            for (int c = 0; c < C::NCH; ++c) {
                uint32_t q[32];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint4 v = real ? __ldg(src + 8 * c + u) : make_uint4(0u, 0u, 0u, 0u);
                    q[4 * u] = v.x, q[4 * u + 1] = v.y, q[4 * u + 2] = v.z, q[4 * u + 3] = v.w;
                }
                tmem_st32(lanes + C::Q_COL + 32 * c, q);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&misc.q_tmem);
        };
        while (true) {
            if (at >= end) {
                if (open) {
                    const bool some = at != misc.job[nth & 1].tiles * C::MT + g;  // (a part of a split may have no tile)
                    if (ok && some) {
                        const uint32_t v = at - C::MT;  // this tile's last item
                        ok = mbar_wait_warp(&misc.o_done[v & 1], C::MT == 1 ? (v >> 1) & 1 : misc.job[nth & 1].asked & 1);
                        tc_fence_after();
                    }
                    if constexpr (C::QT) {
                        // the next block's queries before this one's output: no MMA reads the old ones any more
                        Job next;
                        asked = ok && splits == 1 && job_at(nth + 1, next) && next.n >= 0 && next.past >= 0;
                        if (asked) put_queries(next);
                    }
                    if (!ok && lane == 0) {
                        *abort_flag = 1;
                        if (a.status != nullptr) record_error(a.status, MLRA_ERR_DEVICE_TIMEOUT);
                    }
                    const bool bad = !mbar_wait_warp(&misc.checked[nth & 1], (nth >> 1) & 1) || misc.bad[nth & 1] != 0 || !ok;
                    const Job job = misc.job[nth & 1];  // (again: registers are short in the loop above)
                    const int row = job.row0 + g * 128 + r, rows = job.rows;
                    __nv_bfloat16* dst = a.out + (size_t)(job.out0 + row) * W + job.b * DC + rank * C::DL;
                    if (splits == 1) {
                        const float inv = a.out_scale / l;
#pragma unroll 1
                        for (int c = 0; c < C::VN / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld32(o_addr + 32 * c, o);
                            tmem_wait_ld();
                            reg_tie<32>(o);
#pragma unroll
                            for (int j = 0; j < 32; j += 2)
                                o[j / 2] = bad ? 0u : pack_bf16(__uint_as_float(o[j]) * inv, __uint_as_float(o[j + 1]) * inv);
                            if constexpr (C::MT == 2) {
                                // lane i of four takes the i-th 16 bytes of each of their rows: a store
                                // covers 64 bytes of eight rows, not 16 of 32 (packed prompts 49 us against
                                // 54; with one warp on a scheduler the exchange costs more: d_c = 512 240
                                // against 234)
                                swap_quarters<1>(o, lane);
                                swap_quarters<2>(o, lane);
                                const int i = lane & 3;
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    if (row - i + k < rows)
                                        *reinterpret_cast<uint4*>(dst + (long long)(k - i) * (long long)W + 32 * c + 8 * i) =
                                            make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                            } else if (row < rows) {
#pragma unroll
                                for (int k = 0; k < 4; ++k)
                                    *reinterpret_cast<uint4*>(dst + 32 * c + 8 * k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                            }
                        }
                    } else {
                        // ---------------------------------------------------- the join of the parts
                        // Every part's maximum m and sum l of a row, its O scaled to the common
                        // maximum in shared memory (the operands there are done with), then each
                        // part sums 1 / splits of the columns over the parts, in their order.
                        constexpr int ROWS = 128 * C::MT;
                        float2* stat = reinterpret_cast<float2*>(sm);                 // [row] (m, l)
                        float4* stage = reinterpret_cast<float4*>(sm + ROWS * 8);     // [four columns][row]
                        static_assert(ROWS * 8 + ROWS * C::VN * 4 <= C::OFF_MISC, "the stage fits below the barriers");
                        const int tr = g * 128 + r;
                        if (!some) mbar_wait_warp(&misc.q_full, 0);  // (else the first scores have)
                        named_bar_sync<1, 32 * C::SOFT_WARPS>();  // (no MMA of this CTA reads operands any more)
                        stat[tr] = make_float2(mx, l);
                        cluster_sync();
                        float top = -INFINITY, total = 0.f;
                        for (int p = 0; p < splits; ++p) {
                            const float2 v = ld_shared_cluster_f2(map_shared_rank(smem_u32(stat + tr), p * C::NV + rank));
                            const float t = fmaxf(top, v.x);
                            if (t != -INFINITY) total = total * ex2(top - t) + v.y * ex2(v.x - t);
                            top = t;
                        }
                        const float f = mx != -INFINITY ? ex2(mx - top) : 0.f;
#pragma unroll 1
                        for (int c = 0; c < C::VN / 32; ++c) {
                            uint32_t o[32];
                            if (some) {
                                tmem_ld32(o_addr + 32 * c, o);
                                tmem_wait_ld();
                                reg_tie<32>(o);
                            }
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                                if (f != 0.f)
                                    v = make_float4(__uint_as_float(o[j]) * f, __uint_as_float(o[j + 1]) * f, __uint_as_float(o[j + 2]) * f,
                                                    __uint_as_float(o[j + 3]) * f);
                                stage[(c * 8 + j / 4) * ROWS + tr] = v;
                            }
                        }
                        cluster_sync();
                        const float inv = a.out_scale / total;
                        const int c0 = C::VN / 4 * split >> log_splits, c1 = C::VN / 4 * (split + 1) >> log_splits;  // groups of four columns
                        for (int c = c0; c < c1; c += 2) {
                            float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
                            for (int p = 0; p < splits; ++p) {
                                const uint32_t at = map_shared_rank(smem_u32(stage + c * ROWS + tr), p * C::NV + rank);
                                const float4 x = ld_shared_cluster_f4(at), y = ld_shared_cluster_f4(at + ROWS * 16);
                                u.x += x.x, u.y += x.y, u.z += x.z, u.w += x.w;
                                v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
                            }
                            uint4 o = make_uint4(pack_bf16(u.x * inv, u.y * inv), pack_bf16(u.z * inv, u.w * inv), pack_bf16(v.x * inv, v.y * inv),
                                                 pack_bf16(v.z * inv, v.w * inv));
                            if (bad) o = make_uint4(0u, 0u, 0u, 0u);
                            if (row < rows) *reinterpret_cast<uint4*>(dst + 4 * c) = o;
                        }
                    }
                    tc_fence_before();
                    job_done(nth++);
                    if (!ok) break;
                    open = false;
                }
                {
                    Job job;
                    ok = job_at(nth, job);
                    if (!ok && lane == 0) *abort_flag = 1;
                    if (!ok || job.n < 0) break;
                    const int row = job.row0 + g * 128 + r;
                    if (job.past < 0) {  // a bad length: zeros
                        __nv_bfloat16* dst = a.out + (size_t)(job.out0 + row) * W + job.b * DC + rank * C::DL;
                        for (int c = 0; c < C::VN / 8 && row < job.rows; ++c) *reinterpret_cast<uint4*>(dst + 8 * c) = make_uint4(0u, 0u, 0u, 0u);
                        job_done(nth++);
                        continue;
                    }
                    int ntiles;
                    span(job, tok0, ntiles);
                    tok0 *= C::KT;
                    at = job.tiles * C::MT + g;
                    end = (job.tiles + ntiles) * C::MT;
                    pos_first = job.past + min(row - lane, job.rows - 1) / H;  // last token of the warp's first row
                }
                if constexpr (C::QT) {
                    if (!asked) put_queries(misc.job[nth & 1]);
                    asked = false;
                }
                mx = -INFINITY, l = 0.f;
                open = true;
                if (at >= end) continue;
            }
            const uint32_t slot = at & 1, parity = (at >> 1) & 1;
            const uint32_t s_addr = lanes + slot * C::S_COLS;
            ok = mbar_wait_warp(&misc.s_full[slot], parity);
            if (!ok) {
                at = end;
                continue;
            }
            tc_fence_after();
            uint32_t x[C::KT];
#pragma unroll
            for (int c = 0; c < C::KT / 32; ++c) tmem_ld32(s_addr + 32 * c, x + 32 * c);
            tmem_wait_ld();
            reg_tie<C::KT>(x);
            if constexpr (C::PAIR) {
                // plus the scores of the other CTA's columns (a sum of two, so both
                // CTAs have the same bits)
                const float4* here = reinterpret_cast<const float4*>(sm + C::OFF_X + slot * C::X_BYTES) + r;
                ok = mbar_wait_warp(&misc.x_full[slot], parity);
                if (!ok) {
                    at = end;
                    continue;
                }
#pragma unroll
                for (int c = 0; c < C::KT / 4; ++c) {
                    const float4 v = here[c * 128];
                    x[4 * c] = __float_as_uint(__uint_as_float(x[4 * c]) + v.x);
                    x[4 * c + 1] = __float_as_uint(__uint_as_float(x[4 * c + 1]) + v.y);
                    x[4 * c + 2] = __float_as_uint(__uint_as_float(x[4 * c + 2]) + v.z);
                    x[4 * c + 3] = __float_as_uint(__uint_as_float(x[4 * c + 3]) + v.w);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&misc.x_read[slot]);
                // (P will lie over the scores: they have been taken for sending)
                ok = mbar_wait_warp(&misc.x_taken[slot], parity);
                if (!ok) {
                    at = end;
                    continue;
                }
                tc_fence_after();
            }
            // tokens j > limit of the tile are masked (a whole warp's rows at once see it all otherwise)
            if (pos_first - tok0 < C::KT - 1) {
                const Job& job = misc.job[nth & 1];
                const int limit = job.past + min(job.row0 + g * 128 + r, job.rows - 1) / H - tok0;  // of this row
                const uint32_t none = sc < 0.f ? 0x7f800000u : 0xff800000u;
#pragma unroll
                for (int j = 0; j < C::KT; ++j) x[j] = j > limit ? none : x[j];
            }
            // the largest scaled score (the smallest raw one under a negative scale)
            float top[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) top[k] = __uint_as_float(x[k]);
            if (sc < 0.f) {
#pragma unroll
                for (int j = 4; j < C::KT; ++j) top[j & 3] = fminf(top[j & 3], __uint_as_float(x[j]));
                top[0] = fminf(fminf(top[0], top[1]), fminf(top[2], top[3])) * sc;
            } else {
#pragma unroll
                for (int j = 4; j + 8 <= C::KT; j += 8)
#pragma unroll
                    for (int k = 0; k < 4; ++k) top[k] = max3(top[k], __uint_as_float(x[j + 2 * k]), __uint_as_float(x[j + 2 * k + 1]));
#pragma unroll
                for (int k = 0; k < 4; ++k) top[k] = fmaxf(top[k], __uint_as_float(x[C::KT - 4 + k]));
                top[0] = fmaxf(max3(top[0], top[1], top[2]), top[3]) * sc;
            }
            {
                // (a row that has seen no token yet: its O, not begun or of zero weights, stays)
                const bool none = mx == -INFINITY;
                const bool grow = !none && top[0] > mx + kRescale;
                if (none) mx = top[0];
                if (__any_sync(0xffffffffu, grow)) {
                    // O of this warp's rows at the new maximum, once the PV before is done
                    if constexpr (C::MT == 1) {
                        ok = mbar_wait_warp(&misc.o_done[(at - 1) & 1], ((at - 1) >> 1) & 1);
                        if (!ok) {
                            at = end;
                            continue;
                        }
                        tc_fence_after();
                    }
                    const float alpha = grow ? ex2(mx - top[0]) : 1.f;
                    if (grow) mx = top[0];
                    l *= alpha;
#pragma unroll 1
                    for (int c = 0; c < C::VN / 16; ++c) {
                        float o[16];
                        tmem_ld16(o_addr + 16 * c, o);
                        tmem_wait_ld(o);
#pragma unroll
                        for (int j = 0; j < 16; ++j) o[j] *= alpha;
                        tmem_st16(o_addr + 16 * c, o);
                    }
                    tmem_wait_st();
                }
            }
            // slots behind the last token (stale, or another sequence's) become
            // zero before the output MMA reads them: 0 * NaN is NaN
            if (at + C::MT >= end && tok0 + C::KT > misc.job[nth & 1].kv_end) {
                uint8_t* tile = sm + C::OFF_C + (at / C::MT % C::NC) * C::C_BYTES;
                const int dead = tok0 + C::KT - misc.job[nth & 1].kv_end, units = dead * 8;
                for (int e = r; e < units * C::NCH; e += 128)
                    *reinterpret_cast<uint4*>(tile + e / units * C::C_CHUNK + (C::KT - dead) * 128 + e % units * 16) =
                        make_uint4(0u, 0u, 0u, 0u);
                fence_proxy_async_smem();
            }
            // (a row that has seen no token yet: its scores are all -infinity, and so their
            // differences stay)
            const float ref = mx == -INFINITY ? 0.f : mx;
            // The maximum is a rounded product, the difference below takes it exactly: off by
            // half a step, which from 2^31 on is 2^7 and more, a weight of infinity or none.
            // From 2^30 on scores are scaled by the power of two that brings the largest below
            // 2^31: their steps are 2^6 and more still, so all but the largest weigh nothing.
            // (8192 tokens 1068 us against 1065 without; other forms, with a vote and the
            // differences taken beforehand, 1077 to 1124; 512-wide branch 235 us against 232.)
            const float s = __uint_as_float(min(127u << 23, ((127u + 157u) << 23) - (__float_as_uint(ref) & 0x7f800000u)));
            const float fac = sc * s, neg = -ref * s;
            const uint64_t sc2 = pack2(fac, fac), mx2 = pack2(neg, neg);
            uint64_t sum[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < C::KT; j += 2) {
                float p0, p1;
                unpack2(fma2(pack2(x[j], x[j + 1]), sc2, mx2), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                sum[j / 2 & 1] = add2(sum[j / 2 & 1], pack2(p0, p1));
                x[j / 2] = pack_bf16(p0, p1);
            }
#pragma unroll
            for (int c = 0; c < C::KT / 64; ++c) tmem_st32(s_addr + 32 * c, x + 32 * c);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&misc.p_full[slot]);
            float s0, s1;
            unpack2(add2(sum[0], sum[1]), s0, s1);
            l += s0 + s1;
            at += C::MT;
            tok0 += C::KT;
        }
    }
    if (splits > 1 && misc.job[0].n >= 0 && misc.job[0].past >= 0 && (warp < 4 || warp >= 4 + C::SOFT_WARPS)) {  // the softmax warps' meetings in the join
        cluster_sync();
        cluster_sync();
    }
    __syncwarp();
    if (cluster > 1) cluster_sync();  // (no other CTA reads or writes this one's memory any more)
    else __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int DC, int DR>
cudaError_t launch_cfg(const PrefillArgs& a, cudaStream_t stream) {
    using C = Cfg<DC, DR>;
    Maps maps;
    const uint64_t W = (uint64_t)a.branches * DC, q_rows = (uint64_t)a.tokens * a.heads;
    const uint64_t rows = (uint64_t)a.num_pages * a.page_size;
    const uint32_t box = a.page_size < C::KT ? a.page_size : C::KT;
    if (!encode_rows(&maps.q, a.q_lat, 2, W, q_rows, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_rows(&maps.qr, a.q_rope, 2, DR, q_rows, C::RL, 128, rope_swizzle(C::RL)) ||
        !encode_rows(&maps.lat, a.latent, 2, W, rows, 64, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_rows(&maps.rope, a.rope, 2, DR, rows, C::RL, box, rope_swizzle(C::RL)))
        return cudaErrorInvalidValue;
    auto kernel = prefill_kernel<DC, DR>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if constexpr (C::MT == 2) {
        // the softmax warps' registers come out of what the block is launched
        // with; a build that allots less must not launch (they would wait forever)
        static const int regs = [&] {
            cudaFuncAttributes at;
            return cudaFuncGetAttributes(&at, kernel) == cudaSuccess ? at.numRegs : 0;
        }();
        if (regs / 8 * 8 * C::THREADS < 128 * (2 * kSoftRegs + kOtherRegs)) return cudaErrorInvalidConfiguration;
    }
    const long long places = (long long)(q_rows / C::BM) + a.batch;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    cfg.attrs = attr;
    // Row blocks in flight at once: one CTA (or pair) per SM.  Where they leave SMs
    // idle, a row block's tokens are split over a cluster of up to 8 CTAs, four
    // tiles each at least (by the block table, which bounds the lengths) and as
    // many clusters as the device holds at once (a cluster stays within a group of
    // SMs: 74 clusters of 2, 33 of 4, 15 of 8).  One new token after 8191: 30.5 us in
    // 8 parts, 136 in one.  Every sequence has row blocks of its own; the lengths of
    // the runs are not known here, so their average stands for them.  One new token
    // in each of 8, 32, 64 sequences after 8191: 52, 153, 328 us, where the blocks of
    // all rows laid end to end, with more parts, gave 95, 296, 442 (of 1 to 7 tokens
    // after up to 8191: 42, 152, 245 us and 70, 148, 226).  Pairs may be a quarter more
    // than fit at once: 16 sequences of the 512-wide branch in 4 parts take 132 us
    // at one token after 8191 each, 67 ragged, in 2 parts 122 and 117.
    static const auto resident = [&] {
        std::array<int, 4> n{};  // clusters of 1, 2, 4, 8 CTAs
        cudaLaunchConfig_t c = cfg;
        c.numAttrs = 1;
        for (int k = 0; k < 4; ++k) {
            attr[0].val.clusterDim = {1u << k, 1, 1};
            c.gridDim = dim3(1u << k);
            if (cudaOccupancyMaxActiveClusters(&n[k], kernel, &c) != cudaSuccess) n[k] = 0;
        }
        cudaGetLastError();
        return n;
    }();
    const long long runs = a.batch < a.tokens ? a.batch : a.tokens;  // sequences with new tokens, at most
    const long long rows_of_run = (a.tokens + runs - 1) / runs * a.heads;
    const long long blocks = runs * ((rows_of_run + C::BM - 1) / C::BM) * a.branches;
    const long long most = (long long)a.max_pages * a.page_size / (4 * C::KT);
    int log_splits = 0;
    while (C::NV << log_splits < 8 && blocks * 4 <= resident[log_splits + 1 + (C::NV == 2)] * (C::PAIR ? 5 : 4) && 2 << log_splits <= most) ++log_splits;
    const long long grid = places * a.branches * C::NV << log_splits;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)grid);
    attr[0].val.clusterDim = {(unsigned)(C::NV << log_splits), 1, 1};
    attr[1] = attr[0];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = C::NV << log_splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, maps, a, places, log_splits);
}

template <int DC>
cudaError_t launch_dc(const PrefillArgs& a, cudaStream_t stream) {
    return a.d_r == 64 ? launch_cfg<DC, 64>(a, stream) : launch_cfg<DC, 32>(a, stream);
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
