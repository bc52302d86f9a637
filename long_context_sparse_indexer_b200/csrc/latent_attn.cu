// Latent attention in the absorbed form over every visible cached row, paged or not, on the 5th-generation
// tensor cores.
//
//   z_s = sm_scale q . K_s (576), o = softmax(z) V (V = the first 512 elements of the same row), one pass with a
//   running reference maximum and sum.
//
// Units and cut.  The rows of a group (q_group tokens x H heads, one sequence) are taken 128 at a time: a unit,
// whose work is ceil(longest context of its tokens / 64) key tiles.  The tiles of all units, laid end to end, are
// cut into equal runs, one per cluster, so ragged lengths and few tokens load the GPU evenly (few units are cut each by
// itself where that costs little).  A unit that lies in one run is written out; one that is cut leaves FP32 partial results (at most two per cluster), joined by
// latent_merge_kernel.  The cut depends on the inputs only, so results repeat bit for bit.
//
// A cluster is two CTAs and one tcgen05 pair (cta_group::2, M = 128): CTA c holds rows [64 c, 64 c + 64) of the
// unit, on TMEM lanes 0..63 for the first half of each product's columns and 64..127 for the second, so the
// 64 x 512 FP32 accumulator takes 256 columns and leaves room for scores and queries; a single CTA with 128 rows
// would need all 512.  The pair runs at the full rate of both tensor cores (measured: 64 cycles for M = 128,
// N = 256, K = 16).  Of a key tile's 64 keys CTA c loads its own 32 whole, as its half of the B operand of the
// scores; for P V it needs the other 32 as well, in its 256 value dimensions: once the scores are done these are
// loaded over the 256 dimensions of its own keys that only the scores needed.  Every byte crosses to an SM once
// for S and half of them once more for V, against twice the rows for a pair of independent CTAs.
//
// Memory.  TMEM: O [0, 256), two score buffers [256, 320), Q dims 0..383 [320, 512) (each row on lanes r and
// r + 64; a query operand from TMEM spares the shared-memory port, which S alone would fill: 4 KB per 32-cycle
// MMA).  Shared memory: Q dims 384..575, two P buffers (BF16), a ring of five 36 KB stages; a stage is nine
// 64-dim atoms of 32 keys, atoms 0..3 / 4..7 doubling as the value rows of keys 0..31 / 32..63.  Queries arrive
// through two stages of the same ring.
//
// Warps: 0..3 and 4..7 softmax, alternate tiles (thread = TMEM lane = (row, half of the keys); the two halves of a row
// exchange their maxima through shared memory), 8 the MMAs (in CTA 0, for both), 9 the plan of the cluster's segments.
// BF16: 10 and 11 load keys and exchanged rows by TMA.  FP8: 16 loads a tile's codes into the tail of the stage that they
// widen into (bit moves only), eight warps widen them there and four the exchanged rows, one brings the row scales, and
// the plan is 21's.
// All waits are bounded; a CTA that gives up reports LSA_ERR_TIMEOUT.  A parity tells one phase from the next only, so
// every wait is on a barrier each phase of which its warp sees, and none of whose phases ends without that warp's part in
// the one before.
//
// Measured (kernel and join on the device, inputs not in L2; in brackets after a tenth of a second of such calls, when the GPU
// is at its power limit, 1.1-1.6 GHz): 32 tokens of 128 heads at 32K-64K rows 396-416 us [470] (1.1 PFLOP/s, 4.6 TB/s; a tile
// of 64 keys takes 1,470 cycles, 1,244 of them products), FP8 455-463 [530] (2,400 cycles: widening); a chunk of 500 tokens
// behind 15,500 rows 1.50 ms [1.72], 1.46 [1.27] PFLOP/s; one token at 1000 rows 17.3 us, all latency.
#include <cmath>
#include <cstring>
#include <mutex>

#include "kernels.cuh"
#include "tc.cuh"

namespace lsa {

namespace {

constexpr int kD = 576, kDv = 512, kM = 128, kRows = 64;         // unit rows, rows of a CTA
constexpr int kTile = 64, kOwn = 32;                             // keys of a tile, of a CTA
constexpr int kStages = 5, kAtoms = 9, kStageBytes = kAtoms * kOwn * 128;
// A stage's keys: groups of 8 rows, each nine 1 KB atoms of 8 rows x 64 dims.  Any run of 8 rows is one TMA box with
// every dim, whatever the page size, and both operands' strides stay uniform (a group apart, an atom apart).
constexpr int kAtom = 1024, kGroup = kAtoms * kAtom;
constexpr int kQAtom = kOwn * 128;               // queries in a stage: 64-dim atoms of 32 rows
constexpr int kXBytes = 4 * kOwn * 128;
// FP8: the codes of 8 rows land in the tail of the group they widen into, in its order (nine 512-byte atoms), so that
// widening atom after atom never writes over codes not yet read: 1024 (c + 1) <= 4608 + 512 (c + 1) for c < 9.
constexpr int kCodeBytes = kOwn * kD, kCodeAt = kGroup / 2;
constexpr int kQTmem = 6;                                        // query atoms in TMEM, the others in shared memory
constexpr int kSCol = 256, kQCol = 320;
constexpr int kSegs = 3;                                         // published segments
constexpr int kMaxClusters = 80;
constexpr int kMinRun = 2;                       // key tiles of a run at least: a shorter one costs more to join than it saves
constexpr int kSpare = 5;                        // key tiles that a run may be longer to lie in one unit
constexpr int kSoftmaxWarps = 8, kMmaWarp = 8;
// The other warps.  FP8 (24 warps): the four schedulers (warp mod 4) share the widening evenly, the MMAs' with less of it.
template <bool FP8> constexpr int kPlanWarp = FP8 ? 21 : 9;
template <bool FP8> constexpr int kLoadWarp = FP8 ? 16 : 10;     // queries and own keys
template <bool FP8> constexpr int kXWarp = FP8 ? -1 : 11;        // BF16: exchanged rows
constexpr int kKWarps = 8, kXWarps = 4;                          // FP8 converters
static_assert(kQCol + kQTmem * 32 == 512, "TMEM columns");

struct Seg {
    int unit, seq, k0, k1, n, len;               // key tiles [k0, k1) of the unit's n; keys below len; unit < 0: the end
};

struct Smem {
    alignas(1024) uint8_t ring[kStages][kStageBytes];
    alignas(1024) uint8_t q[kAtoms - kQTmem][kRows * 128];
    alignas(1024) uint8_t p[2][kRows * 128];
    float kscale[kStages][kTile];                // FP8: the tile's row scales, times kUp and the softmax scale
    float mx[2][2][128];                         // what the halves of a row exchange, per warpgroup: tile maxima, sums
    float m_ref[128];                            // the reference maximum after the latest decided tile
    float m_last[2][kRows];                      // each warpgroup's last reference, and its sums by half
    union {
        float l_last[2][128];
        struct {                                 // the plan's, before any tile
            long long scan[32];                  // sums of the warps
            int tiles[kMaxClusters];             // of each unit, where there are no more units than clusters
        } plan;
    };
    Seg seg[kSegs];
    uint64_t seg_full[kSegs], seg_empty[kSegs];
    uint64_t k_full[kStages];                    // CTA 0: both CTAs' keys have landed
    uint64_t sc_full[kStages];                   // FP8: kscale is written
    uint64_t code_full[2][kStages], x_code[4];   // FP8: the codes of an even / odd tile in the stage have landed; those of exchanged group g
    uint64_t x_go[kStages], x_full[kStages];     // the scores of the stage are done; its exchanged rows have landed
    uint64_t empty[kStages];
    uint64_t q_full, q_ready;                    // queries staged; (CTA 0) moved to their operand places in both CTAs
    uint64_t s_full[2], s_free[2];               // scores done; (CTA 0) read by both CTAs
    uint64_t p_full[2], pv_done[2];              // (CTA 0) weights and value rows in place; their product done
    uint64_t pair[2][2];                         // softmax warps w and w + 2 of a warpgroup: the halves' values are written
    uint64_t hand[2][4];                         // warpgroup w, quarter q: m_ref of its tile is out
    uint64_t both;                               // every softmax warp has written its last reference and sum
    uint64_t o_read;                             // every softmax warp has read O
    uint64_t q_taken;                            // every softmax warp has read the staged queries
    uint64_t mma_done;
    uint32_t tmem_base;
    int abort;
};

static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory");

// Workspace: a header, then the partial results of 2 kMaxClusters slots.
struct WsHeader {
    int clusters;                                // runs of this call
    int unit[kMaxClusters], k0[kMaxClusters];    // each run's first unit and tile in it
};
constexpr size_t kWsO = 4096;
constexpr size_t kWsLse = kWsO + (size_t)2 * kMaxClusters * kM * kDv * 4;
constexpr size_t kWsBytes = kWsLse + (size_t)2 * kMaxClusters * kM * 4;
static_assert(sizeof(WsHeader) <= kWsO, "header");

// A slot's partial result for a CTA's rows, as the softmax threads hold it: [4-dim group of 64][TMEM lane] float4, lane L = row
// L & 63 and dims 256 (L >> 6) + 4 group .. + 3.
__device__ __forceinline__ float4* part_o(void* ws, int slot, int rank) {
    return reinterpret_cast<float4*>(static_cast<uint8_t*>(ws) + kWsO) + ((size_t)slot * 2 + rank) * (kRows * kDv / 4);
}
__device__ __forceinline__ float* part_lse(void* ws, int slot) {
    return reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kWsLse) + (size_t)slot * kM;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A bounded wait whose slow part is a call: the roles' loops together fill the instruction cache otherwise (with every
// wait inlined and the products issued from three places the FP8 kernel was 140 KB of code, half its time fetching).
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort) { return tc::mbar_wait(bar, parity, abort); }
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return tc::mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort);
}

// ---- pair forms of the tcgen05 and mbarrier operations

__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t n) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(tc::smem_u32(dst)), "r"(n) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t t, uint32_t n) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(t), "r"(n) : "memory");
}
__device__ __forceinline__ void mma2_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" :: "r"(d), "l"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}
__device__ __forceinline__ void mma2_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p; }" :: "r"(d), "r"(a), "l"(b), "r"(id), "r"(acc) : "memory");
}
// Arrives on `bar` of both CTAs once every MMA issued so far has completed.
__device__ __forceinline__ void commit2(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(tc::smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
// Arrive on a barrier of CTA 0.  What it signals stays on this SM (writes to its own shared memory, already
// fenced for the tensor core that reads them, and tensor-memory accesses), so the release is at CTA scope: at
// cluster scope it cost the warp 700 to 1,000 cycles, twice a tile.
__device__ __forceinline__ void arrive0(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];" :: "r"(tc::peer_smem(bar, 0)) : "memory");
}
// 4-D box into this CTA's shared memory, completing on the barrier at shared::cluster address bar of the pair's CTA 0.
__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        :: "r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Boxes completing on a barrier of this CTA.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z, int w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
        :: "r"(tc::smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(tc::smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

// Four e4m3 codes (a word) to BF16 values times 2^-120, exactly (subnormals included): sign, exponent and mantissa moved
// into place, the exponent keeping e4m3's bias of 7 under BF16's of 127.  The factor is made good by the other operands:
// queries and row scales carry kUp, and the results 1 / (kUp * 2^-120) = kUp.  (The row scales also
// carry the softmax scale, for the scores; the results give it back.)
constexpr float kUp = 1152921504606846976.f;     // 2^60
__device__ __forceinline__ uint2 widen4(uint32_t w) {
    // A code's byte below its sign replicated (selectors 8 + i), shifted by 4: sign at bit 15, exponent from bit 7.
    uint32_t lo, hi;
    asm("prmt.b32 %0, %1, 0, 0x9180;" : "=r"(lo) : "r"(w));
    asm("prmt.b32 %0, %1, 0, 0xb3a2;" : "=r"(hi) : "r"(w));
    return make_uint2((lo << 4) & 0x87f087f0u, (hi << 4) & 0x87f087f0u);
}
// Two BF16 values times kUp.
__device__ __forceinline__ uint32_t up2(uint32_t v) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x5d805d80u));
    return r;
}

struct LatentKernelArgs {
    LatentArgs a;
    int units, m_tiles, group_rows;              // units, units of a group, rows of a group
    int clusters;
};

// Page (or sequence, without pages) of a sequence's row and its place in it; -1, reported, for a page outside the pool.
__device__ __noinline__ int page_of(const LatentArgs& a, int seq, int row, int* in_page) {
    if (!a.table) { *in_page = row; return seq; }
    const int pg = row / a.page_size;
    *in_page = row - pg * a.page_size;
    const int id = a.table[seq * a.table_ld + pg];
    if (id >= 0 && id < a.n_pages) return id;
    report(a.status, LSA_ERR_DEVICE_DATA);
    return -1;
}

// Keys that some token of the unit sees (0: padding only), and its sequence.  `tell`: report bad tokens.
__device__ __noinline__ int unit_len(const LatentKernelArgs& k, int u, int* seq, bool tell) {
    const LatentArgs& a = k.a;
    const int g = u / k.m_tiles, r0 = (u - g * k.m_tiles) * kM, r1 = min(k.group_rows, r0 + kM);
    const int t0 = g * a.q_group, ta = t0 + r0 / a.H, tb = t0 + (r1 - 1) / a.H;
    const int b = a.q_seq[t0];
    int pos = a.q_pos[ta], sq = a.q_seq[ta];     // asked for before the sequence's length is
    int sl = 0;
    if (b >= 0 && b < a.B) {
        sl = a.seq_len[b];
        if (sl > a.L_alloc) sl = 0;
    }
    *seq = b;
    int len = 0;
    bool bad = false;
    for (int t = ta;; pos = a.q_pos[t], sq = a.q_seq[t]) {
        if (pos >= 0) {
            if (pos < sl && sq == b) len = max(len, pos + 1);
            else bad = true;
        }
        if (++t > tb) break;
    }
    if (bad && tell) report(a.status, LSA_ERR_DEVICE_DATA);
    return len;
}

template <bool FP8>
constexpr int kThreadsOf = 32 * (FP8 ? 24 : 12);

template <bool FP8>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreadsOf<FP8>, 1)
    latent_attn_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap xmap, const __grid_constant__ LatentKernelArgs k) {
    constexpr int kThreads = kThreadsOf<FP8>;
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const LatentArgs& a = k.a;
    const int rank = blockIdx.x & 1, cluster = blockIdx.x >> 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sm.abort;

    if (threadIdx.x == 0) {
        constexpr int kLoaders = FP8 ? 2 + kKWarps + kXWarps : 2;
        for (int i = 0; i < kSegs; ++i) {
            tc::mbar_init(&sm.seg_full[i], 1);
            tc::mbar_init(&sm.seg_empty[i], kSoftmaxWarps + kLoaders + (rank == 0 ? 1 : 0));
        }
        for (int i = 0; i < kStages; ++i) {
            tc::mbar_init(&sm.k_full[i], FP8 ? kKWarps : 1);     // FP8: four warps of each CTA
            tc::mbar_init(&sm.sc_full[i], 1);
            for (int j = 0; j < 2; ++j) tc::mbar_init(&sm.code_full[j][i], 1);
            tc::mbar_init(&sm.x_go[i], 1);
            tc::mbar_init(&sm.x_full[i], FP8 ? kXWarps : 1);
            tc::mbar_init(&sm.empty[i], 1);
        }
        tc::mbar_init(&sm.q_full, 1);
        tc::mbar_init(&sm.q_ready, 2 * kSoftmaxWarps);
        tc::mbar_init(&sm.q_taken, kSoftmaxWarps);
        tc::mbar_init(&sm.o_read, kSoftmaxWarps);
        tc::mbar_init(&sm.both, kSoftmaxWarps);
        for (int i = 0; i < 4; ++i) tc::mbar_init(&sm.x_code[i], 1);
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&sm.s_full[i], 1);
            tc::mbar_init(&sm.s_free[i], 8);
            tc::mbar_init(&sm.p_full[i], 8);
            tc::mbar_init(&sm.pv_done[i], 1);
            for (int j = 0; j < 2; ++j) tc::mbar_init(&sm.pair[i][j], 2);
            for (int j = 0; j < 4; ++j) tc::mbar_init(&sm.hand[i][j], 1);
        }
        tc::mbar_init(&sm.mma_done, 1);
        sm.abort = 0;
        tc::fence_barrier_init();
    }
    if (warp == kMmaWarp) tmem_alloc2(&sm.tmem_base, 512);
    if (threadIdx.x == 32) {
        tc::prefetch_tmap(&qmap);
        tc::prefetch_tmap(&kmap);
        tc::prefetch_tmap(&xmap);
    }

    // The plan: tiles per unit, summed over the block; each thread takes a run of units.
    const int per = (k.units + kThreads - 1) / kThreads;
    const int ua = min(k.units, (int)threadIdx.x * per), ub = min(k.units, ua + per);
    long long mine = 0;
    int len0 = 0, seq0 = 0;                      // of the thread's last unit
    for (int u = ua; u < ub; ++u) {
        len0 = unit_len(k, u, &seq0, blockIdx.x == 0);
        mine += (len0 + kTile - 1) / kTile;
    }
    long long before = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += v;
    }
    if (lane == 31) sm.plan.scan[warp] = before;
    if (k.units <= k.clusters && threadIdx.x < k.units) sm.plan.tiles[threadIdx.x] = (int)mine;
    __syncthreads();
    long long sums = lane < kThreads / 32 ? sm.plan.scan[lane] : 0;     // of the warps up to this lane's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, sums, o);
        if (lane >= o) sums += v;
    }
    const long long total = __shfl_sync(0xffffffffu, sums, 31), below = __shfl_sync(0xffffffffu, sums, (warp + 31) & 31);
    before += (warp ? below : 0) - mine;
    int n_runs = (int)min((long long)k.clusters, (total + kMinRun - 1) / kMinRun);
    long long lo = 0, hi = 0;
    if (n_runs && total < 0x7fffffffll / kMaxClusters) {           // the common case without 64-bit divisions
        lo = (uint32_t)total * (uint32_t)cluster / (uint32_t)n_runs;
        hi = (uint32_t)total * (uint32_t)(cluster + 1) / (uint32_t)n_runs;
        // A run with parts of two units pays for the second's start, about as much as kSpare tiles: where runs up to so
        // much longer suffice, every unit is cut by itself, evenly (4 tokens at 1000 rows 24.9 -> 21.1 us, 4 verify tokens of 128
        // heads at 4000 rows 34 -> 28; with 10 tiles to spare some longer contexts lose 5%).
        if (k.units > 1 && k.units <= n_runs) {
            int t[3], len = 0;
#pragma unroll
            for (int i = 0; i < 3; ++i) t[i] = i * 32 + lane < k.units ? sm.plan.tiles[i * 32 + lane] : 0;
            const int even = ((int)total + n_runs - 1) / n_runs;
            for (int l = even; l <= even + kSpare && !len; ++l) {
                int runs = 0;
#pragma unroll
                for (int i = 0; i < 3; ++i) runs += (t[i] + l - 1) / l;
                if ((int)__reduce_add_sync(0xffffffffu, runs) <= n_runs) len = l;
            }
            if (len) {
                int r0 = 0, t0 = 0;              // runs and tiles of the units before
#pragma unroll
                for (int i = 0; i < 3; ++i) {
                    if (i * 32 >= k.units) break;
                    const int runs = (t[i] + len - 1) / len;
                    int r = runs, n = t[i];
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const int rv = __shfl_up_sync(0xffffffffu, r, o), nv = __shfl_up_sync(0xffffffffu, n, o);
                        if (lane >= o) { r += rv; n += nv; }
                    }
                    const int j = cluster - (r0 + r - runs);       // of this lane's unit
                    const unsigned mine_is = __ballot_sync(0xffffffffu, j >= 0 && j < runs);
                    if (mine_is) {
                        const uint32_t d = max(runs, 1);
                        const int from = t0 + n - t[i] + (int)((uint32_t)t[i] * (uint32_t)j / d);
                        const int to = t0 + n - t[i] + (int)((uint32_t)t[i] * (uint32_t)(j + 1) / d);
                        lo = __shfl_sync(0xffffffffu, from, __ffs(mine_is) - 1);
                        hi = __shfl_sync(0xffffffffu, to, __ffs(mine_is) - 1);
                    }
                    r0 += __shfl_sync(0xffffffffu, r, 31);
                    t0 += __shfl_sync(0xffffffffu, n, 31);
                }
                n_runs = r0;
            }
        }
    } else if (n_runs) {
        lo = total * cluster / n_runs;
        hi = total * (cluster + 1) / n_runs;
    }
    const bool busy = cluster < n_runs;
    if (busy && before <= lo && lo < before + mine) {              // one thread: the run starts among its units
        long long at = before;
        for (int u = ua; u < ub; ++u) {
            Seg s;
            if (u == ub - 1) { s.len = len0; s.seq = seq0; }
            else s.len = unit_len(k, u, &s.seq, false);
            s.n = (s.len + kTile - 1) / kTile;
            if (lo < at + s.n) {                 // and publishes the first segment at once
                s.unit = u;
                s.k0 = (int)(lo - at);
                s.k1 = (int)min((long long)s.n, s.k0 + hi - lo);
                sm.seg[0] = s;
                tc::mbar_arrive(&sm.seg_full[0]);
                // Its queries, too: the first two stages are free.
                const int g = u / k.m_tiles, q0 = g * k.group_rows + (u - g * k.m_tiles) * kM + rank * kRows;
                tc::mbar_expect_tx(&sm.q_full, 2 * kStageBytes);
                for (int i = 0; i < 2; ++i) tc::tma_load_3d(sm.ring[i], &qmap, &sm.q_full, 0, q0 + i * 32, 0);
                if (rank == 0) {
                    WsHeader* w = static_cast<WsHeader*>(a.ws);
                    w->unit[cluster] = u;
                    w->k0[cluster] = s.k0;
                }
                break;
            }
            at += s.n;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) static_cast<WsHeader*>(a.ws)->clusters = n_runs;
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync_all();                      // both CTAs' barriers and TMEM exist
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    tc::tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    // Segments, as every role but the plan takes them.
    int seg_i = 0;
    auto next_seg = [&](Seg& s) -> bool {
        const int d = seg_i % kSegs;
        const bool ok = __all_sync(0xffffffffu, wait(&sm.seg_full[d], (seg_i / kSegs) & 1, abort_flag));
        s = sm.seg[d];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.seg_empty[d]);
        ++seg_i;
        return ok && s.unit >= 0;
    };
    // Queries of a segment into the two stages at ring position r (one warp).  The segment before must have taken
    // its own: their barrier counts one phase at a time.  The first segment's are on their way since the plan.
    auto load_q = [&](const Seg& s, int r, int seg) -> bool {
        if (seg == 0) return true;
        const int g = s.unit / k.m_tiles, q0 = g * k.group_rows + (s.unit - g * k.m_tiles) * kM + rank * kRows;
        bool ok = __all_sync(0xffffffffu, wait(&sm.q_taken, (seg - 1) & 1, abort_flag));
        for (int i = 0; i < 2 && ok; ++i) {
            ok = __all_sync(0xffffffffu, wait(&sm.empty[(r + i) % kStages], (((r + i) / kStages) + 1) & 1, abort_flag));
            if (ok && lane == 0) {
                if (i == 0) tc::mbar_expect_tx(&sm.q_full, 2 * kStageBytes);
                tc::tma_load_3d(sm.ring[(r + i) % kStages], &qmap, &sm.q_full, 0, q0 + i * 32, 0);
            }
        }
        return ok;
    };

    if (warp == kPlanWarp<FP8>) {
        // ---------------- plan: the run's segments, then the units that hold padding only
        if (busy) {
            int seg = 1, u = sm.seg[0].unit + 1; // the first is out
            long long left = hi - lo - (sm.seg[0].k1 - sm.seg[0].k0);
            bool ok = true;
            while (ok && left > 0) {
                // 32 units at a time.
                int seq = 0;
                const int len = u + lane < k.units ? unit_len(k, u + lane, &seq, false) : 0;
                for (int i = 0; i < 32 && left > 0 && u + i < k.units; ++i) {
                    Seg s;
                    s.unit = u + i;
                    s.len = __shfl_sync(0xffffffffu, len, i);
                    s.seq = __shfl_sync(0xffffffffu, seq, i);
                    s.n = (s.len + kTile - 1) / kTile;
                    if (s.n == 0) continue;
                    s.k0 = 0;
                    s.k1 = (int)min((long long)s.n, left);
                    left -= s.k1;
                    const int d = seg % kSegs;
                    ok = __all_sync(0xffffffffu, wait(&sm.seg_empty[d], ((seg / kSegs) + 1) & 1, abort_flag));
                    if (!ok) break;
                    if (lane == 0) {
                        sm.seg[d] = s;
                        tc::mbar_arrive(&sm.seg_full[d]);
                    }
                    ++seg;
                }
                u += 32;
                if (u >= k.units) break;
            }
            const int d = seg % kSegs;
            if (ok) ok = __all_sync(0xffffffffu, wait(&sm.seg_empty[d], ((seg / kSegs) + 1) & 1, abort_flag));
            if (ok && lane == 0) {
                sm.seg[d].unit = -1;
                tc::mbar_arrive(&sm.seg_full[d]);
            }
        }
        for (int u0 = blockIdx.x; u0 < k.units; u0 += 32 * gridDim.x) {
            int seq;
            const int u = u0 + lane * gridDim.x;
            unsigned none = __ballot_sync(0xffffffffu, u < k.units && unit_len(k, u, &seq, false) == 0);
            for (; none; none &= none - 1) {
                const int v = u0 + (__ffs(none) - 1) * gridDim.x, g = v / k.m_tiles, r0 = (v - g * k.m_tiles) * kM;
                const size_t row = (size_t)g * k.group_rows + r0;
                const int n = min(k.group_rows - r0, kM), eb = a.o_f32 ? 4 : 2;
                uint4* o = reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.o) + row * kDv * eb);
                for (int i = lane; i < n * kDv * eb / 16; i += 32) o[i] = make_uint4(0, 0, 0, 0);
                if (a.lse)
                    for (int i = lane; i < n; i += 32) a.lse[row + i] = kNegInf;
            }
        }
    } else if (busy && warp == kMmaWarp) {
        // ---------------- MMA issuer (CTA 0)
        if (rank == 0) {
            const uint32_t idesc_s = tc::idesc_f16(128, kTile, 1), idesc_o = tc::idesc_f16_bmn(128, 256, 1);
            int r = 0, tile = 0, seg = 0;        // ring position, key tiles so far, segments so far
            uint32_t k_ph = 0;                   // parity of each stage's next keys
            const bool leader = tc::elect_one();
            bool ok = true, any = false;
            Seg s;
            while (ok && next_seg(s)) {
                r += 2;                          // the queries' stages
                const int n = s.k1 - s.k0;
                if (leader) {
                    ok = wait(&sm.q_ready, seg & 1, abort_flag);
                    auto score = [&](int i) {
                        const int st = (r + i) % kStages, bf = (tile + i) & 1;
                        ok = ok && wait(&sm.s_free[bf], (((tile + i) >> 1) + 1) & 1, abort_flag) &&
                             wait(&sm.k_full[st], (k_ph >> st) & 1, abort_flag);
                        if (!ok) return;
                        k_ph ^= 1u << st;
                        tc::tc_fence_after();
                        const uint32_t ka = tc::smem_u32(sm.ring[st]), qa = tc::smem_u32(sm.q[0]);
#pragma unroll
                        for (int at = 0; at < kAtoms; ++at)
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk) {
                                const uint64_t bd = tc::sdesc_sw128_lbo(ka + at * kAtom + kk * 32, 16, kGroup);
                                if (at < kQTmem) mma2_ts(tmem + kSCol + bf * 32, tmem + kQCol + at * 32 + kk * 8, bd, idesc_s, (at | kk) != 0);
                                else mma2_ss(tmem + kSCol + bf * 32, tc::sdesc_sw128(qa + (at - kQTmem) * (kRows * 128) + kk * 32), bd, idesc_s, 1u);
                            }
                        commit2(&sm.s_full[bf]);
                        commit2(&sm.x_go[st]);
                        any = true;
                    };
                    auto weigh = [&](int i) {
                        const int st = (r + i) % kStages, pb = (tile + i) & 1;
                        ok = ok && wait(&sm.p_full[pb], ((tile + i) >> 1) & 1, abort_flag);
                        if (!ok) return;
                        tc::tc_fence_after();
                        const uint32_t va = tc::smem_u32(sm.ring[st]), pa = tc::smem_u32(sm.p[pb]);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const uint64_t ad = tc::sdesc_sw128(pa + kk * 32);
                            const uint32_t vk = va + (kk >> 1) * 4 * kAtom + (kk & 1) * 2 * kGroup;
#pragma unroll
                            for (int ob = 0; ob < 2; ++ob)
                                mma2_ss(tmem + ob * 128, ad, tc::sdesc_sw128_lbo(vk + ob * 2 * kAtom, kAtom, kGroup), idesc_o,
                                        (i | kk) != 0);
                        }
                        commit2(&sm.empty[st]);
                        commit2(&sm.pv_done[pb]);
                    };
                    // S runs two tiles ahead of P V.
#pragma unroll 1
                    for (int i = -2; i < n && ok; ++i) {
                        if (i + 2 < n) score(i + 2);
                        if (ok && i >= 0) weigh(i);
                    }
                }
                ok = __all_sync(0xffffffffu, ok);
                r += n;
                tile += n;
                ++seg;
            }
            if (leader && any) {                 // drain before TMEM is freed
                volatile int drain = 0;
                commit2(&sm.mma_done);
                wait(&sm.mma_done, 0, &drain);
            }
        }
    } else if (busy && warp < kSoftmaxWarps) {
        // ---------------- softmax: lane L of TMEM = row L & 63, keys 32 (L >> 6) .. + 31 of a tile.  Warpgroup wg takes
        // the tiles of score buffer and P buffer wg
        const int wg = warp >> 2, quarter = warp & 3, L = quarter * 32 + lane, row = L & 63, hf = L >> 6;
        const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
        int r = 0, tile = 0, seg = 0;            // ring position and key tiles before the segment, segments so far
        uint32_t stage_ph = 0, hand_ph = 0;      // parity of each stage's next phase; of the next hand-over
        bool alive = true;
        Seg s;
        // Queries of the next segment from the two stages at ring position r to their operand places; each warpgroup
        // takes half the atoms.
        auto take_q = [&](int r) {
            alive = alive && __all_sync(0xffffffffu, wait(&sm.q_full, seg & 1, abort_flag));
            if (!alive) return;
            const uint8_t* src = sm.ring[(r + (row >> 5)) % kStages] + (row & 31) * 128;
#pragma unroll
            for (int a3 = 0; a3 < kQTmem / 2; ++a3) {
                const int at = wg * (kQTmem / 2) + a3;
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    const uint4 v = *reinterpret_cast<const uint4*>(src + at * kQAtom + ((c ^ (row & 7)) << 4));
                    w[4 * c] = v.x; w[4 * c + 1] = v.y; w[4 * c + 2] = v.z; w[4 * c + 3] = v.w;
                }
                if constexpr (FP8)
#pragma unroll
                    for (int c = 0; c < 32; ++c) w[c] = up2(w[c]);
                tc::tmem_st32(tmem + kQCol + at * 32 + lane_off, w);
            }
            // The other atoms keep their swizzle: bytes move as they are, a quarter of a row per thread (rows side by side at different
            // chunks: other banks).
#pragma unroll
            for (int at = kQTmem; at < kAtoms; ++at)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint4 v = *reinterpret_cast<const uint4*>(src + at * kQAtom + ((4 * hf + 2 * wg + c ^ row & 7) << 4));
                    if constexpr (FP8) v = make_uint4(up2(v.x), up2(v.y), up2(v.z), up2(v.w));
                    *reinterpret_cast<uint4*>(sm.q[at - kQTmem] + row * 128 + ((4 * hf + 2 * wg + c ^ row & 7) << 4)) = v;
                }
            tc::fence_proxy_async_smem();
            tc::tmem_wait_st();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                tc::mbar_arrive(&sm.q_taken);
                arrive0(&sm.q_ready);
            }
            if (warp == 0) {                     // the stages are free once every warp has read them
                alive = __all_sync(0xffffffffu, wait(&sm.q_taken, seg & 1, abort_flag));
                if (alive && lane == 0) {
                    tc::mbar_arrive(&sm.empty[r % kStages]);
                    tc::mbar_arrive(&sm.empty[(r + 1) % kStages]);
                }
            }
        };
        // The value of the other half of this row (its thread is two warps away in the warpgroup).
        int swaps = 0;
        auto swap = [&](float v) -> float {
            const int bf = swaps & 1;
            sm.mx[wg][bf][L] = v;
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&sm.pair[wg][quarter & 1]);
            alive = alive && __all_sync(0xffffffffu, wait(&sm.pair[wg][quarter & 1], swaps & 1, abort_flag));
            ++swaps;
            return sm.mx[wg][bf][L ^ 64];
        };
        // Per segment: its queries, then the epilogue of the one before (so that the new scores run meanwhile), then its tiles.
        Seg cur;                                 // the segment whose tiles are done
        int g = 0, grow = 0;                     // its group; this thread's row in it
        float m = kNegInf, l = 0.f;              // reference maximum this warpgroup last used, its sum
#pragma unroll 1
        for (bool first = true; alive; first = false) {
            const bool have = next_seg(s);
            int lim = 0;                         // keys this row sees in the new segment
            if (have) {
                const int g1 = s.unit / k.m_tiles, row1 = (s.unit - g1 * k.m_tiles) * kM + rank * kRows + row;
                if (row1 < k.group_rows) {
                    const int t = g1 * a.q_group + row1 / a.H;
                    const int pos = a.q_pos[t], seq = a.q_seq[t], sl = a.seq_len[s.seq];        // together, then compared
                    lim = pos >= 0 && seq == s.seq && pos < sl ? pos + 1 : 0;
                }
            }
            if (!first) {
                // Both warpgroups' sums at the larger of their references; past this barrier both have seen their last scores,
                // so the queries may be replaced.
                if (hf == 0) sm.m_last[wg][row] = m;
                sm.l_last[wg][L] = l;
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.both);
                alive = __all_sync(0xffffffffu, wait(&sm.both, (seg - 1) & 1, abort_flag));
                if (!alive) break;
                const float m0 = sm.m_last[0][row], m1 = sm.m_last[1][row];
                m = fmaxf(m0, m1);
                // No reference yet: the sum is 0, or NaN.
                l = (m0 == kNegInf ? sm.l_last[0][L] : sm.l_last[0][L] * ex2(m0 - m)) +
                    (m1 == kNegInf ? sm.l_last[1][L] : sm.l_last[1][L] * ex2(m1 - m));
                l += swap(l);                        // x + y = y + x: both halves hold the same sum
            }
            if (have) take_q(r);
            if (!alive) break;
            if (!first) {
                for (int j = max(0, tile - 2); j < tile; ++j)          // both buffers' last products
                    alive = alive && __all_sync(0xffffffffu, wait(&sm.pv_done[j & 1], (j >> 1) & 1, abort_flag));
                if (!alive) break;
                tc::tc_fence_after();
                // A sum of 0 means that the row saw no key; NaN (a query that is not finite) stays NaN.
                const float inv = l == 0.f ? 0.f : (FP8 ? kUp / a.sm_scale_log2 : 1.f) / l;
                const float lse = l == 0.f ? kNegInf : (m + log2f(l)) * 0.69314718055994530942f;
                const bool whole = cur.k0 == 0 && cur.k1 == cur.n;
                const int slot = 2 * cluster + (cur.k0 == 0 ? 1 : 0);
                const bool write = grow < k.group_rows;
                const size_t orow = (size_t)g * k.group_rows + grow;
                float4* part = part_o(a.ws, slot, rank) + L;        // rows past the group's are not written
                if (hf == 0 && wg == 0 && write) {
                    if (!whole) part_lse(a.ws, slot)[rank * kRows + row] = lse;
                    else if (a.lse) a.lse[orow] = lse;
                }
                uint8_t* stage = sm.p[wg] + quarter * 2048;        // its product is done
#pragma unroll 1
                for (int c = wg * 128; c < wg * 128 + 128; c += 32) {
                    uint32_t ov[32];
                    tc::tmem_ld32(tmem + c + lane_off, ov);
                    tc::tmem_wait_ld();
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = l == 0.f ? 0.f : __uint_as_float(ov[e]) * inv;
                    if (!whole) {                // lanes side by side
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (write) part[(c / 4 + e) * 128] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    } else if (a.o_f32) {
                        float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.o) + orow * kDv + hf * 256 + c);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (write) d[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    } else {                     // 64 bytes of 32 rows through shared memory: 8 rows a store
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            *reinterpret_cast<uint4*>(stage + lane * 64 + ((e ^ (lane >> 1 & 3)) << 4)) =
                                make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                           pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
                        __syncwarp();
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int rr = e * 8 + lane / 4, ch = lane & 3;
                            if (grow - row + (rr + quarter * 32 & 63) < k.group_rows)
                                *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + (orow - row + (rr + quarter * 32 & 63)) * kDv + hf * 256 + c + ch * 8) =
                                    *reinterpret_cast<const uint4*>(stage + rr * 64 + ((ch ^ (rr >> 1 & 3)) << 4));
                        }
                    }
                    __syncwarp();
                }
                // The next segment's first product overwrites O: not before both warpgroups have read theirs.
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&sm.o_read);
                if (have) alive = alive && __all_sync(0xffffffffu, wait(&sm.o_read, (seg - 1) & 1, abort_flag));
            }
            if (!have || !alive) break;
            cur = s;
            ++seg;
            r += 2;
            const int n = s.k1 - s.k0;
            g = s.unit / k.m_tiles;
            grow = (s.unit - g * k.m_tiles) * kM + rank * kRows + row;
            m = kNegInf;
            l = 0.f;
            for (int i = (tile ^ wg) & 1; i < n; i += 2) {
                const int tl = tile + i, st = (r + i) % kStages, key0 = (s.k0 + i) * kTile;
                alive = __all_sync(0xffffffffu, wait(&sm.s_full[wg], (tl >> 1) & 1, abort_flag));
                if (!alive) break;
                tc::tc_fence_after();
                // A stage comes round every kStages tiles; its phases before this tile's are complete, since the tile's keys
                // replaced a stage whose product was done.
                const uint32_t turn = (stage_ph >> st ^ i / kStages) & 1;
                if (FP8) {
                    alive = __all_sync(0xffffffffu, wait(&sm.sc_full[st], turn, abort_flag));
                    if (!alive) break;
                }
                uint32_t w[32];
                tc::tmem_ld32(tmem + kSCol + wg * 32 + lane_off, w);
                tc::tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive0(&sm.s_free[wg]);
                // Scores in log2 units: x = w * sc for BF16 (sc folded into the exponent's multiply-add), w for FP8 after the
                // rows' scales.
                float x[32];
                const float sc = FP8 ? 1.f : a.sm_scale_log2;
                if constexpr (FP8) {
                    const float4* ks = reinterpret_cast<const float4*>(&sm.kscale[st][hf * 32]);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float4 v = ks[e];
                        x[4 * e + 0] = __uint_as_float(w[4 * e + 0]) * v.x;
                        x[4 * e + 1] = __uint_as_float(w[4 * e + 1]) * v.y;
                        x[4 * e + 2] = __uint_as_float(w[4 * e + 2]) * v.z;
                        x[4 * e + 3] = __uint_as_float(w[4 * e + 3]) * v.w;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(w[e]);
                }
                const int left = lim - key0 - hf * 32;
                if (__any_sync(0xffffffffu, left < 32)) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (e >= left) x[e] = kNegInf;
                }
                float mx[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) mx[e] = fmaxf(fmaxf(x[e], x[e + 8]), fmaxf(x[e + 16], x[e + 24]));
                float mt = fmaxf(fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), fmaxf(fmaxf(mx[4], mx[5]), fmaxf(mx[6], mx[7]))) * sc;
                mt = fmaxf(mt, swap(mt));
                // The reference rises only when the tile exceeds it by more than 2^8 (both halves alike).  These decisions are
                // one chain over the segment's tiles, handed from one warpgroup to the other.
                float m_prev = m;
                if (i > 0) {
                    alive = alive && __all_sync(0xffffffffu, wait(&sm.hand[wg ^ 1][quarter], hand_ph, abort_flag));
                    hand_ph ^= 1;
                    m_prev = sm.m_ref[L];
                }
                if (!alive) break;
                float alpha = 1.f, m_new = m_prev;
                bool rescale = false;
                if (mt > m_prev + 8.f) {
                    if (m_prev != kNegInf) { alpha = ex2(m_prev - mt); rescale = true; }
                    m_new = mt;
                }
                if (i + 1 < n) {
                    sm.m_ref[L] = m_new;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sm.hand[wg][quarter]);
                }
                if (m_new != m) {                // this warpgroup's sum to the new reference
                    if (m != kNegInf) l *= ex2(m - m_new);
                    m = m_new;
                }
                const float mref = m == kNegInf ? 0.f : m;
                const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-mref, -mref);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                uint32_t pw[16];
                const float2* vs = reinterpret_cast<const float2*>(&sm.kscale[st][hf * 32]);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float2 p = ffma2(make_float2(x[2 * e], x[2 * e + 1]), sc2, m2);
                    p.x = ex2(p.x);
                    p.y = ex2(p.y);
                    sum[e & 1].x += p.x;
                    sum[e & 1].y += p.y;
                    if constexpr (FP8) {                           // the row's scale goes into its weight
                        const float2 v = vs[e];
                        p.x *= v.x;
                        p.y *= v.y;
                    }
                    pw[e] = pack_bf16x2(p.x, p.y);
                }
                l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
                // P into its buffer once the product two tiles ago has read it.
                if (tl >= 2) alive = __all_sync(0xffffffffu, wait(&sm.pv_done[wg], ((tl >> 1) - 1) & 1, abort_flag));
                if (!alive) break;
                uint8_t* prow = sm.p[wg] + row * 128;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    *reinterpret_cast<uint4*>(prow + (((4 * hf + c) ^ (row & 7)) << 4)) =
                        make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
                if (__any_sync(0xffffffffu, rescale)) {
                    // O must hold every product before this tile's: P V of the tile before, whose barrier's earlier phase
                    // (three tiles ago) is complete -- this tile's scores were issued after that product.
                    if (i > 0) {
                        alive = __all_sync(0xffffffffu, wait(&sm.pv_done[wg ^ 1], ((tl - 1) >> 1) & 1, abort_flag));
                        if (!alive) break;
                    }
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int c = 0; c < 256; c += 32) {
                        uint32_t ov[32];
                        tc::tmem_ld32(tmem + c + lane_off, ov);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tc::tmem_st32(tmem + c + lane_off, ov);
                    }
                    tc::tmem_wait_st();
                }
                // Not before the tile's value rows are there.
                alive = __all_sync(0xffffffffu, wait(&sm.x_full[st], turn, abort_flag));
                if (!alive) break;
                if (!FP8 && key0 + kTile > s.len) {                // value rows behind the last key: zero
                    const int from = s.len - key0;
                    for (int j = L; j < (kTile - from) * 32; j += 128) {
                        const int rr = from + (j >> 5), c = j & 31;
                        *reinterpret_cast<uint4*>(sm.ring[st] + ((rr & 31) >> 3) * kGroup + ((rr >> 5) * 4 + (c >> 3)) * kAtom + (rr & 7) * 128 + (c & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                }
                tc::fence_proxy_async_smem();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive0(&sm.p_full[wg]);
            }
            // Keys seen, but every score -inf (an infinite query): no reference came of the segment's first tile.
            if (wg == (tile & 1) && m == kNegInf && lim > s.k0 * kTile) l = __int_as_float(0x7fc00000);
            // The stages' parities move on for the tiles of both warpgroups.
            if (n / kStages & 1) stage_ph ^= (1u << kStages) - 1;
            for (int i = n - n % kStages; i < n; ++i) stage_ph ^= 1u << ((r + i) % kStages);
            r += n;
            tile += n;
        }
    } else if (busy && (warp == kLoadWarp<FP8> || warp == kXWarp<FP8>)) {
        // ---------------- TMA loads.  First warp: queries and own keys (FP8: their codes); second: the exchanged value rows
        const bool xw = warp == kXWarp<FP8>;
        const int my0 = xw ? (rank ^ 1) * kOwn : rank * kOwn;      // first key in a tile of the rows this warp loads
        int r = 0, tile = 0, seg = 0;
        uint32_t go_ph = 0;
        bool ok = true;
        Seg s;
        while (ok && next_seg(s)) {
            if (!xw) ok = load_q(s, r, seg++);
            r += 2;
            const int n = s.k1 - s.k0;
            // Lane l: page and first row of 8-row group l % 4 of tile base + l / 4; 8 tiles at a time.
            auto fetch = [&](int base, int* in_page) -> int {
                const int key = (s.k0 + base + lane / 4) * kTile + my0 + (lane % 4) * 8;
                *in_page = 0;
                if (base + lane / 4 >= n || key >= s.len) return a.n_pages;        // outside the map: zeros
                const int pg = page_of(a, s.seq, key, in_page);
                // Sequences or pages that share their rows (stride 0) are one in the map.
                return pg < 0 ? a.n_pages : (a.seq_b ? pg : 0);
            };
            int nrow, npg = fetch(0, &nrow), crow = 0, cpg = 0;
            for (int i = 0; i < n && ok; ++i, ++r, ++tile) {
                const int o = i % 8;
                if (o == 0) {
                    crow = nrow; cpg = npg;
                    npg = fetch(i + 8, &nrow);
                }
                const int st = r % kStages;
                if (xw) {
                    ok = __all_sync(0xffffffffu, wait(&sm.x_go[st], (go_ph >> st) & 1, abort_flag));
                    go_ph ^= 1u << st;
                } else {
                    ok = __all_sync(0xffffffffu, wait(&sm.empty[st], ((r / kStages) + 1) & 1, abort_flag));
                }
                if (!ok) break;
                const uint32_t bar0 = tc::peer_smem(&sm.k_full[st], 0);
                if (lane == 0) {
                    if (xw) tc::mbar_expect_tx(&sm.x_full[st], kXBytes);
                    else if (FP8) tc::mbar_expect_tx(&sm.code_full[tile & 1][st], kCodeBytes);
                    else if (rank == 0) tc::mbar_expect_tx(&sm.k_full[st], 2 * kStageBytes);
                }
                __syncwarp();
                const int pg = __shfl_sync(0xffffffffu, cpg, o * 4 + (lane & 3)), rw = __shfl_sync(0xffffffffu, crow, o * 4 + (lane & 3));
                if (xw) {                        // 256 dims of 8 rows a box
                    if (lane < 4) tma_load_4d(sm.ring[st] + lane * kGroup + (rank ^ 1) * 4 * kAtom, &xmap, &sm.x_full[st], 0, rw, rank * 4, pg);
                } else if (FP8) {
                    if (lane < 4) tma_load_4d(sm.ring[st] + lane * kGroup + kCodeAt, &kmap, &sm.code_full[tile & 1][st], 0, rw, 0, pg);
                } else if (lane < 4) {           // 8 rows a box
                    tma_load_4d_pair(sm.ring[st] + lane * kGroup, &kmap, bar0, 0, rw, 0, pg);
                }
            }
        }
    } else if (busy && FP8) {
        // ---------------- FP8.  Eight warps widen the own keys' codes landed in the stage, four the exchanged rows', one brings
        // the row scales.
        // Own keys 0..7: warps 9, 10, 11, 12 and 13, 14, 15, 17; exchanged rows 8..11: 18, 19, 20, 23; scales 12: 22.
        const int w = warp < 16 ? warp - 9 : (warp == 17 ? 7 : (warp == 22 ? 12 : (warp == 23 ? 11 : warp - 10)));
        int r = 0, tile = 0;
        uint32_t ph = 0;                         // parity of each stage's next phase (codes landed, by set; scores done)
        bool ok = true;
        Seg s;
        // n atoms of codes at `from` to n atoms at `to` (this lane's 16 codes of each).
        auto widen = [&](const uint8_t* from, uint8_t* to, int n) {
            uint8_t* to2 = reinterpret_cast<uint8_t*>((uintptr_t)to ^ 16);         // the next 8 dims under the swizzle
            uint4 next = *reinterpret_cast<const uint4*>(from);
#pragma unroll 3                                 // the roles share the instruction caches: unrolled whole, 537 instead of 447 us
            for (int c = 0; c < n; ++c) {        // for 32 tokens of 128 heads at 32K-64K
                const uint4 v = next;
                from += kAtom / 2;
                if (c + 1 < n) next = *reinterpret_cast<const uint4*>(from);
                __syncwarp();                    // atom c + 1 is read before atom c is written
                const uint2 w0 = widen4(v.x), w1 = widen4(v.y), w2 = widen4(v.z), w3 = widen4(v.w);
                *reinterpret_cast<uint4*>(to) = make_uint4(w0.x, w0.y, w1.x, w1.y);
                *reinterpret_cast<uint4*>(to2) = make_uint4(w2.x, w2.y, w3.x, w3.y);
                to += kAtom;
                to2 += kAtom;
            }
        };
        if (w < kKWarps) {
            // Warps 0..3 take the even tiles, 4..7 the odd ones; warp = 8-row group, which only it reads and writes.  Lane: 16
            // codes of an atom, row lane / 4.
            const int g = w & 3, set = w >> 2, r8 = lane >> 2;
            const int src = g * kGroup + kCodeAt + lane * 16, dst = g * kGroup + r8 * 128 + (((lane & 3) * 2 ^ r8) << 4);
            while (ok && next_seg(s)) {
                r += 2;
                const int n = s.k1 - s.k0;
                for (int i = (tile ^ set) & 1; i < n; i += 2) {
                    // The stage's barrier of this set: its phases are this set's tiles alone, none of which completes unless the warp
                    // saw the one before.  (A warp must not wait on what goes on without it: such a phase can be over, and the next
                    // one too, before it looks, and the parity then says "not yet" for good.)
                    const int st = (r + i) % kStages;
                    ok = __all_sync(0xffffffffu, wait(&sm.code_full[set][st], (ph >> st) & 1, abort_flag));
                    if (!ok) break;
                    ph ^= 1u << st;
                    // A row whose codes are NaN (stored so by the append for a row with a NaN or an infinity; widening moves
                    // bits and would make them numbers) gets a NaN among its rotary dims, which only the scores read.
                    const bool bad = (sm.ring[st][src + (kAtoms - 1) * (kAtom / 2)] & 0x7f) == 0x7f;
                    widen(sm.ring[st] + src, sm.ring[st] + dst, kAtoms);
                    if (bad) *reinterpret_cast<uint32_t*>(sm.ring[st] + dst + (kAtoms - 1) * kAtom) = 0x7fc07fc0u;
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) arrive0(&sm.k_full[st]);
                }
                r += n;
                tile += n;
            }
        } else if (w < kKWarps + kXWarps) {
            // Warp = 8-row group of the exchanged rows: once the scores have read the dims that they replace, their codes land
            // in the tail of that place (the other CTA has brought them into L2) and widen as the keys do, four atoms.
            const int g = w - kKWarps, r8 = lane >> 2;
            const int at = g * kGroup + (rank ^ 1) * 4 * kAtom;
            const int src = at + 2 * kAtom + lane * 16, dst = at + r8 * 128 + (((lane & 3) * 2 ^ r8) << 4);
            while (ok && next_seg(s)) {
                r += 2;
                const int n = s.k1 - s.k0;
                // Lane l: page and row of the group in tile base + l.
                auto fetch = [&](int base, int* row) -> int {
                    const int key = (s.k0 + base + lane) * kTile + (rank ^ 1) * kOwn + g * 8;
                    *row = 0;
                    if (base + lane >= n || key >= s.len) return a.n_pages;        // outside the map: zeros
                    const int pg = page_of(a, s.seq, key, row);
                    return pg < 0 ? a.n_pages : (a.seq_b ? pg : 0);
                };
                int nrow, npg = fetch(0, &nrow), crow = 0, cpg = 0;
                for (int i = 0; i < n; ++i, ++r, ++tile) {
                    if (i % 32 == 0) {
                        crow = nrow; cpg = npg;
                        npg = fetch(i + 32, &nrow);
                    }
                    const int st = r % kStages;
                    ok = __all_sync(0xffffffffu, wait(&sm.x_go[st], (ph >> st) & 1, abort_flag));
                    ph ^= 1u << st;
                    if (!ok) break;
                    if (lane == i % 32) {
                        tc::mbar_expect_tx(&sm.x_code[g], 4 * kAtom / 2);
                        tma_load_4d(sm.ring[st] + at + 2 * kAtom, &xmap, &sm.x_code[g], 0, crow, rank * 4, cpg);
                    }
                    ok = __all_sync(0xffffffffu, wait(&sm.x_code[g], tile & 1, abort_flag));
                    if (!ok) break;
                    widen(sm.ring[st] + src, sm.ring[st] + dst, 4);
                    tc::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sm.x_full[st]);
                }
            }
        } else {
            // Row scales, lane l: keys l and l + 32, loaded a tile ahead.  They are put out once the tile's codes have landed: its
            // stage is free then, and every phase of those barriers is seen (the stage's own has phases of queries between, which
            // end before the products of the tiles in front of them).
            const float up = kUp * a.sm_scale_log2;
            while (ok && next_seg(s)) {
                r += 2;
                const int n = s.k1 - s.k0;
                // Lane l: index of the first scale of 8-row group l % 8 of tile base + l / 8; 4 tiles at a time, a batch ahead.
                auto fetch = [&](int base) -> int64_t {
                    const int key = (s.k0 + base + lane / 8) * kTile + (lane % 8) * 8;
                    if (base + lane / 8 >= n || key >= s.len) return -1;
                    int rw;
                    const int pg = page_of(a, s.seq, key, &rw);
                    return pg < 0 ? -1 : pg * a.scale_seq + rw;
                };
                int64_t at = fetch(0), at_next = fetch(4);
                float n0 = 0.f, n1 = 0.f;
                auto load = [&](int i) {
                    if (i % 4 == 0 && i > 0) {
                        at = at_next;
                        at_next = fetch(i + 4);
                    }
                    const int left = s.len - (s.k0 + i) * kTile;
                    const int64_t o0 = __shfl_sync(0xffffffffu, at, (i % 4) * 8 + lane / 8), o1 = __shfl_sync(0xffffffffu, at, (i % 4) * 8 + 4 + lane / 8);
                    n0 = i < n && o0 >= 0 && lane < left ? __ldg(a.kv_scale + o0 + lane % 8) : 0.f;
                    n1 = i < n && o1 >= 0 && lane + 32 < left ? __ldg(a.kv_scale + o1 + lane % 8) : 0.f;
                };
                load(0);
                for (int i = 0; i < n; ++i, ++r, ++tile) {
                    const float s0 = n0, s1 = n1;
                    load(i + 1);
                    const int st = r % kStages, bit = (tile & 1) * kStages + st;
                    ok = __all_sync(0xffffffffu, wait(&sm.code_full[tile & 1][st], (ph >> bit) & 1, abort_flag));
                    if (!ok) break;
                    ph ^= 1u << bit;
                    sm.kscale[st][lane] = s0 * up;
                    sm.kscale[st][32 + lane] = s1 * up;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sm.sc_full[st]);
                }
            }
        }
    }
    __syncwarp();
    if (*abort_flag) {                           // copies in flight land well within this time
        const uint64_t t0 = tc::global_ns();
        while (tc::global_ns() - t0 < 2000000ull) __nanosleep(1000);
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::cluster_sync_all();                      // no CTA leaves while the other may still signal it
    if (sm.abort && threadIdx.x == 0) report(a.status, LSA_ERR_TIMEOUT);
    if (warp == kMmaWarp) {
        tc::tc_fence_after();
        tmem_dealloc2(tmem, 512);
    }
}

// Joins the partial results of the units that a run's start cuts.  Block (x, y): with one group (P = 1) run x + 1's first
// unit, when that run is the first to start inside it, else unit x; a CTA's rows and 4 V dims of each half-row.  Thread = lane of the partial results, in
// one of P groups; a group takes every P-th part in key order with weights exp(lse - its own maximum), and the groups'
// results are joined in order the same way.  Launched while the attention still runs: it waits for its end.
template <int V, int P>
__global__ void __launch_bounds__(128 * P) latent_merge_kernel(const __grid_constant__ LatentKernelArgs k) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const LatentArgs& a = k.a;
    const WsHeader* ws = static_cast<const WsHeader*>(a.ws);
    __shared__ WsHeader sh;                      // read at once: the runs of a unit are counted one after another
    __shared__ float4 acc_s[P > 1 ? P - 1 : 1][V][P > 1 ? 128 : 1];
    __shared__ float2 stat_s[P > 1 ? P - 1 : 1][P > 1 ? 128 : 1];
    WsHeader* w = &sh;
    for (int i = threadIdx.x; i < kMaxClusters; i += blockDim.x) { w->unit[i] = ws->unit[i]; w->k0[i] = ws->k0[i]; }
    const int n_runs = ws->clusters;
    int c, u, last;                              // runs c .. last start inside unit u
    if constexpr (P == 1) {
        c = blockIdx.x + 1;
        __syncthreads();
        if (c >= n_runs || w->k0[c] == 0) return;
        u = w->unit[c];
        if (w->unit[c - 1] == u && w->k0[c - 1] > 0) return;       // an earlier run is the first
        last = c;
        while (last + 1 < n_runs && w->unit[last + 1] == u) ++last;
    } else {
        __shared__ int first;
        u = blockIdx.x;
        if (threadIdx.x == 0) first = kMaxClusters;
        __syncthreads();
        const int i = threadIdx.x;
        const bool in = i < n_runs && w->unit[i] == u && w->k0[i] > 0;
        if (in) atomicMin(&first, i);
        const int n_in = __syncthreads_count(in);
        if (n_in == 0) return;
        c = first;
        last = c + n_in - 1;
    }
    constexpr int kSlices = 64 / V;
    const int rank = blockIdx.y / kSlices, c4 = (blockIdx.y % kSlices) * V;
    const int L = threadIdx.x & 127, part = threadIdx.x >> 7, row = L & 63;
    const int g = u / k.m_tiles, grow = (u - g * k.m_tiles) * kM + rank * kRows + row;
    const bool live = grow < k.group_rows;
    auto slot = [&](int i) { return i == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + i); };
    const int n = last - c + 2;
    float m = kNegInf, sum = 0.f;
    float4 acc[V];
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int e, float x, float4 v) {
        acc[e].x = fmaf(x, v.x, acc[e].x);
        acc[e].y = fmaf(x, v.y, acc[e].y);
        acc[e].z = fmaf(x, v.z, acc[e].z);
        acc[e].w = fmaf(x, v.w, acc[e].w);
    };
    if (live) {
#pragma unroll 8
        for (int i = part; i < n; i += P) m = fmaxf(m, part_lse(a.ws, slot(i))[rank * kRows + row]);
#pragma unroll 8
        for (int i = part; i < n; i += P) {
            const float lse = part_lse(a.ws, slot(i))[rank * kRows + row];
            const float x = lse == kNegInf ? 0.f : expf(lse - m);  // a part without keys holds zeros
            const float4* p = part_o(a.ws, slot(i), rank) + (size_t)c4 * 128 + L;
            sum += x;
#pragma unroll
            for (int e = 0; e < V; ++e) add(e, x, p[e * 128]);
        }
    }
    if constexpr (P > 1) {
        if (part > 0) {
            stat_s[part - 1][L] = make_float2(m, sum);
#pragma unroll
            for (int e = 0; e < V; ++e) acc_s[part - 1][e][L] = acc[e];
        }
        __syncthreads();
        if (part > 0) return;
        float mm = m;
#pragma unroll
        for (int j = 0; j < P - 1; ++j) mm = fmaxf(mm, stat_s[j][L].x);
        const float x0 = m == kNegInf ? 0.f : expf(m - mm);
        sum *= x0;
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = make_float4(acc[e].x * x0, acc[e].y * x0, acc[e].z * x0, acc[e].w * x0);
#pragma unroll
        for (int j = 0; j < P - 1; ++j) {
            const float2 t = stat_s[j][L];
            const float x = t.x == kNegInf ? 0.f : expf(t.x - mm);
            sum = fmaf(x, t.y, sum);
#pragma unroll
            for (int e = 0; e < V; ++e) add(e, x, acc_s[j][e][L]);
        }
        m = mm;
    }
    if (!live) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;                // 0: no key in any part
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = make_float4(acc[e].x * inv, acc[e].y * inv, acc[e].z * inv, acc[e].w * inv);
    const size_t orow = (size_t)g * k.group_rows + grow, at = orow * kDv + (L >> 6) * 256 + c4 * 4;
    if (a.o_f32) {
#pragma unroll
        for (int e = 0; e < V; ++e) reinterpret_cast<float4*>(static_cast<float*>(a.o) + at)[e] = acc[e];
    } else {
#pragma unroll
        for (int e = 0; e < V; e += 2)
            reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + at)[e / 2] =
                make_uint4(pack_bf16x2(acc[e].x, acc[e].y), pack_bf16x2(acc[e].z, acc[e].w),
                           pack_bf16x2(acc[e + 1].x, acc[e + 1].y), pack_bf16x2(acc[e + 1].z, acc[e + 1].w));
    }
    if (L < kRows && c4 == 0 && a.lse) a.lse[orow] = sum == 0.f ? kNegInf : m + logf(sum);
}

// The cache as (64 dims, rows, 9 chunks of dims, pages), box 64 x 8 x `chunks` x 1; BF16 under the 128-byte swizzle, codes plain.
bool make_kv_map(const LatentArgs& a, CUtensorMap* m, int chunks) {
    const bool one = a.n_pages == 1 || a.seq_b == 0, fp8 = a.kv_scale != nullptr;
    const cuuint64_t d[4] = {64, (cuuint64_t)a.page_size, kAtoms, (cuuint64_t)(one ? 1 : a.n_pages)};
    const cuuint64_t s[3] = {(cuuint64_t)a.tok_b, (cuuint64_t)(fp8 ? 64 : 128), (cuuint64_t)(one ? a.tok_b : a.seq_b)};
    const cuuint32_t box[4] = {64, 8, (cuuint32_t)chunks, 1}, e[4] = {1, 1, 1, 1};
    return tc::encode_tiled()(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                              const_cast<uint8_t*>(a.kv), d, s, box, e, CU_TENSOR_MAP_INTERLEAVE_NONE,
                              fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Clusters that run at once on the current device (asked once per device).
template <bool FP8>
int cluster_count(size_t smem) {
    static std::mutex mu;
    static int known[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev]) return known[dev];
    if (cudaFuncSetAttribute(latent_attn_kernel<FP8>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return 0;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * kMaxClusters);
    cfg.blockDim = dim3(kThreadsOf<FP8>);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {2, 1, 1};
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, latent_attn_kernel<FP8>, &cfg) != cudaSuccess || n < 1) return 0;
    return known[dev] = n < kMaxClusters ? n : kMaxClusters;
}

template <bool FP8>
cudaError_t launch_t(const CUtensorMap& qm, const CUtensorMap& km, const CUtensorMap& xm, LatentKernelArgs& k, cudaStream_t st) {
    const size_t smem = sizeof(Smem) + 1024;
    k.clusters = cluster_count<FP8>(smem);
    if (k.clusters < 1) return cudaErrorInvalidConfiguration;
    // No more clusters than the allocated rows can need: a short context launches few, and one alone has nothing to join.
    const int64_t tiles = (int64_t)k.units * ((k.a.L_alloc + kTile - 1) / kTile);
    if ((tiles + kMinRun - 1) / kMinRun < k.clusters) k.clusters = (int)((tiles + kMinRun - 1) / kMinRun);
    latent_attn_kernel<FP8><<<2 * k.clusters, kThreadsOf<FP8>, smem, st>>>(qm, km, xm, k);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || k.clusters == 1) return e;
    // The join is launched while the attention runs, and waits for its end on the device.
    cudaLaunchConfig_t cfg{};
    // Units of eight parts and more: four groups of a block share them.  Units of few: small blocks that wait resident
    // beside the attention (12 units of 6 parts 45.9 us so, 50.4 in groups; one token at 48752 rows, 74 parts, 46.4 us in
    // groups and 73 in one).  The large blocks are few, units x 64: they cannot wait beside the attention, and one set per
    // run, most of it leaving at once, took 31.5 instead of 26.4 us for one token at 27,000 rows.
    const bool wide = k.units * 8 <= k.clusters;
    cfg.gridDim = dim3(wide ? k.units : k.clusters - 1, wide ? 64 : 32);
    cfg.blockDim = dim3(wide ? 512 : 128);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return wide ? cudaLaunchKernelEx(&cfg, latent_merge_kernel<2, 4>, k) : cudaLaunchKernelEx(&cfg, latent_merge_kernel<4, 1>, k);
}

}  // namespace

size_t latent_attn_ws(int, int, int) { return kWsBytes; }

cudaError_t launch_latent_attn(const LatentArgs& a, cudaStream_t st) {
    if (tc::encode_tiled() == nullptr) return cudaErrorNotSupported;
    LatentKernelArgs k{};
    k.a = a;
    k.group_rows = a.q_group * a.H;
    k.m_tiles = (k.group_rows + kM - 1) / kM;
    k.units = a.T / a.q_group * k.m_tiles;
    CUtensorMap qm, km, xm;
    memset(&km, 0, sizeof(km));
    memset(&xm, 0, sizeof(xm));
    {
        const cuuint64_t d[3] = {64, (cuuint64_t)a.T * a.H, kAtoms}, s[2] = {kD * 2, 128};
        const cuuint32_t box[3] = {64, 32, kAtoms}, e[3] = {1, 1, 1};
        if (tc::encode_tiled()(&qm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(a.q), d, s, box, e,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    if (!make_kv_map(a, &km, kAtoms)) return cudaErrorInvalidValue;
    if (!make_kv_map(a, &xm, 4)) return cudaErrorInvalidValue;
    if (a.kv_scale) return launch_t<true>(qm, km, xm, k, st);
    return launch_t<false>(qm, km, xm, k, st);
}

}  // namespace lsa
