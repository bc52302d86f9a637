// Latent attention in the expanded form on the 5th-generation tensor cores: packed prompts with per-head keys
// and values, 64 rotary dimensions shared by the heads.
//
//   z = sm_scale (q[0:128] . k_nope + q[128:192] . k_rope), o = softmax(z) v, one pass over the keys with a
//   running reference maximum and sum.
//
// Work split.  CTA = 256 queries of one (sequence, head) as two tiles of M = 128 rows, against 128 keys at a
// time: each key tile is loaded once for both.  The two tiles take turns on the tensor pipe -- while one
// tile's 128 x 128 scores are in the softmax, the other's products run (O0 += P0 V, S0', O1 += P1 V, S1', ...).
// Per key tile and query tile the pipe needs 12 + 8 MMAs of 64 cycles (S: K = 192; P V: K = 128, N = 128), the
// softmax 16,384 exponentials of 16 a cycle = 1,024 cycles: both pipes are close to full, the tensor one first.
//
// Memory.  TMEM (512 columns): S0, S1 (128 each; the softmax writes P as BF16 over the S it has read), O0, O1
// (128 each).  Shared memory: Q (2 x 3 swizzled 64-dim atoms, 96 KB) and a ring of eight 16 KB units: a key
// tile is five units, three K atoms (64 dims x 128 keys; two of k_nope, the rotary one) and two V units (64 keys
// x 128 dims), each released as soon as its last product is issued.
//
// Items.  A CTA that runs takes over grid blocks that have not been launched yet (cluster launch control), so that the
// start of one block's work -- its plan, queries and first scores -- runs under the end of another's; the order of the
// grid, heaviest query tiles of a head first, stays.  The next block is asked for a few key tiles before the end of the
// one in work, so that no CTA holds two while another has none.
//
// Warps: 0..3 softmax of query tile 0 (thread = row = TMEM lane), 4..7 of tile 1, 8 issues the MMAs, 9 loads keys and
// values by TMA, 10 clears the rows of a sequence's last key tile that lie behind the sequence (0 x whatever they hold
// would reach O), 11 takes the blocks, plans them and loads their queries.  All waits are bounded; a CTA that gives up
// reports LSA_ERR_TIMEOUT.  The waits of warps 9 and 11 take the limit of lsa_set_wait_limit_ns, and every other wait
// ends with the flag that they set; what is in flight then is waited for with the 2 s bound, each with a flag of its own.
//
// Measured on the device: 2048 queries behind 2048 keys, 128 heads, causal: 419-430 us, 1.2 PFLOP/s; 490 us after a tenth of a
// second of such calls, at the power limit (1.5 GHz).  A pair of query tiles takes about 3,700 cycles a key tile where its
// products take 2,560: the chain score, softmax, product shows.
#include <cmath>
#include <cstring>

#include "kernels.cuh"
#include "tc.cuh"

namespace lsa {

namespace {

constexpr int kThreads = 384;
constexpr int kM = 128, kN = 128;                // query rows of a tile, keys of a tile
constexpr int kDn = 128, kDr = 64, kD = kDn + kDr, kDv = 128;
constexpr int kUnits = 8, kUnitBytes = 16384;    // ring
constexpr int kPerTile = 5;                      // units of a key tile: K atoms 0..2, V keys 0..63, 64..127
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kOtherRegs <= kThreads * 168, "register split within the launch's registers");

struct Item {
    int q0, rows, k0, nk, shift;                 // first query row (packed), queries here, first key row, keys, nk - nq
    int i0;                                      // index of the first query in its sequence
    int n[2];                                    // key tiles of each query tile
    int h;
    int more;                                    // 0: no item, the end
};

constexpr int kItems = 2;                        // published items
constexpr int kConsumers = 11;                   // warps that read them
constexpr int kAskAhead = 6;                     // key tiles before an item's end at which the next block is asked for

struct Smem {
    alignas(1024) uint8_t q[2][3][kM * 128];     // query tiles, 64-dim atoms
    alignas(1024) uint8_t ring[kUnits][kUnitBytes];
    alignas(16) uint8_t answer[16];              // of the request for a block
    Item item[kItems];
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t asked, ask;                         // the answer is there; the loads are close to the item's end
    uint64_t full[kUnits], empty[kUnits];
    uint64_t q_full, q_free;                     // the item's queries have landed; its last scores are done
    uint64_t v_last[2];                          // a partial last tile's V units: landed, not yet cleared behind the sequence
    uint64_t mma_done;                           // committed once, after the last MMA (the issuer's drain)
    uint64_t s_full[2], p_full[2][2], o_done[2]; // p_full[tile][keys 0..63 / 64..127]
    uint32_t tmem_base;
    int abort;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A wait under a limit, its slow part a call: the roles share the instruction caches (2048 queries behind 2048 keys, 128
// heads: 444 us with both ways of polling inlined, 428 so).
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    return tc::mbar_wait(bar, parity, abort, limit_ns);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint64_t limit_ns) {
    return tc::mbar_test_wait(bar, parity) || wait_slow(bar, parity, abort, limit_ns);
}

template <int R>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(R)); }
template <int R>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(R)); }

__global__ void __launch_bounds__(kThreads, 1)
    latent_expanded_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                           const __grid_constant__ CUtensorMap rmap, const __grid_constant__ CUtensorMap vmap,
                           const __grid_constant__ ExpandedArgs a) {
    extern __shared__ uint8_t smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sm.abort;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i) {
            tc::mbar_init(&sm.item_full[i], 1);
            tc::mbar_init(&sm.item_empty[i], kConsumers);
        }
        tc::mbar_init(&sm.asked, 1);
        tc::mbar_init(&sm.ask, 1);
        for (int i = 0; i < kUnits; ++i) {
            tc::mbar_init(&sm.full[i], 1);
            tc::mbar_init(&sm.empty[i], 1);
        }
        tc::mbar_init(&sm.q_full, 1);
        tc::mbar_init(&sm.q_free, 1);
        tc::mbar_init(&sm.v_last[0], 1);
        tc::mbar_init(&sm.v_last[1], 1);
        tc::mbar_init(&sm.mma_done, 1);
        for (int t = 0; t < 2; ++t) {
            tc::mbar_init(&sm.s_full[t], 1);
            tc::mbar_init(&sm.p_full[t][0], 4);
            tc::mbar_init(&sm.p_full[t][1], 4);
            tc::mbar_init(&sm.o_done[t], 1);
        }
        sm.abort = 0;
        tc::fence_barrier_init();
    }
    if (warp == 8) tc::tmem_alloc(&sm.tmem_base, 512);
    if (threadIdx.x == 9 * 32) {
        tc::prefetch_tmap(&qmap);
        if (a.S > 0) {                           // without keys the other maps are not encoded, and not touched
            tc::prefetch_tmap(&kmap);
            tc::prefetch_tmap(&rmap);
            tc::prefetch_tmap(&vmap);
        }
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    // Items, as every role but warp 11 takes them.
    int item_i = 0;
    auto next_item = [&](Item& p) -> bool {
        const int d = item_i % kItems;
        const bool ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.item_full[d], (item_i / kItems) & 1, abort_flag));
        p = sm.item[d];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&sm.item_empty[d]);
        ++item_i;
        return ok && p.more;
    };
    auto tiles = [](const Item& p) { return max(p.n[0], p.n[1]); };
    auto is_partial = [&](const Item& p) { return tiles(p) * kN > p.nk; };         // the last key tile reaches behind the sequence

    if (warp >= 8) {
        reg_dec<kOtherRegs>();
        Item p;
        if (warp == 11) {
            // ---------------- blocks: the grid's own, then those not launched yet
            if (tc::elect_one()) {
                int x = blockIdx.x, h = blockIdx.y, b = blockIdx.z, published = 0, loaded = 0, asked = 0;
                bool ok = true, more = true;
                while (ok && more) {
                    const int qs = a.q_start[b], qe = a.q_start[b + 1], ks = a.k_start[b], ke = a.k_start[b + 1];
                    const bool inside = qs >= 0 && qe >= qs && qe <= a.T && ks >= 0 && ke >= ks && ke <= a.S;
                    const int nq = inside ? qe - qs : 0, todo = min(nq, a.max_q);
                    if ((!inside || nq > a.max_q) && x == 0 && h == 0) report(a.status, LSA_ERR_DEVICE_DATA);
                    // The longest query tiles of a causal sequence first.
                    p.i0 = ((todo + 2 * kM - 1) / (2 * kM) - 1 - x) * 2 * kM;
                    if (p.i0 >= 0) {
                        p.q0 = qs + p.i0;
                        p.rows = min(2 * kM, todo - p.i0);
                        p.k0 = ks;
                        p.nk = ke - ks;
                        p.shift = p.nk - nq;
                        p.h = h;
                        p.more = 1;
                        for (int t = 0; t < 2; ++t) {
                            const int r = min(kM, p.rows - t * kM);               // rows of the tile
                            const int end = r <= 0 ? 0 : (a.causal ? min(p.nk, max(0, p.i0 + t * kM + r + p.shift)) : p.nk);
                            p.n[t] = (end + kN - 1) / kN;
                        }
                        const int d = published % kItems;
                        ok = wait(&sm.item_empty[d], ((published / kItems) + 1) & 1, abort_flag, a.wait_ns);
                        if (!ok) break;
                        sm.item[d] = p;
                        tc::mbar_arrive(&sm.item_full[d]);
                        ++published;
                        if (tiles(p) > 0) {
                            ok = loaded == 0 || wait(&sm.q_free, (loaded - 1) & 1, abort_flag, a.wait_ns);
                            if (!ok) break;
                            const int hq = a.qh ? h : 0, n_q = p.rows > kM ? 2 : 1;        // a broadcast head has no stride
                            tc::mbar_expect_tx(&sm.q_full, n_q * 3 * kM * 128);
                            for (int t = 0; t < n_q; ++t)
                                for (int c = 0; c < 3; ++c)
                                    tc::tma_load_3d(sm.q[t][c], &qmap, &sm.q_full, c * 64, hq, p.q0 + t * kM);
                            ok = wait(&sm.ask, loaded & 1, abort_flag, a.wait_ns);
                            ++loaded;
                            if (!ok) break;
                        }
                    }
                    tc::fence_proxy_async_smem();            // the last answer has been read
                    tc::mbar_expect_tx(&sm.asked, 16);
                    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];"
                                 :: "r"(tc::smem_u32(sm.answer)), "r"(tc::smem_u32(&sm.asked)) : "memory");
                    ok = wait(&sm.asked, asked & 1, abort_flag, a.wait_ns);
                    ++asked;
                    if (!ok) break;
                    const volatile uint64_t* an = reinterpret_cast<const volatile uint64_t*>(sm.answer);
                    uint32_t got, cx, cy, cz;
                    asm volatile("{ .reg .b128 r; .reg .pred p; .reg .b32 w;\n"
                                 "mov.b128 r, {%4, %5};\n"
                                 "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n"
                                 "selp.u32 %0, 1, 0, p;\n"
                                 "mov.b32 %1, 0; mov.b32 %2, 0; mov.b32 %3, 0;\n"
                                 "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, %3, w}, r; }"
                                 : "=r"(got), "=r"(cx), "=r"(cy), "=r"(cz) : "l"(an[0]), "l"(an[1]) : "memory");
                    more = got != 0;
                    x = (int)cx;
                    h = (int)cy;
                    b = (int)cz;
                }
                if (ok) ok = wait(&sm.item_empty[published % kItems], ((published / kItems) + 1) & 1, abort_flag, a.wait_ns);
                if (ok) {
                    sm.item[published % kItems].more = 0;
                    tc::mbar_arrive(&sm.item_full[published % kItems]);
                }
                // No copy and no answer outlives the CTA.
                volatile int drain_q = 0, drain_a = 0;
                if (loaded) tc::mbar_wait(&sm.q_full, (loaded - 1) & 1, &drain_q);
                if (asked) tc::mbar_wait(&sm.asked, (asked - 1) & 1, &drain_a);
            }
        } else if (warp == 9) {
            // ---------------- keys and values: the ring's units in the order of their use
            const bool leader = tc::elect_one();
            int u = 0, partials = 0, last[2] = {-kUnits, -kUnits};  // next unit; partial tiles so far, and the units of the latest
            uint32_t last_ph[2] = {0, 0};        // the phases of v_last that those complete
            bool ok = true;
            while (ok && next_item(p)) {
                const int n_tiles = tiles(p);
                if (leader && n_tiles > 0) {
                    const bool partial = is_partial(p);
                    const int hk = a.kh ? p.h : 0, hv = a.vh ? p.h : 0;
                    for (int j = 0; j < n_tiles && ok; ++j) {
                        if (j == max(0, n_tiles - kAskAhead)) tc::mbar_arrive(&sm.ask);
                        const int row = p.k0 + j * kN;
                        for (int c = 0; c < kPerTile; ++c, ++u) {
                            const int s = u % kUnits;
                            ok = wait(&sm.empty[s], ((u / kUnits) + 1) & 1, abort_flag, a.wait_ns);
                            uint64_t* bar = &sm.full[s];
                            if (ok && c >= 3 && partial && j == n_tiles - 1) {
                                // The V units of a partial last tile pass through warp 10, which then completes `full`; it must be
                                // through with the latest one (unless that unit's place has been used again since).
                                const int w = last[c - 3];
                                if (w > u - kUnits && partials > 0) ok = wait(&sm.full[w % kUnits], (w / kUnits) & 1, abort_flag, a.wait_ns);
                                if (ok) {
                                    bar = &sm.v_last[c - 3];
                                    last[c - 3] = u;
                                    last_ph[c - 3] = partials & 1;
                                }
                            }
                            if (!ok) break;
                            tc::mbar_expect_tx(bar, kUnitBytes);
                            if (c < 2) tc::tma_load_3d(sm.ring[s], &kmap, bar, c * 64, hk, row);
                            else if (c == 2) tc::tma_load_2d(sm.ring[s], &rmap, bar, 0, row);
                            else {
                                tc::tma_load_3d(sm.ring[s], &vmap, bar, 0, hv, row + (c - 3) * 64);
                                tc::tma_load_3d(sm.ring[s] + 8192, &vmap, bar, 64, hv, row + (c - 3) * 64);
                            }
                        }
                    }
                    if (partial && ok) ++partials;
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            // No copy outlives the CTA: all have landed, at once unless a wait gave up.
            if (leader)
                for (int v = max(0, u - kUnits); v < u; ++v) {
                    volatile int drain = 0;
                    const int c = v == last[0] ? 0 : (v == last[1] ? 1 : -1);
                    if (c >= 0) tc::mbar_wait(&sm.v_last[c], last_ph[c], &drain);      // `full` is warp 10's to complete
                    else tc::mbar_wait(&sm.full[v % kUnits], (v / kUnits) & 1, &drain);
                }
        } else if (warp == 8) {
            // ---------------- MMA issuer
            const uint32_t idesc_s = tc::idesc_f16(kM, kN, 1), idesc_o = tc::idesc_f16_bmn(kM, kDv, 1);
            const bool leader = tc::elect_one();
            int u0 = 0, items = 0, done0 = 0, done1 = 0;           // the item's first unit; items with keys; score tiles before it
            bool ok = true, any = false;
            while (ok && next_item(p)) {
                const int n_tiles = tiles(p);
                if (leader && n_tiles > 0) {
                    auto unit = [&](int j, int c) { return (u0 + j * kPerTile + c) % kUnits; };
                    auto landed = [&](int j, int c) {
                        const int u = u0 + j * kPerTile + c;
                        ok = ok && tc::mbar_wait(&sm.full[u % kUnits], (u / kUnits) & 1, abort_flag);
                    };
                    auto score = [&](int t, int j) {             // S_t = Q_t K_j^T
#pragma unroll
                        for (int c = 0; c < 3; ++c) {
                            landed(j, c);
                            if (!ok) return;
                            const uint32_t qa = tc::smem_u32(sm.q[t][c]), ka = tc::smem_u32(sm.ring[unit(j, c)]);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_f16_ss(tmem + t * kN, tc::sdesc_sw128(qa + k * 32), tc::sdesc_sw128(ka + k * 32),
                                               idesc_s, (c | k) != 0);
                        }
                        tc::mma_commit(&sm.s_full[t]);
                    };
                    auto weigh = [&](int t, int j, int done) {   // O_t += P_t V_j
#pragma unroll
                        for (int hf = 0; hf < 2; ++hf) {
                            landed(j, 3 + hf);
                            ok = ok && tc::mbar_wait(&sm.p_full[t][hf], (done + j) & 1, abort_flag);
                            if (!ok) return;
                            tc::tc_fence_after();
                            const uint32_t va = tc::smem_u32(sm.ring[unit(j, 3 + hf)]);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tc::mma_f16_ts(tmem + 256 + t * kDv, tmem + t * kN + hf * 32 + k * 8,
                                               tc::sdesc_sw128_lbo(va + k * 2048, 8192, 1024), idesc_o, (j | hf | k) != 0);
                        }
                        if (j == p.n[t] - 1) tc::mma_commit(&sm.o_done[t]);
                    };
                    auto release = [&](int j, int c0, int c1) {
                        for (int c = c0; c < c1; ++c) tc::mma_commit(&sm.empty[unit(j, c)]);
                    };
                    any = true;
                    ok = tc::mbar_wait(&sm.q_full, items & 1, abort_flag);
                    // One step ahead of the products: j = -1 issues the first scores only.
#pragma unroll 1
                    for (int j = -1; j < n_tiles && ok; ++j) {
                        if (j >= 0 && j < p.n[0]) weigh(0, j, done0);
                        if (ok && j + 1 < p.n[0]) score(0, j + 1);
                        if (ok && j >= 0 && j < p.n[1]) weigh(1, j, done1);
                        if (ok && j >= 0) release(j, 3, 5);
                        if (ok && j + 1 < p.n[1]) score(1, j + 1);
                        if (ok && j + 1 < n_tiles) release(j + 1, 0, 3);
                        if (ok && j + 2 == n_tiles) tc::mma_commit(&sm.q_free);    // the last scores are issued
                    }
                    ++items;
                    done0 += p.n[0];
                    done1 += p.n[1];
                    u0 += n_tiles * kPerTile;
                }
                ok = __all_sync(0xffffffffu, ok);
            }
            // Drain before TMEM is freed: a commit completes after every MMA issued.
            if (leader && any) {
                volatile int drain = 0;
                if (!ok) *abort_flag = 1;
                tc::mma_commit(&sm.mma_done);
                tc::mbar_wait(&sm.mma_done, 0, &drain);
            }
        } else {
            // ---------------- rows of a partial last tile behind the sequence: zero
            int u0 = 0, partials = 0;
            bool ok = true;
            while (ok && next_item(p)) {
                const int n_tiles = tiles(p);
                if (n_tiles > 0 && is_partial(p)) {
                    const int j = n_tiles - 1, from = p.nk - j * kN;
                    for (int hf = 0; hf < 2; ++hf) {
                        ok = __all_sync(0xffffffffu, tc::mbar_wait(&sm.v_last[hf], partials & 1, abort_flag));
                        if (!ok) break;
                        const int s = (u0 + j * kPerTile + 3 + hf) % kUnits, r0 = max(0, from - hf * 64);
                        for (int i = lane; i < (64 - min(64, r0)) * 16; i += 32)
                            *reinterpret_cast<uint4*>(sm.ring[s] + ((i >> 3) & 1) * 8192 + (r0 + (i >> 4)) * 128 + (i & 7) * 16) =
                                make_uint4(0, 0, 0, 0);
                        tc::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) tc::mbar_arrive(&sm.full[s]);
                    }
                    ++partials;
                }
                u0 += n_tiles * kPerTile;
            }
        }
    } else {
        reg_inc<kSoftmaxRegs>();
        // ---------------- softmax and epilogue: thread = query row
        const int t = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + t * kN + lane_off, o_col = tmem + 256 + t * kDv + lane_off;
        const float sc = a.sm_scale_log2;
        int done = 0, outs = 0;                      // score tiles, and items with keys, of this query tile so far
        bool alive = true;
        Item p;
        while (alive && next_item(p)) {
            const int n = p.n[t], i = p.i0 + t * kM + row;
            const bool live = t * kM + row < p.rows;
            const int lim = a.causal ? min(p.nk, max(0, i + 1 + p.shift)) : p.nk;     // keys this row sees
            float m = kNegInf, l = 0.f;              // reference maximum (log2 units) and sum
            for (int j = 0; j < n; ++j, ++done) {
                if (!__all_sync(0xffffffffu, tc::mbar_wait(&sm.s_full[t], done & 1, abort_flag))) { alive = false; break; }
                tc::tc_fence_after();
                uint32_t w[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tc::tmem_ld32(s_col + c * 32, w[c]);
                tc::tmem_wait_ld();
                const int left = lim - j * kN;           // keys of this tile that the row sees
                if (__any_sync(0xffffffffu, left < kN)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (c * 32 + e >= left) w[c][e] = 0xff800000u;
                }
                float mx[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mx[c] = __uint_as_float(w[c][0]);
#pragma unroll
                    for (int e = 1; e < 32; ++e) mx[c] = fmaxf(mx[c], __uint_as_float(w[c][e]));
                }
                const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
                // The reference rises only when the tile exceeds it by more than 2^8; weights stay below 2^8.
                float alpha = 1.f;
                bool rescale = false;
                if (mt > m + 8.f) {
                    if (m != kNegInf) { alpha = ex2(m - mt); rescale = true; }
                    l *= alpha;
                    m = mt;
                }
                if (__any_sync(0xffffffffu, rescale)) {  // O holds P V of the tiles before: their MMAs precede this S
#pragma unroll 1
                    for (int c = 0; c < kDv / 32; ++c) {
                        uint32_t ov[32];
                        tc::tmem_ld32(o_col + c * 32, ov);
                        tc::tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        tc::tmem_st32(o_col + c * 32, ov);
                    }
                }
                const float mref = m == kNegInf ? 0.f : m;
                const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-mref, -mref);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    uint32_t pw[32];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const uint32_t* s2 = &w[2 * hf + c][e];
                            float2 x = ffma2(make_float2(__uint_as_float(s2[0]), __uint_as_float(s2[1])), sc2, m2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            sum[(e >> 1) & 1] = ffma2(x, make_float2(1.f, 1.f), sum[(e >> 1) & 1]);
                            pw[c * 16 + e / 2] = pack_bf16x2(x.x, x.y);
                        }
                    tc::tmem_st32(s_col + hf * 32, pw);
                    tc::tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&sm.p_full[t][hf]);
                }
                l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
            }
            if (n > 0 && alive) {
                alive = __all_sync(0xffffffffu, tc::mbar_wait(&sm.o_done[t], outs & 1, abort_flag));
                ++outs;
            }
            tc::tc_fence_after();
            // Zero for a row that sees no key; with keys every finite row has a positive sum, and a query that is not finite
            // gives NaN.
            const bool none = lim <= 0;
            if (!none && !(l > 0.f)) l = __int_as_float(0x7fc00000);
            const float inv = 1.f / l;
            const size_t orow = (size_t)(p.q0 + t * kM + row) * a.H + p.h;
#pragma unroll 1
            for (int c = 0; c < kDv / 32; ++c) {
                uint32_t ov[32];
                if (n > 0 && alive) {
                    tc::tmem_ld32(o_col + c * 32, ov);
                    tc::tmem_wait_ld();
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) ov[e] = 0u;
                }
                __syncwarp();
                if (live) {
                    float f[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) f[e] = none ? 0.f : __uint_as_float(ov[e]) * inv;
                    if (a.o_f32) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.o) + orow * kDv + c * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.o) + orow * kDv + c * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(pack_bf16x2(f[8 * e], f[8 * e + 1]), pack_bf16x2(f[8 * e + 2], f[8 * e + 3]),
                                                pack_bf16x2(f[8 * e + 4], f[8 * e + 5]), pack_bf16x2(f[8 * e + 6], f[8 * e + 7]));
                    }
                }
                __syncwarp();
            }
            if (live && a.lse) a.lse[orow] = none ? kNegInf : (m + log2f(l)) * 0.69314718055994530942f;
            tc::tc_fence_before();                   // the next item's first product overwrites O after this warp's p_full
        }
    }
    __syncwarp();
    tc::tc_fence_before();
    __syncthreads();
    if (sm.abort && threadIdx.x == 0) report(a.status, LSA_ERR_TIMEOUT);
    if (warp == 8) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem, 512);
    }
}

// [tokens][heads][dims] BF16 as a 3-D tensor, box 64 dims x 1 head x `rows` tokens, 128-byte swizzle.  A dimension of
// one element, or a broadcast one (stride 0, taken at coordinate 0), has extent 1 and any valid stride.
bool make_map(CUtensorMap* m, const uint16_t* base, int dims, int heads, int64_t head_stride, int tokens,
              int64_t tok_stride, int rows) {
    const bool one = heads == 1 || head_stride == 0;
    const cuuint64_t d[3] = {(cuuint64_t)dims, (cuuint64_t)(one ? 1 : heads), (cuuint64_t)tokens};
    const cuuint64_t s[2] = {(cuuint64_t)(one ? dims : head_stride) * 2, (cuuint64_t)(tok_stride ? tok_stride : dims) * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows};
    const cuuint32_t e[3] = {1, 1, 1};
    return tc::encode_tiled()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(base), d, s, box, e,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_latent_expanded(const ExpandedArgs& a, cudaStream_t st) {
    if (tc::encode_tiled() == nullptr) return cudaErrorNotSupported;
    CUtensorMap qm, km, rm, vm;
    memset(&km, 0, sizeof(km));
    memset(&rm, 0, sizeof(rm));
    memset(&vm, 0, sizeof(vm));
    if (!make_map(&qm, a.q, kD, a.H, a.qh, a.T, a.qt, kM)) return cudaErrorInvalidValue;
    if (a.S > 0) {
        const cuuint64_t d[2] = {kDr, (cuuint64_t)a.S}, s[1] = {(cuuint64_t)(a.rt ? a.rt : kDr) * 2};
        const cuuint32_t box[2] = {64, kN}, e[2] = {1, 1};
        if (!make_map(&km, a.kn, kDn, a.H, a.kh, a.S, a.kt, kN) || !make_map(&vm, a.v, kDv, a.H, a.vh, a.S, a.vt, 64) ||
            tc::encode_tiled()(&rm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(a.kr), d, s, box, e,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    }
    const size_t smem = sizeof(Smem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(latent_expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    latent_expanded_kernel<<<dim3((a.max_q + 2 * kM - 1) / (2 * kM), a.H, a.B), kThreads, smem, st>>>(qm, km, rm, vm, a);
    return cudaGetLastError();
}

}  // namespace lsa
