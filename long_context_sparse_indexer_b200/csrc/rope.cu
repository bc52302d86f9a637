// Rotary positions: frequencies (host) and the rotation of query heads.
//
// (u, w) -> mscale (u cos a - w sin a, w cos a + u sin a) per pair of dimensions, a = position * frequency;
// the gradient is the rotation by -a.  One read and one write of every element, 3 multiply-adds a pair:
// bound by memory (8192 tokens x 64 heads of 128 in 54 us, 5.0 TB/s, 76% of the copy rate), so the split keeps loads in flight and indexing
// cheap.  A block takes a run of (token, head) rows,
// first the dimensions that are only copied, then the rotary ones, so that no warp mixes the two (mixed, every warp
// paid for the rotation: 104 us instead of 54 for 8192 tokens x 64 heads of 128, half rotated).  A thread keeps one
// item of the row -- 16 bytes to copy, or the 16 (interleaved) or 2 x 16 bytes (half layout) of whole pairs -- and walks
// down the rows, several of them loaded before any is used.  The sines and cosines (one per token and pair, whatever
// the number of heads) are made once in shared memory, before the copies, and stay in registers from one head to the
// next.
#include <cmath>

#include "kernels.cuh"
#include "rope.cuh"

namespace lsa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kCopyBatch = 4, kRotBatch = 2;     // rows in flight per thread
constexpr int kMaxTokens = 16;                   // tokens of a block (their table in shared memory)

struct RopeArgs {
    RopeTable r;
    const int32_t* pos;
    const void* x;
    void* y;
    int64_t xt, xh, yt, yh;                      // strides, elements
    int T, H, D, off;
    int tokens, heads;                           // tokens and heads of a block
    int copy;                                    // 0: y is x, the other dimensions are in place
    float sign;                                  // -1: backward
};

__device__ __forceinline__ float to_f(uint16_t v) { return bf16_bits_to_float(v); }
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ void from_f(uint16_t& d, float v) { d = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ void from_f(float& d, float v) { d = v; }

// E elements of type T moved as one access: 16 bytes, or single elements for rows aligned to no more.
template <typename T, int E>
struct alignas(sizeof(T) * E) Pack { T v[E]; };

// Rotary items of a row.  Scalars (E = 1): a pair per item.
template <int E, bool INTER>
__host__ __device__ inline int rot_items(int rd) { return INTER && E > 1 ? rd / E : rd / 2 / E; }

// Walks the rows of a block (nh heads of each token) with `n` items each: item(c) is called for each item column of this
// thread, then rows(tokens, heads, count) for BATCH rows at a time, count of them live.
template <int BATCH, typename Item, typename Rows>
__device__ __forceinline__ void walk(int n, int rows, int nh, Item item, Rows body) {
    const int cols = min(n, kRopeThreads), step = kRopeThreads / cols;             // items and rows of a pass
    const int r0 = threadIdx.x / cols, dt = step / nh, dh = step - dt * nh;
    if (r0 >= step) return;
    for (int c = threadIdx.x - r0 * cols; c < n; c += cols) {
        item(c);
        int t = r0 / nh, h = r0 - t * nh;
        for (int row = r0; row < rows; row += step * BATCH) {
            int tt[BATCH], hh[BATCH];
#pragma unroll
            for (int u = 0; u < BATCH; ++u) {
                tt[u] = t;
                hh[u] = h;
                t += dt;
                h += dh;
                if (h >= nh) { h -= nh; ++t; }
            }
            body(tt, hh, (rows - row + step - 1) / step);
        }
    }
}

template <typename T, int E, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
    extern __shared__ float2 cs[];               // [tokens][rd / 2]
    using P = Pack<T, E>;
    constexpr bool kIn = INTER && E > 1;         // both of a pair in the same pack
    constexpr int kPairs = kIn ? E / 2 : E;      // pairs of a rotary item
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
    const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.H - h0);
    const int rd = p.r.rot_dim, half = rd / 2;
    const T* x = static_cast<const T*>(p.x) + t0 * p.xt + h0 * p.xh;
    T* y = static_cast<T*>(p.y) + t0 * p.yt + h0 * p.yh;
    for (int k = threadIdx.x; k < nt * half; k += kRopeThreads) {
        const int t = k / half, i = k - t * half;
        float2 v = rope_cs(p.pos[t0 + t], p.r.rev_freq[i], p.r.mscale);
        v.y *= p.sign;
        cs[k] = v;
    }
    if (p.copy && p.D > rd) {
        int d = 0;
        walk<kCopyBatch>((p.D - rd) / E, nt * nh, nh, [&](int c) { d = c * E < p.off ? c * E : c * E + rd; },
            [&](const int* tt, const int* hh, int n) {
                P a[kCopyBatch];
#pragma unroll
                for (int u = 0; u < kCopyBatch; ++u)
                    if (u < n) a[u] = *reinterpret_cast<const P*>(x + tt[u] * p.xt + hh[u] * p.xh + d);
#pragma unroll
                for (int u = 0; u < kCopyBatch; ++u)
                    if (u < n) *reinterpret_cast<P*>(y + tt[u] * p.yt + hh[u] * p.yh + d) = a[u];
            });
    }
    __syncthreads();
    const int d2 = INTER ? 1 : half;             // where an item's partners are (interleaved packs hold both)
    int d = 0, pair = 0, have = -1;
    float2 c[kPairs];
    walk<kRotBatch>(rot_items<E, INTER>(rd), nt * nh, nh,
        [&](int it) {
            pair = it * kPairs;
            d = p.off + (INTER ? 2 * pair : pair);
            have = -1;
        },
        [&](const int* tt, const int* hh, int n) {
            P a[kRotBatch], b[kRotBatch];
#pragma unroll
            for (int u = 0; u < kRotBatch; ++u)
                if (u < n) {
                    const T* s = x + tt[u] * p.xt + hh[u] * p.xh + d;
                    a[u] = *reinterpret_cast<const P*>(s);
                    if (!kIn) b[u] = *reinterpret_cast<const P*>(s + d2);
                }
#pragma unroll
            for (int u = 0; u < kRotBatch; ++u)
                if (u < n) {
                    if (tt[u] != have) {
                        have = tt[u];
#pragma unroll
                        for (int e = 0; e < kPairs; ++e) c[e] = cs[have * half + pair + e];
                    }
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        T& fu = a[u].v[kIn ? 2 * e : e];
                        T& gu = kIn ? a[u].v[2 * e + (kIn ? 1 : 0)] : b[u].v[e];
                        const float f = to_f(fu), g = to_f(gu);
                        from_f(fu, f * c[e].x - g * c[e].y);
                        from_f(gu, g * c[e].x + f * c[e].y);
                    }
                    T* o = y + tt[u] * p.yt + hh[u] * p.yh + d;
                    *reinterpret_cast<P*>(o) = a[u];
                    if (!kIn) *reinterpret_cast<P*>(o + d2) = b[u];
                }
        });
}

template <typename T, int E, bool INTER>
cudaError_t launch_rope_i(RopeArgs& p, cudaStream_t st) {
    // Rows per block: about 16 items a thread, so that a block's start (its table) is a small part of it; fewer when the
    // grid would not cover the 148 SMs a few times.
    const int n_row = rot_items<E, INTER>(p.r.rot_dim) + (p.copy ? (p.D - p.r.rot_dim) / E : 0);
    const int64_t want = 16 * kRopeThreads;
    p.heads = p.H;
    p.tokens = 1;
    if ((int64_t)p.H * n_row > want) p.heads = (int)((want + n_row - 1) / n_row);
    else while (p.tokens < kMaxTokens && (int64_t)2 * p.tokens * p.H * n_row <= want) p.tokens *= 2;
    auto blocks = [&] { return (int64_t)((p.T + p.tokens - 1) / p.tokens) * ((p.H + p.heads - 1) / p.heads); };
    while (blocks() < 4 * 148 && (int64_t)p.tokens * p.heads * n_row > kRopeThreads) {
        if (p.tokens > 1) p.tokens /= 2;
        else if (p.heads > 1) p.heads = (p.heads + 1) / 2;
        else break;
    }
    dim3 grid((p.T + p.tokens - 1) / p.tokens, (p.H + p.heads - 1) / p.heads);
    rope_kernel<T, E, INTER><<<grid, kRopeThreads, (size_t)p.tokens * p.r.rot_dim / 2 * sizeof(float2), st>>>(p);
    return cudaGetLastError();
}

template <typename T, int E>
cudaError_t launch_rope_t(RopeArgs& p, cudaStream_t st) {
    return p.r.interleaved ? launch_rope_i<T, E, true>(p, st) : launch_rope_i<T, E, false>(p, st);
}

}  // namespace

RopeTable rope_table(const lsa_rope* r) {
    RopeTable t{};
    t.rot_dim = r->rot_dim;
    t.interleaved = r->interleaved != 0;
    t.mscale = r->mscale;
    for (int i = 0; i < r->rot_dim / 2; ++i) t.rev_freq[i] = r->inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
    return t;
}

cudaError_t launch_rope(const lsa_rope* r, int T, int H, int D, int off, const int32_t* pos, bool bf16, const void* x,
                        int64_t xt, int64_t xh, void* y, int64_t yt, int64_t yh, bool backward, cudaStream_t st) {
    RopeArgs p{};
    p.r = rope_table(r);
    p.pos = pos; p.x = x; p.y = y; p.xt = xt; p.xh = xh; p.yt = yt; p.yh = yh;
    p.T = T; p.H = H; p.D = D; p.off = off; p.copy = x != y; p.sign = backward ? -1.f : 1.f;
    // 16-byte accesses need every row, every run and the pairs in whole packs.
    const int E = bf16 ? 8 : 4;
    auto ok = [&](int64_t v) { return v % E == 0; };
    const bool vec = ok(xt) && ok(xh) && ok(yt) && ok(yh) && ok(off) && ok(D) && ok(r->interleaved ? r->rot_dim : r->rot_dim / 2) &&
                     ((uintptr_t)x & 15) == 0 && ((uintptr_t)y & 15) == 0;
    if (bf16) return vec ? launch_rope_t<uint16_t, 8>(p, st) : launch_rope_t<uint16_t, 1>(p, st);
    return vec ? launch_rope_t<float, 4>(p, st) : launch_rope_t<float, 1>(p, st);
}

// Frequencies of an lsa_rope.  YaRN: pair(turns) is the pair that makes `turns` turns over the original length;
// pairs up to floor(pair(beta_fast)) keep their frequency, those from ceil(pair(beta_slow)) on are divided by
// the factor, linearly between.
lsa_status rope_init(lsa_rope* r, int rd, int interleaved, double theta, int scaling, double factor, int64_t orig_len,
                     double beta_fast, double beta_slow, double mscale) {
    if (!r || rd < 2 || rd > LSA_ROPE_MAX_DIM || rd % 2 || (interleaved != 0 && interleaved != 1)) return LSA_ERR_INVALID_ARG;
    if (!(theta > 1.0) || !std::isfinite(theta) || !std::isfinite(mscale)) return LSA_ERR_INVALID_ARG;
    if (scaling < LSA_ROPE_PLAIN || scaling > LSA_ROPE_YARN) return LSA_ERR_UNSUPPORTED;
    if (scaling != LSA_ROPE_PLAIN && (!(factor > 0.0) || !std::isfinite(factor))) return LSA_ERR_INVALID_ARG;
    if (scaling == LSA_ROPE_NTK && rd == 2) return LSA_ERR_INVALID_ARG;
    if (scaling == LSA_ROPE_YARN && (orig_len < 1 || !(beta_fast > 0.0) || !(beta_slow > 0.0) ||
                                     !std::isfinite(beta_fast) || !std::isfinite(beta_slow)))
        return LSA_ERR_INVALID_ARG;
    if (scaling == LSA_ROPE_NTK) theta *= std::pow(factor, rd / (rd - 2.0));
    if (!(theta > 1.0) || !std::isfinite(theta)) return LSA_ERR_INVALID_ARG;
    double lo = 0.0, hi = 0.0;
    if (scaling == LSA_ROPE_YARN) {
        auto pair = [&](double turns) { return rd * std::log(orig_len / (turns * 6.283185307179586477)) / (2.0 * std::log(theta)); };
        lo = std::fmax(0.0, std::floor(pair(beta_fast)));
        hi = std::fmin(rd - 1.0, std::ceil(pair(beta_slow)));
    }
    *r = lsa_rope{};
    r->rot_dim = rd;
    r->interleaved = interleaved;
    r->mscale = (float)mscale;
    for (int i = 0; i < rd / 2; ++i) {
        double f = std::pow(theta, -2.0 * i / rd);
        if (scaling == LSA_ROPE_LINEAR) f /= factor;
        if (scaling == LSA_ROPE_YARN) {
            const double ramp = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
            f = f / factor * ramp + f * (1.0 - ramp);
        }
        r->inv_freq[i] = f;
    }
    return LSA_OK;
}

}  // namespace lsa
