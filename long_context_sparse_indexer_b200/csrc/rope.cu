// Rotary positions: frequencies (host) and the rotation of query heads.
//
// (u, w) -> mscale (u cos a - w sin a, w cos a + u sin a) per pair of dimensions, a = position * frequency;
// the gradient is the rotation by -a.  One read and one write of every element, 3 multiply-adds a pair:
// bound by memory, so the split serves loads in flight.  A block takes one run of (token, head) rows of a
// few tokens; its sines and cosines (one per token and pair, whatever the number of heads) are made once in
// shared memory while the first loads travel.  A work item is 16 bytes of dimensions that are only copied,
// or the 16 (interleaved) or 2 x 16 bytes (half layout) of whole pairs; kBatch items are loaded per thread
// before any is used.
#include <cmath>

#include "kernels.cuh"
#include "rope.cuh"

namespace lsa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kBatch = 4;                        // items in flight per thread
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

// An item's loaded elements: `a` from dimension d0, and `b` its partners (rotary items, half layout: from d0 + rd / 2).
template <typename T, int E>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs p) {
    extern __shared__ float2 cs[];               // [tokens][rd / 2]
    using P = Pack<T, E>;
    const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
    const int h0 = blockIdx.y * p.heads, nh = min(p.heads, p.H - h0);
    const int rd = p.r.rot_dim, half = rd / 2;
    const bool inter = p.r.interleaved;
    // A row's items: the rotary ones first, then the copied runs before and behind the rotary dimensions.
    // Scalars (E = 1): a pair per rotary item, one element per copied item.
    const int n_rot = inter ? (E > 1 ? rd / E : half) : half / E;
    const int n_row = n_rot + (p.copy ? (p.D - rd) / E : 0);
    const int n = nt * nh * n_row;
    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    bool ready = false;
    for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < n; i0 += kRopeThreads * kBatch) {
        P a[kBatch], b[kBatch];
        int64_t ya[kBatch];
        int rot[kBatch];                         // table index of the item's first pair, or -1
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kRopeThreads;
            rot[u] = -2;
            if (i >= n) continue;
            const int row = i / n_row, it = i - row * n_row;
            const int tl = row / nh, h = h0 + row - tl * nh, t = t0 + tl;
            const int64_t xa = t * p.xt + h * p.xh;
            int d;
            if (it < n_rot) {
                const int pair = inter ? it * (E > 1 ? E / 2 : 1) : it * E;
                rot[u] = tl * half + pair;
                d = p.off + (inter ? 2 * pair : pair);
                if (!inter) b[u] = *reinterpret_cast<const P*>(x + xa + d + half);
                else if (E == 1) b[u] = *reinterpret_cast<const P*>(x + xa + d + 1);
            } else {
                rot[u] = -1;
                d = (it - n_rot) * E;
                if (d >= p.off) d += rd;
            }
            a[u] = *reinterpret_cast<const P*>(x + xa + d);
            ya[u] = t * p.yt + h * p.yh + d;
        }
        if (!ready) {                            // the table, once, under the first loads
            for (int k = threadIdx.x; k < nt * half; k += kRopeThreads) {
                const int tl = k / half, i = k - tl * half;
                float2 v = rope_cs(p.pos[t0 + tl], p.r.rev_freq[i], p.r.mscale);
                v.y *= p.sign;
                cs[k] = v;
            }
            __syncthreads();
            ready = true;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (rot[u] == -2) continue;
            if (rot[u] >= 0) {
                if (inter && E > 1) {
#pragma unroll
                    for (int e = 0; e + 1 < E; e += 2) {
                        const float2 c = cs[rot[u] + e / 2];
                        const float f = to_f(a[u].v[e]), g = to_f(a[u].v[e + 1]);
                        from_f(a[u].v[e], f * c.x - g * c.y);
                        from_f(a[u].v[e + 1], g * c.x + f * c.y);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        const float2 c = cs[rot[u] + e];
                        const float f = to_f(a[u].v[e]), g = to_f(b[u].v[e]);
                        from_f(a[u].v[e], f * c.x - g * c.y);
                        from_f(b[u].v[e], g * c.x + f * c.y);
                    }
                    *reinterpret_cast<P*>(y + ya[u] + (inter ? 1 : half)) = b[u];
                }
            }
            *reinterpret_cast<P*>(y + ya[u]) = a[u];
        }
    }
}

template <typename T, int E>
cudaError_t launch_rope_t(RopeArgs& p, cudaStream_t st) {
    // Tokens per block so that a block has about two rounds of items (32 KB), heads per block so that the
    // grid covers the GPU: few tokens split their heads, many tokens with few heads share a block.
    const int n_row = (p.r.interleaved ? (E > 1 ? p.r.rot_dim / E : p.r.rot_dim / 2) : p.r.rot_dim / 2 / E) +
                      (p.copy ? (p.D - p.r.rot_dim) / E : 0);
    const int want = 2 * kBatch * kRopeThreads;
    p.heads = p.H;
    p.tokens = 1;
    if ((int64_t)p.H * n_row > want) p.heads = (want + n_row - 1) / n_row;
    else while (p.tokens < kMaxTokens && (int64_t)2 * p.tokens * p.H * n_row <= want) p.tokens *= 2;
    // Too few blocks for 148 SMs: smaller ones, down to one round of items each.
    auto blocks = [&] { return (int64_t)((p.T + p.tokens - 1) / p.tokens) * ((p.H + p.heads - 1) / p.heads); };
    while (blocks() < 2 * 148 && (int64_t)p.tokens * p.heads * n_row > kRopeThreads) {
        if (p.tokens > 1) p.tokens /= 2;
        else if (p.heads > 1) p.heads = (p.heads + 1) / 2;
        else break;
    }
    dim3 grid((p.T + p.tokens - 1) / p.tokens, (p.H + p.heads - 1) / p.heads);
    rope_kernel<T, E><<<grid, kRopeThreads, (size_t)p.tokens * p.r.rot_dim / 2 * sizeof(float2), st>>>(p);
    return cudaGetLastError();
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
