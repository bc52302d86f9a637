// Cache append: one new row per token, normalised, rotated, rounded and stored at its position.
//
// h = norm(x[0:n]) (RMS or layer norm), then the rotation of the rotary part, then BF16 or e4m3 codes with
// scale = max|row| / 448.  Every element is read once and written once with a few operations in between:
// bound for many rows by the latency of the chain load, reductions, exchange, store with one row ahead (instructions fill
// about 40% of the issue slots), for few by that of one row (on the device, inputs not in L2: 32,764 latent rows to BF16
// pages 29 us, 2.6 TB/s, to FP8 39; as many 128-element keys to FP8 17.5; a decode step's 32 rows 4.2).  LANES lanes
// (32, 16 or 8, the fewest that hold a row in up to four 16-byte chunks each) take a row and keep it in registers, so
// that its loads travel together and the reductions are shuffles.  A warp takes several rows one after another: the
// loads that find their places depend on one another (position and sequence, then length and page), so lanes find
// them for all its rows at once, and a row's elements are loaded while the one before is in work.  The only shared
// memory is the rotary part and its sines and cosines, which lanes exchange because a pair's halves sit in different
// lanes in the half layout.
#include <cuda_fp8.h>

#include "kernels.cuh"
#include "rope.cuh"

namespace lsa {

namespace {

constexpr int kMaxSlots = 4;                     // 8-element chunks per lane: rows of up to 1024 elements

template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct AppendKernelArgs {
    AppendArgs a;
    RopeTable r;
};

// Eight floats of a vector, read through L1; `whole`: it is 16-byte aligned.
__device__ __forceinline__ void load8(const float* p, bool whole, float2 (&v)[4]) {
    if (whole) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
        v[0] = make_float2(a.x, a.y); v[1] = make_float2(a.z, a.w);
        v[2] = make_float2(b.x, b.y); v[3] = make_float2(b.z, b.w);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = make_float2(__ldg(p + 2 * e), __ldg(p + 2 * e + 1));
    }
}

// Packed FP32 pairs, each rounded as the scalar operation.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{ .reg .b64 ra, rb, rd;\n"
        "mov.b64 ra, {%2, %3}; mov.b64 rb, {%4, %5};\n"
        "mul.rn.f32x2 rd, ra, rb;\n"
        "mov.b64 {%0, %1}, rd; }"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// rope_cs with the hardware's sine and cosine: absolute error below 2^-20 on a reduced angle, far inside the rounding
// of what is stored (2^-9 at best), for a third of the instructions.
__device__ __forceinline__ float2 rope_cs_fast(int pos, double rev_freq, float mscale) {
    const double turns = (double)pos * rev_freq;
    float s, c;
    __sincosf((float)(turns - rint(turns)) * 6.28318530717958647692f, &s, &c);
    return make_float2(c * mscale, s * mscale);
}

template <int LANES, int SLOTS, bool FP8>
__global__ void __launch_bounds__(256, SLOTS == 1 ? 4 : 3) append_kernel(const __grid_constant__ AppendKernelArgs k, int chunk) {
    extern __shared__ __align__(16) float smem[];                  // per warp: the frequencies; per row in work: rot_dim rotary elements,
                                                                   // rot_dim / 2 (cos, sin)
    constexpr int kSide = 32 / LANES;            // rows side by side in a warp
    const AppendArgs& p = k.a;
    const int wl = threadIdx.x & 31, lane = wl % LANES, side = wl / LANES;
    const int base = (blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) * chunk * kSide;        // the warp's first row
    if (base >= p.T) return;                     // whole warps; no block barrier below
    const int chunks = p.dim / 8, nc = p.norm == LSA_NORM_NONE ? 0 : p.norm_dim / 8, rd = p.rope ? k.r.rot_dim : 0;
    double* freq = reinterpret_cast<double*>(smem + (size_t)(threadIdx.x >> 5) * (1 + 2 * kSide) * rd);
    float* rot = reinterpret_cast<float*>(freq) + rd + side * 2 * rd;
    float2* cs = reinterpret_cast<float2*>(rot + rd);
    for (int j = wl; j < rd / 2; j += 32) freq[j] = k.r.rev_freq[j];               // lanes' indices differ: once from the parameters
    // Chunks of 8 dims wholly inside or outside the rotary part, and with it their partners: no element takes a test.
    const bool even = p.rope_off % 8 == 0 && rd % 16 == 0;
    const uint16_t* x = p.x + (int64_t)(base + side) * p.ld_x + lane * 8;          // this group's next row
    auto load = [&](int i, uint4 (&raw)[SLOTS]) {                  // its i-th
        const bool in = i < chunk && base + i * kSide + side < p.T;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            raw[s] = in && s * LANES + lane < chunks ? ldg_nc16(x + s * LANES * 8) : make_uint4(0, 0, 0, 0);
        x += kSide * p.ld_x;
    };
    uint4 next[SLOTS];
    load(0, next);
    if (nc)
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (s * LANES + lane < nc) {
                if (p.gamma) asm volatile("prefetch.global.L1 [%0];" :: "l"(p.gamma + (s * LANES + lane) * 8));
                if (p.beta) asm volatile("prefetch.global.L1 [%0];" :: "l"(p.beta + (s * LANES + lane) * 8));
            }
    // Lane l: where row base + l goes -- byte offset in the cache (-1: nowhere), index of its scale.
    int my_pos = -1;
    int64_t my_off = -1, my_sc = 0;
    if (wl < chunk * kSide && base + wl < p.T) {
        const int t = base + wl, b = p.q_seq[t];
        my_pos = p.q_pos[t];
        if (my_pos >= 0) {
            bool ok = b >= 0 && b < p.B;
            if (ok) {
                const int len = p.seq_len[b];
                int64_t lead = b, row = my_pos;
                ok = my_pos < len && len <= p.L_alloc;
                if (p.table && ok) {             // entries behind the last position are not read
                    const int pg = my_pos / p.page_size;
                    row = my_pos - pg * p.page_size;
                    lead = p.table[b * p.table_ld + pg];
                    ok = lead >= 0 && lead < p.n_pages;
                }
                if (ok) {
                    my_off = lead * p.seq_b + row * p.tok_b;
                    my_sc = lead * p.scale_seq + row;
                }
            }
            if (!ok) report(p.status, LSA_ERR_DEVICE_DATA);
        }
    }
    const float inv_n = 1.f / (float)max(1, p.norm_dim);
    const bool g_whole = ((uintptr_t)p.gamma & 15) == 0, b_whole = ((uintptr_t)p.beta & 15) == 0;
#pragma unroll 1
    for (int i = 0; i < chunk && base + i * kSide < p.T; ++i) {
        const int pos = __shfl_sync(0xffffffffu, my_pos, i * kSide + side);
        const int64_t off = __shfl_sync(0xffffffffu, my_off, i * kSide + side);
        const bool ok = off >= 0;
        float2 v[SLOTS][4];
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const uint32_t w[4] = {next[s].x, next[s].y, next[s].z, next[s].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) v[s][e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
        }
        load(i + 1, next);
        if (rd) {
            __syncwarp();                        // the row before has been read
            for (int j = lane; j < rd / 2; j += LANES) cs[j] = rope_cs_fast(pos, freq[j], k.r.mscale);
        }
        if (nc) {
            float2 sq = make_float2(0.f, 0.f);
            if (p.norm == LSA_NORM_LAYER) {
                float sum = 0.f;
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (s * LANES + lane < nc)
#pragma unroll
                        for (int e = 0; e < 4; ++e) sum += v[s][e].x + v[s][e].y;
                const float mean = lanes_sum<LANES>(sum) * inv_n;
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
                    if (s * LANES + lane < nc)
#pragma unroll
                        for (int e = 0; e < 4; ++e) { v[s][e].x -= mean; v[s][e].y -= mean; }
            }
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s * LANES + lane < nc)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sq = ffma2(v[s][e], v[s][e], sq);
            const float rs = rsqrtf(lanes_sum<LANES>(sq.x + sq.y) * inv_n + p.eps);
            const float2 rs2 = make_float2(rs, rs);
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s * LANES + lane < nc) {
                    float2 w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[s][e] = mul2(v[s][e], rs2);
                    if (p.gamma) {
                        load8(p.gamma + (s * LANES + lane) * 8, g_whole, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[s][e] = mul2(v[s][e], w[e]);
                    }
                    if (p.beta) {
                        load8(p.beta + (s * LANES + lane) * 8, b_whole, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) { v[s][e].x += w[e].x; v[s][e].y += w[e].y; }
                    }
                }
        }
        if (rd) {
            const int half = rd / 2;
            const bool inter = k.r.interleaved;
            if (even && inter) {                 // pairs side by side in the lane
                __syncwarp();
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const int d0 = (s * LANES + lane) * 8 - p.rope_off;
                    if (d0 < 0 || d0 >= rd) continue;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 c = cs[d0 / 2 + e];
                        const float f = v[s][e].x, g = v[s][e].y;
                        v[s][e] = make_float2(f * c.x - g * c.y, g * c.x + f * c.y);
                    }
                }
            } else if (even) {                   // a chunk's partners are a chunk, in another lane
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const int d0 = (s * LANES + lane) * 8 - p.rope_off;
                    if (d0 < 0 || d0 >= rd) continue;
                    float4* w = reinterpret_cast<float4*>(rot + d0);
                    w[0] = make_float4(v[s][0].x, v[s][0].y, v[s][1].x, v[s][1].y);
                    w[1] = make_float4(v[s][2].x, v[s][2].y, v[s][3].x, v[s][3].y);
                }
                __syncwarp();
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const int d0 = (s * LANES + lane) * 8 - p.rope_off;
                    if (d0 < 0 || d0 >= rd) continue;
                    const bool second = d0 >= half;
                    const int o0 = second ? d0 - half : d0 + half, pair = second ? o0 : d0;
                    const float4 x0 = reinterpret_cast<const float4*>(rot + o0)[0], x1 = reinterpret_cast<const float4*>(rot + o0)[1];
                    const float o[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
                    const float sign = second ? 1.f : -1.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 c0 = cs[pair + 2 * e], c1 = cs[pair + 2 * e + 1];
                        v[s][e] = make_float2(v[s][e].x * c0.x + sign * o[2 * e] * c0.y, v[s][e].y * c1.x + sign * o[2 * e + 1] * c1.y);
                    }
                }
            } else {                             // any offset, either layout
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const int d0 = (s * LANES + lane) * 8 - p.rope_off;
                    if (d0 <= -8 || d0 >= rd) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (d0 + e >= 0 && d0 + e < rd) rot[d0 + e] = e & 1 ? v[s][e / 2].y : v[s][e / 2].x;
                }
                __syncwarp();
#pragma unroll
                for (int s = 0; s < SLOTS; ++s) {
                    const int d0 = (s * LANES + lane) * 8 - p.rope_off;
                    if (d0 <= -8 || d0 >= rd) continue;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = d0 + e;
                        if (d < 0 || d >= rd) continue;
                        const bool second = inter ? d & 1 : d >= half;
                        const int pair = inter ? d >> 1 : (second ? d - half : d);
                        const float o = rot[inter ? d ^ 1 : (second ? d - half : d + half)];
                        const float2 c = cs[pair];
                        float& me = e & 1 ? v[s][e / 2].y : v[s][e / 2].x;
                        me = second ? me * c.x + o * c.y : me * c.x - o * c.y;
                    }
                }
            }
        }
        // The row as it stands here: left to itself the compiler carries every path of the rotation through to its own store, in
        // more registers than there are (rows to BF16 28 us so, 23 us pinned).
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) asm volatile("" : "+f"(v[s][e].x), "+f"(v[s][e].y));
        // 0 x element: zero, or NaN for an infinity or a NaN.
        float2 none = make_float2(0.f, 0.f);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int e = 0; e < 4; ++e) none = ffma2(v[s][e], make_float2(0.f, 0.f), none);
        bool bad = none.x != 0.f || none.y != 0.f;                 // of this lane's elements
        float amax = 0.f;
        if constexpr (FP8) {
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fmaxf(fabsf(v[s][e].x), fabsf(v[s][e].y)));
            if (bad) amax = __int_as_float(0x7f800000);            // through the reduction, to the row's other lanes
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            bad = amax == __int_as_float(0x7f800000);
        }
        if (ok && bad) report(p.status, LSA_ERR_DEVICE_DATA);
        uint8_t* dst = p.data + off;
        if constexpr (FP8) {
            // 448 / amax would overflow for the tiniest rows: those are taken 2^64 times.
            const float up = amax < 0x1p-60f ? 0x1p64f : 1.f;
            if (up != 1.f) {
#pragma unroll
                for (int s = 0; s < SLOTS; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[s][e] = mul2(v[s][e], make_float2(up, up));
            }
            const float inv = amax > 0.f ? 448.f / (amax * up) : 1.f;
            const int64_t sc = __shfl_sync(0xffffffffu, my_sc, i * kSide + side);
            if (ok && lane == 0) p.scale[sc] = bad || !(amax > 0.f) ? 1.f : amax / 448.f;
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int c = s * LANES + lane;
                if (!ok || c >= chunks) continue;
                uint32_t w[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t lo = __nv_cvt_float2_to_fp8x2(mul2(v[s][2 * h], make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
                    const uint32_t hi = __nv_cvt_float2_to_fp8x2(mul2(v[s][2 * h + 1], make_float2(inv, inv)), __NV_SATFINITE, __NV_E4M3);
                    w[h] = bad ? 0x7f7f7f7fu : lo | hi << 16;
                }
                *reinterpret_cast<uint2*>(dst + c * 8) = make_uint2(w[0], w[1]);
            }
        } else {
#pragma unroll
            for (int s = 0; s < SLOTS; ++s) {
                const int c = s * LANES + lane;
                if (!ok || c >= chunks) continue;
                *reinterpret_cast<uint4*>(dst + c * 16) =
                    make_uint4(pack_bf16x2(v[s][0].x, v[s][0].y), pack_bf16x2(v[s][1].x, v[s][1].y),
                               pack_bf16x2(v[s][2].x, v[s][2].y), pack_bf16x2(v[s][3].x, v[s][3].y));
            }
        }
    }
}

template <int LANES, int SLOTS>
cudaError_t launch_append_t(const AppendKernelArgs& k, cudaStream_t st) {
    // Few rows: one each, a warp per block, so that they spread over the SMs.  Many: as many in turn as make the grid one
    // wave of the blocks that fit the SMs (3 of 8 warps by registers, 4 for single-slot rows), at most the 32 rows whose
    // places a warp finds at once.
    const int side = 32 / LANES, resident = 148 * (SLOTS == 1 ? 4 : 3) * 8 * side;
    const bool few = k.a.T <= 8 * 148 * side;
    const int in_turn = (k.a.T + resident - 1) / resident;
    const int chunk = few ? 1 : (in_turn < LANES ? in_turn : LANES), warps = few ? 1 : 8, per_block = warps * chunk * side;
    const size_t smem = (size_t)warps * (1 + 2 * side) * (k.a.rope ? k.r.rot_dim : 0) * sizeof(float);
    const int grid = (k.a.T + per_block - 1) / per_block;
    if (k.a.scale) append_kernel<LANES, SLOTS, true><<<grid, warps * 32, smem, st>>>(k, chunk);
    else append_kernel<LANES, SLOTS, false><<<grid, warps * 32, smem, st>>>(k, chunk);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, const lsa_rope* rope, cudaStream_t st) {
    AppendKernelArgs k{};
    k.a = a;
    k.a.rope = rope != nullptr;
    if (rope) k.r = rope_table(rope);
    const int chunks = a.dim / 8;
    if (chunks <= 8) return launch_append_t<8, 1>(k, st);
    if (chunks <= 16) return launch_append_t<16, 1>(k, st);
    if (chunks <= 32) return launch_append_t<32, 1>(k, st);
    if (chunks <= 96) return launch_append_t<32, 3>(k, st);
    return launch_append_t<32, kMaxSlots>(k, st);
}

}  // namespace lsa
