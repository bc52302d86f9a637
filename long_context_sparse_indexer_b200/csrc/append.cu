// Cache append: one new row per token, normalised, rotated, rounded and stored at its position.
//
// h = norm(x[0:n]) (RMS or layer norm), then the rotation of the rotary part, then BF16 or e4m3 codes with
// scale = max|row| / 448.  Every element is read once and written once with a few operations in between:
// bound by memory for many rows and by the latency of one row for few.  So a warp takes a row and keeps it
// in registers (8 elements per lane and slot, up to 4 slots): all its loads travel together, the two or
// three reductions are shuffles, and the only shared memory is the warp's rotary part and its sines and
// cosines, which lanes exchange because a pair's halves sit in different lanes in the half layout.
#include <cuda_fp8.h>

#include "kernels.cuh"
#include "rope.cuh"

namespace lsa {

namespace {

constexpr int kMaxSlots = 4;                     // 8-element chunks per lane: rows of up to 1024 elements

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

struct AppendKernelArgs {
    AppendArgs a;
    RopeTable r;
};

template <int SLOTS, bool FP8>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendKernelArgs k) {
    extern __shared__ float smem[];              // per warp: rot_dim rotary elements, rot_dim / 2 (cos, sin)
    const AppendArgs& p = k.a;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t = blockIdx.x * warps + warp;
    if (t >= p.T) return;                        // whole warps; no block barrier below
    const int pos = p.q_pos[t];
    if (pos < 0) return;
    const int b = p.q_seq[t];
    bool ok = b >= 0 && b < p.B && pos < p.seq_len[b] && p.seq_len[b] <= p.L_alloc;
    int64_t lead = b, row = pos;
    if (ok && p.table) {
        const int pg = pos / p.page_size;
        row = pos - pg * p.page_size;
        lead = p.table[b * p.table_ld + pg];
        ok = lead >= 0 && lead < p.n_pages;
    }
    if (!ok) {
        if (lane == 0) report(p.status, LSA_ERR_DEVICE_DATA);
        return;
    }
    const int chunks = p.dim / 8, rd = p.rope ? k.r.rot_dim : 0;
    const uint16_t* x = p.x + (int64_t)t * p.ld_x;
    uint4 raw[SLOTS];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const int c = s * 32 + lane;
        raw[s] = c < chunks ? ldg_nc16(x + c * 8) : make_uint4(0, 0, 0, 0);
    }
    float* rot = smem + (size_t)warp * 2 * rd;
    float2* cs = reinterpret_cast<float2*>(rot + rd);
    for (int i = lane; i < rd / 2; i += 32) cs[i] = rope_cs(pos, k.r.rev_freq[i], k.r.mscale);
    float v[SLOTS][8];
#pragma unroll
    for (int s = 0; s < SLOTS; ++s) {
        const uint32_t w[4] = {raw[s].x, raw[s].y, raw[s].z, raw[s].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[s][2 * e] = __uint_as_float(w[e] << 16);
            v[s][2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
    }
    if (p.norm != LSA_NORM_NONE) {
        const int nc = p.norm_dim / 8;
        const float inv_n = 1.f / (float)p.norm_dim;
        float mean = 0.f, sum = 0.f;
        if (p.norm == LSA_NORM_LAYER) {
#pragma unroll
            for (int s = 0; s < SLOTS; ++s)
                if (s * 32 + lane < nc)
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum += v[s][e];
            mean = warp_sum(sum) * inv_n;
        }
        float sq = 0.f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
            if (s * 32 + lane < nc)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[s][e] -= mean;
                    sq = fmaf(v[s][e], v[s][e], sq);
                }
        const float rs = 1.f / sqrtf(warp_sum(sq) * inv_n + p.eps);
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int c = s * 32 + lane;
            if (c >= nc) continue;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[s][e] *= rs;
            if (p.gamma)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[s][e] *= __ldg(p.gamma + c * 8 + e);
            if (p.beta)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[s][e] += __ldg(p.beta + c * 8 + e);
        }
    }
    if (rd) {
        // The rotary part through shared memory: any offset, either layout.
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = (s * 32 + lane) * 8 + e - p.rope_off;
                if (d >= 0 && d < rd) rot[d] = v[s][e];
            }
        __syncwarp();
        const int half = rd / 2;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = (s * 32 + lane) * 8 + e - p.rope_off;
                if (d < 0 || d >= rd) continue;
                const bool second = k.r.interleaved ? d & 1 : d >= half;
                const int pair = k.r.interleaved ? d >> 1 : (second ? d - half : d);
                const float o = rot[k.r.interleaved ? d ^ 1 : (second ? d - half : d + half)];
                const float2 c = cs[pair];
                v[s][e] = second ? v[s][e] * c.x + o * c.y : v[s][e] * c.x - o * c.y;
            }
    }
    float amax = 0.f;
    bool bad = false;
#pragma unroll
    for (int s = 0; s < SLOTS; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            amax = fmaxf(amax, fabsf(v[s][e]));
            bad |= !(fabsf(v[s][e]) < __int_as_float(0x7f800000));
        }
    bad = __any_sync(0xffffffffu, bad);
    if (bad && lane == 0) report(p.status, LSA_ERR_DEVICE_DATA);
    uint8_t* dst = p.data + lead * p.seq_b + row * p.tok_b;
    if constexpr (FP8) {
        amax = warp_max(amax);
        const float inv = amax > 0.f ? 448.f / amax : 1.f;
        if (lane == 0) p.scale[lead * p.scale_seq + row] = bad || !(amax > 0.f) ? 1.f : amax / 448.f;
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int c = s * 32 + lane;
            if (c >= chunks) continue;
            uint32_t w[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float* f = v[s] + 4 * h;
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0] * inv, f[1] * inv), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2] * inv, f[3] * inv), __NV_SATFINITE, __NV_E4M3);
                w[h] = bad ? 0x7f7f7f7fu : lo | hi << 16;
            }
            *reinterpret_cast<uint2*>(dst + c * 8) = make_uint2(w[0], w[1]);
        }
    } else {
#pragma unroll
        for (int s = 0; s < SLOTS; ++s) {
            const int c = s * 32 + lane;
            if (c >= chunks) continue;
            *reinterpret_cast<uint4*>(dst + c * 16) =
                make_uint4(pack_bf16x2(v[s][0], v[s][1]), pack_bf16x2(v[s][2], v[s][3]),
                           pack_bf16x2(v[s][4], v[s][5]), pack_bf16x2(v[s][6], v[s][7]));
        }
    }
}

template <int SLOTS>
cudaError_t launch_append_t(const AppendKernelArgs& k, cudaStream_t st) {
    // Few rows: a block per row, so that they spread over the SMs; many: 8 warps a block.
    const int warps = k.a.T <= 2 * 148 ? 1 : 8;
    const size_t smem = (size_t)warps * 2 * (k.a.rope ? k.r.rot_dim : 0) * sizeof(float);
    const int grid = (k.a.T + warps - 1) / warps;
    if (k.a.scale) append_kernel<SLOTS, true><<<grid, warps * 32, smem, st>>>(k);
    else append_kernel<SLOTS, false><<<grid, warps * 32, smem, st>>>(k);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(const AppendArgs& a, const lsa_rope* rope, cudaStream_t st) {
    AppendKernelArgs k{};
    k.a = a;
    k.a.rope = rope != nullptr;
    if (rope) k.r = rope_table(rope);
    const int slots = (a.dim / 8 + 31) / 32;
    if (slots <= 1) return launch_append_t<1>(k, st);
    if (slots <= 3) return launch_append_t<3>(k, st);
    return launch_append_t<kMaxSlots>(k, st);
}

}  // namespace lsa
