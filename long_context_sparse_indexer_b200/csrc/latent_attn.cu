// Latent attention in the absorbed form over every visible cached row, paged or not.
//
//   z_s = sm_scale q . K_s (576), o = softmax(z) V (V = the first 512 elements of the same row).
//
// One pass with a running maximum and sum.  Block = (16 heads, token): the heads' queries in shared memory
// as FP32, rows brought in tiles of 16 and widened, each thread two of the 16 x 16 scores, then each thread
// 4 dimensions of all 16 heads' accumulators in registers.  CUDA cores, FP32 throughout: bound by them.
#include <cmath>

#include "kernels.cuh"

namespace lsa {

namespace {

constexpr int kThreads = 128, kHeads = 16, kRows = 16, kD = 576, kDv = 512;

struct Smem {
    float q[kHeads][kD + 1];
    float k[kRows][kD + 1];
    float p[kHeads][kRows];
    float m[kHeads], l[kHeads], alpha[kHeads];
    int64_t row[kRows];                          // byte offset of each row, or -1
    float scale[kRows];
};

__global__ void __launch_bounds__(kThreads) latent_attn_kernel(LatentArgs a) {
    extern __shared__ uint8_t raw[];
    Smem& s = *reinterpret_cast<Smem*>(raw);
    const int t = blockIdx.x, h0 = blockIdx.y * kHeads, tid = threadIdx.x;
    const int nh = min(kHeads, a.H - h0);
    const int g0 = t / a.q_group * a.q_group;
    const int b = a.q_seq[g0], pos = a.q_pos[t];
    int n = 0;
    if (pos >= 0) {
        const bool ok = b >= 0 && b < a.B && a.q_seq[t] == b && pos < a.seq_len[b] && a.seq_len[b] <= a.L_alloc;
        if (ok) n = pos + 1;
        else if (tid == 0) report(a.status, LSA_ERR_DEVICE_DATA);
    }
    for (int i = tid; i < kHeads * kD; i += kThreads) {
        const int h = i / kD, d = i % kD;
        s.q[h][d] = h < nh ? bf16_bits_to_float(a.q[((size_t)t * a.H + h0 + h) * kD + d]) * a.sm_scale_log2 : 0.f;
    }
    if (tid < kHeads) { s.m[tid] = kNegInf; s.l[tid] = 0.f; }
    float acc[kHeads][4];
#pragma unroll
    for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[h][e] = 0.f;
    for (int r0 = 0; r0 < n; r0 += kRows) {
        __syncthreads();
        if (tid < kRows) {
            const int r = r0 + tid;
            int64_t off = -1;
            float sc = 1.f;
            if (r < n) {
                int64_t lead = b, row = r;
                if (a.table) {
                    const int pg = r / a.page_size;
                    row = r - pg * a.page_size;
                    lead = a.table[b * a.table_ld + pg];
                }
                if (lead >= 0 && lead < a.n_pages) {
                    off = lead * a.seq_b + row * a.tok_b;
                    if (a.kv_scale) sc = a.kv_scale[lead * a.scale_seq + row];
                } else report(a.status, LSA_ERR_DEVICE_DATA);
            }
            s.row[tid] = off;
            s.scale[tid] = sc;
        }
        __syncthreads();
        for (int i = tid; i < kRows * kD; i += kThreads) {
            const int r = i / kD, d = i % kD;
            float v = 0.f;
            if (s.row[r] >= 0) {
                const uint8_t* p = a.kv + s.row[r];
                if (a.kv_scale) v = __half2float(__ushort_as_half((unsigned short)(e4m3x2_to_f16x2(p[d]) & 0xffff))) * s.scale[r];
                else v = bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[d]);
            }
            s.k[r][d] = v;
        }
        __syncthreads();
        for (int i = tid; i < kHeads * kRows; i += kThreads) {
            const int h = i / kRows, r = i % kRows;
            float z = 0.f;
            for (int d = 0; d < kD; ++d) z = fmaf(s.q[h][d], s.k[r][d], z);
            s.p[h][r] = s.row[r] >= 0 ? z : kNegInf;
        }
        __syncthreads();
        if (tid < kHeads) {
            float m = s.m[tid];
            for (int r = 0; r < kRows; ++r) m = fmaxf(m, s.p[tid][r]);
            const float ref = m == kNegInf ? 0.f : m;
            const float al = exp2f(s.m[tid] - ref);
            float l = s.l[tid] * al;
            for (int r = 0; r < kRows; ++r) {
                s.p[tid][r] = exp2f(s.p[tid][r] - ref);
                l += s.p[tid][r];
            }
            s.m[tid] = m; s.l[tid] = l; s.alpha[tid] = al;
        }
        __syncthreads();
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
            const float al = s.alpha[h];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float v = acc[h][e] * al;
                for (int r = 0; r < kRows; ++r) v = fmaf(s.p[h][r], s.k[r][tid + e * kThreads], v);
                acc[h][e] = v;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
        if (h >= nh) continue;
        const float l = s.l[h], inv = l > 0.f ? 1.f / l : 0.f;
        const size_t row = (size_t)t * a.H + h0 + h;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const size_t i = row * kDv + tid + e * kThreads;
            if (a.o_f32) static_cast<float*>(a.o)[i] = acc[h][e] * inv;
            else static_cast<__nv_bfloat16*>(a.o)[i] = __float2bfloat16_rn(acc[h][e] * inv);
        }
        if (tid == 0 && a.lse) a.lse[row] = l > 0.f ? (s.m[h] + log2f(l)) * 0.69314718055994530942f : kNegInf;
    }
}

}  // namespace

size_t latent_attn_ws(int, int, int) { return 256; }

cudaError_t launch_latent_attn(const LatentArgs& a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(latent_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    latent_attn_kernel<<<dim3(a.T, (a.H + kHeads - 1) / kHeads), kThreads, sizeof(Smem), st>>>(a);
    return cudaGetLastError();
}

}  // namespace lsa
