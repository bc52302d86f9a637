// Latent attention in the expanded form: packed prompts with per-head keys and values, 64 shared rotary
// dimensions.
//
//   z = sm_scale (q[0:128] . k_nope + q[128:192] . k_rope), o = softmax(z) v.
//
// One pass with a running maximum and sum.  Block = (16 queries of a sequence, head): FP32 on CUDA cores,
// tiles of 16 keys, each thread two of the 16 x 16 scores and one of the 128 value dimensions of all 16 queries.
#include <cmath>

#include "kernels.cuh"

namespace lsa {

namespace {

constexpr int kThreads = 128, kQ = 16, kRows = 16, kDn = 128, kDr = 64, kD = kDn + kDr, kDv = 128;

struct Smem {
    float q[kQ][kD + 1];
    float k[kRows][kD + 1];
    float v[kRows][kDv];
    float p[kQ][kRows];
    float m[kQ], l[kQ], alpha[kQ];
};

__global__ void __launch_bounds__(kThreads) latent_expanded_kernel(ExpandedArgs a) {
    extern __shared__ uint8_t raw[];
    Smem& s = *reinterpret_cast<Smem*>(raw);
    const int i0 = blockIdx.x * kQ, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int qs = a.q_start[b], nq = a.q_start[b + 1] - qs, ks = a.k_start[b], nk = a.k_start[b + 1] - ks;
    const bool ok = qs >= 0 && nq >= 0 && nq <= a.max_q && qs + (int64_t)nq <= a.T && ks >= 0 && nk >= 0 && ks + (int64_t)nk <= a.S;
    if (!ok && i0 == 0 && h == 0 && tid == 0) report(a.status, LSA_ERR_DEVICE_DATA);
    if (qs < 0 || nq < 0 || qs + (int64_t)nq > a.T || ks < 0 || nk < 0 || ks + (int64_t)nk > a.S) return;
    const int n = min(kQ, min(nq, a.max_q) - i0);
    if (n <= 0) return;
    for (int i = tid; i < kQ * kD; i += kThreads) {
        const int r = i / kD, d = i % kD;
        s.q[r][d] = r < n ? bf16_bits_to_float(a.q[(qs + i0 + r) * a.qt + h * a.qh + d]) * a.sm_scale_log2 : 0.f;
    }
    if (tid < kQ) { s.m[tid] = kNegInf; s.l[tid] = 0.f; }
    float acc[kQ];
#pragma unroll
    for (int r = 0; r < kQ; ++r) acc[r] = 0.f;
    const int end = a.causal ? min(nk, i0 + n + nk - nq) : nk;
    for (int k0 = 0; k0 < end; k0 += kRows) {
        __syncthreads();
        for (int i = tid; i < kRows * kD; i += kThreads) {
            const int r = i / kD, d = i % kD;
            const int64_t j = ks + k0 + r;
            s.k[r][d] = k0 + r >= end ? 0.f
                : bf16_bits_to_float(d < kDn ? a.kn[j * a.kt + h * a.kh + d] : a.kr[j * a.rt + d - kDn]);
            if (d < kDv) s.v[r][d] = k0 + r >= end ? 0.f : bf16_bits_to_float(a.v[j * a.vt + h * a.vh + d]);
        }
        __syncthreads();
        for (int i = tid; i < kQ * kRows; i += kThreads) {
            const int r = i / kRows, j = i % kRows;
            float z = 0.f;
            for (int d = 0; d < kD; ++d) z = fmaf(s.q[r][d], s.k[j][d], z);
            const bool seen = k0 + j < end && (!a.causal || k0 + j <= i0 + r + nk - nq);
            s.p[r][j] = seen ? z : kNegInf;
        }
        __syncthreads();
        if (tid < kQ) {
            float m = s.m[tid];
            for (int j = 0; j < kRows; ++j) m = fmaxf(m, s.p[tid][j]);
            const float ref = m == kNegInf ? 0.f : m;
            const float al = exp2f(s.m[tid] - ref);
            float l = s.l[tid] * al;
            for (int j = 0; j < kRows; ++j) {
                s.p[tid][j] = exp2f(s.p[tid][j] - ref);
                l += s.p[tid][j];
            }
            s.m[tid] = m; s.l[tid] = l; s.alpha[tid] = al;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < kQ; ++r) {
            float v = acc[r] * s.alpha[r];
            for (int j = 0; j < kRows; ++j) v = fmaf(s.p[r][j], s.v[j][tid], v);
            acc[r] = v;
        }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kQ; ++r) {
        if (r >= n) continue;
        const float l = s.l[r], inv = l > 0.f ? 1.f / l : 0.f;
        const size_t row = (size_t)(qs + i0 + r) * a.H + h;
        if (a.o_f32) static_cast<float*>(a.o)[row * kDv + tid] = acc[r] * inv;
        else static_cast<__nv_bfloat16*>(a.o)[row * kDv + tid] = __float2bfloat16_rn(acc[r] * inv);
        if (tid == 0 && a.lse) a.lse[row] = l > 0.f ? (s.m[r] + log2f(l)) * 0.69314718055994530942f : kNegInf;
    }
}

}  // namespace

cudaError_t launch_latent_expanded(const ExpandedArgs& a, cudaStream_t st) {
    cudaError_t e = cudaFuncSetAttribute(latent_expanded_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
    if (e != cudaSuccess) return e;
    latent_expanded_kernel<<<dim3((a.max_q + kQ - 1) / kQ, a.H, a.B), kThreads, sizeof(Smem), st>>>(a);
    return cudaGetLastError();
}

}  // namespace lsa
