// gdn_scan.cu -- the gated linear recurrence per channel (sm_100a), its gradients
// and one decode step.
//
//   h_t = a_t h_{t-1} + x_t,  a_t = exp(log_alpha_t)
//
// Gradients: with u_t = a_t g_t (what token t hands back to token t - 1),
//   u_t = a_t (dh_t + u_{t+1}),  dx_t = dh_t + u_{t+1},  dlog_alpha_t = u_t h_{t-1},
// u behind the last token being dh_final, and dh0 = u at the first token.
//
// All of it is HBM-bound: 3 flops and one exp per element.
#include <cuda_bf16.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}

// Token range [lo, hi) of sequence n, kept within the T rows.
__device__ __forceinline__ void range_of(const int32_t* cu, int n, int T, int& lo, int& hi) {
    lo = cu ? min(max(cu[n], 0), T) : 0;
    hi = cu ? min(max(cu[n + 1], lo), T) : T;
}

// Grid (N, channel blocks): one thread walks one channel of one sequence.
template <typename IO, typename G>
__global__ void __launch_bounds__(128) scan_kernel(const ScanArgs p) {
    const int n = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x;
    if (c >= p.C) return;
    int lo, hi;
    range_of(p.cu_seqlens, n, p.T, lo, hi);
    float h = p.h0 ? p.h0[(int64_t)n * p.C + c] : 0.f;
#pragma unroll 8
    for (int64_t t = lo; t < hi; ++t) {
        const float a = expf(to_f(static_cast<const G*>(p.la)[t * p.la_stride + c]));
        h = fmaf(a, h, to_f(static_cast<const IO*>(p.x)[t * p.x_stride + c]));
        static_cast<IO*>(p.h)[t * p.h_stride + c] = from_f<IO>(h);
    }
    if (p.h_final) p.h_final[(int64_t)n * p.C + c] = h;
}

template <typename IO, typename G>
__global__ void __launch_bounds__(128) scan_backward_kernel(const ScanGradArgs p) {
    const int n = blockIdx.x;
    const int64_t c = (int64_t)blockIdx.y * 128 + threadIdx.x;
    if (c >= p.C) return;
    int lo, hi;
    range_of(p.cu_seqlens, n, p.T, lo, hi);
    float u = p.dh_final ? p.dh_final[(int64_t)n * p.C + c] : 0.f;
    for (int64_t t = hi - 1; t >= lo; --t) {
        const float a = expf(to_f(static_cast<const G*>(p.la)[t * p.la_stride + c]));
        const float g = u + to_f(static_cast<const IO*>(p.dh)[t * p.dh_stride + c]);
        const float before = t > lo ? to_f(static_cast<const IO*>(p.h)[(t - 1) * p.h_stride + c])
                                    : (p.h0 ? p.h0[(int64_t)n * p.C + c] : 0.f);
        u = a * g;
        static_cast<IO*>(p.dx)[t * p.dx_stride + c] = from_f<IO>(g);
        static_cast<G*>(p.dla)[t * p.dla_stride + c] = from_f<G>(u * before);
    }
    if (p.dh0) p.dh0[(int64_t)n * p.C + c] = u;
}

template <typename IO, typename G>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanArgs p) {
    const int64_t n = (int64_t)p.T * p.C;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t b = i / p.C, c = i - b * p.C;
        const float a = expf(to_f(static_cast<const G*>(p.la)[b * p.la_stride + c]));
        const float h = fmaf(a, p.h_final[i], to_f(static_cast<const IO*>(p.x)[b * p.x_stride + c]));
        p.h_final[i] = h;
        static_cast<IO*>(p.h)[b * p.h_stride + c] = from_f<IO>(h);
    }
}

}  // namespace

// One call of `fn<IO, G>` for the types of a scan.
#define GDN_SCAN_TYPES(fn, ...)                                                                \
    (bf16 ? (gate_bf16 ? fn<__nv_bfloat16, __nv_bfloat16> __VA_ARGS__                         \
                       : fn<__nv_bfloat16, float> __VA_ARGS__)                                 \
          : (gate_bf16 ? fn<float, __nv_bfloat16> __VA_ARGS__ : fn<float, float> __VA_ARGS__))

cudaError_t launch_scan(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream) {
    const dim3 grid(a.N, (a.C + 127) / 128);
    GDN_SCAN_TYPES(scan_kernel, <<<grid, 128, 0, stream>>>(a));
    return cudaGetLastError();
}

cudaError_t launch_scan_backward(const ScanGradArgs& a, bool bf16, bool gate_bf16,
                                 cudaStream_t stream) {
    const dim3 grid(a.N, (a.C + 127) / 128);
    GDN_SCAN_TYPES(scan_backward_kernel, <<<grid, 128, 0, stream>>>(a));
    return cudaGetLastError();
}

cudaError_t launch_scan_step(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream) {
    const int64_t blocks = ((int64_t)a.T * a.C + 255) / 256;
    const int grid = (int)(blocks < 148 * 64 ? blocks : 148 * 64);
    GDN_SCAN_TYPES(scan_step_kernel, <<<grid, 256, 0, stream>>>(a));
    return cudaGetLastError();
}

}  // namespace gdn
