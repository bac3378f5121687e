// gdn_sums.cuh -- the second step of a gradient that is a sum over tokens: kernels leave one
// row of partial sums per run of tokens, and these are added in an order that does not depend
// on timing.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdn {

// The second step's launch does not wait for the first one's end: its blocks come in as the
// first one's leave, and those that read what the first wrote wait for its end themselves.
// Every block of the first step allows that (once they all have, the second may start); the
// last block of the second ends behind the first, so what follows in the stream is ordered
// behind both.
__device__ __forceinline__ void allow_next_step() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_first_step() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_second_step(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t stream,
                               const A&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// out = column sums of part [rows, cols].
struct ColumnSums {
    const float* part;
    float* out;
    int rows, cols;
};

// Columns 32 bx .. of a, by a block of 32 x RT threads.  Bound by the latency of its loads:
// RT rows at once, eight loads in flight per thread.
template <int RT>
__device__ __forceinline__ void column_sums(const ColumnSums& a, int bx) {
    __shared__ float sm[RT][33];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = bx * 32 + tx;
    float s = 0.f;
    if (c < a.cols)
        for (int r = ty; r < a.rows; r += 8 * RT) {
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = r + k * RT < a.rows ? a.part[(int64_t)(r + k * RT) * a.cols + c] : 0.f;
#pragma unroll
            for (int k = 0; k < 8; ++k) s += v[k];
        }
    sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < a.cols) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < RT; ++q) s += sm[q][tx];
        a.out[c] = s;
    }
}

}  // namespace gdn
