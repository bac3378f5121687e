// gdn_norm.cu -- the norm behind a mixer (sm_100a): per token and head, channels
// last, with its activation or activated gate, and its gradients.
//
//   m = mean (or 0), r = 1 / sqrt(mean (x - m)^2 + eps), xh = (x - m) r,
//   n = w xh + b;  y = n act(z) with a gate, act(n) without.
//
// Gradients, with dn = dy act(z) (gated) or dy act'(n), and e = dn w:
//   dz = dy n act'(z),  dw = sum dn xh,  db = sum dn,
//   dx = r (e - [mean e] - xh mean(e xh))      (mean e only when centred).
//
// Both directions are HBM-bound: one pass over the data, a group's channels in
// the registers of LG lanes, its statistics by shuffles.  A lane group keeps one
// head and walks over the tokens, so that the weights stay in registers and the
// sums of dw and db run in registers over all its tokens.
#include <cuda_bf16.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"

namespace gdn {

namespace {

constexpr int NT = 256;       // threads per block
constexpr int FWD_BLOCKS = 8;  // blocks per SM the grids are sized for
constexpr int BWD_BLOCKS = 4;

// VE consecutive channels as floats.
template <typename IO, int VE>
struct Chan;
template <>
struct Chan<__nv_bfloat16, 8> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                       pack_bf16x2(v[6], v[7]));
    }
};
template <>
struct Chan<float, 4> {
    static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
    }
    static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <>
struct Chan<__nv_bfloat16, 1> {
    static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[1]) {
        v[0] = __bfloat162float(*p);
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[1]) {
        *p = __float2bfloat16_rn(v[0]);
    }
};
template <>
struct Chan<float, 1> {
    static __device__ __forceinline__ void load(const float* p, float (&v)[1]) { v[0] = *p; }
    static __device__ __forceinline__ void store(float* p, const float (&v)[1]) { *p = v[0]; }
};

struct NormParams {
    const void *x, *z, *dy;
    void *y, *dz;            // y: the output, or dx
    const float *w, *b;
    float *dw_part, *db_part;
    int64_t xs, zs, dys, ys, dzs;  // row strides in elements
    int T, H, d, nvec, streams;
    bool per_head, centred, silu, has_bias;
    float eps, inv_d;
};

__device__ __forceinline__ float sigmoid_fast(float y) { return __fdividef(1.f, 1.f + __expf(-y)); }

template <int LG>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = LG / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Where a lane group works: lane group g of the grid takes head g % H and the
// tokens g / H, g / H + streams, ...  (neighbours take neighbouring heads of a
// token, so a warp's loads are contiguous).
template <int LG>
struct Place {
    int lane, head, trips;
    int64_t row;
    bool active;
    __device__ __forceinline__ explicit Place(const NormParams& p) {
        constexpr int GPB = NT / LG;
        lane = threadIdx.x % LG;
        const int64_t g = (int64_t)blockIdx.x * GPB + threadIdx.x / LG;
        active = g < (int64_t)p.streams * p.H;
        head = (int)(g % p.H);
        row = g / p.H;
        // the whole warp makes the trips of its first lane group, which has the most
        const int64_t g0 = (int64_t)blockIdx.x * GPB + (threadIdx.x & ~31) / LG;
        const int64_t row0 = g0 / p.H;
        trips = row0 < p.T && g0 < (int64_t)p.streams * p.H
                    ? (int)((p.T - row0 + p.streams - 1) / p.streams)
                    : 0;
    }
};

// xh and 1 / sqrt(...) of one group, from its channels in v (zeros outside it).
template <int LG, int NV, int VE>
__device__ __forceinline__ float normalise(float (&v)[NV][VE], int lane, int nvec, bool centred,
                                           float inv_d, float eps) {
    if (centred) {
        float s = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < VE; ++i) s += v[j][i];
        const float m = group_sum<LG>(s) * inv_d;
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (lane + LG * j < nvec)
#pragma unroll
                for (int i = 0; i < VE; ++i) v[j][i] -= m;
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) ss = fmaf(v[j][i], v[j][i], ss);
    const float r = rsqrtf(fmaf(group_sum<LG>(ss), inv_d, eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) v[j][i] *= r;
    return r;
}

template <typename IO, int VE, int LG, int NV, bool GATED>
__global__ void __launch_bounds__(NT) group_norm_kernel(const NormParams p) {
    const Place<LG> at(p);
    float w[NV][VE], b[NV][VE];
    const int wo = p.per_head ? at.head * p.d : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const int vec = at.lane + LG * j;
            const bool in = vec < p.nvec;
            w[j][i] = in ? p.w[wo + vec * VE + i] : 0.f;
            b[j][i] = in && p.has_bias ? p.b[wo + vec * VE + i] : 0.f;
        }
    const int col = at.head * p.d + at.lane * VE;
    int64_t row = at.row;
    for (int it = 0; it < at.trips; ++it, row += p.streams) {
        const bool ok = at.active && row < p.T;
        float v[NV][VE], g[NV][VE];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = ok && at.lane + LG * j < p.nvec;
#pragma unroll
            for (int i = 0; i < VE; ++i) v[j][i] = 0.f, g[j][i] = 0.f;
            if (in) {
                Chan<IO, VE>::load(static_cast<const IO*>(p.x) + row * p.xs + col + LG * VE * j,
                                   v[j]);
                if (GATED)
                    Chan<IO, VE>::load(
                        static_cast<const IO*>(p.z) + row * p.zs + col + LG * VE * j, g[j]);
            }
        }
        normalise<LG>(v, at.lane, p.nvec, p.centred, p.inv_d, ok ? p.eps : 1.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float n = fmaf(v[j][i], w[j][i], b[j][i]);
                const float a = GATED ? g[j][i] : n;
                const float s = p.silu ? a * sigmoid_fast(a) : a;
                v[j][i] = GATED ? n * s : s;
            }
            if (ok && at.lane + LG * j < p.nvec)
                Chan<IO, VE>::store(static_cast<IO*>(p.y) + row * p.ys + col + LG * VE * j, v[j]);
        }
    }
}

template <typename IO, int VE, int LG, int NV, bool GATED>
__global__ void __launch_bounds__(NT) group_norm_backward_kernel(const NormParams p) {
    constexpr int GPB = NT / LG;
    extern __shared__ float part[];  // [GPB][d], for the sums over a block's groups
    const Place<LG> at(p);
    float w[NV][VE], b[NV][VE], dw[NV][VE], db[NV][VE];
    const int wo = p.per_head ? at.head * p.d : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const int vec = at.lane + LG * j;
            const bool in = vec < p.nvec;
            w[j][i] = in ? p.w[wo + vec * VE + i] : 0.f;
            b[j][i] = in && p.has_bias ? p.b[wo + vec * VE + i] : 0.f;
            dw[j][i] = db[j][i] = 0.f;
        }
    const int col = at.head * p.d + at.lane * VE;
    int64_t row = at.row;
    for (int it = 0; it < at.trips; ++it, row += p.streams) {
        const bool ok = at.active && row < p.T;
        float v[NV][VE], g[NV][VE], dn[NV][VE];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const bool in = ok && at.lane + LG * j < p.nvec;
#pragma unroll
            for (int i = 0; i < VE; ++i) v[j][i] = 0.f, g[j][i] = 0.f, dn[j][i] = 0.f;
            if (in) {
                const int c = col + LG * VE * j;
                Chan<IO, VE>::load(static_cast<const IO*>(p.x) + row * p.xs + c, v[j]);
                Chan<IO, VE>::load(static_cast<const IO*>(p.dy) + row * p.dys + c, dn[j]);
                if (GATED) Chan<IO, VE>::load(static_cast<const IO*>(p.z) + row * p.zs + c, g[j]);
            }
        }
        // (a lane group past the last token adds exact zeros to its sums)
        const float r =
            normalise<LG>(v, at.lane, p.nvec, p.centred, p.inv_d, ok ? p.eps : 1.f);
        float se = 0.f, sx = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float n = fmaf(v[j][i], w[j][i], b[j][i]);
                const float a = GATED ? g[j][i] : n;
                float value = a, slope = 1.f;
                if (p.silu) {
                    const float s = sigmoid_fast(a);
                    value = a * s;
                    slope = fmaf(value, 1.f - s, s);
                }
                const float dy = dn[j][i];
                if (GATED) {
                    g[j][i] = dy * n * slope;
                    dn[j][i] = dy * value;
                } else {
                    dn[j][i] = dy * slope;
                }
                dw[j][i] = fmaf(dn[j][i], v[j][i], dw[j][i]);
                db[j][i] += dn[j][i];
                dn[j][i] *= w[j][i];
                se += dn[j][i];
                sx = fmaf(dn[j][i], v[j][i], sx);
            }
            if (GATED && ok && at.lane + LG * j < p.nvec)
                Chan<IO, VE>::store(static_cast<IO*>(p.dz) + row * p.dzs + col + LG * VE * j, g[j]);
        }
        const float cx = group_sum<LG>(sx) * p.inv_d;
        const float ce = p.centred ? group_sum<LG>(se) * p.inv_d : 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < VE; ++i) v[j][i] = r * (dn[j][i] - ce - v[j][i] * cx);
            if (ok && at.lane + LG * j < p.nvec)
                Chan<IO, VE>::store(static_cast<IO*>(p.y) + row * p.ys + col + LG * VE * j, v[j]);
        }
    }

    // partial sums: one row per stream of a head, or one row per block
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* out = which ? p.db_part : p.dw_part;
        if (!out) continue;
        if (p.per_head) {
            if (at.active) {
                const int64_t g = (int64_t)blockIdx.x * GPB + threadIdx.x / LG;
                float* o = out + (g / p.H) * ((int64_t)p.H * p.d) + at.head * p.d;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < VE; ++i)
                        if (at.lane + LG * j < p.nvec)
                            o[(at.lane + LG * j) * VE + i] = which ? db[j][i] : dw[j][i];
            }
        } else {
            float* mine = part + (threadIdx.x / LG) * p.d;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < VE; ++i)
                    if (at.lane + LG * j < p.nvec)
                        mine[(at.lane + LG * j) * VE + i] = which ? db[j][i] : dw[j][i];
            __syncthreads();
            for (int c = threadIdx.x; c < p.d; c += NT) {
                float s = 0.f;
                for (int q = 0; q < GPB; ++q) s += part[q * p.d + c];
                out[(int64_t)blockIdx.x * p.d + c] = s;
            }
        }
    }
}

// Column sums of part [rows, cols] into out (blockIdx.y: the first pair, then the
// second), in an order that does not depend on timing.
__global__ void __launch_bounds__(256)
    column_sums_kernel(const float* part0, const float* part1, float* out0, float* out1, int rows,
                       int cols) {
    __shared__ float sm[8][33];
    const float* part = blockIdx.y ? part1 : part0;
    float* out = blockIdx.y ? out1 : out0;
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + tx;
    float s = 0.f;
    if (c < cols)
#pragma unroll 4
        for (int r = ty; r < rows; r += 8) s += part[(int64_t)r * cols + c];
    sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && c < cols) {
#pragma unroll
        for (int q = 1; q < 8; ++q) s += sm[q][tx];
        out[c] = s;
    }
}

int lanes_for(int nvec) {
    int lg = 1;
    while (lg < 32 && lg < nvec) lg *= 2;
    return lg;
}

// Blocks of a grid of lane groups, and the tokens walked side by side per head.
struct Shape {
    int lg, blocks, streams;
};
Shape shape_of(int T, int H, int nvec, int blocks_per_sm) {
    Shape s;
    s.lg = lanes_for(nvec);
    const long long gpb = NT / s.lg, groups = (long long)T * H;
    const long long need = (groups + gpb - 1) / gpb, least = (H + gpb - 1) / gpb;
    long long blocks = (long long)device_sms() * blocks_per_sm;
    if (blocks < least) blocks = least;
    if (blocks > need) blocks = need;
    s.blocks = (int)blocks;
    s.streams = (int)(blocks * gpb / H);
    if (s.streams > T) s.streams = T;
    return s;
}

template <typename IO, int VE, int LG, int NV>
void launch_one(const NormParams& p, int blocks, bool backward, cudaStream_t stream) {
    if (backward) {
        const size_t smem = p.per_head ? 0 : (size_t)(NT / LG) * p.d * sizeof(float);
        if (p.z)
            group_norm_backward_kernel<IO, VE, LG, NV, true><<<blocks, NT, smem, stream>>>(p);
        else
            group_norm_backward_kernel<IO, VE, LG, NV, false><<<blocks, NT, smem, stream>>>(p);
    } else {
        if (p.z)
            group_norm_kernel<IO, VE, LG, NV, true><<<blocks, NT, 0, stream>>>(p);
        else
            group_norm_kernel<IO, VE, LG, NV, false><<<blocks, NT, 0, stream>>>(p);
    }
}

template <typename IO, int VE>
cudaError_t launch_ve(NormParams p, int blocks_per_sm, bool backward, cudaStream_t stream) {
    p.nvec = p.d / VE;
    const Shape s = shape_of(p.T, p.H, p.nvec, blocks_per_sm);
    p.streams = s.streams;
    constexpr int MAXNV = GDN_MAX_GROUP_DIM / VE / 32;
    switch (s.lg) {
        case 1: launch_one<IO, VE, 1, 1>(p, s.blocks, backward, stream); break;
        case 2: launch_one<IO, VE, 2, 1>(p, s.blocks, backward, stream); break;
        case 4: launch_one<IO, VE, 4, 1>(p, s.blocks, backward, stream); break;
        case 8: launch_one<IO, VE, 8, 1>(p, s.blocks, backward, stream); break;
        case 16: launch_one<IO, VE, 16, 1>(p, s.blocks, backward, stream); break;
        default: {
            const int nv = (p.nvec + 31) / 32;
            if (nv <= 1) launch_one<IO, VE, 32, 1>(p, s.blocks, backward, stream);
            else if (nv <= 2) launch_one<IO, VE, 32, 2>(p, s.blocks, backward, stream);
            else if (nv <= 4) launch_one<IO, VE, 32, 4>(p, s.blocks, backward, stream);
            else if constexpr (MAXNV > 4) {
                if (nv <= 8) launch_one<IO, VE, 32, 8>(p, s.blocks, backward, stream);
                else if constexpr (MAXNV > 8) {
                    if (nv <= 16) launch_one<IO, VE, 32, 16>(p, s.blocks, backward, stream);
                    else launch_one<IO, VE, 32, 32>(p, s.blocks, backward, stream);
                }
            }
        }
    }
    return cudaGetLastError();
}

// Channels per access: 16 bytes where every pointer, stride and the group allow it, else one.
int vector_of(const NormParams& p, bool bf16) {
    const int ve = bf16 ? 8 : 4;
    const void* ptrs[] = {p.x, p.z, p.dy, p.y, p.dz};
    const int64_t strides[] = {p.xs, p.zs, p.dys, p.ys, p.dzs};
    if (p.d % ve) return 1;
    for (int i = 0; i < 5; ++i)
        if (ptrs[i] && (reinterpret_cast<uintptr_t>(ptrs[i]) % 16 || strides[i] % ve)) return 1;
    return ve;
}

cudaError_t launch_any(const NormParams& p, bool bf16, int blocks_per_sm, bool backward,
                       cudaStream_t stream) {
    if (vector_of(p, bf16) > 1)
        return bf16 ? launch_ve<__nv_bfloat16, 8>(p, blocks_per_sm, backward, stream)
                    : launch_ve<float, 4>(p, blocks_per_sm, backward, stream);
    return bf16 ? launch_ve<__nv_bfloat16, 1>(p, blocks_per_sm, backward, stream)
                : launch_ve<float, 1>(p, blocks_per_sm, backward, stream);
}

NormParams params_of(const GroupNormArgs& a) {
    NormParams p{};
    p.x = a.x, p.z = a.z, p.dy = a.dy, p.y = a.y, p.dz = a.dz, p.w = a.weight, p.b = a.bias;
    p.xs = a.x_stride, p.zs = a.z_stride, p.dys = a.dy_stride, p.ys = a.y_stride;
    p.dzs = a.dz_stride;
    p.T = a.T, p.H = a.H, p.d = a.d, p.per_head = a.weight_heads != 1;
    p.centred = a.centred, p.silu = a.silu, p.has_bias = a.bias != nullptr;
    p.eps = a.eps, p.inv_d = 1.f / (float)a.d;
    return p;
}

// Rows of partial sums that the backward kernel writes: one per stream (weights
// per head) or one per block.
int partial_rows(int T, int H, int d, bool per_head, int ve) {
    const Shape s = shape_of(T, H, d / ve, BWD_BLOCKS);
    return per_head ? s.streams : s.blocks;
}

}  // namespace

cudaError_t launch_column_sums(const float* part0, const float* part1, float* out0, float* out1,
                               int rows, int cols, cudaStream_t stream) {
    column_sums_kernel<<<dim3((cols + 31) / 32, out1 ? 2 : 1), 256, 0, stream>>>(
        part0, part1, out0, out1, rows, cols);
    return cudaGetLastError();
}

cudaError_t launch_group_norm(const GroupNormArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    return launch_any(params_of(a), a.bf16, FWD_BLOCKS, false, stream);
}

size_t group_norm_backward_workspace_bytes(int T, int H, int d, int weight_heads, bool bf16) {
    if (T == 0) return 0;
    const bool per_head = weight_heads != 1;
    const size_t cols = (size_t)(per_head ? H : 1) * d;
    // enough for either access width: the pointers are not known here
    size_t rows = 0;
    for (const int ve : {bf16 ? 8 : 4, 1})
        if (d % ve == 0) {
            const size_t r = (size_t)partial_rows(T, H, d, per_head, ve);
            rows = r > rows ? r : rows;
        }
    return 2 * ((rows * cols * sizeof(float) + 255) / 256 * 256);
}

cudaError_t launch_group_norm_backward(const GroupNormArgs& a, float* dweight, float* dbias,
                                       void* workspace, cudaStream_t stream) {
    const bool per_head = a.weight_heads != 1;
    const int cols = (per_head ? a.H : 1) * a.d;
    NormParams p = params_of(a);
    int rows = 0;
    if (a.T > 0) {
        const size_t half =
            group_norm_backward_workspace_bytes(a.T, a.H, a.d, a.weight_heads, a.bf16) / 2;
        p.dw_part = static_cast<float*>(workspace);
        if (dbias) p.db_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + half);
        const cudaError_t e = launch_any(p, a.bf16, BWD_BLOCKS, true, stream);
        if (e != cudaSuccess) return e;
        rows = partial_rows(a.T, a.H, a.d, per_head, vector_of(p, a.bf16));
    }
    return launch_column_sums(p.dw_part, p.db_part, dweight, dbias, rows, cols, stream);
}

}  // namespace gdn
