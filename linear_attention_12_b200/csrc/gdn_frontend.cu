// gdn_frontend.cu -- the GDN front end (sm_100a): short causal convolution of
// the q, k, v channels, L2 normalisation of q and k, gate activations.
//
// What it computes (the jianying88.com article "Qwen3.8-Flash-Next混合注意力
// 深度解析…", section 三: the GDN layer stacks a short convolution of kernel
// width 4, config linear_conv_kernel_dim 4; the pages print no formula):
//
//   y[t, c] = sum_{i=0..3} w[c, i] x[t - 3 + i, c]    (x = 0 before the sequence start)
//   y = act(y)                                        (none, or SiLU y sigmoid(y))
//   q, k = y / sqrt(sum_head y^2 + eps)               (per token and head)
//   log_alpha = -softplus(a),  beta = sigmoid(b)
//
// The normalisation and the gate activations follow the recipes of the
// workloads the layer is measured on.  Channels are ordered q (head-major),
// k, v; the weight is [(2 H_qk + H_v) d, 4] fp32.
//
// The work is HBM-bound.  The prefill form stages each block's rows in shared
// memory with bulk copies (up to 35 KB in flight per block, six blocks per
// SM), then one warp per head convolves them with a rolling window, each lane
// holding 4 channels; outputs leave as one coalesced 256-byte (bf16) or
// 512-byte (fp32) row segment per warp.
#include <cuda_bf16.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_sums.cuh"

namespace gdn {

namespace {

constexpr int FD = 128;      // head dim

template <typename IO>
struct Vec4;
template <>
struct Vec4<__nv_bfloat16> {
    using Raw = uint2;  // 4 channels as stored
    static __device__ __forceinline__ Raw load_raw(const __nv_bfloat16* p) {
        return *reinterpret_cast<const uint2*>(p);
    }
    static __device__ __forceinline__ Raw zero() { return make_uint2(0u, 0u); }
    static __device__ __forceinline__ float4 widen(Raw u) {
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
        return make_float4(a.x, a.y, b.x, b.y);
    }
    static __device__ __forceinline__ float4 load(const __nv_bfloat16* p) {
        return widen(load_raw(p));
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, float4 v) {
        uint2 u;
        u.x = pack_bf16x2(v.x, v.y);
        u.y = pack_bf16x2(v.z, v.w);
        *reinterpret_cast<uint2*>(p) = u;
    }
};
template <>
struct Vec4<float> {
    using Raw = float4;
    static __device__ __forceinline__ Raw load_raw(const float* p) {
        return *reinterpret_cast<const float4*>(p);
    }
    static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
    static __device__ __forceinline__ float4 widen(Raw u) { return u; }
    static __device__ __forceinline__ float4 load(const float* p) { return load_raw(p); }
    static __device__ __forceinline__ void store(float* p, float4 v) {
        *reinterpret_cast<float4*>(p) = v;
    }
};

__device__ __forceinline__ float silu(float y) { return y / (1.f + expf(-y)); }

__device__ __forceinline__ float4 act4(float4 y, int act) {
    if (act == GDN_ACT_SILU) return make_float4(silu(y.x), silu(y.y), silu(y.z), silu(y.w));
    return y;
}

// y = w0 x_{t-3} + w1 x_{t-2} + w2 x_{t-1} + w3 x_t for 4 channels
__device__ __forceinline__ float4 conv4(const float4 (&w)[4], float4 x3, float4 x2, float4 x1,
                                        float4 x0) {
    float4 y;
    y.x = fmaf(w[0].x, x3.x, fmaf(w[1].x, x2.x, fmaf(w[2].x, x1.x, w[3].x * x0.x)));
    y.y = fmaf(w[0].y, x3.y, fmaf(w[1].y, x2.y, fmaf(w[2].y, x1.y, w[3].y * x0.y)));
    y.z = fmaf(w[0].z, x3.z, fmaf(w[1].z, x2.z, fmaf(w[2].z, x1.z, w[3].z * x0.z)));
    y.w = fmaf(w[0].w, x3.w, fmaf(w[1].w, x2.w, fmaf(w[2].w, x1.w, w[3].w * x0.w)));
    return y;
}

// Scale 4 channels of a head row to unit L2 norm over the head (the warp holds
// the whole 128-channel row).
__device__ __forceinline__ float4 l2norm_row(float4 y, float eps) {
    float ss = y.x * y.x + y.y * y.y + y.z * y.z + y.w * y.w;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float r = rsqrtf(ss + eps);
    return make_float4(y.x * r, y.y * r, y.z * r, y.w * r);
}

// softplus(a) = max(a, 0) + log(1 + e^{-|a|}), without overflow
__device__ __forceinline__ float softplus(float a) { return fmaxf(a, 0.f) + log1pf(expf(-fabsf(a))); }
__device__ __forceinline__ float sigmoidf(float b) { return 1.f / (1.f + expf(-b)); }

// Start of the sequence that holds token t (the last cu[n] <= t).
__device__ __forceinline__ int seq_start(const int32_t* cu, int N, int t) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return cu[lo];
}

struct FrontendParams {
    const void* x[3];      // q_raw, k_raw, v_raw
    void* y[3];            // q, k, v
    const float* w;        // [(2 H_qk + H_v) d, 4]
    const float* a;        // [T, H_v]
    const float* b;
    float* log_alpha;
    float* beta;
    const int32_t* cu_seqlens;
    int N, T, H_qk, H_v;
    int act;
    float eps;
};

// ---- prefill front end: rows staged in shared memory by bulk copies ----
//
// A block handles FE_TC consecutive tokens of a group of HG heads of one
// kind (HG = 4 for bf16, 2 for fp32: 1 KB of each token row).  One thread
// issues one bulk copy per token row -- the three rows of history before the
// tile and its FE_TC tokens -- so that the whole tile (up to 35 KB) is in
// flight at once; warp w then convolves head w of the group from shared
// memory with a rolling window, each lane holding 4 channels.
constexpr int FE_TC = 32;                         // tokens per block
constexpr int FE_ROWS = FE_TC + 3;                // staged rows: history + tile
constexpr uint32_t FE_ROWB = 1024;                // shared-memory bytes of one staged row
constexpr uint32_t FE_SMEM = FE_ROWS * FE_ROWB + 16;  // + mbarrier and abort flag
static_assert(FE_TC <= 32, "lane j handles token j of a tile (gates, sequence starts)");

template <typename IO>
__host__ __device__ constexpr int fe_heads() { return FE_ROWB / (FD * sizeof(IO)); }

// Grid: token tiles x head groups (q groups, then k, then v), the group index
// varying fastest so that the blocks resident at one time read whole token rows.
template <typename IO, int ACT>
__global__ void __launch_bounds__(fe_heads<IO>() * 32)
    frontend_kernel(const FrontendParams p) {
    constexpr int HG = fe_heads<IO>();
    extern __shared__ __align__(128) uint8_t fe_sm[];
    uint64_t* bar = reinterpret_cast<uint64_t*>(fe_sm + FE_ROWS * FE_ROWB);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(fe_sm + FE_ROWS * FE_ROWB + 8);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int gq = (p.H_qk + HG - 1) / HG, gv = (p.H_v + HG - 1) / HG;
    const int NG = 2 * gq + gv;
    const int grp = blockIdx.x % NG, tile = blockIdx.x / NG;
    const int kind = grp < gq ? 0 : (grp < 2 * gq ? 1 : 2);  // q, k, v
    const int head0 = HG * (kind == 0 ? grp : (kind == 1 ? grp - gq : grp - 2 * gq));
    const int H = kind == 2 ? p.H_v : p.H_qk;
    const int nh = min(HG, H - head0);
    const int t0 = tile * FE_TC;  // < T: the grid holds exactly the tiles that start inside
    const int t1 = min(t0 + FE_TC, p.T);
    const size_t rs = (size_t)H * FD;  // row stride in elements
    // (the pointers are picked without indexing the parameter arrays at run time)
    const IO* x = static_cast<const IO*>(kind == 0 ? p.x[0] : (kind == 1 ? p.x[1] : p.x[2]));
    IO* y = static_cast<IO*>(kind == 0 ? p.y[0] : (kind == 1 ? p.y[1] : p.y[2]));

    // staged row i holds token t0 - 3 + i; rows before token 0 are not loaded
    const int r_lo = max(0, t0 - 3);
    if (threadIdx.x == 0) {
        mbar_init(bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        const uint32_t row_bytes = (uint32_t)nh * FD * sizeof(IO);
        mbar_arrive_expect_tx(bar, (uint32_t)(t1 - r_lo) * row_bytes);
        for (int t = r_lo; t < t1; ++t)
            bulk_load(fe_sm + (t - (t0 - 3)) * FE_ROWB, x + (size_t)t * rs + (size_t)head0 * FD,
                      row_bytes, bar);
    }

    // while the rows land: weights, gate inputs, sequence starts
    const bool active = warp < nh;
    const int head = head0 + min(warp, nh - 1);
    const int hid = (kind == 0 ? 0 : (kind == 1 ? p.H_qk : 2 * p.H_qk)) + head;
    float4 w[4];
    {
        const float4* wp = reinterpret_cast<const float4*>(p.w + ((size_t)hid * FD + 4 * lane) * 4);
        // 4 channels x 4 taps, channel-major -> per-tap float4 over the channels
        const float4 c0 = wp[0], c1 = wp[1], c2 = wp[2], c3 = wp[3];
        w[0] = make_float4(c0.x, c1.x, c2.x, c3.x);
        w[1] = make_float4(c0.y, c1.y, c2.y, c3.y);
        w[2] = make_float4(c0.z, c1.z, c2.z, c3.z);
        w[3] = make_float4(c0.w, c1.w, c2.w, c3.w);
    }
    const int tg = t0 + lane;  // lane <-> token for the gates and the sequence starts
    float ga = 0.f, gb = 0.f;
    const bool gate = kind == 2 && active && tg < t1;
    if (gate) {
        ga = p.a[(size_t)tg * p.H_v + head];
        gb = p.b[(size_t)tg * p.H_v + head];
    }
    const int s_mine = seq_start(p.cu_seqlens, p.N, min(tg, t1 - 1));
    const bool one_seq = __all_sync(0xffffffffu, s_mine <= t0 - 3);

    __syncthreads();  // the barrier is initialised before anyone waits on it
    const bool ok = mbar_wait(bar, 0, abort_flag);
    if (!__syncthreads_and(ok)) {
        // the copies may still land: wait for them (bounded) before the block exits
        if (threadIdx.x == 0) {
            const unsigned long long ts = globaltimer();
            while (!mbar_try_wait(smem_u32(bar), 0) && globaltimer() - ts < kWaitLimitNs) {
            }
        }
        __syncthreads();
        return;
    }

    if (active) {
        const uint8_t* rp = fe_sm + (warp * FD + 4 * lane) * sizeof(IO);
        float4 x3 = Vec4<IO>::widen(*reinterpret_cast<const typename Vec4<IO>::Raw*>(rp));
        float4 x2 = Vec4<IO>::widen(*reinterpret_cast<const typename Vec4<IO>::Raw*>(rp + FE_ROWB));
        float4 x1 =
            Vec4<IO>::widen(*reinterpret_cast<const typename Vec4<IO>::Raw*>(rp + 2 * FE_ROWB));
        IO* yt = y + (size_t)t0 * rs + (size_t)head * FD + 4 * lane;
        const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int j = 0; j < FE_TC; ++j) {
            const float4 x0 = Vec4<IO>::widen(
                *reinterpret_cast<const typename Vec4<IO>::Raw*>(rp + (j + 3) * FE_ROWB));
            float4 a3 = x3, a2 = x2, a1 = x1;
            if (!one_seq) {  // taps before the start of token t's sequence are zero
                const int t = t0 + j, s = __shfl_sync(0xffffffffu, s_mine, j);
                a3 = (t - 3 >= s) ? a3 : z;
                a2 = (t - 2 >= s) ? a2 : z;
                a1 = (t - 1 >= s) ? a1 : z;
            }
            float4 v = act4(conv4(w, a3, a2, a1, x0), ACT);
            if (kind < 2) v = l2norm_row(v, p.eps);
            if (t0 + j < t1) Vec4<IO>::store(yt, v);
            yt += rs;
            x3 = x2;
            x2 = x1;
            x1 = x0;
        }
    }
    if (gate) {
        p.log_alpha[(size_t)tg * p.H_v + head] = -softplus(ga);
        p.beta[(size_t)tg * p.H_v + head] = sigmoidf(gb);
    }
}

template <typename IO, int ACT>
cudaError_t launch_frontend_t(const FrontendParams& prm, int T, int H_qk, int H_v,
                              cudaStream_t stream) {
    constexpr int HG = fe_heads<IO>();
    const cudaError_t attr = cudaFuncSetAttribute(
        frontend_kernel<IO, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, FE_SMEM);
    if (attr != cudaSuccess) return attr;
    const long long groups = 2LL * ((H_qk + HG - 1) / HG) + (H_v + HG - 1) / HG;
    const long long blocks = ((long long)T + FE_TC - 1) / FE_TC * groups;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    frontend_kernel<IO, ACT><<<(unsigned)blocks, HG * 32, FE_SMEM, stream>>>(prm);
    return cudaGetLastError();
}

// Grid (B, 2 H_qk + H_v), one warp: one decode step of one head of one sequence.
// state [B, 3, C] (io dtype) holds the last three raw input rows, oldest first;
// it is shifted in place.
template <typename IO>
__global__ void __launch_bounds__(32)
    frontend_decode_kernel(const FrontendParams p, IO* state, int C) {
    const int lane = threadIdx.x;
    const int bi = blockIdx.x, hid = blockIdx.y;
    const int kind = hid < p.H_qk ? 0 : (hid < 2 * p.H_qk ? 1 : 2);
    const int head = kind == 0 ? hid : (kind == 1 ? hid - p.H_qk : hid - 2 * p.H_qk);
    const int H = kind == 2 ? p.H_v : p.H_qk;
    const size_t off = ((size_t)bi * H + head) * FD + 4 * lane;
    float4 w[4];
    {
        const float4* wp = reinterpret_cast<const float4*>(p.w + ((size_t)hid * FD + 4 * lane) * 4);
        const float4 c0 = wp[0], c1 = wp[1], c2 = wp[2], c3 = wp[3];
        w[0] = make_float4(c0.x, c1.x, c2.x, c3.x);
        w[1] = make_float4(c0.y, c1.y, c2.y, c3.y);
        w[2] = make_float4(c0.z, c1.z, c2.z, c3.z);
        w[3] = make_float4(c0.w, c1.w, c2.w, c3.w);
    }
    IO* sp = state + (size_t)bi * 3 * C + (size_t)hid * FD + 4 * lane;
    const float4 x3 = Vec4<IO>::load(sp), x2 = Vec4<IO>::load(sp + C),
                 x1 = Vec4<IO>::load(sp + 2 * C);
    const void* xk = kind == 0 ? p.x[0] : (kind == 1 ? p.x[1] : p.x[2]);
    void* yk = kind == 0 ? p.y[0] : (kind == 1 ? p.y[1] : p.y[2]);
    const float4 x0 = Vec4<IO>::load(static_cast<const IO*>(xk) + off);
    float4 v = act4(conv4(w, x3, x2, x1, x0), p.act);
    if (kind < 2) v = l2norm_row(v, p.eps);
    Vec4<IO>::store(static_cast<IO*>(yk) + off, v);
    // the raw rows are stored as given (exact in the io dtype)
    Vec4<IO>::store(sp, x2);
    Vec4<IO>::store(sp + C, x1);
    Vec4<IO>::store(sp + 2 * C, x0);
    if (kind == 2 && lane < 2) {
        const size_t gi = (size_t)bi * p.H_v + head;
        if (lane == 0) p.log_alpha[gi] = -softplus(p.a[gi]);
        else p.beta[gi] = sigmoidf(p.b[gi]);
    }
}

// ---- gradients of the front end ----
//
// With y the convolution, u = act(y) and r = 1 / sqrt(sum u^2 + eps) of a q or k head:
//   du = r (dq - u r^2 <u, dq>)  (v: du = dv),   dy = du act'(y),
//   dx[s] = sum_i w_i dy[s + 3 - i],   dw_i = sum_t dy[t] x[t - 3 + i].
//
// HBM-bound: raw rows and output gradients read once, raw gradients written once.
// One warp walks a run of consecutive tokens of its channels: a rolling window of three raw
// rows feeds the convolution, three partial rows of dx wait for the tokens ahead of them,
// and dw runs in registers.  Runs overlap by the three rows behind and ahead of them.
//
// Every warp keeps three tiles of rows (x and the output gradient) on their way by TMA into its
// own part of shared memory; within a tile nothing but the window joins the rows, so their
// latencies overlap.  The arithmetic goes two channels to an instruction.  A warp holds a whole
// head, for the sums over a head of q or k and because rows of 256 bytes keep the memory busy
// (with rows of 128 bytes v's part took 246 us instead of 210 us even with its arithmetic left
// out).  12 warps an SM at 168 registers: with 128 registers and 16 warps the spills cost more
// than the warps bring (32,768 tokens of 16/48 bf16 heads: 428 us against 395 us).
constexpr int FG_BLOCKS = 12;                   // blocks (of one warp) per SM: all runs at once
constexpr int FG_STAGES = 4;                    // of a ring (a power of two), three on their way
constexpr int FG_HALF = 8 * FD * 2;             // bytes of a stage's rows of x: 8 of bf16, 4 of fp32
constexpr int FG_RING = FG_STAGES * 2 * FG_HALF;  // bytes of a warp's ring
constexpr int FG_SMEM = FG_RING + FG_STAGES * 8 + 16;

// Runs of a kind of head: `runs` of `len` tokens each, and their partial sums of dw
// [runs, the kind's channels, 4].
struct GradRuns {
    int runs, len;
    float* part;
};
struct FrontendGradParams {
    FrontendGradArgs a;
    GradRuns qk, v;
};
struct FrontendGradMaps {
    CUtensorMap x[3], dout[3];
};

// A lane's channels: 2 P neighbours.
constexpr int P = 2;
struct Chans {
    float2 c[P];
};
__device__ __forceinline__ Chans zeros() {
    Chans r;
#pragma unroll
    for (int i = 0; i < P; ++i) r.c[i] = both(0.f);
    return r;
}
__device__ __forceinline__ Chans fma_c(const Chans& a, const Chans& b, const Chans& c) {
    Chans r;
#pragma unroll
    for (int i = 0; i < P; ++i) r.c[i] = fma2(a.c[i], b.c[i], c.c[i]);
    return r;
}
__device__ __forceinline__ Chans mul_c(const Chans& a, const Chans& b) {
    Chans r;
#pragma unroll
    for (int i = 0; i < P; ++i) r.c[i] = mul2(a.c[i], b.c[i]);
    return r;
}
__device__ __forceinline__ float dot_c(const Chans& a, const Chans& b) {
    float2 s = mul2(a.c[0], b.c[0]);
#pragma unroll
    for (int i = 1; i < P; ++i) s = fma2(a.c[i], b.c[i], s);
    return s.x + s.y;
}
__device__ __forceinline__ Chans load_c(const __nv_bfloat16* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const uint32_t u[P] = {v.x, v.y};
    Chans r;
#pragma unroll
    for (int i = 0; i < P; ++i)
        r.c[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    return r;
}
__device__ __forceinline__ Chans load_c(const float* p) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    Chans r;
    r.c[0] = make_float2(v.x, v.y), r.c[1] = make_float2(v.z, v.w);
    return r;
}
__device__ __forceinline__ void store_c(__nv_bfloat16* p, const Chans& v) {
    *reinterpret_cast<uint2*>(p) =
        make_uint2(pack_bf16x2(v.c[0].x, v.c[0].y), pack_bf16x2(v.c[1].x, v.c[1].y));
}
__device__ __forceinline__ void store_c(float* p, const Chans& v) {
    *reinterpret_cast<float4*>(p) = make_float4(v.c[0].x, v.c[0].y, v.c[1].x, v.c[1].y);
}

// What a warp carries from row to row.
struct GradState {
    Chans w[4], dw[4];
    Chans x1, x2, x3;  // raw rows t - 1, t - 2, t - 3 (zeros before the sequence)
    Chans d1, d2, d3;  // dx of tokens t - 1, t - 2, t - 3 so far
    int lo;               // the first token whose dx is pending or stored here
};

// Rows t .. t + NR - 1 of one sequence: x and dout at xs, gs (rows `pitch` elements apart);
// dx of tokens t - 3 .. t + NR - 4 is complete after it and stored.  ALL: every one of them
// belongs to the run.
template <int NR, bool L2, bool SILU, bool DW, bool ALL, typename IO>
__device__ __forceinline__ void grad_rows(GradState& s, int t, const IO* xs, const IO* gs,
                                          int64_t pitch, IO* dx, int64_t rs, float eps) {
    Chans x[NR + 3], u[NR], slope[NR], dy[NR];
    x[0] = s.x3, x[1] = s.x2, x[2] = s.x1;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        x[i + 3] = load_c(xs + i * pitch);
        dy[i] = load_c(gs + i * pitch);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        const Chans y = fma_c(
            s.w[0], x[i],
            fma_c(s.w[1], x[i + 1], fma_c(s.w[2], x[i + 2], mul_c(s.w[3], x[i + 3]))));
        u[i] = y;
        if (SILU) {
#pragma unroll
            for (int c = 0; c < P; ++c) {
                const float2 g = sigmoid2(y.c[c]);
                u[i].c[c] = mul2(y.c[c], g);
                slope[i].c[c] = fma2(u[i].c[c], fma2(g, both(-1.f), both(1.f)), g);
            }
        }
    }
    if (L2) {
        float2 su[NR];  // <u, u> and <u, dout>
#pragma unroll
        for (int i = 0; i < NR; ++i) su[i] = make_float2(dot_c(u[i], u[i]), dot_c(u[i], dy[i]));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < NR; ++i)
                su[i] = add2(su[i], make_float2(__shfl_xor_sync(0xffffffffu, su[i].x, o),
                                                __shfl_xor_sync(0xffffffffu, su[i].y, o)));
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const float r = rsqrtf(su[i].x + eps);
            // (r^3 alone leaves fp32 for rows far from unit size; r <u, dout> does not)
            const float2 r2 = both(r), k = both(-r * (r * (r * su[i].y)));
#pragma unroll
            for (int c = 0; c < P; ++c) dy[i].c[c] = fma2(u[i].c[c], k, mul2(r2, dy[i].c[c]));
        }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        if (SILU) dy[i] = mul_c(dy[i], slope[i]);
        if (DW)
#pragma unroll
            for (int k = 0; k < 4; ++k) s.dw[k] = fma_c(dy[i], x[i + k], s.dw[k]);
        const Chans done = fma_c(s.w[0], dy[i], s.d3);
        if (ALL || t + i - 3 >= s.lo) store_c(dx + (t + i - 3) * rs, done);
        s.d3 = fma_c(s.w[1], dy[i], s.d2);
        s.d2 = fma_c(s.w[2], dy[i], s.d1);
        s.d1 = mul_c(s.w[3], dy[i]);
    }
    s.x3 = x[NR], s.x2 = x[NR + 1], s.x1 = x[NR + 2];
}

// Nothing follows token t - 1 in its sequence or run: what waits is complete.
template <typename IO>
__device__ __forceinline__ void grad_flush(const GradState& s, int t, int tb, IO* dx, int64_t rs) {
    if (t - 3 >= s.lo && t - 3 < tb) store_c(dx + (t - 3) * rs, s.d3);
    if (t - 2 >= s.lo && t - 2 < tb) store_c(dx + (t - 2) * rs, s.d2);
    if (t - 1 >= s.lo && t - 1 < tb) store_c(dx + (t - 1) * rs, s.d1);
}

template <typename IO, bool SILU, bool L2>
__device__ __forceinline__ void grad_run(const FrontendGradArgs& a, GradState& s,
                                         const IO* x, const IO* go, IO* dx, int64_t rs, int ta,
                                         int tb, int T_end, const CUtensorMap* mx,
                                         const CUtensorMap* mg, int c0, uint8_t* ring,
                                         uint64_t* full, volatile int* abort_flag) {
    constexpr int ROWS = FG_HALF / (FD * (int)sizeof(IO)), STAGES = FG_STAGES;
    const int lane = threadIdx.x & 31;
    // (the three tokens ahead of the run's last are read too, for the run's dx alone)
    const int te = min(tb + 3, T_end), tiles = (te - ta + ROWS - 1) / ROWS;
    const auto fetch = [&](int i) {
        if (i >= tiles || lane != 0) return;
        uint8_t* d = ring + (i & (STAGES - 1)) * (2 * FG_HALF);
        uint64_t* bar = &full[i & (STAGES - 1)];
        mbar_arrive_expect_tx(bar, 2 * FG_HALF);
        tma_load_2d(d, mx, c0, ta + i * ROWS, bar);
        tma_load_2d(d + FG_HALF, mg, c0, ta + i * ROWS, bar);
    };
    for (int i = 0; i < STAGES - 1; ++i) fetch(i);

    // the sequence of token ta, and where the next one starts
    int n = 0, first = 0, next = T_end;
    if (a.cu_seqlens) {
        int hi = a.N - 1;
        while (n < hi) {
            const int mid = (n + hi + 1) >> 1;
            if (a.cu_seqlens[mid] <= ta) n = mid; else hi = mid - 1;
        }
        first = max(a.cu_seqlens[n], 0);
        next = a.cu_seqlens[n + 1];
    }
    s.x1 = ta - 1 >= first ? load_c(x + (ta - 1) * rs) : zeros();
    s.x2 = ta - 2 >= first ? load_c(x + (ta - 2) * rs) : zeros();
    s.x3 = ta - 3 >= first ? load_c(x + (ta - 3) * rs) : zeros();
    s.d1 = s.d2 = s.d3 = zeros();
    s.lo = max(first, ta);
    const auto start = [&](int t) {  // a sequence starts at token t
        grad_flush(s, t, tb, dx, rs);
        s.x1 = s.x2 = s.x3 = s.d1 = s.d2 = s.d3 = zeros();
        s.lo = t;
        do {
            ++n;
        } while (n + 1 < a.N && a.cu_seqlens[n + 1] <= t);
        next = a.cu_seqlens[n + 1];
    };

    for (int i = 0; i < tiles; ++i) {
        // (the lanes give up together: those that went on would wait for the others in a shuffle)
        if (!__all_sync(0xffffffffu,
                        mbar_wait(&full[i & (STAGES - 1)], (i / STAGES) & 1, abort_flag))) {
            // the copies may still land: wait for them (bounded) before the block ends
            const unsigned long long ts = globaltimer();
            for (int k = i; k < min(i + STAGES - 1, tiles); ++k)
                while (!mbar_try_wait(smem_u32(&full[k & (STAGES - 1)]), (k / STAGES) & 1) &&
                       globaltimer() - ts < kWaitLimitNs) {
                }
            return;
        }
        const IO* xs =
            reinterpret_cast<const IO*>(ring + (i & (STAGES - 1)) * (2 * FG_HALF)) + 2 * P * lane;
        const IO* gs = xs + ROWS * FD;
        const int t0 = ta + i * ROWS;
        if (t0 == next) start(t0);
        if (t0 + ROWS <= tb && next >= t0 + ROWS) {
            // a whole tile within the run and the sequence, as almost all are
            constexpr int NR = 4;
            if (t0 - 3 >= s.lo) {
#pragma unroll
                for (int r = 0; r < ROWS; r += NR)
                    grad_rows<NR, L2, SILU, true, true>(s, t0 + r, xs + r * FD, gs + r * FD,
                                                        FD, dx, rs, a.eps);
            } else {  // the first one
#pragma unroll
                for (int r = 0; r < ROWS; r += NR)
                    grad_rows<NR, L2, SILU, true, false>(s, t0 + r, xs + r * FD, gs + r * FD,
                                                         FD, dx, rs, a.eps);
            }
        } else {
#pragma unroll 1
            for (int r = 0; r < ROWS && t0 + r < te; ++r) {
                const int t = t0 + r;
                if (t == next) start(t);
                if (t < tb)
                    grad_rows<1, L2, SILU, true, false>(s, t, xs + r * FD, gs + r * FD, FD,
                                                        dx, rs, a.eps);
                else if (s.lo < tb)
                    grad_rows<1, L2, SILU, false, false>(s, t, xs + r * FD, gs + r * FD, FD,
                                                         dx, rs, a.eps);
            }
        }
        // Into the place of the tile before this one: everything read from that has gone into
        // the rows stored since (this one's last rows still wait in registers), and each lane
        // orders its reads before the copy, which comes through another proxy.
        fence_proxy_async_smem();
        __syncwarp();
        fetch(i + STAGES - 1);
    }
    grad_flush(s, te, tb, dx, rs);
}

template <typename IO, int ACT>
__global__ void __launch_bounds__(32, FG_BLOCKS)
    frontend_grad_kernel(const __grid_constant__ FrontendGradMaps maps, const FrontendGradParams p) {
    const FrontendGradArgs& a = p.a;
    const int T_end = a.cu_seqlens ? min(max(a.cu_seqlens[a.N], 0), a.T) : a.T;
    extern __shared__ __align__(128) uint8_t fg_sm[];
    allow_next_step();
    const int lane = threadIdx.x;
    uint8_t* ring = fg_sm;
    uint64_t* full = reinterpret_cast<uint64_t*>(fg_sm + FG_RING);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(fg_sm + FG_RING + FG_STAGES * 8);
    if (lane == 0) {
        *abort_flag = 0;
        for (int i = 0; i < FG_STAGES; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncwarp();
    // unit: a run of a head, those of q and k first
    const int units_qk = p.qk.runs * 2 * a.H_qk;
    const int unit = blockIdx.x;
    const bool is_v = unit >= units_qk;
    const GradRuns& runs = is_v ? p.v : p.qk;
    const int heads = is_v ? a.H_v : 2 * a.H_qk;
    const int run = (is_v ? unit - units_qk : unit) / heads;
    const int head = (is_v ? unit - units_qk : unit) - run * heads;  // among the kind's
    const int hid = is_v ? 2 * a.H_qk + head : head;
    const int kind = hid < a.H_qk ? 0 : (hid < 2 * a.H_qk ? 1 : 2);  // q, k, v
    const int c0 = (hid - (kind == 0 ? 0 : (kind == 1 ? a.H_qk : 2 * a.H_qk))) * FD;
    const int64_t rs = (int64_t)(kind == 2 ? a.H_v : a.H_qk) * FD;
    const int64_t off = c0 + 4 * lane;
    const IO* x = static_cast<const IO*>(kind == 0 ? a.x[0] : (kind == 1 ? a.x[1] : a.x[2])) + off;
    const IO* go =
        static_cast<const IO*>(kind == 0 ? a.dout[0] : (kind == 1 ? a.dout[1] : a.dout[2])) + off;
    IO* dx = static_cast<IO*>(kind == 0 ? a.dx[0] : (kind == 1 ? a.dx[1] : a.dx[2])) + off;
    const int64_t wc = (int64_t)hid * FD + 4 * lane;  // the lane's channel of the weight

    GradState s;
    // the lane's channels x 4 taps, channel-major -> the taps' pairs of channels
    const float4* wp = reinterpret_cast<const float4*>(a.w) + wc;
#pragma unroll
    for (int c = 0; c < P; ++c) {
        const float4 u = wp[2 * c], v = wp[2 * c + 1];
        s.w[0].c[c] = make_float2(u.x, v.x);
        s.w[1].c[c] = make_float2(u.y, v.y);
        s.w[2].c[c] = make_float2(u.z, v.z);
        s.w[3].c[c] = make_float2(u.w, v.w);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) s.dw[k] = zeros();
    const int64_t first = (int64_t)run * runs.len;
    const int ta = (int)min(first, (int64_t)T_end), tb = (int)min(first + runs.len, (int64_t)T_end);
    if (ta < tb) {
        if (kind == 2)
            grad_run<IO, ACT == GDN_ACT_SILU, false>(a, s, x, go, dx, rs, ta, tb, T_end, &maps.x[2],
                                                     &maps.dout[2], c0, ring, full, abort_flag);
        else
            grad_run<IO, ACT == GDN_ACT_SILU, true>(
                a, s, x, go, dx, rs, ta, tb, T_end, kind == 0 ? &maps.x[0] : &maps.x[1],
                kind == 0 ? &maps.dout[0] : &maps.dout[1], c0, ring, full, abort_flag);
    }
    float4* o = reinterpret_cast<float4*>(runs.part) + ((int64_t)run * heads + head) * FD + 4 * lane;
#pragma unroll
    for (int c = 0; c < P; ++c) {
        o[2 * c] = make_float4(s.dw[0].c[c].x, s.dw[1].c[c].x, s.dw[2].c[c].x, s.dw[3].c[c].x);
        o[2 * c + 1] = make_float4(s.dw[0].c[c].y, s.dw[1].c[c].y, s.dw[2].c[c].y, s.dw[3].c[c].y);
    }
}

// The last step: the gates (blockIdx.y 0), which need nothing of the first and fill the SMs as
// its warps end (at the start of the blocks of v they took 45 us for 32,768 tokens of 48
// heads), and dw from the partial sums of q and k (1) and of v (2).
constexpr int FG_LAST = 256;
__global__ void __launch_bounds__(FG_LAST)
    frontend_grad_last_kernel(const FrontendGradArgs a, const ColumnSums qk, const ColumnSums v) {
    if (blockIdx.y > 0) {
        wait_for_first_step();
        column_sums<FG_LAST / 32>(blockIdx.y == 1 ? qk : v, blockIdx.x);
        return;
    }
    const int T_end = a.cu_seqlens ? min(max(a.cu_seqlens[a.N], 0), a.T) : a.T;
    const int64_t n = (int64_t)T_end * a.H_v, all = (int64_t)gridDim.x * FG_LAST;
    for (int64_t i = (int64_t)blockIdx.x * FG_LAST + threadIdx.x; i < n; i += 4 * all) {
        float va[4], vb[4], ga[4], gb[4];  // (all loads before the first store)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t j = i + k * all < n ? i + k * all : i;
            va[k] = a.a[j], vb[k] = a.b[j], ga[k] = a.dlog_alpha[j], gb[k] = a.dbeta[j];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t j = i + k * all;
            const float be = sigmoidf(vb[k]);
            if (j < n) {
                a.da[j] = -sigmoidf(va[k]) * ga[k];
                a.db[j] = be * (1.f - be) * gb[k];
            }
        }
    }
}

// Runs per head: all warps at once, runs of at least 32 tokens, whole tiles of rows; 1.3 to
// 1.4 times as many for q and k as for v, whose rows take less arithmetic (with as many for each
// the last warps of q and k ran alone: 485 us against 420 us for 32,768 tokens of 16/48 bf16
// heads).
void frontend_grad_runs(int T, int H_qk, int H_v, GradRuns& qk, GradRuns& v) {
    const long long warps = (long long)known_sms() * FG_BLOCKS;
    const auto cut = [T](long long runs) {
        const long long most = ((long long)T + 31) / 32;
        if (runs > most) runs = most;
        if (runs < 1) runs = 1;
        long long len = (T + runs - 1) / runs;
        len = (len + 7) / 8 * 8;
        return GradRuns{(int)((T + len - 1) / len), (int)len, nullptr};
    };
    v = cut(warps / (26ll * H_qk / 10 + H_v));
    qk = cut((warps - v.runs * (long long)H_v) / (2ll * H_qk));
}

template <typename IO, int ACT>
cudaError_t launch_frontend_grad(const FrontendGradParams& p, cudaStream_t stream) {
    const FrontendGradArgs& a = p.a;
    FrontendGradMaps maps{};
    constexpr int rows = FG_HALF / (FD * (int)sizeof(IO));
    for (int k = 0; k < 3; ++k) {
        const int64_t C = (int64_t)(k == 2 ? a.H_v : a.H_qk) * FD;
        if (!tile_map(&maps.x[k], a.x[k], a.bf16, a.T, C, C, FD, rows) ||
            !tile_map(&maps.dout[k], a.dout[k], a.bf16, a.T, C, C, FD, rows))
            return cudaErrorInvalidValue;
    }
    const auto kernel = frontend_grad_kernel<IO, ACT>;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FG_SMEM);
    if (e != cudaSuccess) return e;
    const long long units = (long long)p.qk.runs * 2 * a.H_qk + (long long)p.v.runs * a.H_v;
    if (units > 0x7fff0000LL) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)units, 32, FG_SMEM, stream>>>(maps, p);
    return cudaGetLastError();
}

}  // namespace

size_t frontend_backward_workspace_bytes(int T, int H_qk, int H_v) {
    if (T == 0) return 0;
    GradRuns qk, v;
    frontend_grad_runs(T, H_qk, H_v, qk, v);
    return ((size_t)qk.runs * 2 * H_qk + (size_t)v.runs * H_v) * FD * 4 * sizeof(float);
}

cudaError_t launch_frontend_backward(const FrontendGradArgs& a, void* workspace,
                                     cudaStream_t stream) {
    const int cq = 2 * a.H_qk * FD * 4, cv = a.H_v * FD * 4;
    FrontendGradParams p{};
    p.a = a;
    if (a.T > 0) {
        frontend_grad_runs(a.T, a.H_qk, a.H_v, p.qk, p.v);
        p.qk.part = static_cast<float*>(workspace);
        p.v.part = p.qk.part + (size_t)p.qk.runs * cq;
        const cudaError_t e =
            a.bf16 ? (a.silu ? launch_frontend_grad<__nv_bfloat16, GDN_ACT_SILU>(p, stream)
                             : launch_frontend_grad<__nv_bfloat16, GDN_ACT_NONE>(p, stream))
                   : (a.silu ? launch_frontend_grad<float, GDN_ACT_SILU>(p, stream)
                             : launch_frontend_grad<float, GDN_ACT_NONE>(p, stream));
        if (e != cudaSuccess) return e;
    }
    const int blocks = ((cq > cv ? cq : cv) + 31) / 32;
    return launch_second_step(frontend_grad_last_kernel, dim3(blocks, 3), FG_LAST, stream, a,
                              ColumnSums{p.qk.part, a.dw, p.qk.runs, cq},
                              ColumnSums{p.v.part, a.dw + cq, p.v.runs, cv});
}

cudaError_t launch_frontend(const void* q_raw, const void* k_raw, const void* v_raw,
                            const float* conv_w, const float* a, const float* b,
                            const int32_t* cu_seqlens, int N, int T, int H_qk, int H_v,
                            bool bf16, int act, float eps, void* q, void* k, void* v,
                            float* log_alpha, float* beta, cudaStream_t stream) {
    if (T == 0) return cudaSuccess;
    FrontendParams prm{{q_raw, k_raw, v_raw}, {q, k, v}, conv_w, a, b, log_alpha, beta,
                       cu_seqlens, N, T, H_qk, H_v, act, eps};
    if (bf16)
        return act == GDN_ACT_SILU
                   ? launch_frontend_t<__nv_bfloat16, GDN_ACT_SILU>(prm, T, H_qk, H_v, stream)
                   : launch_frontend_t<__nv_bfloat16, GDN_ACT_NONE>(prm, T, H_qk, H_v, stream);
    return act == GDN_ACT_SILU ? launch_frontend_t<float, GDN_ACT_SILU>(prm, T, H_qk, H_v, stream)
                               : launch_frontend_t<float, GDN_ACT_NONE>(prm, T, H_qk, H_v, stream);
}

cudaError_t launch_frontend_decode(const void* q_raw, const void* k_raw, const void* v_raw,
                                   const float* conv_w, const float* a, const float* b,
                                   void* conv_state, int B, int H_qk, int H_v, bool bf16, int act,
                                   float eps, void* q, void* k, void* v, float* log_alpha,
                                   float* beta, cudaStream_t stream) {
    if (B == 0) return cudaSuccess;
    FrontendParams prm{{q_raw, k_raw, v_raw}, {q, k, v}, conv_w, a, b, log_alpha, beta,
                       nullptr, 0, 0, H_qk, H_v, act, eps};
    const int C = (2 * H_qk + H_v) * FD;
    dim3 grid(B, 2 * H_qk + H_v);
    if (bf16)
        frontend_decode_kernel<__nv_bfloat16><<<grid, 32, 0, stream>>>(
            prm, static_cast<__nv_bfloat16*>(conv_state), C);
    else
        frontend_decode_kernel<float><<<grid, 32, 0, stream>>>(prm, static_cast<float*>(conv_state),
                                                               C);
    return cudaGetLastError();
}

}  // namespace gdn
