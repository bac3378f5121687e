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
// sums of dw and db run in registers over all its tokens; the next token's
// channels are on their way while one is computed.  The arithmetic goes two
// channels to an instruction: at one each, the gradients' ~35 instructions per
// channel take as long as their 10 bytes.
#include <cuda_bf16.h>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_internal.h"
#include "gdn_sums.cuh"

namespace gdn {

namespace {

constexpr int NT = 256;        // threads per block
// Blocks per SM that the grids are sized for, so that all run at once: as many as the
// registers allow without spills in the loop.  (The gradients with bias or mean and bf16's
// eight channels a lane need 128: at three blocks 516 us, at two 379 us, for 32,768 x 48 x 128.
// The others took 332 us at three and 371 us at two.  Forward, with a gate: 201 us at four
// and 295 us at five; without gate, mean and bias: 152 us and 143 us.)
constexpr int fwd_blocks(bool gated, bool plain) { return !gated && plain ? 5 : 4; }
constexpr int bwd_blocks(bool plain, bool bf16_wide) { return !plain && bf16_wide ? 2 : 3; }
// Tokens that a lane group of the gradients walks over at least: its partial sums (fp32, one
// row per stream for weights per head) cost as much traffic as two to four tokens.
constexpr int BWD_TOKENS = 4;

struct NormParams {
    const void *x, *z, *dy;
    void *y, *dz;            // y: the output, or dx
    const float *w, *b;
    float *dw_part, *db_part;
    int64_t xs, zs, dys, ys, dzs;  // row strides in elements
    int T, H, d, streams;
    bool per_head, centred, silu, has_bias;
    float eps, inv_d;
};

// How a lane reads and writes its channels, by what the alignment allows: 16 bytes at once, a
// pair of bf16 (4 bytes; 32,768 x 16 x 258 centred with bias: 192 us against 476 us one by one),
// or one by one.
enum Access { WIDE, PAIR, SINGLE };

// The channels of a group that a lane holds, in NV vectors of NP pairs.  WIDE: channels
// (lane + LG j) VE .. + VE - 1 of vector j.  Else one pair each: neighbours 2 (lane + LG j) and
// one further (PAIR), or lane + 2 LG j and LG further, so that single accesses stay coalesced.
template <typename IO, Access A, int LG>
struct Vec {
    static constexpr int VE = A == WIDE ? 16 / (int)sizeof(IO) : 2;
    static constexpr int NP = VE / 2;
    static constexpr int STEP = A == SINGLE ? LG : 1;  // from a pair's first channel to its second
    static constexpr bool PACKED = A != SINGLE && sizeof(IO) == 2;  // bf16 pairs, as stored
    struct Raw {
        uint32_t u[A == WIDE ? 4 : 2];
    };
    static __device__ __forceinline__ int channel(int lane, int j, int i) {
        return A == SINGLE ? lane + 2 * LG * j : (lane + LG * j) * VE + 2 * i;
    }
    // p: the group's first channel
    static __device__ __forceinline__ Raw load(const IO* p, int lane, int j, int d, bool ok) {
        Raw r;
        const int c = channel(lane, j, 0);
        if constexpr (A == WIDE) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u);
            if (ok && c < d) u = *reinterpret_cast<const uint4*>(p + c);
            r.u[0] = u.x, r.u[1] = u.y, r.u[2] = u.z, r.u[3] = u.w;
        } else if constexpr (A == PAIR) {  // (d is even)
            r.u[0] = ok && c < d ? *reinterpret_cast<const uint32_t*>(p + c) : 0u;
        } else {
            const float a = ok && c < d ? (float)p[c] : 0.f;
            const float b = ok && c + STEP < d ? (float)p[c + STEP] : 0.f;
            r.u[0] = __float_as_uint(a), r.u[1] = __float_as_uint(b);
        }
        return r;
    }
    static __device__ __forceinline__ float2 pair(const Raw& r, int i) {
        if constexpr (PACKED)
            return make_float2(__uint_as_float(r.u[i] << 16), __uint_as_float(r.u[i] & 0xffff0000u));
        else
            return make_float2(__uint_as_float(r.u[2 * i]), __uint_as_float(r.u[2 * i + 1]));
    }
    // (streaming: 32,768 x 48 x 128 gated forward 195 us against 207 us, passes back to back)
    static __device__ __forceinline__ void store(IO* p, int lane, int j, int d, bool ok,
                                                 const float2 (&v)[NP]) {
        const int c = channel(lane, j, 0);
        if constexpr (A == WIDE && sizeof(IO) == 2) {
            if (ok && c < d)
                __stcs(reinterpret_cast<uint4*>(p + c),
                       make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y),
                                  pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y)));
        } else if constexpr (A == WIDE) {
            if (ok && c < d)
                __stcs(reinterpret_cast<float4*>(p + c),
                       make_float4(v[0].x, v[0].y, v[1].x, v[1].y));
        } else if constexpr (A == PAIR) {
            if (ok && c < d) *reinterpret_cast<uint32_t*>(p + c) = pack_bf16x2(v[0].x, v[0].y);
        } else {
            if (ok && c < d) p[c] = (IO)v[0].x;
            if (ok && c + STEP < d) p[c + STEP] = (IO)v[0].y;
        }
    }
    static __device__ __forceinline__ float2 weight(const float* w, int lane, int j, int i, int d) {
        const int c = channel(lane, j, i);
        return make_float2(c < d ? w[c] : 0.f, c + STEP < d ? w[c + STEP] : 0.f);
    }
    static __device__ __forceinline__ void put_weight(float* w, int lane, int j, int i, int d,
                                                      float2 v) {
        const int c = channel(lane, j, i);
        if (c < d) w[c] = v.x;
        if (c + STEP < d) w[c + STEP] = v.y;
    }
    // zero what lies outside the group
    static __device__ __forceinline__ float2 inside(float2 v, int lane, int j, int i, int d) {
        const int c = channel(lane, j, i);
        return make_float2(c < d ? v.x : 0.f, c + STEP < d ? v.y : 0.f);
    }
};

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
    int64_t row, group;
    bool active;
    __device__ __forceinline__ explicit Place(const NormParams& p) {
        constexpr int GPB = NT / LG;
        lane = threadIdx.x % LG;
        group = (int64_t)blockIdx.x * GPB + threadIdx.x / LG;
        active = group < (int64_t)p.streams * p.H;
        head = (int)(group % p.H);
        row = group / p.H;
        // the whole warp makes the trips of its first lane group, which has the most
        const int64_t g0 = (int64_t)blockIdx.x * GPB + (threadIdx.x & ~31) / LG;
        const int64_t row0 = g0 / p.H;
        trips = row0 < p.T && g0 < (int64_t)p.streams * p.H
                    ? (int)((p.T - row0 + p.streams - 1) / p.streams)
                    : 0;
    }
};

// xh and 1 / sqrt(...) of one group, from its channels in v (zeros outside it).
template <typename V, int LG, int NV>
__device__ __forceinline__ float normalise(float2 (&v)[NV][V::NP], int lane, int d, bool centred,
                                           float inv_d, float eps) {
    if (centred) {
        float2 s = both(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V::NP; ++i) s = add2(s, v[j][i]);
        const float2 m = both(-group_sum<LG>(s.x + s.y) * inv_d);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V::NP; ++i)
                v[j][i] = V::inside(add2(v[j][i], m), lane, j, i, d);
    }
    float2 ss = both(0.f);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V::NP; ++i) ss = fma2(v[j][i], v[j][i], ss);
    const float r = rsqrtf(fmaf(group_sum<LG>(ss.x + ss.y), inv_d, eps));
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V::NP; ++i) v[j][i] = mul2(v[j][i], both(r));
    return r;
}

// PLAIN: RMS without bias, the common form; it saves the bias's registers (built for the wide
// access alone).
template <typename IO, Access A, int LG, int NV, bool GATED, bool PLAIN>
__global__ void __launch_bounds__(NT, NV == 1 ? fwd_blocks(GATED, PLAIN) : 1)
    group_norm_kernel(const NormParams p) {
    using V = Vec<IO, A, LG>;
    const Place<LG> at(p);
    const int lane = at.lane, d = p.d;
    float2 w[NV][V::NP], b[NV][V::NP];
    const int wo = p.per_head ? at.head * d : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V::NP; ++i) {
            w[j][i] = V::weight(p.w + wo, lane, j, i, d);
            b[j][i] = !PLAIN && p.has_bias ? V::weight(p.b + wo, lane, j, i, d) : both(0.f);
        }
    const int64_t col = (int64_t)at.head * d;
    const IO* px = static_cast<const IO*>(p.x) + at.row * p.xs + col;
    const IO* pz = GATED ? static_cast<const IO*>(p.z) + at.row * p.zs + col : nullptr;
    IO* py = static_cast<IO*>(p.y) + at.row * p.ys + col;
    const int64_t sx = p.streams * p.xs, sz = p.streams * p.zs, sy = p.streams * p.ys;
    int64_t row = at.row;
    typename V::Raw xr[NV], zr[NV];
    const auto fetch = [&](bool ok) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            xr[j] = V::load(px, lane, j, d, ok);
            if (GATED) zr[j] = V::load(pz, lane, j, d, ok);
        }
        px += sx;
        if (GATED) pz += sz;
    };
    fetch(at.active && row < p.T);
    for (int it = 0; it < at.trips; ++it, row += p.streams, py += sy) {
        const bool ok = at.active && row < p.T;
        float2 v[NV][V::NP], g[NV][V::NP];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V::NP; ++i) {
                v[j][i] = V::pair(xr[j], i);
                if (GATED) g[j][i] = V::pair(zr[j], i);
            }
        fetch(at.active && row + p.streams < p.T);
        normalise<V, LG, NV>(v, lane, d, !PLAIN && p.centred, p.inv_d, ok ? p.eps : 1.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < V::NP; ++i) {
                const float2 n = PLAIN ? mul2(v[j][i], w[j][i]) : fma2(v[j][i], w[j][i], b[j][i]);
                float2 a = GATED ? g[j][i] : n;
                if (p.silu) a = mul2(a, sigmoid2(a));
                v[j][i] = GATED ? mul2(n, a) : a;
            }
            V::store(py, lane, j, d, ok, v[j]);
        }
    }
}

template <typename IO, Access A, int LG, int NV, bool GATED, bool PLAIN>
__global__ void __launch_bounds__(NT, NV == 1 ? bwd_blocks(PLAIN, A == WIDE && sizeof(IO) == 2) : 1)
    group_norm_backward_kernel(const NormParams p) {
    using V = Vec<IO, A, LG>;
    constexpr int GPB = NT / LG;
    extern __shared__ float part[];  // [GPB][d], for the sums over a block's groups
    allow_next_step();
    const Place<LG> at(p);
    const int lane = at.lane, d = p.d;
    float2 w[NV][V::NP], b[NV][V::NP], dw[NV][V::NP], db[NV][V::NP];
    const int wo = p.per_head ? at.head * d : 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < V::NP; ++i) {
            w[j][i] = V::weight(p.w + wo, lane, j, i, d);
            b[j][i] = !PLAIN && p.has_bias ? V::weight(p.b + wo, lane, j, i, d) : both(0.f);
            dw[j][i] = db[j][i] = both(0.f);
        }
    const int64_t col = (int64_t)at.head * d;
    const IO* px = static_cast<const IO*>(p.x) + at.row * p.xs + col;
    const IO* pd = static_cast<const IO*>(p.dy) + at.row * p.dys + col;
    const IO* pz = GATED ? static_cast<const IO*>(p.z) + at.row * p.zs + col : nullptr;
    IO* py = static_cast<IO*>(p.y) + at.row * p.ys + col;
    IO* pg = GATED ? static_cast<IO*>(p.dz) + at.row * p.dzs + col : nullptr;
    const int64_t sx = p.streams * p.xs, sd = p.streams * p.dys, sz = p.streams * p.zs;
    const int64_t sy = p.streams * p.ys, sg = p.streams * p.dzs;
    int64_t row = at.row;
    typename V::Raw xr[NV], dr[NV], zr[NV];
    const auto fetch = [&](bool ok) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            xr[j] = V::load(px, lane, j, d, ok);
            dr[j] = V::load(pd, lane, j, d, ok);
            if (GATED) zr[j] = V::load(pz, lane, j, d, ok);
        }
        px += sx;
        pd += sd;
        if (GATED) pz += sz;
    };
    fetch(at.active && row < p.T);
    for (int it = 0; it < at.trips; ++it, row += p.streams, py += sy) {
        const bool ok = at.active && row < p.T;
        float2 v[NV][V::NP], g[NV][V::NP], dn[NV][V::NP];
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int i = 0; i < V::NP; ++i) {
                v[j][i] = V::pair(xr[j], i);
                dn[j][i] = V::pair(dr[j], i);
                if (GATED) g[j][i] = V::pair(zr[j], i);
            }
        fetch(at.active && row + p.streams < p.T);
        // (a lane group past the last token adds exact zeros to its sums)
        const float r = normalise<V, LG, NV>(v, lane, d, !PLAIN && p.centred, p.inv_d,
                                             ok ? p.eps : 1.f);
        float2 se = both(0.f), sx2 = both(0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < V::NP; ++i) {
                const float2 n = PLAIN ? mul2(v[j][i], w[j][i]) : fma2(v[j][i], w[j][i], b[j][i]);
                const float2 a = GATED ? g[j][i] : n;
                float2 value = a, slope = both(1.f);
                if (p.silu) {
                    const float2 s = sigmoid2(a);
                    value = mul2(a, s);
                    slope = fma2(value, fma2(s, both(-1.f), both(1.f)), s);
                }
                const float2 dy = dn[j][i];
                if (GATED) {
                    g[j][i] = mul2(mul2(dy, n), slope);
                    dn[j][i] = mul2(dy, value);
                } else {
                    dn[j][i] = mul2(dy, slope);
                }
                dw[j][i] = fma2(dn[j][i], v[j][i], dw[j][i]);
                if (!PLAIN) db[j][i] = add2(db[j][i], dn[j][i]);
                dn[j][i] = mul2(dn[j][i], w[j][i]);
                if (!PLAIN) se = add2(se, dn[j][i]);
                sx2 = fma2(dn[j][i], v[j][i], sx2);
            }
            if (GATED) V::store(pg, lane, j, d, ok, g[j]);
        }
        const float2 cx = both(-group_sum<LG>(sx2.x + sx2.y) * p.inv_d);
        const float2 ce =
            both(!PLAIN && p.centred ? -group_sum<LG>(se.x + se.y) * p.inv_d : 0.f);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int i = 0; i < V::NP; ++i) {
                float2 e = fma2(v[j][i], cx, dn[j][i]);
                if (!PLAIN) e = add2(e, ce);
                v[j][i] = mul2(e, both(r));
            }
            V::store(py, lane, j, d, ok, v[j]);
        }
        if (GATED) pg += sg;
    }

    // partial sums: one row per stream of a head, or one row per block
#pragma unroll
    for (int which = 0; which < (PLAIN ? 1 : 2); ++which) {
        float* out = which ? p.db_part : p.dw_part;
        if (!out) continue;
        if (p.per_head) {
            if (at.active) {
                float* o = out + (at.group / p.H) * ((int64_t)p.H * d) + col;
#pragma unroll
                for (int j = 0; j < NV; ++j)
#pragma unroll
                    for (int i = 0; i < V::NP; ++i)
                        V::put_weight(o, lane, j, i, d, which ? db[j][i] : dw[j][i]);
            }
        } else {
            float* mine = part + (threadIdx.x / LG) * d;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
                for (int i = 0; i < V::NP; ++i)
                    V::put_weight(mine, lane, j, i, d, which ? db[j][i] : dw[j][i]);
            __syncthreads();
            for (int c = threadIdx.x; c < d; c += NT) {
                float s = 0.f;
                for (int q = 0; q < GPB; ++q) s += part[q * d + c];
                out[(int64_t)blockIdx.x * d + c] = s;
            }
        }
    }
}

// Column sums of up to two matrices (blockIdx.y).
template <int RT>
__global__ void __launch_bounds__(32 * RT) column_sums_kernel(const ColumnSums a, const ColumnSums b) {
    wait_for_first_step();
    column_sums<RT>(blockIdx.y ? b : a, blockIdx.x);
}

// Lanes of a group: a power of two that its vectors fill, 4 to 32.
int lanes_for(int nvec) {
    int lg = 4;
    while (lg < 32 && lg < nvec) lg *= 2;
    return lg;
}

// Blocks of a grid of lane groups, and the tokens walked side by side per head.
struct Shape {
    int lg, blocks, streams;
};
Shape shape_of(int T, int H, int d, bool wide, bool bf16, int blocks_per_sm, int tokens) {
    Shape s;
    s.lg = wide ? lanes_for(d / (bf16 ? 8 : 4)) : 32;
    const long long gpb = NT / s.lg, groups = (long long)T * H;
    const long long need = (groups + gpb * tokens - 1) / (gpb * tokens);
    const long long least = (H + gpb - 1) / gpb;
    long long blocks = (long long)known_sms() * blocks_per_sm;
    if (blocks > need) blocks = need;
    if (blocks < least) blocks = least;
    s.blocks = (int)blocks;
    s.streams = (int)(blocks * gpb / H);
    if (s.streams > T) s.streams = T;
    return s;
}

// How every pointer, stride and the group itself let the channels be accessed.
Access access_of(const NormParams& p, bool bf16) {
    const int ve = bf16 ? 8 : 4;
    const void* ptrs[] = {p.x, p.z, p.dy, p.y, p.dz};
    const int64_t strides[] = {p.xs, p.zs, p.dys, p.ys, p.dzs};
    bool wide = p.d % ve == 0, pair = bf16 && p.d % 2 == 0;
    for (int i = 0; i < 5; ++i) {
        if (!ptrs[i]) continue;
        const uintptr_t at = reinterpret_cast<uintptr_t>(ptrs[i]);
        wide = wide && at % 16 == 0 && strides[i] % ve == 0;
        pair = pair && at % 4 == 0 && strides[i] % 2 == 0;
    }
    return wide ? WIDE : (pair ? PAIR : SINGLE);
}
bool is_plain(const NormParams& p, bool wide) {
    return wide && !p.centred && !p.has_bias && !p.db_part;  // (dbias may be asked for without bias)
}
Shape backward_shape(int T, int H, int d, bool wide, bool bf16, bool plain) {
    return shape_of(T, H, d, wide, bf16, bwd_blocks(plain, wide && bf16), BWD_TOKENS);
}

template <typename IO, Access A, int LG, int NV, bool GATED, bool PLAIN>
void launch_one(const NormParams& p, int blocks, bool backward, cudaStream_t stream) {
    if (backward) {
        const size_t smem = p.per_head ? 0 : (size_t)(NT / LG) * p.d * sizeof(float);
        group_norm_backward_kernel<IO, A, LG, NV, GATED, PLAIN><<<blocks, NT, smem, stream>>>(p);
    } else {
        group_norm_kernel<IO, A, LG, NV, GATED, PLAIN><<<blocks, NT, 0, stream>>>(p);
    }
}

template <typename IO, Access A, int LG, int NV>
void launch_form(const NormParams& p, int blocks, bool backward, cudaStream_t stream) {
    if constexpr (A == WIDE) {
        if (is_plain(p, true)) {
            p.z ? launch_one<IO, A, LG, NV, true, true>(p, blocks, backward, stream)
                : launch_one<IO, A, LG, NV, false, true>(p, blocks, backward, stream);
            return;
        }
    }
    p.z ? launch_one<IO, A, LG, NV, true, false>(p, blocks, backward, stream)
        : launch_one<IO, A, LG, NV, false, false>(p, blocks, backward, stream);
}

template <typename IO, Access A>
cudaError_t launch_io(NormParams p, bool backward, cudaStream_t stream) {
    const bool plain = is_plain(p, A == WIDE);
    const Shape s = backward ? backward_shape(p.T, p.H, p.d, A == WIDE, sizeof(IO) == 2, plain)
                             : shape_of(p.T, p.H, p.d, A == WIDE, sizeof(IO) == 2,
                                        fwd_blocks(p.z != nullptr, plain), 1);
    p.streams = s.streams;
    constexpr int PER = A == WIDE ? 32 * 16 / (int)sizeof(IO) : 64;  // channels of 32 lanes' vectors
    const int nv = (p.d + PER - 1) / PER;
    if constexpr (A == WIDE) {
        if (s.lg == 4) launch_form<IO, A, 4, 1>(p, s.blocks, backward, stream);
        else if (s.lg == 8) launch_form<IO, A, 8, 1>(p, s.blocks, backward, stream);
        else if (s.lg == 16) launch_form<IO, A, 16, 1>(p, s.blocks, backward, stream);
        else if (nv <= 1) launch_form<IO, A, 32, 1>(p, s.blocks, backward, stream);
        else if (nv <= 2) launch_form<IO, A, 32, 2>(p, s.blocks, backward, stream);
        else if (nv <= 4) launch_form<IO, A, 32, 4>(p, s.blocks, backward, stream);
        else if constexpr (GDN_MAX_GROUP_DIM > 4 * PER)
            launch_form<IO, A, 32, 8>(p, s.blocks, backward, stream);
    } else {
        if (nv <= 1) launch_form<IO, A, 32, 1>(p, s.blocks, backward, stream);
        else if (nv <= 2) launch_form<IO, A, 32, 2>(p, s.blocks, backward, stream);
        else if (nv <= 3) launch_form<IO, A, 32, 3>(p, s.blocks, backward, stream);
        else if (nv <= 5) launch_form<IO, A, 32, 5>(p, s.blocks, backward, stream);
        else if (nv <= 8) launch_form<IO, A, 32, 8>(p, s.blocks, backward, stream);
        else launch_form<IO, A, 32, 16>(p, s.blocks, backward, stream);
    }
    return cudaGetLastError();
}

cudaError_t launch_any(const NormParams& p, bool bf16, bool backward, cudaStream_t stream) {
    switch (access_of(p, bf16)) {
        case WIDE:
            return bf16 ? launch_io<__nv_bfloat16, WIDE>(p, backward, stream)
                        : launch_io<float, WIDE>(p, backward, stream);
        case PAIR: return launch_io<__nv_bfloat16, PAIR>(p, backward, stream);
        default:
            return bf16 ? launch_io<__nv_bfloat16, SINGLE>(p, backward, stream)
                        : launch_io<float, SINGLE>(p, backward, stream);
    }
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
int partial_rows(int T, int H, int d, bool per_head, bool wide, bool bf16, bool plain) {
    const Shape s = backward_shape(T, H, d, wide, bf16, plain);
    return per_head ? s.streams : s.blocks;
}

}  // namespace

cudaError_t launch_group_norm(const GroupNormArgs& a, cudaStream_t stream) {
    if (a.T == 0) return cudaSuccess;
    return launch_any(params_of(a), a.bf16, false, stream);
}

size_t group_norm_backward_workspace_bytes(int T, int H, int d, int weight_heads, bool bf16) {
    if (T == 0) return 0;
    const bool per_head = weight_heads != 1;
    const size_t cols = (size_t)(per_head ? H : 1) * d;
    // enough for every form of the call: pointers, bias and norm are not known here
    size_t rows = 0;
    for (const bool wide : {false, true})
        for (const bool plain : {false, true}) {
            const size_t r = (size_t)partial_rows(T, H, d, per_head, wide, bf16, plain);
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
        const cudaError_t e = launch_any(p, a.bf16, true, stream);
        if (e != cudaSuccess) return e;
        const bool wide = access_of(p, a.bf16) == WIDE;
        rows = partial_rows(a.T, a.H, a.d, per_head, wide, a.bf16, is_plain(p, wide));
    }
    const ColumnSums sw{p.dw_part, dweight, rows, cols}, sb{p.db_part, dbias, rows, cols};
    const dim3 grid((cols + 31) / 32, dbias ? 2 : 1);
    return rows > 64 ? launch_second_step(column_sums_kernel<32>, grid, 1024, stream, sw, sb)
                     : launch_second_step(column_sums_kernel<8>, grid, 256, stream, sw, sb);
}

}  // namespace gdn
