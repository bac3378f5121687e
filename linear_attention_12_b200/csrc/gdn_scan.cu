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
#include "gdn_tiles.cuh"

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

// ---- the scan over many tokens ----
//
// A scan step is the map s -> A s + B, and maps compose, so a long sequence can be cut
// anywhere: every piece forms its (A, B) from s = 0 side by side, the pieces' maps are
// joined in order, and every piece then runs again from the state that enters it.  Here
// the data is read once and stays in registers between the two runs:
//
//   * A block takes a tile of TT = 8 ST tokens x 64 channels; warp g holds ST consecutive
//     tokens, each lane two channels.
//   * A cluster of R blocks takes R consecutive tiles of the same 64 channels at a time and
//     walks over all tokens.  Each block sends its tile's (A, B) into the shared memory of
//     all R (st.async, completing on their mbarriers); every block joins them in rank order,
//     so each knows the state entering its own tile and the next R tiles.
//
// No block waits for anything outside its cluster, nothing goes through global memory, and
// the order of every sum is fixed by the sizes alone.  A ninth warp keeps STAGES tiles on
// their way by TMA and works out which rows start or end a sequence.
//
// Packed sequences are one token axis: a row that starts a sequence (for the gradients,
// run backwards: ends one) drops the state that comes in and adds its own.  Maps across such
// a row carry A = -1 and drop the state by selection, not by a product with 0, so that an
// infinity or a NaN cannot cross.
constexpr int CW = 64;             // channels of a tile
constexpr int WARPS = 8;           // consumer warps: time groups of a tile
constexpr int THREADS = (WARPS + 1) * 32;
constexpr int MAX_CLUSTER = 8;
constexpr int SCAN_BAR = 1;        // named barrier of the consumer warps

struct ScanParams {
    const void *x, *la, *h;        // forward: x; gradients: dh, and h the forward's output
    const float *init, *h0;        // the state that a reset row adds; h0 for the gradients
    const int32_t* cu;
    void *out, *dla;               // h, or dx and dlog_alpha
    float* last;                   // h_final, or dh0
    int64_t xs, las, hs, outs, dlas;
    int N, T, C;
};

// Two neighbouring channels.
__device__ __forceinline__ float2 two(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 two(const __nv_bfloat16* p) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ void put_two(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void put_two(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
}

// The map (A, B) of two channels, the later one q after p, and a map applied to a state.
__device__ __forceinline__ void compose1(float& pa, float& pb, float qa, float qb) {
    pb = qa < 0.f ? qb : fmaf(qa, pb, qb);
    pa = qa < 0.f || pa < 0.f ? -1.f : pa * qa;
}
__device__ __forceinline__ float apply1(float qa, float qb, float s) {
    return qa < 0.f ? qb : fmaf(qa, s, qb);
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void st_async(uint32_t addr, float4 v, uint32_t bar) {
    asm volatile(
        "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
        "[%5];" ::"r"(addr),
        "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
        : "memory");
}
// mbar_wait for data that other blocks of the cluster wrote.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort) {
    const uint32_t addr = smem_u32(bar);
    if (mbar_try_wait_cluster(addr, parity)) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (mbar_try_wait_cluster(addr, parity)) return true;
        if (*abort) return false;
        if (globaltimer() - t0 > kWaitLimitNs) {
            atomicOr(&g_status, GDN_DEV_TIMEOUT);
            *abort = 1;
            return false;
        }
    }
}

// Shared memory of a block.
template <typename IO, typename G, bool BWD, bool TMA, int ST, int STAGES>
struct ScanSmem {
    static constexpr int TT = WARPS * ST;
    static constexpr int X = TMA ? TT * CW * (int)sizeof(IO) : 0;
    static constexpr int L = TMA ? TT * CW * (int)sizeof(G) : 0;
    static constexpr int DATA = X + L + (BWD ? X : 0);  // x (dh), log_alpha, h
    struct Meta {
        uint32_t reset[WARPS], emit[WARPS];  // one bit per row of a time group, scan order
        int reset_n[TT], emit_n[TT];         // their sequences
    };
    static constexpr int META = STAGES * DATA;
    static constexpr int AGG = META + STAGES * (int)sizeof(Meta);
    static constexpr int SLOT = AGG + 2 * WARPS * 32 * 16;
    static constexpr int BARS = SLOT + 2 * MAX_CLUSTER * 32 * 16;
    static constexpr int BYTES = BARS + (2 * STAGES + 2) * 8 + 16;
    static_assert(sizeof(Meta) % 16 == 0 && DATA % 128 == 0, "regions stay aligned");
};

template <typename IO, typename G, bool BWD, bool TMA, int ST, int STAGES, int MINB>
__global__ void __launch_bounds__(THREADS, MINB)
    scan_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_la,
                const __grid_constant__ CUtensorMap map_h, const ScanParams p, const int R) {
    using SM = ScanSmem<IO, G, BWD, TMA, ST, STAGES>;
    using Meta = typename SM::Meta;
    constexpr int TT = SM::TT;
    extern __shared__ __align__(128) uint8_t sm[];
    Meta* metas = reinterpret_cast<Meta*>(sm + SM::META);
    float4* agg = reinterpret_cast<float4*>(sm + SM::AGG);    // [2][WARPS][32]
    float4* slot = reinterpret_cast<float4*>(sm + SM::SLOT);  // [2][MAX_CLUSTER][32]
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + SM::BARS);
    uint64_t* empty = full + STAGES;
    uint64_t* joined = empty + STAGES;  // [2]
    volatile int* abort_flag = reinterpret_cast<volatile int*>(joined + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int c0 = (int)(blockIdx.x / R) * CW;
    const int T_end = p.cu ? min(max(p.cu[p.N], 0), p.T) : p.T;
    const int ntiles = (T_end + TT - 1) / TT, iters = (ntiles + R - 1) / R;

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 2);
            mbar_init(&empty[i], WARPS);
        }
        mbar_init(&joined[0], 1);
        mbar_init(&joined[1], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    cluster_sync();  // every block's barriers are ready before anyone sends to them

    if (warp == WARPS) {
        // ---- producer: tiles by TMA, and the rows where sequences start and end ----
        int it = 0;
        for (; it * R + rank < ntiles; ++it) {
            const int st = it % STAGES, k = it * R + rank;
            const int row0 = (BWD ? ntiles - 1 - k : k) * TT;
            if (it >= STAGES) mbar_wait(&empty[st], (it / STAGES - 1) & 1, abort_flag);
            if (lane == 0) {
                if (TMA) {
                    uint8_t* d = sm + st * SM::DATA;
                    mbar_arrive_expect_tx(&full[st], SM::DATA);
                    tma_load_2d(d, &map_x, c0, row0, &full[st]);
                    tma_load_2d(d + SM::X, &map_la, c0, row0, &full[st]);
                    if (BWD) tma_load_2d(d + SM::X + SM::L, &map_h, c0, row0 - 1, &full[st]);
                } else {
                    mbar_arrive(&full[st]);
                }
            }
            Meta& m = metas[st];
            if (lane < WARPS) m.reset[lane] = m.emit[lane] = 0u;
            __syncwarp();
            int n = 0;  // the last sequence that starts at or before row0
            if (p.cu) {
                int hi = p.N - 1;
                while (n < hi) {
                    const int mid = (n + hi + 1) >> 1;
                    if (p.cu[mid] <= row0) n = mid; else hi = mid - 1;
                }
            }
            for (n += lane;; n += 32) {
                const bool in = n < p.N;
                const int lo = in ? (p.cu ? p.cu[n] : 0) : 0x7fffffff;
                const int hi = in ? (p.cu ? min(p.cu[n + 1], T_end) : T_end) : 0;
                if (lo < hi) {
                    // (bit j of a time group is its j-th row in scan order)
                    const int f = BWD ? TT - 1 - (lo - row0) : lo - row0;
                    const int l = BWD ? TT - 1 - (hi - 1 - row0) : hi - 1 - row0;
                    if (f >= 0 && f < TT) {
                        (BWD ? m.emit_n : m.reset_n)[f] = n;
                        atomicOr(BWD ? &m.emit[f / ST] : &m.reset[f / ST], 1u << (f % ST));
                    }
                    if (l >= 0 && l < TT) {
                        (BWD ? m.reset_n : m.emit_n)[l] = n;
                        atomicOr(BWD ? &m.reset[l / ST] : &m.emit[l / ST], 1u << (l % ST));
                    }
                }
                if (__any_sync(0xffffffffu, lo >= row0 + TT)) break;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[st]);
        }
        if (*abort_flag && lane == 0) {
            // copies may still be landing: let them (bounded) before the block ends
            const unsigned long long ts = globaltimer();
            for (int j = max(0, it - STAGES); j < it; ++j)
                while (!mbar_try_wait(smem_u32(&full[j % STAGES]), (j / STAGES) & 1) &&
                       globaltimer() - ts < kWaitLimitNs) {
                }
        }
        __syncwarp();
    } else {
        // ---- consumers ----
        const int c = c0 + 2 * lane;
        const bool has0 = c < p.C, has1 = c + 1 < p.C;
        // sequences without tokens hand their state through
        if (p.last && (p.cu || T_end == 0)) {
            for (int n0 = (rank * WARPS + warp) * 32; n0 < p.N; n0 += R * WARPS * 32) {
                const int n = n0 + lane;
                uint32_t none = __ballot_sync(
                    0xffffffffu, n < p.N && (!p.cu || p.cu[n] >= p.cu[min(n, p.N - 1) + 1]));
                while (none) {
                    const int64_t o = (int64_t)(n0 + __ffs(none) - 1) * p.C + c;
                    none &= none - 1;
                    if (has0) p.last[o] = p.init ? p.init[o] : 0.f;
                    if (has1) p.last[o + 1] = p.init ? p.init[o + 1] : 0.f;
                }
            }
        }
        float s0 = 0.f, s1 = 0.f;  // the state entering the R tiles of this iteration
        for (int it = 0; it < iters; ++it) {
            const int st = it % STAGES, k = it * R + rank, b = it & 1;
            const bool live = k < ntiles;
            const int row0 = (BWD ? ntiles - 1 - k : k) * TT;
            float2 a[ST], x[ST], before[BWD ? ST : 1];
            uint32_t reset = 0u, emit = 0u;
            float A0 = 1.f, A1 = 1.f, B0 = 0.f, B1 = 0.f;
            if (live) {
                const Meta& m = metas[st];
                if (mbar_wait(&full[st], (it / STAGES) & 1, abort_flag)) {
                    reset = m.reset[warp];
                    emit = m.emit[warp];
                }
                const uint8_t* d = sm + st * SM::DATA;
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    const int r = BWD ? TT - 1 - (warp * ST + j) : warp * ST + j;
                    float2 l;
                    if (TMA) {
                        x[j] = two(reinterpret_cast<const IO*>(d) + r * CW + 2 * lane);
                        l = two(reinterpret_cast<const G*>(d + SM::X) + r * CW + 2 * lane);
                        if (BWD)
                            before[j] =
                                two(reinterpret_cast<const IO*>(d + SM::X + SM::L) + r * CW + 2 * lane);
                    } else {
                        const int64_t t = row0 + r;
                        const bool in = t < T_end;
                        const IO* px = static_cast<const IO*>(p.x) + t * p.xs + c;
                        const G* pl = static_cast<const G*>(p.la) + t * p.las + c;
                        x[j] = make_float2(in && has0 ? to_f(px[0]) : 0.f, in && has1 ? to_f(px[1]) : 0.f);
                        l = make_float2(in && has0 ? to_f(pl[0]) : 0.f, in && has1 ? to_f(pl[1]) : 0.f);
                        if (BWD) {
                            const bool inb = in && t > 0;
                            const IO* ph = static_cast<const IO*>(p.h) + (t - 1) * p.hs + c;
                            before[j] = make_float2(inb && has0 ? to_f(ph[0]) : 0.f,
                                                    inb && has1 ? to_f(ph[1]) : 0.f);
                        }
                    }
                    a[j] = make_float2(expf(l.x), expf(l.y));
                }
                if (reset | emit) {
                    // rows that add the state of their sequence
#pragma unroll
                    for (int j = 0; j < ST; ++j) {
                        if (reset >> j & 1 && p.init) {
                            const int64_t o = (int64_t)m.reset_n[warp * ST + j] * p.C + c;
                            const float i0 = has0 ? p.init[o] : 0.f, i1 = has1 ? p.init[o + 1] : 0.f;
                            // (the gradients multiply by the gate behind the sum)
                            x[j].x = BWD ? x[j].x + i0 : fmaf(a[j].x, i0, x[j].x);
                            x[j].y = BWD ? x[j].y + i1 : fmaf(a[j].y, i1, x[j].y);
                        }
                        if (BWD && emit >> j & 1) {
                            const int64_t o = (int64_t)m.emit_n[warp * ST + j] * p.C + c;
                            before[j].x = p.h0 && has0 ? p.h0[o] : 0.f;
                            before[j].y = p.h0 && has1 ? p.h0[o + 1] : 0.f;
                        }
                    }
                }
                if (!emit) {  // nothing of the stage is read again
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&empty[st]);
                }
                // the map of these ST rows
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    if (reset >> j & 1) B0 = B1 = 0.f;
                    if (BWD) {
                        B0 = a[j].x * (B0 + x[j].x);
                        B1 = a[j].y * (B1 + x[j].y);
                    } else {
                        B0 = fmaf(a[j].x, B0, x[j].x);
                        B1 = fmaf(a[j].y, B1, x[j].y);
                    }
                    A0 *= a[j].x;
                    A1 *= a[j].y;
                }
                if (reset) A0 = A1 = -1.f;
            }
            agg[(b * WARPS + warp) * 32 + lane] = make_float4(A0, B0, A1, B1);
            bar_sync<SCAN_BAR, WARPS * 32>();
            // the map of the time groups before this one, within the tile
            float pa0 = 1.f, pa1 = 1.f, pb0 = 0.f, pb1 = 0.f;
            for (int q = 0; q < warp; ++q) {
                const float4 v = agg[(b * WARPS + q) * 32 + lane];
                compose1(pa0, pb0, v.x, v.y);
                compose1(pa1, pb1, v.z, v.w);
            }
            if (warp == WARPS - 1) {  // the whole tile's map goes to every block
                if (lane == 0) mbar_arrive_expect_tx(&joined[b], R * 32 * 16);
                float4 v = make_float4(pa0, pb0, pa1, pb1);
                compose1(v.x, v.y, A0, B0);
                compose1(v.z, v.w, A1, B1);
                const uint32_t to = smem_u32(&slot[(b * MAX_CLUSTER + rank) * 32 + lane]);
                const uint32_t bar = smem_u32(&joined[b]);
                for (int r = 0; r < R; ++r) st_async(map_rank(to, r), v, map_rank(bar, r));
            }
            mbar_wait_cluster(&joined[b], (it >> 1) & 1, abort_flag);
            float h0 = s0, h1 = s1;
            for (int r = 0; r < R; ++r) {
                if (r == rank) h0 = s0, h1 = s1;
                const float4 v = slot[(b * MAX_CLUSTER + r) * 32 + lane];
                s0 = apply1(v.x, v.y, s0);
                s1 = apply1(v.z, v.w, s1);
            }
            if (!live) continue;
            h0 = apply1(pa0, pb0, h0);
            h1 = apply1(pa1, pb1, h1);
            // the rows once more, from the state that enters them
            const Meta& m = metas[st];
#pragma unroll
            for (int j = 0; j < ST; ++j) {
                const int r = BWD ? TT - 1 - (warp * ST + j) : warp * ST + j;
                const int64_t t = row0 + r;
                if (reset >> j & 1) h0 = h1 = 0.f;
                float2 o, g;
                if (BWD) {
                    o = make_float2(x[j].x + h0, x[j].y + h1);
                    h0 = a[j].x * o.x;
                    h1 = a[j].y * o.y;
                    g = make_float2(h0 * before[j].x, h1 * before[j].y);
                } else {
                    h0 = fmaf(a[j].x, h0, x[j].x);
                    h1 = fmaf(a[j].y, h1, x[j].y);
                    o = make_float2(h0, h1);
                }
                if (t < T_end) {
                    IO* po = static_cast<IO*>(p.out) + t * p.outs + c;
                    G* pg = BWD ? static_cast<G*>(p.dla) + t * p.dlas + c : nullptr;
                    if (TMA && has1) {
                        put_two(po, o);
                        if (BWD) put_two(pg, g);
                    } else {
                        if (has0) po[0] = from_f<IO>(o.x);
                        if (has1) po[1] = from_f<IO>(o.y);
                        if (BWD && has0) pg[0] = from_f<G>(g.x);
                        if (BWD && has1) pg[1] = from_f<G>(g.y);
                    }
                }
                if (emit >> j & 1 && p.last) {
                    const int64_t at = (int64_t)m.emit_n[warp * ST + j] * p.C + c;
                    if (has0) p.last[at] = h0;
                    if (has1) p.last[at + 1] = h1;
                }
            }
            if (emit) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
        }
    }
    cluster_sync();  // nobody ends while others may still send to it
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

// A [T, C] tensor as boxes of `rows` x CW; false if the driver refuses it.
bool tile_map(CUtensorMap* map, const void* base, bool bf16, int64_t T, int64_t C, int64_t stride,
              int rows) {
    using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void* fn = nullptr;
        cudaDriverEntryPointQueryResult found = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            fn = nullptr;
        return reinterpret_cast<Encode>(fn);
    }();
    if (!encode) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)C, (cuuint64_t)T};
    const cuuint64_t strides[1] = {(cuuint64_t)stride * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {CW, (cuuint32_t)rows}, ones[2] = {1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                  const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool wide_rows(const void* ptr, int64_t stride, int elem) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && stride * elem % 16 == 0;
}

template <typename IO, typename G, bool BWD, bool TMA, int ST, int STAGES, int MINB>
cudaError_t launch_tiles(const ScanParams& p, cudaStream_t stream) {
    using SM = ScanSmem<IO, G, BWD, TMA, ST, STAGES>;
    const auto kernel = scan_kernel<IO, G, BWD, TMA, ST, STAGES, MINB>;
    CUtensorMap mx{}, ml{}, mh{};
    if (TMA && p.T > 0) {
        if (!tile_map(&mx, p.x, sizeof(IO) == 2, p.T, p.C, p.xs, SM::TT) ||
            !tile_map(&ml, p.la, sizeof(G) == 2, p.T, p.C, p.las, SM::TT) ||
            (BWD && !tile_map(&mh, p.h, sizeof(IO) == 2, p.T, p.C, p.hs, SM::TT)))
            return cudaErrorInvalidValue;
    }
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::BYTES);
    if (e != cudaSuccess) return e;
    // blocks per cluster: as many as the SMs hold at once, and no more than there are tiles
    const long long groups = ((long long)p.C + CW - 1) / CW;
    const long long tiles = ((long long)p.T + SM::TT - 1) / SM::TT;
    const long long room = (long long)device_sms() * MINB;
    int R = 1;
    while (R < MAX_CLUSTER && R < tiles && groups * (2 * R) <= room) R *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(groups * R));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SM::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = R;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, mx, ml, mh, p, R);
}

template <typename IO, typename G, bool BWD>
cudaError_t launch_types(const ScanParams& p, cudaStream_t stream) {
    const int e = sizeof(IO), ge = sizeof(G);
    const bool wide = wide_rows(p.x, p.xs, e) && wide_rows(p.la, p.las, ge) &&
                      wide_rows(p.out, p.outs, e) &&
                      (!BWD || (wide_rows(p.h, p.hs, e) && wide_rows(p.dla, p.dlas, ge)));
    constexpr int STAGES = 2;
    constexpr int MINB = BWD ? 2 : 3;
    if (wide) return launch_tiles<IO, G, BWD, true, 8, STAGES, MINB>(p, stream);
    return launch_tiles<IO, G, BWD, false, 8, STAGES, MINB>(p, stream);
}

template <bool BWD>
cudaError_t launch_direction(const ScanParams& p, bool bf16, bool gate_bf16, cudaStream_t stream) {
    if (bf16)
        return gate_bf16 ? launch_types<__nv_bfloat16, __nv_bfloat16, BWD>(p, stream)
                         : launch_types<__nv_bfloat16, float, BWD>(p, stream);
    return gate_bf16 ? launch_types<float, __nv_bfloat16, BWD>(p, stream)
                     : launch_types<float, float, BWD>(p, stream);
}

}  // namespace

cudaError_t launch_scan(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream) {
    ScanParams p{};
    p.x = a.x, p.la = a.la, p.init = a.h0, p.cu = a.cu_seqlens, p.out = a.h, p.last = a.h_final;
    p.xs = a.x_stride, p.las = a.la_stride, p.outs = a.h_stride;
    p.N = a.N, p.T = a.T, p.C = a.C;
    return launch_direction<false>(p, bf16, gate_bf16, stream);
}

cudaError_t launch_scan_backward(const ScanGradArgs& a, bool bf16, bool gate_bf16,
                                 cudaStream_t stream) {
    ScanParams p{};
    p.x = a.dh, p.la = a.la, p.h = a.h, p.init = a.dh_final, p.h0 = a.h0, p.cu = a.cu_seqlens;
    p.out = a.dx, p.dla = a.dla, p.last = a.dh0;
    p.xs = a.dh_stride, p.las = a.la_stride, p.hs = a.h_stride, p.outs = a.dx_stride;
    p.dlas = a.dla_stride;
    p.N = a.N, p.T = a.T, p.C = a.C;
    return launch_direction<true>(p, bf16, gate_bf16, stream);
}

cudaError_t launch_scan_step(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream) {
    const int64_t blocks = ((int64_t)a.T * a.C + 255) / 256;
    const int grid = (int)(blocks < 148 * 64 ? blocks : 148 * 64);
    if (bf16) {
        if (gate_bf16) scan_step_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 256, 0, stream>>>(a);
        else scan_step_kernel<__nv_bfloat16, float><<<grid, 256, 0, stream>>>(a);
    } else {
        if (gate_bf16) scan_step_kernel<float, __nv_bfloat16><<<grid, 256, 0, stream>>>(a);
        else scan_step_kernel<float, float><<<grid, 256, 0, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace gdn
