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

#include <atomic>

#include "../../include/gdn.h"
#include "gdn_common.cuh"
#include "gdn_granules.h"
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
//   * A block takes a tile of TT = WARPS ST tokens x 64 channels; warp g holds ST consecutive
//     tokens, each lane two channels.
//   * A cluster of R blocks takes R consecutive tiles of the same 64 channels at a time and
//     walks over all tokens.  Each block sends its tile's (A, B) into the shared memory of
//     all R (st.async, completing on their mbarriers); every block joins them in rank order,
//     so each knows the state entering its own tile and the next R tiles.
//
// No block waits for anything outside its cluster, nothing goes through global memory, and
// the order of every sum is fixed by the sizes alone.  One more warp keeps one or two tiles on
// their way by TMA and works out which rows start or end a sequence.
//
// Packed sequences are one token axis: a row that starts a sequence (for the gradients,
// run backwards: ends one) drops the state that comes in and adds its own.  Maps across such
// a row carry A = -1 and drop the state by selection, not by a product with 0, so that an
// infinity or a NaN cannot cross.
constexpr int CW = 64;             // channels of a tile
constexpr int MAX_CLUSTER = 16;    // (above 8 only where the device grants it)
constexpr int SCAN_BAR = 1;        // named barrier of the consumer warps
constexpr unsigned long long kTestWaitNs = 20000000ull;  // limit of the waits that a test lets run out

struct ScanParams {
    const void *x, *la, *h;        // forward: x; gradients: dh, and h the forward's output
    const float *init, *h0;        // the state that a reset row adds; h0 for the gradients
    const int32_t* cu;
    void *out, *dla;               // h, or dx and dlog_alpha
    float* last;                   // h_final, or dh0
    int64_t xs, las, hs, outs, dlas;
    int N, T, C;
    int drop = -1;  // a test's: this tile (in scan order) never comes
    unsigned long long limit = kWaitLimitNs;
};

// Two neighbouring channels, as stored (bf16 pairs stay packed in one register) and widened.
template <typename T>
struct Pair;
template <>
struct Pair<float> {
    using Raw = float2;
    static __device__ __forceinline__ float2 widen(Raw v) { return v; }
};
template <>
struct Pair<__nv_bfloat16> {
    using Raw = uint32_t;
    static __device__ __forceinline__ float2 widen(Raw u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
};
// A tile in shared memory and its two channels of a lane.  TILED: rows of CW channels as the
// tensor copy wrote them, neighbours 2 lane and 2 lane + 1.  Else: rows of 16-byte granules
// whose first holds the row's first channel somewhere inside (`shift` bytes in, another one
// for every row), channels lane and lane + 32, which keeps the scalar accesses coalesced.
template <typename T, bool TILED>
struct Tile {
    static constexpr int PITCH = CW * (int)sizeof(T) + (TILED ? 0 : 16);
    // Where in its first granule a row starts, and what that moves by from row to row.
    static __device__ __forceinline__ uint32_t shift(const void* base, int row, int64_t stride,
                                                     int c0) {
        const uint32_t at = (uint32_t)reinterpret_cast<uintptr_t>(base);
        return (at + ((uint32_t)row * (uint32_t)stride + (uint32_t)c0) * (uint32_t)sizeof(T)) & 15u;
    }
    static __device__ __forceinline__ uint32_t shift_step(int64_t stride) {
        return (uint32_t)stride * (uint32_t)sizeof(T);
    }
    static __device__ __forceinline__ typename Pair<T>::Raw at(const uint8_t* tile, int r, int lane,
                                                               uint32_t shift) {
        if constexpr (TILED) {
            return reinterpret_cast<const typename Pair<T>::Raw*>(tile + r * PITCH)[lane];
        } else if constexpr (sizeof(T) == 2) {
            const uint16_t* p = reinterpret_cast<const uint16_t*>(tile + r * PITCH + shift) + lane;
            return (uint32_t)p[0] | (uint32_t)p[32] << 16;
        } else {
            const float* p = reinterpret_cast<const float*>(tile + r * PITCH + shift) + lane;
            return make_float2(p[0], p[32]);
        }
    }
};
__device__ __forceinline__ void put_two(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
__device__ __forceinline__ void put_two(__nv_bfloat16* p, float2 v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
}

// exp by the base-2 instruction: its own error is 2 ulp, and the product with log2(e) adds
// |v| 2^-24, which is small where the gate is not.  (expf's range checks cost 6 more
// instructions per element, and instructions are what this kernel runs out of first.)
__device__ __forceinline__ float2 exp2ch(float2 v) {
    const float2 w = mul2(v, make_float2(1.4426950408889634f, 1.4426950408889634f));
    float2 r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(w.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(w.y));
    return r;
}

// A lane's two channels of a row: neighbours, or 32 apart.
template <bool TILED>
__device__ __forceinline__ void put_both(float* p, float2 v) {
    if (TILED) {
        put_two(p, v);
    } else {
        p[0] = v.x;
        p[32] = v.y;
    }
}
template <bool TILED>
__device__ __forceinline__ void put_both(__nv_bfloat16* p, float2 v) {
    if (TILED) {
        put_two(p, v);
    } else {
        const uint32_t u = pack_bf16x2(v.x, v.y);
        reinterpret_cast<uint16_t*>(p)[0] = (uint16_t)u;
        reinterpret_cast<uint16_t*>(p)[32] = (uint16_t)(u >> 16);
    }
}

// A map s -> A s + B of two channels.
struct Map {
    float2 a, b;
};
__device__ __forceinline__ float4 as4(const Map& m) {
    return make_float4(m.a.x, m.a.y, m.b.x, m.b.y);
}
__device__ __forceinline__ Map as_map(float4 v) {
    return Map{make_float2(v.x, v.y), make_float2(v.z, v.w)};
}
// q after p, and q applied to a state; A < 0: the state that comes in is dropped.
__device__ __forceinline__ Map compose(const Map& p, const Map& q) {
    if (q.a.x < 0.f) return q;  // (both channels reset together)
    Map r;
    r.b = fma2(q.a, p.b, q.b);
    r.a = p.a.x < 0.f ? p.a : mul2(p.a, q.a);
    return r;
}
__device__ __forceinline__ float2 apply(const Map& q, float2 s) {
    return q.a.x < 0.f ? q.b : fma2(q.a, s, q.b);
}

// Asynchronous copies of a thread, in groups: 16 bytes, of which `bytes` are read and the others
// zeros.
__device__ __forceinline__ void cp_async16(void* to, const void* from, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
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
// mbar_wait of a whole warp, whose lanes give up together (those that went on alone would meet
// the others at no barrier).  CLUSTER: for data that other blocks wrote; such a wait gives up by
// its limit alone.  (A vote with every try costs nothing; one lane's tries for the others took
// 387 us instead of 205 us for 32,768 x 6144 bf16.)
template <bool CLUSTER>
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort,
                                          unsigned long long limit) {
    const uint32_t addr = smem_u32(bar);
    const auto there = [&] {
        return __all_sync(0xffffffffu, CLUSTER ? mbar_try_wait_cluster(addr, parity)
                                               : mbar_try_wait(addr, parity)) != 0;
    };
    if (there()) return true;
    const unsigned long long t0 = globaltimer();
    for (;;) {
        if (there()) return true;
        const bool late = globaltimer() - t0 > limit;
        if (late) atomicOr(&g_status, GDN_DEV_TIMEOUT);
        if (__any_sync(0xffffffffu, late || (!CLUSTER && *abort))) {
            *abort = 1;
            return false;
        }
    }
}

// When a wait runs out, all of a cluster unwinds, and its output is void (the status says so):
//   * The producer issues nothing more, and waits for what it has issued.
//   * A consumer warp waits, reads and writes no more and only takes part in the block's barriers
//     of the turns that are left (leaving the loop by a vote of the block instead took 215 us
//     where this takes 205 us, 32,768 x 6144 bf16).
//   * The block's map is sent no more, so that the others wait for it in vain and unwind in
//     turn; their limit is longer than any wait of a block before it sends.
// Nobody ends before all have come to the cluster's last barrier, and a map has then arrived or
// its sender has waited in vain for the others' since: none is on its way any more.

// Shared memory of a block.
template <typename IO, typename G, bool BWD, bool TMA, int WARPS, int ST>
struct ScanSmem {
    static constexpr int TT = WARPS * ST;
    static constexpr int X = TT * Tile<IO, TMA>::PITCH;
    static constexpr int L = TT * Tile<G, TMA>::PITCH;
    static constexpr int DATA = X + L + (BWD ? X : 0);  // x (dh), log_alpha, h
    struct Meta {
        uint32_t reset[WARPS], emit[WARPS];  // one bit per row of a time group, scan order
        int reset_n[TT], emit_n[TT];         // their sequences
    };
    static constexpr int METAS = 3;  // read until the tile is written, one tile longer
    static constexpr int META = 2 * DATA;
    static constexpr int AGG = META + METAS * (int)sizeof(Meta);
    static constexpr int SLOT = AGG + 2 * WARPS * 32 * 16;
    static constexpr int BARS = SLOT + 2 * MAX_CLUSTER * 32 * 16;
    static constexpr int BYTES = BARS + 6 * 8 + 16;
    static_assert(sizeof(Meta) % 16 == 0 && X % 128 == 0 && L % 128 == 0, "regions stay aligned");
};

template <typename IO, typename G, bool BWD, bool TMA, int WARPS, int ST, int MINB>
__global__ void __launch_bounds__((WARPS + 1) * 32, MINB)
    scan_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_la,
                const __grid_constant__ CUtensorMap map_h, const ScanParams p, const int R,
                const int two_stages) {
    using SM = ScanSmem<IO, G, BWD, TMA, WARPS, ST>;
    using Meta = typename SM::Meta;
    constexpr int TT = SM::TT;
    extern __shared__ __align__(128) uint8_t sm[];
    Meta* metas = reinterpret_cast<Meta*>(sm + SM::META);
    float4* agg = reinterpret_cast<float4*>(sm + SM::AGG);    // [2][WARPS][32]
    float4* slot = reinterpret_cast<float4*>(sm + SM::SLOT);  // [2][MAX_CLUSTER][32]
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + SM::BARS);
    uint64_t* empty = full + 2;
    uint64_t* joined = empty + 2;
    volatile int* abort_flag = reinterpret_cast<volatile int*>(joined + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const int c0 = (int)(blockIdx.x / R) * CW;
    const int T_end = p.cu ? min(max(p.cu[p.N], 0), p.T) : p.T;
    const int ntiles = (T_end + TT - 1) / TT, iters = (ntiles + R - 1) / R;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], TMA ? 2 : 1);  // the copies, and the rows' marks
            mbar_init(&empty[i], 1);
            mbar_init(&joined[i], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    cluster_sync();  // every block's barriers are ready before anyone sends to them

    if (warp == WARPS) {
        // ---- producer: tiles by TMA, and the rows where sequences start and end ----
        int it = 0;  // tiles issued
        for (; it * R + rank < ntiles; ++it) {
            const int st = it & two_stages, turn = it >> two_stages, k = it * R + rank;
            const int row0 = (BWD ? ntiles - 1 - k : k) * TT;
            if (k == p.drop) break;
            if (turn > 0 && !warp_wait<false>(&empty[st], (turn - 1) & 1, abort_flag, p.limit)) break;
            if (TMA && lane == 0) {
                uint8_t* d = sm + st * SM::DATA;
                mbar_arrive_expect_tx(&full[st], SM::DATA);
                tma_load_2d(d, &map_x, c0, row0, &full[st]);
                tma_load_2d(d + SM::X, &map_la, c0, row0, &full[st]);
                if (BWD) tma_load_2d(d + SM::X + SM::L, &map_h, c0, row0 - 1, &full[st]);
            }
            Meta& m = metas[it % SM::METAS];
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
        // the last copies have landed (bounded) before the block ends, whatever ended the loop
        if (lane == 0)
            for (int j = max(0, it - 1 - two_stages); j < it; ++j)
                mbar_wait_drain(&full[j & two_stages], (j >> two_stages) & 1);
    } else {
        // ---- consumers ----
        constexpr int NEXT = TMA ? 1 : 32;  // a lane's second channel
        const int c = c0 + (TMA ? 2 * lane : lane);
        const bool has0 = c < p.C, has1 = c + NEXT < p.C;
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
                    if (has1) p.last[o + NEXT] = p.init ? p.init[o + NEXT] : 0.f;
                }
            }
        }
        // Unaligned rows: every warp copies its own, the 16-byte granules that hold them, two
        // turns ahead (rows that are not used stay out); 32 / ST lanes to a row.
        const auto fetch = [&](int it) {
            const int k = it * R + rank;
            if (k < ntiles) {
                constexpr int LPR = 32 / ST;
                const int row0 = (BWD ? ntiles - 1 - k : k) * TT;
                const int r = (BWD ? TT - (warp + 1) * ST : warp * ST) + lane / LPR;
                uint8_t* d = sm + (it & 1) * SM::DATA;
                const auto copy = [&](auto t, uint8_t* tile, const void* base, int back, int64_t s) {
                    using E = decltype(t);
                    constexpr int PITCH = Tile<E, TMA>::PITCH;
                    if (row0 + r >= T_end || row0 + r - back < 0) return;
                    const E* whole = static_cast<const E*>(base);
                    const uintptr_t at = reinterpret_cast<uintptr_t>(
                        whole + (int64_t)(row0 + r - back) * s + c0);
                    const uint8_t* from = reinterpret_cast<const uint8_t*>(at & ~(uintptr_t)15);
                    uint8_t* to = tile + r * PITCH;
                    copy_granules<E, LPR, (PITCH / 16 + LPR - 1) / LPR>(
                        at, at + min(CW, p.C - c0) * (int)sizeof(E),
                        reinterpret_cast<uintptr_t>(whole),
                        reinterpret_cast<uintptr_t>(whole + (int64_t)(p.T - 1) * s + p.C),
                        lane % LPR, [&](int o, int bytes) { cp_async16(to + o, from + o, bytes); },
                        [&](int o) {
                            *reinterpret_cast<E*>(to + o) = *reinterpret_cast<const E*>(from + o);
                        });
                };
                copy(G(), d + SM::X, p.la, 0, p.las);
                copy(IO(), d, p.x, 0, p.xs);
                if (BWD) copy(IO(), d + SM::X + SM::L, p.h, 1, p.hs);
            }
            cp_async_commit();
        };
        if (!TMA)
            for (int it = 0; it < 2; ++it) fetch(it);

        float2 state = make_float2(0.f, 0.f);  // entering the R tiles of this iteration
        for (int it = 0; it < iters; ++it) {
            const int st = it & two_stages, k = it * R + rank, b = it & 1;
            const bool live = k < ntiles;
            const int row0 = (BWD ? ntiles - 1 - k : k) * TT;
            const Meta& m = metas[it % SM::METAS];
            float2 a[ST];
            typename Pair<IO>::Raw x[ST], before[BWD ? ST : 1];
            uint32_t reset = 0u, emit = 0u;
            Map mine{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
            // channels of a row of states
            const auto states = [&](const float* base, int n) {
                if (!base) return make_float2(0.f, 0.f);
                base += (int64_t)n * p.C + c;
                return make_float2(has0 ? base[0] : 0.f, has1 ? base[NEXT] : 0.f);
            };
            // The state given to the group's last sequence and h0 of its first: almost always the
            // only ones, and asked for early.  (The first matters for more: where that sequence
            // ends in another warp, its result may take the given state's place before this warp
            // runs again.)
            int last_reset = -1, first_emit = -1;
            float2 kept = make_float2(0.f, 0.f), kept_h0 = kept;
            // h (or u) of a row, from the row's before it in scan order
            const auto step = [](float2 aj, typename Pair<IO>::Raw xj, float2 s) {
                const float2 v = Pair<IO>::widen(xj);
                return BWD ? mul2(aj, add2(s, v)) : fma2(aj, s, v);
            };
            if (live) {
                if (!warp_wait<false>(&full[st], (it >> two_stages) & 1, abort_flag, p.limit)) {
                    for (; it < iters; ++it) bar_sync<SCAN_BAR, WARPS * 32>();
                    break;
                }
                reset = m.reset[warp];
                emit = m.emit[warp];
                if (reset) {
                    last_reset = 31 - __clz(reset);
                    kept = states(p.init, m.reset_n[warp * ST + last_reset]);
                }
                if (BWD && emit) {
                    first_emit = __ffs(emit) - 1;
                    kept_h0 = states(p.h0, m.emit_n[warp * ST + first_emit]);
                }
                const uint8_t* d = sm + st * SM::DATA;
                if (!TMA) {
                    cp_async_wait<1>();
                    __syncwarp();
                }
                typename Pair<G>::Raw l[ST];
                // (the shifts of unaligned rows, from the group's lowest row up)
                const int low = BWD ? TT - (warp + 1) * ST : warp * ST;
                uint32_t sl = 0, sx = 0, sh = 0;
                if (!TMA) {
                    sl = Tile<G, TMA>::shift(p.la, row0 + low, p.las, c0);
                    sx = Tile<IO, TMA>::shift(p.x, row0 + low, p.xs, c0);
                    if (BWD) sh = Tile<IO, TMA>::shift(p.h, row0 + low - 1, p.hs, c0);
                }
#pragma unroll
                for (int i = 0; i < ST; ++i) {
                    const int j = BWD ? ST - 1 - i : i, r = low + i;
                    l[j] = Tile<G, TMA>::at(d + SM::X, r, lane, sl);
                    x[j] = Tile<IO, TMA>::at(d, r, lane, sx);
                    if (BWD) before[j] = Tile<IO, TMA>::at(d + SM::X + SM::L, r, lane, sh);
                    if (!TMA) {
                        sl = (sl + Tile<G, TMA>::shift_step(p.las)) & 15u;
                        sx = (sx + Tile<IO, TMA>::shift_step(p.xs)) & 15u;
                        if (BWD) sh = (sh + Tile<IO, TMA>::shift_step(p.hs)) & 15u;
                    }
                }
#pragma unroll
                for (int j = 0; j < ST; ++j) a[j] = exp2ch(Pair<G>::widen(l[j]));
                // the map of these ST rows (only what follows the last reset counts)
                if (reset) {
#pragma unroll
                    for (int j = 0; j < ST; ++j)
                        mine.b = step(a[j], x[j], j == last_reset ? kept : mine.b);
                    mine.a = make_float2(-1.f, -1.f);
                } else {
#pragma unroll
                    for (int j = 0; j < ST; ++j) {
                        mine.b = step(a[j], x[j], mine.b);
                        mine.a = mul2(mine.a, a[j]);
                    }
                }
            }
            agg[(b * WARPS + warp) * 32 + lane] = as4(mine);
            // The tile is free again behind the warps' barrier, which no read of it can pass, with
            // each lane's reads ordered before the next copy, another proxy's write, by a fence.
            // (An arrive of every warp right behind its reads did not hold them: a tile was now
            // and then overwritten under the last of them when the code behind came from a cold
            // cache, and the gradients' h is not even needed before the second run.)
            if (TMA) fence_proxy_async_smem();
            bar_sync<SCAN_BAR, WARPS * 32>();
            if (live && threadIdx.x == 0) mbar_arrive(&empty[st]);
            // the map of the time groups before this one, within the tile
            Map pre{make_float2(1.f, 1.f), make_float2(0.f, 0.f)};
            for (int q = 0; q < warp; ++q)
                pre = compose(pre, as_map(agg[(b * WARPS + q) * 32 + lane]));
            if (warp == WARPS - 1) {  // the whole tile's map goes to every block
                if (lane == 0) mbar_arrive_expect_tx(&joined[b], R * 32 * 16);
                const float4 v = as4(compose(pre, mine));
                const uint32_t to = smem_u32(&slot[(b * MAX_CLUSTER + rank) * 32 + lane]);
                const uint32_t bar = smem_u32(&joined[b]);
                for (int r = 0; r < R; ++r) st_async(map_rank(to, r), v, map_rank(bar, r));
            }
            if (!TMA && live) fetch(it + 2);  // (while the maps travel)
            if (!warp_wait<true>(&joined[b], (it >> 1) & 1, abort_flag, 2 * p.limit)) {
                while (++it < iters) bar_sync<SCAN_BAR, WARPS * 32>();
                break;
            }
            float2 h = state;
#pragma unroll 4
            for (int r = 0; r < R; ++r) {
                if (r == rank) h = state;
                state = apply(as_map(slot[(b * MAX_CLUSTER + r) * 32 + lane]), state);
            }
            if (!live) continue;
            h = apply(pre, h);
            // the rows once more, from the state that enters them
            const int r0 = BWD ? TT - 1 - warp * ST : warp * ST;
            constexpr int DIR = BWD ? -1 : 1;
            IO* po = static_cast<IO*>(p.out) + (int64_t)(row0 + r0) * p.outs + c;
            G* pg = BWD ? static_cast<G*>(p.dla) + (int64_t)(row0 + r0) * p.dlas + c : nullptr;
            // o: the row's output, g: its second one (the gradients' dlog_alpha)
            const auto run = [&](int j, float2& o, float2& g, float2 w) {
                o = BWD ? add2(h, Pair<IO>::widen(x[j])) : step(a[j], x[j], h);
                h = BWD ? mul2(a[j], o) : o;
                if (BWD) g = mul2(h, w);
            };
            const auto put = [&](int j, float2 o, float2 g) {
                if (row0 + r0 + DIR * j < T_end) {
                    if (has0) po[0] = from_f<IO>(o.x);
                    if (has1) po[NEXT] = from_f<IO>(o.y);
                    if (BWD && has0) pg[0] = from_f<G>(g.x);
                    if (BWD && has1) pg[NEXT] = from_f<G>(g.y);
                }
                po += DIR * p.outs;
                if (BWD) pg += DIR * p.dlas;
            };
            const auto finish = [&](int j, float2 s) {  // the state behind a sequence
                if (!p.last) return;
                float* to = p.last + (int64_t)m.emit_n[warp * ST + j] * p.C + c;
                if (has0) to[0] = s.x;
                if (has1) to[NEXT] = s.y;
            };
            // Three forms of the same loop: rows without marks, groups with one boundary (no branch
            // inside: the rows' instructions interleave, which halves the time), and the rest.
            if (!(reset | emit) && row0 + TT <= T_end && c0 + CW <= p.C) {
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    float2 o, g;
                    run(j, o, g, Pair<IO>::widen(before[BWD ? j : 0]));
                    put_both<TMA>(po, o);
                    po += DIR * p.outs;
                    if (BWD) {
                        put_both<TMA>(pg, g);
                        pg += DIR * p.dlas;
                    }
                }
            } else if (!(reset & (reset - 1)) && !(emit & (emit - 1))) {
                const int emit_at = emit ? __ffs(emit) - 1 : -1;
                float2 ended = h;
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    float2 o, g;
                    if (j == last_reset) h = kept;
                    run(j, o, g,
                        BWD && j == emit_at ? kept_h0 : Pair<IO>::widen(before[BWD ? j : 0]));
                    if (j == emit_at) ended = h;
                    put(j, o, g);
                }
                if (emit) finish(emit_at, ended);
            } else {
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    float2 o, g;
                    if (reset >> j & 1)
                        h = j == last_reset ? kept : states(p.init, m.reset_n[warp * ST + j]);
                    float2 w = Pair<IO>::widen(before[BWD ? j : 0]);
                    if (BWD && emit >> j & 1)
                        w = j == first_emit ? kept_h0 : states(p.h0, m.emit_n[warp * ST + j]);
                    run(j, o, g, w);
                    if (emit >> j & 1) finish(j, h);
                    put(j, o, g);
                }
            }
        }
        cp_async_wait<0>();
    }
    __syncwarp();
    cluster_sync();  // nobody ends while others may still send to it
}

// ---- one token of each of B sequences ----
//
// Bound by bytes at large B and by the launch at small: one pass, V channels a thread
// (4 where rows are aligned: 16-byte accesses to the state; 256 x 6144 bf16 took 14.3 us with
// one channel a thread).
constexpr int STEP_THREADS = 128;

template <typename T, int V>
__device__ __forceinline__ void load_chans(const T* p, float2 (&v)[(V + 1) / 2]) {
    if constexpr (V == 4 && sizeof(T) == 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        v[0] = Pair<__nv_bfloat16>::widen(u.x), v[1] = Pair<__nv_bfloat16>::widen(u.y);
    } else if constexpr (V == 4) {
        const float4 u = *reinterpret_cast<const float4*>(p);
        v[0] = make_float2(u.x, u.y), v[1] = make_float2(u.z, u.w);
    } else {
        v[0] = make_float2(to_f(p[0]), 0.f);
    }
}

template <typename IO, typename G, int V>
__global__ void __launch_bounds__(STEP_THREADS) scan_step_kernel(const ScanArgs p, const int cblocks) {
    constexpr int NP = (V + 1) / 2;
    const int64_t b = blockIdx.x / cblocks;
    const int c = ((int)(blockIdx.x - b * cblocks) * STEP_THREADS + threadIdx.x) * V;
    if (c >= p.C) return;
    float* state = p.h_final + b * p.C + c;
    IO* h = static_cast<IO*>(p.h) + b * p.h_stride + c;
    float2 l[NP], x[NP], s[NP];
    load_chans<float, V>(state, s);
    load_chans<G, V>(static_cast<const G*>(p.la) + b * p.la_stride + c, l);
    load_chans<IO, V>(static_cast<const IO*>(p.x) + b * p.x_stride + c, x);
#pragma unroll
    for (int i = 0; i < NP; ++i) s[i] = fma2(exp2ch(l[i]), s[i], x[i]);
    if constexpr (V == 4) {
        *reinterpret_cast<float4*>(state) = make_float4(s[0].x, s[0].y, s[1].x, s[1].y);
        put_two(h, s[0]);
        put_two(h + 2, s[1]);
    } else {
        state[0] = s[0].x;
        h[0] = from_f<IO>(s[0].x);
    }
}

bool wide_rows(const void* ptr, int64_t stride, int elem) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && stride * elem % 16 == 0;
}

template <typename IO, typename G, bool BWD, bool TMA, int WARPS, int ST, int MINB>
cudaError_t launch_tiles(const ScanParams& p, cudaStream_t stream) {
    using SM = ScanSmem<IO, G, BWD, TMA, WARPS, ST>;
    const auto kernel = scan_kernel<IO, G, BWD, TMA, WARPS, ST, MINB>;
    CUtensorMap mx{}, ml{}, mh{};
    if (TMA && p.T > 0) {
        if (!tile_map(&mx, p.x, sizeof(IO) == 2, p.T, p.C, p.xs, CW, SM::TT) ||
            !tile_map(&ml, p.la, sizeof(G) == 2, p.T, p.C, p.las, CW, SM::TT) ||
            (BWD && !tile_map(&mh, p.h, sizeof(IO) == 2, p.T, p.C, p.hs, CW, SM::TT)))
            return cudaErrorInvalidValue;
    }
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // the kernel's attributes and how many clusters of R blocks a device holds: asked once
    static std::atomic<int> ready[kKnownDevices];
    static std::atomic<int> room[kKnownDevices][MAX_CLUSTER + 1];  // 0: not asked yet
    const bool known = dev < kKnownDevices;
    if (!known || !ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::BYTES);
        if (e != cudaSuccess) return e;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        if (known) ready[dev].store(1, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3((WARPS + 1) * 32);
    cfg.dynamicSmemBytes = SM::BYTES;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Blocks per cluster: the most with which all clusters run at once (a second wave costs as
    // much as the first), and no more than there are tiles.
    const long long groups = ((long long)p.C + CW - 1) / CW;
    const long long tiles = ((long long)p.T + SM::TT - 1) / SM::TT;
    int R = (int)(tiles < MAX_CLUSTER ? (tiles < 1 ? 1 : tiles) : MAX_CLUSTER);
    for (; R > 1; --R) {
        int fit = known ? room[dev][R].load(std::memory_order_relaxed) : 0;
        if (fit == 0) {
            cfg.gridDim = dim3(R);
            attr[0].val.clusterDim.x = R;
            if (cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg) != cudaSuccess || fit < 1) {
                cudaGetLastError();
                fit = -1;
            }
            if (known) room[dev][R].store(fit, std::memory_order_relaxed);
        }
        if (groups <= fit) break;
    }
    attr[0].val.clusterDim.x = R;
    cfg.gridDim = dim3((unsigned)(groups * R));
    // A second tile on its way hides the first one's latency.  The gradients' five streams
    // stand more in flight badly: past what the memory system needs it only lengthens the
    // queues, clusters progress unevenly and the last ones run alone.  32,768 x 6144 bf16
    // gradients took 410 us with 18.9 MB in flight and 339 us with 9.4 MB (344 us now); the forward
    // with fp32 gates took 246 us with 18.9 MB (242 us now) and 270 us with 9.4 MB.
    const int two = !BWD || !TMA || groups * R * (2ll * SM::DATA) <= (15 << 20);
    return cudaLaunchKernelEx(&cfg, kernel, mx, ml, mh, p, R, two);
}

template <typename IO, typename G, bool BWD>
cudaError_t launch_types(const ScanParams& p, cudaStream_t stream) {
    const int e = sizeof(IO), ge = sizeof(G);
    const bool wide = wide_rows(p.x, p.xs, e) && wide_rows(p.la, p.las, ge) &&
                      wide_rows(p.out, p.outs, e) &&
                      (!BWD || (wide_rows(p.h, p.hs, e) && wide_rows(p.dla, p.dlas, ge)));
    // Few channels leave one block an SM or less: larger tiles then, for fewer turns of the
    // cluster (131,072 x 128 bf16 forward: 217 us against 315 us when this was chosen; 133 us now).
    const bool few = ((long long)p.C + CW - 1) / CW * 8 <= known_sms();
    if (few) {
        // (16 rows a warp do not fit the shared memory where three unaligned fp32 tiles are held)
        constexpr int ST = BWD && sizeof(IO) + sizeof(G) == 8 ? 8 : 16;
        return wide ? launch_tiles<IO, G, BWD, true, 8, 16, 1>(p, stream)
                    : launch_tiles<IO, G, BWD, false, 8, ST, 1>(p, stream);
    }
    // Unaligned tiles always come two at a time; smaller ones then, but for two streams of bf16, so
    // as not to queue (32,768 x 3,001: fp32 gradients 449 us against 1713 us with 16 rows a warp,
    // bf16 gradients 357 us against 709 us, fp32 forward 321 us against 379 us, bf16 forward 272 us
    // against 250 us; now, the tensors' ends checked: 461, 368, 308 and 242 us).
    constexpr int ST = BWD || sizeof(IO) + sizeof(G) > 4 ? 8 : 16;
    // (the shared memory of three fp32 tiles leaves room for two blocks an SM: their registers then)
    constexpr int MINB = BWD && sizeof(IO) == 4 ? 2 : 3;
    return wide ? launch_tiles<IO, G, BWD, true, 4, 16, MINB>(p, stream)
                : launch_tiles<IO, G, BWD, false, 4, ST, 3>(p, stream);
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

bool tile_map(CUtensorMap* map, const void* base, bool bf16, int64_t T, int64_t C, int64_t stride,
              int cols, int rows) {
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
    const cuuint32_t box[2] = {(cuuint32_t)cols, (cuuint32_t)rows}, ones[2] = {1, 1};
    return encode(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2,
                  const_cast<void*>(base), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_scan(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream) {
    ScanParams p{};
    p.x = a.x, p.la = a.la, p.init = a.h0, p.cu = a.cu_seqlens, p.out = a.h, p.last = a.h_final;
    p.xs = a.x_stride, p.las = a.la_stride, p.outs = a.h_stride;
    p.N = a.N, p.T = a.T, p.C = a.C;
    if (a.drop >= 0) p.drop = a.drop, p.limit = kTestWaitNs;
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
    if (a.drop >= 0) p.drop = a.drop, p.limit = kTestWaitNs;
    return launch_direction<true>(p, bf16, gate_bf16, stream);
}

template <typename IO, typename G>
static cudaError_t launch_step(const ScanArgs& a, cudaStream_t stream) {
    const bool wide = a.C % 4 == 0 && reinterpret_cast<uintptr_t>(a.h_final) % 16 == 0 &&
                      wide_rows(a.x, a.x_stride, sizeof(IO)) &&
                      wide_rows(a.la, a.la_stride, sizeof(G)) &&
                      wide_rows(a.h, a.h_stride, sizeof(IO));
    const int per = STEP_THREADS * (wide ? 4 : 1), cblocks = (a.C + per - 1) / per;
    const long long blocks = (long long)a.T * cblocks;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    if (wide)
        scan_step_kernel<IO, G, 4><<<(unsigned)blocks, STEP_THREADS, 0, stream>>>(a, cblocks);
    else
        scan_step_kernel<IO, G, 1><<<(unsigned)blocks, STEP_THREADS, 0, stream>>>(a, cblocks);
    return cudaGetLastError();
}

cudaError_t launch_scan_step(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream) {
    if (bf16)
        return gate_bf16 ? launch_step<__nv_bfloat16, __nv_bfloat16>(a, stream)
                         : launch_step<__nv_bfloat16, float>(a, stream);
    return gate_bf16 ? launch_step<float, __nv_bfloat16>(a, stream)
                     : launch_step<float, float>(a, stream);
}

}  // namespace gdn
