// gdn_internal.h -- launchers behind the C ABI (not part of the public header).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

cudaError_t launch_decode_step(const void* q, const void* k, const void* v,
                               const float* log_alpha, const float* beta, float* S, int B,
                               int H_qk, int H_v, bool bf16, void* o, cudaStream_t stream);
cudaError_t launch_decode_multi(const void* q, const void* k, const void* v,
                                const float* log_alpha, const float* beta, const float* S_in,
                                float* S_steps, int B, int M, int H_qk, int H_v, bool bf16,
                                void* o, cudaStream_t stream);

// Workspace bytes the prefill needs with P segments per sequence (fp32 I/O
// also stages bf16 copies of q, k, v).
size_t prefill_workspace_bytes(int N, int T, int H_qk, int H_v, bool bf16, int P);

// Devices (by index) whose properties are remembered between calls.
constexpr int kKnownDevices = 64;

// SM count of the current device (148 when there is none).
int device_sms();
// The same, remembered for each device (for calls that ask several times).
int known_sms();

// Segments per sequence the prefill uses when the caller leaves it to the
// library: 1 unless splitting the sequences fills more of the SMs.
int choose_segments(int N, int T, int H_v, int sms);

// Which implementation runs the state pass that writes the prefill's outputs.
constexpr int STATE_PASS_AUTO = 0;  // the faster one for the slice width
constexpr int STATE_PASS_TC = 1;    // tcgen05, accumulators in tensor memory
constexpr int STATE_PASS_MMA = 2;   // warp-level mma.sync, accumulators in registers

// P segments per sequence (P <= 0: choose_segments).
cudaError_t launch_prefill(const void* q, const void* k, const void* v, const float* log_alpha,
                           const float* beta, const float* S0, const int32_t* cu_seqlens, int N,
                           int T, int H_qk, int H_v, bool bf16, void* o, float* S_final,
                           void* workspace, int P, int state_pass, cudaStream_t stream);

// Records and chunk-entering states (bf16 images) of a prefill with bf16
// q, k, v, for its gradients; with o non-null also its outputs (bf16 or fp32)
// and final states.
cudaError_t launch_prefill_save(const void* q, const void* k, const void* v,
                                const float* log_alpha, const float* beta, const float* S0,
                                const int32_t* cu_seqlens, int N, int T, int H_qk, int H_v,
                                uint8_t* records, uint8_t* S_saved, void* o, float* S_final,
                                bool out_bf16, cudaStream_t stream);
size_t prefill_record_bytes(int N, int T, int H_v);

// Gradients of a bf16 prefill: workspace bytes, and the launches (the forward
// pass saving every chunk's state, the reverse chain, the per-chunk gradients).
size_t prefill_backward_workspace_bytes(int N, int T, int H_qk, int H_v, bool bf16);
cudaError_t launch_prefill_backward(const void* q, const void* k, const void* v,
                                    const float* log_alpha, const float* beta, const float* S0,
                                    const int32_t* cu_seqlens, const void* dO,
                                    const float* dS_final, int N, int T, int H_qk, int H_v,
                                    bool bf16, void* dq, void* dk, void* dv, float* dlog_alpha,
                                    float* dbeta, float* dS0, void* workspace, bool recompute,
                                    cudaStream_t stream);
// The prefill (outputs, final states) that also leaves in `workspace` (laid
// out as launch_prefill_backward's) the records and entering states its
// gradients read; launch_prefill_backward with recompute = false then skips
// the forward re-run.
cudaError_t launch_prefill_train(const void* q, const void* k, const void* v,
                                 const float* log_alpha, const float* beta, const float* S0,
                                 const int32_t* cu_seqlens, int N, int T, int H_qk, int H_v,
                                 bool bf16, void* o, float* S_final, void* workspace,
                                 cudaStream_t stream);

cudaError_t launch_frontend(const void* q_raw, const void* k_raw, const void* v_raw,
                            const float* conv_w, const float* a, const float* b,
                            const int32_t* cu_seqlens, int N, int T, int H_qk, int H_v,
                            bool bf16, int act, float eps, void* q, void* k, void* v,
                            float* log_alpha, float* beta, cudaStream_t stream);

cudaError_t launch_frontend_decode(const void* q_raw, const void* k_raw, const void* v_raw,
                                   const float* conv_w, const float* a, const float* b,
                                   void* conv_state, int B, int H_qk, int H_v, bool bf16, int act,
                                   float eps, void* q, void* k, void* v, float* log_alpha,
                                   float* beta, cudaStream_t stream);

// The tensor map of a [T, C] tensor (row stride in elements) read in boxes of rows x cols,
// rows and columns outside it as zeros; false if the driver refuses it.
bool tile_map(CUtensorMap* map, const void* base, bool bf16, int64_t T, int64_t C, int64_t stride,
              int cols, int rows);

// The per-channel recurrence (row strides in elements; the step's T is its B and
// its h_final the state).
struct ScanArgs {
    const void *x, *la;
    const float* h0;
    const int32_t* cu_seqlens;
    void* h;
    float* h_final;
    int64_t x_stride, la_stride, h_stride;
    int N, T, C;
    int drop = -1;  // a test's: this tile never comes, and the waits are short
};
struct ScanGradArgs {
    const void *la, *h, *dh;
    const float *h0, *dh_final;
    const int32_t* cu_seqlens;
    void *dx, *dla;
    float* dh0;
    int64_t la_stride, h_stride, dh_stride, dx_stride, dla_stride;
    int N, T, C;
    int drop = -1;
};
cudaError_t launch_scan(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream);
cudaError_t launch_scan_backward(const ScanGradArgs& a, bool bf16, bool gate_bf16,
                                 cudaStream_t stream);
cudaError_t launch_scan_step(const ScanArgs& a, bool bf16, bool gate_bf16, cudaStream_t stream);

// Group norm over heads (strides in elements; y is dx in the backward form).
struct GroupNormArgs {
    const void *x, *z, *dy;
    void *y, *dz;
    const float *weight, *bias;
    int64_t x_stride, z_stride, dy_stride, y_stride, dz_stride;
    int T, H, d, weight_heads;
    bool centred, silu, bf16;
    float eps;
};
cudaError_t launch_group_norm(const GroupNormArgs& a, cudaStream_t stream);
size_t group_norm_backward_workspace_bytes(int T, int H, int d, int weight_heads, bool bf16);
cudaError_t launch_group_norm_backward(const GroupNormArgs& a, float* dweight, float* dbias,
                                       void* workspace, cudaStream_t stream);

// Gradients of the front end.
struct FrontendGradArgs {
    const void* x[3];     // q_raw, k_raw, v_raw
    const void* dout[3];  // dq, dk, dv
    void* dx[3];
    const float *w, *a, *b, *dlog_alpha, *dbeta;
    float *dw, *da, *db;
    const int32_t* cu_seqlens;
    int N, T, H_qk, H_v;
    bool bf16, silu;
    float eps;
};
size_t frontend_backward_workspace_bytes(int T, int H_qk, int H_v);
cudaError_t launch_frontend_backward(const FrontendGradArgs& a, void* workspace,
                                     cudaStream_t stream);

cudaError_t read_and_clear_status(unsigned int* status, cudaStream_t stream);

// Fixed-size device scratch used by gdn_prefill_noalloc (bytes, and its address
// on the current device; the address is looked up once per device).
size_t noalloc_scratch_bytes();
cudaError_t noalloc_scratch_address(void** out);

}  // namespace gdn
