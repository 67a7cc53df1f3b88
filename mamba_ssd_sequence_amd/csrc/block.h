// Internal launchers and workspace sizes of the gated linear recurrence
// (gated_scan.hip) and of the norms around a mixer block (norms.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ssd {

// The recurrence h_t = a_t h_{t-1} + beta_t g_t x_t over BH independent
// [N, DH] matrices; scale: ssd_input_scale; I, h0, hf may be NULL.
size_t gated_scan_floats(int64_t BH, int64_t N, int64_t DH);
bool gated_scan_fits(bool bf16, int64_t BH, int64_t N, int64_t DH);  // a head fits a launch
hipError_t launch_gated_scan(bool bf16, int scale, const void* x, const void* A, const void* I,
                             const float* h0, int64_t BH, int64_t N, int64_t DH, float* y,
                             float* hf, float* ws, hipStream_t stream);

// One token of n independent channels (out may be state).
hipError_t launch_gated_scan_step(bool bf16, int scale, const void* x, const void* A,
                                  const void* I, const float* state, int64_t n, float* out,
                                  hipStream_t stream);

// Its gradients; I, dI, h0, dlast, dh0 may be NULL.
size_t gated_scan_backward_floats(int64_t BH, int64_t N, int64_t DH);
bool gated_scan_backward_fits(int64_t BH, int64_t N, int64_t DH);
hipError_t launch_gated_scan_backward(bool bf16, int scale, const void* x, const void* A,
                                      const void* I, const float* h0, const float* y,
                                      const float* dy, const float* dlast, int64_t BH, int64_t N,
                                      int64_t DH, float* dx, float* dA, float* dI, float* dh0,
                                      float* ws, hipStream_t stream);

// r' = r + s p, u = w r' / rms(r'); p, s may be NULL.
hipError_t launch_norm_in(bool bf16, const float* r, const void* p, const float* s, const float* w,
                          int64_t rows, int64_t E, float eps, float* r_out, void* u,
                          hipStream_t stream);
size_t norm_in_backward_floats(int64_t rows, int64_t E);
hipError_t launch_norm_in_backward(bool bf16, const void* du, const float* dr_out, const float* r,
                                   const void* p, const float* s, const float* w, int64_t rows,
                                   int64_t E, float eps, float* dr, float* dp, float* dw, float* ds,
                                   float* ws, hipStream_t stream);

// o = norm and gate of y, from head order to token order.
hipError_t launch_norm_out(bool bf16, bool gate_first, const float* y, const void* z,
                           const float* w, int64_t B, int64_t H, int64_t N, int64_t DH,
                           int64_t groups, float eps, void* o, hipStream_t stream);
size_t norm_out_backward_floats(int64_t B, int64_t H, int64_t N, int64_t DH, int64_t groups);
hipError_t launch_norm_out_backward(bool bf16, bool gate_first, const void* d_out, const float* y,
                                    const void* z, const float* w, int64_t B, int64_t H, int64_t N,
                                    int64_t DH, int64_t groups, float eps, float* dy, float* dz,
                                    float* dw, float* ws, hipStream_t stream);

}  // namespace ssd
