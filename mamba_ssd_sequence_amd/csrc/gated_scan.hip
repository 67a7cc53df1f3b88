// ssd_gated_scan, ssd_gated_scan_step, ssd_gated_scan_backward: the linear
// recurrence with a gate for every channel and token,
//     a = exp(-softplus(A_P)) = 1 / (1 + e^{A_P}),  g = sigmoid(I_P) or 1,
//     h_t = a_t h_{t-1} + beta_t g_t x_t,           y = h,
// beta = 1, 1 - a or sqrt(1 - a^2), and its gradients by the reverse recurrence
//     lam_t = dy_t + a_{t+1} lam_{t+1}.
#include "block.h"
#include "common.h"

#include <type_traits>

namespace ssd {

// e^x for x <= 0 to about 1.5 ulp: 2^(x log2 e) on the hardware exponential
// with the rounding of the product and of log2 e put back to first order.
// Below -104 the result is 0; NaN stays NaN.
__device__ __forceinline__ float exp_neg(float x) {
  x = x < -104.f ? -104.f : x;
  const float t = x * LOG2E;
  const float lo = fmaf(x, 1.925963033500011e-08f, fmaf(x, LOG2E, -t));  // x log2 e - t
  const float e = exp2_fast(t);
  return fmaf(e, lo * 0.6931471805599453f, e);
}

// sigmoid(x) and 1 - sigmoid(x) = sigmoid(-x).  The smaller of the two is
// e / (1 + e) with e = e^{-|x|} and has its own relative accuracy; the larger
// is one minus it, a single rounding: a decay near 1 is then right to half an
// ulp, without the bias of a reciprocal that a thousand tokens would add up.
__device__ __forceinline__ void sigmoid_pair(float x, float& s, float& rest) {
  const float e = exp_neg(-fabsf(x));
  const float small = e * __builtin_amdgcn_rcpf(1.f + e);
  const float large = 1.f - small;
  s = x > 0.f ? large : small;
  rest = x > 0.f ? small : large;
}

__device__ __forceinline__ float sigmoid_v(float x) {
  float s, rest;
  sigmoid_pair(x, s, rest);
  return s;
}

enum { IN_PLAIN = 0, IN_CONVEX = 1, IN_UNIT = 2 };

// a, 1 - a, beta(a) and, for the backward pass, d beta / d A_P
template <int SCALE>
__device__ __forceinline__ void decay_of(float A, float& a, float& rest, float& beta, float& dbeta) {
  sigmoid_pair(A, rest, a);
  if constexpr (SCALE == IN_PLAIN) {
    beta = 1.f;
    dbeta = 0.f;
  } else if constexpr (SCALE == IN_CONVEX) {
    beta = rest;
    dbeta = a * rest;
  } else {
    // beta = sqrt(q), dbeta = a^2 (1 - a) / beta, q = 1 - a^2 without cancellation
    const float q = rest * (1.f + a);
    const float inv = q == 0.f ? 0.f : __builtin_amdgcn_rsqf(q);
    beta = q * inv;
    dbeta = a * a * rest * inv;
  }
}

// One thread per channel, a token after the other.
template <typename T, int SCALE>
__global__ __launch_bounds__(64) void k_gated_scan(const T* __restrict__ x, const T* __restrict__ A,
                                                   const T* __restrict__ I,
                                                   const float* __restrict__ h0, int64_t N,
                                                   int64_t DH, int64_t slabs, float* __restrict__ y,
                                                   float* __restrict__ hf) {
  const int64_t bh = blockIdx.x / slabs;
  const int64_t c = (blockIdx.x - bh * slabs) * 64 + threadIdx.x;
  if (c >= DH) return;
  float h = h0 ? h0[bh * DH + c] : 0.f;
  int64_t at = bh * N * DH + c;
  for (int64_t t = 0; t < N; ++t, at += DH) {
    float a, rest, beta, db;
    decay_of<SCALE>(Elem<T>::ld(A, at), a, rest, beta, db);
    const float g = I ? sigmoid_v(Elem<T>::ld(I, at)) : 1.f;
    h = fmaf(a, h, beta * g * Elem<T>::ld(x, at));
    y[at] = h;
  }
  if (hf) hf[bh * DH + c] = h;
}

template <typename T, int SCALE>
__global__ __launch_bounds__(64) void k_gated_scan_bwd(
    const T* __restrict__ x, const T* __restrict__ A, const T* __restrict__ I,
    const float* __restrict__ h0, const float* __restrict__ y, const float* __restrict__ dy,
    const float* __restrict__ dlast, int64_t N, int64_t DH, int64_t slabs, float* __restrict__ dx,
    float* __restrict__ dA, float* __restrict__ dI, float* __restrict__ dh0) {
  const int64_t bh = blockIdx.x / slabs;
  const int64_t c = (blockIdx.x - bh * slabs) * 64 + threadIdx.x;
  if (c >= DH) return;
  float carry = dlast ? dlast[bh * DH + c] : 0.f;  // a_{t+1} lam_{t+1}
  int64_t at = (bh * N + N - 1) * DH + c;
  for (int64_t t = N - 1; t >= 0; --t, at -= DH) {
    float a, rest, beta, db;
    decay_of<SCALE>(Elem<T>::ld(A, at), a, rest, beta, db);
    const float g = I ? sigmoid_v(Elem<T>::ld(I, at)) : 1.f;
    const float xv = Elem<T>::ld(x, at);
    const float prev = t ? y[at - DH] : (h0 ? h0[bh * DH + c] : 0.f);
    const float lam = dy[at] + carry;
    dx[at] = lam * beta * g;
    dA[at] = lam * (db * g * xv - a * rest * prev);
    if (dI) dI[at] = lam * beta * xv * g * (1.f - g);
    carry = a * lam;
  }
  if (dh0) dh0[bh * DH + c] = carry;
}

template <typename T, int SCALE>
__global__ __launch_bounds__(256) void k_gated_step(const T* __restrict__ x, const T* __restrict__ A,
                                                    const T* __restrict__ I, const float* state,
                                                    int64_t n, float* out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  float a, rest, beta, db;
  decay_of<SCALE>(Elem<T>::ld(A, i), a, rest, beta, db);
  const float g = I ? sigmoid_v(Elem<T>::ld(I, i)) : 1.f;
  out[i] = fmaf(a, state[i], beta * g * Elem<T>::ld(x, i));
}

size_t gated_scan_floats(int64_t, int64_t, int64_t) { return 0; }
size_t gated_scan_backward_floats(int64_t, int64_t, int64_t) { return 0; }

// calls f<T, SCALE>()
template <typename F>
static hipError_t by_type(bool bf16, int scale, F&& f) {
  auto with = [&](auto t) {
    switch (scale) {
      case IN_PLAIN: return f(t, std::integral_constant<int, IN_PLAIN>{});
      case IN_CONVEX: return f(t, std::integral_constant<int, IN_CONVEX>{});
      default: return f(t, std::integral_constant<int, IN_UNIT>{});
    }
  };
  return bf16 ? with(uint16_t{}) : with(float{});
}

hipError_t launch_gated_scan(bool bf16, int scale, const void* x, const void* A, const void* I,
                             const float* h0, int64_t BH, int64_t N, int64_t DH, float* y,
                             float* hf, float*, hipStream_t stream) {
  const int64_t slabs = (DH + 63) / 64;
  return by_type(bf16, scale, [&](auto t, auto sc) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_gated_scan<T, sc.value>), dim3((unsigned)(BH * slabs)), dim3(64), 0, stream,
                       (const T*)x, (const T*)A, (const T*)I, h0, N, DH, slabs, y, hf);
    return hipGetLastError();
  });
}

hipError_t launch_gated_scan_step(bool bf16, int scale, const void* x, const void* A,
                                  const void* I, const float* state, int64_t n, float* out,
                                  hipStream_t stream) {
  return by_type(bf16, scale, [&](auto t, auto sc) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_gated_step<T, sc.value>), dim3((unsigned)((n + 255) / 256)), dim3(256), 0,
                       stream, (const T*)x, (const T*)A, (const T*)I, state, n, out);
    return hipGetLastError();
  });
}

hipError_t launch_gated_scan_backward(bool bf16, int scale, const void* x, const void* A,
                                      const void* I, const float* h0, const float* y,
                                      const float* dy, const float* dlast, int64_t BH, int64_t N,
                                      int64_t DH, float* dx, float* dA, float* dI, float* dh0,
                                      float*, hipStream_t stream) {
  const int64_t slabs = (DH + 63) / 64;
  return by_type(bf16, scale, [&](auto t, auto sc) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_gated_scan_bwd<T, sc.value>), dim3((unsigned)(BH * slabs)), dim3(64), 0,
                       stream, (const T*)x, (const T*)A, (const T*)I, h0, y, dy, dlast, N, DH, slabs,
                       dx, dA, dI, dh0);
    return hipGetLastError();
  });
}

}  // namespace ssd
