// ssd_norm_in, ssd_norm_out and their gradients: the RMS norms, the SiLU gate
// and the residual scale at the two ends of a mixer block.
//     norm in:   r' = r + s p,  u = w r' k,  k = 1 / sqrt(mean r'^2 + eps)
//     norm out:  t = y silu(z), o = w t k   or   o = w silu(z) y k,
//                k over the groups of a token's channels; y in head order
//                [B,H,N,d_h], z and o in token order [B,N,H d_h]
#include "block.h"
#include "common.h"

namespace ssd {

constexpr int NT = 256;  // threads of a workgroup

template <typename T> struct Out;
template <> struct Out<float> {
  static __device__ __forceinline__ void st(float* p, int64_t i, float v) { p[i] = v; }
};
template <> struct Out<uint16_t> {
  static __device__ __forceinline__ void st(uint16_t* p, int64_t i, float v) {
    reinterpret_cast<__bf16*>(p)[i] = f32_to_bf16(v);
  }
};

// the sums of two values over the workgroup
__device__ __forceinline__ void block_sum2(float& a, float& b) {
  __shared__ float sa[NT / WAVE], sb[NT / WAVE];
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    a += __shfl_xor(a, o, WAVE);
    b += __shfl_xor(b, o, WAVE);
  }
  __syncthreads();  // an earlier sum's slots are read
  if (threadIdx.x % WAVE == 0) {
    sa[threadIdx.x / WAVE] = a;
    sb[threadIdx.x / WAVE] = b;
  }
  __syncthreads();
  a = b = 0.f;
#pragma unroll
  for (int i = 0; i < NT / WAVE; ++i) {
    a += sa[i];
    b += sb[i];
  }
}

// 1 / sqrt(sum / E + eps)
__device__ __forceinline__ float inv_rms(float sum, int64_t E, float eps) {
  return 1.f / sqrtf(sum / (float)E + eps);
}

__device__ __forceinline__ float sigmoid_f(float z) {
  const float e = expf(-fabsf(z));
  const float r = 1.f / (1.f + e);
  return z >= 0.f ? r : e * r;
}

// a workgroup per row, the row read twice
template <typename T>
__global__ __launch_bounds__(NT) void k_norm_in(const float* __restrict__ r, const T* __restrict__ p,
                                                const float* __restrict__ s,
                                                const float* __restrict__ w, int64_t rows, int64_t E,
                                                float eps, float* __restrict__ r_out,
                                                T* __restrict__ u) {
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t at = row * E;
    auto value = [&](int64_t e) {
      const float v = r[at + e];
      if (!p) return v;
      return fmaf(s ? s[e] : 1.f, Elem<T>::ld(p, at + e), v);
    };
    float sum = 0.f, none = 0.f;
    for (int64_t e = threadIdx.x; e < E; e += NT) {
      const float v = value(e);
      if (p) r_out[at + e] = v;
      sum = fmaf(v, v, sum);
    }
    block_sum2(sum, none);
    const float k = inv_rms(sum, E, eps);
    for (int64_t e = threadIdx.x; e < E; e += NT) Out<T>::st(u, at + e, value(e) * k * w[e]);
  }
}

// rows of a workgroup's share: its partial sums go to part[blockIdx.x]
template <typename T>
__global__ __launch_bounds__(NT) void k_norm_in_bwd(
    const T* __restrict__ du, const float* __restrict__ dr_out, const float* __restrict__ r,
    const T* __restrict__ p, const float* __restrict__ s, const float* __restrict__ w, int64_t rows,
    int64_t E, float eps, float* __restrict__ dr, float* __restrict__ dp, float* __restrict__ part) {
  float* dw = part + (int64_t)blockIdx.x * E;
  float* ds = part + (int64_t)(gridDim.x + blockIdx.x) * E;
  for (int64_t e = threadIdx.x; e < E; e += NT) {
    dw[e] = 0.f;
    if (s) ds[e] = 0.f;
  }
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t at = row * E;
    float sq = 0.f, cr = 0.f;
    for (int64_t e = threadIdx.x; e < E; e += NT) {
      const float v = r[at + e];
      sq = fmaf(v, v, sq);
      cr = fmaf(Elem<T>::ld(du, at + e) * w[e], v, cr);
    }
    block_sum2(sq, cr);
    const float k = inv_rms(sq, E, eps), m = k * k * k * (cr / (float)E);
    for (int64_t e = threadIdx.x; e < E; e += NT) {
      const float v = r[at + e], d = Elem<T>::ld(du, at + e);
      const float g = fmaf(-m, v, fmaf(k, d * w[e], dr_out ? dr_out[at + e] : 0.f));
      dr[at + e] = g;
      dw[e] = fmaf(d, v * k, dw[e]);
      if (s) {
        dp[at + e] = s[e] * g;
        ds[e] = fmaf(g, Elem<T>::ld(p, at + e), ds[e]);
      }
    }
  }
}

// out[e] = sum over n partial rows, in their order
__global__ __launch_bounds__(NT) void k_sum_rows(const float* __restrict__ part, int64_t n, int64_t E,
                                                 float* __restrict__ out) {
  const int64_t e = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (e >= E) return;
  float sum = 0.f;
  for (int64_t i = 0; i < n; ++i) sum += part[i * E + e];
  out[e] = sum;
}

// the arrays' places of channel e of a unit (token bn, group g of EG channels)
struct Place {
  int64_t H, N, DH, EG;
  __device__ __forceinline__ int64_t y(int64_t bn, int64_t e) const {
    const int64_t b = bn / N, n = bn - b * N, h = e / DH;
    return ((b * H + h) * N + n) * DH + (e - h * DH);
  }
};

template <typename T>
__global__ __launch_bounds__(NT) void k_norm_out(const float* __restrict__ y, const T* __restrict__ z,
                                                 const float* __restrict__ w, int64_t units,
                                                 int64_t groups, Place pl, bool gate_first, float eps,
                                                 T* __restrict__ o) {
  const int64_t E = pl.EG * groups;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t bn = unit / groups, e0 = (unit - bn * groups) * pl.EG;
    float sum = 0.f, none = 0.f;
    for (int64_t e = e0 + threadIdx.x; e < e0 + pl.EG; e += NT) {
      float t = y[pl.y(bn, e)];
      if (gate_first) {
        const float zv = Elem<T>::ld(z, bn * E + e);
        t *= zv * sigmoid_f(zv);
      }
      sum = fmaf(t, t, sum);
    }
    block_sum2(sum, none);
    const float k = inv_rms(sum, pl.EG, eps);
    for (int64_t e = e0 + threadIdx.x; e < e0 + pl.EG; e += NT) {
      const float zv = Elem<T>::ld(z, bn * E + e);
      Out<T>::st(o, bn * E + e, y[pl.y(bn, e)] * (zv * sigmoid_f(zv)) * k * w[e]);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(NT) void k_norm_out_bwd(
    const T* __restrict__ d_out, const float* __restrict__ y, const T* __restrict__ z,
    const float* __restrict__ w, int64_t tokens, int64_t groups, Place pl, bool gate_first, float eps,
    float* __restrict__ dy, float* __restrict__ dz, float* __restrict__ part) {
  const int64_t E = pl.EG * groups;
  float* dw = part + (int64_t)blockIdx.x * E;
  for (int64_t e = threadIdx.x; e < E; e += NT) dw[e] = 0.f;
  for (int64_t bn = blockIdx.x; bn < tokens; bn += gridDim.x)
    for (int64_t e0 = 0; e0 < E; e0 += pl.EG) {
      __syncthreads();  // dw[e] of the next group belongs to another thread
      float sq = 0.f, ct = 0.f;
      for (int64_t e = e0 + threadIdx.x; e < e0 + pl.EG; e += NT) {
        const float zv = Elem<T>::ld(z, bn * E + e), gate = zv * sigmoid_f(zv), yv = y[pl.y(bn, e)];
        const float t = gate_first ? yv * gate : yv;
        sq = fmaf(t, t, sq);
        ct = fmaf(Elem<T>::ld(d_out, bn * E + e) * w[e] * (gate_first ? 1.f : gate), t, ct);
      }
      block_sum2(sq, ct);
      const float k = inv_rms(sq, pl.EG, eps), m = k * k * k * (ct / (float)pl.EG);
      for (int64_t e = e0 + threadIdx.x; e < e0 + pl.EG; e += NT) {
        const float zv = Elem<T>::ld(z, bn * E + e), sig = sigmoid_f(zv), gate = zv * sig;
        const float slope = sig * (1.f + zv * (1.f - sig));
        const int64_t ya = pl.y(bn, e);
        const float yv = y[ya], d = Elem<T>::ld(d_out, bn * E + e);
        const float t = gate_first ? yv * gate : yv;
        const float dt = k * d * w[e] * (gate_first ? 1.f : gate) - m * t;
        dy[ya] = gate_first ? dt * gate : dt;
        dz[bn * E + e] = gate_first ? dt * yv * slope : d * w[e] * yv * k * slope;
        dw[e] = fmaf(d, t * k * (gate_first ? 1.f : gate), dw[e]);
      }
    }
}

static unsigned grid_of(int64_t rows) { return (unsigned)(rows < 2048 ? rows : 2048); }

hipError_t launch_norm_in(bool bf16, const float* r, const void* p, const float* s, const float* w,
                          int64_t rows, int64_t E, float eps, float* r_out, void* u,
                          hipStream_t stream) {
  auto go = [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_norm_in<T>), dim3(grid_of(rows)), dim3(NT), 0, stream, r, (const T*)p, s, w,
                       rows, E, eps, r_out, (T*)u);
    return hipGetLastError();
  };
  return bf16 ? go(uint16_t{}) : go(float{});
}

static int64_t parts_of(int64_t rows) { return rows < 512 ? rows : 512; }

size_t norm_in_backward_floats(int64_t rows, int64_t E) { return (size_t)(2 * parts_of(rows) * E); }

hipError_t launch_norm_in_backward(bool bf16, const void* du, const float* dr_out, const float* r,
                                   const void* p, const float* s, const float* w, int64_t rows,
                                   int64_t E, float eps, float* dr, float* dp, float* dw, float* ds,
                                   float* ws, hipStream_t stream) {
  const int64_t n = parts_of(rows);
  auto go = [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_norm_in_bwd<T>), dim3((unsigned)n), dim3(NT), 0, stream, (const T*)du, dr_out,
                       r, (const T*)p, s, w, rows, E, eps, dr, dp, ws);
    return hipGetLastError();
  };
  hipError_t e = hipSuccess;
  if (n) e = bf16 ? go(uint16_t{}) : go(float{});
  const unsigned grid = (unsigned)((E + NT - 1) / NT);
  if (e == hipSuccess) {
    hipLaunchKernelGGL(k_sum_rows, dim3(grid), dim3(NT), 0, stream, ws, n, E, dw);
    e = hipGetLastError();
  }
  if (e == hipSuccess && s) {
    hipLaunchKernelGGL(k_sum_rows, dim3(grid), dim3(NT), 0, stream, ws + n * E, n, E, ds);
    e = hipGetLastError();
  }
  return e;
}

hipError_t launch_norm_out(bool bf16, bool gate_first, const float* y, const void* z,
                           const float* w, int64_t B, int64_t H, int64_t N, int64_t DH,
                           int64_t groups, float eps, void* o, hipStream_t stream) {
  const Place pl{H, N, DH, H / groups * DH};
  auto go = [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_norm_out<T>), dim3(grid_of(B * N * groups)), dim3(NT), 0, stream, y,
                       (const T*)z, w, B * N * groups, groups, pl, gate_first, eps, (T*)o);
    return hipGetLastError();
  };
  return bf16 ? go(uint16_t{}) : go(float{});
}

size_t norm_out_backward_floats(int64_t B, int64_t H, int64_t N, int64_t DH, int64_t) {
  return (size_t)(parts_of(B * N) * H * DH);
}

hipError_t launch_norm_out_backward(bool bf16, bool gate_first, const void* d_out, const float* y,
                                    const void* z, const float* w, int64_t B, int64_t H, int64_t N,
                                    int64_t DH, int64_t groups, float eps, float* dy, float* dz,
                                    float* dw, float* ws, hipStream_t stream) {
  const Place pl{H, N, DH, H / groups * DH};
  const int64_t n = parts_of(B * N), E = H * DH;
  auto go = [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_norm_out_bwd<T>), dim3((unsigned)n), dim3(NT), 0, stream, (const T*)d_out, y,
                       (const T*)z, w, B * N, groups, pl, gate_first, eps, dy, dz, ws);
    return hipGetLastError();
  };
  hipError_t e = hipSuccess;
  if (n) e = bf16 ? go(uint16_t{}) : go(float{});
  if (e == hipSuccess) {
    hipLaunchKernelGGL(k_sum_rows, dim3((unsigned)((E + NT - 1) / NT)), dim3(NT), 0, stream, ws, n, E,
                       dw);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace ssd
