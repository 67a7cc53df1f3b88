// ssd_norm_in, ssd_norm_out and their gradients: the RMS norms, the SiLU gate
// and the residual scale at the two ends of a mixer block.
//     norm in:   r' = r + s p,  u = w r' k,  k = 1 / sqrt(mean r'^2 + eps)
//     norm out:  t = y silu(z), o = w t k   or   o = w silu(z) y k,
//                k over the groups of a token's channels; y in head order
//                [B,H,N,d_h], z and o in token order [B,N,H d_h]
// All four are bound by memory: every array is read once and written once, a
// row (a token's group of channels) lives in registers between its sums and its
// outputs, and norm out reads y where the mixer left it.
//
// A row belongs to TPR threads, each with NV pieces of V channels; a workgroup
// holds NT / TPR rows at a time and walks over the tokens, so that the weights
// (and, backwards, the weights' gradients) stay in registers.  The gradients'
// per-workgroup sums go to the workspace and are added by k_sum_parts, in an
// order that the sizes alone fix.
#include "block.h"
#include "common.h"
#include "elem.h"

#include <type_traits>

namespace ssd {

template <int V_, int TPR_, int NV_>
struct Row {
  static constexpr int V = V_, TPR = TPR_, NV = NV_;
  static constexpr int NT = TPR > 512 ? TPR : 512;  // threads of a workgroup
  static constexpr int SLOTS = NT / TPR;            // rows it holds
};

// Which rows a workgroup takes: `gpw` groups of `tpw` tokens at a time; there
// are `blocks` workgroups for the groups of a token, and `parts` sets of them
// that share the tokens.
struct Geo {
  int64_t tokens;
  int groups, EG;  // groups of a token, channels of a group
  int gpw, tpw, blocks, parts;
  bool nt_in, nt_out;  // nontemporal loads, stores
};

// A thread's place: its row's group and token, its channels.
template <typename R>
struct Seat {
  int slot, lane, g, part;
  bool seated;  // the slot has a row at all
  __device__ __forceinline__ explicit Seat(const Geo& q) {
    slot = threadIdx.x / R::TPR;
    if constexpr (R::TPR >= WAVE) slot = __builtin_amdgcn_readfirstlane(slot);  // rows have uniform addresses
    lane = threadIdx.x % R::TPR;
    part = blockIdx.x / q.blocks;
    g = (blockIdx.x - part * q.blocks) * q.gpw + slot % q.gpw;
    seated = g < q.groups && slot / q.gpw < q.tpw;
    if (!seated) g = 0;
  }
  // the row's channel of piece k, or `none` past its end
  __device__ __forceinline__ int channel(int k) const { return (k * R::TPR + lane) * R::V; }
};

// Sums of a and b over the TPR threads of each row.  With more than a wave a
// row, through LDS: `turn` alternates between two sets of slots, so that one
// barrier a call is enough.  Every thread of the workgroup calls it.
template <typename R>
__device__ __forceinline__ void row_sums(float& a, float& b, int turn) {
#pragma unroll
  for (int o = 1; o < (R::TPR < WAVE ? R::TPR : WAVE); o <<= 1) {
    a += __shfl_xor(a, o, WAVE);
    b += __shfl_xor(b, o, WAVE);
  }
  if constexpr (R::TPR > WAVE) {
    __shared__ float2 sums[2][R::NT / WAVE];
    const int wave = threadIdx.x / WAVE;
    if (threadIdx.x % WAVE == 0) sums[turn][wave] = make_float2(a, b);
    __syncthreads();
    constexpr int W = R::TPR / WAVE;
    const float2* mine = sums[turn] + wave / W * W;
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      a += mine[i].x;
      b += mine[i].y;
    }
  }
}

// 1 / sqrt(sum / n + eps)
__device__ __forceinline__ float inv_rms(float sum, float inv_n, float eps) {
  return 1.f / sqrtf(fmaf(sum, inv_n, eps));
}

template <typename T, typename R>
__global__ __launch_bounds__(R::NT) void k_norm_in(const float* __restrict__ r, const T* __restrict__ p,
                                                   const float* __restrict__ s,
                                                   const float* __restrict__ w, Geo q, float eps,
                                                   float* __restrict__ r_out, T* __restrict__ u) {
  constexpr int V = R::V, NV = R::NV;
  const Seat<R> seat(q);
  const float inv_n = 1.f / (float)q.EG;
  Raw<float, V> rw[NV], rs[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = seat.channel(k) < q.EG ? seat.channel(k) : 0;
    rw[k].load(w + e);
    if (s) rs[k].load(s + e);
  }
  int turn = 0;
  for (int64_t t = (int64_t)seat.part * q.tpw; t < q.tokens; t += (int64_t)q.parts * q.tpw, turn ^= 1) {
    const int64_t row = t + seat.slot;
    const bool live = row < q.tokens;
    const int64_t at = (live ? row : q.tokens - 1) * q.EG;
    Raw<float, V> rr[NV];
    Raw<T, V> rp[NV];
    either(q.nt_in, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = seat.channel(k) < q.EG ? seat.channel(k) : 0;
        rr[k].template load<nt.value>(r + at + e);
        if (p) rp[k].template load<nt.value>(p + at + e);
      }
    });
    float x[NV][V], sum = 0.f, none = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = seat.channel(k) < q.EG;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float y = rr[k].get(v);
        if (p) y = s ? fmaf(rs[k].get(v), rp[k].get(v), y) : y + rp[k].get(v);
        x[k][v] = y;
        sum = in ? fmaf(y, y, sum) : sum;
      }
      if (p && live && in)
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(r_out + at + seat.channel(k), x[k]); });
    }
    row_sums<R>(sum, none, turn);
    const float inv = inv_rms(sum, inv_n, eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[k][v] = x[k][v] * inv * rw[k].get(v);
      if (live && seat.channel(k) < q.EG)
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(u + at + seat.channel(k), x[k]); });
    }
  }
}

// The sums of the workgroup's rows, channel by channel, to `part` (the group's
// channels of this workgroup's partial sums): the slots of one group are added
// in their order.
template <typename R>
__device__ __forceinline__ void store_part(const Seat<R>& seat, const Geo& q, const float (&d)[R::NV][R::V],
                                           float* part) {
  constexpr int V = R::V, NV = R::NV, L = R::TPR * NV * V;
  if constexpr (R::SLOTS == 1) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (seat.channel(k) < q.EG) store_row<V>(part + seat.channel(k), d[k]);
  } else {
    __shared__ float sums[R::SLOTS * L];
    __syncthreads();  // an earlier call's sums are read
#pragma unroll
    for (int k = 0; k < NV; ++k) store_row<V>(sums + seat.slot * L + seat.channel(k), d[k]);
    __syncthreads();
    if (seat.seated && seat.slot < q.gpw)
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = d[k][v];
        for (int i = 1; i < q.tpw; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) sum[v] += sums[(seat.slot + i * q.gpw) * L + seat.channel(k) + v];
        if (seat.channel(k) < q.EG) store_row<V>(part + seat.channel(k), sum);
      }
  }
}

template <typename T, typename R>
__global__ __launch_bounds__(R::NT) void k_norm_in_bwd(
    const T* __restrict__ du, const float* __restrict__ dr_out, const float* __restrict__ r,
    const T* __restrict__ p, const float* __restrict__ s, const float* __restrict__ w, Geo q, float eps,
    float* __restrict__ dr, float* __restrict__ dp, float* __restrict__ part) {
  constexpr int V = R::V, NV = R::NV;
  const Seat<R> seat(q);
  const float inv_n = 1.f / (float)q.EG;
  Raw<float, V> rw[NV], rs[NV];
  float dw[NV][V], ds[NV][V];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = seat.channel(k) < q.EG ? seat.channel(k) : 0;
    rw[k].load(w + e);
    if (s) rs[k].load(s + e);
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = ds[k][v] = 0.f;
  }
  int turn = 0;
  for (int64_t t = (int64_t)seat.part * q.tpw; t < q.tokens; t += (int64_t)q.parts * q.tpw, turn ^= 1) {
    const int64_t row = t + seat.slot;
    const bool live = row < q.tokens;
    const int64_t at = (live ? row : q.tokens - 1) * q.EG;
    Raw<float, V> rr[NV], ro[NV];
    Raw<T, V> rp[NV], rd[NV];
    either(q.nt_in, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = seat.channel(k) < q.EG ? seat.channel(k) : 0;
        rr[k].template load<nt.value>(r + at + e);
        rd[k].template load<nt.value>(du + at + e);
        if (dr_out) ro[k].template load<nt.value>(dr_out + at + e);
        if (s) rp[k].template load<nt.value>(p + at + e);
      }
    });
    float sq = 0.f, cr = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = seat.channel(k) < q.EG;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = rr[k].get(v);
        sq = in ? fmaf(y, y, sq) : sq;
        cr = in ? fmaf(rd[k].get(v) * rw[k].get(v), y, cr) : cr;
      }
    }
    row_sums<R>(sq, cr, turn);
    const float inv = inv_rms(sq, inv_n, eps), m = inv * inv * inv * (cr * inv_n);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = live && seat.channel(k) < q.EG;
      float g[V], h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = rr[k].get(v), d = rd[k].get(v);
        g[v] = fmaf(-m, y, inv * (d * rw[k].get(v)));
        if (dr_out) g[v] += ro[k].get(v);
        dw[k][v] = in ? fmaf(d, y * inv, dw[k][v]) : dw[k][v];
        if (s) {
          h[v] = rs[k].get(v) * g[v];
          ds[k][v] = in ? fmaf(g[v], rp[k].get(v), ds[k][v]) : ds[k][v];
        }
      }
      if (in) {
        either(q.nt_out, [&](auto nt) {
          store_row<V, nt.value>(dr + at + seat.channel(k), g);
          if (s) store_row<V, nt.value>(dp + at + seat.channel(k), h);
        });
      }
    }
  }
  store_part<R>(seat, q, dw, part + (int64_t)seat.part * q.EG);
  if (s) store_part<R>(seat, q, ds, part + (int64_t)(q.parts + seat.part) * q.EG);
}

// out[i][e] = sum over n partial rows of set i, e < E: a workgroup takes 32
// columns, its 32 row slices of lanes add every 32nd row, then each other.
__global__ __launch_bounds__(1024) void k_sum_parts(const float* __restrict__ part, int n, int64_t E,
                                                    float* __restrict__ out0, float* __restrict__ out1) {
  __shared__ float sums[32][32];
  const int64_t e = (int64_t)blockIdx.x * 32 + threadIdx.x % 32;
  const int slice = threadIdx.x / 32;
  const float* src = part + (int64_t)blockIdx.y * n * E + (e < E ? e : 0);
  float sum = 0.f;
#pragma unroll 8
  for (int i = slice; i < n; i += 32) sum += src[i * E];
  sums[slice][threadIdx.x % 32] = sum;
  __syncthreads();
  if (slice || e >= E) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) sum += sums[i][threadIdx.x];
  (blockIdx.y ? out1 : out0)[e] = sum;
}

// The places of a row of y in head order: channel e0 + e of the token is
// element y[off] of the token's first head's row; off is computed once, the
// token's row (`base`) for every token.
struct Heads {
  int64_t H, N, DH;
  __device__ __forceinline__ int64_t off(int e) const {
    const int d = (int)DH, h = e / d;
    return (int64_t)h * N * DH + (e - h * d);
  }
  __device__ __forceinline__ int64_t base(int64_t token) const {
    const unsigned n = (unsigned)N, b = (unsigned)token / n;
    return ((int64_t)b * H * N + ((unsigned)token - b * n)) * DH;
  }
};

template <typename T, typename R, bool FIRST>
__global__ __launch_bounds__(R::NT) void k_norm_out(const float* __restrict__ y, const T* __restrict__ z,
                                                    const float* __restrict__ w, Geo q, Heads hd,
                                                    float eps, T* __restrict__ o) {
  constexpr int V = R::V, NV = R::NV;
  const Seat<R> seat(q);
  const int64_t E = (int64_t)q.groups * q.EG;
  const int e0 = seat.g * q.EG;
  const float inv_n = 1.f / (float)q.EG;
  Raw<float, V> rw[NV];
  int64_t off[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = e0 + (seat.channel(k) < q.EG ? seat.channel(k) : 0);
    rw[k].load(w + e);
    off[k] = hd.off(e);
  }
  int turn = 0;
  for (int64_t t = (int64_t)seat.part * q.tpw; t < q.tokens; t += (int64_t)q.parts * q.tpw, turn ^= 1) {
    const int64_t mine = t + seat.slot / q.gpw, token = mine < q.tokens ? mine : q.tokens - 1;
    const bool live = seat.seated && mine < q.tokens;
    const int64_t base = hd.base(token), at = token * E + e0;
    Raw<float, V> ry[NV];
    Raw<T, V> rz[NV];
    either(q.nt_in, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rz[k].template load<nt.value>(z + at + (seat.channel(k) < q.EG ? seat.channel(k) : 0));
        ry[k].template load<nt.value>(y + base + off[k]);
      }
    });
    float x[NV][V], sum = 0.f, none = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = seat.channel(k) < q.EG;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v);
        x[k][v] = yv * (zv * sigmoid_v(zv));
        const float n = FIRST ? x[k][v] : yv;
        sum = in ? fmaf(n, n, sum) : sum;
      }
    }
    row_sums<R>(sum, none, turn);
    const float inv = inv_rms(sum, inv_n, eps);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[k][v] = x[k][v] * inv * rw[k].get(v);
      if (live && seat.channel(k) < q.EG)
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(o + at + seat.channel(k), x[k]); });
    }
  }
}

template <typename T, typename R, bool FIRST>
__global__ __launch_bounds__(R::NT) void k_norm_out_bwd(
    const T* __restrict__ d_out, const float* __restrict__ y, const T* __restrict__ z,
    const float* __restrict__ w, Geo q, Heads hd, float eps, float* __restrict__ dy,
    float* __restrict__ dz, float* __restrict__ part) {
  constexpr int V = R::V, NV = R::NV;
  const Seat<R> seat(q);
  const int64_t E = (int64_t)q.groups * q.EG;
  const int e0 = seat.g * q.EG;
  const float inv_n = 1.f / (float)q.EG;
  Raw<float, V> rw[NV];
  float dw[NV][V];
  int64_t off[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int e = e0 + (seat.channel(k) < q.EG ? seat.channel(k) : 0);
    rw[k].load(w + e);
    off[k] = hd.off(e);
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = 0.f;
  }
  int turn = 0;
  for (int64_t t = (int64_t)seat.part * q.tpw; t < q.tokens; t += (int64_t)q.parts * q.tpw, turn ^= 1) {
    const int64_t mine = t + seat.slot / q.gpw, token = mine < q.tokens ? mine : q.tokens - 1;
    const bool live = seat.seated && mine < q.tokens;
    const int64_t base = hd.base(token), at = token * E + e0;
    Raw<float, V> ry[NV];
    Raw<T, V> rz[NV], rd[NV];
    either(q.nt_in, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int e = seat.channel(k) < q.EG ? seat.channel(k) : 0;
        rz[k].template load<nt.value>(z + at + e);
        rd[k].template load<nt.value>(d_out + at + e);
        ry[k].template load<nt.value>(y + base + off[k]);
      }
    });
    // sig = silu'(z)'s logistic; kept between the sums and the outputs
    float sig[NV][V], sq = 0.f, ct = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = seat.channel(k) < q.EG;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v), gate = zv * (sig[k][v] = sigmoid_v(zv));
        const float x = FIRST ? yv * gate : yv, c = rd[k].get(v) * rw[k].get(v) * (FIRST ? 1.f : gate);
        sq = in ? fmaf(x, x, sq) : sq;
        ct = in ? fmaf(c, x, ct) : ct;
      }
    }
    row_sums<R>(sq, ct, turn);
    const float inv = inv_rms(sq, inv_n, eps), m = inv * inv * inv * (ct * inv_n);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = live && seat.channel(k) < q.EG;
      float gy[V], gz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v), d = rd[k].get(v), dwv = d * rw[k].get(v);
        const float gate = zv * sig[k][v], slope = sig[k][v] * fmaf(zv, 1.f - sig[k][v], 1.f);
        const float x = FIRST ? yv * gate : yv;
        const float dx = fmaf(-m, x, inv * (FIRST ? dwv : dwv * gate));
        gy[v] = FIRST ? dx * gate : dx;
        gz[v] = FIRST ? dx * yv * slope : dwv * (yv * inv) * slope;
        dw[k][v] = in ? fmaf(FIRST ? d : d * gate, x * inv, dw[k][v]) : dw[k][v];
      }
      if (in) {
        either(q.nt_out, [&](auto nt) {
          store_row<V, nt.value>(dy + base + off[k], gy);
          store_row<V, nt.value>(dz + at + seat.channel(k), gz);
        });
      }
    }
  }
  store_part<R>(seat, q, dw, part + seat.part * E + e0);
}

// ---- launches ----

// calls f(R) with the row shape for groups of EG channels: 8 channels a thread
// (4 in rows of up to 256, 16 beyond 8192, 32 beyond 16384), so that a row with
// its weights and their gradients leaves room for 16 waves a CU and more.
// `wide`: whole pieces of 4 channels (EG and the heads' width multiples of 4).
template <typename F>
static auto by_row(int64_t EG, bool wide, F&& f) {
  if (wide) {
    if (EG <= 64) return f(Row<4, 16, 1>{});
    if (EG <= 256) return f(Row<4, 64, 1>{});
    if (EG <= 512) return f(Row<4, 64, 2>{});
    if (EG <= 1024) return f(Row<4, 128, 2>{});
    if (EG <= 2048) return f(Row<4, 256, 2>{});
    if (EG <= 4096) return f(Row<4, 512, 2>{});
    if (EG <= 8192) return f(Row<4, 1024, 2>{});
    if (EG <= 16384) return f(Row<4, 1024, 4>{});
    return f(Row<4, 1024, 8>{});
  }
  if (EG <= 64) return f(Row<1, 16, 4>{});
  if (EG <= 512) return f(Row<1, 64, 8>{});
  if (EG <= 2048) return f(Row<1, 256, 8>{});
  if (EG <= 8192) return f(Row<1, 1024, 8>{});
  return f(Row<1, 1024, 32>{});
}

// Workgroups: enough to fill the 256 CUs with 2048 threads each (backwards with
// 1024, whose sums then add up over fewer parts), no more than there is work for.
// Nontemporal loads where a call moves more than the last-level cache (256 MB)
// holds, nontemporal stores too where it moves 768 MB and more (below that the
// cache still takes up much of what is written).  Norm in, E 1024 (plain / loads /
// both): 101 MB 16.0 / 18.1 / 18.4 us, 403 MB 74.3 / 61.8 / 69.3, 805 MB 150 / 149
// / 140; backwards 168 MB 33.1 / 33.4 / 35.0, 671 MB 129 / 108 / 118, 1342 MB 260 /
// 259 / 233.
template <typename R>
static Geo geo_of(R, int64_t tokens, int64_t groups, int64_t EG, bool backward, int64_t bytes) {
  Geo q{};
  q.nt_in = bytes >= CACHE_BYTES;
  q.nt_out = bytes >= 3 * CACHE_BYTES;
  q.tokens = tokens;
  q.groups = (int)groups;
  q.EG = (int)EG;
  q.gpw = groups < R::SLOTS ? (int)groups : R::SLOTS;
  q.tpw = R::SLOTS / q.gpw;
  q.blocks = (int)((groups + q.gpw - 1) / q.gpw);
  const int64_t want = (tokens + q.tpw - 1) / q.tpw;
  int64_t most = 256 * (backward ? 1024 : 2048) / R::NT / q.blocks;
  if (most < 1) most = 1;
  q.parts = (int)(want < most ? want : most);
  return q;
}

static Geo geo_by(int64_t tokens, int64_t groups, int64_t EG, bool wide, bool backward, int64_t bytes) {
  return by_row(EG, wide, [&](auto row) { return geo_of(row, tokens, groups, EG, backward, bytes); });
}

static hipError_t launch_sum_parts(const float* part, int n, int64_t E, float* out0, float* out1,
                                   hipStream_t stream) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((E + 31) / 32), out1 ? 2 : 1), dim3(1024), 0, stream, part,
                     n, E, out0, out1);
  return hipGetLastError();
}

// calls f(T, row)
template <typename F>
static hipError_t by_call(bool bf16, int64_t EG, bool wide, F&& f) {
  return by_row(EG, wide, [&](auto row) { return bf16 ? f(uint16_t{}, row) : f(float{}, row); });
}

hipError_t launch_norm_in(bool bf16, const float* r, const void* p, const float* s, const float* w,
                          int64_t rows, int64_t E, float eps, float* r_out, void* u,
                          hipStream_t stream) {
  const int64_t size = bf16 ? 2 : 4;
  return by_call(bf16, E, E % 4 == 0, [&](auto t, auto row) {
    using T = decltype(t);
    using R = decltype(row);
    const Geo q = geo_of(row, rows, 1, E, false, rows * E * (p ? 8 + 2 * size : 4 + size));
    hipLaunchKernelGGL((k_norm_in<T, R>), dim3((unsigned)q.parts), dim3(R::NT), 0, stream, r, (const T*)p,
                       s, w, q, eps, r_out, (T*)u);
    return hipGetLastError();
  });
}

size_t norm_in_backward_floats(int64_t rows, int64_t E) {
  return (size_t)(2 * geo_by(rows, 1, E, E % 4 == 0, true, 0).parts * E);
}

hipError_t launch_norm_in_backward(bool bf16, const void* du, const float* dr_out, const float* r,
                                   const void* p, const float* s, const float* w, int64_t rows,
                                   int64_t E, float eps, float* dr, float* dp, float* dw, float* ds,
                                   float* ws, hipStream_t stream) {
  const int64_t size = bf16 ? 2 : 4;
  const Geo q = geo_by(rows, 1, E, E % 4 == 0, true, rows * E * (8 + size + (dr_out ? 4 : 0) + (s ? 4 + size : 0)));
  if (rows) {
    const hipError_t e = by_call(bf16, E, E % 4 == 0, [&](auto t, auto row) {
      using T = decltype(t);
      using R = decltype(row);
      hipLaunchKernelGGL((k_norm_in_bwd<T, R>), dim3((unsigned)q.parts), dim3(R::NT), 0, stream,
                         (const T*)du, dr_out, r, (const T*)p, s, w, q, eps, dr, dp, ws);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  return launch_sum_parts(ws, rows ? q.parts : 0, E, dw, ds, stream);
}

static bool heads_wide(int64_t DH) { return DH % 4 == 0; }

hipError_t launch_norm_out(bool bf16, bool gate_first, const float* y, const void* z,
                           const float* w, int64_t B, int64_t H, int64_t N, int64_t DH,
                           int64_t groups, float eps, void* o, hipStream_t stream) {
  const int64_t EG = H / groups * DH;
  return by_call(bf16, EG, heads_wide(DH), [&](auto t, auto row) {
    using T = decltype(t);
    using R = decltype(row);
    const Geo q = geo_of(row, B * N, groups, EG, false, B * N * H * DH * (bf16 ? 8 : 12));
    auto go = [&](auto first) {
      hipLaunchKernelGGL((k_norm_out<T, R, first.value>), dim3((unsigned)(q.parts * q.blocks)), dim3(R::NT),
                         0, stream, y, (const T*)z, w, q, Heads{H, N, DH}, eps, (T*)o);
      return hipGetLastError();
    };
    return gate_first ? go(std::true_type{}) : go(std::false_type{});
  });
}

size_t norm_out_backward_floats(int64_t B, int64_t H, int64_t N, int64_t DH, int64_t groups) {
  return (size_t)(geo_by(B * N, groups, H / groups * DH, heads_wide(DH), true, 0).parts * H * DH);
}

hipError_t launch_norm_out_backward(bool bf16, bool gate_first, const void* d_out, const float* y,
                                    const void* z, const float* w, int64_t B, int64_t H, int64_t N,
                                    int64_t DH, int64_t groups, float eps, float* dy, float* dz,
                                    float* dw, float* ws, hipStream_t stream) {
  const int64_t EG = H / groups * DH, tokens = B * N;
  const Geo q = geo_by(tokens, groups, EG, heads_wide(DH), true, tokens * H * DH * (bf16 ? 16 : 20));
  if (tokens) {
    const hipError_t e = by_call(bf16, EG, heads_wide(DH), [&](auto t, auto row) {
      using T = decltype(t);
      using R = decltype(row);
      auto go = [&](auto first) {
        hipLaunchKernelGGL((k_norm_out_bwd<T, R, first.value>), dim3((unsigned)(q.parts * q.blocks)),
                           dim3(R::NT), 0, stream, (const T*)d_out, y, (const T*)z, w, q,
                           Heads{H, N, DH}, eps, dy, dz, ws);
        return hipGetLastError();
      };
      return gate_first ? go(std::true_type{}) : go(std::false_type{});
    });
    if (e != hipSuccess) return e;
  }
  return launch_sum_parts(ws, tokens ? q.parts : 0, H * DH, dw, nullptr, stream);
}

}  // namespace ssd
