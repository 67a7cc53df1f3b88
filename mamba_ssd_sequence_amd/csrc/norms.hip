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
//
// Pieces never cross a head (norm in: the row is one head): ceil(d / 4) pieces
// of 4 channels each, of which the last is moved back to end with the head.  Its
// first channels are then also the piece's before it; they count once in the
// row's sums, and are computed and written twice with the same values.
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
  // What registers hold: the weights up to 8 channels a thread, the row up to
  // 16.  Longer rows read them again (from the L2).
  static constexpr bool HOLD_W = NV * V <= 8, HOLD_ROW = NV * V <= 16;
};

// Which rows a workgroup takes: `gpw` groups of `tpw` tokens at a time; there
// are `blocks` workgroups for the groups of a token, and `parts` sets of them
// that share the tokens.
struct Geo {
  int64_t tokens;
  int groups, EG;      // groups of a token, channels of a group
  int width, pieces;   // channels of a head, pieces of a group
  int gpw, tpw, blocks, parts;
  bool nt_in, nt_out;  // nontemporal loads, stores
};

// A thread's place: its row's group and token, its pieces' channels.
template <typename R>
struct Seat {
  int slot, lane, g, part;
  bool seated;             // the slot has a row at all
  unsigned at[R::NV];      // a piece's first channel in the group (0 past the end)
  int head[R::NV];         // the head it is in
  int skip[R::NV];         // channels of it that are not its own (V: no piece)
  __device__ __forceinline__ explicit Seat(const Geo& q) {
    slot = threadIdx.x / R::TPR;
    if constexpr (R::TPR >= WAVE) slot = __builtin_amdgcn_readfirstlane(slot);  // rows have uniform addresses
    lane = threadIdx.x % R::TPR;
    part = blockIdx.x / q.blocks;
    g = (blockIdx.x - part * q.blocks) * q.gpw + slot % q.gpw;
    seated = g < q.groups && slot / q.gpw < q.tpw;
    if (!seated) g = 0;
    const int each = (q.width + R::V - 1) / R::V;
#pragma unroll
    for (int k = 0; k < R::NV; ++k) {
      const int piece = k * R::TPR + lane;
      const bool is = piece < q.pieces;
      head[k] = is ? piece / each : 0;
      const int c = is ? (piece - head[k] * each) * R::V : 0, moved = c < q.width - R::V ? c : q.width - R::V;
      at[k] = head[k] * q.width + moved;
      skip[k] = is ? c - moved : R::V;
    }
  }
  __device__ __forceinline__ bool is(int k) const { return skip[k] < R::V; }
  // the piece's place among the pieces of the row
  __device__ __forceinline__ int nominal(int k) const { return (k * R::TPR + lane) * R::V; }
};

// A long row's pieces are taken one after the other: their loads stay where they
// are written, or the registers that all of them need would go to scratch.
template <typename R>
__device__ __forceinline__ void piece_by_piece() {
  if constexpr (!R::HOLD_W) __builtin_amdgcn_sched_barrier(0);
}

// The same address, as one that nothing is known of: what is read from it is
// not kept from an earlier read.
template <typename P>
__device__ __forceinline__ P* afresh(P* p) {
  asm volatile("" : "+s"(p));
  return p;
}

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
  if constexpr (R::HOLD_W)
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      rw[k].load(element(w, seat.at[k]));
      if (s) rs[k].load(element(s, seat.at[k]));
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
        rr[k].template load<nt.value>(element(r + at, seat.at[k]));
        if (p) rp[k].template load<nt.value>(element(p + at, seat.at[k]));
      }
    });
    if constexpr (!R::HOLD_W) s = s ? afresh(s) : s;
    float x[NV][V], sum = 0.f, none = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W)
        if (s) rs[k].load(element(s, seat.at[k]));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float y = rr[k].get(v);
        if (p) y = s ? fmaf(rs[k].get(v), rp[k].get(v), y) : y + rp[k].get(v);
        x[k][v] = y;
        sum = v >= seat.skip[k] ? fmaf(y, y, sum) : sum;
      }
      if (p && live && seat.is(k))
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(element(r_out + at, seat.at[k]), x[k]); });
    }
    row_sums<R>(sum, none, turn);
    const float inv = inv_rms(sum, inv_n, eps);
    if constexpr (!R::HOLD_W) w = afresh(w);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W) rw[k].load(element(w, seat.at[k]));
#pragma unroll
      for (int v = 0; v < V; ++v) x[k][v] = x[k][v] * inv * rw[k].get(v);
      if (live && seat.is(k))
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(element(u + at, seat.at[k]), x[k]); });
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
      if (seat.is(k)) store_row<V>(element(part, seat.at[k]), d[k]);
  } else {
    __shared__ float sums[R::SLOTS * L];
    __syncthreads();  // an earlier call's sums are read
#pragma unroll
    for (int k = 0; k < NV; ++k) store_row<V>(sums + seat.slot * L + seat.nominal(k), d[k]);
    __syncthreads();
    if (seat.seated && seat.slot < q.gpw)
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        float sum[V];
#pragma unroll
        for (int v = 0; v < V; ++v) sum[v] = d[k][v];
        for (int i = 1; i < q.tpw; ++i)
#pragma unroll
          for (int v = 0; v < V; ++v) sum[v] += sums[(seat.slot + i * q.gpw) * L + seat.nominal(k) + v];
        if (seat.is(k)) store_row<V>(element(part, seat.at[k]), sum);
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
    if constexpr (R::HOLD_W) {
      rw[k].load(element(w, seat.at[k]));
      if (s) rs[k].load(element(s, seat.at[k]));
    }
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
    either(q.nt_in && R::HOLD_ROW, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rr[k].template load<nt.value>(element(r + at, seat.at[k]));
        rd[k].template load<nt.value>(element(du + at, seat.at[k]));
        if constexpr (R::HOLD_ROW) {
          if (dr_out) ro[k].template load<nt.value>(element(dr_out + at, seat.at[k]));
          if (s) rp[k].template load<nt.value>(element(p + at, seat.at[k]));
        }
      }
    });
    if constexpr (!R::HOLD_W) w = afresh(w);
    float sq = 0.f, cr = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W) rw[k].load(element(w, seat.at[k]));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = rr[k].get(v), c = rd[k].get(v) * rw[k].get(v);
        sq = v >= seat.skip[k] ? fmaf(y, y, sq) : sq;
        cr = v >= seat.skip[k] ? fmaf(c, y, cr) : cr;
      }
    }
    row_sums<R>(sq, cr, turn);
    const float inv = inv_rms(sq, inv_n, eps), m = inv * inv * inv * (cr * inv_n);
    if constexpr (!R::HOLD_W) {
      w = afresh(w);
      s = s ? afresh(s) : s;
    }
    if constexpr (!R::HOLD_ROW) {
      r = afresh(r);
      du = afresh(du);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W) {
        rw[k].load(element(w, seat.at[k]));
        if (s) rs[k].load(element(s, seat.at[k]));
      }
      if constexpr (!R::HOLD_ROW) {
        rr[k].load(element(r + at, seat.at[k]));
        rd[k].load(element(du + at, seat.at[k]));
        if (dr_out) ro[k].load(element(dr_out + at, seat.at[k]));
        if (s) rp[k].load(element(p + at, seat.at[k]));
      }
      float g[V], h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = rr[k].get(v), d = rd[k].get(v);
        g[v] = fmaf(-m, y, inv * (d * rw[k].get(v)));
        if (dr_out) g[v] += ro[k].get(v);
        dw[k][v] = live ? fmaf(d, y * inv, dw[k][v]) : dw[k][v];
        if (s) {
          h[v] = rs[k].get(v) * g[v];
          ds[k][v] = live ? fmaf(g[v], rp[k].get(v), ds[k][v]) : ds[k][v];
        }
      }
      if (live && seat.is(k))
        either(q.nt_out, [&](auto nt) {
          store_row<V, nt.value>(element(dr + at, seat.at[k]), g);
          if (s) store_row<V, nt.value>(element(dp + at, seat.at[k]), h);
        });
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

// The places of a row of y in head order: channel c of head h of a token is
// element base(token) + h N d + c.
struct Heads {
  int64_t H, N, DH;
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
  const int e0 = seat.g * q.EG, h0 = e0 / q.width;
  const float inv_n = 1.f / (float)q.EG;
  Raw<float, V> rw[NV];
  int64_t off[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if constexpr (R::HOLD_W) rw[k].load(element(w + e0, seat.at[k]));
    off[k] = (h0 + seat.head[k]) * hd.N * hd.DH + ((int)seat.at[k] - seat.head[k] * q.width);
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
        rz[k].template load<nt.value>(element(z + at, seat.at[k]));
        ry[k].template load<nt.value>(y + base + off[k]);
      }
    });
    float x[NV][V], sum = 0.f, none = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v);
        x[k][v] = yv * (zv * sigmoid_v(zv));
        const float n = FIRST ? x[k][v] : yv;
        sum = v >= seat.skip[k] ? fmaf(n, n, sum) : sum;
      }
    row_sums<R>(sum, none, turn);
    const float inv = inv_rms(sum, inv_n, eps);
    if constexpr (!R::HOLD_W) w = afresh(w);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W) rw[k].load(element(w + e0, seat.at[k]));
#pragma unroll
      for (int v = 0; v < V; ++v) x[k][v] = x[k][v] * inv * rw[k].get(v);
      if (live && seat.is(k))
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(element(o + at, seat.at[k]), x[k]); });
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
  const int e0 = seat.g * q.EG, h0 = e0 / q.width;
  const float inv_n = 1.f / (float)q.EG;
  Raw<float, V> rw[NV];
  float dw[NV][V];
  int64_t off[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if constexpr (R::HOLD_W) rw[k].load(element(w + e0, seat.at[k]));
    off[k] = (h0 + seat.head[k]) * hd.N * hd.DH + ((int)seat.at[k] - seat.head[k] * q.width);
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
    either(q.nt_in && R::HOLD_ROW, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rz[k].template load<nt.value>(element(z + at, seat.at[k]));
        rd[k].template load<nt.value>(element(d_out + at, seat.at[k]));
        ry[k].template load<nt.value>(y + base + off[k]);
      }
    });
    if constexpr (!R::HOLD_W) w = afresh(w);
    float sq = 0.f, ct = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W) rw[k].load(element(w + e0, seat.at[k]));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v), gate = zv * sigmoid_v(zv);
        const float x = FIRST ? yv * gate : yv, c = rd[k].get(v) * rw[k].get(v) * (FIRST ? 1.f : gate);
        sq = v >= seat.skip[k] ? fmaf(x, x, sq) : sq;
        ct = v >= seat.skip[k] ? fmaf(c, x, ct) : ct;
      }
    }
    row_sums<R>(sq, ct, turn);
    const float inv = inv_rms(sq, inv_n, eps), m = inv * inv * inv * (ct * inv_n);
    if constexpr (!R::HOLD_W) w = afresh(w);
    if constexpr (!R::HOLD_ROW) {
      y = afresh(y);
      z = afresh(z);
      d_out = afresh(d_out);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      piece_by_piece<R>();
      if constexpr (!R::HOLD_W) rw[k].load(element(w + e0, seat.at[k]));
      if constexpr (!R::HOLD_ROW) {
        rz[k].load(element(z + at, seat.at[k]));
        rd[k].load(element(d_out + at, seat.at[k]));
        ry[k].load(y + base + off[k]);
      }
      float gy[V], gz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v), d = rd[k].get(v), dwv = d * rw[k].get(v);
        const float sig = sigmoid_v(zv), gate = zv * sig, slope = sig * fmaf(zv, 1.f - sig, 1.f);
        const float x = FIRST ? yv * gate : yv;
        const float dx = fmaf(-m, x, inv * (FIRST ? dwv : dwv * gate));
        gy[v] = FIRST ? dx * gate : dx;
        gz[v] = FIRST ? dx * yv * slope : dwv * (yv * inv) * slope;
        dw[k][v] = live ? fmaf(FIRST ? d : d * gate, x * inv, dw[k][v]) : dw[k][v];
      }
      if (live && seat.is(k))
        either(q.nt_out, [&](auto nt) {
          store_row<V, nt.value>(dy + base + off[k], gy);
          store_row<V, nt.value>(element(dz + at, seat.at[k]), gz);
        });
    }
  }
  store_part<R>(seat, q, dw, part + seat.part * E + e0);
}

// ---- launches ----

// calls f(R) with the row shape for `heads` heads of `width` channels: 8 channels
// a thread (4 in rows of up to 256, 16 beyond 8192, 32 beyond 16384), so that a
// row with its weights and their gradients leaves room for 16 waves a CU and
// more.  Single channels where heads have fewer than 4, or so few more than 4
// that the pieces of a row outnumber the largest shape's.
static int64_t row_pieces(int64_t heads, int64_t width) {
  const int64_t wide = heads * ((width + 3) / 4);
  return width < 4 || wide > 8192 ? 0 : wide;
}

template <typename F>
static auto by_row(int64_t heads, int64_t width, F&& f) {
  const int64_t n = row_pieces(heads, width), EG = heads * width;
  if (n) {
    if (n <= 16) return f(Row<4, 16, 1>{});
    if (n <= 32) return f(Row<4, 32, 1>{});
    if (n <= 64) return f(Row<4, 64, 1>{});
    if (n <= 128) return f(Row<4, 64, 2>{});
    if (n <= 256) return f(Row<4, 128, 2>{});
    if (n <= 512) return f(Row<4, 256, 2>{});
    if (n <= 1024) return f(Row<4, 512, 2>{});
    if (n <= 2048) return f(Row<4, 1024, 2>{});
    if (n <= 4096) return f(Row<4, 1024, 4>{});
    return f(Row<4, 1024, 8>{});
  }
  if (EG <= 64) return f(Row<1, 16, 4>{});
  if (EG <= 512) return f(Row<1, 64, 8>{});
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
static Geo geo_of(R, int64_t tokens, int64_t groups, int64_t heads, int64_t width, bool backward,
                  int64_t bytes) {
  Geo q{};
  q.nt_in = bytes >= CACHE_BYTES;
  q.nt_out = bytes >= 3 * CACHE_BYTES;
  q.tokens = tokens;
  q.groups = (int)groups;
  q.EG = (int)(heads * width);
  q.width = (int)width;
  q.pieces = (int)(R::V == 4 ? row_pieces(heads, width) : heads * width);
  q.gpw = groups < R::SLOTS ? (int)groups : R::SLOTS;
  q.tpw = R::SLOTS / q.gpw;
  q.blocks = (int)((groups + q.gpw - 1) / q.gpw);
  const int64_t want = (tokens + q.tpw - 1) / q.tpw;
  int64_t most = 256 * (backward ? 1024 : 2048) / R::NT / q.blocks;
  if (most < 1) most = 1;
  q.parts = (int)(want < most ? want : most);
  return q;
}

static Geo geo_by(int64_t tokens, int64_t groups, int64_t heads, int64_t width, bool backward,
                  int64_t bytes) {
  return by_row(heads, width,
                [&](auto row) { return geo_of(row, tokens, groups, heads, width, backward, bytes); });
}

static hipError_t launch_sum_parts(const float* part, int n, int64_t E, float* out0, float* out1,
                                   hipStream_t stream) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((E + 31) / 32), out1 ? 2 : 1), dim3(1024), 0, stream, part,
                     n, E, out0, out1);
  return hipGetLastError();
}

// calls f(T, row)
template <typename F>
static hipError_t by_call(bool bf16, int64_t heads, int64_t width, F&& f) {
  return by_row(heads, width, [&](auto row) { return bf16 ? f(uint16_t{}, row) : f(float{}, row); });
}

hipError_t launch_norm_in(bool bf16, const float* r, const void* p, const float* s, const float* w,
                          int64_t rows, int64_t E, float eps, float* r_out, void* u,
                          hipStream_t stream) {
  const int64_t size = bf16 ? 2 : 4;
  return by_call(bf16, 1, E, [&](auto t, auto row) {
    using T = decltype(t);
    using R = decltype(row);
    const Geo q = geo_of(row, rows, 1, 1, E, false, rows * E * (p ? 8 + 2 * size : 4 + size));
    hipLaunchKernelGGL((k_norm_in<T, R>), dim3((unsigned)q.parts), dim3(R::NT), 0, stream, r, (const T*)p,
                       s, w, q, eps, r_out, (T*)u);
    return hipGetLastError();
  });
}

size_t norm_in_backward_floats(int64_t rows, int64_t E) {
  return (size_t)(2 * geo_by(rows, 1, 1, E, true, 0).parts * E);
}

hipError_t launch_norm_in_backward(bool bf16, const void* du, const float* dr_out, const float* r,
                                   const void* p, const float* s, const float* w, int64_t rows,
                                   int64_t E, float eps, float* dr, float* dp, float* dw, float* ds,
                                   float* ws, hipStream_t stream) {
  const int64_t size = bf16 ? 2 : 4;
  const Geo q = geo_by(rows, 1, 1, E, true, rows * E * (8 + size + (dr_out ? 4 : 0) + (s ? 4 + size : 0)));
  if (rows) {
    const hipError_t e = by_call(bf16, 1, E, [&](auto t, auto row) {
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

hipError_t launch_norm_out(bool bf16, bool gate_first, const float* y, const void* z,
                           const float* w, int64_t B, int64_t H, int64_t N, int64_t DH,
                           int64_t groups, float eps, void* o, hipStream_t stream) {
  return by_call(bf16, H / groups, DH, [&](auto t, auto row) {
    using T = decltype(t);
    using R = decltype(row);
    const Geo q = geo_of(row, B * N, groups, H / groups, DH, false, B * N * H * DH * (bf16 ? 8 : 12));
    auto go = [&](auto first) {
      hipLaunchKernelGGL((k_norm_out<T, R, first.value>), dim3((unsigned)(q.parts * q.blocks)), dim3(R::NT),
                         0, stream, y, (const T*)z, w, q, Heads{H, N, DH}, eps, (T*)o);
      return hipGetLastError();
    };
    return gate_first ? go(std::true_type{}) : go(std::false_type{});
  });
}

size_t norm_out_backward_floats(int64_t B, int64_t H, int64_t N, int64_t DH, int64_t groups) {
  return (size_t)(geo_by(B * N, groups, H / groups, DH, true, 0).parts * H * DH);
}

hipError_t launch_norm_out_backward(bool bf16, bool gate_first, const void* d_out, const float* y,
                                    const void* z, const float* w, int64_t B, int64_t H, int64_t N,
                                    int64_t DH, int64_t groups, float eps, float* dy, float* dz,
                                    float* dw, float* ws, hipStream_t stream) {
  const int64_t tokens = B * N;
  const Geo q = geo_by(tokens, groups, H / groups, DH, true, tokens * H * DH * (bf16 ? 16 : 20));
  if (tokens) {
    const hipError_t e = by_call(bf16, H / groups, DH, [&](auto t, auto row) {
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
