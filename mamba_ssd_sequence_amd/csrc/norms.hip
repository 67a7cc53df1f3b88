// ssd_norm_in, ssd_norm_out and their gradients: the RMS norms, the SiLU gate
// and the residual scale at the two ends of a mixer block.
//     norm in:   r' = r + s p,  u = w r' k,  k = 1 / sqrt(mean r'^2 + eps)
//     norm out:  t = y silu(z), o = w t k   or   o = w silu(z) y k,
//                k over the groups of a token's channels; y in head order
//                [B,H,N,d_h], z and o in token order [B,N,H d_h]
// Backwards with t^ = t k, the row over its own size:
//     dt = k (c - t^ mean(c t^)),  mean(c t^) = k mean(c t),
// so that no power of k is formed: k^3 leaves fp32's range at rows of 1e13 (and,
// with eps = 0, of 1e-13) while the gradients and the squares are well inside it.
// All four are bound by memory: every array is read once and written once, a
// row (a token's group of channels) lives in registers between its sums and its
// outputs, and norm out reads y where the mixer left it.  bf16, E 1024: norm in
// 65536 rows 805 MB in 141 us (5.7 TB/s), backwards 8192 rows 168 MB in 33.9 us with
// the sum of the weight gradients (4 us); norm out 2 x 16 heads of 4096 tokens 67 MB
// in 12.1 us, backwards 4 x 16 of 2048 134 MB in 27.1 us.
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
//
// Rows of more than 2048 pieces (8192 channels) do not fit that way: backwards a
// thread would hold 128 values and more, and spilled (16384 channels, 1024 rows:
// 216 us).  Backwards one kernel then leaves each row's two means, and another takes
// blocks of 256 pieces down the rows (91 us, 3.7 TB/s of the bytes that have to move).
// Forwards, where a row would be fewer registers, a workgroup walks along it twice
// all the same (norm in 1024 x 16384 51 us, 300 x 32768 40 us: 3.9 and 2.9 TB/s).
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
  int groups, EG;      // groups of a token, channels of a group
  int width, pieces;   // channels of a head, pieces of a group
  int gpw, tpw, blocks, parts;
  bool nt_in, nt_out;  // nontemporal loads, stores
};

// A piece of a group's row: its first channel there, the head it is in, and how
// many of its channels are not its own (V: there is no such piece).
struct Piece {
  unsigned at;
  int head, skip;
};

template <int V>
__device__ __forceinline__ Piece piece_of(int i, const Geo& q) {
  const int each = (q.width + V - 1) / V;
  const bool is = i < q.pieces;
  const int head = is ? i / each : 0;
  const int c = is ? (i - head * each) * V : 0, moved = c < q.width - V ? c : q.width - V;
  return {(unsigned)(head * q.width + moved), head, is ? c - moved : V};
}

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
#pragma unroll
    for (int k = 0; k < R::NV; ++k) {
      const Piece p = piece_of<R::V>(k * R::TPR + lane, q);
      at[k] = p.at;
      head[k] = p.head;
      skip[k] = p.skip;
    }
  }
  __device__ __forceinline__ bool is(int k) const { return skip[k] < R::V; }
  // the piece's place among the pieces of the row
  __device__ __forceinline__ int nominal(int k) const { return (k * R::TPR + lane) * R::V; }
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
    float x[NV][V], sum = 0.f, none = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
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
#pragma unroll
    for (int k = 0; k < NV; ++k) {
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

template <typename T, typename R, bool SCALED, bool ADDED>
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
    rw[k].load(element(w, seat.at[k]));
    if constexpr (SCALED) rs[k].load(element(s, seat.at[k]));
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
        rr[k].template load<nt.value>(element(r + at, seat.at[k]));
        rd[k].template load<nt.value>(element(du + at, seat.at[k]));
        if constexpr (ADDED) ro[k].template load<nt.value>(element(dr_out + at, seat.at[k]));
        if constexpr (SCALED) rp[k].template load<nt.value>(element(p + at, seat.at[k]));
      }
    });
    float sq = 0.f, cr = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = rr[k].get(v), c = rd[k].get(v) * rw[k].get(v);
        sq = v >= seat.skip[k] ? fmaf(y, y, sq) : sq;
        cr = v >= seat.skip[k] ? fmaf(c, y, cr) : cr;
      }
    }
    row_sums<R>(sq, cr, turn);
    const float inv = inv_rms(sq, inv_n, eps), m = inv * (cr * inv_n);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float g[V], h[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float hat = rr[k].get(v) * inv, d = rd[k].get(v);
        g[v] = inv * fmaf(-m, hat, d * rw[k].get(v));
        if constexpr (ADDED) g[v] += ro[k].get(v);
        dw[k][v] = live ? fmaf(d, hat, dw[k][v]) : dw[k][v];
        if constexpr (SCALED) {
          h[v] = rs[k].get(v) * g[v];
          ds[k][v] = live ? fmaf(g[v], rp[k].get(v), ds[k][v]) : ds[k][v];
        }
      }
      if (live && seat.is(k))
        either(q.nt_out, [&](auto nt) {
          store_row<V, nt.value>(element(dr + at, seat.at[k]), g);
          if constexpr (SCALED) store_row<V, nt.value>(element(dp + at, seat.at[k]), h);
        });
    }
  }
  store_part<R>(seat, q, dw, part + (int64_t)seat.part * q.EG);
  if constexpr (SCALED) store_part<R>(seat, q, ds, part + (int64_t)(q.parts + seat.part) * q.EG);
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
    rw[k].load(element(w + e0, seat.at[k]));
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
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) x[k][v] = x[k][v] * inv * rw[k].get(v);
      if (live && seat.is(k))
        either(q.nt_out, [&](auto nt) { store_row<V, nt.value>(element(o + at, seat.at[k]), x[k]); });
    }
  }
}

// One channel's gradients: k = inv, m = k mean(c x).
template <bool FIRST>
__device__ __forceinline__ void norm_out_slopes(float z, float y, float d, float w, float inv, float m,
                                                float& dy, float& dz, float& dw) {
  const float sig = sigmoid_v(z), gate = z * sig, slope = sig * fmaf(z, 1.f - sig, 1.f);
  const float c = d * w, hat = (FIRST ? y * gate : y) * inv;
  const float dx = inv * fmaf(-m, hat, FIRST ? c : c * gate);
  dy = FIRST ? dx * gate : dx;
  dz = FIRST ? dx * y * slope : c * hat * slope;
  dw = fmaf(FIRST ? d : d * gate, hat, dw);
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
    rw[k].load(element(w + e0, seat.at[k]));
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
    either(q.nt_in, [&](auto nt) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        rz[k].template load<nt.value>(element(z + at, seat.at[k]));
        rd[k].template load<nt.value>(element(d_out + at, seat.at[k]));
        ry[k].template load<nt.value>(y + base + off[k]);
      }
    });
    float sq = 0.f, ct = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz[k].get(v), yv = ry[k].get(v), gate = zv * sigmoid_v(zv);
        const float x = FIRST ? yv * gate : yv, c = rd[k].get(v) * rw[k].get(v) * (FIRST ? 1.f : gate);
        sq = v >= seat.skip[k] ? fmaf(x, x, sq) : sq;
        ct = v >= seat.skip[k] ? fmaf(c, x, ct) : ct;
      }
    }
    row_sums<R>(sq, ct, turn);
    const float inv = inv_rms(sq, inv_n, eps), m = inv * (ct * inv_n);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float gy[V], gz[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float more = dw[k][v];
        norm_out_slopes<FIRST>(rz[k].get(v), ry[k].get(v), rd[k].get(v), rw[k].get(v), inv, m, gy[v], gz[v], more);
        dw[k][v] = live ? more : dw[k][v];
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

// ---- long rows ----

constexpr int LT = 1024;  // threads along a row

// the sums of a and b over the workgroup of LT threads
__device__ __forceinline__ void long_sums(float& a, float& b) {
  row_sums<Row<4, LT, 1>>(a, b, 0);
  __syncthreads();  // the slots are free for the next row
}

// A row per workgroup and turn, read twice (the second time from the L2).
template <typename T, int V>
__global__ __launch_bounds__(LT) void k_long_in(const float* __restrict__ r, const T* __restrict__ p,
                                                const float* __restrict__ s, const float* __restrict__ w,
                                                Geo q, float eps, float* __restrict__ r_out,
                                                T* __restrict__ u) {
  for (int64_t row = blockIdx.x; row < q.tokens; row += gridDim.x) {
    const int64_t at = row * q.EG;
    auto value = [&](const Piece& pc, float(&x)[V]) {
      Raw<float, V> rr, rs;
      Raw<T, V> rp;
      rr.load(element(r + at, pc.at));
      if (p) rp.load(element(p + at, pc.at));
      if (s) rs.load(element(s, pc.at));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[v] = rr.get(v);
        if (p) x[v] = s ? fmaf(rs.get(v), rp.get(v), x[v]) : x[v] + rp.get(v);
      }
    };
    float sum = 0.f, none = 0.f;
    for (int i = threadIdx.x; i < q.pieces; i += LT) {
      const Piece pc = piece_of<V>(i, q);
      float x[V];
      value(pc, x);
#pragma unroll
      for (int v = 0; v < V; ++v) sum = v >= pc.skip ? fmaf(x[v], x[v], sum) : sum;
      if (p) store_row<V>(element(r_out + at, pc.at), x);
    }
    long_sums(sum, none);
    const float inv = inv_rms(sum, 1.f / (float)q.EG, eps);
    for (int i = threadIdx.x; i < q.pieces; i += LT) {
      const Piece pc = piece_of<V>(i, q);
      float x[V];
      Raw<float, V> rw;
      value(pc, x);
      rw.load(element(w, pc.at));
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = x[v] * inv * rw.get(v);
      store_row<V>(element(u + at, pc.at), x);
    }
  }
}

// k and k mean(c r) of every row
template <typename T, int V>
__global__ __launch_bounds__(LT) void k_long_in_means(const T* __restrict__ du, const float* __restrict__ r,
                                                      const float* __restrict__ w, Geo q, float eps,
                                                      float2* __restrict__ means) {
  const float inv_n = 1.f / (float)q.EG;
  for (int64_t row = blockIdx.x; row < q.tokens; row += gridDim.x) {
    const int64_t at = row * q.EG;
    float sq = 0.f, cr = 0.f;
    for (int i = threadIdx.x; i < q.pieces; i += LT) {
      const Piece pc = piece_of<V>(i, q);
      Raw<float, V> rr, rw;
      Raw<T, V> rd;
      rr.load(element(r + at, pc.at));
      rd.load(element(du + at, pc.at));
      rw.load(element(w, pc.at));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float y = rr.get(v), c = rd.get(v) * rw.get(v);
        sq = v >= pc.skip ? fmaf(y, y, sq) : sq;
        cr = v >= pc.skip ? fmaf(c, y, cr) : cr;
      }
    }
    long_sums(sq, cr);
    const float inv = inv_rms(sq, inv_n, eps);
    if (threadIdx.x == 0) means[row] = make_float2(inv, inv * (cr * inv_n));
  }
}

// a thread per piece, down the rows part, part + parts, ..
template <typename T, int V>
__global__ __launch_bounds__(256) void k_long_in_bwd(
    const T* __restrict__ du, const float* __restrict__ dr_out, const float* __restrict__ r,
    const T* __restrict__ p, const float* __restrict__ s, const float* __restrict__ w,
    const float2* __restrict__ means, Geo q, float* __restrict__ dr, float* __restrict__ dp,
    float* __restrict__ part) {
  const Piece pc = piece_of<V>(blockIdx.x * 256 + threadIdx.x, q);
  if (pc.skip == V) return;
  Raw<float, V> rw, rs;
  float dw[V], ds[V];
  rw.load(element(w, pc.at));
  if (s) rs.load(element(s, pc.at));
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = ds[v] = 0.f;
  for (int64_t row = blockIdx.y; row < q.tokens; row += q.parts) {
    const int64_t at = row * q.EG;
    Raw<float, V> rr, ro;
    Raw<T, V> rd, rp;
    rr.load(element(r + at, pc.at));
    rd.load(element(du + at, pc.at));
    if (dr_out) ro.load(element(dr_out + at, pc.at));
    if (s) rp.load(element(p + at, pc.at));
    const float2 mean = means[row];
    float g[V], h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float hat = rr.get(v) * mean.x, d = rd.get(v);
      g[v] = mean.x * fmaf(-mean.y, hat, d * rw.get(v));
      if (dr_out) g[v] += ro.get(v);
      dw[v] = fmaf(d, hat, dw[v]);
      if (s) {
        h[v] = rs.get(v) * g[v];
        ds[v] = fmaf(g[v], rp.get(v), ds[v]);
      }
    }
    store_row<V>(element(dr + at, pc.at), g);
    if (s) store_row<V>(element(dp + at, pc.at), h);
  }
  store_row<V>(element(part + (int64_t)blockIdx.y * q.EG, pc.at), dw);
  if (s) store_row<V>(element(part + (int64_t)(q.parts + blockIdx.y) * q.EG, pc.at), ds);
}

// Rows of norm out: unit = token x group.
template <typename T, int V, bool FIRST>
__global__ __launch_bounds__(LT) void k_long_out(const float* __restrict__ y, const T* __restrict__ z,
                                                 const float* __restrict__ w, Geo q, Heads hd, float eps,
                                                 T* __restrict__ o) {
  const int64_t E = (int64_t)q.groups * q.EG, units = q.tokens * q.groups;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t token = unit / q.groups, e0 = (unit - token * q.groups) * q.EG, h0 = e0 / q.width;
    const int64_t base = hd.base(token), at = token * E + e0;
    auto value = [&](const Piece& pc, float(&x)[V], float(&n)[V]) {
      Raw<float, V> ry;
      Raw<T, V> rz;
      ry.load(y + base + ((h0 + pc.head) * hd.N * hd.DH + ((int)pc.at - pc.head * q.width)));
      rz.load(element(z + at, pc.at));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz.get(v);
        x[v] = ry.get(v) * (zv * sigmoid_v(zv));
        n[v] = FIRST ? x[v] : ry.get(v);
      }
    };
    float sum = 0.f, none = 0.f;
    for (int i = threadIdx.x; i < q.pieces; i += LT) {
      const Piece pc = piece_of<V>(i, q);
      float x[V], n[V];
      value(pc, x, n);
#pragma unroll
      for (int v = 0; v < V; ++v) sum = v >= pc.skip ? fmaf(n[v], n[v], sum) : sum;
    }
    long_sums(sum, none);
    const float inv = inv_rms(sum, 1.f / (float)q.EG, eps);
    for (int i = threadIdx.x; i < q.pieces; i += LT) {
      const Piece pc = piece_of<V>(i, q);
      float x[V], n[V];
      Raw<float, V> rw;
      value(pc, x, n);
      rw.load(element(w + e0, pc.at));
#pragma unroll
      for (int v = 0; v < V; ++v) x[v] = x[v] * inv * rw.get(v);
      store_row<V>(element(o + at, pc.at), x);
    }
  }
}

template <typename T, int V, bool FIRST>
__global__ __launch_bounds__(LT) void k_long_out_means(const T* __restrict__ d_out, const float* __restrict__ y,
                                                       const T* __restrict__ z, const float* __restrict__ w,
                                                       Geo q, Heads hd, float eps, float2* __restrict__ means) {
  const int64_t E = (int64_t)q.groups * q.EG, units = q.tokens * q.groups;
  const float inv_n = 1.f / (float)q.EG;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t token = unit / q.groups, e0 = (unit - token * q.groups) * q.EG, h0 = e0 / q.width;
    const int64_t base = hd.base(token), at = token * E + e0;
    float sq = 0.f, ct = 0.f;
    for (int i = threadIdx.x; i < q.pieces; i += LT) {
      const Piece pc = piece_of<V>(i, q);
      Raw<float, V> ry, rw;
      Raw<T, V> rz, rd;
      ry.load(y + base + ((h0 + pc.head) * hd.N * hd.DH + ((int)pc.at - pc.head * q.width)));
      rz.load(element(z + at, pc.at));
      rd.load(element(d_out + at, pc.at));
      rw.load(element(w + e0, pc.at));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float zv = rz.get(v), gate = zv * sigmoid_v(zv);
        const float x = FIRST ? ry.get(v) * gate : ry.get(v);
        const float c = rd.get(v) * rw.get(v) * (FIRST ? 1.f : gate);
        sq = v >= pc.skip ? fmaf(x, x, sq) : sq;
        ct = v >= pc.skip ? fmaf(c, x, ct) : ct;
      }
    }
    long_sums(sq, ct);
    const float inv = inv_rms(sq, inv_n, eps);
    if (threadIdx.x == 0) means[unit] = make_float2(inv, inv * (ct * inv_n));
  }
}

// a thread per piece of a group, down the tokens part, part + parts, ..
template <typename T, int V, bool FIRST>
__global__ __launch_bounds__(256) void k_long_out_bwd(
    const T* __restrict__ d_out, const float* __restrict__ y, const T* __restrict__ z,
    const float* __restrict__ w, const float2* __restrict__ means, Geo q, Heads hd,
    float* __restrict__ dy, float* __restrict__ dz, float* __restrict__ part) {
  const int g = blockIdx.x / q.blocks;
  const Piece pc = piece_of<V>((blockIdx.x - g * q.blocks) * 256 + threadIdx.x, q);
  if (pc.skip == V) return;
  const int64_t E = (int64_t)q.groups * q.EG, e0 = (int64_t)g * q.EG, h0 = e0 / q.width;
  const int64_t off = (h0 + pc.head) * hd.N * hd.DH + ((int)pc.at - pc.head * q.width);
  Raw<float, V> rw;
  float dw[V];
  rw.load(element(w + e0, pc.at));
#pragma unroll
  for (int v = 0; v < V; ++v) dw[v] = 0.f;
  for (int64_t token = blockIdx.y; token < q.tokens; token += q.parts) {
    const int64_t base = hd.base(token), at = token * E + e0;
    Raw<float, V> ry;
    Raw<T, V> rz, rd;
    ry.load(y + base + off);
    rz.load(element(z + at, pc.at));
    rd.load(element(d_out + at, pc.at));
    const float2 mean = means[token * q.groups + g];
    float gy[V], gz[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      norm_out_slopes<FIRST>(rz.get(v), ry.get(v), rd.get(v), rw.get(v), mean.x, mean.y, gy[v], gz[v], dw[v]);
    store_row<V>(dy + base + off, gy);
    store_row<V>(element(dz + at, pc.at), gz);
  }
  store_row<V>(element(part + (int64_t)blockIdx.y * E + e0, pc.at), dw);
}

// ---- launches ----

// Pieces of a group's row: of 4 channels, or of one where heads have fewer than 4.
static int64_t row_pieces(int64_t heads, int64_t width) {
  return width < 4 ? heads * width : heads * ((width + 3) / 4);
}

// Rows that do not fit a workgroup's registers, 8 channels a thread (512 channels
// of such narrow heads).
static bool is_long(int64_t heads, int64_t width) {
  return row_pieces(heads, width) > (width < 4 ? 512 : 2048);
}

// calls f(R) with the row shape for `heads` heads of `width` channels: 8 channels
// a thread (4 in rows of up to 256), so that a row with its weights and their
// gradients leaves room for 16 waves a CU and more.
// DEEP, norm out forwards, which holds least and whose rows come from many places:
// a row of 513 to 1024 channels to one wave, 16 channels a thread and no barrier
// in its sum, from 2048 rows on, whose workgroups of 8 rows are then one to a CU.
// One wave / two a row, 16 heads of 64: 256 rows 4.1 / 3.4 us, 1024 4.3 / 3.7, 2048
// 4.6 / 5.0, 8192 11.9 / 14.7, 2 x 8192 23.0 / 26.9, 32768 48.2 / 50.2, 65536 96.5 /
// 92.6; 12 heads, 16384 rows 18.8 / 20.9; 8 of 128, 32768 rows 53.1 / 50.4.  Longer rows
// have their barrier either way, and win with 16 channels as often as they lose
// (32 heads 0.88 to 1.09 of the time of 8, 64 heads 0.90 to 1.31, 128 heads 0.97 to
// 1.05); norm in 8192 rows 16.8 / 16.0.  They keep 8.
template <bool DEEP, typename F>
static auto by_row(int64_t heads, int64_t width, int64_t rows, F&& f) {
  const int64_t n = row_pieces(heads, width);
  if (width < 4) {
    if (n <= 64) return f(Row<1, 16, 4>{});
    return f(Row<1, 64, 8>{});
  }
  if (n <= 16) return f(Row<4, 16, 1>{});
  if (n <= 32) return f(Row<4, 32, 1>{});
  if (n <= 64) return f(Row<4, 64, 1>{});
  if (n <= 128) return f(Row<4, 64, 2>{});
  if constexpr (DEEP)
    if (n <= 256 && rows >= 2048) return f(Row<4, 64, 4>{});
  if (n <= 256) return f(Row<4, 128, 2>{});
  if (n <= 512) return f(Row<4, 256, 2>{});
  if (n <= 1024) return f(Row<4, 512, 2>{});
  return f(Row<4, 1024, 2>{});
}

// Workgroups: enough to fill the 256 CUs with 2048 threads each (backwards with
// 1024, whose sums then add up over fewer parts), no more than there is work for.
// Nontemporal stores where a call moves 128 MB and more, half of the last-level
// cache, loads too from 192 MB on; smaller calls find their arrays in the cache and
// leave them there.  Plain / stores / loads / both: norm in, bf16, E 1024, 101 MB 16.0 /
// 16.4 / 18.5 / 18.9 us, 403 MB 74.9 / 72.7 / 73.4 / 69.3; norm out backwards 134 MB
// 31.3 / 27.0 / 31.1 / 30.5; norm in backwards 168 MB 37.0 / 34.7 / 34.6 / 35.2, 671 MB
// 130 / 125 / 127 / 121, 1342 MB 258 / 249 / 256 / 243.
template <typename R>
static Geo geo_of(R, int64_t tokens, int64_t groups, int64_t heads, int64_t width, bool backward,
                  int64_t bytes) {
  Geo q{};
  q.nt_in = bytes >= (int64_t)192 << 20;
  q.nt_out = bytes >= (int64_t)128 << 20;
  q.tokens = tokens;
  q.groups = (int)groups;
  q.EG = (int)(heads * width);
  q.width = (int)width;
  q.pieces = (int)row_pieces(heads, width);
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
  return by_row<false>(heads, width, tokens * groups,
                       [&](auto row) { return geo_of(row, tokens, groups, heads, width, backward, bytes); });
}

// Long rows: the rows' grid, and the backward's blocks of 256 pieces x parts of
// the tokens (some 2048 workgroups); its workspace has the means behind the parts.
static Geo long_geo(int64_t tokens, int64_t groups, int64_t heads, int64_t width) {
  Geo q{};
  q.tokens = tokens;
  q.groups = (int)groups;
  q.EG = (int)(heads * width);
  q.width = (int)width;
  q.pieces = (int)row_pieces(heads, width);
  q.blocks = (q.pieces + 255) / 256;
  const int64_t want = 2048 / (q.blocks * groups) + 1;
  q.parts = (int)(tokens < want ? tokens : want);
  return q;
}

static unsigned long_grid(int64_t rows) { return (unsigned)(rows < 1024 ? rows : 1024); }

// calls f(T, V)
template <typename F>
static hipError_t by_long(bool bf16, int64_t width, F&& f) {
  if (width < 4)
    return bf16 ? f(uint16_t{}, std::integral_constant<int, 1>{}) : f(float{}, std::integral_constant<int, 1>{});
  return bf16 ? f(uint16_t{}, std::integral_constant<int, 4>{}) : f(float{}, std::integral_constant<int, 4>{});
}

static hipError_t launch_sum_parts(const float* part, int n, int64_t E, float* out0, float* out1,
                                   hipStream_t stream) {
  hipLaunchKernelGGL(k_sum_parts, dim3((unsigned)((E + 31) / 32), out1 ? 2 : 1), dim3(1024), 0, stream, part,
                     n, E, out0, out1);
  return hipGetLastError();
}

// calls f(T, row)
template <bool DEEP = false, typename F>
static hipError_t by_call(bool bf16, int64_t heads, int64_t width, int64_t rows, F&& f) {
  return by_row<DEEP>(heads, width, rows, [&](auto row) { return bf16 ? f(uint16_t{}, row) : f(float{}, row); });
}

hipError_t launch_norm_in(bool bf16, const float* r, const void* p, const float* s, const float* w,
                          int64_t rows, int64_t E, float eps, float* r_out, void* u,
                          hipStream_t stream) {
  const int64_t size = bf16 ? 2 : 4;
  if (is_long(1, E))
    return by_long(bf16, E, [&](auto t, auto v) {
      using T = decltype(t);
      hipLaunchKernelGGL((k_long_in<T, v.value>), dim3(long_grid(rows)), dim3(LT), 0, stream, r, (const T*)p, s, w,
                         long_geo(rows, 1, 1, E), eps, r_out, (T*)u);
      return hipGetLastError();
    });
  return by_call(bf16, 1, E, rows, [&](auto t, auto row) {
    using T = decltype(t);
    using R = decltype(row);
    const Geo q = geo_of(row, rows, 1, 1, E, false, rows * E * (p ? 8 + 2 * size : 4 + size));
    hipLaunchKernelGGL((k_norm_in<T, R>), dim3((unsigned)q.parts), dim3(R::NT), 0, stream, r, (const T*)p,
                       s, w, q, eps, r_out, (T*)u);
    return hipGetLastError();
  });
}

size_t norm_in_backward_floats(int64_t rows, int64_t E) {
  if (is_long(1, E)) return (size_t)(2 * long_geo(rows, 1, 1, E).parts * ((E + 1) / 2 * 2) + 2 * rows);
  return (size_t)(2 * geo_by(rows, 1, 1, E, true, 0).parts * E);
}

hipError_t launch_norm_in_backward(bool bf16, const void* du, const float* dr_out, const float* r,
                                   const void* p, const float* s, const float* w, int64_t rows,
                                   int64_t E, float eps, float* dr, float* dp, float* dw, float* ds,
                                   float* ws, hipStream_t stream) {
  if (rows && is_long(1, E)) {
    const Geo q = long_geo(rows, 1, 1, E);
    float2* means = (float2*)(ws + 2 * q.parts * ((E + 1) / 2 * 2));
    const hipError_t e = by_long(bf16, E, [&](auto t, auto v) {
      using T = decltype(t);
      hipLaunchKernelGGL((k_long_in_means<T, v.value>), dim3(long_grid(rows)), dim3(LT), 0, stream, (const T*)du,
                         r, w, q, eps, means);
      hipLaunchKernelGGL((k_long_in_bwd<T, v.value>), dim3((unsigned)q.blocks, (unsigned)q.parts), dim3(256), 0,
                         stream, (const T*)du, dr_out, r, (const T*)p, s, w, means, q, dr, dp, ws);
      return hipGetLastError();
    });
    return e != hipSuccess ? e : launch_sum_parts(ws, q.parts, E, dw, ds, stream);
  }
  const int64_t size = bf16 ? 2 : 4;
  const Geo q = geo_by(rows, 1, 1, E, true, rows * E * (8 + size + (dr_out ? 4 : 0) + (s ? 4 + size : 0)));
  if (rows) {
    const hipError_t e = by_call(bf16, 1, E, rows, [&](auto t, auto row) {
      using T = decltype(t);
      using R = decltype(row);
      auto go = [&](auto scaled, auto added) {
        hipLaunchKernelGGL((k_norm_in_bwd<T, R, scaled.value, added.value>), dim3((unsigned)q.parts),
                           dim3(R::NT), 0, stream, (const T*)du, dr_out, r, (const T*)p, s, w, q, eps, dr, dp, ws);
        return hipGetLastError();
      };
      if (s) return dr_out ? go(std::true_type{}, std::true_type{}) : go(std::true_type{}, std::false_type{});
      return dr_out ? go(std::false_type{}, std::true_type{}) : go(std::false_type{}, std::false_type{});
    });
    if (e != hipSuccess) return e;
  }
  return launch_sum_parts(ws, rows ? q.parts : 0, E, dw, ds, stream);
}

hipError_t launch_norm_out(bool bf16, bool gate_first, const float* y, const void* z,
                           const float* w, int64_t B, int64_t H, int64_t N, int64_t DH,
                           int64_t groups, float eps, void* o, hipStream_t stream) {
  if (is_long(H / groups, DH))
    return by_long(bf16, DH, [&](auto t, auto v) {
      using T = decltype(t);
      auto go = [&](auto first) {
        hipLaunchKernelGGL((k_long_out<T, v.value, first.value>), dim3(long_grid(B * N * groups)), dim3(LT), 0,
                           stream, y, (const T*)z, w, long_geo(B * N, groups, H / groups, DH), Heads{H, N, DH}, eps,
                           (T*)o);
        return hipGetLastError();
      };
      return gate_first ? go(std::true_type{}) : go(std::false_type{});
    });
  return by_call<true>(bf16, H / groups, DH, B * N * groups, [&](auto t, auto row) {
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
  if (is_long(H / groups, DH))
    return (size_t)(long_geo(B * N, groups, H / groups, DH).parts * ((H * DH + 1) / 2 * 2) + 2 * B * N * groups);
  return (size_t)(geo_by(B * N, groups, H / groups, DH, true, 0).parts * H * DH);
}

hipError_t launch_norm_out_backward(bool bf16, bool gate_first, const void* d_out, const float* y,
                                    const void* z, const float* w, int64_t B, int64_t H, int64_t N,
                                    int64_t DH, int64_t groups, float eps, float* dy, float* dz,
                                    float* dw, float* ws, hipStream_t stream) {
  const int64_t tokens = B * N;
  if (tokens && is_long(H / groups, DH)) {
    const Geo q = long_geo(tokens, groups, H / groups, DH);
    float2* means = (float2*)(ws + q.parts * ((H * DH + 1) / 2 * 2));
    const hipError_t e = by_long(bf16, DH, [&](auto t, auto v) {
      using T = decltype(t);
      auto go = [&](auto first) {
        hipLaunchKernelGGL((k_long_out_means<T, v.value, first.value>), dim3(long_grid(tokens * groups)), dim3(LT),
                           0, stream, (const T*)d_out, y, (const T*)z, w, q, Heads{H, N, DH}, eps, means);
        hipLaunchKernelGGL((k_long_out_bwd<T, v.value, first.value>),
                           dim3((unsigned)(q.blocks * groups), (unsigned)q.parts), dim3(256), 0, stream,
                           (const T*)d_out, y, (const T*)z, w, means, q, Heads{H, N, DH}, dy, dz, ws);
        return hipGetLastError();
      };
      return gate_first ? go(std::true_type{}) : go(std::false_type{});
    });
    return e != hipSuccess ? e : launch_sum_parts(ws, q.parts, H * DH, dw, nullptr, stream);
  }
  const Geo q = geo_by(tokens, groups, H / groups, DH, true, tokens * H * DH * (bf16 ? 16 : 20));
  if (tokens) {
    const hipError_t e = by_call(bf16, H / groups, DH, tokens * groups, [&](auto t, auto row) {
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
