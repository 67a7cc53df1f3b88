// ssd_gated_scan, ssd_gated_scan_step, ssd_gated_scan_backward: the linear
// recurrence with a gate for every channel and token,
//     a = exp(-softplus(A_P)) = 1 / (1 + e^{A_P}),  g = sigmoid(I_P) or 1,
//     h_t = a_t h_{t-1} + beta_t g_t x_t,           y = h,
// beta = 1, 1 - a or sqrt(1 - a^2), and its gradients by the reverse recurrence
//     lam_t = dy_t + a_{t+1} lam_{t+1}.
#include "block.h"
#include "common.h"
#include "elem.h"

#include <type_traits>

namespace ssd {

enum { IN_PLAIN = 0, IN_CONVEX = 1, IN_UNIT = 2 };

// a and beta(a) from the logit
template <int SCALE>
__device__ __forceinline__ void decay_of(float A, float& a, float& beta) {
  float rest;
  sigmoid_pair(A, rest, a);
  if constexpr (SCALE == IN_PLAIN) beta = 1.f;
  if constexpr (SCALE == IN_CONVEX) beta = rest;
  // 1 - a^2 = (1 - a)(1 + a) without cancellation
  if constexpr (SCALE == IN_UNIT) beta = __builtin_amdgcn_sqrtf(fmaf(rest, a, rest));
}

// a, 1 - a, beta and d beta / d A_P, for the gradients
template <int SCALE>
__device__ __forceinline__ void decay_slope(float A, float& a, float& rest, float& beta, float& dbeta) {
  sigmoid_pair(A, rest, a);
  if constexpr (SCALE == IN_PLAIN) {
    beta = 1.f;
    dbeta = 0.f;
  } else if constexpr (SCALE == IN_CONVEX) {
    beta = rest;
    dbeta = a * rest;
  } else {
    // beta = sqrt(q), dbeta = a^2 (1 - a) / beta (0 where a = 1), q = 1 - a^2
    const float q = fmaf(rest, a, rest);
    const float inv = q == 0.f ? 0.f : __builtin_amdgcn_rsqf(q);
    beta = q * inv;
    dbeta = a * a * rest * inv;
  }
}

// ---- whole sequences ----
//
// One workgroup takes a tile: TOKENS consecutive tokens of C channels of one
// head, read once, held in registers as decays and inputs, and written once.
// Lane l of a wave owns V channels (l % LPR) of TT consecutive tokens (its
// group l / LPR); groups, then waves, follow each other along the tokens.
//  1. Each thread composes its TT steps h -> a h + u to one step (P, U); the
//     wave scans its groups' steps by lane shuffles, the waves' steps go to LDS.
//  2. The first wave, a lane per channel, composes them to the tile's step and
//     publishes it.  The steps of the earlier tiles of the same span of SPAN
//     tiles are read by all waves, some by each, and composed wave by wave; with
//     the state that enters the span the first wave then has the state entering
//     the tile and each of its waves.
//  3. Every thread runs its tokens from its own entering state and writes y.
// The alternative, a pass over the inputs for the segments' steps and a second
// one for the outputs, reads x, A_P and I_P twice.  Memory bounds both directions:
// 1 x 16 heads of 65536 tokens x 64 channels, bf16 with gate, 671 MB that have to
// move and 677 MB that the counters see, 129 us (5.2 TB/s; a copy of that size
// makes 5.1 to 5.3); 4 x 16 heads of 2048 tokens 84 MB in 17.9 us (loading, joining and
// storing do not overlap when every tile is resident at once), backwards 218 MB in
// 46 to 51 us, by the card.  A tile's 39 instruction slots an element would take half of that.
//
// Waiting.  A workgroup takes the next tile of its head from a counter, so the
// tiles before its own belong to workgroups that have started; each publishes
// its tile's step before it waits for anything.  The state entering a span is
// published by the last tile of the span before, after waits on steps and on
// the state entering that span: by induction from the first span, which waits
// for no state, every wait ends, in whatever order workgroups are scheduled.
// What is published is one 8-byte word a channel, stored and read by relaxed
// atomics of the whole device: the word itself says whether it is there, so no
// fence (a write-back of the XCD's L2) is needed.  A step's word holds P and U,
// marked by P's sign bit (P is a product of decays in [0, 1], or NaN, whose sign
// says nothing); a state's word holds the state and a mark.  Counters and words
// are cleared by a kernel in front.
// The order of every composition is fixed by the sizes alone, so the same call
// gives the same bits.

constexpr int SPAN = 32;

typedef unsigned long long word_t;

constexpr unsigned MARK = 0x80000000u;

__device__ __forceinline__ void put_word(word_t* p, unsigned hi, float lo) {
  __hip_atomic_store(p, (word_t)hi << 32 | __float_as_uint(lo), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ word_t get_word(const word_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ bool is_there(word_t w) { return (w >> 63) != 0; }
__device__ __forceinline__ float step_p(word_t w) { return __uint_as_float((unsigned)(w >> 32) & ~MARK); }
__device__ __forceinline__ float low_value(word_t w) { return __uint_as_float((unsigned)w); }

// The shape of a tile.  NW waves; TT tokens a thread.
template <int V_, int LPR_, int NW_, int TT_>
struct Tile {
  static constexpr int V = V_, LPR = LPR_, NW = NW_, TT = TT_;
  static constexpr int TG = WAVE / LPR;       // groups of a wave
  static constexpr int C = LPR * V;           // channels
  static constexpr int TOKENS = NW * TG * TT;
};

// Words and counters of the tiles of one channel slab of one head, `tiles` > 1:
// [tiles][C] words (steps), [spans][C] words (states entering the spans).
__host__ __device__ inline int64_t span_count(int64_t tiles) { return (tiles + SPAN - 1) / SPAN; }
__host__ __device__ inline int64_t slab_words(int64_t tiles, int C) {
  return (tiles + span_count(tiles)) * C;
}

__global__ __launch_bounds__(256) void k_clear_words(uint4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = make_uint4(0, 0, 0, 0);
}

// Steps (P, U) of the groups of a wave along its tokens (reverse: from the last
// group to the first) -> for each group the composition of the groups before it;
// the whole wave's composition goes to LDS, channel c on (lanes without channels
// of their own have channel 0's values, and write them once more).
template <typename TL, bool REVERSE>
__device__ __forceinline__ void scan_groups(float (&P)[TL::V], float (&U)[TL::V], int lane, int c,
                                            float* sP, float* sU) {
  const int tg = REVERSE ? TL::TG - 1 - lane / TL::LPR : lane / TL::LPR;
  auto before = [](float x, int groups) {
    return REVERSE ? __shfl_down(x, groups * TL::LPR, WAVE) : __shfl_up(x, groups * TL::LPR, WAVE);
  };
#pragma unroll
  for (int o = 1; o < TL::TG; o <<= 1)
#pragma unroll
    for (int v = 0; v < TL::V; ++v) {
      const float p = before(P[v], o), u = before(U[v], o);
      if (tg >= o) {
        U[v] = fmaf(P[v], u, U[v]);
        P[v] *= p;
      }
    }
  if (tg == TL::TG - 1) {
    store_row<TL::V>(sP + c, P);
    store_row<TL::V>(sU + c, U);
  }
#pragma unroll
  for (int v = 0; v < TL::V; ++v) {
    const float p = before(P[v], 1), u = before(U[v], 1);
    P[v] = tg ? p : 1.f;
    U[v] = tg ? u : 0.f;
  }
}

// LDS of a workgroup: the steps of its waves, the composed steps of the earlier
// tiles of the span (each wave's share), the states entering its waves.
template <typename TL>
struct Joint {
  float P[TL::NW * TL::C], U[TL::NW * TL::C], spanP[TL::NW * TL::C], spanU[TL::NW * TL::C],
      H[TL::NW * TL::C];
};

// From the waves' steps in LDS (complete) to the state entering each wave
// (j.H, complete on return), by way of the other tiles; lane c < C of a wave is
// channel c, `exists` says whether the head has it.  `order`: the tile's place
// in the scan's direction; `first`: in the first wave's lanes, the state
// entering the whole sequence.  Returns, there, the state that leaves the tile.
template <typename TL, bool REVERSE>
__device__ __forceinline__ float join_tiles(Joint<TL>& j, int wave, int c, bool exists, int order,
                                           int tiles, float first, word_t* words) {
  constexpr int C = TL::C, NW = TL::NW, EACH = SPAN / NW;
  static_assert(SPAN % NW == 0, "a span's tiles are shared out to the waves");
  auto slot = [&](int i) { return (REVERSE ? NW - 1 - i : i) * C + c; };
  const int span = order / SPAN, start = span * SPAN;
  word_t* states = words + (int64_t)tiles * C + c;
  words += c;
  float P = 1.f, U = 0.f;
  if (wave == 0 && exists && tiles > 1) {
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      U = fmaf(j.P[slot(i)], U, j.U[slot(i)]);
      P *= j.P[slot(i)];
    }
    if (order % SPAN != SPAN - 1 && order + 1 < tiles)  // someone may read the tile's step
      put_word(words + (int64_t)order * C, __float_as_uint(P) | MARK, U);
  }
  if (order > start) {
    const int t0 = start + wave * EACH;
    if (exists) {
      float p = 1.f, u = 0.f;
      if (t0 < order) {
        word_t w[EACH];
        bool all;
        do {
          all = true;
#pragma unroll
          for (int i = 0; i < EACH; ++i) w[i] = get_word(words + (int64_t)(t0 + i < order ? t0 + i : t0) * C);
#pragma unroll
          for (int i = 0; i < EACH; ++i) all = all && is_there(w[i]);
        } while (!all);
#pragma unroll
        for (int i = 0; i < EACH; ++i)
          if (t0 + i < order) {
            u = fmaf(step_p(w[i]), u, low_value(w[i]));
            p *= step_p(w[i]);
          }
      }
      j.spanP[wave * C + c] = p;
      j.spanU[wave * C + c] = u;
    }
    __syncthreads();
  }
  float h = first;
  if (wave == 0 && exists) {
    if (span) {
      word_t s;
      while (!is_there(s = get_word(states + (int64_t)span * C))) __builtin_amdgcn_s_sleep(1);
      h = low_value(s);
    }
    if (order > start)
#pragma unroll
      for (int i = 0; i < NW; ++i) h = fmaf(j.spanP[i * C + c], h, j.spanU[i * C + c]);
    if (order % SPAN == SPAN - 1 && order + 1 < tiles)
      put_word(states + ((int64_t)span + 1) * C, MARK, fmaf(P, h, U));
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      j.H[slot(i)] = h;
      h = fmaf(j.P[slot(i)], h, j.U[slot(i)]);
    }
  }
  __syncthreads();
  return h;
}

// the next tile of this workgroup's head (in the scan's order)
__device__ __forceinline__ int take_tile(int tiles, unsigned* counter) {
  if (tiles == 1) return 0;
  __shared__ unsigned mine;
  if (threadIdx.x == 0)
    mine = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(mine);
}

// The channels of a slab: `width` of them (a multiple of V; a slab's lanes past
// them are idle) from `start`.  Pieces of 4 that would pass the head's last
// channel are moved back to end with it, and a slab that would begin with fewer
// than 4 channels left begins 4 before the end: lanes or slabs then share
// channels, compute the same values for them and write them twice.
template <typename TL>
__device__ __forceinline__ int slab_start(int slab, int width, int DH) {
  return slab * width < DH - TL::V ? slab * width : DH - TL::V;
}

// Where a workgroup and a thread are: every array is addressed from a uniform
// pointer at the tile's first row by 32-bit byte offsets (at most 512 rows of at
// most SSD_GATED_MAX = 2^20 channels, more rows only of 32 channels and less), so
// that offsets past 2^32 elements cost no registers.
template <typename TL>
struct Spot {
  int64_t base;      // element of the tile's first row and the slab's first channel
  int tok, rows, c;  // the thread's first token in the tile, the tile's tokens, its channel in the slab
  bool live;         // it has channels of its own
  __device__ __forceinline__ Spot(int64_t bh, int start, int tile, int64_t N, int DH, int width) {
    const int lane = threadIdx.x % WAVE, nominal = lane % TL::LPR * TL::V;
    const int64_t left = N - (int64_t)tile * TL::TOKENS;
    rows = left < TL::TOKENS ? (int)left : TL::TOKENS;
    base = (bh * N + (int64_t)tile * TL::TOKENS) * DH + start;
    tok = (threadIdx.x / WAVE * TL::TG + lane / TL::LPR) * TL::TT;
    live = nominal < width && start + nominal < DH;
    c = !live ? 0 : start + nominal + TL::V <= DH ? nominal : DH - TL::V - start;
  }
  // offset of row tok + i, or of the last row
  __device__ __forceinline__ unsigned at(int i, int DH) const {
    return (unsigned)(tok + i < rows ? tok + i : rows - 1) * (unsigned)DH + (unsigned)c;
  }
};

template <typename T, int SCALE, bool GATE, typename TL>
__global__ __launch_bounds__(TL::NW* WAVE, 4) void k_gated_scan(
    const T* __restrict__ x, const T* __restrict__ A, const T* __restrict__ I,
    const float* __restrict__ h0, int64_t N, int DH, int width, int slabs, int heads, int tiles, int runs,
    bool nt_row, float* __restrict__ y, float* __restrict__ hf, unsigned* counters, word_t* words) {
  constexpr int V = TL::V, TT = TL::TT, C = TL::C;
  __shared__ Joint<TL> j;
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  const int hs = blockIdx.x % heads;  // head and slab
  const int start = slab_start<TL>(hs % slabs, width, DH);
  const int64_t bh = hs / slabs, state = bh * DH + start;  // the head, its state's first channel here
  const int taken = take_tile(tiles, counters + hs);
  const bool exists = lane < width && start + lane < DH;
  float enter = 0.f;  // in the first wave: the state entering the sequence, then each next tile
  if (wave == 0 && exists && h0) enter = h0[state + lane];
  for (int k = 0; k < runs; ++k) {
    const int tile = taken + k;
    asm("" : "+s"(DH));  // a tile's offsets are not worth registers over the loop
    const Spot<TL> sp(bh, start, tile, N, DH, width);
    const T *xt = x + sp.base, *At = A + sp.base, *It = I + sp.base;
    float* yt = y + sp.base;

    Raw<T, V> rx[TT], rA[TT], rI[TT];
    either(nt_row, [&](auto nt) {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const unsigned at = sp.at(i, DH);
        rA[i].template load<nt.value>(element(At, at));
        if constexpr (GATE) rI[i].template load<nt.value>(element(It, at));
        rx[i].template load<nt.value>(element(xt, at));
      }
    });
    float a[TT][V], u[TT][V], P[V], U[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.f;
      U[v] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      rA[i].or_else(sp.tok + i < sp.rows, 0xff80u);  // tokens past the end leave the state alone:
      rx[i].or_else(sp.tok + i < sp.rows, 0u);       // A_P = -inf, x = 0
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float beta, g = 1.f;
        decay_of<SCALE>(rA[i].get(v), a[i][v], beta);
        if constexpr (GATE) g = sigmoid_v(rI[i].get(v));
        u[i][v] = beta * g * rx[i].get(v);
        U[v] = fmaf(a[i][v], U[v], u[i][v]);
        P[v] *= a[i][v];
      }
    }
    scan_groups<TL, false>(P, U, lane, sp.c, j.P + wave * C, j.U + wave * C);
    __syncthreads();
    enter = join_tiles<TL, false>(j, wave, lane, exists, tiles > 1 ? tile : 0, tiles, enter,
                                  words + hs * slab_words(tiles, C));
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = fmaf(P[v], j.H[wave * C + sp.c + v], U[v]);
    const bool last = tile == tiles * runs - 1 && hf;
#pragma unroll
    for (int i = 0; i < TT; ++i) {
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = fmaf(a[i][v], h[v], u[i][v]);
      if (sp.live && sp.tok + i < sp.rows) {
        either(nt_row, [&](auto nt) { store_row<V, nt.value>(element(yt, sp.at(i, DH)), h); });
        if (last && sp.tok + i == sp.rows - 1) store_row<V>(hf + state + sp.c, h);
      }
    }
  }
}

// The gradients: the same tiles from the last token to the first, with the
// state c_t = a_t lam_t, c_t = a_t (dy_t + c_{t+1}), c_N = d_final_state and
// lam_t = dy_t + c_{t+1}; c_0 is the gradient of the initial state.  Only A_P
// and dy are needed for a tile's step; x, I_P and the states before each token
// (y one token earlier) are loaded right behind them, to arrive while the tiles
// are joined, and wait in registers for the tile's entering c.
template <typename T, int SCALE, bool GATE, typename TL>
__global__ __launch_bounds__(TL::NW* WAVE, 4) void k_gated_scan_bwd(
    const T* __restrict__ x, const T* __restrict__ A, const T* __restrict__ I,
    const float* __restrict__ h0, const float* __restrict__ y, const float* __restrict__ dy,
    const float* __restrict__ dlast, int64_t N, int DH, int width, int slabs, int heads, int tiles, int runs,
    bool nt_row, float* __restrict__ dx, float* __restrict__ dA, float* __restrict__ dI,
    float* __restrict__ dh0, unsigned* counters, word_t* words) {
  constexpr int V = TL::V, TT = TL::TT, C = TL::C;
  __shared__ Joint<TL> j;
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  const int hs = blockIdx.x % heads;
  const int start = slab_start<TL>(hs % slabs, width, DH);
  const int64_t bh = hs / slabs, state = bh * DH + start;
  const int taken = take_tile(tiles, counters + hs);
  const bool exists = lane < width && start + lane < DH;
  float enter = 0.f;  // in the first wave: d_final_state, then the c that leaves each tile
  if (wave == 0 && exists && dlast) enter = dlast[state + lane];
  for (int k = 0; k < runs; ++k) {
    const int order = taken + k, tile = tiles * runs - 1 - order;
    asm("" : "+s"(DH));  // a tile's offsets are not worth registers over the loop
    const Spot<TL> sp(bh, start, tile, N, DH, width);
    const T *xt = x + sp.base, *At = A + sp.base, *It = I + sp.base;
    const float *dyt = dy + sp.base, *yt = y + sp.base - DH;  // yt: a row before, the states before each token
    float *dxt = dx + sp.base, *dAt = dA + sp.base, *dIt = dI + sp.base;
    const bool first = tile == 0 && sp.tok == 0;  // the sequence's first token: the state before it is h0

    Raw<T, V> rA[TT], rx[TT], rI[TT];
    Raw<float, V> rd[TT], rp[TT], r0;
    either(nt_row, [&](auto nt) {
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        rA[i].template load<nt.value>(element(At, sp.at(i, DH)));
        rd[i].template load<nt.value>(element(dyt, sp.at(i, DH)));
      }
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const unsigned at = sp.at(i, DH);
        rx[i].template load<nt.value>(element(xt, at));
        if constexpr (GATE) rI[i].template load<nt.value>(element(It, at));
        // the row before; before the sequence's first row there is none, and its own is read without use
        rp[i].template load<nt.value>(element(yt, tile == 0 && at < (unsigned)DH ? at + DH : at));
      }
    });
    if (tile == 0 && h0) r0.load(h0 + state + sp.c);
    float P[V], U[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] = 1.f;
      U[v] = 0.f;
    }
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
      rA[i].or_else(sp.tok + i < sp.rows, 0xff80u);  // tokens past the end: a = 1, dy = 0
      rd[i].or_else(sp.tok + i < sp.rows, 0u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, rest;
        sigmoid_pair(rA[i].get(v), rest, a);
        U[v] = a * (rd[i].get(v) + U[v]);
        P[v] *= a;
      }
    }
    scan_groups<TL, true>(P, U, lane, sp.c, j.P + wave * C, j.U + wave * C);
    __syncthreads();
    enter = join_tiles<TL, true>(j, wave, lane, exists, tiles > 1 ? order : 0, tiles, enter,
                                 words + hs * slab_words(tiles, C));
    // the decays are computed again rather than held over the wait
#pragma unroll
    for (int i = 0; i < TT; ++i) rA[i].forget();
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = fmaf(P[v], j.H[wave * C + sp.c + v], U[v]);
#pragma unroll
    for (int i = TT - 1; i >= 0; --i) {
      if (!sp.live || sp.tok + i >= sp.rows) continue;
      float ox[V], oA[V], oI[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a, rest, beta, db, g = 1.f;
        decay_slope<SCALE>(rA[i].get(v), a, rest, beta, db);
        const float lam = rd[i].get(v) + carry[v], xv = rx[i].get(v);
        if constexpr (GATE) {
          float ng;
          sigmoid_pair(rI[i].get(v), g, ng);
          oI[v] = lam * beta * xv * g * ng;
        }
        float prev = rp[i].get(v);
        if (i == 0 && first) prev = h0 ? r0.get(v) : 0.f;
        ox[v] = lam * beta * g;
        oA[v] = lam * (SCALE == IN_PLAIN ? -(a * rest) * prev : fmaf(db * g, xv, -(a * rest) * prev));
        carry[v] = a * lam;
      }
      const unsigned at = sp.at(i, DH);
      either(nt_row, [&](auto nt) {
        store_row<V, nt.value>(element(dxt, at), ox);
        store_row<V, nt.value>(element(dAt, at), oA);
        if constexpr (GATE) store_row<V, nt.value>(element(dIt, at), oI);
      });
      if (i == 0 && first && dh0) store_row<V>(dh0 + state + sp.c, carry);
    }
  }
}

// ---- single tokens ----

// 4 channels a thread, the last n % 4 by one thread one by one (a piece moved
// back to the end would read channels that the step in place has written).
template <typename T, int SCALE, int V>
__device__ __forceinline__ void step_piece(const T* x, const T* A, const T* I, const float* state, int64_t i,
                                           float* out) {
  Raw<T, V> rx, rA, rI;
  Raw<float, V> rh;
  rA.load(A + i);
  if (I) rI.load(I + i);
  rx.load(x + i);
  rh.load(state + i);
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a, beta;
    decay_of<SCALE>(rA.get(v), a, beta);
    const float g = I ? sigmoid_v(rI.get(v)) : 1.f;
    h[v] = fmaf(a, rh.get(v), beta * g * rx.get(v));
  }
  store_row<V>(out + i, h);
}

template <typename T, int SCALE>
__global__ __launch_bounds__(256) void k_gated_step(const T* __restrict__ x, const T* __restrict__ A,
                                                    const T* __restrict__ I, const float* state,
                                                    int64_t n, float* out) {
  int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i + 4 <= n) {
    step_piece<T, SCALE, 4>(x, A, I, state, i, out);
  } else {
    for (; i < n; ++i) step_piece<T, SCALE, 1>(x, A, I, state, i, out);
  }
}

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

// The tile of a call: 4 channels a lane, 64 a tile (32 when the head has no
// more); heads of fewer than 4 channels a channel a lane, 4 a tile.
enum { WIDE64, WIDE32, NARROW };
static int tile_kind(int64_t DH) { return DH < 4 ? NARROW : DH > 32 ? WIDE64 : WIDE32; }
constexpr int kind_lpr(int k) { return k == WIDE64 ? 16 : k == WIDE32 ? 8 : 4; }
constexpr int kind_v(int k) { return k == NARROW ? 1 : 4; }

// Tokens a thread: what its registers hold (16 waves of 128 a CU).
constexpr int fwd_tokens(bool bf16) { return bf16 ? 8 : 4; }
constexpr int BWD_TOKENS = 4;

// How a call is cut.  A workgroup of 16 waves has the larger tile, so fewer
// steps to publish and wait for, but a CU holds only one: it pays within one round
// of the 256 CUs and where its tiles fill more than three quarters of two, three
// or four rounds, short of four whole ones (4 x 16 heads of 2048 tokens, bf16, one
// round: 17.9 us against 20.4 of 8 waves; of 3500, 1.75: 30.8 against 34.1; backwards
// 2048, two: 45.6 against 49.1).  Else workgroups of 8 waves take turns at loading
// and storing (4 x 16 of 2304 tokens, 1.25 rounds: 24.6 us against 27.0; of 8192,
// four: 65.0 against 65.8).
// From 512 heads and slabs on the chip can be full without cutting sequences: a
// workgroup then runs its head's tiles one after the other and nothing is published.
// That pays for up to 8 tiles a head, if the last round of 256 workgroups leaves
// less than a tenth of the rounds empty (heads of 600 tokens, one after the other /
// shared out: 512 39.8 / 45.3 us, backwards 104 / 107; 2048 150 / 161, 404 / 407; 736
// 58.6 / 62.0; but 528 53.7 / 48.0, backwards 130 / 110.  Of 2048 tokens, 8 tiles, 16
// backwards: 512 119 / 123, 337 / 333; 528 152 / 128, 424 / 344; 832 211 / 197, 585 / 540.
// Of 8192: 512 474 / 470, 640 643 / 593.  The border's own losses: 1600 of 300 tokens
// 73.3 / 78.2, 512 of 2304 140 / 146).
struct Split {
  int64_t slabs, heads, tiles;  // tiles: those that workgroups of one head share out
  int waves, runs, C, width;    // runs: tiles that a workgroup takes one after the other (then tiles = 1);
                                // width: channels of a slab, at most the tile's C
  // floats: the counters, padded, then the words
  size_t counters() const { return (size_t)((heads + 63) & ~(int64_t)63); }
  size_t floats() const { return tiles > 1 ? counters() + (size_t)(heads * slab_words(tiles, C)) * 2 : 0; }
};

static Split split_of(int64_t BH, int64_t N, int64_t DH, int tokens) {
  const int k = tile_kind(DH), lpr = kind_lpr(k), C = lpr * kind_v(k);
  const int64_t slabs = (DH + C - 1) / C, heads = BH * slabs;
  const int even = (int)((DH + slabs - 1) / slabs), width = k == NARROW ? even : (even + 3) / 4 * 4;
  auto tiles = [&](int waves) {
    const int64_t per = (int64_t)waves * (WAVE / lpr) * tokens;
    return (N + per - 1) / per;
  };
  const int64_t wide = heads * tiles(16), rounds = (wide + 255) / 256;
  if (rounds <= 1 || (wide < 4 * 256 && 4 * wide > 3 * 256 * rounds))
    return {slabs, heads, tiles(16), 16, 1, C, width};
  if (heads >= 512 && tiles(8) <= 8 && 10 * heads > 9 * 256 * ((heads + 255) / 256))
    return {slabs, heads, 1, 8, (int)tiles(8), C, width};
  return {slabs, heads, tiles(8), 8, 1, C, width};
}

// for either element type
size_t gated_scan_floats(int64_t BH, int64_t N, int64_t DH) {
  const size_t a = split_of(BH, N, DH, fwd_tokens(true)).floats();
  const size_t b = split_of(BH, N, DH, fwd_tokens(false)).floats();
  return a > b ? a : b;
}

size_t gated_scan_backward_floats(int64_t BH, int64_t N, int64_t DH) {
  return split_of(BH, N, DH, BWD_TOKENS).floats();
}

// A launch holds less than 2^32 threads: so many heads go into one (0: a single
// head has more), and the heads of a call into one launch after the other.
static int64_t heads_of_launch(const Split& s) {
  return (int64_t)(0xffffffffu / (unsigned)(s.waves * WAVE)) / s.tiles / s.slabs;
}

bool gated_scan_fits(bool bf16, int64_t BH, int64_t N, int64_t DH) {
  return heads_of_launch(split_of(BH, N, DH, fwd_tokens(bf16))) > 0;
}

bool gated_scan_backward_fits(int64_t BH, int64_t N, int64_t DH) {
  return heads_of_launch(split_of(BH, N, DH, BWD_TOKENS)) > 0;
}

// One launch's heads: their number, and where their arrays begin.
struct Share {
  int64_t heads, token, state;  // elements of [BH,N,DH] and of [BH,DH] before them
  unsigned* counters;
  word_t* words;
  unsigned grid(const Split& s) const { return (unsigned)(heads * s.tiles); }
  template <typename T> T* tokens(T* p) const { return p ? p + token : nullptr; }
  template <typename T> T* states(T* p) const { return p ? p + state : nullptr; }
};

// calls go(share) for one launch after the other
template <typename F>
static hipError_t by_share(const Split& s, int64_t BH, int64_t N, int64_t DH, float* ws, F&& go) {
  const int64_t most = heads_of_launch(s);
  for (int64_t b = 0; b < BH; b += most) {
    Share sh{(BH - b < most ? BH - b : most) * s.slabs, b * N * DH, b * DH, nullptr, nullptr};
    if (s.tiles > 1) {
      sh.counters = (unsigned*)ws + b * s.slabs;
      sh.words = (word_t*)(ws + s.counters()) + b * s.slabs * slab_words(s.tiles, s.C);
    }
    const hipError_t e = go(sh);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Inputs and outputs pass through once: nontemporal accesses where rows are whole
// 128-byte lines of fp32 (plain / nontemporal, bf16 with gate: 4 x 16 heads of 2048
// tokens 19.0 / 17.8 us, 1 x 16 of 65536 143 / 129; backwards 57.8 / 45.0); else
// two rows share a line, which has to stay for the second (33 channels,
// backwards: 34.7 / 59.0).
static bool passing(int64_t DH) { return DH % 32 == 0; }

static hipError_t clear_words(const Split& s, float* ws, hipStream_t stream) {
  const int64_t n = (int64_t)((s.floats() + 3) / 4), want = (n + 255) / 256;
  if (!n) return hipSuccess;
  hipLaunchKernelGGL(k_clear_words, dim3((unsigned)(want < 256 ? want : 256)), dim3(256), 0, stream,
                     (uint4*)ws, n);
  return hipGetLastError();
}

// calls f(T, SCALE, GATE, kind, NW) with types for the call's element type, scale, gate, tile and waves
template <typename F>
static hipError_t by_call(bool bf16, int scale, bool gate, int64_t DH, int waves, F&& f) {
  return by_type(bf16, scale, [&](auto t, auto sc) {
    auto with = [&](auto g, auto k) {
      return waves == 16 ? f(t, sc, g, k, std::integral_constant<int, 16>{})
                         : f(t, sc, g, k, std::integral_constant<int, 8>{});
    };
    auto by_kind = [&](auto g) {
      switch (tile_kind(DH)) {
        case WIDE64: return with(g, std::integral_constant<int, WIDE64>{});
        case WIDE32: return with(g, std::integral_constant<int, WIDE32>{});
        default: return with(g, std::integral_constant<int, NARROW>{});
      }
    };
    return gate ? by_kind(std::true_type{}) : by_kind(std::false_type{});
  });
}

hipError_t launch_gated_scan(bool bf16, int scale, const void* x, const void* A, const void* I,
                             const float* h0, int64_t BH, int64_t N, int64_t DH, float* y,
                             float* hf, float* ws, hipStream_t stream) {
  const Split s = split_of(BH, N, DH, fwd_tokens(bf16));
  const hipError_t e = clear_words(s, ws, stream);
  if (e != hipSuccess) return e;
  return by_call(bf16, scale, I != nullptr, DH, s.waves, [&](auto t, auto sc, auto g, auto k, auto nw) {
    using T = decltype(t);
    using TL = Tile<kind_v(k.value), kind_lpr(k.value), nw.value, fwd_tokens(sizeof(T) == 2)>;
    return by_share(s, BH, N, DH, ws, [&](const Share& sh) {
      hipLaunchKernelGGL((k_gated_scan<T, sc.value, g.value, TL>), dim3(sh.grid(s)), dim3(TL::NW * WAVE), 0, stream,
                         sh.tokens((const T*)x), sh.tokens((const T*)A), sh.tokens((const T*)I), sh.states(h0), N,
                         (int)DH, s.width, (int)s.slabs, (int)sh.heads, (int)s.tiles, s.runs, passing(DH),
                         sh.tokens(y), sh.states(hf), sh.counters, sh.words);
      return hipGetLastError();
    });
  });
}

hipError_t launch_gated_scan_step(bool bf16, int scale, const void* x, const void* A,
                                  const void* I, const float* state, int64_t n, float* out,
                                  hipStream_t stream) {
  return by_type(bf16, scale, [&](auto t, auto sc) {
    using T = decltype(t);
    hipLaunchKernelGGL((k_gated_step<T, sc.value>), dim3((unsigned)((n + 1023) / 1024)), dim3(256), 0,
                       stream, (const T*)x, (const T*)A, (const T*)I, state, n, out);
    return hipGetLastError();
  });
}

hipError_t launch_gated_scan_backward(bool bf16, int scale, const void* x, const void* A,
                                      const void* I, const float* h0, const float* y,
                                      const float* dy, const float* dlast, int64_t BH, int64_t N,
                                      int64_t DH, float* dx, float* dA, float* dI, float* dh0,
                                      float* ws, hipStream_t stream) {
  const Split s = split_of(BH, N, DH, BWD_TOKENS);
  const hipError_t e = clear_words(s, ws, stream);
  if (e != hipSuccess) return e;
  return by_call(bf16, scale, I != nullptr, DH, s.waves, [&](auto t, auto sc, auto g, auto k, auto nw) {
    using T = decltype(t);
    using TL = Tile<kind_v(k.value), kind_lpr(k.value), nw.value, BWD_TOKENS>;
    return by_share(s, BH, N, DH, ws, [&](const Share& sh) {
      hipLaunchKernelGGL((k_gated_scan_bwd<T, sc.value, g.value, TL>), dim3(sh.grid(s)), dim3(TL::NW * WAVE), 0,
                         stream, sh.tokens((const T*)x), sh.tokens((const T*)A), sh.tokens((const T*)I),
                         sh.states(h0), sh.tokens(y), sh.tokens(dy), sh.states(dlast), N, (int)DH, s.width,
                         (int)s.slabs, (int)sh.heads, (int)s.tiles, s.runs, passing(DH), sh.tokens(dx),
                         sh.tokens(dA), sh.tokens(dI), sh.states(dh0), sh.counters, sh.words);
      return hipGetLastError();
    });
  });
}

}  // namespace ssd
