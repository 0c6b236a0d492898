// Products of a few rows of unquantized activations with packed MXFP4 weights:
//   y[m][n] = alpha sum_k x[m][k] deq(W)[n][k]
// -- the single-token (decode) form of a layer whose weights are kept packed,
// and the same per expert of a mixture-of-experts layer, with the routed rows'
// ranges and sources read on the device.
//
// What bounds it: a tile of rows of x (16 of a bf16 x, 4 of a float32 x) reads and
// decodes all the weights, 17/32 byte each.  For one row tile that read is the bound,
// HBM's rate or, where the weights stay in it, the Infinity Cache's, or the latency of
// one pass where there is little to read; from two row tiles on it is the decoding and
// the products, which are done again for each.  The products run on
// V_MFMA_F32_16X16X32_BF16: E2M1 values times a power of two are exact in bf16 (one
// conversion instruction per two codes), the products are exact in float32 and the sums
// are float32.  A bf16 x goes in as it is; a float32 x is split exactly into three bf16
// terms (8 significant bits each, by truncation), which take three of an MFMA's columns.
//
// Lane layout: lane l holds MFMA row l & 15 (a weight row) or column l & 15 (a row of
// x) and the 8 contraction values of group l >> 4.  The contraction may run in any
// order as long as both operands agree, so in a step of 128 values group g takes the
// step's block g (32 values): one 16-byte load of codes and one scale byte a lane feed
// four MFMAs, the j-th with values 8j .. 8j+7 of the block.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "mx_device.h"
#include "mx_host.h"

namespace mx {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));

struct GemvArgs {
  const void* x;
  int64_t ldx;
  const uint8_t* codes;
  const uint8_t* scales;
  int64_t scale_ld, scale_end;  // bytes between scale rows; end of the last one
  const int64_t* offs;  // grouped: device offsets [groups + 1]
  const int32_t* src;   // grouped: slot of each row, or NULL
  int64_t N;
  void* y;
  float* partial;  // [slices][M][N] where the contraction is sliced
  int64_t ldy, ntiles;
  int M, K, top_k, groups, x_rows, y_bf16, window, rounds, slices;  // M: rows of y
  float alpha;
};

// 8 codes (element i in nibble i) under a block scale, as bf16.
__device__ __forceinline__ v8bf decode8_bf16(uint32_t w, float scale) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3);
  v8bf v;
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  return v;
}

// x as kTerms bf16 planes: take() gives the next plane of a lane's 8 consecutive values
// (words of bf16 pairs) and leaves the rest of the values in w.
template <typename T>
struct XTerms;
template <>
struct XTerms<uint16_t> {
  static constexpr int kTerms = 1;
  static __device__ __forceinline__ uint4 take(uint32_t w[4]) {
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct XTerms<float> {
  static constexpr int kTerms = 3;
  // The upper half of a float holds its 8 leading significant bits; the rest is exact.  Inf
  // has no rest, and a NaN stays one even if only its low bits say so.
  static __device__ __forceinline__ uint4 take(uint32_t w[8]) {
    uint32_t t[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      uint32_t u[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t v = w[2 * p + i], m = v & 0x7FFFFFFFu;
        u[i] = m > 0x7F800000u ? 0x7FC00000u : v;
        const float rest = __uint_as_float(v) - __uint_as_float(v & 0xFFFF0000u);
        w[2 * p + i] = m >= 0x7F800000u ? 0u : __float_as_uint(rest);
      }
      t[p] = __builtin_amdgcn_perm(u[1], u[0], 0x07060302u);  // the two upper halves
    }
    return make_uint4(t[0], t[1], t[2], t[3]);
  }
};

// Orders a wave's LDS accesses around an exchange between its lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// A workgroup barrier for LDS alone: global loads stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// The first `left` of V neighbouring sums, at T's alignment.
template <int V, typename T>
__device__ __forceinline__ void store_sums(T* p, const float (&sum)[V], int left) {
  T v[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 2) v[i] = (T)f32_to_bf16_rne(sum[i]);
    else v[i] = sum[i];
  }
  if (left >= V) {
    __builtin_memcpy(p, v, sizeof(v));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < left) p[i] = v[i];
  }
}

// The row tiles (of R rows) of all groups in one sequence.  Every lane holds two groups:
// their rows [lo, hi) within [0, rows) and the number of row tiles up to their end.
template <int R>
struct GroupTiles {
  int lo[2], hi[2], end[2];

  __device__ __forceinline__ void load(const int64_t* __restrict__ offs, int groups, int rows) {
    const int lane = threadIdx.x & 63;
    int64_t o[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int e = min(64 * h + lane, groups - 1);
      o[h][0] = offs[e];
      o[h][1] = offs[e + 1];
    }
    int before = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lo[h] = (int)max<int64_t>(min<int64_t>(o[h][0], rows), 0);
      hi[h] = (int)max<int64_t>(min<int64_t>(o[h][1], rows), 0);
      int n = 64 * h + lane < groups && hi[h] > lo[h] ? (hi[h] - lo[h] - 1) / R + 1 : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int up = __shfl_up(n, d);
        n += lane >= d ? up : 0;
      }
      end[h] = n + before;
      before = __builtin_amdgcn_readlane(end[h], 63);
    }
  }
  __device__ __forceinline__ int total() const { return __builtin_amdgcn_readlane(end[1], 63); }
  // Row tile v: its group, first row and rows.
  __device__ __forceinline__ int find(int v, int& m0, int& mrows) const {
    const uint64_t low = __ballot(end[0] > v);
    const int h = low ? 0 : 1;
    const int l = __ffsll((unsigned long long)(low ? low : __ballot(end[1] > v))) - 1;
    const int first = __builtin_amdgcn_readlane(h ? lo[1] : lo[0], l);
    const int last = __builtin_amdgcn_readlane(h ? hi[1] : hi[0], l);
    const int tiles = __builtin_amdgcn_readlane(h ? end[1] : end[0], l);
    m0 = first + (v - (tiles - ((last - first - 1) / R + 1))) * R;
    mrows = min(R, last - m0);
    return 64 * h + l;
  }
};

// Measured (one launch): one bf16 row of 14336 x 4096, 31 MB of weights, 8.4 us (3.7 TB/s,
// its start and end in it) with three such weights in turn, which the Infinity Cache holds,
// and 8.9 with 21, which it does not; 61 tokens x 4 of 32 experts 5760 x 2880, 285 MB, 60.6
// us (4.7 TB/s); 16 float32 tokens x 4 of 32, 2880 x 2880, 32.6 us; 47 bf16 rows of 4096 x
// 14336 25.6 us and 64 float32 rows 67.5 us.  Of the 61 tokens' time the loads alone take 53
// us and the rest alone some 40; the 47 rows are bound by the rest, each of their three row
// tiles decoding the weights, and the 64 rows' 16 row tiles the more so.
//
// One workgroup per compute unit: two of them, with smaller windows, took 68 us for the 61
// tokens where one takes 63, and several row tiles per workgroup, decoded once, 36 us for the
// 47 rows where one each takes 30 (more x to stage, registers for it, fewer loads ahead).
// That is for the eight waves of 1024 values and more.  Shorter contractions have a wave per
// 128 values and leave the card idle with it: four bf16 rows of 262144 x 768, x 384 and x 128
// take 35, 35 and 41 us, 3.1, 1.5 and 0.4 TB/s.
// The alternative of x in LDS and whole rows of weights per wave, without sums across
// waves, computes faster but reads 64-byte pieces of 128 rows at once: 73 us for the 61
// tokens.
//
// A tile is kGemvTile columns of y (weight rows) for up to R rows of x; a workgroup takes a
// run of consecutive tiles, column tiles first, so that it keeps its rows of x while the
// group and row tile stay.  Its waves split the contraction into windows of up to 4 S
// blocks (wave w takes windows w, w + W, ...): a wave holds a window's x operands in
// registers and walks the tile's weight rows, 16 at a time, Q loads of them ahead of
// their use -- also across tiles, so that the weight stream does not stop at a tile's
// end.  Its sums go to LDS, where the waves' are added in wave order.
//
// The 16 columns of an MFMA are 16 bf16 rows of x, or the three terms of four float32
// rows (term p of row q in column 4 p + q): the terms' sums are added at the end.
constexpr int kMaxWaves = 8, kGemvTile = 64;

template <typename T, int S, bool GROUPED>
__global__ __launch_bounds__(64 * kMaxWaves) void k_gemv(const GemvArgs a) {
  constexpr int X = XTerms<T>::kTerms;
  constexpr int XW = 2 * sizeof(T);        // words of 8 values of x
  constexpr int R = X == 1 ? 16 : 4;       // rows of x in an MFMA's columns
  constexpr int Q = S <= 2 ? 4 : 2;        // subtiles in flight (61 tokens, S = 3: 4 took 66.7 us, 2 63.4)
  extern __shared__ uint4 s_stage[];       // [waves][4 rows][64 runs], then
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int nblk = a.K / 32, rounds = a.rounds;
  constexpr int tile_n = kGemvTile, subs = tile_n / 16;
  constexpr int ldp = tile_n + 4;          // LDS column pitch: columns on different banks
  const uint32_t kbytes = a.K / 2;
  const T* const x = static_cast<const T*>(a.x);
  uint4* const stage = s_stage + 256 * wave;
  uint4* const s_scale = s_stage + 256 * waves;                          // [waves][64 rows] of 16 bytes
  float* const s_part = reinterpret_cast<float*>(s_scale + 64 * waves);  // [2][waves][16][ldp]
  int turn = 0;  // the sums of consecutive tiles alternate: one barrier a tile

  // this workgroup's run of tiles [t, t_end)
  GroupTiles<R> groups;
  int64_t row_tiles = ((int64_t)a.M + R - 1) / R;
  if constexpr (GROUPED) {
    groups.load(a.offs, a.groups, a.M);
    row_tiles = groups.total();
  }
  const int64_t tiles = row_tiles * a.slices * a.ntiles;
  const int64_t t0 = tiles * blockIdx.x / gridDim.x, t_end = tiles * (blockIdx.x + 1) / gridDim.x;
  if (t0 >= t_end) return;

  struct Place {
    int v, ks, nt;  // row tile, slice of the contraction, column tile
    int grp, m0, mrows, ncols;
  };
  const auto find = [&](Place& p) {
    p.ncols = (int)min<int64_t>(tile_n, a.N - (int64_t)p.nt * tile_n);
    p.grp = 0;
    if constexpr (GROUPED) {
      p.grp = groups.find(p.v, p.m0, p.mrows);
    } else {
      p.m0 = p.v * R;
      p.mrows = min(R, a.M - p.m0);
    }
  };
  const auto step_tile = [&](Place& p) {
    if (++p.nt == a.ntiles) {
      p.nt = 0;
      if (++p.ks == a.slices) p.ks = 0, ++p.v;
    }
    find(p);
  };
  Place cur;
  const int64_t strip = t0 / a.ntiles;
  cur.nt = (int)(t0 - strip * a.ntiles);
  cur.v = (int)(strip / a.slices);
  cur.ks = (int)(strip - (int64_t)cur.v * a.slices);
  find(cur);

  // The weight stream.  Offsets within a tile fit 32 bits (K < 2^26); rows past the last
  // read the last, lanes past the last block read block 0.  Past the workgroup's last
  // tile it repeats that tile's last rows.
  Place ahead = cur;
  int64_t t_ahead = t0;
  int round_ahead = 0, sub_ahead = 0;
  const uint8_t* codes;
  uint4 scale16;
  uint32_t c_at, c_end, b_at[S];
  const auto stream = [&]() {
    const int64_t row = (GROUPED ? ahead.grp * a.N : 0) + (int64_t)ahead.nt * tile_n;
    codes = a.codes + row * kbytes;
    const int b0 = ((ahead.ks * rounds + round_ahead) * waves + wave) * a.window;
    const int b1 = min(b0 + a.window, nblk);
    c_at = min(r16, ahead.ncols - 1) * kbytes;
    c_end = (ahead.ncols - 1) * kbytes;
#pragma unroll
    for (int s = 0; s < S; ++s) b_at[s] = (b0 + 4 * s + g < b1 ? b0 + 4 * s + g : 0) * 16;
    // The window's scale bytes of the tile's rows, a row a lane (at most 64): 16 bytes at
    // any alignment, byte by byte where the array ends within them.  Loaded with the codes,
    // a byte a lane, they touch as many cache lines as those: a kernel that only reads 265 MB
    // of weights took 70 us that way and 46 us without.
    const int64_t at = (row + min(lane, ahead.ncols - 1)) * a.scale_ld + b0;
    if (at + 16 <= a.scale_end) {
      __builtin_memcpy(&scale16, a.scales + at, 16);
    } else {
      uint64_t w[2] = {0, 0};
#pragma unroll 1
      for (int i = 0; at + i < a.scale_end; ++i) {
        const uint64_t byte = (uint64_t)a.scales[at + i] << (8 * (i & 7));
        w[0] |= i < 8 ? byte : 0;
        w[1] |= i < 8 ? 0 : byte;
      }
      scale16 = make_uint4((uint32_t)w[0], (uint32_t)(w[0] >> 32), (uint32_t)w[1],
                           (uint32_t)(w[1] >> 32));
    }
  };
  uint4 c[Q][S];
  const auto fetch = [&](int q) {
    if (sub_ahead == subs && (round_ahead + 1 < rounds || t_ahead + 1 < t_end)) {
      sub_ahead = 0;
      if (++round_ahead == rounds) {
        round_ahead = 0;
        ++t_ahead;
        step_tile(ahead);
      }
      stream();
    }
    ++sub_ahead;
#pragma unroll
    for (int s = 0; s < S; ++s)  // kept in the caches (non-temporal: 80 us for 63)
      c[q][s] = *reinterpret_cast<const uint4*>(codes + (c_at + b_at[s]));
    c_at = min(c_at + 16 * kbytes, c_end);
  };

  // The x operands.  Rows of x, 8 values a lane, go through the wave's LDS four at a time,
  // 64 runs of 8 values a row, and are read back by the lanes of their columns: block p's
  // run j.  Run 4 p + j lies at 4 p + (j ^ p / 4), which spreads the blocks over the banks.
  constexpr int kFours = R / 4;
  v8bf xt[S][4];
#pragma unroll
  for (int s = 0; s < S; ++s)
#pragma unroll
    for (int j = 0; j < 4; ++j) xt[s][j] = v8bf{};
  uint32_t xv[4][XW];     // four rows on their way
  int row_of = 0;         // lane q: the row of x of the tile's row q
  uint64_t real = ~0ull;  // the tile's rows whose row of x exists
  const auto x_rows = [&]() {
    row_of = cur.m0 + min(lane, cur.mrows - 1);
    if constexpr (GROUPED) {
      if (a.src) {
        const int slot = a.src[row_of];
        row_of = slot < 0 ? -1 : slot / a.top_k;
      }
      real = __ballot(row_of >= 0 && row_of < a.x_rows);
      if (row_of < 0 || row_of >= a.x_rows) row_of = 0;  // not stored below
    }
  };
  const auto x_load = [&](int four, int b0, int b1) {
    const int k0 = 32 * b0 + 8 * lane;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
#pragma unroll
      for (int k = 0; k < XW; ++k) xv[q][k] = 0;
      if (4 * four + q < cur.mrows && k0 < 32 * b1) {
        const int64_t r = __builtin_amdgcn_readlane(row_of, 4 * four + q);
        __builtin_memcpy(xv[q], x + (r * a.ldx + k0), 4 * XW);  // at T's alignment
      }
    }
  };
  const auto x_put = [&](int four, int b0, int b1) {
    const int row = min(r16 & 3, cur.mrows - 4 * four - 1);  // columns past the last row repeat it
#pragma unroll
    for (int k = 0; k < X; ++k) {
      wave_sync();
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (4 * four + q < cur.mrows)
          stage[64 * q + (lane ^ lane >> 4)] = XTerms<T>::take(xv[q]);
      wave_sync();
      if (k == X - 1 && four + 1 < kFours && 4 * four + 4 < cur.mrows) x_load(four + 1, b0, b1);
      if (r16 >> 2 == (X == 1 ? four : k)) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            xt[s][j] = __builtin_bit_cast(v8bf, stage[64 * row + 16 * s + 4 * g + (j ^ s)]);
      }
    }
  };

  // The waves' sums of a tile, cols() neighbouring columns a thread.
  const auto join = [&](auto cols) {
    constexpr int V = decltype(cols)::value;
    for (int o = threadIdx.x; o < cur.mrows * (tile_n / V); o += blockDim.x) {
      const int m = o / (tile_n / V), n = V * (o % (tile_n / V)), left = cur.ncols - n;
      if (left <= 0 || !(real >> m & 1)) continue;
      float sum[V] = {};
      if (nblk) {
        const float* const p = s_part + (turn * waves * 16 + m) * ldp + n;
        float v[X][kMaxWaves][V];  // all reads in flight, then the sum in order
#pragma unroll
        for (int k = 0; k < X; ++k)
#pragma unroll
          for (int w = 0; w < kMaxWaves; ++w)
            __builtin_memcpy(
                v[k][w], __builtin_assume_aligned(p + (min(w, waves - 1) * 16 + 4 * k) * ldp, 4 * V), 4 * V);
#pragma unroll
        for (int k = X - 1; k >= 0; --k)
#pragma unroll
          for (int w = 0; w < kMaxWaves; ++w)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[i] += w < waves ? v[k][w][i] : 0.0f;
      }
      const int64_t col = (int64_t)cur.nt * tile_n + n;
      if (a.slices > 1) {
        store_sums<V>(a.partial + ((int64_t)cur.ks * a.M + cur.m0 + m) * a.N + col, sum, left);
        continue;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) sum[i] *= a.alpha;
      const int64_t at = (int64_t)(cur.m0 + m) * a.ldy + col;
      if (a.y_bf16) store_sums<V>(static_cast<uint16_t*>(a.y) + at, sum, left);
      else store_sums<V>(static_cast<float*>(a.y) + at, sum, left);
    }
  };

  x_rows();
  if (nblk) {
    stream();
    fetch(0);
    const int b0 = (cur.ks * rounds * waves + wave) * a.window;
    x_load(0, b0, min(b0 + a.window, nblk));  // in front of the stream's second half
#pragma unroll
    for (int q = 1; q < Q; ++q) fetch(q);
  }
  bool fresh = true;
  for (int64_t t = t0;;) {
    for (int round = 0; round < rounds; ++round) {
      const int b0 = ((cur.ks * rounds + round) * waves + wave) * a.window;
      const int b1 = min(b0 + a.window, nblk);
      if (fresh || rounds > 1) {
        if (t > t0 || round > 0) {
          x_rows();
          x_load(0, b0, b1);
        }
#pragma unroll
        for (int four = 0; four < kFours; ++four)
          if (4 * four < cur.mrows) x_put(four, b0, b1);
      }
      if (nblk) {
        // these windows' scale bytes: the stream is at most a tile's subtiles ahead, so it has not
        // come to the next windows' yet
        wave_sync();
        s_scale[64 * wave + lane] = scale16;
        wave_sync();
        const uint8_t* const sb = reinterpret_cast<const uint8_t*>(s_scale + 64 * wave) + 16 * r16 + g;
#pragma unroll 1
        for (int sub = 0; sub < subs; sub += Q) {
          float f[Q][S];  // block scales; x is 0 past the window's end, but NaN and Inf times 0 are not
#pragma unroll
          for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int s = 0; s < S; ++s) {
              const uint32_t byte = sb[256 * (sub + q) + 4 * s];
              f[q][s] = scale_of(b0 + 4 * s + g < b1 ? byte : 127u);
            }
#pragma unroll
          for (int q = 0; q < Q; ++q) {
            v4f* const p = reinterpret_cast<v4f*>(s_part + ((turn * waves + wave) * 16 + r16) * ldp +
                                                  16 * (sub + q) + 4 * g);
            v4f acc[2] = {};  // two chains of sums
            if (round) acc[1] = *p;
#pragma unroll
            for (int s = 0; s < S; ++s) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint4 u = c[q][s];
                const uint32_t eight = j == 0 ? u.x : j == 1 ? u.y : j == 2 ? u.z : u.w;
                acc[j & 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    decode8_bf16(eight, f[q][s]), xt[s][j], acc[j & 1], 0, 0, 0);
              }
            }
            fetch(q);
            // lane 16 g + m holds weight rows 4 g .. 4 g + 3 of column m
            *p = acc[0] + acc[1];
          }
        }
      }
    }
    lds_barrier();
    // Four columns a thread keep this to half of the waves; with few rows it is the latency
    // that counts.  One and four columns a thread: 61 tokens x 4 of 32 experts (8 rows a tile)
    // 64.9 and 60.5 us, 1024 rows of 4096 x 4096 83.7 and 70.9, one token's 4 rows 10.7 and
    // 11.0.  A float32 x has four rows and three terms to read: two columns (256 rows of
    // 2880 x 2880 41.9 and 38.2 us).
    if constexpr (X == 3) join(std::integral_constant<int, 2>());
    else if (cur.mrows <= 4) join(std::integral_constant<int, 1>());
    else join(std::integral_constant<int, 4>());
    if (++t == t_end) break;
    turn ^= 1;
    const int grp = cur.grp, m0 = cur.m0, ks = cur.ks;
    step_tile(cur);
    fresh = cur.m0 != m0 || cur.grp != grp || cur.ks != ks;
  }
}

// y = alpha times the slices' sums, added in slice order.  Latency bound: 4.1 us for 47
// rows of 4096 in four slices (3.9 MB).
__global__ __launch_bounds__(256) void k_gemv_sum(const float* __restrict__ partial, int slices,
                                                  int64_t M, int64_t N, float alpha, void* y,
                                                  int y_bf16, int64_t ldy) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < M * N; i += (int64_t)gridDim.x * 256) {
    float sum = 0.0f;
    for (int k = 0; k < slices; ++k) sum += partial[k * M * N + i];
    const int64_t m = i / N, at = m * ldy + (i - m * N);
    sum *= alpha;
    if (y_bf16) static_cast<uint16_t*>(y)[at] = (uint16_t)f32_to_bf16_rne(sum);
    else static_cast<float*>(y)[at] = sum;
  }
}

// How a product is cut: steps of a window, waves, blocks of a wave's window, rounds of
// windows in one workgroup and slices over workgroups.
struct GemvPlan {
  int steps, waves, window, rounds, slices;
};

static constexpr int rows_per_tile(int x_dtype) { return x_dtype == MX_BF16 ? 16 : 4; }

constexpr int64_t kMaxPartial = (int64_t)1 << 26;  // floats of the slices' sums

static GemvPlan gemv_plan(int x_dtype, int64_t rows, int64_t N, int64_t K, bool grouped) {
  const int nblk = K ? (int)(K / 32) : 1;
  GemvPlan p;
  p.waves = (int)hmin(cdiv(nblk, 4), kMaxWaves);
  const auto passes = [&](int steps) { return (int)cdiv(nblk, 4 * steps * p.waves); };
  const int n = passes(4);
  p.steps = 1;
  while (passes(p.steps) > n) ++p.steps;
  // A contraction longer than a workgroup's windows goes in n rounds, which fetch x again
  // for every tile, or in n slices over workgroups and one more launch for their sums.
  // Slices pay where x is many rows or the tiles leave compute units idle.  Sliced and in
  // rounds, us: bf16 8192 x 8192 (n = 2) one row 14.1 and 11.3, 8 rows 14.4 and 14.6, 16
  // rows 15.1 and 18.5; 14336 x 14336 (n = 4) 8 rows 31.9 and 30.0, 40 rows 73.7 and 91.4;
  // one row of 4096 x 14336 (64 tiles) 13.9 and 18.8; float32 14336 x 14336 2 rows 30.5 and
  // 29.1, 4 rows 32.7 and 35.1; bf16 4096 x 14336 64 rows 32.6 and 34.8, 2048 rows 654 and
  // 854.  The sums take at most 256 MiB: past that it is rounds, for the workspace's sake.
  const bool slice = !grouped && n > 1 && rows * N <= kMaxPartial / n &&
                     (rows > rows_per_tile(x_dtype) / 2 || (n > 2 && cdiv(N, kGemvTile) <= 64));
  p.rounds = slice ? 1 : n;
  p.slices = slice ? n : 1;
  p.window = (int)cdiv(cdiv(nblk, (int64_t)n * p.waves), 4) * 4;
  return p;
}

template <typename T, int S, bool GROUPED>
static int gemv_launch(GemvArgs a, const GemvPlan& p, int64_t groups, hipStream_t st) {
  constexpr int R = rows_per_tile(sizeof(T) == 2 ? MX_BF16 : MX_F32);
  constexpr int kBytes = 5120 + 2 * 16 * (kGemvTile + 4) * 4;  // LDS of a wave
  static_assert(kMaxWaves * kBytes <= 160 * 1024, "the sums of all waves fit LDS");
  a.ntiles = cdiv(a.N, kGemvTile);
  a.window = p.window;
  a.rounds = p.rounds;
  a.slices = p.slices;
  // a group adds less than one row tile to the rows'
  const int64_t row_tiles = GROUPED ? cdiv(a.M, R) + groups : cdiv(a.M, R);
  const unsigned grid = (unsigned)hmin(row_tiles * p.slices * a.ntiles, device_cu_count());
  k_gemv<T, S, GROUPED><<<grid, 64 * p.waves, (size_t)p.waves * kBytes, st>>>(a);
  if (p.slices > 1)
    k_gemv_sum<<<(unsigned)hmin(cdiv(a.M * a.N, 256), 4096), 256, 0, st>>>(
        a.partial, p.slices, a.M, a.N, a.alpha, a.y, a.y_bf16, a.ldy);
  return launch_status();
}

template <typename T, bool GROUPED>
static int gemv_steps(const GemvArgs& a, const GemvPlan& p, int64_t groups, hipStream_t st) {
  if (p.steps == 1) return gemv_launch<T, 1, GROUPED>(a, p, groups, st);
  if (p.steps == 2) return gemv_launch<T, 2, GROUPED>(a, p, groups, st);
  if (p.steps == 3) return gemv_launch<T, 3, GROUPED>(a, p, groups, st);
  return gemv_launch<T, 4, GROUPED>(a, p, groups, st);
}

template <bool GROUPED>
static int gemv_any(const GemvArgs& a, const GemvPlan& p, int x_dtype, int64_t groups, hipStream_t st) {
  return x_dtype == MX_BF16 ? gemv_steps<uint16_t, GROUPED>(a, p, groups, st)
                            : gemv_steps<float, GROUPED>(a, p, groups, st);
}

static int gemv_check(const void* x, int x_dtype, int64_t ldx, const uint8_t* w_codes,
                      const uint8_t* w_scales, int64_t w_scale_ld, int64_t M, int64_t N, int64_t K,
                      const void* y, int y_dtype, int64_t ldy) {
  constexpr int64_t kMax31 = (int64_t)1 << 31;
  MX_REQUIRE((x_dtype == MX_F32 || x_dtype == MX_BF16) && (y_dtype == MX_F32 || y_dtype == MX_BF16),
             MX_ERR_ENUM);
  constexpr int64_t kMaxK = (int64_t)1 << 26;  // a tile's offsets stay within 32 bits
  MX_REQUIRE(M >= 0 && M < kMax31 && N >= 0 && N < kMax31 && K >= 0 && K < kMaxK && K % 32 == 0 &&
                 ldx >= K && ldy >= N && w_scale_ld >= K / 32 && w_scale_ld < kMaxK, MX_ERR_SHAPE);
  if (M == 0 || N == 0) return MX_OK;
  MX_REQUIRE(y, MX_ERR_NULL);
  if (K) MX_REQUIRE(x && w_codes && w_scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(x) && aligned16(w_codes) && aligned16(w_scales) && aligned16(y), MX_ERR_ALIGN);
  return MX_OK;
}

}  // namespace mx

using namespace mx;

extern "C" size_t mx_gemv_workspace_size(int x_dtype, int64_t M, int64_t N, int64_t K) {
  constexpr int64_t kMax31 = (int64_t)1 << 31;
  if ((x_dtype != MX_F32 && x_dtype != MX_BF16) || M <= 0 || N <= 0 || K < 0 || M >= kMax31 ||
      N >= kMax31 || K >= (int64_t)1 << 26 || K % 32)
    return 0;
  const GemvPlan p = gemv_plan(x_dtype, M, N, K, false);
  return p.slices > 1 ? (size_t)p.slices * M * N * sizeof(float) : 0;
}

extern "C" int mx_gemv(const void* x, int x_dtype, int64_t ldx, const uint8_t* w_codes,
                       const uint8_t* w_scales, int64_t w_scale_ld, int64_t M, int64_t N, int64_t K,
                       float alpha, void* y, int y_dtype, int64_t ldy, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const int bad = gemv_check(x, x_dtype, ldx, w_codes, w_scales, w_scale_ld, M, N, K, y, y_dtype, ldy);
  if (bad != MX_OK || M == 0 || N == 0) return bad;
  const size_t need = mx_gemv_workspace_size(x_dtype, M, N, K);
  if (need) {
    MX_REQUIRE(workspace && workspace_bytes >= need, MX_ERR_WORKSPACE);
    MX_REQUIRE(aligned16(workspace), MX_ERR_ALIGN);
  }
  const GemvPlan p = gemv_plan(x_dtype, M, N, K, false);
  GemvArgs a = {};
  a.x = x; a.ldx = ldx; a.x_rows = (int)M; a.M = (int)M; a.N = N; a.K = (int)K;
  a.codes = w_codes; a.scales = w_scales; a.scale_ld = w_scale_ld;
  a.scale_end = (N - 1) * w_scale_ld + K / 32;
  a.alpha = K ? alpha : 0.0f;  // an empty sum is 0 under any alpha
  a.y = y; a.y_bf16 = y_dtype == MX_BF16; a.ldy = ldy;
  a.partial = static_cast<float*>(workspace);
  return gemv_any<false>(a, p, x_dtype, 0, as_stream(stream));
}

extern "C" int mx_gemv_grouped(const void* x, int x_dtype, int64_t ldx, int64_t x_rows,
                               const int32_t* src, int64_t top_k, const uint8_t* w_codes,
                               const uint8_t* w_scales, int64_t w_scale_ld, const int64_t* offs,
                               int64_t groups, int64_t rows, int64_t N, int64_t K, float alpha,
                               void* y, int y_dtype, int64_t ldy, void* stream) {
  const int bad = gemv_check(x, x_dtype, ldx, w_codes, w_scales, w_scale_ld, rows, N, K, y, y_dtype, ldy);
  if (bad != MX_OK) return bad;
  MX_REQUIRE(groups >= 1 && groups <= MX_MAX_GROUPS && x_rows >= 0 && x_rows <= INT32_MAX &&
                 top_k >= 1 && top_k <= INT32_MAX, MX_ERR_SHAPE);
  if (rows == 0 || N == 0 || x_rows == 0) return MX_OK;
  MX_REQUIRE(offs, MX_ERR_NULL);
  MX_REQUIRE(aligned16(offs) && aligned16(src), MX_ERR_ALIGN);
  const int64_t held = hmin(groups, rows);  // at most `rows` groups hold rows
  const GemvPlan p = gemv_plan(x_dtype, rows, N, K, true);
  GemvArgs a = {};
  a.x = x; a.ldx = ldx; a.x_rows = (int)x_rows; a.src = src; a.top_k = (int)top_k;
  a.M = (int)rows; a.N = N; a.K = (int)K; a.offs = offs; a.groups = (int)groups;
  a.codes = w_codes; a.scales = w_scales; a.scale_ld = w_scale_ld;
  a.scale_end = (groups * N - 1) * w_scale_ld + K / 32;
  a.alpha = K ? alpha : 0.0f;  // an empty sum is 0 under any alpha
  a.y = y; a.y_bf16 = y_dtype == MX_BF16; a.ldy = ldy;
  return gemv_any<true>(a, p, x_dtype, held, as_stream(stream));
}
