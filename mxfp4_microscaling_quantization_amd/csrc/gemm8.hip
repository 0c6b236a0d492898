// Products of 8-bit block-scaled matrices:
//   C[m][n] = alpha sum_k deq(A)[m][k] deq(B)[n][k]
// A [M, K] and B [N, K] hold E4M3 codes and one E8M0 byte per 128 values of k.
//
// Two kinds of products.  A bf16 C takes the scaled 8-bit matrix instructions, which take the codes
// and scale bytes as they are (one byte per 32 values of k and row; a block of 128 gives the same
// byte four times).  They add the products of eight neighbouring values with about 14 bits below the
// largest of the eight before these sums meet in float32 (measured: a product 2^-13 of its neighbour
// survives, 2^-14 is lost, between groups 2^-23 survives): 2e-5 of C's norm for normal operands,
// against the 2e-3 of C's own rounding.  A float32 C takes V_MFMA_F32_*_BF16 instead (wide), half the
// rate: a code times a power of two is exact in bf16 (down to bits of 2^-133), and every product joins a
// float32 sum.
//
// Many rows are bound by the matrix units at the clock that power leaves (1.7 GHz in the 8-bit loop):
// 8192x14336x4096, bf16 360 to 380 us (2.6 PFLOP/s; its loop without loads and LDS reads 322);
// 4096x4096x4096 55 to 61 us, float32 106 to 111 (1.25 PFLOP/s).  Few rows are bound by reading B: one row of 14336x4096
// 12 us (4.9 TB/s).
//
// Per lane an operand is 32 bytes of one row: row (lane % 32), k [32 (lane / 32), + 32) of the 64 of
// V_MFMA_SCALE_F32_32X32X64_F8F6F4.  The bf16 instructions take a quarter of those each, 8 values a
// lane: k may run in any order as long as both operands agree.  B goes in first, so that a lane
// holds consecutive columns of a row of C.
//
// Code rows are padded with zeros to a multiple of 16 bytes (K is that multiple here), scale
// rows to whole dwords, which hold the bytes of 512 values of k.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gemm8_plan.h"
#include "mx_device8.h"
#include "mx_host8.h"

namespace mx {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

constexpr int kFmtE4m3 = 0;  // cbsz / blgp operand format

struct Gemm8Args {
  const uint8_t* a;
  const uint8_t* sa;
  const uint8_t* b;
  const uint8_t* sb;
  int64_t lda, lsa, ldb, lsb, M, N, K;
  void* c;
  int64_t ldc;
  float* part;    // sums of the sliced tiles: [slices][sliced tiles][128][128]
  int tiles_m, tiles_n;
  int whole;      // tiles in front of the sliced ones
  int slices;
  int64_t slice;  // contraction values a slice, a multiple of 512
  float alpha;
};

// Eight codes times a scale (0xFF: +Inf, which gives NaN), as bf16.
__device__ __forceinline__ v8bf widen8(uint32_t lo, uint32_t hi, float scale) {
  const v2bf a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const v2bf b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const v2bf c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const v2bf d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  v8bf v;
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  return v;
}

// The first n of a run of consecutive outputs (RAW: their 8 or 16 bytes) at T's alignment.  Nontemporal stores
// of whole lines take as long (8192x14336x4096 380 us, 12608x1536x384 20) and the next launch a little longer
// (with the gate of C behind it 445 and 441 us); of rows that start within lines, much longer (6385x11240 of
// K 32 68 and 41.5).
template <typename T, typename RAW>
__device__ __forceinline__ void store_run8(T* p, const RAW& raw, int64_t n) {
  typedef RAW avec __attribute__((aligned(sizeof(T))));
  constexpr int V = sizeof(RAW) / sizeof(T);
  if (n >= V) {
    *reinterpret_cast<avec*>(p) = raw;
  } else {
    T v[V];
    __builtin_memcpy(v, &raw, sizeof(raw));
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = v[i];
  }
}
template <typename T>
__device__ __forceinline__ void store_four8(T* p, const float* v, int64_t n) {
  if constexpr (sizeof(T) == 2) {
    const v2i raw = {(int)bf16_pair(v[0], v[1]), (int)bf16_pair(v[2], v[3])};
    store_run8(p, raw, n);
  } else {
    const v4f raw = {v[0], v[1], v[2], v[3]};
    store_run8(p, raw, n);
  }
}

// s_waitcnt with only the vector-memory counter constrained (gfx9 encoding).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

typedef __attribute__((address_space(3))) void* lds8_ptr_t;
// Direct global -> LDS loads from a scalar base and a 32-bit offset a lane: lane i's 16 (4) bytes
// land at LDS address M0 + 16 i (4 i).  Written as asm so that the compiler does not wait for
// them by itself; the kernel counts them and waits before its barriers.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void lds_load16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_load4(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
               :
               : "s"(lds), "v"(off), "s"(base)
               : "memory", "m0");
}
// A load from any address: the last step of a contraction takes its missing codes from here.
__device__ const uint4 kZero16 = {0, 0, 0, 0};
__device__ __forceinline__ void lds_load16_at(bool yes, const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %2\n\ts_mov_b32 exec_hi, %2\n\tglobal_load_lds_dwordx4 %1, off\n\ts_mov_b64 exec, -1"
               :
               : "s"(lds), "v"(p), "s"(__builtin_amdgcn_readfirstlane(yes ? -1 : 0))
               : "memory", "m0");
}
// The same loads if `yes`, without a branch (a branch between the products of a step would let the
// compiler move them past it): by no lane otherwise.  Every lane is active around them.
__device__ __forceinline__ void lds_load4_if(bool yes, const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_mov_b32 exec_lo, %3\n\ts_mov_b32 exec_hi, %3\n\tglobal_load_lds_dword %1, %2\n\ts_mov_b64 exec, -1"
               :
               : "s"(lds), "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(yes ? -1 : 0))
               : "memory", "m0");
}
__device__ __forceinline__ void lds_load4_at(const uint8_t* p, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" : : "s"(lds), "v"(p) : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ int64_t lmin8(int64_t a, int64_t b) { return a < b ? a : b; }

// ============================================================== tiles
// A tile's outputs.  A lane holds C[m = lr][n = 8 q + 4 lh + i] of each 32x32 accumulator.  A wave stages
// 64 rows at a time, in C's type, in its quarter of the idle LDS ring (16-byte chunks XORed with row & 15)
// and stores whole row segments.  It is alone on its SIMD, and every instruction counts: with bf16 rounded by
// integer operations after a float32 staging this took 6 of a tile's 57 us.
struct Out8 {
  void* c;
  int64_t m0, n0, M, N, ldc;
  float alpha;
};
template <int W, typename TY>
__device__ __forceinline__ void store_tile8(const Out8& g, v16f (&acc)[W][W], uint8_t* ring) {
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * W * 32, wn = (wave & 1) * W * 32;
  constexpr int RB = W * 32 * sizeof(TY);    // bytes a row
  constexpr int CH = RB / 16, MASK = CH < 16 ? CH - 1 : 15;
  constexpr int V = 16 / sizeof(TY);         // outputs a lane and store
  wait_vm<0>();
  __syncthreads();
  uint8_t* stg = ring + wave * 64 * RB;
  TY* c = static_cast<TY*>(g.c);
  const float alpha = g.alpha;
#pragma unroll
  for (int p = 0; p < W / 2; ++p) {
    auto stage = [&](auto SCALED) {
#pragma unroll
      for (int bb = 0; bb < 2; ++bb) {
        const int r = bb * 32 + lr;
#pragma unroll
        for (int a = 0; a < W; ++a)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = decltype(SCALED)::value ? acc[a][2 * p + bb][4 * q + e] * alpha : acc[a][2 * p + bb][4 * q + e];
            if constexpr (sizeof(TY) == 2)
              *reinterpret_cast<uint2*>(stg + r * RB + ((a * 4 + q) ^ (r & MASK)) * 16 + lh * 8) =
                  make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
            else
              *reinterpret_cast<float4*>(stg + r * RB + ((a * 8 + q * 2 + lh) ^ (r & MASK)) * 16) =
                  make_float4(v[0], v[1], v[2], v[3]);
          }
      }
    };
    // a float32 C has its factor always: a second copy of this would spill registers
    if (sizeof(TY) == 2 && alpha == 1.0f) stage(std::false_type{});
    else stage(std::true_type{});
#pragma unroll 4
    for (int it = 0; it < CH; ++it) {
      const int r = it * (64 / CH) + lane / CH, at = lane % CH;
      const v4i raw = *reinterpret_cast<const v4i*>(stg + r * RB + (at ^ (r & MASK)) * 16);
      const int64_t m = g.m0 + wm + p * 64 + r, n = g.n0 + wn + at * V;
      if (m < g.M && n < g.N) store_run8(c + m * g.ldc + n, raw, g.N - n);
    }
  }
}

// Which tile and slice a workgroup takes.  Workgroups are dealt round-robin over 8 dies: consecutive
// tiles go to one die; tile rows are walked four together, so that B tiles are read again from L2.
struct Place8 {
  int64_t m0, n0, k0, klen;
  int part;  // of the sliced tiles' sums; -1: a whole tile
};
template <int T>
__device__ __forceinline__ void tile8_at(const Gemm8Args& g, int id, int64_t* m0, int64_t* n0) {
  constexpr int kRows = 4;
  const int span = kRows * g.tiles_n, first_m = id / span * kRows;
  const int gm = min(g.tiles_m - first_m, kRows);
  *m0 = (int64_t)(first_m + id % span % gm) * T;
  *n0 = (int64_t)(id % span / gm) * T;
}
template <int T, bool SLICED>
__device__ __forceinline__ Place8 place8(const Gemm8Args& g, int block, int total) {
  Place8 p{0, 0, 0, g.K, -1};
  const bool sliced = SLICED && block >= g.whole;
  if (SLICED) {
    block -= sliced ? g.whole : 0;
    total = sliced ? total - g.whole : g.whole;
  }
  const int q = total / 8, r = total % 8, x = block % 8;
  int id = x * q + min(x, r) + block / 8;
  if (sliced) {
    const int tiles = g.tiles_m * g.tiles_n - g.whole, slice = id / tiles;
    p.part = id;
    id += g.whole - slice * tiles;
    p.k0 = slice * g.slice;
    p.klen = lmin8(g.slice, g.K - p.k0);
  }
  tile8_at<T>(g, id, &p.m0, &p.n0);
  return p;
}

template <int W, typename TY, bool SLICED>
__device__ __forceinline__ void finish8(const Gemm8Args& g, const Place8& at, v16f (&acc)[W][W], uint8_t* ring) {
  constexpr int T = W * 64;
  if constexpr (SLICED) {
    if (at.part >= 0) {
      store_tile8<W, float>(Out8{g.part + (int64_t)at.part * T * T, 0, 0, T, T, T, 1.0f}, acc, ring);
      return;
    }
  }
  store_tile8<W, TY>(Out8{g.c, at.m0, at.n0, g.M, g.N, g.ldc, g.alpha}, acc, ring);
}

// This wave's LDS reads have landed, then the workgroup's barrier.
__device__ __forceinline__ void barrier8() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int W>
__device__ __forceinline__ void clear8(v16f (&acc)[W][W]) {
#pragma unroll
  for (int a = 0; a < W; ++a)
#pragma unroll
    for (int b = 0; b < W; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[a][b][e] = 0.f;
}

// How many of n things are due before turn `at` of `turns`.
constexpr int due8(int at, int turns, int n) { return at <= 0 ? 0 : (at >= turns ? n : n * at / turns); }

// What a step knows of the loads that it issues: they are whole, or may end within the contraction or be past it,
// or there are none (a product's last two steps; the wide kernel without masked loads there, and with whole ones in
// its prologue, 12608x1536x384 28.8 -> 25.7 us; the 8-bit one spills by it).
struct Whole8 {
  static constexpr bool sure = true, none = false;
};
struct Maybe8 {
  static constexpr bool sure = false, none = false;
};
struct None8 {
  static constexpr bool sure = false, none = true;
};

// The 8-bit instructions' kernel.  A wave holds the A fragments of a whole step and goes through its W column
// tiles of B one after the other ("turns" of 2 W products).  In turn b it reads column tile b + 1, in the second
// half of a step also the next step's A.  So A's part of a stage is free as soon as its step begins, and B's
// tile by tile; the loads of step p + 2 follow at once, in two groups, each behind a barrier that ends the
// reads of what it overwrites:
//   first half of step p    B tiles W/2+1 .. W-1 of step p + 1, A of step p + 2
//   second half of step p   B tiles 0 .. W/2 of step p + 2
// Everything is on its way for a step at least before the barrier in front of its first read, where
// its wave waits for it.  Between two products of a wave there is room for a read or a load: 64 cycles.
template <int T, typename TY, bool SLICED>
__device__ __forceinline__ void tile8(const Gemm8Args& g, int block, int blocks, uint8_t* ring, uint32_t (&s_scale)[2][2 * T]) {
  constexpr int W = T / 64;
  constexpr int LA = T / 32;                   // A loads a wave and step (8 rows each)
  constexpr int NB = W / 2 + 1;                // B tiles loaded in the second half of a step (2 loads each)
  constexpr int kFirst = 2 * (W - NB) + LA, kSecond = 2 * NB;
  constexpr int LS = T / 128;                  // scale loads a wave and four steps (64 rows each)
  constexpr int STAGE = 2 * T * 128;

  const Place8 at = place8<T, SLICED>(g, block, blocks);
  const int64_t m0 = at.m0, n0 = at.n0, klen = at.klen;
  const int KT = (int)((klen + 127) / 128);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = (wave >> 1) * (T / 2), wn = (wave & 1) * (T / 2);
  const int lr = lane & 31, lh = lane >> 5;
  const uint32_t ring0 = (uint32_t)(uintptr_t)(lds8_ptr_t)ring;
  const uint32_t scale0 = (uint32_t)(uintptr_t)(lds8_ptr_t)s_scale;

  // Sources, rows past the matrix clamped to its last (they feed outputs that are not stored).  A
  // wave loads T/4 rows of A, and of each B tile (32 rows of either half) 16 rows.
  const uint8_t* abase = g.a + m0 * g.lda + at.k0;
  const uint8_t* bbase = g.b + n0 * g.ldb + at.k0;
  const int64_t alast = g.M - m0 - 1, blast = g.N - n0 - 1;
  auto a_row = [&](int j) { return wave * (T / 4) + j * 8; };
  auto b_row = [&](int j) { return (wave >> 1) * (T / 2) + (j >> 1) * 32 + (wave & 1) * 16 + (j & 1) * 8; };
  const int dr = lane >> 3;
  auto chunk = [&](int row0) { return ((lane & 7) ^ (((row0 + dr) >> 1) & 7)) * 16; };  // of this lane's load
  uint32_t aoff[LA], boff[2 * W];
#pragma unroll
  for (int j = 0; j < LA; ++j) aoff[j] = (uint32_t)(lmin8(a_row(j) + dr, alast) * g.lda) + chunk(a_row(j));
#pragma unroll
  for (int j = 0; j < 2 * W; ++j) boff[j] = (uint32_t)(lmin8(b_row(j) + dr, blast) * g.ldb) + chunk(b_row(j));
  const bool isA = wave < 2;
  const uint8_t* sbase = (isA ? g.sa + m0 * g.lsa : g.sb + n0 * g.lsb) + at.k0 / 128;
  uint32_t soff[LS];
#pragma unroll
  for (int j = 0; j < LS; ++j)
    soff[j] = (uint32_t)(lmin8((wave & 1) * (T / 2) + j * 64 + lane, isA ? alast : blast) * (isA ? g.lsa : g.lsb));

  // A load of step p (j < LA: A's j-th, else B's).  SURE: the step exists and is whole.  Else chunks
  // past the contraction are zeros, and steps past it are not loaded.
  auto issue_one = [&](int p, int j, auto SURE) {
    const int row0 = j < LA ? a_row(j) : T + b_row(j - LA);
    const uint32_t to = ring0 + (uint32_t)(p & 1) * STAGE + (uint32_t)row0 * 128;
    const uint8_t* base = (j < LA ? abase : bbase) + (int64_t)p * 128;
    const uint32_t off = j < LA ? aoff[j] : boff[j - LA];
    if constexpr (decltype(SURE)::sure) {
      lds_load16(base, off, to);
    } else {
      const int c = chunk(j < LA ? a_row(j) : b_row(j - LA));
      lds_load16_at(p < KT, (int64_t)p * 128 + c < klen ? base + off : reinterpret_cast<const uint8_t*>(&kZero16), to);
    }
  };
  auto issue_first = [&](int p, int i, auto SURE) {   // load i of the first half of step p
    if (i < 2 * (W - NB)) issue_one(p + 1, LA + 2 * NB + i, SURE);
    else issue_one(p + 2, i - 2 * (W - NB), SURE);
  };
  auto issue_scales = [&](int grp, bool yes) {        // of steps 4 grp .. 4 grp + 3
#pragma unroll
    for (int j = 0; j < LS; ++j)
      lds_load4_if(yes, sbase + grp * 4, soff[j],
                   scale0 + (uint32_t)((grp & 1) * 2 * T + wave * (T / 2) + j * 64) * 4);
  };

  v16f acc[W][W];
  clear8(acc);

  // Fragments: both 64-halves of the rows of A, of this step and the next, and of two B tiles.  Half h of a
  // row's 128 bytes: chunks 4 h + 2 lh and the next.
  v8i fa[2][W][2], fb[2][2];
  uint32_t sa[W], sb[W], na[W], nb[W];
  const uint8_t *pa[4], *pb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = ((4 * (i >> 1) + 2 * lh + (i & 1)) ^ ((lr >> 1) & 7)) * 16;
    pa[i] = ring + (wm + lr) * 128 + c;
    pb[i] = ring + (T + wn + lr) * 128 + c;
  }
  auto put = [&](v8i& f, int e, const v4i& c) {
    f = e ? __builtin_shufflevector(f, __builtin_shufflevector(c, c, 0, 1, 2, 3, 0, 1, 2, 3), 0, 1, 2, 3, 8, 9, 10, 11)
          : __builtin_shufflevector(c, c, 0, 1, 2, 3, -1, -1, -1, -1);
  };
  auto read_a = [&](auto P, int p, int i) {           // read i of 4 W: tile i / 4
    constexpr int q = decltype(P)::value;
    put(fa[q][i >> 2][(i >> 1) & 1], i & 1,
        *reinterpret_cast<const v4i*>(pa[i & 3] + (p & 1) * STAGE + (i >> 2) * 32 * 128));
  };
  auto read_b = [&](int p, int tile, int i) {         // read i of 4
    put(fb[tile & 1][i >> 1], i & 1, *reinterpret_cast<const v4i*>(pb[i] + (p & 1) * STAGE + tile * 32 * 128));
  };
  auto read_scales = [&](int p, uint32_t (&x)[W], uint32_t (&y)[W]) {
    const uint8_t* s = reinterpret_cast<const uint8_t*>(s_scale[(p >> 2) & 1]) + (p & 3);
#pragma unroll
    for (int t = 0; t < W; ++t) {
      x[t] = s[(wm + t * 32 + lr) * 4];
      y[t] = s[(T + wn + t * 32 + lr) * 4];
    }
  };
  // Prologue, in the order of the steps: scales, step 0 but for its last B tiles; those and A of step 1;
  // the first B tiles of step 1.
  issue_scales(0, true);
#pragma unroll
  for (int j = 0; j < LA + 2 * NB; ++j) issue_one(0, j, Maybe8{});
#pragma unroll
  for (int i = 0; i < kFirst; ++i) issue_first(-1, i, Maybe8{});
#pragma unroll
  for (int i = 0; i < kSecond; ++i) issue_one(1, LA + i, Maybe8{});
  if (KT > 1) wait_vm<2 * (NB - 1) + kFirst + kSecond>();
  else wait_vm<0>();
  barrier8();
  read_scales(0, sa, sb);
#pragma unroll
  for (int i = 0; i < 4 * W; ++i) read_a(std::integral_constant<int, 0>{}, 0, i);
#pragma unroll
  for (int i = 0; i < 4; ++i) read_b(0, 0, i);

  // Turn B of step p, p % 2 == P.  SURE: steps p + 1 and p + 2 exist and are whole.
  auto turn = [&](int p, auto P, auto B, auto SURE) {
    constexpr int q = decltype(P)::value, b = decltype(B)::value;
    constexpr bool sure = decltype(SURE)::sure;
    constexpr bool second = b >= W / 2;
    constexpr int kTurn = 2 * W, kHalf = kTurn * W / 2;  // products
    if constexpr (b == 0) {  // B tiles 1 .. W/2 of this step have landed
      if (sure || p + 1 < KT) wait_vm<kFirst + kSecond>();
      else wait_vm<2 * (W - NB)>();
      barrier8();
      issue_scales((p >> 2) + 1, (p & 3) == 0 && p + 4 < KT);
    }
    if constexpr (b == W / 2) {  // the other B tiles, A and B tile 0 of the next step have landed
      if (sure || p + 2 < KT) wait_vm<2 * (NB - 1) + kFirst>();
      else if (p + 1 < KT) wait_vm<2 * (NB - 1) + 2 * (W - NB)>();
      else wait_vm<0>();
      barrier8();
    }
    if constexpr (b == W - 1) read_scales(p + 1, na, nb);
    constexpr int kReads = second ? 4 + 8 : 4;  // of this turn
#pragma unroll
    for (int i = 0; i < kTurn; ++i) {
      const int h = i / W, a = i % W;
      acc[b][a] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[b & 1][h], fa[q][a][h], acc[b][a], kFmtE4m3,
                                                                  kFmtE4m3, 0, (int)sb[b], 0, (int)sa[a]);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = due8(i, kTurn, kReads); r < due8(i + 1, kTurn, kReads); ++r) {
        if (r < 4) read_b(b == W - 1 ? p + 1 : p, (b + 1) % W, r);
        else read_a(std::integral_constant<int, 1 - q>{}, p + 1, (b - W / 2) * 8 + r - 4);
      }
      const int done = (second ? b - W / 2 : b) * kTurn + i;
      if constexpr (second) {
#pragma unroll
        for (int l = due8(done, kHalf, kSecond); l < due8(done + 1, kHalf, kSecond); ++l) issue_one(p + 2, LA + l, SURE);
      } else {
#pragma unroll
        for (int l = due8(done, kHalf, kFirst); l < due8(done + 1, kHalf, kFirst); ++l) issue_first(p, l, SURE);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  auto step = [&](int p, auto P, auto SURE) {
    turn(p, P, std::integral_constant<int, 0>{}, SURE);
    turn(p, P, std::integral_constant<int, 1>{}, SURE);
    if constexpr (W == 4) {
      turn(p, P, std::integral_constant<int, 2>{}, SURE);
      turn(p, P, std::integral_constant<int, 3>{}, SURE);
    }
#pragma unroll
    for (int t = 0; t < W; ++t) sa[t] = na[t], sb[t] = nb[t];
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  int p = 0;
  for (; (int64_t)(p + 4) * 128 <= klen; p += 2) {
    step(p, I0{}, Whole8{});
    step(p + 1, I1{}, Whole8{});
  }
  for (; p < KT; p += 2) {
    step(p, I0{}, Maybe8{});
    if (p + 1 < KT) step(p + 1, I1{}, Maybe8{});
  }
  finish8<W, TY, SLICED>(g, at, acc, ring);
}

// The wide kernel's loads and LDS reads: two stages as above.  (The 8-bit kernel has them in its own body:
// through this struct it took some more registers, which spilled, and 374 us became 397.)
template <int T>
struct Feed8 {
  static constexpr int W = T / 64;           // accumulators of 32x32 of a wave along m and n
  static constexpr int LA = T / 32;          // A loads a wave and step (8 rows each)
  static constexpr int LB = T / 32;          // B loads: of each tile of 32 columns (of either half) two
  static constexpr int LS = T / 128;         // scale loads a wave and four steps (64 rows each)
  static constexpr int STAGE = 2 * T * 128;
  uint8_t* ring;
  uint32_t* scales;                          // [2][2 T]: the bytes of four steps
  const uint8_t *abase, *bbase, *sbase;
  uint32_t aoff[LA], boff[LB], soff[LS];
  uint32_t ring0, scale0;
  int64_t klen;
  int KT, wave, dr, lane;
  uint32_t pa[4], pb[4];                     // fragment chunks in a stage: half i / 2 of the step, 16 bytes i % 2

  __device__ __forceinline__ int a_row(int j) const { return wave * (T / 4) + j * 8; }
  __device__ __forceinline__ int b_row(int j) const {
    return (wave >> 1) * (T / 2) + (j >> 1) * 32 + (wave & 1) * 16 + (j & 1) * 8;
  }
  __device__ __forceinline__ int chunk(int row0) const { return ((lane & 7) ^ (((row0 + dr) >> 1) & 7)) * 16; }

  __device__ __forceinline__ Feed8(const Gemm8Args& g, const Place8& at, uint8_t* r, uint32_t* s) : ring(r), scales(s) {
    const int tid = threadIdx.x;
    lane = tid & 63;
    dr = lane >> 3;
    wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    ring0 = (uint32_t)(uintptr_t)(lds8_ptr_t)ring;
    scale0 = (uint32_t)(uintptr_t)(lds8_ptr_t)scales;
    klen = at.klen;
    KT = (int)((klen + 127) / 128);
    abase = g.a + at.m0 * g.lda + at.k0;
    bbase = g.b + at.n0 * g.ldb + at.k0;
    const int64_t alast = g.M - at.m0 - 1, blast = g.N - at.n0 - 1;
#pragma unroll
    for (int j = 0; j < LA; ++j) aoff[j] = (uint32_t)(lmin8(a_row(j) + dr, alast) * g.lda) + chunk(a_row(j));
#pragma unroll
    for (int j = 0; j < LB; ++j) boff[j] = (uint32_t)(lmin8(b_row(j) + dr, blast) * g.ldb) + chunk(b_row(j));
    const bool isA = wave < 2;
    sbase = (isA ? g.sa + at.m0 * g.lsa : g.sb + at.n0 * g.lsb) + at.k0 / 128;
#pragma unroll
    for (int j = 0; j < LS; ++j)
      soff[j] = (uint32_t)(lmin8((wave & 1) * (T / 2) + j * 64 + lane, isA ? alast : blast) * (isA ? g.lsa : g.lsb));
    const int lr = lane & 31, lh = lane >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = ((4 * (i >> 1) + 2 * lh + (i & 1)) ^ ((lr >> 1) & 7)) * 16;
      pa[i] = ((wave >> 1) * (T / 2) + lr) * 128 + c;
      pb[i] = (T + (wave & 1) * (T / 2) + lr) * 128 + c;
    }
  }

  // A load of step p (j < LA: A's j-th, else B's).  SURE: the step exists and is whole.  Else chunks
  // past the contraction are zeros, and steps past it are not loaded.
  template <bool SURE>
  __device__ __forceinline__ void issue(int p, int j) const {
    const int row0 = j < LA ? a_row(j) : T + b_row(j - LA);
    const uint32_t to = ring0 + (uint32_t)(p & 1) * STAGE + (uint32_t)row0 * 128;
    const uint8_t* base = (j < LA ? abase : bbase) + (int64_t)p * 128;
    uint32_t off = j < LA ? aoff[j] : boff[j - LA];
    if constexpr (SURE) {
      lds_load16(base, off, to);
    } else {
      int c = ((lane & 7) ^ ((dr >> 1) & 7)) * 16;  // chunk() of this row
      c = j & 1 ? c ^ 64 : c;
      asm volatile("" : "+v"(off), "+v"(c));  // kept from being held, added up, over the last steps' loop
      lds_load16_at(p < KT, (int64_t)p * 128 + c < klen ? base + off : reinterpret_cast<const uint8_t*>(&kZero16), to);
    }
  }
  __device__ __forceinline__ void issue_scales(int grp, bool yes) const {  // of steps 4 grp .. 4 grp + 3
#pragma unroll
    for (int j = 0; j < LS; ++j)
      lds_load4_if(yes, sbase + grp * 4, soff[j],
                   scale0 + (uint32_t)((grp & 1) * 2 * T + wave * (T / 2) + j * 64) * 4);
  }
  // 16 bytes e of half h of this lane's row of A's (B's) tile t of step p, into operand f
  static __device__ __forceinline__ void put(v8i& f, int e, const v4i& c) {
    f = e ? __builtin_shufflevector(f, __builtin_shufflevector(c, c, 0, 1, 2, 3, 0, 1, 2, 3), 0, 1, 2, 3, 8, 9, 10, 11)
          : __builtin_shufflevector(c, c, 0, 1, 2, 3, -1, -1, -1, -1);
  }
  __device__ __forceinline__ void read_a(v8i& f, int p, int t, int h, int e) const {
    put(f, e, *reinterpret_cast<const v4i*>(ring + pa[2 * h + e] + (p & 1) * STAGE + t * 32 * 128));
  }
  __device__ __forceinline__ void read_b(v8i& f, int p, int t, int h, int e) const {
    put(f, e, *reinterpret_cast<const v4i*>(ring + pb[2 * h + e] + (p & 1) * STAGE + t * 32 * 128));
  }
  __device__ __forceinline__ void read_scales(int p, uint32_t (&x)[W], uint32_t (&y)[W]) const {
    const uint8_t* s = reinterpret_cast<const uint8_t*>(scales + ((p >> 2) & 1) * 2 * T) + (p & 3);
    const int lr = lane & 31;
#pragma unroll
    for (int t = 0; t < W; ++t) {
      x[t] = s[((wave >> 1) * (T / 2) + t * 32 + lr) * 4];
      y[t] = s[(T + (wave & 1) * (T / 2) + t * 32 + lr) * 4];
    }
  }
};

// The wide kernel: a wave holds the fragments of two halves of a step (64 values of k each), reads the next
// half's while one half's products run, 4 W^2 of 32 cycles, and widens them 8 values a lane at a time.  One
// barrier a step, in front of its second half: by then every wave has that half in registers, so the step's
// stage is free for the loads of step p + 2, and the loads of step p + 1, issued a step ago, have landed.
template <int T, typename TY, bool SLICED>
__device__ __forceinline__ void wide8(const Gemm8Args& g, int block, int blocks, uint8_t* ring, uint32_t (&s_scale)[2][2 * T]) {
  using Feed = Feed8<T>;
  constexpr int W = Feed::W, L = Feed::LA + Feed::LB;
  const Place8 at = place8<T, SLICED>(g, block, blocks);
  const Feed feed(g, at, ring, s_scale[0]);
  const int KT = feed.KT;

  v16f acc[W][W];
  clear8(acc);
  v8i fa[2][W], fb[2][W];
  uint32_t sa[W], sb[W], na[W], nb[W];
  auto read_one = [&](auto H, int p, int i) {  // read i of 4 W of half H of step p
    constexpr int h = decltype(H)::value;
    if (i & 2) feed.read_b(fb[h][i >> 2], p, i >> 2, h, i & 1);
    else feed.read_a(fa[h][i >> 2], p, i >> 2, h, i & 1);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  feed.issue_scales(0, true);
  auto prologue = [&](auto SURE) {
#pragma unroll
    for (int j = 0; j < 2 * L; ++j) feed.template issue<decltype(SURE)::sure>(j / L, j % L);
  };
  if (feed.klen >= 256) prologue(Whole8{});
  else prologue(Maybe8{});
  if (KT > 1) wait_vm<L>();
  else wait_vm<0>();
  barrier8();
  feed.read_scales(0, sa, sb);
#pragma unroll
  for (int i = 0; i < 4 * W; ++i) read_one(I0{}, 0, i);

  // Half H of step p.  SURE: step p + 2 exists and is whole.
  auto half = [&](int p, auto H, auto SURE) {
    constexpr int h = decltype(H)::value;
    if constexpr (h == 1) {
      wait_vm<0>();
      barrier8();
      feed.issue_scales((p >> 2) + 1, (p & 3) == 0 && p + 4 < KT);
      feed.read_scales(p + 1, na, nb);
    }
    constexpr int kProducts = 4 * W * W;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v8bf xa[W], xb[W];
#pragma unroll
      for (int t = 0; t < W; ++t) {
        xa[t] = widen8(fa[h][t][2 * j], fa[h][t][2 * j + 1], scale_of(sa[t]));
        xb[t] = widen8(fb[h][t][2 * j], fb[h][t][2 * j + 1], scale_of(sb[t]));
      }
#pragma unroll
      for (int i = 0; i < W * W; ++i) {
        const int a = i / W, b = i % W, done = j * W * W + i;
        acc[a][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(xb[a], xa[b], acc[a][b], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int r = due8(done, kProducts, 4 * W); r < due8(done + 1, kProducts, 4 * W); ++r)
          read_one(std::integral_constant<int, 1 - h>{}, p + h, r);
        if constexpr (h == 1 && !decltype(SURE)::none) {
#pragma unroll
          for (int l = due8(done, kProducts, L); l < due8(done + 1, kProducts, L); ++l)
            feed.template issue<decltype(SURE)::sure>(p + 2, l);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (h == 1) {
#pragma unroll
      for (int t = 0; t < W; ++t) sa[t] = na[t], sb[t] = nb[t];
    }
  };
  int p = 0;
  for (; (int64_t)(p + 3) * 128 <= feed.klen; ++p) {
    half(p, I0{}, Whole8{});
    half(p, I1{}, Whole8{});
  }
  for (; p + 2 < KT; ++p) {
    half(p, I0{}, Maybe8{});
    half(p, I1{}, Maybe8{});
  }
  for (; p < KT; ++p) {
    half(p, I0{}, None8{});
    if ((int64_t)p * 128 + 64 < feed.klen) half(p, I1{}, None8{});
  }
  finish8<W, TY, SLICED>(g, at, acc, ring);
}

template <int T, typename TY, bool SLICED>
__global__ __launch_bounds__(256, T == 256 ? 1 : 2) void k_gemm8_tile(const Gemm8Args g) {
  __shared__ __align__(16) uint8_t ring[4 * T * 128];
  __shared__ __align__(16) uint32_t s_scale[2][2 * T];
  tile8<T, TY, SLICED>(g, blockIdx.x, gridDim.x, ring, s_scale);
}
template <int T, typename TY, bool SLICED>
__global__ __launch_bounds__(256, T == 256 ? 1 : 2) void k_gemm8_wide(const Gemm8Args g) {
  __shared__ __align__(16) uint8_t ring[4 * T * 128];
  __shared__ __align__(16) uint32_t s_scale[2][2 * T];
  wide8<T, TY, SLICED>(g, blockIdx.x, gridDim.x, ring, s_scale);
}

// Two products in one launch in tiles of 128, x's C of type TY and w's float32: w's workgroups in front, or
// behind x's.  The second's begin at a multiple of 8, so that each die has whole runs of either's tiles.  One's
// last, partial round of workgroups runs beside the other's first (the layer's backward, 12608x1536x384 64.1 us
// by a launch each, 55.5 so; 2048x2048x2048 49 and 41.5; 500x384x384 20.2 and 15.4; 4096x2048x2048 float32 72 and 64).
template <typename TY>
__global__ __launch_bounds__(256, 2) void k_gemm8_two(const Gemm8Args x, int x_blocks, const Gemm8Args w, int w_blocks,
                                                      int w_front) {
  constexpr int T = 128;
  __shared__ __align__(16) uint8_t ring[4 * T * 128];
  __shared__ __align__(16) uint32_t s_scale[2][2 * T];
  const int front = ((w_front ? w_blocks : x_blocks) + 7) & ~7;
  const bool behind = (int)blockIdx.x >= front, of_w = behind != (bool)w_front;
  const int block = behind ? (int)blockIdx.x - front : (int)blockIdx.x, blocks = of_w ? w_blocks : x_blocks;
  if (block >= blocks) return;
  if (of_w) wide8<T, float, true>(w, block, blocks, ring, s_scale);
  else if constexpr (sizeof(TY) == 4) wide8<T, TY, true>(x, block, blocks, ring, s_scale);
  else tile8<T, TY, true>(x, block, blocks, ring, s_scale);
}

// The sliced tiles of C: alpha times their slices' sums, in their order.  Eight rows a workgroup.
template <typename TY>
__global__ __launch_bounds__(256) void k_gemm8_sum(const Gemm8Args g) {
  constexpr int T = 128;
  const int tiles = g.tiles_m * g.tiles_n - g.whole, tile = (int)blockIdx.x / 16;
  const int row = (int)blockIdx.x % 16 * 8 + (int)threadIdx.x / 32, col = (int)threadIdx.x % 32 * 4;
  int64_t m, n;
  tile8_at<T>(g, g.whole + tile, &m, &n);
  m += row;
  n += col;
  if (m >= g.M || n >= g.N) return;
  const float* p = g.part + ((int64_t)tile * T + row) * T + col;
  const int64_t step = (int64_t)tiles * T * T;
  v4f s = *reinterpret_cast<const v4f*>(p);
#pragma unroll 4
  for (int k = 1; k < g.slices; ++k) s += *reinterpret_cast<const v4f*>(p + k * step);
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = s[e] * g.alpha;
  store_four8(static_cast<TY*>(g.c) + m * g.ldc + n, v, g.N - n);
}

// ============================================================== few rows
// Up to 64 rows of A: the weights are read once, and that read is the bound.  A wave takes 16 NT columns,
// all rows (8 XD of them) and a part of K, and streams both operands through a ring of its own in LDS, four
// steps of 128 deep: no barrier until the waves' sums meet.  The detour keeps loads whole: eight lanes take a
// line of 128 bytes (into the operand registers directly, neighbouring lanes take different rows, 16 bytes a
// clock: one row of 14336x4096 14.8 us, 12.1 so, 47 of 4096x14336 35 us, 17 so), and holds what is
// in flight, 4 KB a step and up.  Layout of a step as in the tiles: row r's chunks in the order c ^ ((r >> 1) & 7).
constexpr int kRowsDepth = 4;
constexpr int rows8_step(int xd, int nt) { return (2 * nt + xd) * 1024; }         // bytes in LDS
constexpr int rows8_scales(int xd, int nt) { return (16 * nt + 8 * xd + 63) / 64; } // loads per four steps
constexpr int rows8_lds(int xd, int nt) { return kRowsDepth * rows8_step(xd, nt) + 2 * rows8_scales(xd, nt) * 256; }

struct Rows8Args {
  Gemm8Args g;
  int steps, per;  // steps of the contraction and of a wave (a multiple of 4)
};

template <int XD, int NT, typename TY>
__global__ __launch_bounds__(512) void k_gemm8_rows(const Rows8Args r) {
  constexpr int MT = (XD + 1) / 2;                       // row tiles of 16
  constexpr int LC = 2 * NT + XD, LS = rows8_scales(XD, NT);
  constexpr int STEP = rows8_step(XD, NT);
  static_assert((kRowsDepth - 1) * LC + LS < 64 && MT * NT * 1024 <= kRowsDepth * STEP, "loads in flight, room for the sums");
  extern __shared__ __align__(16) uint8_t lds[];
  const Gemm8Args& g = r.g;
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = blockDim.x >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * NT);
  uint8_t* ring = lds + wave * rows8_lds(XD, NT);
  uint8_t* scales = ring + kRowsDepth * STEP;
  const uint32_t ring0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds8_ptr_t)ring);
  const int first = wave * r.per, end = min(first + r.per, r.steps);

  const int dr = lane >> 3;
  const uint8_t* wbase = g.b + n0 * g.ldb;
  uint32_t off[LC];  // this lane's chunk of step 0: B's loads (from wbase), then A's
#pragma unroll
  for (int j = 0; j < LC; ++j) {
    const int row = (j < 2 * NT ? j : j - 2 * NT) * 8 + dr;
    off[j] = (uint32_t)(j < 2 * NT ? lmin8(row, g.N - 1 - n0) * g.ldb : lmin8(row, g.M - 1) * g.lda) +
             ((lane & 7) ^ ((row >> 1) & 7)) * 16;
  }
  const uint8_t* ssrc[LS];  // scale rows: B's 16 NT, then A's
#pragma unroll
  for (int j = 0; j < LS; ++j) {
    const int row = j * 64 + lane;
    ssrc[j] = row < 16 * NT ? g.sb + lmin8(n0 + row, g.N - 1) * g.lsb
                            : g.sa + lmin8(row - 16 * NT, g.M - 1) * g.lsa;
  }
  auto issue = [&](int s) {
    if ((s & 3) == 0) {
#pragma unroll
      for (int j = 0; j < LS; ++j)
        lds_load4_at(ssrc[j] + s, ring0 + kRowsDepth * STEP + (((s >> 2) & 1) * LS + j) * 256);
    }
    const int64_t k = (int64_t)s * 128;
    const uint32_t to = ring0 + (s % kRowsDepth) * STEP;
    if (k + 128 <= g.K) {
#pragma unroll
      for (int j = 0; j < LC; ++j) lds_load16((j < 2 * NT ? wbase : g.a) + k, off[j], to + j * 1024);
    } else {  // the last step: chunks past the contraction are zeros
      const int c0 = ((lane & 7) ^ ((dr >> 1) & 7)) * 16;
#pragma unroll
      for (int j = 0; j < LC; ++j) {  // odd loads: rows 8 further, the chunk's bit 2 flipped
        const bool in = k + (j & 1 ? c0 ^ 64 : c0) < g.K;
        lds_load16_at(true, in ? (j < 2 * NT ? wbase : g.a) + k + off[j] : reinterpret_cast<const uint8_t*>(&kZero16),
                      to + j * 1024);
      }
    }
  };

  v4f acc[NT][MT];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[a][b][e] = 0.f;

#pragma unroll
  for (int i = 0; i < kRowsDepth; ++i)
    if (first + i < end) issue(first + i);
  const uint8_t *at[2], *last[2];  // this lane's chunks of a tile; of the last one, which has 8 rows where XD is odd
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = XD & 1 ? l16 & 7 : l16;
    at[h] = ring + l16 * 128 + ((2 * kg + h) ^ ((l16 >> 1) & 7)) * 16;
    last[h] = ring + (NT + MT - 1) * 2048 + row * 128 + ((2 * kg + h) ^ ((row >> 1) & 7)) * 16;
  }
  for (int s = first; s < end; ++s) {
    // steps s + 1 .. s + 3 may stay in flight
    if (s + 3 < end) wait_vm<3 * LC>();
    else if (s + 2 < end) wait_vm<2 * LC>();
    else if (s + 1 < end) wait_vm<LC>();
    else wait_vm<0>();
    asm volatile("" ::: "memory");
    const int step = (s % kRowsDepth) * STEP;
    v8i f[NT + MT];
    uint32_t sc[NT + MT];
#pragma unroll
    for (int t = 0; t < NT + MT; ++t) {
      const v4i lo = *reinterpret_cast<const v4i*>((t < NT + MT - 1 ? at[0] + t * 2048 : last[0]) + step);
      const v4i hi = *reinterpret_cast<const v4i*>((t < NT + MT - 1 ? at[1] + t * 2048 : last[1]) + step);
      f[t] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      sc[t] = scales[((s >> 2) & 1) * LS * 256 + (t * 16 + l16) * 4 + (s & 3)];
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read: the step's room can be filled again
    if (s + kRowsDepth < end) issue(s + kRowsDepth);
    if constexpr (sizeof(TY) == 2) {
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int b = 0; b < MT; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(f[a], f[NT + b], acc[a][b], kFmtE4m3, kFmtE4m3, 0,
                                                                       (int)sc[a], 0, (int)sc[NT + b]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v8bf x[NT + MT];
#pragma unroll
        for (int t = 0; t < NT + MT; ++t) x[t] = widen8(f[t][2 * j], f[t][2 * j + 1], scale_of(sc[t]));
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int b = 0; b < MT; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[a], x[NT + b], acc[a][b], 0, 0, 0);
      }
    }
  }
  // The waves' sums, in their order.  The second eight rows of a half tile (XD odd) are not stored.
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int b = 0; b < MT; ++b)
      *reinterpret_cast<v4f*>(ring + ((a * MT + b) * 64 + lane) * 16) = acc[a][b];
  __syncthreads();
  for (int t = wave; t < NT * MT; t += waves) {
    v4f sum = *reinterpret_cast<const v4f*>(lds + (t * 64 + lane) * 16);
    for (int w = 1; w < waves; ++w)
      sum += *reinterpret_cast<const v4f*>(lds + w * rows8_lds(XD, NT) + (t * 64 + lane) * 16);
    const int64_t m = t % MT * 16 + l16, n = n0 + t / MT * 16 + kg * 4;
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = sum[e] * g.alpha;
    if (m < g.M && n < g.N) store_four8(static_cast<TY*>(g.c) + m * g.ldc + n, v, g.N - n);
  }
}

// C = 0: an empty contraction, without touching the operands.
template <typename TY>
__global__ __launch_bounds__(256) void k_gemm8_zero(int64_t M, int64_t N, TY* __restrict__ c, int64_t ldc) {
  const int64_t runs = (N + 3) / 4, total = M * runs;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const float zero[4] = {};
    store_four8(c + i / runs * ldc + i % runs * 4, zero, N - i % runs * 4);
  }
}

// ============================================================== launches
size_t gemm8_workspace(int64_t M, int64_t N, int64_t K) {  // for C of either type
  const size_t a = plan8_bytes(gemm8_plan(M, N, round16(K), false), M, N);
  const size_t b = plan8_bytes(gemm8_plan(M, N, round16(K), true), M, N);
  return a > b ? a : b;
}

constexpr int64_t kMaxItems8 = 0xFFFFFFFFll;  // the work-items of a dispatch

// The grid of a product in tiles of T, its tiles from `whole` on in slices; 0: too many.
template <int T>
static int64_t place_tiles(Gemm8Args& g, int64_t whole) {
  const int64_t tm = cdiv(g.M, T), tn = cdiv(g.N, T), blocks = whole + (tm * tn - whole) * g.slices;
  if (blocks > kMaxItems8 / 256) return 0;
  g.tiles_m = (int)tm;
  g.tiles_n = (int)tn;
  g.whole = (int)whole;
  return blocks;
}

template <typename TY>
static int launch_sum(const Gemm8Args& g, hipStream_t st) {
  k_gemm8_sum<TY><<<dim3((unsigned)(g.tiles_m * g.tiles_n - g.whole) * 16), 256, 0, st>>>(g);
  return launch_status();
}

template <int T, typename TY, bool SLICED, bool WIDE>
static int launch_tiles(Gemm8Args g, int64_t whole, hipStream_t st) {
  const int64_t blocks = place_tiles<T>(g, whole);
  if (!blocks) return MX_ERR_SHAPE;
  const dim3 grid((unsigned)blocks);
  if constexpr (!WIDE) {
    k_gemm8_tile<T, TY, SLICED><<<grid, 256, 0, st>>>(g);
  } else {
    k_gemm8_wide<T, TY, SLICED><<<grid, 256, 0, st>>>(g);
  }
  if constexpr (SLICED) {
    if (const int s = launch_status()) return s;
    return launch_sum<TY>(g, st);
  }
  return launch_status();
}

template <int XD, int NT, typename TY>
static int launch_rows(const Gemm8Args& g, hipStream_t st) {
  // The waves of a workgroup share K: as many as leave room for two workgroups a compute unit, or for one
  // where there are no more workgroups than units or half the room takes one wave.  14336x4096, weights from HBM
  // and, second, the same ones each time: 47 rows float32 by one wave 25.3 and 24.5 us, by three 24.0 and 21.3,
  // bf16 18.0 and 16.2, and 19.9 and 15.9; 17 rows bf16 by two waves 14.5 and 12.7, by four 16.0 and 13.1.
  const int64_t tiles = cdiv(g.N, 16 * NT), steps = cdiv(g.K, 128), units = cdiv(steps, 4);
  constexpr int64_t kLds = 160 * 1024, kWave = rows8_lds(XD, NT);
  const int64_t room = tiles > device_cu_count() && kLds / 2 >= 2 * kWave ? kLds / 2 : kLds;
  const int64_t most = hmin(hmin(room / kWave, 8), units), per = cdiv(units, most);
  const Rows8Args r{g, (int)steps, (int)per * 4};
  const unsigned waves = (unsigned)cdiv(units, per);
  if (tiles > kMaxItems8 / (waves * 64)) return MX_ERR_SHAPE;
  k_gemm8_rows<XD, NT, TY><<<dim3((unsigned)tiles), waves * 64, waves * rows8_lds(XD, NT), st>>>(r);
  return launch_status();
}

template <typename TY>
static int gemm8_launch(Gemm8Args g, void* workspace, hipStream_t st) {
  if (g.K == 0) {
    const dim3 flat((unsigned)hmin(cdiv(g.M * cdiv(g.N, 4), 256), 4096));
    k_gemm8_zero<TY><<<flat, 256, 0, st>>>(g.M, g.N, static_cast<TY*>(g.c), g.ldc);
    return launch_status();
  }
  constexpr bool kWide = sizeof(TY) == 4;
  const Plan8 p = gemm8_plan(g.M, g.N, g.K, kWide);
  g.slices = p.slices;
  g.slice = p.slice;
  if (p.rows) {
    // 32 columns a wave halve the reads of A, where that leaves a workgroup for each compute unit (64 rows of
    // 8192x8192 20 us, by 16 columns 29)
    const bool two = g.N > 32 * 255;
#define MX_ROWS8(XD) (two ? launch_rows<XD, 2, TY>(g, st) : launch_rows<XD, 1, TY>(g, st))
    if (g.M <= 8) return MX_ROWS8(1);
    if (g.M <= 16) return MX_ROWS8(2);
    if (g.M <= 32) return MX_ROWS8(4);
    if (g.M <= 48) return MX_ROWS8(6);
    return MX_ROWS8(8);
#undef MX_ROWS8
  }
  if (p.big) return launch_tiles<256, TY, false, kWide>(g, 0, st);
  if (p.slices == 1) return launch_tiles<128, TY, false, kWide>(g, 0, st);
  g.part = static_cast<float*>(workspace);
  return launch_tiles<128, TY, true, kWide>(g, p.whole, st);
}

static Gemm8Args args8(const Product8& p) {
  return {p.a, p.sa, p.b, p.sb, p.lda, p.lsa, p.ldb, p.lsb, p.M, p.N, round16(p.K), p.c, p.ldc, nullptr, 0, 0, 0, 1, 0, p.alpha};
}

int gemm8_impl(const Product8& p, void* workspace, hipStream_t st) {
  if (p.M == 0 || p.N == 0) return MX_OK;
  return p.c_dtype == MX_F32 ? gemm8_launch<float>(args8(p), workspace, st) : gemm8_launch<uint16_t>(args8(p), workspace, st);
}

size_t gemm8_two_workspace(int64_t Mx, int64_t Nx, int64_t Kx, int64_t Mw, int64_t Nw, int64_t Kw) {
  return gemm8_workspace(Mx, Nx, Kx) + gemm8_workspace(Mw, Nw, Kw);  // whole tiles of 64 KB
}

template <typename TY>
static int launch_two(Gemm8Args x, const Plan8& px, Gemm8Args w, const Plan8& pw, hipStream_t st) {
  const int64_t bx = place_tiles<128>(x, px.whole), bw = place_tiles<128>(w, pw.whole);
  const bool front = pw.slice > px.slice;  // the longer workgroups first
  const int64_t blocks = cdiv(front ? bw : bx, 8) * 8 + (front ? bx : bw);
  if (!bx || !bw || blocks > kMaxItems8 / 256) return MX_ERR_SHAPE;
  k_gemm8_two<TY><<<dim3((unsigned)blocks), 256, 0, st>>>(x, (int)bx, w, (int)bw, front);
  int s = launch_status();
  if (s == MX_OK && px.slices > 1) s = launch_sum<TY>(x, st);
  if (s == MX_OK && pw.slices > 1) s = launch_sum<float>(w, st);
  return s;
}

// The plan of a product beside another: the tiles behind full rounds stay whole, the other's fill their round
// (both of 4093x5760x2880 float32 294 us, so 287).
static Plan8 beside(Plan8 p, const Product8& of) {
  if (p.slices > 1 && p.whole) p.whole = cdiv(of.M, 128) * cdiv(of.N, 128), p.slices = 1, p.slice = round16(of.K);
  return p;
}

int gemm8_two_impl(const Product8& x, const Product8& w, void* workspace, hipStream_t st) {
  const Plan8 px = beside(gemm8_plan(x.M, x.N, round16(x.K), x.c_dtype == MX_F32), x);
  const Plan8 pw = beside(gemm8_plan(w.M, w.N, round16(w.K), true), w);
  void* after = static_cast<uint8_t*>(workspace) + gemm8_workspace(x.M, x.N, x.K);
  if (px.rows || px.big || pw.rows || pw.big) {
    const int s = gemm8_impl(x, workspace, st);
    return s == MX_OK ? gemm8_impl(w, after, st) : s;
  }
  Gemm8Args gx = args8(x), gw = args8(w);
  gx.slices = px.slices, gx.slice = px.slice, gx.part = static_cast<float*>(workspace);
  gw.slices = pw.slices, gw.slice = pw.slice, gw.part = static_cast<float*>(after);
  return x.c_dtype == MX_F32 ? launch_two<float>(gx, px, gw, pw, st) : launch_two<uint16_t>(gx, px, gw, pw, st);
}

}  // namespace mx

using namespace mx;

static bool gemm8_shape(int64_t M, int64_t N, int64_t K) {
  return M >= 0 && N >= 0 && K >= 0 && M < kMax8 && N < kMax8 && K <= kMaxAxis8;
}

extern "C" size_t mx_gemm8_workspace_size(int64_t M, int64_t N, int64_t K) {
  return gemm8_shape(M, N, K) && M && N && K ? gemm8_workspace(M, N, K) : 0;
}

extern "C" int mx_gemm8(const uint8_t* a_codes, int64_t lda, const uint8_t* a_scales, int64_t a_scale_ld,
                        const uint8_t* b_codes, int64_t ldb, const uint8_t* b_scales, int64_t b_scale_ld,
                        int64_t M, int64_t N, int64_t K, float alpha, void* c, int c_dtype, int64_t ldc,
                        void* workspace, size_t workspace_bytes, void* stream) {
  MX_REQUIRE(float_type(c_dtype), MX_ERR_ENUM);
  MX_REQUIRE(gemm8_shape(M, N, K) && ldc >= N, MX_ERR_SHAPE);
  MX_REQUIRE(matrix8(K, lda, a_scale_ld) && matrix8(K, ldb, b_scale_ld), MX_ERR_SHAPE);
  if (M == 0 || N == 0) return MX_OK;
  MX_REQUIRE(c && (K == 0 || (a_codes && a_scales && b_codes && b_scales)), MX_ERR_NULL);
  MX_REQUIRE(aligned16(c) && aligned16(a_codes) && aligned16(a_scales) && aligned16(b_codes) &&
                 aligned16(b_scales), MX_ERR_ALIGN);
  const size_t need = mx_gemm8_workspace_size(M, N, K);
  if (need) {
    MX_REQUIRE(workspace && workspace_bytes >= need, MX_ERR_WORKSPACE);
    MX_REQUIRE(aligned16(workspace), MX_ERR_ALIGN);
  }
  return gemm8_impl({a_codes, a_scales, b_codes, b_scales, lda, a_scale_ld, ldb, b_scale_ld, M, N, K, alpha, c, c_dtype, ldc},
                    workspace, as_stream(stream));
}
