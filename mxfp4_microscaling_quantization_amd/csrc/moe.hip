// Routing of a mixture-of-experts layer around the grouped products: token
// slots sorted by expert, rows copied or quantized into expert order, expert
// rows added up per token with the router's weights, and the gradients.
//
// A slot s = token * top_k + j is one of a token's top_k choices.  With pos[s]
// the sorted row of slot s (-1: the slot takes part in nothing),
//   dispatch          out[pos[t,j]] = w[t,j] x[t]          (w = 1 without weights)
//   combine           y[t] = sum_j w[t,j] z[pos[t,j]]
//   combine gradient  dz[pos[t,j]] = w[t,j] dy[t],  dw[t,j] = <dy[t], z[pos[t,j]]>
// Dispatch and combine are each other's transposes, so combine without weights
// is the gradient of a dispatch.  All of them move rows once and compute little:
// HBM bandwidth bounds them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device.h"
#include "mx_host.h"

namespace mx {

// ============================================================== plan
// Stable counting sort of the slots by expert; slots without an expert form one
// more bin behind the last expert, whose rows get src = -1.  Chunks of
// consecutive slots are counted (k_plan_count), then every chunk places its
// slots (k_plan_place): rows of bin e start at the total of the bins before it,
// a chunk's rows of the bin at the sum of the chunks before it, and a slot's
// place among its own wave's slots of the same bin comes from ballots over the
// bits of the bin number.  Sums of whole numbers: the result does not depend on
// the order in which atomics arrive.
// Latency bound: 16384 x 4 slots of 32 experts (1 MB in all) take 2.4 us to count
// and 4.7 us to place in 64 chunks, a chunk alone (24 x 4 slots) 2.8 us without the
// count's launch.  Chunks of one slot a thread keep the ranks a single pass.
constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kPlanMaxChunks = 256;
constexpr int kPlanBins = MX_MAX_GROUPS + 1;

struct PlanShape {
  int64_t slots, chunk;
  int chunks, experts;
};

template <typename ID>
__device__ __forceinline__ int plan_bin(const ID* ids, int64_t s, int experts) {
  const ID e = ids[s];
  return e >= 0 && e < (ID)experts ? (int)e : experts;
}

template <typename ID>
__global__ __launch_bounds__(kPlanThreads) void k_plan_count(const ID* __restrict__ ids,
                                                             const PlanShape p,
                                                             int32_t* __restrict__ counts) {
  __shared__ int32_t s_cnt[kPlanBins];
  const int bins = p.experts + 1;
  for (int e = threadIdx.x; e < bins; e += kPlanThreads) s_cnt[e] = 0;
  __syncthreads();
  const int64_t end = min<int64_t>(p.slots, (blockIdx.x + 1) * p.chunk);
  for (int64_t s = blockIdx.x * p.chunk + threadIdx.x; s < end; s += kPlanThreads)
    atomicAdd(&s_cnt[plan_bin(ids, s, p.experts)], 1);
  __syncthreads();
  for (int e = threadIdx.x; e < bins; e += kPlanThreads)
    counts[(int64_t)blockIdx.x * bins + e] = s_cnt[e];
}

template <typename ID>
__global__ __launch_bounds__(kPlanThreads) void k_plan_place(const ID* __restrict__ ids,
                                                             const PlanShape p,
                                                             const int32_t* __restrict__ counts,
                                                             int64_t* __restrict__ offs,
                                                             int32_t* __restrict__ src,
                                                             int32_t* __restrict__ pos) {
  __shared__ int32_t s_total[kPlanBins];            // slots of each bin
  __shared__ int32_t s_base[kPlanBins];             // next row of each bin in this chunk
  __shared__ int32_t s_wave[kPlanWaves][kPlanBins]; // slots of a bin in each wave's 64
  const int bins = p.experts + 1;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (int e = tid; e < bins; e += kPlanThreads) s_total[e] = s_base[e] = 0;
  __syncthreads();
  const int64_t begin = (int64_t)blockIdx.x * p.chunk;
  const int64_t end = min<int64_t>(p.slots, begin + p.chunk);
  if (p.chunks == 1) {
    for (int64_t s = tid; s < end; s += kPlanThreads)
      atomicAdd(&s_total[plan_bin(ids, s, p.experts)], 1);
  } else {
    for (int i = tid; i < p.chunks * bins; i += kPlanThreads) {
      const int c = i / bins, e = i - c * bins;
      const int32_t n = counts[i];
      atomicAdd(&s_total[e], n);
      if (c < (int)blockIdx.x) atomicAdd(&s_base[e], n);
    }
  }
  __syncthreads();
  if (wave == 0) {  // rows of the bins before each: lanes hold 64 bins at a time
    int32_t before = 0;
    for (int e0 = 0; e0 < bins; e0 += 64) {
      const int e = e0 + lane;
      const int32_t n = e < bins ? s_total[e] : 0;
      int32_t upto = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t up = __shfl_up(upto, d);
        upto += lane >= d ? up : 0;
      }
      if (e < bins) {
        if (blockIdx.x == 0) offs[e] = before + upto - n;
        s_base[e] += before + upto - n;
      }
      before += __shfl(upto, 63);
    }
  }
  for (int64_t s0 = begin; s0 < end; s0 += kPlanThreads) {
    for (int i = tid; i < kPlanWaves * kPlanBins; i += kPlanThreads) (&s_wave[0][0])[i] = 0;
    __syncthreads();
    const int64_t s = s0 + tid;
    const bool in = s < end;
    const int bin = in ? plan_bin(ids, s, p.experts) : 0;
    uint64_t same = __ballot(in);
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t set = __ballot((bin >> b) & 1);
      same &= ((bin >> b) & 1) ? set : ~set;
    }
    const int before = __popcll(same & ((1ull << lane) - 1));
    if (in && before == 0) s_wave[wave][bin] = __popcll(same);
    __syncthreads();
    for (int e = tid; e < bins; e += kPlanThreads) {
      int32_t n[kPlanWaves], row = s_base[e];
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) n[w] = s_wave[w][e];
#pragma unroll
      for (int w = 0; w < kPlanWaves; ++w) {
        s_wave[w][e] = row;
        row += n[w];
      }
      s_base[e] = row;
    }
    __syncthreads();
    if (in) {
      const int32_t row = s_wave[wave][bin] + before;
      const bool real = bin < p.experts;
      pos[s] = real ? row : -1;
      src[row] = real ? (int32_t)s : -1;
    }
    __syncthreads();
  }
}

static PlanShape plan_shape(int64_t slots, int64_t experts) {
  PlanShape p;
  p.slots = slots;
  p.experts = (int)experts;
  const int64_t per = cdiv(cdiv(slots, kPlanMaxChunks), kPlanThreads);
  p.chunk = (per > 1 ? per : 1) * kPlanThreads;
  p.chunks = (int)cdiv(slots, p.chunk);
  return p;
}

// ============================================================== rows
// A run is 8 consecutive values of a row.  Rows start at any multiple of their type's
// size: the vector accesses carry that alignment, which the hardware takes.  Where the
// width is no multiple of 8 the last run starts early and covers values of the run before
// it once more (they are stored twice alike, and summed once).  One value a thread took
// 206 us where such runs take 165 (combine of 2885 columns, float32 to bf16), and a branch
// for a short last run cost whole ones too (a copy of 2880 bf16 columns 146 us, not 93).
// NARROW: rows of fewer than 8 values, one run of n of them.
template <typename T, bool NARROW>
__device__ __forceinline__ void load_run(const T* p, int n, float v[8]) {
  if constexpr (!NARROW) {
    T raw[8];
    __builtin_memcpy(raw, p, sizeof(raw));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (sizeof(T) == 2) v[i] = bf16_lo(raw[i]);
      else v[i] = raw[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (i < n) {
        if constexpr (sizeof(T) == 2) v[i] = bf16_lo(p[i]);
        else v[i] = p[i];
      }
    }
  }
}

template <typename T, bool NARROW>
__device__ __forceinline__ void store_run(T* p, int n, const float v[8]) {
  T raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 2) raw[i] = (T)f32_to_bf16_rne(v[i]);
    else raw[i] = v[i];
  }
  if constexpr (!NARROW) {
    __builtin_memcpy(p, raw, sizeof(raw));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = raw[i];
  }
}

// Position of a thread's run in the flat order (token, run of the row): the
// workgroup's first index is divided once, the threads' by a 32-bit division.
struct RowRun {
  int64_t token;
  int run;
};
__device__ __forceinline__ RowRun row_run(int64_t first, int at, int runs) {
  const int64_t t0 = first / runs;
  const uint32_t r = (uint32_t)(first - t0 * runs) + (uint32_t)at;
  const uint32_t q = r / (uint32_t)runs;
  return {t0 + q, (int)(r - q * (uint32_t)runs)};
}

// ============================================================== dispatch
// One read of a token's run, top_k writes: bound by the writes.  The copy moves 16-byte
// runs of elements whatever they hold, so NaN patterns stay as they are.  16384 x 2880
// bf16 to 4 rows each: 93 us, 5.1 TB/s; the weighted form 113 us of 2885 columns.
template <typename T, bool NARROW>
__global__ __launch_bounds__(256) void k_dispatch_copy(const T* __restrict__ x, int64_t ldx,
                                                       const int32_t* __restrict__ pos,
                                                       int64_t tokens, int top_k, int64_t rows,
                                                       int cols, int runs, T* __restrict__ out,
                                                       int64_t ldo) {
  constexpr int E = 16 / sizeof(T);
  const int64_t total = tokens * runs;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowRun r = row_run(first, threadIdx.x, runs);
    const int n = min(E, cols), col = min(r.run * E, cols - n);
    const T* p = x + r.token * ldx + col;
    T v[E];
    if constexpr (!NARROW) {
      __builtin_memcpy(v, p, 16);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < n) v[i] = p[i];
    }
    for (int j = 0; j < top_k; ++j) {
      const int32_t to = pos[r.token * top_k + j];
      if (to < 0 || to >= rows) continue;
      T* o = out + to * ldo + col;
      if constexpr (!NARROW) {
        __builtin_memcpy(o, v, 16);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (i < n) o[i] = v[i];
      }
    }
  }
}

template <typename T, bool NARROW>
__global__ __launch_bounds__(256) void k_dispatch_scaled(const T* __restrict__ x, int64_t ldx,
                                                         const int32_t* __restrict__ pos,
                                                         int64_t tokens, int top_k, int64_t rows,
                                                         int cols, int runs,
                                                         const float* __restrict__ weights,
                                                         T* __restrict__ out, int64_t ldo) {
  const int64_t total = tokens * runs;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowRun r = row_run(first, threadIdx.x, runs);
    const int n = min(8, cols), col = min(r.run * 8, cols - n);
    float v[8];
    load_run<T, NARROW>(x + r.token * ldx + col, n, v);
    for (int j = 0; j < top_k; ++j) {
      const int32_t to = pos[r.token * top_k + j];
      if (to < 0 || to >= rows) continue;
      const float w = weights[r.token * top_k + j];
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = w * v[i];
      store_run<T, NARROW>(out + to * ldo + col, n, u);
    }
  }
}

// Q_D of a token's 1x32 blocks (a quad of lanes per block, 8 values a lane) once,
// its codes and scale byte written to the token's top_k rows: the values are the
// same in each, so one conversion serves them all.  Every lane of a quad gets the
// block's 16 bytes of codes and stores them to one of the rows, four rows at a time
// (4 bytes a lane to every row took 51 us for 16384 x 2880 to 4 rows each, this 44.7 us,
// 4.4 TB/s; two or four runs of x a thread 48 us).
template <typename T>
__global__ __launch_bounds__(256) void k_dispatch_quant(const T* __restrict__ x, int64_t ldx,
                                                        const int32_t* __restrict__ pos,
                                                        int64_t tokens, int top_k, int64_t rows,
                                                        int runs, uint32_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales,
                                                        int64_t scale_ld) {
  const int64_t total = tokens * runs;  // runs of 8: a multiple of 4 per row
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;  // whole quads: total is a multiple of 4
    const RowRun r = row_run(first, threadIdx.x, runs);
    float v[8];
    load_run<T, false>(x + r.token * ldx + (int64_t)r.run * 8, 8, v);
    const uint32_t byte = scale_byte_of(quad_max_u32(amax_bits<8>(v)));
    uint32_t w = 0;
    if (byte != 255u) {
      const float sc = scale_of(byte);
#pragma unroll
      for (int i = 0; i < 4; ++i) w |= (cvt_rne_pair(v[2 * i], v[2 * i + 1], sc) & 0xFFu) << (8 * i);
    }
    const uint4 block = make_uint4(dpp_u32<0x00>(w), dpp_u32<0x55>(w), dpp_u32<0xAA>(w), dpp_u32<0xFF>(w));
    for (int j = r.run & 3; j < top_k; j += 4) {
      const int32_t to = pos[r.token * top_k + j];
      if (to < 0 || to >= rows) continue;
      *reinterpret_cast<uint4*>(codes + (int64_t)to * runs + (r.run & ~3)) = block;
      scales[(int64_t)to * scale_ld + (r.run >> 2)] = (uint8_t)byte;
    }
  }
}

// ============================================================== combine
// A token's slots are taken four at a time, so that four rows of z are on their way
// together.  A slot left out, or missing where top_k is no multiple of four, loads row 0
// and adds nothing.  65536 rows of 2880 float32 as top_k = 1, 2, 3, 4, 6 and 8 rows of bf16
// tokens: 264, 187, 171, 162, 154 and 149 us (4.3, 5.1, 5.2, 5.2, 5.3 and 5.4 TB/s), their
// gradient 334, 266, 245, 240, 238 and 236 us (4.5, 5.0, 5.1, 5.1, 5.0 and 5.0); top_k = 4
// with 40 % padding tokens 108 and 162 us (5.1 and 4.6).
constexpr int kSlots = 4;

struct Slots {
  int32_t row[kSlots];
  float w[kSlots];
  bool real[kSlots];
};
__device__ __forceinline__ Slots load_slots(const int32_t* __restrict__ pos,
                                            const float* __restrict__ weights, int64_t first,
                                            int left, int64_t rows) {
  Slots s;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int64_t at = first + min(i, left - 1);
    s.row[i] = pos[at];
    s.w[i] = weights ? weights[at] : 1.0f;
  }
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    s.real[i] = i < left && s.row[i] >= 0 && s.row[i] < rows;
    s.row[i] = s.real[i] ? s.row[i] : 0;
  }
  return s;
}

// Sums in float32 in slot order, each product rounded first.  HBM bound: 16384 x 4 rows of
// 2880 float32 into bf16 161 us, 5.3 TB/s (164 us one row at a time).
template <typename TZ, typename TY, bool NARROW>
__global__ __launch_bounds__(256) void k_combine(const TZ* __restrict__ z, int64_t ldz, int64_t rows,
                                                 const int32_t* __restrict__ pos,
                                                 const float* __restrict__ weights, int64_t tokens,
                                                 int top_k, int cols, int runs,
                                                 TY* __restrict__ y, int64_t ldy) {
  const int64_t total = tokens * runs;
  for (int64_t first = (int64_t)blockIdx.x * 256; first < total; first += (int64_t)gridDim.x * 256) {
    if (first + threadIdx.x >= total) continue;
    const RowRun r = row_run(first, threadIdx.x, runs);
    const int n = min(8, cols), col = min(r.run * 8, cols - n);
    float acc[8] = {};
    for (int j = 0; j < top_k && rows; j += kSlots) {
      const Slots s = load_slots(pos, weights, r.token * top_k + j, top_k - j, rows);
      float v[kSlots][8];
#pragma unroll
      for (int k = 0; k < kSlots; ++k) load_run<TZ, NARROW>(z + s.row[k] * ldz + col, n, v[k]);
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = s.real[k] ? acc[i] + s.w[k] * v[k][i] : acc[i];
    }
    store_run<TY, NARROW>(y + r.token * ldy + col, n, acc);
  }
}

// One workgroup per token: dz rows as a weighted dispatch, and each slot's inner
// product <dy, z> as per-thread sums, then a fixed tree over lanes and waves.  HBM bound:
// 240 us for 16384 x 4 rows of 2880 (bf16 dy and dz, float32 z), 5.1 TB/s.
template <typename TY, typename TZ, bool NARROW>
__global__ __launch_bounds__(256) void k_combine_bwd(
    const TY* __restrict__ dy, int64_t lddy, const TZ* __restrict__ z, int64_t ldz, int64_t rows,
    const int32_t* __restrict__ pos, const float* __restrict__ weights, int64_t tokens, int top_k,
    int cols, int runs, TY* __restrict__ dz, int64_t lddz, float* __restrict__ dw) {
  __shared__ float s_part[2][4][kSlots];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  int turn = 0;  // the two halves of s_part alternate: one barrier a turn
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j = 0; j < top_k; j += kSlots, turn ^= 1) {
      const Slots s = load_slots(pos, weights, t * top_k + j, top_k - j, rows);
      float part[kSlots] = {};
      if (rows) {
        for (int r = threadIdx.x; r < runs; r += blockDim.x) {
          const int n = min(8, cols), col = min(r * 8, cols - n);
          const int again = r * 8 - col;  // values that the run before has
          float g[8], v[kSlots][8], u[8];
          load_run<TY, NARROW>(dy + t * lddy + col, n, g);
#pragma unroll
          for (int k = 0; k < kSlots; ++k) load_run<TZ, NARROW>(z + s.row[k] * ldz + col, n, v[k]);
#pragma unroll
          for (int k = 0; k < kSlots; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              part[k] = i < again ? part[k] : part[k] + g[i] * v[k][i];
              u[i] = s.w[k] * g[i];
            }
            if (s.real[k]) store_run<TY, NARROW>(dz + s.row[k] * lddz + col, n, u);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
#pragma unroll
        for (int d = 32; d; d >>= 1) part[k] += __shfl_xor(part[k], d);
        if (lane == 0) s_part[turn][wave][k] = part[k];
      }
      __syncthreads();
      if (threadIdx.x < kSlots && j + (int)threadIdx.x < top_k) {
        float sum = 0.0f;
        for (int w = 0; w < waves; ++w) sum += s_part[turn][w][threadIdx.x];
        bool real = false;
#pragma unroll
        for (int k = 0; k < kSlots; ++k) real = (int)threadIdx.x == k ? s.real[k] : real;
        dw[t * top_k + j + threadIdx.x] = real ? sum : 0.0f;
      }
    }
  }
}

// ============================================================== launches
static unsigned row_grid(int64_t work_items) {
  return (unsigned)hmin(cdiv(work_items, 256), (int64_t)device_cu_count() * 64);
}

static bool is_float_type(int t) { return t == MX_F32 || t == MX_BF16; }
constexpr int64_t kMax31 = (int64_t)1 << 31;

// Sizes every row call shares: tokens * top_k and the output rows fit 32-bit positions.
static bool routed_shape(int64_t tokens, int64_t top_k, int64_t cols, int64_t rows) {
  return tokens >= 0 && top_k >= 1 && top_k < kMax31 && cols >= 0 && cols < kMax31 && rows >= 0 &&
         rows < kMax31 && tokens <= (kMax31 - 1) / top_k;
}

}  // namespace mx

using namespace mx;

extern "C" size_t mx_moe_plan_workspace_size(int64_t tokens, int64_t top_k, int64_t experts) {
  if (!routed_shape(tokens, top_k, 0, 0) || experts < 1 || experts > MX_MAX_GROUPS) return 0;
  const PlanShape p = plan_shape(tokens * top_k, experts);
  return p.chunks > 1 ? (size_t)p.chunks * (experts + 1) * sizeof(int32_t) : 0;
}

extern "C" int mx_moe_plan(const void* ids, int id_type, int64_t tokens, int64_t top_k,
                           int64_t experts, int64_t* offs, int32_t* src, int32_t* pos,
                           void* workspace, size_t workspace_bytes, void* stream) {
  MX_REQUIRE(routed_shape(tokens, top_k, 0, 0) && experts >= 1 && experts <= MX_MAX_GROUPS,
             MX_ERR_SHAPE);
  MX_REQUIRE(id_type == MX_I32 || id_type == MX_I64, MX_ERR_ENUM);
  MX_REQUIRE(offs, MX_ERR_NULL);
  const int64_t slots = tokens * top_k;
  if (slots) MX_REQUIRE(ids && src && pos, MX_ERR_NULL);
  MX_REQUIRE(aligned16(ids) && aligned16(offs) && aligned16(src) && aligned16(pos), MX_ERR_ALIGN);
  const PlanShape p = plan_shape(slots, experts);
  const size_t need = mx_moe_plan_workspace_size(tokens, top_k, experts);
  if (need) {
    MX_REQUIRE(workspace && workspace_bytes >= need, MX_ERR_WORKSPACE);
    MX_REQUIRE(aligned16(workspace), MX_ERR_ALIGN);
  }
  const hipStream_t st = as_stream(stream);
  int32_t* counts = static_cast<int32_t*>(workspace);
  const unsigned grid = p.chunks ? p.chunks : 1;  // no slots: one workgroup writes offs = 0
  if (id_type == MX_I32) {
    const int32_t* e = static_cast<const int32_t*>(ids);
    if (need) k_plan_count<<<grid, kPlanThreads, 0, st>>>(e, p, counts);
    k_plan_place<<<grid, kPlanThreads, 0, st>>>(e, p, counts, offs, src, pos);
  } else {
    const int64_t* e = static_cast<const int64_t*>(ids);
    if (need) k_plan_count<<<grid, kPlanThreads, 0, st>>>(e, p, counts);
    k_plan_place<<<grid, kPlanThreads, 0, st>>>(e, p, counts, offs, src, pos);
  }
  return launch_status();
}

extern "C" int mx_moe_dispatch(const void* x, int dtype, int64_t ldx, const int32_t* pos,
                               const float* weights, int64_t tokens, int64_t top_k, int64_t rows,
                               int64_t cols, void* out, int64_t ldo, void* stream) {
  MX_REQUIRE(is_float_type(dtype), MX_ERR_ENUM);
  MX_REQUIRE(routed_shape(tokens, top_k, cols, rows) && ldx >= cols && ldo >= cols, MX_ERR_SHAPE);
  if (tokens == 0 || cols == 0 || rows == 0) return MX_OK;
  MX_REQUIRE(x && pos && out, MX_ERR_NULL);
  MX_REQUIRE(aligned16(x) && aligned16(pos) && aligned16(out) && aligned16(weights), MX_ERR_ALIGN);
  const int run = weights || dtype == MX_BF16 ? 8 : 4;
  const int runs = (int)cdiv(cols, run);
  const dim3 grid(row_grid(tokens * runs));
  const hipStream_t st = as_stream(stream);
#define MX_DISPATCH_WIDTH(T, NARROW)                                                          \
  do {                                                                                       \
    const T* xt = static_cast<const T*>(x);                                                  \
    T* o = static_cast<T*>(out);                                                             \
    if (weights)                                                                             \
      k_dispatch_scaled<T, NARROW><<<grid, 256, 0, st>>>(xt, ldx, pos, tokens, (int)top_k, rows, \
                                                       (int)cols, runs, weights, o, ldo);    \
    else                                                                                     \
      k_dispatch_copy<T, NARROW><<<grid, 256, 0, st>>>(xt, ldx, pos, tokens, (int)top_k, rows, \
                                                     (int)cols, runs, o, ldo);               \
  } while (0)
#define MX_DISPATCH(T)                            \
  do {                                             \
    if (cols < run) MX_DISPATCH_WIDTH(T, true);    \
    else MX_DISPATCH_WIDTH(T, false);              \
  } while (0)
  if (dtype == MX_F32) MX_DISPATCH(float);
  else MX_DISPATCH(uint16_t);
#undef MX_DISPATCH
#undef MX_DISPATCH_WIDTH
  return launch_status();
}

extern "C" int mx_moe_dispatch_quantize(const void* x, int dtype, int64_t ldx, const int32_t* pos,
                                        int64_t tokens, int64_t top_k, int64_t rows, int64_t cols,
                                        uint8_t* codes, uint8_t* scales, int64_t scale_ld,
                                        void* stream) {
  MX_REQUIRE(is_float_type(dtype), MX_ERR_ENUM);
  MX_REQUIRE(routed_shape(tokens, top_k, cols, rows) && cols % 32 == 0 && ldx >= cols &&
                 scale_ld >= cols / 32, MX_ERR_SHAPE);
  if (tokens == 0 || cols == 0 || rows == 0) return MX_OK;
  MX_REQUIRE(x && pos && codes && scales, MX_ERR_NULL);
  MX_REQUIRE(aligned16(x) && aligned16(pos) && aligned16(codes) && aligned16(scales), MX_ERR_ALIGN);
  const int runs = (int)(cols / 8);
  const dim3 grid(row_grid(tokens * runs));
  const hipStream_t st = as_stream(stream);
#define MX_DISPATCHQ(T)                                                                        \
  k_dispatch_quant<T><<<grid, 256, 0, st>>>(static_cast<const T*>(x), ldx, pos, tokens,         \
                                            (int)top_k, rows, runs,                             \
                                            reinterpret_cast<uint32_t*>(codes), scales, scale_ld)
  if (dtype == MX_F32) MX_DISPATCHQ(float);
  else MX_DISPATCHQ(uint16_t);
#undef MX_DISPATCHQ
  return launch_status();
}

extern "C" int mx_moe_combine(const void* z, int z_dtype, int64_t ldz, int64_t rows,
                              const int32_t* pos, const float* weights, int64_t tokens,
                              int64_t top_k, int64_t cols, void* y, int y_dtype, int64_t ldy,
                              void* stream) {
  MX_REQUIRE(is_float_type(z_dtype) && is_float_type(y_dtype), MX_ERR_ENUM);
  MX_REQUIRE(routed_shape(tokens, top_k, cols, rows) && ldz >= cols && ldy >= cols, MX_ERR_SHAPE);
  if (tokens == 0 || cols == 0) return MX_OK;
  MX_REQUIRE(pos && y, MX_ERR_NULL);
  if (rows) MX_REQUIRE(z, MX_ERR_NULL);  // no rows: y = 0, z is not read
  MX_REQUIRE(aligned16(z) && aligned16(pos) && aligned16(weights) && aligned16(y), MX_ERR_ALIGN);
  const int runs = (int)cdiv(cols, 8);
  const dim3 grid(row_grid(tokens * runs));
  const hipStream_t st = as_stream(stream);
#define MX_COMBINE_WIDTH(TZ, TY, NARROW)                                                      \
  k_combine<TZ, TY, NARROW><<<grid, 256, 0, st>>>(static_cast<const TZ*>(z), ldz, rows, pos, \
                                                weights, tokens, (int)top_k, (int)cols, runs, \
                                                static_cast<TY*>(y), ldy)
#define MX_COMBINE(TZ, TY)                            \
  do {                                                 \
    if (cols < 8) MX_COMBINE_WIDTH(TZ, TY, true);      \
    else MX_COMBINE_WIDTH(TZ, TY, false);              \
  } while (0)
  if (z_dtype == MX_F32) {
    if (y_dtype == MX_F32) MX_COMBINE(float, float);
    else MX_COMBINE(float, uint16_t);
  } else {
    if (y_dtype == MX_F32) MX_COMBINE(uint16_t, float);
    else MX_COMBINE(uint16_t, uint16_t);
  }
#undef MX_COMBINE
#undef MX_COMBINE_WIDTH
  return launch_status();
}

extern "C" int mx_moe_combine_bwd(const void* dy, int dy_dtype, int64_t lddy, const void* z,
                                  int z_dtype, int64_t ldz, int64_t rows, const int32_t* pos,
                                  const float* weights, int64_t tokens, int64_t top_k,
                                  int64_t cols, void* dz, int64_t lddz, float* dweights,
                                  void* stream) {
  MX_REQUIRE(is_float_type(dy_dtype) && is_float_type(z_dtype), MX_ERR_ENUM);
  MX_REQUIRE(routed_shape(tokens, top_k, cols, rows) && lddy >= cols && ldz >= cols && lddz >= cols,
             MX_ERR_SHAPE);
  if (tokens == 0) return MX_OK;
  MX_REQUIRE(pos && dweights, MX_ERR_NULL);
  if (rows && cols) MX_REQUIRE(dy && z && dz, MX_ERR_NULL);
  MX_REQUIRE(aligned16(dy) && aligned16(z) && aligned16(pos) && aligned16(weights) &&
                 aligned16(dz) && aligned16(dweights), MX_ERR_ALIGN);
  const int runs = (int)cdiv(cols, 8);
  const dim3 grid((unsigned)hmin(tokens, (int64_t)device_cu_count() * 64));
  // the workgroup whose last pass over the row leaves the fewest threads idle
  int threads = 256;
  for (int n = 192; n >= 64; n -= 64)
    if (cdiv(runs, n) * n < cdiv(runs, threads) * threads) threads = n;
  const hipStream_t st = as_stream(stream);
#define MX_COMBINE_BWD_WIDTH(TY, TZ, NARROW)                                                   \
  k_combine_bwd<TY, TZ, NARROW><<<grid, threads, 0, st>>>(                                    \
      static_cast<const TY*>(dy), lddy, static_cast<const TZ*>(z), ldz, rows, pos, weights,  \
      tokens, (int)top_k, (int)cols, runs, static_cast<TY*>(dz), lddz, dweights)
#define MX_COMBINE_BWD(TY, TZ)                            \
  do {                                                     \
    if (cols < 8) MX_COMBINE_BWD_WIDTH(TY, TZ, true);      \
    else MX_COMBINE_BWD_WIDTH(TY, TZ, false);              \
  } while (0)
  if (dy_dtype == MX_F32) {
    if (z_dtype == MX_F32) MX_COMBINE_BWD(float, float);
    else MX_COMBINE_BWD(float, uint16_t);
  } else {
    if (z_dtype == MX_F32) MX_COMBINE_BWD(uint16_t, float);
    else MX_COMBINE_BWD(uint16_t, uint16_t);
  }
#undef MX_COMBINE_BWD
#undef MX_COMBINE_BWD_WIDTH
  return launch_status();
}
