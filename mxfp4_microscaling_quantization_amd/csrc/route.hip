// Router of a mixture-of-experts layer: each token's softmax over the experts, its top_k choices
// and their weights, the slots each expert gets, the balance loss, and the gradients.
//
// With s the softmax of a token's logits, n the tokens that take part, c_e the slots of expert e:
//   p_j = s_{id_j}, or s_{id_j} / sum_i s_{id_i}
//   loss = E sum_e f_e P_e,  f_e = c_e / (n k),  P_e = 1/n sum_t s_te
// The choices and counts are constants of the gradient:
//   dlogits_e = s_e (G_e - <s, G>) + [e = id_j] p_j (dp_j - C)      renormalized
//   dlogits_e = s_e (G_e - <s, G> - C) + [e = id_j] p_j dp_j        otherwise
// with G_e = dloss E f_e / n and C = sum_j p_j dp_j.
//
// 16 lanes hold a token, expert e in lane e % 16, so that sums and maxima stay within a row of
// lanes; a wave takes 4 tokens.  There is little to read (2 MB for 16384 tokens of 32 experts, 0.5 us):
// the launches and the chain of top_k selections bound it.  16384 tokens of 32 experts, four each, float32: 5.6 us,
// the sums 3.3, backward 4.6; 5000 of 128, eight each, bf16: 7.6, 5.4 and 6.9; one launch of 3 to 4 us for a
// batch of decoding.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mx_device8.h"
#include "mx_host8.h"

namespace mx {

constexpr int kRouteMaxK = 16;       // slot j's choice is kept by lane j
constexpr int kRouteGroups = 256;    // workgroups whose sums the second launch adds up
// Up to so many tokens one workgroup does all: 64 tokens of 32 experts, four each, 5.0 us and in two launches 6.8,
// 128 7.3 and 6.9; 64 of 128 experts, eight each, 9.6 and 11.4, 256 29 and 12.
constexpr int kRouteAlone = 64;
// Threads of a workgroup: as many as its tokens, or those of 256 workgroups, have lanes for, 512 or 1024 (24 tokens of
// 128 experts 6.7 and 9.4 us; 8192 12.8 and 15.2, 65536 42 and 37).
static int route_threads(int64_t tokens) {
  return tokens <= 32 || (tokens > kRouteAlone && tokens <= 32 * kRouteGroups) ? 512 : 1024;
}
static int64_t route_groups(int64_t tokens) { return hmin(cdiv(tokens, route_threads(tokens) / 16), kRouteGroups); }

// Sums and extremes over the 16 lanes of a row, the same bits in each: neighbours, pairs, halves
// and the row are mirrored onto each other.
template <typename F>
__device__ __forceinline__ float row16_f32(float v, F f) {
  v = f(v, dpp_f32<kQuadSwap1>(v));
  v = f(v, dpp_f32<kQuadSwap2>(v));
  v = f(v, dpp_f32<0x141>(v));  // lane i of 8 reads lane 7 - i
  v = f(v, dpp_f32<0x140>(v));  // lane i of 16 reads lane 15 - i
  return v;
}
__device__ __forceinline__ float row16_sum(float v) {
  return row16_f32(v, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float row16_max(float v) {
  return row16_f32(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ __forceinline__ uint32_t row16_min_u32(uint32_t v) {
  v = min(v, dpp_u32<kQuadSwap1>(v));
  v = min(v, dpp_u32<kQuadSwap2>(v));
  v = min(v, dpp_u32<0x141>(v));
  v = min(v, dpp_u32<0x140>(v));
  return v;
}

__device__ __forceinline__ float route_value(const float* p) { return *p; }
__device__ __forceinline__ float route_value(const uint16_t* p) { return bf16_lo(*p); }
__device__ __forceinline__ void route_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void route_store(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_rne(v); }

constexpr float kClosed = -__builtin_huge_valf();  // the logit of an expert that takes no token

// A token's logits in its lanes, the largest of them (NaN passed over), and whether it takes part:
// a logit other than -Inf.  A NaN or +Inf among them makes its softmax NaN.
template <int EPL>
struct Token {
  float v[EPL], top;
  bool in;
  template <typename T>
  __device__ __forceinline__ void load(const T* __restrict__ row, int lane, int experts, bool real) {
    float m = kClosed;
    uint32_t some = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 16 + lane;
      v[i] = real && e < experts ? route_value(row + e) : kClosed;
      m = fmaxf(m, v[i]);
      some |= !(v[i] == kClosed);
    }
    top = row16_max(m);
    in = row16_max_u32(some) != 0;
  }
};

struct RouteArgs {
  const void* logits;
  int64_t ld, tokens;
  const uint8_t* mask;
  int experts, top_k, renormalize;
};

// The workgroup's sums of s and of slots, from its token groups' registers: partial [E] floats and
// [E + 1] counts (the last: tokens that take part).
template <typename T, int EPL, int THREADS>
__device__ __forceinline__ void route_tokens(const RouteArgs& a, int32_t* __restrict__ ids, float* __restrict__ p,
                                             float (&s_sum)[THREADS / 64][128], int32_t (&s_cnt)[129]) {
  const int tid = threadIdx.x, lane = tid & 15, group = tid >> 4, wave = tid >> 6;
  for (int e = tid; e <= a.experts; e += THREADS) s_cnt[e] = 0;
  __syncthreads();
  float sum[EPL] = {};
  constexpr int kPer = THREADS / 16;
  const int64_t stride = (int64_t)gridDim.x * kPer;
  for (int64_t t0 = (int64_t)blockIdx.x * kPer; t0 < a.tokens; t0 += stride) {
    const int64_t t = t0 + group;
    const bool there = t < a.tokens;
    Token<EPL> x;
    x.load(static_cast<const T*>(a.logits) + (there ? t : 0) * a.ld, lane, a.experts,
           there && (!a.mask || a.mask[t] != 0));
    float e[EPL], total = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      e[i] = x.in ? expf(x.v[i] - x.top) : 0.0f;
      total += e[i];
    }
    total = row16_sum(total);
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum[i] += x.in ? e[i] / total : 0.0f;
    // the largest that is left, the first of equals, top_k times
    int32_t my_id = -1;
    float my_e = 0.0f, share = 0.0f;
    for (int j = 0; j < a.top_k; ++j) {
      float best = kClosed;
      uint32_t at = ~0u;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (x.v[i] > best) best = x.v[i], at = i * 16 + lane;
      const float top = row16_max(best);
      const uint32_t id = row16_min_u32(best == top && top > kClosed ? at : ~0u);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (id == (uint32_t)(i * 16 + lane)) x.v[i] = kClosed;
      const float ej = id != ~0u ? expf(top - x.top) : 0.0f;
      share += ej;
      if (lane == j) my_id = (int32_t)id, my_e = ej;
    }
    if (there && lane < a.top_k) {
      ids[t * a.top_k + lane] = my_id;
      const float of = a.renormalize ? share : total;
      // a NaN in the row shows in each of the weights
      p[t * a.top_k + lane] = my_id >= 0 ? (total == total ? my_e / of : total) : 0.0f;
      if (my_id >= 0) atomicAdd(&s_cnt[my_id], 1);
    }
    if (lane == 0 && x.in) atomicAdd(&s_cnt[a.experts], 1);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    sum[i] += __shfl_xor(sum[i], 16);
    sum[i] += __shfl_xor(sum[i], 32);
    if ((tid & 48) == 0) s_sum[wave][i * 16 + lane] = sum[i];
  }
  __syncthreads();
}

// Counts, sums and loss from their totals in LDS (one workgroup).
__device__ __forceinline__ void route_loss(int experts, int top_k, const double* total, const int32_t* cnt,
                                           int32_t* __restrict__ counts, float* __restrict__ sums,
                                           float* __restrict__ loss) {
  const int e = threadIdx.x;
  if (e <= experts) counts[e] = cnt[e];
  if (e < experts) sums[e] = (float)total[e];
  if (e < 64) {
    double l = 0.0;
    for (int i = e; i < experts; i += 64) l += (double)cnt[i] * total[i];
#pragma unroll
    for (int d = 32; d; d >>= 1) l += __shfl_xor(l, d);
    const double n = cnt[experts];
    if (e == 0) *loss = n > 0 ? (float)(experts * l / (n * n * top_k)) : 0.0f;
  }
}

template <typename T, int EPL, int THREADS, bool ALONE>
__global__ __launch_bounds__(THREADS) void k_route(const RouteArgs a, int32_t* __restrict__ ids,
                                                              float* __restrict__ p, float* __restrict__ part_sum,
                                                              int32_t* __restrict__ part_cnt,
                                                              int32_t* __restrict__ counts,
                                                              float* __restrict__ sums, float* __restrict__ loss) {
  __shared__ float s_sum[THREADS / 64][128];
  __shared__ int32_t s_cnt[129];
  __shared__ double s_total[128];
  route_tokens<T, EPL, THREADS>(a, ids, p, s_sum, s_cnt);
  const int e = threadIdx.x;
  if (e < a.experts) {
    double total = 0.0;
    for (int w = 0; w < THREADS / 64; ++w) total += s_sum[w][e];
    if constexpr (ALONE) s_total[e] = total;
    else part_sum[(int64_t)blockIdx.x * a.experts + e] = (float)total;
  }
  if constexpr (ALONE) {
    __syncthreads();
    route_loss(a.experts, a.top_k, s_total, s_cnt, counts, sums, loss);
  } else {
    if (e <= a.experts) part_cnt[(int64_t)blockIdx.x * (a.experts + 1) + e] = s_cnt[e];
  }
}

// The workgroups' sums in their order: a thread an expert and a run of 4 EPL workgroups, then the runs.  Every
// load is on its way before the first sum (256 workgroups' sums of 32 experts one after the other 14.7 us, by
// eight runs whatever the experts 7.2, so 3.3; 79 of 128 experts 7.1 and 5.2).
template <int EPL>
__global__ __launch_bounds__(1024) void k_route_sum(const float* __restrict__ part_sum,
                                                    const int32_t* __restrict__ part_cnt, int groups, int experts,
                                                    int top_k, int32_t* __restrict__ counts,
                                                    float* __restrict__ sums, float* __restrict__ loss) {
  constexpr int kWide = 16 * EPL, kRuns = 1024 / kWide, kRun = kRouteGroups / kRuns;
  __shared__ double s_run[kRuns][kWide];
  __shared__ int32_t s_crun[kRuns][kWide];
  __shared__ double s_total[128];
  __shared__ int32_t s_cnt[129];
  const int tid = threadIdx.x, e = tid % kWide, run = tid / kWide, at = min(e, experts - 1);
  if (tid == 0) s_cnt[experts] = 0;
  float x[kRun];
  int32_t n[kRun];
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    const int g = min(run * kRun + i, groups - 1);
    x[i] = part_sum[g * experts + at];
    n[i] = part_cnt[g * (experts + 1) + at];
  }
  int32_t tokens = tid < groups ? part_cnt[tid * (experts + 1) + experts] : 0;
  double total = 0.0;
  int32_t slots = 0;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    total += run * kRun + i < groups ? x[i] : 0.0f;
    slots += run * kRun + i < groups ? n[i] : 0;
  }
  s_run[run][e] = total;
  s_crun[run][e] = slots;
#pragma unroll
  for (int d = 32; d; d >>= 1) tokens += __shfl_xor(tokens, d);
  __syncthreads();
  if (tokens && (tid & 63) == 0) atomicAdd(&s_cnt[experts], tokens);
  if (tid < experts) {
    total = 0.0, slots = 0;
#pragma unroll
    for (int r = 0; r < kRuns; ++r) total += s_run[r][tid], slots += s_crun[r][tid];
    s_total[tid] = total;
    s_cnt[tid] = slots;
  }
  __syncthreads();
  route_loss(experts, top_k, s_total, s_cnt, counts, sums, loss);
}

template <typename T, int EPL>
__global__ __launch_bounds__(256) void k_route_bwd(const RouteArgs a, const int32_t* __restrict__ ids,
                                                   const int32_t* __restrict__ counts,
                                                   const float* __restrict__ dp, const float* __restrict__ dloss,
                                                   T* __restrict__ dlogits, int64_t ldd) {
  const int tid = threadIdx.x, lane = tid & 15, group = tid >> 4;
  float G[EPL];
  const double n = counts[a.experts];
  const double of = dloss && n > 0 ? (double)*dloss * a.experts / (n * n * a.top_k) : 0.0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 16 + lane;
    G[i] = e < a.experts ? (float)(of * counts[e]) : 0.0f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * 16; t0 < a.tokens; t0 += (int64_t)gridDim.x * 16) {
    const int64_t t = t0 + group;
    const bool there = t < a.tokens;
    Token<EPL> x;
    const T* row = static_cast<const T*>(a.logits) + (there ? t : 0) * a.ld;
    x.load(row, lane, a.experts, there && (!a.mask || a.mask[t] != 0));
    float s[EPL], total = 0.0f, sg = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      s[i] = x.in ? expf(x.v[i] - x.top) : 0.0f;
      total += s[i];
    }
    total = x.in ? row16_sum(total) : 1.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] /= total, sg += s[i] * G[i];
    sg = row16_sum(sg);
    // lane j: slot j's weight and its gradient
    int32_t id = -1;
    float pj = 0.0f, dj = 0.0f;
    if (there && x.in && lane < a.top_k && dp) {
      id = ids[t * a.top_k + lane];
      if (id >= 0 && id < a.experts) {
        const float v = route_value(row + id);
        pj = v == kClosed ? 0.0f : expf(v - x.top);
        dj = dp[t * a.top_k + lane];
      } else {
        id = -1;
      }
    }
    const float share = row16_sum(pj);
    pj = id >= 0 ? pj / (a.renormalize ? share : total) : 0.0f;
    const float C = row16_sum(pj * dj);
    const float mine = a.renormalize ? pj * (dj - C) : pj * dj;
    float d[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = s[i] * (G[i] - sg - (a.renormalize ? 0.0f : C));
    for (int j = 0; j < a.top_k; ++j) {
      const int32_t to = __shfl(id, (tid & 48) + j);
      const float term = __shfl(mine, (tid & 48) + j);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (to == i * 16 + lane) d[i] += term;
    }
    if (there) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = i * 16 + lane;
        if (e < a.experts) route_store(dlogits + t * ldd + e, x.in ? d[i] : 0.0f);
      }
    }
  }
}

// ============================================================== launches
static bool route_shape(int64_t tokens, int64_t experts, int64_t top_k) {
  return tokens >= 0 && experts >= 1 && experts <= MX_MAX_GROUPS && top_k >= 1 && top_k <= kRouteMaxK &&
         top_k <= experts && tokens <= (kMax8 - 1) / top_k;
}

}  // namespace mx

using namespace mx;

extern "C" size_t mx_moe_route_workspace_size(int64_t tokens, int64_t experts, int64_t top_k) {
  if (!route_shape(tokens, experts, top_k) || tokens <= kRouteAlone) return 0;
  return (size_t)route_groups(tokens) * (2 * experts + 1) * 4;
}

#define MX_ROUTE_WIDTH(CALL, T)            \
  do {                                     \
    if (experts <= 16) CALL(T, 1);         \
    else if (experts <= 32) CALL(T, 2);    \
    else if (experts <= 64) CALL(T, 4);    \
    else CALL(T, 8);                       \
  } while (0)

extern "C" int mx_moe_route(const void* logits, int dtype, int64_t ld, const uint8_t* mask, int64_t tokens,
                            int64_t experts, int64_t top_k, int renormalize, int32_t* ids, float* weights,
                            int32_t* counts, float* sums, float* loss, void* workspace, size_t workspace_bytes,
                            void* stream) {
  MX_REQUIRE(float_type(dtype) && (renormalize == 0 || renormalize == 1), MX_ERR_ENUM);
  MX_REQUIRE(route_shape(tokens, experts, top_k) && ld >= experts, MX_ERR_SHAPE);
  MX_REQUIRE(counts && sums && loss, MX_ERR_NULL);
  if (tokens) MX_REQUIRE(logits && ids && weights, MX_ERR_NULL);
  MX_REQUIRE(aligned16(logits) && aligned16(ids) && aligned16(weights) && aligned16(counts) && aligned16(sums) &&
                 (reinterpret_cast<uintptr_t>(loss) & 3) == 0, MX_ERR_ALIGN);
  const size_t need = mx_moe_route_workspace_size(tokens, experts, top_k);
  if (need) {
    MX_REQUIRE(workspace && workspace_bytes >= need, MX_ERR_WORKSPACE);
    MX_REQUIRE(aligned16(workspace), MX_ERR_ALIGN);
  }
  const RouteArgs a{logits, ld, tokens, mask, (int)experts, (int)top_k, renormalize};
  const hipStream_t st = as_stream(stream);
  const int groups = (int)route_groups(tokens);
  const bool half = route_threads(tokens) == 512;
  float* part = static_cast<float*>(workspace);
  int32_t* cnt = reinterpret_cast<int32_t*>(part + (need ? groups * experts : 0));
#define MX_ROUTE_TOKENS(T, EPL, THREADS)                                                                        \
  do {                                                                                                          \
    if (need)                                                                                                   \
      k_route<T, EPL, THREADS, false><<<groups, THREADS, 0, st>>>(a, ids, weights, part, cnt, counts, sums, loss); \
    else                                                                                                        \
      k_route<T, EPL, THREADS, true><<<1, THREADS, 0, st>>>(a, ids, weights, part, cnt, counts, sums, loss);     \
  } while (0)
#define MX_ROUTE(T, EPL)                                                                                          \
  do {                                                                                                            \
    if (half) MX_ROUTE_TOKENS(T, EPL, 512);                                                                       \
    else MX_ROUTE_TOKENS(T, EPL, 1024);                                                                           \
    if (need)                                                                                                     \
      k_route_sum<EPL><<<1, 1024, 0, st>>>(part, cnt, groups, (int)experts, (int)top_k, counts, sums, loss);       \
  } while (0)
  if (dtype == MX_F32) MX_ROUTE_WIDTH(MX_ROUTE, float);
  else MX_ROUTE_WIDTH(MX_ROUTE, uint16_t);
#undef MX_ROUTE
#undef MX_ROUTE_TOKENS
  return launch_status();
}

extern "C" int mx_moe_route_bwd(const void* logits, int dtype, int64_t ld, const uint8_t* mask, int64_t tokens,
                                int64_t experts, int64_t top_k, int renormalize, const int32_t* ids,
                                const int32_t* counts, const float* dweights, const float* dloss, void* dlogits,
                                int64_t ldd, void* stream) {
  MX_REQUIRE(float_type(dtype) && (renormalize == 0 || renormalize == 1), MX_ERR_ENUM);
  MX_REQUIRE(route_shape(tokens, experts, top_k) && ld >= experts && ldd >= experts, MX_ERR_SHAPE);
  if (tokens == 0) return MX_OK;
  MX_REQUIRE(logits && ids && counts && dlogits, MX_ERR_NULL);
  MX_REQUIRE(aligned16(logits) && aligned16(ids) && aligned16(counts) && aligned16(dweights) &&
                 aligned16(dlogits) && (reinterpret_cast<uintptr_t>(dloss) & 3) == 0, MX_ERR_ALIGN);
  const RouteArgs a{logits, ld, tokens, mask, (int)experts, (int)top_k, renormalize};
  const hipStream_t st = as_stream(stream);
  const dim3 grid((unsigned)hmin(cdiv(tokens, 16), (int64_t)device_cu_count() * 8));
#define MX_ROUTE_BWD(T, EPL)                                                                        \
  k_route_bwd<T, EPL><<<grid, 256, 0, st>>>(a, ids, counts, dweights, dloss, static_cast<T*>(dlogits), ldd)
  if (dtype == MX_F32) MX_ROUTE_WIDTH(MX_ROUTE_BWD, float);
  else MX_ROUTE_WIDTH(MX_ROUTE_BWD, uint16_t);
#undef MX_ROUTE_BWD
  return launch_status();
}
