// Router of the routed feed-forward: top-k selection and weights from router logits, and the
// gradient of the logits ([P1] "Concurrency, not sparsity, is the lever" names the routed model;
// the formulas are in sp24.h).
//
// One warp per token; lane l holds the logits l, l + 32, l + 64, ... of its row in registers, and works
// on them mapped to unsigned integers of the same order.
//
// Selection.  The topk-th largest of the 32 lanes' maxima is a floor under the topk largest logits
// (that many lanes have one at or above it).  The few logits at or above the floor, 32 at most, are
// gathered in shared memory and ranked against each other; that costs about a third of topk rounds
// of "largest one left, take it away" (T = 4096, E = 512, topk = 10: 5.4 against 9.0 us), which remain
// for rows whose ties leave more than 32, and for E <= 64, where a round is cheap (T = 16384, E = 64,
// topk = 8: 7.8 against 8.6 us).
//
// The logits of 4096 tokens over 512 experts are 8.4 MB, 1.3 us at the copy rate.  Forward 5.5 us (16-bit
// logits 5.4), gradient 4.5 us (16-bit 3.9; dense, softmax over all experts, 6.7 for 17 MB); 8 tokens 2.3 and
// 2.2 us.  A launch and one dependent load are 2.2 us of it.  Not bound by issue (46 % of its
// slots) nor by HBM (10 %): a token's chain of load, sort of maxima, gather and ranking is latency, with
// few warps to hide it.  The forward for 512 experts holds 80 registers, so six CTAs fit an SM, and
// 4096 tokens are 1024 CTAs, 1.15 times what the chip holds at once.
#include "sp24_launch.cuh"

namespace sp24 {
namespace {

constexpr int kMaxE = 1024, kMaxTopk = 32;
constexpr int kThreads = 128;  // four tokens per CTA
constexpr uint32_t kFull = 0xffffffffu;
constexpr uint32_t kKeyNegInf = 0x007fffffu;  // order_key(-inf): nothing at or below it is selected

template <int DT>
__device__ __forceinline__ float load_as_f32(const void* p, int64_t i) {
  if (DT == SP24_F32) return reinterpret_cast<const float*>(p)[i];
  if (DT == SP24_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(reinterpret_cast<const __half*>(p)[i]);
}

template <int DT>
__device__ __forceinline__ void store_f32(void* p, int64_t i, float v) {
  if (DT == SP24_F32)
    reinterpret_cast<float*>(p)[i] = v;
  else if (DT == SP24_BF16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half*>(p)[i] = __float2half_rn(v);
}

// A float as an unsigned integer of the same order; -0 as +0, NaN below everything.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  const uint32_t k = b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
  return v == v ? k : 0u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

template <int DT, int NV>
__global__ void __launch_bounds__(kThreads) route_topk_kernel(const void* logits, int64_t T, int E,
                                                              int topk, int scoring, int renorm,
                                                              int32_t* routing,
                                                              float* router_w) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  begin();
  if (t >= T) return;
  uint32_t key[NV];
  float raw[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    raw[j] = e < E ? load_as_f32<DT>(logits, t * E + e) : -INFINITY;
  }
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    key[j] = order_key(raw[j]);
    best = max(best, key[j]);
  }
  float total = 0.0f;  // softmax over all experts: its denominator about the row's maximum
  if (scoring == SP24_ROUTE_SOFTMAX && !renorm) {
    const float m = key_value(__reduce_max_sync(kFull, best));
#pragma unroll
    for (int j = 0; j < NV; ++j) total += expf(raw[j] - m);
    total = warp_sum(total);
  }
  // lane s is to keep slot s
  uint32_t mine = 0;
  int mine_id = -1;
  bool gathered = false;
  if constexpr (NV > 2) {
    uint32_t floor_key = best;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
      for (int d = size / 2; d; d /= 2) {  // bitonic, largest first
        const uint32_t other = __shfl_xor_sync(kFull, floor_key, d);
        const bool upper = (lane & d) != 0, rising = (lane & size) != 0 && size < 32;
        floor_key = upper == rising ? max(floor_key, other) : min(floor_key, other);
      }
    floor_key = max(__shfl_sync(kFull, floor_key, topk - 1), kKeyNegInf + 1);
    int count = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) count += key[j] >= floor_key;
    const int total_count = __reduce_add_sync(kFull, count);
    __shared__ uint2 table[kThreads / 32][2][32];
    gathered = total_count <= 32;
    if (gathered) {
      uint2* const found = table[threadIdx.x >> 5][0];
      uint2* const ranked = table[threadIdx.x >> 5][1];
      int at = count;  // exclusive sum over the lanes
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(kFull, at, d);
        if (lane >= d) at += o;
      }
      at -= count;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (key[j] >= floor_key) found[at++] = make_uint2(key[j], lane + 32 * j);
      __syncwarp();
      const uint2 own = lane < total_count ? found[lane] : make_uint2(0, 0);
      int rank = 0;
      for (int i = 0; i < total_count; ++i) {
        const uint2 other = found[i];
        rank += other.x > own.x || (other.x == own.x && other.y < own.y);
      }
      if (lane < total_count) ranked[rank] = own;
      __syncwarp();
      if (lane < min(total_count, topk)) {
        mine = ranked[lane].x;
        mine_id = (int)ranked[lane].y;
      }
    }
  }
  if (!gathered) {
    for (int s = 0; s < topk; ++s) {
      const uint32_t top = __reduce_max_sync(kFull, best);
      if (top <= kKeyNegInf) break;
      int at = INT32_MAX;
#pragma unroll
      for (int j = NV - 1; j >= 0; --j)
        if (key[j] == top) at = lane + 32 * j;
      at = __reduce_min_sync(kFull, at);
      if (lane == s) {
        mine = top;
        mine_id = at;
      }
      best = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (at == lane + 32 * j) key[j] = 0;
        best = max(best, key[j]);
      }
    }
  }
  const bool live = mine_id >= 0;
  const float v = live ? key_value(mine) : -INFINITY;
  float w = 0.0f;
  if (scoring == SP24_ROUTE_SOFTMAX) {
    const float m = __shfl_sync(kFull, v, 0);  // slot 0 holds the maximum
    w = live ? expf(v - m) : 0.0f;
  } else {
    w = live ? sigmoid(v) : 0.0f;
  }
  if (renorm) total = warp_sum(w);
  if (scoring == SP24_ROUTE_SOFTMAX || renorm) w = live && total != 0.0f ? w / total : 0.0f;
  if (lane < topk) {
    routing[t * topk + lane] = mine_id;
    router_w[t * topk + lane] = w;
  }
}

template <int DT, int NV>
__global__ void __launch_bounds__(kThreads) route_backward_kernel(const void* logits, int64_t T, int E,
                                                                  int topk, int scoring, int renorm,
                                                                  const int32_t* routing,
                                                                  const float* d_router_w,
                                                                  void* dlogits) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  begin();
  if (t >= T) return;
  int id = lane < topk ? routing[t * topk + lane] : -1;
  if (id < 0 || id >= E) {
    if (id != -1) set_dev_error(SP24_ERR_INVALID_ARG);
    id = -1;
  }
  const bool live = id >= 0;
  const float g = live ? d_router_w[t * topk + lane] : 0.0f;
  const float v = live ? load_as_f32<DT>(logits, t * E + id) : -INFINITY;
  const bool any = __any_sync(kFull, live);

  float part = 0.0f;    // this slot's share of its expert's gradient
  float p_scale = 0.0f; // softmax over all experts: dl_e = share_e - exp(l_e - m) * p_scale
  float m = 0.0f;
  float raw[NV];
  const bool dense = scoring == SP24_ROUTE_SOFTMAX && !renorm && any;
  if (scoring == SP24_ROUTE_SOFTMAX) {
    if (dense) {
      m = -INFINITY;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int e = lane + 32 * j;
        raw[j] = e < E ? load_as_f32<DT>(logits, t * E + e) : -INFINITY;
        m = fmaxf(m, raw[j]);
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
      float total = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        raw[j] = expf(raw[j] - m);
        total += raw[j];
      }
      total = warp_sum(total);
      const float w = live ? expf(v - m) / total : 0.0f;
      const float dot = warp_sum(w * g);
      p_scale = dot / total;
      part = w * g;
    } else {
      m = v;
#pragma unroll
      for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
      float w = live ? expf(v - m) : 0.0f;
      const float total = warp_sum(w);
      w = live ? w / total : 0.0f;
      const float dot = warp_sum(w * g);
      part = live ? w * (g - dot) : 0.0f;
    }
  } else {
    const float up = live ? sigmoid(v) : 0.0f;
    const float slope = live ? up * sigmoid(-v) : 0.0f;
    if (renorm) {
      const float total = warp_sum(up);
      const float dot = total != 0.0f ? warp_sum(up * g) / total : 0.0f;
      part = live && total != 0.0f ? slope * (g - dot) / total : 0.0f;
    } else {
      part = slope * g;
    }
  }
  // an expert met by several slots: the first of them writes the sum, in slot order
  float sum = 0.0f;
  bool first = live;
  for (int s = 0; s < topk; ++s) {
    const int other = __shfl_sync(kFull, id, s);
    const float add = __shfl_sync(kFull, part, s);
    if (other == id) {
      sum += add;
      if (s < lane) first = false;
    }
  }
  if (dense) sum -= expf(v - m) * p_scale;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = lane + 32 * j;
    if (e < E) store_f32<DT>(dlogits, t * E + e, dense ? -raw[j] * p_scale : 0.0f);
  }
  __syncwarp();  // the shares below overwrite entries that other lanes have just stored
  if (live && first) store_f32<DT>(dlogits, t * E + id, sum);
}

template <template <int, int> class Launch, int DT, typename... A>
int by_experts(int64_t E, A... a) {
  if (E <= 32) return Launch<DT, 1>::go(a...);
  if (E <= 64) return Launch<DT, 2>::go(a...);
  if (E <= 128) return Launch<DT, 4>::go(a...);
  if (E <= 256) return Launch<DT, 8>::go(a...);
  if (E <= 512) return Launch<DT, 16>::go(a...);
  return Launch<DT, 32>::go(a...);
}

template <template <int, int> class Launch, typename... A>
int by_type(int dtype, int64_t E, A... a) {
  if (dtype == SP24_F32) return by_experts<Launch, SP24_F32>(E, a...);
  if (dtype == SP24_BF16) return by_experts<Launch, SP24_BF16>(E, a...);
  return by_experts<Launch, SP24_F16>(E, a...);
}

unsigned token_ctas(int64_t T) { return (unsigned)((T + kThreads / 32 - 1) / (kThreads / 32)); }

template <int DT, int NV>
struct LaunchTopk {
  static int go(const void* l, int64_t T, int64_t E, int k, int sc, int rn, int32_t* r, float* w, cudaStream_t s) {
    return launch_after(route_topk_kernel<DT, NV>, token_ctas(T), kThreads, 0, s, l, T, (int)E, k, sc, rn, r, w);
  }
};
template <int DT, int NV>
struct LaunchBackward {
  static int go(const void* l, int64_t T, int64_t E, int k, int sc, int rn, const int32_t* r, const float* g, void* d,
                cudaStream_t s) {
    return launch_after(route_backward_kernel<DT, NV>, token_ctas(T), kThreads, 0, s, l, T, (int)E, k, sc, rn, r, g, d);
  }
};

int check_route(int dtype, int64_t T, int64_t E, int topk, int scoring) {
  if (!elem_bytes(dtype)) return SP24_ERR_DTYPE;
  if (scoring != SP24_ROUTE_SOFTMAX && scoring != SP24_ROUTE_SIGMOID) return SP24_ERR_INVALID_ARG;
  if (T < 0 || E < 1 || topk < 1 || topk > E) return SP24_ERR_SHAPE;
  if (E > kMaxE || topk > kMaxTopk || T > INT32_MAX) return SP24_ERR_UNSUPPORTED;
  return SP24_OK;
}

}  // namespace
}  // namespace sp24

using namespace sp24;

extern "C" int sp24_moe_route(const void* logits, int dtype, int64_t T, int64_t E, int topk, int scoring,
                              int renormalize, int32_t* routing, float* router_w, void* stream) {
  const int st = check_route(dtype, T, E, topk, scoring);
  if (st) return st;
  if (T == 0) return SP24_OK;
  if (!logits || !routing || !router_w) return SP24_ERR_INVALID_ARG;
  if (!aligned(logits, elem_bytes(dtype)) || !aligned(routing, 4) || !aligned(router_w, 4)) return SP24_ERR_ALIGN;
  return by_type<LaunchTopk>(dtype, E, logits, T, E, topk, scoring, renormalize, routing, router_w, as_stream(stream));
}

extern "C" int sp24_moe_route_backward(const void* logits, int dtype, const int32_t* routing, const float* d_router_w,
                                       int64_t T, int64_t E, int topk, int scoring, int renormalize, void* dlogits,
                                       void* stream) {
  const int st = check_route(dtype, T, E, topk, scoring);
  if (st) return st;
  if (T == 0) return SP24_OK;
  if (!logits || !routing || !d_router_w || !dlogits) return SP24_ERR_INVALID_ARG;
  if (!aligned(logits, elem_bytes(dtype)) || !aligned(dlogits, elem_bytes(dtype)) || !aligned(routing, 4) ||
      !aligned(d_router_w, 4))
    return SP24_ERR_ALIGN;
  return by_type<LaunchBackward>(dtype, E, logits, T, E, topk, scoring, renormalize, routing, d_router_w, dlogits,
                                 as_stream(stream));
}
