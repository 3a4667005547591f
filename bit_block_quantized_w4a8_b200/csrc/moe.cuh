// moe.cuh -- the token side of a mixture-of-experts layer around the grouped
// GEMM: routing (logits -> experts and weights), dispatch (rows grouped by
// expert and quantized into that order) and combine (weighted sum of a
// token's expert outputs).
#pragma once
#include <cuda_bf16.h>

#include <cstdint>
#include "ptx.cuh"
#include "quant.cuh"

namespace w4a8 {

// ------------------------------------------------------------------ routing
// One warp per token.  The E logits of a token sit in registers; the choice
// is k rounds of a warp-wide maximum over order-preserving integer keys
// (redux.sync), ties to the lowest expert.
//
// Keys.  Without a bias an expert's score grows with its logit, so the order
// of the logits IS the order of the scores and no arithmetic can blur it.
// With a bias (or when a group is scored by the sum of its two best) the keys
// are sums of a score and a number, and two of them can be closer than fp32
// tells apart; they are computed in fp64, whose units on this chip run at half
// the fp32 rate, so that the chosen experts are those of the definition.
// Weights are fp32.
//
// Layout.  The lanes are divided evenly among the groups (rounded up to a
// power of two), so a group's score is a few shuffles among its own lanes
// for all groups at once; with one group every lane holds every 32nd expert.
constexpr int kRouteWarps = 4;
constexpr float kMaskedLogit = -3.3895313892515355e38f;  // bf16's lowest finite value

struct RouteParams {
  const void* logits;
  int bf16;             // logits type: 0 = fp32, 1 = bf16
  int M, E, k;
  int sigmoid;
  const float* bias;    // [E] or nullptr
  int groups, top_groups, group_top;
  int lanes_per_group;  // power of two, lanes_per_group * ceil2(groups) = 32
  int renormalize;
  float scale;
  int* ids;
  float* weights;
};

__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 and +0 are one value
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
// warp maximum of a key: one redux for 32 bits, two for 64
__device__ __forceinline__ uint32_t warp_max_key(uint32_t v) {
  return __reduce_max_sync(0xffffffffu, v);
}
__device__ __forceinline__ uint64_t warp_max_key(uint64_t v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo = __reduce_max_sync(
      0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// MODE 0: logit keys, groups (if any) scored by their best logit;
// MODE 1: logit keys, groups scored by sums of two fp64 scores;
// MODE 2: fp64 keys score + bias.
template <int MODE> struct RouteKey { using type = uint32_t; };
template <> struct RouteKey<2> { using type = uint64_t; };

template <int NV, int MODE>
__global__ void __launch_bounds__(kRouteWarps * 32) route_kernel(const RouteParams p) {
  using Key = typename RouteKey<MODE>::type;
  constexpr uint32_t kFull = 0xffffffffu;
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const long long m = (long long)blockIdx.x * kRouteWarps + (threadIdx.x >> 5);
  if (m >= p.M) return;
  const int lg = p.lanes_per_group;
  const int sub = lane & (lg - 1), grp = lane / lg;
  const int size = p.E / p.groups;
  const int e0 = grp * size + sub;
  const float* lf = static_cast<const float*>(p.logits) + m * p.E;
  const __nv_bfloat16* lb = static_cast<const __nv_bfloat16*>(p.logits) + m * p.E;
  float l[NV];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const bool in = grp < p.groups && sub + i * lg < size;
    float v = -INFINITY;
    if (in) v = p.bf16 ? __bfloat162float(lb[e0 + i * lg]) : lf[e0 + i * lg];
    l[i] = v > kMaskedLogit ? v : -INFINITY;  // (false for NaN)
    mx = fmaxf(mx, l[i]);
  }
  mx = warp_max(mx);

  // the softmax's denominator, where something needs it
  double inv_sum = 1.0;
  float sum_f = 1.0f;
  if (MODE != 0 && !p.sigmoid) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (l[i] > -INFINITY) s += l[i] == mx ? 1.0 : exp((double)l[i] - (double)mx);
    s = warp_sum(s);
    inv_sum = s > 0.0 ? 1.0 / s : 0.0;
  }
  if (!p.renormalize && !p.sigmoid) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (l[i] > -INFINITY) s += l[i] == mx ? 1.0f : expf(l[i] - mx);
    sum_f = warp_sum(s);
  }
  auto score = [&](float x) -> double {  // x unmasked
    if (p.sigmoid) return 1.0 / (1.0 + exp(-(double)x));
    return x == mx ? inv_sum : exp((double)x - (double)mx) * inv_sum;
  };

  Key key[NV];  // 0 = masked
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    key[i] = 0;
    if (l[i] > -INFINITY) {
      if constexpr (MODE == 2)
        key[i] = order_key(score(l[i]) + (double)__ldg(p.bias + e0 + i * lg));
      else
        key[i] = order_key(l[i]);
    }
  }

  if (p.groups > 1) {
    uint64_t gkey = 0;  // 0 = no expert of the group is left
    if constexpr (MODE == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) gkey = max(gkey, (uint64_t)key[i]);
      for (int o = lg / 2; o > 0; o >>= 1)
        gkey = max(gkey, (uint64_t)__shfl_xor_sync(kFull, (uint32_t)gkey, o));
    } else {
      // the two best scores of the group (a missing one is -inf)
      double a = -INFINITY, b = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (!(l[i] > -INFINITY)) continue;
        double v;
        if constexpr (MODE == 2) {
          const uint64_t u = key[i];  // the key is the score's bits
          v = __longlong_as_double((long long)((u >> 63) ? u & 0x7fffffffffffffffull : ~u));
        } else {
          v = score(l[i]);
        }
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      for (int o = lg / 2; o > 0; o >>= 1) {
        const double a2 = __shfl_xor_sync(kFull, a, o), b2 = __shfl_xor_sync(kFull, b, o);
        const double hi = fmax(a, a2), lo = fmin(a, a2);
        b = fmax(lo, a == hi ? b : b2);
        a = hi;
      }
      if (a > -INFINITY) gkey = order_key(p.group_top == 2 && b > -INFINITY ? a + b : a);
    }
    int before = 0;
    for (int h = 0; h < p.groups; ++h) {
      const uint64_t o = __shfl_sync(kFull, gkey, h * lg);
      before += o > gkey || (o == gkey && h < grp);
    }
    if (before >= p.top_groups) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = 0;
    }
  }

  // k rounds: the largest key, the lowest expert among equals.  Lane j keeps
  // the j-th choice.
  int mine = -1;
  for (int j = 0; j < p.k; ++j) {
    Key best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const Key top = warp_max_key(best);
    if (top == 0) break;  // nothing is left
    const uint32_t e = __reduce_min_sync(
        kFull, best == top ? (uint32_t)(e0 + at * lg) : 0xffffffffu);
    if (lane == j) mine = (int)e;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (best == top && (uint32_t)(e0 + i * lg) == e) key[i] = 0;
  }

  // weights: lane j holds the j-th choice's logit
  const bool has = mine >= 0;
  float x = -INFINITY;
  if (has) x = p.bf16 ? __bfloat162float(lb[mine]) : lf[mine];
  float w = 0.0f;
  if (!p.sigmoid) {
    // renormalised: relative to the largest chosen logit, so that chosen
    // experts far below the row's maximum keep their proportions
    const float ref = p.renormalize ? warp_max(x) : mx;
    if (has) w = x == ref ? 1.0f : expf(x - ref);
    const float s = p.renormalize ? warp_sum(w) : sum_f;
    if (has) w = w / s;
  } else {
    // sigmoid(x) = exp(min(x, 0)) / (1 + exp(-|x|)); the renormalised form
    // takes the largest chosen exponent out of both sides
    const float t = fminf(x, 0.0f);
    const float ref = p.renormalize ? warp_max(t) : 0.0f;
    if (has) w = (t == ref ? 1.0f : expf(t - ref)) / (1.0f + expf(-fabsf(x)));
    if (p.renormalize) {
      const float s = warp_sum(w);
      if (has) w = w / s;
    }
  }
  if (lane < p.k) {
    p.ids[m * p.k + lane] = mine;
    p.weights[m * p.k + lane] = has ? w * p.scale : 0.0f;
  }
}

// ----------------------------------------------------------------- grouping
// Stable counting sort of n small integers: offsets[g] = how many valid ids
// are below g, pos[i] = the place of pair i (-1 where its id is outside
// [0, groups)), rows[pos[i]] = i.  One CTA, or one cluster of kGroupCluster
// CTAs that exchange their counts through distributed shared memory.  Every
// warp owns a contiguous stretch of the ids and ranks 32 of them at a time
// with match.any, so places follow the order of the pairs and the result does
// not depend on timing.
constexpr int kGroupThreads = 1024;
constexpr int kGroupCluster = 8;
constexpr int kMaxGroups = 1024;

inline size_t group_rows_smem(int groups) { return (size_t)(32 + 2) * groups * sizeof(int); }

__global__ void __launch_bounds__(kGroupThreads) group_rows_kernel(
    const int* __restrict__ ids, int n, int groups, int ctas, int* __restrict__ offsets,
    int* __restrict__ rows, int* __restrict__ pos) {
  extern __shared__ int gsm[];
  __shared__ int wsum[32];
  int* hist = gsm;                   // [32][groups]: counts, then places within the CTA
  int* total = gsm + 32 * groups;    // [groups]: this CTA's counts
  int* start = total + groups;       // [groups]: first place of this CTA's pairs
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ctas > 1 ? (int)cluster_ctarank() : 0;
  for (int i = tid; i < 32 * groups; i += kGroupThreads) hist[i] = 0;
  pdl_wait();  // ids may be written by the preceding kernel
  pdl_launch_dependents();
  __syncthreads();
  const int chunks = ctas * 32;
  const int per = ((n + chunks - 1) / chunks + 31) & ~31;
  const int lo = (int)min((long long)n, (long long)(rank * 32 + warp) * per);
  const int hi = min(n, lo + per);
  int* mine = hist + warp * groups;
  for (int b = lo; b < hi; b += 32) {
    const int i = b + lane;
    const int e = i < hi ? ids[i] : -1;
    const bool ok = (unsigned)e < (unsigned)groups;
    const unsigned same = __match_any_sync(0xffffffffu, ok ? e : -1);
    if (ok && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  int own = 0;
  if (tid < groups) {
#pragma unroll 8
    for (int w = 0; w < 32; ++w) {
      const int c = hist[w * groups + tid];
      hist[w * groups + tid] = own;
      own += c;
    }
    total[tid] = own;
  }
  if (ctas > 1) cluster_sync_all();
  int base = 0, all = own;
  if (ctas > 1 && tid < groups) {
    all = 0;
    for (int c = 0; c < ctas; ++c) {
      const int v = dsmem_ld_s32(dsmem_map(smem_u32(total + tid), c));
      if (c < rank) base += v;
      all += v;
    }
  }
  int incl = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = wsum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    wsum[lane] = v;
  }
  __syncthreads();
  if (tid < groups) {
    const int first = incl - all + (warp > 0 ? wsum[warp - 1] : 0);
    start[tid] = first + base;
    if (rank == 0) {
      offsets[tid] = first;
      if (tid == groups - 1) offsets[groups] = first + all;
    }
  }
  __syncthreads();
  for (int b = lo; b < hi; b += 32) {
    const int i = b + lane;
    const int e = i < hi ? ids[i] : -1;
    const bool ok = (unsigned)e < (unsigned)groups;
    const unsigned same = __match_any_sync(0xffffffffu, ok ? e : -1);
    int at = -1;
    if (ok) at = start[e] + mine[e] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (ok && lane == __ffs(same) - 1) mine[e] += __popc(same);
    __syncwarp();
    if (ok) rows[at] = i;
    if (pos != nullptr && i < hi) pos[i] = at;
  }
  // no CTA leaves while another may still read its counts
  if (ctas > 1) cluster_sync_all();
}

// ----------------------------------------------------------------- dispatch
// One CTA per token: the row is read once, quantized by the rule of
// act_quant_kernel (the same codes and scale), its codes are laid out in
// shared memory, and one bulk copy per kept slot writes them to their rows.
// Bound by HBM: K s bytes in, K bytes out per kept slot.
//
// SMALL (M * top_k <= kDispatchSmall): the CTA also finds its slots' places
// itself, by counting the pairs that come before them (all ids fit the CTA's
// registers), and one more CTA writes the offsets: one launch.  Otherwise
// group_rows_kernel ran before, and this kernel (launched so that it may
// start early) reads and quantizes its row before it waits for the places.
constexpr int kDispatchThreads = 256;
constexpr int kDispatchIds = 8;  // ids per thread (SMALL)
constexpr int kDispatchSmall = kDispatchThreads * kDispatchIds;
constexpr int kMaxTopK = 32;

template <bool BF16>
struct RowVec;
template <>
struct RowVec<false> {
  static constexpr int kElems = 4;
  using Raw = float4;
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
  static __device__ __forceinline__ float absmax(Raw v) { return absmax4(v); }
  static __device__ __forceinline__ void store(uint8_t* codes, int idx, Raw v, float s, float y,
                                               bool rcp) {
    reinterpret_cast<uint32_t*>(codes)[idx] = rcp ? quant4_rcp(v, s, y) : quant4(v, s);
  }
};
template <>
struct RowVec<true> {
  static constexpr int kElems = 8;
  using Raw = uint4;
  static __device__ __forceinline__ Raw zero() { return make_uint4(0, 0, 0, 0); }
  static __device__ __forceinline__ float4 low(Raw v) {
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u),
                       __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
  static __device__ __forceinline__ float4 high(Raw v) {
    return make_float4(__uint_as_float(v.z << 16), __uint_as_float(v.z & 0xffff0000u),
                       __uint_as_float(v.w << 16), __uint_as_float(v.w & 0xffff0000u));
  }
  static __device__ __forceinline__ float absmax(Raw v) {
    return fmaxf(absmax4(low(v)), absmax4(high(v)));
  }
  static __device__ __forceinline__ void store(uint8_t* codes, int idx, Raw v, float s, float y,
                                               bool rcp) {
    const float4 a = low(v), b = high(v);
    reinterpret_cast<uint2*>(codes)[idx] =
        rcp ? make_uint2(quant4_rcp(a, s, y), quant4_rcp(b, s, y))
            : make_uint2(quant4(a, s), quant4(b, s));
  }
};

template <bool BF16, bool SMALL>
__global__ void __launch_bounds__(kDispatchThreads) dispatch_kernel(
    const void* __restrict__ X, int M, int K, const int* __restrict__ ids, int top_k, int groups,
    int8_t* __restrict__ Xq, float* __restrict__ s_x, int* __restrict__ offsets,
    int* __restrict__ rows, int* __restrict__ pos) {
  using V = RowVec<BF16>;
  constexpr int kRegs = 8192 / (V::kElems * kDispatchThreads);  // a row of 8192 stays in registers
  extern __shared__ __align__(16) uint8_t codes[];              // [K]
  __shared__ float red[kDispatchThreads / 32];
  __shared__ int place[kMaxTopK];
  __shared__ int hist[SMALL ? kMaxGroups : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int m = blockIdx.x;
  if (SMALL) {
    pdl_launch_dependents();
    pdl_wait();
    if (m == M) {  // the offsets
      for (int g = tid; g < groups; g += kDispatchThreads) hist[g] = 0;
      __syncthreads();
      for (int i = tid; i < M * top_k; i += kDispatchThreads) {
        const int e = ids[i];
        if ((unsigned)e < (unsigned)groups) atomicAdd(hist + e, 1);
      }
      __syncthreads();
      if (warp == 0) {
        int sum = 0;
        for (int g0 = 0; g0 < groups; g0 += 32) {
          const int c = g0 + lane < groups ? hist[g0 + lane] : 0;
          int incl = c;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
          }
          if (g0 + lane < groups) offsets[g0 + lane] = sum + incl - c;
          sum += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) offsets[groups] = sum;
      }
      return;
    }
  }
  const typename V::Raw* row = reinterpret_cast<const typename V::Raw*>(
      static_cast<const uint8_t*>(X) + (size_t)m * K * (BF16 ? 2 : 4));
  const int nv = K / V::kElems;
  typename V::Raw v[kRegs];
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const int idx = tid + i * kDispatchThreads;
    v[i] = idx < nv ? __ldg(row + idx) : V::zero();
  }
  if (SMALL) {
    if (tid < top_k) place[tid] = 0;
    int id[kDispatchIds];
    const int n = M * top_k;
#pragma unroll
    for (int i = 0; i < kDispatchIds; ++i) {
      const int at = tid + i * kDispatchThreads;
      id[i] = at < n ? ids[at] : -1;
    }
    __syncthreads();
    for (int j = 0; j < top_k; ++j) {
      const int self = m * top_k + j;
      const int e = ids[self];
      int c = 0;
#pragma unroll
      for (int i = 0; i < kDispatchIds; ++i)
        c += id[i] >= 0 && (id[i] < e || (id[i] == e && tid + i * kDispatchThreads < self));
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0 && c) atomicAdd(place + j, c);
    }
  }
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) amax = fmaxf(amax, V::absmax(v[i]));
  for (int idx = tid + kRegs * kDispatchThreads; idx < nv; idx += kDispatchThreads)
    amax = fmaxf(amax, V::absmax(__ldg(row + idx)));
  amax = warp_max(amax);
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < kDispatchThreads / 32; ++w) amax = fmaxf(amax, red[w]);
  const float s = __fdiv_rn(amax, 127.0f);
  const bool rcp = rcp_quant_ok(s);
  const float y = rcp ? __fdiv_rn(1.0f, s) : 0.0f;
#pragma unroll
  for (int i = 0; i < kRegs; ++i) {
    const int idx = tid + i * kDispatchThreads;
    if (idx < nv) V::store(codes, idx, v[i], s, y, rcp);
  }
  for (int idx = tid + kRegs * kDispatchThreads; idx < nv; idx += kDispatchThreads)
    V::store(codes, idx, __ldg(row + idx), s, y, rcp);
  fence_proxy_async_smem();  // the codes are read by the bulk copies
  if (!SMALL) pdl_wait();    // the places, from group_rows_kernel
  __syncthreads();
  if (!SMALL) pdl_launch_dependents();
  if (tid < top_k) {
    int p = -1;
    if (SMALL) {
      const int e = ids[m * top_k + tid];
      if ((unsigned)e < (unsigned)groups) p = place[tid];
      pos[m * top_k + tid] = p;
      if (p >= 0) rows[p] = m * top_k + tid;
    } else {
      p = pos[m * top_k + tid];
    }
    if (p >= 0) {
      bulk_s2g(Xq + (size_t)p * K, smem_u32(codes), (uint32_t)K);
      s_x[p] = s;
    }
    bulk_commit_group();
    bulk_wait_group_read_all();  // the codes stay until they are read
  }
}

// ------------------------------------------------------------------ combine
// out[m] = sum_j weights[m][j] * Y[pos[m][j]] in fp32, slot by slot, rounded
// once.  One thread per VEC adjacent columns; the rows of a token's slots
// are read kCombineBatch at a time.  Bound by HBM: 2 N bytes per slot.
constexpr int kCombineThreads = 256;
constexpr int kCombineBatch = 8;

__device__ __forceinline__ void store_out(float* out, size_t i, const float (&a)[8]) {
  float4* o = reinterpret_cast<float4*>(out + i);
  o[0] = make_float4(a[0], a[1], a[2], a[3]);
  o[1] = make_float4(a[4], a[5], a[6], a[7]);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}
__device__ __forceinline__ void store_out(__nv_bfloat16* out, size_t i, const float (&a)[8]) {
  *reinterpret_cast<uint4*>(out + i) =
      make_uint4(pack_bf16(a[0], a[1]), pack_bf16(a[2], a[3]), pack_bf16(a[4], a[5]),
                 pack_bf16(a[6], a[7]));
}
__device__ __forceinline__ void store_out(float* out, size_t i, const float (&a)[1]) {
  out[i] = a[0];
}
__device__ __forceinline__ void store_out(__nv_bfloat16* out, size_t i, const float (&a)[1]) {
  out[i] = __float2bfloat16_rn(a[0]);
}

template <typename OutT, int VEC>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(
    const uint16_t* __restrict__ Y, int rows, int N, const int* __restrict__ pos,
    const float* __restrict__ weights, int top_k, OutT* __restrict__ out) {
  __shared__ int sp[kMaxTopK];
  __shared__ float sw[kMaxTopK];
  pdl_launch_dependents();
  pdl_wait();
  const size_t m = blockIdx.x;
  if (threadIdx.x < top_k) {
    const int p = pos[m * top_k + threadIdx.x];
    sp[threadIdx.x] = (unsigned)p < (unsigned)rows ? p : -1;
    sw[threadIdx.x] = weights[m * top_k + threadIdx.x];
  }
  __syncthreads();
  const int col = (blockIdx.y * kCombineThreads + threadIdx.x) * VEC;
  if (col >= N) return;
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < top_k; j0 += kCombineBatch) {
    if constexpr (VEC == 8) {
      uint4 v[kCombineBatch];
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {
        const int p = j0 + b < top_k ? sp[j0 + b] : -1;
        v[b] = make_uint4(0, 0, 0, 0);
        if (p >= 0) v[b] = __ldg(reinterpret_cast<const uint4*>(Y + (size_t)p * N + col));
      }
#pragma unroll
      for (int b = 0; b < kCombineBatch; ++b) {
        if (j0 + b >= top_k || sp[j0 + b] < 0) continue;
        const float w = sw[j0 + b];
        const float4 lo = RowVec<true>::low(v[b]), hi = RowVec<true>::high(v[b]);
        const float x[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, x[i], acc[i]);
      }
    } else {
      for (int b = 0; b < kCombineBatch && j0 + b < top_k; ++b) {
        const int p = sp[j0 + b];
        if (p >= 0)
          acc[0] = fmaf(sw[j0 + b],
                        __uint_as_float((uint32_t)__ldg(Y + (size_t)p * N + col) << 16), acc[0]);
      }
    }
  }
  store_out(out, m * N + col, acc);
}

}  // namespace w4a8
