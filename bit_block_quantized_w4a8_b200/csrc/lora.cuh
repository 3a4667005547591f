// lora.cuh -- low-rank adapters of many requests beside a shared projection:
//   Y[m] += scale[a] * B[a] (A[a] x_m),   a = the adapter of row m,
// A [L][r][K], B [L][N][r] bf16, X fp32 or bf16, Y bf16 (the projection's
// output, updated in place; rows without an adapter are not touched).
//
// One launch does both products.  Rows are taken in tiles that share an
// adapter: the grouped order of group_rows_kernel, or for a few rows the
// order that each CTA finds from the ids by itself (a launch less).  A
// cluster of CTAs owns a tile: each CTA multiplies its stretch of K (t = A x, summed over the
// CTA's warps in shared memory and over the cluster through distributed
// shared memory), then updates its stretch of N.  t never leaves the chip.
//
// Bound by HBM (X and Y once, A and B once per adapter and tile, mostly from
// L2): at ranks up to 64 the tensor work is far below the bytes, so warp
// level MMAs (m16n8k16) fed straight from global memory carry it.  Both
// products may sum their index in any order, so each lane takes 8 adjacent
// elements of a row (16-byte loads) and calls them the four k pairs that its
// MMA fragments want; the same trick gives each lane 8 adjacent output
// columns.
//
// Rounding: fp32 activations and t enter the MMAs as two bf16 terms (the
// value rounded to bf16, and the rest rounded to bf16), which keeps 16
// bits of them: the error left is below 2^-16 of the value, far under the
// one rounding of the sum to Y's bf16 (2^-8).  All sums are fp32; y + delta
// is rounded once.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>
#include "moe.cuh"
#include "ptx.cuh"

namespace w4a8 {

constexpr int kLoraThreads = 256;
constexpr int kLoraWarps = kLoraThreads / 32;
constexpr int kLoraMaxRank = 128;
constexpr int kLoraMaxAdapters = kMaxGroups;
constexpr int kLoraIdsMax = kLoraThreads;  // rows that a CTA groups by itself

struct LoraParams {
  const void* X;
  long long ldx;
  int M, K, N, rank, adapters;
  const uint16_t* A;
  const uint16_t* B;
  const float* scale;  // [adapters] or nullptr (1)
  const int* ids;      // [M], or nullptr with the rows grouped already:
  const int* offsets;  // [adapters + 1]
  const int* rows;     // [M]
  uint16_t* Y;
  long long ldy;
  int y_vec;           // rows of Y are 16-byte aligned
  int ctas;            // cluster size
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// x0, x1 as two bf16 pairs whose sum is them to 16 bits
__device__ __forceinline__ void split_bf16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(x0, x1);
  lo = pack_bf16(x0 - __uint_as_float(hi << 16), x1 - __uint_as_float(hi & 0xffff0000u));
}

template <int NT, int WR>
struct LoraCfg {
  static constexpr int kTileRows = 16 * WR;
  static constexpr int kWarpsK = kLoraWarps / WR;
  static constexpr int kPitch = NT * 8 + 4;  // floats per row of t
  static constexpr int kPartFloats = kTileRows * kPitch;
  static constexpr int kSmemBytes = (kWarpsK + 1) * kPartFloats * 4;
};

// NT: tiles of 8 ranks (ranks past p.rank are zero); WR: tiles of 16 rows.
template <bool BF16X, int NT, int WR>
__global__ void __launch_bounds__(kLoraThreads, 2) lora_kernel(const LoraParams p) {
  using C = LoraCfg<NT, WR>;
  constexpr int TM = C::kTileRows, WK = C::kWarpsK, RP = C::kPitch;
  extern __shared__ __align__(16) float tsm[];
  float* part = tsm;                          // [WK][TM][RP]
  float* full = tsm + WK * C::kPartFloats;    // [TM][RP]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const int wr = warp % WR, wk = warp / WR;
  const int rank_c = p.ctas > 1 ? (int)cluster_ctarank() : 0;
  const int slot = blockIdx.x / p.ctas;
  pdl_launch_dependents();
  pdl_wait();  // ids (or the plan), X and Y may be written by the preceding kernel

  // the slot-th tile that holds rows: its adapter, and its rows in toks
  __shared__ int toks[TM];
  int adapter = -1, cnt = 0;
  if (p.ids != nullptr) {
    // few rows (one per thread), not grouped yet: a row that has a multiple
    // of TM rows of its adapter before it opens a tile, and tiles count in
    // the order of the rows that open them
    __shared__ __align__(16) int sid[kLoraIdsMax];
    __shared__ int opens[kLoraWarps];
    __shared__ int found[3];  // adapter, first rank, rows
    int id = tid < p.M ? p.ids[tid] : -1;
    if ((unsigned)id >= (unsigned)p.adapters) id = -1;
    sid[tid] = id;
    if (tid < TM) toks[tid] = -1;
    if (tid < 3) found[tid] = tid == 0 ? -1 : 0;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < tid; i += 4) {
      const int4 v = *reinterpret_cast<const int4*>(sid + i);
      before += (v.x == id) + (v.y == id && i + 1 < tid) + (v.z == id && i + 2 < tid) +
                (v.w == id && i + 3 < tid);
    }
    const bool open = id >= 0 && before % TM == 0;
    const unsigned mask = __ballot_sync(0xffffffffu, open);
    if (lane == 0) opens[warp] = __popc(mask);
    __syncthreads();
    int at = __popc(mask & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) at += opens[w];
    if (open && at == slot) {
      found[0] = id;
      found[1] = before;
    }
    __syncthreads();
    adapter = found[0];
    if (adapter < 0) return;  // the whole cluster: a slot past the last tile
    const int r = before - found[1];
    if (id == adapter && (unsigned)r < (unsigned)TM) {
      toks[r] = tid;
      atomicAdd(found + 2, 1);
    }
    __syncthreads();
    cnt = found[2];
  } else {
    int seen = 0, r0 = 0;
    for (int a0 = 0; a0 < p.adapters && adapter < 0; a0 += 32) {
      const int a = a0 + lane;
      int o0 = 0, o1 = 0;
      if (a < p.adapters) {
        o0 = p.offsets[a];
        o1 = p.offsets[a + 1];
        if (o0 < 0 || o1 < o0 || o1 > p.M) o1 = o0 = 0;
      }
      const int t = (o1 - o0 + TM - 1) / TM;
      int incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, seen + incl > slot);
      if (hit) {
        const int src = __ffs(hit) - 1;
        adapter = a0 + src;
        const int first = __shfl_sync(0xffffffffu, seen + incl - t, src);
        r0 = __shfl_sync(0xffffffffu, o0, src) + (slot - first) * TM;
        cnt = min(TM, __shfl_sync(0xffffffffu, o1, src) - r0);
      }
      seen += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (adapter < 0) return;  // the whole cluster: a slot past the last tile
    if (tid < TM) {
      const int m = tid < cnt ? p.rows[r0 + tid] : -1;
      toks[tid] = (unsigned)m < (unsigned)p.M ? m : -1;
    }
    __syncthreads();
  }

  // this lane's two rows of the warp's 16
  const int tok[2] = {toks[wr * 16 + g], toks[wr * 16 + g + 8]};

  // ---- t = A x over this CTA's stretch of K, 32 k per step
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.0f;
  {
    const int nkb = p.K / 32;
    const int kb1 = (int)((long long)nkb * (rank_c + 1) / p.ctas);
    const uint16_t* Aw = p.A + ((size_t)adapter * p.rank + g) * p.K + 8 * c;
    const int nt = p.rank / 8;
    for (int kb = (int)((long long)nkb * rank_c / p.ctas) + wk; kb < kb1; kb += WK) {
      const int k = kb * 32;
      uint4 b[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        b[j] = make_uint4(0, 0, 0, 0);
        if (j < nt) b[j] = __ldg(reinterpret_cast<const uint4*>(Aw + (size_t)(8 * j) * p.K + k));
      }
      // hi and lo words: [row half][k pair]
      uint32_t hi[2][4], lo[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (BF16X) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (tok[h] >= 0)
            v = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.X) +
                                                     (size_t)tok[h] * p.ldx + k + 8 * c));
          hi[h][0] = v.x;
          hi[h][1] = v.y;
          hi[h][2] = v.z;
          hi[h][3] = v.w;
        } else {
          float4 u = make_float4(0.f, 0.f, 0.f, 0.f), v = u;
          if (tok[h] >= 0) {
            const float4* x = reinterpret_cast<const float4*>(
                static_cast<const float*>(p.X) + (size_t)tok[h] * p.ldx + k + 8 * c);
            u = __ldg(x);
            v = __ldg(x + 1);
          }
          split_bf16(u.x, u.y, hi[h][0], lo[h][0]);
          split_bf16(u.z, u.w, hi[h][1], lo[h][1]);
          split_bf16(v.x, v.y, hi[h][2], lo[h][2]);
          split_bf16(v.z, v.w, hi[h][3], lo[h][3]);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if (j >= nt) continue;
        mma_bf16(acc[j], hi[0][0], hi[1][0], hi[0][1], hi[1][1], b[j].x, b[j].y);
        mma_bf16(acc[j], hi[0][2], hi[1][2], hi[0][3], hi[1][3], b[j].z, b[j].w);
        if constexpr (!BF16X) {
          mma_bf16(acc[j], lo[0][0], lo[1][0], lo[0][1], lo[1][1], b[j].x, b[j].y);
          mma_bf16(acc[j], lo[0][2], lo[1][2], lo[0][3], lo[1][3], b[j].z, b[j].w);
        }
      }
    }
  }
  {
    float* mine = part + wk * C::kPartFloats + (wr * 16 + g) * RP + 2 * c;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      *reinterpret_cast<float2*>(mine + 8 * j) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(mine + 8 * RP + 8 * j) = make_float2(acc[j][2], acc[j][3]);
    }
  }
  __syncthreads();
  // sums over the warps' stretches of K, then over the cluster's, each in a
  // fixed order; ranks past p.rank and rows past cnt are zero already
  const float s = p.scale != nullptr ? __ldg(p.scale + adapter) : 1.0f;
  for (int i = tid; i < TM * NT * 8; i += kLoraThreads) {
    const int at = i / (NT * 8) * RP + i % (NT * 8);
    float v = part[at];
#pragma unroll
    for (int w = 1; w < WK; ++w) v += part[w * C::kPartFloats + at];
    if (p.ctas > 1)
      part[at] = v;
    else
      full[at] = v * s;
  }
  if (p.ctas > 1) {
    cluster_sync_all();
    for (int i = tid; i < TM * NT * 8; i += kLoraThreads) {
      const int r = i / (NT * 8), at = r * RP + i % (NT * 8);
      float v = 0.0f;
      if (r < cnt)
        for (int q = 0; q < p.ctas; ++q)
          v += __int_as_float(dsmem_ld_s32(dsmem_map(smem_u32(part + at), q)));
      full[at] = v * s;
    }
    cluster_arrive();  // this CTA has read its peers' sums
  }
  __syncthreads();

  // ---- Y += t B^T over this CTA's stretch of N, 32 columns per step
  constexpr int KW = NT == 2 ? 4 : 8;   // adjacent ranks per lane
  constexpr int NB = NT * 8 / (4 * KW); // rank blocks
  uint32_t th[NB][2][KW / 2], tl[NB][2][KW / 2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < KW / 2; ++i) {
        const float2 v = *reinterpret_cast<const float2*>(
            full + (wr * 16 + g + 8 * h) * RP + b * 4 * KW + KW * c + 2 * i);
        split_bf16(v.x, v.y, th[b][h][i], tl[b][h][i]);
      }
  const int slices = (p.N + 31) / 32;
  const int parts = p.ctas * gridDim.y, my = blockIdx.y * p.ctas + rank_c;
  const int s1 = (int)((long long)slices * (my + 1) / parts);
  const uint16_t* Bw = p.B + (size_t)adapter * p.N * p.rank + KW * c;
  const int jcol = (g >> 1) * 8 + (g & 1);  // + 2 q: the column of MMA column g, n tile q
  for (int sl = (int)((long long)slices * my / parts) + wk; sl < s1; sl += WK) {
    const int n = sl * 32, col = n + 8 * c;
    uint16_t* yp[2];
    uint4 y[2];
    const bool whole = p.y_vec && col + 8 <= p.N;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      yp[h] = p.Y + (size_t)(tok[h] < 0 ? 0 : tok[h]) * p.ldy + col;
      y[h] = make_uint4(0, 0, 0, 0);
      if (tok[h] >= 0) {
        if (whole) {
          y[h] = *reinterpret_cast<const uint4*>(yp[h]);
        } else {
          uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < p.N) w[i / 2] |= (uint32_t)yp[h][i] << (16 * (i & 1));
          y[h] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    float d[4][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {y[h].x, y[h].y, y[h].z, y[h].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        d[q][2 * h] = __uint_as_float(w[q] << 16);
        d[q][2 * h + 1] = __uint_as_float(w[q] & 0xffff0000u);
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool in = b * 4 * KW + KW * c < p.rank;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int bc = n + jcol + 2 * q;
        uint32_t w[KW / 2];
        const uint16_t* src = Bw + (size_t)bc * p.rank + b * 4 * KW;
        if constexpr (KW == 8) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (in && bc < p.N) v = __ldg(reinterpret_cast<const uint4*>(src));
          w[0] = v.x;
          w[1] = v.y;
          w[2] = v.z;
          w[3] = v.w;
        } else {
          uint2 v = make_uint2(0, 0);
          if (in && bc < p.N) v = __ldg(reinterpret_cast<const uint2*>(src));
          w[0] = v.x;
          w[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < KW / 2; i += 2) {
          mma_bf16(d[q], th[b][0][i], th[b][1][i], th[b][0][i + 1], th[b][1][i + 1], w[i],
                   w[i + 1]);
          mma_bf16(d[q], tl[b][0][i], tl[b][1][i], tl[b][0][i + 1], tl[b][1][i + 1], w[i],
                   w[i + 1]);
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (tok[h] < 0) continue;
      const uint32_t w[4] = {pack_bf16(d[0][2 * h], d[0][2 * h + 1]),
                             pack_bf16(d[1][2 * h], d[1][2 * h + 1]),
                             pack_bf16(d[2][2 * h], d[2][2 * h + 1]),
                             pack_bf16(d[3][2 * h], d[3][2 * h + 1])};
      if (whole) {
        *reinterpret_cast<uint4*>(yp[h]) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < p.N) yp[h][i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
      }
    }
  }
  if (p.ctas > 1) cluster_wait();  // nobody still reads this CTA's sums
}

}  // namespace w4a8
