// Joins the partial results of attention over a paged cache. Every partial of
// a row is (O unnormalised, m, l) of some of its keys:
//
//   M = max m_s, O = sum_s 2^(m_s - M) O_s / L, L = sum_s 2^(m_s - M) l_s,
//   LSE = (M + log2 L) ln 2
//
// One, four or eight warps per output row, each for every W-th partial.
// Which work ranges hold a row's partials follows from the same arithmetic on
// the work line as in the attention kernel; rows
// that one worker finished by itself are left alone, and a row without keys gets
// O = 0, LSE = -inf. The order of the sum is fixed: the result does not depend
// on timing.
#include <cstdint>
#include <math_constants.h>

#include "kv_work.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace fa {

namespace {

struct Partials {
  int ca;             // first range that holds a part, of n
  int ua;             // first unit of the item
  int whole;          // slot of an item that one worker holds
  int n;
  int ranges, U;      // the line it is on
};

__device__ __forceinline__ Partials partials_of(int ua, int units, int ranges, int U, int whole) {
  Partials q{0, ua, whole, 0, min(ranges, U), U};
  if (units == 0 || U == 0) return q;
  q.ca = range_of(ua, q.ranges, U);
  q.n = range_of(ua + units - 1, q.ranges, U) - q.ca + 1;
  return q;
}
// in units of Hk slots
__device__ __forceinline__ int slot_of(const Partials& q, int i) {
  if (q.n == 1) return q.whole;
  const int c = q.ca + i;
  return 2 * c + (range_start(c, q.ranges, q.U) >= q.ua ? 0 : 1);
}

// W warps a row; with one, a CTA takes four rows.
template <int D, int W>
__global__ void __launch_bounds__(W == 1 ? 128 : 32 * W) kv_merge_kernel(const __grid_constant__ KvMergeParams mp) {
  constexpr int V = D / 32;   // elements of a lane
  __shared__ float part[W][D], stat[W][2];
  const KvAttnParams& p = mp.p;
  const int64_t row = W == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  const int warp = W == 1 ? 0 : threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = (int)(row / p.Hq), h = (int)(row - (int64_t)t * p.Hq);
  const int b = t < p.s.total ? seq_of_row(p.s, t) : -1;
  SeqWork w;
  w.bad = true;
  if (b >= 0) w = seq_work(p, b, mp.own.rt, mp.own.unit);
  // What follows reads what the attention kernels wrote. Every thread waits,
  // those with nothing to do too: this kernel must not end before those.
  wait_for_predecessor();
  if (w.bad || t < w.first || t >= w.first + w.n) return;
  const int hk = h / p.G, gq = h - hk * p.G;
  // (plain loads: the kernel before wrote it, perhaps while this one was resident)
  const int own_U = p.cum[p.s.B];

  Partials own, pre{0, 0, 0, 0, 0, 0};
  int own_r, pre_r = 0;
  {
    const int rt = mp.own.rt;
    const int R = (t - w.first) * p.G + gq;
    const int mt = R / rt;
    own_r = R - mt * rt;
    own = partials_of(mp.own.pre_total + p.cum[b] + mt * w.units, w.units, mp.own.ranges, mp.own.pre_total + own_U,
                      mp.own.whole + whole_slot(p, rt, b, w.first, mt));
    if (own.n == 1 && p.prefix_tiles == 0) return;   // finished by the worker that had all of it
  }
  if (p.prefix_tiles > 0) {
    const int rt = mp.pre.rt;
    const int R = t * p.G + gq;
    const int mt = R / rt;
    const int units = (p.prefix_len + mp.pre.unit - 1) / mp.pre.unit;
    pre_r = R - mt * rt;
    pre = partials_of(mt * units, units, mp.pre.ranges, mp.pre.pre_total + (mp.pre.own ? own_U : 0), mp.pre.whole + mt);
  }
  if (own.n == 0 && w.units > 0) return;   // the line was not worked through (scan_units)
  const int n = own.n + pre.n;
  // row of partial i in its launch's part of the workspace
  auto at = [&](int i) -> int64_t {
    return i < pre.n ? ((int64_t)slot_of(pre, i) * p.Hk + hk) * mp.pre.rt + pre_r
                     : ((int64_t)slot_of(own, i - pre.n) * p.Hk + hk) * mp.own.rt + own_r;
  };
  // each warp joins every W-th partial, 32 at a time: lane i has the (m, l) and
  // row of partial i0 + W i
  float M = -CUDART_INF_F, L = 0.f;
  float acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  for (int i0 = warp; i0 < n; i0 += 32 * W) {
    const int mine = i0 + W * lane;
    int64_t r = 0;
    float2 ml = make_float2(-CUDART_INF_F, 0.f);
    if (mine < n) {
      r = at(mine);
      ml = *reinterpret_cast<const float2*>((mine < pre.n ? mp.pre.ml : mp.own.ml) + 2 * r);
    }
    float x = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (x > M) {
      const float f = M == -CUDART_INF_F ? 0.f : ptx::ex2(M - x);
      L *= f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] *= f;
      M = x;
    }
    const float wgt = ml.y == 0.f ? 0.f : ml.x == M ? 1.f : ptx::ex2(ml.x - M);
    const int top = min(32, (n - i0 + W - 1) / W);
#pragma unroll 4
    for (int k = 0; k < top; ++k) {
      const float f = __shfl_sync(0xffffffffu, wgt, k), lk = __shfl_sync(0xffffffffu, ml.y, k);
      const int64_t rk = __shfl_sync(0xffffffffu, r, k);
      if (lk == 0.f) continue;
      const float* src = (i0 + W * k < pre.n ? mp.pre.o : mp.own.o) + rk * D;
      L = fmaf(f, lk, L);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const float2 v = *reinterpret_cast<const float2*>(src + 2 * lane + 64 * j);
        acc[2 * j] = fmaf(f, v.x, acc[2 * j]);
        acc[2 * j + 1] = fmaf(f, v.y, acc[2 * j + 1]);
      }
    }
  }
  uint16_t* const o = static_cast<uint16_t*>(p.o) + row * D;
  if constexpr (W == 1) {
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float x0 = acc[2 * j] * inv, x1 = acc[2 * j + 1] * inv;
      *reinterpret_cast<uint32_t*>(o + 2 * lane + 64 * j) = p.q_bf16 ? ptx::pack_bf16(x0, x1) : ptx::pack_f16(x0, x1);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      part[warp][2 * lane + 64 * j] = acc[2 * j];
      part[warp][2 * lane + 64 * j + 1] = acc[2 * j + 1];
    }
    if (lane == 0) {
      stat[warp][0] = M;
      stat[warp][1] = L;
    }
    __syncthreads();
    // and the warps' results are joined in their order
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, stat[w][0]);
    L = 0.f;
    float fw[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float l = stat[w][1];
      fw[w] = l == 0.f ? 0.f : stat[w][0] == M ? 1.f : ptx::ex2(stat[w][0] - M);
      L += fw[w] * l;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    for (int e = 2 * threadIdx.x; e < D; e += 64 * W) {
      float x[2] = {0.f, 0.f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (stat[w][1] == 0.f) continue;
        x[0] = fmaf(fw[w], part[w][e], x[0]);
        x[1] = fmaf(fw[w], part[w][e + 1], x[1]);
      }
      x[0] *= inv;
      x[1] *= inv;
      *reinterpret_cast<uint32_t*>(o + e) = p.q_bf16 ? ptx::pack_bf16(x[0], x[1]) : ptx::pack_f16(x[0], x[1]);
    }
  }
  if (warp == 0 && lane == 0) {
    const float lse = L == 0.f ? -CUDART_INF_F : (M + __log2f(L)) * kLn2;
    if (p.s.cu != nullptr)
      p.lse[(int64_t)h * p.s.total + t] = lse;
    else
      p.lse[((int64_t)b * p.Hq + h) * p.s.S + (t - w.first)] = lse;
  }
}

}  // namespace

cudaError_t launch_kv_merge(const KvMergeParams& m, int D, cudaStream_t stream) {
  const int64_t rows = (int64_t)m.p.s.total * m.p.Hq;
  if (rows == 0) return cudaSuccess;
  if (rows > 0x7fffffff) return cudaErrorInvalidValue;
  // Eight warps a row where few rows leave the machine empty and have many
  // partials each; one where there are so many rows that the CTAs' starts count.
  // Whole calls, e4m3, 32 query and 8 K/V heads of 128, one, four and eight
  // warps: 32 rows (8192 keys) 61.0, 27.9, 16.7 us; 256 rows 30.4, 23.5, 22.1; 512
  // rows 21.3, 18.6, 17.8; 1024 rows 24.1, 22.6, 25.7; 1536 rows 34.9, 36.2, 39.5;
  // 2048 rows 117.4, 119.2, 124.9; 8192 rows 96.2, 107.7, 128.4; 32000 rows (up to
  // 30 keys) 42.3, 72.2, 118.5. Heads of 256: 512 rows 65.7, 63.0, 62.1; 1152 rows
  // 124.2, 122.4, 125.4; 1536 rows 157.2, 157.9, 161.8; 8192 rows 165.7, 176.2,
  // 195.2. Heads of 64: 1536 rows 25.3, 24.7, 28.1; 8192 rows 64.1, 73.9, 90.4.
  auto run = [&](auto one, auto four, auto eight) {
    if (rows >= 1536) return launch_early(one, (int)((rows + 3) / 4), 128, 0, stream, true, m);
    return rows > 512 ? launch_early(four, (int)rows, 128, 0, stream, true, m)
                      : launch_early(eight, (int)rows, 256, 0, stream, true, m);
  };
  if (D == 64) return run(kv_merge_kernel<64, 1>, kv_merge_kernel<64, 4>, kv_merge_kernel<64, 8>);
  if (D == 128) return run(kv_merge_kernel<128, 1>, kv_merge_kernel<128, 4>, kv_merge_kernel<128, 8>);
  return run(kv_merge_kernel<256, 1>, kv_merge_kernel<256, 4>, kv_merge_kernel<256, 8>);
}

}  // namespace fa
