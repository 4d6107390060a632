// Rotary positions with several axes (time, height, width, ...), forward and
// backward, of a query and a key tensor in one launch.
//
// Pair j of a head holds two elements (a, b); axis x(j) gives its position
// p = positions[x(j), t] and w_j its frequency, phi = p w_j:
//
//   a' = a cos phi - b sin phi,   b' = b cos phi + a sin phi
//
// The map is orthogonal, so the backward pass is the same kernel with -phi.
// Elements past rot_dim pass through.
//
// The angle is reduced in integers: the host gives w_j / 2 pi as a 64-bit binary
// fraction of a turn, rounded once, and the integer product p * fraction,
// modulo 2^64, is the fraction of a turn left after all whole turns are dropped.
// A position of 2^31 leaves an error of 2^-34 turns from the fraction's rounding;
// an fp32 product would be off by whole radians there. sincospif takes the upper
// 32 bits, which drops less than 2^-32 turns.
//
// HBM-bound: every element is read once and written once, 2 * 2 bytes. A CTA
// takes a few tokens, computes their sines and cosines once into shared
// memory (they are the same for every head), then streams all heads of these
// tokens, 32 bytes at a time in two 16-byte accesses (with 16 bytes T = 16383,
// 32 heads of 80 took 35 us, with 32 it takes 32). Measured: T = 32768, 40
// heads of 128: 102 us, 6.6 TB/s, 96 % of a copy's rate.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_codes.cuh"
#include "kv_internal.h"

namespace fa {

namespace {

constexpr int kRopeThreads = 256;

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (BF16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <bool BF16>
__device__ __forceinline__ float load1(const uint16_t* p) {
  return BF16 ? __uint_as_float((uint32_t)*p << 16) : __half2float(*reinterpret_cast<const __half*>(p));
}
template <bool BF16>
__device__ __forceinline__ uint16_t store1(float x) {
  if (BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return __half_as_ushort(__float2half_rn(x));
}

// (a, b) -> (a cos - b sin, b cos + a sin); one product of each sum is rounded,
// then the sum, all in fp32
__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = fmaf(a, cs.x, -(b * cs.y));
  b = fmaf(b, cs.x, a * cs.y);
  a = x;
}

// VEC: 16-byte accesses; a unit is 8 pairs (half layout: 8 elements of each
// half; interleaved: 16 adjacent elements, the last unit perhaps 8) or 8
// elements that pass through. Otherwise a unit is one pair or one element, for
// widths, strides and addresses that 16 bytes do not divide.
template <bool BF16, bool VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p, int tokens) {
  extern __shared__ float2 cs[];   // [tokens][rot_dim / 2]
  __shared__ uint64_t freq[kRopeMaxPairs];
  __shared__ int axis[kRopeMaxPairs];
  const int half = p.rot / 2;
  if ((int)threadIdx.x < half) {
    freq[threadIdx.x] = p.freq[threadIdx.x];
    axis[threadIdx.x] = p.axis[threadIdx.x];
  }
  __syncthreads();
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, p.T - t0);
  for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
    const int t = i / half, j = i - t * half;
    const int pos = __ldg(p.pos + (int64_t)axis[j] * p.T + t0 + t);
    const uint64_t turns = (uint64_t)(int64_t)pos * freq[j];
    // upper 32 bits as a signed fraction: [-1/2, 1/2) of a turn = [-1, 1) half turns
    const float x = (float)(int32_t)(uint32_t)(turns >> 32) * 0x1p-31f;
    float s, c;
    sincospif(x, &s, &c);
    cs[i] = make_float2(c, p.inverse ? -s : s);
  }
  __syncthreads();

  const int rot_units = VEC ? (INTERLEAVED ? (p.rot + 15) / 16 : half / 8) : half;
  const int U = rot_units + (VEC ? (p.D - p.rot) / 8 : p.D - p.rot);   // units of one head
  const int HH = p.H[0] + p.H[1];
  const int n = nt * HH * U;
  // unit i of this CTA: where it is read and written, and its sines and cosines
  struct Unit {
    const uint16_t* src;
    uint16_t* dst;
    const float2* c;
    int u;
    bool skip;   // passes through and is there already
  };
  auto unit = [&](int i) {
    Unit x;
    const int row = i / U;
    x.u = i - row * U;
    const int t = row / HH;
    int h = row - t * HH;
    // q or k: selected, not indexed (an index that varies by thread makes a
    // parameter read serial: T = 32768, 40 heads of 128, 104 us against 102)
    const bool k = h >= p.H[0];
    if (k) h -= p.H[0];
    const int64_t tt = t0 + t;
    x.src = static_cast<const uint16_t*>(k ? p.x[1] : p.x[0]) + tt * (k ? p.xs_t[1] : p.xs_t[0]) +
            h * (k ? p.xs_h[1] : p.xs_h[0]);
    x.dst = static_cast<uint16_t*>(k ? p.y[1] : p.y[0]) + tt * (k ? p.ys_t[1] : p.ys_t[0]) +
            h * (k ? p.ys_h[1] : p.ys_h[0]);
    x.c = cs + t * half;
    x.skip = x.u >= rot_units && (k ? p.in_place[1] : p.in_place[0]);
    return x;
  };
  // one unit at a time at 32 registers a thread beat two and four at a time at
  // 48 and 71: T = 32768, 40 heads of 128, 104 us against 111 and 130
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kRopeThreads) {
    const Unit x = unit(i);
    if (x.skip) continue;
    const int u = x.u;
    if (VEC) {
      if (u >= rot_units) {
        const int e = p.rot + 8 * (u - rot_units);
        *reinterpret_cast<uint4*>(x.dst + e) = *reinterpret_cast<const uint4*>(x.src + e);
      } else if (INTERLEAVED) {
        uint4 v[2];
        const bool both = 16 * u + 8 < p.rot;
        v[0] = *reinterpret_cast<const uint4*>(x.src + 16 * u);
        if (both) v[1] = *reinterpret_cast<const uint4*>(x.src + 16 * u + 8);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          uint32_t* r = reinterpret_cast<uint32_t*>(&v[a]);
          if (a == 1 && !both) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float2 f = unpack2<BF16>(r[j]);
            rotate(f.x, f.y, x.c[8 * u + 4 * a + j]);
            r[j] = pack2<BF16>(f.x, f.y);
          }
          *reinterpret_cast<uint4*>(x.dst + 16 * u + 8 * a) = v[a];
        }
      } else {
        uint4 va = *reinterpret_cast<const uint4*>(x.src + 8 * u);
        uint4 vb = *reinterpret_cast<const uint4*>(x.src + half + 8 * u);
        uint32_t* ra = reinterpret_cast<uint32_t*>(&va);
        uint32_t* rb = reinterpret_cast<uint32_t*>(&vb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 a = unpack2<BF16>(ra[j]), b = unpack2<BF16>(rb[j]);
          const float4 c2 = *reinterpret_cast<const float4*>(x.c + 8 * u + 2 * j);
          rotate(a.x, b.x, make_float2(c2.x, c2.y));
          rotate(a.y, b.y, make_float2(c2.z, c2.w));
          ra[j] = pack2<BF16>(a.x, a.y);
          rb[j] = pack2<BF16>(b.x, b.y);
        }
        *reinterpret_cast<uint4*>(x.dst + 8 * u) = va;
        *reinterpret_cast<uint4*>(x.dst + half + 8 * u) = vb;
      }
    } else {
      if (u >= rot_units) {
        const int e = p.rot + u - rot_units;
        x.dst[e] = x.src[e];
      } else {
        const int ea = INTERLEAVED ? 2 * u : u, eb = INTERLEAVED ? 2 * u + 1 : half + u;
        float a = load1<BF16>(x.src + ea), b = load1<BF16>(x.src + eb);
        rotate(a, b, x.c[u]);
        x.dst[ea] = store1<BF16>(a);
        x.dst[eb] = store1<BF16>(b);
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, int num_sms, cudaStream_t stream) {
  if (p.T == 0 || p.H[0] + p.H[1] == 0) return cudaSuccess;
  const int half = p.rot / 2;
  bool vec = p.D % 8 == 0 && (interleaved ? p.rot % 8 == 0 : half % 8 == 0);
  for (int w = 0; w < 2; ++w) {
    if (p.H[w] == 0) continue;
    for (int64_t s : {p.xs_t[w], p.xs_h[w], p.ys_t[w], p.ys_h[w]}) vec = vec && s % 8 == 0;
    for (const void* a : {p.x[w], (const void*)p.y[w]}) vec = vec && (reinterpret_cast<uintptr_t>(a) & 15u) == 0;
  }
  // tokens of a CTA: as many as leave about eight CTAs per SM, at most 4
  int tokens = p.T / (8 * (num_sms > 0 ? num_sms : 1));
  tokens = tokens < 1 ? 1 : (tokens > 4 ? 4 : tokens);
  const unsigned grid = (unsigned)(((int64_t)p.T + tokens - 1) / tokens);
  const size_t smem = (size_t)tokens * half * sizeof(float2);
  auto run = [&](auto kern) { kern<<<grid, kRopeThreads, smem, stream>>>(p, tokens); };
  if (bf16) {
    if (vec) interleaved ? run(rope_kernel<true, true, true>) : run(rope_kernel<true, true, false>);
    else interleaved ? run(rope_kernel<true, false, true>) : run(rope_kernel<true, false, false>);
  } else {
    if (vec) interleaved ? run(rope_kernel<false, true, true>) : run(rope_kernel<false, true, false>);
    else interleaved ? run(rope_kernel<false, false, true>) : run(rope_kernel<false, false, false>);
  }
  return cudaGetLastError();
}

}  // namespace fa
