// The paged K/V cache: quantised as it is written (append) and read back.
//
// Append. A row is one token of one K/V head, D elements of K or of V:
//   scale = max(amax / M, 2^-126), M = 448 (e4m3) or 127 (int8),
//   code  = round(x * (1 / scale)), to nearest even.
// The scale's floor keeps its reciprocal finite; a row of zeros gets codes 0.
// A row that holds an infinity or a NaN gets scale NaN and codes 0, so every
// element of it reads back as NaN and the codes themselves stay finite (the
// attention kernels rely on that: a masked row's codes meet a zero weight).
// One scale per row lets a token be appended without touching earlier rows.
// Every step is one correctly rounded fp32 operation, so the codes are the
// same wherever they are computed. 16-bit caches take the bits as they are.
//
// Read. x = code * scale in fp32, rounded once to the output type.
//
// Both are HBM-bound and move every element once; what has to be kept small is
// the instructions per element. D / 16 lanes own a row, each two chunks of
// eight elements, half a row apart, so that every access of a warp covers
// whole lines; the row's amax is two to four shuffles, and the scale and its
// reciprocal are worked out once per sixteen elements. A group of lanes stays
// with one head of K or V and walks down the CTA's tokens, four loads ahead of
// their use. One thread per token finds its sequence, position and page first.
// Four CTAs per SM (at most 64 registers) rather than three: append 142 -> 128 us.
// Measured: 32 prompts of 128 .. 8192 tokens, 8 heads of 128: append from bf16
// to int8 128 us, 6.3 TB/s, 93 % of a copy's rate; read from e4m3 to bf16
// 122 us, 6.6 TB/s, 97 %.
#include <cstdint>

#include "kv_codes.cuh"
#include "kv_internal.h"
#include "ptx.cuh"

namespace fa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 16;   // tokens of a CTA

// Row of the cache (page * page_size + offset) of row t, -1 where nothing is to
// be done, -2 for a bad page entry. `append`: the rows are the last of their
// sequence's seqlens_k keys (positions below 0 are padding and skipped);
// otherwise row i of a sequence is its position i.
__device__ __forceinline__ int64_t cache_row(const PagedSeqs& s, int t, bool append) {
  const int b = seq_of_row(s, t);
  if (b < 0) return -1;
  int first, n;
  const int len = __ldg(s.seqlens_k + b);
  if (!seq_rows(s, b, first, n) || len < 0 || (int64_t)len > (int64_t)s.max_pages * s.page_size ||
      (!append && n > len)) {
    atomicOr(s.status, kDevBadSeqlens);
    return -1;
  }
  const int i = t - first;
  if (i < 0 || i >= n) return -1;
  const int pos = append ? len - n + i : i;
  if (pos < 0) return -1;
  int index, offset;
  page_of(s, pos, index, offset);
  const int page = __ldg(s.block_table + (int64_t)b * s.max_pages + index);
  if (page < 0 || page >= s.num_pages) {
    atomicOr(s.status, kDevBadSeqlens);
    return -2;
  }
  return (int64_t)page * s.page_size + offset;
}

// a packed sequence whose bounds are broken is reported even if none of its
// rows is found
__device__ __forceinline__ void report_bad(const PagedSeqs& s) {
  if (s.cu == nullptr || blockIdx.x != 0) return;
  for (int b = threadIdx.x; b < s.B; b += kThreads) {
    int first, n;
    if (!seq_rows(s, b, first, n)) atomicOr(s.status, kDevBadSeqlens);
  }
}

// One row's sixteen elements of this lane -> codes (2 x 8 bytes) and the scale.
template <int KIND, bool BF16, int L>
__device__ __forceinline__ float quantise(const uint4 (&v)[2], uint2 (&c)[2]) {
  // the largest magnitude, as bits: orders finite < infinity < NaN
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                               __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu)));
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const bool bad = m >= (BF16 ? 0x7f80u : 0x7c00u);
  const float amax = unpack2<BF16>(m).x;
  const float scale = fmaxf(__fdiv_rn(amax, KIND == kCacheE4M3 ? 448.f : 127.f), 0x1p-126f);
  const float inv = __frcp_rn(scale);
  const uint64_t inv2 = ptx::f2pack(inv, inv);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t r[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
    uint32_t out[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 a = unpack2<BF16>(r[2 * j]), b = unpack2<BF16>(r[2 * j + 1]);
      float x0, x1, x2, x3;
      ptx::f2unpack(ptx::mul2(ptx::f2pack(a.x, a.y), inv2), x0, x1);
      ptx::f2unpack(ptx::mul2(ptx::f2pack(b.x, b.y), inv2), x2, x3);
      if (KIND == kCacheE4M3) {
        out[j] = ptx::pack_e4m3x4(x0, x1, x2, x3);
      } else {
        // adding 1.5 2^23 rounds to an integer (to nearest even), whose low
        // byte is the code
        const float k = 12582912.f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(x0, k)), __float_as_uint(__fadd_rn(x1, k)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(x2, k)), __float_as_uint(__fadd_rn(x3, k)), 0x0040);
        out[j] = __byte_perm(lo, hi, 0x5410);
      }
      if (bad) out[j] = 0;
    }
    c[i] = make_uint2(out[0], out[1]);
  }
  return bad ? __uint_as_float(0x7fffffffu) : scale;
}

// sixteen codes -> sixteen 16-bit elements
template <int KIND, bool BF16>
__device__ __forceinline__ void dequantise(const uint2 (&c)[2], float scale, uint4 (&v)[2]) {
  const uint64_t s2 = ptx::f2pack(scale, scale);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t cw[2] = {c[i].x, c[i].y};
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t lo, hi;   // f16 pairs, exact
      codes_to_f16<KIND>(cw[j], lo, hi);
      const float2 a = unpack2<false>(lo), b = unpack2<false>(hi);
      float x0, x1, x2, x3;
      ptx::f2unpack(ptx::mul2(ptx::f2pack(a.x, a.y), s2), x0, x1);
      ptx::f2unpack(ptx::mul2(ptx::f2pack(b.x, b.y), s2), x2, x3);
      out[2 * j] = BF16 ? ptx::pack_bf16(x0, x1) : ptx::pack_f16(x0, x1);
      out[2 * j + 1] = BF16 ? ptx::pack_bf16(x2, x3) : ptx::pack_f16(x2, x3);
    }
    v[i] = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

// APPEND: rows -> pages; else pages -> rows. 16-bit caches: the bits as they are.
template <int KIND, bool BF16, int D, bool APPEND>
__global__ void __launch_bounds__(kThreads, 4) kv_move_kernel(const __grid_constant__ CacheParams p, int tokens) {
  constexpr int L = D / 16;                   // lanes of a row
  constexpr int GROUPS = kThreads / L;
  constexpr int AHEAD = 4;                    // rows loaded before the first is used
  constexpr bool k8 = cache_is_8bit(KIND);
  __shared__ int64_t rows[kMaxTokens];        // row of the cache, -1: nothing to do, -2: bad page
  __shared__ int64_t srow[kMaxTokens];        // element of the scales, for head 0
  const int t0 = blockIdx.x * tokens;
  const int nt = min(tokens, p.s.total - t0);
  if ((int)threadIdx.x < nt) {
    const int64_t row = cache_row(p.s, t0 + threadIdx.x, APPEND);
    rows[threadIdx.x] = row;
    if (k8 && row >= 0) {
      const int64_t page = row / p.s.page_size;
      srow[threadIdx.x] = page * p.H * p.s.page_size + (row - page * p.s.page_size);
    }
  }
  report_bad(p.s);
  __syncthreads();
  const int group = threadIdx.x / L, u = threadIdx.x % L;
  const int combos = 2 * p.H;                 // heads of K, then of V
  const int par = combos < GROUPS ? GROUPS / combos : 1;   // tokens side by side
  const int tg = group / combos;              // this group's token among them (combos >= GROUPS: 0)
  // every lane of a warp makes the same turns in both loops (the shuffles)
  for (int base = 0; base < combos; base += GROUPS) {
    const int combo = combos < GROUPS ? group - tg * combos : base + group;
    const bool mine = tg < par && combo < combos;
    const int hw = mine ? combo : 0;
    const int w = hw >= p.H ? 1 : 0, h = hw - w * p.H;
    uint16_t* const x = static_cast<uint16_t*>(p.x[w]) + (int64_t)t0 * p.xs_t[w] + (int64_t)h * p.xs_h[w] + 8 * u;
    uint8_t* const pages = static_cast<uint8_t*>(p.pages[w]) + ((int64_t)h * D + 8 * u) * (k8 ? 1 : 2);
    float* const scales = k8 ? p.scale[w] + (int64_t)h * p.s.page_size : nullptr;
    for (int t = 0; t < nt; t += par * AHEAD) {
      uint4 v[AHEAD][2];
      uint2 c[AHEAD][2];
      float sc[AHEAD];
      int64_t row[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        const int tt = t + i * par + tg;
        row[i] = mine && tt < nt ? rows[tt] : -1;
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        c[i][0] = c[i][1] = make_uint2(0, 0);
        sc[i] = 0.f;
        if (row[i] < 0) continue;
        if (APPEND) {
          const uint16_t* src = x + tt * p.xs_t[w];
          v[i][0] = *reinterpret_cast<const uint4*>(src);
          v[i][1] = *reinterpret_cast<const uint4*>(src + D / 2);
        } else if (k8) {
          const uint8_t* src = pages + row[i] * p.H * D;
          c[i][0] = *reinterpret_cast<const uint2*>(src);
          c[i][1] = *reinterpret_cast<const uint2*>(src + D / 2);
          sc[i] = scales[srow[tt]];
        } else {
          const uint16_t* src = reinterpret_cast<const uint16_t*>(pages) + row[i] * p.H * D;
          v[i][0] = *reinterpret_cast<const uint4*>(src);
          v[i][1] = *reinterpret_cast<const uint4*>(src + D / 2);
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (t + i * par >= nt) break;
        const int tt = t + i * par + tg;
        if (APPEND) {
          if (k8) {
            const float scale = quantise<KIND, BF16, L>(v[i], c[i]);
            if (row[i] >= 0) {
              uint8_t* dst = pages + row[i] * p.H * D;
              *reinterpret_cast<uint2*>(dst) = c[i][0];
              *reinterpret_cast<uint2*>(dst + D / 2) = c[i][1];
              if (u == 0) scales[srow[tt]] = scale;
            }
          } else if (row[i] >= 0) {
            uint16_t* dst = reinterpret_cast<uint16_t*>(pages) + row[i] * p.H * D;
            *reinterpret_cast<uint4*>(dst) = v[i][0];
            *reinterpret_cast<uint4*>(dst + D / 2) = v[i][1];
          }
        } else if (row[i] != -1) {   // a bad page reads as zeros
          if (k8) dequantise<KIND, BF16>(c[i], sc[i], v[i]);
          uint16_t* dst = x + tt * p.xs_t[w];
          *reinterpret_cast<uint4*>(dst) = v[i][0];
          *reinterpret_cast<uint4*>(dst + D / 2) = v[i][1];
        }
      }
    }
  }
}

int tokens_per_cta(int total, int num_sms) {
  int t = total / (4 * (num_sms > 0 ? num_sms : 1));
  return t < 1 ? 1 : (t > kMaxTokens ? kMaxTokens : t);
}

template <bool APPEND, int KIND, bool BF16>
cudaError_t launch_move_d(const CacheParams& p, int num_sms, cudaStream_t stream) {
  if (p.s.total == 0) return cudaSuccess;
  const int tokens = tokens_per_cta(p.s.total, num_sms);
  const unsigned grid = (unsigned)(((int64_t)p.s.total + tokens - 1) / tokens);
  auto run = [&](auto kern) { kern<<<grid, kThreads, 0, stream>>>(p, tokens); };
  if (p.D == 64) run(kv_move_kernel<KIND, BF16, 64, APPEND>);
  else if (p.D == 128) run(kv_move_kernel<KIND, BF16, 128, APPEND>);
  else run(kv_move_kernel<KIND, BF16, 256, APPEND>);
  return cudaGetLastError();
}
template <bool APPEND>
cudaError_t launch_move(const CacheParams& p, int kind, bool bf16, int num_sms, cudaStream_t stream) {
  if (kind == kCacheE4M3)
    return bf16 ? launch_move_d<APPEND, kCacheE4M3, true>(p, num_sms, stream)
                : launch_move_d<APPEND, kCacheE4M3, false>(p, num_sms, stream);
  if (kind == kCacheI8)
    return bf16 ? launch_move_d<APPEND, kCacheI8, true>(p, num_sms, stream)
                : launch_move_d<APPEND, kCacheI8, false>(p, num_sms, stream);
  return launch_move_d<APPEND, kCacheF16, false>(p, num_sms, stream);
}

}  // namespace

cudaError_t launch_kv_append(const CacheParams& p, int kind, bool bf16, int num_sms, cudaStream_t stream) {
  return launch_move<true>(p, kind, bf16, num_sms, stream);
}
cudaError_t launch_kv_read(const CacheParams& p, int kind, bool bf16, int num_sms, cudaStream_t stream) {
  return launch_move<false>(p, kind, bf16, num_sms, stream);
}

}  // namespace fa
