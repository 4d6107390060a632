// The work line of the attention kernels over a paged cache: how the keys of
// all sequences are cut into units and handed to the CTAs, and where partial
// results go. The merge kernel repeats the same arithmetic.
//
// An item is (sequence, tile of rt rows), or, for the shared prefix, a tile of
// the rows of all sequences. Its keys are cut into units; the units of all
// items form one line (prefix first), and range r of n is the units [r U / n,
// (r + 1) U / n): every range the same, whatever the lengths. A worker (a warp,
// or a CTA) takes one range for one K/V head, and the workers of a range's
// heads sit side by side: a token's heads are neighbours in a page, 128 bytes
// each at D = 128 in 8 bits, and are best read at about the same time (B = 64,
// up to 8192 keys, e4m3: 6.0 TB/s; 4.0 with the heads apart on the line, before
// other steps).
#pragma once

#include <cstdint>

#include "kv_internal.h"

namespace fa {

// The next kernel of the stream, launched with programmatic serialisation, may
// be set up from here on; it waits for this one's end before it reads results.
__device__ __forceinline__ void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_predecessor() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- work line
// Row tiles and units of sequence b; zero where there is nothing to do. Bad
// sequences (reported once by the caller) have nothing to do.
struct SeqWork {
  int first, n, len;   // first query row, query rows, keys
  int mtiles, units;
  bool bad;
};
__device__ __forceinline__ SeqWork seq_work(const KvAttnParams& p, int b, int rt, int unit) {
  SeqWork w;
  w.bad = !seq_rows(p.s, b, w.first, w.n);
  w.len = __ldg(p.s.seqlens_k + b);
  if (w.len < 0 || (int64_t)w.len > (int64_t)p.s.max_pages * p.s.page_size) w.bad = true;
  if (w.bad) w.n = w.len = 0;
  w.mtiles = (w.n * p.G + rt - 1) / rt;
  w.units = w.mtiles > 0 ? (w.len + unit - 1) / unit : 0;
  return w;
}
// range c of n is the units [c U / n, (c + 1) U / n)
__device__ __forceinline__ int range_start(int c, int n, int U) { return (int)((int64_t)c * U / n); }
__device__ __forceinline__ int range_of(int u, int n, int U) { return (int)((((int64_t)u + 1) * n - 1) / U); }

// Whole items have a slot each, in Hk's: that of tile mt of sequence b, by the
// rows before the sequence's (a short last tile moves the next sequences on by
// one), so there are total * G / rt + B at most, whatever bounds the lengths.
__device__ __forceinline__ int whole_slot(const KvAttnParams& p, int rt, int b, int first, int mt) {
  return first * p.G / rt + b + mt;
}

// Part of a work item that one worker takes.
struct KvSegment {
  int pre, b, hk, mt;         // shared prefix?; sequence, K/V head, row tile
  int len, first, rows, Lq;   // keys; first query row, rows of the item's matrix, queries of the sequence
  int at, take;               // first unit and number of units (0: the end)
  int slot, direct;           // where its partial goes; direct: it is the whole item, O and LSE are written
};
// Slots: two per worker (range r of `ranges`, head hk) for the items that it
// shares with its neighbours (the one it begins with, the one it ends with),
// then one per whole item and head where even those are joined with others (a
// prefix).
__device__ __forceinline__ KvSegment find_segment(const KvAttnParams& p, int rt, int unit, const int* cum, int u, int u_begin,
                                                  int u_end, int pre_units, int pre_total, int r, int ranges, int hk) {
  KvSegment s;
  int units;
  s.b = s.first = s.Lq = s.take = s.direct = 0;
  s.hk = hk;
  s.pre = u < pre_total;
  if (s.pre) {
    units = pre_units;
    s.mt = u / units;
    s.at = u - s.mt * units;
    s.len = p.prefix_len;
    s.rows = p.s.total * p.G;
    s.slot = (2 * ranges + (p.pass_own ? p.s.total * p.G / rt + p.s.B : 0) + s.mt) * p.Hk + hk;
  } else {
    const int v = u - pre_total;
    int lo = 0, hi = p.s.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cum[mid] <= v) lo = mid; else hi = mid;
    }
    const SeqWork w = seq_work(p, lo, rt, unit);
    units = w.units;
    if (units <= 0 || w.mtiles * units != cum[lo + 1] - cum[lo]) return s;   // the lengths changed under the call
    s.b = lo;
    s.mt = (v - cum[lo]) / units;
    s.at = v - cum[lo] - s.mt * units;
    s.len = w.len;
    s.Lq = w.n;
    s.first = w.first;
    s.rows = w.n * p.G;
    s.slot = (2 * ranges + whole_slot(p, rt, lo, w.first, s.mt)) * p.Hk + hk;
  }
  s.take = min(units - s.at, u_end - u);
  if (s.take < units)
    s.slot = (2 * r + (u == u_begin ? 0 : 1)) * p.Hk + hk;
  else
    s.direct = p.direct;
  return s;
}

// Units before each sequence, cum[0 .. B], by a scan over the block (all its
// threads; sm_warp: one int per warp). Ends with a barrier. Valid sequences have
// at most p.most_units (counted in 32 bits): all of them together have no more
// rows than `total`. Sequences that overlap (prefix sums that go down in between)
// can have more; sums stop one above, and then nothing is done and it is reported.
__device__ __forceinline__ void scan_units(const KvAttnParams& p, int rt, int unit, int threads, int* cum, int* sm_warp) {
  const uint32_t most = (uint32_t)p.most_units;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = threads >> 5;
  uint32_t carry = 0;
  for (int b0 = 0; b0 < p.s.B; b0 += threads) {
    const int b = b0 + threadIdx.x;
    uint32_t x = 0;
    if (b < p.s.B) {
      const SeqWork w = seq_work(p, b, rt, unit);
      x = min((uint32_t)(w.mtiles * w.units), most + 1u);
      if (w.bad && blockIdx.x == 0) atomicOr(p.s.status, kDevBadSeqlens);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = min(x + y, most + 1u);
    }
    if (lane == 31) sm_warp[warp] = (int)x;
    __syncthreads();
    uint32_t before = carry;
    for (int i = 0; i < warps; ++i) {
      if (i == warp) before = carry;
      carry = min(carry + (uint32_t)sm_warp[i], most + 1u);
    }
    if (b < p.s.B) cum[b + 1] = (int)min(before + x, most + 1u);
    __syncthreads();
  }
  if (threadIdx.x == 0) cum[0] = 0;
  if (carry > most) {   // the same in every thread
    for (int b = threadIdx.x; b <= p.s.B; b += threads) cum[b] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.s.status, kDevBadSeqlens);
  }
  __syncthreads();
}

// Keys that row R of a segment sees: the first `lim` of the segment's len.
__device__ __forceinline__ int row_limit(const KvAttnParams& p, const KvSegment& s, int R) {
  const int t = R / p.G;
  int l = s.len;
  if (!s.pre) {
    if (p.causal) l = t + s.len - s.Lq + 1;
  } else {
    const int sq = seq_of_row(p.s, t);
    l = 0;
    if (sq >= 0) {
      const SeqWork w = seq_work(p, sq, 1, 1);
      if (!w.bad) l = p.causal ? t - w.first + s.len + w.len - w.n + 1 : s.len;
    }
  }
  return max(min(l, s.len), 0);
}

}  // namespace fa
