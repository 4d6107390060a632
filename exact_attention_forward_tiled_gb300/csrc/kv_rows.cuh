// Attention of many query rows over a paged K/V cache: a prefix that a batch
// shares (the rows of all its sequences against the same keys), drafted tokens
// of models with many heads per K/V head, chunks of prompts. The few-row kernel
// (kv_attn.cuh) has the formulas and the arithmetic of 8-bit caches; this one
// runs them on tcgen05.
//
// With 256 rows a block of 128 keys of 128 elements costs 16.8 million
// operations, 1.3 us of an SM's share of the tensor cores, and 33 KB (e4m3),
// 0.75 us of its share of HBM. One CTA per SM, up to 256 rows (two 128-row
// tiles; one at D = 256 or for up to 128 rows) against 128-key blocks:
//
//   load warp       finds the work (kv_work.cuh), hands it to the others
//                   through a small ring, loads pages with TMA: 16-bit tiles
//                   straight into the operand slots, 8-bit codes into a ring
//                   of their own
//   convert warps   four; 8-bit codes -> f16 operand tiles in the swizzled layout
//                   the tensor core reads (exact); rows past the last key are
//                   made zeros (whatever the page held there, 0 times a NaN is
//                   not 0), which is all that two do for 16-bit caches
//   scale warps     two, 8-bit caches only: a block's scales into shared memory
//   MMA thread      S_t = Q_t K^T, O_t += P_t V, accumulators in tensor memory
//   softmax warps   four per tile, a thread owns a row: scores, weights, P back
//                   into tensor memory over the scores, row sums
//
// An 8-bit block is converted once for 256 rows, behind the products of the
// block before. The products' order for two tiles (QK0_j, PV1_{j-1}, QK1_j,
// PV0_j) gives each tile's softmax the other tile's two products to run behind.
//
// P is rounded to f16 (8-bit and fp16 caches) or bf16; l takes it unrounded.
//
// Measured: 256 rows, 8 K/V heads of 128, 32768 shared keys, e4m3: 70 us; 25 us
// for the first block and the ends (131072 keys: 199 us), then 3.2 us for each
// block of 128 keys. 16-bit: 41 and 117 us, 1.7 us a block, 5.8 TB/s. The 8-bit
// form is bound by no unit (tensor core 20 %, issue slots 36 %, shared memory
// 29 %) but by a tile's chain scores, max, weights, P, product. Slower or no
// faster: 8 convert warps, two warps to a row, longer rings, scores read ahead
// or in the layout of an mma's accumulator.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <type_traits>

#include "kv_codes.cuh"
#include "kv_work.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace fa {

template <int D_, int KIND_, int QT_>
struct RowsCfg {
  static constexpr int D = D_, KIND = KIND_, QT = QT_;
  static constexpr bool k8 = cache_is_8bit(KIND);
  static constexpr int RT = 128 * QT;
  static constexpr int BOX = D / 64;                        // operand boxes of 64 elements x 128 rows
  static constexpr int kBoxBytes = 128 * 128;
  static constexpr int kTileBytes = BOX * kBoxBytes;
  static constexpr int NS = D == 64 ? 6 : D == 128 ? 4 : 2;   // operand slots
  // 8-bit: codes arrive in parts of RK keys
  static constexpr int RK = rows_box(D, 1);
  static constexpr int PARTS = 128 / RK;
  static constexpr int RS = D == 64 ? 8 : 3;   // slots of codes (none for 16-bit caches)
  static constexpr int RS_USED = k8 ? RS : 0;
  static constexpr int RB = D < 128 ? D : 128;              // bytes of a code box row
  static constexpr int RBOX = D / RB;
  static constexpr int kRawBytes = RK * D;
  static constexpr int kLoadSlots = k8 ? RS : NS;           // slots that TMA fills
  static constexpr int kQkSteps = D / 16, kPvSteps = 8;
  static constexpr float kTau = 8.f;
  static constexpr int kSoftmaxWarps = 4 * QT;
  // MMA warp, load warp, then two scale warps and four convert warps (8-bit
  // caches) or two convert warps
  static constexpr int kMmaWarp = kSoftmaxWarps, kLoadWarp = kMmaWarp + 1;
  static constexpr int kScaleWarps = k8 ? 2 : 0, kScaleWarp = kMmaWarp + 2, kConvWarp = kScaleWarp + kScaleWarps;
  static constexpr int kConvWarps = k8 ? 4 : 2;
  static constexpr int kConvLanes = 32 * kConvWarps;
  static constexpr int kThreads = 32 * (kSoftmaxWarps + 2 + kScaleWarps + kConvWarps);
  // registers: at launch, and then of the softmax warpgroups and of the others
  static constexpr bool kRebalance = kThreads > 256;
  static constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
  static constexpr int kRegsHigh = QT == 2 ? (k8 ? 184 : 216) : 232;
  static constexpr int kRegsLow = QT == 2 ? (k8 ? 72 : 64) : 136;
  static_assert(!kRebalance || kThreads * kRegsLaunch >= 32 * kSoftmaxWarps * kRegsHigh + (kThreads - 32 * kSoftmaxWarps) * kRegsLow,
                "register split");
  static constexpr int kTmemCols = 512;
  __host__ __device__ static constexpr uint32_t col_s(uint32_t b) { return b ? 128u : 0u; }
  __host__ __device__ static constexpr uint32_t col_o(uint32_t t) { return 256u + t * D; }
  static constexpr int SCR = 4;                             // blocks of scales in their ring
  static constexpr int SEGS = 4;                            // segments in their ring
  // shared memory, from a 1024-byte aligned base
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = QT * kTileBytes;
  static constexpr int kOffRaw = kOffKV + NS * kTileBytes;
  static constexpr int kOffScale = kOffRaw + RS_USED * kRawBytes;           // [SCR][2][128] fp32
  static constexpr int kOffBar = kOffScale + (k8 ? SCR * 1024 : 0);
  static constexpr int kBarLoadFull = 0, kBarRawEmpty = kBarLoadFull + kLoadSlots, kBarKVFull = kBarRawEmpty + RS_USED,
                       kBarKVEmpty = kBarKVFull + NS, kBarQFull = kBarKVEmpty + NS, kBarSFull = kBarQFull + 2,
                       kBarPFull = kBarSFull + 2, kBarOFull = kBarPFull + 2, kBarPVDone = kBarOFull + 2,
                       kBarMmaDone = kBarPVDone + 1, kBarScale = kBarMmaDone + 1, kBarScaleEmpty = kBarScale + SCR,
                       kBarSegFull = kBarScaleEmpty + SCR,
                       kBarSegEmpty = kBarSegFull + SEGS, kNumBars = kBarSegEmpty + SEGS;
  static constexpr int kOffSeg = (kOffBar + kNumBars * 8 + 15) & ~15;  // [SEGS] 64 bytes each
  static constexpr int kOffMisc = kOffSeg + SEGS * 64;                 // tmem address, abort flag, warp sums
  static constexpr int kOffCum = kOffMisc + 16 + 64;                   // cum[B + 1]
  static constexpr int kSmemFixed = kOffCum + 1024;
  static_assert(D == 64 || D == 128 || D == 256, "head dimension");
  static_assert(256 + QT * D <= kTmemCols, "tensor memory");
  static_assert(kSmemFixed + (kRowsMaxSeqs + 1) * 4 <= 232448, "shared memory");
};

// A segment and its key blocks.
struct RowsSegment {
  KvSegment s;
  int nblk;   // 128-key blocks from s.at on
};

template <class C>
struct RowsSync {
  uint32_t bars;
  Waiter wt;
  RowsSegment* segs;   // 64 bytes apart
  __device__ __forceinline__ uint32_t bar(int i) const { return bars + 8u * i; }
  __device__ __forceinline__ RowsSegment* seg(int j) const {
    return reinterpret_cast<RowsSegment*>(reinterpret_cast<uint8_t*>(segs) + 64 * (j % C::SEGS));
  }
  // segment j for a consumer (a whole warp, or one thread); false at the end
  __device__ __forceinline__ bool next(int j, bool warp_wide, bool lead, RowsSegment& out) const {
    const uint32_t par = (j / C::SEGS) & 1u;
    const uint32_t full = bar(C::kBarSegFull + j % C::SEGS);
    if (!(warp_wide ? wt.wait_warp(full, par, 0x30) : wt.wait(full, par, 0x30))) return false;
    out = *seg(j);
    if (warp_wide) __syncwarp();
    if (lead) ptx::mbar_arrive(bar(C::kBarSegEmpty + j % C::SEGS));
    return out.s.take > 0;
  }
};

// ------------------------------------------------------------------ load warp
template <class C>
__device__ void rows_load_role(const CUtensorMap* tk, const CUtensorMap* tv, const KvAttnParams& p, uint32_t sbase,
                               const RowsSync<C>& sy, const int* cum, int u_begin, int u_end, int pre_units, int pre_total) {
  const int lane = threadIdx.x & 31;
  const bool lead = lane == 0;
  // a TMA fill: KEYS keys, (KEYS / box_rows) x BOXES boxes, one lane each
  constexpr int KEYS = C::k8 ? C::RK : 128;
  constexpr int BOXES = C::k8 ? C::RBOX : C::BOX;
  constexpr int ROW_BYTES = C::k8 ? C::RB : 128, COLS = C::k8 ? C::RB : 64;
  constexpr int kFillBytes = C::k8 ? C::kRawBytes : C::kTileBytes;
  const int box_row = lane / BOXES * p.box_rows, box_col = lane % BOXES;
  const bool mine = box_row < KEYS;
  const uint32_t dst0 = sbase + (C::k8 ? C::kOffRaw : C::kOffKV) + box_col * (KEYS * ROW_BYTES) + box_row * ROW_BYTES;
  const int empty0 = C::k8 ? C::kBarRawEmpty : C::kBarKVEmpty;
  const int dead_row = p.s.num_pages * p.s.page_size;   // past the cache: TMA fills zeros
  uint32_t fills = 0;
  bool ok = true;
  auto wait0 = [&](uint32_t b, uint32_t parity, int where) -> bool {
    bool r = true;
    if (lead) r = sy.wt.wait(b, parity, where);
    return __shfl_sync(0xffffffffu, r ? 1 : 0, 0) != 0;
  };
  int u = u_begin;
  for (int j = 0; ok; ++j) {
    if (!(ok = wait0(sy.bar(C::kBarSegEmpty + j % C::SEGS), ((j / C::SEGS) & 1u) ^ 1u, 0x31))) break;
    if (lead) {
      RowsSegment rs;
      rs.s.take = 0;
      rs.nblk = 0;
      if (u < u_end) {
        rs.s = find_segment(p, C::RT, kRowsUnit, cum, u, u_begin, u_end, pre_units, pre_total, (int)blockIdx.x / p.Hk,
                            p.ranges, (int)blockIdx.x % p.Hk);
        if (rs.s.take > 0) {
          int end = min(rs.s.len, (rs.s.at + rs.s.take) * kRowsUnit);
          if (!rs.s.pre && p.causal) {   // the last row sees the most
            const int last = (min(rs.s.rows, (rs.s.mt + 1) * C::RT) - 1) / p.G;
            end = min(end, last + rs.s.len - rs.s.Lq + 1);
          }
          rs.nblk = max((end - rs.s.at * kRowsUnit + kRowsUnit - 1) / kRowsUnit, 0);
        }
      }
      *sy.seg(j) = rs;
      ptx::mbar_arrive(sy.bar(C::kBarSegFull + j % C::SEGS));
    }
    __syncwarp();
    const RowsSegment rs = *sy.seg(j);   // stays until this warp passes here again
    if (rs.s.take <= 0) break;
    u += rs.s.take;
    const int* const table = rs.s.pre ? p.prefix_pages : p.s.block_table + (int64_t)rs.s.b * p.s.max_pages;
    const int per_tile = C::k8 ? C::PARTS : 1;
    const int n = rs.nblk * 2 * per_tile;
    // fill f: part f % per_tile of K or V (f / per_tile even or odd) of block f / (2 per_tile)
    int pg = -2, off = 0;
    auto lookup = [&](int f) {
      const int key = (rs.s.at + f / (2 * per_tile)) * kRowsUnit + (f % per_tile) * KEYS + box_row;
      pg = -2;
      if (f < n && mine && key < rs.s.len) {
        int index;
        page_of(p.s, key, index, off);
        pg = __ldg(table + index);
      }
    };
    lookup(0);
    for (int f = 0; ok && f < n; ++f) {
      const int s = fills % C::kLoadSlots;
      if (!(ok = wait0(sy.bar(empty0 + s), ((fills / C::kLoadSlots) & 1u) ^ 1u, 0x32))) break;
      const uint32_t b = sy.bar(C::kBarLoadFull + s);
      if (lead) ptx::mbar_arrive_expect_tx(b, kFillBytes);
      __syncwarp();
      if (mine) {
        int row = dead_row;
        if (pg >= 0 && pg < p.s.num_pages)
          row = pg * p.s.page_size + off;
        else if (pg != -2)
          atomicOr(p.s.status, kDevBadSeqlens);
        ptx::tma_load_2d(dst0 + s * kFillBytes, (f / per_tile) & 1 ? tv : tk, rs.s.hk * C::D + box_col * COLS, row, b);
      }
      ++fills;
      lookup(f + 1);
    }
  }
  if (lead && *sy.wt.abort_flag) {
    // let the copies in flight land before the CTA's memory goes away
    const uint32_t first = fills > (uint32_t)C::kLoadSlots ? fills - C::kLoadSlots : 0u;
    for (uint32_t c = first; c < fills; ++c)
      sy.wt.drain(sy.bar(C::kBarLoadFull + (int)(c % C::kLoadSlots)), (c / C::kLoadSlots) & 1u);
  }
}

// ------------------------------------------------------------------ scale warps
// Two keys a lane: the K scales (times c = scale log2 e) and V scales of a
// block into shared memory.
template <class C>
__device__ void rows_scale_role(const KvAttnParams& p, uint32_t sbase, const RowsSync<C>& sy, int w) {
  const int lane = threadIdx.x & 31;
  const bool lead = lane == 0;
  const int idx = w * 32 + lane;
  uint32_t blk = 0;
  RowsSegment rs;
  for (int j = 0; sy.next(j, true, lead, rs); ++j) {
    const int* const table = rs.s.pre ? p.prefix_pages : p.s.block_table + (int64_t)rs.s.b * p.s.max_pages;
    // the page of the block after the next and the scales of the next one are
    // on their way while a block waits for its slot
    auto page = [&](int i) -> int {
      const int key = (rs.s.at + i) * kRowsUnit + 2 * idx;
      if (i >= rs.nblk || key >= rs.s.len) return -1;
      int index, off;
      page_of(p.s, key, index, off);
      return __ldg(table + index);
    };
    float2 ks, vs;
    auto scales = [&](int i, int pg) {
      ks = vs = make_float2(0.f, 0.f);
      if ((unsigned)pg >= (unsigned)p.s.num_pages) return;
      const int key = (rs.s.at + i) * kRowsUnit + 2 * idx;
      int index, off;
      page_of(p.s, key, index, off);
      const int64_t at = ((int64_t)pg * p.Hk + rs.s.hk) * p.s.page_size + off;
      ks = __ldg(reinterpret_cast<const float2*>(p.k_scale + at));
      vs = __ldg(reinterpret_cast<const float2*>(p.v_scale + at));
      // what a page holds past the last key must not enter the block's bounds
      if (key + 1 >= rs.s.len) ks.y = vs.y = 0.f;
    };
    scales(0, page(0));
    int pg = page(1);
    for (int i = 0; i < rs.nblk; ++i, ++blk) {
      const int s = blk % C::SCR;
      if (!sy.wt.wait_warp(sy.bar(C::kBarScaleEmpty + s), ((blk / C::SCR) & 1u) ^ 1u, 0x3d)) return;
      const uint32_t dst = sbase + C::kOffScale + s * 1024u + idx * 8;
      // + 0: a scale of -0 becomes 0 (the bounds compare bits)
      st_shared_f2(dst, make_float2(fmaf(ks.x, p.c, 0.f), fmaf(ks.y, p.c, 0.f)));
      st_shared_f2(dst + 512, make_float2(vs.x + 0.f, vs.y + 0.f));
      __syncwarp();
      if (lead) ptx::mbar_arrive(sy.bar(C::kBarScale + s));
      scales(i + 1, pg);
      pg = page(i + 2);
    }
  }
}

// ------------------------------------------------------------------ convert warps
template <class C>
__device__ void rows_convert_role(uint32_t sbase, const RowsSync<C>& sy, int cw) {
  const int lane = threadIdx.x & 31;
  const bool lead = lane == 0;
  const int idx = cw * 32 + lane;
  // Eight lanes take four 16-code chunks of two rows, r and r ^ 5 of a group of
  // eight: under both swizzles their 16-byte reads, and their two writes each,
  // then cover all banks once. The lanes step down the rows by whole groups, so
  // a lane's place in its row and in the swizzle never changes.
  constexpr int CPR = C::D / 16;                          // chunks of a row
  constexpr int PER = C::RK / 2 * (CPR / 4) / (C::kConvLanes / 8);   // chunks of a lane in a part
  constexpr int STEP = C::RK / PER;                       // rows between them
  static_assert(!C::k8 || (PER * STEP == C::RK && STEP % 8 == 0), "whole groups of rows");
  const int un = idx >> 3, hi = (idx >> 2) & 1, c4 = idx & 3;
  const int rp = un / (CPR / 4), c = (un % (CPR / 4)) * 4 + c4;
  const int r7 = (rp & 3) ^ (5 * hi), row = (rp >> 2) * 8 + r7;
  const uint32_t src0 = C::RB == 128 ? (c / 8) * (C::RK * 128) + row * 128 + (((c & 7) ^ r7) << 4)
                                     : row * 64 + ((c ^ (r7 >> 1)) << 4);
  const uint32_t dst0 = (c / 4) * C::kBoxBytes + row * 128 + (((2 * c4) ^ r7) << 4);
  uint32_t raw = 0, tile = 0;   // code parts and operand tiles so far
  RowsSegment rs;
  for (int j = 0; sy.next(j, true, lead, rs); ++j) {
    for (int i = 0; i < 2 * rs.nblk; ++i, ++tile) {   // K, V of block i / 2
      const int left = rs.s.len - (rs.s.at + (i >> 1)) * kRowsUnit;   // rows that exist from the block's first on
      const int s = tile % C::NS;
      const uint32_t dst = sbase + C::kOffKV + s * C::kTileBytes;
      if (!C::k8) {
        // the tile is there already; V's rows past the end become zeros
        if (!sy.wt.wait_warp(sy.bar(C::kBarLoadFull + s), (tile / C::NS) & 1u, 0x33)) return;
        if ((i & 1) && left < 128) {
          for (int q = idx; q < (128 - left) * C::BOX * 8; q += C::kConvLanes) {
            const int r = left + q / (C::BOX * 8), x = q % (C::BOX * 8);
            st_shared_zero16(dst + (x / 8) * C::kBoxBytes + r * 128 + (x % 8) * 16);
          }
          ptx::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lead) ptx::mbar_arrive(sy.bar(C::kBarKVFull + s));
        continue;
      }
      if (!sy.wt.wait_warp(sy.bar(C::kBarKVEmpty + s), ((tile / C::NS) & 1u) ^ 1u, 0x34)) return;
#pragma unroll 1
      for (int part = 0; part < C::PARTS; ++part, ++raw) {
        const int r = raw % C::RS;
        if (!sy.wt.wait_warp(sy.bar(C::kBarLoadFull + r), (raw / C::RS) & 1u, 0x35)) return;
        const uint32_t src = sbase + C::kOffRaw + r * C::kRawBytes + src0;
        const uint32_t out = dst + part * C::RK * 128 + dst0;
        uint4 v[PER];
#pragma unroll
        for (int q = 0; q < PER; ++q) v[q] = lds128(src + q * STEP * C::RB);
        if (left < 128) {
#pragma unroll
          for (int q = 0; q < PER; ++q)
            if (part * C::RK + row + q * STEP >= left) v[q] = make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < PER; ++q) {
          uint4 x, y;
          codes_to_f16<C::KIND>(v[q].x, x.x, x.y);
          codes_to_f16<C::KIND>(v[q].y, x.z, x.w);
          codes_to_f16<C::KIND>(v[q].z, y.x, y.y);
          codes_to_f16<C::KIND>(v[q].w, y.z, y.w);
          sts128(out + q * STEP * 128, x);
          sts128((out + q * STEP * 128) ^ 16u, y);
        }
        __syncwarp();
        if (lead) ptx::mbar_arrive(sy.bar(C::kBarRawEmpty + r));
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lead) ptx::mbar_arrive(sy.bar(C::kBarKVFull + s));
    }
  }
}

// ------------------------------------------------------------------ MMA thread
template <class C>
__device__ void rows_mma_role(uint32_t sbase, uint32_t tmem, const RowsSync<C>& sy) {
  constexpr uint32_t fmt = C::KIND == kCacheBF16 ? 1u : 0u;
  constexpr uint32_t idesc_qk = ptx::make_idesc(fmt, false, 128, 128);
  constexpr uint32_t idesc_pv = ptx::make_idesc(fmt, true, 128, C::D);
  const uint32_t sq = sbase + C::kOffQ;
  auto slot = [&](uint32_t c) { return (int)(c % C::NS); };
  auto addr = [&](uint32_t c) { return sbase + C::kOffKV + slot(c) * C::kTileBytes; };
  auto qk = [&](uint32_t s_col, uint32_t q_addr, uint32_t k_addr) {
#pragma unroll
    for (int kk = 0; kk < C::kQkSteps; ++kk) {
      const uint32_t off = (kk / 4) * C::kBoxBytes + (kk % 4) * 32;
      ptx::mma_f16_ss(tmem + s_col, ptx::smem_desc_sw128(q_addr + off, 16, 1024), ptx::smem_desc_sw128(k_addr + off, 16, 1024),
                      idesc_qk, kk > 0);
    }
  };
  auto pv = [&](uint32_t o_col, uint32_t p_col, uint32_t v_addr, bool acc, int pbuf, uint32_t parity) -> bool {
    if (!sy.wt.wait(sy.bar(C::kBarPFull + pbuf), parity, 0x36)) return false;
    ptx::tc_fence_after();
#pragma unroll
    for (int kk = 0; kk < C::kPvSteps; ++kk)
      ptx::mma_f16_ts(tmem + o_col, tmem + p_col + kk * 8, ptx::smem_desc_sw128(v_addr + kk * 16 * 128, C::kBoxBytes, 1024),
                      idesc_pv, (acc || kk > 0) ? 1u : 0u);
    return true;
  };
  auto ready = [&](uint32_t c) {
    const bool r = sy.wt.wait(sy.bar(C::kBarKVFull + slot(c)), (c / C::NS) & 1u, 0x37);
    ptx::tc_fence_after();
    return r;
  };
  uint32_t kvc = 0, it = 0, tiles = 0;
  bool ok = true;
  RowsSegment rs;
  for (int j = 0; ok && sy.next(j, false, true, rs); ++j) {
    const int n = rs.nblk;
    if (n == 0) continue;
    const uint32_t qpar = tiles & 1u;
    ++tiles;
    if (!(ok = sy.wt.wait(sy.bar(C::kBarQFull), qpar, 0x38))) break;
    ptx::tc_fence_after();
    if (C::QT == 2) {
      if (!(ok = ready(kvc))) break;
      qk(C::col_s(0), sq, addr(kvc));
      ptx::mma_commit(sy.bar(C::kBarSFull));
      if (!(ok = sy.wt.wait(sy.bar(C::kBarQFull + 1), qpar, 0x38))) break;
      ptx::tc_fence_after();
      for (int i = 0; i < n; ++i) {
        const uint32_t ck = kvc + 2 * i, cv = ck + 1;
        if (i > 0) {
          if (!(ok = pv(C::col_o(1), C::col_s(1), addr(cv - 2), i - 1 > 0, 1, (it + i - 1) & 1u))) break;
          ptx::mma_commit(sy.bar(C::kBarKVEmpty + slot(cv - 2)));
        }
        qk(C::col_s(1), sq + C::kTileBytes, addr(ck));
        ptx::mma_commit(sy.bar(C::kBarSFull + 1));
        ptx::mma_commit(sy.bar(C::kBarKVEmpty + slot(ck)));
        if (!(ok = ready(cv))) break;
        if (!(ok = pv(C::col_o(0), C::col_s(0), addr(cv), i > 0, 0, (it + i) & 1u))) break;
        if (i == n - 1) ptx::mma_commit(sy.bar(C::kBarOFull));
        if (i + 1 < n) {
          if (!(ok = ready(ck + 2))) break;
          qk(C::col_s(0), sq, addr(ck + 2));
          ptx::mma_commit(sy.bar(C::kBarSFull));
        }
      }
      if (!ok) break;
      const uint32_t cl = kvc + 2 * n - 1;
      if (!(ok = pv(C::col_o(1), C::col_s(1), addr(cl), n - 1 > 0, 1, (it + n - 1) & 1u))) break;
      ptx::mma_commit(sy.bar(C::kBarKVEmpty + slot(cl)));
      ptx::mma_commit(sy.bar(C::kBarOFull + 1));
    } else {
      // K_0, V_0, K_1, ... lie in the slots in this order; the products run
      // K_0, K_1, V_0, K_2, V_1, ... with scores double-buffered
      if (!(ok = ready(kvc))) break;
      qk(C::col_s(it & 1u), sq, addr(kvc));
      ptx::mma_commit(sy.bar(C::kBarSFull + (int)(it & 1u)));
      ptx::mma_commit(sy.bar(C::kBarKVEmpty + slot(kvc)));
      for (int i = 0; i < n; ++i) {
        const uint32_t x = it + i;
        const uint32_t cv = kvc + 2 * i + 1, ck = cv + 1;
        if (i + 1 < n) {
          if (!(ok = ready(ck))) break;
          qk(C::col_s((x + 1) & 1u), sq, addr(ck));
          ptx::mma_commit(sy.bar(C::kBarSFull + (int)((x + 1) & 1u)));
          ptx::mma_commit(sy.bar(C::kBarKVEmpty + slot(ck)));
        }
        if (!(ok = ready(cv))) break;
        if (!(ok = pv(C::col_o(0), C::col_s(x & 1u), addr(cv), i > 0, (int)(x & 1u), (x >> 1) & 1u))) break;
        ptx::mma_commit(sy.bar(C::kBarKVEmpty + slot(cv)));
        ptx::mma_commit(sy.bar(C::kBarPVDone));
        if (i == n - 1) ptx::mma_commit(sy.bar(C::kBarOFull));
      }
    }
    kvc += 2 * n;
    it += n;
  }
  // all issued products complete before tensor memory is released
  ptx::mma_commit(sy.bar(C::kBarMmaDone));
  sy.wt.drain(sy.bar(C::kBarMmaDone), 0);
}

// ------------------------------------------------------------------ softmax warps
template <class C>
__device__ void rows_softmax_role(const KvAttnParams& p, uint32_t sbase, uint32_t tmem, const RowsSync<C>& sy, int t, int quarter) {
  constexpr int D = C::D;
  constexpr float kNone = -3e38f;   // m of a row that has seen no key
  const int lane = threadIdx.x & 31;
  const int r = quarter * 32 + lane;
  const uint32_t tl = tmem + ((uint32_t)(quarter * 32) << 16);
  const uint32_t o_addr = tl + C::col_o(C::QT == 2 ? t : 0);
  uint32_t it = 0, tiles = 0;
  RowsSegment rs;
  for (int j = 0; sy.next(j, true, lane == 0, rs); ++j) {
    const KvSegment& sg = rs.s;
    const int R = sg.mt * C::RT + 128 * t + r;
    const bool have = R < sg.rows;
    const int tok = have ? R / p.G : 0;
    const int hq = sg.hk * p.G + (have ? R - tok * p.G : 0);
    const int64_t row_at = have ? ((int64_t)(sg.first + tok) * p.Hq + hq) * D : -1;   // in q and in o
    float m_ref = kNone, l = 0.f, rowf = p.c;
    int lr = C::k8 ? 100 : 0;
    bool ok = true;
    if (rs.nblk > 0) {
      // ---- the warp's rows of Q into the operand tile, LPR lanes to a row
      // (8-bit caches, bf16 queries: scaled by a power of two and made f16)
      constexpr int LPR = D / 8, RPI = 32 / LPR;
      const int ch = lane % LPR;
      uint4 v[LPR];
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, (long long)row_at, i * RPI + lane / LPR);
        v[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + at) + ch) : make_uint4(0, 0, 0, 0);
      }
      if (C::k8) rowf = 1.f;
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        if (C::k8 && p.q_bf16) {
          uint32_t m = __vmaxu2(__vmaxu2(v[i].x & 0x7fff7fffu, v[i].y & 0x7fff7fffu),
                                __vmaxu2(v[i].z & 0x7fff7fffu, v[i].w & 0x7fff7fffu));
#pragma unroll
          for (int x = LPR / 2; x >= 1; x >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, x));
          const uint32_t e = max(m & 0xffffu, m >> 16);
          float f = 1.f, qs = 1.f;
          if (e != 0 && e < 0x7f80u) {
            // the largest element times 2^sh is in [2^14, 2^15) (less where it is below 2^-100)
            const int sh = min(14 - ((int)(e >> 7) - 127), 114);
            f = __uint_as_float((uint32_t)(127 + sh) << 23);
            qs = __uint_as_float((uint32_t)(127 - sh) << 23);
          }
          qs = __shfl_sync(0xffffffffu, qs, lane % RPI * LPR);
          if (lane / RPI == i) rowf = qs;   // the row of this lane
          uint32_t* x = reinterpret_cast<uint32_t*>(&v[i]);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            x[k] = ptx::pack_f16(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f);
        }
        const int rr = quarter * 32 + i * RPI + lane / LPR;
        sts128(sbase + C::kOffQ + t * C::kTileBytes + (ch / 8) * C::kBoxBytes + rr * 128 + (((ch % 8) ^ (rr & 7)) << 4), v[i]);
      }
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(sy.bar(C::kBarQFull + t));
    }
    // (behind Q, whose product can begin)
    const int lim = have ? row_limit(p, sg, R) : sg.len;   // a missing row asks for no mask
    for (int i = 0; i < rs.nblk; ++i, ++it) {
      const int key0 = (sg.at + i) * kRowsUnit;
      const int buf = C::QT == 2 ? t : (int)(it & 1u);
      const uint32_t par = C::QT == 2 ? (it & 1u) : ((it >> 1) & 1u);
      const uint32_t sc = sbase + C::kOffScale + (it % C::SCR) * 1024u;
      if (C::k8 && !(ok = sy.wt.wait_warp(sy.bar(C::kBarScale + (int)(it % C::SCR)), (it / C::SCR) & 1u, 0x39))) break;
      // while the scores are on their way: bounds on the block's scales
      float thr = C::kTau, k_hi = 0.f, k_lo = 0.f;
      uint32_t v_hi = 0, v_lo = 0;
      if (C::k8) {
        const float4 f = lds128f(sc + 16 * lane), w = lds128f(sc + 512 + 16 * lane);
        const uint32_t hi = max(max(__float_as_uint(f.x), __float_as_uint(f.y)), max(__float_as_uint(f.z), __float_as_uint(f.w)));
        const uint32_t lo = min(min(__float_as_uint(f.x), __float_as_uint(f.y)), min(__float_as_uint(f.z), __float_as_uint(f.w)));
        const uint32_t e = max(max(__float_as_uint(w.x), __float_as_uint(w.y)), max(__float_as_uint(w.z), __float_as_uint(w.w)));
        k_hi = __uint_as_float(__reduce_max_sync(0xffffffffu, hi));
        k_lo = __uint_as_float(__reduce_min_sync(0xffffffffu, lo));
        v_hi = __reduce_max_sync(0xffffffffu, e);
        v_lo = __reduce_min_sync(0xffffffffu, min(min(__float_as_uint(w.x), __float_as_uint(w.y)),
                                                  min(__float_as_uint(w.z), __float_as_uint(w.w))));
        // 15 - log2 of a bound on the block's V scales, less what the weights are held at
        thr = (float)(15 + 126 - (int)(v_hi >> 23) - lr);
      }
      if (!(ok = sy.wt.wait_warp(sy.bar(C::kBarSFull + buf), par, 0x3a))) break;
      ptx::tc_fence_after();
      const uint32_t s_addr = tl + C::col_s(buf);
      const int seen = lim - key0;
      const bool masked = __any_sync(0xffffffffu, seen < 128);
      // 32 columns of this row's scores; with an 8-bit cache still without ks
      auto take = [&](uint32_t (&v)[32], float (&s)[32]) {   // what tmem_ld32 has brought
        ptx::tmem_wait_ld();
        ptx::reg_fence(v);
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = __uint_as_float(v[k]);
      };
      auto load = [&](int ch, float (&s)[32]) {
        uint32_t v[32];
        ptx::tmem_ld32(s_addr + 32 * ch, v);
        take(v, s);
      };
      auto times_ks = [&](int ch, float (&s)[32]) {   // the scales hold c = scale log2 e already
#pragma unroll
        for (int k = 0; k < 32; k += 4) {
          const float4 f = lds128f(sc + 4 * (32 * ch + k));
          ptx::f2unpack(ptx::mul2(ptx::f2pack(s[k], s[k + 1]), ptx::f2pack(f.x, f.y)), s[k], s[k + 1]);
          ptx::f2unpack(ptx::mul2(ptx::f2pack(s[k + 2], s[k + 3]), ptx::f2pack(f.z, f.w)), s[k + 2], s[k + 3]);
        }
      };
      auto hide = [&](int ch, float (&s)[32]) {
#pragma unroll
        for (int k = 0; k < 32; ++k) s[k] = 32 * ch + k < seen ? s[k] : -CUDART_INF_F;
      };
      auto max32 = [&](const float (&s)[32]) {
        float x[11];
#pragma unroll
        for (int k = 0; k < 10; ++k) x[k] = ptx::max3(s[3 * k], s[3 * k + 1], s[3 * k + 2]);
        x[10] = fmaxf(s[30], s[31]);
        return fmaxf(fmaxf(ptx::max3(x[0], x[1], x[2]), ptx::max3(x[3], x[4], x[5])),
                     ptx::max3(fmaxf(x[6], x[7]), x[8], fmaxf(x[9], x[10])));
      };
      // The scores are read from tensor memory twice, 32 columns at a time in
      // rolled loops, for the max and for the weights: held all at once (128
      // registers, code unrolled 128 times) the instruction fetches and spills
      // cost more than the second read.
      float mx = -CUDART_INF_F;
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        float s[32];
        load(ch, s);
        if (masked) hide(ch, s);
        mx = fmaxf(mx, max32(s));
      }
      // m + up: a bound on the row's largest score; 8-bit: the largest product
      // times the largest (if negative, the smallest) scale, good enough to see
      // that nothing has to move
      if (C::k8) mx = mx == -CUDART_INF_F ? mx : mx * (mx > 0.f ? k_hi : k_lo);
      const float up = mx == -CUDART_INF_F ? mx : fmaf(mx, rowf, -m_ref);
      // (not <=: a NaN scale has to get through, too)
      if (__any_sync(0xffffffffu, !(up <= fminf(C::kTau, thr)) || (C::k8 && thr < 0.f))) {
        float cr = 1.f;
        if (C::k8) {
          mx = -CUDART_INF_F;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            float s[32];
            load(ch, s);
            times_ks(ch, s);
            if (masked) hide(ch, s);
            mx = fmaxf(mx, max32(s));
          }
        }
        const float x = mx == -CUDART_INF_F ? mx : mx * rowf;
        if (x > m_ref + C::kTau) {
          if (m_ref != kNone) cr = ptx::ex2(m_ref - x);   // else nothing was summed yet
          m_ref = x;
        }
        if (C::k8) {
          // the largest weight at the new m; where it belongs: [2^6, 2^7) (as
          // in the few-row kernel)
          float um = 0.f;
          const bool top = mx == -CUDART_INF_F || x == m_ref;   // a row's largest weight is 1 (or it has none)
          if (__all_sync(0xffffffffu, top) && v_lo > 0 && v_hi < 0x7f800000u && (v_hi >> 23) - (v_lo >> 23) <= 4) {
            // scales within 2^5 of one another (most first blocks): the bound
            // 1 * the largest does, at [2^1, 2^7)
            um = mx == -CUDART_INF_F ? 0.f : __uint_as_float(v_hi);
          } else {
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
              float s[32];
              load(ch, s);
              times_ks(ch, s);
              if (masked) hide(ch, s);
#pragma unroll
              for (int k = 0; k < 32; k += 4) {
                const float4 f = lds128f(sc + 512 + 4 * (32 * ch + k));
                const float w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  um = fmaxf(um, s[k + q] == -CUDART_INF_F ? 0.f : ptx::ex2(fmaf(s[k + q], rowf, -m_ref)) * w[q]);
              }
            }
          }
          const int e = um > 0.f ? (int)(__float_as_uint(um) >> 23) - 127 : -200;
          const int old = lr;
          if (e + old >= 15) lr = 6 - e;
          else if (cr < 1.f) lr = min(6 - e, old + (cr > 0.f ? 126 - (int)(__float_as_uint(cr) >> 23) : 200));
          lr = max(min(lr, 100), -120);
          cr = cr == 0.f ? 0.f : cr * ptx::ex2((float)(lr - old));
        }
        l *= cr;
        if (i > 0) {   // the first block's product starts O anew
          if (C::QT == 1) {
            // the product before must have landed in O
            if (!(ok = sy.wt.wait_warp(sy.bar(C::kBarPVDone), (it - 1) & 1u, 0x3b))) break;
            ptx::tc_fence_after();
          }
          const uint64_t a2 = ptx::f2pack(cr, cr);
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            uint32_t v[32];
            ptx::tmem_ld32(o_addr + 32 * ch, v);
            ptx::tmem_wait_ld();
            ptx::reg_fence(v);
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              float lo, hi;
              ptx::f2unpack(ptx::mul2(ptx::f2pack(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), a2), lo, hi);
              v[k] = __float_as_uint(lo);
              v[k + 1] = __float_as_uint(hi);
            }
            ptx::tmem_st32(o_addr + 32 * ch, v);
          }
          ptx::tmem_wait_st();
        }
      }
      const float mu = (float)lr - m_ref;
      const uint64_t f2 = ptx::f2pack(rowf, rowf), mu2 = ptx::f2pack(mu, mu);
      uint64_t sum = ptx::f2pack(0.f, 0.f);
      // weights of 32 columns and, at half the columns, P over the scores read
      // (one branch on the mask: selects in the common path would double its
      // integer work)
      auto weights = [&](auto mask) {
        constexpr bool kMask = decltype(mask)::value;
        auto part = [&](int ch, float (&s)[32]) {
          if (C::k8) times_ks(ch, s);
          uint32_t pk[16];
          uint64_t ps[8];
#pragma unroll
          for (int k = 0; k < 32; k += 4) {
            float x[4];
            ptx::f2unpack(ptx::fma2(ptx::f2pack(s[k], s[k + 1]), f2, mu2), x[0], x[1]);
            ptx::f2unpack(ptx::fma2(ptx::f2pack(s[k + 2], s[k + 3]), f2, mu2), x[2], x[3]);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              x[q] = ptx::ex2(x[q]);
              if (kMask) x[q] = 32 * ch + k + q < seen ? x[q] : 0.f;
            }
            ps[k / 4] = ptx::add2(ptx::f2pack(x[0], x[1]), ptx::f2pack(x[2], x[3]));
            if (C::k8) {
              const float4 f = lds128f(sc + 512 + 4 * (32 * ch + k));
              ptx::f2unpack(ptx::mul2(ptx::f2pack(x[0], x[1]), ptx::f2pack(f.x, f.y)), x[0], x[1]);
              ptx::f2unpack(ptx::mul2(ptx::f2pack(x[2], x[3]), ptx::f2pack(f.z, f.w)), x[2], x[3]);
              if (kMask) {   // whatever the scale holds
#pragma unroll
                for (int q = 0; q < 4; ++q) x[q] = 32 * ch + k + q < seen ? x[q] : 0.f;
              }
            }
            pk[k / 2] = C::KIND == kCacheBF16 ? ptx::pack_bf16(x[0], x[1]) : ptx::pack_f16(x[0], x[1]);
            pk[k / 2 + 1] = C::KIND == kCacheBF16 ? ptx::pack_bf16(x[2], x[3]) : ptx::pack_f16(x[2], x[3]);
          }
          ptx::tmem_st16(s_addr + 16 * ch, pk);
#pragma unroll
          for (int w = 4; w >= 1; w >>= 1)
#pragma unroll
            for (int k = 0; k < w; ++k) ps[k] = ptx::add2(ps[k], ps[k + w]);
          sum = ptx::add2(sum, ps[0]);
        };
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          float s[32];
          load(ch, s);
          part(ch, s);
        }
      };
      if (masked)
        weights(std::true_type{});
      else
        weights(std::false_type{});
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        ptx::mbar_arrive(sy.bar(C::kBarPFull + buf));
        if (C::k8) ptx::mbar_arrive(sy.bar(C::kBarScaleEmpty + (int)(it % C::SCR)));
      }
      float a0, a1;
      ptx::f2unpack(sum, a0, a1);
      l += a0 + a1;
    }
    if (!ok) return;
    // ---- the segment's result: O and LSE, or a partial
    const float un = C::k8 ? __uint_as_float((uint32_t)(127 - lr) << 23) : 1.f;   // the power of two that O and l carry
    if (rs.nblk > 0) {
      if (!sy.wt.wait_warp(sy.bar(C::kBarOFull + (C::QT == 2 ? t : 0)), tiles & 1u, 0x3c)) return;
      ++tiles;
      ptx::tc_fence_after();
    }
    const float f = sg.direct ? (l == 0.f ? 0.f : 1.f / l) : un;
    const int64_t prow = (int64_t)sg.slot * C::RT + 128 * t + r;
    // through shared memory (the rows of Q, which no product reads any more), so
    // that a warp writes whole lines: a row to a thread costs 32 lines a store
    const uint32_t stage = sbase + C::kOffQ + t * C::kTileBytes + quarter * 4096;
    uint16_t* const o = static_cast<uint16_t*>(p.o);
    float* const part = p.part_o + (prow - lane) * D;
#pragma unroll 1
    for (int ch = 0; ch < D / 32; ++ch) {
      uint32_t v[32];
      if (rs.nblk > 0) {
        ptx::tmem_ld32(o_addr + 32 * ch, v);
        ptx::tmem_wait_ld();
        ptx::reg_fence(v);
      } else {
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = 0u;
      }
      __syncwarp();   // the chunk before was read
      if (sg.direct) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float a = __uint_as_float(v[8 * k + 2 * q]) * f, b = __uint_as_float(v[8 * k + 2 * q + 1]) * f;
            w[q] = p.q_bf16 ? ptx::pack_bf16(a, b) : ptx::pack_f16(a, b);
          }
          sts128(stage + lane * 128 + ((k ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int rr = 8 * i + lane / 4;
          const int64_t at = __shfl_sync(0xffffffffu, (long long)row_at, rr);
          const uint4 x = lds128(stage + rr * 128 + (((lane & 3) ^ (rr & 7)) << 4));
          if (at >= 0) *reinterpret_cast<uint4*>(o + at + 32 * ch + 8 * (lane & 3)) = x;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) w[q] = __float_as_uint(__uint_as_float(v[4 * k + q]) * f);
          sts128(stage + lane * 128 + ((k ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + lane / 8;
          const uint4 x = lds128(stage + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4));
          if (R - lane + rr < sg.rows) *reinterpret_cast<uint4*>(part + rr * D + 32 * ch + 4 * (lane & 7)) = x;
        }
      }
    }
    __syncwarp();   // before the next segment's Q
    if (have) {
      if (sg.direct) {
        const float lse = l == 0.f ? -CUDART_INF_F : (m_ref + __log2f(l) - (float)lr) * kLn2;
        if (p.s.cu != nullptr)
          p.lse[(int64_t)hq * p.s.total + sg.first + tok] = lse;
        else
          p.lse[((int64_t)sg.b * p.Hq + hq) * p.s.S + tok] = lse;
      } else {
        *reinterpret_cast<float2*>(p.part_ml + 2 * prow) = make_float2(l == 0.f ? -CUDART_INF_F : m_ref, l * un);
      }
    }
    // the next segment's product may overwrite O, and its Q rows this one's,
    // only after these reads
    ptx::tc_fence_before();
  }
}

// ------------------------------------------------------------------ kernel
template <class C>
__global__ void __launch_bounds__(C::kThreads, 1)
    kv_rows_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ KvAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* const tmem_holder = reinterpret_cast<uint32_t*>(smem + C::kOffMisc);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc + 4);
  int* const sm_warp = reinterpret_cast<int*>(smem + C::kOffMisc + 16);
  int* const cum = reinterpret_cast<int*>(smem + C::kOffCum);
  const uint32_t bars = sbase + C::kOffBar;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      uint32_t count = 1;
      if (i >= C::kBarRawEmpty && i < C::kBarKVEmpty) count = C::kConvWarps;   // raw_empty, kv_full
      if (i >= C::kBarQFull && i < C::kBarSFull) count = 4;        // a tile's four warps
      if (i >= C::kBarPFull && i < C::kBarOFull) count = 4;
      if (i >= C::kBarScale && i < C::kBarScaleEmpty) count = 2;   // both scale warps
      if (i >= C::kBarScaleEmpty && i < C::kBarSegFull) count = C::kSoftmaxWarps;
      if (i >= C::kBarSegEmpty) count = 1 + C::kScaleWarps + C::kConvWarps + C::kSoftmaxWarps;
      ptx::mbar_init(bars + 8u * i, count);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tk);
    ptx::prefetch_tmap(&tv);
  }
  if (warp == C::kMmaWarp) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_holder), C::kTmemCols);
    ptx::tmem_relinquish();
  }
  int own_total = 0;
  if (p.pass_own) {
    scan_units(p, C::RT, kRowsUnit, C::kThreads, cum, sm_warp);
    own_total = cum[p.s.B];
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= p.s.B; b += C::kThreads) p.cum[b] = cum[b];
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  launch_dependents();
  const int pre_units = (p.prefix_len + kRowsUnit - 1) / kRowsUnit;
  const int pre_total = p.prefix_tiles * pre_units;
  const int U = pre_total + own_total;
  const int n_ranges = min(p.ranges, U), my_range = blockIdx.x / p.Hk;
  int u_begin = 0, u_end = 0;
  if (my_range < n_ranges) {
    u_begin = range_start(my_range, n_ranges, U);
    u_end = range_start(my_range + 1, n_ranges, U);
  }
  const RowsSync<C> sy{bars, Waiter{abort_flag, p.s.status}, reinterpret_cast<RowsSegment*>(smem + C::kOffSeg)};
  if (warp >= C::kSoftmaxWarps) {
    if constexpr (C::kRebalance) ptx::setmaxnreg_dec<C::kRegsLow>();
    if (warp == C::kLoadWarp)
      rows_load_role<C>(&tk, &tv, p, sbase, sy, cum, u_begin, u_end, pre_units, pre_total);
    else if (warp == C::kMmaWarp) {
      if (lane == 0) rows_mma_role<C>(sbase, tmem, sy);
    } else if (C::k8 && warp < C::kConvWarp)
      rows_scale_role<C>(p, sbase, sy, warp - C::kScaleWarp);
    else
      rows_convert_role<C>(sbase, sy, warp - C::kConvWarp);
  } else {
    if constexpr (C::kRebalance) ptx::setmaxnreg_inc<C::kRegsHigh>();
    rows_softmax_role<C>(p, sbase, tmem, sy, warp >> 2, warp & 3);
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == C::kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, C::kTmemCols);
  }
  // set up early itself, this kernel must not end before its predecessor: the
  // merge waits for this one only
  wait_for_predecessor();
}

template <int D, int KIND, int QT>
cudaError_t launch_kv_rows_kind(const KvAttnLaunch& L) {
  using C = RowsCfg<D, KIND, QT>;
  const int smem = C::kSmemFixed + (L.p.s.B + 1) * 4;
  if (smem > 232448 && L.p.pass_own) return cudaErrorInvalidValue;
  auto kern = kv_rows_kernel<C>;
  static std::atomic<uint64_t> allowed{0};
  const uint64_t bit = 1ull << (L.device & 63);
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  return launch_early(kern, L.grid, C::kThreads, L.p.pass_own ? smem : C::kSmemFixed, L.stream, L.early, L.tk, L.tv, L.p);
}

template <int D, int KIND>
cudaError_t launch_kv_rows_qt(const KvAttnLaunch& L) {
  if constexpr (rows_max_qt(D) == 2) {
    if (L.qt == 2) return launch_kv_rows_kind<D, KIND, 2>(L);
  }
  return launch_kv_rows_kind<D, KIND, 1>(L);
}

template <int D>
cudaError_t launch_kv_rows(const KvAttnLaunch& L) {
  switch (L.kind) {
    case kCacheF16: return launch_kv_rows_qt<D, kCacheF16>(L);
    case kCacheBF16: return launch_kv_rows_qt<D, kCacheBF16>(L);
    case kCacheE4M3: return launch_kv_rows_qt<D, kCacheE4M3>(L);
    default: return launch_kv_rows_qt<D, kCacheI8>(L);
  }
}

}  // namespace fa
