// Attention of a few query rows over a paged K/V cache: single-token and
// drafted-token decoding, shared K/V heads, 16-bit or 8-bit caches, with or
// without a prefix that every sequence of the batch shares.
//
// Row (i, g) of a work item is query token i of head hk * G + g: the G query
// heads that share a K/V head and all query tokens of a sequence (or, for the
// shared prefix, of all sequences) are rows of one matrix product, so K and V
// are read once for every 16 of them.
//
//   x_ij = (q_i . kcode_j) ks_j scale log2 e,  p_ij = 2^(x_ij - m_i),
//   l_i = sum_j p_ij,  O_i = (sum_j p_ij vs_j vcode_j) / l_i,
//   LSE_i = (m_i + log2 l_i) ln 2
//
// with the running max m_i moved lazily (O and l are rescaled only when a
// tile's max exceeds it by more than 8, so p <= 2^8).
//
// HBM-bound: a K/V byte is used by at most 8 * NB rows. The tensor core is
// used through mma.sync, keys and head elements on its 16-row side, query rows
// on its 8-column side, so that eight rows (single tokens, up to eight shared
// heads) waste nothing. A tcgen05 product is 128 rows high and needs its
// operands as 16-bit tiles in shared memory, which an 8-bit cache does not
// give; here the codes go from shared memory to registers and become f16 there.
//
// Arithmetic with an 8-bit cache. Both products run in f16, where every code is
// exact, with fp32 accumulation. Query rows are scaled by a power of two so that
// their largest element is in [2^14, 2^15) (bf16 queries; fp16 ones are taken as
// they are): every element is held to 2^-38 of the row's largest. (e4m3 products
// on the raw codes, a query as the sum of two or three e4m3 numbers per element,
// lose what lies below 2^-17 of the largest, and are slower where it counts: 8
// rows 124 against 123 us, 16 rows 172 against 134, B = 64 of 2048 .. 8192 keys,
// 8 heads of 128.) The weights p vs, whose range is that of the V scales, are
// held at a power of two per row, 2^lr, lr <= 100, chosen such that the largest
// is about 2^6 and none reaches 2^16, and rounded to f16 (11 bits). 2^lr sits in
// the exponent's argument, so O and l both carry it; it moves only when it has
// to. l takes the unrounded p.
//
// Work split. The keys of every (sequence, K/V head, row tile) are cut into
// tiles of 16 or 32 keys; all tiles form one line, cut into equal contiguous
// ranges, one per warp (kv_work.cuh), whatever the lengths: a ragged batch loads
// every warp alike. A warp that holds all tiles of an item
// writes O and LSE; otherwise it writes a partial (O unnormalised, m, l) and a
// second kernel joins them. Nothing is shared between warps, so there is no
// barrier after the start, and the end of one item overlaps the loads of the
// next: each warp streams its range through a private ring of slots, K and V
// tiles in turn, that its lanes fill with TMA boxes (a box is a page, or part
// of one), running ahead across items. (A range per CTA, its warps' partials
// joined through shared memory, spent a third of its time on the barriers and
// empty pipelines at the items' ends.) Measured: B = 64, 2048 .. 8192 keys, 32
// query and 8 K/V heads of 128, e4m3: 118 us alone, 5.9 TB/s, 86 % of a copy's
// rate.
//
// Lane layout. The products' operand order along a contracted axis is free,
// so it is chosen such that every shared-memory read is a 16-byte vector
// without bank conflicts under the swizzle that TMA wrote: thread (g, c) =
// (lane / 4, lane % 4) reads of the key rows g, g + 8 of 16 the chunks 2c,
// 2c + 1 of each 128-byte box (K), and of the key rows 2c, 2c + 1, 2c + 8,
// 2c + 9 the chunk g (V), whose elements are interleaved in pairs of keys. The
// weights change sides between the products by 8 x 8 transposes (movmatrix).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <type_traits>

#include "kv_codes.cuh"
#include "kv_work.cuh"
#include "pipeline.cuh"
#include "ptx.cuh"

namespace fa {

template <int D_, int KIND_, int NB_>
struct KvCfg {
  static constexpr int D = D_, KIND = KIND_, NB = NB_;
  static constexpr bool k8 = cache_is_8bit(KIND);
  static constexpr int EB = k8 ? 1 : 2;
  static constexpr int RB = D * EB < 128 ? D * EB : 128;    // bytes of a box row
  static constexpr int BC = RB / EB;                         // elements of a box row
  static constexpr int BOXES = D / BC;
  static constexpr int CH = RB / 64;                         // 16-byte chunks of a K box row per thread
  static constexpr int EPC = 16 / EB;                        // elements of a chunk
  static constexpr int SPC = EPC / 4;                        // k16 steps of a chunk
  static constexpr int VB = RB / 8;                          // bytes of a V box row per thread (16, or 8)
  static constexpr int VE = VB / EB;                         // its elements
  static constexpr KvAttnGeom geom = kv_attn_geom(D, EB, NB);
  static constexpr int W = geom.warps, KT = geom.keys, NS = geom.slots, CTAS = geom.ctas;
  static constexpr int RT = 8 * NB;
  static constexpr int kBoxBytes = KT * RB;
  static constexpr int kSlotBytes = BOXES * kBoxBytes;       // K or V of a tile
  static constexpr int MT = KT / 16, OT = D / 16, QS = D / 16;
  static constexpr int kThreads = 32 * W;
  static constexpr float kTau = 8.f;
  static constexpr int QW = D / 8;                           // Q fragments, 4 bytes each: two of a k16 step
  static constexpr bool kQRegs = D * NB <= 128;              // they are in registers, else in shared memory
  static constexpr int SR = NS <= 4 ? 2 : 4;                 // tiles whose scales are held
  static constexpr int SEGS = 4;                             // segments found ahead: at most (NS - 1) / 2 + 2 are open
  // shared memory, from a 1024-byte aligned base; all but cum is per warp
  static constexpr int kOffQ = W * NS * kSlotBytes;                        // [W][NB][QW / 2][32] uint2
  static constexpr int kOffScale = kOffQ + (kQRegs ? 0 : W * NB * QW * 128);   // [W][SR][2][KT] fp32
  static constexpr int kOffSeg = kOffScale + (k8 ? W * SR * 2 * KT * 4 : 0);   // [W][SEGS] KvSegment
  static constexpr int kOffBar = kOffSeg + W * SEGS * 64;
  static constexpr int kOffMisc = kOffBar + W * NS * 8;                    // abort flag, warp sums
  static constexpr int kOffCum = kOffMisc + 16 + 64;                       // cum[B + 1]
  static constexpr int kSmemFixed = kOffCum + 1024;
  static_assert(kSmemFixed == kv_attn_smem(D, EB, NB), "shared memory of the geometry");
  static_assert(BOXES * (KT / 16) <= 32, "one lane per TMA box");
  static_assert(sizeof(KvSegment) <= 64, "segment slots");
  static_assert(NS >= 3 && CTAS * (kSmemFixed + 2048) <= 233472, "shared memory");
};

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, bool bf16) {
  if (bf16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit elements, two per thread, transposed across the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ---------------------------------------------------------------- kernel
template <class C>
__global__ void __launch_bounds__(C::kThreads, C::CTAS)
    kv_attn_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ KvAttnParams p) {
  constexpr int D = C::D, W = C::W, KT = C::KT, NS = C::NS, NB = C::NB, RT = C::RT, RB = C::RB, MT = C::MT;
  constexpr float kNone = -3e38f;   // m of a row that has seen no key
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = ptx::smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, c = lane & 3;
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  int* const sm_warp = reinterpret_cast<int*>(smem + C::kOffMisc + 16);
  int* const cum = reinterpret_cast<int*>(smem + C::kOffCum);
  const uint32_t bar0 = sbase + C::kOffBar + 8u * (warp * NS);
  const uint32_t ring = sbase + warp * NS * C::kSlotBytes;
  const uint32_t sring = sbase + C::kOffScale + warp * C::SR * 2 * KT * 4;
  const uint32_t qbuf = sbase + C::kOffQ + warp * NB * C::QW * 128;
  uint8_t* const segs = smem + C::kOffSeg + warp * C::SEGS * 64;

  if (threadIdx.x == 0) {
    for (int i = 0; i < W * NS; ++i) ptx::mbar_init(sbase + C::kOffBar + 8u * i, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tk);
    ptx::prefetch_tmap(&tv);
  }
  scan_units(p, RT, KT, C::kThreads, cum, sm_warp);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= p.s.B; b += C::kThreads) p.cum[b] = cum[b];
  const int pre_units = (p.prefix_len + KT - 1) / KT;
  const int pre_total = p.prefix_tiles * pre_units;
  const int U = pre_total + cum[p.s.B];
  const int worker = blockIdx.x * W + warp;
  const int my_range = worker / p.Hk, my_head = worker - my_range * p.Hk;
  const int n_ranges = min(p.ranges, U);
  launch_dependents();
  int u_begin = 0, u_end = 0;
  if (my_range < n_ranges) {
    u_begin = range_start(my_range, n_ranges, U);
    u_end = range_start(my_range + 1, n_ranges, U);
  }
  const Waiter wt{abort_flag, p.s.status};

  // this lane's part of a tile's copies: box (box_row, box_col) of K, and of V
  const int box_row = lane / C::BOXES * p.box_rows, box_col = lane % C::BOXES;
  const bool box_mine = box_row < KT;
  const uint32_t box_dst = ring + box_col * C::kBoxBytes + box_row * RB;
  const int dead_row = p.s.num_pages * p.s.page_size;   // past the cache: TMA fills zeros

  // ---- the filling side: runs up to NS - 1 halves (K or V of a tile) ahead
  int u_fill = u_begin;              // next tile to be looked up
  int f_seg = 0;                     // segments found so far
  const int* f_table = nullptr;
  int f_key = 0, f_last = 0, f_len = 0;   // next key, end of the segment's tiles, of the keys
  int f_tiles = 0;                   // tiles whose copies have begun
  // the tile to be copied next: first key (-1: no tile), this lane's page
  // (as read, until the copy of K begins; then -1 for none)
  int t_key = -1, pg = -1;
  bool pg_live = false;
  uint32_t is_slot = 0, issued = 0;
  // find the next tile of the range: its first key and this lane's page
  auto next_tile = [&]() {
    t_key = -1;
    if (f_key >= f_last) {
      if (u_fill >= u_end) return;
      KvSegment sg;
      if (lane == 0) {
        sg = find_segment(p, RT, KT, cum, u_fill, u_begin, u_end, pre_units, pre_total, my_range, p.ranges, my_head);
        *reinterpret_cast<KvSegment*>(segs + 64 * (f_seg % C::SEGS)) = sg;
      }
      __syncwarp();
      sg = *reinterpret_cast<const KvSegment*>(segs + 64 * (f_seg % C::SEGS));
      if (sg.take <= 0) {            // the lengths changed under the call: no more
        u_fill = u_end;
        return;
      }
      ++f_seg;
      u_fill += sg.take;
      f_table = sg.pre ? p.prefix_pages : p.s.block_table + (int64_t)sg.b * p.s.max_pages;
      f_len = sg.len;
      f_key = sg.at * KT;
      f_last = f_key + sg.take * KT;
    }
    t_key = f_key;
    f_key += KT;
    const int key = t_key + lane;
    pg_live = lane < KT && key < f_len;
    if (pg_live) {
      int index, off;
      page_of(p.s, key, index, off);
      pg = __ldg(f_table + index);   // looked at when the copy begins, one product later
    }
  };
  // begin the copy of K (with the tile's scales) or V of the tile found
  auto issue = [&](bool is_v) {
    if (t_key >= 0) {
      const uint32_t b = bar0 + 8u * is_slot;
      if (!is_v) {
        if (pg_live && (unsigned)pg >= (unsigned)p.s.num_pages) {
          atomicOr(p.s.status, kDevBadSeqlens);
          pg_live = false;
        }
        if (!pg_live) pg = -1;
      }
      if (lane == 0) ptx::mbar_arrive_expect_tx(b, C::kSlotBytes);
      const int box_page = __shfl_sync(0xffffffffu, pg, box_row & 31);   // also orders the lanes
      if (box_mine) {
        int index, off;
        page_of(p.s, t_key + box_row, index, off);
        ptx::tma_load_2d(box_dst + is_slot * C::kSlotBytes, is_v ? &tv : &tk, my_head * D + box_col * C::BC,
                         box_page >= 0 ? box_page * p.s.page_size + off : dead_row, b);
      }
      if (C::k8 && !is_v && lane < KT) {
        int index, off;
        page_of(p.s, t_key + lane, index, off);
        const int64_t at = pg >= 0 ? ((int64_t)pg * p.Hk + my_head) * p.s.page_size + off : 0;
        const uint32_t sd = sring + ((f_tiles % C::SR) * 2 * KT + lane) * 4;
        cp_async4(sd, p.k_scale + at, pg >= 0);
        cp_async4(sd + KT * 4, p.v_scale + at, pg >= 0);
      }
      is_slot = is_slot + 1 == NS ? 0 : is_slot + 1;
      ++issued;
      if (is_v) {
        ++f_tiles;
        next_tile();
      }
    }
    cp_async_commit();
  };
  next_tile();
#pragma unroll
  for (int h = 0; h < NS - 1; ++h) issue(h & 1);

  uint32_t cs_slot = 0, cs_phase = 0, read = 0;   // slot to be read next; halves read
  int tile = 0;                                   // tiles read
  bool ok = true;
  int u = u_begin;
  for (int seg = 0; ok && u < u_end; ++seg) {
    __syncwarp();
    if (seg >= f_seg) break;           // the filling side found no more
    const KvSegment sg = *reinterpret_cast<const KvSegment*>(segs + 64 * (seg % C::SEGS));
    const int hk = my_head, row0 = sg.mt * RT, len = sg.len;
    u += sg.take;

    // ---- how many keys the rows 2c, 2c + 1 of each eight see
    int lim[NB][2];
    int min_lim = len;
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int R = row0 + 8 * b + 2 * c + j;
        lim[b][j] = R < sg.rows ? row_limit(p, sg, R) : len;   // a missing row asks for no mask
        min_lim = min(min_lim, lim[b][j]);
      }
    min_lim = __reduce_min_sync(0xffffffffu, min_lim);

    // ---- Q fragments: row g of each eight, the elements of this thread's
    // chunks in order (box, chunk, element), four (two words) at a time; and the
    // rows' factors: the scores of a row are its products times rowf
    uint32_t qf[C::kQRegs ? NB : 1][C::QW];
    float rowf[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int R = row0 + 8 * b + g;
      uint2 v[C::QS];
      const bool have = R < sg.rows;
      const int t = have ? R / p.G : 0;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                            ((int64_t)(sg.first + t) * p.Hq + hk * p.G + (have ? R - t * p.G : 0)) * D;
      uint32_t m = 0;
#pragma unroll
      for (int s = 0; s < C::QS; s += 2) {   // eight elements at a time
        const int st = s % C::SPC, i = (s / C::SPC) % C::CH, bx = s / (C::SPC * C::CH);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (have) x = __ldg(reinterpret_cast<const uint4*>(src + bx * C::BC + (c * C::CH + i) * C::EPC + 4 * st));
        v[s] = make_uint2(x.x, x.y);
        v[s + 1] = make_uint2(x.z, x.w);
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
      }
      float qs = 1.f;
      if (C::k8 && p.q_bf16) {
        uint32_t e = max(m & 0xffffu, m >> 16);
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
        float f = 1.f;
        if (e != 0 && e < 0x7f80u) {
          // the largest element times 2^sh is in [2^14, 2^15) (less where it is
          // below 2^-100); sh in [-113, 114]
          const int sh = min(14 - ((int)(e >> 7) - 127), 114);
          f = __uint_as_float((uint32_t)(127 + sh) << 23);
          qs = __uint_as_float((uint32_t)(127 - sh) << 23);
        }
#pragma unroll
        for (int s = 0; s < C::QS; ++s) {
          v[s].x = ptx::pack_f16(__uint_as_float(v[s].x << 16) * f, __uint_as_float(v[s].x & 0xffff0000u) * f);
          v[s].y = ptx::pack_f16(__uint_as_float(v[s].y << 16) * f, __uint_as_float(v[s].y & 0xffff0000u) * f);
        }
      }
#pragma unroll
      for (int s = 0; s < C::QS; ++s) {
        if (C::kQRegs) {
          qf[C::kQRegs ? b : 0][2 * s] = v[s].x;
          qf[C::kQRegs ? b : 0][2 * s + 1] = v[s].y;
        } else {
          sts64(qbuf + ((b * C::QS + s) * 32 + lane) * 8, v[s]);   // read back by the same lane
        }
      }
      rowf[b][0] = C::k8 ? __shfl_sync(0xffffffffu, qs, 8 * c) : p.c;
      rowf[b][1] = C::k8 ? __shfl_sync(0xffffffffu, qs, 8 * c + 4) : p.c;
    }
    auto q_words = [&](int b, int s) -> uint2 {   // fragments 2 s, 2 s + 1
      return C::kQRegs ? make_uint2(qf[C::kQRegs ? b : 0][2 * s], qf[C::kQRegs ? b : 0][2 * s + 1])
                       : lds64(qbuf + ((b * C::QS + s) * 32 + lane) * 8);
    };

    // ---- the warp's online softmax over its tiles
    float o[NB][C::OT][4];
    float m_ref[NB][2], l[NB][2];
    int lr[NB][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int t = 0; t < C::OT; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[b][t][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m_ref[b][j] = kNone;
        l[b][j] = 0.f;
        lr[b][j] = C::k8 ? 100 : 0;
      }
    }
    for (int i = 0; i < sg.take; ++i, ++tile) {
      const int key0 = (sg.at + i) * KT;
      // ---- S = K Q^T: 16 keys by 8 rows at a time
      issue((NS - 1) & 1);
      cp_async_wait<NS - 1>();
      if (!(ok = wt.wait_warp(bar0 + 8u * cs_slot, cs_phase, 0x20))) break;
      __syncwarp();   // the other lanes' scales are in shared memory too
      const uint32_t kbuf = ring + cs_slot * C::kSlotBytes;
      float sc[MT][NB][4];
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) sc[t][b][j] = 0.f;
#pragma unroll
      for (int bx = 0; bx < C::BOXES; ++bx)
#pragma unroll
        for (int ch = 0; ch < C::CH; ++ch) {
          uint4 kw[MT][2];
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int chunk = (c * C::CH + ch) ^ (RB == 128 ? g : (g >> 1) & 3);
              kw[t][r] = lds128(kbuf + bx * C::kBoxBytes + (16 * t + 8 * r + g) * RB + chunk * 16);
            }
#pragma unroll
          for (int st = 0; st < C::SPC; ++st) {
            const int s = (bx * C::CH + ch) * C::SPC + st;
            uint2 q[NB];
#pragma unroll
            for (int b = 0; b < NB; ++b) q[b] = q_words(b, s);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              const uint32_t w0[4] = {kw[t][0].x, kw[t][0].y, kw[t][0].z, kw[t][0].w};
              const uint32_t w1[4] = {kw[t][1].x, kw[t][1].y, kw[t][1].z, kw[t][1].w};
              uint32_t a[4];
              if (C::k8) {
                codes_to_f16<C::KIND>(w0[st], a[0], a[2]);
                codes_to_f16<C::KIND>(w1[st], a[1], a[3]);
              } else {
                a[0] = w0[(2 * st) & 3];
                a[2] = w0[(2 * st + 1) & 3];
                a[1] = w1[(2 * st) & 3];
                a[3] = w1[(2 * st + 1) & 3];
              }
#pragma unroll
              for (int b = 0; b < NB; ++b) mma_16816(sc[t][b], a, q[b].x, q[b].y, C::KIND == kCacheBF16);
            }
          }
        }
      ++read;
      cs_slot = cs_slot + 1 == NS ? (cs_phase ^= 1u, 0u) : cs_slot + 1;

      // ---- scores -> weights; element (t, b, j): key 16 t + g + 8 (j >> 1),
      // row 8 b + 2 c + (j & 1)
      const bool masked = key0 + KT > min_lim;
      const uint32_t srow = sring + ((tile % C::SR) * 2 * KT) * 4;
      if (C::k8) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = lds32(srow + (16 * t + 8 * r + g) * 4) * p.c;
            const uint64_t f2 = ptx::f2pack(f, f);
#pragma unroll
            for (int b = 0; b < NB; ++b)
              ptx::f2unpack(ptx::mul2(ptx::f2pack(sc[t][b][2 * r], sc[t][b][2 * r + 1]), f2), sc[t][b][2 * r], sc[t][b][2 * r + 1]);
          }
      }
      if (masked) {
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (key0 + 16 * t + g + 8 * (j >> 1) >= lim[b][j & 1]) sc[t][b][j] = -CUDART_INF_F;
      }
      float vs[MT][2];
      float thr0 = C::kTau;      // 8-bit: 15 - log2 of a bound on the tile's V scales
      if (C::k8) {
        const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(lane < KT ? lds32(srow + (KT + lane) * 4) : 0.f) >> 23);
        thr0 = (float)(15 + 126 - (int)e);
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
          for (int r = 0; r < 2; ++r) vs[t][r] = lds32(srow + (KT + 16 * t + 8 * r + g) * 4);
      }
      float mx[NB][2];
      bool need = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaxf(sc[0][b][j], sc[0][b][2 + j]);
#pragma unroll
          for (int t = 1; t < MT; ++t) x = ptx::max3(x, sc[t][b][j], sc[t][b][2 + j]);
          mx[b][j] = x;
          // how far above m_ref: not past tau, and no weight past 2^15
          const float up = x == -CUDART_INF_F ? x : fmaf(x, rowf[b][j], -m_ref[b][j]);
          const float thr = C::k8 ? thr0 - (float)lr[b][j] : C::kTau;
          need = need || up > fminf(C::kTau, thr) || (C::k8 && thr < 0.f);
        }
      if (__any_sync(0xffffffffu, need)) {
        float corr[NB][2];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float x = mx[b][j];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            x = x == -CUDART_INF_F ? x : x * rowf[b][j];
            float cr = 1.f;
            if (x > m_ref[b][j] + C::kTau) {
              if (m_ref[b][j] != kNone) cr = ptx::ex2(m_ref[b][j] - x);   // else nothing was summed yet
              m_ref[b][j] = x;
            }
            if (C::k8) {
              // the largest weight at the new m; where it belongs: [2^6, 2^7).
              // The power goes up by at most what O goes down by, and down as
              // far as it takes
              float um = 0.f;
#pragma unroll
              for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int r = 0; r < 2; ++r)
                  um = fmaxf(um, sc[t][b][2 * r + j] == -CUDART_INF_F
                                     ? 0.f : ptx::ex2(fmaf(sc[t][b][2 * r + j], rowf[b][j], -m_ref[b][j])) * vs[t][r]);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) um = fmaxf(um, __shfl_xor_sync(0xffffffffu, um, d));
              const int e = um > 0.f ? (int)(__float_as_uint(um) >> 23) - 127 : -200;
              const int old = lr[b][j];
              int now = old;
              if (e + old >= 15) now = 6 - e;
              else if (cr < 1.f) now = min(6 - e, old + (cr > 0.f ? 126 - (int)(__float_as_uint(cr) >> 23) : 200));
              now = max(min(now, 100), -120);
              cr = cr == 0.f ? 0.f : cr * ptx::ex2((float)(now - old));
              lr[b][j] = now;
            }
            l[b][j] *= cr;
            corr[b][j] = cr;
          }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint64_t c2 = ptx::f2pack(corr[b][0], corr[b][1]);
#pragma unroll
          for (int t = 0; t < C::OT; ++t) {
            ptx::f2unpack(ptx::mul2(ptx::f2pack(o[b][t][0], o[b][t][1]), c2), o[b][t][0], o[b][t][1]);
            ptx::f2unpack(ptx::mul2(ptx::f2pack(o[b][t][2], o[b][t][3]), c2), o[b][t][2], o[b][t][3]);
          }
        }
      }
      uint32_t pw[MT][NB][2];   // weights of 8 keys by 8 rows, rows first
      // (one branch on the mask: selects in the common path cost as much as the rest)
      auto weights = [&](auto mask) {
        constexpr bool kMask = decltype(mask)::value;
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          const uint64_t f2 = ptx::f2pack(rowf[b][0], rowf[b][1]);
          const uint64_t mu2 = ptx::f2pack((float)lr[b][0] - m_ref[b][0], (float)lr[b][1] - m_ref[b][1]);
          uint64_t sum = ptx::f2pack(l[b][0], l[b][1]);
#pragma unroll
          for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              float x0, x1;
              ptx::f2unpack(ptx::fma2(ptx::f2pack(sc[t][b][2 * r], sc[t][b][2 * r + 1]), f2, mu2), x0, x1);
              x0 = ptx::ex2(x0);
              x1 = ptx::ex2(x1);
              const int key = key0 + 16 * t + g + 8 * r;
              if (kMask) {   // with scale 0, -inf * 0 would be NaN
                if (key >= lim[b][0]) x0 = 0.f;
                if (key >= lim[b][1]) x1 = 0.f;
              }
              sum = ptx::add2(sum, ptx::f2pack(x0, x1));
              if (C::k8) {
                ptx::f2unpack(ptx::mul2(ptx::f2pack(x0, x1), ptx::f2pack(vs[t][r], vs[t][r])), x0, x1);
                if (kMask) {   // whatever the scale holds
                  if (key >= lim[b][0]) x0 = 0.f;
                  if (key >= lim[b][1]) x1 = 0.f;
                }
              }
              pw[t][b][r] = transpose8(C::KIND == kCacheBF16 ? ptx::pack_bf16(x0, x1) : ptx::pack_f16(x0, x1));
            }
          ptx::f2unpack(sum, l[b][0], l[b][1]);
        }
      };
      if (masked)
        weights(std::true_type{});
      else
        weights(std::false_type{});

      // ---- O += V^T P
      issue(NS & 1);
      cp_async_wait<NS - 1>();
      if (!(ok = wt.wait_warp(bar0 + 8u * cs_slot, cs_phase, 0x21))) break;
      const uint32_t vbuf = ring + cs_slot * C::kSlotBytes;
      if (key0 + KT > len) {
        // rows past the end hold whatever the page held: their weights are 0,
        // but 0 times a NaN is not
        for (int r = len - key0; r < KT; ++r)
          for (int q = lane; q < C::BOXES * RB / 16; q += 32) {
            const uint32_t a = vbuf + (q / (RB / 16)) * C::kBoxBytes + r * RB + (q % (RB / 16)) * 16;
            asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(0) : "memory");
          }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int bx = 0; bx < C::BOXES; ++bx) {
          constexpr int NW = C::VB / 4;   // words of a row that a thread reads: 4, or 2
          uint32_t w[4][NW];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int row = 16 * t + 2 * c + (r & 1) + 8 * (r >> 1);
            const uint32_t a0 = vbuf + bx * C::kBoxBytes + row * RB;
            if (RB == 128) {
              const uint4 v = lds128(a0 + ((g ^ ((2 * c + (r & 1)) & 7)) << 4));
              w[r][0] = v.x;
              w[r][1] = v.y;
              w[r][NW - 2] = v.z;
              w[r][NW - 1] = v.w;
            } else {
              const uint2 v = lds64(a0 + (((g >> 1) ^ c) << 4) + (g & 1) * 8);
              w[r][0] = v.x;
              w[r][1] = v.y;
            }
          }
#pragma unroll
          for (int q = 0; q < NW; ++q) {
            constexpr int TW = 2 / C::EB;   // 16-row tiles of O per word
            const int ot = bx * (C::BC / 16) + TW * q;
            if (C::k8) {
              // bytes of two keys interleaved, then two elements of each pair
              uint32_t a[2][4];
              codes_to_f16<C::KIND>(__byte_perm(w[0][q], w[1][q], 0x5140), a[0][0], a[0][1]);
              codes_to_f16<C::KIND>(__byte_perm(w[2][q], w[3][q], 0x5140), a[0][2], a[0][3]);
              codes_to_f16<C::KIND>(__byte_perm(w[0][q], w[1][q], 0x7362), a[1][0], a[1][1]);
              codes_to_f16<C::KIND>(__byte_perm(w[2][q], w[3][q], 0x7362), a[1][2], a[1][3]);
#pragma unroll
              for (int x = 0; x < TW; ++x)
#pragma unroll
                for (int b = 0; b < NB; ++b) mma_16816(o[b][ot + x], a[x], pw[t][b][0], pw[t][b][1], false);
            } else {
              const uint32_t a[4] = {__byte_perm(w[0][q], w[1][q], 0x5410), __byte_perm(w[0][q], w[1][q], 0x7632),
                                     __byte_perm(w[2][q], w[3][q], 0x5410), __byte_perm(w[2][q], w[3][q], 0x7632)};
#pragma unroll
              for (int b = 0; b < NB; ++b) mma_16816(o[b][ot], a, pw[t][b][0], pw[t][b][1], C::KIND == kCacheBF16);
            }
          }
        }
      ++read;
      cs_slot = cs_slot + 1 == NS ? (cs_phase ^= 1u, 0u) : cs_slot + 1;
      __syncwarp();   // every lane has read both slots: they may be filled again
    }
    if (!ok) break;

    // ---- the segment's result: O and LSE, or a partial
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 8 * b + 2 * c + j, R = row0 + r;
        float x = l[b][j];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        if (R >= sg.rows) continue;
        // the power of two that O and l carry
        const float un = C::k8 ? __uint_as_float((uint32_t)(127 - lr[b][j]) << 23) : 1.f;
        // tile t holds elements 2 t, 2 t + 1 of the thread's VE of a box
        if (sg.direct) {
          const int t = R / p.G, hq = hk * p.G + (R - t * p.G);
          const float inv = x == 0.f ? 0.f : 1.f / x;
          uint16_t* dst = static_cast<uint16_t*>(p.o) + ((int64_t)(sg.first + t) * p.Hq + hq) * D + g * C::VE;
#pragma unroll
          for (int bx = 0; bx < C::BOXES; ++bx)
#pragma unroll
            for (int e = 0; e < C::VE; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int t2 = bx * (C::BC / 16) + e / 2 + q;
                const float lo = o[b][t2][j] * inv, hi = o[b][t2][2 + j] * inv;
                w[q] = p.q_bf16 ? ptx::pack_bf16(lo, hi) : ptx::pack_f16(lo, hi);
              }
              *reinterpret_cast<uint4*>(dst + bx * C::BC + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          if (g == 0) {
            const float lse = x == 0.f ? -CUDART_INF_F : (m_ref[b][j] + __log2f(x) - (float)lr[b][j]) * kLn2;
            if (p.s.cu != nullptr)
              p.lse[(int64_t)hq * p.s.total + sg.first + t] = lse;
            else
              p.lse[((int64_t)sg.b * p.Hq + hq) * p.s.S + t] = lse;
          }
        } else {
          const int64_t prow = (int64_t)sg.slot * RT + r;
          float* dst = p.part_o + prow * D + g * C::VE;
#pragma unroll
          for (int bx = 0; bx < C::BOXES; ++bx)
#pragma unroll
            for (int e = 0; e < C::VE; e += 4) {
              const int t2 = bx * (C::BC / 16) + e / 2;
              *reinterpret_cast<float4*>(dst + bx * C::BC + e) =
                  make_float4(o[b][t2][j] * un, o[b][t2][2 + j] * un, o[b][t2 + 1][j] * un, o[b][t2 + 1][2 + j] * un);
            }
          if (g == 0)
            *reinterpret_cast<float2*>(p.part_ml + 2 * prow) = make_float2(x == 0.f ? -CUDART_INF_F : m_ref[b][j], x * un);
        }
      }
  }
  cp_async_wait<0>();
  // copies that nobody waited for (a wait gave up): let them land
  for (; read < issued; ++read) {
    wt.drain(bar0 + 8u * cs_slot, cs_phase);
    cs_slot = cs_slot + 1 == NS ? (cs_phase ^= 1u, 0u) : cs_slot + 1;
  }
  // set up early itself, this kernel must not end before its predecessor: the
  // merge waits for this one only
  wait_for_predecessor();
}

template <int D, int KIND, int NB>
cudaError_t launch_kv_attn_kind(const KvAttnLaunch& L) {
  using C = KvCfg<D, KIND, NB>;
  const int smem = C::kSmemFixed + (L.p.s.B + 1) * 4;
  if (smem > 232448) return cudaErrorInvalidValue;
  auto kern = kv_attn_kernel<C>;
  // once per device: the most shared memory there is, so that later calls need not ask
  static std::atomic<uint64_t> allowed{0};
  const uint64_t bit = 1ull << (L.device & 63);
  if (!(allowed.load(std::memory_order_acquire) & bit)) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_release);
  }
  return launch_early(kern, L.grid, C::kThreads, smem, L.stream, L.early, L.tk, L.tv, L.p);
}

template <int D, int KIND>
cudaError_t launch_kv_attn_nb(const KvAttnLaunch& L) {
  return L.nb == 1 ? launch_kv_attn_kind<D, KIND, 1>(L) : launch_kv_attn_kind<D, KIND, 2>(L);
}

template <int D>
cudaError_t launch_kv_attn(const KvAttnLaunch& L) {
  switch (L.kind) {
    case kCacheF16: return launch_kv_attn_nb<D, kCacheF16>(L);
    case kCacheBF16: return launch_kv_attn_nb<D, kCacheBF16>(L);
    case kCacheE4M3: return launch_kv_attn_nb<D, kCacheE4M3>(L);
    default: return launch_kv_attn_nb<D, kCacheI8>(L);
  }
}

}  // namespace fa
