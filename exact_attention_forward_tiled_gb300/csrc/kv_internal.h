// Internal interface of the cache-side operators (rotary positions, the paged
// K/V cache that is quantised as it is written, attention over it) between
// their C-ABI front end (kv_api.cu) and the kernel translation units.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

// The current device's state (fa_api.cu): its number, SM count and status word. FA_OK or
// the FA_ERR_* code to report.
int device_state(int* device, int* num_sms, int** status);
// 2-D tensor map over a [rows, cols] row-major matrix (fa_api.cu).
int encode_map(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int elem_bytes, uint64_t cols, uint64_t rows,
               uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle);

// ------------------------------------------------------------------ rotary
constexpr int kRopeMaxPairs = 128;   // D <= 256
struct RopeParams {
  const void* x[2];            // q, k: [T, H, D] by strides (elements)
  void* y[2];
  int64_t xs_t[2], xs_h[2], ys_t[2], ys_h[2];
  int H[2];
  int in_place[2];             // y is x with the same strides: what passes through is there already
  const int* pos;              // [n_axes, T]
  int T, D, rot;
  int inverse;
  uint64_t freq[kRopeMaxPairs];   // frequency of each pair, in 2^-64 turns per position
  uint8_t axis[kRopeMaxPairs];
};
cudaError_t launch_rope(const RopeParams& p, bool bf16, bool interleaved, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------------ paged cache
// Element kinds of a cache.
enum CacheKind : int { kCacheF16 = 0, kCacheBF16 = 1, kCacheE4M3 = 2, kCacheI8 = 3 };
constexpr bool cache_is_8bit(int kind) { return kind >= kCacheE4M3; }

// What append, read and the attention kernels know of a cache and of the
// sequences in it.
struct PagedSeqs {
  const int* block_table;   // [B, max_pages]
  const int* seqlens_k;     // [B]
  const int* cu;            // packed rows: prefix sums [B + 1], or nullptr (fixed: S rows per sequence)
  int B, S;                 // sequences; rows of each (fixed) or at most (packed)
  int total;                // rows of the packed (or B * S) side
  int num_pages, page_size, page_shift, max_pages;   // page_shift: log2(page_size), -1 if none
  int* status;
};

struct CacheParams {
  PagedSeqs s;
  // append: k, v [total, H, D] 16-bit by strides (elements) -> pages;
  // read: pages -> k, v [total, H, D] contiguous
  void* x[2];
  int64_t xs_t[2], xs_h[2];
  void* pages[2];           // [num_pages, page_size, H, D]
  float* scale[2];          // [num_pages, H, page_size], 8-bit caches only
  int H, D;
};
cudaError_t launch_kv_append(const CacheParams& p, int kind, bool bf16, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_read(const CacheParams& p, int kind, bool bf16, int num_sms, cudaStream_t stream);

// ------------------------------------------------------------------ attention over the cache
struct KvAttnParams {
  PagedSeqs s;              // cu / S / total: the query side
  const void* q;            // [total, Hq, D] 16-bit
  void* o;                  // [total, Hq, D], type of q
  float* lse;               // fixed: [B, Hq, S]; packed: [Hq, total]
  const float* k_scale;     // [num_pages, Hk, page_size], 8-bit caches
  const float* v_scale;
  int Hq, Hk, G;            // G = Hq / Hk query heads share a K/V head
  int q_bf16;
  int causal;
  float c;                  // softmax scale * log2(e)
  // shared prefix: keys 0 .. prefix_len - 1 of every sequence, in the pages of
  // prefix_pages [ceil(prefix_len / page_size)]; the sequence's own keys follow
  const int* prefix_pages;
  int prefix_len;
  int prefix_tiles;         // row tiles of the prefix, 0 if it is no part of this launch
  int ranges;               // of the work line; workers: ranges * Hk
  int pass_own;             // the sequences' own keys are part of this launch's work line
  int most_units;           // of the sequences' own keys, for any lengths and row counts within their bounds
  int direct;               // an item that one worker holds whole is written to O and LSE (no prefix to join)
  int box_rows;             // rows of a TMA box of the cache
  // workspace
  float* part_o;            // [slots, row tile, D] unnormalised partial O
  float* part_ml;           // [slots, row tile, 2] running max (log2 units) and sum
  int* cum;                 // [B + 1] work units before each sequence
};

struct KvAttnLaunch {
  CUtensorMap tk, tv;       // caches as [num_pages * page_size, Hk * D]
  KvAttnParams p;
  int D, kind;
  int nb;                   // few-row kernel: query rows of a work item / 8, 1 or 2
  int qt;                   // many-row kernel: 128-row query tiles of a work item, 1 or 2
  bool early;               // set up while the launch before it still runs (it reads nothing of that one's)
  int grid;
  int device;
  cudaStream_t stream;
};

// Geometry that the front end, the kernels and the merge share.
struct KvAttnGeom {
  int ctas;                 // CTAs per SM
  int warps, keys, slots;   // warps of a CTA; keys of a tile, the unit of work; slots (K or V of a tile) of a warp's ring
};
// nb: query rows of an item / 8. As many warps as leave each the registers its
// accumulators (D * nb / 4) and operands need: 12 in two CTAs (168 registers a
// thread), or 8 or 6 in one (255). More warps with less spill in the inner loop
// and lose, whole calls, D = 128, e4m3, B = 64 of 2048 .. 8192 keys: nb = 1, 16
// warps (128 registers) 129 us, 12 warps 121 us; nb = 2, 10 warps 151 us, 8 warps
// 134 us.
constexpr KvAttnGeom kv_attn_geom(int D, int elem_bytes, int nb) {
  const int keys = D * elem_bytes <= 128 ? 32 : 16;
  const int slot = keys * D * elem_bytes;
  const int ctas = D * nb <= 128 ? 2 : 1;
  const int warps = D * nb >= 256 && slot <= 4096 ? 8 : 6;
  // 192 KB per SM for the rings and, where they are not in registers (D * nb >
  // 128), each warp's query fragments
  const int q = D * nb > 128 ? nb * D * 16 : 0;
  int slots = (196608 / (ctas * warps) - q) / slot;
  slots = slots > 6 ? 6 : slots;
  return KvAttnGeom{ctas, warps, keys, slots};
}

// Shared memory of a CTA without the work line's sums (kv_attn.cuh lays it out),
// and the CTAs that an SM holds with those of B sequences: two become one past
// B = 2875 (D = 128, 8 bits) or 3643 (16 bits). The line is cut for those that
// fit: cut for two, the second half of the grid started behind the first (B =
// 3000 of 75 .. 300 keys, D = 128, e4m3: 393 us, 384 with this; B = 2800: 234).
constexpr int kv_attn_smem(int D, int elem_bytes, int nb) {
  const KvAttnGeom g = kv_attn_geom(D, elem_bytes, nb);
  const int q = D * nb > 128 ? nb * D * 16 : 0;
  const int scales = elem_bytes == 1 ? (g.slots <= 4 ? 2 : 4) * 2 * g.keys * 4 : 0;
  return g.warps * (g.slots * (g.keys * D * elem_bytes + 8) + q + scales + 4 * 64) + 16 + 64 + 1024;
}
constexpr int kv_attn_ctas(int D, int elem_bytes, int nb, int B) {
  const int ctas = kv_attn_geom(D, elem_bytes, nb).ctas;
  return ctas == 2 && 2 * (kv_attn_smem(D, elem_bytes, nb) + (B + 1) * 4 + 1024) > 233472 ? 1 : ctas;
}

cudaError_t launch_kv_attn_d64(const KvAttnLaunch& L);
cudaError_t launch_kv_attn_d128(const KvAttnLaunch& L);
cudaError_t launch_kv_attn_d256(const KvAttnLaunch& L);
// The many-row kernel (kv_rows.cuh): items of up to 128 * qt rows, units of 128 keys.
constexpr int kRowsUnit = 128;
constexpr int kRowsMaxSeqs = 1024;   // sequences of its work line (their prefix sums sit in shared memory)
constexpr int rows_max_qt(int D) { return D <= 128 ? 2 : 1; }
// rows of its TMA boxes at most: 16-bit tiles are loaded whole, 8-bit ones in
// parts of 64 keys (D = 256: 32) that are then converted
constexpr int rows_box(int D, int elem_bytes) { return elem_bytes == 2 ? 128 : D == 256 ? 32 : 64; }
cudaError_t launch_kv_rows_d64(const KvAttnLaunch& L);
cudaError_t launch_kv_rows_d128(const KvAttnLaunch& L);
cudaError_t launch_kv_rows_d256(const KvAttnLaunch& L);

// Where one launch left its partials, as the merge needs it.
struct KvPartials {
  const float* o;           // [slots, rt, D]
  const float* ml;          // [slots, rt, 2]
  int rt, unit, ranges;
  int pre_total;            // units of the prefix on that launch's line
  int whole;                // first of the whole items' slots, in Hk's
  int own;                  // the line also holds the sequences' own units
};
struct KvMergeParams {
  KvAttnParams p;
  KvPartials own, pre;      // the sequences' own keys; the prefix (p.prefix_tiles > 0)
};
cudaError_t launch_kv_merge(const KvMergeParams& m, int D, cudaStream_t stream);

#ifdef __CUDACC__
// Launch, optionally with programmatic serialisation: the kernel may be set up
// while the one before it in the stream still runs.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kern)(Params...), int grid, int threads, int smem, cudaStream_t stream, bool early,
                         const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// page and row of position `pos` within its page
__device__ __forceinline__ void page_of(const PagedSeqs& s, int pos, int& index, int& offset) {
  if (s.page_shift >= 0) {
    index = pos >> s.page_shift;
    offset = pos & (s.page_size - 1);
  } else {
    index = pos / s.page_size;
    offset = pos - index * s.page_size;
  }
}

// first row and number of rows of sequence b on the packed (or fixed) side;
// false if its bounds are broken
__device__ __forceinline__ bool seq_rows(const PagedSeqs& s, int b, int& first, int& n) {
  if (s.cu == nullptr) {
    first = b * s.S;
    n = s.S;
    return true;
  }
  const int r0 = __ldg(s.cu + b), r1 = __ldg(s.cu + b + 1);
  first = r0;
  n = r1 - r0;
  return r0 >= 0 && r1 >= r0 && r1 <= s.total && n <= s.S;
}

// sequence of row t: the last b with cu[b] <= t (cu nondecreasing), or -1
__device__ __forceinline__ int seq_of_row(const PagedSeqs& s, int t) {
  if (s.cu == nullptr) return t / s.S;
  if (t >= __ldg(s.cu + s.B)) return -1;
  int lo = -1, hi = s.B;   // cu[lo] <= t < cu[hi], with cu[-1] taken as below every row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(s.cu + mid) <= t) lo = mid; else hi = mid;
  }
  return lo;
}
#endif

}  // namespace fa
