// C-ABI front end of the cache-side operators: argument checks, tensor maps,
// workspace layout and launches. See include/fa.h for the contract.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fa.h"
#include "kv_internal.h"

namespace {

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return FA_OK;
  cudaGetLastError();
  return FA_ERR_CUDA;
}

// Checks that every operator on a paged cache shares. dtype: the 16-bit side.
int check_cache(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                const int* block_table, const int* seqlens_k, int B, int Hk, int S, int D, int num_pages,
                int page_size, int max_pages, const int* cu, int total, int dtype, int cache_dtype) {
  if (dtype != FA_FP16 && dtype != FA_BF16) return dtype == FA_FP8_E4M3 ? FA_ERR_UNSUPPORTED : FA_ERR_INVALID_ARG;
  if (cache_dtype != FA_FP16 && cache_dtype != FA_BF16 && cache_dtype != FA_FP8_E4M3 && cache_dtype != FA_INT8)
    return FA_ERR_INVALID_ARG;
  const bool k8 = cache_dtype == FA_FP8_E4M3 || cache_dtype == FA_INT8;
  if (!k8 && cache_dtype != dtype) return FA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256) return FA_ERR_UNSUPPORTED;
  if (B < 0 || Hk <= 0 || S < 0 || total < 0 || num_pages <= 0 || max_pages <= 0) return FA_ERR_INVALID_ARG;
  if (!(page_size == 16 || page_size == 32 || page_size == 64 || (page_size > 0 && page_size % 128 == 0)))
    return FA_ERR_INVALID_ARG;
  if ((int64_t)num_pages * page_size + 128 > INT32_MAX || (int64_t)max_pages * page_size > INT32_MAX ||
      (int64_t)B * max_pages > INT32_MAX || (cu == nullptr && (int64_t)B * S > INT32_MAX) ||
      (int64_t)Hk * D * 2 > INT32_MAX)
    return FA_ERR_INVALID_ARG;
  if (cu != nullptr && B > 0 && S == 0 && total > 0) return FA_ERR_INVALID_ARG;   // rows, but no sequence may have any
  if (B == 0 || S == 0 || (cu != nullptr && total == 0)) return FA_OK;   // nothing to do
  if (!k_cache || !v_cache || !block_table || !seqlens_k) return FA_ERR_INVALID_ARG;
  if (k8 && (!k_scale || !v_scale)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16)) return FA_ERR_ALIGNMENT;
  if (k8 && (!aligned(k_scale, 16) || !aligned(v_scale, 16))) return FA_ERR_ALIGNMENT;
  for (const void* p : {(const void*)block_table, (const void*)seqlens_k, (const void*)cu})
    if (!aligned(p, 4)) return FA_ERR_ALIGNMENT;
  return FA_OK;
}

void fill_seqs(fa::PagedSeqs& s, const int* block_table, const int* seqlens_k, const int* cu, int B, int S, int total,
               int num_pages, int page_size, int max_pages, int* status) {
  s.block_table = block_table;
  s.seqlens_k = seqlens_k;
  s.cu = cu;
  s.B = B;
  s.S = S;
  s.total = cu != nullptr ? total : B * S;
  s.num_pages = num_pages;
  s.page_size = page_size;
  s.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz((unsigned)page_size) : -1;
  s.max_pages = max_pages;
  s.status = status;
}

int cache_kind(int cache_dtype) {
  return cache_dtype == FA_FP16 ? fa::kCacheF16
         : cache_dtype == FA_BF16 ? fa::kCacheBF16
         : cache_dtype == FA_FP8_E4M3 ? fa::kCacheE4M3 : fa::kCacheI8;
}

// One launch of an attention call over a cache: which kernel takes which part.
struct Pass {
  bool rows;                // the many-row kernel
  int nb, qt, rt, unit, grid;
  int ranges;               // of the work line; each has a worker per K/V head
  int64_t whole, slots;     // slots of partials, in Hk's: two per range, then the whole items
  size_t off_o, off_ml;
};
// The call: `own` for the sequences' own keys (and the prefix too, if there is
// one and `pre` is unused), `pre` for the prefix by itself.
struct Shape {
  Pass own, pre;
  bool split;
  int64_t prefix_tiles;     // row tiles of the prefix, in the pass that takes it
  size_t off_cum, bytes;
};

// The few-row kernel takes tiles of up to 16 rows and reads the keys once for
// each; the many-row kernel reads them once for up to 256 rows, and pays for
// 128. 16-bit caches change at 16 rows, 8-bit caches, whose codes it has to
// convert for 128 rows however few there are, at 32. Measured, few-row against
// many-row kernel, B = 64, 8 K/V heads, 2048 to 8192 keys:
//   16-bit, D = 128: 16 rows 223, 268 us; 20 rows 412, 275; 64 rows 815, 290
//   16-bit, 20 rows: D = 64 205, 189; D = 256 754, 736
//   e4m3, D = 128: 16 rows 134, 299; 32 rows 251, 304; 36 rows 357, 304
//   e4m3, 32 rows: D = 64 165, 287; D = 256 522, 703; 36 rows: 234, 288; 761, 704
//   int8, 32 rows: D = 64 183, 293; D = 128 280, 312; D = 256 567, 727
//   int8, 36 rows: D = 64 260, 294; D = 128 403, 313; D = 256 829, 728
// (one bound for all head sizes: at D = 64 the 8-bit few-row kernel would still
// win up to 48 rows)
// `rows` bounds an item's rows, `mean` is what they are on average: that is
// what the few-row kernel's time goes with (24 packed sequences of 4 to 20
// rows, 12 on average, 16-bit, D = 256: 133, 208 us).
// Its work line holds kRowsMaxSeqs sequences; beyond, the few-row kernel does
// it all.
void choose(Pass& z, int64_t rows, int64_t mean, int B, int Hk, int D, int elem_bytes, bool can_rows, int sms) {
  z.rows = mean > (elem_bytes == 1 ? 32 : 16) && can_rows;
  z.qt = z.rows && rows > 128 && fa::rows_max_qt(D) == 2 ? 2 : 1;
  z.nb = rows <= 8 ? 1 : 2;
  int workers = sms, per_cta = 1;
  if (z.rows) {
    z.rt = 128 * z.qt;
    z.unit = fa::kRowsUnit;
  } else {
    const fa::KvAttnGeom g = fa::kv_attn_geom(D, elem_bytes, z.nb);
    z.rt = 8 * z.nb;
    z.unit = g.keys;
    workers *= fa::kv_attn_ctas(D, elem_bytes, z.nb, B) * g.warps;
    per_cta = g.warps;
  }
  z.ranges = std::max(1, workers / Hk);
  z.grid = (int)(((int64_t)z.ranges * Hk + per_cta - 1) / per_cta);
}

bool shape_of(Shape& z, int B, int Hq, int Hk, int S, int D, int elem_bytes, int total, bool prefix, int sms) {
  const int64_t G = Hq / Hk;
  const int64_t rows_own = (int64_t)S * G, rows_pre = (int64_t)total * G;
  // A prefix that more than 32 rows share gets a pass of its own; fewer rows go
  // on one work line with the sequences' own keys, with the few-row kernel (e4m3,
  // 32768 shared keys, up to 1024 own ones: 48 rows 53 us split, 58 on one line;
  // 32 rows 48 and 43, and with 100 own and 300 shared keys 19 and 15).
  z.split = prefix && rows_pre > 32;
  const bool one_line = prefix && !z.split;
  choose(z.own, one_line ? rows_pre : rows_own, (rows_pre + B - 1) / B, B, Hk, D, elem_bytes,
         !one_line && B <= fa::kRowsMaxSeqs, sms);
  choose(z.pre, rows_pre, rows_pre, B, Hk, D, elem_bytes, true, sms);
  const int rt_pre = z.split ? z.pre.rt : z.own.rt;
  z.prefix_tiles = prefix ? (rows_pre + rt_pre - 1) / rt_pre : 0;
  z.own.whole = 2 * (int64_t)z.own.ranges;
  z.own.slots = z.own.whole + (prefix ? rows_pre / z.own.rt + B : 0);
  if (prefix && !z.split) {
    z.pre = z.own;
    z.pre.whole = z.own.slots;
    z.own.slots += z.prefix_tiles;
    z.pre.slots = 0;
  } else {
    z.pre.whole = 2 * (int64_t)z.pre.ranges;
    z.pre.slots = prefix ? z.pre.whole + z.prefix_tiles : 0;
  }
  if (z.own.slots * Hk > INT32_MAX || z.pre.slots * Hk > INT32_MAX) return false;
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t off = at;
    at += round256(n);
    return off;
  };
  z.own.off_o = take((size_t)z.own.slots * Hk * z.own.rt * D * sizeof(float));
  z.own.off_ml = take((size_t)z.own.slots * Hk * z.own.rt * 2 * sizeof(float));
  if (z.pre.slots > 0) {
    z.pre.off_o = take((size_t)z.pre.slots * Hk * z.pre.rt * D * sizeof(float));
    z.pre.off_ml = take((size_t)z.pre.slots * Hk * z.pre.rt * 2 * sizeof(float));
  } else {
    z.pre.off_o = z.own.off_o;
    z.pre.off_ml = z.own.off_ml;
  }
  z.off_cum = take(((size_t)B + 1) * sizeof(int));
  z.bytes = at;
  return true;
}

// Tensor maps of a pass over the caches, and the launch.
int launch_pass(fa::KvAttnLaunch& L, const Pass& z, const void* k_cache, const void* v_cache, int D, int kind, char* ws) {
  const int eb = fa::cache_is_8bit(kind) ? 1 : 2;
  const fa::PagedSeqs& s = L.p.s;
  L.p.box_rows = std::min(s.page_size, z.rows ? fa::rows_box(D, eb) : fa::kv_attn_geom(D, eb, z.nb).keys);
  L.p.part_o = reinterpret_cast<float*>(ws + z.off_o);
  L.p.part_ml = reinterpret_cast<float*>(ws + z.off_ml);
  const uint64_t cols = (uint64_t)L.p.Hk * D, rows = (uint64_t)s.num_pages * s.page_size;
  const CUtensorMapDataType dt = eb == 1                  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : kind == fa::kCacheF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                          : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const uint32_t box_cols = (uint32_t)(std::min(D * eb, 128) / eb), box_rows = (uint32_t)L.p.box_rows;
  const CUtensorMapSwizzle sw = D * eb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  int st;
  if ((st = fa::encode_map(&L.tk, k_cache, dt, eb, cols, rows, box_cols, box_rows, sw)) != FA_OK) return st;
  if ((st = fa::encode_map(&L.tv, v_cache, dt, eb, cols, rows, box_cols, box_rows, sw)) != FA_OK) return st;
  L.D = D;
  L.kind = kind;
  L.nb = z.nb;
  L.qt = z.qt;
  L.grid = z.grid;
  L.p.ranges = z.ranges;
  auto* launch = z.rows ? (D == 64 ? fa::launch_kv_rows_d64 : D == 128 ? fa::launch_kv_rows_d128 : fa::launch_kv_rows_d256)
                        : (D == 64 ? fa::launch_kv_attn_d64 : D == 128 ? fa::launch_kv_attn_d128 : fa::launch_kv_attn_d256);
  return cuda_status(launch(L));
}

constexpr int kMaxSeqs = 4096;   // the work line's prefix sums sit in shared memory

int attention(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
              const int* prefix_pages, int prefix_len, const int* block_table, const int* seqlens_k, void* o, float* lse,
              int B, int Hq, int Hk, int Sq, int D, int num_pages, int page_size, int max_pages, float scale, int causal,
              const int* cu_seqlens_q, int total_q, void* workspace, size_t workspace_bytes, int dtype, int cache_dtype,
              void* stream) {
  if (Hk <= 0 || Hq <= 0 || Hq % Hk != 0) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale < 0.f) return FA_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return FA_ERR_INVALID_ARG;
  if (prefix_len < 0) return FA_ERR_INVALID_ARG;
  int st = check_cache(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, B, Hk, Sq, D, num_pages, page_size,
                       max_pages, cu_seqlens_q, total_q, dtype, cache_dtype);
  if (st != FA_OK) return st;
  if (B == 0 || Sq == 0 || (cu_seqlens_q != nullptr && total_q == 0)) return FA_OK;
  if (B > kMaxSeqs) return FA_ERR_UNSUPPORTED;
  const int total = cu_seqlens_q != nullptr ? total_q : B * Sq;
  Sq = std::min(Sq, total);   // a loose bound on the rows of a packed sequence
  if (prefix_len > 0 && !prefix_pages) return FA_ERR_INVALID_ARG;
  if (!q || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(prefix_pages, 4)) return FA_ERR_ALIGNMENT;
  // positions are counted in 32 bits, up to the end of a tile that the last key begins
  if ((int64_t)prefix_len + (int64_t)max_pages * page_size + Sq + 256 > INT32_MAX) return FA_ERR_INVALID_ARG;
  const int64_t G = Hq / Hk;
  if ((int64_t)total * Hq > INT32_MAX || (int64_t)Sq * G > INT32_MAX) return FA_ERR_INVALID_ARG;

  int device = 0, sms = 0, *status = nullptr;
  if ((st = fa::device_state(&device, &sms, &status)) != FA_OK) return st;
  Shape z;
  const bool prefix = prefix_len > 0;
  const int kind = cache_kind(cache_dtype);
  const int eb = fa::cache_is_8bit(kind) ? 1 : 2;
  if (!shape_of(z, B, Hq, Hk, Sq, D, eb, total, prefix, sms)) return FA_ERR_UNSUPPORTED;
  if (workspace == nullptr || workspace_bytes < z.bytes) return FA_ERR_INVALID_ARG;
  if (!aligned(workspace, 256)) return FA_ERR_ALIGNMENT;
  // the work lines are counted in 32 bits
  const int64_t own_tiles = std::min((int64_t)B * ((Sq * G + z.own.rt - 1) / z.own.rt), total * G / z.own.rt + B);
  const int64_t own_units = own_tiles * (((int64_t)max_pages * page_size + z.own.unit - 1) / z.own.unit);
  const int64_t pre_units = z.prefix_tiles * (((int64_t)prefix_len + z.pre.unit - 1) / z.pre.unit);
  if (own_units + pre_units >= INT32_MAX) return FA_ERR_UNSUPPORTED;

  fa::KvMergeParams M;
  std::memset(&M, 0, sizeof(M));
  fa::KvAttnParams& P = M.p;
  fill_seqs(P.s, block_table, seqlens_k, cu_seqlens_q, B, Sq, total_q, num_pages, page_size, max_pages, status);
  P.q = q;
  P.o = o;
  P.lse = lse;
  P.k_scale = k_scale;
  P.v_scale = v_scale;
  P.Hq = Hq;
  P.Hk = Hk;
  P.G = (int)G;
  P.q_bf16 = dtype == FA_BF16;
  P.causal = causal;
  P.c = (float)((double)scale * 1.4426950408889634);
  P.prefix_pages = prefix_pages;
  P.prefix_len = prefix_len;
  P.direct = !prefix;
  P.most_units = (int)own_units;
  char* ws = static_cast<char*>(workspace);
  P.cum = reinterpret_cast<int*>(ws + z.off_cum);
  fa::KvAttnLaunch L;
  std::memset(&L, 0, sizeof(L));
  L.p = P;
  L.device = device;
  L.stream = static_cast<cudaStream_t>(stream);
  if (z.split) {
    L.p.prefix_tiles = (int)z.prefix_tiles;
    L.p.pass_own = 0;
    if ((st = launch_pass(L, z.pre, k_cache, v_cache, D, kind, ws)) != FA_OK) return st;
    L.p.prefix_tiles = 0;
    L.early = true;   // the prefix is nothing to the sequences' own keys
  } else {
    L.p.prefix_tiles = (int)z.prefix_tiles;
  }
  L.p.pass_own = 1;
  if ((st = launch_pass(L, z.own, k_cache, v_cache, D, kind, ws)) != FA_OK) return st;
  auto partials = [&](const Pass& x, int64_t pre_total, int own) {
    return fa::KvPartials{reinterpret_cast<float*>(ws + x.off_o), reinterpret_cast<float*>(ws + x.off_ml), x.rt, x.unit,
                          x.ranges, (int)pre_total, (int)x.whole, own};
  };
  P.prefix_tiles = (int)z.prefix_tiles;
  M.own = partials(z.own, z.split ? 0 : pre_units, 1);
  M.pre = partials(z.pre, pre_units, z.split ? 0 : 1);
  return cuda_status(fa::launch_kv_merge(M, D, L.stream));
}

int move(bool append, void* const x[2], const long long* strides, void* k_cache, void* v_cache, float* k_scale,
         float* v_scale, const int* block_table, const int* seqlens_k, int B, int Hk, int S, int D, int num_pages,
         int page_size, int max_pages, const int* cu, int total, int dtype, int cache_dtype, void* stream) {
  int st = check_cache(k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, B, Hk, S, D, num_pages, page_size,
                       max_pages, cu, total, dtype, cache_dtype);
  if (st != FA_OK) return st;
  if (B == 0 || S == 0 || (cu != nullptr && total == 0)) return FA_OK;
  if (!x[0] || !x[1]) return FA_ERR_INVALID_ARG;
  if (!aligned(x[0], 16) || !aligned(x[1], 16)) return FA_ERR_ALIGNMENT;
  // a CTA counts its work, 16 tokens of K and V, in 32 bits
  if ((int64_t)Hk * D > (1 << 24)) return FA_ERR_UNSUPPORTED;
  fa::CacheParams P;
  std::memset(&P, 0, sizeof(P));
  for (int w = 0; w < 2; ++w) {
    P.x[w] = x[w];
    P.xs_t[w] = strides ? strides[2 * w] : (long long)Hk * D;
    P.xs_h[w] = strides ? strides[2 * w + 1] : D;
    if (P.xs_t[w] < 0 || P.xs_h[w] < 0) return FA_ERR_INVALID_ARG;
    if (P.xs_t[w] % 8 || P.xs_h[w] % 8) return FA_ERR_ALIGNMENT;
  }
  int device = 0, sms = 0, *status = nullptr;
  if ((st = fa::device_state(&device, &sms, &status)) != FA_OK) return st;
  fill_seqs(P.s, block_table, seqlens_k, cu, B, S, total, num_pages, page_size, max_pages, status);
  P.pages[0] = k_cache;
  P.pages[1] = v_cache;
  P.scale[0] = k_scale;
  P.scale[1] = v_scale;
  P.H = Hk;
  P.D = D;
  auto* launch = append ? fa::launch_kv_append : fa::launch_kv_read;
  return cuda_status(launch(P, cache_kind(cache_dtype), dtype == FA_BF16, sms, static_cast<cudaStream_t>(stream)));
}

// Radians -> the fraction of a turn, in 2^-64 (whole turns per position change
// nothing: positions are integers). 1 / 2 pi as the sum of two doubles, so that
// the fraction is within one unit for |w| up to 2^40; one double alone leaves 53
// bits, and positions of 2^31 off by 2^-25 turns.
uint64_t turn_fraction(double w) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double a = std::fabs(w);
  const double p = std::fma(a, kHi, 0.0);   // (a product could be fused with what follows)
  const double rest = std::fma(a, kLo, std::fma(a, kHi, -p));   // a / 2 pi = p + rest
  const double t = (p - std::floor(p)) * 0x1p64;
  const uint64_t whole = (uint64_t)t;
  const uint64_t u = std::fabs(rest) < 0.25 ? whole + (uint64_t)(int64_t)std::floor(t - (double)whole + rest * 0x1p64 + 0.5)
                                            : whole + (uint64_t)((rest - std::floor(rest)) * 0x1p64);   // |w| past 2^50
  return w < 0.0 ? 0 - u : u;
}

}  // namespace

extern "C" {

int fa_rope(const void* q, const void* k, void* q_out, void* k_out, const int* positions, int T, int Hq, int Hk, int D,
            int rot_dim, int n_axes, const double* inv_freq, const signed char* axis, int interleaved, int inverse,
            const long long* strides, int dtype, void* stream) {
  if (dtype == FA_FP8_E4M3) return FA_ERR_UNSUPPORTED;
  if (dtype != FA_FP16 && dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (T < 0 || Hq < 0 || Hk < 0 || n_axes <= 0 || rot_dim < 2 || rot_dim % 2 || rot_dim > D) return FA_ERR_INVALID_ARG;
  if (D > 2 * fa::kRopeMaxPairs) return FA_ERR_UNSUPPORTED;
  if ((interleaved & ~1) || (inverse & ~1) || !inv_freq || !axis) return FA_ERR_INVALID_ARG;
  // the CTAs count their work in 32 bits, four tokens at a time
  if (((int64_t)Hq + Hk) * D > (1 << 28)) return FA_ERR_UNSUPPORTED;
  fa::RopeParams P;
  std::memset(&P, 0, sizeof(P));
  for (int j = 0; j < rot_dim / 2; ++j) {
    if (axis[j] < 0 || axis[j] >= n_axes || !std::isfinite(inv_freq[j])) return FA_ERR_INVALID_ARG;
    P.axis[j] = (uint8_t)axis[j];
    P.freq[j] = turn_fraction(inv_freq[j]);
  }
  if (T == 0 || (Hq == 0 && Hk == 0)) return FA_OK;
  if (!positions || (Hq > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out))) return FA_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return FA_ERR_ALIGNMENT;
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int H[2] = {Hq, Hk};
  for (int w = 0; w < 2; ++w) {
    P.x[w] = in[w];
    P.y[w] = out[w];
    P.H[w] = H[w];
    if (H[w] == 0) continue;
    if (!aligned(in[w], 2) || !aligned(out[w], 2)) return FA_ERR_ALIGNMENT;
    const long long dense[4] = {(long long)H[w] * D, D, (long long)H[w] * D, D};
    const long long* s = strides ? strides + 4 * w : dense;
    P.xs_t[w] = s[0];
    P.xs_h[w] = s[1];
    P.ys_t[w] = s[2];
    P.ys_h[w] = s[3];
    for (int i = 0; i < 4; ++i)
      if (s[i] < 0) return FA_ERR_INVALID_ARG;
    // two rows of an output in one place would race
    const bool token_inner = s[2] <= s[3];
    const long long inner = token_inner ? s[2] : s[3], outer = token_inner ? s[3] : s[2];
    const long long n_inner = token_inner ? T : H[w], n_outer = token_inner ? H[w] : T;
    if ((n_inner > 1 && inner < D) || (n_outer > 1 && outer < (n_inner > 1 ? (n_inner - 1) * inner : 0) + D))
      return FA_ERR_INVALID_ARG;
    P.in_place[w] = in[w] == out[w] && s[0] == s[2] && s[1] == s[3];
  }
  P.pos = positions;
  P.T = T;
  P.D = D;
  P.rot = rot_dim;
  P.inverse = inverse;
  int device = 0, sms = 0, *status = nullptr;
  const int st = fa::device_state(&device, &sms, &status);
  if (st != FA_OK) return st;
  return cuda_status(fa::launch_rope(P, dtype == FA_BF16, interleaved != 0, sms, static_cast<cudaStream_t>(stream)));
}

int fa_kv_append(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale, float* v_scale,
                 const int* block_table, const int* seqlens_k, int B, int Hk, int Sq, int D, int num_pages,
                 int page_size, int max_pages, const long long* strides, const int* cu_seqlens_q, int total_q, int dtype,
                 int cache_dtype, void* stream) {
  void* const x[2] = {const_cast<void*>(k), const_cast<void*>(v)};
  return move(true, x, strides, k_cache, v_cache, k_scale, v_scale, block_table, seqlens_k, B, Hk, Sq, D, num_pages,
              page_size, max_pages, cu_seqlens_q, total_q, dtype, cache_dtype, stream);
}

int fa_kv_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
               const int* block_table, const int* seqlens_k, const int* cu_seqlens_k, void* k, void* v, int B, int Hk,
               int D, int num_pages, int page_size, int max_pages, int total_k, int dtype, int cache_dtype,
               void* stream) {
  if (B < 0 || total_k < 0 || (B > 0 && total_k > 0 && !cu_seqlens_k)) return FA_ERR_INVALID_ARG;
  if (B == 0 || total_k == 0) return FA_OK;
  // a sequence's rows are bounded by its seqlens_k entry, on the device
  const int64_t most = page_size > 0 ? (int64_t)max_pages * page_size : 0;
  if (most <= 0 || most > INT32_MAX) return FA_ERR_INVALID_ARG;
  void* const x[2] = {k, v};
  return move(false, x, nullptr, const_cast<void*>(k_cache), const_cast<void*>(v_cache), const_cast<float*>(k_scale),
              const_cast<float*>(v_scale), block_table, seqlens_k, B, Hk, (int)most, D, num_pages, page_size, max_pages,
              cu_seqlens_k, total_k, dtype, cache_dtype, stream);
}

size_t fa_fwd_kvcache_workspace_size(int B, int Hq, int Hk, int Sq, int D, int total_q, int prefix_len) {
  if (B <= 0 || Hk <= 0 || Hq <= 0 || Hq % Hk || Sq <= 0 || (D != 64 && D != 128 && D != 256)) return 0;
  int device = 0, sms = 0, *status = nullptr;
  if (fa::device_state(&device, &sms, &status) != FA_OK) return 0;
  Shape z;
  const int64_t total = total_q > 0 ? total_q : (int64_t)B * Sq;
  if (total > INT32_MAX) return 0;
  Sq = (int)std::min<int64_t>(Sq, total);
  // enough for 8-bit and 16-bit caches
  size_t most = 0;
  for (int eb = 1; eb <= 2; ++eb) {
    if (!shape_of(z, B, Hq, Hk, Sq, D, eb, (int)total, prefix_len > 0, sms)) return 0;
    most = std::max(most, z.bytes);
  }
  return most;
}

int fa_fwd_kvcache(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                   const int* block_table, const int* seqlens_k, void* o, float* lse, int B, int Hq, int Hk, int Sq,
                   int D, int num_pages, int page_size, int max_pages, float scale, int causal, const int* cu_seqlens_q,
                   int total_q, void* workspace, size_t workspace_bytes, int dtype, int cache_dtype, void* stream) {
  return attention(q, k_cache, v_cache, k_scale, v_scale, nullptr, 0, block_table, seqlens_k, o, lse, B, Hq, Hk, Sq, D,
                   num_pages, page_size, max_pages, scale, causal, cu_seqlens_q, total_q, workspace, workspace_bytes,
                   dtype, cache_dtype, stream);
}

int fa_fwd_prefix(const void* q, const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale,
                  const int* prefix_pages, int prefix_len, const int* block_table, const int* seqlens_k, void* o,
                  float* lse, int B, int Hq, int Hk, int Sq, int D, int num_pages, int page_size, int max_pages,
                  float scale, int causal, const int* cu_seqlens_q, int total_q, void* workspace, size_t workspace_bytes,
                  int dtype, int cache_dtype, void* stream) {
  return attention(q, k_cache, v_cache, k_scale, v_scale, prefix_pages, prefix_len, block_table, seqlens_k, o, lse, B,
                   Hq, Hk, Sq, D, num_pages, page_size, max_pages, scale, causal, cu_seqlens_q, total_q, workspace,
                   workspace_bytes, dtype, cache_dtype, stream);
}

}  // extern "C"
