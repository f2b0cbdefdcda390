// kvappend.cuh - append new K/V rows to a paged e4m3 cache, rotating keys and
// queries by their positions on the way.
//
// Sequence b's new rows take positions pos = cache_len[b] + i.  Rotation of a
// pair (x, y) of a head by the angle a of (pos, pair index), from a table of
// (cos a, sin a):   x' = x cos a - y sin a,   y' = y cos a + x sin a
// (every product and sum rounded to fp32, never contracted, so that the bits
// do not depend on the compiler).  The rows of one page and kv head share a
// power-of-two scale 2^e:
//   e    = the smallest integer with max |x| <= 448 2^e over the page's new
//          rows (finite values only), clamped to [-40, 100];
//   kept = rows of the page below cache_len[b]: e is at least their old scale
//          (even one above 100, in a page of another origin), and if it grew
//          their codes are rounded again to the new one;
//   code = e4m3(x 2^-e), nearest, ties to even, saturating.
// A power of two makes both the scaling and a later attention's dequantisation
// exact, and a re-rounding loses bits only where codes turn subnormal.
//
// One unit = one page of one kv head of K or of V.  Its 2 page threads hold all
// its rows in registers as fp32 (a row is read once, and its maximum is known
// before its codes are formed): a thread owns the two 8-element chunks that
// rotate with each other, so a rotation needs no exchange.  Queries are
// rotated by further CTAs of the same launch; a thread keeps one row's angles
// for several heads.  Rows are read once, past the caches' usual order.
//
// Bound by HBM for long prompts: four of up to 4096 rows (8 kv and 16 query
// heads of 128) in 32 us, 4.8 TB/s, 73% of the measured copy rate, with a third
// of the SM's warps resident (three CTAs: 80 registers with the rows held in
// fp32, and at hd 128 still 104 bytes of spill loads) and 45% of its issue
// slots taken by conversions and rotation.  Canvases and single
// tokens are launch and latency: 3 to 7 us.
#pragma once

#include <cuda_fp8.h>
#include <float.h>

#include "dg_common.cuh"

namespace dg {
namespace paged {

constexpr int SCALE_MIN = -40;   // exponents of a page's scale; stored with a bias of 127
constexpr int SCALE_MAX = 100;

// The batch of ragged new rows that append and attention share.
struct Batch {
  int B, T, max_new, max_pages, page, log_page, n_pages;
  const int32_t* tok_start;   // [B + 1] first token row of each sequence
  const int32_t* cache_len;   // [B] rows cached before the new ones
  const int32_t* page_table;  // [B, max_pages]
};

struct Seq {
  int t0, n, c0;  // first token row, new rows, cached rows
};

// Sequence b's extent.  One that does not fit its buffers (or the bounds that
// the launch was planned with) is recorded as a device check and left out.
__device__ __forceinline__ Seq load_seq(const Batch& p, int b, int max_prefix, uint32_t site,
                                        bool report) {
  Seq s;
  s.t0 = p.tok_start[b];
  const long long n = static_cast<long long>(p.tok_start[b + 1]) - s.t0;
  s.c0 = p.cache_len[b];
  const long long cap = static_cast<long long>(p.max_pages) << p.log_page;
  const bool ok = s.t0 >= 0 && n >= 0 && n <= p.max_new && s.t0 + n <= p.T && s.c0 >= 0 &&
                  s.c0 <= max_prefix && s.c0 + n <= cap;
  if (!ok && report) raise_error(ERR_CHECK | site, static_cast<uint32_t>(b));
  s.n = ok ? static_cast<int>(n) : 0;
  return s;
}

// The smallest e in [SCALE_MIN, SCALE_MAX] with amax <= 448 2^e = 1.75 2^(e + 8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, SCALE_MIN), SCALE_MAX);
}

// 2^e for normal results
__device__ __forceinline__ float pow2(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint2 pack_e4m3x8(const float (&x)[8], float f) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i] * f, x[2 * i + 1] * f), __NV_SATFINITE,
                                    __NV_E4M3);
  return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

__device__ __forceinline__ void unpack_e4m3x8(uint2 v, float (&x)[8]) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void unpack_bf16x8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void rotate(float& x, float& y, float2 cs) {
  const float a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
  y = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
  x = a;
}

// Half h of the eight pairs that the chunks a and b of a pair index form: their
// elements 4 h .. 4 h + 3 with each other, or the adjacent pairs of one chunk.
__device__ __forceinline__ void rotate_half(float (&a)[8], float (&b)[8], const float2 (&cs)[4],
                                            int h, bool interleaved) {
  if (interleaved) {
    float(&x)[8] = h ? b : a;
#pragma unroll
    for (int j = 0; j < 4; ++j) rotate(x[2 * j], x[2 * j + 1], cs[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) rotate(a[4 * h + j], b[4 * h + j], cs[j]);
  }
}

struct AppendParams {
  Batch bt;
  int Hq, Hkv;
  int half;         // rotated pairs per head (a multiple of 8; 0: no rotation)
  int interleaved;  // pairs (2i, 2i + 1) instead of (i, i + half)
  int rope_len;
  const float2* rope;  // [rope_len, half] (cos, sin)
  const __nv_bfloat16 *k, *v, *q;
  __nv_bfloat16* q_out;
  int ldkv, ldq, ldqo;
  uint8_t *k_pages, *v_pages;  // [n_pages, Hkv, page, hd]
  uint8_t *k_exp, *v_exp;      // [n_pages, Hkv]
  int kv_blocks;  // CTAs per (sequence, page) for keys and values; further ones for queries
};

constexpr int APPEND_THREADS = 256;
constexpr int Q_HEADS = 4;  // query heads per thread

// The chunk indices (8 elements each) of pair index i.
__device__ __forceinline__ void chunk_pair(const AppendParams& p, int i, int* a, int* b) {
  const int rc = p.half >> 3;
  if (p.interleaved || i >= rc) {
    *a = 2 * i;  // also the unrotated rest: 2 rc + 2 (i - rc)
    *b = 2 * i + 1;
  } else {
    *a = i;
    *b = i + rc;
  }
}

// Angles 4 h .. 4 h + 3 of pair index i's eight.
__device__ __forceinline__ void load_angles(const AppendParams& p, int pos, int i, int h,
                                            float2 (&cs)[4]) {
  const float4* t = reinterpret_cast<const float4*>(p.rope + static_cast<int64_t>(pos) * p.half) +
                    4 * i + 2 * h;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 f = __ldg(t + j);
    cs[2 * j] = make_float2(f.x, f.y);
    cs[2 * j + 1] = make_float2(f.z, f.w);
  }
}

// Grid: z = sequence, y = page that its new rows touch, x = units of that page
// and then its rows' queries.  Every index below is a shift: at 16 elements a
// thread, divisions would be most of the instructions.
template <int HD>
__global__ void __launch_bounds__(APPEND_THREADS, 3) append_kernel(const AppendParams p) {
  constexpr int PAIRS = HD / 16;  // chunk pairs per row
  constexpr int LOG_PAIRS = HD == 128 ? 3 : 2;
  constexpr int ROWS = HD / 32;   // rows per thread of a unit
  __shared__ float red[APPEND_THREADS / 32];
  griddep_launch();
  griddep_wait();
  const Batch& bt = p.bt;
  const int b = blockIdx.z;
  const int slot = blockIdx.y;
  const int blk = blockIdx.x;
  const bool report = slot == 0 && blk == 0 && threadIdx.x == 0;
  Seq s = load_seq(bt, b, INT_MAX, 0x501, report);
  if (p.half > 0 && s.n > 0 && s.n > p.rope_len - s.c0) {
    if (report) raise_error(ERR_CHECK | 0x502, b);
    s.n = 0;
  }
  const int page_idx = (s.c0 >> bt.log_page) + slot;
  const int base = page_idx << bt.log_page;  // position of the page's first row
  // the page's rows [r_beg, r_end) are new
  const int r_beg = max(s.c0 - base, 0);
  const int r_end = min(s.c0 + s.n - base, bt.page);
  if (s.n == 0 || r_beg >= r_end) return;

  if (blk >= p.kv_blocks) {
    // ------------------------------------------------------------ queries
    const int item = (blk - p.kv_blocks) * APPEND_THREADS + static_cast<int>(threadIdx.x);
    const int i = item & (PAIRS - 1);
    const int r = (item >> LOG_PAIRS) & (bt.page - 1);
    const int h0 = (item >> (LOG_PAIRS + bt.log_page)) * Q_HEADS;
    if (r < r_beg || r >= r_end || h0 >= p.Hq) return;
    int ca, cb;
    chunk_pair(p, i, &ca, &cb);
    const int64_t row = s.t0 + base + r - s.c0;
    const __nv_bfloat16* src = p.q + row * p.ldq + h0 * HD;
    __nv_bfloat16* dst = p.q_out + row * p.ldqo + h0 * HD;
    const bool turn = i * 8 < p.half;
    const int heads = min(Q_HEADS, p.Hq - h0);
    uint4 ra[Q_HEADS], rb[Q_HEADS];
#pragma unroll
    for (int u = 0; u < Q_HEADS; ++u) {
      if (u < heads) {
        ra[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * HD + ca * 8));
        rb[u] = __ldcs(reinterpret_cast<const uint4*>(src + u * HD + cb * 8));
      }
    }
    if (turn) {
      float2 cs[2][4];
      load_angles(p, base + r, i, 0, cs[0]);
      load_angles(p, base + r, i, 1, cs[1]);
#pragma unroll
      for (int u = 0; u < Q_HEADS; ++u) {
        float a[8], c[8];
        unpack_bf16x8(ra[u], a);
        unpack_bf16x8(rb[u], c);
        rotate_half(a, c, cs[0], 0, p.interleaved != 0);
        rotate_half(a, c, cs[1], 1, p.interleaved != 0);
        ra[u] = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]),
                           pack_bf16x2(a[4], a[5]), pack_bf16x2(a[6], a[7]));
        rb[u] = make_uint4(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]),
                           pack_bf16x2(c[4], c[5]), pack_bf16x2(c[6], c[7]));
      }
    }
#pragma unroll
    for (int u = 0; u < Q_HEADS; ++u) {
      if (u < heads) {
        *reinterpret_cast<uint4*>(dst + u * HD + ca * 8) = ra[u];
        *reinterpret_cast<uint4*>(dst + u * HD + cb * 8) = rb[u];
      }
    }
    return;
  }

  // -------------------------------------------------------------- keys and values
  const int pg = bt.page_table[static_cast<int64_t>(b) * bt.max_pages + page_idx];
  if (pg < 0 || pg >= bt.n_pages) {
    if (blk == 0 && threadIdx.x == 0) raise_error(ERR_CHECK | 0x503, b);
    return;
  }
  const int log_threads = bt.log_page + 1;  // of one unit: 2 page
  const int unit = (blk << (8 - log_threads)) + (static_cast<int>(threadIdx.x) >> log_threads);
  const bool live = unit < 2 * p.Hkv;
  const bool is_v = unit >= p.Hkv;
  const int g = live ? (is_v ? unit - p.Hkv : unit) : 0;
  const int tu = static_cast<int>(threadIdx.x) & ((1 << log_threads) - 1);
  const int i = tu & (PAIRS - 1);
  const int row0 = tu >> LOG_PAIRS;
  const int row_step = 1 << (log_threads - LOG_PAIRS);
  int ca, cb;
  chunk_pair(p, i, &ca, &cb);
  const __nv_bfloat16* src =
      (is_v ? p.v : p.k) + static_cast<int64_t>(s.t0 + base - s.c0) * p.ldkv + g * HD;
  const int64_t head = static_cast<int64_t>(pg) * p.Hkv + g;
  uint8_t* dst = (is_v ? p.v_pages : p.k_pages) + (head << bt.log_page) * HD;
  uint8_t* exp_at = (is_v ? p.v_exp : p.k_exp) + head;
  const bool keeps = r_beg > 0;  // rows of earlier appends stay in this page
  const int e_old = keeps ? static_cast<int>(*exp_at) - 127 : SCALE_MIN;

  uint4 ra[ROWS], rb[ROWS];
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int r = row0 + u * row_step;
    ra[u] = rb[u] = make_uint4(0u, 0u, 0u, 0u);
    if (live && r >= r_beg && r < r_end) {
      const __nv_bfloat16* at = src + static_cast<int64_t>(r) * p.ldkv;
      ra[u] = __ldcs(reinterpret_cast<const uint4*>(at + ca * 8));
      rb[u] = __ldcs(reinterpret_cast<const uint4*>(at + cb * 8));
    }
  }
  float a[ROWS][8], c[ROWS][8];
  float amax = 0.f;
  const bool turn = !is_v && i * 8 < p.half;
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int r = row0 + u * row_step;
    unpack_bf16x8(ra[u], a[u]);
    unpack_bf16x8(rb[u], c[u]);
    if (turn && r >= r_beg && r < r_end) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 cs[4];
        load_angles(p, base + r, i, h, cs);
        rotate_half(a[u], c[u], cs, h, p.interleaved != 0);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(a[u][e]), fabsf(c[u][e])));
  }
  if (!(amax <= FLT_MAX)) {  // infinities are left out (the maximum drops NaN by itself)
    amax = 0.f;
#pragma unroll
    for (int u = 0; u < ROWS; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = fabsf(a[u][e]), y = fabsf(c[u][e]);
        amax = fmaxf(amax, fmaxf(x <= FLT_MAX ? x : 0.f, y <= FLT_MAX ? y : 0.f));
      }
  }
  // magnitudes order as their bits
  const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
  amax = __uint_as_float(top);
  if (log_threads > 5) {  // the same for every unit of the launch
    if (lane_id() == 0) red[warp_id()] = amax;
    __syncthreads();
    const int w0 = (static_cast<int>(threadIdx.x) >> log_threads) << (log_threads - 5);
    for (int w = 0; w < 1 << (log_threads - 5); ++w) amax = fmaxf(amax, red[w0 + w]);
  }
  if (!live) return;
  const int e = max(scale_exponent(amax), e_old);
  const float f = e < 127 ? pow2(-e) : __uint_as_float(0x800000u >> (e - 126));  // subnormal
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int r = row0 + u * row_step;
    uint2* da = reinterpret_cast<uint2*>(dst + r * HD + ca * 8);
    uint2* db = reinterpret_cast<uint2*>(dst + r * HD + cb * 8);
    if (r >= r_beg && r < r_end) {
      *da = pack_e4m3x8(a[u], f);
      *db = pack_e4m3x8(c[u], f);
    } else if (r < r_beg && e > e_old) {
      const float down = exp2f(static_cast<float>(e_old - e));
      float x[8];
      unpack_e4m3x8(*da, x);
      *da = pack_e4m3x8(x, down);
      unpack_e4m3x8(*db, x);
      *db = pack_e4m3x8(x, down);
    }
  }
  __syncwarp();  // a one-warp unit has read its old exponent (larger ones passed the barrier)
  if (tu == 0) *exp_at = static_cast<uint8_t>(e + 127);
}

}  // namespace paged
}  // namespace dg
