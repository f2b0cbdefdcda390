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
//   kept = rows of the page below cache_len[b]: e is at least their old scale,
//          and if it grew their codes are rounded again to the new one;
//   code = e4m3(x 2^-e), nearest, ties to even, saturating.
// A power of two makes both the scaling and a later attention's dequantisation
// exact, and a re-rounding loses bits only where codes turn subnormal.
//
// One unit = one page of one kv head of K or of V.  Its 2 page threads hold all
// its rows in registers as fp32 (a row is read once, and its maximum is known
// before its codes are formed): a thread owns the two 8-element chunks that
// rotate with each other, so a rotation needs no exchange.  Queries are
// rotated by further CTAs of the same launch; a thread keeps one row's angles
// for several heads.
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

// The two chunks of pair index i (8 pairs of elements); both layouts take the
// angles of pairs 8 i .. 8 i + 7.
__device__ __forceinline__ void rotate_chunks(float (&a)[8], float (&b)[8], const float2 (&cs)[8],
                                              bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rotate(a[2 * j], a[2 * j + 1], cs[j]);
      rotate(b[2 * j], b[2 * j + 1], cs[4 + j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) rotate(a[j], b[j], cs[j]);
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
  int slots;      // pages that one sequence's new rows can touch
  int kv_blocks;  // CTAs per (sequence, page slot)
  int q_blocks;   // CTAs per sequence for the queries
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

__device__ __forceinline__ void load_angles(const AppendParams& p, int pos, int i,
                                            float2 (&cs)[8]) {
  const float4* t = reinterpret_cast<const float4*>(p.rope + static_cast<size_t>(pos) * p.half) +
                    4 * i;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 f = __ldg(t + j);
    cs[2 * j] = make_float2(f.x, f.y);
    cs[2 * j + 1] = make_float2(f.z, f.w);
  }
}

template <int HD>
__global__ void __launch_bounds__(APPEND_THREADS) append_kernel(const AppendParams p) {
  constexpr int PAIRS = HD / 16;  // chunk pairs per row
  constexpr int ROWS = HD / 32;   // rows per thread of a unit
  __shared__ float red[APPEND_THREADS / 32];
  griddep_launch();
  griddep_wait();
  const Batch& bt = p.bt;
  const int kv_total = bt.B * p.slots * p.kv_blocks;
  const bool rotated = p.half > 0;

  if (static_cast<int>(blockIdx.x) >= kv_total) {
    // ------------------------------------------------------------ queries
    const int x = static_cast<int>(blockIdx.x) - kv_total;
    const int b = x / p.q_blocks;
    const Seq s = load_seq(bt, b, INT_MAX, 0x501, false);
    const int groups = (p.Hq + Q_HEADS - 1) / Q_HEADS;
    const int item = (x % p.q_blocks) * APPEND_THREADS + static_cast<int>(threadIdx.x);
    const int i = item % PAIRS;
    const int hg = (item / PAIRS) % groups;
    const int row = item / (PAIRS * groups);
    if (row >= s.n || s.c0 + row >= p.rope_len) return;
    int ca, cb;
    chunk_pair(p, i, &ca, &cb);
    const __nv_bfloat16* src = p.q + static_cast<size_t>(s.t0 + row) * p.ldq;
    __nv_bfloat16* dst = p.q_out + static_cast<size_t>(s.t0 + row) * p.ldqo;
    const bool turn = i * 8 < p.half;
    float2 cs[8];
    if (turn) load_angles(p, s.c0 + row, i, cs);
    const int h1 = min(p.Hq, (hg + 1) * Q_HEADS);
#pragma unroll
    for (int u = 0; u < Q_HEADS; ++u) {
      const int h = hg * Q_HEADS + u;
      if (h >= h1) break;
      const uint4 ra = *reinterpret_cast<const uint4*>(src + h * HD + ca * 8);
      const uint4 rb = *reinterpret_cast<const uint4*>(src + h * HD + cb * 8);
      uint4 wa = ra, wb = rb;
      if (turn) {
        float a[8], c[8];
        unpack_bf16x8(ra, a);
        unpack_bf16x8(rb, c);
        rotate_chunks(a, c, cs, p.interleaved != 0);
        wa = make_uint4(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]), pack_bf16x2(a[4], a[5]),
                        pack_bf16x2(a[6], a[7]));
        wb = make_uint4(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]), pack_bf16x2(c[4], c[5]),
                        pack_bf16x2(c[6], c[7]));
      }
      *reinterpret_cast<uint4*>(dst + h * HD + ca * 8) = wa;
      *reinterpret_cast<uint4*>(dst + h * HD + cb * 8) = wb;
    }
    return;
  }

  // -------------------------------------------------------------- keys and values
  const int b = static_cast<int>(blockIdx.x) / (p.slots * p.kv_blocks);
  const int slot = (static_cast<int>(blockIdx.x) / p.kv_blocks) % p.slots;
  const int blk = static_cast<int>(blockIdx.x) % p.kv_blocks;
  Seq s = load_seq(bt, b, INT_MAX, 0x501, slot == 0 && blk == 0 && threadIdx.x == 0);
  if (rotated && s.c0 + s.n > p.rope_len && s.n > 0) {
    if (slot == 0 && blk == 0 && threadIdx.x == 0) raise_error(ERR_CHECK | 0x502, b);
    s.n = 0;
  }
  const int page_idx = (s.c0 >> bt.log_page) + slot;
  const int base = page_idx << bt.log_page;  // position of the page's first row
  if (s.n == 0 || base >= s.c0 + s.n) return;
  const int pg = bt.page_table[static_cast<size_t>(b) * bt.max_pages + page_idx];
  if (pg < 0 || pg >= bt.n_pages) {
    if (blk == 0 && threadIdx.x == 0) raise_error(ERR_CHECK | 0x503, b);
    return;
  }

  const int threads = 2 * bt.page;  // of one unit
  const int unit = blk * (APPEND_THREADS / threads) + static_cast<int>(threadIdx.x) / threads;
  const bool live = unit < 2 * p.Hkv;
  const bool is_v = unit >= p.Hkv;
  const int g = live ? (is_v ? unit - p.Hkv : unit) : 0;
  const int tu = static_cast<int>(threadIdx.x) % threads;
  const int i = tu % PAIRS;
  const int row0 = tu / PAIRS;
  const int row_step = threads / PAIRS;
  int ca, cb;
  chunk_pair(p, i, &ca, &cb);
  const __nv_bfloat16* src = (is_v ? p.v : p.k) + static_cast<size_t>(g) * HD;
  const size_t head = static_cast<size_t>(pg) * p.Hkv + g;
  uint8_t* dst = (is_v ? p.v_pages : p.k_pages) + (head << bt.log_page) * HD;
  uint8_t* exp_at = (is_v ? p.v_exp : p.k_exp) + head;
  const bool keeps = base < s.c0;  // rows of earlier appends stay in this page
  const int e_old = keeps ? min(static_cast<int>(*exp_at) - 127, SCALE_MAX) : SCALE_MIN;

  uint4 ra[ROWS], rb[ROWS];
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int pos = base + row0 + u * row_step;
    ra[u] = rb[u] = make_uint4(0u, 0u, 0u, 0u);
    if (live && pos >= s.c0 && pos < s.c0 + s.n) {
      const __nv_bfloat16* r = src + static_cast<size_t>(s.t0 + pos - s.c0) * p.ldkv;
      ra[u] = *reinterpret_cast<const uint4*>(r + ca * 8);
      rb[u] = *reinterpret_cast<const uint4*>(r + cb * 8);
    }
  }
  float a[ROWS][8], c[ROWS][8];
  float amax = 0.f;
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int pos = base + row0 + u * row_step;
    unpack_bf16x8(ra[u], a[u]);
    unpack_bf16x8(rb[u], c[u]);
    if (!is_v && i * 8 < p.half && pos >= s.c0 && pos < s.c0 + s.n) {
      float2 cs[8];
      load_angles(p, pos, i, cs);
      rotate_chunks(a[u], c[u], cs, p.interleaved != 0);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = fabsf(a[u][e]), y = fabsf(c[u][e]);
      amax = fmaxf(amax, x <= FLT_MAX ? x : 0.f);
      amax = fmaxf(amax, y <= FLT_MAX ? y : 0.f);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (threads > 32) {  // the same for every unit of the launch
    if (lane_id() == 0) red[warp_id()] = amax;
    __syncthreads();
    const int w0 = (static_cast<int>(threadIdx.x) / threads) * (threads / 32);
    for (int w = 0; w < threads / 32; ++w) amax = fmaxf(amax, red[w0 + w]);
  }
  if (!live) return;
  const int e = max(scale_exponent(amax), e_old);
  const float f = pow2(-e);
#pragma unroll
  for (int u = 0; u < ROWS; ++u) {
    const int row = row0 + u * row_step;
    const int pos = base + row;
    uint2* da = reinterpret_cast<uint2*>(dst + static_cast<size_t>(row) * HD + ca * 8);
    uint2* db = reinterpret_cast<uint2*>(dst + static_cast<size_t>(row) * HD + cb * 8);
    if (pos >= s.c0 && pos < s.c0 + s.n) {
      *da = pack_e4m3x8(a[u], f);
      *db = pack_e4m3x8(c[u], f);
    } else if (pos < s.c0 && e > e_old) {
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
