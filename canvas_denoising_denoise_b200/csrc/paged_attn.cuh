// paged_attn.cuh - attention of ragged new rows over a paged e4m3 KV cache.
//
// Sequence b's new rows (already appended) attend to its cache_len[b] + n_b
// cached rows, all of them (canvas) or up to their own position (causal):
//   s_ij = scale q_i . k_j,   out_i = sum_j softmax_j(s_ij) v_j,
// with k_j = 2^ek code, v_j = 2^ev code, one exponent per page and kv head.
// The query rows of a kv head's group are packed token by token (row = token
// * group + head in group), so a tile holds them whatever the group size.
//
// Rounding.  Codes enter the tensor core as they are cached; no key is ever
// expanded.  A bf16 query row, scaled by a power of two to at most 448, is
// split into two e4m3 values hi + lo (4 + 4 significant bits: exact for
// elements down to 2^-10 of the row's largest, below that to 2^-18 of it), and
// both halves are multiplied by the same key codes with fp32 accumulation.
// The probabilities are f16 (2^-11 of themselves): an 8-bit one would lose 2^-4.
// With many rows V codes become f16 times a power of two relative to the CTA's
// largest page scale (exactly for scales down to 2^-22 of that, below to 2^-32
// of it), and weights below 2^-21 of the largest are held to 2^-32 of it.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "attn.cuh"
#include "dg_common.cuh"
#include "kvappend.cuh"

namespace dg {
namespace paged {

constexpr int BQ = 128;
constexpr int BKV = 128;
constexpr int MAX_TILES = 128;  // key tiles per CTA: their page ids and scales sit in shared memory

__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
constexpr int MAX_CLUSTER = 8;  // portable cluster size

// Largest value over a warp (NaN ignored).
__device__ __forceinline__ float warp_top(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Order this thread's shared-memory writes before later accesses of the async
// proxy (the tensor core's operand reads).
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 64-byte-swizzled counterpart of sdesc_sw128 (rows of 64 bytes, 512-byte
// atoms of 8 rows; 16-byte chunk c of row r sits at c ^ ((r >> 1) & 3)).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t lbo_bytes,
                                               uint32_t sbo_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo_bytes >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo_bytes >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(4) << 61;  // 64-byte swizzle
  return d;
}

// Instruction descriptor, kind::f16 with f16 A/B and fp32 D, B MN-major.
__host__ __device__ constexpr uint32_t idesc_f16_f32_bmn(int M, int N) {
  return (1u << 4) | (1u << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Descriptor of a K-major 8-bit tile with rows of HD bytes.
template <int HD>
__device__ __forceinline__ uint64_t sdesc_rows(uint32_t saddr) {
  if constexpr (HD == 128) return sdesc_sw128(saddr, 16, 1024);
  return sdesc_sw64(saddr, 16, 512);
}

// Byte offset of 16-byte chunk c of row r in such a tile.
template <int HD>
__device__ __forceinline__ int swz(int r, int c) {
  if constexpr (HD == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}


// Two fp32 operations in one instruction, and the largest of three values: the
// softmax warps are bound by how many instructions they issue.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi));
  return v;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The larger value; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

struct AttnParams {
  Batch bt;
  int Hq, Hkv, group, causal;
  uint32_t group_mul, group_shift;  // token_of()
  int max_prefix;
  int n_pairs;           // query-row blocks (of 256 packed rows) per kv head
  int tiles_per_split;   // key tiles per CTA
  int n_splits;
  int sorted;            // CTAs outnumber the slots: longest sequences first
  int merge;             // the splits of a unit form a cluster, which merges them
  float scale_log2;      // scale * log2(e)
  const __nv_bfloat16* q;
  int ldq;
  const uint8_t *k_exp, *v_exp;  // [n_pages, Hkv]
  __nv_bfloat16* out;
  int ldo;
  float* lse;       // [T, Hq] or null
  float* part_o;    // [n_splits, T, Hq, hd] (n_splits > 1 without merge)
  float* part_lse;  // [n_splits, T, Hq]
};

// Token of a packed row below 2^31: row / group by a multiplication.  With c =
// ceil(log2 group), mul = floor(2^(31 + c) / group) + 1 and shift = 31 + c the
// error row (mul - 2^shift / group) / 2^shift stays below 1 / group.
__device__ __forceinline__ int token_of(const AttnParams& p, int row) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(row)) * p.group_mul) >>
                          p.group_shift);
}

// Walks packed rows in equal steps: token, head of the group, and the element
// offset token * ld + head * HD that they stand for (a division only at the start).
template <int HD>
struct RowWalk {
  int tok, head;
  int64_t at;
  int step_tok, step_head;
  int64_t step, wrap;
  __device__ __forceinline__ RowWalk(const AttnParams& p, int row, int by, int ld) {
    tok = token_of(p, row);
    head = row - tok * p.group;
    at = static_cast<int64_t>(tok) * ld + head * HD;
    step_tok = token_of(p, by);
    step_head = by - step_tok * p.group;
    step = static_cast<int64_t>(step_tok) * ld + step_head * HD;
    wrap = static_cast<int64_t>(ld) - p.group * HD;
  }
  __device__ __forceinline__ void next(const AttnParams& p) {
    tok += step_tok;
    head += step_head;
    at += step;
    if (head >= p.group) {
      head -= p.group;
      ++tok;
      at += wrap;
    }
  }
};

// The smallest e with amax <= 448 2^e = 1.75 2^(e + 8), at least -100, from
// the bf16 bits of a finite amax.
__device__ __forceinline__ int q_exponent(uint32_t top) {
  return max(static_cast<int>(top >> 7) - 135 + ((top & 0x7Fu) > 0x60u ? 1 : 0), -100);
}

// Eight scaled query elements as e4m3 hi + lo.  x f (f a power of two) fits f16
// exactly down to 2^-17, far below what lo can still hold (2^-10).
__device__ __forceinline__ void split_q(uint4 raw, float f, uint2* hi, uint2* lo) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t h[4], r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 x = __floats2half2_rn(__uint_as_float(w[i] << 16) * f,
                                        __uint_as_float(w[i] & 0xFFFF0000u) * f);
    h[i] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 back = __half2(
        __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(h[i]), __NV_E4M3));
    r[i] = __nv_cvt_halfraw2_to_fp8x2(__half2_raw(__hsub2(x, back)), __NV_SATFINITE, __NV_E4M3);
  }
  *hi = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  *lo = make_uint2(r[0] | (r[1] << 16), r[2] | (r[3] << 16));
}

// 16 bytes global -> shared, asynchronously; zeros when !valid (src is not read).
__device__ __forceinline__ void copy16_async(void* dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}

// A warp brings rows [r0, r0 + ROWS) of a tile of packed query rows (first row
// `first` of `rows` in the kv head's group) into shared memory as hi / lo
// tiles, and stores each row's factor scale_log2 * 2^e.  A row that holds an
// infinity or a NaN gets a NaN factor, so that its scores are NaN; rows past
// the end are zero.  The bf16 row first lands, all rows in flight together, in
// the bytes that its two halves will take: its 16-byte chunk c in chunk
// c % (hd / 16) of hi, then of lo.
template <int HD, int ROWS>
__device__ __forceinline__ void load_q_rows(const AttnParams& p, const Seq& s, int g, int first,
                                            int rows, uint8_t* hi, uint8_t* lo, float* factor,
                                            int r0) {
  constexpr int LANES = HD / 8;                   // lanes per row
  constexpr int PER = 32 / LANES;                 // rows per pass
  constexpr int PASSES = (ROWS + PER - 1) / PER;
  const int lane = lane_id();
  const int c8 = lane % LANES;
  uint8_t* raw = c8 < HD / 16 ? hi : lo;
#pragma unroll 2
  for (int u = 0; u < PASSES; ++u) {
    const int i = u * PER + lane / LANES;
    const int pr = first + r0 + i;
    const int tok = token_of(p, pr);
    const bool valid = pr < rows;
    const __nv_bfloat16* src =
        p.q + (valid ? static_cast<size_t>(s.t0 + tok) * p.ldq +
                           static_cast<size_t>(g * p.group + pr - tok * p.group) * HD + c8 * 8
                     : 0);
    if (i < ROWS) copy16_async(raw + swz<HD>(r0 + i, c8 % (HD / 16)), src, valid);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
#pragma unroll 2
  for (int u = 0; u < PASSES; ++u) {
    const int i = u * PER + lane / LANES;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (i < ROWS)
      x = *reinterpret_cast<const uint4*>(raw + swz<HD>(r0 + i, c8 % (HD / 16)));
    // largest magnitude of the row as bf16 bits (an integer order in which
    // infinities and NaN come last)
    uint32_t top = __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                            __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    top = max(top & 0xFFFFu, top >> 16);
    const bool fine = top < 0x7F80u;
    const int e = q_exponent(top);
    uint2 vh = make_uint2(0u, 0u), vl = make_uint2(0u, 0u);
    if (fine) split_q(x, pow2(-e), &vh, &vl);
    __syncwarp();  // the row has been read
    if (i < ROWS) {
      const int r = r0 + i;
      const int at = swz<HD>(r, c8 >> 1) + (c8 & 1) * 8;
      *reinterpret_cast<uint2*>(hi + at) = vh;
      *reinterpret_cast<uint2*>(lo + at) = vl;
      if (c8 == 0) factor[r] = fine ? p.scale_log2 * pow2(e) : __int_as_float(0x7FC00000);
    }
  }
}

// The same for a 128-row tile by its four softmax warps, a thread per row: a row
// is too long a chain of shuffles and conversions to walk 32 of them per warp
// (6.5 us of a CTA's time; 3.3 us this way, 1.3 us of them the conversions'
// pipe cycles).  The bf16 rows land in `raw` (rows of 2 HD bytes, 16-byte chunk
// c at c ^ (r & 7)): shared memory of ring stages that are not yet in use.
template <int HD>
__device__ __forceinline__ void load_q_tile(const AttnParams& p, const Seq& s, int g, int first,
                                            int rows, uint8_t* raw, uint8_t* hi, uint8_t* lo,
                                            float* factor, int r0, int row) {
  constexpr int LANES = HD / 8;  // 16-byte chunks per row
  constexpr int PER = 32 / LANES;
  const int lane = lane_id();
  const int c8 = lane % LANES;
  const __nv_bfloat16* base = p.q + static_cast<int64_t>(s.t0) * p.ldq +
                              static_cast<int64_t>(g) * p.group * HD + c8 * 8;
  RowWalk<HD> walk(p, first + r0 + lane / LANES, PER, p.ldq);
#pragma unroll 4
  for (int u = 0; u < 32 / PER; ++u) {
    const int r = r0 + u * PER + lane / LANES;
    copy16_async(raw + r * (2 * HD) + ((c8 ^ (r & 7)) << 4), base + walk.at, first + r < rows);
    walk.next(p);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const uint8_t* mine = raw + row * (2 * HD);
  uint32_t top = 0;
#pragma unroll
  for (int c = 0; c < LANES; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(mine + ((c ^ (row & 7)) << 4));
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                                 __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
  }
  top = max(top & 0xFFFFu, top >> 16);
  const bool fine = top < 0x7F80u;
  const int e = fine ? q_exponent(top) : 0;
  factor[row] = fine ? p.scale_log2 * pow2(e) : __int_as_float(0x7FC00000);
  const float f = fine ? pow2(-e) : 0.f;  // a bad row's codes do not matter
#pragma unroll 1
  for (int c0 = 0; c0 < LANES; c0 += 8) {
    uint4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      x[i] = *reinterpret_cast<const uint4*>(mine + (((c0 + i) ^ (row & 7)) << 4));
    uint2 h[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split_q(x[i], f, &h[i], &l[i]);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const int at = swz<HD>(row, (c0 + i) >> 1);
      *reinterpret_cast<uint4*>(hi + at) = make_uint4(h[i].x, h[i].y, h[i + 1].x, h[i + 1].y);
      *reinterpret_cast<uint4*>(lo + at) = make_uint4(l[i].x, l[i].y, l[i + 1].x, l[i + 1].y);
    }
  }
}

// The sequence that comes `want`-th by cached and new rows, longest first (ties
// to the lower index): CTAs start in grid order, and with more of them than fit
// at once the long ones must not be the last.  Every thread of the CTA calls it.
constexpr int MAX_SORTED = 256;
__device__ __forceinline__ int nth_longest(const Batch& bt, int want, int* scratch, int threads) {
  int* len = scratch + 1;
  for (int i = threadIdx.x; i < bt.B; i += threads) {
    const int n = bt.tok_start[i + 1] - bt.tok_start[i];
    len[i] = n > 0 ? bt.cache_len[i] + n : 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < bt.B; i += threads) {
    const int mine = len[i];
    int before = 0;
#pragma unroll 8
    for (int k = 0; k < bt.B; ++k) {
      const int v = len[k];
      before += (v > mine || (v == mine && k < i)) ? 1 : 0;
    }
    if (before == want) *scratch = i;
  }
  __syncthreads();
  return *scratch;
}

// ---------------------------------------------------------------------------
// Many query rows per kv head: two 128-row query tiles per CTA
// ---------------------------------------------------------------------------
// Four warpgroups, with registers moved to the softmax (setmaxnreg):
//   warps 0..3    0 = TMA producer, 1 = TMEM owner + MMA issuer (80 registers)
//   warps 4..11   softmax of tile A / B, one query row per thread (192)
//   warps 12..15  V expansion: codes -> f16 tiles in shared memory, rows past
//                 the visible keys zeroed (48)
// Per key tile and query tile the tensor core does 4 hd 128 128 FLOP as eight
// e4m3 products of the scores (hi, lo) and eight f16 ones with V: 1024 cycles,
// and the special function unit 1024 for the exponentials.  The two query tiles
// take turns: while one's warps form probabilities, the other's products run.
// A pair of tiles takes about 3700 cycles (1.8 us) where 2048 would fill the
// tensor core: what is left is the softmax's own latency (TMEM loads, one warp
// per scheduler) plus the way P -> P V -> next scores, 1300 cycles that only the
// other tile's work covers.  A softmax thread holds its 128 scores in
// registers (read once), and hands P over in two halves of 64 keys, so that P V
// starts while the second half is still being formed.
// Measured: 32 heads x 256 rows over 32768 + 256 keys (hd 128) in 150 us with
// the merge, 0.92 PFLOP/s, 57% of the measured bf16 rate; a 4096-row causal
// prompt behind 1031 rows in 120 us, 54%.  With hd 64 a tile has half the FLOP
// and the same softmax: 133 and 110 us.  Where the key range is short the
// set-up and epilogue of a CTA (8 us) weigh as much as its tiles.  16 bytes of
// a thread's state are spilled.
constexpr int WIDE_THREADS = 512;
constexpr float P_SHIFT = 7.f;  // probabilities are held as 2^(s - m + 7): at most 2^15 in f16
constexpr int V_SHIFT = 7;      // V codes as code 2^(ev - emax + 7): at most 57344 in f16

template <int HD>
struct Wide {
  static constexpr int T_BYTES = BKV * HD;       // K or V codes of a tile; also a hi or lo tile of Q
  static constexpr int V16_BYTES = BKV * HD * 2;
  static constexpr int KST = 3, VST = 2, HST = 2;  // stages of K codes, V codes, V f16
  static constexpr int RING = KST * T_BYTES + VST * T_BYTES + HST * V16_BYTES;
  static constexpr int MAX_PAGES = MAX_TILES * (BKV / 16);
  static constexpr int SMEM_BYTES = 1024 + 4 * T_BYTES + RING + MAX_PAGES * 5 + 2 * BQ * 4 + 512;
  static constexpr uint32_t IDESC_S = idesc_e4m3_f32(BQ, BKV);
  static constexpr uint32_t IDESC_PV = idesc_f16_f32_bmn(BQ, HD);
  static_assert(RING >= 2 * BQ * HD * 4, "O staging does not fit the rings");
  static_assert(V16_BYTES == BQ * HD * 2 && (KST - 1) * T_BYTES >= BQ * HD * 2 && HST == 2,
                "raw query rows do not fit the stages that they pass through");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
  static_assert(80 + 2 * 192 + 48 == 512, "register shares exceed the launch's 128 a thread");
};

template <int HD>
__global__ void __launch_bounds__(WIDE_THREADS, 1)
    wide_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ AttnParams p) {
  using CF = Wide<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;                              // [2 tiles][hi, lo]
  uint8_t* sV16 = sQ + 4 * CF::T_BYTES;            // HST tiles [halves][128][128 B]
  uint8_t* sK = sV16 + CF::HST * CF::V16_BYTES;    // KST tiles, swizzled
  uint8_t* sV8 = sK + CF::KST * CF::T_BYTES;       // VST tiles, plain rows
  float* sQf = reinterpret_cast<float*>(sV8 + CF::VST * CF::T_BYTES);  // [256] row factors
  float* sKf = sQf + 2 * BQ;                                           // [MAX_PAGES] 2^ek
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKf + CF::MAX_PAGES);
  uint64_t* q_full = bars;
  uint64_t* meta_full = q_full + 1;           // page scales are in shared memory
  uint64_t* k_full = meta_full + 1;           // [KST]
  uint64_t* k_empty = k_full + CF::KST;       // [KST]
  uint64_t* v8_full = k_empty + CF::KST;      // [VST]
  uint64_t* v8_empty = v8_full + CF::VST;     // [VST]
  uint64_t* v16_full = v8_empty + CF::VST;    // [HST]
  uint64_t* v16_empty = v16_full + CF::HST;   // [HST]
  uint64_t* s_full = v16_empty + CF::HST;     // [2] per query tile
  uint64_t* p_full = s_full + 2;              // [2 tiles][2 halves]
  uint64_t* o_final = p_full + 4;
  uint64_t* drain = o_final + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* s_emax = reinterpret_cast<int*>(tmem_holder + 2);       // [4]
  uint8_t* sVe = reinterpret_cast<uint8_t*>(tmem_holder + 8);  // [MAX_PAGES] biased ev

  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 8);
    mbar_init(meta_full, 4);
    for (int i = 0; i < CF::KST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < CF::VST; ++i) {
      mbar_init(&v8_full[i], 1);
      mbar_init(&v8_empty[i], 4);
    }
    for (int i = 0; i < CF::HST; ++i) {
      mbar_init(&v16_full[i], 4);
      mbar_init(&v16_empty[i], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    for (int i = 0; i < 4; ++i) mbar_init(&p_full[i], BQ);
    mbar_init(o_final, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();
  const Batch& bt = p.bt;
  // Causal launches take their heaviest row blocks (the last) first, so that
  // the light ones fill the tail of the grid.
  const int nbg = p.Hkv * bt.B;
  const int pi = p.causal ? p.n_pairs - 1 - static_cast<int>(blockIdx.x) / nbg
                          : static_cast<int>(blockIdx.x) % p.n_pairs;
  const int gb = p.causal ? static_cast<int>(blockIdx.x) % nbg
                          : static_cast<int>(blockIdx.x) / p.n_pairs;
  const int g = gb % p.Hkv;
  const int b = p.sorted ? nth_longest(bt, gb / p.Hkv, reinterpret_cast<int*>(sQ), WIDE_THREADS)
                         : gb / p.Hkv;
  const int split = blockIdx.y;
  const Seq s = load_seq(bt, b, p.max_prefix, 0x511,
                         threadIdx.x == 0 && split == 0 && pi == 0 && g == 0);
  const int rows = s.n * p.group;
  const int first = pi * 2 * BQ;
  if (first >= rows) return;
  const bool vB = first + BQ < rows;
  const int total = s.c0 + s.n;
  const int last_tok = token_of(p, min(rows, first + 2 * BQ) - 1);
  const int visible = p.causal ? s.c0 + last_tok + 1 : total;  // keys that this CTA's rows see
  const int tiles = (visible + BKV - 1) / BKV;
  const int t_beg = split * p.tiles_per_split;
  const int n = min(tiles, t_beg + p.tiles_per_split) - t_beg;
  if (n <= 0) return;
  const int log_ppt = 7 - bt.log_page;  // log2(pages per tile)
  const int page_beg = t_beg << log_ppt;
  const int n_pages = ((min(visible, (t_beg + n) * BKV) + bt.page - 1) >> bt.log_page) - page_beg;
  const int32_t* table = bt.page_table + static_cast<size_t>(b) * bt.max_pages + page_beg;

  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch();  // only now: a successor's CTA must not take the TMEM before this one
  const uint32_t tmem = *tmem_holder;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      // Lane l loads page l of the tile.  A page outside the pool is reported
      // by the V expansion and read as zeros (a box past the tensor's end).
      const int ppt = 1 << log_ppt;
      const int page_bytes = bt.page * HD;
      int issued = 0;
      int next = lane < min(ppt, n_pages) ? table[lane] : -1;  // one tile ahead
      for (int j = 0; j < n; ++j) {
        const int ks = j % CF::KST, vs = j % CF::VST;
        const int pages = min(ppt, n_pages - (j << log_ppt));
        const int pg = next;
        if (lane < ppt && ((j + 1) << log_ppt) + lane < n_pages)
          next = table[((j + 1) << log_ppt) + lane];
        bool ok = j == 1 ? mbar_wait(q_full, 0, abort_flag, 0x525)
                         : j < CF::KST ||
                               mbar_wait(&k_empty[ks], ((j / CF::KST) - 1) & 1, abort_flag, 0x521);
        ok = ok && (j < CF::VST ||
                    mbar_wait(&v8_empty[vs], ((j / CF::VST) - 1) & 1, abort_flag, 0x522));
        if (!__all_sync(0xffffffffu, ok)) break;
        if (lane == 0) {
          mbar_expect_tx(&k_full[ks], pages * page_bytes);
          mbar_expect_tx(&v8_full[vs], pages * page_bytes);
        }
        __syncwarp();
        if (lane < pages) {
          const int y = (pg < 0 || pg >= bt.n_pages) ? bt.n_pages * p.Hkv * bt.page
                                                     : (pg * p.Hkv + g) * bt.page;
          tma_load_2d(sK + ks * CF::T_BYTES + lane * page_bytes, &tm_k, &k_full[ks], 0, y);
          tma_load_2d(sV8 + vs * CF::T_BYTES + lane * page_bytes, &tm_v, &v8_full[vs], 0, y);
        }
        issued = j + 1;
      }
      if (*abort_flag && lane == 0) {
        for (int j = max(0, issued - CF::KST); j < issued; ++j)
          mbar_wait(&k_full[j % CF::KST], (j / CF::KST) & 1, nullptr, 0x523);
        for (int j = max(0, issued - CF::VST); j < issued; ++j)
          mbar_wait(&v8_full[j % CF::VST], (j / CF::VST) & 1, nullptr, 0x524);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMA issuer
      // The whole warp walks the schedule, so that descriptors stay in uniform
      // registers; an elected lane issues.
      auto wait_all = [&](uint64_t* bar, uint32_t parity, uint32_t site) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, site));
      };
      bool ok = wait_all(q_full, 0, 0x531);
      // Descriptors advance by adding to their address field (16-byte units).
      const uint64_t q_desc = sdesc_rows<HD>(smem_u32(sQ));
      const uint64_t k_desc = sdesc_rows<HD>(smem_u32(sK));
      const uint64_t v_desc = sdesc_sw128(smem_u32(sV16), BKV * 128, 1024);
      constexpr int TD = CF::T_BYTES >> 4;
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) umma_commit(bar);
      };
      auto issue_s = [&](int X, int ks) {  // S_X = (hi + lo) K^T
        const uint64_t kd = k_desc + ks * TD, qd = q_desc + 2 * X * TD;
        if (elect_one()) {
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int kk = 0; kk < HD / 32; ++kk)
              umma_ss_f8(tmem + X * 128, qd + (part * TD + kk * 2), kd + kk * 2, CF::IDESC_S,
                         (part | kk) ? 1u : 0u);
          umma_commit(&s_full[X]);
        }
      };
      auto issue_pv = [&](int X, int j, int hs) -> bool {
        const uint64_t vd = v_desc + hs * (CF::V16_BYTES >> 4);
        const uint32_t d = tmem + 256 + X * 128, a = tmem + X * 128;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!wait_all(&p_full[2 * X + half], j & 1, 0x533)) return false;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int kk = half * (BKV / 32); kk < (half + 1) * (BKV / 32); ++kk)
              umma_ts(d, a + kk * 8, vd + kk * (16 * 128 / 16), CF::IDESC_PV,
                      kk ? 1u : (j ? 1u : 0u));
          }
        }
        return true;
      };
      if (ok) ok = wait_all(&k_full[0], 0, 0x532);
      if (ok) {
        tc_fence_after();
        issue_s(0, 0);
        if (vB) issue_s(1, 0);
        commit(&k_empty[0]);
      }
      int ks = 0, kph = 0, hs = 0, hph = 0;  // stages and phases of K and of V f16
      for (int j = 0; ok && j < n; ++j) {
        if (++ks == CF::KST) {
          ks = 0;
          kph ^= 1;
        }
        const bool more = j + 1 < n;
        ok = wait_all(&v16_full[hs], hph, 0x534);
        if (ok && more) ok = wait_all(&k_full[ks], kph, 0x532);
        if (ok) ok = issue_pv(0, j, hs);
        if (ok && more) issue_s(0, ks);
        if (ok && vB) ok = issue_pv(1, j, hs);
        if (ok) commit(&v16_empty[hs]);
        if (ok && more) {
          if (vB) issue_s(1, ks);
          commit(&k_empty[ks]);
        }
        if (++hs == CF::HST) {
          hs = 0;
          hph ^= 1;
        }
      }
      if (ok) commit(o_final);
      commit(drain);
      mbar_wait(drain, 0, nullptr, 0x535);
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ V expansion
    asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
    const int tid = static_cast<int>(threadIdx.x) - 384;
    // scales of the whole key range, and the largest V scale among them
    int emax = 0;
    for (int i = tid; i < (n << log_ppt); i += 128) {
      float kf = 1.f;
      int ve = 0;
      if (i < n_pages) {
        const int pg = table[i];
        if (pg < 0 || pg >= bt.n_pages) {
          raise_error(ERR_CHECK | 0x512, static_cast<uint32_t>(b));
        } else {
          const size_t at = static_cast<size_t>(pg) * p.Hkv + g;
          kf = __uint_as_float(static_cast<uint32_t>(p.k_exp[at]) << 23);
          ve = p.v_exp[at];
        }
      }
      sKf[i] = kf;
      sVe[i] = static_cast<uint8_t>(ve);
      emax = max(emax, ve);
    }
    emax = __reduce_max_sync(0xffffffffu, emax);
    if (lane == 0) s_emax[warp - 12] = emax;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    emax = max(max(s_emax[0], s_emax[1]), max(s_emax[2], s_emax[3]));
    if (lane == 0) mbar_arrive(meta_full);
    constexpr int CPR = HD / 16;            // 16-code chunks per row
    constexpr int RSTEP = 128 / CPR;        // rows per pass
    constexpr int PASSES = BKV / RSTEP;
    const int c = tid % CPR;
    const int r0 = tid / CPR;
    // 16 codes -> two 16-byte chunks 2 (c % 4), + 1 of half c / 4, swizzled;
    // the halves write their chunks in opposite order (no bank conflicts)
    const int half_off = (c >> 2) * (BKV * 128);
    const int odd = (c >> 2) & 1;
    const int ch0 = (2 * (c & 3)) | odd;
    for (int j = 0; j < n; ++j) {
      const int vs = j % CF::VST, hs = j % CF::HST;
      bool ok = mbar_wait(&v8_full[vs], (j / CF::VST) & 1, abort_flag, 0x541);
      ok = ok && (j == 0 || (j == 1 ? mbar_wait(q_full, 0, abort_flag, 0x543)
                                    : mbar_wait(&v16_empty[hs], ((j / CF::HST) - 1) & 1,
                                                abort_flag, 0x542)));
      if (!__all_sync(0xffffffffu, ok)) break;
      const uint8_t* src = sV8 + vs * CF::T_BYTES;
      uint8_t* dst = sV16 + hs * CF::V16_BYTES + half_off;
      const int live = visible - (t_beg + j) * BKV;  // rows of this tile that were loaded
#pragma unroll 2
      for (int u = 0; u < PASSES; ++u) {
        const int r = r0 + u * RSTEP;
        uint4 lo = make_uint4(0u, 0u, 0u, 0u), hi = lo;
        if (r < live) {
          const int k = static_cast<int>(sVe[(j << log_ppt) + (r >> bt.log_page)]) - emax + V_SHIFT;
          const uint32_t fb = k >= -14 ? static_cast<uint32_t>(k + 15) << 10
                                       : (k >= -24 ? 1u << (k + 24) : 0u);
          const __half2 f = __half2(__ushort_as_half(static_cast<unsigned short>(fb)),
                                    __ushort_as_half(static_cast<unsigned short>(fb)));
          const uint4 raw = *reinterpret_cast<const uint4*>(src + r * HD + c * 16);
          const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
          uint32_t o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(
                static_cast<__nv_fp8x2_storage_t>((w[e >> 1] >> (16 * (e & 1))) & 0xFFFFu),
                __NV_E4M3));
            const __half2 m = __hmul2(h, f);
            o[e] = *reinterpret_cast<const uint32_t*>(&m);
          }
          lo = make_uint4(o[0], o[1], o[2], o[3]);
          hi = make_uint4(o[4], o[5], o[6], o[7]);
        }
        uint8_t* row = dst + r * 128;
        *reinterpret_cast<uint4*>(row + ((ch0 ^ (r & 7)) << 4)) = odd ? hi : lo;
        *reinterpret_cast<uint4*>(row + (((ch0 ^ 1) ^ (r & 7)) << 4)) = odd ? lo : hi;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&v16_full[hs]);
        mbar_arrive(&v8_empty[vs]);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax (tile X)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    const int X = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const int qrow = first + X * BQ + r;  // packed row
    bool ok = X == 0 || vB;
    // The raw rows pass through V f16's second stage (tile A) and the K codes'
    // second and third (tile B); their first writers wait for q_full.
    if (ok)
      load_q_tile<HD>(p, s, g, first + X * BQ, rows,
                      X == 0 ? sV16 + CF::V16_BYTES : sK + CF::T_BYTES, sQ + 2 * X * CF::T_BYTES,
                      sQ + (2 * X + 1) * CF::T_BYTES, sQf + X * BQ, quarter * 32, r);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    if (ok) {
      ok = __all_sync(0xffffffffu, mbar_wait(meta_full, 0, abort_flag, 0x552));
    }
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t tS = tmem + X * 128 + lane_off;
    const uint32_t tO = tmem + 256 + X * 128 + lane_off;
    float m = -INFINITY;  // running max in log2 units
    float l = 0.f;
    const float sc = ok ? sQf[X * BQ + r] : 0.f;
    // keys [0, sees) are visible to this row
    const int sees = p.causal ? min(total, s.c0 + token_of(p, qrow) + 1) : total;
    // keys [0, open_keys) are visible to every row of the CTA
    const int open_keys = p.causal ? s.c0 + token_of(p, first) + 1 : total;
    for (int j = 0; j < n && ok; ++j) {
      // row factor times the page scale, per 16 columns; never zero, which a
      // masked score of -infinity must not meet
      float scg[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        scg[q] = max_nan(sc * sKf[(j << log_ppt) + ((q * 16) >> bt.log_page)], FLT_MIN);
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[X], j & 1, abort_flag, 0x551))) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sa[128];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        tmem_ld32(tS + h * 32, *reinterpret_cast<uint32_t(*)[32]>(&sa[32 * h]));
      const int lim = sees - (t_beg + j) * BKV - 1;  // columns [0, lim] are visible
      const bool edge = (t_beg + j + 1) * BKV > open_keys;
      tmem_ld_wait();
      if (edge) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > lim) sa[c] = __float_as_uint(-INFINITY);
      }
      // 32 keys' probabilities as packed f16 pairs, their sums added to rs
      uint64_t rs[2] = {0, 0};
      auto probs = [&](const uint32_t* x, float f0, float f1, float neg_m, uint32_t* pk) {
        const uint64_t m2 = pack2(neg_m, neg_m);
        const uint64_t ff[2] = {pack2(f0, f0), pack2(f1, f1)};
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float2 e = unpack2(fma2(pack2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])),
                                        ff[c >> 3], m2));
          const float p0 = attn::fast_exp2(e.x), p1 = attn::fast_exp2(e.y);
          rs[c & 1] = add2(rs[c & 1], pack2(p0, p1));
          const __half2 a = __floats2half2_rn(p0, p1);
          pk[c] = *reinterpret_cast<const uint32_t*>(&a);
        }
      };
      // The first 64 keys' exponentials are formed with the maximum as it
      // stands while the tile's own maximum is found beside them (the special
      // function unit is what bounds this loop; the maximum is free there).
      // Only where it grew by more than 2^8 are they formed again.
      uint32_t pk[32];
      float tmax = -INFINITY;
      {
        const float neg_m = P_SHIFT - m;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          probs(&sa[32 * h], scg[2 * h], scg[2 * h + 1], neg_m, &pk[16 * h]);
#pragma unroll
          for (int q = 4 * h; q < 4 * h + 4; ++q) {
            float m0 = __uint_as_float(sa[16 * q]), m1 = __uint_as_float(sa[16 * q + 1]);
#pragma unroll
            for (int c = 2; c < 14; c += 4) {
              m0 = max3(m0, __uint_as_float(sa[16 * q + c]), __uint_as_float(sa[16 * q + c + 1]));
              m1 = max3(m1, __uint_as_float(sa[16 * q + c + 2]), __uint_as_float(sa[16 * q + c + 3]));
            }
            m0 = max3(m0, __uint_as_float(sa[16 * q + 14]), __uint_as_float(sa[16 * q + 15]));
            tmax = fmaxf(tmax, fmaxf(m0, m1) * scg[q]);
          }
        }
      }
      const bool want = tmax > m + attn::kRescaleThreshold || m == -INFINITY;
      if (__any_sync(0xffffffffu, want)) {
        // Raise the maximum (1/l keeps a lagging one exact).  PV_X(j-1) is
        // complete because S_X(j) is.
        const float m_new = fmaxf(tmax, m);
        if (j > 0) {
          const float f = (m == -INFINITY) ? 0.f : attn::fast_exp2(m - m_new);
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(tO + c * 16, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(tO + c * 16, o);
          }
          l *= f;
        }
        m = m_new;
        const float neg_m = (m == -INFINITY) ? 0.f : P_SHIFT - m;
        rs[0] = rs[1] = 0;
        // (from TMEM again: kept in registers, the scores would cost spills)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t again[32];
          tmem_ld32(tS + h * 32, again);
          tmem_ld_wait();
          if (edge) {
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (h * 32 + c > lim) again[c] = __float_as_uint(-INFINITY);
          }
          probs(again, scg[2 * h], scg[2 * h + 1], neg_m, &pk[16 * h]);
        }
      }
      // P takes the first half of S's columns
      tmem_st32(tS, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[2 * X]);
      const float neg_m = (m == -INFINITY) ? 0.f : P_SHIFT - m;
      probs(&sa[64], scg[4], scg[5], neg_m, &pk[0]);
      probs(&sa[96], scg[6], scg[7], neg_m, &pk[16]);
      tmem_st32(tS + 32, pk);
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[2 * X + 1]);
      const float2 sum = unpack2(add2(rs[0], rs[1]));
      l += sum.x + sum.y;
    }
    const bool fin = __all_sync(0xffffffffu, ok && mbar_wait(o_final, 0, abort_flag, 0x553));
    // Stage O_X in the idle rings (rows XOR-swizzled by 16-byte chunk), then
    // write whole rows: coalesced stores, fp32 partials or bf16 results.
    if (fin) {
      float* stage = reinterpret_cast<float*>(sV16) + X * (BQ * HD);
      int emax = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) emax = max(emax, s_emax[i]);
      // probabilities carry 2^P_SHIFT in O and in l alike; V carries 2^(V_SHIFT - emax)
      const int e_out = emax - 127 - V_SHIFT;
      const float inv = l == 0.f ? 0.f : exp2f(static_cast<float>(max(e_out, -64))) / l;
      // what a very small scale lacks, so that the quotient keeps its bits
      const float rest = exp2f(static_cast<float>(min(e_out + 64, 0)));
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < HD / 64; ++c) {
        uint32_t o[2][32];
        tmem_ld32(tO + c * 64, o[0]);
        tmem_ld32(tO + c * 64 + 32, o[1]);
        tmem_ld_wait();
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const uint32_t* x = &o[v >> 3][(v & 7) * 4];
          float4 y = make_float4(__uint_as_float(x[0]) * inv, __uint_as_float(x[1]) * inv,
                                 __uint_as_float(x[2]) * inv, __uint_as_float(x[3]) * inv);
          if (e_out < -64) {
            y.x *= rest;
            y.y *= rest;
            y.z *= rest;
            y.w *= rest;
          }
          reinterpret_cast<float4*>(stage + r * HD)[(c * 16 + v) ^ (r & 7)] = y;
        }
      }
      if (qrow < rows) {
        const int tok = token_of(p, qrow);
        const size_t at =
            static_cast<size_t>(s.t0 + tok) * p.Hq + g * p.group + qrow - tok * p.group;
        const float z = l == 0.f ? -INFINITY : (m - P_SHIFT + log2f(l)) * 0.69314718055994531f;
        if (p.n_splits > 1)
          p.part_lse[static_cast<size_t>(split) * bt.T * p.Hq + at] = z;
        else if (p.lse)
          p.lse[at] = z;
      }
      __syncwarp();  // a warp writes the rows that it staged
      constexpr int CPR = HD / 4;
      constexpr int RPW = 32 / CPR;  // rows per pass (1 or 2)
      const int cc = lane % CPR;
      constexpr int BATCH = 8;  // loads ahead of the stores: the compiler keeps their order
      const int pr0 = first + X * BQ + quarter * 32 + lane / CPR;
      // partial rows [split][token][head][HD] or results [token][ldo]
      const bool direct = p.n_splits == 1;
      RowWalk<HD> walk(p, pr0, RPW, direct ? p.ldo : p.Hq * HD);
      const int64_t base = static_cast<int64_t>(g) * p.group * HD + cc * 4;
      __nv_bfloat16* out = p.out + static_cast<int64_t>(s.t0) * p.ldo + base;
      float* part = p.part_o +
                    (static_cast<int64_t>(split) * bt.T + s.t0) * p.Hq * HD + base;
#pragma unroll 1
      for (int k0 = 0; k0 < 32; k0 += BATCH * RPW) {
        float4 v[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int rr = quarter * 32 + k0 + i * RPW + lane / CPR;
          v[i] = reinterpret_cast<const float4*>(stage + rr * HD)[cc ^ (rr & 7)];
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          if (pr0 + k0 + i * RPW < rows) {
            if (direct)
              *reinterpret_cast<uint2*>(out + walk.at) =
                  make_uint2(pack_bf16x2(v[i].x, v[i].y), pack_bf16x2(v[i].z, v[i].w));
            else
              *reinterpret_cast<float4*>(part + walk.at) = v[i];
          }
          walk.next(p);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Few query rows per kv head (decoding): keys along the tensor core's M
// ---------------------------------------------------------------------------
// With R = group * n_b <= 32 rows a 128-row query tile would be mostly padding,
// and one softmax thread would walk all 128 keys of a tile alone.  So the
// products are transposed: per tile of 128 keys
//     S^T [keys x 2 NR]  = K [hi | lo]^T      A = K tile, B = query halves
//     O^T [hd x 4 NR]   += V^T [p0 p1 p2 p3]  A = V tile (M-major), B = P
// NR (16 or 32) holds the rows.  A thread owns one key: its page's scales are
// per-thread constants and its NR probabilities are 4 x NR bytes, one 16-byte
// store per 16.  A probability p (times the page's V scale) is rounded to f16
// and enters as four e4m3 terms p0 + p1/32 + p2/32^2 + p3/32^3, each the
// rounding of what the terms before left.  Up to p = 2^8 a term's remainder
// times 32 stays within e4m3's range, and the four hold every f16 value
// exactly (the last one's smallest step is f16's, 2^-24): weights keep 2^-11
// of themselves down to 2^-18 of the largest and 2^-29 of that below, so that
// many small ones beside a large one are not lost.  Both products read the
// codes as TMA delivered them: the kernel streams the cache and does nothing
// else to it, and is bound by HBM once there are enough keys.
//
// The running maximum m is common to all keys of the CTA; the first tile sets
// it, and it is only raised when a p would pass 2^8 (the largest starts at 2^4):
// the test costs one barrier with an OR a tile, the raise itself is rare.
//
// Value scales.  With e the exponent of the key's page and E a reference common
// to the CTA, p = 2^(s - m + e - E + 4) goes into the product and p 2^(E - e)
// into the sum.  E is the first tile's largest e and follows one that lies more
// than 2 above it (in a raise); an e below E - 48 counts as E - 48, and its
// values, too small to matter, as zero.  So m is at most 2 above the largest s,
// whatever the scales: when E grows, and with it the product's unit, p keeps
// 2^-27 of the largest probability at the largest scale.  The largest weight's
// part of the sum lies between 2^2 and 2^56, and weights down to 2^-80 of it
// are not lost.
// Measured: 64 sequences of 8193 keys, 32 / 8 heads, hd 128: 164 us, 6.5 TB/s,
// the measured copy rate; of 20 to 100% of that length 109 us, 90%; one
// sequence of 4097 keys 9.9 us, which is launch, first loads and the merge.
// Otherwise a tile's chain of scores, barrier, P and P V bounds it.  With hd 64
// a tile has half the bytes and the same chain: 136 us for the 64 of 8193,
// where the bytes need 82.  With 17 to 32 rows a thread holds 32 scores and
// sums (254 registers, one CTA an SM): 16 sequences of 8193 keys in 93 us at 20
// rows and 108 at 32, where the bytes need 41.
// Two CTAs an SM for NR = 16: 146 registers, no spills.  With hd 64 shared
// memory would hold three, at 96 registers and 340 bytes of spill loads: 162 us
// instead of 136, 300 sequences of 301 keys 65 instead of 70.
//
// Warps: 0 = TMA producer, 1 = TMEM owner + MMA issuer, 2..5 = softmax (thread
// = key; at the end thread = element of the head).
constexpr int NARROW_THREADS = 192;
constexpr float N_SHIFT = 4.f;
constexpr float N_LIMIT = 8.f;
constexpr int V_SPREAD = 48;     // value scales further below the reference are left out
constexpr int V_LAG = 2;         // how far one may lie above it (0: 0.4 us of 10 and 1 of 109 more)
constexpr int P_TERMS = 4;       // e4m3 terms of a probability
constexpr float P_STEP = 32.f;   // between them

template <int HD, int NR>
struct Narrow {
  static constexpr int T_BYTES = BKV * HD;
  static constexpr int STAGES = 3;
  static constexpr int PB = 4 * NR;  // bytes of a P row
  static constexpr int P_BYTES = BKV * PB;
  static constexpr int Q_BYTES = 2 * NR * HD;
  static constexpr int TMEM = 8 * NR;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * 2 * T_BYTES + P_BYTES + Q_BYTES + NR * 4 * 8 + 256;
  static_assert((1 + 4 * STAGES + 5) * 8 + 3 * 4 + 4 * 4 <= 256, "barriers, flags and exponents");
  static constexpr uint32_t IDESC_S = idesc_e4m3_f32(BKV, 2 * NR);
  // A and B both M/N-major; the M = 128 lanes beyond a head of 64 are unused
  static constexpr uint32_t IDESC_PV = idesc_e4m3_f32(128, 4 * NR) | (1u << 15) | (1u << 16);
  static_assert(2 * (SMEM_BYTES + 1024) <= 228 * 1024 || NR > 16, "two CTAs per SM");
  // Padding rows are left out from a few places on only: a test every four rows
  // would keep the rows' instructions apart (32 rows: 38 -> 45 us).
  static __device__ __forceinline__ bool stops(int r, int rows) {
    return (NR == 16 ? r == 4 || r == 8 : r == 24) && r >= rows;
  }
  static __device__ __forceinline__ bool skips(int r, int rows) {
    return NR == 16 ? (r >= 8 ? rows <= 8 : r >= 4 && rows <= 4) : r >= 24 && rows <= 24;
  }
};

// OR of a predicate over the named barrier's threads.
__device__ __forceinline__ bool bar_any(int id, int threads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// 16-byte chunk c of P row r (rows of 64 or 128 bytes, swizzled over their width)
template <int NR>
__device__ __forceinline__ int p_swz(int r, int c) {
  return NR == 16 ? swz<64>(r, c) : swz<128>(r, c);
}

template <int HD, int NR>
__global__ void __launch_bounds__(NARROW_THREADS, NR == 32 ? 1 : 2)
    narrow_kernel(const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ AttnParams p) {
  using CF = Narrow<HD, NR>;
  constexpr int ST = CF::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sK = smem;                        // ST tiles
  uint8_t* sV = sK + ST * CF::T_BYTES;       // ST tiles (a head of 64 reads 512 bytes past one)
  uint8_t* sP = sV + ST * CF::T_BYTES;       // [128 keys][p0 | p1 | p2 | p3]
  uint8_t* sQ = sP + CF::P_BYTES;            // [NR hi rows][NR lo rows]
  float* sF = reinterpret_cast<float*>(sQ + CF::Q_BYTES);  // [NR] row factors
  float* sM = sF + NR;                                     // [2][NR] running maxima (log2 units)
  int* sSees = reinterpret_cast<int*>(sM + 2 * NR);        // [NR] visible keys
  float* sRed = reinterpret_cast<float*>(sSees + NR);      // [4][NR]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sRed + 4 * NR);
  uint64_t* q_full = bars;
  uint64_t* k_full = q_full + 1;       // [ST]
  uint64_t* k_empty = k_full + ST;     // [ST]
  uint64_t* v_full = k_empty + ST;     // [ST]
  uint64_t* v_empty = v_full + ST;     // [ST]
  uint64_t* s_full = v_empty + ST;     // [2]
  uint64_t* p_full = s_full + 2;
  uint64_t* pv_done = p_full + 1;
  uint64_t* drain = pv_done + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* s_fail = abort_flag + 1;  // a softmax thread gave up waiting
  int* sE = reinterpret_cast<int*>(tmem_holder + 3);  // [4] largest value exponents of the warps

  const int warp = warp_id();
  const int lane = lane_id();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 4);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(p_full, 128);
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *s_fail = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  griddep_wait();
  const Batch& bt = p.bt;
  const int g = static_cast<int>(blockIdx.x) % p.Hkv;
  const int bx = static_cast<int>(blockIdx.x) / p.Hkv;
  const int b = p.sorted ? nth_longest(bt, bx, reinterpret_cast<int*>(sP), NARROW_THREADS) : bx;
  const int split = blockIdx.y;
  const Seq s = load_seq(bt, b, p.max_prefix, 0x511, threadIdx.x == 0 && split == 0 && g == 0);
  const int rows = s.n * p.group;
  if (rows == 0) return;
  const int total = s.c0 + s.n;
  const int tiles = (total + BKV - 1) / BKV;
  const int t_beg = split * p.tiles_per_split;
  const int n = min(tiles, t_beg + p.tiles_per_split) - t_beg;
  const bool idle = n <= 0;  // no key of this split exists
  if (idle && !p.merge) return;
  const int log_ppt = 7 - bt.log_page;
  const int pages = (total + bt.page - 1) >> bt.log_page;  // of the sequence
  const int32_t* table = bt.page_table + static_cast<size_t>(b) * bt.max_pages;

  if (warp == 1 && !idle) {
    tmem_alloc(tmem_holder, CF::TMEM);
    tmem_relinquish();
  }
  if (threadIdx.x >= 64 && threadIdx.x < 64 + NR) {
    const int r = static_cast<int>(threadIdx.x) - 64;
    sM[r] = 0.f;
    sSees[r] = p.causal ? min(total, s.c0 + token_of(p, r) + 1) : total;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch();  // only now: a successor's CTA must not take the TMEM before this one
  const uint32_t tmem = *tmem_holder;

  if (idle) {
    if (threadIdx.x < NR) sF[threadIdx.x] = 0.f;  // no weight
  } else if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int ppt = 1 << log_ppt;
    const int page_bytes = bt.page * HD;
    int issued_k = 0, issued_v = 0;
    int next = -1;  // page id of the next tile, loaded one tile ahead
    if (lane < ppt && (t_beg << log_ppt) + lane < pages) next = table[(t_beg << log_ppt) + lane];
    for (int j = 0; j < n; ++j) {
      const int st = j % ST;
      const int base = (t_beg + j) << log_ppt;
      const int here = min(ppt, pages - base);
      int pg = next;
      if (j + 1 < n && lane < ppt && base + ppt + lane < pages) next = table[base + ppt + lane];
      const int y = (pg < 0 || pg >= bt.n_pages) ? bt.n_pages * p.Hkv * bt.page
                                                 : (pg * p.Hkv + g) * bt.page;
      bool ok = j < ST || mbar_wait(&k_empty[st], ((j / ST) - 1) & 1, abort_flag, 0x561);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_expect_tx(&k_full[st], here * page_bytes);
      __syncwarp();
      if (lane < here)
        tma_load_2d(sK + st * CF::T_BYTES + lane * page_bytes, &tm_k, &k_full[st], 0, y);
      issued_k = j + 1;
      ok = j < ST || mbar_wait(&v_empty[st], ((j / ST) - 1) & 1, abort_flag, 0x562);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) mbar_expect_tx(&v_full[st], here * page_bytes);
      __syncwarp();
      if (lane < here)
        tma_load_2d(sV + st * CF::T_BYTES + lane * page_bytes, &tm_v, &v_full[st], 0, y);
      issued_v = j + 1;
    }
    if (*abort_flag && lane == 0) {
      for (int j = max(0, issued_k - ST); j < issued_k; ++j)
        mbar_wait(&k_full[j % ST], (j / ST) & 1, nullptr, 0x563);
      for (int j = max(0, issued_v - ST); j < issued_v; ++j)
        mbar_wait(&v_full[j % ST], (j / ST) & 1, nullptr, 0x564);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      bool ok = mbar_wait(q_full, 0, abort_flag, 0x571);
      const uint64_t q_desc = sdesc_rows<HD>(smem_u32(sQ));
      const uint64_t k_desc = sdesc_rows<HD>(smem_u32(sK));
      // 32 keys a step: four 8-row groups of V and of P
      const uint64_t v_desc = HD == 128 ? sdesc_sw128(smem_u32(sV), 1024, 1024)
                                        : sdesc_sw64(smem_u32(sV), 512, 512);
      const uint64_t p_desc = NR == 16 ? sdesc_sw64(smem_u32(sP), 512, 512)
                                       : sdesc_sw128(smem_u32(sP), 1024, 1024);
      auto issue_s = [&](int j) -> bool {
        const int st = j % ST;
        if (!mbar_wait(&k_full[st], (j / ST) & 1, abort_flag, 0x572)) return false;
        tc_fence_after();
        const uint64_t kd = k_desc + st * (CF::T_BYTES >> 4);
#pragma unroll
        for (int kk = 0; kk < HD / 32; ++kk)
          umma_ss_f8(tmem + (j & 1) * 2 * NR, kd + kk * 2, q_desc + kk * 2, CF::IDESC_S,
                     kk ? 1u : 0u);
        umma_commit(&s_full[j & 1]);
        umma_commit(&k_empty[st]);
        return true;
      };
      if (ok) ok = issue_s(0);
      if (ok && n > 1) ok = issue_s(1);
      for (int j = 0; ok && j < n; ++j) {
        const int st = j % ST;
        ok = mbar_wait(&v_full[st], (j / ST) & 1, abort_flag, 0x573);
        if (ok) ok = mbar_wait(p_full, j & 1, abort_flag, 0x574);
        if (!ok) break;
        tc_fence_after();
        const uint64_t vd = v_desc + st * (CF::T_BYTES >> 4);
#pragma unroll
        for (int kk = 0; kk < BKV / 32; ++kk)
          umma_ss_f8(tmem + 4 * NR, vd + kk * (32 * HD / 16), p_desc + kk * (32 * CF::PB / 16),
                     CF::IDESC_PV, kk ? 1u : (j ? 1u : 0u));
        umma_commit(pv_done);
        umma_commit(&v_empty[st]);
        if (j + 2 < n) ok = issue_s(j + 2);
      }
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr, 0x575);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quarter = warp & 3;
    const int kl = quarter * 32 + lane;  // key of the tile; later element of the head
    const uint32_t tl = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    // page scales of this thread's key, one tile ahead
    auto page_id = [&](int j) -> int {
      const int at = ((t_beg + j) << log_ppt) + (kl >> bt.log_page);
      return j < n && at < pages ? table[at] : -1;
    };
    auto page_exps = [&](int pg, int* ke, int* ve) {
      *ke = 127;
      *ve = 0;  // no page: below every reference
      if (pg >= 0 && pg < bt.n_pages) {
        const size_t at = static_cast<size_t>(pg) * p.Hkv + g;
        *ke = p.k_exp[at];
        *ve = p.v_exp[at];
      }
    };
    auto check_page = [&](int j, int pg) {
      if ((pg < 0 || pg >= bt.n_pages) && (kl & (bt.page - 1)) == 0 &&
          ((t_beg + j) << log_ppt) + (kl >> bt.log_page) < pages)
        raise_error(ERR_CHECK | 0x512, static_cast<uint32_t>(b));
    };
    int ke, ve;
    int pg = page_id(0);
    load_q_rows<HD, NR / 4>(p, s, g, 0, rows, sQ, sQ + NR * HD, sF, (warp - 2) * (NR / 4));
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    page_exps(pg, &ke, &ve);
    check_page(0, pg);
    pg = page_id(1);
    auto warp_exponents = [&](int e) {
      const int top = __reduce_max_sync(0xffffffffu, e);
      if (lane == 0) sE[quarter] = top;
    };
    auto top_exponent = [&]() { return max(max(sE[0], sE[1]), max(sE[2], sE[3])); };
    warp_exponents(ve);
    const int open_keys = p.causal ? s.c0 + 1 : total;  // keys below are visible to every row
    float l[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) l[r] = 0.f;
    bar_any(1, 128, false);  // row factors and exponents are in place
    int e_ref = top_exponent();
    bool ok = true;
    int cur = 0;  // which of sM holds the maxima
    int j = 0;
    for (; j < n; ++j) {
      const float kf = __uint_as_float(static_cast<uint32_t>(ke) << 23);
      const int ve_now = ve;
      int eff = max(ve_now, e_ref - V_SPREAD);
      const float shift = static_cast<float>(eff - e_ref) + N_SHIFT;
      if (j + 1 < n) {
        page_exps(pg, &ke, &ve);
        check_page(j + 1, pg);
        pg = page_id(j + 2);
      }
      const int pos = (t_beg + j) * BKV + kl;
      const bool edge = (t_beg + j + 1) * BKV > open_keys;
      const uint32_t tS = tl + (j & 1) * 2 * NR;
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(&s_full[j & 1], (j >> 1) & 1, abort_flag, 0x581));
      tc_fence_after();
      float x[NR];
      // x = score in log2 units + shift (the V scale) - running maximum
      const float* m_now = sM + cur * NR;
      bool above = ve_now > e_ref + V_LAG;
#pragma unroll
      for (int c = 0; c < NR; c += 16) {
        uint32_t hi[16], lo[16];
        tmem_ld16(tS + c, hi);
        tmem_ld16(tS + NR + c, lo);
        tmem_ld_wait();
#pragma unroll
        for (int q = 0; q < 16; q += 4) {
          if (CF::stops(c + q, rows)) break;
          const float4 f = *reinterpret_cast<const float4*>(sF + c + q);
          const float4 m = *reinterpret_cast<const float4*>(m_now + c + q);
          const float ff[4] = {f.x, f.y, f.z, f.w}, mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sum = __uint_as_float(hi[q + e]) + __uint_as_float(lo[q + e]);
            x[c + q + e] = fmaf(sum, ff[e] * kf, shift - mm[e]);
            if (edge && pos >= sSees[c + q + e]) x[c + q + e] = -INFINITY;
            above = above || x[c + q + e] > N_LIMIT;
          }
        }
      }
      bool raise = j == 0;  // the first tile sets the maxima without a test
      if (j > 0) {
        if (!ok) *s_fail = 1;
        raise = bar_any(1, 128, above || !ok);
      } else if (!ok) {
        *s_fail = 1;
      }
      if (raise) {
        float shrink = 1.f;  // 2^ of how far the reference exponent falls behind
        if (j > 0) {
          warp_exponents(ve_now);
          bar_any(1, 128, false);
          const int top = top_exponent();
          if (top > e_ref + V_LAG) {
            const int was = eff;
            eff = max(eff, top - V_SPREAD);
            const float move = static_cast<float>(eff - was - (top - e_ref));
            shrink = attn::fast_exp2(static_cast<float>(e_ref - top));
#pragma unroll
            for (int r = 0; r < NR; ++r) x[r] += move;
            e_ref = top;
          }
        }
        // raise the maxima to this tile's
#pragma unroll
        for (int r = 0; r < NR; r += 4) {
          if (CF::stops(r, rows)) break;
          const float4 v = make_float4(warp_top(x[r]), warp_top(x[r + 1]), warp_top(x[r + 2]),
                                       warp_top(x[r + 3]));
          if (lane == 0) *reinterpret_cast<float4*>(sRed + quarter * NR + r) = v;
        }
        if (j > 0) {
          ok = __all_sync(0xffffffffu, ok && mbar_wait(pv_done, (j - 1) & 1, abort_flag, 0x582));
          tc_fence_after();
        }
        bar_any(1, 128, false);
        // s_fail is written before a barrier only, and read only behind the
        // next: every thread sees the same
        if (*s_fail) break;
        float* m_next = sM + (cur ^ 1) * NR;
        float mine = 0.f;
#pragma unroll
        for (int c = 0; c < NR; c += 16) {
          float fac[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int r = c + e;
            fac[e] = 1.f;
            if (CF::skips(r, rows)) continue;
            // how far the tile's maximum lies above the running one; the first
            // tile's becomes the running one either way, unless the row sees no key
            const float d = fmaxf(fmaxf(sRed[r], sRed[NR + r]),
                                  fmaxf(sRed[2 * NR + r], sRed[3 * NR + r])) - N_SHIFT;
            const float up = d == -INFINITY ? 0.f : (j > 0 ? fmaxf(d, 0.f) : d);
            // (the first tile, with nothing summed before it, has an up of any
            // sign: 2^-up may be infinite, and times the empty sums NaN)
            fac[e] = attn::fast_exp2(-fmaxf(up, 0.f));
            l[r] *= fac[e];
            x[r] -= up;
            if (r == kl) mine = m_now[r] + up;
          }
          if (j > 0) {
#pragma unroll
            for (int term = 0; term < P_TERMS; ++term) {
              uint32_t o[16];
              tmem_ld16(tl + 4 * NR + term * NR + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e)
                o[e] = __float_as_uint(__uint_as_float(o[e]) * (fac[e] * shrink));
              tmem_st16(tl + 4 * NR + term * NR + c, o);
            }
          }
        }
        tmem_st_wait();
        if (kl < NR) m_next[kl] = mine;
        cur ^= 1;
        bar_any(1, 128, false);
      }
      const float l_scale = pow2(e_ref - eff);
      // P rows may be rewritten once the previous product has read them
      if (j > 0)
        ok = __all_sync(0xffffffffu, ok && mbar_wait(pv_done, (j - 1) & 1, abort_flag, 0x583));
#pragma unroll
      for (int c = 0; c < NR; c += 16) {
        uint32_t w[P_TERMS][4] = {};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (CF::stops(c + 4 * q, rows)) break;
          uint32_t term[P_TERMS][2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = c + 4 * q + 2 * e;
            const float p0 = attn::fast_exp2(x[r]), p1 = attn::fast_exp2(x[r + 1]);
            l[r] = fmaf(p0, l_scale, l[r]);
            l[r + 1] = fmaf(p1, l_scale, l[r + 1]);
            __half2 rest = __floats2half2_rn(p0, p1);
#pragma unroll
            for (int t = 0; t < P_TERMS; ++t) {
              const __nv_fp8x2_storage_t code =
                  __nv_cvt_halfraw2_to_fp8x2(__half2_raw(rest), __NV_SATFINITE, __NV_E4M3);
              term[t][e] = code;
              if (t < P_TERMS - 1)
                rest = __hmul2(__hsub2(rest, __half2(__nv_cvt_fp8x2_to_halfraw2(code, __NV_E4M3))),
                               __float2half2_rn(P_STEP));
            }
          }
#pragma unroll
          for (int t = 0; t < P_TERMS; ++t) w[t][q] = term[t][0] | (term[t][1] << 16);
        }
#pragma unroll
        for (int t = 0; t < P_TERMS; ++t)
          *reinterpret_cast<uint4*>(sP + p_swz<NR>(kl, t * (NR / 16) + c / 16)) =
              make_uint4(w[t][0], w[t][1], w[t][2], w[t][3]);
      }
      if (ve_now < eff) {  // (the values count as zero, but the weights as weights)
#pragma unroll
        for (int c = 0; c < 4 * NR / 16; ++c)
          *reinterpret_cast<uint4*>(sP + p_swz<NR>(kl, c)) = make_uint4(0u, 0u, 0u, 0u);
      }
      if (pos >= total) {
        // whatever lies behind the sequence's end must not meet the product
        const int st = j % ST;
        ok = mbar_wait(&v_full[st], (j / ST) & 1, abort_flag, 0x584) && ok;
#pragma unroll
        for (int c = 0; c < HD / 16; ++c)
          reinterpret_cast<uint4*>(sV + st * CF::T_BYTES + kl * HD)[c] =
              make_uint4(0u, 0u, 0u, 0u);
      }
      fence_async_smem();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    // ------------------------------------------------------------ results
    ok = __all_sync(0xffffffffu, ok && j == n &&
                                     mbar_wait(pv_done, (n - 1) & 1, abort_flag, 0x585));
    tc_fence_after();
    if (kl < NR && cur) sM[kl] = sM[NR + kl];
    // sum of l over the warp's 32 keys for all rows at once: each exchange
    // halves the rows that a lane still carries
#pragma unroll
    for (int half = NR / 2, bit = 16; bit > 0; bit >>= 1, half >>= 1) {
      const bool up = (lane & bit) != 0;
      if (half > 0) {
#pragma unroll
        for (int r = 0; r < half; ++r) {
          const float give = up ? l[r] : l[r + half];
          const float keep = up ? l[r + half] : l[r];
          l[r] = keep + __shfl_xor_sync(0xffffffffu, give, bit);
        }
      } else {
        l[0] += __shfl_xor_sync(0xffffffffu, l[0], bit);
      }
    }
    // lane bits from the top select the row: bit 16 its highest bit, and so on
    {
      const int r = NR == 32 ? lane : lane >> 1;
      if (NR == 32 || (lane & 1) == 0) sRed[quarter * NR + r] = l[0];
    }
    bar_any(1, 128, false);
    // O^T, a thread per element of the head: value of row r in terms of 2^-m
    float* sO = reinterpret_cast<float*>(sK);  // [NR][HD]; the K stages are idle now
    const int64_t part = static_cast<int64_t>(split) * bt.T * p.Hq;
    float sum = 0.f;
    if (kl < NR) {
      sum = (sRed[kl] + sRed[NR + kl]) + (sRed[2 * NR + kl] + sRed[3 * NR + kl]);
      if (!ok) sum = 0.f;
      sRed[kl] = sum == 0.f ? 0.f : 1.f / sum;  // this thread alone reads it above
      sF[kl] = sum;
    }
    const float v_scale = pow2(e_ref - 127);
    if (kl < rows && !p.merge) {
      const int tok = token_of(p, kl);
      const int64_t at = static_cast<int64_t>(s.t0 + tok) * p.Hq + g * p.group + kl - tok * p.group;
      const float z = sum == 0.f ? -INFINITY
                                 : (sM[kl] - N_SHIFT + log2f(sum)) * 0.69314718055994531f;
      if (p.n_splits > 1)
        p.part_lse[part + at] = z;
      else if (p.lse)
        p.lse[at] = z;
    }
    bar_any(1, 128, false);
    int tok = 0, hh = 0;
#pragma unroll
    for (int c = 0; c < NR; c += 16) {
      if (c >= rows) break;
      uint32_t o[P_TERMS][16];
#pragma unroll
      for (int t = 0; t < P_TERMS; ++t) tmem_ld16(tl + (4 + t) * NR + c, o[t]);
      tmem_ld_wait();
      if (kl < HD) {
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int r = c + e;
          if (r >= rows) break;
          float v = __uint_as_float(o[P_TERMS - 1][e]);
#pragma unroll
          for (int t = P_TERMS - 2; t >= 0; --t)
            v = fmaf(v, 1.f / P_STEP, __uint_as_float(o[t][e]));
          v = v * sRed[r] * v_scale;  // (their product might overflow)
          const int h = g * p.group + hh;
          if (p.merge)
            sO[r * HD + kl] = v;
          else if (p.n_splits > 1)
            p.part_o[(part + static_cast<int64_t>(s.t0 + tok) * p.Hq + h) * HD + kl] = v;
          else
            p.out[static_cast<int64_t>(s.t0 + tok) * p.ldo + h * HD + kl] = __float2bfloat16_rn(v);
          if (++hh == p.group) {
            hh = 0;
            ++tok;
          }
        }
      }
    }
  }
  if (p.merge) {
    // Every split's results, sums (sF) and maxima (sM) lie in its CTA's shared
    // memory; the CTAs of the cluster share the rows x hd results.
    cluster_arrive_wait();
    if (threadIdx.x >= 64) {
      const int S = p.n_splits;
      uint32_t o_at[MAX_CLUSTER], f_at[MAX_CLUSTER], m_at[MAX_CLUSTER];
#pragma unroll
      for (int k = 0; k < MAX_CLUSTER; ++k) {
        o_at[k] = cluster_addr(sK, min(k, S - 1));
        f_at[k] = cluster_addr(sF, min(k, S - 1));
        m_at[k] = cluster_addr(sM, min(k, S - 1));
      }
      for (int i = split * 128 + static_cast<int>(threadIdx.x) - 64; i < rows * HD; i += S * 128) {
        const int r = i / HD;
        float o[MAX_CLUSTER], f[MAX_CLUSTER], m[MAX_CLUSTER];
#pragma unroll
        for (int k = 0; k < MAX_CLUSTER; ++k) {
          m[k] = k < S ? ld_cluster(m_at[k] + r * 4) : -INFINITY;
          f[k] = k < S ? ld_cluster(f_at[k] + r * 4) : 0.f;
          o[k] = k < S ? ld_cluster(o_at[k] + i * 4) : 0.f;
        }
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < MAX_CLUSTER; ++k)
          if (f[k] != 0.f) top = fmaxf(top, m[k]);
        float sum = 0.f, v = 0.f;
#pragma unroll
        for (int k = 0; k < MAX_CLUSTER; ++k) {
          // a split without a visible key weighs nothing, whatever it left
          if (f[k] != 0.f) f[k] *= attn::fast_exp2(m[k] - top);
          sum += f[k];
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int k = 0; k < MAX_CLUSTER; ++k)
          if (f[k] != 0.f) v = fmaf(f[k] * inv, o[k], v);
        const int tok = token_of(p, r);
        const int h = g * p.group + r - tok * p.group;
        p.out[static_cast<int64_t>(s.t0 + tok) * p.ldo + h * HD + (i & (HD - 1))] =
            __float2bfloat16_rn(v);
        if (p.lse && (i & (HD - 1)) == 0)
          p.lse[static_cast<int64_t>(s.t0 + tok) * p.Hq + h] =
              sum == 0.f ? -INFINITY : (top - N_SHIFT + log2f(sum)) * 0.69314718055994531f;
      }
    }
    cluster_arrive_wait();  // no CTA leaves while another reads its shared memory
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1 && !idle) {
    tc_fence_after();
    tmem_dealloc(tmem, CF::TMEM);
  }
}

// ---------------------------------------------------------------------------
// Merge of the key-range splits: out = sum_s w_s O_s / sum_s w_s with
// w_s = 2^(lse_s - max).  A warp per (token, head); only the splits that the
// row's visible keys reach were written, and only those are read, in order.
// The sum is kept divided by its weights, so that it stays as large as a value.
// ---------------------------------------------------------------------------
// Lane s reads split s's log-sum-exp, so every weight is known after one load,
// beside which the first COMBINE_BATCH partial rows are already on their way.
constexpr int COMBINE_THREADS = 256;
constexpr int COMBINE_BATCH = 12;

template <int HD>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(const AttnParams p) {
  constexpr int PER = HD / 32;
  griddep_launch();
  griddep_wait();
  const int b = blockIdx.y;
  const int lane = lane_id();
  const int item = static_cast<int>(blockIdx.x) * (COMBINE_THREADS / 32) + warp_id();
  const Seq s = load_seq(p.bt, b, p.max_prefix, 0x511, false);
  const int tok = item / p.Hq;
  if (tok >= s.n) return;
  const int h = item - tok * p.Hq;
  const int sees = p.causal ? s.c0 + tok + 1 : s.c0 + s.n;
  const int S = (((sees + BKV - 1) / BKV) + p.tiles_per_split - 1) / p.tiles_per_split;
  const size_t row = static_cast<size_t>(s.t0 + tok) * p.Hq + h;
  const size_t stride = static_cast<size_t>(p.bt.T) * p.Hq;
  float mx = -INFINITY, wsum = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int s0 = 0; s0 < S; s0 += 32) {
    const int here = min(32, S - s0);
    float v[COMBINE_BATCH][PER];
    auto load = [&](int k0) {
#pragma unroll
      for (int k = 0; k < COMBINE_BATCH; ++k) {
        const float* src = p.part_o + ((s0 + k0 + k) * stride + row) * HD + lane * PER;
#pragma unroll
        for (int e = 0; e < PER; e += 2) {
          const float2 x = k0 + k < here ? *reinterpret_cast<const float2*>(src + e)
                                         : make_float2(0.f, 0.f);
          v[k][e] = x.x;
          v[k][e + 1] = x.y;
        }
      }
    };
    load(0);  // in flight beside the log-sum-exps
    const float z = lane < here ? p.part_lse[(s0 + lane) * stride + row] : -INFINITY;
    const float top = fmaxf(warp_top(z), mx);
    const float f = mx == -INFINITY ? 0.f : expf(mx - top);
    // a split without a visible key weighs nothing; a NaN one makes the row NaN
    float w = z == -INFINITY ? 0.f : z != z ? z : expf(z - top);
    const float before = wsum * f;
    wsum = before + warp_sum(w);
    const float inv = wsum == 0.f ? 0.f : 1.f / wsum;
    w *= inv;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] *= before * inv;
    mx = top;
    for (int k0 = 0; k0 < here; k0 += COMBINE_BATCH) {
      if (k0 > 0) load(k0);
#pragma unroll
      for (int k = 0; k < COMBINE_BATCH; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, (k0 + k) & 31);
        if (k0 + k < here) {
#pragma unroll
          for (int e = 0; e < PER; ++e) acc[e] = wk == 0.f ? acc[e] : fmaf(wk, v[k][e], acc[e]);
        }
      }
    }
  }
  __nv_bfloat16* out = p.out + static_cast<size_t>(s.t0 + tok) * p.ldo +
                       static_cast<size_t>(h) * HD + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e], acc[e + 1]);
  if (p.lse && lane == 0) p.lse[row] = wsum == 0.f ? -INFINITY : mx + logf(wsum);
}

}  // namespace paged
}  // namespace dg
