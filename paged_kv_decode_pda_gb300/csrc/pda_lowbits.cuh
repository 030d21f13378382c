// Caches in fewer bits: the writers that find the scales of what they write
// (e4m3 with a scale per token and kv head; e2m1 with a scale per 16 dims) and
// the readers that give a cache's values back as bf16.
//
// The 4-bit record of (block b, kv head h) is 144 * block_size bytes at
// (b * Hk + h) * 144 * block_size:
//   K codes   [bs][64]   byte j of a token: dims 2j (low nibble), 2j + 1
//   V codes   [bs][64]   the same, byte j of slot o at j ^ (o & 2 ? 32 : 0)
//   K scales  [bs][8]    e4m3, one per 16 dims
//   V scales  [bs/16][8][16]   slot t of its 16 at fp4_scale_place(t)
// A value is e2m1 * block scale * tensor scale. e2m1 has 2 significant bits and
// e4m3 4, so e2m1 * block scale is exact in f16 (2^-10 .. 2688). V's order is the
// decode kernel's: its lanes read four tokens' bytes of one block free of bank
// conflicts, and those tokens' scales as one word.
//
// Every rounding to 8 or 4 bits is that of the real quotient (nearest, ties to
// even), whatever the scales' low bits: the quotient is made with a reciprocal,
// off by less than 2^-21, both ends of that range are rounded, and where they
// differ the sign of one fused multiply-add, which is exact, decides.
#pragma once

#include "pda_device.cuh"

namespace pda {

constexpr int kFp4TokenBytes = 144;   // K and V of one (token, kv head): 2 * 64 codes, 2 * 8 scales

// Where slot t of 16 has its V scale: the four tokens of one lane of the decode
// kernel (t & 3 = l, or l ^ 1 in the second and fourth quarter) side by side.
__host__ __device__ __forceinline__ int fp4_scale_place(int t) { return 4 * ((t & 3) ^ ((t >> 2) & 1)) + (t >> 2); }

// Four bytes of e2m1 pairs -> four f16x2 (low nibble in the low half), exact.
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight fp32 -> e2m1 nibbles, v[0] lowest; nearest even, saturating.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) { return f16lo_f32(e4m3x2_lo_to_f16x2(code)); }

// The margin of a quotient made with a reciprocal: three roundings of 2^-24.
constexpr float kQuotLo = 1.f - 4.76837158203125e-07f;   // 1 -+ 2^-21
constexpr float kQuotHi = 1.f + 4.76837158203125e-07f;

// Which of two neighbouring codes (magnitudes lo, lo + 1, whose midpoint is
// `mid` units) is nearest to |x|: |x| - mid * unit, rounded once, has the
// difference's own sign; a tie takes the even code.
__device__ __forceinline__ uint32_t settle(uint32_t lo, float mid, float unit, float ax) {
  const float r = fmaf(-mid, unit, ax);
  return r > 0.f ? lo + 1u : r < 0.f ? lo : lo + (lo & 1u);
}

// Eight bf16 values (w) as e4m3 codes of x / scale, the first in the lowest
// byte of .x. inv is 1 / scale rounded.
__device__ __forceinline__ uint2 e4m3_codes8(const uint32_t (&w)[4], float scale, float inv) {
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float x[4] = {bf16lo_f32(w[2 * i]), bf16hi_f32(w[2 * i]), bf16lo_f32(w[2 * i + 1]), bf16hi_f32(w[2 * i + 1])};
    float y[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = x[j] * inv;
    uint32_t lo = f32x2_to_e4m3x2(y[0] * kQuotLo, y[1] * kQuotLo) | (f32x2_to_e4m3x2(y[2] * kQuotLo, y[3] * kQuotLo) << 16);
    const uint32_t hi =
        f32x2_to_e4m3x2(y[0] * kQuotHi, y[1] * kQuotHi) | (f32x2_to_e4m3x2(y[2] * kQuotHi, y[3] * kQuotHi) << 16);
    if (lo != hi) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = (lo >> (8 * j)) & 0x7Fu, b = (hi >> (8 * j)) & 0x7Fu;
        if (a != b) {
          const float mid = 0.5f * (e4m3_value(a) + e4m3_value(b));
          lo = (lo & ~(0x7Fu << (8 * j))) | (settle(a, mid, scale, fabsf(x[j])) << (8 * j));
        }
      }
    }
    c[i] = lo;
  }
  return make_uint2(c[0], c[1]);
}

// Largest magnitude of eight bf16 values as bits (order like the values; NaN
// and infinities are >= 0x7F80).
__device__ __forceinline__ uint32_t amax_bits8(const uint32_t (&w)[4]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
  return max(m & 0xFFFFu, m >> 16);
}
// The same over the finite values only.
__device__ __forceinline__ uint32_t finite_amax_bits8(const uint32_t (&w)[4]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFFu, b = (w[i] >> 16) & 0x7FFFu;
    m = max(m, a < 0x7F80u ? a : 0u);
    m = max(m, b < 0x7F80u ? b : 0u);
  }
  return m;
}

struct LowbitsWriteParams {
  const __nv_bfloat16* k;        // row of (token t, kv head h) at k + t * k_tok + h * k_head
  const __nv_bfloat16* v;
  long long k_tok, k_head, v_tok, v_head;
  uint8_t* k_cache;              // slot scales: the two caches; 4 bits: the records (k_cache)
  uint8_t* v_cache;
  float* k_scales;               // slot scales: [NB][Hk][bs]
  float* v_scales;
  const int64_t* slot_mapping;   // [T]
  int num_tokens;
  int num_kv_heads;
  int block_size;
  long long num_slots;           // num_blocks * block_size
  float min_scale;               // slot scales
  float k_scale, v_scale;        // 4 bits: the tensors' scales
  float k_inv6, v_inv6;          // 4 bits: 1 / (6 * scale), rounded
};

constexpr int kLowbitsThreads = 256;

// 16 bytes (eight values) of a row; kVec: row and strides on the 16-byte grid.
template <bool kVec>
__device__ __forceinline__ void load8(const __nv_bfloat16* src, uint32_t (&w)[4]) {
  if constexpr (kVec) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src));
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
  } else {
    const unsigned short* s = reinterpret_cast<const unsigned short*>(src);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = (uint32_t)__ldg(s + 2 * i) | ((uint32_t)__ldg(s + 2 * i + 1) << 16);
  }
}

// The slot of token t, or -1 when there is nothing to write.
__device__ __forceinline__ long long write_slot(const LowbitsWriteParams& p, int t, bool report) {
  const long long slot = __ldg(p.slot_mapping + t);
  if (slot < p.num_slots) return slot;
  if (report) atomicOr(&g_status, kStatusBadSlot);
  return -1;
}

// ------------------------------------------------- e4m3, a scale per slot

// The scale of a row whose 16 lanes (a half warp) hold eight values each.
__device__ __forceinline__ float slot_scale(const uint32_t (&w)[4], float min_scale) {
  uint32_t m = amax_bits8(w);
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
    m = finite_amax_bits8(w);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  return fmaxf(__fdiv_rn(__uint_as_float(m << 16), 448.f), min_scale);
}

// One warp per (token, kv head): lanes 0-15 the key row, 16-31 the value row.
template <bool kVec>
__global__ void __launch_bounds__(kLowbitsThreads) pda_write_slot_scales_kernel(const LowbitsWriteParams p) {
  const long long item = (long long)blockIdx.x * (kLowbitsThreads / 32) + (threadIdx.x >> 5);
  if (item >= (long long)p.num_tokens * p.num_kv_heads) return;   // whole warps
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const int t = (int)(item / p.num_kv_heads), h = (int)(item % p.num_kv_heads);
  const long long slot = write_slot(p, t, lane == 0);
  if (slot < 0) return;
  uint32_t w[4];
  load8<kVec>((is_v ? p.v + t * p.v_tok + h * p.v_head : p.k + t * p.k_tok + h * p.k_head) + 8 * l, w);
  const float scale = slot_scale(w, p.min_scale);
  const uint2 c = e4m3_codes8(w, scale, __frcp_rn(scale));
  const int bs = p.block_size;
  const long long row = (slot / bs) * p.num_kv_heads + h;
  const int o = (int)(slot % bs);
  if (l == 0) (is_v ? p.v_scales : p.k_scales)[row * bs + o] = scale;
  if (!is_v) {
    *reinterpret_cast<uint2*>(p.k_cache + row * (128 * bs) + ((l >> 1) * bs + o) * 16 + 8 * (l & 1)) = c;
  } else {
    uint8_t* dst = p.v_cache + row * (128 * bs) + (8 * l) * bs + o;
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i * bs] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// ------------------------------------------------------------------ e2m1

// This lane's eight values (two lanes a block of 16) as e2m1 nibbles of
// x / (s * g), and the block's e4m3 scale code s = E4M3(amax / (6 g)).
// A NaN in the block makes the scale NaN; an infinity saturates.
__device__ __forceinline__ uint32_t e2m1_codes8(uint32_t (&w)[4], float g, float inv6, uint32_t* scale_code) {
  uint32_t m = amax_bits8(w);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  bool nan = false;
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
    nan = m > 0x7F80u;   // of the block's largest bits
    m = finite_amax_bits8(w);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    // infinities as the largest finite value (they saturate all the same, and 0 * inf is no NaN)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((w[i] & 0x7FFFu) == 0x7F80u) w[i] = (w[i] & 0xFFFF8000u) | 0x7F7Fu;
      if (((w[i] >> 16) & 0x7FFFu) == 0x7F80u) w[i] = (w[i] & 0x8000FFFFu) | 0x7F7F0000u;
    }
  }
  const float a = __uint_as_float(m << 16);
  const float y0 = a * inv6;
  const uint32_t sc = f32x2_to_e4m3x2(y0 * kQuotLo, y0 * kQuotHi);
  uint32_t s = sc & 0x7Fu;
  const uint32_t s_hi = (sc >> 8) & 0x7Fu;
  if (s != s_hi) s = settle(s, 3.f * (e4m3_value(s) + e4m3_value(s_hi)), g, a);   // midpoint * 6
  *scale_code = nan ? 0x7Fu : s;
  const float sf = e4m3_value(s);
  const float inv = s == 0u ? 0.f : __frcp_rn(sf * g);
  float x[8], lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo_f32(w[i]);
    x[2 * i + 1] = bf16hi_f32(w[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = x[i] * inv;
    lo[i] = y * kQuotLo;
    hi[i] = y * kQuotHi;
  }
  uint32_t c = f32x8_to_e2m1(lo);
  const uint32_t d = c ^ f32x8_to_e2m1(hi);
  if (d != 0u && !nan) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((d >> (4 * i)) & 7u) {
        const uint32_t q = (c >> (4 * i)) & 7u;
        // 4 * midpoint of codes q and q + 1
        const float mid4 = (float)((0x00140E0A07050301ull >> (8 * q)) & 0xFFull);
        c = (c & ~(7u << (4 * i))) | (settle(q, 0.25f * mid4 * sf, g, fabsf(x[i])) << (4 * i));
      }
    }
  }
  return c;
}

// Items (a token's kv head) of kItems per warp, lanes 0-15 the key row, 16-31
// the value row: 16 bytes a lane in, 4 bytes of codes out.
template <bool kVec, int kItems>
__global__ void __launch_bounds__(kLowbitsThreads) pda_write_fp4_kernel(const LowbitsWriteParams p) {
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const long long items = (long long)p.num_tokens * p.num_kv_heads;
  const long long first = ((long long)blockIdx.x * (kLowbitsThreads / 32) + (threadIdx.x >> 5)) * kItems;
  uint32_t w[kItems][4];
  long long slot[kItems];
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    slot[i] = -1;
    if (first + i < items) {
      const int t = (int)((first + i) / p.num_kv_heads), h = (int)((first + i) % p.num_kv_heads);
      slot[i] = write_slot(p, t, lane == 0);
      load8<kVec>((is_v ? p.v + t * p.v_tok + h * p.v_head : p.k + t * p.k_tok + h * p.k_head) + 8 * l, w[i]);
    }
  }
  const int bs = p.block_size;
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (slot[i] < 0) continue;   // whole warps
    const int h = (int)((first + i) % p.num_kv_heads);
    uint32_t s;
    const uint32_t c = e2m1_codes8(w[i], is_v ? p.v_scale : p.k_scale, is_v ? p.v_inv6 : p.k_inv6, &s);
    const int o = (int)(slot[i] % bs);
    uint8_t* rec = p.k_cache + ((slot[i] / bs) * p.num_kv_heads + h) * (long long)(kFp4TokenBytes * bs);
    const int at = is_v ? 64 * bs + 64 * o + ((4 * l) ^ (16 * (o & 2))) : 64 * o + 4 * l;
    *reinterpret_cast<uint32_t*>(rec + at) = c;
    if ((l & 1) == 0) {
      const int b = l >> 1;
      rec[is_v ? 136 * bs + (o >> 4) * 128 + b * 16 + fp4_scale_place(o & 15) : 128 * bs + 8 * o + b] = (uint8_t)s;
    }
  }
}

// --------------------------------------------------------------- readers

struct GatherParams {
  __nv_bfloat16* k_out;          // [T][Hk][128]
  __nv_bfloat16* v_out;
  const uint8_t* k_cache;        // 4 bits: the records
  const uint8_t* v_cache;
  const float* k_scales;         // slot scales, or nullptr
  const float* v_scales;
  const int32_t* block_tables;   // [S][MB]
  const int32_t* token_starts;   // [S + 1]
  const int32_t* first;          // [S] or nullptr (0)
  int num_tokens;
  int num_seqs;
  int num_kv_heads;
  int block_size;
  int max_blocks;
  long long num_blocks;
  float k_scale, v_scale;
  int v_shuffled;
  int rows_per_cta;              // 4-bit reader
  int heads_per_cta;             // e4m3 reader
};

constexpr int kRowNone = -1;     // of no sequence: left as it is
constexpr int kRowBad = -2;      // outside its table row or the pool: zeros

// Block (or kRowNone / kRowBad) and slot in it of output row r.
__device__ __forceinline__ int2 gather_row(const GatherParams& p, int r) {
  int lo = 0, hi = p.num_seqs;   // first sequence that ends behind r
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.token_starts + mid + 1) > r) hi = mid;
    else lo = mid + 1;
  }
  if (lo == p.num_seqs) return make_int2(kRowNone, 0);
  const int start = __ldg(p.token_starts + lo);
  if (start > r) return make_int2(kRowNone, 0);
  const long long pos = (long long)r - start + (p.first ? (long long)__ldg(p.first + lo) : 0ll);
  if (pos >= 0 && pos < (long long)p.max_blocks * p.block_size) {
    const int b = __ldg(p.block_tables + (size_t)lo * p.max_blocks + (size_t)(pos / p.block_size));
    if (b >= 0 && b < p.num_blocks) return make_int2(b, (int)(pos % p.block_size));
  }
  atomicOr(&g_status, kStatusBadBlock);
  return make_int2(kRowBad, 0);
}

__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr int kGatherRows = 16;        // e4m3 reader: rows of a CTA
constexpr int kGatherMaxRows4 = 32;    // 4-bit reader: rows of a CTA at most

// 4 bits: one warp per (row, kv head), lanes 0-15 the key, 16-31 the value;
// 4 bytes of codes and one scale byte a lane in, 16 bytes out.
__global__ void __launch_bounds__(kLowbitsThreads) pda_gather_fp4_kernel(const GatherParams p) {
  __shared__ int2 rows[kGatherMaxRows4];
  const int r0 = blockIdx.x * p.rows_per_cta;
  const int n = min(p.rows_per_cta, p.num_tokens - r0);
  if (threadIdx.x < n) rows[threadIdx.x] = gather_row(p, r0 + threadIdx.x);
  __syncthreads();
  const int lane = threadIdx.x & 31, l = lane & 15, warp = threadIdx.x >> 5;
  const bool is_v = lane >= 16;
  const int bs = p.block_size, Hk = p.num_kv_heads;
  const float g = is_v ? p.v_scale : p.k_scale;
  __nv_bfloat16* out = is_v ? p.v_out : p.k_out;
  const int items = n * Hk;
  constexpr int kAhead = 4, kWarps = kLowbitsThreads / 32;
  for (int i0 = warp; i0 < items; i0 += kWarps * kAhead) {
    uint32_t c[kAhead], s[kAhead];
    int blk[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j * kWarps;
      blk[j] = kRowNone;
      c[j] = s[j] = 0u;
      if (i < items) {
        const int2 at = rows[i / Hk];
        blk[j] = at.x;
        if (at.x >= 0) {
          const int o = at.y;
          const uint8_t* rec = p.k_cache + ((long long)at.x * Hk + i % Hk) * (long long)(kFp4TokenBytes * bs);
          c[j] = __ldg(reinterpret_cast<const uint32_t*>(
              rec + (is_v ? 64 * bs + 64 * o + ((4 * l) ^ (16 * (o & 2))) : 64 * o + 4 * l)));
          s[j] = __ldg(rec + (is_v ? 136 * bs + (o >> 4) * 128 + (l >> 1) * 16 + fp4_scale_place(o & 15)
                                   : 128 * bs + 8 * o + (l >> 1)));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (blk[j] == kRowNone) continue;
      const int i = i0 + j * kWarps;
      const float f = e4m3_value(s[j]);
      uint32_t x[4], y[4];
      e2m1x8_to_f16x2(c[j], x);
#pragma unroll
      for (int u = 0; u < 4; ++u) y[u] = bf16x2_of((f16lo_f32(x[u]) * f) * g, (f16hi_f32(x[u]) * f) * g);
      const long long row = (long long)(r0 + i / Hk) * Hk + i % Hk;
      *reinterpret_cast<uint4*>(out + row * 128 + 8 * l) = make_uint4(y[0], y[1], y[2], y[3]);
    }
  }
}

// 16 e4m3 codes * scale -> 16 bf16 at dst.
__device__ __forceinline__ void store16(__nv_bfloat16* dst, const uint4& c, float scale) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = e4m3x2_lo_to_f16x2(w[i]), b = e4m3x2_hi_to_f16x2(w[i]);
    y[2 * i] = bf16x2_of(f16lo_f32(a) * scale, f16hi_f32(a) * scale);
    y[2 * i + 1] = bf16x2_of(f16lo_f32(b) * scale, f16hi_f32(b) * scale);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(y[0], y[1], y[2], y[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(y[4], y[5], y[6], y[7]);
}

// e4m3: 16 rows a CTA, thread 8j + c row j, dims 16c..16c+15; V, whose pages
// hold a dim's tokens side by side, passes through shared memory: thread d
// reads dim d's 16-byte group of tokens and hands out the rows' bytes.
__global__ void __launch_bounds__(128) pda_gather_kernel(const GatherParams p) {
  __shared__ int2 rows[kGatherRows];
  __shared__ __align__(16) uint8_t vt[kGatherRows][128];
  const int tid = threadIdx.x, j = tid >> 3, c = tid & 7;
  const int r0 = blockIdx.x * kGatherRows;
  if (tid < kGatherRows) rows[tid] = r0 + tid < p.num_tokens ? gather_row(p, r0 + tid) : make_int2(kRowNone, 0);
  __syncthreads();
  const int bs = p.block_size, Hk = p.num_kv_heads;
  const int h_end = min(Hk, (int)(blockIdx.y + 1) * p.heads_per_cta);
  const int2 at = rows[j];
  for (int h = blockIdx.y * p.heads_per_cta; h < h_end; ++h) {
    uint4 kq = make_uint4(0u, 0u, 0u, 0u);
    float ks = p.k_scale, vs = p.v_scale;
    if (at.x >= 0) {
      const long long row = (long long)at.x * Hk + h;
      kq = __ldg(reinterpret_cast<const uint4*>(p.k_cache + row * (128 * bs) + (c * bs + at.y) * 16));
      if (p.k_scales) {
        ks = __ldg(p.k_scales + row * bs + at.y);
        vs = __ldg(p.v_scales + row * bs + at.y);
      }
    } else {
      ks = vs = 0.f;
    }
    {
      uint4 grp = make_uint4(0u, 0u, 0u, 0u);
      int have_b = kRowNone, have_g = -1;
#pragma unroll
      for (int i = 0; i < kGatherRows; ++i) {
        const int2 a = rows[i];
        if (a.x >= 0 && (a.x != have_b || (a.y >> 4) != have_g)) {   // the same for all threads
          have_b = a.x;
          have_g = a.y >> 4;
          const uint8_t* page = p.v_cache + ((long long)a.x * Hk + h) * (128 * bs);
          grp = __ldg(reinterpret_cast<const uint4*>(page + (p.v_shuffled ? (have_g * 128 + tid) * 16
                                                                          : tid * bs + have_g * 16)));
        }
        const int o = a.y & 15;
        const uint32_t w = o < 8 ? (o < 4 ? grp.x : grp.y) : (o < 12 ? grp.z : grp.w);
        vt[i][tid] = a.x >= 0 ? (uint8_t)(w >> (8 * (o & 3))) : (uint8_t)0;
      }
    }
    __syncthreads();
    if (at.x != kRowNone) {
      const long long row = (long long)(r0 + j) * Hk + h;
      store16(p.k_out + row * 128 + 16 * c, kq, ks);
      store16(p.v_out + row * 128 + 16 * c, *reinterpret_cast<const uint4*>(&vt[j][16 * c]), vs);
    }
    __syncthreads();
  }
}

}  // namespace pda
