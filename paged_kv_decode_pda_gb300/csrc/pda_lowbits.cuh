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
// off by less than 2^-21, and next to a midpoint the sign of one fused
// multiply-add, which is exact, decides.
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

// 1 / x to 2^-23 of itself.
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t code) { return f16lo_f32(e4m3x2_lo_to_f16x2(code)); }

// The margin of a quotient made with a reciprocal: roundings of unit, shifted ends and
// product (2^-24 each) and the reciprocal's 2^-23.
constexpr float kQuotLo = 1.f - 4.76837158203125e-07f;   // 1 -+ 2^-21
constexpr float kQuotHi = 1.f + 4.76837158203125e-07f;

// Which of two neighbouring codes (magnitudes lo, lo + 1, whose midpoint is
// `mid` units) is nearest to |x|: |x| - mid * unit, rounded once, has the
// difference's own sign; a tie takes the even code.
__device__ __forceinline__ uint32_t settle(uint32_t lo, float mid, float unit, float ax) {
  const float r = fmaf(-mid, unit, ax);
  return r > 0.f ? lo + 1u : r < 0.f ? lo : lo + (lo & 1u);
}

// Two products, two sums, two fused products and sums at once (fp32, each rounded on its own).
__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  unsigned long long x, y, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(r));
  return d;
}
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  unsigned long long x, y, z, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(z) : "f"(c.x), "f"(c.y));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(r));
  return d;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  unsigned long long x, y, r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(a.x), "f"(a.y));
  asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(b.x), "f"(b.y));
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  float2 d;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(r));
  return d;
}

// The quotient x / scale for a rounding to e4m3: an approximate one, at most 2^-19
// of itself too large, cut to 16 significant bits (midpoints have 5, so that a
// quotient at or just past one is cut to it), and moved to the side on which the
// exact one lies, which the sign of one fused multiply-add tells. above: 1 / scale, a
// little too large.
__device__ __forceinline__ float e4m3_quotient(float x, float scale, float above) {
  const uint32_t c = __float_as_uint(x * above) & 0xFFFFFF00u;   // (NaN and infinities stay)
  const float r = copysignf(1.f, x) * fmaf(-__uint_as_float(c), scale, x);   // of the magnitudes
  return __uint_as_float(c + (r > 0.f ? 1u : 0u) - (r < 0.f ? 1u : 0u));     // (c == 0: r >= 0)
}

// A row's scale, and where it is amax / 448 rounded the factor that moves a cut
// quotient (e4m3_quotient) to its exact side: 448 x / amax is a midpoint or at least
// 2^-13 of itself from all (x and amax have 8 significant bits, a midpoint 5), so the
// quotients next to midpoints are those at them but for the scale's own rounding, and
// lie all on the side that its error tells. 0: another scale, each quotient by itself.
struct RowScale {
  float scale, step;
};

// Eight bf16 values (w) as e4m3 codes of x / scale, the first in the lowest byte of .x.
// (Exact and near ties are common, as a row's largest value is 448 scales: with a branch
// for them two of three warps took it. Each quotient by itself: 19.9 us for 8192 tokens
// of 8 heads, 16.6 by the row's factor.)
__device__ __forceinline__ uint2 e4m3_codes8(const uint32_t (&w)[4], RowScale s) {
  const float above = rcp_approx(s.scale) * (1.f + 9.5367431640625e-07f);   // 1 + 2^-20
  uint32_t c[4];
  if (__all_sync(0xffffffffu, s.step != 0.f)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 q = mul_f32x2(make_float2(bf16lo_f32(w[i]), bf16hi_f32(w[i])), make_float2(above, above));
      const float2 r = mul_f32x2(make_float2(__uint_as_float(__float_as_uint(q.x) & 0xFFFFFF00u),
                                             __uint_as_float(__float_as_uint(q.y) & 0xFFFFFF00u)),
                                 make_float2(s.step, s.step));
      c[i] = f32x2_to_e4m3x2(r.x, r.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = f32x2_to_e4m3x2(e4m3_quotient(bf16lo_f32(w[i]), s.scale, above), e4m3_quotient(bf16hi_f32(w[i]), s.scale, above));
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
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
__device__ __forceinline__ RowScale slot_scale(const uint32_t (&w)[4], float min_scale) {
  uint32_t m = amax_bits8(w);
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (__any_sync(0xffffffffu, m >= 0x7F80u)) {
    m = finite_amax_bits8(w);
#pragma unroll
    for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  // amax / 448 rounded to nearest: a product with the rounded reciprocal and one step
  // from its exact remainder (right for all 128 significands of a bf16)
  const float amax = __uint_as_float(m << 16), c = 1.f / 448.f, q = amax * c;
  const float s = fmaf(fmaf(-q, 448.f, amax), c, q), r = fmaf(s, 448.f, -amax);   // r: 448 times the scale's error
  RowScale row;
  row.scale = fmaxf(s, min_scale);
  row.step = r == 0.f ? 1.f : r > 0.f ? 1.f - 9.5367431640625e-07f : 1.f + 9.5367431640625e-07f;   // 1 -+ 2^-20
  if (s < min_scale) row.step = 0.f;
  return row;
}

// One warp per (token, kv head): lanes 0-15 the key row, 16-31 the value row. What
// bounds it are V's 1-byte stores, and latency: 256 tokens of 8 heads 4.7 us.
template <bool kVec>
__global__ void __launch_bounds__(kLowbitsThreads) pda_write_slot_scales_kernel(const LowbitsWriteParams p) {
  grid_dependency_wait();
  const long long item = (long long)blockIdx.x * (kLowbitsThreads / 32) + (threadIdx.x >> 5);
  if (item >= (long long)p.num_tokens * p.num_kv_heads) return;   // whole warps
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const int t = (int)(item / p.num_kv_heads), h = (int)(item % p.num_kv_heads);
  const long long slot = write_slot(p, t, lane == 0);
  if (slot < 0) return;
  uint32_t w[4];
  load8<kVec>((is_v ? p.v + t * p.v_tok + h * p.v_head : p.k + t * p.k_tok + h * p.k_head) + 8 * l, w);
  const RowScale scale = slot_scale(w, p.min_scale);
  const uint2 c = e4m3_codes8(w, scale);
  const int bs = p.block_size;
  const long long row = (slot / bs) * p.num_kv_heads + h;
  const int o = (int)(slot % bs);
  if (l == 0) (is_v ? p.v_scales : p.k_scales)[row * bs + o] = scale.scale;
  if (!is_v) {
    *reinterpret_cast<uint2*>(p.k_cache + row * (128 * bs) + ((l >> 1) * bs + o) * 16 + 8 * (l & 1)) = c;
  } else {
    uint8_t* dst = p.v_cache + row * (128 * bs) + (8 * l) * bs + o;
#pragma unroll
    for (int i = 0; i < 8; ++i) dst[i * bs] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
  }
}

// V pages hold a dim's tokens side by side, rows a token's dims: 16 slots x 4 dims
// of bytes turned in registers. in[i] = the 16 slots of dim i (four words), out[s] =
// the 4 dims of slot s; and back.
__device__ __forceinline__ void turn4(const uint32_t (&a)[4], uint32_t (&b)[4]) {
  const uint32_t t0 = __byte_perm(a[0], a[1], 0x5140), t1 = __byte_perm(a[2], a[3], 0x5140);
  const uint32_t t2 = __byte_perm(a[0], a[1], 0x7362), t3 = __byte_perm(a[2], a[3], 0x7362);
  b[0] = __byte_perm(t0, t1, 0x5410);
  b[1] = __byte_perm(t0, t1, 0x7632);
  b[2] = __byte_perm(t2, t3, 0x5410);
  b[3] = __byte_perm(t2, t3, 0x7632);
}

// A tile of 16 rows by the groups of 16 slots that hold them: group k is slots
// 16 * part .. + 15 of block `block`; `mask` says which of them are rows of the tile,
// `map` (4 bits a slot) which rows. Where two rows name one slot, rows make groups
// alone. One warp; returns the number of groups.
struct SlotGroup {
  int block, part;
  unsigned mask;
  unsigned long long map;
};
__device__ __forceinline__ int slot_groups(int block, int slot, bool live, int lane, SlotGroup* groups) {
  unsigned left = __ballot_sync(0xffffffffu, live && lane < 16);
  int n = 0;
  while (left != 0u) {
    const int lead = __ffs((int)left) - 1;
    const int b = __shfl_sync(0xffffffffu, block, lead), part = __shfl_sync(0xffffffffu, slot, lead) >> 4;
    const bool mine = (left >> lane & 1u) && block == b && (slot >> 4) == part;
    unsigned mask = __reduce_or_sync(0xffffffffu, mine ? 1u << (slot & 15) : 0u);
    bool take = mine;
    if (__popc((int)mask) != __popc((int)__ballot_sync(0xffffffffu, mine))) {   // a slot named twice: one row alone
      take = lane == lead;
      mask = 1u << (__shfl_sync(0xffffffffu, slot, lead) & 15);
    }
    const unsigned long long place = take ? (unsigned long long)lane << (4 * (slot & 15)) : 0ull;
    const unsigned lo = __reduce_or_sync(0xffffffffu, (unsigned)place);
    const unsigned hi = __reduce_or_sync(0xffffffffu, (unsigned)(place >> 32));
    if (lane == 0) {
      groups[n].block = b;
      groups[n].part = part;
      groups[n].mask = mask;
      groups[n].map = (unsigned long long)hi << 32 | lo;
    }
    ++n;
    left &= ~__ballot_sync(0xffffffffu, take);
  }
  return n;
}

// Where a tile's key row r has its 16-byte chunk c: read or written by rows and by
// columns without bank conflicts.
__device__ __forceinline__ int key_at(int r, int c) { return 16 * (c ^ (r & 7)); }

// Tiles of 16 tokens, a warp per kv head: the rows' codes pass through shared memory,
// K to go out 16 bytes (a chunk of a row) at a time, V by groups of 16 slots, turned
// in registers: 16-byte rows of whole groups, and what a group holds of the tile
// where it is cut or scattered. 8192 tokens of 8 heads in whole blocks 15.3 us, 3.3 TB/s:
// one partly filled wave of CTAs (6.7 an SM, a third of the warps) bounds it, neither
// bytes (24 % of DRAM) nor instructions (issue 54 %, ALU 52 %) alone. Prompts of odd
// lengths, whose tiles lie across two groups of slots, 31 us, scattered slots 73. (Keys
// and values to warps of their own, twice the CTAs: 16.8 against 16.4.)
constexpr int kWriteTileThreads = 128;
template <bool kVec>
__global__ void __launch_bounds__(kWriteTileThreads) pda_write_slot_scales_tile_kernel(const LowbitsWriteParams p) {
  grid_dependency_wait();
  __shared__ int2 rows[16];
  __shared__ SlotGroup groups[16];
  __shared__ int num_groups;
  __shared__ __align__(16) uint8_t tile[kWriteTileThreads / 32][2][16][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int half = lane >> 4, l = lane & 15;
  const int t0 = blockIdx.x * 16, bs = p.block_size, Hk = p.num_kv_heads;
  // 8 rows of a head, two at once: row 8 * (part & 1) + 2 i + half of the keys (parts 0
  // and 1) or values, 16 bytes a lane
  auto load = [&](uint32_t (&w)[4][4], int h, int part) {
    const __nv_bfloat16* src = part >= 2 ? p.v + h * p.v_head : p.k + h * p.k_head;
    const long long step = part >= 2 ? p.v_tok : p.k_tok;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + 8 * (part & 1) + 2 * i + half;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i][j] = 0u;
      if (t < p.num_tokens) load8<kVec>(src + t * step + 8 * l, w[i]);
    }
  };
  uint32_t w[4][4], next[4][4];
  const int h = blockIdx.y * (kWriteTileThreads / 32) + warp;   // the launch has a warp for every head
  if (h < Hk) load(w, h, 0);   // on their way while the slots are sorted out
  if (warp == 0) {
    const long long slot = lane < 16 && t0 + lane < p.num_tokens ? write_slot(p, t0 + lane, blockIdx.y == 0) : -1;
    const int2 at = slot < 0 ? make_int2(-1, 0) : make_int2((int)(slot / bs), (int)(slot % bs));
    if (lane < 16) rows[lane] = at;
    const int n = slot_groups(at.x, at.y, at.x >= 0, lane, groups);
    if (lane == 0) num_groups = n;
  }
  __syncthreads();
  if (num_groups == 0) return;
  const size_t page = (size_t)(128 * bs);
  uint8_t(*kt)[128] = tile[warp][0];
  uint8_t(*vt)[128] = tile[warp][1];
  if (h >= Hk) return;
  // (one part a turn of the loop: 33.2 us in place of 31.1 for prompts of odd lengths)
#pragma unroll 2
  for (int part = 0; part < 4; ++part) {
    const bool is_v = part >= 2;
    if (part < 3) load(next, h, part + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 8 * (part & 1) + 2 * i + half;
      const int2 at = rows[r];
      const RowScale scale = slot_scale(w[i], p.min_scale);
      *reinterpret_cast<uint2*>(is_v ? &vt[r][8 * l] : &kt[r][key_at(r, l >> 1) + 8 * (l & 1)]) = e4m3_codes8(w[i], scale);
      if (l == 0 && at.x >= 0) (is_v ? p.v_scales : p.k_scales)[((size_t)at.x * Hk + h) * bs + at.y] = scale.scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[i][j] = next[i][j];
    }
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // consecutive lanes: consecutive rows of one chunk
    const int r = lane & 15, c = half + 2 * i;
    const int2 at = rows[r];
    if (at.x >= 0)
      *reinterpret_cast<uint4*>(p.k_cache + ((size_t)at.x * Hk + h) * page + (c * bs + at.y) * 16) =
          *reinterpret_cast<const uint4*>(&kt[r][key_at(r, c)]);
  }
  for (int k = 0; k < num_groups; ++k) {
    const SlotGroup gr = groups[k];
    uint8_t* dst = p.v_cache + ((size_t)gr.block * Hk + h) * page + 4 * lane * bs + gr.part * 16;
    if ((gr.mask & (gr.mask - 1u)) == 0u) {   // a token alone
      const int s = __ffs((int)gr.mask) - 1;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(&vt[(int)(gr.map >> (4 * s)) & 15][4 * lane]);
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[i * bs + s] = (uint8_t)(c >> (8 * i));
      continue;
    }
    uint32_t v[4][4];   // [dim][four slots]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t in[4], out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = 4 * q + i;
        in[i] = gr.mask >> s & 1u ? *reinterpret_cast<const uint32_t*>(&vt[(int)(gr.map >> (4 * s)) & 15][4 * lane]) : 0u;
      }
      turn4(in, out);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i][q] = out[i];
    }
    if (gr.mask == 0xFFFFu) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4*>(dst + i * bs) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const unsigned m = gr.mask >> (4 * q) & 15u;
        if (m == 0u) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint8_t* d = dst + i * bs + 4 * q;
          if (m == 15u) {
            *reinterpret_cast<uint32_t*>(d) = v[i][q];
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (m >> j & 1u) d[j] = (uint8_t)(v[i][q] >> (8 * j));
          }
        }
      }
    }
  }
}

// ------------------------------------------------------------------ e2m1

// Eight e2m1 codes c, of which those in d are uncertain between c and c + 1: the
// exact sign decides. (Rare unless the tensor's scale is a power of two, and so a
// call.)
__device__ __noinline__ uint32_t settle_e2m1x8(uint32_t c, uint32_t d, uint4 w, float sf, float g) {
#pragma unroll 1
  while (d != 0u) {
    const int i = (__ffs((int)d) - 1) >> 2;
    d &= ~(15u << (4 * i));
    const uint32_t q = (c >> (4 * i)) & 7u;
    const uint32_t x = (i < 4 ? (i < 2 ? w.x : w.y) : (i < 6 ? w.z : w.w)) >> (16 * (i & 1)) & 0x7FFFu;
    const float mid4 = (float)((0x00140E0A07050301ull >> (8 * q)) & 0xFFull);   // 4 * midpoint of q and q + 1
    c = (c & ~(7u << (4 * i))) | (settle(q, 0.25f * mid4 * sf, g, __uint_as_float(x << 16)) << (4 * i));
  }
  return c;
}

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
  const float inv = s == 0u ? 0.f : rcp_approx(sf * g);
  const float2 inv_lo = make_float2(inv * kQuotLo, inv * kQuotLo), inv_hi = make_float2(inv * kQuotHi, inv * kQuotHi);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = make_float2(bf16lo_f32(w[i]), bf16hi_f32(w[i]));
    const float2 a2 = mul_f32x2(x, inv_lo), b2 = mul_f32x2(x, inv_hi);
    lo[2 * i] = a2.x, lo[2 * i + 1] = a2.y;
    hi[2 * i] = b2.x, hi[2 * i + 1] = b2.y;
  }
  const uint32_t c = f32x8_to_e2m1(lo), d = f32x8_to_e2m1(hi);
  return c == d || nan ? c : settle_e2m1x8(c, c ^ d, make_uint4(w[0], w[1], w[2], w[3]), sf, g);
}

// One warp per token and kItems of its kv heads (blockIdx.y counts them), lanes 0-15
// the key rows, 16-31 the value rows: 16 bytes a lane in, 4 bytes of codes out. Bound by
// instructions (issue 74 %): 16384 tokens of 8 heads 19 us, 4.5 TB/s.
template <bool kVec, int kItems>
__global__ void __launch_bounds__(kLowbitsThreads) pda_write_fp4_kernel(const LowbitsWriteParams p) {
  grid_dependency_wait();
  const int lane = threadIdx.x & 31, l = lane & 15;
  const bool is_v = lane >= 16;
  const long long t = (long long)blockIdx.x * (kLowbitsThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.num_tokens) return;   // whole warps
  const int h0 = blockIdx.y * kItems, n = min(kItems, p.num_kv_heads - h0);
  const long long slot = write_slot(p, (int)t, lane == 0 && h0 == 0);
  const __nv_bfloat16* src = is_v ? p.v + t * p.v_tok : p.k + t * p.k_tok;
  const long long head = is_v ? p.v_head : p.k_head;
  uint32_t w[kItems][4];
#pragma unroll
  for (int i = 0; i < kItems; ++i)
    if (i < n) load8<kVec>(src + (h0 + i) * head + 8 * l, w[i]);
  if (slot < 0) return;
  const int bs = p.block_size, o = (int)(slot % bs);
  const size_t rec = (size_t)(kFp4TokenBytes * bs);
  uint8_t* base = p.k_cache + ((size_t)(slot / bs) * p.num_kv_heads + h0) * rec;
  const int code = is_v ? 64 * bs + 64 * o + ((4 * l) ^ (16 * (o & 2))) : 64 * o + 4 * l;
  const int scale = is_v ? 136 * bs + (o >> 4) * 128 + (l >> 1) * 16 + fp4_scale_place(o & 15) : 128 * bs + 8 * o + (l >> 1);
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
    if (i >= n) break;
    uint32_t s;
    const uint32_t c = e2m1_codes8(w[i], is_v ? p.v_scale : p.k_scale, is_v ? p.v_inv6 : p.k_inv6, &s);
    *reinterpret_cast<uint32_t*>(base + i * rec + code) = c;
    if ((l & 1) == 0) base[i * rec + scale] = (uint8_t)s;
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
  int v_wide;                    // a group's V rows lie side by side, on the 32-byte grid
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

// 4 bits: a warp per (row, kv head), lanes 0-15 the key, 16-31 the value; 4 bytes
// of codes and one scale byte a lane in, 16 bytes out. The warps of a CTA take rows
// each, or share a row's heads where a CTA has fewer rows than warps. Bound by bytes in
// long calls (64 contexts of 1 to 4000: 103.8 us, 6.1 TB/s); by the way from a row to
// its page in short ones (16384 tokens: 17.6 us, 4.9 TB/s; each warp looking its rows up
// without the CTA's barrier: 62 registers, or spills, and 107 and 18.6 us).
__global__ void __launch_bounds__(kLowbitsThreads) pda_gather_fp4_kernel(const GatherParams p) {
  grid_dependency_wait();
  __shared__ int2 rows[kGatherMaxRows4];
  const int r0 = blockIdx.x * p.rows_per_cta;
  const int n = min(p.rows_per_cta, p.num_tokens - r0);
  if (threadIdx.x < n) rows[threadIdx.x] = gather_row(p, r0 + threadIdx.x);
  __syncthreads();
  constexpr int kWarps = kLowbitsThreads / 32, kAhead = 8;   // (64 contexts of 1 to 4000: 104 us, 118 with 4)
  const int lane = threadIdx.x & 31, l = lane & 15, warp = threadIdx.x >> 5;
  const bool is_v = lane >= 16;
  const int bs = p.block_size, Hk = p.num_kv_heads;
  const float g = is_v ? p.v_scale : p.k_scale;
  // rows_per_cta is a power of two
  const int share = p.rows_per_cta < kWarps ? kWarps / p.rows_per_cta : 1;   // warps of a row
  const size_t rec = (size_t)(kFp4TokenBytes * bs);
  for (int r = warp / share; r < n; r += kWarps / share) {
    const int2 at = rows[r];
    if (at.x == kRowNone) continue;
    const int o = at.y, h_first = warp % share;
    const bool ok = at.x >= 0;   // else zeros
    const uint8_t* base = p.k_cache + (ok ? (size_t)at.x : 0) * Hk * rec;
    const uint8_t* code = base + (is_v ? 64 * bs + 64 * o + ((4 * l) ^ (16 * (o & 2))) : 64 * o + 4 * l);
    const uint8_t* scale = base + (is_v ? 136 * bs + (o >> 4) * 128 + (l >> 1) * 16 + fp4_scale_place(o & 15)
                                        : 128 * bs + 8 * o + (l >> 1));
    __nv_bfloat16* out = (is_v ? p.v_out : p.k_out) + ((size_t)(r0 + r) * Hk) * 128 + 8 * l;
    for (int h0 = h_first; h0 < Hk; h0 += kAhead * share) {
      uint32_t c[kAhead], s[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = h0 + j * share;
        c[j] = s[j] = 0u;
        if (ok && h < Hk) {
          c[j] = __ldg(reinterpret_cast<const uint32_t*>(code + h * rec));
          s[j] = __ldg(scale + h * rec);
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int h = h0 + j * share;
        if (h >= Hk) break;
        const uint32_t s2 = e4m3x2_lo_to_f16x2(s[j] | (s[j] << 8));
        uint32_t x[4], y[4];
        e2m1x8_to_f16x2(c[j], x);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t v = mul_f16x2(x[u], s2);   // exact
          y[u] = bf16x2_of(f16lo_f32(v) * g, f16hi_f32(v) * g);
        }
        *reinterpret_cast<uint4*>(out + (size_t)h * 128) = make_uint4(y[0], y[1], y[2], y[3]);
      }
    }
  }
}

// e4m3: 16 rows a CTA, a warp per kv head. Both tensors pass through shared memory
// as [row][128] bytes: K 16 bytes (a chunk of a row) at a time, V by groups of 16
// slots turned in registers; from there a half warp writes a row. What bounds it
// beside the bytes are L1's passes over scattered 16-byte loads: 32 contexts of 1 to
// 4000 tokens, 16-token blocks, 71.6 us with V's 16 bytes and K's rows a lane eighth
// at a time, 66.0 (5.9 TB/s) with V's 32 bytes at a time and K's rows side by side
// (64 registers and 24 bytes spilled: 69).
constexpr int kGatherThreads = 128;
// 32 bytes on their grid in one load.
__device__ __forceinline__ void ldg_32(const uint8_t* src, uint4& a, uint4& b) {
  asm("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
      : "l"(src));
}
__global__ void __launch_bounds__(kGatherThreads) pda_gather_kernel(const GatherParams p) {
  grid_dependency_wait();
  __shared__ int2 rows[kGatherRows];
  __shared__ SlotGroup groups[kGatherRows];
  __shared__ int num_groups;
  __shared__ __align__(16) uint8_t tile[kGatherThreads / 32][2][kGatherRows][128];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r0 = blockIdx.x * kGatherRows;
  if (warp == 0) {
    const int2 at = lane < kGatherRows && r0 + lane < p.num_tokens ? gather_row(p, r0 + lane) : make_int2(kRowNone, 0);
    if (lane < kGatherRows) rows[lane] = at;
    const int n = slot_groups(at.x, at.y, at.x >= 0, lane, groups);
    if (lane == 0) num_groups = n;
  }
  __syncthreads();
  const int bs = p.block_size, Hk = p.num_kv_heads;
  const int half = lane >> 4, l = lane & 15;
  const int h_end = min(Hk, (int)(blockIdx.y + 1) * p.heads_per_cta);
  const size_t page = (size_t)(128 * bs);
  const int2 own = rows[l];   // this lane's row, for its scale
  for (int h = blockIdx.y * p.heads_per_cta + warp; h < h_end; h += kGatherThreads / 32) {
    uint8_t(*kt)[128] = tile[warp][0];
    uint8_t(*vt)[128] = tile[warp][1];
    float scale = half ? p.v_scale : p.k_scale;   // of row l, key (lanes 0-15) or value
    if (p.k_scales && own.x >= 0) scale = __ldg((half ? p.v_scales : p.k_scales) + ((size_t)own.x * Hk + h) * bs + own.y);
    uint4 kq[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // consecutive lanes: consecutive rows of one chunk
      kq[i] = make_uint4(0u, 0u, 0u, 0u);
      if (own.x >= 0)
        kq[i] = __ldg(reinterpret_cast<const uint4*>(p.k_cache + ((size_t)own.x * Hk + h) * page + ((half + 2 * i) * bs + own.y) * 16));
    }
    for (int k = 0; k < num_groups; ++k) {   // (the next group's loads ahead: 104 registers, and 84 us for 72)
      const SlotGroup gr = groups[k];
      const uint8_t* src = p.v_cache + ((size_t)gr.block * Hk + h) * page;
      src += p.v_shuffled ? (gr.part * 128 + 4 * lane) * 16 : 4 * lane * bs + gr.part * 16;
      const int step = p.v_shuffled ? 16 : bs;
      uint4 v[4];
      if (p.v_wide) {   // the four rows side by side
        ldg_32(src, v[0], v[1]);
        ldg_32(src + 32, v[2], v[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(src + i * step));
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t in[4] = {q == 0 ? v[0].x : q == 1 ? v[0].y : q == 2 ? v[0].z : v[0].w,
                                q == 0 ? v[1].x : q == 1 ? v[1].y : q == 2 ? v[1].z : v[1].w,
                                q == 0 ? v[2].x : q == 1 ? v[2].y : q == 2 ? v[2].z : v[2].w,
                                q == 0 ? v[3].x : q == 1 ? v[3].y : q == 2 ? v[3].z : v[3].w};
        uint32_t out[4];
        turn4(in, out);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int s = 4 * q + i;
          if (gr.mask >> s & 1u) *reinterpret_cast<uint32_t*>(&vt[(int)(gr.map >> (4 * s)) & 15][4 * lane]) = out[i];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(&kt[l][key_at(l, half + 2 * i)]) = kq[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kGatherRows; ++i) {
      // two rows at once: keys of rows 0 .. 15, then values
      const int r = (2 * i + half) & 15;
      const bool is_v = i >= kGatherRows / 2;
      const int st = rows[r].x;
      const float f = __shfl_sync(0xffffffffu, scale, r + (is_v ? 16 : 0));
      const uint2 c = *reinterpret_cast<const uint2*>(is_v ? &vt[r][8 * l] : &kt[r][key_at(r, l >> 1) + 8 * (l & 1)]);
      if (st == kRowNone) continue;
      uint32_t y[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t w = u < 2 ? c.x : c.y;
        const uint32_t x = u & 1 ? e4m3x2_hi_to_f16x2(w) : e4m3x2_lo_to_f16x2(w);
        y[u] = bf16x2_of(f16lo_f32(x) * f, f16hi_f32(x) * f);
      }
      uint4 o = make_uint4(y[0], y[1], y[2], y[3]);
      if (st < 0) o = make_uint4(0u, 0u, 0u, 0u);
      *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + ((size_t)(r0 + r) * Hk + h) * 128 + 8 * l) = o;
    }
    __syncwarp();   // the tile is read
  }
}

}  // namespace pda
