// Decode attention over the 4-bit cache (records: pda_lowbits.cuh).
//
//   out = sum_t e^(z_t) v_t / (sum_t e^(z_t) + e^sink),  z_t = scale q . k_t
//
// over the tokens max(0, L - window) .. L - 1 of a sequence. What it cannot do
// without: 144 bytes per (token, kv head) against 256 for e4m3, so the same
// bandwidth brings 1.8 times the tokens, and converting and multiplying them is
// what comes close to bounding the kernel.
//
// Work. A unit is a (sequence, group of kv heads): four heads where the pages have
// at most 64 tokens, whose records lie side by side, so that one copy brings a
// page of all four and each consumer warp works on a head of its own, alone; two
// or one where pages are larger or the heads do not divide, a head's tokens then
// shared by two or four warps, whose rows are merged in shared memory (256 x 4096 tokens
// of 8/2 heads 62 us for a floor of 45, of 8/1 heads 40 for 22). A unit's tokens go in
// chunks of whole pages, 256 / heads tokens at most. All units' chunks, one after the
// other, are cut into runs wherever the cuts fall, one per resident CTA, so that every
// batch (a few long sequences, many ragged ones) loads all SMs alike. The pieces (O, m,
// l) of a unit that a cut divides go to the workspace, and a second kernel joins them.
// (Smaller runs for the last quarter, taken from a queue as CTAs come free: all CTAs
// end within 4 % of each other, not 20 %, and the pieces this adds cost as much, 219
// against 222 us at 256 x 4096 tokens of 32/8 heads, 120 against 119 at 256 x 1 to
// 4000 of 40/8, 83 against 67 at 2 x 131072 of 64/8, at two tiles a warp.)
// (Joined in this kernel, by the warp that brings a unit's last piece: 256 x 4096
// tokens of 32/8 heads took 242 us against 212, as a warp that waits for counts and
// other warps' rows holds up its CTA's ring.)
//
// A CTA. One producer warp copies chunks into a ring; four consumer warps take four
// 16-token tiles of each (what a chunk costs beside its tiles, half a microsecond a
// CTA, is spread over them: with two a warp 222 us against 200 at 256 x 4096 tokens
// of 32/8 heads), or two in batches too short for even runs of so large chunks:
//   S^T = K (16 tokens x 128) Q^T (128 x 8 heads), O^T += V^T (128 x 16) P^T
// on warp MMAs whose A fragments are made in registers: e2m1 -> f16 by the
// conversion instruction, times the block's scale, exact (6 significant bits).
// These MMAs are the bound: 8 of them take 18 cycles of an SM, and little else issues
// meanwhile, so that a tile (16 MMAs, 64 conversions, 64 products, 60 others) takes 84
// with 12 or with 16 warps, where HBM would bring one every 91; 256 x 4096 tokens take
// 192 us without any copies and 201 with them.
// Q enters as in pda_decode (shifted by a power of two into f16), P as one f16, held
// 2^7 times as large (up to 2^15, with the lag below): off by at most 2^-11 of itself
// down to 2^-21 of the running maximum, by 2^-32 of that below (held as it is, by 2^-25:
// the weights behind one far token, 2^-24 of it each, were off by up to half of
// themselves). The normaliser sums P unrounded in fp32, in the same units, so that they
// cancel but for the sinks.
//
// The contraction's order is free, so each lane takes what lies side by side:
// of a K row 16 bytes (32 dims), of four V rows one 8-byte block of 16 dims each,
// whose single scale then serves all its dims. MMA row r holds token
// fp4_row_token(r) and V's k slots the same tokens, chosen so that both kinds of
// loads spread over all banks.
//
// The running maximum is let fall up to 8 (log2) behind: P stays below 2^8, 2^15 as it
// is held, inside f16, and nearly every tile passes with one vote in place of a maximum
// over the lanes and a rescale. The reference is an unscaled logit, taken off the
// others before the scale, so that the weight of the reference itself is exactly 1
// at any size (a scaled one leaves the rounding of a product as a power of two:
// infinite in f16 from 2^27 on).
#pragma once

#include "pda_kernels.cuh"
#include "pda_lowbits.cuh"

namespace pda {

constexpr int kF4Warps = 4;                                    // consumer warps
constexpr int kF4Threads = kF4Warps * 32 + 32;
constexpr int kF4CtasPerSm = 3;
constexpr int kF4Stages = 2;
constexpr int kF4Tiles = 4;                                    // 16-token tiles of a chunk per consumer warp at most
constexpr int kF4ChunkTokens = 16 * kF4Tiles * kF4Warps;
constexpr uint32_t kF4StageBytes = kF4ChunkTokens * kFp4TokenBytes;
constexpr int kF4MergeStride = kHeadDim + 4;
static_assert(kF4Warps * kMaxGqa * (kF4MergeStride + 2) * 4 <= kF4StageBytes, "merge rows fit a stage");
constexpr float kF4Lag = 8.f;                                  // the running reference's lag behind the maximum, log2
constexpr float kF4Shift = 7.f;                                // P and its sums are held in units of 2^-7
static_assert(kF4Lag + kF4Shift < 16.f, "f16 holds P");
constexpr int kF4MaxCtas = 512;
constexpr int kF4RowFloats = kMaxGqa * (kHeadDim + 2);         // a piece: O rows, then (m, l) pairs

// Workspace: the join's CTAs that are done and the numbers of cut units, zero
// between calls; the cut units {sequence, first kv head, first run, pieces} in no
// order, those of few pieces from the front, those of many from the back; then the
// pieces, two per run and warp.
constexpr int kF4FewPieces = 8;
struct Fp4Head {
  unsigned joined, cuts[2];
  unsigned pad[61];
  int4 cut[kF4MaxCtas];
};

// The runs: C chunks over G CTAs, the first `more` of which take one more.
struct Fp4Runs {
  unsigned each, more;

  __device__ __forceinline__ void plan(unsigned C, unsigned G) {
    each = C / G;
    more = C - each * G;
  }
  __device__ __forceinline__ unsigned first(unsigned r) const { return r * each + min(r, more); }
  __device__ __forceinline__ unsigned owner(unsigned x) const {   // run of chunk x
    const unsigned wide = more * (each + 1u);
    return x < wide ? x / (each + 1u) : more + (x - wide) / each;
  }
};

struct Fp4DecodeParams {
  void* out;
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const float* sinks;
  Fp4Head* head;
  float* pieces;
  int num_seqs;
  int num_heads;
  int num_kv_heads;
  int gqa;
  int block_size;
  int max_blocks;
  int num_blocks;
  int window;
  int pages_per_chunk;
  int group;                // kv heads of a unit: 4, 2 or 1
  int tiles;                // of a chunk per consumer warp: 4 or 2
  unsigned long long bs_inverse, chunk_inverse;   // ceil(2^37 / d) of block_size and pages_per_chunk
  float logit_scale_log2;   // |scale * k_scale| * log2(e)
  int negate;
  float v_scale;
  int out_fp8;
  float out_scale;
};

// Pages [first, first + n) and tokens [lo, hi) of a sequence.
struct Fp4Span {
  int first, n, lo, hi;
};

// A chunk's note, written by the producer with its copies.
struct __align__(16) Fp4Chunk {
  int flags;                // kHdrFirst, kHdrLast: of this CTA's part of the unit; kF4Full
  int t0;                   // the chunk's first token
  int lo, hi;               // tokens that count (hi: also not past the chunk's pages)
  int s, kvh;               // sequence, first kv head of the unit
  int run0, piece, pieces;  // run of the unit's first piece; this one of how many
  int pad[3];
};
constexpr int kF4Full = 8;  // a whole chunk, all of whose tokens count

// Ring, notes, barriers (full, empty, consumers), scan sums and flag,
// and the chunks before each thread's sequences.
constexpr uint32_t kF4Smem = 128 + kF4Stages * (kF4StageBytes + (uint32_t)sizeof(Fp4Chunk)) + (2 * kF4Stages + 1) * 8 + 64 +
                             kF4Threads * 4;

__device__ __forceinline__ int fp4_row_token(int r) {
  const int t = (r >> 1) & 3;
  return ((r & 1) ? (t ^ 1) + 4 : t) + (r & 8);
}

// x / d with ceil(2^37 / d), for tokens (x < 2^30 + 128, d = 16 .. 128) and pages
// (x <= 2^26, d = 1 .. 16): before it is cut the result is off by less than x / 2^37
// (nothing where d is a power of two), less than 1 / d, and x / d lies at least 1 / d
// below the next integer; the product stays below 2^64.
__device__ __forceinline__ int fp4_divide(int x, unsigned long long inverse) {
  return (int)(((unsigned long long)(unsigned)x * inverse) >> 37);
}
__device__ __forceinline__ Fp4Span fp4_span(const Fp4DecodeParams& p, int s) {
  Fp4Span a;
  a.hi = max(0, min(__ldg(p.seq_lens + s), p.max_blocks * p.block_size));
  a.lo = p.window > 0 ? max(0, a.hi - p.window) : 0;
  a.first = a.lo > 0 ? fp4_divide(a.lo, p.bs_inverse) : 0;
  a.n = fp4_divide(a.hi + p.block_size - 1, p.bs_inverse) - a.first;
  return a;
}
// An empty sequence has one chunk too: somebody writes its zeros.
__device__ __forceinline__ int fp4_chunks(const Fp4DecodeParams& p, int pages) {
  return pages > 0 ? fp4_divide(pages + p.pages_per_chunk - 1, p.chunk_inverse) : 1;
}

// A consumer warp's share of a unit.
struct Fp4Worker {
  int gid, tig;
  uint32_t k_off, v_off, ks_off, vs_off;
  uint32_t qf[kChunks][2];
  float2 lsc;               // log2 units of an unscaled logit, >= 0
  float2 nr;                // minus the running reference: an unscaled logit, at most the lag below the maximum
  float l0, l1;             // sums, in units of 2^-kF4Shift, as o
  float t0, t1;             // unscaled logits past which the reference moves
  float o[kChunks][4];      // dims 16 gid + 2 mt (0, 1) and 16 gid + 2 mt + 1 (2, 3); heads 2 tig, 2 tig + 1

  __device__ __forceinline__ void setup(int lane) {
    gid = lane >> 2;
    tig = lane & 3;
    const int tok = fp4_row_token(gid);
    k_off = (uint32_t)(tok * 64 + 16 * tig);
    ks_off = (uint32_t)(tok * 8 + 2 * tig);
    v_off = (uint32_t)(tig * 64) + ((uint32_t)(8 * gid) ^ (uint32_t)((tig & 2) << 4));
    vs_off = (uint32_t)(gid * 16 + 4 * tig);
  }
  // The state of a unit, when one has ended: nothing of it is held in registers
  // through what ends it.
  __device__ __forceinline__ void reset() {
    nr.x = nr.y = INFINITY;
    t0 = t1 = -INFINITY;
    l0 = l1 = lsc.x = lsc.y = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) qf[i][0] = qf[i][1] = 0u;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // The reference in log2 units.
  __device__ __forceinline__ float m0() const { return nr.x == INFINITY ? -INFINITY : -nr.x * lsc.x; }
  __device__ __forceinline__ float m1() const { return nr.y == INFINITY ? -INFINITY : -nr.y * lsc.y; }

  // Q^T fragments of the row at qrow: k step c's slots (2 tig, 2 tig + 1),
  // (2 tig + 8, 2 tig + 9) are dims 32 tig + 4c .. + 3. Each row is shifted by a
  // power of two that puts its largest |q| into [2^14, 2^15).
  __device__ __forceinline__ void load_q(const __nv_bfloat16* qrow, bool live, float unit, bool negate) {
    uint2 v[kChunks];
    uint32_t mx = 0u;
#pragma unroll
    for (int c = 0; c < kChunks; c += 2) {
      const uint4 x = live ? __ldg(reinterpret_cast<const uint4*>(qrow + 32 * tig + 4 * c)) : make_uint4(0u, 0u, 0u, 0u);
      v[c] = make_uint2(x.x, x.y);
      v[c + 1] = make_uint2(x.z, x.w);
      mx = __vmaxu2(__vmaxu2(mx, x.x & 0x7FFF7FFFu), x.y & 0x7FFF7FFFu);
      mx = __vmaxu2(__vmaxu2(mx, x.z & 0x7FFF7FFFu), x.w & 0x7FFF7FFFu);
    }
    mx = max(mx & 0xFFFFu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = mx == 0u ? 0 : min(max((int)(mx >> 7) - 127 - 14, -100), 113);
    const float down = negate ? -exp2_int(-e) : exp2_int(-e);
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      qf[c][0] = pack_f16x2(bf16lo_f32(v[c].x) * down, bf16hi_f32(v[c].x) * down);
      qf[c][1] = pack_f16x2(bf16lo_f32(v[c].y) * down, bf16hi_f32(v[c].y) * down);
    }
    lsc.x = unit * exp2_int(__shfl_sync(0xffffffffu, e, 8 * tig));
    lsc.y = unit * exp2_int(__shfl_sync(0xffffffffu, e, 8 * tig + 4));
  }

  // Unscaled logits of a tile: z[0], z[1] token row gid, z[2], z[3] row gid + 8.
  __device__ __forceinline__ void scores(uint32_t k, uint32_t ks, float (&z)[4]) const {
    uint32_t wa[4], wb[4];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(wa[0]), "=r"(wa[1]), "=r"(wa[2]), "=r"(wa[3]) : "r"(k + k_off));
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(wb[0]), "=r"(wb[1]), "=r"(wb[2]), "=r"(wb[3]) : "r"(k + k_off + 512u));
    unsigned short ua, ub;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(ua) : "r"(ks + ks_off));
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(ub) : "r"(ks + ks_off + 64u));
    const uint32_t sa = e4m3x2_lo_to_f16x2(ua), sb = e4m3x2_lo_to_f16x2(ub);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // words 0, 1 lie in the row's block 2 tig, words 2, 3 in 2 tig + 1
      const uint32_t fa = __byte_perm(sa, 0, j < 2 ? 0x1010 : 0x3232), fb = __byte_perm(sb, 0, j < 2 ? 0x1010 : 0x3232);
      uint32_t a[4], b[4];
      e2m1x8_to_f16x2(wa[j], a);
      e2m1x8_to_f16x2(wb[j], b);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = mul_f16x2(a[i], fa);
        b[i] = mul_f16x2(b[i], fb);
      }
      if (j == 0) mma_f16_first(z, a[0], b[0], a[1], b[1], qf[0][0], qf[0][1]);
      else mma_f16(z, a[0], b[0], a[1], b[1], qf[2 * j][0], qf[2 * j][1]);
      mma_f16(z, a[2], b[2], a[3], b[3], qf[2 * j + 1][0], qf[2 * j + 1][1]);
    }
  }

  // O^T += V^T P^T of a tile; p in scores' order. [lo, hi): the tile's tokens
  // that count (the others' scales may hold anything, also NaN).
  template <bool kMasked>
  __device__ __forceinline__ void values(uint32_t v, uint32_t vs, const float (&p)[4], int lo, int hi) {
    const uint32_t pb0 = movmatrix_trans(pack_f16x2(p[0], p[1]));
    const uint32_t pb1 = movmatrix_trans(pack_f16x2(p[2], p[3]));
    const uint2 w0 = ld_shared_v2(v + v_off);                                             // token tig
    const uint2 w1 = ld_shared_v2(v + v_off + ((tig & 1) ? 192u : 320u));                 // (tig ^ 1) + 4
    const uint2 w2 = ld_shared_v2(v + v_off + 512u);                                      // tig + 8
    const uint2 w3 = ld_shared_v2(v + v_off + 512u + ((tig & 1) ? 192u : 320u));          // (tig ^ 1) + 12
    uint32_t s;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(s) : "r"(vs + vs_off));
    if (kMasked && (lo > 0 || hi < 16)) {
      const int t1 = (tig ^ 1) + 4;
      if (tig < lo || tig >= hi) s &= 0xFFFFFF00u;
      if (t1 < lo || t1 >= hi) s &= 0xFFFF00FFu;
      if (tig + 8 < lo || tig + 8 >= hi) s &= 0xFF00FFFFu;
      if (t1 + 8 < lo || t1 + 8 >= hi) s &= 0x00FFFFFFu;
    }
    const uint32_t f01 = e4m3x2_lo_to_f16x2(s), f23 = e4m3x2_hi_to_f16x2(s);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t x0 = j ? w0.y : w0.x, x1 = j ? w1.y : w1.x, x2 = j ? w2.y : w2.x, x3 = j ? w3.y : w3.x;
      // bytes (token, token') of the even dims, of the odd dims
      uint32_t e01[4], o01[4], e23[4], o23[4];
      e2m1x8_to_f16x2((x0 & 0x0F0F0F0Fu) | ((x1 << 4) & 0xF0F0F0F0u), e01);
      e2m1x8_to_f16x2(((x0 >> 4) & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u), o01);
      e2m1x8_to_f16x2((x2 & 0x0F0F0F0Fu) | ((x3 << 4) & 0xF0F0F0F0u), e23);
      e2m1x8_to_f16x2(((x2 >> 4) & 0x0F0F0F0Fu) | (x3 & 0xF0F0F0F0u), o23);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        mma_f16(o[4 * j + i], mul_f16x2(e01[i], f01), mul_f16x2(o01[i], f01), mul_f16x2(e23[i], f23),
                mul_f16x2(o23[i], f23), pb0, pb1);
    }
  }

  // kN tiles at once: tile i's K codes at code[i] (V's v_step further), its K scales
  // at scale[i] (V's vs_step further); kMasked: only the tokens [lo[i], hi[i]) of
  // its 16 count (at least one).
  template <int kN, bool kMasked>
  __device__ __forceinline__ void tiles(const uint32_t (&code)[kN], const uint32_t (&scale)[kN], uint32_t v_step,
                                        uint32_t vs_step, const int (&lo)[kN], const int (&hi)[kN]) {
    float z[kN][4];
    bool far = false;   // a logit more than the lag past the running maximum
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      scores(code[i], scale[i], z[i]);
      if (kMasked && (lo[i] > 0 || hi[i] < 16)) {
        const int ta = fp4_row_token(gid), tb = ta + 8;
        if (ta < lo[i] || ta >= hi[i]) z[i][0] = z[i][1] = -INFINITY;
        if (tb < lo[i] || tb >= hi[i]) z[i][2] = z[i][3] = -INFINITY;
      }
      far = far || z[i][0] > t0 || z[i][1] > t1 || z[i][2] > t0 || z[i][3] > t1;
    }
    if (__any_sync(0xffffffffu, far)) {
      float x0 = fmaxf(z[0][0], z[0][2]), x1 = fmaxf(z[0][1], z[0][3]);
#pragma unroll
      for (int i = 1; i < kN; ++i) {
        x0 = fmaxf(x0, fmaxf(z[i][0], z[i][2]));
        x1 = fmaxf(x1, fmaxf(z[i][1], z[i][3]));
      }
      x0 = warp_max_over_gid(x0);
      x1 = warp_max_over_gid(x1);
      const float n0 = fmaxf(-nr.x, x0), n1 = fmaxf(-nr.y, x1);
      const float c0 = nr.x == INFINITY ? 0.f : fast_exp2((-nr.x - n0) * lsc.x);
      const float c1 = nr.y == INFINITY ? 0.f : fast_exp2((-nr.y - n1) * lsc.y);
      nr = make_float2(-n0, -n1);
      // (never more than the lag, which bounds P; infinite where all logits are 0)
      t0 = __fadd_rd(n0, kF4Lag * (1.f - 0x1p-20f) * rcp_approx(lsc.x));
      t1 = __fadd_rd(n1, kF4Lag * (1.f - 0x1p-20f) * rcp_approx(lsc.y));
      l0 *= c0;
      l1 *= c1;
#pragma unroll
      for (int mt = 0; mt < kChunks; ++mt) {
        o[mt][0] *= c0;
        o[mt][1] *= c1;
        o[mt][2] *= c0;
        o[mt][3] *= c1;
      }
    }
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      // (a masked -inf stays -inf unless lsc is 0, so it is asked for again)
      const float2 up = make_float2(kF4Shift, kF4Shift);
      const float2 a = fma_f32x2(add_f32x2(make_float2(z[i][0], z[i][1]), nr), lsc, up);
      const float2 b = fma_f32x2(add_f32x2(make_float2(z[i][2], z[i][3]), nr), lsc, up);
      float p[4] = {fast_exp2(a.x), fast_exp2(a.y), fast_exp2(b.x), fast_exp2(b.y)};
      if (kMasked) {
        if (z[i][0] == -INFINITY) p[0] = p[1] = 0.f;
        if (z[i][2] == -INFINITY) p[2] = p[3] = 0.f;
      }
      l0 += p[0] + p[2];
      l1 += p[1] + p[3];
      values<kMasked>(code[i] + v_step, scale[i] + vs_step, p, lo[i], hi[i]);
    }
  }

  // (m, l, O) into the CTA's merge rows: mo [warp][kMaxGqa][stride], then ml.
  __device__ __forceinline__ void store_merge(float* mo, float* mml, int warp) {
    l0 = warp_sum_over_gid(l0);
    l1 = warp_sum_over_gid(l1);
    float* r0 = mo + (warp * kMaxGqa + 2 * tig) * kF4MergeStride + 16 * gid;
#pragma unroll
    for (int mt = 0; mt < kChunks; mt += 2) {
      *reinterpret_cast<float4*>(r0 + 2 * mt) = make_float4(o[mt][0], o[mt][2], o[mt + 1][0], o[mt + 1][2]);
      *reinterpret_cast<float4*>(r0 + kF4MergeStride + 2 * mt) = make_float4(o[mt][1], o[mt][3], o[mt + 1][1], o[mt + 1][3]);
    }
    if (gid == 0) {
      float* ml = mml + (warp * kMaxGqa + 2 * tig) * 2;
      ml[0] = m0();
      ml[1] = l0;
      ml[2] = m1();
      ml[3] = l1;
    }
  }

  // (m, l, O) straight to a piece's rows.
  __device__ __forceinline__ void store_piece(float* rows, int g) {
    l0 = warp_sum_over_gid(l0);
    l1 = warp_sum_over_gid(l1);
    const int h = 2 * tig;
    float* r0 = rows + h * kHeadDim + 16 * gid;
#pragma unroll
    for (int mt = 0; mt < kChunks; mt += 2) {
      if (h < g) __stcg(reinterpret_cast<float4*>(r0 + 2 * mt), make_float4(o[mt][0], o[mt][2], o[mt + 1][0], o[mt + 1][2]));
      if (h + 1 < g)
        __stcg(reinterpret_cast<float4*>(r0 + kHeadDim + 2 * mt), make_float4(o[mt][1], o[mt][3], o[mt + 1][1], o[mt + 1][3]));
    }
    if (gid == 0) __stcg(reinterpret_cast<float4*>(rows + kMaxGqa * kHeadDim + 4 * tig), make_float4(m0(), l0, m1(), l1));
  }

  // The unit's output rows; h0: its first query head.
  __device__ __forceinline__ void store_out_rows(const Fp4DecodeParams& p, int s, int h0, bool any) {
    l0 = warp_sum_over_gid(l0);
    l1 = warp_sum_over_gid(l1);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int hh = 2 * tig + e;
      if (hh >= p.gqa) continue;
      const float zs = p.sinks ? __ldg(p.sinks + h0 + hh) * 1.4426950408889634f + kF4Shift : -INFINITY;
      const float M = e ? m1() : m0(), den = e ? l1 : l0;
      const size_t at = ((size_t)s * p.num_heads + h0 + hh) * kHeadDim + 16 * gid;
      float r[16];
#pragma unroll
      for (int i = 0; i < 16; ++i)
        r[i] = any ? finish(o[i >> 1][e + 2 * (i & 1)], den, M, zs, p.v_scale) : 0.f;
      if (p.out_fp8) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] = f32x2_to_e4m3x2(__fdiv_rn(r[4 * i], p.out_scale), __fdiv_rn(r[4 * i + 1], p.out_scale)) |
                 f32x2_to_e4m3x2(__fdiv_rn(r[4 * i + 2], p.out_scale), __fdiv_rn(r[4 * i + 3], p.out_scale)) << 16;
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + at) = make_uint4(c[0], c[1], c[2], c[3]);
      } else {
        uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at);
        dst[0] = make_uint4(bf16x2_of(r[0], r[1]), bf16x2_of(r[2], r[3]), bf16x2_of(r[4], r[5]), bf16x2_of(r[6], r[7]));
        dst[1] = make_uint4(bf16x2_of(r[8], r[9]), bf16x2_of(r[10], r[11]), bf16x2_of(r[12], r[13]), bf16x2_of(r[14], r[15]));
      }
    }
  }
};

// A unit's pieces: piece i of one that begins in run c0 is run (c0 + i)'s; a run's
// slot 0 holds a piece that an earlier run began, slot 1 one that begins with it.
// Each has room for four kv heads' rows.
__device__ __forceinline__ int fp4_slot(int c0, int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); }
constexpr size_t kF4PieceFloats = (size_t)kF4Warps * kF4RowFloats;
constexpr int kF4Slots = 2 * kF4MaxCtas;

__global__ void __launch_bounds__(kF4Threads, kF4CtasPerSm) pda_fp4_decode_kernel(const Fp4DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  grid_dependents_launch();   // the join kernel may start its launch: it waits for this grid's results
  uint8_t* ring = smem + ((128u - (smem_u32(smem) & 127u)) & 127u);
  Fp4Chunk* notes = reinterpret_cast<Fp4Chunk*>(ring + kF4Stages * kF4StageBytes);
  uint64_t* bars = reinterpret_cast<uint64_t*>(notes + kF4Stages);
  int* sums = reinterpret_cast<int*>(bars + 2 * kF4Stages + 1);   // scan [5]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sums + 8);
  unsigned* pre = reinterpret_cast<unsigned*>(sums + 16);
  const uint32_t ring_u32 = smem_u32(ring);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * kF4Stages, cons_bar = empty0 + 8u * kF4Stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = p.block_size, PPC = p.pages_per_chunk, Hk = p.num_kv_heads, g = p.gqa, hw = p.group, tiles = p.tiles;
  const int HG = Hk / hw;     // units of a sequence

  if (threadIdx.x == 0) {
    for (int i = 0; i < kF4Stages; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, kF4Warps);
    }
    mbar_init(cons_bar, kF4Warps);
    *abort_flag = 0;
    fence_barrier_init();
  }
  grid_dependency_wait();   // nothing above reads what a kernel in front may write

  // ---- the chunks of all sequences: thread i counts sequences [i * each, ...)
  const int each = (p.num_seqs + kF4Threads - 1) / kF4Threads;
  const int s_a = min(p.num_seqs, (int)threadIdx.x * each), s_b = min(p.num_seqs, s_a + each);
  unsigned mine = 0u;
  for (int s = s_a; s < s_b; ++s) mine += (unsigned)fp4_chunks(p, fp4_span(p, s).n);
  unsigned scan = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const unsigned y = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += y;
  }
  if (lane == 31) sums[warp] = (int)scan;
  __syncthreads();
  unsigned before = scan - mine, all = 0u;
#pragma unroll
  for (int w = 0; w < kF4Threads / 32; ++w) {
    if (w < warp) before += (unsigned)sums[w];
    all += (unsigned)sums[w];
  }
  pre[threadIdx.x] = before * (unsigned)HG;
  const unsigned C = all * (unsigned)HG, G = min(gridDim.x, C), run = blockIdx.x;
  if (run >= G) return;   // (whole CTA)
  __syncthreads();

  if (warp == kF4Warps) {
    // ---------------------------------------------------------- producer
    Fp4Runs runs;
    runs.plan(C, G);
    unsigned x = runs.first(run);
    const unsigned end = runs.first(run + 1u);
    int s, n, hg, ci;
    unsigned unit0;                            // the unit's first chunk
    Fp4Span a;
    {
      // the thread whose sequences hold chunk x, then the sequence, 32 at a time
      int i = 0;
      for (int j = lane; j - lane < kF4Threads; j += 32) i += __popc(__ballot_sync(0xffffffffu, pre[j] <= x));
      unsigned at = pre[i - 1];
      s = (i - 1) * each;
      for (;;) {
        const int sl = s + lane;
        const unsigned m = sl < p.num_seqs ? (unsigned)fp4_chunks(p, fp4_span(p, sl).n) * (unsigned)HG : 0u;
        unsigned sum = m;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const unsigned y = __shfl_up_sync(0xffffffffu, sum, d);
          if (lane >= d) sum += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at + sum > x);
        if (past != 0u || s + 32 >= p.num_seqs) {
          const int l = past != 0u ? __ffs((int)past) - 1 : 31;
          unit0 = at + __shfl_sync(0xffffffffu, sum - m, l);
          s = min(s + l, p.num_seqs - 1);
          break;
        }
        at += __shfl_sync(0xffffffffu, sum, 31);
        s += 32;
      }
      a = fp4_span(p, s);
      n = fp4_chunks(p, a.n);
      hg = min((int)((x - unit0) / (unsigned)n), HG - 1);
      unit0 += (unsigned)hg * (unsigned)n;
      ci = (int)(x - unit0);
    }
    bool fresh = true, ok = true;              // fresh: first chunk of a unit (or of the run)
    int run0 = 0, pieces = 1, fill = 0;
    const uint64_t once = evict_first_policy();   // pages are read once: the pieces stay in L2 instead
    const uint32_t page_bytes = (uint32_t)(kFp4TokenBytes * bs * hw);   // of the unit's heads, side by side
    auto entry = [&]() {
      const int pg = ci * PPC + lane;
      return lane < PPC && pg < a.n ? __ldg(p.block_tables + (size_t)s * p.max_blocks + a.first + pg) : 0;
    };
    int block = entry();
    uint32_t stage = 0, parity = 1;
    for (; x < end; ++x, ++fill) {
      const bool done = x + 1u == end, last = ci + 1 == n || done;
      if (fresh) {
        run0 = (int)runs.owner(unit0);
        pieces = (int)runs.owner(unit0 + (unsigned)n - 1u) - run0 + 1;
      }
      // a unit that this run begins and another ends
      if (done && lane == 0 && pieces > 1 && (int)run == run0) {
        const int many = pieces > kF4FewPieces ? 1 : 0;
        const unsigned at = atomicAdd(&p.head->cuts[many], 1u);
        if (at < (unsigned)kF4MaxCtas) p.head->cut[many ? kF4MaxCtas - 1u - at : at] = make_int4(s, hg * hw, run0, pieces);
      }
      const int np = min(PPC, a.n - ci * PPC), t0 = (a.first + ci * PPC) * bs;
      const bool got = mbar_wait_bounded(empty0 + 8u * stage, parity, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) {
          atomicOr(&g_status, kStatusEmptyWaitTimeout);
          *abort_flag = 1;
        }
        ok = false;
        break;
      }
      const uint32_t bar = full0 + 8u * stage;
      if (fresh) {
        // the queries that the consumers read when the chunk is there
        const __nv_bfloat16* q = p.q + ((size_t)s * p.num_heads + (size_t)(hg * hw) * g) * kHeadDim;
        for (int i = lane; i < hw * g * 2; i += 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i * 64));
      }
      if (lane == 0) {
        Fp4Chunk* c = notes + stage;
        const int hi = min(a.hi, t0 + np * bs);
        c->flags = (fresh ? kHdrFirst : 0) | (last ? kHdrLast : 0) |
                   (t0 >= a.lo && t0 + 16 * kF4Warps * tiles / hw <= hi ? kF4Full : 0);
        c->t0 = t0;
        c->lo = a.lo, c->hi = hi;
        c->s = s, c->kvh = hg * hw;
        c->run0 = run0, c->piece = (int)run - run0, c->pieces = pieces;
        if (np > 0) mbar_arrive_expect_tx(bar, (uint32_t)np * page_bytes);
        else mbar_arrive(bar);
      }
      __syncwarp();
      if (lane < np) {
        const int b = checked_block(block, (uint32_t)p.num_blocks);
        bulk_g2s_hint(ring_u32 + stage * kF4StageBytes + (uint32_t)lane * page_bytes,
                      p.cache + ((size_t)b * HG + hg) * page_bytes, page_bytes, bar, once);
      }
      // the next chunk; its table entries are under way while its stage is awaited
      fresh = last;
      if (++ci == n) {
        ci = 0;
        unit0 += (unsigned)n;
        if (++hg == HG) {
          hg = 0;
          s = min(s + 1, p.num_seqs - 1);
          a = fp4_span(p, s);
          n = fp4_chunks(p, a.n);
        }
      }
      if (!done) block = entry();
      if (++stage == kF4Stages) stage = 0, parity ^= 1u;
      __syncwarp();
    }
    if (ok) {
      // end mark: a note without copies
      const bool got = mbar_wait_bounded(empty0 + 8u * stage, parity, abort_flag, kWaitLimitNs);
      if (__all_sync(0xffffffffu, got)) {
        if (lane == 0) {
          notes[stage].flags = kHdrEnd;
          mbar_arrive(full0 + 8u * stage);
        }
        ++fill;
      } else if (lane == 0) {
        atomicOr(&g_status, kStatusEmptyWaitTimeout);
        *abort_flag = 1;
      }
      __syncwarp();
    }
    // never leave the CTA with copies still landing in its shared memory
    for (int f = max(0, fill - kF4Stages); f < fill; ++f) {
      if (!mbar_wait_bounded(full0 + 8u * (f % kF4Stages), (uint32_t)(f / kF4Stages) & 1u, nullptr, kWaitLimitNs)) {
        if (lane == 0) atomicOr(&g_status, kStatusDrainTimeout);
        break;
      }
    }
    return;
  }

  // ------------------------------------------------------------- consumers
  Fp4Worker w;
  w.setup(lane);
  w.reset();
  // this warp's head of the unit, and its first token of a chunk
  const int head = warp % hw, tok = 16 * tiles * (warp / hw);
  const uint32_t rec = (uint32_t)(kFp4TokenBytes * bs);
  uint32_t code_off[kF4Tiles], scale_off[kF4Tiles];
#pragma unroll
  for (int i = 0; i < kF4Tiles; ++i) {
    const int t = tok + 16 * i;
    const uint32_t at = ((uint32_t)(t / bs) * hw + head) * rec;
    code_off[i] = at + (uint32_t)(t % bs) * 64u;
    scale_off[i] = at + (uint32_t)(128 * bs) + (uint32_t)(t % bs) * 8u;
  }
  uint32_t cons_phase = 0, parity = 0;
  for (uint32_t stage = 0;; stage = stage + 1 < kF4Stages ? stage + 1 : 0u, parity ^= stage == 0u ? 1u : 0u) {
    const bool got = mbar_wait_bounded(full0 + 8u * stage, parity, abort_flag, kWaitLimitNs);
    if (!__all_sync(0xffffffffu, got)) {
      if (lane == 0) {
        atomicOr(&g_status, kStatusFullWaitTimeout);
        *abort_flag = 1;
      }
      return;
    }
    const uint32_t base = ring_u32 + stage * kF4StageBytes;
    const Fp4Chunk* c = notes + stage;
    const int flags = c->flags;
    if (flags & kHdrEnd) return;
    if (flags & kHdrFirst) {
      const __nv_bfloat16* q = p.q + ((size_t)c->s * p.num_heads + (size_t)(c->kvh + head) * g) * kHeadDim;
      w.load_q(q + (w.gid < g ? w.gid : 0) * kHeadDim, w.gid < g, p.logit_scale_log2, p.negate != 0);
    }
    // (Pages of 48, 80, 96 or 112 tokens do not fill a chunk, and all their tiles are masked:
    // 256 x 4096 tokens of 32/8 heads 259 us in 48-token blocks, 202 in 16-token ones.)
    if (flags & kF4Full) {
#pragma unroll
      for (int i = 0; i < kF4Tiles; i += 2) {
        if (i >= tiles) break;
        const uint32_t code[2] = {base + code_off[i], base + code_off[i + 1]};
        const uint32_t scale[2] = {base + scale_off[i], base + scale_off[i + 1]};
        const int none[2] = {0, 0}, all16[2] = {16, 16};
        w.tiles<2, false>(code, scale, 64u * bs, 8u * bs, none, all16);
      }
    } else {
      // the tiles that hold tokens that count, one at a time
#pragma unroll 1
      for (int i = 0; i < tiles; ++i) {
        const int t0 = c->t0 + tok + 16 * i;
        const int lo[1] = {max(c->lo - t0, 0)}, hi[1] = {min(c->hi - t0, 16)};
        if (lo[0] >= hi[0]) continue;
        const int tt = tok + 16 * i;
        const uint32_t at = base + ((uint32_t)(tt / bs) * hw + head) * rec;
        const uint32_t code[1] = {at + (uint32_t)(tt % bs) * 64u}, scale[1] = {at + (uint32_t)(128 * bs + tt % bs * 8)};
        w.tiles<1, true>(code, scale, 64u * bs, 8u * bs, lo, hi);
      }
    }
    if (!(flags & kHdrLast)) {
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8u * stage);
      continue;
    }
    const Fp4Chunk hd = *c;
    float* rows = p.pieces + (size_t)fp4_slot(hd.run0, hd.piece) * kF4PieceFloats;
    if (hw == kF4Warps) {
      // the head was this warp's alone
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8u * stage);
      if (hd.pieces == 1) {
        w.store_out_rows(p, hd.s, (hd.kvh + head) * g, hd.hi > hd.lo);
      } else {
        w.store_piece(rows + head * kF4RowFloats, g);
      }
      w.reset();
      continue;
    }
    // All warps are done with the stage: its memory takes the merge rows.
    if (!consumer_sync(cons_bar, cons_phase, lane, abort_flag)) return;
    float* mo = reinterpret_cast<float*>(ring + stage * kF4StageBytes);
    float* mml = mo + kF4Warps * kMaxGqa * kF4MergeStride;
    w.store_merge(mo, mml, warp);
    w.reset();
    if (!consumer_sync(cons_bar, cons_phase, lane, abort_flag)) return;
    for (int r = warp; r < hw * g; r += kF4Warps) {
      const int hh = r / hw, kh = r % hw;   // query head of the group, kv head of the unit
      float M = -INFINITY, den = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = kh; i < kF4Warps; i += hw) {
        const float2 ml = *reinterpret_cast<const float2*>(mml + (i * kMaxGqa + hh) * 2);
        const float4 y = *reinterpret_cast<const float4*>(mo + (i * kMaxGqa + hh) * kF4MergeStride + 4 * lane);
        if (ml.x != -INFINITY) lse_fold(M, den, acc, ml.x, ml.y, y);   // a warp without a tile: nothing
      }
      if (hd.pieces == 1) {
        store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, hd.s, (hd.kvh + kh) * g + hh, lane,
                     hd.hi > hd.lo, M, den, acc, kF4Shift);
      } else {
        float* to = rows + kh * kF4RowFloats;
        __stcg(reinterpret_cast<float4*>(to + hh * kHeadDim) + lane, acc);
        if (lane == 0) __stcg(reinterpret_cast<float2*>(to + kMaxGqa * kHeadDim) + hh, make_float2(M, den));
      }
    }
    // the merge rows were written through the generic proxy; copies come next
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) mbar_arrive(empty0 + 8u * stage);
  }
}

// The join, a programmatic dependent of the decode kernel. Rows of few pieces: a
// warp each. Rows of many (long sequences): a CTA each, its warps taking every
// eighth piece. The order of the additions is the pieces' alone. It runs and
// empties the lists also when CTAs of the decode kernel gave up on a wait.
constexpr int kF4JoinThreads = 256;
constexpr int kF4JoinWarps = kF4JoinThreads / 32;
constexpr int kF4JoinCtas = 760;

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// One row's pieces first, first + step, ... (k <= 32 of them), added up by a warp:
// lane i weighs piece i while the rows are on their way, four at a time.
__device__ __forceinline__ void fp4_add_pieces(const float* pieces, int run0, int first, int step, int k, int kh, int hh,
                                               int lane, float& M, float& den, float4& acc) {
  auto piece = [&](int i) {
    return pieces + (size_t)fp4_slot(run0, first + i * step) * kF4PieceFloats + kh * kF4RowFloats;
  };
  constexpr int kAhead = 4;
  float4 y[kAhead];
  auto load = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      y[j] = j0 + j < k ? __ldcg(reinterpret_cast<const float4*>(piece(j0 + j) + hh * kHeadDim) + lane)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
  };
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < k) ml = __ldcg(reinterpret_cast<const float2*>(piece(lane) + kMaxGqa * kHeadDim) + hh);
  load(0);
  M = warp_max(ml.x);
  const float f = lane < k ? fast_exp2(ml.x - M) : 0.f;   // 0 past the last piece
  den = warp_sum(f * ml.y);
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int j0 = 0; j0 < k; j0 += kAhead) {
    if (j0 > 0) load(j0);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const float v = __shfl_sync(0xffffffffu, f, (j0 + j) & 31);
      acc.x = fmaf(v, y[j].x, acc.x);
      acc.y = fmaf(v, y[j].y, acc.y);
      acc.z = fmaf(v, y[j].z, acc.z);
      acc.w = fmaf(v, y[j].w, acc.w);
    }
  }
}

__global__ void __launch_bounds__(kF4JoinThreads, 5) pda_fp4_join_kernel(const Fp4DecodeParams p) {
  __shared__ int cuts[2];
  __shared__ float part_ml[kF4JoinWarps][2];
  __shared__ float4 part_o[kF4JoinWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = p.gqa, per = p.group * g;   // rows of a unit
  grid_dependency_wait();
  if (threadIdx.x < 2) cuts[threadIdx.x] = min((int)__ldcg(&p.head->cuts[threadIdx.x]), kF4MaxCtas);
  __syncthreads();
  // Entry i of the lists; whatever it holds, what it names lies in bounds.
  auto cut_of = [&](int i) {
    int4 c = __ldcg(p.head->cut + i);
    if (c.x < 0 || c.x >= p.num_seqs || c.y < 0 || c.y + p.group > p.num_kv_heads || c.z < 0 || c.w > kF4MaxCtas - c.z)
      c.w = 0;
    return c;
  };
  for (int r = blockIdx.x * kF4JoinWarps + warp; r < cuts[0] * per; r += gridDim.x * kF4JoinWarps) {
    const int4 c = cut_of(r / per);
    const int kh = r % per / g, hh = r % per % g;
    if (c.w < 1) continue;
    float M, den;
    float4 acc;
    fp4_add_pieces(p.pieces, c.z, 0, 1, min(c.w, kF4FewPieces), kh, hh, lane, M, den, acc);
    store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, c.x, (c.y + kh) * g + hh, lane, true, M, den,
                 acc, kF4Shift);
  }
#pragma unroll 1
  for (int r = blockIdx.x; r < cuts[1] * per; r += gridDim.x) {
    const int4 c = cut_of(kF4MaxCtas - 1 - r / per);   // the same for the whole CTA
    const int kh = r % per / g, hh = r % per % g;
    if (c.w <= kF4FewPieces) continue;
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = warp; b < c.w; b += 32 * kF4JoinWarps) {   // more than 8 pieces: every warp has one
      float m1, d1;
      float4 a1;
      fp4_add_pieces(p.pieces, c.z, b, kF4JoinWarps, min(32, (c.w - b + kF4JoinWarps - 1) / kF4JoinWarps), kh, hh, lane, m1, d1,
                     a1);
      lse_fold(M, den, acc, m1, d1, a1);
    }
    if (lane == 0) part_ml[warp][0] = M, part_ml[warp][1] = den;
    part_o[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
      M = -INFINITY, den = 0.f;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int v = 0; v < kF4JoinWarps; ++v) lse_fold(M, den, acc, part_ml[v][0], part_ml[v][1], part_o[v][lane]);
      store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, c.x, (c.y + kh) * g + hh, lane, true, M,
                   den, acc, kF4Shift);
    }
    __syncthreads();
  }
  // The last CTA leaves the lists empty (each has read their lengths).
  if (threadIdx.x == 0 && atomicInc(&p.head->joined, gridDim.x - 1u) == gridDim.x - 1u) p.head->cuts[0] = p.head->cuts[1] = 0u;
}

}  // namespace pda
