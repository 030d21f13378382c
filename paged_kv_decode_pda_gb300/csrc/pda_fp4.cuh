// Decode attention over the 4-bit cache (records: pda_lowbits.cuh).
//
//   out = sum_t e^(z_t) v_t / (sum_t e^(z_t) + e^sink),  z_t = scale q . k_t
//
// over the tokens max(0, L - window) .. L - 1 of a sequence. What it cannot do
// without: 144 bytes per (token, kv head) against 256 for e4m3, so the same
// bandwidth brings 1.8 times the tokens, and converting and multiplying them is
// what comes close to bounding the kernel.
//
// Work. A unit is a (sequence, kv head), its tokens in chunks of whole pages
// (up to kF4ChunkTokens tokens). All units' chunks, one after the other, are cut
// into equal runs, one per resident CTA, wherever the cuts fall: every batch (a
// few long sequences, many ragged ones) loads all SMs alike, with no queue and
// one launch. A unit cut by a run's end is joined from its pieces (O, m, l) in
// the workspace by whichever CTA brings the last one, in the pieces' order, so
// the result does not depend on which CTA that is.
//
// A CTA. One producer warp copies a chunk's records (K, V and both scales of a
// page are one contiguous piece: one bulk copy per page) into a ring; four
// consumer warps take two of its 16-token tiles each:
//   S^T = K (16 tokens x 128) Q^T (128 x 8 heads), O^T += V^T (128 x 16) P^T
// on warp MMAs whose A fragments are made in registers: e2m1 -> f16 by the
// conversion instruction, times the block's scale, exact (6 significant bits).
// Q enters as in pda_decode (shifted by a power of two into f16), P as one f16,
// off by at most 2^-11 of itself; the normaliser sums P unrounded in fp32.
//
// The contraction's order is free, so each lane takes what lies side by side:
// of a K row 16 bytes (32 dims), of four V rows one 8-byte block of 16 dims each,
// whose single scale then serves all its dims. MMA row r holds token
// fp4_row_token(r) and V's k slots the same tokens, chosen so that both kinds of
// loads spread over all banks.
//
// The running maximum is let fall up to 8 (log2) behind: P stays below 2^8, well
// inside f16, and nearly every tile passes with one vote in place of a maximum
// over the lanes and a rescale.
#pragma once

#include "pda_kernels.cuh"
#include "pda_lowbits.cuh"

namespace pda {

constexpr int kF4ChunkTokens = 128;
constexpr int kF4Tiles = 2;                                    // 16-token tiles of a chunk per consumer warp
static_assert(kF4ChunkTokens == 16 * kF4Tiles * kConsumerWarps, "a chunk's tiles go round the warps");
constexpr int kF4MaxPages = kF4ChunkTokens / 16;
constexpr int kF4Stages = 3;
constexpr int kF4CtasPerSm = 3;
constexpr uint32_t kF4StageBytes = kF4ChunkTokens * kFp4TokenBytes;
constexpr uint32_t kF4QBytes = kMaxGqa * kHeadDim * 2;
constexpr int kF4MergeStride = kHeadDim + 4;
static_assert(kConsumerWarps * kMaxGqa * (kF4MergeStride + 2) * 4 <= kF4StageBytes, "merge rows fit a stage");
constexpr float kF4Lag = 8.f;                                  // the running maximum's lag, log2
constexpr int kF4MaxCtas = 1024;
constexpr int kF4FoldGroup = 16;                               // pieces folded at once where a unit has many
constexpr int kF4RowFloats = kMaxGqa * (kHeadDim + 2);         // a piece: O rows, then (m, l) pairs

// Workspace: a header that starts at zero, then 4 piece slots per CTA (two of
// its own, two for folded groups).
struct Fp4Head {
  unsigned epoch;                                              // calls finished
  unsigned done;                                               // CTAs of this call that have left
  unsigned long long arrived[3 * kF4MaxCtas];                  // epoch + 1 (high), pieces that have come (low)
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
  float logit_scale_log2;   // |scale * k_scale| * log2(e)
  int negate;
  float v_scale;
  int out_fp8;
  float out_scale;
};

// A chunk's header, written by the producer with its copies.
struct Fp4Chunk {
  int s, kvh;
  int tok0, tokens;         // first token of the chunk's pages, tokens in them (0: an empty sequence)
  int lo, hi;               // tokens of the sequence that count
  int flags;
  int piece, pieces;        // this CTA's piece of the unit
  int pad;
};
constexpr uint32_t kF4AuxBytes = kF4QBytes + ((sizeof(Fp4Chunk) + 15) / 16) * 16;

// Ring, side entries, barriers (full, empty, consumers), scan sums and flags.
constexpr uint32_t kF4Smem = 128 + kF4Stages * (kF4StageBytes + kF4AuxBytes) + (2 * kF4Stages + 1) * 8 + 128;

__device__ __forceinline__ int fp4_row_token(int r) {
  const int t = (r >> 1) & 3;
  return ((r & 1) ? (t ^ 1) + 4 : t) + (r & 8);
}

// Pages [first, first + n) and tokens [lo, hi) of a sequence.
struct Fp4Span {
  int first, n, lo, hi;
};
__device__ __forceinline__ Fp4Span fp4_span(const Fp4DecodeParams& p, int s) {
  Fp4Span a;
  a.hi = max(0, min(__ldg(p.seq_lens + s), p.max_blocks * p.block_size));
  a.lo = p.window > 0 ? max(0, a.hi - p.window) : 0;
  a.first = a.lo / p.block_size;
  a.n = (a.hi + p.block_size - 1) / p.block_size - a.first;
  return a;
}
// An empty sequence has one chunk too: somebody writes its zeros.
__device__ __forceinline__ int fp4_chunks(int pages, int per) { return pages > 0 ? (pages + per - 1) / per : 1; }

// A consumer warp's share of a unit.
struct Fp4Worker {
  int gid, tig;
  uint32_t k_off, v_off, ks_off, vs_off;
  uint32_t qf[kChunks][2];
  float lsc0, lsc1;
  float m0, m1, l0, l1;
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
  __device__ __forceinline__ void reset() {
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // Q^T fragments of the row at qrow (shared): k step c's slots (2 tig, 2 tig
  // + 1), (2 tig + 8, 2 tig + 9) are dims 32 tig + 4c .. + 3. Each row is shifted
  // by a power of two that puts its largest |q| into [2^14, 2^15).
  __device__ __forceinline__ void load_q(uint32_t qrow, bool live, float lsc, bool negate) {
    uint2 v[kChunks];
    uint32_t mx = 0u;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      v[c] = live ? ld_shared_v2(qrow + (uint32_t)(64 * tig + 8 * c)) : make_uint2(0u, 0u);
      mx = __vmaxu2(mx, v[c].x & 0x7FFF7FFFu);
      mx = __vmaxu2(mx, v[c].y & 0x7FFF7FFFu);
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
    lsc0 = lsc * exp2_int(__shfl_sync(0xffffffffu, e, 8 * tig));
    lsc1 = lsc * exp2_int(__shfl_sync(0xffffffffu, e, 8 * tig + 4));
  }

  // Logits (log2) of a tile: z[0], z[1] token row gid, z[2], z[3] row gid + 8.
  __device__ __forceinline__ void scores(uint32_t k, uint32_t ks, float (&z)[4]) const {
    uint32_t wa[4], wb[4];
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(wa[0]), "=r"(wa[1]), "=r"(wa[2]), "=r"(wa[3]) : "r"(k + k_off));
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(wb[0]), "=r"(wb[1]), "=r"(wb[2]), "=r"(wb[3]) : "r"(k + k_off + 512u));
    unsigned short ua, ub;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(ua) : "r"(ks + ks_off));
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(ub) : "r"(ks + ks_off + 64u));
    const uint32_t sa = e4m3x2_lo_to_f16x2(ua), sb = e4m3x2_lo_to_f16x2(ub);
    float sc[4] = {0.f, 0.f, 0.f, 0.f}, sd[4] = {0.f, 0.f, 0.f, 0.f};
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
      mma_f16(sc, a[0], b[0], a[1], b[1], qf[2 * j][0], qf[2 * j][1]);
      mma_f16(sd, a[2], b[2], a[3], b[3], qf[2 * j + 1][0], qf[2 * j + 1][1]);
    }
    z[0] = (sc[0] + sd[0]) * lsc0;
    z[1] = (sc[1] + sd[1]) * lsc1;
    z[2] = (sc[2] + sd[2]) * lsc0;
    z[3] = (sc[3] + sd[3]) * lsc1;
  }

  // O^T += V^T P^T of a tile; p in scores' order. [lo, hi): the tile's tokens
  // that count (the others' scales may hold anything, also NaN).
  __device__ __forceinline__ void values(uint32_t v, uint32_t vs, const float (&p)[4], int lo, int hi) {
    const uint32_t pb0 = movmatrix_trans(pack_f16x2(p[0], p[1]));
    const uint32_t pb1 = movmatrix_trans(pack_f16x2(p[2], p[3]));
    const uint2 w0 = ld_shared_v2(v + v_off);                                             // token tig
    const uint2 w1 = ld_shared_v2(v + v_off + ((tig & 1) ? 192u : 320u));                 // (tig ^ 1) + 4
    const uint2 w2 = ld_shared_v2(v + v_off + 512u);                                      // tig + 8
    const uint2 w3 = ld_shared_v2(v + v_off + 512u + ((tig & 1) ? 192u : 320u));          // (tig ^ 1) + 12
    uint32_t s;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(s) : "r"(vs + vs_off));
    if (lo > 0 || hi < 16) {
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

  // kN tiles at once; tile i's records at k[i], v[i], ks[i], vs[i], the tokens
  // [lo[i], hi[i]) of its 16 counting (at least one).
  template <int kN>
  __device__ __forceinline__ void tiles(const uint32_t (&k)[kF4Tiles], const uint32_t (&v)[kF4Tiles],
                                        const uint32_t (&ks)[kF4Tiles], const uint32_t (&vs)[kF4Tiles],
                                        const int (&lo)[kF4Tiles], const int (&hi)[kF4Tiles]) {
    float z[kN][4];
    float x0 = -INFINITY, x1 = -INFINITY;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      scores(k[i], ks[i], z[i]);
      if (lo[i] > 0 || hi[i] < 16) {
        const int ta = fp4_row_token(gid), tb = ta + 8;
        if (ta < lo[i] || ta >= hi[i]) z[i][0] = z[i][1] = -INFINITY;
        if (tb < lo[i] || tb >= hi[i]) z[i][2] = z[i][3] = -INFINITY;
      }
      x0 = fmaxf(x0, fmaxf(z[i][0], z[i][2]));
      x1 = fmaxf(x1, fmaxf(z[i][1], z[i][3]));
    }
    if (__any_sync(0xffffffffu, x0 > m0 + kF4Lag || x1 > m1 + kF4Lag)) {
      const float n0 = fmaxf(m0, warp_max_over_gid(x0)), n1 = fmaxf(m1, warp_max_over_gid(x1));
      const float c0 = fast_exp2(m0 - n0), c1 = fast_exp2(m1 - n1);   // 0 while m is -inf
      m0 = n0;
      m1 = n1;
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
      const float p[4] = {fast_exp2(z[i][0] - m0), fast_exp2(z[i][1] - m1), fast_exp2(z[i][2] - m0),
                          fast_exp2(z[i][3] - m1)};
      l0 += p[0] + p[2];
      l1 += p[1] + p[3];
      values(v[i], vs[i], p, lo[i], hi[i]);
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
      ml[0] = m0;
      ml[1] = l0;
      ml[2] = m1;
      ml[3] = l1;
    }
  }
};

// One thread: piece counter i gains one piece; true for the last of `pieces`,
// which leaves it at zero. A word of another call counts as zero, so a call that
// gave up leaves nothing to the next.
__device__ __forceinline__ bool fp4_arrive(Fp4Head* head, int i, unsigned epoch, unsigned pieces) {
  const unsigned long long mine = (unsigned long long)(epoch + 1u) << 32;
  unsigned long long old = __ldcg(head->arrived + i);
  for (;;) {
    const unsigned come = (old >> 32) == (mine >> 32) ? (unsigned)old + 1u : 1u;
    const unsigned long long now = come == pieces ? 0ull : mine | come;
    const unsigned long long seen = atomicCAS(head->arrived + i, old, now);
    if (seen == old) return come == pieces;
    old = seen;
  }
}

// Slot of piece i of a unit whose first piece is CTA c0's: a CTA's slot 0 holds
// a piece that an earlier CTA began, slot 1 one that begins with it.
__device__ __forceinline__ int fp4_slot(int c0, int i) { return 2 * (c0 + i) + (i == 0 ? 1 : 0); }

// Head row hh of `n` pieces folded in order (one warp, lane 4 dims).
template <class Slot>
__device__ __forceinline__ void fp4_fold(const float* pieces, const Slot& slot, int n, int hh, int lane, float& M,
                                         float& den, float4& acc) {
  M = -INFINITY;
  den = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* r = pieces + (size_t)slot(i) * kF4RowFloats;
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(r + kMaxGqa * kHeadDim) + hh);
    const float4 x = __ldcg(reinterpret_cast<const float4*>(r + hh * kHeadDim) + lane);
    lse_fold(M, den, acc, ml.x, ml.y, x);
  }
}
__device__ __forceinline__ void fp4_store_piece(float* pieces, int slot, int hh, int lane, float M, float den,
                                                const float4& acc) {
  float* r = pieces + (size_t)slot * kF4RowFloats;
  __stcg(reinterpret_cast<float4*>(r + hh * kHeadDim) + lane, acc);
  if (lane == 0) __stcg(reinterpret_cast<float2*>(r + kMaxGqa * kHeadDim) + hh, make_float2(M, den));
}

__global__ void __launch_bounds__(kThreads, kF4CtasPerSm) pda_fp4_decode_kernel(const Fp4DecodeParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + ((128u - (smem_u32(smem) & 127u)) & 127u);
  uint8_t* aux = ring + kF4Stages * kF4StageBytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(aux + kF4Stages * kF4AuxBytes);
  long long* where = reinterpret_cast<long long*>(bars + 2 * kF4Stages + 1);   // first chunk of the first sequence
  int* sums = reinterpret_cast<int*>(where + 1);                               // scan [5], first sequence, vote
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sums + 8);
  const uint32_t ring_u32 = smem_u32(ring), aux_u32 = smem_u32(aux);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8u * kF4Stages, cons_bar = full0 + 16u * kF4Stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int bs = p.block_size, PPC = p.pages_per_chunk, Hk = p.num_kv_heads, g = p.gqa;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kF4Stages; ++i) {
      mbar_init(full0 + 8u * i, 1);
      mbar_init(empty0 + 8u * i, kConsumerWarps);
    }
    mbar_init(cons_bar, kConsumerWarps);
    *abort_flag = 0;
    *where = 0;
    sums[5] = 0;
    fence_barrier_init();
  }

  // ---- this CTA's run of chunks, and the sequence that it begins in
  const int per = (p.num_seqs + kThreads - 1) / kThreads;
  const int s_a = min(p.num_seqs, (int)threadIdx.x * per), s_b = min(p.num_seqs, s_a + per);
  int mine = 0;
  for (int s = s_a; s < s_b; ++s) mine += fp4_chunks(fp4_span(p, s).n, PPC);
  int scan = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int x = __shfl_up_sync(0xffffffffu, scan, d);
    if (lane >= d) scan += x;
  }
  if (lane == 31) sums[warp] = scan;
  const unsigned epoch = __ldcg(&p.head->epoch);
  __syncthreads();
  int before = scan - mine, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  const long long C = (long long)all * Hk;
  const long long G = (long long)gridDim.x < C ? (long long)gridDim.x : C;
  const long long cta = blockIdx.x;
  const long long begin = cta < G ? cta * C / G : 0, end = cta < G ? (cta + 1) * C / G : 0;
  if (begin < end && begin >= (long long)before * Hk && begin < (long long)(before + mine) * Hk) {
    long long at = before;
    for (int s = s_a; s < s_b; ++s) {
      const int n = fp4_chunks(fp4_span(p, s).n, PPC);
      if (begin < (at + n) * Hk) {
        *where = at * Hk;
        sums[5] = s;
        break;
      }
      at += n;
    }
  }
  __syncthreads();

  if (warp == kConsumerWarps) {
    // ---------------------------------------------------------- producer
    int fill = 0;
    bool ok = true;
    if (begin < end) {
      int s = sums[5];
      Fp4Span a = fp4_span(p, s);
      int n = fp4_chunks(a.n, PPC);
      long long unit0 = *where;   // the unit's first chunk
      int kvh = min((int)((begin - unit0) / n), Hk - 1);
      unit0 += (long long)kvh * n;
      int ci = (int)(begin - unit0);
      bool fresh = true;          // first chunk of a unit (or of the run)
      int piece = 0, pieces = 1;
      auto entry = [&](const Fp4Span& b, int seq, int c) {
        const int pg = c * PPC + lane;
        return lane < PPC && pg < b.n ? __ldg(p.block_tables + (size_t)seq * p.max_blocks + b.first + pg) : 0;
      };
      int block = entry(a, s, ci);
      for (long long x = begin; x < end; ++x, ++fill) {
        if (fresh) {
          const long long c0 = ((unit0 + 1) * G - 1) / C, c1 = ((unit0 + n) * G - 1) / C;
          piece = (int)(cta - c0);
          pieces = (int)(c1 - c0) + 1;
        }
        // the next chunk, its table entries under way while this one's slot is awaited
        const bool last = ci + 1 == n || x + 1 == end;
        int s2 = s, kvh2 = kvh, ci2 = ci + 1, n2 = n;
        long long unit2 = unit0;
        Fp4Span a2 = a;
        if (ci2 == n) {
          ci2 = 0;
          unit2 += n;
          if (++kvh2 == Hk) {
            kvh2 = 0;
            s2 = min(s + 1, p.num_seqs - 1);
            if (x + 1 < end) {
              a2 = fp4_span(p, s2);
              n2 = fp4_chunks(a2.n, PPC);
            }
          }
        }
        const int block2 = x + 1 < end ? entry(a2, s2, ci2) : 0;

        const int np = min(PPC, a.n - ci * PPC);
        const int stage = fill % kF4Stages;
        const bool got = mbar_wait_bounded(empty0 + 8u * stage, ((uint32_t)(fill / kF4Stages) & 1u) ^ 1u, abort_flag,
                                           kWaitLimitNs);
        if (!__all_sync(0xffffffffu, got)) {
          if (lane == 0) {
            atomicOr(&g_status, kStatusEmptyWaitTimeout);
            *abort_flag = 1;
          }
          ok = false;
          break;
        }
        const uint32_t bar = full0 + 8u * stage;
        const uint32_t page_bytes = (uint32_t)(kFp4TokenBytes * bs);
        if (lane == 0) {
          Fp4Chunk* hd = reinterpret_cast<Fp4Chunk*>(aux + (size_t)stage * kF4AuxBytes + kF4QBytes);
          hd->s = s;
          hd->kvh = kvh;
          hd->tok0 = (a.first + ci * PPC) * bs;
          hd->tokens = np * bs;
          hd->lo = a.lo;
          hd->hi = a.hi;
          hd->flags = (fresh ? kHdrFirst : 0) | (last ? kHdrLast : 0);
          hd->piece = piece;
          hd->pieces = pieces;
          if (np > 0) {
            const uint32_t q_bytes = fresh ? (uint32_t)(g * kHeadDim * 2) : 0u;
            mbar_arrive_expect_tx(bar, (uint32_t)np * page_bytes + q_bytes);
            if (fresh)
              bulk_g2s(aux_u32 + (uint32_t)stage * kF4AuxBytes, p.q + ((size_t)s * p.num_heads + (size_t)kvh * g) * kHeadDim,
                       q_bytes, bar);
          } else {
            mbar_arrive(bar);
          }
        }
        __syncwarp();
        if (lane < np) {
          const int b = checked_block(block, (uint32_t)p.num_blocks);
          bulk_g2s(ring_u32 + (uint32_t)stage * kF4StageBytes + (uint32_t)lane * page_bytes,
                   p.cache + ((size_t)b * Hk + kvh) * page_bytes, page_bytes, bar);
        }
        __syncwarp();
        fresh = last;
        s = s2, kvh = kvh2, ci = ci2, n = n2, unit0 = unit2, a = a2, block = block2;
      }
    }
    if (ok) {
      // end marker: a header without copies
      const int stage = fill % kF4Stages;
      const bool got = mbar_wait_bounded(empty0 + 8u * stage, ((uint32_t)(fill / kF4Stages) & 1u) ^ 1u, abort_flag,
                                         kWaitLimitNs);
      if (__all_sync(0xffffffffu, got)) {
        if (lane == 0) {
          reinterpret_cast<Fp4Chunk*>(aux + (size_t)stage * kF4AuxBytes + kF4QBytes)->flags = kHdrEnd;
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
  } else {
    // --------------------------------------------------------- consumers
    Fp4Worker w;
    w.setup(lane);
    w.reset();
    uint32_t cons_phase = 0;
    const int tpp = bs / 16;
    // this warp's tiles of a chunk: warp, warp + 4
    uint32_t code_off[kF4Tiles], scale_off[kF4Tiles];
#pragma unroll
    for (int i = 0; i < kF4Tiles; ++i) {
      const int tile = warp + i * kConsumerWarps;
      const uint32_t page = (uint32_t)(tile / tpp * (kFp4TokenBytes * bs));
      code_off[i] = page + (uint32_t)(tile % tpp) * 1024u;
      scale_off[i] = page + (uint32_t)(128 * bs) + (uint32_t)(tile % tpp) * 128u;
    }
    for (int fill = 0;; ++fill) {
      const int stage = fill % kF4Stages;
      const bool got = mbar_wait_bounded(full0 + 8u * stage, (uint32_t)(fill / kF4Stages) & 1u, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) {
        if (lane == 0) {
          atomicOr(&g_status, kStatusFullWaitTimeout);
          *abort_flag = 1;
        }
        break;
      }
      const uint32_t sbase = ring_u32 + (uint32_t)stage * kF4StageBytes;
      const Fp4Chunk hd = *reinterpret_cast<const Fp4Chunk*>(aux + (size_t)stage * kF4AuxBytes + kF4QBytes);
      if (hd.flags & kHdrEnd) break;
      if (hd.flags & kHdrFirst) {
        w.reset();
        if (hd.tokens > 0)
          w.load_q(aux_u32 + (uint32_t)stage * kF4AuxBytes + (uint32_t)(w.gid < g ? w.gid : 0) * (kHeadDim * 2), w.gid < g,
                   p.logit_scale_log2, p.negate != 0);
      }
      // tiles of the chunk that hold tokens that count, the first ones of k, v, ...
      uint32_t k[kF4Tiles], v[kF4Tiles], ks[kF4Tiles], vs[kF4Tiles];
      int lo[kF4Tiles], hi[kF4Tiles], n = 0;
#pragma unroll
      for (int i = 0; i < kF4Tiles; ++i) {
        const int t0 = 16 * (warp + i * kConsumerWarps);
        const int a = hd.lo - hd.tok0 - t0, b = min(hd.hi - hd.tok0, hd.tokens) - t0;
        if (a < 16 && b > 0) {
          // (kept at constant indexes: registers)
          if (n == 0) {
            k[0] = sbase + code_off[i], ks[0] = sbase + scale_off[i], lo[0] = max(a, 0), hi[0] = min(b, 16);
          } else {
            k[1] = sbase + code_off[i], ks[1] = sbase + scale_off[i], lo[1] = max(a, 0), hi[1] = min(b, 16);
          }
          ++n;
        }
      }
#pragma unroll
      for (int i = 0; i < kF4Tiles; ++i) {
        if (i >= n) k[i] = ks[i] = 0u, lo[i] = 0, hi[i] = 16;
        v[i] = k[i] + (uint32_t)(64 * bs);
        vs[i] = ks[i] + (uint32_t)(8 * bs);
      }
      if (n == 2) w.tiles<2>(k, v, ks, vs, lo, hi);
      else if (n == 1) w.tiles<1>(k, v, ks, vs, lo, hi);

      if (hd.flags & kHdrLast) {
        // All warps are done with the stage: its memory takes the merge rows.
        if (!consumer_sync(cons_bar, cons_phase, lane, abort_flag)) break;
        float* mo = reinterpret_cast<float*>(ring + (size_t)stage * kF4StageBytes);
        float* mml = mo + kConsumerWarps * kMaxGqa * kF4MergeStride;
        w.store_merge(mo, mml, warp);
        if (!consumer_sync(cons_bar, cons_phase, lane, abort_flag)) break;
        const int c0 = blockIdx.x - hd.piece;
        for (int hh = warp; hh < g; hh += kConsumerWarps) {
          float M = -INFINITY, den = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int i = 0; i < kConsumerWarps; ++i) {
            const float2 ml = *reinterpret_cast<const float2*>(mml + (i * kMaxGqa + hh) * 2);
            const float4 x = *reinterpret_cast<const float4*>(mo + (i * kMaxGqa + hh) * kF4MergeStride + 4 * lane);
            if (ml.x != -INFINITY) lse_fold(M, den, acc, ml.x, ml.y, x);   // a warp without a tile: nothing
          }
          if (hd.pieces == 1)
            store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, hd.s, hd.kvh * g + hh, lane,
                         hd.tokens > 0, M, den, acc);
          else
            fp4_store_piece(p.pieces, fp4_slot(c0, hd.piece), hh, lane, M, den, acc);
        }
        if (hd.pieces > 1) {
          // Join: the pieces as they are, or where there are many in groups first.
          const bool grouped = hd.pieces > 2 * kF4FoldGroup;
          const int group = hd.piece / kF4FoldGroup, g0 = group * kF4FoldGroup;
          const int gn = min(kF4FoldGroup, hd.pieces - g0), groups = (hd.pieces + kF4FoldGroup - 1) / kF4FoldGroup;
          const int fold_base = 2 * gridDim.x;   // slots of folded groups
          bool live = true;
#pragma unroll 1
          for (int level = grouped ? 0 : 1; level < 2 && live; ++level) {
            __threadfence();   // this thread's part of the piece, before the arrival
            if (!consumer_sync(cons_bar, cons_phase, lane, abort_flag)) {
              live = false;
              break;
            }
            if (threadIdx.x == 0) {
              const bool all_here =
                  level == 0 ? fp4_arrive(p.head, fp4_slot(c0, g0), epoch, (unsigned)gn)
                             : fp4_arrive(p.head, 2 * kF4MaxCtas + c0, epoch, (unsigned)(grouped ? groups : hd.pieces));
              __threadfence();
              sums[6] = all_here ? 1 : 0;
            }
            if (!consumer_sync(cons_bar, cons_phase, lane, abort_flag)) {
              live = false;
              break;
            }
            if (*reinterpret_cast<volatile int*>(sums + 6) == 0) break;
            for (int hh = warp; hh < g; hh += kConsumerWarps) {
              float M, den;
              float4 acc;
              if (level == 0) {
                fp4_fold(p.pieces, [&](int i) { return fp4_slot(c0, g0 + i); }, gn, hh, lane, M, den, acc);
                fp4_store_piece(p.pieces, fold_base + fp4_slot(c0, g0), hh, lane, M, den, acc);
              } else {
                if (grouped)
                  fp4_fold(p.pieces, [&](int i) { return fold_base + fp4_slot(c0, i * kF4FoldGroup); }, groups, hh, lane, M,
                           den, acc);
                else
                  fp4_fold(p.pieces, [&](int i) { return fp4_slot(c0, i); }, hd.pieces, hh, lane, M, den, acc);
                store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, hd.s, hd.kvh * g + hh, lane,
                             true, M, den, acc);
              }
            }
          }
          if (!live) break;
        }
        // the merge rows were written through the generic proxy; copies come next
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8u * stage);
    }
  }
  // Every CTA counts itself out, also one that gave up; the last one starts the
  // next call's epoch, to which counters that a call left unfinished mean nothing.
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&p.head->done, 1u) == gridDim.x - 1u) {
      atomicExch(&p.head->done, 0u);
      atomicAdd(&p.head->epoch, 1u);
    }
  }
}

}  // namespace pda
