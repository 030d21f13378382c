// Attention of a chunk of new tokens per sequence over the paged e4m3 cache
// (pda_extend), on the fifth-generation tensor cores.
//
// One CTA holds up to 256 query rows of one (sequence, kv head): the g heads
// of a group share K and V, so row r is token r / g, head r % g of the tile.
// With S = Q K^T and c the row's factor from S to logits in log2 units, each
// row keeps a reference m, a value of S, and
//   P = 2^(S c + b),  l = sum P,  O += P V,   out = v_scale O / l,
// with b close to 7 - m c (extend_exponent). The reference follows the running
// maximum lazily: while S c + b stays at or below 15, O stays as it is and P
// grows (P <= 2^15 fits f16; the offset of 7 leaves f16 31 binades below the
// maximum for small weights); only a larger step rescales O and l. S, l, O and
// the references are fp32; P rounds once to f16 (2^-11 relative, while l sums
// it unrounded), Q is exact in f16 after a shift of its row by a power of two,
// K and V are exact in f16.
//
// Roles (16 warps):
//   warps 0-3, 4-7    softmax of rows 0..127 (block A) and 128..255 (block B):
//                     thread = row, a row of S read from tensor memory into
//                     registers, P written back over it
//   warps 8-11        K and V: 16-byte loads through the block table, e4m3 ->
//                     f16 in registers, stores in the matrix units' layout
//   warps 12, 13      issue the products of block A, B
//   warp 14           takes and describes the next work item (15 idle:
//                     registers are traded by groups of four warps)
// Tensor memory (512 columns): S_A, S_B (128 each; P takes the first 64 of
// its block's), O_A, O_B. Shared memory: Q 64 KiB, two K stages and three V
// stages of 128 tokens, 32 KiB each, in the layout without swizzle: 8 x 16
// byte core matrices, 16-byte column c of row r at c * 2048 + r * 16, which
// lanes with consecutive rows store without bank conflicts.
// While block A is in its softmax the tensor core works for block B.
//
// With at most 128 rows in the tile (a few tokens per sequence) both blocks
// take the same rows, A the even and B the odd tiles of 128 tokens, and their
// (O, m, l) are joined at the end, so the two softmax groups still overlap.
#pragma once

#include "pda_kernels.cuh"

namespace pda {

// What the order holds. The items of the last, partial round over the CTAs
// are cut into pieces of their KV range, so that more CTAs share them.
struct ExtendHead {
  int tiles;                    // tiles in the order
  int whole;                    // work items handed out whole
  int tail;                     // items behind them (fewer than CTAs)
  int pieces;                   // pieces of each of those
};

struct ExtendParams {
  void* out;                    // [T][H][128]
  const __nv_bfloat16* q;       // [T][H][128]
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* block_tables;  // [S][MB]
  const int32_t* seq_lens;      // [S]
  const int32_t* query_starts;  // [S + 1]
  int num_tokens;
  int num_seqs;
  int num_heads;
  int num_kv_heads;
  int gqa;
  int gqa_inverse;              // ceil(2^16 / gqa): see token_of
  int block_size;
  int max_blocks;
  int window;
  float logit_scale_log2;       // |scale * k_scale| * log2(e)
  int negate;                   // scale * k_scale < 0: the queries are negated
  float v_scale;
  const float* sinks;
  int out_fp8;
  float out_scale;
  int v_shuffled;
  uint32_t block_limit;
  int tile_tokens;              // tokens of a full tile: 256 / g
  int tiles;                    // tile slots
  int nsplit;                   // KV splits
  const int2* order;            // (sequence, first token) of the tiles, longest first; nullptr: by slot
  const ExtendHead* head;       // with an order: what it holds
  float* tail_o;                // pieces of the last items: [item][256 rows][pieces][128]
  float* tail_ml;               // and their (reference, l)
  unsigned* queue;              // next work item, CTAs done (both left at zero); nullptr: items dealt out in turn
  float* part_o;                // [T][H][nsplit][128]   (nsplit > 1)
  float* part_ml;               // [T][H][nsplit][2]: reference (log2 units), l
  uint32_t zero;                // 0 (see release_item)
};

constexpr int kExtRows = 128;                         // rows of a block
constexpr int kExtTile = 128;                         // tokens of a KV tile
constexpr int kExtThreads = 16 * 32;
// Registers per thread: at launch, then after the warps have traded them.
constexpr int kExtLaunchRegs = 128;
constexpr int kExtSoftmaxRegs = 192;
constexpr int kExtConvertRegs = 88;
constexpr int kExtIssueRegs = 40;
static_assert(256 * kExtSoftmaxRegs + 128 * kExtConvertRegs + 128 * kExtIssueRegs <= kExtThreads * kExtLaunchRegs,
              "the warps' registers come out of the CTA's own");
constexpr uint32_t kExtOperand = 128u * 128u * 2u;    // one f16 operand tile: 32 KiB
constexpr uint32_t kExtColumn = 128u * 16u;           // one 16-byte column of an operand
constexpr uint32_t kExtKStages = 2, kExtVStages = 3;
constexpr uint32_t kExtQOff = 0;
constexpr uint32_t kExtKOff = 2 * kExtOperand;
constexpr uint32_t kExtVOff = kExtKOff + kExtKStages * kExtOperand;
constexpr uint32_t kExtBarOff = kExtVOff + kExtVStages * kExtOperand;
constexpr int kExtAhead = 4;                          // tiles before an item's end that the next one is taken
constexpr int kExtSlots = 2;                          // work items known ahead
enum : int {                                          // barriers (8 bytes each)
  kBarItemFull = 0,                                   // a work item described
  kBarItemFree = kBarItemFull + kExtSlots,            // read by the 14 warps that work on it
  kBarQ = kBarItemFree + kExtSlots,                   // queries of block A, B stored (4 warps), a pair per item slot
  kBarKFull = kBarQ + 2 * kExtSlots,                              // f16 tiles (4 warps), up to 2 stages of K, 3 of V
  kBarKFree = kBarKFull + 2,                          // and let go of by both blocks
  kBarVFull = kBarKFree + 2,
  kBarVFree = kBarVFull + 3,
  kBarS = kBarVFree + 3,                              // S of block A, B ready
  kBarP = kBarS + 2,                                  // P's halves, of block A, B ready (4 warps)
  kBarO = kBarP + 4,                                  // O of block A, B final
  kBarTurn = kBarO + 2,                               // block A's, B's turn to issue
  kBarSums = kBarTurn + 2,                            // both blocks' (m, l) exchanged (8 warps)
  kBarJoined = kBarSums + 1,                          // both blocks' O read (8 warps)
  kBarAhead = kBarJoined + 1,                         // the item's end is near: the next one may be taken (4 warps)
  kBarCount = kBarAhead + 1
};
constexpr uint32_t kExtItemOff = kExtBarOff + ((kBarCount * 8u + 15u) & ~15u);
constexpr uint32_t kExtSumsOff = kExtItemOff + kExtSlots * 64u;
constexpr uint32_t kExtMiscOff = kExtSumsOff + 2u * 128u * 8u;   // tensor memory base, abort flag
constexpr uint32_t kExtSmem = kExtMiscOff + 16u;
static_assert(kExtSmem <= 232448, "shared memory of one CTA");
constexpr float kExtOffset = 7.f;                     // P = 2^(S c + b), b = kExtOffset - m c
constexpr float kExtLimit = 15.f;                     // largest S c + b that leaves m as it is

// Token of a tile's row: row / gqa, exact for rows below 256 and gqa <= 8
// (the inverse is at most 8 / 2^16 too large, relative to 1 / gqa >= 1 / 8).
__device__ __forceinline__ int token_of(const ExtendParams& p, int row) { return row * p.gqa_inverse >> 16; }

// The exponent of the weights of a row with reference m (finite): S c + b, for
// logits S c0. Logits may reach 2^126, and b rounds where m c0 is large; what
// counts is that P at the reference, 2^(m c + b), is a small power of two, and
// that it is known. Up to 2^28 it is: b is off by half its last place, 8 at
// most, so m c + b is in [-1, 15]. From there on neighbouring values of S are
// 16 or more apart in logits, which carry S's 24 bits and no more, so c may be
// another factor as long as neighbours stay far apart: the power of two that
// takes m c to [2^29, 2^30), and b = -m c is exact.
// (Subtracting m from each S instead costs 346 us where this takes 336, for
// chunks of 2 x 2048 at 8192.)
__device__ __forceinline__ void extend_exponent(float m, float c0, float& c, float& b) {
  c = c0;
  b = fmaf(-m, c0, kExtOffset);
  if (fabsf(m) * c0 >= 268435456.f) {
    c = exp2_int(29 - (int)((__float_as_uint(m) >> 23 & 255u) - 127u));
    b = -m * c;
  }
}

// ------------------------------------------------- tensor core primitives

__device__ __forceinline__ void tmem_alloc(uint32_t smem_dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns));
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// Arrives on `bar` once every product this warp's elected lane has issued is done.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}

// f16 x f16 -> fp32 instruction descriptor, M = N = 128, both operands K-major.
constexpr uint32_t kExtIdesc = (1u << 4) | ((128u >> 3) << 17) | ((128u >> 4) << 24);

// Descriptor of a K-major operand without swizzle: core matrices of 8 rows x
// 16 bytes, the next 16-byte column kExtColumn on (low word), the next 8 rows
// 128 bytes on (high word). The products of a tile walk the low word.
__device__ __forceinline__ uint32_t operand_desc_lo(uint32_t addr) { return (addr >> 4) | ((kExtColumn >> 4) << 16); }
constexpr uint32_t kExtDescHi = (128u >> 4) | (1u << 14);
constexpr uint32_t kExtDescStep = (2u * kExtColumn) >> 4;   // 16 elements of the summed dimension
// One tile's product, eight instructions of 16 elements of the summed
// dimension each, issued by the warp's elected lane (all lanes call). One
// block of assembly, so that the descriptors are made by adding constants:
// with the instructions issued one by one the issue took longer than the
// products.
#define PDA_MMA_SS(k)                                                                         \
  "add.u32 x, %1, " #k "*256;\n\tadd.u32 y, %2, " #k "*256;\n\tmov.b64 a, {x, %5};\n\t"     \
  "mov.b64 b, {y, %5};\n\t@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, q;\n\t"
#define PDA_MMA_TS(k)                                                                         \
  "add.u32 x, %1, " #k "*8;\n\tadd.u32 y, %2, " #k "*256;\n\tmov.b64 b, {y, %5};\n\t"       \
  "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %3, q;\n\t"
// d = A B^T, both operands' tiles in shared memory.
__device__ __forceinline__ void mma_tile_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo) {
  static_assert(kExtDescStep == 256u, "descriptor step of PDA_MMA_SS and PDA_MMA_TS");
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 a, b;\n\t.reg .b32 x, y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t" PDA_MMA_SS(1) PDA_MMA_SS(2) PDA_MMA_SS(3)
          PDA_MMA_SS(4) PDA_MMA_SS(5) PDA_MMA_SS(6) PDA_MMA_SS(7) "}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(kExtIdesc), "r"(0u), "r"(kExtDescHi)
      : "memory");
}
// d (+)= A B^T over half the summed dimension, A in tensor memory.
__device__ __forceinline__ void mma_half_ts(uint32_t d, uint32_t a, uint32_t b_lo, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 b;\n\t.reg .b32 x, y;\n\t"
      "elect.sync _|e, 0xffffffff;\n\tsetp.ne.u32 p, %4, 0;\n\tsetp.eq.u32 q, 0, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t" PDA_MMA_TS(1) PDA_MMA_TS(2) PDA_MMA_TS(3)
      "}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(kExtIdesc), "r"(add ? 1u : 0u), "r"(kExtDescHi)
      : "memory");
}

#define PDA_R8(x, i) "=r"(x[i]), "=r"(x[i + 1]), "=r"(x[i + 2]), "=r"(x[i + 3]), "=r"(x[i + 4]), "=r"(x[i + 5]), \
      "=r"(x[i + 6]), "=r"(x[i + 7])
#define PDA_W8(x, i) "r"(x[i]), "r"(x[i + 1]), "r"(x[i + 2]), "r"(x[i + 3]), "r"(x[i + 4]), "r"(x[i + 5]), \
      "r"(x[i + 6]), "r"(x[i + 7])
// 32 columns of this warp's 32 lanes <-> 32 registers per lane.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : PDA_R8(x, 0), PDA_R8(x, 8), PDA_R8(x, 16), PDA_R8(x, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      PDA_W8(x, 0), PDA_W8(x, 8), PDA_W8(x, 16), PDA_W8(x, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* x) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : PDA_R8(x, 0), PDA_R8(x, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      PDA_W8(x, 0), PDA_W8(x, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// 16 e4m3 bytes -> 16 f16 (two 16-byte columns' worth), exact.
__device__ __forceinline__ void e4m3x16_to_f16(const uint4& x, uint4& lo, uint4& hi) {
  lo = make_uint4(e4m3x2_lo_to_f16x2(x.x), e4m3x2_hi_to_f16x2(x.x), e4m3x2_lo_to_f16x2(x.y), e4m3x2_hi_to_f16x2(x.y));
  hi = make_uint4(e4m3x2_lo_to_f16x2(x.z), e4m3x2_hi_to_f16x2(x.z), e4m3x2_lo_to_f16x2(x.w), e4m3x2_hi_to_f16x2(x.w));
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}
// 16 bytes from p, or zeros where `in` is false, without a branch.
__device__ __forceinline__ uint4 ld_nc_v4_if(const void* p, bool in) {
  uint4 r;
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@q ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
      : "=&r"(r.x), "=&r"(r.y), "=&r"(r.z), "=&r"(r.w)
      : "l"(p), "r"((uint32_t)in));
  return r;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A work item: a tile of query rows, a kv head and a share of the KV range.
// Tiles of 128 tokens [j0, j1) hold what block A's and B's rows attend to.
struct __align__(16) ExtendItem {
  int more;                     // 0: no further item; 1: one; 2 + i: a piece of tail item i
  int seq, row0, rows;          // first query row (token) in the packing; rows (token, head) of the tile
  int pos0;                     // position of the first token
  int kv_lo, kv_hi;             // tokens some row attends to
  int j0a, j1a, j0b, j1b;
  int jmin, jmax;
  int both;                     // both blocks hold the same rows
  int kvh, split;               // split | splits << 8 of the KV range
};
static_assert(sizeof(ExtendItem) == 64, "one slot");

// The sequence of a tile slot, and the slot's first token in it. Sequence s
// starts at slot starts[s] / tile_tokens + s, which leaves each sequence room
// for its tiles whatever the lengths are; `first` is past its rows where the
// slot is spare. The whole warp searches, probing 32 sequences at a time.
__device__ __forceinline__ int2 extend_slot(const ExtendParams& p, int slot) {
  const int lane = threadIdx.x & 31;
  const int base = __ldg(p.query_starts);
  auto first_slot = [&](int s) { return (__ldg(p.query_starts + s) - base) / p.tile_tokens + s; };
  int s = 0;
  for (int n = p.num_seqs; n > 1;) {
    const int step = (n + 31) / 32, probe = lane * step;
    const unsigned hit = __ballot_sync(0xffffffffu, probe < n && first_slot(s + probe) <= slot);
    const int k = hit ? (31 - __clz(hit)) * step : 0;
    s += k;
    n = min(step, n - k);
  }
  return make_int2(s, (slot - first_slot(s)) * p.tile_tokens);
}

// Describes the tile of sequence s from token `first` on (t.more, t.kvh and
// t.split are set); false where it has no rows.
__device__ __forceinline__ bool extend_item(const ExtendParams& p, int s, int first, int start, int end, int len0,
                                            ExtendItem& t) {
  start = max(0, min(start, p.num_tokens));
  end = max(start, min(end, p.num_tokens));
  const int n = end - start;
  if (first < 0 || first >= n) return false;
  const int tokens = min(p.tile_tokens, n - first);
  const int len = (int)max(0ll, min((long long)len0, (long long)p.max_blocks * p.block_size));
  t.seq = s;
  t.row0 = start + first;
  t.rows = tokens * p.gqa;
  t.pos0 = len - n + first;
  t.both = t.rows <= kExtRows;
  t.kv_lo = p.window > 0 ? max(0, t.pos0 - p.window + 1) : 0;
  t.kv_hi = max(0, t.pos0 + tokens);
  // tiles of the block of tokens [t0, t1)
  auto tiles_of = [&](int t0, int t1, int& j0, int& j1) {
    const int p0 = t.pos0 + t0, p1 = t.pos0 + t1;
    j0 = (p.window > 0 ? max(0, p0 - p.window + 1) : 0) / kExtTile;
    j1 = p1 > 0 && t1 > t0 ? (p1 - 1) / kExtTile + 1 : j0;
  };
  tiles_of(0, t.both ? tokens : min(tokens, (kExtRows - 1) / p.gqa + 1), t.j0a, t.j1a);
  tiles_of(t.both ? 0 : kExtRows / p.gqa, tokens, t.j0b, t.j1b);
  t.jmin = t.j0a;
  t.jmax = max(t.j1a, t.j1b);
  if (const int splits = t.split >> 8; splits > 1) {
    const int per = (t.jmax - t.jmin + splits - 1) / splits;
    const int a = t.jmin + (t.split & 255) * per, b = min(t.jmax, a + per);
    t.jmin = min(a, t.jmax);
    t.jmax = max(t.jmin, b);
    t.j0a = max(t.j0a, t.jmin), t.j1a = max(t.j0a, min(t.j1a, t.jmax));
    t.j0b = max(t.j0b, t.jmin), t.j1b = max(t.j0b, min(t.j1b, t.jmax));
  }
  return true;
}

__device__ __forceinline__ bool extend_item(const ExtendParams& p, int s, int first, ExtendItem& t) {
  return extend_item(p, s, first, __ldg(p.query_starts + s), __ldg(p.query_starts + s + 1), __ldg(p.seq_lens + s), t);
}

// The tiles block x takes: j0, j0 + step, ... below j1.
__device__ __forceinline__ void block_tiles(const ExtendItem& t, int x, int& j0, int& j1, int& step) {
  j0 = (x ? t.j0b : t.j0a) + (t.both ? x : 0);
  j1 = x ? t.j1b : t.j1a;
  step = t.both ? 2 : 1;
  if (j0 > j1) j0 = j1;
}

// Persistent: one CTA per SM works through items; every role goes from one
// item to the next by itself, so K and V of the next item arrive, and its
// queries, under the end of this one.
__global__ void __launch_bounds__(kExtThreads, 1) pda_extend_kernel(const ExtendParams p) {
  extern __shared__ __align__(1024) uint8_t ext_smem[];
  uint8_t* const smem = ext_smem;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sm = smem_u32(smem);
  const uint32_t bars = sm + kExtBarOff;
  auto bar = [&](int i) { return bars + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + kExtMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kExtMiscOff + 4);
  if (tid == 0) {
    *abort_flag = 0;
    for (int i = 0; i < kExtSlots; ++i) mbar_init(bar(kBarItemFull + i), 1), mbar_init(bar(kBarItemFree + i), 14);
    for (int i = 0; i < 2 * kExtSlots; ++i) mbar_init(bar(kBarQ + i), 4);
    for (int i = 0; i < 2; ++i) mbar_init(bar(kBarKFull + i), 4), mbar_init(bar(kBarKFree + i), 2);
    for (int i = 0; i < 3; ++i) mbar_init(bar(kBarVFull + i), 4), mbar_init(bar(kBarVFree + i), 2);
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar(kBarS + x), 1);
      mbar_init(bar(kBarP + 2 * x), 4);
      mbar_init(bar(kBarP + 2 * x + 1), 4);
      mbar_init(bar(kBarO + x), 1);
      mbar_init(bar(kBarTurn + x), 1);
    }
    mbar_init(bar(kBarSums), 8);
    mbar_init(bar(kBarJoined), 8);
    mbar_init(bar(kBarAhead), 4);
    fence_barrier_init();
  }
  // Up to 32 sequences: the scheduling warp holds their starts and lengths,
  // asked for while the CTA sets itself up.
  const bool few = p.num_seqs <= 32;
  int my_start = 0, my_end = 0, my_len = 0;
  if (warp == 14 && few) {
    const int s = min(lane, p.num_seqs - 1);
    my_start = __ldg(p.query_starts + s);
    my_end = __ldg(p.query_starts + s + 1);
    my_len = __ldg(p.seq_lens + s);
  }
  if (warp == 12) tmem_alloc(sm + kExtMiscOff, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Bounded: a wait that gives up records it and sends every role to the end.
  // The whole warp calls; the common case is the first line alone.
  auto warp_wait = [&](int i, uint32_t parity) -> bool {
    if (__builtin_expect(__all_sync(0xffffffffu, mbar_try_wait(bar(i), parity)), 1)) return true;
    const bool got = mbar_wait_bounded(bar(i), parity, const_cast<volatile int*>(abort_flag), kWaitLimitNs);
    if (!got) {
      if (!*abort_flag) atomicOr(&g_status, kStatusFullWaitTimeout);
      *abort_flag = 1;
    }
    return __all_sync(0xffffffffu, got) != 0;
  };
  auto read_item = [&](int it, ExtendItem& t) {
    const uint32_t src = sm + kExtItemOff + (uint32_t)(it % kExtSlots) * 64u;
    int4* dst = reinterpret_cast<int4*>(&t);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm volatile("ld.shared.v4.s32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(dst[i].x), "=r"(dst[i].y), "=r"(dst[i].z), "=r"(dst[i].w)
                   : "r"(src + 16u * i));
  };
  // Lets the slot go once the four loads have delivered: an arrival can
  // overtake loads that still stand in the shared-memory queue, but not where
  // its address depends on their results.
  auto release_item = [&](int it, const ExtendItem& t) {
    const uint32_t z = (uint32_t)(t.more | t.pos0 | t.j1a | t.split) & p.zero;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarItemFree + it % kExtSlots) + z);
  };
  // Item number it, or false at the end (or on abort).
  auto next_item = [&](int it, ExtendItem& t) -> bool {
    if (!warp_wait(kBarItemFull + it % kExtSlots, (uint32_t)(it / kExtSlots) & 1u)) return false;
    read_item(it, t);
    return t.more != 0;
  };

  if (warp < 8) {
    regs_inc<kExtSoftmaxRegs>();
    // ---------------------------------------------------------- softmax
    const int x = warp >> 2;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;        // lane 32 * (warp mod 4) in bits 16..
    const uint32_t s_addr = tmem + lanes + (uint32_t)x * 128u;
    const uint32_t o_addr = s_addr + 256u;
    // the warp's 32 rows of its block's query tile
    const uint32_t own = sm + kExtQOff + (uint32_t)x * kExtOperand + (uint32_t)(warp & 3) * 512u;
    float2* sums = reinterpret_cast<float2*>(smem + kExtSumsOff);   // [block][row]: reference, l
    uint32_t s_phase = 0, o_phase = 0, join_phase = 0;
    bool ok = true;
    ExtendItem t;
#pragma unroll 1
    for (int it = 0; ok && next_item(it, t); ++it) {
      const int row = t.both ? (tid & 127) : tid;             // of the tile
      const int tok = token_of(p, row);
      const bool live = row < t.rows;
      // The row's queries: shifted by a power of two into f16 (its largest |q|
      // in [2^14, 2^15)), stored as this row of the A operand. The products
      // that read the last item's are complete: its O has been waited for.
      // Lanes are 8 rows x 4 pieces of 16 bytes: a load touches 8 rows' 64
      // bytes instead of 32 rows' 16 (an eighth of the cache lines per load of
      // a row per lane), and 8 lanes' stores to one column have no conflicts.
      float c = 0.f;
      {
        const int r8 = lane & 7, piece = lane >> 3;
        const int wrow = (t.both ? (tid & 96) : tid & ~31);    // the warp's first row
        uint4 vv[4][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = wrow + 8 * q + r8, rt = token_of(p, r);
          const uint4* src = reinterpret_cast<const uint4*>(
              p.q + ((size_t)(t.row0 + rt) * p.num_heads + t.kvh * p.gqa + r - rt * p.gqa) * kHeadDim) + piece;
#pragma unroll
          for (int i = 0; i < 4; ++i) vv[q][i] = r < t.rows ? __ldg(src + 4 * i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint4(&v)[4] = vv[q];
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mx = __vmaxu2(mx, v[i].x & 0x7FFF7FFFu);
            mx = __vmaxu2(mx, v[i].y & 0x7FFF7FFFu);
            mx = __vmaxu2(mx, v[i].z & 0x7FFF7FFFu);
            mx = __vmaxu2(mx, v[i].w & 0x7FFF7FFFu);
          }
          mx = max(mx & 0xFFFFu, mx >> 16);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
          const int e = mx == 0u ? 0 : min(max((int)(mx >> 7) - 127 - 14, -100), 113);
          const float down = p.negate ? -exp2_int(-e) : exp2_int(-e);
          // row `lane` of the warp is this thread's own
          if (piece == q) c = fmaxf(p.logit_scale_log2 * exp2_int(e), 1.17549435e-38f);
          if (x == 0 || !t.both) {
            const uint32_t dst = own + (uint32_t)(8 * q + r8) * 16u + (uint32_t)piece * kExtColumn;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              st_shared_v4(dst + (uint32_t)(4 * i) * kExtColumn,
                           make_uint4(pack_f16x2(bf16lo_f32(v[i].x) * down, bf16hi_f32(v[i].x) * down),
                                      pack_f16x2(bf16lo_f32(v[i].y) * down, bf16hi_f32(v[i].y) * down),
                                      pack_f16x2(bf16lo_f32(v[i].z) * down, bf16hi_f32(v[i].z) * down),
                                      pack_f16x2(bf16lo_f32(v[i].w) * down, bf16hi_f32(v[i].w) * down)));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQ + 2 * (it % kExtSlots) + x));
      }
      const int hi = live ? t.pos0 + tok : -1;                // last token of the row
      const int lo = p.window > 0 ? max(0, hi - p.window + 1) : 0;
      // tiles inside [in_lo, in_hi] need no mask for any live row of the block
      const int last_row = min(t.rows, t.both ? kExtRows : (x + 1) * kExtRows) - 1;
      const int first_row = t.both ? 0 : x * kExtRows;
      const int in_hi = t.pos0 + token_of(p, first_row);
      const int in_lo = p.window > 0 ? t.pos0 + token_of(p, last_row) - p.window + 1 : 0;
      int j, j1, step;
      block_tiles(t, x, j, j1, step);
      const bool any = j < j1;
      float m = -INFINITY, l = 0.f;
      const float c0 = c;
      float b = 3e38f;                                        // no reference yet: any logit is past the limit
      bool first = true;
      const bool idle = (row & ~31) >= t.rows;                // no row of the warp is live
#pragma unroll 1
      for (; j < j1; j += step, first = false) {
        if (!warp_wait(kBarS + x, s_phase)) {
          ok = false;
          break;
        }
        s_phase ^= 1;
        if (idle) {
          // rows of P that are nobody's may hold anything: they reach their own rows of O alone
          if (lane < 2) mbar_arrive(bar(kBarP + 2 * x + lane));
          continue;
        }
        tc_fence_after();
        const int t0 = j * kExtTile;
        uint32_t s[128];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32(s_addr + 32u * q, s + 32 * q);
        tmem_wait_ld();
        if (t0 < in_lo || t0 + kExtTile - 1 > in_hi) {
          const int first_c = lo - t0, last_c = hi - t0;
#pragma unroll
          for (int i = 0; i < 128; ++i)
            if (i < first_c || i > last_c) s[i] = 0xFF800000u;   // -inf
        }
        float mx[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx[i] = __uint_as_float(s[i]);
#pragma unroll
        for (int i = 4; i < 128; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = i + k + 4 < 128 ? fmaxf(mx[k], fmaxf(__uint_as_float(s[i + k]), __uint_as_float(s[(i + k + 4) & 127])))
                                    : fmaxf(mx[k], __uint_as_float(s[i + k]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool grow = fmaf(top, c, b) > kExtLimit;     // no reference yet: at the row's first visible token
        if (__any_sync(0xffffffffu, grow)) {
          float f = 1.f;
          if (grow) {
            const float was = m == -INFINITY ? 0.f : fmaf(m, c, b);   // log2 of P at the reference
            extend_exponent(top, c0, c, b);
            if (m != -INFINITY) f = fast_exp2((m - top) * c0 + (fmaf(top, c, b) - was));
            m = top;
          }
          // O holds earlier tiles' sums (their product is complete: S was issued after it)
          if (!first && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              uint32_t o[16];
              tmem_ld16(o_addr + 16u * i, o);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(o_addr + 16u * i, o);
            }
          }
          l *= f;
        }
        const uint64_t cc = pack_f32x2(c, c), bb = pack_f32x2(b, b);
        uint64_t s0 = 0, s1 = 0;                         // two fp32 sums each
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t* w = s + 64 * h + 2 * i;
            const float2 z = unpack_f32x2(
                fma_f32x2(pack_f32x2(__uint_as_float(w[0]), __uint_as_float(w[1])), cc, bb));
            const float pa = fast_exp2(z.x), pe = fast_exp2(z.y);
            if (i & 1)
              s1 = add_f32x2(s1, pack_f32x2(pa, pe));
            else
              s0 = add_f32x2(s0, pack_f32x2(pa, pe));
            pk[i] = pack_f16x2(pa, pe);
          }
          tmem_st32(s_addr + 32u * h, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kBarP + 2 * x + h));   // its product starts under the other half's weights
        }
        const float2 both_sums = unpack_f32x2(add_f32x2(s0, s1));
        l += both_sums.x + both_sums.y;
      }
      // -------------------------------------------------------- output
      if (any && ok) {
        ok = warp_wait(kBarO + x, o_phase);
        o_phase ^= 1;
      }
      if (!ok) break;
      tc_fence_after();
      // read again rather than held in registers through the tiles
      read_item(it, t);
      release_item(it, t);
      const int row2 = t.both ? (tid & 127) : tid, tok2 = token_of(p, row2);
      const bool live2 = row2 < t.rows;
      const int head2 = t.kvh * p.gqa + row2 - tok2 * p.gqa;
      const size_t orow2 = (size_t)(t.row0 + tok2) * p.num_heads + head2;
      // factors of this block's O and the other's, which take P at the reference to 1
      float top = m, den = l, fa = m == -INFINITY ? 0.f : fast_exp2(-fmaf(m, c, b)), fb = 0.f;
      if (t.both) {
        // Both blocks hold the rows: they exchange (m, l), and each reads
        // half the columns of both O's.
        sums[x * 128 + row2] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarSums));
        if (!warp_wait(kBarSums, join_phase)) break;
        const float2 o = sums[(1 - x) * 128 + row2];
        top = fmaxf(m, o.x);
        if (m != -INFINITY) fa *= fast_exp2((m - top) * c0);
        if (o.x != -INFINITY) {
          float co, bo;
          extend_exponent(o.x, c0, co, bo);
          fb = fast_exp2((o.x - top) * c0 - fmaf(o.x, co, bo));
        }
        den = l * fa + o.y * fb;
        tc_fence_after();
      } else {
        den *= fa;
      }
      const float M = top * c0;                                 // the reference in logits
      // Splits leave (O, reference, l): of a row of the call, or of the tail item's
      const int split = t.split & 255, splits = t.split >> 8;
      const bool partial = splits > 1;
      const size_t prow =
          (t.more >= 2 ? (size_t)(t.more - 2) * (2 * kExtRows) + row2 : orow2) * splits + split;
      if (!partial) {
        const float zs = p.sinks && live2 ? __ldg(p.sinks + head2) * 1.4426950408889634f : -INFINITY;
        const float r = live2 && t.pos0 + tok2 >= 0 ? finish(1.f, den, M, zs, p.v_scale) : 0.f;
        fa *= r;
        fb *= r;
      } else if (live2 && (x == 0 || !t.both)) {
        *reinterpret_cast<float2*>((t.more >= 2 ? p.tail_ml : p.part_ml) + prow * 2) = make_float2(M, den);
      }
      const int i0 = t.both ? 4 * x : 0, i1 = t.both ? 4 * x + 4 : 8;
#pragma unroll 1
      for (int i = i0; i < i1; ++i) {
        uint32_t o[16], u[16];
        __syncwarp();
        tmem_ld16(o_addr + 16u * i, o);
        if (t.both) tmem_ld16((o_addr ^ 128u) + 16u * i, u);
        tmem_wait_ld();
        float r[16];
        // a factor of 0: that block saw nothing, and its O may be anything
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          r[k] = fa != 0.f ? __uint_as_float(o[k]) * fa : 0.f;
          if (t.both && fb != 0.f) r[k] += __uint_as_float(u[k]) * fb;
        }
        if (partial) {
          if (live2) {
            float4* dst = reinterpret_cast<float4*>((t.more >= 2 ? p.tail_o : p.part_o) + prow * kHeadDim + 16 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) dst[k] = make_float4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
          }
        } else if (p.out_fp8) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            w[k] = f32x2_to_e4m3x2(__fdiv_rn(r[4 * k], p.out_scale), __fdiv_rn(r[4 * k + 1], p.out_scale)) |
                   (f32x2_to_e4m3x2(__fdiv_rn(r[4 * k + 2], p.out_scale), __fdiv_rn(r[4 * k + 3], p.out_scale)) << 16);
          st_shared_v4(own + lane * 16u + (uint32_t)i * kExtColumn, make_uint4(w[0], w[1], w[2], w[3]));
        } else {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[k]) : "f"(r[2 * k + 1]), "f"(r[2 * k]));
          st_shared_v4(own + lane * 16u + (uint32_t)(2 * i) * kExtColumn, make_uint4(w[0], w[1], w[2], w[3]));
          st_shared_v4(own + lane * 16u + (uint32_t)(2 * i + 1) * kExtColumn, make_uint4(w[4], w[5], w[6], w[7]));
        }
      }
      if (!partial) {
        // The rows went to the warp's own part of the query tile, a 16-byte
        // column apart (its products are done), and leave from there 8 rows x
        // 64 bytes at a time, as the queries came.
        __syncwarp();
        const int r8 = lane & 7, piece = lane >> 3;
        const int wrow = (t.both ? (tid & 96) : tid & ~31);
        const int cols = p.out_fp8 ? 8 : 16;
        const int c0 = t.both ? cols / 2 * x : 0, c1 = t.both ? c0 + cols / 2 : cols;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          const int rr = wrow + 8 * q + r8, rt = token_of(p, rr);
          if (rr < t.rows) {
            uint8_t* dst = static_cast<uint8_t*>(p.out) +
                           ((size_t)(t.row0 + rt) * p.num_heads + t.kvh * p.gqa + rr - rt * p.gqa) * (size_t)(cols * 16);
            for (int k = c0 + piece; k < c1; k += 4)
              *reinterpret_cast<uint4*>(dst + k * 16) =
                  ld_shared_v4(own + (uint32_t)(8 * q + r8) * 16u + (uint32_t)k * kExtColumn);
          }
        }
      }
      __syncwarp();
      tc_fence_before();
      if (t.both) {
        // the next item's products may overwrite O, and its queries Q, once both blocks are here
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarJoined));
        if (!warp_wait(kBarJoined, join_phase)) break;
        join_phase ^= 1;
        tc_fence_after();
      }
    }
  } else if (warp < 12) {
    regs_dec<kExtConvertRegs>();
    // ------------------------------------------------- K and V to f16
    const int me = tid & 127;                                 // token of the tile (K), dim (V)
    const uint32_t bs = (uint32_t)p.block_size;
    const uint32_t per_page = bs / 16u;                       // 16-token units of a page
    // Zeroes the tokens of 16 in front of kv_lo, at or behind kv_hi.
    auto clip = [&](uint4& x, int ti, int kv_lo, int kv_hi) {
      const int a = kv_lo - ti, b = kv_hi - ti;
      if (a <= 0 && b >= 16) return;
      auto below = [](int n) { return n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u); };
      x.x &= below(b) & ~below(a);
      x.y &= below(b - 4) & ~below(a - 4);
      x.z &= below(b - 8) & ~below(a - 8);
      x.w &= below(b - 12) & ~below(a - 12);
    };
    auto store = [&](const uint4 (&x)[8], uint32_t dst) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint4 a, b;
        e4m3x16_to_f16(x[i], a, b);
        st_shared_v4(dst + (uint32_t)(2 * i) * kExtColumn, a);
        st_shared_v4(dst + (uint32_t)(2 * i + 1) * kExtColumn, b);
      }
    };
    auto signal = [&](int b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(b));
    };
    bool ok = true;
    ExtendItem t;
    // 16-byte loads through the block table, a tile ahead: K: the 8 chunks
    // of 16 dims of a token; V: the 8 units of 16 tokens of a dim. What no
    // row attends to is not read: zeros stand in (a masked weight of 0
    // times a NaN would be NaN).
    const uint32_t magic = per_page == 1 ? 0u : 0xFFFFFFFFu / per_page + 1u;
    auto page_of = [&](uint32_t unit) { return per_page == 1 ? unit : __umulhi(unit, magic); };
    const uint32_t block_bytes = (uint32_t)kHeadDim * bs * (uint32_t)p.num_kv_heads;   // < 2^31: bs <= 128, 65535 heads
    const uint32_t unit_bytes = p.v_shuffled ? kHeadDim * 16u : 16u;   // V: from a page's unit to the next
    auto checked = [&](int id) { return p.block_limit ? checked_block(id, p.block_limit) : id; };
    uint32_t n = 0;                                         // tiles so far
    uint4 k[8], v[8];
    int k_id = -1, v_id[8];
#pragma unroll 1
    for (int it = 0; ok && next_item(it, t); ++it) {
      release_item(it, t);
      const int kv_lo = t.kv_lo, kv_hi = t.kv_hi, jmin = t.jmin, jmax = t.jmax;
      const int near = max(jmin, jmax - kExtAhead);
      const int32_t* table = p.block_tables + (size_t)t.seq * p.max_blocks;
      const uint8_t* k_cache = p.k_cache + (size_t)t.kvh * kHeadDim * bs;
      const uint8_t* v_cache = p.v_cache + (size_t)t.kvh * kHeadDim * bs + (uint32_t)me * (p.v_shuffled ? 16u : bs);
      // Block ids, two tiles ahead: lane i mod 8 has unit i's page. They are
      // handed round (K: the unit of the thread's token; V: all) in front of a
      // tile's stores: shuffles stand in the shared-memory queue too, and
      // behind the stores they would wait for all of them. (A load of every id
      // by every thread took 400 to 1400 cycles a tile to issue.)
      auto look_up = [&](int j) -> int {
        const int tk = j * kExtTile + 16 * (lane & 7);
        return tk + 16 > kv_lo && tk < kv_hi ? checked(__ldg(table + page_of((uint32_t)tk >> 4))) : -1;
      };
      auto hand_round = [&](int ids, int j) {
        const int tk = j * kExtTile + me;
        k_id = __shfl_sync(0xffffffffu, ids, me >> 4);
        if (tk < kv_lo || tk >= kv_hi) k_id = -1;
#pragma unroll
        for (int i = 0; i < 8; ++i) v_id[i] = __shfl_sync(0xffffffffu, ids, i);
      };
      auto load_k = [&](int j) {
        const uint32_t tk = (uint32_t)(j * kExtTile + me);
        const uint8_t* src = k_cache + ((uint64_t)(uint32_t)k_id * block_bytes + (tk - page_of(tk >> 4) * bs) * 16u);
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = ld_nc_v4_if(src + i * bs * 16u, k_id != -1);
      };
      auto load_v = [&](int j) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t unit = (uint32_t)(j * (kExtTile / 16) + i);
          v[i] = ld_nc_v4_if(v_cache + ((uint64_t)(uint32_t)v_id[i] * block_bytes +
                                        (unit - page_of(unit) * per_page) * unit_bytes),
                             v_id[i] != -1);
        }
      };
      int ids = -1;                                           // of tile j + 1
      if (jmin < jmax) {
        hand_round(look_up(jmin), jmin);
        load_k(jmin);
        load_v(jmin);
        if (jmin + 1 < jmax) ids = look_up(jmin + 1);
      } else {
        signal(kBarAhead);
      }
#pragma unroll 1
      for (int j = jmin; j < jmax; ++j, ++n) {
        if (j == near) signal(kBarAhead);
        const bool more = j + 1 < jmax;
        hand_round(ids, j + 1);
        if (j + 2 < jmax) ids = look_up(j + 2);
        uint32_t st = n % kExtKStages;
        if (n >= kExtKStages) ok = warp_wait(kBarKFree + (int)st, (n / kExtKStages - 1u) & 1u);
        if (!ok) break;
        store(k, sm + kExtKOff + st * kExtOperand + (uint32_t)me * 16u);
        if (more) load_k(j + 1);
        fence_async_smem();
        signal(kBarKFull + (int)st);
        st = n % kExtVStages;
        if (n >= kExtVStages) ok = warp_wait(kBarVFree + (int)st, (n / kExtVStages - 1u) & 1u);
        if (!ok) break;
        if (j * kExtTile < kv_lo || (j + 1) * kExtTile > kv_hi) {
#pragma unroll
          for (int i = 0; i < 8; ++i) clip(v[i], j * kExtTile + 16 * i, kv_lo, kv_hi);
        }
        store(v, sm + kExtVOff + st * kExtOperand + (uint32_t)me * 16u);
        if (more) load_v(j + 1);
        fence_async_smem();
        signal(kBarVFull + (int)st);
      }
    }
  } else {
    regs_dec<kExtIssueRegs>();
    const int x = __shfl_sync(0xffffffffu, warp - 12, 0);    // uniform, for the compiler too
    if (x < 2) {
      // ---------------------------------------------- the products
      const uint32_t s_tm = tmem + (uint32_t)x * 128u, o_tm = s_tm + 256u;
      uint32_t s_count = 0;     // S products so far: P's phases
      uint32_t n0 = 0;          // tiles of earlier items: the rings' phases
      uint32_t turn = 0;        // turns so far
      bool ok = true;
      ExtendItem t;
#pragma unroll 1
      for (int it = 0; ok && next_item(it, t); ++it) {
        int j0, j1, step;
        block_tiles(t, x, j0, j1, step);
        const uint32_t qd = operand_desc_lo(sm + kExtQOff + (t.both ? 0u : (uint32_t)x * kExtOperand));
        int prev = -1;          // tile (from jmin) whose P V is due
        bool started = false;   // O holds something
        const int tiles = t.jmax - t.jmin;
        // The slot is let go of behind these waits: a softmax group whose block
        // has no tiles goes on without the products, but it can store the
        // queries of the slot's next item only once this one's have been seen.
        const int q_bar = kBarQ + 2 * (it % kExtSlots);
        const uint32_t q_phase = (uint32_t)(it / kExtSlots) & 1u;
        ok = warp_wait(q_bar + x, q_phase);
        if (ok && t.both && x) ok = warp_wait(q_bar, q_phase);
        if (!ok) break;
        release_item(it, t);
#pragma unroll 1
        for (int i = 0; ok && i <= tiles; ++i) {             // the last round: what is left
          const int j = t.jmin + i;
          const bool mine = i < tiles && j >= j0 && j < j1 && (step == 1 || ((j - j0) & 1) == 0);
          const bool due = prev >= 0 && (mine || j >= j1);
          const uint32_t n = n0 + (uint32_t)i, np = n0 + (uint32_t)prev;
          const uint32_t ks = n % kExtKStages, vs = np % kExtVStages;
          if (due) ok = warp_wait(kBarVFull + vs, (np / kExtVStages) & 1u);
          if (ok && mine) ok = warp_wait(kBarKFull + ks, (n / kExtKStages) & 1u);
          // The blocks issue in turn. Left to themselves they fall into step:
          // both wait for both products, then both are in their softmax.
          const bool turns = step == 1 && i < tiles;
          if (ok && turns && (x || turn)) ok = warp_wait(kBarTurn + x, (x ? turn : turn - 1u) & 1u);
          const uint32_t p_phase = (s_count - 1u) & 1u;
          const uint32_t vd = operand_desc_lo(sm + kExtVOff + vs * kExtOperand);
          if (ok && due && (ok = warp_wait(kBarP + 2 * x, p_phase))) {
            tc_fence_after();
            mma_half_ts(o_tm, s_tm, vd, started);
          }
          if (ok && due) ok = warp_wait(kBarP + 2 * x + 1, p_phase);
          if (!ok) break;
          tc_fence_after();
          if (due) {
            mma_half_ts(o_tm, s_tm + 32u, vd + 4u * kExtDescStep, true);
            tc_commit(bar(kBarVFree + vs));
            if (!mine) tc_commit(bar(kBarO + x));
            started = true;
            prev = -1;
          }
          if (mine) {
            mma_tile_ss(s_tm, qd, operand_desc_lo(sm + kExtKOff + ks * kExtOperand));
            tc_commit(bar(kBarS + x));
            tc_commit(bar(kBarKFree + ks));
            prev = i;
            ++s_count;
          }
          if (turns) {
            if (lane == 0) mbar_arrive(bar(kBarTurn + 1 - x));
            ++turn;
          }
          if (!mine && i < tiles) {
            // the other block's tile: a stage is free when both have let go of it
            const uint32_t v2 = n % kExtVStages;
            ok = warp_wait(kBarKFull + ks, (n / kExtKStages) & 1u);
            if (ok && lane == 0) mbar_arrive(bar(kBarKFree + ks));
            ok = ok && warp_wait(kBarVFull + v2, (n / kExtVStages) & 1u);
            if (ok && lane == 0) mbar_arrive(bar(kBarVFree + v2));
          }
        }
        n0 += (uint32_t)tiles;
      }
    } else if (x == 2) {
      // ---------------------------------------------- the next items
      // The order comes from the kernel in front, which this one does not
      // wait for as a whole.
      if (p.order) grid_dependency_wait();
      const unsigned heads = (unsigned)p.num_kv_heads;
      ExtendHead head = {p.tiles, 0, 0, 1};
      if (p.order) head = *reinterpret_cast<const ExtendHead*>(p.head);
      else head.whole = (int)((unsigned)p.tiles * heads * (unsigned)p.nsplit);
      const unsigned total = (unsigned)head.whole + (unsigned)(head.tail * head.pieces);
      unsigned ticket = blockIdx.x;
      auto take = [&]() {
        if (p.queue) {
          if (lane == 0) ticket = gridDim.x + atomicAdd(p.queue, 1u);
          ticket = __shfl_sync(0xffffffffu, ticket, 0);
        } else {
          ticket += gridDim.x;
        }
      };
      bool ok = true;
      for (int it = 0; ok; ++it) {
        // Taken late, so that no CTA sits on an item while others are idle.
        if (it > 0 && !warp_wait(kBarAhead, (uint32_t)(it - 1) & 1u)) break;
        if (it > 0) take();
        ExtendItem t;
        bool found = false;
        while (ticket < total) {
          // heads, then splits, then tiles: CTAs that run together share
          // tables; without an order, later tiles of a sequence (which see
          // more tokens) go first
          unsigned item = ticket;
          t.more = 1;
          if (ticket >= (unsigned)head.whole) {
            const unsigned at = ticket - (unsigned)head.whole;
            item = (unsigned)head.whole + at / (unsigned)head.pieces;
            t.more = 2 + (int)(at / (unsigned)head.pieces);
            t.split = (int)(at % (unsigned)head.pieces) | head.pieces << 8;
          }
          t.kvh = (int)(item % heads);
          unsigned tile = item / heads;
          if (!p.order) {
            t.split = (int)(tile % (unsigned)p.nsplit) | p.nsplit << 8;
            tile /= (unsigned)p.nsplit;
          } else if (t.more == 1) {
            t.split = 1 << 8;
          }
          const int slot = p.tiles - 1 - (int)tile;
          int2 at;
          if (p.order) {
            at = __ldcg(p.order + tile);
          } else if (few) {
            const int first_slot = (my_start - __shfl_sync(0xffffffffu, my_start, 0)) / p.tile_tokens + lane;
            const unsigned hit = __ballot_sync(0xffffffffu, lane < p.num_seqs && first_slot <= slot);
            at.x = hit ? 31 - __clz((int)hit) : 0;
            at.y = (slot - __shfl_sync(0xffffffffu, first_slot, at.x)) * p.tile_tokens;
          } else {
            at = extend_slot(p, slot);
          }
          found = few ? extend_item(p, at.x, at.y, __shfl_sync(0xffffffffu, my_start, at.x),
                                    __shfl_sync(0xffffffffu, my_end, at.x), __shfl_sync(0xffffffffu, my_len, at.x), t)
                      : extend_item(p, at.x, at.y, t);
          if (found) break;
          take();
        }
        if (!found) t.more = 0;
        const int place = it % kExtSlots;
        if (it >= kExtSlots) ok = warp_wait(kBarItemFree + place, (uint32_t)(it / kExtSlots - 1) & 1u);
        if (!ok) break;
        if (lane == 0) {
          *reinterpret_cast<ExtendItem*>(smem + kExtItemOff + place * 64) = t;
          mbar_arrive(bar(kBarItemFull + place));
        }
        if (!t.more) break;
      }
      // the last CTA to stop taking items leaves the queue at zero
      if (p.queue && lane == 0) {
        __threadfence();
        if (atomicAdd(p.queue + 1, 1u) == gridDim.x - 1) {
          p.queue[0] = 0u;
          p.queue[1] = 0u;
        }
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 12) {
    if (*abort_flag) {
      // products still in flight end by themselves, within this time by far
      const unsigned long long t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000ull) {}
    }
    tc_fence_after();
    tmem_free(tmem, 512);
  }
}

// pda_extend_order_kernel: the tiles of a call with more work items than CTAs,
// longest KV range first (a counting sort by 128-token tiles, one block), so
// that the items that come last are short; the last, partial round of them is
// cut into pieces for the CTAs it would leave idle (pda_extend_tail_kernel joins
// them). GB300, us without either / with the order / with both: 2 x 2048
// tokens at 8192 (3.4 items a CTA) 349 / 361 / 338, 64 x 4 tokens over
// 2000-4000 152 / 157 / 152, a mixed batch of 24 sequences (6.9 items)
// 159 / 153 / 156.
constexpr int kExtOrderThreads = 1024;
constexpr int kExtMaxOrdered = 16384;                 // tile slots
constexpr int kExtMaxPieces = 4;
constexpr int kExtMinPiece = 4;                       // KV tiles
__global__ void __launch_bounds__(kExtOrderThreads) pda_extend_order_kernel(const ExtendParams p, int2* order,
                                                                            ExtendHead* head, int ctas) {
  __shared__ int hist[kExtOrderThreads], sums[32];
  grid_dependents_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  hist[tid] = 0;
  __syncthreads();
  // KV tiles of a slot (-1: spare), 1023 at most; the thread's own search
  auto size_of = [&](int slot, int2& at) -> int {
    const int base = __ldg(p.query_starts);
    int lo = 0, hi = p.num_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((__ldg(p.query_starts + mid) - base) / p.tile_tokens + mid <= slot)
        lo = mid;
      else
        hi = mid - 1;
    }
    at = make_int2(lo, (slot - ((__ldg(p.query_starts + lo) - base) / p.tile_tokens + lo)) * p.tile_tokens);
    ExtendItem t;
    t.kvh = t.split = 0;
    if (!extend_item(p, at.x, at.y, t)) return -1;
    return min(t.jmax - t.jmin, kExtOrderThreads - 1);
  };
  for (int slot = tid; slot < p.tiles; slot += kExtOrderThreads) {
    int2 at;
    const int n = size_of(slot, at);
    if (n >= 0) atomicAdd(&hist[kExtOrderThreads - 1 - n], 1);
  }
  __syncthreads();
  // exclusive prefix over the sizes, largest first
  const int mine = hist[tid];
  int x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int v = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    sums[lane] = v;
  }
  __syncthreads();
  const int before = (warp ? sums[warp - 1] : 0) + x - mine;
  hist[tid] = before;
  // The thread whose size holds the first item of the last, partial round
  // (the largest of them) cuts that round: into as many pieces as leave no
  // CTA two of them, of at least kExtMinPiece tiles for that item.
  const int tiles = sums[31];
  const int items = tiles * p.num_kv_heads;
  const int rest = items > ctas ? items % ctas : 0;
  const int cut = rest ? (items - rest) / p.num_kv_heads : 0;    // tile of that item
  if (rest ? (before <= cut && cut < before + mine) : tid == 0) {
    int n = rest ? min(ctas / rest, (kExtOrderThreads - 1 - tid) / kExtMinPiece) : 1;
    n = max(1, min(n, kExtMaxPieces));
    const int whole = n > 1 ? items - rest : items;
    *head = ExtendHead{tiles, whole, items - whole, n};
  }
  __syncthreads();
  // Scatter in slot order within a size (warp after warp, so that the same
  // state always gives the same order, and with it the same pieces).
  for (int slot0 = 0; slot0 < p.tiles; slot0 += kExtOrderThreads) {
    int2 at = make_int2(0, 0);
    const int n = slot0 + tid < p.tiles ? size_of(slot0 + tid, at) : -1;
    const unsigned peers = __match_any_sync(0xffffffffu, n);
    const int leader = __ffs((int)peers) - 1;
    int pos = 0;
#pragma unroll 1
    for (int w = 0; w < kExtOrderThreads / 32; ++w) {
      if (w == warp && n >= 0 && lane == leader) {
        pos = hist[kExtOrderThreads - 1 - n];
        hist[kExtOrderThreads - 1 - n] = pos + __popc(peers);
      }
      __syncthreads();
    }
    pos = __shfl_sync(0xffffffffu, pos, leader) + __popc(peers & ((1u << lane) - 1u));
    if (n >= 0) order[pos] = at;
  }
}

// Joins the pieces of the last items: a warp per row of a tail item's tile, a
// block 8 rows at a time and kExtTailBlocks blocks an item; those past the
// tail return at once. (Joined by the piece that is done last, in the kernel
// itself, 2 x 2048 tokens at 8192 took 379 us against 337: the softmax loop's
// code came out worse.)
constexpr int kExtTailRows = 8, kExtTailBlocks = 8;
__global__ void __launch_bounds__(kExtTailRows * 32) pda_extend_tail_kernel(const ExtendParams p) {
  grid_dependency_wait();
  const ExtendHead head = *p.head;
  const int item = (int)blockIdx.y;
  if (item >= head.tail) return;
  const int lane = threadIdx.x & 31;
  const int at = head.whole + item;
  const int2 tile = __ldcg(p.order + at / p.num_kv_heads);
  ExtendItem t;
  t.kvh = at % p.num_kv_heads;
  t.split = 0;
  if (!extend_item(p, tile.x, tile.y, t)) return;
  for (int row = (int)blockIdx.x * kExtTailRows + (threadIdx.x >> 5); row < t.rows;
       row += kExtTailBlocks * kExtTailRows) {
    float M = -INFINITY, den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t first = ((size_t)item * (2 * kExtRows) + row) * head.pieces;
#pragma unroll 4
    for (int i = 0; i < head.pieces; ++i) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.tail_ml) + (first + i));
      const float4 o = __ldcg(reinterpret_cast<const float4*>(p.tail_o + (first + i) * kHeadDim) + lane);
      if (ml.x != -INFINITY) lse_fold(M, den, acc, ml.x, ml.y, o);
    }
    const int tok = token_of(p, row);
    store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, t.row0 + tok,
                 t.kvh * p.gqa + row - tok * p.gqa, lane, M != -INFINITY, M, den, acc);
  }
}

// Joins the KV splits: one warp per (token, head) row.
struct ExtendMergeParams {
  void* out;
  const float* part_o;
  const float* part_ml;
  const int32_t* query_starts;
  int num_tokens;
  int num_seqs;
  int num_heads;
  int nsplit;
  float v_scale;
  const float* sinks;
  int out_fp8;
  float out_scale;
};
__global__ void __launch_bounds__(kHeadDim) pda_extend_merge_kernel(const ExtendMergeParams p) {
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kMergeRowsPerBlock + (threadIdx.x >> 5);
  if (item >= (long long)p.num_tokens * p.num_heads) return;
  const int row = (int)(item / p.num_heads), h = (int)(item % p.num_heads);
  const int first = __ldg(p.query_starts), end = __ldg(p.query_starts + p.num_seqs);
  grid_dependency_wait();
  if (row < first || row >= end) return;       // a row of no sequence
  float M = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < p.nsplit; ++i) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (item * p.nsplit + i));
    const float4 o = __ldcg(reinterpret_cast<const float4*>(p.part_o + (item * p.nsplit + i) * kHeadDim) + lane);
    if (ml.x != -INFINITY) lse_fold(M, den, acc, ml.x, ml.y, o);
  }
  store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, row, h, lane, M != -INFINITY, M, den,
               acc);
}

}  // namespace pda
