// Rotary positions (sm_103a): pda_rope_kernel rotates query and key heads,
// and, in its cache build, quantises the rotated keys and the values into the
// paged e4m3 cache on the way.
//
// Mathematics. Pair i < R/2 of a head turns by pos * inv_freq_i radians:
//   (a, b) -> magnitude * (a cos - b sin, a sin + b cos)
// with (a, b) = (x[i], x[i + R/2]) or, interleaved, (x[2i], x[2i + 1]); dims
// from R on pass through. The angle is reduced exactly in integers: the host
// hands over turns_i = inv_freq_i / 2 pi in units of 2^-64 turn, and
// pos * turns_i modulo 2^64 is the fraction of a turn whatever the position
// (negative positions turn back). Its top 32 bits, rounded, go to sincospi,
// so an angle is off by about 1e-7 rad plus |pos| * 2^-54 turns of the
// frequency's own 64-bit rounding, at position 1 and at position 10^6 alike.
//
// Bound: bytes (6 flops per 4 bytes moved). One CTA holds kTok tokens and one
// group of heads: it computes the (cos, sin) table of its tokens once and
// rotates every head of the group with it, each thread keeping its token's
// eight pairs in registers. What counts then is how many loads are in flight:
// each thread runs a ring of four heads of asynchronous copies into shared
// memory, private to it, so no barrier stands between them, and 8 (with the
// cache 7) CTAs fit an SM. 16,384 tokens of 40/8 heads take 62.7 us (6.4 TB/s),
// 8192 of 64/8 with the cache 55.7 us (5.7 TB/s), against 75 and 71 with two
// heads in registers. Rings of 2, 3 and 6 heads: 67.1, 65.0 and 66.2 us with
// the cache where 4 took 64.6 (half of its accesses then half-sectors).
// These are figures of slots in aligned runs of 16; packed prompts that start
// between the CTAs' bounds take 110.8 us at 8192 tokens of 64/8 heads, by their
// 1-byte stores of V.
#pragma once

#include "pda_kernels.cuh"

namespace pda {

constexpr int kRopeMaxPairs = kHeadDim / 2;
constexpr int kRopeThreads = 128;

struct RopeParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;          // cache build only
  __nv_bfloat16* q_out;
  __nv_bfloat16* k_out;            // without the cache
  const int64_t* positions;
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head;      // strides, elements
  long long qo_tok, qo_head, ko_tok, ko_head;
  int num_tokens;
  int num_heads;
  int num_kv_heads;
  int groups;                      // head groups (grid y); the cache build: kv heads
  int pairs;                       // R / 2
  int interleaved;
  float magnitude;
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int64_t* slot_mapping;
  int block_size;
  long long num_slots;
  float k_scale, v_scale;
  int v_shuffled;
  uint64_t turns[kRopeMaxPairs];   // inv_freq / 2 pi, units of 2^-64 turn
};

// 16 dims of a head as a thread holds them: two 16-byte vectors.
struct RopeItem {
  uint4 a, b;
};

// Dims of item j's two vectors. With R a multiple of 16 a head is 8 items:
// item j < R/16 holds dims 8j.. and 8j + R/2.. of the rotated part (the two
// sides of pairs 8j .. 8j+7; interleaved, pairs 4j .. 4j+3 and R/4 + 4j ..),
// the others dims of the rest, likewise in two halves: lanes next to each
// other touch vectors next to each other, so an access fills its sectors.
__device__ __forceinline__ void rope_item_dims(int j, int pairs, int& da, int& db) {
  const bool turned = j < pairs / 8;
  da = turned ? 8 * j : pairs + 8 * j;
  db = da + (turned ? pairs : kHeadDim / 2 - pairs);
}

// Rotates item j in fp32: r[0..7] vector a's dims, r[8..15] vector b's. t:
// (cos, sin) of its pairs, two to a float4.
__device__ __forceinline__ void rope_rotate(const RopeItem& x, int j, int pairs, bool interleaved, const float4 (&t)[4],
                                            float (&r)[16]) {
  const uint32_t wa[4] = {x.a.x, x.a.y, x.a.z, x.a.w}, wb[4] = {x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r[2 * i] = bf16lo_f32(wa[i]);
    r[2 * i + 1] = bf16hi_f32(wa[i]);
    r[8 + 2 * i] = bf16lo_f32(wb[i]);
    r[8 + 2 * i + 1] = bf16hi_f32(wb[i]);
  }
  if (j >= pairs / 8) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 c = t[i];
    if (interleaved) {
      const float a0 = r[4 * i], b0 = r[4 * i + 1], a1 = r[4 * i + 2], b1 = r[4 * i + 3];
      r[4 * i] = a0 * c.x - b0 * c.y;
      r[4 * i + 1] = a0 * c.y + b0 * c.x;
      r[4 * i + 2] = a1 * c.z - b1 * c.w;
      r[4 * i + 3] = a1 * c.w + b1 * c.z;
    } else {
      const float a0 = r[2 * i], b0 = r[8 + 2 * i], a1 = r[2 * i + 1], b1 = r[8 + 2 * i + 1];
      r[2 * i] = a0 * c.x - b0 * c.y;
      r[8 + 2 * i] = a0 * c.y + b0 * c.x;
      r[2 * i + 1] = a1 * c.z - b1 * c.w;
      r[8 + 2 * i + 1] = a1 * c.w + b1 * c.z;
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 pack_bf16x8(const float* r) {
  return make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]),
                    pack_bf16x2(r[6], r[7]));
}
// Eight e4m3 codes of r / scale (the IEEE binary32 quotient, as the cache
// writers do; a product with 1 / scale and the quotient only near the borders
// between codes was slower: 78 against 72 us for 8192 tokens of 64/8 heads).
__device__ __forceinline__ uint2 quantize8(const float* r, float scale) {
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = f32x2_to_e4m3x2(__fdiv_rn(r[2 * i], scale), __fdiv_rn(r[2 * i + 1], scale));
  return make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
}

// The thread's cp.async copies since the last call form a group; waits until
// at most n groups are in flight.
__device__ __forceinline__ void cp_async_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// kTok tokens x one head group per 128-thread CTA. 8 threads hold one head
// of one token, so 16 / kTok heads go side by side.
constexpr int kRopeDepth = 4;           // heads in flight per thread
template <int kTok, bool kCache>
__global__ void __launch_bounds__(kRopeThreads, kCache ? 7 : 8) pda_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int kSide = 16 / kTok;     // heads side by side
  // (cos, sin) of a token's pairs: the two pairs of an item's i-th float4 (see
  // rope_item_dims) are entry 8i + j, so that the 8 threads of a token read
  // entry i of each without conflicts
  __shared__ float4 cs[kTok][kRopeMaxPairs / 2];
  __shared__ __align__(16) uint8_t kt[kCache ? kTok : 1][kHeadDim];
  __shared__ __align__(16) uint8_t vt[kCache ? kTok : 1][kHeadDim];
  __shared__ long long slots[kTok];
  __shared__ uint4 ring[kRopeDepth][2][kRopeThreads];   // each thread's own items
  const int tid = threadIdx.x;
  const int j = tid & 7;
  const int tl = (tid >> 3) % kTok;
  const int side = (tid >> 3) / kTok;
  const int y = blockIdx.y;
  const long long t = (long long)blockIdx.x * kTok + tl;
  const bool in = t < p.num_tokens;
  const int q0 = (int)((long long)p.num_heads * y / p.groups), q1 = (int)((long long)p.num_heads * (y + 1) / p.groups);
  const int k0 = (int)((long long)p.num_kv_heads * y / p.groups);
  const int k1 = (int)((long long)p.num_kv_heads * (y + 1) / p.groups);
  const int nq = q1 - q0, nk = nq + k1 - k0;
  const int nh = kCache ? nk + 1 : nk;   // the cache build: its V head comes last
  const bool il = p.interleaved != 0;
  int da, db;
  rope_item_dims(j, p.pairs, da, db);

  const uint32_t mine_at = smem_u32(&ring[0][0][tid]);
  // one copy group per step, empty past the last head
  auto load = [&](int step) {
    const int h = step * kSide + side;
    if (in && h < nh) {
      const uint32_t at = mine_at + (uint32_t)((unsigned)step % kRopeDepth) * (2 * kRopeThreads * 16);
      if (kCache && h >= nk) {
        const __nv_bfloat16* s = p.v + t * p.v_tok + (long long)y * p.v_head + 8 * j;
        cp_async_16(at, s);
        cp_async_16(at + kRopeThreads * 16, s + kHeadDim / 2);
      } else {
        const __nv_bfloat16* s =
            h < nq ? p.q + t * p.q_tok + (q0 + h) * p.q_head : p.k + t * p.k_tok + (k0 + h - nq) * p.k_head;
        cp_async_16(at, s + da);
        cp_async_16(at + kRopeThreads * 16, s + db);
      }
    }
    cp_async_close();
  };
#pragma unroll
  for (int d = 0; d < kRopeDepth; ++d) load(d);
  if constexpr (kCache) {
    if (side == 0 && j == 0) {
      long long slot = in ? __ldg(p.slot_mapping + t) : -1;
      if (slot >= p.num_slots) {
        atomicOr(&g_status, kStatusBadSlot);
        slot = -1;
      }
      slots[tl] = slot;
    }
  }
  // Lanes run over tokens first: the 64-bit frequencies sit in constant
  // memory, where lanes of one address share a read.
  for (int i = tid; i < kTok * p.pairs; i += kRopeThreads) {
    const int tt = i % kTok, pr = i / kTok;
    const long long tok = (long long)blockIdx.x * kTok + tt;
    if (tok < p.num_tokens) {
      const uint64_t turn = (uint64_t)__ldg(p.positions + tok) * p.turns[pr];
      const int frac = (int)(uint32_t)((turn + 0x80000000ull) >> 32);
      float sn, cn;
      sincospif((float)frac * 4.656612873077393e-10f, &sn, &cn);   // 2^-31 half turns
      const int hi = pr >= p.pairs / 2, pp = hi ? pr - p.pairs / 2 : pr;
      const int e = il ? 8 * (2 * hi + ((pp >> 1) & 1)) + (pp >> 2) : 8 * ((pr >> 1) & 3) + (pr >> 3);
      reinterpret_cast<float2*>(&cs[tt][e])[pr & 1] =
          make_float2(cn * p.magnitude, sn * p.magnitude);
    }
  }
  __syncthreads();
  // a thread stays with its token and pairs through all heads
  float4 mine[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) mine[i] = cs[tl][8 * i + j];

  const int steps = (nh + kSide - 1) / kSide;
  for (int step = 0; step < steps; ++step) {
    const int h = step * kSide + side;
    cp_async_wait<kRopeDepth - 1>();
    if (in && h < nh) {
      RopeItem x;
      x.a = ring[(unsigned)step % kRopeDepth][0][tid];
      x.b = ring[(unsigned)step % kRopeDepth][1][tid];
      float r[16];
      if (kCache && h >= nk) {
        rope_rotate(x, kHeadDim, p.pairs, il, mine, r);
        *reinterpret_cast<uint2*>(&vt[kCache ? tl : 0][8 * j]) = quantize8(r, p.v_scale);
        *reinterpret_cast<uint2*>(&vt[kCache ? tl : 0][kHeadDim / 2 + 8 * j]) = quantize8(r + 8, p.v_scale);
      } else {
        rope_rotate(x, j, p.pairs, il, mine, r);
        if (kCache && h >= nq) {
          *reinterpret_cast<uint2*>(&kt[kCache ? tl : 0][da]) = quantize8(r, p.k_scale);
          *reinterpret_cast<uint2*>(&kt[kCache ? tl : 0][db]) = quantize8(r + 8, p.k_scale);
        } else {
          __nv_bfloat16* d = h < nq ? p.q_out + t * p.qo_tok + (q0 + h) * p.qo_head
                                    : p.k_out + t * p.ko_tok + (k0 + h - nq) * p.ko_head;
          *reinterpret_cast<uint4*>(d + da) = pack_bf16x8(r);
          *reinterpret_cast<uint4*>(d + db) = pack_bf16x8(r + 8);
        }
      }
    }
    // the stores above waited for this slot's reads
    load(step + kRopeDepth);
  }
  if constexpr (kCache) {
    __syncthreads();
    const int bs = p.block_size;
    // K: one 16-byte row of a token per thread
    if (side == 0 && slots[tl] >= 0) {
      const long long b = slots[tl] / bs;
      const int o = (int)(slots[tl] % bs);
      *reinterpret_cast<uint4*>(p.k_cache + ((size_t)b * p.num_kv_heads + y) * (size_t)kHeadDim * bs +
                                ((size_t)j * bs + o) * 16) = *reinterpret_cast<const uint4*>(&kt[tl][16 * j]);
    }
    // V: rows run over tokens. 16 slots in one aligned run store 16-byte
    // rows; else a warp writes a token's 128 codes, 4 per lane.
    bool run = kTok == kCacheWriteTokens;
    if constexpr (kTok == kCacheWriteTokens) {
      const long long first = slots[0];
      run = __syncthreads_and(first >= 0 && first % kCacheWriteTokens == 0 && slots[tl] == first + tl);
      if (run) {
        const int d = tid;
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = (uint32_t)vt[4 * i][d] | ((uint32_t)vt[4 * i + 1][d] << 8) | ((uint32_t)vt[4 * i + 2][d] << 16) |
                 ((uint32_t)vt[4 * i + 3][d] << 24);
        const long long b = first / bs;
        const int o = (int)(first % bs);
        const size_t off = p.v_shuffled ? ((size_t)(o / 16) * kHeadDim + d) * 16 : (size_t)d * bs + o;
        *reinterpret_cast<uint4*>(p.v_cache + ((size_t)b * p.num_kv_heads + y) * (size_t)kHeadDim * bs + off) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    if (!run) {
      const int d0 = 4 * (tid & 31);
      const size_t vstride = p.v_shuffled ? 16 : (size_t)bs;
#pragma unroll
      for (int jj = tid >> 5; jj < kTok; jj += kRopeThreads / 32) {
        const long long sl = slots[jj];
        if (sl < 0) continue;
        const long long b = sl / bs;
        const int o = (int)(sl % bs);
        const uint32_t v = *reinterpret_cast<const uint32_t*>(&vt[jj][d0]);
        uint8_t* vrow = p.v_cache + ((size_t)b * p.num_kv_heads + y) * (size_t)kHeadDim * bs +
                        (p.v_shuffled ? ((size_t)(o / 16) * kHeadDim + d0) * 16 + (o % 16) : (size_t)d0 * bs + o);
#pragma unroll
        for (int i = 0; i < 4; ++i) vrow[(size_t)i * vstride] = (uint8_t)(v >> (8 * i));
      }
    }
  }
}

// Any even R, any alignment and stride: one warp per (token, head), two
// pairs (or passed-through dims) per lane in 2-byte accesses. Rotary sizes
// that are no multiple of 16 and views off the 16-byte grid come here: 8192
// tokens of 40/8 heads take 86.6 us at R = 20, 186.7 us at R = 128 off the grid
// (35.1 us by the kernel above at R = 128). Every warp makes its angles anew.
template <bool kCache>
__global__ void __launch_bounds__(kRopeThreads) pda_rope_any_kernel(const __grid_constant__ RopeParams p) {
  const int lane = threadIdx.x & 31;
  const int per = p.num_heads + p.num_kv_heads * (kCache ? 2 : 1);
  const long long item = (long long)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  if (item >= (long long)p.num_tokens * per) return;
  const long long t = item / per;
  const int h = (int)(item % per);
  const int kind = h < p.num_heads ? 0 : (h < p.num_heads + p.num_kv_heads ? 1 : 2);   // q, k, v
  const int hh = h - (kind == 0 ? 0 : (kind == 1 ? p.num_heads : p.num_heads + p.num_kv_heads));
  const __nv_bfloat16* s = kind == 0 ? p.q + t * p.q_tok + hh * p.q_head
                                     : (kind == 1 ? p.k + t * p.k_tok + hh * p.k_head : p.v + t * p.v_tok + hh * p.v_head);
  long long slot = -1;
  if (kCache && kind) {
    slot = __ldg(p.slot_mapping + t);
    if (slot >= p.num_slots) {
      if (lane == 0) atomicOr(&g_status, kStatusBadSlot);
      slot = -1;
    }
    if (slot < 0) return;
  }
  const int64_t pos = __ldg(p.positions + t);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = lane + 32 * u;
    const bool turn = kind < 2 && i < p.pairs;
    int d0 = i < p.pairs ? (p.interleaved ? 2 * i : i) : 2 * i;
    int d1 = i < p.pairs ? (p.interleaved ? 2 * i + 1 : i + p.pairs) : 2 * i + 1;
    float a = __bfloat162float(s[d0]), b = __bfloat162float(s[d1]);
    if (turn) {
      const uint64_t turns = (uint64_t)pos * p.turns[i];
      const int frac = (int)(uint32_t)((turns + 0x80000000ull) >> 32);
      float sn, cn;
      sincospif((float)frac * 4.656612873077393e-10f, &sn, &cn);
      sn *= p.magnitude;
      cn *= p.magnitude;
      const float ra = a * cn - b * sn, rb = a * sn + b * cn;
      a = ra;
      b = rb;
    }
    if (kCache && kind) {
      const float scale = kind == 1 ? p.k_scale : p.v_scale;
      const uint32_t c = f32x2_to_e4m3x2(__fdiv_rn(a, scale), __fdiv_rn(b, scale));
      const int bs = p.block_size;
      const long long blk = slot / bs;
      const int o = (int)(slot % bs);
      uint8_t* page = (kind == 1 ? p.k_cache : p.v_cache) + ((size_t)blk * p.num_kv_heads + hh) * (size_t)kHeadDim * bs;
      auto at = [&](int d) -> size_t {
        if (kind == 1) return ((size_t)(d / 16) * bs + o) * 16 + d % 16;
        return p.v_shuffled ? ((size_t)(o / 16) * kHeadDim + d) * 16 + o % 16 : (size_t)d * bs + o;
      };
      page[at(d0)] = (uint8_t)c;
      page[at(d1)] = (uint8_t)(c >> 8);
    } else {
      __nv_bfloat16* d = kind == 0 ? p.q_out + t * p.qo_tok + hh * p.qo_head : p.k_out + t * p.ko_tok + hh * p.ko_head;
      d[d0] = __float2bfloat16_rn(a);
      d[d1] = __float2bfloat16_rn(b);
    }
  }
}

}  // namespace pda
