// Attention of a chunk of new tokens per sequence over the paged e4m3 cache
// (pda_extend): one warp per (new token, query head).
#pragma once

#include "pda_kernels.cuh"

namespace pda {

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
  int block_size;
  int max_blocks;
  int window;
  float logit_scale_log2;       // scale * k_scale * log2(e)
  float v_scale;
  const float* sinks;
  int out_fp8;
  float out_scale;
  int v_shuffled;
  uint32_t block_limit;
};

constexpr int kExtendWarps = 4;

// First s with query_starts[s + 1] > row, or num_seqs.
__device__ __forceinline__ int sequence_of_row(const int32_t* starts, int num_seqs, int row) {
  int lo = 0, hi = num_seqs;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(starts + mid + 1) > row)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kExtendWarps * 32) pda_extend_row_kernel(const ExtendParams p) {
  __shared__ float qs[kExtendWarps][kHeadDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * kExtendWarps + warp;
  if (item >= (long long)p.num_tokens * p.num_heads) return;
  const int row = (int)(item / p.num_heads), h = (int)(item % p.num_heads);
  const int s = sequence_of_row(p.query_starts, p.num_seqs, row);
  if (s >= p.num_seqs || row < __ldg(p.query_starts + s)) return;
  const int start = __ldg(p.query_starts + s), n = __ldg(p.query_starts + s + 1) - start;
  const int bs = p.block_size;
  const int len = (int)max(0ll, min((long long)__ldg(p.seq_lens + s), (long long)p.max_blocks * bs));
  const int pos = len - n + row - start;
  const int lo = p.window > 0 ? max(0, pos - p.window + 1) : 0;
  const size_t o0 = ((size_t)row * p.num_heads + h) * kHeadDim;
  for (int d = lane; d < kHeadDim; d += 32) qs[warp][d] = __bfloat162float(p.q[o0 + d]);
  __syncwarp();
  const int kvh = h / p.gqa;
  const size_t page_bytes = (size_t)kHeadDim * bs;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = lo & ~31; t0 <= pos; t0 += 32) {
    const int t = t0 + lane;
    const bool seen = t >= lo && t <= pos;
    float z = -INFINITY;
    size_t page = 0;
    if (seen) {
      const int b = checked_block(__ldg(p.block_tables + (size_t)s * p.max_blocks + t / bs), p.block_limit);
      page = ((size_t)b * p.num_kv_heads + kvh) * page_bytes;
      float a = 0.f;
      for (int c = 0; c < kChunks; ++c) {
        const uint4 x = *reinterpret_cast<const uint4*>(p.k_cache + page + ((size_t)c * bs + t % bs) * 16);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        for (int i = 0; i < 4; ++i) {
          const uint32_t e = e4m3x2_lo_to_f16x2(w[i]), f = e4m3x2_hi_to_f16x2(w[i]);
          const float* qq = &qs[warp][16 * c + 4 * i];
          a += qq[0] * f16lo_f32(e) + qq[1] * f16hi_f32(e) + qq[2] * f16lo_f32(f) + qq[3] * f16hi_f32(f);
        }
      }
      z = a * p.logit_scale_log2;
    }
    float mx = z;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(m, mx);
    const float f = m == -INFINITY ? 0.f : fast_exp2(m - mn);
    const float pr = seen ? fast_exp2(z - mn) : 0.f;
    float sum = pr;
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    l = l * f + sum;
    m = mn;
    acc.x *= f, acc.y *= f, acc.z *= f, acc.w *= f;
    for (int i = 0; i < 32; ++i) {
      const int ti = t0 + i;
      if (ti < lo || ti > pos) continue;
      const float pi = __shfl_sync(0xffffffffu, pr, i);
      const size_t pg = __shfl_sync(0xffffffffu, (unsigned long long)page, i);
      const int o = ti % bs;
      float vv[4];
      for (int u = 0; u < 4; ++u) {
        const int d = 4 * lane + u;
        const size_t at = p.v_shuffled ? ((size_t)(o / 16) * kHeadDim + d) * 16 + o % 16 : (size_t)d * bs + o;
        vv[u] = f16lo_f32(e4m3x2_lo_to_f16x2(p.v_cache[pg + at]));
      }
      acc.x += pi * vv[0], acc.y += pi * vv[1], acc.z += pi * vv[2], acc.w += pi * vv[3];
    }
  }
  store_merged(p.out, p.sinks, p.out_fp8, p.out_scale, p.v_scale, p.num_heads, row, h, lane, pos >= 0, m, l, acc);
}

}  // namespace pda
