// Entry points of the caches in fewer bits: writers, readers and the decode
// attention over 4 bits. Included by pda_api.cu, whose validation helpers,
// workspace and error conventions they share.
#pragma once

namespace {

// Rows (a token's kv head) up to which the slot-scale writer gives each a warp.
constexpr long long kSlotScalesMaxRows = 4096;

// Scales that the quantising writers take: with them every midpoint's product
// is a normal number whose last bit binary32 holds, so that its sign is exact.
bool scale_in_range(float x) { return x >= 0x1p-100f && x <= 0x1p100f; }   // false for NaN

// A programmatic launch: the kernel sets up its CTAs while the one in front of it ends,
// and waits for that one's results (grid_dependency_wait) before it touches memory. That
// one has waited for what is in front of it, as every programmatic kernel here does. us
// without / with it, calls in turn on one stream: slot-scale write of 8192 tokens 18.5 /
// 15.9, 4-bit write and read of 16384 41.0 / 36.3, 4-bit read of 64 contexts 105.6 / 103.0,
// decode of 16 x 1024 18.2 / 15.7. (Writers and readers that also let the next kernel's
// CTAs in early, with grid_dependents_launch: 17.6, 36.6, 103.3, and a write of 256
// tokens in a graph 6.7 where this takes 4.7.)
template <typename P>
bool launch_behind(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t stream, const P& p) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = grid;
  lc.blockDim = dim3((unsigned)threads);
  lc.dynamicSmemBytes = smem;
  lc.stream = stream;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, p) == cudaSuccess;
}

pda_status write_checks(const pda_token_rows* key, const pda_token_rows* value, int num_tokens, int num_kv_heads,
                        int head_size, int block_size, long long num_blocks) {
  if (!key || !value || num_tokens < 0 || num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 || num_blocks < 0)
    return PDA_ERR_INVALID_ARG;
  if (head_size != kHeadDim || block_size % 16 != 0 || block_size > 128 || num_kv_heads > 65535 ||
      num_blocks > INT32_MAX || num_tokens > INT32_MAX - 64)
    return PDA_ERR_UNSUPPORTED;
  return PDA_OK;
}

pda_status write_fill(pda::LowbitsWriteParams& p, const pda_token_rows* key, const pda_token_rows* value,
                      const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int block_size,
                      long long num_blocks, bool* vec) {
  if (!key->base || !value->base || !slot_mapping || misaligned(slot_mapping, 8) || misaligned(key->base, 2) ||
      misaligned(value->base, 2))
    return PDA_ERR_INVALID_ARG;
  p.k = static_cast<const __nv_bfloat16*>(key->base);
  p.v = static_cast<const __nv_bfloat16*>(value->base);
  p.k_tok = key->token_stride, p.k_head = key->head_stride;
  p.v_tok = value->token_stride, p.v_head = value->head_stride;
  p.slot_mapping = slot_mapping;
  p.num_tokens = num_tokens;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_slots = num_blocks * (long long)block_size;
  *vec = rope_on_grid(p.k, p.k_tok, p.k_head) && rope_on_grid(p.v, p.v_tok, p.v_head);
  return PDA_OK;
}

pda_status gather_checks(int num_tokens, int num_seqs, int num_kv_heads, int head_size, int block_size, int max_blocks,
                         long long num_blocks) {
  if (num_tokens < 0 || num_seqs < 0 || num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 || max_blocks < 0 ||
      num_blocks < 0)
    return PDA_ERR_INVALID_ARG;
  if (head_size != kHeadDim || block_size % 16 != 0 || block_size > 128 || num_kv_heads > 65535 ||
      num_blocks > INT32_MAX || (long long)max_blocks * block_size > (long long)INT32_MAX / 2 ||
      num_tokens > INT32_MAX - 64)
    return PDA_ERR_UNSUPPORTED;
  return PDA_OK;
}

pda_status gather_fill(pda::GatherParams& p, void* k_out, void* v_out, const int32_t* block_tables,
                       const int32_t* token_starts, const int32_t* first, int num_tokens, int num_seqs,
                       int num_kv_heads, int block_size, int max_blocks, long long num_blocks) {
  if (!k_out || !v_out || k_out == v_out || !token_starts || (max_blocks > 0 && !block_tables) || !aligned16(k_out) || !aligned16(v_out) ||
      misaligned(block_tables, 4) || misaligned(token_starts, 4) || misaligned(first, 4))
    return PDA_ERR_INVALID_ARG;
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.block_tables = block_tables;
  p.token_starts = token_starts;
  p.first = first;
  p.num_tokens = num_tokens;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks = max_blocks;
  p.num_blocks = num_blocks;
  return PDA_OK;
}

pda_status gather_e4m3(pda::GatherParams& p, const void* k_cache, const void* v_cache, cudaStream_t stream) {
  if (!k_cache || !v_cache || !aligned16(k_cache) || !aligned16(v_cache)) return PDA_ERR_INVALID_ARG;
  p.k_cache = static_cast<const uint8_t*>(k_cache);
  p.v_cache = static_cast<const uint8_t*>(v_cache);
  p.v_wide = (p.v_shuffled || p.block_size == 16) && !misaligned(v_cache, 32);
  const int tiles = (p.num_tokens + pda::kGatherRows - 1) / pda::kGatherRows;
  // Heads of a CTA of four warps: all, unless that leaves fewer than 4 CTAs an SM.
  int per = p.num_kv_heads;
  while (per > 4 && (long long)tiles * ((p.num_kv_heads + per - 1) / per) < 4 * 152) per = (per + 1) / 2;
  p.heads_per_cta = per;
  const dim3 grid((unsigned)tiles, (unsigned)((p.num_kv_heads + per - 1) / per));
  return launch_behind(pda::pda_gather_kernel, grid, pda::kGatherThreads, 0, stream, p) ? PDA_OK : PDA_ERR_CUDA;
}

// Resident CTAs of the 4-bit decode kernel on device `dev`; opts it in to its
// shared memory, once per device.
pda_status fp4_resident(int dev, int* ctas) {
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& di = g_devices[dev];
  if (di.fp4_ctas == 0) {
    int sms = 0, occ = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(pda::pda_fp4_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)pda::kF4Smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, pda::pda_fp4_decode_kernel, pda::kF4Threads, pda::kF4Smem) !=
            cudaSuccess ||
        occ < 1)
      return PDA_ERR_CUDA;
    const int n = sms * occ;
    di.fp4_ctas = n < pda::kF4MaxCtas ? n : pda::kF4MaxCtas;
  }
  *ctas = di.fp4_ctas;
  return PDA_OK;
}

constexpr size_t kFp4HeadBytes = (sizeof(pda::Fp4Head) + 255) / 256 * 256;

// One size for every call.
pda_status fp4_workspace(int dev, cudaStream_t stream, void** ws) {
  const size_t bytes = kFp4HeadBytes + (size_t)pda::kF4Slots * pda::kF4PieceFloats * sizeof(float);
  return grow_workspace(g_fp4_ws, dev, stream, bytes, kFp4HeadBytes, ws);
}

}  // namespace

extern "C" {

pda_status pda_reshape_and_cache_slot_scales(const pda_token_rows* key, const pda_token_rows* value, void* k_cache,
                                             void* v_cache, float* k_scales, float* v_scales,
                                             const int64_t* slot_mapping, int num_tokens, int num_kv_heads,
                                             int head_size, int block_size, long long num_blocks, float min_scale,
                                             cudaStream_t stream) {
  pda_status st = write_checks(key, value, num_tokens, num_kv_heads, head_size, block_size, num_blocks);
  if (st != PDA_OK) return st;
  if (!std::isfinite(min_scale) || min_scale <= 0.f) return PDA_ERR_INVALID_ARG;
  if (!scale_in_range(min_scale)) return PDA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PDA_OK;
  pda::LowbitsWriteParams p = {};
  bool vec = false;
  st = write_fill(p, key, value, slot_mapping, num_tokens, num_kv_heads, block_size, num_blocks, &vec);
  if (st != PDA_OK) return st;
  if (!k_cache || !v_cache || !k_scales || !v_scales || !aligned16(k_cache) || !aligned16(v_cache) ||
      misaligned(k_scales, 4) || misaligned(v_scales, 4))
    return PDA_ERR_INVALID_ARG;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.min_scale = min_scale;
  // Few rows: a warp each, whatever the slots. More: tiles of 16 tokens, whose V codes
  // go out by groups of slots (us with a warp a row / tiles, 8 kv heads: 256 tokens in
  // whole blocks 6.3 / 7.2, scattered 5.5 / 15.7; 512 9.8 / 7.3, 8.2 / 16.2; 1024 16.3 /
  // 7.2, 12.5 / 18.6; 8192 82.7 / 16.2, 75.5 / 74.2). The number of rows alone decides, as
  // the host does not see the slots: scattered calls from 513 tokens on lose by it.
  const long long items = (long long)num_tokens * num_kv_heads;
  bool done;
  if (items <= kSlotScalesMaxRows) {
    const dim3 grid((unsigned)((items + pda::kLowbitsThreads / 32 - 1) / (pda::kLowbitsThreads / 32)));
    done = launch_behind(vec ? pda::pda_write_slot_scales_kernel<true> : pda::pda_write_slot_scales_kernel<false>, grid,
                         pda::kLowbitsThreads, 0, stream, p);
  } else {
    const int warps = pda::kWriteTileThreads / 32;
    const dim3 grid((unsigned)((num_tokens + 15) / 16), (unsigned)((num_kv_heads + warps - 1) / warps));
    done = launch_behind(vec ? pda::pda_write_slot_scales_tile_kernel<true> : pda::pda_write_slot_scales_tile_kernel<false>,
                         grid, pda::kWriteTileThreads, 0, stream, p);
  }
  return done ? PDA_OK : PDA_ERR_CUDA;
}

pda_status pda_reshape_and_cache_fp4(const pda_token_rows* key, const pda_token_rows* value, void* kv_cache,
                                     const int64_t* slot_mapping, int num_tokens, int num_kv_heads, int head_size,
                                     int block_size, long long num_blocks, float k_scale, float v_scale,
                                     cudaStream_t stream) {
  pda_status st = write_checks(key, value, num_tokens, num_kv_heads, head_size, block_size, num_blocks);
  if (st != PDA_OK) return st;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f)
    return PDA_ERR_INVALID_ARG;
  if (!scale_in_range(k_scale) || !scale_in_range(v_scale)) return PDA_ERR_UNSUPPORTED;
  if (num_tokens == 0) return PDA_OK;
  pda::LowbitsWriteParams p = {};
  bool vec = false;
  st = write_fill(p, key, value, slot_mapping, num_tokens, num_kv_heads, block_size, num_blocks, &vec);
  if (st != PDA_OK) return st;
  if (!kv_cache || !aligned16(kv_cache)) return PDA_ERR_INVALID_ARG;
  p.k_cache = static_cast<uint8_t*>(kv_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_inv6 = (float)(1.0 / (6.0 * (double)k_scale));
  p.v_inv6 = (float)(1.0 / (6.0 * (double)v_scale));
  // Heads of a warp: four, whose loads overlap; one where four leave fewer than 16
  // warps an SM.
  const bool four = (long long)num_tokens * num_kv_heads >= 4ll * 16 * 152;
  const int per = four ? 4 : 1;
  const dim3 grid((unsigned)((num_tokens + pda::kLowbitsThreads / 32 - 1) / (pda::kLowbitsThreads / 32)),
                  (unsigned)((num_kv_heads + per - 1) / per));
  const auto kernel = four ? (vec ? pda::pda_write_fp4_kernel<true, 4> : pda::pda_write_fp4_kernel<false, 4>)
                           : (vec ? pda::pda_write_fp4_kernel<true, 1> : pda::pda_write_fp4_kernel<false, 1>);
  return launch_behind(kernel, grid, pda::kLowbitsThreads, 0, stream, p) ? PDA_OK : PDA_ERR_CUDA;
}

pda_status pda_gather_cache(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* token_starts, const int32_t* first,
                            int num_tokens, int num_seqs, int num_kv_heads, int head_size, int block_size,
                            int max_num_blocks_per_seq, long long num_blocks, float k_scale, float v_scale,
                            int kv_layout, cudaStream_t stream) {
  pda_status st = gather_checks(num_tokens, num_seqs, num_kv_heads, head_size, block_size, max_num_blocks_per_seq,
                                num_blocks);
  if (st != PDA_OK) return st;
  if (kv_layout != PDA_KV_NATIVE && kv_layout != PDA_KV_SHUFFLED_V) return PDA_ERR_INVALID_ARG;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale)) return PDA_ERR_INVALID_ARG;
  if (num_tokens == 0 || num_seqs == 0) return PDA_OK;
  pda::GatherParams p = {};
  st = gather_fill(p, k_out, v_out, block_tables, token_starts, first, num_tokens, num_seqs, num_kv_heads, block_size,
                   max_num_blocks_per_seq, num_blocks);
  if (st != PDA_OK) return st;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.v_shuffled = kv_layout == PDA_KV_SHUFFLED_V ? 1 : 0;
  return gather_e4m3(p, k_cache, v_cache, stream);
}

pda_status pda_gather_cache_slot_scales(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                        const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                        const int32_t* token_starts, const int32_t* first, int num_tokens,
                                        int num_seqs, int num_kv_heads, int head_size, int block_size,
                                        int max_num_blocks_per_seq, long long num_blocks, cudaStream_t stream) {
  pda_status st = gather_checks(num_tokens, num_seqs, num_kv_heads, head_size, block_size, max_num_blocks_per_seq,
                                num_blocks);
  if (st != PDA_OK) return st;
  if (num_tokens == 0 || num_seqs == 0) return PDA_OK;
  pda::GatherParams p = {};
  st = gather_fill(p, k_out, v_out, block_tables, token_starts, first, num_tokens, num_seqs, num_kv_heads, block_size,
                   max_num_blocks_per_seq, num_blocks);
  if (st != PDA_OK) return st;
  if (!k_scales || !v_scales || misaligned(k_scales, 4) || misaligned(v_scales, 4)) return PDA_ERR_INVALID_ARG;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  return gather_e4m3(p, k_cache, v_cache, stream);
}

pda_status pda_gather_cache_fp4(void* k_out, void* v_out, const void* kv_cache, const int32_t* block_tables,
                                const int32_t* token_starts, const int32_t* first, int num_tokens, int num_seqs,
                                int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                                long long num_blocks, float k_scale, float v_scale, cudaStream_t stream) {
  pda_status st = gather_checks(num_tokens, num_seqs, num_kv_heads, head_size, block_size, max_num_blocks_per_seq,
                                num_blocks);
  if (st != PDA_OK) return st;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale)) return PDA_ERR_INVALID_ARG;
  if (num_tokens == 0 || num_seqs == 0) return PDA_OK;
  pda::GatherParams p = {};
  st = gather_fill(p, k_out, v_out, block_tables, token_starts, first, num_tokens, num_seqs, num_kv_heads, block_size,
                   max_num_blocks_per_seq, num_blocks);
  if (st != PDA_OK) return st;
  if (!kv_cache || !aligned16(kv_cache)) return PDA_ERR_INVALID_ARG;
  p.k_cache = static_cast<const uint8_t*>(kv_cache);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  int rows = pda::kGatherMaxRows4;
  while (rows > 1 && (num_tokens + rows - 1) / rows < 8 * 152) rows /= 2;
  p.rows_per_cta = rows;
  const dim3 grid((unsigned)((num_tokens + rows - 1) / rows));
  return launch_behind(pda::pda_gather_fp4_kernel, grid, pda::kLowbitsThreads, 0, stream, p) ? PDA_OK : PDA_ERR_CUDA;
}

pda_status pda_decode_fp4(void* out, const void* q, const void* kv_cache, const int32_t* block_tables,
                          const int32_t* seq_lens, int num_seqs, int num_heads, int num_kv_heads, int head_size,
                          int block_size, int max_num_blocks_per_seq, long long num_blocks, float scale, float k_scale,
                          float v_scale, int window, const float* sinks, int out_dtype, float output_scale,
                          cudaStream_t stream) {
  pda_status st = validate_sizes(num_seqs, num_heads, num_kv_heads, head_size, block_size, max_num_blocks_per_seq,
                                 scale, k_scale, v_scale);
  if (st != PDA_OK) return st;
  if (window < 0 || num_blocks < 0) return PDA_ERR_INVALID_ARG;
  if (out_dtype != PDA_OUT_BF16 && out_dtype != PDA_OUT_E4M3) return PDA_ERR_INVALID_ARG;
  if (out_dtype == PDA_OUT_E4M3 && !(std::isfinite(output_scale) && output_scale > 0.f)) return PDA_ERR_INVALID_ARG;
  if (misaligned(sinks, 4)) return PDA_ERR_INVALID_ARG;
  if (num_blocks > INT32_MAX || (long long)num_seqs * max_num_blocks_per_seq > INT32_MAX) return PDA_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PDA_OK;
  // Heads of a unit, as many as share a chunk of whole pages (see pda_fp4.cuh), and
  // the chunks at the longest lengths, for `tiles` tiles a warp.
  int tiles = pda::kF4Tiles, group = 0, per = 0;
  long long most = 0;
  auto cut = [&] {
    const int tokens = 16 * pda::kF4Warps * tiles;
    group = 4;
    while (group > 1 && (num_kv_heads % group != 0 || block_size * group > tokens)) group /= 2;
    per = tokens / group / block_size;
    most = (long long)num_seqs * (num_kv_heads / group) *
           (max_num_blocks_per_seq > per ? (max_num_blocks_per_seq + per - 1) / per : 1);
  };
  cut();
  if (most > INT32_MAX) return PDA_ERR_UNSUPPORTED;
  if (num_blocks == 0 || !out || !q || !kv_cache || !seq_lens || (max_num_blocks_per_seq > 0 && !block_tables))
    return PDA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(kv_cache) || misaligned(block_tables, 4) || misaligned(seq_lens, 4))
    return PDA_ERR_INVALID_ARG;
  return guarded([&]() -> pda_status {
    int dev = 0, ctas = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PDA_ERR_CUDA;
    pda_status st = fp4_resident(dev, &ctas);
    if (st != PDA_OK) return st;
    void* ws = nullptr;
    st = fp4_workspace(dev, stream, &ws);
    if (st != PDA_OK) return st;
    // Half as large chunks where large ones are too few for even runs: below four a CTA
    // (us with 4 / 2 tiles a warp, 32/8 heads: 16 x 1024 tokens 16.3 / 15.0, 32 x 1024
    // 20.9 / 19.1, 64 x 1024 25.2 / 25.3, 128 x 1 to 2048 43.7 / 48.8). But not where a
    // large chunk holds a whole sequence, so that nothing is to be joined (64 x 50 tokens
    // 10.0, and 11.8 with the join). All this goes by the table's width, as the host does not
    // see the lengths: with 8192 entries a row 16 x 1024 take 17.0, 64 x 50 11.8.
    if (most < 4ll * ctas) {
      const int whole = per;
      tiles = 2;
      cut();
      if (max_num_blocks_per_seq > per && max_num_blocks_per_seq <= whole) {
        tiles = pda::kF4Tiles;
        cut();
      }
    }
    const double logit = (double)scale * (double)k_scale * 1.4426950408889634;
    pda::Fp4DecodeParams p = {};
    p.out = out;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.cache = static_cast<const uint8_t*>(kv_cache);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.sinks = sinks;
    p.head = static_cast<pda::Fp4Head*>(ws);
    p.pieces = reinterpret_cast<float*>(static_cast<char*>(ws) + kFp4HeadBytes);
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.gqa = num_heads / num_kv_heads;
    p.block_size = block_size;
    p.max_blocks = max_num_blocks_per_seq;
    p.num_blocks = (int)num_blocks;
    p.window = window;
    p.pages_per_chunk = per;
    p.group = group;
    p.tiles = tiles;
    p.bs_inverse = ((1ull << 37) + block_size - 1) / block_size;
    p.chunk_inverse = ((1ull << 37) + per - 1) / per;
    p.logit_scale_log2 = (float)std::fabs(logit);
    p.negate = logit < 0.0 ? 1 : 0;
    p.v_scale = v_scale;
    p.out_fp8 = out_dtype == PDA_OUT_E4M3;
    p.out_scale = output_scale;
    const unsigned grid = (unsigned)(most < ctas ? most : ctas);
    std::lock_guard<std::mutex> lk(g_ops_mu);   // the two kernels follow each other
    if (!launch_behind(pda::pda_fp4_decode_kernel, dim3(grid), pda::kF4Threads, pda::kF4Smem, stream, p)) return PDA_ERR_CUDA;
    if (max_num_blocks_per_seq <= per) return PDA_OK;   // units of one chunk: no cut divides them
    const long long rows = (long long)num_seqs * num_heads;
    const dim3 join((unsigned)(rows < pda::kF4JoinCtas ? rows : pda::kF4JoinCtas));
    if (launch_behind(pda::pda_fp4_join_kernel, join, pda::kF4JoinThreads, 0, stream, p)) return PDA_OK;
    cudaMemsetAsync(ws, 0, kFp4HeadBytes, stream);   // the lists that the join would have emptied
    return PDA_ERR_CUDA;
  });
}

pda_status pda_reserve_fp4(cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    int dev = 0, ctas = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PDA_ERR_CUDA;
    const pda_status st = fp4_resident(dev, &ctas);
    if (st != PDA_OK) return st;
    void* ws = nullptr;
    return fp4_workspace(dev, stream, &ws);
  });
}

}  // extern "C"
