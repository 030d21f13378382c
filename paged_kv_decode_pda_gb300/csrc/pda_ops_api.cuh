// Entry points around the decode call: rotary positions (alone and with the
// cache write), attention of a chunk of new tokens, and the pages'
// bookkeeping. Included by pda_api.cu, whose validation helpers, workspace
// and error conventions they share.
#pragma once

namespace {

// Runs an entry point's body so that no C++ exception (a failed allocation
// in a map) crosses the C boundary.
template <typename F>
pda_status guarded(F&& body) {
  try {
    return body();
  } catch (...) {
    return PDA_ERR_CUDA;
  }
}

// Held over the launches of a call that leaves something from one kernel to
// the next, in the workspace or (the page calls) in the tables and counts, and
// over those of every call that must not fall between: calls of several threads
// on one stream follow each other whole.
std::mutex g_ops_mu;

bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// ------------------------------------------------------------- rotary

// Frequencies as 2^-64ths of a turn per position. Frequencies up to half a
// turn per position in size (pi radians) are representable; rope's are <= 1.
pda_status rope_turns(const double* inv_freq, int pairs, uint64_t* turns) {
  for (int i = 0; i < pairs; ++i) {
    const double t = inv_freq[i] * 0.15915494309189533577;   // 1 / 2 pi
    if (!(t >= -0.5 && t < 0.5)) return PDA_ERR_INVALID_ARG;  // also NaN
    turns[i] = (uint64_t)(int64_t)std::nearbyint(t * 18446744073709551616.0);
  }
  return PDA_OK;
}

pda_status rope_fill(pda::RopeParams& p, const pda_rope_heads* q, const pda_rope_heads* k, const int64_t* positions,
                     int num_tokens, const double* inv_freq, int rot_dim, int interleaved, float magnitude) {
  if (!q || num_tokens < 0 || q->num_heads <= 0 || (k && k->num_heads < 0)) return PDA_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim % 2 != 0 || !std::isfinite(magnitude)) return PDA_ERR_INVALID_ARG;
  if (rot_dim > kHeadDim) return PDA_ERR_UNSUPPORTED;
  if (rot_dim > 0 && !inv_freq) return PDA_ERR_INVALID_ARG;
  const int hk = k ? k->num_heads : 0;
  if (q->num_heads > 65535 || hk > 65535) return PDA_ERR_UNSUPPORTED;
  p.num_tokens = num_tokens;
  p.num_heads = q->num_heads;
  p.num_kv_heads = hk;
  p.pairs = rot_dim / 2;
  p.interleaved = interleaved ? 1 : 0;
  p.magnitude = magnitude;
  p.positions = positions;
  p.q = static_cast<const __nv_bfloat16*>(q->in);
  p.q_out = static_cast<__nv_bfloat16*>(q->out);
  p.q_tok = q->in_token_stride, p.q_head = q->in_head_stride;
  p.qo_tok = q->out_token_stride, p.qo_head = q->out_head_stride;
  if (k) {
    p.k = static_cast<const __nv_bfloat16*>(k->in);
    p.k_out = static_cast<__nv_bfloat16*>(k->out);
    p.k_tok = k->in_token_stride, p.k_head = k->in_head_stride;
    p.ko_tok = k->out_token_stride, p.ko_head = k->out_head_stride;
  }
  return rope_turns(inv_freq, p.pairs, p.turns);
}

// 16-byte accesses: the base and both strides on the 16-byte grid.
bool rope_on_grid(const void* base, long long tok, long long head) {
  return aligned16(base) && tok % 8 == 0 && head % 8 == 0;
}

template <bool kCache>
pda_status rope_launch(pda::RopeParams& p, bool vec, cudaStream_t stream) {
  const long long T = p.num_tokens;
  if (!vec || p.pairs % 8 != 0) {
    const long long items = T * (p.num_heads + (long long)p.num_kv_heads * (kCache ? 2 : 1));
    const long long blocks = (items + pda::kRopeThreads / 32 - 1) / (pda::kRopeThreads / 32);
    if (blocks > INT32_MAX) return PDA_ERR_UNSUPPORTED;
    pda::pda_rope_any_kernel<kCache><<<(unsigned)blocks, pda::kRopeThreads, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
  }
  // Heads of a CTA: with the cache a kv head's; else as many as leave about
  // four CTAs an SM (every CTA makes its tokens' angles anew).
  const int heads = p.num_heads + p.num_kv_heads;
  const long long tiles4 = (T + 3) / 4, tiles16 = (T + 15) / 16;
  long long groups = kCache ? p.num_kv_heads : (608 + tiles4 - 1) / tiles4;
  if (!kCache && groups > (heads + 7) / 8) groups = (heads + 7) / 8;
  p.groups = (int)groups;
  // Tokens per CTA. With the cache 16, which store whole V rows where the CTA's
  // slots are one run from a multiple of 16 on (us with 16 / 4, 64/8 heads and
  // 64-token blocks: 1024 tokens 12.3 / 22.7, 8192 57.8 / 132.6), from two CTAs
  // an SM on. Other slots take 1-byte stores of V either way: 8192 tokens of
  // packed prompts that start between the CTAs' bounds 110.8 / 133.0, 8192
  // scattered ones 116.2 / 120.6, 2000 37.4 / 35.3.
  if constexpr (kCache) {
    if (tiles16 * groups >= 304) {
      const dim3 grid((unsigned)tiles16, (unsigned)p.groups);
      pda::pda_rope_kernel<16, kCache><<<grid, pda::kRopeThreads, 0, stream>>>(p);
      return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
    }
  }
  // Else 4, or one for the steps of the fewest tokens, which it spreads over
  // more SMs (us with 4 / one a CTA: 256 tokens of 40/8 heads 4.4 / 6.0, with
  // the cache 32/8 heads 7.0 / 10.1, 64 tokens with it 5.8 / 6.2; 16 tokens of
  // 32/8 heads 3.6 / 3.3).
  if (tiles4 * groups >= 128) {
    const dim3 grid((unsigned)tiles4, (unsigned)p.groups);
    pda::pda_rope_kernel<4, kCache><<<grid, pda::kRopeThreads, 0, stream>>>(p);
  } else {
    const dim3 grid((unsigned)T, (unsigned)p.groups);
    pda::pda_rope_kernel<1, kCache><<<grid, pda::kRopeThreads, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

// ------------------------------------------------- attention of new tokens

struct ExtendPlan {
  int tile_tokens;   // new tokens of a full tile (256 rows of g heads)
  int tiles;         // tile slots: room for every sequence's tiles, whatever the lengths
  int nsplit;
  int sms;
  bool ordered;      // more items than SMs: longest first
  size_t bytes;      // of the work queue, and the order or the split partials
};

// What the order holds, the order, and the rows of up to one piece per CTA.
size_t extend_order_bytes(int tiles, int sms) {
  return 256 + align256((size_t)tiles * sizeof(int2)) +
         (size_t)sms * 2 * pda::kExtRows * (kHeadDim + 2) * sizeof(float);
}
size_t extend_split_bytes(long long rows, long long nsplit) {
  return (size_t)(rows * nsplit) * (kHeadDim + 2) * sizeof(float);
}

// The most workspace that a call of up to these sizes (the heads and the block
// size as given) asks for. Fewer tiles get more splits, so each number of tiles
// that is split is looked at, with the most tokens that make so many.
size_t extend_most_bytes(int sms, int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int block_size,
                         int max_blocks) {
  const int tile_tokens = 2 * pda::kExtRows / (num_heads / num_kv_heads);
  const long long tiles = num_tokens / tile_tokens + (long long)num_seqs;
  const int ordered = (int)(tiles < pda::kExtMaxOrdered ? tiles : pda::kExtMaxOrdered);
  size_t most = (long long)ordered * num_kv_heads > sms ? extend_order_bytes(ordered, sms) : 0;
  const long long kv_tiles = ((long long)max_blocks * block_size + pda::kExtTile - 1) / pda::kExtTile;
  for (long long t = 1; t <= tiles; ++t) {
    long long n = sms / (t * num_kv_heads);
    n = n < kv_tiles / 2 ? n : kv_tiles / 2;
    if (n < 2) break;
    const long long tokens = t * tile_tokens - 1 < num_tokens ? t * tile_tokens - 1 : num_tokens;
    const size_t b = extend_split_bytes(tokens * num_heads, n);
    most = b > most ? b : most;
  }
  return kQueueBytes + most;
}

// The tiles, and how many splits of the KV range each gets: one, unless the
// tiles of all kv heads leave SMs idle (one CTA per SM); then as many as fill
// the SMs, of at least two 128-token tiles each at the longest context (GB300,
// us with at least 1 / 2 / 4 tiles: 4 new tokens at 2048 16.1 / 13.2 / 14.7, 16
// at 512 13.4 / 12.8 / 13.7).
// Also opts the kernel in to its shared memory, once per device.
pda_status extend_plan(int dev, int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int block_size,
                       int max_blocks, int window, ExtendPlan* pl) {
  int sms = 0;
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    DeviceInfo& di = g_devices[dev];
    if (!di.extend_set) {
      // The warps trade registers inside what the CTA was launched with: a
      // build with another count must not run.
      cudaFuncAttributes fa;
      if (cudaFuncGetAttributes(&fa, pda::pda_extend_kernel) != cudaSuccess || fa.numRegs != pda::kExtLaunchRegs ||
          cudaFuncSetAttribute(pda::pda_extend_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)pda::kExtSmem) != cudaSuccess)
        return PDA_ERR_CUDA;
      if (cudaDeviceGetAttribute(&di.extend_sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return PDA_ERR_CUDA;
      di.extend_set = true;
    }
    sms = di.extend_sms;
  }
  const int g = num_heads / num_kv_heads;
  pl->tile_tokens = 2 * pda::kExtRows / g;
  pl->tiles = num_tokens / pl->tile_tokens + num_seqs;
  long long tokens = (long long)max_blocks * block_size;
  const long long seen = (long long)window + pl->tile_tokens + pda::kExtTile;   // of a tile's rows, whole KV tiles
  if (window > 0 && seen < tokens) tokens = seen;
  const long long kv_tiles = (tokens + pda::kExtTile - 1) / pda::kExtTile;
  const long long ctas = (long long)pl->tiles * num_kv_heads;
  long long n = sms / ctas;
  n = n < kv_tiles / 2 ? n : kv_tiles / 2;
  pl->nsplit = n < 1 ? 1 : (int)n;
  pl->sms = sms;
  pl->ordered = ctas > sms && pl->tiles <= pda::kExtMaxOrdered;   // then there is one split
  pl->bytes = kQueueBytes;
  if (pl->ordered) pl->bytes += extend_order_bytes(pl->tiles, sms);
  if (pl->nsplit > 1) pl->bytes += extend_split_bytes((long long)num_tokens * num_heads, pl->nsplit);
  return PDA_OK;
}

// -------------------------------------------------------------- pages

// Workspace of a page call (in g_ops_ws, apart from the decode workspace,
// whose queue words have to stay as they are).
size_t page_ws_bytes(long long num_blocks, long long num_rows, long long n) {
  const size_t NB = align256((size_t)num_blocks * 4);
  return kQueueBytes + 256 + align256((size_t)num_rows * 4) + align256((size_t)n * 8) + 3 * NB;
}

pda::PageWs page_ws_layout(void* ptr, long long num_blocks, long long num_rows, long long n) {
  const size_t NB = align256((size_t)num_blocks * 4);
  char* c = static_cast<char*>(ptr) + kQueueBytes;   // pda_extend's queue words stay as they are
  pda::PageWs w;
  w.head = reinterpret_cast<int32_t*>(c);
  c += 256;
  w.fresh = reinterpret_cast<int32_t*>(c);
  c += NB;
  w.moved = reinterpret_cast<int32_t*>(c);
  c += NB;
  w.remap = reinterpret_cast<int32_t*>(c);
  c += NB;
  w.claims = reinterpret_cast<int32_t*>(c);
  c += align256((size_t)num_rows * 4);
  w.reqs = reinterpret_cast<int2*>(c);
  return w;
}

pda_status get_page_workspace(cudaStream_t stream, size_t bytes, void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PDA_ERR_CUDA;
  return grow_workspace(g_ops_ws, dev, stream, bytes, kQueueBytes, out);
}

pda_status page_state(const pda_page_table* t, pda::PageState* st) {
  if (!t || t->num_blocks < 0 || t->num_rows < 0 || t->max_num_blocks_per_seq < 0 || t->block_size <= 0)
    return PDA_ERR_INVALID_ARG;
  if (t->block_size % 16 != 0 || t->block_size > 128 || t->num_blocks > INT32_MAX / 2 ||
      (long long)t->max_num_blocks_per_seq * t->block_size > (long long)INT32_MAX / 2)
    return PDA_ERR_UNSUPPORTED;
  if ((t->num_blocks > 0 && !t->ref_counts) || (t->num_rows > 0 && !t->seq_lens) ||
      (t->num_rows > 0 && t->max_num_blocks_per_seq > 0 && !t->block_tables) || misaligned(t->ref_counts, 4) ||
      misaligned(t->block_tables, 4) || misaligned(t->seq_lens, 4))
    return PDA_ERR_INVALID_ARG;
  st->refs = t->ref_counts;
  st->tables = t->block_tables;
  st->lens = t->seq_lens;
  st->num_blocks = (int)t->num_blocks;
  st->num_rows = t->num_rows;
  st->max_blocks = t->max_num_blocks_per_seq;
  st->block_size = t->block_size;
  return PDA_OK;
}

pda_status check_arrays(const pda_page_array* arrays, int num_arrays) {
  if (num_arrays < 0 || (num_arrays > 0 && !arrays)) return PDA_ERR_INVALID_ARG;
  for (int i = 0; i < num_arrays; ++i)
    if (!arrays[i].base || !aligned16(arrays[i].base) || arrays[i].bytes_per_block <= 0 ||
        arrays[i].bytes_per_block % 16 != 0 || arrays[i].bytes_per_block > (1ll << 40))
      return PDA_ERR_INVALID_ARG;
  return PDA_OK;
}

// A cluster kernel over the pool: one CTA while a pass over the counts is
// short, else a cluster of kPageCluster.
template <typename P>
pda_status launch_cluster(void (*fn)(const P), const P& p, int num_blocks, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  const unsigned ctas = num_blocks <= 8 * pda::kPageThreads ? 1 : pda::kPageCluster;
  lc.gridDim = dim3(ctas);
  lc.blockDim = dim3(pda::kPageThreads);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, fn, p) == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
}

// The copies of p's mode over all arrays, kMaxPageArrays a launch. max_pairs:
// the most pages a call can move. The table entries go with the last launch
// (and a fork's lengths with them): a decode of another thread that falls
// between two of them reads the old ids in arrays that still hold the old pages
// (targets of copies were free).
pda_status launch_copies(pda::CopyParams& p, const pda_page_array* arrays, int num_arrays, long long max_pairs,
                         bool table_work, bool after, cudaStream_t stream) {
  for (int a0 = 0; a0 < num_arrays || (a0 == 0 && table_work); a0 += pda::kMaxPageArrays) {
    const bool last = num_arrays - a0 <= pda::kMaxPageArrays;
    p.tables = table_work && last;
    p.num_arrays = last ? num_arrays - a0 : pda::kMaxPageArrays;
    long long most = 0;
    for (int i = 0; i < p.num_arrays; ++i) {
      p.arrays[i].base = static_cast<uint8_t*>(arrays[a0 + i].base);
      p.arrays[i].bytes = arrays[a0 + i].bytes_per_block;
      most = p.arrays[i].bytes > most ? p.arrays[i].bytes : most;
    }
    p.chunks = (int)((most + pda::kCopyChunk - 1) / pda::kCopyChunk);
    long long items = max_pairs * p.num_arrays * p.chunks;
    if (p.tables) {
      const long long entries = p.mode == pda::kCopyFork
                                    ? (long long)p.n * ((p.st.max_blocks + 127) / 128) * 32
                                    : (long long)p.st.num_rows * p.st.max_blocks;
      const long long t = (entries + pda::kCopyThreads - 1) / pda::kCopyThreads;
      items = t > items ? t : items;
    }
    if (items <= 0) continue;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(items < 152 * 8 ? items : 152 * 8));
    lc.blockDim = dim3(pda::kCopyThreads);
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    if (after && a0 == 0) {
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      lc.attrs = attr;
      lc.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&lc, pda::pda_page_copy_kernel, p) != cudaSuccess) return PDA_ERR_CUDA;
  }
  return PDA_OK;
}

// Grow and fork: the allocation, shared.
pda_status page_alloc(const pda_page_table* table, const int32_t* rows, const int32_t* add, const int32_t* children,
                      int n, pda::AllocParams* p, cudaStream_t stream) {
  void* ws = nullptr;
  pda_status st = get_page_workspace(stream, page_ws_bytes(table->num_blocks, table->num_rows, n), &ws);
  if (st != PDA_OK) return st;
  p->ws = page_ws_layout(ws, table->num_blocks, table->num_rows, n);
  p->rows = rows;
  p->add = add;
  p->children = children;
  p->n = n;
  return launch_cluster(pda::pda_page_alloc_kernel, *p, p->st.num_blocks, stream);
}

}  // namespace

extern "C" {

pda_status pda_rope_frequencies(double* inv_freq, double* magnitude, int rot_dim, double base, int scaling,
                                double factor, double original_length, double low, double high) {
  if (!inv_freq || rot_dim <= 0 || rot_dim % 2 != 0 || rot_dim > kHeadDim) return PDA_ERR_INVALID_ARG;
  if (!std::isfinite(base) || base <= 1.0) return PDA_ERR_INVALID_ARG;
  if (scaling < PDA_ROPE_PLAIN || scaling > PDA_ROPE_BANDS) return PDA_ERR_INVALID_ARG;
  if (scaling != PDA_ROPE_PLAIN && !(std::isfinite(factor) && factor >= 1.0)) return PDA_ERR_INVALID_ARG;
  const bool lengths = scaling == PDA_ROPE_RAMP || scaling == PDA_ROPE_BANDS;
  if (lengths && (!(std::isfinite(original_length) && original_length > 0.0) ||
                  !(std::isfinite(low) && std::isfinite(high) && low > 0.0 && high > low)))
    return PDA_ERR_INVALID_ARG;
  if (scaling == PDA_ROPE_BASE && rot_dim <= 2) return PDA_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  const int n = rot_dim / 2;
  double b = base;
  if (scaling == PDA_ROPE_BASE) b = base * std::pow(factor, rot_dim / (rot_dim - 2.0));
  double ramp0 = 0.0, ramp1 = 0.0;
  if (scaling == PDA_ROPE_RAMP) {
    // the pair index that makes `turns` turns over the original length
    auto at = [&](double turns) {
      return rot_dim * std::log(original_length / (turns * two_pi)) / (2.0 * std::log(base));
    };
    ramp0 = std::fmax(0.0, std::floor(at(high)));
    ramp1 = std::fmin(rot_dim - 1.0, std::ceil(at(low)));
  }
  for (int i = 0; i < n; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == PDA_ROPE_LINEAR) {
      f /= factor;
    } else if (scaling == PDA_ROPE_RAMP) {
      const double t = std::fmin(1.0, std::fmax(0.0, (i - ramp0) / std::fmax(ramp1 - ramp0, 0.001)));
      f = f * (1.0 - t) + f / factor * t;
    } else if (scaling == PDA_ROPE_BANDS) {
      const double turns = original_length * f / two_pi;   // over the original length
      if (turns < low) {
        f /= factor;
      } else if (turns <= high) {
        const double t = (turns - low) / (high - low);
        f = (1.0 - t) * f / factor + t * f;
      }
    }
    inv_freq[i] = f;
  }
  if (magnitude) *magnitude = scaling == PDA_ROPE_RAMP ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return PDA_OK;
}

pda_status pda_rope(const pda_rope_heads* q, const pda_rope_heads* k, const int64_t* positions, int num_tokens,
                    int head_size, const double* inv_freq, int rot_dim, int interleaved, float magnitude,
                    cudaStream_t stream) {
  if (head_size <= 0) return PDA_ERR_INVALID_ARG;
  if (head_size != kHeadDim) return PDA_ERR_UNSUPPORTED;
  pda::RopeParams p = {};
  const pda_status st = rope_fill(p, q, k, positions, num_tokens, inv_freq, rot_dim, interleaved, magnitude);
  if (st != PDA_OK || num_tokens == 0) return st;
  const bool keys = k && k->num_heads > 0;
  if (!positions || misaligned(positions, 8) || !p.q || !p.q_out || (keys && (!p.k || !p.k_out)))
    return PDA_ERR_INVALID_ARG;
  if (misaligned(p.q, 2) || misaligned(p.q_out, 2) || misaligned(p.k, 2) || misaligned(p.k_out, 2))
    return PDA_ERR_INVALID_ARG;
  const bool vec = rope_on_grid(p.q, p.q_tok, p.q_head) && rope_on_grid(p.q_out, p.qo_tok, p.qo_head) &&
                   (!keys || (rope_on_grid(p.k, p.k_tok, p.k_head) && rope_on_grid(p.k_out, p.ko_tok, p.ko_head)));
  return rope_launch<false>(p, vec, stream);
}

pda_status pda_rope_and_cache(const pda_rope_heads* q, const pda_rope_heads* k, const pda_rope_heads* v,
                              const int64_t* positions, const int64_t* slot_mapping, int num_tokens, int head_size,
                              const double* inv_freq, int rot_dim, int interleaved, float magnitude, void* k_cache,
                              void* v_cache, int block_size, long long num_blocks, float k_scale, float v_scale,
                              int kv_layout, cudaStream_t stream) {
  if (head_size <= 0 || block_size <= 0 || num_blocks < 0 || !k || !v) return PDA_ERR_INVALID_ARG;
  if (kv_layout != PDA_KV_NATIVE && kv_layout != PDA_KV_SHUFFLED_V) return PDA_ERR_INVALID_ARG;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale == 0.f || v_scale == 0.f)
    return PDA_ERR_INVALID_ARG;
  if (k->num_heads <= 0 || v->num_heads != k->num_heads) return PDA_ERR_INVALID_ARG;
  if (head_size != kHeadDim || block_size % 16 != 0 || block_size > 128) return PDA_ERR_UNSUPPORTED;
  pda::RopeParams p = {};
  const pda_status st = rope_fill(p, q, k, positions, num_tokens, inv_freq, rot_dim, interleaved, magnitude);
  if (st != PDA_OK || num_tokens == 0) return st;
  p.v = static_cast<const __nv_bfloat16*>(v->in);
  p.v_tok = v->in_token_stride, p.v_head = v->in_head_stride;
  p.k_cache = static_cast<uint8_t*>(k_cache);
  p.v_cache = static_cast<uint8_t*>(v_cache);
  p.slot_mapping = slot_mapping;
  p.block_size = block_size;
  p.num_slots = num_blocks * (long long)block_size;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.v_shuffled = kv_layout == PDA_KV_SHUFFLED_V ? 1 : 0;
  if (!positions || misaligned(positions, 8) || !slot_mapping || misaligned(slot_mapping, 8) || !p.q || !p.q_out ||
      !p.k || !p.v || !k_cache || !v_cache)
    return PDA_ERR_INVALID_ARG;
  if (!aligned16(k_cache) || !aligned16(v_cache) || misaligned(p.q, 2) || misaligned(p.q_out, 2) ||
      misaligned(p.k, 2) || misaligned(p.v, 2))
    return PDA_ERR_INVALID_ARG;
  const bool vec = rope_on_grid(p.q, p.q_tok, p.q_head) && rope_on_grid(p.q_out, p.qo_tok, p.qo_head) &&
                   rope_on_grid(p.k, p.k_tok, p.k_head) && rope_on_grid(p.v, p.v_tok, p.v_head);
  return rope_launch<true>(p, vec, stream);
}

pda_status pda_extend(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const int32_t* query_starts, int num_tokens, int num_seqs,
                      int num_heads, int num_kv_heads, int head_size, int block_size, int max_num_blocks_per_seq,
                      float scale, float k_scale, float v_scale, int window, int kv_layout, const float* sinks,
                      int out_dtype, float output_scale, cudaStream_t stream) {
  pda_status st = validate_sizes(num_seqs, num_heads, num_kv_heads, head_size, block_size, max_num_blocks_per_seq,
                                 scale, k_scale, v_scale);
  if (st != PDA_OK) return st;
  if (num_tokens < 0 || window < 0) return PDA_ERR_INVALID_ARG;
  if (kv_layout != PDA_KV_NATIVE && kv_layout != PDA_KV_SHUFFLED_V) return PDA_ERR_INVALID_ARG;
  if (out_dtype != PDA_OUT_BF16 && out_dtype != PDA_OUT_E4M3) return PDA_ERR_INVALID_ARG;
  if (out_dtype == PDA_OUT_E4M3 && !(std::isfinite(output_scale) && output_scale > 0.f)) return PDA_ERR_INVALID_ARG;
  if (misaligned(sinks, 4)) return PDA_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0) return PDA_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_starts) return PDA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || misaligned(block_tables, 4) ||
      misaligned(seq_lens, 4) || misaligned(query_starts, 4))
    return PDA_ERR_INVALID_ARG;
  if ((long long)num_tokens * num_heads > INT32_MAX) return PDA_ERR_UNSUPPORTED;
  return guarded([&]() -> pda_status {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PDA_ERR_CUDA;
    pda::ExtendParams p = {};
    const double logit = (double)scale * (double)k_scale * 1.4426950408889634;
    p.out = out;
    p.q = static_cast<const __nv_bfloat16*>(q);
    p.k_cache = static_cast<const uint8_t*>(k_cache);
    p.v_cache = static_cast<const uint8_t*>(v_cache);
    p.block_tables = block_tables;
    p.seq_lens = seq_lens;
    p.query_starts = query_starts;
    p.num_tokens = num_tokens;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.gqa = num_heads / num_kv_heads;
    p.gqa_inverse = (65536 + p.gqa - 1) / p.gqa;
    p.block_size = block_size;
    p.max_blocks = max_num_blocks_per_seq;
    p.window = window < (1 << 30) ? window : 1 << 30;   // no position is that large
    p.logit_scale_log2 = (float)std::fabs(logit);
    p.negate = logit < 0.0 ? 1 : 0;
    p.v_scale = v_scale;
    p.sinks = sinks;
    p.out_fp8 = out_dtype == PDA_OUT_E4M3;
    p.out_scale = output_scale;
    p.v_shuffled = kv_layout == PDA_KV_SHUFFLED_V ? 1 : 0;
    p.block_limit = g_block_limit.load();
    ExtendPlan pl;
    pda_status st = extend_plan(dev, num_tokens, num_seqs, num_heads, num_kv_heads, block_size,
                                max_num_blocks_per_seq, window, &pl);
    if (st != PDA_OK) return st;
    void* ws = nullptr;
    std::lock_guard<std::mutex> lk(g_ops_mu);
    st = grow_workspace(g_ops_ws, dev, stream, pl.bytes, kQueueBytes, &ws);
    if (st == PDA_ERR_WORKSPACE) {
      // captured without pda_reserve_extend: one split, and the items dealt
      // out in turn, need no workspace
      pl.nsplit = 1;
      st = PDA_OK;
    }
    if (st != PDA_OK) return st;
    p.tile_tokens = pl.tile_tokens;
    p.tiles = pl.tiles;
    p.nsplit = pl.nsplit;
    p.queue = static_cast<unsigned*>(ws);
    if (pl.nsplit > 1) {
      p.part_o = reinterpret_cast<float*>(static_cast<char*>(ws) + kQueueBytes);
      p.part_ml = p.part_o + (size_t)num_tokens * num_heads * pl.nsplit * kHeadDim;
    }
    const long long items = (long long)pl.tiles * num_kv_heads * pl.nsplit;
    if (items > INT32_MAX / 2) return PDA_ERR_UNSUPPORTED;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3((unsigned)(items < pl.sms ? items : pl.sms));
    lc.blockDim = dim3(pda::kExtThreads);
    lc.dynamicSmemBytes = pda::kExtSmem;
    lc.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    if (pl.ordered && ws) {
      char* at = static_cast<char*>(ws) + kQueueBytes;
      pda::ExtendHead* head = reinterpret_cast<pda::ExtendHead*>(at);
      int2* order = reinterpret_cast<int2*>(at + 256);
      p.tail_o = reinterpret_cast<float*>(at + 256 + align256((size_t)pl.tiles * sizeof(int2)));
      p.tail_ml = p.tail_o + (size_t)pl.sms * 2 * pda::kExtRows * kHeadDim;
      pda::pda_extend_order_kernel<<<1, pda::kExtOrderThreads, 0, stream>>>(p, order, head, pl.sms);
      if (cudaGetLastError() != cudaSuccess) return PDA_ERR_CUDA;
      p.order = order;
      p.head = head;
      lc.attrs = attr;
      lc.numAttrs = 1;
    }
    if (cudaLaunchKernelEx(&lc, pda::pda_extend_kernel, p) != cudaSuccess) return PDA_ERR_CUDA;
    if (p.order) {
      lc.gridDim = dim3(pda::kExtTailBlocks, (unsigned)(pl.sms + 1) / 2);   // two pieces an item at least
      lc.blockDim = dim3(pda::kExtTailRows * 32);
      lc.dynamicSmemBytes = 0;
      return cudaLaunchKernelEx(&lc, pda::pda_extend_tail_kernel, p) == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
    }
    if (pl.nsplit == 1) return PDA_OK;
    pda::ExtendMergeParams m = {};
    m.out = out;
    m.part_o = p.part_o;
    m.part_ml = p.part_ml;
    m.query_starts = query_starts;
    m.num_tokens = num_tokens;
    m.num_seqs = num_seqs;
    m.num_heads = num_heads;
    m.nsplit = pl.nsplit;
    m.v_scale = v_scale;
    m.sinks = sinks;
    m.out_fp8 = p.out_fp8;
    m.out_scale = output_scale;
    const long long rows = (long long)num_tokens * num_heads;
    lc.gridDim = dim3((unsigned)((rows + pda::kMergeRowsPerBlock - 1) / pda::kMergeRowsPerBlock));
    lc.blockDim = dim3(kHeadDim);
    lc.dynamicSmemBytes = 0;
    lc.attrs = attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, pda::pda_extend_merge_kernel, m) == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
  });
}

pda_status pda_reserve_extend(int num_tokens, int num_seqs, int num_heads, int num_kv_heads,
                              int max_num_blocks_per_seq, int block_size, cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    pda_status st = validate_sizes(num_seqs, num_heads, num_kv_heads, kHeadDim, block_size, max_num_blocks_per_seq,
                                   1.f, 1.f, 1.f);
    if (st != PDA_OK) return st;
    if (num_tokens < 0) return PDA_ERR_INVALID_ARG;
    if ((long long)num_tokens * num_heads > INT32_MAX) return PDA_ERR_UNSUPPORTED;
    if (num_tokens == 0 || num_seqs == 0) return PDA_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PDA_ERR_CUDA;
    ExtendPlan pl;
    st = extend_plan(dev, num_tokens, num_seqs, num_heads, num_kv_heads, block_size, max_num_blocks_per_seq, 0, &pl);
    if (st != PDA_OK) return st;
    const size_t bytes = extend_most_bytes(pl.sms, num_tokens, num_seqs, num_heads, num_kv_heads, block_size,
                                           max_num_blocks_per_seq);
    void* ws = nullptr;
    return grow_workspace(g_ops_ws, dev, stream, bytes, kQueueBytes, &ws);
  });
}

pda_status pda_copy_pages(const pda_page_array* arrays, int num_arrays, const int32_t* src, const int32_t* dst,
                          int num_pairs, long long num_blocks, cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    const pda_status st = check_arrays(arrays, num_arrays);
    if (st != PDA_OK) return st;
    if (num_pairs < 0 || num_blocks < 0) return PDA_ERR_INVALID_ARG;
    if (num_blocks > INT32_MAX) return PDA_ERR_UNSUPPORTED;
    if (num_pairs == 0 || num_arrays == 0) return PDA_OK;
    if (!src || !dst || misaligned(src, 4) || misaligned(dst, 4)) return PDA_ERR_INVALID_ARG;
    pda::CopyParams p = {};
    p.mode = pda::kCopyPairs;
    p.src = src;
    p.dst = dst;
    p.n = num_pairs;
    p.st.num_blocks = (int)num_blocks;
    std::lock_guard<std::mutex> lk(g_ops_mu);
    return launch_copies(p, arrays, num_arrays, num_pairs, false, false, stream);
  });
}

pda_status pda_grow_pages(const pda_page_table* table, const int32_t* rows, const int32_t* add, int n,
                          cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    pda::AllocParams p = {};
    const pda_status st = page_state(table, &p.st);
    if (st != PDA_OK) return st;
    if (n < 0) return PDA_ERR_INVALID_ARG;
    if (n == 0) return PDA_OK;
    if (!rows || !add || misaligned(rows, 4) || misaligned(add, 4)) return PDA_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lk(g_ops_mu);
    return page_alloc(table, rows, add, nullptr, n, &p, stream);
  });
}

pda_status pda_fork_pages(const pda_page_table* table, const int32_t* parents, const int32_t* children, int n,
                          const pda_page_array* arrays, int num_arrays, cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    pda::AllocParams p = {};
    pda_status st = page_state(table, &p.st);
    if (st == PDA_OK) st = check_arrays(arrays, num_arrays);
    if (st != PDA_OK) return st;
    if (n < 0) return PDA_ERR_INVALID_ARG;
    if (n == 0) return PDA_OK;
    if (!parents || !children || misaligned(parents, 4) || misaligned(children, 4)) return PDA_ERR_INVALID_ARG;
    std::lock_guard<std::mutex> lk(g_ops_mu);
    st = page_alloc(table, parents, nullptr, children, n, &p, stream);
    if (st != PDA_OK) return st;
    pda::CopyParams c = {};
    c.st = p.st;
    c.ws = p.ws;
    c.mode = pda::kCopyFork;
    c.rows = parents;
    c.children = children;
    c.n = n;
    return launch_copies(c, arrays, num_arrays, n, true, true, stream);
  });
}

pda_status pda_free_pages(const pda_page_table* table, const int32_t* rows, int n, cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    pda::FreeParams p = {};
    const pda_status st = page_state(table, &p.st);
    if (st != PDA_OK) return st;
    if (n < 0) return PDA_ERR_INVALID_ARG;
    if (n == 0) return PDA_OK;
    if (!rows || misaligned(rows, 4)) return PDA_ERR_INVALID_ARG;
    p.rows = rows;
    p.n = n;
    std::lock_guard<std::mutex> lk(g_ops_mu);
    pda::pda_page_free_kernel<<<(unsigned)n, 128, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? PDA_OK : PDA_ERR_CUDA;
  });
}

pda_status pda_compact_pages(const pda_page_table* table, const pda_page_array* arrays, int num_arrays,
                             int32_t* new_ids, cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    pda::CompactParams p = {};
    pda_status st = page_state(table, &p.st);
    if (st == PDA_OK) st = check_arrays(arrays, num_arrays);
    if (st == PDA_OK && misaligned(new_ids, 4)) st = PDA_ERR_INVALID_ARG;
    if (st != PDA_OK || table->num_blocks == 0) return st;
    p.new_ids = new_ids;
    void* ws = nullptr;
    std::lock_guard<std::mutex> lk(g_ops_mu);
    st = get_page_workspace(stream, page_ws_bytes(table->num_blocks, table->num_rows, 0), &ws);
    if (st != PDA_OK) return st;
    p.ws = page_ws_layout(ws, table->num_blocks, table->num_rows, 0);
    st = launch_cluster(pda::pda_page_compact_kernel, p, p.st.num_blocks, stream);
    if (st != PDA_OK) return st;
    pda::CopyParams c = {};
    c.st = p.st;
    c.ws = p.ws;
    c.mode = pda::kCopyCompact;
    return launch_copies(c, arrays, num_arrays, table->num_blocks / 2 + 1, true, true, stream);
  });
}

pda_status pda_reserve_pages(long long num_blocks, int num_rows, int max_requests, cudaStream_t stream) {
  return guarded([&]() -> pda_status {
    if (num_blocks < 0 || num_rows < 0 || max_requests < 0) return PDA_ERR_INVALID_ARG;
    if (num_blocks > INT32_MAX / 2) return PDA_ERR_UNSUPPORTED;
    void* ws = nullptr;
    return get_page_workspace(stream, page_ws_bytes(num_blocks, num_rows, max_requests), &ws);
  });
}

}  // extern "C"
