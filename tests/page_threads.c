/* Calls of several threads on one stream, without an interpreter between them. */
#include <pthread.h>
#include <stddef.h>

#include "pda.h"

struct work {
  const pda_page_table* table;
  const pda_page_array* arrays;
  int num_arrays;
  const int32_t* rows;
  const int32_t* add;
  int n, loops;
  cudaStream_t stream;
  int status;
};

static void* churn(void* arg) {
  struct work* w = arg;
  for (int i = 0; i < w->loops && w->status == PDA_OK; ++i) {
    for (int j = 0; j < w->n && w->status == PDA_OK; ++j)
      w->status = pda_free_pages(w->table, w->rows + j, 1, w->stream);
    if (w->status == PDA_OK) w->status = pda_grow_pages(w->table, w->rows, w->add, w->n, w->stream);
  }
  return NULL;
}

static void* compact(void* arg) {
  struct work* w = arg;
  for (int i = 0; i < w->loops && w->status == PDA_OK; ++i)
    w->status = pda_compact_pages(w->table, w->arrays, w->num_arrays, NULL, w->stream);
  return NULL;
}

/* Two threads free and grow rows of their own (the holes of one make the
 * compaction move the other's pages), a third compacts. Returns the first
 * status that is not PDA_OK. */
int churn_beside_compaction(const pda_page_table* table, const pda_page_array* arrays, int num_arrays,
                            const int32_t* rows, const int32_t* add, int n, int loops, cudaStream_t stream) {
  struct work w[3];
  pthread_t t[3];
  int started = 0, status = PDA_OK;
  for (int i = 0; i < 3; ++i) {
    w[i] = (struct work){table, arrays, num_arrays, rows + (i == 1 ? n : 0), add, n, loops, stream, PDA_OK};
    if (pthread_create(&t[i], NULL, i < 2 ? churn : compact, &w[i]) != 0) break;
    ++started;
  }
  for (int i = 0; i < started; ++i) {
    pthread_join(t[i], NULL);
    if (status == PDA_OK) status = w[i].status;
  }
  return started == 3 ? status : -1;
}

struct decodes {
  const pda_page_table* table;
  const void *q, *k, *v;
  char* out;
  size_t out_bytes;   /* of one call's output */
  int heads, kv_heads, loops;
  cudaStream_t stream;
  pthread_barrier_t* gate;
  int status;
};

static void* decode(void* arg) {
  struct decodes* w = arg;
  const pda_page_table* t = w->table;
  pthread_barrier_wait(w->gate);
  for (int i = 0; i < w->loops && w->status == PDA_OK; ++i)
    w->status = pda_decode(w->out + (size_t)i * w->out_bytes, w->q, w->k, w->v, t->block_tables, t->seq_lens, t->num_rows,
                           w->heads, w->kv_heads, 128, t->block_size, t->max_num_blocks_per_seq, 0.1f, 0.05f, 0.05f,
                           w->stream);
  return NULL;
}

/* One thread decodes every row of the table `loops` times, one output behind
 * the other, while the caller's compacts (parents NULL) or forks. */
int decode_beside_pages(const pda_page_table* table, const pda_page_array* arrays, int num_arrays,
                        const int32_t* parents, const int32_t* children, int n, const void* q, int heads, int kv_heads,
                        void* out, size_t out_bytes, int loops, cudaStream_t stream) {
  pthread_barrier_t gate;
  if (pthread_barrier_init(&gate, NULL, 2) != 0) return -1;
  struct decodes w = {table, q, arrays[0].base, arrays[num_arrays - 1].base, out, out_bytes, heads, kv_heads, loops,
                      stream, &gate, PDA_OK};
  pthread_t t;
  if (pthread_create(&t, NULL, decode, &w) != 0) return -1;
  pthread_barrier_wait(&gate);
  const int status = parents ? pda_fork_pages(table, parents, children, n, arrays, num_arrays, stream)
                             : pda_compact_pages(table, arrays, num_arrays, NULL, stream);
  pthread_join(t, NULL);
  pthread_barrier_destroy(&gate);
  return status != PDA_OK ? status : w.status;
}
