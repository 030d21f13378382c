/* Page calls of three threads on one stream, without an interpreter between
 * them: two free and grow rows of their own (the holes of one make the
 * compaction move the other's pages), the third compacts. Returns the first
 * status that is not PDA_OK. */
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
