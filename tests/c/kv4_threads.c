/* Calls of csa_kv4_decode from several host threads at once: `repeat` of each
 * of n calls, a thread to a call.  Returns the largest status that came back. */
#include <pthread.h>
#include <stdint.h>

#include "csa.h"

typedef struct {
  const csa_shape* shape;
  const csa_kv4* cache;
  int T, repeat;
  const void* q;
  const csa_strides* qs;
  const int64_t* len;
  float* o;
  void* workspace;
  size_t workspace_bytes;
  void* stream;
  int status;
} call;

static void* run(void* p) {
  call* c = (call*)p;
  for (int i = 0; i < c->repeat; ++i) {
    const int st = csa_kv4_decode(c->shape, c->cache, c->T, c->q, c->qs, c->len, 0, c->o, 0, c->workspace,
                                  c->workspace_bytes, c->stream);
    if (st > c->status) c->status = st;
  }
  return 0;
}

int run_calls(call* calls, int n) {
  pthread_t id[16];
  int made = 0, worst = 0;
  for (; made < n && made < 16; ++made)
    if (pthread_create(&id[made], 0, run, &calls[made])) break;
  for (int i = 0; i < made; ++i) {
    pthread_join(id[i], 0);
    if (calls[i].status > worst) worst = calls[i].status;
  }
  return made == n ? worst : -1;
}
