/* Two kinds of ccl_moe_sort in host threads of one process: sorts that need 72
 * KB of shared memory per CTA and sorts that need 49 KB, each thread on a stream
 * of its own.  Neither may be refused for what the other one asks.  Exit status
 * 0 when every call of every thread returned CCL_OK, 1 otherwise (the first
 * failing call's reason is on stderr). */
#include <pthread.h>
#include <stdio.h>
#include <stdlib.h>

#include <cuda_runtime_api.h>

#include "ccl.h"

enum { TOKENS = 20000, CALLS = 20000, THREADS = 4 };

static void* sorts(void* arg) {
  const int experts = *(const int*)arg;
  const size_t tokens = TOKENS;
  int32_t* base = NULL;
  cudaStream_t stream = NULL;
  if (cudaMalloc((void**)&base, sizeof(int32_t) * (2 * TOKENS + 2048)) != cudaSuccess ||
      cudaMemset(base, 0, sizeof(int32_t) * TOKENS) != cudaSuccess || cudaStreamCreate(&stream) != cudaSuccess ||
      cudaDeviceSynchronize() != cudaSuccess) {
    fprintf(stderr, "set-up failed\n");
    return arg;
  }
  const int32_t* ids[1] = {base};
  int32_t* rows[1] = {base + TOKENS};
  int32_t* offsets[1] = {base + 2 * TOKENS};
  void* bad = NULL;
  for (int i = 0; i < CALLS && bad == NULL; ++i) {
    if (ccl_moe_sort(ids, &tokens, 1, 1, experts, NULL, offsets, rows, stream) != CCL_OK) {
      fprintf(stderr, "call %d of %d experts: %s\n", i, experts, ccl_last_error());
      bad = arg;
    }
  }
  if (cudaStreamSynchronize(stream) != cudaSuccess) bad = arg;
  cudaStreamDestroy(stream);
  cudaFree(base);
  return bad;
}

int main(void) {
  static int experts[THREADS] = {1024, 700, 1024, 700};
  pthread_t threads[THREADS];
  int failed = 0;
  for (int i = 0; i < THREADS; ++i)
    if (pthread_create(&threads[i], NULL, sorts, &experts[i]) != 0) return 2;
  for (int i = 0; i < THREADS; ++i) {
    void* bad = NULL;
    pthread_join(threads[i], &bad);
    failed |= bad != NULL;
  }
  return failed;
}
