/*
 * c_experts_client.c -- a layer of FP4 experts from plain C: the routing sort,
 * tokens into expert order, capture with tiled scales, the product with and
 * without a workspace, the weighted sum back and its gradients, through the C ABI
 * in include/trace_fp4.h.  A few argument errors are checked on the way.  Inputs
 * and outputs go to a binary file for the test:  c_experts_client OUT_FILE
 *
 * Output file, in this order: ids (int32), weights (float), x and w (bf16), offsets
 * (int64[E+2]), rows, slots (int32), y (bf16 [slots, COLS]), a codes, a scales
 * (tiled), a gscale (float[E+1]), w codes, w scales (row-major), w gscale
 * (float[E]), product twice (bf16 [slots, N]), out (bf16 [T, N]), grad_y (bf16),
 * grad_weights (float).  The gradient of out is out itself.
 */
#include <cuda_runtime_api.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "trace_fp4.h"

#define T 50
#define K 3
#define E 4
#define COLS 192
#define N 72
#define S (T * K)

static uint32_t lcg_state = 99u;
static uint32_t lcg(void) {
  lcg_state = lcg_state * 1664525u + 1013904223u;
  return lcg_state >> 8;
}

#define CK(call)                                                         \
  do {                                                                   \
    cudaError_t e_ = (call);                                             \
    if (e_ != cudaSuccess) {                                             \
      fprintf(stderr, "%s failed: %s\n", #call, cudaGetErrorString(e_)); \
      return 2;                                                          \
    }                                                                    \
  } while (0)

#define TK(call, want)                                                 \
  do {                                                                 \
    int s_ = (call);                                                   \
    if (s_ != (want)) {                                                \
      fprintf(stderr, "%s returned %d (%s), expected %d\n", #call, s_, \
              trace_strerror(s_), (want));                             \
      return 3;                                                        \
    }                                                                  \
  } while (0)

static uint16_t rand_bf16(void) { /* 2^-3 .. 2^3, either sign */
  return (uint16_t)(((lcg() & 1u) << 15) | ((124u + lcg() % 6u) << 7) | (lcg() & 0x7Fu));
}

static int put(FILE* f, const void* device, size_t bytes) {
  void* h = malloc(bytes);
  if (cudaMemcpy(h, device, bytes, cudaMemcpyDeviceToHost) != cudaSuccess) return 1;
  const int bad = fwrite(h, 1, bytes, f) != bytes;
  free(h);
  return bad;
}

int main(int argc, char** argv) {
  if (argc != 2) return 1;
  static int32_t ids[S];
  static float p[S];
  static uint16_t x[T * COLS], w[E * N * COLS];
  int64_t w_bounds[E + 1];
  for (int i = 0; i < S; ++i) ids[i] = (int32_t)(lcg() % (E + 2)) - 1; /* both ends dropped */
  for (int i = 0; i < S; ++i) p[i] = (float)(lcg() % 1000u) / 1000.0f;
  for (int i = 0; i < T * COLS; ++i) x[i] = rand_bf16();
  for (int i = 0; i < E * N * COLS; ++i) w[i] = rand_bf16();
  for (int e = 0; e <= E; ++e) w_bounds[e] = (int64_t)e * N;

  /* one allocation for each array, in the order of the file */
  enum { IDS, P, X, W, OFFS, ROWS, SLOTS, Y, AC, AS, AG, WC, WS, WG, OUT1, OUT2, OUT, GY, GP,
         MB, WB, SORT_WS, CAP_WS, MM_WS, COUNT };
  const size_t as_bytes = trace_scale_bytes(S, COLS, 16, TRACE_SCALES_TILED_128x4);
  const size_t sort_ws = trace_moe_sort_workspace_bytes(T, K, E);
  const size_t cap_ws = trace_capture_workspace_bytes(E * N, COLS, E + 1);
  const size_t mm_ws = trace_fp4_matmul_workspace_bytes(S, COLS, E + 1, TRACE_SCALES_TILED_128x4, N,
                                                        E, TRACE_SCALES_ROW_MAJOR);
  const size_t bytes[COUNT] = {sizeof ids, sizeof p, sizeof x, sizeof w, (E + 2) * 8, S * 4, S * 4,
                               S * COLS * 2, S * COLS / 2, as_bytes, (E + 1) * 4, E * N * COLS / 2,
                               E * N * COLS / 16, E * 4, S * N * 2, S * N * 2, T * N * 2, S * N * 2,
                               S * 4, E * N * COLS / 8, sizeof w_bounds, sort_ws, cap_ws,
                               mm_ws ? mm_ws : 256};
  void* d[COUNT];
  for (int i = 0; i < COUNT; ++i) {
    CK(cudaMalloc(&d[i], bytes[i]));
    CK(cudaMemset(d[i], i == CAP_WS || i == AS ? 0 : 0xA5, bytes[i]));
  }
  CK(cudaMemcpy(d[IDS], ids, sizeof ids, cudaMemcpyHostToDevice));
  CK(cudaMemcpy(d[P], p, sizeof p, cudaMemcpyHostToDevice));
  CK(cudaMemcpy(d[X], x, sizeof x, cudaMemcpyHostToDevice));
  CK(cudaMemcpy(d[W], w, sizeof w, cudaMemcpyHostToDevice));
  CK(cudaMemcpy(d[WB], w_bounds, sizeof w_bounds, cudaMemcpyHostToDevice));
  cudaStream_t st;
  CK(cudaStreamCreate(&st));

  /* argument errors return before anything is enqueued */
  TK(trace_moe_sort(d[IDS], 3, T, K, E, d[OFFS], d[ROWS], d[SLOTS], d[SORT_WS], sort_ws, st),
     TRACE_ERR_SHAPE);
  TK(trace_moe_combine(d[Y], T, K, N + 8, d[ROWS], d[P], d[OUT], st), TRACE_ERR_SHAPE);
  TK(trace_fp4_matmul(d[AC], d[AS], NULL, S, COLS, E + 1, d[OFFS], 1, d[WC], d[WS], d[WG], N, E, 0,
                      d[OUT1], st), TRACE_ERR_NULL);

  TK(trace_capture(d[W], E * N, COLS, E, d[WB], d[WC], d[MB], d[WS], d[WG], d[CAP_WS], cap_ws, st),
     TRACE_OK);
  TK(trace_moe_sort(d[IDS], 4, T, K, E, d[OFFS], d[ROWS], d[SLOTS], d[SORT_WS], sort_ws, st),
     TRACE_OK);
  TK(trace_moe_dispatch(d[X], T, K, COLS, d[ROWS], d[SLOTS], d[Y], st), TRACE_OK);
  TK(trace_capture_ex(d[Y], S, COLS, E + 1, d[OFFS], d[AC], d[MB], d[AS], d[AG], d[CAP_WS], cap_ws,
                      TRACE_SCALES_TILED_128x4, st), TRACE_OK);
  TK(trace_fp4_matmul(d[AC], d[AS], d[AG], S, COLS, E + 1, d[OFFS], TRACE_SCALES_TILED_128x4, d[WC],
                      d[WS], d[WG], N, E, TRACE_SCALES_ROW_MAJOR, d[OUT1], st), TRACE_OK);
  TK(trace_fp4_matmul_ws(d[AC], d[AS], d[AG], S, COLS, E + 1, d[OFFS], TRACE_SCALES_TILED_128x4,
                         d[WC], d[WS], d[WG], N, E, TRACE_SCALES_ROW_MAJOR, d[OUT2], d[MM_WS],
                         bytes[MM_WS], st), TRACE_OK);
  TK(trace_matmul_status(st), TRACE_OK);
  /* rows of N columns are no multiple of 32 for the token kernels: the first 64 go back */
  const int64_t back = 64;
  CK(cudaMemcpy2DAsync(d[Y], back * 2, d[OUT1], N * 2, back * 2, S, cudaMemcpyDeviceToDevice, st));
  TK(trace_moe_combine(d[Y], T, K, back, d[ROWS], d[P], d[OUT], st), TRACE_OK);
  TK(trace_moe_combine_bwd(d[OUT], d[Y], T, K, back, d[ROWS], d[SLOTS], d[P], d[GY], d[GP], st),
     TRACE_OK);
  TK(trace_moe_dispatch(d[X], T, K, COLS, d[ROWS], d[SLOTS], d[Y], st), TRACE_OK);
  CK(cudaStreamSynchronize(st));

  FILE* f = fopen(argv[1], "wb");
  if (!f) return 5;
  for (int i = 0; i <= GP; ++i)
    if (put(f, d[i], bytes[i])) return 6;
  fclose(f);
  printf("c_experts_client: ok\n");
  return 0;
}
