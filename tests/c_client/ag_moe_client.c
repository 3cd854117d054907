/*
 * A plain C user of include/ag_moe.h: three tokens, two experts, one choice each, small
 * whole numbers.  Routes, gathers, multiplies by the experts' matrices (the unit matrix
 * and twice it) and combines; prints what it finds wrong.  Exit status 0 on success.
 */
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "ag_moe.h"

enum { T = 3, E = 2, TOP_K = 1, K = 8, N = 8 };

#define CUDA_OK(call)                                             \
  do {                                                            \
    cudaError_t e_ = (call);                                      \
    if (e_ != cudaSuccess) {                                      \
      fprintf(stderr, "%s: %s\n", #call, cudaGetErrorString(e_)); \
      return 1;                                                   \
    }                                                             \
  } while (0)
#define AG_OK(call)                                                  \
  do {                                                               \
    if ((call) < 0) {                                                \
      fprintf(stderr, "%s: %s\n", #call, ag_gemm_last_error_message()); \
      return 1;                                                      \
    }                                                                \
  } while (0)
#define SAME(got, want)                                    \
  do {                                                     \
    if (memcmp((got), (want), sizeof(want)) != 0) {        \
      fprintf(stderr, "%s differs from %s\n", #got, #want); \
      return 1;                                            \
    }                                                      \
  } while (0)

/* fp16 bits of a whole number from 0 to 16 */
static uint16_t half_of(int v) {
  int e = 0;
  if (v == 0) return 0;
  while ((v >> e) > 1) ++e;
  return (uint16_t)(((15 + e) << 10) | ((v - (1 << e)) << (10 - e)));
}

int main(void) {
  const float logits[T * E] = {1, 0, 0, 1, 2, 1};
  const int32_t want_offsets[E + 1] = {0, 2, 3}, want_order[T] = {0, 2, 1}, want_slots[T] = {0, 2, 1};
  const float one[T] = {1, 1, 1};
  uint16_t x[T * K], w[E * K * N];
  float want[T * N], y[T * N], weights[T], out[T * N];
  int32_t offsets[E + 1], order[T], slots[T];
  void *d_logits, *d_weights, *d_experts, *d_offsets, *d_order, *d_slots, *d_x, *d_rows, *d_w, *d_y, *d_out;
  ag_moe_plan* plan;
  int t, i, e;

  for (t = 0; t < T; ++t)
    for (i = 0; i < K; ++i) {
      x[t * K + i] = half_of(t + i);
      want[t * N + i] = (float)((t + i) * (t == 1 ? 2 : 1)); /* token 1 goes to expert 1 */
    }
  memset(w, 0, sizeof(w));
  for (e = 0; e < E; ++e)
    for (i = 0; i < K; ++i) w[(e * K + i) * N + i] = half_of(e + 1);

  if (ag_moe_route_workspace(T, 0, TOP_K) != AG_GEMM_ERR_INVALID || ag_moe_plan_create(E, K, 12, AG_GEMM_F16) != NULL ||
      ag_gemm_last_error() != AG_GEMM_ERR_INVALID) {
    fprintf(stderr, "bad sizes were accepted\n");
    return 1;
  }
  CUDA_OK(cudaMalloc(&d_logits, sizeof(logits)));
  CUDA_OK(cudaMalloc(&d_weights, sizeof(weights)));
  CUDA_OK(cudaMalloc(&d_experts, T * 4));
  CUDA_OK(cudaMalloc(&d_offsets, sizeof(offsets)));
  CUDA_OK(cudaMalloc(&d_order, sizeof(order)));
  CUDA_OK(cudaMalloc(&d_slots, sizeof(slots)));
  CUDA_OK(cudaMalloc(&d_x, sizeof(x)));
  CUDA_OK(cudaMalloc(&d_rows, sizeof(x)));
  CUDA_OK(cudaMalloc(&d_w, sizeof(w)));
  CUDA_OK(cudaMalloc(&d_y, sizeof(y)));
  CUDA_OK(cudaMalloc(&d_out, sizeof(out)));
  CUDA_OK(cudaMemcpy(d_logits, logits, sizeof(logits), cudaMemcpyHostToDevice));
  CUDA_OK(cudaMemcpy(d_x, x, sizeof(x), cudaMemcpyHostToDevice));
  CUDA_OK(cudaMemcpy(d_w, w, sizeof(w), cudaMemcpyHostToDevice));

  if (ag_moe_route_workspace(T, E, TOP_K) != 0) return 1;
  AG_OK(ag_moe_route(T, E, TOP_K, AG_MOE_F32, d_logits, E, 1, d_weights, d_experts, d_offsets, d_order, d_slots, NULL,
                     NULL));
  AG_OK(ag_moe_gather(T, TOP_K, K, AG_GEMM_F16, d_x, K, d_order, d_rows, NULL));
  plan = ag_moe_plan_create(E, K, N, AG_GEMM_F16);
  if (!plan) {
    fprintf(stderr, "%s\n", ag_gemm_last_error_message());
    return 1;
  }
  AG_OK(ag_moe_forward(plan, T * TOP_K, d_rows, K, d_offsets, d_w, N, K * N, d_y, N, AG_MOE_F32, NULL));
  AG_OK(ag_moe_combine(T, TOP_K, N, AG_MOE_F32, d_y, N, d_slots, d_weights, d_out, NULL));
  AG_OK(ag_moe_plan_status(plan));
  ag_moe_plan_destroy(plan);

  CUDA_OK(cudaMemcpy(offsets, d_offsets, sizeof(offsets), cudaMemcpyDeviceToHost));
  CUDA_OK(cudaMemcpy(order, d_order, sizeof(order), cudaMemcpyDeviceToHost));
  CUDA_OK(cudaMemcpy(slots, d_slots, sizeof(slots), cudaMemcpyDeviceToHost));
  CUDA_OK(cudaMemcpy(weights, d_weights, sizeof(weights), cudaMemcpyDeviceToHost));
  CUDA_OK(cudaMemcpy(out, d_out, sizeof(out), cudaMemcpyDeviceToHost));
  SAME(offsets, want_offsets);
  SAME(order, want_order);
  SAME(slots, want_slots);
  SAME(weights, one);
  SAME(out, want);
  return 0;
}
