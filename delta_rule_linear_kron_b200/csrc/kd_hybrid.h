// kd_hybrid.h -- internal launch interface of the operators that stand beside
// the delta rules in a hybrid stack: rotary positions, sliding-window
// attention, the element-wise gated linear recurrence.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kd_kernels.h"

namespace kd {

struct RotaryArgs {
  const void* x[2];  // q, k
  void* y[2];
  int heads[2];
  const double* freqs;
  const long long* pos;
  long long rows;  // B * T
  int T, d, rot, interleaved, inverse, dtype;
  float scale;
};
cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st);

struct SwaArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  const void *o, *dO;  // backward: the forward's output and its gradient
  const float* lse_in;
  void *dq, *dk, *dv;
  int B, T, H, Hk, d, window, sinks, dtype;
  float scale;
  void* olo;            // bf16: the output's rounding, written by the forward
  const void* olo_in;
  char* ws;             // backward scratch (SwaBwdLayout)
  int* err = nullptr;   // the library's device error word
};

// Backward scratch.  lse2 and delta are [B][H][Tp] fp32 (Tp = T rounded up to
// 128; lse2 = lse * log2 e, +inf behind T, so that the probability is 0
// there).  The far queries of a first token, those beyond the band of its key
// tile, are taken by `pieces` work items per query head, and each writes its
// part of dk and dv of the first `sinks` rows: part[2][piece][B][H][sinks][d].
// The band items write theirs to band[2][B][Hk][sinks][d].
struct SwaBwdLayout {
  int Tp = 0, pieces = 0;
  size_t lse2 = 0, delta = 0, part = 0, band = 0, bytes = 0;
};
// queries of one far item; backward in us with 1024, 2048, 4096: 307, 300, 296 at
// T16384 H16 Hk4 window 256 (the sums grow with the pieces), 76, 81, 104 at B2
// T4096 H8 Hk2 d64 window 128 (too few items)
constexpr int kSwaPiece = 2048;
SwaBwdLayout swa_bwd_layout(int B, int T, int H, int Hk, int d, int window, int sinks);

bool swa_tc_supported(int dtype);
cudaError_t launch_swa_fwd_simt(const SwaArgs& a, cudaStream_t st);
cudaError_t launch_swa_bwd_simt(const SwaArgs& a, cudaStream_t st);
cudaError_t launch_swa_fwd_tc(const SwaArgs& a, cudaStream_t st);
cudaError_t launch_swa_bwd_tc(const SwaArgs& a, cudaStream_t st);
// the backward's passes around the products, shared by both paths
cudaError_t launch_swa_delta(const SwaArgs& a, const SwaBwdLayout& L, cudaStream_t st);
cudaError_t launch_swa_sink_sum(const SwaArgs& a, const SwaBwdLayout& L, int tile, cudaStream_t st);

struct SwaDecodeArgs {
  const void *q, *k, *v;
  void *k_cache, *v_cache;
  const long long* pos;
  void* out;
  int B, H, Hk, d, window, sinks, dtype;
  float scale;
  float* part;  // partial results of more splits than a cluster joins, or null
  int splits;
};
// number of parts that a sequence's cache is read in, and the scratch they need
int swa_decode_splits(int B, int H, int Hk, int window, int sinks, int dtype);
size_t swa_decode_bytes(int B, int H, int d, int splits);
cudaError_t launch_swa_decode(const SwaDecodeArgs& a, cudaStream_t st);

struct SwaFillArgs {
  const void *k, *v;
  const long long* lens;
  void *k_cache, *v_cache;
  int B, T, Hk, d, window, sinks, dtype;
};
cudaError_t launch_swa_fill(const SwaFillArgs& a, cudaStream_t st);

// largest cluster of CTAs along the sequence (each writes a part of da_log)
constexpr int kGlrMaxCluster = 8;

struct GlrArgs {
  const void *x, *i_pre, *f_pre;
  const float *a_log, *h0;
  void* out;
  float* hT;
  const void* dh;
  const float* dhT;
  void *dx, *di_pre, *df_pre;
  float *da_log, *dh0;
  float* states;           // forward: state at the start of each chunk [B][NC][D], or null
  const float* states_in;  // backward
  float* part;             // backward: parts of da_log [B][cluster][D]
  int B, T, D, dtype;
  int* err = nullptr;      // the library's device error word
};
cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st);
cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st);
cudaError_t launch_glr_decode(const GlrArgs& a, cudaStream_t st);

}  // namespace kd
