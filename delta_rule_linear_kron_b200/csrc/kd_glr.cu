// kd_glr.cu -- element-wise gated linear recurrence: forward, backward, step.
//
// Per channel, with a = e^{a_log}:
//   l_t = a log sigma(f~_t),  f_t = e^{l_t},  m_t = sqrt(1 - f_t^2),  i_t = sigma(i~_t)
//   h_t = f_t h_{t-1} + m_t i_t x_t
// Backward for <dh, out> + <dhT, hT>, with u_t = f_t g_t:
//   g_t = dh_t + u_{t+1}  (u_T = dhT),   dh0 = u_0
//   dx = g m i,  di~ = g m x i (1 - i),  dl = g (f h_{t-1} - i x f^2 / m)
//   df~ = dl a sigma(-f~),  da_log = sum dl l
//
// HBM-bound in bytes (8 per element forward, 14.25 backward with bf16), but
// close to the instruction rate too: the gates are about 45 instructions per
// element, so nothing may be computed twice.  One pass: a cluster of C CTAs
// takes 64 channels and C consecutive chunks of 64 tokens at a time.  A warp
// holds 8 tokens, a lane 2 channels; each thread scans its 8 tokens from zero,
// the warps' (prod f, h) pairs combine through shared memory and the CTAs'
// through distributed shared memory, and the thread then adds its start
// state's part, from registers.  The chain along the sequence is then only
// ceil(T / 64C) cluster exchanges long.
//
// The state's error builds up over 1 / (1 - f) steps, so f and 1 - f^2 are
// formed through expm1 (f = 1 + y, 1 - f^2 = -y (1 + f)): f is then within
// half an fp32 step, without a bias, where the hardware exponential alone is
// off by up to two.
#include "kd_hybrid.h"
#include "kd_rows.cuh"
#include "kd_tc.cuh"

namespace kd {

namespace {

constexpr int kWarps = 8, kTok = 8;    // a chunk: 8 warps of 8 tokens
constexpr int kChans = 64;             // channels of a CTA, 2 per lane
static_assert(kWarps * kTok == kChunk, "a CTA takes one chunk at a time");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rsq(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.44269504088896f;

// log(1 + e), 0 <= e <= 1: 2 artanh(s) with s = e / (2 + e) <= 1/3, seven
// terms of its series (the eighth is below 2e-8 of the sum).
__device__ __forceinline__ float log1p01(float e) {
  const float s = e * rcp(2.f + e), z = s * s;
  float p = fmaf(z, 1.f / 13, 1.f / 11);
  p = fmaf(z, p, 1.f / 9);
  p = fmaf(z, p, 1.f / 7);
  p = fmaf(z, p, 1.f / 5);
  p = fmaf(z, p, 1.f / 3);
  return 2.f * fmaf(s * z, p, s);
}

struct Gates {
  float l, f, w, i;  // w = 1 - f^2
  float e;           // e^{-|f~|}
};

__device__ __forceinline__ Gates gates(float zf, float zi, float a) {
  Gates g;
  g.e = ex2(-kLog2e * fabsf(zf));
  // f~ at the type's lowest value starts a new sequence: l stays finite so
  // that the backward's dl l is 0 there and not 0 * infinity
  g.l = fmaxf(-a * (fmaxf(-zf, 0.f) + log1p01(g.e)), -1e30f);
  // e^l - 1 on [-1/2, 0] by its series up to l^8 / 8! (the next term is below
  // 1e-8 of the sum); below that nothing cancels
  const float l = g.l;
  float p = fmaf(l, 1.f / 40320, 1.f / 5040);
  p = fmaf(l, p, 1.f / 720);
  p = fmaf(l, p, 1.f / 120);
  p = fmaf(l, p, 1.f / 24);
  p = fmaf(l, p, 1.f / 6);
  p = fmaf(l, p, 0.5f);
  p = fmaf(l, p, 1.f) * l;
  const float far = ex2(kLog2e * l);
  const bool near = l > -0.5f;
  g.f = near ? 1.f + p : far;
  const float y = near ? p : far - 1.f;
  g.w = -y * (1.f + g.f);
  g.i = rcp(1.f + ex2(-kLog2e * zi));
  return g;
}

// 1 / m.  A gate so close to 1 that w leaves the range of the reciprocal root
// writes nothing (m < 1e-15) and takes no gradient through m.
__device__ __forceinline__ float inv_m(float w) { return w > 1e-30f ? rsq(w) : 0.f; }

template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
  using type = __nv_bfloat162;
  static __device__ __forceinline__ float2 f(type v) { return __bfloat1622float2(v); }
  static __device__ __forceinline__ type of(float a, float b) { return __floats2bfloat162_rn(a, b); }
};
template <> struct Pair<float> {
  using type = float2;
  static __device__ __forceinline__ float2 f(type v) { return v; }
  static __device__ __forceinline__ type of(float a, float b) { return make_float2(a, b); }
};

__device__ __forceinline__ void st_cluster(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}

template <typename T>
__global__ void __launch_bounds__(kWarps * 32) glr_fwd_kernel(const T* __restrict__ x, const T* __restrict__ ip,
                                                              const T* __restrict__ fp,
                                                              const float* __restrict__ a_log,
                                                              const float* __restrict__ h0, T* __restrict__ out,
                                                              float* __restrict__ hT, float* __restrict__ states,
                                                              int T_, int D, int NC, int C) {
  using P = Pair<T>;
  using V = typename P::type;
  __shared__ float4 wagg[2][kWarps][32];  // (f products, states) of a warp's tokens, two channels
  __shared__ float4 cagg[2][kGlrMaxCluster][32];       // the same of the cluster's CTAs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)tc::cluster_rank() : 0;
  const int b = blockIdx.y, c = (int)(blockIdx.x / C) * kChans + lane * 2;
  const bool live = c < D;
  const size_t base = (size_t)b * T_ * D + c;
  float a0 = 1.f, a1 = 1.f;
  float2 carry = make_float2(0.f, 0.f);
  if (live) {
    a0 = expf(a_log[c]);
    a1 = expf(a_log[c + 1]);
    if (h0) carry = *reinterpret_cast<const float2*>(h0 + (size_t)b * D + c);
  }
  if (C > 1) tc::cluster_sync();  // every CTA of the cluster has started
  const int steps = (NC + C - 1) / C;
  for (int s = 0; s < steps; ++s) {
    const int n = s * C + rank, par = s & 1;
    const long long t0 = (long long)n * kChunk + warp * kTok;
    const long long left = T_ - t0;
    const int k = !live || left <= 0 ? 0 : left < kTok ? (int)left : kTok;  // tokens of this thread
    const size_t off = base + (size_t)t0 * D;
    V rx[kTok], ri[kTok], rf[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < k) {
        rf[j] = __ldcs(reinterpret_cast<const V*>(fp + off + (size_t)j * D));
        ri[j] = __ldcs(reinterpret_cast<const V*>(ip + off + (size_t)j * D));
        rx[j] = __ldcs(reinterpret_cast<const V*>(x + off + (size_t)j * D));
      }
    float F0[kTok], F1[kTok], H0[kTok], H1[kTok];
    float p0 = 1.f, p1 = 1.f, q0 = 0.f, q1 = 0.f;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (j < k) {
        const float2 vx = P::f(rx[j]), vi = P::f(ri[j]), vf = P::f(rf[j]);
        const Gates g0 = gates(vf.x, vi.x, a0), g1 = gates(vf.y, vi.y, a1);
        p0 *= g0.f;
        p1 *= g1.f;
        q0 = fmaf(g0.f, q0, g0.w * inv_m(g0.w) * g0.i * vx.x);
        q1 = fmaf(g1.f, q1, g1.w * inv_m(g1.w) * g1.i * vx.y);
      }
      F0[j] = p0; F1[j] = p1; H0[j] = q0; H1[j] = q1;
    }
    wagg[par][warp][lane] = make_float4(p0, p1, q0, q1);
    __syncthreads();
    float4 pre = make_float4(1.f, 1.f, 0.f, 0.f), all = pre;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) pre = all;
      const float4 v = wagg[par][w][lane];
      all = make_float4(all.x * v.x, all.y * v.y, fmaf(v.x, all.z, v.z), fmaf(v.y, all.w, v.w));
    }
    float2 mine = carry;  // state at the start of this CTA's chunk
    if (C > 1) {
      // warp w hands the chunk's pair to CTA w; the buffer's last readers have
      // arrived at the barrier of the step before
      if (warp < C) st_cluster(tc::mapa(tc::smem_u32(&cagg[par][rank][lane]), warp), all);
      tc::cluster_sync();
      for (int r = 0; r < C; ++r) {
        if (r == rank) mine = carry;
        const float4 v = cagg[par][r][lane];
        carry = make_float2(fmaf(v.x, carry.x, v.z), fmaf(v.y, carry.y, v.w));
      }
    } else {
      carry = make_float2(fmaf(all.x, carry.x, all.z), fmaf(all.y, carry.y, all.w));
    }
    const float s0 = fmaf(pre.x, mine.x, pre.z), s1 = fmaf(pre.y, mine.y, pre.w);
    if (states && warp == 0 && live && n < NC)
      *reinterpret_cast<float2*>(states + ((size_t)b * NC + n) * D + c) = mine;
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < k)
        __stcs(reinterpret_cast<V*>(out + off + (size_t)j * D),
               P::of(fmaf(F0[j], s0, H0[j]), fmaf(F1[j], s1, H1[j])));
  }
  if (hT && rank == 0 && warp == 0 && live) *reinterpret_cast<float2*>(hT + (size_t)b * D + c) = carry;
}

// The backward walks the chunks from the last.  The states h_{t-1} come from
// the chunk's saved start state, run forward again over the tokens in
// registers, so they are fp32 (the bf16 output would put its rounding into
// df~ and da_log).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32, 2) glr_bwd_kernel(
    const T* __restrict__ x, const T* __restrict__ ip, const T* __restrict__ fp, const float* __restrict__ a_log,
    const float* __restrict__ states, const T* __restrict__ dh, const float* __restrict__ dhT, T* __restrict__ dx,
    T* __restrict__ di, T* __restrict__ df, float* __restrict__ part, float* __restrict__ dh0, int T_, int D, int NC,
    int C) {
  using P = Pair<T>;
  using V = typename P::type;
  __shared__ float4 wagg[2][kWarps][32];  // (f products, forward states)
  __shared__ float2 uagg[2][kWarps][32];  // reverse terms u
  __shared__ float4 cagg[2][kGlrMaxCluster][32];       // (f products, u) of the cluster's CTAs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = C > 1 ? (int)tc::cluster_rank() : 0;
  const int b = blockIdx.y, c = (int)(blockIdx.x / C) * kChans + lane * 2;
  const bool live = c < D;
  const size_t base = (size_t)b * T_ * D + c;
  float a0 = 1.f, a1 = 1.f;
  float2 carry = make_float2(0.f, 0.f);
  if (live) {
    a0 = expf(a_log[c]);
    a1 = expf(a_log[c + 1]);
    if (dhT) carry = *reinterpret_cast<const float2*>(dhT + (size_t)b * D + c);
  }
  float da0 = 0.f, da1 = 0.f;
  if (C > 1) tc::cluster_sync();  // every CTA of the cluster has started
  const int steps = (NC + C - 1) / C;
  for (int s = steps - 1; s >= 0; --s) {
    const int n = s * C + rank, par = s & 1;
    const long long t0 = (long long)n * kChunk + warp * kTok;
    const long long left = T_ - t0;
    const int k = !live || left <= 0 ? 0 : left < kTok ? (int)left : kTok;
    const size_t off = base + (size_t)t0 * D;
    V rx[kTok], ri[kTok], rf[kTok], rg[kTok];
#pragma unroll
    for (int j = 0; j < kTok; ++j)
      if (j < k) {
        rf[j] = __ldcs(reinterpret_cast<const V*>(fp + off + (size_t)j * D));
        ri[j] = __ldcs(reinterpret_cast<const V*>(ip + off + (size_t)j * D));
        rx[j] = __ldcs(reinterpret_cast<const V*>(x + off + (size_t)j * D));
        rg[j] = __ldcs(reinterpret_cast<const V*>(dh + off + (size_t)j * D));
      }
    float2 start = make_float2(0.f, 0.f);
    if (live && n < NC) start = *reinterpret_cast<const float2*>(states + ((size_t)b * NC + n) * D + c);
    float F[2][kTok], Bx[2][kTok], Wr[2][kTok], I[2][kTok];  // f, m i x, 1 / m, i
    float p0 = 1.f, p1 = 1.f, q0 = 0.f, q1 = 0.f;
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      F[0][j] = F[1][j] = 1.f;
      Bx[0][j] = Bx[1][j] = Wr[0][j] = Wr[1][j] = I[0][j] = I[1][j] = 0.f;
      if (j < k) {
        const float2 vx = P::f(rx[j]), vi = P::f(ri[j]), vf = P::f(rf[j]);
        const Gates g0 = gates(vf.x, vi.x, a0), g1 = gates(vf.y, vi.y, a1);
        F[0][j] = g0.f;
        F[1][j] = g1.f;
        I[0][j] = g0.i;
        I[1][j] = g1.i;
        Wr[0][j] = inv_m(g0.w);
        Wr[1][j] = inv_m(g1.w);
        Bx[0][j] = g0.w * Wr[0][j] * g0.i * vx.x;
        Bx[1][j] = g1.w * Wr[1][j] * g1.i * vx.y;
        p0 *= g0.f;
        p1 *= g1.f;
        q0 = fmaf(g0.f, q0, Bx[0][j]);
        q1 = fmaf(g1.f, q1, Bx[1][j]);
      }
    }
    float u0 = 0.f, u1 = 0.f;
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j)
      if (j < k) {
        const float2 g = P::f(rg[j]);
        u0 = F[0][j] * (g.x + u0);
        u1 = F[1][j] * (g.y + u1);
      }
    wagg[par][warp][lane] = make_float4(p0, p1, q0, q1);
    uagg[par][warp][lane] = make_float2(u0, u1);
    __syncthreads();
    // forward: state before this warp's first token
    float2 hs = start;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
      if (w < warp) {
        const float4 v = wagg[par][w][lane];
        hs = make_float2(fmaf(v.x, hs.x, v.z), fmaf(v.y, hs.y, v.w));
      }
    // backward: what this warp's last token gets from the later ones
    float4 post = make_float4(1.f, 1.f, 0.f, 0.f), all = post;
#pragma unroll
    for (int w = kWarps - 1; w >= 0; --w) {
      if (w == warp) post = all;
      const float4 v = wagg[par][w][lane];
      const float2 u = uagg[par][w][lane];
      all = make_float4(all.x * v.x, all.y * v.y, fmaf(v.x, all.z, u.x), fmaf(v.y, all.w, u.y));
    }
    float2 mine = carry;
    if (C > 1) {
      if (warp < C) st_cluster(tc::mapa(tc::smem_u32(&cagg[par][rank][lane]), warp), all);
      tc::cluster_sync();
      for (int r = C - 1; r >= 0; --r) {
        if (r == rank) mine = carry;
        const float4 v = cagg[par][r][lane];
        carry = make_float2(fmaf(v.x, carry.x, v.z), fmaf(v.y, carry.y, v.w));
      }
    } else {
      carry = make_float2(fmaf(all.x, carry.x, all.z), fmaf(all.y, carry.y, all.w));
    }
    float Hp[2][kTok];  // h_{t-1}
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      Hp[0][j] = hs.x;
      Hp[1][j] = hs.y;
      hs = make_float2(fmaf(F[0][j], hs.x, Bx[0][j]), fmaf(F[1][j], hs.y, Bx[1][j]));
    }
    float v0 = fmaf(post.x, mine.x, post.z), v1 = fmaf(post.y, mine.y, post.w);
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j)
      if (j < k) {
        const float2 vx = P::f(rx[j]), vf = P::f(rf[j]), vg = P::f(rg[j]);
        float o[3][2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float a = q ? a1 : a0, xx = q ? vx.y : vx.x, zf = q ? vf.y : vf.x;
          const float g = (q ? vg.y : vg.x) + (q ? v1 : v0);
          const float f = F[q][j], i = I[q][j], r = Wr[q][j];
          const float u = f * g;
          (q ? v1 : v0) = u;
          // 1 - f^2 again from its reciprocal root, so that it stays out of the registers
          const float m = r > 0.f ? rcp(r) : 0.f;
          o[0][q] = g * m * i;
          o[1][q] = g * Bx[q][j] * (1.f - i);
          const float dl = u * (Hp[q][j] - i * xx * f * r);
          const float e = ex2(-kLog2e * fabsf(zf)), den = rcp(1.f + e);
          const float l = fmaxf(-a * (fmaxf(-zf, 0.f) + log1p01(e)), -1e30f);
          o[2][q] = dl * a * (zf >= 0.f ? e * den : den);
          (q ? da1 : da0) += dl * l;
        }
        const size_t at = off + (size_t)j * D;
        __stcs(reinterpret_cast<V*>(dx + at), P::of(o[0][0], o[0][1]));
        __stcs(reinterpret_cast<V*>(di + at), P::of(o[1][0], o[1][1]));
        __stcs(reinterpret_cast<V*>(df + at), P::of(o[2][0], o[2][1]));
      }
  }
  if (dh0 && rank == 0 && warp == 0 && live) *reinterpret_cast<float2*>(dh0 + (size_t)b * D + c) = carry;
  // da_log: the warps' sums in a fixed order, one row per CTA of the cluster
  __syncthreads();
  uagg[0][warp][lane] = make_float2(da0, da1);
  __syncthreads();
  if (warp == 0 && live) {
    float2 t = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 v = uagg[0][w][lane];
      t.x += v.x;
      t.y += v.y;
    }
    *reinterpret_cast<float2*>(part + ((size_t)b * C + rank) * D + c) = t;
  }
}

__global__ void __launch_bounds__(256) glr_dalog_kernel(const float* __restrict__ part, int rows, int D,
                                                        float* __restrict__ da_log) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  float t = 0.f;
  for (int r = 0; r < rows; ++r) t += part[(size_t)r * D + c];
  da_log[c] = t;
}

template <typename T>
__global__ void __launch_bounds__(128) glr_decode_kernel(const T* __restrict__ x, const T* __restrict__ ip,
                                                         const T* __restrict__ fp, const float* __restrict__ a_log,
                                                         float* __restrict__ h, T* __restrict__ out, long long n,
                                                         int D) {
  using P = Pair<T>;
  using V = typename P::type;
  const long long at = ((long long)blockIdx.x * 128 + threadIdx.x) * 2;
  if (at >= n) return;
  const int c = (int)(at % D);
  const float2 vx = P::f(*reinterpret_cast<const V*>(x + at)), vi = P::f(*reinterpret_cast<const V*>(ip + at));
  const float2 vf = P::f(*reinterpret_cast<const V*>(fp + at));
  float2 s = *reinterpret_cast<const float2*>(h + at);
  const Gates g0 = gates(vf.x, vi.x, expf(a_log[c])), g1 = gates(vf.y, vi.y, expf(a_log[c + 1]));
  s.x = fmaf(g0.f, s.x, g0.w * inv_m(g0.w) * g0.i * vx.x);
  s.y = fmaf(g1.f, s.y, g1.w * inv_m(g1.w) * g1.i * vx.y);
  *reinterpret_cast<float2*>(h + at) = s;
  *reinterpret_cast<V*>(out + at) = P::of(s.x, s.y);
}

// CTAs of a cluster (chunks taken at a time): enough CTAs for two on each of
// 148 SMs, as far as the sequence has chunks, and at most the portable 8.
int cluster_size(const GlrArgs& a, int NC) {
  const long long lanes = (long long)((a.D + kChans - 1) / kChans) * a.B;
  int C = 1;
  while (C < kGlrMaxCluster && C < NC && lanes * C < 2 * 148) C *= 2;
  return C;
}

template <typename K, typename... A>
cudaError_t launch_cluster(K kernel, dim3 grid, int C, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = C;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t glr_fwd_t(const GlrArgs& a, cudaStream_t st) {
  const int NC = (a.T + kChunk - 1) / kChunk, C = cluster_size(a, NC);
  const dim3 grid((unsigned)((a.D + kChans - 1) / kChans) * C, a.B);
  prof_begin(st, "glr_fwd");
  const cudaError_t e =
      launch_cluster(glr_fwd_kernel<T>, grid, C, st, static_cast<const T*>(a.x), static_cast<const T*>(a.i_pre),
                     static_cast<const T*>(a.f_pre), a.a_log, a.h0, static_cast<T*>(a.out), a.hT, a.states, a.T, a.D,
                     NC, C);
  prof_end(st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t glr_bwd_t(const GlrArgs& a, cudaStream_t st) {
  const int NC = (a.T + kChunk - 1) / kChunk, C = cluster_size(a, NC);
  const dim3 grid((unsigned)((a.D + kChans - 1) / kChans) * C, a.B);
  prof_begin(st, "glr_bwd");
  cudaError_t e =
      launch_cluster(glr_bwd_kernel<T>, grid, C, st, static_cast<const T*>(a.x), static_cast<const T*>(a.i_pre),
                     static_cast<const T*>(a.f_pre), a.a_log, a.states_in, static_cast<const T*>(a.dh), a.dhT,
                     static_cast<T*>(a.dx), static_cast<T*>(a.di_pre), static_cast<T*>(a.df_pre), a.part, a.dh0, a.T,
                     a.D, NC, C);
  prof_end(st);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  prof_begin(st, "glr_dalog");
  glr_dalog_kernel<<<(a.D + 255) / 256, 256, 0, st>>>(a.part, a.B * C, a.D, a.da_log);
  prof_end(st);
  return cudaGetLastError();
}

template <typename T>
cudaError_t glr_decode_t(const GlrArgs& a, cudaStream_t st) {
  const long long n = (long long)a.B * a.D;
  prof_begin(st, "glr_decode");
  glr_decode_kernel<T><<<(unsigned)((n / 2 + 127) / 128), 128, 0, st>>>(
      static_cast<const T*>(a.x), static_cast<const T*>(a.i_pre), static_cast<const T*>(a.f_pre), a.a_log, a.hT,
      static_cast<T*>(a.out), n, a.D);
  prof_end(st);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? glr_fwd_t<__nv_bfloat16>(a, st) : glr_fwd_t<float>(a, st);
}
cudaError_t launch_glr_bwd(const GlrArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? glr_bwd_t<__nv_bfloat16>(a, st) : glr_bwd_t<float>(a, st);
}
cudaError_t launch_glr_decode(const GlrArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? glr_decode_t<__nv_bfloat16>(a, st) : glr_decode_t<float>(a, st);
}

}  // namespace kd
