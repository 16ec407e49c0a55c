// kd_swa_decode.cu -- one token per sequence over the ring cache of
// sliding-window attention, and the cache's fill after a prefill.
//
// The cache keeps sinks + window slots per sequence; position p lives in slot
// p (p < sinks) or sinks + (p - sinks) mod window, so the slots in use, the
// first min(p + 1, sinks + window), are exactly the keys that the token sees,
// in an order that a softmax does not depend on.
//
// HBM-bound: every key and value in use is read once, for all query heads of
// its group.  A row of d channels is one 16-byte vector per lane, so a warp
// takes 32 / (d / vector) keys at a time: dot products per lane, a butterfly
// over the row's lanes, one running maximum and sum per warp and head, and
// the values weighted in the same layout.  A warp's lanes hold partial sums
// over its keys; they are joined at the end, over the warps through shared
// memory, and over the parts of a long cache by a second kernel.
#include "kd_hybrid.h"
#include "kd_rows.cuh"

namespace kd {

namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 8;  // rows of keys (then of values) in flight per lane
constexpr float kLog2e = 1.44269504088896f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ long long slot_of(long long p, int W, int S) { return p < S ? p : S + (p - S) % W; }

template <typename T, int D>
struct Row {
  static constexpr int E = 16 / sizeof(T);  // channels per lane
  static constexpr int lanes = D / E;       // lanes per row
  static constexpr int rows = 32 / lanes;   // rows per warp and load
};

// GC: query heads of a key head that a CTA takes.
template <typename T, int D, int GC>
__global__ void __launch_bounds__(kWarps * 32) swa_decode_kernel(SwaDecodeArgs a) {
  using R = Row<T, D>;
  constexpr int E = R::E;
  using P = Pack<T, E>;
  __shared__ float sh_m[kWarps][GC], sh_l[kWarps][GC], sh_o[kWarps][GC][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / R::lanes, c = (lane % R::lanes) * E;
  const int group = a.H / a.Hk, chunks = (group + GC - 1) / GC;
  const int hk = blockIdx.y / chunks, g0 = blockIdx.y % chunks * GC;
  const size_t b = blockIdx.z;
  const int slots = a.window + a.sinks;
  const long long pos = a.pos[b];
  const int n = pos < 0 ? 0 : pos + 1 < slots ? (int)pos + 1 : slots;
  const int mine = pos < 0 ? -1 : (int)slot_of(pos, a.window, a.sinks);
  const int per = (n + a.splits - 1) / a.splits;
  const int lo = blockIdx.x * per < n ? blockIdx.x * per : n, hi = lo + per < n ? lo + per : n;

  const size_t pitch = (size_t)a.Hk * D;
  T* kc = static_cast<T*>(a.k_cache) + (b * slots * a.Hk + hk) * D;
  T* vc = static_cast<T*>(a.v_cache) + (b * slots * a.Hk + hk) * D;
  const T* kn = static_cast<const T*>(a.k) + (b * a.Hk + hk) * D;
  const T* vn = static_cast<const T*>(a.v) + (b * a.Hk + hk) * D;
  // The new token is stored by one CTA and read by all from the arguments.
  if (mine >= lo && mine < hi && g0 == 0 && warp == 0 && sub == 0) {
    *reinterpret_cast<P*>(kc + mine * pitch + c) = *reinterpret_cast<const P*>(kn + c);
    *reinterpret_cast<P*>(vc + mine * pitch + c) = *reinterpret_cast<const P*>(vn + c);
  }

  float q[GC][E], o[GC][E], m[GC], l[GC];
#pragma unroll
  for (int g = 0; g < GC; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
    P v{};
    if (g0 + g < group) v = *reinterpret_cast<const P*>(static_cast<const T*>(a.q) + (b * a.H + hk * group + g0 + g) * D + c);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[g][e] = g0 + g < group ? to_f(v.x[e]) * (a.scale * kLog2e) : 0.f;
      o[g][e] = 0.f;
    }
  }
  for (int j0 = lo + warp * R::rows * kBatch; j0 < hi; j0 += kWarps * R::rows * kBatch) {
    P kk[kBatch], vv[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + u * R::rows + sub;
      if (j < hi) kk[u] = *reinterpret_cast<const P*>((j == mine ? kn : kc + j * pitch) + c);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = j0 + u * R::rows + sub;
      if (j < hi) vv[u] = *reinterpret_cast<const P*>((j == mine ? vn : vc + j * pitch) + c);
    }
#pragma unroll
    for (int g = 0; g < GC; ++g) {
      float s[kBatch], top = m[g];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        float d = 0.f;
        const bool in = j0 + u * R::rows + sub < hi;
        if (in) {
#pragma unroll
          for (int e = 0; e < E; ++e) d = fmaf(q[g][e], to_f(kk[u].x[e]), d);
        }
        d = group_sum<R::lanes>(d);
        s[u] = in ? d : -INFINITY;
        top = fmaxf(top, s[u]);
      }
#pragma unroll
      for (int w = R::lanes; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float f = ex2(m[g] - top);  // top is finite: the warp's first row is in range
      m[g] = top;
      l[g] *= f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] *= f;
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (j0 + u * R::rows + sub < hi) {
          const float p = ex2(s[u] - top);
          l[g] += p;
#pragma unroll
          for (int e = 0; e < E; ++e) o[g][e] = fmaf(p, to_f(vv[u].x[e]), o[g][e]);
        }
    }
  }
  // join the warp's rows, then the warps
#pragma unroll
  for (int g = 0; g < GC; ++g) {
#pragma unroll
    for (int w = R::lanes; w < 32; w <<= 1) {
      l[g] += __shfl_xor_sync(0xffffffffu, l[g], w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] += __shfl_xor_sync(0xffffffffu, o[g][e], w);
    }
    if (lane == 0) {
      sh_m[warp][g] = m[g];
      sh_l[warp][g] = l[g];
    }
    if (sub == 0)
#pragma unroll
      for (int e = 0; e < E; ++e) sh_o[warp][g][c + e] = o[g][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < GC * D; i += kWarps * 32) {
    const int g = i / D, ch = i % D, h = hk * group + g0 + g;
    if (g0 + g >= group) continue;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w][g]);
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sh_m[w][g] == -INFINITY ? 0.f : ex2(sh_m[w][g] - top);
      sum = fmaf(f, sh_l[w][g], sum);
      acc = fmaf(f, sh_o[w][g][ch], acc);
    }
    if (a.splits == 1) {
      static_cast<T*>(a.out)[(b * a.H + h) * D + ch] = from_f<T>(n ? acc / sum : 0.f);
    } else {
      float* part = a.part + ((b * a.H + h) * a.splits + blockIdx.x) * (size_t)(D + 2);
      part[2 + ch] = acc;
      if (ch == 0) {
        part[0] = top;
        part[1] = sum;
      }
    }
  }
}

// Joins the parts of one head: weights of the parts first, then the channels.
template <typename T, int D>
__global__ void __launch_bounds__(D) swa_decode_join_kernel(const float* __restrict__ part, int splits,
                                                            T* __restrict__ out) {
  const float* p = part + (size_t)blockIdx.x * splits * (D + 2);
  float top = -INFINITY;
  for (int s = 0; s < splits; ++s) top = fmaxf(top, p[(size_t)s * (D + 2)]);
  float sum = 0.f, acc = 0.f;
  if (top != -INFINITY)
    for (int s = 0; s < splits; ++s) {
      const float* q = p + (size_t)s * (D + 2);
      const float f = ex2(q[0] - top);  // 0 for an empty part
      sum = fmaf(f, q[1], sum);
      acc = fmaf(f, q[2 + threadIdx.x], acc);
    }
  out[(size_t)blockIdx.x * D + threadIdx.x] = from_f<T>(sum > 0.f ? acc / sum : 0.f);
}

template <typename T, int D, int GC>
cudaError_t decode_gc(const SwaDecodeArgs& a, cudaStream_t st) {
  const int chunks = (a.H / a.Hk + GC - 1) / GC;
  prof_begin(st, "swa_decode");
  swa_decode_kernel<T, D, GC><<<dim3(a.splits, a.Hk * chunks, a.B), kWarps * 32, 0, st>>>(a);
  prof_end(st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.splits == 1) return e;
  prof_begin(st, "swa_decode_join");
  swa_decode_join_kernel<T, D><<<a.B * a.H, D, 0, st>>>(a.part, a.splits, static_cast<T*>(a.out));
  prof_end(st);
  return cudaGetLastError();
}

int heads_per_cta(int group) { return group >= 3 ? 4 : group; }

template <typename T, int D>
cudaError_t decode_d(const SwaDecodeArgs& a, cudaStream_t st) {
  switch (heads_per_cta(a.H / a.Hk)) {
    case 1: return decode_gc<T, D, 1>(a, st);
    case 2: return decode_gc<T, D, 2>(a, st);
    default: return decode_gc<T, D, 4>(a, st);
  }
}

template <typename T>
cudaError_t decode_t(const SwaDecodeArgs& a, cudaStream_t st) {
  return a.d == 32 ? decode_d<T, 32>(a, st) : a.d == 64 ? decode_d<T, 64>(a, st) : decode_d<T, 128>(a, st);
}

// Per slot: the newest of the first n tokens that belongs there.
__global__ void __launch_bounds__(256) swa_fill_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                                                       const long long* __restrict__ lens, uint4* __restrict__ kc,
                                                       uint4* __restrict__ vc, int T_, int row, int W, int S,
                                                       long long total) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= total) return;
  const long long rs = i / row;
  const int c = (int)(i - rs * row), slots = W + S;
  const long long b = rs / slots;
  const int slot = (int)(rs - b * slots);
  long long n = lens[b];
  n = n < 0 ? 0 : n > T_ ? T_ : n;
  const long long p = slot < S ? slot : slot >= n ? n : n - 1 - (n - 1 - slot) % W;
  if (p >= n) return;
  const long long from = (b * T_ + p) * row + c;
  kc[i] = k[from];
  vc[i] = v[from];
}

}  // namespace

// Parts of a cache: enough CTAs for four on each of 148 SMs, but at least 64
// slots to a part.
int swa_decode_splits(int B, int H, int Hk, int d, int window, int sinks, int dtype) {
  const int gc = heads_per_cta(H / Hk);
  const long long units = (long long)B * Hk * ((H / Hk + gc - 1) / gc);
  const long long most = ((long long)window + sinks + 63) / 64;
  long long s = (592 + units - 1) / units;
  if (s > most) s = most;
  return s < 1 ? 1 : (int)s;
}

size_t swa_decode_bytes(int B, int H, int d, int splits) {
  return splits == 1 ? 0 : (size_t)B * H * splits * (d + 2) * sizeof(float);
}

cudaError_t launch_swa_decode(const SwaDecodeArgs& a, cudaStream_t st) {
  return a.dtype == 1 ? decode_t<__nv_bfloat16>(a, st) : decode_t<float>(a, st);
}

cudaError_t launch_swa_fill(const SwaFillArgs& a, cudaStream_t st) {
  const int row = a.Hk * a.d * (a.dtype == 1 ? 2 : 4) / 16;
  const long long total = (long long)a.B * (a.window + a.sinks) * row;
  prof_begin(st, "swa_fill");
  swa_fill_kernel<<<(unsigned)((total + 255) / 256), 256, 0, st>>>(
      static_cast<const uint4*>(a.k), static_cast<const uint4*>(a.v), a.lens, static_cast<uint4*>(a.k_cache),
      static_cast<uint4*>(a.v_cache), a.T, row, a.window, a.sinks, total);
  prof_end(st);
  return cudaGetLastError();
}

}  // namespace kd
