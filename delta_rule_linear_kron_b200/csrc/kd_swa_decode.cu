// kd_swa_decode.cu -- one token per sequence over the ring cache of
// sliding-window attention, and the cache's fill after a prefill.
//
// The cache keeps sinks + window slots per sequence; position p lives in slot
// p (p < sinks) or sinks + (p - sinks) mod window, so the slots in use, the
// first min(p + 1, sinks + window), are exactly the keys that the token sees,
// in an order that a softmax does not depend on.
//
// HBM-bound: every key and value in use is read once, for all query heads of
// its group.  256 sequences, 16 + 4 heads of 128 bf16, 2052 slots in use (1.08 GB):
// 182 us, 5.9 TB/s, 90% of what a copy does.  Where there are few sequences, a cache is read in parts by
// several CTAs.  Up to 8 parts are a cluster, whose CTAs join them through
// distributed shared memory; more (a long window) are joined by a second
// kernel from the workspace.
//
// bf16: m16n8k16 products, the (up to 16) query heads of a key head as the 16
// rows.  tcgen05 would want 128 rows, of which a group fills 1 to 16, and the
// products are an eighth of what the tensor cores can do while the cache
// streams in; what matters is that the cache's bytes are in flight.  So each
// warp works alone: its own ring of 16-key tiles, filled by 16-byte async
// copies two tiles ahead, its own running maximum and sum, and no barrier
// until the warps' results are joined.  The weights go into the value product
// as bf16 high and low parts (2^-16 of themselves): the second product costs
// nothing here, and the output is as exact as with fp32 weights.
//
// fp32: CUDA cores.  A row of d channels is one 16-byte vector per lane, so a
// warp takes 32 / (d / 4) keys at a time: dot products per lane, a butterfly
// over the row's lanes, the values weighted in the same layout.  256 sequences
// as above 666 us, 3.2 TB/s: with four heads' rows in 200 registers an SM holds
// 8 warps, too few to hide that a warp's batch of loads, its arithmetic and its
// butterflies follow one another (43% of the issue slots, HBM at 37%).
#include "kd_hybrid.h"
#include "kd_rows.cuh"
#include "kd_tc.cuh"

namespace kd {

namespace {

constexpr int kWarps = 4;
constexpr int kDecodeCluster = 8;
constexpr int kDecodeParts = 64;
// slots times bytes per channel up to which a cluster's 8 parts are used where
// more would be wanted.  One sequence, d = 128 bf16 (d = 64 fp32), us by a
// cluster and by 64 parts and a second kernel: 5.3 and 5.8 (6.9 and 6.4) for
// 1024 slots, 9.5 and 8.0 (17 and 8.7) for 4096, 24 and 10.5 (58 and 14) for
// 16384; the second kernel costs the caller 5 us of launch and workspace.
constexpr int kDecodeClusterBytes = 2 * (4096 + 128);
// CTAs of a call that run at once: two on each of 148 SMs, less what clusters
// leave free.  64 x 4 key heads in 2, 1 parts: 31, 25 us (512, 256 CTAs); 16 x 4
// in 5, 4, 3, 2 parts: 36, 25, 27, 27 us; 24 x 4 in 3, 2 parts: 50, 37 us.
constexpr int kDecodeCtas = 272;
constexpr int kBatch = 8;  // rows of keys (then of values) in flight per lane
constexpr float kLog2e = 1.44269504088896f;
// where running maxima start.  Finite, so that a score of -infinity (a product
// that overflows, an infinite key) weighs 0 and not NaN also before any other
// has been seen.
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ long long slot_of(long long p, int W, int S) { return p < S ? p : S + (p - S) % W; }

__device__ __forceinline__ float2 peer_f2(const float* p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(tc::mapa(tc::smem_u32(p), rank))
               : "memory");
  return v;
}

// A CTA's results for `heads` query heads from h0 on: sh_m, sh_l [warp][R] and
// sh_o [warp][R][D] of its warps become its part, and the parts the output.
template <typename T, int D, int R>
__device__ __forceinline__ void finish(const SwaDecodeArgs& a, size_t b, int h0, int heads, int n, float* sh_m,
                                       float* sh_l, float* sh_o) {
  const int tid = threadIdx.x;
  const bool cluster = a.splits > 1 && !a.part;
  // two channels per thread: the CTA's own (maximum, sum, weighted values), in
  // place of warp 0's
  for (int i = tid; i < heads * (D / 2); i += kWarps * 32) {
    const int r = i / (D / 2), c = i % (D / 2) * 2;
    float top = kLowest;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w * R + r]);
    float sum = 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = sh_m[w * R + r] == kLowest ? 0.f : ex2(sh_m[w * R + r] - top);
      const float2 v = *reinterpret_cast<const float2*>(sh_o + (w * R + r) * D + c);
      sum = fmaf(f, sh_l[w * R + r], sum);
      acc = make_float2(fmaf(f, v.x, acc.x), fmaf(f, v.y, acc.y));
    }
    if (a.splits == 1) {
      T* out = static_cast<T*>(a.out) + (b * a.H + h0 + r) * D + c;
      out[0] = from_f<T>(n ? acc.x / sum : 0.f);
      out[1] = from_f<T>(n ? acc.y / sum : 0.f);
    } else if (!cluster) {
      float* part = a.part + ((b * a.H + h0 + r) * a.splits + blockIdx.x) * (size_t)(D + 2);
      *reinterpret_cast<float2*>(part + 2 + c) = acc;
      if (c == 0) *reinterpret_cast<float2*>(part) = make_float2(top, n ? sum : -1.f);
    } else {
      *reinterpret_cast<float2*>(sh_o + r * D + c) = acc;  // only this thread reads these two of warp 0
    }
  }
  if (!cluster) return;
  __syncthreads();  // every thread has read the warps' maxima and sums
  for (int r = tid; r < heads; r += kWarps * 32) {
    float top = kLowest, sum = 0.f;
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh_m[w * R + r]);
    for (int w = 0; w < kWarps; ++w)
      sum += sh_m[w * R + r] == kLowest ? 0.f : ex2(sh_m[w * R + r] - top) * sh_l[w * R + r];
    *reinterpret_cast<float2*>(sh_o + R * D + r * 2) = make_float2(top, sum);  // over warp 1's values
  }
  tc::cluster_sync();
  // each CTA a share of the channels of every head
  for (int i = blockIdx.x * kWarps * 32 + tid; i < heads * (D / 2); i += a.splits * kWarps * 32) {
    const int r = i / (D / 2), c = i % (D / 2) * 2;
    float2 ms[8], v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < a.splits) {
        ms[s] = peer_f2(sh_o + R * D + r * 2, s);
        v[s] = peer_f2(sh_o + r * D + c, s);
      }
    float top = kLowest, sum = 0.f;
    float2 acc = make_float2(0.f, 0.f);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < a.splits) top = fmaxf(top, ms[s].x);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (s < a.splits) {
        const float f = ms[s].x == kLowest ? 0.f : ex2(ms[s].x - top);  // 0 for an empty part
        sum = fmaf(f, ms[s].y, sum);
        acc = make_float2(fmaf(f, v[s].x, acc.x), fmaf(f, v[s].y, acc.y));
      }
    T* out = static_cast<T*>(a.out) + (b * a.H + h0 + r) * D + c;
    out[0] = from_f<T>(n ? acc.x / sum : 0.f);
    out[1] = from_f<T>(n ? acc.y / sum : 0.f);
  }
  tc::cluster_sync();  // no CTA leaves while another still reads its part
}

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
  __shared__ float sh_m[kWarps][GC], sh_l[kWarps][GC];
  __shared__ __align__(16) float sh_o[kWarps][GC][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / R::lanes, c = (lane % R::lanes) * E;
  const int group = a.H / a.Hk, chunks = (group + GC - 1) / GC;
  const int hk = blockIdx.y / chunks, g0 = blockIdx.y % chunks * GC;
  const size_t b = blockIdx.z;
  const int slots = a.window + a.sinks;
  const long long pos = a.pos[b];
  const int n = pos < 0 ? 0 : pos < slots ? (int)pos + 1 : slots;
  const int mine = pos < 0 ? -1 : (int)slot_of(pos, a.window, a.sinks);
  const int per = (n + a.splits - 1) / a.splits;
  const int lo = (int)min((long long)blockIdx.x * per, (long long)n), hi = min((long long)lo + per, (long long)n);

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
    m[g] = kLowest;
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
      const float f = ex2(m[g] - top);
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
  finish<T, D, GC>(a, b, hk * group + g0, min(GC, group - g0), n, &sh_m[0][0], &sh_l[0][0], &sh_o[0][0][0]);
}

// ---- bf16 -------------------------------------------------------------------

template <int D>
struct MmaCfg {
  static constexpr int CH = D / 8;              // 16-byte chunks of a row
  static constexpr int TILE = 16 * D * 2;       // bytes of 16 keys (or values)
  static constexpr int STAGES = D == 128 ? 3 : 4;
  static constexpr int WARP = STAGES * 2 * TILE;
  static constexpr int BYTES = kWarps * WARP;
  // byte offset of chunk c of row r: the eight rows that one ldmatrix reads at
  // a chunk lie in eight different 16-byte bank groups
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    return (uint32_t)(r * CH + (D == 32 ? c ^ ((r >> 1) & 3) : c ^ (r & 7))) * 16u;
  }
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool in) {  // zeros where !in
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool kTrans>
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
  if (kTrans)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// the part of (lo, hi) that pack2 leaves
__device__ __forceinline__ uint32_t rest2(float lo, float hi, uint32_t packed) {
  return pack2(lo - __uint_as_float(packed << 16), hi - __uint_as_float(packed & 0xffff0000u));
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) swa_decode_mma_kernel(SwaDecodeArgs a) {
  using Cf = MmaCfg<D>;
  using T = __nv_bfloat16;
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ float sh_m[kWarps][16], sh_l[kWarps][16];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, tq = lane & 3;
  const int group = a.H / a.Hk, chunks = (group + 15) / 16;
  const int hk = blockIdx.y / chunks, g0 = blockIdx.y % chunks * 16, heads = min(16, group - g0);
  const size_t b = blockIdx.z;
  const int slots = a.window + a.sinks;
  const long long pos = a.pos[b];
  const int n = pos < 0 ? 0 : pos < slots ? (int)pos + 1 : slots;
  const int mine = pos < 0 ? -1 : (int)slot_of(pos, a.window, a.sinks);
  const int per = (n + a.splits - 1) / a.splits;
  const int lo = (int)min((long long)blockIdx.x * per, (long long)n), hi = (int)min((long long)lo + per, (long long)n);

  const size_t pitch = (size_t)a.Hk * D;
  T* kc = static_cast<T*>(a.k_cache) + (b * slots * a.Hk + hk) * D;
  T* vc = static_cast<T*>(a.v_cache) + (b * slots * a.Hk + hk) * D;
  const T* kn = static_cast<const T*>(a.k) + (b * a.Hk + hk) * D;
  const T* vn = static_cast<const T*>(a.v) + (b * a.Hk + hk) * D;
  const uint32_t ring = smem_addr(sm) + warp * Cf::WARP;
  const int tiles = hi - lo > warp * 16 ? (hi - lo - warp * 16 + kWarps * 16 - 1) / (kWarps * 16) : 0;

  const auto load = [&](int it) {
    if (it < tiles) {
      const int j0 = lo + (it * kWarps + warp) * 16;
      const uint32_t dst = ring + it % Cf::STAGES * 2 * Cf::TILE;
#pragma unroll
      for (int i = 0; i < Cf::CH / 2; ++i) {
        const int r = (lane + 32 * i) / Cf::CH, c = (lane + 32 * i) % Cf::CH, j = j0 + r;
        const bool in = j < hi, fresh = j == mine;  // the new token comes from the arguments
        const size_t off = (size_t)(in ? j : lo) * pitch;
        copy16(dst + Cf::at(r, c), (fresh ? kn : kc + off) + c * 8, in);
        copy16(dst + Cf::TILE + Cf::at(r, c), (fresh ? vn : vc + off) + c * 8, in);
      }
    }
    copy_commit();
  };
#pragma unroll
  for (int i = 0; i < Cf::STAGES - 1; ++i) load(i);
  // The new token is stored by one CTA; all read it from the arguments.
  if (mine >= lo && mine < hi && g0 == 0 && warp == 0 && lane < Cf::CH) {
    *reinterpret_cast<uint4*>(kc + mine * pitch + lane * 8) = *reinterpret_cast<const uint4*>(kn + lane * 8);
    *reinterpret_cast<uint4*>(vc + mine * pitch + lane * 8) = *reinterpret_cast<const uint4*>(vn + lane * 8);
  }

  uint32_t q[D / 16][4];
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = g + (i & 1) * 8, c = s * 16 + (i >> 1) * 8 + tq * 2;
      q[s][i] = r < heads ? *reinterpret_cast<const uint32_t*>(static_cast<const T*>(a.q) +
                                                               (b * a.H + hk * group + g0 + r) * D + c)
                          : 0u;
    }
  float o[D / 8][4], m0 = kLowest, m1 = kLowest, l0 = 0.f, l1 = 0.f;
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  const float s2 = a.scale * kLog2e;
  const int mat = lane >> 3, mr = lane & 7;
  for (int it = 0; it < tiles; ++it) {
    copy_wait<Cf::STAGES - 2>();
    __syncwarp();
    load(it + Cf::STAGES - 1);
    const uint32_t kt = ring + it % Cf::STAGES * 2 * Cf::TILE, vt = kt + Cf::TILE;
    float x[2][4] = {};
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      uint32_t f[4];  // keys 0-7 and 8-15, channels 16s .. 16s + 15
      ldm4<false>(kt + Cf::at((mat >> 1) * 8 + mr, 2 * s + (mat & 1)), f);
      mma16816(x[0], q[s], f[0], f[1]);
      mma16816(x[1], q[s], f[2], f[3]);
    }
    const int j0 = lo + (it * kWarps + warp) * 16;
    float t0 = m0, t1 = m1;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[h][e] = j0 + h * 8 + tq * 2 + (e & 1) < hi ? x[h][e] * s2 : -INFINITY;
        if (e < 2) t0 = fmaxf(t0, x[h][e]);
        else t1 = fmaxf(t1, x[h][e]);
      }
#pragma unroll
    for (int w = 1; w <= 2; w <<= 1) {
      t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, w));
      t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, w));
    }
    if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
      const float f0 = ex2(m0 - t0), f1 = ex2(m1 - t1);
      m0 = t0;
      m1 = t1;
      l0 *= f0;
      l1 *= f1;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f0;
        o[i][2] *= f1;
        o[i][3] *= f1;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[h][e] = ex2(x[h][e] - (e < 2 ? m0 : m1));
        if (e < 2) l0 += x[h][e];
        else l1 += x[h][e];
      }
    const uint32_t ph[4] = {pack2(x[0][0], x[0][1]), pack2(x[0][2], x[0][3]), pack2(x[1][0], x[1][1]),
                            pack2(x[1][2], x[1][3])};
    const uint32_t pl[4] = {rest2(x[0][0], x[0][1], ph[0]), rest2(x[0][2], x[0][3], ph[1]),
                            rest2(x[1][0], x[1][1], ph[2]), rest2(x[1][2], x[1][3], ph[3])};
#pragma unroll
    for (int c = 0; c < Cf::CH; c += 2) {
      uint32_t f[4];  // values: channels 8c .. 8c + 7 of keys 0-7, 8-15, then the next eight channels
      ldm4<true>(vt + Cf::at((mat & 1) * 8 + mr, c + (mat >> 1)), f);
      mma16816(o[c], ph, f[0], f[1]);
      mma16816(o[c + 1], ph, f[2], f[3]);
      mma16816(o[c], pl, f[0], f[1]);
      mma16816(o[c + 1], pl, f[2], f[3]);
    }
    __syncwarp();  // the slot is filled again by all lanes in the next round
  }
  copy_wait<0>();
  __syncthreads();
  float* so = reinterpret_cast<float*>(sm);  // [warp][16][D] over the rings
#pragma unroll
  for (int w = 1; w <= 2; w <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, w);
    l1 += __shfl_xor_sync(0xffffffffu, l1, w);
  }
  if (tq == 0) {
    sh_m[warp][g] = m0;
    sh_m[warp][g + 8] = m1;
    sh_l[warp][g] = l0;
    sh_l[warp][g + 8] = l1;
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i) {
    *reinterpret_cast<float2*>(so + (warp * 16 + g) * D + i * 8 + tq * 2) = make_float2(o[i][0], o[i][1]);
    if (heads > 8)
      *reinterpret_cast<float2*>(so + (warp * 16 + g + 8) * D + i * 8 + tq * 2) = make_float2(o[i][2], o[i][3]);
  }
  __syncthreads();
  finish<T, D, 16>(a, b, hk * group + g0, heads, n, &sh_m[0][0], &sh_l[0][0], so);
}

// Joins the parts (at most kDecodeParts) of one head: the parts' weights first,
// in shared memory, then each channel's sum with its loads in flight together.
// An idle sequence, whose out is zero, is told by its parts' sum of -1: a live
// one's is not negative, but it may be NaN, which is then the answer.
template <typename T, int D>
__global__ void __launch_bounds__(D) swa_decode_join_kernel(const float* __restrict__ part, int splits,
                                                            T* __restrict__ out) {
  __shared__ float m[kDecodeParts], w[kDecodeParts];
  const float* p = part + (size_t)blockIdx.x * splits * (D + 2);
  for (int s = threadIdx.x; s < splits; s += D) {
    const float2 v = *reinterpret_cast<const float2*>(p + (size_t)s * (D + 2));
    m[s] = v.x;
    w[s] = v.y;
  }
  __syncthreads();
  float top = kLowest, sum = 0.f, acc = 0.f;
  for (int s = 0; s < splits; ++s) top = fmaxf(top, m[s]);
#pragma unroll 8
  for (int s = 0; s < splits; ++s) {
    const float f = m[s] == kLowest ? 0.f : ex2(m[s] - top);  // 0 for an empty part
    sum = fmaf(f, w[s], sum);
    acc = fmaf(f, p[(size_t)s * (D + 2) + 2 + threadIdx.x], acc);
  }
  out[(size_t)blockIdx.x * D + threadIdx.x] = from_f<T>(w[0] < 0.f ? 0.f : acc / sum);
}

int pieces_of(long long slots) { return (int)((slots + 63) / 64 < kDecodeParts ? (slots + 63) / 64 : kDecodeParts); }

// Query heads of a key head that one CTA takes.  bf16: all, up to the 16 rows
// of a product.  fp32, where each costs arithmetic: the fewest of 1, 2, 4 whose
// CTAs still run at once when a cluster shares each cache.  H16 Hk4 d128 window
// 1024, us with 4, 2, 1: 12, 10, 9 for one sequence, 14, 12, 13 for 4, 23, 24,
// 40 for 16, 90, 106, 152 for 64 (each in its best number of parts).
int heads_per_cta(int B, int H, int Hk, int window, int sinks, int dtype) {
  if (dtype == 1) return 16;
  const int group = H / Hk, parts = pieces_of((long long)window + sinks);
  int gc = 1;
  while (gc < 4 && gc < group &&
         (long long)B * Hk * ((group + gc - 1) / gc) * (parts < kDecodeCluster ? parts : kDecodeCluster) > kDecodeCtas)
    gc *= 2;
  return gc;
}

// One CTA per part, key head (or 16, 4 of its query heads) and sequence; the
// parts of up to kDecodeCluster are a cluster.
template <typename T, int D, typename K>
cudaError_t decode_go(const SwaDecodeArgs& a, K kernel, size_t smem, cudaStream_t st) {
  const int gc = heads_per_cta(a.B, a.H, a.Hk, a.window, a.sinks, a.dtype);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.splits, a.Hk * ((a.H / a.Hk + gc - 1) / gc), a.B);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = a.part ? 1 : a.splits;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = a.splits > 1 && !a.part ? 1 : 0;
  prof_begin(st, "swa_decode");
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  prof_end(st);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  prof_begin(st, "swa_decode_join");
  swa_decode_join_kernel<T, D><<<a.B * a.H, D, 0, st>>>(a.part, a.splits, static_cast<T*>(a.out));
  prof_end(st);
  return cudaGetLastError();
}

template <int D>
cudaError_t decode_f32(const SwaDecodeArgs& a, cudaStream_t st) {
  switch (heads_per_cta(a.B, a.H, a.Hk, a.window, a.sinks, 0)) {
    case 1: return decode_go<float, D>(a, swa_decode_kernel<float, D, 1>, 0, st);
    case 2: return decode_go<float, D>(a, swa_decode_kernel<float, D, 2>, 0, st);
    default: return decode_go<float, D>(a, swa_decode_kernel<float, D, 4>, 0, st);
  }
}

template <int D>
cudaError_t decode_bf16(const SwaDecodeArgs& a, cudaStream_t st) {
  using Cf = MmaCfg<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(swa_decode_mma_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::BYTES);
  return e != cudaSuccess ? e : decode_go<__nv_bfloat16, D>(a, swa_decode_mma_kernel<D>, Cf::BYTES, st);
}

// Per slot: the newest of the first n tokens that belongs there.  One 16-byte
// vector per thread; 16 x 2052 slots of 4 x 128 bf16 (135 MB): 27 us, 5 TB/s.
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

// Parts of a cache: as many as run at once, at least 64 slots to a part.
int swa_decode_splits(int B, int H, int Hk, int window, int sinks, int dtype) {
  const int gc = heads_per_cta(B, H, Hk, window, sinks, dtype);
  const long long units = (long long)B * Hk * ((H / Hk + gc - 1) / gc), slots = (long long)window + sinks;
  long long s = kDecodeCtas / units;
  if (s > pieces_of(slots)) s = pieces_of(slots);
  if (s > kDecodeCluster && slots * (dtype == 1 ? 2 : 4) <= kDecodeClusterBytes) s = kDecodeCluster;
  return s < 1 ? 1 : (int)s;
}

size_t swa_decode_bytes(int B, int H, int d, int splits) {
  return splits <= kDecodeCluster ? 0 : (size_t)B * H * splits * (d + 2) * sizeof(float);
}

cudaError_t launch_swa_decode(const SwaDecodeArgs& a, cudaStream_t st) {
  if (a.dtype == 1)
    return a.d == 32 ? decode_bf16<32>(a, st) : a.d == 64 ? decode_bf16<64>(a, st) : decode_bf16<128>(a, st);
  return a.d == 32 ? decode_f32<32>(a, st) : a.d == 64 ? decode_f32<64>(a, st) : decode_f32<128>(a, st);
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
