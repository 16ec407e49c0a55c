// kd_rotary.cu -- rotary positions of q and k, and their backward.
//
// Pair j of a token at position p turns by theta = p w_j:
//   (y1, y2) = s (x1 cos theta - x2 sin theta, x1 sin theta + x2 cos theta),
// the backward by -theta.  Pairs are (j, j + rot/2) or (2j, 2j + 1); channels
// from rot on are copied.
//
// The angle is a product in 64 bits, reduced to a fraction of a turn there
// (at position 2^20 an fp32 product is off by 0.06 rad), and only the fraction
// goes to fp32's sincospi.
//
// Every element is read and written once.  One sine and cosine serve all heads
// of a token, so a CTA takes whole tokens: it fills a table of its tokens' rot/2
// pairs in shared memory, then moves the heads' rows as vectors, x threads to a
// row and y rows at a time.  16384 tokens of 16 + 4 heads of 128 bf16 (168 MB):
// 33 to 35 us, 5 TB/s.  What bounds it is the table's reads: the shared-memory
// pipe is at 73% of its rate, three quarters of that for the table, whose vectors
// for a row's threads lie in the same banks and are read one after another.  With
// two and four rows in flight per thread 53 and 68 us (more registers, fewer
// CTAs), with a thread's first row loaded ahead of the table 43.
#include "kd_hybrid.h"
#include "kd_rows.cuh"

namespace kd {

namespace {

constexpr int kRotThreads = 256;

struct RotaryShape {
  int heads0, heads1, d, rot, tokens;  // tokens per CTA
  int pairs;                           // rot / 2
  int turn_items;                      // vectors of V pairs in a row
  int items;                           // + vectors of the copied channels
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&o)[V]) {
  const Pack<T, V> t = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) o[i] = to_f(t.x[i]);
}

// V: pairs per item.  P: channels per copied vector.
template <typename T, int V, int P, bool kInter>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const T* x0, const T* x1, T* y0, T* y1,
                                                             const double* __restrict__ freqs,
                                                             const long long* __restrict__ pos, long long rows,
                                                             int T_, float scale, float sign, RotaryShape s) {
  extern __shared__ float2 table[];  // [tokens][pairs]: s cos, s sin
  const long long first = (long long)blockIdx.x * s.tokens;
  const int n = (int)(rows - first < s.tokens ? rows - first : s.tokens);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, threads = blockDim.x * blockDim.y;
  for (int i = tid; i < n * s.pairs; i += threads) {
    const int t = i / s.pairs, j = i - t * s.pairs;
    const long long p = pos ? pos[first + t] : (first + t) % T_;
    const double turns = (double)p * freqs[j] * 0.15915494309189533577;  // 1 / (2 pi)
    float sn, cs;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
    table[i] = make_float2(scale * cs, sign * scale * sn);
  }
  __syncthreads();
  const int heads = s.heads0 + s.heads1, it = threadIdx.x;
  for (int r = threadIdx.y; r < n * heads; r += blockDim.y) {
    const int t = r / heads, h = r - t * heads;
    const size_t row = (size_t)(first + t);
    const bool second = h >= s.heads0;
    const size_t off = (second ? row * s.heads1 + (h - s.heads0) : row * s.heads0 + h) * s.d;
    const T* x = (second ? x1 : x0) + off;
    T* y = (second ? y1 : y0) + off;
    if (it < s.turn_items) {
      const float2* cs = table + t * s.pairs + it * V;
      if (kInter) {
        float a[2 * V];
        load_vec<T, 2 * V>(x + it * 2 * V, a);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u = a[2 * i], w = a[2 * i + 1];
          a[2 * i] = u * cs[i].x - w * cs[i].y;
          a[2 * i + 1] = u * cs[i].y + w * cs[i].x;
        }
        store_row<T, 2 * V>(y + it * 2 * V, a);
      } else {
        float a[V], b[V];
        load_vec<T, V>(x + it * V, a);
        load_vec<T, V>(x + s.pairs + it * V, b);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float u = a[i], w = b[i];
          a[i] = u * cs[i].x - w * cs[i].y;
          b[i] = u * cs[i].y + w * cs[i].x;
        }
        store_row<T, V>(y + it * V, a);
        store_row<T, V>(y + s.pairs + it * V, b);
      }
    } else {
      const int c = s.rot + (it - s.turn_items) * P;
      *reinterpret_cast<Pack<T, P>*>(y + c) = *reinterpret_cast<const Pack<T, P>*>(x + c);
    }
  }
}

template <typename T, int V, int P, bool kInter>
cudaError_t rotary_go(const RotaryArgs& a, RotaryShape s, cudaStream_t st) {
  s.turn_items = s.pairs / V;
  s.items = s.turn_items + (s.d - s.rot) / P;
  const dim3 block(s.items, kRotThreads / s.items);
  const long long grid = (a.rows + s.tokens - 1) / s.tokens;
  prof_begin(st, a.inverse ? "rotary_bwd" : "rotary_fwd");
  rotary_kernel<T, V, P, kInter><<<(unsigned)grid, block, (size_t)s.tokens * s.pairs * sizeof(float2), st>>>(
      static_cast<const T*>(a.x[0]), static_cast<const T*>(a.x[1]), static_cast<T*>(a.y[0]),
      static_cast<T*>(a.y[1]), a.freqs, a.pos, a.rows, a.T, a.scale, a.inverse ? -1.f : 1.f, s);
  prof_end(st);
  return cudaGetLastError();
}

int pow2_in(int n, int most) {
  int v = most;
  while (n % v) v >>= 1;
  return v;
}

// Copied channels start at rot, so their vectors divide rot (and d - rot).
template <typename T, int V, bool kInter>
cudaError_t rotary_copy(const RotaryArgs& a, const RotaryShape& s, cudaStream_t st) {
  switch (pow2_in(s.rot, 16 / (int)sizeof(T))) {
    case 8: return rotary_go<T, V, 16 / sizeof(T), kInter>(a, s, st);
    case 4: return rotary_go<T, V, 4, kInter>(a, s, st);
    default: return rotary_go<T, V, 2, kInter>(a, s, st);
  }
}

template <typename T>
cudaError_t rotary_t(const RotaryArgs& a, const RotaryShape& s, cudaStream_t st) {
  // 16-byte vectors where the number of pairs allows them (at 16384 x 32 heads
  // of 128 bf16 48 us; 4-byte ones 66, single channels 108): a half-layout
  // item is two vectors of V channels, an interleaved one a vector of 2V
  constexpr int W = 16 / sizeof(T);
  if (a.interleaved) {
    switch (pow2_in(s.pairs, W / 2)) {
      case 4: return rotary_copy<T, W / 2, true>(a, s, st);
      case 2: return rotary_copy<T, 2, true>(a, s, st);
      default: return rotary_copy<T, 1, true>(a, s, st);
    }
  }
  switch (pow2_in(s.pairs, W)) {
    case 8: return rotary_copy<T, W, false>(a, s, st);
    case 4: return rotary_copy<T, 4, false>(a, s, st);
    case 2: return rotary_copy<T, 2, false>(a, s, st);
    default: return rotary_copy<T, 1, false>(a, s, st);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, cudaStream_t st) {
  RotaryShape s{};
  s.heads0 = a.heads[0];
  s.heads1 = a.heads[1];
  s.d = a.d;
  s.rot = a.rot;
  s.pairs = a.rot / 2;
  // Tokens per CTA: up to 8 while that leaves 512 CTAs and at most 32 KB to one.
  // 1 and 4 (8) tokens, us: 2.8 and 4.1 for 256 tokens of 16 + 16 heads of 128
  // bf16, 14.7 and 13.9 for 4096, 57.7 and 48.4 for 16384; 25.6 and 10.2 (9.5)
  // for 16384 of 8 + 2 heads of 64.
  const long long row = (long long)(a.heads[0] + a.heads[1]) * a.d * (a.dtype == 1 ? 2 : 4);
  s.tokens = 1;
  while (s.tokens < 8 && a.rows / (2 * s.tokens) >= 512 && 2 * s.tokens * row <= 32768) s.tokens *= 2;
  return a.dtype == 1 ? rotary_t<__nv_bfloat16>(a, s, st) : rotary_t<float>(a, s, st);
}

}  // namespace kd
