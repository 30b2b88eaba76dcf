// k_attention_bwd.cu -- attention over volume tokens, backward.
//
// One warp per query row (gq) or key row (gk, gv): a dot product per pair
// across the lanes.
#include "ffdp_tokens.h"

namespace ffdp {

namespace {

constexpr int kWarps = 8;
constexpr int kE = 4;  // channels per lane (head_dim <= 128)

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <class T>
__device__ __forceinline__ void row(const HeadsView& t, int b, int s, int h, int D, float* f) {
  const T* p = static_cast<const T*>(t.p) + b * t.sb + s * t.st + h * t.sh;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int c = (threadIdx.x & 31) + 32 * e;
    f[e] = c < D ? to_f32<T>(p[c]) : 0.0f;
  }
}

template <class T>
__device__ __forceinline__ void put(const HeadsView& t, int b, int s, int h, int D, const float* f) {
  T* p = static_cast<T*>(t.p) + b * t.sb + s * t.st + h * t.sh;
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    const int c = (threadIdx.x & 31) + 32 * e;
    if (c < D) p[c] = from_f32<T>(f[e]);
  }
}

__device__ __forceinline__ float dot(const float* a, const float* b) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < kE; ++e) s = fmaf(a[e], b[e], s);
  return warp_sum(s);
}

__device__ __forceinline__ bool visible(const AttnArgs& a, int b, int i, int j) {
  if (a.causal && j > i + a.Sk - a.Sq && (!a.prefix || j >= a.prefix[b])) return false;
  if (a.doc_q) {
    const int d = a.doc_q[b * a.doc_q_sb + i];
    if (d < 0 || d != a.doc_k[b * a.doc_k_sb + j]) return false;
  }
  return true;
}

// score of a pair from its product, and d score / d (scale product)
__device__ __forceinline__ float score(const AttnArgs& a, int b, int h, int i, int j, float qk, float* slope) {
  float s = qk * a.scale;
  *slope = 1.0f;
  if (a.cap > 0.0f) {
    const float t = tanhf(s / a.cap);
    s = a.cap * t;
    *slope = 1.0f - t * t;
  }
  for (int x = 0; x < a.axes; ++x)
    s -= a.slopes[h * a.axes + x] *
         fabsf(a.pos_q[b * a.pos_q_sb + (int64_t)i * a.axes + x] - a.pos_k[b * a.pos_k_sb + (int64_t)j * a.axes + x]);
  return s;
}

template <class T>
__global__ void __launch_bounds__(kWarps * 32) k_attn_bwd_q(const AttnArgs a) {
  const int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (r >= (int64_t)a.B * a.Hq * a.Sq) return;
  const int i = (int)(r % a.Sq), h = (int)(r / a.Sq % a.Hq), b = (int)(r / a.Sq / a.Hq), g = h / a.G;
  float q[kE], o[kE], go[kE], gq[kE] = {};
  row<T>(a.q, b, i, h, a.D, q);
  row<T>(a.o, b, i, h, a.D, o);
  row<T>(a.go, b, i, h, a.D, go);
  const float delta = dot(o, go), lse = a.lse[r];
  if ((threadIdx.x & 31) == 0) a.delta[r] = delta;
  for (int j = 0; j < a.Sk; ++j) {
    if (!visible(a, b, i, j)) continue;
    float k[kE], v[kE], slope;
    row<T>(a.k, b, j, g, a.D, k);
    row<T>(a.v, b, j, g, a.D, v);
    const float p = expf(score(a, b, h, i, j, dot(q, k), &slope) - lse);
    const float ds = p * (dot(go, v) - delta) * slope * a.scale;
#pragma unroll
    for (int e = 0; e < kE; ++e) gq[e] = fmaf(ds, k[e], gq[e]);
  }
  put<T>(a.gq, b, i, h, a.D, gq);
}

template <class T>
__global__ void __launch_bounds__(kWarps * 32) k_attn_bwd_kv(const AttnArgs a) {
  const int64_t r = (int64_t)blockIdx.x * kWarps + threadIdx.x / 32;
  if (r >= (int64_t)a.B * a.Hk * a.Sk) return;
  const int j = (int)(r % a.Sk), g = (int)(r / a.Sk % a.Hk), b = (int)(r / a.Sk / a.Hk);
  float k[kE], v[kE], gk[kE] = {}, gv[kE] = {};
  row<T>(a.k, b, j, g, a.D, k);
  row<T>(a.v, b, j, g, a.D, v);
  for (int h = g * a.G; h < (g + 1) * a.G; ++h)
    for (int i = 0; i < a.Sq; ++i) {
      if (!visible(a, b, i, j)) continue;
      float q[kE], go[kE], slope;
      row<T>(a.q, b, i, h, a.D, q);
      row<T>(a.go, b, i, h, a.D, go);
      const int64_t at = ((int64_t)b * a.Hq + h) * a.Sq + i;
      const float p = expf(score(a, b, h, i, j, dot(q, k), &slope) - a.lse[at]);
      const float ds = p * (dot(go, v) - a.delta[at]) * slope * a.scale;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        gv[e] = fmaf(p, go[e], gv[e]);
        gk[e] = fmaf(ds, q[e], gk[e]);
      }
    }
  put<T>(a.gk, b, j, g, a.D, gk);
  put<T>(a.gv, b, j, g, a.D, gv);
}

unsigned blocks(int64_t rows) { return (unsigned)((rows + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_attention_bwd(int dt, const AttnArgs& a, cudaStream_t s) {
  if (a.Sq) {
    note_launch_begin("k_attn_bwd_q", s);
    FFDP_TOK_SWITCH16(dt, T, (k_attn_bwd_q<T><<<blocks((int64_t)a.B * a.Hq * a.Sq), kWarps * 32, 0, s>>>(a)));
    note_launch_end(s);
  }
  if (a.Sk) {
    note_launch_begin("k_attn_bwd_kv", s);
    FFDP_TOK_SWITCH16(dt, T, (k_attn_bwd_kv<T><<<blocks((int64_t)a.B * a.Hk * a.Sk), kWarps * 32, 0, s>>>(a)));
    note_launch_end(s);
  }
  return cudaGetLastError();
}

}  // namespace ffdp
