// ffdp_attention.cuh -- what the attention kernels share: visibility of pairs
// of tiles and of single pairs, 16-bit packing, base-2 softmax arithmetic.
#pragma once

#include "ffdp_tc.cuh"
#include "ffdp_tokens.h"

namespace ffdp {

constexpr int kTile = 128;           // tokens per tile, queries and keys
constexpr int kPanel = kTile * 128;  // bytes of 64 channels of a tile in shared memory
constexpr int kMaxCodes = 4096;      // tile codes a CTA keeps; longer ranges are split

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

template <class T> __device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// Whether either half of a packed pair is infinite or NaN.
template <class T> __device__ __forceinline__ bool bad2(uint32_t u);
template <> __device__ __forceinline__ bool bad2<__half>(uint32_t u) {
  return (u & 0x7c00u) == 0x7c00u || (u & 0x7c000000u) == 0x7c000000u;
}
template <> __device__ __forceinline__ bool bad2<__nv_bfloat16>(uint32_t u) {
  return (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
}

// Documents of a tile: range of the valid ids, whether any token is padding.
struct DocRange {
  int lo, hi, pad, unused;
};
__device__ __forceinline__ bool docs_apart(const DocRange& q, const DocRange& k) { return q.hi < k.lo || k.hi < q.lo; }
__device__ __forceinline__ bool docs_one(const DocRange& q, const DocRange& k) {
  return !q.pad && !k.pad && q.lo == q.hi && k.lo == k.hi && q.lo == k.lo;
}

// Number of keys before the first one that query i does not see (documents
// aside): all of them, or the larger of the causal line and the prefix.
__device__ __forceinline__ int key_limit(const AttnArgs& a, int prefix, int i) {
  if (!a.causal) return a.Sk;
  const int c = i + a.Sk - a.Sq + 1;
  return max(0, min(a.Sk, max(prefix, c)));
}
__device__ __forceinline__ int prefix_of(const AttnArgs& a, int b) { return a.prefix ? a.prefix[b] : 0; }

// Tile pair codes: nothing visible, everything visible, some pairs masked.
enum { kSkip = 0, kFull = 1, kMasked = 2 };

// Queries [i0, i1) against keys [k0, k1), each range inside one tile of 128;
// k1 may pass the last key.
__device__ __forceinline__ int pair_code(const AttnArgs& a, int prefix, int b, int i0, int i1, int k0, int k1,
                                         const DocRange* dq, const DocRange* dk) {
  if (i0 >= i1) return kSkip;
  if (k0 >= key_limit(a, prefix, i1 - 1)) return kSkip;
  int code = k1 > key_limit(a, prefix, i0) ? kMasked : kFull;
  if (dq) {
    const DocRange q = dq[(int64_t)b * ((a.Sq + kTile - 1) / kTile) + i0 / kTile];
    const DocRange k = dk[(int64_t)b * ((a.Sk + kTile - 1) / kTile) + k0 / kTile];
    if (docs_apart(q, k)) return kSkip;
    if (!docs_one(q, k)) code = kMasked;
  }
  return code;
}

// A row of a [rows][64 channels per panel] tile in shared memory holds an
// infinity or NaN: zero it (its products with masked weights must vanish) and
// say so.
template <class T>
__device__ __forceinline__ bool clear_bad_row(char* tile, int panels, int panel_bytes, int row) {
  bool bad = false;
  for (int p = 0; p < panels; ++p) {
    const uint4* r = reinterpret_cast<const uint4*>(tile + p * panel_bytes + row * 128);
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 u = r[c];
      bad |= bad2<T>(u.x) || bad2<T>(u.y) || bad2<T>(u.z) || bad2<T>(u.w);
    }
  }
  if (bad)
    for (int p = 0; p < panels; ++p) {
      uint4* r = reinterpret_cast<uint4*>(tile + p * panel_bytes + row * 128);
#pragma unroll
      for (int c = 0; c < 8; ++c) r[c] = make_uint4(0, 0, 0, 0);
    }
  return bad;
}

// Tensor map of [batch][tokens][heads][head_dim]: axes (channel, token, head,
// batch), boxes of 64 channels x `tokens` x `heads`.
inline cudaError_t heads_map(CUtensorMap* m, int dt, const HeadsView& v, int B, int S, int H, int D, int tokens, int heads) {
  const int64_t far = 8 * ((D + 7) / 8);  // any legal stride for extents of one
  const int64_t ext[4] = {D, S > 0 ? S : 1, H, B};
  const int64_t str[3] = {v.st ? v.st : far, v.sh ? v.sh : far, v.sb ? v.sb : far};
  const int box[4] = {64, tokens, heads, 1};
  return make_tensor_map(m, dt, v.p, 4, ext, str, box);
}

cudaError_t launch_doc_ranges(const AttnArgs& a, DocRange* dq, DocRange* dk, cudaStream_t s);

}  // namespace ffdp
