// k_attention_few.cu -- attention of few queries over many keys, forward.
//
// With at most 16 rows (tokens times the query heads of a key head) the keys
// and values are read once and that is the cost: HBM bounds it.  A tile of 128
// rows on tcgen05 would leave one warp with the arithmetic of a whole key tile;
// here every warp takes blocks of 16 keys of its own and runs the products as
// 16 x 8 x 16 register-level matrix instructions, straight from global loads,
// with no shared memory or barrier until the warps' results are joined.  Both
// products are free to permute the summed index, so that each thread's 16-byte
// load is its operand: channels of k, and channels of v for the output.
#include "ffdp_attention.cuh"

namespace ffdp {

namespace {

constexpr int kWarps = 8, kThreads = kWarps * 32;

template <class T>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__half>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const void* p) { return __ldg(static_cast<const uint4*>(p)); }

// DP: channels rounded up to 64 or 128.
template <class T, int DP, bool AXES, bool CAP>
__global__ void __launch_bounds__(kThreads, 1) k_attn_few(const AttnArgs a, const FewArgs f) {
  __shared__ float buf[kWarps / 2][16][DP];
  __shared__ float sm_m[kWarps][16], sm_l[kWarps][16];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, q4 = lane % 4, g8 = lane / 4;
  const int split = blockIdx.x % f.splits, bg = blockIdx.x / f.splits, b = bg / a.Hk, g = bg - b * a.Hk;
  const int rows = a.G * a.Sq, prefix = prefix_of(a, b);
  // this thread's two rows
  int i[2], h[2], limit[2], doc[2];
  bool valid[2];
  float pq[2][3], sl[2][3];
  uint32_t qa[DP / 32][2][4];  // [32 channels][half of a thread's 8][A registers]
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    const int r = g8 + 8 * y;
    valid[y] = r < rows;
    const int hl = valid[y] ? r / a.Sq : 0;
    i[y] = valid[y] ? r - hl * a.Sq : 0;
    h[y] = g * a.G + hl;
    limit[y] = valid[y] ? key_limit(a, prefix, i[y]) : a.Sk;
    doc[y] = a.doc_q ? a.doc_q[b * a.doc_q_sb + i[y]] : 0;
    if (doc[y] < 0) doc[y] = -2;
    if (AXES) {
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        pq[y][x] = x < a.axes ? a.pos_q[b * a.pos_q_sb + (int64_t)i[y] * a.axes + x] : 0.0f;
        sl[y][x] = x < a.axes ? a.slopes[h[y] * a.axes + x] * kLog2e : 0.0f;
      }
    }
    const T* p = static_cast<const T*>(a.q.p) + b * a.q.sb + (int64_t)i[y] * a.q.st + h[y] * a.q.sh;
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
      const int ch = 32 * c + 8 * q4;
      const uint4 u = valid[y] && ch < a.D ? load16(p + ch) : make_uint4(0, 0, 0, 0);
      qa[c][0][y] = u.x;
      qa[c][0][2 + y] = u.y;
      qa[c][1][y] = u.z;
      qa[c][1][2 + y] = u.w;
    }
  }
  // blocks of 16 keys of this split (the last query of a causal call sees the last key)
  const int nb = (a.Sk + 15) / 16;
  const int n0 = (int)((int64_t)nb * split / f.splits), n1 = (int)((int64_t)nb * (split + 1) / f.splits);
  float o[DP / 64][8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {};
  const T* kbase = static_cast<const T*>(a.k.p) + b * a.k.sb + g * a.k.sh;
  const T* vbase = static_cast<const T*>(a.v.p) + b * a.v.sb + g * a.v.sh;
#pragma unroll 1
  for (int n = n0 + warp; n < n1; n += kWarps) {
    const int j0 = n * 16;
    uint4 kw[2][DP / 32], vw[4][DP / 64];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int j = j0 + 8 * t + g8;
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        const int ch = 32 * c + 8 * q4;
        kw[t][c] = j < a.Sk && ch < a.D ? load16(kbase + (int64_t)j * a.k.st + ch) : make_uint4(0, 0, 0, 0);
      }
    }
    int key[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // keys 2 q4, 2 q4 + 1, and both + 8
      key[e] = j0 + 2 * q4 + (e & 1) + 8 * (e >> 1);
#pragma unroll
      for (int c = 0; c < DP / 64; ++c) {
        const int ch = 64 * c + 8 * g8;
        vw[e][c] = key[e] < a.Sk && ch < a.D ? load16(vbase + (int64_t)key[e] * a.v.st + ch) : make_uint4(0, 0, 0, 0);
      }
    }
    float s[2][4] = {};  // [8 keys][row 0: two keys, row 1: two keys]
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int c = 0; c < DP / 32; ++c) {
        mma16816<T>(s[t], qa[c][0], kw[t][c].x, kw[t][c].y);
        mma16816<T>(s[t], qa[c][1], kw[t][c].z, kw[t][c].w);
      }
    bool hidden = false;
    bool see[2][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float pk[3];
      if (AXES) {
#pragma unroll
        for (int x = 0; x < 3; ++x)
          pk[x] = x < a.axes && key[e] < a.Sk ? __ldg(a.pos_k + b * a.pos_k_sb + (int64_t)key[e] * a.axes + x) : 0.0f;
      }
      const int dk = a.doc_k && key[e] < a.Sk ? __ldg(a.doc_k + b * a.doc_k_sb + key[e]) : 0;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float& v = s[e >> 1][2 * y + (e & 1)];
        if (CAP) {
          v = fmaf(-2.0f * f.cap2, rcp(1.0f + ex2(v * f.cap_in)), f.cap2);
        } else {
          v *= f.c;
        }
        if (AXES) {
#pragma unroll
          for (int x = 0; x < 3; ++x) v = fmaf(-sl[y][x], fabsf(pq[y][x] - pk[x]), v);
        }
        see[y][e] = key[e] < limit[y] && (!a.doc_q || dk == doc[y]);
        hidden |= valid[y] && key[e] < a.Sk && !see[y][e];
        if (!see[y][e]) v = -INFINITY;
      }
    }
    if ((a.causal || a.doc_q) && __any_sync(0xffffffffu, hidden)) {
      // a value row that is not finite must not reach the rows that do not see
      // it: cleared, and the rows that see it become NaN
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t z = 0;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c) {
          z = zero_times<T>(vw[e][c].x, z);
          z = zero_times<T>(vw[e][c].y, z);
          z = zero_times<T>(vw[e][c].z, z);
          z = zero_times<T>(vw[e][c].w, z);
        }
        z &= 0x7fff7fffu;
        z |= __shfl_xor_sync(0xffffffffu, z, 4);
        z |= __shfl_xor_sync(0xffffffffu, z, 8);
        z |= __shfl_xor_sync(0xffffffffu, z, 16);
        if (z) {
#pragma unroll
          for (int c = 0; c < DP / 64; ++c) vw[e][c] = make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (see[y][e]) s[e >> 1][2 * y + (e & 1)] = NAN;
        }
      }
    }
    float top[2];
    bool grow = false;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      top[y] = fmaxf(max3(s[0][2 * y], s[0][2 * y + 1], s[1][2 * y]), s[1][2 * y + 1]);
      top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 1));
      top[y] = fmaxf(top[y], __shfl_xor_sync(0xffffffffu, top[y], 2));
      grow |= top[y] > m[y] + 8.0f || (m[y] == -INFINITY && top[y] > m[y]);
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float mn = fmaxf(m[y], top[y]), w = mn == -INFINITY ? 1.0f : ex2(m[y] - mn);
        m[y] = mn;
        l[y] *= w;
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) o[c][j][2 * y] *= w, o[c][j][2 * y + 1] *= w;
      }
    }
    uint32_t p[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const float mm = m[y] == -INFINITY ? 0.0f : m[y];
        const float p0 = ex2(s[t][2 * y] - mm), p1 = ex2(s[t][2 * y + 1] - mm);
        l[y] += p0 + p1;
        p[2 * t + y] = pack2<T>(p0, p1);
      }
#pragma unroll
    for (int c = 0; c < DP / 64; ++c) {
      const uint32_t w[4][4] = {{vw[0][c].x, vw[0][c].y, vw[0][c].z, vw[0][c].w}, {vw[1][c].x, vw[1][c].y, vw[1][c].z, vw[1][c].w},
                                {vw[2][c].x, vw[2][c].y, vw[2][c].z, vw[2][c].w}, {vw[3][c].x, vw[3][c].y, vw[3][c].z, vw[3][c].w}};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned half = j & 1 ? 0x7632u : 0x5410u;
        mma16816<T>(o[c][j], p, __byte_perm(w[0][j / 2], w[1][j / 2], half), __byte_perm(w[2][j / 2], w[3][j / 2], half));
      }
    }
  }
  // join the warps: common maximum, sums in the order of the warps
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
    l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
    if (q4 == 0) sm_m[warp][g8 + 8 * y] = m[y], sm_l[warp][g8 + 8 * y] = l[y];
  }
  __syncthreads();
  float mt[2], lt[2];
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    mt[y] = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mt[y] = fmaxf(mt[y], sm_m[w][g8 + 8 * y]);
    const float ref = mt[y] == -INFINITY ? 0.0f : mt[y];
    lt[y] = 0.0f;
    for (int w = 0; w < kWarps; ++w) lt[y] += sm_l[w][g8 + 8 * y] * ex2(sm_m[w][g8 + 8 * y] - ref);
    const float w = ex2(m[y] - ref);
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) o[c][j][2 * y] *= w, o[c][j][2 * y + 1] *= w;
  }
  // row r, channels 64 c + 16 q4 + {0 .. 15} of this thread: o[c][j][2 y] is channel j, [2 y + 1] channel 8 + j
  for (int step = kWarps / 2; step; step >>= 1) {
    if (warp >= step && warp < 2 * step) {
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            buf[warp - step][g8 + 8 * y][64 * c + 16 * q4 + j] = o[c][j][2 * y];
            buf[warp - step][g8 + 8 * y][64 * c + 16 * q4 + 8 + j] = o[c][j][2 * y + 1];
          }
    }
    __syncthreads();
    if (warp < step) {
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int c = 0; c < DP / 64; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            o[c][j][2 * y] += buf[warp][g8 + 8 * y][64 * c + 16 * q4 + j];
            o[c][j][2 * y + 1] += buf[warp][g8 + 8 * y][64 * c + 16 * q4 + 8 + j];
          }
    }
    __syncthreads();
  }
  if (warp != 0) return;
#pragma unroll
  for (int y = 0; y < 2; ++y) {
    if (!valid[y]) continue;
    const float inv = lt[y] == 0.0f ? 0.0f : 1.0f / lt[y], lse2 = lt[y] == 0.0f ? -INFINITY : mt[y] + log2f(lt[y]);
    const int64_t row = ((int64_t)b * a.Hq + h[y]) * a.Sq + i[y], all = (int64_t)a.B * a.Hq * a.Sq;
    if (q4 == 0) {
      if (f.splits > 1)
        f.part[all * a.D * f.splits + split * all + row] = lse2;
      else if (a.lse)
        a.lse[row] = lse2 * kLn2;
    }
#pragma unroll
    for (int c = 0; c < DP / 64; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int ch = 64 * c + 16 * q4 + 8 * e;
        if (ch >= a.D) continue;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = lt[y] == 0.0f ? 0.0f : o[c][j][2 * y + e] * inv;
        if (f.splits > 1) {
          float4* p = reinterpret_cast<float4*>(f.part + (split * all + row) * a.D + ch);
          p[0] = make_float4(v[0], v[1], v[2], v[3]);
          p[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
          T* p = static_cast<T*>(a.o.p) + b * a.o.sb + (int64_t)i[y] * a.o.st + h[y] * a.o.sh + ch;
          *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(v[0], v[1]), pack2<T>(v[2], v[3]), pack2<T>(v[4], v[5]), pack2<T>(v[6], v[7]));
        }
      }
  }
}

template <class T, int DP>
void pick(const AttnArgs& a, const FewArgs& f, unsigned grid, cudaStream_t s) {
  if (a.axes) {
    if (a.cap > 0.0f) k_attn_few<T, DP, true, true><<<grid, kThreads, 0, s>>>(a, f);
    else k_attn_few<T, DP, true, false><<<grid, kThreads, 0, s>>>(a, f);
  } else {
    if (a.cap > 0.0f) k_attn_few<T, DP, false, true><<<grid, kThreads, 0, s>>>(a, f);
    else k_attn_few<T, DP, false, false><<<grid, kThreads, 0, s>>>(a, f);
  }
}

}  // namespace

// One CTA per SM: as many splits as fill the SMs, each with a block of 16 keys
// per warp at least.
int few_splits(int64_t pairs, int64_t keys, int sms) {
  int64_t s = pairs < 1 ? 1 : sms / pairs;
  const int64_t most = keys / (16 * kWarps);
  if (s > most) s = most;
  return (int)(s < 1 ? 1 : s);
}

cudaError_t launch_attention_few(int dt, const AttnArgs& a, const FewArgs& f, cudaStream_t s) {
  const unsigned grid = (unsigned)((int64_t)a.B * a.Hk * f.splits);
  note_launch_begin("k_attn_few", s);
  FFDP_TOK_SWITCH16(dt, T, {
    if (a.D <= 64)
      pick<T, 64>(a, f, grid, s);
    else
      pick<T, 128>(a, f, grid, s);
  });
  note_launch_end(s);
  return cudaGetLastError();
}

}  // namespace ffdp
