// k_linear.cu -- matrix products of the linear operator and its gradients.
//
// C[m][n] = sum_k A(m, k) B(n, k): the forward product (x w^T), gx = gz w and
// gw = gz^T x are this product with other strides.
#include "ffdp_tokens.h"

namespace ffdp {

namespace {

constexpr int kTile = 64, kStep = 16;

__device__ __forceinline__ float act_fwd(int act, float z) {
  switch (act) {
    case 1: return fmaxf(z, 0.0f);
    case 2: return 0.5f * z * (1.0f + erff(z * 0.70710678f));
    case 3: return z / (1.0f + expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ float act_grad(int act, float z) {
  switch (act) {
    case 1: return z > 0.0f ? 1.0f : 0.0f;
    case 2: return 0.5f * (1.0f + erff(z * 0.70710678f)) + z * expf(-0.5f * z * z) * 0.39894228f;
    case 3: {
      const float g = 1.0f / (1.0f + expf(-z));
      return g * (1.0f + z * (1.0f - g));
    }
    default: return 1.0f;
  }
}

template <class T>
__global__ void __launch_bounds__(256) k_linear(const LinearArgs a, int tiles_n) {
  __shared__ float sa[kStep][kTile + 1], sb[kStep][kTile + 1];
  const int m0 = blockIdx.x / tiles_n * kTile, n0 = blockIdx.x % tiles_n * kTile;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float c[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kStep) {
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int ka = a.ak == 1 ? i % kStep : i / kTile, ra = a.ak == 1 ? i / kStep : i % kTile;
      sa[ka][ra] = m0 + ra < a.M && k0 + ka < a.K ? to_f32<T>(static_cast<const T*>(a.a)[(m0 + ra) * a.am + (k0 + ka) * a.ak]) : 0.0f;
      const int kb = a.bk == 1 ? i % kStep : i / kTile, rb = a.bk == 1 ? i / kStep : i % kTile;
      sb[kb][rb] = n0 + rb < a.N && k0 + kb < a.K ? to_f32<T>(static_cast<const T*>(a.b)[(n0 + rb) * a.bn + (k0 + kb) * a.bk]) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kStep; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], c[i][j]);
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      float z = c[i][j];
      if (a.bias) z += to_f32<T>(static_cast<const T*>(a.bias)[n]);
      if (a.z) static_cast<T*>(a.z)[m * a.ldz + n] = from_f32<T>(z);
      z = act_fwd(a.act, z);
      if (a.res) z += to_f32<T>(static_cast<const T*>(a.res)[m * a.ldr + n]);
      static_cast<T*>(a.c)[m * a.ldc + n] = from_f32<T>(z);
    }
}

// One thread per column and chunk of rows.
template <class T>
__global__ void __launch_bounds__(128) k_linear_gz(const LinearGradArgs a, int rows) {
  const int n = blockIdx.x * 128 + threadIdx.x;
  if (n >= a.N) return;
  const int m0 = blockIdx.y * rows, m1 = min(a.M, m0 + rows);
  float sum = 0.0f;
  for (int64_t m = m0; m < m1; ++m) {
    float g = to_f32<T>(static_cast<const T*>(a.gy)[m * a.ldgy + n]);
    if (a.gz) {
      g *= act_grad(a.act, to_f32<T>(static_cast<const T*>(a.z)[m * a.ldz + n]));
      static_cast<T*>(a.gz)[m * a.ldgz + n] = from_f32<T>(g);
    }
    sum += g;
  }
  if (a.partial) a.partial[(int64_t)blockIdx.y * a.N + n] = sum;
}

template <class T>
__global__ void __launch_bounds__(128) k_linear_gb(const LinearGradArgs a) {
  const int n = blockIdx.x * 128 + threadIdx.x;
  if (n >= a.N) return;
  float sum = 0.0f;
  for (int c = 0; c < a.chunks; ++c) sum += a.partial[(int64_t)c * a.N + n];
  static_cast<T*>(a.gb)[n] = from_f32<T>(sum);
}

}  // namespace

cudaError_t launch_linear(int dt, const LinearArgs& a, cudaStream_t s) {
  const int tn = (a.N + kTile - 1) / kTile;
  const int64_t grid = (int64_t)((a.M + kTile - 1) / kTile) * tn;
  note_launch_begin("k_linear", s);
  FFDP_TOK_SWITCH16(dt, T, (k_linear<T><<<(unsigned)grid, 256, 0, s>>>(a, tn)));
  note_launch_end(s);
  return cudaGetLastError();
}

int linear_grad_chunks(int M, int N, int sms) {
  const int cols = (N + 127) / 128;
  int c = (sms * 8 + cols - 1) / cols;
  const int most = (M + 31) / 32;
  c = c < most ? c : most;
  return c < 1 ? 1 : c;
}

cudaError_t launch_linear_grad(int dt, const LinearGradArgs& a, cudaStream_t s) {
  const int cols = (a.N + 127) / 128, rows = (a.M + a.chunks - 1) / a.chunks;
  note_launch_begin("k_linear_gz", s);
  FFDP_TOK_SWITCH16(dt, T, (k_linear_gz<T><<<dim3(cols, a.chunks), 128, 0, s>>>(a, rows)));
  note_launch_end(s);
  if (a.gb) {
    note_launch_begin("k_linear_gb", s);
    FFDP_TOK_SWITCH16(dt, T, (k_linear_gb<T><<<cols, 128, 0, s>>>(a)));
    note_launch_end(s);
  }
  return cudaGetLastError();
}

}  // namespace ffdp
