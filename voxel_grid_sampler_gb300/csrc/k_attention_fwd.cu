// k_attention_fwd.cu -- attention over volume tokens, forward.
//
// One CTA holds two tiles of 128 query rows that share their keys: the rows of
// a tile are 128 tokens of one head, or, with few queries, the tokens of
// several heads of one key head.  Per key tile: S = Q K^T on tcgen05 into TMEM;
// a warpgroup per query tile (one row per thread) turns S into scores, keeps
// the running maximum and sum, and writes P = 2^(score - maximum) back to TMEM
// in 16 bits; O += P V on tcgen05.  The two tiles take turns on the tensor
// cores and the arithmetic units.  Warps: 0-3 and 4-7 softmax of tiles 0 and
// 1, 8 loads (TMA), 9 multiplies, 10 prepares the key tile's positions,
// documents and non-finite rows.  Registers: 384 threads start with 168 each; the
// softmax warps, which hold a row of 128 scores, take 208 and leave 88.
#include <atomic>

#include "ffdp_attention.cuh"

namespace ffdp {

namespace {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kMaxStages = 4;
constexpr unsigned kTmemCols = 512;
constexpr float kRescale = 8.0f;  // O and the sum are rescaled when the maximum grew by 2^8

struct FwdArgs {
  AttnArgs a;
  const DocRange *dq, *dk;
  int packed;       // rows of a tile are `rh` tokens of `gb` heads
  int rh, gb;
  int tiles, pairs; // query tiles and pairs of them per key head
  int splits, nk;   // splits of the key tiles, key tiles in all
  int panels, stages;
  uint32_t idesc_s, idesc_o;
  float c;          // |scale| log2 e
  float cap_in, cap2;  // 2 log2 e |scale| / cap, cap log2 e
  float* part;      // splits > 1: [splits][B Hq Sq][D] results, then [splits][B Hq Sq] lse (base 2)
  unsigned* error;
};

// Per key-tile slot: positions (per query tile, scaled by its head's slopes,
// or raw when the tile's heads differ), documents, non-finite rows of V.
struct alignas(16) Aux {
  float pos[2][3][kTile];
  int doc[kTile];
  unsigned bad[4];
};

template <class T, int AXES, bool CAP, bool PACKED>
__global__ void __launch_bounds__(kThreads, 1)
    k_attn_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
               const __grid_constant__ CUtensorMap mv, const FwdArgs f) {
  extern __shared__ char raw[];
  char* base = reinterpret_cast<char*>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
  __shared__ uint64_t bars[1 + 5 * kMaxStages + 7];
  __shared__ unsigned dead, tmem_slot;
  __shared__ uint8_t codes[kMaxCodes];
  __shared__ __align__(16) Aux aux[kMaxStages];
  const AttnArgs& a = f.a;
  const int NS = f.stages, tile_bytes = f.panels * kPanel;
  char *sq = base, *sk = sq + 2 * tile_bytes, *sv = sk + NS * tile_bytes;
  const uint32_t qfull = smem_addr(bars), kfull = qfull + 8, kempty = kfull + 8 * kMaxStages, vfull = kempty + 8 * kMaxStages,
                 vempty = vfull + 8 * kMaxStages, ready = vempty + 8 * kMaxStages, sfull = ready + 8 * kMaxStages,
                 pfull = sfull + 16, pvdone = pfull + 16, drain = pvdone + 16;
  const Guard guard{&dead, f.error};
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const int split = blockIdx.x % f.splits, rest = blockIdx.x / f.splits;
  const int bg = rest / f.pairs, b = bg / a.Hk, g = bg - b * a.Hk;
  int pair = rest - bg * f.pairs;
  if (a.causal) pair = f.pairs - 1 - pair;  // the longest rows first
  const int prefix = prefix_of(a, b);
  // head and first token of this CTA's tiles
  int head[2], i0[2], i1[2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int x = 2 * pair + t;
    if (PACKED) {
      head[t] = g * a.G + x * f.gb;
      i0[t] = 0;
      i1[t] = x < f.tiles ? a.Sq : 0;
    } else {
      head[t] = g * a.G + x % a.G;
      i0[t] = x / a.G * kTile;
      i1[t] = x < f.tiles ? min(a.Sq, i0[t] + kTile) : i0[t];
    }
  }
  const int j0 = (int)((int64_t)f.nk * split / f.splits), j1 = (int)((int64_t)f.nk * (split + 1) / f.splits);
  for (int j = j0 + threadIdx.x; j < j1; j += kThreads)
    codes[j - j0] = (uint8_t)(pair_code(a, prefix, b, i0[0], i1[0], j * kTile, (j + 1) * kTile, f.dq, f.dk) |
                              pair_code(a, prefix, b, i0[1], i1[1], j * kTile, (j + 1) * kTile, f.dq, f.dk) << 2);
  if (threadIdx.x == 0) {
    dead = 0;
    bar_init(qfull, 1);
    for (int i = 0; i < kMaxStages; ++i) {
      bar_init(kfull + 8 * i, 1);
      bar_init(kempty + 8 * i, 1);
      bar_init(vfull + 8 * i, 1);
      bar_init(vempty + 8 * i, 1);
      bar_init(ready + 8 * i, 1);
    }
    for (int t = 0; t < 2; ++t) {
      bar_init(sfull + 8 * t, 1);
      bar_init(pfull + 8 * t, 4);
      bar_init(pvdone + 8 * t, 1);
    }
    bar_init(drain, 1);
    bar_init_fence();
  }
  if (warp == 9) tmem_alloc(smem_addr(&tmem_slot), kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_slot;
  // TMEM columns: S of the two tiles, then O of the two; up to 64 channels P
  // has columns of its own, above that it takes S's place
  const bool own_p = f.panels == 1;
  const uint32_t o_cols = own_p ? 64 : 128;
  auto s_at = [&](int t) { return tmem + t * 128; };
  auto o_at = [&](int t) { return tmem + 256 + t * o_cols; };
  auto p_at = [&](int t) { return own_p ? tmem + 384 + t * 64 : tmem + t * 128; };
  const int n = j1 - j0;
  int cur = 0;
  auto next_tile = [&](int j) {  // first key tile at or after j that either query tile sees
    while (j < n && codes[j] == 0) ++j;
    return j;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 && elect_one()) {
      cur = next_tile(0);
      if (cur < n) {
        unsigned issued = 0;
        const int rows = f.rh * f.gb;
        const int valid = i1[1] > i0[1] ? 2 : 1;
        bar_expect(qfull, valid * f.panels * rows * 128);
        for (int t = 0; t < valid; ++t)
          for (int p = 0; p < f.panels; ++p)
            tma_load_4d(smem_addr(sq + t * tile_bytes + p * kPanel), &mq, p * 64, i0[t], head[t], b, qfull);
        int slot = 0;
        unsigned phase = 0;
        for (; cur < n; cur = next_tile(cur + 1)) {
          if (!bar_wait(kempty + 8 * slot, phase ^ 1u, guard)) break;
          bar_expect(kfull + 8 * slot, tile_bytes);
          for (int p = 0; p < f.panels; ++p)
            tma_load_4d(smem_addr(sk + slot * tile_bytes + p * kPanel), &mk, p * 64, (j0 + cur) * kTile, g, b, kfull + 8 * slot);
          const bool ok = bar_wait(vempty + 8 * slot, phase ^ 1u, guard);
          if (!ok) {
            bar_drain(kfull + 8 * slot, phase);
            break;
          }
          bar_expect(vfull + 8 * slot, tile_bytes);
          for (int p = 0; p < f.panels; ++p)
            tma_load_4d(smem_addr(sv + slot * tile_bytes + p * kPanel), &mv, p * 64, (j0 + cur) * kTile, g, b, vfull + 8 * slot);
          ++issued;
          if (++slot == NS) slot = 0, phase ^= 1u;
        }
        bar_drain(qfull, 0);
        for (unsigned i = issued > (unsigned)NS ? issued - NS : 0; i < issued; ++i) {
          bar_drain(kfull + 8 * (i % NS), (i / NS) & 1);
          bar_drain(vfull + 8 * (i % NS), (i / NS) & 1);
        }
      }
    } else if (warp == 9 && elect_one()) {
      const int ksteps = (a.D + 15) / 16;
      int ks = 0, vs = 0;
      unsigned kp = 0, vp = 0, done[2] = {0, 0};  // products P V issued per query tile
      auto scores = [&](int t, int slot) {
        for (int k = 0; k < ksteps; ++k) {
          const uint32_t off = (k / 4) * kPanel + (k % 4) * 32;
          mma_ss(s_at(t), smem_desc(smem_addr(sq + t * tile_bytes) + off, 16, 1024),
                 smem_desc(smem_addr(sk + slot * tile_bytes) + off, 16, 1024), f.idesc_s, k > 0);
        }
        mma_commit(sfull + 8 * t);
      };
      cur = next_tile(0);
      bool ok = cur < n && bar_wait(qfull, 0, guard) && bar_wait(kfull, 0, guard);
      if (ok) {
        fence_after();
        for (int t = 0; t < 2; ++t)
          if ((codes[cur] >> (2 * t)) & 3) scores(t, 0);
        mma_commit(kempty);
        if (++ks == NS) ks = 0, kp ^= 1u;
      }
      while (ok) {
        const int nxt = next_tile(cur + 1), code = codes[cur], ncode = nxt < n ? codes[nxt] : 0;
        if (ncode && !(ok = bar_wait(kfull + 8 * ks, kp, guard))) break;
        bool v_seen = false;
        for (int t = 0; ok && t < 2; ++t) {
          const bool now = (code >> (2 * t)) & 3, then = (ncode >> (2 * t)) & 3;
          if (now) {
            if (!(ok = bar_wait(pfull + 8 * t, done[t] & 1u, guard))) break;
            fence_after();
          }
          if (own_p && then) scores(t, ks);
          if (now) {
            if (!v_seen) {
              if (!(ok = bar_wait(ready + 8 * vs, vp, guard))) break;
              fence_after();
              v_seen = true;
            }
            for (int k = 0; k < kTile / 16; ++k)
              mma_ts(o_at(t), p_at(t) + k * 8, smem_desc(smem_addr(sv + vs * tile_bytes) + k * 2048, kPanel, 1024), f.idesc_o,
                     done[t] || k > 0);
            ++done[t];
            mma_commit(pvdone + 8 * t);
          }
          if (!own_p && then) {  // S takes P's place: after the product that reads P
            if (done[t] && !(ok = bar_wait(pvdone + 8 * t, (done[t] - 1) & 1u, guard))) break;
            scores(t, ks);
          }
        }
        if (!ok) break;
        mma_commit(vempty + 8 * vs);
        if (++vs == NS) vs = 0, vp ^= 1u;
        if (ncode) {
          mma_commit(kempty + 8 * ks);
          if (++ks == NS) ks = 0, kp ^= 1u;
        }
        cur = nxt;
        if (cur >= n) break;
      }
      mma_commit(drain);
      bar_drain(drain, 0);
    } else if (warp == 10) {
      int slot = 0;
      unsigned phase = 0;
      float slope[2][3];
      if (AXES) {
  #pragma unroll
        for (int t = 0; t < 2; ++t)
  #pragma unroll
          for (int x = 0; x < 3; ++x)
            slope[t][x] = PACKED ? 1.0f : (x < a.axes && i1[t] > i0[t] ? a.slopes[head[t] * a.axes + x] * kLog2e : 0.0f);
      }
      for (cur = next_tile(0); cur < n; cur = next_tile(cur + 1)) {
        const int code = codes[cur];
        const bool masked = (code & 3) == kMasked || (code >> 2) == kMasked;
        float pos[4][3];
        int doc[4];
  #pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = (j0 + cur) * kTile + i * 32 + lane;
          if (AXES) {
  #pragma unroll
            for (int x = 0; x < 3; ++x)
              pos[i][x] = x < a.axes && j < a.Sk ? a.pos_k[b * a.pos_k_sb + (int64_t)j * a.axes + x] : 0.0f;
          }
          doc[i] = a.doc_k && masked && j < a.Sk ? a.doc_k[b * a.doc_k_sb + j] : -1;
        }
        if (!bar_wait_warp(vfull + 8 * slot, phase, guard)) break;
        Aux& x = aux[slot];
        if (AXES) {
  #pragma unroll
          for (int i = 0; i < 4; ++i)
  #pragma unroll
            for (int c = 0; c < 3; ++c) {
              x.pos[0][c][i * 32 + lane] = pos[i][c] * slope[0][c];
              if (!PACKED) x.pos[1][c][i * 32 + lane] = pos[i][c] * slope[1][c];
            }
        }
        if (masked) {
  #pragma unroll
          for (int i = 0; i < 4; ++i) {
            x.doc[i * 32 + lane] = doc[i];
            const unsigned m = __ballot_sync(0xffffffffu, clear_bad_row<T>(sv + slot * tile_bytes, f.panels, kPanel, i * 32 + lane));
            if (lane == 0) x.bad[i] = m;
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) bar_arrive(ready + 8 * slot);
        if (++slot == NS) slot = 0, phase ^= 1u;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp / 4;
    const int r = (warp % 4) * 32 + lane;  // row of the tile, lane of TMEM
    const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;
    int i, h;
    bool valid;
    if (PACKED) {
      const int hl = r / f.rh;
      i = r - hl * f.rh;
      h = head[t] + hl;
      valid = hl < f.gb && h < (g + 1) * a.G && i < i1[t];
    } else {
      i = i0[t] + r;
      h = head[t];
      valid = i < i1[t];
    }
    if (!valid) i = i0[t], h = g * a.G;
    const int limit = key_limit(a, prefix, i);
    const int doc_q = a.doc_q && i1[t] > i0[t] ? a.doc_q[b * a.doc_q_sb + i] : 0;
    float pq[3], sl[3];
    if (AXES) {
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        sl[x] = x < a.axes && i1[t] > i0[t] ? a.slopes[h * a.axes + x] * kLog2e : 0.0f;
        pq[x] = x < a.axes && i1[t] > i0[t] ? a.pos_q[b * a.pos_q_sb + (int64_t)i * a.axes + x] : 0.0f;
        if (!PACKED) pq[x] *= sl[x];
      }
    }
    float m = -INFINITY, l = 0.0f;  // maximum (base-2 units) that P is relative to, sum of P
    unsigned sp = 0, count = 0;
    int slot = 0;
    unsigned phase = 0;
    bool ok = true;
    for (cur = next_tile(0); cur < n; cur = next_tile(cur + 1)) {
      const int code = (codes[cur] >> (2 * t)) & 3;
      if (code) {
        if (AXES || code == kMasked) {
          if (!(ok = bar_wait_warp(ready + 8 * slot, phase, guard))) break;
        }
        const Aux& x = aux[slot];
        if (!(ok = bar_wait_warp(sfull + 8 * t, sp, guard))) break;
        sp ^= 1u;
        fence_after();
        float s[kTile];
#pragma unroll
        for (int c = 0; c < kTile; c += 32) tmem_ld32(s_at(t) + lanes + c, s + c);
        tmem_wait_ld();
        if (CAP) {
          // cap tanh(y) = cap - 2 cap / (1 + e^2y): two special-function
          // operations with an error of 1e-7 cap, and right at infinities
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] = fmaf(-2.0f * f.cap2, rcp(1.0f + ex2(s[c] * f.cap_in)), f.cap2);
        } else if (AXES) {
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] *= f.c;
        }
        if (AXES) {
#pragma unroll
          for (int ax = 0; ax < 3; ++ax) {
            const float4* kp = reinterpret_cast<const float4*>(x.pos[PACKED ? 0 : t][ax]);
#pragma unroll
            for (int c = 0; c < kTile; c += 4) {
              const float4 k = kp[c / 4];
              if (PACKED) {
                s[c] = fmaf(-sl[ax], fabsf(pq[ax] - k.x), s[c]);
                s[c + 1] = fmaf(-sl[ax], fabsf(pq[ax] - k.y), s[c + 1]);
                s[c + 2] = fmaf(-sl[ax], fabsf(pq[ax] - k.z), s[c + 2]);
                s[c + 3] = fmaf(-sl[ax], fabsf(pq[ax] - k.w), s[c + 3]);
              } else {
                s[c] -= fabsf(pq[ax] - k.x);
                s[c + 1] -= fabsf(pq[ax] - k.y);
                s[c + 2] -= fabsf(pq[ax] - k.z);
                s[c + 3] -= fabsf(pq[ax] - k.w);
              }
            }
          }
        }
        const float c2 = CAP || AXES ? 1.0f : f.c;
        if (code == kMasked) {
          const int left = limit - (j0 + cur) * kTile;  // keys of this tile before the limit
#pragma unroll
          for (int c = 0; c < kTile; ++c) s[c] = c < left ? s[c] : -INFINITY;
          if (a.doc_q) {
            const int4* kd = reinterpret_cast<const int4*>(x.doc);
#pragma unroll
            for (int c = 0; c < kTile; c += 4) {
              const int4 d = kd[c / 4];
              s[c] = d.x == doc_q && doc_q >= 0 ? s[c] : -INFINITY;
              s[c + 1] = d.y == doc_q && doc_q >= 0 ? s[c + 1] : -INFINITY;
              s[c + 2] = d.z == doc_q && doc_q >= 0 ? s[c + 2] : -INFINITY;
              s[c + 3] = d.w == doc_q && doc_q >= 0 ? s[c + 3] : -INFINITY;
            }
          }
          if (x.bad[0] | x.bad[1] | x.bad[2] | x.bad[3]) {  // a visible non-finite value makes the row NaN
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if ((x.bad[c / 32] >> (c % 32)) & 1u) s[c] = s[c] == -INFINITY ? s[c] : NAN;
          }
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int c = 4; c < kTile; ++c) mx[c % 4] = fmaxf(mx[c % 4], s[c]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
        // own columns for P, or a rescaling of O: the last product must be done
        const bool grow = top > m + kRescale || (m == -INFINITY && top > m);
        const bool rescale = __any_sync(0xffffffffu, grow);
        if (count && (own_p || rescale)) {
          if (!(ok = bar_wait_warp(pvdone + 8 * t, (count - 1) & 1u, guard))) break;
          fence_after();
        }
        if (rescale) {
          const float mn = grow ? top : m, w = grow ? ex2(m - mn) : 1.0f;  // 2^-inf = 0: no row before
          m = mn;
          l *= w;
          if (count) {
            for (int c = 0; c < a.D; c += 32) {
              float o[32];
              tmem_ld32(o_at(t) + lanes + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= w;
              tmem_st32(o_at(t) + lanes + c, o);
            }
          }
        }
        const float mm = m == -INFINITY ? 0.0f : m;
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kTile; c += 32) {
          uint32_t u[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = ex2(fmaf(s[c + e], c2, -mm)), p1 = ex2(fmaf(s[c + e + 1], c2, -mm));
            sum[e % 4] += p0;
            sum[e % 4 + 1] += p1;
            u[e / 2] = pack2<T>(p0, p1);
          }
          tmem_st16(p_at(t) + lanes + c / 2, u);
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(pfull + 8 * t);
        ++count;
      }
      if (++slot == NS) slot = 0, phase ^= 1u;
    }
    // results: o = O / l, lse; of a split, both in 32 bits to the workspace
    if (ok && count) ok = bar_wait_warp(pvdone + 8 * t, (count - 1) & 1u, guard);
    fence_after();
    if (i1[t] > i0[t]) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l, lse2 = l == 0.0f ? -INFINITY : m + log2f(l);
      const int64_t row = ((int64_t)b * a.Hq + h) * a.Sq + i, rows = (int64_t)a.B * a.Hq * a.Sq;
      if (valid) {
        if (f.splits > 1)
          f.part[rows * a.D * f.splits + split * rows + row] = lse2;
        else if (a.lse)
          a.lse[row] = lse2 * kLn2;
      }
      for (int c = 0; c < a.D; c += 32) {
        float o[32];
        if (ok && count) {
          tmem_ld32(o_at(t) + lanes + c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0.0f : o[e] * inv;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          if (!valid || c + e >= a.D) continue;
          if (f.splits > 1) {
            float* p = f.part + (split * rows + row) * a.D + c + e;
            *reinterpret_cast<float4*>(p) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            *reinterpret_cast<float4*>(p + 4) = make_float4(o[e + 4], o[e + 5], o[e + 6], o[e + 7]);
          } else {
            T* p = static_cast<T*>(a.o.p) + b * a.o.sb + (int64_t)i * a.o.st + h * a.o.sh + c + e;
            *reinterpret_cast<uint4*>(p) = make_uint4(pack2<T>(o[e], o[e + 1]), pack2<T>(o[e + 2], o[e + 3]),
                                                      pack2<T>(o[e + 4], o[e + 5]), pack2<T>(o[e + 6], o[e + 7]));
          }
        }
        __syncwarp();
      }
    }
  }
  fence_before();
  __syncwarp();
  __syncthreads();
  fence_after();
  if (warp == 9) tmem_free(tmem, kTmemCols);
}

// Joins the splits of a row: o = sum 2^(lse_s - lse) o_s.  One warp per row.
template <class T>
__global__ void __launch_bounds__(256) k_attn_join(const FwdArgs f) {
  const AttnArgs& a = f.a;
  const int64_t rows = (int64_t)a.B * a.Hq * a.Sq, row = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (row >= rows) return;
  const int lane = threadIdx.x % 32;
  const float* ls = f.part + rows * a.D * f.splits;
  float top = -INFINITY;
  for (int s = lane; s < f.splits; s += 32) {
    const float v = ls[s * rows + row];
    top = v > top || v != v ? v : top;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float v = __shfl_xor_sync(0xffffffffu, top, o);
    top = v > top || v != v ? v : top;
  }
  const float ref = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, acc[4] = {};
  for (int s = 0; s < f.splits; ++s) {
    const float w = ex2(ls[s * rows + row] - ref);
    sum += w;
    if (4 * lane < a.D) {
      const float4 o = *reinterpret_cast<const float4*>(f.part + (s * rows + row) * a.D + 4 * lane);
      acc[0] = fmaf(w, o.x, acc[0]);
      acc[1] = fmaf(w, o.y, acc[1]);
      acc[2] = fmaf(w, o.z, acc[2]);
      acc[3] = fmaf(w, o.w, acc[3]);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int i = (int)(row % a.Sq), h = (int)(row / a.Sq % a.Hq), b = (int)(row / a.Sq / a.Hq);
  if (4 * lane < a.D) {
    T* p = static_cast<T*>(a.o.p) + b * a.o.sb + (int64_t)i * a.o.st + h * a.o.sh + 4 * lane;
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv));
  }
  if (a.lse && lane == 0) a.lse[row] = (top == -INFINITY ? top : ref + log2f(sum)) * kLn2;
}

// One warp per tile of one sequence, queries' tiles first.
__global__ void __launch_bounds__(256) k_doc_ranges(const AttnArgs a, DocRange* dq, DocRange* dk) {
  const int nq = (a.Sq + kTile - 1) / kTile, nk = (a.Sk + kTile - 1) / kTile;
  const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  if (w >= (int64_t)a.B * (nq + nk)) return;
  const int b = (int)(w / (nq + nk)), x = (int)(w % (nq + nk)), lane = threadIdx.x % 32;
  const bool q = x < nq;
  const int tile = q ? x : x - nq, len = q ? a.Sq : a.Sk;
  const int* d = q ? a.doc_q + b * a.doc_q_sb : a.doc_k + b * a.doc_k_sb;
  int lo = INT32_MAX, hi = -1, pad = 0;
  for (int i = tile * kTile + lane; i < min(len, (tile + 1) * kTile); i += 32) {
    const int v = d[i];
    if (v < 0) {
      pad = 1;
    } else {
      lo = min(lo, v);
      hi = max(hi, v);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  pad = __any_sync(0xffffffffu, pad);
  if (lane == 0) (q ? dq + (int64_t)b * nq : dk + (int64_t)b * nk)[tile] = DocRange{lo, hi, pad, 0};
}

template <class T, int AXES, bool CAP, bool PACKED>
cudaError_t run(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FwdArgs& f, cudaStream_t s) {
  static std::atomic<unsigned long long> granted{0};
  const size_t smem = 1024 + (size_t)(2 + 2 * f.stages) * f.panels * kPanel;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(granted.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_attn_fwd<T, AXES, CAP, PACKED>, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + 12 * kPanel);
    if (e != cudaSuccess) return e;
    granted.fetch_or(bit, std::memory_order_relaxed);
  }
  const unsigned grid = (unsigned)((int64_t)f.a.B * f.a.Hk * f.pairs * f.splits);
  note_launch_begin("k_attn_fwd", s);
  k_attn_fwd<T, AXES, CAP, PACKED><<<grid, kThreads, smem, s>>>(mq, mk, mv, f);
  note_launch_end(s);
  if (f.splits > 1) {
    const int64_t rows = (int64_t)f.a.B * f.a.Hq * f.a.Sq;
    note_launch_begin("k_attn_join", s);
    k_attn_join<T><<<(unsigned)((rows + 7) / 8), 256, 0, s>>>(f);
    note_launch_end(s);
  }
  return cudaGetLastError();
}

template <class T>
cudaError_t pick(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const FwdArgs& f, cudaStream_t s) {
  const bool cap = f.a.cap > 0.0f;
  if (f.packed) {
    if (f.a.axes) return cap ? run<T, 3, true, true>(mq, mk, mv, f, s) : run<T, 3, false, true>(mq, mk, mv, f, s);
    return cap ? run<T, 0, true, true>(mq, mk, mv, f, s) : run<T, 0, false, true>(mq, mk, mv, f, s);
  }
  if (f.a.axes) return cap ? run<T, 3, true, false>(mq, mk, mv, f, s) : run<T, 3, false, false>(mq, mk, mv, f, s);
  return cap ? run<T, 0, true, false>(mq, mk, mv, f, s) : run<T, 0, false, false>(mq, mk, mv, f, s);
}

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace

cudaError_t launch_doc_ranges(const AttnArgs& a, DocRange* dq, DocRange* dk, cudaStream_t s) {
  const int64_t w = (int64_t)a.B * ((a.Sq + kTile - 1) / kTile + (a.Sk + kTile - 1) / kTile);
  if (w == 0) return cudaSuccess;
  note_launch_begin("k_doc_ranges", s);
  k_doc_ranges<<<(unsigned)((w + 7) / 8), 256, 0, s>>>(a, dq, dk);
  note_launch_end(s);
  return cudaGetLastError();
}

// Rows of a query tile, and how the key tiles are split: a call whose tiles
// leave SMs idle splits its keys over them, at least two key tiles each.
AttnPlan attention_plan(const AttnArgs& a, int sms) {
  AttnPlan p{};
  p.nq = (a.Sq + kTile - 1) / kTile;
  p.nk = (a.Sk + kTile - 1) / kTile;
  p.packed = a.Sq > 0 && a.Sq <= kTile / 2 && a.G > 1;
  if (p.packed) {
    p.rh = a.Sq;
    p.gb = kTile / a.Sq < a.G ? kTile / a.Sq : a.G;
    p.tiles = (a.G + p.gb - 1) / p.gb;
  } else {
    p.rh = a.Sq < kTile ? (a.Sq > 0 ? a.Sq : 1) : kTile;
    p.gb = 1;
    p.tiles = p.nq * a.G;
  }
  p.pairs = (p.tiles + 1) / 2;
  const int64_t ctas = (int64_t)a.B * a.Hk * p.pairs;
  int64_t s = ctas > 0 && 2 * ctas <= sms ? sms / ctas : 1;
  if (s > p.nk / 2) s = p.nk / 2;
  const int64_t least = (p.nk + kMaxCodes - 1) / kMaxCodes;
  if (s < least) s = least;
  p.splits = (int)(s < 1 ? 1 : s);
  const int64_t rows = (int64_t)a.B * a.Hq * a.Sq;
  p.ranges_bytes = round256((size_t)a.B * p.nq * sizeof(DocRange)) + round256((size_t)a.B * p.nk * sizeof(DocRange));
  p.part_bytes = p.splits > 1 ? round256((size_t)rows * p.splits * (a.D + 1) * 4) : 0;
  return p;
}

cudaError_t launch_attention_fwd(int dt, const AttnArgs& a, int sms, void* ws, cudaStream_t s) {
  const AttnPlan p = attention_plan(a, sms);
  FwdArgs f{};
  f.a = a;
  char* w = static_cast<char*>(ws);
  DocRange* dq = reinterpret_cast<DocRange*>(w);
  DocRange* dk = reinterpret_cast<DocRange*>(w + round256((size_t)a.B * p.nq * sizeof(DocRange)));
  f.part = reinterpret_cast<float*>(w + p.ranges_bytes);
  if (a.doc_q) {
    f.dq = dq;
    f.dk = dk;
    const cudaError_t e = launch_doc_ranges(a, dq, dk, s);
    if (e != cudaSuccess) return e;
  }
  f.packed = p.packed;
  f.rh = p.rh;
  f.gb = p.gb;
  f.tiles = p.tiles;
  f.pairs = p.pairs;
  f.splits = p.splits;
  f.nk = p.nk;
  f.panels = (a.D + 63) / 64;
  f.stages = f.panels == 1 ? 4 : 2;
  f.idesc_s = tc::mma_idesc(dt == 2, false, false, kTile, kTile) | (a.scale < 0.0f ? 1u << 13 : 0u);  // negate A
  f.idesc_o = tc::mma_idesc(dt == 2, false, true, kTile, (a.D + 15) / 16 * 16);
  f.c = fabsf(a.scale) * kLog2e;
  if (a.cap > 0.0f) {
    f.cap_in = 2.0f * kLog2e * fabsf(a.scale) / a.cap;
    f.cap2 = a.cap * kLog2e;
  }
  cudaError_t e = device_error_word(&f.error);
  CUtensorMap mq, mk, mv;
  if (e == cudaSuccess) e = heads_map(&mq, dt, a.q, a.B, a.Sq, a.Hq, a.D, p.rh, p.gb);
  // without keys no tile is loaded: any valid address serves the maps
  HeadsView k = a.k, v = a.v;
  if (a.Sk == 0) k = v = a.q;
  if (e == cudaSuccess) e = heads_map(&mk, dt, k, a.B, a.Sk, a.Hk, a.D, kTile, 1);
  if (e == cudaSuccess) e = heads_map(&mv, dt, v, a.B, a.Sk, a.Hk, a.D, kTile, 1);
  if (e != cudaSuccess) return e;
  FFDP_TOK_SWITCH16(dt, T, { return pick<T>(mq, mk, mv, f, s); });
}

}  // namespace ffdp
