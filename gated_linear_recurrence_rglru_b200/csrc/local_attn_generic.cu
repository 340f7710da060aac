// Windowed attention with sinks on CUDA cores, forward and backward
// (include/rglru_attn.h), for fp32 and for bf16 heads other than 64, 128 or 256
// wide; and the kernels that every backward shares (the rows' dot products of
// dout and out, the join of partial key gradients).
//
//   forward    S = scale Q K^T, running max m and sum l, O = O 2^(m - m') + P V
//   backward   P = exp(S - lse), dP = dO V^T, dS = P (dP - delta),
//              delta = rowsum(dO * O); dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO
//
// Bound by the CUDA cores' fp32 rate. Tiles of BT queries by BT keys (64, or, in
// the backward of heads over 128 wide, whose four operand tiles fill shared memory,
// 48) in float in shared memory; 16 x 16 threads, each BT/16 rows by BT/16 columns of
// S and BT/16 rows by dh/16 columns of a product, from 16-byte shared loads.
// Rows of shared memory are padded by 16 bytes, so the 8 rows that a quarter
// warp reads fall into different banks. Tiles outside the mask are skipped.
// Hidden keys get weight zero by selection, never by arithmetic on what lies
// there, and rows past a sequence are read as zeros.
#include "attn_cluster.cuh"
#include "attn_kernels.h"
#include "attn_mask.cuh"
#include "common.cuh"

namespace rglru {
namespace {

constexpr int kThreads = 256;

// Rows r0 .. r0+BT-1 of one head (row stride st) to dst[BT][pitch]; rows before
// first, at or past n, and columns dh .. 64*NC-1, as zeros.
template <typename T, int BT, int NC>
__device__ __forceinline__ void fill(float *dst, const T *src, long long st, int r0, int n, int dh, int first = 0) {
  constexpr int W = NC * 64, kPitch = W + 4, kV = W / 4;
  for (int i = threadIdx.x; i < BT * kV; i += kThreads) {
    const int r = i / kV, c = (i % kV) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r >= first && r0 + r < n && c < dh) {
      const T *s = src + (r0 + r) * st + c;
      if constexpr (sizeof(T) == 4) {
        v = __ldg(reinterpret_cast<const float4 *>(s));
      } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(s));
        v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                        __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
      }
    }
    *reinterpret_cast<float4 *>(dst + r * kPitch + c) = v;
  }
}

// The same ahead of use: fp32 rows by cp.async, in flight until fill_wait.
template <typename T, int BT, int NC>
__device__ __forceinline__ void fill_ahead(float *dst, const T *src, long long st, int r0, int n, int dh) {
  if constexpr (sizeof(T) == 4) {
    constexpr int W = NC * 64, kPitch = W + 4, kV = W / 4;
    for (int i = threadIdx.x; i < BT * kV; i += kThreads) {
      const int r = i / kV, c = (i % kV) * 4;
      const bool in = r0 + r < n && c < dh;
      const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst + r * kPitch + c));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d),
                   "l"(in ? src + (r0 + r) * st + c : src), "r"(in ? 16 : 0)
                   : "memory");
    }
  } else {
    fill<T, BT, NC>(dst, src, st, r0, n, dh);
  }
}
__device__ __forceinline__ void fill_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void fill_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// acc[i][j] = sum_d a[ty + 16 i][d] b[tx + 16 j][d]
template <int N, int NC>
__device__ __forceinline__ void dot_rows(float (&acc)[N][N], const float *a, const float *b, int tx,
                                         int ty) {
  constexpr int kPitch = NC * 64 + 4;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < N; ++j) acc[i][j] = 0.0f;
#pragma unroll 4
  for (int d = 0; d < NC * 64; d += 4) {
    float4 av[N], bv[N];
#pragma unroll
    for (int i = 0; i < N; ++i) av[i] = *reinterpret_cast<const float4 *>(a + (ty + 16 * i) * kPitch + d);
#pragma unroll
    for (int j = 0; j < N; ++j) bv[j] = *reinterpret_cast<const float4 *>(b + (tx + 16 * j) * kPitch + d);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        acc[i][j] = fmaf(av[i].x, bv[j].x, acc[i][j]);
        acc[i][j] = fmaf(av[i].y, bv[j].y, acc[i][j]);
        acc[i][j] = fmaf(av[i].z, bv[j].z, acc[i][j]);
        acc[i][j] = fmaf(av[i].w, bv[j].w, acc[i][j]);
      }
  }
}

// The rows of a thread's part of a product whose weights are stored key-major: four
// together where it has four, for one load.
template <int N> __device__ __forceinline__ int part_row(int ty, int i) { return N == 4 ? ty * 4 + i : ty + 16 * i; }

// o[i][c] += sum_k w[k][row i] v[k][4 tx + 64 c ..]: weights stored key-major
// (wt[k][row], pitch BT + 4; rows of part_row) or row-major (w[row][k]; rows ty + 16 i).
template <int BT, int NC, bool kTransposed>
__device__ __forceinline__ void add_product(float4 (&o)[BT / 16][NC], const float *w, const float *v,
                                            int tx, int ty) {
  constexpr int kPitch = NC * 64 + 4, kWp = BT + 4, N = BT / 16;
#pragma unroll 2
  for (int k = 0; k < BT; k += 4) {
    float wv[N][4];
    if constexpr (kTransposed && N == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 x = *reinterpret_cast<const float4 *>(w + (k + e) * kWp + ty * 4);
        wv[0][e] = x.x;
        wv[1][e] = x.y;
        wv[2][e] = x.z;
        wv[3][e] = x.w;
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (kTransposed) {
        if (N == 4) break;
#pragma unroll
        for (int e = 0; e < 4; ++e) wv[i][e] = w[(k + e) * kWp + ty + 16 * i];
      } else {
        const float4 x = *reinterpret_cast<const float4 *>(w + (ty + 16 * i) * kWp + k);
        wv[i][0] = x.x;
        wv[i][1] = x.y;
        wv[i][2] = x.z;
        wv[i][3] = x.w;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 x = *reinterpret_cast<const float4 *>(v + (k + e) * kPitch + tx * 4 + c * 64);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          o[i][c].x = fmaf(wv[i][e], x.x, o[i][c].x);
          o[i][c].y = fmaf(wv[i][e], x.y, o[i][c].y);
          o[i][c].z = fmaf(wv[i][e], x.z, o[i][c].z);
          o[i][c].w = fmaf(wv[i][e], x.w, o[i][c].w);
        }
      }
  }
}

template <typename T> __device__ __forceinline__ void store4(T *p, float4 v, float f);
template <> __device__ __forceinline__ void store4<float>(float *p, float4 v, float f) {
  *reinterpret_cast<float4 *>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
template <> __device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16 *p, float4 v, float f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z * f, v.w * f);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                             *reinterpret_cast<const uint32_t *>(&b));
}

template <typename T>
__device__ __forceinline__ const T *head_of(const Strided &x, int b, int h) {
  return static_cast<const T *>(x.p) + b * x.sb + h * x.sh;
}

// max / sum over the 16 threads tx of a row
__device__ __forceinline__ float row_max16(float v) {
#pragma unroll
  for (int x = 8; x > 0; x >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, x));
  return v;
}
__device__ __forceinline__ float row_sum16(float v) {
#pragma unroll
  for (int x = 8; x > 0; x >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, x);
  return v;
}

template <int BT, int NC> constexpr int fwd_smem() {
  return (5 * BT * (NC * 64 + 4) + BT * (BT + 4)) * 4;
}
template <int BT, int NC> constexpr int bwd_smem() {
  return (4 * BT * (NC * 64 + 4) + 2 * BT * (BT + 4) + 2 * BT) * 4;
}

// kSplit: the blocks of a cluster of `blocks` share a query tile's keys.
template <typename T, int BT, int NC, bool kSplit>
__global__ void __launch_bounds__(kThreads) attn_fwd_generic_kernel(const AttnArgs p, const int blocks) {
  extern __shared__ __align__(16) float smf[];
  constexpr int kPitch = NC * 64 + 4, N = BT / 16, kWp = BT + 4;
  float *qs = smf, *kvs = qs + BT * kPitch, *ps = kvs + 4 * BT * kPitch;   // K and V: two buffers
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int parts = kSplit ? blocks : 1;
  const int part = blockIdx.x % parts, row = blockIdx.x / parts, h = row % p.Hq, b = row / p.Hq;
  // the last queries first: they see the most keys
  const int q0 = (gridDim.y - 1 - blockIdx.y) * BT, off = p.S - p.T;
  const RowLens n = row_lens(p, b);
  if (q0 >= n.nq) return;
  const int kvh = h / (p.Hq / p.Hkv);
  const T *qp = head_of<T>(p.q, b, h), *kp = head_of<T>(p.k, b, kvh), *vp = head_of<T>(p.v, b, kvh);
  fill<T, BT, NC>(qs, qp, p.q.st, q0, n.nq, p.dh);
  const int qe = min(q0 + BT, n.nq) - 1;
  const KeyTiles kt = key_tiles(q0 + off, qe + off, n.nk, p.window, p.sinks, BT);
  float4 o[N][NC];
  float m[N], l[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  // positions of the tile's queries bound which keys any of them sees
  const int seen_lo = p.window > 0 ? q0 + off - p.window + 1 : 0, seen_hi = qe + off;
  const int x0 = kt.n * part / parts, x1 = kt.n * (part + 1) / parts;   // this block's tiles
  auto ahead = [&](int x) {
    if (x < x1) {
      float *d = kvs + (x & 1) * 2 * BT * kPitch;
      fill_ahead<T, BT, NC>(d, kp, p.k.st, kt.tile(x) * BT, n.nk, p.dh);
      fill_ahead<T, BT, NC>(d + BT * kPitch, vp, p.v.st, kt.tile(x) * BT, n.nk, p.dh);
    }
    fill_commit();
  };
  ahead(x0);
  for (int x = x0; x < x1; ++x) {
    const int k0 = kt.tile(x) * BT;
    float *ks = kvs + (x & 1) * 2 * BT * kPitch, *vs = ks + BT * kPitch;
    ahead(x + 1);
    fill_wait<1>();
    __syncthreads();
    // value rows that no query here sees count as zeros, whatever they hold
    for (int i = threadIdx.x; i < BT * NC * 16; i += kThreads) {
      const int r = i / (NC * 16), j = k0 + r;
      if (j > seen_hi || (j < seen_lo && j >= p.sinks))
        *reinterpret_cast<float4 *>(vs + r * kPitch + (i % (NC * 16)) * 4) =
            make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float s[N][N];
    dot_rows<N, NC>(s, qs, ks, tx, ty);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int pos = q0 + ty + 16 * i + off;
      float mx = -INFINITY;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const int key = k0 + tx + 16 * j;
        s[i][j] = key < n.nk && attn_visible(key, pos, p.window, p.sinks) ? s[i][j] * p.scale
                                                                           : -INFINITY;
        mx = fmaxf(mx, s[i][j]);
      }
      const float mn = fmaxf(m[i], row_max16(mx));
      const float f = m[i] == -INFINITY ? 0.0f : expf(m[i] - mn);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float w = s[i][j] == -INFINITY ? 0.0f : expf(s[i][j] - mn);   // (NaN stays NaN)
        sum += w;
        ps[(ty + 16 * i) * kWp + tx + 16 * j] = w;
      }
      l[i] = l[i] * f + row_sum16(sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        o[i][c].x *= f;
        o[i][c].y *= f;
        o[i][c].z *= f;
        o[i][c].w *= f;
      }
    }
    __syncthreads();
    add_product<BT, NC, false>(o, ps, vs, tx, ty);
    __syncthreads();                               // the buffer may be filled again
  }
  fill_wait<0>();
  if constexpr (kSplit) {
    // O (not divided yet), m and l to shared memory, where Q was, for the cluster's
    // blocks; each joins its share of the rows
    const int share = BT / parts, r0 = part * share;
    float *ml = kvs, *fs = ml + 2 * BT;
    if (x0 == x1) __syncthreads();                       // (Q was filled, not used)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = ty + 16 * i;
#pragma unroll
      for (int c = 0; c < NC; ++c) *reinterpret_cast<float4 *>(qs + r * kPitch + tx * 4 + c * 64) = o[i][c];
      if (tx == 0) *reinterpret_cast<float2 *>(ml + 2 * r) = make_float2(m[i], l[i]);
    }
    tc::cluster_sync();
    const uint32_t o_at = tc::smem_u32(qs), ml_at = tc::smem_u32(ml);
    for (int r = threadIdx.x; r < share; r += kThreads) {
      const int t = q0 + r0 + r;
      float f[8], top, sum;
      join_factors<false>(ml_at + 2 * (r0 + r) * 4, parts, f, top, sum);
#pragma unroll
      for (int i = 0; i < 8; ++i) fs[r * 8 + i] = f[i];
      if (t < n.nq && p.lse != nullptr)
        p.lse[(static_cast<long long>(b) * p.Hq + h) * p.T + t] = sum == 0.0f ? -INFINITY : top + logf(sum);
    }
    __syncthreads();
    for (int z = threadIdx.x; z < share * NC * 16; z += kThreads) {
      const int r = z / (NC * 16), c = z % (NC * 16) * 4, t = q0 + r0 + r;
      if (t >= n.nq || c >= p.dh) continue;
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const float f = fs[r * 8 + i];
        const float4 x = ld_cluster4(tc::mapa_shared(o_at + ((r0 + r) * kPitch + c) * 4, i));
        if (f != 0.0f) a = make_float4(fmaf(x.x, f, a.x), fmaf(x.y, f, a.y), fmaf(x.z, f, a.z), fmaf(x.w, f, a.w));
      }
      store4<T>(static_cast<T *>(p.out) + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * p.dh + c, a, 1.0f);
    }
    tc::cluster_sync();                                  // the others have read this block's part
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = q0 + ty + 16 * i;
      if (t >= n.nq) continue;
      const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
      T *dst = static_cast<T *>(p.out) + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * p.dh;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (tx * 4 + c * 64 < p.dh) store4<T>(dst + tx * 4 + c * 64, o[i][c], inv);
      if (p.lse != nullptr && tx == 0)
        p.lse[(static_cast<long long>(b) * p.Hq + h) * p.T + t] =
            l[i] == 0.0f ? -INFINITY : m[i] + logf(l[i]);
    }
  }
}

// The weights and score gradients of one tile pair, from the four operand tiles:
// thread (ty, tx) holds rows ty + 16 i (queries) and columns tx + 16 j (keys).
template <int BT, int NC>
__device__ __forceinline__ void tile_grads(const AttnArgs &p, const float *qs, const float *dos,
                                           const float *ks, const float *vs, const float *lses,
                                           const float *deltas, int q0, int k0, int off, RowLens n,
                                           float (&w)[BT / 16][BT / 16], float (&ds)[BT / 16][BT / 16],
                                           int tx, int ty) {
  constexpr int N = BT / 16;
  dot_rows<N, NC>(w, qs, ks, tx, ty);
  dot_rows<N, NC>(ds, dos, vs, tx, ty);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = ty + 16 * i, t = q0 + r;
    const float lse = lses[r], dl = deltas[r];
    const bool lone = attn_lone(t + off, p.window, p.sinks);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int key = k0 + tx + 16 * j;
      const bool ok = t < n.nq && key < n.nk && attn_visible(key, t + off, p.window, p.sinks);
      w[i][j] = ok ? expf(w[i][j] * p.scale - lse) : 0.0f;
      ds[i][j] = ok && !lone ? w[i][j] * (ds[i][j] - dl) * p.scale : 0.0f;
    }
  }
}

// dQ: a block takes BT queries of one head and walks the keys they see.
template <typename T, int BT, int NC, bool kSplit>
__global__ void __launch_bounds__(kThreads)
attn_dq_generic_kernel(const AttnArgs p, const float *delta, const int blocks) {
  extern __shared__ __align__(16) float smf[];
  constexpr int kPitch = NC * 64 + 4, N = BT / 16, kWp = BT + 4;
  float *qs = smf, *dos = qs + BT * kPitch, *ks = dos + BT * kPitch, *vs = ks + BT * kPitch;
  float *dss = vs + BT * kPitch, *lses = dss + 2 * BT * kWp, *deltas = lses + BT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int parts = kSplit ? blocks : 1;
  const int part = blockIdx.x % parts, row = blockIdx.x / parts, h = row % p.Hq, b = row / p.Hq;
  const int q0 = (gridDim.y - 1 - blockIdx.y) * BT, off = p.S - p.T;
  const RowLens n = row_lens(p, b);
  if (q0 >= n.nq) return;
  const int kvh = h / (p.Hq / p.Hkv);
  const T *kp = head_of<T>(p.k, b, kvh), *vp = head_of<T>(p.v, b, kvh);
  const long long dst_row = static_cast<long long>(p.Hq) * p.dh;
  const T *dop = static_cast<const T *>(p.dout) + (static_cast<long long>(b) * p.T * p.Hq + h) * p.dh;
  fill<T, BT, NC>(qs, head_of<T>(p.q, b, h), p.q.st, q0, n.nq, p.dh);
  fill<T, BT, NC>(dos, dop, dst_row, q0, n.nq, p.dh);
  const long long srow = (static_cast<long long>(b) * p.Hq + h) * p.T;
  for (int i = threadIdx.x; i < BT; i += kThreads) {
    lses[i] = q0 + i < n.nq ? p.lse[srow + q0 + i] : 0.0f;
    deltas[i] = q0 + i < n.nq ? delta[srow + q0 + i] : 0.0f;
  }
  const int qe = min(q0 + BT, n.nq) - 1;
  const KeyTiles kt = key_tiles(q0 + off, qe + off, n.nk, p.window, p.sinks, BT);
  const int seen_lo = p.window > 0 ? q0 + off - p.window + 1 : 0, seen_hi = qe + off;
  float4 o[N][NC];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int x1 = kt.n * (part + 1) / parts;                  // this block's tiles
  for (int x = kt.n * part / parts; x < x1; ++x) {
    const int k0 = kt.tile(x) * BT;
    __syncthreads();
    fill<T, BT, NC>(ks, kp, p.k.st, k0, n.nk, p.dh);
    fill<T, BT, NC>(vs, vp, p.v.st, k0, n.nk, p.dh);
    __syncthreads();
    float w[N][N], ds[N][N];
    tile_grads<BT, NC>(p, qs, dos, ks, vs, lses, deltas, q0, k0, off, n, w, ds, tx, ty);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) dss[(ty + 16 * i) * kWp + tx + 16 * j] = ds[i][j];
    __syncthreads();
    // key rows that no query here sees count as zeros in the product
    for (int i = threadIdx.x; i < BT * NC * 16; i += kThreads) {
      const int r = i / (NC * 16), j = k0 + r;
      if (j > seen_hi || (j < seen_lo && j >= p.sinks))
        *reinterpret_cast<float4 *>(ks + r * kPitch + (i % (NC * 16)) * 4) =
            make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    add_product<BT, NC, false>(o, dss, ks, tx, ty);
  }
  if constexpr (kSplit) {
    // each block of the cluster adds its share of the rows up, in the order of the parts
    const int share = BT / parts, r0 = part * share;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int c = 0; c < NC; ++c)
        *reinterpret_cast<float4 *>(qs + (ty + 16 * i) * kPitch + tx * 4 + c * 64) = o[i][c];
    tc::cluster_sync();
    const uint32_t at = tc::smem_u32(qs);
    for (int z = threadIdx.x; z < share * NC * 16; z += kThreads) {
      const int r = z / (NC * 16), c = z % (NC * 16) * 4, t = q0 + r0 + r;
      if (t >= n.nq || c >= p.dh) continue;
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
      for (int i = 0; i < parts; ++i) {
        const float4 x = ld_cluster4(tc::mapa_shared(at + ((r0 + r) * kPitch + c) * 4, i));
        a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
      }
      store4<T>(static_cast<T *>(p.dq) + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * p.dh + c, a, 1.0f);
    }
    tc::cluster_sync();                                  // the others have read this block's part
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = q0 + ty + 16 * i;
      if (t >= n.nq) continue;
      T *dst = static_cast<T *>(p.dq) + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * p.dh;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (tx * 4 + c * 64 < p.dh) store4<T>(dst + tx * 4 + c * 64, o[i][c], 1.0f);
    }
  }
}

// dK and dV: a block takes one piece of a tile of BT keys (PiecePlan).
template <typename T, int BT, int NC>
__global__ void __launch_bounds__(kThreads)
attn_dkv_generic_kernel(const AttnArgs p, const float *delta, const PiecePlan pl, float *parts) {
  extern __shared__ __align__(16) float smf[];
  constexpr int kPitch = NC * 64 + 4, N = BT / 16, kWp = BT + 4;
  float *qs = smf, *dos = qs + BT * kPitch, *ks = dos + BT * kPitch, *vs = ks + BT * kPitch;
  float *ws = vs + BT * kPitch, *dss = ws + BT * kWp, *lses = dss + BT * kWp, *deltas = lses + BT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int kvh = blockIdx.y % p.Hkv, b = blockIdx.y / p.Hkv;
  const PieceAt at = piece_at(pl, blockIdx.x);
  const int k0 = at.tile * BT, off = p.S - p.T, G = p.Hq / p.Hkv;
  const RowLens n = row_lens(p, b);
  if (k0 >= n.nk) return;
  const Steps st = steps_of(query_range(k0, BT, n.nq, n.nk, off, p.window, p.sinks), BT, G);
  const Piece pc = piece_of(pl, st.n, at.piece);
  const int first = pc.first, last = pc.last;
  if (first >= last && at.piece > 0) return;
  fill<T, BT, NC>(ks, head_of<T>(p.k, b, kvh), p.k.st, k0, n.nk, p.dh);
  fill<T, BT, NC>(vs, head_of<T>(p.v, b, kvh), p.v.st, k0, n.nk, p.dh);
  float4 dk[N][NC], dv[N][NC];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int c = 0; c < NC; ++c) dk[i][c] = dv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int x = first; x < last; ++x) {
    const int h = kvh * G + x / st.nq, q0 = (st.q0 + x % st.nq) * BT;
    const T *dop = static_cast<const T *>(p.dout) + (static_cast<long long>(b) * p.T * p.Hq + h) * p.dh;
    const long long srow = (static_cast<long long>(b) * p.Hq + h) * p.T;
    __syncthreads();
    // (queries before -off see no key: their rows count as zeros, whatever they hold)
    fill<T, BT, NC>(qs, head_of<T>(p.q, b, h), p.q.st, q0, n.nq, p.dh, -off);
    fill<T, BT, NC>(dos, dop, static_cast<long long>(p.Hq) * p.dh, q0, n.nq, p.dh, -off);
    for (int i = threadIdx.x; i < BT; i += kThreads) {
      lses[i] = q0 + i < n.nq ? p.lse[srow + q0 + i] : 0.0f;
      deltas[i] = q0 + i < n.nq ? delta[srow + q0 + i] : 0.0f;
    }
    __syncthreads();
    float w[N][N], ds[N][N];
    tile_grads<BT, NC>(p, qs, dos, ks, vs, lses, deltas, q0, k0, off, n, w, ds, tx, ty);
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < N; ++j) {
        ws[(ty + 16 * i) * kWp + tx + 16 * j] = w[i][j];
        dss[(ty + 16 * i) * kWp + tx + 16 * j] = ds[i][j];
      }
    __syncthreads();
    add_product<BT, NC, true>(dv, ws, dos, tx, ty);
    add_product<BT, NC, true>(dk, dss, qs, tx, ty);
  }
  const bool whole = st.n <= pl.len;               // the tile's only piece
  const size_t slot = (static_cast<size_t>(blockIdx.y) * pl.slots + first_slot(pl, at.tile) + at.piece) *
                      2 * BT * p.dh;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int r = part_row<N>(ty, i), j = k0 + r;
    if (j >= n.nk) continue;
    const size_t dst = ((static_cast<size_t>(b) * p.S + j) * p.Hkv + kvh) * p.dh;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int d = tx * 4 + c * 64;
      if (d >= p.dh) continue;
      if (whole) {
        store4<T>(static_cast<T *>(p.dk) + dst + d, dk[i][c], 1.0f);
        store4<T>(static_cast<T *>(p.dv) + dst + d, dv[i][c], 1.0f);
      } else {
        store4<float>(parts + slot + static_cast<size_t>(r) * p.dh + d, dk[i][c], 1.0f);
        store4<float>(parts + slot + static_cast<size_t>(BT + r) * p.dh + d, dv[i][c], 1.0f);
      }
    }
  }
}

// 8 elements of a row, as loaded.
template <typename T> struct Row8 {
  uint4 w[sizeof(T) / 2] = {};
  __device__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
  }
  __device__ float dot(const Row8 &o, float s) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      const uint32_t a[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, c[4] = {o.w[i].x, o.w[i].y, o.w[i].z, o.w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
          s = fmaf(__uint_as_float(a[k]), __uint_as_float(c[k]), s);
        } else {
          s = fmaf(__uint_as_float(a[k] << 16), __uint_as_float(c[k] << 16), s);
          s = fmaf(__uint_as_float(a[k] & 0xFFFF0000u), __uint_as_float(c[k] & 0xFFFF0000u), s);
        }
      }
    }
    return s;
  }
};

// delta[b, h, t] = sum_d dout * out of row (b, t, h). A query that sees few keys gets it
// from them instead, as sum_j p_j (dout . v_j): the stored out is rounded, and that
// error is in each of the row's score gradients alike, where it adds up while their own
// roundings average; its share falls with the number of keys (bf16, rows of 4 tokens,
// 10 heads of 256: dQ and dK off by 3.2e-3 with out's, 2.4e-3 so; rows of 74 tokens
// 2.6e-3 and 2.4e-3). Those are the queries at the first kFew positions, or all where
// window and sinks come to no more. They are a warp each, in the first blocks, so that
// their walks over the keys run beside the others (3 us more on 4 x 2048 tokens, 10
// heads of 256); the others are 8 lanes each.
constexpr int kFew = 16;

// The first tokens of a row whose queries see few keys.
int few_tokens(const AttnArgs &p) {
  if (p.window > 0 && static_cast<long long>(p.window) + p.sinks <= kFew) return p.T;
  const long long n = kFew - (static_cast<long long>(p.S) - p.T);
  return static_cast<int>(n < 0 ? 0 : n < p.T ? n : p.T);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
attn_delta_kernel(const AttnArgs p, float *delta, const int few, const unsigned few_blocks) {
  const bool walk = blockIdx.x < few_blocks;
  const int lanes = walk ? 32 : 8, lane = threadIdx.x & (lanes - 1);
  const long long heads = static_cast<long long>(p.B) * p.Hq, rows = (walk ? few : p.T) * heads;
  // tokens slowest
  const long long item = walk ? static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)
                              : few * heads + static_cast<long long>(blockIdx.x - few_blocks) * (kThreads / 8) +
                                    (threadIdx.x >> 3);
  if (item >= rows) return;                         // whole groups of lanes
  const int h = static_cast<int>(item % p.Hq);
  const long long tb = item / p.Hq;
  const int b = static_cast<int>(tb % p.B), t = static_cast<int>(tb / p.B);
  const long long row = (static_cast<long long>(b) * p.T + t) * p.Hq + h;
  const long long at = (static_cast<long long>(b) * p.Hq + h) * p.T + t;
  const T *x = static_cast<const T *>(p.dout) + row * p.dh;
  const RowLens n = row_lens(p, b);
  float s = 0.0f;
  if (walk) {
    // the keys first .. last, and those before first that are sinks
    const int pos = t + p.S - p.T, last = t < n.nq ? min(pos, n.nk - 1) : -1;
    const int first = p.window > 0 ? max(pos - p.window + 1, 0) : 0, head = min(p.sinks, first);
    const int keys = last < 0 ? 0 : head + max(last - first + 1, 0);
    // a key to 8, 16 or 32 lanes of 8 dims each (dh is 256 at most), and four such at once
    const int wide = p.dh <= 64 ? 8 : p.dh <= 128 ? 16 : 32, slot = lane / wide, d = (lane & (wide - 1)) * 8;
    const int kvh = h / (p.Hq / p.Hkv), at_once = 32 / wide;
    const T *q = head_of<T>(p.q, b, h) + t * p.q.st, *k = head_of<T>(p.k, b, kvh), *v = head_of<T>(p.v, b, kvh);
    const bool in = d < p.dh && keys > 0;
    const float lse = keys > 0 ? p.lse[at] : 0.0f;
    Row8<T> qs, xs;
    if (in) {
      qs.load(q + d);
      xs.load(x + d);
    }
    for (int i0 = slot; i0 < keys + slot; i0 += 4 * at_once) {             // (uniform in the warp)
      Row8<T> ks[4], vs[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int z = min(i0 + i * at_once, keys - 1), j = z < head ? z : first + z - head;
        if (in) {
          ks[i].load(k + j * p.k.st + d);
          vs[i].load(v + j * p.v.st + d);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float qk = qs.dot(ks[i], 0.0f), dv = xs.dot(vs[i], 0.0f);
        for (int w = wide / 2; w > 0; w >>= 1) {
          qk += __shfl_xor_sync(0xFFFFFFFFu, qk, w);
          dv += __shfl_xor_sync(0xFFFFFFFFu, dv, w);
        }
        if (i0 + i * at_once < keys) s = fmaf(expf(qk * p.scale - lse), dv, s);
      }
    }
    for (int w = wide; w < 32; w <<= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, w);
  } else {
    if (t < n.nq) {
      const T *y = static_cast<const T *>(p.out) + row * p.dh;
      for (int d = lane * 8; d < p.dh; d += 64) {
        Row8<T> c, e;
        c.load(x + d);
        e.load(y + d);
        s = c.dot(e, s);
      }
    }
    const unsigned mask = 0xFFu << (threadIdx.x & 24);
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) s += __shfl_xor_sync(mask, s, w);
  }
  if (lane == 0) delta[at] = s;
}

// Sums of the pieces of every tile that has more than one, in their order.
// parts[(b * Hkv + kvh) * slots + slot][dk, dv][tile][dh].
template <typename T>
__global__ void __launch_bounds__(kThreads)
attn_join_kernel(const AttnArgs p, const PiecePlan pl, const float *__restrict__ parts) {
  const int kvh = blockIdx.z % p.Hkv, b = blockIdx.z / p.Hkv;
  const int tile = blockIdx.y, off = p.S - p.T, k0 = tile * pl.tile;
  const RowLens n = row_lens(p, b);
  const Steps st = steps_of(query_range(k0, pl.tile, n.nq, n.nk, off, p.window, p.sinks), pl.step,
                            p.Hq / p.Hkv);
  if (k0 >= n.nk || st.n <= pl.len) return;         // stored by its only piece
  // the pieces that are not empty (rounding the even length up can leave the last so)
  const int asked = (st.n + pl.len - 1) / pl.len, each = (st.n + asked - 1) / asked;
  const int np = (st.n + each - 1) / each;
  const size_t one = static_cast<size_t>(2) * pl.tile * p.dh;
  const float *src = parts + (static_cast<size_t>(blockIdx.z) * pl.slots + first_slot(pl, tile)) * one;
  const int per_row = p.dh / 4;
  for (int i = blockIdx.x * kThreads + threadIdx.x; i < 2 * pl.tile * per_row; i += gridDim.x * kThreads) {
    const int r = (i / per_row) % pl.tile, d = (i % per_row) * 4, j = k0 + r;
    if (j >= n.nk) continue;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int x = 0; x < np; ++x) {
      const float4 v = *reinterpret_cast<const float4 *>(src + x * one + static_cast<size_t>(i) * 4);
      s.x += v.x;
      s.y += v.y;
      s.z += v.z;
      s.w += v.w;
    }
    T *dst = static_cast<T *>(i < pl.tile * per_row ? p.dk : p.dv);
    store4<T>(dst + ((static_cast<size_t>(b) * p.S + j) * p.Hkv + kvh) * p.dh + d, s, 1.0f);
  }
}

// Launches a kernel with a block for each query tile of BT; where those are few, its
// split form with a cluster of blocks for each (fp32, 30 queries, 4 heads of 64: 2048
// keys 183 us in one block, 27 in 8; 128 keys 14.0 in one, 9.9 in two, 7.2 in four of
// one tile each).
template <int BT, typename K, typename... Args>
cudaError_t run_queries(K kernel, K split, int smem, const AttnArgs &p, std::atomic<unsigned long long> (&done)[2],
                        ClusterRoom *room, cudaStream_t st, Args... args) {
  const int tiles = ceil_div(p.T, BT), last = (tiles - 1) * BT + p.S - p.T;
  const long long units = static_cast<long long>(p.B) * p.Hq * tiles;
  int parts = 1;
  cudaError_t e = cluster_parts(split, kThreads, smem, &done[1], room, static_cast<unsigned>(units < 149 ? units : 149),
                                key_tiles(last, p.S - 1, p.S, p.window, p.sinks, BT).n, &parts);
  if (e != cudaSuccess) return e;
  dim3 grid(static_cast<unsigned>(p.B) * p.Hq, tiles);
  if (parts > 1) {
    grid.x *= parts;
    cudaLaunchAttribute attr;
    const cudaLaunchConfig_t cfg = cluster_config(&attr, parts, grid, kThreads, smem, st);
    return cudaLaunchKernelEx(&cfg, split, args..., parts);
  }
  e = opt_in_smem(kernel, smem, done[0]);
  if (e != cudaSuccess) return e;
  kernel<<<grid, kThreads, smem, st>>>(args..., 1);
  return cudaGetLastError();
}

template <typename T, int BT, int NC>
cudaError_t run_fwd(const AttnArgs &p, cudaStream_t st) {
  constexpr int smem = fwd_smem<BT, NC>();
  static_assert(smem <= kMaxSmem, "shared memory");
  static std::atomic<unsigned long long> done[2];
  static ClusterRoom room;
  return run_queries<BT>(attn_fwd_generic_kernel<T, BT, NC, false>, attn_fwd_generic_kernel<T, BT, NC, true>, smem, p,
                         done, &room, st, p);
}

template <typename T, int BT, int NC>
cudaError_t run_bwd(const AttnArgs &p, const float *delta, const PiecePlan &pl, float *parts,
                    cudaStream_t st) {
  constexpr int smem = bwd_smem<BT, NC>();
  static_assert(smem <= kMaxSmem, "shared memory");
  static std::atomic<unsigned long long> done_q[2], done_kv{0};
  static ClusterRoom room;
  cudaError_t e = run_queries<BT>(attn_dq_generic_kernel<T, BT, NC, false>, attn_dq_generic_kernel<T, BT, NC, true>,
                                  smem, p, done_q, &room, st, p, delta);
  if (e != cudaSuccess) return e;
  e = opt_in_smem(attn_dkv_generic_kernel<T, BT, NC>, smem, done_kv);
  if (e != cudaSuccess) return e;
  const dim3 gk(pl.slots, static_cast<unsigned>(p.B) * p.Hkv);
  attn_dkv_generic_kernel<T, BT, NC><<<gk, kThreads, smem, st>>>(p, delta, pl, parts);
  return cudaGetLastError();
}

int bwd_tile(int dh) { return dh <= 128 ? 64 : 48; }

// Pieces of one step and more: a step takes longer than a partial sum (fp32, 256
// queries, 4 heads of 64: 68 us with 4 steps or more, 48 with 2, 36 with 1). Four
// pieces an SM: shorter ones even the blocks out and keep the fp32 sums short (5 x 1009,
// 20/2 heads of 64: 2.27 ms and 7.2e-7 of dK off with one an SM, 1.70 ms and 4.9e-7
// with four; 2 x 1024, 8/1 heads, window 256: 230 us and 156).
PiecePlan generic_plan_of(const AttnArgs &p) {
  const int bt = bwd_tile(p.dh);
  return attn_plan(p.B, p.T, p.S, p.Hq, p.Hkv, p.window, p.sinks, bt, bt, 592, 1);
}

template <typename T> cudaError_t bwd_typed(const AttnArgs &p, void *ws, cudaStream_t st) {
  const PiecePlan pl = generic_plan_of(p);
  float *delta = static_cast<float *>(ws);
  float *parts = delta + align_up(static_cast<size_t>(p.B) * p.Hq * p.T, 64);
  cudaError_t e = launch_attn_delta(p, sizeof(T) == 4 ? RGLRU_IO_F32 : RGLRU_IO_BF16, delta, st);
  if (e != cudaSuccess) return e;
  switch (ceil_div(p.dh, 64)) {
    case 1: e = run_bwd<T, 64, 1>(p, delta, pl, parts, st); break;
    case 2: e = run_bwd<T, 64, 2>(p, delta, pl, parts, st); break;
    case 3: e = run_bwd<T, 48, 3>(p, delta, pl, parts, st); break;
    default: e = run_bwd<T, 48, 4>(p, delta, pl, parts, st); break;
  }
  if (e != cudaSuccess) return e;
  return launch_attn_join(p, sizeof(T) == 4 ? RGLRU_IO_F32 : RGLRU_IO_BF16, pl, parts, st);
}

// Tiles of 64 queries, fewer where the operands of wide heads leave no room; 32 of
// heads up to 128 wide when there are fewer tiles of 64 than SMs (fp32, 2 x 500
// queries, 4 heads of 64, window 256: 42 us with 64, 30 with 32; 192 wide 32 take
// as long as 48).
template <typename T> cudaError_t fwd_typed(const AttnArgs &p, cudaStream_t st) {
  const bool few = static_cast<long long>(p.B) * p.Hq * ceil_div(p.T, 64) < 148;
  switch (ceil_div(p.dh, 64)) {
    case 1: if (few) return run_fwd<T, 32, 1>(p, st); break;
    case 2: if (few) return run_fwd<T, 32, 2>(p, st); break;
    default: break;
  }
  switch (ceil_div(p.dh, 64)) {
    case 1: return run_fwd<T, 64, 1>(p, st);
    case 2: return run_fwd<T, 64, 2>(p, st);
    case 3: return run_fwd<T, 48, 3>(p, st);
    default: return run_fwd<T, 32, 4>(p, st);
  }
}

}  // namespace

PiecePlan attn_plan(int B, int T, int S, int Hq, int Hkv, int window, int sinks, int tile,
                    int step, int target_blocks, int least) {
  PiecePlan pl;
  pl.tile = tile;
  pl.step = step;
  pl.n_tiles = ceil_div(S, tile);
  const long long ns = window > 0 ? (static_cast<long long>(sinks) + tile - 1) / tile : 0;
  pl.n_sink_tiles = static_cast<int>(ns < pl.n_tiles ? ns : pl.n_tiles);
  const int G = Hq / Hkv, off = S - T;
  long long total = 0;
  int most = 0, most_sink = 0;
  for (int i = 0; i < pl.n_tiles; ++i) {
    const int n = steps_of(query_range(i * tile, tile, T, S, off, window, sinks), step, G).n;
    total += n;
    if (i < pl.n_sink_tiles)
      most_sink = n > most_sink ? n : most_sink;
    else
      most = n > most ? n : most;
  }
  total *= static_cast<long long>(B) * Hkv;
  // pieces of the average block's share, never shorter than `least` steps: a piece
  // costs a partial sum of its tile, written and read again
  long long len = (total + target_blocks - 1) / target_blocks;
  if (len < least) len = least;
  pl.len = static_cast<int>(len);
  pl.pieces = most > 0 ? ceil_div(most, pl.len) : 1;
  pl.sink_pieces = most_sink > 0 ? ceil_div(most_sink, pl.len) : 1;
  pl.slots = pl.n_sink_tiles * pl.sink_pieces + (pl.n_tiles - pl.n_sink_tiles) * pl.pieces;
  return pl;
}

size_t attn_delta_bytes(const AttnArgs &p) {
  return align_up(static_cast<size_t>(p.B) * p.Hq * p.T, 64) * sizeof(float);
}

size_t attn_parts_bytes(const AttnArgs &p, const PiecePlan &pl) {
  if (pl.pieces <= 1 && pl.sink_pieces <= 1) return 0;
  return static_cast<size_t>(p.B) * p.Hkv * pl.slots * 2 * pl.tile * p.dh * sizeof(float);
}

cudaError_t launch_attn_delta(const AttnArgs &p, int io, float *delta, cudaStream_t st) {
  const long long heads = static_cast<long long>(p.B) * p.Hq;
  const int few = few_tokens(p);
  const unsigned few_blocks = static_cast<unsigned>((few * heads + kThreads / 32 - 1) / (kThreads / 32));
  const unsigned blocks =
      few_blocks + static_cast<unsigned>(((p.T - few) * heads + kThreads / 8 - 1) / (kThreads / 8));
  if (io == RGLRU_IO_F32)
    attn_delta_kernel<float><<<blocks, kThreads, 0, st>>>(p, delta, few, few_blocks);
  else
    attn_delta_kernel<__nv_bfloat16><<<blocks, kThreads, 0, st>>>(p, delta, few, few_blocks);
  return cudaGetLastError();
}

cudaError_t launch_attn_join(const AttnArgs &p, int io, const PiecePlan &pl, const float *parts,
                             cudaStream_t st) {
  if (pl.pieces <= 1 && pl.sink_pieces <= 1) return cudaSuccess;
  const int per_tile = ceil_div(2 * pl.tile * p.dh / 4, kThreads);
  const dim3 grid(per_tile < 8 ? per_tile : 8, pl.n_tiles, static_cast<unsigned>(p.B) * p.Hkv);
  if (io == RGLRU_IO_F32)
    attn_join_kernel<float><<<grid, kThreads, 0, st>>>(p, pl, parts);
  else
    attn_join_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(p, pl, parts);
  return cudaGetLastError();
}

cudaError_t launch_attn_fwd_generic(const AttnArgs &p, int io, cudaStream_t st) {
  return io == RGLRU_IO_F32 ? fwd_typed<float>(p, st) : fwd_typed<__nv_bfloat16>(p, st);
}

size_t attn_bwd_generic_workspace_bytes(const AttnArgs &p) {
  return attn_delta_bytes(p) + attn_parts_bytes(p, generic_plan_of(p));
}

cudaError_t launch_attn_bwd_generic(const AttnArgs &p, int io, void *ws, cudaStream_t st) {
  return io == RGLRU_IO_F32 ? bwd_typed<float>(p, ws, st) : bwd_typed<__nv_bfloat16>(p, ws, st);
}

}  // namespace rglru
