// Norms of queries and keys per head and their position rotation, in one pass
// over HBM: forward, the serving form that writes a paged cache, and backward
// (include/rglru_attn.h).
//
//   n = x * r * w,  r = rsqrt(mean(x^2) + eps)
//   y_i = n_i cos - n_j sin,  y_j = n_j cos + n_i sin,  j = i + rot/2, i < rot/2
//
// Backward, with g = the rotation's transpose applied to dy:
//   dw = sum over rows of g * x r,   dx = r (g w - x r^2 mean(g w x))
//
// Bound by HBM: x (and dy) read once, y (dx) written once (8 x 2048 tokens, 10 + 1 heads
// of 256: 45 us, 4.1 TB/s; backward of 8 x 2047 tokens, 16 + 4 heads of 128: 62 us, 4.1
// TB/s; the rest of HBM's rate is lost to the rows' arithmetic, some 60 instructions a
// pair of elements, and its latency). One warp takes one
// token and a run of its heads; a lane holds 8 consecutive elements of a row
// (16 bytes of bf16), a row is dh/8 lanes, so narrow heads put several rows in
// a warp, and a lane has 64 bytes of loads in flight. Norm sums are warp shuffles;
// the rotation's partner sits rot/16 lanes away at the same place of its lane (rot
// is a multiple of 16), one shuffle.
// Sine and cosine are formed once per token and warp for all of the run's
// heads. The angle of pair i is position * phase[i] in 64-bit integers, phase
// a fraction of a turn times 2^64: the product modulo 2^64 is the exact
// position within the turn, so far positions keep full precision without
// 64-bit floating point (the phase's own rounding, 2^-65 of a turn, times
// 2^31 positions is 2^-34 of a turn).
#include "attn_kernels.h"
#include "common.cuh"

namespace rglru {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Rows that a lane has in flight: 64 bytes (of q; as much of dy in the backward).
template <typename T> constexpr int rows_in_flight() { return 8 / sizeof(T); }
constexpr int kMaxBlocks = 148 * 3;   // resident at once
constexpr int kBwdBlocks = 148 * 2;   // resident at once; each leaves one partial sum of dw

// 8 elements of a row: as loaded, and as floats.
template <typename T> struct Raw {
  uint4 w[sizeof(T) / 2];
};

struct Row8 {
  float v[8];
};

template <typename T> __device__ __forceinline__ Raw<T> load_raw(const T *p, bool live) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    r.w[i] = live ? __ldg(reinterpret_cast<const uint4 *>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
  return r;
}

__device__ __forceinline__ Row8 floats(const Raw<float> &a) {
  return {{__uint_as_float(a.w[0].x), __uint_as_float(a.w[0].y), __uint_as_float(a.w[0].z),
           __uint_as_float(a.w[0].w), __uint_as_float(a.w[1].x), __uint_as_float(a.w[1].y),
           __uint_as_float(a.w[1].z), __uint_as_float(a.w[1].w)}};
}

__device__ __forceinline__ Row8 floats(const Raw<__nv_bfloat16> &a) {
  const uint32_t w[4] = {a.w[0].x, a.w[0].y, a.w[0].z, a.w[0].w};
  Row8 r;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    r.v[2 * e] = __uint_as_float(w[e] << 16);
    r.v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
  return r;
}

__device__ __forceinline__ void store8(float *p, const Row8 &r) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Row8 &r) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(r.v[2 * e], r.v[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Moved as they are (v into its cache).
template <typename T> __device__ __forceinline__ void store_raw(T *d, const Raw<T> &r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4 *>(d)[i] = r.w[i];
}

template <int LPR> __device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// What a lane needs of the rotation at one token: whether its elements turn,
// the lane that holds their partners, and (cos, +-sin) of each. The first of a
// pair takes -sin (forward), the second +sin; `back` turns the other way.
struct Turn {
  float c[8], s[8];
  bool on;
  int partner;
};

// Sine and cosine of pi x, |x| <= 1: to the last places for fp32 rows; for bf16
// rows by the hardware's instructions, off by at most 2^-21 on this range, far
// below the 2^-8 of the row's own rounding (48 -> 45 us on 185 MB).
__device__ __forceinline__ void turn_of(float x, float &s, float &c, float) { sincospif(x, &s, &c); }
__device__ __forceinline__ void turn_of(float x, float &s, float &c, __nv_bfloat16) {
  __sincosf(x * 3.14159265358979f, &s, &c);
}

template <typename T>
__device__ __forceinline__ void set_turn(Turn &t, const unsigned long long *phase, int pos, int e0,
                                         int half, bool back) {
  if (!t.on) return;
  const bool first = e0 < half;
  const int i0 = first ? e0 : e0 - half;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const unsigned long long turn =
        phase[i0 + e] * static_cast<unsigned long long>(static_cast<long long>(pos));
    // the top 32 bits as a signed fraction of a turn, -1/2 .. 1/2
    const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;
    turn_of(x, t.s[e], t.c[e], T());  // angle = pi x, x = 2 * fraction
    if (first != back) t.s[e] = -t.s[e];
  }
}

__device__ __forceinline__ void rotate(Row8 &n, const Turn &t) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float o = __shfl_sync(0xFFFFFFFFu, n.v[e], t.partner);
    if (t.on) n.v[e] = n.v[e] * t.c[e] + o * t.s[e];
  }
}

// A warp's place: LPR lanes a row (dh/8 of them in use), 32/LPR rows at once.
template <int LPR> struct Place {
  int sub, e0;
  bool in;
  __device__ Place(int lane, int dh) : sub(lane / LPR), e0((lane % LPR) * 8), in(e0 < dh) {}
};

template <int LPR> __device__ __forceinline__ Turn make_turn(int lane, int e0, int rot) {
  Turn t;
  const int half = rot / 2;
  t.on = e0 < rot;
  t.partner = !t.on ? lane : e0 < half ? lane + half / 8 : lane - half / 8;
  return t;
}

__device__ __forceinline__ void stage_phases(unsigned long long *dst, const QkArgs &p) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kThreads) dst[i] = p.phase[i];
}

// This lane's weights, kept as loaded (half the registers in bf16).
template <typename T>
__device__ __forceinline__ Raw<T> weights(const void *w, int e0, bool in) {
  if (w != nullptr) return load_raw(static_cast<const T *>(w) + e0, in);
  const uint32_t one = sizeof(T) == 4 ? 0x3F800000u : 0x3F803F80u;
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.w[i] = make_uint4(one, one, one, one);
  return r;
}

// Rows h0 .. h1-1 (heads of one token) normed and rotated: src and dst at the
// token's head 0 and this lane's elements, sh and dh elements between heads.
template <typename T, int LPR>
__device__ __forceinline__ void norm_rows(const T *src, long long sh, T *dst, int dh, int h0, int h1,
                                          const Place<LPR> &at, const Raw<T> &raw_w,
                                          const Turn &turn, float inv, float eps) {
  constexpr int R = 32 / LPR, kRows = rows_in_flight<T>();
  const Row8 w = floats(raw_w);
  for (int h = h0; h < h1; h += R * kRows) {
    Raw<T> raw[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int hh = h + u * R + at.sub;
      raw[u] = load_raw(src + hh * sh, at.in && hh < h1);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int hh = h + u * R + at.sub;
      if (h + u * R >= h1) break;                       // (the warp's rows all past the end)
      Row8 x = floats(raw[u]);
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x.v[e], x.v[e], ss);
      const float r = rsqrtf(row_sum<LPR>(ss) * inv + eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x.v[e] *= r * w.v[e];
      rotate(x, turn);
      if (at.in && hh < h1) store8(dst + static_cast<long long>(hh) * dh, x);
    }
  }
}

// Their backward: dw is added to, dx written; dy and dx dense.
template <typename T, int LPR>
__device__ __forceinline__ void grad_rows(const T *src, long long sh, const T *dy, T *dx, int dh, int h0,
                                          int h1, const Place<LPR> &at, const Raw<T> &raw_w, Row8 &dw,
                                          const Turn &turn, float inv, float eps) {
  constexpr int R = 32 / LPR, kRows = rows_in_flight<T>();
  const Row8 w = floats(raw_w);
  for (int h = h0; h < h1; h += R * kRows) {
    Raw<T> raw[kRows], rawg[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int hh = h + u * R + at.sub;
      const bool live = at.in && hh < h1;
      raw[u] = load_raw(src + hh * sh, live);
      rawg[u] = load_raw(dy + static_cast<long long>(hh) * dh, live);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int hh = h + u * R + at.sub;
      if (h + u * R >= h1) break;
      const Row8 x = floats(raw[u]);
      Row8 g = floats(rawg[u]);
      float ss = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(x.v[e], x.v[e], ss);
      const float root = rsqrtf(row_sum<LPR>(ss) * inv + eps);
      // (no row here: without eps its root is infinite, and 0 times that would be NaN in dw)
      const float r = hh < h1 ? root : 0.0f;
      rotate(g, turn);
      float gx = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw.v[e] = fmaf(g.v[e], x.v[e] * r, dw.v[e]);
        g.v[e] *= w.v[e];
        gx = fmaf(g.v[e], x.v[e], gx);
      }
      const float c = row_sum<LPR>(gx) * inv * r * r;
#pragma unroll
      for (int e = 0; e < 8; ++e) g.v[e] = r * (g.v[e] - x.v[e] * c);
      if (at.in && hh < h1) store8(dx + static_cast<long long>(hh) * dh, g);
    }
  }
}

// Work item: one token and one of n_runs runs of `run` heads of the list q heads,
// k heads. Tokens times runs stay below 2^31 (there is more than one run only
// where tokens are few).
struct Item {
  unsigned tok;
  int b, t, h0, h1;
  __device__ Item(const QkArgs &p, unsigned it, int run, int n_runs) {
    tok = it;
    h0 = 0;
    if (n_runs > 1) {
      tok = it / static_cast<unsigned>(n_runs);
      h0 = static_cast<int>(it - tok * static_cast<unsigned>(n_runs)) * run;
    }
    b = static_cast<int>(tok / static_cast<unsigned>(p.T));
    t = static_cast<int>(tok - static_cast<unsigned>(b) * static_cast<unsigned>(p.T));
    h1 = min(h0 + run, p.Hq + p.Hkv);
  }
};

template <typename T> __device__ __forceinline__ const T *token_of(const Strided &x, const Item &i, int e0) {
  return static_cast<const T *>(x.p) + i.b * x.sb + i.t * x.st + e0;
}

// Forward (kAppend: k and v rows go to the cache).
template <typename T, int LPR, bool kAppend>
__global__ void __launch_bounds__(kThreads, 3) qk_fwd_kernel(const __grid_constant__ QkArgs p,
                                                             int run, int n_runs) {
  __shared__ unsigned long long phase[kMaxPairs];
  stage_phases(phase, p);
  __syncthreads();
  constexpr int R = 32 / LPR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place<LPR> at(lane, p.dh);
  const Raw<T> wq = weights<T>(p.w_q, at.e0, at.in), wk = weights<T>(p.w_k, at.e0, at.in);
  Turn turn = make_turn<LPR>(lane, at.e0, p.rot);
  const float inv = 1.0f / static_cast<float>(p.dh);
  const unsigned items = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.T) * n_runs;
  for (unsigned x = blockIdx.x * kWarps + warp; x < items; x += gridDim.x * kWarps) {
    const Item it(p, x, run, n_runs);
    const int pos = p.positions ? __ldg(p.positions + it.tok) : it.t;
    T *q_out = static_cast<T *>(p.q_out) + static_cast<long long>(it.tok) * p.Hq * p.dh + at.e0;
    T *k_out = nullptr;
    long long slot = 0;
    const int k0 = max(it.h0 - p.Hq, 0), k1 = it.h1 - p.Hq;
    if (kAppend) {
      if (pos < 0) {                                    // padding (the warp's one token)
        for (int h = it.h0 + at.sub; h < min(it.h1, p.Hq); h += R)
          if (at.in) store8(q_out + static_cast<long long>(h) * p.dh, Row8{});
        continue;
      }
      const int pg = pos / p.page_size;
      const int page = pg < p.max_pages
                           ? __ldg(p.page_table + static_cast<long long>(it.b) * p.max_pages + pg)
                           : -1;
      if (page >= 0 && page < p.num_pages) {
        slot = (static_cast<long long>(page) * p.page_size + pos % p.page_size) * p.Hkv * p.dh + at.e0;
        k_out = static_cast<T *>(p.k_cache) + slot;
      } else if (p.dev_status && lane == 0) {
        atomicCAS(p.dev_status, 0, RGLRU_ERR_INVALID_ARG);
      }
    } else {
      k_out = static_cast<T *>(p.k_out) + static_cast<long long>(it.tok) * p.Hkv * p.dh + at.e0;
    }
    set_turn<T>(turn, phase, pos, at.e0, p.rot / 2, false);
    norm_rows<T, LPR>(token_of<T>(p.q, it, at.e0), p.q.sh, q_out, p.dh, it.h0, min(it.h1, p.Hq), at, wq,
                      turn, inv, p.eps);
    if (k_out == nullptr) continue;                     // no cache slot (the warp's one token)
    norm_rows<T, LPR>(token_of<T>(p.k, it, at.e0), p.k.sh, k_out, p.dh, k0, k1, at, wk, turn, inv, p.eps);
    if (kAppend) {
      const T *v = token_of<T>(p.v, it, at.e0);
      for (int h = k0 + at.sub; h < k1; h += R)
        if (at.in)
          store_raw(static_cast<T *>(p.v_cache) + slot + static_cast<long long>(h) * p.dh,
                    load_raw(v + h * p.v.sh, true));
    }
  }
}

// Backward; each block leaves its sums of dw_q and dw_k in partial[block][2][dh].
// A lane adds up a few rows of dw in registers, at least kFold steps of its warp's rows
// and at most a token's more, and then folds them into a sum in shared memory that keeps
// what each addition rounds off, so that the error does not grow with the number of rows
// (4 x 2^20 equal fp32 rows: 2.4e-6 off in one 32-bit sum a lane, nothing so; 8 x 2047
// random tokens, 16 heads of 128: 1.5e-7 and 8e-8, what the terms themselves are off by,
// in 85.8 and 88.4 us). bf16 rows, whose arithmetic does not hide behind HBM, fold less
// often (60.8 -> 61.5 us on 16/4 heads of 128; every 8 steps 63.5 us).
template <typename T> constexpr int kFold = sizeof(T) == 4 ? 8 : 64;

// s + x, s as a rounded sum and what it lacks (Knuth's exact sum of two numbers).
__device__ __forceinline__ float2 add_exact(float2 s, float x) {
  const float t = __fadd_rn(s.x, x), z = __fsub_rn(t, s.x);
  const float lost = __fadd_rn(__fsub_rn(s.x, __fsub_rn(t, z)), __fsub_rn(x, z));
  return make_float2(t, s.y + lost);
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kThreads, 2) qk_bwd_kernel(const __grid_constant__ QkArgs p,
                                                             int run, int n_runs, double *partial) {
  __shared__ unsigned long long phase[kMaxPairs];
  __shared__ float2 sums[16][kThreads + 1];             // [q, k][8 elements] of each lane
  stage_phases(phase, p);
#pragma unroll
  for (int e = 0; e < 16; ++e) sums[e][threadIdx.x] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Place<LPR> at(lane, p.dh);
  const Raw<T> wq = weights<T>(p.w_q, at.e0, at.in), wk = weights<T>(p.w_k, at.e0, at.in);
  Turn turn = make_turn<LPR>(lane, at.e0, p.rot);
  Row8 dwq = {}, dwk = {};
  int steps = 0;
  auto fold = [&]() {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sums[e][threadIdx.x] = add_exact(sums[e][threadIdx.x], dwq.v[e]);
      sums[8 + e][threadIdx.x] = add_exact(sums[8 + e][threadIdx.x], dwk.v[e]);
    }
    dwq = dwk = Row8{};
    steps = 0;
  };
  const float inv = 1.0f / static_cast<float>(p.dh);
  const unsigned items = static_cast<unsigned>(p.B) * static_cast<unsigned>(p.T) * n_runs;
  for (unsigned x = blockIdx.x * kWarps + warp; x < items; x += gridDim.x * kWarps) {
    const Item it(p, x, run, n_runs);
    const int pos = p.positions ? __ldg(p.positions + it.tok) : it.t;
    set_turn<T>(turn, phase, pos, at.e0, p.rot / 2, true);
    const long long oq = static_cast<long long>(it.tok) * p.Hq * p.dh + at.e0;
    const long long ok = static_cast<long long>(it.tok) * p.Hkv * p.dh + at.e0;
    grad_rows<T, LPR>(token_of<T>(p.q, it, at.e0), p.q.sh, static_cast<const T *>(p.dq_out) + oq,
                      static_cast<T *>(p.q_out) + oq, p.dh, it.h0, min(it.h1, p.Hq), at, wq, dwq, turn,
                      inv, p.eps);
    grad_rows<T, LPR>(token_of<T>(p.k, it, at.e0), p.k.sh, static_cast<const T *>(p.dk_out) + ok,
                      static_cast<T *>(p.k_out) + ok, p.dh, max(it.h0 - p.Hq, 0), it.h1 - p.Hq, at, wk,
                      dwk, turn, inv, p.eps);
    steps += run * LPR / 32 + 1;
    if (steps >= kFold<T>) fold();
  }
  fold();
  __syncthreads();
  // the lanes LPR apart, of every warp, hold the same elements: kGroup threads a column
  constexpr int kLanes = kThreads / LPR, kGroup = LPR < 16 ? 16 / LPR : 1;
  const int g = threadIdx.x % kGroup;
  for (int i = threadIdx.x / kGroup; i < 2 * p.dh; i += kThreads / kGroup) {
    const int d = i % p.dh;
    double s = 0.0;
    float lost = 0.0f;
#pragma unroll 8
    for (int x = g; x < kLanes; x += kGroup) {
      const float2 v = sums[i / p.dh * 8 + d % 8][x * LPR + d / 8];
      s += static_cast<double>(v.x);
      lost += v.y;
    }
    s += static_cast<double>(lost);
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (g == 0) partial[static_cast<size_t>(blockIdx.x) * 2 * p.dh + i] = s;
  }
}

// dw[i] = sum over the blocks of partial[block][i]: one warp a
// column, lanes over the blocks, a fixed order.
__global__ void __launch_bounds__(kThreads) qk_dw_kernel(const double *__restrict__ partial,
                                                         int blocks, int dh, float *dw_q,
                                                         float *dw_k) {
  const int i = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (i >= 2 * dh) return;
  double s = 0.0;
  for (int b = lane; b < blocks; b += 32) s += partial[static_cast<size_t>(b) * 2 * dh + i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  float *dst = i < dh ? dw_q : dw_k;
  if (lane == 0 && dst != nullptr) dst[i % dh] = static_cast<float>(s);
}

// Heads per work item: all of a token's (its sines are then formed once), or
// fewer when that leaves warps without work.
int heads_per_item(long long tokens, int heads, int rows_at_once) {
  const long long warps = 148ll * 4 * kWarps;
  int n_runs = 1;
  if (tokens < warps) n_runs = static_cast<int>((warps + tokens - 1) / (tokens > 0 ? tokens : 1));
  const int most = ceil_div(heads, rows_at_once);
  if (n_runs > most) n_runs = most;
  const int run = ceil_div(heads, n_runs);
  return ceil_div(run, rows_at_once) * rows_at_once;
}

int lanes_per_row(int dh) {
  int l = 1;
  while (l * 8 < dh) l *= 2;
  return l;
}

template <typename T, int LPR>
cudaError_t launch(const QkArgs &p, int mode, double *partial, int blocks, int run, int n_runs,
                   cudaStream_t st) {
  if (mode == 0)
    qk_fwd_kernel<T, LPR, false><<<blocks, kThreads, 0, st>>>(p, run, n_runs);
  else if (mode == 1)
    qk_fwd_kernel<T, LPR, true><<<blocks, kThreads, 0, st>>>(p, run, n_runs);
  else
    qk_bwd_kernel<T, LPR><<<blocks, kThreads, 0, st>>>(p, run, n_runs, partial);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_lpr(const QkArgs &p, int mode, double *partial, int blocks, int run, int n_runs,
                       cudaStream_t st) {
  switch (lanes_per_row(p.dh)) {
    case 1: return launch<T, 1>(p, mode, partial, blocks, run, n_runs, st);
    case 2: return launch<T, 2>(p, mode, partial, blocks, run, n_runs, st);
    case 4: return launch<T, 4>(p, mode, partial, blocks, run, n_runs, st);
    case 8: return launch<T, 8>(p, mode, partial, blocks, run, n_runs, st);
    case 16: return launch<T, 16>(p, mode, partial, blocks, run, n_runs, st);
    default: return launch<T, 32>(p, mode, partial, blocks, run, n_runs, st);
  }
}

int qk_blocks(int B, int T, int Hq, int Hkv, int dh, int most, int *run, int *n_runs) {
  const int heads = Hq + Hkv;
  *run = heads_per_item(static_cast<long long>(B) * T, heads, 32 / lanes_per_row(dh));
  *n_runs = ceil_div(heads, *run);
  const long long items = static_cast<long long>(B) * T * *n_runs;
  const long long blocks = (items + kWarps - 1) / kWarps;
  return static_cast<int>(blocks < most ? blocks : most);
}

cudaError_t run_mode(const QkArgs &p, int io, int mode, cudaStream_t st) {
  int run, n_runs;
  const int blocks = qk_blocks(p.B, p.T, p.Hq, p.Hkv, p.dh, kMaxBlocks, &run, &n_runs);
  return io == RGLRU_IO_F32 ? launch_lpr<float>(p, mode, nullptr, blocks, run, n_runs, st)
                            : launch_lpr<__nv_bfloat16>(p, mode, nullptr, blocks, run, n_runs, st);
}

}  // namespace

cudaError_t launch_qk_fwd(const QkArgs &p, int io, cudaStream_t st) { return run_mode(p, io, 0, st); }

cudaError_t launch_qk_append(const QkArgs &p, int io, cudaStream_t st) {
  return run_mode(p, io, 1, st);
}

size_t qk_bwd_workspace_bytes(int B, int T, int Hq, int Hkv, int dh) {
  int run, n_runs;
  const int blocks = qk_blocks(B, T, Hq, Hkv, dh, kBwdBlocks, &run, &n_runs);
  return static_cast<size_t>(blocks) * 2 * dh * sizeof(double);
}

cudaError_t launch_qk_bwd(const QkArgs &p, int io, void *ws, cudaStream_t st) {
  int run, n_runs;
  const int blocks = qk_blocks(p.B, p.T, p.Hq, p.Hkv, p.dh, kBwdBlocks, &run, &n_runs);
  double *partial = static_cast<double *>(ws);
  const cudaError_t e =
      io == RGLRU_IO_F32 ? launch_lpr<float>(p, 2, partial, blocks, run, n_runs, st)
                         : launch_lpr<__nv_bfloat16>(p, 2, partial, blocks, run, n_runs, st);
  if (e != cudaSuccess || (p.dw_q == nullptr && p.dw_k == nullptr)) return e;
  qk_dw_kernel<<<ceil_div(2 * p.dh, kWarps), kThreads, 0, st>>>(partial, blocks, p.dh, p.dw_q,
                                                                p.dw_k);
  return cudaGetLastError();
}

}  // namespace rglru
