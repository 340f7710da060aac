// Attention of one new token of each sequence over its paged cache
// (include/rglru_attn.h): out = softmax(scale q K^T) V over the visible keys.
//
// Bound by HBM: the visible K and V rows are read once, everything else is
// small. The visible keys of a sequence (its first `sinks`, then its last
// `window`) are numbered without the gap between them, so that the kernels walk
// one range and only its end is ragged. The range is cut into chunks of a fixed
// number of keys, one thread block a (chunk, sequence, key head, up to 16 query
// heads of the group): long caches of few sequences fill the GPU, and ragged
// lengths stay balanced, since a block's work does not depend on its sequence's
// length. Blocks past a sequence's end return at once. With more than one chunk
// a sequence, each leaves (max, sum, unnormalised out) in float and
// decode_join_kernel joins them in the order of the chunks.
//
// A key whose page number is out of range is hidden (and reported).
#include <math.h>

#include <algorithm>

#include "attn_kernels.h"
#include "common.cuh"

namespace rglru {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The visible keys of sequence b: u = 0 .. nk-1 stands for key u (u < head) or
// u + jump. Keys past what the table names are hidden (and the length reported);
// the window stays where the length puts it.
struct Keys {
  int nk, head, jump;
};

__device__ __forceinline__ Keys visible_keys(const DecodeArgs &p, int b) {
  const int n = __ldg(p.lens + b), cap = p.max_pages * p.page_size;
  if (n > cap && p.dev_status && threadIdx.x == 0) atomicCAS(p.dev_status, 0, RGLRU_ERR_INVALID_ARG);
  const int end = max(min(n, cap), 0);
  Keys k = {end, end, 0};
  if (p.window > 0 && n > p.window) {
    const int start = n - p.window;                // the window's first key
    k.head = min(p.sinks, min(start, end));
    k.nk = k.head + max(end - start, 0);
    k.jump = start - k.head;
  }
  return k;
}

// Row of the cache (in rows of Hkv * dh elements) that holds visible key u of
// sequence b, or -1 when its page is out of range.
__device__ __forceinline__ long long cache_row(const DecodeArgs &p, int b, const Keys &k, int u) {
  const int j = u < k.head ? u : u + k.jump;
  const int pg = j / p.page_size;
  const int page = __ldg(p.page_table + static_cast<long long>(b) * p.max_pages + pg);
  if (page < 0 || page >= p.num_pages) {
    if (p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_INVALID_ARG);
    return -1;
  }
  return static_cast<long long>(page) * p.page_size + (j - pg * p.page_size);
}

__device__ __forceinline__ uint32_t saddr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// 16 bytes to shared memory; zeros when !full.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool full) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(full ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 2^x by the hardware's instruction (2 units in the last place, 0 for -inf).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Parts {
  float *o;      // [B][Hq][chunks][dh] unnormalised sums
  float2 *ml;    // [B][Hq][chunks] (max in log2 units, sum); max = -inf: nothing seen
  int chunks, chunk;
};

// Block -> (chunk, sequence, key head, slice of the group's query heads).
struct Unit {
  int c, b, kvh, g0;
};
__device__ __forceinline__ Unit unit_of(const DecodeArgs &p, int slices, int per) {
  unsigned x = blockIdx.x;
  Unit u;
  u.g0 = static_cast<int>(x % slices) * per;
  x /= slices;
  u.kvh = static_cast<int>(x % p.Hkv);
  x /= p.Hkv;
  u.b = static_cast<int>(x % p.B);
  u.c = static_cast<int>(x / p.B);
  return u;
}

// -------------------------------------------------- bf16, 64/128/256-wide heads
//
// The 16 query heads of a group that share a key head make the 16 rows of
// mma.m16n8k16 (the tensor core is needed: 10 heads over one 256-wide bf16 key
// are 20 flop a byte, more than CUDA cores do at HBM speed; the tcgen05 MMA's
// 128 rows would hold 16 useful ones, and the 16-row instruction has margin: 64
// MMAs per 16 KB of K and V, under a third of the time HBM needs for them).
// Every warp works alone: its own 16-key groups, its own ring of cp.async
// stages, its own running max, sum and out; the four warps are joined once at
// the end, so the loop has no block barrier. A row of the ring is XOR-swizzled
// in 16-byte pieces, so ldmatrix reads without bank conflicts. Each step's rows
// of the page table are read one step ahead of the copies that need them.
constexpr int kDecWarps = 4;
constexpr int kStages = 3;

template <int DH> constexpr int decode_smem() {
  return kDecWarps * kStages * 2 * 16 * DH * 2 + kDecWarps * (kStages * 4 + 16 * 8) + 64;
}

template <int DH>
__global__ void __launch_bounds__(kDecWarps * 32)
paged_decode_kernel(const DecodeArgs p, const Parts parts, int slices) {
  extern __shared__ __align__(128) unsigned char sm[];
  constexpr int kRow = DH * 2;                     // bytes of a K or V row
  constexpr int kHalf = 16 * kRow;                 // one group's K (or V)
  constexpr int kPer = DH / 8;                     // 16-byte pieces of a row
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Unit un = unit_of(p, slices, 16);
  const Keys ks = visible_keys(p, un.b);
  const int u0 = un.c * parts.chunk, u1 = u0 + min(parts.chunk, ks.nk - u0);   // (the sums stay below 2^31)
  const int G = p.Hq / p.Hkv, g = min(16, G - un.g0);
  const long long hrow = static_cast<long long>(un.b) * p.Hq + un.kvh * G + un.g0;
  if (u0 >= u1) {
    if (un.c == 0) {                               // an empty sequence
      __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + hrow * DH;
      for (int i = threadIdx.x; i < g * DH; i += blockDim.x) o[i] = __float2bfloat16_rn(0.0f);
    }
    return;
  }
  unsigned char *ring = sm + warp * (kStages * 2 * kHalf);
  const uint32_t ring_s = saddr(ring);
  uint32_t *vmask = reinterpret_cast<uint32_t *>(sm + kDecWarps * kStages * 2 * kHalf) + warp * kStages;
  float2 *ml_s = reinterpret_cast<float2 *>(sm + kDecWarps * kStages * 2 * kHalf +
                                            kDecWarps * kStages * 4);

  const long long head_off = static_cast<long long>(un.kvh) * DH;
  const long long row_len = static_cast<long long>(p.Hkv) * DH;
  const __nv_bfloat16 *kc = static_cast<const __nv_bfloat16 *>(p.k_cache) + head_off;
  const __nv_bfloat16 *vc = static_cast<const __nv_bfloat16 *>(p.v_cache) + head_off;

  // q as the A operand: rows lane/4 and lane/4 + 8, two consecutive k a register
  uint32_t qa[DH / 16][4];
  {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + hrow * DH;
    const int r = lane >> 2, c = (lane & 3) * 2;
#pragma unroll
    for (int k = 0; k < DH / 16; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r + (i & 1) * 8, col = k * 16 + c + (i >> 1) * 8;
        qa[k][i] = row < g ? __ldg(reinterpret_cast<const uint32_t *>(q + row * DH + col)) : 0u;
      }
  }

  // this warp's groups: u0 + 16 * (warp + 4 i)
  const int n = u1 - u0 > warp * 16 ? (u1 - u0 - warp * 16 + 63) / 64 : 0;
  auto row_of = [&](int i) -> long long {          // lanes 0..15: the group's cache rows
    const int x = 16 * (warp + kDecWarps * i) + lane;
    return (i < n && lane < 16 && x < u1 - u0) ? cache_row(p, un.b, ks, u0 + x) : -1;
  };
  auto issue = [&](int i, long long row) {
    const int s = i % kStages;
    const uint32_t valid = __ballot_sync(0xFFFFFFFFu, row >= 0) & 0xFFFFu;
    if (i < n) {
      if (lane == 0) vmask[s] = valid;
      const long long off = row < 0 ? 0 : row * row_len;
      const uint32_t dst = ring_s + s * 2 * kHalf;
#pragma unroll
      for (int it = 0; it < 16 * kPer / 32; ++it) {
        const int id = it * 32 + lane, r = id / kPer, c = id % kPer;
        const long long o = __shfl_sync(0xFFFFFFFFu, off, r) + c * 8;
        const bool in = (valid >> r) & 1u;
        const uint32_t d = dst + r * kRow + ((c ^ (r & 7)) << 4);
        cp16(d, kc + o, in);
        cp16(d + kHalf, vc + o, in);
      }
    }
    cp_commit();
  };

  float o[DH / 8][4];
#pragma unroll
  for (int i = 0; i < DH / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  const float sc = p.scale * kLog2e;

#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i, row_of(i));
  long long next = row_of(kStages - 1);
  for (int i = 0; i < n; ++i) {
    __syncwarp();                                  // the slot's readers are done
    issue(i + kStages - 1, next);
    next = row_of(i + kStages);
    cp_wait<kStages - 1>();
    __syncwarp();
    const int s = i % kStages;
    const uint32_t kb = ring_s + s * 2 * kHalf, vb = kb + kHalf;
    const uint32_t valid = vmask[s];
    // S = q K^T: 16 heads x 16 keys, even and odd k steps in separate sums
    float acc[2][2][4] = {};
    const int mi = lane >> 3, mr = lane & 7;
#pragma unroll
    for (int k = 0; k < DH / 16; ++k) {
      uint32_t b[4];
      const int key = (mi >> 1) * 8 + mr;
      ldsm4(b, kb + key * kRow + (((k * 2 + (mi & 1)) ^ mr) << 4));
      mma16816(acc[k & 1][0], qa[k], b[0], b[1]);
      mma16816(acc[k & 1][1], qa[k], b[2], b[3]);
    }
    float sv[2][4];
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int key = t * 8 + (lane & 3) * 2 + (e & 1);
        sv[t][e] = (valid >> key) & 1u ? (acc[0][t][e] + acc[1][t][e]) * sc : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], sv[t][e]);
      }
    bool grow = false;
    float mn[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xFFFFFFFFu, mx[h], 2));
      // the reference maximum moves only when it is 8 or more behind (weights up
      // to 2^8 keep their relative precision), so out is seldom rescaled
      mn[h] = mx[h] > m[h] + 8.0f || m[h] == -INFINITY ? fmaxf(mx[h], m[h]) : m[h];
      grow |= mn[h] != m[h];
    }
    if (__any_sync(0xFFFFFFFFu, grow)) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f[h] = m[h] == -INFINITY ? 0.0f : ex2(m[h] - mn[h]);
        l[h] *= f[h];
        m[h] = mn[h];
      }
#pragma unroll
      for (int t = 0; t < DH / 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][e] *= f[e >> 1];
    }
    uint32_t pa[4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float base = m[h] == -INFINITY ? 0.0f : m[h];
        const float a = ex2(sv[t][2 * h] - base), b = ex2(sv[t][2 * h + 1] - base);
        l[h] += a + b;
        pa[t * 2 + h] = pack_bf16(a, b);
      }
#pragma unroll
    for (int d = 0; d < DH / 16; ++d) {
      uint32_t b[4];
      const int key = (mi & 1) * 8 + mr;
      ldsm4t(b, vb + key * kRow + (((d * 2 + (mi >> 1)) ^ mr) << 4));
      mma16816(o[2 * d], pa, b[0], b[1]);
      mma16816(o[2 * d + 1], pa, b[2], b[3]);
    }
  }
  cp_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 1);
    l[h] += __shfl_xor_sync(0xFFFFFFFFu, l[h], 2);
  }
  __syncthreads();                                 // every ring is free
  float *ow = reinterpret_cast<float *>(sm) + warp * 16 * DH;
  const int r = lane >> 2;
#pragma unroll
  for (int t = 0; t < DH / 8; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2 *>(ow + (r + 8 * h) * DH + t * 8 + (lane & 3) * 2) =
          make_float2(o[t][2 * h], o[t][2 * h + 1]);
  if ((lane & 3) == 0)
#pragma unroll
    for (int h = 0; h < 2; ++h) ml_s[warp * 16 + r + 8 * h] = make_float2(m[h], l[h]);
  __syncthreads();
  const float *os = reinterpret_cast<const float *>(sm);
  for (int i = threadIdx.x; i < g * (DH / 4); i += blockDim.x) {
    const int row = i / (DH / 4), d = (i % (DH / 4)) * 4;
    float mm = -INFINITY, ll = 0.0f;
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) mm = fmaxf(mm, ml_s[w * 16 + row].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kDecWarps; ++w) {
      const float2 ml = ml_s[w * 16 + row];
      const float f = ml.y == 0.0f ? 0.0f : ex2(ml.x - mm);   // (NaN scores leave NaN sums)
      const float4 v = *reinterpret_cast<const float4 *>(os + (w * 16 + row) * DH + d);
      ll = fmaf(f, ml.y, ll);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    if (parts.chunks == 1) {
      const float inv = ll == 0.0f ? 0.0f : 1.0f / ll;
      *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + (hrow + row) * DH + d) =
          make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
    } else {
      const long long part = (hrow + row) * parts.chunks + un.c;
      *reinterpret_cast<float4 *>(parts.o + part * DH + d) = acc;
      if (d == 0) parts.ml[part] = make_float2(mm, ll);
    }
  }
}

// ------------------------------------------------------- fp32, and other widths
//
// CUDA cores in fp32. A block of 8 warps takes 8 query heads and walks tiles of
// 32 keys, double-buffered by cp.async. Scores: lane = key, the warps share out
// the row's pieces of 4 elements, their sums meet in shared memory; then warp g
// owns head g (max, sum and the tile's weights, lane = key); then thread = one
// dim of out for all 8 heads (narrow heads: several groups of keys).
constexpr int kGenThreads = 256;
constexpr int kGenHeads = 8;
constexpr int kGenKeys = 32;

struct GenLayout {
  int pitch;          // bytes of a K or V row in shared memory
  int stage;          // bytes of K and V of one tile
  int off_q, off_s, off_p, off_misc, total;
};

__host__ __device__ inline GenLayout gen_layout(int dh, int eb) {
  GenLayout L;
  L.pitch = dh * eb + 16;
  L.stage = 2 * kGenKeys * L.pitch;
  L.off_q = 2 * L.stage;
  L.off_s = L.off_q + kGenHeads * dh * 4;
  L.off_p = L.off_s + 8 * kGenHeads * kGenKeys * 4;
  L.off_misc = L.off_p + kGenKeys * kGenHeads * 4;
  L.total = L.off_misc + kGenHeads * 4 + kGenHeads * 8 + 16;
  return L;
}

__device__ __forceinline__ float4 four(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 four(const __nv_bfloat16 *p) {
  const uint2 w = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xFFFF0000u));
}

template <typename T>
__global__ void __launch_bounds__(kGenThreads)
paged_decode_generic_kernel(const DecodeArgs p, const Parts parts, int slices) {
  extern __shared__ __align__(128) unsigned char sm[];
  const int dh = p.dh;
  const GenLayout L = gen_layout(dh, sizeof(T));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Unit un = unit_of(p, slices, kGenHeads);
  const Keys ks = visible_keys(p, un.b);
  const int u0 = un.c * parts.chunk, u1 = u0 + min(parts.chunk, ks.nk - u0);   // (the sums stay below 2^31)
  const int G = p.Hq / p.Hkv, g = min(kGenHeads, G - un.g0);
  const long long hrow = static_cast<long long>(un.b) * p.Hq + un.kvh * G + un.g0;
  if (u0 >= u1) {
    if (un.c == 0)
      for (int i = tid; i < g * dh; i += kGenThreads)
        static_cast<T *>(p.out)[hrow * dh + i] = from_f32<T>(0.0f);
    return;
  }
  float *qs = reinterpret_cast<float *>(sm + L.off_q);
  float *ss = reinterpret_cast<float *>(sm + L.off_s);   // [8 warps][8 heads][32 keys]
  float *ps = reinterpret_cast<float *>(sm + L.off_p);   // [32 keys][8 heads]
  float *fs = reinterpret_cast<float *>(sm + L.off_misc);        // [8] rescaling
  float2 *mls = reinterpret_cast<float2 *>(sm + L.off_misc + 32);  // [8]
  unsigned char *vmask = sm + L.off_misc + 32 + 64;               // [2 stages][8], 4 keys each
  for (int i = tid; i < kGenHeads * dh; i += kGenThreads)
    qs[i] = i < g * dh ? to_f32<T>(static_cast<const T *>(p.q)[hrow * dh + i]) : 0.0f;

  const int n = (u1 - u0 + kGenKeys - 1) / kGenKeys;
  const long long row_len = static_cast<long long>(p.Hkv) * dh;
  const long long head_off = static_cast<long long>(un.kvh) * dh;
  const int pieces = dh * static_cast<int>(sizeof(T)) / 16;
  constexpr int kE = 16 / sizeof(T);
  auto issue = [&](int i) {
    if (i < n) {
      // 8 threads a key
      const int key = tid >> 3, x = i * kGenKeys + key;
      const long long row = x < u1 - u0 ? cache_row(p, un.b, ks, u0 + x) : -1;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, row >= 0);  // keys 4 warp .. +3, 8 bits each
      if (lane == 0) {
        const uint32_t bits = (m & 1u) | ((m >> 7) & 2u) | ((m >> 14) & 4u) | ((m >> 21) & 8u);
        vmask[(i & 1) * 8 + warp] = static_cast<unsigned char>(bits);
      }
      unsigned char *st = sm + (i & 1) * L.stage + key * L.pitch;
      const long long o = (row < 0 ? 0 : row) * row_len + head_off;
      for (int c = tid & 7; c < pieces; c += 8) {
        cp16(saddr(st + c * 16), static_cast<const T *>(p.k_cache) + o + c * kE, row >= 0);
        cp16(saddr(st + kGenKeys * L.pitch + c * 16), static_cast<const T *>(p.v_cache) + o + c * kE,
             row >= 0);
      }
    }
    cp_commit();
  };

  int groups = 1, dhp = 1;
  while (dhp < dh) dhp *= 2;
  groups = kGenThreads / dhp;                      // groups of keys of the second product
  const int d = tid % dhp, kg = tid / dhp;
  float o[kGenHeads] = {};
  float m = -INFINITY, l = 0.0f;                   // of head `warp`
  const float sc = p.scale * kLog2e;
  issue(0);
  for (int i = 0; i < n; ++i) {
    issue(i + 1);
    cp_wait<1>();
    __syncthreads();
    const unsigned char *kt = sm + (i & 1) * L.stage, *vt = kt + kGenKeys * L.pitch;
    {
      float acc[kGenHeads] = {};
      const T *kr = reinterpret_cast<const T *>(kt + lane * L.pitch);
      for (int c = warp; c < dh / 4; c += 8) {
        const float4 kv = four(kr + c * 4);
#pragma unroll
        for (int h = 0; h < kGenHeads; ++h) {
          const float4 qv = *reinterpret_cast<const float4 *>(qs + h * dh + c * 4);
          acc[h] = fmaf(kv.x, qv.x, fmaf(kv.y, qv.y, fmaf(kv.z, qv.z, fmaf(kv.w, qv.w, acc[h]))));
        }
      }
#pragma unroll
      for (int h = 0; h < kGenHeads; ++h) ss[(warp * kGenHeads + h) * kGenKeys + lane] = acc[h];
    }
    __syncthreads();
    {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) s += ss[(w * kGenHeads + warp) * kGenKeys + lane];
      s = (vmask[(i & 1) * 8 + (lane >> 2)] >> (lane & 3)) & 1 ? s * sc : -INFINITY;
      float mx = s;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
      const float mn = fmaxf(m, mx);
      const float w = s == -INFINITY ? 0.0f : exp2f(s - mn);
      const float f = m == -INFINITY ? 0.0f : exp2f(m - mn);
      float sum = w;
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
      l = l * f + sum;
      m = mn;
      ps[lane * kGenHeads + warp] = w;
      if (lane == 0) fs[warp] = f;
    }
    __syncthreads();
    if (d < dh) {
#pragma unroll
      for (int h = 0; h < kGenHeads; ++h) o[h] *= fs[h];
      for (int key = kg; key < kGenKeys; key += groups) {
        const float v = to_f32<T>(reinterpret_cast<const T *>(vt + key * L.pitch)[d]);
        const float4 a = *reinterpret_cast<const float4 *>(ps + key * kGenHeads);
        const float4 b = *reinterpret_cast<const float4 *>(ps + key * kGenHeads + 4);
        o[0] = fmaf(a.x, v, o[0]);
        o[1] = fmaf(a.y, v, o[1]);
        o[2] = fmaf(a.z, v, o[2]);
        o[3] = fmaf(a.w, v, o[3]);
        o[4] = fmaf(b.x, v, o[4]);
        o[5] = fmaf(b.y, v, o[5]);
        o[6] = fmaf(b.z, v, o[6]);
        o[7] = fmaf(b.w, v, o[7]);
      }
    }
    __syncthreads();                               // the tile's buffer is free
  }
  cp_wait<0>();
  if (lane == 0) mls[warp] = make_float2(m, l);
  float *red = reinterpret_cast<float *>(sm);      // [groups][8][dh]: at most 8 KB, the ring's start
  if (d < dh)
#pragma unroll
    for (int h = 0; h < kGenHeads; ++h) red[(kg * kGenHeads + h) * dh + d] = o[h];
  __syncthreads();
  for (int i = tid; i < g * dh; i += kGenThreads) {
    const int h = i / dh;
    float s = 0.0f;
    for (int x = 0; x < groups; ++x) s += red[x * kGenHeads * dh + i];
    const float2 ml = mls[h];
    if (parts.chunks == 1) {
      static_cast<T *>(p.out)[hrow * dh + i] = from_f32<T>(ml.y == 0.0f ? 0.0f : s / ml.y);
    } else {
      const long long part = (hrow + h) * parts.chunks + un.c;
      parts.o[part * dh + i % dh] = s;
      if (i % dh == 0) parts.ml[part] = ml;
    }
  }
}

// --------------------------------------------------------------------- the join
//
// One block a (sequence, query head): out = sum_c 2^(m_c - M) o_c / sum_c 2^(m_c - M) l_c.
// Threads are dh/4 columns of 4 dims by groups that share out the chunks.
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads)
decode_join_kernel(const DecodeArgs p, const Parts parts) {
  __shared__ float4 red[kJoinThreads];
  __shared__ float red_m[kJoinThreads / 32], red_l[kJoinThreads];
  const int dh = p.dh, cols = dh / 4, tid = threadIdx.x;
  const int b = blockIdx.x / p.Hq;
  const Keys ks = visible_keys(p, b);
  if (ks.nk == 0) return;                          // written by chunk 0's block
  const int n = (ks.nk - 1) / parts.chunk + 1;
  const long long row = static_cast<long long>(blockIdx.x) * parts.chunks;
  float mm = -INFINITY;
  for (int c = tid; c < n; c += kJoinThreads) mm = fmaxf(mm, parts.ml[row + c].x);
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, x));
  if ((tid & 31) == 0) red_m[tid >> 5] = mm;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) mm = fmaxf(mm, red_m[w]);
  const int groups = kJoinThreads / cols, col = tid % cols, gr = tid / cols;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.0f;
  if (gr < groups) {
#pragma unroll 4
    for (int c = gr; c < n; c += groups) {
      const float2 ml = parts.ml[row + c];
      const float4 v = *reinterpret_cast<const float4 *>(parts.o + (row + c) * dh + col * 4);
      const float f = ml.y == 0.0f ? 0.0f : exp2f(ml.x - mm);
      l = fmaf(f, ml.y, l);
      a.x = fmaf(f, v.x, a.x);
      a.y = fmaf(f, v.y, a.y);
      a.z = fmaf(f, v.z, a.z);
      a.w = fmaf(f, v.w, a.w);
    }
  }
  red[tid] = a;
  red_l[tid] = l;
  __syncthreads();
  if (tid >= cols) return;
  for (int x = 1; x < groups; ++x) {
    const float4 v = red[x * cols + tid];
    a.x += v.x;
    a.y += v.y;
    a.z += v.z;
    a.w += v.w;
    l += red_l[x * cols + tid];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  T *o = static_cast<T *>(p.out) + static_cast<long long>(blockIdx.x) * dh + tid * 4;
  o[0] = from_f32<T>(a.x * inv);
  o[1] = from_f32<T>(a.y * inv);
  o[2] = from_f32<T>(a.z * inv);
  o[3] = from_f32<T>(a.w * inv);
}

// ------------------------------------------------------------------------- host

bool tensor_path(const DecodeArgs &p, int io) {
  return io == RGLRU_IO_BF16 && (p.dh == 64 || p.dh == 128 || p.dh == 256);
}

int slices_of(const DecodeArgs &p, int io) {
  return ceil_div(p.Hq / p.Hkv, tensor_path(p, io) ? 16 : kGenHeads);
}

// Keys of a chunk. More chunks fill the GPU and even out ragged sequences; each
// costs its block a start and an end (the chain length, page table, first keys,
// and the joining of its warps: about 3 us) and more than one costs the join (5
// us). The time of every number of chunks is estimated for sequences as long as
// their tables and window allow, in waves of resident blocks that share HBM (44
// bytes a ns and SM; 60 for an SM that runs beside idle ones), and the most chunks
// within 5 % of the best are taken: 128 sequences of 1028 visible 256-wide keys
// get one chunk (three took 47 us, one 31), 4 sequences of 131072 keys, ragged,
// get 74 rather than 37 (128 us, 146 with 37).
Parts parts_of(const DecodeArgs &p, int io) {
  const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
  long long most = cap;
  if (p.window > 0 && static_cast<long long>(p.window) + p.sinks < cap)
    most = static_cast<long long>(p.window) + p.sinks;
  const long long units = static_cast<long long>(p.B) * p.Hkv * slices_of(p, io);
  const int resident = !tensor_path(p, io) ? 1 : p.dh == 256 ? 1 : p.dh == 128 ? 2 : 4;
  const double slots = 148.0 * resident, key_bytes = 2.0 * p.dh * (io == RGLRU_IO_F32 ? 4 : 2);
  auto chunk_of = [&](long long chunks) { return ((most + chunks - 1) / chunks + 63) / 64 * 64; };
  auto time_of = [&](long long chunks) {               // ns
    const double blocks = static_cast<double>(units) * chunks;
    const double waves = ceil(blocks / slots);
    const double share = blocks < slots ? fmin(60.0, 44.0 * slots / blocks) : 44.0;
    return waves * (3000.0 + chunk_of(chunks) * key_bytes / (share / resident)) + (chunks > 1 ? 5000.0 : 0.0);
  };
  const long long limit = most / 128 > 1 ? (most / 128 < 1024 ? most / 128 : 1024) : 1;
  double best = time_of(1);
  for (long long c = 2; c <= limit; c += 1 + c / 16) best = fmin(best, time_of(c));
  long long chunks = 1;
  for (long long c = 1; c <= limit; c += 1 + c / 16)
    if (time_of(c) <= 1.05 * best) chunks = c;
  Parts r;
  r.o = nullptr;
  r.ml = nullptr;
  r.chunk = static_cast<int>(std::min(chunk_of(chunks), 1ll << 30));   // (offsets past its end stay below 2^31)
  r.chunks = static_cast<int>((most + r.chunk - 1) / r.chunk);
  return r;
}

template <int DH>
cudaError_t launch_tensor(const DecodeArgs &p, const Parts &parts, int slices, unsigned grid,
                          cudaStream_t st) {
  constexpr int smem = decode_smem<DH>();
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(paged_decode_kernel<DH>, smem, done);
  if (e != cudaSuccess) return e;
  paged_decode_kernel<DH><<<grid, kDecWarps * 32, smem, st>>>(p, parts, slices);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_generic(const DecodeArgs &p, const Parts &parts, int slices, unsigned grid,
                           cudaStream_t st) {
  const int smem = gen_layout(p.dh, sizeof(T)).total;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(paged_decode_generic_kernel<T>, kMaxSmem, done);
  if (e != cudaSuccess) return e;
  paged_decode_generic_kernel<T><<<grid, kGenThreads, smem, st>>>(p, parts, slices);
  return cudaGetLastError();
}

}  // namespace

size_t paged_decode_workspace_bytes(const DecodeArgs &p, int io) {
  const Parts parts = parts_of(p, io);
  if (parts.chunks == 1) return 0;
  const size_t rows = static_cast<size_t>(p.B) * p.Hq * parts.chunks;
  return rows * p.dh * sizeof(float) + rows * sizeof(float2);
}

cudaError_t launch_paged_decode(const DecodeArgs &p, int io, void *ws, cudaStream_t st) {
  Parts parts = parts_of(p, io);
  const int slices = slices_of(p, io);
  if (parts.chunks > 1) {
    const size_t rows = static_cast<size_t>(p.B) * p.Hq * parts.chunks;
    parts.o = static_cast<float *>(ws);
    parts.ml = reinterpret_cast<float2 *>(parts.o + rows * p.dh);
  }
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(parts.chunks) * p.B * p.Hkv * slices);
  cudaError_t e;
  if (tensor_path(p, io)) {
    if (p.dh == 64)
      e = launch_tensor<64>(p, parts, slices, grid, st);
    else if (p.dh == 128)
      e = launch_tensor<128>(p, parts, slices, grid, st);
    else
      e = launch_tensor<256>(p, parts, slices, grid, st);
  } else if (io == RGLRU_IO_F32) {
    e = launch_generic<float>(p, parts, slices, grid, st);
  } else {
    e = launch_generic<__nv_bfloat16>(p, parts, slices, grid, st);
  }
  if (e != cudaSuccess || parts.chunks == 1) return e;
  const unsigned rows = static_cast<unsigned>(p.B) * p.Hq;
  if (io == RGLRU_IO_F32)
    decode_join_kernel<float><<<rows, kJoinThreads, 0, st>>>(p, parts);
  else
    decode_join_kernel<__nv_bfloat16><<<rows, kJoinThreads, 0, st>>>(p, parts);
  return cudaGetLastError();
}

}  // namespace rglru
