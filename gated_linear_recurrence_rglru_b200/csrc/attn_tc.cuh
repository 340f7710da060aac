// What the tensor-core attention kernels share beside tc_primitives.cuh: 4-D
// TMA tile loads and their maps, packed fp32 pairs, 2^x, 32-byte stores, and
// the zeroing of rows that no query sees.
#pragma once

#include <cudaTypedefs.h>

#include <mutex>

#include "attn_kernels.h"
#include "attn_mask.cuh"
#include "common.cuh"
#include "tc_primitives.cuh"

namespace rglru {
namespace tc {

__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The warp's index, the same value in every lane by construction, so that what
// depends on it (an MMA warp's descriptors above all) stays in uniform registers.
__device__ __forceinline__ int warp_index() {
  return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x >> 5), 0);
}

// MMAs from descriptors split into words: within a tile only the address field
// (the low word, 16-byte units) changes, by 32-bit adds. `hi` is kDescHi with the
// SBO of 1024 bytes that all tiles here have; `lo` carries address and LBO.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return ((saddr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi)
      : "memory");
}

// A warp group's registers a thread from here on: more (N > 0) or fewer (N < 0).
template <int N> __device__ __forceinline__ void set_registers() {
  if constexpr (N > 0)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(-N));
}

// N threads of the softmax warps meet.
template <int N> __device__ __forceinline__ void bar_sync_softmax() {
  asm volatile("bar.sync 1, %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 consecutive TMEM columns of this thread's lane, as raw words.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// Waits for this thread's TMEM loads; v, one of them, counts as written here, so
// that nothing that reads it can be moved before the wait.
__device__ __forceinline__ void tmem_wait_ld32(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]),
                 "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}

// The same for 32 or 16 columns: load, wait, and store of their bf16 pairs.
__device__ __forceinline__ void tmem_wait_ld16(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]),
                 "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]),
                 "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
__device__ __forceinline__ void ld_cols(uint32_t t, float (&v)[32]) {
  tmem_ld32(t, v);
  tmem_wait_ld32(v);
}
__device__ __forceinline__ void ld_cols(uint32_t t, float (&v)[16]) {
  tmem_ld16(t, v);
  tmem_wait_ld16(v);
}
__device__ __forceinline__ void st_bf16(uint32_t t, const float (&v)[32]) {
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = bf16x2(v[2 * e], v[2 * e + 1]);
  tmem_st16u(t, w);
}
__device__ __forceinline__ void st_bf16(uint32_t t, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] = bf16x2(v[2 * e], v[2 * e + 1]);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
               "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// 2^x by the hardware's instruction (2 units in the last place, 0 for -inf).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Pairs of floats in one 64-bit register: one instruction for both.
__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b,
                                                   unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest; NaN if any is.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max2(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// 2^a, 2^b for a, b <= 127 on the FMA pipes: 2^x = 2^n 2^f with n the nearest whole
// number (read off the low bits of x + 1.5 * 2^23) and f in [-1/2, 1/2], 2^f by the
// polynomial of degree 4 of least relative error there (2.6e-6, by Remez exchange),
// times 2^n. Below -126 the result is 2^-126 to a factor of sqrt 2. For NaN it is NaN with
// kNaN; without, where n is added to the exponent's bits instead of one product more, it
// is the largest finite number, and the caller has to see to the NaN.
template <bool kNaN> __device__ __forceinline__ void ex2_pair(float &a, float &b) {
  constexpr float kMagic = 12582912.0f;
  const unsigned long long x = pair(max2(a, -126.0f), max2(b, -126.0f));
  const unsigned long long z = add2(x, pair(kMagic, kMagic));
  const unsigned long long n = add2(z, pair(-kMagic, -kMagic));
  const unsigned long long f = fma2(n, pair(-1.0f, -1.0f), x);
  unsigned long long r = fma2(f, pair(9.570101911e-03f, 9.570101911e-03f), pair(5.591786032e-02f, 5.591786032e-02f));
  r = fma2(r, f, pair(2.402474483e-01f, 2.402474483e-01f));
  r = fma2(r, f, pair(6.931218147e-01f, 6.931218147e-01f));
  r = fma2(r, f, pair(9.999992614e-01f, 9.999992614e-01f));
  float za, zb;
  unpair(z, za, zb);
  const int na = __float_as_int(za) << 23, nb = __float_as_int(zb) << 23;
  if constexpr (kNaN) {
    constexpr int kOne = 0x3F800000;
    unpair(mul2(r, pair(__int_as_float(na + kOne), __int_as_float(nb + kOne))), a, b);
  } else {
    unpair(r, a, b);
    a = __int_as_float(__float_as_int(a) + na);
    b = __int_as_float(__float_as_int(b) + nb);
  }
}

// N floats as bf16 (2 N bytes) at dst; v8: dst is 32-byte aligned.
template <int N>
__device__ __forceinline__ void store_row(__nv_bfloat16 *dst, const float (&v)[N], float f, bool v8) {
  uint32_t w[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) w[e] = bf16x2(v[2 * e] * f, v[2 * e + 1] * f);
  if (v8) {
#pragma unroll
    for (int q = 0; q < N / 16; ++q)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst + q * 16),
                   "r"(w[8 * q]), "r"(w[8 * q + 1]), "r"(w[8 * q + 2]), "r"(w[8 * q + 3]),
                   "r"(w[8 * q + 4]), "r"(w[8 * q + 5]), "r"(w[8 * q + 6]), "r"(w[8 * q + 7])
                   : "memory");
  } else {
#pragma unroll
    for (int q = 0; q < N / 8; ++q)
      reinterpret_cast<uint4 *>(dst)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
  }
}

// Bits lo .. hi (ends included, any values) of 32.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  const uint32_t upto = hi >= 31 ? 0xFFFFFFFFu : hi < 0 ? 0u : (2u << hi) - 1u;
  const uint32_t from = lo <= 0 ? 0xFFFFFFFFu : lo > 31 ? 0u : 0xFFFFFFFFu << lo;
  return upto & from;
}

// What has no bit set becomes `to`; nothing is done where all of a warp's have.
template <int N> __device__ __forceinline__ void hide(float (&v)[N], uint32_t bits, float to) {
  if (__all_sync(0xFFFFFFFFu, bits == 0xFFFFFFFFu)) return;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (!((bits >> e) & 1u)) v[e] = to;
}

// Keys that no query of the call sees: [sinks, dead_lo) and [nk, S). Their rows
// may hold anything, so a tile's rows among them are zeroed in shared memory
// (weight 0 times NaN would be NaN).
struct DeadKeys {
  int sinks, lo, nk, S;
  __device__ bool in(int j) const { return (j >= sinks && j < lo) || j >= nk; }
  __device__ bool any(int k0, int tile) const {
    return (k0 + tile > nk && nk < S) || max(k0, sinks) < min(k0 + tile, lo);
  }
};

__device__ __forceinline__ DeadKeys dead_keys(const AttnArgs &p, int nk) {
  return {p.sinks, p.window > 0 ? p.S - p.T - p.window + 1 : 0, nk, p.S};
}

// Map of a strided bf16 (B, T, H, dh) tensor as boxes of 64 columns x `rows`
// tokens of one head, 128-byte swizzle; rows past T read as zeros.
inline PFN_cuTensorMapEncodeTiled_v12000 attn_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

inline bool attn_map(CUtensorMap *m, const Strided &x, int B, int T, int H, int dh, int rows) {
  auto enc = attn_encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dh), static_cast<cuuint64_t>(T),
                              static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(x.st) * 2, static_cast<cuuint64_t>(x.sh) * 2,
                                 static_cast<cuuint64_t>(x.sb) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(x.p), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace tc
}  // namespace rglru
