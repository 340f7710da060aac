// Windowed attention with sinks on the 5th-generation tensor core, forward
// (include/rglru_attn.h), for bf16 heads 64, 128 or 256 wide.
//
//   S = Q K^T (128 queries x 128 keys), p = 2^(S c - m), c = scale log2 e,
//   l = l 2^(m - m') + sum p,  O = O 2^(m - m') + P V,  out = O / l
//
// One block takes 128 queries of one head and walks the key tiles that its mask
// leaves. Warps 0-7 are the softmax, thread = query row = TMEM lane, warp group
// g the columns 64 g ..: a row's maximum is one exchange through shared memory
// between two threads. Warp 8 issues the TMA copies (K and V through one ring of
// slots, 128 keys x up to 128 columns each, in the order of use), warp 9 the
// MMAs: S from shared memory (Q and K both K-major), P V with P as the TMEM
// operand (bf16, written over the scores it came from) and V MN-major as TMA
// left it. The accumulator O
// stays in TMEM for the whole walk; the reference maximum m moves only when it
// is 8 or more behind in log2 units (weights up to 2^8 keep their relative
// precision), so O is seldom rescaled.
//
// Heads 64 and 128 wide: one score buffer, 256 TMEM columns and under half the
// shared memory a block, so two blocks share an SM and one's softmax runs under
// the other's MMAs. 256 wide: O takes 256 columns; one block an SM with two
// score buffers, S of the next tile is made while the softmax works on this one.
// Only tiles that the mask cuts test it, element by element.
//
// Every wait is bounded; on expiry the kernel records RGLRU_ERR_TIMEOUT (wait
// site 7), drains what it issued and returns.
#include "attn_tc.cuh"

namespace rglru {
namespace {

using namespace tc;

constexpr int kBM = 128, kBN = 128;
constexpr int kThreads = 320;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kSite = 7;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;

template <int DH> struct Cfg {
  static constexpr int kCols = DH < 128 ? DH : 128;      // columns of a slot
  static constexpr int kPer = DH / kCols;                // slots of a tile
  static constexpr int kSlotBytes = kBN * kCols * 2;
  static constexpr int kSlots = DH == 256 ? 5 : DH == 128 ? 2 : 4;
  static constexpr int kNS = DH == 256 ? 2 : 1;          // score buffers
  static constexpr int kTmem = DH == 256 ? 512 : 256;
  static constexpr int kQBytes = kBM * DH * 2;
  static constexpr int kOffRing = kQBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
  static constexpr int kNumBars = 2 * kSlots + 1 + 2 * kNS + 2;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMax = kOffMisc + 16;            // [2][2 groups][128 rows]
  static constexpr int kSmem = kOffMax + 2 * 2 * kBM * 4;
  static constexpr int kBlocks = DH == 256 ? 1 : 2;      // per SM
  static constexpr bool kReread = kBlocks == 2;
};
static_assert(Cfg<256>::kSmem <= kMaxSmem && 2 * (Cfg<128>::kSmem + 1024) <= 233472, "shared memory");

struct Params {
  AttnArgs a;
  int n_qt;      // query tiles
  int v8;        // out rows may be stored 32 bytes at a time
  float c;       // scale * log2 e
};

template <int DH>
__global__ void __launch_bounds__(kThreads, Cfg<DH>::kBlocks)
attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ Params prm) {
  using C = Cfg<DH>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const AttnArgs &p = prm.a;
  if ((smem_u32(sm) & 1023u) != 0u) {
    if (threadIdx.x == 0 && p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_UNSUPPORTED);
    return;
  }
  // heads fastest (they share keys), then rows, then query tiles from the last
  // (the longest walks of an unwindowed causal mask start first)
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.Hq));
  const unsigned rest = blockIdx.x / static_cast<unsigned>(p.Hq);
  const int b = static_cast<int>(rest % static_cast<unsigned>(p.B));
  const int q0 = (prm.n_qt - 1 - static_cast<int>(rest / static_cast<unsigned>(p.B))) * kBM;
  const RowLens n = row_lens(p, b);
  if (q0 >= n.nq) return;
  const int off = p.S - p.T, kvh = h / (p.Hq / p.Hkv);
  const int q_last = min(q0 + kBM, n.nq) - 1;
  const KeyTiles kt = key_tiles(q0 + off, q_last + off, n.nk, p.window, p.sinks, kBN);
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
  if (kt.n == 0) {                                       // no query of the tile sees a key
    for (int i = tid; i < (q_last - q0 + 1) * (DH / 8); i += kThreads) {
      const int t = q0 + i / (DH / 8);
      reinterpret_cast<uint4 *>(out + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * DH)[i % (DH / 8)] =
          make_uint4(0u, 0u, 0u, 0u);
    }
    if (p.lse != nullptr)
      for (int i = tid; i <= q_last - q0; i += kThreads)
        p.lse[(static_cast<long long>(b) * p.Hq + h) * p.T + q0 + i] = -INFINITY;
    return;
  }

  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  uint64_t *empty = full + C::kSlots;
  uint64_t *q_full = empty + C::kSlots;
  uint64_t *s_full = q_full + 1;
  uint64_t *p_full = s_full + C::kNS;
  uint64_t *o_done = p_full + C::kNS;
  uint64_t *all_done = o_done + 1;                       // every MMA of the block
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::kOffMisc);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + C::kOffMisc + 4);
  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(q_full, 1);
    for (int s = 0; s < C::kNS; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 8);
    }
    mbar_init(o_done, 1);
    mbar_init(all_done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t t_o = tmem, t_s = tmem + DH;            // O, then the score buffers
  auto give_up = [&]() {
    if (!*abort) {
      if (p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_TIMEOUT | (kSite << 8) |
                                                       (static_cast<int>(blockIdx.x & 0x7FFFu) << 16));
      *abort = 1;
    }
  };

  // Slots in order of use: the K and V of tile i are fills at(i, is_v) ..+kPer-1.
  // One score buffer: K0 V0 K1 V1 ...; two: K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
  auto at = [&](int i, bool is_v) -> int {
    if (C::kNS == 1) return (2 * i + (is_v ? 1 : 0)) * C::kPer;
    if (!is_v) return (i == 0 ? 0 : 2 * i - 1) * C::kPer;
    return (i + 1 < kt.n ? 2 * i + 2 : 2 * i + 1) * C::kPer;
  };

  if (warp == 8) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      mbar_arrive_expect_tx(q_full, C::kQBytes);
      for (int c = 0; c < DH / 64; ++c)
        tma_load_4d(sm + c * (kBM * 128), &tmap_q, q_full, c * 64, q0, h, b);
      const int fills = 2 * kt.n * C::kPer;
      int f = 0;
      // walk K and V in the order of `at`
      int ik = 0, iv = 0;
      while (f < fills) {
        bool is_v;
        int i;
        if (ik < kt.n && at(ik, false) == f) {
          is_v = false;
          i = ik++;
        } else {
          is_v = true;
          i = iv++;
        }
        bool ok = true;
        for (int x = 0; x < C::kPer && ok; ++x, ++f) {
          const int s = f % C::kSlots;
          if (!mbar_wait(&empty[s], ((f / C::kSlots) & 1) ^ 1, abort, kWaitNs)) {
            give_up();
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], C::kSlotBytes);
          for (int c = 0; c < C::kCols / 64; ++c)
            tma_load_4d(sm + C::kOffRing + s * C::kSlotBytes + c * (kBN * 128),
                        is_v ? &tmap_v : &tmap_k, &full[s], x * C::kCols + c * 64, kt.tile(i) * kBN,
                        kvh, b);
        }
        if (!ok) break;
      }
      if (*abort) {
        mbar_wait_drain(q_full, 0, kDrainNs);
        for (int j = f - 1; j >= 0 && j >= f - C::kSlots; --j)
          mbar_wait_drain(&full[j % C::kSlots], (j / C::kSlots) & 1, kDrainNs);
      }
    }
  } else if (warp == 9) {
    // ============================= MMA issuer =============================
    // The whole warp walks, one elected lane issues.
    constexpr uint32_t id_s = idesc_bf16_f32(kBM, kBN, false, false);
    constexpr uint32_t id_o = idesc_bf16_f32(kBM, C::kCols, false, true);
    const uint32_t base = smem_u32(sm);
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok && !mbar_wait(bar, parity, abort, kWaitNs)) {
        give_up();
        ok = false;
      }
      if (ok) tc_fence_after();
      return ok;
    };
    auto scores = [&](int i) {
      const int f0 = at(i, false);
      const uint32_t d = t_s + (i % C::kNS) * kBN;
      for (int x = 0; x < C::kPer; ++x) {
        const int s = (f0 + x) % C::kSlots;
        if (!wait(&full[s], ((f0 + x) / C::kSlots) & 1)) return;
        const uint32_t ad = desc_lo(base + x * (C::kCols / 64) * (kBM * 128), 16);
        const uint32_t bd = desc_lo(base + C::kOffRing + s * C::kSlotBytes, 16);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < C::kCols / 16; ++k) {
            // a K step of 16 moves 32 bytes along the 128-byte row; 64-column
            // blocks lie 128 rows x 128 bytes apart
            const uint32_t o = ((k & 3) * 32 + (k >> 2) * (kBN * 128)) >> 4;
            mma_ss(d, ad + o, bd + o, id_s, k > 0 ? 1u : x > 0);
          }
          mma_commit(&empty[s]);
          if (x == C::kPer - 1) mma_commit(&s_full[i % C::kNS]);
        }
        __syncwarp();
      }
    };
    auto values = [&](int i) {
      if (!wait(&p_full[i % C::kNS], (i / C::kNS) & 1)) return;
      const int f0 = at(i, true);
      const uint32_t a = t_s + (i % C::kNS) * kBN;
      for (int x = 0; x < C::kPer; ++x) {
        const int s = (f0 + x) % C::kSlots;
        if (!wait(&full[s], ((f0 + x) / C::kSlots) & 1)) return;
        const uint32_t bd = desc_lo(base + C::kOffRing + s * C::kSlotBytes, kBN * 128);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kBN / 16; ++k)
            mma_ts(t_o + x * C::kCols, a + (k >> 2) * 64 + (k & 3) * 8, bd + ((k * 16 * 128) >> 4), id_o, k > 0 ? 1u : i > 0);
          mma_commit(&empty[s]);
          if (x == C::kPer - 1) mma_commit(o_done);
        }
        __syncwarp();
      }
    };
    wait(q_full, 0);
    if (ok) scores(0);
    for (int i = 0; i < kt.n && ok; ++i) {
      if (C::kNS == 2 && i + 1 < kt.n) scores(i + 1);
      if (ok) values(i);
      if (C::kNS == 1 && ok && i + 1 < kt.n) scores(i + 1);
    }
    if (elect_one()) mma_commit(all_done);
    if (*abort) mbar_wait_drain(all_done, 0, kDrainNs);
  } else {
    // =============================== softmax ==============================
    // Warp group g: columns 64 g .. of a tile. Thread = row = TMEM lane.
    const int g = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int pos = q0 + row + off;
    const DeadKeys dead = dead_keys(p, n.nk);
    float *shared_max = reinterpret_cast<float *>(sm + C::kOffMax);
    float m = -INFINITY, l = 0.0f;
    bool ok = true;                  // a warp whose wait expired still meets the block barriers
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok && !mbar_wait(bar, parity, abort, kWaitNs)) {
        give_up();
        ok = false;
      }
      if (ok) tc_fence_after();
      return ok;
    };
    for (int i = 0; i < kt.n; ++i) {
      const int s = i % C::kNS, k0 = kt.tile(i) * kBN;
      const uint32_t ts = t_s + s * kBN + g * 64 + lanes;
      // whether every query of the tile sees every key of the tile
      const bool whole = k0 + kBN - 1 <= min(q0 + off, n.nk - 1) &&
                         (p.window == 0 || k0 > q0 + kBM - 1 + off - p.window || k0 + kBN <= p.sinks);
      const int hi = min(pos, n.nk - 1) - k0;
      const int lo = p.window > 0 ? pos - p.window + 1 - k0 : -1, sk = p.sinks - k0;
      auto mask = [&](float (&v)[32], int c) {
        if (whole) return;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int j = g * 64 + c * 32 + e;
          if (!(j <= hi && (j >= lo || j < sk))) v[e] = -INFINITY;
        }
      };
      float v[2][32], mx[2] = {-INFINITY, -INFINITY};
      if (wait(&s_full[s], (i / C::kNS) & 1)) {
        // two blocks an SM leave a thread under 102 registers: the scores are read
        // 32 at a time, once for the maximum and once for the weights
        if constexpr (!C::kReread) {
          tmem_ld32(ts, v[0]);
          tmem_ld32(ts + 32, v[1]);
          tmem_wait_ld32(v[0]);
          tmem_wait_ld32(v[1]);
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float(&u)[32] = v[C::kReread ? 0 : x];
          if constexpr (C::kReread) {
            tmem_ld32(ts + x * 32, u);
            tmem_wait_ld32(u);
          }
          mask(u, x);
#pragma unroll
          for (int e = 0; e < 32; e += 2) mx[x] = max3(mx[x], u[e], u[e + 1]);
        }
      }
      const float mine = fmaxf(mx[0], mx[1]);
      shared_max[((i & 1) * 2 + g) * kBM + row] = mine;
      bar_sync_softmax();
      if (!ok) continue;
      const float top = fmaxf(mine, shared_max[((i & 1) * 2 + (g ^ 1)) * kBM + row]) * prm.c;
      const bool grow = top > m + kSlack || m == -INFINITY;
      const float mn = grow ? fmaxf(top, m) : m;
      if (__any_sync(0xFFFFFFFFu, mn != m)) {
        const float f = m == -INFINITY ? 0.0f : ex2(m - mn);
        l *= f;
        m = mn;
        if (i > 0 && wait(o_done, (i - 1) & 1)) {        // O so far: P V of the last tile is done
#pragma unroll 1
          for (int c = 0; c < DH / 64; ++c) {
            const uint32_t to = t_o + lanes + g * (DH / 2) + c * 32;
            float o[32];
            tmem_ld32(to, o);
            tmem_wait_ld32(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= f;
            tmem_st32(to, o);
          }
          tmem_wait_st();
        }
        if (!ok) continue;
      }
      const float base = m == -INFINITY ? 0.0f : m;
      const unsigned long long cc = pair(prm.c, prm.c), mm = pair(-base, -base);
      unsigned long long sum[2] = {0ull, 0ull};
      // the weights of this group's columns go to the first half of its score columns
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float(&u)[32] = v[C::kReread ? 0 : c];
        if constexpr (C::kReread) {
          tmem_ld32(ts + c * 32, u);
          tmem_wait_ld32(u);
          mask(u, c);
        }
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          float a, bb;
          unpair(fma2(pair(u[e], u[e + 1]), cc, mm), a, bb);
          a = ex2(a);
          bb = ex2(bb);
          sum[(e >> 1) & 1] = add2(sum[(e >> 1) & 1], pair(a, bb));
          w[e / 2] = bf16x2(a, bb);
        }
        tmem_st16u(ts + c * 16, w);
      }
      float s0, s1;
      unpair(add2(sum[0], sum[1]), s0, s1);
      l += s0 + s1;
      if (dead.any(k0, kBN)) {
        // zero the value rows that no query sees, once V is there
        const int f0 = at(i, true);
        for (int x = 0; x < C::kPer; ++x) {
          const int sl = (f0 + x) % C::kSlots;
          if (wait(&full[sl], ((f0 + x) / C::kSlots) & 1) && g == 0 && dead.in(k0 + row))
            for (int c = 0; c < C::kCols / 64; ++c)
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4 *>(sm + C::kOffRing + sl * C::kSlotBytes + c * (kBN * 128) +
                                           row * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[s]);
    }
    // the row's sum, from both groups
    shared_max[((kt.n & 1) * 2 + g) * kBM + row] = l;
    bar_sync_softmax();
    l += shared_max[((kt.n & 1) * 2 + (g ^ 1)) * kBM + row];
    if (wait(all_done, 0)) {
      const int t = q0 + row;
      const bool live = t < n.nq;
      const float inv = m == -INFINITY ? 0.0f : 1.0f / l;
      __nv_bfloat16 *dst = out + ((static_cast<long long>(b) * p.T + t) * p.Hq + h) * DH + g * (DH / 2);
#pragma unroll 1
      for (int c = 0; c < DH / 64; ++c) {
        float o[32];
        tmem_ld32(t_o + lanes + g * (DH / 2) + c * 32, o);
        tmem_wait_ld32(o);
        if (live) {
          if (m == -INFINITY) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0.0f;
          }
          store_row32(dst + c * 32, o, inv, prm.v8 != 0);
        }
      }
      if (live && g == 0 && p.lse != nullptr)
        p.lse[(static_cast<long long>(b) * p.Hq + h) * p.T + t] =
            m == -INFINITY ? -INFINITY : m * kLn2 + logf(l);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, C::kTmem);
}

template <int DH> cudaError_t launch(const AttnArgs &p, cudaStream_t st) {
  using C = Cfg<DH>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(attn_fwd_tc_kernel<DH>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!attn_map(&mq, p.q, p.B, p.T, p.Hq, DH, kBM) || !attn_map(&mk, p.k, p.B, p.S, p.Hkv, DH, kBN) ||
      !attn_map(&mv, p.v, p.B, p.S, p.Hkv, DH, kBN))
    return cudaErrorInvalidValue;
  Params prm;
  prm.a = p;
  prm.n_qt = ceil_div(p.T, kBM);
  prm.v8 = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0 ? 1 : 0;
  prm.c = p.scale * kLog2e;
  const unsigned grid = static_cast<unsigned>(static_cast<long long>(prm.n_qt) * p.B * p.Hq);
  attn_fwd_tc_kernel<DH><<<grid, kThreads, C::kSmem, st>>>(mq, mk, mv, prm);
  return cudaGetLastError();
}

}  // namespace

bool attn_tc_supported(const AttnArgs &p, int io) {
  return io == RGLRU_IO_BF16 && (p.dh == 64 || p.dh == 128 || p.dh == 256);
}

cudaError_t launch_attn_fwd_tc(const AttnArgs &p, cudaStream_t st) {
  switch (p.dh) {
    case 64: return launch<64>(p, st);
    case 128: return launch<128>(p, st);
    default: return launch<256>(p, st);
  }
}

}  // namespace rglru
