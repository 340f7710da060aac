// Windowed attention with sinks on the 5th-generation tensor core, forward
// (include/rglru_attn.h), for bf16 heads 64, 128 or 256 wide.
//
//   S = Q K^T (128 queries x 128 keys), p = 2^(S c - m), c = scale log2 e,
//   l = l 2^(m - m') + sum p,  O = O 2^(m - m') + P V,  out = O / l
//
// Blocks are resident, one an SM, and take unit after unit: 128-query tiles of a
// head and the key tiles that their mask leaves, the next unit's copies and first
// scores running while the softmax warps store the last one's rows. Heads 64 and
// 128 wide: a block works on two query tiles at once, which share every K and V
// tile (two heads of a group, or two tiles of one head): while the softmax works on
// one's scores, the tensor core does the other's P V and next S. 256 wide: one query
// tile (O takes 256 TMEM columns) with two score buffers, S of the next key tile is
// made while the softmax works on this one. Where units would leave SMs idle, a
// cluster of blocks shares a unit's key tiles (join).
//
// Eight softmax warps, thread = query row = TMEM lane: with two query tiles a thread
// has all 128 scores of its row and key tile in registers (16 warps with half a row
// each: 25 % slower, for the exchange of the maximum and the spills); with one, two
// warp groups share the columns, and a row's maximum is one exchange through shared
// memory between two threads. One warp issues the TMA copies (K and V through one
// ring of slots, 128 keys x up to 128 columns each, in the order of use), one or two
// the MMAs: S from shared memory (Q and K both K-major), P V with P as the TMEM
// operand (bf16, written over the scores it came from, or, 64 wide, to columns of its
// own) and V MN-major as TMA left it. Weights are handed over in halves, so that P V
// starts while the second half is formed. The accumulator O stays in TMEM for a unit's
// whole walk; the reference maximum m moves only when it is 8 or more behind in log2
// units (weights up to 2^8 keep their relative precision), so O is seldom rescaled.
// Where the mask cuts a tile, the keys that a row sees are bits, and only warps that
// have a hidden one apply them. Weights are rounded to bf16 for the product with V, as
// its operand has to be, and summed before that.
//
// Bound by the way round from scores to weights and back, of which a query tile's
// softmax is half: 8192 tokens, 16/4 heads of 128, window 2048, take 128 us (940
// TFLOP/s, the tensor pipe half busy); 4 x 2048 tokens, 10 query heads on one 256-wide
// key head, window 1024, 72 us (890 TFLOP/s); short windows of ragged rows (5 x 777, 16
// heads of 64, window 256) 27 us, half of it the starts and ends of units.
//
// Every wait is bounded; on expiry the kernel records RGLRU_ERR_TIMEOUT (wait
// site 7), drains what it issued and returns.
#include "attn_cluster.cuh"
#include "attn_tc.cuh"

namespace rglru {
namespace {

using namespace tc;

constexpr int kBM = 128, kBN = 128;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kSite = 7;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;
constexpr int kLeast = 2;                                // key tiles of a part of a unit

template <int DH> struct Cfg {
  static constexpr int kNQ = DH == 256 ? 1 : 2;          // query tiles of a block
  static constexpr int kNS = DH == 256 ? 2 : 1;          // score buffers of a query tile
  static constexpr bool kApart = DH == 64;               // weights in columns of their own
  static constexpr bool kAhead = kNS == 2 || kApart;     // S of a tile before P V of the last
  static constexpr int kIssuers = DH == 64 ? 2 : 1;      // warps that issue MMAs
  static constexpr int kCols = DH < 128 ? DH : 128;      // columns of a slot
  static constexpr int kPer = DH / kCols;                // slots of a tile
  static constexpr int kSlotBytes = kBN * kCols * 2;
  static constexpr int kSlots = DH == 64 ? 8 : 5;
  static constexpr int kQBytes = kBM * DH * 2;           // of one query tile
  static constexpr int kPoly = 2;                        // of 16 pairs of scores (weights32)
  static constexpr int kG = kNQ == 2 ? 1 : 2;            // warp groups that share a tile's columns
  static constexpr int kSoftmax = 8;                     // softmax warps
  static constexpr int kThreads = (kSoftmax + 4) * 32;   // whole warp groups, for the register split
  static constexpr int kOffRing = kNQ * kQBytes;
  static constexpr int kOffBar = kOffRing + kSlots * kSlotBytes;
  static constexpr int kNumBars = 2 * kSlots + kNQ * (3 * kNS + 6) + 1;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffMax = kOffMisc + 16;          // [2][2 groups][128 rows]
  static constexpr int kSmem = kOffMax + (kG == 2 ? 2 * 2 * kBM * 4 : 0);
  static constexpr int kOffS = kNQ * DH;                 // TMEM columns: O, scores, weights
  static constexpr int kOffP = kOffS + kNQ * kNS * kBN;
  static_assert(kSmem <= kMaxSmem && kOffP + (kApart ? kNQ * kBN / 2 : 0) <= 512, "shared memory, TMEM");
};

// The largest of N x 32 scores, in four chains; NaN if any is.
template <int N> __device__ __forceinline__ float max_of(const float (&v)[N][32]) {
  float m[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) m[x] = max2(v[0][2 * x], v[0][2 * x + 1]);
#pragma unroll
  for (int c = 0; c < N; ++c)
#pragma unroll
    for (int e = c == 0 ? 8 : 0; e < 32; e += 2) m[(e >> 1) & 3] = max3(m[(e >> 1) & 3], v[c][e], v[c][e + 1]);
  return max2(max3(m[0], m[1], m[2]), m[3]);
}

// 32 scores of a row to weights 2^(v c - m), packed as bf16; sum gains them. kPoly
// of the 16 pairs go by ex2_pair: the hardware's 2^x gives 16 results a cycle and
// SM, as long for a tile of 128 x 128 scores as the tensor core needs for a 128-wide
// head, while the FMA pipes have room (8192 tokens, 16/4 heads of 128: 131 us with none
// of them, 128 with 2, 129 with 4, 136 with 8; with 2 that keep a NaN, 131). A NaN among
// the scores makes m NaN (softmax warps), so that the hardware's results, and with them
// the row's sum and product, are NaN.
template <int kPoly>
__device__ __forceinline__ void weights32(const float (&v)[32], unsigned long long cc,
                                          unsigned long long mm, unsigned long long (&sum)[2],
                                          uint32_t (&packed)[16]) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float a, b;
    unpair(fma2(pair(v[2 * e], v[2 * e + 1]), cc, mm), a, b);
    if ((e * kPoly) % 16 < kPoly) {                       // spread evenly
      ex2_pair<false>(a, b);
    } else {
      a = ex2(a);
      b = ex2(b);
    }
    sum[e & 1] = add2(sum[e & 1], pair(a, b));
    packed[e] = bf16x2(a, b);
  }
}

struct Params {
  AttnArgs a;
  int n_qt;        // query tiles of a row; pairs of them when `rows2`
  unsigned n_h;    // heads of a row; pairs of them when a block's two tiles are two heads
  int rows2;       // a block's two query tiles follow each other in one head
  unsigned units;
  int parts;       // blocks of a cluster that share a unit's key tiles (kSplit)
  int v8;          // out rows may be stored 32 bytes at a time
  float c;         // scale * log2 e
};

// One unit of work: a block's query tiles (128 queries of one head each) and the
// key tiles that any of them sees. Two tiles are two heads that share keys, or,
// where heads are odd in a group, two tiles of one head. Heads fastest (they share
// keys), then rows, then query tiles from the last (the longest walks of an
// unwindowed causal mask come first).
// kSplit: the part-th of prm.parts shares of the unit's key tiles.
template <int NQ, bool kSplit> struct Unit {
  int h, b, q0, rows2, first_tile;
  RowLens n;
  KeyTiles kt;
  __device__ Unit(const Params &prm, unsigned u) {
    const AttnArgs &p = prm.a;
    rows2 = NQ == 2 ? prm.rows2 : 0;
    const unsigned rest = u / prm.n_h, far = rest / static_cast<unsigned>(p.B);
    h = static_cast<int>(u - rest * prm.n_h) * (NQ == 2 && !rows2 ? 2 : 1);
    b = static_cast<int>(rest - far * static_cast<unsigned>(p.B));
    q0 = (prm.n_qt - 1 - static_cast<int>(far)) * kBM * (1 + rows2);
    n = row_lens(p, b);
    kt = {0, 0, 0};
    if (q0 < n.nq)
      kt = key_tiles(q0 + p.S - p.T, min(q0 + kBM * (1 + rows2), n.nq) - 1 + p.S - p.T, n.nk, p.window,
                     p.sinks, kBN);
    if constexpr (kSplit) {
      const int part = static_cast<int>(blockIdx.x) % prm.parts;
      first_tile = kt.n * part / prm.parts;
      kt.n = kt.n * (part + 1) / prm.parts - first_tile;
      kt.win += max(first_tile - kt.sink_end, 0);
      kt.sink_end = max(kt.sink_end - first_tile, 0);
    }
  }
  __device__ int tile(int i) const { return (kSplit && i < kt.sink_end ? first_tile : 0) + kt.tile(i); }
  __device__ int head(int q) const { return h + (NQ == 2 && !rows2 ? q : 0); }
  __device__ int first(int q) const { return q0 + (NQ == 2 && rows2 ? q * kBM : 0); }
  // whether any query of tile q sees any key of key tile i
  __device__ bool sees(const AttnArgs &p, int q, int i) const {
    if (NQ == 1 || !rows2) return true;
    const int f = first(q), off = p.S - p.T, k0 = tile(i) * kBN;
    return f < n.nq && k0 <= min(f + kBM, n.nq) - 1 + off &&
           (p.window == 0 || k0 + kBN - 1 > f + off - p.window || k0 < p.sinks);
  }
  // the last key tile that tile q sees, or -1
  __device__ int last(const AttnArgs &p, int q) const {
    if (NQ == 1 || !rows2) return kt.n - 1;
    const int f = first(q), hi = min(min(f + kBM, n.nq) - 1 + p.S - p.T, n.nk - 1);
    if (f >= n.nq || hi < 0) return -1;
    if constexpr (kSplit) {
      int x = kt.n - 1;
      while (x >= 0 && !sees(p, q, x)) --x;
      return x;
    }
    const int x = hi / kBN;
    return x < kt.win ? x : kt.sink_end + x - kt.win;
  }
};

// The block's r-th unit: units come sorted by length, and every second round runs
// backwards over the blocks, so that their sums stay close.
template <bool kSplit> __device__ __forceinline__ unsigned unit_at(const Params &prm, unsigned r) {
  if (kSplit) return r == 0 ? blockIdx.x / static_cast<unsigned>(prm.parts) : prm.units;
  return r * gridDim.x + ((r & 1u) ? gridDim.x - 1u - blockIdx.x : blockIdx.x);
}

// Ring fills of a unit in order of use: the K and V of tile i are fills
// fill_of(i, is_v) .. + kPer - 1. K0 V0 K1 V1 ..., or, with the next scores ahead,
// K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
template <int DH> __device__ __forceinline__ int fill_of(int i, bool is_v, int n) {
  using C = Cfg<DH>;
  if (!C::kAhead) return (2 * i + (is_v ? 1 : 0)) * C::kPer;
  if (!is_v) return (i == 0 ? 0 : 2 * i - 1) * C::kPer;
  return (i + 1 < n ? 2 * i + 2 : 2 * i + 1) * C::kPer;
}

// The parts of a split unit to its rows: every block of the cluster leaves O (not
// divided yet), m and l of its keys in its shared memory, where the operands were, and
// each joins its share of the rows (half of them at most) from all.
template <int DH, typename Un>
__device__ __forceinline__ void join(const Params &prm, const Un &un, uint32_t t_o, bool some, int q, int g,
                                     int row, float m, float l, unsigned char *sm) {
  using C = Cfg<DH>;
  constexpr int kPitch = DH + 4, kOut = DH / C::kG, kRows = C::kNQ * kBM;
  static_assert(kRows * (kPitch + 2 + 4) * 4 <= C::kOffBar, "the parts' room");
  const AttnArgs &p = prm.a;
  float *part = reinterpret_cast<float *>(sm), *ml = part + kRows * kPitch, *fs = ml + 2 * kRows;
  asm volatile("bar.sync 2, 256;" ::: "memory");         // no product of the block reads its operands now
  const int at = q * kBM + row;
  if (some) {
#pragma unroll 1
    for (int c = 0; c < kOut; c += 32) {
      float o[32];
      tmem_ld32(t_o + c, o);
      tmem_wait_ld32(o);
#pragma unroll
      for (int e = 0; e < 32; e += 4)
        *reinterpret_cast<float4 *>(part + at * kPitch + g * kOut + c + e) =
            make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
  }
  // (m = -inf: no key seen, or none with a score above -inf)
  if (g == 0) *reinterpret_cast<float2 *>(ml + 2 * at) = make_float2(m, some && m != -INFINITY ? l : 0.0f);
  cluster_sync();
  const int tid = threadIdx.x, parts = prm.parts, share = kRows / parts;
  const int x0 = static_cast<int>(cluster_ctarank()) * share;            // this block's rows
  const uint32_t mine = smem_u32(part);
  if (tid < share) {                                     // f_i / L of a row
    const int x = x0 + tid, y = x / kBM, t = un.first(y) + x % kBM;
    float f[8], top, sum;
    join_factors<true>(mine + (kRows * kPitch + 2 * x) * 4, parts, f, top, sum);
#pragma unroll
    for (int i = 0; i < 8; ++i) fs[tid * 8 + i] = f[i];
    if (t < un.n.nq && p.lse != nullptr)
      p.lse[(static_cast<long long>(un.b) * p.Hq + un.head(y)) * p.T + t] =
          sum == 0.0f ? -INFINITY : top * kLn2 + logf(sum);
  }
  asm volatile("bar.sync 2, 256;" ::: "memory");
  constexpr int kV = DH / 4, kN = 4;                     // 16-byte pieces of a row; at once of a thread
  for (int z = tid; z < share * kV; z += 256 * kN) {
    float4 acc[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) acc[e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int i = 0; i < parts; ++i) {
      const uint32_t from = mapa_shared(mine, i);
      float4 o[kN];
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const int w = min(z + e * 256, share * kV - 1);
        o[e] = ld_cluster4(from + ((x0 + w / kV) * kPitch + w % kV * 4) * 4);
      }
#pragma unroll
      for (int e = 0; e < kN; ++e) {
        const float f = fs[min(z + e * 256, share * kV - 1) / kV * 8 + i];
        if (f != 0.0f) {                                 // (else what lies there may not be O)
          acc[e].x = fmaf(o[e].x, f, acc[e].x);
          acc[e].y = fmaf(o[e].y, f, acc[e].y);
          acc[e].z = fmaf(o[e].z, f, acc[e].z);
          acc[e].w = fmaf(o[e].w, f, acc[e].w);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      const int w = z + e * 256, x = x0 + w / kV, y = x / kBM, t = un.first(y) + x % kBM;
      if (w < share * kV && t < un.n.nq)
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) +
                                   ((static_cast<long long>(un.b) * p.T + t) * p.Hq + un.head(y)) * DH +
                                   w % kV * 4) = make_uint2(bf16x2(acc[e].x, acc[e].y), bf16x2(acc[e].z, acc[e].w));
    }
  }
  cluster_sync();                                        // the others have read this block's part
}

template <int DH, bool kSplit>
__global__ void __launch_bounds__(Cfg<DH>::kThreads, 1)
attn_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ Params prm) {
  using C = Cfg<DH>;
  using Un = Unit<C::kNQ, kSplit>;
  constexpr int kTma = C::kSoftmax, kMma = C::kSoftmax + 1;       // warps
  extern __shared__ __align__(1024) unsigned char sm[];
  const AttnArgs &p = prm.a;
  if ((smem_u32(sm) & 1023u) != 0u) {
    if (threadIdx.x == 0 && p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_UNSUPPORTED);
    return;
  }
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int off = p.S - p.T;
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  uint64_t *empty = full + C::kSlots;
  uint64_t *q_full = empty + C::kSlots, *q_empty = q_full + C::kNQ;      // [kNQ]
  uint64_t *s_full = q_empty + C::kNQ;                   // [kNQ][kNS]
  uint64_t *p_full = s_full + C::kNQ * C::kNS;           // [halves][kNQ][kNS]
  uint64_t *o_done = p_full + 2 * C::kNQ * C::kNS;       // [kNQ] a tile's P V
  uint64_t *all_done = o_done + C::kNQ;                  // [kNQ] a unit's last P V
  uint64_t *o_free = all_done + C::kNQ;                  // [kNQ] a unit's O was read
  uint64_t *s_free = o_free + C::kNQ;                    // [kNQ] scores apart from weights were read
  uint64_t *drained = s_free + C::kNQ;                   // used when a wait expired
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::kOffMisc);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + C::kOffMisc + 4);
  if (tid == 0) {
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], C::kIssuers);
    }
    mbar_init(drained, C::kIssuers);
    for (int s = 0; s < C::kNQ * C::kNS; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], 4 * C::kG);
      mbar_init(&p_full[C::kNQ * C::kNS + s], 4 * C::kG);
    }
    for (int q = 0; q < C::kNQ; ++q) {
      mbar_init(&q_full[q], 1);
      mbar_init(&q_empty[q], 1);
      mbar_init(&o_done[q], 1);
      mbar_init(&all_done[q], 1);
      mbar_init(&o_free[q], 4 * C::kG);
      mbar_init(&s_free[q], 4 * C::kG);
    }
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kMma) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;                      // O of each query tile, then the scores
  auto give_up = [&]() {
    if (!*abort) {
      if (p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_TIMEOUT | (kSite << 8) |
                                                       (static_cast<int>(blockIdx.x & 0x7FFFu) << 16));
      *abort = 1;
    }
  };

  // The block is launched with 168 registers a thread (12 warps); the copy and MMA
  // warps give up some of theirs to the softmax warps: 8 x 208 + 4 x 88 = 12 x 168.
  if (warp >= kTma) {
    set_registers<-88>();
    if (warp == kTma) {
      // ============================ TMA producer ============================
      if (lane == 0) {
        int f = 0, nu[2] = {0, 0};                         // fills and query tiles issued
        bool ok = true;
        for (unsigned r = 0, u; (u = unit_at<kSplit>(prm, r)) < prm.units && ok; ++r) {
          const Un un(prm, u);
          if (un.kt.n == 0) continue;
          const int kvh = un.h / (p.Hq / p.Hkv);
          const int fills = 2 * un.kt.n * C::kPer;
          // K and V tiles in the order of fill_of; Q after the first of them, which
          // may come while the last unit still uses its Q
          int ik = 0, iv = 0;
          for (int g = 0; g < fills && ok;) {
            const bool is_v = !(ik < un.kt.n && fill_of<DH>(ik, false, un.kt.n) == g);
            const int i = is_v ? iv++ : ik++;
            for (int x = 0; x < C::kPer && ok; ++x, ++g, ++f) {
              const int s = f % C::kSlots;
              if (!mbar_wait(&empty[s], ((f / C::kSlots) & 1) ^ 1, abort, kWaitNs)) {
                give_up();
                ok = false;
                break;
              }
              mbar_arrive_expect_tx(&full[s], C::kSlotBytes);
              for (int c = 0; c < C::kCols / 64; ++c)
                tma_load_4d(sm + C::kOffRing + s * C::kSlotBytes + c * (kBN * 128), is_v ? &tmap_v : &tmap_k,
                            &full[s], x * C::kCols + c * 64, un.tile(i) * kBN, kvh, un.b);
            }
            if (ok && !is_v && i == 0) {
              for (int q = 0; q < C::kNQ && ok; ++q) {
                if (!mbar_wait(&q_empty[q], (nu[q] & 1) ^ 1, abort, kWaitNs)) {
                  give_up();
                  ok = false;
                  break;
                }
                mbar_arrive_expect_tx(&q_full[q], C::kQBytes);
                for (int c = 0; c < DH / 64; ++c)
                  tma_load_4d(sm + q * C::kQBytes + c * (kBM * 128), &tmap_q, &q_full[q], c * 64, un.first(q),
                              un.head(q), un.b);
                ++nu[q];
              }
            }
          }
        }
        if (*abort) {
          for (int q = 0; q < C::kNQ; ++q)
            if (nu[q] > 0) mbar_wait_drain(&q_full[q], (nu[q] - 1) & 1, kDrainNs);
          for (int j = f - 1; j >= 0 && j >= f - C::kSlots; --j)
            mbar_wait_drain(&full[j % C::kSlots], (j / C::kSlots) & 1, kDrainNs);
        }
      }
    } else if (warp < kMma + C::kIssuers) {
      // ============================ MMA issuers =============================
      // The whole warp walks, one elected lane issues. 64 wide, where the softmax
      // takes longer than the tensor core, each query tile has a warp of its own, so
      // that neither waits for the other's (batch of short windows: 31 -> 27 us). 128
      // wide, one warp takes turns with the two: on their own, both would want the
      // tensor core at once and the softmax units at once (128 -> 153 us on 8192
      // tokens, 16 heads).
      constexpr int kMine = C::kNQ / C::kIssuers;          // query tiles of this warp
      constexpr uint32_t id_s = idesc_bf16_f32(kBM, kBN, false, false);
      constexpr uint32_t id_o = idesc_bf16_f32(kBM, C::kCols, false, true);
      const uint32_t base = smem_u32(sm);
      const int first_q = warp - kMma;
      bool ok = true;
      int f0 = 0, units = 0;                               // fills and units before this unit
      int js[kMine] = {}, jp[kMine] = {}, nu[kMine] = {};  // tiles scored, tiles added, units with a key
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (ok && !mbar_wait(bar, parity, abort, kWaitNs)) {
          give_up();
          ok = false;
        }
        if (ok) tc_fence_after();
        return ok;
      };
      // a tile that this warp's query tiles do not see: its slots are the other warp's alone
      auto pass = [&](int f) {
        for (int x = 0; kMine == 1 && x < C::kPer; ++x) {  // (of two, one sees it)
          const int s = (f + x) % C::kSlots;
          if (!wait(&full[s], ((f + x) / C::kSlots) & 1)) return;
          if (elect_one()) mbar_arrive(&empty[s]);
          __syncwarp();
        }
      };
      // S of key tile i; `last`: Q has no later reader; `free`: nor has K, of this warp
      auto scores = [&](const Un &un, int y, int i, bool last, bool free) {
        const int q = first_q + y;
        const int f = f0 + fill_of<DH>(i, false, un.kt.n), sb = q * C::kNS + js[y] % C::kNS;
        const uint32_t d = tmem + C::kOffS + sb * kBN;
        if (C::kApart && js[y] > 0 && !wait(&s_free[q], (js[y] - 1) & 1)) return;
        for (int x = 0; x < C::kPer; ++x) {
          const int s = (f + x) % C::kSlots;
          if (!wait(&full[s], ((f + x) / C::kSlots) & 1)) return;
          const uint32_t ad = desc_lo(base + q * C::kQBytes + x * (C::kCols / 64) * (kBM * 128), 16);
          const uint32_t bd = desc_lo(base + C::kOffRing + s * C::kSlotBytes, 16);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < C::kCols / 16; ++k) {
              // a K step of 16 moves 32 bytes along the 128-byte row; 64-column
              // blocks lie 128 rows x 128 bytes apart
              const uint32_t o = ((k & 3) * 32 + (k >> 2) * (kBN * 128)) >> 4;
              mma_ss(d, ad + o, bd + o, id_s, k > 0 ? 1u : x > 0);
            }
            if (free) mma_commit(&empty[s]);
            if (x == C::kPer - 1) {
              mma_commit(&s_full[sb]);
              if (last) mma_commit(&q_empty[q]);
            }
          }
          __syncwarp();
        }
        ++js[y];
      };
      // O gains P V of key tile i, in the two halves in which the softmax warps hand
      // the weights over; `first`, `done`: of the unit
      auto values = [&](const Un &un, int y, int i, bool first, bool done, bool free) {
        const int q = first_q + y;
        const int f = f0 + fill_of<DH>(i, true, un.kt.n), sb = q * C::kNS + jp[y] % C::kNS;
        const uint32_t a = tmem + (C::kApart ? C::kOffP + q * (kBN / 2) : C::kOffS + sb * kBN);
        if (first && nu[y] > 0 && !wait(&o_free[q], (nu[y] - 1) & 1)) return;
        for (int x = 0; x < C::kPer; ++x)
          if (!wait(&full[(f + x) % C::kSlots], ((f + x) / C::kSlots) & 1)) return;
        for (int half = 0; half < 2; ++half) {
          if (!wait(&p_full[half * C::kNQ * C::kNS + sb], (jp[y] / C::kNS) & 1)) return;
          for (int x = 0; x < C::kPer; ++x) {
            const int s = (f + x) % C::kSlots;
            const uint32_t bd = desc_lo(base + C::kOffRing + s * C::kSlotBytes, kBN * 128);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kBN / 32; ++k) {
                // the first half of each group's columns, then the second
                const int ks = C::kG == 2 ? (k >> 1) * 4 + half * 2 + (k & 1) : half * 4 + k;
                mma_ts(tmem + q * DH + x * C::kCols, a + (C::kG == 2 ? (ks >> 2) * 64 + (ks & 3) * 8 : ks * 8),
                       bd + ((ks * 16 * 128) >> 4), id_o, half + k > 0 ? 1u : !first);
              }
              if (half == 1) {
                if (free) mma_commit(&empty[s]);
                if (x == C::kPer - 1) {
                  mma_commit(&o_done[q]);
                  if (done) mma_commit(&all_done[q]);
                }
              }
            }
            __syncwarp();
          }
        }
        ++jp[y];
      };
      for (unsigned r = 0, u; (u = unit_at<kSplit>(prm, r)) < prm.units && ok; ++r) {
        const Un un(prm, u);
        const int n = un.kt.n;
        if (n == 0) continue;
        int end[kMine];                                    // the last tile that each sees
        bool begun[kMine] = {};
#pragma unroll
        for (int y = 0; y < kMine; ++y) {
          wait(&q_full[first_q + y], units & 1);
          end[y] = un.last(p, first_q + y);
          if (end[y] < 0 && ok) {                          // none: Q is not read
            if (elect_one()) mbar_arrive(&q_empty[first_q + y]);
            __syncwarp();
          }
        }
        ++units;
        auto next = [&](int y, int i) {
          if (!ok || i >= n) return;
          if (un.sees(p, first_q + y, i)) scores(un, y, i, i == end[y], y == kMine - 1 || !un.sees(p, kMine - 1, i));
          else pass(f0 + fill_of<DH>(i, false, n));
        };
        for (int i = -1; i < n && ok; ++i) {
#pragma unroll
          for (int y = 0; y < kMine; ++y) {
            if (C::kAhead) next(y, i + 1);
            if (ok && i >= 0) {
              if (un.sees(p, first_q + y, i)) {
                values(un, y, i, !begun[y], i == end[y], y == kMine - 1 || !un.sees(p, kMine - 1, i));
                begun[y] = true;
              } else {
                pass(f0 + fill_of<DH>(i, true, n));
              }
            }
            if (!C::kAhead) next(y, i + 1);
          }
        }
#pragma unroll
        for (int y = 0; y < kMine; ++y) nu[y] += begun[y] ? 1 : 0;
        f0 += 2 * n * C::kPer;
      }
      if (*abort) {                                        // let what was issued finish
        if (elect_one()) mma_commit(drained);
        mbar_wait_drain(drained, 0, kDrainNs);
      }
    }
  } else {
    set_registers<208>();
    // =============================== softmax ==============================
    // Thread = row = TMEM lane, and kCols of a key tile's columns: all 128, or, one
    // query tile a block, half of them (warp group g).
    constexpr int kCols = kBN / C::kG, kOut = DH / C::kG;
    const int q = C::kNQ == 2 ? warp >> 2 : 0, g = C::kG == 2 ? warp >> 2 : 0, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_o = tmem + lanes + q * DH + g * kOut;
    const uint32_t t_s = tmem + lanes + C::kOffS + q * C::kNS * kBN + g * kCols;
    float *shared_max = reinterpret_cast<float *>(sm + C::kOffMax);
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.out);
    bool ok = true;                  // a warp whose wait expired still meets the block barriers
    int f0 = 0, j = 0, nu = 0;       // fills before this unit; tiles so far; units
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok && !mbar_wait(bar, parity, abort, kWaitNs)) {
        give_up();
        ok = false;
      }
      if (ok) tc_fence_after();
      return ok;
    };
    // the other group's value for this row; buffers alternate from call to call
    auto exchange = [&](float x, int buffer) -> float {
      shared_max[(buffer * 2 + g) * kBM + row] = x;
      bar_sync_softmax<256>();
      return shared_max[(buffer * 2 + (g ^ 1)) * kBM + row];
    };
    for (unsigned r = 0, u; (u = unit_at<kSplit>(prm, r)) < prm.units; ++r) {
      const Un un(prm, u);
      const int q0 = un.first(q), t = q0 + row;
      const long long out_row = (static_cast<long long>(un.b) * p.T + t) * p.Hq + un.head(q);
      const long long lse_row = (static_cast<long long>(un.b) * p.Hq + un.head(q)) * p.T + t;
      float m = -INFINITY, l = 0.0f;
      bool begun = false;
      const DeadKeys dead = dead_keys(p, un.n.nk);
      for (int i = 0; i < un.kt.n; ++i) {
        if (!un.sees(p, q, i)) continue;
        const bool first = !begun;
        begun = true;
        const int s = j % C::kNS, k0 = un.tile(i) * kBN;
        const uint32_t ts = t_s + s * kBN;
        const uint32_t tp = C::kApart ? tmem + lanes + C::kOffP + q * (kBN / 2) : ts;
        // Where every query of the tile sees every key of it, the scores stay in
        // registers from the maximum to the weights. Elsewhere they are read twice, 32
        // columns at a time in rolled loops (unrolled over a row, that path alone
        // outran the instruction cache: 7000 cycles a tile), with the keys that this
        // row sees of 32 as bits.
        const bool whole = k0 + kBN - 1 <= min(q0 + off, un.n.nk - 1) &&
                           (p.window == 0 || k0 > q0 + kBM - 1 + off - p.window || k0 + kBN <= p.sinks);
        auto seen = [&](int c) -> uint32_t {
          const int key = k0 + g * kCols + c, hi = min(t + off, un.n.nk - 1) - key;
          const int lo = p.window > 0 ? t + off - p.window + 1 - key : 0;
          return bits_between(lo, hi) | bits_between(0, min(hi, p.sinks - key - 1));
        };
        // the scores' columns may take the next tile's (where weights lie apart from them)
        auto read = [&]() {
          if constexpr (C::kApart) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_free[q]);
          }
        };
        float v[kCols / 32][32], top = -INFINITY;
        if (wait(&s_full[q * C::kNS + s], (j / C::kNS) & 1)) {
          if (whole) {
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_ld32(ts + c * 32, v[c]);
#pragma unroll
            for (int c = 0; c < kCols / 32; ++c) tmem_wait_ld32(v[c]);
            read();
            top = max_of(v);
          } else {
#pragma unroll 1
            for (int c = 0; c < kCols; c += 32) {
              const uint32_t bits = seen(c);
              // (columns that none of a warp's rows sees: worth a test where a thread has
              // all 128, 31.5 -> 29.7 us on a batch of short windows)
              if (C::kG == 1 && !__any_sync(0xFFFFFFFFu, bits != 0u)) continue;
              float w[1][32];
              tmem_ld32(ts + c, w[0]);
              tmem_wait_ld32(w[0]);
              hide(w[0], bits, -INFINITY);
              top = max2(top, max_of(w));
            }
          }
        }
        if constexpr (C::kG == 2) top = max2(top, exchange(top, j & 1));
        if (!ok) {
          ++j;
          continue;
        }
        top *= prm.c;
        // (a NaN moves m too and stays in it, and a score of +inf makes it one: its weight
        // would be inf - inf, which the polynomial does not show)
        const float mn = top <= m + kSlack ? m : max2(top, m) + (top - top);
        if (__any_sync(0xFFFFFFFFu, mn != m)) {
          const float f = m == -INFINITY ? 0.0f : ex2(m - mn);
          l *= f;
          m = mn;
          if (!first && wait(&o_done[q], (j - 1) & 1)) {  // O so far: P V of the last tile is done
#pragma unroll 1
            for (int c = 0; c < kOut; c += 32) {
              float o[32];
              tmem_ld32(t_o + c, o);
              tmem_wait_ld32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= f;
              tmem_st32(t_o + c, o);
            }
            tmem_wait_st();
          }
        }
        if (dead.any(k0, kBN)) {
          // zero the value rows that no query sees, once V is there (each query tile
          // does, before its own product: zeros over zeros)
          const int f = f0 + fill_of<DH>(i, true, un.kt.n);
          for (int x = 0; x < C::kPer; ++x) {
            const int sl = (f + x) % C::kSlots;
            if (wait(&full[sl], ((f + x) / C::kSlots) & 1) && g == 0 && dead.in(k0 + row))
              for (int c = 0; c < C::kCols / 64; ++c)
                for (int e = 0; e < 8; ++e)
                  *reinterpret_cast<uint4 *>(sm + C::kOffRing + sl * C::kSlotBytes + c * (kBN * 128) +
                                             row * 128 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (C::kApart && !first) wait(&o_done[q], (j - 1) & 1);   // the last tile's weights were read
        // half of the thread's weights are in TMEM: the tensor core may use them
        auto publish = [&](int half) {
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&p_full[(half * C::kNQ + q) * C::kNS + s]);
        };
        const float base = m == -INFINITY ? 0.0f : m;
        const unsigned long long cc = pair(prm.c, prm.c), mm = pair(-base, -base);
        unsigned long long sum[2] = {0ull, 0ull};
        // The weights of a group's columns go to the first half of its score columns,
        // or to columns of their own. The first half of them is handed over when the
        // next 32 are computed, so that its stores have long ended.
        if (whole) {
#pragma unroll
          for (int c = 0; c < kCols / 32; ++c) {
            uint32_t packed[16];
            weights32<C::kPoly>(v[c], cc, mm, sum, packed);
            if (c == kCols / 64) publish(0);
            tmem_st16u(tp + c * 16, packed);
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < kCols; c += 32) {
            const uint32_t bits = seen(c);
            uint32_t packed[16] = {};
            if (C::kG == 2 || __any_sync(0xFFFFFFFFu, bits != 0u)) {
              float w[32];
              tmem_ld32(ts + c, w);
              tmem_wait_ld32(w);
              hide(w, bits, -INFINITY);
              weights32<0>(w, cc, mm, sum, packed);      // hidden scores give 0 exactly
            }
            if (c == kCols / 2) publish(0);
            tmem_st16u(tp + c / 2, packed);
          }
          read();
        }
        publish(1);
        float s0, s1;
        unpair(add2(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
        ++j;
      }
      if constexpr (kSplit) {
        // (a Q that no product reads has to have landed too: join writes over it)
        if (un.kt.n > 0) wait(begun ? &all_done[q] : &q_full[q], 0);
        if (C::kG == 2) l += exchange(l, j & 1);
        join<DH>(prm, un, t_o, ok && begun, q, g, row, m, l, sm);
        break;
      }
      f0 += 2 * un.kt.n * C::kPer;
      const bool live = t < un.n.nq;
      if (!begun) {                                      // sees no key
        if (live) {
          for (int e = 0; e < kOut / 8; ++e)
            reinterpret_cast<uint4 *>(out + out_row * DH + g * kOut)[e] = make_uint4(0u, 0u, 0u, 0u);
          if (g == 0 && p.lse != nullptr) p.lse[lse_row] = -INFINITY;
        }
        continue;
      }
      if constexpr (C::kG == 2) {
        l += exchange(l, j & 1);                         // the row's sum, from both groups
        bar_sync_softmax<256>();                               // the next unit's first tile writes there
      }
      if (wait(&all_done[q], nu & 1)) {
        // a row that sees no key, or none with a score above -inf (to which the polynomial
        // gives 2^-126); NaN scores leave m and l NaN
        const bool none = m == -INFINITY;
        const float inv = none ? 0.0f : 1.0f / l;
        __nv_bfloat16 *dst = out + out_row * DH + g * kOut;
#pragma unroll 1
        for (int c = 0; c < kOut; c += 64) {
          float o[2][32];
          tmem_ld32(t_o + c, o[0]);
          tmem_ld32(t_o + c + 32, o[1]);
          tmem_wait_ld32(o[0]);
          tmem_wait_ld32(o[1]);
          if (c + 64 == kOut) {                          // O may be written again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[q]);
          }
          if (live) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (none) {
#pragma unroll
                for (int e = 0; e < 32; ++e) o[x][e] = 0.0f;
              }
              store_row(dst + c + x * 32, o[x], inv, prm.v8 != 0);
            }
          }
        }
        if (live && g == 0 && p.lse != nullptr)
          p.lse[lse_row] = none ? -INFINITY : m * kLn2 + logf(l);
      }
      ++nu;
    }
  }
  if constexpr (kSplit) {
    if (warp >= kTma) {                                  // the softmax warps' barriers of join
      cluster_sync();
      cluster_sync();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMma) tmem_dealloc(tmem, 512);
}

template <int DH, bool kSplit> cudaError_t start(const AttnArgs &p, const Params &prm, cudaStream_t st) {
  using C = Cfg<DH>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(attn_fwd_tc_kernel<DH, kSplit>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv;
  if (!attn_map(&mq, p.q, p.B, p.T, p.Hq, DH, kBM) || !attn_map(&mk, p.k, p.B, p.S, p.Hkv, DH, kBN) ||
      !attn_map(&mv, p.v, p.B, p.S, p.Hkv, DH, kBN))
    return cudaErrorInvalidValue;
  if constexpr (kSplit) {
    cudaLaunchAttribute attr;
    const unsigned parts = static_cast<unsigned>(prm.parts);
    const cudaLaunchConfig_t cfg = cluster_config(&attr, parts, dim3(prm.units * parts), C::kThreads, C::kSmem, st);
    return cudaLaunchKernelEx(&cfg, attn_fwd_tc_kernel<DH, true>, mq, mk, mv, prm);
  }
  attn_fwd_tc_kernel<DH, kSplit>
      <<<prm.units < 148u ? prm.units : 148u, C::kThreads, C::kSmem, st>>>(mq, mk, mv, prm);
  return cudaGetLastError();
}

template <int DH> cudaError_t launch(const AttnArgs &p, cudaStream_t st) {
  using C = Cfg<DH>;
  Params prm;
  prm.a = p;
  prm.rows2 = C::kNQ == 2 && (p.Hq / p.Hkv) % 2 != 0 ? 1 : 0;
  prm.n_qt = ceil_div(p.T, kBM * (1 + prm.rows2));
  prm.n_h = static_cast<unsigned>(C::kNQ == 2 && !prm.rows2 ? p.Hq / 2 : p.Hq);
  prm.units = static_cast<unsigned>(static_cast<long long>(prm.n_qt) * p.B * prm.n_h);
  prm.v8 = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0 ? 1 : 0;
  prm.c = p.scale * kLog2e;
  // While units leave half of the SMs idle, a cluster of 2, 4 or 8 blocks takes each,
  // kLeast key tiles or more a block, as long as all clusters fit on the GPU at once
  // (16 queries, 32768 keys, 16/4 heads of 128: 472 us in one block a unit, 74 in 8).
  // Two tiles are the least that pay: 128 queries of 16/8 heads of 128 over 512 keys
  // take 15.3 us whole, 14.8 in two parts and 13.9 in four of one tile, but over 256
  // keys 11.7 whole and 12.6 in two parts of one tile (256 wide 10.0 and 12.0).
  const int last = (prm.n_qt - 1) * kBM * (1 + prm.rows2) + p.S - p.T;
  const int most = key_tiles(last, p.S - 1, p.S, p.window, p.sinks, kBN).n;
  static std::atomic<unsigned long long> done{0};
  static ClusterRoom room;
  const cudaError_t e = cluster_parts(attn_fwd_tc_kernel<DH, true>, C::kThreads, C::kSmem, &done, &room, prm.units,
                                      most / kLeast, &prm.parts);
  if (e != cudaSuccess) return e;
  return prm.parts > 1 ? start<DH, true>(p, prm, st) : start<DH, false>(p, prm, st);
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
