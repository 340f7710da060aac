// Windowed attention with sinks on the 5th-generation tensor core, backward
// (include/rglru_attn.h), for bf16 heads 64, 128 or 256 wide.
//
//   P = 2^(S c - lse log2 e), dP = dO V^T, dS = P (dP - delta),
//   dQ = scale dS K, dK = scale dS^T Q, dV = P^T dO
//
// Every block keeps 128 rows of one side resident and walks tiles of the other,
// so each gradient is summed in TMEM in a fixed order, without atomics: query
// rows against the keys they see (dQ), key rows against the queries that see
// them, head by head over the group that shares the key head (dK, dV). Both
// are one walk: with resident rows X, Y and walked tiles U, W
//   query rows  X = Q, Y = dO, U = K, W = V;   key rows  X = K, Y = V, U = Q, W = dO
//   S = X U^T,  dP = Y W^T,  first += dS U,  second += P W
// (key rows hold S and dP transposed, lse and delta then vary along the columns
// and are read from shared memory). dQ sums `first`; dK and dV are `first` and
// `second`. 256-wide heads have no room in TMEM for both sums (2 x 256 of 512
// columns): dK and dV are blocks of their own there, at the price of a second S.
// Seven products (eight for 256-wide heads) instead of the five of one pass that
// adds dQ up in memory by atomics, whose order would change the result.
//
// Warps 0-15 turn scores into weights, warp group g a quarter of a tile's columns,
// thread = row = TMEM lane; P and dS go back to TMEM as bf16 over the scores
// they came from and are the A operand of their product. Warp 16 issues the TMA
// copies, warps 18 and 19 fetch lse and delta, warp 17 issues the MMAs in an order that
// keeps the tensor core fed: the next tile's S runs while dS is formed, and P of the
// next tile is formed during `first` and dP.
//
// P and dS are rounded to bf16, as the operands of their products have to be: that
// rounding's share of a gradient's error is about the store's own (together 1.3 to 1.5
// times the error of fp32 products that are stored in bf16). Sums are fp32.
//
// Bound by the tensor core and the hand-overs between it and the weight warps: 4 x 2048
// tokens, 10 query heads on one 256-wide key head, window 1024, take 265 us with the row
// sums' 22 (608 TFLOP/s of the five products that the gradients need, 0.97 PFLOP/s of
// the eight done); 2 x 4096 tokens, 16/4 heads of 128, 395 us (870; 1.22 PFLOP/s of the
// seven done). Short walks (3 x 1535 ragged tokens, 16 heads of 64, window 512: 68 us of
// 1152 blocks) spend 2300 cycles before the first scores, 2500 a step, of which the
// exponentials are half, and 2600 after the last.
//
// All kinds of a call are one grid, the key-row blocks first. Key rows' steps
// are cut into pieces (PiecePlan), joined by attn_join_kernel.
//
// Every wait is bounded; on expiry the kernel records RGLRU_ERR_TIMEOUT (wait
// site 8), drains what it issued and returns.
#include "attn_tc.cuh"

namespace rglru {
namespace {

using namespace tc;

constexpr int kBM = 128;
constexpr int kWarps = 16;                             // weight warps; then copies, MMAs, stats (2)
constexpr int kThreads = (kWarps + 4) * 32;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;
constexpr int kSite = 8;
constexpr float kLog2e = 1.4426950408889634f;

struct Params {
  AttnArgs a;
  PiecePlan pl;
  const float *delta;
  float *parts;
  int n_qt;
  unsigned n_kv;     // key-row blocks of one kind
  int v8;            // gradients' rows may be stored 32 bytes at a time
  float c;           // scale * log2 e
};

// kFirst: sum dS U; kSecond: sum P W.
template <int DH, bool kFirst, bool kSecond> struct Cfg {
  static constexpr int kBN = DH == 256 ? 64 : 128;         // rows of a walked tile
  // 256 wide: X lives in TMEM. Read from shared memory for each of a tile's 64-row
  // products, it made S bound by shared memory's bandwidth (6 KB in 32 cycles), and
  // its 64 KB there are a third U and a second W buffer now.
  static constexpr bool kXT = DH == 256;
  static constexpr int kNS = kFirst && DH != 64 ? 1 : 2;   // score buffers
  static constexpr int kNU = 3, kNW = kXT && !kFirst ? 3 : 2;
  static constexpr int kXBytes = kBM * DH * 2;
  static constexpr int kTile = kBN * DH * 2;
  static constexpr int kOffY = kXT ? 0 : kXBytes;
  static constexpr int kOffU = kOffY + (kFirst ? kXBytes : 0);
  static constexpr int kOffW = kOffU + kNU * kTile;
  static constexpr int kOffX = kXT ? kOffW : 0;            // in TMEM: on its way there
  static constexpr int kOffStat = kOffW + kNW * kTile;     // [2][lse, delta][kBN]
  static constexpr int kOffBar = kOffStat + 2 * 2 * kBN * 4;
  static constexpr int kNumBars = 3 + 2 * (kNU + kNW) + 2 * 4 + 3;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmem = kOffMisc + 16;
  static constexpr int kTSecond = kFirst ? DH : 0;         // TMEM columns
  static constexpr int kTS = kTSecond + (kSecond ? DH : 0);
  static constexpr int kTdP = kTS + kNS * kBN;
  static constexpr int kTX = kTdP + (kFirst ? kBN : 0);
  static_assert(kSmem <= kMaxSmem && kTX + (kXT ? DH / 2 : 0) <= 512, "shared memory, TMEM");
  static_assert(!kXT || kNW * kTile >= kXBytes, "X on its way to TMEM");
};

template <int DH> constexpr int smem_bytes() {
  if constexpr (DH == 256)
    return Cfg<256, true, false>::kSmem > Cfg<256, false, true>::kSmem ? Cfg<256, true, false>::kSmem
                                                                      : Cfg<256, false, true>::kSmem;
  else
    return Cfg<DH, true, true>::kSmem;
}

// Where a block stands: its rows, and the walk over the other side.
struct Walk {
  int b, h, kvh;       // h: query rows only
  int r0;              // first row
  RowLens len;
  int n;               // steps
  KeyTiles kt;         // query rows
  Steps st;            // key rows: steps first .. first + n - 1
  int first;
};

// The walk's place: a step's head (key rows), and the first row of its tile; moved
// on without divisions.
template <bool kKeys, int kBN> struct Step {
  int i, h, t0;
  __device__ Step(const Walk &w, int G) : i(0), h(w.kvh * G), t0(0) {
    if (kKeys) {
      h += w.first / w.st.nq;
      t0 = (w.st.q0 + w.first % w.st.nq) * kBN;
    } else {
      h = w.kvh;
      t0 = w.kt.tile(0) * kBN;
    }
  }
  __device__ void next(const Walk &w) {
    ++i;
    if (kKeys) {
      t0 += kBN;
      if (t0 == (w.st.q0 + w.st.nq) * kBN) {
        t0 = w.st.q0 * kBN;
        ++h;
      }
    } else {
      t0 = w.kt.tile(i) * kBN;
    }
  }
};

template <int DH, bool kKeys, bool kFirst, bool kSecond>
__device__ __forceinline__ void walk(const Params &prm, const CUtensorMap *mx, const CUtensorMap *my,
                                     const CUtensorMap *mu, const CUtensorMap *mw, const Walk &wk,
                                     bool whole_tile, size_t slot, unsigned char *sm) {
  using C = Cfg<DH, kFirst, kSecond>;
  constexpr int kBN = C::kBN, kW = kBN / 4;             // columns of a warp group
  const AttnArgs &p = prm.a;
  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int G = p.Hq / p.Hkv, off = p.S - p.T;
  uint64_t *x_full = reinterpret_cast<uint64_t *>(sm + C::kOffBar);
  uint64_t *y_full = x_full + 1, *x_done = y_full + 1;    // x_done: X is in TMEM
  uint64_t *u_full = x_done + 1, *u_empty = u_full + C::kNU;
  uint64_t *w_full = u_empty + C::kNU, *w_empty = w_full + C::kNW;
  uint64_t *s_full = w_empty + C::kNW;                    // [kNS]
  uint64_t *p_full = s_full + 2;                          // [kNS] P is in TMEM (kSecond) or S was read
  uint64_t *stat_full = p_full + 2, *stat_empty = stat_full + 2;   // [2] key rows
  uint64_t *dp_full = stat_empty + 2, *ds_full = dp_full + 1, *done = ds_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + C::kOffMisc);
  volatile int *abort = reinterpret_cast<volatile int *>(sm + C::kOffMisc + 4);
  float *stat = reinterpret_cast<float *>(sm + C::kOffStat);
  if (tid == 0) {
    mbar_init(x_full, 1);
    mbar_init(y_full, 1);
    mbar_init(x_done, kWarps);
    for (int s = 0; s < C::kNU; ++s) {
      mbar_init(&u_full[s], 1);
      mbar_init(&u_empty[s], 1);
    }
    for (int s = 0; s < C::kNW; ++s) {
      mbar_init(&w_full[s], 1);
      mbar_init(&w_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&p_full[s], kWarps);
      mbar_init(&stat_full[s], 2);
      mbar_init(&stat_empty[s], kWarps);
    }
    mbar_init(dp_full, 1);
    mbar_init(ds_full, kWarps);
    mbar_init(done, 1);
    *abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarps + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&]() {
    if (!*abort) {
      if (p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_TIMEOUT | (kSite << 8) |
                                                       (static_cast<int>(blockIdx.x & 0x7FFFu) << 16));
      *abort = 1;
    }
  };

  if (warp == kWarps) {
    // ============================ TMA producer ============================
    if (lane == 0) {
      const int xh = kKeys ? wk.kvh : wk.h;
      mbar_arrive_expect_tx(x_full, C::kXBytes);
      for (int c = 0; c < DH / 64; ++c)
        tma_load_4d(sm + C::kOffX + c * (kBM * 128), mx, x_full, c * 64, wk.r0, xh, wk.b);
      if (kFirst) {
        mbar_arrive_expect_tx(y_full, C::kXBytes);
        for (int c = 0; c < DH / 64; ++c)
          tma_load_4d(sm + C::kOffY + c * (kBM * 128), my, y_full, c * 64, wk.r0, xh, wk.b);
      }
      int w_issued = 0, u_issued = 0;
      for (Step<kKeys, kBN> st(wk, G); st.i < wk.n; st.next(wk)) {
        const int i = st.i, h = st.h, t0 = st.t0;
        const int u = i % C::kNU, w = i % C::kNW;
        if (!mbar_wait(&u_empty[u], ((i / C::kNU) & 1) ^ 1, abort, kWaitNs)) {
          give_up();
          break;
        }
        mbar_arrive_expect_tx(&u_full[u], C::kTile);
        for (int c = 0; c < DH / 64; ++c)
          tma_load_4d(sm + C::kOffU + u * C::kTile + c * (kBN * 128), mu, &u_full[u], c * 64, t0, h, wk.b);
        u_issued = i + 1;
        // the W buffers hold X on its way to TMEM at first
        if ((C::kXT && i == 0 && !mbar_wait(x_done, 0, abort, kWaitNs)) ||
            !mbar_wait(&w_empty[w], ((i / C::kNW) & 1) ^ 1, abort, kWaitNs)) {
          give_up();
          break;
        }
        mbar_arrive_expect_tx(&w_full[w], C::kTile);
        for (int c = 0; c < DH / 64; ++c)
          tma_load_4d(sm + C::kOffW + w * C::kTile + c * (kBN * 128), mw, &w_full[w], c * 64, t0, h, wk.b);
        w_issued = i + 1;
      }
      if (*abort) {
        mbar_wait_drain(x_full, 0, kDrainNs);
        if (kFirst) mbar_wait_drain(y_full, 0, kDrainNs);
        for (int j = u_issued - 1; j >= 0 && j >= u_issued - C::kNU; --j)
          mbar_wait_drain(&u_full[j % C::kNU], (j / C::kNU) & 1, kDrainNs);
        for (int j = w_issued - 1; j >= 0 && j >= w_issued - C::kNW; --j)
          mbar_wait_drain(&w_full[j % C::kNW], (j / C::kNW) & 1, kDrainNs);
      }
    }
  } else if (warp >= kWarps + 2) {
    // ===================== lse and delta of key rows' queries =====================
    if (kKeys) {
      const int second = warp - (kWarps + 2);             // the lse's warp, the delta's
      const float *src = second ? prm.delta : p.lse;
      const float f = second ? 1.0f : kLog2e;
      for (Step<kKeys, kBN> st(wk, G); st.i < wk.n; st.next(wk)) {
        float v[kBN / 32] = {};
        if (!second || kFirst) {
          const float *row = src + (static_cast<long long>(wk.b) * p.Hq + st.h) * p.T;
#pragma unroll
          for (int x = 0; x < kBN / 32; ++x)
            if (st.t0 + x * 32 + lane < wk.len.nq) v[x] = __ldg(row + st.t0 + x * 32 + lane) * f;
        }
        const int s = st.i & 1;
        if (!mbar_wait(&stat_empty[s], ((st.i >> 1) & 1) ^ 1, abort, kWaitNs)) {
          give_up();
          break;
        }
#pragma unroll
        for (int x = 0; x < kBN / 32; ++x) stat[(s * 2 + second) * kBN + x * 32 + lane] = v[x];
        __syncwarp();
        if (lane == 0) mbar_arrive(&stat_full[s]);
      }
    }
  } else if (warp == kWarps + 1) {
    // ============================= MMA issuer =============================
    // The whole warp walks, one elected lane issues.
    constexpr uint32_t id_s = idesc_bf16_f32(kBM, kBN, false, false);
    constexpr uint32_t id_o = idesc_bf16_f32(kBM, DH, false, true);
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
    // (one lane) rows (K-major, resident) times tile (K-major): D = R T^T over DH
    auto scores = [&](uint32_t d, uint32_t rows, uint32_t tile) {
      const uint32_t ad = desc_lo(base + rows, 16), bd = desc_lo(base + tile, 16);
#pragma unroll
      for (int k = 0; k < DH / 16; ++k)
        mma_ss(d, ad + (((k & 3) * 32 + (k >> 2) * (kBM * 128)) >> 4),
               bd + (((k & 3) * 32 + (k >> 2) * (kBN * 128)) >> 4), id_s, k > 0 ? 1u : 0u);
    };
    // (one lane) the same with the rows in TMEM
    auto scores_t = [&](uint32_t d, uint32_t tile) {
      const uint32_t bd = desc_lo(base + tile, 16);
#pragma unroll
      for (int k = 0; k < DH / 16; ++k)
        mma_ts(d, tmem + C::kTX + k * 8, bd + (((k & 3) * 32 + (k >> 2) * (kBN * 128)) >> 4), id_s,
               k > 0 ? 1u : 0u);
    };
    // (one lane) weights in TMEM (each group's columns at the start of its
    // scores) times tile (MN-major): D += A T
    auto product = [&](uint32_t d, uint32_t a, uint32_t tile, bool add) {
      const uint32_t bd = desc_lo(base + tile, kBN * 128);
#pragma unroll
      for (int k = 0; k < kBN / 16; ++k)
        mma_ts(d, a + (k / (kW / 16)) * kW + (k % (kW / 16)) * 8, bd + ((k * 16 * 128) >> 4),
               id_o, k > 0 ? 1u : add);
    };
    auto u_at = [&](int i) { return static_cast<uint32_t>(C::kOffU + (i % C::kNU) * C::kTile); };
    auto w_at = [&](int i) { return static_cast<uint32_t>(C::kOffW + (i % C::kNW) * C::kTile); };
    auto issue_s = [&](int i) {
      if (!wait(&u_full[i % C::kNU], (i / C::kNU) & 1)) return;
      if (elect_one()) {
        if (C::kXT)
          scores_t(tmem + C::kTS + (i % C::kNS) * kBN, u_at(i));
        else
          scores(tmem + C::kTS + (i % C::kNS) * kBN, C::kOffX, u_at(i));
        mma_commit(&s_full[i % C::kNS]);
        if (!kFirst) mma_commit(&u_empty[i % C::kNU]);
      }
      __syncwarp();
    };
    auto issue_dp = [&](int i) {
      if (!wait(&w_full[i % C::kNW], (i / C::kNW) & 1)) return;
      if (elect_one()) {
        scores(tmem + C::kTdP, C::kOffY, w_at(i));
        mma_commit(dp_full);
        if (!kSecond) mma_commit(&w_empty[i % C::kNW]);
      }
      __syncwarp();
    };
    auto issue_second = [&](int i) {
      if (!kFirst && !wait(&w_full[i % C::kNW], (i / C::kNW) & 1)) return;
      if (elect_one()) {
        product(tmem + C::kTSecond, tmem + C::kTS + (i % C::kNS) * kBN, w_at(i), i > 0);
        mma_commit(&w_empty[i % C::kNW]);
      }
      __syncwarp();
    };
    wait(C::kXT ? x_done : x_full, 0);
    if (ok) issue_s(0);
    if (kFirst && wait(y_full, 0)) issue_dp(0);
    for (int i = 0; i < wk.n && ok; ++i) {
      if (!kFirst) {
        if (i + 1 < wk.n) issue_s(i + 1);
        if (wait(&p_full[i & 1], (i >> 1) & 1)) issue_second(i);
        continue;
      }
      // P is in place, or S was read: the score columns are free after `second`, or,
      // with two buffers, after the last tile's
      if (C::kNS == 2 && i + 1 < wk.n) issue_s(i + 1);
      if (!wait(&p_full[i % C::kNS], (i / C::kNS) & 1)) break;
      if (kSecond) issue_second(i);
      if (C::kNS == 1 && ok && i + 1 < wk.n) issue_s(i + 1);
      if (wait(ds_full, i & 1)) {
        if (elect_one()) {
          product(tmem, tmem + C::kTdP, u_at(i), i > 0);
          mma_commit(&u_empty[i % C::kNU]);
        }
        __syncwarp();
        if (i + 1 < wk.n) issue_dp(i + 1);
      }
    }
    if (elect_one()) mma_commit(done);
    if (*abort) mbar_wait_drain(done, 0, kDrainNs);
  } else {
    // =============================== weights ==============================
    // Thread = row = TMEM lane, warp group g the columns kW g .. of a tile.
    const int g = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int r = wk.r0 + row;                             // this thread's query or key
    const int nq = wk.len.nq, nk = wk.len.nk;
    float row_lse = 0.0f, row_delta = 0.0f;
    if (!kKeys && r < nq) {
      const long long x = (static_cast<long long>(wk.b) * p.Hq + wk.h) * p.T + r;
      row_lse = __ldg(p.lse + x) * kLog2e;
      if (kFirst) row_delta = __ldg(prm.delta + x);
    }
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (ok && !mbar_wait(bar, parity, abort, kWaitNs)) {
        give_up();
        ok = false;
      }
      if (ok) tc_fence_after();
      return ok;
    };
    if constexpr (C::kXT) {                                // X to TMEM: 64 columns of a row a thread
      if (wait(x_full, 0)) {
        uint32_t w[32];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 x = *reinterpret_cast<const uint4 *>(sm + C::kOffX + g * (kBM * 128) + row * 128 +
                                                           ((c ^ (row & 7)) << 4));
          w[4 * c] = x.x;
          w[4 * c + 1] = x.y;
          w[4 * c + 2] = x.z;
          w[4 * c + 3] = x.w;
        }
        tmem_st32u(tmem + lanes + C::kTX + g * 32, w);
        tmem_wait_st();
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(x_done);
      }
    }
    Step<kKeys, kBN> st(wk, G);
    for (int i = 0; i < wk.n && ok; ++i, st.next(wk)) {
      const int t0 = st.t0;
      // the columns that this row sees, as bits; all of them where the whole tile is
      // seen by every row
      bool all;
      uint32_t bits = 0xFFFFFFFFu, ds_bits = 0xFFFFFFFFu;  // and those whose scores have a gradient
      if (kKeys)
        all = t0 + kBN <= nq && t0 + off >= wk.r0 + kBM - 1 &&
              (p.window == 0 || wk.r0 + kBM <= p.sinks || t0 + kBN - 1 + off < wk.r0 + p.window);
      else
        all = t0 + kBN - 1 <= min(wk.r0 + off, nk - 1) &&
              (p.window == 0 || t0 > wk.r0 + kBM - 1 + off - p.window || t0 + kBN <= p.sinks);
      if (!all) {
        const int t1 = t0 + g * kW;                        // the first column's query or key
        if (kKeys) {
          const int lo = r - off - t1;
          const int hi = (p.window > 0 && r >= p.sinks ? min(nq - t1, lo + p.window) : nq - t1) - 1;
          bits = bits_between(lo, hi);
          // a query that sees one key: the one at position 0, or all of a window of one
          ds_bits = p.window == 1 && p.sinks == 0 ? 0u : bits & ~bits_between(-off - t1, -off - t1);
        } else {
          const int hi = min(r + off, nk - 1) - t1;
          bits = bits_between(p.window > 0 ? r + off - p.window + 1 - t1 : 0, hi) |
                 bits_between(0, min(hi, p.sinks - t1 - 1));
          ds_bits = attn_lone(r + off, p.window, p.sinks) ? 0u : bits;
        }
      }
      const int sb = i % C::kNS;
      const float *ls = stat + (i & 1) * 2 * kBN + g * kW;
      const uint32_t ts = tmem + lanes + C::kTS + sb * kBN + g * kW;
      float v[kW];
      if (kKeys && !wait(&stat_full[i & 1], (i >> 1) & 1)) break;
      if (!wait(&s_full[sb], (i / C::kNS) & 1)) break;
      {
        ld_cols(ts, v);
        if (kFirst && !kSecond) {                          // the scores may be overwritten
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[sb]);
        }
        const unsigned long long cc = pair(prm.c, prm.c), mm = pair(-row_lse, -row_lse);
#pragma unroll
        for (int c = 0; c < kW; c += 4) {
          unsigned long long m0 = mm, m1 = mm;
          if (kKeys) {
            const float4 x = *reinterpret_cast<const float4 *>(ls + c);
            m0 = pair(-x.x, -x.y);
            m1 = pair(-x.z, -x.w);
          }
          unpair(fma2(pair(v[c], v[c + 1]), cc, m0), v[c], v[c + 1]);
          unpair(fma2(pair(v[c + 2], v[c + 3]), cc, m1), v[c + 2], v[c + 3]);
          // an eighth of them on the FMA pipes (2 x 4096 tokens, 16/4 heads of 128: 395 us
          // with none, 392 with an eighth, 391 to 394 with more; 64 wide 92 with none and
          // an eighth, 95 and more with a quarter)
          if (c % 16 == 0) {
            ex2_pair<true>(v[c], v[c + 1]);
          } else {
            v[c] = ex2(v[c]);
            v[c + 1] = ex2(v[c + 1]);
          }
          v[c + 2] = ex2(v[c + 2]);
          v[c + 3] = ex2(v[c + 3]);
        }
        hide(v, bits, 0.0f);
        // walked rows that nobody sees, or that see nothing, zeroed before a product reads them
        bool dead = false;
        if (kKeys)
          dead = (t0 + kBN > nq && nq < p.T) || t0 + off < 0;
        else
          dead = dead_keys(p, nk).any(t0, kBN);
        if (dead) {
          if (kFirst && kSecond && !wait(dp_full, i & 1)) break;
          if (!kFirst && !wait(&w_full[i % C::kNW], (i / C::kNW) & 1)) break;
          const bool mine = tid < kBN && (kKeys ? t0 + tid >= nq || t0 + tid + off < 0
                                                : dead_keys(p, nk).in(t0 + tid));
          if (mine)
            for (int c = 0; c < DH / 64; ++c)
              for (int e = 0; e < 8; ++e) {
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                const int o = c * (kBN * 128) + tid * 128 + e * 16;
                if (kFirst) *reinterpret_cast<uint4 *>(sm + C::kOffU + (i % C::kNU) * C::kTile + o) = z;
                if (kSecond) *reinterpret_cast<uint4 *>(sm + C::kOffW + (i % C::kNW) * C::kTile + o) = z;
              }
          fence_proxy_async_smem();
        }
        if (kSecond) {
          st_bf16(ts, v);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[sb]);
        }
      }
      if (kFirst) {
        if (!wait(dp_full, i & 1)) break;
        {
          const uint32_t td = tmem + lanes + C::kTdP + g * kW;
          const unsigned long long dd = pair(-row_delta, -row_delta);
          float d[kW];
          ld_cols(td, d);
#pragma unroll
          for (int e = 0; e < kW; e += 4) {
            unsigned long long d0 = dd, d1 = dd;
            if (kKeys) {
              const float4 x = *reinterpret_cast<const float4 *>(ls + kBN + e);
              d0 = pair(-x.x, -x.y);
              d1 = pair(-x.z, -x.w);
            }
            unpair(mul2(add2(pair(d[e], d[e + 1]), d0), pair(v[e], v[e + 1])), d[e], d[e + 1]);
            unpair(mul2(add2(pair(d[e + 2], d[e + 3]), d1), pair(v[e + 2], v[e + 3])), d[e + 2], d[e + 3]);
          }
          hide(d, ds_bits, 0.0f);                          // whatever dP holds there
          st_bf16(td, d);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(ds_full);
        }
      }
      if (kKeys) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&stat_empty[i & 1]);
      }
    }
    if (wait(done, 0)) {
      const bool live = r < (kKeys ? nk : nq);
      constexpr int kCols = DH / 4, kStep = kCols < 32 ? kCols : 32;   // of this warp group
#pragma unroll
      for (int part = 0; part < 2; ++part) {               // first, second
        if (part == 0 ? !kFirst : !kSecond) continue;
        const uint32_t t = tmem + lanes + (part == 0 ? 0 : C::kTSecond) + g * kCols;
        const float f = part == 0 ? p.scale : 1.0f;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(part == 1 ? p.dv : kKeys ? p.dk : p.dq);
        dst += kKeys ? ((static_cast<long long>(wk.b) * p.S + r) * p.Hkv + wk.kvh) * DH
                     : ((static_cast<long long>(wk.b) * p.T + r) * p.Hq + wk.h) * DH;
        float *part_dst = prm.parts + slot + static_cast<size_t>(part * kBM + row) * DH;
#pragma unroll
        for (int c = 0; c < kCols; c += kStep) {
          float o[kStep];
          ld_cols(t + c, o);
          if (!live) continue;
          if (whole_tile) {
            store_row(dst + g * kCols + c, o, f, prm.v8 != 0);
          } else {
#pragma unroll
            for (int e = 0; e < kStep; e += 4)
              *reinterpret_cast<float4 *>(part_dst + g * kCols + c + e) =
                  make_float4(o[e] * f, o[e + 1] * f, o[e + 2] * f, o[e + 3] * f);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWarps + 1) tmem_dealloc(tmem, 512);
}

template <int DH>
__global__ void __launch_bounds__(kThreads, 1)
attn_bwd_tc_kernel(const __grid_constant__ CUtensorMap q_rows, const __grid_constant__ CUtensorMap do_rows,
                   const __grid_constant__ CUtensorMap k_rows, const __grid_constant__ CUtensorMap v_rows,
                   const __grid_constant__ CUtensorMap q_tile, const __grid_constant__ CUtensorMap do_tile,
                   const __grid_constant__ CUtensorMap k_tile, const __grid_constant__ CUtensorMap v_tile,
                   const __grid_constant__ Params prm) {
  extern __shared__ __align__(1024) unsigned char sm[];
  const AttnArgs &p = prm.a;
  if ((smem_u32(sm) & 1023u) != 0u) {
    if (threadIdx.x == 0 && p.dev_status) atomicCAS(p.dev_status, 0, RGLRU_ERR_UNSUPPORTED);
    return;
  }
  constexpr int kBN = DH == 256 ? 64 : 128;
  constexpr unsigned kKinds = DH == 256 ? 2 : 1;
  const int off = p.S - p.T, G = p.Hq / p.Hkv;
  Walk w = {};
  if (blockIdx.x < kKinds * prm.n_kv) {
    const bool second = blockIdx.x >= prm.n_kv;            // 256 wide: dK blocks, then dV blocks
    const unsigned x = second ? blockIdx.x - prm.n_kv : blockIdx.x;
    const unsigned heads = static_cast<unsigned>(p.B) * p.Hkv;
    const int bk = static_cast<int>(x % heads);
    w.b = bk / p.Hkv;
    w.kvh = bk % p.Hkv;
    w.len = row_lens(p, w.b);
    const PieceAt at = piece_at(prm.pl, static_cast<int>(x / heads));
    w.r0 = at.tile * kBM;
    if (w.r0 >= w.len.nk) return;
    w.st = steps_of(query_range(w.r0, kBM, w.len.nq, w.len.nk, off, p.window, p.sinks), kBN, G);
    const Piece pc = piece_of(prm.pl, w.st.n, at.piece);
    if (pc.first >= pc.last && at.piece > 0) return;
    w.first = pc.first;
    w.n = pc.last - pc.first;
    const bool whole = w.st.n <= prm.pl.len;
    const size_t slot =
        (static_cast<size_t>(bk) * prm.pl.slots + first_slot(prm.pl, at.tile) + at.piece) * 2 * kBM * DH;
    if (w.n == 0) {                                        // seen by no query: zero gradients
      const int rows = min(kBM, w.len.nk - w.r0);
      for (int part = 0; part < 2; ++part) {
        if (DH == 256 && (part == 1) != second) continue;
        __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(part == 1 ? p.dv : p.dk);
        for (int i = threadIdx.x; i < rows * (DH / 8); i += kThreads)
          reinterpret_cast<uint4 *>(
              dst + ((static_cast<long long>(w.b) * p.S + w.r0 + i / (DH / 8)) * p.Hkv + w.kvh) * DH)[i % (DH / 8)] =
              make_uint4(0u, 0u, 0u, 0u);
      }
      return;
    }
    if constexpr (DH == 256) {
      if (second)
        walk<DH, true, false, true>(prm, &k_rows, &v_rows, &q_tile, &do_tile, w, whole, slot, sm);
      else
        walk<DH, true, true, false>(prm, &k_rows, &v_rows, &q_tile, &do_tile, w, whole, slot, sm);
    } else {
      walk<DH, true, true, true>(prm, &k_rows, &v_rows, &q_tile, &do_tile, w, whole, slot, sm);
    }
    return;
  }
  unsigned x = blockIdx.x - kKinds * prm.n_kv;
  w.h = static_cast<int>(x % static_cast<unsigned>(p.Hq));
  x /= static_cast<unsigned>(p.Hq);
  w.b = static_cast<int>(x % static_cast<unsigned>(p.B));
  w.kvh = w.h / G;
  w.r0 = (prm.n_qt - 1 - static_cast<int>(x / static_cast<unsigned>(p.B))) * kBM;
  w.len = row_lens(p, w.b);
  if (w.r0 >= w.len.nq) return;
  const int last = min(w.r0 + kBM, w.len.nq) - 1;
  w.kt = key_tiles(w.r0 + off, last + off, w.len.nk, p.window, p.sinks, kBN);
  w.n = w.kt.n;
  if (w.n == 0) {                                          // sees no key: zero gradients
    __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.dq);
    for (int i = threadIdx.x; i < (last - w.r0 + 1) * (DH / 8); i += kThreads)
      reinterpret_cast<uint4 *>(
          dst + ((static_cast<long long>(w.b) * p.T + w.r0 + i / (DH / 8)) * p.Hq + w.h) * DH)[i % (DH / 8)] =
          make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  walk<DH, false, true, false>(prm, &q_rows, &do_rows, &k_tile, &v_tile, w, true, 0, sm);
}

// A call's steps are its key-row steps (twice for 256-wide heads) and about as many
// query-row steps, over 148 SMs. A tile of keys is cut only where one piece would be
// longer than 1.15 times an SM's share of them: a cut costs partial sums that are written and
// read again (4 rows of 2048, 10 query heads on one 256-wide key head: 257 us
// without cuts, 283 us with pieces of half, 318 us of a fifth of a tile).
PiecePlan plan_of(const AttnArgs &p) {
  return attn_plan(p.B, p.T, p.S, p.Hq, p.Hkv, p.window, p.sinks, kBM, p.dh == 256 ? 64 : 128,
                   p.dh == 256 ? 43 : 64, 4);
}

template <int DH>
cudaError_t launch(const AttnArgs &p, const PiecePlan &pl, const float *delta, float *parts, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = opt_in_smem(attn_bwd_tc_kernel<DH>, smem_bytes<DH>(), done);
  if (e != cudaSuccess) return e;
  constexpr int kBN = DH == 256 ? 64 : 128;
  const Strided dout = {p.dout, static_cast<long long>(p.T) * p.Hq * DH, static_cast<long long>(p.Hq) * DH, DH};
  CUtensorMap m[8];
  const bool ok = attn_map(&m[0], p.q, p.B, p.T, p.Hq, DH, kBM) && attn_map(&m[1], dout, p.B, p.T, p.Hq, DH, kBM) &&
                  attn_map(&m[2], p.k, p.B, p.S, p.Hkv, DH, kBM) && attn_map(&m[3], p.v, p.B, p.S, p.Hkv, DH, kBM) &&
                  attn_map(&m[4], p.q, p.B, p.T, p.Hq, DH, kBN) && attn_map(&m[5], dout, p.B, p.T, p.Hq, DH, kBN) &&
                  attn_map(&m[6], p.k, p.B, p.S, p.Hkv, DH, kBN) && attn_map(&m[7], p.v, p.B, p.S, p.Hkv, DH, kBN);
  if (!ok) return cudaErrorInvalidValue;
  Params prm;
  prm.a = p;
  prm.pl = pl;
  prm.delta = delta;
  prm.parts = parts;
  prm.n_qt = ceil_div(p.T, kBM);
  prm.n_kv = static_cast<unsigned>(static_cast<long long>(pl.slots) * p.B * p.Hkv);
  const uintptr_t outs = reinterpret_cast<uintptr_t>(p.dq) | reinterpret_cast<uintptr_t>(p.dk) |
                         reinterpret_cast<uintptr_t>(p.dv);
  prm.v8 = (outs & 31u) == 0 ? 1 : 0;
  prm.c = p.scale * kLog2e;
  const unsigned grid = (DH == 256 ? 2u : 1u) * prm.n_kv +
                        static_cast<unsigned>(static_cast<long long>(prm.n_qt) * p.B * p.Hq);
  attn_bwd_tc_kernel<DH><<<grid, kThreads, smem_bytes<DH>(), st>>>(m[0], m[1], m[2], m[3], m[4], m[5], m[6], m[7], prm);
  return cudaGetLastError();
}

}  // namespace

size_t attn_bwd_tc_workspace_bytes(const AttnArgs &p) {
  return attn_delta_bytes(p) + attn_parts_bytes(p, plan_of(p));
}

cudaError_t launch_attn_bwd_tc(const AttnArgs &p, void *ws, cudaStream_t st) {
  const PiecePlan pl = plan_of(p);
  float *delta = static_cast<float *>(ws);
  float *parts = delta + attn_delta_bytes(p) / sizeof(float);
  cudaError_t e = launch_attn_delta(p, RGLRU_IO_BF16, delta, st);
  if (e != cudaSuccess) return e;
  switch (p.dh) {
    case 64: e = launch<64>(p, pl, delta, parts, st); break;
    case 128: e = launch<128>(p, pl, delta, parts, st); break;
    default: e = launch<256>(p, pl, delta, parts, st); break;
  }
  if (e != cudaSuccess) return e;
  return launch_attn_join(p, RGLRU_IO_BF16, pl, parts, st);
}

}  // namespace rglru
