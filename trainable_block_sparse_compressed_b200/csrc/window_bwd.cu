// window_bwd.cu -- gradients of the windowed attention with sinks
// (window_attn.cu).  With P = softmax(scale Q K^T) recomputed from lse over the
// visible keys and D = rowsum(dO * O):
//   dV = P^T dO,   dS = P * (dO V^T - D),   dQ = scale dS K,   dK = scale dS^T Q.
//
// Three passes (and a merge), no atomics, so results repeat exactly:
//
//   stats  D and lse (log2 units) of every row, packed by query tile.
//   dkv    a CTA holds one 128-key tile and streams the query tiles that see
//          it; per tile S^T = K Q^T and dP^T = V dO^T (keys on the 128 lanes),
//          then dV += P^T dO and dK += dS^T Q with P^T, dS^T as the A operand
//          in tensor memory.
//   dq     a CTA holds one query tile and streams its key tiles: S = Q K^T,
//          dP = dO V^T, dQ += dS K.
//
// S and dP are computed in both passes: 7 products instead of 5.  One pass
// would have to add dQ up across CTAs in memory: in an order that changes from
// run to run, or in turns (not tried).
//
// dkv: S(j+1) is issued as soon as the warps have read S(j), so P goes through
// shared memory (32 KB) instead of over S; dS goes over dP, which dP(j+1) reuses
// after dK(j).  Four 128-column accumulators fill tensor memory.  (With P over S,
// P(j), dV(j), S(j+1), P(j+1) were one chain: 3870 cycles a tile.)  The
// query tiles of all key tiles in a row are cut into equal ranges, one per CTA
// (sinks and the causal triangle make key tiles very unequal); a key tile that
// a range cuts is summed from fp32 partials in order.
//
// dq double-buffers S: S(j+1) and dP(j+1) run while the warps form dS(j).
//
// P and dS are rounded to bf16 for the tensor core (half a step is 2^-8 relative,
// as for the outputs themselves), and D takes the forward's bf16 O; sums stay in
// fp32.
//
// One B200, B=2, T=4096, 32 heads on 2, causal, each launch alone: stats 30 us (135
// MB), dkv 488, dq 341, merge 11, after a forward of 284; the whole step in a row
// 1250-1270.  The tensor pipe is active 64 % of dkv and 66 % of dq.  dkv is
// bound by shared memory: operands of S, dP and dV (A and B), dK (B), P and the
// TMA's writes are 320 KB a query tile, 2500 of its ~3300 cycles; dq by its
// elementwise warps.  Q and dO come from L2 (88 MB of 2.2 GB from HBM).  Tried:
// one issuer for all products (dq 377 us), P over S (S then waits for dV), 16
// elementwise warps of 32 columns (equal), L2 prefetch of Q and dO (equal).
#include "window.cuh"

namespace infllmv2 {
namespace {

constexpr int kThreads = 384;          // 4 role warps, 8 elementwise warps
constexpr int kTile = 128 * 256;       // 128 rows x 128 channels bf16
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kItemUnits = 4;          // what a key tile costs beyond its query tiles
constexpr int kMinUnits = 8;

struct BwdArgs {
  Visible vis;
  int B, T, Hq, Hkv;
  int n_qt;                 // query tiles per (b, g)
  int n_kt;                 // key tiles
  float scale, scale_log2;
  const float* stats;       // [B * Hkv * n_qt][2][128]: lse (log2), D
  __nv_bfloat16 *dQ, *dK, *dV;
  // dkv schedule
  long long per, per_bg;    // units per CTA, units per (b, g)
  float* part;              // [2 * CTAs][2][128][128] partial dV, dK
  int4* part_item;          // [CTAs] (bg, key tile, first CTA, 1) of the key tile a CTA ends
};

// Query tiles that see key tile kt: [q0, q1].
struct QRange {
  int q0, q1;
};
template <int TPT>
__host__ __device__ inline QRange query_tiles(const Visible& v, int T, int kt) {
  const int k0 = kt * kKeyTile;
  const long long last = static_cast<long long>(k0) + kKeyTile - 1 + v.window - 1;
  const int t1 = k0 < v.n_sink || last > T - 1 ? T - 1 : static_cast<int>(last);
  return QRange{k0 / TPT, t1 / TPT};
}

// ---------------------------------------------------------------------------
// stats: one block per query tile; O and dO are read once, a half-warp per row
// and four rows in flight per half-warp (HBM-bound); rows with few keys take D
// from their keys, in blocks of their own
// ---------------------------------------------------------------------------
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t *x = &a.x, *y = &b.x;
  float d = 0.f;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float2 u = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(x + c));
    const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(y + c));
    d = fmaf(u.x, v.x, fmaf(u.y, v.y, d));
  }
  return d;
}

// Rows with no more visible keys than this take D from their keys, not from O:
// the rounding of O (and of the forward's P) is 2^-8 of values as large as V
// there, and through D moved dQ and dK by twice their own rounding (2 keys:
// 4.8e-3 relative, 16 keys: 2.5e-3, against 2.4e-3 without it). Such rows are
// t < kFewKeys, or all of them under a small window. Blocks of their own take
// them, first in the launch: read within the rows' sums, the keys one after the
// other left the last blocks 20 us behind the rest.
constexpr int kFewKeys = 16;

struct FewRows {
  int tokens;     // tokens 0 .. tokens-1 of every sequence are such
  int64_t rows;   // B * tokens * Hq
};

template <int G>
__global__ void __launch_bounds__(512, 2) stats_kernel(
    const __nv_bfloat16* __restrict__ Q, const __nv_bfloat16* __restrict__ K,
    const __nv_bfloat16* __restrict__ V, const __nv_bfloat16* __restrict__ O,
    const __nv_bfloat16* __restrict__ dO, const float* __restrict__ lse,
    float* __restrict__ stats, int T, int Hkv, int n_qt, Visible vis, float scale_log2,
    FewRows few, int n_bg, int* status) {
  grid_launch_next();
  constexpr int TPT = 128 / G;
  const int Hq = Hkv * G;
  const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
  const uint32_t lanes = 0xffffu << (threadIdx.x & 16);
  auto sum16 = [&](float x) {
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) x += __shfl_xor_sync(lanes, x, k);
    return x;
  };
  auto load = [&](const __nv_bfloat16* x, int64_t row) {
    return __ldg(reinterpret_cast<const uint4*>(x + row * kHeadDim + 8 * sub));
  };
  const int64_t few_blocks = (few.rows + 31) / 32;
  if (blockIdx.x < few_blocks) {
    // a half-warp per row: D = sum_c P_c (dO . V_c) / sum_c P_c over its keys
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + half;
    if (i >= few.rows) return;
    const int h = static_cast<int>(i % Hq), g = h / G;
    const int t = static_cast<int>(i / Hq % few.tokens), b = static_cast<int>(i / Hq / few.tokens);
    const int64_t row = (static_cast<int64_t>(b) * T + t) * Hq + h;
    const int64_t key0 = static_cast<int64_t>(b) * T;
    const uint4 q = load(Q, row), go = load(dO, row);
    float l2 = __ldg(lse + (static_cast<int64_t>(b) * Hq + h) * T + t) * kLog2e;
    if (l2 == -INFINITY) l2 = INFINITY;  // every score is -inf: P = 0, D = 0
    const int begin = window_begin(vis, t), sinks = min(vis.n_sink, begin);
    const int n = t - begin + 1 + sinks;
    float pd = 0.f, pl = 0.f;
    for (int j0 = 0; j0 < n; j0 += 2) {
      uint4 k[2], v[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int j = min(j0 + x, n - 1);
        const int64_t at = (key0 + (j < sinks ? j : begin + j - sinks)) * Hkv + g;
        k[x] = load(K, at);
        v[x] = load(V, at);
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float s = sum16(dot8(q, k[x])), dp = sum16(dot8(go, v[x]));
        const float p = j0 + x < n ? fast_exp2(fmaf(s, scale_log2, -l2)) : 0.f;
        pd = fmaf(p, dp, pd);
        pl += p;
      }
    }
    if (sub == 0 && INFLLMV2_CHECK(status, b * Hkv + g < n_bg && t < T))
      stats[((static_cast<int64_t>(b) * Hkv + g) * n_qt + t / TPT) * 256 + 128 + (t % TPT) * G + h % G] =
          pl == 0.f ? 0.f : pd / pl;
    return;
  }
  const int tile = static_cast<int>(blockIdx.x - few_blocks);
  const int bg = tile / n_qt, qt = tile % n_qt;
  const int b = bg / Hkv, g = bg % Hkv;
  if (!INFLLMV2_CHECK(status, bg < n_bg)) return;
  float* out = stats + static_cast<int64_t>(tile) * 256;
  uint4 o[4], g4[4];
  float l2[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 32 * i + half, t = qt * TPT + r / G;  // row of the tile, its token
    o[i] = g4[i] = make_uint4(0, 0, 0, 0);
    // a row behind the last token, or without a visible key: P = exp2(s - inf) = 0
    l2[i] = INFINITY;
    if (t < T) {
      const int64_t row = (static_cast<int64_t>(b) * T + t) * Hq + g * G + r % G;
      o[i] = load(O, row);
      g4[i] = load(dO, row);
      if (sub == 0) {
        l2[i] = __ldg(lse + (static_cast<int64_t>(b) * Hq + g * G + r % G) * T + t) * kLog2e;
        if (l2[i] == -INFINITY) l2[i] = INFINITY;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 32 * i + half, t = qt * TPT + r / G;
    const float d = sum16(dot8(o[i], g4[i]));
    if (sub == 0) {
      out[r] = l2[i];
      if (t >= few.tokens) out[128 + r] = d;
    }
  }
}

// A row that sees one key alone has P = 1 whatever its score: its dS is zero, set
// so rather than left to two roundings of the same product.  Row 0 always; every
// row with a window of 1 and no sinks.
__device__ __forceinline__ bool always_one_key(const Visible& v) {
  return v.window == 1 && v.n_sink == 0;
}

__device__ __forceinline__ void pack16(const float* v, uint32_t (&pk)[16]) {
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * c], v[2 * c + 1]);
    pk[c] = *reinterpret_cast<uint32_t*>(&b2);
  }
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
struct DkvSmem {
  float stats[2][2][128];
  uint64_t kv_full, kv_empty, q_full[2], q_empty[2], do_full[2], do_empty[2];
  uint64_t s_full, s_read, p_ready, p_free, dp_full, ds_ready, acc_full, acc_free, drain[2];
  uint32_t tmem_base;
  int abort_flag;
  int bg, kt, off;
  long long units;
};
constexpr size_t kDkvSmem = 7 * kTile + sizeof(DkvSmem);
static_assert(kDkvSmem <= 232448, "shared memory");

struct DkvItem {
  int b, g, bg, kt;
  int q0, q1;      // the piece of the query tiles
  bool begins, ends;
  int off;         // units of the key tile before the piece
};

template <int G>
struct DkvWalk {
  static constexpr int TPT = 128 / G;
  const BwdArgs& a;
  long long left;
  int bg, kt, off;
  __device__ DkvWalk(const BwdArgs& args, const DkvSmem& sm)
      : a(args), left(sm.units), bg(sm.bg), kt(sm.kt), off(sm.off) {}
  __device__ __forceinline__ bool next(DkvItem& r) {
    while (left > 0) {
      const QRange q = query_tiles<TPT>(a.vis, a.T, kt);
      const int n = q.q1 - q.q0 + 1;
      const int take = static_cast<int>(min(static_cast<long long>(n + kItemUnits - off), left));
      r.bg = bg;
      r.b = bg / a.Hkv;
      r.g = bg % a.Hkv;
      r.kt = kt;
      r.off = off;
      const int i0 = off, i1 = min(n, off + take);
      r.q0 = q.q0 + i0;
      r.q1 = q.q0 + i1 - 1;
      r.begins = i0 == 0;
      r.ends = i1 == n;
      left -= take;
      off = 0;
      if (++kt == a.n_kt) kt = 0, ++bg;
      if (i0 < i1) return true;
    }
    return false;
  }
};

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    dkv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
               const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const BwdArgs a, DevCtx ctx) {
  constexpr int TPT = 128 / G;
  extern __shared__ uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) report_status(ctx.status, INFLLMV2_STATUS_CHECK);
    return;
  }
  uint8_t* sK = smem_raw;
  uint8_t* sV = sK + kTile;
  uint8_t* sQ = sV + kTile;
  uint8_t* sdO = sQ + 2 * kTile;
  uint8_t* sP = sdO + 2 * kTile;
  DkvSmem& sm = *reinterpret_cast<DkvSmem*>(sP + kTile);
  const int warp = uniform(warp_id()), lane = lane_id();
  if (threadIdx.x == 0) {
    // counts of 2: a commit from each of the two issuers
    mbar_init(&sm.kv_full, 1);
    mbar_init(&sm.kv_empty, 2);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 2);
      mbar_init(&sm.do_full[s], 1);
      mbar_init(&sm.do_empty[s], 2);
      mbar_init(&sm.drain[s], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_read, 8);
    mbar_init(&sm.p_ready, 8);
    mbar_init(&sm.p_free, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.ds_ready, 8);
    mbar_init(&sm.acc_full, 2);
    mbar_init(&sm.acc_free, 8);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == 1) {  // where this CTA's range begins
    const long long w0 = a.per * blockIdx.x;
    const long long total = a.per_bg * a.B * a.Hkv;
    const long long mine = max(0ll, min(a.per, total - w0));
    long long r = w0 % a.per_bg;
    int kt = 0, off = 0;
    if (mine > 0) {
      for (int base = 0; base < a.n_kt; base += 32) {
        const int k = base + lane;
        int u = 0;
        if (k < a.n_kt) {
          const QRange q = query_tiles<TPT>(a.vis, a.T, k);
          u = q.q1 - q.q0 + 1 + kItemUnits;
        }
        long long x = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, r < x);
        if (hit) {
          const int l = __ffs(hit) - 1;
          kt = base + l;
          off = static_cast<int>(r - __shfl_sync(0xffffffffu, x - u, l));
          break;
        }
        r -= __shfl_sync(0xffffffffu, x, 31);
      }
    }
    if (lane == 0) {
      sm.units = mine;
      sm.bg = static_cast<int>(w0 / a.per_bg);
      sm.kt = kt;
      sm.off = off;
    }
  }
  grid_wait();
  grid_launch_next();
  if (threadIdx.x == 0) a.part_item[blockIdx.x] = make_int4(0, 0, 0, 0);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const uint32_t tS = tmem, tdP = tmem + 128, tdV = tmem + 256, tdK = tmem + 384;
  volatile int* abort_flag = &sm.abort_flag;

  // 168 registers a thread at launch: 384 x 168 = 128 x (56 + 224 + 224)
  if (warp < 4) {
    reg_dec<56>();
    DkvWalk<G> walk(a, sm);
    DkvItem it;
    if (warp < 2) {
      // warp 0: K, V and the dO tiles; warp 1: Q tiles and their stats
      if (lane == 0) {
        int ik = 0;
        long long n = 0;
        bool ok = true;
        uint64_t* full = warp == 0 ? sm.do_full : sm.q_full;
        uint64_t* empty = warp == 0 ? sm.do_empty : sm.q_empty;
        while (ok && walk.next(it)) {
          if (warp == 0) {
            if (ik > 0 && !(ok = guarded_wait(&sm.kv_empty, (ik - 1) & 1, ctx, abort_flag))) break;
            mbar_arrive_expect_tx(&sm.kv_full, 2 * kTile);
            for (int h = 0; h < 2; ++h) {
              tma_load_4d(sK + h * 16384, &tmK, &sm.kv_full, 64 * h, it.g, it.kt * kKeyTile, it.b);
              tma_load_4d(sV + h * 16384, &tmV, &sm.kv_full, 64 * h, it.g, it.kt * kKeyTile, it.b);
            }
            ++ik;
          }
          for (int q = it.q0; q <= it.q1; ++q, ++n) {
            const int s = static_cast<int>(n & 1);
            if (n >= 2 && !(ok = guarded_wait(&empty[s], ((n >> 1) & 1) ^ 1, ctx, abort_flag))) break;
            uint8_t* dst = (warp == 0 ? sdO : sQ) + s * kTile;
            mbar_arrive_expect_tx(&full[s], warp == 0 ? kTile : kTile + 1024);
            for (int h = 0; h < 2; ++h)
              tma_load_4d(dst + h * 16384, warp == 0 ? &tmdO : &tmQ, &full[s], 64 * h, it.g * G,
                          q * TPT, it.b);
            if (warp == 1)
              bulk_load(sm.stats[s], a.stats + (static_cast<int64_t>(it.bg) * a.n_qt + q) * 256, 1024,
                        &full[s]);
          }
        }
        if (ik > 0) mbar_wait(&sm.kv_full, (ik - 1) & 1, ctx.wait_ns);
        for (long long q = n - 1; q >= 0 && q >= n - 2; --q)
          mbar_wait(&full[q & 1], (q >> 1) & 1, ctx.wait_ns);
      }
    } else {
      // MMA issuers: warp 2 S(j+1) as soon as the warps have read S(j), then
      // dV(j); warp 3 dK(j), then dP(j+1) over dS(j)
      const uint32_t elect = lane == 0;
      const uint32_t kA = smem_u32(sK), vA = smem_u32(sV), qA = smem_u32(sQ), dA = smem_u32(sdO);
      int ik = 0;
      uint32_t n = 0;  // query tiles before this item
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return warp_wait(bar, phase & 1, ctx, abort_flag);
      };
      if (warp == 2) {
        auto issue_s = [&](uint32_t j) -> bool {
          if (!wait(&sm.q_full[j & 1], j >> 1)) return false;
          if (j > 0 && !wait(&sm.s_read, j - 1)) return false;
          tc_fence_after();
          mma_rows(tS, kA, qA + (j & 1) * kTile, elect);
          commit_if(&sm.s_full, elect);
          commit_if(&sm.q_empty[j & 1], elect);
          return true;
        };
        for (; ok && walk.next(it); ++ik) {
          const uint32_t cnt = it.q1 - it.q0 + 1;
          if (!(ok = wait(&sm.kv_full, ik) && issue_s(n))) break;
          if (ik > 0 && !(ok = wait(&sm.acc_free, ik - 1))) break;
          for (uint32_t i = 0; i < cnt; ++i) {
            const uint32_t j = n + i;
            if (i + 1 < cnt && !(ok = issue_s(j + 1))) break;
            if (!(ok = wait(&sm.do_full[j & 1], j >> 1) && wait(&sm.p_ready, j))) break;
            tc_fence_after();
            mma_rows_cols(tdV, smem_u32(sP), dA + (j & 1) * kTile, i == 0, elect);
            commit_if(&sm.p_free, elect);
            commit_if(&sm.do_empty[j & 1], elect);
          }
          if (!ok) break;
          commit_if(&sm.acc_full, elect);
          commit_if(&sm.kv_empty, elect);
          n += cnt;
        }
      } else {
        auto issue_dp = [&](uint32_t j) -> bool {
          if (!wait(&sm.do_full[j & 1], j >> 1)) return false;
          tc_fence_after();
          mma_rows(tdP, vA, dA + (j & 1) * kTile, elect);
          commit_if(&sm.dp_full, elect);
          commit_if(&sm.do_empty[j & 1], elect);
          return true;
        };
        for (; ok && walk.next(it); ++ik) {
          const uint32_t cnt = it.q1 - it.q0 + 1;
          if (!(ok = wait(&sm.kv_full, ik) && issue_dp(n))) break;
          if (ik > 0 && !(ok = wait(&sm.acc_free, ik - 1))) break;
          for (uint32_t i = 0; i < cnt; ++i) {
            const uint32_t j = n + i;
            if (!(ok = wait(&sm.q_full[j & 1], j >> 1) && wait(&sm.ds_ready, j))) break;
            tc_fence_after();
            mma_cols(tdK, tdP, 64, qA + (j & 1) * kTile, i == 0, elect);
            commit_if(&sm.q_empty[j & 1], elect);
            if (i + 1 < cnt && !(ok = issue_dp(j + 1))) break;
          }
          if (!ok) break;
          commit_if(&sm.acc_full, elect);
          commit_if(&sm.kv_empty, elect);
          n += cnt;
        }
      }
      commit_if(&sm.drain[warp - 2], elect);
      if (lane == 0) mbar_wait(&sm.drain[warp - 2], 0, ctx.wait_ns);
    }
  } else {
    reg_inc<224>();
    DkvWalk<G> walk(a, sm);
    DkvItem it;
    // warpgroup w: the query rows 64 w .. 64 w + 63 (columns) of every tile for
    // all 128 keys (lanes)
    const int w = (warp - 4) >> 2;
    const int key_r = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    long long n = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, long long phase) {
      return warp_wait(bar, static_cast<uint32_t>(phase & 1), ctx, abort_flag);
    };
    for (int ik = 0; ok && walk.next(it); ++ik) {
      const int k0 = it.kt * kKeyTile, key = k0 + key_r;
      for (int q = it.q0; q <= it.q1; ++q, ++n) {
        const int t0 = q * TPT;
        const bool full = t0 >= k0 + kKeyTile - 1 &&
                          (t0 + TPT - 1 < k0 + static_cast<long long>(a.vis.window) ||
                           k0 + kKeyTile <= a.vis.n_sink);
        if (!(ok = wait(&sm.q_full[n & 1], n >> 1))) break;   // the stats
        if (!(ok = wait(&sm.s_full, n))) break;
        tc_fence_after();
        float p[64];
        tmem_ld32(tS + lane_addr + 64 * w, *reinterpret_cast<float(*)[32]>(p));
        tmem_ld32(tS + lane_addr + 64 * w + 32, *reinterpret_cast<float(*)[32]>(p + 32));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_read);
        if (!full) {
          // column c: token t0 + (64 w + c) / G; the key is seen by the tokens
          // lo .. hi-1 of the tile
          const int lo = key - t0;
          const int hi = key < a.vis.n_sink ? TPT : max(0, min(lo + a.vis.window, TPT));
          mask_columns(p, max(lo, 0) * G - 64 * w, hi * G - 64 * w, 0);
        }
        const float4* l4 = reinterpret_cast<const float4*>(&sm.stats[n & 1][0][64 * w]);
        const float4* d4 = reinterpret_cast<const float4*>(&sm.stats[n & 1][1][64 * w]);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 l = l4[c];
          float2 x = fma2(make_float2(p[4 * c], p[4 * c + 1]), sl2, make_float2(-l.x, -l.y));
          float2 y = fma2(make_float2(p[4 * c + 2], p[4 * c + 3]), sl2, make_float2(-l.z, -l.w));
          p[4 * c] = fast_exp2(x.x);
          p[4 * c + 1] = fast_exp2(x.y);
          p[4 * c + 2] = fast_exp2(y.x);
          p[4 * c + 3] = fast_exp2(y.y);
        }
        // P^T, K-major with 128-byte swizzle: row = key, half w = these columns
        if (n > 0 && !(ok = wait(&sm.p_free, n - 1))) break;
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
          pack16(p + 32 * hf, pk);
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(sP + w * 16384 + key_r * 128 +
                                      (((4 * hf + c) ^ (key_r & 7)) * 16)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_ready);
        if (q == 0 && w == 0) {  // token 0's rows see one key
#pragma unroll
          for (int c = 0; c < G && c < 64; ++c) p[c] = 0.f;
        }
        if (!(ok = wait(&sm.dp_full, n))) break;
        tc_fence_after();
        float dp[64];
        tmem_ld32(tdP + lane_addr + 64 * w, *reinterpret_cast<float(*)[32]>(dp));
        tmem_ld32(tdP + lane_addr + 64 * w + 32, *reinterpret_cast<float(*)[32]>(dp + 32));
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float4 d = d4[c];
          const float2 x = mul2(make_float2(p[4 * c], p[4 * c + 1]),
                                add2(make_float2(dp[4 * c], dp[4 * c + 1]), make_float2(-d.x, -d.y)));
          const float2 y = mul2(make_float2(p[4 * c + 2], p[4 * c + 3]),
                                add2(make_float2(dp[4 * c + 2], dp[4 * c + 3]), make_float2(-d.z, -d.w)));
          dp[4 * c] = x.x;
          dp[4 * c + 1] = x.y;
          dp[4 * c + 2] = y.x;
          dp[4 * c + 3] = y.y;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
          pack16(dp + 32 * hf, pk);
          tmem_st16(tdP + lane_addr + 64 * w + 16 * hf, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ds_ready);
      }
      if (!ok) break;
      // the key tile's sums: warpgroup 0 stores dV, 1 dK
      if (!(ok = wait(&sm.acc_full, ik))) break;
      tc_fence_after();
      const bool whole = it.begins && it.ends;
      const float f = w ? (always_one_key(a.vis) ? 0.f : a.scale) : 1.f;
      const uint32_t acc = (w ? tdK : tdV) + lane_addr;
      __nv_bfloat16* out = (w ? a.dK : a.dV) +
                           ((static_cast<int64_t>(it.b) * a.T + key) * a.Hkv + it.g) * kHeadDim;
      const bool store = INFLLMV2_CHECK(ctx.status, it.bg < a.B * a.Hkv && it.kt < a.n_kt &&
                                                        it.q0 >= 0 && it.q1 < a.n_qt);
      const int slot = 2 * blockIdx.x + (it.begins ? 1 : 0);
      float* part = a.part + ((static_cast<int64_t>(slot) * 2 + w) * 128 + key_r) * kHeadDim;
#pragma unroll 1
      for (int c = 0; c < 128; c += 16) {
        float v[16];
        tmem_ld16(acc + c, v);
        tmem_ld_wait();
        uint32_t u[8];
        if (!store) continue;
        if (!whole) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[8 * x + j]);
            store_sector(part + c + 8 * x, u);
          }
        } else if (key < a.T) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j] * f, v[2 * j + 1] * f);
            u[j] = *reinterpret_cast<uint32_t*>(&b2);
          }
          store_sector(out + c, u);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_free);
      if (threadIdx.x == kThreads - 1 && !it.begins && it.ends && store)
        a.part_item[blockIdx.x] =
            make_int4(it.bg, it.kt, static_cast<int>((a.per * blockIdx.x - it.off) / a.per), 1);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Sums the partials of the key tile that CTA c ended (CTA c0, which began it,
// left its piece in slot 2 c0 + 1, the others in slot 2 j), in order.  Blocks
// (c, part of the 2 x 128 x 128 values).
constexpr int kMergeSplit = 32;
__global__ void __launch_bounds__(256) dkv_merge_kernel(const BwdArgs a, int* status) {
  grid_wait();
  const int4 it = a.part_item[blockIdx.x];
  if (it.w == 0) return;
  const int c = blockIdx.x, c0 = it.z;
  if (!INFLLMV2_CHECK(status, c0 >= 0 && c0 < c && it.x < a.B * a.Hkv)) return;
  constexpr int kN = 2 * 128 * 32 / kMergeSplit;  // float4 per block
  for (int i = blockIdx.y * kN + threadIdx.x; i < (blockIdx.y + 1) * kN; i += blockDim.x) {
    const int w = i >> 12, r = (i >> 5) & 127, ch = (i & 31) * 4;
    const int key = it.y * kKeyTile + r;
    if (key >= a.T) continue;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int j = c0; j <= c; ++j) {
      const int slot = 2 * j + (j == c0 ? 1 : 0);
      const float4 x = *reinterpret_cast<const float4*>(
          a.part + ((static_cast<int64_t>(slot) * 2 + w) * 128 + r) * kHeadDim + ch);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    const float f = w ? (always_one_key(a.vis) ? 0.f : a.scale) : 1.f;
    __nv_bfloat162 b0 = __floats2bfloat162_rn(s.x * f, s.y * f);
    __nv_bfloat162 b1 = __floats2bfloat162_rn(s.z * f, s.w * f);
    __nv_bfloat16* out = (w ? a.dK : a.dV) +
                         ((static_cast<int64_t>(it.x / a.Hkv) * a.T + key) * a.Hkv + it.x % a.Hkv) *
                             kHeadDim + ch;
    *reinterpret_cast<uint2*>(out) =
        make_uint2(*reinterpret_cast<uint32_t*>(&b0), *reinterpret_cast<uint32_t*>(&b1));
  }
}

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
constexpr int kDqK = 3, kDqV = 2;  // ring stages: a K tile is read by S and, later, by dQ
struct DqSmem {
  uint64_t q_full, q_empty, k_full[kDqK], k_empty[kDqK], v_full[kDqV], v_empty[kDqV];
  uint64_t s_full[2], dp_full, dp_free, ds_ready[2], dq_full, dq_free, drain[2];
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kDqSmem = (2 + kDqK + kDqV) * kTile + sizeof(DqSmem);

struct DqItem {
  int b, g, qt, t0, n_tok;
  KeyTiles kt;
};

template <int G>
__device__ __forceinline__ DqItem dq_item(const BwdArgs& a, long long k) {
  constexpr int TPT = 128 / G;
  DqItem r;
  const int bgn = a.B * a.Hkv;
  r.qt = a.n_qt - 1 - static_cast<int>(k / bgn);  // the latest (heaviest) tokens first
  const int bg = static_cast<int>(k % bgn);
  r.b = bg / a.Hkv;
  r.g = bg % a.Hkv;
  r.t0 = r.qt * TPT;
  r.n_tok = min(TPT, a.T - r.t0);
  r.kt = key_tiles(a.vis, r.t0, r.t0 + r.n_tok - 1);
  return r;
}

template <int G>
__global__ void __launch_bounds__(kThreads, 1)
    dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmdO,
              const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const BwdArgs a, DevCtx ctx) {
  extern __shared__ uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) report_status(ctx.status, INFLLMV2_STATUS_CHECK);
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* sdO = sQ + kTile;
  uint8_t* sK = sdO + kTile;
  uint8_t* sV = sK + kDqK * kTile;
  DqSmem& sm = *reinterpret_cast<DqSmem*>(sV + kDqV * kTile);
  const int warp = uniform(warp_id()), lane = lane_id();
  const long long n_items = static_cast<long long>(a.B) * a.Hkv * a.n_qt;
  if (threadIdx.x == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);  // both issuers
    for (int s = 0; s < kDqK; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], 1);
    for (int s = 0; s < kDqV; ++s) mbar_init(&sm.v_full[s], 1), mbar_init(&sm.v_empty[s], 1);
    mbar_init(&sm.s_full[0], 1);
    mbar_init(&sm.s_full[1], 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.dp_free, 8);
    // two: dP(j+1) is issued before dS(j) is waited for
    mbar_init(&sm.ds_ready[0], 8);
    mbar_init(&sm.ds_ready[1], 8);
    mbar_init(&sm.dq_full, 1);
    mbar_init(&sm.dq_free, 8);
    mbar_init(&sm.drain[0], 1);
    mbar_init(&sm.drain[1], 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  grid_wait();
  grid_launch_next();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  const uint32_t tS = tmem, tdP = tmem + 256, tdQ = tmem + 384;  // S: two buffers
  volatile int* abort_flag = &sm.abort_flag;

  // 168 registers a thread at launch: 384 x 168 = 128 x (56 + 224 + 224)
  if (warp < 4) {
    reg_dec<56>();
    if (warp < 2) {
      // warp 0: Q, dO and the K tiles; warp 1: V tiles
      if (lane == 0) {
        const int stages = warp == 0 ? kDqK : kDqV;
        uint64_t* full = warp == 0 ? sm.k_full : sm.v_full;
        uint64_t* empty = warp == 0 ? sm.k_empty : sm.v_empty;
        int ik = 0, st = 0;
        uint32_t ph = 0;
        long long n = 0;
        bool ok = true;
        for (long long k = blockIdx.x; ok && k < n_items; k += gridDim.x) {
          const DqItem it = dq_item<G>(a, k);
          if (warp == 0) {
            if (ik > 0 && !(ok = guarded_wait(&sm.q_empty, (ik - 1) & 1, ctx, abort_flag))) break;
            mbar_arrive_expect_tx(&sm.q_full, 2 * kTile);
            for (int h = 0; h < 2; ++h) {
              tma_load_4d(sQ + h * 16384, &tmQ, &sm.q_full, 64 * h, it.g * G, it.t0, it.b);
              tma_load_4d(sdO + h * 16384, &tmdO, &sm.q_full, 64 * h, it.g * G, it.t0, it.b);
            }
            ++ik;
          }
          for (int i = 0; i < it.kt.n; ++i, ++n) {
            if (n >= stages && !(ok = guarded_wait(&empty[st], ph ^ 1, ctx, abort_flag))) break;
            uint8_t* dst = (warp == 0 ? sK : sV) + st * kTile;
            mbar_arrive_expect_tx(&full[st], kTile);
            for (int h = 0; h < 2; ++h)
              tma_load_4d(dst + h * 16384, warp == 0 ? &tmK : &tmV, &full[st], 64 * h, it.g,
                          it.kt.tile(i) * kKeyTile, it.b);
            if (++st == stages) st = 0, ph ^= 1;
          }
        }
        if (ik > 0) mbar_wait(&sm.q_full, (ik - 1) & 1, ctx.wait_ns);
        for (long long q = n - 1; q >= 0 && q >= n - stages; --q)
          mbar_wait(&full[q % stages], (q / stages) & 1, ctx.wait_ns);
      }
    } else {
      // MMA issuers: warp 2 S(j+1), then dQ(j) once dS(j) is written; warp 3 dP
      const uint32_t elect = lane == 0;
      const uint32_t qA = smem_u32(sQ), dA = smem_u32(sdO), kA = smem_u32(sK), vA = smem_u32(sV);
      int ik = 0;
      uint32_t n = 0;  // key tiles before this item
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t phase) {
        return warp_wait(bar, phase & 1, ctx, abort_flag);
      };
      if (warp == 2) {
        auto issue_s = [&](uint32_t j) -> bool {
          const uint32_t s = j % kDqK;
          if (!wait(&sm.k_full[s], j / kDqK)) return false;
          tc_fence_after();
          mma_rows(tS + (j & 1) * 128, qA, kA + s * kTile, elect);
          commit_if(&sm.s_full[j & 1], elect);
          return true;
        };
        for (long long k = blockIdx.x; ok && k < n_items; k += gridDim.x, ++ik) {
          const DqItem it = dq_item<G>(a, k);
          const uint32_t cnt = it.kt.n;
          if (!(ok = wait(&sm.q_full, ik) && issue_s(n))) break;
          if (cnt == 1) commit_if(&sm.q_empty, elect);  // S has read Q
          if (ik > 0 && !(ok = wait(&sm.dq_free, ik - 1))) break;
          for (uint32_t i = 0; i < cnt; ++i) {
            const uint32_t j = n + i, s = j % kDqK;
            if (i + 1 < cnt && !(ok = issue_s(j + 1))) break;
            if (i + 2 == cnt) commit_if(&sm.q_empty, elect);
            if (!(ok = wait(&sm.ds_ready[j & 1], j >> 1))) break;
            tc_fence_after();
            mma_cols(tdQ, tS + (j & 1) * 128, 64, kA + s * kTile, i == 0, elect);
            commit_if(&sm.k_empty[s], elect);
          }
          if (!ok) break;
          commit_if(&sm.dq_full, elect);
          n += cnt;
        }
      } else {
        for (long long k = blockIdx.x; ok && k < n_items; k += gridDim.x, ++ik) {
          const DqItem it = dq_item<G>(a, k);
          const uint32_t cnt = it.kt.n;
          if (!(ok = wait(&sm.q_full, ik))) break;
          for (uint32_t i = 0; i < cnt; ++i) {
            const uint32_t j = n + i, s = j % kDqV;
            if (!(ok = wait(&sm.v_full[s], j / kDqV))) break;
            // the warps have read dP of the tile before
            if (j > 0 && !(ok = wait(&sm.dp_free, j - 1))) break;
            tc_fence_after();
            mma_rows(tdP, dA, vA + s * kTile, elect);
            commit_if(&sm.dp_full, elect);
            commit_if(&sm.v_empty[s], elect);
          }
          if (!ok) break;
          commit_if(&sm.q_empty, elect);  // dP has read dO
          n += cnt;
        }
      }
      commit_if(&sm.drain[warp - 2], elect);
      if (lane == 0) mbar_wait(&sm.drain[warp - 2], 0, ctx.wait_ns);
    }
  } else {
    reg_inc<224>();
    // warpgroup w: the keys 64 w .. 64 w + 63 (columns) of every tile for all
    // 128 query rows (lanes)
    const int w = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
    long long n = 0;
    int ik = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, long long phase) {
      return warp_wait(bar, static_cast<uint32_t>(phase & 1), ctx, abort_flag);
    };
    for (long long k = blockIdx.x; ok && k < n_items; k += gridDim.x, ++ik) {
      const DqItem it = dq_item<G>(a, k);
      const int t = it.t0 + r / G;
      const int wb = window_begin(a.vis, t);
      const float* st =
          a.stats + ((static_cast<int64_t>(it.b) * a.Hkv + it.g) * a.n_qt + it.qt) * 256 + r;
      const float l2 = __ldg(st), D = __ldg(st + 128);
      const float2 ml = make_float2(-l2, -l2), mD = make_float2(-D, -D);
      for (int i = 0; i < it.kt.n; ++i, ++n) {
        const int lo = it.kt.tile(i) * kKeyTile + 64 * w;
        if (!(ok = wait(&sm.s_full[n & 1], n >> 1))) break;
        tc_fence_after();
        const uint32_t s_addr = tS + (n & 1) * 128 + lane_addr + 64 * w;
        float p[64];
        tmem_ld32(s_addr, *reinterpret_cast<float(*)[32]>(p));
        tmem_ld32(s_addr + 32, *reinterpret_cast<float(*)[32]>(p + 32));
        tmem_ld_wait();
        const bool full = lo + 63 <= t && (lo >= wb || lo + 64 <= a.vis.n_sink);
        if (__any_sync(0xffffffffu, !full)) {
          mask_columns(p, wb - lo, t - lo + 1, a.vis.n_sink - lo);
        }
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 x = fma2(make_float2(p[c], p[c + 1]), sl2, ml);
          p[c] = fast_exp2(x.x);
          p[c + 1] = fast_exp2(x.y);
        }
        if (!(ok = wait(&sm.dp_full, n))) break;
        tc_fence_after();
        float dp[64];
        tmem_ld32(tdP + lane_addr + 64 * w, *reinterpret_cast<float(*)[32]>(dp));
        tmem_ld32(tdP + lane_addr + 64 * w + 32, *reinterpret_cast<float(*)[32]>(dp + 32));
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.dp_free);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float2 x = mul2(make_float2(p[c], p[c + 1]), add2(make_float2(dp[c], dp[c + 1]), mD));
          dp[c] = x.x;
          dp[c + 1] = x.y;
        }
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pk[16];
          pack16(dp + 32 * hf, pk);
          tmem_st16(s_addr + 16 * hf, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ds_ready[n & 1]);
      }
      if (!ok) break;
      if (!(ok = wait(&sm.dq_full, ik))) break;
      tc_fence_after();
      const float f = t == 0 || always_one_key(a.vis) ? 0.f : a.scale;
      __nv_bfloat16* out = a.dQ + ((static_cast<int64_t>(it.b) * a.T + t) * a.Hq + it.g * G + r % G) *
                                      kHeadDim + 64 * w;
#pragma unroll 1
      for (int c = 0; c < 64; c += 16) {
        float v[16];
        tmem_ld16(tdQ + lane_addr + 64 * w + c, v);
        tmem_ld_wait();
        if (t < a.T && INFLLMV2_CHECK(ctx.status, it.qt >= 0 && it.b < a.B)) {
          uint32_t u[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * j] * f, v[2 * j + 1] * f);
            u[j] = *reinterpret_cast<uint32_t*>(&b2);
          }
          store_sector(out + c, u);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.dq_free);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

int query_tile_count(const Geometry& g) {
  const int tpt = 128 / g.G;
  return (g.T + tpt - 1) / tpt;
}

size_t stats_bytes(const Geometry& g) {
  return align256(static_cast<size_t>(g.B) * g.Hkv * query_tile_count(g) * 1024);
}

size_t part_bytes() { return static_cast<size_t>(sm_count()) * 2 * 2 * 128 * kHeadDim * 4; }

template <int G>
int launch_g(const void* Q, const void* K, const void* V, const void* O, const float* lse,
             const void* dO, BwdArgs a,
             const CUtensorMap& tq, const CUtensorMap& tdo, const CUtensorMap& tk,
             const CUtensorMap& tv, const DevCtx& ctx, cudaStream_t st) {
  constexpr int TPT = 128 / G;
  const int sms = sm_count();
  a.per_bg = 0;
  for (int kt = 0; kt < a.n_kt; ++kt) {
    const QRange q = query_tiles<TPT>(a.vis, a.T, kt);
    a.per_bg += q.q1 - q.q0 + 1 + kItemUnits;
  }
  const long long total = a.per_bg * a.B * a.Hkv;
  a.per = (total + sms - 1) / sms;
  if (a.per < kMinUnits) a.per = kMinUnits;
  const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * a.n_qt;
  // visible keys of the last token: no row has more
  const int most = a.T - window_begin(a.vis, a.T - 1) +
                   (a.vis.n_sink < window_begin(a.vis, a.T - 1) ? a.vis.n_sink
                                                                : window_begin(a.vis, a.T - 1));
  FewRows few;
  few.tokens = most <= kFewKeys || a.T < kFewKeys ? a.T : kFewKeys;
  few.rows = static_cast<int64_t>(a.B) * few.tokens * a.Hq;
  const int64_t stat_blocks = items + (few.rows + 31) / 32;
  if (stat_blocks > INT32_MAX)
    return INFLLMV2_ERR_UNSUPPORTED;  // beyond any GPU's memory
  stats_kernel<G><<<static_cast<unsigned>(stat_blocks), 512, 0, st>>>(
      static_cast<const __nv_bfloat16*>(Q), static_cast<const __nv_bfloat16*>(K),
      static_cast<const __nv_bfloat16*>(V), static_cast<const __nv_bfloat16*>(O),
      static_cast<const __nv_bfloat16*>(dO), lse, const_cast<float*>(a.stats), a.T, a.Hkv, a.n_qt,
      a.vis, a.scale_log2, few, a.B * a.Hkv, ctx.status);
  static std::atomic<uint64_t> kv_set{0}, q_set{0};
  if (int e = set_smem_limit(dkv_kernel<G>, kDkvSmem, kv_set)) return e;
  if (int e = set_smem_limit(dq_kernel<G>, kDqSmem, q_set)) return e;
  const int ctas = static_cast<int>((total + a.per - 1) / a.per);
  if (cudaGetLastError() != cudaSuccess) return INFLLMV2_ERR_CUDA;
  if (int e = launch_waiting(dkv_kernel<G>, ctas, kThreads, kDkvSmem, st, tq, tdo, tk, tv, a, ctx))
    return e;
  const unsigned q_ctas = static_cast<unsigned>(items < sms ? items : sms);
  if (int e = launch_waiting(dq_kernel<G>, q_ctas, kThreads, kDqSmem, st, tq, tdo, tk, tv, a, ctx))
    return e;
  return launch_waiting(dkv_merge_kernel, dim3(ctas, kMergeSplit), 256, 0, st, a, ctx.status);
}

// [B, T, heads, 128] bf16, boxes of 64 channels x box_heads x box_rows.
int bthd_map(CUtensorMap* tm, const void* x, const Geometry& g, int heads, int box_heads,
             int box_rows) {
  const uint64_t row = static_cast<uint64_t>(heads) * kHeadDim * 2;
  const uint64_t dims[4] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(g.T), static_cast<uint64_t>(g.B)};
  const uint64_t strides[3] = {static_cast<uint64_t>(kHeadDim) * 2, row, row * g.T};
  const uint32_t box[4] = {64u, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_rows),
                           1u};
  return make_tmap_bf16_4d(tm, x, dims, strides, box);
}

}  // namespace

// Row statistics, dK/dV partials, cut key tiles.
size_t window_bwd_ws_bytes(const Geometry& g) {
  return stats_bytes(g) + part_bytes() + static_cast<size_t>(sm_count()) * sizeof(int4);
}

int launch_window_bwd(const Geometry& g, int window, int n_sink, const void* Q, const void* K,
                      const void* V, const void* O, const float* lse, const void* dO, void* dQ,
                      void* dK, void* dV, void* ws, const DevCtx& ctx, cudaStream_t st) {
  BwdArgs a{};
  a.vis = visible(window, n_sink);
  a.B = g.B;
  a.T = g.T;
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.n_qt = query_tile_count(g);
  a.n_kt = (g.T + kKeyTile - 1) / kKeyTile;
  a.scale = g.scale;
  a.scale_log2 = g.scale_log2;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.stats = reinterpret_cast<float*>(w);
  a.part = reinterpret_cast<float*>(w + stats_bytes(g));
  a.part_item = reinterpret_cast<int4*>(w + stats_bytes(g) + part_bytes());
  a.dQ = static_cast<__nv_bfloat16*>(dQ);
  a.dK = static_cast<__nv_bfloat16*>(dK);
  a.dV = static_cast<__nv_bfloat16*>(dV);
  CUtensorMap tq, tdo, tk, tv;
  if (int e = bthd_map(&tq, Q, g, g.Hq, g.G, 128 / g.G)) return e;
  if (int e = bthd_map(&tdo, dO, g, g.Hq, g.G, 128 / g.G)) return e;
  if (int e = bthd_map(&tk, K, g, g.Hkv, 1, kKeyTile)) return e;
  if (int e = bthd_map(&tv, V, g, g.Hkv, 1, kKeyTile)) return e;
  switch (g.G) {
    case 1: return launch_g<1>(Q, K, V, O, lse, dO, a, tq, tdo, tk, tv, ctx, st);
    case 2: return launch_g<2>(Q, K, V, O, lse, dO, a, tq, tdo, tk, tv, ctx, st);
    case 4: return launch_g<4>(Q, K, V, O, lse, dO, a, tq, tdo, tk, tv, ctx, st);
    case 8: return launch_g<8>(Q, K, V, O, lse, dO, a, tq, tdo, tk, tv, ctx, st);
    case 16: return launch_g<16>(Q, K, V, O, lse, dO, a, tq, tdo, tk, tv, ctx, st);
    default: return INFLLMV2_ERR_UNSUPPORTED;
  }
}

}  // namespace infllmv2
