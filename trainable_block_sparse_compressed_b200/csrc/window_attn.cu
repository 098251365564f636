// window_attn.cu -- causal softmax attention with a sliding window and sinks,
// over contiguous keys (training, prefill) or over a paged cache (chunks of
// new tokens and single tokens).
//
//   keys(t) = { c <= t : c > t - window or c < n_sink },
//   O[t] = sum_{c in keys(t)} softmax_c(scale q_t . K_c) V_c,
//   lse[t] = log sum_{c in keys(t)} exp(scale q_t . K_c);
//   no visible key: O = 0, lse = -inf.
//
// A query tile is 128 rows: 128/G consecutive tokens x the G query heads of
// one group.  A work item is up to two query tiles of one (sequence, kv head)
// against a list of 128-key tiles: the tiles of the sinks, then those of the
// window (window.cuh), so keys outside both are not read.  Two streams share
// the CTA, each with its own softmax warpgroup, its own MMA issuer, 128 tensor
// memory columns for S and P and 128 for O:
//
//   pair    two query tiles: stream w runs query tile w over every key tile,
//           so a loaded K/V tile serves 256 rows;
//   single  one query tile (the last of a sequence, single tokens): stream w
//           takes every second key tile, and the two results are merged.
//
// A stream's S columns are two regions of 64 keys' scores.  Key tile j has its
// first half in region j % 2; P(j), 64 columns of bf16 pairs, goes over it, and
// the other region takes S(j+1)'s first half as soon as S(j) has been read, so
// the warps go on to tile j+1 while the tensor core runs P V(j) and then S(j+1)'s
// second half over P(j).  Stream 1 of a pair starts half a tile behind stream 0,
// so that one forms exponentials while the other's products run (T=8192, window
// 128: 63.0 -> 58.8 us, 256: 76.6 -> 69.9, 512: 102 -> 95).  The exponentials
// take the reference maximum of the keys before them; the maximum of their own
// keys is formed beside them, and only where it passes the reference by more
// than 8 (log2 units) is the reference raised, O_w rescaled and the half formed
// again.  P = exp2(s - m) is rounded to bf16 for the tensor core (2^-9 relative
// on average, the size of the output's own rounding); its sum is kept in fp32.
//
// What bounds it (clock stamps, pair items): a softmax warp spends ~1000 cycles
// on the exponentials of 64 keys (512 on the special-function unit alone, which
// two warps of a scheduler share) and ~700 on loads, stores and barriers; the
// tensor core's four products are done in ~2500 of the ~3500 cycles of a tile.
// In a long run the power cap lowers the clock to ~1.4 GHz.  One B200, calls in a
// row: T=32768, 32 heads, window 4096, 64 sinks 2.0-2.1 ms (1.0 PFLOP/s).  Single
// tokens are bound by HBM: 16 x 131072 tokens, 2.15 GB, 340-370 us from card to
// card (5.8-6.3 TB/s).
// Tried and slower: S in one 128-wide product per tile (P V, S and the softmax
// of a stream then wait for each other, 4350 cycles; with the streams taking
// turns at the exponentials), two softmax warpgroups per stream (a barrier per
// tile for the common reference), P V in two halves, a V ring of two stages
// (3 %), a quarter or an eighth of the exponentials by a polynomial (2-5 %: the
// issue slots are no freer than the special-function unit).
//
// Warps: 0 loads Q and K, 1 V (TMA, rings of 2 K and 3 V stages of 32 KB),
// 2 and 3 issue stream 0's and 1's MMAs, 4-7 and 8-11 are the softmax.
#include "window.cuh"

namespace infllmv2 {
namespace {

constexpr int kKStages = 2, kVStages = 3;
constexpr int kTileBytes = 128 * 256;   // 128 rows x 128 channels bf16
constexpr int kThreads = 384;           // 4 role warps, 2 x 4 softmax warps
constexpr float kSlack = 8.0f;          // log2 units
constexpr float kLn2 = 0.6931471805599453f;
// Windows of up to this many keys take a variant that leaves out the halves of
// key tiles that no row of a warp sees (half of all halves at 128) and writes
// whole lines of O.  T=8192, 32 heads, with and without: window 128 54.1 and 58.8
// us, 256 67.5 and 69.9, 512 94 and 94, 2048 260 and 250, 4096 (T=32768) 2050 and
// 2000: both cost a long item more than its few edge tiles save.
constexpr int kNarrow = 256;
// Work units of the paged schedule: an item costs its key tiles plus this for
// its query load, pipeline fill and epilogue.
constexpr int kItemUnits = 2;
// A CTA of the paged schedule takes at least this many units: a key tile and its
// item's share.  With 2 the joins of long items cost more (one sequence of 8192
// tokens: 16.4 -> 17.8 us), with 4 short ones wait longer (one of 100 tokens:
// 9.9 -> 13.1 us).
constexpr int kMinUnits = 3;
constexpr int kSlotRows = 256;          // rows of a partial result

struct FwdArgs {
  __nv_bfloat16* O;       // [rows, Hq, 128]
  float* lse;             // contiguous: [B, Hq, T]; paged: [rows, Hq]
  Visible vis;
  int Hq, Hkv;
  int item_tiles;         // query tiles per item: 2 or 1
  float scale_log2;
  int B, T;               // contiguous
  // paged
  const int32_t* table;   // [n_seqs, max_pages]
  const int32_t* cu_q;    // [n_seqs + 1]
  const int32_t* seqlens; // [n_seqs] keys, the new tokens' included
  int n_seqs, max_pages, n_pages, page, n_tokens;
  float* part;            // [2 * CTAs][256][128] partial outputs (normalised)
  float* part_lse;        // [2 * CTAs][256] their log2 sums
  int4* part_item;        // [CTAs] (first row, rows, first CTA, head) of the item a CTA ends
};

struct FwdSmem {
  uint64_t q_full, q_empty;
  uint64_t k_full[kKStages], k_empty[kKStages], v_full[kVStages], v_empty[kVStages];
  // by stream; s_full by half of the key tile too
  uint64_t s_full[2][2], s_read[2], turn, p_full[2], pv_done[2], o_full[2], o_free[2], drain[2];
  uint32_t tmem_base;
  int abort_flag;
  // the paged schedule's start: units to do, then where
  long long units, start, per;
  int seq, g, q, off;
  long long scan[kThreads / 32 + 1];
  float xch[2][2][128];   // single items: each stream's (m, l) per row
};

constexpr size_t kFwdSmem = 2 * kTileBytes + (kKStages + kVStages) * kTileBytes + sizeof(FwdSmem);
static_assert(kFwdSmem <= 232448, "shared memory");

struct FwdItem {
  int b, g;          // sequence, kv head
  int tok0, n_tok;   // contiguous: token of the sequence; paged: row of Q
  int t0;            // position of the first token
  int pair;
  KeyTiles kt;
  int k0, k1;        // the piece of the key tile list
};

struct SeqLens {
  int row0, n_q, t0;  // first row, new tokens, position of the first
  int n_past;         // rows behind them whose positions lie past the table
};

// Lengths of sequence i with every value brought into range: nothing that the
// arrays hold leads outside Q, O, lse or the table.
__device__ __forceinline__ SeqLens seq_lens(const FwdArgs& a, int i) {
  SeqLens s;
  const int r0 = __ldg(a.cu_q + i), r1 = __ldg(a.cu_q + i + 1);
  const int c0 = max(0, min(r0, a.n_tokens)), c1 = max(0, min(r1, a.n_tokens));
  // (rows past n_tokens are cut, the others keep their positions)
  const long long len = min(max(static_cast<long long>(r1) - r0, 0ll), 1ll << 28);
  s.t0 = max(0, min(__ldg(a.seqlens + i), 1 << 30)) - static_cast<int>(len);
  s.row0 = c0;
  const int rows = max(0, c1 - c0);
  s.n_q = max(0, min(rows, a.max_pages * a.page - s.t0));
  s.n_past = rows - s.n_q;
  return s;
}

// Walks this CTA's work in the same order in every role.
template <int G, bool PAGED>
struct Walk {
  static constexpr int TPT = 128 / G;
  const FwdArgs& a;
  int it;                       // tokens per item
  // contiguous: the query item and (batch, head), and a CTA stride's steps
  int qi, bg, dq, dbg, bgn;
  // paged
  long long left;
  int seq, g, q, off;
  SeqLens s;

  __device__ Walk(const FwdArgs& args, const FwdSmem& sm) : a(args) {
    it = a.item_tiles * TPT;
    if (PAGED) {
      left = sm.units;
      seq = sm.seq, g = sm.g, q = sm.q, off = sm.off;
      if (left > 0) s = seq_lens(a, seq);
    } else {
      // the latest (heaviest) tokens first; CTAs of one wave share their keys
      bgn = a.B * a.Hkv;
      qi = (a.T + it - 1) / it - 1 - static_cast<int>(blockIdx.x) / bgn;
      bg = static_cast<int>(blockIdx.x) % bgn;
      dq = static_cast<int>(gridDim.x) / bgn;
      dbg = static_cast<int>(gridDim.x) % bgn;
    }
  }

  __device__ __forceinline__ void fill(FwdItem& r, int first, int n_q, int t_first) const {
    r.n_tok = min(it, n_q - first);
    r.t0 = t_first + first;
    r.pair = r.n_tok > TPT;
    r.kt = key_tiles(a.vis, r.t0, r.t0 + r.n_tok - 1);
  }

  __device__ __forceinline__ bool next(FwdItem& r) {
    if constexpr (!PAGED) {
      if (qi < 0) return false;
      r.b = bg / a.Hkv;
      r.g = bg % a.Hkv;
      r.tok0 = qi * it;
      fill(r, r.tok0, a.T, 0);
      r.k0 = 0;
      r.k1 = r.kt.n;
      qi -= dq;
      bg += dbg;
      if (bg >= bgn) bg -= bgn, --qi;
      return true;
    } else {
    while (left > 0) {
      fill(r, q * it, s.n_q, s.t0);
      r.b = seq;
      r.g = g;
      r.tok0 = s.row0 + q * it;
      const int units = r.kt.n + kItemUnits;
      const int take = static_cast<int>(min(static_cast<long long>(units - off), left));
      r.k0 = off;
      r.k1 = min(r.kt.n, off + take);
      left -= take;
      off = 0;
      if (left > 0) {  // the item is done: on to the next
        if ((q + 1) * it < s.n_q) {
          ++q;
        } else {
          q = 0;
          if (++g == a.Hkv) {
            g = 0;
            do {
              if (++seq >= a.n_seqs) {
                left = 0;
                break;
              }
              s = seq_lens(a, seq);
            } while (s.n_q == 0);
          }
        }
      }
      if (r.k0 < r.k1) return true;
    }
    return false;
    }
  }
};

// sum_{k < n} floor(max(x + k STEP, 0) / 128) for a STEP that divides 128 or is a
// multiple of it.
template <int STEP>
__device__ long long tile_sum(long long x, long long n) {
  static_assert(kKeyTile == 128 && (128 % STEP == 0 || STEP % 128 == 0), "steps");
  if (x < 0) {  // the terms below zero
    const long long k = (-x + STEP - 1) / STEP;
    n -= k;
    x += k * STEP;
  }
  if (n <= 0) return 0;
  const long long whole = n * (x / 128);
  if constexpr (STEP >= 128) {
    return whole + STEP / 128 * (n * (n - 1) / 2);
  } else {
    // + sum_{k < n} floor((y + k) / p), y < p: u whole groups of p equal terms
    constexpr int p = 128 / STEP;
    const long long m = x % 128 / STEP + n, u = m / p;
    return whole + p * (u * (u - 1) / 2) + (m - u * p) * u;
  }
}

// Units of the first n items of one kv head, all of IT tokens: an item has hi -
// lo + min(sink tiles, lo) + 1 = hi - max(lo - sink tiles, 0) + 1 key tiles.
template <int IT>
__device__ long long units_before(const Visible& v, int t0, int n) {
  if (n <= 0) return 0;
  const long long sinks = (v.n_sink + kKeyTile - 1) / kKeyTile;
  return tile_sum<IT>(static_cast<long long>(t0) + IT - 1, n) -
         tile_sum<IT>(t0 + 1ll - v.window - kKeyTile * sinks, n) + n * (1ll + kItemUnits);
}

// Units of one kv head of a sequence: its last item may be shorter.  (In closed
// form: counted item by item, a chunk of 8192 tokens under a window of 128 took
// 125 us instead of 76, one of 32768 tokens 540 instead of 335.)
template <int IT>
__device__ long long head_units(const FwdArgs& a, const SeqLens& s) {
  if (s.n_q == 0) return 0;
  const int last = (s.n_q - 1) / IT;
  return units_before<IT>(a.vis, s.t0, last) +
         key_tiles(a.vis, s.t0 + last * IT, s.t0 + s.n_q - 1).n + kItemUnits;
}

// The rows of tokens that found no place in the table: O = 0, lse = -inf.  One
// thread of each CTA calls it, which takes every gridDim.x-th row.
__device__ __forceinline__ void no_place(const FwdArgs& a, const SeqLens& s) {
  for (int r = s.n_q + blockIdx.x; r < s.n_q + s.n_past; r += gridDim.x) {
    const int64_t at = (static_cast<int64_t>(s.row0) + r) * a.Hq;
    uint4* o = reinterpret_cast<uint4*>(a.O + at * kHeadDim);
    for (int c = 0; c < a.Hq * (kHeadDim / 8); ++c) o[c] = make_uint4(0, 0, 0, 0);
    for (int h = 0; h < a.Hq; ++h) a.lse[at + h] = -INFINITY;
  }
}

// The paged schedule: the units of all items in a row (sequence, head, query
// tiles) are cut into equal ranges, one per CTA; an item cut by a range's end
// gets partial results that the merge kernel joins.  Every CTA derives its own
// range from the lengths.
template <int G>
__device__ void paged_schedule(const FwdArgs& a, FwdSmem& sm) {
  constexpr int IT = 2 * (128 / G);  // tokens of two query tiles
  const int lane = lane_id(), warp = warp_id();
  long long total = 0, mine0 = 0;  // mine0: the first strip's sequence of this thread
  for (int i0 = 0; i0 < a.n_seqs; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    if (i < a.n_seqs) {
      const SeqLens s = seq_lens(a, i);
      const long long u = a.Hkv * head_units<IT>(a, s);
      if (i0 == 0) mine0 = u;
      total += u;
      if (s.n_past > 0) no_place(a, s);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) sm.scan[warp] = total;
  __syncthreads();
  total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += sm.scan[w];
  const long long per = max((total + gridDim.x - 1) / gridDim.x, static_cast<long long>(kMinUnits));
  const long long w0 = per * blockIdx.x;
  const long long mine = max(0ll, min(per, total - w0));
  if (threadIdx.x == 0) sm.per = per, sm.units = mine, sm.seq = sm.g = sm.q = sm.off = 0;
  __syncthreads();
  if (mine == 0) return;
  // the sequence that holds unit w0
  long long base = 0;
  for (int i0 = 0; i0 < a.n_seqs && base <= w0; i0 += kThreads) {
    const int i = i0 + threadIdx.x;
    const long long u = i0 == 0 ? mine0
                        : i < a.n_seqs ? a.Hkv * head_units<IT>(a, seq_lens(a, i)) : 0;
    long long x = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) sm.scan[warp] = x;
    __syncthreads();
    long long before = base;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sm.scan[w];
      base += sm.scan[w];
    }
    before += x - u;
    if (before <= w0 && w0 < before + u) {
      sm.seq = i;
      sm.start = w0 - before;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const SeqLens s = seq_lens(a, sm.seq);
    const long long hu = head_units<IT>(a, s);
    sm.g = static_cast<int>(sm.start / hu);
    const long long r = sm.start - sm.g * hu;
    int q = 0, end = (s.n_q - 1) / IT;  // the last item that starts at or before r
    while (q < end) {
      const int mid = q + (end - q + 1) / 2;
      if (units_before<IT>(a.vis, s.t0, mid) <= r) q = mid; else end = mid - 1;
    }
    sm.q = q;
    sm.off = static_cast<int>(r - units_before<IT>(a.vis, s.t0, q));
  }
}

template <int G, bool PAGED, bool NARROW>
__global__ void __launch_bounds__(kThreads, 1)
    window_attn_kernel(const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const FwdArgs a, DevCtx ctx) {
  constexpr int TPT = 128 / G;
  extern __shared__ uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {  // 128-byte swizzled tiles
    if (threadIdx.x == 0) report_status(ctx.status, INFLLMV2_STATUS_CHECK);
    return;
  }
  uint8_t* sQ = smem_raw;
  uint8_t* sK = sQ + 2 * kTileBytes;
  uint8_t* sV = sK + kKStages * kTileBytes;
  FwdSmem& sm = *reinterpret_cast<FwdSmem*>(sV + kVStages * kTileBytes);
  const int warp = uniform(warp_id()), lane = lane_id();

  if (threadIdx.x == 0) {
    mbar_init(&sm.turn, 4);
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);
    for (int s = 0; s < kKStages; ++s) mbar_init(&sm.k_full[s], 1), mbar_init(&sm.k_empty[s], 2);
    for (int s = 0; s < kVStages; ++s) mbar_init(&sm.v_full[s], 1), mbar_init(&sm.v_empty[s], 2);
    for (int w = 0; w < 2; ++w) {
      mbar_init(&sm.s_full[w][0], 1);
      mbar_init(&sm.s_full[w][1], 1);
      mbar_init(&sm.s_read[w], 4);
      mbar_init(&sm.p_full[w], 4);
      mbar_init(&sm.pv_done[w], 1);
      mbar_init(&sm.o_full[w], 1);
      mbar_init(&sm.o_free[w], 8);
      mbar_init(&sm.drain[w], 1);
    }
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (PAGED) {
    grid_launch_next();  // the merge's blocks come as soon as SMs are free
    paged_schedule<G>(a, sm);
    if (threadIdx.x == 0) a.part_item[blockIdx.x] = make_int4(0, 0, 0, 0);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;

  // 168 registers a thread at launch: 384 x 168 = 128 x (56 + 224 + 224)
  if (warp < 4) {
    reg_dec<56>();
  Walk<G, PAGED> walk(a, sm);
  FwdItem item;
  if (warp < 2) {
    // ------------------------------ producers -----------------------------
    const bool v_role = warp == 1;
    const CUtensorMap* tm = v_role ? &tmV : &tmK;
    if (lane == 0) {
      tma_prefetch_desc(tm);
      if (!v_role) tma_prefetch_desc(&tmQ);
    }
    const int stages = v_role ? kVStages : kKStages;
    uint64_t* full = v_role ? sm.v_full : sm.k_full;
    uint64_t* empty = v_role ? sm.v_empty : sm.k_empty;
    uint8_t* ring = v_role ? sV : sK;
    int ik = 0, st = 0;
    uint32_t ph = 0;            // parity of the ring's current round
    long long n = 0;            // tiles issued
    bool ok = true;
    while (ok && walk.next(item)) {
      if (!v_role) {
        if (ik > 0 && !(ok = warp_wait(&sm.q_empty, (ik - 1) & 1, ctx, abort_flag))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full, (1 + item.pair) * kTileBytes);
          for (int x = 0; x <= item.pair; ++x)
            for (int h = 0; h < 2; ++h)
              tma_load_4d(sQ + x * kTileBytes + h * 16384, &tmQ, &sm.q_full, 64 * h, item.g * G,
                          item.tok0 + x * TPT, PAGED ? 0 : item.b);
        }
        ++ik;
      }
      const int t_last = item.t0 + item.n_tok - 1;
      const int w_begin = window_begin(a.vis, max(item.t0, 0));
      // paged: lane l takes the l-th page of a tile, its id loaded a tile ahead
      const int ppt = PAGED ? kKeyTile / a.page : 1;
      const int32_t* row = PAGED ? a.table + static_cast<int64_t>(item.b) * a.max_pages : nullptr;
      auto needs = [&](int i) -> bool {  // the page has a visible key
        const int col = item.kt.tile(i) * ppt + lane;
        const int c0 = col * a.page;
        return i < item.k1 && lane < ppt && col < a.max_pages && c0 <= t_last &&
               (c0 + a.page > w_begin || c0 < a.vis.n_sink);
      };
      auto page_id = [&](int i, bool needed) -> int {
        return needed ? __ldg(row + item.kt.tile(i) * ppt + lane) : 0;
      };
      bool next_need = PAGED && needs(item.k0);
      int next_id = PAGED ? page_id(item.k0, next_need) : 0;
      for (int i = item.k0; i < item.k1; ++i, ++n) {
        const int id = next_id;
        const bool need = next_need;
        if (PAGED) next_need = needs(i + 1), next_id = page_id(i + 1, next_need);
        if (n >= stages && !(ok = warp_wait(&empty[st], ph ^ 1, ctx, abort_flag))) break;
        uint8_t* dst = ring + st * kTileBytes;
        if (PAGED) {
          const uint32_t box = static_cast<uint32_t>(a.page) * 128;
          const uint32_t cnt = __popc(__ballot_sync(0xffffffffu, need));
          if (lane == 0) mbar_arrive_expect_tx(&full[st], cnt * 2 * box);
          __syncwarp();
          if (need) {
            // any id outside the pool counts as -1: a page in front of the tensor,
            // of which the copies read zeros
            const bool bad = id < 0 || id >= a.n_pages;
            if (bad) report_status(ctx.status, INFLLMV2_STATUS_BAD_PAGE);
            for (int h = 0; h < 2; ++h)
              tma_load_4d(dst + h * 16384 + lane * box, tm, &full[st], 64 * h, item.g, 0,
                          bad ? -1 : id);
          }
        } else if (lane == 0) {
          mbar_arrive_expect_tx(&full[st], kTileBytes);
          for (int h = 0; h < 2; ++h)
            tma_load_4d(dst + h * 16384, tm, &full[st], 64 * h, item.g,
                        item.kt.tile(i) * kKeyTile, item.b);
        }
        if (++st == stages) st = 0, ph ^= 1;
      }
    }
    // never leave with copies of this CTA in flight
    if (!v_role && ik > 0) mbar_wait(&sm.q_full, (ik - 1) & 1, ctx.wait_ns);
    for (long long q = n - 1; q >= 0 && q >= n - stages; --q)
      mbar_wait(&full[q % stages], (q / stages) & 1, ctx.wait_ns);
  } else {
    // ----------------------------- MMA issuers ----------------------------
    // Per key tile j of the stream: S(j+1)'s first half as soon as the warps
    // have read S(j) whole (its second region is free then), P V(j) when P(j)
    // is written, S(j+1)'s second half over P(j).
    const int w = warp - 2;
    const uint32_t elect = lane == 0;
    const uint32_t s_tmem = tmem + w * 128, o_tmem = tmem + 256 + w * 128;
    uint32_t base = 0;    // key tiles of the items before this one
    uint32_t tiles = 0;   // key tiles of this stream so far
    int ik = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      return PAGED ? warp_wait(bar, parity & 1, ctx, abort_flag)
                   : warp_poll(bar, parity & 1, ctx, abort_flag);
    };
    for (; ok && walk.next(item); ++ik) {
      const uint32_t step = item.pair ? 1 : 2;
      const uint32_t first = item.pair ? 0 : w;
      const uint32_t n_kt = item.k1 - item.k0;
      // Up to 16 rows (a single token of a group): products of 64 rows, whose
      // first 16 lie in the same lanes.  The padding rows' work costs no time
      // here but power, which lowers the clock: 16 x 131072 tokens in a loop,
      // 395 -> 358 us.
      const bool few = PAGED && !item.pair && item.n_tok * G <= 16;
      const uint32_t q_addr = smem_u32(sQ + (item.pair ? w : 0) * kTileBytes);
      const int t_last = item.t0 + item.n_tok - 1;
      const int w_begin = window_begin(a.vis, max(item.t0, 0));
      // half hf of S of the item's tile i, the stream's tile number j
      auto issue_s = [&](uint32_t i, uint32_t j, int hf) -> bool {
        const uint32_t kc = base + i, s = kc % kKStages;
        if (hf == 0 && !wait(&sm.k_full[s], kc / kKStages)) return false;
        tc_fence_after();
        mma_rows<64>(s_tmem + ((j + hf) & 1) * 64, q_addr,
                     smem_u32(sK + s * kTileBytes) + hf * 8192, elect, few);
        commit_if(&sm.s_full[w][hf], elect);
        if (hf == 1) {
          commit_if(&sm.k_empty[s], elect);
          if (!item.pair) commit_if(&sm.k_empty[s], elect);  // the tile has one reader
          if (i + step >= n_kt) commit_if(&sm.q_empty, elect);
        }
        return true;
      };
      if (!(ok = wait(&sm.q_full, ik))) break;
      if (first < n_kt) {
        // the regions are free: P V of the stream's last tile has been issued
        // and its S read
        if (tiles > 0 && !(ok = wait(&sm.s_read[w], tiles - 1))) break;
        if (!(ok = issue_s(first, tiles, 0) && issue_s(first, tiles, 1))) break;
      } else if (lane == 0) {
        umma_commit(&sm.q_empty);
      }
      if (ik > 0 && !(ok = wait(&sm.o_free[w], ik - 1))) break;
      for (uint32_t i = first; i < n_kt; i += step, ++tiles) {
        const bool more = i + step < n_kt;
        if (more && !(ok = wait(&sm.s_read[w], tiles) && issue_s(i + step, tiles + 1, 0))) break;
        const uint32_t vc = base + i, s = vc % kVStages;
        if (!(ok = wait(&sm.v_full[s], vc / kVStages))) break;
        const uint32_t v_addr = smem_u32(sV + s * kTileBytes);
        if (PAGED) {
          // P = 0 meets the V rows that no row of the item sees: zero them,
          // whatever the cache (or an unloaded page's stage) holds there
          const int lo = item.kt.tile(item.k0 + i) * kKeyTile;
          const bool whole = lo + kKeyTile - 1 <= t_last &&
                             (lo >= w_begin || lo + kKeyTile <= a.vis.n_sink);
          if (!whole) {
            // eight lanes a row: no bank conflicts (8 chunks of 300: 41.5 -> 38 us)
            auto zero = [&](int r0, int r1) {
              for (int x = max(r0, 0) * 8 + lane; x < min(r1, kKeyTile) * 8; x += 32) {
                uint4* p = reinterpret_cast<uint4*>(sV + s * kTileBytes) + x;
                p[0] = p[1024] = make_uint4(0, 0, 0, 0);  // channels 0-63, 64-127
              }
            };
            zero(a.vis.n_sink - lo, w_begin - lo);
            zero(t_last + 1 - lo, kKeyTile);
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (!(ok = wait(&sm.p_full[w], tiles))) break;
        tc_fence_after();
        mma_cols(o_tmem, s_tmem + (tiles & 1) * 64, 32, v_addr, i == first, elect, few);
        commit_if(&sm.pv_done[w], elect);
        commit_if(&sm.v_empty[s], elect);
        if (!item.pair) commit_if(&sm.v_empty[s], elect);
        if (more && !(ok = issue_s(i + step, tiles + 1, 1))) break;
      }
      if (!ok) break;
      if (lane == 0) umma_commit(&sm.o_full[w]);
      __syncwarp();
      base += n_kt;
    }
    // every MMA of this warp completes before tensor memory is released
    if (lane == 0) {
      umma_commit(&sm.drain[w]);
      mbar_wait(&sm.drain[w], 0, ctx.wait_ns);
    }
  }
  } else {
    // ------------------------------- softmax ------------------------------
    // Warpgroup w is stream w: thread = tensor memory lane = query row.  The
    // stream's 128 columns are two regions of 64: tile j has the scores of its
    // first 64 keys in region j % 2, of the others in the other one, and P(j)
    // goes over the first.
    reg_inc<224>();
    Walk<G, PAGED> walk(a, sm);
    FwdItem item;
    const int w = (warp - 4) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;       // row of the query tile
    const int tok = r / G, h = r % G;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t s_base = lane_addr + w * 128, o_addr = lane_addr + 256 + w * 128;
    const float sl2 = a.scale_log2;
    const float2 sl2x2 = make_float2(sl2, sl2);
    uint32_t tiles = 0, turns = 0;
    int ik = 0;
    // After a wait that ran out the warps go on without results, so that their
    // named barriers stay matched.
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity) {
      ok = __all_sync(0xffffffffu, ok && guarded_wait(b, parity & 1, ctx, abort_flag));
    };
    auto arrive = [&](uint64_t* b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    for (; walk.next(item); ++ik) {
      const int step = item.pair ? 1 : 2;
      const int first = item.pair ? 0 : w;
      const int n_kt = item.k1 - item.k0;
      const int my_tok = (item.pair ? w * TPT : 0) + tok;   // token of the item
      const bool row_ok = my_tok < item.n_tok;
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int t = item.t0 + my_tok;
      const int wb = window_begin(a.vis, max(t, 0));
      const int t_min = item.t0 + (item.pair ? w * TPT : 0);
      const int wb_max = window_begin(a.vis, max(item.t0 + item.n_tok - 1, 0));
      // the warp's rows: last token, first key of the first one's window
      const int t_warp0 = t_min + quad * 32 / G;
      const int t_warp1 = t_min + (quad * 32 + 31) / G, wb_warp0 = window_begin(a.vis, max(t_warp0, 0));
      float m = -INFINITY, l = 0.f;
      // 64 scores of the row: a half of a tile
      float x[64];
      auto fetch = [&](uint32_t at) {
        tmem_ld32(at, *reinterpret_cast<float(*)[32]>(x));
        tmem_ld32(at + 32, *reinterpret_cast<float(*)[32]>(x + 32));
      };
      // Stream 1 starts when stream 0 has formed P of its first 64 keys: in step,
      // both would want the exponentials and then both the tensor core.  (Of
      // two tiles or more: stream 0 cannot be at the next item before stream 1
      // has read its first S.)
      const bool stagger = item.pair && n_kt > 1;
      if (stagger && w == 1) wait(&sm.turn, turns);
      turns += stagger;
      if (first < n_kt) {
        wait(&sm.s_full[w][0], tiles);
        if (warp_ok && ok) {
          tc_fence_after();
          fetch(s_base + (tiles & 1) * 64);
        }
      }
      for (int i = first; i < n_kt; i += step, ++tiles) {
        const int lo = item.kt.tile(item.k0 + i) * kKeyTile;
        const uint32_t reg0 = s_base + (tiles & 1) * 64, reg1 = s_base + (~tiles & 1) * 64;
        // some row of the stream may not see all of the tile (rows behind the
        // last token count as seeing every key: their results are not stored)
        const bool edge = lo + kKeyTile - 1 > t_min ||
                          (lo < wb_max && lo + kKeyTile > a.vis.n_sink);
        uint32_t pk[32];
        float2 s2[2];
        auto mask = [&](int hf) {
          if (edge)
            mask_columns(x, row_ok ? wb - lo - 64 * hf : 0, row_ok ? t - lo + 1 - 64 * hf : 64,
                         a.vis.n_sink - lo - 64 * hf);
        };
        auto row_max = [&]() {
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 8) {
#pragma unroll
            for (int q = 0; q < 4; ++q) mx[q] = fmax3(mx[q], x[c + 2 * q], x[c + 2 * q + 1]);
          }
          return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
        };
        // P of the 64 keys, packed, and its sum.  The exponentials take the
        // reference of the keys before them, with the maximum formed beside
        // them; where that passes the reference by more than the slack,
        // raise() moves it and they are formed again.
        auto expo = [&]() {
          const float mo = m > -INFINITY ? -m : 0.f;  // no key yet: every x is -inf
          const float2 mo2 = make_float2(mo, mo);
          s2[0] = s2[1] = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 e = fma2(make_float2(x[2 * c], x[2 * c + 1]), sl2x2, mo2);
            const float2 p = make_float2(fast_exp2(e.x), fast_exp2(e.y));
            s2[c & 1] = add2(s2[c & 1], p);
            __nv_bfloat162 b2 = __floats2bfloat162_rn(p.x, p.y);
            pk[c] = *reinterpret_cast<uint32_t*>(&b2);
          }
        };
        auto raise = [&](int hf, float top) {
          // (no row of the warp has seen a key: P and O are 0 as they are)
          const bool seen = __any_sync(0xffffffffu, m > -INFINITY);
          float alpha = 1.f;
          if (top > m + kSlack) {
            alpha = fast_exp2(m - top);  // 0 while the row had no key
            m = top;
          }
          l *= alpha;
          const float2 al = make_float2(alpha, alpha);
          if (seen && i != first) {  // (the stream's first tile of the item overwrites O_w)
            wait(&sm.pv_done[w], tiles - 1);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 16) {
              float o[16];
              tmem_ld16(o_addr + c, o);
              tmem_ld_wait();
              uint32_t u[16];
#pragma unroll
              for (int j = 0; j < 16; j += 2) {
                const float2 v = mul2(make_float2(o[j], o[j + 1]), al);
                u[j] = __float_as_uint(v.x);
                u[j + 1] = __float_as_uint(v.y);
              }
              tmem_st16(o_addr + c, u);
            }
          }
          if (seen && hf == 1) {  // P of the first half, already written
            tmem_st_wait();
#pragma unroll 1
            for (int c = 0; c < 32; c += 16) {
              float o[16];
              tmem_ld16(reg0 + c, o);
              tmem_ld_wait();
              uint32_t u[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const uint32_t b = __float_as_uint(o[j]);
                const float2 v = mul2(make_float2(__uint_as_float(b << 16),
                                                  __uint_as_float(b & 0xffff0000u)), al);
                __nv_bfloat162 b2 = __floats2bfloat162_rn(v.x, v.y);
                u[j] = *reinterpret_cast<uint32_t*>(&b2);
              }
              tmem_st16(reg0 + c, u);
            }
          }
          tmem_st_wait();
        };
        // no row of the warp sees a key of half hf: its P is zero
        auto unseen = [&](int hf) {
          const int c0 = lo + 64 * hf;
          return NARROW && edge && c0 >= a.vis.n_sink && (c0 > t_warp1 || c0 + 64 <= wb_warp0);
        };
        auto half = [&](int hf) {
          if (unseen(hf)) {
#pragma unroll
            for (int c = 0; c < 32; ++c) pk[c] = 0u;
            return;
          }
          mask(hf);
          float top = row_max();
          if (hf == 0 && i == first) m = top;  // the item's first reference
          expo();
          while (ok && __any_sync(0xffffffffu, top > m + kSlack)) {
            raise(hf, top);
            expo();
          }
          l += (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
        };
        if (warp_ok && ok) {
          tmem_ld_wait();
          half(0);
          tmem_st32u(reg0, pk);
        }
        if (stagger && w == 0 && i == 0) arrive(&sm.turn);
        wait(&sm.s_full[w][1], tiles);
        if (warp_ok && ok) {
          tc_fence_after();
          fetch(reg1);
          tmem_ld_wait();
          tc_fence_before();
        }
        arrive(&sm.s_read[w]);  // S is read: its second region takes S of the next tile
        if (warp_ok && ok) {
          half(1);
          tmem_st32u(reg0 + 32, pk);
          tmem_st_wait();
          tc_fence_before();
        }
        arrive(&sm.p_full[w]);
        if (i + step < n_kt) {
          wait(&sm.s_full[w][0], tiles + 1);
          if (warp_ok && ok) {
            tc_fence_after();
            fetch(reg1);
          }
        }
      }
      // ---- the item's result ----
      float L = l, M = m;
      wait(&sm.o_full[w], ik);
      float c0 = 0.f, c1 = 0.f;  // single: weights of O_0 and O_1
      if (!item.pair) {  // join the streams, each warpgroup 64 channels
        sm.xch[0][w][r] = m;
        sm.xch[1][w][r] = l;
        named_bar_sync(1, 256);
        const float m0 = sm.xch[0][0][r], m1 = sm.xch[0][1][r];
        M = fmaxf(m0, m1);
        c0 = m0 > -INFINITY ? fast_exp2(m0 - M) : 0.f;
        c1 = m1 > -INFINITY ? fast_exp2(m1 - M) : 0.f;
        L = sm.xch[1][0][r] * c0 + sm.xch[1][1][r] * c1;
        wait(&sm.o_full[w ^ 1], ik);
        named_bar_sync(2, 256);  // the exchange is free for the next item
      }
      if (ok && warp_ok) {
        tc_fence_after();
        // pair: the stream's 128 channels; single: 64 of both accumulators
        float o[4][32];
#pragma unroll
        for (int k = 0; k < 4; ++k)
          tmem_ld32(lane_addr + 256 + (item.pair ? 128 * w + 32 * k
                                                 : 128 * (k >> 1) + 64 * w + 32 * (k & 1)), o[k]);
        const float inv = L > 0.f ? 1.f / L : (L != L ? L : 0.f);  // a NaN sum stays NaN
        const bool whole = !PAGED || (item.k0 == 0 && item.k1 == item.kt.n);
        const int64_t row = static_cast<int64_t>(PAGED ? 0 : item.b) * a.T + item.tok0 + my_tok;
        const int head = item.g * G + h;
        const int slot = 2 * blockIdx.x + (item.k0 > 0 ? 0 : 1);
        const int64_t prow = static_cast<int64_t>(slot) * kSlotRows + (item.pair ? w * 128 : 0) + r;
        const bool write =
            row_ok && INFLLMV2_CHECK(ctx.status, item.g < a.Hkv &&
                                                     (PAGED ? row >= 0 && row < a.n_tokens
                                                            : item.b < a.B && item.tok0 + my_tok < a.T));
        auto store = [&](const float (&v)[32], int c) {  // channels c .. c + 31
          uint32_t u[8];
          if (whole) {
            __nv_bfloat16* dst = a.O + (row * a.Hq + head) * kHeadDim + c;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                __nv_bfloat162 b2 = __floats2bfloat162_rn(v[16 * x + 2 * j], v[16 * x + 2 * j + 1]);
                u[j] = *reinterpret_cast<uint32_t*>(&b2);
              }
              store_sector(dst + 16 * x, u);
            }
          } else {
            float* dst = a.part + prow * kHeadDim + c;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
#pragma unroll
              for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(v[8 * x + j]);
              store_sector(dst + 8 * x, u);
            }
          }
        };
        tmem_ld_wait();
        tc_fence_before();
        if (item.pair) {
          if (NARROW && whole) {  // (uniform in the warp, as warp_ok is)
            // Four lanes exchange 32-byte pieces, so that a store writes 8 whole
            // lines instead of a sector of 32: step d writes piece lane % 4 of
            // the row of lane ^ d.
            const __nv_bfloat16* mine =
                write ? a.O + (row * a.Hq + head) * kHeadDim : nullptr;
            const int j = lane & 3;
            uint64_t to[4];
#pragma unroll
            for (int d = 0; d < 4; ++d)
              to[d] = __shfl_xor_sync(0xffffffffu, reinterpret_cast<uint64_t>(mine), d);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {  // 64 channels: a line of the row
              uint32_t u[4][8];
#pragma unroll
              for (int q = 0; q < 4; ++q) {
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                  const float* v = o[k + (q >> 1)] + 16 * (q & 1) + 2 * z;
                  __nv_bfloat162 b2 = __floats2bfloat162_rn(v[0] * inv, v[1] * inv);
                  u[q][z] = *reinterpret_cast<uint32_t*>(&b2);
                }
              }
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                uint32_t got[8];
#pragma unroll
                for (int z = 0; z < 8; ++z) {  // piece (lane ^ d) % 4 of the own row, sent there
                  const uint32_t even = (j ^ d) & 2 ? u[2][z] : u[0][z];
                  const uint32_t odd = (j ^ d) & 2 ? u[3][z] : u[1][z];
                  const uint32_t v = (j ^ d) & 1 ? odd : even;
                  got[z] = d ? __shfl_xor_sync(0xffffffffu, v, d) : v;
                }
                if (to[d])
                  store_sector(reinterpret_cast<__nv_bfloat16*>(to[d]) + 32 * k + 16 * j, got);
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
              for (int j = 0; j < 32; ++j) o[k][j] *= inv;
              if (write) store(o[k], 32 * k);
            }
          }
        } else {
          const float f0 = c0 * inv, f1 = c1 * inv;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float v = o[k][j] * f0;
              o[k][j] = n_kt > 1 ? fmaf(o[k + 2][j], f1, v) : v;  // else stream 1 had no tile
            }
            if (write) store(o[k], 64 * w + 32 * k);
          }
        }
        if (write && (item.pair || w == 0)) {
          const float l2 = L > 0.f ? M + __log2f(L) : (L != L ? L : -INFINITY);
          if (!whole)
            a.part_lse[prow] = l2;
          else if (PAGED)
            a.lse[row * a.Hq + head] = l2 * kLn2;
          else
            a.lse[(static_cast<int64_t>(item.b) * a.Hq + head) * a.T + item.tok0 + my_tok] = l2 * kLn2;
        }
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.o_free[item.pair ? w : 0]);
        mbar_arrive(&sm.o_free[item.pair ? w : 1]);
      }
      // the CTA that ends a cut item names it for the merge
      if (PAGED && ok && threadIdx.x == kThreads - 1 && item.k0 > 0 && item.k1 == item.kt.n)
        a.part_item[blockIdx.x] =
            make_int4(item.tok0, item.n_tok,
                      static_cast<int>((sm.per * blockIdx.x - item.k0) / sm.per), item.g);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the partial results of the items that the schedule cut.  Block c takes
// the item that CTA c ended: CTA c0, which began it, left its piece in slot
// 2 c0 + 1, every later one in slot 2 j.  One warp per row (kMergeSplit blocks
// share an item's rows), a lane holding 4 of its 128 channels; the pieces are
// added in order, so results repeat exactly.
constexpr int kMergeThreads = 256, kMergeSplit = 16;

__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const FwdArgs a, int G,
                                                                    int* status) {
  grid_wait();
  const int4 it = a.part_item[blockIdx.x];
  const int c = blockIdx.x, c0 = it.z;
  const int lane = lane_id();
  if (!INFLLMV2_CHECK(status, it.y == 0 || (c0 >= 0 && c0 < c && it.y * G <= kSlotRows && it.x >= 0 &&
                                            it.x + it.y <= a.n_tokens && it.w < a.Hkv)))
    return;
  constexpr int kWarps = kMergeThreads / 32;
  for (int r = blockIdx.y * kWarps + warp_id(); r < it.y * G; r += kWarps * kMergeSplit) {
    auto prow = [&](int j) {
      return static_cast<int64_t>(2 * j + (j == c0 ? 1 : 0)) * kSlotRows + r;
    };
    float M = -INFINITY;
    for (int j = c0 + lane; j <= c; j += 32) M = fmaxf(M, a.part_lse[prow(j)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float Mo = M > -INFINITY ? M : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
#pragma unroll 4
    for (int j = c0; j <= c; ++j) {
      const int64_t p = prow(j);
      const float wt = fast_exp2(a.part_lse[p] - Mo);
      const float4 o = *reinterpret_cast<const float4*>(a.part + p * kHeadDim + 4 * lane);
      L += wt;
      acc.x = fmaf(wt, o.x, acc.x);
      acc.y = fmaf(wt, o.y, acc.y);
      acc.z = fmaf(wt, o.z, acc.z);
      acc.w = fmaf(wt, o.w, acc.w);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const int64_t row = it.x + r / G;
    const int head = it.w * G + r % G;
    __nv_bfloat162 b0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    __nv_bfloat162 b1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    uint2 u = make_uint2(*reinterpret_cast<uint32_t*>(&b0), *reinterpret_cast<uint32_t*>(&b1));
    *reinterpret_cast<uint2*>(a.O + (row * a.Hq + head) * kHeadDim + 4 * lane) = u;
    if (lane == 0)
      a.lse[row * a.Hq + head] = L == 0.f ? -INFINITY : (Mo + __log2f(L)) * kLn2;
  }
}

template <int G, bool PAGED, bool NARROW>
int launch_g(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const FwdArgs& a,
             int grid, const DevCtx& ctx, cudaStream_t st) {
  static std::atomic<uint64_t> smem_set{0};
  if (int e = set_smem_limit(window_attn_kernel<G, PAGED, NARROW>, kFwdSmem, smem_set)) return e;
  window_attn_kernel<G, PAGED, NARROW><<<grid, kThreads, kFwdSmem, st>>>(tq, tk, tv, a, ctx);
  return cudaGetLastError() == cudaSuccess ? INFLLMV2_OK : INFLLMV2_ERR_CUDA;
}

template <bool PAGED, bool NARROW>
int launch_n(int G, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
           const FwdArgs& a, int grid, const DevCtx& ctx, cudaStream_t st) {
  switch (G) {
    case 1: return launch_g<1, PAGED, NARROW>(tq, tk, tv, a, grid, ctx, st);
    case 2: return launch_g<2, PAGED, NARROW>(tq, tk, tv, a, grid, ctx, st);
    case 4: return launch_g<4, PAGED, NARROW>(tq, tk, tv, a, grid, ctx, st);
    case 8: return launch_g<8, PAGED, NARROW>(tq, tk, tv, a, grid, ctx, st);
    case 16: return launch_g<16, PAGED, NARROW>(tq, tk, tv, a, grid, ctx, st);
    default: return INFLLMV2_ERR_UNSUPPORTED;
  }
}

template <bool PAGED>
int launch(int G, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
           const FwdArgs& a, int grid, const DevCtx& ctx, cudaStream_t st) {
  const bool narrow = a.vis.window <= kNarrow;
  return narrow ? launch_n<PAGED, true>(G, tq, tk, tv, a, grid, ctx, st)
                : launch_n<PAGED, false>(G, tq, tk, tv, a, grid, ctx, st);
}

// [n, rows, heads, 128] bf16, rows `row_stride` elements apart; boxes of 64
// channels x box_heads x box_rows.
int rows_map(CUtensorMap* tm, const void* x, int64_t n, int64_t rows, int heads,
             int64_t row_stride, int box_heads, int box_rows) {
  const uint64_t dims[4] = {static_cast<uint64_t>(kHeadDim), static_cast<uint64_t>(heads),
                            static_cast<uint64_t>(rows), static_cast<uint64_t>(n)};
  const uint64_t strides[3] = {static_cast<uint64_t>(kHeadDim) * 2,
                               static_cast<uint64_t>(row_stride) * 2,
                               static_cast<uint64_t>(row_stride) * rows * 2};
  const uint32_t box[4] = {64u, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_rows),
                           1u};
  return make_tmap_bf16_4d(tm, x, dims, strides, box);
}

}  // namespace

int launch_window_attn(const Geometry& g, int window, int n_sink, const void* Q, const void* K,
                       const void* V, void* O, float* lse, const DevCtx& ctx, cudaStream_t st) {
  FwdArgs a{};
  a.O = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  a.vis = visible(window, n_sink);
  a.Hq = g.Hq;
  a.Hkv = g.Hkv;
  a.scale_log2 = g.scale_log2;
  a.B = g.B;
  a.T = g.T;
  const int tpt = 128 / g.G;
  // Two query tiles per item halve the K/V traffic; with fewer such items
  // than SMs, single tiles (keys split between the streams) fill more of them.
  const int64_t pairs = static_cast<int64_t>(g.B) * g.Hkv * ((g.T + 2 * tpt - 1) / (2 * tpt));
  a.item_tiles = pairs >= sm_count() ? 2 : 1;
  const int64_t items = static_cast<int64_t>(g.B) * g.Hkv *
                        ((g.T + a.item_tiles * tpt - 1) / (a.item_tiles * tpt));
  const int grid = static_cast<int>(items < sm_count() ? items : sm_count());
  CUtensorMap tq, tk, tv;
  const int64_t qs = static_cast<int64_t>(g.Hq) * kHeadDim, ks = static_cast<int64_t>(g.Hkv) * kHeadDim;
  if (int e = rows_map(&tq, Q, g.B, g.T, g.Hq, qs, g.G, tpt)) return e;
  if (int e = rows_map(&tk, K, g.B, g.T, g.Hkv, ks, 1, kKeyTile)) return e;
  if (int e = rows_map(&tv, V, g.B, g.T, g.Hkv, ks, 1, kKeyTile)) return e;
  return launch<false>(g.G, tq, tk, tv, a, grid, ctx, st);
}

// Partial results, their log2 sums, and the cut items.
size_t paged_ws_bytes() {
  const size_t n = static_cast<size_t>(sm_count());
  return n * 2 * kSlotRows * (kHeadDim + 1) * sizeof(float) + n * sizeof(int4);
}

int launch_paged_attn(const infllmv2_paged_params& p, float scale_log2, const void* Q,
                      int64_t q_stride, const void* K_pages, const void* V_pages,
                      const int32_t* table, const int32_t* cu_q, const int32_t* seqlens, void* O,
                      float* lse, void* ws, const DevCtx& ctx, cudaStream_t st) {
  FwdArgs a{};
  a.O = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  a.vis = visible(p.window, p.n_sink);
  a.Hq = p.Hq;
  a.Hkv = p.Hkv;
  a.scale_log2 = scale_log2;
  a.item_tiles = 2;
  a.table = table;
  a.cu_q = cu_q;
  a.seqlens = seqlens;
  a.n_seqs = p.n_seqs;
  a.max_pages = p.max_pages;
  a.n_pages = p.n_pages;
  a.page = p.page_size;
  a.n_tokens = p.n_tokens;
  const int grid = sm_count(), G = p.Hq / p.Hkv;
  a.part = static_cast<float*>(ws);
  a.part_lse = a.part + static_cast<size_t>(grid) * 2 * kSlotRows * kHeadDim;
  a.part_item = reinterpret_cast<int4*>(a.part_lse + static_cast<size_t>(grid) * 2 * kSlotRows);
  CUtensorMap tq, tk, tv;
  const int64_t ks = static_cast<int64_t>(p.Hkv) * kHeadDim;
  if (int e = rows_map(&tq, Q, 1, p.n_tokens, p.Hq, q_stride, G, 128 / G)) return e;
  if (int e = rows_map(&tk, K_pages, p.n_pages, p.page_size, p.Hkv, ks, 1, p.page_size)) return e;
  if (int e = rows_map(&tv, V_pages, p.n_pages, p.page_size, p.Hkv, ks, 1, p.page_size)) return e;
  if (int e = launch<true>(G, tq, tk, tv, a, grid, ctx, st)) return e;
  return launch_waiting(merge_kernel, dim3(grid, kMergeSplit), kMergeThreads, 0, st, a, G, ctx.status);
}

}  // namespace infllmv2
