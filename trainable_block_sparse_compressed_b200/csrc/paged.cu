// paged.cu -- the paged key/value cache: block tables and slot maps built on
// the GPU from the requests' lengths, and the append of new keys and values.
//
// Measured on one B200, replayed in a graph: tables of 16 requests 4.6 us, of
// 1024 requests with 44000 new tokens 9 us; append of 16 tokens 1.8 us, of 8192
// tokens of 8 kv heads (67 MB) 12.4 us from HBM (5.4 TB/s).  Calls in a row from
// Python: 6.2, 10.3, 4 and 14.4 us.
//
// Tables.  For request i with kv_i cached and q_i new tokens, pages of P:
//   have_i = ceil(kv_i / P), want_i = ceil((kv_i + q_i) / P), neither more than max_pages,
//   cu_q = exclusive sum of q,  first_i = sum_{j<i} (want_j - have_j),
//   table[i, c] = free_pages[free_count - 1 - first_i - (c - have_i)],  have_i <= c < want_i,
//   token j of i: position kv_i + j, slot = table[i, position / P] * P + position % P.
// A few hundred bytes per request: latency-bound.  One launch of one cluster
// of up to 8 CTAs; every CTA scans all requests into shared memory (redundantly,
// it costs less than handing the sums over) and the CTAs share the table
// entries and tokens.  A cluster barrier between the last read of the inputs
// and the first write lets outputs replace inputs (seqlens over kv_lens, the
// free count in place), so that a captured step can be replayed.
//
// Append.  A copy with scattered rows; bound by HBM.
#include <cooperative_groups.h>

#include "common.cuh"
#include "sm100.cuh"

namespace infllmv2 {
namespace {

constexpr int kTblThreads = 1024;
constexpr int kMaxLen = 1 << 28;  // a longer length is cut
// Sums are kept in 64 bits and stored no larger than this, so that nonsense
// lengths leave the offsets ascending.
constexpr long long kMostRows = 0x7fffffff;

struct TblArgs {
  const int32_t *kv_lens, *q_lens, *free_pages, *free_count;
  int32_t *table, *cu_q, *seqlens, *slots, *positions, *free_left;
  int n_seqs, max_pages, n_pages, page_shift, n_tokens;
};

// Shared memory, per request: first row of its tokens, pages taken before it (one
// more entry of these two: the totals), cached and new tokens.
__global__ void __launch_bounds__(kTblThreads) tables_kernel(const TblArgs a, DevCtx ctx) {
  namespace cg = cooperative_groups;
  extern __shared__ int32_t sh[];
  __shared__ long long warp_sum[2][kTblThreads / 32];
  int32_t* cu = sh;
  int32_t* first = cu + a.n_seqs + 1;
  int32_t* kv = first + a.n_seqs + 1;
  int32_t* qs = kv + a.n_seqs;
  const int lane = lane_id(), warp = warp_id();
  const int P1 = (1 << a.page_shift) - 1;
  const int free_count = max(0, __ldg(a.free_count));
  long long rows = 0, pages = 0;  // of the requests before the strip
  bool too_long = false;          // a token found no column, or no row
  for (int i0 = 0; i0 < a.n_seqs; i0 += kTblThreads) {
    const int i = i0 + threadIdx.x;
    int k = 0, q = 0, need = 0;
    if (i < a.n_seqs) {
      k = max(0, min(a.kv_lens[i], kMaxLen));
      q = max(0, min(a.q_lens[i], kMaxLen));
      need = min((k + q + P1) >> a.page_shift, a.max_pages) -
             min((k + P1) >> a.page_shift, a.max_pages);
      too_long = too_long || (q > 0 && k + q > a.max_pages << a.page_shift);
    }
    long long x = q, y = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long px = __shfl_up_sync(0xffffffffu, x, o), py = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) x += px, y += py;
    }
    if (lane == 31) warp_sum[0][warp] = x, warp_sum[1][warp] = y;
    __syncthreads();
    // kTblThreads / 32 == 32: every warp scans the warps' sums
    long long sx = warp_sum[0][lane], sy = warp_sum[1][lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long px = __shfl_up_sync(0xffffffffu, sx, o), py = __shfl_up_sync(0xffffffffu, sy, o);
      if (lane >= o) sx += px, sy += py;
    }
    const long long tx = __shfl_sync(0xffffffffu, sx, 31), ty = __shfl_sync(0xffffffffu, sy, 31);
    const int before = warp ? warp - 1 : 0;
    const long long bx = __shfl_sync(0xffffffffu, sx, before), by = __shfl_sync(0xffffffffu, sy, before);
    if (i < a.n_seqs) {
      cu[i] = static_cast<int>(min(rows + (warp ? bx : 0) + x - q, kMostRows));
      first[i] = static_cast<int>(min(pages + (warp ? by : 0) + y - need, kMostRows));
      kv[i] = k;
      qs[i] = q;
    }
    rows += tx;
    pages += ty;
    __syncthreads();
  }
  const int n_rows = static_cast<int>(min(rows, kMostRows));
  const int n_new = static_cast<int>(min(pages, kMostRows));
  if (threadIdx.x == 0) cu[a.n_seqs] = n_rows, first[a.n_seqs] = n_new;
  // every CTA has read the lengths and the count before any is replaced
  cg::this_cluster().sync();

  const int n_thr = gridDim.x * kTblThreads;
  const int me = blockIdx.x * kTblThreads + threadIdx.x;
  // the page that request i's table holds, or will hold, in column c
  auto new_page = [&](int i, int k) -> int {  // its k-th new page
    const int at = free_count - 1 - first[i] - k;
    return at >= 0 && at < free_count ? __ldg(a.free_pages + at) : -1;
  };
  for (int i = me; i <= a.n_seqs; i += n_thr) {
    a.cu_q[i] = cu[i];
    if (i < a.n_seqs) a.seqlens[i] = kv[i] + qs[i];
  }
  if (me == 0) a.free_left[0] = max(0, free_count - n_new);
  // new table entries: entry e of all requests' new pages in a row
  auto find = [&](const int32_t* v, int e) -> int {  // last i with v[i] <= e
    int lo = 0, hi = a.n_seqs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (v[mid] <= e) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  for (int64_t e64 = me; e64 < n_new; e64 += n_thr) {
    const int e = static_cast<int>(e64), i = find(first, e);
    const int k = e - first[i];
    const int c = ((kv[i] + P1) >> a.page_shift) + k;
    if (INFLLMV2_CHECK(ctx.status, c >= 0 && c < a.max_pages))
      a.table[static_cast<int64_t>(i) * a.max_pages + c] = new_page(i, k);
  }
  // slots and positions, four rows a thread: one search, and a page looked up
  // again only where the request or the page changes; rows behind the last
  // token get -1.  A token whose column holds no page of the pool is reported: the
  // list ran out now, or in an earlier step that left the entry at -1.
  bool no_page = me == 0 && n_new > free_count;
  const bool wide = ((reinterpret_cast<uintptr_t>(a.slots) |
                      reinterpret_cast<uintptr_t>(a.positions)) & 15u) == 0;
  for (int64_t r0 = 4 * static_cast<int64_t>(me); r0 < a.n_tokens; r0 += 4 * static_cast<int64_t>(n_thr)) {
    int slot[4] = {-1, -1, -1, -1}, pos[4] = {-1, -1, -1, -1};
    int i = r0 < n_rows ? find(cu, static_cast<int>(r0)) : 0;
    int c_last = -1, page = -1;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int r = static_cast<int>(r0) + x;
      if (r0 + x >= n_rows) break;
      while (r >= cu[i + 1]) ++i, c_last = -1;  // (requests without new tokens)
      pos[x] = kv[i] + r - cu[i];
      const int c = pos[x] >> a.page_shift;
      if (c != c_last) {
        c_last = c;
        const int have = (kv[i] + P1) >> a.page_shift;
        page = -1;
        if (c < a.max_pages)
          page = c >= have ? new_page(i, c - have)
                           : a.table[static_cast<int64_t>(i) * a.max_pages + c];
      }
      if (page >= 0 && page < a.n_pages)
        slot[x] = (page << a.page_shift) + (pos[x] & P1);
      else if (c < a.max_pages && r < a.n_tokens)
        no_page = true;
    }
    if (wide && r0 + 4 <= a.n_tokens) {
      *reinterpret_cast<int4*>(a.slots + r0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (r0 + x < a.n_tokens) a.slots[r0 + x] = slot[x], a.positions[r0 + x] = pos[x];
    }
  }
  if (no_page) report_status(ctx.status, INFLLMV2_STATUS_NO_PAGE);
  if (too_long || (me == 0 && n_rows > a.n_tokens)) report_status(ctx.status, INFLLMV2_STATUS_SEQ_FULL);
}

// Rows of `chunks` 16-byte pieces (Hkv x 128 channels); K and V alike.  Four
// pieces of each a thread, all loaded before the first is stored; I: the index
// type of the pieces (32 bits where they suffice, for the division's sake).
template <typename I>
__global__ void __launch_bounds__(256) append_kernel(const int32_t* __restrict__ slots,
                                                     const uint4* __restrict__ k_new,
                                                     const uint4* __restrict__ v_new,
                                                     uint4* __restrict__ K_pages,
                                                     uint4* __restrict__ V_pages, I n, I chunks,
                                                     int64_t k_stride, int64_t v_stride,
                                                     int64_t n_slots) {
  const I first = static_cast<I>(blockIdx.x) * 1024 + threadIdx.x;
  uint4 k[4], v[4];
  int64_t at[4];
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const I i = first + 256 * x;
    at[x] = -1;
    if (i < n) {
      const I t = i / chunks, c = i - t * chunks;
      const int64_t slot = __ldg(slots + t);
      if (slot >= 0 && slot < n_slots) {
        at[x] = slot * static_cast<int64_t>(chunks) + c;
        k[x] = __ldg(k_new + static_cast<int64_t>(t) * k_stride + c);
        v[x] = __ldg(v_new + static_cast<int64_t>(t) * v_stride + c);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (at[x] >= 0) K_pages[at[x]] = k[x], V_pages[at[x]] = v[x];
}

}  // namespace

int launch_paged_tables(const infllmv2_paged_params& p, const int32_t* kv_lens,
                        const int32_t* q_lens, const int32_t* free_pages,
                        const int32_t* free_count, int32_t* table, int32_t* cu_q,
                        int32_t* seqlens, int32_t* slots, int32_t* positions, int32_t* free_left,
                        const DevCtx& ctx, cudaStream_t st) {
  TblArgs a{kv_lens, q_lens, free_pages, free_count, table, cu_q, seqlens, slots, positions,
            free_left, p.n_seqs, p.max_pages, p.n_pages, 0, p.n_tokens};
  while ((1 << a.page_shift) < p.page_size) ++a.page_shift;
  const size_t smem = (4 * static_cast<size_t>(p.n_seqs) + 2) * sizeof(int32_t);
  static std::atomic<uint64_t> smem_set{0};
  constexpr size_t kMost = (4 * static_cast<size_t>(INFLLMV2_MAX_PAGED_SEQS) + 2) * sizeof(int32_t);
  if (int e = set_smem_limit(tables_kernel, kMost, smem_set)) return e;
  const int64_t tokens = (static_cast<int64_t>(p.n_tokens) + 3) / 4;
  const int64_t work = tokens > p.n_seqs ? tokens : p.n_seqs;
  int ctas = 1;
  while (ctas < 8 && static_cast<int64_t>(ctas) * kTblThreads < work) ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kTblThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, tables_kernel, a, ctx));
}

int launch_paged_append(const infllmv2_paged_params& p, const int32_t* slots, const void* k_new,
                        int64_t k_stride, const void* v_new, int64_t v_stride, void* K_pages,
                        void* V_pages, cudaStream_t st) {
  const int chunks = p.Hkv * kHeadDim / 8;
  const int64_t n = static_cast<int64_t>(p.n_tokens) * chunks;
  const int64_t blocks = (n + 1023) / 1024;
  if (blocks > INT32_MAX) return INFLLMV2_ERR_UNSUPPORTED;  // beyond any GPU's memory
  const auto* k = static_cast<const uint4*>(k_new);
  const auto* v = static_cast<const uint4*>(v_new);
  auto* K = static_cast<uint4*>(K_pages);
  auto* V = static_cast<uint4*>(V_pages);
  const int64_t n_slots = static_cast<int64_t>(p.n_pages) * p.page_size;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (n < (int64_t{1} << 31))
    append_kernel<uint32_t><<<grid, 256, 0, st>>>(slots, k, v, K, V, static_cast<uint32_t>(n),
                                                  static_cast<uint32_t>(chunks), k_stride / 8,
                                                  v_stride / 8, n_slots);
  else
    append_kernel<int64_t><<<grid, 256, 0, st>>>(slots, k, v, K, V, n, chunks, k_stride / 8,
                                                 v_stride / 8, n_slots);
  return cudaGetLastError() == cudaSuccess ? INFLLMV2_OK : INFLLMV2_ERR_CUDA;
}

}  // namespace infllmv2
