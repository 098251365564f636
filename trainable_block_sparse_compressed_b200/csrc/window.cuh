// window.cuh -- the visible keys of causal attention with a sliding window and
// sinks, shared by its forward (window_attn.cu) and backward (window_bwd.cu).
//
// Key c is visible to the token at position t iff
//   c <= t  and  (c > t - window  or  c < n_sink),
// window <= 0 standing for no window (every key c <= t).
#pragma once

#include "common.cuh"
#include "sm100.cuh"

namespace infllmv2 {

constexpr int kKeyTile = 128;  // keys per tile
constexpr int kNoWindow = 1 << 30;

struct Visible {
  int window;  // kNoWindow: none
  int n_sink;
};

__host__ __device__ inline Visible visible(int window, int n_sink) {
  return Visible{window > 0 && window < kNoWindow ? window : kNoWindow,
                 n_sink < kNoWindow ? n_sink : kNoWindow};
}

// First key of the window of position t (0 where the window covers them all).
__host__ __device__ inline int window_begin(const Visible& v, int t) {
  return t >= v.window ? t - v.window + 1 : 0;
}

// The key tiles that positions t0 .. t1 (t0 <= t1) can see: tiles 0 .. ns-1
// that hold sinks alone, then tiles lo .. lo+n-ns-1.  At least one tile, so
// that rows without a visible key (t1 < 0) still get their result.
struct KeyTiles {
  int ns, lo, n;
  __host__ __device__ int tile(int i) const { return i < ns ? i : lo + i - ns; }
};

__host__ __device__ inline KeyTiles key_tiles(const Visible& v, int t0, int t1) {
  KeyTiles k;
  const int hi = t1 > 0 ? t1 / kKeyTile : 0;
  k.lo = window_begin(v, t0 > 0 ? t0 : 0) / kKeyTile;
  const int sink_tiles = (v.n_sink + kKeyTile - 1) / kKeyTile;
  k.ns = sink_tiles < k.lo ? sink_tiles : k.lo;
  k.n = k.ns + hi - k.lo + 1;
  return k;
}

// A bounded wait of one thread that gives up at once when another thread of the
// CTA has.
__device__ __forceinline__ bool guarded_wait(uint64_t* bar, uint32_t parity, const DevCtx& ctx,
                                             volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  if (*abort_flag) return false;
  if (mbar_wait(bar, parity, ctx.wait_ns)) return true;
  report_status(ctx.status, INFLLMV2_STATUS_TIMEOUT);
  *abort_flag = 1;
  return false;
}

// The same for a warp that goes on together: decided by a vote.  (Decided lane by
// lane, a barrier that completes just as some lanes give up would leave the others
// waiting, without a bound, for the lanes that left, at their next shuffle, ballot
// or __syncwarp.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const DevCtx& ctx,
                                          volatile int* abort_flag) {
  return __all_sync(0xffffffffu, guarded_wait(bar, parity, ctx, abort_flag));
}

// Likewise, with a vote at every poll instead of one behind them: the loop keeps
// the warp's values in uniform registers.  For the issuers of contiguous items
// (T=32768, window 4096: 2013 us, with warp_wait 2050); mixed chunks over pages
// take warp_wait (48.5 us, with warp_poll 49.0).
__device__ __forceinline__ bool warp_poll(uint64_t* bar, uint32_t parity, const DevCtx& ctx,
                                          volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t n = 0;; ++n) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((n & 63) == 0) {
      const bool late = global_timer_ns() - t0 > ctx.wait_ns;
      if (__any_sync(0xffffffffu, late || *abort_flag)) {
        if (late) report_status(ctx.status, INFLLMV2_STATUS_TIMEOUT);
        *abort_flag = 1;
        return false;
      }
    }
  }
}

// Moves registers between the warpgroups of a CTA (all four warps of a
// warpgroup call it); the shares may not exceed what the launch gave the CTA.
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Programmatic launch: lets the next kernel of the stream be launched; waits for
// the kernel before to have finished and its writes to be visible.
__device__ __forceinline__ void grid_launch_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Launches a kernel that calls grid_wait() before it touches memory: its blocks
// may start, and set up, while the kernel before it in the stream still runs.
template <typename... P, typename... A>
int launch_waiting(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                   A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return launched(cudaLaunchKernelEx(&cfg, kernel, static_cast<A&&>(args)...));
}

// Bits 0 .. n-1 of a 32-bit word.
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : 0xffffffffu >> (32 - min(n, 32));
}

// Sets the columns outside [begin, end) to -inf, but for those below `extra`
// that lie before `begin` (sinks).  One bit test and one select per column: a
// comparison per bound and column compiled to branches cost ten times that.
template <int N>
__device__ __forceinline__ void mask_columns(float (&x)[N], int begin, int end, int extra) {
#pragma unroll
  for (int q = 0; q < N / 32; ++q) {
    const uint32_t see = bits_below(end - 32 * q) &
                         (~bits_below(begin - 32 * q) | bits_below(extra - 32 * q));
#pragma unroll
    for (int c = 0; c < 32; ++c)
      x[32 * q + c] = (see >> c) & 1u ? x[32 * q + c] : -INFINITY;
  }
}

// ---------------------------------------------------------------------------
// Products of one 128 x 128 x 128 step.  The shared-memory
// descriptors of a tile differ in their low word's address alone, so each MMA
// costs one or two integer additions (building whole descriptors in a loop took
// ~160 cycles an MMA, more than the tensor core's 64).  A whole warp runs them,
// its warp index broadcast (uniform()), so that addresses stay in uniform
// registers and barriers need no loop over lanes: 5 % of the attention's time.
// ---------------------------------------------------------------------------
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);  // SBO, version, swizzle

__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr >> 4) & 0x3fffu) | ((lbo >> 4) << 16);
}

// A value that is the same in all lanes, in a form that the compiler knows to be.
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// D = A B^T, both K-major tiles of 128 rows x 128 channels (two 16 KB halves of
// 64 channels, 128-byte swizzle); N < 128: as many rows of B.  Called by a whole
// warp, issued by the lane with elect != 0.
template <int N = 128>
__device__ __forceinline__ void mma_rows(uint32_t d, uint32_t a_addr, uint32_t b_addr,
                                         uint32_t elect, bool few = false) {
  const uint32_t idesc = uniform(instr_desc_bf16(few ? 64 : 128, N, 0, 0));
  const uint32_t a = uniform(desc_lo(a_addr, 16)), b = uniform(desc_lo(b_addr, 16));
  const uint32_t du = uniform(d);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(du),
        "r"(a + off), "r"(b + off), "r"(kDescHi), "r"(idesc), "r"(kk > 0 ? 1u : 0u), "r"(elect)
        : "memory");
  }
}

// D (+)= A B: A 128 rows x 16 STEPS in tensor memory (bf16 pairs: columns a ..
// a+31, then a+half ..); B the rows of a tile that are summed over (MN-major).
template <int STEPS = 8>
__device__ __forceinline__ void mma_cols(uint32_t d, uint32_t a, uint32_t half, uint32_t b_addr,
                                         bool first, uint32_t elect, bool few = false) {
  const uint32_t idesc = uniform(instr_desc_bf16(few ? 64 : 128, 128, 0, 1));
  const uint32_t b = uniform(desc_lo(b_addr, 16384)), au = uniform(a), du = uniform(d);
  const uint32_t acc = uniform(first ? 0u : 1u);
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(du),
        "r"(au + (kk >> 2) * half + (kk & 3) * 8), "r"(b + kk * (2048 >> 4)), "r"(kDescHi),
        "r"(idesc), "r"(kk == 0 ? acc : 1u), "r"(elect)
        : "memory");
}

// D (+)= A B, both in shared memory: A a K-major tile (two halves of 64 columns),
// B a tile whose 128 rows are summed over.
__device__ __forceinline__ void mma_rows_cols(uint32_t d, uint32_t a_addr, uint32_t b_addr,
                                              bool first, uint32_t elect) {
  constexpr uint32_t idesc = instr_desc_bf16(128, 128, 0, 1);
  const uint32_t a = uniform(desc_lo(a_addr, 16)), b = uniform(desc_lo(b_addr, 16384));
  const uint32_t du = uniform(d), acc = uniform(first ? 0u : 1u);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 e, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(du),
        "r"(a + (((kk >> 2) * 16384 + (kk & 3) * 32) >> 4)), "r"(b + kk * (2048 >> 4)),
        "r"(kDescHi), "r"(idesc), "r"(kk == 0 ? acc : 1u), "r"(elect)
        : "memory");
}

// umma_commit, likewise.
__device__ __forceinline__ void commit_if(uint64_t* bar, uint32_t elect) {
  asm volatile(
      "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
          smem_u32(bar)),
      "r"(elect)
      : "memory");
}

// 32-byte global store (one full sector per thread).
__device__ __forceinline__ void store_sector(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

}  // namespace infllmv2
