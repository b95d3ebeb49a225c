// Chunked-prefill attention with a sliding window and sinks on the 5th-generation tensor cores.
//
// What it computes: query i of sequence s's chunk, at position p = len_s - C_s + i, sees the keys t <= p with
// t > p - window or t < n_sink; out = softmax(scale q K^T) V over those (bf16, f16 and E4M3 pools, d_head 128, and 64
// for the 16-bit pools; the block size a multiple of 16).
//
// Work: an item is a (sequence, KV head, pair of query blocks); its rows are two M = 128 tiles A and B of (query, head)
// pairs (row r = query r / G, head r % G).  The keys that some query of the item sees are a list of 16-token slabs --
// the sinks' slabs, then those from the window's start to the last query -- taken a key tile at a time, so that a few
// sinks cost one slab, not a tile of their own.  Slabs lie in pool blocks of their own: each is one or two TMA boxes.
// A window makes items short (1,024 keys are 9 key tiles), so what surrounds them counts: the grid is persistent, and
// loads, products and softmax of the next item start while this one's rows are written.
//
// What bounds it: 4 d flops a (row, key) on the tensor cores, one exponential on the CUDA cores, and the chain between
// them: Q K, softmax, P V of a key tile follow each other, and only the other row tile fills the gaps.
//   * 16-bit pools: 128-key tiles (N = 128 products keep their shared-memory reads, 8 KB a K = 16 step, in step with the
//     multiplies).  S of both tiles and O fill TMEM, so S has one buffer; A and B take turns at the tensor cores, (P V,
//     Q K) of one, then of the other, and P V starts with half of P.  8 x 512 queries, window 4,096: 398 us,
//     0.73 of cuBLAS's rate (567 us for the kernel of the calls without a window, given this mask).  Of a key tile's 3,300
//     cycles the tensor cores work 2,050.  Measured and not kept: 64-key tiles with two S buffers (445 us: the products of
//     N = 64 wait for shared memory), issuing without turns (530 us: both tiles' softmaxes run at once, then both
//     products), two threads a row (534 us).
//   * E4M3 pools: 64-key tiles and two S buffers; codes are converted to binary16 operands by 8 warps (K by 4, V by 4),
//     which share the multi-function units with the exponentials.  Prompts of 1,500 to 2,500 tokens, window 1,024: 305 us,
//     0.42 of cuBLAS's 16-bit rate (450 us for the other kernel).  128-key tiles leave too few operand buffers (403 us);
//     K codes as operands as they are, q as the sum of two E4M3 numbers, cost as much in splitting q (427 us).
//
// Roles (warps): 0-3 softmax and epilogue of A, 4-7 of B (a thread a row, its TMEM lane); 8 loads K and V; 9 and 11
// issue the products of A and of B; 10 looks the items up, loads Q and zeroes V rows that no row sees (0 times whatever
// lies there must stay 0); E4M3 pools: 12-15 convert K and q of A, 16-19 V and q of B.
// TMEM: S of A and B (128 columns each; P overwrites scores that have been read), O of A and B from column 256 on.
// A tile's products are issued by one thread and taken in order, ..., P V(j), Q K(j + 1), ...: Q K may go over P(j).
//
// Few items (a short chunk, one sequence) leave SMs idle: there a cluster of up to 8 CTAs takes one item, each a
// range of its key tiles, and the partial (m, l, O) meet in shared memory.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <string>

#include "pkv_attn.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

constexpr int WP_TBL = 256;  // entries of the table that finds an item's sequence

template <bool KV8, int D>
struct WpCfg {
  static constexpr int THREADS = KV8 ? 640 : 384;
  static constexpr int KEYS = KV8 ? 64 : 128, SLABS = KEYS / TILE;  // a key tile
  static constexpr int NCH = D / 64;                      // 64-wide chunks of d (128 bytes, the swizzle's width)
  static constexpr int Q_TILE = 128 * D * 2;              // one Q tile
  static constexpr int KV_TILE = KEYS * D * 2;            // one K or V tile as an operand (16-bit)
  static constexpr int STG_TILE = KEYS * D;               // one K or V tile of E4M3 codes
  static constexpr int KS = KV8 ? 6 : (D == 64 ? 8 : 5);  // operand ring: K and V tiles in turn
  static constexpr int FS = KV8 ? 8 : 0;                  // staging ring
  static constexpr int BARS = 3 + 3 * KS + 2 * 4 + 5 * 2 + 4 + 2 * FS;
  static constexpr int READERS = THREADS / 32 - 1;        // warps that follow the items
  static constexpr int DATA = 2 * Q_TILE + KS * KV_TILE + FS * STG_TILE;
  static constexpr int SMEM = 1024 + DATA + (BARS + 1) * 8 + 16 + 2 * 64 + 96 + (WP_TBL + 1) * 4;
  // registers: the launch's share is 65,536 / THREADS rounded down to a multiple of 8
  static constexpr int R_LAUNCH = KV8 ? 96 : 168;
  static constexpr int R_SOFTMAX = KV8 ? 160 : 208, R_CONTROL = KV8 ? 64 : 88, R_CONVERT = 48;
  static_assert(256 * R_SOFTMAX + 128 * R_CONTROL + (KV8 ? 256 * R_CONVERT : 0) <= THREADS * R_LAUNCH, "register split");
  static_assert(SMEM <= 232448, "shared memory per CTA");
};

__device__ __forceinline__ bool wait_hint(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\nselp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// true in one lane of the (converged) warp, the same one every time
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}

// two binary32 products and sums, or sums, an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n.reg .b64 x, y, z, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 r, x, y, z;\nmov.b64 {%0, %1}, r;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, r;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 r, x, y;\nmov.b64 {%0, %1}, r;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// the lowest n of 16 bits
__device__ __forceinline__ uint32_t below(int n) {
  const int k = max(0, min(TILE, n));
  return (1u << k) - 1u;
}

// four E4M3 codes to binary16 (exact), and two bfloat16 rounded to binary16, the first of each pair low
__device__ __forceinline__ void f16_of_e4m3(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t f16_of_bf16(uint32_t x) {
  const __half2 h = __floats2half2_rn(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t cluster_peer(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// One item: where its rows and keys are (16 words: it travels through shared memory).
template <int SLABS>
struct __align__(16) ItemT {
  int32_t s, g;
  int32_t qbeg, i0, i1, nq;              // chunk's first row; its queries i0 .. i1 - 1; tiles with rows (1, 2)
  int32_t P, nkeys;                      // position of query 0; keys up to the last query
  int32_t sink_end, lo;                  // a key t is hidden from every row if sink_end <= t < lo
  int32_t sink_slabs, first, nslab;      // the slab list: 0 .. sink_slabs - 1, then from `first` on
  int32_t j0, j1;                        // this CTA's key tiles
  int32_t work;                          // 0: no item (any more)
  __device__ __forceinline__ int32_t slab(int32_t u) const { return u < sink_slabs ? u : first + u - sink_slabs; }
  __device__ __forceinline__ int32_t slabs_of(int32_t j) const { return min(SLABS, nslab - j * SLABS); }
  __device__ __forceinline__ bool hidden(int32_t t) const { return t >= nkeys || (t >= sink_end && t < lo); }
  __device__ __forceinline__ bool ragged(int32_t u) const {  // slab u holds a key hidden from every row
    return hidden(slab(u) * TILE) || hidden(slab(u) * TILE + TILE - 1) ||
           (sink_end < lo && slab(u) * TILE < lo && slab(u) * TILE + TILE > sink_end);
  }
  // tile j holds such a slab: only the last with sinks, the first after them and the last can
  __device__ __forceinline__ bool zeroes(int32_t j) const {
    const int32_t a = j * SLABS, b = a + slabs_of(j);
    auto at = [&](int32_t u) { return u >= a && u < b && ragged(u); };
    return at(sink_slabs - 1) || at(sink_slabs) || at(nslab - 1);
  }
};

template <typename T, bool KV8, int D>
__global__ void __launch_bounds__(WpCfg<KV8, D>::THREADS, 1)
    prefill_win_kernel(const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                       const __grid_constant__ CUtensorMap tmv, const DecodeArgs a, const int32_t* __restrict__ q_off,
                       int32_t max_q, int32_t csize, int64_t most_items) {
  using C = WpCfg<KV8, D>;
  using Item = ItemT<C::SLABS>;
  constexpr int WP_KEYS = C::KEYS, WP_SLABS = C::SLABS;
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value && !KV8;  // operand type of the products
  using TP = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int KS = C::KS, FS = C::FS;
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.G, QB = 128 / G;  // queries a tile
  const int rank = csize > 1 ? blockIdx.x % csize : 0;

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t qs = smem_u32(base), ring = qs + 2 * C::Q_TILE;
  uint8_t* ring_p = base + 2 * C::Q_TILE;
  uint8_t* stg_p = ring_p + KS * C::KV_TILE;
  uint8_t* bar_p = base + C::DATA;
  const uint32_t q_full = smem_u32(bar_p), q_ready = q_full + 8, q_empty = q_full + 16;
  const uint32_t full = q_full + 24, empty = full + 8 * KS, land = empty + 8 * KS;  // operand ring; V tiles to be zeroed
  // per tile A, B: S and P (E4M3: of an even and of an odd key tile); half of P, P V done; the item's O done;
  // the turn to issue; after an abort
  const uint32_t s_full = land + 8 * KS, p_full = s_full + 32, p_most = p_full + 32, o_done = p_most + 16;
  const uint32_t o_full = o_done + 16, turn = o_full + 16, drain = turn + 16;
  const uint32_t sf_full = drain + 16, sf_empty = sf_full + 8 * FS;  // staging ring
  const uint32_t it_full = sf_full + 16 * FS, it_empty = it_full + 16;  // items, two places
  uint8_t* tail_p = bar_p + (C::BARS + 1) / 2 * 16;
  Item* items_p = reinterpret_cast<Item*>(tail_p);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tail_p + 2 * sizeof(Item));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int32_t* wsum = reinterpret_cast<int32_t*>(tslot + 4);
  int32_t* pre = wsum + 24;  // [groups + 1]: query-block pairs of the sequences before a group of them

  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_ready, 8);  // one arrival a warp
    mbar_init(q_empty, 2);
    for (int k = 0; k < KS; ++k) {
      mbar_init(full + 8 * k, KV8 ? 4 : 1);
      mbar_init(empty + 8 * k, 2);  // both tiles' products
      mbar_init(land + 8 * k, 1);
    }
    for (int x = 0; x < 2; ++x) {
      for (int b = 0; b < 2; ++b) {
        mbar_init(s_full + 16 * x + 8 * b, 1);
        mbar_init(p_full + 16 * x + 8 * b, 4);  // one arrival a warp
      }
      mbar_init(p_most + 8 * x, 4);
      mbar_init(o_done + 8 * x, 1);
      mbar_init(turn + 8 * x, 1);
      mbar_init(o_full + 8 * x, 1);
      mbar_init(drain + 8 * x, 1);
    }
    for (int k = 0; k < FS; ++k) {
      mbar_init(sf_full + 8 * k, 1);
      mbar_init(sf_empty + 8 * k, 4);
    }
    for (int k = 0; k < 2; ++k) {
      mbar_init(it_full + 8 * k, 1);
      mbar_init(it_empty + 8 * k, C::READERS);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(smem_u32(tslot), 512);

  // ---- the items, counted ahead so that ragged chunks leave no holes: a thread counts the query-block pairs of
  // `per` sequences (one, up to WP_TBL of them), and the table holds the sums before each such group
  const int most = (max_q + 2 * QB - 1) / (2 * QB);  // query-block pairs of a chunk at most
  const int per = (a.n_seq + WP_TBL - 1) / WP_TBL, groups = (a.n_seq + per - 1) / per;
  auto pairs_of = [&](int s, bool record) -> int {
    const int q0 = q_off[s], c = q_off[s + 1] - q0;
    if (q0 < 0 || c < 0 || c > a.n_tok - q0) {
      if (record) record_error(a.err, DERR_PREFILL_CHUNK, s);
      return 0;
    }
    return min(most, (c + 2 * QB - 1) / (2 * QB));
  };
  {
    int n = 0;
    if (tid < groups)
      for (int s = tid * per; s < min(a.n_seq, (tid + 1) * per); ++s) n += pairs_of(s, blockIdx.x == 0);
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    for (int k = 0; k < warp; ++k) incl += wsum[k];
    if (tid < groups) pre[tid + 1] = incl;
    if (tid == 0) pre[0] = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const int64_t n_items = min(static_cast<int64_t>(pre[groups]) * a.H_kv, most_items);
  const int64_t step = csize > 1 ? n_items : gridDim.x;  // a cluster takes one item
  const int64_t begin = csize > 1 ? blockIdx.x / csize : blockIdx.x;

  // item idx (called by a whole warp); false for one without work.  `record` reports bad values.
  auto get = [&](int64_t idx, Item& w, bool record) __attribute__((always_inline)) -> bool {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(pre[mid]) * a.H_kv <= idx) lo = mid; else hi = mid - 1;
    }
    int64_t r = idx - static_cast<int64_t>(pre[lo]) * a.H_kv;
    w.s = lo * per;
    int nb = 0;
    if (per == 1) {
      nb = pairs_of(w.s, false);
    } else {  // among the group's sequences, 32 at a time
      const int end = min(a.n_seq, w.s + per);
      for (; w.s < end && nb == 0; w.s += 32) {
        const int n = w.s + lane < end ? pairs_of(w.s + lane, false) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(0xffffffffu, static_cast<int64_t>(incl) * a.H_kv > r);
        const int at = past ? __ffs(past) - 1 : 31;  // the lane whose sequence holds the item
        if (past) {
          nb = __shfl_sync(0xffffffffu, n, at);
          r -= static_cast<int64_t>(__shfl_sync(0xffffffffu, incl, at) - nb) * a.H_kv;
          w.s += at;
          break;
        }
        r -= static_cast<int64_t>(__shfl_sync(0xffffffffu, incl, 31)) * a.H_kv;
      }
    }
    if (nb == 0 || r < 0 || r >= static_cast<int64_t>(nb) * a.H_kv) return false;
    w.g = static_cast<int>(r) / nb;
    const int qb = static_cast<int>(r) - w.g * nb;
    w.qbeg = q_off[w.s];
    const int Cs = q_off[w.s + 1] - w.qbeg, len = a.seq_lens[w.s];
    record = record && qb == 0 && w.g == 0;
    if (record && Cs > max_q) record_error(a.err, DERR_PREFILL_CHUNK, w.s);
    w.i0 = qb * 2 * QB;
    if (w.i0 >= Cs) return false;
    if (len < Cs || len > static_cast<int64_t>(a.W) * a.B) {
      if (record) record_error(a.err, DERR_DECODE_LEN, w.s);
      return false;
    }
    w.nq = w.i0 + QB < Cs ? 2 : 1;
    w.i1 = min(Cs, w.i0 + w.nq * QB);
    w.P = len - Cs;
    w.nkeys = w.P + w.i1;
    const Visible v = visible_at(a.window, a.n_sink, w.P + w.i0);
    w.sink_end = v.ns;
    w.lo = v.lo;
    w.sink_slabs = (v.ns + TILE - 1) / TILE;
    w.first = max(w.sink_slabs, v.lo / TILE);
    w.nslab = w.sink_slabs + (w.nkeys + TILE - 1) / TILE - w.first;
    const int nt = (w.nslab + WP_SLABS - 1) / WP_SLABS;
    w.j0 = csize > 1 ? static_cast<int>(static_cast<int64_t>(nt) * rank / csize) : 0;
    w.j1 = csize > 1 ? static_cast<int>(static_cast<int64_t>(nt) * (rank + 1) / csize) : nt;
    w.work = 1;
    return true;
  };

  // bounded wait that also gives up once another role has given up
  auto wait = [&](uint32_t bar, uint32_t parity, int where) -> bool {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (;;) {
      if (wait_hint(bar, parity)) return true;
      if (*abort_flag) return false;
      if (global_ns() - t0 > kWaitNs) {
        *abort_flag = 1;
        record_error(a.err, DERR_DECODE_TIMEOUT, where);
        return false;
      }
    }
  };
  // after an abort: bounded wait for copies or products already started
  auto settle = [&](uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_ns();
    while (!mbar_try_wait(bar, parity) && global_ns() - t0 < kWaitNs) {
    }
  };
  auto warp_ok = [&](bool ok) { return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0; };
  // The next item, looked up by warp 10 while the last ones were at work; false after the last (or an abort).
  uint32_t n_it = 0;
  auto next_item = [&](Item& w) -> bool {
    const uint32_t k = n_it & 1;
    if (!__all_sync(0xffffffffu, wait(it_full + 8 * k, (n_it >> 1) & 1, 900))) return false;
    w = items_p[k];
    __syncwarp();
    if (lane == 0) mbar_arrive(it_empty + 8 * k);
    ++n_it;
    return w.work != 0;
  };

  Item w;
  bool ok = true;
  if (warp >= 8 && warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_CONTROL));
    if (warp == 8) {
      // ------------------------------------------------------------ K and V tiles, in turn, into the ring
      // Lane i holds the pool row of slab 32 k + i of the list (the next 32 are looked up ahead); the 8 lanes of tile
      // j copy its slabs.  16-bit pools: a K slab as one box per 64-wide chunk ([chunk][128 keys][128 B]), a V slab
      // as one box of all chunks ([slab][chunk][16 keys][128 B]); E4M3 pools: 2 KB of codes into the staging ring.
      constexpr int RS = KV8 ? FS : KS;
      const uint32_t r_full = KV8 ? sf_full : full, r_empty = KV8 ? sf_empty : empty;
      const uint32_t r_data = KV8 ? smem_u32(stg_p) : ring;
      uint32_t c = 0;  // tiles loaded so far
      uint32_t on_land = 0;  // of the last RS tiles, those whose bytes arrive at `land` (bit c % RS)
      uint32_t land_par = 0;  // bit k: parity of the uses of `land` slot k
      while (ok && next_item(w)) {
        auto row_of = [&](int u) -> int {
          if (u >= w.nslab) return 0;
          const int t0 = w.slab(u) * TILE, lb = t0 / a.B;
          int blk = a.tables[static_cast<int64_t>(w.s) * a.W + lb];
          if (blk < 0 || blk >= a.num_blocks) {
            record_error(a.err, DERR_DECODE_BLOCK, blk);
            blk = 0;
          }
          return ((blk * a.L + a.layer) * a.H_kv + w.g) * a.B + (t0 - lb * a.B);
        };
        constexpr int TPG = 32 / WP_SLABS;  // key tiles a group of 32 slabs
        int row = row_of(w.j0 * WP_SLABS + lane);
        int next = w.j0 + TPG < w.j1 ? row_of((w.j0 + TPG) * WP_SLABS + lane) : 0;
        for (int j = w.j0; j < w.j1 && ok; ++j) {
          const int q = (j - w.j0) % TPG;
          if (q == 0 && j > w.j0) {
            row = next;
            if (j + TPG < w.j1) next = row_of((j + TPG) * WP_SLABS + lane);
          }
          const int ns = w.slabs_of(j), i = lane - q * WP_SLABS;  // this lane's slab of the tile
          const bool mine = i >= 0 && i < ns;
          for (int kv = 0; kv < 2 && ok; ++kv, ++c) {
            const uint32_t slot = c % RS;
            const bool zero = !KV8 && kv == 1 && w.zeroes(j);
            const uint32_t bar = zero ? land + 8 * slot : r_full + 8 * slot;
            if (lane == 0) {
              if (c >= RS) ok = wait(r_empty + 8 * slot, ((c / RS) - 1) & 1, 100);
              if (ok) mbar_arrive_expect_tx(bar, ns * TILE * D * (KV8 ? 1 : 2));
            }
            ok = warp_ok(ok);  // also orders the expect_tx before the copies
            if (!ok) break;
            on_land = (on_land & ~(1u << slot)) | (zero ? 1u << slot : 0u);
            if (zero) land_par ^= 1u << slot;
            const uint32_t dst = r_data + slot * (KV8 ? C::STG_TILE : C::KV_TILE);
            if (mine) {
              if constexpr (KV8) {
                tma_load_2d(dst + i * TILE * 128, kv ? &tmv : &tmk, 0, row, bar);
              } else if (kv == 0) {
#pragma unroll
                for (int h = 0; h < C::NCH; ++h)
                  tma_load_2d(dst + h * (WP_KEYS * 128) + i * TILE * 128, &tmk, 64 * h, row, bar);
              } else if constexpr (D == 128) {
                tma_load_3d(dst + i * 2 * TILE * 128, &tmv, 0, row, 0, bar);
              } else {
                tma_load_2d(dst + i * TILE * 128, &tmv, 0, row, bar);
              }
            }
          }
        }
      }
      if (*abort_flag && lane == 0)  // copies may still be landing in the last ring's slots
        for (uint32_t k = c > RS ? c - RS : 0; k < c; ++k) {
          const uint32_t slot = k % RS;
          if (!KV8 && (on_land >> slot & 1)) settle(land + 8 * slot, ~(land_par >> slot) & 1);
          else settle(r_full + 8 * slot, (k / RS) & 1);
        }
    } else if (warp == 9 || warp == 11) {
      // ------------------------------------------------------------ the products of tile X (9: A, 11: B)
      // The whole warp walks the items, so that descriptors stay warp-uniform, and one elected lane issues: a
      // divergent thread on its own needs some 140 cycles a product to bring its operands into uniform registers.
      // 16-bit pools: A and B take turns, so that S of A arrives while B's products run and the two softmaxes stay half a
      // period apart.  E4M3 pools: S has two buffers, so that Q K of the next key tile runs while this one's softmax does.
      // A tile without rows (nq = 1) has its turns, and its part in the operand ring, all the same.
      // (the broadcasts from lane 0 are what tells the compiler that a value is the same in all lanes)
      auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
      const int X = uni(warp == 9 ? 0 : 1);
      const uint32_t s_tm = uni(tmem) + 128 * X, o_tm = uni(tmem) + 256 + 128 * X;
      const uint32_t idesc_o = umma_idesc_f16(BF16, 128, D, true);
      // operand descriptors: the first, and a step of the address field (16-byte units) from there on
      const uint64_t q_desc = umma_desc_sw128(uni(qs) + X * C::Q_TILE, 16, 1024);
      const uint64_t k_desc = umma_desc_sw128(uni(ring), 16, 1024);
      const uint64_t v_desc = umma_desc_sw128(uni(ring), TILE * 128, 1024);
      const uint32_t bars = uni(q_full);  // the barriers from here on
      const uint32_t u_empty = bars + (empty - q_full), u_q_empty = bars + 16;
      const uint32_t u_s_full = bars + (s_full - q_full) + 16 * X, u_o_full = bars + (o_full - q_full) + 8 * X;
      const uint32_t u_o_done = bars + (o_done - q_full) + 8 * X;
      const uint32_t u_turn = bars + (turn - q_full) + 8 * (1 - X);  // the other tile's
      auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
        return __all_sync(0xffffffffu, wait(bar, parity, where)) != 0;
      };
      auto commit = [&](uint32_t bar) {
        if (elect_one()) umma_commit(bar);
      };
      uint32_t c = 0, items = 0, ns_ = 0, np = 0, turns = 0;  // ring position; items; S and P tiles; turns had
      while (ok && next_item(w)) {
        if (w.j0 == w.j1) continue;  // a cluster rank without a key tile
        const bool live = uni(X < w.nq) != 0;
        const int nt = uni(w.j1 - w.j0), nslab = uni(w.nslab - w.j0 * WP_SLABS);
        ok = wait_all(KV8 ? q_ready : q_full, items++ & 1, 200);
        if constexpr (KV8) {
          // S of the item's i-th key tile (its K is at ring position c + 2 i)
          auto qk = [&](int i) -> bool {
            const uint32_t at = c + 2 * i, slot = at % KS;
            if (!wait_all(full + 8 * slot, (at / KS) & 1, 210)) return false;
            tc_fence_after();
            const uint64_t kd = k_desc + slot * (C::KV_TILE / 16);
            const uint32_t idesc_s = umma_idesc_f16(BF16, 128, min(WP_SLABS, nslab - i * WP_SLABS) * TILE, false);
            const uint32_t b = ns_ & 1;
            if (elect_one()) {
              if (live) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)  // 64-wide chunk; 16 elements along its 128-byte row
                  umma_ss(s_tm + 64 * b, q_desc + ((k >> 2) * 16384 + (k & 3) * 32) / 16,
                          kd + ((k >> 2) * (WP_KEYS * 128) + (k & 3) * 32) / 16, idesc_s, k > 0);
                umma_commit(u_s_full + 8 * b);
                umma_commit(u_empty + 8 * slot);  // this tile's use of the operand is over once its products are done
                if (i + 1 == nt) umma_commit(u_q_empty);
              } else {
                mbar_arrive(empty + 8 * slot);
                if (i + 1 == nt) mbar_arrive(q_empty);
              }
            }
            __syncwarp();
            ++ns_;
            return true;
          };
          auto pv = [&](int i) -> bool {
            const uint32_t at = c + 2 * i + 1, slot = at % KS, b = np & 1;
            if (!wait_all(full + 8 * slot, (at / KS) & 1, 220)) return false;
            if (live && !wait_all(p_full + 16 * X + 8 * b, (np >> 1) & 1, 230)) return false;
            tc_fence_after();
            const uint64_t vd = v_desc + slot * (C::KV_TILE / 16);
            const int n = min(WP_SLABS, nslab - i * WP_SLABS);
            if (elect_one()) {
              if (live) {
#pragma unroll
                for (int k = 0; k < WP_SLABS; ++k)
                  if (k < n)
                    umma_ts(o_tm, s_tm + 64 * b + 8 * k, vd + k * (C::NCH * TILE * 128 / 16), idesc_o, i > 0 || k > 0 ? 1u : 0u);
                umma_commit(u_o_done);
                if (i + 1 == nt) umma_commit(u_o_full);
                umma_commit(u_empty + 8 * slot);
              } else {
                mbar_arrive(empty + 8 * slot);
              }
            }
            __syncwarp();
            ++np;
            return true;
          };
          if (ok) ok = qk(0);
          for (int i = 0; i < nt && ok; ++i) {
            if (i + 1 < nt) ok = qk(i + 1);
            if (ok) ok = pv(i);
          }
          c += 2 * nt;
          if (!live) ns_ -= nt, np -= nt;  // no S or P of this tile
        }
        for (int i = -1; !KV8 && i < nt && ok; ++i) {  // P V of the item's i-th key tile, then Q K of the next
          // everything is waited for before the turn: within it the products follow each other without a gap
          const bool has_pv = i >= 0, has_qk = i + 1 < nt;
          const uint32_t vs = c % KS, ks = (c + has_pv) % KS;
          if (has_pv) {
            ok = wait_all(full + 8 * vs, (c / KS) & 1, 210);
            ++c;
          }
          if (ok && has_qk) {
            ok = wait_all(full + 8 * ks, (c / KS) & 1, 220);
            ++c;
          }
          if (ok && has_pv && live) ok = wait_all(p_most + 8 * X, np & 1, 230);
          if (ok && (X == 1 || turns > 0)) ok = wait_all(turn + 8 * X, (turns - 1 + X) & 1, 240);
          if (!ok) break;
          ++turns;
          tc_fence_after();
          const uint64_t vd = v_desc + vs * (C::KV_TILE / 16), kd = k_desc + ks * (C::KV_TILE / 16);
          const int nv = has_pv ? min(WP_SLABS, nslab - i * WP_SLABS) : 0;
          const uint32_t idesc_s =
              umma_idesc_f16(BF16, 128, has_qk ? min(WP_SLABS, nslab - (i + 1) * WP_SLABS) * TILE : TILE, false);
          // P of keys 64 .. 127 comes first (slabs 4 .. 7, where the tile has them)
          const int k0 = nv > 4 ? 4 : 0;
          auto pv = [&](int k) {
            if (k < nv)
              umma_ts(o_tm, s_tm + 64 + 8 * k, vd + k * (C::NCH * TILE * 128 / 16), idesc_o, i > 0 || k != k0 ? 1u : 0u);
          };
          bool came = true;
          if (elect_one()) {
            if (live) {
              if (has_pv) {  // half of P, then (it comes meanwhile) the rest
#pragma unroll
                for (int k = 0; k < WP_SLABS; ++k)
                  if (k >= 4) pv(k);
                came = wait(p_full + 16 * X, np & 1, 250);
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < 4; ++k) pv(k);
              }
              if (has_qk) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {  // 64-wide chunk; 16 elements along its 128-byte row
                  // the other tile's warp is let go two products early, which hides its start
                  if (k == D / 16 - 2) mbar_arrive(u_turn);
                  umma_ss(s_tm, q_desc + ((k >> 2) * 16384 + (k & 3) * 32) / 16,
                          kd + ((k >> 2) * (WP_KEYS * 128) + (k & 3) * 32) / 16, idesc_s, k > 0);
                }
                umma_commit(u_s_full);
              } else {
                mbar_arrive(u_turn);
                umma_commit(u_o_full);
              }
              // this tile's use of the operands is over once its products so far are done
              if (has_pv) umma_commit(u_empty + 8 * vs);
              if (has_qk) umma_commit(u_empty + 8 * ks);
              if (i + 2 == nt) umma_commit(u_q_empty);
            } else {
              mbar_arrive(u_turn);
              if (has_pv) mbar_arrive(u_empty + 8 * vs);
              if (has_qk) mbar_arrive(u_empty + 8 * ks);
              if (i + 2 == nt) mbar_arrive(u_q_empty);
            }
          }
          np += live && has_pv;
          ok = __all_sync(0xffffffffu, came);
        }
      }
      if (*abort_flag) {
        commit(drain + 8 * X);
        settle(drain + 8 * X, 0);
      }
    } else {
      // ------------------------------------------------------------ Q; V rows hidden from every row of the item
      uint32_t c = 0, uses = 0, items = 0;  // ring position; bit k: parity of `land` uses of slot k; items
      int64_t idx = begin;
      auto publish = [&](uint32_t n) -> bool {  // the n-th item (or the end) into its place
        bool room = true;
        if (lane == 0 && n >= 2) room = wait(it_empty + 8 * (n & 1), ((n >> 1) - 1) & 1, 910);
        if (!warp_ok(room)) return false;
        w.work = 0;
        for (; idx < n_items && !w.work; idx += step)
          if (!get(idx, w, lane == 0 && rank == 0)) w.work = 0;
        if (lane == 0) {
          items_p[n & 1] = w;
          mbar_arrive(it_full + 8 * (n & 1));
        }
        __syncwarp();
        return true;
      };
      ok = publish(0);
      for (uint32_t n = 0; ok; ++n) {
        if (!items_p[n & 1].work) break;
        ok = publish(n + 1);  // one ahead of what the others work on
        if (!ok) break;
        w = items_p[n & 1];
        if (w.j0 == w.j1) continue;
        if (lane == 0) {
          if (items > 0) ok = wait(q_empty, (items - 1) & 1, 400);
          if (ok) {
            fence_proxy_async();
            mbar_arrive_expect_tx(q_full, w.nq * G * QB * D * 2);  // G * QB rows a tile (126 for G = 3)
            for (int x = 0; x < w.nq; ++x)
              for (int h = 0; h < C::NCH; ++h)
                tma_load_3d(qs + x * C::Q_TILE + h * 16384, &tmq, 64 * h, w.g * G, w.qbeg + w.i0 + x * QB, q_full);
            ++items;
          }
        }
        ok = warp_ok(ok);
        for (int j = w.j0; j < w.j1 && ok && !KV8; ++j, c += 2) {  // (E4M3: the conversion writes the zeros)
          if (!w.zeroes(j)) continue;
          const uint32_t slot = (c + 1) % KS;
          if (lane == 0) ok = wait(land + 8 * slot, uses >> slot & 1, 300);
          ok = warp_ok(ok);
          if (!ok) break;
          uses ^= 1u << slot;
          uint8_t* vt = ring_p + slot * C::KV_TILE;
          for (int i = 0; i < w.slabs_of(j); ++i) {
            const int u = j * WP_SLABS + i;
            if (!w.ragged(u)) continue;
            const int t0 = w.slab(u) * TILE;
            for (int k = lane; k < TILE * 8 * C::NCH; k += 32) {  // 16-byte pieces of the slab
              const int r = k / (8 * C::NCH), p = k % (8 * C::NCH);
              if (w.hidden(t0 + r))
                *reinterpret_cast<int4*>(vt + i * (C::NCH * TILE * 128) + p / 8 * (TILE * 128) + r * 128 + p % 8 * 16) =
                    make_int4(0, 0, 0, 0);
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(full + 8 * slot);
        }
      }
      if (*abort_flag && lane == 0 && items > 0) settle(q_full, (items - 1) & 1);
    }
  } else if (warp >= 12) {
    // -------------------------------------------------------------- E4M3: q and the staged codes to binary16
    if constexpr (KV8) {
      // warps 12-15: q of tile A, then the K tiles; 16-19: q of B, the V tiles
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_CONVERT));
      const int r = tid & 127, kv = warp >= 16;
      uint32_t c = kv, items = 0;
      while (ok && next_item(w)) {
        if (w.j0 == w.j1) continue;
        ok = __all_sync(0xffffffffu, wait(q_full, items++ & 1, 500));
        if (!ok) break;
        uint4* qt = reinterpret_cast<uint4*>(base + kv * C::Q_TILE);
        if (kv < w.nq)
#pragma unroll 4
          for (int k = r; k < C::Q_TILE / 16; k += 128) {
            uint4 v = qt[k];
            v = make_uint4(f16_of_bf16(v.x), f16_of_bf16(v.y), f16_of_bf16(v.z), f16_of_bf16(v.w));
            qt[k] = v;
          }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
        for (int j = w.j0; j < w.j1 && ok; ++j, c += 2) {
            const uint32_t f = c % FS, slot = c % KS;
            bool here = wait(sf_full + 8 * f, (c / FS) & 1, 510);
            if (here && c >= KS) here = wait(empty + 8 * slot, ((c / KS) - 1) & 1, 520);
            ok = __all_sync(0xffffffffu, here);
            if (!ok) break;
            const uint8_t* src = stg_p + f * C::STG_TILE;
            uint8_t* dst = ring_p + slot * C::KV_TILE;
            const int ns = w.slabs_of(j);
            const bool zero = kv == 1 && w.zeroes(j);
            // staging row rr of slab i holds d = 16 u .. 16 u + 15 in 16-byte unit u ^ (rr & 7); the operand rows hold
            // d in two 64-wide chunks of eight units, unit t at t ^ (row & 7).  Thread r: row r / 8, unit r % 8 of slab i
            const int rr = r >> 3, u = r & 7, cc = u >> 2, t = (u & 3) * 2, sw = rr & 7;
#pragma unroll 4
            for (int i = 0; i < ns; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(src + i * (TILE * 128) + rr * 128 + ((u ^ sw) << 4));
              uint4 o0, o1;
              f16_of_e4m3(v.x, o0.x, o0.y);
              f16_of_e4m3(v.y, o0.z, o0.w);
              f16_of_e4m3(v.z, o1.x, o1.y);
              f16_of_e4m3(v.w, o1.z, o1.w);
              if (zero && w.hidden(w.slab(j * WP_SLABS + i) * TILE + rr)) o0 = o1 = make_uint4(0, 0, 0, 0);
              uint8_t* p = kv == 0 ? dst + cc * (WP_KEYS * 128) + (i * TILE + rr) * 128
                                   : dst + i * (2 * TILE * 128) + cc * (TILE * 128) + rr * 128;
              *reinterpret_cast<uint4*>(p + ((t ^ sw) << 4)) = o0;
              *reinterpret_cast<uint4*>(p + (((t + 1) ^ sw) << 4)) = o1;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(full + 8 * slot);
              mbar_arrive(sf_empty + 8 * f);
            }
          }
      }
    }
  } else {
    // -------------------------------------------------------------- softmax and epilogue of tile X
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::R_SOFTMAX));
    const int X = warp >> 2, r = tid & 127;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_tile = lane_addr + 128 * X, o_addr = lane_addr + 256 + 128 * X;
    const float sl = a.scale_log2;
    uint32_t n_s = 0, no = 0;  // S tiles and outputs taken
    while (ok && next_item(w)) {
      if (X >= w.nq) continue;
      const int qi = w.i0 + X * QB + r / G;
      const bool valid = r < QB * G && qi < w.i1;
      const int lim = valid ? w.P + qi : w.nkeys - 1;                  // last visible key
      const int low = visible_at(a.window, a.n_sink, lim).lo;          // from here on visible, before only the sinks
      // a tile's other rows (past the chunk, past QB G) hold whatever lies there: their m stays as it is, so that no
      // vote of the warp, and with it no rounding of a row, depends on them
      float m = valid ? -INFINITY : 0.f, l = 0.f, mx;
      float2 ls[4];
      for (int j = w.j0; j < w.j1 && ok; ++j, ++n_s) {
        const uint32_t b = KV8 ? n_s & 1 : 0, s_addr = s_tile + 64 * b;
        ok = __all_sync(0xffffffffu, wait(s_full + 16 * X + 8 * b, (KV8 ? n_s >> 1 : n_s) & 1, 600));
        if (!ok) break;
        tc_fence_after();
        // the tile's last 64 keys and, 16-bit pools, its first 64
        uint32_t sb[2][32], sa[KV8 ? 1 : 2][32];
        constexpr int B0 = KV8 ? 0 : 64;
        tmem_ld32(s_addr + B0, sb[0]);
        tmem_ld32(s_addr + B0 + 32, sb[1]);
        // mask only tiles that hold a key hidden from a row of the warp (or columns that were not computed)
        const int u0 = j * WP_SLABS, n = w.slabs_of(j);
        const int t_first = w.slab(u0) * TILE, t_last = w.slab(u0 + n - 1) * TILE + TILE - 1;
        const bool edge = __any_sync(0xffffffffu, n < WP_SLABS || t_last > lim || t_first < low);
        auto mask = [&](uint32_t (&x)[2][32], int i0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // the slab's visible elements as bits: up to the row's last key, less those between its sinks and its
            // window (selects, no branches: 128 short branches cost ten times the softmax itself)
            const int t0 = w.slab(u0 + i0 + i) * TILE;
            const uint32_t vis = i0 + i < n ? below(lim + 1 - t0) & ~(below(low - t0) & ~below(a.n_sink - t0)) : 0u;
            if (__any_sync(0xffffffffu, vis != 0xffffu)) {
#pragma unroll
              for (int e = 0; e < TILE; ++e) {
                uint32_t& v = x[i >> 1][(i & 1) * TILE + e];
                v = (vis & (1u << e)) ? v : __float_as_uint(-INFINITY);
              }
            }
          }
        };
        auto largest = [&](const uint32_t (&x)[2][32], float from) {
          float mx4[4] = {from, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int t = 0; t < 4; ++t)
                mx4[t] = fmaxf(mx4[t], fmaxf(__uint_as_float(x[c][e + t]), __uint_as_float(x[c][e + t + 4])));
          return fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        };
        // P = 2^(scale s - m), 16-bit, two keys a column, over scores that have been read; a row that has seen no key
        // yet keeps m = -inf, and 0 stands in for it
        auto exps = [&](const uint32_t (&x)[32], uint32_t at) {
          const float neg_m = m == -INFINITY ? 0.f : -m;
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 p = fma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), make_float2(sl, sl),
                            make_float2(neg_m, neg_m));
            p = make_float2(fast_exp2(p.x), fast_exp2(p.y));
            ls[e & 3] = add2(ls[e & 3], p);
            pw[e] = pack2<TP>(p.x, p.y);
          }
          tmem_st16(at, pw);
        };
        auto arrive = [&](uint32_t bar) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        };
        constexpr int P0 = KV8 ? 0 : 64;  // P's columns in S (16-bit pools: keys 64 .. are in the last 32 of them)
        auto first_exps = [&] {
          exps(sb[0], s_addr + P0 + (KV8 ? 0 : 32));
          exps(sb[1], s_addr + P0 + (KV8 ? 16 : 48));
        };
        // The reference maximum of a row moves only when the row's grows by more than 2^8 (until then P and l share the
        // old one), which is rare after the first tile.  E4M3 pools take the exponentials with the old one while the new
        // maximum is found, and once more if it moves (305 -> 303 us; with 16-bit pools' longer turns it costs 9 %).
        const bool early = KV8 && !__any_sync(0xffffffffu, m == -INFINITY);
        if (early)
#pragma unroll
          for (int t = 0; t < 4; ++t) ls[t] = make_float2(0.f, 0.f);
        tmem_ld_wait();
        if constexpr (!KV8) {
          tmem_ld32(s_addr, sa[0]);
          tmem_ld32(s_addr + 32, sa[1]);
        }
        if (edge) mask(sb, KV8 ? 0 : 4);
        if (early) first_exps();
        mx = largest(sb, -INFINITY);
        if constexpr (!KV8) {
          tmem_ld_wait();
          if (edge) mask(sa, 0);
          if constexpr (!KV8) mx = largest(sa, mx);
        }
        const float m_new = valid ? fmaxf(m, mx * sl) : m;
        const bool moves = __any_sync(0xffffffffu, m_new > m + 8.f);
        if (moves) {
          // l and O so far are rescaled, once O holds P V(j - 1) (16-bit pools: S(j) is here, so it does)
          const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m - m_new);
          if (j > w.j0) {
            if constexpr (KV8) {
              ok = __all_sync(0xffffffffu, wait(o_done + 8 * X, (n_s - 1) & 1, 610));
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(o_addr + 32 * c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
              tmem_st32(o_addr + 32 * c, o);
            }
          }
          l *= alpha;
          m = m_new;
        }
        if (!early || moves) {
#pragma unroll
          for (int t = 0; t < 4; ++t) ls[t] = make_float2(0.f, 0.f);
          first_exps();
        }
        if constexpr (!KV8) {
          arrive(p_most + 8 * X);  // P V may begin with half of the keys
          exps(sa[0], s_addr + P0);
          exps(sa[1], s_addr + P0 + 16);
        }
        arrive(p_full + 16 * X + 8 * b);
        const float2 l2 = add2(add2(ls[0], ls[1]), add2(ls[2], ls[3]));
        l += l2.x + l2.y;
      }
      if (!ok) break;
      if (w.j0 < w.j1) {
        ok = __all_sync(0xffffffffu, wait(o_full + 8 * X, no & 1, 700));
        // a cluster's partial goes over the operands: not before the products of the other tile are done, too
        if (ok && csize > 1 && w.nq == 2) ok = __all_sync(0xffffffffu, wait(o_full + 8 * (1 - X), 0, 710));
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      if (csize == 1) {
        const float inv = a.v_mul / l;  // v_scale of an E4M3 pool, else 1
        // the 16-byte pieces of four rows change places within a quad of lanes, so that a store covers 64 bytes
        // in a row of eight rows, not 16 of 32: piece p of 32 columns of the quad's row i in lane p
        T* out[4];
        const int r4 = r & ~3, q4 = lane & 3;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int qr = w.i0 + X * QB + (r4 + i) / G, hr = (r4 + i) % G;
          const bool there = r4 + i < QB * G && qr < w.i1;
          out[i] = there ? static_cast<T*>(a.out) + (static_cast<int64_t>(w.qbeg + qr) * a.H_q + w.g * G + hr) * D + 8 * q4
                         : nullptr;
        }
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32], v[4][4];
          tmem_ld32(o_addr + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int p = 0; p < 4; ++p)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[p][e] = pack2<T>(__uint_as_float(o[8 * p + 2 * e]) * inv, __uint_as_float(o[8 * p + 2 * e + 1]) * inv);
#pragma unroll
          for (int bit = 1; bit < 4; bit *= 2)
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              if (p & bit) continue;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const bool up = q4 & bit;
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[p][e] : v[p | bit][e], bit);
                v[p][e] = up ? got : v[p][e];
                v[p | bit][e] = up ? v[p | bit][e] : got;
              }
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (out[i]) *reinterpret_cast<uint4*>(out[i] + 32 * c) = make_uint4(v[i][0], v[i][1], v[i][2], v[i][3]);
        }
        tc_fence_before();
      } else {
        // this CTA's partial of the row, over the operand room (its products are done, its loads were all used):
        // (m, l) of the 256 rows, then O; 16-byte pieces rotated by the row so that neighbours share no bank
        if (w.j0 < w.j1) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_addr + 32 * c, o);
            tmem_ld_wait();
            if (valid) {
#pragma unroll
              for (int v = 0; v < 8; ++v)
                *reinterpret_cast<uint4*>(base + 2048 + (X * 128 + r) * (D * 4) + ((8 * c + v + r) % (D / 4)) * 16) =
                    make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
            }
          }
          tc_fence_before();
        }
        *reinterpret_cast<float2*>(base + (X * 128 + r) * 8) = make_float2(m, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_dealloc(tmem, 512);
  if (csize > 1) {
    // every thread of the cluster; an item is the same for all its CTAs, and so is its absence
    const Item it = items_p[0];
    const bool has = it.work != 0;
    cluster_barrier();
    if (has && !*abort_flag) {
      constexpr int PC = D / 4;  // 16-byte pieces of a row's O
      const int rows = (it.i1 - it.i0) * G;  // rows of A (QB G of them), then of B
      for (int k = rank * blockDim.x + tid; k < rows * PC; k += csize * blockDim.x) {
        const int row = k / PC, pc = k - row * PC;
        const int x = row / (QB * G), r = row - x * QB * G, at = x * 128 + r;
        float m = -INFINITY;
        for (int p = 0; p < csize; ++p) {
          float pm;
          asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(pm) : "r"(cluster_peer(qs + at * 8, p)) : "memory");
          m = fmaxf(m, pm);
        }
        float l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int p = 0; p < csize; ++p) {
          float pm, pl;
          asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                       : "=f"(pm), "=f"(pl)
                       : "r"(cluster_peer(qs + at * 8, p))
                       : "memory");
          if (pm == -INFINITY) continue;  // no key of the row in that CTA's range: its O holds nothing
          float4 v;
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                       : "r"(cluster_peer(qs + 2048 + at * (D * 4) + ((pc + r) % PC) * 16, p))
                       : "memory");
          const float e = fast_exp2(pm - m);
          l += pl * e;
          o.x += v.x * e;
          o.y += v.y * e;
          o.z += v.z * e;
          o.w += v.w * e;
        }
        const float inv = a.v_mul / l;
        T* out = static_cast<T*>(a.out) +
                 (static_cast<int64_t>(it.qbeg + it.i0 + x * QB + r / G) * a.H_q + it.g * G + r % G) * D + 4 * pc;
        *reinterpret_cast<uint2*>(out) = make_uint2(pack2<T>(o.x * inv, o.y * inv), pack2<T>(o.z * inv, o.w * inv));
      }
    }
    cluster_barrier();  // peers may still read this CTA's partials
  }
}

int encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* p, const cuuint64_t* dims,
           const cuuint64_t* strides, const cuuint32_t* box, const char* what) {
  const cuuint32_t ones[3] = {1, 1, 1};
  const CUresult r = encode_fn()(map, type, rank, const_cast<void*>(p), dims, strides, box, ones,
                                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(PKV_ERR_CUDA, std::string("cuTensorMapEncodeTiled (") + what + ") failed: " + std::to_string(r));
  return PKV_OK;
}

template <typename T, bool KV8, int D>
int launch_t(Pool& P, DecodeArgs& a, CUtensorMap* maps, const int32_t* q_off, int32_t max_q, int32_t n_tok,
             cudaStream_t st) {
  using C = WpCfg<KV8, D>;
  max_q = std::min(max_q, n_tok);  // no chunk is longer than that
  const void* k = reinterpret_cast<const void*>(&prefill_win_kernel<T, KV8, D>);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("device query: ") + cudaGetErrorString(e));
  // items at most: by rows (each sequence adds a ragged pair of blocks) and by the longest chunk
  const int64_t two = 2 * (128 / a.G), most = (static_cast<int64_t>(max_q) + two - 1) / two;
  int64_t items =
      std::min(most * a.n_seq, static_cast<int64_t>(n_tok) / two + a.n_seq) * P.geo.H_kv;
  // key tiles of an item at most: the table's, or those of the sinks, the window and the item's queries
  const int64_t keys = std::min(static_cast<int64_t>(a.W) * a.B,
                                static_cast<int64_t>(a.n_sink) + a.window + std::min<int64_t>(max_q, two) + 2 * TILE);
  int32_t csize = 1;
  while (csize < 8 && items * csize * 2 <= sms && keys >= 2 * csize * C::KEYS) csize *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(csize > 1 ? items * csize : std::min<int64_t>(items, sms)));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = csize > 1 ? 1 : 0;
  void* args[] = {&maps[0], &maps[1], &maps[2], &a, const_cast<int32_t**>(&q_off), &max_q, &csize, &items};
  e = cudaLaunchKernelExC(&cfg, k, args);
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("windowed prefill launch: ") + cudaGetErrorString(e));
  count_launch();
  return PKV_OK;
}

}  // namespace

// The geometries that the kernel takes.
bool win_prefill_ok(const pkv_geometry& g) {
  const bool dt = ((g.dtype == PKV_BF16 || g.dtype == PKV_F16) && (g.d_head == 64 || g.d_head == 128)) ||
                  (g.dtype == PKV_E4M3 && g.d_head == 128);
  return dt && g.H_q / g.H_kv <= 128 && g.block_size % TILE == 0 &&
         g.num_blocks * g.L * g.H_kv * g.block_size < (int64_t(1) << 31) && encode_fn() != nullptr;
}

int launch_prefill_window(Pool& P, DecodeArgs& a, const void* q, const int32_t* q_off, int32_t n_tok, int32_t max_q,
                          const void* k_pool, const void* v_pool, cudaStream_t st) {
  const auto& g = P.geo;
  const cuuint64_t d = static_cast<cuuint64_t>(g.d_head);
  const cuuint64_t rows = static_cast<cuuint64_t>(g.num_blocks) * g.L * g.H_kv * g.block_size;
  const CUtensorMapDataType act =
      g.dtype == PKV_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;  // q: bf16 for E4M3
  CUtensorMap maps[3];
  if (int rc = get_tensor_maps(P, k_pool, v_pool, &maps[1], &maps[2])) return rc;
  {  // q: a {64, G, 128 / G} box lands as (query, head) rows of 128 bytes
    const cuuint64_t dims[3] = {d, static_cast<cuuint64_t>(g.H_q), static_cast<cuuint64_t>(n_tok)};
    const cuuint64_t strides[2] = {d * 2, d * 2 * static_cast<cuuint64_t>(g.H_q)};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(128 / a.G)};
    if (int rc = encode(&maps[0], act, 3, q, dims, strides, box, "q")) return rc;
  }
  if (g.dtype != PKV_E4M3 && g.d_head == 128) {  // V: a {64, 16, 2} box is a slab, chunk after chunk
    const cuuint64_t dims[3] = {64, rows, 2}, strides[2] = {256, 128};
    const cuuint32_t box[3] = {64, TILE, 2};
    if (int rc = encode(&maps[2], act, 3, v_pool, dims, strides, box, "v slabs")) return rc;
  }
  if (g.dtype == PKV_E4M3) return launch_t<__nv_bfloat16, true, 128>(P, a, maps, q_off, max_q, n_tok, st);
  const bool bf = g.dtype == PKV_BF16;
  if (g.d_head == 128)
    return bf ? launch_t<__nv_bfloat16, false, 128>(P, a, maps, q_off, max_q, n_tok, st)
              : launch_t<__half, false, 128>(P, a, maps, q_off, max_q, n_tok, st);
  return bf ? launch_t<__nv_bfloat16, false, 64>(P, a, maps, q_off, max_q, n_tok, st)
            : launch_t<__half, false, 64>(P, a, maps, q_off, max_q, n_tok, st);
}

}  // namespace pkv
