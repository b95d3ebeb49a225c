// Chunked-prefill attention with a sliding window and sinks on the 5th-generation tensor cores.
//
// What it computes: query i of sequence s's chunk, at position p = len_s - C_s + i, sees the keys t <= p with
// t > p - window or t < n_sink; out = softmax(scale q K^T) V over those (bf16, f16 and E4M3 pools, d_head 128, and 64
// for the 16-bit pools; the block size a multiple of 16).
//
// Work: an item is a (sequence, KV head, pair of query blocks); its rows are two M = 128 tiles A and B of (query, head)
// pairs (row r = query r / G, head r % G).  The keys that some query of the item sees are a list of 16-token slabs --
// the sinks' slabs, then those from the window's start to the last query -- taken 8 slabs (128 keys) at a time, so that a
// few sinks cost one slab, not a tile of their own.  Slabs lie in pool blocks of their own: each is one or two TMA boxes.
//
// What bounds it: 4 d flops a (row, key) on the tensor cores, against 128 exponentials a row and key tile on the CUDA
// cores; the two products of a tile (A) run while the softmax of the other (B) does, so the longer of the two counts.
// N = 128 keys a product lets its shared-memory reads (A and B operands, 8 KB a K = 16 step) keep up with the
// multiplies, which N = 64 does not.  A window makes items short (a window of 1,024 is 9 key tiles), so what surrounds them
// counts: the grid is persistent, and loads, products and softmax of the next item start while this one's rows are written.
//
// Roles (warps): 0-3 softmax and epilogue of A, 4-7 of B (a thread a row, its TMEM lane); 8 loads K and V; 9 and 11
// issue the products of A and of B; 10 loads Q and zeroes V rows that no row sees (0 times whatever lies there must
// stay 0).  E4M3 pools: K codes are an operand as they are, with q as the sum of two E4M3 numbers (two products at
// twice the rate), and V codes are converted to binary16, both by warps 12-15.
// TMEM: S of A and B (128 columns each; P overwrites its last 64), O of A and B from column 256 on.
// A tile's products are issued by one thread and taken in order, ..., P V(j), Q K(j + 1), ...: S(j + 1) may go over
// P(j), and its arrival says that O holds P V(j).
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

constexpr int WP_KEYS = 128, WP_SLABS = WP_KEYS / TILE;

template <bool KV8, int D>
struct WpCfg {
  static constexpr int THREADS = KV8 ? 512 : 384;
  static constexpr int TBL = KV8 ? 128 : 256;             // entries of the table that finds an item's sequence
  static constexpr int NCH = D / 64;                      // 64-wide chunks of d (128 bytes, the swizzle's width)
  static constexpr int Q_TILE = 128 * D * 2;              // one Q tile (E4M3: its two parts, below)
  static constexpr int KV_TILE = WP_KEYS * D * 2;         // one K or V tile of 16-bit operands
  static constexpr int F8_TILE = WP_KEYS * D;             // one of E4M3 codes
  // 16-bit pools: one ring of KS operands, K and V tiles in turn.  E4M3 pools: KS K tiles, FS staged V tiles and VS
  // converted ones.
  static constexpr int KS = KV8 ? 4 : (D == 64 ? 8 : 5), FS = KV8 ? 2 : 0, VS = KV8 ? 2 : 0;
  static constexpr int DATA = 2 * Q_TILE + (KV8 ? KS * F8_TILE + VS * KV_TILE + FS * F8_TILE : KS * KV_TILE);
  static constexpr int BARS = 3 + 3 * KS + 6 * 2 + 4 + 2 * FS + 2 * VS;
  static constexpr int READERS = THREADS / 32 - 1;        // warps that follow the items
  static constexpr int SMEM = 1024 + DATA + (BARS + 1) * 8 + 16 + 2 * 64 + 96 + (TBL + 1) * 4 + (KV8 ? 512 : 0);
  // registers: the launch's share is 65,536 / THREADS rounded down to a multiple of 8
  static constexpr int R_LAUNCH = KV8 ? 128 : 168;
  static constexpr int R_SOFTMAX = KV8 ? 168 : 208, R_CONTROL = KV8 ? 72 : 88, R_CONVERT = 96;
  static_assert(256 * R_SOFTMAX + 128 * R_CONTROL + (KV8 ? 128 * R_CONVERT : 0) <= THREADS * R_LAUNCH, "register split");
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

// four E4M3 codes to binary16 (exact), the first of each pair low
__device__ __forceinline__ void f16_of_e4m3(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
// two values to E4M3 codes (the first low), and the rest that the codes leave of them, as codes
__device__ __forceinline__ void e4m3_split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
  uint32_t h2;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(h2) : "r"(hi));
  const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&h2));
  lo = __nv_cvt_float2_to_fp8x2(make_float2(x - back.x, y - back.y), __NV_SATFINITE, __NV_E4M3);
}

// D(tmem) (+)= A(smem) B(smem)^T on 8-bit operands, K = 32
__device__ __forceinline__ void umma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\ntcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor of kind::f8f6f4: binary32 accumulator, A and B both E4M3 (format 0) and K-major
__host__ __device__ constexpr uint32_t umma_idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
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
struct __align__(16) Item {
  int32_t s, g;
  int32_t qbeg, i0, i1, nq;              // chunk's first row; its queries i0 .. i1 - 1; tiles with rows (1, 2)
  int32_t P, nkeys;                      // position of query 0; keys up to the last query
  int32_t sink_end, lo;                  // a key t is hidden from every row if sink_end <= t < lo
  int32_t sink_slabs, first, nslab;      // the slab list: 0 .. sink_slabs - 1, then from `first` on
  int32_t j0, j1;                        // this CTA's key tiles
  int32_t work;                          // 0: no item (any more)
  __device__ __forceinline__ int32_t slab(int32_t u) const { return u < sink_slabs ? u : first + u - sink_slabs; }
  __device__ __forceinline__ int32_t slabs_of(int32_t j) const { return min(WP_SLABS, nslab - j * WP_SLABS); }
  __device__ __forceinline__ bool hidden(int32_t t) const { return t >= nkeys || (t >= sink_end && t < lo); }
  __device__ __forceinline__ bool ragged(int32_t u) const {  // slab u holds a key hidden from every row
    return hidden(slab(u) * TILE) || hidden(slab(u) * TILE + TILE - 1) ||
           (sink_end < lo && slab(u) * TILE < lo && slab(u) * TILE + TILE > sink_end);
  }
  // tile j holds such a slab: only the last with sinks, the first after them and the last can
  __device__ __forceinline__ bool zeroes(int32_t j) const {
    const int32_t a = j * WP_SLABS, b = a + slabs_of(j);
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
  constexpr bool BF16 = std::is_same<T, __nv_bfloat16>::value && !KV8;  // type of P and V as operands
  using TP = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int KS = C::KS, FS = C::FS, VS = C::VS;
  extern __shared__ uint8_t smem_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = a.G, QB = 128 / G;  // queries a tile
  const int rank = csize > 1 ? blockIdx.x % csize : 0;

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t qs = smem_u32(base), ring = qs + 2 * C::Q_TILE;
  uint8_t* ring_p = base + 2 * C::Q_TILE;
  uint8_t* vop_p = ring_p + KS * C::F8_TILE;  // E4M3: converted V tiles, then staged ones
  uint8_t* stg_p = vop_p + VS * C::KV_TILE;
  uint8_t* bar_p = base + C::DATA;
  const uint32_t q_full = smem_u32(bar_p), q_ready = q_full + 8, q_empty = q_full + 16;
  const uint32_t full = q_full + 24, empty = full + 8 * KS, land = empty + 8 * KS;  // operand ring; V tiles to be zeroed
  // per tile A, B: S; the first three quarters of P, all of it; the item's O; the turn to issue; after an abort
  const uint32_t s_full = land + 8 * KS, p_most = s_full + 16, p_full = p_most + 16, o_full = p_full + 16;
  const uint32_t turn = o_full + 16, drain = turn + 16;
  const uint32_t sf_full = drain + 16, sf_empty = sf_full + 8 * FS;             // staged V (E4M3)
  const uint32_t vo_full = sf_empty + 8 * FS, vo_empty = vo_full + 8 * VS;      // converted V
  const uint32_t it_full = vo_empty + 8 * VS, it_empty = it_full + 16;          // items, two places
  uint8_t* tail_p = bar_p + (C::BARS + 1) / 2 * 16;
  Item* items_p = reinterpret_cast<Item*>(tail_p);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tail_p + 2 * sizeof(Item));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  int32_t* wsum = reinterpret_cast<int32_t*>(tslot + 4);
  int8_t* q_exp = reinterpret_cast<int8_t*>(wsum + 24);  // E4M3: exponents of the rows' q, of two items in turn
  int32_t* pre = wsum + 24 + (KV8 ? 128 : 0);  // [groups + 1]: query-block pairs of the sequences before a group of them

  if (tid == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_ready, 4);  // one arrival a warp
    mbar_init(q_empty, 2);
    for (int k = 0; k < KS; ++k) {
      mbar_init(full + 8 * k, 1);
      mbar_init(empty + 8 * k, 2);  // both tiles' products
      mbar_init(land + 8 * k, 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(s_full + 8 * x, 1);
      mbar_init(p_most + 8 * x, 4);  // one arrival a warp
      mbar_init(p_full + 8 * x, 4);
      mbar_init(turn + 8 * x, 1);
      mbar_init(o_full + 8 * x, 1);
      mbar_init(drain + 8 * x, 1);
    }
    for (int k = 0; k < FS; ++k) {
      mbar_init(sf_full + 8 * k, 1);
      mbar_init(sf_empty + 8 * k, 4);
    }
    for (int k = 0; k < VS; ++k) {
      mbar_init(vo_full + 8 * k, 4);
      mbar_init(vo_empty + 8 * k, 2);
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
  // `per` sequences (one, up to C::TBL of them), and the table holds the sums before each such group
  const int most = (max_q + 2 * QB - 1) / (2 * QB);  // query-block pairs of a chunk at most
  const int per = (a.n_seq + C::TBL - 1) / C::TBL, groups = (a.n_seq + per - 1) / per;
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

  // item idx; false for one without work.  `record` reports bad values.
  auto get = [&](int64_t idx, Item& w, bool record) __attribute__((always_inline)) -> bool {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(pre[mid]) * a.H_kv <= idx) lo = mid; else hi = mid - 1;
    }
    int64_t r = idx - static_cast<int64_t>(pre[lo]) * a.H_kv;
    w.s = lo * per;
    int nb = pairs_of(w.s, false);
    while (r >= static_cast<int64_t>(nb) * a.H_kv && w.s + 1 < a.n_seq) {
      r -= static_cast<int64_t>(nb) * a.H_kv;
      nb = pairs_of(++w.s, false);
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
      uint32_t c = 0;  // tiles loaded so far (E4M3: pairs of them)
      uint32_t on_land = 0;  // of the last KS tiles, those whose bytes arrive at `land` (bit c % KS)
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
          if constexpr (KV8) {
            const uint32_t ks = c % KS, fs = c % FS;
            if (lane == 0) {
              if (c >= KS) ok = wait(empty + 8 * ks, ((c / KS) - 1) & 1, 100);
              if (ok) mbar_arrive_expect_tx(full + 8 * ks, ns * TILE * D);
            }
            ok = warp_ok(ok);  // also orders the expect_tx before the copies
            if (!ok) break;
            if (mine) tma_load_2d(ring + ks * C::F8_TILE + i * TILE * 128, &tmk, 0, row, full + 8 * ks);
            if (lane == 0) {
              if (c >= FS) ok = wait(sf_empty + 8 * fs, ((c / FS) - 1) & 1, 110);
              if (ok) mbar_arrive_expect_tx(sf_full + 8 * fs, ns * TILE * D);
            }
            ok = warp_ok(ok);
            if (!ok) {
              ++c;  // K is on its way
              break;
            }
            if (mine) tma_load_2d(smem_u32(stg_p) + fs * C::F8_TILE + i * TILE * 128, &tmv, 0, row, sf_full + 8 * fs);
            ++c;
          } else {
            for (int kv = 0; kv < 2 && ok; ++kv, ++c) {
              const uint32_t slot = c % KS;
              const bool zero = kv == 1 && w.zeroes(j);
              const uint32_t bar = zero ? land + 8 * slot : full + 8 * slot;
              if (lane == 0) {
                if (c >= KS) ok = wait(empty + 8 * slot, ((c / KS) - 1) & 1, 100);
                if (ok) mbar_arrive_expect_tx(bar, ns * TILE * D * 2);
              }
              ok = warp_ok(ok);
              if (!ok) break;
              on_land = (on_land & ~(1u << slot)) | (zero ? 1u << slot : 0u);
              if (zero) land_par ^= 1u << slot;
              const uint32_t dst = ring + slot * C::KV_TILE;
              if (mine) {
                if (kv == 0) {
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
      }
      if (*abort_flag && lane == 0) {  // copies may still be landing in the rings' last slots
        for (uint32_t k = c > KS ? c - KS : 0; k < c; ++k) {
          const uint32_t slot = k % KS;
          if (!KV8 && (on_land >> slot & 1)) settle(land + 8 * slot, ~(land_par >> slot) & 1);
          else settle(full + 8 * slot, (k / KS) & 1);
        }
        if constexpr (KV8)
          for (uint32_t k = c > FS ? c - FS : 0; k < c; ++k) settle(sf_full + 8 * (k % FS), (k / FS) & 1);
      }
    } else if (warp == 9 || warp == 11) {
      // ------------------------------------------------------------ the products of tile X (9: A, 11: B)
      // The whole warp walks the items, so that descriptors stay warp-uniform, and one elected lane issues: a
      // divergent thread on its own needs some 140 cycles a product to bring its operands into uniform registers.
      // A and B take turns, (P V, Q K) of one, then of the other, so that S of A arrives while B's products run and the
      // two softmaxes stay half a period apart; issued side by side, the products of both end together, and then both
      // softmaxes run while the tensor cores wait.  A tile without rows (nq = 1) has its turns all the same.
      // (the broadcasts from lane 0 are what tells the compiler that a value is the same in all lanes)
      auto uni = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
      const int X = uni(warp == 9 ? 0 : 1);
      const uint32_t s_tm = uni(tmem) + 128 * X, o_tm = uni(tmem) + 256 + 128 * X;
      const uint32_t idesc_o = umma_idesc_f16(BF16, 128, D, true);
      // operand descriptors: the first, and a step of the address field (16-byte units) from there on
      const uint64_t q_desc = umma_desc_sw128(uni(qs) + X * C::Q_TILE, 16, 1024);
      const uint64_t k_desc = umma_desc_sw128(uni(ring), 16, 1024);
      const uint64_t v_desc = umma_desc_sw128(uni(KV8 ? smem_u32(vop_p) : ring), TILE * 128, 1024);
      const uint32_t bars = uni(q_full);  // the barriers from here on
      const uint32_t u_empty = bars + (empty - q_full), u_q_empty = bars + 16;
      const uint32_t u_v_empty = bars + ((KV8 ? vo_empty : empty) - q_full);
      const uint32_t u_s_full = bars + (s_full - q_full) + 8 * X, u_o_full = bars + (o_full - q_full) + 8 * X;
      const uint32_t u_turn = bars + (turn - q_full) + 8 * (1 - X);  // the other tile's
      auto wait_all = [&](uint32_t bar, uint32_t parity, int where) {
        return __all_sync(0xffffffffu, wait(bar, parity, where)) != 0;
      };
      auto commit = [&](uint32_t bar) {
        if (elect_one()) umma_commit(bar);
      };
      constexpr uint32_t VS_ = VS > 0 ? VS : 1;
      uint32_t c = 0, vc = 0, items = 0, np = 0, turns = 0;  // ring positions; items; P tiles taken; turns had
      while (ok && next_item(w)) {
        if (w.j0 == w.j1) continue;  // a cluster rank without a key tile
        const bool live = uni(X < w.nq) != 0;
        const int nt = uni(w.j1 - w.j0), nslab = uni(w.nslab - w.j0 * WP_SLABS);
        ok = wait_all(KV8 ? q_ready : q_full, items++ & 1, 200);
        for (int i = -1; i < nt && ok; ++i) {  // P V of the item's i-th key tile, then Q K of the next
          // everything is waited for before the turn: within it the products follow each other without a gap
          const bool has_pv = i >= 0, has_qk = i + 1 < nt;
          // 16-bit pools: ring position c, V and K tiles in turn; E4M3 pools: key tile c of each of the two rings
          const uint32_t vs = KV8 ? vc % VS_ : c % KS, ks = (KV8 ? c : c + has_pv) % KS;
          if (has_pv) {
            ok = KV8 ? wait_all(vo_full + 8 * vs, (vc / VS_) & 1, 210) : wait_all(full + 8 * vs, (c / KS) & 1, 210);
            if (KV8) ++vc; else ++c;
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
          const uint64_t vd = v_desc + vs * (C::KV_TILE / 16), kd = k_desc + ks * ((KV8 ? C::F8_TILE : C::KV_TILE) / 16);
          const int nv = has_pv ? min(WP_SLABS, nslab - i * WP_SLABS) : 0;
          const int nk = has_qk ? min(WP_SLABS, nslab - (i + 1) * WP_SLABS) * TILE : TILE;
          const uint32_t idesc_s = KV8 ? umma_idesc_e4m3(128, nk) : umma_idesc_f16(BF16, 128, nk, false);
          // P of keys 0 .. 31 and 64 .. 127 comes first (slabs 0, 1, 4 .. 7; slab 0 is always there)
          auto pv = [&](int k) {
            if (k < nv)
              umma_ts(o_tm, s_tm + 64 + 8 * k, vd + k * (C::NCH * TILE * 128 / 16), idesc_o, i > 0 || k > 0 ? 1u : 0u);
          };
          if (live && has_pv) {  // three quarters of P, then (it came meanwhile) the rest
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < WP_SLABS; ++k)
                if (k < 2 || k >= 4) pv(k);
            }
            __syncwarp();
            ok = wait_all(p_full + 8 * X, np++ & 1, 250);
            if (!ok) break;
            tc_fence_after();
          }
          if (elect_one()) {
            if (live) {
#pragma unroll
              for (int k = 2; k < 4; ++k) pv(k);
              if (has_qk) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  // the other tile's warp is let go two products early, which hides its start
                  if (k == D / 16 - 2) mbar_arrive(u_turn);
                  // 16-bit: 64-wide chunk k / 4; 32 bytes along its 128-byte row.  E4M3: part k / 4 of q; all of d is one row
                  const uint64_t qk = q_desc + ((k >> 2) * 16384 + (k & 3) * 32) / 16;
                  if constexpr (KV8) umma_f8(s_tm, qk, kd + (k & 3) * 2, idesc_s, k > 0);
                  else umma_ss(s_tm, qk, kd + ((k >> 2) * (WP_KEYS * 128) + (k & 3) * 32) / 16, idesc_s, k > 0);
                }
                umma_commit(u_s_full);
              } else {
                mbar_arrive(u_turn);
                umma_commit(u_o_full);
              }
              // this tile's use of the operands is over once its products so far are done
              if (has_pv) umma_commit(u_v_empty + 8 * vs);
              if (has_qk) umma_commit(u_empty + 8 * ks);
              if (i + 2 == nt) umma_commit(u_q_empty);
            } else {
              mbar_arrive(u_turn);
              if (has_pv) mbar_arrive(u_v_empty + 8 * vs);
              if (has_qk) mbar_arrive(u_empty + 8 * ks);
              if (i + 2 == nt) mbar_arrive(u_q_empty);
            }
          }
          __syncwarp();
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
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::R_CONVERT));
      const int r = tid & 127;
      uint32_t c = 0, items = 0;
      while (ok && next_item(w)) {
        if (w.j0 == w.j1) continue;
        ok = __all_sync(0xffffffffu, wait(q_full, items & 1, 500));
        if (!ok) break;
        // Row r of each tile, 128 bf16 in two 128-byte rows of eight 16-byte units (unit u at u ^ (r & 7)), scaled by a power
        // of two that brings its largest element to [128, 256), becomes x = hi + lo, both E4M3, 128 bytes each in the
        // same two places: bf16 has 8 significant bits and E4M3 4, so the rest after hi is an E4M3 number again, down to
        // 2^-10 (2^-17 of the row's largest).
        for (int x = 0; x < w.nq; ++x) {
          uint8_t* qr = base + x * C::Q_TILE + r * 128;
          uint32_t mx = 0;  // the largest magnitude as bf16 bits, two side by side
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const uint4 v = *reinterpret_cast<const uint4*>(qr + (u >> 3) * 16384 + (((u & 7) ^ (r & 7)) << 4));
            mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                       __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
          }
          mx = max(mx & 0xffffu, mx >> 16);
          // a row with an infinity or a NaN is NaN throughout (0 times it is)
          const int e = max(-120, min(120, 134 - static_cast<int>(mx >> 7)));
          const float f = mx >= 0x7f80u ? __uint_as_float(0x7fc00000u) : __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
          q_exp[(items & 1) * 256 + x * 128 + r] = static_cast<int8_t>(e);
          uint4 hi[8], lo[8];  // all read before any is written
#pragma unroll
          for (int u = 0; u < 16; ++u) {
            const uint4 v = *reinterpret_cast<const uint4*>(qr + (u >> 3) * 16384 + (((u & 7) ^ (r & 7)) << 4));
            const uint32_t p[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4], l[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              e4m3_split(__uint_as_float(p[k] << 16) * f, __uint_as_float(p[k] & 0xffff0000u) * f, h[k], l[k]);
            uint32_t* ho = &hi[u >> 1].x + 2 * (u & 1);
            uint32_t* lw = &lo[u >> 1].x + 2 * (u & 1);
            ho[0] = h[0] | h[1] << 16, ho[1] = h[2] | h[3] << 16;
            lw[0] = l[0] | l[1] << 16, lw[1] = l[2] | l[3] << 16;
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            *reinterpret_cast<uint4*>(qr + ((u ^ (r & 7)) << 4)) = hi[u];
            *reinterpret_cast<uint4*>(qr + 16384 + ((u ^ (r & 7)) << 4)) = lo[u];
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_ready);
        ++items;
        for (int j = w.j0; j < w.j1 && ok; ++j, ++c) {
            const uint32_t f = c % 2, slot = c % 2;
            bool here = wait(sf_full + 8 * f, (c / 2) & 1, 510);
            if (here && c >= 2) here = wait(vo_empty + 8 * slot, ((c / 2) - 1) & 1, 520);
            ok = __all_sync(0xffffffffu, here);
            if (!ok) break;
            const uint8_t* src = stg_p + f * C::F8_TILE;
            uint8_t* dst = vop_p + slot * C::KV_TILE;
            const int ns = w.slabs_of(j);
            const bool zero = w.zeroes(j);
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
              uint8_t* p = dst + i * (2 * TILE * 128) + cc * (TILE * 128) + rr * 128;
              *reinterpret_cast<uint4*>(p + ((t ^ sw) << 4)) = o0;
              *reinterpret_cast<uint4*>(p + (((t + 1) ^ sw) << 4)) = o1;
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(vo_full + 8 * slot);
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
    const uint32_t s_addr = lane_addr + 128 * X, o_addr = lane_addr + 256 + 128 * X;
    uint32_t n_s = 0, no = 0, items = 0;  // S tiles and outputs taken; items
    while (ok && next_item(w)) {
      const uint32_t item = w.j0 < w.j1 ? items++ : 0;
      if (X >= w.nq) continue;
      const int qi = w.i0 + X * QB + r / G;
      const bool valid = r < QB * G && qi < w.i1;
      const int lim = valid ? w.P + qi : w.nkeys - 1;                  // last visible key
      const int low = visible_at(a.window, a.n_sink, lim).lo;          // from here on visible, before only the sinks
      float m = -INFINITY, l = 0.f, sl = a.scale_log2;
      for (int j = w.j0; j < w.j1 && ok; ++j, ++n_s) {
        ok = __all_sync(0xffffffffu, wait(s_full + 8 * X, n_s & 1, 600));
        if (!ok) break;
        tc_fence_after();
        if (KV8 && j == w.j0)  // the row's q is scaled by 2^e
          sl *= __uint_as_float(static_cast<uint32_t>(127 - q_exp[(item & 1) * 256 + X * 128 + r]) << 23);
        uint32_t sa[2][32], sb[2][32];  // the first 64 keys and the others
        tmem_ld32(s_addr, sa[0]);
        tmem_ld32(s_addr + 32, sa[1]);
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
        float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        auto largest = [&](const uint32_t (&x)[2][32]) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 32; e += 8)
#pragma unroll
              for (int t = 0; t < 4; ++t)
                mx4[t] = fmaxf(mx4[t], fmaxf(__uint_as_float(x[c][e + t]), __uint_as_float(x[c][e + t + 4])));
        };
        tmem_ld_wait();
        tmem_ld32(s_addr + 64, sb[0]);  // on their way during the first half's maximum
        tmem_ld32(s_addr + 96, sb[1]);
        if (edge) mask(sa, 0);
        largest(sa);
        tmem_ld_wait();
        if (edge) mask(sb, 4);
        largest(sb);
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        const float m_new = fmaxf(m, mx * sl);
        // the reference maximum moves when a row's grows by more than 2^8 (until then P and l share the old one):
        // l and O so far are rescaled; S(j) is here, so O holds P V(j - 1)
        if (__any_sync(0xffffffffu, m_new > m + 8.f)) {
          const float alpha = m_new == -INFINITY ? 1.f : fast_exp2(m - m_new);
          if (j > w.j0) {
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
        // P = 2^(scale s - m), 16-bit, two keys a column, over S of the other keys, which are taken first: E4M3 pools,
        // whose softmax has fewer registers, read S of the first 64 a second time instead of keeping it; a row that
        // has seen no key yet keeps m = -inf, and 0 stands in for it
        const float neg_m = m == -INFINITY ? 0.f : -m;
        float2 ls[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) ls[t] = make_float2(0.f, 0.f);
        auto exps = [&](const uint32_t (&x)[32], uint32_t at) {
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
        exps(sb[0], s_addr + 96);
        exps(sb[1], s_addr + 112);
        if constexpr (KV8) {
          tmem_ld32(s_addr, sa[0]);
          tmem_ld32(s_addr + 32, sa[1]);
          tmem_ld_wait();
          if (edge) mask(sa, 0);
        }
        exps(sa[0], s_addr + 64);
        arrive(p_most + 8 * X);  // P V may begin with three quarters of the keys
        exps(sa[1], s_addr + 80);
        arrive(p_full + 8 * X);
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
  while (csize < 8 && items * csize * 2 <= sms && keys >= 2 * csize * WP_KEYS) csize *= 2;
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
