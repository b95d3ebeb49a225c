// One 16-token tile of paged decode attention on tensor cores, shared by the decode kernels: the
// tile's shared-memory layout, the keys of a sequence that a launch attends to, and the step that
// folds a tile into a warp's running softmax.
#pragma once

#include "pkv_attn.cuh"

namespace pkv {

// The keys of sequence s that this kernel attends to: `len` tokens from table block `kb` on.
// kb is the shared prefix's block count (share[s].x) when one is given and leaves at least one
// token, else 0 (an out-of-range value is recorded and ignored); len is the length clamped to
// the table's capacity [0, W*B], minus the prefix.  `record` reports bad values.
struct Span {
  int32_t len, kb;
};
__device__ __forceinline__ Span seq_span(const DecodeArgs& a, int s, bool record) {
  int32_t len = a.seq_lens[s];
  const int64_t maxlen = static_cast<int64_t>(a.W) * a.B;
  if (len < 0 || len > maxlen) {
    if (record) record_error(a.err, DERR_DECODE_LEN, s);
    len = len < 0 ? 0 : static_cast<int32_t>(maxlen);
  }
  int32_t kb = 0;
  if (a.share) {
    kb = a.share[s].x;
    if (kb < 0 || static_cast<int64_t>(kb) * a.B >= len) {
      if (record && kb != 0) record_error(a.err, DERR_SHARE, s);
      kb = 0;
    }
  }
  return Span{len - kb * a.B, kb};
}
__device__ __forceinline__ int32_t clamped_len(const DecodeArgs& a, int s, bool record) {
  return seq_span(a, s, record).len;
}

// With a window: the tiles of sequence s that hold a visible key -- sink tiles 0 .. sink_tiles - 1,
// then from tile `first` on -- and which keys those are.  Every one of them has a visible key.
struct WinTiles {
  int32_t len, ns, lo, sink_tiles, first, n;
  __device__ __forceinline__ int32_t token0(int32_t j) const {  // first token of the j-th of them
    return (j < sink_tiles ? j : first + j - sink_tiles) * TILE;
  }
};
__device__ __forceinline__ WinTiles win_tiles(const DecodeArgs& a, int s, bool record) {
  WinTiles w;
  w.len = clamped_len(a, s, record);
  const Visible v = visible_at(a.window, a.n_sink, w.len - 1);
  w.ns = v.ns;
  w.lo = v.lo;
  w.sink_tiles = (v.ns + TILE - 1) / TILE;
  w.first = max(w.sink_tiles, v.lo / TILE);
  w.n = w.sink_tiles + (w.len + TILE - 1) / TILE - w.first;
  return w;
}
// Tiles of sequence s that the launch attends to.
template <bool WIN>
__device__ __forceinline__ int32_t seq_tiles(const DecodeArgs& a, int s, bool record) {
  if constexpr (WIN) return win_tiles(a, s, record).n;
  return (clamped_len(a, s, record) + TILE - 1) / TILE;
}

// --------------------------------------------------------------------------- tensor-core tiles

// EB: bytes per stored K/V element; NB: 8-head column blocks of the mma N dimension (1 for
// G <= 8, 2 for 9 <= G <= 16: every K/V fragment loaded from shared memory feeds NB mmas).
template <int D, int EB = 2, int NB = 1>
struct TcCfg {
  static constexpr int GP = GPAD * NB;                     // query rows held per group (padded)
  static constexpr int KV_TILE_BYTES = TILE * D * EB;     // one 16 x D tile of K (or V)
  static constexpr int Q_BYTES = GP * D * 2;               // up to GP query rows (16-bit)
  static constexpr int STAGE_BYTES = 2 * KV_TILE_BYTES + Q_BYTES;
  static constexpr int NBOX = D * EB / 128;                // 128-byte TMA boxes per tile row
  static constexpr int BOX_ELEMS = 128 / EB;
  static constexpr int NKC = D / 16;                       // 16-wide chunks of d_head
  static constexpr int OFL = NKC * 32 * 4;                 // floats of one head block's O^T fragments
  // floats per partial slot: the O^T fragments of each head block, then m[GP], then l[GP]
  static constexpr int PSTRIDE = NB * OFL + 2 * GP;
  static_assert(STAGE_BYTES % 1024 == 0, "stages must keep 1024-byte alignment for the swizzle");
};

// Four E4M3 codes (bytes 0..3 of w) to binary16 pairs (exact): lo = (b0, b1), hi = (b2, b3),
// the first of each pair in the low half.
__device__ __forceinline__ void e4m3x4_to_f16x2x2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// Two bfloat16 values (low half first) to two binary16 values (round to nearest).
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t w) {
  __half2 h = __floats2half2_rn(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w));
}

// Descriptor of one tile, built by the warp a batch at a time:
//   x = TMA row coordinate of the slab, y = pair id (s * H_kv + g),
//   z = valid tokens | first-of-pair << 8 | last-of-pair << 9 | new-pair-in-range << 10,
//   w = tiles of the sequences before s (the pair's place in the batch's tile order).
// With a window z also holds which rows of the tile are hidden, those from row (z >> 16) & 31 (the
// sinks' end) up to row (z >> 24) & 31 (the window's start), none when the first is not below.
constexpr int F_FIRST = 1 << 8, F_LAST = 1 << 9, F_NEWPAIR = 1 << 10;

// Fold one tile (K then V in shared memory at `stage`, its shared address sk, 128-byte swizzle) into a warp's running
// softmax of the group's query heads.  z: the tile's valid tokens and hidden rows (above).  qf: the
// warp's q fragments; per head block nb the O^T fragments o, running maxima m (base 2) and sums l
// of heads 8 nb + 2 (lane & 3) and + 1 (l: this lane's part).
template <typename T, int D, int NB, bool WIN>
__device__ __forceinline__ void attend_tile(uint8_t* stage, uint32_t sk, int z, float scale_log2, int lane,
                                            const uint32_t (&qf)[NB][D / 16][2], float (&o)[NB][D / 16][4],
                                            float (&m)[NB][2], float (&l)[NB][2]) {
  constexpr bool F8 = std::is_same<T, E4M3>::value;
  using TM = typename std::conditional<F8, __half, T>::type;
  constexpr bool BF16 = std::is_same<TM, __nv_bfloat16>::value;
  using C = TcCfg<D, F8 ? 1 : 2, NB>;
  const uint32_t sv = sk + C::KV_TILE_BYTES;
  // per-lane ldmatrix geometry (128-byte swizzle: chunk c of row r sits at c ^ (r & 7))
  const int r8 = lane & 7, mi = lane >> 3;
  const int k_row = r8 + 8 * (mi & 1), k_add = mi >> 1;  // QK: A = K tile (t x d)
  const int v_row = r8 + 8 * (mi >> 1), v_add = mi & 1;  // PV: A = V^T via .trans
  const int trow = lane >> 2;                            // token row of c0/c1 (c2/c3: +8)
  const int c4 = lane & 3;
  // ---- S^T = K q^T  (16 tokens x 8 heads per block), two accumulation chains per block
  float sa[NB][4], sb[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int r = 0; r < 4; ++r) sa[nb][r] = sb[nb][r] = 0.f;
  if constexpr (F8) {
    // K rows trow and trow + 8, bytes 32 c4 .. 32 c4 + 31 (16-byte chunks 2c4, 2c4 + 1; swizzle
    // XOR = row & 7 = trow); step c takes bytes 4c .. 4c + 3 of each row
    const uint4 ka0 = lds128(sk + trow * 128 + (((2 * c4) ^ trow) << 4));
    const uint4 ka1 = lds128(sk + trow * 128 + (((2 * c4 + 1) ^ trow) << 4));
    const uint4 kb0 = lds128(sk + (trow + 8) * 128 + (((2 * c4) ^ trow) << 4));
    const uint4 kb1 = lds128(sk + (trow + 8) * 128 + (((2 * c4 + 1) ^ trow) << 4));
#pragma unroll
    for (int c = 0; c < C::NKC; ++c) {
      const uint32_t wa = word_of(c < 4 ? ka0 : ka1, c & 3), wb = word_of(c < 4 ? kb0 : kb1, c & 3);
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_f16x2x2(wa, a0, a2);
      e4m3x4_to_f16x2x2(wb, a1, a3);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (c & 1) mma_16816<BF16>(sb[nb], a0, a1, a2, a3, qf[nb][c][0], qf[nb][c][1]);
        else mma_16816<BF16>(sa[nb], a0, a1, a2, a3, qf[nb][c][0], qf[nb][c][1]);
      }
    }
  } else {
#pragma unroll
    for (int c = 0; c < C::NKC; ++c) {
      const int chunk = 2 * (c & 3) + k_add;
      const uint32_t addr = sk + (c >> 2) * (TILE * 128) + k_row * 128 + ((chunk ^ r8) << 4);
      uint32_t a0, a1, a2, a3;
      ldmatrix_x4(addr, a0, a1, a2, a3);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (c & 1) mma_16816<BF16>(sb[nb], a0, a1, a2, a3, qf[nb][c][0], qf[nb][c][1]);
        else mma_16816<BF16>(sa[nb], a0, a1, a2, a3, qf[nb][c][0], qf[nb][c][1]);
      }
    }
  }
  float sc[NB][4];  // scores (base-2 logits): c0, c1 token trow, heads h0, h0 + 1; c2, c3 token trow + 8
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int r = 0; r < 4; ++r) sc[nb][r] = (sa[nb][r] + sb[nb][r]) * scale_log2;
  const int valid = z & 0xff;
  if constexpr (WIN) {
    const int hid0 = (z >> 16) & 31, hid1 = (z >> 24) & 31;  // rows the window hides
    if (valid < TILE || hid0 < hid1) {
      auto hidden = [&](int r) { return r >= valid || (r >= hid0 && r < hid1); };
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        if (hidden(trow)) sc[nb][0] = sc[nb][1] = -INFINITY;
        if (hidden(trow + 8)) sc[nb][2] = sc[nb][3] = -INFINITY;
      }
      // zero the hidden V rows so that 0 * (whatever lies there) cannot make NaN
      uint8_t* vrows = stage + C::KV_TILE_BYTES;
      for (int k = lane; k < TILE * 8 * C::NBOX; k += 32)
        if (hidden(k / 8 % TILE))
          *reinterpret_cast<int4*>(vrows + k / (8 * TILE) * (TILE * 128) + k / 8 % TILE * 128 + k % 8 * 16) =
              make_int4(0, 0, 0, 0);
      __syncwarp();
    }
  } else if (valid < TILE) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      if (trow >= valid) sc[nb][0] = sc[nb][1] = -INFINITY;
      if (trow + 8 >= valid) sc[nb][2] = sc[nb][3] = -INFINITY;
    }
    // zero the V rows past the end so that 0 * (stale value) cannot make NaN
    uint8_t* vrows = stage + C::KV_TILE_BYTES;
    for (int k = lane; k < (TILE - valid) * 8 * C::NBOX; k += 32) {
      const int b = k / ((TILE - valid) * 8);
      const int rem = k - b * (TILE - valid) * 8;
      const int r = valid + rem / 8, c16 = rem & 7;
      *reinterpret_cast<int4*>(vrows + b * (TILE * 128) + r * 128 + c16 * 16) = make_int4(0, 0, 0, 0);
    }
    __syncwarp();
  }

  // ---- online softmax over this tile (per head: columns h0, h0 + 1 of each block)
  uint32_t pb[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    float x0 = fmaxf(sc[nb][0], sc[nb][2]), x1 = fmaxf(sc[nb][1], sc[nb][3]);
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
    }
    const float n0 = fmaxf(m[nb][0], x0), n1 = fmaxf(m[nb][1], x1);
    const float c0 = exp2f(m[nb][0] - n0), c1 = exp2f(m[nb][1] - n1);
    m[nb][0] = n0;
    m[nb][1] = n1;
    const float p0 = exp2f(sc[nb][0] - n0), p2 = exp2f(sc[nb][2] - n0);
    const float p1 = exp2f(sc[nb][1] - n1), p3 = exp2f(sc[nb][3] - n1);
    l[nb][0] = l[nb][0] * c0 + (p0 + p2);
    l[nb][1] = l[nb][1] * c1 + (p1 + p3);
#pragma unroll
    for (int c = 0; c < C::NKC; ++c) {
      o[nb][c][0] *= c0;
      o[nb][c][1] *= c1;
      o[nb][c][2] *= c0;
      o[nb][c][3] *= c1;
    }
    // P^T (16 tokens x 8 heads) from the accumulator layout into the B-operand layout
    pb[nb][0] = movmatrix_trans(pack2<TM>(p0, p1));
    pb[nb][1] = movmatrix_trans(pack2<TM>(p2, p3));
  }

  // ---- O^T += V^T P^T  (d_head x 8 heads per block)
  if constexpr (F8) {
    // token rows 2c4, 2c4 + 1, 2c4 + 8, 2c4 + 9, bytes 16 trow .. 16 trow + 15 of each (chunk trow;
    // swizzle XOR = row & 7); step c takes d = 16 trow + 2c (A rows trow) and + 1 (rows trow + 8)
    const int r0 = 2 * c4;
    const uint4 v0 = lds128(sv + r0 * 128 + ((trow ^ r0) << 4));
    const uint4 v1 = lds128(sv + (r0 + 1) * 128 + ((trow ^ (r0 + 1)) << 4));
    const uint4 v2 = lds128(sv + (r0 + 8) * 128 + ((trow ^ r0) << 4));
    const uint4 v3 = lds128(sv + (r0 + 9) * 128 + ((trow ^ (r0 + 1)) << 4));
#pragma unroll
    for (int c = 0; c < C::NKC; ++c) {
      // bytes 2c, 2c + 1 of the 16: word c / 2, byte 2 (c & 1); interleave tokens (2c4, 2c4 + 1)
      const unsigned sel = (c & 1) ? 0x7362u : 0x5140u;
      const uint32_t x = __byte_perm(word_of(v0, c >> 1), word_of(v1, c >> 1), sel);
      const uint32_t y = __byte_perm(word_of(v2, c >> 1), word_of(v3, c >> 1), sel);
      uint32_t a0, a1, a2, a3;
      e4m3x4_to_f16x2x2(x, a0, a1);
      e4m3x4_to_f16x2x2(y, a2, a3);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_16816<BF16>(o[nb][c], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < C::NKC; ++c) {
      const int chunk = 2 * (c & 3) + v_add;
      const uint32_t addr = sv + (c >> 2) * (TILE * 128) + v_row * 128 + ((chunk ^ r8) << 4);
      uint32_t a0, a1, a2, a3;
      ldmatrix_x4_trans(addr, a0, a1, a2, a3);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) mma_16816<BF16>(o[nb][c], a0, a1, a2, a3, pb[nb][0], pb[nb][1]);
    }
  }
}

}  // namespace pkv
