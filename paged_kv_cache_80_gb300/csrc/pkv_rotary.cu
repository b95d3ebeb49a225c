// Append with the position rotation applied on the way: the new tokens' queries and keys are
// rotated by their positions, keys and values written at their slots of the paged pool, in one
// pass ("PagedAttention", programmer.ie Inference ch. 14, "The real cache": each new key and
// value is written at its block and offset; the rotation of the pair (x1, x2) of frequency i by
// the angle w = p * inv_freq[i] is the product (x1 + i x2) e^{i w}).
//
// The angle.  A 32-bit product p * inv_freq is off by up to p * 2^-24, a whole radian at far
// positions, and 64-bit floating point is slow on this machine, so the angle is kept in turns as a
// 64-bit fixed-point fraction: u = 2^64 frac(inv_freq / 2 pi), made once per frequency and CTA in
// double, and p * u mod 2^64, whose wrap-around is the reduction of the angle, exactly.  The error
// is that of u, at most 2^-53 * inv_freq / 2 pi + 2^-64 turns a position: below 2^-24 turns over all
// int32 positions for inv_freq <= 1.  sincospif of the phase's upper 32 bits follows.
// The rotation is done in 32 bits and rounded once, to the activation type (q), the pool's type
// (k), or the E4M3 code nearest to the 32-bit quotient by the pool's scale.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include "pkv_attn.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

namespace {

struct RotaryArgs {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  void* k_pool;
  void* v_pool;
  const float* inv_freq;
  const int32_t* positions;  // [n_axes][n_tok]
  const int32_t* slots;
  int* err;
  int64_t q_stride, k_stride, v_stride, q_out_stride;  // elements between tokens
  int64_t n_slots;
  int32_t n_tok, H_q, H_kv, d, B, L, layer, rot;
  float k_scale, v_scale;
  uint8_t axis[128];
};

// 2^64 frac(f / 2 pi)
__device__ __forceinline__ unsigned long long turns_of(float f) {
  double r = static_cast<double>(f) * 0.15915494309189535;
  r -= floor(r);
  return __double2ull_rz(r * 18446744073709551616.0);
}

// (cos, sin) of the angle p * f, u = turns_of(f)
__device__ __forceinline__ float2 cos_sin(unsigned long long u, int32_t p) {
  const unsigned long long phase = u * static_cast<unsigned long long>(static_cast<long long>(p));
  const float half_turns = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float2 r;
  sincospif(half_turns, &r.y, &r.x);
  return r;
}

__device__ __forceinline__ uint8_t e4m3_of(float x, float scale) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(x, scale), __NV_SATFINITE, __NV_E4M3);
}

// Any even rotary_dim, head size and alignment: one thread per pair of elements of a (token, row);
// the rows of a token are its H_q query, H_kv key and H_kv value heads.
template <typename TA, bool F8, bool INTER>
__global__ void __launch_bounds__(256) rotary_append_any_kernel(const __grid_constant__ RotaryArgs a) {
  using TS = typename std::conditional<F8, uint8_t, TA>::type;
  __shared__ unsigned long long turns[128];
  const int half = a.rot / 2, pairs = a.d / 2, rows = a.H_q + 2 * a.H_kv;
  for (int i = threadIdx.x; i < half; i += blockDim.x) turns[i] = turns_of(a.inv_freq[i]);
  __syncthreads();
  const int64_t total = static_cast<int64_t>(a.n_tok) * rows * pairs;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t idx = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; idx < total; idx += stride) {
    const int64_t r = idx / pairs;
    const int i = static_cast<int>(idx - r * pairs);
    const int64_t t = r / rows;
    const int row = static_cast<int>(r - t * rows);
    const bool is_q = row < a.H_q, is_k = !is_q && row < a.H_q + a.H_kv;
    if (is_q && !a.q) continue;
    const int h = is_q ? row : (is_k ? row - a.H_q : row - a.H_q - a.H_kv);
    const bool turned = (is_q || is_k) && i < half;
    const int e1 = turned && !INTER ? i : 2 * i, e2 = turned && !INTER ? i + half : 2 * i + 1;
    const TA* src = is_q   ? static_cast<const TA*>(a.q) + t * a.q_stride
                    : is_k ? static_cast<const TA*>(a.k) + t * a.k_stride
                           : static_cast<const TA*>(a.v) + t * a.v_stride;
    src += static_cast<int64_t>(h) * a.d;
    float x1 = to_f(src[e1]), x2 = to_f(src[e2]);
    if (turned) {
      const float2 cs = cos_sin(turns[i], a.positions[static_cast<int64_t>(a.axis[i]) * a.n_tok + t]);
      const float y1 = x1 * cs.x - x2 * cs.y;
      x2 = x2 * cs.x + x1 * cs.y;
      x1 = y1;
    }
    if (is_q) {
      TA* dst = static_cast<TA*>(a.q_out) + t * a.q_out_stride + static_cast<int64_t>(h) * a.d;
      dst[e1] = f_to<TA>(x1);
      dst[e2] = f_to<TA>(x2);
      continue;
    }
    const int32_t slot = a.slots[t];
    if (slot < 0 || slot >= a.n_slots) {
      if (i == 0 && is_k && h == 0) record_error(a.err, DERR_APPEND_SLOT, slot);
      continue;
    }
    const int64_t blk = slot / a.B, off = slot - blk * a.B;
    TS* dst = static_cast<TS*>(is_k ? a.k_pool : a.v_pool) +
              (((blk * a.L + a.layer) * a.H_kv + h) * a.B + off) * a.d;
    if constexpr (F8) {
      const float scale = is_k ? a.k_scale : a.v_scale;
      dst[e1] = e4m3_of(x1, scale);
      dst[e2] = e4m3_of(x2, scale);
    } else {
      dst[e1] = f_to<TA>(x1);
      dst[e2] = f_to<TA>(x2);
    }
  }
}

// Rows made of 16-byte vectors (d_head and rotary_dim multiples of 2 E, E elements a vector; every row and
// pool on a 16-byte boundary).  A thread handles chunk c of a row, two vectors that hold both elements of E
// pairs: elements E c .. and rotary_dim / 2 + E c .. of a rotated head in halves, 2 E c .. (adjacent pairs), or
// 2 E neighbours past rotary_dim; c stays the same for all of a thread's rows.  A CTA takes
// its tokens (or, when there are few, one of `splits` parts of one token's rows): the first rows' vectors are
// on their way while each thread makes the cosines and sines of one frequency, which all H_q + H_kv heads of a
// token share through shared memory, as float4 entries [token][E / 2][chunk] that neighbouring threads read
// without bank conflicts.  A CTA's tokens are a range of its own, taken `tokens` at a time.  The work is the bytes moved: everything else has to hide behind them.
template <typename TA>
struct RowVec {
  static constexpr int E = 16 / sizeof(TA);
  static __device__ __forceinline__ void unpack(const uint4& w, float (&f)[E]) {
    const TA* p = reinterpret_cast<const TA*>(&w);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = to_f(p[e]);
  }
  static __device__ __forceinline__ uint4 pack(const float (&f)[E]) {
    uint4 w;
    if constexpr (E == 4) {
      w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      w = make_uint4(pack2<TA>(f[0], f[1]), pack2<TA>(f[2], f[3]), pack2<TA>(f[4], f[5]), pack2<TA>(f[6], f[7]));
    }
    return w;
  }
};

// eight values to E4M3 codes of x / scale
__device__ __forceinline__ uint2 codes_of(const float (&f)[8], float scale) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e >> 2] |= static_cast<uint32_t>(e4m3_of(f[e], scale)) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}

constexpr int kRotThreads = 256;
constexpr int kRotUnroll = 2;  // rows a thread has in flight
constexpr int kRotCtas = 4;    // resident CTAs an SM the registers have to allow

template <typename TA, bool F8, bool INTER>
__global__ void __launch_bounds__(kRotThreads, kRotCtas) rotary_append_kernel(const __grid_constant__ RotaryArgs a, int tokens,
                                                                     int splits) {
  using RV = RowVec<TA>;
  constexpr int E = RV::E, U = kRotUnroll;
  extern __shared__ float4 cs4[];  // [tokens][E / 2][nch]: (cos, sin) of two frequencies
  const int half = a.rot / 2, nch = half / E, nct = a.d / (2 * E), all_rows = a.H_q + 2 * a.H_kv;
  const int first_row = a.q ? 0 : a.H_q;
  const int per = (all_rows - first_row + splits - 1) / splits;
  const int tid = threadIdx.x;
  const int c = tid % nct, r0 = tid / nct, rpp = kRotThreads / nct;
  const int o0 = c >= nch ? a.rot + 2 * E * (c - nch) : (INTER ? 2 * E * c : E * c);
  const int o1 = c >= nch || INTER ? o0 + E : half + E * c;
  const int fi = tid % half, ft = tid / half, tpp = kRotThreads / half;  // this thread's frequency and first token
  unsigned long long u = 0;
  const int32_t* pos = a.positions + static_cast<int64_t>(a.axis[fi]) * a.n_tok;
  float2* cs_out = reinterpret_cast<float2*>(cs4) + (((fi % E) / 2) * nch + fi / E) * 2 + (fi & 1);
  const int groups = gridDim.x / splits, group = blockIdx.x / splits, sp = blockIdx.x - group * splits;
  const int rb = first_row + sp * per, nr = min(all_rows, rb + per) - rb;  // this split's rows
  const int64_t t_end = static_cast<int64_t>(a.n_tok) * (group + 1) / groups;
  bool first = true;
  for (int64_t t0 = static_cast<int64_t>(a.n_tok) * group / groups; t0 < t_end; t0 += tokens) {
    const int nt = static_cast<int>(min(static_cast<int64_t>(tokens), t_end - t0));
    int t = 0, row = r0;  // the next row to load: token t of the tile, row rb + row
    auto settle = [&] {
      while (row >= nr && t < nt) {
        row -= nr;
        ++t;
      }
    };
    if (r0 >= rpp || nr <= 0) t = nt;
    settle();
    uint4 x0[U], x1[U];
    int xt[U], xr[U], xs[U];
    auto load = [&](int k) {
      xt[k] = t;
      xr[k] = rb + row;
      if (t >= nt) return;
      const int64_t tok = t0 + t;
      const int r = rb + row;
      const TA* src = r < a.H_q ? static_cast<const TA*>(a.q) + tok * a.q_stride + static_cast<int64_t>(r) * a.d
                      : r < a.H_q + a.H_kv
                          ? static_cast<const TA*>(a.k) + tok * a.k_stride + static_cast<int64_t>(r - a.H_q) * a.d
                          : static_cast<const TA*>(a.v) + tok * a.v_stride + static_cast<int64_t>(r - a.H_q - a.H_kv) * a.d;
      x0[k] = *reinterpret_cast<const uint4*>(src + o0);
      x1[k] = *reinterpret_cast<const uint4*>(src + o1);
      if (r >= a.H_q) xs[k] = a.slots[tok];
      row += rpp;
      settle();
    };
#pragma unroll
    for (int k = 0; k < U; ++k) load(k);
    int32_t p = ft < nt ? pos[t0 + ft] : 0;
    if (first) u = turns_of(a.inv_freq[fi]);
    else __syncthreads();  // every thread is done with the last tile's angles
    first = false;
    if (ft < tpp)
      for (int k = ft; k < nt; k += tpp) {
        cs_out[k * half] = cos_sin(u, p);
        if (k + tpp < nt) p = pos[t0 + k + tpp];
      }
    __syncthreads();
    while (xt[0] < nt) {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        if (xt[k] >= nt) break;
        const int64_t tok = t0 + xt[k];
        const int r = xr[k];
        const bool is_v = r >= a.H_q + a.H_kv;
        float f0[E], f1[E];
        RV::unpack(x0[k], f0);
        RV::unpack(x1[k], f1);
        if (c < nch && !is_v) {
          const float4* cs = cs4 + static_cast<int64_t>(xt[k]) * (E / 2) * nch + c;
#pragma unroll
          for (int j = 0; j < E / 2; ++j) {
            const float4 v = cs[j * nch];
            if constexpr (INTER) {  // pairs (2i, 2i + 1): frequencies E c + 2j, + 1 lie in elements 4j .. 4j + 3 of the chunk
              float* f = 4 * j < E ? f0 + 4 * j : f1 + (4 * j - E);
              const float a0 = f[0], a1 = f[1], b0 = f[2], b1 = f[3];
              f[0] = a0 * v.x - a1 * v.y;
              f[1] = a1 * v.x + a0 * v.y;
              f[2] = b0 * v.z - b1 * v.w;
              f[3] = b1 * v.z + b0 * v.w;
            } else {
              const float a0 = f0[2 * j], a1 = f1[2 * j], b0 = f0[2 * j + 1], b1 = f1[2 * j + 1];
              f0[2 * j] = a0 * v.x - a1 * v.y;
              f1[2 * j] = a1 * v.x + a0 * v.y;
              f0[2 * j + 1] = b0 * v.z - b1 * v.w;
              f1[2 * j + 1] = b1 * v.z + b0 * v.w;
            }
          }
        }
        if (r < a.H_q) {
          TA* dst = static_cast<TA*>(a.q_out) + tok * a.q_out_stride + static_cast<int64_t>(r) * a.d;
          *reinterpret_cast<uint4*>(dst + o0) = RV::pack(f0);
          *reinterpret_cast<uint4*>(dst + o1) = RV::pack(f1);
        } else {
          const int32_t slot = xs[k];
          const int h = is_v ? r - a.H_q - a.H_kv : r - a.H_q;
          if (slot < 0 || slot >= a.n_slots) {
            if (c == 0 && h == 0 && !is_v) record_error(a.err, DERR_APPEND_SLOT, slot);
          } else {
            const int64_t blk = slot / a.B, off = slot - blk * a.B;
            const int64_t at = (((blk * a.L + a.layer) * a.H_kv + h) * a.B + off) * a.d;
            void* pool = is_v ? a.v_pool : a.k_pool;
            if constexpr (F8) {
              const float scale = is_v ? a.v_scale : a.k_scale;
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at + o0) = codes_of(f0, scale);
              *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at + o1) = codes_of(f1, scale);
            } else {
              *reinterpret_cast<uint4*>(static_cast<TA*>(pool) + at + o0) = RV::pack(f0);
              *reinterpret_cast<uint4*>(static_cast<TA*>(pool) + at + o1) = RV::pack(f1);
            }
          }
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) load(k);
    }
  }
}

int sm_count() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (!cache[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cache[dev] = n > 0 ? n : 152;
  }
  return cache[dev];
}

// Whether every row is made of whole 16-byte vectors on 16-byte boundaries (the vector kernel's rows).
bool vector_rows(const RotaryArgs& a, int act, int elem) {
  const int E = 16 / act;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out) |
                      reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                      static_cast<uintptr_t>((a.q_stride | a.k_stride | a.v_stride | a.q_out_stride) * act);
  const uintptr_t pools = reinterpret_cast<uintptr_t>(a.k_pool) | reinterpret_cast<uintptr_t>(a.v_pool);
  return a.d % (2 * E) == 0 && a.rot % (2 * E) == 0 && p % 16 == 0 && pools % (E * elem) == 0;
}

template <typename TA, bool F8, bool INTER>
void launch_t(const RotaryArgs& a, cudaStream_t st) {
  constexpr int E = RowVec<TA>::E;
  const int64_t sms = sm_count();
  if (!vector_rows(a, sizeof(TA), F8 ? 1 : sizeof(TA))) {
    const int64_t items = static_cast<int64_t>(a.n_tok) * (a.H_q + 2 * a.H_kv) * (a.d / 2);
    const int grid = static_cast<int>(std::min<int64_t>((items + 255) / 256, sms * 8));
    rotary_append_any_kernel<TA, F8, INTER><<<grid, 256, 0, st>>>(a);
    return;
  }
  // Few tokens: a token's rows over as many CTAs as one resident wave has room for.  Many: tiles of
  // kTokens tokens over a resident grid.
  constexpr int kTokens = 8;
  const int64_t cap = sms * kRotCtas;
  const int rows = (a.q ? a.H_q : 0) + 2 * a.H_kv, rpp = kRotThreads / (a.d / (2 * E));
  const int64_t passes = (rows + rpp - 1) / rpp;
  const int splits = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(passes, cap / a.n_tok)));
  const int groups = static_cast<int>(std::min<int64_t>(a.n_tok, cap / splits));
  const int64_t share = (static_cast<int64_t>(a.n_tok) + groups - 1) / groups;  // a CTA's tokens, in even tiles
  const int64_t rounds = (share + kTokens - 1) / kTokens;
  const int tokens = static_cast<int>((share + rounds - 1) / rounds), grid = groups * splits;
  const size_t smem = static_cast<size_t>(tokens) * a.rot / 2 * sizeof(float2);
  rotary_append_kernel<TA, F8, INTER><<<grid, kRotThreads, smem, st>>>(a, tokens, splits);
}

}  // namespace

int launch_append_rotary(const Pool& P, int32_t layer, const pkv_rotary& rot, const void* q, int64_t q_stride,
                         const void* k_new, int64_t k_stride, const void* v_new, int64_t v_stride,
                         const int32_t* positions, const int32_t* slots, int32_t n_tok, void* q_out,
                         int64_t q_out_stride, void* k_pool, void* v_pool, void* stream) {
  void* err = nullptr;
  if (int rc = device_error_word(&err)) return rc;
  const auto& g = P.geo;
  RotaryArgs a{};
  a.q = q;
  a.k = k_new;
  a.v = v_new;
  a.q_out = q_out;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.inv_freq = rot.inv_freq;
  a.positions = positions;
  a.slots = slots;
  a.err = static_cast<int*>(err);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.n_slots = g.num_blocks * g.block_size;
  a.n_tok = n_tok;
  a.H_q = g.H_q;
  a.H_kv = g.H_kv;
  a.d = g.d_head;
  a.B = g.block_size;
  a.L = g.L;
  a.layer = layer;
  a.rot = rot.rotary_dim;
  a.k_scale = P.k_scale;
  a.v_scale = P.v_scale;
  std::copy(rot.axis, rot.axis + 128, a.axis);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool inter = rot.interleaved != 0;
  switch (g.dtype) {
    case PKV_F32: inter ? launch_t<float, false, true>(a, st) : launch_t<float, false, false>(a, st); break;
    case PKV_F16: inter ? launch_t<__half, false, true>(a, st) : launch_t<__half, false, false>(a, st); break;
    case PKV_BF16: inter ? launch_t<__nv_bfloat16, false, true>(a, st) : launch_t<__nv_bfloat16, false, false>(a, st); break;
    default: inter ? launch_t<__nv_bfloat16, true, true>(a, st) : launch_t<__nv_bfloat16, true, false>(a, st); break;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("rotary append launch: ") + cudaGetErrorString(e));
  count_launch();
  return PKV_OK;
}

}  // namespace pkv
