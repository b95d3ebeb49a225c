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

template <typename TA, bool F8>
void launch_t(const RotaryArgs& a, bool interleaved, cudaStream_t st) {
  const int64_t items = static_cast<int64_t>(a.n_tok) * (a.H_q + 2 * a.H_kv) * (a.d / 2);
  const int grid = static_cast<int>(std::min<int64_t>((items + 255) / 256, static_cast<int64_t>(sm_count()) * 8));
  if (interleaved) rotary_append_any_kernel<TA, F8, true><<<grid, 256, 0, st>>>(a);
  else rotary_append_any_kernel<TA, F8, false><<<grid, 256, 0, st>>>(a);
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
    case PKV_F32: launch_t<float, false>(a, inter, st); break;
    case PKV_F16: launch_t<__half, false>(a, inter, st); break;
    case PKV_BF16: launch_t<__nv_bfloat16, false>(a, inter, st); break;
    default: launch_t<__nv_bfloat16, true>(a, inter, st); break;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("rotary append launch: ") + cudaGetErrorString(e));
  count_launch();
  return PKV_OK;
}

}  // namespace pkv
