// Windowed decode attention for small batches: one cluster of CTAs per (sequence, KV head) pair.
//
// What it computes: for sequence s of length n and query head h (KV head g = floor(h / G)),
//   out[s][h] = sum_t softmax_t(scale * q[s][h] . K_s[t]) V_s[t]  over t < n_sink or n - window <= t < n.
//
// What bounds it: with few pairs there is little to read (a window of 1,024 keys of one sequence with
// 8 KV heads is 4 MB, 0.6 us of the memory's time), so the time is the chain of dependent steps:
// length, table entry, K/V tile, scores, merge.  The pair's tiles are cut over all warps of a cluster
// of up to 8 CTAs, whose partial (m, l, O) meet in shared memory, read across the cluster: two cluster
// barriers, against the global stores, fences, counters and loads with which the persistent
// kernel (pkv_decode.cu) joins a pair that is split over its grid, and no workspace.  Every warp loads up
// to S tiles at once, so the chain holds one memory latency for tiles.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <string>

#include "pkv_attn.cuh"
#include "pkv_device.cuh"
#include "pkv_internal.h"
#include "pkv_tile.cuh"

namespace pkv {

namespace {

constexpr int WD_WARPS = 8;
constexpr int WD_WARP_KB = 16;  // tiles a warp has in flight, in bytes: 8 warps' worth fill one CTA an SM

template <int D, int EB, int NB>
struct WdCfg {
  using C = TcCfg<D, EB, NB>;
  static constexpr int STAGE = 2 * C::KV_TILE_BYTES;  // K tile, V tile
  static constexpr int S = WD_WARP_KB * 1024 / STAGE;
  static constexpr int WARP_BYTES = S * STAGE + 64 * 16 + S * 8;
  static constexpr int WARP_STRIDE = (WARP_BYTES + 1023) / 1024 * 1024;
  static constexpr int PART = NB * C::OFL + 2 * C::GP;  // floats of a partial: O^T fragments, m, l
  static constexpr int CTA_PART = WD_WARPS * WARP_STRIDE;  // the CTA's own partial, behind its warps' rooms
  static constexpr int SMEM = CTA_PART + PART * 4 + 1024;
  static_assert(PART * 4 <= S * STAGE, "a warp's partial takes its stages' room");
};

__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
// Every thread of the cluster: its earlier writes to shared memory are seen by all after the wait.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Unit u = (head block, d-chunk) of n partials: a lane's O^T fragment, relative to 2^m, and the (m, l) of its
// two heads.  at(i): shared address of partial i (of this CTA or a peer), 0 for one that holds nothing.
struct Merged {
  float4 o;
  float m0, m1, l0, l1;
};
template <int NB, typename C, typename At>
__device__ __forceinline__ Merged merge_unit(int n, int u, int lane, const At& at) {
  constexpr int U = 8;  // partials in flight
  const int nb = u / C::NKC, c = u - nb * C::NKC, h = GPAD * nb + 2 * (lane & 3);
  Merged r{make_float4(0.f, 0.f, 0.f, 0.f), -INFINITY, -INFINITY, 0.f, 0.f};
  for (int i0 = 0; i0 < n; i0 += U) {
    float2 pm[U], pl[U];
    float4 po[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const uint32_t p = i0 + k < n ? at(i0 + k) : 0u;
      pm[k] = make_float2(-INFINITY, -INFINITY);
      pl[k] = make_float2(0.f, 0.f);
      po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p) {
        pm[k] = ld_peer2(p + 4 * (NB * C::OFL + h));
        pl[k] = ld_peer2(p + 4 * (NB * C::OFL + C::GP + h));
        po[k] = ld_peer4(p + 4 * nb * C::OFL + 16 * (c * 32 + lane));
      }
    }
    float n0 = r.m0, n1 = r.m1;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      n0 = fmaxf(n0, pm[k].x);
      n1 = fmaxf(n1, pm[k].y);
    }
    // -inf: nothing seen yet (0 stands in for a maximum that is not there)
    const float s0 = n0 == -INFINITY ? 0.f : n0, s1 = n1 == -INFINITY ? 0.f : n1;
    const float r0 = exp2f(r.m0 - s0), r1 = exp2f(r.m1 - s1);
    r.l0 *= r0;
    r.l1 *= r1;
    r.o = make_float4(r.o.x * r0, r.o.y * r1, r.o.z * r0, r.o.w * r1);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float e0 = exp2f(pm[k].x - s0), e1 = exp2f(pm[k].y - s1);
      r.l0 += pl[k].x * e0;
      r.l1 += pl[k].y * e1;
      r.o.x += po[k].x * e0;
      r.o.y += po[k].y * e1;
      r.o.z += po[k].z * e0;
      r.o.w += po[k].w * e1;
    }
    r.m0 = n0;
    r.m1 = n1;
  }
  return r;
}

// O^T fragment of chunk c: 16-bit pools hold d = 16c + trow (x, y) and + 8 (z, w), FP8 pools 16 trow + 2c and + 1;
// x, z the lane's first head and y, w its second
template <typename TA, int D, bool F8, int NB>
__device__ __forceinline__ void store_unit(const DecodeArgs& a, TA* out, int u, const Merged& r, int lane) {
  constexpr int NKC = D / 16;
  const int nb = u / NKC, c = u - nb * NKC, h = GPAD * nb + 2 * (lane & 3), trow = lane >> 2;
  const int da = F8 ? 16 * trow + 2 * c : 16 * c + trow, db = F8 ? da + 1 : da + 8;
  const float i0 = a.v_mul / r.l0, i1 = a.v_mul / r.l1;
  TA* oh = out + static_cast<int64_t>(h) * D;
  if (h < a.G) {
    oh[da] = from_float<TA>(r.o.x * i0);
    oh[db] = from_float<TA>(r.o.z * i0);
  }
  if (h + 1 < a.G) {
    oh[D + da] = from_float<TA>(r.o.y * i1);
    oh[D + db] = from_float<TA>(r.o.w * i1);
  }
}

template <typename T, int D, int NB>
__global__ void __launch_bounds__(WD_WARPS * 32) decode_win_kernel(const __grid_constant__ CUtensorMap tmk,
                                                                   const __grid_constant__ CUtensorMap tmv,
                                                                   const DecodeArgs a, int csize) {
  constexpr bool F8 = std::is_same<T, E4M3>::value;
  using TA = typename std::conditional<F8, __nv_bfloat16, T>::type;
  constexpr int EB = F8 ? 1 : 2, NW = WD_WARPS;
  using C = TcCfg<D, EB, NB>;
  using W = WdCfg<D, EB, NB>;
  constexpr int S = W::S;
  extern __shared__ uint8_t smem_raw[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pair = blockIdx.x / csize, rank = blockIdx.x - pair * csize;
  const int s = pair / a.H_kv, g = pair - s * a.H_kv;
  const int c4 = lane & 3, trow = lane >> 2, h0 = 2 * c4;

  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* region = base + warp * W::WARP_STRIDE;
  int4* desc = reinterpret_cast<int4*>(region + S * W::STAGE);
  const uint32_t bar0 = smem_u32(region + S * W::STAGE + 64 * 16);
  const uint32_t stage0 = smem_u32(region);

  const WinTiles wt = win_tiles(a, s, g == 0 && rank == 0 && threadIdx.x == 0);
  TA* out = static_cast<TA*>(a.out) + (static_cast<int64_t>(s) * a.H_q + g * a.G) * D;
  if (wt.n == 0) {  // an empty sequence attends to nothing: zero output (the whole cluster leaves)
    if (rank == 0)
      for (int k = threadIdx.x; k < a.G * D / 8; k += NW * 32) reinterpret_cast<uint4*>(out)[k] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int total = csize * NW;
  auto first_tile = [&](int i) { return static_cast<int>(static_cast<int64_t>(wt.n) * i / total); };  // of warp i
  const int me = rank * NW + warp, t0 = first_tile(me), n_my = first_tile(me + 1) - t0;

  // tiles [k, k + 32) of this warp: their row in the pool, valid and hidden rows
  auto fill = [&](int k) {
    const int t = k + lane;
    if (t < n_my) {
      const int tok0 = wt.token0(t0 + t), lb = tok0 / a.B;
      int blk = a.tables[static_cast<int64_t>(s) * a.W + lb];
      if (blk < 0 || blk >= a.num_blocks) {
        record_error(a.err, DERR_DECODE_BLOCK, blk);
        blk = 0;
      }
      const int z = min(TILE, wt.len - tok0) | max(0, min(TILE, wt.ns - tok0)) << 16 | max(0, min(TILE, wt.lo - tok0)) << 24;
      desc[t & 63] = make_int4(((blk * a.L + a.layer) * a.H_kv + g) * a.B + tok0 - lb * a.B, z, 0, 0);
    }
    __syncwarp();
  };
  auto issue = [&](int t) {  // lane 0 only
    const int row = desc[t & 63].x;
    const uint32_t bar = bar0 + 8 * (t % S), sk = stage0 + (t % S) * W::STAGE, sv = sk + C::KV_TILE_BYTES;
    fence_proxy_async();
    mbar_arrive_expect_tx(bar, W::STAGE);
#pragma unroll
    for (int b = 0; b < C::NBOX; ++b) {
      tma_load_2d(sk + b * (TILE * 128), &tmk, b * C::BOX_ELEMS, row, bar);
      tma_load_2d(sv + b * (TILE * 128), &tmv, b * C::BOX_ELEMS, row, bar);
    }
  };
  if (lane == 0) {
    for (int st = 0; st < S; ++st) mbar_init(bar0 + 8 * st, 1);
    fence_barrier_init();
  }
  __syncwarp();
  fill(0);
  if (n_my > 32) fill(32);
  if (lane == 0)
    for (int t = 0; t < S && t < n_my; ++t) issue(t);

  // q fragments straight from memory, while the first tiles are on their way
  uint32_t qf[NB][C::NKC][2];
  float o[NB][C::NKC][4], m[NB][2], l[NB][2];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    m[nb][0] = m[nb][1] = -INFINITY;
    l[nb][0] = l[nb][1] = 0.f;
    const int hq = trow + GPAD * nb;
    const TA* q = static_cast<const TA*>(a.q) + (static_cast<int64_t>(s) * a.H_q + g * a.G + hq) * D;
#pragma unroll
    for (int c = 0; c < C::NKC; ++c) {
      o[nb][c][0] = o[nb][c][1] = o[nb][c][2] = o[nb][c][3] = 0.f;
      qf[nb][c][0] = qf[nb][c][1] = 0u;
      if (hq < a.G) {
        if constexpr (F8) {  // step c of q K^T covers d = 32 c4 + 4c .. + 3
          const uint2 w = *reinterpret_cast<const uint2*>(q + (D / 4) * c4 + 4 * c);
          qf[nb][c][0] = bf16x2_to_f16x2(w.x);
          qf[nb][c][1] = bf16x2_to_f16x2(w.y);
        } else {
          qf[nb][c][0] = *reinterpret_cast<const uint32_t*>(q + 16 * c + h0);
          qf[nb][c][1] = *reinterpret_cast<const uint32_t*>(q + 16 * c + h0 + 8);
        }
      }
    }
  }

  for (int i = 0; i < n_my; ++i) {
    if (i >= 32 && (i & 31) == 0 && i + 32 < n_my) fill(i + 32);
    if (!mbar_wait_bounded(bar0 + 8 * (i % S), (i / S) & 1, kWaitNs)) {
      if (lane == 0) record_error(a.err, DERR_DECODE_TIMEOUT, i);
      for (int k = 1; k < S && i + k < n_my; ++k)  // let the other stages' loads land (bounded) before their room is used
        mbar_wait_bounded(bar0 + 8 * ((i + k) % S), ((i + k) / S) & 1, kWaitNs);
      break;
    }
    attend_tile<T, D, NB, true>(region + (i % S) * W::STAGE, stage0 + (i % S) * W::STAGE, desc[i & 63].y, a.scale_log2,
                                lane, qf, o, m, l);
    __syncwarp();  // every lane is done with this stage
    if (lane == 0 && i + S < n_my) issue(i + S);
  }

  // this warp's partial, over its stages (their loads have all landed and been read)
  __syncwarp();
  if (n_my > 0) {
    float* ps = reinterpret_cast<float*>(region);
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      float L0 = l[nb][0], L1 = l[nb][1];
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        L0 += __shfl_xor_sync(0xffffffffu, L0, off);
        L1 += __shfl_xor_sync(0xffffffffu, L1, off);
      }
#pragma unroll
      for (int c = 0; c < C::NKC; ++c)
        reinterpret_cast<float4*>(ps + nb * C::OFL)[c * 32 + lane] =
            make_float4(o[nb][c][0], o[nb][c][1], o[nb][c][2], o[nb][c][3]);
      if (lane < 4) {
        *reinterpret_cast<float2*>(ps + NB * C::OFL + GPAD * nb + h0) = make_float2(m[nb][0], m[nb][1]);
        *reinterpret_cast<float2*>(ps + NB * C::OFL + C::GP + GPAD * nb + h0) = make_float2(L0, L1);
      }
    }
  }
  // merge ("Chunked prefill mechanics" rule), a (head block, d-chunk) unit of a warp at a time: the CTA's
  // warps first, then the CTAs of the cluster
  const uint32_t base_s = smem_u32(base);
  constexpr int UNITS = NB * C::NKC;
  __syncthreads();
  for (int u = warp; u < UNITS; u += NW) {
    const Merged r = merge_unit<NB, C>(NW, u, lane, [&](int i) -> uint32_t {
      return first_tile(rank * NW + i + 1) > first_tile(rank * NW + i) ? base_s + i * W::WARP_STRIDE : 0u;
    });
    if (csize == 1) {
      store_unit<TA, D, F8, NB>(a, out, u, r, lane);
    } else {
      float* part = reinterpret_cast<float*>(base + W::CTA_PART);
      reinterpret_cast<float4*>(part)[u * 32 + lane] = r.o;
      if (u % C::NKC == 0 && lane < 4) {
        const int h = GPAD * (u / C::NKC) + h0;
        *reinterpret_cast<float2*>(part + NB * C::OFL + h) = make_float2(r.m0, r.m1);
        *reinterpret_cast<float2*>(part + NB * C::OFL + C::GP + h) = make_float2(r.l0, r.l1);
      }
    }
  }
  if (csize == 1) return;
  cluster_sync();
  for (int u = rank + csize * warp; u < UNITS; u += csize * NW) {
    const Merged r =
        merge_unit<NB, C>(csize, u, lane, [&](int i) -> uint32_t { return peer_smem(base_s + W::CTA_PART, i); });
    store_unit<TA, D, F8, NB>(a, out, u, r, lane);
  }
  cluster_sync();  // peers may still read this CTA's partial
}

template <typename T, int D, int NB>
const void* kernel_of(int* smem) {
  *smem = WdCfg<D, std::is_same<T, E4M3>::value ? 1 : 2, NB>::SMEM;
  return reinterpret_cast<const void*>(&decode_win_kernel<T, D, NB>);
}

template <int NB>
const void* pick(const pkv_geometry& g, int* smem) {
  if (g.dtype == PKV_E4M3) return kernel_of<E4M3, 128, NB>(smem);
  const bool bf = g.dtype == PKV_BF16;
  if (g.d_head == 128) return bf ? kernel_of<__nv_bfloat16, 128, NB>(smem) : kernel_of<__half, 128, NB>(smem);
  return bf ? kernel_of<__nv_bfloat16, 64, NB>(smem) : kernel_of<__half, 64, NB>(smem);
}

}  // namespace

// CTAs per pair of the cluster kernel for a batch of `pairs` pairs of at most `tiles` tiles each: a power
// of two, at most 8, doubled while every warp keeps a tile and all CTAs are resident at once (one an
// SM); 0 when the pairs alone are more than that: the persistent kernel's even split of the bytes
// wins there.  Measured (64 q / 8 KV heads, d 128, bf16; cluster against persistent kernel): one
// sequence, 128 keys 5.4 against 12.9 us (1 CTA a pair; 8 CTAs 6.0), 1,024 keys 6.7 against 46 us (8 CTAs; 4
// CTAs 7.8, 1 CTA 10.3), 8,192 keys 12.2 against 70 us; 16 sequences of 4,096 keys 45 against 57 us; 48 of
// 4,096 keys 143 against 131 us.
int win_cluster_size(int64_t pairs, int64_t tiles, int sms) {
  if (pairs > sms) return 0;
  int c = 1;
  while (c < 8 && pairs * c * 2 <= sms && tiles >= 2 * c * WD_WARPS) c *= 2;
  return c;
}

int launch_decode_clusters(const Pool& P, DecodeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv, int csize,
                           cudaStream_t st) {
  int smem = 0;
  const void* k = a.G > GPAD ? pick<2>(P.geo, &smem) : pick<1>(P.geo, &smem);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("cudaFuncSetAttribute: ") + cudaGetErrorString(e));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_seq * a.H_kv * csize));
  cfg.blockDim = dim3(WD_WARPS * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = csize;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {const_cast<CUtensorMap*>(&tk), const_cast<CUtensorMap*>(&tv), &a, &csize};
  e = cudaLaunchKernelExC(&cfg, k, args);
  if (e != cudaSuccess) return fail(PKV_ERR_CUDA, std::string("windowed decode launch: ") + cudaGetErrorString(e));
  count_launch();
  return PKV_OK;
}

}  // namespace pkv
