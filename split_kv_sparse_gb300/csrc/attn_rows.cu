// Attention of packed queries over a paged cache or over packed K and V: one
// warp per (token, query head).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"
#include "softmax_util.cuh"

namespace skv {
namespace {

// 16 consecutive elements as fp32.
template <bool kE4m3>
__device__ __forceinline__ void load16(const void* base, int64_t off, float (&x)[16]) {
  if constexpr (kE4m3) {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + off);
    const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(ws[i >> 1] >> (16 * (i & 1))),
                                                       __NV_E4M3);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
    const uint4 a = p[0], b = p[1];
    const uint32_t ws[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[2 * i] = __uint_as_float(ws[i] << 16);
      x[2 * i + 1] = __uint_as_float(ws[i] & 0xffff0000u);
    }
  }
}

// Lanes 8c .. 8c + 7 take the keys = c mod 4, 16 dims a lane, each group with its
// own running maximum and sum; the four are merged at the end.
template <bool kE4m3>
__global__ void __launch_bounds__(256) attn_rows_kernel(const AttnArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  grid_dependency_wait();
  const int t = static_cast<int>(row / a.h_q), j = static_cast<int>(row - static_cast<int64_t>(t) * a.h_q);
  if (t >= a.total_q || t < a.cu_q[0] || t >= a.cu_q[a.batch]) return;
  int b = 0;
  for (int hi = a.batch; hi - b > 1;) {
    const int mid = (b + hi) >> 1;
    if (a.cu_q[mid] <= t) b = mid;
    else hi = mid;
  }
  int64_t k0 = 0;
  int len;
  if (a.table != nullptr) {
    const int64_t most = static_cast<int64_t>(a.table_width) << a.page_shift;
    len = static_cast<int>(min(static_cast<int64_t>(max(a.kv_lens[b], 0)), most));
  } else {
    k0 = min(max(a.cu_kv[b], 0), a.total_kv);
    len = max(min(a.cu_kv[b + 1], a.total_kv) - static_cast<int>(k0), 0);
  }
  const int seen = min(len - (a.cu_q[b + 1] - t) + 1, len);   // keys this query sees
  const int g = j / a.group;
  const int c = lane >> 3, x0 = (lane & 7) * 16;
  const float dq = a.descale_q ? *a.descale_q : 1.f, dk = a.descale_k ? *a.descale_k : 1.f,
              dv = a.descale_v ? *a.descale_v : 1.f;
  const float sc = dq * dk * a.scale_log2;
  float q[16], o[16];
  load16<kE4m3>(a.q, t * a.q_ts + j * a.q_hs + x0, q);
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  float m = -INFINITY, l = 0.f;
  for (int key0 = 0; key0 < seen; key0 += 4) {
    const int key = key0 + c;
    bool ok = key < seen;
    int64_t at = (k0 + key) * a.kv_rs;
    if (a.table != nullptr && ok) {
      const int page = a.table[static_cast<size_t>(b) * a.table_width + (key >> a.page_shift)];
      ok = page >= 0 && page < a.num_pages;
      at = page * a.kv_ps + (key & ((1 << a.page_shift) - 1)) * a.kv_rs;
    }
    at += g * a.kv_hs + x0;
    float k[16], v[16], s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) k[i] = v[i] = 0.f;
    if (ok) {
      load16<kE4m3>(a.k, at, k);
      load16<kE4m3>(a.v, at, v);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) s = fmaf(q[i], k[i], s);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 4);
    s = ok ? s * sc : -INFINITY;
    const float mn = fmaxf(m, s);
    const float al = m == -INFINITY ? 0.f : exp2f(m - mn);
    const float p = ok ? exp2f(s - mn) : 0.f;
    m = mn;
    l = fmaf(l, al, p);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(o[i], al, p * v[i]);
  }
  float M = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
  M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 16));
  const float w = m == -INFINITY ? 0.f : exp2f(m - M);
  l *= w;
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  l += __shfl_xor_sync(0xffffffffu, l, 16);
  const float inv = M == -INFINITY ? 0.f : dv / l;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    o[i] = m == -INFINITY ? 0.f : o[i] * w;
    o[i] += __shfl_xor_sync(0xffffffffu, o[i], 8);
    o[i] += __shfl_xor_sync(0xffffffffu, o[i], 16);
    o[i] = M == -INFINITY ? 0.f : o[i] * inv;
    amax = fmaxf(amax, fabsf(o[i]));
  }
  const int64_t at = row * 128 + x0;
  if (c == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (a.out_dtype == 0) static_cast<float*>(a.out)[at + i] = o[i];
      else if (a.out_dtype == 1) static_cast<__nv_bfloat16*>(a.out)[at + i] = __float2bfloat16_rn(o[i]);
      else
        static_cast<uint8_t*>(a.out)[at + i] =
            static_cast<uint8_t>(__nv_cvt_float_to_fp8(o[i] * a.inv_scale, __NV_SATFINITE, __NV_E4M3));
    }
  }
  if (lane == 0 && a.lse_out != nullptr) a.lse_out[row] = M == -INFINITY ? -INFINITY : M + log2f(l);
  if (a.amax != nullptr) {
#pragma unroll
    for (int x = 4; x > 0; x >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
    if (lane == 0) atomicMax(reinterpret_cast<int*>(a.amax), __float_as_int(amax));
  }
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, int dtype, cudaStream_t stream) {
  const int64_t blocks = (static_cast<int64_t>(a.total_q) * a.h_q + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  if (dtype == 2) attn_rows_kernel<true><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  else attn_rows_kernel<false><<<static_cast<unsigned>(blocks), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace skv
