// The paged KV cache's bookkeeping and append: block tables and slot maps from
// request lengths, and the copy (or e4m3 cast) of new K/V rows into their slots.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "attn_common.cuh"

namespace skv {
namespace {

// ------------------------------------------------------------------ the map --
//
// With h_b, p_b the pages a request holds and shall hold, two prefix sums over
// the batch, of max(h_b - p_b, 0) and of max(p_b - h_b, 0), give every freed and
// every wanted page its ordinal, so the free list is pushed and popped without
// atomics and always in request order. One CTA does that part: a step changes
// few pages, so it is latency, not bandwidth, that counts.

constexpr int kMapThreads = 1024;
constexpr int kMapRun = 8;
// Rows whose slots the same CTA writes; more get a grid of their own behind it.
constexpr int kMapFusedRows = 4096;

__device__ __forceinline__ int pages_of(int n, int page_size, int width) {
  const int p = n <= 0 ? 0 : (n - 1) / page_size + 1;
  return p < width ? p : width;
}

// The last i in [0, n) with off[i] <= x, for off[0] = 0 <= x and off non-decreasing.
__device__ __forceinline__ int segment_of(const int* off, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (off[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Exclusive prefix sum of v over the CTA; *total = the sum. `part` holds a word a warp and
// alternates between two places, so one barrier a call is enough.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T (*part)[kMapThreads / 32], int& turn, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  T* p = part[turn];
  turn ^= 1;
  if (lane == 31) p[warp] = x;
  __syncthreads();
  T s = p[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const T before = __shfl_sync(0xffffffffu, s, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : 0) + x - v;
}

__device__ __forceinline__ void slot_of_row(const PagesMapArgs& a, const int32_t* cu, int r) {
  int64_t slot = -1;
  int pos_out = -1;
  if (r < cu[a.batch] && r >= cu[0]) {
    const int b = segment_of(cu, a.batch, r);
    const int pos = a.lens[b] - (cu[b + 1] - r);
    if (pos >= 0 && pos / a.page_size < a.width) {
      pos_out = pos;
      const int page = a.table[static_cast<size_t>(b) * a.width + pos / a.page_size];
      if (page >= 0) slot = static_cast<int64_t>(page) * a.page_size + pos % a.page_size;
    }
  }
  a.slots[r] = slot;
  if (a.positions != nullptr) a.positions[r] = pos_out;
}

__global__ void __launch_bounds__(kMapThreads, 1) pages_map_kernel(const PagesMapArgs a) {
  extern __shared__ int dyn[];
  int* freed = dyn;                   // [batch + 1] exclusive prefix sums
  int* wanted = dyn + a.batch + 1;    // [batch + 1]
  __shared__ uint64_t part[2][kMapThreads / 32];
  int turn = 0;
  grid_dependency_wait();
  const int n0 = min(max(a.free_in[0], 0), a.capacity);
  uint64_t carry = 0;                 // freed pages in the high word, wanted ones in the low
  for (int b0 = 0; b0 < a.batch; b0 += kMapThreads) {
    const int b = b0 + threadIdx.x;
    uint64_t v = 0;
    if (b < a.batch) {
      const int h = pages_of(a.held[b], a.page_size, a.width), p = pages_of(a.lens[b], a.page_size, a.width);
      v = (static_cast<uint64_t>(max(h - p, 0)) << 32) | static_cast<uint64_t>(max(p - h, 0));
    }
    uint64_t total;
    const uint64_t x = carry + block_scan(v, part, turn, &total);
    if (b < a.batch) {
      freed[b] = static_cast<int>(x >> 32);
      wanted[b] = static_cast<int>(x & 0xffffffffu);
    }
    carry += total;
  }
  const int all_freed = static_cast<int>(carry >> 32), all_wanted = static_cast<int>(carry & 0xffffffffu);
  __syncthreads();

  // push: the freed entries in order, without those that hold no page; kMapRun consecutive ones a thread, all loads
  // in flight at once
  int n = n0;
  for (int i0 = 0; i0 < all_freed; i0 += kMapThreads * kMapRun) {
    const int first = i0 + threadIdx.x * kMapRun;
    int page[kMapRun], held = 0;
    int b = first < all_freed ? segment_of(freed, a.batch, first) : 0;
#pragma unroll
    for (int k = 0; k < kMapRun; ++k) {
      const int i = first + k;
      page[k] = -1;
      if (i < all_freed) {
        while (b + 1 < a.batch && freed[b + 1] <= i) ++b;
        page[k] = a.table[static_cast<size_t>(b) * a.width + pages_of(a.lens[b], a.page_size, a.width) + (i - freed[b])];
      }
    }
#pragma unroll
    for (int k = 0; k < kMapRun; ++k) held += page[k] >= 0 ? 1 : 0;
    uint64_t t;
    int at = n + static_cast<int>(block_scan(static_cast<uint64_t>(held), part, turn, &t));
#pragma unroll
    for (int k = 0; k < kMapRun; ++k)
      if (page[k] >= 0) {
        if (at < a.capacity) a.free_pages[at] = page[k];
        ++at;
      }
    n += static_cast<int>(t);
  }
  n = min(n, a.capacity);
  __syncthreads();   // the pushed pages are read below

  // pop
  for (int j0 = threadIdx.x; j0 < all_wanted; j0 += kMapThreads * 4) {
    int page[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + k * kMapThreads;
      page[k] = j < all_wanted && j < n ? a.free_pages[n - 1 - j] : -1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int j = j0 + k * kMapThreads;
      if (j >= all_wanted) break;
      const int b = segment_of(wanted, a.batch, j);
      a.table[static_cast<size_t>(b) * a.width + pages_of(a.held[b], a.page_size, a.width) + (j - wanted[b])] = page[k];
    }
  }
  if (threadIdx.x == 0) {
    a.free_out[0] = max(n - all_wanted, 0);
    a.free_out[1] = max(all_wanted - n, 0);
  }
  if (a.total_q <= kMapFusedRows) {
    __syncthreads();   // the table entries written above
    for (int r = threadIdx.x; r < a.total_q; r += blockDim.x) slot_of_row(a, a.cu_q, r);
  }
}

__global__ void __launch_bounds__(256) pages_slots_kernel(const PagesMapArgs a) {
  grid_dependency_wait();
  const int r = blockIdx.x * 256 + threadIdx.x;
  if (r < a.total_q) slot_of_row(a, a.cu_q, r);
}

// --------------------------------------------------------------- the append --

__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t bf16x2, float descale) {
  const float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&bf16x2));
  return __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(x.x, descale), __fdiv_rn(x.y, descale)), __NV_SATFINITE,
                                  __NV_E4M3);
}

// One thread takes 16 consecutive elements of a K row and the same of the V row.
template <bool kE4m3>
__global__ void __launch_bounds__(256) pages_write_kernel(const PagesWriteArgs a) {
  grid_dependency_wait();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int per_row = a.h_kv * 8;
  const int64_t r = i / per_row;
  if (r >= a.rows) return;
  const int c = static_cast<int>(i - r * per_row);
  const int g = c >> 3, x = (c & 7) * 16;
  const int64_t slot = a.slots[r];
  if (slot < 0 || slot >= a.num_slots) return;
  const int64_t src = r * a.token_stride + g * a.head_stride + x;
  const int64_t page = slot >> a.page_shift, row = slot & ((int64_t{1} << a.page_shift) - 1);
  const int64_t dst = page * a.page_stride + row * a.row_stride + g * a.cache_head_stride + x;
  const uint4* ks = reinterpret_cast<const uint4*>(a.k_new + src);
  const uint4* vs = reinterpret_cast<const uint4*>(a.v_new + src);
  const uint4 k0 = ks[0], k1 = ks[1], v0 = vs[0], v1 = vs[1];
  if constexpr (kE4m3) {
    const float dk = a.descale_k ? *a.descale_k : 1.f, dv = a.descale_v ? *a.descale_v : 1.f;
    auto pack = [](uint32_t lo, uint32_t hi, float d) { return e4m3x2_of(lo, d) | (e4m3x2_of(hi, d) << 16); };
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.k) + dst) =
        make_uint4(pack(k0.x, k0.y, dk), pack(k0.z, k0.w, dk), pack(k1.x, k1.y, dk), pack(k1.z, k1.w, dk));
    *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.v) + dst) =
        make_uint4(pack(v0.x, v0.y, dv), pack(v0.z, v0.w, dv), pack(v1.x, v1.y, dv), pack(v1.z, v1.w, dv));
  } else {
    uint4* kd = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.k) + dst);
    uint4* vd = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.v) + dst);
    kd[0] = k0;
    kd[1] = k1;
    vd[0] = v0;
    vd[1] = v1;
  }
}

constexpr int kMapMaxBatch = 16384;

}  // namespace

cudaError_t launch_pages_map(const PagesMapArgs& a, cudaStream_t stream) {
  const size_t smem = 2 * (static_cast<size_t>(a.batch) + 1) * sizeof(int);
  const cudaError_t e = launch_pdl(pages_map_kernel, 1, kMapThreads, smem, stream, a);
  if (e != cudaSuccess || a.total_q <= kMapFusedRows) return e;
  return launch_pdl(pages_slots_kernel, (a.total_q + 255u) / 256u, 256, 0, stream, a);
}

cudaError_t launch_pages_write(const PagesWriteArgs& a, int dtype, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int64_t blocks = (a.rows * a.h_kv * 8 + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(dtype == 2 ? pages_write_kernel<true> : pages_write_kernel<false>,
                          static_cast<unsigned>(blocks), 256, 0, stream, a);
}

cudaError_t prepare_paged_kernels() {
  return cudaFuncSetAttribute(pages_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              2 * (kMapMaxBatch + 1) * static_cast<int>(sizeof(int)));
}

}  // namespace skv
