// The paged KV cache's bookkeeping and append: block tables and slot maps from
// request lengths, and the copy (or e4m3 cast) of new K/V rows into their slots.
#include <cuda_bf16.h>

#include <algorithm>

#include "attn_common.cuh"
#include "quant.cuh"

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

__device__ __forceinline__ uint2 e4m3x8_of(const uint4& x, const Divider& by) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x0 = __uint_as_float(w[i] << 16), x1 = __uint_as_float(w[i] & 0xffff0000u);
    most = fmax3(most, fabsf(__fmul_rn(x0, by.y)), fabsf(__fmul_rn(x1, by.y)));
    c[i] = e4m3x2(quotient(x0, by.d, by.y), quotient(x1, by.d, by.y));
  }
  if (by.plain || most > 1e30f) {
#pragma unroll 1
    for (int i = 0; i < 4; ++i) {
      const uint32_t v = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
      const uint32_t code = e4m3x2(__fdiv_rn(__uint_as_float(v << 16), by.d), __fdiv_rn(__uint_as_float(v & 0xffff0000u), by.d));
      c[0] = i == 0 ? code : c[0];
      c[1] = i == 1 ? code : c[1];
      c[2] = i == 2 ? code : c[2];
      c[3] = i == 3 ? code : c[3];
    }
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// One warp takes a row's h_kv x 128 elements of K or of V, in pieces that give 16 bytes
// of cache (8 elements, or 16 that become codes), several of a lane's loads in flight at
// once, the slot's among them. HBM bounds the copy (16,001 rows of 8 heads into bf16, 131 MB: 21.2 us). Into e4m3, 98 MB,
// they take 20.1 us, 0.72 of the copy rate: a warp's one burst of loads is followed by its conversions.
template <bool kE4m3>
__global__ void __launch_bounds__(256) pages_write_kernel(const PagesWriteArgs a) {
  constexpr int kFlight = kE4m3 ? 2 : 4;
  constexpr int kLoads = kE4m3 ? 2 : 1;          // 16-byte loads a piece
  constexpr int kPieces = kE4m3 ? 8 : 16;        // pieces a head
  const int lane = threadIdx.x & 31;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t r = w >> 1;
  const bool is_v = w & 1;
  grid_dependency_wait();
  if (r >= a.rows) return;
  const int64_t slot = a.slots[r];
  const float* descale = is_v ? a.descale_v : a.descale_k;
  const Divider by = divider(kE4m3 && descale ? *descale : 1.f);
  const uint16_t* src = (is_v ? a.v_new : a.k_new) + r * a.token_stride;
  const int64_t page = slot >> a.page_shift, row = slot & ((int64_t{1} << a.page_shift) - 1);
  const int64_t to = page * a.page_stride + row * a.row_stride;
  const bool keep = slot >= 0 && slot < a.num_slots;
  const int n = a.h_kv * kPieces;
  for (int c0 = lane; c0 < n; c0 += 32 * kFlight) {
    uint4 x[kFlight][kLoads];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int c = c0 + 32 * k;
      if (c < n) {
        const uint4* from = reinterpret_cast<const uint4*>(src + (c / kPieces) * a.head_stride + (c % kPieces) * 8 * kLoads);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) x[k][i] = __ldg(from + i);
      }
    }
    if (!keep) continue;
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int c = c0 + 32 * k;
      if (c < n) {
        const int64_t dst = to + (c / kPieces) * a.cache_head_stride + (c % kPieces) * 8 * kLoads;
        if constexpr (kE4m3) {
          const uint2 lo = e4m3x8_of(x[k][0], by), hi = e4m3x8_of(x[k][kLoads - 1], by);
          *reinterpret_cast<uint4*>(static_cast<uint8_t*>(is_v ? a.v : a.k) + dst) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(is_v ? a.v : a.k) + dst) = x[k][0];
        }
      }
    }
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
  const int64_t blocks = (2 * a.rows + 7) / 8;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(dtype == 2 ? pages_write_kernel<true> : pages_write_kernel<false>,
                          static_cast<unsigned>(blocks), 256, 0, stream, a);
}

cudaError_t prepare_paged_kernels() {
  return cudaFuncSetAttribute(pages_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              2 * (kMapMaxBatch + 1) * static_cast<int>(sizeof(int)));
}

}  // namespace skv
