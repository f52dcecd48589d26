// Rows of the paged cache with arithmetic on the way: the append that rotates by position, the append into 4-bit
// pages, and the way back from pages of any type to bf16 rows.
//
// Both kernels are copies: every byte is read and written once and HBM bounds them, latency a call of few rows. Back-to-back calls of 16,001
// rows of 32 + 2 x 8 heads: into bf16 60 us (6.6 TB/s), q and cache into e4m3 63 (4.8), into 4 bits 69 (5.1; 8,192 rows 40), K and V alone
// 30.5 (2.8): the codes' arithmetic beside the loads. 20,000 rows back: of 4 bits 17.8 (5.9), of e4m3 20.5 (6.0), of bf16 26.4 (6.2).
#include <algorithm>

#include "attn_common.cuh"
#include "quant.cuh"

namespace skv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[2][4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i >> 1][2 * (i & 1)] = __uint_as_float(w[i] << 16);
    x[i >> 1][2 * (i & 1) + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[2][4]) {
  return make_uint4(pack_bf16x2(x[0][0], x[0][1]), pack_bf16x2(x[0][2], x[0][3]), pack_bf16x2(x[1][0], x[1][1]),
                    pack_bf16x2(x[1][2], x[1][3]));
}

// The append: y = x turned by the angles of its row's position (q and k heads), then to q_out, k_out and the cache.
// The products and their sum are rounded to fp32 one by one, so a code follows from plain fp32 arithmetic.
// Eight threads take a head, 16 of its dims each in two pieces of eight: with halves turned against each other
// thread t < R / 16 has the pieces t and t + R / 16, whose dims are pairs; the other threads, and all with neighbours paired, have
// two pieces side by side. A row is chunks of four heads, those of q, then those of k and v; a warp takes `per` of them one after the
// other, the loads of the next two on their way meanwhile, and keeps its angles in shared memory. (Four heads' loads at once,
// unrolled for each kind of output, left 16 warps an SM, each fetching its instructions anew: 8,192 rows into 4 bits 66 us.)
// kTurn: 0 no rotation, 1 halves, 2 neighbours.
template <int kCache, int kTurn, bool kQ8>
__global__ void __launch_bounds__(kThreads, kCache == 1 && !kQ8 ? 4 : 3) pages_append_kernel(const PagesAppendArgs a, const int per) {
  __shared__ float4 angles[kThreads / 32][4][8];
  const int lane = threadIdx.x & 31, t = lane & 7, sub = lane >> 3;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int q_chunks = (a.h_q + 3) >> 2, chunks = q_chunks + ((a.h_kv + 1) >> 1);
  const int parts = (chunks + per - 1) / per;
  const int64_t r = w / parts;
  const int first = static_cast<int>(w - r * parts) * per, last = min(first + per, chunks);
  const bool turning = kTurn != 0 && t < (a.rot >> 4), apart = kTurn == 1 && turning;
  const int p0 = apart ? t : kTurn == 1 ? (a.rot >> 3) + 2 * (t - (a.rot >> 4)) : 2 * t;
  const int p1 = apart ? t + (a.rot >> 4) : p0 + 1;
  grid_dependency_wait();
  if (r >= a.rows) return;
  // (q and k may be written in place, by the thread that has read them: plain loads)
  auto load = [&](int ch, uint4 (&x)[2]) {
    if (ch >= last) return;
    const uint16_t* src = nullptr;
    if (ch < q_chunks) {
      const int h = 4 * ch + sub;
      if (h < a.h_q) src = a.q + r * a.q_ts + h * a.q_hs;
    } else {
      const int i = 4 * (ch - q_chunks) + sub;
      if (i < 2 * a.h_kv) src = (i < a.h_kv ? a.k_new + i * a.head_stride : a.v_new + (i - a.h_kv) * a.head_stride) + r * a.token_stride;
    }
    if (src != nullptr) {
      x[0] = *reinterpret_cast<const uint4*>(src + 8 * p0);
      x[1] = *reinterpret_cast<const uint4*>(src + 8 * p1);
    }
  };
  uint4 ahead[2][2];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    ahead[b][0] = ahead[b][1] = make_uint4(0, 0, 0, 0);
    load(first + b, ahead[b]);
  }
  int64_t pos = 0;
  if (kTurn != 0) pos = a.positions[r];
  const int64_t slot = a.slots[r];
  const float dq = kQ8 && a.descale_q ? *a.descale_q : 1.f, dk = kCache != 1 && a.descale_k ? *a.descale_k : 1.f,
              dv = kCache != 1 && a.descale_v ? *a.descale_v : 1.f;
  if (kTurn != 0 && (pos < 0 || pos >= a.num_positions)) return;   // padding: nothing of the row is written
  float4(&mine)[4][8] = angles[threadIdx.x >> 5];                  // cosines of this thread's first and last four pairs, sines
  if (kTurn != 0 && turning && sub < 2) {
    const float* row = a.cos_sin + pos * a.rot + 8 * t + (sub ? a.rot >> 1 : 0);
    mine[2 * sub][t] = reinterpret_cast<const float4*>(row)[0];
    mine[2 * sub + 1][t] = reinterpret_cast<const float4*>(row)[1];
  }
  __syncwarp();
  auto pair = [](float& u, float& v, float cs, float sn) {
    const float u1 = __fsub_rn(__fmul_rn(u, cs), __fmul_rn(v, sn));
    v = __fadd_rn(__fmul_rn(v, cs), __fmul_rn(u, sn));
    u = u1;
  };
  auto turn = [&](float (&y)[2][2][4]) {                  // [piece][half of it][dim]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 c = mine[h][t], s = mine[2 + h][t];
      if constexpr (kTurn == 2) {
        pair(y[h][0][0], y[h][0][1], c.x, s.x);
        pair(y[h][0][2], y[h][0][3], c.y, s.y);
        pair(y[h][1][0], y[h][1][1], c.z, s.z);
        pair(y[h][1][2], y[h][1][3], c.w, s.w);
      } else {
        pair(y[0][h][0], y[1][h][0], c.x, s.x);
        pair(y[0][h][1], y[1][h][1], c.y, s.y);
        pair(y[0][h][2], y[1][h][2], c.z, s.z);
        pair(y[0][h][3], y[1][h][3], c.w, s.w);
      }
    }
  };
  auto put16 = [&](void* base, int64_t to, const float (&y)[2][2][4]) {
    uint16_t* dst = static_cast<uint16_t*>(base) + to;
    *reinterpret_cast<uint4*>(dst + 8 * p0) = pack8(y[0]);
    *reinterpret_cast<uint4*>(dst + 8 * p1) = pack8(y[1]);
  };
  auto put8 = [&](void* base, int64_t to, float (&y)[2][2][4], const Divider& by) {
    uint8_t* dst = static_cast<uint8_t*>(base) + to;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      divide4(y[e][0], by);
      divide4(y[e][1], by);
      *reinterpret_cast<uint2*>(dst + 8 * (e ? p1 : p0)) = make_uint2(pack_e4m3x4(y[e][0][0], y[e][0][1], y[e][0][2], y[e][0][3]),
                                                                      pack_e4m3x4(y[e][1][0], y[e][1][1], y[e][1][2], y[e][1][3]));
    }
  };
  const bool keep = slot >= 0 && slot < a.num_slots;
  const int64_t page = slot >> a.page_shift, at = slot & ((int64_t{1} << a.page_shift) - 1);
  auto chunk = [&](int ch, uint4 (&x)[2]) {
    float y[2][2][4];
    unpack8(x[0], y[0]);
    unpack8(x[1], y[1]);
    load(ch + 2, x);
    if (ch < q_chunks) {
      if (kTurn != 0 && turning) turn(y);
      const int h = 4 * ch + sub;
      if (h >= a.h_q) return;
      const int64_t to = r * a.qo_ts + h * a.qo_hs;
      if constexpr (kQ8) put8(a.q_out, to, y, divider(dq));
      else put16(a.q_out, to, y);
      return;
    }
    const int i = 4 * (ch - q_chunks) + sub;
    const bool is_k = i < a.h_kv, to_cache = keep && i < 2 * a.h_kv;
    const int g = is_k ? i : i - a.h_kv;
    if (kTurn != 0 && is_k) {
      if (turning) turn(y);
      if (a.k_out != nullptr) put16(a.k_out, r * a.ko_ts + g * a.ko_hs, y);
    }
    const int64_t to = page * a.page_stride + at * a.row_stride + g * a.cache_head_stride;
    void* cache = is_k ? a.k : a.v;
    if constexpr (kCache == 1) {
      if (to_cache) put16(cache, to, y);
    } else if constexpr (kCache == 2) {
      if (to_cache) put8(cache, to, y, divider(is_k ? dk : dv));
    } else {
      // 16 dims with one scale: this thread's pieces, or each with the neighbour's
      const Divider by = divider(is_k ? dk : dv);
      float most[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          divide4(y[e][h], by);
#pragma unroll
          for (int k = 0; k < 4; ++k) most[e] = max_abs_nan(most[e], y[e][h][k]);
        }
      const float other0 = __shfl_xor_sync(0xffffffffu, most[0], 1), other1 = __shfl_xor_sync(0xffffffffu, most[1], 1);
      const float m0 = max_abs_nan(most[0], apart ? other0 : most[1]), m1 = max_abs_nan(most[1], apart ? other1 : most[0]);
      if (!(m0 <= 1e30f) || !(m1 <= 1e30f)) {             // (infinities and NaN; beyond 6 * 448 every code is the largest)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k) y[e][h][k] = fminf(fmaxf(y[e][h][k], -4096.f), 4096.f);
      }
      if (to_cache) {
        const uint32_t s0 = scale_code(m0), s1 = scale_code(m1);
        uint8_t* codes = static_cast<uint8_t*>(cache) + to;
        *reinterpret_cast<uint32_t*>(codes + 4 * p0) = e2m1x8(y[0], e4m3_value(s0));
        *reinterpret_cast<uint32_t*>(codes + 4 * p1) = e2m1x8(y[1], e4m3_value(s1));
        uint8_t* scales = (is_k ? a.k_scales : a.v_scales) + page * a.scale_page_stride + g * a.scale_head_stride + 8 * at;
        if (!apart || !(t & 1)) scales[p0 >> 1] = static_cast<uint8_t>(s0);
        if (apart && !(t & 1)) scales[p1 >> 1] = static_cast<uint8_t>(s1);
      }
    }
  };
#pragma unroll 1
  for (int ch = first; ch < last; ch += 2) {
    chunk(ch, ahead[0]);
    if (ch + 1 < last) chunk(ch + 1, ahead[1]);
  }
}

// The way back: 16 dims a thread, code x scale (exact) x descale in fp32, rounded to bf16 (a bf16 cache's bits as they are).
template <int kCache, int kFlight>
__global__ void __launch_bounds__(kThreads) pages_read_kernel(const PagesAppendArgs a) {
  const int lane = threadIdx.x & 31, p = lane & 7;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int heads = 2 * a.h_kv;
  const int chunks = (heads + 4 * kFlight - 1) / (4 * kFlight);
  const int64_t r = w / chunks;
  const int h0 = static_cast<int>(w - r * chunks) * 4 * kFlight + (lane >> 3);
  grid_dependency_wait();
  if (r >= a.rows) return;
  const int64_t slot = a.slots[r];
  if (slot < 0 || slot >= a.num_slots) return;
  const int64_t page = slot >> a.page_shift, at = slot & ((int64_t{1} << a.page_shift) - 1);
  uint4 x[kFlight][kCache == 1 ? 2 : 1];
  uint32_t scale[kFlight];
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    const int h = h0 + 4 * k;
    if (h >= heads) continue;
    const bool is_k = h < a.h_kv;
    const int g = is_k ? h : h - a.h_kv;
    const void* cache = is_k ? a.k : a.v;
    const int64_t src = page * a.page_stride + at * a.row_stride + g * a.cache_head_stride;
    if constexpr (kCache == 1) {
      const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + src + 16 * p);
      x[k][0] = from[0];
      x[k][1] = from[1];
    } else if constexpr (kCache == 2) {
      x[k][0] = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + src + 16 * p);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + src + 8 * p);
      x[k][0].x = v.x;
      x[k][0].y = v.y;
      scale[k] = (is_k ? a.k_scales : a.v_scales)[page * a.scale_page_stride + g * a.scale_head_stride + 8 * at + p];
    }
  }
  const float dk = a.descale_k ? *a.descale_k : 1.f, dv = a.descale_v ? *a.descale_v : 1.f;
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    const int h = h0 + 4 * k;
    if (h >= heads) continue;
    const bool is_k = h < a.h_kv;
    const int g = is_k ? h : h - a.h_kv;
    uint16_t* dst = (is_k ? a.k_out : a.v_out) + r * a.ko_ts + g * a.ko_hs + 16 * p;
    uint32_t v[8];
    if constexpr (kCache == 1) {
      v[0] = x[k][0].x, v[1] = x[k][0].y, v[2] = x[k][0].z, v[3] = x[k][0].w;
      v[4] = x[k][1].x, v[5] = x[k][1].y, v[6] = x[k][1].z, v[7] = x[k][1].w;
    } else {
      const float d = is_k ? dk : dv;
      uint32_t f[8];                     // pairs in f16 (exact)
      if constexpr (kCache == 2) {
        const uint32_t c[4] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = f16x2_of_e4m3(c[i]);
          f[2 * i + 1] = f16x2_of_e4m3(c[i] >> 16);
        }
      } else {
        const uint32_t both = f16x2_of_e4m3(scale[k] | (scale[k] << 8));
        uint32_t lo[4], hi[4];
        f16_of_e2m1x8(x[k][0].x, lo);
        f16_of_e2m1x8(x[k][0].y, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[i] = mul_f16x2(lo[i], both);
          f[4 + i] = mul_f16x2(hi[i], both);
        }
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
        v[i] = pack_bf16x2(y.x * d, y.y * d);
      }
    }
    st_global_32(dst, v, (reinterpret_cast<uintptr_t>(dst) & 31) == 0);
  }
}

// Warps of an SM that keep HBM busy: where a call has fewer it takes the smallest pieces.
constexpr int64_t kSmWarps = 16;

unsigned blocks_of(int64_t warps) {
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  return blocks > 0x7fffffff ? 0u : static_cast<unsigned>(blocks);
}

template <int kCache>
cudaError_t launch_rows(const PagesAppendArgs& a, bool read, cudaStream_t stream) {
  const int64_t full = kSmWarps * a.num_sms;
  if (read) {
    const bool many = a.rows * 2 * a.h_kv >= 16 * full;
    const int64_t each = many ? 16 : 4;
    const unsigned grid = blocks_of(a.rows * ((2ll * a.h_kv + each - 1) / each));
    if (grid == 0) return cudaErrorInvalidValue;
    return launch_pdl(many ? pages_read_kernel<kCache, 4> : pages_read_kernel<kCache, 1>, grid, kThreads, 0, stream, a);
  }
  const int chunks = (a.h_q + 3) / 4 + (a.h_kv + 1) / 2;
  // A warp's start waits for the position and then the angles: it takes many chunks where the rows fill the SMs, in bf16 at most six
  // (16,001 rows of 32 + 2 x 8 heads in bf16, graphs: 6 chunks 61.0 us, all 12 65.4, 1 122; 8,192 into 4 bits: all 40, 6 48.3, 1 98).
  // A row's warps take even parts, and no more than leaves every SM its warps (parts of six and a rest: bf16, 28 + 2 x 4 heads 49.8
  // us, even 48.6; 40 + 2 x 8 74.9 and 72.4; 20 + 2 x 4 44.1 and 39.8; whole rows in 4 bits: 1,000 of 64 + 2 x 64 heads 33.6, so 28.7).
  int per = 1;
  if (a.rows * chunks >= 12 * full) {
    const int64_t most = std::min<int64_t>(kCache == 1 ? 6 : chunks, a.rows * chunks / full);
    const int64_t parts = (chunks + most - 1) / most;
    per = static_cast<int>((chunks + parts - 1) / parts);
  }
  const unsigned grid = blocks_of(a.rows * ((chunks + per - 1) / per));
  if (grid == 0) return cudaErrorInvalidValue;
  if constexpr (kCache == 4) {   // (the other types' append without a turn is pages_write_kernel)
    if (a.positions == nullptr) return launch_pdl(pages_append_kernel<4, 0, false>, grid, kThreads, 0, stream, a, per);
  }
  const bool q8 = a.h_q > 0 && a.q_out_e4m3;
  return launch_pdl(a.interleaved ? (q8 ? pages_append_kernel<kCache, 2, true> : pages_append_kernel<kCache, 2, false>)
                                  : (q8 ? pages_append_kernel<kCache, 1, true> : pages_append_kernel<kCache, 1, false>),
                    grid, kThreads, 0, stream, a, per);
}

cudaError_t launch_rows(const PagesAppendArgs& a, int dtype, bool read, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  return dtype == 1 ? launch_rows<1>(a, read, stream) : dtype == 2 ? launch_rows<2>(a, read, stream) : launch_rows<4>(a, read, stream);
}

}  // namespace

cudaError_t launch_pages_append(const PagesAppendArgs& a, int dtype, cudaStream_t stream) { return launch_rows(a, dtype, false, stream); }
cudaError_t launch_pages_read(const PagesAppendArgs& a, int dtype, cudaStream_t stream) { return launch_rows(a, dtype, true, stream); }

}  // namespace skv
