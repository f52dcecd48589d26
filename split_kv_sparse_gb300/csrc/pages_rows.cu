// Rows of the paged cache with arithmetic on the way: the append that rotates by position, the append into 4-bit
// pages, and the way back from pages of any type to bf16 rows.
//
// Both kernels are copies: every byte is read and written once and HBM bounds them, latency a call of a few rows. Eight
// threads take a head, 16 of its 128 dims each (two 16-byte pieces), a warp four heads at a time; with kFlight = 4 a
// thread has four heads of the row in flight and keeps its angles for all of them, with 1 a call of few rows spreads
// over more warps.
#include "attn_common.cuh"
#include "quant.cuh"

namespace skv {
namespace {

constexpr int kD = kAttnDim;
constexpr int kThreads = 256;
// Rows x heads from which a warp takes 16 heads of a row: 16 warps an SM have work then.
constexpr int64_t kManyHeads = 16ll * 16 * 152;

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ uint2 codes8(float (&x)[8], const Divider& by) {
  divide8(x, by);
  return make_uint2(pack_e4m3x4(x[0], x[1], x[2], x[3]), pack_e4m3x4(x[4], x[5], x[6], x[7]));
}

// Piece numbers (of eight dims) of thread p of a head: with halves rotated against each other, thread p < R / 16 has
// the pieces p and p + R / 16, whose dims are pairs; the other threads, and all with neighbours paired, have two
// pieces side by side.
__device__ __forceinline__ int2 pieces_of(int p, int rot, bool interleaved) {
  const int turning = interleaved ? 0 : rot >> 4;
  if (p < turning) return make_int2(p, p + turning);
  const int first = 2 * turning + 2 * (p - turning);
  return make_int2(first, first + 1);
}

// The append: y = x turned by the angles of its row's position (q and k heads), then to q_out, k_out and the cache.
// The products and their sum are rounded to fp32 one by one, so a code follows from plain fp32 arithmetic.
template <int kCache, int kFlight>
__global__ void __launch_bounds__(kThreads) pages_append_kernel(const PagesAppendArgs a) {
  const int lane = threadIdx.x & 31, p = lane & 7;
  const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  const int heads = a.h_q + 2 * a.h_kv;
  const int chunks = (heads + 4 * kFlight - 1) / (4 * kFlight);
  const int64_t r = w / chunks;
  const int h0 = static_cast<int>(w - r * chunks) * 4 * kFlight + (lane >> 3);
  const int2 piece = pieces_of(p, a.rot, a.interleaved);
  grid_dependency_wait();
  if (r >= a.rows) return;
  // (q and k may be written in place, by the thread that has read them: plain loads)
  uint4 x[kFlight][2];
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    const int h = h0 + 4 * k;
    if (h < heads) {
      const uint16_t* src = h < a.h_q ? a.q + r * a.q_ts + h * a.q_hs
                            : (h < a.h_q + a.h_kv ? a.k_new + (h - a.h_q) * a.head_stride : a.v_new + (h - a.h_q - a.h_kv) * a.head_stride) +
                                  r * a.token_stride;
      x[k][0] = *reinterpret_cast<const uint4*>(src + 8 * piece.x);
      x[k][1] = *reinterpret_cast<const uint4*>(src + 8 * piece.y);
    }
  }
  const int64_t slot = a.slots[r];
  int64_t pos = 0;
  if (a.positions != nullptr) pos = a.positions[r];
  const bool turning = p < (a.rot >> 4);
  if (a.positions != nullptr && (pos < 0 || pos >= a.num_positions)) return;   // padding: nothing of the row is written
  float c[8], s[8];
  if (turning) {
    const float* row = a.cos_sin + pos * a.rot + 8 * p;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 u = __ldg(reinterpret_cast<const float4*>(row) + i), v = __ldg(reinterpret_cast<const float4*>(row + (a.rot >> 1)) + i);
      c[4 * i] = u.x, c[4 * i + 1] = u.y, c[4 * i + 2] = u.z, c[4 * i + 3] = u.w;
      s[4 * i] = v.x, s[4 * i + 1] = v.y, s[4 * i + 2] = v.z, s[4 * i + 3] = v.w;
    }
  }
  const bool keep = slot >= 0 && slot < a.num_slots;
  const int64_t page = slot >> a.page_shift, at = slot & ((int64_t{1} << a.page_shift) - 1);
  const float dq = a.descale_q ? *a.descale_q : 1.f, dk = kCache != 1 && a.descale_k ? *a.descale_k : 1.f,
              dv = kCache != 1 && a.descale_v ? *a.descale_v : 1.f;
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    const int h = h0 + 4 * k;
    const bool is_q = h < a.h_q, is_k = !is_q && h < a.h_q + a.h_kv;
    float y[2][8];
    unpack8(x[k][0], y[0]);
    unpack8(x[k][1], y[1]);
    if (turning && (is_q || is_k)) {
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float& u = y[i >> 2][2 * (i & 3)];
          float& v = y[i >> 2][2 * (i & 3) + 1];
          const float u1 = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(v, s[i]));
          v = __fadd_rn(__fmul_rn(v, c[i]), __fmul_rn(u, s[i]));
          u = u1;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float u1 = __fsub_rn(__fmul_rn(y[0][i], c[i]), __fmul_rn(y[1][i], s[i]));
          y[1][i] = __fadd_rn(__fmul_rn(y[1][i], c[i]), __fmul_rn(y[0][i], s[i]));
          y[0][i] = u1;
        }
      }
    }
    if (is_q) {
      if (a.q_out_e4m3) {
        uint8_t* dst = static_cast<uint8_t*>(a.q_out) + r * a.qo_ts + h * a.qo_hs;
        const Divider by = divider(dq);
        *reinterpret_cast<uint2*>(dst + 8 * piece.x) = codes8(y[0], by);
        *reinterpret_cast<uint2*>(dst + 8 * piece.y) = codes8(y[1], by);
      } else {
        uint16_t* dst = static_cast<uint16_t*>(a.q_out) + r * a.qo_ts + h * a.qo_hs;
        *reinterpret_cast<uint4*>(dst + 8 * piece.x) = pack8(y[0]);
        *reinterpret_cast<uint4*>(dst + 8 * piece.y) = pack8(y[1]);
      }
    }
    if (is_k && a.k_out != nullptr) {
      uint16_t* dst = a.k_out + r * a.ko_ts + (h - a.h_q) * a.ko_hs;
      *reinterpret_cast<uint4*>(dst + 8 * piece.x) = pack8(y[0]);
      *reinterpret_cast<uint4*>(dst + 8 * piece.y) = pack8(y[1]);
    }
    const bool to_cache = keep && !is_q && h < heads;
    const int g = is_k ? h - a.h_q : h - a.h_q - a.h_kv;
    const int64_t dst = page * a.page_stride + at * a.row_stride + g * a.cache_head_stride;
    void* cache = is_k ? a.k : a.v;
    if constexpr (kCache == 1) {
      if (to_cache) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + dst + 8 * piece.x) = pack8(y[0]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + dst + 8 * piece.y) = pack8(y[1]);
      }
    } else if constexpr (kCache == 2) {
      if (to_cache) {
        const Divider by = divider(is_k ? dk : dv);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst + 8 * piece.x) = codes8(y[0], by);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst + 8 * piece.y) = codes8(y[1], by);
      }
    } else {
      const Divider by = divider(is_k ? dk : dv);
      float most[2] = {0.f, 0.f};
      if (to_cache) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          divide8(y[e], by);
#pragma unroll
          for (int i = 0; i < 8; ++i) most[e] = max_abs_nan(most[e], y[e][i]);
        }
      }
      // 16 dims with one scale: this thread's pieces, or each with the neighbour's
      const float other0 = __shfl_xor_sync(0xffffffffu, most[0], 1), other1 = __shfl_xor_sync(0xffffffffu, most[1], 1);
      const bool apart = turning && !a.interleaved;
      const float m0 = max_abs_nan(most[0], apart ? other0 : most[1]), m1 = max_abs_nan(most[1], apart ? other1 : most[0]);
      if (to_cache) {
        const uint32_t s0 = scale_code(m0), s1 = scale_code(m1);
        uint8_t* codes = static_cast<uint8_t*>(cache) + dst;
        *reinterpret_cast<uint32_t*>(codes + 4 * piece.x) = e2m1x8(y[0], e4m3_value(s0));
        *reinterpret_cast<uint32_t*>(codes + 4 * piece.y) = e2m1x8(y[1], e4m3_value(s1));
        uint8_t* scales = (is_k ? a.k_scales : a.v_scales) + page * a.scale_page_stride + g * a.scale_head_stride + 8 * at;
        if (!apart || !(p & 1)) scales[piece.x >> 1] = static_cast<uint8_t>(s0);
        if (apart && !(p & 1)) scales[piece.y >> 1] = static_cast<uint8_t>(s1);
      }
    }
  }
}

// The way back: 16 dims a thread, code x scale x descale rounded once to bf16 (a bf16 cache's bits as they are).
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
      x[k][0] = __ldg(from);
      x[k][1] = __ldg(from + 1);
    } else if constexpr (kCache == 2) {
      x[k][0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(cache) + src + 16 * p));
    } else {
      const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + src + 8 * p));
      x[k][0].x = v.x;
      x[k][0].y = v.y;
      scale[k] = __ldg((is_k ? a.k_scales : a.v_scales) + page * a.scale_page_stride + g * a.scale_head_stride + 8 * at + p);
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

template <int kCache>
cudaError_t launch_rows(const PagesAppendArgs& a, bool read, cudaStream_t stream) {
  const int64_t heads = read ? 2ll * a.h_kv : a.h_q + 2ll * a.h_kv;
  const bool many = a.rows * heads >= kManyHeads;
  const int64_t each = many ? 16 : 4;
  const int64_t warps = a.rows * ((heads + each - 1) / each);
  const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (read)
    return launch_pdl(many ? pages_read_kernel<kCache, 4> : pages_read_kernel<kCache, 1>, grid, kThreads, 0, stream, a);
  return launch_pdl(many ? pages_append_kernel<kCache, 4> : pages_append_kernel<kCache, 1>, grid, kThreads, 0, stream, a);
}

cudaError_t launch_rows(const PagesAppendArgs& a, int dtype, bool read, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  return dtype == 1 ? launch_rows<1>(a, read, stream) : dtype == 2 ? launch_rows<2>(a, read, stream) : launch_rows<4>(a, read, stream);
}

}  // namespace

cudaError_t launch_pages_append(const PagesAppendArgs& a, int dtype, cudaStream_t stream) { return launch_rows(a, dtype, false, stream); }
cudaError_t launch_pages_read(const PagesAppendArgs& a, int dtype, cudaStream_t stream) { return launch_rows(a, dtype, true, stream); }

}  // namespace skv
