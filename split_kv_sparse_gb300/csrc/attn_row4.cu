// Attention of few query rows (at most 8 or 16: the tokens x the heads of one group) over a paged cache in 4 bits: decode.
// A key's K and V are 144 bytes a KV head, so at the rate of HBM an SM has to widen and multiply four fifths more
// keys than with e4m3: the instructions of a key bound the kernel beside the bytes. Both products are therefore taken
// the other way round than in the kernel of wider types, S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16, with 16 keys
// or dims as M and 8 query rows as N: K and V are widened once, straight into the registers of the A operand, and a
// group of 4 or 8 heads wastes half as many products as with 16 rows as M.
//
// Everything else is that kernel's: four warps a CTA, two CTAs an SM, each warp with key blocks (64 keys), a TMA ring, a
// running maximum and a sum of its own, merged at a job's end; equal shares of the batch's key tiles (AttnShares).
//
// Widening: a byte of two e2m1 codes is one conversion to an f16 pair, times its e4m3 scale in f16: exact (6
// significant bits, 2^-10 to 2688). The order of the contracted dims of S is free as long as Q has the same, so a lane takes
// 32 consecutive dims of a key (16 bytes: one load); for O a lane has 16 dims of four keys, and a pair of one dim of two
// keys is made by putting their codes into one byte before the conversion. Keys are taken in the order kPerm within
// eight, which keeps the loads of K and of V free of bank conflicts under the 64-byte swizzle.
// Q is held in f16 at a power of two of its row (largest element in [2^14, 2^15)): exact down to 2^-28 of that element, whose
// smaller ones are rounded by at most 2^-39 of it.
#include "attn_common.cuh"
#include "quant.cuh"

namespace skv {
namespace {

constexpr int kD = kAttnDim;
constexpr int kTile = kAttnKeyTile;
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kBlock = 64;                              // keys of a block
constexpr int kCodes = kBlock * kD / 2;                 // bytes of its K or V codes
constexpr int kScales = kBlock * 8;
constexpr int kOffV = kCodes, kOffKs = 2 * kCodes, kOffVs = kOffKs + kScales;
constexpr int kStageBytes = 2 * (kCodes + kScales);
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kOffBars = kWarps * kWarpBytes;
constexpr int kOffStats = kOffBars + kWarps * kStages * 8;   // float2 [kWarps][16]: m, l
constexpr int kOffAbort = kOffStats + kWarps * 16 * 8;
constexpr int kOffStage = kOffAbort + 16;               // int [kWarps]: the stage that holds a warp's result
constexpr int kSmem = kOffStage + 16 + 1024;
static_assert(16 * kD * 4 <= kStageBytes && kStageBytes % 512 == 0, "a warp's result goes through one stage; 64-byte swizzle");
static_assert(kRowCtasPerSm * (kSmem + 1024) <= 233472, "two CTAs an SM");
// A piece's start and end, in key tiles of an equal share.
constexpr int kRowHead = 2;

enum : uint32_t { W_R_FULL = 301, W_R_DRAIN };

// Row i of a tile's eight is key kPerm(i) = 0, 3, 1, 2, 4, 7, 5, 6.
__device__ __forceinline__ int perm8(int i) { return static_cast<int>((0x65742130u >> (4 * i)) & 7u); }

__device__ __forceinline__ void mma_f16_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
// kN: query rows of a job in eights.
template <int kN, bool kPoll>
__global__ void __launch_bounds__(kWarps * 32, kRowCtasPerSm)
    attn_row4_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs, const AttnArgs a,
                     const int box_rows) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, q4 = lane & 3;
  const uint32_t ring = sbase + warp * kWarpBytes;
  auto bar = [&](int st) -> uint32_t { return sbase + kOffBars + (warp * kStages + st) * 8; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  if (lane == 0) {
    for (int st = 0; st < kStages; ++st) mbar_init(bar(st), 1);
    if (warp == 0) *abort_flag = 0;
    mbar_init_fence();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_ks);
    tma_prefetch_desc(&tm_vs);
  }
  if (warp == 1) attn_prefetch(a, lane);
  __syncthreads();
  grid_dependency_wait();

  const int tokens = 8 * kN / a.group;
  // every warp for itself: the pieces of an equal share, or one job where the split count is given
  AttnShares<1, kRowHead> shares;
  AttnPiece next;
  if (a.adaptive == kShares) {
    shares.init(a, tokens, lane);
    next = shares.next(a);
  } else {
    AttnJobs jobs;
    jobs.init<false>(a, tokens, lane);
    next = jobs.find<true>(a, blockIdx.x, lane);
  }
  grid_launch_dependents();

  // ---- this warp's loads: they run ahead of its products, into the next piece
  const int box_shift = box_rows == 64 ? 6 : box_rows == 32 ? 5 : 4;
  const int boxes = kBlock >> box_shift;                 // pages (or parts of one) of a block: 1, 2 or 4
  struct Loads {                      // a piece: the warp's first key, its blocks, the sequence's keys, KV head, table
    int key, cnt, kv, g;
    const int32_t* table;
  };
  auto loads_of = [&](const AttnPiece& p) {
    const AttnSeq seq = attn_seq(a, p.b);
    const int key0 = p.tile0 * kTile;
    // up to the last token's keys
    const int key_end = static_cast<int>(min(key0 + static_cast<int64_t>(p.tiles) * kTile,
                                             static_cast<int64_t>(seq.kv - seq.sq + min((p.j + 1) * tokens, seq.sq))));
    const int blocks = key_end > key0 ? (key_end - key0 + kBlock - 1) / kBlock : 0;
    Loads x;
    x.key = key0 + warp * kBlock;
    x.cnt = blocks > warp ? (blocks - warp + kWarps - 1) / kWarps : 0;
    x.kv = seq.kv;
    x.g = p.g;
    x.table = a.table + static_cast<size_t>(p.b) * a.table_width;
    return x;
  };
  // lane's (block, box) of a group of 32: the page, or num_pages (zeros) where there is none
  auto lookup = [&](const Loads& x, int first) {
    const int e = first + lane;
    const int key = x.key + kWarps * kBlock * (e / boxes) + (e & (boxes - 1)) * box_rows;
    int page = a.num_pages;
    if (e < x.cnt * boxes && key < x.kv) {
      const int p = x.table[key >> a.page_shift];
      if (p >= 0 && p < a.num_pages) page = p;
    }
    return page;
  };
  int loaded = 0, issued = 0;         // blocks of earlier pieces; blocks whose loads were started
  uint32_t have = 0;                  // four bits a block in flight: its boxes' pages exist
  Loads in = {0, 0, 0, 0, nullptr}, then = in;   // the piece that the loads are in, the next one
  bool more = false;                  // `then` is there and not entered yet
  int at = 0, group0 = 0;             // next block of `in`; first (block, box) of `pages`
  int pages = 0, pages_next = 0, pages_then = 0;
  auto announce = [&](const AttnPiece& p) {   // `then` = p
    more = p.b >= 0;
    if (more) {
      then = loads_of(p);
      pages_then = lookup(then, 0);
    }
  };
  auto load_ahead = [&](int seen) {   // until every stage is in flight
    while (issued - seen < kStages) {
      if (at == in.cnt) {
        if (!more) break;
        more = false;
        in = then;
        at = group0 = 0;
        pages = pages_then;
        pages_next = lookup(in, 32);
        continue;
      }
      if (at * boxes - group0 >= 32) {
        pages = pages_next;
        group0 += 32;
        pages_next = lookup(in, group0 + 32);
      }
      const int box = lane & (boxes - 1);
      const int page = __shfl_sync(0xffffffffu, pages, (at * boxes - group0 + box) & 31);
      const unsigned got = __ballot_sync(0xffffffffu, lane < boxes && page != a.num_pages);
      have = (have & ~(15u << (4 * (issued & 7)))) | (got << (4 * (issued & 7)));
      const int st = issued % kStages;
      if (lane == 0) mbar_arrive_expect_tx(bar(st), kStageBytes);
      __syncwarp();
      if (lane < 4 * boxes) {          // a lane a box of K's or V's codes or scales
        const int which = lane >> (6 - box_shift);
        const int key = in.key + kWarps * kBlock * at + box * box_rows;
        const int row = key & ((1 << a.page_shift) - 1);
        const uint32_t dst = ring + st * kStageBytes;
        if (which < 2)
          tma_load_4d(dst + which * kOffV + box * box_rows * 64, which ? &tm_v : &tm_k, 0, row, page, in.g, bar(st));
        else
          tma_load_4d(dst + kOffKs + (which - 2) * kScales + box * box_rows * 8, which == 3 ? &tm_vs : &tm_ks, 2 * row, 0, page, in.g,
                      bar(st));
      }
      ++at;
      ++issued;
    }
  };
  auto drain = [&](int seen) {        // what was started may not be writing shared memory any more when the CTA ends
    bool done = true;
    for (int k = seen; k < issued; ++k)
      done = wait_drain(bar(k % kStages), (k / kStages) & 1, a.drain_limit_ns) && done;
    if (!done && lane == 0) atomicCAS(&a.status[1], 0u, W_R_DRAIN);
  };
  // shared memory offsets of this lane's rows of a tile of 16 keys
  const int k_row = perm8(quad);                          // keys of tile rows quad, and 8 on
  const uint32_t k_off = k_row * 64 + ((q4 ^ ((k_row >> 1) & 3)) << 4), ks_off = kOffKs + k_row * 8 + 2 * q4;
  uint32_t v_off[2], vs_off[2];                           // tile rows 2 q4 and 2 q4 + 1, and 8 on: dims 16 quad ..
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = perm8(2 * q4 + e);
    v_off[e] = kOffV + row * 64 + (((quad >> 1) ^ ((row >> 1) & 3)) << 4) + 8 * (quad & 1);
    vs_off[e] = kOffVs + row * 8 + quad;
  }
  announce(next);
#pragma unroll 1
  while (next.b >= 0) {
  const AttnPiece job = next;
  const AttnSeq seq = attn_seq(a, job.b);
  const int tok0 = job.j * tokens;
  const int ntok = min(tokens, seq.sq - tok0);
  load_ahead(loaded);                 // (every earlier block has been used, so the loads are in this piece now)
  const int first_key = in.key, cnt = in.cnt;   // this warp's
  next.b = -1;
  if (a.adaptive == kShares) next = shares.next(a);
  announce(next);

  // ---- Q fragments: row 8 n + quad (token r / group, head r % group), dims 32 q4 .. + 31, four a step
  const float dq = a.descale_q ? *a.descale_q : 1.f, dk = a.descale_k ? *a.descale_k : 1.f,
              dv = a.descale_v ? *a.descale_v : 1.f;
  const float sc = dq * dk * a.scale_log2;
  const bool raw_ok = sc > 0.f;
  uint32_t qf[kN][8][2];
  int lim[kN][2];                                         // last keys of rows 8 n + 2 q4 and + 1
  float esc[kN][2];
  int least = 0x7fffffff;
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    const int r = 8 * n + quad;
    const int t = r / a.group;
    const bool live = t < ntok;
    const int last = live ? seq.kv - seq.sq + tok0 + t : -1;
    least = min(least, live ? last : 0x7fffffff);
    uint32_t w[16];
    uint32_t top = 0;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + static_cast<int64_t>(seq.q0 + tok0 + t) * a.q_ts +
                                                       static_cast<int64_t>(job.g * a.group + (r - t * a.group)) * a.q_hs + 32 * q4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (live) v = from[i];
      w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = static_cast<int>(top >> 7);             // the largest element's exponent
    const float up = __int_as_float(min(268 - e, 254) << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      qf[n][i >> 1][i & 1] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
    const float down = e > 14 ? __int_as_float((e - 14) << 23) : __int_as_float(1 << 22);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      lim[n][k] = __shfl_sync(0xffffffffu, last, 8 * q4 + 4 * k);
      esc[n][k] = sc * __shfl_sync(0xffffffffu, down, 8 * q4 + 4 * k);
      if (raw_ok) esc[n][k] = fmaxf(esc[n][k], 1.17549435e-38f);   // (0 times a masked score's infinity would be a NaN)
    }
  }
  const int lim_min = min(__reduce_min_sync(0xffffffffu, least), seq.kv - 1);   // keys up to here are seen by every live row

  float o[8][kN][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[i][n][k] = 0.f;
  float m[kN][2], l[kN][2], lc[kN][2];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      m[n][k] = -INFINITY;
      l[n][k] = lc[n][k] = 0.f;
    }
  const uint32_t limit = wait_limit(a);
  bool ok = true;
  int nb = 0;
#pragma unroll 1
  for (; nb < cnt; ++nb) {
    load_ahead(loaded + nb);
    const int st = (loaded + nb) % kStages;
    if (!wait_for<kPoll>(bar(st), ((loaded + nb) / kStages) & 1, limit)) {
      ok = false;
      break;
    }
    const uint32_t stage = ring + st * kStageBytes;
    const int key = first_key + kWarps * kBlock * nb;
    if (key + kBlock > seq.kv) {
      // rows past the sequence's end: 0 * NaN would reach the result, and only a scale can be NaN
      for (int r = seq.kv - key + lane; r < kBlock; r += 32)
        *reinterpret_cast<uint2*>(smem + warp * kWarpBytes + st * kStageBytes + kOffVs + 8 * r) = make_uint2(0, 0);
      fence_proxy_async_smem();        // (a later load writes the stage)
      __syncwarp();
    }
    float s[4][kN][4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[t][n][k] = 0.f;
      uint32_t lo[4], hi[4];
      lds128(stage + k_off + t * 1024, lo);
      lds128(stage + k_off + t * 1024 + 512, hi);
      const uint32_t slo = f16x2_of_e4m3(lds16(stage + ks_off + t * 128)), shi = f16x2_of_e4m3(lds16(stage + ks_off + t * 128 + 64));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bl = __byte_perm(slo, 0, j < 2 ? 0x1010 : 0x3232), bh = __byte_perm(shi, 0, j < 2 ? 0x1010 : 0x3232);
        uint32_t x[4], y[4];
        f16_of_e2m1x8(lo[j], x);
        f16_of_e2m1x8(hi[j], y);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] = mul_f16x2(x[i], bl);
          y[i] = mul_f16x2(y[i], bh);
        }
#pragma unroll
        for (int n = 0; n < kN; ++n) {
          mma_f16_16x8(s[t][n], x[0], y[0], x[1], y[1], qf[n][2 * j][0], qf[n][2 * j][1]);
          mma_f16_16x8(s[t][n], x[2], y[2], x[3], y[3], qf[n][2 * j + 1][0], qf[n][2 * j + 1][1]);
        }
      }
    }
    if (!raw_ok) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[t][n][k] *= esc[n][k & 1];
    }
    const uint32_t there = (have >> (4 * ((loaded + nb) & 7))) & 15u;
    if (key + kBlock - 1 > lim_min || there != (1u << boxes) - 1u) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at_key = key + 16 * t + k_row + 8 * (k >> 1);
            if (at_key > lim[n][k & 1] || !((there >> ((16 * t) >> box_shift)) & 1u)) s[t][n][k] = -INFINITY;
          }
    }
    float mx[kN][2];
    bool need = false;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = fmaxf(s[0][n][k], s[0][n][k + 2]);
#pragma unroll
        for (int t = 1; t < 4; ++t) x = fmax3(x, s[t][n][k], s[t][n][k + 2]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        mx[n][k] = raw_ok ? x * esc[n][k] : x;
        need = need || new_reference<true>(mx[n][k], m[n][k]);
      }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (new_reference<true>(mx[n][k], m[n][k])) {
            const float al = m[n][k] == -INFINITY ? 0.f : ex2_approx(m[n][k] - mx[n][k]);
            m[n][k] = mx[n][k];
            l[n][k] *= al;
            lc[n][k] *= al;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][n][k] *= al;
              o[i][n][k + 2] *= al;
            }
          }
    }
    uint32_t pf[4][kN][2];                                 // P^T: keys 2 q4, 2 q4 + 1 (and + 8) of row quad
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float nm0 = minus_reference<true>(m[n][0]), nm1 = minus_reference<true>(m[n][1]);
      const float e0 = raw_ok ? esc[n][0] : 1.f, e1 = raw_ok ? esc[n][1] : 1.f;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int k = 0; k < 4; ++k) s[t][n][k] = ex2_approx(fmaf(s[t][n][k], k & 1 ? e1 : e0, k & 1 ? nm1 : nm0));
        sum[0] += s[t][n][0] + s[t][n][2];
        sum[1] += s[t][n][1] + s[t][n][3];
        pf[t][n][0] = transpose_8x8(pack_f16x2(s[t][n][0], s[t][n][1]));
        pf[t][n][1] = transpose_8x8(pack_f16x2(s[t][n][2], s[t][n][3]));
      }
      add_compensated(l[n][0], lc[n][0], sum[0]);
      add_compensated(l[n][1], lc[n][1], sum[1]);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      uint32_t w[2][2][2];                                 // [key + 8][key of the pair][eight dims]
      uint32_t sv[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lds64(stage + v_off[0] + t * 1024 + h * 512, w[h][0]);
        lds64(stage + v_off[1] + t * 1024 + h * 512, w[h][1]);
        sv[h] = f16x2_of_e4m3(lds8(stage + vs_off[0] + t * 128 + h * 64) | (lds8(stage + vs_off[1] + t * 128 + h * 64) << 8));
      }
      uint32_t x[2][2][8];                                 // [key + 8][dims + 8][dim]: a pair of keys
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const uint32_t u = w[h][0][d], v = w[h][1][d];
          uint32_t even[4], odd[4];
          f16_of_e2m1x8((u & 0x0f0f0f0fu) | ((v << 4) & 0xf0f0f0f0u), even);
          f16_of_e2m1x8(((u >> 4) & 0x0f0f0f0fu) | (v & 0xf0f0f0f0u), odd);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[h][d][2 * i] = mul_f16x2(even[i], sv[h]);
            x[h][d][2 * i + 1] = mul_f16x2(odd[i], sv[h]);
          }
        }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int n = 0; n < kN; ++n)
          mma_f16_16x8(o[i][n], x[0][0][i], x[0][1][i], x[1][0][i], x[1][1][i], pf[t][n][0], pf[t][n][1]);
    }
    __syncwarp();                                          // every lane has read the stage
  }
  if (!ok) {
    if (lane == 0) *abort_flag = 1;   // read at the merge
    give_up(a, W_R_FULL);
    drain(loaded + nb);
  }

  // ---- merge of the four warps' results
  // A warp's rows x 128 fp32 go through the stage that the next load will take (at most two are in flight now). Row r's
  // 16-byte piece c lies at c ^ c / 8 ^ r / 2 within its eight: no bank conflicts on either side.
  auto piece_at = [](int row, int c) { return row * 512 + (((c & 24) | ((c ^ (c >> 3) ^ ((row >> 1) & 3)) & 7)) << 4); };
  volatile int* stage_of = reinterpret_cast<volatile int*>(smem + kOffStage);
  uint8_t* mine = smem + warp * kWarpBytes + (issued % kStages) * kStageBytes;
  if (lane == 0) stage_of[warp] = issued % kStages;
  float2* stats = reinterpret_cast<float2*>(smem + kOffStats);
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float z = l[n][k];
      z += __shfl_xor_sync(0xffffffffu, z, 4);
      z += __shfl_xor_sync(0xffffffffu, z, 8);
      z += __shfl_xor_sync(0xffffffffu, z, 16);
      const int r = 8 * n + 2 * q4 + k;
#pragma unroll
      for (int h = 0; h < 2; ++h)                          // dims 16 quad + 8 h ..
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>(mine + piece_at(r, 4 * quad + 2 * h + j)) =
              make_float4(o[4 * j][n][2 * h + k], o[4 * j + 1][n][2 * h + k], o[4 * j + 2][n][2 * h + k], o[4 * j + 3][n][2 * h + k]);
      if (quad == 0) stats[warp * 16 + r] = make_float2(m[n][k], z);
    }
  __syncthreads();
  if (*abort_flag) {
    if (ok) drain(loaded + cnt);
    return;
  }
  const int row = threadIdx.x >> 3, x0 = (threadIdx.x & 7) * 16;
  const int rt = row / a.group;
  const bool live = row < 8 * kN && rt < ntok;
  float amax = 0.f;
  if (live) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stats[w * 16 + row].x);
    float tot = 0.f, y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 st = stats[w * 16 + row];
      const float f = st.x == -INFINITY ? 0.f : ex2_approx(st.x - M);
      tot = fmaf(st.y, f, tot);
      const uint8_t* r = smem + w * kWarpBytes + stage_of[w] * kStageBytes;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = *reinterpret_cast<const float4*>(r + piece_at(row, (x0 >> 2) + i));
        y[4 * i] = fmaf(v.x, f, y[4 * i]);
        y[4 * i + 1] = fmaf(v.y, f, y[4 * i + 1]);
        y[4 * i + 2] = fmaf(v.z, f, y[4 * i + 2]);
        y[4 * i + 3] = fmaf(v.w, f, y[4 * i + 3]);
      }
    }
    const bool some = tot > 0.f || tot != tot;
    const float inv = some ? dv / tot : 0.f;
    const float lse = some ? lse_of<true>(M, tot) : -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      y[i] = some ? y[i] * inv : 0.f;
      amax = fmaxf(amax, fabsf(y[i]));
    }
    const bool part = job.slot >= 0;
    const int64_t orow = static_cast<int64_t>(seq.q0 + tok0 + rt) * a.h_q + job.g * a.group + (row - rt * a.group);
    const int64_t prow = static_cast<int64_t>(job.slot) * kRowRows + row;
    if (part) store_row(a.o_part, 0, prow * kD + x0, y, 1.f);
    else store_row(a.out, a.out_dtype, orow * kD + x0, y, a.inv_scale);
    if (x0 == 0) {
      if (part) a.lse_part[prow] = lse;
      else if (a.lse_out != nullptr) a.lse_out[orow] = lse;
      if (a.row_map != nullptr && (job.S > 0 || !part) && row == rt * a.group)
        a.row_map[static_cast<int64_t>(seq.q0 + tok0 + rt) * a.h_kv + job.g] = make_int2(static_cast<int>(prow), part ? job.S : 0);
    }
  }
  if (job.slot < 0 && a.amax != nullptr) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
    if (lane == 0) atomicMax(reinterpret_cast<int*>(a.amax), __float_as_int(amax));
  }
  if (next.b < 0) break;
  loaded += cnt;
  fence_proxy_async_smem();            // stages were read and written here; TMA writes them next
  __syncthreads();
  }
}

using Row4Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, AttnArgs, int);
// [rows / 8 - 1][polling waits]
constexpr Row4Kernel kRow4Kernels[2][2] = {{attn_row4_kernel<1, false>, attn_row4_kernel<1, true>},
                                           {attn_row4_kernel<2, false>, attn_row4_kernel<2, true>}};

}  // namespace

int attn_row4_box(int page_size) { return page_size < kBlock ? page_size : kBlock; }

cudaError_t prepare_attn_row4() {
  for (int k = 0; k < 4; ++k) {
    const cudaError_t e = cudaFuncSetAttribute(kRow4Kernels[k >> 1][k & 1], cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_attn_row4(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const CUtensorMap& tm_ks, const CUtensorMap& tm_vs,
                             const AttnArgs& a, int rows, int64_t grid, cudaStream_t stream) {
  if (grid < 1 || grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(kRow4Kernels[rows > 8][a.wait_limit_ns < kSuspendNs], static_cast<unsigned>(grid), kWarps * 32, kSmem, stream,
                    tm_k, tm_v, tm_ks, tm_vs, a, attn_row4_box(1 << a.page_shift));
}

}  // namespace skv
