// Attention of many query rows over a paged cache or packed K and V on the tensor
// cores: S = Q K^T (scaled to log2 units), an online softmax, O += P V.
//
// One CTA an SM takes job after job (sequence, KV head, query tile, split). A job's rows are
// tokens x the heads of one group, up to two blocks of 128 rows, so every K and V tile (128
// keys) is loaded once for the whole group. Two streams run through the tensor
// pipe in turn, so one stream's softmax overlaps the other's products:
//   two row blocks: stream i has row block i, both walk the same key tiles;
//   one row block:  both have it, stream i walks the tiles of parity i, and the two
//                   results are merged in shared memory.
//   warps 0-3, 4-7  softmax, rescale and epilogue of stream 0 and 1: a thread is a
//                   row (a TMEM lane), so no reduction crosses threads.
//   warps 8, 10     tcgen05 issue, in turn: S = Q_i K^T; O_i += P_i V with P_i read from
//                   tensor memory.
//   warps 9, 11     TMA: Q and the K tiles, the V tiles, each into a ring of slots, page by page;
//                   warp 11 also looks for the CTA's jobs and (bf16) clears the V rows past
//                   a sequence's end (0 * NaN would reach a result).
//   warps 12-15     e4m3: convert each V tile to f16 (exact), rows past the end to 0. 4 bits: convert Q's rows, and
//                   widen each K and V tile, to f16.
// TMEM: S (128 columns, one buffer for both streams: a stream's scores leave it for
// registers as soon as they are there), P_0, P_1 (64 each), O_0, O_1 (128 each).
// P is rounded to V's MMA type (bf16; f16 for V in e4m3 or 4 bits, whose values f16 holds exactly);
// the sums are taken over the unrounded fp32 values. bf16 P costs 2^-8 relative a
// term at most, as much as the rounding of a bf16 result, and also where the result is fp32 (a pair as in the 16-row kernel
// would double the PV products of a kernel that the tensor pipe bounds).
// The tensor pipe bounds the bf16 kernel (prompt of 16,384 tokens, 32/8 heads: 1.13 ms, 1.95 PFLOP/s, a call of a burst
// of 20; 1.28 ms, 1.71 PFLOP/s, one of 500, where the power cap takes the clock to 1.55 GHz), the softmax's latency the e4m3 one (2,900 clocks a tile of two streams, of which the products take
// 1,560; 7 ragged prompts: 234 us, 1.56 PFLOP/s). Between two jobs the pipe waits for the first one's epilogue
// (2.2 us into bf16 rows, 4 us into fp32 partials).
// 4 bits: much the same (2,048 tokens over 32,768 keys 612 to 640 us, 1.7 PFLOP/s; ragged chunks over pages of 16 358 us). Widening does not
// bound it (no gain without), the softmax and its code do: with a mask for the last keys, one for pages and a path for negative scales of their
// own, as the other types have them, 685 and 367 us; with the converting warps' code ahead of the softmax 818 and 390.
#include "attn_common.cuh"
#include "quant.cuh"

namespace skv {
namespace {

constexpr int kD = kAttnDim;
constexpr int kTile = kAttnKeyTile;
// A piece's start and end, in halves of a key tile of an equal share (2 to 12 measure alike).
constexpr int kTileHead = 4;

// kType: of the pages (1 bf16, 2 e4m3, 4 in 4 bits).
template <int kType>
struct Cfg {
  static constexpr bool kF8 = kType == 2, kF4 = kType == 4;
  static constexpr int kThreads = kF8 || kF4 ? 512 : 384;
  static constexpr int kQBytes = 128 * kD * (kF8 ? 1 : 2);   // one row block
  static constexpr int kCodeBytes = kTile * kD / 2;          // 4 bits: the codes of a tile, its scales behind them
  static constexpr int kItemBytes = kF4 ? kCodeBytes + kTile * 8 : kTile * kD * (kF8 ? 1 : 2);   // one K or V tile
  static constexpr int kHalves = kF8 ? 1 : 2;            // 128-byte column blocks of a row of Q (bf16: of K and V)
  static constexpr int kKSlots = kF8 ? 4 : 3;            // K(t) in slot t % kKSlots of its ring, V(t) in t % kVSlots
  static constexpr int kVSlots = kF8 ? 4 : kF4 ? 1 : 2;  // (4 bits: none, V lies in the ring of K, in the order item_of)
  static constexpr int kWideBytes = kF8 || kF4 ? kTile * kD * 2 : 0;   // a tile in f16
  static constexpr int kOffQ = 0;
  static constexpr int kOffK16 = 2 * kQBytes;
  static constexpr int kOffK = kOffK16 + (kF4 ? 2 * kWideBytes : 0);
  static constexpr int kOffV = kOffK + (kF4 ? 0 : kKSlots * kItemBytes);
  static constexpr int kOffV16 = kOffV + (kF4 ? kKSlots : kVSlots) * kItemBytes;
  static constexpr int kOffBars = kOffV16 + 2 * kWideBytes;
  static constexpr int kOffMisc = kOffBars + 352;
  static constexpr int kOffStats = kOffMisc + 384;       // float2 [128 rows]: m, l of stream 1
  static constexpr int kOffShares = kOffStats + 1024;
  static constexpr int kOffRow = kOffShares + 128;       // 4 bits: float [2 jobs][256 rows], what undoes a row's power of two
  static constexpr int kSmem = kOffRow + (kF4 ? 2048 : 0) + 1024;
  static_assert(kSmem <= 232448, "shared memory budget");
  static_assert(kOffV16 % 1024 == 0 && kOffK % 1024 == 0, "swizzle atoms");
  static constexpr int kConsumers = kF8 || kF4 ? 16 : 12;   // warps that read a job's description
};
// Where the scales of 4-bit pages lie; nothing for other types.
template <int kType>
struct ScalesOf {};
template <>
struct ScalesOf<4> {
  KvScales at;
};

enum {
  B_Q = 0, B_QDONE, B_S0, B_S1, B_SFREE, B_P0, B_P1, B_O0, B_O1, B_TURN_QK, B_TURN_PV, B_VLAND, B_END, B_DRAIN,
  B_DRAIN2, B_V16F0, B_V16F1, B_V16E0, B_V16E1, B_JOB0, B_JOB1, B_READ0, B_READ1, B_CLC, B_STAT,
  B_OREAD, B_KFULL,
  B_KEMPTY = B_KFULL + 4, B_VFULL = B_KEMPTY + 4, B_VEMPTY = B_VFULL + 4,
  B_Q16 = B_VEMPTY + 4, kNumBars   // (the last one: 4 bits alone, Q's rows are f16)
};
static_assert(kNumBars * 8 <= 352, "barrier area");
// 4 bits: the place of a tile in the order in which a job's K and V tiles are loaded and widened, K a tile ahead (K_0, K_1, V_0,
// K_2, V_1, .., V_n-2, V_n-1): V_t has to wait for the product of V_t-2, and the scores of later tiles not for that.
__device__ __forceinline__ int item_of(int t, int tiles, bool is_v) {
  return is_v ? (t == tiles - 1 ? 2 * tiles - 1 : 2 * t + 2) : (t == 0 ? 0 : 2 * t - 1);
}
// 4 bits: K tiles in f16, written and free (the places of the V ring's barriers, which has no ring of its own)
constexpr int B_K16F0 = B_VFULL, B_K16E0 = B_VEMPTY;

enum : uint32_t { W_T_SOFTMAX = 201, W_T_MMA, W_T_LOAD, W_T_CONVERT, W_T_DRAIN };   // whose wait ran out

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemP = 128, kTmemO = 256;   // S; P_0, P_1 (64 each); O_0, O_1 (128 each)

// What the roles need of a job, worked out once by the scheduler warp; two of them are
// in flight.
enum {
  J_B, J_G, J_S, J_SLOT, J_Q0, J_SQ, J_K0, J_KV,
  J_TOK0,             // first token (of the sequence) of row block 0
  J_TILE0, J_TILES,   // first key tile and count that the job walks
  J_ONE,              // one row block
  J_CNT0, J_CNT1,     // key tiles of each stream
  J_TAIL,             // the local tile that holds the sequence's ragged end, or -1
  kJobWords
};
enum { M_TMEM = 0, M_CLC = 4, M_JOBS = 8, M_MASK = M_JOBS + 2 * kJobWords, kMaskRing = 16, M_LAST = M_MASK + kMaskRing };
static_assert((M_LAST + 6) * 4 <= 384, "misc area");

// kPages: 0 packed K and V, jobs never split; 1 pages; 2 pages in equal shares (kernels of their
// own, since the loops' code has to stay near in the instruction caches).
template <int kType, int kPages, bool kPoll>
__global__ void __launch_bounds__(Cfg<kType>::kThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const AttnArgs a, const ScalesOf<kType> scales) {
  using C = Cfg<kType>;
  constexpr bool kF8 = C::kF8, kF4 = C::kF4;
  constexpr bool kF16 = kF8 || kF4;   // P and V are multiplied in f16
  constexpr bool kPaged = kPages > 0;
  constexpr int kRescaleUnroll = kF4 ? 2 : 8;   // (of O's rare rescaling; 4 bits: for its code's size)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + C::kOffMisc);
  auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBars + 8 * i; };

  const int tokens = 128 / a.group;   // of one row block
  if (threadIdx.x == 0) {
    // Arrivals: of four warps, of a tile's converting warps, of all that read a job's description; of 4-bit codes' bytes and each lane's
    // copies of scales. (An expression for each kind: with Q16 among the barriers of e4m3 too its kernels' loops lay elsewhere in
    // the code, and ragged chunks over pages of 16 took 141.3 us instead of 139, 1 to 16 tokens 40.6 instead of 39.6.)
    for (int i = 0; i < (kF4 ? kNumBars : B_Q16); ++i) {
      const int n = kF4 ? (i == B_STAT || i == B_OREAD || i == B_SFREE || i == B_P0 || i == B_P1 || i == B_V16F0 || i == B_V16F1 ||
                                   i == B_Q16 || (i >= B_KEMPTY && i < B_KEMPTY + 4) || i == B_K16F0 || i == B_K16F0 + 1
                               ? 4
                           : i >= B_KFULL && i < B_KEMPTY       ? 33
                           : i == B_READ0 || i == B_READ1       ? C::kConsumers
                                                                : 1)
                    : i == B_STAT || i == B_OREAD || i == B_SFREE || i == B_P0 || i == B_P1 || i == B_V16F0 || i == B_V16F1 ||
                            (kF8 && i >= B_VEMPTY)
                        ? 4
                    : i == B_READ0 || i == B_READ1 ? C::kConsumers
                                                   : 1;
      mbar_init(bar(i), n);
    }
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(smem_u32(smem + C::kOffMisc), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dependency_wait();
  grid_launch_dependents();
  const uint32_t tmem = static_cast<uint32_t>(misc[M_TMEM]);
  const uint32_t limit = wait_limit(a);
  // Job number k of this CTA: waits until the scheduler has described it and returns its words (negative J_B: no more).
  auto job_at = [&](int k, volatile int*& words) {
    words = misc + M_JOBS + (k & 1) * kJobWords;
    return wait_for<kPoll>(bar(B_JOB0 + (k & 1)), (k >> 1) & 1, limit);
  };
  // The words have been copied.
  auto job_read = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_READ0 + (k & 1)));
  };

  if (warp < 8) {
    // ================================================= softmax + epilogue ===
    if constexpr (kF16) regs_inc<192>();
    else regs_inc<208>();
    const int i = warp >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts = tmem + lanes + kTmemS, tp = tmem + lanes + kTmemP + 64 * i, to = tmem + lanes + kTmemO + 128 * i;
    const int rt = row / a.group;                          // token of the block
    const float dq = a.descale_q ? *a.descale_q : 1.f, dk = a.descale_k ? *a.descale_k : 1.f,
                dv = a.descale_v ? *a.descale_v : 1.f;
    const float sc = dq * dk * a.scale_log2;
    const bool raw_ok = sc > 0.f;      // then the scale commutes with the maximum and goes into the exponent's FMA
    const float unit = raw_ok ? sc : 1.f;
    int su = 0, ends = 0, ones = 0, mask0 = 0;   // this stream's tiles, jobs with tiles, jobs of one row block, all tiles
#pragma unroll 1
    for (int job = 0;; ++job) {
    volatile int* w;
    if (!job_at(job, w) || w[J_B] < 0) break;
    const int g = w[J_G], S = w[J_S], slot0 = w[J_SLOT], q0 = w[J_Q0], sq = w[J_SQ], kv = w[J_KV],
              tok0 = w[J_TOK0], tile0 = w[J_TILE0], tiles = w[J_TILES], cnt0 = w[J_CNT0], cnt1 = w[J_CNT1];
    const bool one = w[J_ONE] != 0;
    job_read(job);
    const int cnt = i ? cnt1 : cnt0;
    const int tok = tok0 + (one ? 0 : i * tokens) + rt;    // token of the sequence
    const bool live = rt < tokens && tok < sq;
    const int lim = live ? kv - sq + tok : kv - 1;   // last key the row sees (a dead row's result goes nowhere)
    float m_run = -INFINITY, l = 0.f, lc = 0.f;
    bool bad = false;
    float esc = unit;                  // (4 bits: of this row of the job, with what undoes its power of two; the sign is in Q)
#pragma unroll 1
    for (int u = 0; u < cnt; ++u) {
      const int t = one ? 2 * u + i : u;
      if (!wait_for<kPoll>(bar(B_S0 + i), (su + u) & 1, limit)) {
        bad = true;
        break;
      }
      tc_fence_after();
      if (kF4 && u == 0) {
        // (written before the scores' product was issued. No wait for Q's own barrier here: behind a long epilogue it may be two jobs
        // further on, and its parity would say nothing)
        const float x = fabsf(sc) * reinterpret_cast<volatile float*>(smem + C::kOffRow)[256 * (ends & 1) + (one ? 0 : 128 * i) + row];
        esc = x == x ? fmaxf(x, 1.17549435e-38f) : x;   // (0 times a masked score's infinity would be a NaN)
      }
      uint32_t pages4 = 0xffu;           // 4 bits: 16-key groups with a page (read here, not behind the scores: 655 -> 634 us)
      if constexpr (kF4) pages4 = static_cast<uint32_t>(misc[M_MASK + ((mask0 + t) & (kMaskRing - 1))]);
      uint32_t r[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(ts + 32 * c, r[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_wait_ld_x32(r[c]);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_SFREE));   // the other stream's scores may come
      float(&x)[4][32] = reinterpret_cast<float(&)[4][32]>(r);
      if (!kF4 && !raw_ok) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int k = 0; k < 32; ++k) x[c][k] *= sc;
      }
      const int kmax = lim - (tile0 + t) * kTile;          // last visible key of the tile
      if constexpr (kF4) {
        // (both masks in one block: rarely run, but the loop's code that it parts has to be fetched around it)
        if (__any_sync(0xffffffffu, kmax < kTile - 1 || pages4 != 0xffu)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int last = kmax - 32 * c;
            const uint32_t seen = (last >= 31 ? 0xffffffffu : last < 0 ? 0u : (2u << last) - 1u) &
                                  (((pages4 >> (2 * c)) & 1u ? 0xffffu : 0u) | ((pages4 >> (2 * c + 1)) & 1u ? 0xffff0000u : 0u));
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (!((seen >> k) & 1u)) x[c][k] = -INFINITY;
          }
        }
      } else {
        if (__any_sync(0xffffffffu, kmax < kTile - 1)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (32 * c + k > kmax) x[c][k] = -INFINITY;
        }
        const uint32_t pages = !kPaged ? 0xffu : static_cast<uint32_t>(misc[M_MASK + ((mask0 + t) & (kMaskRing - 1))]);   // 16-key groups with a page
        if (pages != 0xffu) {
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (!((pages >> c) & 1u)) {
#pragma unroll
              for (int k = 0; k < 16; ++k) x[c >> 1][16 * (c & 1) + k] = -INFINITY;
            }
        }
      }
      const float mx = fmaxf(fmaxf(max32(x[0]), max32(x[1])), fmaxf(max32(x[2]), max32(x[3]))) * esc;
      const bool need = new_reference<kF16>(mx, m_run);
      // O_i's last product is done: P_i may be written again, O_i rescaled
      if (u > 0 && !wait_for<kPoll>(bar(B_O0 + i), (su + u - 1) & 1, limit)) {
        bad = true;
        break;
      }
      tc_fence_after();
      if (__any_sync(0xffffffffu, need)) {
        float al = 1.f;
        if (need) {
          al = m_run == -INFINITY ? 0.f : ex2_approx(m_run - mx);
          m_run = mx;
          l *= al;
          lc *= al;
        }
        if (u > 0) {
#pragma unroll kRescaleUnroll
          for (int c = 0; c < 8; ++c) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(to + 16 * c, o);
            tmem_wait_ld_x16(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al);
            tmem_st_32x32b_x16(to + 16 * c, o);
          }
        }
      }
      const float nm = minus_reference<kF16>(m_run);
      const uint64_t esc2 = pair_f32(esc, esc), nm2 = pair_f32(nm, nm);
      uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t p[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float e0, e1;
          unpair_f32(fma_f32x2(pair_f32(x[c][2 * k], x[c][2 * k + 1]), esc2, nm2), e0, e1);
          e0 = ex2_approx(e0);
          e1 = ex2_approx(e1);
          sum[k & 3] = add_f32x2(sum[k & 3], pair_f32(e0, e1));
          p[k] = kF16 ? pack_f16x2(e0, e1) : pack_bf16x2(e0, e1);
        }
        tmem_st_32x32b_x16(tp + 16 * c, p);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_P0 + i));
      float s0, s1;
      unpair_f32(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), s0, s1);
      add_compensated(l, lc, s0 + s1);
    }

    // ---- epilogue
    if (!bad && cnt > 0) bad = !wait_for<kPoll>(bar(B_O0 + i), (su + cnt - 1) & 1, limit);
    // one row block: stream 0 takes both results from tensor memory (they lie in the same lanes)
    if (one && tiles > 0 && !bad) bad = !wait_for<kPoll>(bar(B_END), ends & 1, limit);
    tc_fence_after();
    float2* stats = reinterpret_cast<float2*>(smem + C::kOffStats);
    if (one && i == 1) {
      stats[row] = make_float2(m_run, l);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_STAT));
      bad = !wait_for<kPoll>(bar(B_OREAD), ones & 1, limit) || bad;   // stream 0 has read O_1
    } else {
      float w0 = 1.f, w1 = 0.f;
      if (one) {
        bad = !wait_for<kPoll>(bar(B_STAT), ones & 1, limit) || bad;
        const float2 st = stats[row];
        const float M = fmaxf(m_run, st.x);
        w0 = m_run == -INFINITY ? 0.f : ex2_approx(m_run - M);
        w1 = st.x == -INFINITY ? 0.f : ex2_approx(st.x - M);
        l = l * w0 + st.y * w1;
        m_run = M;
      }
      if (!bad) {
        const bool some = l > 0.f || l != l;   // a NaN score stays a NaN result
        const float inv = some ? dv / l : 0.f;
        const float lse = some ? lse_of<kF16>(m_run, l) : -INFINITY;
        const int64_t orow = static_cast<int64_t>(q0 + tok) * a.h_q + g * a.group + (row - rt * a.group);
        const int64_t prow = static_cast<int64_t>(slot0) * kTileRows + (one ? 0 : 128 * i) + row;
        const bool part = kPaged && slot0 >= 0;
        if (live) {
          if (part) a.lse_part[prow] = lse;
          else if (a.lse_out != nullptr) a.lse_out[orow] = lse;
          if (kPaged && a.row_map != nullptr && (S > 0 || !part) && row == rt * a.group)
            a.row_map[static_cast<int64_t>(q0 + tok) * a.h_kv + g] = make_int2(static_cast<int>(prow), part ? S : 0);
        }
        // A thread stores its own row, whole 32-byte sectors at a time: no place in shared memory is needed, so the next
        // job's Q can be loaded, and its first scores computed, meanwhile (8 prompts of 2,048 tokens: 219 us with the rows
        // staged in Q's place, 194 so).
        const int dst_type = part ? 0 : a.out_dtype;
        uint8_t* dst = part ? reinterpret_cast<uint8_t*>(a.o_part + prow * kD)
                            : static_cast<uint8_t*>(a.out) + orow * (dst_type == 0 ? kD * 4 : dst_type == 1 ? kD * 2 : kD);
        const bool wide = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
        float amax = 0.f;
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          __syncwarp();
          float y[32];
          if (cnt > 0) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 32 * c, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = some ? __uint_as_float(o[k]) : 0.f;
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = 0.f;
          }
          if (one && cnt1 > 0) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + 128 + 32 * c, o);
            tmem_wait_ld_x32(o);
#pragma unroll
            for (int k = 0; k < 32; ++k) y[k] = y[k] * w0 + (w1 != 0.f ? __uint_as_float(o[k]) * w1 : 0.f);
          }
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            y[k] *= inv;
            amax = fmaxf(amax, fabsf(y[k]));
          }
          if (live) {
            if (dst_type == 0) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = __float_as_uint(y[8 * k + e]);
                st_global_32(dst + 128 * c + 32 * k, v, wide);
              }
            } else if (dst_type == 1) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                uint32_t v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = pack_bf16x2(y[16 * k + 2 * e], y[16 * k + 2 * e + 1]);
                st_global_32(dst + 64 * c + 32 * k, v, wide);
              }
            } else {
              uint32_t v[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                v[e] = pack_e4m3x4(y[4 * e] * a.inv_scale, y[4 * e + 1] * a.inv_scale, y[4 * e + 2] * a.inv_scale,
                                   y[4 * e + 3] * a.inv_scale);
              st_global_32(dst + 32 * c, v, wide);
            }
          }
        }
        if (!part && a.amax != nullptr) {
          if (!live) amax = 0.f;
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          if (lane == 0) atomicMax(reinterpret_cast<int*>(a.amax), __float_as_int(amax));
        }
      }
      if (one) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_OREAD));
      }
    }
    tc_fence_before();
    su += cnt;
    mask0 += tiles;
    ends += tiles > 0 ? 1 : 0;
    ones += one ? 1 : 0;
    if (bad) {
      give_up(a, W_T_SOFTMAX);
      break;
    }
    }
  } else {
    if constexpr (kF16) regs_dec<64>();
    else regs_dec<88>();
    if (warp == 8 || warp == 10) {
      // ====================================================== MMA issuers ===
      // The whole warp walks its loop, so addresses stay uniform; one elected lane issues. The pipe takes the order
      // QK_0(u), PV_0(u - 1), QK_1(u), PV_1(u - 1): S is one buffer, and stream 0 takes S_0(u) into registers while PV_0(u - 1)
      // runs; a stream has the time of four products for its softmax. An issue blocks until the pipe is two MMAs
      // from idle, so a wait on one warp alone would be idle time, and two warps in no order would stretch both
      // products: each warp waits for its own operands ahead, then for its turn. PV number m follows QK number m + 2.
      // 128-byte-swizzled operands with 1024-byte atoms: one high word for all but V's leading stride (its low word)
      const uint32_t hi = static_cast<uint32_t>(sdesc_sw128(sbase, 16, 1024) >> 32);
      const bool is_qk = warp == 8;
      constexpr uint32_t kIdescQK = idesc_make(128, 128, kF16 ? 0 : 1, false, false);
      constexpr uint32_t kIdescPV = idesc_make(128, 128, kF16 ? 0 : 1, false, true);   // f16 or bf16; V is MN-major
      const uint32_t q_lo = static_cast<uint32_t>(sdesc_sw128(sbase + C::kOffQ, 16, 1024));
      const uint32_t k_lo = static_cast<uint32_t>(sdesc_sw128(sbase + (kF4 ? C::kOffK16 : C::kOffK), 16, 1024));
      // K and V tiles: the 64-dim column blocks one after the other (8-row atoms 1024 bytes apart), or with kv_wide
      // beside one another (atoms 2048 bytes apart, the second block 1024 bytes on)
      const bool wide = kPaged && !kF16 && a.kv_wide != 0;
      const uint32_t block = wide ? 1024 : kTile * 128;
      const uint32_t kv_hi = wide ? static_cast<uint32_t>(sdesc_sw128(sbase, 16, 2048) >> 32) : hi;
      const uint32_t v_step = (wide ? 4096 : 2048) >> 4;   // 16 keys
      const uint32_t v_lo = static_cast<uint32_t>(sdesc_sw128(sbase + (kF16 ? C::kOffV16 : C::kOffV), block, 1024));
      bool ok = true;
      int tile_base = 0;     // tiles of earlier jobs
      int n = 0;             // this warp's products so far
      int with_tiles = 0;    // jobs that had any
      int seen0 = 0, seen1 = 0;
#pragma unroll 1
      for (int job = 0; ok; ++job) {
        volatile int* w;
        ok = job_at(job, w);
        if (!ok || w[J_B] < 0) break;
        const int tiles = w[J_TILES], cnt0 = w[J_CNT0], cnt1 = w[J_CNT1];
        const bool one = w[J_ONE] != 0;
        job_read(job);
        if (tiles == 0) continue;
        const int steps = max(cnt0, cnt1);
        auto tile_at = [&](int i, int u) { return one ? 2 * u + i : u; };
        if (is_qk) {
          const uint32_t d = tmem + kTmemS;
          const int first = n;   // (a job's first products have none of its own to follow)
          // (the last job's products are all done, so the turns below start afresh; its rows may still be on their way out)
          ok = wait_for<kPoll>(bar(kF4 ? B_Q16 : B_Q), with_tiles & 1, limit) &&
               (with_tiles == 0 || wait_for<kPoll>(bar(B_END), (with_tiles - 1) & 1, limit));
#pragma unroll 1
          for (int u = 0; ok && u < steps; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || u >= (i ? cnt1 : cnt0)) continue;
              const int t = tile_base + tile_at(i, u);
              ok = (kF4 ? wait_for<kPoll>(bar(B_K16F0 + (t & 1)), (t >> 1) & 1, limit)
                        : wait_for<kPoll>(bar(B_KFULL + t % C::kKSlots), (t / C::kKSlots) & 1, limit)) &&
                   (n < first + 3 || wait_for<kPoll>(bar(B_TURN_QK), (n - 3) & 1, limit)) &&
                   (n == 0 || wait_for<kPoll>(bar(B_SFREE), (n - 1) & 1, limit));
              if (!ok) break;
              ++n;
              tc_fence_after();
              if (elect_one()) {
                const uint32_t qa = q_lo + (one ? 0 : i) * (C::kQBytes >> 4);
                const uint32_t kb = k_lo + (kF4 ? static_cast<uint32_t>(t & 1) * (C::kWideBytes >> 4)
                                                : static_cast<uint32_t>(t % C::kKSlots) * (C::kItemBytes >> 4));
                if constexpr (kF8) {
                  mma_f8_wc<0>(d, qa, kb, hi, kIdescQK);
                  mma_f8_wc<1>(d, qa + 2, kb + 2, hi, kIdescQK);
                  mma_f8_wc<1>(d, qa + 4, kb + 4, hi, kIdescQK);
                  mma_f8_wc<1>(d, qa + 6, kb + 6, hi, kIdescQK);
                } else {
                  const uint32_t kb2 = kb + (block >> 4);   // 64 dims a column block, 16 an MMA
                  mma_f16_wc2<0>(d, qa, hi, kb, kv_hi, kIdescQK);
#pragma unroll
                  for (int k = 1; k < 8; ++k)
                    mma_f16_wc2<1>(d, qa + (k >> 2) * (128 * 128 >> 4) + (k & 3) * 2, hi, (k < 4 ? kb : kb2) + (k & 3) * 2, kv_hi,
                                   kIdescQK);
                }
                mbar_arrive(bar(B_TURN_PV));
                mma_commit(bar(B_S0 + i));
                if (one || i == 1) mma_commit(bar(kF4 ? B_K16E0 + (t & 1) : B_KEMPTY + t % C::kKSlots));
              }
              __syncwarp();
            }
          }
          if (ok && elect_one()) mma_commit(bar(B_QDONE));
          __syncwarp();
        } else {
          const int last = n + cnt0 + cnt1 - 1;   // the job's last product
#pragma unroll 1
          for (int u = 0; ok && u < steps; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || u >= (i ? cnt1 : cnt0)) continue;
              const int t = tile_base + tile_at(i, u);
              if constexpr (kF16) ok = wait_for<kPoll>(bar(B_V16F0 + (t & 1)), (t >> 1) & 1, limit);
              else
                ok = wait_for<kPoll>(bar(B_VFULL + t % C::kVSlots), (t / C::kVSlots) & 1, limit);
              // (the job's last two products have no later QK to follow; the turn is an order, P is the dependency)
              ok = ok && wait_for<kPoll>(bar(B_P0 + i), (i ? seen1 : seen0) & 1, limit) &&
                   (n + 2 > last || wait_for<kPoll>(bar(B_TURN_PV), (n + 2) & 1, limit));
              if (!ok) break;
              ++n;
              if (i) ++seen1;
              else ++seen0;
              tc_fence_after();
              if (elect_one()) {
                uint32_t vb = v_lo;
                if constexpr (kF16) vb += static_cast<uint32_t>(t & 1) * (C::kWideBytes >> 4);
                else vb += static_cast<uint32_t>(t % C::kVSlots) * (C::kItemBytes >> 4);
                const uint32_t pa = tmem + kTmemP + 64 * i, d = tmem + kTmemO + 128 * i;
#pragma unroll
                for (int k = 0; k < 8; ++k)   // 16 keys an MMA: 8 columns of P, two 8-row atoms of V
                  mma_f16_ts(d, pa + 8 * k, vb + k * v_step, kv_hi, kIdescPV, k > 0 ? 1u : (u > 0 ? 1u : 0u));
                mbar_arrive(bar(B_TURN_QK));
                mma_commit(bar(B_O0 + i));
                if (one || i == 1) {
                  if constexpr (kF16) mma_commit(bar(B_V16E0 + (t & 1)));
                  else mma_commit(bar(B_VEMPTY + t % C::kVSlots));
                }
              }
              __syncwarp();
            }
          }
          if (ok && elect_one()) mma_commit(bar(B_END));
          __syncwarp();
        }
        tile_base += tiles;
        ++with_tiles;
      }
      if (!ok) {
        give_up(a, W_T_MMA);
        const int drain = is_qk ? B_DRAIN : B_DRAIN2;
        if (elect_one()) mma_commit(bar(drain));
        __syncwarp();
        if (!wait_drain(bar(drain), 0, a.drain_limit_ns)) atomicExch(&a.status[1], W_T_DRAIN);
      }
    } else if (warp == 9 || warp == 11) {
      // ============================================ loads (K and Q; V) and jobs ===
      // Warp 9 loads Q and the K tiles, warp 11 the V tiles: with pages of 16 rows a tile is eight boxes, and one warp's
      // issue of K and V would bound the kernel. Warp 11 also describes the jobs: this CTA's own, then, each time the
      // loads of one have all been started, that of a CTA that was not launched yet and that it takes over.
      const bool is_k = warp == 9;
      const int page_rows = kPaged ? min(1 << a.page_shift, kTile) : kTile;
      const int boxes = kTile / page_rows;                 // of one tile (and column block)
      bool ok = true;
      int done = 0;                                        // tiles whose loads were started
      int with_tiles = 0, landed = 0;                      // jobs that had any; V tiles that went by B_VLAND
      int tile_base = 0, older[3] = {-1, -1, -1};          // 4 bits: tiles of earlier jobs, this warp's last items
      AttnJobs jobs;
      // (in shared memory between the jobs: the loads' loop needs the registers)
      auto shares_at = reinterpret_cast<AttnShares<2, kTileHead>*>(smem + C::kOffShares);
      static_assert(sizeof(AttnShares<2, kTileHead>) <= 128, "shares area");
      constexpr bool shared = kPages == 2;
      int idx = blockIdx.x, asked = 0;
      auto take_over = [&]() {                             // the index of a CTA that was pending, or -1
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_CLC), 16);
          try_cancel_cta(sbase + C::kOffMisc + 4 * M_CLC, bar(B_CLC));
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, wait_drain(bar(B_CLC), asked & 1, a.drain_limit_ns));
        ++asked;
        const int x = ok ? canceled_cta(sbase + C::kOffMisc + 4 * M_CLC) : -1;
        fence_proxy_async_smem();
        __syncwarp();
        return x;
      };
      if (!is_k) {
        if (lane == 0) {
          tma_prefetch_desc(&tm_q);
          tma_prefetch_desc(&tm_k);
          tma_prefetch_desc(&tm_v);
        }
        if constexpr (shared) {
          AttnShares<2, kTileHead> shares;
          shares.init(a, 2 * tokens, lane);
          if (lane == 0) *shares_at = shares;
          __syncwarp();
        } else {
          jobs.init<kPaged>(a, 2 * tokens, lane);
        }
      }
      // Works out job number `job` and writes its words.
      auto describe = [&](int job) {
        AttnPiece next = {-1, 0, 0, 0, 0, -1, 0};
        if constexpr (shared) {
          AttnShares<2, kTileHead> shares = *shares_at;
          next = shares.next(a);
          __syncwarp();
          if (lane == 0) *shares_at = shares;
          __syncwarp();
        } else {
          if (job > 0) idx = take_over();
          while (ok && idx >= 0) {
            next = jobs.find<kPaged>(a, idx, lane);
            if (next.b >= 0) break;
            idx = take_over();   // (an index past the batch's jobs; the grid is sized by a bound)
          }
        }
        volatile int* w = misc + M_JOBS + (job & 1) * kJobWords;
        ok = ok && (job < 2 || wait_for<kPoll>(bar(B_READ0 + (job & 1)), ((job >> 1) - 1) & 1, limit));
        if (!ok) return;
        if (lane == 0) {
          w[J_B] = next.b;
          if (next.b >= 0) {
            const AttnSeq seq = attn_seq(a, next.b);
            const int tok0 = next.j * 2 * tokens;
            const int tiles_all = (seq.kv + kTile - 1) / kTile;
            const int tile0 = next.tile0, nt = max(min(next.tiles, tiles_all - tile0), 0);
            // key tiles of row block i: up to the position of its last token
            auto tiles_of = [&](int i) {
              const int last = min(tok0 + (i + 1) * tokens, seq.sq) - 1;
              if (last < tok0 + i * tokens) return 0;
              const int keys = seq.kv - seq.sq + last + 1;
              return min(max((keys + kTile - 1) / kTile - tile0, 0), nt);
            };
            const bool one = tok0 + tokens >= seq.sq;
            const int n0 = tiles_of(0), n1 = tiles_of(1);  // n1 >= n0 where there is a second block
            const int tiles = one ? n0 : n1;
            w[J_G] = next.g;
            w[J_S] = next.S;
            w[J_SLOT] = next.slot;
            w[J_Q0] = seq.q0;
            w[J_SQ] = seq.sq;
            w[J_K0] = seq.k0;
            w[J_KV] = seq.kv;
            w[J_TOK0] = tok0;
            w[J_TILE0] = tile0;
            w[J_TILES] = tiles;
            w[J_ONE] = one;
            w[J_CNT0] = one ? (tiles + 1) >> 1 : n0;
            w[J_CNT1] = one ? tiles >> 1 : n1;
            w[J_TAIL] = (seq.kv & (kTile - 1)) != 0 && tiles_all - 1 - tile0 < tiles ? tiles_all - 1 - tile0 : -1;
          }
          mbar_arrive(bar(B_JOB0 + (job & 1)));
        }
        __syncwarp();
      };
#pragma unroll 1
      for (int job = 0; ok; ++job) {
        if (!is_k) describe(job);
        volatile int* w;
        ok = ok && job_at(job, w);
        if (!ok || w[J_B] < 0) break;
        const int job_b = w[J_B], g = w[J_G], q0 = w[J_Q0], k0 = w[J_K0], kv = w[J_KV], tok0 = w[J_TOK0], tile0 = w[J_TILE0],
                  tiles = w[J_TILES], tail = w[J_TAIL];
        const bool one = w[J_ONE] != 0;
        job_read(job);
        // this lane's page of tile t: (page, row), page = num_pages (zeros) where there is none
        auto lookup = [&](int t, int& page, int& row) {
          const int key = (tile0 + t) * kTile + lane * page_rows;
          if (!kPaged) {
            page = 0;
            row = k0 + key;
            return true;
          }
          page = a.num_pages;
          row = key & ((1 << a.page_shift) - 1);
          if (lane < boxes && key < kv) {
            const int p = a.table[static_cast<size_t>(job_b) * a.table_width + (key >> a.page_shift)];
            if (p >= 0 && p < a.num_pages) page = p;
          }
          return page != a.num_pages;
        };
        int page = 0, row = 0;
        bool have = tiles > 0 && lookup(0, page, row);
        const int slots = is_k || kF4 ? C::kKSlots : C::kVSlots, full = is_k || kF4 ? B_KFULL : B_VFULL,
                  empty = is_k || kF4 ? B_KEMPTY : B_VEMPTY;
        const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
          int page_n = 0, row_n = 0;
          bool have_n = false;
          if (t + 1 < tiles) have_n = lookup(t + 1, page_n, row_n);
          const int item = kF4 ? 2 * tile_base + item_of(t, tiles, !is_k) : done;
          const int sl = item % slots;
          if (item >= slots && !wait_for<kPoll>(bar(empty + sl), ((item / slots) - 1) & 1, limit)) {
            ok = false;
            break;
          }
          if (kPaged && is_k) {
            // the tile's 16-key groups that have a page (those past the sequence's end are masked anyway)
            const unsigned got = __ballot_sync(0xffffffffu, have);
            unsigned groups = 0;
            for (int i = 0; i < 8; ++i)
              if ((got >> (i * 16 / page_rows)) & 1u) groups |= 1u << i;
            if (lane == 0) misc[M_MASK + (done & (kMaskRing - 1))] = static_cast<int>(groups);
          }
          // (V's rows past the sequence's end are cleared before its tile counts as there)
          const uint32_t there = bar(!kF16 && !is_k && t == tail ? static_cast<int>(B_VLAND) : full + sl);
          if (lane == 0) mbar_arrive_expect_tx(there, kF4 ? C::kCodeBytes : C::kItemBytes);
          __syncwarp();
          if constexpr (kF4) {
            // scales by cp.async, a lane those of rows 2 l, 2 l + 1 and of 64 on; 0 past the sequence's end and without a page (a
            // box of TMA would bring 128 bytes of a page of 16, at about 90 clocks of this warp: ragged chunks 374 us)
            const KvScales& from = scales.at;
            const uint8_t* base = is_k ? from.k : from.v;
            const uint32_t to = sbase + C::kOffK + sl * C::kItemBytes + C::kCodeBytes + 16 * lane;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = 64 * h + 2 * lane, key = (tile0 + t) * kTile + r;
              const int p = __shfl_sync(0xffffffffu, page, r / page_rows);
              const bool there_is = p != a.num_pages;
              const int64_t off = static_cast<int64_t>(there_is ? p : 0) * from.page_stride + g * from.head_stride +
                                  8 * (key & ((1 << a.page_shift) - 1));
              cp_async_16(to + 512 * h, base + off, there_is ? 8 * min(max(kv - key, 0), 2) : 0);
            }
            cp_async_arrive_noinc(there);
          }
          if (lane < boxes) {
            const uint32_t dst = sbase + (is_k || kF4 ? C::kOffK : C::kOffV) + sl * C::kItemBytes;
            if constexpr (kF4) {
              tma_load_4d(dst + lane * page_rows * 64, tm, 0, row, page, g, there);
            } else if (kPaged && !kF8 && a.kv_wide != 0) {
              const int groups = a.kv_wide == 2 ? g << (a.page_shift - 3) : 0;
              tma_load_5d(dst + lane * page_rows * 256, tm, 0, 0, a.kv_wide == 1 ? 2 * g : 0, groups + (row >> 3), page,
                          there);
            } else {
              for (int h = 0; h < C::kHalves; ++h)
                tma_load_4d(dst + lane * page_rows * 128 + h * kTile * 128, tm, 64 * h, row, page, g, there);
            }
          }
          ++done;   // at once: a wait below may run out, and what was started is drained by this count
          if constexpr (kF4) {
            older[2] = older[1];
            older[1] = older[0];
            older[0] = item;
          }
          page = page_n;
          row = row_n;
          have = have_n;
          if (is_k && t == 0) {
            // Q once the products of the job before have read its place
            ok = with_tiles == 0 || wait_for<kPoll>(bar(B_QDONE), (with_tiles - 1) & 1, limit);
            if (!ok) break;
            if (lane == 0) {
              const int blocks = one ? 1 : 2;
              mbar_arrive_expect_tx(bar(B_Q), blocks * C::kHalves * tokens * a.group * 128);
              for (int i = 0; i < blocks; ++i)
                for (int h = 0; h < C::kHalves; ++h)
                  tma_load_3d(sbase + C::kOffQ + i * C::kQBytes + h * 128 * 128, &tm_q, 64 * h, g * a.group,
                              q0 + tok0 + i * tokens, bar(B_Q));
            }
            ++with_tiles;
          }
        }
        if (!ok) break;
        tile_base += tiles;
        // the ragged end lies in the last tile: clear V's rows past it
        if (!kF16 && !is_k && tail >= 0) {
          const int sl = (done - 1) % C::kVSlots;
          ok = wait_for<kPoll>(bar(B_VLAND), landed & 1, limit);
          if (!ok && !wait_drain(bar(B_VLAND), landed & 1, a.drain_limit_ns)) atomicExch(&a.status[1], W_T_DRAIN);
          ++landed;
          if (ok) {
            uint8_t* v = smem + C::kOffV + sl * C::kItemBytes;
            const bool wide = kPaged && a.kv_wide != 0;
            for (int p = (kv & (kTile - 1)) * 8 + lane; p < kTile * 8; p += 32) {
              uint8_t* at = v + (wide ? (p >> 6) * 2048 + (p & 63) * 16 : p * 16);   // 64 pieces an 8-row atom
              *reinterpret_cast<uint4*>(at) = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(at + (wide ? 1024 : kTile * 128)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_VFULL + sl));
        }
      }
      if (!ok) give_up(a, W_T_LOAD);
      if constexpr (kF4) cp_async_wait_all();
      // nothing that was started may still be writing shared memory when the CTA ends
      __syncwarp();
      if (lane == 0) {
        const int slots = is_k ? C::kKSlots : kF4 ? 1 : C::kVSlots, full = is_k ? B_KFULL : B_VFULL;
        bool quiet = with_tiles == 0 || wait_drain(bar(B_Q), (with_tiles - 1) & 1, a.drain_limit_ns);
        if constexpr (kF4) {           // (two warps' tiles in one ring: drained behind the last barrier)
          done = 0;
          for (int k = 0; k < 3; ++k) misc[M_LAST + (is_k ? 0 : 3) + k] = older[k];
        }
        for (int k = max(0, done - slots); k < done; ++k)
          quiet = wait_drain(bar(full + k % slots), (k / slots) & 1, a.drain_limit_ns) && quiet;
        if (!quiet) atomicExch(&a.status[1], W_T_DRAIN);
      }
    } else if (kF8 && warp >= 12) {
      // ================================================== V e4m3 -> f16 ===
      const int key = threadIdx.x - 32 * 12;               // this thread's row of every tile
      const int r8 = key & 7;
      int tile_base = 0;
      bool ok = true;
#pragma unroll 1
      for (int job = 0; ok; ++job) {
      volatile int* jw;
      ok = job_at(job, jw);
      if (!ok || jw[J_B] < 0) break;
      const int kv = jw[J_KV], tile0 = jw[J_TILE0], tiles = jw[J_TILES];
      job_read(job);
#pragma unroll 1
      for (int tl = 0; tl < tiles; ++tl) {
        const int t = tile_base + tl;
        const int sl = t % C::kVSlots;
        ok = wait_for<kPoll>(bar(B_VFULL + sl), (t / C::kVSlots) & 1, limit) &&
             (t < 2 || wait_for<kPoll>(bar(B_V16E0 + (t & 1)), ((t >> 1) - 1) & 1, limit));
        if (!ok) break;
        const uint8_t* src = smem + C::kOffV + sl * C::kItemBytes + key * 128;
        uint8_t* dst = smem + C::kOffV16 + (t & 1) * C::kWideBytes + key * 128;
        const bool in = (tile0 + tl) * kTile + key < kv;
#pragma unroll
        for (int half = 0; half < 2; ++half) {               // 64 dims
          uint4 w[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            w[c] = in ? *reinterpret_cast<const uint4*>(src + (((4 * half + c) ^ r8) << 4)) : make_uint4(0, 0, 0, 0);
          uint8_t* blk = dst + half * kTile * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t ws[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
            uint32_t h[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %2;\n  cvt.rn.f16x2.e4m3x2 %0, lo;\n"
                  "  cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
                  : "=r"(h[2 * k]), "=r"(h[2 * k + 1])
                  : "r"(ws[k]));
            }
            *reinterpret_cast<uint4*>(blk + (((2 * c) ^ r8) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
            *reinterpret_cast<uint4*>(blk + (((2 * c + 1) ^ r8) << 4)) = make_uint4(h[4], h[5], h[6], h[7]);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(B_V16F0 + (t & 1)));
          mbar_arrive(bar(B_VEMPTY + sl));
        }
      }
      tile_base += tiles;
      }
      if (!ok) give_up(a, W_T_CONVERT);
    } else if (kF4 && warp >= 12) {
      // ================================ Q bf16 -> f16; K and V codes x scales -> f16 ===
      // A thread is a row of Q, then a key of every tile. Q's rows are taken to f16 in place at a power of two of their own (f16_row_up) with
      // the sign of the scores' scale. A code times its scale is exact in f16.
      const int key = threadIdx.x - 32 * 12;
      const int r8 = key & 7, r4 = (key >> 1) & 3;
      const float sign = (a.descale_q ? *a.descale_q : 1.f) * (a.descale_k ? *a.descale_k : 1.f) * a.scale_log2;   // of the scores' scale
      int tile_base = 0, with_tiles = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = true;
#pragma unroll 1
      for (int job = 0; ok; ++job) {
      volatile int* jw;
      ok = job_at(job, jw);
      if (!ok || jw[J_B] < 0) break;
      const int tiles = jw[J_TILES], blocks = jw[J_ONE] != 0 ? 1 : 2;
      job_read(job);
      if (tiles == 0) continue;
      ok = wait_for<kPoll>(bar(B_Q), with_tiles & 1, limit);
      if (!ok) break;
#pragma unroll 1
      for (int i = 0; i < blocks; ++i) {
        uint8_t* q = smem + C::kOffQ + i * C::kQBytes + key * 128;
        uint32_t top = 0;
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          const uint4 v = *reinterpret_cast<const uint4*>(q + (c >> 3) * 128 * 128 + (((c & 7) ^ r8) << 4));
          const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max(ws[k] & 0x7fffu, (ws[k] >> 16) & 0x7fffu));
        }
        const int e = static_cast<int>(top >> 7);          // the largest element's exponent
        const float up = copysignf(f16_row_up(e), sign);
#pragma unroll 4
        for (int c = 0; c < 16; ++c) {
          uint4* at = reinterpret_cast<uint4*>(q + (c >> 3) * 128 * 128 + (((c & 7) ^ r8) << 4));
          const uint4 v = *at;
          const uint32_t ws[4] = {v.x, v.y, v.z, v.w};
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) h[k] = pack_f16x2(__uint_as_float(ws[k] << 16) * up, __uint_as_float(ws[k] & 0xffff0000u) * up);
          *at = make_uint4(h[0], h[1], h[2], h[3]);
        }
        reinterpret_cast<volatile float*>(smem + C::kOffRow)[256 * (with_tiles & 1) + 128 * i + key] = f16_row_down(e);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_Q16));
      ++with_tiles;
      // A tile's codes come to registers while the wait for a free place of its values runs: their slot is free at once.
      uint32_t w[4][4], sc[2];
      // item `it` of the job (the inverse of item_of)
      auto kind = [&](int it) { return it == 2 * tiles - 1 || (it > 0 && !(it & 1)); };   // V?
      auto tile_of = [&](int it) {
        return it == 2 * tiles - 1 ? tiles - 1 : it & 1 ? (it + 1) >> 1 : max((it >> 1) - 1, 0);
      };
      auto take = [&](int it) {
        ok = wait_for<kPoll>(bar(B_KFULL + slot), phase, limit);
        if (!ok) return;
        const uint32_t src = sbase + C::kOffK + slot * C::kItemBytes;
        lds64(src + C::kCodeBytes + key * 8, sc);
#pragma unroll
        for (int c = 0; c < 4; ++c) lds128((src + key * 64 + (r4 << 4)) ^ (c << 4), w[c]);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_KEMPTY + slot));
        slot = slot == C::kKSlots - 1 ? 0 : slot + 1;
        phase ^= slot == 0 ? 1u : 0u;
      };
      take(0);
#pragma unroll 1
      for (int it = 0; ok && it < 2 * tiles; ++it) {
        const bool is_v = kind(it);
        const int t = tile_base + tile_of(it);
        ok = t < 2 || wait_for<kPoll>(bar((is_v ? B_V16E0 : B_K16E0) + (t & 1)), ((t >> 1) - 1) & 1, limit);
        if (!ok) break;
        const uint32_t dst = sbase + (is_v ? C::kOffV16 : C::kOffK16) + (t & 1) * C::kWideBytes + key * 128 + (r8 << 4);
#pragma unroll
        for (int c = 0; c < 4; ++c) {                        // 32 dims, two scales
          const uint32_t two = f16x2_of_e4m3(sc[c >> 1] >> (16 * (c & 1)));
#pragma unroll
          for (int k = 0; k < 4; ++k) {                      // 8 dims: one piece of 16 bytes
            const uint32_t by = __byte_perm(two, 0, k < 2 ? 0x1010 : 0x3232);
            uint32_t h[4];
            f16_of_e2m1x8(w[c][k], h);
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = mul_f16x2(h[e], by);
            const int piece = 4 * c + k;
            sts128((dst ^ ((piece & 7) << 4)) + (piece >> 3) * kTile * 128, h);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar((is_v ? B_V16F0 : B_K16F0) + (t & 1)));
        if (it + 1 < 2 * tiles) take(it + 1);
      }
      tile_base += tiles;
      }
      if (!ok) give_up(a, W_T_CONVERT);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (kF4 && warp == 9 && lane == 0) {
    // each slot's last tile, of whichever warp loaded it (a warp's last three hold all of its own among the ring's last three)
    bool quiet = true;
    for (int sl = 0; sl < C::kKSlots; ++sl) {
      int last = -1;
      for (int k = 0; k < 6; ++k)
        if (misc[M_LAST + k] >= 0 && misc[M_LAST + k] % C::kKSlots == sl) last = max(last, misc[M_LAST + k]);
      if (last >= 0) quiet = wait_drain(bar(B_KFULL + sl), (last / C::kKSlots) & 1, a.drain_limit_ns) && quiet;
    }
    if (!quiet) atomicExch(&a.status[1], W_T_DRAIN);
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ combine --

// One warp per kHeads heads of a (token, KV head): M = max_s LSE_s, w_s = 2^(LSE_s -
// M), O = sum_s w_s O_s / sum_s w_s. Lane (32 / kHeads) h + s holds the LSE of head h and
// split s (mod 32 / kHeads), every lane four columns of each head, several splits in
// flight, the first ones beside the LSE. A row has two loads in a chain (with three, 8 e4m3
// sequences of 2,048 keys took 15.2 us, so 14.4), so many rows take four heads a warp
// (measured on 47 thousand rows of 3 splits: 31 -> 14 us), few rows one, to spread over
// the SMs (256 rows: 1.3 us less). A token whose job was not split is left alone.
template <int kHeads>
__global__ void __launch_bounds__(256, 2) attn_combine_kernel(const AttnArgs a, const int rows_per_slot) {
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  const int begin = a.cu_q[0], end = a.cu_q[a.batch];   // (a token's map is on its way before these are there)
  float amax = 0.f;
  constexpr int kLanes = 32 / kHeads;            // lanes of a head: splits looked at together
  constexpr int kFlight = kHeads == 1 ? 8 : 4;   // splits of a head in flight
  const int parts = (a.group + kHeads - 1) / kHeads;
  const int64_t per_token = static_cast<int64_t>(a.h_kv) * parts;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); item < a.total_q * per_token;
       item += static_cast<int64_t>(gridDim.x) * 8) {
    const int tok = static_cast<int>(item / per_token), rest = static_cast<int>(item - tok * per_token);
    const int g = rest / parts, h0 = (rest - g * parts) * kHeads;
    const int2 map = a.row_map[static_cast<int64_t>(tok) * a.h_kv + g];
    if (tok < begin || tok >= end) continue;
    const int S = map.y;
    // (a token of no job, which only offsets that decrease can leave, has no entry: nothing outside the partials is read)
    if (S < 1 || S > a.num_splits || map.x < 0 ||
        map.x + a.group > static_cast<int64_t>(a.max_slots) * rows_per_slot ||
        map.x + (S - 1ll) * rows_per_slot - a.part_gap + a.group > static_cast<int64_t>(a.max_slots) * rows_per_slot ||
        (S > 1 && map.x + rows_per_slot - a.part_gap < 0))
      continue;
    {
      // split s > 0 lies at the first one's place + s slots - part_gap rows
      const int64_t p0 = static_cast<int64_t>(map.x) + h0;
      auto row_of = [&](int s) { return p0 + static_cast<int64_t>(s) * rows_per_slot - (s > 0 ? a.part_gap : 0); };
      const int heads = min(kHeads, a.group - h0);
      const int hl = lane / kLanes, sl = lane & (kLanes - 1);
      auto lse_at = [&](int s0) {
        const int s = s0 + sl;
        return hl < heads && s < S ? a.lse_part[row_of(s) + hl] : -INFINITY;
      };
      float4 x[kHeads][kFlight];
      auto load = [&](int s0) {
#pragma unroll
        for (int h = 0; h < kHeads; ++h)
#pragma unroll
          for (int k = 0; k < kFlight; ++k) {
            x[h][k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (h < heads && s0 + k < S) x[h][k] = __ldcs(reinterpret_cast<const float4*>(a.o_part + (row_of(s0 + k) + h) * kD) + lane);
          }
      };
      load(0);   // beside the LSE (the row of an empty split holds zeros)
      const float first = lse_at(0);
      float M = first, z = 0.f;
      for (int s0 = kLanes; s0 < S; s0 += kLanes) M = fmaxf(M, lse_at(s0));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      float4 acc[kHeads];
#pragma unroll
      for (int h = 0; h < kHeads; ++h) acc[h] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = 0; s0 < S; s0 += kLanes) {
        const float l = s0 == 0 ? first : lse_at(s0);
        const float w = l == -INFINITY ? 0.f : exp2f(l - M);
        z += w;
        for (int s1 = 0; s1 < kLanes && s0 + s1 < S; s1 += kFlight) {
          if (s0 + s1 > 0) load(s0 + s1);
#pragma unroll
          for (int h = 0; h < kHeads; ++h)
#pragma unroll
            for (int k = 0; k < kFlight; ++k) {
              const float ws = __shfl_sync(0xffffffffu, w, kLanes * h + s1 + k);
              acc[h].x = fmaf(ws, x[h][k].x, acc[h].x);
              acc[h].y = fmaf(ws, x[h][k].y, acc[h].y);
              acc[h].z = fmaf(ws, x[h][k].z, acc[h].z);
              acc[h].w = fmaf(ws, x[h][k].w, acc[h].w);
            }
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
      const int64_t row0 = static_cast<int64_t>(tok) * a.h_q + g * a.group + h0;
      if (sl == 0 && hl < heads && a.lse_out != nullptr)
        a.lse_out[row0 + hl] = z == 0.f ? -INFINITY : M + log2f(z);   // (a NaN partial's weight, and so z, is NaN)
      const float inv_l = z == 0.f ? 0.f : 1.f / z;
#pragma unroll
      for (int h = 0; h < kHeads; ++h) {
        const float inv = __shfl_sync(0xffffffffu, inv_l, kLanes * h);
        if (h >= heads) continue;
        const float4 y = make_float4(acc[h].x * inv, acc[h].y * inv, acc[h].z * inv, acc[h].w * inv);
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
        const int64_t at = (row0 + h) * kD + 4 * lane;
        if (a.out_dtype == 0) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
        else if (a.out_dtype == 1)
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
        else
          *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + at) =
              pack_e4m3x4(y.x * a.inv_scale, y.y * a.inv_scale, y.z * a.inv_scale, y.w * a.inv_scale);
      }
    }
  }
  if (a.amax != nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (lane == 0 && amax > 0.f) atomicMax(reinterpret_cast<int*>(a.amax), __float_as_int(amax));
  }
}

}  // namespace

namespace {
template <int kType>
using TileKernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, AttnArgs, ScalesOf<kType>);
// [pages][polling waits]; bf16 takes no equal shares, and 4 bits are a form of pages
template <int kType>
constexpr TileKernel<kType> kTileKernels[3][2] = {{attn_tile_kernel<kType, 0, false>, attn_tile_kernel<kType, 0, true>},
                                                  {attn_tile_kernel<kType, 1, false>, attn_tile_kernel<kType, 1, true>},
                                                  {attn_tile_kernel<kType, 2, false>, attn_tile_kernel<kType, 2, true>}};
template <>
constexpr TileKernel<1> kTileKernels<1>[3][2] = {{attn_tile_kernel<1, 0, false>, attn_tile_kernel<1, 0, true>},
                                                 {attn_tile_kernel<1, 1, false>, attn_tile_kernel<1, 1, true>},
                                                 {nullptr, nullptr}};
template <>
constexpr TileKernel<4> kTileKernels<4>[3][2] = {{nullptr, nullptr},
                                                 {attn_tile_kernel<4, 1, false>, attn_tile_kernel<4, 1, true>},
                                                 {attn_tile_kernel<4, 2, false>, attn_tile_kernel<4, 2, true>}};

template <int kType>
cudaError_t prepare() {
  for (int k = 0; k < 6; ++k) {
    if (kTileKernels<kType>[k >> 1][k & 1] == nullptr) continue;
    const cudaError_t e = cudaFuncSetAttribute(kTileKernels<kType>[k >> 1][k & 1], cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Cfg<kType>::kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}
template <int kType>
cudaError_t launch(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a,
                   const ScalesOf<kType>& scales, int64_t grid, cudaStream_t stream) {
  const int pages = a.table == nullptr ? 0 : a.adaptive == kShares ? 2 : 1;
  const TileKernel<kType> kernel = kTileKernels<kType>[pages][a.wait_limit_ns < kSuspendNs];
  if (kernel == nullptr || grid < 1 || grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(kernel, static_cast<unsigned>(grid), Cfg<kType>::kThreads, Cfg<kType>::kSmem, stream, tm_q, tm_k, tm_v, a, scales);
}
}  // namespace

cudaError_t prepare_attn_tile() {
  cudaError_t e = prepare<1>();
  if (e == cudaSuccess) e = prepare<2>();
  if (e == cudaSuccess) e = prepare<4>();
  return e;
}

cudaError_t launch_attn_tile(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                             const AttnArgs& a, int dtype, int64_t grid, cudaStream_t stream) {
  if (dtype == 2) return launch<2>(tm_q, tm_k, tm_v, a, {}, grid, stream);
  return launch<1>(tm_q, tm_k, tm_v, a, {}, grid, stream);
}

cudaError_t launch_attn_tile4(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a,
                              const KvScales& scales, int64_t grid, cudaStream_t stream) {
  return launch<4>(tm_q, tm_k, tm_v, a, {scales}, grid, stream);
}

cudaError_t launch_attn_combine(const AttnArgs& a, int rows_per_slot, cudaStream_t stream) {
  // one head a warp while the rows fit four warps of every scheduler
  const int64_t rows = static_cast<int64_t>(a.total_q) * a.h_q;
  const bool many = rows > 16ll * a.num_sms && a.group > 1;
  const int heads = many ? 4 : 1;
  const int64_t blocks = (static_cast<int64_t>(a.total_q) * a.h_kv * ((a.group + heads - 1) / heads) + 7) / 8;
  const int64_t most = 2ll * a.num_sms;
  return launch_pdl(many ? attn_combine_kernel<4> : attn_combine_kernel<1>, static_cast<unsigned>(blocks < most ? blocks : most),
                    256, 0, stream, a, rows_per_slot);
}

}  // namespace skv
