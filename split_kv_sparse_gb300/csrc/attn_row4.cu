// Attention of few query rows (at most 8 or 16: the tokens x the heads of one group) over a paged cache in 4 bits: decode.
// A key's K and V are 144 bytes a KV head, so at the rate of HBM an SM has to widen and multiply four fifths more
// keys than with e4m3: the instructions of a key bound the kernel beside the bytes. Both products are therefore taken
// the other way round than in the kernel of wider types, S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16, with 16 keys
// or dims as M and 8 query rows as N: K and V are widened once, straight into the registers of the A operand, and a
// group of 4 or 8 heads wastes half as many products as with 16 rows as M.
//
// Two CTAs an SM, each with four warps that compute and four that load: every computing warp walks key blocks (64 keys, every
// fourth of a job's) of its own with a running maximum and a sum of its own, merged at a job's end; a loading warp fills
// its ring by TMA, page by page, ahead into the next job. Equal shares of the batch's key tiles (AttnShares). Back-to-back calls: 4 x 100,000 to
// 131,072 keys, 64 / 8 heads, 99 us, 5.3 TB/s; 96 x 100 to 12,000, 32 / 8 heads, pages of 16, 142 us, 4.7 TB/s.
//
// Widening: a byte of two e2m1 codes is one conversion to an f16 pair, times its e4m3 scale in f16: exact (6
// significant bits, 2^-10 to 2688). The order of the contracted dims of S is free as long as Q has the same, so a lane takes
// 32 consecutive dims of a key (16 bytes: one load); for O a lane has 16 dims of four keys, and a pair of one dim of two
// keys is made by putting their codes into one byte before the conversion. Keys are taken in the order kPerm within
// eight, which keeps the loads of K and of V free of bank conflicts under the 64-byte swizzle.
// Q is held in f16 at a power of two of its row (f16_row_up).
#include "attn_common.cuh"
#include "quant.cuh"

namespace skv {
namespace {

constexpr int kD = kAttnDim;
constexpr int kTile = kAttnKeyTile;
constexpr int kWarps = 4;                               // that compute; as many load
constexpr int kThreads = 64 * kWarps;
constexpr int kStages = 3;
constexpr int kBlock = 64;                              // keys of a block
constexpr int kTiles = kBlock / 16;
constexpr int kCodes = kBlock * kD / 2;                 // bytes of its K or V codes
constexpr int kScales = kBlock * 8;
constexpr int kOffV = kCodes, kOffKs = 2 * kCodes, kOffVs = kOffKs + kScales;
constexpr int kStageBytes = 2 * (kCodes + kScales);
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kOffFull = kWarps * kWarpBytes;           // barriers [kWarps][kStages]: a block is there; its place is free
constexpr int kOffEmpty = kOffFull + kWarps * kStages * 8;
constexpr int kOffHave = kOffEmpty + kWarps * kStages * 8;   // int [kWarps][kStages]: a bit for each box that has a page
constexpr int kOffStats = kOffHave + kWarps * kStages * 8;   // float2 [kWarps][16]: m, l
constexpr int kOffAbort = kOffStats + kWarps * 16 * 8;
constexpr int kOffStage = kOffAbort + 16;               // int [kWarps]: the stage that holds a warp's result
constexpr int kSmem = kOffStage + 16 + 1024;
static_assert(16 * kD * 4 <= kStageBytes, "a warp's result goes through one stage");
static_assert(kRowCtasPerSm * (kSmem + 1024) <= 233472, "two CTAs an SM");
// Registers of a thread that loads, and that computes: 256 of two threads of a launch (jobs of 8 rows, 4 x 100,000 to 131,072 keys,
// 64 / 8 heads: 40 + 216 108.4 us, 56 + 200 105.2, 72 + 184 102.7, 88 + 168 103.5; of 16 rows, 32 x 3 tokens over 4,096 to 8,192 keys, 32 / 8
// heads: 40 + 216 75.7, 48 + 208 77.0, 56 + 200 77.7, 72 + 184 83.5). With 16 rows the compiler spills all the same (448 bytes of stores, 376
// of loads; none with 8), and e4m3 pages of the same lengths are quicker, 71.3 us.
template <int kN>
constexpr int kLoadRegs = kN == 1 ? 72 : 40;
template <int kN>
constexpr int kRegs = 256 - kLoadRegs<kN>;
// A piece's start and end, in units of an equal share (256 keys; 96 sequences of 100 to 12,000 keys: 0 150.6 us, 1 148.4, 2 145.1, 3 146.4).
constexpr int kRowHead = 2;

enum : uint32_t { W_R_FULL = 301, W_R_DRAIN, W_R_EMPTY };

// Row i of a tile's eight is key kPerm(i) = 0, 3, 1, 2, 4, 7, 5, 6.
__device__ __forceinline__ int perm8(int i) { return static_cast<int>((0x65742130u >> (4 * i)) & 7u); }

__device__ __forceinline__ void mma_f16_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// kN: query rows of a job in eights.
template <int kN, bool kPoll>
__global__ void __launch_bounds__(kThreads, kRowCtasPerSm)
    attn_row4_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ CUtensorMap tm_ks, const __grid_constant__ CUtensorMap tm_vs, const AttnArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane >> 2, q4 = lane & 3;
  auto full = [&](int w, int st) -> uint32_t { return sbase + kOffFull + (w * kStages + st) * 8; };
  auto empty = [&](int w, int st) -> uint32_t { return sbase + kOffEmpty + (w * kStages + st) * 8; };
  volatile int* have = reinterpret_cast<volatile int*>(smem + kOffHave);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  if (threadIdx.x < kWarps * kStages) {
    for (int k = 0; k < 2; ++k) mbar_init(sbase + kOffFull + 8 * (threadIdx.x + k * kWarps * kStages), 1);
    if (threadIdx.x == 0) *abort_flag = 0;
    mbar_init_fence();
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
  const uint32_t limit = wait_limit(a);
  // a piece's blocks of keys: up to the last token's keys
  auto blocks_of = [&](const AttnPiece& p, const AttnSeq& seq) {
    const int key0 = p.tile0 * kTile;
    const int end = static_cast<int>(min(key0 + static_cast<int64_t>(p.tiles) * kTile,
                                         static_cast<int64_t>(seq.kv - seq.sq + min((p.j + 1) * tokens, seq.sq))));
    return end > key0 ? (end - key0 + kBlock - 1) / kBlock : 0;
  };

  if (warp >= kWarps) {
    // ============================================================ loads ===
    regs_dec<kLoadRegs<kN>>();
    const int w = warp - kWarps;                           // whose
    const uint32_t ring = sbase + w * kWarpBytes;
    // A lane loads a box (a page's rows, or 64 of one) of K's or V's codes or scales. Rows without a page become zeros.
    const int box_shift = min(a.page_shift, 6);
    const int boxes = kBlock >> box_shift;                 // of a block: 1, 2 or 4
    const int box = lane & (boxes - 1), which = lane >> (6 - box_shift);
    const bool is_v = which & 1, is_scale = which >= 2;
    const uint32_t dst = ring + (is_scale ? (is_v ? kOffVs : kOffKs) + (box << (box_shift + 3)) : (is_v ? kOffV : 0) + (box << (box_shift + 6)));
    const CUtensorMap* tm = is_scale ? (is_v ? &tm_vs : &tm_ks) : (is_v ? &tm_v : &tm_k);
    const int row_mask = (1 << a.page_shift) - 1;
    if (lane < 4) tma_prefetch_desc(lane == 0 ? &tm_k : lane == 1 ? &tm_v : lane == 2 ? &tm_ks : &tm_vs);
    int used = 0, st = 0;                                  // blocks so far, the next one's stage and parity
    uint32_t parity = 0;
    bool ok = true;
#pragma unroll 1
    while (ok && next.b >= 0) {
      const AttnSeq seq = attn_seq(a, next.b);
      const int key0 = next.tile0 * kTile + w * kBlock, all = blocks_of(next, seq);
      const int cnt = all > w ? (all - w + kWarps - 1) / kWarps : 0;   // this warp's blocks
      const int32_t* table = a.table + static_cast<size_t>(next.b) * a.table_width;
      const int head = next.g;
      // lane's box of a group of 32: the page, or num_pages (zeros) where there is none
      auto lookup = [&](int first) {
        const int e = first + lane;
        const int key = key0 + kWarps * kBlock * (e / boxes) + ((e & (boxes - 1)) << box_shift);
        int page = a.num_pages;
        if (e < cnt * boxes && key < seq.kv) {
          const int p = table[key >> a.page_shift];
          if (p >= 0 && p < a.num_pages) page = p;
        }
        return page;
      };
      int group0 = 0, pages = lookup(0), pages_next = lookup(32);
      next.b = -1;
      if (a.adaptive == kShares) next = shares.next(a);
#pragma unroll 1
      for (int at = 0; at < cnt; ++at) {
        if (at * boxes - group0 >= 32) {
          pages = pages_next;
          group0 += 32;
          pages_next = lookup(group0 + 32);
        }
        ok = used < kStages || wait_for<kPoll>(empty(w, st), parity ^ 1u, limit);
        if (!ok) break;
        ++used;
        const int page = __shfl_sync(0xffffffffu, pages, (at * boxes - group0 + box) & 31);
        const unsigned got = __ballot_sync(0xffffffffu, lane < boxes && page != a.num_pages);
        if (lane == 0) {
          have[w * kStages + st] = static_cast<int>(got);
          mbar_arrive_expect_tx(full(w, st), kStageBytes);
        }
        __syncwarp();
        if (lane < 4 * boxes) {
          const int row = (key0 + kWarps * kBlock * at + (box << box_shift)) & row_mask;
          tma_load_4d(dst + st * kStageBytes, tm, is_scale ? 2 * row : 0, is_scale ? 0 : row, page, head, full(w, st));
        }
        st = st == kStages - 1 ? 0 : st + 1;
        parity ^= st == 0 ? 1u : 0u;
      }
    }
    if (!ok) give_up(a, W_R_EMPTY);
    // what was started may not be writing shared memory any more when the CTA ends
    bool quiet = true;
    for (int k = max(0, used - kStages); k < used; ++k)
      quiet = wait_drain(full(w, k % kStages), (k / kStages) & 1, a.drain_limit_ns) && quiet;
    if (!quiet && lane == 0) atomicExch(&a.status[1], W_R_DRAIN);
    return;
  }

  // ============================================================ products ===
  regs_inc<kRegs<kN>>();
  const int box_shift = min(a.page_shift, 6), boxes = kBlock >> box_shift;
  const uint32_t ring = sbase + warp * kWarpBytes;
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
  int loaded = 0;                     // blocks of earlier pieces
  int st = 0;                         // the next block's stage, its barrier's parity, whether it was seen there
  uint32_t parity = 0;
  bool seen = false;
  AttnSeq seq_next = {0, 0, 0, 0};
  if (next.b >= 0) seq_next = attn_seq(a, next.b);
#pragma unroll 1
  while (next.b >= 0) {
  const AttnPiece job = next;
  const AttnSeq seq = seq_next;
  const int tok0 = job.j * tokens;
  const int ntok = min(tokens, seq.sq - tok0);
  const int first_key = job.tile0 * kTile + warp * kBlock;
  const int all = blocks_of(job, seq), cnt = all > warp ? (all - warp + kWarps - 1) / kWarps : 0;   // this warp's
  next.b = -1;
  if (a.adaptive == kShares) next = shares.next(a);
  if (next.b >= 0) seq_next = attn_seq(a, next.b);

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
    const float up = f16_row_up(e);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      qf[n][i >> 1][i & 1] = pack_f16x2(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
    const float down = f16_row_down(e);
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
  bool ok = true;
  int nb = 0;
#pragma unroll 1
  for (; nb < cnt; ++nb) {
    if (!seen && !wait_for<kPoll>(full(warp, st), parity, limit)) {
      ok = false;
      break;
    }
    const uint32_t stage = ring + st * kStageBytes;
    const int key = first_key + kWarps * kBlock * nb;
    const uint32_t there = static_cast<uint32_t>(have[warp * kStages + st]);   // a bit a box
    float s[kTiles][kN][4];
#pragma unroll
    for (int t0 = 0; t0 < kTiles; t0 += 2) {               // two tiles side by side: their products do not wait for one another
      uint32_t w[2][2][4], sc2[2][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = t0 + e;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[t][n][k] = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          lds128(stage + k_off + t * 1024 + h * 512, w[e][h]);
          sc2[e][h] = f16x2_of_e4m3(lds16(stage + ks_off + t * 128 + h * 64));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t x[2][2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t by = __byte_perm(sc2[e][h], 0, j < 2 ? 0x1010 : 0x3232);
            f16_of_e2m1x8(w[e][h][j], x[e][h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[e][h][i] = mul_f16x2(x[e][h][i], by);
          }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < kN; ++n)
              mma_f16_16x8(s[t0 + e][n], x[e][0][2 * i], x[e][1][2 * i], x[e][0][2 * i + 1], x[e][1][2 * i + 1], qf[n][2 * j + i][0],
                           qf[n][2 * j + i][1]);
      }
    }
    if (!raw_ok) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[t][n][k] *= esc[n][k & 1];
    }
    if (key + kBlock - 1 > lim_min || there != (1u << boxes) - 1u) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int at_key = key + 16 * t + k_row + 8 * (k >> 1);
            if (at_key > lim[n][k & 1] || !((there >> ((16 * t) >> box_shift)) & 1u)) s[t][n][k] = -INFINITY;
          }
    }
    // a row's keys lie over the eight lanes of a column: their maximum is needed only where a lane's asks for a new reference
    float mx[kN][2];
    bool need = false;
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = fmaxf(s[0][n][k], s[0][n][k + 2]);
#pragma unroll
        for (int t = 1; t < kTiles; ++t) x = fmax3(x, s[t][n][k], s[t][n][k + 2]);
        mx[n][k] = raw_ok ? x * esc[n][k] : x;
        need = need || new_reference<true>(mx[n][k], m[n][k]);
      }
    if (__any_sync(0xffffffffu, need)) {
#pragma unroll
      for (int n = 0; n < kN; ++n)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float x = mx[n][k];
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          if (new_reference<true>(x, m[n][k])) {
            const float al = m[n][k] == -INFINITY ? 0.f : ex2_approx(m[n][k] - x);
            m[n][k] = x;
            l[n][k] *= al;
            lc[n][k] *= al;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i][n][k] *= al;
              o[i][n][k + 2] *= al;
            }
          }
        }
    }
    uint32_t pf[kTiles][kN][2];                                 // P^T: keys 2 q4, 2 q4 + 1 (and + 8) of row quad
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const float nm0 = minus_reference<true>(m[n][0]), nm1 = minus_reference<true>(m[n][1]);
      const float e0 = raw_ok ? esc[n][0] : 1.f, e1 = raw_ok ? esc[n][1] : 1.f;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
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
    const int st_next = st == kStages - 1 ? 0 : st + 1;
    const uint32_t parity_next = parity ^ (st_next == 0 ? 1u : 0u);
    seen = nb + 1 < cnt && mbar_test_wait(full(warp, st_next), parity_next);
    if (seq.kv - key < kBlock) {
      // rows past the sequence's end: 0 * NaN would reach the result, and only a scale can be NaN
      for (int r = seq.kv - key + lane; r < kBlock; r += 32)
        *reinterpret_cast<uint2*>(smem + warp * kWarpBytes + st * kStageBytes + kOffVs + 8 * r) = make_uint2(0, 0);
      fence_proxy_async_smem();        // (a later load writes the stage)
      __syncwarp();
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
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
    if (lane == 0 && nb + 1 < cnt) mbar_arrive(empty(warp, st));   // (the last one holds the warp's result first)
    st = st_next;
    parity = parity_next;
  }
  if (!ok) {
    if (lane == 0) *abort_flag = 1;   // read at the merge
    give_up(a, W_R_FULL);
  }

  // ---- merge of the four warps' results
  // A warp's rows x 128 fp32 go through the stage of its last block. Row r's 16-byte piece c lies at c ^ c / 8 ^ r / 2 within its
  // eight: no bank conflicts on either side.
  auto piece_at = [](int row, int c) { return row * 512 + (((c & 24) | ((c ^ (c >> 3) ^ ((row >> 1) & 3)) & 7)) << 4); };
  volatile int* stage_of = reinterpret_cast<volatile int*>(smem + kOffStage);
  const int last = (loaded + max(cnt, 1) - 1) % kStages;
  uint8_t* mine = smem + warp * kWarpBytes + last * kStageBytes;
  if (lane == 0) stage_of[warp] = cnt > 0 ? last : -1;
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
      if (cnt > 0) {
#pragma unroll
        for (int h = 0; h < 2; ++h)                        // dims 16 quad + 8 h ..
#pragma unroll
          for (int j = 0; j < 2; ++j)
            *reinterpret_cast<float4*>(mine + piece_at(r, 4 * quad + 2 * h + j)) =
                make_float4(o[4 * j][n][2 * h + k], o[4 * j + 1][n][2 * h + k], o[4 * j + 2][n][2 * h + k], o[4 * j + 3][n][2 * h + k]);
      }
      if (quad == 0) stats[warp * 16 + r] = make_float2(m[n][k], z);
    }
  named_bar_sync(1, 32 * kWarps);
  if (*abort_flag) return;
  const bool part = job.slot >= 0;
  float amax = 0.f;
#pragma unroll 1
  for (int row = warp; row < 8 * kN; row += kWarps) {     // a warp a row, four dims a lane
    const int rt = row / a.group;
    if (rt >= ntok) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, stats[w * 16 + row].x);
    float tot = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (stage_of[w] < 0) continue;
      const float2 st = stats[w * 16 + row];
      const float f = st.x == -INFINITY ? 0.f : ex2_approx(st.x - M);
      tot = fmaf(st.y, f, tot);
      const float4 v = *reinterpret_cast<const float4*>(smem + w * kWarpBytes + stage_of[w] * kStageBytes + piece_at(row, lane));
      y.x = fmaf(v.x, f, y.x);
      y.y = fmaf(v.y, f, y.y);
      y.z = fmaf(v.z, f, y.z);
      y.w = fmaf(v.w, f, y.w);
    }
    const bool some = tot > 0.f || tot != tot;
    const float inv = some ? dv / tot : 0.f;
    const float lse = some ? lse_of<true>(M, tot) : -INFINITY;
    y = some ? make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv) : make_float4(0.f, 0.f, 0.f, 0.f);
    amax = fmaxf(amax, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
    const int64_t orow = static_cast<int64_t>(seq.q0 + tok0 + rt) * a.h_q + job.g * a.group + (row - rt * a.group);
    const int64_t prow = static_cast<int64_t>(job.slot) * kRowRows + row;
    const int64_t to = (part ? prow : orow) * kD + 4 * lane;
    if (part) *reinterpret_cast<float4*>(a.o_part + to) = y;
    else if (a.out_dtype == 0) *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = y;
    else if (a.out_dtype == 1)
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + to) = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    else
      *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.out) + to) =
          pack_e4m3x4(y.x * a.inv_scale, y.y * a.inv_scale, y.z * a.inv_scale, y.w * a.inv_scale);
    if (lane == 0) {
      if (part) a.lse_part[prow] = lse;
      else if (a.lse_out != nullptr) a.lse_out[orow] = lse;
      if (a.row_map != nullptr && (job.S > 0 || !part) && row == rt * a.group)
        a.row_map[static_cast<int64_t>(seq.q0 + tok0 + rt) * a.h_kv + job.g] = make_int2(static_cast<int>(prow), part ? job.S : 0);
    }
  }
  if (!part && a.amax != nullptr) {
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
    if (lane == 0) atomicMax(reinterpret_cast<int*>(a.amax), __float_as_int(amax));
  }
  if (next.b < 0) break;
  fence_proxy_async_smem();            // the stages were read and written here; TMA writes them next
  named_bar_sync(1, 32 * kWarps);      // the results have been read
  if (lane == 0 && cnt > 0) mbar_arrive(empty(warp, last));
  loaded += cnt;
  }
}

using Row4Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, AttnArgs);
// [rows / 8 - 1][polling waits]
constexpr Row4Kernel kRow4Kernels[2][2] = {{attn_row4_kernel<1, false>, attn_row4_kernel<1, true>},
                                           {attn_row4_kernel<2, false>, attn_row4_kernel<2, true>}};

}  // namespace

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
  return launch_pdl(kRow4Kernels[rows > 8][a.wait_limit_ns < kSuspendNs], static_cast<unsigned>(grid), kThreads, kSmem, stream, tm_k,
                    tm_v, tm_ks, tm_vs, a);
}

}  // namespace skv
