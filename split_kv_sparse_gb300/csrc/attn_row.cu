// Attention of few query rows (at most 16: the tokens x the heads of one group) over
// a paged cache: decode. Every K and V element is read once and used for 16 rows, so
// HBM bounds it, and the kernel is built around bytes in flight (196 KB an SM): four warps a CTA,
// two CTAs an SM; each warp walks key blocks of its own (every fourth of a job's), with a
// ring of its own that TMA fills page by page, and its own running maximum and sum, so no
// warp waits for another until the four results of a job are merged. Where the plan forces
// no split count, a CTA takes an equal share of the batch's work (AttnShares): pieces of one or more
// jobs, one after the other, the loads running ahead into the next. Measured with 32 query and 8
// KV heads: 96 sequences of 100 to 12,000 bf16 keys 339 us (6.4 TB/s; with one job a CTA a tenth more),
// 256 of 500 95 us, 8 of 65,536 e4m3 keys 166 us (6.5 TB/s), 8 of 1,024 to 16,384 34.5 us.
//
// The products are mma.sync with the 16 rows as M: a tcgen05 tile has at least 64, and
// the tensor work of 16 rows is far below either pipe's rate. bf16: blocks of 16 keys
// (8 KB of K and V), P as a bf16 pair hi + lo (two products: an error of 2^-16, where one bf16
// costs 2^-8); e4m3: blocks of 32 keys (8 KB), Q K^T on the codes, V converted to f16
// (exact) in registers and P in f16. e4m3 V needs no transpose: lane 4 g + q loads the 16
// dims 16 g .. 16 g + 15 of keys 2 q, 2 q + 1 (and + 8), and MMA i of 16 takes dim 16 g + i
// as its column g, so each lane ends with 32 consecutive dims of its rows.
#include "attn_common.cuh"

namespace skv {
namespace {

constexpr int kD = kAttnDim;
constexpr int kTile = kAttnKeyTile;
constexpr int kWarps = 4;
constexpr int kStages = 3;
constexpr int kStageBytes = 8192;                       // K then V of one block
constexpr int kWarpBytes = kStages * kStageBytes;
constexpr int kOffBars = kWarps * kWarpBytes;
constexpr int kOffStats = kOffBars + kWarps * kStages * 8;   // float2 [kWarps][16]: m, l
constexpr int kOffAbort = kOffStats + kWarps * 16 * 8;
constexpr int kOffStage = kOffAbort + 16;               // int [kWarps]: the stage that holds a warp's result
constexpr int kSmem = kOffStage + 16 + 1024;
static_assert(16 * kD * 4 <= kStageBytes, "a warp's result goes through one stage");
// A piece's start and end, in key tiles of an equal share (128 sequences of 2,048 e4m3 keys: 0 97.9 us, 1 97.8, 2
// 96.7; 8 of 8,192: 33.0, 32.8, 32.4).
constexpr int kRowHead = 2;

enum : uint32_t { W_R_FULL = 301, W_R_DRAIN };

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16s(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes (the low half of w) as an f16 pair.
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t w, bool high) {
  uint32_t h;
  if (high)
    asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(h) : "r"(w));
  else
    asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(w));
  return h;
}

template <bool kF8, bool kPoll>
__global__ void __launch_bounds__(kWarps * 32, kRowCtasPerSm)
    attn_row_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const AttnArgs a,
                    const int box_rows) {
  constexpr int kBlock = kF8 ? 32 : 16;                  // keys of a block
  constexpr int kNt = kBlock / 8;                        // 8-key column groups of its scores
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
  }
  if (warp == 1) attn_prefetch(a, lane);
  __syncthreads();
  grid_dependency_wait();

  const int tokens = kRowRows / a.group;
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
  const int boxes = kBlock / box_rows;                   // pages (or parts of one) of a block: 1 or 2
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
    const int key = x.key + kWarps * kBlock * (e / boxes) + (e % boxes) * box_rows;
    int page = a.num_pages;
    if (e < x.cnt * boxes && key < x.kv) {
      const int p = x.table[key >> a.page_shift];
      if (p >= 0 && p < a.num_pages) page = p;
    }
    return page;
  };
  int loaded = 0, issued = 0;         // blocks of earlier pieces; blocks whose loads were started
  uint32_t have = 0;                  // two bits a block in flight: its boxes' pages exist
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
      const int page = __shfl_sync(0xffffffffu, pages, (at * boxes - group0 + (lane & (boxes - 1))) & 31);
      const unsigned got = __ballot_sync(0xffffffffu, lane < boxes && page != a.num_pages);
      const uint32_t two = boxes == 1 ? (got & 1u) * 3u : (got & 3u);
      have = (have & ~(3u << (2 * (issued & 7)))) | (two << (2 * (issued & 7)));
      const int st = issued % kStages;
      if (lane == 0) mbar_arrive_expect_tx(bar(st), kStageBytes);
      __syncwarp();
      if (lane < boxes) {
        const int key = in.key + kWarps * kBlock * at + lane * box_rows;
        const int row = key & ((1 << a.page_shift) - 1);
        const uint32_t dst = ring + st * kStageBytes + lane * box_rows * 128;
        tma_load_4d(dst, &tm_k, 0, row, page, in.g, bar(st));
        if constexpr (!kF8) tma_load_4d(dst + kBlock * 128, &tm_k, 64, row, page, in.g, bar(st));
        tma_load_4d(dst + kStageBytes / 2, &tm_v, 0, row, page, in.g, bar(st));
        if constexpr (!kF8) tma_load_4d(dst + kStageBytes / 2 + kBlock * 128, &tm_v, 64, row, page, in.g, bar(st));
      }
      ++at;
      ++issued;
    }
  };
  auto drain = [&](int seen) {        // what was started may not be writing shared memory any more when the CTA ends
    bool done = true;
    for (int k = seen; k < issued; ++k)
      done = wait_drain(bar(k % kStages), (k / kStages) & 1, a.drain_limit_ns) && done;
    if (!done && lane == 0) atomicExch(&a.status[1], W_R_DRAIN);
  };
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

  // ---- Q fragments: rows quad and quad + 8 (token r / group, head r % group)
  constexpr int kKs = kF8 ? 4 : 8;                       // MMA steps over the 128 dims
  uint32_t qf[kKs][4];
  int lim[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = quad + 8 * h;
    const int t = r / a.group;
    const bool live = t < ntok;
    lim[h] = live ? seq.kv - seq.sq + tok0 + t : -1;
    const int64_t off = static_cast<int64_t>(seq.q0 + tok0 + t) * a.q_ts +
                        static_cast<int64_t>(job.g * a.group + (r - t * a.group)) * a.q_hs;
#pragma unroll
    for (int k = 0; k < kKs; ++k) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {                      // 16-byte half of the step's dims
        uint32_t v = 0;
        if (live) {
          if constexpr (kF8) v = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.q) + off + 32 * k + 16 * p + 4 * q4);
          else v = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(a.q) + off + 16 * k + 8 * p + 2 * q4);
        }
        qf[k][2 * p + h] = v;
      }
    }
  }
  const float dq = a.descale_q ? *a.descale_q : 1.f, dk = a.descale_k ? *a.descale_k : 1.f,
              dv = a.descale_v ? *a.descale_v : 1.f;
  const float sc = dq * dk * a.scale_log2;
  const bool raw_ok = sc > 0.f;
  const float esc = raw_ok ? sc : 1.f;
  const int lim_min = min(__reduce_min_sync(0xffffffffu, min(lim[0] < 0 ? 0x7fffffff : lim[0], lim[1] < 0 ? 0x7fffffff : lim[1])),
                          seq.kv - 1);                   // keys up to here are seen by every live row

  float o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, lc[2] = {0.f, 0.f};
  const uint32_t limit = wait_limit(a);
  bool ok = true;
  int n = 0;
#pragma unroll 1
  for (; n < cnt; ++n) {
    load_ahead(loaded + n);
    const int st = (loaded + n) % kStages;
    if (!wait_for<kPoll>(bar(st), ((loaded + n) / kStages) & 1, limit)) {
      ok = false;
      break;
    }
    const uint32_t ks = ring + st * kStageBytes, vs = ks + kStageBytes / 2;
    const int key = first_key + kWarps * kBlock * n;
    if (key + kBlock > seq.kv) {
      // rows past the sequence's end: 0 * NaN would reach the result
      uint8_t* v = smem + warp * kWarpBytes + st * kStageBytes + kStageBytes / 2;
      for (int p = (seq.kv - key) * 8 + lane; p < kBlock * 8; p += 32) {
        *reinterpret_cast<uint4*>(v + p * 16) = make_uint4(0, 0, 0, 0);
        if constexpr (!kF8) *reinterpret_cast<uint4*>(v + kBlock * 128 + p * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();        // (a later load writes the stage)
      __syncwarp();
    }
    float s[kNt][4];
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
    {
      // matrices of an x4: (keys 0-7, piece 2k), (keys 0-7, piece 2k + 1), (keys 8-15, ...) x 2
      const int mr = (lane & 7) + ((lane >> 4) << 3), mp = (lane >> 3) & 1;
#pragma unroll
      for (int k = 0; k < kKs; ++k) {
#pragma unroll
        for (int h = 0; h < kBlock / 16; ++h) {
          const int row = 16 * h + mr;
          const int piece = 2 * k + mp;
          const uint32_t addr = ks + (kF8 ? 0 : (piece >> 3) * kBlock * 128) + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
          uint32_t b[4];
          ldmatrix_x4(addr, b);
          if constexpr (kF8) {
            mma_e4m3(s[2 * h], qf[k], b[0], b[1]);
            mma_e4m3(s[2 * h + 1], qf[k], b[2], b[3]);
          } else {
            mma_bf16(s[2 * h], qf[k], b[0], b[1]);
            mma_bf16(s[2 * h + 1], qf[k], b[2], b[3]);
          }
        }
      }
    }
    if (!raw_ok) {
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] *= sc;
    }
    const uint32_t two = (have >> (2 * ((loaded + n) & 7))) & 3u;
    if (key + kBlock - 1 > lim_min || two != 3u) {
#pragma unroll
      for (int i = 0; i < kNt; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int at = 8 * i + 2 * q4 + (k & 1);
          const bool gone = boxes == 2 ? !((two >> (i >> 1)) & 1u) : two == 0u;
          if (key + at > lim[k >> 1] || gone) s[i][k] = -INFINITY;
        }
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int i = 0; i < kNt; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) mx[k >> 1] = fmaxf(mx[k >> 1], s[i][k]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
      mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2)) * esc;
    }
    const bool need0 = new_reference<kF8>(mx[0], m[0]), need1 = new_reference<kF8>(mx[1], m[1]);
    if (__any_sync(0xffffffffu, need0 || need1)) {
      float al[2] = {1.f, 1.f};
      if (need0) {
        al[0] = m[0] == -INFINITY ? 0.f : ex2_approx(m[0] - mx[0]);
        m[0] = mx[0];
      }
      if (need1) {
        al[1] = m[1] == -INFINITY ? 0.f : ex2_approx(m[1] - mx[1]);
        m[1] = mx[1];
      }
      l[0] *= al[0];
      l[1] *= al[1];
      lc[0] *= al[0];
      lc[1] *= al[1];
#pragma unroll
      for (int i = 0; i < 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][k] *= al[k >> 1];
    }
    const float nm0 = minus_reference<kF8>(m[0]), nm1 = minus_reference<kF8>(m[1]);
#pragma unroll
    for (int i = 0; i < kNt; ++i) {
#pragma unroll
      for (int k = 0; k < 4; ++k) s[i][k] = ex2_approx(fmaf(s[i][k], esc, k < 2 ? nm0 : nm1));
    }
    float more[2] = {s[0][0] + s[0][1], s[0][2] + s[0][3]};
#pragma unroll
    for (int i = 1; i < kNt; ++i) {
      more[0] += s[i][0] + s[i][1];
      more[1] += s[i][2] + s[i][3];
    }
    add_compensated(l[0], lc[0], more[0]);
    add_compensated(l[1], lc[1], more[1]);
    if constexpr (kF8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {                       // 16 keys
        uint32_t pf[4] = {pack_f16x2(s[2 * h][0], s[2 * h][1]), pack_f16x2(s[2 * h][2], s[2 * h][3]),
                          pack_f16x2(s[2 * h + 1][0], s[2 * h + 1][1]), pack_f16x2(s[2 * h + 1][2], s[2 * h + 1][3])};
        uint32_t w[4][4];                                 // keys 2 q4, + 1, + 8, + 9: dims 16 quad .. + 15
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * h + 2 * q4 + (e & 1) + 8 * (e >> 1);
          const uint32_t addr = vs + row * 128 + ((quad ^ (row & 7)) << 4);
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                       : "r"(addr));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo0 = __byte_perm(w[0][j], w[1][j], 0x5140), hi0 = __byte_perm(w[0][j], w[1][j], 0x7362);
          const uint32_t lo1 = __byte_perm(w[2][j], w[3][j], 0x5140), hi1 = __byte_perm(w[2][j], w[3][j], 0x7362);
          mma_f16s(o[4 * j], pf, f16x2_of_e4m3x2(lo0, false), f16x2_of_e4m3x2(lo1, false));
          mma_f16s(o[4 * j + 1], pf, f16x2_of_e4m3x2(lo0, true), f16x2_of_e4m3x2(lo1, true));
          mma_f16s(o[4 * j + 2], pf, f16x2_of_e4m3x2(hi0, false), f16x2_of_e4m3x2(hi1, false));
          mma_f16s(o[4 * j + 3], pf, f16x2_of_e4m3x2(hi0, true), f16x2_of_e4m3x2(hi1, true));
        }
      }
    } else {
      uint32_t ph[4], pl[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = s[e >> 1][2 * (e & 1)], x1 = s[e >> 1][2 * (e & 1) + 1];
        ph[e] = pack_bf16x2(x0, x1);
        pl[e] = pack_bf16x2(x0 - __uint_as_float(ph[e] << 16), x1 - __uint_as_float(ph[e] & 0xffff0000u));
      }
      // matrices of a transposing x4: (keys 0-7, piece 2i), (keys 8-15, piece 2i), then piece 2i + 1
      const int row = lane & 15, mp = lane >> 4;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int piece = 2 * i + mp;
        const uint32_t addr = vs + (piece >> 3) * kBlock * 128 + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
        uint32_t b[4];
        ldmatrix_x4_trans(addr, b);
        mma_bf16(o[2 * i], ph, b[0], b[1]);
        mma_bf16(o[2 * i + 1], ph, b[2], b[3]);
        mma_bf16(o[2 * i], pl, b[0], b[1]);
        mma_bf16(o[2 * i + 1], pl, b[2], b[3]);
      }
    }
    __syncwarp();                                          // every lane has read the stage
  }
  if (!ok) {
    if (lane == 0) *abort_flag = 1;   // read at the merge
    give_up(a, W_R_FULL);
    drain(loaded + n);
  }

  // ---- merge of the four warps' results
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  // A warp's 16 x 128 fp32 go through the stage that the next load will take (at most two are in flight now). Row r's
  // 16-byte piece c lies at c ^ c / 8 ^ 4 (r % 2) ^ r & 2 within its eight: no bank conflicts on either side.
  auto piece_at = [](int row, int c) { return row * 512 + (((c & 24) | ((c ^ (c >> 3) ^ ((row & 1) << 2) ^ (row & 2)) & 7)) << 4); };
  volatile int* stage_of = reinterpret_cast<volatile int*>(smem + kOffStage);
  uint8_t* mine = smem + warp * kWarpBytes + (issued % kStages) * kStageBytes;
  if (lane == 0) stage_of[warp] = issued % kStages;
  float2* stats = reinterpret_cast<float2*>(smem + kOffStats);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = quad + 8 * h;
    if constexpr (kF8) {
#pragma unroll
      for (int c = 0; c < 2; ++c)                          // dims 32 q4 + 16 c .. + 15
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *reinterpret_cast<float4*>(mine + piece_at(r, 8 * q4 + 4 * c + j)) =
              make_float4(o[4 * j][2 * h + c], o[4 * j + 1][2 * h + c], o[4 * j + 2][2 * h + c], o[4 * j + 3][2 * h + c]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float2*>(mine + piece_at(r, 2 * i + (q4 >> 1)) + 8 * (q4 & 1)) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
    }
    if (q4 == 0) stats[warp * 16 + quad + 8 * h] = make_float2(m[h], l[h]);
  }
  __syncthreads();
  if (*abort_flag) {
    if (ok) drain(loaded + cnt);
    return;
  }
  const int row = threadIdx.x >> 3, x0 = (threadIdx.x & 7) * 16;
  const int rt = row / a.group;
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
  const float lse = some ? lse_of<kF8>(M, tot) : -INFINITY;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    y[i] = some ? y[i] * inv : 0.f;
    amax = fmaxf(amax, fabsf(y[i]));
  }
  const bool live = rt < ntok;
  const bool part = job.slot >= 0;
  const int64_t orow = static_cast<int64_t>(seq.q0 + tok0 + rt) * a.h_q + job.g * a.group + (row - rt * a.group);
  const int64_t prow = static_cast<int64_t>(job.slot) * kRowRows + row;
  if (live) {
    if (part) store_row(a.o_part, 0, prow * kD + x0, y, 1.f);
    else store_row(a.out, a.out_dtype, orow * kD + x0, y, a.inv_scale);
    if (x0 == 0) {
      if (part) a.lse_part[prow] = lse;
      else if (a.lse_out != nullptr) a.lse_out[orow] = lse;
      if (a.row_map != nullptr && (job.S > 0 || !part) && row == rt * a.group)
        a.row_map[static_cast<int64_t>(seq.q0 + tok0 + rt) * a.h_kv + job.g] = make_int2(static_cast<int>(prow), part ? job.S : 0);
    }
  }
  if (!part && a.amax != nullptr) {
    if (!live) amax = 0.f;
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

}  // namespace

int attn_row_box(int dtype, int page_size) {
  const int block = dtype == 2 ? 32 : 16;
  return page_size < block ? page_size : block;
}

namespace {
using RowKernel = void (*)(CUtensorMap, CUtensorMap, AttnArgs, int);
// [e4m3][polling waits]
constexpr RowKernel kRowKernels[2][2] = {{attn_row_kernel<false, false>, attn_row_kernel<false, true>},
                                         {attn_row_kernel<true, false>, attn_row_kernel<true, true>}};
}  // namespace

cudaError_t prepare_attn_row() {
  for (int k = 0; k < 4; ++k) {
    const cudaError_t e = cudaFuncSetAttribute(kRowKernels[k >> 1][k & 1], cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_attn_row(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const AttnArgs& a, int dtype,
                            int64_t grid, cudaStream_t stream) {
  if (grid < 1 || grid > 0x7fffffff) return cudaErrorInvalidValue;
  const int box = attn_row_box(dtype, 1 << a.page_shift);
  return launch_pdl(kRowKernels[dtype == 2][a.wait_limit_ns < kSuspendNs], static_cast<unsigned>(grid), kWarps * 32, kSmem,
                    stream, tm_k, tm_v, a, box);
}

}  // namespace skv
