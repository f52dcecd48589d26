// Shared by the kernels of attention over paged or packed K and V: a sequence's
// lengths, the search for a CTA's job, and waits that can be inlined.
#pragma once

#include "kernels.h"
#include "ptx.cuh"
#include "softmax_util.cuh"

namespace skv {

constexpr int kAttnDim = 128;
constexpr int kAttnKeyTile = 128;   // keys per tile, the unit of a split

struct AttnSeq {
  int q0, sq;   // first query row and query count
  int k0, kv;   // packed: first key row; key count
};

// Lengths of sequence b, cut to what the buffers hold whatever the device arrays say.
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  AttnSeq s;
  s.q0 = min(max(a.cu_q[b], 0), a.total_q);
  s.sq = max(min(a.cu_q[b + 1], a.total_q) - s.q0, 0);
  if (a.table != nullptr) {
    const int64_t most = min(static_cast<int64_t>(a.table_width) << a.page_shift, int64_t{0x7fff0000});
    s.k0 = 0;
    s.kv = static_cast<int>(min(static_cast<int64_t>(max(a.kv_lens[b], 0)), most));
  } else {
    s.k0 = min(max(a.cu_kv[b], 0), a.total_kv);
    s.kv = min(max(min(a.cu_kv[b + 1], a.total_kv) - s.k0, 0), 0x7fff0000);
  }
  return s;
}

// Pages: brings the lengths and this CTA's share of the block table towards L2, by one warp,
// before grid_dependency_wait: a prefetch returns nothing, so it may run ahead of the
// kernel that writes them, and the first loads after the wait are L2 hits.
__device__ __forceinline__ void attn_prefetch(const AttnArgs& a, int lane) {
  for (int b = 32 * lane; b <= a.batch && b < 32 * 32; b += 32 * 32) {
    prefetch_l2_line(a.cu_q + b);
    if (b < a.batch) prefetch_l2_line(a.kv_lens + b);
  }
  const int64_t lines = (static_cast<int64_t>(a.batch) * a.table_width + 31) / 32;
  const int64_t each = (lines + gridDim.x - 1) / gridDim.x;
  const int64_t first = each * blockIdx.x;
  if (lane < each && each <= 32 && first + lane < lines) prefetch_l2_line(a.table + 32 * (first + lane));
}

__device__ __forceinline__ int warp_scan_incl(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}
__device__ __forceinline__ int warp_sum_int(int v) { return __reduce_add_sync(0xffffffffu, v); }

// ceil(x / y) for 0 <= x < 2^24 (a sequence's key tiles), y >= 1: x is a float, and below 2^23 the quotient's two last places
// are less than one, so it is off by one at most and the remainder puts it right; above, the result may be off by one,
// where a count of splits is cut to 64 anyway.
__device__ __forceinline__ int ceil_div(int x, int y) {
  int q = __float2int_rz(__fdividef(static_cast<float>(x), static_cast<float>(y)));
  const int r = x - q * y;
  q += r > y ? 2 : r > 0 ? 1 : r <= -y ? -1 : 0;
  return q;
}

struct AttnPiece {
  int b, j, g;       // sequence (-1: none), query tile, KV head
  int tile0, tiles;  // key tiles (perhaps more than the sequence has)
  int slot;          // the piece's place among the partials, or -1: the whole job
  int S;             // pieces of the job where this is its first, else 0
};

// The batch's jobs, found by one warp (lane by lane a sequence). Sequence b has n_b =
// ceil(s_b / tokens) query tiles and S_b splits: num_splits of them where the plan
// forces a count, else, with T = the key tiles a job should walk, clamp(ceil(tiles_b / T),
// 1, num_splits). If the unsplit jobs fit one wave of num_sms, T is the smallest whose
// jobs do too; otherwise T is a third of an SM's share of the work (ragged chunks and e4m3
// chunks both lose with two thirds or a whole one: fewer jobs to even out), or the next
// (by quarters) whose split jobs fit the workspace's max_slots.
// Jobs are listed sequence by sequence; within one the last query tiles first (they
// see the most keys), then the splits, the KV heads fastest.
struct AttnJobs {
  int tokens, groups;
  int n_first, tiles_first;   // the first 32 sequences stay in registers
  int T;                      // 0: S_b = num_splits
  int from, from_base, from_slots;   // the group of 32 sequences of the last job found, jobs and slots before it

  __device__ __forceinline__ void load(const AttnArgs& a, int i, int lane, int& n, int& tiles) const {
    n = tiles = 0;
    const int b = 32 * i + lane;
    if (b < a.batch) {
      const AttnSeq q = attn_seq(a, b);
      n = (q.sq + tokens - 1) / tokens;
      tiles = (q.kv + kAttnKeyTile - 1) / kAttnKeyTile;
    }
  }
  __device__ __forceinline__ void shape(const AttnArgs& a, int i, int lane, int& n, int& tiles) const {
    if (i == 0) {
      n = n_first;
      tiles = tiles_first;
    } else {
      load(a, i, lane, n, tiles);
    }
  }
  __device__ __forceinline__ int splits(const AttnArgs& a, int tiles) const {
    return T == 0 ? a.num_splits : min(a.num_splits, max(1, ceil_div(tiles, T)));
  }

  // kSplits: false where no job is ever split.
  template <bool kSplits>
  __device__ __forceinline__ void init(const AttnArgs& a, int job_tokens, int lane) {
    tokens = job_tokens;
    groups = (a.batch + 31) / 32;
    T = 0;
    from = from_base = from_slots = 0;
    load(a, 0, lane, n_first, tiles_first);
    if (!kSplits || a.adaptive != kByLength || a.num_splits <= 1) return;
    // The sums are floats (exact to 2^-23), and the bounds below give way by more than that. (64-bit integers cost a
    // microsecond at the start of every launch.)
    int jobs = 0, most = 1;
    float work = 0.f;
    for (int i = 0; i < groups; ++i) {
      int n, tiles;
      shape(a, i, lane, n, tiles);
      jobs += warp_sum_int(n);
      most = max(most, __reduce_max_sync(0xffffffffu, n > 0 ? tiles : 0));
      float w = static_cast<float>(n) * static_cast<float>(tiles);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      work += w;
    }
    work *= static_cast<float>(a.h_kv);
    const float unsplit = static_cast<float>(jobs) * static_cast<float>(a.h_kv);
    const float wave = static_cast<float>(a.num_sms);
    if (unsplit > wave) {
      T = max(1, static_cast<int>(fminf(ceilf(work / (3.f * wave)), 16777216.f)));   // (above any sequence's tiles)
      for (;;) {
        int split_jobs = 0;
        for (int i = 0; i < groups; ++i) {
          int n, tiles;
          shape(a, i, lane, n, tiles);
          const int s = splits(a, tiles);
          split_jobs += warp_sum_int(s > 1 ? n * s : 0);
        }
        if (static_cast<long long>(split_jobs) * a.h_kv <= a.max_slots) return;
        T += (T + 3) >> 2;
      }
    }
    // jobs(T) <= work / T + unsplit, so from work / (wave - unsplit) on they fit
    int lo = max(1, static_cast<int>(work * 0.9999f / wave));
    int hi = most;
    if (unsplit < wave) hi = min(hi, static_cast<int>(fminf(work * 1.0001f / (wave - unsplit), 16777216.f)) + 2);
    hi = max(hi, lo);
    while (lo < hi) {
      T = (lo + hi) >> 1;
      int total = warp_sum_int(n_first * splits(a, tiles_first));
      for (int i = 1; i < groups; ++i) {
        int n, tiles;
        load(a, i, lane, n, tiles);
        total += warp_sum_int(n * splits(a, tiles));
      }
      if (static_cast<long long>(total) * a.h_kv <= a.num_sms) hi = T;
      else lo = T + 1;
    }
    T = hi;
  }

  // (a CTA's jobs come in rising order, as a rule)
  template <bool kSplits>
  __device__ __forceinline__ AttnPiece find(const AttnArgs& a, int idx, int lane) {
    AttnPiece job = {-1, 0, 0, 0, 0, -1, 0};
    if (idx < from_base) from = from_base = from_slots = 0;
    int base = from_base, slots = from_slots;
    for (int i = from; i < groups; ++i) {
      int n, tiles;
      shape(a, i, lane, n, tiles);
      const int s = kSplits ? splits(a, tiles) : 1;
      const int count = n * s * a.h_kv;
      const int split_count = s > 1 ? count : 0;
      const int incl = warp_scan_incl(count, lane), sincl = kSplits ? warp_scan_incl(split_count, lane) : 0;
      const int local = idx - base - (incl - count);
      const unsigned hit = __ballot_sync(0xffffffffu, local >= 0 && local < count);
      if (hit != 0) {
        from = i;
        from_base = base;
        from_slots = slots;
        const int src = __ffs(hit) - 1;
        const int l = __shfl_sync(0xffffffffu, local, src);
        const int nn = __shfl_sync(0xffffffffu, n, src);
        const int all = __shfl_sync(0xffffffffu, tiles, src);
        const int first = kSplits ? __shfl_sync(0xffffffffu, slots + sincl - split_count, src) : 0;
        const int S = kSplits ? __shfl_sync(0xffffffffu, s, src) : 1;
        const int rest = l / a.h_kv;
        job.b = 32 * i + src;
        job.g = l - rest * a.h_kv;
        job.j = nn - 1 - rest;
        job.tiles = all;
        if (S > 1) {
          const int tile = rest / S, at = rest - tile * S;
          job.j = nn - 1 - tile;
          const int each = all / S, more = all - each * S;
          job.tile0 = at * each + min(at, more);
          job.tiles = each + (at < more ? 1 : 0);
          job.slot = first + (job.j * a.h_kv + job.g) * S + at;
          job.S = at == 0 ? S : 0;
          // (offsets that decrease can name more split jobs than the workspace holds)
          if (static_cast<unsigned>(job.slot) >= static_cast<unsigned>(a.max_slots)) job.b = -1;
        }
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
      if (kSplits) slots += __shfl_sync(0xffffffffu, sincl, 31);
    }
    return job;
  }
};

// Equal shares of the batch's work for one wave of CTAs. Its jobs (sequence, query tile,
// group of side heads) lie one after the other on a line, each as kHead units for its start
// and end and then kWeight units for every 2^share_shift key tiles that its tokens see (or
// one more; half as many where a job of the tile kernel has one row block only). Range r of R
// takes the units [r U, (r + 1) U), by one CTA for each of the side heads: the heads of a row
// lie side by side in memory, and read at one time they share DRAM rows (decode of 128 sequences of
// 2,048 e4m3 keys, 8 KV heads: 97 us when it came, with the heads one after the other on the line 141; one
// job a CTA 118). A job that crosses no boundary is written at once; the pieces of one
// that does are partials. A CTA has at most one piece that begins a cut job (slot R side + h R +
// r, h its head of the group) and one that goes on with one (slot h R + r), so the pieces of a
// job lie at R side + h R + r, then h R + r + 1, h R + r + 2, ..
template <int kWeight, int kHead>
struct AttnShares {
  int tokens;               // of a job
  int R, r, h;              // ranges; this CTA's range and head of a group
  int U, pos, end;          // units of a range; the next one of this CTA, its last
  int b, n, sq, kv;         // the sequence at pos: query tiles, tokens, keys
  int job, group, off;      // in it: the job (its last query tile is job 0), head group, units before pos
  uint32_t frac;            // running sum of the key tiles before the job: what was rounded off

  // Job i of a sequence sees ceil(x_i / 128) key tiles, x_i = kv - sq + (n - i) tokens (all of the sequence's where
  // it has fewer keys than tokens). The running sum of (x_i + 127) / 128, rounded down, gives each job at least as many.
  // (kWeight 1: a job has at most 16 tokens, and counts all of its sequence's tiles.)
  __device__ __forceinline__ uint32_t keys_up(const AttnArgs& a, int i) const {
    if constexpr (kWeight == 1) {
      const uint32_t up = (1u << (7 + a.share_shift)) - 1u;
      return (max(kv, 1) + up) & ~up;
    }
    const bool behind = kv >= sq && kv > 0;
    const uint32_t x = (behind ? kv - sq : max(kv, 1)) + (1u << (7 + a.share_shift)) - 1u;
    return x + (behind ? static_cast<uint32_t>(tokens * (n - i)) : 0u);
  }
  // 128 << share_shift times the key tiles of the jobs before i.
  __device__ __forceinline__ unsigned long long sum_before(const AttnArgs& a, int i) const {
    const unsigned long long first = keys_up(a, 0), step = kv >= sq && kv > 0 ? tokens : 0, m = i;
    return m * first - step * (m * (m - (i > 0)) / 2);
  }
  // (kWeight 2: a job of at most tokens / 2 tokens has one row block)
  __device__ __forceinline__ int weight_of(int i) const {
    return kWeight == 2 && i == 0 && sq - (n - 1) * tokens <= tokens / 2 ? 1 : kWeight;
  }
  __device__ __forceinline__ int units_before(const AttnArgs& a, int i) const {
    const int sh = 7 + a.share_shift;
    if constexpr (kWeight == 1) return i * (kHead + static_cast<int>(keys_up(a, 0) >> sh));
    const int one = i > 0 && weight_of(0) < kWeight ? static_cast<int>(keys_up(a, 0) >> sh) : 0;
    return i * kHead + kWeight * static_cast<int>(sum_before(a, i) >> sh) - one;
  }
  __device__ __forceinline__ void load(const AttnArgs& a, int seq) {
    b = seq;
    n = sq = kv = 0;
    if (b < a.batch) {
      const AttnSeq q = attn_seq(a, b);
      sq = q.sq;
      kv = q.kv;
      n = (sq + tokens - 1) / tokens;
    }
  }

  __device__ __forceinline__ void init(const AttnArgs& a, int job_tokens, int lane) {
    tokens = job_tokens;
    const int groups = a.h_kv / a.side;
    R = gridDim.x / a.side;
    r = blockIdx.x / a.side;
    h = blockIdx.x - r * a.side;
    int total = 0, most = 0, count = 0;
    for (int i = (a.batch - 1) / 32; i >= 0; --i) {   // (the first 32 sequences last: they stay for the search)
      load(a, 32 * i + lane);
      count = groups * units_before(a, n);
      total += warp_sum_int(count);
      most = max(most, __reduce_max_sync(0xffffffffu, n > 0 ? (max(kv, 1) + tokens) >> (7 + a.share_shift) : 0));
    }
    // (a job of num_splits - 1 shares touches num_splits ranges at most; a share has a key tile of every job in it)
    U = max(max((total + R - 1) / R, kWeight * (most + 2) / (a.num_splits - 1) + 1), kWeight);
    const long long first = static_cast<long long>(U) * r;
    pos = static_cast<int>(first < total ? first : total);
    end = total - pos < U ? total : pos + U;
    if (pos >= end) return;
    int base = 0, at = -1;
    for (int i = 0; 32 * i < a.batch; ++i) {
      if (i > 0) {
        load(a, 32 * i + lane);
        count = groups * units_before(a, n);
      }
      const int incl = warp_scan_incl(count, lane);
      const int local = pos - base - (incl - count);
      const unsigned hit = __ballot_sync(0xffffffffu, local >= 0 && local < count);
      if (hit != 0) {
        const int src = __ffs(hit) - 1;
        b = 32 * i + src;
        n = __shfl_sync(0xffffffffu, n, src);
        sq = __shfl_sync(0xffffffffu, sq, src);
        kv = __shfl_sync(0xffffffffu, kv, src);
        at = __shfl_sync(0xffffffffu, local, src);
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (at < 0) {                    // (offsets that decrease)
      pos = end;
      return;
    }
    job = 0;
    if constexpr (kWeight == 1) {
      if (n > 1) job = at / (groups * units_before(a, 1));
    } else {
      for (int hi = n; hi - job > 1;) {
        const int mid = (job + hi) >> 1;
        if (groups * units_before(a, mid) <= at) job = mid;
        else hi = mid;
      }
    }
    const int before = units_before(a, job);
    off = at - groups * before;
    group = 0;
    if (groups > 1) {
      const int units = units_before(a, job + 1) - before;
      group = off / units;
      off -= group * units;
    }
    frac = kWeight == 1 ? 0u : static_cast<uint32_t>(sum_before(a, job)) & ((128u << a.share_shift) - 1u);
  }

  // The next piece of this CTA.
  __device__ __forceinline__ AttnPiece next(const AttnArgs& a) {
    AttnPiece p = {-1, 0, 0, 0, 0, -1, 0};
    while (pos < end && p.b < 0) {
      const uint32_t sum = frac + keys_up(a, job);
      const int weight = weight_of(job), k_all = static_cast<int>(sum >> (7 + a.share_shift));
      const int units = kHead + weight * k_all;
      const int start = pos - off, stop = min(end, start + units);
      // key tile k (of 2^share_shift) is the unit start + kHead + weight k
      auto ceil_w = [&](int x) { return x <= 0 ? 0 : kWeight == 2 && weight == 2 ? (x + 1) >> 1 : x; };
      const int k0 = ceil_w(off - kHead), k1 = ceil_w(stop - start - kHead);
      if (k1 > k0) {                   // (else the job's first key tile is the next range's)
        p.b = b;
        p.g = group * a.side + h;
        p.j = n - 1 - job;
        p.tile0 = k0 << a.share_shift;
        p.tiles = (k1 - k0) << a.share_shift;
        if (k0 > 0) {
          p.slot = h * R + r;
        } else if (k1 < k_all) {
          p.slot = gridDim.x + h * R + r;
          p.S = (start + kHead + weight * (k_all - 1)) / U - r + 1;
        }
      }
      pos = start + units;
      off = 0;
      if (pos < end && (++group) * a.side == a.h_kv) {
        group = 0;
        frac = sum & ((128u << a.share_shift) - 1u);
        if (++job == n) {
          job = 0;
          frac = 0;
          do load(a, b + 1);
          while (n == 0 && b < a.batch);
          if (b >= a.batch) pos = end;   // (offsets that decrease)
        }
      }
    }
    return p;
  }
};

// Waits for the phase with the given parity of `bar`, at most `limit` ns. All lanes of
// a converged warp call it and leave it together (one barrier word, one timer). It
// is kept this small because it is inlined at some thirty places: with the status
// word and the CTA's abort flag handled in its loop, or with a vote behind it, these
// kernels lose 30 to 40 % of their rate (e4m3 prompt of 16,384 tokens: 1.2 -> 2.0 ms). A role that gives up
// says so once (give_up); the others run into their own limit.
// kPoll: test_wait, for limits below kSuspendNs: the hardware suspends a try_wait for
// longer than a load from memory takes, so such a limit could never run out. Limits
// that short are for tests of the way out, and have kernels of their own.
constexpr uint64_t kSuspendNs = 20000;
template <bool kPoll>
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, uint32_t limit) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint32_t t0 = globaltimer_lo();
  do {
    if (kPoll ? mbar_test_wait(bar, parity) : mbar_try_wait(bar, parity)) return true;
  } while (globaltimer_lo() - t0 <= limit);
  return false;
}
// The limit of wait_for: the caller's (mla_set_wait_limit_ns), at most what 32 bits of
// nanoseconds can tell apart.
__device__ __forceinline__ uint32_t wait_limit(const AttnArgs& a) {
  return a.wait_limit_ns < 4000000000ull ? static_cast<uint32_t>(a.wait_limit_ns) : 4000000000u;
}
// Records that a role's wait ran out.
__device__ __forceinline__ void give_up(const AttnArgs& a, uint32_t site) {
  if ((threadIdx.x & 31) == 0) {
    atomicOr(&a.status[0], 1u);
    atomicCAS(&a.status[1], 0u, site);
  }
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// P for e4m3 V is f16, which ends at 2^-25 below: its reference is therefore taken 2^kF16Shift under the running maximum, P
// = 2^(s - m + kF16Shift), and the sums carry the same factor, so O / l needs nothing and the LSE a multiplication.
// Weights down to 2^-32 of the largest then count (the numerator alone lost what fell below 2^-25: 32,768 keys of 2^-26
// behind a key whose V is 0 gave O = 0). At the top a reference that lags by kRescaleThreshold leaves P at
// 2^15, finite in f16.
constexpr float kF16Shift = 7.0f;
constexpr float kRescaleThreshold = 8.0f;   // log2 units a row's reference may lag behind its maximum
// Whether the maximum mx asks for a new reference. f16: mx and s - m are rounded to scores' own steps, which grow with them;
// the lag allowed shrinks with |m| (8 at 0, none from 2^20 on), so that P stays in range.
template <bool kF16>
__device__ __forceinline__ bool new_reference(float mx, float m) {
  if constexpr (kF16) return mx > fmaxf(m, fmaf(fabsf(m), -0x1p-17f, m + kRescaleThreshold));
  return mx > m + kRescaleThreshold;
}
// l += x, compensated (Kahan, "Further remarks on reducing truncation errors", 1965): c is what l holds too much. A long
// row's small terms would be lost behind a large one (16,384 keys of 2^-25 behind a sink: 4e-5 of the LSE by plain
// sums). Under 1 % of the time (decode of 128 sequences of 2,048 e4m3 keys 95.0 -> 95.7 us, 7 ragged e4m3 prompts 233 -> 235).
__device__ __forceinline__ void add_compensated(float& l, float& c, float x) {
  const float y = x - c, s = l + y;
  c = (s - l) - y;
  l = s;
}
// The fp32 term of the exponent, and l without the shift's factor.
template <bool kF16>
__device__ __forceinline__ float minus_reference(float m) {
  return m == -INFINITY ? 0.f : (kF16 ? kF16Shift : 0.f) - m;
}
template <bool kF16>
__device__ __forceinline__ float lse_of(float m, float l) {
  return m + log2f(kF16 ? l * 0x1p-7f : l);
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
// N (16 or 32) consecutive elements at element offset `at` of an output of type
// out_dtype (MLA_OUT_*: 0 fp32, 1 bf16, 2 e4m3).
template <int N>
__device__ __forceinline__ void store_row(void* out, int out_dtype, int64_t at, const float (&x)[N], float inv_scale) {
  if (out_dtype == 0) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) p[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  } else if (out_dtype == 1) {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + at);
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      p[i] = make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                        pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
  } else {
    uint4* p = reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) + at);
#pragma unroll
    for (int i = 0; i < N / 16; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = pack_e4m3x4(x[16 * i + 4 * k] * inv_scale, x[16 * i + 4 * k + 1] * inv_scale,
                           x[16 * i + 4 * k + 2] * inv_scale, x[16 * i + 4 * k + 3] * inv_scale);
      p[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// The kernels here set up while the preceding kernel of the stream ends
// (grid_dependency_wait before the first read or write of global memory).
template <typename K, typename... A>
cudaError_t launch_pdl(K kernel, unsigned grid, unsigned block, size_t smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace skv
