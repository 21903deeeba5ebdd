// What a serving step needs before its attention: the plan of its tokens in a paged cache, and the norms and the
// rotation of its queries and keys.
#include "tl_serve.cuh"
#include "tl_softmax.cuh"

namespace tl {

// ---------------------------------------------------------------------------- plan
// Sequence b holds n_b rows and gets c_b more: it needs ceil((n_b + c_b) / page) pages and has ceil(n_b / page), so
// its new pages are free_pages[taken + sum of the needs before it ..].  Every CTA takes both prefix sums over
// the batch for itself (4096 sequences at most), so one launch does without a hand-over between CTAs; then each
// packed token finds its sequence by bisection of the bounds in shared memory (mostly it is that of the lane's token before),
// and the token that opens a page writes the page's entry.  New pages are read from the free list and not from the table, so nothing waits for
// a write.  Lengths (and `taken`) that are brought up to date in place may only be written once every CTA has read
// them: a grid of up to 8 CTAs is one cluster then, with a barrier between; behind a larger one a second launch of one
// CTA works them out again (37 sequences with 76000 new tokens and the slots of 189000 rows, in place: 7.5 us, as one cluster 40; one of
// 3000 tokens, a cluster of 6: 4.0 to 4.1, not in place 3.7).
// The launch and some four waits bound it: lengths, two rounds of sums, the table's entry, the stores.  Not in place: a step of 64
// sequences 3.4 us (in place 2.9 to 3.4); 37 sequences with 76000 new tokens and the slots of all 189000 rows 5.4 us; the slots of 8.3
// million rows of 1000 sequences 22.8 us (each by a bisection of its own 61; four of a lane's pages read at once 24.7, and pages of one
// row 37 instead of 44).
struct PlanParams {
  DevStatus* status;
  const int* lengths;
  const int* counts;  // null: 1 each
  int* table;
  const int* free_pages;
  const int* taken;
  int* taken_out;
  int* new_lengths;
  int* cu_q;
  int* cu_k;       // may be null
  int* slots;
  int* positions;  // may be null
  int* kv_slots;   // may be null
  int batch, max_pages, num_free, page_size, tokens, kv_tokens;
  int parts;       // plan::kTokens, plan::kLengths
  FastDiv by_page;
};

namespace plan {
constexpr int kMaxBatch = 4096, kThreads = 1024, kFewThreads = 512;  // threads of a CTA, and for up to as many sequences
constexpr int kTokens = 1, kLengths = 2;  // what a launch writes: bounds, slots, pages; lengths and pages taken
constexpr uint32_t kMost = 0x7fffffffu;
// Sums stop at 2^31 - 1 (in any order): whatever lies there is past every buffer.
__device__ __forceinline__ uint32_t sat(uint32_t a, uint32_t b) { return min(a + b, kMost); }
// The sums over all threads before this one, and those over all, of N numbers.
template <int kWarps, int N>
__device__ __forceinline__ void scan(uint32_t (&v)[N], uint32_t (*warps)[kWarps], uint32_t (&all)[N]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s[N];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    s[n] = v[n];
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, s[n], x);
      if (lane >= x) s[n] = sat(s[n], o);
    }
    if (lane == 31) warps[n][warp] = s[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    uint32_t t = lane < kWarps ? warps[n][lane] : 0u;
#pragma unroll
    for (int x = 1; x < kWarps; x <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, t, x);
      if (lane >= x) t = sat(t, o);
    }
    all[n] = __shfl_sync(0xffffffffu, t, kWarps - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, t, warp ? warp - 1 : 0);
    const uint32_t up = __shfl_up_sync(0xffffffffu, s[n], 1);
    v[n] = sat(warp ? before : 0u, lane ? up : 0u);
  }
}
// The last b of lo .. n - 1 with bounds[b] <= i, for bounds[lo] <= i (so it holds i if any does).
__device__ __forceinline__ int find(const int* bounds, int lo, int n, int i) {
  int hi = n;  // bounds[lo] <= i < bounds[hi] (or past the end)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (bounds[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}
}  // namespace plan

template <bool Cluster, int kThreads>
__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanParams p) {
  using namespace plan;
  constexpr int kWarps = kThreads / 32, kChunk = kThreads == kFewThreads ? 1 : kMaxBatch / kThreads;  // sequences of a thread, at most
  extern __shared__ int smem[];
  __shared__ uint32_t s_warps[4][kWarps];
  int* const s_q = smem;                       // [batch + 1] first new token of a sequence
  int* const s_k = s_q + p.batch + 1;          // [batch + 1] its first row among all
  int* const s_len = s_k + p.batch + 1;        // [batch] rows held; ~rows if it gets none of its new ones
  int* const s_first = s_len + p.batch;        // [batch] place of its first new page in the free list
  const int chunk = (p.batch + kThreads - 1) / kThreads, b0 = static_cast<int>(threadIdx.x) * chunk;
  const long long cap = static_cast<long long>(p.max_pages) * p.page_size;
  const bool report = blockIdx.x == 0;

  const int taken = *p.taken;
  const bool taken_ok = taken >= 0 && taken <= p.num_free;
  const uint32_t left = taken_ok ? static_cast<uint32_t>(p.num_free - taken) : 0u;
  int raw[kChunk], len[kChunk], cnt[kChunk];
  uint32_t need[kChunk], sum_q = 0, sum_p = 0;
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    const int b = b0 + i;
    raw[i] = len[i] = cnt[i] = 0;
    need[i] = 0;
    if (i >= chunk || b >= p.batch) continue;
    raw[i] = len[i] = p.lengths[b];
    cnt[i] = p.counts ? p.counts[b] : 1;
    if (len[i] < 0 || cnt[i] < 0 || static_cast<long long>(len[i]) + cnt[i] > cap) {
      if (report) report_index(p.status, static_cast<unsigned long long>(b));
      if (len[i] < 0 || len[i] > cap) len[i] = 0;
      cnt[i] = 0;
    }
    need[i] = divide(len[i] + cnt[i] + p.page_size - 1, p.by_page) - divide(len[i] + p.page_size - 1, p.by_page);
    sum_q = sat(sum_q, cnt[i]);
    sum_p = sat(sum_p, need[i]);
  }
  uint32_t at[2] = {sum_q, sum_p}, all[2];
  scan(at, s_warps, all);
  uint32_t &at_q = at[0], &at_p = at[1];
  // A sequence gets its tokens if they and its pages are there: those that do not fit are the last ones.
  uint32_t sum_k = 0, used = 0;
#pragma unroll
  for (int i = 0; i < kChunk; ++i) {
    const int b = b0 + i;
    if (i >= chunk || b >= p.batch) continue;
    s_q[b] = static_cast<int>(at_q);
    s_first[b] = static_cast<int>(taken + at_p);
    at_q = sat(at_q, cnt[i]);
    at_p = sat(at_p, need[i]);
    const bool fits = at_q <= static_cast<uint32_t>(p.tokens) && (need[i] == 0 || at_p <= left);
    if (!fits && cnt[i] > 0) {
      if (report) report_index(p.status, static_cast<unsigned long long>(b));
      cnt[i] = -1;
    } else if (need[i] > 0) {
      used = at_p;
    }
    s_len[b] = cnt[i] < 0 ? ~len[i] : len[i];
    sum_k = sat(sum_k, len[i] + max(cnt[i], 0));
  }
  if (threadIdx.x == 0) s_q[p.batch] = static_cast<int>(all[0]);
  if (p.cu_k || p.kv_slots) {
    uint32_t at_k[1] = {sum_k}, all_k[1];
    scan(at_k, s_warps + 2, all_k);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const int b = b0 + i;
      if (i >= chunk || b >= p.batch) continue;
      s_k[b] = static_cast<int>(at_k[0]);
      at_k[0] = sat(at_k[0], len[i] + max(cnt[i], 0));
    }
    if (threadIdx.x == 0) s_k[p.batch] = static_cast<int>(all_k[0]);
  }
  // the most pages that a sequence which gets its tokens ends at
  {
    const uint32_t top = __reduce_max_sync(0xffffffffu, used);
    if ((threadIdx.x & 31) == 0) s_warps[3][threadIdx.x >> 5] = top;
  }
  if constexpr (Cluster) asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
  __syncthreads();

  const bool tokens = p.parts & kTokens;
  if (blockIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const int b = b0 + i;
      if (i >= chunk || b >= p.batch) continue;
      if (p.parts & kLengths) p.new_lengths[b] = cnt[i] > 0 ? len[i] + cnt[i] : raw[i];
      if (tokens) p.cu_q[b] = s_q[b];
      if (tokens && p.cu_k) p.cu_k[b] = s_k[b];
    }
    if (threadIdx.x == 0) {
      uint32_t top = 0;
      for (int w = 0; w < kWarps; ++w) top = max(top, s_warps[3][w]);
      if (p.parts & kLengths) *p.taken_out = taken + static_cast<int>(top);
      if (tokens) p.cu_q[p.batch] = s_q[p.batch];
      if (tokens && p.cu_k) p.cu_k[p.batch] = s_k[p.batch];
      if (!taken_ok || (p.kv_slots && s_k[p.batch] > p.kv_tokens)) report_index(p.status, static_cast<unsigned long long>(p.batch));
    }
  }
  if (!tokens) return;

  // Each warp has a range of packed tokens, a lane every 32nd of it: the sequence of one is mostly that of the lane's next one.
  const int lane = threadIdx.x & 31;
  const long long warps = static_cast<long long>(gridDim.x) * kWarps, warp = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  struct Sequence {
    int b, begin, past;  // its packed tokens
    int held, has;       // rows and pages held; held is ~rows if it gets none of its new ones
    const int* table;
    const int* fresh;    // new pages, of page `has` on
  };
  auto enter = [&](const int* bounds, Sequence& q, int t) {
    q.b = find(bounds, q.b, p.batch, t);
    q.begin = bounds[q.b];
    q.past = bounds[q.b + 1];
    q.held = s_len[q.b];
    q.has = static_cast<int>(divide(static_cast<uint32_t>((q.held < 0 ? ~q.held : q.held) + p.page_size - 1), p.by_page));
    q.table = p.table + static_cast<long long>(q.b) * p.max_pages;
    q.fresh = p.free_pages + s_first[q.b] - q.has;
  };
  // The slot of row `pos`: its page is in the table, or a new one.  -1 where there is none.
  auto slot_of = [&](const Sequence& q, int pos, int& page_at, int& page) {
    page_at = static_cast<int>(divide(static_cast<uint32_t>(pos), p.by_page));
    page = page_at < q.has ? q.table[page_at] : __ldg(q.fresh + page_at);
    const long long slot = static_cast<long long>(page) * p.page_size + (pos - page_at * p.page_size);
    if (page < 0 || slot > static_cast<long long>(kMost)) {
      report_index(p.status, static_cast<unsigned long long>(q.b));
      return -1;
    }
    return static_cast<int>(slot);
  };
  auto each = [&](int n, const int* bounds, auto&& token) {
    const long long range = ((n + warps - 1) / warps + 31) / 32 * 32, begin = warp * range, end = begin + range < n ? begin + range : n;
    const int total = bounds[p.batch];
    Sequence q = {};
    for (long long i = begin + lane; i < end; i += 32) {
      const int t = static_cast<int>(i);
      if (t < total && t >= q.past) enter(bounds, q, t);
      token(t, t < total, q);
    }
  };
  each(p.tokens, s_q, [&](int t, bool there, const Sequence& q) {
    int slot = -1, pos = 0;
    if (there) {
      pos = (q.held < 0 ? ~q.held : q.held) + t - q.begin;
      if (q.held >= 0) {
        int page_at, page;
        slot = slot_of(q, pos, page_at, page);
        // its first row opens a page
        if (pos == page_at * p.page_size) p.table[static_cast<long long>(q.b) * p.max_pages + page_at] = page;
      }
    }
    p.slots[t] = slot;
    if (p.positions) p.positions[t] = pos;
  });
  if (p.kv_slots)
    each(p.kv_tokens, s_k, [&](int t, bool there, const Sequence& q) {
      int page_at, page;
      p.kv_slots[t] = there ? slot_of(q, t - q.begin, page_at, page) : -1;
    });
}

// ---------------------------------------------------------------------------- norms and rotation
// A row x of d values (one head of one token) becomes
//   y = x / sqrt(mean x^2 + eps) * w,   (y_i, y_j) -> (y_i cos a - y_j sin a, y_i sin a + y_j cos a)
// for its r / 2 pairs, with the angle a = position * inv_freq of the pair.
// HBM bounds it: each value is read and written once for some 6 operations.  D / 16 threads hold a row, 16 values
// each: two vectors of 8 whose places are those of eight pairs, so that neither the rotation nor the store needs another
// thread, and the mean takes 3 (d 64: 2) exchanges.  A CTA has some rows of a token, the same ones of each of its tokens; its
// threads work out the next token's angles, one pair each, before they turn to their rows of this one, and each thread's
// next row is on its way.
// 8192 tokens of 32 and 8 heads of 128: 30.3 to 30.6 us, 5.5 TB/s, 0.81 of the copy rate (without the norms 29.3; 64 and 8 heads 51,
// 0.87; interleaved pairs, which pass through single fp32 arithmetic, 33.7 to 34.5, 0.72; angles in every thread for itself 36.7, with
// 24 warps an SM for their registers; frequencies in turns kept from token to token 32.2).  One step of 64: 2.7 to 3.0 us, the launch
// and two waits.
//
// Angles: a position may be far and a frequency any number, and fp32 would leave a turn of 2^20 with 4 bits
// behind the point.  So a frequency is held in turns as a 64-bit fraction, F = inv_freq / (2 pi) 2^64, whose product with
// the position modulo 2^64 is the angle's fraction of a turn, off by at most position (1 + |inv_freq| / 2) 2^-64 turns (F is cut to a
// whole number, and 1 / (2 pi) is rounded to 64 bits) and exact in all the turns before it.  sin and cos of the rest, within
// [-pi, pi], are off by 2^-21 at most (__sincosf), far below half a step of the 16-bit result.
struct RopeParams {
  const uint8_t* x[2];  // q, k
  uint8_t* y[2];
  const void* weight[2];  // [D] of T or fp32; null: no norm
  long long x_token[2], x_head[2], y_token[2], y_head[2];  // bytes
  int heads[2];
  const int* positions;
  const float* inv_freq;  // [rotary / 2]
  int tokens, rotary, weight_f32;
  float eps;
};

namespace rope {
constexpr int kMaxThreads = 256;
// Rows whose squares' sum is below kSmall, times kUp: from bf16's smallest value on the squares are normal numbers then.
constexpr float kSmall = 0x1p-90f, kUp = 0x1p80f;
// inv_freq / (2 pi) in units of 2^-64 turns, modulo one turn.
__device__ __forceinline__ unsigned long long turns(float f) {
  constexpr unsigned long long kInv2Pi = 2935890503282001226ull;  // 2^64 / (2 pi), rounded
  const uint32_t bits = __float_as_uint(f), e = (bits >> 23) & 0xffu;
  const unsigned long long m = (bits & 0x7fffffu) | (e ? 0x800000u : 0u);
  const unsigned long long lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int s = 150 - static_cast<int>(e ? e : 1);  // f = m 2^-s
  unsigned long long v;
  if (s > 64) v = s < 128 ? hi >> (s - 64) : 0;
  else if (s == 64) v = hi;
  else if (s > 0) v = (lo >> s) | (hi << (64 - s));
  else v = -s < 64 ? lo << -s : 0;
  return bits >> 31 ? 0 - v : v;
}
__device__ __forceinline__ float2 unit(unsigned long long turn, int position) {
  const long long a = static_cast<long long>(turn * static_cast<unsigned long long>(static_cast<long long>(position)));
  float2 cs;
  __sincosf(static_cast<float>(static_cast<int>(a >> 32)) * 1.4629180792671596e-9f, &cs.y, &cs.x);  // 2 pi 2^-32
  return cs;
}
}  // namespace rope

// A CTA has the same blockDim / (D / 16) rows of each of its tokens, a thread the same part of one row: its places and weights
// stay in registers.
template <class T, int D, bool Interleaved>
__global__ void __launch_bounds__(rope::kMaxThreads, 4) rope_kernel(const RopeParams p) {
  using namespace rope;
  constexpr int kPer = D / 16;  // threads of a row
  // cosines and sines of a token's pairs, and of the next one's
  __shared__ __align__(16) float s_cos[2][D / 2], s_sin[2][D / 2];
  const int j = threadIdx.x % kPer;
  // The vectors (of 8 values) of this thread: a pair's two places lie in both, or side by side in one.  (Interleaved pairs
  // have vectors half a row apart too, so that neighbours read neighbouring ones.)
  const int half = p.rotary / 16;
  int va, vb;
  bool turn, turn_b;  // (turn_b: of the second vector of interleaved pairs)
  if constexpr (Interleaved) {
    va = j;
    vb = j + kPer;
    turn = va < 2 * half;
    turn_b = vb < 2 * half;
  } else {
    turn = j < half;
    turn_b = false;
    va = j < half ? j : 2 * j;
    vb = j < half ? j + half : 2 * j + 1;
  }
  const int r = blockIdx.y * (blockDim.x / kPer) + threadIdx.x / kPer;
  const bool there = r < p.heads[0] + p.heads[1];
  const uint32_t group_mask = ((1u << kPer) - 1u) << (threadIdx.x % 32 / kPer * kPer);
  const int w = r >= p.heads[0], h = w ? r - p.heads[0] : r;
  int t = blockIdx.x;
  // the next token's row is on its way while this one's is worked on
  const uint8_t* src = p.x[w] + t * p.x_token[w] + h * p.x_head[w];
  uint8_t* dst = p.y[w] + t * p.y_token[w] + h * p.y_head[w];
  const long long src_step = gridDim.x * p.x_token[w], dst_step = gridDim.x * p.y_token[w];
  uint4 next_a = make_uint4(0, 0, 0, 0), next_b = next_a;
  if (there) {
    next_a = reinterpret_cast<const uint4*>(src)[va];
    next_b = reinterpret_cast<const uint4*>(src)[vb];
  }
  auto angles = [&](int token, int slot) {
    for (int i = threadIdx.x; i < p.rotary / 2; i += blockDim.x) {
      const float2 cs = unit(turns(__ldg(p.inv_freq + i)), __ldg(p.positions + token));
      s_cos[slot][i] = cs.x;
      s_sin[slot][i] = cs.y;
    }
  };
  angles(t, 0);
  const bool norm = there && p.weight[w] != nullptr;
  unsigned long long ua[4], ub[4];
  if (norm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ia = 8 * va + 2 * i, ib = 8 * vb + 2 * i;
      if (p.weight_f32) {
        const float* f = static_cast<const float*>(p.weight[w]);
        ua[i] = f2(f[ia], f[ia + 1]);
        ub[i] = f2(f[ib], f[ib + 1]);
      } else {
        const T* f = static_cast<const T*>(p.weight[w]);
        ua[i] = f2(static_cast<float>(f[ia]), static_cast<float>(f[ia + 1]));
        ub[i] = f2(static_cast<float>(f[ib]), static_cast<float>(f[ib + 1]));
      }
    }
  }

  for (int slot = 0; t < p.tokens; t += gridDim.x, slot ^= 1, dst += dst_step) {
    __syncthreads();  // this token's angles are there, and the one before is done with its own
    const bool more = t + static_cast<int>(gridDim.x) < p.tokens;
    if (more) angles(t + static_cast<int>(gridDim.x), slot ^ 1);
    if (there) {
      const uint32_t au[4] = {next_a.x, next_a.y, next_a.z, next_a.w}, bu[4] = {next_b.x, next_b.y, next_b.z, next_b.w};
      if (more) {
        src += src_step;
        next_a = reinterpret_cast<const uint4*>(src)[va];
        next_b = reinterpret_cast<const uint4*>(src)[vb];
      }
      unsigned long long a[4], b[4];  // two values each
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = to_f32x2<T>(au[i]), y = to_f32x2<T>(bu[i]);
        a[i] = f2(x.x, x.y);
        b[i] = f2(y.x, y.y);
      }
      if (norm) {
        unsigned long long s0 = fmul2(a[0], a[0]), s1 = fmul2(b[0], b[0]);
#pragma unroll
        for (int i = 1; i < 4; ++i) {
          s0 = ffma2(a[i], a[i], s0);
          s1 = ffma2(b[i], b[i], s1);
        }
        float x, y;
        f2_split(fadd2(s0, s1), x, y);
        auto row_sum = [&](float v) {
#pragma unroll
          for (int k = 1; k < kPer; k <<= 1) v += __shfl_xor_sync(group_mask, v, k);
          return v;
        };
        const float ss = row_sum(x + y);
        float inv = rsqrtf(ss * (1.f / D) + p.eps);
        // Squares of small bf16 values leave fp32's range below, which shows where eps is next to nothing: such a row is brought up
        // by a power of two first.  (The same in all threads of a row; 8192 tokens 30.6 us, without it 30.5.)
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          if (ss < kSmall && p.eps < kSmall) {
            const unsigned long long up = f2(kUp, kUp);
            s0 = s1 = f2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              a[i] = fmul2(a[i], up);
              b[i] = fmul2(b[i], up);
              s0 = ffma2(a[i], a[i], s0);
              s1 = ffma2(b[i], b[i], s1);
            }
            f2_split(fadd2(s0, s1), x, y);
            inv = rsqrtf(row_sum(x + y) * (1.f / D) + p.eps * kUp * kUp);
          }
        }
        const unsigned long long both = f2(inv, inv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = fmul2(fmul2(a[i], both), ua[i]);
          b[i] = fmul2(fmul2(b[i], both), ub[i]);
        }
      }
      auto table = [&](const float* values, int at, unsigned long long(&v)[2]) {  // four of a table's entries
        const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(values + at);
        v[0] = u.x;
        v[1] = u.y;
      };
      if constexpr (Interleaved) {
        auto rotate = [&](unsigned long long(&v)[4], int at) {
          const float4 c4 = *reinterpret_cast<const float4*>(s_cos[slot] + at), n4 = *reinterpret_cast<const float4*>(s_sin[slot] + at);
          const float c[4] = {c4.x, c4.y, c4.z, c4.w}, n[4] = {n4.x, n4.y, n4.z, n4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x, y;
            f2_split(v[i], x, y);
            v[i] = f2(x * c[i] - y * n[i], x * n[i] + y * c[i]);
          }
        };
        if (turn) rotate(a, 4 * va);
        if (turn_b) rotate(b, 4 * vb);
      } else if (turn) {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          unsigned long long cos[2], sin[2];
          table(s_cos[slot], 8 * j + 2 * i, cos);
          table(s_sin[slot], 8 * j + 2 * i, sin);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const unsigned long long x = a[i + e], y = b[i + e], xs = fmul2(x, sin[e]), ys = fmul2(y, sin[e]);
            float p0, p1;
            f2_split(ys, p0, p1);
            a[i + e] = ffma2(x, cos[e], f2(-p0, -p1));
            b[i + e] = ffma2(y, cos[e], xs);
          }
        }
      }
      auto pack = [](const unsigned long long(&v)[4]) {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float x, y;
          f2_split(v[i], x, y);
          r[i] = from_f32x2<T>(x, y);
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
      };
      reinterpret_cast<uint4*>(dst)[va] = pack(a);
      reinterpret_cast<uint4*>(dst)[vb] = pack(b);
    }
  }
}

template <class T, int D>
static void rope_launch(const RopeParams& p, bool interleaved, dim3 grid, int threads, cudaStream_t stream) {
  if (interleaved) rope_kernel<T, D, true><<<grid, threads, 0, stream>>>(p);
  else rope_kernel<T, D, false><<<grid, threads, 0, stream>>>(p);
}

constexpr int kRopeWarps = 32;  // resident on an SM (at 64 registers)

}  // namespace tl

using namespace tl;

extern "C" int tl_cache_plan(tl_ctx* ctx, const int* lengths, const int* counts, int batch, int page_size, int* page_table,
                             int max_pages, const int* free_pages, int num_free, const int* taken, int* taken_out,
                             int* new_lengths, int* cu_q, int* cu_k, int* slots, int* positions, int tokens, int* kv_slots,
                             int kv_tokens, tl_stream_t stream) {
  if (!ctx || batch < 0 || batch > plan::kMaxBatch || page_size < 1 || max_pages < 0 || num_free < 0 || tokens < 0 ||
      kv_tokens < 0)
    return TL_ERR_INVALID;
  if (static_cast<long long>(max_pages) * page_size >= (1LL << 31) - page_size) return TL_ERR_INVALID;
  if (!taken || !taken_out || !cu_q || (batch > 0 && (!lengths || !new_lengths)) || (tokens > 0 && !slots) ||
      (batch > 0 && max_pages > 0 && !page_table) || (num_free > 0 && !free_pages) || (kv_tokens > 0 && !kv_slots))
    return TL_ERR_INVALID;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  PlanParams p;
  p.status = ctx->status;
  p.lengths = lengths;
  p.counts = counts;
  p.table = page_table;
  p.free_pages = free_pages;
  p.taken = taken;
  p.taken_out = taken_out;
  p.new_lengths = new_lengths;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.slots = slots;
  p.positions = positions;
  p.kv_slots = kv_slots;
  p.batch = batch;
  p.max_pages = max_pages;
  p.num_free = num_free;
  p.page_size = page_size;
  p.tokens = tokens;
  p.kv_tokens = kv_tokens;
  p.by_page = fast_div(page_size);
  // More than 512 sequences go to CTAs of 1024 threads (a step of 4000: 10.5 us, with 512 threads 13.5; one of 64: 4.4 and 3.4),
  // two packed tokens a thread up to 1024 threads an SM (one: a step of 4000 9.3 us instead of 10.7, the others the same; eight: 13.2,
  // and 37 prompts 6.2 us instead of 5.4; 500 sequences with the slots of 4.1 million rows 12.7 us, with 512 threads an SM 16.5, with
  // 2048 14.8).
  const int threads = batch > plan::kFewThreads ? plan::kThreads : plan::kFewThreads, smem = (4 * batch + 2) * 4;
  const long long items = static_cast<long long>(tokens) + kv_tokens;
  long long ctas = (items + 2 * threads - 1) / (2 * threads);
  const int most = (threads == plan::kFewThreads ? 2 : 1) * ctx->sms;
  if (ctas > most) ctas = most;
  if (ctas < 1) ctas = 1;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool in_place = lengths == new_lengths || taken == taken_out;
  static std::atomic<unsigned long long> ready[4];
  auto launch = [&](int parts, long long grid, bool cluster) {
    p.parts = parts;
    using namespace plan;
    auto kern = threads == kFewThreads ? (cluster ? plan_kernel<true, kFewThreads> : plan_kernel<false, kFewThreads>)
                                       : (cluster ? plan_kernel<true, plan::kThreads> : plan_kernel<false, plan::kThreads>);
    if (smem > (48 << 10) - 1024 && !smem_ready(ready[2 * cluster + (threads == kFewThreads)], ctx->device, reinterpret_cast<const void*>(kern),
                                                (4 * plan::kMaxBatch + 2) * 4))
      return static_cast<int>(TL_ERR_CUDA);
    if (!cluster) {
      kern<<<static_cast<unsigned>(grid), threads, smem, st>>>(p);
      return launched();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(grid);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess) return static_cast<int>(TL_OK);
    (void)cudaGetLastError();
    return static_cast<int>(TL_ERR_CUDA);
  };
  if (!in_place || ctas == 1) return launch(plan::kTokens | plan::kLengths, ctas, false);  // (or a CTA's own barrier is enough)
  if (ctas <= 8) return launch(plan::kTokens | plan::kLengths, ctas, true);
  const int rc = launch(plan::kTokens, ctas, false);
  return rc == TL_OK ? launch(plan::kLengths, 1, false) : rc;
}

extern "C" int tl_norm_rope(tl_ctx* ctx, int dtype, const void* q, long long q_token_stride, long long q_head_stride,
                            const void* k, long long k_token_stride, long long k_head_stride, const void* q_weight,
                            const void* k_weight, int weight_dtype, float eps, const int* positions, const float* inv_freq,
                            int rotary, int interleaved, void* q_out, long long q_out_token_stride,
                            long long q_out_head_stride, void* k_out, long long k_out_token_stride,
                            long long k_out_head_stride, int tokens, int heads, int kv_heads, int d, tl_stream_t stream) {
  if (!ctx || (dtype != TL_BF16 && dtype != TL_FP16) || (weight_dtype != dtype && weight_dtype != TL_FP32) || tokens < 0 ||
      heads < 0 || kv_heads < 0 || (d != 64 && d != 128) || rotary < 0 || rotary > d || rotary % 16 != 0 ||
      (interleaved != 0 && interleaved != 1) || !(eps >= 0.f) || eps > 3.0e38f)
    return TL_ERR_INVALID;
  const long long strides[8] = {q_token_stride, q_head_stride, k_token_stride, k_head_stride, q_out_token_stride,
                                q_out_head_stride, k_out_token_stride, k_out_head_stride};
  for (long long s : strides)
    if (!esize_ok(s, 2)) return TL_ERR_INVALID;
  if (tokens == 0 || heads + static_cast<long long>(kv_heads) == 0) return TL_OK;
  if (heads + static_cast<long long>(kv_heads) > 65536 || tokens >= (1 << 30)) return TL_ERR_INVALID;
  if ((heads > 0 && (!q || !q_out || !aligned16(q) || !aligned16(q_out))) ||
      (kv_heads > 0 && (!k || !k_out || !aligned16(k) || !aligned16(k_out))) || (rotary > 0 && (!positions || !inv_freq)))
    return TL_ERR_INVALID;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  RopeParams p;
  p.x[0] = static_cast<const uint8_t*>(q);
  p.x[1] = static_cast<const uint8_t*>(k);
  p.y[0] = static_cast<uint8_t*>(q_out);
  p.y[1] = static_cast<uint8_t*>(k_out);
  p.weight[0] = heads > 0 ? q_weight : nullptr;
  p.weight[1] = kv_heads > 0 ? k_weight : nullptr;
  for (int w = 0; w < 2; ++w) {
    p.x_token[w] = 2 * strides[2 * w];
    p.x_head[w] = 2 * strides[2 * w + 1];
    p.y_token[w] = 2 * strides[4 + 2 * w];
    p.y_head[w] = 2 * strides[5 + 2 * w];
  }
  p.heads[0] = heads;
  p.heads[1] = kv_heads;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.tokens = tokens;
  p.rotary = rotary;
  p.weight_f32 = weight_dtype == TL_FP32;
  p.eps = eps;
  // A token's rows in as few CTAs as 256 threads allow, evenly (32 and 8 heads of 128: two of 160 threads, 30.2 us for 8192 tokens; of
  // 128 threads at most 32.2), as many CTAs as are resident: one more would wait for all others (64 and 8 heads 51 us, then 80).
  const int per = d / 16, rows = heads + kv_heads;
  const int rounds = (rows * per + rope::kMaxThreads - 1) / rope::kMaxThreads, at_once = (rows + rounds - 1) / rounds;
  const int threads = (at_once * per + 31) / 32 * 32, parts = (rows + threads / per - 1) / (threads / per);
  long long places = static_cast<long long>(kRopeWarps / (threads / 32)) * ctx->sms / parts;
  if (places < 1) places = 1;
  const dim3 grid(static_cast<unsigned>(tokens < places ? tokens : places), parts, 1);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TL_BF16) {
    if (d == 64) rope_launch<__nv_bfloat16, 64>(p, interleaved, grid, threads, s);
    else rope_launch<__nv_bfloat16, 128>(p, interleaved, grid, threads, s);
  } else {
    if (d == 64) rope_launch<__half, 64>(p, interleaved, grid, threads, s);
    else rope_launch<__half, 128>(p, interleaved, grid, threads, s);
  }
  return launched();
}
