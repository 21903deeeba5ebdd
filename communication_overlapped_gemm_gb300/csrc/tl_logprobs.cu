// Log probabilities of chosen tokens, with the entropy of the distribution and its most likely tokens.
#include "tl_serve.cuh"
#include "tl_softmax.cuh"

namespace tl {

// For a row x of logits, c the scale, m the maximum and l = c log2 e, one pass gives
//   z = l (x - m),  S = sum 2^z,  T = sum z 2^z,
//   lse = c m + ln S,   logprob = c (x_t - m) - ln S,   entropy = ln S - ln 2 T / S.
// (x - m comes first: l x of a mask's lowest value would be -inf, and a row of nothing else has no maximum then.)
// Every logit is read once for some thirteen instructions, so HBM bounds it.  A CTA streams a row, or a part of one
// where there are few rows; thread i has the vectors i, i + threads, .. with its own m, S and T.  The parts of a row are
// joined by the CTA that finishes the last one, in their order.
// Measured: 2048 rows of 50001 fp32 logits with the best token 73 to 76 us, 5.4 TB/s, 0.80 of the copy rate (without 68.3, 0.88; with
// the best 20 94), of bf16 51 (46; 65), where instructions bound it (16 bytes of spills at 64 registers); 64 rows of 131072 bf16 with
// the best 5 12.5 us (without 8.6 to 9.5); one row of 131072 fp32 with the best 20 8.7 us, without 5.1: the launch, the logits, the bound, the second look, the part, and the join are waited for in turn.  (One line of all rows cut
// evenly over CTAs that stay: 83 to 99 us and 12; rows beyond the last full round cut in two or three: 81 to 84.)
//
// The most likely k <= 32 tokens need nothing in that loop but the maximum that a thread has anyway.  The k-th
// largest of 32 maxima, of a lane of all warps each, is a bound that at least k logits reach (and few more than k, in no
// order), and only threads whose maximum reaches it can hold one: their vectors are read a second time, from L2, and of
// the logits that reach the bound each counts how many are larger: its place.  An order of 64-bit keys, the value's bits above
// the complement of its index, has no ties (of equal logits the lower index is the larger key).  Logits that are alike in
// great number (masks, rows of one value) would make too many candidates: then only those above the bound are taken, from a
// higher bound if these too are many, and the first ones equal to it are looked up from the row's start, 32 at a time by one
// warp.  That is short where they begin early, as masks do.  Where they lie in the last 2000 of 131072 logits, with lower ones
// before them, one row (cut into parts) takes 53 us, 600 uncut rows 2.3 ms.
struct ScoreParams {
  DevStatus* status;
  const uint8_t* x;
  long long stride;  // bytes
  const int* targets;
  float* logprob;
  float* entropy;
  float* lse;
  float* top_logprob;
  int* top_id;
  float* part;        // [row][split][kPart]
  unsigned* counter;  // [row]
  int rows, vocab, top, splits;
  float scale;
};

namespace score {
constexpr int kTop = 32, kThreads = 256;
// More short rows than there are places for CTAs of 256 threads go to CTAs of 64.  fp32 with the best token: 610 rows of 300 logits 4.6
// us (with 256 threads 8.3), of 4000 6.3 (8.6), of 8000 7.8 (10.1); 2048 rows 7.7 (18.4), 11.1 (19.5), 17.2 (25.3); bf16 with the best
// 5, 610 rows of 8000 8.1 (10.2); 100 rows of 8000 11.7 (6.0).
constexpr int kFewThreads = 64, kShortRow = 8192;
constexpr int kAgain = 2;  // vectors that a thread reads again at once
constexpr int kCandidates = 1024;    // (a join never has more, see below)
constexpr int kPart = 4 + 2 * kTop;  // floats of a part: m, S, T, then its best keys
constexpr int kMaxSplitRows = 2400;  // (a counter for each row that is split)
constexpr int kScoreParts = 640;     // parts of all rows together, beside one a row
using Key = unsigned long long;

// Larger values, larger numbers; NaN the lowest; a zero has one sign.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return o == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ Key key_of(float x, int i) {
  return (static_cast<Key>(order_of(x)) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ int index_of(Key k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

// The k-th largest of the lanes' numbers.
__device__ __forceinline__ uint32_t kth_of_warp(uint32_t v, int k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int j = n / 2; j > 0; j >>= 1) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, v, j);
      v = ((lane & j) == 0) == ((lane & n) == 0) ? max(v, o) : min(v, o);
    }
  return __shfl_sync(0xffffffffu, v, k - 1);
}
// Puts the k largest of n keys (none twice) in their order; the CTA's barrier before and after it.
__device__ __forceinline__ void place_best(const Key* keys, int n, Key* best, int k) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const Key mine = keys[i];
    int larger = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) larger += keys[j] > mine;
    if (larger < k) best[larger] = mine;
  }
}

struct Sums {
  float m, s, t;
};
// Two parts of a row as one.
__device__ __forceinline__ Sums join(Sums a, Sums b, float l2) {
  const float m = fmaxf(a.m, b.m), base = m == -INFINITY ? 0.f : m;
  const float da = a.m == -INFINITY ? 0.f : (a.m - base) * l2, db = b.m == -INFINITY ? 0.f : (b.m - base) * l2;
  const float fa = ex2_approx(da), fb = ex2_approx(db);
  Sums c;
  c.m = m;
  c.s = __fadd_rn(__fmul_rn(a.s, fa), __fmul_rn(b.s, fb));  // (either way round the same)
  // (a part so far below the other that nothing is left of it)
  c.t = __fadd_rn(fa == 0.f ? 0.f : fa * (a.t + da * a.s), fb == 0.f ? 0.f : fb * (b.t + db * b.s));
  return c;
}
// The same in all lanes, whatever their order in a pair.
__device__ __forceinline__ Sums join_warp(Sums a, float l2) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    Sums o;
    o.m = __shfl_xor_sync(0xffffffffu, a.m, j);
    o.s = __shfl_xor_sync(0xffffffffu, a.s, j);
    o.t = __shfl_xor_sync(0xffffffffu, a.t, j);
    a = join(a, o, l2);
  }
  return a;
}

// A 16-byte vector of logits.
template <class T>
struct Logits {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNone = std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;  // -inf
  __device__ static float2 pair(const uint4& v, int i) {
    return to_f32x2<T>(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};
template <>
struct Logits<float> {
  static constexpr int kVec = 4;
  static constexpr uint32_t kNone = 0xff800000u;
  __device__ static float2 pair(const uint4& v, int i) {
    return i == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y)) : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
};

// A row, or a part of it: its logits have the places [off, end), counted from the 16-byte boundary at or before the row.
template <class T>
struct Row {
  static constexpr int kVec = Logits<T>::kVec;
  const uint8_t* base;
  int off, end;
  __device__ float one(int place) const {
    return static_cast<float>(*reinterpret_cast<const T*>(base + static_cast<long long>(place) * static_cast<int>(sizeof(T))));
  }
  // The vector at `place` (a multiple of kVec); -inf where the row is not.
  __device__ uint4 load(long long place) const {
    const uint8_t* at = base + place * static_cast<int>(sizeof(T));
    if (place >= off && place + kVec <= end) return __ldg(reinterpret_cast<const uint4*>(at));
    uint32_t u[4] = {Logits<T>::kNone, Logits<T>::kNone, Logits<T>::kNone, Logits<T>::kNone};
    if (place < end) {
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        if (place + i >= off && place + i < end) {
          if constexpr (sizeof(T) == 4) u[i] = *reinterpret_cast<const uint32_t*>(at + 4 * i);
          else u[i / 2] = __byte_perm(u[i / 2], *reinterpret_cast<const uint16_t*>(at + 2 * i), i & 1 ? 0x5410 : 0x3254);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
}  // namespace score

template <class T, int NV, int kThreads>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) score_kernel(const ScoreParams p) {
  using namespace score;
  constexpr int kVec = Logits<T>::kVec, kWarps = kThreads / 32;
  __shared__ uint32_t s_order[kWarps][32];
  __shared__ Key s_cand[kCandidates], s_best[kTop];
  __shared__ uint8_t s_flag[kThreads];
  __shared__ Sums s_sums[kWarps];
  __shared__ int s_count, s_flags;
  __shared__ unsigned s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  const int target = p.targets ? __ldg(p.targets + row) : 0;
  const uint8_t* x0 = p.x + row * p.stride;
  Row<T> r;
  r.off = static_cast<int>(reinterpret_cast<uintptr_t>(x0) & 15u) / static_cast<int>(sizeof(T));
  r.end = r.off + p.vocab;
  r.base = x0 - r.off * static_cast<int>(sizeof(T));
  const int off = r.off;
  const float l2 = p.scale * kLog2E;
  // this CTA's vectors
  const long long all = (static_cast<long long>(r.end) + kVec - 1) / kVec;
  const int v0 = static_cast<int>(all * split / p.splits), v1 = static_cast<int>(all * (split + 1) / p.splits);
  if (v1 * static_cast<long long>(kVec) < r.end) r.end = v1 * kVec;
  const long long first = static_cast<long long>(v0) * kVec;
  const int count = (v1 - v0 + kThreads - 1) / kThreads;  // vectors of a thread, at most
  if (first > r.off) r.off = static_cast<int>(first);

  Sums sums = {-INFINITY, 0.f, 0.f};
  {
    const long long mine = first + static_cast<int>(threadIdx.x) * kVec;
    uint4 next[NV];
    // The vectors of steps i to i + NV - 1; but at a row's ends all of the CTA's lie within it.
    const int inner = r.end - static_cast<int>(first) >= kThreads * kVec ? (r.end - static_cast<int>(first)) / (kThreads * kVec) : 0;
    auto fetch = [&](int i) {
      if (i + NV <= inner && (i > 0 || first >= r.off)) {
        const uint4* at = reinterpret_cast<const uint4*>(r.base + mine * static_cast<int>(sizeof(T))) + static_cast<long long>(i) * kThreads;
#pragma unroll
        for (int v = 0; v < NV; ++v) next[v] = __ldg(at + v * kThreads);
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v) next[v] = r.load(mine + static_cast<long long>(i + v) * (kThreads * kVec));
      }
    };
    fetch(0);
    if (target < 0) return;
    if (target >= p.vocab) {
      if (split == 0 && threadIdx.x == 0) report_index(p.status, static_cast<unsigned long long>(row));
      return;
    }
    for (int i = 0; i < count; i += NV) {
      uint4 x[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) x[v] = next[v];
      if (i + NV < count) fetch(i + NV);
      float m = sums.m;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {
          const float2 f = Logits<T>::pair(x[v], e);
          m = fmax3(m, f.x, f.y);
        }
      if (m > sums.m) sums = join(sums, Sums{m, 0.f, 0.f}, l2);
      const float top = m == -INFINITY ? 0.f : m;
      const unsigned long long lm = f2(-top, -top), ll = f2(l2, l2);
      unsigned long long ss = f2(0.f, 0.f), tt = ss;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < kVec / 2; ++e) {
          const float2 f = Logits<T>::pair(x[v], e);
          float z0, z1;
          f2_split(fmul2(fadd2(f2(f.x, f.y), lm), ll), z0, z1);
          const unsigned long long w = f2(ex2_approx(z0), ex2_approx(z1));
          ss = fadd2(ss, w);
          tt = ffma2(w, f2(fmaxf(z0, -200.f), fmaxf(z1, -200.f)), tt);  // (of a masked logit 0 times -inf)
        }
      float a, b;
      f2_split(ss, a, b);
      sums.s += a + b;
      f2_split(tt, a, b);
      sums.t += a + b;
    }
  }

  // ---------------------------------------------------------------- the best of the CTA's part
  if (p.top) {
    if (threadIdx.x == 0) s_count = s_flags = 0;
    if (threadIdx.x < kTop) s_best[threadIdx.x] = 0;
    s_order[warp][lane] = order_of(sums.m);
    __syncthreads();
    uint32_t o = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) o = max(o, s_order[w][lane]);
    float bound = value_of(kth_of_warp(o, p.top));
    bool equal = bound > -INFINITY;  // (masked logits, if they are wanted at all, are looked up below)
    int n;
    for (;;) {
      if (equal ? sums.m >= bound : sums.m > bound) s_flag[atomicAdd(&s_flags, 1)] = static_cast<uint8_t>(threadIdx.x);
      __syncthreads();
      const int flags = s_flags, items = flags * count;
      for (int i0 = threadIdx.x; i0 < items; i0 += kAgain * kThreads) {
        uint4 x[kAgain];
        long long place[kAgain];
#pragma unroll
        for (int u = 0; u < kAgain; ++u) {
          const int i = i0 + u * kThreads, nth = i / flags;
          place[u] = i < items ? first + (static_cast<long long>(nth) * kThreads + s_flag[i - nth * flags]) * kVec : r.end;
          x[u] = r.load(place[u]);
        }
#pragma unroll
        for (int u = 0; u < kAgain; ++u) {
          float top = -INFINITY;
#pragma unroll
          for (int e = 0; e < kVec / 2; ++e) {
            const float2 f = Logits<T>::pair(x[u], e);
            top = fmax3(top, f.x, f.y);
          }
          if (equal ? top >= bound : top > bound)
#pragma unroll
            for (int e = 0; e < kVec; ++e) {
              const float2 f = Logits<T>::pair(x[u], e / 2);
              const float y = e & 1 ? f.y : f.x;
              const long long at = place[u] + e;
              if ((equal ? y >= bound : y > bound) && at >= r.off && at < r.end) {
                const int k = atomicAdd(&s_count, 1);
                if (k < kCandidates) s_cand[k] = key_of(y, static_cast<int>(at) - off);
              }
            }
        }
      }
      __syncthreads();
      n = s_count;
      place_best(s_cand, n < kCandidates ? n : kCandidates, s_best, p.top);
      __syncthreads();
      if (n <= kCandidates) break;
      if (!equal) bound = value_of(static_cast<uint32_t>(s_best[p.top - 1] >> 32));
      equal = false;
      if (threadIdx.x == 0) s_count = s_flags = 0;
      __syncthreads();
      if (threadIdx.x < kTop) s_best[threadIdx.x] = 0;
    }
    if (warp == 0 && n < p.top) {
      // fewer than k above the bound: the first ones equal to it, then NaN (and where both are too few, the part is)
      for (int pass = equal ? 1 : 0; pass < 2 && n < p.top; ++pass)
        for (int i = r.off; i < r.end && n < p.top; i += 32) {
          const bool there = i + lane < r.end;
          const float y = there ? r.one(i + lane) : 0.f;
          const bool hit = there && (pass ? y != y : y == bound);
          const unsigned hits = __ballot_sync(0xffffffffu, hit);
          const int nth = n + __popc(hits & ((1u << lane) - 1u));
          if (hit && nth < p.top) s_best[nth] = key_of(y, i + lane - off);
          n += __popc(hits);
        }
      __syncwarp();
    }
  }

  // ---------------------------------------------------------------- the CTA's part of the row
  sums = join_warp(sums, l2);
  if (lane == 0) s_sums[warp] = sums;
  __syncthreads();
  if (warp == 0) sums = join_warp(lane < kWarps ? s_sums[lane] : Sums{-INFINITY, 0.f, 0.f}, l2);
  if (p.splits > 1) {
    const float* parts = p.part + static_cast<size_t>(row) * p.splits * kPart;
    if (warp == 0) {
      float* part = p.part + (static_cast<size_t>(row) * p.splits + split) * kPart;
      if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(sums.m, sums.s, sums.t, 0.f);
      if (p.top) reinterpret_cast<Key*>(part + 4)[lane] = s_best[lane];
      __threadfence();
      __syncwarp();
      if (lane == 0) {
        const unsigned done = atomicAdd(p.counter + row, 1u) + 1u;
        s_last = done == static_cast<unsigned>(p.splits);
        if (s_last) p.counter[row] = 0u;
        __threadfence();
      }
    }
    __syncthreads();
    if (!s_last) return;
    if (p.top) {
      // With j = k / splits and need = k / j (both rounded up), `need` of the parts' j-th keys reach the need-th largest of them: so do
      // k keys.  No part has more than k, and of the other parts fewer than j each reach it: need k + (splits - need) (j - 1) at
      // most, which is k k for j = 1 and less otherwise.
      static_assert(kTop * kTop <= kCandidates && kScoreParts <= kCandidates, "a join's keys");
      const Key* keys = reinterpret_cast<const Key*>(parts + 4);
      constexpr int kStride = kPart / 2;
      const int nth = (p.top + p.splits - 1) / p.splits, need = (p.top + nth - 1) / nth;
      if (threadIdx.x == 0) s_count = 0;
      for (int s = threadIdx.x; s < p.splits; s += kThreads) s_cand[s] = __ldcg(keys + static_cast<size_t>(s) * kStride + nth - 1);
      constexpr int kAhead = 4;  // keys of a thread that are on their way meanwhile
      const int all_keys = p.splits * kTop;
      Key held[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = threadIdx.x + u * kThreads;
        held[u] = i < all_keys && i % kTop < p.top ? __ldcg(keys + static_cast<size_t>(i / kTop) * kStride + i % kTop) : 0;
      }
      __syncthreads();
      for (int s = threadIdx.x; s < p.splits; s += kThreads) {
        // (equal ones are zeros, from parts of fewer keys)
        const Key mine = s_cand[s];
        int larger = 0, same = 0;
#pragma unroll 8
        for (int i = 0; i < p.splits; ++i) {
          larger += s_cand[i] > mine;
          same += s_cand[i] == mine && i < s;
        }
        if (larger + same == need - 1) s_best[0] = mine;
      }
      __syncthreads();
      const Key bound = s_best[0] > 0 ? s_best[0] : 1;
      __syncthreads();
      if (threadIdx.x < kTop) s_best[threadIdx.x] = 0;
      auto keep = [&](Key k) {
        if (k >= bound) {
          const int c = atomicAdd(&s_count, 1);
          if (c < kCandidates) s_cand[c] = k;
        }
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u) keep(held[u]);
      for (int i = threadIdx.x + kAhead * kThreads; i < all_keys; i += kThreads)
        if (i % kTop < p.top) keep(__ldcg(keys + static_cast<size_t>(i / kTop) * kStride + i % kTop));
      __syncthreads();
      place_best(s_cand, min(s_count, kCandidates), s_best, p.top);
      __syncthreads();
    }
    if (warp == 0) {
      sums = {-INFINITY, 0.f, 0.f};
      for (int s = lane; s < p.splits; s += 32) {
        const float4 o = __ldcg(reinterpret_cast<const float4*>(parts + static_cast<size_t>(s) * kPart));
        sums = join(sums, Sums{o.x, o.y, o.z}, l2);
      }
      sums = join_warp(sums, l2);
    }
  }
  if (warp != 0) return;
  const bool none = sums.m == -INFINITY && sums.s == 0.f;  // every logit is -inf
  const float ln = logf(sums.s);
  if (lane == 0) {
    if (p.logprob) p.logprob[row] = none ? -INFINITY : (r.one(off + target) - sums.m) * p.scale - ln;
    if (p.entropy) p.entropy[row] = none ? 0.f : ln - kLn2 * (sums.t / sums.s);
    if (p.lse) p.lse[row] = none ? -INFINITY : fmaf(sums.m, p.scale, ln);
  }
  if (lane < p.top) {
    const long long at = static_cast<long long>(row) * p.top + lane;
    const Key best = s_best[lane];
    p.top_id[at] = index_of(best);
    p.top_logprob[at] = none ? -INFINITY : (value_of(static_cast<uint32_t>(best >> 32)) - sums.m) * p.scale - ln;
  }
}

// The parts that a row is cut into: three CTAs an SM of all rows (64 bf16 rows of 131072 without best tokens 9.5 us; two 10.1, four
// 10.7; 300 fp32 rows with 5 33, 33 and 43), none of less than 4096 logits (one row with the best 20: 8.9 us; 2048 10.4, 8192 9.5).
static int score_splits(int rows, int vocab, int sms) {
  if (rows <= 0 || rows > score::kMaxSplitRows) return 1;
  int places = 3 * sms < score::kScoreParts ? 3 * sms : score::kScoreParts;
  const int s = (places + rows - 1) / rows, most = vocab / (score::kThreads * 16);
  return s < most ? s : most < 1 ? 1 : most;
}

}  // namespace tl

using namespace tl;

extern "C" size_t tl_token_logprobs_workspace_bytes(int rows, int vocab, int top) {
  if (rows < 0 || vocab < 1 || top < 0 || top > score::kTop || top > vocab) return 0;
  const size_t parts = rows > score::kMaxSplitRows ? 0 : static_cast<size_t>(rows) + score::kScoreParts;
  return kCounterBytes + parts * score::kPart * 4;
}

extern "C" int tl_token_logprobs(tl_ctx* ctx, int dtype, const void* logits, long long row_stride, const int* targets,
                                 float* logprob, float* entropy, float* lse, float* top_logprobs, int* top_ids, int top,
                                 float scale, int rows, int vocab, void* workspace, size_t workspace_bytes,
                                 tl_stream_t stream) {
  if (!ctx || (dtype != TL_BF16 && dtype != TL_FP16 && dtype != TL_FP32) || rows < 0 || vocab < 1 || vocab > (1 << 30) || top < 0 ||
      top > score::kTop || top > vocab || row_stride < 0 || !scale_ok(scale))
    return TL_ERR_INVALID;
  if (rows == 0) return TL_OK;
  if (rows > (1 << 24) || !logits || reinterpret_cast<uintptr_t>(logits) % (dtype == TL_FP32 ? 4 : 2) != 0 || !workspace || !aligned16(workspace) || (logprob && !targets) ||
      (top > 0 && (!top_logprobs || !top_ids)))
    return TL_ERR_INVALID;
  if (workspace_bytes < tl_token_logprobs_workspace_bytes(rows, vocab, top)) return TL_ERR_WORKSPACE;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  ScoreParams p;
  const int es = dtype == TL_FP32 ? 4 : 2;
  p.status = ctx->status;
  p.x = static_cast<const uint8_t*>(logits);
  p.stride = row_stride * es;
  p.targets = targets;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.top_logprob = top_logprobs;
  p.top_id = top_ids;
  p.counter = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  p.rows = rows;
  p.vocab = vocab;
  p.top = top;
  p.scale = scale;
  p.splits = score_splits(rows, vocab, ctx->sms);
  const unsigned grid = static_cast<unsigned>(rows) * p.splits;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (vocab <= score::kShortRow && rows > 4 * ctx->sms) {
    if (dtype == TL_FP32) score_kernel<float, 5, score::kFewThreads><<<grid, score::kFewThreads, 0, s>>>(p);
    else if (dtype == TL_BF16) score_kernel<__nv_bfloat16, 4, score::kFewThreads><<<grid, score::kFewThreads, 0, s>>>(p);
    else score_kernel<__half, 4, score::kFewThreads><<<grid, score::kFewThreads, 0, s>>>(p);
  } else {
    if (dtype == TL_FP32) score_kernel<float, 5, score::kThreads><<<grid, score::kThreads, 0, s>>>(p);
    else if (dtype == TL_BF16) score_kernel<__nv_bfloat16, 4, score::kThreads><<<grid, score::kThreads, 0, s>>>(p);
    else score_kernel<__half, 4, score::kThreads><<<grid, score::kThreads, 0, s>>>(p);
  }
  return launched();
}
