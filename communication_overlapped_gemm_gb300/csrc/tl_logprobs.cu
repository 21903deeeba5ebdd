// Log probabilities of chosen tokens, with the entropy of the distribution and its most likely tokens.
#include "tl_serve.cuh"

namespace tl {

// For a row x of logits, c the scale, m the maximum and l = c log2 e, one pass gives
//   z = l (x - m),  S = sum 2^z,  T = sum z 2^z,
//   lse = c m + ln S,   logprob = c (x_t - m) - ln S,   entropy = ln S - ln 2 T / S.
// (x - m comes first: l x of a mask's lowest value would be -inf, and a row of nothing else has no maximum then.)
// Every logit is read once for some ten instructions, so HBM bounds it.  A CTA takes a chunk of a row at a time
// into registers, 32 values a thread, each thread with its own m, S and T; few rows are cut into parts, which the CTA
// that finishes a row's last part joins.
//
// The most likely k <= 32 tokens: an order of 64-bit keys, the value's bits above the complement of its index, has
// no ties (equal values: the lower index is the larger key).  In a chunk the k-th largest of the 256
// threads' maxima is a bound that at least k keys reach, and only the k threads with such a maximum can hold one: at
// most 32 k candidates, whatever the logits are (ties, masked stretches, sorted rows).  A warp sorts 32 keys by
// exchanges between lanes, and two sorted lists merge into their best 32 in 6 steps.
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
  int rows, vocab, top, splits, chunks;  // chunks of a row
  float scale;
};

namespace score {
constexpr int kThreads = 256, kWarps = kThreads / 32, kTop = 32;
constexpr int kPart = 4 + 2 * kTop;  // floats of a part: m, S, T, then its best keys
constexpr int kMaxSplitRows = 1024;  // (a counter for each row that is split)
using Key = unsigned long long;

__device__ __forceinline__ Key key_of(float x, int i) {
  const uint32_t b = __float_as_uint(x + 0.f);  // (a zero has one sign)
  const uint32_t o = x != x ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return (static_cast<Key>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float value_of(Key k) {
  const uint32_t o = static_cast<uint32_t>(k >> 32);
  return o == 0u ? __uint_as_float(0x7fffffffu) : __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int index_of(Key k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

__device__ __forceinline__ Key exchange(Key k, int j, bool larger) {
  const Key o = __shfl_xor_sync(0xffffffffu, k, j);
  return (k > o) == larger ? k : o;
}
// The largest first, a key a lane.
__device__ __forceinline__ Key sort32(Key k) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 2; n <= 32; n <<= 1)
#pragma unroll
    for (int j = n / 2; j > 0; j >>= 1) k = exchange(k, j, ((lane & j) == 0) == ((lane & n) == 0));
  return k;
}
// The best 32 of two sorted lists, sorted.
__device__ __forceinline__ Key merge32(Key a, Key b) {
  const int lane = threadIdx.x & 31;
  const Key o = __shfl_xor_sync(0xffffffffu, b, 31);
  Key k = a > o ? a : o;
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) k = exchange(k, j, (lane & j) == 0);
  return k;
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
  c.s = a.s * fa + b.s * fb;
  // (a part so far below the other that nothing is left of it)
  c.t = (fa == 0.f ? 0.f : fa * (a.t + da * a.s)) + (fb == 0.f ? 0.f : fb * (b.t + db * b.s));
  return c;
}
}  // namespace score

template <class T>
struct Logits {
  static constexpr int kVec = 8;
  __device__ static void unpack(uint4 v, float* x) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = to_f32x2<T>(u[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  __device__ static float one(const uint8_t* p) { return static_cast<float>(*reinterpret_cast<const T*>(p)); }
};
template <>
struct Logits<float> {
  static constexpr int kVec = 4;
  __device__ static void unpack(uint4 v, float* x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  __device__ static float one(const uint8_t* p) { return *reinterpret_cast<const float*>(p); }
};

template <class T, int NV>
__global__ void __launch_bounds__(score::kThreads) score_kernel(const ScoreParams p) {
  using namespace score;
  constexpr int kVec = Logits<T>::kVec, kVals = NV * kVec, kChunk = kThreads * kVals;
  __shared__ Key s_list[kWarps][kTop];
  __shared__ Key s_cand[kTop * kVals];
  __shared__ Sums s_sums[kWarps];
  __shared__ int s_count;
  __shared__ unsigned s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x / p.splits, split = blockIdx.x - row * p.splits;
  int target = 0;
  if (p.targets) {
    target = __ldg(p.targets + row);
    if (target < 0) return;
    if (target >= p.vocab) {
      if (split == 0 && threadIdx.x == 0) report_index(p.status, static_cast<unsigned long long>(row));
      return;
    }
  }
  const uint8_t* x0 = p.x + row * p.stride;
  // places are counted from the 16-byte boundary at or before the row
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x0) & 15u) / static_cast<int>(sizeof(T));
  const int end = off + p.vocab;
  const uint8_t* base = x0 - off * static_cast<int>(sizeof(T));
  const float l2 = p.scale * kLog2E;
  const int c0 = static_cast<int>(static_cast<long long>(p.chunks) * split / p.splits);
  const int c1 = static_cast<int>(static_cast<long long>(p.chunks) * (split + 1) / p.splits);

  Sums sums = {-INFINITY, 0.f, 0.f};
  Key best = 0;  // warp 0: the best keys so far, sorted
  Key bound = 0; // the k-th of them
  for (int c = c0; c < c1; ++c) {
    const long long first = static_cast<long long>(c) * kChunk;
    if (first >= end) break;
    float x[kVals];
    int at[NV];  // the place of a vector's first value
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const long long place = first + (v * kThreads + static_cast<int>(threadIdx.x)) * kVec;
      at[v] = place < end ? static_cast<int>(place) : end;
      if (at[v] >= off && at[v] + kVec <= end) {
        Logits<T>::unpack(__ldcs(reinterpret_cast<const uint4*>(base + static_cast<long long>(at[v]) * static_cast<int>(sizeof(T)))), x + v * kVec);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int e = at[v] + i;
          x[v * kVec + i] = e >= off && e < end ? Logits<T>::one(base + static_cast<long long>(e) * static_cast<int>(sizeof(T))) : -INFINITY;
        }
      }
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kVals; ++i) m = fmaxf(m, x[i]);
    sums = join(sums, Sums{m, 0.f, 0.f}, l2);
    const float top = sums.m == -INFINITY ? 0.f : sums.m;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const float z = (x[i] - top) * l2, w = ex2_approx(z);
      sums.s += w;
      sums.t = fmaf(w, fmaxf(z, -200.f), sums.t);
    }
    if (p.top == 0) continue;
    // ---------------------------------------------------------------- the best of this chunk
    Key mine = 0;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int e = at[v] + i;
        if (e >= off && e < end) {
          const Key k = key_of(x[v * kVec + i], e - off);
          if (k > mine) mine = k;
        }
      }
    if (!__syncthreads_or(mine > bound)) continue;
    if (threadIdx.x == 0) s_count = 0;
    Key list = sort32(mine);
    s_list[warp][lane] = list;
    __syncthreads();
#pragma unroll
    for (int n = kWarps / 2; n > 0; n >>= 1) {
      if (warp < n) {
        list = merge32(list, s_list[warp + n][lane]);
        s_list[warp][lane] = list;
      }
      __syncthreads();
    }
    const Key low = s_list[0][p.top - 1], least = low > bound ? low : bound;
    if (mine >= least && mine > 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const int e = at[v] + i;
          if (e >= off && e < end) {
            const Key k = key_of(x[v * kVec + i], e - off);
            if (k >= least) s_cand[atomicAdd(&s_count, 1)] = k;
          }
        }
    }
    __syncthreads();
    if (warp == 0) {
      const int n = s_count;
      for (int i = 0; i < n; i += 32) best = merge32(best, sort32(i + lane < n ? s_cand[i + lane] : 0));
      s_list[0][lane] = best;
    }
    __syncthreads();
    bound = s_list[0][p.top - 1];
    __syncthreads();
  }

  // ---------------------------------------------------------------- the CTA's part of the row
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) {
    Sums o;
    o.m = __shfl_xor_sync(0xffffffffu, sums.m, j);
    o.s = __shfl_xor_sync(0xffffffffu, sums.s, j);
    o.t = __shfl_xor_sync(0xffffffffu, sums.t, j);
    sums = join(sums, o, l2);
  }
  if (lane == 0) s_sums[warp] = sums;
  __syncthreads();
  if (warp != 0 && p.splits == 1) return;
  if (warp == 0) {
    sums = s_sums[0];
    for (int w = 1; w < kWarps; ++w) sums = join(sums, s_sums[w], l2);
  }
  if (p.splits > 1) {
    float* part = p.part + (static_cast<size_t>(row) * p.splits + split) * kPart;
    if (warp == 0) {
      if (lane == 0) *reinterpret_cast<float4*>(part) = make_float4(sums.m, sums.s, sums.t, 0.f);
      if (p.top) reinterpret_cast<Key*>(part + 4)[lane] = best;
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
    // the row's parts, in their order
    if (warp != 0) return;
    sums = {-INFINITY, 0.f, 0.f};
    best = 0;
    for (int s = 0; s < p.splits; ++s) {
      const float* src = p.part + (static_cast<size_t>(row) * p.splits + s) * kPart;
      const float4 o = __ldcg(reinterpret_cast<const float4*>(src));
      sums = join(sums, Sums{o.x, o.y, o.z}, l2);
      if (p.top) best = merge32(best, __ldcg(reinterpret_cast<const Key*>(src + 4) + lane));
    }
  }
  const bool none = sums.m == -INFINITY && sums.s == 0.f;  // every logit is -inf
  const float ln = logf(sums.s);
  if (lane == 0) {
    if (p.logprob)
      p.logprob[row] = none ? -INFINITY : (Logits<T>::one(x0 + target * static_cast<long long>(sizeof(T))) - sums.m) * p.scale - ln;
    if (p.entropy) p.entropy[row] = none ? 0.f : ln - kLn2 * (sums.t / sums.s);
    if (p.lse) p.lse[row] = none ? -INFINITY : fmaf(sums.m, p.scale, ln);
  }
  if (lane < p.top) {
    const long long at = static_cast<long long>(row) * p.top + lane;
    p.top_id[at] = index_of(best);
    p.top_logprob[at] = none ? -INFINITY : (value_of(best) - sums.m) * p.scale - ln;
  }
}

// The parts that a row is cut into: as many as fill the SMs, no finer than a chunk.
static int score_splits(int rows, int chunks, int sms) {
  if (rows <= 0 || rows > score::kMaxSplitRows) return 1;
  int s = (2 * sms + rows - 1) / rows;
  return s < chunks ? s : chunks;
}
constexpr int kScoreVals = 32;  // values of a thread
static int score_chunks(int vocab) { return (vocab + 7 + score::kThreads * kScoreVals - 1) / (score::kThreads * kScoreVals); }

}  // namespace tl

using namespace tl;

extern "C" size_t tl_token_logprobs_workspace_bytes(int rows, int vocab, int top) {
  if (rows < 0 || vocab < 1 || top < 0 || top > score::kTop || top > vocab) return 0;
  const size_t split_rows = rows < score::kMaxSplitRows ? rows : score::kMaxSplitRows;
  // (at most 2 splits for each of at most 320 SMs beside one a row)
  const size_t chunks = score_chunks(vocab);
  const size_t parts = split_rows + 640 < split_rows * chunks ? split_rows + 640 : split_rows * chunks;
  return kCounterBytes + parts * score::kPart * 4;
}

extern "C" int tl_token_logprobs(tl_ctx* ctx, int dtype, const void* logits, long long row_stride, const int* targets,
                                 float* logprob, float* entropy, float* lse, float* top_logprobs, int* top_ids, int top,
                                 float scale, int rows, int vocab, void* workspace, size_t workspace_bytes,
                                 tl_stream_t stream) {
  if (!ctx || (dtype != TL_BF16 && dtype != TL_FP16 && dtype != TL_FP32) || rows < 0 || vocab < 1 || vocab > (1 << 30) || top < 0 ||
      top > score::kTop || top > vocab || row_stride < 0 || !(scale > 0.f) || scale > 3.0e38f)
    return TL_ERR_INVALID;
  if (rows == 0) return TL_OK;
  if (rows > (1 << 24) || !logits || !aligned16(logits) || !workspace || !aligned16(workspace) || (logprob && !targets) ||
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
  p.chunks = score_chunks(vocab);
  p.splits = score_splits(rows, p.chunks, ctx->sms < 320 ? ctx->sms : 320);
  const unsigned grid = static_cast<unsigned>(rows) * p.splits;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TL_FP32) score_kernel<float, 8><<<grid, score::kThreads, 0, s>>>(p);
  else if (dtype == TL_BF16) score_kernel<__nv_bfloat16, 4><<<grid, score::kThreads, 0, s>>>(p);
  else score_kernel<__half, 4><<<grid, score::kThreads, 0, s>>>(p);
  return launched();
}
