// The paged key/value cache: appending new rows, and the attention of one new token over it.
#include "tl_serve.cuh"

namespace tl {

struct CacheArgs {
  uint8_t* k;
  uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  long long page_stride, row_stride, head_stride;  // bytes
  int num_pages, page_size, kv_heads;
};

// ---------------------------------------------------------------------------- append
// One thread per 8 elements of a K and of a V row: 16 bytes read and 16 (8 for e4m3) written.
struct AppendParams {
  CacheArgs c;
  DevStatus* status;
  const uint8_t* k;
  const uint8_t* v;
  long long k_token, k_head, v_token, v_head;  // bytes
  const int* slots;
  int tokens;
};

// 8 elements of T divided by the scale, as e4m3 (nearest even, saturating; NaN stays NaN).
template <class T>
__device__ __forceinline__ uint2 quantise8(uint4 x, float scale) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = to_f32x2<T>(in[i]);
    out[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, scale), __fdiv_rn(f.y, scale)), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
}

template <class T, bool Fp8, int D>
__global__ void __launch_bounds__(256) append_kernel(const AppendParams p) {
  constexpr int kVec = D / 8;
  const long long n = static_cast<long long>(p.tokens) * p.c.kv_heads * kVec;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<long long>(gridDim.x) * blockDim.x) {
    const int vec = static_cast<int>(i % kVec);
    const long long th = i / kVec;
    const int h = static_cast<int>(th % p.c.kv_heads), t = static_cast<int>(th / p.c.kv_heads);
    const int slot = p.slots[t];
    if (slot < 0) continue;
    const int page = slot / p.c.page_size;
    if (page >= p.c.num_pages) {
      if (h == 0 && vec == 0) report_index(p.status, static_cast<unsigned long long>(t));
      continue;
    }
    const long long at = page * p.c.page_stride + (slot - page * p.c.page_size) * p.c.row_stride + h * p.c.head_stride;
    const uint4 k = __ldg(reinterpret_cast<const uint4*>(p.k + t * p.k_token + h * p.k_head) + vec);
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.v + t * p.v_token + h * p.v_head) + vec);
    if constexpr (Fp8) {
      reinterpret_cast<uint2*>(p.c.k + at)[vec] = quantise8<T>(k, p.c.k_scale ? p.c.k_scale[h] : 1.f);
      reinterpret_cast<uint2*>(p.c.v + at)[vec] = quantise8<T>(v, p.c.v_scale ? p.c.v_scale[h] : 1.f);
    } else {
      reinterpret_cast<uint4*>(p.c.k + at)[vec] = k;
      reinterpret_cast<uint4*>(p.c.v + at)[vec] = v;
    }
  }
}

// ---------------------------------------------------------------------------- attention of one token
struct PagedParams {
  CacheArgs c;
  DevStatus* status;
  const uint8_t* q;
  uint8_t* out;
  float* lse;
  long long q_seq, q_head, out_seq, out_head;  // bytes
  const int* table;
  const int* lengths;
  int max_pages, batch, heads;
  float scale;
  int window, sinks;
};

// The visible rows of a sequence of n, counted from 0: the first `head` are rows [0, head), the
// rest rows [skip + head, n).
struct Visible {
  int count, head, skip;
};
__device__ __forceinline__ Visible visible_rows(int n, int window, int sinks) {
  Visible v;
  if (window == 0 || n <= window || sinks >= n - window) {
    v.count = n;
    v.head = n;
    v.skip = 0;
  } else {
    v.head = sinks;
    v.skip = n - window - sinks;
    v.count = window + sinks;
  }
  return v;
}

// One CTA per (sequence, query head), a warp per key in turn with its own running maximum and
// sum, joined at the end: the plain form of the operator.
template <class T, bool Fp8, int D>
__global__ void __launch_bounds__(256) paged_kernel(const PagedParams p) {
  constexpr int kPer = D / 32, kWarps = 8;
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int b = blockIdx.x, h = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = h / (p.heads / p.c.kv_heads);
  int n = p.lengths[b];
  const long long cap = static_cast<long long>(p.max_pages) * p.c.page_size;
  if (n < 0 || n > cap) {
    if (threadIdx.x == 0) report_index(p.status, static_cast<unsigned long long>(b));
    n = n < 0 ? 0 : static_cast<int>(cap);
  }
  const Visible vis = visible_rows(n, p.window, p.sinks);
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
  const T* qp = reinterpret_cast<const T*>(p.q + b * p.q_seq + h * p.q_head);
  const float sc = p.scale * kLog2E * (Fp8 && p.c.k_scale ? p.c.k_scale[hk] : 1.f);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = static_cast<float>(qp[lane * kPer + i]);
    o[i] = 0.f;
  }
  for (int i = warp; i < vis.count; i += kWarps) {
    const int row = i < vis.head ? i : i + vis.skip;
    const int pg = row / p.c.page_size;
    const int page = p.table[static_cast<long long>(b) * p.max_pages + pg];
    if (page < 0 || page >= p.c.num_pages) {
      if (lane == 0) report_index(p.status, static_cast<unsigned long long>(b));
      continue;
    }
    const long long at = page * p.c.page_stride + (row - pg * p.c.page_size) * p.c.row_stride + hk * p.c.head_stride;
    float k[kPer], v[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if constexpr (Fp8) {
        k[j] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(p.c.k + at)[lane * kPer + j]);
        v[j] = static_cast<float>(reinterpret_cast<const __nv_fp8_e4m3*>(p.c.v + at)[lane * kPer + j]);
      } else {
        k[j] = static_cast<float>(reinterpret_cast<const T*>(p.c.k + at)[lane * kPer + j]);
        v[j] = static_cast<float>(reinterpret_cast<const T*>(p.c.v + at)[lane * kPer + j]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < kPer; ++j) s += q[j] * k[j];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= sc;
    const float mn = fmaxf(m, s);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - mn), w = s == -INFINITY ? 0.f : exp2f(s - mn);
    m = mn;
    l = l * keep + w;
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] = o[j] * keep + w * v[j];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) s_o[warp][lane * kPer + j] = o[j];
  __syncthreads();
  if (threadIdx.x >= D) return;
  float mm = -INFINITY, ll = 0.f, acc = 0.f;
  for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
  for (int w = 0; w < kWarps; ++w) {
    const float f = s_m[w] == -INFINITY ? 0.f : exp2f(s_m[w] - mm);
    ll += f * s_l[w];
    acc += f * s_o[w][threadIdx.x];
  }
  const bool none = ll == 0.f;
  const float vs = Fp8 && p.c.v_scale ? p.c.v_scale[hk] : 1.f;
  reinterpret_cast<T*>(p.out + b * p.out_seq + h * p.out_head)[threadIdx.x] = static_cast<T>(none ? 0.f : acc / ll * vs);
  if (p.lse && threadIdx.x == 0)
    p.lse[static_cast<long long>(b) * p.heads + h] = none ? -INFINITY : mm * kLn2 + logf(ll);
}

// ---------------------------------------------------------------------------- host side
static bool cache_ok(const tl_paged_cache* c, int dtype) {
  if (!c || (dtype != TL_BF16 && dtype != TL_FP16) || (c->dtype != dtype && c->dtype != TL_E4M3)) return false;
  const int es = c->dtype == TL_E4M3 ? 1 : 2;
  if (c->num_pages < 0 || c->page_size < 1 || c->kv_heads < 0 || (c->d != 64 && c->d != 128)) return false;
  if (static_cast<long long>(c->num_pages) * c->page_size >= (1LL << 31)) return false;
  if (!esize_ok(c->page_stride, es) || !esize_ok(c->row_stride, es) || !esize_ok(c->head_stride, es)) return false;
  if (c->dtype != TL_E4M3 && (c->k_scale || c->v_scale)) return false;
  if (c->num_pages > 0 && c->kv_heads > 0 && (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v))) return false;
  return true;
}

static CacheArgs cache_args(const tl_paged_cache* c) {
  const int es = c->dtype == TL_E4M3 ? 1 : 2;
  CacheArgs a;
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  a.k_scale = c->k_scale;
  a.v_scale = c->v_scale;
  a.page_stride = c->page_stride * es;
  a.row_stride = c->row_stride * es;
  a.head_stride = c->head_stride * es;
  a.num_pages = c->num_pages;
  a.page_size = c->page_size;
  a.kv_heads = c->kv_heads;
  return a;
}

static int launched() {
  if (cudaGetLastError() != cudaSuccess) return TL_ERR_CUDA;
  return TL_OK;
}

// f(T{}, Fp8, D) for the call's types, as compile-time values.
template <class F>
static int dispatch(int dtype, int cache_dtype, int d, F&& f) {
  const bool fp8 = cache_dtype == TL_E4M3;
  auto with_d = [&](auto t, auto fp8c) {
    return d == 64 ? f(t, fp8c, std::integral_constant<int, 64>{}) : f(t, fp8c, std::integral_constant<int, 128>{});
  };
  auto with_t = [&](auto t) { return fp8 ? with_d(t, std::true_type{}) : with_d(t, std::false_type{}); };
  return dtype == TL_BF16 ? with_t(__nv_bfloat16{}) : with_t(__half{});
}

}  // namespace tl

using namespace tl;

extern "C" int tl_kv_append(tl_ctx* ctx, const tl_paged_cache* cache, int dtype, const void* k, const void* v,
                            long long k_token_stride, long long k_head_stride, long long v_token_stride,
                            long long v_head_stride, const int* slots, int tokens, tl_stream_t stream) {
  if (!ctx || !cache_ok(cache, dtype) || tokens < 0) return TL_ERR_INVALID;
  if (!esize_ok(k_token_stride, 2) || !esize_ok(k_head_stride, 2) || !esize_ok(v_token_stride, 2) ||
      !esize_ok(v_head_stride, 2))
    return TL_ERR_INVALID;
  if (tokens == 0 || cache->kv_heads == 0) return TL_OK;
  if (!k || !v || !slots || !aligned16(k) || !aligned16(v)) return TL_ERR_INVALID;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  AppendParams p;
  p.c = cache_args(cache);
  p.status = ctx->status;
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.k_token = 2 * k_token_stride;
  p.k_head = 2 * k_head_stride;
  p.v_token = 2 * v_token_stride;
  p.v_head = 2 * v_head_stride;
  p.slots = slots;
  p.tokens = tokens;
  const long long n = static_cast<long long>(tokens) * cache->kv_heads * (cache->d / 8);
  const long long need = (n + 255) / 256, most = 8LL * ctx->sms;
  return dispatch(dtype, cache->dtype, cache->d, [&](auto t, auto fp8, auto d) {
    append_kernel<decltype(t), decltype(fp8)::value, decltype(d)::value>
        <<<static_cast<unsigned>(need < most ? need : most), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched();
  });
}

extern "C" size_t tl_paged_attention_workspace_bytes(int batch, int heads, int kv_heads, int d) {
  if (batch < 0 || batch > 4096 || !heads_ok(heads, kv_heads, d)) return 0;
  return 256;
}

extern "C" int tl_paged_attention(tl_ctx* ctx, const tl_paged_cache* cache, int dtype, const void* q,
                                  long long q_seq_stride, long long q_head_stride, const int* page_table, int max_pages,
                                  const int* lengths, void* out, long long out_seq_stride, long long out_head_stride,
                                  float* lse, int batch, int heads, float scale, int window, int sinks, void* workspace,
                                  size_t workspace_bytes, tl_stream_t stream) {
  if (!ctx || !cache_ok(cache, dtype) || batch < 0 || batch > 4096 || !heads_ok(heads, cache->kv_heads, cache->d) ||
      max_pages < 0 || window < 0 || sinks < 0 || !(scale > 0.f) || scale > 3.0e38f)
    return TL_ERR_INVALID;
  if (static_cast<long long>(max_pages) * cache->page_size >= (1LL << 31)) return TL_ERR_INVALID;
  if (!esize_ok(q_seq_stride, 2) || !esize_ok(q_head_stride, 2) || !esize_ok(out_seq_stride, 2) ||
      !esize_ok(out_head_stride, 2))
    return TL_ERR_INVALID;
  if (batch == 0 || heads == 0) return TL_OK;
  if (!q || !out || !lengths || (!page_table && max_pages > 0) || !workspace || !aligned16(q) || !aligned16(out) ||
      !aligned16(workspace))
    return TL_ERR_INVALID;
  if (workspace_bytes < tl_paged_attention_workspace_bytes(batch, heads, cache->kv_heads, cache->d))
    return TL_ERR_WORKSPACE;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  PagedParams p;
  p.c = cache_args(cache);
  p.status = ctx->status;
  p.q = static_cast<const uint8_t*>(q);
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.q_seq = 2 * q_seq_stride;
  p.q_head = 2 * q_head_stride;
  p.out_seq = 2 * out_seq_stride;
  p.out_head = 2 * out_head_stride;
  p.table = page_table;
  p.lengths = lengths;
  p.max_pages = max_pages;
  p.batch = batch;
  p.heads = heads;
  p.scale = scale;
  p.window = window;
  p.sinks = sinks;
  return dispatch(dtype, cache->dtype, cache->d, [&](auto t, auto fp8, auto d) {
    paged_kernel<decltype(t), decltype(fp8)::value, decltype(d)::value>
        <<<dim3(batch, heads), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched();
  });
}
