// Causal attention of packed prompts with a sliding window and sinks.
#include "tl_serve.cuh"

namespace tl {

struct WindowParams {
  DevStatus* status;
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* out;
  float* lse;
  long long q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;  // bytes
  const int* cu_q;
  const int* cu_k;
  int batch, total_q, total_k, heads, group;
  float sl2;  // scale * log2(e)
  int window, sinks;
};

// The keys a query at position p sees, of n: [0, head) and [from, p].
struct Seen {
  int head, from;
};
__device__ __forceinline__ Seen seen_keys(int p, int window, int sinks) {
  Seen s;
  s.from = window == 0 || p < window ? 0 : p - window + 1;
  s.head = sinks < s.from ? sinks : s.from;
  return s;
}

// One row (query, head) by one warp: keys in turn, each lane D / 32 of the head dims, with a
// running maximum and sum in fp32.  Reads the visible keys only.
template <class T, int D>
__device__ __forceinline__ void window_row(const WindowParams& p, int token, int h, int pos, int k0, int lane) {
  constexpr int kPer = D / 32;
  const int hk = h / p.group;
  float q[kPer], o[kPer], m = -INFINITY, l = 0.f;
  const T* qp = reinterpret_cast<const T*>(p.q + token * p.q_token + h * p.q_head) + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    q[i] = static_cast<float>(qp[i]);
    o[i] = 0.f;
  }
  const Seen s = seen_keys(pos, p.window, p.sinks);
  const int count = pos < 0 ? 0 : s.head + pos - s.from + 1;
  for (int i = 0; i < count; ++i) {
    const int j = k0 + (i < s.head ? i : i - s.head + s.from);
    const T* kp = reinterpret_cast<const T*>(p.k + j * p.k_token + hk * p.k_head) + lane * kPer;
    const T* vp = reinterpret_cast<const T*>(p.v + j * p.v_token + hk * p.v_head) + lane * kPer;
    float x = 0.f;
#pragma unroll
    for (int c = 0; c < kPer; ++c) x += q[c] * static_cast<float>(kp[c]);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) x += __shfl_xor_sync(0xffffffffu, x, w);
    x *= p.sl2;
    const float mn = fmaxf(m, x);
    const float keep = m == -INFINITY ? 0.f : exp2f(m - mn), w = x == -INFINITY ? 0.f : exp2f(x - mn);
    m = mn;
    l = l * keep + w;
#pragma unroll
    for (int c = 0; c < kPer; ++c) o[c] = o[c] * keep + w * static_cast<float>(vp[c]);
  }
  T* op = reinterpret_cast<T*>(p.out + token * p.out_token + h * p.out_head) + lane * kPer;
#pragma unroll
  for (int c = 0; c < kPer; ++c) op[c] = static_cast<T>(l == 0.f ? 0.f : o[c] / l);
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(token) * p.heads + h] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
}

// A warp per (query, head).
template <class T, int D>
__global__ void __launch_bounds__(256) window_kernel(const WindowParams p) {
  const int lane = threadIdx.x & 31;
  const long long n = static_cast<long long>(p.total_q) * p.heads;
  for (long long i = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; i < n;
       i += (static_cast<long long>(gridDim.x) * blockDim.x) >> 5) {
    const int token = static_cast<int>(i / p.heads), h = static_cast<int>(i % p.heads);
    for (int b = 0; b < p.batch; ++b) {
      const int q0 = p.cu_q[b], q1 = p.cu_q[b + 1], k0 = p.cu_k[b], k1 = p.cu_k[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k) {
        if (lane == 0) report_index(p.status, static_cast<unsigned long long>(b));
        continue;
      }
      if (token < q0 || token >= q1) continue;
      window_row<T, D>(p, token, h, (k1 - k0) - (q1 - q0) + (token - q0), k0, lane);
      break;
    }
  }
}

}  // namespace tl

using namespace tl;

extern "C" int tl_window_attention(tl_ctx* ctx, int dtype, const void* q, long long q_token_stride,
                                   long long q_head_stride, const void* k, long long k_token_stride,
                                   long long k_head_stride, const void* v, long long v_token_stride,
                                   long long v_head_stride, const int* cu_q, const int* cu_k, void* out,
                                   long long out_token_stride, long long out_head_stride, float* lse, int batch,
                                   int total_q, int total_k, int heads, int kv_heads, int d, float scale, int window,
                                   int sinks, tl_stream_t stream) {
  if (!ctx || (dtype != TL_BF16 && dtype != TL_FP16) || !heads_ok(heads, kv_heads, d) || heads / kv_heads > 128 ||
      batch < 0 || batch > 1024 || total_q < 0 || total_k < 0 || window < 0 || sinks < 0 || !(scale > 0.f) ||
      scale > 3.0e38f || static_cast<long long>(total_q) * heads >= (1LL << 31))
    return TL_ERR_INVALID;
  for (long long s : {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                      out_token_stride, out_head_stride})
    if (!esize_ok(s, 2)) return TL_ERR_INVALID;
  if (total_q == 0 || heads == 0 || batch == 0) return TL_OK;
  if (!q || !out || !cu_q || !cu_k || !aligned16(q) || !aligned16(out)) return TL_ERR_INVALID;
  if (total_k > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return TL_ERR_INVALID;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  WindowParams p;
  p.status = ctx->status;
  p.q = static_cast<const uint8_t*>(q);
  p.k = static_cast<const uint8_t*>(k);
  p.v = static_cast<const uint8_t*>(v);
  p.out = static_cast<uint8_t*>(out);
  p.lse = lse;
  p.q_token = 2 * q_token_stride;
  p.q_head = 2 * q_head_stride;
  p.k_token = 2 * k_token_stride;
  p.k_head = 2 * k_head_stride;
  p.v_token = 2 * v_token_stride;
  p.v_head = 2 * v_head_stride;
  p.out_token = 2 * out_token_stride;
  p.out_head = 2 * out_head_stride;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.batch = batch;
  p.total_q = total_q;
  p.total_k = total_k;
  p.heads = heads;
  p.group = heads / kv_heads;
  p.sl2 = scale * kLog2E;
  p.window = window;
  p.sinks = sinks;
  const long long need = (static_cast<long long>(total_q) * heads + 7) / 8, most = 64LL * ctx->sms;
  const unsigned grid = static_cast<unsigned>(need < most ? need : most);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TL_BF16) {
    if (d == 64) window_kernel<__nv_bfloat16, 64><<<grid, 256, 0, st>>>(p);
    else window_kernel<__nv_bfloat16, 128><<<grid, 256, 0, st>>>(p);
  } else {
    if (d == 64) window_kernel<__half, 64><<<grid, 256, 0, st>>>(p);
    else window_kernel<__half, 128><<<grid, 256, 0, st>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? TL_OK : TL_ERR_CUDA;
}
