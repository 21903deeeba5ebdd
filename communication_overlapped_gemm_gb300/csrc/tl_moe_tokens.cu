// The MoE layer for the few tokens of a decoding step.
#include "tl_serve.cuh"

namespace tl {

namespace moet {
constexpr int kMaxT = 128, kMaxTopk = 8, kMaxE = 256, kMaxA = kMaxT * kMaxTopk;
}

struct MoeTokParams {
  const __nv_bfloat16* x;
  const float* logits;
  const __nv_bfloat16* w_gate;
  const __nv_bfloat16* w_up;
  const __nv_bfloat16* w_down;
  float* out;
  int* experts_out;
  float* gates_out;
  int* experts;  // [T topk]
  float* gates;  // [T topk]
  float* h;      // [T topk][F]
  int T, H, E, F, topk, renorm;
};

// The routing of one token by one warp: the topk largest logits (ties to the lower expert, NaN
// the lowest), and the softmax over all E logits taken at them.
__device__ __forceinline__ void route_token(const float* row, int E, int topk, int renorm, int lane, int* experts,
                                            float* gates) {
  constexpr int kPer = moet::kMaxE / 32;
  float v[kPer], mx = -INFINITY, s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < E ? row[e] : -INFINITY;
    mx = fmaxf(mx, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < E) s += expf(v[i] - mx);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  uint32_t taken = 0;
  float sum = 0.f;
  for (int j = 0; j < topk; ++j) {
    // order key: NaN -> -inf; a free expert always beats "none" (index beyond every expert)
    float bv = -INFINITY;
    int bi = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = lane + 32 * i;
      const float x = v[i] == v[i] ? v[i] : -INFINITY;
      if (e < E && !(taken & (1u << i)) && (x > bv || (x == bv && e < bi))) {
        bv = x;
        bi = e;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
      }
    }
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (lane + 32 * i == bi) {
        taken |= 1u << i;
        mine = v[i];
      }
    const float g = expf(__shfl_sync(0xffffffffu, mine, bi & 31) - mx) / s;
    sum += g;
    if (lane == 0) {
      experts[j] = bi;
      gates[j] = g;
    }
  }
  __syncwarp();
  if (renorm)
    for (int j = lane; j < topk; j += 32) gates[j] /= sum;
}

__global__ void __launch_bounds__(128) moet_route_kernel(const MoeTokParams p) {
  const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (t >= p.T) return;
  route_token(p.logits + static_cast<size_t>(t) * p.E, p.E, p.topk, p.renorm, lane, p.experts + t * p.topk,
              p.gates + t * p.topk);
  __syncwarp();
  for (int j = lane; j < p.topk; j += 32) {
    if (p.experts_out) p.experts_out[t * p.topk + j] = p.experts[t * p.topk + j];
    if (p.gates_out) p.gates_out[t * p.topk + j] = p.gates[t * p.topk + j];
  }
}

// h = SiLU(x Wg) * (x Wu): one thread per column of F, one CTA row per assignment.
__global__ void __launch_bounds__(64) moet_up_kernel(const MoeTokParams p) {
  const int a = blockIdx.y, f = blockIdx.x * 64 + threadIdx.x;
  if (f >= p.F) return;
  const size_t w0 = static_cast<size_t>(p.experts[a]) * p.H * p.F + f;
  const __nv_bfloat16* x = p.x + static_cast<size_t>(a / p.topk) * p.H;
  float g = 0.f, u = 0.f;
#pragma unroll 8
  for (int k = 0; k < p.H; ++k) {
    const float xv = __bfloat162float(x[k]);
    g += xv * __bfloat162float(p.w_gate[w0 + static_cast<size_t>(k) * p.F]);
    u += xv * __bfloat162float(p.w_up[w0 + static_cast<size_t>(k) * p.F]);
  }
  p.h[static_cast<size_t>(a) * p.F + f] = g / (1.f + expf(-g)) * u;
}

// out = sum_j gate_j h_j Wd: one thread per column of H, one CTA row per token.
__global__ void __launch_bounds__(64) moet_down_kernel(const MoeTokParams p) {
  const int t = blockIdx.y, c = blockIdx.x * 64 + threadIdx.x;
  if (c >= p.H) return;
  float out = 0.f;
  for (int j = 0; j < p.topk; ++j) {
    const int a = t * p.topk + j;
    const size_t w0 = static_cast<size_t>(p.experts[a]) * p.F * p.H + c;
    const float* h = p.h + static_cast<size_t>(a) * p.F;
    float y = 0.f;
#pragma unroll 8
    for (int k = 0; k < p.F; ++k) y += h[k] * __bfloat162float(p.w_down[w0 + static_cast<size_t>(k) * p.H]);
    out += p.gates[a] * y;
  }
  p.out[static_cast<size_t>(t) * p.H + c] = out;
}

}  // namespace tl

using namespace tl;

static bool moet_shape_ok(int T, int H, int E, int F, int topk) {
  return T >= 1 && T <= moet::kMaxT && topk >= 1 && topk <= moet::kMaxTopk && E >= topk && E <= moet::kMaxE && H > 0 &&
         F > 0 && H % 8 == 0 && F % 8 == 0 && H <= (1 << 20) && F <= (1 << 20);
}

extern "C" size_t tl_moe_tokens_workspace_bytes(int T, int H, int E, int F, int topk) {
  if (!moet_shape_ok(T, H, E, F, topk)) return 0;
  const size_t a = static_cast<size_t>(T) * topk;
  return 2 * align256(a * 4) + align256(a * F * 4);
}

extern "C" int tl_moe_tokens(tl_ctx* ctx, const void* x, const float* logits, int topk, const void* w_gate,
                             const void* w_up, const void* w_down, float* out, int* experts_out, float* gates_out,
                             void* workspace, size_t workspace_bytes, int T, int H, int E, int F, tl_stream_t stream) {
  if (!ctx || !moet_shape_ok(T, H, E, F, topk)) return TL_ERR_INVALID;
  if (!x || !logits || !w_gate || !w_up || !w_down || !out || !workspace) return TL_ERR_INVALID;
  for (const void* q : {x, static_cast<const void*>(logits), w_gate, w_up, w_down, static_cast<const void*>(out),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return TL_ERR_INVALID;
  if (workspace_bytes < tl_moe_tokens_workspace_bytes(T, H, E, F, topk)) return TL_ERR_WORKSPACE;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  const size_t a = static_cast<size_t>(T) * topk;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeTokParams p;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.logits = logits;
  p.w_gate = static_cast<const __nv_bfloat16*>(w_gate);
  p.w_up = static_cast<const __nv_bfloat16*>(w_up);
  p.w_down = static_cast<const __nv_bfloat16*>(w_down);
  p.out = out;
  p.experts_out = experts_out;
  p.gates_out = gates_out;
  p.experts = reinterpret_cast<int*>(ws);
  p.gates = reinterpret_cast<float*>(ws + align256(a * 4));
  p.h = reinterpret_cast<float*>(ws + 2 * align256(a * 4));
  p.T = T;
  p.H = H;
  p.E = E;
  p.F = F;
  p.topk = topk;
  p.renorm = ctx->cfg.moe_renorm;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  moet_route_kernel<<<(T + 3) / 4, 128, 0, st>>>(p);
  moet_up_kernel<<<dim3((F + 63) / 64, T * topk), 64, 0, st>>>(p);
  moet_down_kernel<<<dim3((H + 63) / 64, T), 64, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? TL_OK : TL_ERR_CUDA;
}
