// The MoE layer for the few tokens of a decoding step.
//
//   h_a = SiLU(x_t Wg_e) * (x_t Wu_e),   out_t = sum_j gate_tj h_a Wd_e,   a = (t, j), e the expert of a
// With a handful of tokens at each expert the weights are read once and meet one or two tokens, so
// HBM bounds the layer: 6 H F bytes for each distinct expert, 6 H F flops for each assignment.  Two
// launches, one per product; the second is a dependent launch whose CTAs fit beside the first's, so
// its weights are already being loaded while the first ends.
//
// Each CTA (one per SM and kernel) works out the routing by itself, so nothing has to pass between
// CTAs before the first load: the topk of every token, the assignments in the order (expert, t, j),
// and the items: an expert with up to 8 NT (8 or 16) of its assignments.  (item, 64 or 128 columns, 64 rows
// of the weights) is a unit of 16 KB; all units form one line, cut into equal ranges, one per CTA:
// even work for any routing.  One warp keeps a ring of TMA loads full, two groups of four
// warps multiply, a unit each in turn.
//
// The products run on mma.sync m16n8k16: columns of the weights are its 16 rows (transposed by ldmatrix from
// the 128-byte-swizzled tile), the tokens its 8 columns, which wastes least for 1 to 8 tokens; a
// tcgen05 tile would be 128 rows of tokens.  The k order inside 32 rows is permuted so
// that a thread's part of x is 16 contiguous bytes and ldmatrix rows fall in different banks: thread t
// holds k = 8 t .. 8 t + 7 as four pairs, and pair (i + t) mod 4 is its i-th.
// h goes to the second product as a sum of three bf16 (24 bits), three products for one load of
// the weights, so the layer keeps fp32 precision between the two.
//
// Tiles whose units lie in several CTAs: each CTA stores its fp32 sums, and the one that finishes
// last (a counter, left at zero again) adds them in the order of the line.  In the second product
// the last item of a column block to finish combines the block's rows, sum over j in order.  The order of
// every sum is fixed by the routing; nothing waits on another CTA.
#include <type_traits>

#include "tl_serve.cuh"

namespace tl {

namespace moet {
constexpr int kMaxT = 128, kMaxTopk = 8, kMaxE = 256, kMaxA = kMaxT * kMaxTopk, kMaxCtas = 512;
// Two groups of four warps take every other unit: one group's loads of x and products hide the other's.
constexpr int kGroup = 128, kThreads = 2 * kGroup + 32;
constexpr int kUnitBytes = 16384;
// Stages: an even number, so that a stage always serves the same group.  (With an odd one, a group could
// be a whole ring ahead of a load that the other one still waits for, and take the barrier's
// phase before it for its own.)  For up to 8 tokens the second product's CTAs fit beside the first's
// (registers too) with four.
template <bool Down, int NT>
struct Ring {
  static constexpr int kStages = Down && NT == 1 ? 4 : 6;
  static_assert(kStages % 2 == 0, "a stage belongs to one group");
  static constexpr int kBarOff = kStages * kUnitBytes;
  static constexpr int kHandOff = kBarOff + 128;  // group 1's sums: [2][8 NT][128 threads] floats
  static_assert(2 * kStages * 8 <= 128, "barriers");
  static constexpr int kSmem = kHandOff + 2 * kGroup * 8 * NT * 4 + 1024;  // 1024: the ring's alignment
};
}  // namespace moet

struct MoeTokParams {
  CUtensorMap w0;  // gate, or down: {columns, rows, E}, box {64, 64, 1}
  CUtensorMap w1;  // up
  Common common;
  const __nv_bfloat16* x;
  const float* logits;
  float* out;
  int* experts_out;
  float* gates_out;
  __nv_bfloat16* h;    // [3][T topk][F]: h = h0 + h1 + h2, rows in the order (expert, t, j)
  float* y;            // [T topk][H]
  float* part;         // [CTA][2][8 NT][128 threads] sums of a cut tile
  float* gates;        // [T topk]
  unsigned* cut_ctr;   // [CTA]: CTAs done with the cut tile that starts in this one
  unsigned* col_ctr;   // [column block]: items done (second product)
  int T, H, E, F, topk, renorm;
};

// What a CTA derives from the logits.
struct MoeTables {
  uint8_t expert[moet::kMaxA];   // of assignment a = t topk + j
  uint16_t at[moet::kMaxA];      // row of assignment a
  uint16_t order[moet::kMaxA];   // assignment of a row
  uint16_t start[moet::kMaxE + 1];  // rows of expert e: [start[e], start[e + 1])
  uint16_t item_expert[moet::kMaxA];
  uint16_t item_row[moet::kMaxA];   // first row
  int items;
  unsigned last;
};

// An order-preserving key of a logit; NaN is the lowest, as -inf.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);  // + 0: -0 equals 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp: the topk experts of a token, best first, ties to the lower index.  Lane l holds
// experts l, l + 32, ...; key 0 marks "none" (below the key of -inf).
__device__ __forceinline__ void route_token(const float* row, int E, int topk, int lane, uint8_t* experts) {
  constexpr int kPer = moet::kMaxE / 32;
  uint32_t key[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) key[i] = lane + 32 * i < E ? logit_key(__ldg(row + lane + 32 * i)) : 0u;
  for (int j = 0; j < topk; ++j) {
    uint32_t best = 0u;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (32 * i < E && key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const uint32_t e = __reduce_min_sync(0xffffffffu, best == top ? lane + 32 * at : 0xffffffffu);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (static_cast<uint32_t>(lane + 32 * i) == e) key[i] = 0u;
    if (lane == 0) experts[j] = static_cast<uint8_t>(e);
  }
}

// All threads of the CTA: routing, order and items (groups of `group` rows of an expert).
__device__ __forceinline__ void moet_tables(const MoeTokParams& p, MoeTables& tb, int group) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.T * p.topk;
  for (int t = warp; t < p.T; t += moet::kThreads / 32)
    route_token(p.logits + static_cast<size_t>(t) * p.E, p.E, p.topk, lane, tb.expert + t * p.topk);
  for (int a = n + static_cast<int>(threadIdx.x); a < ((n + 3) & ~3); a += moet::kThreads) tb.expert[a] = 0xff;  // never an assignment below
  __syncthreads();
  // counts, then rows, of the experts of this thread: a byte compare over all assignments.  (E = 256
  // uses 0xff too, so entries past n are cut off by index.)
  const uint32_t* words = reinterpret_cast<const uint32_t*>(tb.expert);
  for (int e = threadIdx.x; e < p.E; e += moet::kThreads) {
    int c = 0;
    for (int w = 0; 4 * w < n; ++w) {
      const uint32_t eq = __vcmpeq4(words[w], e * 0x01010101u);
      c += __popc((4 * w + 4 <= n ? eq : eq & ((1u << (8 * (n - 4 * w))) - 1u)) & 0x01010101u);
    }
    tb.start[e + 1] = static_cast<uint16_t>(c);
  }
  __syncthreads();
  if (warp == 0) {
    int rows = 0, items = 0;
    for (int e0 = 0; e0 < p.E; e0 += 32) {
      const int c = e0 + lane < p.E ? tb.start[e0 + lane + 1] : 0, k = (c + group - 1) / group;
      int sr = c, si = k;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int r = __shfl_up_sync(0xffffffffu, sr, x), i = __shfl_up_sync(0xffffffffu, si, x);
        if (lane >= x) {
          sr += r;
          si += i;
        }
      }
      __syncwarp();
      if (e0 + lane < p.E) tb.start[e0 + lane + 1] = static_cast<uint16_t>(rows + sr);
      for (int i = 0; i < k; ++i) {
        tb.item_expert[items + si - k + i] = static_cast<uint16_t>(e0 + lane);
        tb.item_row[items + si - k + i] = static_cast<uint16_t>(rows + sr - c + i * group);
      }
      rows += __shfl_sync(0xffffffffu, sr, 31);
      items += __shfl_sync(0xffffffffu, si, 31);
    }
    if (lane == 0) {
      tb.start[0] = 0;
      tb.items = items;
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += moet::kThreads) {
    int r = tb.start[e];
    if (r == tb.start[e + 1]) continue;
    for (int w = 0; 4 * w < n; ++w) {
      uint32_t eq = __vcmpeq4(words[w], e * 0x01010101u) & 0x01010101u;
      for (; eq; eq &= eq - 1) {
        const int a = 4 * w + ((__ffs(eq) - 1) >> 3);
        if (a >= n) break;
        tb.at[a] = static_cast<uint16_t>(r);
        tb.order[r++] = static_cast<uint16_t>(a);
      }
    }
  }
  __syncthreads();
}

// Four pairs of a 16-byte part of x (or h) in the order that thread t uses them: pair (i + t) mod 4 i-th.
__device__ __forceinline__ void rotate_pairs(const uint4& v, int t, uint32_t (&r)[4]) {
  const uint32_t a0 = t & 1 ? v.y : v.x, a1 = t & 1 ? v.z : v.y, a2 = t & 1 ? v.w : v.z, a3 = t & 1 ? v.x : v.w;
  r[0] = t & 2 ? a2 : a0;
  r[1] = t & 2 ? a3 : a1;
  r[2] = t & 2 ? a0 : a2;
  r[3] = t & 2 ? a1 : a3;
}

// A 16-byte load that another kernel's writes may precede (not through the read-only path).
__device__ __forceinline__ uint4 ld_global128(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// One warp: the gates of a token, the softmax over all E logits taken at its experts.
__device__ __forceinline__ void token_gates(const MoeTokParams& p, const MoeTables& tb, int tok, int lane) {
  const float* row = p.logits + static_cast<size_t>(tok) * p.E;
  float top = -INFINITY, sum = 0.f;
  for (int e = lane; e < p.E; e += 32) top = fmaxf(top, row[e]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  for (int e = lane; e < p.E; e += 32) sum += expf(row[e] - top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float gate = lane < p.topk ? expf(row[tb.expert[tok * p.topk + lane]] - top) / sum : 0.f;
  if (p.renorm) {
    float all = gate;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);  // topk <= 8
    gate /= all;
  }
  if (lane < p.topk) {
    p.gates[tok * p.topk + lane] = gate;
    if (p.gates_out) p.gates_out[tok * p.topk + lane] = gate;
  }
}

// Down: false for the first product (gate and up, 64 columns of each), true for the second (down,
// 128 columns).  NT: groups of 8 tokens in an item.
template <bool Down, int NT>
__global__ void __launch_bounds__(moet::kThreads, 1) moet_kernel(const __grid_constant__ MoeTokParams p) {
  using namespace moet;
  using R = Ring<Down, NT>;
  constexpr int kStages = R::kStages;
  constexpr int kParts = Down ? 3 : 1;            // 16-bit terms of the left operand
  constexpr int kCols = Down ? 128 : 64;          // columns of a tile
  extern __shared__ uint8_t smem_raw[];
  __shared__ MoeTables tb;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + R::kBarOff);
  uint64_t* empty = full + kStages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 4);  // the warps of one group
    }
    fence_mbar_init();
    tma_prefetch_map(&p.w0);
    if (!Down) tma_prefetch_map(&p.w1);
  }
  if (!Down) grid_dep_launch();
  moet_tables(p, tb, 8 * NT);
  const int K = Down ? p.F : p.H, N = Down ? p.H : p.F;
  const int nk = (K + 63) / 64, nc = (N + kCols - 1) / kCols;
  // the line of units: the first product item by item, the second column block by column block, so
  // that blocks are combined while others are still multiplied
  const uint32_t tiles = static_cast<uint32_t>(tb.items) * nc, total = tiles * nk;
  const uint32_t per = (total + gridDim.x - 1) / gridDim.x, first = per * blockIdx.x;
  const int n = first >= total ? 0 : static_cast<int>(per < total - first ? per : total - first);
  const int item0 = n ? (Down ? (first / nk) % tb.items : first / nk / nc) : 0;
  const int col0 = n ? (Down ? first / nk / tb.items : (first / nk) % nc) : 0;
  const int k0 = n ? first % nk : 0;
  auto next_tile = [&](int& item, int& col) {
    if (Down) {
      if (++item == tb.items) {
        item = 0;
        ++col;
      }
    } else if (++col == nc) {
      col = 0;
      ++item;
    }
  };

  if (warp == 2 * kGroup / 32) {
    // ------------------------------------------------------------ loads (they wait for no other kernel)
    if (lane == 0) {
      int item = item0, col = col0, k = k0, i = 0;
      bool ok = true;
      for (; i < n && ok; ++i) {
        const int s = i % kStages;
        ok = mbar_wait(&empty[s], ((i / kStages) & 1) ^ 1, p.common, kSiteEmpty);
        if (!ok) break;
        mbar_arrive_expect_tx(&full[s], kUnitBytes);
        const int e = tb.item_expert[item];
        uint8_t* dst = ring + s * kUnitBytes;
        tma_load_3d(dst, &p.w0, &full[s], col * kCols, k * 64, e);
        tma_load_3d(dst + kUnitBytes / 2, Down ? &p.w0 : &p.w1, &full[s], col * kCols + (Down ? 64 : 0), k * 64, e);
        if (++k == nk) {
          k = 0;
          next_tile(item, col);
        }
      }
      if (!ok)  // gave up: what was issued has landed before the CTA ends
        for (int j = i > kStages ? i - kStages : 0; j < i; ++j) mbar_wait(&full[j % kStages], (j / kStages) & 1, p.common, kSiteDrain);
    }
    __syncwarp();
    if (!Down)
      for (int tok = blockIdx.x; tok < p.T; tok += gridDim.x) token_gates(p, tb, tok, lane);
    return;
  }

  // -------------------------------------------------------------- products
  const int grp = warp >> 2, wq = warp & 3, tid = threadIdx.x & (kGroup - 1), g = lane >> 2, t = lane & 3;
  if (Down) grid_dep_wait();  // h is written
  if (!Down && blockIdx.x == 0 && p.experts_out)
    for (int a = threadIdx.x; a < p.T * p.topk; a += 2 * kGroup) p.experts_out[a] = tb.expert[a];
  // the rows of an item
  auto item_rows = [&](int item, int& row0) {
    row0 = tb.item_row[item];
    const int end = tb.start[tb.item_expert[item] + 1];
    return end - row0 < 8 * NT ? end - row0 : 8 * NT;
  };
  // this thread's part of the left operand for the next unit of its group, loaded a unit ahead
  int x_item = item0, x_col = col0, x_k = k0, x_rows = 0;
  uint4 xv[kParts][NT][2];
  const __nv_bfloat16* src[NT];
  const size_t plane = static_cast<size_t>(p.T) * p.topk * p.F;
  auto x_tile = [&]() {
    int row0;
    x_rows = item_rows(x_item, row0);
#pragma unroll
    for (int b = 0; b < NT; ++b) {
      src[b] = nullptr;
      if (8 * b + g < x_rows) {
        const int r = row0 + 8 * b + g;
        src[b] = Down ? p.h + static_cast<size_t>(r) * p.F : p.x + static_cast<size_t>(tb.order[r] / p.topk) * p.H;
      }
    }
  };
  auto x_step = [&]() {
    if (++x_k == nk) {
      x_k = 0;
      next_tile(x_item, x_col);
      return true;
    }
    return false;
  };
  auto load_x = [&]() {
#pragma unroll
    for (int q = 0; q < kParts; ++q)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          xv[q][b][w] = make_uint4(0u, 0u, 0u, 0u);
          const int at = x_k * 64 + 32 * w + 8 * t;
          if (8 * b < x_rows && src[b] && at < K)
            xv[q][b][w] = Down ? ld_global128(src[b] + q * plane + at) : __ldg(reinterpret_cast<const uint4*>(src[b] + at));
        }
  };
  if (grp && n > 1) x_step();
  if (grp < n) {
    x_tile();
    load_x();
  }
  // ldmatrix rows: lane l gives row l & 7 of matrix l >> 3; matrices 0, 1: k pairs 2s, columns 0-7 and
  // 8-15; matrices 2, 3: k pairs 2s + 1
  const int lt = (lane & 7) >> 1, lbit = lane & 1, lhi = lane >> 4, lcol = (lane >> 3) & 1;
  float* hand = reinterpret_cast<float*>(ring + R::kHandOff) + tid * 4;
  float acc[2][NT][4];
  bool ok = true;
  int item = item0, col = col0;
  for (int begin = 0, seg = 0; begin < n; ++seg) {
    // this CTA's units [begin, end) of one tile
    const uint32_t tile = (first + begin) / nk;
    const int left = static_cast<int>((tile + 1) * nk - (first + begin));
    const int end = left < n - begin ? begin + left : n;
    int row0;
    const int rows = item_rows(item, row0);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][b][j] = 0.f;
    for (int i = begin + ((begin ^ grp) & 1); i < end; i += 2) {
      uint32_t xr[2][kParts][NT][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < kParts; ++q)
#pragma unroll
          for (int b = 0; b < NT; ++b) rotate_pairs(xv[q][b][h], t, xr[h][q][b]);
      if (i + 2 < n) {
        const bool one = x_step(), two = x_step();
        if (one || two) x_tile();
        load_x();
      }
      const int s = i % kStages;
      if (ok) ok = mbar_wait(&full[s], (i / kStages) & 1, p.common, kSiteFull);  // after a timeout: on, without waits
      const uint32_t w = smem_u32(ring + s * kUnitBytes);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int s2 = 0; s2 < 2; ++s2) {
          const int kr = 32 * h + 8 * lt + 2 * ((2 * s2 + lhi + lt) & 3) + lbit;
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            // first product: m = gate, up, columns 16 wq of each; second: columns 32 wq + 16 m
            const int chunk = (Down ? 4 * (wq & 1) + 2 * m : 2 * wq) + lcol;
            const uint32_t box = w + (Down ? (wq >> 1) : m) * (kUnitBytes / 2);
            uint32_t a[4];
            ldsm4t(a, box + kr * 128 + ((chunk ^ (kr & 7)) << 4));
#pragma unroll
            for (int b = 0; b < NT; ++b)
              if (8 * b < rows)
#pragma unroll
                for (int q = 0; q < kParts; ++q)
                  mma16816<__nv_bfloat16>(acc[m][b], a, xr[h][q][b][2 * s2], xr[h][q][b][2 * s2 + 1]);
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ------------------------------------------------------------ the end of a tile, or of the CTA's part of it
    // Group 1 hands its sums over (two buffers: it cannot pass the next barrier before group 0 has read
    // these) and goes on with the next tile; group 0 adds and finishes.
    const int this_col = col;
    const uint32_t seg_first = first + begin;
    begin = end;
    next_tile(item, col);
    float* buf = hand + (seg & 1) * kGroup * 8 * NT;
    if (grp) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int b = 0; b < NT; ++b)
          if (8 * b < rows)
            *reinterpret_cast<float4*>(buf + (m * NT + b) * kGroup * 4) = make_float4(acc[m][b][0], acc[m][b][1], acc[m][b][2], acc[m][b][3]);
    }
    named_bar_sync(1, 2 * kGroup);
    if (grp) continue;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b)
        if (8 * b < rows) {
          const float4 v = *reinterpret_cast<const float4*>(buf + (m * NT + b) * kGroup * 4);
          acc[m][b][0] += v.x;
          acc[m][b][1] += v.y;
          acc[m][b][2] += v.z;
          acc[m][b][3] += v.w;
        }
    const bool starts = seg_first == tile * nk, ends = first + end == (tile + 1) * nk;
    if (!starts || !ends) {
      const uint32_t c0 = tile * nk / per, c1 = (tile * nk + nk - 1) / per;
      constexpr int kSlot = kGroup * 8 * NT;
      float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (starts ? 1 : 0)) * kSlot + tid * 4;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int b = 0; b < NT; ++b)
          if (8 * b < rows)
            *reinterpret_cast<float4*>(part + (m * NT + b) * kGroup * 4) = make_float4(acc[m][b][0], acc[m][b][1], acc[m][b][2], acc[m][b][3]);
      named_bar_sync(2, kGroup);
      if (tid == 0) {
        __threadfence();  // the CTA's part, seen by this thread through the barrier, before the count
        const unsigned done = atomicAdd(p.cut_ctr + c0, 1u) + 1u;
        tb.last = done == c1 - c0 + 1;
        if (tb.last) p.cut_ctr[c0] = 0u;
        __threadfence();
      }
      named_bar_sync(2, kGroup);
      if (!tb.last) continue;
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int b = 0; b < NT; ++b)
          if (8 * b < rows) {
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (uint32_t c = c0; c <= c1; ++c) {
              const float4 v = __ldcg(reinterpret_cast<const float4*>(
                  p.part + (static_cast<size_t>(c) * 2 + (c == c0 ? 1 : 0)) * kSlot + (m * NT + b) * kGroup * 4 + tid * 4));
              sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
            }
            acc[m][b][0] = sum.x;
            acc[m][b][1] = sum.y;
            acc[m][b][2] = sum.z;
            acc[m][b][3] = sum.w;
          }
    }
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 8 * b + 2 * t + (j & 1);  // columns of the products are rows of the item
        if (r >= rows) continue;
        if constexpr (!Down) {
          const int f = this_col * 64 + wq * 16 + g + 8 * (j >> 1);
          if (f < N) {
            const float a = acc[0][b][j], v = a / (1.f + expf(-a)) * acc[1][b][j];
            const __nv_bfloat16 h0 = __float2bfloat16_rn(v);
            const float r1 = v - __bfloat162float(h0);
            const __nv_bfloat16 h1 = __float2bfloat16_rn(r1);
            const size_t at = static_cast<size_t>(row0 + r) * p.F + f;
            p.h[at] = h0;
            p.h[plane + at] = h1;
            p.h[2 * plane + at] = __float2bfloat16_rn(r1 - __bfloat162float(h1));
          }
        } else {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int c = this_col * 128 + wq * 32 + m * 16 + g + 8 * (j >> 1);
            if (c < N) p.y[static_cast<size_t>(row0 + r) * p.H + c] = acc[m][b][j];
          }
        }
      }
    if constexpr (Down) {
      // the block's last item combines its rows
      named_bar_sync(2, kGroup);
      if (tid == 0) {
        __threadfence();
        const unsigned done = atomicAdd(p.col_ctr + this_col, 1u) + 1u;
        tb.last = done == static_cast<unsigned>(tb.items);
        if (tb.last) p.col_ctr[this_col] = 0u;
        __threadfence();
      }
      named_bar_sync(2, kGroup);
      if (tb.last) {
        for (int v = tid; v < p.T * 32; v += kGroup) {
          const int tok = v >> 5, c = this_col * 128 + (v & 31) * 4;
          if (c >= N) continue;
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int j = 0; j < p.topk; ++j) {
            const int a = tok * p.topk + j;
            const float gate = __ldcg(p.gates + a);
            const float4 u = __ldcg(reinterpret_cast<const float4*>(p.y + static_cast<size_t>(tb.at[a]) * p.H + c));
            sum = make_float4(sum.x + gate * u.x, sum.y + gate * u.y, sum.z + gate * u.z, sum.w + gate * u.w);
          }
          *reinterpret_cast<float4*>(p.out + static_cast<size_t>(tok) * p.H + c) = sum;
        }
      }
    }
  }
}

}  // namespace tl

using namespace tl;

static bool moet_shape_ok(int T, int H, int E, int F, int topk) {
  return T >= 1 && T <= moet::kMaxT && topk >= 1 && topk <= moet::kMaxTopk && E >= topk && E <= moet::kMaxE && H > 0 &&
         F > 0 && H % 8 == 0 && F % 8 == 0 && H <= 32768 && F <= 32768;
}

// Tokens in an item, in eights: an expert with more of them is read again, from L2.  Most experts have
// one or two tokens whatever T, and 16 tokens' operands are what the registers hold twice.
static int moet_eights(int T) { return T <= 8 ? 1 : 2; }

struct MoetLayout {
  size_t gates, h, y, part, total;
};
static MoetLayout moet_layout(int T, int H, int F, int topk) {
  const size_t a = static_cast<size_t>(T) * topk;
  MoetLayout L;
  L.gates = kCounterBytes;
  L.h = L.gates + align256(a * 4);
  L.y = L.h + align256(3 * a * F * 2);
  L.part = L.y + align256(a * H * 4);
  L.total = L.part + static_cast<size_t>(moet::kMaxCtas) * 2 * moet::kGroup * 8 * moet_eights(T) * 4;
  return L;
}

extern "C" size_t tl_moe_tokens_workspace_bytes(int T, int H, int E, int F, int topk) {
  if (!moet_shape_ok(T, H, E, F, topk)) return 0;
  return moet_layout(T, H, F, topk).total;
}

template <bool Down, int NT>
static int moet_launch(tl_ctx* ctx, const MoeTokParams& p, cudaStream_t st) {
  auto kern = moet_kernel<Down, NT>;
  static std::atomic<unsigned long long> ready{0};
  if (!smem_ready(ready, ctx->device, reinterpret_cast<const void*>(kern), moet::Ring<Down, NT>::kSmem)) return TL_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctx->ctas < moet::kMaxCtas ? ctx->ctas : moet::kMaxCtas, 1, 1);
  cfg.blockDim = dim3(moet::kThreads, 1, 1);
  cfg.dynamicSmemBytes = moet::Ring<Down, NT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = Down ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return TL_ERR_CUDA;
  }
  return TL_OK;
}

extern "C" int tl_moe_tokens(tl_ctx* ctx, const void* x, const float* logits, int topk, const void* w_gate,
                             const void* w_up, const void* w_down, float* out, int* experts_out, float* gates_out,
                             void* workspace, size_t workspace_bytes, int T, int H, int E, int F, tl_stream_t stream) {
  if (!ctx || !moet_shape_ok(T, H, E, F, topk)) return TL_ERR_INVALID;
  if (!x || !logits || !w_gate || !w_up || !w_down || !out || !workspace) return TL_ERR_INVALID;
  for (const void* q : {x, static_cast<const void*>(logits), w_gate, w_up, w_down, static_cast<const void*>(out),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return TL_ERR_INVALID;
  const MoetLayout L = moet_layout(T, H, F, topk);
  if (workspace_bytes < L.total) return TL_ERR_WORKSPACE;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeTokParams p;
  std::memset(&p, 0, sizeof(p));
  CUtensorMap down;
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!tmap_3d(&p.w0, BF, 2, w_gate, F, H, E, 64, 64, 1) || !tmap_3d(&p.w1, BF, 2, w_up, F, H, E, 64, 64, 1) ||
      !tmap_3d(&down, BF, 2, w_down, H, F, E, 64, 64, 1))
    return TL_ERR_CUDA;
  p.common = make_common(ctx);
  p.common.trace_hdr = nullptr;  // these kernels record no trace spans
  p.common.trace = nullptr;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.logits = logits;
  p.out = out;
  p.experts_out = experts_out;
  p.gates_out = gates_out;
  p.cut_ctr = reinterpret_cast<unsigned*>(ws);
  p.col_ctr = reinterpret_cast<unsigned*>(ws) + kCutCounters;
  p.gates = reinterpret_cast<float*>(ws + L.gates);
  p.h = reinterpret_cast<__nv_bfloat16*>(ws + L.h);
  p.y = reinterpret_cast<float*>(ws + L.y);
  p.part = reinterpret_cast<float*>(ws + L.part);
  p.T = T;
  p.H = H;
  p.E = E;
  p.F = F;
  p.topk = topk;
  p.renorm = ctx->cfg.moe_renorm;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  auto both = [&](auto nt) {
    const int rc = moet_launch<false, decltype(nt)::value>(ctx, p, st);
    if (rc != TL_OK) return rc;
    p.w0 = down;
    return moet_launch<true, decltype(nt)::value>(ctx, p, st);
  };
  return moet_eights(T) == 1 ? both(std::integral_constant<int, 1>{}) : both(std::integral_constant<int, 2>{});
}
