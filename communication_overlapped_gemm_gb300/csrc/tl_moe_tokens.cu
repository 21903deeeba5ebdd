// The MoE layer for the few tokens of a decoding step, in one launch.
//
//   h_a = SiLU(x_t Wg_e) * (x_t Wu_e),   out_t = sum_j gate_tj h_a Wd_e,   a = (t, j), e the expert of a
// With a handful of tokens at each expert the weights are read once and meet one or two tokens, so
// HBM bounds the layer: 6 H F bytes for each distinct expert, 6 H F flops for each assignment.
// Measured (H 2048, F 1408, 64 experts, top 2): 64 tokens 158 us, 6.1 TB/s, 0.90 of the copy rate; 8 tokens 52;
// one token, two experts, 18.5 us against 5.1 for its bytes: routing, first loads, the tiles' joins and the
// combine are waited for in turn.  An expert with more than 16 tokens is several items and is read for each: of 8
// experts of 17 MB 64 tokens take 52 us and 128 71, with 140 and 148 MB from HBM for 138 MB of weights; of 8 experts
// of 352 MB (H 4096, F 14336) 32, 64 and 128 tokens take 450, 606 and 1005 us, the later readings from HBM too.
//
// Each CTA (one per SM, a cooperative launch) works out the routing by itself, so nothing has to
// pass between CTAs before the first load: the topk of every token, the assignments in the order
// (expert, t, j), and the items: an expert with up to 8 NT (8 or 16) of its assignments.  (item, 128
// columns of gate and up or 256 of down, 32 rows) is a unit of 16 KB; all units of a product form one
// line, cut into equal ranges, one per CTA: even work for any routing.  A CTA takes its range of
// the first product, then its range of the second.  One warp keeps a ring of TMA loads of the
// weights full across both, a second one copies the tokens' parts of x (then h) beside them; two
// groups of four warps multiply, a unit each in turn.  (With the parts of x loaded by the multiplying
// warps from L2 a unit ahead, 64 tokens took 251 us against 194 without those loads.  Boxes
// side by side read 256 or 512 bytes of a row at a time: 128 bytes reached 0.8 of HBM.)
//
// The second product of an item waits (bounded) until its h is complete.  No unit of the first waits
// for anything, every CTA is resident, and both lines are item by item, so the h that a CTA needs comes
// from itself and its neighbours; its weights are in the ring by then.
//
// The products run on mma.sync m16n8k16: columns of the weights are its 16 rows (transposed by
// ldmatrix from the 128-byte-swizzled tile), the tokens its 8 columns, which wastes least for 1 to 8
// tokens; a tcgen05 tile would be 128 rows of tokens.
// h goes to the second product as a sum of three bf16 (24 bits), three products for one load of
// the weights, so the layer keeps fp32 precision between the two.
//
// Tiles whose units lie in several CTAs: each CTA stores its fp32 sums, and the one that finishes
// last (a counter) adds them in the order of the line.  The last of a token's topk rows to be finished
// in a block of 256 columns adds them up, in the order j = 0, 1, ...  So the order of every sum is
// fixed by the routing.  Every counter is left at zero.
#include <type_traits>

#include "tl_serve.cuh"

namespace tl {

namespace moet {
constexpr int kMaxT = 128, kMaxTopk = 8, kMaxE = 256, kMaxA = kMaxT * kMaxTopk, kMaxCtas = 256;
// Two groups of four warps take every other unit: one group's loads of x and products hide the other's.
constexpr int kGroup = 128, kThreads = 2 * kGroup + 64;
constexpr int kRows = 32, kBox = 4096, kUnitBytes = 4 * kBox;  // rows of a unit; 64 columns of them; 4 boxes
constexpr int kXPitch = 80;  // bytes from a token's 32 values to the next one's: ldmatrix rows in different banks
// Stages: an even number, so that a stage always serves the same group.  (With an odd one, a group could
// be a whole ring ahead of a load that the other one still waits for, and take the barrier's
// phase before it for its own.)
template <int NT>
struct Ring {
  static constexpr int kStages = NT == 1 ? 10 : 8;
  static_assert(kStages % 2 == 0, "a stage belongs to one group");
  static constexpr int kXPart = 8 * NT * kXPitch;  // one 16-bit term of the tokens' 32 values
  static constexpr int kStageBytes = (kUnitBytes + 3 * kXPart + 1023) / 1024 * 1024;
  static constexpr int kBarOff = kStages * kStageBytes;
  static constexpr int kHandOff = kBarOff + 256;  // sums handed over: [2][16 NT][128 threads] floats
  static_assert(2 * kStages * 8 <= 256, "barriers");
  static_assert(2 * kGroup * 16 * NT * 4 >= kMaxA / 32 * kMaxE * 2, "the routing's counts go there first");
  static constexpr int kSmem = kHandOff + 2 * kGroup * 16 * NT * 4 + 1024;  // 1024: the ring's alignment
};
static_assert(2 * kMaxCtas <= kCutCounters, "a counter per product and CTA");
}  // namespace moet

struct MoeTokParams {
  CUtensorMap gate, up, down;  // {columns, rows, E}, box {64, 32, 1}
  Common common;
  const __nv_bfloat16* x;
  const float* logits;
  float* out;
  int* experts_out;
  float* gates_out;
  __nv_bfloat16* h;    // [3][T topk][F]: h = h0 + h1 + h2, rows in the order (expert, t, j)
  float* y;            // [T topk][H]
  float* part;         // [product][CTA][2][16 NT][128 threads] sums of a cut tile
  unsigned* cut_ctr;   // [product][CTA]: CTAs done with the cut tile that starts in this one
  unsigned* item_ctr;  // [item]: tiles done, of both products
  unsigned* tok_ctr;   // [token][column block]: rows done
  int T, H, E, F, topk, renorm;
};

// What a CTA derives from the logits.
struct MoeTables {
  alignas(16) uint8_t expert[moet::kMaxA];  // of assignment a = t topk + j
  uint8_t rank[moet::kMaxA];     // among the assignments of the same expert in its group of 32
  float gate[moet::kMaxA];       // of assignment a
  uint16_t at[moet::kMaxA];      // row of assignment a
  uint16_t order[moet::kMaxA];   // assignment of a row
  uint16_t start[moet::kMaxE + 1];  // rows of expert e: [start[e], start[e + 1])
  uint16_t item_expert[moet::kMaxA];
  uint16_t item_row[moet::kMaxA];   // first row
  uint16_t first_item[moet::kMaxE];  // of an expert
  int items;
  uint32_t last;
};

// An order-preserving key of a logit; NaN is the lowest, as -inf.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t b = __float_as_uint(v == v ? v + 0.f : -INFINITY);  // + 0: -0 equals 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// One warp: the topk experts of tokens t, t + step, .. (kBatch of them, below T), best first, ties to
// the lower index.  Lane l holds experts l, l + 32, ...; key 0 marks "none" (below the key of -inf).
// Each token is a chain of loads and reductions, so several go side by side, without a branch between them.
template <int kBatch, int kPer>
__device__ __forceinline__ void route_tokens(const MoeTokParams& p, int t, int step, int lane, MoeTables& tb) {
  uint32_t key[kBatch][kPer], mine[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const float* row = p.logits + static_cast<size_t>(t + b * step < p.T ? t + b * step : t) * p.E;
#pragma unroll
    for (int i = 0; i < kPer; ++i) key[b][i] = lane + 32 * i < p.E ? logit_key(__ldg(row + lane + 32 * i)) : 0u;
  }
  for (int j = 0; j < p.topk; ++j) {
    uint32_t best[kBatch], e[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      best[b] = key[b][0];
      e[b] = lane;
#pragma unroll
      for (int i = 1; i < kPer; ++i) {
        e[b] = key[b][i] > best[b] ? lane + 32 * i : e[b];
        best[b] = max(best[b], key[b][i]);
      }
    }
    uint32_t high[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) high[b] = __reduce_max_sync(0xffffffffu, best[b]);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) e[b] = __reduce_min_sync(0xffffffffu, best[b] == high[b] ? e[b] : 0xffffffffu);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      mine[b] = lane == j ? e[b] : mine[b];
#pragma unroll
      for (int i = 0; i < kPer; ++i) key[b][i] = lane + 32 * i == static_cast<int>(e[b]) ? 0u : key[b][i];
    }
  }
#pragma unroll
  for (int b = 0; b < kBatch; ++b)
    if (lane < p.topk && t + b * step < p.T) tb.expert[(t + b * step) * p.topk + lane] = static_cast<uint8_t>(mine[b]);
}

// One warp: the gates of kBatch tokens (as above), the softmax over all E logits taken at the chosen experts.
template <int kBatch>
__device__ __forceinline__ void token_gates(const MoeTokParams& p, int t, int step, int lane, MoeTables& tb) {
  const float* row[kBatch];
  float top[kBatch], sum[kBatch], gate[kBatch];
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    row[b] = p.logits + static_cast<size_t>(t + b * step < p.T ? t + b * step : t) * p.E;
    top[b] = -INFINITY;
    sum[b] = 0.f;
  }
  for (int e = lane; e < p.E; e += 32)
#pragma unroll
    for (int b = 0; b < kBatch; ++b) top[b] = fmaxf(top[b], __ldg(row[b] + e));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int b = 0; b < kBatch; ++b) top[b] = fmaxf(top[b], __shfl_xor_sync(0xffffffffu, top[b], o));
  for (int e = lane; e < p.E; e += 32)
#pragma unroll
    for (int b = 0; b < kBatch; ++b) sum[b] += expf(__ldg(row[b] + e) - top[b]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int b = 0; b < kBatch; ++b) sum[b] += __shfl_xor_sync(0xffffffffu, sum[b], o);
#pragma unroll
  for (int b = 0; b < kBatch; ++b) {
    const int a = (t + b * step < p.T ? t + b * step : t) * p.topk + (lane < p.topk ? lane : 0);
    gate[b] = lane < p.topk ? expf(__ldg(row[b] + tb.expert[a]) - top[b]) / sum[b] : 0.f;
    if (p.renorm) {
      float all = gate[b];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);  // topk <= 8
      gate[b] /= all;
    }
    if (lane < p.topk && t + b * step < p.T) tb.gate[a] = gate[b];
  }
}

template <int kPer>
__device__ __forceinline__ void route_all(const MoeTokParams& p, int warp, int lane, MoeTables& tb) {
  constexpr int kWarps = moet::kThreads / 32, kBatch = 8 / kPer;
  if (p.T <= kWarps) {
    if (warp < p.T) route_tokens<1, kPer>(p, warp, kWarps, lane, tb);
  } else {
    for (int t = warp; t < p.T; t += kBatch * kWarps) route_tokens<kBatch, kPer>(p, t, kWarps, lane, tb);
  }
}

// All threads of the CTA: routing, order and items (groups of `group` rows of an expert).  `seen`:
// a count for each 32 assignments and expert, 16 KB of shared memory that nothing else uses yet.
__device__ __forceinline__ void moet_tables(const MoeTokParams& p, MoeTables& tb, uint16_t* seen, int group) {
  using namespace moet;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = p.T * p.topk, chunks = (n + 31) / 32;
  for (int i = threadIdx.x; i < chunks * p.E; i += kThreads) seen[i] = 0;
  if (p.E <= 64)
    route_all<2>(p, warp, lane, tb);
  else
    route_all<8>(p, warp, lane, tb);
  __syncthreads();
  // Up to 8 tokens (kernels of that group): by one warp, a lane per assignment, an item per expert (one token 19.2
  // -> 18.7 us; also compiled into the other kernels it cost them 0.5).
  if (group == 8 && n <= 32) {
    if (warp == 0) {
      const uint32_t key = lane < n ? tb.expert[lane] * 32u + lane : 0xffffffffu;
      int row = 0, before = 0;  // assignments, and those of other experts, that come first
      for (int i = 0; i < n; ++i) {
        const uint32_t other = __shfl_sync(0xffffffffu, key, i);
        row += other < key;
        before += other >> 5 < key >> 5;
      }
      const uint32_t same = __match_any_sync(0xffffffffu, key >> 5);
      const bool lead = lane < n && row == before;
      int item = 0;
      for (uint32_t leads = __ballot_sync(0xffffffffu, lead); leads; leads &= leads - 1)
        item += __shfl_sync(0xffffffffu, key, __ffs(leads) - 1) >> 5 < key >> 5;
      if (lane < n) {
        const uint32_t e = key >> 5;
        tb.at[lane] = static_cast<uint16_t>(row);
        tb.order[row] = static_cast<uint16_t>(lane);
        if (lead) {
          tb.start[e] = static_cast<uint16_t>(row);
          tb.start[e + 1] = static_cast<uint16_t>(row + __popc(same));
          tb.first_item[e] = static_cast<uint16_t>(item);
          tb.item_expert[item] = static_cast<uint16_t>(e);
          tb.item_row[item] = static_cast<uint16_t>(row);
        }
      }
      const int items = __popc(__ballot_sync(0xffffffffu, lead));
      if (lane == 0) tb.items = items;
    }
    __syncthreads();
    return;
  }
  for (int c = warp; c < chunks; c += kThreads / 32) {
    const int a = 32 * c + lane;
    const uint32_t same = __match_any_sync(0xffffffffu, a < n ? static_cast<uint32_t>(tb.expert[a]) : 0x100u + lane);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (a < n) {
      tb.rank[a] = static_cast<uint8_t>(rank);
      if (rank == 0) seen[c * p.E + tb.expert[a]] = static_cast<uint16_t>(__popc(same));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += kThreads) {  // counts become the rows before each group of 32
    int sum = 0;
    for (int c = 0; c < chunks; ++c) {
      const int here = seen[c * p.E + e];
      seen[c * p.E + e] = static_cast<uint16_t>(sum);
      sum += here;
    }
    tb.start[e + 1] = static_cast<uint16_t>(sum);
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
      if (e0 + lane < p.E) tb.start[e0 + lane + 1] = static_cast<uint16_t>(rows + sr);
      if (e0 + lane < p.E) tb.first_item[e0 + lane] = static_cast<uint16_t>(items + si - k);
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
  for (int a = threadIdx.x; a < n; a += kThreads) {
    const int e = tb.expert[a], row = tb.start[e] + seen[(a >> 5) * p.E + e] + tb.rank[a];
    tb.at[a] = static_cast<uint16_t>(row);
    tb.order[row] = static_cast<uint16_t>(a);
  }
  __syncthreads();
}

// Adds to a counter, releasing what this thread has seen and acquiring what others released; the sum.
__device__ __forceinline__ unsigned count_up(unsigned* ctr, unsigned by = 1u) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(ctr), "r"(by) : "memory");
  return old + by;
}

__device__ __forceinline__ void count_up_async(unsigned* ctr) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(ctr) : "memory");
}

// Wait (bounded) until an item's h is complete; one lane polls.
__device__ __forceinline__ bool wait_item(const unsigned* ctr, unsigned want, const Common& c, int lane) {
  bool ok = true;
  if (lane == 0) {
    uint64_t t0 = 0;
    for (int i = 0;; ++i) {
      unsigned v;
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ctr) : "memory");
      if (v >= want) break;
      if (i == 64) t0 = globaltimer();  // (a read of the timer costs as much as the load)
      if (i > 64 && (i & 15) == 0 && globaltimer() - t0 > c.timeout_ns) {
        report_timeout(c.status, kSiteSignal, 0);
        ok = false;
        break;
      }
    }
  }
  __syncwarp();  // orders the other lanes' reads of h after lane 0's acquire; the shuffle orders no memory
  return __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
}

// A CTA's range of one product's line of units (item by item, column block by column block, k).
template <bool Down>
struct MoeLine {
  static constexpr int kCols = Down ? 256 : 128;  // columns of a tile
  int K, N, nk, nc, n;
  uint32_t per, first;
  int item0, col0, k0;
  __device__ __forceinline__ MoeLine(const MoeTokParams& p, int items) {
    K = Down ? p.F : p.H;
    N = Down ? p.H : p.F;
    nk = (K + moet::kRows - 1) / moet::kRows;
    nc = (N + kCols - 1) / kCols;
    const uint32_t total = static_cast<uint32_t>(items) * nc * nk;
    per = (total + gridDim.x - 1) / gridDim.x;
    first = per * blockIdx.x;
    n = first >= total ? 0 : static_cast<int>(per < total - first ? per : total - first);
    const uint32_t tile = n ? first / nk : 0;
    k0 = n ? first % nk : 0;
    item0 = tile / nc;
    col0 = tile % nc;
  }
  __device__ __forceinline__ void next_tile(int& item, int& col) const {
    if (++col == nc) {
      col = 0;
      ++item;
    }
  }
};

// The rows of an item.
template <int NT>
__device__ __forceinline__ int item_rows(const MoeTables& tb, int item, int& row0) {
  row0 = tb.item_row[item];
  const int end = tb.start[tb.item_expert[item] + 1];
  return end - row0 < 8 * NT ? end - row0 : 8 * NT;
}

// The loads of a line's weights, by one thread; u counts units over both lines.
template <bool Down, int NT>
__device__ __forceinline__ bool moet_load_w(const MoeTokParams& p, const MoeTables& tb, uint8_t* ring, uint64_t* full,
                                            uint64_t* empty, int& u) {
  using namespace moet;
  using R = Ring<NT>;
  const MoeLine<Down> ln(p, tb.items);
  int item = ln.item0, col = ln.col0, k = ln.k0;
  for (int i = 0; i < ln.n; ++i, ++u) {
    const int s = u % R::kStages;
    if (!mbar_wait(&empty[s], ((u / R::kStages) & 1) ^ 1, p.common, kSiteEmpty)) return false;
    mbar_arrive_expect_tx(&full[s], kUnitBytes);
    const int e = tb.item_expert[item], x = col * ln.kCols, y = k * kRows;
    uint8_t* dst = ring + s * R::kStageBytes;
#pragma unroll
    for (int box = 0; box < 4; ++box)
      tma_load_3d(dst + box * kBox, Down ? &p.down : box < 2 ? &p.gate : &p.up, &full[s], x + 64 * (Down ? box : box & 1), y, e);
    if (++k == ln.nk) {
      k = 0;
      ln.next_tile(item, col);
    }
  }
  return true;
}

// Arrive on a barrier (one of its counted arrivals) once this thread's earlier cp.async have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The tokens' 32 values of x, or of the three terms of h, for each unit, by one warp: lane l copies
// 16 bytes, values 8 (l mod 4) on, of rows l / 4 and l / 4 + 8.
template <bool Down, int NT>
__device__ __forceinline__ bool moet_load_x(const MoeTokParams& p, const MoeTables& tb, uint8_t* ring, uint64_t* full,
                                            uint64_t* empty, int& u) {
  using namespace moet;
  using R = Ring<NT>;
  const MoeLine<Down> ln(p, tb.items);
  const int lane = threadIdx.x & 31, r = lane >> 2, ch = lane & 3;
  const int nc1 = (p.F + MoeLine<false>::kCols - 1) / MoeLine<false>::kCols;  // tiles of an item in the first product
  const size_t plane = static_cast<size_t>(p.T) * p.topk * p.F;
  int item = ln.item0, col = ln.col0, k = ln.k0, seen = -1, rows = 0;
  const __nv_bfloat16* src[NT];
  for (int i = 0; i < ln.n; ++i, ++u) {
    if (item != seen) {
      seen = item;
      if (Down && !wait_item(p.item_ctr + item, nc1, p.common, lane)) return false;
      int row0;
      rows = item_rows<NT>(tb, item, row0);
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        const int row = row0 + (r + 8 * b < rows ? r + 8 * b : 0);
        src[b] = (Down ? p.h + static_cast<size_t>(row) * p.F : p.x + static_cast<size_t>(tb.order[row] / p.topk) * p.H) + 8 * ch;
      }
    }
    const int s = u % R::kStages;
    if (!__all_sync(0xffffffffu, mbar_wait(&empty[s], ((u / R::kStages) & 1) ^ 1, p.common, kSiteEmpty))) return false;
    const uint32_t dst = smem_u32(ring + s * R::kStageBytes + kUnitBytes) + r * kXPitch + ch * 16;
    const uint32_t bytes = k * kRows + 8 * ch < ln.K ? 16u : 0u;  // past K: zeros, nothing is read
#pragma unroll
    for (int b = 0; b < NT; ++b)
      if (r + 8 * b < rows)
#pragma unroll
        for (int q = 0; q < (Down ? 3 : 1); ++q)
          cp_async16(dst + q * R::kXPart + b * 8 * kXPitch, src[b] + (bytes ? q * plane + k * kRows : 0), bytes);
    cp_async_arrive(&full[s]);
    if (++k == ln.nk) {
      k = 0;
      ln.next_tile(item, col);
    }
  }
  return true;
}

__device__ __forceinline__ void put_routing(const MoeTokParams& p, const MoeTables& tb, int tok, int col, int lane) {
  if (col == 0 && lane < p.topk) {
    if (p.experts_out) p.experts_out[tok * p.topk + lane] = tb.expert[tok * p.topk + lane];
    if (p.gates_out) p.gates_out[tok * p.topk + lane] = tb.gate[tok * p.topk + lane];
  }
}

// By a warp: 64 of a token's 256 columns of a block, the gates times all pieces of its topk rows (whole tiles in
// y, those of cut ones by CTA), in the order j, then that of the line.
template <int Slot, int Group>
__device__ __forceinline__ void add_pieces(const MoeTokParams& p, const MoeTables& tb, const MoeLine<true>& ln,
                                           const float* parts, int tok, int col, int wq, int lane) {
  using namespace moet;
  constexpr int kBatch = 16;
  const int c = col * ln.kCols + wq * 64 + lane * 2;
  // lane j: the CTAs with pieces of the token's j-th row, and how many pieces are before theirs
  uint32_t c0 = 0, pieces = 0, row = 0, in = 0;
  float gate = 0.f;
  if (lane < p.topk) {
    const int a = tok * p.topk + lane, e = tb.expert[a];
    row = tb.at[a];
    in = (row - tb.start[e]) % Group;
    const uint32_t unit = ((tb.first_item[e] + (row - tb.start[e]) / Group) * ln.nc + col) * ln.nk;
    c0 = unit / ln.per;
    pieces = (unit + ln.nk - 1) / ln.per - c0 + 1;
    gate = tb.gate[a];
  }
  uint32_t before = pieces;
#pragma unroll
  for (int x = 1; x < kMaxTopk; x <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, before, x);
    if (lane >= x) before += v;
  }
  const uint32_t all = __shfl_sync(0xffffffffu, before, kMaxTopk - 1);
  before -= pieces;
  float2 sum = make_float2(0.f, 0.f);
  for (uint32_t q0 = 0; q0 < all; q0 += 32) {
    // lane q: where piece q0 + q lies, and its gate
    int j = 0;
#pragma unroll
    for (int x = 1; x < kMaxTopk; ++x) {
      const uint32_t start = __shfl_sync(0xffffffffu, before, x);
      if (x < p.topk && q0 + lane >= start) j = x;
    }
    const uint32_t k = q0 + lane - __shfl_sync(0xffffffffu, before, j), cta = __shfl_sync(0xffffffffu, c0, j) + k;
    const bool cut = __shfl_sync(0xffffffffu, pieces, j) > 1;
    const uint32_t r = __shfl_sync(0xffffffffu, in, j), y_row = __shfl_sync(0xffffffffu, row, j);
    const float f = __shfl_sync(0xffffffffu, gate, j);
    const float* at = cut ? parts + (static_cast<size_t>(cta) * 2 + (k == 0 ? 1 : 0)) * Slot + r * ln.kCols
                          : p.y + static_cast<size_t>(y_row) * p.H + col * ln.kCols;
    const int here = all - q0 < 32 ? all - q0 : 32;
    for (int q = 0; q < here; q += kBatch) {
      float2 v[kBatch];
      float fs[kBatch];
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const auto from = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(at), q + x));
        fs[x] = __shfl_sync(0xffffffffu, f, q + x);
        v[x] = q + x < here && c < ln.N ? __ldcg(reinterpret_cast<const float2*>(from + wq * 64 + lane * 2)) : make_float2(0.f, 0.f);
      }
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (q + x >= here) break;
        sum.x = fmaf(fs[x], v[x].x, sum.x);
        sum.y = fmaf(fs[x], v[x].y, sum.y);
      }
    }
  }
  if (c < ln.N) *reinterpret_cast<float2*>(p.out + static_cast<size_t>(tok) * p.H + c) = sum;
  if (wq == 0) put_routing(p, tb, tok, col, lane);
}

// The products of a line, by the two groups; u0: units of the line before it.
template <bool Down, int NT>
__device__ __forceinline__ void moet_multiply(const MoeTokParams& p, MoeTables& tb, uint8_t* ring, uint64_t* full,
                                              uint64_t* empty, int u0, int& segs, bool& ok) {
  using namespace moet;
  using R = Ring<NT>;
  constexpr int kStages = R::kStages;
  constexpr int kParts = Down ? 3 : 1;  // 16-bit terms of the left operand
  constexpr int kSlot = kGroup * 16 * NT;  // sums of a tile
  // Up to 8 tokens: the pieces of the second product's cut tiles are added up with the tokens' rows at once, not
  // tile by tile before, one hand-over less (one token 20.4 -> 19.2 us, 4 tokens 36.5 -> 34.8; 64 tokens 158 -> 162).
  constexpr bool kPieces = Down && NT == 1;
  const MoeLine<Down> ln(p, tb.items);
  const int nk = ln.nk, N = ln.N, n = ln.n;
  const uint32_t per = ln.per, first = ln.first;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wq = warp & 3, tid = threadIdx.x & (kGroup - 1), g = lane >> 2, t = lane & 3;
  const int grp = warp >> 2, par = (u0 ^ grp) & 1;  // this group's units are those with i & 1 == par
  const size_t plane = static_cast<size_t>(p.T) * p.topk * p.F;
  // Weights, 16 columns m of this warp: rows k are lines of 128 bytes, their 16-byte chunks permuted by k
  // mod 8; ldmatrix matrices 0, 1: rows 0-7, columns 0-7 and 8-15; 2, 3: rows 8-15.  First product:
  // m = 0, 1 gate, 2, 3 up, columns 32 wq of the tile on; second: columns 64 wq on.
  uint32_t w_off[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    const int box = Down ? wq : (wq >> 1) + (m & 2), chunk = (Down ? 2 * m : 4 * (wq & 1) + 2 * (m & 1)) + ((lane >> 3) & 1);
    w_off[m] = box * kBox + ((lane & 7) + ((lane >> 4) << 3)) * 128 + ((chunk ^ (lane & 7)) << 4);
  }
  const uint32_t x_off = kUnitBytes + (lane & 7) * kXPitch + (lane >> 3) * 16;  // tokens 0-7, 8 of the 32 values per matrix
  float* hand = reinterpret_cast<float*>(ring + R::kHandOff) + tid * 4;
  float acc[4][NT][4];
  int item = ln.item0, col = ln.col0;
  for (int begin = 0; begin < n; ++segs) {
    // this CTA's units [begin, end) of one tile
    const uint32_t tile = (first + begin) / nk;
    const int left = static_cast<int>((tile + 1) * nk - (first + begin));
    const int end = left < n - begin ? begin + left : n;
    int row0;
    const int rows = item_rows<NT>(tb, item, row0);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][b][j] = 0.f;
    for (int i = begin + ((begin ^ par) & 1); i < end; i += 2) {
      const int s = (u0 + i) % kStages;
      if (ok)  // the same in all lanes; after a timeout: on, without waits
        ok = __all_sync(0xffffffffu, mbar_wait(&full[s], ((u0 + i) / kStages) & 1, p.common, kSiteFull));
      const uint32_t st = smem_u32(ring + s * R::kStageBytes);
      uint32_t x[NT][kParts][4];
#pragma unroll
      for (int b = 0; b < NT; ++b)
        if (8 * b < rows)
#pragma unroll
          for (int q = 0; q < kParts; ++q) {
            ldsm4(x[b][q], st + x_off + q * R::kXPart + b * 8 * kXPitch);
          }
      // A unit's products start from zero and are then added in fp32: the tensor core cuts what it adds to
      // a long sum off, which over 2048 rows cost a relative 4e-6, rounded additions a tenth of it.
      uint32_t a[2][4][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int m = 0; m < 4; ++m) ldsm4t(a[h][m], st + w_off[m] + h * 2048);
#pragma unroll
      for (int b = 0; b < NT; ++b)
        if (8 * b < rows) {
          float d[4][4];
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[m][j] = 0.f;
#pragma unroll
          for (int q = kParts - 1; q >= 0; --q)  // the small terms first
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int m = 0; m < 4; ++m) mma16816<__nv_bfloat16>(d[m], a[h][m], x[b][q][2 * h], x[b][q][2 * h + 1]);
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][b][j] += d[m][j];
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // ------------------------------------------------------------ the end of a tile, or of the CTA's part of it
    // The groups finish tiles in turn: the other one hands its sums over and goes on with the next
    // tile.  Two buffers and two barriers: it cannot reach the tile after next, and write this buffer
    // again, before the finisher, which hands over the next one, has read this one.
    const int this_col = col, this_item = item;
    const uint32_t seg_first = first + begin;
    begin = end;
    ln.next_tile(item, col);
    float* buf = hand + (segs & 1) * kGroup * 16 * NT;
    const uint32_t bar = 1 + (segs & 1);
    if ((segs & 1) != grp) {
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int b = 0; b < NT; ++b)
          if (8 * b < rows)
            *reinterpret_cast<float4*>(buf + (m * NT + b) * kGroup * 4) = make_float4(acc[m][b][0], acc[m][b][1], acc[m][b][2], acc[m][b][3]);
      named_bar_arrive(bar, 2 * kGroup);
      continue;
    }
    named_bar_sync(bar, 2 * kGroup);
#pragma unroll
    for (int m = 0; m < 4; ++m)
#pragma unroll
      for (int b = 0; b < NT; ++b)
        if (8 * b < rows) {
          const float4 v = *reinterpret_cast<const float4*>(buf + (m * NT + b) * kGroup * 4);
          acc[m][b][0] += v.x;
          acc[m][b][1] += v.y;
          acc[m][b][2] += v.z;
          acc[m][b][3] += v.w;
        }
    const bool whole = seg_first == tile * nk && first + end == (tile + 1) * nk;
    // (each product has parts and counters of its own: a CTA is in the second one while its
    // neighbour still works on their common tile of the first)
    float* parts = p.part + (Down ? static_cast<size_t>(kMaxCtas) * 2 * kSlot : 0);
    float* mine = parts + (static_cast<size_t>(blockIdx.x) * 2 + (seg_first == tile * nk ? 1 : 0)) * kSlot;  // slot 1 starts a tile
    if (!kPieces && !whole) {
      const uint32_t c0 = tile * nk / per, c1 = (tile * nk + nk - 1) / per;
      unsigned* ctr = p.cut_ctr + (Down ? kMaxCtas : 0) + c0;
      float* part = mine + tid * 4;
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int b = 0; b < NT; ++b)
          if (8 * b < rows)
            *reinterpret_cast<float4*>(part + (m * NT + b) * kGroup * 4) = make_float4(acc[m][b][0], acc[m][b][1], acc[m][b][2], acc[m][b][3]);
      named_bar_sync(3, kGroup);
      if (tid == 0) {  // releases the whole CTA's part, which it has seen through the barrier
        tb.last = count_up(ctr) == c1 - c0 + 1;
        if (tb.last) *ctr = 0u;
      }
      named_bar_sync(3, kGroup);
      if (!tb.last) continue;
#pragma unroll
      for (int b = 0; b < NT; ++b)
        if (8 * b < rows) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[m][b][j] = 0.f;
          const float* from = parts + (static_cast<size_t>(c0) * 2 + 1) * kSlot + b * kGroup * 4 + tid * 4;
          for (uint32_t c = c0; c <= c1;) {
            constexpr int kBatch = NT == 1 ? 8 : 4;
            float4 v[kBatch][4];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
#pragma unroll
              for (int m = 0; m < 4; ++m)
                v[x][m] = c + x <= c1 ? __ldcg(reinterpret_cast<const float4*>(from + m * NT * kGroup * 4)) : make_float4(0.f, 0.f, 0.f, 0.f);
              from += c + x == c0 ? kSlot : 2 * kSlot;
            }
            c += kBatch;
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
#pragma unroll
              for (int m = 0; m < 4; ++m) {
                acc[m][b][0] += v[x][m].x;
                acc[m][b][1] += v[x][m].y;
                acc[m][b][2] += v[x][m].z;
                acc[m][b][3] += v[x][m].w;
              }
          }
        }
    }
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = 8 * b + 2 * t + (j & 1);  // columns of the products are rows of the item
        if (r >= rows) continue;
        if constexpr (!Down) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int f = this_col * ln.kCols + wq * 32 + m * 16 + g + 8 * (j >> 1);
            if (f < N) {
              const float a = acc[m][b][j], v = a / (1.f + expf(-a)) * acc[2 + m][b][j];
              // (a value that rounds to infinity is cut off to bf16's largest instead; an infinity has no remainder)
              __nv_bfloat16 h0 = __float2bfloat16_rn(v);
              if (__hisinf(h0)) h0 = __float2bfloat16_rz(v);
              const float f0 = __bfloat162float(h0), r1 = v == f0 ? 0.f : v - f0;
              const __nv_bfloat16 h1 = __float2bfloat16_rn(r1);
              const size_t at = static_cast<size_t>(row0 + r) * p.F + f;
              p.h[at] = h0;
              p.h[plane + at] = h1;
              p.h[2 * plane + at] = __float2bfloat16_rn(r1 - __bfloat162float(h1));
            }
          }
        } else {
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int c = wq * 64 + m * 16 + g + 8 * (j >> 1), at = this_col * ln.kCols + c;
            if (kPieces && !whole) mine[r * ln.kCols + c] = acc[m][b][j];
            else if (at < N) p.y[static_cast<size_t>(row0 + r) * p.H + at] = acc[m][b][j];
          }
        }
      }
    named_bar_sync(3, kGroup);
    if constexpr (!Down) {
      if (tid == 0) count_up_async(p.item_ctr + this_item);
    } else {
      // A token's topk rows of this block: who finishes the last of them (kPieces: the last unit) adds them up.
      // The item's last sets the item's counter back: nothing waits on it any more.
      const unsigned units = kPieces ? static_cast<unsigned>(first + end - seg_first) : 1u, tile_units = kPieces ? nk : 1;
      if (wq == 0) {
        bool done = false;
        if (lane < rows) {
          unsigned* ctr = p.tok_ctr + (tb.order[row0 + lane] / p.topk) * ln.nc + this_col;
          done = count_up(ctr, units) == static_cast<unsigned>(p.topk) * tile_units;
          if (done) *ctr = 0u;
        }
        const uint32_t mask = __ballot_sync(0xffffffffu, done);
        if (lane == 0) tb.last = mask;
      } else if (tid == kGroup - 1) {
        const int nc1 = (p.F + MoeLine<false>::kCols - 1) / MoeLine<false>::kCols;
        if (count_up(p.item_ctr + this_item, units) == nc1 + ln.nc * tile_units) p.item_ctr[this_item] = 0u;
      }
      named_bar_sync(3, kGroup);
      uint32_t mask = tb.last;
      if constexpr (kPieces) {
        for (; mask; mask &= mask - 1)  // a quarter of the block per warp
          add_pieces<kSlot, 8 * NT>(p, tb, ln, parts, tb.order[row0 + __ffs(mask) - 1] / p.topk, this_col, wq, lane);
      } else {
        for (int x = 0; mask; ++x, mask &= mask - 1) {  // two tokens at a time, half a block per warp
          if ((x & 1) != (wq >> 1)) continue;
          const int tok = tb.order[row0 + __ffs(mask) - 1] / p.topk, c = this_col * ln.kCols + (wq & 1) * 128 + lane * 4;
          if (c < N) {
            float4 v[kMaxTopk], sum = make_float4(0.f, 0.f, 0.f, 0.f);
  #pragma unroll
            for (int j = 0; j < kMaxTopk; ++j)
              if (j < p.topk)
                v[j] = __ldcg(reinterpret_cast<const float4*>(p.y + static_cast<size_t>(tb.at[tok * p.topk + j]) * p.H + c));
  #pragma unroll
            for (int j = 0; j < kMaxTopk; ++j)
              if (j < p.topk) {
                const float f = tb.gate[tok * p.topk + j];
                sum = make_float4(sum.x + f * v[j].x, sum.y + f * v[j].y, sum.z + f * v[j].z, sum.w + f * v[j].w);
              }
            *reinterpret_cast<float4*>(p.out + static_cast<size_t>(tok) * p.H + c) = sum;
          }
          if ((wq & 1) == 0) put_routing(p, tb, tok, this_col, lane);
        }
      }
    }
  }
}

// NT: groups of 8 tokens in an item.
template <int NT>
__global__ void __launch_bounds__(moet::kThreads, 1) moet_kernel(const __grid_constant__ MoeTokParams p) {
  using namespace moet;
  using R = Ring<NT>;
  constexpr int kStages = R::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ MoeTables tb;
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + R::kBarOff);
  uint64_t* empty = full + kStages;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1 + 32);  // weights, a lane's x each
      mbar_init(&empty[s], 4);  // the warps of one group
    }
    fence_mbar_init();
    tma_prefetch_map(&p.gate);
    tma_prefetch_map(&p.up);
    tma_prefetch_map(&p.down);
  }
  moet_tables(p, tb, reinterpret_cast<uint16_t*>(ring + R::kHandOff), 8 * NT);
  if (threadIdx.x >= 2 * kGroup) {
    int u = 0;
    bool ok = true;
    const bool one = (threadIdx.x & 31) == 0;
    if (threadIdx.x >= 2 * kGroup + 32)
      ok = moet_load_x<false, NT>(p, tb, ring, full, empty, u) && moet_load_x<true, NT>(p, tb, ring, full, empty, u);
    else if (one)
      ok = moet_load_w<false, NT>(p, tb, ring, full, empty, u) && moet_load_w<true, NT>(p, tb, ring, full, empty, u);
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!ok && one) {
      // Gave up: what was issued lands before the CTA ends (bounded: the other warp may not have joined
      // in a stage's barrier, and then the wait runs out long after the copies are in).
      for (int j = u > kStages ? u - kStages : 0; j < u; ++j) mbar_wait(&full[j % kStages], (j / kStages) & 1, p.common, kSiteDrain);
    }
    return;
  }
  // the gates, while the first loads are under way; a tile's barriers lie between here and their first use
  for (int t = threadIdx.x >> 5; t < p.T; t += 4 * (2 * kGroup / 32)) token_gates<4>(p, t, 2 * kGroup / 32, threadIdx.x & 31, tb);
  int segs = 0;
  bool ok = true;
  moet_multiply<false, NT>(p, tb, ring, full, empty, 0, segs, ok);
  moet_multiply<true, NT>(p, tb, ring, full, empty, MoeLine<false>(p, tb.items).n, segs, ok);
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
  size_t h, y, part, total;
};
static MoetLayout moet_layout(int T, int H, int F, int topk) {
  const size_t a = static_cast<size_t>(T) * topk;
  MoetLayout L;
  L.h = kCounterBytes;
  L.y = L.h + align256(3 * a * F * 2);
  L.part = L.y + align256(a * H * 4);
  L.total = L.part + 2 * static_cast<size_t>(moet::kMaxCtas) * 2 * moet::kGroup * 16 * moet_eights(T) * 4;
  return L;
}

extern "C" size_t tl_moe_tokens_workspace_bytes(int T, int H, int E, int F, int topk) {
  if (!moet_shape_ok(T, H, E, F, topk)) return 0;
  return moet_layout(T, H, F, topk).total;
}

template <int NT>
static int moet_launch(tl_ctx* ctx, const MoeTokParams& p, cudaStream_t st) {
  auto kern = moet_kernel<NT>;
  static std::atomic<unsigned long long> ready{0};
  if (!smem_ready(ready, ctx->device, reinterpret_cast<const void*>(kern), moet::Ring<NT>::kSmem)) return TL_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctx->ctas < moet::kMaxCtas ? ctx->ctas : moet::kMaxCtas, 1, 1);
  cfg.blockDim = dim3(moet::kThreads, 1, 1);
  cfg.dynamicSmemBytes = moet::Ring<NT>::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // every CTA resident: the second product waits on the first
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return e == cudaErrorCooperativeLaunchTooLarge ? TL_ERR_UNSUPPORTED : TL_ERR_CUDA;
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
  const auto BF = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  if (!tmap_3d(&p.gate, BF, 2, w_gate, F, H, E, 64, moet::kRows, 1) || !tmap_3d(&p.up, BF, 2, w_up, F, H, E, 64, moet::kRows, 1) ||
      !tmap_3d(&p.down, BF, 2, w_down, H, F, E, 64, moet::kRows, 1))
    return TL_ERR_CUDA;
  p.common = make_common(ctx);
  p.common.trace_hdr = nullptr;  // this kernel records no trace spans
  p.common.trace = nullptr;
  p.x = static_cast<const __nv_bfloat16*>(x);
  p.logits = logits;
  p.out = out;
  p.experts_out = experts_out;
  p.gates_out = gates_out;
  p.cut_ctr = reinterpret_cast<unsigned*>(ws);
  p.item_ctr = p.cut_ctr + kCutCounters;
  p.tok_ctr = p.item_ctr + kItemCounters;
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
  return moet_eights(T) == 1 ? moet_launch<1>(ctx, p, st) : moet_launch<2>(ctx, p, st);
}
