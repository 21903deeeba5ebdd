// Causal attention of packed prompts with a sliding window and sinks, on the tensor cores.
//
//   S = sl2 Q K^T,  P = 2^(S - m),  O = P V,  l = sum P,  out = O / l,  lse = ln 2 (m + log2 l)
// over the keys that each query sees, with the running maximum m of a row (base 2).
//
// A tile is 128 rows: the G = heads / kv_heads query heads of one kv head for 128 / G consecutive tokens
// (TMA reads them as one box), so short prompts fill tiles, a tile's window is narrow, and K and V
// are read once for all G heads.  An item is two tiles side by side of one sequence and kv head, which
// share every K and V block in shared memory; persistent CTAs take items in turn, the longest
// first (WinPlan).  An item's keys are walked in blocks of 128:
// first the sinks that lie before its windows (up to 32 of them as a block of 32), then from
// the first window's start to its last query.  Blocks start anywhere (a TMA row coordinate has no alignment), so a window of 1024 takes 9.
//
//   warp 0    TMA: Q of both tiles, K and V blocks through a ring
//   warps 1, 2  the MMAs of tile 0 and 1, tcgen05.mma M = 128, issued by one thread each:
//               S_t = Q_t K^T        N = 128 keys, K = head dim, both K-major from shared memory
//               O_t += P_t V         N = head dim, K = 128 keys, P_t from TMEM, V MN-major
//   warp 3    the list of the CTA's items, if it is long
//   warps 4-7, 8-11   softmax of tile 0 and 1, one row per thread
// TMEM: S_0, S_1 (128 columns each; P_t as 16-bit pairs takes the first 64 of S_t once they are
// read), O_0, O_1.  The two warps issue in turn, S_0 S_1 | PV_0 S_0' | PV_1 S_1' | ..: while one tile is in its
// softmax the tensor cores work for the other.  MMAs of a thread complete in order, so S_t' needs
// no wait for PV_t before it, and "S_t' is there" also says that PV_t is complete: the softmax
// rescales O_t then, and only when a row's maximum grew by more than 2^8 (until then weights
// stay below 2^8 and the stale maximum cancels in O / l).
// (The tensor cores take an MMA in 66 cycles, 35 at N = 64, but an issuing warp whose descriptors are not uniform
// values needs 45 for it, and several times that while the softmax's long unrolled code has the instruction
// caches: one warp for both tiles was busy throughout, 3300 cycles a block.  Hence two warps, uniform bases plus
// constants, predicates in place of branches: causal 8192 tokens 374 -> 333 us.  Without the turns both tiles fall
// into step, softmax with softmax and MMAs with MMAs: 421 us.)
// P is rounded to the 16-bit type of V (half a step each; fp16 ones are held times 2^7, kWeightBits, m being 7
// less); l sums it unrounded in fp32.
//
// Bound: for a block of 128 keys of both tiles the MMAs take 2100 cycles (1100 at d 64), one tile's chain of
// softmax (1200 alone, more beside the other's), barriers and its own MMAs about 2700.  Measured (32 heads on 8,
// bf16, d 128, 8192 tokens): causal 317 to 324 us, 1700 TFLOP/s of visible pairs, 0.85 of the peak; window 1024 and 4
// sinks 113 us, 1141 TFLOP/s, 9 and a quarter blocks walked for 8 seen.  Two sequences of 4k after 513 keys, 16
// heads on 2, d 64: 93 us, 855 TFLOP/s.
//
// A key that a row does not see gets weight 0 there, but 0 times a NaN or infinity in V still reaches the row
// through the product.  (One in K does not: the scores of unseen keys are replaced.  So a sum l that is NaN
// comes from a key that the row sees, and the row is NaN.)  Items with rows whose l is finite and whose result is not are
// noted, and after the last item, when no other warp waits for anything, their non-finite results are computed once
// more from what the rows see (window_again).  One prompt of 4096 tokens, 8 heads on 2, d 128, causal, 0.09 ms: with a
// NaN in K 0.07 ms, with one in V 1.4 ms (row by row and key by key inside the loop it was 56 ms for either), with
// NaN in a dim of every V 2.6 ms.
#include <atomic>
#include <climits>

#include "tl_serve.cuh"
#include "tl_softmax.cuh"

namespace tl {

namespace win {
constexpr int kKeys = 128, kNarrow = 32, kMaxBatch = 1024;
constexpr int kLevels = 256, kSorted = 32;  // order of items: see WinPlan
constexpr int kHeld = 32, kReaders = 11;    // items listed; warps that walk them
constexpr int kThreads = 384;          // warps 0-3, softmax warpgroups 4-7 and 8-11
constexpr float kRescale = 8.f;
template <int D>
struct Shape {
  static constexpr int kHalves = D / 64;             // 64-column SW128 boxes of a row
  static constexpr int kBox = 128 * 128;             // 128 rows of 64 columns
  static constexpr int kTileBytes = kHalves * kBox;  // Q of a tile, a K block, a V block
  static constexpr int kSlots = 4;                   // K and V blocks in flight, two of each
  static constexpr int kRingOff = 2 * kTileBytes;
  static constexpr int kBarOff = kRingOff + kSlots * kTileBytes;
  static constexpr int kCumOff = kBarOff + 256;
  static constexpr int kPlanOff = kCumOff + (kMaxBatch + 4) * 4;
  static constexpr int kHeldOff = kPlanOff + (kLevels + 4 + 2 * kSorted) * 4;
  static constexpr int kAgainOff = kHeldOff + kHeld * 64;  // a softmax warp's first and last item for window_again
  static constexpr int kSmem = 1024 + kAgainOff + 9 * 8;                // (and the plan's numbers for it)
};
constexpr uint32_t kColS = 0, kColO = 256;  // TMEM columns: S_t at 128 t, O_t at 256 + 128 t
}  // namespace win

struct WindowParams {
  CUtensorMap tq;  // {d, heads, total_q}, box {64, G, 128 / G}
  CUtensorMap tk;  // {d, kv_heads, total_k}, box {64, 1, 128}
  CUtensorMap tv;
  Common common;
  const uint8_t* q;
  const uint8_t* k;
  const uint8_t* v;
  uint8_t* out;
  float* lse;
  long long q_token, q_head, k_token, k_head, v_token, v_head, out_token, out_head;  // bytes
  const int* cu_q;
  const int* cu_k;
  int batch, total_q, total_k, heads, kv_heads, group;
  int tokens;  // of a tile: 128 / group
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

// A sequence's bounds, as rows of q and k; nothing (n = 0) if they are out of order or range.
struct WinSeq {
  int q0, k0, n, off;  // first rows, queries, position of the first query
};
__device__ __forceinline__ WinSeq win_seq(const WindowParams& p, int b, bool report) {
  const int q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1), k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
  WinSeq s;
  if (q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k) {
    if (report) report_index(p.common.status, static_cast<unsigned long long>(b));
    s.q0 = s.k0 = s.n = s.off = 0;
  } else {
    s.q0 = q0;
    s.k0 = k0;
    s.n = q1 - q0;
    s.off = (k1 - k0) - s.n;
  }
  return s;
}

// The order of the items.  Of 2 to 32 sequences with several items a CTA, those whose tiles stand further into their keys come first,
// in 256 levels of `gran` positions, so that a round of CTAs has items of about the same length; otherwise
// sequence by sequence, the last tiles first.  (Sequence by sequence and so, 32 heads on 8, d 128, causal: 2 of up to 8k
// tokens 571 and 536 us, 8 of up to 4k 503 and 454, 32 of up to 4k 1295 and 1242; short ones lose, 32 of up to 600 101
// and 107.  A lane has a sequence, hence 32; a batch of 33 of up to 4k takes what it takes by sequence, 786.)
struct WinPlan {
  bool sorted;
  int* cum;    // [batch + 1]: items before each sequence (if not sorted)
  int* above;  // [kLevels + 1]: above[0] all pairs of tiles, above[v + 1] those that start at (v + 1) gran or later
  int* off;    // [kSorted]: position of a sequence's first query
  int* pairs;  // [kSorted]: its pairs of tiles
  int gran, items;
};
// Of a sequence's pairs of tiles, those that start at position x or later.
__device__ __forceinline__ int pairs_from(int pairs, int off, int step, int x) {
  const int first = x <= off ? 0 : (x - off + step - 1) / step;
  return first < pairs ? pairs - first : 0;
}

// An item and the key blocks it walks.
struct alignas(16) WinItem {
  WinSeq s;
  int hk, i0;     // kv head, first query
  bool two;       // its second tile has queries
  int lo;         // first key of the blocks after the sinks'
  int sinks;      // keys [0, sinks) of the sinks' blocks
  int nh, nb;     // blocks of sinks, all blocks
  bool narrow;    // the sinks fit in kNarrow keys: their block is that wide
};
// (a whole warp at once)
__device__ __forceinline__ WinItem win_item(const WindowParams& p, const WinPlan& plan, int idx, int lane) {
  const int step = 2 * p.tokens;
  WinItem w;
  int b, pair;
  if (plan.sorted) {
    const int rank = idx / p.kv_heads;
    w.hk = idx - rank * p.kv_heads;
    int lo = 0, hi = win::kLevels;  // the level v with above[v + 1] <= rank < above[v]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (plan.above[mid + 1] <= rank) hi = mid; else lo = mid + 1;
    }
    const int n = lane < p.batch ? plan.pairs[lane] : 0, off = lane < p.batch ? plan.off[lane] : 0;
    const int after = pairs_from(n, off, step, (lo + 1) * plan.gran);
    const int here = (lo ? pairs_from(n, off, step, lo * plan.gran) : n) - after;
    int sum = here;
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, sum, x);
      if (lane >= x) sum += o;
    }
    const int in = rank - plan.above[lo + 1];
    b = __popc(__ballot_sync(0xffffffffu, sum <= in));
    pair = __shfl_sync(0xffffffffu, n - after - 1 - (in - (sum - here)), b);
  } else {
    int lo = 0, hi = p.batch;  // the sequence that holds the item: cum[b] <= idx < cum[b + 1]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (plan.cum[mid] <= idx) lo = mid; else hi = mid;
    }
    b = lo;
    const int in = idx - plan.cum[lo], pairs = (plan.cum[lo + 1] - plan.cum[lo]) / p.kv_heads;
    w.hk = in % p.kv_heads;
    pair = pairs - 1 - in / p.kv_heads;
  }
  w.s = win_seq(p, b, false);
  w.i0 = pair * step;
  w.two = w.i0 + p.tokens < w.s.n;
  const int end = min(w.i0 + step, w.s.n);  // one past the last query
  const int first = w.s.off + w.i0, last = w.s.off + end - 1;  // positions
  w.lo = p.window == 0 || first < p.window ? 0 : first - p.window + 1;
  w.sinks = min(p.sinks, w.lo);
  w.nh = (w.sinks + win::kKeys - 1) / win::kKeys;
  w.nb = last < 0 ? 0 : w.nh + (last - w.lo) / win::kKeys + 1;
  if (last < 0) w.nh = 0;
  w.narrow = w.nh == 1 && w.sinks <= win::kNarrow;
  return w;
}
__device__ __forceinline__ int win_start(const WinItem& w, int j) {
  return j < w.nh ? j * win::kKeys : w.lo + (j - w.nh) * win::kKeys;
}

// A CTA's k-th item: one of each round of gridDim.x, forwards and backwards in turn, so that the one with the
// longest item of a round has the shortest of the next (one causal prompt of 8k: 408 us forwards, 370 so).
// From `items` on there is none.
__device__ __forceinline__ int win_index(int k) {
  const int grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  return k * grid + (k & 1 ? grid - 1 - cta : cta);
}

// MMAs (kind::f16, one CTA) and commits by the thread of a converged warp that has `lead`: a predicate on each
// instruction, no branch, so that what they take is computed once a warp.
__device__ __forceinline__ void mma_ss(uint32_t lead, uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(lead)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}
// A value that is the same in the whole warp, in a uniform register.
__device__ __forceinline__ int uniform(int v) { return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(v))); }

// umma_desc_sw128 without its address.
__host__ __device__ constexpr uint64_t umma_desc_base(uint32_t lbo) {
  return static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16 | static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// True in one thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// 16 fp32 columns of this warp's lanes, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n\t"
      "tcgen05.wait::st.sync.aligned;" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// The register share of this warpgroup, of those that the CTA was launched with.
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The first n of 32 bits.
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// The results of 16 rows of a tile that are not finite, once more by one warp, on mma.sync m16n8k16 with the rows as its
// rows: 16 keys at a time, of those that any of the rows sees, with a running maximum and sum.  V's elements that are not
// finite are taken as 0 in the product, and each is then added, times its weight in fp32, to the rows that see its
// key.  Results that are finite keep their bits.
template <class T, int D>
__device__ __forceinline__ void window_again(const WindowParams& p, const WinItem& w, int t, int r0, int lane) {
  constexpr uint32_t kExp = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;  // all ones: not finite
  const int g = lane >> 2, c2 = 2 * (lane & 3);  // this thread: rows g and g + 8, columns c2 and c2 + 1 of every 8
  auto odd = [](uint32_t v) { return (v & kExp) == kExp; };
  auto load = [](const uint8_t* at) { return *reinterpret_cast<const uint32_t*>(at); };
  const uint8_t* qp[2];
  uint8_t* op[2];
  bool live[2], any = false;
  int pos[2], from[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = r0 + g + 8 * x, tok = row / p.group, h = w.hk * p.group + row - tok * p.group;
    const int i = w.i0 + t * p.tokens + tok;
    live[x] = tok < p.tokens && i < w.s.n;
    pos[x] = live[x] ? w.s.off + i : -1;
    from[x] = live[x] ? seen_keys(pos[x], p.window, p.sinks).from : INT_MAX;
    qp[x] = p.q + (w.s.q0 + i) * p.q_token + h * p.q_head + c2 * 2;
    op[x] = p.out + (w.s.q0 + i) * p.out_token + h * p.out_head + c2 * 2;
    if (live[x])
#pragma unroll 4
      for (int n = 0; n < D / 8; ++n) {
        const uint32_t v = load(op[x] + 16 * n);
        any |= odd(v) || odd(v >> 16);
      }
  }
  if (!__any_sync(0xffffffffu, any)) return;
  const int last = __reduce_max_sync(0xffffffffu, max(pos[0], pos[1]));
  const int first = __reduce_min_sync(0xffffffffu, min(from[0], from[1]));
  const int sinks = p.sinks;
  auto sees = [&](int x, int j) { return j <= pos[x] && (j >= from[x] || j < sinks); };
  const uint8_t* kb = p.k + w.s.k0 * p.k_token + w.hk * p.k_head;
  const uint8_t* vb = p.v + w.s.k0 * p.v_token + w.hk * p.v_head;
  float o[D / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int n = 0; n < D / 8; ++n)
#pragma unroll
    for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
  for (int j0 = 0; j0 <= last; j0 += 16) {
    if (j0 >= sinks && j0 + 16 <= first) j0 = first & ~15;
    float s[2][4];  // rows g (0, 1) and g + 8 (2, 3), keys c2 and c2 + 1 of both eights
    const uint8_t* kp[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      kp[e] = kb + min(j0 + 8 * e + g, last) * p.k_token + c2 * 2;  // (past the last key: that key again, without weight)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[e][x] = 0.f;
    }
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t q[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) q[x] = live[x & 1] ? load(qp[x & 1] + 32 * d + 16 * (x >> 1)) : 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e) mma16816<T>(s[e], q, load(kp[e] + 32 * d), load(kp[e] + 32 * d + 16));
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float top = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& v = s[e >> 1][2 * x + (e & 1)];
        v = sees(x, j0 + 8 * (e >> 1) + c2 + (e & 1)) ? v * p.sl2 : -INFINITY;
        top = fmaxf(top, v);
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float mn = fmaxf(m[x], top - kWeightBits<T>), keep = m[x] == -INFINITY ? 0.f : ex2_approx(m[x] - mn);
      m[x] = mn;
      l[x] *= keep;
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        o[n][2 * x] *= keep;
        o[n][2 * x + 1] *= keep;
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float& v = s[e >> 1][2 * x + (e & 1)];
        v = v == -INFINITY ? 0.f : ex2_approx(v - mn);
        l[x] += v;
      }
    }
    const uint32_t a[4] = {from_f32x2<T>(s[0][0], s[0][1]), from_f32x2<T>(s[0][2], s[0][3]), from_f32x2<T>(s[1][0], s[1][1]),
                           from_f32x2<T>(s[1][2], s[1][3])};
    uint32_t some = 0;  // eights of dims with a V that is not finite
    const uint16_t* vp[4];  // this thread's keys c2, c2 + 1 of both eights, dim g of every 8
#pragma unroll
    for (int x = 0; x < 4; ++x)
      vp[x] = reinterpret_cast<const uint16_t*>(vb + min(j0 + 8 * (x >> 1) + c2 + (x & 1), last) * p.v_token) + g;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      uint32_t v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        v[x] = vp[x][8 * n];
        if (odd(v[x])) {
          some |= 1u << n;
          v[x] = 0u;
        }
      }
      mma16816<T>(o[n], a, v[0] | v[1] << 16, v[2] | v[3] << 16);
    }
    some = __reduce_or_sync(0xffffffffu, some);
    if (some) {
      const int keys = min(16, last + 1 - j0);
#pragma unroll
      for (int n = 0; n < D / 8; ++n) {
        if (!(some >> n & 1u)) continue;
#pragma unroll 4
        for (int k = 0; k < 16; ++k) {
          const uint32_t v = k < keys ? load(vb + (j0 + k) * p.v_token + 16 * n + c2 * 2) : 0u;
          const float2 f = to_f32x2<T>(v);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float even = k & 8 ? s[1][2 * x] : s[0][2 * x], uneven = k & 8 ? s[1][2 * x + 1] : s[0][2 * x + 1];
            const float weight = __shfl_sync(0xffffffffu, k & 1 ? uneven : even, (lane & ~3) + ((k & 7) >> 1));
            if (odd(v) && sees(x, j0 + k)) o[n][2 * x] += weight * f.x;
            if (odd(v >> 16) && sees(x, j0 + k)) o[n][2 * x + 1] += weight * f.y;
          }
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 1);
    l[x] += __shfl_xor_sync(0xffffffffu, l[x], 2);
    if (!live[x]) continue;
    const float inv = 1.f / l[x];
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      uint32_t* at = reinterpret_cast<uint32_t*>(op[x] + 16 * n);
      const uint32_t was = *at, now = l[x] == 0.f ? 0u : from_f32x2<T>(o[n][2 * x] * inv, o[n][2 * x + 1] * inv);
      *at = (odd(was) ? now & 0xffffu : was & 0xffffu) | (odd(was >> 16) ? now & 0xffff0000u : was & 0xffff0000u);
    }
  }
}

template <class T, int D>
__global__ void __launch_bounds__(win::kThreads, 1) window_kernel(const __grid_constant__ WindowParams p) {
  using namespace win;
  using S = Shape<D>;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  // operand formats: bits 7-9 and 10-12, 0 fp16, 1 bf16
  constexpr uint32_t kFormat = kBf16 ? 0u : (1u << 7) | (1u << 10);
  constexpr uint32_t kDescS = umma_idesc_bf16(128, kKeys, false) & ~kFormat;
  constexpr uint32_t kDescNarrow = umma_idesc_bf16(128, kNarrow, false) & ~kFormat;
  constexpr uint32_t kDescO = umma_idesc_bf16(128, D, true) & ~kFormat;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* qfull = reinterpret_cast<uint64_t*>(base + S::kBarOff);
  uint64_t* qempty = qfull + 1;
  uint64_t* full = qfull + 2;              // [kSlots] a K or V block is there
  uint64_t* empty = full + S::kSlots;      // [kSlots] both tiles' MMAs have read it
  uint64_t* sfull = empty + S::kSlots;     // [2] S_t is there, every MMA before it complete
  uint64_t* pready = sfull + 2;            // [2][2] the first, the second 64 keys of P_t are there (and O_t rescaled)
  uint64_t* ofull = pready + 4;            // [2] the item's last PV_t is complete
  uint64_t* turn = ofull + 2;              // [2] tile t's MMAs may be issued
  uint64_t* listed = turn + 2;             // [2] a half of the list of items is written anew
  uint64_t* used = listed + 2;             // [2] all warps have read it
  uint64_t* drain = used + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(drain + 1);
  WinPlan plan;
  plan.cum = reinterpret_cast<int*>(base + S::kCumOff);
  plan.above = reinterpret_cast<int*>(base + S::kPlanOff);
  plan.off = plan.above + kLevels + 1;
  plan.pairs = plan.off + kSorted;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Common& c = p.common;

  for (int b = threadIdx.x; b < p.batch; b += kThreads) {
    const WinSeq s = win_seq(p, b, blockIdx.x == 0);
    const int pairs = (s.n + 2 * p.tokens - 1) / (2 * p.tokens);
    plan.cum[b + 1] = pairs * p.kv_heads;
    if (b < kSorted) {
      plan.off[b] = s.off;
      plan.pairs[b] = pairs;
    }
  }
  if (threadIdx.x == 0) {
    mbar_init(qfull, 1);
    mbar_init(qempty, 2);
    for (int i = 0; i < S::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sfull[t], 1);
      mbar_init(&pready[2 * t], 4);
      mbar_init(&pready[2 * t + 1], 4);
      mbar_init(&ofull[t], 1);
      mbar_init(&turn[t], 1);
      mbar_init(&listed[t], 1);
      mbar_init(&used[t], kReaders);
    }
    mbar_init(drain, 2);
    fence_mbar_init();
    tma_prefetch_map(&p.tq);
    tma_prefetch_map(&p.tk);
    tma_prefetch_map(&p.tv);
  }
  if (warp == 1) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  plan.gran = kKeys;
  plan.sorted = false;
  if (p.batch > 1 && p.batch <= kSorted) {  // in every warp alike
    int end = lane < p.batch ? plan.off[lane] + plan.pairs[lane] * 2 * p.tokens : 0, all = lane < p.batch ? plan.pairs[lane] : 0;
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
      end = max(end, __shfl_xor_sync(0xffffffffu, end, x));
      all += __shfl_xor_sync(0xffffffffu, all, x);
    }
    plan.gran = max(plan.gran, (end + kLevels - 1) / kLevels);
    plan.sorted = all * p.kv_heads > static_cast<int>(gridDim.x);
  }
  if (plan.sorted) {
    for (int v = threadIdx.x; v <= kLevels; v += kThreads) {
      int sum = 0;
      for (int b = 0; b < p.batch; ++b)
        sum += v ? pairs_from(plan.pairs[b], plan.off[b], 2 * p.tokens, v * plan.gran) : plan.pairs[b];
      plan.above[v] = sum;
    }
  } else if (warp == 0) {
    int sum = 0;
    for (int b0 = 0; b0 < p.batch; b0 += 32) {
      int v = b0 + lane < p.batch ? plan.cum[b0 + lane + 1] : 0;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, v, x);
        if (lane >= x) v += o;
      }
      if (b0 + lane < p.batch) plan.cum[b0 + lane + 1] = sum + v;
      sum += __shfl_sync(0xffffffffu, v, 31);
    }
    if (lane == 0) plan.cum[0] = 0;
  }
  __syncthreads();
  const int items = plan.sorted ? plan.above[0] * p.kv_heads : plan.cum[p.batch];
  if (threadIdx.x == 0) reinterpret_cast<int2*>(base + S::kAgainOff)[8] = make_int2(plan.sorted, plan.gran);
  // The list of the CTA's items: the first kHeld looked up by all warps at once, later ones by warp 3, half a list at a
  // time.  (Looked up by each warp as it came to them, the code in every role cost 4%: instruction fetch.)
  WinItem* held = reinterpret_cast<WinItem*>(base + S::kHeldOff);
  static_assert(sizeof(WinItem) <= 64, "room");
  for (int k = warp; k < kHeld && win_index(k) < items; k += kThreads / 32) {
    const WinItem w = win_item(p, plan, win_index(k), lane);
    if (lane == 0) held[k] = w;
  }
  __syncthreads();
  auto item = [&](int k, bool& ok) {
    constexpr int kHalf = kHeld / 2;
    const int h = k / kHalf & 1;
    if (k >= kHeld && k % kHalf == 0) ok = __all_sync(0xffffffffu, mbar_wait(&listed[h], (k / kHeld - 1) & 1, c, kSiteFull)) != 0;
    const WinItem w = held[k % kHeld];
    if (k % kHalf == kHalf - 1) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&used[h]);
    }
    return w;
  };
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);
  // Registers: 128 x 104 + 256 x 200 = 384 x 168, what the CTA has at launch.
  if (warp < 4) {
    regs_down<104>();
  if (warp == 0) {
    // ------------------------------------------------------------ loads (lane 0; the whole warp finds the items)
    bool ok = true;
    int u = 0, nq = 0;  // blocks and items loaded
    const uint32_t q_bytes = static_cast<uint32_t>(p.tokens * p.group) * 128 * S::kHalves;
    for (int k = 0; ok && win_index(k) < items; ++k) {
      const WinItem w = item(k, ok);
      if (w.nb == 0 || !ok) continue;
      if (lane == 0) {
        ok = mbar_wait(qempty, (nq & 1) ^ 1, c, kSiteEmpty);
        if (ok) {
          mbar_arrive_expect_tx(qfull, q_bytes * (w.two ? 2 : 1));
          for (int t = 0; t < (w.two ? 2 : 1); ++t)
            for (int h = 0; h < S::kHalves; ++h)
              tma_load_3d(base + t * S::kTileBytes + h * S::kBox, &p.tq, qfull, 64 * h, w.hk * p.group,
                          w.s.q0 + w.i0 + t * p.tokens);
          ++nq;
        }
        for (int j = 0; j < w.nb && ok; ++j)
          for (int kv = 0; kv < 2 && ok; ++kv) {
            const int s = u % S::kSlots;
            ok = mbar_wait(&empty[s], ((u / S::kSlots) & 1) ^ 1, c, kSiteEmpty);
            if (!ok) break;
            mbar_arrive_expect_tx(&full[s], S::kTileBytes);
            for (int h = 0; h < S::kHalves; ++h)
              tma_load_3d(base + S::kRingOff + s * S::kTileBytes + h * S::kBox, kv ? &p.tv : &p.tk, &full[s], 64 * h, w.hk,
                          w.s.k0 + win_start(w, j));
            ++u;
          }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    }
    // every load has landed before the CTA ends (at once, unless a wait ran out)
    if (lane == 0) {
      if (nq) mbar_wait(qfull, (nq - 1) & 1, c, kSiteDrain);
      for (int j = u > S::kSlots ? u - S::kSlots : 0; j < u; ++j) mbar_wait(&full[j % S::kSlots], (j / S::kSlots) & 1, c, kSiteDrain);
    }
    __syncwarp();
  } else if (warp <= 2) {
    // ------------------------------------------------------------ MMAs
    // A warp for each tile.  It walks along as a whole and one thread of it issues; the tiles' MMAs are issued in
    // turn, S_0 S_1 | PV_0 S_0' | PV_1 S_1' | ..  Descriptors are a uniform base and constants: slots 0 and 2 hold K
    // blocks, 1 and 3 V blocks.
    {
      const uint32_t lead = elect_one() ? 1u : 0u, t = uniform(warp - 1), tm = uniform(tmem) + 128 * t;
      const uint32_t s0 = uniform((smem_u32(base) & 0x3FFFFu) >> 4), q0 = s0 + t * (S::kTileBytes >> 4);
      const int n_items = uniform(items);
      bool ok = true;
      int nq = 0, np = 0, nt = 0, g = 0;  // items, P blocks consumed, turns, blocks gone by
      auto wait = [&](uint64_t* bar, int n, unsigned site) { return __all_sync(0xffffffffu, mbar_wait(bar, n & 1, c, site)) != 0; };
      constexpr uint64_t kDescK = umma_desc_base(16), kDescMn = umma_desc_base(S::kBox);
      auto my_turn = [&](bool two) { return !two || (t == 0 && nt == 0) || wait(&turn[t], t ? nt : nt - 1, kSiteFull); };
      auto next_turn = [&](bool two) {
        if (!two) return;
        ++nt;
        if (lane == 0) mbar_arrive(&turn[1 - t]);
      };
      // S_t = Q_t K^T; then this tile needs the slot (and after the item's last block, Q) no more
      auto mma_s = [&](auto slot, uint32_t desc, bool last_block) {
        constexpr int kAt = S::kRingOff + decltype(slot)::value * S::kTileBytes;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * S::kBox + (k & 3) * 32;
          mma_ss(lead, tm + kColS, kDescK | (q0 + (off >> 4)), kDescK | (s0 + ((kAt + off) >> 4)), desc, k ? 1u : 0u);
        }
        mma_commit(lead, &sfull[t]);
        mma_commit(lead, &empty[decltype(slot)::value]);
        if (last_block) mma_commit(lead, qempty);
      };
      // O_t += P_t V over 64 keys (kNarrow and none of a narrow block)
      auto mma_o = [&](auto slot, auto hf, bool narrow, uint32_t onto) {
        constexpr int kFirst = decltype(hf)::value * (kKeys / 32), kAt = S::kRingOff + decltype(slot)::value * S::kTileBytes;
#pragma unroll
        for (int k = 0; k < kKeys / 32; ++k) {
          if (narrow && kFirst + k >= kNarrow / 16) break;
          mma_ts(lead, tm + kColO, tm + kColS + (kFirst + k) * 8, kDescMn | (s0 + ((kAt + (kFirst + k) * 2048) >> 4)), kDescO,
                 kFirst + k ? 1u : onto);
        }
      };
      // V of block g is in slot 2 kPar + 1, K of the next in the other K slot
      auto block = [&](auto par, bool two, bool narrow, uint32_t onto, bool more, bool last_k) {
        constexpr int kPar = decltype(par)::value;
        using Next = std::integral_constant<int, 2 * (1 - kPar)>;
        using V = std::integral_constant<int, 2 * kPar + 1>;
        if (!wait(&full[V::value], g >> 1, kSiteFull) || !wait(&pready[2 * t], np, kSiteTmemFull) || !my_turn(two)) return false;
        tc_fence_after();
        mma_o(V(), std::integral_constant<int, 0>(), narrow, onto);
        if (!wait(&pready[2 * t + 1], np, kSiteTmemFull)) return false;
        tc_fence_after();
        mma_o(V(), std::integral_constant<int, 1>(), narrow, 1u);
        mma_commit(lead, &empty[V::value]);
        if (!more) mma_commit(lead, &ofull[t]);
        ++np;
        ++g;
        if (more) {
          if (!wait(&full[Next::value], g >> 1, kSiteFull)) return false;
          mma_s(Next(), kDescS, last_k);
        }
        next_turn(two);
        return true;
      };
      for (int it = 0; ok && win_index(it) < n_items; ++it) {
        const WinItem w = item(it, ok);
        const int nb = uniform(w.nb);
        const bool two = uniform(w.two) != 0, narrow = uniform(w.narrow) != 0;
        if (nb == 0 || !ok) continue;
        ok = wait(qfull, nq, kSiteFull);
        if (!ok) break;
        ++nq;
        if (t && !two) {  // nothing to do, but the loads go by
          for (int j = 0; j < nb && ok; ++j, ++g)
            for (int kv = 0; kv < 2 && ok; ++kv) {
              const int slot = 2 * (g & 1) + kv;
              ok = wait(&full[slot], g >> 1, kSiteFull);
              if (ok && lane == 0) mbar_arrive(&empty[slot]);
            }
          if (lane == 0) mbar_arrive(qempty);
          continue;
        }
        ok = wait(&full[2 * (g & 1)], g >> 1, kSiteFull) && my_turn(two);
        if (!ok) break;
        tc_fence_after();
        const uint32_t desc = narrow ? kDescNarrow : kDescS;
        if (g & 1) mma_s(std::integral_constant<int, 2>(), desc, nb == 1);
        else mma_s(std::integral_constant<int, 0>(), desc, nb == 1);
        next_turn(two);
        for (int j = 0; j < nb && ok; ++j) {
          const bool more = j + 1 < nb, nar = narrow && j == 0, last_k = j + 2 == nb;
          ok = g & 1 ? block(std::integral_constant<int, 1>(), two, nar, j > 0, more, last_k)
                     : block(std::integral_constant<int, 0>(), two, nar, j > 0, more, last_k);
        }
      }
      mma_commit(lead, drain);
      mbar_wait(drain, 0, c, kSiteDrain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ the list of items, from the kHeld-th on
    constexpr int kHalf = kHeld / 2;
    bool ok = true;
    for (int k = kHeld; ok && win_index(k) < items; k += kHalf) {
      const int h = k / kHalf & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(&used[h], (k / kHeld - 1) & 1, c, kSiteEmpty)) != 0;
      if (!ok) break;
      for (int x = k; x < k + kHalf && win_index(x) < items; ++x) {
        const WinItem w = win_item(p, plan, win_index(x), lane);
        if (lane == 0) held[x % kHeld] = w;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&listed[h]);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    regs_up<200>();
    const int t = (warp - 4) >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + kColS + 128 * t + lanes, to = tmem + kColO + 128 * t + lanes;
    const int tok = row / p.group, hg = row - tok * p.group;
    int2* const again = reinterpret_cast<int2*>(base + S::kAgainOff) + warp - 4;
    if (lane == 0) *again = make_int2(-1, -1);
    bool ok = true;
    int ns = 0, no = 0;  // S blocks and items seen
    for (int it = 0; ok && win_index(it) < items; ++it) {
      const WinItem w = item(it, ok);
      if ((t && !w.two) || !ok) continue;
      const int i = w.i0 + t * p.tokens + tok;  // this row's query
      const bool live = tok < p.tokens && i < w.s.n;
      const int pos = live ? w.s.off + i : -1;
      const int from = p.window == 0 || pos < p.window ? 0 : pos - p.window + 1;  // first key of its window
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < w.nb && ok; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sfull[t], ns & 1, c, kSiteTmemFull));
        if (!ok) break;
        ++ns;
        tc_fence_after();
        // the keys of this block that the row sees: [a, z), or before s2
        const int start = win_start(w, j);
        const bool head = j < w.nh;
        // (rows without a query are not cut: what they compute goes nowhere)
        const int z = !live ? kKeys : (head ? min(w.sinks, pos + 1) : pos + 1) - start;
        const int a = head || !live ? 0 : from - start, s2 = head ? 0 : p.sinks - start;
        if (w.narrow && j == 0) {  // the sinks, in kNarrow columns; an item's first block
          uint32_t r[kNarrow], pk[kNarrow / 2];
          tmem_ld32_issue(ts, r);
          tmem_ld_wait(r);
          float top = -INFINITY;
#pragma unroll
          for (int k = 0; k < kNarrow; ++k) {
            if (k >= z) r[k] = 0xff800000u;
            top = fmaxf(top, __uint_as_float(r[k]));
          }
          m = top * p.sl2 - kWeightBits<T>;
          const float nm = m == -INFINITY ? 0.f : -m;
#pragma unroll
          for (int k = 0; k < kNarrow / 2; ++k) {
            const float e0 = ex2_approx(fmaf(__uint_as_float(r[2 * k]), p.sl2, nm));
            const float e1 = ex2_approx(fmaf(__uint_as_float(r[2 * k + 1]), p.sl2, nm));
            l += e0 + e1;
            pk[k] = from_f32x2<T>(e0, e1);
          }
          tmem_st16(ts, pk);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&pready[2 * t]);
            mbar_arrive(&pready[2 * t + 1]);
          }
          continue;
        }
        const bool cut = __any_sync(0xffffffffu, z < kKeys || (a > 0 && s2 < kKeys));
        uint32_t seen[4] = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
        if (cut)
#pragma unroll
          for (int q = 0; q < 4; ++q) seen[q] = low_bits(z - 32 * q) & (~low_bits(a - 32 * q) | low_bits(s2 - 32 * q));
        // all 128 scores at once
        uint32_t r[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld32_issue(ts + 32 * q, r[q]);
        tmem_ld_wait(r[0]);
#pragma unroll
        for (int q = 1; q < 4; ++q) tmem_ld_after(r[q]);
        if (cut)
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int k = 0; k < 32; ++k) r[q][k] = (seen[q] >> k) & 1u ? r[q][k] : 0xff800000u;  // -inf
        float mx[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = __uint_as_float(r[0][k]);
#pragma unroll
        for (int i = 8; i < 120; i += 16)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mx[k] = fmax3(mx[k], __uint_as_float(r[(i + k) >> 5][(i + k) & 31]), __uint_as_float(r[(i + 8 + k) >> 5][(i + 8 + k) & 31]));
#pragma unroll
        for (int k = 0; k < 8; ++k) mx[k] = fmaxf(mx[k], __uint_as_float(r[3][24 + k]));
        const float top = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * p.sl2 - kWeightBits<T>;  // sl2 > 0
        // (a row without a query has no vote: what it holds, of another sequence or left by an earlier call, would move
        // the others' maxima and so their last bits)
        if (__any_sync(0xffffffffu, live && top > m + kRescale)) {
          const float mn = fmaxf(m, top), keep = mn == -INFINITY ? 1.f : ex2_approx(m - mn);
          m = mn;
          l *= keep;
          if (j > 0) {  // PV_t of the blocks before is complete (it precedes this S_t)
#pragma unroll 1
            for (int q = 0; q < D / 16; ++q) {
              uint32_t o[16];
              tmem_ld16(to + 16 * q, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
              tmem_st16(to + 16 * q, o);
            }
          }
        }
        // weights, 64 keys at a time; P's columns lie over scores that are read
        const float nm = m == -INFINITY ? 0.f : -m;
        const unsigned long long sl2x2 = f2(p.sl2, p.sl2), nmx2 = f2(nm, nm);
        unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t pk[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int i = 64 * half + 2 * k;
            float y0, y1;
            f2_split(ffma2(f2(__uint_as_float(r[i >> 5][i & 31]), __uint_as_float(r[i >> 5][(i & 31) + 1])), sl2x2, nmx2), y0, y1);
            const float e0 = ex2_approx(y0), e1 = ex2_approx(y1);
            sum[k & 1] = fadd2(sum[k & 1], f2(e0, e1));
            pk[k] = from_f32x2<T>(e0, e1);
          }
          tmem_st32_raw(ts + 32 * half, pk);
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pready[2 * t + half]);
        }
        float a0, a1;
        f2_split(fadd2(sum[0], sum[1]), a0, a1);
        l += a0 + a1;
      }
      if (!ok) break;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      unsigned long long zero = 0ull;  // 0 times every sum: NaN if one is not finite
      if (w.nb) {
        ok = __all_sync(0xffffffffu, mbar_wait(&ofull[t], no & 1, c, kSiteTmemFull));
        if (!ok) break;
        ++no;
        tc_fence_after();
      }
      // Four lanes hold four rows; they exchange 16-byte pieces so that a store covers 64 bytes of each of
      // eight rows instead of 16 of 32.  Lane 4 r + x then stores piece x of rows 4 r .. 4 r + 3.
      const long long mine = (w.s.q0 + i) * p.out_token + (w.hk * p.group + hg) * p.out_head;
      const uint32_t lives = __ballot_sync(0xffffffffu, live);
      uint8_t* dst[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) dst[x] = p.out + __shfl_sync(0xffffffffu, mine, (lane & ~3) + x) + 16 * (lane & 3);
#pragma unroll 1
      for (int q = 0; q < D / 32; ++q) {
        float o[32];
        if (w.nb) {
          tmem_ld32(to + 32 * q, o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0.f;
        }
        uint32_t v[4][4];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          zero = ffma2(f2(o[2 * k], o[2 * k + 1]), 0ull, zero);
          v[k >> 2][k & 3] = from_f32x2<T>(o[2 * k] * inv, o[2 * k + 1] * inv);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // the transpose, by pairs at distance 1, then 2
          const bool up = (lane >> h) & 1;
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int lo = h ? x : 2 * x, hi = lo + (1 << h);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? v[lo][k] : v[hi][k], 1 << h);
              if (up) v[lo][k] = got;
              else v[hi][k] = got;
            }
          }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if ((lives >> ((lane & ~3) + x)) & 1u)
            *reinterpret_cast<uint4*>(dst[x] + 64 * q) = make_uint4(v[x][0], v[x][1], v[x][2], v[x][3]);
      }
      float z0, z1;
      f2_split(zero, z0, z1);
      if (__any_sync(0xffffffffu, live && l == l && !(z0 + z1 == 0.f))) {
        if (lane == 0) {
          if (again->x < 0) again->x = it;
          again->y = it;
        }
      }
      if (live && p.lse)
        p.lse[static_cast<long long>(w.s.q0 + i) * p.heads + w.hk * p.group + hg] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
      tc_fence_before();
      __syncwarp();
    }
    __syncwarp();
    const int2 range = *again;
    if (ok && range.x >= 0) {  // (the rows were stored by other lanes: the barriers above)
      // (the plan from shared memory: registers would hold it all along)
      WinPlan late;
      const int2 numbers = reinterpret_cast<const int2*>(base + S::kAgainOff)[8];
      late.sorted = numbers.x != 0;
      late.gran = numbers.y;
      late.cum = reinterpret_cast<int*>(base + S::kCumOff);
      late.above = reinterpret_cast<int*>(base + S::kPlanOff);
      late.off = late.above + kLevels + 1;
      late.pairs = late.off + kSorted;
      for (int it = range.x; it <= range.y; ++it) {
        const WinItem w = win_item(p, late, win_index(it), lane);
        if (w.nb == 0 || (t && !w.two)) continue;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) window_again<T, D>(p, w, t, (warp & 3) * 32 + 16 * h, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <class T, int D>
static int window_launch(tl_ctx* ctx, const WindowParams& p, cudaStream_t st) {
  auto kern = window_kernel<T, D>;
  static std::atomic<unsigned long long> ready{0};
  if (!smem_ready(ready, ctx->device, reinterpret_cast<const void*>(kern), win::Shape<D>::kSmem)) return TL_ERR_CUDA;
  const long long most = (p.total_q / (2LL * p.tokens) + p.batch) * p.kv_heads;  // items there can be
  const int grid = most < ctx->ctas ? static_cast<int>(most) : ctx->ctas;
  kern<<<grid, win::kThreads, win::Shape<D>::kSmem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? TL_OK : TL_ERR_CUDA;
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
      batch < 0 || batch > 1024 || total_q < 0 || total_k < 0 || window < 0 || sinks < 0 || !scale_ok(scale) ||
      static_cast<long long>(total_q) * heads >= (1LL << 31))
    return TL_ERR_INVALID;
  for (long long s : {q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                      out_token_stride, out_head_stride})
    if (!esize_ok(s, 2)) return TL_ERR_INVALID;
  if (total_q == 0 || heads == 0 || batch == 0) return TL_OK;
  // (a row read as another one, by a stride of 0, is refused: a tensor map has none)
  if ((total_q > 1 && !q_token_stride) || (heads > 1 && !q_head_stride)) return TL_ERR_INVALID;
  if ((total_k > 1 && (!k_token_stride || !v_token_stride)) || (total_k > 0 && kv_heads > 1 && (!k_head_stride || !v_head_stride)))
    return TL_ERR_INVALID;
  if (!q || !out || !cu_q || !cu_k || !aligned16(q) || !aligned16(out)) return TL_ERR_INVALID;
  if (total_k > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return TL_ERR_INVALID;
  if (cudaSetDevice(ctx->device) != cudaSuccess) return TL_ERR_CUDA;
  WindowParams p;
  std::memset(&p, 0, sizeof(p));
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
  p.kv_heads = kv_heads;
  p.tokens = 128 / p.group;
  const auto dt = dtype == TL_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  // a dimension of one entry has any stride; a map wants a valid one
  auto stride = [&](long long bytes, int n) { return static_cast<uint64_t>(n > 1 ? bytes : 2 * d); };
  const int rows_k = total_k > 0 ? total_k : 1, heads_k = total_k > 0 ? kv_heads : 1;  // (no keys: a map of q, never read)
  if (!tmap_3d_strided(&p.tq, dt, q, d, heads, total_q, stride(p.q_head, heads), stride(p.q_token, total_q), 64, p.group,
                       p.tokens) ||
      !tmap_3d_strided(&p.tk, dt, total_k > 0 ? k : q, d, heads_k, rows_k, stride(p.k_head, heads_k),
                       stride(p.k_token, total_k), 64, 1, win::kKeys) ||
      !tmap_3d_strided(&p.tv, dt, total_k > 0 ? v : q, d, heads_k, rows_k, stride(p.v_head, heads_k),
                       stride(p.v_token, total_k), 64, 1, win::kKeys))
    return TL_ERR_CUDA;
  p.common = make_common(ctx);
  p.common.trace_hdr = nullptr;  // this kernel records no trace spans
  p.common.trace = nullptr;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == TL_BF16) return d == 64 ? window_launch<__nv_bfloat16, 64>(ctx, p, st) : window_launch<__nv_bfloat16, 128>(ctx, p, st);
  return d == 64 ? window_launch<__half, 64>(ctx, p, st) : window_launch<__half, 128>(ctx, p, st);
}
