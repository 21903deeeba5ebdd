// The paged key/value cache: appending new rows, and the attention of one new token over it.
#include <atomic>
#include <type_traits>

#include "tl_serve.cuh"
#include "tl_softmax.cuh"

namespace tl {

struct CacheArgs {
  uint8_t* k;
  uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  long long page_stride, row_stride, head_stride;  // bytes
  int num_pages, page_size, kv_heads;
};

// n / d for n < 2^31 as (umulhi(n, mul) + n) >> shift, exact.
struct FastDiv {
  uint32_t mul, shift;
};
__device__ __forceinline__ uint32_t divide(uint32_t n, FastDiv d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// ---------------------------------------------------------------------------- append
// Each thread copies 16 bytes of a K and of a V row (8 bytes written for e4m3): a row a thread, all threads of an
// SM resident, the rows' loads beside that of the slot, which only the stores need.  HBM and the ramp of a short
// launch bound a prompt's rows (8192 tokens of 8 heads of 128: bf16 12.3 us, 0.81 of the copy rate; into e4m3
// 11.8 us, 0.63; two or four rows a thread 15.3 and 18.6, with the slot first 13.0), the launch a step's (64
// tokens: 1.8 us).
struct AppendParams {
  CacheArgs c;
  DevStatus* status;
  const uint8_t* k;
  const uint8_t* v;
  long long k_token, k_head, v_token, v_head;  // bytes
  const int* slots;
  FastDiv by_heads, by_page;
  uint32_t rows;  // tokens * kv_heads
};

// 8 elements of T divided by the scale, as e4m3 (nearest even, saturating; NaN stays NaN).  The quotient is the
// IEEE one, from the scale's reciprocal y, which a thread needs once: q += (x - q s) y twice from q = x y.  The first
// step leaves q within a unit in the last place, and then the second is exact (Markstein 1990: for y the
// rounded reciprocal and a remainder by a fused multiply-add).  That asks for a positive scale whose reciprocal and
// remainders do not leave the range (a quotient that small is 0 in e4m3 either way) and finite quotients;
// anything else is divided.  (With divisions throughout 8192 tokens take 12.8 us instead of 11.8.)
struct Scale {
  float s, y;
  bool plain;
};
__device__ __forceinline__ Scale read_scale(const float* scales, int head) {
  Scale c;
  c.s = scales ? __ldg(scales + head) : 1.f;
  c.y = __frcp_rn(c.s);
  c.plain = c.s >= 0x1p-60f && c.s <= 0x1p60f;
  return c;
}
template <class T>
__device__ __forceinline__ uint2 quantise8(uint4 x, Scale c) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  const unsigned long long y = f2(c.y, c.y), ms = f2(-c.s, -c.s);
  uint32_t out[4];
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = to_f32x2<T>(in[i]);
    const unsigned long long a = f2(f.x, f.y);
    unsigned long long q = fmul2(a, y);
    q = ffma2(ffma2(q, ms, a), y, q);
    q = ffma2(ffma2(q, ms, a), y, q);
    float2 d;
    f2_split(q, d.x, d.y);
    top = fmax3(top, fabsf(f.x), fabsf(f.y));
    // (the sum above loses the sign of a zero)
    out[i] = __nv_cvt_float2_to_fp8x2(make_float2(copysignf(d.x, f.x), copysignf(d.y, f.y)), __NV_SATFINITE, __NV_E4M3);
  }
  if (!c.plain || top > 0x1p60f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = to_f32x2<T>(in[i]);
      out[i] = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, c.s), __fdiv_rn(f.y, c.s)), __NV_SATFINITE, __NV_E4M3);
    }
  }
  return make_uint2(out[0] | (out[1] << 16), out[2] | (out[3] << 16));
}

template <class T, bool Fp8, int D>
__global__ void __launch_bounds__(256, 8) append_kernel(const AppendParams p) {
  constexpr int kVec = D / 8;
  const int vec = threadIdx.x % kVec;
  const uint32_t r = blockIdx.x * (256 / kVec) + threadIdx.x / kVec;
  if (r >= p.rows) return;
  const uint32_t t = divide(r, p.by_heads), h = r - t * p.c.kv_heads;
  const int slot = __ldg(p.slots + t);
  const uint4 k = __ldg(reinterpret_cast<const uint4*>(p.k + t * p.k_token + h * p.k_head) + vec);
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p.v + t * p.v_token + h * p.v_head) + vec);
  if (slot < 0) return;
  const uint32_t page = divide(static_cast<uint32_t>(slot), p.by_page);
  if (page >= static_cast<uint32_t>(p.c.num_pages)) {
    if (h == 0 && vec == 0) report_index(p.status, t);
    return;
  }
  const long long at = page * p.c.page_stride + (slot - static_cast<int>(page) * p.c.page_size) * p.c.row_stride + h * p.c.head_stride;
  if constexpr (Fp8) {
    reinterpret_cast<uint2*>(p.c.k + at)[vec] = quantise8<T>(k, read_scale(p.c.k_scale, h));
    reinterpret_cast<uint2*>(p.c.v + at)[vec] = quantise8<T>(v, read_scale(p.c.v_scale, h));
  } else {
    reinterpret_cast<uint4*>(p.c.k + at)[vec] = k;
    reinterpret_cast<uint4*>(p.c.v + at)[vec] = v;
  }
}

// ---------------------------------------------------------------------------- attention of one token
// For each sequence and kv head, G = heads / kv_heads query rows meet the same K and V rows:
//   s = sc K q^T,  p = 2^(s - m),  O^T = V^T p,  l = sum p,  out = O / l
// with the running maximum m (base 2: sc folds in log2 e).  m moves, and O and l are rescaled, only when a
// score exceeds it by more than 8, so weights stay below 2^8 and most tiles need no reduction over keys.
// Every K and V byte is read once and each meets 2 G flops, far below the ridge of the tensor
// cores, so HBM bounds it.  The products run on mma.sync m16n8k16 with keys (then head dims) as the 16
// rows and 8 query heads as the columns (twice 8 for G > 8): 64 keys x 8 queries is far too small a tile for
// a tcgen05 instruction, and CUDA cores alone would need G fused multiply-adds per element, 27 T/s
// at G = 8 and full HBM rate of the 39 T/s that the SMs have.
// Measured (32 heads on 8, d 128): 32 bf16 sequences of up to 8k 88 us, 6.19 TB/s, 0.91 of the copy rate; 64 heads
// over 128 e4m3 sequences of up to 16k 352 us, 0.91; one sequence of 4k 9.0 us against 2.5 for its bytes: length, table
// entry, row, part, counter and the parts again are waited for in turn.
//
// Work: an item is (sequence, kv head, block of 8 or 16 query heads), a tile 64 of its visible keys.
// (Rows of less than 256 bytes that lie side by side, the heads of a token, are read together: an item
// is then `wh` kv heads, 2 or 4, and a tile 64 / wh keys; a warp has one of the heads.  With pieces of 128
// bytes read far apart HBM gave 0.80 of its copy rate, with 64 bytes 0.45.)  All tiles of
// all items form one line, cut into equal ranges, one per CTA, so ragged batches are even and few
// long sequences are spread over all SMs.  Each CTA derives the plan from the lengths by a prefix
// sum.  A CTA's part of an item is a segment; warp w takes keys [16 w, 16 w + 16) of each of its
// tiles, with its own m, l, O and its own ring of cp.async stages: inside a segment no warp waits
// for another, and loads of the next segment are in flight while one ends.  At a segment's end the
// warps of a head merge in shared memory.  A whole item is written at once; a part goes to the workspace (at
// most two per CTA), and the CTA that finishes an item's last part (a counter, left at zero again)
// joins all parts in the order of the line.  Nothing waits, and the order of the sums is fixed by
// the lengths.
//
// e4m3 rows are widened to fp16 (exact) in registers; q is brought to fp16 by a power of two per row
// that puts its largest element in [1, 2) (exact but for elements 2^-14 below it), so both products
// run in fp16.  Weights meet V in the products' 16-bit type, fp16 ones held times 2^7 (kWeightBits, m being 7 less): over
// a 16-bit cache as a sum of two terms, off by half a step of half a step, so that a bf16 output is off by its own
// rounding (relative 1.6e-3; with one term 2.2e-3, and 0.6% less time: the tensor pipe waits for HBM), over an
// e4m3 cache, whose rows have 4 bits, as one fp16 term.  l sums them unrounded in fp32.
namespace paged {
constexpr int kWarps = 4, kThreads = 32 * kWarps, kKeys = 16, kTile = kWarps * kKeys;
template <bool Fp8, int D, int NB>
struct Shape {
  static constexpr int kRows = 8 * NB;                   // query heads of an item
  static constexpr int kRowBytes = D * (Fp8 ? 1 : 2);
  static constexpr int kHalf = kKeys * kRowBytes;        // one warp's K (or V) rows of a stage
  // CTAs per SM, and the stages that fit: 64 KB of ring at two CTAs, 48 KB at three.  A step of
  // 8-bit or short rows brings few bytes for its instructions and wants the warps; the registers
  // allow three CTAs there.
  static constexpr int kCtas = D == 64 || (Fp8 && NB == 1) ? 3 : 2;
  static constexpr int kFit = (kCtas == 3 ? 49152 : 65536) / (kWarps * 2 * kHalf);
  static constexpr int kStages = kFit > 6 ? 6 : kFit;
  static constexpr int kPitch = D + 4;                   // floats of a merged row
  static constexpr int kMergeOff = kStages * kWarps * 2 * kHalf;
  static constexpr int kMlOff = kMergeOff + kWarps * kRows * kPitch * 4;
  static constexpr int kSmem = kMlOff + kWarps * kRows * 2 * 4;
  static constexpr int kPartRows = NB == 1 ? 32 : 16;    // query heads of an item's kv heads, at most
  static constexpr int kPart = kPartRows * (D + 2);      // floats of a segment's part: O, then m and l
};
}  // namespace paged

constexpr int kPagedMaxCtas = 640;
static_assert(kPagedMaxCtas <= kCutCounters, "a counter per CTA");

struct PagedParams {
  CacheArgs c;
  DevStatus* status;
  const uint8_t* q;
  uint8_t* out;
  float* lse;
  long long q_seq, q_head, out_seq, out_head;  // bytes
  const int* table;
  const int* lengths;
  float* part;        // [CTA][2][rows][D + 2]: O, m, l of a segment
  unsigned* counter;  // [CTA]: segments done of the split item that starts in this one
  int max_pages, batch, heads, group, blocks;  // blocks: items per kv head
  int lw;             // log2 of the kv heads of an item
  FastDiv by_page;
  float sl2;          // scale * log2(e)
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

// The length of sequence b, cut to what its table holds (reported once, by CTA 0).
__device__ __forceinline__ int paged_length(const PagedParams& p, int b, bool report) {
  const int n = __ldg(p.lengths + b);
  const long long cap = static_cast<long long>(p.max_pages) * p.c.page_size;
  if (n < 0 || n > cap) {
    if (report) report_index(p.status, static_cast<unsigned long long>(b));
    return n < 0 ? 0 : static_cast<int>(cap);
  }
  return n;
}
__device__ __forceinline__ int paged_tiles(int count, int lw) { return (count + (paged::kTile >> lw) - 1) >> (6 - lw); }

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
// Four e4m3 values as two pairs of fp16, exactly.
__device__ __forceinline__ void widen_e4m3(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi) : "r"(v));
}

// Where a CTA stands on the line of tiles.
struct PagedAt {
  int b;        // sequence
  int sub;      // kv head * blocks + block
  int tile;     // of this item
  int tiles;    // of this item
  Visible vis;  // of this sequence
};

// The transpose of an 8 x 8 matrix of 16-bit elements, a row's pair per thread.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

template <class T, bool Fp8, int D, int NB>
__global__ void __launch_bounds__(paged::kThreads, (paged::Shape<Fp8, D, NB>::kCtas)) paged_kernel(const PagedParams p) {
  using namespace paged;
  using S = Shape<Fp8, D, NB>;
  using M = typename std::conditional<Fp8, __half, T>::type;  // the products' type
  constexpr int kSteps = D / 16, kStages = S::kStages, kRows = S::kRows;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint32_t s_sum[kThreads], s_warp[kWarps];
  __shared__ unsigned s_last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int subs = (p.c.kv_heads >> p.lw) * p.blocks;
  // this warp's kv head of an item's, and its 16 keys of a tile's
  const int hw = warp & ((1 << p.lw) - 1), kb = warp >> p.lw;

  // ---------------------------------------------------------------- plan
  // Thread i sums the tiles of sequences [i chunk, (i + 1) chunk); s_sum holds the sums inside a warp.
  const int chunk = (p.batch + kThreads - 1) / kThreads;
  {
    uint32_t sum = 0;
    for (int i = 0; i < chunk; ++i) {
      const int b = static_cast<int>(threadIdx.x) * chunk + i;
      if (b >= p.batch) break;
      const int count = visible_rows(paged_length(p, b, blockIdx.x == 0), p.window, p.sinks).count;
      sum += paged_tiles(count, p.lw);
      if (count == 0 && b % gridDim.x == blockIdx.x) {  // nothing visible: no item
        for (int h = 0; h < p.heads; ++h) {
          uint4* o = reinterpret_cast<uint4*>(p.out + b * p.out_seq + h * p.out_head);
          for (int v = 0; v < D / 8; ++v) o[v] = make_uint4(0, 0, 0, 0);
          if (p.lse) p.lse[static_cast<long long>(b) * p.heads + h] = -INFINITY;
        }
      }
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, sum, x);
      if (lane >= x) sum += o;
    }
    s_sum[threadIdx.x] = sum;
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
  }
  uint32_t total = 0;  // below 2^31 (the host checks)
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += s_warp[w];
  total *= subs;
  // Tiles of a CTA: an even share, but, by the mean item, no more than 32 parts of an item, and no more than 16 if
  // that takes a CTA up to 2 tiles (4 or 8 of the shorter ones of `wh` heads): a join waits for 16 parts at a
  // time.  One sequence of 2k and 8k rows by the even share alone: bf16 8.3 and 11.3 us, e4m3 15.4 and 21.5; so
  // 7.6, 11.4, 9.8 and 15.5.
  const uint32_t mean = (total + p.batch * subs - 1) / (p.batch * subs);
  const uint32_t per = max(max((total + gridDim.x - 1) / gridDim.x, (mean + 31) / 32), min((mean + 15) / 16, 2u << p.lw));
  // (where an item's parts are limited, `per` is up to grid / 32 even shares: 20 times the line does not fit 32 bits)
  const unsigned long long line = static_cast<unsigned long long>(per) * blockIdx.x;
  if (line >= total) return;
  const uint32_t first = static_cast<uint32_t>(line);
  const int nsteps = static_cast<int>(per < total - first ? per : total - first);

  PagedAt at;
  uint32_t item_begin;  // position on the line of the current item's first tile
  {
    // the warp, then the thread, whose sequences hold `first`
    uint32_t pos = 0;
    int w = 0;
    while (pos + s_warp[w] * subs <= first) pos += s_warp[w++] * subs;
    const int i = __popc(__ballot_sync(0xffffffffu, pos + s_sum[32 * w + lane] * subs <= first));
    if (i > 0) pos += s_sum[32 * w + i - 1] * subs;
    at.b = (32 * w + i) * chunk;
    for (;;) {
      at.vis = visible_rows(paged_length(p, at.b, false), p.window, p.sinks);
      at.tiles = paged_tiles(at.vis.count, p.lw);
      const uint32_t here = static_cast<uint32_t>(at.tiles) * subs;
      if (first < pos + here) break;
      pos += here;
      ++at.b;
    }
    at.sub = static_cast<int>((first - pos) / static_cast<uint32_t>(at.tiles));
    at.tile = static_cast<int>(first - pos) - at.sub * at.tiles;
    item_begin = first - at.tile;
  }
  // One tile on; past the last one of the CTA's range the position is not used.
  auto advance = [&](PagedAt& a) {
    if (++a.tile < a.tiles) return;
    a.tile = 0;
    if (++a.sub < subs) return;
    a.sub = 0;
    while (++a.b < p.batch) {
      a.vis = visible_rows(paged_length(p, a.b, false), p.window, p.sinks);
      a.tiles = paged_tiles(a.vis.count, p.lw);
      if (a.tiles > 0) return;
    }
  };

  // ---------------------------------------------------------------- loads
  // The rows of a step are looked up (page table) one step before they are loaded, the first kStages - 1 steps' all at
  // once; nothing waits for an entry before its loads.  Lanes l and l + 16 hold key l's.  A stage's mask has a
  // bit for each key that is there.
  PagedAt load_at = at;
  int step_loaded = 0;  // steps issued
  struct Place {
    int page;        // as the table has it
    bool wanted;
    long long rest;  // from the page's start to the row's
    int b;
  };
  auto look_up = [&](const PagedAt& a, bool more) {
    Place w;
    w.page = 0;
    w.wanted = false;
    w.rest = 0;
    w.b = a.b;
    const int i = a.tile * (kTile >> p.lw) + kb * kKeys + (lane & 15);
    if (more && i < a.vis.count) {
      const int row = i < a.vis.head ? i : i + a.vis.skip;
      const uint32_t pg = divide(static_cast<uint32_t>(row), p.by_page);
      w.page = __ldg(p.table + static_cast<long long>(a.b) * p.max_pages + pg);
      w.wanted = true;
      w.rest = (row - static_cast<int>(pg) * p.c.page_size) * p.c.row_stride +
               (((NB == 1 ? a.sub : a.sub / p.blocks) << p.lw) + hw) * p.c.head_stride;
    }
    return w;
  };
  const uint32_t ring = smem_u32(smem) + warp * (2 * S::kHalf);
  auto stage_addr = [&](int s) { return ring + s * (kWarps * 2 * S::kHalf); };
  uint32_t masks[kStages];  // one per stage, the same in all lanes
  auto issue = [&](int s, uint32_t& mask, const Place& w) {
    const bool row_ok = w.wanted && w.page >= 0 && w.page < p.c.num_pages;
    if (w.wanted && !row_ok) report_index(p.status, static_cast<unsigned long long>(w.b));
    const long long row_off = row_ok ? w.page * p.c.page_stride + w.rest : 0;
    mask = __ballot_sync(0xffffffffu, row_ok) & 0xffffu;
    if (step_loaded < nsteps) {
      constexpr int kChunks = S::kRowBytes / 16, kPer = 32 / kChunks;  // rows a warp-wide copy covers
      const uint32_t sk = stage_addr(s), sv = sk + S::kHalf;
      const int c = lane % kChunks;
#pragma unroll
      for (int j = 0; j < kKeys / kPer; ++j) {
        const int key = j * kPer + lane / kChunks;
        const long long off = __shfl_sync(0xffffffffu, row_off, key) + c * 16;
        const uint32_t bytes = (mask >> key) & 1u ? 16u : 0u;  // 0: filled with zeros, nothing is read
        uint32_t ck, cv;  // 16-byte chunks are permuted within a row so that no read below conflicts
        if constexpr (!Fp8) {
          ck = cv = key * S::kRowBytes + ((c ^ (key & 7)) << 4);
        } else if constexpr (D == 128) {
          ck = key * 128 + ((c ^ ((key & 1) << 2)) << 4);
          cv = key * 128 + ((c ^ (((key >> 1) & 3) << 1)) << 4);
        } else {
          ck = key * 64 + (c << 4);
          cv = key * 64 + ((c ^ ((key >> 1) & 3)) << 4);
        }
        cp_async16(sk + ck, p.c.k + off, bytes);
        cp_async16(sv + cv, p.c.v + off, bytes);
      }
      ++step_loaded;
    }
    cp_async_commit();
  };

  // ---------------------------------------------------------------- the running state of a segment
  // Columns are query heads: thread (g, t) holds those of 8 b + 2t and 8 b + 2t + 1.
  float o[D / 16][NB][4], m[NB][2], l[NB][2], sc[NB][2];
  uint32_t qf[kSteps][NB][2];
  Place next;
  {
    Place places[kStages - 1];
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
      places[s] = look_up(load_at, s < nsteps);
      if (s + 1 < nsteps) advance(load_at);
    }
    next = look_up(load_at, kStages - 1 < nsteps);
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) issue(s, masks[s], places[s]);
  }

  int step = 0;
  while (step < nsteps) {
    // a segment: this CTA's tiles of one item
    const int seg_tile = at.tile;
    const int seg = nsteps - step < at.tiles - at.tile ? nsteps - step : at.tiles - at.tile;
    const int hk0 = (NB == 1 ? at.sub : at.sub / p.blocks) << p.lw, hk = hk0 + hw;  // (NB 1: one block)
    const int r0 = NB == 1 ? 0 : at.sub % p.blocks * kRows, h0 = hk * p.group + r0;
    const int rows = p.group - r0 < kRows ? p.group - r0 : kRows;
    // q as the products' B: column g of block b (zero past the group)
    const float sl2 = Fp8 && p.c.k_scale ? p.sl2 * __ldg(p.c.k_scale + hk) : p.sl2;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool there = g + 8 * b < rows;
      const uint8_t* qp = p.q + at.b * p.q_seq + (h0 + g + 8 * b) * p.q_head;
      if constexpr (Fp8) {
        float top = 0.f;
        float2 x[kSteps * 2];
#pragma unroll
        for (int h = 0; h < D / 64; ++h)
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint4 v = there ? __ldg(reinterpret_cast<const uint4*>(qp + (64 * h + 16 * t) * 2) + w) : make_uint4(0, 0, 0, 0);
            x[h * 8 + w * 4] = to_f32x2<T>(v.x);
            x[h * 8 + w * 4 + 1] = to_f32x2<T>(v.y);
            x[h * 8 + w * 4 + 2] = to_f32x2<T>(v.z);
            x[h * 8 + w * 4 + 3] = to_f32x2<T>(v.w);
          }
#pragma unroll
        for (int i = 0; i < kSteps * 2; ++i) top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^-e and 2^e for top in [2^e, 2^(e+1)), e kept to where both are normal
        int e = static_cast<int>(__float_as_uint(top) >> 23);
        e = e < 2 ? 2 : e > 252 ? 252 : e;
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        sc[b][0] = sl2 * __shfl_sync(0xffffffffu, up, 8 * t);      // column 2t lives in lanes g = 2t
        sc[b][1] = sl2 * __shfl_sync(0xffffffffu, up, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          qf[i][b][0] = from_f32x2<__half>(x[2 * i].x * down, x[2 * i].y * down);
          qf[i][b][1] = from_f32x2<__half>(x[2 * i + 1].x * down, x[2 * i + 1].y * down);
        }
      } else {
        sc[b][0] = sc[b][1] = sl2;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          qf[i][b][0] = there ? __ldg(reinterpret_cast<const uint32_t*>(qp + (16 * i + 2 * t) * 2)) : 0u;
          qf[i][b][1] = there ? __ldg(reinterpret_cast<const uint32_t*>(qp + (16 * i + 8 + 2 * t) * 2)) : 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m[b][j] = -INFINITY;
        l[b][j] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][b][j] = 0.f;
    }

    for (int i = 0; i < seg; ++i, ++step) {
      // the stage of step - 1 is free (every lane has read it): fill it with step + kStages - 1
      __syncwarp();
      const int s = step % kStages, sn = (step + kStages - 1) % kStages;
      uint32_t mask = 0, fresh;
      issue(sn, fresh, next);
      if (step_loaded < nsteps) advance(load_at);
      next = look_up(load_at, step_loaded < nsteps);
#pragma unroll
      for (int x = 0; x < kStages; ++x) {
        if (x == sn) masks[x] = fresh;
        if (x == s) mask = masks[x];
      }
      cp_async_wait<kStages - 1>();
      __syncwarp();
      const uint32_t sk = stage_addr(s), sv = sk + S::kHalf;
      float x[NB][4];  // scores of keys g (0, 1) and g + 8 (2, 3) at columns 2t, 2t + 1
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[b][j] = 0.f;
      if constexpr (!Fp8) {
        const int key = lane & 15;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          uint32_t a[4];
          ldsm4(a, sk + key * S::kRowBytes + (((2 * k + (lane >> 4)) ^ (key & 7)) << 4));
#pragma unroll
          for (int b = 0; b < NB; ++b) mma16816<M>(x[b], a, qf[k][b][0], qf[k][b][1]);
        }
      } else {
        // 16 bytes per thread and row: k index 2t, 2t + 1, 8 + 2t, 9 + 2t of step (h, k) is head dim
        // 64 h + 16 t + 4 k + 0..3, for q above likewise
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          const int c = 4 * h + t;
          const uint4 u = lds128(sk + g * S::kRowBytes + ((D == 128 ? c ^ ((g & 1) << 2) : c) << 4));
          const uint4 w = lds128(sk + (g + 8) * S::kRowBytes + ((D == 128 ? c ^ ((g & 1) << 2) : c) << 4));
          const uint32_t lo[4] = {u.x, u.y, u.z, u.w}, hi[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t a[4];
            widen_e4m3(lo[k], a[0], a[2]);
            widen_e4m3(hi[k], a[1], a[3]);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816<M>(x[b], a, qf[4 * h + k][b][0], qf[4 * h + k][b][1]);
          }
        }
      }
      bool moved = false;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[b][j] *= sc[b][j & 1];
          if (mask != 0xffffu && !((mask >> (g + 8 * (j >> 1))) & 1u)) x[b][j] = -INFINITY;
          moved |= x[b][j] > m[b][j & 1] + (8.f + kWeightBits<M>);
        }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(x[b][j], x[b][j + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float mn = fmaxf(m[b][j], top - kWeightBits<M>);
            const float keep = mn == -INFINITY ? 0.f : ex2_approx(m[b][j] - mn);
            m[b][j] = mn;
            l[b][j] *= keep;
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
              o[d][b][j] *= keep;
              o[d][b][j + 2] *= keep;
            }
          }
      }
      // the weights as the next product's B: keys by pairs in a column of queries; for a 16-bit cache as a sum of two terms
      constexpr int kTerms = Fp8 ? 1 : 2;
      uint32_t pf[NB][kTerms][2];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          w[j] = ex2_approx(x[b][j] - (m[b][j & 1] == -INFINITY ? 0.f : m[b][j & 1]));
          l[b][j & 1] += w[j];
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t top = from_f32x2<M>(w[2 * e], w[2 * e + 1]);
          pf[b][0][e] = transpose8x8(top);
          if constexpr (!Fp8) {
            const float2 f = to_f32x2<M>(top);
            pf[b][1][e] = transpose8x8(from_f32x2<M>(w[2 * e] - f.x, w[2 * e + 1] - f.y));
          }
        }
      }
      if constexpr (!Fp8) {
        const int key = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          uint32_t a[4];
          ldsm4t(a, sv + key * S::kRowBytes + (((2 * d + ((lane >> 3) & 1)) ^ (key & 7)) << 4));
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = kTerms - 1; e >= 0; --e) mma16816<M>(o[d][b], a, pf[b][e][0], pf[b][e][1]);
        }
      } else {
        // rows 2t, 2t + 1, 8 + 2t, 9 + 2t at head dims [g D/8, (g + 1) D/8), transposed bytewise: rows
        // g and g + 8 of product n are head dims g D/8 + 2n and + 2n + 1
        constexpr int kW = D / 32;  // words
        uint32_t w[4][kW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 2 * t + (k & 1) + 8 * (k >> 1);
          if constexpr (D == 128) {
            const uint4 v = lds128(sv + key * 128 + ((g ^ (((key >> 1) & 3) << 1)) << 4));
            w[k][0] = v.x;
            w[k][1] = v.y;
            w[k][2] = v.z;
            w[k][3] = v.w;
          } else {
            const uint2 v = lds64(sv + key * 64 + (((g >> 1) ^ ((key >> 1) & 3)) << 4) + (g & 1) * 8);
            w[k][0] = v.x;
            w[k][1] = v.y;
          }
        }
#pragma unroll
        for (int i = 0; i < kW; ++i)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            uint32_t a[4];
            widen_e4m3(__byte_perm(w[0][i], w[1][i], z ? 0x7362 : 0x5140), a[0], a[1]);
            widen_e4m3(__byte_perm(w[2][i], w[3][i], z ? 0x7362 : 0x5140), a[2], a[3]);
#pragma unroll
            for (int b = 0; b < NB; ++b) mma16816<M>(o[2 * i + z][b], a, pf[b][0][0], pf[b][0][1]);
          }
      }
    }

    // ---------------------------------------------------------------- the segment's end
    float* merge = reinterpret_cast<float*>(smem + S::kMergeOff);
    float2* ml = reinterpret_cast<float2*>(smem + S::kMlOff);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        l[b][j] += __shfl_xor_sync(0xffffffffu, l[b][j], 4);
        l[b][j] += __shfl_xor_sync(0xffffffffu, l[b][j], 8);
        l[b][j] += __shfl_xor_sync(0xffffffffu, l[b][j], 16);
        const int row = 8 * b + 2 * t + j;
        if (row < rows) {
          float* dst = merge + (warp * kRows + row) * S::kPitch;
          if (g == 0) ml[warp * kRows + row] = make_float2(m[b][j], l[b][j]);
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            if constexpr (!Fp8) {
              dst[16 * n + g] = o[n][b][j];
              dst[16 * n + g + 8] = o[n][b][j + 2];
            } else {
              *reinterpret_cast<float2*>(dst + g * (D / 8) + 2 * n) = make_float2(o[n][b][j], o[n][b][j + 2]);
            }
          }
        }
      }
    __syncthreads();
    const bool whole = seg == at.tiles;
    const int all = rows << p.lw, vecs = all * (D / 4);  // the item's query heads; float4s of them
    float* part = p.part + (static_cast<size_t>(blockIdx.x) * 2 + (seg_tile ? 0 : 1)) * S::kPart;
    auto head_of = [&](int r) { return NB == 1 ? (r >= rows) + (r >= 2 * rows) + (r >= 3 * rows) : 0; };  // of the item's
    auto write_out = [&](int r, int d, float4 v, float mm, float ll) {
      const int head = head_of(r), kv = hk0 + head, h = kv * p.group + r0 + r - head * rows;
      const float vs = Fp8 && p.c.v_scale ? __ldg(p.c.v_scale + kv) : 1.f, inv = ll == 0.f ? 0.f : vs / ll;
      *reinterpret_cast<uint2*>(p.out + at.b * p.out_seq + h * p.out_head + d * 2) =
          make_uint2(from_f32x2<T>(v.x * inv, v.y * inv), from_f32x2<T>(v.z * inv, v.w * inv));
      if (p.lse && d == 0)
        p.lse[static_cast<long long>(at.b) * p.heads + h] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
    };
    auto add = [](float4& acc, float f, const float4& v) {
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    };
    for (int i = threadIdx.x; i < vecs; i += kThreads) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      const int head = head_of(r), row = r - head * rows;
      float mm = -INFINITY, ll = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = head; w < kWarps; w += 1 << p.lw) mm = fmaxf(mm, ml[w * kRows + row].x);
      const float base = mm == -INFINITY ? 0.f : mm;
      for (int w = head; w < kWarps; w += 1 << p.lw) {
        const float2 z = ml[w * kRows + row];
        const float f = ex2_approx(z.x - base);
        ll += f * z.y;
        add(acc, f, *reinterpret_cast<const float4*>(merge + (w * kRows + row) * S::kPitch + d));
      }
      if (whole) {
        write_out(r, d, acc, mm, ll);
      } else {
        *reinterpret_cast<float4*>(part + r * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(part + S::kPartRows * D + 2 * r) = make_float2(mm, ll);
      }
    }
    if (!whole) {
      // the item's parts lie in CTAs [c0, c1]: the first in slot 1 (it starts the item), the others in slot 0
      const int c0 = static_cast<int>(item_begin / per), c1 = static_cast<int>((item_begin + at.tiles - 1) / per);
      __syncthreads();
      if (threadIdx.x == 0) {
        __threadfence();  // the CTA's part, seen by this thread through the barrier, before the count
        unsigned* ctr = p.counter + c0;
        const unsigned done = atomicAdd(ctr, 1u) + 1u;
        s_last = done == static_cast<unsigned>(c1 - c0 + 1);
        if (s_last) *ctr = 0u;
        __threadfence();
      }
      __syncthreads();
      if (s_last) {
        // Part c of c0 + 1.. is `stride` floats after part c - 1; the first one lies apart.
        constexpr int kStride = 2 * S::kPart;
        const float* one = p.part + (static_cast<size_t>(c0) * 2 + 1) * S::kPart;
        const float* rest = p.part + static_cast<size_t>(c0 + 1) * kStride;
        const int parts = c1 - c0 + 1;
        // Few rows leave threads over: `teams` of them share the parts of a row, merged at the end.
        const int teams = vecs < kThreads ? kThreads / vecs : 1;
        for (int i0 = 0; i0 < vecs * teams; i0 += kThreads) {
          const int i = i0 + threadIdx.x, team = teams > 1 ? i / vecs : 0, v = i - team * vecs;
          const bool mine = i < vecs * teams;
          const int row = v / (D / 4), d = (v % (D / 4)) * 4;
          float mm = -INFINITY, ll = 0.f;
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          if (mine) {
            constexpr int kBatch = 16;  // a round trip to L2, often the other die's, each
            for (int c = team; c < parts; c += kBatch * teams) {
              float2 z[kBatch];
              float4 u[kBatch];
#pragma unroll
              for (int x = 0; x < kBatch; ++x) {
                const int k = c + x * teams;
                const float* src = k == 0 ? one : rest + static_cast<size_t>(k - 1) * kStride;
                z[x] = make_float2(-INFINITY, 0.f);
                u[x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (k < parts) {
                  z[x] = __ldcg(reinterpret_cast<const float2*>(src + S::kPartRows * D + 2 * row));
                  u[x] = __ldcg(reinterpret_cast<const float4*>(src + row * D + d));
                }
              }
              float top = mm;
#pragma unroll
              for (int x = 0; x < kBatch; ++x) top = fmaxf(top, z[x].x);
              const float base = top == -INFINITY ? 0.f : top, keep = ex2_approx(mm - base);
              acc = make_float4(acc.x * keep, acc.y * keep, acc.z * keep, acc.w * keep);
              ll *= keep;
              mm = top;
#pragma unroll
              for (int x = 0; x < kBatch; ++x) {
                const float f = ex2_approx(z[x].x - base);
                ll += f * z[x].y;
                add(acc, f, u[x]);
              }
            }
          }
          if (teams > 1) {  // one round (vecs * teams <= kThreads); the merged rows are not needed any more
            float* hold = merge + threadIdx.x * 8;
            *reinterpret_cast<float4*>(hold) = acc;
            *reinterpret_cast<float2*>(hold + 4) = make_float2(mm, ll);
            __syncthreads();
            if (mine && team == 0) {
              for (int x = 1; x < teams; ++x) mm = fmaxf(mm, merge[(threadIdx.x + x * vecs) * 8 + 4]);
              const float base = mm == -INFINITY ? 0.f : mm;
              acc = make_float4(0.f, 0.f, 0.f, 0.f);
              ll = 0.f;
              for (int x = 0; x < teams; ++x) {
                const float* other = merge + (threadIdx.x + x * vecs) * 8;
                const float f = ex2_approx(other[4] - base);
                ll += f * other[5];
                add(acc, f, *reinterpret_cast<const float4*>(other));
              }
            }
          }
          if (mine && team == 0) write_out(row, d, acc, mm, ll);
        }
      }
    }
    __syncthreads();  // merge, ml and s_last are read: the next segment may write them
    at.tile += seg - 1;
    item_begin += at.tiles;
    advance(at);
  }
  cp_async_wait<0>();
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

static FastDiv fast_div(int d) {
  FastDiv f;
  f.shift = 0;
  while ((1ull << f.shift) < static_cast<unsigned long long>(d)) ++f.shift;
  f.mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
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
  if (static_cast<long long>(tokens) * cache->kv_heads >= (1LL << 30)) return TL_ERR_INVALID;
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
  p.rows = static_cast<uint32_t>(tokens) * cache->kv_heads;
  p.by_heads = fast_div(cache->kv_heads);
  p.by_page = fast_div(cache->page_size);
  const long long per_cta = 256 / (cache->d / 8);
  const long long ctas = (p.rows + per_cta - 1) / per_cta;
  return dispatch(dtype, cache->dtype, cache->d, [&](auto t, auto fp8, auto d) {
    append_kernel<decltype(t), decltype(fp8)::value, decltype(d)::value>
        <<<static_cast<unsigned>(ctas), 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
    return launched();
  });
}

// Workspace: the counters, then the parts of split items (two per CTA of the largest grid).
static int paged_rows(int heads, int kv_heads) { return heads / kv_heads > 8 ? 16 : 8; }  // query heads of an item
static int paged_blocks(int heads, int kv_heads) {
  return (heads / kv_heads + paged_rows(heads, kv_heads) - 1) / paged_rows(heads, kv_heads);
}

extern "C" size_t tl_paged_attention_workspace_bytes(int batch, int heads, int kv_heads, int d) {
  if (batch < 0 || batch > 4096 || !heads_ok(heads, kv_heads, d)) return 0;
  const int rows = paged_rows(heads, kv_heads) == 8 ? 32 : 16;  // Shape::kPartRows
  return kCounterBytes + static_cast<size_t>(kPagedMaxCtas) * 2 * rows * (d + 2) * 4;
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
  p.group = heads / cache->kv_heads;
  p.blocks = paged_blocks(heads, cache->kv_heads);
  p.counter = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  p.sl2 = scale * kLog2E;
  p.window = window;
  p.sinks = sinks;
  p.by_page = fast_div(cache->page_size);
  // no more CTAs than tiles there can be
  long long cap = static_cast<long long>(max_pages) * cache->page_size;
  if (window > 0 && cap > static_cast<long long>(window) + sinks) cap = static_cast<long long>(window) + sinks;
  // kv heads read together: side by side, as many as make 256 bytes of a token
  const int es = cache->dtype == TL_E4M3 ? 1 : 2;
  p.lw = 0;
  if (p.group <= 8 && cache->head_stride == cache->d)
    while (p.lw < 2 && ((cache->d * es) << p.lw) < 256 && cache->kv_heads % (2 << p.lw) == 0) ++p.lw;
  const long long most = batch * static_cast<long long>(cache->kv_heads >> p.lw) * p.blocks * (cap / (paged::kTile >> p.lw) + 1);
  if (most >= (1LL << 31)) return TL_ERR_INVALID;
  return dispatch(dtype, cache->dtype, cache->d, [&](auto t, auto fp8, auto d) {
    auto launch = [&](auto nb) {
      using S = paged::Shape<decltype(fp8)::value, decltype(d)::value, decltype(nb)::value>;
      auto kern = paged_kernel<decltype(t), decltype(fp8)::value, decltype(d)::value, decltype(nb)::value>;
      static std::atomic<unsigned long long> ready{0};  // devices on which the kernel may use its shared memory
      if (!smem_ready(ready, ctx->device, reinterpret_cast<const void*>(kern), S::kSmem)) return static_cast<int>(TL_ERR_CUDA);
      long long grid = static_cast<long long>(S::kCtas) * ctx->ctas;
      if (grid > kPagedMaxCtas) grid = kPagedMaxCtas;
      if (grid > most) grid = most;
      kern<<<static_cast<unsigned>(grid), paged::kThreads, S::kSmem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
      return launched();
    };
    return p.group > 8 ? launch(std::integral_constant<int, 2>{}) : launch(std::integral_constant<int, 1>{});
  });
}
