// Attention of a batch over one shared prefix and each sequence's own tail, keys and values
// in a paged cache (sm_100a).
//
// The softmax runs in one pass over the keys: a row keeps a reference maximum m and the sum
// l of 2^(s - m), and its accumulator O = sum 2^(s - m) v is rescaled only when the maximum
// grows by more than 2^8.  Results over disjoint sets of keys are joined by their log-sums:
// LSE = log2(2^a + 2^b), O = 2^(a - LSE) Oa + 2^(b - LSE) Ob.
//
// Work.  An item is a tile of up to 256 query rows of one key head and a run of 128-key
// tiles.  The heads that share a key head are rows too (row = query * G + head in group), so
// a key tile is read once for all of them.
//   * own mode (a sequence has at least 256 rows per key head, or 128 and a short prefix): an
//     item is up to 256 rows of one sequence and walks the prefix, then the sequence's tail;
//   * shared mode (fewer rows): the rows of ALL sequences are tiled together for the
//     prefix, so its keys and values leave HBM once for the batch; each sequence's tail is
//     one more item, and every result is a part that the join kernel joins.
// Items of at most 16 rows (single tokens of a group of heads) are walked by few_rows(), whose
// warps stream keys on their own; the others as described next.
// The unit of scheduling is one key tile.  A CTA (one per SM) first takes whole items, one
// per round while all CTAs have one (own mode, items of one length); what is left over is cut
// into runs of equal length, so no SM waits for a long item: runs wherever they fall inside
// items, or, with items of one length, items dealt out to CTAs of their own.  Item lengths
// follow from the device's tail lengths: every CTA sums the units and finds its run
// itself, so a captured launch follows the lengths of its replay.
//
// A CTA has two softmax warpgroups ("slots"), each with a 128 x 128 f32 score buffer and a
// 128 x D accumulator in TMEM (512 columns at D = 128).  With more than 128 rows the slots
// are the tile's two halves and share each key tile ("dual"); otherwise both hold the same
// rows and take alternate key tiles.  One warp streams K and V tiles with TMA (128-byte
// swizzle; the pages of a tile are copied by different lanes), one issues the MMAs, two
// gather Q.  Step t of the issuer is O += P V of step t - 2, then S of step t into the
// buffer it frees, so one slot's MMAs run under the other's softmax.  P replaces S in TMEM
// as 16-bit pairs and is the A operand of P V.
//
// Rows of V past a length are zeroed in shared memory (a cache slot there may hold NaN, and
// 0 * NaN would reach O); scores past a length are replaced by -inf.
//
// Long items are bound by the tensor pipe and the softmax's issue slots between two MMAs of a
// slot (a tile of 256 rows: 2.1 us, 1.8 with the MMAs alone): 2 x 7,168 tokens over 14,336 keys,
// 24 heads, D = 128: 2.15 ms, 1.18 PF/s.  A prefix shared by single tokens is bound by HBM:
// 32 tokens over 32768 keys and tails up to 1500, 227 MB: 60 us, of which the bytes take 38.
// Half as large score tiles, a second issuer, four softmax warpgroups, five stages, and masked
// tiles on the one-pass path (more registers) were all slower.
#include <math.h>

#include <atomic>

#include <cudaTypedefs.h>

#include "history.cuh"

namespace nabla {

PFN_cuTensorMapEncodeTiled_v12000 get_encode_fn();   // attn_fwd.cu

namespace {

constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;          // warps 4..7 = slot 0, 8..11 = slot 1
constexpr int kMaxCtas = 148;
constexpr int kRowCtas = 2 * kMaxCtas;    // most CTAs of rows_attn_kernel
constexpr int kFewRows = 16;              // most rows of an item with few rows
constexpr int kKeys = 128;                // keys per tile
constexpr int kRows = 256;                // query rows per item
constexpr int kLaunchRegs = 168;
constexpr int kPolyPairs = 2;             // of 8 pairs of weights, by poly_exp2
constexpr int kRegProducer = 72;
constexpr int kRegSoftmax = 216;
static_assert(128 * kRegProducer + 256 * kRegSoftmax <= kThreads * kLaunchRegs,
              "register split exceeds the block's launch budget");

// n / d and n % d for 0 <= n < 2^31 by a multiplication: m = floor(2^32 / d) + 1 overshoots
// 2^32 / d by at most 1, so the product's high word is the quotient or one more.
struct FastDiv {
  uint32_t d, m;
  __host__ void init(uint32_t v) {
    d = v;
    m = v > 1 ? static_cast<uint32_t>((1ull << 32) / v) + 1u : 0u;
  }
  __device__ __forceinline__ int div(int n, int* rem) const {
    if (d == 1) {
      *rem = 0;
      return n;
    }
    int q = static_cast<int>(__umulhi(static_cast<uint32_t>(n), m));
    int r = n - q * static_cast<int>(d);
    if (r < 0) {
      --q;
      r += static_cast<int>(d);
    }
    *rem = r;
    return q;
  }
};

struct AttnParams {
  // queries and outputs
  const void* q;
  long long q_b, q_h, q_s;
  void* o;
  long long o_b, o_h, o_s;
  int o_f32;
  float* lse;
  const void* part_o;
  long long po_b, po_h, po_s;
  int part_f32;
  const float* part_lse;
  int B, Hq, Hkv, G, Sq, R;         // R = Sq * G rows per sequence and key head
  FastDiv div_r, div_g, div_rt, div_kv;
  // keys
  const int32_t* prefix_pages;
  const int32_t* tail_pages;
  const int32_t* tail_len;
  const int32_t* q_len;
  int P, tail_width, page, page_shift, n_pages;
  int causal;
  float scale_log2;
  // schedule
  int shared;                       // shared mode
  int n_rt;                         // row tiles: of a sequence (own), of the batch (shared)
  int n_prefix;                     // prefix items (shared mode)
  int n_items, whole;               // whole: rounds of whole items
  int few0, few1;                   // items [few0, few1) have few rows
  int apart;                        // rows_attn_kernel: CTAs for each item, one tile each (0: runs)
  int uniform;                      // length of every item before few0 if the host knows it
  int tail_rows;                    // rows of a tail part
  // workspace
  uint32_t* cta_status;             // ranks of device status codes
  int32_t* cta_done;                // own mode: the split item that CTA c completes, or -1
  int32_t* first;                   // first / last CTA of an item (relative to whole * grid)
  int32_t* last;
  float* part_l;                    // log2 sums of parts
  float* part_acc;                  // normalised f32 accumulators of parts
  long long tail_base, few_base;    // rows at which the tail parts and the few-row parts start
};

struct Item {
  int b, kvh, row0, rows;           // b = -1: rows of all sequences
  int np, nt;                       // key tiles of the prefix and of the tail
  bool dual;
};

__device__ __forceinline__ int clamp_len(int v, int top) { return v < 0 ? 0 : (v > top ? top : v); }

__device__ __forceinline__ int queries_of(const AttnParams& p, int b) {
  return p.q_len == nullptr ? p.Sq : clamp_len(__ldg(p.q_len + b), p.Sq);
}
__device__ __forceinline__ int tail_of(const AttnParams& p, int b) {
  return p.tail_pages == nullptr ? 0 : clamp_len(__ldg(p.tail_len + b), p.tail_width * p.page);
}
__device__ __forceinline__ int tiles(int keys) { return (keys + kKeys - 1) / kKeys; }

// Keys visible to query s of a sequence with n queries and a tail of L keys (s < n).
__device__ __forceinline__ int visible(const AttnParams& p, int L, int n, int s) {
  if (!p.causal) return p.P + L;
  return max(p.P + L - n + s + 1, 0);
}

__device__ __forceinline__ Item item_of(const AttnParams& p, int i) {
  Item t;
  if (p.shared && i < p.n_prefix) {
    t.b = -1;
    int rt;
    t.kvh = p.div_rt.div(i, &rt);
    t.row0 = rt * kRows;
    t.rows = min(kRows, p.B * p.R - t.row0);
    t.np = tiles(p.P);
    t.nt = 0;
    t.dual = t.rows > 128;
    return t;
  }
  int j = i, rt = 0;
  if (p.shared) {
    j = i - p.n_prefix;
  } else {
    j = p.div_rt.div(i, &rt);
    if (p.causal) rt = p.n_rt - 1 - rt;       // the longest first
  }
  t.b = p.div_kv.div(j, &t.kvh);
  t.row0 = rt * kRows;
  t.rows = min(kRows, p.R - t.row0);
  t.dual = !p.shared || t.rows > 128;
  const int n = queries_of(p, t.b), L = tail_of(p, t.b);
  int rem;
  const int s0 = p.div_g.div(t.row0, &rem), s1 = min(p.div_g.div(t.row0 + t.rows - 1, &rem), n - 1);
  t.np = t.nt = 0;
  if (s0 < n) {
    const int v = visible(p, L, n, s1);
    if (!p.shared) t.np = tiles(min(p.P, v));
    t.nt = tiles(max(v - p.P, 0));
  }
  return t;
}
__device__ __forceinline__ int length_of(const Item& t) { return max(t.np + t.nt, 1); }

// A CTA's share of the work, part by part: key tiles [x0, x1) of an item.  An item counts as
// its tiles and `setup` more (its Q, its pipeline's fill and its epilogue); a run that ends
// inside an item's setup leaves the item to the next CTA.
struct Walk {
  int round, item, x0, setup;
  int left;
  struct Part {
    int i;
    Item t;
    int x0, x1, total;
    int n;        // key tiles of the part (0: an item without keys)
  };
  __device__ __forceinline__ bool next(const AttnParams& p, Part* o) {
    if (round < p.whole) {
      o->i = round * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
      ++round;
      o->t = item_of(p, o->i);
      o->x0 = 0;
      o->x1 = o->total = length_of(o->t);
    } else {
      if (left <= 0) return false;
      o->i = item;
      o->t = item_of(p, item);
      o->total = length_of(o->t);
      const int end = left < o->total + setup - x0 ? x0 + left : o->total + setup;
      o->x0 = max(x0 - setup, 0);
      o->x1 = max(end - setup, 0);
      left -= end - x0;
      ++item;
      x0 = 0;
      if (o->x1 == 0) return false;
    }
    o->n = o->t.np + o->t.nt == 0 ? 0 : o->x1 - o->x0;
    return true;
  }
};

// Items [i0, i1) are cut into runs of equal length, one per CTA of those that share them.  The
// units before a thread's items and in them, by a block-wide scan of the items' lengths.
// `scratch`: kBlock / 32 + 8 words of shared memory; all threads call it.
constexpr int kSetup = 4, kSetupFew = 2;
// Where long items and items of few rows share the CTAs, a tile of the former counts twice: its
// MMAs and exponentials take a CTA longer (factors 1.75, 2, 2.5: 8 sequences of 4 tokens over
// 16384 and 4000 of their own 50, 45, 53 us; 64 tokens over 4096 and 500 46, 43, 40.5; 32
// tokens over 32768 59.8, 59.8, 63.4).
constexpr float kLongWeight = 2.0f;
struct Units {
  int a, b, at, sum, total;
};
template <int kBlock>
__device__ __forceinline__ Units scan_units(const AttnParams& p, int i0, int i1, int setup, int32_t* scratch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int32_t* sums = scratch + 8;
  if (threadIdx.x < 8) scratch[threadIdx.x] = 0;
  const int n = i1 - i0, per = (n + kBlock - 1) / kBlock;
  Units u;
  u.a = min(static_cast<int>(threadIdx.x) * per, n);
  u.b = min(u.a + per, n);
  u.sum = u.total = 0;
  for (int i = u.a; i < u.b; ++i) u.sum += length_of(item_of(p, i0 + i)) + setup;
  int inc = u.sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  u.at = inc - u.sum;
  for (int w = 0; w < kBlock / 32; ++w) {
    if (w < warp) u.at += sums[w];
    u.total += sums[w];
  }
  return u;
}

// Run c of n when `total` units are cut into runs that differ by one unit at most, with at
// least one each (the parts of an item are then those of neighbouring CTAs): start and length.
__device__ __forceinline__ int run_of(int total, int c, int n, int* u0) {
  const int q = total / n, more = total - q * n;
  *u0 = q * c + min(c, more);
  return q + (c < more ? 1 : 0);
}

// The thread whose items hold the run's start finds it (all threads call; `out`: four words of
// the scan's scratch).
__device__ __forceinline__ Walk find_run(const AttnParams& p, const Units& u, int i0, int c, int n, int setup,
                                         int32_t* out) {
  int u0;
  const int mine = run_of(u.total, c, n, &u0);
  if (mine > 0 && u0 >= u.at && u0 < u.at + u.sum) {
    int i = u.a, at = u.at;
    for (; i < u.b; ++i) {
      const int len = length_of(item_of(p, i0 + i)) + setup;
      if (u0 < at + len) break;
      at += len;
    }
    out[0] = i0 + i;
    out[1] = u0 - at;
    out[2] = mine;
  }
  __syncthreads();
  Walk w;
  w.round = 1 << 30;
  w.setup = setup;
  w.item = out[0];
  w.x0 = out[1];
  w.left = out[2];
  return w;
}

// n items of `len` tiles and `ctas` CTAs: every item gets CTAs of its own (each with a tile at
// least), unless runs cut anywhere are shorter even with the change of items in some of them.
__device__ __forceinline__ bool items_apart(int len, int n, int ctas) {
  if (n > ctas || len < (ctas + n - 1) / n) return false;
  return len / (ctas / n) <= static_cast<int>(static_cast<float>(n) * len / ctas) + kSetup;
}

// The same for items i0 .. i0 + n - 1 of one length.
__device__ __forceinline__ Walk find_run_of_equals(int len, int i0, int n, int c, int ctas) {
  Walk w;
  w.round = 1 << 30;
  if (items_apart(len, n, ctas)) {
    const int i = c * n / ctas;
    const int c0 = (i * ctas + n - 1) / n, of = ((i + 1) * ctas + n - 1) / n - c0;
    w.setup = 0;
    w.item = i0 + i;
    w.left = run_of(len, c - c0, of, &w.x0);
  } else {
    int u0;
    w.setup = kSetup;
    w.left = run_of(n * (len + kSetup), c, ctas, &u0);
    w.item = i0 + u0 / (len + kSetup);
    w.x0 = u0 % (len + kSetup);
  }
  return w;
}

struct Bars {
  uint64_t full[8], empty[8];       // K/V stages: landed / read
  uint64_t v_part;                  // a partial V tile landed (its tail rows are then zeroed)
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2];    // S landed / P written
  uint64_t o_done[2], o_free[2];    // the part's last P V landed / the accumulator was read
  uint64_t drain;
  uint32_t tmem;
  int32_t scratch[kThreads / 32 + 8];
  float stat[8][16][2];             // few_rows()
};

template <int D>
struct Cfg {
  static constexpr int kPanels = D / 64;
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr int kOffKv = 2 * kTileBytes;
  static constexpr int kOffOut = kOffKv + kStages * kTileBytes;    // 8 warps x 32 rows x 128 bytes
  static constexpr int kOffBar = kOffOut + 8 * 4096;
  static constexpr int kSmemBytes = kOffBar + 1024 + static_cast<int>(sizeof(Bars));
  static_assert(kSmemBytes <= 232448, "shared memory");
  static __device__ __forceinline__ uint32_t col_s(int s) { return s * 128u; }
  static __device__ __forceinline__ uint32_t col_o(int s) { return 256u + s * 128u; }
};

// A CTA's status word holds the largest rank of what its threads recorded.  (The reduction
// itself: with atomicMax() ptxas loads 64 bytes more of spills in the long items' kernel.)
__device__ __forceinline__ void record_rank(uint32_t* status, uint32_t code) {
  asm volatile("red.global.max.u32 [%0], %1;" ::"l"(__cvta_generic_to_global(status)), "r"(status_rank(code))
               : "memory");
}

// mbar_wait() for short hand-overs: probes without reading the timer, which is looked at (and
// the limit applied) every 256 probes only.
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t parity, uint32_t* status, uint32_t code) {
  uint64_t t0 = 0;
  for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 255u) == 0u) {
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) {
        record_rank(status, code);
        return false;
      }
      // another wait of the CTA gave up (a bad page ends none)
      if (is_timeout_rank(*reinterpret_cast<volatile uint32_t*>(status))) return false;
    }
  }
  return true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Barrier of two warps (ids 1 ..; 0 is __syncthreads).
__device__ __forceinline__ void pair_sync(int id) { asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory"); }

// The next kernel of the call may be set up from here on / waits here for the ones before.
__device__ __forceinline__ void next_kernel_may_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Rows of a part in the workspace (row-major: rows of D floats, and one log-sum each).
__device__ __forceinline__ long long part_row(const AttnParams& p, int i, int cta, bool cont, int half, int row) {
  if (!p.shared) return (static_cast<long long>(2 * cta + (cont ? 0 : 1)) * 2 + half) * 128 + row;
  if (i < p.n_prefix) return (static_cast<long long>(i + cta) * 2 + half) * 128 + row;
  return p.tail_base + static_cast<long long>(i - p.n_prefix + cta) * p.tail_rows + half * 128 + row;
}

// 2^y for a pair of arguments, without the special-function unit: y = n + f with n
// whole and |f| <= 1/2 (adding 1.5 * 2^23 leaves n in the low mantissa bits), 2^f by the
// minimax polynomial of degree 4 (Remez exchange on [-1/2, 1/2]: relative error 2.65e-6 by its
// coefficients, 2.8e-6 with the f32 steps), and n added to the exponent.  Results end at 2^-126
// and 2^127; a NaN gives 2^127, which no row's sum may hold, so its tile is done again without
// the polynomial.
__device__ __forceinline__ float2 poly_exp2(float2 y) {
  const float2 magic = make_float2(12582912.f, 12582912.f), back = make_float2(-12582912.f, -12582912.f);
  y.x = fmaxf(fminf(y.x, 127.f), -126.f);
  y.y = fmaxf(fminf(y.y, 127.f), -126.f);
  const float2 t = __fadd2_rn(y, magic);
  const float2 n = __fadd2_rn(t, back);
  const float2 f = __ffma2_rn(n, make_float2(-1.f, -1.f), y);
  float2 r = __ffma2_rn(make_float2(0.0095701021f, 0.0095701021f), f, make_float2(0.0559178591f, 0.0559178591f));
  r = __ffma2_rn(r, f, make_float2(0.2402474433f, 0.2402474433f));
  r = __ffma2_rn(r, f, make_float2(0.6931217909f, 0.6931217909f));
  r = __ffma2_rn(r, f, make_float2(0.9999992847f, 0.9999992847f));
  return make_float2(__uint_as_float(__float_as_uint(r.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(r.y) + (__float_as_uint(t.y) << 23)));
}

// log2(2^a + 2^b)
__device__ __forceinline__ float join(float a, float b) {
  const float m = fmaxf(a, b);
  if (m == -INFINITY) return a + b;          // -inf, or NaN if one of them is
  return m + log2f(exp2f(a - m) + exp2f(b - m));
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
  if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2*>(&v));
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  return F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
}

// ------------------------------------------------------------------------------------
// Items of at most 16 rows.  Bound by the cache's bytes, and by latency when those are few:
// a 128-row MMA tile would be mostly padding and its pipeline (8 us from launch to result)
// longer than the work.  Four warps take a run of units as above; each streams every fourth
// group of 16 keys through its own ring of 24 KB in shared memory (cp.async; one stage of it is
// being read, so 16 KB are in flight a warp and 128 an SM at D = 128, 20 and 160 at D = 64),
// multiplies with m16n8k16 MMAs (the rows as M, so the scores' registers are the
// second product's A operand), and keeps m, l and O in registers.  The warps' results are
// joined through shared memory at the part's end.
//
// A call with such items only runs rows_attn_kernel (two runs an SM).  One with a prefix tiled
// for many rows as well gives them some of the CTAs of prefix_attn_kernel, each of whose softmax
// warpgroups does the same: one kernel fills the GPU, where two in turn each ramped up and ran
// out (32 tokens over 32768: 60 us, 63.6 in turn; 12 sequences of 5 drafted tokens over 4099:
// 25 us, 28 in turn).  Alone: 4 tokens over 1000 + 150 keys 10.4 us, join included (latency);
// 32 tokens over tails up to 1500, 98 MB: 30 us.
// ------------------------------------------------------------------------------------
constexpr int kFewThreads = 128;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kGroup = 16;                 // keys of a ring stage

template <int D>
struct FewCfg {
  static constexpr int kHalf = kGroup * D * 2;           // bytes of K (or V) of a group
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kWarpBytes = kStages * 2 * kHalf;
  static constexpr int kSmemBytes = kFewThreads / 32 * kWarpBytes;
  static_assert(kFewRows * (D + 4) * 4 <= kWarpBytes, "the joined results reuse the rings");
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// 16 bytes, or zeros
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool read) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}

// A run's parts by four warps (`warp`: 0 .. 3), which share barrier `bar`.
template <int D, bool F16>
__device__ __forceinline__ void few_rows(const AttnParams& p, Walk walk, int run, const uint16_t* __restrict__ k_pool,
                                         const uint16_t* __restrict__ v_pool, unsigned char* smem,
                                         float (*stat)[kFewRows][2], int warp, int bar, uint32_t* status) {
  using C = FewCfg<D>;
  const int lane = threadIdx.x & 31;
  constexpr int kWarps = kFewWarps;
  auto sync = [&] { asm volatile("barrier.cta.sync %0, %1;" ::"r"(bar), "n"(kWarps * 32) : "memory"); };
  const uint32_t ring = smem_u32(smem) + warp * C::kWarpBytes;
  constexpr float kBias = F16 ? 7.0f : 0.0f;       // as in prefix_attn_kernel
  constexpr int kChunks = D / 8;                   // 16-byte pieces of a row
  constexpr int kRowsPerCopy = 32 / kChunks;       // rows that one copy of the warp covers
  const int c_row = lane / kChunks, c_ch = lane % kChunks;
  const int q0 = lane >> 2, kq = (lane & 3) * 2;   // fragment row (and row + 8), column pair
  Walk::Part part;
  while (walk.next(p, &part)) {
    const Item& t = part.t;
    const bool pre = t.b < 0;
    const int L = pre ? p.P : tail_of(p, t.b);
    const int32_t* list = pre ? p.prefix_pages : p.tail_pages + static_cast<long long>(t.b) * p.tail_width;
    const int key0 = part.x0 * kKeys;
    const int key1 = part.n > 0 ? min(part.x1 * kKeys, L) : key0;
    const int groups = (key1 - key0 + kGroup - 1) / kGroup;
    const int mine = groups > warp ? (groups - warp + kWarps - 1) / kWarps : 0;
    // page numbers of the warp's groups, 32 at a time, one per lane
    int ids = 0;
    auto look_up = [&](int j) {                    // groups j .. j + 31 of the warp
      const int key = key0 + (warp + (j + lane) * kWarps) * kGroup;
      ids = -1;
      if (j + lane < mine) {
        const int id = __ldg(list + (key >> p.page_shift));
        if (id < 0 || id >= p.n_pages) record_rank(status, kDevBadPage);
        else ids = id;
      }
    };
    auto load = [&](int j) {                       // group j of the warp into stage j % kStages
      if (j > 0 && (j & 31) == 0) look_up(j);
      const int id = __shfl_sync(0xffffffffu, ids, j & 31);
      if (j < mine) {
        const int key = key0 + (warp + j * kWarps) * kGroup;
        const long long off = static_cast<long long>(max(id, 0)) * p.Hkv * p.page * D +
                              (static_cast<long long>(t.kvh) * p.page + (key & (p.page - 1))) * D;
        const uint32_t st = ring + (j % C::kStages) * 2 * C::kHalf;
#pragma unroll
        for (int i = 0; i < kGroup / kRowsPerCopy; ++i) {
          const int r = i * kRowsPerCopy + c_row;
          const uint32_t dst = st + r * D * 2 + ((c_ch ^ (r & 7)) << 4);
          // a bad page, and slots past the length, are read as zeros
          const bool read = id >= 0 && key + r < key1;
          const long long src = off + (read ? r * D + c_ch * 8 : 0);
          cp_async16_or_zero(dst, k_pool + src, read);
          cp_async16_or_zero(dst + C::kHalf, v_pool + src, read);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    look_up(0);
    // The thread's two rows: keys they see, and their Q in A-operand registers (requested
    // before the first keys, whose traffic would hold it up).
    int lim[2];
    uint32_t qf[D / 16][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = q0 + 8 * e;
      const uint16_t* src = nullptr;
      lim[e] = 0;
      if (r < t.rows) {
        int b = t.b, rr = t.row0 + r, g;
        if (b < 0) b = p.div_r.div(rr, &rr);
        const int s = p.div_g.div(rr, &g);
        const int n = queries_of(p, b);
        if (s < n) {
          const int v = visible(p, tail_of(p, b), n, s);
          lim[e] = pre ? min(v, p.P) : v - p.P;
          src = static_cast<const uint16_t*>(p.q) + b * p.q_b + (t.kvh * p.G + g) * p.q_h + s * p.q_s + kq;
        }
      }
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        qf[c][e] = src != nullptr ? *reinterpret_cast<const uint32_t*>(src + c * 16) : 0u;
        qf[c][2 + e] = src != nullptr ? *reinterpret_cast<const uint32_t*>(src + c * 16 + 8) : 0u;
      }
    }
#pragma unroll
    for (int j = 0; j < C::kStages - 1; ++j) load(j);
    float o[D / 8][4];
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[c][i] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (int j = 0; j < mine; ++j) {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::kStages - 2) : "memory");
      __syncwarp();                                // every lane's copies of group j; stage j - 1 is read
      load(j + C::kStages - 1);
      const uint32_t st = ring + (j % C::kStages) * 2 * C::kHalf;
      const int key = key0 + (warp + j * kWarps) * kGroup;
      float sc[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[n][i] = 0.f;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {         // 32 channels: four 8 x 8 matrices
          const int r = n * 8 + (lane & 7), ch = c * 4 + (lane >> 3);
          uint32_t kf[4];
          ldmatrix_x4(kf, st + r * D * 2 + ((ch ^ (r & 7)) << 4));
          mma_16816<F16>(sc[n], qf[2 * c], kf[0], kf[1]);
          mma_16816<F16>(sc[n], qf[2 * c + 1], kf[2], kf[3]);
        }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = i >> 1;
          if (key + n * 8 + kq + (i & 1) >= lim[e]) sc[n][i] = -INFINITY;
          mx[e] = fmaxf(mx[e], sc[n][i]);
        }
      float factor[2] = {1.f, 1.f};
      bool rescale = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
        const float rm = mx[e] * p.scale_log2 - kBias;
        if (mx[e] != -INFINITY && rm > m[e] + 8.0f) {
          if (m[e] != -INFINITY) {
            factor[e] = fast_exp2(m[e] - rm);
            rescale = true;
          }
          m[e] = rm;
        }
      }
      if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll
        for (int c = 0; c < D / 8; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[c][i] *= factor[i >> 1];
        l[0] *= factor[0];
        l[1] *= factor[1];
      }
      uint32_t pf[4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float neg = m[e] == -INFINITY ? 0.f : -m[e];
          const float x = fast_exp2(fmaf(sc[n][2 * e], p.scale_log2, neg));
          const float y = fast_exp2(fmaf(sc[n][2 * e + 1], p.scale_log2, neg));
          l[e] += x + y;
          pf[2 * n + e] = pack2<F16>(x, y);
        }
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {           // 16 channels: two tiles of 8, two halves of the keys
        const int r = (lane & 7) + (lane & 8), ch = c * 2 + (lane >> 4);
        uint32_t vf[4];
        ldmatrix_x4_trans(vf, st + C::kHalf + r * D * 2 + ((ch ^ (r & 7)) << 4));
        mma_16816<F16>(o[2 * c], pf, vf[0], vf[1]);
        mma_16816<F16>(o[2 * c + 1], pf, vf[2], vf[3]);
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
    }
    // Join the warps (the rings are free now): rows of D values, then m and l.
    sync();
    constexpr int kPitch = D + 4;
    float* acc = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *reinterpret_cast<float2*>(acc + (warp * kFewRows + q0 + 8 * e) * kPitch + c * 8 + kq) =
            make_float2(o[c][2 * e], o[c][2 * e + 1]);
    }
    if ((lane & 3) == 0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        stat[warp][q0 + 8 * e][0] = m[e];
        stat[warp][q0 + 8 * e][1] = l[e];
      }
    }
    sync();
    if (warp == 0 && lane == 0) {
      if (part.x0 == 0) p.first[part.i] = run;
      if (part.x1 == part.total) p.last[part.i] = run;
    }
    constexpr int kPerRow = 32 * kWarps / kFewRows;                 // threads a row
    const int thread = warp * 32 + lane, r = thread / kPerRow;
    if (r < t.rows) {
      int b = t.b, rr = t.row0 + r, g;
      if (b < 0) b = p.div_r.div(rr, &rr);
      const int s = p.div_g.div(rr, &g);
      if (s < queries_of(p, b)) {
        float top = -INFINITY, sum = 0.f, w[kWarps];
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, stat[k][r][0]);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float lk = stat[k][r][1];
          w[k] = lk == 0.f ? 0.f : exp2f(stat[k][r][0] - top);
          sum += lk == 0.f ? 0.f : w[k] * lk;
        }
        const long long row = p.few_base + static_cast<long long>(part.i - p.few0 + run) * kFewRows + r;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (thread % kPerRow == 0) p.part_l[row] = sum == 0.f ? -INFINITY : top + log2f(sum);
#pragma unroll
        for (int i = 0; i < D / (4 * kPerRow); ++i) {
          const int d = 4 * (thread % kPerRow + i * kPerRow);
          float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int k = 0; k < kWarps; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(acc + (k * kFewRows + r) * kPitch + d);
            f.x += w[k] * x.x; f.y += w[k] * x.y; f.z += w[k] * x.z; f.w += w[k] * x.w;
          }
          *reinterpret_cast<float4*>(p.part_acc + row * D + d) = make_float4(f.x * inv, f.y * inv, f.z * inv, f.w * inv);
        }
      }
    }
    sync();
  }
}

template <int D, bool F16>
__global__ void __launch_bounds__(kFewThreads, 2) rows_attn_kernel(const uint16_t* __restrict__ k_pool,
                                                                    const uint16_t* __restrict__ v_pool,
                                                                    const __grid_constant__ AttnParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int32_t scratch[kFewThreads / 32 + 8];
  __shared__ float stat[kFewThreads / 32][kFewRows][2];
  uint32_t* status = p.cta_status + blockIdx.x;
  next_kernel_may_start();
  if (threadIdx.x == 0) *status = 0;
  __syncthreads();         // any warp may record into the word from here on
  Walk walk;
  int run = blockIdx.x;
  if (p.apart > 0) {
    // (every item's first tile, then the second ones: the busy CTAs are on SMs of their own)
    const int n = p.few1 - p.few0, j = static_cast<int>(blockIdx.x) / n, i = static_cast<int>(blockIdx.x) - j * n;
    walk.round = 1 << 30;
    walk.setup = 0;
    walk.item = p.few0 + i;
    walk.x0 = j;
    walk.left = j < p.apart && j < length_of(item_of(p, walk.item)) ? 1 : 0;
    run = i * p.apart + j;
  } else {
    walk = find_run(p, scan_units<kFewThreads>(p, p.few0, p.few1, kSetupFew, scratch), p.few0, blockIdx.x, gridDim.x,
                    kSetupFew, scratch);
  }
  few_rows<D, F16>(p, walk, run, k_pool, v_pool, smem, stat, threadIdx.x >> 5, 0, status);
}

template <int D, bool F16>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_attn_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                       const uint16_t* __restrict__ k_pool, const uint16_t* __restrict__ v_pool,
                       const __grid_constant__ AttnParams p) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* sKV = smem + C::kOffKv;
  Bars& B = *reinterpret_cast<Bars*>(smem + C::kOffBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint32_t* status = p.cta_status + blockIdx.x;

  next_kernel_may_start();
  if (threadIdx.x == 0) {
    *status = 0;
    p.cta_done[blockIdx.x] = -1;
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&B.full[i], 1);
      mbar_init(&B.empty[i], 1);
    }
    mbar_init(&B.v_part, 1);
    mbar_init(&B.q_full, 64);
    mbar_init(&B.q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&B.s_full[s], 1);
      mbar_init(&B.p_full[s], 4);
      mbar_init(&B.o_done[s], 1);
      mbar_init(&B.o_free[s], 4);
    }
    mbar_init(&B.drain, 1);
    fence_mbarrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&B.tmem, 512);
    tmem_relinquish();
  }
  // The CTA's run: among the long items, or, where a call has items of few rows as well, among
  // those; each kind gets a share of the CTAs by its units.
  const int c = blockIdx.x, ctas = gridDim.x;
  const int i0 = p.whole * ctas, n_left = p.few0 - i0;
  Walk walk;
  int few_cta = -1;                 // its index among the CTAs of the items of few rows
  if (p.few1 > p.few0) {
    const Units u = scan_units<kThreads>(p, p.few0, p.few1, kSetupFew, B.scratch);
    const float long_units = kLongWeight * n_left * (p.uniform + kSetup);
    int n_long = min(max(static_cast<int>(ctas * long_units / (long_units + u.total) + 0.5f), 1), ctas - 1);
    if (n_long >= 2 * n_left) {        // the same number of CTAs for each item
      n_long = (n_long + n_left / 2) / n_left * n_left;
      if (n_long >= ctas) n_long -= n_left;
    }
    if (c >= n_long) few_cta = c - n_long;
    if (few_cta >= 0) {                // a run for each of its two softmax warpgroups
      const Walk w0 = find_run(p, u, p.few0, 2 * few_cta, 2 * (ctas - n_long), kSetupFew, B.scratch);
      const Walk w1 = find_run(p, u, p.few0, 2 * few_cta + 1, 2 * (ctas - n_long), kSetupFew, B.scratch + 4);
      walk = warp < kSoftmaxWarp0 + 4 ? w0 : w1;
    } else {
      walk = find_run_of_equals(p.uniform, i0, n_left, c, n_long);
    }
  } else if (p.uniform > 0 && n_left > 0) {
    walk = find_run_of_equals(p.uniform, i0, n_left, c, ctas);
  } else {
    walk = find_run(p, scan_units<kThreads>(p, i0, p.few0, kSetup, B.scratch), i0, c, ctas, kSetup, B.scratch);
  }
  if (p.whole > 0) walk.round = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = B.tmem;
  Walk::Part part;

  if (warp < kSoftmaxWarp0) {
    reg_dealloc<kRegProducer>();
    if (few_cta >= 0) walk.left = 0;       // few_rows() is the other warps' work
    if (warp == 0) {
      // ------------------------------------------------------------------ K and V tiles
      // A tile is K then V, in successive stages of one ring.  Its pages (or, for large
      // pages, its one page) are copied by different lanes, panel by panel.
      if (lane == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
      }
      const int rows_pp = min(p.page, kKeys);            // rows per piece
      const int piece = lane / C::kPanels, panel = lane % C::kPanels;
      uint32_t g = 0;           // stages filled
      // A partial V tile's missing rows are zeroed once it has landed, and only then is it
      // handed on; the next K is requested first.
      uint32_t n_cut = 0;       // partial V tiles
      int cut_stage = -1, cut_valid = 0;
      bool ok = true;
      auto wait_all = [&](uint64_t* bar, uint32_t parity, uint32_t code) -> bool {
        return __all_sync(0xffffffffu, bar_wait(bar, parity, status, code));
      };
      auto finish_cut = [&]() -> bool {
        if (cut_stage < 0) return true;
        if (!wait_all(&B.v_part, n_cut & 1, kDevTimeoutTmaFull)) return false;
        ++n_cut;
        unsigned char* dst = sKV + cut_stage * C::kTileBytes;
        for (int e = cut_valid * 8 + lane; e < kKeys * 8; e += 32)
#pragma unroll
          for (int pn = 0; pn < C::kPanels; ++pn)
            *reinterpret_cast<uint4*>(dst + pn * 16384 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.full[cut_stage]);
        __syncwarp();
        cut_stage = -1;
        return true;
      };
      while (ok && walk.next(p, &part)) {
        const int L = part.t.b >= 0 ? tail_of(p, part.t.b) : 0;
        // Page of this lane's piece of tile x (-1: past the length, nothing to copy).
        auto lookup = [&](int x) -> int {
          const bool pre = x < part.t.np;
          const int base = (pre ? x : x - part.t.np) * kKeys + piece * rows_pp;
          if (piece * rows_pp >= kKeys || base >= (pre ? p.P : L)) return -1;
          const int32_t* list = pre ? p.prefix_pages : p.tail_pages + static_cast<long long>(part.t.b) * p.tail_width;
          const int id = __ldg(list + (base >> p.page_shift));
          if (id < 0 || id >= p.n_pages) {
            record_rank(status, kDevBadPage);
            return p.n_pages;                            // out of bounds: the copy fills zeros
          }
          return id;
        };
        const int xe = part.x0 + part.n;
        int id = part.n > 0 ? lookup(part.x0) : -1;
        for (int x = part.x0; ok && x < xe; ++x) {
          const bool pre = x < part.t.np;
          const int base = (pre ? x : x - part.t.np) * kKeys;
          const int valid = min((pre ? p.P : L) - base, kKeys);
          const uint32_t bytes = static_cast<uint32_t>((valid + rows_pp - 1) / rows_pp * rows_pp) * D * 2;
          const int slot = (base + piece * rows_pp) & (p.page - 1);
          const int cur = id;
          if (x + 1 < xe) id = lookup(x + 1);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const uint32_t st = g % C::kStages;
            if (g >= C::kStages &&
                !wait_all(&B.empty[st], (g / C::kStages - 1) & 1, kDevTimeoutKvEmpty)) {
              ok = false;
              break;
            }
            unsigned char* dst = sKV + st * C::kTileBytes;
            const bool cut = kv == 1 && valid < kKeys;
            uint64_t* bar = cut ? &B.v_part : &B.full[st];
            if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
            __syncwarp();
            if (cur >= 0)
              tma_load_4d(dst + panel * 16384 + piece * rows_pp * 128, kv ? &map_v : &map_k, bar, panel * 64, slot,
                          part.t.kvh, cur);
            __syncwarp();
            if (kv == 0) {
              if (!finish_cut()) {
                ok = false;
                break;
              }
            } else if (cut) {
              cut_stage = static_cast<int>(st);
              cut_valid = valid;
            }
            ++g;
          }
        }
      }
      if (ok) ok = finish_cut();
      if (!ok && cut_stage >= 0) bar_wait(&B.v_part, n_cut & 1, status, kDevTimeoutDrain);
      // Copies still in flight must land before the CTA exits.
      for (uint32_t x = g > C::kStages ? g - C::kStages : 0; x < g; ++x)
        bar_wait(&B.full[x % C::kStages], (x / C::kStages) & 1, status, kDevTimeoutDrain);
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------------ MMA issuer
      // One elected lane.  (elect.sync, not a lane comparison: the compiler then keeps
      // descriptors in uniform registers, and eight MMAs issue back to back.)
      if (elect_one()) {
        constexpr uint32_t idesc_s = F16 ? idesc_f16_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idesc_o = F16 ? idesc_f16_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
        constexpr uint32_t kTile16 = C::kTileBytes >> 4;       // descriptors count 16 bytes
        const uint64_t desc_q = sdesc_sw128(smem_u32(smem), 16, 1024);
        const uint64_t desc_k = sdesc_sw128(smem_u32(sKV), 16, 1024);
        const uint64_t desc_v = sdesc_sw128(smem_u32(sKV), 16384, 1024);
        uint32_t g0 = 0;                // stages of earlier parts
        uint32_t n_q = 0;               // parts with keys
        uint32_t n_p0 = 0, n_p1 = 0;    // P V issued per slot
        uint32_t n_o0 = 0, n_o1 = 0;    // parts finished per slot
        bool ok = true;
        auto full = [&](uint32_t g) -> bool {
          return bar_wait(&B.full[g % C::kStages], (g / C::kStages) & 1, status, kDevTimeoutTmaFull);
        };
        while (ok && walk.next(p, &part)) {
          if (part.n == 0) continue;
          const int dual = part.t.dual ? 1 : 0;
          const int steps = part.n << dual;
          if (!bar_wait(&B.q_full, n_q & 1, status, kDevTimeoutQFull)) break;
          ++n_q;
          for (int t = 0; t < steps + 2; ++t) {
            const uint32_t s = t & 1;
            if (t >= 2) {
              // O += P V of step t - 2 (same slot)
              const uint32_t x = static_cast<uint32_t>(t - 2) >> dual;
              const uint32_t gv = g0 + 2 * x + 1;
              const bool first = dual ? x == 0 : x < 2;
              const uint32_t n_p = s ? n_p1 : n_p0, n_o = s ? n_o1 : n_o0;
              if (!bar_wait(&B.p_full[s], n_p & 1, status, kDevTimeoutPFull) || !full(gv) ||
                  (first && n_o > 0 && !bar_wait(&B.o_free[s], (n_o - 1) & 1, status, kDevTimeoutOBar))) {
                ok = false;
                break;
              }
              if (s) ++n_p1; else ++n_p0;
              tc_fence_after();
              const uint64_t v = desc_v + gv % C::kStages * kTile16;
              const uint32_t o_t = tmem + C::col_o(s), p_t = tmem + C::col_s(s);
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_bf16_ts(o_t, p_t + kk * 8, v + kk * (2048 >> 4), idesc_o, (!first || kk > 0) ? 1u : 0u);
              if (!dual || s == 1) mma_commit(&B.empty[gv % C::kStages]);
              if (t >= steps) {          // the slot's last step
                mma_commit(&B.o_done[s]);
                if (s) ++n_o1; else ++n_o0;
              }
            }
            if (t < steps) {
              const uint32_t gk = g0 + 2 * (static_cast<uint32_t>(t) >> dual);
              if (!full(gk)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint64_t qd = desc_q + (dual ? s : 0u) * kTile16;
              const uint64_t kd = desc_k + gk % C::kStages * kTile16;
              const uint32_t s_t = tmem + C::col_s(s);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                mma_bf16_ss(s_t, qd + off, kd + off, idesc_s, kk > 0 ? 1u : 0u);
              }
              mma_commit(&B.s_full[s]);
              if (!dual || s == 1) mma_commit(&B.empty[gk % C::kStages]);
              if (t == steps - 1) mma_commit(&B.q_empty);
            }
          }
          g0 += 2 * part.n;
        }
        mma_commit(&B.drain);
        bar_wait(&B.drain, 0, status, kDevTimeoutDrain);
      }
      __syncwarp();
    } else {
      // ------------------------------------------------------------------ Q rows
      // Two warps gather the tile's rows into the K-major 128-byte-swizzled layout, each every
      // other 32 rows: a lane finds one row, then the warp copies the rows, D / 8 lanes a row.
      // Rows that do not exist, or lie behind their sequence's queries, are zeros: what a padded
      // batch holds there (NaN, say) would fail the sum check of the whole warp in every tile
      // (5 uneven causal prompts, NaN behind them: 379 us, 266 as zeros, with a cold L2).
      constexpr int kChunks = D / 8;
      constexpr int kStep = 32 / kChunks;
      const int c = lane % kChunks;
      const uint16_t* q = static_cast<const uint16_t*>(p.q);
      uint32_t n_q = 0;
      bool ok = true;
      while (ok && walk.next(p, &part)) {
        if (part.n == 0) continue;
        const int n_rows = part.t.dual ? 256 : 128;
        if (n_q > 0) ok = __all_sync(0xffffffffu, bar_wait(&B.q_empty, (n_q - 1) & 1, status, kDevTimeoutQFull));
        if (!ok) break;
        ++n_q;
        for (int r0 = (warp - 2) * 32; r0 < n_rows; r0 += 64) {
          long long off = -1;
          if (r0 + lane < part.t.rows) {
            int b = part.t.b, rr = part.t.row0 + r0 + lane, g;
            if (b < 0) b = p.div_r.div(rr, &rr);
            const int s = p.div_g.div(rr, &g);
            if (s < queries_of(p, b)) off = b * p.q_b + (part.t.kvh * p.G + g) * p.q_h + s * p.q_s;
          }
#pragma unroll 4
          for (int i = 0; i < 32; i += kStep) {
            const int r = r0 + i + lane / kChunks;
            const long long from = __shfl_sync(0xffffffffu, off, r & 31);
            unsigned char* dst = smem + (r >> 7) * C::kTileBytes + (c >> 3) * 16384 + (r & 127) * 128 +
                                 (((c & 7) ^ (r & 7)) << 4);
            if (from >= 0) cp_async16(smem_u32(dst), q + from + c * 8);
            else *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        fence_proxy_async_smem();
        mbar_arrive(&B.q_full);
      }
      __syncwarp();
    }
  } else {
    reg_alloc<kRegSoftmax>();
    if (few_cta >= 0) {
      const int half = (warp - kSoftmaxWarp0) >> 2;
      few_rows<D, F16>(p, walk, 2 * few_cta + half, k_pool, v_pool, smem + half * FewCfg<D>::kSmemBytes,
                       B.stat + half * kFewWarps, warp & 3, 5 + half, status);
      walk.left = 0;
    }
    // -------------------------------------------------------------------- softmax of a slot
    const int slot = (warp - kSoftmaxWarp0) >> 2;
    const int row = ((warp - kSoftmaxWarp0) & 3) * 32 + lane;       // TMEM lane
    const uint32_t lane_base = static_cast<uint32_t>(((warp - kSoftmaxWarp0) & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + C::col_s(slot);
    const uint32_t o_col = tmem + lane_base + C::col_o(slot);
    const float sl2 = p.scale_log2;
    const float2 sl2v = make_float2(sl2, sl2);
    // The largest weight of a row lies in [2^kBias, 2^(kBias + 8)]: for fp16 as high as its
    // range allows, so that weights down to 2^-31 of it are kept (2^-24 without the bias; a
    // long prefix has enough small ones to matter).
    constexpr float kBias = F16 ? 7.0f : 0.0f;
    uint32_t n_s = 0, n_o = 0;
    const int pair = 1 + (warp & 3);     // barrier of the two slots' warps of the same TMEM lanes
    unsigned char* stage = smem + C::kOffOut + (warp - kSoftmaxWarp0) * 4096;
    // A wait that gives up (never, short of a fault) only ends the waiting: the slots' warps go
    // on through the same barriers, so neither is left at one.
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t code) {
      if (!dead) dead = !__all_sync(0xffffffffu, bar_wait(bar, parity, status, code));
    };
    while (walk.next(p, &part)) {
      // the row: its sequence, query and head, and the keys it sees
      const int r = part.t.dual ? slot * 128 + row : row;
      int b = part.t.b, s = 0, gh = 0;
      bool valid = r < part.t.rows;
      int lim_p = 0x7FFFFFFF, lim_t = 0x7FFFFFFF;     // rows that are never written need no mask
      if (valid) {
        int rr = part.t.row0 + r;
        if (b < 0) b = p.div_r.div(rr, &rr);
        s = p.div_g.div(rr, &gh);
        const int n = queries_of(p, b), L = tail_of(p, b);
        valid = s < n;
        if (valid) {
          const int v = visible(p, L, n, s);
          lim_p = min(v, p.P);
          lim_t = v - p.P;
        }
      }
      const int stride = part.t.dual ? 1 : 2;
      const int x_first = part.x0 + (part.t.dual ? 0 : slot);
      const int xe = part.x0 + part.n;
      float m_ref = -INFINITY, l = 0.f;
      bool any = false, started = false;       // started: an earlier tile set the rows' references
      for (int x = x_first; x < xe; x += stride) {
        any = true;
        wait(&B.s_full[slot], n_s & 1, kDevTimeoutSFull);
        tc_fence_after();
        const int seen = x < part.t.np ? lim_p - x * kKeys : lim_t - (x - part.t.np) * kKeys;
        float2 acc = make_float2(0.f, 0.f);
        bool done = false;
        const bool full = __all_sync(0xffffffffu, seen >= kKeys);
        if (full) {
          if (!started) {
            // A row's first reference: the maximum of its first 32 scores (any near one does).
            uint32_t sv[32];
            tmem_ld32(s_col, sv);
            tmem_wait_ld();
            reg_fence32(sv);
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 32; i += 2) mx = fmax3(mx, __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
            m_ref = mx * sl2 - kBias;
          }
          // Usual tile: weights against the reference of the tiles before, 32 keys at a time as
          // they arrive, some of the exponentials on the FMA pipe.  Their sum decides whether
          // the reference still holds: up to 2^15 no weight is too large (for fp16 either),
          // and NaN or infinity fails; the scores are intact until then.
          const float2 negv = make_float2(-m_ref, -m_ref);
          uint32_t buf[2][32], pk[64];       // scores; weights as 16-bit pairs
          tmem_ld32(s_col, buf[0]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_wait_ld();
            reg_fence32(buf[c & 1]);
            if (c < 3) tmem_ld32(s_col + 32 * (c + 1), buf[(c + 1) & 1]);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 z = make_float2(__uint_as_float(buf[c & 1][2 * e]), __uint_as_float(buf[c & 1][2 * e + 1]));
              const float2 y = __ffma2_rn(z, sl2v, negv);
              const float2 pr = (e & 7) < kPolyPairs ? poly_exp2(y) : make_float2(fast_exp2(y.x), fast_exp2(y.y));
              acc = __fadd2_rn(acc, pr);
              pk[16 * c + e] = pack2<F16>(pr.x, pr.y);
            }
          }
          done = __all_sync(0xffffffffu, acc.x + acc.y <= 32768.f);
          if (!started && !done) m_ref = -INFINITY;
          if (done) {
            l += acc.x + acc.y;
            tmem_st32(s_col, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
            tmem_st32(s_col + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
          }
        }
        if (!done) {
          // First tile, a masked one, or a maximum that has grown: one pass over the scores
          // for the maximum, one for the weights.
          float mx = -INFINITY;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t sv[32];
            tmem_ld32(s_col + 32 * c, sv);
            tmem_wait_ld();
            reg_fence32(sv);
#pragma unroll
            for (int i = 0; i < 32; ++i) mx = fmaxf(mx, 32 * c + i < seen ? __uint_as_float(sv[i]) : -INFINITY);
          }
          float factor = 1.f;
          bool rescale = false;
          const float rm = mx * sl2 - kBias;
          // (after a failed check the reference follows any growth: the next tiles pass)
          if (mx != -INFINITY && rm > m_ref + (full ? 0.f : 8.f)) {
            if (m_ref != -INFINITY) {
              factor = fast_exp2(m_ref - rm);
              rescale = true;
            }
            m_ref = rm;
          }
          const float neg = m_ref == -INFINITY ? 0.f : -m_ref;
          const float2 negv = make_float2(neg, neg);
          acc = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            // the weights of keys 32 c .. go to columns 16 c .., whose scores have been read
            uint32_t sv[32], pk[16];
            tmem_ld32(s_col + 32 * c, sv);
            tmem_wait_ld();
            reg_fence32(sv);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i = 32 * c + 2 * e;
              const float2 z = make_float2(i < seen ? __uint_as_float(sv[2 * e]) : -INFINITY,
                                           i + 1 < seen ? __uint_as_float(sv[2 * e + 1]) : -INFINITY);
              const float2 y = __ffma2_rn(z, sl2v, negv);
              const float2 pr = make_float2(fast_exp2(y.x), fast_exp2(y.y));
              acc = __fadd2_rn(acc, pr);
              pk[e] = pack2<F16>(pr.x, pr.y);
            }
            tmem_st16(s_col + 16 * c, pk);
          }
          // Every earlier P V of the slot was issued before this S, so its completion covers
          // them: the accumulator may be rescaled at once.
          if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
            for (int o0 = 0; o0 < D; o0 += 16) {
              uint32_t ov[16];
              tmem_ld16(o_col + o0, ov);
              tmem_wait_ld();
              reg_fence16(ov);
#pragma unroll
              for (int i = 0; i < 16; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * factor);
              tmem_st16(o_col + o0, ov);
            }
          }
          l = l * factor + (acc.x + acc.y);
        }
        started = true;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[slot]);
        ++n_s;
      }
      // ------------------------------------------------------------------ the part's result
      if (any) {
        wait(&B.o_done[slot], n_o & 1, kDevTimeoutOBar);
        ++n_o;
        tc_fence_after();
      }
      // l is NaN where a visible score is: such a row is NaN, not empty
      float inv = l == 0.f ? 0.f : 1.f / l;
      float sum2 = l == 0.f ? -INFINITY : m_ref + log2f(l);
      // With the same rows in both slots, their results are joined here: each slot's warps
      // read both accumulators and write half of the channels.
      const bool dual = part.t.dual;
      float inv_other = 0.f;
      const bool any_other = !dual && part.n > 1 - slot;
      if (!dual) {
        volatile float* mine = reinterpret_cast<volatile float*>(stage + lane * 8);
        mine[0] = m_ref;
        mine[1] = l;
        tc_fence_before();
        pair_sync(pair);
        tc_fence_after();
        const volatile float* x = reinterpret_cast<const volatile float*>(
            smem + C::kOffOut + ((warp - kSoftmaxWarp0) ^ 4) * 4096 + lane * 8);
        const float m_o = x[0], l_o = x[1];
        pair_sync(pair);                 // the staging areas may be overwritten
        const float top = fmaxf(m_ref, m_o);
        const float wa = l == 0.f ? 0.f : exp2f(m_ref - top), wb = l_o == 0.f ? 0.f : exp2f(m_o - top);
        const float sum = (l == 0.f ? 0.f : wa * l) + (l_o == 0.f ? 0.f : wb * l_o);
        sum2 = sum == 0.f ? -INFINITY : top + log2f(sum);
        inv = sum == 0.f ? 0.f : wa / sum;
        inv_other = sum == 0.f ? 0.f : wb / sum;
      }
      const bool whole = !p.shared && part.x0 == 0 && part.x1 == part.total;
      // where the row goes: bit 0 of `how` = written, bit 1 = merged with the caller's part
      long long at = 0, part_at = 0;
      float pw = 0.f;
      int how = 0;
      if (whole) {
        if (valid) {
          const int h = part.t.kvh * p.G + gh;
          const long long flat = (static_cast<long long>(b) * p.Hq + h) * p.Sq + s;
          how = 1;
          if (p.part_lse != nullptr) {
            const float a = p.part_lse[flat] * 1.4426950408889634f;
            if (a != -INFINITY) {
              const float both = join(sum2, a);
              inv *= sum2 == -INFINITY ? 0.f : exp2f(sum2 - both);
              pw = exp2f(a - both);
              sum2 = both;
              part_at = b * p.po_b + h * p.po_h + s * p.po_s;
              how = 3;
            }
          }
          if (p.lse != nullptr) p.lse[flat] = sum2 * 0.69314718055994531f;
          at = b * p.o_b + h * p.o_h + s * p.o_s;
        }
      } else {
        if (part.x0 == 0 && threadIdx.x == kSoftmaxWarp0 * 32) p.first[part.i - p.whole * gridDim.x] = blockIdx.x;
        if (part.x1 == part.total && threadIdx.x == kSoftmaxWarp0 * 32) {
          p.last[part.i - p.whole * gridDim.x] = blockIdx.x;
          if (!p.shared && part.x0 > 0) p.cta_done[blockIdx.x] = part.i;
        }
        if (valid) {
          const long long w = part_row(p, part.i, blockIdx.x, part.x0 > 0, dual ? slot : 0, row);
          if (dual || slot == 0) p.part_l[w] = sum2;
          how = sum2 != -INFINITY ? 1 : 0;
          at = w * D;
        }
      }
      // 32 channels at a time the warp's 32 rows go through shared memory, so that a store
      // covers whole 128-byte lines (8 lanes a row) instead of 16 bytes of 32 rows: 5 us
      // less per item of 128 f32 rows.
      const bool to_f32 = !whole || p.o_f32;
      // the rows whose channels 4 ch .. 4 ch + 3 (of every 32) this lane stores
      const int ch = lane & 7;
      long long to[8];
      uint32_t hows = 0;
#pragma unroll
      for (int it = 0; it < 8; ++it) {
        const int rr = 4 * it + (lane >> 3);
        to[it] = __shfl_sync(0xffffffffu, at, rr) + 4 * ch;
        hows |= static_cast<uint32_t>(__shfl_sync(0xffffffffu, how, rr)) << (2 * it);
      }
      const bool merge = __any_sync(0xffffffffu, (how & 2) != 0);
      const int d_end = dual ? D : (slot + 1) * (D / 2);
#pragma unroll 1
      for (int d0 = dual ? 0 : slot * (D / 2); d0 < d_end; d0 += 32) {
        float a[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i] = 0.f;
        if (any) {
          uint32_t x[32];
          tmem_ld32(o_col + d0, x);
          tmem_wait_ld();
          reg_fence32(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] = inv == 0.f ? 0.f : __uint_as_float(x[i]) * inv;
        }
        if (any_other) {
          uint32_t x[32];
          tmem_ld32(tmem + lane_base + C::col_o(slot ^ 1) + d0, x);
          tmem_wait_ld();
          reg_fence32(x);
#pragma unroll
          for (int i = 0; i < 32; ++i) a[i] += inv_other == 0.f ? 0.f : __uint_as_float(x[i]) * inv_other;
        }
        if (d0 + 32 == d_end) {
          tc_fence_before();
          if (!dual) pair_sync(pair);      // the other slot's warp has read it too
          __syncwarp();
          if (any && lane == 0) mbar_arrive(&B.o_free[slot]);
        }
        float4 y[8];
        if (merge) {
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const long long from = __shfl_sync(0xffffffffu, part_at, 4 * it + (lane >> 3)) + 4 * ch + d0;
            y[it] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (hows >> (2 * it) & 2) {
              if (p.part_f32) {
                y[it] = *reinterpret_cast<const float4*>(static_cast<const float*>(p.part_o) + from);
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.part_o) + from);
                const float2 y0 = unpack2<F16>(v.x), y1 = unpack2<F16>(v.y);
                y[it] = make_float4(y0.x, y0.y, y1.x, y1.y);
              }
            }
          }
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4*>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
        __syncwarp();
        float4 f[8];
#pragma unroll
        for (int it = 0; it < 8; ++it) {
          const int rr = 4 * it + (lane >> 3);
          f[it] = *reinterpret_cast<const float4*>(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
        }
        if (merge) {
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const float w = __shfl_sync(0xffffffffu, pw, 4 * it + (lane >> 3));
            f[it].x += w * y[it].x; f[it].y += w * y[it].y; f[it].z += w * y[it].z; f[it].w += w * y[it].w;
          }
        }
        if (to_f32) {
          float* base = (whole ? static_cast<float*>(p.o) : p.part_acc) + d0;
#pragma unroll
          for (int it = 0; it < 8; ++it)
            if (hows >> (2 * it) & 1) *reinterpret_cast<float4*>(base + to[it]) = f[it];
        } else {
          uint16_t* base = static_cast<uint16_t*>(p.o) + d0;
#pragma unroll
          for (int it = 0; it < 8; ++it)
            if (hows >> (2 * it) & 1)
              *reinterpret_cast<uint2*>(base + to[it]) =
                  make_uint2(pack2<F16>(f[it].x, f[it].y), pack2<F16>(f[it].z, f[it].w));
        }
      }
    }
  }
  // ---------------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joining the parts of split items, merging the caller's part and writing the rows; the last
// block gathers the CTAs' status words and looks the lengths over (in a block of its own:
// behind its rows' work, or before it, one block would end 3 us after the others).
constexpr int kJoinThreads = 256;

__device__ __forceinline__ void gather_status(const AttnParams& p, uint32_t* status, int ctas) {
  __shared__ uint32_t found;
  if (threadIdx.x == 0) found = 0;
  __syncthreads();
  uint32_t w = 0;
#pragma unroll
  for (int c0 = 0; c0 < kRowCtas; c0 += kJoinThreads) {
    const int c = c0 + static_cast<int>(threadIdx.x);
    const uint32_t x = c < ctas ? p.cta_status[c] : 0u;
    w = max(w, x);
  }
  for (int i = threadIdx.x; i < p.B; i += kJoinThreads) {
    if (p.q_len != nullptr && queries_of(p, i) != p.q_len[i]) w = max(w, status_rank(kDevBadLength));
    if (p.tail_pages != nullptr && tail_of(p, i) != p.tail_len[i]) w = max(w, status_rank(kDevBadLength));
  }
  if (w != 0) atomicMax(&found, w);
  __syncthreads();
  if (threadIdx.x == 0) *status = status_of_rank(found);
}

// Own mode: many rows with few parts each.  A warp joins eight rows at a time, four lanes a
// row for the log-sums (four parts at a time), then all lanes for a row's channels.  Bound by
// the latency of its loads: 12 tiles in 12 parts each 15 us with cold caches (four rows a warp
// and four parts in flight: no faster).
constexpr int kOwnJoinBlocks = kRows / 64;
template <int D, bool F16>
__global__ void __launch_bounds__(kJoinThreads) own_join_kernel(const __grid_constant__ AttnParams p, uint32_t* status,
                                                                int ctas) {
  constexpr int kPer = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_kernel_before();
  if (blockIdx.x == ctas) {
    if (blockIdx.y == 0) gather_status(p, status, ctas);
    return;
  }
  const int i = p.cta_done[blockIdx.x];
  if (i < 0) return;
  const Item t = item_of(p, i);
  const int first = p.first[i - p.whole * ctas], last = p.last[i - p.whole * ctas];
  if (first < 0 || last < first || last >= ctas) return;       // only after a wait gave up
  const int n = last - first + 1, row0 = blockIdx.y * 64 + warp * 8;
  if (row0 >= t.rows) return;
  const int mine = row0 + (lane >> 2);       // the row of this lane's group of four
  int gh = 0;
  const int s = mine < t.rows ? p.div_g.div(t.row0 + mine, &gh) : 0;
  const bool live = mine < t.rows && s < queries_of(p, t.b);
  // workspace row of part j of item row r: part_row(...) + r
  auto base_of = [&](int j) { return part_row(p, i, first + j, j > 0, 0, 0); };
  float m = -INFINITY, sum = 0.f;
  bool nan = false;
  float acc[8][kPer];
#pragma unroll
  for (int r = 0; r < 8; ++r)
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[r][k] = 0.f;
  for (int jc = 0; jc < n; jc += 4) {
    const int j = jc + (lane & 3);
    const float v = live && j < n ? p.part_l[base_of(j) + mine] : -INFINITY;
    nan |= v != v;
    float top = v;
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = fmaxf(top, m);
    const float f = m == -INFINITY ? 0.f : exp2f(m - top);
    float e = v == -INFINITY || top == -INFINITY ? 0.f : exp2f(v - top);
    float es = e;
    es += __shfl_xor_sync(0xffffffffu, es, 1);
    es += __shfl_xor_sync(0xffffffffu, es, 2);
    sum = sum * f + es;
    m = top;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const float fr = __shfl_sync(0xffffffffu, f, 4 * r);
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[r][k] *= fr;
    }
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      if (jc + jj >= n) break;
      const float* src = p.part_acc + (base_of(jc + jj) + row0) * D + lane * kPer;
      float x[8][kPer], w[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        w[r] = __shfl_sync(0xffffffffu, e, 4 * r + jj);
#pragma unroll
        for (int k = 0; k < kPer; k += 2) {
          const float2 y = w[r] != 0.f ? *reinterpret_cast<const float2*>(src + r * D + k) : make_float2(0.f, 0.f);
          x[r][k] = y.x;
          x[r][k + 1] = y.y;
        }
      }
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int k = 0; k < kPer; ++k) acc[r][k] += w[r] * x[r][k];
    }
  }
  nan |= __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), 1) != 0;
  nan |= __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), 2) != 0;
  float lse2 = sum > 0.f ? m + log2f(sum) : -INFINITY;
  float wa = sum > 0.f ? 1.f / sum : 0.f, wb = 0.f;
  if (nan) lse2 = wa = __int_as_float(0x7FC00000);
  const int h = t.kvh * p.G + gh;
  const long long flat = (static_cast<long long>(t.b) * p.Hq + h) * p.Sq + s;
  if (p.part_lse != nullptr && live) {
    const float a = p.part_lse[flat] * 1.4426950408889634f;
    if (a != -INFINITY) {
      const float both = join(lse2, a);
      wa *= lse2 == -INFINITY ? 0.f : exp2f(lse2 - both);
      wb = exp2f(a - both);
      lse2 = both;
    }
  }
  __syncwarp();        // every lane has read part_lse, which may be lse
  if (p.lse != nullptr && live && (lane & 3) == 0) p.lse[flat] = lse2 * 0.69314718055994531f;
  const long long to = t.b * p.o_b + h * p.o_h + s * p.o_s, from = t.b * p.po_b + h * p.po_h + s * p.po_s;
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const bool go = __shfl_sync(0xffffffffu, static_cast<int>(live), 4 * r) != 0;
    const float a = __shfl_sync(0xffffffffu, wa, 4 * r), b = __shfl_sync(0xffffffffu, wb, 4 * r);
    const long long off = __shfl_sync(0xffffffffu, to, 4 * r) + lane * kPer;
    const long long poff = __shfl_sync(0xffffffffu, from, 4 * r) + lane * kPer;
    if (!go) continue;
#pragma unroll
    for (int k = 0; k < kPer; k += 2) {
      float2 y = make_float2(0.f, 0.f);
      if (b != 0.f) {
        if (p.part_f32) y = *reinterpret_cast<const float2*>(static_cast<const float*>(p.part_o) + poff + k);
        else y = unpack2<F16>(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.part_o) + poff + k));
      }
      const float u = acc[r][k] * a + y.x * b, v = acc[r][k + 1] * a + y.y * b;
      if (p.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + off + k) = make_float2(u, v);
      else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + off + k) = pack2<F16>(u, v);
    }
  }
}

// Shared mode.  Bound by latency (about 4 us: first and last CTA, log-sums, accumulators).
// Four warps share a row: a long prefix leaves a row a part in every CTA, and they are read in
// parallel (every fourth part by one warp, always the same ones, so results do not depend on
// timing).  With more rows than are resident that way a warp has a row to itself (a call with
// 52,080 rows in two parts: 74 us, 147 with four warps each).
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kFewJoinRows = kMaxCtas * (2048 / kJoinThreads) * (kJoinWarps / 4);

// Parts of one item that hold a row: the first in workspace row r0, part j > 0 in r1 +
// (j - 1) step.
struct PartList {
  int n;
  long long r0, r1;
  int step;
  __device__ __forceinline__ long long at(int j) const { return j == 0 ? r0 : r1 + static_cast<long long>(j - 1) * step; }
};

__device__ __forceinline__ PartList parts_of(const AttnParams& p, int i, int first, int last, int lrow, int ctas) {
  PartList l;
  l.n = 0;
  const bool few = i >= p.few0 && i < p.few1;
  if (first < 0 || last < first || last >= (few ? kRowCtas : ctas)) return l;       // only after a wait gave up
  if (few) {
    l.n = last - first + 1;
    l.step = kFewRows;
    l.r0 = p.few_base + static_cast<long long>(i - p.few0 + first) * kFewRows + lrow;
    l.r1 = l.r0 + l.step;
    return l;
  }
  const int half = lrow >> 7, row = lrow & 127;
  l.r0 = part_row(p, i, first, false, half, row);
  l.n = last - first + 1;
  l.step = i < p.n_prefix ? kRows : p.tail_rows;
  l.r1 = l.r0 + l.step;
  return l;
}

template <int D, bool F16, int kRowWarps>
__global__ void __launch_bounds__(kJoinThreads) prefix_join_kernel(const __grid_constant__ AttnParams p,
                                                                   uint32_t* status, int ctas) {
  constexpr int kPer = D / 32;
  constexpr int kJoinRows = kJoinWarps / kRowWarps;     // rows at a time
  __shared__ float acc_s[kRowWarps > 1 ? kJoinRows : 1][kRowWarps][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  wait_for_kernel_before();
  if (blockIdx.x == gridDim.x - 1) {
    gather_status(p, status, ctas);
    return;
  }
  const int slot = warp / kRowWarps, sub = warp % kRowWarps;
  const long long n_rows = static_cast<long long>(p.Hkv) * p.B * p.R;
  const long long row0 = static_cast<long long>(blockIdx.x) * kJoinRows, stride = static_cast<long long>(gridDim.x - 1) * kJoinRows;
  for (long long base = row0; base < n_rows; base += stride) {
    const long long id = base + slot;
    bool live = id < n_rows;
    int b = 0, kvh = 0, rr = 0, s = 0, gh = 0;
    PartList l0, l1;
    l0.n = l1.n = 0;
    if (live) {
      const int per = p.B * p.R;
      kvh = n_rows < 1LL << 31 ? static_cast<int>(static_cast<uint32_t>(id) / static_cast<uint32_t>(per))
                               : static_cast<int>(id / per);
      const int rg = static_cast<int>(id - static_cast<long long>(kvh) * per);
      b = p.div_r.div(rg, &rr);
      const int rt = rg / kRows, i0 = kvh * p.n_rt + rt, i1 = p.n_prefix + b * p.Hkv + kvh;
      int f0 = -1, e0 = -1, f1 = -1, e1 = -1;            // (all requested at once)
      if (p.n_prefix > 0) {
        f0 = p.first[i0];
        e0 = p.last[i0];
      }
      if (p.tail_pages != nullptr) {
        f1 = p.first[i1];
        e1 = p.last[i1];
      }
      l0 = parts_of(p, i0, f0, e0, rg - rt * kRows, ctas);
      l1 = parts_of(p, i1, f1, e1, rr, ctas);
      s = p.div_g.div(rr, &gh);
      live = s < queries_of(p, b);
    }
    const int total = l0.n + l1.n;
    float m = -INFINITY, sum = 0.f, acc[kPer];
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    if (live) {
      auto where = [&](int j) { return j < l0.n ? l0.at(j) : l1.at(j - l0.n); };
      for (int j = lane; j < total; j += 32) {
        const float v = p.part_l[where(j)];
        nan |= v != v;
        m = fmaxf(m, v);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      nan = __any_sync(0xffffffffu, nan);
      if (m != -INFINITY) {
        for (int j = lane; j < total; j += 32) sum += exp2f(p.part_l[where(j)] - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
#pragma unroll 4
        for (int j = sub; j < total; j += kRowWarps) {
          const long long w = where(j);
          const float v = p.part_l[w];
          const float e = exp2f(v - m);
          const float* src = p.part_acc + w * D + lane * kPer;
          float x[kPer];
#pragma unroll
          for (int i = 0; i < kPer; i += 2) *reinterpret_cast<float2*>(&x[i]) = *reinterpret_cast<const float2*>(src + i);
          // a part without keys wrote no accumulator
#pragma unroll
          for (int i = 0; i < kPer; ++i) acc[i] += v == -INFINITY ? 0.f : e * x[i];
        }
      }
    }
    if constexpr (kRowWarps > 1) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc_s[slot][sub][lane * kPer + i] = acc[i];
      __syncthreads();
    }
    if (live && sub == 0) {
      if constexpr (kRowWarps > 1) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          float x = 0.f;
#pragma unroll
          for (int k = 0; k < kRowWarps; ++k) x += acc_s[slot][k][lane * kPer + i];
          acc[i] = x;
        }
      }
      float lse2 = m == -INFINITY ? -INFINITY : m + log2f(sum);
      if (nan) lse2 = __int_as_float(0x7FC00000);
      const float inv = nan ? lse2 : (sum > 0.f ? 1.f / sum : 0.f);
#pragma unroll
      for (int i = 0; i < kPer; ++i) acc[i] *= inv;
      const int h = kvh * p.G + gh;
      const long long flat = (static_cast<long long>(b) * p.Hq + h) * p.Sq + s;
      if (p.part_lse != nullptr) {
        const float a = p.part_lse[flat] * 1.4426950408889634f;
        if (a != -INFINITY) {
          const float both = join(lse2, a);
          const float wa = lse2 == -INFINITY ? 0.f : exp2f(lse2 - both), wb = exp2f(a - both);
          const long long off = b * p.po_b + h * p.po_h + s * p.po_s + lane * kPer;
#pragma unroll
          for (int i = 0; i < kPer; i += 2) {
            float2 y;
            if (p.part_f32) y = *reinterpret_cast<const float2*>(static_cast<const float*>(p.part_o) + off + i);
            else y = unpack2<F16>(*reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.part_o) + off + i));
            acc[i] = acc[i] * wa + y.x * wb;
            acc[i + 1] = acc[i + 1] * wa + y.y * wb;
          }
          lse2 = both;
        }
      }
      __syncwarp();        // every lane has read part_lse, which may be lse
      if (p.lse != nullptr && lane == 0) p.lse[flat] = lse2 * 0.69314718055994531f;
      const long long off = b * p.o_b + h * p.o_h + s * p.o_s + lane * kPer;
#pragma unroll
      for (int i = 0; i < kPer; i += 2) {
        if (p.o_f32) *reinterpret_cast<float2*>(static_cast<float*>(p.o) + off + i) = make_float2(acc[i], acc[i + 1]);
        else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.o) + off + i) = pack2<F16>(acc[i], acc[i + 1]);
      }
    }
    if constexpr (kRowWarps > 1) __syncthreads();
  }
}

// 4-D map of a pool [n_pages, H, page, D]: box = 64 channels x min(page, 128) tokens of one
// head of one page, 128-byte swizzle; a page number of n_pages fills zeros.
bool make_map_pool(CUtensorMap* map, const void* base, const nabla_cache& c) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = get_encode_fn();
  if (!enc) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(c.D) * 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.D), static_cast<cuuint64_t>(c.page),
                        static_cast<cuuint64_t>(c.H), static_cast<cuuint64_t>(c.n_pages)};
  cuuint64_t strides[3] = {row, row * c.page, row * c.page * c.H};
  cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(c.page < kKeys ? c.page : kKeys), 1u, 1u};
  cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
  return enc(map, c.dtype == NABLA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Shared mode, for R rows per sequence and key head and a prefix of P tokens.  From 128 rows on a
// sequence fills at least half of an item by itself: over a short prefix the padding of its
// 256 rows costs less than parts and their join.  Own against shared, us: 130 rows over 300,
// 1000, 3000 tokens 38 : 45, 48 : 49, 73 : 66; 168 rows over 1000, 3000, 6000 79 : 109, 140 :
// 154, 221 : 214; 200 rows over 3000, 12000 134 : 155, 367 : 374 (there the rule takes the
// second, 2% slower).  The rule knows neither the number of sequences nor of key heads, on which the cost of
// reading the prefix again and of joining parts depends.
bool is_shared(long long R, long long P) {
  if (R < kRows / 2 || R >= kRows) return R < kRows;
  return (kRows - R) * ((P + kKeys - 1) / kKeys) > 16 * R;
}

// How a call is cut into items, and its workspace.
struct Plan {
  bool shared;
  long long n_rt, n_prefix, n_tail, n_items;
  bool few_prefix, few_tail;             // items of rows_attn_kernel
  long long prefix_rows, tail_rows, few_rows;      // rows of parts
  size_t off_first, off_last, off_l, off_acc, bytes;
};

Plan make_plan(long long B, long long Hkv, long long G, long long Sq, int D, bool shared) {
  Plan a;
  const long long R = G * Sq;
  a.shared = shared;
  if (a.shared) {
    a.n_rt = (B * R + kRows - 1) / kRows;
    a.n_prefix = Hkv * a.n_rt;
    a.n_tail = B * Hkv;
    a.n_items = a.n_prefix + a.n_tail;
    a.few_prefix = B * R <= kFewRows;
    a.few_tail = R <= kFewRows;
    a.prefix_rows = a.few_prefix ? 0 : (a.n_prefix + kMaxCtas) * kRows;
    a.tail_rows = a.few_tail ? 0 : (a.n_tail + kMaxCtas) * (R <= 128 ? R : kRows);
    a.few_rows = a.few_tail ? (a.n_items + kRowCtas) * kFewRows : 0;
  } else {
    a.few_prefix = a.few_tail = false;
    a.few_rows = 0;
    a.n_rt = (R + kRows - 1) / kRows;
    a.n_prefix = a.n_tail = 0;
    a.n_items = B * Hkv * a.n_rt;
    a.prefix_rows = 2LL * kMaxCtas * kRows;
    a.tail_rows = 0;
  }
  a.off_first = kStatusBytes + 2048 + 1024;
  a.off_last = a.off_first + align_up(a.n_items * 4, 256);
  a.off_l = a.off_last + align_up(a.n_items * 4, 256);
  const long long rows = a.prefix_rows + a.tail_rows + a.few_rows;
  a.off_acc = a.off_l + align_up(rows * 4, 256);
  a.bytes = a.off_acc + static_cast<size_t>(rows) * D * 4;
  return a;
}

nabla_status check_sizes(int64_t B, int64_t Hq, int64_t Hkv, int64_t Sq, int D) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Sq < 1 || Hq % Hkv) return NABLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return NABLA_ERR_UNSUPPORTED;
  // rows of a key head, items and their units are counted in 32 bits
  const double rows = static_cast<double>(B) * (Hq / Hkv) * Sq;
  if (rows >= 1073741824.0 || static_cast<double>(B) * Hkv + rows / 256 * Hkv >= 1048576.0 * 8) return NABLA_ERR_UNSUPPORTED;
  return NABLA_OK;
}

// A launch that may be set up while the kernel before it in the stream still runs (that
// kernel lets it, and the kernel itself waits where it must).
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), dim3 grid, int block, size_t smem, cudaStream_t st,
                          Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What a launch needs to know of the current device, looked up once per context (a device
// reset gives a new context id): SMs, and that the kernels' shared memory was allowed.
constexpr int kMaxDevices = 64;

bool current_context_id(unsigned long long* id) {
  static std::atomic<PFN_cuCtxGetCurrent_v4000> get_current{nullptr};
  static std::atomic<PFN_cuCtxGetId_v12000> get_id{nullptr};
  if (get_id.load() == nullptr) {
    void *a = nullptr, *b = nullptr;
    cudaDriverEntryPointQueryResult r1, r2;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &a, cudaEnableDefault, &r1) != cudaSuccess ||
        r1 != cudaDriverEntryPointSuccess ||
        cudaGetDriverEntryPoint("cuCtxGetId", &b, cudaEnableDefault, &r2) != cudaSuccess ||
        r2 != cudaDriverEntryPointSuccess)
      return false;
    get_current.store(reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(a));
    get_id.store(reinterpret_cast<PFN_cuCtxGetId_v12000>(b));
  }
  CUcontext ctx = nullptr;
  *id = 0;
  return get_current.load()(&ctx) == CUDA_SUCCESS && (ctx == nullptr || get_id.load()(ctx, id) == CUDA_SUCCESS);
}

template <int D, bool F16>
nabla_status set_up(int* sms) {
  static std::atomic<unsigned long long> ready[kMaxDevices];   // context id + 1
  static std::atomic<int> n_sms[kMaxDevices];
  int dev = -1;
  unsigned long long id = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || !current_context_id(&id)) return NABLA_ERR_CUDA;
  if (dev >= kMaxDevices) return NABLA_ERR_UNSUPPORTED;
  if (id == 0 || ready[dev].load() != id + 1) {
    int n = 0;
    cudaFuncAttributes fa;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaFuncSetAttribute(prefix_attn_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Cfg<D>::kSmemBytes) != cudaSuccess ||
        cudaFuncSetAttribute(rows_attn_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             FewCfg<D>::kSmemBytes) != cudaSuccess ||
        cudaFuncGetAttributes(&fa, prefix_attn_kernel<D, F16>) != cudaSuccess)
      return NABLA_ERR_CUDA;
    // The register split needs the block to launch with kLaunchRegs a thread.
    if (fa.numRegs != kLaunchRegs) return NABLA_ERR_UNSUPPORTED;
    n_sms[dev].store(n);
    if (id != 0)   // (0: no context was current yet; the next call notes it)
      ready[dev].store(id + 1);
  }
  *sms = n_sms[dev].load();
  return NABLA_OK;
}

template <int D, bool F16>
nabla_status launch(const AttnParams& p, const nabla_cache& cache, uint32_t* status, cudaStream_t st) {
  using C = Cfg<D>;
  int sms = 0;
  nabla_status rc = set_up<D, F16>(&sms);
  if (rc != NABLA_OK) return rc;
  if (sms < 2) return NABLA_ERR_UNSUPPORTED;
  const bool only_few = p.few0 == 0;
  const int sm = sms < kMaxCtas ? sms : kMaxCtas, ctas = only_few ? 2 * sm : sm;
  AttnParams a = p;
  // Whole rounds keep the CTAs on few key heads at a time (the L2 cache holds their keys);
  // items of different lengths would make a round as long as its longest (uneven prompts:
  // 327 us in rounds, 261 in runs at the time).
  a.whole = a.shared || a.uniform == 0 ? 0 : a.n_items / ctas;
  const uint16_t* k = static_cast<const uint16_t*>(cache.k);
  const uint16_t* v = static_cast<const uint16_t*>(cache.v);
  cudaError_t e;
  if (only_few) {
    // A small call has a CTA for every tile that its page tables can hold: no scan of the lengths
    // (32 sequences' tails of up to 100 tokens, 8 heads: 11.4 us after 12.4).
    const int per = ctas / a.n_items, most = a.P > a.tail_width * a.page ? a.P : a.tail_width * a.page;
    a.apart = (most + kKeys - 1) / kKeys <= per ? per : 0;
    rows_attn_kernel<D, F16><<<ctas, kFewThreads, FewCfg<D>::kSmemBytes, st>>>(k, v, a);
  } else {
    CUtensorMap mk, mv;
    if (!make_map_pool(&mk, cache.k, cache) || !make_map_pool(&mv, cache.v, cache)) return NABLA_ERR_CUDA;
    prefix_attn_kernel<D, F16><<<ctas, kThreads, C::kSmemBytes, st>>>(mk, mv, k, v, a);
  }
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  if (a.shared) {
    const long long rows = static_cast<long long>(a.Hkv) * a.B * a.R;
    const bool few = rows <= kFewJoinRows;
    const int at_once = few ? kJoinWarps / 4 : kJoinWarps;
    const long long blocks = (rows + at_once - 1) / at_once;
    e = launch_behind(few ? prefix_join_kernel<D, F16, 4> : prefix_join_kernel<D, F16, 1>,
                      dim3(static_cast<unsigned>(blocks < 1 << 20 ? blocks : 1 << 20) + 1), kJoinThreads, 0, st, a, status,
                      ctas);
  } else {
    e = launch_behind(own_join_kernel<D, F16>, dim3(ctas + 1, kOwnJoinBlocks), kJoinThreads, 0, st, a, status, ctas);
  }
  return cuda_status(e);
}

}  // namespace
}  // namespace nabla

using namespace nabla;

extern "C" size_t nabla_prefix_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t Sq, int32_t D) {
  if (check_sizes(B, Hq, Hkv, Sq, D) != NABLA_OK) return 0;
  const int G = Hq / Hkv;
  const size_t shared = make_plan(B, Hkv, G, Sq, D, true).bytes, own = make_plan(B, Hkv, G, Sq, D, false).bytes;
  const long long R = static_cast<long long>(G) * Sq;
  if (R < kRows / 2 || R >= kRows) return R < kRows ? shared : own;
  return shared > own ? shared : own;            // the prefix's length decides
}

extern "C" nabla_status nabla_prefix_attn(nabla_heads q, int32_t B, int32_t Sq, nabla_cache cache,
                                          const int32_t* prefix_pages, int32_t prefix_len,
                                          const int32_t* tail_pages, int32_t tail_width, const int32_t* tail_len,
                                          const int32_t* q_len, int32_t causal, float scale, nabla_heads part_o,
                                          const float* part_lse, nabla_heads o, float* lse, void* workspace,
                                          size_t workspace_bytes, nabla_stream_t stream) {
  nabla_status rc = check_cache(cache);
  if (rc != NABLA_OK) return rc;
  if ((rc = check_sizes(B, q.H, cache.H, Sq, cache.D)) != NABLA_OK) return rc;
  if ((rc = check_heads(q, B, Sq, false)) != NABLA_OK || (rc = check_heads(o, B, Sq, true)) != NABLA_OK) return rc;
  if (q.dtype != cache.dtype || o.H != q.H) return NABLA_ERR_INVALID_ARG;
  if (o.dtype != q.dtype && o.dtype != NABLA_F32) return NABLA_ERR_INVALID_ARG;
  if (prefix_len < 0 || (prefix_len > 0 && !prefix_pages)) return NABLA_ERR_INVALID_ARG;
  if (tail_pages ? (tail_width < 1 || !tail_len) : (tail_len != nullptr)) return NABLA_ERR_INVALID_ARG;
  const int64_t tail_cap = tail_pages ? static_cast<int64_t>(tail_width) * cache.page : 0;
  if (prefix_len + tail_cap + Sq > 2147483000LL) return NABLA_ERR_UNSUPPORTED;
  if (causal != 0 && causal != 1) return NABLA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !isfinite(scale)) return NABLA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(prefix_pages), static_cast<const void*>(tail_pages),
                        static_cast<const void*>(tail_len), static_cast<const void*>(q_len),
                        static_cast<const void*>(part_lse), static_cast<const void*>(lse)})
    if (reinterpret_cast<uintptr_t>(x) & 3) return NABLA_ERR_INVALID_ARG;
  // units of work are summed in 32 bits
  const double rows = static_cast<double>(B) * (q.H / cache.H) * Sq;
  const double keys = static_cast<double>(prefix_len) + static_cast<double>(tail_cap);
  if ((rows / 256 + B + 1) * cache.H * (keys / 128 + 2 + kSetup) >= 2147483648.0) return NABLA_ERR_UNSUPPORTED;
  const bool part = part_o.ptr != nullptr;
  if (part != (part_lse != nullptr)) return NABLA_ERR_INVALID_ARG;
  if (part) {
    if ((rc = check_heads(part_o, B, Sq, false)) != NABLA_OK) return rc;
    if (part_o.H != q.H || (part_o.dtype != NABLA_F32 && part_o.dtype != q.dtype)) return NABLA_ERR_INVALID_ARG;
  }
  // outputs over inputs: refused, but for the merge in place
  const char* o0 = static_cast<const char*>(o.ptr);
  const char* o1 = heads_end(o, B, Sq, cache.D);
  const int64_t pool = static_cast<int64_t>(cache.n_pages) * cache.H * cache.page * cache.D * 2;
  const int64_t lse_bytes = static_cast<int64_t>(B) * q.H * Sq * 4;
  auto hits = [](const void* a0, const void* a1, const void* b0, const void* b1) { return a0 < b1 && b0 < a1; };
  auto end = [](const void* x, int64_t n) { return static_cast<const void*>(static_cast<const char*>(x) + n); };
  if (heads_overlap(q, o, B, Sq, cache.D) || hits(o0, o1, cache.k, end(cache.k, pool)) ||
      hits(o0, o1, cache.v, end(cache.v, pool)))
    return NABLA_ERR_INVALID_ARG;
  if (part) {
    const bool same = part_o.ptr == o.ptr && part_o.dtype == o.dtype && part_o.stride_b == o.stride_b &&
                      part_o.stride_h == o.stride_h && part_o.stride_s == o.stride_s;
    if (!same && heads_overlap(part_o, o, B, Sq, cache.D)) return NABLA_ERR_INVALID_ARG;
    if (hits(o0, o1, part_lse, end(part_lse, lse_bytes))) return NABLA_ERR_INVALID_ARG;
  }
  if (lse) {
    const void* l1 = end(lse, lse_bytes);
    if (hits(lse, l1, o0, o1) || hits(lse, l1, q.ptr, heads_end(q, B, Sq, cache.D)) ||
        hits(lse, l1, cache.k, end(cache.k, pool)) || hits(lse, l1, cache.v, end(cache.v, pool)))
      return NABLA_ERR_INVALID_ARG;
    if (part && ((part_lse != lse && hits(lse, l1, part_lse, end(part_lse, lse_bytes))) ||
                 hits(lse, l1, part_o.ptr, heads_end(part_o, B, Sq, cache.D))))
      return NABLA_ERR_INVALID_ARG;
  }
  const int G = q.H / cache.H;
  const Plan plan = make_plan(B, cache.H, G, Sq, cache.D, is_shared(static_cast<int64_t>(G) * Sq, prefix_len));
  if (!workspace || workspace_bytes < plan.bytes || (reinterpret_cast<uintptr_t>(workspace) & 255))
    return NABLA_ERR_WORKSPACE;
  AttnParams p = {};
  p.q = q.ptr;
  p.q_b = q.stride_b; p.q_h = q.stride_h; p.q_s = q.stride_s;
  p.o = o.ptr;
  p.o_b = o.stride_b; p.o_h = o.stride_h; p.o_s = o.stride_s;
  p.o_f32 = o.dtype == NABLA_F32;
  p.lse = lse;
  if (part) {
    p.part_o = part_o.ptr;
    p.po_b = part_o.stride_b; p.po_h = part_o.stride_h; p.po_s = part_o.stride_s;
    p.part_f32 = part_o.dtype == NABLA_F32;
    p.part_lse = part_lse;
  }
  p.B = B; p.Hq = q.H; p.Hkv = cache.H; p.G = G; p.Sq = Sq; p.R = Sq * G;
  p.div_r.init(p.R);
  p.div_g.init(G);
  p.prefix_pages = prefix_pages;
  p.tail_pages = tail_pages;
  p.tail_len = tail_len;
  p.q_len = q_len;
  p.P = prefix_len;
  p.tail_width = tail_pages ? tail_width : 0;
  p.page = cache.page;
  while ((1 << p.page_shift) < cache.page) ++p.page_shift;
  p.n_pages = cache.n_pages;
  p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.shared = plan.shared;
  p.n_rt = static_cast<int>(plan.n_rt);
  p.div_rt.init(p.n_rt);
  p.div_kv.init(cache.H);
  // without tails (or without a prefix) shared mode has only the other kind of items
  p.n_prefix = plan.shared && (prefix_len > 0 || !tail_pages) ? static_cast<int>(plan.n_prefix) : 0;
  p.n_items = plan.shared ? p.n_prefix + (tail_pages ? static_cast<int>(plan.n_tail) : 0) : static_cast<int>(plan.n_items);
  p.tail_rows = p.R <= 128 ? p.R : kRows;
  p.few0 = !plan.few_tail ? p.n_items : (plan.few_prefix ? 0 : p.n_prefix);
  p.few1 = p.n_items;
  p.uniform = plan.shared ? (p.few0 <= p.n_prefix ? (prefix_len + kKeys - 1) / kKeys : 0)
                          : (!tail_pages && !q_len && !causal ? (prefix_len + kKeys - 1) / kKeys : 0);
  char* ws = static_cast<char*>(workspace);
  p.cta_status = reinterpret_cast<uint32_t*>(ws + kStatusBytes);
  p.cta_done = reinterpret_cast<int32_t*>(ws + kStatusBytes + 2048);
  p.first = reinterpret_cast<int32_t*>(ws + plan.off_first);
  p.last = reinterpret_cast<int32_t*>(ws + plan.off_last);
  p.part_l = reinterpret_cast<float*>(ws + plan.off_l);
  p.part_acc = reinterpret_cast<float*>(ws + plan.off_acc);
  p.tail_base = plan.prefix_rows;
  p.few_base = plan.prefix_rows + plan.tail_rows;
  uint32_t* status = static_cast<uint32_t*>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cache.D == 64)
    return cache.dtype == NABLA_F16 ? launch<64, true>(p, cache, status, st) : launch<64, false>(p, cache, status, st);
  return cache.dtype == NABLA_F16 ? launch<128, true>(p, cache, status, st) : launch<128, false>(p, cache, status, st);
}
