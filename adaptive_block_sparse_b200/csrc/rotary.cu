// Rotary positions for Q and K, and the append of K (rotated on the way) and V to a paged
// cache.
//
// A pair (x0, x1) of channels is turned by the angle a = position * inv_freq[pair] and
// scaled by a magnitude m:
//   y0 = m (x0 cos a - x1 sin a),  y1 = m (x1 cos a + x0 sin a);
// the adjoint (the gradient's direction) turns by -a.  Angles are formed in fp64 as turns,
// t = position * inv_freq / (2 pi), and reduced to t - rint(t) before the f32 sine and
// cosine, so a position of 10^6 is as exact as one of 10 (in f32 its angle would be off by
// up to 0.03 rad).
//
// Bound by HBM: every element is read once and written once (720p-like Q and K, 3.3 GB: 501 us,
// 6.6 TB/s; 7,168 tokens appended, 176 MB: 37 us).  A thread owns 8 pairs of one
// token (two 16-byte vectors of a 16-bit tensor) and walks a group of heads with them, so
// the fp64 angles and the sines are computed once for the whole group; it keeps the loads
// of two heads in flight.  The angles come first, so calls of one or two waves (the appended
// tokens above) show their latency; in larger ones other warps hide it.  Neighbouring threads
// own a token's neighbouring pairs and then the neighbouring tokens, so a head's accesses are
// contiguous runs.
//
// Half-split pairs (i, i + dim / 2) with dim / 2 no multiple of 8 have no common 16-byte
// alignment of their parts: rotary_staged_kernel turns them in shared memory (97 MB of f32
// rows with 38 pairs: 26 us; 38.5 us with partners read one by one from L1; vectors that
// divide dim / 2 ran at 1 TB/s where it is odd).
#include <math.h>

#include <type_traits>

#include "history.cuh"

namespace nabla {
namespace {

constexpr int kThreads = 128;
enum { kInterleaved = 0, kHalf = 1 };   // pairing

// One tensor to move: source and destination views (strides in elements).
struct Stream {
  const void* src;
  void* dst;
  long long s_b, s_h, s_s, d_b, d_h, d_s;
  int end;                    // one past its last head in the call's list of heads
};

struct RotaryParams {
  Stream st[3];               // Q, K, V; V is copied unrotated (cache append only)
  int heads;                  // all heads of the call
  int group;                  // heads per thread
  int tokens, S;              // B * S, S
  int Hg, W;                  // grid of a frame (3 axes or a reordered layout)
  int T0, H0, W0;             // position of the first token
  int axes;
  int src_blocks, dst_blocks; // token order of sources / destinations is the block order
  int half;                   // rotated pairs
  int ax1, ax2;               // first pair of the second and third axis
  float sign, magnitude;
  const double* inv_freq;
  const int32_t* positions;   // [B, S, axes] or NULL
  // cache append
  const int32_t* table;       // [B, table_w]; NULL: plain rotary
  const int32_t* start;
  const int32_t* counts;
  long long pos0;
  int table_w, n_pages, page, page_shift;
  long long page_stride;      // elements between pages
  uint32_t* status;
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

// V consecutive elements, whole 16-byte words.
template <typename T, int V>
struct Vec {
  using W = uint4;
  static constexpr int kWords = V * sizeof(T) / 16;
  union {
    W w[kWords];
    T e[V];
  };
  __device__ __forceinline__ Vec() {}
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __ldg(reinterpret_cast<const W*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) reinterpret_cast<W*>(p)[i] = w[i];
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_float(e[i]);
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < V; i += 2)
        reinterpret_cast<uint32_t*>(w)[i / 2] =
            std::is_same<T, __half>::value ? pack_f16x2(f[i], f[i + 1]) : pack_bf16x2(f[i], f[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = f[i];
    }
  }
};

// The same elements in another type (a plain copy when the types agree).
template <typename TD, typename TS, int V>
__device__ __forceinline__ Vec<TD, V> convert(const Vec<TS, V>& x) {
  if constexpr (std::is_same<TD, TS>::value) {
    return x;
  } else {
    float f[V];
    x.get(f);
    Vec<TD, V> y;
    y.set(f);
    return y;
  }
}

// What a thread knows about its token.
struct Token {
  long long pos[3];
  long long src[3], dst[3];   // element offsets of the streams at head 0
  bool stored;                // K and V have a destination (always, without a cache)
};

// Index in the block order (8 x 8 patches of a frame, row-major) of natural token n.
__device__ __forceinline__ int block_index(int n, int Hg, int W) {
  const int t = n / (Hg * W), r = n - t * Hg * W;
  const int h = r / W, w = r - h * W;
  return t * Hg * W + ((h >> 3) * (W >> 3) + (w >> 3)) * 64 + (h & 7) * 8 + (w & 7);
}

__device__ __forceinline__ Token locate(const RotaryParams& p, int token) {
  Token k;
  const int b = token / p.S, n = token - b * p.S;
  k.stored = true;
  long long page_off = 0;
  if (p.table != nullptr) {
    const long long at = static_cast<long long>(p.start[b]) + n;
    if (p.counts != nullptr) {
      const int c = p.counts[b];
      k.stored = n < c;
      if (n == 0 && (c < 0 || c > p.S)) record_status(p.status, kDevBadLength);
    }
    if (k.stored) {
      const long long pg = at >> p.page_shift;
      int id = -1;
      if (at < 0 || pg >= p.table_w) {
        record_status(p.status, kDevBadLength);
        k.stored = false;
      } else {
        id = p.table[static_cast<long long>(b) * p.table_w + pg];
        if (id < 0 || id >= p.n_pages) {
          record_status(p.status, kDevBadPage);
          k.stored = false;
        }
      }
      page_off = k.stored ? id * p.page_stride + (at & (p.page - 1)) * p.st[1].d_s : 0;
    }
    const long long q = p.pos0 + at;
    k.pos[0] = q;
    if (p.axes == 3 && p.positions == nullptr) {
      const long long hw = static_cast<long long>(p.Hg) * p.W;
      const long long t = q / hw, r = q - t * hw;
      k.pos[0] = t; k.pos[1] = r / p.W; k.pos[2] = r % p.W;
    }
  } else if (p.axes == 3) {
    const int t = n / (p.Hg * p.W), r = n - t * p.Hg * p.W;
    k.pos[0] = static_cast<long long>(t) + p.T0;
    k.pos[1] = static_cast<long long>(r / p.W) + p.H0;
    k.pos[2] = static_cast<long long>(r % p.W) + p.W0;
  } else {
    k.pos[0] = static_cast<long long>(n) + p.T0;
  }
  if (p.positions != nullptr) {
    const int32_t* e = p.positions + static_cast<long long>(token) * p.axes;
    k.pos[0] = e[0];
    if (p.axes == 3) { k.pos[1] = e[1]; k.pos[2] = e[2]; }
  }
  const int blk = (p.src_blocks | p.dst_blocks) ? block_index(n, p.Hg, p.W) : n;
  const int ns = p.src_blocks ? blk : n, nd = p.dst_blocks ? blk : n;
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    k.src[i] = b * p.st[i].s_b + ns * p.st[i].s_s;
    k.dst[i] = (p.table != nullptr && i > 0) ? page_off : b * p.st[i].d_b + nd * p.st[i].d_s;
  }
  return k;
}

// cos and sin (times the magnitude) of pair i at the token's position.
__device__ __forceinline__ void angle(const RotaryParams& p, const Token& k, int i, float* c, float* s) {
  long long pos = k.pos[0];
  if (p.axes == 3) pos = i < p.ax1 ? k.pos[0] : (i < p.ax2 ? k.pos[1] : k.pos[2]);
  const double turns = static_cast<double>(pos) * __ldg(p.inv_freq + i) * 0.15915494309189533577;   // 1 / (2 pi)
  float sn, cs;
  sincospif(static_cast<float>(2.0 * (turns - rint(turns))), &sn, &cs);
  *c = cs * p.magnitude;
  *s = sn * p.magnitude * p.sign;
}

template <int PAIRING, int D, typename TS, typename TD>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int V = 8;
  constexpr int kLanes = D / (2 * V);                      // threads per token
  constexpr int kUnroll = 2;                               // heads in flight
  const long long gid = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const long long token = gid / kLanes;
  if (token >= p.tokens) return;
  const int u = static_cast<int>(gid & (kLanes - 1));
  const Token k = locate(p, static_cast<int>(token));
  const int h_begin = blockIdx.y * p.group;
  const int h_end = min(h_begin + p.group, p.heads);

  // Element offsets of the thread's two vectors, and its pairs' factors.  A pair that is
  // not rotated is copied, not multiplied by one: its values may be infinite.
  int e0, e1;
  bool turn[V];
  float c[V], s[V];
  if constexpr (PAIRING == kHalf) {
    const bool rot = V * u < p.half;
    e0 = rot ? V * u : 2 * p.half + (V * u - p.half) * 2;
    e1 = rot ? p.half + V * u : e0 + V;
  } else {
    e0 = 2 * V * u;
    e1 = e0 + V;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    turn[j] = V * u + j < p.half;
    c[j] = 1.f;
    s[j] = 0.f;
    if (turn[j]) angle(p, k, V * u + j, &c[j], &s[j]);
  }

  // A head of the list -> its stream, whether it is rotated and whether it is written.
  auto stream_of = [&](int h) { return h < p.st[0].end ? 0 : (h < p.st[1].end ? 1 : 2); };
  auto source = [&](int i, int hh) {
    return static_cast<const TS*>(p.st[i].src) + (i == 0 ? k.src[0] : (i == 1 ? k.src[1] : k.src[2])) + hh * p.st[i].s_h;
  };
  auto target = [&](int i, int hh) {
    return static_cast<TD*>(p.st[i].dst) + (i == 0 ? k.dst[0] : (i == 1 ? k.dst[1] : k.dst[2])) + hh * p.st[i].d_h;
  };
  for (int h0 = h_begin; h0 < h_end; h0 += kUnroll) {
    const TS* src[kUnroll];
    TD* dst[kUnroll];
    bool go[kUnroll], rot[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      const int h = h0 + x;
      const int i = stream_of(h);
      const int hh = h - (i == 0 ? 0 : p.st[i - 1].end);
      go[x] = h < h_end && (i == 0 || k.stored);
      rot[x] = i < 2;
      src[x] = source(i, hh);
      dst[x] = target(i, hh);
    }
    Vec<TS, V> a[kUnroll], b[kUnroll];
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      if (go[x]) {
        a[x].load(src[x] + e0);
        b[x].load(src[x] + e1);
      }
    }
#pragma unroll
    for (int x = 0; x < kUnroll; ++x) {
      if (!go[x]) continue;
      Vec<TD, V> ya, yb;
      if (rot[x]) {
        float f[V], g[V];
        a[x].get(f);
        b[x].get(g);
        if constexpr (PAIRING == kHalf) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            if (turn[j]) {
              const float x0 = f[j], x1 = g[j];
              f[j] = x0 * c[j] - x1 * s[j];
              g[j] = x1 * c[j] + x0 * s[j];
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            if (turn[j]) {
              const float x0 = f[2 * j], x1 = f[2 * j + 1];
              f[2 * j] = x0 * c[j] - x1 * s[j];
              f[2 * j + 1] = x1 * c[j] + x0 * s[j];
            }
            if (turn[V / 2 + j]) {
              const float x0 = g[2 * j], x1 = g[2 * j + 1];
              g[2 * j] = x0 * c[V / 2 + j] - x1 * s[V / 2 + j];
              g[2 * j + 1] = x1 * c[V / 2 + j] + x0 * s[V / 2 + j];
            }
          }
        }
        ya.set(f);
        yb.set(g);
      } else {
        ya = convert<TD>(a[x]);
        yb = convert<TD>(b[x]);
      }
      ya.store(dst[x] + e0);
      yb.store(dst[x] + e1);
    }
  }
}

// Any dim / 2.  A warp owns a token and a run of heads, eight at a time: rows come in
// 16-byte vectors, are widened into shared memory, turned there (a lane has pairs lane and
// lane + 32) and leave in 16-byte vectors.  (Eight tokens of one head at a time, with their
// angles in shared memory, was slower: 186 against 145 us on 588 MB.)
constexpr int kStagedRows = 8, kStagedWarps = 8;
template <int D, typename TS, typename TD>
__global__ void __launch_bounds__(kThreads) rotary_staged_kernel(const __grid_constant__ RotaryParams p) {
  constexpr int kVs = 16 / sizeof(TS), kVd = 16 / sizeof(TD);            // elements of a vector
  constexpr int kLoads = kStagedRows * D / (kVs * 32), kStores = kStagedRows * D / (kVd * 32);
  constexpr int kPairs = D / 64;                                         // pairs of a lane
  __shared__ __align__(16) float rows[kThreads / 32][kStagedRows][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long token = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  if (token >= p.tokens) return;                                         // whole warps
  const Token k = locate(p, static_cast<int>(token));
  const int h_begin = blockIdx.y * p.group;
  const int h_end = min(h_begin + p.group, p.heads);
  float c[kPairs], s[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j)
    if (lane + 32 * j < p.half) angle(p, k, lane + 32 * j, &c[j], &s[j]);
  float(*row)[D] = rows[warp];
  auto written = [&](int h) { return h < h_end && (h < p.st[0].end || k.stored); };
  for (int h0 = h_begin; h0 < h_end; h0 += kStagedRows) {
    Vec<TS, kVs> a[kLoads];
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int f = n * 32 + lane, h = h0 + f / (D / kVs), e = f % (D / kVs) * kVs;
      const int i = h < p.st[0].end ? 0 : (h < p.st[1].end ? 1 : 2);
      if (written(h))
        a[n].load(static_cast<const TS*>(p.st[i].src) + (i == 0 ? k.src[0] : (i == 1 ? k.src[1] : k.src[2])) +
                  (h - (i == 0 ? 0 : p.st[i - 1].end)) * p.st[i].s_h + e);
    }
#pragma unroll
    for (int n = 0; n < kLoads; ++n) {
      const int f = n * 32 + lane, r = f / (D / kVs), e = f % (D / kVs) * kVs;
      if (!written(h0 + r)) continue;
      float x[kVs];
      a[n].get(x);
#pragma unroll
      for (int v = 0; v < kVs; v += 4) *reinterpret_cast<float4*>(&row[r][e + v]) = make_float4(x[v], x[v + 1], x[v + 2], x[v + 3]);
    }
    __syncwarp();
    const int turned = min(min(h_end, p.st[1].end) - h0, kStagedRows);
    for (int r = 0; r < turned; ++r) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        const int i = lane + 32 * j;
        if (i < p.half) {
          const float x0 = row[r][i], x1 = row[r][i + p.half];
          row[r][i] = x0 * c[j] - x1 * s[j];
          row[r][i + p.half] = x1 * c[j] + x0 * s[j];
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kStores; ++n) {
      const int f = n * 32 + lane, r = f / (D / kVd), h = h0 + r, e = f % (D / kVd) * kVd;
      const int i = h < p.st[0].end ? 0 : (h < p.st[1].end ? 1 : 2);
      if (!written(h)) continue;
      float x[kVd];
#pragma unroll
      for (int v = 0; v < kVd; v += 4) {
        const float4 y = *reinterpret_cast<const float4*>(&row[r][e + v]);
        x[v] = y.x; x[v + 1] = y.y; x[v + 2] = y.z; x[v + 3] = y.w;
      }
      Vec<TD, kVd> y;
      y.set(x);
      y.store(static_cast<TD*>(p.st[i].dst) + (i == 0 ? k.dst[0] : (i == 1 ? k.dst[1] : k.dst[2])) +
              (h - (i == 0 ? 0 : p.st[i - 1].end)) * p.st[i].d_h + e);
    }
    __syncwarp();
  }
}

template <int PAIRING, int D, typename TS, typename TD>
cudaError_t go(RotaryParams p, cudaStream_t st) {
  constexpr int kLanes = D / 16;
  const long long lanes = static_cast<long long>(p.tokens) * kLanes;
  // Heads per thread: as many as launch about 8 warps of threads for each of the GPU's 592
  // schedulers, so that the angles (about 3 us of latency) are shared by many heads; a small
  // call spreads its heads over threads instead.  6 of the 8 are resident with 80 registers
  // (16 bits, interleaved), 5 with 90 (half-split): calls of the rule's size end in a partly
  // empty wave (3 x 4,097 tokens 1,538 blocks on 740 places, 7,168 appended ones 1,344 on 888).
  // Sequences [3, 4097] of 24 heads: 118 us at one head a thread, 33 us at four and more.  One
  // sequence of 7,168 tokens, 48 heads: 37 us at 8 warps, 43 at 6 and at 4, 39 at 12.  Blocks of
  // 128 threads and two heads in flight beat 256 and four (720p-like Q and K 499 against 507 us).
  long long g = lanes * p.heads / (148LL * 1024);
  g = g < 1 ? 1 : (g > p.heads ? p.heads : g);
  const int groups = static_cast<int>((p.heads + g - 1) / g);
  p.group = (p.heads + groups - 1) / groups;
  dim3 grid(static_cast<unsigned>((lanes + kThreads - 1) / kThreads), groups);
  rotary_kernel<PAIRING, D, TS, TD><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D, typename TS, typename TD>
cudaError_t go_staged(RotaryParams p, cudaStream_t st) {
  // heads per warp: as many as leave about 8 warps on each scheduler
  long long g = static_cast<long long>(p.tokens) * p.heads / (592LL * kStagedWarps);
  if (g > kStagedRows) g = (g + kStagedRows - 1) / kStagedRows * kStagedRows;
  g = g < 1 ? 1 : (g > p.heads ? p.heads : g);
  p.group = static_cast<int>(g);
  constexpr int kWarps = kThreads / 32;
  dim3 grid(static_cast<unsigned>((static_cast<long long>(p.tokens) + kWarps - 1) / kWarps),
            static_cast<unsigned>((p.heads + g - 1) / g));
  rotary_staged_kernel<D, TS, TD><<<grid, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <int D, typename TS, typename TD>
cudaError_t by_pairing(const RotaryParams& p, int style, cudaStream_t st) {
  if (style == NABLA_ROPE_INTERLEAVED) return go<kInterleaved, D, TS, TD>(p, st);
  return p.half % 8 == 0 ? go<kHalf, D, TS, TD>(p, st) : go_staged<D, TS, TD>(p, st);
}

template <typename TS, typename TD>
cudaError_t by_width(const RotaryParams& p, int style, int D, cudaStream_t st) {
  return D == 64 ? by_pairing<64, TS, TD>(p, style, st) : by_pairing<128, TS, TD>(p, style, st);
}

cudaError_t by_dtype(const RotaryParams& p, int style, int D, int src, int dst, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (src == NABLA_BF16) return dst == NABLA_BF16 ? by_width<bf, bf>(p, style, D, st) : by_width<bf, float>(p, style, D, st);
  if (src == NABLA_F16) return dst == NABLA_F16 ? by_width<__half, __half>(p, style, D, st) : by_width<__half, float>(p, style, D, st);
  return dst == NABLA_F32    ? by_width<float, float>(p, style, D, st)
         : dst == NABLA_BF16 ? by_width<float, bf>(p, style, D, st)
                             : by_width<float, __half>(p, style, D, st);
}

nabla_status check_rope(const nabla_rope& r, int D) {
  if (r.style != NABLA_ROPE_INTERLEAVED && r.style != NABLA_ROPE_HALF) return NABLA_ERR_INVALID_ARG;
  if (r.axes != 1 && r.axes != 3) return NABLA_ERR_INVALID_ARG;
  if (r.dim < 2 || (r.dim & 1) || r.dim > D) return NABLA_ERR_INVALID_ARG;
  if (r.axes == 3) {
    int sum = 0;
    for (int a = 0; a < 3; ++a) {
      if (r.axis_dim[a] < 0 || (r.axis_dim[a] & 1) || r.axis_dim[a] > D) return NABLA_ERR_INVALID_ARG;
      sum += r.axis_dim[a];
    }
    if (sum != r.dim) return NABLA_ERR_INVALID_ARG;
  }
  if (!r.inv_freq || (reinterpret_cast<uintptr_t>(r.inv_freq) & 7)) return NABLA_ERR_INVALID_ARG;
  if (!isfinite(r.magnitude)) return NABLA_ERR_INVALID_ARG;
  return NABLA_OK;
}

void set_rope(RotaryParams* p, const nabla_rope& r) {
  p->axes = r.axes;
  p->half = r.dim / 2;
  p->ax1 = r.axes == 3 ? r.axis_dim[0] / 2 : p->half;
  p->ax2 = r.axes == 3 ? p->ax1 + r.axis_dim[1] / 2 : p->half;
  p->magnitude = r.magnitude;
  p->inv_freq = r.inv_freq;
}

void set_src(Stream* s, const nabla_heads& x) {
  s->src = x.ptr;
  s->s_b = x.stride_b; s->s_h = x.stride_h; s->s_s = x.stride_s;
}
void set_dst(Stream* s, const nabla_heads& x) {
  s->dst = x.ptr;
  s->d_b = x.stride_b; s->d_h = x.stride_h; s->d_s = x.stride_s;
}

}  // namespace
}  // namespace nabla

using namespace nabla;

extern "C" nabla_status nabla_rotary_freqs(int32_t dim, double base, nabla_rope_scaling scaling, double factor,
                                           double trained_len, double* inv_freq, double* magnitude) {
  if (dim < 2 || (dim & 1) || !inv_freq) return NABLA_ERR_INVALID_ARG;
  if (!(base > 1.0) || !isfinite(base) || !(factor >= 1.0) || !isfinite(factor)) return NABLA_ERR_INVALID_ARG;
  if (scaling < NABLA_ROPE_PLAIN || scaling > NABLA_ROPE_PARTS) return NABLA_ERR_INVALID_ARG;
  if (scaling == NABLA_ROPE_PARTS && (!(trained_len >= 1.0) || !isfinite(trained_len))) return NABLA_ERR_INVALID_ARG;
  const double pi = 3.14159265358979323846;
  double b = base;
  if (scaling == NABLA_ROPE_BASE && dim > 2) b = base * pow(factor, static_cast<double>(dim) / (dim - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == NABLA_ROPE_PARTS) {
    // pair whose wavelength fits `turns` times into the trained length
    auto pair_at = [&](double turns) { return dim * log(trained_len / (turns * 2.0 * pi)) / (2.0 * log(base)); };
    lo = fmax(floor(pair_at(32.0)), 0.0);
    hi = fmin(ceil(pair_at(1.0)), dim - 1.0);
  }
  for (int j = 0; j < dim / 2; ++j) {
    double f = pow(b, -2.0 * j / dim);
    if (scaling == NABLA_ROPE_LINEAR) f /= factor;
    if (scaling == NABLA_ROPE_PARTS) {
      const double ramp = fmin(fmax((j - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    inv_freq[j] = f;
  }
  if (magnitude) *magnitude = scaling == NABLA_ROPE_PARTS ? 0.1 * log(factor) + 1.0 : 1.0;
  return NABLA_OK;
}

extern "C" nabla_status nabla_rotary(nabla_heads q_src, nabla_heads q_dst, nabla_heads k_src, nabla_heads k_dst,
                                     int32_t B, nabla_grid grid, int32_t D, nabla_rope rope, nabla_grid origin,
                                     const int32_t* positions, nabla_layout src_layout, nabla_layout dst_layout,
                                     int32_t adjoint, nabla_stream_t stream) {
  if (B < 1 || grid.T < 1 || grid.Hg < 1 || grid.W < 1) return NABLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return NABLA_ERR_UNSUPPORTED;
  nabla_status rc = check_rope(rope, D);
  if (rc != NABLA_OK) return rc;
  if (adjoint != 0 && adjoint != 1) return NABLA_ERR_INVALID_ARG;
  for (const nabla_layout l : {src_layout, dst_layout}) {
    if (l != NABLA_LAYOUT_NATURAL && l != NABLA_LAYOUT_REORDERED) return NABLA_ERR_INVALID_ARG;
    if (l == NABLA_LAYOUT_REORDERED && (grid.Hg % 8 || grid.W % 8)) return NABLA_ERR_INVALID_ARG;
  }
  const double tokens = static_cast<double>(B) * grid.T * grid.Hg * grid.W;
  if (tokens >= 2147483648.0) return NABLA_ERR_UNSUPPORTED;
  const int64_t S = static_cast<int64_t>(grid.T) * grid.Hg * grid.W;
  if (positions && (reinterpret_cast<uintptr_t>(positions) & 3)) return NABLA_ERR_INVALID_ARG;
  const bool has_q = q_src.ptr || q_dst.ptr, has_k = k_src.ptr || k_dst.ptr;
  if (!has_q && !has_k) return NABLA_ERR_INVALID_ARG;
  const nabla_heads* in[2] = {&q_src, &k_src};
  const nabla_heads* out[2] = {&q_dst, &k_dst};
  const bool has[2] = {has_q, has_k};
  RotaryParams p = {};
  int heads = 0, sdt = -1, ddt = -1;
  for (int i = 0; i < 2; ++i) {
    if (has[i]) {
      if ((rc = check_heads(*in[i], B, S, false)) != NABLA_OK || (rc = check_heads(*out[i], B, S, true)) != NABLA_OK) return rc;
      if (in[i]->H != out[i]->H) return NABLA_ERR_INVALID_ARG;
      if (sdt >= 0 && (sdt != in[i]->dtype || ddt != out[i]->dtype)) return NABLA_ERR_INVALID_ARG;
      sdt = in[i]->dtype;
      ddt = out[i]->dtype;
      for (int j = 0; j < 2; ++j)
        if (has[j] && heads_overlap(*in[j], *out[i], B, S, D)) return NABLA_ERR_INVALID_ARG;
      set_src(&p.st[i], *in[i]);
      set_dst(&p.st[i], *out[i]);
      if (in[i]->H > 65535 - heads) return NABLA_ERR_UNSUPPORTED;
      heads += in[i]->H;
    }
    p.st[i].end = heads;
  }
  if (has_q && has_k && q_dst.ptr == k_dst.ptr) return NABLA_ERR_INVALID_ARG;
  if (sdt != ddt && sdt != NABLA_F32 && ddt != NABLA_F32) return NABLA_ERR_INVALID_ARG;   // bf16 <-> fp16
  p.st[2].end = heads;
  p.heads = heads;
  p.tokens = static_cast<int>(tokens);
  p.S = static_cast<int>(S);
  p.Hg = grid.Hg; p.W = grid.W;
  p.T0 = origin.T; p.H0 = origin.Hg; p.W0 = origin.W;
  p.src_blocks = src_layout == NABLA_LAYOUT_REORDERED;
  p.dst_blocks = dst_layout == NABLA_LAYOUT_REORDERED;
  p.sign = adjoint ? -1.f : 1.f;
  set_rope(&p, rope);
  p.positions = positions;
  return cuda_status(by_dtype(p, rope.style, D, sdt, ddt, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" nabla_status nabla_cache_append(nabla_heads k, nabla_heads v, nabla_heads q_src, nabla_heads q_dst,
                                           int32_t B, int32_t S, nabla_cache cache, const int32_t* page_table,
                                           int32_t table_width, const int32_t* start, const int32_t* counts,
                                           const nabla_rope* rope, nabla_grid frame, int64_t pos0,
                                           const int32_t* positions, uint32_t* status, nabla_stream_t stream) {
  if (B < 1 || S < 1) return NABLA_ERR_INVALID_ARG;
  nabla_status rc = check_cache(cache);
  if (rc != NABLA_OK) return rc;
  if (rope) {
    if ((rc = check_rope(*rope, cache.D)) != NABLA_OK) return rc;
    if (rope->axes == 3 && !positions && (frame.Hg < 1 || frame.W < 1)) return NABLA_ERR_INVALID_ARG;
  }
  if (static_cast<double>(B) * S >= 2147483648.0) return NABLA_ERR_UNSUPPORTED;
  if (!page_table || table_width < 1 || !start) return NABLA_ERR_INVALID_ARG;
  if (static_cast<int64_t>(table_width) * cache.page > 2147483647LL) return NABLA_ERR_UNSUPPORTED;
  if (pos0 < 0 || pos0 > (1LL << 40)) return NABLA_ERR_INVALID_ARG;
  for (const void* x : {static_cast<const void*>(page_table), static_cast<const void*>(start),
                        static_cast<const void*>(counts), static_cast<const void*>(positions),
                        static_cast<const void*>(status)})
    if (reinterpret_cast<uintptr_t>(x) & 3) return NABLA_ERR_INVALID_ARG;
  if ((rc = check_heads(k, B, S, false)) != NABLA_OK || (rc = check_heads(v, B, S, false)) != NABLA_OK) return rc;
  if (k.H != cache.H || v.H != cache.H || k.dtype != cache.dtype || v.dtype != cache.dtype) return NABLA_ERR_INVALID_ARG;
  // the pools are written page by page: they may not hold each other or a source
  const int64_t pool = static_cast<int64_t>(cache.n_pages) * cache.H * cache.page * cache.D;
  nabla_heads kc = {cache.k, cache.dtype, 1, 0, 0, cache.D}, vc = {cache.v, cache.dtype, 1, 0, 0, cache.D};
  auto hits = [&](const nabla_heads& x, const nabla_heads& pl) {
    return static_cast<const char*>(x.ptr) < static_cast<const char*>(pl.ptr) + pool * 2 &&
           static_cast<const char*>(pl.ptr) < heads_end(x, B, S, cache.D);
  };
  if (static_cast<const char*>(kc.ptr) < static_cast<const char*>(vc.ptr) + pool * 2 &&
      static_cast<const char*>(vc.ptr) < static_cast<const char*>(kc.ptr) + pool * 2)
    return NABLA_ERR_INVALID_ARG;
  if (hits(k, kc) || hits(k, vc) || hits(v, kc) || hits(v, vc)) return NABLA_ERR_INVALID_ARG;
  const bool has_q = q_src.ptr || q_dst.ptr;
  RotaryParams p = {};
  int heads = 0;
  if (has_q) {
    if (!rope) return NABLA_ERR_INVALID_ARG;   // nothing would happen to Q
    if ((rc = check_heads(q_src, B, S, false)) != NABLA_OK || (rc = check_heads(q_dst, B, S, true)) != NABLA_OK) return rc;
    if (q_src.H != q_dst.H || q_src.dtype != cache.dtype || q_dst.dtype != cache.dtype) return NABLA_ERR_INVALID_ARG;
    if (hits(q_src, kc) || hits(q_src, vc) || hits(q_dst, kc) || hits(q_dst, vc)) return NABLA_ERR_INVALID_ARG;
    if (heads_overlap(q_src, q_dst, B, S, cache.D) || heads_overlap(k, q_dst, B, S, cache.D) ||
        heads_overlap(v, q_dst, B, S, cache.D))
      return NABLA_ERR_INVALID_ARG;
    set_src(&p.st[0], q_src);
    set_dst(&p.st[0], q_dst);
    heads = q_src.H;
  }
  if (cache.H > 16383 || heads > 32767) return NABLA_ERR_UNSUPPORTED;
  p.st[0].end = heads;
  p.st[1].end = heads + cache.H;
  p.st[2].end = heads + 2 * cache.H;
  set_src(&p.st[1], k);
  set_src(&p.st[2], v);
  p.st[1].dst = cache.k;
  p.st[2].dst = cache.v;
  for (int i = 1; i < 3; ++i) {
    p.st[i].d_s = cache.D;
    p.st[i].d_h = static_cast<long long>(cache.page) * cache.D;
  }
  p.heads = heads + 2 * cache.H;
  p.tokens = B * S;
  p.S = S;
  p.Hg = frame.Hg; p.W = frame.W;
  p.sign = 1.f;
  int style = NABLA_ROPE_INTERLEAVED;
  if (rope) {
    set_rope(&p, *rope);
    style = rope->style;
    p.positions = positions;
  } else {
    p.axes = 1;
    p.half = 0;      // no pair is rotated: K is copied
  }
  p.table = page_table;
  p.table_w = table_width;
  p.start = start;
  p.counts = counts;
  p.pos0 = pos0;
  p.n_pages = cache.n_pages;
  p.page = cache.page;
  while ((1 << p.page_shift) < cache.page) ++p.page_shift;
  p.page_stride = static_cast<long long>(cache.H) * cache.page * cache.D;
  p.status = status;
  return cuda_status(by_dtype(p, style, cache.D, cache.dtype, cache.dtype, reinterpret_cast<cudaStream_t>(stream)));
}
