// block_select.cuh -- the cheap score of block-selected attention: key-block
// means, and the selection of the best-scoring blocks per query.
//
//   c_j = mean of the keys of block j (64 tokens, the last one ragged), bf16
//   s_rj = sum over the G query heads of a KV head of q_gr . c_j
//        = (sum_g q_gr) . c_j
//
// Row r takes the first n_first and the last n_local of its visible blocks,
// and fills the rest of its n_sel slots with the best scores among the other
// visible blocks, equal scores to the lower index.  The list is written in
// ascending order, -1 in slots left over.
//
// The chosen set is the one the exact scores give.  Scores are first formed
// in float32 (tensor core in the prompt form) together with a bound e on
// their error; blocks within 2 e of the cut are scored again in float64 and
// ranked by that (a few per cent of the rows have any).
#pragma once

#include "decode_mma.cuh"

namespace blasst {

constexpr int kSelBlock = 64;  // keys per selection block

// ---------------------------------------------------------------------------
// Block means
// ---------------------------------------------------------------------------
struct MeansArgs {
  const __nv_bfloat16* k;  // [B, Hkv, L, d], or the pool
  __nv_bfloat16* means;    // [B, Hkv, max_blocks, d]
  int Hkv, L, nblk;        // L: keys (contiguous), upper bound (paged)
  int max_blocks;          // blocks per (sequence, head) in means
  // paged
  const int* block_table;
  const int* seq_lens;
  long long page_stride;
  int log2_page, max_pages, num_pages, n_new;
};

// One CTA of 128 threads per block: a thread sums 8 columns (16 bytes) of
// every (128 / (D/8))-th row, all its loads in flight at once; the row groups
// are added through a shuffle and shared memory in a fixed order.  Bound by
// HBM: the keys are read once (16K keys x 8 heads, 34 MB: 8.4 us from HBM, 4.2
// from L2; a decode step's last blocks, batch 32 x 8 heads: 3 us, latency).
template <int D, bool PAGED>
__global__ void __launch_bounds__(128) block_means_kernel(const MeansArgs a) {
  constexpr int CH = D / 8;        // 16-byte chunks of a row
  constexpr int RG = 128 / CH;     // row groups
  constexpr int NR = kSelBlock / RG;
  __shared__ float red[4][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = tid % CH, rg = tid / CH;
  const int bh = PAGED ? (int)blockIdx.x : (int)(blockIdx.x / a.nblk);
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  int L = a.L, j;
  const int* bt = nullptr;
  if constexpr (PAGED) {
    L = __ldg(a.seq_lens + b);
    if (L < 0 || L > a.L) {  // uniform across the CTA
      if (tid == 0) record_error(kBadSeqLen, (unsigned)b, (unsigned)L, 0);
      return;
    }
    // the blocks the last n_new tokens lie in (all of them for 0)
    const int first = a.n_new > 0 && a.n_new < L ? L - a.n_new : 0;
    const long long jl = first / kSelBlock + (long long)blockIdx.y;
    if (jl * kSelBlock >= L) return;
    j = (int)jl;
    bt = a.block_table + (size_t)b * a.max_pages;
  } else {
    j = (int)(blockIdx.x - (unsigned)bh * (unsigned)a.nblk);
  }
  const int t0 = j * kSelBlock;
  const int n = min(kSelBlock, L - t0);
  uint4 w[NR];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = i * RG + rg;
    w[i] = make_uint4(0, 0, 0, 0);
    if (row < n) {
      const __nv_bfloat16* src;
      if constexpr (PAGED) {
        const int t = t0 + row;
        const int id = __ldg(bt + (t >> a.log2_page));
        if (id < 0 || id >= a.num_pages) {
          record_error(kBadPageId, (unsigned)b, (unsigned)(t >> a.log2_page),
                       (unsigned)id);
          bad = true;
          continue;
        }
        const int ps = 1 << a.log2_page;
        src = a.k + (long long)id * a.page_stride +
              ((long long)h * ps + (t & (ps - 1))) * D;
      } else {
        src = a.k + ((size_t)bh * a.L + t0 + row) * D;
      }
      w[i] = __ldg(reinterpret_cast<const uint4*>(src) + chunk);
    }
  }
  if constexpr (PAGED) {
    if (__syncthreads_or(bad)) return;  // the block's mean stays as it was
  }
  float s[8];
#pragma unroll
  for (int x = 0; x < 8; ++x) s[x] = 0.f;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      s[2 * x] += bf16lo(u[x]);
      s[2 * x + 1] += bf16hi(u[x]);
    }
  }
#pragma unroll
  for (int o = CH; o < 32; o <<= 1)  // lanes of the warp on the same chunk
#pragma unroll
    for (int x = 0; x < 8; ++x) s[x] += __shfl_xor_sync(0xffffffffu, s[x], o);
  if (lane < CH) {
#pragma unroll
    for (int x = 0; x < 8; ++x) red[warp][chunk * 8 + x] = s[x];
  }
  __syncthreads();
  if (tid < D / 2) {
    const float fn = (float)n;
    float m[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = 2 * tid + e;
      m[e] = ((red[0][c] + red[1][c]) + (red[2][c] + red[3][c])) / fn;
    }
    reinterpret_cast<uint32_t*>(a.means + ((size_t)bh * a.max_blocks + j) *
                                              D)[tid] = pack_bf16x2(m[0], m[1]);
  }
}

// ---------------------------------------------------------------------------
// Selection among the scores of one row
// ---------------------------------------------------------------------------
// Warp-wide maximum and minimum (one instruction each on sm_100).
__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float redux_min(float x) {
  float y;
  asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The threads that work on one row: a warp, or a whole CTA.
struct WarpGroup {
  static constexpr int kThreads = 32;
  int id, warp, nwarps;
  __device__ WarpGroup() : id(threadIdx.x & 31), warp(0), nwarps(1) {}
  __device__ void sync() { __syncwarp(); }
  __device__ int add(int x) { return (int)__reduce_add_sync(~0u, (unsigned)x); }
  __device__ float max(float x) { return redux_max(x); }
  // exclusive rank of the set flags, and their number
  __device__ int rank(bool f, int& total) {
    const unsigned m = __ballot_sync(~0u, f);
    total = __popc(m);
    return __popc(m & ((1u << id) - 1u));
  }
};

template <int NT>
struct CtaGroup {
  static constexpr int kThreads = NT;
  static constexpr int kWarps = NT / 32;
  int id, warp, nwarps, flip;
  uint32_t* scratch;  // [2][kWarps] shared
  __device__ explicit CtaGroup(uint32_t* s)
      : id(threadIdx.x), warp(threadIdx.x >> 5), nwarps(kWarps), flip(0),
        scratch(s) {}
  __device__ void sync() { __syncthreads(); }
  // Each reduction writes its own half of the scratch words, alternating, so
  // one barrier per reduction separates readers from the next writers.
  __device__ const uint32_t* share(uint32_t x) {
    uint32_t* s = scratch + flip * kWarps;
    flip ^= 1;
    if ((id & 31) == 0) s[warp] = x;
    __syncthreads();
    return s;
  }
  __device__ int add(int x) {
    const uint32_t* s = share(__reduce_add_sync(~0u, (unsigned)x));
    int t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += (int)s[w];
    return t;
  }
  __device__ float max(float x) {
    const uint32_t* s = share(__float_as_uint(redux_max(x)));
    float t = __uint_as_float(s[0]);
#pragma unroll
    for (int w = 1; w < kWarps; ++w) t = fmaxf(t, __uint_as_float(s[w]));
    return t;
  }
  __device__ int rank(bool f, int& total) {
    const unsigned m = __ballot_sync(~0u, f);
    const uint32_t* s = share(__popc(m));
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += (int)s[w];
      total += (int)s[w];
    }
    return before + __popc(m & ((1u << (id & 31)) - 1u));
  }
};

// Cut of the k largest of s[0..n): every s > v is in, and of those equal to
// v the lowest indices fill up; a is the smallest value taken, b the largest
// left (a == b when equal values straddle the cut).  1 <= k < n; s holds no
// NaN.  Bisection on the value between the extremes, ended early by a
// midpoint that separates exactly k.
struct Cut {
  float v, a, b;
};
template <class GroupT>
__device__ Cut find_cut(GroupT& g, const float* s, int n, int k) {
  float mx = -INFINITY, mn = INFINITY;  // of the finite values
  int n_hi = 0, n_fin = 0;
  for (int i = g.id; i < n; i += GroupT::kThreads) {
    const float x = s[i];
    if (x == INFINITY) ++n_hi;
    if (fabsf(x) < INFINITY) {
      ++n_fin;
      mx = fmaxf(mx, x);
      mn = fminf(mn, x);
    }
  }
  n_hi = g.add(n_hi);
  n_fin = g.add(n_fin);
  mx = g.max(mx);
  mn = -g.max(-mn);
  if (n_hi > k) return {INFINITY, INFINITY, INFINITY};
  if (n_hi + n_fin < k) return {-INFINITY, -INFINITY, -INFINITY};
  // in [lo, hi): at least k values are >= lo, fewer than k are >= hi
  float t;  // a threshold that exactly k values reach
  bool exact = false;
  if (n_hi == k) {
    t = INFINITY;
    exact = true;
  } else {
    float lo = mn, hi = INFINITY;
    int c = n_hi + n_fin;
    t = mn;
    if (c == k) exact = true;
    bool first = true;
    while (!exact) {
      float mid;
      if (first) {
        mid = mx;
        first = false;
        if (!(mid > lo)) break;  // all finite values equal
      } else {
        mid = 0.5f * lo + 0.5f * hi;
        if (!(mid > lo && mid < hi)) break;
      }
      c = 0;
      for (int i = g.id; i < n; i += GroupT::kThreads) c += s[i] >= mid;
      c = g.add(c);
      if (c == k) {
        t = mid;
        exact = true;
      } else if (c > k) {
        lo = mid;
        if (mid == mx) break;  // more than k values equal the largest
      } else {
        hi = mid;
      }
    }
    if (!exact) return {lo, lo, lo};
  }
  float a = INFINITY, b = -INFINITY;
  for (int i = g.id; i < n; i += GroupT::kThreads) {
    const float x = s[i];
    if (x >= t) a = fminf(a, x);
    else b = fmaxf(b, x);
  }
  a = -g.max(-a);
  b = g.max(b);
  return {a, a, b};
}

// One row's candidates for a warp: the k best of blocks [f, f + n) by the
// approximate scores s, each off by at most eps, go to out; 0 < k < n.
struct RowTask {
  const float* s;
  int* out;
  int f, n, k;
  float eps;
};

// A row's scores for one warp, lane l holding every 32nd from l: in NR
// registers, or (NR 0) where they are.  each(f) calls f(x, score 32 x + lane),
// -infinity past the end.
template <int NR>
struct RowScores {
  float v[NR];
  __device__ __forceinline__ explicit RowScores(const RowTask& r) {
#pragma unroll
    for (int x = 0; x < NR; ++x) {
      const int i = 32 * x + (int)(threadIdx.x & 31);
      v[x] = i < r.n ? r.s[i] : -INFINITY;
    }
  }
  template <class F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int x = 0; x < NR; ++x) f(x, v[x]);
  }
};
template <>
struct RowScores<0> {
  const float* s;
  int n;
  __device__ __forceinline__ explicit RowScores(const RowTask& r)
      : s(r.s), n(r.n) {}
  template <class F>
  __device__ __forceinline__ void each(F f) const {
    const int lane = threadIdx.x & 31;
#pragma unroll 4
    for (int x = 0; x < (n + 31) / 32; ++x)
      f(x, 32 * x + lane < n ? s[32 * x + lane] : -INFINITY);
  }
};

// The same cut by one warp for n finite scores:
// t splits off exactly k (split), or equal values at t (or a float step above
// it) straddle the cut.  A prompt has a row per token and KV head, so this
// sets the selection's time.  The first thresholds come from the normal
// distribution of the scores' mean and variance (a score sums d products) and
// from its density there, the next from bisection: about 4 passes of NR
// compares and one warp reduction where bisection alone takes 9.
template <class ScoresT>
__device__ __forceinline__ void find_cut(const RowTask& r, const ScoresT& v,
                                         float& t, bool& split) {
  const int lane = threadIdx.x & 31;
  // at least k values are >= lo; fewer than k are >= hi, or hi is the maximum
  float lo = INFINITY, hi = -INFINITY, s1 = 0.f, s2 = 0.f;
  v.each([&](int x, float z) {
    const bool in = 32 * x + lane < r.n;
    hi = fmaxf(hi, z);
    lo = fminf(lo, in ? z : INFINITY);
    z = in ? z : 0.f;
    s1 += z;
    s2 = fmaf(z, z, s2);
  });
  hi = redux_max(hi);
  lo = redux_min(lo);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    s1 += __shfl_xor_sync(~0u, s1, o);
    s2 += __shfl_xor_sync(~0u, s2, o);
  }
  // the k / n quantile of a normal distribution (Abramowitz and Stegun,
  // 26.2.22: within 3e-3) and 1 / (n times its density there)
  const float n = (float)r.n;
  const float mu = s1 / n, sd = sqrtf(fmaxf(s2 / n - mu * mu, 0.f));
  const float p = (float)r.k / n, q = fminf(p, 1.f - p);
  const float w = sqrtf(-2.f * __logf(q));
  const float z = w - __fdividef(2.30753f + 0.27061f * w,
                                 1.f + w * (0.99229f + 0.04481f * w));
  const float gain = __fdividef(2.5066283f * sd, n) * __expf(0.5f * z * z);
  t = p < 0.5f ? fmaf(z, sd, mu) : fmaf(-z, sd, mu);
  split = false;
  if (!(t > lo && t < hi)) t = 0.5f * lo + 0.5f * hi;
  if (!(t > lo && t < hi)) t = lo;  // one value, or no float between two
  for (int pass = 0; t > lo; ++pass) {
    int c = 0;
    v.each([&](int, float y) { c += y >= t; });
    const int d = (int)__reduce_add_sync(~0u, (unsigned)c) - r.k;
    if (d == 0) {
      split = true;
      return;
    }
    if (d > 0) lo = t;
    else hi = t;
    t = fmaf((float)d, gain, t);
    if (pass >= 3 || !(t > lo && t < hi)) t = 0.5f * lo + 0.5f * hi;
    if (!(t > lo && t < hi)) t = lo;
  }
}

// The take of one row after its cut.  When the cut is not wider than 2 eps,
// the blocks within 2 eps of it (2 or 3, on a few rows of a hundred) get a
// lane each for their float64 score and are ranked there.  (Without a split
// the equal values lie within a float step of t, far inside 2 eps.)  Returns
// false, with nothing written, when they are more than 32, or when equal
// scores straddle the cut and eps is 0.
template <class ScoresT, class ExactT>
__device__ __forceinline__ bool take_cut(const RowTask& r, const ScoresT& v,
                                         float t, bool split, ExactT exact) {
  const int lane = threadIdx.x & 31;
  const unsigned below = (1u << lane) - 1u;
  int* out = r.out;
  float a = t, b = t;  // smallest taken, largest left
  if (split) {
    a = INFINITY;
    b = -INFINITY;
    v.each([&](int, float y) {
      if (y >= t) a = fminf(a, y);
      else b = fmaxf(b, y);
    });
    a = redux_min(a);
    b = redux_max(b);
    if (a - b > 2.f * r.eps) {
      v.each([&](int x, float y) {
        const unsigned m = __ballot_sync(~0u, y >= t);
        if (y >= t) out[__popc(m & below)] = r.f + 32 * x + lane;
        out += __popc(m);
      });
      return true;
    }
  } else if (r.eps == 0.f) {
    return false;
  }
  const float up = b + 2.f * r.eps;  // above: taken for certain
  const float dn = a - 2.f * r.eps;  // below: left for certain
  int sure = 0, cnt = 0;
  v.each([&](int, float y) {
    sure += __popc(__ballot_sync(~0u, y > up));
    cnt += __popc(__ballot_sync(~0u, y >= dn && y <= up));
  });
  if (cnt > 32) return false;
  // lane o gets the o-th doubtful block, in ascending order
  int mine_at = 0, at = 0;
  v.each([&](int x, float y) {
    unsigned m = __ballot_sync(~0u, y >= dn && y <= up);
    for (; m; m &= m - 1, ++at)
      if (lane == at) mine_at = 32 * x + __ffs(m) - 1;
  });
  double mine = 0.0;
  for (int o = 0; o < cnt; ++o) {
    const double e = exact(r.f + __shfl_sync(~0u, mine_at, o));
    if (lane == o) mine = e;
  }
  int ahead = 0;  // doubtful blocks that go before this lane's
  for (int o = 0; o < cnt; ++o) {
    const double e = __shfl_sync(~0u, mine, o);
    ahead += e > mine || (e == mine && o < lane);
  }
  unsigned won = __ballot_sync(~0u, lane < cnt && ahead < r.k - sure);
  v.each([&](int x, float y) {
    const bool doubt = y >= dn && y <= up;
    unsigned m = __ballot_sync(~0u, doubt);
    const bool take = y > up || (doubt && ((won >> __popc(m & below)) & 1u));
    const int c = __popc(m);
    won = c < 32 ? won >> c : 0u;
    m = __ballot_sync(~0u, take);
    if (take) out[__popc(m & below)] = r.f + 32 * x + lane;
    out += __popc(m);
  });
  return true;
}

// Cut and take of one row (n <= 32 NR, or NR 0); false: left to take_general.
template <int NR, class ExactT>
__device__ __forceinline__ bool take_row(const RowTask& r, ExactT exact) {
  const RowScores<NR> v(r);
  float t;
  bool split;
  find_cut(r, v, t, split);
  return take_cut(r, v, t, split, exact);
}

// The take of one row in general, by a warp or a CTA, for any n: s is
// overwritten where the cut needs it.  exact(j) (taken by a whole warp) is the
// float64 score of block j.
//
// Blocks whose place a cut leaves open are scored again, as the distance of
// their exact score to a reference among them, rounded.  Rounding keeps the
// order, so after another cut only blocks that tie there are open; the next
// round takes the first of them as its reference, and the rounds end when the
// tied blocks equal it in float64.
template <class GroupT, class ExactT>
__device__ void take_general(GroupT& g, float* s, const RowTask& r,
                             ExactT exact) {
  const int n = r.n, k = r.k;
  const float eps = r.eps;
  const int lane = threadIdx.x & 31;
  int* out = r.out;
  Cut c;
  float lo = -INFINITY, hi = INFINITY;  // open: lo <= s <= hi
  double ref = 0.0;
  bool again = !(eps < INFINITY);  // a bound that overflowed: all are open
  if (!again) {
    c = find_cut(g, s, n, k);
    // the scores are exact when eps is 0; otherwise the order is certain
    // only when the cut is wider than the two errors: above b + 2 eps is
    // better than every value left out, below a - 2 eps worse than all taken
    again = eps > 0.f && !(c.a - c.b > 2.f * eps);
    lo = c.a - 2.f * eps;
    hi = c.b + 2.f * eps;
    ref = (double)c.v;
  }
  bool nan_only = false;  // -infinities against NaN, which ranks below them
  for (bool start = true; again; start = false) {
    g.sync();
    for (int i0 = 32 * g.warp; i0 < n; i0 += 32 * g.nwarps) {
      const int i = i0 + lane;
      const float x = i < n ? s[i] : 0.f;
      float y = x > hi ? INFINITY : -INFINITY;
      unsigned todo = __ballot_sync(~0u, i < n && x >= lo && x <= hi);
      while (todo) {
        const int t = __ffs(todo) - 1;
        todo &= todo - 1;
        const double e = exact(r.f + i0 + t) - ref;
        if (lane == t) {
          // later rounds: exponent and 12 bits, float64's whole range
          const int u = (int)(__double_as_longlong(fabs(e)) >> 40);
          y = start ? (float)e : copysignf((float)u, (float)e);
          if (nan_only) y = 0.f;
          if (isnan(e)) y = -INFINITY;
        }
      }
      if (i < n) s[i] = y;
    }
    g.sync();
    c = find_cut(g, s, n, k);
    again = c.a == c.b && c.v < INFINITY && !nan_only &&
            (start || c.v != 0.f);
    if (!again) break;
    lo = hi = c.v;
    nan_only = c.v == -INFINITY;
    ref = 0.0;
    if (!nan_only) {
      float first = -INFINITY;
      for (int i = g.id; i < n; i += GroupT::kThreads)
        if (s[i] == c.v) first = fmaxf(first, -(float)i);
      ref = exact(r.f - (int)g.max(first));
    }
  }
  // values above the cut, then equal ones in ascending index
  int left = k;
  {
    int above = 0;
    for (int i = g.id; i < n; i += GroupT::kThreads) above += s[i] > c.v;
    left -= g.add(above);
  }
  for (int i0 = 0; i0 < n; i0 += GroupT::kThreads) {
    const int i = i0 + g.id;
    const float x = i < n ? s[i] : -INFINITY;
    int total;
    const bool eq = i < n && x == c.v;
    const int er = g.rank(eq, total);
    const bool take = i < n && (x > c.v || (eq && er < left));
    left -= min(left, total);
    const int rk = g.rank(take, total);
    if (take) out[rk] = r.f + i;
    out += total;
  }
}

struct SelectArgs {
  const __nv_bfloat16* q;      // [B, Hq, Lq, d]; decode [B, Hq, d]
  const __nv_bfloat16* means;  // [B, Hkv, nblk, d]
  int* sel;                    // [B, Hkv, Lq, n_sel]; decode [B, Hkv, n_sel]
  const int* seq_lens;         // decode
  int Hkv, G, Lq, Lkv, nblk;   // Lkv: upper bound on seq_lens in decode
  int causal, n_sel, n_first, n_local;
  int ntile, ld;               // prompt: row tiles, score row stride (floats)
};

// The row's regions: [0, f) and [m1, end) always taken, k of [f, m1) by score.
struct SelRange {
  int f, m1, end, k;
};
__device__ __forceinline__ SelRange sel_range(int last, int n_sel, int n_first,
                                              int n_local) {
  SelRange r;
  r.end = last + 1;
  r.f = min(n_first, r.end);
  r.m1 = max(r.f, r.end - n_local);
  r.k = n_sel - r.f - (r.end - r.m1);
  return r;
}

// The slots that need no score: blocks [0, f) and [m1, end), all of [f, m1)
// when they fit, and -1 behind them.  Returns whether k of [f, m1) are left to
// be chosen (0 < k < m1 - f), for the slots from f on.
template <class GroupT>
__device__ __forceinline__ bool fill_fixed(GroupT& g, const SelRange& r,
                                           int n_sel, int* out) {
  const int n = r.m1 - r.f;
  const int mid = min(r.k, n);  // slots of [f, m1)
  const int used = r.f + mid + (r.end - r.m1);
  const bool all = mid == n;
  for (int i = g.id; i < n_sel; i += GroupT::kThreads) {
    if (i >= used) out[i] = -1;
    else if (i < r.f || all) out[i] = i;
    else if (i >= r.f + mid) out[i] = r.m1 + i - r.f - mid;
  }
  return !all && mid > 0;
}

// Error bounds of the float32 scores: |w| |c| (2-norms), w the error of each
// term of the dot product per unit of c.
// Tensor core: x = sum_g q_g is split into two bf16 parts, whose rest is known
// exactly; its float32 sum is off by (G - 1) 2^-24 sum_g |q_g|.  The products
// of the parts are exact; a step adds 16 of them to the sum so far, and on
// B200 cuts each of the 17 to a multiple of 2^-25 of the largest one's power
// of two and the result to 24 bits (seen on sums that tell; always towards
// zero).  With |x| |c| above every partial sum a step is off by at most
// (17 + 4) 2^-25 |x| |c|.  The large parts' sum takes d / 16 steps; the small
// parts, 2^-8 of them, are summed apart, so that their steps cut 2^-8 of that;
// in one sum they would double the bound.  (16K prompt, 32 heads on 8: 202 us
// apart and 200 in one; 232 and 242 where the means share a direction 30 times
// their spread and more rows have doubtful blocks.)  The 22nd part covers them
// and the roundings of the norms.
// CUDA cores (no split): the head sum 2^-19 sum_g |q_g| for G <= 32, and 13
// roundings of 2^-24 in the dot product: below 2^-18 sum_g |q_g|.
template <int D>
constexpr float kSelEpsMma = (D / 16) * 22 * 2.98023223876953125e-08f;  // 2^-25
constexpr float kSelEpsFma = 3.814697265625e-06f;  // 2^-18
// Norms are summed over values scaled by 2^40 (the prompt kernel's means are
// not), so that squares of small values stay above float32's smallest (a sum
// that overflows only sends the row to the float64 scores).  What is still
// smaller must not count as nothing: unless every value is 0 a squared norm
// gets kNormFloor, far above what its squares can lose (128 of 2^-149).
constexpr float kNormUp = 1099511627776.f, kNormDown = 1.f / 1099511627776.f;
constexpr float kNormFloor = 4e-36f;

// The largest squared norm of the means at c (n chunks of 16 bytes) from its
// bits; whole CTA of NT threads.
template <int NT>
__device__ __forceinline__ float floor_norm(uint32_t bits,
                                            const __nv_bfloat16* c, int n) {
  if (bits >= __float_as_uint(kNormFloor)) return __uint_as_float(bits);
  uint32_t nz = 0u;  // bits of every value but their signs
  for (int e = threadIdx.x; e < n; e += NT) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(c) + e);
    nz |= (w.x | w.y | w.z | w.w) & 0x7fff7fffu;
  }
  return __syncthreads_or(nz != 0u) ? kNormFloor : 0.f;
}

// nw nc, for the norm nw of w and the largest norm nc of a mean, but no less
// than scores among float32's smallest numbers are off by; infinite where the
// scores themselves may leave float32's range (w is at least 2^-19 of what
// they sum); 0 where all are 0.
__device__ __forceinline__ float score_eps(float nw, float nc) {
  const float e = nw * nc;
  if (!(e < 5e32f)) return INFINITY;
  return nw > 0.f && nc > 0.f ? fmaxf(e, 1e-37f) : 0.f;
}

// The float64 score of one block for the whole warp; qd holds the lane's
// D / 32 head sums.
template <int D>
__device__ __forceinline__ double exact_score(const double (&qd)[D / 32],
                                              const __nv_bfloat16* c) {
  const int lane = threadIdx.x & 31;
  double e = 0.0;
#pragma unroll
  for (int x = 0; x < D / 32; ++x)
    e += qd[x] * (double)__bfloat162float(c[lane * (D / 32) + x]);
#pragma unroll
  for (int o = 16; o; o >>= 1) e += __shfl_xor_sync(~0u, e, o);
  return e;
}

// ---------------------------------------------------------------------------
// One token per sequence: a CTA per (sequence, KV head) scores every block
// (float32 on the CUDA cores: one pass over the means) and selects.  26 MB of
// means at batch 32 x 8 KV heads and 32K take 4 us at HBM's rate; the kernel's
// 13 us are a chain of latencies: lengths, q, means (4), the cut (6), a row's
// doubtful blocks (2).
// ---------------------------------------------------------------------------
constexpr int kSelDecThreads = 512;
constexpr int kSelDecMaxBlocks = 16384;  // their scores fill 64 KB

template <int D>
__global__ void __launch_bounds__(kSelDecThreads, 2)
    block_select_decode_kernel(const SelectArgs a) {
  constexpr int CH = D / 8;           // lanes per block row
  constexpr int RPW = 32 / CH;        // rows a warp reads at once
  constexpr int NW = kSelDecThreads / 32;
  constexpr int UN = 4;
  extern __shared__ float sel_smem[];  // [nblk] scores
  __shared__ float qs[D], qa[D];
  __shared__ uint32_t scratch[2 * NW];
  __shared__ uint32_t cmax_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int L = __ldg(a.seq_lens + b);
  int* out = a.sel + (size_t)bh * a.n_sel;
  if (L < 0 || L > a.Lkv) {  // uniform across the CTA
    if (tid == 0) record_error(kBadSeqLen, (unsigned)b, (unsigned)L, 0);
    for (int i = tid; i < a.n_sel; i += kSelDecThreads) out[i] = -1;
    return;
  }
  if (L == 0) {
    for (int i = tid; i < a.n_sel; i += kSelDecThreads) out[i] = -1;
    return;
  }
  const SelRange r = sel_range((L - 1) / kSelBlock, a.n_sel, a.n_first,
                               a.n_local);
  const __nv_bfloat16* q =
      a.q + ((size_t)b * a.Hkv + h) * (size_t)a.G * D;  // G rows of D
  if (tid == 0) cmax_s = 0u;
  if (tid < D) {
    float x = 0.f, y = 0.f;
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) {
      const float z = __bfloat162float(q[(size_t)g * D + tid]);
      x += z;
      y += fabsf(z);
    }
    qs[tid] = x;
    qa[tid] = y;
  }
  __syncthreads();
  const int n = r.m1 - r.f;
  const __nv_bfloat16* c0 = a.means + (size_t)bh * a.nblk * D;
  if (r.k > 0 && r.k < n) {
    const int chunk = lane % CH, rl = lane / CH;
    float qr[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) qr[x] = qs[chunk * 8 + x];
    float cm = 0.f;
    for (int i0 = warp * RPW * UN; i0 < n; i0 += NW * RPW * UN) {
      uint4 w[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int i = i0 + u * RPW + rl;
        w[u] = i < n ? __ldg(reinterpret_cast<const uint4*>(
                                 c0 + (size_t)(r.f + i) * D) + chunk)
                     : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const uint32_t ww[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        float dot = 0.f, nn = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float lo = bf16lo(ww[x]), hi = bf16hi(ww[x]);
          dot = fmaf(qr[2 * x], lo, dot);
          dot = fmaf(qr[2 * x + 1], hi, dot);
          nn = fmaf(lo * kNormUp, lo * kNormUp, nn);
          nn = fmaf(hi * kNormUp, hi * kNormUp, nn);
        }
#pragma unroll
        for (int o = CH / 2; o; o >>= 1) {
          dot += __shfl_xor_sync(~0u, dot, o);
          nn += __shfl_xor_sync(~0u, nn, o);
        }
        const int i = i0 + u * RPW + rl;
        if (i < n && chunk == 0) {
          sel_smem[i] = isnan(dot) ? -INFINITY : dot;
        }
        // (a NaN's bits compare above every number's)
        cm = __uint_as_float(max(__float_as_uint(cm), __float_as_uint(fabsf(nn))));
      }
    }
    const uint32_t cw = __reduce_max_sync(~0u, __float_as_uint(cm));
    if (lane == 0) atomicMax(&cmax_s, cw);
  }
  __syncthreads();
  float eps = 0.f;
  if (r.k > 0 && r.k < n) {
    float qq = 0.f;
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      const float y = qa[lane + 32 * x];
      qq = fmaf(y * kNormUp, y * kNormUp, y > 0.f ? qq + kNormFloor : qq);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) qq += __shfl_xor_sync(~0u, qq, o);
    eps = score_eps(kSelEpsFma * (sqrtf(qq) * kNormDown),
                    sqrtf(floor_norm<kSelDecThreads>(
                        cmax_s, c0 + (size_t)r.f * D, n * CH)) * kNormDown);
  }
  double qd[D / 32];
  bool have_q = false;
  const RowTask task = {sel_smem, out + r.f, r.f, n, r.k, eps};
  auto exact = [&](int j) {
    if (!have_q) {
      have_q = true;
#pragma unroll
      for (int x = 0; x < D / 32; ++x) {
        qd[x] = 0.0;
        for (int gg = 0; gg < a.G; ++gg)
          qd[x] += (double)__bfloat162float(
              q[(size_t)gg * D + lane * (D / 32) + x]);
      }
    }
    return exact_score<D>(qd, c0 + (size_t)j * D);
  };
  // Up to 1024 blocks (65536 tokens) one warp selects: its reductions cost an
  // instruction where the CTA's cost a barrier (batch 32 x 8 KV heads at 64K:
  // 31 us against 33; at 128K one warp takes 54 us, the CTA 47).  The other
  // warps are done.
  __shared__ int by_cta;
  if (warp == 0) {
    WarpGroup wg;
    bool todo = fill_fixed(wg, r, a.n_sel, out);
    if (todo && eps < INFINITY) {
      if (n <= 256) todo = !take_row<8>(task, exact);
      else if (n <= 512) todo = !take_row<16>(task, exact);
      else if (n <= 1024) todo = !take_row<0>(task, exact);
    }
    if (lane == 0) by_cta = todo;
  }
  __syncthreads();
  if (!by_cta) return;
  CtaGroup<kSelDecThreads> g(scratch);
  take_general(g, sel_smem, task, exact);
}

template <int D>
cudaError_t launch_block_select_decode(const SelectArgs& a, int B, int nblk,
                                       cudaStream_t st) {
  const int smem = nblk * 4;
  // (the limit is the function's, shared by every thread of the process: the
  // same for all calls, so that none takes back what another relies on)
  cudaError_t e = cudaFuncSetAttribute(
      block_select_decode_kernel<D>,
      cudaFuncAttributeMaxDynamicSharedMemorySize, kSelDecMaxBlocks * 4);
  if (e != cudaSuccess) return e;
  block_select_decode_kernel<D>
      <<<(unsigned)(B * a.Hkv), kSelDecThreads, smem, st>>>(a);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Every row of a prompt: a CTA of 8 warps takes 16 rows of one KV head.  The
// head sums are split into two bf16 parts (16 bits of each sum) and scored
// against the means on the tensor core (mma.sync: 2 d deep, far from its
// limit, and the scores land in registers, one shared-memory store away from
// the selection); all scores of the rows stay in shared memory, then each warp
// selects for two of them.  What bounds it is the selection's instructions,
// so what counts is warps to hide their latency: 16 rows take 57 KB at 16K
// keys, three CTAs per SM (32 heads on 8 at 16K: 201 us.  When this was chosen
// 215; 32 rows, two CTAs, 223; 64 rows, one, 336.  B 2, 777 rows on 5K keys:
// 12.1, 19.8, 19.8).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 16-byte asynchronous copy; zeros when !valid (nothing is read then).
__device__ __forceinline__ void cp_async_16(void* dst_smem, const void* src,
                                            bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   smem_u32(dst_smem)),
               "l"(src), "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_but_one() {
  asm volatile("cp.async.wait_group 1;" ::: "memory");
}

constexpr int kSelRows = 16;  // rows per CTA
constexpr int kSelPromptMaxBlocks = 2048;  // 16 rows' scores fill 128 KB

template <int D>
struct SelectCfg {
  static constexpr int TM = kSelRows;
  static constexpr int QROW = 2 * D * 2;  // hi and lo halves of a row, bytes
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_C = OFF_Q + TM * QROW;       // [2][64][D] bf16
  static constexpr int CBYTES = kSelBlock * D * 2;
  static constexpr int OFF_N = OFF_C + 2 * CBYTES;      // f32 [TM] |w|
  static constexpr int OFF_CM = OFF_N + TM * 4;
  static constexpr int OFF_S = (OFF_CM + 4 + 127) / 128 * 128;
  static constexpr int smem(int ld) { return OFF_S + TM * ld * 4; }
};

template <int D>
__global__ void __launch_bounds__(256, 3)
    block_select_kernel(const SelectArgs a) {
  using C = SelectCfg<D>;
  constexpr int TM = kSelRows;
  constexpr int CH = D / 8;
  constexpr int KST = D / 16;
  extern __shared__ __align__(128) uint8_t sel_raw[];
  uint8_t* sq = sel_raw + C::OFF_Q;
  uint8_t* sc = sel_raw + C::OFF_C;
  float* nrm = reinterpret_cast<float*>(sel_raw + C::OFF_N);
  uint32_t* cmax_s = reinterpret_cast<uint32_t*>(sel_raw + C::OFF_CM);
  float* S = reinterpret_cast<float*>(sel_raw + C::OFF_S);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nbh = gridDim.x / a.ntile;
  const int tile = a.ntile - 1 - (int)(blockIdx.x / nbh);  // longest first
  const int bh = blockIdx.x % nbh;
  const int b = bh / a.Hkv, h = bh - b * a.Hkv;
  const int row0 = tile * TM;
  const int nrow = min(TM, a.Lq - row0);
  const int off = a.causal ? a.Lkv - a.Lq : 0;
  // blocks any row of the tile may score
  const int key_end = a.causal ? row0 + nrow - 1 + off : a.Lkv - 1;
  const int ncand = key_end / kSelBlock + 1 - a.n_local;
  const int nct = ncand > 0 ? (ncand + kSelBlock - 1) / kSelBlock : 0;
  const __nv_bfloat16* c0 = a.means + (size_t)bh * a.nblk * D;
  if (tid == 0) *cmax_s = 0u;

  auto load_c = [&](int ct) {
    uint8_t* dst = sc + (ct & 1) * C::CBYTES;
    for (int e = tid; e < kSelBlock * CH; e += 256) {
      const int row = e / CH, ch = e % CH;
      const int j = ct * kSelBlock + row;
      const bool ok = j < a.nblk;
      cp_async_16(dst + row * (D * 2) + ((ch ^ (row & 7)) << 4),
                  c0 + (size_t)(ok ? j : 0) * D + ch * 8, ok);
    }
    cp_async_commit();
  };
  if (nct > 0) load_c(0);
  // head sums of the TM rows: 8 columns per thread and row
  {
    const __nv_bfloat16* q0 =
        a.q + ((size_t)b * a.Hkv + h) * (size_t)a.G * a.Lq * D;
    const float head_eps =
        (float)(a.G - 1) * 5.9604644775390625e-08f * kNormUp;  // 2^-24, scaled
    for (int e = tid; e < TM * CH; e += 256) {
      const int row = e / CH, ch = e % CH;
      float x[8], y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = y[i] = 0.f;
      if (row < nrow) {
        const uint4* src = reinterpret_cast<const uint4*>(
                               q0 + (size_t)(row0 + row) * D) + ch;
        const size_t hs = (size_t)a.Lq * CH;  // 16-byte chunks per head
#pragma unroll 4
        for (int g = 0; g < a.G; ++g) {
          const uint4 w = __ldg(src + g * hs);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = bf16lo(ww[i]), hi = bf16hi(ww[i]);
            x[2 * i] += lo;
            x[2 * i + 1] += hi;
            y[2 * i] += fabsf(lo);
            y[2 * i + 1] += fabsf(hi);
          }
        }
      }
      uint32_t ph[4], pl[4];
      float nn = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ph[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
        pl[i] = pack_bf16x2(x[2 * i] - bf16lo(ph[i]),
                            x[2 * i + 1] - bf16hi(ph[i]));
        // the error of these two columns, see kSelEpsMma, scaled
        const float r0 = fabsf(x[2 * i] - bf16lo(ph[i]) - bf16lo(pl[i]));
        const float r1 = fabsf(x[2 * i + 1] - bf16hi(ph[i]) - bf16hi(pl[i]));
        const float w0 = fmaf(kSelEpsMma<D> * kNormUp, fabsf(x[2 * i]),
                              fmaf(head_eps, y[2 * i], r0 * kNormUp));
        const float w1 = fmaf(kSelEpsMma<D> * kNormUp, fabsf(x[2 * i + 1]),
                              fmaf(head_eps, y[2 * i + 1], r1 * kNormUp));
        nn = fmaf(w0, w0, nn);
        nn = fmaf(w1, w1, nn);
        if (y[2 * i] > 0.f || y[2 * i + 1] > 0.f) nn += kNormFloor;
      }
      uint8_t* dst = sq + row * C::QROW;
      *reinterpret_cast<uint4*>(dst + ((ch ^ (row & 7)) << 4)) =
          make_uint4(ph[0], ph[1], ph[2], ph[3]);
      *reinterpret_cast<uint4*>(dst + (((ch + CH) ^ (row & 7)) << 4)) =
          make_uint4(pl[0], pl[1], pl[2], pl[3]);
#pragma unroll
      for (int o = CH / 2; o; o >>= 1) nn += __shfl_xor_sync(~0u, nn, o);
      if (ch == 0) nrm[row] = sqrtf(nn) * kNormDown;
    }
  }
  __syncthreads();
  // each warp scores all rows against 8 of a tile's 64 blocks
  const int mi = lane >> 3, mr = lane & 7;
  uint32_t ah[KST][4], al[KST][4];
  {
    const int row = (mi & 1) * 8 + mr;
    const uint32_t base = smem_u32(sq) + row * C::QROW;
#pragma unroll
    for (int ks = 0; ks < KST; ++ks) {
      const int ch = 2 * ks + (mi >> 1);
      ldsm_x4(base + ((ch ^ (row & 7)) << 4), ah[ks][0], ah[ks][1], ah[ks][2],
              ah[ks][3]);
      ldsm_x4(base + (((ch + CH) ^ (row & 7)) << 4), al[ks][0], al[ks][1],
              al[ks][2], al[ks][3]);
    }
  }
  for (int ct = 0; ct < nct; ++ct) {
    if (ct + 1 < nct) {
      load_c(ct + 1);
      cp_async_wait_but_one();
    } else {
      cp_async_wait_all();
    }
    __syncthreads();
    const uint32_t ca = smem_u32(sc + (ct & 1) * C::CBYTES);
    // The scores, and the largest |c|^2 among the tile's blocks: the diagonal
    // of c c^T (a row-major A fragment of 8 rows is their B fragment).
    float acc[4] = {0.f, 0.f, 0.f, 0.f}, low[4] = {0.f, 0.f, 0.f, 0.f};
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int p = 0; p < KST / 2; ++p) {
      const int row = warp * 8 + mr;
      uint32_t r0, r1, r2, r3;
      ldsm_x4(ca + row * (D * 2) + (((4 * p + mi) ^ (row & 7)) << 4), r0, r1, r2,
              r3);
      mma16816(acc, ah[2 * p], r0, r1);
      mma16816(low, al[2 * p], r0, r1);
      mma16816(acc, ah[2 * p + 1], r2, r3);
      mma16816(low, al[2 * p + 1], r2, r3);
      mma16816_top(d0, d1, r0, r1, r0, r1);
      mma16816_top(d0, d1, r2, r3, r2, r3);
    }
    {
      const int col = ct * kSelBlock + warp * 8 + 2 * (lane & 3);
      const int row = lane >> 2;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        acc[x] += low[x];
        if (isnan(acc[x])) acc[x] = -INFINITY;
      }
      *reinterpret_cast<float2*>(S + (size_t)row * a.ld + col) =
          make_float2(acc[0], acc[1]);
      *reinterpret_cast<float2*>(S + (size_t)(row + 8) * a.ld + col) =
          make_float2(acc[2], acc[3]);
    }
    // lane: row lane / 4, columns 2 (lane % 4) and the next
    const float nn = (lane >> 2) == 2 * (lane & 3)       ? d0
                     : (lane >> 2) == 2 * (lane & 3) + 1 ? d1
                                                         : 0.f;
    const uint32_t cw = __reduce_max_sync(~0u, __float_as_uint(fabsf(nn)));
    if (lane == 0) atomicMax(cmax_s, cw);
    __syncthreads();
  }
  const float cmax =
      sqrtf(floor_norm<256>(*cmax_s, c0, min(nct * kSelBlock, a.nblk) * CH));
  WarpGroup g;
  for (int rr = warp; rr < nrow; rr += 8) {
    const int row = row0 + rr;
    const int last = (a.causal ? row + off : a.Lkv - 1) / kSelBlock;
    const SelRange r = sel_range(last, a.n_sel, a.n_first, a.n_local);
    int* out = a.sel + ((size_t)bh * a.Lq + row) * a.n_sel;
    if (!fill_fixed(g, r, a.n_sel, out)) continue;
    float* srow = S + (size_t)rr * a.ld + r.f;
    const RowTask task = {srow, out + r.f, r.f, r.m1 - r.f, r.k,
                          score_eps(nrm[rr], cmax)};
    // the float64 score of block j
    double qd[D / 32];
    bool have_q = false;
    auto exact = [&](int j) {
      if (!have_q) {
        have_q = true;
        const __nv_bfloat16* q =
            a.q + (((size_t)b * a.Hkv + h) * a.G * (size_t)a.Lq + row) * D;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) qd[x] = 0.0;
        for (int gg = 0; gg < a.G; ++gg)
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            qd[x] += (double)__bfloat162float(
                q[(size_t)gg * a.Lq * D + lane * (D / 32) + x]);
      }
      return exact_score<D>(qd, c0 + (size_t)j * D);
    };
    bool todo = true;
    if (task.eps < INFINITY) {
      if (task.n <= 64) todo = !take_row<2>(task, exact);
      else if (task.n <= 128) todo = !take_row<4>(task, exact);
      else if (task.n <= 256) todo = !take_row<8>(task, exact);
      else if (task.n <= 512) todo = !take_row<16>(task, exact);
      else todo = !take_row<0>(task, exact);
    }
    if (todo) take_general(g, srow, task, exact);
    __syncwarp();
  }
}

// Score columns kept per row: whole 64-block tiles, plus 8 floats so that the 8
// rows a fragment store writes fall into different banks.
constexpr int select_ld(int nblk) { return (nblk + 63) / 64 * 64 + 8; }

template <int D>
cudaError_t launch_block_select(SelectArgs a, int B, cudaStream_t st) {
  a.ld = select_ld(a.nblk);
  a.ntile = (a.Lq + kSelRows - 1) / kSelRows;
  const int smem = SelectCfg<D>::smem(a.ld);
  constexpr int most = SelectCfg<D>::smem(select_ld(kSelPromptMaxBlocks));
  static_assert(most <= 232448, "shared memory per CTA");
  const long long grid = (long long)a.ntile * B * a.Hkv;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(
      block_select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
      most);  // (of all calls, as above)
  if (e != cudaSuccess) return e;
  block_select_kernel<D><<<(unsigned)grid, 256, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace blasst
