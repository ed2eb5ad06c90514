// select_bwd.cuh -- backward of the block-selected attention (select_attn.cuh)
// with the selection held fixed: the gradients of softmax attention over each
// row's selected, visible keys (d = 128),
//   D_r = dO_r . O_r;  P = exp(scale q k^T - lse) on selected pairs (else 0);
//   dV = P^T dO;  dS = P o (dO V^T - D);  dK = scale dS^T Q;  dQ = scale dS K.
//
// Two passes of tensor-core work, one per side that is summed:
//   select_dkdv_kernel  a CTA keeps one 128-key block (two selection blocks)
//                       and streams the query tiles (TQ tokens x G heads, 128
//                       rows) any of whose tokens selected either half
//   select_dq_kernel    a CTA keeps one query tile and streams the 64-key
//                       blocks its tokens selected, two a step
// One pass over the pairs would need 5 products of 128^3 for each where these
// need 4 and 3 (and 2 more for the dQ pass's accuracy, see there), but it has
// to add every pair's dQ tile (64 KB of float32) to memory: at 8K causal, 32
// heads on 8, 16 blocks a row, the additions alone cost 370 of its 1190 us,
// they leave the tensor memory no room to overlap the products with the
// threads' work, and their order changes the result from run to run.  The dQ
// pass also walks 64-key blocks, a third fewer than the 128-key pairs.  Both
// passes sum in a fixed order.  The dQ pass runs first: it corrects D.
//
// Before them:
//   select_prep_kernel   -D and -lse * log2 e per query row
//   select_lists_kernel  per tile: its blocks and their token bits, and the
//                        bits of every block, block-major
//   select_tiles_kernel  per (KV head, 128-key block): the tiles with a bit,
//                        ascending, and their bits
//   select_order_kernel  the key blocks by the length of their lists
#pragma once

#include "backward.cuh"
#include "select_attn.cuh"

namespace blasst {

struct SelBwdListArgs {
  const unsigned* bits;  // [B*Hkv][nblk2][ntile][wpt]
  int* count;        // [slots], slot = jb * (B*Hkv) + b*Hkv + hkv
  int* list;         // [slots][ntile]
  unsigned* words;   // [slots][ntile][2][wpt]
  int BH, wpt, ntile, nblk2;
};

__global__ void __launch_bounds__(128)
    select_tiles_kernel(const SelBwdListArgs a) {
  __shared__ int wsum[4];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int slot = blockIdx.x;
  const int jb = slot / a.BH;
  const int bh = slot - jb * a.BH;
  const unsigned* b0 =
      a.bits + ((size_t)bh * a.nblk2 + 2 * jb) * a.ntile * a.wpt;
  const unsigned* b1 = b0 + (size_t)a.ntile * a.wpt;
  int at = 0;
  for (int t0 = 0; t0 < a.ntile; t0 += 128) {
    const int t = t0 + tid;
    unsigned any = 0;
    if (t < a.ntile)
      for (int w = 0; w < a.wpt; ++w)
        any |= b0[(size_t)t * a.wpt + w] | b1[(size_t)t * a.wpt + w];
    const unsigned m = __ballot_sync(~0u, any != 0u);
    if (lane == 0) wsum[warp] = __popc(m);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (any) {
      const size_t pos = (size_t)slot * a.ntile + at + before +
                         __popc(m & ((1u << lane) - 1u));
      a.list[pos] = t;
      for (int w = 0; w < a.wpt; ++w) {
        a.words[pos * 2 * a.wpt + w] = b0[(size_t)t * a.wpt + w];
        a.words[pos * 2 * a.wpt + a.wpt + w] = b1[(size_t)t * a.wpt + w];
      }
    }
    at += total;
    __syncthreads();
  }
  if (tid == 0) a.count[slot] = at;
}

// order[rank of slot s] = s, rank = slots with more tiles, or as many and a
// lower index: a permutation of 0 .. n-1, the longest lists first.  A warp per
// slot.
__global__ void __launch_bounds__(256)
    select_order_kernel(const int* count, int n, int* order) {
  const int s = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (s >= n) return;
  const int cs = __ldg(count + s);
  int rank = 0;
#pragma unroll 4
  for (int u = lane; u < n; u += 32) {
    const int cu = __ldg(count + u);
    rank += (cu > cs) || (cu == cs && u < s);
  }
  rank = (int)__reduce_add_sync(0xffffffffu, (unsigned)rank);
  if (lane == 0) order[rank] = s;
}

struct __align__(64) SelBwdParams {
  CUtensorMap tq, tdo;        // query tiles (TQ tokens x G heads)
  CUtensorMap tk, tv;         // box 64 rows
  CUtensorMap tdel, tlse2;    // those rows' -D and -lse * log2 e
  const __nv_bfloat16* o;     // [B, Hq, Lq, D]
  const __nv_bfloat16* dout;  // [B, Hq, Lq, D]
  const float* lse;           // [B, Hq, Lq] natural log
  float* delta;               // [B*Hq][Lqp] -D
  float* lse2;                // [B*Hq][Lqp] -lse * log2 e
  __nv_bfloat16* dq;          // [B, Hq, Lq, D]
  __nv_bfloat16* dk;          // [B, Hkv, Lkv, D]
  __nv_bfloat16* dv;          // [B, Hkv, Lkv, D]
  // dK, dV pass: the tiles of each key block
  const int* order;           // slot of each CTA
  const int* count;
  const int* tlist;
  const unsigned* twords;
  // dQ pass: the blocks of each tile (select_lists_kernel)
  const int* nstep;
  const unsigned* list;
  const unsigned* words;
  int B, Hq, Hkv, Lq, Lqp, Lkv, G, causal;
  int TQ, wpt, ntile, cap;
  unsigned rep;  // repeats a TQ-bit word over 32 bits (TQ < 32), else 1
  float scale;
};

// D_r = sum_e dO_re O_re (f32).  Half a warp per query row, 16 bytes per lane,
// 4 rows in flight per half warp: bound by reading o and dout once.
constexpr int kSelPrepRows = 64;  // per CTA of 256 threads
__global__ void __launch_bounds__(256)
    select_prep_kernel(const __grid_constant__ SelBwdParams p) {
  const long long rows = (long long)p.B * p.Hq * p.Lq;
  const int sub = threadIdx.x & 15;
  const long long row0 =
      (long long)blockIdx.x * kSelPrepRows + (threadIdx.x >> 4);
  uint4 a[4], g[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long row = row0 + 16 * i;
    if (row < rows) {
      a[i] = __ldg(reinterpret_cast<const uint4*>(p.o + row * kBwdD) + sub);
      g[i] = __ldg(reinterpret_cast<const uint4*>(p.dout + row * kBwdD) + sub);
    } else {
      a[i] = g[i] = make_uint4(0, 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const long long row = row0 + 16 * i;
    const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
    const uint32_t y[4] = {g[i].x, g[i].y, g[i].z, g[i].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(bf16lo(x[e]), bf16lo(y[e]), s);
      s = fmaf(bf16hi(x[e]), bf16hi(y[e]), s);
    }
#pragma unroll
    for (int m = 8; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (sub == 0 && row < rows) {
      const long long r = row / p.Lq, q = row - r * p.Lq;
      p.delta[r * p.Lqp + q] = -s;
      p.lse2[r * p.Lqp + q] = -p.lse[row] * kPrefLog2e;
      if (q == p.Lq - 1)  // the row's padding columns: finite, never used
        for (int c = p.Lq; c < p.Lqp; ++c) {
          p.delta[r * p.Lqp + c] = 0.f;
          p.lse2[r * p.Lqp + c] = 0.f;
        }
    }
  }
}

constexpr int kSelNumSm = 148;  // one CTA of either pass per SM
constexpr int kSelBwdThreads = 64 + 256;  // producer, issuer, 8 compute warps

// ---------------------------------------------------------------------------
// dK, dV.  Per tile four products, transposed so that a thread is a key row:
//   S^T  = K_j Q_i^T   -> TMEM [0, 128)      dV += P^T dO_i  -> [256, 384)
//   dP^T = V_j dO_i^T  -> [128, 256)         dK += dS^T Q_i  -> [384, 512)
// P^T and dS^T are the A operands of the second column, written as bf16 over
// the scores they come from.  The issuer's order is
//   [P_n written] dV_n, S^T_{n+1}   [dS_n written] dK_n, dP^T_{n+1}
// so that the threads' dS_n overlaps dV_n and S^T_{n+1}, and their P_{n+1}
// overlaps dK_n and dP^T_{n+1}.  8K causal, 32 heads on 8, 16 blocks a row
// (38.6k pairs): 0.53 ms, the tensor pipe 58% busy; what bounds a pair is the
// hand-offs between its products and the threads' two phases.
// ---------------------------------------------------------------------------
template <bool V>
struct BoolTag {
  static constexpr bool value = V;
};

struct SelDkdvCfg {
  static constexpr int TILE = 128 * kBwdD * 2;  // 32 KB, two 64-column boxes
  static constexpr int BOX = 128 * 128;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + TILE;
  static constexpr int OFF_Q = OFF_V + TILE;        // [2]
  static constexpr int OFF_DO = OFF_Q + 2 * TILE;   // [2]
  static constexpr int OFF_LSE = OFF_DO + 2 * TILE;  // f32 [2][128]
  static constexpr int OFF_DEL = OFF_LSE + 2 * 512;  // f32 [2][128]
  static constexpr int OFF_BAR = OFF_DEL + 2 * 512;
  static constexpr int B_KV = 0;
  static constexpr int B_QF = 1;   // [2] a tile's Q, dO, lse and D
  static constexpr int B_QE = 3;   // [2] that slot free
  static constexpr int B_SF = 5;   // S^T in TMEM
  static constexpr int B_DPF = 6;  // dP^T in TMEM
  static constexpr int B_PR = 7;   // P^T written (one arrival per warp)
  static constexpr int B_DSR = 8;  // dS^T written (one arrival per warp)
  static constexpr int B_OD = 9;   // every product complete
  static constexpr int B_DR = 10;  // drain after a wait gave up
  static constexpr int NBAR = 11;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_TMEM + 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static_assert(SMEM_ALLOC <= 232448, "shared memory per CTA");
};

__global__ void __launch_bounds__(kSelBwdThreads, 1)
    select_dkdv_kernel(const __grid_constant__ SelBwdParams p) {
  using C = SelDkdvCfg;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nbk = p.B * p.Hkv;
  const int slot = p.order ? __ldg(p.order + blockIdx.x) : (int)blockIdx.x;
  const int jb = slot / nbk;       // key block
  const int bk = slot - jb * nbk;  // b * Hkv + hkv
  const int b = bk / p.Hkv;
  const int hkv = bk - b * p.Hkv;
  const int zq = b * p.Hq + hkv * p.G;
  const int off = p.Lkv - p.Lq;
  const int nt = __ldg(p.count + slot);
  const int* tlist = p.tlist + (size_t)slot * p.ntile;

  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  if (threadIdx.x == 0) {
    mbar_init(&bar[C::B_KV], 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar[C::B_QF + s], 1);
      mbar_init(&bar[C::B_QE + s], 1);
    }
    mbar_init(&bar[C::B_SF], 1);
    mbar_init(&bar[C::B_DPF], 1);
    mbar_init(&bar[C::B_PR], 8);
    mbar_init(&bar[C::B_DSR], 8);
    mbar_init(&bar[C::B_OD], 1);
    mbar_init(&bar[C::B_DR], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0 && nt > 0) {
      const uint64_t pol_kv = policy_evict_first();
      const uint64_t pol_q = policy_evict_last();
      mbar_arrive_expect_tx(&bar[C::B_KV], 2 * C::TILE);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int at = c * C::BOX + h * (C::BOX / 2);
          tma_load_3d(smem + C::OFF_K + at, &p.tk, &bar[C::B_KV], c * 64,
                      jb * 128 + h * 64, bk, pol_kv);
          tma_load_3d(smem + C::OFF_V + at, &p.tv, &bar[C::B_KV], c * 64,
                      jb * 128 + h * 64, bk, pol_kv);
        }
      int next = __ldg(tlist), n = 0;
      for (; n < nt; ++n) {
        const int r0 = next * p.TQ;
        if (n + 1 < nt) next = __ldg(tlist + n + 1);
        const int s = n & 1;
        if (n >= 2 && !mbar_wait(&bar[C::B_QE + s], ((n >> 1) - 1) & 1,
                                 kWaitSelect, n, 500 + s))
          break;
        mbar_arrive_expect_tx(&bar[C::B_QF + s], 2 * C::TILE + 1024);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tma_load_3d(smem + C::OFF_Q + s * C::TILE + c * C::BOX, &p.tq,
                      &bar[C::B_QF + s], c * 64, r0, zq, pol_q);
        tma_load_3d(smem + C::OFF_LSE + s * 512, &p.tlse2, &bar[C::B_QF + s],
                    r0, zq, 0, pol_q);
#pragma unroll
        for (int c = 0; c < 2; ++c)
          tma_load_3d(smem + C::OFF_DO + s * C::TILE + c * C::BOX, &p.tdo,
                      &bar[C::B_QF + s], c * 64, r0, zq, pol_q);
        tma_load_3d(smem + C::OFF_DEL + s * 512, &p.tdel, &bar[C::B_QF + s],
                    r0, zq, 0, pol_q);
      }
      // no copy is left in flight, whatever became of its readers
      drain_ring(&bar[C::B_QF], 2, n);
      mbar_wait(&bar[C::B_KV], 0, kWaitSelect, n, 502);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t id_kk = idesc_bf16(128, 128, 0, 0);  // K-major A, B
    constexpr uint32_t id_km = idesc_bf16(128, 128, 0, 1);  // B MN-major
    // K-major operands step 32 bytes in a box, boxes C::BOX apart; MN-major
    // ones 16 rows of 128 bytes
    const uint64_t dK = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
    const uint64_t dV = smem_desc(smem_u32(smem + C::OFF_V), 16, 1024, 2);
    const uint64_t dQk = smem_desc(smem_u32(smem + C::OFF_Q), 16, 1024, 2);
    const uint64_t dOk = smem_desc(smem_u32(smem + C::OFF_DO), 16, 1024, 2);
    const uint64_t dQm = smem_desc(smem_u32(smem + C::OFF_Q), C::BOX, 1024, 2);
    const uint64_t dOm = smem_desc(smem_u32(smem + C::OFF_DO), C::BOX, 1024, 2);
    // D[128 x 128] = A B^T, both K-major in shared memory
    auto mm_ss = [&](uint32_t d, uint64_t a0, uint64_t b0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t st = (uint64_t)(((k >> 2) * C::BOX + (k & 3) * 32) >> 4);
        mma_ss_elect(d, a0 + st, b0 + st, id_kk, k > 0 ? 1u : 0u);
      }
    };
    // D += A B, A bf16 in tensor memory: step k is 8 columns, steps 4 .. 7
    // 64 columns on (each compute group writes at the start of its half)
    auto mm_ts = [&](uint32_t d, uint32_t a0, uint64_t b0, bool first) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_ts_elect(d, a0 + (k >> 2) * 64 + (k & 3) * 8,
                     b0 + (uint64_t)((k * 2048) >> 4), id_km,
                     (first && k == 0) ? 0u : 1u);
    };
    const uint64_t slot_step = (uint64_t)(C::TILE >> 4);
    bool ok = true;
    auto wait = [&](int id, int parity, int step, int what) {
      const bool w = ok && mbar_wait(&bar[id], parity, kWaitSelect, step, what);
      ok = __all_sync(FULL, w);
    };
    if (nt > 0) {
      wait(C::B_KV, 0, 0, 510);
      wait(C::B_QF, 0, 0, 511);
      if (ok) {
        tc_fence_after();
        mm_ss(tmem, dK, dQk);
        mma_commit_elect(&bar[C::B_SF]);
        mm_ss(tmem + 128, dV, dOk);
        mma_commit_elect(&bar[C::B_DPF]);
      }
      for (int n = 0; n < nt && ok; ++n) {
        const uint64_t s = (n & 1) ? slot_step : 0;
        const uint64_t s1 = (n & 1) ? 0 : slot_step;
        const bool more = n + 1 < nt;
        wait(C::B_PR, n & 1, n, 512);
        if (more) wait(C::B_QF + ((n + 1) & 1), ((n + 1) >> 1) & 1, n, 513);
        if (!ok) break;
        tc_fence_after();
        mm_ts(tmem + 256, tmem, dOm + s, n == 0);
        if (more) {
          mm_ss(tmem, dK, dQk + s1);
          mma_commit_elect(&bar[C::B_SF]);
        }
        wait(C::B_DSR, n & 1, n, 514);
        if (!ok) break;
        tc_fence_after();
        mm_ts(tmem + 384, tmem + 128, dQm + s, n == 0);
        mma_commit_elect(&bar[C::B_QE + (n & 1)]);
        if (more) {
          mm_ss(tmem + 128, dV, dOk + s1);
          mma_commit_elect(&bar[C::B_DPF]);
        }
      }
      if (ok)
        mma_commit_elect(&bar[C::B_OD]);
      else
        drain_mma(&bar[C::B_DR]);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- threads
    // Warps 2..5 take query columns 0 .. 63 of a tile, warps 6..9 the rest.
    const int wg = (warp - 2) >> 2;
    const int quad = warp & 3;
    const int rr = quad * 32 + lane;  // TMEM lane: key row of the block
    const uint32_t lane_base =
        tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(wg * 64);
    const int key = jb * 128 + rr;
    const bool key_ok = key < p.Lkv;
    const float sl2 = p.scale * kPrefLog2e;
    const unsigned* wp = p.twords + ((size_t)slot * p.ntile * 2 + (rr >> 6)) *
                                        (size_t)p.wpt;
    const int w0 = (2 * wg) & (p.wpt - 1), w1 = (2 * wg + 1) & (p.wpt - 1);
    bool ok = true;
    // A V row with an infinity or NaN makes its dP so everywhere: where one of
    // the warp's rows has any, dS of hidden entries is set to 0 (a key that
    // nobody selected has no gradient, whatever it holds).
    bool odd_v = false;
    if (nt > 0) {
      const bool w = mbar_wait(&bar[C::B_KV], 0, kWaitSelect, 0, 519);
      ok = __all_sync(FULL, w);
      bool odd = false;
#pragma unroll 4
      for (int e = 0; e < 16; ++e) {
        const uint4 x = *reinterpret_cast<const uint4*>(
            smem + C::OFF_V + (e >> 3) * C::BOX + rr * 128 + (e & 7) * 16);
        const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          odd |= (y[i] & 0x7f800000u) == 0x7f800000u ||
                 (y[i] & 0x7f80u) == 0x7f80u;
      }
      odd_v = __any_sync(FULL, odd);
    }
    // P of a tile from its P phase to its dS phase, float32: a weight far below
    // its row's largest still gives its key a gradient, and the bf16 rounding
    // of dS is the only one that counts.  (Half the registers would hold it as
    // bf16 or fp16: fp16 loses the weights below 3e-8, bf16 adds an error as
    // large as that rounding.)
    float pf[64];
    unsigned m_n[2] = {0u, 0u};  // next tile's token bits
    int t_n = 0;                 // and the tile
    if (nt > 0) {
      t_n = __ldg(tlist);
      m_n[0] = __ldg(wp + w0);
      m_n[1] = __ldg(wp + w1);
    }
    for (int n = 0; n < nt; ++n) {
      // one bit per query column: the token bits of this key's half of the
      // block, cut at the first token that sees the key
      unsigned cm[2];
      {
        const int t0 = p.causal ? key - off - t_n * p.TQ : 0;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int sh = t0 - (u ? w1 : w0) * 32;
          const unsigned see = sh <= 0 ? ~0u : sh >= 32 ? 0u : ~0u << sh;
          cm[u] = key_ok ? (m_n[u] & see) * p.rep : 0u;
        }
      }
      if (n + 1 < nt) {
        t_n = __ldg(tlist + n + 1);
        m_n[0] = __ldg(wp + (size_t)(n + 1) * 2 * p.wpt + w0);
        m_n[1] = __ldg(wp + (size_t)(n + 1) * 2 * p.wpt + w1);
      }
      const int s = n & 1;
      const float4* lse4 = reinterpret_cast<const float4*>(
          smem + C::OFF_LSE + s * 512 + wg * 256);
      const float4* del4 = reinterpret_cast<const float4*>(
          smem + C::OFF_DEL + s * 512 + wg * 256);
      // the tile's lse and D came with its Q (visible to this thread once it
      // has seen the barrier itself)
      bool w = ok && mbar_wait(&bar[C::B_QF + s], (n >> 1) & 1, kWaitSelect, n,
                               520) &&
               mbar_wait(&bar[C::B_SF], n & 1, kWaitSelect, n, 521);
      ok = __all_sync(FULL, w);
      if (!ok) break;
      tc_fence_after();
      // ---- P^T
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t sv[32], st[16];
        tmem_ld32(lane_base + u * 32, sv);
        tc_wait_ld();
        if (__all_sync(FULL, cm[u] == ~0u)) {
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 l4 = lse4[u * 8 + (x >> 2)];
            float p0, p1, p2, p3;
            fma2v(p0, p1, __uint_as_float(sv[x]), __uint_as_float(sv[x + 1]),
                  sl2, l4.x, l4.y);
            fma2v(p2, p3, __uint_as_float(sv[x + 2]), __uint_as_float(sv[x + 3]),
                  sl2, l4.z, l4.w);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            p2 = ex2_approx(p2);
            p3 = ex2_approx(p3);
            st[x >> 1] = pack_bf16x2(p0, p1);
            st[(x >> 1) + 1] = pack_bf16x2(p2, p3);
            pf[u * 32 + x] = p0;
            pf[u * 32 + x + 1] = p1;
            pf[u * 32 + x + 2] = p2;
            pf[u * 32 + x + 3] = p3;
          }
        } else {
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 l4 = lse4[u * 8 + (x >> 2)];
            float* pv = pf + u * 32 + x;
            fma2v(pv[0], pv[1], __uint_as_float(sv[x]), __uint_as_float(sv[x + 1]),
                  sl2, l4.x, l4.y);
            fma2v(pv[2], pv[3], __uint_as_float(sv[x + 2]),
                  __uint_as_float(sv[x + 3]), sl2, l4.z, l4.w);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pv[e] = (cm[u] >> (x + e)) & 1u ? ex2_approx(pv[e]) : 0.f;
            st[x >> 1] = pack_bf16x2(pv[0], pv[1]);
            st[(x >> 1) + 1] = pack_bf16x2(pv[2], pv[3]);
          }
        }
        tmem_st16(lane_base + u * 16, st);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_PR]);
      // ---- dS^T = P^T o (dP^T - D)
      w = mbar_wait(&bar[C::B_DPF], n & 1, kWaitSelect, n, 522);
      ok = __all_sync(FULL, w);
      if (!ok) break;
      tc_fence_after();
      auto d_phase = [&](auto hide) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t dp[32], st[16];
          tmem_ld32(lane_base + 128 + u * 32, dp);
          tc_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            const float4 d4 = del4[u * 8 + (x >> 2)];
            const float* pv = pf + u * 32 + x;
            float ds[4];
            add_mul2(ds[0], ds[1], pv[0], pv[1], __uint_as_float(dp[x]),
                     __uint_as_float(dp[x + 1]), d4.x, d4.y);
            add_mul2(ds[2], ds[3], pv[2], pv[3], __uint_as_float(dp[x + 2]),
                     __uint_as_float(dp[x + 3]), d4.z, d4.w);
            if constexpr (decltype(hide)::value) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                ds[e] = (cm[u] >> (x + e)) & 1u ? ds[e] : 0.f;
            }
            st[x >> 1] = pack_bf16x2(ds[0], ds[1]);
            st[(x >> 1) + 1] = pack_bf16x2(ds[2], ds[3]);
          }
          tmem_st16(lane_base + 128 + u * 16, st);
        }
      };
      if (odd_v)  // warp-uniform
        d_phase(BoolTag<true>());
      else
        d_phase(BoolTag<false>());
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_DSR]);
    }
    // dV (first group) and dK (second) of the block; zero when no tile
    // selected it
    if (ok && nt > 0) {
      const bool w = mbar_wait(&bar[C::B_OD], 0, kWaitSelect, nt, 523);
      ok = __all_sync(FULL, w);
      tc_fence_after();
    }
    if (ok) {
      const uint32_t col = tmem + ((uint32_t)(quad * 32) << 16) + (wg ? 384 : 256);
      const float f = wg ? p.scale : 1.f;
      __nv_bfloat16* out =
          (wg ? p.dk : p.dv) + ((size_t)bk * p.Lkv + key) * kBwdD;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t a[32];
        if (nt > 0) {  // (warp-collective: every lane loads, the rows store)
          tmem_ld32(col + cc * 32, a);
          tc_wait_ld();
        } else {
#pragma unroll
          for (int x = 0; x < 32; ++x) a[x] = 0u;
        }
        if (key_ok) {
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(a[x]) * f, __uint_as_float(a[x + 1]) * f);
            w.y = pack_bf16x2(__uint_as_float(a[x + 2]) * f, __uint_as_float(a[x + 3]) * f);
            w.z = pack_bf16x2(__uint_as_float(a[x + 4]) * f, __uint_as_float(a[x + 5]) * f);
            w.w = pack_bf16x2(__uint_as_float(a[x + 6]) * f, __uint_as_float(a[x + 7]) * f);
            *reinterpret_cast<uint4*>(out + cc * 32 + x) = w;
          }
        }
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

// ---------------------------------------------------------------------------
// dQ.  Per step of two 64-key blocks five products, a thread is a query row:
//   S = Q K_s^T -> TMEM [0, 128)    dP = dO V_s^T -> [128, 256)
//   dQ += dS K_s -> [256, 384)      M += P K_s -> [384, 512)
// The gradient is scale sum_c dS_c k_c, and two roundings in it are large
// beside that of the result (2^-9 of it on average): dS as one bf16 operand
// (as much again), and D = dO . o from the bf16 o, whose error dD adds
// dD sum_c P_c k_c to a row.  So dS goes in as two bf16 parts (two of the five
// products), and the row sum of dS, 0 with the right D, gives dD: it is
// subtracted with M at the end, and the dK, dV pass behind this one gets the
// corrected D.  dQ's error is then its rounding, 0.0017 of its norm, where it
// was 0.0028 to 0.0038, the more the fewer keys a row has.  P and dS are the A operands, written over
// the S and dP they come from.  The issuer's order is
//   [P_s written] M_s, S_{s+1}   [dS_s written] dQ_s, dP_{s+1}
// so that the threads' dS_s overlaps M_s and S_{s+1}, and their P_{s+1}
// overlaps dQ_s and dP_{s+1}.  K_s is needed until dQ_s: three K slots, two V
// slots.  The same 8K case (25k steps): 0.37 ms, the tensor pipe 69% busy; with
// three products (dS one part, no M) 0.27 ms at 55%.
// ---------------------------------------------------------------------------
struct SelDqCfg {
  static constexpr int TILE = 128 * kBwdD * 2;
  static constexpr int BOX = 128 * 128;
  static constexpr int NKS = 3, NVS = 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_DO = OFF_Q + TILE;
  static constexpr int OFF_K = OFF_DO + TILE;
  static constexpr int OFF_V = OFF_K + NKS * TILE;
  static constexpr int OFF_R = OFF_V + NVS * TILE;  // f32 [2][128] sums of dS
  static constexpr int OFF_BAR = OFF_R + 2 * 128 * 4;
  static constexpr int B_Q = 0;
  static constexpr int B_KF = 1;           // [3]
  static constexpr int B_KE = B_KF + NKS;  // [3]
  static constexpr int B_VF = B_KE + NKS;  // [2]
  static constexpr int B_VE = B_VF + NVS;  // [2]
  static constexpr int B_SF = B_VE + NVS;  // S in TMEM
  static constexpr int B_PR = B_SF + 1;    // P written (one arrival per warp)
  static constexpr int B_DPF = B_PR + 1;   // dP in TMEM
  static constexpr int B_DSR = B_DPF + 1;  // dS written (one per warp)
  static constexpr int B_OD = B_DSR + 1;
  static constexpr int B_DR = B_OD + 1;    // drain after a wait gave up
  static constexpr int NBAR = B_DR + 1;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_TMEM + 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static_assert(SMEM_ALLOC <= 232448, "shared memory per CTA");
};

__global__ void __launch_bounds__(kSelBwdThreads, 1)
    select_dq_kernel(const __grid_constant__ SelBwdParams p) {
  using C = SelDqCfg;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // the latest tiles (the longest lists of a causal call) first
  const int nbk = p.B * p.Hkv;
  const int tile = p.ntile - 1 - (int)(blockIdx.x / nbk);
  const int bk = blockIdx.x % nbk;
  const int b = bk / p.Hkv;
  const int hkv = bk - b * p.Hkv;
  const int zq = b * p.Hq + hkv * p.G;
  const size_t slot = (size_t)bk * p.ntile + tile;
  const int ns = __ldg(p.nstep + slot);
  const uint2* list = reinterpret_cast<const uint2*>(p.list + slot * p.cap);

  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
  if (threadIdx.x == 0) {
    mbar_init(&bar[C::B_Q], 1);
    for (int i = 0; i < C::NKS; ++i) {
      mbar_init(&bar[C::B_KF + i], 1);
      mbar_init(&bar[C::B_KE + i], 1);
    }
    for (int i = 0; i < C::NVS; ++i) {
      mbar_init(&bar[C::B_VF + i], 1);
      mbar_init(&bar[C::B_VE + i], 1);
    }
    mbar_init(&bar[C::B_SF], 1);
    mbar_init(&bar[C::B_PR], 8);
    mbar_init(&bar[C::B_DPF], 1);
    mbar_init(&bar[C::B_DSR], 8);
    mbar_init(&bar[C::B_OD], 1);
    mbar_init(&bar[C::B_DR], 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ---------------------------------------------------------------- TMA
    if (lane == 0 && ns > 0) {
      const uint64_t pol_q = policy_evict_first();
      const uint64_t pol_kv = policy_evict_last();
      mbar_arrive_expect_tx(&bar[C::B_Q], 2 * C::TILE);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        tma_load_3d(smem + C::OFF_Q + c * C::BOX, &p.tq, &bar[C::B_Q], c * 64,
                    tile * p.TQ, zq, pol_q);
        tma_load_3d(smem + C::OFF_DO + c * C::BOX, &p.tdo, &bar[C::B_Q], c * 64,
                    tile * p.TQ, zq, pol_q);
      }
      auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full,
                      uint2 e) {
        mbar_arrive_expect_tx(full, C::TILE);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tma_load_3d(dst + c * C::BOX, map, full, c * 64,
                      (int)e.x * kSelBlock, bk, pol_kv);
          tma_load_3d(dst + c * C::BOX + C::BOX / 2, map, full, c * 64,
                      (int)e.y * kSelBlock, bk, pol_kv);
        }
      };
      uint2 next = __ldg(list);
      int nk = 0, nv = 0;  // loads issued
      for (int s = 0; s < ns; ++s) {
        const uint2 e = next;
        if (s + 1 < ns) next = __ldg(list + s + 1);
        const int ks = s % C::NKS, vs = s % C::NVS;
        if (s >= C::NKS && !mbar_wait(&bar[C::B_KE + ks], (s / C::NKS - 1) & 1,
                                      kWaitSelect, s, 530))
          break;
        load(&p.tk, smem + C::OFF_K + ks * C::TILE, &bar[C::B_KF + ks], e);
        ++nk;
        if (s >= C::NVS && !mbar_wait(&bar[C::B_VE + vs], (s / C::NVS - 1) & 1,
                                      kWaitSelect, s, 531))
          break;
        load(&p.tv, smem + C::OFF_V + vs * C::TILE, &bar[C::B_VF + vs], e);
        ++nv;
      }
      // no copy is left in flight, whatever became of its readers
      drain_ring(&bar[C::B_KF], C::NKS, nk);
      drain_ring(&bar[C::B_VF], C::NVS, nv);
      mbar_wait(&bar[C::B_Q], 0, kWaitSelect, nk, 532);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA
    constexpr uint32_t id_kk = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t id_km = idesc_bf16(128, 128, 0, 1);
    const uint64_t dQ = smem_desc(smem_u32(smem + C::OFF_Q), 16, 1024, 2);
    const uint64_t dO = smem_desc(smem_u32(smem + C::OFF_DO), 16, 1024, 2);
    const uint64_t dKk = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
    const uint64_t dKm = smem_desc(smem_u32(smem + C::OFF_K), C::BOX, 1024, 2);
    const uint64_t dV = smem_desc(smem_u32(smem + C::OFF_V), 16, 1024, 2);
    constexpr uint64_t kSlot = (uint64_t)(C::TILE >> 4);
    auto mm_ss = [&](uint32_t d, uint64_t a0, uint64_t b0) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint64_t st = (uint64_t)(((k >> 2) * C::BOX + (k & 3) * 32) >> 4);
        mma_ss_elect(d, a0 + st, b0 + st, id_kk, k > 0 ? 1u : 0u);
      }
    };
    bool ok = true;
    auto wait = [&](int id, int parity, int step, int what) {
      const bool w = ok && mbar_wait(&bar[id], parity, kWaitSelect, step, what);
      ok = __all_sync(FULL, w);
    };
    if (ns > 0) {
      wait(C::B_Q, 0, 0, 540);
      wait(C::B_KF, 0, 0, 541);
      if (ok) {
        tc_fence_after();
        mm_ss(tmem, dQ, dKk);
        mma_commit_elect(&bar[C::B_SF]);
      }
      wait(C::B_VF, 0, 0, 542);
      if (ok) {
        tc_fence_after();
        mm_ss(tmem + 128, dO, dV);
        mma_commit_elect(&bar[C::B_DPF]);
        mma_commit_elect(&bar[C::B_VE]);
      }
      // D += A B, A 128 keys of bf16 in tensor memory: step k is 8 columns,
      // steps 4 .. 7 64 columns on (block h of a step's two writes at 64 h)
      auto mm_ts = [&](uint32_t d, uint32_t a0, uint64_t b0, bool first) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts_elect(d, a0 + (k >> 2) * 64 + (k & 3) * 8,
                       b0 + (uint64_t)((k * 2048) >> 4), id_km,
                       (first && k == 0) ? 0u : 1u);
      };
      int k0 = 0;  // K slot of step s
      for (int s = 0; s < ns && ok; ++s) {
        const bool more = s + 1 < ns;
        const int k1 = k0 + 1 == C::NKS ? 0 : k0 + 1;
        if (more) wait(C::B_KF + k1, ((s + 1) / C::NKS) & 1, s, 543);
        wait(C::B_PR, s & 1, s, 544);
        if (!ok) break;
        tc_fence_after();
        mm_ts(tmem + 384, tmem, dKm + k0 * kSlot, s == 0);
        if (more) {
          mm_ss(tmem, dQ, dKk + k1 * kSlot);
          mma_commit_elect(&bar[C::B_SF]);
          wait(C::B_VF + ((s + 1) & 1), ((s + 1) >> 1) & 1, s, 545);
        }
        wait(C::B_DSR, s & 1, s, 546);
        if (!ok) break;
        tc_fence_after();
        mm_ts(tmem + 256, tmem + 128, dKm + k0 * kSlot, s == 0);
        mm_ts(tmem + 256, tmem + 160, dKm + k0 * kSlot, false);
        mma_commit_elect(&bar[C::B_KE + k0]);
        if (more) {
          mm_ss(tmem + 128, dO, dV + ((s + 1) & 1) * kSlot);
          mma_commit_elect(&bar[C::B_DPF]);
          mma_commit_elect(&bar[C::B_VE + ((s + 1) & 1)]);
        }
        k0 = k1;
      }
      if (ok)
        mma_commit_elect(&bar[C::B_OD]);
      else
        drain_mma(&bar[C::B_DR]);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- threads
    // Two threads share a query row: thread h takes block h of a step.
    const int h = (warp - 2) >> 2;
    const int quad = warp & 3;
    const int rr = quad * 32 + lane;
    const int g = rr / p.TQ;
    const int tt = rr - g * p.TQ;
    const int tok = tile * p.TQ + tt;
    const bool active = tok < p.Lq;
    const int lim = p.causal ? min(tok + (p.Lkv - p.Lq), p.Lkv - 1) : p.Lkv - 1;
    const unsigned* wrow =
        p.words + (slot * p.cap + h) * (size_t)p.wpt + (tt >> 5);
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const float sl2 = p.scale * kPrefLog2e;
    float* del = p.delta + (size_t)(zq + g) * p.Lqp + tok;
    const float ndel = active ? *del : 0.f;
    const float nl2 = active ? __ldg(p.lse2 + (size_t)(zq + g) * p.Lqp + tok) : 0.f;
    float r0 = 0.f, r1 = 0.f;  // sum of this thread's dS
    bool ok = true;
    uint2 e_n = make_uint2(0, 0);
    unsigned w_n = 0;
    if (ns > 0) {
      e_n = __ldg(list);
      w_n = __ldg(wrow);
    }
    for (int s = 0; s < ns; ++s) {
      const unsigned bit = (w_n >> (tt & 31)) & 1u;
      // visible keys of the block for this row
      const int nv =
          bit ? lim - (int)(h ? e_n.y : e_n.x) * kSelBlock + 1 : 0;
      if (s + 1 < ns) {
        e_n = __ldg(list + s + 1);
        w_n = __ldg(wrow + (size_t)(2 * s + 2) * p.wpt);
      }
      bool w = ok && mbar_wait(&bar[C::B_SF], s & 1, kWaitSelect, s, 550);
      ok = __all_sync(FULL, w);
      if (!ok) break;
      tc_fence_after();
      uint32_t sv[2][32];
      tmem_ld32(lane_base + h * 64, sv[0]);
      tmem_ld32(lane_base + h * 64 + 32, sv[1]);
      tc_wait_ld();
      // P in place of S, float32 here and bf16 for M
      const bool plain = __all_sync(FULL, nv <= 0 || nv >= kSelBlock);
      const bool on = nv > 0;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          float e0, e1;
          fma2(e0, e1, __uint_as_float(sv[c][x]), __uint_as_float(sv[c][x + 1]),
               sl2, nl2);
          e0 = ex2_approx(e0);
          e1 = ex2_approx(e1);
          sv[c][x] = on ? __float_as_uint(e0) : 0u;
          sv[c][x + 1] = on ? __float_as_uint(e1) : 0u;
        }
      if (!plain) {
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (c * 32 + x >= nv) sv[c][x] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t st[16];
#pragma unroll
        for (int x = 0; x < 32; x += 2)
          st[x >> 1] = pack_bf16x2(__uint_as_float(sv[c][x]),
                                   __uint_as_float(sv[c][x + 1]));
        tmem_st16(lane_base + h * 64 + c * 16, st);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_PR]);
      w = mbar_wait(&bar[C::B_DPF], s & 1, kWaitSelect, s, 551);
      ok = __all_sync(FULL, w);
      if (!ok) break;
      tc_fence_after();
      // dS = P o (dP - D) over dP: its bf16 value in the first 32 of this
      // thread's 64 columns, bf16 of what that leaves (off by 2^-16 of dS) in
      // the others, those of the first keys behind the load of the second
      const uint32_t col = lane_base + 128 + h * 64;
      uint32_t lo[16];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t dp[32], st[16];
        tmem_ld32(col + c * 32, dp);
        tc_wait_ld();
        if (c == 1) tmem_st16(col + 32, lo);
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          float s0, s1;
          add_mul2(s0, s1, __uint_as_float(sv[c][x]),
                   __uint_as_float(sv[c][x + 1]), __uint_as_float(dp[x]),
                   __uint_as_float(dp[x + 1]), ndel, ndel);
          add2(r0, r1, s0, s1);
          const uint32_t hi = pack_bf16x2(s0, s1);
          st[x >> 1] = hi;
          lo[x >> 1] = pack_bf16x2(s0 - bf16lo(hi), s1 - bf16hi(hi));
        }
        tmem_st16(col + c * 16, st);
      }
      tmem_st16(col + 48, lo);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_DSR]);
    }
    if (ok && ns > 0) {
      const bool w = mbar_wait(&bar[C::B_OD], 0, kWaitSelect, ns, 552);
      ok = __all_sync(FULL, w);
      tc_fence_after();
    }
    // the row's sum of dS, from both its threads: what D was off by
    float* rs = reinterpret_cast<float*>(smem + C::OFF_R) + rr;
    rs[h * 128] = r0 + r1;
    ok = named_sync_and(1 + quad, 64, ok);
    if (ok) {
      const float r = rs[0] + rs[128];
      if (active && h == 0 && fabsf(r) < INFINITY) *del = ndel - r;
      __nv_bfloat16* out =
          p.dq + ((size_t)(zq + g) * p.Lq + tok) * kBwdD + h * 64;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t a[32], b2[32];
        if (ns > 0) {
          tmem_ld32(lane_base + 256 + h * 64 + c * 32, a);
          tmem_ld32(lane_base + 384 + h * 64 + c * 32, b2);
          tc_wait_ld();
        } else {  // nothing selected
#pragma unroll
          for (int x = 0; x < 32; ++x) a[x] = b2[x] = 0u;
        }
        if (active) {
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint32_t v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              float q0, q1;
              fma2v(q0, q1, __uint_as_float(b2[x + 2 * y]),
                    __uint_as_float(b2[x + 2 * y + 1]), -r,
                    __uint_as_float(a[x + 2 * y]),
                    __uint_as_float(a[x + 2 * y + 1]));
              v[y] = pack_bf16x2(q0 * p.scale, q1 * p.scale);
            }
            *reinterpret_cast<uint4*>(out + c * 32 + x) =
                make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
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

// [planes][cols] f32 with a 16-byte row stride, box TQ columns of G rows: the
// values of a tile's 128 rows, head by head.
inline bool encode_packed_rows(CUtensorMap* m, void* base, int cols,
                               long long planes, int TQ, int G) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)planes, 1};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 4,
                           (cuuint64_t)planes * cols * 4};
  cuuint32_t box[3] = {(cuuint32_t)TQ, (cuuint32_t)G, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Workspace, byte offsets (delta comes first).
struct SelBwdWorkspace {
  size_t lse2, bits, count, order, tlist, twords, nstep, list, words, total;
};
inline SelBwdWorkspace sel_bwd_workspace(int B, int Hq, int Hkv, int Lq,
                                         int Lkv) {
  const SelGeom g = sel_geom(Hq / Hkv, Lq, Lkv);
  const size_t bh = (size_t)B * Hkv;
  const size_t nk = ((size_t)Lkv + 127) / 128;
  const size_t slots = bh * nk, tiles = bh * g.ntile;
  const size_t rows = (size_t)B * Hq * ((Lq + 3) & ~3);
  SelBwdWorkspace w;
  w.lse2 = round256(rows * 4);
  w.bits = w.lse2 + round256(rows * 4);
  w.count = w.bits + round256(tiles * 2 * nk * g.wpt * 4);
  w.order = w.count + round256(slots * 4);
  w.tlist = w.order + round256(slots * 4);
  w.twords = w.tlist + round256(slots * g.ntile * 4);
  w.nstep = w.twords + round256(slots * g.ntile * 2 * g.wpt * 4);
  w.list = w.nstep + round256(tiles * 4);
  w.words = w.list + round256(tiles * g.cap * 4);
  w.total = w.words + round256(tiles * g.cap * g.wpt * 4);
  return w;
}

struct SelBwdProblem {
  const void *q, *k, *v, *o, *dout;
  const float* lse;
  const int* sel;
  void *dq, *dk, *dv;
  void* workspace;
  int B, Hq, Hkv, Lq, Lkv, n_sel, causal;
  float scale;
};

inline cudaError_t launch_select_backward(const SelBwdProblem& pr,
                                          cudaStream_t st) {
  const int G = pr.Hq / pr.Hkv;
  const SelGeom gm = sel_geom(G, pr.Lq, pr.Lkv);
  const SelBwdWorkspace w =
      sel_bwd_workspace(pr.B, pr.Hq, pr.Hkv, pr.Lq, pr.Lkv);
  char* ws = static_cast<char*>(pr.workspace);
  const int BH = pr.B * pr.Hkv;
  const int nk = (pr.Lkv + 127) / 128;
  const size_t rows = (size_t)pr.B * pr.Hq * pr.Lq;
  const long long planes = (long long)pr.B * pr.Hq;
  const long long slots = (long long)BH * nk;
  const long long tiles = (long long)BH * gm.ntile;
  const long long prep_blocks =
      (long long)((rows + kSelPrepRows - 1) / kSelPrepRows);
  if (prep_blocks > 0x7fffffffLL || slots > 0x7fffffffLL ||
      tiles > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;

  SelBwdParams p;
  memset(&p, 0, sizeof p);
  p.Lqp = (pr.Lq + 3) & ~3;
  p.delta = reinterpret_cast<float*>(ws);
  p.lse2 = reinterpret_cast<float*>(ws + w.lse2);
  if (!encode_packed_map(&p.tq, pr.q, kBwdD, pr.Lq, planes, gm.TQ, G) ||
      !encode_packed_map(&p.tdo, pr.dout, kBwdD, pr.Lq, planes, gm.TQ, G) ||
      !encode_map(&p.tk, pr.k, kBwdD, pr.Lkv, BH, kSelBlock) ||
      !encode_map(&p.tv, pr.v, kBwdD, pr.Lkv, BH, kSelBlock) ||
      !encode_packed_rows(&p.tdel, p.delta, p.Lqp, planes, gm.TQ, G) ||
      !encode_packed_rows(&p.tlse2, p.lse2, p.Lqp, planes, gm.TQ, G))
    return cudaErrorInvalidValue;
  p.o = static_cast<const __nv_bfloat16*>(pr.o);
  p.dout = static_cast<const __nv_bfloat16*>(pr.dout);
  p.lse = pr.lse;
  p.dq = static_cast<__nv_bfloat16*>(pr.dq);
  p.dk = static_cast<__nv_bfloat16*>(pr.dk);
  p.dv = static_cast<__nv_bfloat16*>(pr.dv);
  p.B = pr.B;
  p.Hq = pr.Hq;
  p.Hkv = pr.Hkv;
  p.Lq = pr.Lq;
  p.Lkv = pr.Lkv;
  p.G = G;
  p.causal = pr.causal;
  p.TQ = gm.TQ;
  p.wpt = gm.wpt;
  p.ntile = gm.ntile;
  p.cap = gm.cap;
  p.rep = gm.TQ >= 32 ? 1u : gm.TQ == 16 ? 0x00010001u
                         : gm.TQ == 8 ? 0x01010101u : 0x11111111u;
  p.scale = pr.scale;

  SelListArgs la;
  cudaError_t e = launch_select_lists(
      &la, pr.sel, reinterpret_cast<int*>(ws + w.nstep),
      reinterpret_cast<unsigned*>(ws + w.list),
      reinterpret_cast<unsigned*>(ws + w.words),
      reinterpret_cast<unsigned*>(ws + w.bits), gm, BH, pr.Lq, pr.Lkv, pr.n_sel,
      pr.causal, st);
  if (e != cudaSuccess) return e;
  p.nstep = la.nstep;
  p.list = la.list;
  p.words = la.words;
  SelBwdListArgs a;
  a.bits = la.bits;
  a.count = reinterpret_cast<int*>(ws + w.count);
  a.list = reinterpret_cast<int*>(ws + w.tlist);
  a.words = reinterpret_cast<unsigned*>(ws + w.twords);
  a.BH = BH;
  a.wpt = gm.wpt;
  a.ntile = gm.ntile;
  a.nblk2 = la.nblk2;
  p.count = a.count;
  p.tlist = a.list;
  p.twords = a.words;
  select_tiles_kernel<<<(unsigned)slots, 128, 0, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the order of the key blocks; none when every one has an SM to itself, or
  // when they are so many that the quadratic rank would cost more
  if (slots > kSelNumSm && slots <= kBwdOrderMaxSlots) {
    int* order = reinterpret_cast<int*>(ws + w.order);
    select_order_kernel<<<(unsigned)((slots + 7) / 8), 256, 0, st>>>(
        a.count, (int)slots, order);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.order = order;
  }

  select_prep_kernel<<<(unsigned)prep_blocks, 256, 0, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // (dQ first: it corrects the rows' D)
  e = cudaFuncSetAttribute(select_dq_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SelDqCfg::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  select_dq_kernel
      <<<(unsigned)tiles, kSelBwdThreads, SelDqCfg::SMEM_ALLOC, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  e = cudaFuncSetAttribute(select_dkdv_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SelDkdvCfg::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  select_dkdv_kernel
      <<<(unsigned)slots, kSelBwdThreads, SelDkdvCfg::SMEM_ALLOC, st>>>(p);
  return cudaGetLastError();
}

}  // namespace blasst
