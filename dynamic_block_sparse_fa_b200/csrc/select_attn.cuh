// select_attn.cuh -- attention of many query rows over the key blocks that
// each row selected (block_select.cuh, or any other list): forward.
//
//   o_r = softmax over the keys c of the row's selected 64-key blocks, c
//         visible (causal: c <= r + Lkv - Lq), of scale q_r . k_c, times v
//
// The selection is one list per query row and KV head.  A list per row would
// leave a tensor-core tile with the G rows of one token; instead a tile packs
// TQ = 128 / G neighbouring tokens of the G heads (row g * TQ + t), walks the
// union of their lists, and masks per row.  Neighbouring tokens choose mostly
// the same blocks, so the union is little longer than one list; at worst it
// is all visible blocks, the dense forward's work.
//
// select_lists_kernel turns the selection into, per pair of tiles (per tile
// for the backward), the ascending list of blocks any of its tokens selected
// and, per listed block, one bit per token.  select_prefill_kernel is the two-tile pipeline of
// prefill2.cuh (a TMA producer warp, an MMA issuer warp, 4 softmax warps per
// tile; S and O in tensor memory, P over S) walking that list two blocks (128
// keys) a step; a tile none of whose tokens selected either block of a step
// does no work in it.
#pragma once

#include "block_select.cuh"
#include "prefill2.cuh"

namespace blasst {

// The largest number of 64-key blocks: a pair's token bits (32 bytes a block
// at one head per KV head) have to fit shared memory.
constexpr int kSelMaxBlocks = 4096;
constexpr unsigned kSelTile0 = 1u << 30, kSelTile1 = 1u << 31;
constexpr unsigned kSelIdMask = (1u << 30) - 1;

// Tokens per tile and 32-bit words of token bits per tile.
struct SelGeom {
  int TQ, wpt, ntile, npair, nblk, cap;
};
inline SelGeom sel_geom(int G, int Lq, int Lkv) {
  SelGeom g;
  g.TQ = 128 / G;
  g.wpt = g.TQ > 32 ? g.TQ / 32 : 1;
  g.ntile = (Lq + g.TQ - 1) / g.TQ;
  g.npair = (g.ntile + 1) / 2;
  g.nblk = (Lkv + kSelBlock - 1) / kSelBlock;
  g.cap = (g.nblk + 1) & ~1;  // list entries of a pair: whole steps
  return g;
}

struct SelListArgs {
  const int* sel;   // [B, Hkv, Lq, n_sel]
  int* nstep;       // [B*Hkv*nlist]
  unsigned* list;   // [B*Hkv*nlist][cap]: block id | which tiles use it
  unsigned* words;  // [B*Hkv*nlist][cap][tiles][wpt]
  int Lq, Lkv, n_sel, causal;
  int TQ, wpt, nlist, nblk, cap;
  int tiles;        // per list: 2 (forward pairs) or 1 (backward)
};

// Sets the bits of the selection rows [row0, row0 + nrow) in shared words
// [nblk][W]: row i's bit is bit i % 32 of word i / 32, where rows are cut into
// groups of TQ that start at whole words (TQ < 32: one word a group).
__device__ __forceinline__ void sel_set_bits(const int* sel, unsigned* bits,
                                             int W, int TQ, int row0, int nrow,
                                             int n_sel, int off, int causal,
                                             int nblk, unsigned where) {
  const int n = nrow * n_sel;
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int i = e / n_sel;
    const int id = __ldg(sel + (size_t)row0 * n_sel + e);
    if (id < 0) continue;
    if (id >= nblk) {  // not read through
      record_error(kBadBlockId, where, (unsigned)(row0 + i), (unsigned)id);
      continue;
    }
    // a block that starts after the row's last visible key holds nothing
    if (causal && id * kSelBlock > row0 + i + off) continue;
    const int grp = i / TQ, x = i - grp * TQ;
    const int wpt = TQ > 32 ? TQ / 32 : 1;
    atomicOr(&bits[(size_t)id * W + grp * wpt + (x >> 5)], 1u << (x & 31));
  }
}

__global__ void __launch_bounds__(256) select_lists_kernel(const SelListArgs a) {
  extern __shared__ unsigned sel_bits[];  // [nblk][tiles * wpt]
  __shared__ int wsum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x / a.nlist;
  const int id = blockIdx.x - bh * a.nlist;
  const int W = a.tiles * a.wpt;
  for (int e = tid; e < a.nblk * W; e += 256) sel_bits[e] = 0u;
  __syncthreads();
  const int row0 = id * a.tiles * a.TQ;
  sel_set_bits(a.sel + (size_t)bh * a.Lq * a.n_sel, sel_bits, W, a.TQ, row0,
               min(a.tiles * a.TQ, a.Lq - row0), a.n_sel, a.Lkv - a.Lq, a.causal,
               a.nblk, (unsigned)bh);
  __syncthreads();
  unsigned* list = a.list + (size_t)blockIdx.x * a.cap;
  unsigned* words = a.words + (size_t)blockIdx.x * a.cap * W;
  int at = 0;
  for (int j0 = 0; j0 < a.nblk; j0 += 256) {
    const int j = j0 + tid;
    unsigned any0 = 0, any1 = 0;
    if (j < a.nblk)
      for (int w = 0; w < a.wpt; ++w) {
        any0 |= sel_bits[j * W + w];
        if (a.tiles == 2) any1 |= sel_bits[j * W + a.wpt + w];
      }
    const bool take = (any0 | any1) != 0u;
    const unsigned m = __ballot_sync(~0u, take);
    if (lane == 0) wsum[warp] = __popc(m);
    __syncthreads();
    int before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w < warp) before += wsum[w];
      total += wsum[w];
    }
    if (take) {
      const int pos = at + before + __popc(m & ((1u << lane) - 1u));
      list[pos] = (unsigned)j | (any0 ? kSelTile0 : 0u) | (any1 ? kSelTile1 : 0u);
      for (int w = 0; w < W; ++w)
        words[(size_t)pos * W + w] = sel_bits[j * W + w];
    }
    at += total;
    __syncthreads();
  }
  if (tid == 0) a.nstep[blockIdx.x] = (at + 1) / 2;
  if ((at & 1) && tid < W) words[(size_t)at * W + tid] = 0u;
  if ((at & 1) && tid == 0)  // the last step's second block: one that the
    list[at] = list[at - 1] & kSelIdMask;  // list holds, with no bit set
}

struct __align__(64) SelPrefillParams {
  CUtensorMap tq, tk, tv;
  __nv_bfloat16* o;
  float* lse;
  const int* nstep;
  const unsigned* list;
  const unsigned* words;
  int B, Hq, Hkv, Lq, Lkv, G, TQ, wpt, npair, cap;
  float scale;
  int causal;
};

template <int D>
struct SelPrefillCfg {
  static constexpr int NKS = 2, NVS = 2;
  static constexpr int BOX_Q = 128 * 128;  // 128 rows x 64 columns
  static constexpr int BOX_K = 128 * 128;  // two blocks of 64 rows
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int KBYTES = 128 * D * 2;
  static constexpr int OFF_Q = 0;  // Q0 then Q1
  static constexpr int OFF_K = OFF_Q + 2 * QBYTES;
  static constexpr int OFF_V = OFF_K + NKS * KBYTES;
  static constexpr int OFF_BAR = OFF_V + NVS * KBYTES;
  static constexpr int B_Q = 0;
  static constexpr int B_KF = 1;
  static constexpr int B_KE = B_KF + NKS;
  static constexpr int B_VF = B_KE + NKS;
  static constexpr int B_VE = B_VF + NVS;
  static constexpr int B_SF = B_VE + NVS;  // [2]
  static constexpr int B_PF = B_SF + 2;    // [2]
  static constexpr int B_OD = B_PF + 2;
  static constexpr int NBAR = B_OD + 1;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int OFF_ABORT = OFF_TMEM + 4;  // int [2]
  static constexpr int SMEM = OFF_ABORT + 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int COL_S = 0;    // tile t at COL_S + t * 128
  static constexpr int COL_O = 256;  // tile t at COL_O + t * 128
  static constexpr int THREADS = 320;
  static_assert(SMEM_ALLOC <= 232448, "shared memory per CTA");
};

template <int D>
__global__ void __launch_bounds__(320, 1)
    select_prefill_kernel(const __grid_constant__ SelPrefillParams p) {
  using C = SelPrefillCfg<D>;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool leader = (lane == 0);

  // KV-head-major, and within a KV head the latest tokens (the longest
  // lists of a causal call) first
  const int bh = blockIdx.x / p.npair;  // b * Hkv + hkv
  const int pair = p.npair - 1 - (int)(blockIdx.x - bh * p.npair);
  const int b = bh / p.Hkv;
  const int hkv = bh - b * p.Hkv;
  const size_t slot = (size_t)bh * p.npair + pair;
  const int ns = __ldg(p.nstep + slot);
  const uint2* list = reinterpret_cast<const uint2*>(p.list + slot * p.cap);
  const int zq = b * p.Hq + hkv * p.G;  // the tile's first query head

  uint8_t* sQ = smem + C::OFF_Q;
  uint8_t* sK = smem + C::OFF_K;
  uint8_t* sV = smem + C::OFF_V;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);

  if (threadIdx.x == 0) {
    mbar_init(&bar[C::B_Q], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar[C::B_KF + i], 1);
      mbar_init(&bar[C::B_KE + i], 1);
      mbar_init(&bar[C::B_VF + i], 1);
      mbar_init(&bar[C::B_VE + i], 1);
      mbar_init(&bar[C::B_SF + i], 1);
      mbar_init(&bar[C::B_PF + i], 4);  // one arrival per softmax warp
    }
    mbar_init(&bar[C::B_OD], 1);
    reinterpret_cast<volatile int*>(smem + C::OFF_ABORT)[0] = 0;
    reinterpret_cast<volatile int*>(smem + C::OFF_ABORT)[1] = 0;
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
    // ------------------------------------------------------------------
    // TMA producer.  Lane i holds step (32 * chunk + i) of the list.
    // ------------------------------------------------------------------
    const uint64_t pol_q = policy_evict_first();
    const uint64_t pol_kv = policy_evict_last();
    uint2 ahead = make_uint2(0, 0);  // K runs two steps ahead of V
    uint2 cur = lane < ns ? __ldg(list + lane) : make_uint2(0, 0);
    if (ns > 32) ahead = 32 + lane < ns ? __ldg(list + 32 + lane) : make_uint2(0, 0);
    // blocks of step s, for s in the current chunk of 32 or the next
    int chunk = 0;
    auto step = [&](int s, unsigned& x, unsigned& y) {
      const bool nxt = (s >> 5) != chunk;
      x = __shfl_sync(FULL, nxt ? ahead.x : cur.x, s & 31) & kSelIdMask;
      y = __shfl_sync(FULL, nxt ? ahead.y : cur.y, s & 31) & kSelIdMask;
    };
    auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* full,
                    unsigned x, unsigned y) {
      mbar_arrive_expect_tx(full, C::KBYTES);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        tma_load_3d(dst + c * C::BOX_K, map, full, c * 64, (int)x * kSelBlock,
                    bh, pol_kv);
        tma_load_3d(dst + c * C::BOX_K + C::BOX_K / 2, map, full, c * 64,
                    (int)y * kSelBlock, bh, pol_kv);
      }
    };
    if (leader && ns > 0) {
      prefetch_tmap(&p.tq);
      prefetch_tmap(&p.tk);
      prefetch_tmap(&p.tv);
      mbar_arrive_expect_tx(&bar[C::B_Q], 2 * C::QBYTES);
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(sQ + t * C::QBYTES + c * C::BOX_Q, &p.tq, &bar[C::B_Q],
                      c * 64, (2 * pair + t) * p.TQ, zq, pol_q);
    }
    __syncwarp();
    for (int s = 0; s < 2 && s < ns; ++s) {
      unsigned x, y;
      step(s, x, y);
      if (leader) load(&p.tk, sK + s * C::KBYTES, &bar[C::B_KF + s], x, y);
    }
    for (int s = 0; s < ns; ++s) {
      if ((s >> 5) != chunk) {
        chunk = s >> 5;
        cur = ahead;
        const int e = 32 * (chunk + 1) + lane;
        ahead = e < ns ? __ldg(list + e) : make_uint2(0, 0);
      }
      const int sl = s & 1;
      unsigned x, y;
      step(s, x, y);
      if (s >= 2) {
        const bool w = mbar_wait(&bar[C::B_VE + sl], ((s >> 1) - 1) & 1,
                                 kWaitSelect, s, 200 + sl);
        if (!__all_sync(FULL, w)) break;
      }
      if (leader) load(&p.tv, sV + sl * C::KBYTES, &bar[C::B_VF + sl], x, y);
      __syncwarp();
      if (s + 2 < ns) {
        step(s + 2, x, y);
        const bool w = mbar_wait(&bar[C::B_KE + sl], (s >> 1) & 1, kWaitSelect,
                                 s, sl);
        if (!__all_sync(FULL, w)) break;
        if (leader) load(&p.tk, sK + sl * C::KBYTES, &bar[C::B_KF + sl], x, y);
        __syncwarp();
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------
    // MMA issuer.  Per step s: [tile 0] P0.V_s, Q0 K_{s+1}; [tile 1] the
    // same; a tile takes part in the steps its flag is set in.
    // ------------------------------------------------------------------
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16(128, D, 0, 1);
    const uint64_t dQ0 = smem_desc(smem_u32(sQ), 16, 1024, 2);
    const uint64_t dQ1 = smem_desc(smem_u32(sQ) + C::QBYTES, 16, 1024, 2);
    const uint64_t dK0 = smem_desc(smem_u32(sK), 16, 1024, 2);
    const uint64_t dK1 = smem_desc(smem_u32(sK) + C::KBYTES, 16, 1024, 2);
    const uint64_t dV0 = smem_desc(smem_u32(sV), C::BOX_K, 1024, 2);
    const uint64_t dV1 = smem_desc(smem_u32(sV) + C::KBYTES, C::BOX_K, 1024, 2);
    auto qk = [&](int t, int s) {
      const uint32_t d_s = tmem + C::COL_S + t * 128;
      const uint64_t da0 = t ? dQ1 : dQ0;
      const uint64_t db0 = (s & 1) ? dK1 : dK0;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t ka = (uint64_t)(((k >> 2) * C::BOX_Q + (k & 3) * 32) >> 4);
        const uint64_t kb = (uint64_t)(((k >> 2) * C::BOX_K + (k & 3) * 32) >> 4);
        mma_ss_elect(d_s, da0 + ka, db0 + kb, idesc_s, k > 0 ? 1u : 0u);
      }
      mma_commit_elect(&bar[C::B_SF + t]);
    };
    // flags of step s: bit t = tile t takes part
    uint2 fl = make_uint2(0, 0);
    int chunk = -1;
    auto flags = [&](int s) -> unsigned {
      if (s >= ns) return 0u;
      if ((s >> 5) != chunk) {
        chunk = s >> 5;
        const int e = 32 * chunk + lane;
        fl = e < ns ? __ldg(list + e) : make_uint2(0, 0);
      }
      return __shfl_sync(FULL, (fl.x | fl.y) >> 30, s & 31);
    };
    if (ns > 0) {
      bool ok = mbar_wait(&bar[C::B_Q], 0, kWaitSelect, 0, 1) &&
                mbar_wait(&bar[C::B_KF], 0, kWaitSelect, 0, 2);
      ok = __all_sync(FULL, ok);
      unsigned f = flags(0);
      tc_fence_after();
      if (ok) {
        for (int t = 0; t < 2; ++t)
          if ((f >> t) & 1u) qk(t, 0);
        mma_commit_elect(&bar[C::B_KE]);
      }
      int npv[2] = {0, 0};
      for (int s = 0; s < ns && ok; ++s) {
        const unsigned fn = flags(s + 1);
        const int sl = s & 1;
        bool have_v = false, have_k = false;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const bool now = (f >> t) & 1u, more = (fn >> t) & 1u;
          if (!ok || !(now || more)) continue;
          if (now) {
            ok = mbar_wait(&bar[C::B_PF + t], npv[t] & 1, kWaitSelect, s,
                           300 + t);
            if (!__all_sync(FULL, ok)) { ok = false; break; }
            if (!have_v) {
              have_v = true;
              ok = mbar_wait(&bar[C::B_VF + sl], (s >> 1) & 1, kWaitSelect, s,
                             210 + sl);
              if (!__all_sync(FULL, ok)) { ok = false; break; }
            }
          }
          if (more && !have_k) {
            have_k = true;
            ok = mbar_wait(&bar[C::B_KF + (sl ^ 1)], ((s + 1) >> 1) & 1,
                           kWaitSelect, s + 1, 100 + (sl ^ 1));
            if (!__all_sync(FULL, ok)) { ok = false; break; }
          }
          tc_fence_after();
          if (now) {
            const uint32_t a_p = tmem + C::COL_S + t * 128;
            const uint64_t dv0 = sl ? dV1 : dV0;
#pragma unroll
            for (int k = 0; k < 8; ++k)
              mma_ts_elect(tmem + C::COL_O + t * 128, a_p + k * 8,
                           dv0 + (uint64_t)((k * 2048) >> 4), idesc_o,
                           (npv[t] > 0 || k > 0) ? 1u : 0u);
            ++npv[t];
          }
          if (more) qk(t, s + 1);
        }
        if (!__all_sync(FULL, ok)) { ok = false; break; }
        mma_commit_elect(&bar[C::B_VE + sl]);
        if (s + 1 < ns) mma_commit_elect(&bar[C::B_KE + (sl ^ 1)]);
        f = fn;
      }
      if (ok) mma_commit_elect(&bar[C::B_OD]);  // every MMA has been issued
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------
    // Softmax: warps 2..5 tile 0, warps 6..9 tile 1; thread = row = (head
    // g, token t) of the tile.
    // ------------------------------------------------------------------
    const int t = (warp - 2) >> 2;
    const int quad = warp & 3;  // the warp's tensor-memory lane quadrant
    const int rr = quad * 32 + lane;
    const int g = rr / p.TQ;
    const int tt = rr - g * p.TQ;
    const int tok = (2 * pair + t) * p.TQ + tt;
    const bool active = tok < p.Lq;
    const int lim = p.causal ? min(tok + (p.Lkv - p.Lq), p.Lkv - 1) : p.Lkv - 1;
    const unsigned* wrow =
        p.words + slot * p.cap * (size_t)(2 * p.wpt) + t * p.wpt + (tt >> 5);
    const int ws = 2 * p.wpt;  // words from one list entry to the next
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_s = C::COL_S + t * 128;  // scores, then P
    const uint32_t col_o = C::COL_O + t * 128;
    const float sl2 = p.scale * kPrefLog2e;
    volatile int* abort_t = reinterpret_cast<volatile int*>(smem + C::OFF_ABORT);
    const unsigned my_flag = t ? kSelTile1 : kSelTile0;

    float m_ref = -INFINITY, m_run = -INFINITY;  // scaled, natural units
    float l = 0.f;
    int n = 0;  // steps this tile has taken part in
    bool ok = true;
    uint2 e_n = make_uint2(0, 0);
    unsigned w0_n = 0, w1_n = 0;
    if (ns > 0) {
      e_n = __ldg(list);
      w0_n = __ldg(wrow);
      w1_n = __ldg(wrow + ws);
    }
    for (int s = 0; s < ns; ++s) {
      const uint2 e = e_n;
      const unsigned b0 = (w0_n >> (tt & 31)) & 1u, b1 = (w1_n >> (tt & 31)) & 1u;
      if (s + 1 < ns) {
        e_n = __ldg(list + s + 1);
        w0_n = __ldg(wrow + (size_t)(2 * s + 2) * ws);
        w1_n = __ldg(wrow + (size_t)(2 * s + 3) * ws);
      }
      if (!((e.x | e.y) & my_flag)) continue;
      if (!mbar_wait(&bar[C::B_SF + t], n & 1, kWaitSelect, s, 400 + t))
        abort_t[t] = 1;
      ++n;
      tc_fence_after();
      uint32_t sr[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + col_s + c * 32, sr[c]);
      tc_wait_ld();
      // visible keys of the two blocks for this row
      int nv[2];
      nv[0] = b0 ? lim - (int)(e.x & kSelIdMask) * kSelBlock + 1 : 0;
      nv[1] = b1 ? lim - (int)(e.y & kSelIdMask) * kSelBlock + 1 : 0;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!__all_sync(FULL, nv[h] >= kSelBlock)) {
#pragma unroll
          for (int c = 2 * h; c < 2 * h + 2; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if ((c & 1) * 32 + x >= nv[h])
                sr[c][x] = __float_as_uint(-INFINITY);
        }
      }
      float mt;
      {
        float m8[8];
#pragma unroll
        for (int x = 0; x < 8; ++x)
          m8[x] = fmaxf(__uint_as_float(sr[0][x]), __uint_as_float(sr[0][x + 8]));
#pragma unroll
        for (int i = 16; i + 16 <= 128; i += 16)
#pragma unroll
          for (int x = 0; x < 8; ++x)
            m8[x] = fmax3(m8[x], __uint_as_float(sr[i >> 5][(i & 31) + x]),
                          __uint_as_float(sr[(i + 8) >> 5][((i + 8) & 31) + x]));
        mt = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                   fmaxf(m8[6], m8[7]));
      }
      const float mt_s = mt * p.scale;  // scale > 0: -inf stays -inf
      tc_fence_before();
      __syncwarp();
      if (__any_sync(FULL, abort_t[t] != 0)) { ok = false; break; }

      m_run = fmaxf(m_run, mt_s);
      float alpha = 1.f;
      bool rescale = false;
      if (m_run > m_ref + kRescaleNats || (m_ref == -INFINITY && m_run > -INFINITY)) {
        alpha = m_ref == -INFINITY ? 0.f
                                   : ex2_approx((m_ref - m_run) * kPrefLog2e);
        m_ref = m_run;
        rescale = true;
      }
      const float mb = m_ref == -INFINITY ? INFINITY : m_ref * kPrefLog2e;
      float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          const float p0 = ex2_approx(fmaf(__uint_as_float(sr[c][x]), sl2, -mb));
          const float p1 = ex2_approx(fmaf(__uint_as_float(sr[c][x + 1]), sl2, -mb));
          rs[(x >> 1) & 3] += p0 + p1;
          pk[x / 2] = pack_bf16x2(p0, p1);
        }
        tmem_st16(lane_base + col_s + c * 16, pk);
      }
      l = alpha * l + ((rs[0] + rs[1]) + (rs[2] + rs[3]));
      tc_wait_st();
      // O is idle: S of this step was issued after the last P.V (the arrival
      // of S certifies that that P.V is complete)
      if (n > 1 && __any_sync(FULL, rescale)) {
        const float f = rescale ? alpha : 1.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orow[32];
          tmem_ld32(lane_base + col_o + c * 32, orow);
          tc_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x)
            orow[x] = __float_as_uint(__uint_as_float(orow[x]) * f);
          tmem_st32(lane_base + col_o + c * 32, orow);
        }
        tc_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_PF + t]);
    }

    bool w = ok;
    if (ok && ns > 0)
      w = mbar_wait(&bar[C::B_OD], 0, kWaitSelect, ns, 600 + t);
    tc_fence_after();
    if (__all_sync(FULL, w)) {
      const float inv_l = 1.f / l;
      const size_t row = ((size_t)(zq + g)) * p.Lq + tok;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orow[32];
        if (n > 0) {
          tmem_ld32(lane_base + col_o + c * 32, orow);
          tc_wait_ld();
        }
        if (active) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c * 32);
#pragma unroll
          for (int x = 0; x < 32; x += 8) {
            uint32_t v[4];
#pragma unroll
            for (int y = 0; y < 4; ++y)
              v[y] = l == 0.f
                         ? 0u  // nothing selected
                         : pack_bf16x2(
                               __uint_as_float(orow[x + 2 * y]) * inv_l,
                               __uint_as_float(orow[x + 2 * y + 1]) * inv_l);
            dst[x / 8] = make_uint4(v[0], v[1], v[2], v[3]);
          }
        }
      }
      if (active && p.lse)
        p.lse[row] = l == 0.f ? -INFINITY : m_ref + __logf(l);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct SelProblem {
  const void *q, *k, *v;
  const int* sel;
  void* o;
  float* lse;
  void* workspace;
  int B, Hq, Hkv, Lq, Lkv, d, n_sel, causal;
  float scale;
};

// 3-D map over [planes, rows, D] bf16, box = 64 columns x TQ rows x G planes:
// TQ tokens of the G heads of a KV head land as 128 rows, head by head.
inline bool encode_packed_map(CUtensorMap* m, const void* base, int D,
                              int rows, long long planes, int TQ, int G) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)planes};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)TQ, (cuuint32_t)G};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
                  dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

// Workspace: steps per pair, block lists, token bits.
struct SelWorkspace {
  size_t list, words, total;  // byte offsets; the step counts come first
};
inline SelWorkspace sel_workspace(int B, int Hq, int Hkv, int Lq, int Lkv) {
  const SelGeom g = sel_geom(Hq / Hkv, Lq, Lkv);
  const size_t pairs = (size_t)B * Hkv * g.npair;
  SelWorkspace w;
  w.list = round256(pairs * 4);
  w.words = w.list + round256(pairs * g.cap * 4);
  w.total = w.words + round256(pairs * g.cap * 2 * g.wpt * 4);
  return w;
}

inline cudaError_t launch_select_lists(SelListArgs* a, const int* sel,
                                       int* nstep, unsigned* list,
                                       unsigned* words, const SelGeom& gm,
                                       int BH, int Lq, int Lkv, int n_sel,
                                       int causal, int tiles,
                                       cudaStream_t st) {
  a->sel = sel;
  a->nstep = nstep;
  a->list = list;
  a->words = words;
  a->Lq = Lq;
  a->Lkv = Lkv;
  a->n_sel = n_sel;
  a->causal = causal;
  a->TQ = gm.TQ;
  a->wpt = gm.wpt;
  a->nlist = tiles == 2 ? gm.npair : gm.ntile;
  a->nblk = gm.nblk;
  a->cap = gm.cap;
  a->tiles = tiles;
  const long long grid = (long long)BH * a->nlist;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int smem = gm.nblk * tiles * gm.wpt * 4;
  cudaError_t e = cudaFuncSetAttribute(
      select_lists_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  select_lists_kernel<<<(unsigned)grid, 256, smem, st>>>(*a);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_select_prefill(const SelProblem& pr, cudaStream_t st) {
  using C = SelPrefillCfg<D>;
  const int G = pr.Hq / pr.Hkv;
  const SelGeom gm = sel_geom(G, pr.Lq, pr.Lkv);
  const SelWorkspace w = sel_workspace(pr.B, pr.Hq, pr.Hkv, pr.Lq, pr.Lkv);
  char* ws = static_cast<char*>(pr.workspace);
  const long long grid = (long long)pr.B * pr.Hkv * gm.npair;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  SelListArgs a;
  cudaError_t e = launch_select_lists(
      &a, pr.sel, reinterpret_cast<int*>(ws),
      reinterpret_cast<unsigned*>(ws + w.list),
      reinterpret_cast<unsigned*>(ws + w.words), gm, pr.B * pr.Hkv, pr.Lq,
      pr.Lkv, pr.n_sel, pr.causal, 2, st);
  if (e != cudaSuccess) return e;

  SelPrefillParams p;
  memset(&p, 0, sizeof p);
  if (!encode_packed_map(&p.tq, pr.q, D, pr.Lq, (long long)pr.B * pr.Hq, gm.TQ, G) ||
      !encode_map(&p.tk, pr.k, D, pr.Lkv, (long long)pr.B * pr.Hkv, kSelBlock) ||
      !encode_map(&p.tv, pr.v, D, pr.Lkv, (long long)pr.B * pr.Hkv, kSelBlock))
    return cudaErrorInvalidValue;
  p.o = static_cast<__nv_bfloat16*>(pr.o);
  p.lse = pr.lse;
  p.nstep = a.nstep;
  p.list = a.list;
  p.words = a.words;
  p.B = pr.B;
  p.Hq = pr.Hq;
  p.Hkv = pr.Hkv;
  p.Lq = pr.Lq;
  p.Lkv = pr.Lkv;
  p.G = G;
  p.TQ = gm.TQ;
  p.wpt = gm.wpt;
  p.npair = gm.npair;
  p.cap = gm.cap;
  p.scale = pr.scale;
  p.causal = pr.causal;
  e = cudaFuncSetAttribute(select_prefill_kernel<D>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  select_prefill_kernel<D>
      <<<(unsigned)grid, C::THREADS, C::SMEM_ALLOC, st>>>(p);
  return cudaGetLastError();
}

}  // namespace blasst
