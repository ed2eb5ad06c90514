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
// select_lists_kernel turns the selection into, per tile, the ascending list
// of blocks any of its tokens selected and, per listed block, one bit per
// token (for the backward also the bits of all blocks, block-major).  select_prefill_kernel (a TMA producer warp, an MMA issuer warp, 8
// softmax warps) walks that list two blocks (128 keys) a step.
#pragma once

#include "block_select.cuh"
#include "prefill.cuh"

namespace blasst {

// The largest number of 64-key blocks: a tile's token bits (16 bytes a block
// at one head per KV head) have to fit shared memory.
constexpr int kSelMaxBlocks = 4096;

// Tokens per tile and 32-bit words of token bits per tile.
struct SelGeom {
  int TQ, wpt, ntile, nblk, cap;
};
inline SelGeom sel_geom(int G, int Lq, int Lkv) {
  SelGeom g;
  g.TQ = 128 / G;
  g.wpt = g.TQ > 32 ? g.TQ / 32 : 1;
  g.ntile = (Lq + g.TQ - 1) / g.TQ;
  g.nblk = (Lkv + kSelBlock - 1) / kSelBlock;
  g.cap = (g.nblk + 1) & ~1;  // list entries of a tile: whole steps
  return g;
}

struct SelListArgs {
  const int* sel;   // [B, Hkv, Lq, n_sel]
  int* nstep;       // [B*Hkv*ntile]
  unsigned* list;   // [B*Hkv*ntile][cap] block ids
  unsigned* words;  // [B*Hkv*ntile][cap][wpt]
  unsigned* bits;   // backward: [B*Hkv][nblk2][ntile][wpt], block-major
  int Lq, Lkv, n_sel, causal;
  int TQ, wpt, ntile, nblk, cap;
  int nblk2;        // nblk rounded up to whole 128 keys
};

// Sets the bits of the selection rows [row0, row0 + nrow) in shared words
// [nblk][W]: row i's bit is bit i % 32 of word i / 32.
__device__ __forceinline__ void sel_set_bits(const int* sel, unsigned* bits,
                                             int W, int row0, int nrow,
                                             int n_sel, int off, int causal,
                                             int nblk, unsigned where) {
  const int n = nrow * n_sel;  // <= 128 * 4096
  const int* base = sel + (size_t)row0 * n_sel;
  // e / n_sel by multiplication: exact while e * n_sel < 2^32
  const unsigned inv = n_sel > 1 ? 0xffffffffu / (unsigned)n_sel + 1u : 0u;
#pragma unroll 4
  for (int e = threadIdx.x; e < n; e += blockDim.x) {
    const int id = __ldg(base + e);
    const int i = n_sel > 1 ? (int)__umulhi((unsigned)e, inv) : e;
    if (id >= nblk) {  // not read through
      record_error(kBadBlockId, where, (unsigned)(row0 + i), (unsigned)id);
      continue;
    }
    // a block that starts after the row's last visible key holds nothing
    if (id < 0 || (causal && id * kSelBlock > row0 + i + off)) continue;
    atomicOr(&bits[id * W + (i >> 5)], 1u << (i & 31));
  }
}

__global__ void __launch_bounds__(256) select_lists_kernel(const SelListArgs a) {
  extern __shared__ unsigned sel_bits[];  // [nblk][wpt]
  __shared__ int wsum[8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bh = blockIdx.x / a.ntile;
  const int tile = blockIdx.x - bh * a.ntile;
  const int W = a.wpt;
  for (int e = tid; e < a.nblk * W; e += 256) sel_bits[e] = 0u;
  __syncthreads();
  const int row0 = tile * a.TQ;
  sel_set_bits(a.sel + (size_t)bh * a.Lq * a.n_sel, sel_bits, W, row0,
               min(a.TQ, a.Lq - row0), a.n_sel, a.Lkv - a.Lq, a.causal,
               a.nblk, (unsigned)bh);
  __syncthreads();
  unsigned* list = a.list + (size_t)blockIdx.x * a.cap;
  unsigned* words = a.words + (size_t)blockIdx.x * a.cap * W;
  int at = 0;
  for (int j0 = 0; j0 < a.nblk; j0 += 256) {
    const int j = j0 + tid;
    unsigned any = 0;
    if (j < a.nblk)
      for (int w = 0; w < W; ++w) any |= sel_bits[j * W + w];
    const bool take = any != 0u;
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
      list[pos] = (unsigned)j;
      for (int w = 0; w < W; ++w)
        words[(size_t)pos * W + w] = sel_bits[j * W + w];
    }
    at += total;
    __syncthreads();
  }
  if (a.bits)
    for (int e = tid; e < a.nblk2 * W; e += 256) {
      const int j = e / W, w = e - j * W;
      a.bits[(((size_t)bh * a.nblk2 + j) * a.ntile + tile) * W + w] =
          j < a.nblk ? sel_bits[e] : 0u;
    }
  if (tid == 0) a.nstep[blockIdx.x] = (at + 1) / 2;
  if ((at & 1) && tid < W) words[(size_t)at * W + tid] = 0u;
  if ((at & 1) && tid == 0)  // the last step's second block: one that the
    list[at] = list[at - 1];  // list holds, with no bit set
}

struct __align__(64) SelPrefillParams {
  CUtensorMap tq, tk, tv;
  __nv_bfloat16* o;
  float* lse;
  const int* nstep;
  const unsigned* list;
  const unsigned* words;
  int B, Hq, Hkv, Lq, Lkv, G, TQ, wpt, ntile, cap;
  float scale;
  int causal;
};

// Waits for the last loads of a ring of n slots into which `issued` loads went
// in order.  After a run without failures every one has been waited for.
__device__ __forceinline__ void drain_ring(uint64_t* full, int n, int issued) {
  for (int u = issued > n ? issued - n : 0; u < issued; ++u)
    mbar_wait(&full[u % n], (uint32_t)(u / n) & 1u, kWaitSelect, u, 900);
}
// Waits, after some other wait gave up, for the products issued so far (whole
// warp): tensor memory is freed and operands are released behind this.
__device__ __forceinline__ void drain_mma(uint64_t* bar) {
  __syncwarp();
  mma_commit_elect(bar);
  mbar_wait(bar, 0, kWaitSelect, 0, 901);
  __syncwarp();
}

template <int D>
struct SelPrefillCfg {
  static constexpr int NKS = 3, NVS = 2;
  static constexpr int BOX = 128 * 128;  // 128 rows x 64 columns
  static constexpr int TILE = 128 * D * 2;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + TILE;
  static constexpr int OFF_V = OFF_K + NKS * TILE;
  static constexpr int OFF_XM = OFF_V + NVS * TILE;
  // float2 [2 groups][128 rows]: (running max, reference) after the group's
  // last step, then (normaliser, reference) at the end
  static constexpr int OFF_XL = OFF_XM + 2 * 128 * 8;
  static constexpr int OFF_BAR = OFF_XL + 2 * 128 * 8;
  static constexpr int B_Q = 0;
  static constexpr int B_KF = 1;           // [3]
  static constexpr int B_KE = B_KF + NKS;  // [3]
  static constexpr int B_VF = B_KE + NKS;  // [2]
  static constexpr int B_VE = B_VF + NVS;  // [2]
  // [2] each: even and odd steps
  static constexpr int B_SF = B_VE + NVS;  // S in its buffer
  static constexpr int B_SR = B_SF + 2;    // S read (one arrival per warp)
  static constexpr int B_PR = B_SR + 2;    // P written, O scaled (per warp)
  static constexpr int B_OF = B_PR + 2;    // P.V complete
  static constexpr int B_MX = B_OF + 2;    // [2][4 quadrants] maxima written
  static constexpr int B_DR = B_MX + 8;    // drain after a wait gave up
  static constexpr int NBAR = B_DR + 1;
  static constexpr int OFF_TMEM = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_TMEM + 8;
  static constexpr int SMEM_ALLOC = SMEM + 1024;
  static constexpr int COL_S = 0;    // buffer i at COL_S + i * 128
  static constexpr int COL_O = 256;
  static constexpr int COL_P = 384;  // buffer i at COL_P + i * 64
  static constexpr int THREADS = 96 + 256;
  static_assert(SMEM_ALLOC <= 232448, "shared memory per CTA");
};

// One query tile per CTA; per step of two blocks S = Q K^T into one of two
// buffers, P (bf16, V's type, as the product wants it: 2^-8 of each term; the
// normaliser sums it in float32) into one of two others, O += P V.  A step's
// softmax is a chain (scores out of tensor memory, maxima, exps, P back) about
// twice as long as its exps alone keep the MUFU busy, so two groups of 4 warps
// (thread = row) take the even and the odd steps and overlap: while one group
// is in its exps the other loads, reduces and stores.  All they share is the
// row's running max and reference, handed over once per step after three
// quarters of its exps, so that the groups' exps follow one another.  S of step
// s + 2 is issued as soon as step s has read its scores, so the chain never
// waits for the tensor core.
//
// 32 heads on 8, 16K causal, 32 blocks a row: 0.82 ms, the tensor pipe and the
// MUFU 48% busy each (1024 cycles of either a step, of about 1.9k); 0.9 PFLOP/s
// of 128 x 128 tiles, 0.62 of the rows' own blocks.
template <int D>
__global__ void __launch_bounds__(352, 1)
    select_prefill_kernel(const __grid_constant__ SelPrefillParams p) {
  using C = SelPrefillCfg<D>;
  constexpr unsigned FULL = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // KV-head-major (resident CTAs share K and V in L2), and within a KV head
  // the latest tokens (the longest lists of a causal call) first
  const int bh = blockIdx.x / p.ntile;  // b * Hkv + hkv
  const int tile = p.ntile - 1 - (int)(blockIdx.x - bh * p.ntile);
  const int b = bh / p.Hkv;
  const int hkv = bh - b * p.Hkv;
  const size_t slot = (size_t)bh * p.ntile + tile;
  const int ns = __ldg(p.nstep + slot);
  const uint2* list = reinterpret_cast<const uint2*>(p.list + slot * p.cap);
  const int zq = b * p.Hq + hkv * p.G;  // the tile's first query head

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
      mbar_init(&bar[C::B_SF + i], 1);
      mbar_init(&bar[C::B_SR + i], 4);
      mbar_init(&bar[C::B_PR + i], 4);
      mbar_init(&bar[C::B_OF + i], 1);
    }
    for (int i = 0; i < 8; ++i) mbar_init(&bar[C::B_MX + i], 1);
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

  if (warp == 0 || warp == 10) {
    // ------------------------------------------------------------------
    // TMA producers: warp 0 Q and K, warp 10 V (a V slot is free only after
    // its P.V, far behind the S that frees a K slot: one producer for both
    // would hold the K loads back)
    // ------------------------------------------------------------------
    if (lane == 0 && ns > 0) {
      const bool is_k = warp == 0;
      const int nslot = is_k ? C::NKS : C::NVS;
      const CUtensorMap* map = is_k ? &p.tk : &p.tv;
      uint8_t* ring = smem + (is_k ? C::OFF_K : C::OFF_V);
      uint64_t* full = &bar[is_k ? C::B_KF : C::B_VF];
      uint64_t* empty = &bar[is_k ? C::B_KE : C::B_VE];
      const uint64_t pol_kv = policy_evict_last();
      if (is_k) {
        const uint64_t pol_q = policy_evict_first();
        mbar_arrive_expect_tx(&bar[C::B_Q], C::TILE);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(smem + C::OFF_Q + c * C::BOX, &p.tq, &bar[C::B_Q], c * 64,
                      tile * p.TQ, zq, pol_q);
      }
      uint2 next = __ldg(list);
      int sl = 0, s = 0;
      uint32_t par = 1;  // of the slot's previous use
      for (; s < ns; ++s) {
        const uint2 e = next;
        if (s + 1 < ns) next = __ldg(list + s + 1);
        if (s >= nslot &&
            !mbar_wait(&empty[sl], par, kWaitSelect, s, 400 + (is_k ? 0 : 1)))
          break;
        mbar_arrive_expect_tx(&full[sl], C::TILE);
        uint8_t* dst = ring + sl * C::TILE;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(dst + c * C::BOX, map, &full[sl], c * 64,
                      (int)e.x * kSelBlock, bh, pol_kv);
          tma_load_3d(dst + c * C::BOX + C::BOX / 2, map, &full[sl], c * 64,
                      (int)e.y * kSelBlock, bh, pol_kv);
        }
        if (++sl == nslot) {
          sl = 0;
          par ^= 1;
        }
      }
      // no copy is left in flight, whatever became of its readers
      drain_ring(full, nslot, s);
      if (is_k) mbar_wait(&bar[C::B_Q], 0, kWaitSelect, s, 402);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------
    // MMA issuer: S_0, S_1, then per step S_{s+2} and P_{s-1} V_{s-1}
    // ------------------------------------------------------------------
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idesc_o = idesc_bf16(128, D, 0, 1);
    const uint64_t dQ = smem_desc(smem_u32(smem + C::OFF_Q), 16, 1024, 2);
    const uint64_t dK = smem_desc(smem_u32(smem + C::OFF_K), 16, 1024, 2);
    const uint64_t dV = smem_desc(smem_u32(smem + C::OFF_V), C::BOX, 1024, 2);
    constexpr uint64_t kSlot = (uint64_t)(C::TILE >> 4);
    bool ok = true;
    auto wait = [&](int id, int parity, int step, int what) {
      const bool w = ok && mbar_wait(&bar[id], parity, kWaitSelect, step, what);
      ok = __all_sync(FULL, w);
    };
    int ks = 0, kp = 0;  // K slot of the next S and its parity
    auto qk = [&](int s) {
      wait(C::B_KF + ks, kp, s, 410);
      if (!ok) return;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t st = (uint64_t)(((k >> 2) * C::BOX + (k & 3) * 32) >> 4);
        mma_ss_elect(tmem + C::COL_S + (s & 1) * 128, dQ + st,
                     dK + ks * kSlot + st, idesc_s, k > 0 ? 1u : 0u);
      }
      mma_commit_elect(&bar[C::B_SF + (s & 1)]);
      mma_commit_elect(&bar[C::B_KE + ks]);
      if (++ks == 3) {
        ks = 0;
        kp ^= 1;
      }
    };
    if (ns > 0) {
      wait(C::B_Q, 0, 0, 411);
      qk(0);
      if (ns > 1) qk(1);
      for (int s = 0; s <= ns && ok; ++s) {
        if (s + 2 < ns) {
          wait(C::B_SR + (s & 1), (s >> 1) & 1, s, 414);
          qk(s + 2);
        }
        if (s == 0) continue;
        const int v = s - 1, vs = v & 1;
        wait(C::B_VF + vs, (v >> 1) & 1, v, 412);
        wait(C::B_PR + vs, (v >> 1) & 1, v, 413);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ts_elect(tmem + C::COL_O, tmem + C::COL_P + vs * 64 + k * 8,
                       dV + vs * kSlot + (uint64_t)((k * 2048) >> 4), idesc_o,
                       (v > 0 || k > 0) ? 1u : 0u);
        mma_commit_elect(&bar[C::B_OF + vs]);
        mma_commit_elect(&bar[C::B_VE + vs]);
      }
      if (!ok) drain_mma(&bar[C::B_DR]);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------
    // Softmax.  Warps 2..5 take the even steps, warps 6..9 the odd ones;
    // thread = row = (head g, token tt) of the tile.
    // ------------------------------------------------------------------
    constexpr int DH = D / 2;
    const int grp = (warp - 2) >> 2;
    const int quad = warp & 3;  // the warp's tensor-memory lane quadrant
    const int rr = quad * 32 + lane;
    const int g = rr / p.TQ;
    const int tt = rr - g * p.TQ;
    const int tok = tile * p.TQ + tt;
    const bool active = tok < p.Lq;
    const int lim = p.causal ? min(tok + (p.Lkv - p.Lq), p.Lkv - 1) : p.Lkv - 1;
    const unsigned* wrow = p.words + slot * p.cap * (size_t)p.wpt + (tt >> 5);
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16);
    const uint32_t col_s = C::COL_S + grp * 128;
    const uint32_t col_p = C::COL_P + grp * 64;
    const float sl2 = p.scale * kPrefLog2e;
    float2* xm = reinterpret_cast<float2*>(smem + C::OFF_XM) + rr;
    float2* xl = reinterpret_cast<float2*>(smem + C::OFF_XL) + rr;

    // The chunk of exps after which the row's max and reference go over: the
    // other group's exps follow this group's.
    constexpr int kTurn = 2;
    float m_ref = -INFINITY;  // reference of l (scaled, natural units)
    float l = 0.f;            // of this group's steps
    bool ok = true;
    uint2 e_n = make_uint2(0, 0);
    unsigned w0_n = 0, w1_n = 0;
    if (grp < ns) {
      e_n = __ldg(list + grp);
      w0_n = __ldg(wrow + 2 * grp * p.wpt);
      w1_n = __ldg(wrow + (2 * grp + 1) * p.wpt);
    }
    for (int s = grp; s < ns; s += 2) {
      const uint32_t par = (s >> 1) & 1;
      // visible keys of the step's blocks for this row
      int nv[2];
      nv[0] = (w0_n >> (tt & 31)) & 1u ? lim - (int)e_n.x * kSelBlock + 1 : 0;
      nv[1] = (w1_n >> (tt & 31)) & 1u ? lim - (int)e_n.y * kSelBlock + 1 : 0;
      if (s + 2 < ns) {
        // (volatile: issued here, a step ahead of their use)
        e_n.x = ld_nc_volatile(&list[s + 2].x);
        e_n.y = ld_nc_volatile(&list[s + 2].y);
        w0_n = ld_nc_volatile(wrow + (2 * s + 4) * p.wpt);
        w1_n = ld_nc_volatile(wrow + (2 * s + 5) * p.wpt);
      }
      bool w = ok && mbar_wait(&bar[C::B_SF + grp], par, kWaitSelect, s, 420);
      ok = __all_sync(FULL, w);
      if (!ok) break;
      tc_fence_after();
      uint32_t sr[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + col_s + c * 32, sr[c]);
      tc_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_SR + grp]);
      // a warp whose rows all see either all 64 keys of a block or none
      // compares no columns
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (__any_sync(FULL, nv[h] > 0 && nv[h] < kSelBlock)) {
#pragma unroll
          for (int c = 2 * h; c < 2 * h + 2; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if ((c & 1) * 32 + x >= nv[h])
                sr[c][x] = __float_as_uint(-INFINITY);
        } else if (!__all_sync(FULL, nv[h] > 0)) {
          const bool on = nv[h] > 0;
#pragma unroll
          for (int c = 2 * h; c < 2 * h + 2; ++c)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              sr[c][x] = on ? sr[c][x] : __float_as_uint(-INFINITY);
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
      if (s >= 2) {  // the P buffer is free: this group's last P.V is over
        w = mbar_wait(&bar[C::B_OF + grp], par ^ 1, kWaitSelect, s, 425);
        ok = __all_sync(FULL, w);
        if (!ok) break;
        tc_fence_after();
      }
      // the row's running max and reference after step s - 1
      float2 m = make_float2(-INFINITY, -INFINITY);
      if (s > 0) {
        w = mbar_wait(&bar[C::B_MX + (grp ^ 1) * 4 + quad], ((s - 1) >> 1) & 1,
                      kWaitSelect, s, 424);
        ok = __all_sync(FULL, w);
        if (!ok) break;
        m = xm[(grp ^ 1) * 128];
      }
      m.x = fmaxf(m.x, mt * p.scale);  // scale > 0: -inf stays -inf
      float alpha = 1.f;  // of O
      bool rescale = false;
      if (m.x > m.y + kRescaleNats || (m.y == -INFINITY && m.x > -INFINITY)) {
        alpha = m.y == -INFINITY ? 0.f : ex2_approx((m.y - m.x) * kPrefLog2e);
        m.y = m.x;
        rescale = true;
      }
      // (free: the other group's step s - 1 read it before it wrote its own)
      xm[grp * 128] = m;
      if (m.y != m_ref) {  // the reference moved since this group's last step
        l *= m_ref == -INFINITY ? 0.f : ex2_approx((m_ref - m.y) * kPrefLog2e);
        m_ref = m.y;
      }
      const float mb = m_ref == -INFINITY ? -INFINITY : -m_ref * kPrefLog2e;
      float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          float a0, a1;
          fma2(a0, a1, __uint_as_float(sr[c][x]), __uint_as_float(sr[c][x + 1]),
               sl2, mb);
          a0 = ex2_approx(a0);
          a1 = ex2_approx(a1);
          add2(rs[x & 2], rs[(x & 2) + 1], a0, a1);
          pk[x / 2] = pack_bf16x2(a0, a1);
        }
        tmem_st16(lane_base + col_p + c * 16, pk);
        if (c == kTurn) {
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar[C::B_MX + grp * 4 + quad]);
        }
      }
      l += (rs[0] + rs[1]) + (rs[2] + rs[3]);
      if (s > 0 && __any_sync(FULL, rescale)) {
        // O is idle once P.V of step s - 1 is complete (the step before it
        // is, so the parity names the right phase)
        w = mbar_wait(&bar[C::B_OF + (grp ^ 1)], ((s - 1) >> 1) & 1,
                      kWaitSelect, s, 421);
        ok = __all_sync(FULL, w);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orow[32];
          tmem_ld32(lane_base + C::COL_O + c * 32, orow);
          tc_wait_ld();
#pragma unroll
          for (int x = 0; x < 32; ++x)
            orow[x] = __float_as_uint(__uint_as_float(orow[x]) * alpha);
          tmem_st32(lane_base + C::COL_O + c * 32, orow);
        }
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar[C::B_PR + grp]);
    }

    if (ns > 0) {
      // the last two P.V, in order
      bool w = ok;
      if (w && ns > 1)
        w = mbar_wait(&bar[C::B_OF + (ns & 1)], ((ns - 2) >> 1) & 1,
                      kWaitSelect, ns, 422);
      w = w && mbar_wait(&bar[C::B_OF + ((ns - 1) & 1)], ((ns - 1) >> 1) & 1,
                         kWaitSelect, ns, 423);
      ok = __all_sync(FULL, w);
      tc_fence_after();
    }
    // the row's normaliser: both groups' parts, in the last step's reference
    xl[grp * 128] = make_float2(l, m_ref);
    ok = named_sync_and(1 + quad, 64, ok);
    if (ok) {
      const int fin = (ns - 1) & 1;  // the group of the last step
      const float2 la = xl[fin * 128], lb = xl[(fin ^ 1) * 128];
      m_ref = la.y;
      l = la.x;
      if (lb.y != -INFINITY)
        l += lb.x * ex2_approx((lb.y - m_ref) * kPrefLog2e);
      const float inv_l = 1.f / l;
      const size_t row = ((size_t)(zq + g)) * p.Lq + tok;
      // each group writes half of the row
#pragma unroll
      for (int c = 0; c < DH / 32; ++c) {
        uint32_t orow[32];
        if (ns > 0) {
          tmem_ld32(lane_base + C::COL_O + grp * DH + c * 32, orow);
          tc_wait_ld();
        }
        if (active) {
          uint4* dst =
              reinterpret_cast<uint4*>(p.o + row * D + grp * DH + c * 32);
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
      if (active && p.lse && grp == 0)
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

// Workspace: steps per tile, block lists, token bits.
struct SelWorkspace {
  size_t list, words, total;  // byte offsets; the step counts come first
};
inline SelWorkspace sel_workspace(int B, int Hq, int Hkv, int Lq, int Lkv) {
  const SelGeom g = sel_geom(Hq / Hkv, Lq, Lkv);
  const size_t tiles = (size_t)B * Hkv * g.ntile;
  SelWorkspace w;
  w.list = round256(tiles * 4);
  w.words = w.list + round256(tiles * g.cap * 4);
  w.total = w.words + round256(tiles * g.cap * g.wpt * 4);
  return w;
}

inline cudaError_t launch_select_lists(SelListArgs* a, const int* sel,
                                       int* nstep, unsigned* list,
                                       unsigned* words, unsigned* bits,
                                       const SelGeom& gm,
                                       int BH, int Lq, int Lkv, int n_sel,
                                       int causal, cudaStream_t st) {
  a->sel = sel;
  a->nstep = nstep;
  a->list = list;
  a->words = words;
  a->bits = bits;
  a->nblk2 = (gm.nblk + 1) & ~1;
  a->Lq = Lq;
  a->Lkv = Lkv;
  a->n_sel = n_sel;
  a->causal = causal;
  a->TQ = gm.TQ;
  a->wpt = gm.wpt;
  a->ntile = gm.ntile;
  a->nblk = gm.nblk;
  a->cap = gm.cap;
  const long long grid = (long long)BH * a->ntile;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int smem = gm.nblk * gm.wpt * 4;
  // the limit of all calls: it is the function's, shared by every thread
  cudaError_t e = cudaFuncSetAttribute(
      select_lists_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
      kSelMaxBlocks * 4 * 4);
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
  const long long grid = (long long)pr.B * pr.Hkv * gm.ntile;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  SelListArgs a;
  cudaError_t e = launch_select_lists(
      &a, pr.sel, reinterpret_cast<int*>(ws),
      reinterpret_cast<unsigned*>(ws + w.list),
      reinterpret_cast<unsigned*>(ws + w.words), nullptr, gm, pr.B * pr.Hkv,
      pr.Lq, pr.Lkv, pr.n_sel, pr.causal, st);
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
  p.ntile = gm.ntile;
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
