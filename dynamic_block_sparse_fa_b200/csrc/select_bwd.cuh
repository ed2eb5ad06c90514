// select_bwd.cuh -- backward of the block-selected attention (select_attn.cuh)
// with the selection held fixed: the gradients of softmax attention over each
// row's selected, visible keys (formulas in backward.cuh).
//
// bwd_dkdv_kernel<SEL = true> does the work: a CTA keeps one 128-key block
// (two selection blocks) and streams the query tiles (TQ tokens x G heads, 128
// rows) any of whose tokens selected either half.  Two kernels prepare its
// lists:
//   select_bits_kernel   per (KV head, tile): the token bits of every block,
//                        stored block-major
//   select_tiles_kernel  per (KV head, 128-key block): the tiles with a bit,
//                        ascending, and their bits
// The CTAs go out by the length of their lists, longest first.
#pragma once

#include "backward.cuh"
#include "select_attn.cuh"

namespace blasst {

struct SelBwdListArgs {
  const int* sel;    // [B, Hkv, Lq, n_sel]
  unsigned* bits;    // [B*Hkv][nblk2][ntile][wpt]
  int* count;        // [slots], slot = jb * (B*Hkv) + b*Hkv + hkv
  int* list;         // [slots][ntile]
  unsigned* words;   // [slots][ntile][2][wpt]
  int BH, Lq, Lkv, n_sel, causal;
  int TQ, wpt, ntile, nblk, nblk2;  // nblk2: nblk rounded up to whole 128 keys
};

__global__ void __launch_bounds__(256)
    select_bits_kernel(const SelBwdListArgs a) {
  extern __shared__ unsigned sel_bits[];  // [nblk][wpt]
  const int bh = blockIdx.x / a.ntile;
  const int tile = blockIdx.x - bh * a.ntile;
  for (int e = threadIdx.x; e < a.nblk * a.wpt; e += 256) sel_bits[e] = 0u;
  __syncthreads();
  const int row0 = tile * a.TQ;
  sel_set_bits(a.sel + (size_t)bh * a.Lq * a.n_sel, sel_bits, a.wpt, a.TQ, row0,
               min(a.TQ, a.Lq - row0), a.n_sel, a.Lkv - a.Lq, a.causal, a.nblk,
               (unsigned)bh);
  __syncthreads();
  for (int e = threadIdx.x; e < a.nblk2 * a.wpt; e += 256) {
    const int j = e / a.wpt, w = e - j * a.wpt;
    a.bits[(((size_t)bh * a.nblk2 + j) * a.ntile + tile) * a.wpt + w] =
        j < a.nblk ? sel_bits[e] : 0u;
  }
}

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

// Byte offsets of the lists behind the backward's own workspace.
struct SelBwdWorkspace {
  size_t bits, count, order, list, words, total;
};
inline SelBwdWorkspace sel_bwd_workspace(int B, int Hq, int Hkv, int Lq,
                                         int Lkv) {
  const SelGeom g = sel_geom(Hq / Hkv, Lq, Lkv);
  const size_t bh = (size_t)B * Hkv;
  const size_t nk = ((size_t)Lkv + 127) / 128;
  const size_t slots = bh * nk;
  SelBwdWorkspace w;
  w.bits = round256(bwd_workspace_bytes(B, Hq, Lq));
  w.count = w.bits + round256(bh * 2 * nk * g.ntile * g.wpt * 4);
  w.order = w.count + round256(slots * 4);
  w.list = w.order + round256(slots * 4);
  w.words = w.list + round256(slots * g.ntile * 4);
  w.total = w.words + round256(slots * g.ntile * 2 * g.wpt * 4);
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
  BwdParams p;
  memset(&p, 0, sizeof p);
  p.nq = gm.ntile;
  p.nk = (pr.Lkv + 127) / 128;
  const size_t rows = (size_t)pr.B * pr.Hq * pr.Lq;
  const long long planes = (long long)pr.B * pr.Hq;
  const long long slots = (long long)BH * p.nk;
  const long long tiles = (long long)BH * gm.ntile;
  const long long prep_blocks = (long long)((rows + 7) / 8);
  const long long conv_blocks = (long long)((rows * (kBwdD / 8) + 255) / 256);
  if (prep_blocks > 0x7fffffffLL || conv_blocks > 0x7fffffffLL ||
      slots > 0x7fffffffLL || tiles > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;

  SelBwdListArgs a;
  a.sel = pr.sel;
  a.bits = reinterpret_cast<unsigned*>(ws + w.bits);
  a.count = reinterpret_cast<int*>(ws + w.count);
  a.list = reinterpret_cast<int*>(ws + w.list);
  a.words = reinterpret_cast<unsigned*>(ws + w.words);
  a.BH = BH;
  a.Lq = pr.Lq;
  a.Lkv = pr.Lkv;
  a.n_sel = pr.n_sel;
  a.causal = pr.causal;
  a.TQ = gm.TQ;
  a.wpt = gm.wpt;
  a.ntile = gm.ntile;
  a.nblk = gm.nblk;
  a.nblk2 = 2 * p.nk;

  p.Lqp = (pr.Lq + 3) & ~3;
  const size_t prow = (size_t)planes * p.Lqp;
  p.dq_acc = reinterpret_cast<float*>(ws);
  p.delta = p.dq_acc + rows * kBwdD;
  p.lse2 = p.delta + ((prow + 63) & ~(size_t)63);
  if (!encode_packed_map(&p.tq, pr.q, kBwdD, pr.Lq, planes, gm.TQ, G) ||
      !encode_packed_map(&p.tdo, pr.dout, kBwdD, pr.Lq, planes, gm.TQ, G) ||
      !encode_map(&p.tk, pr.k, kBwdD, pr.Lkv, BH, 128) ||
      !encode_map(&p.tv, pr.v, kBwdD, pr.Lkv, BH, 128) ||
      !encode_map_f32(&p.tdq, p.dq_acc, pr.Lq, planes, gm.TQ, G) ||
      !encode_rows_f32(&p.tdel, p.delta, p.Lqp, planes, gm.TQ, G) ||
      !encode_rows_f32(&p.tlse2, p.lse2, p.Lqp, planes, gm.TQ, G))
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
  p.scale = pr.scale;
  p.sel_count = a.count;
  p.sel_list = a.list;
  p.sel_words = a.words;
  p.TQ = gm.TQ;
  p.wpt = gm.wpt;
  p.rep = gm.TQ >= 32 ? 1u : gm.TQ == 16 ? 0x00010001u
                         : gm.TQ == 8 ? 0x01010101u : 0x11111111u;
  p.counts = a.count;

  bwd_prep_kernel<<<(unsigned)prep_blocks, 256, 0, st>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem = gm.nblk * gm.wpt * 4;
  e = cudaFuncSetAttribute(select_bits_kernel,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  select_bits_kernel<<<(unsigned)tiles, 256, smem, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  select_tiles_kernel<<<(unsigned)slots, 128, 0, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (slots <= kBwdOrderMaxSlots) {
    int* order = reinterpret_cast<int*>(ws + w.order);
    bwd_order_kernel<<<(unsigned)((slots + 255) / 256), 256, 0, st>>>(p, order);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    p.order = order;
  }
  e = cudaFuncSetAttribute(bwd_dkdv_kernel<true>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize,
                           BwdCfg::SMEM_ALLOC);
  if (e != cudaSuccess) return e;
  bwd_dkdv_kernel<true>
      <<<(unsigned)slots, kBwdThreads, BwdCfg::SMEM_ALLOC, st>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  bwd_dq_kernel<<<(unsigned)conv_blocks, 256, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace blasst
