"""Float64 restatement of block-selected attention (tests only): block means,
selection by score, and attention over a selection with its gradients, as
whole-matrix torch expressions on whatever device the inputs are on."""
import math

import torch

BLK = 64


def nblk(L):
    return -(-L // BLK)


def means(k):
    """k [..., L, d] -> [..., nblk, d] float64."""
    L = k.shape[-2]
    return torch.stack([k[..., j * BLK:min((j + 1) * BLK, L), :].double()
                        .mean(-2) for j in range(nblk(L))], dim=-2)


def select(q, c, last_block, n_sel, n_first, n_local):
    """One KV head: q [G, R, d], c [nb, d], last_block [R] (list) ->
    int32 [R, n_sel].  Ranks by the float64 score, ties to the lower index;
    NaN lowest."""
    s = torch.einsum("grd,jd->rj", q.double(), c.double())
    out = torch.full((q.shape[1], n_sel), -1, dtype=torch.int32)
    for r, lb in enumerate(last_block):
        if lb < 0:
            continue
        vis = range(lb + 1)
        must = [j for j in vis if j < n_first or j > lb - n_local]
        row = [-math.inf if math.isnan(x) else x for x in s[r].tolist()]
        rest = sorted((j for j in vis if j not in set(must)),
                      key=lambda j: (-row[j], j))
        got = sorted(must + rest[:n_sel - len(must)])
        out[r, :len(got)] = torch.tensor(got, dtype=torch.int32)
    return out


def allowed(sel, Lq, Lkv, causal):
    """sel [..., Lq, n_sel] -> bool [..., Lq, Lkv]."""
    nb = nblk(Lkv)
    s = sel.long()
    hit = torch.zeros(*s.shape[:-1], nb + 1, dtype=torch.bool, device=s.device)
    hit.scatter_(-1, torch.where((s >= 0) & (s < nb), s, nb), True)
    a = hit[..., :nb].repeat_interleave(BLK, -1)[..., :Lkv]
    if causal:
        r = torch.arange(Lq, device=s.device)[:, None] + Lkv - Lq
        a = a & (torch.arange(Lkv, device=s.device) <= r)
    return a


def attention(q, k, v, sel, scale, causal, dout=None):
    """dict with o, lse, pv (the row's sum of p |v|, for rounding bounds) and,
    given dout, dq, dk, dv; float64.  q [B,Hq,Lq,d], k/v [B,Hkv,Lkv,d]."""
    B, Hq, Lq, d = q.shape
    Hkv, Lkv = k.shape[1], k.shape[2]
    G = Hq // Hkv
    q5 = q.double().unflatten(1, (Hkv, G))
    k, v = k.double()[:, :, None], v.double()[:, :, None]
    al = allowed(sel, Lq, Lkv, causal)[:, :, None]
    s = (scale * (q5 @ k.transpose(-1, -2))).masked_fill(~al, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(al, torch.exp(s - lse[..., None]), 0.0)
    o = p @ v
    res = dict(o=o.flatten(1, 2), lse=lse.flatten(1, 2),
               pv=(p @ v.abs()).flatten(1, 2))
    if dout is not None:
        do = dout.double().unflatten(1, (Hkv, G))
        ds = p * (do @ v.transpose(-1, -2) - (do * o).sum(-1, keepdim=True))
        res["dv"] = (p.transpose(-1, -2) @ do).sum(2)
        res["dq"] = (scale * (ds @ k)).flatten(1, 2)
        res["dk"] = scale * (ds.transpose(-1, -2) @ q5).sum(2)
    return res


def decode(q, k, v, sel, lens, scale):
    """q [B,Hq,d]; logical caches k/v [B,Hkv,L,d]; sel [B,Hkv,n_sel]."""
    B, Hq, d = q.shape
    Hkv, L = k.shape[1], k.shape[2]
    G = Hq // Hkv
    al = allowed(sel[:, :, None], 1, L, False)
    al = al & (torch.arange(L, device=q.device)
               < torch.as_tensor(lens, device=q.device)[:, None, None, None])
    s = scale * (q.double().unflatten(1, (Hkv, G))
                 @ k.double().transpose(-1, -2))
    s = s.masked_fill(~al, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.where(al, torch.exp(s - lse[..., None]), 0.0)
    vd = torch.nan_to_num(v.double())
    return dict(o=(p @ vd).flatten(1, 2), lse=lse.flatten(1, 2),
                pv=(p @ vd.abs()).flatten(1, 2))


def random_selection(g, B, Hkv, Lq, Lkv, n_sel, causal, device, n_local=1):
    """A selection whose neighbouring rows mostly agree, own block included."""
    nb = nblk(Lkv)
    last = torch.tensor([(r + Lkv - Lq if causal else Lkv - 1) // BLK
                         for r in range(Lq)])
    out = torch.full((B, Hkv, Lq, n_sel), -1, dtype=torch.int32)
    j = torch.arange(nb)
    for b in range(B):
        for h in range(Hkv):
            s = torch.randn(Lq // 40 + 1, nb, generator=g)
            s = s.repeat_interleave(40, 0)[:Lq]
            s = s + 0.3 * torch.randn(Lq, nb, generator=g)
            s = torch.where(j > last[:, None] - n_local, 1e9, s)
            s = torch.where(j > last[:, None], -1e9, s)
            m = min(n_sel, nb)
            top = s.topk(m, dim=1).indices
            top = torch.where(top <= last[:, None], top, -1)
            out[b, h, :, :m] = top.int()
    return out.to(device)
