"""Cases for the block-selected attention operators: key-block means, block
selection by a cheap score, and attention over the selected blocks, each in
its prompt (or training) form and in its single-token form.

A case is a dict of plain values.  ``run`` computes the operator in plain
torch (``own`` false) or through this package's entry points (``own`` true);
``exact`` computes it in 64 bits, separately from the plain form.
"""
import math

import torch

own = False

BLK = 64  # keys per block


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # summaries of a prompt's keys, computed once after prefill
        dict(name="means_prompt_16k", op="means", B=1, Hkv=8, L=16384, d=128),
        # a small ragged batch at the other head dimension
        dict(name="means_prompt_ragged", op="means", B=3, Hkv=2, L=5037, d=64),
        # one decode step of a serving batch: every sequence has one new token
        dict(name="means_step_b32", op="means_paged", B=32, Hkv=8, L=32768,
             d=128, page=64, n_new=1),
        # the selection of a 16K prompt, 4 query heads per KV head
        dict(name="select_prompt_16k", op="select", B=1, Hq=32, Hkv=8,
             Lq=16384, Lkv=16384, d=128, causal=True, n_sel=32, n_first=1,
             n_local=2),
        # the last chunk of a prompt, one query head per KV head
        dict(name="select_chunk_ragged", op="select", B=2, Hq=4, Hkv=4, Lq=777,
             Lkv=5037, d=64, causal=True, n_sel=9, n_first=1, n_local=1),
        # the selection of one decode step at 32K
        dict(name="select_step_b32", op="select_decode", B=32, Hq=32, Hkv=8,
             L=32768, d=128, n_sel=64, n_first=1, n_local=2),
        # prompt attention over the selection (2K of up to 16K keys a row)
        dict(name="prefill_16k", op="prefill", B=1, Hq=32, Hkv=8, Lq=16384,
             Lkv=16384, d=128, causal=True, n_sel=32, n_first=1, n_local=2),
        # a chunk of a prompt against a longer cache, 8 heads per KV head
        dict(name="prefill_chunk_ragged", op="prefill", B=1, Hq=16, Hkv=2,
             Lq=1531, Lkv=4099, d=64, causal=True, n_sel=12, n_first=1,
             n_local=1),
        # a training step of the attention: forward and gradients
        dict(name="train_8k", op="train", B=1, Hq=32, Hkv=8, Lq=8192, Lkv=8192,
             d=128, causal=True, n_sel=16, n_first=1, n_local=2),
        # the same without a causal mask, one head per KV head, odd length
        dict(name="train_ragged", op="train", B=2, Hq=6, Hkv=6, Lq=1289,
             Lkv=1289, d=128, causal=False, n_sel=7, n_first=1, n_local=1),
        # one decode step of a serving batch over 4K of up to 32K keys
        dict(name="decode_b32", op="decode", B=32, Hq=32, Hkv=8, L=32768,
             d=128, page=64, n_sel=64, n_first=1, n_local=2),
        # one long sequence alone, small pages: latency counts
        dict(name="decode_b1_128k", op="decode", B=1, Hq=32, Hkv=4, L=131071,
             d=128, page=16, n_sel=32, n_first=1, n_local=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["means", "means_paged", "select", "select_decode",
                     "prefill", "train", "decode"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "means":
        return dict(op=op, B=rng.randint(1, 4), Hkv=Hkv, L=_log(rng, 1, 16384),
                    d=d)
    if op == "means_paged":
        L = _log(rng, 64, 32768)
        return dict(op=op, B=rng.randint(1, 32), Hkv=Hkv, L=L, d=d,
                    page=rng.choice([16, 32, 64, 128, 256]),
                    n_new=rng.choice([1, 2, 65, 500]))
    n_sel = rng.randint(4, 32)
    n_first, n_local = rng.randint(0, 2), rng.randint(1, 2)
    if op in ("select_decode", "decode"):
        G = rng.choice([1, 2, 4, 8])
        case = dict(op=op, B=rng.randint(1, 32), Hq=Hkv * G, Hkv=Hkv,
                    L=_log(rng, 128, 32768), d=d, n_sel=rng.randint(4, 64),
                    n_first=n_first, n_local=n_local)
        if op == "decode":
            case["page"] = rng.choice([16, 32, 64, 128, 256])
        else:  # more blocks than slots, so that there is something to choose
            case["L"] = _log(rng, 2048, 32768)
            case["n_sel"] = rng.randint(5, min(64, case["L"] // (3 * BLK)))
        return case
    hi = 8192 if op != "train" else 4096
    G = rng.choice([1, 2, 4, 8])
    Lkv = _log(rng, 65 if op != "select" else 1024, hi)
    if op == "select":
        n_sel = rng.randint(5, min(32, Lkv // (3 * BLK)))
    Lq = Lkv if (op == "train" or rng.random() < 0.5) else _log(rng, 1, Lkv)
    return dict(op=op, B=rng.randint(1, 2), Hq=Hkv * G, Hkv=Hkv, Lq=Lq,
                Lkv=Lkv, d=128 if op == "train" else d,
                causal=rng.random() < 0.75, n_sel=n_sel, n_first=n_first,
                n_local=n_local)


def _blocks(L):
    return -(-L // BLK)


def _lens(case):
    """Ragged sequence lengths of a serving batch, longest first: between
    half of L and L (a function of the case alone)."""
    L = case["L"]
    return [L - (977 * b) % max(L // 2, 1) for b in range(case["B"])]


def _row_last(case):
    """Last visible key of each prompt row."""
    Lq, Lkv = case["Lq"], case["Lkv"]
    return [r + Lkv - Lq if case["causal"] else Lkv - 1 for r in range(Lq)]


def work(case):
    op, d, B = case["op"], case["d"], case["B"]
    if op == "means":
        n = B * case["Hkv"] * d
        return dict(bytes=2 * n * (case["L"] + _blocks(case["L"])),
                    flops=n * case["L"])
    if op == "means_paged":
        rows = blks = 0
        for L in _lens(case):
            j0 = max(0, L - case["n_new"]) // BLK
            rows += L - j0 * BLK
            blks += _blocks(L) - j0
        n = case["Hkv"] * d
        return dict(bytes=2 * n * (rows + blks), flops=n * rows)
    Hq, Hkv, n_sel = case["Hq"], case["Hkv"], case["n_sel"]
    G = Hq // Hkv
    if op == "select_decode":
        blks = sum(_blocks(L) for L in _lens(case))
        return dict(bytes=2 * d * (B * Hq + Hkv * blks) + 4 * B * Hkv * n_sel,
                    flops=2 * d * Hkv * blks + B * Hq * d)
    if op == "decode":
        rows = 0
        for L in _lens(case):
            nb = min(n_sel, _blocks(L))
            rows += min(nb * BLK, L) - (_blocks(L) * BLK - L if nb < _blocks(L)
                                        else 0)
        return dict(bytes=4 * d * Hkv * rows + 4 * d * B * Hq
                    + 4 * B * Hkv * n_sel, flops=4 * d * Hq * rows)
    Lq, Lkv = case["Lq"], case["Lkv"]
    last = _row_last(case)
    q_bytes = 2 * B * Hq * Lq * d
    kv_bytes = 2 * B * Hkv * Lkv * d
    sel_bytes = 4 * B * Hkv * Lq * n_sel
    if op == "select":
        pairs = sum(x // BLK + 1 for x in last)
        return dict(bytes=q_bytes + 2 * B * Hkv * _blocks(Lkv) * d + sel_bytes,
                    flops=2 * d * B * Hkv * pairs + B * Hq * Lq * d)
    # the last block a row sees is always selected and ends at its last key
    keys = 0
    for x in last:
        nb = min(n_sel, x // BLK + 1)
        keys += (nb - 1) * BLK + x % BLK + 1
    fl = 4 * d * B * Hq * keys
    if op == "prefill":
        return dict(bytes=2 * q_bytes + 2 * kv_bytes + sel_bytes
                    + 4 * B * Hq * Lq, flops=fl)
    # forward, then five products of the same size backward; q, k, v, dout,
    # sel in, o, lse, dq, dk, dv out
    return dict(bytes=4 * q_bytes + 4 * kv_bytes + sel_bytes + 4 * B * Hq * Lq,
                flops=fl * 7 // 2)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _keys(g, B, Hkv, L, d):
    """Keys with a common direction per block neighbourhood (nearby tokens of
    a context resemble one another) plus noise of their own."""
    base = _randn(g, B, Hkv, L // 256 + 1, d).repeat_interleave(256, dim=2)
    return (0.7 * base[:, :, :L] + 0.7 * _randn(g, B, Hkv, L, d)).bfloat16()


def _pages(g, case, lens):
    """A page pool and its shuffled block table: [P, 2, Hkv, page, d]."""
    ps, Hkv, d, B = case["page"], case["Hkv"], case["d"], case["B"]
    npg = [-(-L // ps) for L in lens]
    P = sum(npg) + 1
    pool = torch.randn(P, 2, Hkv, ps, d, generator=g, device="cuda",
                       dtype=torch.bfloat16)
    perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, max(npg)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(npg):
        table[b, :n] = perm[at:at + n]
        at += n
    return pool, table


def _pick(score, cand, forced, n_sel):
    """The n_sel best candidates of each row (forced ones first, ties to the
    lowest index), ascending, -1 in the slots left over."""
    nb = score.shape[-1]
    s = torch.where(forced, math.inf, torch.where(cand, score, -math.inf))
    top = torch.sort(s, dim=-1, descending=True, stable=True).indices
    top = top[..., :n_sel]
    ok = torch.gather(cand, -1, top)
    top = torch.sort(torch.where(ok, top, nb), dim=-1).values
    top = torch.where(top < nb, top, -1)
    if top.shape[-1] < n_sel:
        pad = top.new_full((*top.shape[:-1], n_sel - top.shape[-1]), -1)
        top = torch.cat([top, pad], dim=-1)
    return top.to(torch.int32)


def _visible(last_block, nb, n_first, n_local):
    """Candidate and forced blocks of rows whose last visible block is given
    ([rows] -> [rows, nb])."""
    j = torch.arange(nb, device=last_block.device)
    lb = last_block[:, None]
    cand = j <= lb
    return cand, cand & ((j < n_first) | (j > lb - n_local))


def _last_blocks(case):
    return torch.tensor([x // BLK for x in _row_last(case)], device="cuda")


def _selection(g, case):
    """A selection as a trained score gives it: neighbouring rows mostly
    agree, with differences of their own."""
    B, Hkv, Lq, nb = case["B"], case["Hkv"], case["Lq"], _blocks(case["Lkv"])
    cand, forced = _visible(_last_blocks(case), nb, case["n_first"],
                            case["n_local"])
    out = torch.empty(B, Hkv, Lq, case["n_sel"], dtype=torch.int32,
                      device="cuda")
    for b in range(B):
        for h in range(Hkv):
            base = _randn(g, Lq // 128 + 1, nb).repeat_interleave(128, dim=0)
            s = base[:Lq] + 0.25 * _randn(g, Lq, nb)
            out[b, h] = _pick(s, cand, forced, case["n_sel"])
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, B, d, Hkv = case["op"], case["B"], case["d"], case["Hkv"]
    st = dict(case=case)
    if op == "means":
        st["k"] = _keys(g, B, Hkv, case["L"], d)
        return st
    if op == "means_paged":
        lens = _lens(case)
        pool, st["table"] = _pages(g, case, lens)
        st["k_pages"] = pool[:, 0]
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["means"] = _randn(g, B, Hkv, _blocks(case["L"]), d).bfloat16()
        return st
    Hq = case["Hq"]
    if op in ("select_decode", "decode"):
        lens = _lens(case)
        nb = _blocks(case["L"])
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["q"] = _randn(g, B, Hq, d).bfloat16()
        if op == "select_decode":
            st["means"] = (0.5 * _randn(g, B, Hkv, nb, d)).bfloat16()
            return st
        pool, st["table"] = _pages(g, case, lens)
        st["k_pages"], st["v_pages"] = pool[:, 0], pool[:, 1]
        last = torch.tensor([_blocks(L) - 1 for L in lens], device="cuda")
        cand, forced = _visible(last, nb, case["n_first"], case["n_local"])
        st["sel"] = _pick(_randn(g, B, Hkv, nb), cand[:, None].expand(
            B, Hkv, nb), forced[:, None].expand(B, Hkv, nb), case["n_sel"])
        return st
    Lq, Lkv = case["Lq"], case["Lkv"]
    st["q"] = _randn(g, B, Hq, Lq, d).bfloat16()
    if op == "select":
        st["means"] = (0.5 * _randn(g, B, Hkv, _blocks(Lkv), d)).bfloat16()
        return st
    st["k"] = _keys(g, B, Hkv, Lkv, d)
    st["v"] = _randn(g, B, Hkv, Lkv, d).bfloat16()
    st["sel"] = _selection(g, case)
    if op == "train":
        st["dout"] = _randn(g, B, Hq, Lq, d).bfloat16()
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(st):
    import dynamic_block_sparse_fa_b200 as bl
    case = st["case"]
    op = case["op"]
    if op == "means":
        return bl.blasst_block_means(st["k"])
    if op == "means_paged":
        return bl.blasst_block_means_paged(
            st["k_pages"], st["table"], st["lens"], st["means"],
            max_seq_len=case["L"], n_new=case["n_new"])
    if op == "select":
        return bl.blasst_block_select(
            st["q"], st["means"], case["Lkv"], causal=case["causal"],
            n_sel=case["n_sel"], n_first=case["n_first"],
            n_local=case["n_local"])
    if op == "select_decode":
        return bl.blasst_block_select_decode(
            st["q"], st["means"], st["lens"], n_sel=case["n_sel"],
            n_first=case["n_first"], n_local=case["n_local"])
    if op == "decode":
        return bl.blasst_select_decode_paged(
            st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
            st["sel"], max_seq_len=case["L"])
    o, lse = bl.blasst_select_prefill(st["q"], st["k"], st["v"], st["sel"],
                                      causal=case["causal"])
    if op == "prefill":
        return o, lse
    dq, dk, dv = bl.blasst_select_prefill_backward(
        st["q"], st["k"], st["v"], o, lse, st["dout"], st["sel"],
        causal=case["causal"])
    return o, lse, dq, dk, dv


def _rows_allowed(case, sel_bh, r0, r1):
    """[r1-r0, Lkv] bool: keys the rows' selections and the causal limit
    leave."""
    Lkv = case["Lkv"]
    nb = _blocks(Lkv)
    sel = sel_bh[r0:r1].long()
    hit = torch.zeros(r1 - r0, nb + 1, dtype=torch.bool, device=sel.device)
    hit.scatter_(1, torch.where(sel >= 0, sel, nb), True)
    allow = hit[:, :nb].repeat_interleave(BLK, dim=1)[:, :Lkv]
    if case["causal"]:
        c = torch.arange(Lkv, device=sel.device)
        r = torch.arange(r0, r1, device=sel.device) + Lkv - case["Lq"]
        allow = allow & (c <= r[:, None])
    return allow


def _run_plain(st):
    case = st["case"]
    op, d = case["op"], case["d"]
    if op == "means":
        k = st["k"].float()
        L = case["L"]
        full = L // BLK
        out = [k[:, :, :full * BLK].unflatten(2, (full, BLK)).mean(3)] \
            if full else []
        if L % BLK:
            out.append(k[:, :, full * BLK:].mean(2, keepdim=True))
        return torch.cat(out, dim=2).bfloat16()
    if op == "means_paged":
        ps = case["page"]
        for b, L in enumerate(_lens(case)):
            j0 = max(0, L - case["n_new"]) // BLK
            t = torch.arange(j0 * BLK, L, device="cuda")
            page = st["table"][b, t // ps].long()
            rows = st["k_pages"][page, :, t % ps].float()
            blk = t // BLK - j0
            nb = _blocks(L) - j0
            s = torch.zeros(nb, *rows.shape[1:], device="cuda")
            s.index_add_(0, blk, rows)
            n = torch.bincount(blk, minlength=nb).float()
            st["means"][b, :, j0:j0 + nb] = (
                s / n[:, None, None]).transpose(0, 1).bfloat16()
        return st["means"]
    B, Hq, Hkv, n_sel = case["B"], case["Hq"], case["Hkv"], case["n_sel"]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d)
    if op == "select":
        last = _last_blocks(case)
        q = st["q"].double().unflatten(1, (Hkv, G)).sum(2)
        out = []
        for b in range(B):
            for h in range(Hkv):
                s = q[b, h] @ st["means"][b, h].double().T
                cand, forced = _visible(last, s.shape[-1], case["n_first"],
                                        case["n_local"])
                out.append(_pick(s, cand, forced, n_sel))
        return torch.stack(out).unflatten(0, (B, Hkv))
    if op == "select_decode":
        q = st["q"].double().unflatten(1, (Hkv, G)).sum(2)
        s = (st["means"].double() @ q[..., None])[..., 0]
        last = (st["lens"].long() - 1) // BLK
        cand, forced = _visible(last, s.shape[-1], case["n_first"],
                                case["n_local"])
        return _pick(s, cand[:, None].expand_as(s),
                     forced[:, None].expand_as(s), n_sel)
    if op == "decode":
        ps = case["page"]
        o = torch.empty(B, Hq, d, device="cuda", dtype=torch.bfloat16)
        lse = torch.empty(B, Hq, device="cuda")
        key = torch.arange(BLK, device="cuda")
        hs = torch.arange(Hkv, device="cuda")[:, None]
        for b in range(B):
            sel = st["sel"][b].long()
            t = (sel.clamp(min=0)[..., None] * BLK + key).flatten(1)
            ok = (sel >= 0).repeat_interleave(BLK, dim=1)
            ok &= t < st["lens"][b]
            t = torch.where(ok, t, 0)
            page = st["table"][b][t // ps].long()
            k = st["k_pages"][page, hs, t % ps].float()
            v = st["v_pages"][page, hs, t % ps].float()
            q = st["q"][b].float().unflatten(0, (Hkv, G))
            s = scale * (q @ k.transpose(1, 2))
            s = s.masked_fill(~ok[:, None], -math.inf)
            m = s.amax(-1, keepdim=True)
            p = torch.exp(s - m)
            den = p.sum(-1, keepdim=True)
            o[b] = ((p @ v) / den).flatten(0, 1).bfloat16()
            lse[b] = (m + torch.log(den)).flatten()
        return o, lse
    Lq, Lkv = case["Lq"], case["Lkv"]
    train = op == "train"
    o = torch.empty_like(st["q"])
    lse = torch.empty(B, Hq, Lq, device="cuda")
    if train:
        dq = torch.empty_like(st["q"])
        dk, dv = torch.empty_like(st["k"]), torch.empty_like(st["v"])
    step = 512
    for b in range(B):
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            k, v = st["k"][b, h].float(), st["v"][b, h].float()
            if train:
                dk32, dv32 = torch.zeros_like(k), torch.zeros_like(v)
            for r0 in range(0, Lq, step):
                r1 = min(r0 + step, Lq)
                n = r1 + Lkv - Lq if case["causal"] else Lkv
                allow = _rows_allowed(case, st["sel"][b, h], r0, r1)[:, :n]
                q = st["q"][b, hq, r0:r1].float()
                s = scale * (q @ k[:n].T)
                s = s.masked_fill(~allow, -math.inf)
                m = s.amax(-1, keepdim=True)
                p = torch.exp(s - m)
                den = p.sum(-1, keepdim=True)
                p = p / den
                ob = p @ v[:n]
                o[b, hq, r0:r1] = ob.bfloat16()
                lse[b, hq, r0:r1] = (m + torch.log(den))[..., 0]
                if train:
                    do = st["dout"][b, hq, r0:r1].float()
                    dv32[:n] += torch.einsum("grk,grd->kd", p, do)
                    dp = do @ v[:n].T
                    ds = p * (dp - (do * ob).sum(-1, keepdim=True))
                    dq[b, hq, r0:r1] = (scale * (ds @ k[:n])).bfloat16()
                    dk32[:n] += scale * torch.einsum("grk,grd->kd", ds, q)
            if train:
                dk[b, h], dv[b, h] = dk32.bfloat16(), dv32.bfloat16()
    return (o, lse, dq, dk, dv) if train else (o, lse)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    op, d, B, Hkv = case["op"], case["d"], case["B"], case["Hkv"]
    if op == "means":
        L, nb = case["L"], _blocks(case["L"])
        k = torch.zeros(B, Hkv, nb * BLK, d, dtype=torch.float64,
                        device="cuda")
        k[:, :, :L] = st["k"]
        n = torch.full((nb, 1), float(BLK), dtype=torch.float64, device="cuda")
        n[-1] = L - (nb - 1) * BLK
        return k.view(B, Hkv, nb, BLK, d).sum(3) / n
    if op == "means_paged":
        out = st["means"].double()
        ps = case["page"]
        for b, L in enumerate(_lens(case)):
            for j in range(max(0, L - case["n_new"]) // BLK, _blocks(L)):
                acc, n = 0.0, 0
                for t0 in range(j * BLK, min((j + 1) * BLK, L), min(ps, BLK)):
                    t1 = min(t0 + min(ps, BLK), L)
                    page = int(st["table"][b, t0 // ps])
                    acc = acc + st["k_pages"][page, :, t0 % ps:t0 % ps + t1
                                              - t0].double().sum(1)
                    n += t1 - t0
                out[b, :, j] = acc / n
        return out
    Hq, n_sel = case["Hq"], case["n_sel"]
    G = Hq // Hkv
    scale = 1.0 / math.sqrt(d)
    if op in ("select", "select_decode"):
        # rank of every block by counting the better ones
        q, c = st["q"].double(), st["means"].double()
        if op == "select_decode":
            q = q[:, :, None]
            lasts = [[(L - 1) // BLK] for L in _lens(case)]
        else:
            lasts = [[x // BLK for x in _row_last(case)]] * B
        nb, R = c.shape[2], q.shape[2]
        out = torch.full((B, Hkv, R, n_sel), -1, dtype=torch.int32,
                         device="cuda")
        j = torch.arange(nb, device="cuda")
        for b in range(B):
            last = torch.tensor(lasts[b], device="cuda")[:, None]
            for h in range(Hkv):
                s = sum(q[b, h * G + g] @ c[b, h].T for g in range(G))
                # class 0: always taken, 1: by score, 2: not visible
                cls = torch.where(j > last, 2, 1)
                cls = torch.where((cls == 1) & ((j < case["n_first"])
                                                | (last - j < case["n_local"])),
                                  0, cls)
                best = torch.argsort(-s, dim=1, stable=True)
                cls_o = torch.gather(cls, 1, best)
                best = torch.gather(best, 1, torch.argsort(cls_o, dim=1,
                                                           stable=True))
                m = min(n_sel, nb)
                pos = torch.arange(m, device="cuda")
                top = torch.where(pos <= last, best[:, :m], nb + 1)
                top = top.sort(dim=1).values
                out[b, h, :, :m] = torch.where(top > nb, -1, top).int()
        return out[:, :, 0] if op == "select_decode" else out
    key = torch.arange(BLK, device="cuda")
    if op == "decode":
        ps = case["page"]
        o = torch.empty(B, Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(B, Hq, dtype=torch.float64, device="cuda")
        for b, L in enumerate(_lens(case)):
            for h in range(Hkv):
                sel = st["sel"][b, h]
                t = (sel[sel >= 0].long()[:, None] * BLK + key).flatten()
                t = t[t < L]
                page = st["table"][b].long()[t // ps]
                k = st["k_pages"][page, h, t % ps].double()
                v = st["v_pages"][page, h, t % ps].double()
                s = scale * (st["q"][b, h * G:(h + 1) * G].double() @ k.T)
                o[b, h * G:(h + 1) * G] = torch.softmax(s, -1) @ v
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
        return o, lse
    # prompt and training: gather each row's own keys
    Lq, Lkv = case["Lq"], case["Lkv"]
    train = op == "train"
    f64 = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.empty(B, Hq, Lq, d, **f64), torch.empty(B, Hq, Lq, **f64)
    if train:
        dq = torch.empty(B, Hq, Lq, d, **f64)
        dk, dv = (torch.zeros(B, Hkv, Lkv, d, **f64) for _ in range(2))
    step = max(1, (1 << 17) // (n_sel * BLK))
    for b in range(B):
        for h in range(Hkv):
            hq = slice(h * G, (h + 1) * G)
            k, v = st["k"][b, h].double(), st["v"][b, h].double()
            for r0 in range(0, Lq, step):
                r1 = min(r0 + step, Lq)
                sel = st["sel"][b, h, r0:r1].long()
                t = (sel.clamp(min=0)[..., None] * BLK + key).flatten(1)
                ok = (sel >= 0).repeat_interleave(BLK, dim=1) & (t < Lkv)
                if case["causal"]:
                    r = torch.arange(r0, r1, device="cuda") + Lkv - Lq
                    ok &= t <= r[:, None]
                t = torch.where(ok, t, 0)
                kt, vt = k[t], v[t]                        # [r, n, d]
                q = st["q"][b, hq, r0:r1].double().transpose(0, 1)
                s = scale * torch.bmm(q, kt.transpose(1, 2))
                s = torch.where(ok[:, None], s, -math.inf)
                le = torch.logsumexp(s, -1)
                p = torch.exp(s - le[..., None])
                ob = torch.bmm(p, vt)
                o[b, hq, r0:r1] = ob.transpose(0, 1)
                lse[b, hq, r0:r1] = le.T
                if train:
                    do = st["dout"][b, hq, r0:r1].double().transpose(0, 1)
                    dp = torch.bmm(do, vt.transpose(1, 2))
                    ds = scale * p * (dp - (do * ob).sum(-1, keepdim=True))
                    dq[b, hq, r0:r1] = torch.bmm(ds, kt).transpose(0, 1)
                    flat = t.flatten()
                    dv[b, h].index_add_(0, flat, torch.bmm(
                        p.transpose(1, 2), do).flatten(0, 1))
                    dk[b, h].index_add_(0, flat, torch.bmm(
                        ds.transpose(1, 2), q).flatten(0, 1))
    return (o, lse, dq, dk, dv) if train else (o, lse)
