"""Block-selected attention where its promises are easiest to break.

Selections are whole numbers and have to be equal.  Other tolerances are
derived where they are used.
"""
import math
import threading

import pytest
import torch

from tests import _select_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    import dynamic_block_sparse_fa_b200 as mod
    return mod


def _clean(m):
    torch.cuda.synchronize()
    st, where = m.blasst_check_device_error()
    assert st == 0, where


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rand(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


# ------------------------------------------------- weights far below the row's
def test_backward_of_weakly_weighted_keys(m):
    """Blocks whose keys score 12 to 20 nats below the others: their dK against
    its own rounding, not the largest gradient's.

    Per term of dK = scale sum_r dS_r q_r: dS is rounded to bf16 (2^-8 of it),
    D uses the bf16 o (2^-8 sum |o dO|), P = exp(s - lse) has the error of s
    and lse (products of these sizes, sum |q k| below 100, truncated at 2^-23
    of the partial sum in 8 steps: under 1e-3 together); the result is rounded
    to bf16.  Likewise dV with P to bf16."""
    Lq, Lkv, d = 64, 512, 128
    g = _gen(2)
    u = torch.zeros(d, device="cuda")
    u[5] = 1.0
    q = (4.0 * u + 0.3 * torch.randn(1, 1, Lq, d, generator=g,
                                     device="cuda")).to(BF)
    k = 0.3 * torch.randn(1, 1, Lkv, d, generator=g, device="cuda")
    for j, w in ((1, 3.0), (2, 4.0), (4, 5.0), (7, 4.5)):
        k[:, :, j * 64:(j + 1) * 64] -= w * u
    k, v = k.to(BF), _rand(g, 1, 1, Lkv, d)
    do = _rand(g, 1, 1, Lq, d)
    sel = torch.arange(8, dtype=torch.int32, device="cuda").expand(
        1, 1, Lq, 8).contiguous()
    o, lse = m.blasst_select_prefill(q, k, v, sel, scale=1.0, causal=False)
    dq, dk, dv = m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel,
                                                  scale=1.0, causal=False)
    _clean(m)
    qd, kd, vd, dod = (t[0, 0].double() for t in (q, k, v, do))
    s = qd @ kd.T
    p = torch.softmax(s, -1)
    low = p.view(Lq, 8, 64)[:, [1, 2, 4, 7]]
    assert low.max() < 1e-4 and low.min() < 1e-9 and low.median() < 1e-6
    od = p @ vd
    dp, D = dod @ vd.T, (dod * od).sum(-1, keepdim=True)
    ds = p * (dp - D)
    Dabs = (dod * od).abs().sum(-1, keepdim=True)
    e_ds = p * (2 ** -8 * (dp - D).abs() + 2 ** -8 * Dabs
                + 1e-3 * (dp.abs() + D.abs()))
    for name, got, ref, tol in (
            ("dk", dk, ds.T @ qd, e_ds.T @ qd.abs()),
            ("dv", dv, p.T @ dod, (2 ** -8 + 1e-3) * (p.T @ dod.abs())),
            ("dq", dq, ds @ kd, e_ds @ kd.abs())):
        err = (got[0, 0].double() - ref).abs()
        tol = tol * (1 + 2 ** -8) + 2 ** -8 * ref.abs()
        assert (err <= tol).all(), (name, (err / tol).max().item())


# ------------------------------------------ scores that only 64 bits tell apart
def _close_means(g, nb, d, f=1.0):
    """Means whose scores against a query agree to 2^-29 of their size: one
    vector, and in the last column 2^-30 (1 + x / 128) with x in some order."""
    c = torch.randn(d, generator=g, device="cuda").repeat(nb, 1)
    x = torch.randperm(nb, generator=g, device="cuda") % 128
    c[:, d - 1] = 2.0 ** -30 * (1 + x / 128)
    return (c.to(BF).float() * f).to(BF)


def _close_query(g, G, R_, d, f=1.0):
    q = torch.randn(G, R_, d, generator=g, device="cuda")
    q[..., d - 1] = q[..., d - 1].abs() + 0.5
    return (q.to(BF).float() * f).to(BF)


def _check_prompt(m, q, c, causal, n, off=0, nf=1, nl=1):
    G, Lq, _ = q.shape
    nb = c.shape[0]
    Lkv = Lq + off if causal else nb * 64
    assert R.nblk(Lkv) == nb
    got = m.blasst_block_select(q[None], c[None, None], Lkv, n_sel=n,
                                n_first=nf, n_local=nl, causal=causal)
    _clean(m)
    last = [(r + off if causal else Lkv - 1) // 64 for r in range(Lq)]
    want = R.select(q.cpu(), c.cpu(), last, n, nf, nl)
    assert torch.equal(got[0, 0].cpu(), want)


def _check_one(m, q, c, n):
    nb = c.shape[0]
    lens = torch.tensor([nb * 64], dtype=torch.int32, device="cuda")
    got = m.blasst_block_select_decode(q[:, 0].contiguous()[None], c[None, None], lens,
                                       n_sel=n)
    _clean(m)
    want = R.select(q[:, :1].cpu(), c.cpu(), [nb - 1], n, 1, 1)[0]
    assert torch.equal(got[0, 0].cpu(), want)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("odd", [math.nan, math.inf, -math.inf])
def test_select_close_scores_beside_a_nonfinite_mean(m, d, odd):
    """A mean that is infinite or NaN takes its own place; the others are
    still told apart beyond float32's resolution."""
    g = _gen(3)
    q = _close_query(g, 2, 40, d)
    c = _close_means(g, 100, d)
    c[30, 7] = odd
    _check_prompt(m, q, c, False, 20)
    # a block that only the last rows of a 16-row tile see, and one that no
    # row of the tile sees
    q2 = _close_query(g, 2, 500, d)
    for at in (50, 51, 55):
        c = _close_means(g, 59, d)
        c[at, 7] = odd
        # rows 0 .. 7 end in block 50, rows 8 .. 71 in block 51
        _check_prompt(m, q2, c, True, 20, off=64 * 51 - 8)
    for nb in (200, 400, 700, 1500):
        c = _close_means(g, nb, d)
        c[nb // 3, 7] = odd
        _check_one(m, q, c, 30)


def test_select_nan_below_minus_infinity(m):
    """A NaN score ranks below every other, -infinity among them."""
    c = torch.ones(70, 64, device="cuda", dtype=BF)
    q = torch.ones(1, 3, 64, device="cuda", dtype=BF)
    c[5, 0] = math.nan
    c[9:20, 0] = -math.inf
    want = torch.tensor([j for j in range(70) if j != 5], dtype=torch.int32)
    got = m.blasst_block_select(q[None], c[None, None], 70 * 64, n_sel=69,
                                causal=False)
    assert (got[0, 0].cpu() == want).all()
    lens = torch.tensor([70 * 64], dtype=torch.int32, device="cuda")
    got = m.blasst_block_select_decode(q[:, 0].contiguous()[None], c[None, None], lens,
                                       n_sel=69)
    _clean(m)
    assert (got[0, 0].cpu() == want).all()


@pytest.mark.parametrize("f", [1e8, 1e17, 1e30])
def test_select_close_scores_of_large_means(m, f):
    g = _gen(4)
    q = _close_query(g, 2, 20, 128)
    _check_prompt(m, q, _close_means(g, 90, 128, f), False, 20)
    _check_one(m, q, _close_means(g, 300, 128, f), 40)


@pytest.mark.parametrize("d", [64, 128])
def test_select_scores_the_tensor_core_cuts_most(m, d):
    """Two blocks whose float32 scores are in the wrong order by more than
    2^-17 |x| |c|: every product of the better one (A) but the first ends just
    below a multiple of 2^-25 of the sum, where the tensor core cuts it off,
    and so do those of the other (B), with the other sign."""
    n = d // 16                  # steps; a d of 64 loses half as much
    x = torch.full((d,), 2.0 ** -12)
    x[0], x[1] = 1.0, 2.0 ** -8
    under = 255 / 128            # the largest bf16 below 2
    a = torch.full((d,), under * 2.0 ** -13)
    a[15::16] /= 2               # 15 products of 1.99, one of 0.996 a step
    a[0], a[1] = 1.0, under * 2.0 ** -17
    for delta in range(356, 380, 4) if d == 128 else range(176, 192, 4):
        b = torch.full((d,), -under * 2.0 ** -14)
        b[0], b[1] = 1.0, delta * 2.0 ** -17
        sa, sb = (x.double() @ y.double() for y in (a, b))
        # (delta less what B loses below what A adds up to)
        want_a = bool(sa > sb)
        for swap in (False, True):
            c = torch.zeros(6, d)
            c[:, 0] = 0.5
            c[1], c[2] = (b, a) if swap else (a, b)
            cb = c.to(BF).cuda()
            assert torch.equal(cb.float().cpu(), c)
            q = x.repeat(1, 3, 1).to(BF).cuda()
            got = m.blasst_block_select(q[None], cb[None, None], 6 * 64,
                                        n_sel=3, causal=False)
            best = (1 if want_a else 2) if not swap else (2 if want_a else 1)
            assert got[0, 0].tolist() == [[0, best, 5]] * 3, (delta, swap, n)
    _clean(m)


# ---------------------------------------------------- the small end of float32
@pytest.mark.parametrize("fq,fc", [(1.0, 1e-20), (1.0, 1e-25), (1e-36, 1.0),
                                   (1e-20, 1e-19), (1e-25, 1e-28)])
def test_select_close_scores_of_small_values(m, fq, fc):
    """Scores near and below float32's smallest numbers are still ranked by
    their exact values."""
    g = _gen(5)
    q = _close_query(g, 2, 20, 128, fq)
    _check_prompt(m, q, _close_means(g, 90, 128, fc), False, 20)
    _check_one(m, q, _close_means(g, 300, 128, fc), 40)


# --------------------------------------------------------------- host threads
def _threads(calls, n):
    """Each C call n times on a host thread and stream of its own, all at once;
    a call is a function and its arguments but the stream."""
    failed = []
    start = threading.Barrier(len(calls))

    def loop(fn, args, stream):
        start.wait()
        for i in range(n):
            st = fn(*args, stream)
            if st:
                failed.append((fn.__name__, i, st))
                return
            if i % 256 == 255:      # bounds the launches in flight
                torch.cuda.current_stream().synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    ts = [threading.Thread(target=loop, args=(*c, s.cuda_stream))
          for c, s in zip(calls, streams)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed


@pytest.mark.parametrize("op", ["select", "select_decode", "prefill"])
def test_threads_with_different_lengths(m, op):
    """Host threads on the longest sequences beside others on short ones:
    none may disturb another's launch."""
    lib = m.blasst._lib
    g = _gen(1)
    keep = []               # what the raw pointers below point to

    def ptr(t):
        keep.append(t)
        return t.data_ptr()

    def make(L):
        if op == "select":
            out = torch.zeros(16, 3, dtype=torch.int32, device="cuda")
            return out, (lib.blasst_block_select, (
                ptr(_rand(g, 16, 64)), ptr(_rand(g, R.nblk(L), 64)), ptr(out),
                1, 1, 1, 16, L, 64, 0, 3, 1, 1))
        if op == "select_decode":
            out = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
            ln = torch.tensor([L], dtype=torch.int32, device="cuda")
            return out, (lib.blasst_block_select_decode, (
                ptr(_rand(g, 1, 64)), ptr(_rand(g, R.nblk(L), 64)), ptr(ln), L,
                R.nblk(L), ptr(out), 1, 1, 1, 64, 3, 1, 1))
        out = torch.zeros(8, 64, dtype=BF, device="cuda")
        n = m.blasst_select_prefill_workspace_size(1, 1, 1, 8, L)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        sel = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
        return out, (lib.blasst_select_prefill, (
            ptr(_rand(g, 8, 64)), ptr(_rand(g, L, 64)), ptr(_rand(g, L, 64)),
            ptr(sel), ptr(out), None, 1, 1, 1, 8, L, 64, 1, 0.1, 0, ptr(ws), n))
    L = {"select": 131072, "select_decode": 1 << 20, "prefill": 262144}[op]
    work = [make(L), make(640), make(64), make(L), make(1), make(640)]
    for out, (fn, args) in work:
        assert fn(*args, None) == 0
    torch.cuda.synchronize()
    want = [out.clone() for out, _ in work]
    for out, _ in work:
        out.zero_()
    torch.cuda.synchronize()
    _threads([call for _, call in work], 4000)
    _clean(m)
    for (out, _), w in zip(work, want):
        assert torch.equal(out, w)


# -------------------------------------------------- streams, graphs, same bits
def _step(m, q, k, v, do, n_sel):
    c = m.blasst_block_means(k)
    sel = m.blasst_block_select(q, c, k.shape[2], n_sel=n_sel, n_local=2)
    o, lse = m.blasst_select_prefill(q, k, v, sel)
    return (c, sel, o, lse) + tuple(m.blasst_select_prefill_backward(
        q, k, v, o, lse, do, sel))


def test_training_steps_have_the_same_bits_everywhere(m):
    """Every output, dq among them, sums in a fixed order: two streams at once,
    a side stream and a replayed graph give what one call alone gave."""
    g = _gen(70)
    ins = []
    for L in (400, 1100):
        ins.append((_rand(g, 1, 8, L, 128), _rand(g, 1, 2, L, 128),
                    _rand(g, 1, 2, L, 128), _rand(g, 1, 8, L, 128), 5))
    want = []
    for x in ins:
        want.append(_step(m, *x))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, captured = [], []
    for x in ins:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            captured.append(_step(m, *x))
    for _ in range(5):
        got = [None, None]
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got[i] = _step(m, *ins[i])
        torch.cuda.synchronize()
        for outs in captured:
            for t in outs:
                t.zero_()
        torch.cuda.synchronize()
        for i, s in enumerate(streams):     # both graphs at once
            with torch.cuda.stream(s):
                graphs[i].replay()
        torch.cuda.synchronize()
        for a, b, w in zip(got, captured, want):
            for name, x, y, z in zip("c sel o lse dq dk dv".split(), a, b, w):
                assert torch.equal(x, z) and torch.equal(y, z), name
    _clean(m)


@pytest.mark.parametrize("Hq,Hkv,Lq,Lkv,causal,n", [
    (8, 4, 161, 161, True, 3), (4, 1, 300, 700, True, 5),
    (2, 2, 90, 500, False, 3), (32, 1, 70, 1000, True, 7)])
def test_backward_dq_is_as_good_as_its_rounding(m, Hq, Hkv, Lq, Lkv, causal, n):
    """dQ against float64, 2-norms: the rounding of the result itself (bf16 of
    the exact gradient), and what is off before it by no more than
    1.3e-4 scale sum_c P_c (|dP_c| + |D|) |k_c| an entry: scores and lse are
    off by 5e-5 each (sum scale |q k| below 10, cut at 2^-25 of the sum, 21
    times in each of 8 steps, and the lse's logarithm), dP by the same share
    of sum |dO v| / |dP|, dS by 2^-16.  (dS as one bf16 number, or D from the
    bf16 o, would add as much again as the result's rounding.)"""
    g = _gen(Lq)
    B, d = 2, 128
    base = torch.randn(B, Hkv, Lkv // 256 + 1, d, generator=g, device="cuda")
    k = (0.7 * base.repeat_interleave(256, 2)[:, :, :Lkv] + 0.7 * torch.randn(
        B, Hkv, Lkv, d, generator=g, device="cuda")).to(BF)
    q, v = _rand(g, B, Hq, Lq, d), _rand(g, B, Hkv, Lkv, d)
    do = _rand(g, B, Hq, Lq, d)
    sel = R.random_selection(torch.Generator().manual_seed(Lq), B, Hkv, Lq,
                             Lkv, n, causal, "cuda")
    scale = 1 / math.sqrt(d)
    o, lse = m.blasst_select_prefill(q, k, v, sel, causal=causal)
    dq, _, _ = m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel,
                                                causal=causal)
    _clean(m)
    ref = R.attention(q, k, v, sel, scale, causal, do)
    G = Hq // Hkv
    kd, vd, dod, od = (t.double().repeat_interleave(r, 1) for t, r in (
        (k, G), (v, G), (do, 1), (ref["o"], 1)))
    al = R.allowed(sel, Lq, Lkv, causal).repeat_interleave(G, 1)
    s = scale * (q.double() @ kd.transpose(-1, -2))
    p = torch.where(al, torch.exp(s - ref["lse"][..., None]), 0.0)
    dp = dod @ vd.transpose(-1, -2)
    D = (dod * od).sum(-1, keepdim=True)
    before = 1.3e-4 * scale * (p * (dp.abs() + D.abs())) @ kd.abs()
    rounding = ref["dq"].to(BF).double() - ref["dq"]
    err = (dq.double() - ref["dq"]).norm()
    lim = rounding.norm() + before.norm()
    size = ref["dq"].norm()
    print(f"{(err / size).item():.5f} of {(lim / size).item():.5f}")
    assert err <= lim
