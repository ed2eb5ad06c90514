"""Block-selected attention on the GPU against its float64 restatement.

Tolerances, from the arithmetic:
 - means: a float32 sum of at most 64 terms (64 * 2^-24 of the largest key),
   then one rounding to bf16 (2^-8 of the value).
 - selections are whole numbers and have to be equal.
 - o: p is rounded to bf16 (2^-8 of each term, so 2^-8 sum p|v|), o to bf16
   (2^-8 |o|); float32 scores of these sizes are off by less than 1e-4, which
   moves p by as much.
 - lse: that error of the scores, 1e-4, and 2^-22 of its own size.
 - gradients: P and dS are rounded to bf16 before their products, D uses the
   bf16 o, the sums are float32, the result is rounded to bf16: each term
   2^-8 relative, so max error 2e-2 of the largest entry and mean error 1e-2 of
   the mean entry (as the backward's own test).
"""
import math

import pytest
import torch

from synth.paged import paginate
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


def _check_means(got, ref, kmax):
    err = (got.double() - ref).abs()
    assert (err <= 2 ** -8 * ref.abs() + 64 * 2 ** -24 * kmax).all()


def _check_o(got, ref, lse=None, name=""):
    err = (got.double() - ref["o"]).abs()
    tol = (2 ** -8 + 1e-4) * ref["pv"] + 2 ** -8 * ref["o"].abs() + 1e-30
    assert (err <= tol).all(), (name, (err / tol).max().item())
    if lse is not None:
        empty = ref["lse"] == -math.inf
        assert ((lse == -math.inf) == empty).all(), name
        e = (lse.double() - ref["lse"])[~empty].abs()
        t = 1e-4 + 2 ** -22 * ref["lse"][~empty].abs()
        assert (e <= t).all(), (name, e.max().item())


def _check_grad(got, ref, name):
    err = (got.double() - ref).abs()
    mx, mean = ref.abs().max().item(), ref.abs().mean().item()
    assert err.max().item() <= 2e-2 * max(mx, 1e-9), (name, err.max(), mx)
    assert err.mean().item() <= 1e-2 * max(mean, 1e-12), (name, err.mean(), mean)


# ----------------------------------------------------------------------- means
@pytest.mark.parametrize("B,H,L,d", [
    (1, 1, 1, 128), (1, 1, 1, 64), (2, 3, 63, 64), (2, 2, 64, 128),
    (1, 5, 65, 128), (3, 2, 1000, 64), (2, 8, 4097, 128)])
def test_means(m, B, H, L, d):
    g = _gen(L + d)
    k = _rand(g, B, H, L, d) * 3
    got = m.blasst_block_means(k)
    _check_means(got, R.means(k), k.abs().max().item())
    _clean(m)


def test_means_nonfinite_stay_in_their_block(m):
    k = _rand(_gen(3), 1, 2, 200, 128)
    k[0, 0, 70, 5] = math.nan
    k[0, 1, 199, 0] = math.inf
    got = m.blasst_block_means(k)
    bad = ~torch.isfinite(got)
    assert bad[0, 0, 1, 5] and bad[0, 1, 3, 0] and bad.sum() == 2


@pytest.mark.parametrize("ps,d", [(16, 128), (32, 64), (64, 128), (128, 64),
                                  (256, 128)])
@pytest.mark.parametrize("n_new", [0, 1, 2, 64, 65, 300])
def test_means_paged(m, ps, d, n_new):
    lens = [0, 1, 63, 64, 65, 130, 700, 257]
    g = _gen(ps + n_new)
    k = _rand(g, len(lens), 2, 700, d)
    pg = paginate(k, k, lens, ps, seed=1, spare_pages=3,
                  poison=(math.nan, math.nan))
    nb = 12
    means = torch.full((len(lens), 2, nb, d), 7.0, dtype=BF, device="cuda")
    out = m.blasst_block_means_paged(pg.k_pages, pg.block_table, pg.seq_lens,
                                     means, n_new=n_new, max_seq_len=700)
    assert out.data_ptr() == means.data_ptr()
    _clean(m)
    for b, L in enumerate(lens):
        j0 = max(0, L - n_new) // 64 if n_new else 0
        if L:
            ref = R.means(k[b, :, :L])
            _check_means(means[b, :, j0:R.nblk(L)], ref[:, j0:],
                         k.abs().max().item())
        else:
            j0 = 0
        assert (means[b, :, :j0] == 7).all(), "blocks before stay"
        assert (means[b, :, R.nblk(L):] == 7).all(), "blocks behind stay"


def test_means_paged_bad_device_arguments(m):
    k = _rand(_gen(4), 2, 1, 128, 64)
    pg = paginate(k, k, [128, 128], 64, seed=1)
    means = torch.full((2, 1, 2, 64), 7.0, dtype=BF, device="cuda")
    bt = pg.block_table.clone()
    bt[1, 1] = pg.num_pages
    m.blasst_block_means_paged(pg.k_pages, bt, pg.seq_lens, means)
    st, where = m.blasst_check_device_error()
    assert st == 1 and where.startswith("101")
    assert (means[1, :, 1] == 7).all() and not (means[1, :, 0] == 7).any()
    bad = torch.tensor([129, -1], dtype=torch.int32, device="cuda")
    means.fill_(7)
    m.blasst_block_means_paged(pg.k_pages, pg.block_table, bad, means)
    st, where = m.blasst_check_device_error()
    assert st == 1 and where.startswith("100") and (means == 7).all()


# ------------------------------------------------------------------- selection
def _ref_select(q, c, Lkv, causal, n_sel, n_first, n_local):
    B, Hq, Lq, d = q.shape
    Hkv = c.shape[1]
    G = Hq // Hkv
    last = [(r + Lkv - Lq if causal else Lkv - 1) // 64 for r in range(Lq)]
    return torch.stack([torch.stack([
        R.select(q[b, h * G:(h + 1) * G].cpu(), c[b, h].cpu(), last, n_sel,
                 n_first, n_local) for h in range(Hkv)]) for b in range(B)])


SELECT = [  # B, Hq, Hkv, Lq, Lkv, d, causal, n_sel, n_first, n_local
    (1, 4, 1, 1, 1, 128, True, 1, 0, 1),
    (1, 1, 1, 5, 64, 64, False, 3, 1, 0),
    (2, 8, 2, 130, 1000, 128, True, 5, 1, 2),
    (1, 3, 1, 70, 1500, 64, True, 4, 0, 1),
    (1, 16, 1, 33, 2000, 128, False, 7, 0, 0),
    (1, 32, 1, 20, 3000, 64, True, 6, 2, 2),
    (1, 2, 2, 300, 300, 128, True, 64, 1, 1),
    (1, 4, 1, 90, 20000, 128, True, 33, 1, 2),     # 32-row tiles
    (1, 4, 2, 40, 60001, 64, True, 16, 1, 1),
    (1, 4, 1, 17, 131072, 128, True, 20, 1, 1),    # 16-row tiles, longest
]


@pytest.mark.parametrize("case", SELECT)
def test_select(m, case):
    B, Hq, Hkv, Lq, Lkv, d, causal, n, nf, nl = case
    g = _gen(Lkv + d)
    q = _rand(g, B, Hq, Lq, d)
    c = _rand(g, B, Hkv, R.nblk(Lkv), d)
    got = m.blasst_block_select(q, c, Lkv, n_sel=n, n_first=nf, n_local=nl,
                                causal=causal)
    _clean(m)
    assert torch.equal(got.cpu(), _ref_select(q, c, Lkv, causal, n, nf, nl))


@pytest.mark.parametrize("d", [64, 128])
def test_select_near_ties_and_ties(m, d):
    """Means that differ by single bf16 steps (scores closer than float32
    resolves), equal means, and rows of zeros: the float64 order decides,
    equal scores go to the lower index."""
    g = _gen(d)
    Lq, nb = 64, 200
    Lkv = nb * 64
    base = _rand(g, d).float()
    c = base.repeat(1, 1, nb, 1)
    pos = torch.randint(0, d, (nb,), generator=g, device="cuda")
    idx = torch.arange(nb, device="cuda")
    c[0, 0, idx, pos] *= 1 + 2.0 ** -7
    c = c.to(BF)
    c[0, 0, 50:60] = c[0, 0, 40:50]
    q = _rand(g, 1, 4, Lq, d)
    q[:, :, 7] = 0
    q[:, 1:, 9] = 0
    q[:, :, 11] *= 1e-15
    for causal in (True, False):
        got = m.blasst_block_select(q, c, Lkv, n_sel=17, causal=causal)
        assert torch.equal(got.cpu(), _ref_select(q, c, Lkv, causal, 17, 1, 1))
    c[:] = c[:, :, :1]
    got = m.blasst_block_select(q, c, Lkv, n_sel=17, causal=False)
    want = torch.tensor([*range(16), nb - 1], dtype=torch.int32)
    assert (got.cpu() == want).all()
    _clean(m)


def test_select_small_and_large_magnitudes(m):
    g = _gen(9)
    q = _rand(g, 1, 2, 40, 128)
    c = _rand(g, 1, 1, 50, 128)
    for fq, fc in ((1e-12, 1e-14), (1e18, 1e17), (2e36, 1.0)):
        qs, cs = q * fq, c * fc
        got = m.blasst_block_select(qs, cs, 3200, n_sel=9, causal=False)
        assert torch.equal(got.cpu(), _ref_select(qs, cs, 3200, False, 9, 1, 1))
    _clean(m)


def test_select_nonfinite(m):
    """NaN scores rank lowest, infinities where they belong, and values in
    blocks a row does not see change nothing."""
    g = _gen(10)
    q = _rand(g, 1, 2, 128, 64).abs()
    c = _rand(g, 1, 1, 32, 64)
    c[0, 0, 5] = math.nan
    c[0, 0, 7, 3] = math.inf
    c[0, 0, 9, 3] = -math.inf
    got = m.blasst_block_select(q, c, 2048, n_sel=8, n_first=0, causal=False)
    assert torch.equal(got.cpu(), _ref_select(q, c, 2048, False, 8, 0, 1))
    got = m.blasst_block_select(q, c, 2048, n_sel=32, n_first=0, causal=False)
    assert (got.cpu() == torch.arange(32, dtype=torch.int32)).all()
    clean = _rand(g, 1, 1, 32, 64)
    dirty = clean.clone()
    dirty[0, 0, 31] = math.nan           # the rows' own block: never scored
    q = q[:, :, :64].contiguous()
    a = m.blasst_block_select(q, clean, 2048, n_sel=8)
    b = m.blasst_block_select(q, dirty, 2048, n_sel=8)
    assert torch.equal(a, b)
    _clean(m)


@pytest.mark.parametrize("Hq,Hkv,d,n,nf,nl", [
    (4, 1, 128, 6, 1, 1), (8, 8, 64, 9, 0, 0), (32, 2, 128, 20, 2, 2),
    (6, 2, 64, 64, 1, 1)])
def test_select_decode(m, Hq, Hkv, d, n, nf, nl):
    lens = [0, 1, 64, 65, 640, 5000, 9999, 10000]
    nb = R.nblk(10000) + 3
    g = _gen(Hq + d)
    B, G = len(lens), Hq // Hkv
    q = _rand(g, B, Hq, d)
    c = _rand(g, B, Hkv, nb, d)
    for b, L in enumerate(lens):
        c[b, :, R.nblk(L):] = math.nan   # past the sequence: not read
    sl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = m.blasst_block_select_decode(q, c, sl, n_sel=n, n_first=nf,
                                       n_local=nl)
    _clean(m)
    for b, L in enumerate(lens):
        for h in range(Hkv):
            ref = R.select(q[b, h * G:(h + 1) * G, None].cpu(), c[b, h].cpu(),
                           [(L - 1) // 64 if L else -1], n, nf, nl)[0]
            assert torch.equal(got[b, h].cpu(), ref), (b, h)


def test_select_decode_ties_and_longest(m):
    g = _gen(12)
    L = 1 << 20
    nb = L // 64
    q = _rand(g, 1, 2, 64)
    c = _rand(g, 1, 1, nb, 64)
    c[0, 0, 8000:8100] = c[0, 0, 100:200] * 0 + c[0, 0, 77]
    sl = torch.tensor([L], dtype=torch.int32, device="cuda")
    got = m.blasst_block_select_decode(q, c, sl, n_sel=500)
    assert torch.equal(got[0, 0].cpu(), R.select(
        q[0, :, None].cpu(), c[0, 0].cpu(), [nb - 1], 500, 1, 1)[0])
    c[:] = 0
    got = m.blasst_block_select_decode(q, c, sl, n_sel=40, n_local=2)
    assert got[0, 0].tolist() == [*range(38), nb - 2, nb - 1]
    bad = torch.tensor([L + 1], dtype=torch.int32, device="cuda")
    got = m.blasst_block_select_decode(q, c, bad, n_sel=40)
    st, where = m.blasst_check_device_error()
    assert st == 1 and where.startswith("100") and (got == -1).all()


# --------------------------------------------------------------------- prefill
PREFILL = [  # B, Hq, Hkv, Lq, Lkv, d, causal, n_sel
    (1, 1, 1, 1, 1, 128, True, 1),
    (1, 4, 1, 1, 200, 64, True, 2),
    (2, 4, 2, 65, 65, 128, True, 2),
    (1, 8, 1, 129, 700, 128, True, 5),
    (1, 4, 4, 300, 300, 64, False, 3),
    (2, 16, 1, 77, 500, 128, True, 4),
    (1, 32, 1, 40, 1000, 64, True, 6),
    (1, 2, 1, 600, 2111, 128, True, 9),
    (1, 8, 2, 1000, 1000, 128, False, 16),
    (1, 4, 1, 520, 6000, 128, True, 70),
]


def _qkv(g, B, Hq, Hkv, Lq, Lkv, d):
    return (_rand(g, B, Hq, Lq, d), _rand(g, B, Hkv, Lkv, d),
            _rand(g, B, Hkv, Lkv, d))


@pytest.mark.parametrize("case", PREFILL)
def test_prefill(m, case):
    B, Hq, Hkv, Lq, Lkv, d, causal, n = case
    g = _gen(Lq * 7 + Lkv)
    q, k, v = _qkv(g, B, Hq, Hkv, Lq, Lkv, d)
    sel = R.random_selection(torch.Generator().manual_seed(Lkv), B, Hkv, Lq,
                             Lkv, n, causal, "cuda")
    scale = 1 / math.sqrt(d)
    o, lse = m.blasst_select_prefill(q, k, v, sel, causal=causal)
    _clean(m)
    _check_o(o, R.attention(q, k, v, sel, scale, causal), lse, case)


def _odd_selection(Lq, nb, seed, n_sel=6):
    """Repeated ids, unsorted, -1 between ids, blocks in a row's future, rows
    with nothing at all, and whole tiles with nothing."""
    g = torch.Generator().manual_seed(seed)
    sel = torch.randint(-2, nb, (1, 1, Lq, n_sel), generator=g).int()
    sel[..., 1] = sel[..., 0]
    sel[0, 0, 3::7] = -1
    sel[0, 0, 64:200] = -1
    return sel.cuda()


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_odd_lists(m, G, causal):
    Lq, Lkv, d = 333, 900, 128
    q, k, v = _qkv(_gen(G), 1, G, 1, Lq, Lkv, d)
    sel = _odd_selection(Lq, R.nblk(Lkv), G)
    ref = R.attention(q, k, v, sel, 0.1, causal)
    o = torch.full_like(q, 5.0)
    lse = torch.full((1, G, Lq), 5.0, device="cuda")
    m.blasst_select_prefill(q, k, v, sel, causal=causal, scale=0.1, o=o,
                            lse=lse)
    _clean(m)
    _check_o(o, ref, lse, G)
    empty = ref["lse"] == -math.inf
    assert empty.any() and (o[empty] == 0).all()


def test_prefill_nothing_selected(m):
    q, k, v = _qkv(_gen(1), 1, 4, 2, 100, 100, 64)
    sel = torch.full((1, 2, 100, 3), -1, dtype=torch.int32, device="cuda")
    o, lse = m.blasst_select_prefill(q, k, v, sel)
    _clean(m)
    assert (o == 0).all() and (lse == -math.inf).all()


def test_prefill_unselected_blocks_are_not_read(m):
    q, k, v = _qkv(_gen(2), 1, 4, 1, 256, 640, 128)
    sel = torch.tensor([1, 4, 9], dtype=torch.int32,
                       device="cuda").expand(1, 1, 256, 3).contiguous()
    ref = R.attention(q, k, v, sel, 0.1, False)
    for j in (0, 2, 3, 5, 6, 7, 8):
        k[:, :, j * 64:(j + 1) * 64] = math.nan
        v[:, :, j * 64:(j + 1) * 64] = math.inf
    o, lse = m.blasst_select_prefill(q, k, v, sel, causal=False, scale=0.1)
    _clean(m)
    _check_o(o, ref, lse)


def test_prefill_masked_keys_may_be_anything(m):
    """K of keys a row's mask hides (the row's future, other rows' blocks) may
    be infinite or NaN, and a query that is NaN stays in its own row."""
    q, k, v = _qkv(_gen(20), 1, 4, 1, 128, 128, 128)
    sel = torch.zeros(1, 1, 128, 1, dtype=torch.int32, device="cuda")
    sel[:, :, 64:] = 1
    ref = R.attention(q, k, v, sel, 0.1, True)
    k[0, 0, 127] = math.nan
    k[0, 0, 126, 3] = math.inf
    q[0, 2, 5] = math.nan
    o, lse = m.blasst_select_prefill(q, k, v, sel, scale=0.1)
    _clean(m)
    assert torch.isnan(o[0, 2, 5]).all()
    keep = torch.ones(1, 4, 128, dtype=torch.bool, device="cuda")
    keep[0, 2, 5] = False
    keep[:, :, 126:] = False
    sub = dict(o=ref["o"][keep], lse=ref["lse"][keep], pv=ref["pv"][keep])
    _check_o(o[keep], sub, lse[keep])


def test_prefill_bad_block_id(m):
    q, k, v = _qkv(_gen(3), 1, 4, 1, 64, 200, 64)
    sel = torch.zeros(1, 1, 64, 2, dtype=torch.int32, device="cuda")
    ref = R.attention(q, k, v, sel, 0.125, False)
    sel[0, 0, 17, 1] = 4
    o, lse = m.blasst_select_prefill(q, k, v, sel, causal=False)
    st, where = m.blasst_check_device_error()
    assert st == 1 and where.startswith("102") and "row 17" in where \
        and "id 4" in where
    _check_o(o, ref, lse)   # the bad id counts for nothing


def test_prefill_everything_selected_is_the_dense_prefill(m):
    q, k, v = _qkv(_gen(5), 1, 8, 2, 384, 640, 128)
    sel = torch.arange(10, dtype=torch.int32, device="cuda").expand(
        1, 2, 384, 10).contiguous()
    o, lse = m.blasst_select_prefill(q, k, v, sel)
    o2, lse2 = m.blasst_prefill(q, k, v, causal=True)
    _clean(m)
    assert (o.float() - o2.float()).abs().max() <= 2e-2
    assert (lse - lse2).abs().max() <= 1e-4


# -------------------------------------------------------------------- backward
BACKWARD = [  # B, Hq, Hkv, Lq, Lkv, causal, n_sel
    (1, 1, 1, 1, 1, True, 1),
    (1, 4, 1, 1, 130, True, 2),
    (1, 4, 2, 65, 65, True, 2),
    (2, 2, 2, 200, 321, True, 3),
    (1, 8, 1, 300, 300, False, 3),
    (1, 16, 1, 100, 700, True, 5),
    (1, 32, 1, 70, 400, True, 4),
    (1, 4, 1, 1000, 1000, True, 6),
    (1, 6, 6, 513, 513, False, 4),
]


def _train(m, q, k, v, sel, do, scale, causal):
    o, lse = m.blasst_select_prefill(q, k, v, sel, scale=scale, causal=causal)
    return m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel,
                                            scale=scale, causal=causal)


@pytest.mark.parametrize("case", BACKWARD)
def test_backward(m, case):
    B, Hq, Hkv, Lq, Lkv, causal, n = case
    g = _gen(Lq + 3 * Lkv)
    q, k, v = _qkv(g, B, Hq, Hkv, Lq, Lkv, 128)
    do = _rand(g, B, Hq, Lq, 128)
    sel = R.random_selection(torch.Generator().manual_seed(Lkv), B, Hkv, Lq,
                             Lkv, n, causal, "cuda")
    scale = 1 / math.sqrt(128)
    got = _train(m, q, k, v, sel, do, scale, causal)
    _clean(m)
    ref = R.attention(q, k, v, sel, scale, causal, do)
    for name, t in zip(("dq", "dk", "dv"), got):
        if case[4] == 1 and name != "dv":
            # one key: dS is 0 in exact arithmetic; what is left is the bf16
            # rounding of o in D, 2^-8 |o| |dO| summed over the columns
            bound = scale * 2 ** -7 * float(
                (do.double() * v.double()).abs().sum(-1).max()) \
                * float(k.abs().max() + q.abs().max())
            assert t.double().abs().max() <= bound
            continue
        _check_grad(t, ref[name], name)


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32])
@pytest.mark.parametrize("causal", [True, False])
def test_backward_odd_lists(m, G, causal):
    Lq, Lkv = 333, 900
    g = _gen(100 + G)
    q, k, v = _qkv(g, 1, G, 1, Lq, Lkv, 128)
    do = _rand(g, 1, G, Lq, 128)
    sel = _odd_selection(Lq, R.nblk(Lkv), G)
    sel[sel == 3] = 2                       # a block nobody selects
    o, lse = m.blasst_select_prefill(q, k, v, sel, scale=0.1, causal=causal)
    dq, dk, dv = (torch.full_like(t, 9.0) for t in (q, k, v))
    m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel, scale=0.1,
                                     causal=causal, dq=dq, dk=dk, dv=dv)
    _clean(m)
    ref = R.attention(q, k, v, sel, 0.1, causal, do)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_grad(t, ref[name], name)
    empty = ref["lse"] == -math.inf
    assert empty.any() and (dq[empty] == 0).all()
    assert (dk[:, :, 192:256] == 0).all() and (dv[:, :, 192:256] == 0).all()


def test_backward_against_differences(m):
    """The derivative along the gradient itself, by central differences of the
    float64 forward: <grad, grad> to the gradients' mean tolerance."""
    g = _gen(31)
    Lq = Lkv = 400
    x = _qkv(g, 1, 4, 2, Lq, Lkv, 128)
    do = _rand(g, 1, 4, Lq, 128)
    sel = R.random_selection(torch.Generator().manual_seed(5), 1, 2, Lq, Lkv,
                             3, True, "cuda")
    grads = _train(m, *x, sel, do, 0.1, True)
    _clean(m)
    h = 1e-4
    for i, gr in enumerate(grads):
        gd = gr.double()
        val = []
        for s in (h, -h):
            y = [t.double() for t in x]
            y[i] = y[i] + s * gd
            val.append((R.attention(*y, sel, 0.1, True)["o"]
                        * do.double()).sum())
        diff = ((val[0] - val[1]) / (2 * h)).item()
        want = (gd * gd).sum().item()
        assert abs(diff - want) <= 1e-2 * want, (i, diff, want)


def test_backward_bad_block_id(m):
    q, k, v = _qkv(_gen(3), 1, 4, 1, 64, 200, 128)
    sel = torch.zeros(1, 1, 64, 2, dtype=torch.int32, device="cuda")
    do = torch.ones_like(q)
    want = _train(m, q, k, v, sel, do, 0.1, False)
    o, lse = m.blasst_select_prefill(q, k, v, sel, scale=0.1, causal=False)
    _clean(m)
    sel[0, 0, 9, 1] = 1 << 20
    got = m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel, scale=0.1,
                                           causal=False)
    st, where = m.blasst_check_device_error()
    assert st == 1 and where.startswith("102")
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------- decode
LENS = [0, 1, 63, 64, 65, 200, 1000, 777]


def _decode_case(seed, Hq, Hkv, d, ps, n_sel, lens=LENS):
    g = _gen(seed)
    B, L = len(lens), max(lens)
    q = _rand(g, B, Hq, d)
    k, v = _rand(g, B, Hkv, L, d), _rand(g, B, Hkv, L, d)
    pg = paginate(k, v, lens, ps, seed=seed, spare_pages=2,
                  poison=(math.nan, math.nan))
    gc = torch.Generator().manual_seed(seed)
    sel = torch.full((B, Hkv, n_sel), -1, dtype=torch.int32)
    for b, ln in enumerate(lens):
        if ln:
            # random ids of the sequence's blocks: repeated and unsorted, with
            # -1 between them
            sel[b] = torch.randint(-1, R.nblk(ln), (Hkv, n_sel),
                                   generator=gc).int()
    return q, k, v, pg, sel.cuda()


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 2), (8, 2), (16, 2), (32, 2),
                                    (32, 1), (256, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_decode_heads(m, Hq, Hkv, d):
    q, k, v, pg, sel = _decode_case(Hq + d, Hq, Hkv, d, 64, 7)
    o, lse = m.blasst_select_decode_paged(q, pg.k_pages, pg.v_pages,
                                          pg.block_table, pg.seq_lens, sel)
    _clean(m)
    _check_o(o, R.decode(q, k, v, sel, LENS, 1 / math.sqrt(d)), lse)


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n_sel,S", [(1, 1), (9, 0), (9, 9), (140, 4),
                                     (512, 3)])
def test_decode_pages_and_splits(m, ps, d, n_sel, S):
    q, k, v, pg, sel = _decode_case(ps + n_sel, 8, 2, d, ps, n_sel)
    # pages nobody selected may hold any id
    bt = pg.block_table.clone()
    al = R.allowed(sel[:, :, None], 1, 1024, False)[:, :, 0].any(1)
    for b in range(len(LENS)):
        for p in range(bt.shape[1]):
            if not al[b, p * ps:(p + 1) * ps].any():
                bt[b, p] = 1 << 30
    o, lse = m.blasst_select_decode_paged(q, pg.k_pages, pg.v_pages, bt,
                                          pg.seq_lens, sel, num_splits=S)
    _clean(m)
    _check_o(o, R.decode(q, k, v, sel, LENS, 1 / math.sqrt(d)), lse)


def test_decode_interleaved_pool_and_slack(m):
    """K and V halves of one pool, and pages further apart than their rows."""
    q, k, v, pg, sel = _decode_case(77, 8, 2, 128, 32, 6)
    P = pg.num_pages
    pool = torch.full((P, 3, 2, 32, 128), math.nan, dtype=BF, device="cuda")
    pool[:, 0], pool[:, 1] = pg.k_pages, pg.v_pages
    o, lse = m.blasst_select_decode_paged(q, pool[:, 0], pool[:, 1],
                                          pg.block_table, pg.seq_lens, sel,
                                          max_seq_len=1000)
    _clean(m)
    _check_o(o, R.decode(q, k, v, sel, LENS, 1 / math.sqrt(128)), lse)


def test_decode_everything_selected_is_the_dense_decode(m):
    lens = [640, 333, 64]
    q, k, v, pg, _ = _decode_case(5, 8, 2, 128, 64, 1, lens)
    sel = torch.full((3, 2, 10), -1, dtype=torch.int32)
    for b, ln in enumerate(lens):
        sel[b, :, :R.nblk(ln)] = torch.arange(R.nblk(ln)).int()
    o, lse = m.blasst_select_decode_paged(q, pg.k_pages, pg.v_pages,
                                          pg.block_table, pg.seq_lens,
                                          sel.cuda())
    o2, lse2 = m.blasst_decode_paged(q, pg.k_pages, pg.v_pages, pg.block_table,
                                     pg.seq_lens)
    _clean(m)
    assert (o.float() - o2.float()).abs().max() <= 2e-2
    assert (lse - lse2).abs().max() <= 1e-4


def test_decode_bad_device_arguments(m):
    q, k, v, pg, sel = _decode_case(8, 4, 1, 64, 64, 4)

    def run(bt=pg.block_table, sl=pg.seq_lens, s=sel):
        m.blasst_select_decode_paged(q, pg.k_pages, pg.v_pages, bt, sl, s,
                                     max_seq_len=1000)
        return m.blasst_check_device_error()
    bad = sel.clone()
    bad[5] = 4                    # 200 tokens: blocks 0 .. 3
    st, where = run(s=bad)
    assert st == 1 and where.startswith("102") and "id 4" in where
    sl = pg.seq_lens.clone()
    sl[6] = 1001
    st, where = run(sl=sl)
    assert st == 1 and where.startswith("100")
    bt = pg.block_table.clone()
    bt[6] = -3
    st, where = run(bt=bt)
    assert st == 1 and where.startswith("101")
    st, where = run()
    assert st == 0


# -------------------------------------------------------- together, as it runs
def _chain_prompt(m, q, k, v, do, n_sel):
    c = m.blasst_block_means(k)
    sel = m.blasst_block_select(q, c, k.shape[2], n_sel=n_sel, n_local=2)
    o, lse = m.blasst_select_prefill(q, k, v, sel)
    return (c, sel, o, lse) + tuple(m.blasst_select_prefill_backward(
        q, k, v, o, lse, do, sel))


def test_training_step(m):
    """Means, selection, forward, backward; each stage against the reference
    on the stage's own inputs."""
    g = _gen(50)
    q, k, v = _qkv(g, 2, 8, 2, 700, 700, 128)
    do = _rand(g, 2, 8, 700, 128)
    c, sel, o, lse, dq, dk, dv = _chain_prompt(m, q, k, v, do, 5)
    _clean(m)
    _check_means(c, R.means(k), k.abs().max().item())
    assert torch.equal(sel.cpu(), _ref_select(q, c, 700, True, 5, 1, 2))
    ref = R.attention(q, k, v, sel, 1 / math.sqrt(128), True, do)
    _check_o(o, ref, lse)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_grad(t, ref[name], name)


def test_serving_steps_in_a_graph(m):
    """Three decode steps of a growing paged cache (append, means, selection,
    attention), captured once on a side stream and replayed."""
    B, Hq, Hkv, d, ps, n_sel = 4, 8, 2, 128, 16, 6
    L0 = [63, 500, 127, 1000]
    g = _gen(60)
    L = 1024
    k, v = _rand(g, B, Hkv, L, d), _rand(g, B, Hkv, L, d)
    pg = paginate(k, v, [L] * B, ps, seed=2)     # the pages to come are there
    lens = torch.tensor(L0, dtype=torch.int32, device="cuda")
    q = _rand(g, B, Hq, d)
    means = torch.zeros(B, Hkv, L // 64, d, dtype=BF, device="cuda")
    m.blasst_block_means_paged(pg.k_pages, pg.block_table, lens, means)
    sel = torch.empty(B, Hkv, n_sel, dtype=torch.int32, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, Hq, device="cuda")
    S = m.blasst_select_decode_splits(B, Hq, Hkv, n_sel)
    ws = torch.empty(m.blasst_decode_workspace_size(B, Hq, d, S),
                     dtype=torch.uint8, device="cuda")

    def step():
        lens.add_(1)
        m.blasst_block_means_paged(pg.k_pages, pg.block_table, lens, means,
                                   n_new=1)
        m.blasst_block_select_decode(q, means, lens, n_sel=n_sel, sel=sel)
        m.blasst_select_decode_paged(q, pg.k_pages, pg.v_pages, pg.block_table,
                                     lens, sel, o=o, lse=lse, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                    # warm up: the first token
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in range(2, 4):
        q.copy_(_rand(g, B, Hq, d))
        graph.replay()
        _clean(m)
        now = [x + t for x in L0]
        assert lens.tolist() == now
        for b, ln in enumerate(now):
            _check_means(means[b, :, :R.nblk(ln)], R.means(k[b, :, :ln]),
                         k.abs().max().item())
            for h in range(Hkv):
                ref = R.select(q[b, h * 4:(h + 1) * 4, None].cpu(),
                               means[b, h].cpu(), [(ln - 1) // 64], n_sel, 1, 1)
                assert torch.equal(sel[b, h].cpu(), ref[0])
        _check_o(o, R.decode(q, k, v, sel, now, 1 / math.sqrt(d)), lse)


def test_training_step_on_two_streams_and_in_a_graph(m):
    g = _gen(70)
    ins = []
    for _ in range(2):
        q, k, v = _qkv(g, 1, 4, 1, 400, 400, 128)
        ins.append((q, k, v, _rand(g, 1, 4, 400, 128)))
    want = [_chain_prompt(m, *x, 4) for x in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for i, s in enumerate(streams):
        with torch.cuda.stream(s):
            got[i] = _chain_prompt(m, *ins[i], 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _chain_prompt(m, *ins[0], 4)
    for t in captured:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    _clean(m)
    # dq (index 4) sums float32 in any order: equal to its bf16 rounding, two
    # neighbouring values at most, and a few float32 steps near zero
    for a, b in ((got[0], want[0]), (got[1], want[1]), (captured, want[0])):
        for i, (x, y) in enumerate(zip(a, b)):
            if i == 4:
                xd, yd = x.double(), y.double()
                assert ((xd - yd).abs() <= 2 ** -7 * yd.abs()
                        + 1e-6 * yd.abs().max()).all()
            else:
                assert torch.equal(x, y), i


def test_binding_refuses(m):
    q, k, v = _qkv(_gen(1), 1, 4, 1, 64, 64, 128)
    sel = torch.zeros(1, 1, 64, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        m.blasst_select_prefill(q, k, v, sel.long())
    with pytest.raises(TypeError):
        m.blasst_select_prefill(q.half(), k, v, sel)
    with pytest.raises(ValueError):
        m.blasst_select_prefill(q, k, v[:, :, :32], sel)
    with pytest.raises(ValueError):
        m.blasst_select_prefill(q, k, v, sel[:, :, :32])
    with pytest.raises(ValueError):
        m.blasst_select_prefill(q, k, v, sel, o=q)
    with pytest.raises(ValueError):
        m.blasst_select_prefill(q.transpose(1, 2).contiguous().transpose(1, 2),
                                k, v, sel)
    with pytest.raises(ValueError):
        m.blasst_select_prefill(q, k.cpu(), v, sel)
    with pytest.raises(ValueError):
        m.blasst_block_select(q, k[:, :, :2].contiguous(), 64, n_sel=2)
    with pytest.raises(m.BlasstError):
        m.blasst_select_prefill(q, k, v, sel, workspace=torch.empty(
            16, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------- what one might trip over
def test_results_are_the_same_bits_every_run(m):
    g = _gen(80)
    q, k, v = _qkv(g, 2, 8, 2, 900, 900, 128)
    do = _rand(g, 2, 8, 900, 128)
    a = _chain_prompt(m, q, k, v, do, 6)
    b = _chain_prompt(m, q, k, v, do, 6)
    _clean(m)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_stream_argument(m):
    """stream=s runs there; its workspace is not handed to the current stream
    while the call still uses it."""
    g = _gen(81)
    q, k, v = _qkv(g, 1, 8, 2, 2000, 2000, 128)
    do = _rand(g, 1, 8, 2000, 128)
    sel = R.random_selection(torch.Generator().manual_seed(8), 1, 2, 2000, 2000,
                             5, True, "cuda")
    o, lse = m.blasst_select_prefill(q, k, v, sel)
    want = m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        o2, lse2 = m.blasst_select_prefill(q, k, v, sel, stream=s)
        got = m.blasst_select_prefill_backward(q, k, v, o2, lse2, do, sel,
                                               stream=s)
        for _ in range(4):       # the current stream allocates and overwrites
            torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    _clean(m)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_offsets_past_32_bits(m):
    """Keys behind element 2^31 (contiguous), and pages behind element 2^32."""
    L = (1 << 31) // (2 * 128) + 1000
    k = torch.empty(1, 3, L, 128, dtype=BF, device="cuda")
    g = _gen(82)
    tail = _rand(g, 1000, 128)
    k[0, 2, -1000:] = tail
    c = m.blasst_block_means(k)
    nb = R.nblk(L)
    first = -(-(L - 1000) // 64)
    n = L - first * 64
    _check_means(c[0, 2, first:], R.means(tail[-n:]), tail.abs().max().item())
    del k, c
    P, H, ps, d = 40, 2, 64, 128
    stride = 1 << 27
    pool = torch.empty((P - 1) * stride + 2 * H * ps * d, dtype=BF,
                       device="cuda")
    pages = pool.as_strided((P, 2, H, ps, d),
                            (stride, H * ps * d, ps * d, d, 1))
    ids = [39, 33, 1, 38]
    kv = _rand(g, 2, H, 4 * ps, d)
    for i, x in enumerate(ids):
        pages[x] = kv[:, :, i * ps:(i + 1) * ps]
    bt = torch.tensor([ids], dtype=torch.int32, device="cuda")
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    means = torch.zeros(1, H, 4, d, dtype=BF, device="cuda")
    m.blasst_block_means_paged(pages[:, 0], bt, lens, means)
    _check_means(means[0], R.means(kv[0, :, :250]), kv.abs().max().item())
    q = _rand(g, 1, 8, d)
    sel = m.blasst_block_select_decode(q, means, lens, n_sel=3)
    o, lse = m.blasst_select_decode_paged(q, pages[:, 0], pages[:, 1], bt, lens,
                                          sel)
    _clean(m)
    _check_o(o, R.decode(q, kv[:1], kv[1:], sel, [250], 1 / math.sqrt(d)), lse)


@pytest.mark.parametrize("L", [64 * 250, 64 * 700, 64 * 1500, 64 * 4000])
def test_select_decode_lengths(m, L):
    """One warp's registers, and beyond them the whole CTA; near ties that
    only the exact score resolves among them."""
    g = _gen(L)
    nb = L // 64
    q = _rand(g, 2, 8, 128)
    c = _rand(g, 2, 2, nb, 128)
    c[1] = c[1, :, :1]
    at = torch.randint(0, 128, (nb,), generator=g, device="cuda")
    c[1, :, torch.arange(nb, device="cuda"), at] *= 1 + 2.0 ** -7
    lens = torch.tensor([L, L], dtype=torch.int32, device="cuda")
    got = m.blasst_block_select_decode(q, c, lens, n_sel=50, n_local=2)
    _clean(m)
    for b in range(2):
        for h in range(2):
            ref = R.select(q[b, h * 4:(h + 1) * 4, None].cpu(), c[b, h].cpu(),
                           [nb - 1], 50, 1, 2)[0]
            assert torch.equal(got[b, h].cpu(), ref), (b, h)


def test_select_scores_as_large_as_their_bound(m):
    """Queries along the means: the products of a score all have one sign, and
    the best scores crowd together."""
    g = _gen(84)
    base = _rand(g, 128).float()
    c = (base + 0.02 * torch.randn(1, 1, 300, 128, generator=g,
                                   device="cuda")).to(BF)
    q = (base + 0.02 * torch.randn(1, 4, 96, 128, generator=g,
                                   device="cuda")).to(BF)
    got = m.blasst_block_select(q, c, 19200, n_sel=40, causal=False)
    _clean(m)
    assert torch.equal(got.cpu(), _ref_select(q, c, 19200, False, 40, 1, 1))


@pytest.mark.parametrize("nb", [600, 2048])
def test_select_near_ties_of_long_rows(m, nb):
    """Rows of more blocks than a warp's registers hold."""
    g = _gen(nb)
    base = _rand(g, 128).float()
    c = base.repeat(1, 1, nb, 1)
    at = torch.randint(0, 128, (nb,), generator=g, device="cuda")
    c[0, 0, torch.arange(nb, device="cuda"), at] *= 1 + 2.0 ** -7
    c = c.to(BF)
    c[0, 0, 300:330] = _rand(g, 30, 128)
    c[0, 0, 500:520] = c[0, 0, 480:500]
    q = _rand(g, 1, 4, 24, 128)
    q[:, :, 3] = 0
    for n in (9, 45):
        got = m.blasst_block_select(q, c, nb * 64, n_sel=n, causal=False)
        _clean(m)
        assert torch.equal(got.cpu(),
                           _ref_select(q, c, nb * 64, False, n, 1, 1))


@pytest.mark.parametrize("G", [1, 4])
def test_longest_prompt_keys(m, G):
    """262144 keys: the whole range of block ids, lists as long as n_sel
    allows, forward and backward."""
    Lq, Lkv = 5, 262144
    g = _gen(90 + G)
    q, k, v = _qkv(g, 1, G, 1, Lq, Lkv, 128)
    do = _rand(g, 1, G, Lq, 128)
    sel = torch.full((1, 1, Lq, 4096), -1, dtype=torch.int32, device="cuda")
    sel[0, 0, 0, :3] = torch.tensor([0, 4095, 2047], device="cuda").int()
    sel[0, 0, 1] = torch.randint(0, 4096, (4096,), generator=g,
                                 device="cuda").int()
    sel[0, 0, 2, 4000:] = 17
    sel[0, 0, 4, ::2] = torch.arange(4095, 2047, -1, device="cuda").int()
    o, lse = m.blasst_select_prefill(q, k, v, sel, scale=0.05)
    got = m.blasst_select_prefill_backward(q, k, v, o, lse, do, sel, scale=0.05)
    _clean(m)
    ref = R.attention(q, k, v, sel, 0.05, True, do)
    _check_o(o, ref, lse, G)
    for name, t in zip(("dq", "dk", "dv"), got):
        _check_grad(t, ref[name], name)


def test_backward_unselected_blocks_may_hold_anything(m):
    """Infinities and NaN in K and V of blocks nobody selected, next to selected
    ones inside the same 128 keys: gradients of the others as without them,
    their own 0."""
    q, k, v = _qkv(_gen(95), 1, 4, 1, 256, 640, 128)
    do = _rand(_gen(96), 1, 4, 256, 128)
    sel = torch.tensor([1, 4, 9], dtype=torch.int32,
                       device="cuda").expand(1, 1, 256, 3).contiguous()
    sel[0, 0, 40:50] = -1
    ref = R.attention(q, k, v, sel, 0.1, False, do)
    for j in (0, 2, 3, 5, 6, 7, 8):
        k[:, :, j * 64:(j + 1) * 64] = math.nan
        v[:, :, j * 64:(j + 1) * 64] = math.inf
    dq, dk, dv = _train(m, q, k, v, sel, do, 0.1, False)
    _clean(m)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_grad(t, ref[name], name)
    hid = torch.ones(640, dtype=torch.bool, device="cuda")
    for j in (1, 4, 9):
        hid[j * 64:(j + 1) * 64] = False
    assert (dk[0, 0, hid] == 0).all() and (dv[0, 0, hid] == 0).all()
