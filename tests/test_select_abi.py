"""Block-selected attention without a GPU: the float64 restatement the GPU
tests compare with is pinned by closed forms, and the C entry points refuse
bad arguments before any CUDA call."""
import ctypes
import math

import pytest
import torch

from tests import _select_ref as R

vp, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float,
                    ctypes.c_size_t)


@pytest.fixture(scope="module")
def lib():
    import dynamic_block_sparse_fa_b200.blasst as b
    return b._lib


# --------------------------------------------------------------- the reference
def test_reference_of_everything_selected_is_dense_attention():
    g = torch.Generator().manual_seed(0)
    q = torch.randn(1, 4, 70, 16, generator=g)
    k = torch.randn(1, 2, 200, 16, generator=g)
    v = torch.randn(1, 2, 200, 16, generator=g)
    sel = torch.arange(4, dtype=torch.int32).expand(1, 2, 70, 4)
    got = R.attention(q, k, v, sel, 0.25, False)
    for h in range(4):
        s = 0.25 * q[0, h].double() @ k[0, h // 2].double().T
        assert torch.allclose(got["o"][0, h], torch.softmax(s, -1)
                              @ v[0, h // 2].double())
        assert torch.allclose(got["lse"][0, h], torch.logsumexp(s, -1))


def test_reference_gradients_are_the_derivatives():
    g = torch.Generator().manual_seed(1)
    B, Hq, Hkv, Lq, Lkv, d = 1, 2, 1, 66, 130, 8
    q = torch.randn(B, Hq, Lq, d, generator=g).double().requires_grad_()
    k = torch.randn(B, Hkv, Lkv, d, generator=g).double().requires_grad_()
    v = torch.randn(B, Hkv, Lkv, d, generator=g).double().requires_grad_()
    do = torch.randn(B, Hq, Lq, d, generator=g).double()
    sel = R.random_selection(g, B, Hkv, Lq, Lkv, 2, True, "cpu")
    out = R.attention(q, k, v, sel, 0.3, True, do)
    grads = torch.autograd.grad((out["o"] * do).sum(), (q, k, v))
    for name, x in zip(("dq", "dk", "dv"), grads):
        assert torch.allclose(out[name], x, atol=1e-10), name


def test_reference_selection_by_hand():
    c = torch.tensor([[0.], [3.], [1.], [3.], [9.], [2.]])
    q = torch.ones(1, 3, 1)
    got = R.select(q, c, [5, 2, -1], 4, 1, 1)
    assert got.tolist() == [[0, 1, 4, 5], [0, 1, 2, -1], [-1] * 4]
    assert R.select(q, c, [5, 5, 5], 2, 0, 0)[0].tolist() == [1, 4]


def test_reference_empty_rows():
    q = torch.ones(1, 1, 2, 4)
    k = torch.ones(1, 1, 64, 4)
    sel = torch.tensor([[[[0], [-1]]]], dtype=torch.int32)
    r = R.attention(q, k, k, sel, 1.0, False, q)
    assert r["lse"][0, 0, 1] == -math.inf
    assert (r["o"][0, 0, 1] == 0).all() and (r["dq"][0, 0, 1] == 0).all()


# -------------------------------------------------------------------- refusals
P1, P2 = 0x1000, 0x2000


def _means(lib, k=P1, m=P2, B=1, Hkv=1, L=64, d=128):
    return lib.blasst_block_means(vp(k), vp(m), B, Hkv, L, d, None)


def test_block_means_refusals(lib):
    assert _means(lib, k=None) == 1 and _means(lib, m=None) == 1
    assert _means(lib, B=0) == 1 and _means(lib, L=0) == 1
    assert _means(lib, d=96) == 2
    assert _means(lib, B=1 << 20, Hkv=1 << 12) == 2
    assert _means(lib, k=0x1008) == 3 and _means(lib, m=0x2004) == 3


def _means_paged(lib, kp=P1, stride=64 * 128, pages=4, ps=64, bt=P1, mp=4,
                 sl=P1, msl=256, n_new=0, m=P2, mb=4, B=1, Hkv=1, d=128):
    return lib.blasst_block_means_paged(
        vp(kp), ctypes.c_longlong(stride), pages, ps, vp(bt), mp, vp(sl), msl,
        n_new, vp(m), mb, B, Hkv, d, None)


def test_block_means_paged_refusals(lib):
    for a in ("kp", "bt", "sl", "m"):
        assert _means_paged(lib, **{a: None}) == 1, a
    assert _means_paged(lib, n_new=-1) == 1
    assert _means_paged(lib, msl=257) == 1          # more than the table holds
    assert _means_paged(lib, mb=3) == 1             # more than means holds
    assert _means_paged(lib, stride=64 * 128 - 8) == 1
    assert _means_paged(lib, stride=64 * 128 + 4) == 1
    assert _means_paged(lib, ps=48) == 2 and _means_paged(lib, ps=512) == 2
    assert _means_paged(lib, d=32) == 2
    assert _means_paged(lib, kp=0x1002) == 3


def _select(lib, q=P1, m=P1, s=P2, B=1, Hq=4, Hkv=1, Lq=64, Lkv=128, d=128,
            causal=1, n=4, nf=1, nl=1):
    return lib.blasst_block_select(vp(q), vp(m), vp(s), B, Hq, Hkv, Lq, Lkv, d,
                                   causal, n, nf, nl, None)


def test_block_select_refusals(lib):
    for a in ("q", "m", "s"):
        assert _select(lib, **{a: None}) == 1, a
    assert _select(lib, Lq=129) == 1                # causal, Lq > Lkv
    assert _select(lib, nl=0) == 1                  # causal needs its own block
    assert _select(lib, n=1) == 1                   # forced blocks do not fit
    assert _select(lib, n=0, nf=0, nl=0) == 1
    assert _select(lib, nf=-1) == 1
    assert _select(lib, nf=0x7fffffff, nl=0x7fffffff) == 1
    assert _select(lib, Hq=3, Hkv=2) == 1
    assert _select(lib, d=96) == 2
    assert _select(lib, Hq=64) == 2                 # 64 heads per KV head
    assert _select(lib, Lkv=131073) == 2
    assert _select(lib, n=4097) == 2
    assert _select(lib, q=0x1008) == 3


def _select_dec(lib, q=P1, m=P1, sl=P1, msl=128, mb=2, s=P2, B=1, Hq=4, Hkv=1,
                d=128, n=4, nf=1, nl=1):
    return lib.blasst_block_select_decode(vp(q), vp(m), vp(sl), msl, mb, vp(s),
                                          B, Hq, Hkv, d, n, nf, nl, None)


def test_block_select_decode_refusals(lib):
    for a in ("q", "m", "sl", "s"):
        assert _select_dec(lib, **{a: None}) == 1, a
    assert _select_dec(lib, msl=129) == 1           # more than means holds
    assert _select_dec(lib, msl=0) == 1
    assert _select_dec(lib, n=1) == 1
    assert _select_dec(lib, msl=(1 << 20) + 1, mb=1 << 20) == 2
    assert _select_dec(lib, msl=0x7fffffff, mb=0x7fffffff) == 2
    assert _select_dec(lib, d=256) == 2
    assert _select_dec(lib, m=0x1004) == 3


def _prefill(lib, q=P1, k=P1, v=P1, s=P1, o=P2, B=1, Hq=4, Hkv=1, Lq=64,
             Lkv=128, d=128, n=4, scale=0.1, causal=1, ws=P2, wsb=1 << 40):
    return lib.blasst_select_prefill(vp(q), vp(k), vp(v), vp(s), vp(o), None,
                                     B, Hq, Hkv, Lq, Lkv, d, n, f32(scale),
                                     causal, vp(ws), sz(wsb), None)


def test_select_prefill_refusals(lib):
    for a in ("q", "k", "v", "s", "o"):
        assert _prefill(lib, **{a: None}) == 1, a
    assert _prefill(lib, n=0) == 1
    assert _prefill(lib, Lq=129) == 1
    for sc in (0.0, -1.0, math.inf, math.nan):
        assert _prefill(lib, scale=sc) == 1, sc
    assert _prefill(lib, Hq=3) == 2 and _prefill(lib, Hq=64) == 2
    assert _prefill(lib, d=192) == 2
    assert _prefill(lib, Lkv=262145) == 2 and _prefill(lib, n=4097) == 2
    assert _prefill(lib, o=0x2008) == 3
    assert _prefill(lib, ws=None) == 7 and _prefill(lib, wsb=16) == 7
    assert _prefill(lib, ws=0x2010) == 3


def _bwd(lib, drop=None, **kw):
    a = dict(B=1, Hq=4, Hkv=1, Lq=64, Lkv=128, d=128, n=4, scale=0.1, causal=1,
             ws=P2, wsb=1 << 40)
    a.update(kw)
    ptrs = [vp(None if x == drop else P1) for x in range(10)]
    return lib.blasst_select_prefill_backward(
        *ptrs, a["B"], a["Hq"], a["Hkv"], a["Lq"], a["Lkv"], a["d"], a["n"],
        f32(a["scale"]), a["causal"], vp(a["ws"]), sz(a["wsb"]), None)


def test_select_backward_refusals(lib):
    for x in range(10):
        assert _bwd(lib, drop=x) == 1, x
    assert _bwd(lib, scale=0.0) == 1 and _bwd(lib, Lq=200) == 1
    assert _bwd(lib, d=64) == 2 and _bwd(lib, Hq=6) == 2
    assert _bwd(lib, ws=None) == 7 and _bwd(lib, wsb=1024) == 7
    assert _bwd(lib, ws=0x2010) == 3


def _dec(lib, q=P1, kp=P1, vpg=P1, stride=64 * 128, pages=4, ps=64, bt=P1,
         mp=4, sl=P1, msl=256, s=P1, n=4, o=P2, B=1, Hq=4, Hkv=1, d=128,
         scale=0.1, S=1, ws=0x4000, wsb=1 << 30):
    return lib.blasst_select_decode_paged(
        vp(q), vp(kp), vp(vpg), ctypes.c_longlong(stride), pages, ps, vp(bt),
        mp, vp(sl), msl, vp(s), n, vp(o), None, B, Hq, Hkv, d, f32(scale), S,
        vp(ws), sz(wsb), None)


def test_select_decode_refusals(lib):
    for a in ("q", "kp", "vpg", "bt", "sl", "s", "o"):
        assert _dec(lib, **{a: None}) == 1, a
    assert _dec(lib, S=5) == 1 and _dec(lib, S=-1) == 1
    assert _dec(lib, msl=257) == 1 and _dec(lib, n=0) == 1
    assert _dec(lib, scale=0.0) == 1 and _dec(lib, stride=8) == 1
    assert _dec(lib, n=513) == 2 and _dec(lib, Hq=12, Hkv=4) == 2
    assert _dec(lib, d=96) == 2 and _dec(lib, ps=20) == 2
    assert _dec(lib, o=0x2008) == 3 and _dec(lib, ws=0x4010) == 3
    assert _dec(lib, ws=None) == 7 and _dec(lib, wsb=64) == 7


def test_host_policies(lib):
    import dynamic_block_sparse_fa_b200 as m
    for B, Hq, Hkv, n in ((1, 32, 4, 32), (32, 32, 8, 64), (1, 1, 1, 1),
                          (4, 256, 1, 100), (148, 64, 8, 512)):
        assert 1 <= m.blasst_select_decode_splits(B, Hq, Hkv, n) <= n
    assert m.blasst_select_decode_splits(0, 1, 1, 4) == 1
    # grows with every length, and holds what the lists need
    for f in (m.blasst_select_prefill_workspace_size,
              m.blasst_select_prefill_backward_workspace_size):
        a, b = f(1, 32, 8, 1024, 4096), f(2, 32, 8, 1024, 8192)
        assert 0 < a < b
        assert f(1, 6, 2, 64, 64) == 0 and f(0, 4, 1, 64, 64) == 0
    # G = 4: 32 tokens a tile; 65 blocks -> at least 65 ids and words a tile
    tiles = 2 * 5
    assert m.blasst_select_prefill_workspace_size(1, 8, 2, 130, 64 * 64 + 1) \
        >= tiles * (4 + 65 * 4 + 65 * 4)


def test_binding_refuses_what_the_abi_cannot_see():
    import dynamic_block_sparse_fa_b200 as m
    k = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16)
    sel = torch.zeros(1, 1, 64, 1, dtype=torch.int32)
    with pytest.raises(ValueError):                 # not on a GPU
        m.blasst_block_means(k)
    with pytest.raises(ValueError):
        m.blasst_select_prefill(k, k, k, sel)
    with pytest.raises(ValueError):
        m.blasst_block_select(k, k[:, :, :1], 64, n_sel=2)
