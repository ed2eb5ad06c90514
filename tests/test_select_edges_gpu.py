"""Block-selected attention where its promises are easiest to break.

Selections are whole numbers and have to be equal.  Other tolerances are
derived where they are used.
"""
import pytest
import torch

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
