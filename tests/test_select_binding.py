"""Outputs of block-selected attention that lie in the cache they read."""
import ctypes

import pytest
import torch

from dynamic_block_sparse_fa_b200.blasst import _lib as lib

vp, ll, f32, sz = (ctypes.c_void_p, ctypes.c_longlong, ctypes.c_float,
                   ctypes.c_size_t)
POOL = 1 << 24              # pages of 64 x 128 elements, 16 KB, 32 KB apart
PAGE, STEP = 1 << 14, 1 << 15
ELSE = 1 << 30              # nowhere near


def _means(at):
    return lib.blasst_block_means_paged(
        vp(POOL), ll(STEP // 2), 3, 64, vp(ELSE), 3, vp(ELSE), 150, 0, vp(at),
        3, 1, 1, 128, None)


def _decode(k=POOL, v=2 * POOL, o=ELSE, lse=ELSE, ws=ELSE):
    return lib.blasst_select_decode_paged(
        vp(ELSE), vp(k), vp(v), ll(STEP // 2), 3, 64, vp(ELSE), 3, vp(ELSE),
        150, vp(ELSE), 2, vp(o), vp(lse), 1, 4, 1, 128, f32(0.1), 2, vp(ws),
        sz(1 << 20), None)


# (calls that are not refused are made on a GPU below: here their pointers
# point nowhere)
@pytest.mark.parametrize("page", [0, 1, 2])
def test_outputs_in_a_page_are_refused(page):
    p = page * STEP
    n = 3 * 128 * 2                       # three means
    for at in (p - n + 16, p, p + 4096, p + PAGE - 16):
        assert _means(POOL + at) == 1, at
    for pool in (POOL, 2 * POOL):
        for at in (p - 4 * 128 * 2 + 16, p, p + PAGE - 16):
            assert _decode(o=pool + at) == 1, at
        for at in (p - 12, p, p + PAGE - 4):
            assert _decode(lse=pool + at) == 1, at
        # 4 heads x 2 splits of 128 floats and of one, a word: 4608 bytes
        for at in (p - 4608 + 256, p, p + PAGE - 256):
            assert _decode(ws=pool + at) == 1, at


def test_an_output_over_all_pages_is_refused():
    assert lib.blasst_block_means_paged(
        vp(POOL), ll(STEP // 2), 3, 64, vp(ELSE), 3, vp(ELSE), 150, 0,
        vp(POOL - STEP), 4096, 1, 1, 128, None) == 1


@pytest.mark.gpu
def test_outputs_may_not_lie_in_the_cache():
    import dynamic_block_sparse_fa_b200 as m
    bf = torch.bfloat16
    # 4 pages of K and V halves with room behind each pair
    pool = torch.zeros(4, 3, 1, 64, 128, dtype=bf, device="cuda")
    kp, vpg = pool[:, 0], pool[:, 1]
    bt = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    sl = torch.tensor([100], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 128, dtype=bf, device="cuda")
    sel = torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")

    def decode(**kw):
        m.blasst_select_decode_paged(q, kp, vpg, bt, sl, sel, **kw)
    with pytest.raises(m.BlasstError, match="invalid argument"):
        m.blasst_block_means_paged(kp, bt, sl,
                                   kp[3, 0, 5:7].view(1, 1, 2, 128))
    for half in (kp, vpg):
        with pytest.raises(m.BlasstError):
            decode(o=half[1, 0, :4].view(1, 4, 128))
        with pytest.raises(m.BlasstError):
            decode(lse=half[3, 0, 63, :8].view(torch.float32).view(1, 4))
        with pytest.raises(m.BlasstError):
            decode(workspace=half[0].view(-1).view(torch.uint8), num_splits=1)
    # between the pages, and before and behind them: fine
    decode(o=pool[1, 2, 0, :4].view(1, 4, 128))
    m.blasst_block_means_paged(kp, bt, sl,
                               pool[1, 2, 0, 8:10].view(1, 1, 2, 128))
    m.blasst_block_means_paged(kp[1:], bt - 1, sl - 100,
                               pool[0, 0, 0, :2].view(1, 1, 2, 128))
    m.blasst_block_means_paged(kp[:3], bt, sl,
                               pool[3, 0, 0, :2].view(1, 1, 2, 128))
    torch.cuda.synchronize()
    assert m.blasst_check_device_error()[0] == 0


def test_stream_of_another_device_is_refused():
    import dynamic_block_sparse_fa_b200 as m

    class Other:                      # a stream of a second GPU
        device = torch.device("cuda", 1)
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    k = torch.zeros(1, 1, 64, 128, dtype=torch.bfloat16, device=dev)
    sel = torch.zeros(1, 1, 64, 1, dtype=torch.int32, device=dev)
    for call in (lambda: m.blasst_block_means(k, stream=Other()),
                 lambda: m.blasst_block_select(q=k, means=k[:, :, :1],
                                               Lkv=64, n_sel=1,
                                               stream=Other()),
                 lambda: m.blasst_select_prefill(k, k, k, sel,
                                                 stream=Other())):
        with pytest.raises(ValueError, match="stream: on cuda:1"):
            call()
