"""The training calls at the ends of what they allow: as many groups as there can be, rows ahead of the first group,
limits of which some are infinite, nearly everything dropped, and passes that run at one time."""
import math

import pytest
import torch

import grouped_gemm_swiglu_b200 as moe
from tests import train_ref as R
from tests.test_gpu_train import BF, DEV, INF, Ffn, ffn_dims, randn

pytestmark = pytest.mark.gpu


def both(f):
    f.forward()
    f.check_forward()
    f.check_backward(f.backward())


def test_as_many_groups_as_there_can_be():
    g = torch.Generator().manual_seed(2)
    sizes = torch.randint(0, 4, (1024,), generator=g)
    sizes[[0, 500, 1023]] = torch.tensor([0, 130, 17])
    both(Ffn(sizes.tolist(), 128, 128, scales=True, limits=True, p=0.1, seed=61))


@pytest.mark.parametrize("limits", [[INF, 0.75, INF, 1.5], [0.75, INF, 1.5, INF]])
def test_limits_of_which_some_are_infinite(limits):
    f = Ffn([40, 300, 7, 90], 256, 256, limit=3.0, seed=62)
    f.limits = torch.tensor(limits, device=DEV)
    both(f)


@pytest.mark.parametrize("p", [0.999, 2.0 ** -30])
def test_nearly_everything_or_nothing_dropped(p):
    both(Ffn([40, 0, 300], 256, 256, limit=1.0, p=p, seed=63))


def test_rows_ahead_of_the_first_group_are_left_as_they_were():
    """offsets[0] > 0: those rows are read by nobody (they hold NaN) and written by nobody."""
    sizes, skip = [37, 0, 90], 21
    f, want = Ffn([skip] + sizes, 256, 128, seed=64), {}
    f.forward()
    dx, dw1, dw2 = f.backward()
    want = dict(gu=f.gu[skip:], h=f.h[skip:], y=f.y[skip:], dx=dx[skip:], dw1=dw1[1:], dw2=dw2[1:])
    f.off = f.off[1:]
    f.offsets = f.offsets[1:].clone()
    f.w1, f.w2 = f.w1[1:].clone(), f.w2[1:].clone()
    f.dims = ffn_dims(f.A, 3, 256, 128)
    for t in (f.x, f.dy):
        t[:skip] = math.nan
    f.forward()
    dx, dw1, dw2 = f.backward()
    for name, t in dict(gu=f.gu, h=f.h, y=f.y, dx=dx).items():
        assert (t[:skip] == -77.0).all() and torch.equal(t[skip:], want[name]), name
    assert torch.equal(dw1, want["dw1"]) and torch.equal(dw2, want["dw2"])
    assert moe.moe_read_status(f.ws_f) == 0 and moe.moe_read_status(f.ws_b) == 0


def test_passes_on_two_streams_at_one_time():
    """Two blocks with outputs and workspaces of their own, forward and backward, over and over on two streams."""
    cases = [Ffn([400, 0, 1000, 77], 512, 384, p=0.2, seed=65), Ffn([9] * 40, 256, 256, limit=0.8, seed=66)]
    want = [list(c.forward()) + c.backward() for c in cases]
    ws = [(c.ws_f, c.ws_b) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(30):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i] = list(c.forward(ws[i][0])) + c.backward(ws[i][1])
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in zip(got[i], want[i]):
            assert torch.equal(a, b)
        assert all(moe.moe_read_status(w) == 0 for w in ws[i])


def test_a_batch_of_no_rows_between_others_in_one_workspace():
    f = Ffn([33, 290], 256, 384, seed=67)
    both(f)
    none = ffn_dims(0, 2, 256, 384)
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    e = lambda w: torch.empty((0, w), dtype=BF, device=DEV)  # noqa: E731
    dw1, dw2 = torch.full_like(f.w1, math.nan), torch.full_like(f.w2, math.nan)
    moe.moe_ffn_forward(e(256), off, f.w1, None, None, None, f.w2, 0.0, None, none, e(768), e(384), e(256), f.ws_f)
    moe.moe_ffn_backward(e(256), e(256), e(768), e(384), off, f.w1, None, None, None, f.w2, 0.0, None, none, e(256), dw1, dw2, f.ws_b)
    assert (dw1 == 0).all() and (dw2 == 0).all()
    f.forward(f.ws_f)
    f.check_forward()
    f.check_backward(f.backward(f.ws_b))


def test_combine_backward_of_dropped_slots():
    """A slot without a row (inverse permutation -1, as the permutation leaves a refused expert id): no gradient of its
    weight, no row written, the other slots as ever."""
    T, H, E, k = 12, 256, 8, 3
    d = moe.MoeDims(T=T, H=H, I=128, E=E, k=k, n_sink=0, n_shared=0, wdtype=moe.MOE_WDTYPE_BF16, score=moe.MOE_SCORE_SOFTMAX,
                    alpha=1.0, beta=0.0, limit=INF, route_scale=1.0)
    ids = torch.stack([torch.arange(T) % E, (torch.arange(T) + 1) % E, (torch.arange(T) + 3) % E], 1).int().to(DEV)
    inv = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k).clone()
    w = torch.softmax(randn(1, T, k, dtype=torch.float32), 1)
    y, dout = randn(2, T * k, H), randn(3, T, H)
    inv[4, 1] = inv[7, 0] = -1
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    dy = torch.full_like(y, -77.0)
    dw, dl = torch.empty(T, k, device=DEV), torch.empty(T, E, device=DEV)
    moe.moe_combine_backward(dout, y, off, inv, ids, w, None, None, d, dy, dw, None, dl, moe.alloc_workspace(d, moe.MOE_WS_COMBINE))
    gone = torch.zeros(T, k, dtype=torch.bool, device=DEV)
    gone[4, 1] = gone[7, 0] = True
    yd, dd = y.double().view(T, k, H), dout.double()
    want = torch.where(gone, 0.0, (yd * dd[:, None]).sum(2))
    err = (yd.abs() * dd.abs()[:, None]).sum(2) * (H + 8) * R.ACC
    R.assert_within(dw, want, err, "dtopk_w")
    rows = dy.view(T, k, H)
    assert (rows[gone] == -77.0).all()
    full = w.double()[..., None] * dd[:, None].expand(T, k, H)
    R.assert_within(rows[~gone], full[~gone], (R.U16 + 2.0 ** -22) * full[~gone].abs(), "dy")
    # dl_j = w_j (dw_j - sum_i w_i dw_i): errors of dw, and of the fp32 weights and sums (k + 4 roundings)
    wd = w.double()
    dl_want = wd * (want - (wd * want).sum(1, keepdim=True))
    dl_err = wd * (err + (wd * err).sum(1, keepdim=True)) + (k + 4) * 2.0 ** -24 * wd * (want.abs() + (wd * want.abs()).sum(1, keepdim=True))
    R.assert_within(dl.gather(1, ids.long()), dl_want, dl_err, "dlogits")
