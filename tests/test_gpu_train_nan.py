"""NaN and infinities through the feed-forward block's training calls: NaN comes out where the definition has it, with
and without a limit, and everywhere else the results are those of the clean inputs."""
import math

import pytest
import torch

from tests import train_ref as R
from tests.test_gpu_train import DEV, INF, Ffn

pytestmark = pytest.mark.gpu
NAN = math.nan

# token blocks of 64, 128 and 256 rows, and weight gradients split along the rows
SIZES = {"64": dict(sizes=[40, 0, 90], H=256, I=256), "128": dict(sizes=[300, 3, 867], H=128, I=1024),
         "256": dict(sizes=[3990, 0, 20, 40, 1, 2, 111], H=128, I=1024), "split": dict(sizes=[4500], H=256, I=128)}
ACTS = [dict(limit=0.8, alpha=1.702, beta=1.0), dict(limit=7.0, p=0.25), dict(limit=INF), dict(limit=INF, p=0.25),
        dict(limits=True, scales=True)]
ids = lambda a: "-".join(f"{k}{v}" for k, v in a.items())  # noqa: E731


def same(got, clean, nan, what):
    """NaN exactly where `nan` says, and the clean result's bits elsewhere."""
    assert torch.equal(torch.isnan(got), nan), f"{what}: {int((torch.isnan(got) != nan).sum())} of {nan.numel()} elements"
    assert torch.equal(got[~nan], clean[~nan]), what


@pytest.mark.parametrize("size", ["64", "128", "256"])
@pytest.mark.parametrize("act", ACTS, ids=ids)
@pytest.mark.parametrize("where", ["x", "gate row", "up row", "both infinities"])
def test_forward_nan(size, act, where):
    f, clean = Ffn(**SIZES[size], **act, seed=31), Ffn(**SIZES[size], **act, seed=31)
    clean.forward()
    I, g = f.dims.I, len(f.off) - 2  # the last group
    nan = torch.zeros(f.A, 2 * I, dtype=torch.bool, device=DEV)  # gate | up
    if where == "x":
        f.x[f.off[g] + 5, 7] = NAN
        nan[f.off[g] + 5] = True
    elif where == "both infinities":  # inf - inf where the two weights have one sign
        f.x[2, 0], f.x[2, 1] = INF, -INF
        w = f.w1[0, :, :2].float()
        nan[2] = (w[:, 0] > 0) == (w[:, 1] > 0)
        assert (w != 0).all()
    else:
        i = 3 + (I if where == "up row" else 0)
        f.w1[g, i, 11] = NAN
        nan[f.off[g]:f.off[g + 1], i] = True
    f.forward()
    if where == "both infinities":  # the other sums of that row are infinite, and what the activation makes of them is not looked at
        assert torch.equal(torch.isnan(f.gu), nan)
        rest = torch.ones(f.A, dtype=torch.bool, device=DEV)
        rest[2] = False
        for a, b in ((f.gu, clean.gu), (f.h, clean.h), (f.y, clean.y)):
            assert torch.equal(a[rest], b[rest])
        m = nan[2, :I] | nan[2, I:]
        if f.keep is not None:
            m &= f.keep[2] > 0
        assert torch.isnan(f.h[2][m]).all() and torch.isnan(f.y[2]).all()
        return
    same(f.gu, clean.gu, nan, "gu")
    nan_h = nan[:, :I] | nan[:, I:]
    if f.keep is not None:
        nan_h &= f.keep > 0  # a dropped element is 0 whatever it was
    assert nan_h.any()
    same(f.h, clean.h, nan_h, "h")
    same(f.y, clean.y, nan_h.any(1, keepdim=True).expand_as(f.y), "y")


@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("act", ACTS, ids=ids)
@pytest.mark.parametrize("where", ["gate", "up"])
def test_backward_nan(size, act, where):
    """NaN in single saved gates or ups, against the definition in 64 bits: a NaN gate makes dgate and dup NaN, a NaN up
    value makes dgate NaN and, as it does not lie within the limits, dup 0."""
    f = Ffn(**SIZES[size], **act, seed=32)
    f.forward()
    I, n = f.dims.I, f.n
    at = [(0, 1), (17, 40), (n - 1, I - 1), (n - 30, 100), (n - 30, 101)]
    for r, i in at:
        f.gu[r, i], f.gu[r, I + i] = 0.125, 0.25  # the other of the two lies within every limit
        f.gu[r, i + (I if where == "up" else 0)] = NAN
    if f.dims.limit < INF:  # infinities beyond the limit: no gradient of their own
        f.gu[9, 5], f.gu[9, I + 6], f.gu[9, I + 7] = INF, INF, -INF
    got = f.backward()
    ref = R.ffn_backward(f.dy, f.x, f.gu, f.h, f.off, f.w1, f.gs, f.us, f.limits, f.w2, f.keep, *f.act)
    rows = torch.zeros(n, 1, dtype=torch.bool, device=DEV)
    feat = torch.zeros(len(f.off) - 1, 2 * I, 1, dtype=torch.bool, device=DEV)
    for r, i in at:
        g = max(e for e in range(len(f.off) - 1) if f.off[e] <= r)
        rows[r] = True
        feat[g, i] = True
        if where == "gate":
            feat[g, I + i] = True
    for have, (want, err), what, nan in zip(got, ref, ("dx", "dw1", "dw2"), (rows, feat, None)):
        nan = torch.zeros_like(have, dtype=torch.bool) if nan is None else nan.expand_as(have)
        assert torch.equal(torch.isnan(want), nan)  # the definition
        assert torch.equal(torch.isnan(have), nan), f"{what}: {int((torch.isnan(have) != nan).sum())} of {nan.numel()} elements"
        R.assert_within(have[~nan], want[~nan], err[~nan], what)


@pytest.mark.parametrize("limit", [0.8, 7.0, INF])
def test_a_diverged_pass_shows_in_every_gradient_it_reaches(limit):
    """A NaN in a row of x or of the weights, forward and backward together."""
    for where in ("x", "w1"):
        f = Ffn([50, 20], 256, 128, limit=limit, seed=33)
        (f.x[55] if where == "x" else f.w1[1, 9])[:] = NAN
        f.forward()
        dx, dw1, dw2 = f.backward()
        rows = slice(55, 56) if where == "x" else slice(50, 70)
        assert torch.isnan(f.y[rows]).all() and torch.isnan(dx[rows]).all()
        assert torch.isnan(dw1[1] if where == "x" else dw1[1, 9]).all()
        assert torch.isnan(dw2[1] if where == "x" else dw2[1, :, 9]).all()
        for t in (f.y[:50], dx[:50], dw1[0], dw2[0]):
            assert torch.isfinite(t).all()
