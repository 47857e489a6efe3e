"""Weight gradients of groups that end inside a 16-row step, next to rows that hold NaN, over and over: the rows past a
group are zeroed in both CTAs of a pair before the tensor cores read them."""
import math

import pytest
import torch

from tests.test_gpu_train import Ffn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sizes,H,I", [([19, 6, 45, 3, 1, 33], 256, 256), ([300, 3, 867, 5], 128, 1024),
                                       ([1009, 20, 1100, 40, 1001, 2, 1017, 7], 256, 1024), ([4507, 9], 256, 128)],
                         ids=["64-row blocks", "128-row blocks", "256-row blocks", "split"])
def test_neighbours_of_nan_rows_stay_clean(sizes, H, I):
    f, clean = Ffn(sizes, H, I, seed=41), Ffn(sizes, H, I, seed=41)
    for c in (f, clean):
        c.forward()
    want = clean.backward()
    clean.check_backward(want)
    good = list(range(0, len(sizes), 2))
    for g in range(1, len(sizes), 2):  # every second group
        for t in (f.x, f.dy, f.gu, f.h):
            t[f.off[g]:f.off[g + 1]] = math.nan
    for _ in range(100):
        _, dw1, dw2 = f.backward(ws=clean.ws_b)
        assert torch.equal(dw1[good], want[1][good]) and torch.equal(dw2[good], want[2][good])
        assert torch.isnan(dw1[1]).all() and torch.isnan(dw2[1]).all()
