"""What MoETraining refuses before it launches anything (CPU)."""
import math

import pytest
import torch

import grouped_gemm_swiglu_b200 as moe
from grouped_gemm_swiglu_b200 import build as B

BF = torch.bfloat16
T, H, I, E = 4, 128, 128, 6


@pytest.fixture(scope="module")
def layer():
    B.build()
    d = moe.MoeDims(T=T, H=H, I=I, E=E, k=2, n_sink=1, n_shared=0, wdtype=moe.MOE_WDTYPE_BF16, score=moe.MOE_SCORE_SIGMOID,
                    alpha=1.0, beta=0.0, limit=math.inf, route_scale=1.0)
    return moe.MoETraining(d, torch.zeros(E, 2 * I, H, dtype=BF), torch.zeros(E, H, I, dtype=BF))


def forward(layer, bias=None, logits=torch.zeros(T, E + 1), x=torch.zeros(T, H, dtype=BF), **kw):
    layer.router_bias = bias
    layer.forward(logits, x, **kw)


@pytest.mark.parametrize("bias", [torch.zeros(E, dtype=BF), torch.zeros(E, dtype=torch.float64), torch.zeros(E - 1), torch.zeros(E + 1),
                                  torch.zeros(1, E), torch.zeros(2 * E)[::2], torch.zeros(1).expand(E), torch.zeros(E, device="meta")],
                         ids=["bf16", "fp64", "short", "with the sink", "two-dimensional", "strided", "expanded", "other device"])
def test_router_bias_is_refused(layer, bias):
    """The router reads E contiguous fp32 words at the address that it is given."""
    with pytest.raises(ValueError, match="router_bias must be a contiguous torch.float32 tensor of shape \\(6,\\)"):
        forward(layer, bias)


def test_the_other_inputs_are_refused_and_good_ones_are_not(layer):
    for name, kw in (("logits", dict(logits=torch.zeros(T, E))), ("logits", dict(logits=torch.zeros(T, E + 1, dtype=BF))),
                     ("x", dict(x=torch.zeros(T, H))), ("x", dict(x=torch.zeros(T, 2 * H, dtype=BF)[:, ::2])),
                     ("residual", dict(residual=torch.zeros(T, H))), ("residual", dict(residual=torch.zeros(T, H + 1, dtype=BF)))):
        with pytest.raises(ValueError, match=name):
            forward(layer, **kw)
    for bias in (None, torch.zeros(E)):  # everything is right, but on the CPU
        with pytest.raises(ValueError, match="cuda device"):
            forward(layer, bias)


@pytest.mark.gpu
def test_a_good_router_bias_ranks_and_has_no_other_part():
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std  # noqa: E731
    d = moe.MoeDims(T=50, H=H, I=I, E=E, k=2, n_sink=0, n_shared=0, wdtype=moe.MOE_WDTYPE_BF16, score=moe.MOE_SCORE_SIGMOID,
                    alpha=1.0, beta=0.0, limit=math.inf, route_scale=1.0)
    w1, w2 = rnd(E, 2 * I, H, std=0.1).to(BF), rnd(E, H, I, std=0.1).to(BF)
    bias = torch.tensor([0.0, 5.0, 0.0, -5.0, 0.0, 2.0], device="cuda")  # further apart than two sigmoids can be
    layer = moe.MoETraining(d, w1, w2, router_bias=bias)
    logits, x, dout = rnd(50, E), rnd(50, H).to(BF), rnd(50, H).to(BF)
    out, saved = layer.forward(logits, x)
    grads = layer.backward(saved, dout)
    assert layer.status() == 0
    assert torch.equal(saved.topk_ids.cpu(), torch.tensor([[1, 5]], dtype=torch.int32).expand(50, 2))
    w = torch.softmax(torch.nn.functional.logsigmoid(logits[:, [1, 5]].double()), 1)
    assert torch.allclose(saved.topk_w.double(), w, rtol=1e-5, atol=0)
    assert (grads["dlogits"][:, [0, 2, 3, 4]] == 0).all() and (grads["dlogits"][:, [1, 5]] != 0).all()
    # the same selection without a bias: the same pass
    low = torch.full_like(logits, -100.0)
    low[:, 1], low[:, 5] = logits[:, 1], logits[:, 5]
    out2, saved2 = moe.MoETraining(d, w1, w2).forward(low, x)
    same = saved2.topk_ids[:, 0] == 1  # the order of the two slots may differ, and with it that of the sum
    assert torch.equal(out2[same], out[same]) and int(same.sum()) > 5
