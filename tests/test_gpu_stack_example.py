"""GPU test of the hybrid stack's end in examples/: gradients of its head through the public calls
against torch's own in fp32."""

import importlib.util
import os

import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_generate.py")


def load():
    spec = importlib.util.spec_from_file_location("hybrid_generate", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    return example


def test_head_gradients():
    note("hybrid example, head gradients")
    model = load().Model(layers=4)
    gen = torch.Generator("cuda").manual_seed(5)
    lens = [40, 7]
    tokens = torch.randint(0, 512, (47,), generator=gen, device="cuda")
    targets = torch.randint(0, 512, (47,), generator=gen, device="cuda").to(torch.int32)
    g = torch.randn(47, generator=gen, device="cuda")
    model.begin(2, 48)
    x, y = model.step(tokens, lens)
    dx, dw, dh = model.head_gradients(x, y, targets, g)
    xf, w, head = x.float().requires_grad_(), model.weights[-1].clone().requires_grad_(), model.head.float().requires_grad_()
    n = xf * torch.rsqrt(xf.square().mean(-1, keepdim=True) + 1e-6) * w
    lp = torch.log_softmax(n @ head, -1).gather(1, targets.long()[:, None])[:, 0]
    want = torch.autograd.grad((lp * g).sum(), (xf, w, head))
    # y, the logits, their gradient, the product's result and the output each round to bf16: 2^-9 of their
    # size on average, the logits' rounding of up to 2^-8 of about 4 changing every q by as much
    for got, ref in zip((dx, dw, dh), want):
        assert (got.float() - ref).norm() <= (4 * 2.0 ** -8 + 4 * 2.0 ** -8) * ref.norm()
