"""The forward calls and their gradients joined into autograd functions, as the
README shows them (its code is what runs here), around experts written in
torch.  Inputs are small whole numbers, for which every product, sum and
rounding is exact, so gradients are compared with torch's own, bit for bit."""

import os
import re

import pytest
import torch

from quantized_linear_gemm_b200 import lq

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "README.md")


def functions():
    with open(README) as f:
        code = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "autograd.Function" in b]
    assert len(code) == 1
    scope = {"torch": torch, "lq": lq}
    exec(code[0], scope)   # noqa: S102 - this repository's own text
    return scope["Permute"], scope["Unpermute"]


@pytest.mark.parametrize("drop", [False, True])
def test_readme_functions(cuda_device, drop):
    permute, unpermute = functions()
    T, k, H, E = 23, 3, 128, 5
    g = torch.Generator().manual_seed(4)
    whole = lambda *s: torch.randint(-2, 3, s, generator=g).float().cuda()   # noqa: E731
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).cuda()
    if drop:
        ids[::4, 1] = -1
    off, order, slots = lq.moe_sort(ids, E)
    x, w, dout = whole(T, H), whole(T, k), whole(T, H).bfloat16()
    factor = whole(E)                                                  # the experts: y = factor[e] x
    rows = torch.bucketize(torch.arange(T * k, device="cuda"), off[1:-1].long(), right=True)

    xa, wa = x.bfloat16().requires_grad_(), w.clone().requires_grad_()
    y = permute.apply(xa, slots) * factor[rows][:, None].bfloat16()
    out = unpermute.apply(y, slots, wa)
    out.backward(dout)

    xb, wb = x.double().requires_grad_(), w.double().requires_grad_()
    kept = (ids >= 0).double()
    ref = ((wb * kept * factor.double()[ids.clamp(min=0)])[..., None] * xb[:, None]).sum(1)
    ref.backward(dout.double())
    assert torch.equal(out.double(), ref)
    assert torch.equal(xa.grad.double(), xb.grad)
    assert torch.equal(wa.grad.double(), wb.grad)


def test_outputs_carry_no_graph(cuda_device):
    """What the documentation says of the calls themselves."""
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda", requires_grad=True)
    slots = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    xs = lq.moe_permute(x, slots)
    assert not xs.requires_grad and not lq.moe_unpermute(xs, slots).requires_grad
