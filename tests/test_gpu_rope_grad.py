"""Gradients of mx_rope through autograd: its backward pass is the inverse rotation."""

import pytest
import torch

from oracle import attention as oa
from tests.gpu_util import dev, import_library

pytestmark = pytest.mark.gpu

mxa = import_library()


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gradients(dtype, layout, inverse):
    g = torch.Generator(device=dev()).manual_seed(3)
    table = torch.from_numpy(oa.rope_table(64, 32, 1e4)).float().to(dev())
    pos = torch.randint(0, 64, (19,), device=dev(), generator=g).int()
    x, w = (torch.randn((19, 3, 96), device=dev(), generator=g).to(dtype) for _ in range(2))
    x.requires_grad_()
    # two uses of a leaf, one of them a slice
    y = mxa.mx_rope(x, pos, table, layout, inverse)
    z = mxa.mx_rope(x[:, 1:], pos, table, layout, inverse)
    grad, = torch.autograd.grad([y, z], x, [w, w[:, 1:]])
    # to the bit, as the rotation itself: FP32 steps, one rounding to the type, then torch's sum of the two
    one = oa.rotate(w.float().cpu().numpy(), pos.cpu().numpy(), table.cpu().numpy(), layout, not inverse)
    want = torch.from_numpy(one).to(dtype)
    want[:, 1:] += want[:, 1:].clone()
    assert torch.equal(grad.cpu(), want)


def test_no_history_where_none_is_asked_for():
    table, pos = mxa.mx_rope_table(8, 64), torch.arange(4, dtype=torch.int32, device=dev())
    x = torch.randn((4, 2, 64), device=dev())
    assert not mxa.mx_rope(x, pos, table).requires_grad
    x.requires_grad_()
    with torch.no_grad():
        assert not mxa.mx_rope(x, pos, table).requires_grad
        mxa.mx_rope(x, pos, table, out=x)
    with pytest.raises(ValueError, match="out"):
        mxa.mx_rope(x, pos, table, out=torch.empty_like(x))


def test_gradients_are_differentiable():
    table, pos = mxa.mx_rope_table(8, 64), torch.arange(4, dtype=torch.int32, device=dev())
    x = torch.randn((4, 2, 64), device=dev(), requires_grad=True)
    w = torch.randn((4, 2, 64), device=dev(), requires_grad=True)
    g, = torch.autograd.grad(mxa.mx_rope(x, pos, table), x, w, create_graph=True)
    back, = torch.autograd.grad(g, w, torch.ones_like(g))
    assert torch.equal(back, mxa.mx_rope(torch.ones_like(w), pos, table))


def test_expanded_gradients_and_streams():
    """The gradient of a sum has no strides of its own; a side stream's backward pass runs on that stream."""
    table, pos = mxa.mx_rope_table(8, 64), torch.arange(4, dtype=torch.int32, device=dev())
    x = torch.randn((4, 2, 64), device=dev(), requires_grad=True)
    want = mxa.mx_rope(torch.ones((4, 2, 64), device=dev()), pos, table, inverse=True)
    mxa.mx_rope(x, pos, table).sum().backward()
    assert torch.equal(x.grad, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g, = torch.autograd.grad(mxa.mx_rope(x, pos, table).sum(), x)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(g, want)
