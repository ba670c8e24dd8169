"""The rotation under autograd: gradients against the formula in 64 bits and against differences, in place, broadcast, twice, captured."""
import numpy as np
import pytest
import torch

import tiered_kv_cache_gqa_gb300 as tkv
from test_gpu_paged import BF16, FP16, FP32, check_rotation, ints

pytestmark = pytest.mark.gpu


def case(dtype, rows=7, heads=5, d=40, pairs=16, axes=2, interleaved=True, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    x, w = (torch.randn(rows, heads, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    axis = [j * axes // pairs for j in range(pairs)]
    rot = tkv.Rotary(tkv.rope_table(1000, 2 * pairs), axis, interleaved)
    return x, w, rot, torch.randint(0, 1000, (axes, rows), generator=g, device="cuda", dtype=torch.int32), axis


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("shape", [dict(), dict(interleaved=False), dict(rows=1, heads=1, d=2, pairs=1, axes=1), dict(rows=130, heads=3, d=128, pairs=64, axes=3),
                                   dict(rows=3, heads=2, d=75, pairs=9, axes=1, interleaved=False)])
@pytest.mark.parametrize("inverse", [False, True])
def test_gradient_is_the_rotation_back(dtype, shape, inverse):
    x, w, rot, pos, axis = case(dtype, **shape)
    plain = tkv.rope(x, rot, pos, inverse=inverse)
    x.requires_grad_()
    y = tkv.rope(x, rot, pos, inverse=inverse)
    assert torch.equal(y, plain) and y.requires_grad
    y.backward(w)
    check_rotation(x.grad, w, rot.table, pos.cpu().numpy(), axis, shape.get("interleaved", True), not inverse)


def test_gradient_by_differences():
    """f(x + e) - f(x), f = sum(w rope(x)), summed in 64 bits; the map is linear, so the step is 1."""
    x, w, rot, pos, _ = case(FP32)
    x.requires_grad_()
    (tkv.rope(x, rot, pos) * w).sum().backward()
    with torch.no_grad():
        base = tkv.rope(x, rot, pos).double()
        for i in range(0, x.numel(), 97):
            e = x.detach().clone()
            e.view(-1)[i] += 1.0
            diff = (w.double() * (tkv.rope(e, rot, pos).double() - base)).sum().item()
            # the two results of a pair and x + 1 are each rounded to half a step of values below 8, times |w| < 8
            assert abs(diff - x.grad.view(-1)[i].item()) <= 2 * 8 * 4 * 8 * 2.0 ** -24


def test_gradients_of_shared_and_broadcast_inputs():
    x, w, rot, pos, _ = case(FP32, rows=6, heads=4, d=32, pairs=16)
    back = tkv.rope(w, rot, pos, inverse=True)
    one = x[:, :1].clone().requires_grad_()                     # a head that four read
    tkv.rope(one.expand_as(x), rot, pos).backward(w)
    assert torch.allclose(one.grad, back.sum(1, keepdim=True), rtol=0, atol=4 * 8 * 2.0 ** -23)
    a = x.clone().requires_grad_()
    tkv.rope(a, rot, pos).sum().backward()                      # a gradient of stride 0
    assert torch.equal(a.grad, tkv.rope(torch.ones_like(x), rot, pos, inverse=True))
    b = x.clone().requires_grad_()
    (tkv.rope(b, rot, pos) + tkv.rope(b, rot, pos)).backward(w)   # two uses of one leaf
    assert torch.equal(b.grad, back + back)
    c = x.transpose(0, 1).contiguous().requires_grad_()
    tkv.rope(c.transpose(0, 1), rot, pos).backward(w)
    assert torch.equal(c.grad.transpose(0, 1), back)
    e = x[:0].clone().requires_grad_()
    tkv.rope(e, rot, pos[:, :0]).sum().backward()
    assert e.grad.shape == e.shape


def test_twice_differentiable():
    x, w, rot, pos, _ = case(FP32, rows=2, heads=2, d=8, pairs=4)
    x.requires_grad_()
    w.requires_grad_()
    g, = torch.autograd.grad((tkv.rope(x, rot, pos) * w).sum(), x, create_graph=True)
    u = torch.randn_like(g)
    back, = torch.autograd.grad((g * u).sum(), w)               # g = R^T w, so d (u . g) / d w = R u
    assert torch.equal(back, tkv.rope(u, rot, pos).detach())


def test_in_place_and_into_a_tensor():
    x, w, rot, pos, _ = case(FP32)
    leaf = x.clone().requires_grad_()
    y = leaf * 2.0
    assert tkv.rope(y, rot, pos, out=y) is y
    y.backward(w)
    assert torch.equal(leaf.grad, tkv.rope(w, rot, pos, inverse=True) * 2.0)
    leaf = x.clone().requires_grad_()
    into = torch.empty_like(x)
    y = tkv.rope(leaf, rot, pos, out=into)
    assert y is into and y.requires_grad
    y.backward(w)
    assert torch.equal(leaf.grad, tkv.rope(w, rot, pos, inverse=True))
    leaf = x.clone().requires_grad_()
    behind = x.clone().requires_grad_()
    wide = torch.cat([behind[:, :1], behind, behind[:, :1]], dim=1)   # a part of a larger tensor, which autograd then follows
    tkv.rope(leaf, rot, pos, out=wide[:, 1:-1])
    u = torch.randn_like(wide)
    (wide * 3.0).backward(u)
    assert torch.equal(leaf.grad, tkv.rope(u[:, 1:-1] * 3.0, rot, pos, inverse=True))
    want = torch.zeros_like(x)                                  # what lay in that part before has no gradient
    want[:, 0] = (u[:, 0] + u[:, -1]) * 3.0
    assert torch.allclose(behind.grad, want, rtol=0, atol=6 * 8 * 2.0 ** -23)
    leaf = x.clone().requires_grad_()
    wide = torch.cat([leaf[:, :1], leaf * 2.0], dim=1)
    part = wide[:, 1:]
    assert tkv.rope(part, rot, pos, out=part) is part           # a part in place
    u = torch.randn_like(wide)
    wide.backward(u)
    want = tkv.rope(u[:, 1:].contiguous(), rot, pos, inverse=True) * 2.0
    want[:, 0] += u[:, 0]
    assert torch.allclose(leaf.grad, want, rtol=0, atol=3 * 16 * 2.0 ** -23)
    leaf = x.clone().requires_grad_()
    both = leaf * 2.0
    tkv.rope(both[:, :3], rot, pos, out=both[:, :3])            # two views of the same part
    both.backward(w)
    want = torch.cat([tkv.rope(w[:, :3].contiguous(), rot, pos, inverse=True), w[:, 3:]], dim=1) * 2.0
    assert torch.equal(leaf.grad, want)
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError):                           # a leaf cannot be overwritten
        tkv.rope(leaf, rot, pos, out=leaf)
    with torch.no_grad():                                       # the user's own business here
        assert tkv.rope(leaf, rot, pos, out=leaf) is leaf and not tkv.rope(leaf, rot, pos).requires_grad
    with torch.inference_mode():
        z = x.clone()
        tkv.rope(z, rot, pos, out=z)


def test_what_a_backward_pass_needs_is_not_overwritten_unnoticed():
    x, w, rot, pos, _ = case(FP32)
    leaf = w.clone().requires_grad_()
    y = leaf * x                                                # keeps x
    tkv.rope(x, rot, pos, out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    for change in (pos, rot.table):
        leaf = w.clone().requires_grad_()
        y = tkv.rope(leaf, rot, pos)
        change.add_(0)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_a_position_outside_the_table_under_autograd():
    x, w, rot, pos, _ = case(FP32)
    pos[0, 2], status = 1000, ints([0])
    x.requires_grad_()
    y = tkv.rope(x, rot, pos, status=status)
    assert status.item() == tkv.TKV_EINVAL
    y.backward(w)
    bad = torch.zeros(x.shape, dtype=torch.bool, device="cuda")
    bad[2, :, :16] = True                                       # adjacent pairs 0 .. 7 follow axis 0
    assert torch.equal(y.isnan(), bad) and torch.equal(x.grad.isnan(), bad)


def test_refusals_under_autograd():
    x, _, rot, pos, _ = case(FP32)
    x.requires_grad_()
    for call in (lambda: tkv.rope(x, rot, None), lambda: tkv.rope(x, rot, pos[:1]), lambda: tkv.rope(x.transpose(1, 2), rot, pos),
                 lambda: tkv.rope(x, rot, pos, out=torch.empty(1, device="cuda")), lambda: tkv.rope(x.double(), rot, pos), lambda: tkv.rope(x.cpu(), rot, pos),
                 lambda: tkv.rope(None, rot, pos, out=x)):
        with pytest.raises(tkv.TkvError) as e:
            call()
        assert e.value.status == tkv.TKV_EINVAL


def test_a_captured_training_step():
    x, w, rot, pos, _ = case(BF16, rows=33, heads=4, d=64, pairs=32, axes=3)
    leaf = x.clone().requires_grad_()

    def step():
        y = tkv.rope(leaf, rot, pos)
        return y, torch.autograd.grad(y, leaf, w)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    with torch.no_grad():
        leaf.neg_()
        w.neg_()
    graph.replay()
    assert all(torch.equal(a.detach(), -b.detach()) for a, b in zip(got, want))
