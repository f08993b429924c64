"""Rotary positions on the GPU against the float64 oracle (oracle/rotary.py), and their gradient."""

import numpy as np
import pytest
import torch

import oracle.rotary as orot
import sparse_attention_lightning_bf16_amd as lx

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def tolerance(x, start, rot, scale, dtype):
    """cos and sin are good to 2^-22 (angle reduced in 64 bits, rounded to fp32, one ulp of the function, the
    scale's product), two products and a sum in fp32: 2^-21 of |a| + |b|; then one rounding to the type."""
    part = np.abs(x[..., start:start + rot]).sum(-1, keepdims=True)
    tol = np.zeros_like(x)
    tol[..., start:start + rot] = 2.0 ** -21 * scale * part
    return tol, torch.finfo(dtype).eps / 2


def check(y, ref, x, start, rot, scale, dtype):
    tol, half = tolerance(x, start, rot, scale, dtype)
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0          # half of fp16's smallest step
    got = y.detach().cpu().double().numpy()
    assert got.shape == ref.shape
    rotated = np.zeros(x.shape[-1], dtype=bool)
    rotated[start:start + rot] = True
    assert np.array_equal(got[..., ~rotated], x[..., ~rotated])
    assert (np.abs(got - ref)[..., rotated] <= (tol + half * np.abs(ref) + tiny)[..., rotated]).all()


@pytest.mark.parametrize("N0,N1,H,D,rot,start,dtype", [
    (1, 1, 1, 64, 64, 0, torch.bfloat16),
    (1, 16, 64, 128, 64, 64, torch.bfloat16),
    (37, 3, 5, 128, 32, 0, torch.float16),
    (300, 1, 0, 128, 64, 0, torch.bfloat16),          # one key per token
    (9, 2, 3, 192, 64, 128, torch.float32),
    (5, 3, 2, 80, 20, 7, torch.float16),              # nothing a multiple of 16 bytes
    (4, 2, 3, 10, 2, 1, torch.float32),
    (3, 1, 2, 1024, 1024, 0, torch.bfloat16),
])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_and_its_gradient_match_the_oracle(N0, N1, H, D, rot, start, dtype, layout):
    g = torch.Generator().manual_seed(N0 + D)
    shape = (N0, N1) + ((H,) if H else ()) + (D,)
    x, dy = (torch.randn(*shape, generator=g).to(dtype) for _ in range(2))
    pos = torch.randint(-1000, 1 << 20, (N0, N1), generator=g, dtype=torch.int32)
    f, _ = lx.rotary_frequencies(rot, device=DEV)
    xd = x.to(DEV).requires_grad_()
    y = lx.rotary(xd, pos.to(DEV), f, layout, start, 1.25)
    (dx,) = torch.autograd.grad(y, xd, dy.to(DEV))
    assert y.dtype == dtype and dx.dtype == dtype
    x4, dy4 = (t.double().numpy().reshape(N0, N1, max(H, 1), D) for t in (x, dy))
    ref = orot.rotary(x4, pos.numpy(), f.cpu().numpy(), layout, start, 1.25)
    check(y.reshape(x4.shape), ref, x4, start, rot, 1.25, dtype)
    back = orot.rotary(dy4, pos.numpy(), f.cpu().numpy(), layout, start, 1.25, inverse=True)
    check(dx.reshape(x4.shape), back, dy4, start, rot, 1.25, dtype)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient_agrees_with_differences(layout):
    g = torch.Generator().manual_seed(5)
    x = torch.randn(3, 2, 2, 16, generator=g).to(DEV)
    dy = torch.randn(3, 2, 2, 16, generator=g).to(DEV)
    pos = torch.tensor([[3, 70], [1, 9], [100000, 0]], dtype=torch.int32, device=DEV)
    f, scale = lx.rotary_frequencies(8, scaling="yarn", factor=8.0, original_max_position=32, device=DEV)
    xr = x.clone().requires_grad_()
    (dx,) = torch.autograd.grad(lx.rotary(xr, pos, f, layout, 4, scale), xr, dy)
    for at in [(0, 0, 0, 3), (0, 1, 1, 4), (2, 0, 1, 9), (1, 1, 0, 11), (2, 1, 1, 15)]:
        up, down = x.clone(), x.clone()
        up[at] += 0.5
        down[at] -= 0.5                                # the map is linear: no truncation error
        d = (lx.rotary(up, pos, f, layout, 4, scale) - lx.rotary(down, pos, f, layout, 4, scale)).double()
        assert abs(float((d * dy.double()).sum()) - float(dx[at])) < 1e-4


def test_far_positions_keep_their_angle():
    # the largest position, frequency 1: fp32 angles would be off by up to 128
    x = torch.zeros(1, 1, 1, 2, device=DEV)
    x[..., 0] = 1.0
    f = torch.ones(1, dtype=torch.float64, device=DEV)
    for p in (2147483647, -2147483648, 1000003):
        y = lx.rotary(x, torch.tensor([[p]], dtype=torch.int32, device=DEV), f)
        assert abs(float(y[0, 0, 0, 0]) - np.cos(float(p))) < 1e-6
        assert abs(float(y[0, 0, 0, 1]) - np.sin(float(p))) < 1e-6


def test_strides_broadcast_positions_and_writing_in_place():
    g = torch.Generator().manual_seed(7)
    wide = torch.randn(20, 3, 12, 72, generator=g).to(torch.bfloat16).to(DEV)
    x = wide[:, :, 4:8, 8:]                            # a slice of a projection
    f, _ = lx.rotary_frequencies(64, device=DEV)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    want = lx.rotary(x.contiguous(), pos[:, None].expand(20, 3).contiguous(), f)
    for p in (pos, pos[:, None], pos[:, None].expand(20, 3)):
        assert torch.equal(lx.rotary(x, p, f), want)
    shifted = wide[:, :, 4:8, 3:67]                    # rows at odd elements
    assert torch.equal(lx.rotary(shifted, pos, f), lx.rotary(shifted.contiguous(), pos, f))
    t = x.transpose(0, 1)
    assert torch.equal(lx.rotary(t, pos[None], f), want.transpose(0, 1))
    before = wide.clone()
    lx.rotary(x, pos, f, out=x)
    assert torch.equal(x, want)
    before[:, :, 4:8, 8:] = want
    assert torch.equal(wide, before)                   # nothing else was written


def test_expanded_gradients():
    f, _ = lx.rotary_frequencies(16, device=DEV)
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    x = torch.randn(6, 2, 3, 16, device=DEV, requires_grad=True)
    lx.rotary(x, pos, f).sum().backward()              # the upstream gradient is one number, broadcast
    got = x.grad.clone()
    want = torch.autograd.grad(lx.rotary(x, pos, f), x, torch.ones_like(x))[0]
    assert torch.equal(got, want)
    shared = torch.randn(6, 2, 1, 16, device=DEV, requires_grad=True)      # one head given to three
    (d,) = torch.autograd.grad(lx.rotary(shared.expand(6, 2, 3, 16), pos, f).sum(), shared)
    assert torch.allclose(d, 3 * want[:, :, :1], rtol=1e-6, atol=1e-6)


def test_the_indexer_rotates_its_inputs():
    S, B, H, D, c, tk = 64, 2, 16, 64, 2, 8
    g = torch.Generator().manual_seed(9)
    q = torch.randn(S, B, H, D, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    k = torch.randn(S // c, B, D, generator=g).to(torch.bfloat16).to(DEV).requires_grad_()
    w = torch.randn(S, B, H, generator=g).to(DEV).requires_grad_()
    f, scale = lx.rotary_frequencies(32, device=DEV)
    how = lx.Rotary(f, "half", 32, scale)
    sc, ix = lx.v4_lighting_indexer(q, k, w, c, tk, rotary=how)
    qp = torch.arange(S, dtype=torch.int32, device=DEV)
    kp = torch.arange(S // c, dtype=torch.int32, device=DEV) * c
    qr, kr = (t.detach().requires_grad_() for t in (lx.rotary(q, qp, f, "half", 32), lx.rotary(k, kp, f, "half", 32)))
    sc2, ix2 = lx.v4_lighting_indexer(qr, kr, w, c, tk)
    assert torch.equal(sc, sc2) and torch.equal(ix, ix2)
    up = torch.where(ix >= 0, torch.ones_like(sc), torch.zeros_like(sc))
    dq, dw = torch.autograd.grad(sc, (q, w), up)
    dqr, dw2 = torch.autograd.grad(sc2, (qr, w), up)
    assert torch.equal(dw, dw2)
    inv = orot.rotary(dqr.double().cpu().numpy(), qp.cpu().numpy()[:, None].repeat(B, 1), f.cpu().numpy(), "half", 32,
                      1.0, inverse=True)
    check(dq, inv, dqr.double().cpu().numpy(), 32, 32, 1.0, torch.bfloat16)


def test_a_captured_rotation_replays_with_new_inputs():
    x = torch.randn(4, 2, 3, 64, device=DEV, dtype=torch.float16)
    pos = torch.arange(4, dtype=torch.int32, device=DEV)
    f, _ = lx.rotary_frequencies(64, device=DEV)
    lx.rotary(x, pos, f)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lx.rotary(x, pos, f)
    for _ in range(3):
        x.copy_(torch.randn(4, 2, 3, 64, device=DEV))
        pos.add_(1000)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, lx.rotary(x, pos, f))
