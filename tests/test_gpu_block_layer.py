"""The operators together: the mixture-of-experts block of
examples/block_fp8_layer.py against the same block in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests.block_cases import (DEV, E4M3, GROUP, dequant_blocks, groups, rms)

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    spec = importlib.util.spec_from_file_location(
        "block_fp8_layer", os.path.join(ROOT, "examples", "block_fp8_layer.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def quantized(v):
    """v rounded to E4M3FN codes times their 1 x 128 groups' scales."""
    M, K = v.shape
    p = np.pad(v, ((0, 0), (0, groups(K) * GROUP - K))).reshape(M, -1, GROUP)
    amax = np.abs(p).max(axis=2, keepdims=True)
    s = np.where(amax > 0, amax / 448, 1.0)
    t = p / s
    _, e = np.frexp(t)
    step = 2.0 ** np.maximum(e - 4, -9).astype(np.float64)
    return (np.round(t / step) * step * s).reshape(M, -1)[:, :K]


def bf16(v):
    return torch.from_numpy(v).to(torch.bfloat16).double().numpy()


def weights(pair):
    return dequant_blocks(pair[0].view(torch.uint8).cpu().numpy(), pair[1].cpu().numpy())


@pytest.mark.parametrize("T", [1, 5, 48, 300])
@pytest.mark.parametrize("hidden,width,experts,topk", [(512, 256, 8, 2), (640, 144, 5, 3)])
def test_block(layer, T, hidden, width, experts, topk):
    print(f"[case] T={T} hidden={hidden} width={width} experts={experts}", flush=True)
    block = layer.MoeBlock(hidden, width, experts, topk)
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    branch = torch.randn(T, hidden, generator=g, device=DEV).to(torch.bfloat16)
    residual = 4 * torch.randn(T, hidden, generator=g, device=DEV)
    out, after = block.forward(branch, residual)

    b, r = branch.double().cpu().numpy(), residual.double().cpu().numpy()
    h = r + rms(b, 1e-6) * block.post_norm.double().cpu().numpy()
    np.testing.assert_allclose(after.double().cpu().numpy(), h, rtol=2e-6, atol=2e-6)
    z = rms(h, 1e-6) * block.norm.double().cpu().numpy()
    x = quantized(z)

    def mlp(x, up, down):
        both = bf16(x @ up.T)
        gate, u = both[:, :width], both[:, width:]
        return bf16(quantized(gate / (1 + np.exp(-gate)) * u) @ down.T)

    want = mlp(x, weights(block.shared_up), weights(block.shared_down))
    # the experts that the block itself chose
    offsets, rows, weight, place = block.route(
        torch.from_numpy(bf16(z)).to(torch.bfloat16).to(DEV))
    off, rows = offsets.cpu().numpy(), rows.cpu().numpy()
    ups, downs = weights(block.up), weights(block.down)
    routed = np.zeros((T * topk, hidden))
    for e in range(experts):
        at = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            routed[at] = mlp(x[rows[at]], ups[e], downs[e])
    want = want + (routed[place.cpu().numpy()] * weight.double().cpu().numpy()[:, :, None]).sum(1)
    got = out.double().cpu().numpy()
    # Both sides round at the same places; a value within 2^-8 of a rounding
    # boundary may fall on either side.  For codes (steps of 2^-3 at most) that
    # is one value in 2^5 by up to 2^-4 of itself: 2^-6.5 of a row's norm, and
    # as much again from the bf16 roundings: 2^-5 with room for both.
    assert np.linalg.norm(got - want) <= 2.0 ** -5 * np.linalg.norm(want)
