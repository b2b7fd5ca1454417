"""The serving calls where their numbers leave the ordinary range (needs a B200): weights times
value norms over many orders; rotary positions in a graph of gradients.  Tolerances as in
test_gpu_serving.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import rrq as orc
from oracle import serving as osv
from random_rotation_kv_b200 import binding as B
from tests.test_gpu_serving import DEV, HALF, _attend, _check_attention, _dev, _part

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ shared attention
def _outlier(rg, tokens, hq, d, at, gap, norm, batch=1):
    """A cache of one kv head and queries for which token `at` scores `gap` nats above all others
    (which score nearly the same) and has the value norm `norm`; the other values are
    alike, so they add up."""
    u = rg.standard_normal(d)
    q = u[None, None, :] + 0.01 * rg.standard_normal((batch, hq, d))
    kc, kn, vc, vn = _part(rg, tokens, d, 4, 4)
    kn *= 1e-3
    key = orc.encode(u[None, :] * np.sign(gap), 4, 42)
    kc[at] = key.packed[0]
    dot = float(orc.decode_exact(key.packed, key.norms, 4, d, 42)[0] @ u)
    kn[at] = key.norms[0] * abs(gap) / abs(dot)
    vc[:] = vc[:4][np.arange(tokens) % 4]
    vn[at] = norm
    return q, (kc, kn, vc, vn)


@pytest.mark.parametrize("d", [64, 128, 256, 512])
@pytest.mark.parametrize("hq,batch", [(3, 1), (40, 1), (8, 9)])
@pytest.mark.parametrize("gap,norm", [(10, 0.0), (18, 0.0), (25, 1e-6), (50, 0.0), (-40, 1e12), (-20, 1e20), (0.5, 1e30)])
def test_attention_shared_outlier_token(d, hq, batch, gap, norm):
    """A token that takes nearly all of the weight with a value of no size (the others make the
    output), or a value of enormous size with next to no weight: first, inside and last."""
    tokens = 1100
    for at in (0, 700, tokens - 1):
        rg = np.random.Generator(np.random.PCG64(d + hq + at))
        q, p = _outlier(rg, tokens, hq, d, at, gap, norm, batch)
        _check_attention(q, p, None, [0] * batch, 1, d, 4, 4, 1.0, torch.bfloat16, f"prefix, token {at}")
        if batch == 1:  # the same cache as a tail behind nothing, and cut in two
            _check_attention(q, None, p, [tokens], 1, d, 4, 4, 1.0, torch.bfloat16, f"tail, token {at}")
            head, tail = tuple(x[:300] for x in p), tuple(x[300:] for x in p)
            _check_attention(q, head, tail, [tokens - 300], 1, d, 4, 4, 1.0, torch.bfloat16, f"both, token {at}")


@pytest.mark.parametrize("d", [64, 256, 512])
@pytest.mark.parametrize("hq", [2, 24])
def test_attention_shared_value_norms_zero(d, hq):
    rg = np.random.Generator(np.random.PCG64(d))
    p = list(_part(rg, 300, d, 4, 4))
    q = rg.standard_normal((1, hq, d))
    p[3][:] = 0
    assert torch.all(_attend(q, p, None, None, 1, d, 4, 4, d ** -0.5, torch.float16) == 0)
    p[3][7] = 1.0  # one value among them
    _check_attention(q, p, None, [0], 1, d, 4, 4, d ** -0.5, torch.bfloat16, "one value")


# --------------------------------------------------------------------------------- rope
@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved,inverse,rot", [(False, False, 64), (True, False, 40), (False, True, 30)])
def test_rope_records_its_gradient(dtype, interleaved, inverse, rot):
    """The gradient of <g, rope(x)> is the transposed map of g, whatever g's strides are."""
    rg = np.random.Generator(np.random.PCG64(rot))
    freqs, factor = B.rrq_rope_frequencies(rot, 10000.0, "yarn", 4.0)
    pos = _dev(np.array([3, 1 << 20, -7], np.int64))
    x = _dev(rg.standard_normal((3, 2, 64)), dtype).requires_grad_()
    for g in (_dev(rg.standard_normal((3, 2, 64)), dtype), _dev(rg.standard_normal((64, 2, 3)), dtype).permute(2, 1, 0),
              torch.ones((), dtype=dtype, device=DEV).expand(3, 2, 64)):
        y = B.rrq_rope(x, pos, freqs, interleaved=interleaved, factor=factor, inverse=inverse)
        with torch.no_grad():
            plain = B.rrq_rope(x, pos, freqs, interleaved=interleaved, factor=factor, inverse=inverse)
        assert torch.equal(y, plain) and not plain.requires_grad
        (got,) = torch.autograd.grad(y, x, g)
        want, size = osv.rope(g.double().cpu().numpy(), pos.cpu().numpy(), freqs, interleaved, factor, not inverse)
        tol = size * (12 * 2.0 ** -24 + 2 * np.pi * (2.0 ** -32 + 2.0 ** 20 * 2.0 ** -65)) + HALF[dtype] * np.abs(want) + 2.0 ** -25
        assert got.dtype == dtype and np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def test_rope_gradient_of_the_gradient_and_what_it_keeps():
    rg = np.random.Generator(np.random.PCG64(3))
    freqs, _ = B.rrq_rope_frequencies(64)
    held = freqs.copy()
    pos = _dev(np.arange(4))
    x = _dev(rg.standard_normal((4, 2, 64)), torch.float32).requires_grad_()
    g = _dev(rg.standard_normal((4, 2, 64)), torch.float32).requires_grad_()
    (gx,) = torch.autograd.grad(B.rrq_rope(x, pos, freqs), x, g, create_graph=True)
    h = _dev(rg.standard_normal((4, 2, 64)), torch.float32)
    (gg,) = torch.autograd.grad(gx, g, h)
    assert torch.equal(gg, B.rrq_rope(h, pos, freqs))
    # the frequencies are the call's own; positions that moved are refused
    y = B.rrq_rope(x, pos, freqs)
    freqs[:] = 0
    (gx,) = torch.autograd.grad(y, x, h)
    assert torch.equal(gx, B.rrq_rope(h, pos, held, inverse=True))
    y = B.rrq_rope(x, pos, held)
    pos += 1
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, x, h)


def test_rope_gradient_captured():
    """Both directions in one graph."""
    rg = np.random.Generator(np.random.PCG64(4))
    freqs, _ = B.rrq_rope_frequencies(64)
    pos = _dev(np.arange(4))
    x = _dev(rg.standard_normal((4, 2, 64)), torch.float32).requires_grad_()
    g = _dev(rg.standard_normal((4, 2, 64)), torch.float32)
    want = B.rrq_rope(x.detach(), pos, freqs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        torch.autograd.grad(B.rrq_rope(x, pos, freqs), x, g)
        with torch.cuda.graph(graph, stream=side):
            y = B.rrq_rope(x, pos, freqs)
            (gx,) = torch.autograd.grad(y, x, g)
    torch.cuda.current_stream().wait_stream(side)
    g.copy_(g.flip(0))
    graph.replay()
    assert torch.equal(y, want) and torch.equal(gx, B.rrq_rope(g, pos, freqs, inverse=True))
