"""The serving calls where their numbers leave the ordinary range (needs a B200): weights times
value norms over many orders.  Tolerances as in test_gpu_serving.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import rrq as orc
from tests.test_gpu_serving import _attend, _check_attention, _part

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
