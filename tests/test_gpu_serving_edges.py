"""The serving calls where their kernels change path or their numbers leave the ordinary range
(needs a B200): weights times value norms over many orders, more sequences and rows than one
pass of the layout takes, every cluster size, addresses that are aligned as the calls ask
and no further, rotary positions in a graph of gradients.  Tolerances as in
test_gpu_serving.py unless a test derives its own."""

from __future__ import annotations

import math
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import rrq as orc
from oracle import serving as osv
from random_rotation_kv_b200 import binding as B
from tests.conftest import ROOT
from tests.test_gpu_serving import DEV, HALF, _attend, _check_attention, _check_mass, _dev, _part

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


@pytest.mark.parametrize("batch,prefix,cap,d,kb,vb", [(300, 130, 40, 64, 4, 4), (300, 0, 200, 128, 4, 4), (513, 70, 1, 64, 2, 3),
                                                      (260, 0, 33, 256, 4, 4), (260, 40, 20, 512, 4, 4)])
def test_attention_shared_many_sequences(batch, prefix, cap, d, kb, vb):
    """More sequences than the layout takes at a time, more query rows than are merged by
    eight warps each; empty tails among them."""
    rg = np.random.Generator(np.random.PCG64(batch + d))
    hkv, hq = 2, 8
    p = _part(rg, prefix * hkv, d, kb, vb) if prefix else None
    t = _part(rg, batch * cap * hkv, d, kb, vb)
    lens = rg.integers(0, cap + 1, size=batch)
    lens[[0, 100, 255, 256, 257]] = [cap, 0, cap, 0, cap]
    _check_attention(rg.standard_normal((batch, hq, d)), p, t, lens, hkv, d, kb, vb, d ** -0.5, torch.bfloat16, f"{batch}")


@pytest.mark.parametrize("d,alpha", [(64, "0x1.429a86p+0"), (128, "0x1.429a86p+0"), (256, "0x1.429a86p+0"), (512, None)])
@pytest.mark.parametrize("hq", [4, 48])
@pytest.mark.parametrize("scale,knorm", [(0.06, 1.0), (0.5, 1.0), (1.0, 1.0), (0.1, 20.0)])
def test_attention_shared_large_scores(d, alpha, hq, scale, knorm):
    """Scores of tens of nats, where one part of 11 bits per query would be off by more than the output's
    bound: against the attention of key levels rounded as the kernel's (fp16 after a factor) the
    output is within 2e-3·Σ p‖v̂‖ and what the queries' 22 bits cost: a score is off by at most
    δ = 2^-22·scale·‖q‖·‖k̂‖, the output by at most 2δ·Σ p‖v̂‖ (δ is 7e-5 to 3e-3 here)."""
    rg = np.random.Generator(np.random.PCG64(77))
    hkv, tokens, cap = 2, 900, 200
    p, t = list(_part(rg, tokens * hkv, d, 4, 4)), list(_part(rg, 3 * cap * hkv, d, 4, 4))
    p[1], t[1] = (p[1] * knorm).astype(np.float32), (t[1] * knorm).astype(np.float32)
    lens = [cap, 0, 77]
    q = rg.standard_normal((3, hq, d))
    got = _attend(q, p, t, lens, hkv, d, 4, 4, scale, torch.bfloat16)
    levels = np.asarray(orc.default_levels(4), np.float32)
    if alpha:  # of 4-bit levels (attention_shared_levels); the kernel for d = 512 takes them as they are
        factor = np.float32(float.fromhex(alpha))
        levels = np.float64(np.float16(levels * factor)) / np.float64(factor)
    seen = _dev(q, torch.bfloat16).double().cpu().numpy()
    ref, weight = osv.attention_shared(seen, p, t, lens, hkv, d, 4, 4, 42, 43, k_levels=levels, scale=float(np.float32(scale)))
    keys = max(np.linalg.norm(orc.dequantize_rotated(orc.unpack_codes(c[0], 4, d), c[1], 4, None), axis=1).max() for c in (p, t))
    delta = 2.0 ** -22 * scale * np.linalg.norm(seen, axis=2) * keys
    err = np.linalg.norm(got.double().cpu().numpy() - ref, axis=2)
    assert np.all(err <= (2e-3 + 2 * delta) * weight + 2.0 ** -8 * np.linalg.norm(ref, axis=2))


@pytest.mark.parametrize("d,hq", [(128, 2), (128, 24), (64, 24), (256, 8)])
def test_attention_shared_norms_a_few_octaves_apart(d, hq):
    """Value norms inside and outside the span for which a tile's largest norm stands for all, the large
    ones where the scores are low."""
    for octaves in (4.9, 5.1, 12.0):
        rg = np.random.Generator(np.random.PCG64(int(octaves * 10) + d + hq))
        p = list(_part(rg, 1000, d, 4, 4))
        big = rg.random(1000) < 0.3
        p[1] = np.where(big, 1e-3, p[1]).astype(np.float32)
        p[3] = np.where(big, 2.0 ** octaves, 1.0).astype(np.float32)
        q = rg.standard_normal((1, hq, d)) * 2
        _check_attention(q, p, None, [0], 1, d, 4, 4, d ** -0.5, torch.bfloat16, f"{octaves}")


@pytest.mark.parametrize("d", [64, 128, 256, 512])
def test_attention_shared_keeps_sequences_apart(d):
    """Queries of one sequence that are NaN or infinite, and NaN norms in its tail, leave the bits of all
    others as they are."""
    rg = np.random.Generator(np.random.PCG64(d + 3))
    p, t = _part(rg, 260 * 2, d, 4, 4), _part(rg, 6 * 150 * 2, d, 4, 4)
    lens = [150, 20, 150, 0, 99, 1]
    for hq in (4, 48):
        q = rg.standard_normal((6, hq, d))
        want = _attend(q, p, t, lens, 2, d, 4, 4, d ** -0.5, torch.float16)
        q[2, 1], q[2, hq - 1, 3] = np.nan, np.inf
        bad = [x.copy() for x in t]
        for a in (bad[1], bad[3]):
            a.reshape(6, 150, 2)[2, 70] = np.nan
        got = _attend(q, p, bad, lens, 2, d, 4, 4, d ** -0.5, torch.float16)
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(got[keep], want[keep]) and torch.all(torch.isnan(got[2]))


def test_attention_shared_on_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own."""
    rg = np.random.Generator(np.random.PCG64(90))
    jobs = []
    for d, batch in ((128, 20), (64, 33)):
        p, t = [_dev(x) for x in _part(rg, 3000 * 2, d, 4, 4)], [_dev(x) for x in _part(rg, batch * 100 * 2, d, 4, 4)]
        q, lens = _dev(rg.standard_normal((batch, 8, d)), torch.float16), _dev(rg.integers(0, 101, size=batch).astype(np.int32))
        jobs.append((d, lambda d=d, p=p, t=t, q=q, lens=lens: B.rrq_attention_shared(q, *p, *t, lens, 2, d, 42, 43, scale=d ** -0.5)))
    want = [f() for _, f in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for _ in range(10):
        for i, (_, f) in enumerate(jobs):
            with torch.cuda.stream(streams[i]):
                got[i].append(f())
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(w, o) for o in outs)


def test_serving_calls_on_nothing():
    """Batches, caches and positions of size zero through the Python entry points."""
    u8, f32 = torch.uint8, torch.float32

    def part(*lead):
        return [x for _ in range(2) for x in (torch.empty(*lead, 32, dtype=u8, device=DEV), torch.empty(*lead, dtype=f32, device=DEV))]

    def q(n):
        return torch.ones(n, 4, 64, dtype=torch.float16, device=DEV)

    none, zero = [None] * 4, torch.zeros(3, dtype=torch.int32, device=DEV)
    assert B.rrq_attention_shared(q(0), *part(5, 2), *none, None, 2, 64, 1, 2).shape == (0, 4, 64)
    for prefix, tails, lens in ((part(0, 2), none, None), (none, part(3, 0, 2), zero), (part(0, 2), part(3, 0, 2), zero),
                                (none, part(3, 7, 2), zero), (none, none, None)):
        assert torch.all(B.rrq_attention_shared(q(3), *prefix, *tails, lens, 2, 64, 1, 2) == 0)
    assert B.rrq_attention_mass(torch.empty(0, 4, 9, device=DEV), 2).shape == (0, 2, 9)
    assert B.rrq_attention_mass(torch.empty(3, 4, 0, device=DEV), 2, lens=zero).shape == (3, 2, 0)
    index, lens, mass, *cut = B.rrq_evict(torch.empty(3, 2, 0, device=DEV), zero, 4, *part(3, 0, 2))
    assert lens.tolist() == [0, 0, 0] and torch.all(index == -1) and torch.all(mass == 0) and cut[0].shape == (3, 4, 2, 32)
    assert B.rrq_evict(torch.empty(0, 2, 5, device=DEV), None, 4, *part(0, 5, 2))[1].shape == (0,)
    assert B.rrq_rope(torch.empty(0, 4, 64, device=DEV), torch.empty(0, dtype=torch.int64, device=DEV), np.ones(8)).shape == (0, 4, 64)


# ------------------------------------------------------------------------------- mass
@pytest.mark.parametrize("batch,hq,hkv,t_len", [(1, 32, 8, 131072),  # clusters of 10
                                                (1, 16, 2, 65536), (1, 8, 8, 100004),
                                                (5, 16, 1, 2048), (2, 40, 2, 1024),  # heads that share the last copy barrier
                                                (80, 1, 1, 20000), (150, 2, 2, 17000)])  # runs longer than a thread's registers
def test_attention_mass_cluster_sizes(batch, hq, hkv, t_len):
    rg = np.random.Generator(np.random.PCG64(batch * 100 + hq + t_len))
    s = (rg.standard_normal((batch, hq, t_len), dtype=np.float32) * 3)
    s[rg.random(s.shape, dtype=np.float32) < 0.02] = -np.inf
    mass = rg.random((batch, hkv, t_len), dtype=np.float32)
    lens = rg.integers(0, t_len + 1, size=batch)
    lens[0] = t_len - 3
    _check_mass(s, hkv, mass, lens, 0.9)
    _check_mass(s, hkv, mass, lens, 1.0, in_place=True)


def _shifted(a, elements):
    """The array at an address `elements` elements behind an aligned one."""
    t = _dev(a)
    buf = torch.empty(t.numel() + elements, dtype=t.dtype, device=DEV)
    view = buf[elements:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("which", ["scores", "mass", "out"])
def test_attention_mass_addresses(which):
    """4-byte alignment is enough for every array, also where T is a multiple of 4."""
    rg = np.random.Generator(np.random.PCG64(8))
    s = rg.standard_normal((2, 8, 1200)).astype(np.float32)
    mass = rg.random((2, 2, 1200)).astype(np.float32)
    lens = _dev(np.array([1200, 601], np.int32))
    want, p, far = osv.attention_mass(s, 2, mass, [1200, 601], 0.5)
    off = {k: int(k == which) for k in ("scores", "mass", "out")}
    out = _shifted(np.zeros_like(mass), off["out"])
    got = B.rrq_attention_mass(_shifted(s, off["scores"]), 2, mass=_shifted(mass, off["mass"]), lens=lens, decay=0.5, out=out)
    tol = (p * (3 * far + 1200 / 256 + 48)).reshape(2, 2, 4, 1200).sum(2) + 7 * np.abs(want)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol * 2.0 ** -24)


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
        tol = size * (12 * 2.0 ** -24 + 2 * math.pi * (2.0 ** -32 + 2.0 ** 20 * 2.0 ** -65)) + HALF[dtype] * np.abs(want) + 2.0 ** -25
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


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [128, 48, 50])
def test_rope_addresses(dtype, interleaved, rot):
    """16-byte alignment is enough, for each array on its own."""
    rg = np.random.Generator(np.random.PCG64(rot))
    freqs, factor = B.rrq_rope_frequencies(rot, 10000.0)
    x = _dev(rg.standard_normal((9, 3, 128)), dtype)
    pos = _dev(np.arange(9) * 1000)
    buf = [torch.empty(x.numel() + 16, dtype=dtype, device=DEV) for _ in range(2)]
    skip = 16 // x.element_size()
    xs, ys = (b[skip:skip + x.numel()].view(x.shape) for b in buf)
    xs.copy_(x)
    assert xs.data_ptr() % 32 == 16 and ys.data_ptr() % 32 == 16
    want, size = osv.rope(x.double().cpu().numpy(), pos.cpu().numpy(), freqs, interleaved, factor)
    for src, dst in ((xs, ys), (xs, torch.empty_like(x)), (x, ys)):
        got = B.rrq_rope(src, pos, freqs, interleaved=interleaved, factor=factor, out=dst).double().cpu().numpy()
        far = 9000.0
        tol = size * (12 * 2.0 ** -24 + 2 * math.pi * (2.0 ** -32 + far * 2.0 ** -65)) + HALF[dtype] * np.abs(want) + 2.0 ** -25
        assert np.all(np.abs(got - want)[..., :rot] <= tol[..., :rot])
        assert np.array_equal(got[..., rot:], x.double().cpu().numpy()[..., rot:])


# ------------------------------------------------------------------------ all together
def test_evicted_caches_grow():
    """Sequences evicted one by one into the beginning of larger caches, a token appended to each, and
    attention over them: against the oracle on the same rows."""
    rg = np.random.Generator(np.random.PCG64(51))
    batch, hq, hkv, d, cap, keep = 3, 8, 2, 128, 90, 40
    t = [_dev(x).view(batch, cap, hkv, *x.shape[1:]) for x in _part(rg, batch * cap * hkv, d, 4, 4)]
    lens = _dev(np.array([90, 25, 41], np.int32))
    mass = _dev(rg.random((batch, hkv, cap)).astype(np.float32))
    new = [torch.zeros_like(x) for x in t]
    new_lens = torch.empty_like(lens)
    for b in range(batch):
        one = slice(b, b + 1)
        B.rrq_evict(mass[one], lens[one], keep, *(x[one] for x in t), sink=2, recent=5, out_lens=new_lens[one],
                    out=[x[one, :keep] for x in new])
    kept = osv.evict(mass.cpu().numpy(), lens.cpu().numpy(), keep, 2, 5)
    assert new_lens.tolist() == [40, 25, 40]
    for x, old in zip(new, t):
        for b in range(batch):
            for g in range(hkv):
                assert torch.equal(x[b, :len(kept[b][g]), g], old[b, torch.from_numpy(kept[b][g]).to(DEV), g])
                assert torch.all(x[b, len(kept[b][g]):, g] == 0)
    at = new_lens.long()
    for w, bits, seed in ((0, 4, 42), (2, 4, 43)):
        codes, norms = B.rrq_encode(_dev(rg.standard_normal((batch, hkv, d)), torch.float16), bits, seed)
        new[w][torch.arange(batch, device=DEV), at], new[w + 1][torch.arange(batch, device=DEV), at] = codes, norms
    host = [x.reshape(-1, *x.shape[3:]).cpu().numpy() for x in new]
    _check_attention(rg.standard_normal((batch, hq, d)), None, host, (at + 1).tolist(), hkv, d, 4, 4, d ** -0.5, torch.float16,
                     "grown")


FIRST_CALLS_CAPTURED = """
import torch
from random_rotation_kv_b200 import binding as B
dev = "cuda:0"
gen = torch.Generator(device=dev).manual_seed(1)

def part(*lead):
    return [x for _ in range(2) for x in (torch.randint(0, 256, (*lead, 64), device=dev, generator=gen).to(torch.uint8),
                                          torch.rand(*lead, device=dev, generator=gen) + 0.5)]

q, pos = torch.randn(3, 8, 128, device=dev, generator=gen).half(), torch.arange(3, device=dev)
p, t, lens = part(200, 2), part(3, 50, 2), torch.tensor([50, 0, 7], dtype=torch.int32, device=dev)
scores, freqs = torch.randn(3, 8, 50, device=dev, generator=gen), B.rrq_rope_frequencies(128)[0]

def step():
    turned = B.rrq_rope(q, pos, freqs)
    out = B.rrq_attention_shared(turned, *p, *t, lens, 2, 128, 1, 2, scale=0.1)
    mass = B.rrq_attention_mass(scores, 2, lens=lens)
    return [turned, out, mass, *B.rrq_evict(mass, lens, 20, *t, sink=1, recent=2)]

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(held, step()))
print("captured")
"""


def test_serving_calls_captured_before_any_other():
    """A process whose first use of the calls is a capture."""
    done = subprocess.run([sys.executable, "-c", FIRST_CALLS_CAPTURED], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert done.returncode == 0 and "captured" in done.stdout, done.stderr[-2000:]
