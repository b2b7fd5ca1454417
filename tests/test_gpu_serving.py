"""GPU-vs-oracle parity of the serving calls around the quantised cache (needs a B200):
rrq_attention_shared, rrq_attention_mass, rrq_evict, rrq_rope, and a run of them together.

Tolerances, each derived before its first run:

* attention: per head ‖out − oracle‖ ≤ 2e-3·Σ_t p_t·‖v̂_t‖ + half a step of the output type
  (the bound of decode attention: each term of a convex combination within the
  reconstruction tolerance), eps/2·‖oracle‖ with eps/2 = 2^-11 (fp16), 2^-8 (bf16);
* weights: a weight e^{s − m}/l with s − m exact to half a step, its product with log2 e to
  two more, a base-2 exponential to 2 steps (4 halves), l as a sum of n terms in an order
  that adds at most n/256 + 32 of them one after another, its reciprocal and the product
  to a few halves: relative error ≤ (3·|s − m| + n/256 + 48)·2^-24; the sum over the
  group and with decay·mass adds group + 3 halves of the result;
* rotary: the angle's remainder is at most π/4, rounded to 2^-24 of itself and cut at
  2^-32 turns and |p|·2^-65 turns; sine and cosine to 2 steps of at most 1 each, the
  factor, two products and the sum: (|a| + |b|)·factor·(12·2^-24 + 2π·(2^-32 + |p|·2^-65)),
  then half a step of the output type;
* eviction: equal (integers and moved bytes).
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import rrq as orc
from oracle import serving as osv
from random_rotation_kv_b200 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


# ------------------------------------------------------------------ shared attention
def _rows(rg, rows, d, bits, size):
    """Random codes and log-normal norms of a cache (the encoder is not under test here)."""
    return (rg.integers(0, 256, size=(rows, d * bits // 8), dtype=np.uint8),
            (np.exp(rg.standard_normal(rows) * 0.5) * size).astype(np.float32))


def _part(rg, rows, d, kb, vb, ksize=None, vsize=None):
    ksize, vsize = ksize or math.sqrt(d), vsize or 0.8 * math.sqrt(d)
    return (*_rows(rg, rows, d, kb, ksize), *_rows(rg, rows, d, vb, vsize))


def _attend(q, prefix, tails, lens, hkv, d, kb, vb, scale, dtype, **kw):
    none = [None] * 4
    return B.rrq_attention_shared(
        _dev(q, dtype), *([_dev(x) for x in prefix] if prefix else none), *([_dev(x) for x in tails] if tails else none),
        None if tails is None else _dev(np.asarray(lens, np.int32)), hkv, d, 42, 43, k_bits=kb, v_bits=vb, scale=scale, **kw)


def _check_attention(q, prefix, tails, lens, hkv, d, kb, vb, scale, dtype, what, **kw):
    got = _attend(q, prefix, tails, lens, hkv, d, kb, vb, scale, dtype, **kw)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    seen = _dev(q, dtype).double().cpu().numpy()  # the queries as the call reads them
    ref, weight = osv.attention_shared(seen, prefix, tails, lens, hkv, d, kb, vb, 42, 43, scale=scale)
    err = np.linalg.norm(got - ref, axis=2)
    bound = 2e-3 * weight + HALF[dtype] * np.linalg.norm(ref, axis=2)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    assert np.all(err <= bound), f"{what}: worst error/bound {np.max(err / np.maximum(bound, 1e-300))}"
    return got


@pytest.mark.parametrize("d,kb,vb", [(128, 4, 4), (64, 1, 2), (64, 3, 4), (128, 2, 3), (256, 4, 1), (256, 3, 2), (512, 4, 2)])
@pytest.mark.parametrize("batch,hq,hkv,prefix,cap", [(1, 4, 4, 1, 0), (3, 8, 2, 300, 70), (2, 6, 2, 129, 200), (37, 8, 1, 257, 5),
                                                     (5, 8, 8, 0, 130), (1, 1, 1, 2000, 1)])
def test_attention_shared_parity(d, kb, vb, batch, hq, hkv, prefix, cap):
    rg = np.random.Generator(np.random.PCG64(d * 100 + kb * 10 + vb + batch + prefix))
    dtype = torch.bfloat16 if (batch + kb) % 2 else torch.float16
    p = _part(rg, prefix * hkv, d, kb, vb) if prefix else None
    t = _part(rg, batch * cap * hkv, d, kb, vb) if cap else None
    lens = rg.integers(0, cap + 1, size=batch) if cap else np.zeros(batch, np.int64)
    if cap:
        lens[0] = cap
    q = rg.standard_normal((batch, hq, d))
    _check_attention(q, p, t, lens, hkv, d, kb, vb, 1 / math.sqrt(d), dtype, f"{d} {kb}/{vb} {batch} {hq}/{hkv} {prefix}+{cap}")


@pytest.mark.parametrize("group", [3, 5, 16, 100, 128])
def test_attention_shared_any_group(group):
    rg = np.random.Generator(np.random.PCG64(group))
    p, t = _part(rg, 150 * 2, 64, 4, 4), _part(rg, 3 * 90 * 2, 64, 4, 4)
    _check_attention(rg.standard_normal((3, 2 * group, 64)), p, t, [90, 0, 33], 2, 64, 4, 4, 0.125, torch.float16, f"group {group}")


@pytest.mark.parametrize("d", [64, 512])
def test_attention_shared_lengths(d):
    """Lengths of 0 and 1, around a tile's end, out of range; a sequence with no token at
    all gets zeros; rows behind a length are not looked at (NaN norms there)."""
    rg = np.random.Generator(np.random.PCG64(d + 1))
    cap, hkv = 260, 2
    lens = np.array([0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 260, -5, 1000])
    t = _part(rg, len(lens) * cap * hkv, d, 4, 2)
    seen = np.clip(lens, 0, cap)
    for b, n in enumerate(seen):
        for a in (t[1], t[3]):
            a.reshape(len(lens), cap, hkv)[b, n:] = np.nan
    q = rg.standard_normal((len(lens), 4, d))
    got = _attend(q, None, t, lens, hkv, d, 4, 2, d ** -0.5, torch.float16)
    assert torch.all(got[seen == 0] == 0)
    clean = tuple(np.nan_to_num(x) if x.dtype == np.float32 else x for x in t)
    ref, weight = osv.attention_shared(q.astype(np.float16), None, clean, lens, hkv, d, 4, 2, 42, 43, scale=d ** -0.5)
    err = np.linalg.norm(got.double().cpu().numpy() - ref, axis=2)
    assert np.all(err <= 2e-3 * weight + 2.0 ** -11 * np.linalg.norm(ref, axis=2))
    # with a prefix nothing is empty
    p = _part(rg, 130 * hkv, d, 4, 2)
    _check_attention(q, p, clean, lens, hkv, d, 4, 2, d ** -0.5, torch.float16, "lengths behind a prefix")


@pytest.mark.parametrize("scale,qsize", [(0.0, 1.0), (50.0, 1.0), (-0.1, 1.0), (0.1, 0.0), (0.1, 300.0), (0.1, 1e-6)])
def test_attention_shared_scales(scale, qsize):
    rg = np.random.Generator(np.random.PCG64(9))
    p, t = _part(rg, 400 * 2, 128, 4, 4), _part(rg, 2 * 40 * 2, 128, 4, 4)
    q = rg.standard_normal((2, 8, 128)) * qsize
    _check_attention(q, p, t, [40, 13], 2, 128, 4, 4, scale, torch.float16, f"scale {scale} q {qsize}")


@pytest.mark.parametrize("vsize", [1e-20, 1e-4, 1e3])
def test_attention_shared_value_norm_range(vsize):
    """Value norms far from 1, spread over several orders within the cache, one of them zero."""
    rg = np.random.Generator(np.random.PCG64(10))
    p, t = list(_part(rg, 700 * 2, 128, 4, 4)), list(_part(rg, 2 * 300 * 2, 128, 4, 4))
    for part in (p, t):
        part[3] = (part[3] * vsize * np.exp(rg.standard_normal(part[3].shape) * 2)).astype(np.float32)
        part[3][5] = 0
    q = rg.standard_normal((2, 8, 128))
    if vsize >= 1e-4:
        _check_attention(q, p, t, [300, 7], 2, 128, 4, 4, 128 ** -0.5, torch.bfloat16, f"v {vsize}")
    else:  # bf16 has the range of fp32
        _check_attention(q, p, t, [300, 7], 2, 128, 4, 4, 128 ** -0.5, torch.bfloat16, f"v {vsize}")


def test_attention_shared_growing_scores():
    """Scores that keep rising and falling by hundreds along the cache: the running maximum
    moves at every step, and early states have to be scaled away."""
    rg = np.random.Generator(np.random.PCG64(11))
    p = list(_part(rg, 1500, 128, 4, 4))
    p[1] = (p[1] * np.linspace(0.1, 60, 1500)).astype(np.float32)
    q = rg.standard_normal((4, 4, 128))
    _check_attention(q, p, None, [0] * 4, 1, 128, 4, 4, 0.1, torch.float16, "rising")
    p[1] = p[1][::-1].copy()
    _check_attention(q, p, None, [0] * 4, 1, 128, 4, 4, 0.1, torch.float16, "falling")


@pytest.mark.parametrize("bits", [1, 2, 3, 4])
def test_attention_shared_codebooks(bits):
    """Codebooks of the caller's own, K and V different, not symmetric."""
    rg = np.random.Generator(np.random.PCG64(12 + bits))
    kl = np.sort(rg.standard_normal(1 << bits)).astype(np.float32) * 3
    vl = np.sort(rg.standard_normal(1 << bits)).astype(np.float32) * 0.2
    p = _part(rg, 200 * 2, 128, bits, bits)
    q = rg.standard_normal((3, 4, 128))
    got = _attend(q, p, None, None, 2, 128, bits, bits, 0.05, torch.float16, k_codebook=kl, v_codebook=vl)
    ref, weight = osv.attention_shared(q.astype(np.float16), p, None, [0] * 3, 2, 128, bits, bits, 42, 43, kl, vl, 0.05)
    err = np.linalg.norm(got.double().cpu().numpy() - ref, axis=2)
    assert np.all(err <= 2e-3 * weight + 2.0 ** -11 * np.linalg.norm(ref, axis=2))


def test_attention_shared_long_prefix_many_rows():
    """Several row tiles, many ranges: sampled rows against the oracle."""
    rg = np.random.Generator(np.random.PCG64(13))
    batch, hq, hkv, d, prefix, cap = 70, 8, 2, 128, 5000, 300
    p, t = _part(rg, prefix * hkv, d, 4, 4), _part(rg, batch * cap * hkv, d, 4, 4)
    lens = rg.integers(0, cap + 1, size=batch)
    q = rg.standard_normal((batch, hq, d))
    got = _attend(q, p, t, lens, hkv, d, 4, 4, d ** -0.5, torch.bfloat16)
    pick = [0, 31, 32, 33, 63, 64, 69]
    tp = [x.reshape(batch, cap * hkv, -1)[pick].reshape(len(pick) * cap * hkv, -1) for x in t]
    tp[1], tp[3] = tp[1].reshape(-1), tp[3].reshape(-1)
    seen = _dev(q, torch.bfloat16).double().cpu().numpy()[pick]
    ref, weight = osv.attention_shared(seen, p, tp, lens[pick], hkv, d, 4, 4, 42, 43, scale=d ** -0.5)
    err = np.linalg.norm(got.double().cpu().numpy()[pick] - ref, axis=2)
    assert np.all(err <= 2e-3 * weight + 2.0 ** -8 * np.linalg.norm(ref, axis=2))


@pytest.mark.parametrize("d,dtype", [(128, torch.float16), (128, torch.bfloat16), (64, torch.float16)])
@pytest.mark.parametrize("batch,cap", [(65, 0), (70, 40)])
def test_attention_shared_few_rows_before_many(d, dtype, batch, cap):
    """130 or 140 rows per kv head leave a last tile of 2 or 12 rows, and some ranges go on from
    it to the next head's 128 rows."""
    rg = np.random.Generator(np.random.PCG64(batch + d))
    hkv, prefix = 4, 6400
    p = _part(rg, prefix * hkv, d, 4, 4)
    t = _part(rg, batch * cap * hkv, d, 4, 4) if cap else None
    q = rg.standard_normal((batch, 2 * hkv, d))
    _check_attention(q, p, t, rg.integers(0, cap + 1, size=batch), hkv, d, 4, 4, d ** -0.5, dtype, f"{batch} x 2 rows, d {d}")


def test_attention_shared_is_decode_attention_for_one_sequence():
    """The same cache through rrq_attention_decode: both within the bound of the exact one."""
    rg = np.random.Generator(np.random.PCG64(14))
    for d, kb, vb in ((128, 4, 4), (64, 2, 3)):
        p = _part(rg, 900 * 2, d, kb, vb)
        q = rg.standard_normal((1, 8, d)).astype(np.float16)
        one = B.rrq_attention_decode(_dev(q[0]), *(_dev(x) for x in p), 2, d, 42, 43, k_bits=kb, v_bits=vb, scale=d ** -0.5)
        many = _attend(q, p, None, None, 2, d, kb, vb, d ** -0.5, torch.float16)
        _, weight = osv.attention_shared(q, p, None, [0], 2, d, kb, vb, 42, 43, scale=d ** -0.5)
        err = np.linalg.norm((one - many[0].float()).double().cpu().numpy(), axis=1)
        assert np.all(err <= 4e-3 * weight[0] + 2.0 ** -11 * np.linalg.norm(one.double().cpu().numpy(), axis=1))


def test_attention_shared_repeats_streams_and_graphs():
    """The same bits on every run, with a used workspace, on another stream, and replayed
    from two graphs that share the workspace and run one after the other."""
    rg = np.random.Generator(np.random.PCG64(15))
    batch, hq, hkv, d, prefix, cap = 9, 8, 2, 128, 1100, 140
    p = [_dev(x) for x in _part(rg, prefix * hkv, d, 4, 4)]
    t = [_dev(x) for x in _part(rg, batch * cap * hkv, d, 4, 4)]
    lens = _dev(rg.integers(0, cap + 1, size=batch).astype(np.int32))
    q = [_dev(rg.standard_normal((batch, hq, d)), torch.float16) for _ in range(2)]
    need = B.rrq_attention_shared_workspace_bytes(batch, hq, hkv, d, prefix, cap)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)

    def call(i, out=None):
        return B.rrq_attention_shared(q[i], *p, *t, lens, hkv, d, 42, 43, scale=d ** -0.5, out=out, workspace=ws)

    want = [call(0).clone(), call(1).clone()]
    assert torch.equal(call(0), want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(1)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[1])
    outs = [torch.zeros_like(q[0]) for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, outs[i])
        graphs.append(g)
    lens2 = torch.clamp(lens - 3, min=0)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    # the lengths are read on the device: a replay sees new ones
    lens.copy_(lens2)
    fresh = call(0).clone()
    graphs[0].replay()
    assert torch.equal(outs[0], fresh) and not torch.equal(fresh, want[0])


# ------------------------------------------------------------------------------- mass
def _check_mass(s, hkv, mass, lens, decay, in_place=False):
    sd, md = _dev(s), None if mass is None else _dev(mass)
    ld = None if lens is None else _dev(np.asarray(lens, np.int32))
    got = B.rrq_attention_mass(sd, hkv, mass=md, lens=ld, decay=decay, out=md if in_place else None)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    ref, p, far = osv.attention_mass(s, hkv, mass, lens, float(np.float32(decay)))
    b, hq, t_len = s.shape
    group = hq // hkv
    tol = (p * (3 * far + t_len / 256 + 48)).reshape(b, hkv, group, t_len).sum(2) + (group + 3) * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol * 2.0 ** -24)
    if lens is not None and mass is not None:
        for i, n in enumerate(np.clip(lens, 0, t_len)):
            assert np.array_equal(got[i, :, n:], mass[i, :, n:].astype(np.float64))


@pytest.mark.parametrize("batch,hq,hkv", [(1, 1, 1), (2, 8, 2), (3, 6, 2), (1, 32, 8), (5, 16, 1), (2, 34, 2)])
@pytest.mark.parametrize("t_len", [1, 2, 31, 513, 2047, 9001])
def test_attention_mass_parity(batch, hq, hkv, t_len):
    rg = np.random.Generator(np.random.PCG64(batch * 100 + hq + t_len))
    s = (rg.standard_normal((batch, hq, t_len)) * 3).astype(np.float32)
    s[rg.random(s.shape) < 0.02] = -np.inf
    mass = rg.random((batch, hkv, t_len)).astype(np.float32)
    lens = rg.integers(0, t_len + 1, size=batch)
    _check_mass(s, hkv, mass, lens, 0.9)
    _check_mass(s, hkv, mass, lens, 1.0, in_place=True)
    _check_mass(s, hkv, None, None, 1.0)


@pytest.mark.parametrize("t_len", [100000, 131072, 1000003])
def test_attention_mass_long(t_len):
    rg = np.random.Generator(np.random.PCG64(t_len))
    s = (rg.standard_normal((1, 4, t_len)) * 2).astype(np.float32)
    _check_mass(s, 2, rg.random((1, 2, t_len)).astype(np.float32), None, 0.5)


@pytest.mark.parametrize("hq,t_len", [(100, 512), (102, 510), (300, 41), (1024, 9), (1024, 700)])
def test_attention_mass_many_heads(hq, t_len):
    """Groups whose share of scores just fits shared memory, or does not."""
    rg = np.random.Generator(np.random.PCG64(hq + t_len))
    s = (rg.standard_normal((1, hq, t_len)) * 2).astype(np.float32)
    _check_mass(s, 1, rg.random((1, 1, t_len)).astype(np.float32), None, 0.5)


def test_attention_mass_masks_and_lengths():
    """Heads with every score −inf add nothing; scores as low as the type goes are not masks;
    what stands behind a length (NaN) is not looked at; lengths out of range count as the
    nearer end."""
    rg = np.random.Generator(np.random.PCG64(5))
    s = rg.standard_normal((4, 4, 700)).astype(np.float32)
    s[0, 1] = -np.inf
    s[1, :2] = -np.inf
    s[2, 0] = np.finfo(np.float32).min
    s[2, 1, :] = np.finfo(np.float32).min
    s[2, 1, 5] = 0
    s[2, 2] = 3e38
    s[3, 3, :699] = -np.inf
    mass = rg.random((4, 2, 700)).astype(np.float32)
    _check_mass(s, 2, mass, None, 0.5)
    _check_mass(s, 2, mass, [-3, 0, 1000, 699], 1.0)
    bad = s.copy()
    bad[1, :, 400:] = np.nan
    got = B.rrq_attention_mass(_dev(bad), 2, mass=_dev(mass), lens=_dev(np.array([700, 400, 700, 700], np.int32)))
    ref, _, _ = osv.attention_mass(np.nan_to_num(s, nan=0.0, neginf=-np.inf), 2, mass, [700, 400, 700, 700])
    assert np.all(np.isfinite(got.cpu().numpy()))
    assert np.allclose(got.double().cpu().numpy(), ref, rtol=1e-4, atol=1e-6)


def test_attention_mass_repeats_and_decode_scores():
    """The scores of rrq_qk_scores as they come ([hq, T]); the same bits on every run."""
    rg = np.random.Generator(np.random.PCG64(6))
    kc, kn = _rows(rg, 3000 * 2, 128, 4, 11.0)
    q = _dev(rg.standard_normal((8, 128)), torch.float16)
    s = B.rrq_qk_scores(q, _dev(kc), _dev(kn), 2, 128, 4, 42, scale=128 ** -0.5)
    got = B.rrq_attention_mass(s, 2)
    assert got.shape == (2, 3000)
    total = got.double().sum(1).cpu().numpy()
    assert np.all(np.abs(total - 4) <= 4 * (3 * 30 + 3000 / 256 + 48) * 2.0 ** -24)
    for _ in range(3):
        assert torch.equal(B.rrq_attention_mass(s, 2), got)


# -------------------------------------------------------------------------------- evict
def _check_evict(rg, mass, lens, keep, sink, recent, d=64, kb=2, vb=3, fill=7):
    batch, hkv, cap = mass.shape
    kv = [x.reshape(batch, cap, hkv, *x.shape[1:]) for x in _part(rg, batch * cap * hkv, d, kb, vb)]
    out = [torch.full((batch, keep, *x.shape[2:]), fill, dtype=torch.uint8 if x.dtype == np.uint8 else torch.float32, device=DEV)
           for x in kv]
    index = torch.full((batch, hkv, keep), -9, dtype=torch.int32, device=DEV)
    om = torch.full((batch, hkv, keep), -9.0, device=DEV)
    got = B.rrq_evict(_dev(mass), None if lens is None else _dev(np.asarray(lens, np.int32)), keep, *(_dev(x) for x in kv),
                      sink=sink, recent=recent, index=index, out_mass=om, out=out)
    torch.cuda.synchronize()
    got = [x.cpu().numpy() for x in got]
    kept = osv.evict(mass, lens, keep, sink, recent)
    for b in range(batch):
        m = kept[b].shape[1]
        assert got[1][b] == m
        assert np.array_equal(got[0][b, :, :m], kept[b])
        assert np.all(got[0][b, :, m:] == -9) and np.all(got[2][b, :, m:] == -9)
        for g in range(hkv):
            assert np.array_equal(got[2][b, g, :m], mass[b, g, kept[b][g]], equal_nan=True)
            for o, x in zip(got[3:], kv):
                assert np.array_equal(o[b, :m, g], x[b, kept[b][g], g])
        for o in got[3:]:
            assert np.all(o[b, m:] == fill)


@pytest.mark.parametrize("cap,keep,sink,recent", [(1, 1, 0, 0), (1, 1, 1, 0), (2, 1, 0, 1), (40, 9, 2, 3), (1000, 1000, 0, 0),
                                                  (1025, 512, 4, 508), (3000, 37, 0, 0), (5000, 4999, 1, 1), (100, 200, 3, 3)])
@pytest.mark.parametrize("batch,hkv", [(1, 1), (3, 4)])
def test_evict_parity(cap, keep, sink, recent, batch, hkv):
    rg = np.random.Generator(np.random.PCG64(cap * 7 + keep + batch))
    mass = rg.random((batch, hkv, cap)).astype(np.float32)
    mass[rg.random(mass.shape) < 0.4] = 0  # ties
    lens = rg.integers(0, cap + 1, size=batch)
    lens[0] = cap
    _check_evict(rg, mass, lens, keep, sink, recent)
    _check_evict(rg, mass, None, keep, sink, recent)


@pytest.mark.parametrize("d,kb,vb", [(64, 1, 1), (64, 3, 1), (128, 4, 4), (128, 3, 2), (256, 1, 4), (512, 4, 4)])
def test_evict_row_sizes(d, kb, vb):
    rg = np.random.Generator(np.random.PCG64(d + kb))
    _check_evict(rg, rg.random((2, 3, 200)).astype(np.float32), [200, 77], 90, 1, 5, d, kb, vb)


def test_evict_values_of_every_kind():
    """All equal; negative, infinite and NaN masses, both zeros; lengths out of range."""
    rg = np.random.Generator(np.random.PCG64(21))
    _check_evict(rg, np.zeros((2, 2, 5000), np.float32), [5000, 4000], 1700, 2, 2)
    m = rg.choice(np.array([-1, -0.0, 0.0, 1, np.inf, -np.inf, np.nan, 1e-45, -1e-45, 3e38], np.float32), size=(3, 2, 700))
    for keep in (1, 100, 350, 600, 699):
        _check_evict(rg, m, [700, -2, 9000], keep, 0, 0)


@pytest.mark.parametrize("cap", [70000, 131072, 300001])
def test_evict_long(cap):
    rg = np.random.Generator(np.random.PCG64(cap))
    mass = (np.round(np.exp(rg.standard_normal((1, 2, cap)) * 2) * 64) / 64).astype(np.float32)
    _check_evict(rg, mass, None, cap // 3, 4, 1000, 64, 1, 1)


# --------------------------------------------------------------------------------- rope
def _check_rope(x, pos, freqs, interleaved, factor, inverse, dtype, in_place=False):
    xd = _dev(x, dtype)
    seen = xd.double().cpu().numpy()
    got = B.rrq_rope(xd, _dev(np.asarray(pos, np.int64)), freqs, interleaved=interleaved, factor=factor, inverse=inverse,
                     out=xd if in_place else None)
    torch.cuda.synchronize()
    got = got.double().cpu().numpy()
    ref, size = osv.rope(seen, pos, freqs, interleaved, factor, inverse)
    far = np.abs(np.asarray(pos, np.float64))[:, None, None]
    tol = size * (12 * 2.0 ** -24 + 2 * math.pi * (2.0 ** -32 + far * 2.0 ** -65)) + HALF[dtype] * np.abs(ref)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25  # half a step of the subnormal values
    rot = 2 * len(freqs)
    assert np.all(np.abs(got - ref)[..., :rot] <= tol[..., :rot])
    assert np.array_equal(got[..., rot:], seen[..., rot:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,heads,d,rot", [(1, 1, 64, 64), (1, 32, 128, 128), (7, 3, 128, 48), (5, 2, 64, 2), (4, 5, 256, 250),
                                           (3, 2, 512, 512), (300, 8, 128, 128), (33, 7, 64, 38)])
def test_rope_parity(dtype, interleaved, n, heads, d, rot):
    rg = np.random.Generator(np.random.PCG64(n * 1000 + rot + heads))
    freqs, factor = osv.rope_frequencies("yarn" if rot > 2 else "none", rot, 10000.0, 4.0)
    x = rg.standard_normal((n, heads, d))
    pos = rg.integers(0, 200000, size=n)
    _check_rope(x, pos, freqs, interleaved, factor, False, dtype)
    _check_rope(x, pos, freqs, interleaved, factor, True, dtype, in_place=True)


def test_rope_far_positions():
    """Positions of any sign and size: the angle keeps every digit that the frequencies have."""
    rg = np.random.Generator(np.random.PCG64(31))
    pos = [0, 1, -1, 2 ** 20, 2 ** 31 - 1, -2 ** 31, 2 ** 33 + 5, 10 ** 12 + 7, -10 ** 12]
    freqs, _ = osv.rope_frequencies("none", 128, 10000.0)
    _check_rope(rg.standard_normal((len(pos), 2, 128)), pos, freqs, False, 1.0, False, torch.float32)
    odd = rg.uniform(-50, 50, size=32)
    odd[:4] = [0.0, math.pi / 2, -math.pi, 2.0 ** 30]
    _check_rope(rg.standard_normal((len(pos), 2, 64)), pos, odd, True, 0.5, True, torch.float32)


def test_rope_gradient():
    """inverse = 1 is the gradient: against the transposed formula (the oracle's) above, and
    here against differences of the map itself, ⟨g, (rope(x + h·e) − rope(x))/h⟩ in 64 bits
    of fp32 outputs; the map is linear, so with h = 1 the difference is exact but for two
    roundings of at most 2^-24·12·(|a| + |b|) each."""
    rg = np.random.Generator(np.random.PCG64(32))
    n, heads, d, rot = 3, 2, 64, 40
    freqs, factor = B.rrq_rope_frequencies(rot, 10000.0, "yarn", 8.0)
    pos = _dev(np.array([5, 100000, 7], np.int64))
    x = rg.standard_normal((n, heads, d)).astype(np.float32)
    g = rg.standard_normal((n, heads, d)).astype(np.float32)
    for interleaved in (False, True):
        def f(v):
            return B.rrq_rope(_dev(v), pos, freqs, interleaved=interleaved, factor=factor).double().cpu().numpy()
        grad = B.rrq_rope(_dev(g), pos, freqs, interleaved=interleaved, factor=factor, inverse=True).double().cpu().numpy()
        base = f(x)
        for at in [(0, 0, 0), (1, 1, 19), (2, 0, 20), (1, 0, 39), (0, 1, 40), (2, 1, 63)]:
            e = x.copy()
            e[at] += 1
            step = float(e[at]) - float(x[at])  # what the addition in fp32 made of 1
            diff = float((g[at[0], at[1]].astype(np.float64) * (f(e) - base)[at[0], at[1]]).sum()) / step
            assert abs(diff - grad[at]) <= 64 * 12 * 2.0 ** -24 * 4 * 4


def test_rope_captured():
    rg = np.random.Generator(np.random.PCG64(33))
    freqs, _ = osv.rope_frequencies("none", 128, 10000.0)
    x, pos = _dev(rg.standard_normal((4, 8, 128)), torch.bfloat16), _dev(np.arange(4))
    out = torch.zeros_like(x)
    B.rrq_rope(x, pos, freqs, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        B.rrq_rope(x, pos, freqs, out=out)
    pos += 100
    g.replay()
    assert torch.equal(out, B.rrq_rope(x, pos, freqs))


# ------------------------------------------------------------------------ all together
def test_serving_loop():
    """Prompt and answers of a small batch: rotary positions, encoding, attention over the
    shared prefix and the tails, accumulated weights of one sequence, eviction of its tail,
    attention again — against the oracle on the codes that the library made."""
    rg = np.random.Generator(np.random.PCG64(41))
    batch, hq, hkv, d, prefix, cap, kb, vb = 3, 8, 2, 128, 200, 60, 4, 4
    freqs, factor = B.rrq_rope_frequencies(d, 10000.0, "linear", 2.0)

    def encode(x, bits, seed):
        c, n = B.rrq_encode(x.contiguous(), bits, seed)
        return c, n

    k = B.rrq_rope(_dev(rg.standard_normal((prefix, hkv, d)), torch.float16), _dev(np.arange(prefix)), freqs, factor=factor)
    p = [*encode(k, kb, 42), *encode(_dev(rg.standard_normal((prefix, hkv, d)), torch.float16), vb, 43)]
    pos = _dev(np.tile(prefix + np.arange(cap), batch))
    k = B.rrq_rope(_dev(rg.standard_normal((batch * cap, hkv, d)), torch.float16), pos, freqs, factor=factor)
    t = [x.view(batch, cap, *x.shape[1:]) for x in
         (*encode(k, kb, 42), *encode(_dev(rg.standard_normal((batch * cap, hkv, d)), torch.float16), vb, 43))]
    lens = _dev(np.array([60, 0, 33], np.int32))
    q = B.rrq_rope(_dev(rg.standard_normal((batch, hq, d)), torch.float16), _dev(prefix + np.array([60, 0, 33])), freqs,
                   factor=factor)

    def check(tails, lengths):
        got = B.rrq_attention_shared(q, *p, *tails, lengths, hkv, d, 42, 43, k_bits=kb, v_bits=vb, scale=d ** -0.5)
        host = [[x.reshape(-1, x.shape[-1]).cpu().numpy() if x.dtype == torch.uint8 else x.reshape(-1).cpu().numpy() for x in c]
                for c in (p, tails)]
        ref, weight = osv.attention_shared(q.double().cpu().numpy(), *host, lengths.cpu().numpy(), hkv, d, kb, vb, 42, 43,
                                           scale=d ** -0.5)
        err = np.linalg.norm(got.double().cpu().numpy() - ref, axis=2)
        assert np.all(err <= 2e-3 * weight + 2.0 ** -11 * np.linalg.norm(ref, axis=2))

    check(t, lens)
    s = torch.stack([B.rrq_qk_scores(q[b], t[0][b].reshape(cap * hkv, -1), t[1][b].reshape(-1), hkv, d, kb, 42, scale=d ** -0.5)
                     for b in range(batch)])
    mass = B.rrq_attention_mass(s, hkv, lens=lens)
    mass = B.rrq_attention_mass(s, hkv, mass=mass, lens=lens, decay=0.9, out=mass)
    assert np.allclose(mass.sum(2).cpu().numpy(), [[7.6] * 2, [0] * 2, [7.6] * 2], atol=1e-3)
    index, new_lens, new_mass, *cut = B.rrq_evict(mass, lens, 20, *t, sink=2, recent=5)
    kept = osv.evict(mass.cpu().numpy(), lens.cpu().numpy(), 20, 2, 5)
    assert new_lens.tolist() == [20, 0, 20]
    for b in (0, 2):
        assert np.array_equal(index[b].cpu().numpy(), kept[b])
    check(cut, new_lens)


def test_serving_calls_captured():
    """A decode step's calls in one graph, replayed on other inputs and lengths: what the calls give
    one by one."""
    b, hq, hkv, d, cap, keep = 3, 8, 2, 128, 300, 90
    freqs, factor = B.rrq_rope_frequencies(d)
    g = torch.Generator(device=DEV).manual_seed(3)
    p = _part(np.random.Generator(np.random.PCG64(3)), 200 * hkv, d, 4, 4)
    t = _part(np.random.Generator(np.random.PCG64(4)), b * cap * hkv, d, 4, 4)
    p, t = [_dev(x) for x in p], [_dev(x) for x in t]
    q = torch.empty(b, hq, d, device=DEV, dtype=torch.float16)
    scores = torch.empty(b, hq, cap, device=DEV)
    pos = torch.empty(b, device=DEV, dtype=torch.int64)
    lens = torch.empty(b, device=DEV, dtype=torch.int32)
    mass = torch.empty(b, hkv, cap, device=DEV)

    def fill(lengths, first):
        q.copy_(torch.randn(q.shape, device=DEV, generator=g))
        scores.copy_(torch.randn(scores.shape, device=DEV, generator=g))
        mass.copy_(torch.rand(mass.shape, device=DEV, generator=g))
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        pos.copy_(torch.arange(b) + first)

    def step():
        turned = B.rrq_rope(q, pos, freqs, factor=factor)
        out = B.rrq_attention_shared(turned, *p, *t, lens, hkv, d, 1, 2, scale=d ** -0.5)
        m = B.rrq_attention_mass(scores, hkv, mass=mass, lens=lens, decay=0.5)
        shaped = [x.view(b, cap, hkv, *x.shape[1:]) for x in t]
        return [turned, out, m, *B.rrq_evict(m, lens, keep, *shaped, sink=4, recent=10)]

    fill([300, 17, 91], 5)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            held = step()
    torch.cuda.current_stream().wait_stream(side)
    for lengths, first in (([300, 17, 91], 9), ([0, 300, 90], 1 << 40), ([1, 2, 299], 0)):
        fill(lengths, first)
        graph.replay()
        torch.cuda.synchronize()
        for got, want in zip(held, step()):
            assert torch.equal(got, want)
