"""The serving calls without a GPU: pins of their oracle, refusals before any launch, the
host-side frequency schedules and workspace sizes."""

from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import rrq as orc
from oracle import serving as osv
from random_rotation_kv_b200 import binding as B

# fake, never-dereferenced device addresses
P = ctypes.c_void_p(0x10000)
P_MIS = ctypes.c_void_p(0x10002)
NULL = ctypes.c_void_p(None)
INVALID, UNSUPPORTED, OK = B.RRQ_ERR_INVALID, B.RRQ_ERR_UNSUPPORTED, B.RRQ_OK


# ------------------------------------------------------------------------- oracle pins
def _cache(rg, rows, d, kb, vb):
    ek = orc.encode(rg.standard_normal((rows, d)), kb, 42)
    ev = orc.encode(rg.standard_normal((rows, d)), vb, 43)
    return ek.packed, ek.norms, ev.packed, ev.norms


def test_shared_attention_oracle_is_decode_attention_for_one_sequence():
    rg = np.random.Generator(np.random.PCG64(1))
    hq, hkv, d, t_len = 8, 2, 64, 40
    c = _cache(rg, t_len * hkv, d, 3, 2)
    q = rg.standard_normal((1, hq, d))
    want = oatt.decode_attention(q[0], *c, t_len, hkv, d, 3, 2, 42, 43, scale=0.2)
    got, _ = osv.attention_shared(q, c, None, [0], hkv, d, 3, 2, 42, 43, scale=0.2)
    assert np.allclose(got[0], want, rtol=0, atol=1e-12)
    # the same tokens as prefix and tail, cut anywhere
    for cut in (0, 1, 17, 40):
        head = tuple(x[:cut * hkv] for x in c) if cut else None
        tail = tuple(x[cut * hkv:] for x in c) if cut < t_len else None
        got, _ = osv.attention_shared(q, head, tail, [t_len - cut], hkv, d, 3, 2, 42, 43, scale=0.2)
        assert np.allclose(got[0], want, rtol=0, atol=1e-12)


def test_mass_oracle_weights_sum_to_one_per_head():
    rg = np.random.Generator(np.random.PCG64(2))
    s = rg.standard_normal((2, 6, 30))
    s[0, 3] = -np.inf  # a head with every token masked adds nothing
    out, _, _ = osv.attention_mass(s, 3, lens=[30, 11])
    assert np.allclose(out.sum(2), [[2, 1, 2], [2, 2, 2]])
    assert np.all(out[1, :, 11:] == 0)


def test_evict_oracle_ties_and_forced_tokens():
    m = np.array([[[5.0, 0, 0, 7, 0, 0, 0, 0]]])
    assert osv.evict(m, None, 4, 0, 0)[0].tolist() == [[0, 1, 2, 3]]
    assert osv.evict(m, None, 4, 0, 2)[0].tolist() == [[0, 3, 6, 7]]
    assert osv.evict(m, [3], 4, 2, 2)[0].tolist() == [[0, 1, 2]]
    m[0, 0, 1] = np.nan
    m[0, 0, 2] = -np.inf
    assert osv.evict(m, None, 7, 0, 0)[0].tolist() == [[0, 2, 3, 4, 5, 6, 7]]


def test_rope_oracle_inverse_and_frequencies():
    rg = np.random.Generator(np.random.PCG64(3))
    x = rg.standard_normal((3, 2, 64))
    f, factor = osv.rope_frequencies("yarn", 32, 10000.0, 4.0)
    assert f[0] == 1.0 and abs(f[-1] - 10000.0 ** (-30 / 32) / 4) < 1e-15 and factor > 1
    y, _ = osv.rope(x, [5, -7, 10 ** 12], f, True, factor)
    z, _ = osv.rope(y, [5, -7, 10 ** 12], f, True, factor, inverse=True)
    want = x.copy()
    want[..., :32] *= factor ** 2
    assert np.allclose(z, want, rtol=0, atol=1e-12)


# --------------------------------------------------------------- host-side schedules
@pytest.mark.parametrize("schedule", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot", [2, 6, 64, 128, 512])
def test_rope_frequencies_match_the_oracle(schedule, rot):
    for base, stretch, original in ((10000.0, 1.0, 8192.0), (500000.0, 8.0, 4096.0)):
        got, factor = B.rrq_rope_frequencies(rot, base, schedule, stretch, original)
        want, wfactor = osv.rope_frequencies(schedule, rot, base, stretch, original)
        # a power, a logarithm, a quotient and a product in 64 bits, each within a few 2^-53;
        # the power's exponent is at most ln(base)·2 ≈ 40, which multiplies its error
        assert np.all(np.abs(got - want) <= 200 * 2.0 ** -53 * want)
        assert abs(factor - wfactor) <= 4 * 2.0 ** -53 * wfactor


def test_rope_refusals():
    lib = B.lib()
    f = (ctypes.c_double * 256)(*([0.5] * 256))
    fp, one = ctypes.cast(f, ctypes.c_void_p), ctypes.c_double()
    op = ctypes.c_void_p(ctypes.addressof(one))

    def freq(schedule=0, rot=64, base=1e4, stretch=1.0, original=8192.0, fast=32.0, slow=1.0, out=fp, fac=op):
        return lib.rrq_rope_frequencies(schedule, rot, base, stretch, original, fast, slow, out, fac)

    assert freq() == OK
    for bad in (dict(schedule=4), dict(schedule=-1), dict(rot=0), dict(rot=3), dict(rot=514), dict(base=1.0),
                dict(base=math.inf), dict(base=math.nan), dict(stretch=0.5), dict(stretch=math.inf),
                dict(schedule=3, original=0.0), dict(schedule=3, fast=0.5), dict(schedule=3, slow=0.0),
                dict(schedule=3, fast=math.nan), dict(out=NULL), dict(fac=NULL)):
        assert freq(**bad) == INVALID, bad

    def rope(x=P, dt=B.RRQ_F16, n=4, heads=2, d=128, rot=64, inter=0, pos=P, freqs=fp, factor=1.0, inv=0, y=P):
        return lib.rrq_rope(x, dt, n, heads, d, rot, inter, pos, freqs, factor, inv, y, None)

    for bad in (dict(n=-1), dict(heads=0), dict(d=96), dict(d=1024), dict(rot=0), dict(rot=7), dict(rot=130),
                dict(inter=2), dict(inv=2), dict(dt=5), dict(factor=math.inf), dict(factor=math.nan), dict(factor=1e300),
                dict(freqs=NULL), dict(x=P_MIS), dict(y=P_MIS), dict(pos=P_MIS), dict(x=NULL), dict(y=NULL),
                dict(pos=NULL)):
        assert rope(**bad) == INVALID, bad
    for v in (math.inf, math.nan, 2.0 ** 31, -2.0 ** 31):
        f[5] = v
        assert rope() == INVALID
    f[5] = 0.5
    assert rope(n=0, x=NULL, y=NULL, pos=NULL) == OK


def test_mass_refusals():
    lib = B.lib()

    def mass(s=P, b=2, hq=8, hkv=2, t=16, lens=P, decay=1.0, m=P, out=P):
        return lib.rrq_attention_mass(s, b, hq, hkv, t, lens, decay, m, out, None)

    for bad in (dict(b=-1), dict(t=-1), dict(t=1 << 31), dict(hq=0), dict(hkv=0), dict(hq=9), dict(decay=math.nan),
                dict(decay=math.inf), dict(s=NULL), dict(out=NULL), dict(s=P_MIS), dict(lens=P_MIS), dict(m=P_MIS),
                dict(out=P_MIS), dict(b=1 << 30)):
        assert mass(**bad) == INVALID, bad
    assert mass(b=(1 << 27) + 1, hq=1, hkv=1) == INVALID
    assert mass(hq=1025, hkv=1) == UNSUPPORTED and mass(hq=1025, hkv=1, t=0) == UNSUPPORTED
    assert mass(b=0, s=NULL, out=NULL) == OK
    assert mass(t=0, s=NULL, out=NULL) == OK


def test_evict_refusals():
    lib = B.lib()
    names = ("m", "kc", "kn", "vc", "vn", "idx", "ol", "om", "okc", "okn", "ovc", "ovn")

    def evict(b=2, hkv=2, cap=16, lens=P, keep=8, sink=2, recent=3, d=128, kb=4, vb=2, **kw):
        p = {n: kw.get(n, P) for n in names}
        return lib.rrq_evict(p["m"], b, hkv, cap, lens, keep, sink, recent, d, kb, vb, p["kc"], p["kn"], p["vc"],
                             p["vn"], p["idx"], p["ol"], p["om"], p["okc"], p["okn"], p["ovc"], p["ovn"], None)

    for bad in (dict(b=-1), dict(hkv=0), dict(cap=-1), dict(cap=1 << 31), dict(keep=0), dict(keep=1 << 31),
                dict(sink=-1), dict(recent=-1), dict(sink=9), dict(recent=9), dict(sink=5, recent=4), dict(d=100),
                dict(kb=0), dict(vb=5), dict(lens=P_MIS), dict(b=1 << 31)):
        assert evict(**bad) == INVALID, bad
    for n in names:
        assert evict(**{n: P_MIS}) == INVALID, n
        if n != "om":
            assert evict(**{n: NULL}) == INVALID, n
    for n in ("kc", "vc", "okc", "ovc"):
        assert evict(**{n: ctypes.c_void_p(0x10008)}) == INVALID, n
    assert evict(b=0, **{n: NULL for n in names}) == OK


def test_shared_attention_refusals():
    lib = B.lib()
    names = ("q", "pkc", "pkn", "pvc", "pvn", "tkc", "tkn", "tvc", "tvn", "lens", "ws", "out")
    keep = []

    def call(dt=B.RRQ_F16, b=2, hq=8, prefix=100, cap=50, hkv=2, d=128, kb=4, kcb=None, vb=4, scale=1.0, size=1 << 40, **kw):
        p = {n: kw.get(n, P) for n in names}
        return lib.rrq_attention_shared(p["q"], dt, b, hq, p["pkc"], p["pkn"], p["pvc"], p["pvn"], prefix, p["tkc"],
                                        p["tkn"], p["tvc"], p["tvn"], cap, p["lens"], hkv, d, kb, 1, kcb, vb, 2, None,
                                        scale, p["ws"], size, p["out"], None)

    bad_cb = (ctypes.c_float * 16)(*([0.0] * 16))
    keep.append(bad_cb)
    for bad in (dict(dt=7), dict(b=-1), dict(hq=0), dict(hq=9), dict(hkv=0), dict(prefix=-1), dict(cap=-1), dict(d=96),
                dict(kb=0), dict(vb=5), dict(scale=math.inf), dict(scale=math.nan), dict(size=64),
                dict(kcb=ctypes.cast(bad_cb, ctypes.c_void_p)), dict(ws=ctypes.c_void_p(0x10010))):
        assert call(**bad) == INVALID, bad
    for n in names:
        assert call(**{n: NULL}) == INVALID, n
        assert call(**{n: P_MIS}) == INVALID, n
    assert call(dt=B.RRQ_F32) == UNSUPPORTED
    assert call(hq=2 * 129) == UNSUPPORTED
    assert call(prefix=1 << 50) == UNSUPPORTED
    assert call(cap=1 << 50) == UNSUPPORTED
    assert call(b=1 << 40) == UNSUPPORTED
    none = {n: NULL for n in names}
    assert call(b=0, prefix=0, **none) == OK


def test_shared_attention_workspace_sizes():
    """0 for what the call refuses; bounded in prefix and tail_cap once every SM has work."""
    ws = B.rrq_attention_shared_workspace_bytes
    assert ws(0, 8, 2, 128, 10, 10) == 0 and ws(1, 9, 2, 128, 10, 10) == 0 and ws(1, 8, 2, 100, 10, 10) == 0
    assert ws(1, 258, 2, 128, 10, 10) == 0
    # tokens are counted in 32 bits, rounded up to a tile
    most = (1 << 31) - 129
    assert ws(1, 1, 1, 64, most, 0) > 0 and ws(1, 1, 1, 64, most + 1, 0) == 0
    assert ws(3, 1, 1, 64, 0, most // 3) > 0 and ws(3, 1, 1, 64, 0, most // 3 + 1) == 0
    for d in (64, 128, 256, 512):
        rows = 4 * 32
        # a head, the queries, and at least one state (a pair and d floats) per row and part
        assert ws(4, 32, 8, d, 100, 0) >= rows * (d * 2 + d * 4 + 8)
        assert ws(4, 32, 8, d, 0, 0) > 0
        big = ws(4, 32, 8, d, 1 << 20, 0)
        assert ws(4, 32, 8, d, 1 << 21, 0) <= 1.2 * big
