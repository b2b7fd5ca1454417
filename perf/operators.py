"""Workloads of the serving operators around the quantised cache, with their plain forms.

Four calls of a serving loop that keeps its K/V cache as b-bit rotated codes plus norms:

* ``rrq_rope``             rotary positions of queries and keys before they are encoded;
* ``rrq_attention_shared`` attention of a batch of queries over one shared quantised prefix
                           and a private quantised tail per sequence;
* ``rrq_attention_mass``   softmax weights of a step's scores added to a running sum per
                           cached token;
* ``rrq_evict``            the tokens with the largest sums kept, their rows moved together.

With ``own`` false, ``run`` computes the same results from elementary torch operations.
"""

import functools
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
K_SEED, V_SEED = 42, 43


# ------------------------------------------------------------------------------- cases
def _attention(name, batch, hq, hkv, d, kb, vb, prefix, cap, dtype):
    return {"name": name, "op": "attention", "batch": batch, "hq": hq, "hkv": hkv, "d": d, "k_bits": kb,
            "v_bits": vb, "prefix": prefix, "cap": cap, "dtype": dtype}


def _mass(name, batch, hq, hkv, t_len, decay):
    return {"name": name, "op": "mass", "batch": batch, "hq": hq, "hkv": hkv, "t_len": t_len, "decay": decay}


def _evict(name, batch, hkv, d, kb, vb, cap, keep, sink, recent):
    return {"name": name, "op": "evict", "batch": batch, "hkv": hkv, "d": d, "k_bits": kb, "v_bits": vb,
            "cap": cap, "keep": keep, "sink": sink, "recent": recent}


def _rope(name, tokens, heads, d, rot, interleaved, scaling, far, inverse, dtype):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "d": d, "rot": rot,
            "interleaved": interleaved, "scaling": scaling, "far": far, "inverse": inverse, "dtype": dtype}


def listed():
    return [
        # one user, a short instruction as the prefix, a few private tokens: latency
        _attention("shared-one", 1, 8, 2, 64, 2, 2, 500, 17, "f16"),
        # a chat server: one system prompt for 16 conversations of a few hundred tokens
        _attention("shared-chat", 16, 32, 8, 128, 4, 4, 4096, 512, "bf16"),
        # many questions on one long document, 4-bit cache of the score workload's heads
        _attention("shared-document", 64, 32, 8, 128, 4, 4, 32768, 1024, "bf16"),
        # a wide head with odd lengths and mixed bit widths
        _attention("shared-wide", 7, 16, 4, 256, 3, 4, 2049, 301, "f16"),
        # private caches only, nothing shared: a batch in the middle of its answers
        _attention("tails-only", 33, 16, 4, 128, 4, 2, 0, 1500, "bf16"),
        # one decode step over the score workload's cache
        _mass("mass-long", 1, 32, 8, 131072, 1.0),
        # a ragged batch of conversations, older steps fading
        _mass("mass-batch", 16, 16, 4, 2047, 0.97),
        # a quarter of a long cache kept
        _evict("evict-long", 1, 8, 128, 4, 4, 131072, 32768, 4, 1024),
        # a ragged batch cut back to a short budget, 2-bit keys and 3-bit values
        _evict("evict-batch", 24, 4, 64, 2, 3, 2000, 511, 3, 100),
        # the query heads of one decode step, far into a scaled context
        _rope("rope-step", 1, 32, 128, 128, False, "yarn", 1000000, False, "bf16"),
        # the keys of a whole prompt
        _rope("rope-prompt", 32768, 8, 128, 128, False, "none", 0, False, "f16"),
        # gradient of an interleaved, partial rotation in fp32
        _rope("rope-gradient", 5001, 12, 128, 48, True, "linear", 100000, True, "f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "mass", "evict", "rope"])
    if op == "attention":
        while True:
            hkv = rng.choice([1, 2, 4, 8])
            c = _attention("", _log(rng, 1, 64), hkv * rng.choice([1, 2, 4, 8]), hkv, rng.choice([64, 128, 128, 256]),
                           rng.randint(1, 4), rng.randint(1, 4), rng.choice([0, 1, 1, 1]) * _log(rng, 1, 32768),
                           _log(rng, 1, 1500), rng.choice(["f16", "bf16"]))
            w = work(c)
            if w["bytes"] <= 2.0e8 and w["flops"] <= 3.4e10 and c["batch"] * c["cap"] * hkv * c["d"] <= 7e7:
                break
    elif op == "mass":
        while True:
            hkv = rng.choice([1, 2, 4, 8])
            c = _mass("", _log(rng, 1, 32), hkv * rng.choice([1, 2, 4, 8]), hkv, _log(rng, 1, 131072),
                      rng.choice([1.0, 0.9, 0.97]))
            if c["batch"] * c["hq"] * c["t_len"] <= 32 * 131072:
                break
    elif op == "evict":
        while True:
            cap = _log(rng, 2, 131072)
            keep = max(1, int(cap * rng.uniform(0.1, 0.9)))
            c = _evict("", _log(rng, 1, 32), rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.randint(1, 4),
                       rng.randint(1, 4), cap, keep, min(keep // 4, 4), keep // rng.choice([2, 4, 8]))
            if c["batch"] * c["hkv"] * cap * c["d"] <= 8 * 131072 * 128:
                break
    else:
        d = rng.choice([64, 128, 256, 512])
        while True:
            c = _rope("", _log(rng, 1, 32768), rng.randint(1, 32), d, 2 * rng.randint(1, d // 2),
                      rng.random() < 0.5, rng.choice(["none", "linear", "ntk", "yarn"]), rng.choice([0, 100000, 1000000]),
                      rng.random() < 0.3, rng.choice(["f32", "f16", "bf16"]))
            if c["tokens"] * c["heads"] * d * (2 if c["dtype"] == "f32" else 1) <= 32768 * 8 * 128:
                break
    del c["name"]
    return c


# ------------------------------------------------------- the format: codebook, signs, codes
@functools.lru_cache(maxsize=None)
def _levels(bits):
    """Lloyd-Max levels of N(0,1), ascending, by alternating midpoints and cell centroids."""
    half = 1 << (bits - 1)
    c = [3.0 * (k + 0.5) / half for k in range(half)]
    for _ in range(20000):
        edge = [0.0] + [(a + b) / 2 for a, b in zip(c, c[1:])] + [math.inf]
        pdf = [0.0 if math.isinf(e) else math.exp(-e * e / 2) / math.sqrt(2 * math.pi) for e in edge]
        tail = [0.0 if math.isinf(e) else math.erfc(e / math.sqrt(2)) / 2 for e in edge]
        new = [(pdf[k] - pdf[k + 1]) / (tail[k] - tail[k + 1]) for k in range(half)]
        moved = max(abs(a - b) for a, b in zip(new, c))
        c = new
        if moved < 1e-15:
            break
    return tuple([-x for x in reversed(c)] + c)


def _signs(seed, d):
    """-1 where bit 63 of SplitMix64 output i of a generator seeded with `seed` is set, else +1."""
    with np.errstate(over="ignore"):
        z = np.uint64(seed) + np.arange(1, d + 1, dtype=np.uint64) * np.uint64(0x9E3779B97F4A7C15)
        z = (z ^ (z >> np.uint64(30))) * np.uint64(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> np.uint64(27))) * np.uint64(0x94D049BB133111EB)
        z = z ^ (z >> np.uint64(31))
    return np.where(z >> np.uint64(63), -1.0, 1.0)


def _rotation(seed, d):
    """The rotation as a dense matrix in 64 bits: row i, column j: (-1)^popcount(i & j) s_j / sqrt(d)."""
    h = np.ones((1, 1))
    while h.shape[0] < d:
        h = np.block([[h, h], [h, -h]])
    return h * _signs(seed, d)[None, :] / math.sqrt(d)


def _cache(gen, rows, d, bits):
    """Codes and norms as the encoder leaves them: nearest levels of N(0,1) coordinates, log-normal norms."""
    edge = torch.tensor([(a + b) / 2 for a, b in zip(_levels(bits), _levels(bits)[1:])], device="cuda")
    packed = torch.empty(rows, d * bits // 8, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // d)
    shift = torch.arange(8, device="cuda") * bits
    for r in range(0, rows, step):
        u = torch.randn(min(step, rows - r), d, device="cuda", generator=gen)
        codes = torch.bucketize(u, edge).view(u.shape[0], d // 8, 8)
        word = (codes << shift).sum(-1)
        packed[r:r + step] = torch.stack([(word >> (8 * k)) & 255 for k in range(bits)], -1).view(u.shape[0], -1)
    norms = torch.randn(rows, device="cuda", generator=gen).mul_(0.5).exp_().mul_(math.sqrt(d))
    return packed, norms


def _unpack(packed, norms, d, bits, levels):
    """Rotated-domain values [..., d] in fp32, levels times norm / sqrt(d)."""
    by = packed.view(*norms.shape, d // 8, bits).to(torch.int32)
    word = by[..., 0]
    for k in range(1, bits):
        word = word | (by[..., k] << (8 * k))
    code = (word.unsqueeze(-1) >> (torch.arange(8, device="cuda", dtype=torch.int32) * bits)) & ((1 << bits) - 1)
    return levels[code].view(*norms.shape, d) * (norms * (1.0 / math.sqrt(d))).unsqueeze(-1)


def _frequencies(rot, scaling):
    """Radians per position of the rot/2 pairs and the factor on cos and sin, in 64 bits."""
    base, stretch, original = 10000.0, 8.0, 8192.0
    i = np.arange(0, rot, 2, dtype=np.float64)
    freq = base ** (-i / rot)
    if scaling == "linear":
        return freq / stretch, 1.0
    if scaling == "ntk" and rot > 2:
        return (base * stretch ** (rot / (rot - 2))) ** (-i / rot), 1.0
    if scaling == "yarn":
        def turn(times):
            return rot * math.log(original / (times * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), rot - 1)
        ramp = np.clip((i / 2 - lo) / max(hi - lo, 0.001), 0.0, 1.0)
        return freq * (1 - ramp) + freq / stretch * ramp, 0.1 * math.log(stretch) + 1.0
    return freq, 1.0


# ------------------------------------------------------------------------------ prepare
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "attention":
        b, hq, hkv, d, cap, prefix = (case[k] for k in ("batch", "hq", "hkv", "d", "cap", "prefix"))
        s["q"] = torch.randn(b, hq, d, device="cuda", generator=gen).to(DTYPES[case["dtype"]])
        kv = [_cache(gen, n * hkv, d, case[w]) for n in (prefix, b * cap) for w in ("k_bits", "v_bits")]
        s["prefix_kv"] = [t.view(prefix, hkv, *t.shape[1:]) for c in kv[:2] for t in c]
        s["tail_kv"] = [t.view(b, cap, hkv, *t.shape[1:]) for c in kv[2:] for t in c]
        # conversations of every length up to the capacity, an empty one among them
        lens = torch.randint(0, cap + 1, (b,), device="cuda", generator=gen)
        lens[0] = cap
        if b > 2:
            lens[b // 2] = 0
        s["lens"] = lens.to(torch.int32)
        s["levels"] = [torch.tensor(_levels(case[w]), device="cuda", dtype=torch.float32) for w in ("k_bits", "v_bits")]
        s["rotation"] = [torch.from_numpy(_rotation(x, d)).to("cuda", torch.float32) for x in (K_SEED, V_SEED)]
    elif case["op"] == "mass":
        b, hq, hkv, t = case["batch"], case["hq"], case["hkv"], case["t_len"]
        s["scores"] = torch.randn(b, hq, t, device="cuda", generator=gen) * 2
        s["scores"][:, :, 0] += 6  # the first token draws much of the weight
        # a few tokens are masked for a head
        s["scores"].masked_fill_(torch.rand(b, hq, t, device="cuda", generator=gen) < 0.01, -math.inf)
        s["mass"] = torch.rand(b, hkv, t, device="cuda", generator=gen).square_()
        lens = torch.randint(0, t + 1, (b,), device="cuda", generator=gen)
        lens[0] = t
        s["lens"] = lens.to(torch.int32)
    elif case["op"] == "evict":
        b, hkv, cap, d = case["batch"], case["hkv"], case["cap"], case["d"]
        # sums over some thousand steps: a heavy tail, and many tokens never looked at (equal sums)
        mass = torch.randn(b, hkv, cap, device="cuda", generator=gen).mul_(2.0).exp_()
        s["mass"] = torch.where(mass < 0.5, torch.zeros_like(mass), (mass * 1024).round_() / 1024)
        kv = [_cache(gen, b * cap * hkv, d, case[w]) for w in ("k_bits", "v_bits")]
        s["kv"] = [t.view(b, cap, hkv, *t.shape[1:]) for c in kv for t in c]
        lens = torch.randint(0, cap + 1, (b,), device="cuda", generator=gen)
        lens[0] = cap
        s["lens"] = lens.to(torch.int32)
        # the new cache: its rows behind the last kept token stay as they are
        s["out"] = [torch.zeros(b, case["keep"], *t.shape[2:], dtype=t.dtype, device="cuda") for t in s["kv"]]
        s["out_mass"] = torch.zeros(b, hkv, case["keep"], device="cuda")
        s["index"] = torch.full((b, hkv, case["keep"]), -1, dtype=torch.int32, device="cuda")
    else:
        n, heads, d = case["tokens"], case["heads"], case["d"]
        s["x"] = torch.randn(n, heads, d, device="cuda", generator=gen).to(DTYPES[case["dtype"]])
        gaps = torch.randint(1, 3, (n,), device="cuda", generator=gen)  # an evicted cache has gaps
        s["positions"] = case["far"] + torch.cumsum(gaps, 0) - 1
        s["freqs"], s["factor"] = _frequencies(case["rot"], case["scaling"])
    return s


# ---------------------------------------------------------------------------------- run
def _plain_attention(s):
    b, hq, hkv, d, cap = s["batch"], s["hq"], s["hkv"], s["d"], s["cap"]
    scale = 1.0 / math.sqrt(d)
    q = (s["q"].float() @ s["rotation"][0].T).view(b, hkv, hq // hkv, d)
    pk = _unpack(s["prefix_kv"][0], s["prefix_kv"][1], d, s["k_bits"], s["levels"][0])  # [T, hkv, d]
    tk = _unpack(s["tail_kv"][0], s["tail_kv"][1], d, s["k_bits"], s["levels"][0])      # [B, cap, hkv, d]
    sp = torch.einsum("bgjd,tgd->bgjt", q, pk) * scale
    st = torch.einsum("bgjd,btgd->bgjt", q, tk) * scale
    gone = torch.arange(cap, device="cuda")[None] >= s["lens"][:, None]
    st = st.masked_fill(gone[:, None, None], -math.inf)
    x = torch.cat([sp, st], -1)
    m = x.max(-1, keepdim=True).values
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    pv = _unpack(s["prefix_kv"][2], s["prefix_kv"][3], d, s["v_bits"], s["levels"][1])
    tv = _unpack(s["tail_kv"][2], s["tail_kv"][3], d, s["v_bits"], s["levels"][1])
    y = torch.einsum("bgjt,tgd->bgjd", p[..., :s["prefix"]], pv) + torch.einsum("bgjt,btgd->bgjd", p[..., s["prefix"]:], tv)
    y = torch.where(total > 0, y / total, 0.0)
    return (y.reshape(b, hq, d) @ s["rotation"][1]).to(s["q"].dtype)


def _plain_mass(s):
    b, hq, hkv, t = s["batch"], s["hq"], s["hkv"], s["t_len"]
    live = torch.arange(t, device="cuda")[None, None] < s["lens"][:, None, None]
    x = s["scores"].masked_fill(~live, -math.inf)
    m = x.max(-1, keepdim=True).values
    p = torch.exp(x - torch.where(m == -math.inf, 0.0, m))
    total = p.sum(-1, keepdim=True)
    p = torch.where(total > 0, p / total, 0.0)
    return torch.where(live, s["decay"] * s["mass"] + p.view(b, hkv, hq // hkv, t).sum(2), s["mass"])


def _plain_evict(s):
    b, hkv, cap, keep = s["batch"], s["hkv"], s["cap"], s["keep"]
    t = torch.arange(cap, device="cuda")[None, None]
    lens = s["lens"][:, None, None].long()
    rank = torch.where((t < s["sink"]) | (t >= lens - s["recent"]), math.inf, s["mass"])
    rank = torch.where(t < lens, rank, -math.inf)
    first = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = torch.clamp(lens, max=keep)
    slot = torch.arange(keep, device="cuda")[None, None]
    first = torch.sort(torch.where(slot < new, first, cap), dim=-1).values  # ascending, what is not kept last
    live = slot < new
    index = torch.where(live, first, -1).to(torch.int32)
    at = torch.where(live, first, 0)
    out = []
    for t_, o in zip(s["kv"], s["out"]):
        if t_.dim() == 4:
            moved = torch.gather(t_, 1, at.transpose(1, 2).unsqueeze(-1).expand(b, keep, hkv, t_.shape[-1]))
            out.append(torch.where(live.transpose(1, 2).unsqueeze(-1), moved, o))
        else:
            out.append(torch.where(live.transpose(1, 2), torch.gather(t_, 1, at.transpose(1, 2)), o))
    mass = torch.where(live, torch.gather(s["mass"], 2, at), s["out_mass"])
    return index, new.view(b).to(torch.int32), mass, *out


def _plain_rope(s):
    rot, x = s["rot"], s["x"].float()
    angle = s["positions"].double()[:, None, None] * torch.from_numpy(s["freqs"]).to("cuda")
    c, sn = (torch.cos(angle) * s["factor"]).float(), (torch.sin(angle) * s["factor"]).float()
    if s["inverse"]:
        sn = -sn
    a, e = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, v = a * c - e * sn, a * sn + e * c
    turned = torch.stack([u, v], -1).flatten(-2) if s["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1).to(s["x"].dtype)


def run(state):
    s = state
    if own:
        from random_rotation_kv_b200 import binding as B
        if s["op"] == "attention":
            return B.rrq_attention_shared(s["q"], *s["prefix_kv"], *s["tail_kv"], s["lens"], s["hkv"], s["d"], K_SEED, V_SEED,
                                          k_bits=s["k_bits"], v_bits=s["v_bits"], scale=1.0 / math.sqrt(s["d"]))
        if s["op"] == "mass":
            return B.rrq_attention_mass(s["scores"], s["hkv"], mass=s["mass"], lens=s["lens"], decay=s["decay"])
        if s["op"] == "evict":
            return B.rrq_evict(s["mass"], s["lens"], s["keep"], *s["kv"], sink=s["sink"], recent=s["recent"],
                               index=s["index"], out_mass=s["out_mass"], out=s["out"])
        return B.rrq_rope(s["x"], s["positions"], s["freqs"], interleaved=s["interleaved"], factor=s["factor"],
                          inverse=s["inverse"])
    return {"attention": _plain_attention, "mass": _plain_mass, "evict": _plain_evict, "rope": _plain_rope}[s["op"]](s)


# --------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "attention":
        row = c["d"] * (c["k_bits"] + c["v_bits"]) / 8 + 8
        tails = c["batch"] * c["cap"] / 2  # lengths are spread evenly over the capacity
        pairs = c["hq"] * (c["batch"] * c["prefix"] + tails)
        return {"bytes": (c["prefix"] + tails) * c["hkv"] * row + c["batch"] * c["hq"] * c["d"] * 4, "flops": 4.0 * c["d"] * pairs}
    if c["op"] == "mass":
        share = 1.0 if c["batch"] == 1 else 0.5 + 0.5 / c["batch"]
        tokens = c["batch"] * c["t_len"] * share
        # the sums behind a sequence's end are handed on as they are
        return {"bytes": tokens * c["hq"] * 4 + 8.0 * c["batch"] * c["t_len"] * c["hkv"], "flops": 6.0 * tokens * c["hq"]}
    if c["op"] == "evict":
        share = 1.0 if c["batch"] == 1 else 0.5 + 0.5 / c["batch"]
        kept = c["batch"] * c["hkv"] * c["keep"] * min(1.0, share * c["cap"] / c["keep"])
        row = c["d"] * (c["k_bits"] + c["v_bits"]) / 8 + 8
        return {"bytes": c["batch"] * c["hkv"] * c["cap"] * share * 4 + kept * (2 * row + 8), "flops": 0.0}
    values = c["tokens"] * c["heads"] * c["d"]
    return {"bytes": values * 2 * (4 if c["dtype"] == "f32" else 2) + 8.0 * c["tokens"], "flops": 3.0 * c["tokens"] * c["heads"] * c["rot"]}


# -------------------------------------------------------------------------------- exact
def _vectors64(packed, norms, d, bits, seed):
    """The stored vectors themselves in 64 bits: [rows, d], rotated back."""
    bit = (packed.view(-1, d * bits // 8, 1) >> torch.arange(8, device="cuda", dtype=torch.uint8)) & 1
    bit = bit.view(-1, d, bits).long()
    code = (bit << torch.arange(bits, device="cuda")).sum(-1)
    lev = torch.tensor(np.float32(_levels(bits)).astype(np.float64), device="cuda")
    y = lev[code] * (norms.reshape(-1, 1).double() / math.sqrt(d))
    return y @ torch.from_numpy(_rotation(seed, d)).to("cuda")


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        b, hq, hkv, d = case["batch"], case["hq"], case["hkv"], case["d"]
        out = torch.zeros(b, hq, d, dtype=torch.float64, device="cuda")
        lens = s["lens"].tolist()
        group = hq // hkv
        for g in range(hkv):
            kc, kn, vc, vn = (t[:, g].contiguous() for t in s["prefix_kv"])
            pk, pv = _vectors64(kc, kn, d, case["k_bits"], K_SEED), _vectors64(vc, vn, d, case["v_bits"], V_SEED)
            for i in range(b):
                kc, kn, vc, vn = (t[i, :lens[i], g].contiguous() for t in s["tail_kv"])
                k = torch.cat([pk, _vectors64(kc, kn, d, case["k_bits"], K_SEED)])
                v = torch.cat([pv, _vectors64(vc, vn, d, case["v_bits"], V_SEED)])
                if k.shape[0]:
                    x = s["q"][i, g * group:(g + 1) * group].double() @ k.T / math.sqrt(d)
                    out[i, g * group:(g + 1) * group] = torch.softmax(x, -1) @ v
        return out
    if case["op"] == "mass":
        out = s["mass"].double()
        group = case["hq"] // case["hkv"]
        for i, n in enumerate(s["lens"].tolist()):
            if n:
                p = torch.softmax(s["scores"][i, :, :n].double(), -1)
                p = torch.where(torch.isnan(p), 0.0, p)  # every token of the head masked
                out[i, :, :n] = case["decay"] * out[i, :, :n] + p.view(case["hkv"], group, n).sum(1)
        return out
    if case["op"] == "evict":
        return None  # whole numbers, bytes and moved values: equal to the plain form's
    x = s["x"].double().cpu().numpy()
    rot, half = case["rot"], case["rot"] // 2
    turn = np.exp(1j * s["positions"].double().cpu().numpy()[:, None, None] * s["freqs"]) * s["factor"]
    turn = np.conj(turn) if case["inverse"] else turn
    at = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, half), slice(half, rot))
    z = (x[..., at[0]] + 1j * x[..., at[1]]) * turn
    x[..., at[0]], x[..., at[1]] = z.real, z.imag
    return x
