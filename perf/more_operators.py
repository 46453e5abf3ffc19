"""The operators of a prompt, as they are measured: listed cases, drawn cases
of the same ranges, their inputs, the plain form of each operator in elementary
torch operations (32 bits, rounded once at the end) and its definition in 64
bits.

* rope: RMS norm of every query and key head (optional) and rotary positions
  with several axes (time, height, width): pair i of a head turns by the angle
  of the token's position on axis axes[i].
* attend: softmax attention of packed prompts of different lengths over their
  own 16-bit keys and values: grouped heads, causal or full, a sliding window,
  more keys than queries (the chunk of a longer prompt), optionally joined with
  the result of attention over other keys (a cached prefix).
"""

import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    r = dict(op="rope", D=128, sections="16+24+24", turns=False, interleaved=False, norm=True, dtype="bf16")
    t = dict(op="attend", D=128, dtype="bf16", ragged=False, causal=True, window=0, more=0, prefix=False)
    return [
        # the token after a prompt with images: latency is everything
        dict(r, name="rope_1_token", T=1, Hq=64, Hkv=8),
        # a prompt chunk of a small model: fp32 projections, narrow heads, neighbouring pairs, the axes taking turns
        dict(r, name="rope_chunk_narrow", T=1031, Hq=20, Hkv=4, D=64, sections="12+10+10", turns=True,
             interleaved=True, dtype="f32"),
        # the patches of images: two axes on half of each head, no norm
        dict(r, name="rope_patches", T=4099, Hq=16, Hkv=16, sections="16+16", norm=False, dtype="f16"),
        # a long prompt of text and pictures
        dict(r, name="rope_prompt", T=8192, Hq=64, Hkv=8),
        # one short question: the smallest call
        dict(t, name="attend_1_short", B=1, nq=37, Hq=32, Hkv=8),
        # a batch of short prompts, narrow heads in odd groups of three
        dict(t, name="attend_batch_narrow", B=13, nq=517, Hq=24, Hkv=8, D=64, ragged=True, dtype="f16"),
        # prompts of several users in one call
        dict(t, name="attend_ragged_prompts", B=9, nq=2500, Hq=32, Hkv=8, ragged=True),
        # a long document
        dict(t, name="attend_long", B=1, nq=8192, Hq=64, Hkv=8),
        # long documents under a sliding window, sixteen query heads on a KV head
        dict(t, name="attend_window", B=2, nq=8192, Hq=64, Hkv=4, window=1024),
        # a chunk of a longer prompt, whose earlier keys are still there in 16 bits
        dict(t, name="attend_chunk", B=1, nq=2048, Hq=64, Hkv=8, more=6144),
        # new turns of conversations whose earlier tokens lie in the cache: joined with the attention over those
        dict(t, name="attend_prefix", B=5, nq=700, Hq=40, Hkv=8, ragged=True, prefix=True),
        # the patches of images see each other, a KV head for each query head
        dict(t, name="attend_images", B=16, nq=1024, Hq=16, Hkv=16, D=64, ragged=True, causal=False, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _split(rng, pairs, axes):
    """Pairs shared out among the axes, each with one at least."""
    cuts = sorted(rng.sample(range(1, pairs), axes - 1))
    return "+".join(str(b - a) for a, b in zip([0] + cuts, cuts + [pairs]))


def _sections(case):
    """The pairs of each axis."""
    return [int(n) for n in case["sections"].split("+")]


def draw(rng):
    Hkv = rng.randint(1, 8)
    D = rng.choice((64, 128))
    if rng.random() < 0.4:
        rot = rng.choice((D, D, D // 2, D - 16))
        return dict(op="rope", T=_log(rng, 1, 8192), Hq=Hkv * rng.randint(1, 8), Hkv=Hkv, D=D,
                    sections=_split(rng, rot // 2, rng.choice((2, 3, 3))), turns=rng.random() < 0.5,
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.6,
                    dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
    G = rng.choice((1, 1, 2, 3, 4, 5, 7, 8, 8, 12, 16))
    causal = rng.random() < 0.8
    B, nq = _log(rng, 1, 32), _log(rng, 1, 8192)
    more = rng.choice((0, 0, 0, _log(rng, 1, 8192)))
    most = 64 * 8192 * 8192                              # no dearer than the largest listed case
    while B > 1 and B * nq * (nq + 2 * more) * Hkv * G * (1 if causal else 2) > most:
        B = (B + 1) // 2
    while nq * (nq + 2 * more) * Hkv * G * (1 if causal else 2) > most:
        nq, more = (nq + 1) // 2, more // 2
    return dict(op="attend", B=B, nq=nq, Hq=Hkv * G, Hkv=Hkv, D=D, dtype=rng.choice(("bf16", "bf16", "f16")),
                ragged=B > 1 and rng.random() < 0.8, causal=causal, more=more,
                window=rng.choice((0, 0, _log(rng, 16, 2048))) if causal else 0, prefix=rng.random() < 0.25)


def _lengths(case):
    """(queries, keys) of every sequence: part of the case."""
    r = random.Random("%(B)d %(nq)d %(more)d %(Hq)d" % case)
    q, k = [], []
    for b in range(case["B"]):
        m = case["nq"]
        if case["ragged"] and b:
            m = r.choice((1, r.randint(0, m), r.randint((m + 1) // 2, m), r.randint((m + 1) // 2, m)))
        q.append(m)
        k.append(m + (r.randint(0, case["more"]) if case["ragged"] and b else case["more"]))
    return q, k


def work(case):
    D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        rot, axes = 2 * sum(_sections(case)), len(_sections(case))
        per = (Hq + Hkv) * D * 2 * size + 4 * rot + 4 * axes
        return {"bytes": case["T"] * per, "flops": case["T"] * (Hq + Hkv) * (3 * rot + (4 * D if case["norm"] else 0))}
    bytes_, flops, w = 0.0, 0.0, case["window"]
    for m, n in zip(*_lengths(case)):
        bytes_ += (2 * m * Hq + 2 * n * Hkv) * D * size + 4 * m * Hq + 8
        if case["prefix"]:
            bytes_ += m * Hq * (D * size + 4)
        if not case["causal"]:
            pairs = m * n
        elif not w:
            pairs = m * (n - m) + m * (m + 1) // 2
        else:
            grow = max(0, min(m, w - (n - m)))           # queries that see fewer than w keys, or just as many
            pairs = grow * (n - m) + grow * (grow + 1) // 2 + (m - grow) * w
        flops += 4.0 * pairs * Hq * D
    return {"bytes": bytes_, "flops": flops}


# ------------------------------------------------------------------ inputs

def _heavy(shape, g, spread):
    """Normal values whose last axis has a few louder channels."""
    x = torch.randn(shape, generator=g, device="cuda")
    loud = torch.rand(shape[-1], generator=g, device="cuda") < 0.04
    return x * torch.where(loud, 3.0 * spread, spread)


def _places(T, axes, g):
    """Positions [axes, T]: stretches of text (the same on every axis) and of pictures (rows and columns of patches)."""
    dev = torch.device("cuda")
    t = torch.arange(T, device=dev)
    first = int(torch.randint(0, 4096, (1,), generator=g, device=dev))
    pos = (first + t).repeat(axes, 1)
    wide = 16 + int(torch.randint(0, 48, (1,), generator=g, device=dev))
    picture = (t // 512) % 2 == 1
    inside = t % 512
    pos[-1] = torch.where(picture, pos[-1] - inside + inside % wide, pos[-1])
    pos[-2] = torch.where(picture, pos[-2] - inside + inside // wide, pos[-2])
    if axes > 2:
        pos[0] = torch.where(picture, pos[0] - inside, pos[0])
    return pos.to(torch.int32).contiguous()


def _axes(case):
    """The axis of each pair: in blocks, or the axes taking turns while they have pairs left."""
    left = _sections(case)
    if not case["turns"]:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    out = []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return tuple(out)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 7919 + 29)
    dev = torch.device("cuda")
    D, Hq, Hkv, dt = case["D"], case["Hq"], case["Hkv"], _TYPES[case["dtype"]]
    st = dict(case=case, D=D, Hq=Hq, Hkv=Hkv, dtype=dt)
    if case["op"] == "rope":
        T, rot = case["T"], 2 * sum(_sections(case))
        # one fused projection: q and k are views of its rows
        qkv = _heavy((T, Hq + 2 * Hkv, D), g, 1.0).to(dt)
        st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        n_pos = 16384
        freq = 10000.0 ** (-torch.arange(0, rot, 2, device=dev, dtype=torch.float64) / rot)
        angle = torch.arange(n_pos, device=dev, dtype=torch.float64)[:, None] * freq
        st["cos"], st["sin"] = angle.cos().float().contiguous(), angle.sin().float().contiguous()
        st["positions"], st["axes"] = _places(T, len(_sections(case)), g), _axes(case)
        st["q_weight"] = st["k_weight"] = None
        if case["norm"]:
            st["q_weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
            st["k_weight"] = 1.0 + 0.2 * torch.randn(D, generator=g, device=dev)
        st["eps"], st["interleaved"] = 1e-6, case["interleaved"]
        return st
    nq, nk = _lengths(case)
    T, Tk = sum(nq), sum(nk)
    if T == Tk:                                          # views of one fused projection
        qkv = _heavy((T, Hq + 2 * Hkv, D), g, 1.0)
        qkv[:, Hq + Hkv:] *= 0.5
        qkv = qkv.to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        st["q"] = _heavy((T, Hq, D), g, 1.0).to(dt)
        st["k"], st["v"] = _heavy((Tk, Hkv, D), g, 1.0).to(dt), _heavy((Tk, Hkv, D), g, 0.5).to(dt)
    cu_q, cu_k = [0], [0]
    for m, n in zip(nq, nk):
        cu_q.append(cu_q[-1] + m)
        cu_k.append(cu_k[-1] + n)
    st["nq"], st["nk"], st["max_q"], st["max_k"] = nq, nk, max(nq), max(nk)
    st["cu_q"] = torch.tensor(cu_q, dtype=torch.int32, device=dev)
    st["cu_k"] = torch.tensor(cu_k, dtype=torch.int32, device=dev) if T != Tk else None
    st["scale"], st["causal"], st["window"] = D ** -0.5, case["causal"], case["window"]
    st["prefix"] = None
    if case["prefix"]:
        # every third sequence is new: nothing of it is in the cache
        z = 5.0 + 2.0 * torch.rand(T, Hq, generator=g, device=dev)
        o = _heavy((T, Hq, D), g, 0.1)
        for b in range(0, len(nq), 3):
            z[cu_q[b]:cu_q[b + 1]] = -math.inf
            o[cu_q[b]:cu_q[b + 1]] = 0.0
        st["prefix"] = o.to(dt), z
    st["out"] = torch.empty(T, Hq, D, dtype=dt, device=dev)
    st["lse"] = torch.empty(T, Hq, dtype=torch.float32, device=dev)
    if own:
        import nvfp4_router_gate_gb300 as R
        st["attention"] = R.PromptAttention(Hq, Hkv, D)
    return st


# ------------------------------------------------------------------- calls

def run(st):
    if own:
        if st["case"]["op"] == "rope":
            import nvfp4_router_gate_gb300 as R
            q, k = R.prompt_rope(st["q"], st["k"], st["positions"], st["cos"], st["sin"], axes=st["axes"],
                                 q_weight=st["q_weight"], k_weight=st["k_weight"], eps=st["eps"],
                                 interleaved=st["interleaved"])
            return {"q": q, "k": k}
        out, lse = st["attention"](st["q"], st["k"], st["v"], cu_q=st["cu_q"], max_q=st["max_q"], cu_k=st["cu_k"],
                                   max_k=st["max_k"], scale=st["scale"], causal=st["causal"], window=st["window"],
                                   prefix=st["prefix"], out=st["out"], lse=st["lse"])
        return {"out": out, "lse": lse}
    return _rope(st) if st["case"]["op"] == "rope" else _attend(st)


def _rope(st):
    rot = 2 * len(st["axes"])
    place = st["positions"][list(st["axes"])].long()                                   # [rot / 2, T]
    pair = torch.arange(rot // 2, device=place.device)[:, None]
    c, s = st["cos"][place, pair].t()[:, None], st["sin"][place, pair].t()[:, None]     # [T, 1, rot / 2]

    def turn(x, weight):
        x = x.float()
        if weight is not None:
            x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + st["eps"])) * weight
        t = x[..., :rot]
        a, b = (t[..., 0::2], t[..., 1::2]) if st["interleaved"] else (t[..., :rot // 2], t[..., rot // 2:])
        p, r = a * c - b * s, b * c + a * s
        t = torch.stack((p, r), -1).flatten(-2) if st["interleaved"] else torch.cat((p, r), -1)
        return torch.cat((t, x[..., rot:]), -1).to(st["dtype"])

    return {"q": turn(st["q"], st["q_weight"]), "k": turn(st["k"], st["k_weight"])}


def _attend(st):
    D, Hq, Hkv = st["D"], st["Hq"], st["Hkv"]
    G, w = Hq // Hkv, st["window"]
    out, lse = torch.empty_like(st["out"]), torch.empty_like(st["lse"])
    q0 = k0 = 0
    for m, n in zip(st["nq"], st["nk"]):
        if m == 0:
            k0 += n
            continue
        k = st["k"][k0:k0 + n].float().transpose(0, 1)                                  # [Hkv, n, D]
        v = st["v"][k0:k0 + n].float().transpose(0, 1)
        key = torch.arange(n, device=k.device)
        step = max(1, (1 << 30) // (Hq * n))                                            # queries at a time
        for i in range(0, m, step):
            j = min(m, i + step)
            q = st["q"][q0 + i:q0 + j].float().unflatten(1, (Hkv, G)).permute(1, 2, 0, 3)   # [Hkv, G, j - i, D]
            s = torch.matmul(q.reshape(Hkv, -1, D), k.transpose(1, 2)).view(Hkv, G, j - i, n) * st["scale"]
            if st["causal"]:
                at = (n - m + torch.arange(i, j, device=k.device))[:, None]
                see = key <= at
                if w:
                    see = see & (key > at - w)
                s = torch.where(see, s, torch.full((), -math.inf, device=s.device))
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(top > -math.inf, top, torch.zeros_like(top)))
            total = p.sum(-1, keepdim=True)
            o = torch.matmul(p.view(Hkv, -1, n), v).view(Hkv, G, j - i, D)
            o = o / torch.where(total > 0, total, torch.ones_like(total))
            z = (torch.log(total) + top).squeeze(-1).permute(2, 0, 1).reshape(j - i, Hq)
            o = o.permute(2, 0, 1, 3).reshape(j - i, Hq, D)
            if st["prefix"] is not None:
                po, pz = st["prefix"][0][q0 + i:q0 + j].float(), st["prefix"][1][q0 + i:q0 + j]
                high = torch.maximum(z, pz)
                a, b = torch.exp(z - high), torch.exp(pz - high)
                o = (o * a[..., None] + po * b[..., None]) / (a + b)[..., None]
                z = high + torch.log(a + b)
            out[q0 + i:q0 + j], lse[q0 + i:q0 + j] = o.to(out.dtype), z
        q0, k0 = q0 + m, k0 + n
    return {"out": out, "lse": lse}


# ------------------------------------------------------- definition, 64 bits

def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    return _rope_64(case, st) if case["op"] == "rope" else _attend_64(case, st)


def _rope_64(case, st):
    res = {}
    pairs = len(st["axes"])
    for name in ("q", "k"):
        x, w = st[name].double(), st[name + "_weight"]
        if w is not None:
            x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + st["eps"]) * w.double()
        y = x.clone()
        for i, axis in enumerate(st["axes"]):
            at = st["positions"][axis].long()
            c, s = st["cos"][at, i].double()[:, None], st["sin"][at, i].double()[:, None]
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + pairs)
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., b] * c + x[..., a] * s
        res[name] = y
    return res


def _attend_64(case, st):
    Hq, Hkv, w = case["Hq"], case["Hkv"], case["window"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for m, n in zip(*_lengths(case)):
        for h in range(Hq):
            k = st["k"][k0:k0 + n, h * Hkv // Hq].double()
            v = st["v"][k0:k0 + n, h * Hkv // Hq].double()
            for i in range(0, m, 1024):
                j = min(m, i + 1024)
                # the keys that any of these queries sees
                hi = n - m + j if case["causal"] else n
                lo = max(0, n - m + i + 1 - w) if w else 0
                x = st["q"][q0 + i:q0 + j, h].double() @ k[lo:hi].t() * st["scale"]
                if case["causal"]:
                    gap = (n - m + torch.arange(i, j, device="cuda"))[:, None] - torch.arange(lo, hi, device="cuda")
                    x = x.masked_fill((gap < 0) | (gap >= w) if w else gap < 0, -math.inf)
                z = torch.logsumexp(x, -1)
                o = torch.exp(x - z[:, None]) @ v[lo:hi]
                if st["prefix"] is not None:
                    pz = st["prefix"][1][q0 + i:q0 + j, h].double()
                    both = torch.logaddexp(z, pz)
                    o = o * torch.exp(z - both)[:, None]
                    o = o + st["prefix"][0][q0 + i:q0 + j, h].double() * torch.exp(pz - both)[:, None]
                    z = both
                out[q0 + i:q0 + j, h], lse[q0 + i:q0 + j, h] = o, z
        q0, k0 = q0 + m, k0 + n
    return {"out": out, "lse": lse}
