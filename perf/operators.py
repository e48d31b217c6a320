"""The position, cache and shared-prefix operators beside the attention calls,
as cases to be timed and compared.

Each case is one pass through one operator:

  rope        rotary position embedding of the queries and keys of a fused QKV
              projection, from token-major [B, N, heads, d] to the head-major
              [B, H, N, d] the attention reads, or (grad) the gradient's way
              back
  append      rotation of new tokens' queries and keys, and the write of their
              keys and values into the paged KV cache
  shared      one query token per sequence against the paged cache, where
              groups of sequences share a long prefix

`own` chooses between the plain form (elementary torch operations in 32 bits,
angles in 64) and the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _rope(name, B, N, Hq, Hkv, d, rotary, interleaved, scaling, start, grad):
    return {"name": name, "op": "rope", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "d": d, "rotary": rotary,
            "interleaved": interleaved, "scaling": scaling, "start": start, "grad": grad}


def _append(name, seqs, new, ctx, Hq, Hkv, d, page, rotary, interleaved, scaling):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "ctx": ctx, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "rotary": rotary, "interleaved": interleaved, "scaling": scaling}


def _shared(name, seqs, groups, prefix, own_len, Hq, Hkv, d, page):
    return {"name": name, "op": "shared", "seqs": seqs, "groups": groups, "prefix": prefix, "own_len": own_len,
            "Hq": Hq, "Hkv": Hkv, "d": d, "page": page}


def listed():
    return [
        # a short prompt in a small model: launch latency
        _rope("rope short prompt", 1, 257, 8, 8, 64, 64, False, "none", 0, False),
        # odd sizes, a quarter of the head rotated, positions far into a stretched context
        _rope("rope odd quarter head", 3, 1021, 6, 2, 128, 32, False, "yarn", 200000, False),
        # the training step's forward rotation at the causal benchmark's shape
        _rope("rope training forward", 4, 4096, 16, 16, 128, 128, False, "none", 0, False),
        # its backward at the grouped-head shape: neighbouring pairs, half the head
        _rope("rope grouped heads backward", 2, 8192, 32, 8, 128, 64, True, "wavelength", 0, True),
        # one sequence decoding one token: pure latency
        _append("append one token", 1, 1, 700, 8, 8, 64, 8, 64, False, "none"),
        # a decode step of the serving batch
        _append("append decode step", 64, 1, 9000, 32, 8, 128, 16, 128, False, "wavelength"),
        # a chunked-prefill step: ragged chunks of many sequences
        _append("append ragged chunks", 32, 1024, 4096, 32, 8, 128, 16, 128, False, "yarn"),
        # whole prompts entering the cache
        _append("append long prompts", 4, 16384, 0, 32, 8, 128, 64, 64, True, "linear"),
        # a few short requests behind a system prompt: latency
        _shared("shared few short", 8, 1, 515, 33, 8, 2, 64, 8),
        # the serving batch behind one long document
        _shared("shared serving batch", 64, 1, 8000, 512, 32, 8, 128, 16),
        # several documents, each with its own readers; small heads, groups of 8
        _shared("shared ragged groups", 96, 6, 5000, 1024, 32, 4, 64, 32),
        # many samples drawn behind one long context: the products count
        _shared("shared many samples", 256, 1, 30000, 256, 32, 8, 128, 16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    scaling = rng.choice(["none", "linear", "ntk", "yarn", "wavelength"])
    d = rng.choice([64, 128])
    page = rng.choice([8, 16, 32, 64])
    op = rng.choice(["rope", "append", "shared"])
    if op == "rope":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 3, 4])
        B = rng.randint(1, 4)
        N = _log(rng, 1, 16384 * 40 // (B * (Hq + Hkv)))
        c = _rope("", B, N, Hq, Hkv, d, rng.choice([d, d // 2, d // 4]), rng.random() < 0.5, scaling,
                  rng.choice([0, 0, 5000, 1000000]), rng.random() < 0.4)
    elif op == "append":
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        seqs = _log(rng, 1, 300)
        most = 700000000 // (4 * (Hq + 2 * Hkv) * d * seqs)
        new = 1 if rng.random() < 0.4 or most < 2 else _log(rng, 2, most)
        c = _append("", seqs, new, _log(rng, 1, 200000 // seqs), Hq, Hkv, d, page, rng.choice([d, d // 2]),
                    rng.random() < 0.5, scaling)
    else:
        Hkv = rng.choice([1, 2, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 8])
        seqs = _log(rng, 2, 200)
        c = _shared("", seqs, rng.randint(1, min(seqs, 5)), _log(rng, 40, 20000), _log(rng, 1, 100000 // seqs + 20),
                    Hq, Hkv, d, page)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# What a case's numbers mean (sizes follow from the case alone, values from the seed)
# ---------------------------------------------------------------------------

def _append_lens(c):
    """New tokens of each sequence, and the keys it has after them."""
    if c["new"] == 1:
        new = [1] * c["seqs"]
    else:
        new = [1 + (i * 7919 + 101) % c["new"] for i in range(c["seqs"])]
        new[0] = c["new"]
        if c["seqs"] > 3:
            new[2] = 0   # a sequence that brings nothing this step
    ctx = [0 if c["ctx"] == 0 else (c["ctx"] * 5 // 8) + (i * 4057) % (c["ctx"] * 3 // 8 + 1) for i in range(c["seqs"])]
    return new, [a + b for a, b in zip(new, ctx)]


def _append_pad(c):
    return 0 if c["new"] == 1 else 5   # rows behind the last sequence, left as they are


def _shared_plan(c):
    """First sequence of each group (and the end), prefix lengths, sequence lengths."""
    n, g = c["seqs"], c["groups"]
    offsets = [i + int((n - g) * (i / g) ** 1.3) for i in range(g)] + [n]
    prefix = [c["prefix"] - (37 * i) % (c["prefix"] // 4 + 1) for i in range(g)]
    lens = [prefix[i] + 1 + (s * 7919 + 11) % c["own_len"] for i in range(g) for s in range(offsets[i], offsets[i + 1])]
    return offsets, prefix, lens


def work(c):
    if c["op"] == "rope":
        n = c["B"] * c["N"] * (c["Hq"] + c["Hkv"])
        return {"bytes": 4 * n * c["d"] + 4 * c["N"] + 4 * c["rotary"], "flops": 3 * n * c["rotary"]}
    if c["op"] == "append":
        new, lens = _append_lens(c)
        n = sum(new)
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": 4 * n * heads * c["d"] + 4 * c["rotary"] + 4 * sum(-(-a // c["page"]) for a in new) + 8 * c["seqs"],
                "flops": 3 * n * (c["Hq"] + c["Hkv"]) * c["rotary"]}
    offsets, prefix, lens = _shared_plan(c)
    keys = sum(prefix) + sum(n - prefix[_group_of(offsets, s)] for s, n in enumerate(lens))
    return {"bytes": 4 * keys * c["Hkv"] * c["d"] + c["seqs"] * c["Hq"] * (4 * c["d"] + 4) + 4 * -(-keys // c["page"]),
            "flops": 4 * sum(lens) * c["Hq"] * c["d"]}


def _group_of(offsets, s):
    return max(i for i in range(len(offsets) - 1) if offsets[i] <= s)


def _frequencies(c):
    """Radians per position of each rotated pair, and the factor on cos and sin."""
    r, base, factor, trained = c["rotary"], 10000.0, 8.0, 8192.0
    kind = c["scaling"]
    if kind == "ntk":
        base *= factor ** (r / (r - 2))
    f = [base ** (-2.0 * i / r) for i in range(r // 2)]
    amp = 1.0
    if kind == "linear":
        f = [x / factor for x in f]
    if kind == "yarn":
        at = [r * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        keep = [1 - min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0) for i in range(r // 2)]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
        amp = 0.1 * math.log(factor) + 1.0
    if kind == "wavelength":
        keep = [min(max((trained * x / (2 * math.pi) - 1.0) / 3.0, 0.0), 1.0) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
    return torch.tensor(f, dtype=torch.float64, device=DEV), amp


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c = case
    gen = torch.Generator(DEV).manual_seed(1000003 * seed + 17)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)

    st = {"case": c, "Hq": c["Hq"], "Hkv": c["Hkv"]}
    if c["op"] == "rope":
        B, N, Hq, Hkv, d = c["B"], c["N"], c["Hq"], c["Hkv"], c["d"]
        st["inv_freq"], st["amp"] = _frequencies(c)
        st["positions"] = torch.arange(N, device=DEV, dtype=torch.int32) + c["start"]
        if c["grad"]:
            st["q"], st["k"] = normal(B, Hq, N, d), normal(B, Hkv, N, d)
        else:
            qkv = normal(B, N, Hq + 2 * Hkv, d)
            st["q"] = qkv[:, :, :Hq].transpose(1, 2)
            st["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        return st
    if c["op"] == "append":
        new, lens = _append_lens(c)
        total = sum(new) + _append_pad(c)
        pages = [-(-n // c["page"]) for n in lens]
        Hq, Hkv, d = c["Hq"], c["Hkv"], c["d"]
        qkv = normal(total, Hq + 2 * Hkv, d)
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["inv_freq"], st["amp"] = _frequencies(c)
        perm = torch.randperm(sum(pages), generator=gen, device=DEV).to(torch.int32)
        st["table"] = torch.full((len(pages), max(pages)), -1, dtype=torch.int32, device=DEV)
        for s, n in enumerate(pages):
            st["table"][s, :n] = perm[sum(pages[:s]):sum(pages[:s]) + n]
        st["cu"] = _i32([0] + [sum(new[:i + 1]) for i in range(len(new))]) if c["new"] > 1 else None
        st["lens"] = _i32(lens)
        st["k_cache"] = normal(sum(pages), Hkv, c["page"], d)
        st["v_cache"] = normal(sum(pages), Hkv, c["page"], d)
        st["q_out"] = torch.zeros(total, Hq, d, dtype=torch.bfloat16, device=DEV)
        return st
    offsets, prefix, lens = _shared_plan(c)
    page, Hkv, d = c["page"], c["Hkv"], c["d"]
    rows, total = [], 0
    for g in range(c["groups"]):
        full = prefix[g] // page
        shared = list(range(total, total + full))
        total += full
        for s in range(offsets[g], offsets[g + 1]):
            n = -(-lens[s] // page) - full
            rows.append(shared + list(range(total, total + n)))
            total += n
    most = max(len(r) for r in rows)
    perm = torch.randperm(total, generator=gen, device=DEV)
    filled = torch.tensor([r + [-1] * (most - len(r)) for r in rows], device=DEV)
    st["table"] = torch.where(filled >= 0, perm[filled.clamp(min=0)], -1).to(torch.int32)
    st["offsets"], st["prefix"], st["lens"] = _i32(offsets), _i32(prefix), _i32(lens)
    st["max_own"] = max(n - prefix[_group_of(offsets, s)] for s, n in enumerate(lens))
    st["k_cache"], st["v_cache"] = normal(total, Hkv, page, d), normal(total, Hkv, page, d)
    for g in range(c["groups"]):   # a prefix that ends inside a page: every reader's copy of that page holds its tail
        tail = prefix[g] % page
        at = st["table"][offsets[g]:offsets[g + 1], prefix[g] // page].long()
        for cache in (st["k_cache"], st["v_cache"]):
            cache[at, :, :tail] = cache[at[:1], :, :tail].clone()
    st["q"] = normal(c["seqs"], c["Hq"], d)
    return st


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"rope": _plain_rope, "append": _plain_append, "shared": _plain_shared}[op](state)


def _own(st, op):
    from tiled_attention_17_b200 import binding
    c = st["case"]
    if op == "rope" and c["grad"]:
        # the gradient goes back into a fused projection gradient's rows
        out = torch.empty(c["B"], c["N"], c["Hq"] + c["Hkv"], c["d"], dtype=torch.bfloat16, device=DEV)
        heads = out.transpose(1, 2)
        binding.rope_backward(st["q"], st["inv_freq"], st["positions"], interleaved=c["interleaved"],
                              amplitude=st["amp"], out=heads[:, :c["Hq"]])
        binding.rope_backward(st["k"], st["inv_freq"], st["positions"], interleaved=c["interleaved"],
                              amplitude=st["amp"], out=heads[:, c["Hq"]:])
        return out
    if op == "rope":
        return tuple(binding.rope(st[x], st["inv_freq"], st["positions"], interleaved=c["interleaved"],
                                  amplitude=st["amp"]) for x in ("q", "k"))
    if op == "append":
        binding.paged_append(st["k"], st["v"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                             cu_seqlens=st["cu"], q=st["q"], q_out=st["q_out"], inv_freq=st["inv_freq"],
                             interleaved=c["interleaved"], amplitude=st["amp"])
        return st["q_out"], st["k_cache"], st["v_cache"]
    o, lse, _ = binding.paged_decode_shared(st["q"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                            st["offsets"], st["prefix"], max_own_len=st["max_own"])
    return o, lse


def _rotate(x, angle, amp, interleaved, sign):
    """x [..., d] in 32 bits; angle [..., r / 2] in 64, over the same leading axes."""
    r = 2 * angle.shape[-1]
    cos, sin = (torch.cos(angle) * amp).float(), (torch.sin(angle) * (amp * sign)).float()
    x = x.float()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, w = a * cos - b * sin, a * sin + b * cos
    head = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((head, x[..., r:]), -1).to(torch.bfloat16)


def _plain_rope(st):
    c = st["case"]
    angle = st["positions"].double()[:, None] * st["inv_freq"]
    sign = -1.0 if c["grad"] else 1.0
    q, k = (_rotate(st[x], angle, st["amp"], c["interleaved"], sign).contiguous() for x in ("q", "k"))
    return torch.cat((q, k), 1).transpose(1, 2).contiguous() if c["grad"] else (q, k)


def _plain_append(st):
    c = st["case"]
    if st["cu"] is None:
        seq, pos = torch.arange(c["seqs"], device=DEV), st["lens"].long() - 1
        n = c["seqs"]
    else:
        n = st["q"].shape[0] - _append_pad(c)
        cu = st["cu"].long()
        token = torch.arange(n, device=DEV)
        seq = torch.searchsorted(cu[1:], token, right=True)
        pos = token - cu[seq + 1] + st["lens"].long()[seq]
    angle = (pos.double()[:, None] * st["inv_freq"])[:, None]
    page = st["table"].long()[seq, pos // c["page"]]
    row = pos % c["page"]
    st["q_out"][:n] = _rotate(st["q"][:n], angle, st["amp"], c["interleaved"], 1.0)
    st["k_cache"][page, :, row] = _rotate(st["k"][:n], angle, st["amp"], c["interleaved"], 1.0)
    st["v_cache"][page, :, row] = st["v"][:n]
    return st["q_out"], st["k_cache"], st["v_cache"]


def _plain_shared(st):
    """The prefix once for each group, the rest for each sequence, one softmax over both."""
    c = st["case"]
    S, Hq, Hkv, d, page = c["seqs"], c["Hq"], c["Hkv"], c["d"], c["page"]
    G, scale = Hq // Hkv, c["d"] ** -0.5
    offsets, prefix, lens, table = st["offsets"].long(), st["prefix"].long(), st["lens"].long(), st["table"].long()
    seq = torch.arange(S, device=DEV)
    group = torch.searchsorted(offsets[1:], seq, right=True)
    place = seq - offsets[group]
    widest, longest = S - c["groups"] + 1, c["prefix"]
    q = st["q"].float().view(S, Hkv, G, d)

    # prefix: [groups, Hkv, places * G, keys]
    t = torch.arange(longest, device=DEV)
    at = table[offsets[:-1]][:, (t // page).clamp(max=table.shape[1] - 1)]
    kp, vp = (x[at.clamp(min=0), :, t % page].float().transpose(1, 2) for x in (st["k_cache"], st["v_cache"]))
    qg = torch.zeros(c["groups"], widest, Hkv, G, d, device=DEV)
    qg[group, place] = q
    sp = qg.permute(0, 2, 1, 3, 4).flatten(2, 3) @ kp.transpose(2, 3) * scale
    sp = torch.where(t < prefix[:, None, None, None], sp, -math.inf).unflatten(2, (widest, G))

    # own keys: [S, Hkv, G, keys]
    u = torch.arange(st["max_own"], device=DEV)
    pos = prefix[group][:, None] + u
    at = table.gather(1, (pos // page).clamp(max=table.shape[1] - 1))
    ko, vo = (x[at.clamp(min=0), :, pos % page].float().transpose(1, 2) for x in (st["k_cache"], st["v_cache"]))
    so = q @ ko.transpose(2, 3) * scale
    so = torch.where((pos < lens[:, None])[:, None, None], so, -math.inf)

    m = torch.maximum(sp.amax(-1)[group, :, place], so.amax(-1))
    mg = torch.zeros(c["groups"], widest, Hkv, G, device=DEV)
    mg[group, place] = m
    pp = torch.exp(sp - mg.permute(0, 2, 1, 3)[..., None])
    po = torch.exp(so - m[..., None])
    total = pp.sum(-1)[group, :, place] + po.sum(-1)
    out = (pp.flatten(2, 3) @ vp).unflatten(2, (widest, G))[group, :, place] + po @ vo
    return (out / total[..., None]).to(torch.bfloat16).view(S, Hq, d), (m + torch.log(total)).view(S, Hq)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "shared":
        offsets, prefix, lens = _shared_plan(c)
        q = st["q"].double() * c["d"] ** -0.5
        o = torch.empty(c["seqs"], c["Hq"], c["d"], dtype=torch.float64, device=DEV)
        lse = torch.empty(c["seqs"], c["Hq"], dtype=torch.float64, device=DEV)
        for s in range(c["seqs"]):
            g = _group_of(offsets, s)
            cut = prefix[g]
            key, value = [], []
            for row, first, last in ((offsets[g], 0, cut), (s, cut, lens[s])):
                t = torch.arange(first, last, device=DEV)
                page = st["table"][row].long()[t // c["page"]]
                key.append(st["k_cache"][page, :, t % c["page"]])
                value.append(st["v_cache"][page, :, t % c["page"]])
            key, value = torch.cat(key).double(), torch.cat(value).double()
            for h in range(c["Hkv"]):
                mine = slice(h * (c["Hq"] // c["Hkv"]), (h + 1) * (c["Hq"] // c["Hkv"]))
                score = torch.einsum("gd,td->gt", q[s, mine], key[:, h])
                lse[s, mine] = torch.logsumexp(score, 1)
                o[s, mine] = torch.einsum("gt,td->gd", torch.softmax(score, 1), value[:, h])
        return o, lse

    r = c["rotary"]
    # the pairs as complex numbers: a turn by the angle is a product with e^(i angle)
    first = torch.arange(0, r, 2, device=DEV) if c["interleaved"] else torch.arange(0, r // 2, device=DEV)
    second = first + (1 if c["interleaved"] else r // 2)

    def turned(x, pos, back=False):
        y = x.double().clone()
        turn = torch.polar(torch.full((len(pos), r // 2), st["amp"], dtype=torch.float64, device=DEV),
                           torch.outer(pos.double(), st["inv_freq"]) * (-1 if back else 1))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if c["op"] == "rope":
        q, k = (turned(st[x], st["positions"], c["grad"]).contiguous() for x in ("q", "k"))
        return torch.cat((q, k), 1).permute(0, 2, 1, 3).contiguous() if c["grad"] else (q, k)
    new, lens = _append_lens(c)
    q_out, k_cache, v_cache = st["q_out"].double(), st["k_cache"].double(), st["v_cache"].double()
    at = 0
    for s in range(c["seqs"]):
        pos = torch.arange(lens[s] - new[s], lens[s], device=DEV)
        here = slice(at, at + new[s])
        page = st["table"][s].long()[pos // c["page"]]
        q_out[here] = turned(st["q"][here].transpose(0, 1), pos).transpose(0, 1)
        k_cache[page, :, pos % c["page"]] = turned(st["k"][here].transpose(0, 1), pos).transpose(0, 1)
        v_cache[page, :, pos % c["page"]] = st["v"][here].double()
        at += new[s]
    return q_out, k_cache, v_cache
