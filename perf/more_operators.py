"""Cases that measure the operators that take prompts and single tokens through linear-attention layers, and rotary positions:

  prompt  rssm_linattn_prompt  linear attention with a decay for each head over packed prompts, states into the slots' pool
  step    rssm_linattn_step    the same recurrence for one token of each row
  rope    rssm_rope            rotary positions of queries and keys

A case is a dict of plain values; lengths follow from its "lens" number, everything else from the seed. With `own` false the
operators run in their plain form (elementary torch operations in float32, decays and angles in float64)."""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}
CHUNK = 128     # tokens of a chunk of the plain form


# --------------------------------------------------------------------------- cases

def _linear(name, op, **kw):
    # h value heads over g key heads of n, values of p: 32 over 16 heads of 128 unless the case says otherwise
    c = {"op": op, "batch": 1, "h": 32, "g": 16, "n": 128, "p": 128, "act": "bf16", "state": "f32", "decay": "token", "w": True,
         "lens": 1}
    if op == "prompt":
        c.update({"len": 190, "resume": False})
    c.update(kw)
    return dict(c, name=name)


def _rope(name, **kw):
    c = {"op": "rope", "batch": 1, "len": 1, "past": 1000, "hq": 32, "hk": 8, "d": 128, "rot": 128, "interleaved": False,
         "act": "bf16", "base": 10000.0, "scaling": "none", "factor": 1.0, "original": 8192, "where": "slots", "lens": 1}
    c.update(kw)
    return dict(c, name=name)


def listed():
    return [
        # one user's short prompt: latency counts
        _linear("prompt 1 row short", "prompt", len=190, lens=1),
        # a serving batch of prompts of different lengths
        _linear("prompt 24 rows", "prompt", batch=24, len=2500, lens=2),
        # one long document: few heads' worth of rows, the work has to be split over its length
        _linear("prompt 1 row 50k", "prompt", len=50001, lens=3),
        # the second part of prompts cut in pieces, in the geometry of the Mamba2 decode workload (128 heads of 64 over 8 groups)
        _linear("prompt 10 rows 128 heads", "prompt", batch=10, len=4001, h=128, g=8, p=64, state="bf16", resume=True, lens=4),
        # float32 activations, small heads, a constant decay for each head
        _linear("prompt f32", "prompt", batch=3, len=700, h=8, g=8, n=64, p=64, act="f32", decay="head", w=False, lens=5),
        # a few tokens for each of many rows (drafts that were accepted, ends of prompts)
        _linear("prompt 300 rows of 24", "prompt", batch=300, len=24, resume=True, lens=6),
        # one user's next token
        _linear("step 1 row", "step", lens=7),
        # a decode batch, float32 states
        _linear("step 256 rows", "step", batch=256, lens=8),
        # a decode batch in the geometry of the Mamba2 decode workload, bf16 states
        _linear("step 512 rows bf16", "step", batch=512, h=128, g=8, p=64, state="bf16", lens=9),
        # one user's next token, rotated before it enters the cache
        _rope("rope 1 token", lens=10),
        # prompts of 9 users: slices of one fused projection, rotated into dense queries and keys
        _rope("rope 9 prompts", batch=9, len=8001, past=40, base=500000.0, lens=11),
        # far positions given as a list, frequencies stretched for long contexts, interleaved pairs in a part of the head
        _rope("rope far interleaved f32", len=5003, past=900000, hq=16, hk=2, d=80, rot=32, interleaved=True, act="f32",
              scaling="yarn", factor=16.0, where="list", lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "prompt", "step", "rope"])
    lens = rng.randrange(1 << 20)
    if op == "rope":
        d = rng.choice([64, 80, 128, 192, 256])
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 2, 4, 8])
        batch = _log(rng, 1, 256)
        n = _log(rng, 1, max(1, 250000000 // (batch * (hq + hk) * d)))
        rot = min(d, rng.choice([d, d, d // 2, 4 * rng.randrange(1, d // 4 + 1)]))
        return {"op": op, "batch": batch, "len": min(n, 20000), "past": _log(rng, 1, 1 << 20), "hq": hq, "hk": hk, "d": d, "rot": rot,
                "interleaved": rng.random() < 0.5, "act": rng.choice(["bf16", "bf16", "f32"]),
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "scaling": rng.choice(["none", "none", "linear", "base", "yarn", "bands"]),
                "factor": rng.choice([2.0, 8.0, 32.0]), "original": rng.choice([4096, 8192]), "where": rng.choice(["slots", "list"]),
                "lens": lens}
    g = rng.choice([1, 2, 4, 8, 16])
    h = g * rng.choice([1, 2, 4, 8, 16])
    c = {"op": op, "h": min(h, 128), "g": g, "n": rng.choice([64, 128]), "p": rng.choice([64, 128]),
         "act": rng.choice(["bf16", "bf16", "bf16", "f32"]), "state": rng.choice(["f32", "f32", "bf16"]),
         "decay": rng.choice(["token", "token", "head"]), "w": rng.random() < 0.5, "lens": lens}
    if op == "step":
        c["batch"] = _log(rng, 1, min(512, 1 + 1000000000 // (c["h"] * c["n"] * c["p"] * BYTES[c["state"]])))
        return c
    most = (300000 if c["act"] == "f32" else 1600000) // c["h"]      # tokens
    c["batch"] = _log(rng, 1, min(300, most, 16000 // c["h"]))
    c["len"] = _log(rng, 1, most // c["batch"])
    c["resume"] = rng.random() < 0.4
    return c


# --------------------------------------------------------------------------- inputs

def _lengths(case):
    """New tokens of each row: the first row has them all, the others a quarter and up (of a few tokens: perhaps none)."""
    r = random.Random(case["lens"])
    n = case["len"]
    return [n] + [r.randint(n // 4, n) for _ in range(case["batch"] - 1)]


def _pasts(case):
    """Tokens of each row before these."""
    r = random.Random(case["lens"] + 1)
    n = case["past"]
    return [n] + [r.randint(n // 4, n) for _ in range(case["batch"] - 1)]


def _cu(counts):
    cu = torch.zeros(len(counts) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(counts, dtype=torch.int64).cumsum(0)
    return cu.to(DEV)


def _slots(g, batch):
    num = batch + max(1, batch // 4)
    return num, torch.randperm(num, generator=g, device=DEV)[:batch].to(torch.int32)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def prepare(case, seed):
    import ssm_linear_attention_gb300 as ssm
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    act = DTYPES[case["act"]]
    batch = case["batch"]
    num_slots, slots = _slots(g, batch)
    st = {"case": case, "slots": slots}
    if case["op"] == "rope":
        lens, past = _lengths(case), _pasts(case)
        n, hq, hk, d = sum(lens), case["hq"], case["hk"], case["d"]
        # slices of one fused projection of queries, keys and values
        fused = _randn(g, n, hq + 2 * hk, d).to(act)
        st["q"], st["k"] = fused[:, :hq], fused[:, hq:hq + hk]
        st["q_out"], st["k_out"] = (torch.empty(n, x, d, device=DEV, dtype=act) for x in (hq, hk))
        st["cu"] = _cu(lens)
        row = torch.repeat_interleave(torch.arange(batch, device=DEV), torch.tensor(lens, device=DEV))
        first = torch.tensor(past, device=DEV)
        st["pos"] = (first[row] + torch.arange(n, device=DEV) - st["cu"][:-1].long()[row]).to(torch.int32)
        st["slot_len"] = torch.zeros(num_slots, device=DEV, dtype=torch.int32)
        st["slot_len"][slots.long()] = first.to(torch.int32)
        st["freq"] = _frequencies(case)
        make = getattr(ssm, "Rotary", None)
        if make is not None:
            scaling = None if case["scaling"] == "none" else \
                {"type": case["scaling"], "factor": case["factor"], "original": case["original"]}
            st["rotary"] = make(hq, hk, d, rot_dim=case["rot"], interleaved=case["interleaved"], base=case["base"],
                                scaling=scaling, act_dtype=act)
        return st
    lens = _lengths(case) if case["op"] == "prompt" else [1] * batch
    n, h, gk, nd, p = sum(lens), case["h"], case["g"], case["n"], case["p"]
    q, k = _randn(g, n, gk, nd), _randn(g, n, gk, nd)
    st["q"] = q.to(act)
    st["k"] = (k / k.norm(dim=-1, keepdim=True)).to(act)
    st["v"] = _randn(g, n, h, p).to(act)
    # memories of two to a few thousand tokens
    rate = torch.exp(torch.empty(h, device=DEV).uniform_(math.log(3e-4), math.log(0.7), generator=g))
    if case["decay"] == "head":
        st["decay"] = -rate
    else:
        st["decay"] = -rate * torch.empty(n, h, device=DEV).uniform_(0.3, 1.7, generator=g)
    st["w"] = torch.empty(n, h, device=DEV).uniform_(0.05, 1.0, generator=g) if case["w"] else None
    st["state"] = (0.1 * _randn(g, num_slots, h, p, nd)).to(DTYPES[case["state"]])
    st["cu"] = _cu(lens) if case["op"] == "prompt" else None
    st["lens"], st["most"] = torch.tensor(lens, device=DEV), max(lens)
    st["resume"] = torch.ones(batch, device=DEV, dtype=torch.uint8) if case.get("resume") else None
    make = getattr(ssm, "LinearAttention", None)
    if make is not None:
        st["layer"] = make(h, gk, nd, p, num_slots, batch, max_tokens=n, scale=nd ** -0.5, state_dtype=DTYPES[case["state"]],
                           act_dtype=act, out_dtype=act, state=st["state"])
    return st


def _frequencies(case):
    """Angle per position of each pair, float64, and the factor of the rotated values."""
    rot, base, f = case["rot"], case["base"], case["factor"]
    at = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    kind = case["scaling"]
    if kind == "base" and rot > 2:
        base = base * f ** (rot / (rot - 2))
    freq = base ** (-2 * at / rot)
    if kind == "linear":
        return freq / f, 1.0
    if kind == "yarn":
        # pairs that turn more than 32 times in the original length keep their frequency, those that turn less than once
        # are stretched, a ramp between
        ends = [rot * math.log(case["original"] / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (32, 1)]
        lo, hi = max(math.floor(ends[0]), 0), min(math.ceil(ends[1]), rot - 1)
        ramp = ((at - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return freq * (1 - ramp) + freq / f * ramp, 0.1 * math.log(f) + 1
    if kind == "bands":
        # by wavelength: up to a quarter of the original length kept, from the original length on stretched
        turns = case["original"] * freq / (2 * math.pi)
        keep = ((turns - 1) / (4 - 1)).clamp(0, 1)
        return freq * keep + freq / f * (1 - keep), 1.0
    return freq, 1.0


# --------------------------------------------------------------------------- one pass

def run(state):
    return {"prompt": run_prompt, "step": run_step, "rope": run_rope}[state["case"]["op"]](state)


def run_prompt(st):
    if own:
        o = st["layer"].prompt(st["q"], st["k"], st["v"], st["decay"], st["slots"], cu_tokens=st["cu"], w=st["w"],
                               resume=st["resume"])
    else:
        o = plain_prompt(st, st["case"])
    return {"o": o, "state": st["state"]}


def run_step(st):
    if own:
        o = st["layer"].step(st["q"], st["k"], st["v"], st["decay"], st["slots"], w=st["w"])
    else:
        o = plain_step(st, st["case"])
    return {"o": o, "state": st["state"]}


def run_rope(st):
    if own:
        if st["case"]["where"] == "list":
            q, k = st["rotary"](st["q"], st["k"], positions=st["pos"], q_out=st["q_out"], k_out=st["k_out"])
        else:
            q, k = st["rotary"](st["q"], st["k"], cache_indices=st["slots"], slot_len=st["slot_len"], cu_tokens=st["cu"],
                                q_out=st["q_out"], k_out=st["k_out"])
        return {"q": q, "k": k}
    return plain_rope(st, st["case"])


def plain_prompt(st, case):
    """All chunks at once: inside a chunk by its matrix of decayed products, between chunks by the decays of whole chunks."""
    b, h, gk = case["batch"], case["h"], case["g"]
    nd, p = case["n"], case["p"]
    c = min(CHUNK, st["most"])
    nc = -(-st["most"] // c)
    at = torch.arange(nc * c, device=DEV)
    valid = at < st["lens"][:, None]                                                # [b, nc c]
    token = (st["cu"][:-1].long()[:, None] + at).clamp(max=st["q"].shape[0] - 1)

    def heads(x, many):                                                             # [b, h, nc, c, ...]
        x = torch.where(valid[:, :, None, None], x[token].float(), 0.0).view(b, nc, c, x.shape[1], -1)
        return x.repeat_interleave(many, 3).permute(0, 3, 1, 2, 4)
    q, k, v = heads(st["q"], h // gk), heads(st["k"], h // gk), heads(st["v"], 1)
    decay = st["decay"].double()
    decay = decay.expand(b, nc * c, h) if case["decay"] == "head" else decay[token]
    total = torch.where(valid[..., None], decay, 0.0).view(b, nc, c, h).permute(0, 3, 1, 2).cumsum(-1)
    w = valid[..., None].float().expand(b, nc * c, h) if st["w"] is None else torch.where(valid[..., None], st["w"][token], 0.0)
    w = w.view(b, nc, c, h).permute(0, 3, 1, 2)                                     # [b, h, nc, c]
    later = torch.ones(c, c, device=DEV, dtype=torch.bool).triu(1)
    s = torch.matmul(q, k.transpose(-1, -2))
    s = s * (total[..., :, None] - total[..., None, :]).masked_fill(later, -math.inf).exp().float() * w[..., None, :]
    o = torch.matmul(s, v)
    del s
    whole = total[..., -1]                                                          # [b, h, nc]
    fade = (whole[..., None] - total).exp().float() * w
    own_part = torch.matmul((v * fade[..., None]).transpose(-1, -2), k)             # [b, h, nc, p, n]
    del v, k
    ends = torch.cat([torch.zeros_like(whole[..., :1]), whole.cumsum(-1)], -1)      # [b, h, nc + 1]
    before = torch.ones(nc + 1, nc, device=DEV, dtype=torch.bool).tril(-1)
    carry = (ends[..., :, None] - ends[..., None, 1:]).masked_fill(~before, -math.inf).exp().float()
    states = torch.matmul(carry, own_part.view(b, h, nc, p * nd))
    del own_part
    slots = st["slots"].long()
    if st["resume"] is not None:
        states += ends.exp().float()[..., None] * st["state"][slots].float().view(b, h, 1, p * nd)
    states = states.view(b, h, nc + 1, p, nd)
    o += total.exp().float()[..., None] * torch.matmul(q, states[:, :, :nc].transpose(-1, -2))
    has = st["lens"] > 0
    st["state"][slots[has]] = states[has, :, nc].to(st["state"].dtype)
    o = (o * nd ** -0.5).permute(0, 2, 3, 1, 4).reshape(b, nc * c, h, p)
    return o[valid].to(DTYPES[case["act"]])


def plain_step(st, case):
    many = case["h"] // case["g"]
    q, k = (st[x].float().repeat_interleave(many, 1) for x in ("q", "k"))
    v = st["v"].float() if st["w"] is None else st["v"].float() * st["w"][..., None]
    slots = st["slots"].long()
    s = st["state"][slots].float() * st["decay"].exp().expand(case["batch"], case["h"])[..., None, None]
    s += v[..., :, None] * k[..., None, :]
    st["state"][slots] = s.to(st["state"].dtype)
    return ((s * q[..., None, :]).sum(-1) * case["n"] ** -0.5).to(DTYPES[case["act"]])


def plain_rope(st, case):
    freq, m = st["freq"]
    a = st["pos"].double()[:, None] * freq
    cos, sin = (m * a.cos()).float()[:, None], (m * a.sin()).float()[:, None]
    rot, half = case["rot"], case["rot"] // 2

    def turn(x):
        y = x.float()
        if case["interleaved"]:
            u, v = y[..., 0:rot:2], y[..., 1:rot:2]
            y = torch.cat([torch.stack([u * cos - v * sin, v * cos + u * sin], -1).flatten(-2), y[..., rot:]], -1)
        else:
            u, v = y[..., :half], y[..., half:rot]
            y = torch.cat([u * cos - v * sin, v * cos + u * sin, y[..., rot:]], -1)
        return y.to(x.dtype)
    return {"q": turn(st["q"]), "k": turn(st["k"])}


# --------------------------------------------------------------------------- the work of one pass

def work(case):
    a = BYTES[case["act"]]
    if case["op"] == "rope":
        n = sum(_lengths(case)) * (case["hq"] + case["hk"])
        return {"bytes": 2 * n * case["d"] * a, "flops": 3 * n * case["rot"]}
    lens = _lengths(case) if case["op"] == "prompt" else [1] * case["batch"]
    n, h = sum(lens), case["h"]
    gates = (h if case["decay"] == "head" else n * h) + (n * h if case["w"] else 0)
    moves = 1 if case["op"] == "prompt" and not case["resume"] else 2              # states read and written
    states = sum(x > 0 for x in lens) * h * case["p"] * case["n"] * BYTES[case["state"]]
    return {"bytes": n * (2 * case["g"] * case["n"] + 2 * h * case["p"]) * a + 4 * gates + moves * states,
            "flops": 4 * n * h * case["p"] * case["n"]}


# --------------------------------------------------------------------------- the same from the definitions, 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        freq, m = st["freq"]
        turn = torch.polar(torch.full((1, 1), m, device=DEV, dtype=torch.float64), st["pos"].double()[:, None] * freq)[:, None]
        out = {}
        for name in ("q", "k"):
            y = st[name].double().clone()
            part = y[..., :case["rot"]]
            pairs = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
            z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            y[..., :case["rot"]] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
            out[name] = y
        return out
    # one token after another, the rows with the most tokens first
    lens = _lengths(case) if case["op"] == "prompt" else [1] * case["batch"]
    order = sorted(range(len(lens)), key=lambda b: -lens[b])
    order = [b for b in order if lens[b]]
    start, at = [], 0
    for x in lens:
        start.append(at)
        at += x
    rows = torch.tensor(order, device=DEV)
    starts = torch.tensor(start, device=DEV)[rows]
    slots = st["slots"].long()[rows]
    many = case["h"] // case["g"]
    pool = st["state"].double()
    s = pool[slots].clone() if case["op"] == "step" or case["resume"] else torch.zeros_like(pool[slots])
    o = torch.zeros(at, case["h"], case["p"], device=DEV, dtype=torch.float64)
    alive = len(order)
    constant = st["decay"].double().exp() if case["decay"] == "head" else None
    for t in range(max(lens)):
        while lens[order[alive - 1]] <= t:
            alive -= 1
        i = starts[:alive] + t
        k, q = (st[x][i].double().repeat_interleave(many, 1) for x in ("k", "q"))
        v = st["v"][i].double()
        if st["w"] is not None:
            v = v * st["w"][i].double()[..., None]
        f = constant.expand(alive, -1) if constant is not None else st["decay"][i].double().exp()
        s[:alive] = torch.addcmul(s[:alive] * f[..., None, None], v[..., None], k[..., None, :])
        o[i] = (s[:alive] * q[..., None, :]).sum(-1) / math.sqrt(case["n"])
    pool[slots] = s
    return {"o": o, "state": pool}
