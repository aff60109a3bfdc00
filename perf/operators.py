"""Cases of the position rotation and the paged key-value cache.

Three operators that belong together around the attention kernels:

  rope    rotary positions on up to four tensors at once: q and k before a
          forward, q, k and their tangents before a forward + JVP, dq and dk
          after a backward (the inverse rotation)
  append  keys and values of new tokens written into a paged cache, the keys
          (and the queries, beside them) rotated to their positions on the way
  decode  attention of one new token per sequence over the paged cache

``run`` computes them in elementary torch operations (``own`` false) or makes
the calls a user makes of ``attention_forward_jvp_gb300.binding`` (``own``
true).  ``exact`` is the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}

# ------------------------------------------------------------------- cases
# fields of every case: op, dtype.  rot: rotated leading elements of a head;
# interleaved: pairs (2i, 2i + 1), else (i, i + rot / 2); scaling / factor /
# orig: how the frequencies are stretched for contexts longer than `orig`.


def listed():
    rope = {"op": "rope", "dtype": "bf16", "base": 10000.0, "interleaved": False, "scaling": "none", "factor": 1.0,
            "orig": 0, "inverse": False, "start": 0, "token_major": False, "jagged": False, "lens_seed": 0}
    app = {"op": "append", "dtype": "bf16", "base": 10000.0, "interleaved": False, "scaling": "none", "factor": 1.0,
           "orig": 0, "page": 64, "idle": 0, "tokens": 1, "head_major": True}
    dec = {"op": "decode", "dtype": "bf16", "page": 64, "idle": 0, "head_major": True, "q_std": 1.5}
    return [
        # the smallest forward + JVP step of the workloads: launch latency
        dict(rope, name="rope_tiny", B=1, N=128, Hq=2, Hk=2, D=64, rot=64, tensors=4),
        # q, k and both tangents of the causal training workload
        dict(rope, name="rope_causal_jvp", B=2, N=4096, Hq=16, Hk=16, D=128, rot=128, tensors=4),
        # dq and dk of a packed batch, half of each head rotated in neighbouring pairs
        dict(rope, name="rope_jagged_grad", dtype="f16", B=64, N=1024, Hq=8, Hk=8, D=64, rot=32, tensors=2,
             interleaved=True, inverse=True, jagged=True, lens_seed=7),
        # one chunk of a long prompt, far from position 0, read out of a packed projection
        dict(rope, name="rope_far_chunk", B=1, N=8192, Hq=32, Hk=8, D=128, rot=128, tensors=2, base=500000.0,
             scaling="by_parts", factor=8.0, orig=8192, start=110000, token_major=True),
        # one new token of a few sequences: launch latency
        dict(app, name="append_few", B=4, Hq=8, Hk=2, Dqk=64, Dv=64, rot=64, len_lo=1, len_hi=512, lens_seed=3, page=16),
        # one new token of a full serving batch, a few of its places idle
        dict(app, name="append_batch", B=256, Hq=32, Hk=8, Dqk=128, Dv=128, rot=128, len_lo=1, len_hi=16384,
             lens_seed=4, idle=12, base=500000.0, scaling="linear", factor=4.0, head_major=False),
        # prompts of many lengths at once, a quarter of each head rotated in neighbouring pairs
        dict(app, name="append_prompts", dtype="f16", B=24, Hq=16, Hk=4, Dqk=256, Dv=128, rot=64, len_lo=1,
             len_hi=2048, lens_seed=5, tokens=1024, page=32, interleaved=True),
        # one short sequence: launch latency
        dict(dec, name="decode_short", B=1, Hq=8, Hk=2, Dqk=64, Dv=64, len_lo=77, len_hi=77, lens_seed=0, page=16),
        # a serving batch of many lengths, small pages, token-major pool
        dict(dec, name="decode_batch", B=64, Hq=32, Hk=8, Dqk=128, Dv=128, len_lo=1, len_hi=8192, lens_seed=1,
             idle=6, page=16, head_major=False),
        # one long document: the work of one sequence split over the card
        dict(dec, name="decode_long", B=1, Hq=32, Hk=4, Dqk=128, Dv=128, len_lo=131071, len_hi=131071, lens_seed=0),
        # every query head with a key head of its own
        dict(dec, name="decode_mha_f16", dtype="f16", B=32, Hq=16, Hk=16, Dqk=64, Dv=64, len_lo=1, len_hi=4096,
             lens_seed=2),
        # one key head for 64 query heads, wide keys
        dict(dec, name="decode_mqa_wide", B=16, Hq=64, Hk=1, Dqk=256, Dv=128, len_lo=2000, len_hi=32768, lens_seed=6,
             page=128),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_rope(rng, c, D):
    c["interleaved"] = rng.random() < 0.4
    c["rot"] = rng.choice([D, D, D, D // 2, D // 4, max(2, D // 2 - 4)])
    c["base"] = rng.choice([10000.0, 100000.0, 500000.0, 1000000.0])
    c["scaling"] = rng.choice(["none", "none", "linear", "base", "by_parts"])
    c["factor"] = 1.0 if c["scaling"] == "none" else float(rng.choice([2, 4, 8, 32]))
    c["orig"] = rng.choice([2048, 4096, 8192])
    if c["rot"] == 2 and c["scaling"] == "base":
        c["scaling"] = "linear"


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "decode"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "lens_seed": rng.randrange(1 << 30)}
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    Hq = Hk * rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
    if op == "rope":
        D = rng.choice([32, 64, 64, 128, 128, 256])
        _draw_rope(rng, c, D)
        c.update(Hq=Hq, Hk=Hk, D=D, inverse=rng.random() < 0.4, tensors=rng.choice([2, 2, 4]),
                 jagged=rng.random() < 0.35, token_major=rng.random() < 0.4)
        most = 60_000_000 // ((Hq + Hk) * D * c["tensors"] // 2)  # token rows
        c["B"] = _log(rng, 1, min(64, max(1, most // 16)))
        c["N"] = _log(rng, 1, max(1, min(16384, most // c["B"])))
        c["start"] = 0 if c["jagged"] else rng.choice([0, 0, rng.randrange(131072)])
        return c
    big = rng.choice([(64, 64), (128, 128), (128, 128), (128, 64), (64, 128), (256, 128), (256, 256), (32, 32), (16, 64)])
    c.update(Hq=Hq, Hk=Hk, Dqk=big[0], Dv=big[1], page=rng.choice([1, 8, 16, 16, 24, 32, 64, 64, 128, 256]),
             head_major=rng.random() < 0.5, idle=rng.choice([0, 0, 10, 40]))
    if op == "append":
        _draw_rope(rng, c, big[0])
        c["tokens"] = rng.choice([1, 1, _log(rng, 2, 1024)])
        c["B"] = _log(rng, 1, 256 if c["tokens"] == 1 else max(1, 12000 // c["tokens"]))
        c["len_lo"] = 1
        c["len_hi"] = _log(rng, 1, 16384)
        return c
    c["q_std"] = rng.choice([0.5, 1.5, 3.0])
    most = 400_000_000 // (Hk * sum(big))  # keys of all sequences, padded to the longest
    c["B"] = _log(rng, 1, min(256, max(1, most // 64)))
    c["len_hi"] = _log(rng, 1, max(1, min(131072, most // c["B"])))
    c["len_lo"] = rng.choice([1, max(1, c["len_hi"] // 2), c["len_hi"]])
    return c


def _lengths(c):
    """Sequence lengths of a case (not of its seed): what the cache holds of
    each sequence after the call; 0 for a place of the batch that is idle."""
    r = random.Random(c["lens_seed"])
    lens = [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])]
    lens[r.randrange(c["B"])] = c["len_hi"]
    return [0 if c["B"] > 1 and r.random() * 100 < c["idle"] and n < c["len_hi"] else n for n in lens]


def _new_tokens(c, lens):
    """Tokens of each sequence that an append brings: one each (an idle place
    brings a row too), or up to `tokens` of the sequence's last ones."""
    r = random.Random(c["lens_seed"] + 1)
    return [1] * c["B"] if c["tokens"] == 1 else [min(n, r.randint(1, c["tokens"])) for n in lens]


# ------------------------------------------------------------------ inputs


def _tables(c, count):
    """What a program that rotates by hand keeps: cos and sin of every
    position and frequency, taken in 64 bits and held in 32."""
    f = torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"]
    base = c["base"]
    if c["scaling"] == "base":
        base = base * c["factor"] ** (c["rot"] / (c["rot"] - 2))
    f = base ** -f
    scale = 1.0
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] == "by_parts":
        keep = ((c["orig"] / (2 * math.pi) * f - 1.0) / 31.0).clamp(0, 1)
        f = f * keep + f / c["factor"] * (1 - keep)
        scale = 0.1 * math.log(c["factor"]) + 1.0
    angle = torch.arange(count, dtype=torch.float64, device="cuda")[:, None] * f
    return (angle.cos() * scale).float(), (angle.sin() * scale).float()


def _own_rope(c):
    from attention_forward_jvp_gb300 import binding
    by_parts = c["scaling"] == "by_parts"
    return binding.Rope(c["rot"], base=c["base"], interleaved=c["interleaved"],
                        scaling=None if c["scaling"] == "none" else c["scaling"], factor=c["factor"],
                        orig_len=c["orig"], low_turns=1.0, high_turns=32.0,
                        out_scale=0.1 * math.log(c["factor"]) + 1.0 if by_parts else 1.0)


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _pool(g, c, lens, first):
    """A pool of pages in random order, filled with keys and values (and with
    whatever else a pool holds), the table of each sequence's pages and the
    lengths.  The pages before first[b] of sequence b are in nobody's hands
    (an append does not look at them): their entries are 0, as are those
    behind its last page."""
    last = [-(-n // c["page"]) for n in lens]
    count = sum(n - f for n, f in zip(last, first)) + 3
    order = torch.randperm(count, generator=g, device="cuda")
    table = torch.zeros((c["B"], max(max(last), 1) + 1), dtype=torch.int64, device="cuda")
    at = torch.arange(table.shape[1], device="cuda")[None]
    held = (at >= torch.tensor(first, device="cuda")[:, None]) & (at < torch.tensor(last, device="cuda")[:, None])
    table[held] = order[: count - 3]
    page, dt = c["page"], TYPES[c["dtype"]]
    shapes = [(count, c["Hk"], page, d) if c["head_major"] else (count, page, c["Hk"], d) for d in (c["Dqk"], c["Dv"])]
    k, v = (_randn(g, shape, dt) for shape in shapes)
    if not c["head_major"]:  # the same view of either pool: [pages, heads, page, d]
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    return {"k_cache": k, "v_cache": v, "page_table": table.int(),
            "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "rope":
        heads = [c["Hq"], c["Hk"]] * (c["tensors"] // 2)
        if c["jagged"]:
            lens = _lengths(dict(c, len_lo=1, len_hi=c["N"], idle=0))
            off = torch.tensor([0] + lens, device="cuda").cumsum(0)
            T = sum(lens)
            s["offsets"] = off.int()
            s["x"] = [_randn(g, (T, h, c["D"]), dt).transpose(0, 1) if c["token_major"] else _randn(g, (h, T, c["D"]), dt)
                      for h in heads]
        else:
            s["positions"] = (torch.arange(c["N"], dtype=torch.int32, device="cuda") + c["start"]).expand(c["B"], -1)
            if c["token_major"]:  # views of one packed projection, as a model's first product leaves it
                packed = _randn(g, (c["B"], c["N"], sum(heads), c["D"]), dt)
                s["x"] = [t.transpose(1, 2) for t in packed.split(heads, 2)]
            else:
                s["x"] = [_randn(g, (c["B"], h, c["N"], c["D"]), dt) for h in heads]
        count = c["start"] + c["N"]
    elif c["op"] == "append":
        lens = _lengths(c)
        new = _new_tokens(c, lens)
        s.update(_pool(g, c, lens, [max(0, n - m) // c["page"] for n, m in zip(lens, new)]))
        s["offsets"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
        T = sum(new)
        s["k"], s["v"], s["q"] = (_randn(g, (T, h, d), dt) for h, d in
                                  ((c["Hk"], c["Dqk"]), (c["Hk"], c["Dv"]), (c["Hq"], c["Dqk"])))
        count = max(lens) + 1
    else:
        s.update(_pool(g, c, _lengths(c), [0] * c["B"]))
        s["q"] = _randn(g, (c["B"], c["Hq"], c["Dqk"]), dt, c["q_std"])
    if c["op"] != "decode":
        if own:
            s["rope"] = _own_rope(c)
        else:
            s["cos"], s["sin"] = _tables(c, count)
    if own and c["op"] != "rope":
        from attention_forward_jvp_gb300 import binding
        s["cache"] = binding.PagedCache(s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"])
    return s


# --------------------------------------------------------------------- run


def _rotate(x, cos, sin, interleaved):
    """x [..., d] in 32 bits; cos, sin [..., rot / 2], broadcast over heads."""
    half = cos.shape[-1]
    x = x.float()
    if interleaved:
        a, b = x[..., 0 : 2 * half : 2], x[..., 1 : 2 * half : 2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half : 2 * half]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., 2 * half :]), -1)


def _plain_rope(s):
    c = s["case"]
    if c["jagged"]:
        off = s["offsets"].long()
        t = torch.arange(s["x"][0].shape[1], device="cuda")
        pos = t - off[(t[:, None] >= off[1:]).sum(1)]
    else:
        pos = s["positions"].long()[:, None]
    cos, sin = s["cos"][pos], s["sin"][pos]
    sin = -sin if c["inverse"] else sin
    return [_rotate(x, cos, sin, c["interleaved"]).to(x.dtype) for x in s["x"]]


def _plain_append(s):
    c = s["case"]
    off, lens = s["offsets"].long(), s["seq_lens"].long()
    t = torch.arange(s["k"].shape[0], device="cuda")
    seq = (t[:, None] >= off[1:]).sum(1)
    pos = t - off[seq + 1] + lens[seq]
    live = pos >= 0  # an idle place's row has no position: nothing is written, its q is zero
    cos, sin = s["cos"][pos.clamp(min=0)][:, None], s["sin"][pos.clamp(min=0)][:, None]
    q = (_rotate(s["q"], cos, sin, c["interleaved"]) * live[:, None, None]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, c["interleaved"]).to(s["k"].dtype)
    page = s["page_table"].long()[seq, pos.clamp(min=0) // c["page"]]
    slot = pos.clamp(min=0) % c["page"]
    s["k_cache"][page[live], :, slot[live]] = k[live]
    s["v_cache"][page[live], :, slot[live]] = s["v"][live]
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": q}


def _plain_decode(s):
    c = s["case"]
    B, Hq, Dqk = s["q"].shape
    table, lens = s["page_table"].long(), s["seq_lens"].long()
    k = s["k_cache"][table].transpose(1, 2).flatten(2, 3).float()  # [B, Hk, keys, Dqk]
    v = s["v_cache"][table].transpose(1, 2).flatten(2, 3).float()
    q = s["q"].float().view(B, c["Hk"], Hq // c["Hk"], Dqk)
    z = q @ k.transpose(-1, -2) * Dqk**-0.5
    z = z.masked_fill((torch.arange(z.shape[-1], device="cuda") >= lens[:, None])[:, None, None], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    o = p @ v / total.masked_fill(total == 0, 1.0)  # a sequence without keys: zeros, and -inf below
    return {"o": o.view(B, Hq, -1).to(s["q"].dtype), "lse": (total.log() + top).view(B, Hq)}


def run(state):
    s = state
    c = s["case"]
    if not own:
        if c["op"] == "rope":
            return _plain_rope(s)
        return _plain_append(s) if c["op"] == "append" else _plain_decode(s)
    from attention_forward_jvp_gb300 import binding
    if c["op"] == "rope":
        if c["jagged"]:
            return binding.attn_rope(s["x"], s["rope"], offsets=s["offsets"], inverse=c["inverse"])
        return binding.attn_rope(s["x"], s["rope"], positions=s["positions"], inverse=c["inverse"])
    if c["op"] == "append":
        off = s["offsets"] if c["tokens"] != 1 else None
        q = binding.attn_paged_append(s["cache"], s["k"], s["v"], rope=s["rope"], q=s["q"], offsets=off)
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "q": q}
    o, lse = binding.attn_paged_decode(s["cache"], s["q"])
    return {"o": o, "lse": lse}


def work(case):
    c = case
    if c["op"] == "rope":
        rows = sum(_lengths(dict(c, len_lo=1, len_hi=c["N"], idle=0))) if c["jagged"] else c["B"] * c["N"]
        elements = rows * (c["Hq"] + c["Hk"]) * (c["tensors"] // 2)
        return {"bytes": 4 * elements * c["D"], "flops": 3 * elements * c["rot"]}
    lens = _lengths(c)
    if c["op"] == "append":
        new = _new_tokens(c, lens)
        rows = sum(m for m, n in zip(new, lens) if n)
        elements = rows * (c["Hk"] * (c["Dqk"] + c["Dv"]) + c["Hq"] * c["Dqk"])
        return {"bytes": 4 * elements + 8 * c["B"], "flops": 3 * rows * (c["Hk"] + c["Hq"]) * c["rot"]}
    keys = sum(lens)
    wide = c["Dqk"] + c["Dv"]
    return {"bytes": 2 * keys * c["Hk"] * wide + c["B"] * c["Hq"] * (2 * wide + 4) + 4 * sum(-(-n // c["page"]) for n in lens),
            "flops": 2 * keys * c["Hq"] * wide}


# ------------------------------------------------------------------- exact


def _turn(c, pos, x, inverse=False):
    """The rotation as a product of complex numbers, in 64 bits: x [..., T, d],
    pos a list of T positions."""
    rot = c["rot"]
    i = np.arange(rot // 2, dtype=np.float64)
    if c["scaling"] == "base":
        w = np.exp(-2.0 * i / rot * math.log(c["base"]) - 2.0 * i / (rot - 2) * math.log(c["factor"]))
    else:
        w = np.exp(-2.0 * i / rot * math.log(c["base"]))
    size = 1.0
    if c["scaling"] == "linear":
        w = w / c["factor"]
    elif c["scaling"] == "by_parts":
        turns = c["orig"] * w / (2.0 * np.pi)
        slow = 1.0 - np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        w = w * (1.0 - slow * (1.0 - 1.0 / c["factor"]))
        size = 1.0 + 0.1 * math.log(c["factor"])
    angle = np.asarray(pos, dtype=np.float64)[:, None] * w[None]
    unit = torch.from_numpy(size * np.exp((-1j if inverse else 1j) * angle)).to(x.device)
    x = x.double()
    head = x[..., :rot]
    if c["interleaved"]:
        y = torch.view_as_real(torch.complex(head[..., 0::2], head[..., 1::2]) * unit).reshape(head.shape)
    else:
        z = torch.complex(head[..., : rot // 2], head[..., rot // 2 :]) * unit
        y = torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., rot:]), -1)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        if c["jagged"]:
            pos = [p for n in _lengths(dict(c, len_lo=1, len_hi=c["N"], idle=0)) for p in range(n)]
        else:
            pos = range(c["start"], c["start"] + c["N"])
        return [_turn(c, pos, x, c["inverse"]) for x in s["x"]]
    lens = _lengths(c)
    if c["op"] == "append":
        k_all, v_all = s["k_cache"].double(), s["v_cache"].double()
        q_out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        table, at = s["page_table"].tolist(), 0
        for b, m in enumerate(_new_tokens(c, lens)):
            rows, at = slice(at, at + m), at + m
            if m == 0 or lens[b] == 0:
                continue
            pos = list(range(lens[b] - m, lens[b]))
            q_out[rows] = _turn(c, pos, s["q"][rows].transpose(0, 1)).transpose(0, 1)
            k = _turn(c, pos, s["k"][rows].transpose(0, 1)).transpose(0, 1)
            page = torch.tensor([table[b][p // c["page"]] for p in pos], device="cuda")
            slot = torch.tensor([p % c["page"] for p in pos], device="cuda")
            k_all[page, :, slot] = k
            v_all[page, :, slot] = s["v"][rows].double()
        return {"k_cache": k_all, "v_cache": v_all, "q": q_out}
    group = c["Hq"] // c["Hk"]
    o = torch.zeros((c["B"], c["Hq"], c["Dv"]), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pages = s["page_table"][b, : -(-n // c["page"])].long()
        for h in range(c["Hk"]):
            heads = slice(h * group, (h + 1) * group)
            k = s["k_cache"][pages, h].flatten(0, 1)[:n].double()
            v = s["v_cache"][pages, h].flatten(0, 1)[:n].double()
            z = torch.einsum("gd,jd->gj", s["q"][b, heads].double(), k) / math.sqrt(c["Dqk"])
            lse[b, heads] = torch.logsumexp(z, -1)
            o[b, heads] = torch.einsum("gj,jd->gd", torch.softmax(z, -1), v)
    return {"o": o, "lse": lse}
