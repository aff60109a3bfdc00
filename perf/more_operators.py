"""Cases of the operators that make a paged key-value cache smaller, and read it back.

  append4  keys and values of new tokens rounded to 4 bits and written into a
           paged cache, the keys (and the queries, beside them) rotated to
           their positions on the way; then read back as the cache holds
           them, as a prompt's own attention takes them
  gather   the last tokens of each sequence, of a cache in 16 or 4 bits, as
           the dense jagged tensors that the attention kernels take
  decode4  attention of one new token per sequence over a cache in 4 bits
  weights  the attention weight that a token's query heads gave each key,
           added up in 32 bits beside the cache (16 or 4 bits)
  evict    the keys with the largest such weights, the first and the most
           recent ones, copied into fewer pages, head by head

A cache in 4 bits holds 64 neighbouring elements of a row (32 where the head
has no more) as whole numbers n of 0 .. 15 with a scale s and a least value m
in fp16: x = m + n s.

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
MOST_HALF = 65504.0

# ------------------------------------------------------------------- cases
# fields of every case: op, dtype (of q, new tokens and outputs), bits (of the
# cache), Hk key heads, B sequences of len_lo .. len_hi tokens (drawn from
# lens_seed), pages of `page` tokens, head_major: pools [page, head, token, D],
# else [page, token, head, D]; idle: per cent of empty places.


def listed():
    base = {"dtype": "bf16", "bits": 4, "page": 64, "idle": 0, "head_major": True, "len_lo": 1, "lens_seed": 0}
    app = dict(base, op="append4", base=10000.0, interleaved=False, tokens=1)
    gat = dict(base, op="gather")
    dec = dict(base, op="decode4", q_std=1.5)
    wei = dict(base, op="weights", q_std=1.5, decay=1.0)
    evi = dict(base, op="evict", sinks=4)
    return [
        # one new token of a few sequences: launch latency
        dict(app, name="append4_few", B=4, Hq=8, Hk=2, Dqk=64, Dv=64, rot=64, len_hi=512, lens_seed=3, page=16),
        # prompts of many lengths at once, a quarter of each head rotated in neighbouring pairs
        dict(app, name="append4_prompts", dtype="f16", B=24, Hq=16, Hk=4, Dqk=256, Dv=128, rot=64, len_hi=2048,
             lens_seed=5, tokens=1024, page=32, interleaved=True),
        # what a batch holds, for the attention of the next chunks of its prompts
        dict(gat, name="gather_batch", bits=16, B=16, Hk=8, Dqk=128, Dv=128, len_hi=8192, lens_seed=8, tokens=8192,
             page=16, head_major=False),
        # one long shared prefix out of 4 bits
        dict(gat, name="gather_prefix4", B=1, Hk=8, Dqk=128, Dv=128, len_lo=30001, len_hi=30001, tokens=30001),
        # one short sequence: launch latency
        dict(dec, name="decode4_short", B=1, Hq=8, Hk=2, Dqk=64, Dv=64, len_lo=77, len_hi=77, page=16),
        # a serving batch of many lengths, small pages, token-major pool
        dict(dec, name="decode4_batch", B=64, Hq=32, Hk=8, Dqk=128, Dv=128, len_hi=8192, lens_seed=1, idle=6, page=16,
             head_major=False),
        # one long document: the work of one sequence split over the card
        dict(dec, name="decode4_long", B=1, Hq=32, Hk=4, Dqk=128, Dv=128, len_lo=262143, len_hi=262143),
        # few key heads for many query heads, wide keys
        dict(dec, name="decode4_wide_f16", dtype="f16", B=16, Hq=32, Hk=2, Dqk=256, Dv=128, len_lo=2000, len_hi=32768,
             lens_seed=6, page=128),
        # the weights of a serving batch's step, older ones fading
        dict(wei, name="weights_batch", bits=16, B=64, Hq=32, Hk=8, Dqk=128, Dv=128, len_hi=8192, lens_seed=1, idle=6,
             page=16, head_major=False, decay=0.98),
        # those of one long document, added up
        dict(wei, name="weights_long4", B=1, Hq=32, Hk=4, Dqk=128, Dv=128, len_lo=131071, len_hi=131071),
        # a batch cut down to its budget
        dict(evi, name="evict_batch", bits=16, B=32, Hk=8, Dqk=128, Dv=128, len_hi=8192, lens_seed=9, keep=2048,
             recent=256),
        # a quarter of one long document kept
        dict(evi, name="evict_long4", B=1, Hk=4, Dqk=128, Dv=128, len_lo=131071, len_hi=131071, keep=32768, recent=1024),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append4", "gather", "decode4", "decode4", "weights", "evict"])
    c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f16"]), "lens_seed": rng.randrange(1 << 30),
         "bits": 4 if op in ("append4", "decode4") else rng.choice([4, 16]),
         "page": rng.choice([1, 8, 16, 16, 24, 32, 64, 64, 128, 256]), "head_major": rng.random() < 0.5,
         "idle": rng.choice([0, 0, 10, 40])}
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    big = rng.choice([(64, 64), (128, 128), (128, 128), (128, 64), (64, 128), (256, 128), (256, 256), (32, 32), (32, 64)])
    c.update(Hk=Hk, Dqk=big[0], Dv=big[1])
    if op in ("append4", "decode4", "weights"):
        c["Hq"] = Hk * rng.choice([1, 1, 2, 3, 4, 6, 8, 16])
    if op == "append4":
        c["interleaved"] = rng.random() < 0.4
        c["rot"] = rng.choice([big[0], big[0], big[0], big[0] // 2, big[0] // 2 - 4])
        c["base"] = rng.choice([10000.0, 100000.0, 500000.0, 1000000.0])
        c["tokens"] = rng.choice([1, _log(rng, 2, 1024)])
        c["B"] = _log(rng, 1, 256 if c["tokens"] == 1 else max(1, 12000 // c["tokens"]))
        c["len_hi"] = _log(rng, 1, 16384)
        c["len_lo"] = 1
        return c
    most = (400_000_000 if op == "decode4" else 120_000_000) // (Hk * sum(big))  # keys, padded to the longest
    c["B"] = _log(rng, 1, min(128, max(1, most // 64)))
    c["len_hi"] = _log(rng, 1, max(1, min(131072, most // c["B"])))
    c["len_lo"] = rng.choice([1, max(1, c["len_hi"] // 2), c["len_hi"]])
    if op == "gather":
        c["tokens"] = rng.choice([c["len_hi"], _log(rng, 1, c["len_hi"])])
    elif op == "evict":
        c["keep"] = max(1, int(c["len_hi"] * rng.choice([0.05, 0.25, 0.5, 0.9])))
        c["recent"] = rng.choice([0, 1, 32, c["keep"] // 4])
        c["sinks"] = rng.choice([0, 0, 4])
    else:
        c["q_std"] = rng.choice([0.5, 1.5, 3.0])
        c["decay"] = rng.choice([1.0, 0.98, 0.0])
    return c


def _lengths(c):
    """Sequence lengths of a case (not of its seed): what the cache holds of
    each sequence after the call; 0 for a place of the batch that is idle."""
    r = random.Random(c["lens_seed"])
    lens = [r.randint(c["len_lo"], c["len_hi"]) for _ in range(c["B"])]
    lens[r.randrange(c["B"])] = c["len_hi"]
    return [0 if c["B"] > 1 and r.random() * 100 < c["idle"] and n < c["len_hi"] else n for n in lens]


def _last_tokens(c, lens):
    """Tokens of each sequence that an append brings or a gather takes: one
    each (an idle place brings a row too), or up to `tokens` of its last."""
    r = random.Random(c["lens_seed"] + 1)
    if c["op"] == "append4":
        return [1] * c["B"] if c["tokens"] == 1 else [min(n, r.randint(1, c["tokens"])) for n in lens]
    return [min(n, c["tokens"]) for n in lens]


# ------------------------------------------------------------ 4-bit values


def _groups(d):
    return max(1, d // 64)


def _round4(x):
    """x [..., d] in 32 bits -> bytes [..., d / 2], element 2i in the low half
    of byte i, and fp16 [..., 2, groups]: scales, then least values."""
    d = x.shape[-1]
    x = x.clamp(-MOST_HALF, MOST_HALF).unflatten(-1, (_groups(d), -1))
    low = x.amin(-1, keepdim=True).half()
    step = ((x.amax(-1, keepdim=True) - low.float()) / 15.0).half()
    s = step.float()
    n = ((x - low.float()) / torch.where(s > 0, s, 1.0)).round().clamp(0, 15)
    n = torch.where(s > 0, n, 0.0).flatten(-2).to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), torch.stack((step[..., 0], low[..., 0]), -2)


def _values4(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    g = scales.shape[-1]
    n = n.unflatten(-1, (g, -1)) * scales[..., 0, :, None].float() + scales[..., 1, :, None].float()
    return n.flatten(-2)


# ------------------------------------------------------------------ inputs


def _randn(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).to(dtype)


def _pool(g, c, lens, first, spare):
    """A pool of pages in random order, filled with keys and values (and with
    whatever else a pool holds), the table of each sequence's pages and the
    lengths.  Pages before first[b] of sequence b are in nobody's hands: their
    entries are 0, as are those behind its last.  `spare`: further pages, in
    nobody's hands either; their numbers are returned beside."""
    last = [-(-n // c["page"]) for n in lens]
    used = sum(n - f for n, f in zip(last, first))
    count = used + spare + 3
    order = torch.randperm(count, generator=g, device="cuda")
    table = torch.zeros((c["B"], max(max(last), 1) + 1), dtype=torch.int64, device="cuda")
    at = torch.arange(table.shape[1], device="cuda")[None]
    held = (at >= torch.tensor(first, device="cuda")[:, None]) & (at < torch.tensor(last, device="cuda")[:, None])
    table[held] = order[:used]
    s = {"page_table": table.int(), "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    for name, d in (("k", c["Dqk"]), ("v", c["Dv"])):
        lead = (count, c["Hk"], c["page"]) if c["head_major"] else (count, c["page"], c["Hk"])
        if c["bits"] == 16:
            parts = [_randn(g, lead + (d,), TYPES[c["dtype"]])]
        else:
            parts = [torch.empty(lead + (d // 2,), dtype=torch.uint8, device="cuda"),
                     torch.empty(lead + (2, _groups(d)), dtype=torch.float16, device="cuda")]
            step = max(1, (1 << 26) // (c["Hk"] * c["page"] * d))
            for at in range(0, count, step):
                n = min(step, count - at)
                for whole, part in zip(parts, _round4(_randn(g, (n,) + lead[1:] + (d,), torch.float32))):
                    whole[at : at + n] = part
        # the same view of either layout: [pages, heads, page, ...]
        parts = [t if c["head_major"] else t.transpose(1, 2) for t in parts]
        s[name + "_cache"] = parts[0]
        if c["bits"] == 4:
            s[name + "_scale"] = parts[1]
    return s, order[used : used + spare]


def _own_cache(c, s, table="page_table", lens="seq_lens"):
    from attention_forward_jvp_gb300 import binding
    if c["bits"] == 16:
        return binding.PagedCache(s["k_cache"], s["v_cache"], s[table], s[lens])
    return binding.PagedCache4(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s[table], s[lens],
                               dtype=TYPES[c["dtype"]])


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = TYPES[c["dtype"]]
    lens = _lengths(c)
    first = [0] * c["B"]
    if c["op"] in ("append4", "gather"):
        new = _last_tokens(c, lens)
        if c["op"] == "append4":
            first = [max(0, n - m) // c["page"] for n, m in zip(lens, new)]
    pages = -(-c["keep"] // c["page"]) if c["op"] == "evict" else 0
    s, spare = _pool(g, c, lens, first, pages * c["B"])
    s["case"] = c
    if c["op"] in ("append4", "gather"):
        s["offsets"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
        s["T"] = sum(new)
    if c["op"] == "append4":
        s["k"], s["v"], s["q"] = (_randn(g, (s["T"], h, d), dt) for h, d in
                                  ((c["Hk"], c["Dqk"]), (c["Hk"], c["Dv"]), (c["Hq"], c["Dqk"])))
        if own:
            from attention_forward_jvp_gb300 import binding
            s["rope"] = binding.Rope(c["rot"], base=c["base"], interleaved=c["interleaved"])
        else:  # what a program that rotates by hand keeps: cos and sin, taken in 64 bits and held in 32
            f = c["base"] ** -(torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda") / c["rot"])
            angle = torch.arange(max(lens) + 1, dtype=torch.float64, device="cuda")[:, None] * f
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    if c["op"] in ("decode4", "weights"):
        s["q"] = _randn(g, (c["B"], c["Hq"], c["Dqk"]), dt, c["q_std"])
    if c["op"] == "weights":  # as the step's decode left them, and older weights
        s["lse"] = torch.logsumexp(_scores(s), -1).float().view(c["B"], c["Hq"])
        s["weights"] = torch.rand((c["B"], c["Hk"], s["page_table"].shape[1] * c["page"]), generator=g, device="cuda")
        s["weights"] *= _live(s)[:, None]
    if c["op"] == "evict":
        s["pages"] = spare.view(c["B"], pages).int()
        # a few keys with much of the weight; a fifth of them never looked at
        shape = (c["B"], c["Hk"], s["page_table"].shape[1] * c["page"])
        w = torch.randn(shape, generator=g, device="cuda").mul_(2.0).exp_()
        w *= torch.rand(shape, generator=g, device="cuda") > 0.2
        s["weights"] = w * _live(s)[:, None]
        # what the program's cache becomes: the same pools, another table and lengths
        s["after_table"], s["after_lens"] = torch.zeros_like(s["page_table"]), torch.zeros_like(s["seq_lens"])
        s["after_weights"] = torch.zeros_like(s["weights"])
        left = [min(n, c["keep"]) for n in lens]
        s["offsets"] = torch.tensor([0] + left, device="cuda").cumsum(0).int()
        s["T"] = sum(left)
    if own:
        s["cache"] = _own_cache(c, s)
        if c["op"] == "evict":
            s["after"] = _own_cache(c, s, "after_table", "after_lens")
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


def _live(s):
    """[B, places of a table row]: whether a sequence holds a token there."""
    count = s["page_table"].shape[1] * s["case"]["page"]
    return torch.arange(count, device="cuda") < s["seq_lens"].long()[:, None]


def _held(s, name, page, head, slot):
    """Rows of a pool at these places (index tensors that broadcast), in 32 bits."""
    if s["case"]["bits"] == 16:
        return s[name + "_cache"][page, head, slot].float()
    return _values4(s[name + "_cache"][page, head, slot], s[name + "_scale"][page, head, slot])


def _padded(s, name):
    """All places of every table row: [B, Hk, places, d] in 32 bits."""
    c, table = s["case"], s["page_table"].long()
    head = torch.arange(c["Hk"], device="cuda")[None, :, None, None]
    slot = torch.arange(c["page"], device="cuda")
    return _held(s, name, table[:, None, :, None], head, slot).flatten(2, 3)


def _scores(s):
    """sm_scale q k, -inf behind the lengths: [B, Hk, group, places]."""
    c = s["case"]
    q = s["q"].float().view(c["B"], c["Hk"], -1, c["Dqk"])
    z = q @ _padded(s, "k").transpose(-1, -2) * c["Dqk"] ** -0.5
    return z.masked_fill(~_live(s)[:, None, None], -math.inf)


def _token_places(s, table, offsets, lens, T):
    """Sequence, position and place of each of the T packed last tokens."""
    off = offsets.long()
    t = torch.arange(T, device="cuda")
    seq = (t[:, None] >= off[1:]).sum(1)
    pos = t - off[seq + 1] + lens.long()[seq]
    at = pos.clamp(min=0)
    return seq, pos, table.long()[seq, at // s["case"]["page"]], at % s["case"]["page"]


def _plain_gather(s, table, lens):
    c = s["case"]
    _, pos, page, slot = _token_places(s, table, s["offsets"], lens, s["T"])
    head = torch.arange(c["Hk"], device="cuda")[:, None]
    live = (pos >= 0)[:, None]
    return {n: (_held(s, n, page, head, slot) * live).to(TYPES[c["dtype"]]) for n in ("k", "v")}


def _plain_append4(s):
    c = s["case"]
    seq, pos, page, slot = _token_places(s, s["page_table"], s["offsets"], s["seq_lens"], s["T"])
    live = pos >= 0  # an idle place's row has no position: nothing is written, its q is zero
    cos, sin = s["cos"][pos.clamp(min=0)][:, None], s["sin"][pos.clamp(min=0)][:, None]
    q = (_rotate(s["q"], cos, sin, c["interleaved"]) * live[:, None, None]).to(s["q"].dtype)
    k_codes, k_scales = _round4(_rotate(s["k"], cos, sin, c["interleaved"]))
    v_codes, v_scales = _round4(s["v"].float())
    s["k_cache"][page[live], :, slot[live]] = k_codes[live]
    s["k_scale"][page[live], :, slot[live]] = k_scales[live]
    s["v_cache"][page[live], :, slot[live]] = v_codes[live]
    s["v_scale"][page[live], :, slot[live]] = v_scales[live]
    return dict(_plain_gather(s, s["page_table"], s["seq_lens"]), q=q)


def _plain_decode4(s):
    c = s["case"]
    z = _scores(s)
    top = z.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = (z - top).exp()
    total = p.sum(-1, keepdim=True)
    o = p @ _padded(s, "v") / total.masked_fill(total == 0, 1.0)  # a sequence without keys: zeros, and -inf below
    return {"o": o.view(c["B"], c["Hq"], -1).to(s["q"].dtype), "lse": (total.log() + top).view(c["B"], c["Hq"])}


def _plain_weights(s):
    c = s["case"]
    lse = s["lse"].view(c["B"], c["Hk"], -1, 1)
    p = (_scores(s) - lse.masked_fill(lse == -math.inf, 0.0)).exp().sum(2)
    return torch.where(_live(s)[:, None], s["weights"] * c["decay"] + p, s["weights"])


def _plain_evict(s):
    c = s["case"]
    lens, live = s["seq_lens"].long(), _live(s)
    over = lens > c["keep"]
    at = torch.arange(live.shape[1], device="cuda")
    recent = min(c["recent"], c["keep"])
    sinks = min(c["sinks"], c["keep"] - recent)
    sure = (at < sinks) | (at >= (lens - recent)[:, None])
    key = s["weights"].masked_fill(sure[:, None], math.inf).masked_fill(~live[:, None], -math.inf)
    best = key.sort(dim=-1, descending=True, stable=True).indices[..., : c["keep"]]  # ties: the lowest index
    kept = torch.zeros_like(key, dtype=torch.bool).scatter_(-1, best, True) & (live & over[:, None])[:, None]
    b, h, old = kept.nonzero(as_tuple=True)
    new = (kept.cumsum(-1) - 1)[b, h, old]
    src = s["page_table"].long()[b, old // c["page"]]
    dst = s["pages"].long()[b, new // c["page"]]
    parts = ["k_cache", "v_cache"] + (["k_scale", "v_scale"] if c["bits"] == 4 else [])
    s.update({n: s[n].index_put_((dst, h, new % c["page"]), s[n][src, h, old % c["page"]]) for n in parts})
    w = torch.zeros_like(s["weights"])
    w[b, h, new] = s["weights"][b, h, old]
    w = torch.where(over[:, None, None], w, s["weights"])
    table = s["page_table"].clone()
    table[:, : s["pages"].shape[1]] = torch.where(over[:, None], s["pages"], table[:, : s["pages"].shape[1]])
    after = lens.clamp(max=c["keep"]).int()
    kv = {n: s[n] for n in parts} if c["bits"] == 16 else _plain_gather(s, table, after)
    return dict(kv, page_table=table, seq_lens=after, weights=w)


def run(state):
    s = state
    c = s["case"]
    if not own:
        if c["op"] == "gather":
            return _plain_gather(s, s["page_table"], s["seq_lens"])
        return {"append4": _plain_append4, "decode4": _plain_decode4, "weights": _plain_weights,
                "evict": _plain_evict}[c["op"]](s)
    from attention_forward_jvp_gb300 import binding
    if c["op"] == "append4":
        off = s["offsets"] if c["tokens"] != 1 else None
        q = binding.attn_paged_append(s["cache"], s["k"], s["v"], rope=s["rope"], q=s["q"], offsets=off)
        k, v = binding.attn_paged_gather(s["cache"], s["offsets"], s["T"])
        return {"k": k, "v": v, "q": q}
    if c["op"] == "gather":
        k, v = binding.attn_paged_gather(s["cache"], s["offsets"], s["T"])
        return {"k": k, "v": v}
    if c["op"] == "decode4":
        o, lse = binding.attn_paged_decode(s["cache"], s["q"])
        return {"o": o, "lse": lse}
    if c["op"] == "weights":
        return binding.attn_paged_weights(s["cache"], s["q"], s["lse"], s["weights"], decay=c["decay"])
    table, lens, w = binding.attn_paged_evict(s["cache"], s["weights"], c["keep"], s["pages"], sinks=c["sinks"],
                                              recent=c["recent"], out=(s["after_table"], s["after_lens"], s["after_weights"]))
    got = {"page_table": table, "seq_lens": lens, "weights": w}
    if c["bits"] == 16:
        got.update(k_cache=s["k_cache"], v_cache=s["v_cache"])
    else:  # what is left, as the values that the cache holds
        got["k"], got["v"] = binding.attn_paged_gather(s["after"], s["offsets"], s["T"])
    return got


def _row_bytes(c, d):
    return 2 * d if c["bits"] == 16 else d // 2 + 4 * _groups(d)


def work(case):
    c = case
    lens = _lengths(c)
    row = _row_bytes(c, c["Dqk"]) + _row_bytes(c, c["Dv"])
    wide = c["Dqk"] + c["Dv"]
    if c["op"] == "append4":
        rows = sum(m for m, n in zip(_last_tokens(c, lens), lens) if n)
        return {"bytes": rows * (c["Hk"] * (4 * wide + row) + 4 * c["Hq"] * c["Dqk"]) + 8 * c["B"],
                "flops": rows * (3 * (c["Hk"] + c["Hq"]) * c["rot"] + 4 * c["Hk"] * wide)}
    if c["op"] == "gather":
        rows = sum(_last_tokens(c, lens))
        return {"bytes": rows * c["Hk"] * (row + 2 * wide) + 8 * c["B"], "flops": 2 * rows * c["Hk"] * wide}
    keys = sum(lens)
    if c["op"] == "decode4":
        return {"bytes": keys * c["Hk"] * row + c["B"] * c["Hq"] * (2 * wide + 4) + 4 * sum(-(-n // c["page"]) for n in lens),
                "flops": 2 * keys * c["Hq"] * wide}
    if c["op"] == "weights":
        return {"bytes": keys * c["Hk"] * (_row_bytes(c, c["Dqk"]) + (8 if c["decay"] else 4))
                + c["B"] * c["Hq"] * (2 * c["Dqk"] + 4) + 4 * sum(-(-n // c["page"]) for n in lens),
                "flops": 2 * keys * c["Hq"] * c["Dqk"]}
    over = sum(n > c["keep"] for n in lens)
    left = sum(min(n, c["keep"]) for n in lens)
    dense = 2 * left * wide if c["bits"] == 4 else 0
    return {"bytes": c["Hk"] * (2 * over * c["keep"] * row + 4 * keys + 4 * left + dense) + 8 * c["B"], "flops": keys * c["Hk"]}


# ------------------------------------------------------------------- exact


def _turn(c, pos, x):
    """The rotation as a product of complex numbers, in 64 bits: x [T, heads, d],
    pos [T]."""
    rot = c["rot"]
    w = np.exp(-2.0 * np.arange(rot // 2, dtype=np.float64) / rot * math.log(c["base"]))
    unit = torch.from_numpy(np.exp(1j * np.asarray(pos, dtype=np.float64)[:, None, None] * w)).to(x.device)
    x = x.double()
    head = x[..., :rot]
    if c["interleaved"]:
        y = torch.view_as_real(torch.complex(head[..., 0::2], head[..., 1::2]) * unit).reshape(head.shape)
    else:
        z = torch.complex(head[..., : rot // 2], head[..., rot // 2 :]) * unit
        y = torch.cat((z.real, z.imag), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _nearest4(x):
    """The values that a cache in 4 bits holds for x [..., d], in 64 bits."""
    g = torch.stack(x.double().chunk(_groups(x.shape[-1]), -1), -2)
    low = g.min(-1, keepdim=True).values.half().double()
    step = ((g.max(-1, keepdim=True).values - low) / 15).half().double()
    n = torch.where(step > 0, torch.round((g - low) / step), torch.zeros_like(g)).clamp(0, 15)
    return (low + n * step).flatten(-2)


def _sequence(c, s, name, b, h, n):
    """Keys or values 0 .. n of a sequence's head, in 64 bits."""
    pages = s["page_table"][b, : -(-n // c["page"])].long()
    x = s[name + "_cache"][pages, h].flatten(0, 1)[:n]
    if c["bits"] == 16:
        return x.double()
    scale = s[name + "_scale"][pages, h].flatten(0, 1)[:n].double()
    d = 2 * x.shape[-1]
    out = torch.empty((n, d), dtype=torch.float64, device="cuda")
    out[:, 0::2], out[:, 1::2] = (x % 16).double(), (x // 16).double()
    each = d // _groups(d)
    return out * scale[:, 0].repeat_interleave(each, -1) + scale[:, 1].repeat_interleave(each, -1)


def _chosen(c, w, n):
    """Places that an eviction keeps of a head's n keys with weights w (an array)."""
    recent = min(c["recent"], c["keep"])
    sinks = min(c["sinks"], c["keep"] - recent)
    rest = np.arange(sinks, n - recent)
    order = rest[np.lexsort((rest, -w[rest].astype(np.float64)))]
    return np.sort(np.concatenate((np.arange(sinks), order[: c["keep"] - recent - sinks], np.arange(n - recent, n))))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    lens = _lengths(c)
    if c["op"] == "append4":
        new = _last_tokens(c, lens)
        pos = [n - m + i for n, m in zip(lens, new) for i in range(m)]
        live = torch.tensor([p >= 0 for p in pos], device="cuda")[:, None, None]
        k = _nearest4(_turn(c, pos, s["k"])) * live
        v = _nearest4(s["v"]) * live
        return {"k": k.transpose(0, 1), "v": v.transpose(0, 1), "q": _turn(c, pos, s["q"]) * live}
    if c["op"] == "gather":
        take = [(b, n, m) for b, (n, m) in enumerate(zip(lens, _last_tokens(c, lens))) if n]
        return {name: torch.stack([torch.cat([_sequence(c, s, name, b, h, n)[n - m :] for b, n, m in take])
                                   for h in range(c["Hk"])]) for name in ("k", "v")}
    if c["op"] == "evict":
        w_in, table = s["weights"].cpu().numpy(), s["page_table"].cpu().numpy().copy()
        w_out = np.zeros_like(w_in)
        parts = [n for n in ("k_cache", "v_cache") if c["bits"] == 16]
        pools = {n: s[n].clone() for n in parts}
        rows = {"k": [], "v": []}
        for b, n in enumerate(lens):
            more = n > c["keep"]
            heads = {"k": [], "v": []}
            for h in range(c["Hk"]):
                kept = _chosen(c, w_in[b, h], n) if more else np.arange(n)
                w_out[b, h, : len(kept)] = w_in[b, h, kept]
                if c["bits"] == 4:
                    at = torch.from_numpy(kept).cuda()
                    for name in rows:
                        heads[name].append(_sequence(c, s, name, b, h, n)[at])
                elif more:
                    at, to = torch.from_numpy(kept).cuda(), torch.arange(len(kept), device="cuda")
                    src, dst = s["page_table"][b].long()[at // c["page"]], s["pages"][b].long()[to // c["page"]]
                    for name in parts:
                        pools[name][dst, h, to % c["page"]] = s[name][src, h, at % c["page"]]
            if c["bits"] == 4 and n:
                for name in rows:
                    rows[name].append(torch.stack(heads[name]))
            if more:
                table[b, : s["pages"].shape[1]] = s["pages"][b].cpu().numpy()
        got = {"page_table": table, "seq_lens": np.array([min(n, c["keep"]) for n in lens], dtype=np.int32),
               "weights": w_out.astype(np.float64)}
        if c["bits"] == 4:
            got.update({name: torch.cat(x, 1) for name, x in rows.items()})
        got.update({name: x.double() for name, x in pools.items()})
        return got
    group = c["Hq"] // c["Hk"]
    if c["op"] == "weights":
        out = s["weights"].double()
    else:
        o = torch.zeros((c["B"], c["Hq"], c["Dv"]), dtype=torch.float64, device="cuda")
        lse = torch.full((c["B"], c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        for h in range(c["Hk"] if n else 0):
            heads = slice(h * group, (h + 1) * group)
            z = torch.einsum("gd,jd->gj", s["q"][b, heads].double(), _sequence(c, s, "k", b, h, n)) / math.sqrt(c["Dqk"])
            if c["op"] == "weights":
                p = torch.exp(z - s["lse"][b, heads, None].double()).sum(0)
                out[b, h, :n] = c["decay"] * out[b, h, :n] + p
            else:
                lse[b, heads] = torch.logsumexp(z, -1)
                o[b, heads] = torch.einsum("gj,jd->gd", torch.softmax(z, -1), _sequence(c, s, "v", b, h, n))
    return out if c["op"] == "weights" else {"o": o, "lse": lse}
