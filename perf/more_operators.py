"""What the cache's further dense operators are measured on: appends whose rotary positions have several
axes, attention with capped scores, distance bias and masks over the paged pool (a prompt's chunk or
single tokens), and the pool read back.

`run` computes a case's operator in its plain form (elementary torch operations in 32 bits), or,
where `own` is true, through the library's entry points. `exact` gives the same in 64 bits.
"""

import math

import torch

own = False

POSITIONS = 131072  # rows of the cos / sin table: the longest context of the repository's workloads
FMT_CODE = {"bf16": 0, "int8_side": 1, "int8_inline": 2, "e4m3": 3, "f16": 4}  # qkv_format of qkv.h
ACT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _append(name, T, hq, hkv, d, rot, fmt, woven, act="bf16", pairs=False, block=0):
    """T tokens of text, images and frames, three axes. woven: the pairs take the axes in turn, else in runs."""
    return {"name": name, "op": "append", "tokens": T, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "fmt": fmt,
            "woven": woven, "act": act, "pairs": pairs, "block": block}


def _attn(name, seqs, rows, ctx, hq, hkv, d, fmt, block, mask="causal", doc=0, window=0, cap=0.0, bias=False, hole=0,
          act="bf16"):
    """`seqs` sequences with rows[0] to rows[1] new tokens behind ctx[0] to ctx[1] older ones. mask "docs": documents
    of about `doc` tokens; "prefix": the context and half of the new tokens are seen by all. Every `hole`-th
    row sees nothing."""
    return {"name": name, "op": "attn", "seqs": seqs, "rlo": rows[0], "rhi": rows[1], "clo": ctx[0], "chi": ctx[1],
            "hq": hq, "hkv": hkv, "d": d, "fmt": fmt, "block": block, "mask": mask, "doc": doc, "window": window,
            "cap": cap, "bias": bias, "hole": hole, "act": act}


def _read(name, seqs, lo, hi, hkv, d, fmt, out, block, rot=0, pairs=False):
    """`seqs` sequences of lo to hi tokens, read whole; rot: K is turned back to before its rotation."""
    return {"name": name, "op": "read", "seqs": seqs, "lo": lo, "hi": hi, "hkv": hkv, "d": d, "fmt": fmt, "out": out,
            "block": block, "rot": rot, "pairs": pairs}


def listed():
    return [
        # a decode step of a model with image positions: nothing but latency
        _append("append one token 3 axes", 1, 16, 1, 256, 128, "int8_side", False),
        # an odd batch of image patches: half activations, inline records, adjacent pairs, woven axes
        _append("append 1369 patches inline", 1369, 16, 2, 128, 96, "int8_inline", True, act="f16", pairs=True, block=5),
        # a packed video prompt into an unquantised pool, the repository's largest append
        _append("append 16384 video bf16", 16384, 32, 8, 128, 128, "bf16", False, block=64),
        # one request decodes one token in a layer with a sliding window and capped scores: latency
        _attn("decode 1 row capped window", 1, (1, 1), (8191, 8191), 16, 1, 256, "int8_side", 16, window=4096, cap=50.0),
        # a serving batch of ragged lengths, capped scores
        _attn("decode 64 rows capped e4m3", 64, (1, 1), (0, 8191), 64, 8, 128, "e4m3", 64, cap=30.0),
        # draft tokens of a model with a distance bias, unquantised pool
        _attn("decode 8 x 5 drafts bias bf16", 8, (5, 5), (1000, 30000), 32, 4, 128, "bf16", 32, bias=True),
        # a whole prompt, the repository's chunked-prefill length, capped scores
        _attn("prompt 8192 capped int8", 1, (8192, 8192), (0, 0), 16, 1, 256, "int8_side", 16, cap=50.0),
        # prompts packed of documents that do not see one another, with a window
        _attn("prompts documents bf16", 6, (300, 4000), (0, 0), 32, 8, 128, "bf16", 32, mask="docs", doc=700, window=1024),
        # odd sizes everywhere: prefix mask, distance bias, half activations, groups of 12, blocks of 7, empty rows
        _attn("prompts prefix mask bias odd", 3, (77, 1501), (0, 999), 24, 2, 256, "e4m3", 7, mask="prefix", bias=True,
              hole=29, act="f16"),
        # the largest: the last chunk of the long context
        _attn("chunk 2048 behind 129024 int8", 1, (2048, 2048), (129024, 129024), 16, 1, 256, "int8_side", 64),
        # a short document's keys turned back, to be appended at another place
        _read("read 333 turned back f16", 1, 333, 333, 2, 128, "int8_inline", "f16", 5, rot=96, pairs=True),
        # a long conversation handed to another program
        _read("read 131072 int8 to bf16", 1, 131072, 131072, 1, 256, "int8_side", "bf16", 16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    d = rng.choice([128, 256])
    hkv = rng.choice([1, 1, 2, 4, 8])
    hq = hkv * rng.choice([1, 4, 5, 8, 12, 16])
    fmt = rng.choice(["bf16", "int8_side", "int8_inline", "e4m3", "f16"])
    act = fmt if fmt in ACT else rng.choice(["bf16", "f16"])
    block = rng.choice([1, 5, 16, 32, 64, 128])
    kind = rng.random()
    if kind < 0.25:
        top = 16384 * 48 * 128 // ((hq + 2 * hkv) * d)
        c = _append("", _log(rng, 1, min(16384, top)), hq, hkv, d, 16 * rng.randint(1, d // 16), fmt, rng.random() < 0.5,
                    act, rng.random() < 0.5, rng.choice([0, block]))
    elif kind < 0.45:
        seqs = rng.choice([1, 2, 7, 30])
        hi = _log(rng, 1, min(131072, 131072 * 256 // (d * hkv)) // seqs)
        c = _read("", seqs, rng.choice([hi, max(1, hi // 3)]), hi, hkv, d, fmt, rng.choice(["bf16", "f16", "f32"]), block,
                  rng.choice([0, 16 * rng.randint(1, d // 16)]), rng.random() < 0.5)
    else:
        kw = {"mask": rng.choice(["causal", "causal", "docs", "prefix"]), "doc": _log(rng, 20, 4000),
              "window": rng.choice([0, 0, _log(rng, 16, 8192)]), "cap": rng.choice([0.0, 30.0, 50.0]),
              "bias": rng.random() < 0.4, "hole": rng.choice([0, 0, 23]), "act": act}
        if rng.random() < 0.5:  # single tokens and drafts
            per = rng.choice([1, 1, 2, 5])
            seqs = _log(rng, 1, 128 // per)
            hi = _log(rng, 1, max(1, min(32768, 64 * 4096 * 8 * 128 // (seqs * per * hkv * d))))
            c = _attn("", seqs, (per, per), (rng.choice([0, hi // 2, hi]), hi), hq, hkv, d, fmt, block, **kw)
        else:  # prompts' chunks
            seqs = rng.choice([1, 1, 2, 5])
            hi = _log(rng, 16, 8192 // seqs)
            ctx = min(rng.choice([0, _log(rng, 1, 60000)]), 2048 * 131072 * 16 * 256 // (2 * seqs * hi * hq * d) // 2)
            c = _attn("", seqs, (max(1, hi // rng.choice([1, 3])), hi), (ctx // 2, ctx), hq, hkv, d, fmt, block, **kw)
    del c["name"]
    return c


def _spread(n, lo, hi):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _doc_starts(length, doc):
    """First position of every document: lengths from half of `doc` to one and a half."""
    at, k, starts = 0, 0, []
    while at < length:
        starts.append(at)
        at += max(1, doc * (50 + 37 * k % 101) // 100)
        k += 1
    return starts


def _row_masks(case, i):
    """What sequence i's rows see: lists of (start, end, position), and its length. Longer contexts have fewer new tokens."""
    n, ctx = _spread(case["seqs"], case["rlo"], case["rhi"])[i], _spread(case["seqs"], case["chi"], case["clo"])[i]
    starts = _doc_starts(ctx + n, case["doc"]) if case["mask"] == "docs" else [0]
    shared = ctx + (n + 1) // 2 if case["mask"] == "prefix" else 0
    rows, at = [], 0
    for k in range(n):
        p = ctx + k
        while at + 1 < len(starts) and starts[at + 1] <= p:
            at += 1
        empty = case["hole"] and k % case["hole"] == case["hole"] - 1
        rows.append((starts[at], 0 if empty else max(p + 1, shared), p))
    return rows, ctx + n


# ------------------------------------------------------------------ inputs
def _tokens(n, case, gen):
    """n tokens' K or V heads: N(0, 1), one token in a hundred four times as large."""
    x = torch.randn((n, case["hkv"], case["d"]), device="cuda", generator=gen)
    big = torch.rand((n, 1, 1), device="cuda", generator=gen) < 0.01
    return x * torch.where(big, 4.0, 1.0)


def _empty_pool(slots, case):
    s = {}
    shape = (slots, case["hkv"], case["d"])
    for x in "kv":
        if case["fmt"] in ACT:
            s[x + "_cache"] = torch.zeros(shape, dtype=ACT[case["fmt"]], device="cuda")
        elif case["fmt"] == "int8_inline":
            s[x + "_cache"] = torch.zeros((*shape[:2], case["d"] + 4), dtype=torch.uint8, device="cuda")
        else:
            s[x + "_cache"] = torch.zeros(shape, dtype=torch.int8 if case["fmt"] == "int8_side" else torch.uint8, device="cuda")
            if case["fmt"] == "int8_side":
                s[x + "_scale"] = torch.zeros(shape[:2], dtype=torch.float32, device="cuda")
    # the per-layer scales of an E4M3 pool, calibrated for values up to about 28
    s["k_layer"], s["v_layer"] = (0.0625, 0.0546875) if case["fmt"] == "e4m3" else (1.0, 1.0)
    return s


def _angles(rot):
    half = rot // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(POSITIONS, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _pair_axis(case):
    """Each pair's axis: a quarter time and the rest height and width in runs, or the three in turn and time for the last quarter."""
    n = case["rot"] // 2
    if case["woven"]:
        return [i % 3 if i < n - n // 4 else 0 for i in range(n)]
    return [0 if i < n // 4 else 1 if i < n // 4 + (n - n // 4) // 2 else 2 for i in range(n)]


def _table(lengths, block, gen):
    """A block table of sequences of these lengths, its blocks scattered over the pool; and the pool's slots."""
    need = [-(-n // block) for n in lengths]
    ids = torch.randperm(max(1, sum(need)), device="cuda", generator=gen).int()
    table = torch.full((len(lengths), max(1, max(need))), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = ids[at:at + n]
        at += n
    return table, len(ids) * block


def _prepare_append(case, gen):
    T, d = case["tokens"], case["d"]
    act = ACT[case["act"]]
    # q, k and v are slices of the packed projection's output, as a model has them
    packed = torch.cat([torch.randn((T, case["hq"], d), device="cuda", generator=gen),
                        _tokens(T, case, gen), _tokens(T, case, gen)], 1).to(act)
    s = {"q": packed[:, :case["hq"]], "k": packed[:, case["hq"]:case["hq"] + case["hkv"]],
         "v": packed[:, case["hq"] + case["hkv"]:], "q_out": torch.zeros((T, case["hq"], d), dtype=act, device="cuda"),
         "cos_sin": _angles(case["rot"]), "pair_axis": _pair_axis(case)}
    # a tenth of the tokens are text, whose axes agree; the others lie on grids of 37 x 37, one after the other
    t = torch.arange(T, device="cuda")
    first = torch.randint(0, POSITIONS - T - 64, (1,), device="cuda", generator=gen)
    grid = t - T // 10
    axes = torch.stack([grid // 1369, grid % 1369 // 37, grid % 37]) + T // 10
    s["axis_pos"] = (first + torch.where(t < T // 10, t, axes)).int()
    if case["block"]:
        s["block_table"], slots = _table([T], case["block"], gen)
        s["token_seq"], s["token_pos"] = torch.zeros_like(t).int(), t.int()
    else:
        slots = T + 255
        s["slot_mapping"] = torch.randperm(slots, device="cuda", generator=gen)[:T]
    return s | _empty_pool(slots, case)


def _fill(s, case, slots, gen):
    s |= _empty_pool(slots, case)
    act = ACT[case.get("act", "bf16")]
    for x in "kv":
        _store(s, case, x, torch.arange(slots, device="cuda"), _tokens(slots, case, gen).to(act).float())
    return s


def _prepare_attn(case, gen):
    order = torch.randperm(case["seqs"], generator=gen, device="cuda").tolist()
    per_seq = [_row_masks(case, i) for i in order]
    s = {"rows_of": [len(rows) for rows, _ in per_seq]}
    s["block_table"], slots = _table([n for _, n in per_seq], case["block"], gen)
    flat = [(i, *row) for i, (rows, _) in enumerate(per_seq) for row in rows]
    seq, start, end, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*flat))
    s |= {"row_seq": seq, "row_start": start if case["mask"] == "docs" else None, "row_end": end,
          "row_pos": pos if case["mask"] == "prefix" else None, "max_row_end": max(n for _, n in per_seq)}
    # the keys that each row may see, for the plain form's loops
    s["seen"] = [(max(a, p + 1 - case["window"]) if case["window"] else a, e) for _, a, e, p in flat]
    R, act = len(flat), ACT[case["act"]]
    # scores that are capped have a spread worth capping
    s["q"] = (torch.randn((R, case["hq"], case["d"]), device="cuda", generator=gen) * (2.0 if case["cap"] else 1.0)).to(act)
    s["out"] = torch.zeros((R, case["hq"], case["d"]), dtype=act, device="cuda")
    s["lse"] = torch.zeros((R, case["hq"]), dtype=torch.float32, device="cuda")
    s["slopes"] = None
    if case["bias"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, case["hq"] + 1, device="cuda") / case["hq"])
    s["workspace"] = torch.empty(512 << 20, dtype=torch.uint8, device="cuda")
    return _fill(s, case, slots, gen)


def _prepare_read(case, gen):
    lengths = _spread(case["seqs"], case["lo"], case["hi"])
    s = {}
    s["block_table"], slots = _table(lengths, case["block"], gen)
    s["token_seq"] = torch.repeat_interleave(torch.arange(case["seqs"]), torch.tensor(lengths)).int().cuda()
    s["token_pos"] = torch.cat([torch.arange(n) for n in lengths]).int().cuda()
    if case["rot"]:
        s["cos_sin"] = _angles(case["rot"])
    for x in "kv":
        s[x + "_out"] = torch.zeros((sum(lengths), case["hkv"], case["d"]), dtype=ACT[case["out"]], device="cuda")
    return _fill(s, case, slots, gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"append": _prepare_append, "attn": _prepare_attn, "read": _prepare_read}[case["op"]](case, gen)
    s["case"] = case
    return s


# ------------------------------------------------------------------ the plain forms
def _store(s, case, x, slots, vals):
    """fp32 head rows [n, Hkv, D] into the pool of `x` at `slots`, in its format."""
    cache = s[x + "_cache"]
    if case["fmt"] in ACT:
        cache[slots] = vals.to(cache.dtype)
        return
    if case["fmt"] == "e4m3":
        y = vals / torch.full_like(vals, s[x + "_layer"])
        cache[slots] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return
    amax = vals.abs().amax(-1, keepdim=True)
    scale = amax / torch.full_like(amax, 127.0)
    codes = torch.where(scale > 0, (vals / scale).round().clamp(-127, 127), 0.0).to(torch.int8)
    if case["fmt"] == "int8_side":
        cache[slots] = codes
        s[x + "_scale"][slots] = scale[..., 0]
    else:
        cache[slots] = torch.cat([codes.view(torch.uint8), scale.view(torch.uint8)], -1)


def _load(s, case, x, slots):
    """The fp32 head rows [..., Hkv, D] that the pool of `x` holds at `slots`."""
    got = s[x + "_cache"][slots]
    if case["fmt"] in ACT:
        return got.float()
    if case["fmt"] == "e4m3":
        return got.view(torch.float8_e4m3fn).float() * s[x + "_layer"]
    if case["fmt"] == "int8_side":
        return got.float() * s[x + "_scale"][slots][..., None]
    return got[..., :case["d"]].view(torch.int8).float() * got[..., case["d"]:].contiguous().view(torch.float32)


def _pool_values(s, case):
    """The pool after an append, as the values that it stands for (an E4M3 pool: as E4M3 values)."""
    if case["fmt"] in ACT:
        return {"k": s["k_cache"], "v": s["v_cache"]}
    if case["fmt"] == "e4m3":
        return {"k": s["k_cache"].view(torch.float8_e4m3fn), "v": s["v_cache"].view(torch.float8_e4m3fn)}
    if case["fmt"] == "int8_side":
        return {"k": s["k_cache"] * s["k_scale"][..., None], "v": s["v_cache"] * s["v_scale"][..., None],
                "k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    d = case["d"]
    return {x: s[x + "_cache"][..., :d].view(torch.int8) * s[x + "_cache"][..., d:].view(torch.float32) for x in "kv"}


def _rotate(x, cos, sin, rot, pairs):
    """fp32 rows [T, H, D] rotated by their tokens' angles: each product and the sum rounded to fp32."""
    if pairs:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), x[..., rot:]], -1)
    a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., rot:]], -1)


def _slots_at(table, pos, block):
    return table[..., pos // block].long().clamp(min=0) * block + pos % block


def _paged_slots(s, case):
    pos = s["token_pos"].long()
    return s["block_table"][s["token_seq"].long(), pos // case["block"]].long() * case["block"] + pos % case["block"]


def _plain_append(s, case):
    rot, half = case["rot"], case["rot"] // 2
    pair = torch.arange(half, device="cuda")
    at = s["axis_pos"].long()[torch.tensor(s["pair_axis"], device="cuda")].t()  # [T, pairs]
    cos, sin = s["cos_sin"][at, pair][:, None], s["cos_sin"][at, half + pair][:, None]
    slots = _paged_slots(s, case) if case["block"] else s["slot_mapping"]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, rot, case["pairs"]))
    _store(s, case, "k", slots, _rotate(s["k"].float(), cos, sin, rot, case["pairs"]))
    _store(s, case, "v", slots, s["v"].float())
    return {"q": s["q_out"], **_pool_values(s, case)}


def _plain_read(s, case):
    slots, rot = _paged_slots(s, case), case["rot"]
    k = _load(s, case, "k", slots)
    if rot:
        angle = s["cos_sin"][s["token_pos"].long()][:, None]
        k = _rotate(k, angle[..., :rot // 2], -angle[..., rot // 2:], rot, case["pairs"])
    s["k_out"].copy_(k)
    s["v_out"].copy_(_load(s, case, "v", slots))
    return {"k": s["k_out"], "v": s["v_out"]}


def _scores(s, case, z, dist, masked):
    """Logits [..., G, n] to scores: capped, less the bias of their distance [..., 1, n], -inf where masked."""
    if case["cap"]:
        z = torch.tanh(z / case["cap"]) * case["cap"]
    if case["bias"]:
        z = z - s["slopes"].view(case["hkv"], -1, 1) * dist
    return z.masked_fill(masked, -math.inf)


def _softmax(z):
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = (z - m).exp()
    total = e.sum(-1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), m + total.log()


def _plain_rows(s, case, r0, r1):
    """Rows that each gather their own keys."""
    d, hkv, b = case["d"], case["hkv"], case["block"]
    seen = s["seen"][r0:r1]
    span = max(1, max(e - a for a, e in seen))
    lo = torch.tensor([a for a, _ in seen], device="cuda").clamp(min=0)[:, None]
    pos = lo + torch.arange(span, device="cuda")
    rows = s["block_table"][s["row_seq"][r0:r1].long()]
    at = (pos // b).clamp(max=rows.shape[1] - 1)
    slots = rows.gather(1, at).long().clamp(min=0) * b + pos % b
    end = s["row_end"][r0:r1, None]
    own_pos = (s["row_pos"][r0:r1, None] if s["row_pos"] is not None else end - 1)
    z = s["q"][r0:r1].float().view(r1 - r0, hkv, -1, d) * d ** -0.5 @ _load(s, case, "k", slots).permute(0, 2, 3, 1)
    w, lse = _softmax(_scores(s, case, z, (own_pos - pos).abs()[:, None, None].float(), (pos >= end)[:, None, None]))
    s["out"][r0:r1] = (w @ _load(s, case, "v", slots).transpose(1, 2)).view(r1 - r0, -1, d).to(s["out"].dtype)
    s["lse"][r0:r1] = lse.view(r1 - r0, -1)


def _plain_chunk(s, case, seq, r0, r1):
    """Rows of one sequence against the keys that any of them sees."""
    d, hkv, b, n = case["d"], case["hkv"], case["block"], r1 - r0
    seen = [x for x in s["seen"][r0:r1] if x[0] < x[1]] or [(0, 1)]
    pos = torch.arange(max(0, min(a for a, _ in seen)), max(e for _, e in seen), device="cuda")
    slots = _slots_at(s["block_table"][seq], pos, b)
    end = s["row_end"][r0:r1, None]
    own_pos = s["row_pos"][r0:r1, None] if s["row_pos"] is not None else end - 1
    masked = pos >= end
    if s["row_start"] is not None:
        masked |= pos < s["row_start"][r0:r1, None]
    if case["window"]:
        masked |= pos <= own_pos - case["window"]
    q = s["q"][r0:r1].float().view(n, hkv, -1, d) * d ** -0.5
    z = (q.transpose(0, 1).reshape(hkv, -1, d) @ _load(s, case, "k", slots).permute(1, 2, 0)).view(hkv, n, -1, len(pos))
    w, lse = _softmax(_scores(s, case, z.transpose(0, 1), (own_pos - pos).abs()[:, None, None].float(), masked[:, None, None]))
    o = w.transpose(0, 1).reshape(hkv, -1, len(pos)) @ _load(s, case, "v", slots).transpose(0, 1)
    s["out"][r0:r1] = o.view(hkv, n, -1, d).transpose(0, 1).reshape(n, -1, d).to(s["out"].dtype)
    s["lse"][r0:r1] = lse.reshape(n, -1)


def _plain_attn(s, case):
    if case["rhi"] <= 8:  # single tokens: all rows at once, as far as their keys fit
        R = len(s["seen"])
        span = max(1, max(e - a for a, e in s["seen"]))
        step = max(1, (1 << 30) // (span * case["hkv"] * case["d"]))
        for r in range(0, R, step):
            _plain_rows(s, case, r, min(R, r + step))
    else:
        r = 0
        step = max(1, (1 << 29) // (s["max_row_end"] * case["hq"]))
        for seq, n in enumerate(s["rows_of"]):
            for i in range(0, n, step):
                _plain_chunk(s, case, seq, r + i, r + min(n, i + step))
            r += n
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the library's calls
def _own_append(s, case):
    import quantized_kv_cache_write_gb300 as qkv
    qkv.qkv_append_axes(s["k"], s["v"], FMT_CODE[case["fmt"]], s["k_cache"], s["v_cache"], s["cos_sin"], s["axis_pos"],
                        s["pair_axis"], q=s["q"], q_out=s["q_out"], slot_mapping=s.get("slot_mapping"),
                        token_seq=s.get("token_seq"), token_pos=s.get("token_pos"), block_table=s.get("block_table"),
                        block_size=max(1, case["block"]), k_scale=s.get("k_scale"), v_scale=s.get("v_scale"),
                        k_scale_layer=s["k_layer"], v_scale_layer=s["v_layer"], interleaved=case["pairs"])
    return {"q": s["q_out"], **_pool_values(s, case)}


def _own_attn(s, case):
    import quantized_kv_cache_write_gb300 as qkv
    qkv.qkv_masked_attn(s["q"], FMT_CODE[case["fmt"]], s["k_cache"], s["v_cache"], s["block_table"], s["row_seq"],
                        s["row_end"], case["block"], case["d"] ** -0.5, max_row_end=s["max_row_end"],
                        num_kv_heads=case["hkv"], row_start=s["row_start"], row_pos=s["row_pos"], window=case["window"],
                        softcap=case["cap"], slopes=s["slopes"], k_scale_tok=s.get("k_scale"), v_scale_tok=s.get("v_scale"),
                        k_scale_layer=s["k_layer"], v_scale_layer=s["v_layer"], out=s["out"], lse=s["lse"],
                        workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_read(s, case):
    import quantized_kv_cache_write_gb300 as qkv
    qkv.qkv_read(FMT_CODE[case["fmt"]], s["k_cache"], s["v_cache"], k_out=s["k_out"], v_out=s["v_out"],
                 token_seq=s["token_seq"], token_pos=s["token_pos"], block_table=s["block_table"],
                 block_size=case["block"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), k_scale_layer=s["k_layer"],
                 v_scale_layer=s["v_layer"], cos_sin=s.get("cos_sin"),
                 axis_pos=s["token_pos"][None] if case["rot"] else None, interleaved=case["pairs"])
    return {"k": s["k_out"], "v": s["v_out"]}


def run(state):
    case = state["case"]
    forms = {"append": (_plain_append, _own_append), "attn": (_plain_attn, _own_attn), "read": (_plain_read, _own_read)}
    return forms[case["op"]][bool(own)](state, case)


# ------------------------------------------------------------------ work
def _record_bytes(case):
    """Bytes of one head row of the pool, its per-token scale included."""
    return case["d"] * (2 if case["fmt"] in ACT else 1) + (4 if case["fmt"].startswith("int8") else 0)


def work(case):
    d = case["d"]
    if case["op"] == "append":
        token = 2 * (2 * case["hq"] + 2 * case["hkv"]) * d + 2 * case["hkv"] * _record_bytes(case)
        token += 4 * case["rot"] + 12 + 8  # the angles, three positions, the slot id or its sequence and block
        return {"bytes": case["tokens"] * token, "flops": case["tokens"] * (case["hq"] + case["hkv"]) * case["rot"] * 3}
    if case["op"] == "read":
        n = sum(_spread(case["seqs"], case["lo"], case["hi"]))
        token = 2 * case["hkv"] * (_record_bytes(case) + d * ACT[case["out"]].itemsize) + 8 + 4 * case["rot"]
        return {"bytes": n * token, "flops": n * case["hkv"] * (2 * d + 3 * case["rot"])}
    rows = seen = keys = 0
    for i in range(case["seqs"]):
        masks, _ = _row_masks(case, i)
        spans = [(max(0, a, p + 1 - case["window"]) if case["window"] else a, e) for a, e, p in masks]
        spans = [x for x in spans if x[0] < x[1]]
        rows += len(masks)
        seen += sum(e - a for a, e in spans)
        at = 0  # the keys that any row sees, once; later rows neither start nor end earlier
        for a, e in spans:
            keys += max(0, e - max(a, at))
            at = max(at, e)
    return {"bytes": keys * 2 * case["hkv"] * _record_bytes(case) + rows * case["hq"] * (2 * 2 * d + 4),
            "flops": 4 * seen * case["hq"] * d}


# ------------------------------------------------------------------ 64 bits
def _turned(x, c, w, rot, pairs):
    """64-bit rows [T, H, D] turned by cosines c and sines w [T, pairs], dim by dim."""
    j = torch.arange(rot, device="cuda")
    if pairs:
        mate, pair, sign = j ^ 1, j // 2, torch.where(j % 2 == 0, -1.0, 1.0)
    else:
        mate, pair, sign = (j + rot // 2) % rot, j % (rot // 2), torch.where(j < rot // 2, -1.0, 1.0)
    y = x.clone()
    y[..., :rot] = x[..., :rot] * c[:, pair][:, None] + x[..., mate] * (w[:, pair] * sign.double())[:, None]
    return y


def _exact_slots(s, case):
    p, q, tab = s["token_pos"].tolist(), s["token_seq"].tolist(), s["block_table"].cpu()
    b = case["block"]
    seq, pos = torch.tensor(q), torch.tensor(p)
    return (tab[seq, torch.div(pos, b, rounding_mode="floor")].long() * b + torch.remainder(pos, b)).cuda()


def _exact_append(s, case):
    rot, d = case["rot"], case["d"]
    c, w = [], []
    for i, axis in enumerate(s["pair_axis"]):
        row = s["axis_pos"][axis].long()
        c.append(s["cos_sin"][:, i].double()[row])
        w.append(s["cos_sin"][:, rot // 2 + i].double()[row])
    c, w = torch.stack(c, 1), torch.stack(w, 1)
    slots = _exact_slots(s, case) if case["block"] else s["slot_mapping"]
    shape = (s["k_cache"].shape[0], case["hkv"], d)
    got = {"q": _turned(s["q"].double(), c, w, rot, case["pairs"])}
    for x, rows in (("k", _turned(s["k"].double(), c, w, rot, case["pairs"])), ("v", s["v"].double())):
        pool = torch.zeros(shape, dtype=torch.float64, device="cuda")
        if case["fmt"] in ACT:
            pool[slots] = rows
        elif case["fmt"] == "e4m3":
            pool[slots] = (rows / s[x + "_layer"]).clamp(-448, 448)
        else:
            # by definition the scale is held in fp32, and a code is the integer next to the quotient by it
            # in fp32: 16-bit values often fall on a border exactly
            scale = (rows.abs().amax(-1) / 127).float().double()
            pool[slots] = (rows / scale[..., None]).float().double().round() * scale[..., None]
            if case["fmt"] == "int8_side":
                full = torch.zeros(shape[:2], dtype=torch.float64, device="cuda")
                full[slots] = scale
                got[x + "_scale"] = full
        # an int8 K code next to a rounding border goes by the 32-bit roundings of the rotation
        got[x] = None if x == "k" and case["fmt"].startswith("int8") else pool
    return got


def _exact_rows(s, case, x, slots):
    """64-bit head rows [n, Hkv, D] of the pool of `x`."""
    if case["fmt"] in ACT:
        return s[x + "_cache"][slots].double()
    if case["fmt"] == "e4m3":
        return s[x + "_cache"][slots].view(torch.float8_e4m3fn).double() * s[x + "_layer"]
    if case["fmt"] == "int8_side":
        return s[x + "_cache"][slots].double() * s[x + "_scale"].double()[slots].unsqueeze(-1)
    rec = s[x + "_cache"][slots]
    return rec[..., :case["d"]].view(torch.int8).double() * rec[..., case["d"]:].contiguous().view(torch.float32).double()


def _exact_read(s, case):
    slots, rot = _exact_slots(s, case), case["rot"]
    k = _exact_rows(s, case, "k", slots)
    if rot:
        angle = s["cos_sin"].double().index_select(0, s["token_pos"].long())
        k = _turned(k, angle[:, :rot // 2], -angle[:, rot // 2:], rot, case["pairs"])
    return {"k": k, "v": _exact_rows(s, case, "v", slots)}


def _exact_attn(s, case):
    d, hkv, b, hq = case["d"], case["hkv"], case["block"], case["hq"]
    R = len(s["seen"])
    out = torch.zeros((R, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((R, hq), -math.inf, dtype=torch.float64, device="cuda")
    slope = None if s["slopes"] is None else s["slopes"].double()
    ends = s["row_end"].tolist()
    where = ends if s["row_pos"] is None else [p + 1 for p in s["row_pos"].tolist()]
    first = 0
    for seq, n in enumerate(s["rows_of"]):
        live = [r for r in range(first, first + n) if s["seen"][r][0] < s["seen"][r][1]]
        first += n
        if not live:
            continue
        t = torch.arange(max(0, min(s["seen"][r][0] for r in live)), max(ends[r] for r in live), device="cuda")
        base = int(t[0])
        slots = s["block_table"][seq].long()[torch.div(t, b, rounding_mode="floor")] * b + torch.remainder(t, b)
        k, v = (_exact_rows(s, case, x, slots) for x in "kv")
        step = max(1, (1 << 28) // (len(t) * hq))
        for i in range(0, len(live), step):
            rows = live[i:i + step]
            a, e = max(0, min(s["seen"][r][0] for r in rows)) - base, max(ends[r] for r in rows) - base
            idx = torch.tensor(rows, device="cuda")
            place = torch.tensor([where[r] - 1 for r in rows], device="cuda").view(-1, 1)
            lo = torch.tensor([s["seen"][r][0] for r in rows], device="cuda").view(-1, 1)
            hi = torch.tensor([ends[r] for r in rows], device="cuda").view(-1, 1)
            q = s["q"][idx].double().view(len(rows), hkv, hq // hkv, d)
            z = torch.einsum("rhgd,phd->rhgp", q, k[a:e]) / math.sqrt(d)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if slope is not None:
                z -= slope.view(1, hkv, -1, 1) * (place - t[a:e]).abs().double()[:, None, None]
            hidden = (t[a:e] < lo) | (t[a:e] >= hi)
            z = torch.where(hidden[:, None, None], -math.inf, z)
            total = torch.logsumexp(z, -1)
            o = torch.einsum("rhgp,phd->rhgd", torch.exp(z - total[..., None]), v[a:e])
            out[idx], lse[idx] = o.reshape(len(rows), hq, d), total.reshape(len(rows), hq)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "read": _exact_read}[case["op"]](s, case)
