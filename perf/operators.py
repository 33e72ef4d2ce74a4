"""What the cache's dense operators are measured on: keys and values appended to the slot pool with
the position rotation applied on the way, and decode attention for a batch that shares a prefix.

`run` computes a case's operator in its plain form (elementary torch operations in 32 bits), or,
where `own` is true, through the library's entry points. `exact` gives the same in 64 bits.
"""

import math

import torch

own = False

POSITIONS = 131072  # rows of the cos / sin table: the longest context of the repository's workloads
FMT_CODE = {"bf16": 0, "int8_side": 1, "int8_inline": 2, "e4m3": 3, "f16": 4}  # qkv_format of qkv.h
ACT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases
def _append(name, T, hq, hkv, d, rot, fmt, act="bf16", pairs=False, block=0, spare=0):
    """`block` 0: tokens go to slot ids; otherwise through a block table. The pool holds the tokens
    of the call and `spare` more."""
    return {"name": name, "op": "append", "tokens": T, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "fmt": fmt,
            "act": act, "pairs": pairs, "block": block, "spare": spare}


def _prefix(name, seqs, per, hq, hkv, d, fmt, prefix, lo, hi, block, act="bf16"):
    """`seqs` sequences of `per` query rows; behind the prefix each has `lo` to `hi` tokens of its own."""
    return {"name": name, "op": "prefix", "seqs": seqs, "per": per, "hq": hq, "hkv": hkv, "d": d, "fmt": fmt,
            "act": act, "prefix": prefix, "lo": lo, "hi": hi, "block": block}


def listed():
    return [
        # one sequence decodes one token: nothing but latency
        _append("append one token", 1, 16, 1, 256, 64, "int8_side", spare=255),
        # a speculative step: 8 sequences with 5 new positions each, through a block table of 16
        _append("append 8 x 5 drafts, e4m3", 40, 16, 1, 256, 64, "e4m3", block=16, spare=600),
        # a prefill chunk of 8192 tokens, the repository's chunked-prefill shape
        _append("append 8192 chunk, int8", 8192, 16, 1, 256, 256, "int8_side"),
        # the largest: a packed prefill of a model with 128-wide heads into an unquantised pool
        _append("append 16384 chunk, bf16", 16384, 32, 8, 128, 128, "bf16", block=64),
        # a mixed catch-up batch of odd length: half activations, inline records, adjacent pairs
        _append("append 1237 mixed, inline", 1237, 16, 2, 128, 96, "int8_inline", act="f16", pairs=True, block=5),
        # two requests behind a short system prompt: latency
        _prefix("prefix, 2 short rows", 2, 1, 16, 1, 256, "int8_side", 200, 1, 40, 16),
        # the long-context speculative step: 8 sequences x 5 positions, 131072 tokens, most of them shared
        _prefix("prefix, 8 x 5 drafts, 131072", 8, 5, 16, 1, 256, "int8_side", 126976, 5, 4096, 16),
        # a serving batch behind one long document, 8 KV heads
        _prefix("prefix, 64 rows, e4m3", 64, 1, 64, 8, 128, "e4m3", 32768, 1, 1024, 64),
        # an unquantised pool, a prefix that ends inside a block, long private parts
        _prefix("prefix, 128 rows, bf16", 128, 1, 32, 4, 128, "bf16", 8191, 16, 2048, 32),
        # odd sizes everywhere: 37 rows, groups of 12, blocks of 7, half activations, rows with nothing of their own
        _prefix("prefix, 37 odd rows, f16", 37, 1, 24, 2, 256, "f16", 1000, 0, 333, 7, act="f16"),
        # nothing shared: plain paged decode over ragged lengths, one of them empty
        _prefix("no prefix, 64 rows, e4m3", 64, 1, 64, 8, 128, "e4m3", 0, 0, 8192, 64),
        # the largest: 256 requests behind 65536 shared tokens, half activations on an int8 pool
        _prefix("prefix, 256 rows, 65536", 256, 1, 16, 1, 256, "int8_side", 65536, 1, 256, 16, act="f16"),
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
    if rng.random() < 0.5:
        top = 16384 * 48 * 128 // ((hq + 2 * hkv) * d)
        c = _append("", _log(rng, 1, min(16384, top)), hq, hkv, d, 16 * rng.randint(1, d // 16), fmt, act,
                    rng.random() < 0.5, rng.choice([0, block]), rng.choice([0, 17, 300]))
    else:
        per = rng.choice([1, 1, 1, 2, 5])
        seqs = _log(rng, 1, 256 // per)
        prefix = rng.choice([0, _log(rng, 1, 131072), _log(rng, 1, 131072), _log(rng, 1, 131072)])
        prefix = min(prefix, 256 * 16 * 65536 * 256 // (seqs * per * hq * d))
        hi = _log(rng, per, max(per, min(8192, 64 * 4096 * 8 * 128 // (seqs * per * hkv * d))))
        c = _prefix("", seqs, per, hq, hkv, d, fmt, prefix, rng.choice([per, max(per, hi // 2)]), hi, block, act)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _own_lengths(case):
    """Tokens of its own that each sequence has behind the prefix: evenly spread from lo to hi."""
    n = case["seqs"]
    return [case["lo"] + (case["hi"] - case["lo"]) * i // max(1, n - 1) for i in range(n)]


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


def _prepare_append(case, gen):
    T, d = case["tokens"], case["d"]
    act = ACT[case["act"]]
    # q, k and v are slices of the packed projection's output, as a model has them
    packed = torch.cat([torch.randn((T, case["hq"], d), device="cuda", generator=gen),
                        _tokens(T, case, gen), _tokens(T, case, gen)], 1).to(act)
    s = {"q": packed[:, :case["hq"]], "k": packed[:, case["hq"]:case["hq"] + case["hkv"]],
         "v": packed[:, case["hq"] + case["hkv"]:], "q_out": torch.zeros((T, case["hq"], d), dtype=act, device="cuda")}
    half = case["rot"] // 2
    freq = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
    angle = torch.arange(POSITIONS, dtype=torch.float64, device="cuda")[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    slots = T + case["spare"]
    if case["block"]:  # sequences of up to 4096 new tokens that start anywhere in the context
        b = case["block"]
        per = min(T, 5 if T <= 64 else 4096)
        seqs = -(-T // per)
        t = torch.arange(T, device="cuda")
        s["token_seq"] = (t // per).int()
        start = torch.randint(0, POSITIONS - per, (seqs,), device="cuda", generator=gen)
        s["token_pos"] = (start[t // per] + t % per).int()
        wide = -(-POSITIONS // b)
        need = per // b + 2  # blocks that a sequence's new tokens may touch
        slots = seqs * need * b + case["spare"]
        ids = torch.randperm(seqs * need, device="cuda", generator=gen).int()
        table = torch.full((seqs, wide), -1, dtype=torch.int32, device="cuda")
        at = (start // b)[:, None] + torch.arange(need, device="cuda")
        ok = at < wide
        table[torch.arange(seqs, device="cuda")[:, None].expand_as(at)[ok], at[ok]] = ids.view(seqs, need)[ok]
        s["block_table"] = table
    else:
        s["token_pos"] = torch.randint(0, POSITIONS, (T,), device="cuda", generator=gen).int()
        s["slot_mapping"] = torch.randperm(slots, device="cuda", generator=gen)[:T]
    return s | _empty_pool(slots, case)


def _prepare_prefix(case, gen):
    d, b, P = case["d"], case["block"], case["prefix"]
    order = torch.randperm(case["seqs"], generator=gen, device="cuda").tolist()
    lengths = _own_lengths(case)
    total = [P + lengths[i] for i in order]
    wide = max(1, -(-max(total) // b))
    shared = -(-P // b)
    private = [max(0, -(-n // b) - P // b) for n in total]  # blocks of its own: those that reach past the prefix
    ids = torch.randperm(shared + sum(private), device="cuda", generator=gen).int()
    s = {"prefix_blocks": ids[:shared].clone(), "prefix_len": P, "max_row_len": max(total)}
    table = torch.full((case["seqs"], wide), -1, dtype=torch.int32, device="cuda")
    if P:
        table[:, :P // b] = ids[:P // b]
    at = shared
    for i, n in enumerate(private):
        table[i, P // b:P // b + n] = ids[at:at + n]
        at += n
    s["block_table"] = table
    lens = torch.tensor(total, dtype=torch.int32, device="cuda")
    per = case["per"]
    s["row_seq"] = torch.arange(case["seqs"], device="cuda").repeat_interleave(per).int()
    back = torch.arange(per - 1, -1, -1, device="cuda").repeat(case["seqs"])  # a row does not see the positions after it
    s["row_len"] = (lens[s["row_seq"].long()] - back).int()
    rows = case["seqs"] * per
    act = ACT[case["act"]]
    s["q"] = torch.randn((rows, case["hq"], d), device="cuda", generator=gen).to(act)
    s["out"] = torch.zeros((rows, case["hq"], d), dtype=act, device="cuda")
    s["lse"] = torch.zeros((rows, case["hq"]), dtype=torch.float32, device="cuda")
    s["workspace"] = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    s |= _empty_pool(len(ids) * b, case)
    for x in "kv":
        _store(s, case, x, torch.arange(len(ids) * b, device="cuda"), _tokens(len(ids) * b, case, gen).to(act).float())
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = _prepare_append(case, gen) if case["op"] == "append" else _prepare_prefix(case, gen)
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


def _slots_of_tokens(s, case):
    if not case["block"]:
        return s["slot_mapping"]
    pos = s["token_pos"].long()
    return s["block_table"][s["token_seq"].long(), pos // case["block"]].long() * case["block"] + pos % case["block"]


def _plain_append(s, case):
    rot = case["rot"]
    angle = s["cos_sin"][s["token_pos"].long()][:, None]
    cos, sin = angle[..., :rot // 2], angle[..., rot // 2:]
    slots = _slots_of_tokens(s, case)
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, rot, case["pairs"]))
    _store(s, case, "k", slots, _rotate(s["k"].float(), cos, sin, rot, case["pairs"]))
    _store(s, case, "v", slots, s["v"].float())
    return {"q": s["q_out"], **_pool_values(s, case)}


def _slots_at(table, pos, block):
    return table[..., pos // block].long().clamp(min=0) * block + pos % block


def _plain_prefix(s, case):
    d, hkv, b, P = case["d"], case["hkv"], case["block"], case["prefix"]
    rows, g = case["seqs"] * case["per"], case["hq"] // hkv
    q = s["q"].float().view(rows, hkv, g, d) * d ** -0.5
    own_pos = P + torch.arange(s["max_row_len"] - P, device="cuda")
    # the shared part, computed once: [Hkv, rows * G, P]
    slots = _slots_at(s["prefix_blocks"], torch.arange(P, device="cuda"), b)
    k, v = _load(s, case, "k", slots), _load(s, case, "v", slots)
    sp = (q.transpose(0, 1).reshape(hkv, rows * g, d) @ k.permute(1, 2, 0)).view(hkv, rows, g, P).transpose(0, 1)
    sp = sp.masked_fill((s["row_len"] <= 0)[:, None, None, None], -math.inf)
    # each row's own part, padded to the longest: [rows, Hkv, G, L]
    own_slots = _slots_at(s["block_table"][s["row_seq"].long()], own_pos, b)
    ko, vo = _load(s, case, "k", own_slots), _load(s, case, "v", own_slots)
    so = q @ ko.permute(0, 2, 3, 1)
    so = so.masked_fill((own_pos >= s["row_len"][:, None])[:, None, None], -math.inf)
    both = torch.cat([sp, so], -1)
    m = both.amax(-1, keepdim=True) if both.shape[-1] else torch.full((rows, hkv, g, 1), -math.inf, device="cuda")
    m = torch.where(m == -math.inf, 0.0, m)
    e = (both - m).exp()
    total = e.sum(-1, keepdim=True)
    o = (e[..., :P].transpose(0, 1).reshape(hkv, rows * g, P) @ v.transpose(0, 1)).view(hkv, rows, g, d).transpose(0, 1)
    o = o + e[..., P:] @ vo.transpose(1, 2)
    o = o / torch.where(total > 0, total, 1.0)
    s["out"].copy_(o.reshape(rows, hkv * g, d))
    s["lse"].copy_((m + total.log()).view(rows, hkv * g))
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ the library's calls
def _own_append(s, case):
    import quantized_kv_cache_write_gb300 as qkv
    qkv.qkv_append_rope(s["k"], s["v"], FMT_CODE[case["fmt"]], s["k_cache"], s["v_cache"], s["cos_sin"], s["token_pos"],
                        q=s["q"], q_out=s["q_out"], slot_mapping=s.get("slot_mapping"), token_seq=s.get("token_seq"),
                        block_table=s.get("block_table"), block_size=case["block"], k_scale=s.get("k_scale"),
                        v_scale=s.get("v_scale"), k_scale_layer=s["k_layer"], v_scale_layer=s["v_layer"],
                        interleaved=case["pairs"])
    return {"q": s["q_out"], **_pool_values(s, case)}


def _own_prefix(s, case):
    import quantized_kv_cache_write_gb300 as qkv
    qkv.qkv_prefix_attn(s["q"], FMT_CODE[case["fmt"]], s["k_cache"], s["v_cache"], s["block_table"], s["row_seq"],
                        s["row_len"], case["block"], case["d"] ** -0.5, prefix_blocks=s["prefix_blocks"],
                        prefix_len=s["prefix_len"], max_row_len=s["max_row_len"], num_kv_heads=case["hkv"],
                        k_scale_tok=s.get("k_scale"), v_scale_tok=s.get("v_scale"), k_scale_layer=s["k_layer"],
                        v_scale_layer=s["v_layer"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    case = state["case"]
    if case["op"] == "append":
        return _own_append(state, case) if own else _plain_append(state, case)
    return _own_prefix(state, case) if own else _plain_prefix(state, case)


# ------------------------------------------------------------------ work
def _record_bytes(case):
    """Bytes of one head row of the pool, its per-token scale included."""
    return case["d"] * (2 if case["fmt"] in ACT else 1) + (4 if case["fmt"].startswith("int8") else 0)


def work(case):
    d = case["d"]
    if case["op"] == "append":
        T = case["tokens"]
        token = 2 * (2 * case["hq"] + 2 * case["hkv"]) * d + 2 * case["hkv"] * _record_bytes(case)
        token += 4 * case["rot"] + 4 + 8  # the angles, the position, the slot id or its sequence and block
        return {"bytes": T * token, "flops": T * (case["hq"] + case["hkv"]) * case["rot"] * 3}
    own_tokens = _own_lengths(case)
    rows = case["seqs"] * case["per"]
    seen = sum(max(0, case["prefix"] + n - i) for n in own_tokens for i in range(case["per"]))  # keys of all rows
    return {"bytes": (case["prefix"] + sum(own_tokens)) * 2 * case["hkv"] * _record_bytes(case)
            + rows * case["hq"] * (2 * 2 * d + 4),
            "flops": 4 * seen * case["hq"] * d}


# ------------------------------------------------------------------ 64 bits
def _exact_append(s, case):
    rot, d, T = case["rot"], case["d"], case["tokens"]
    j = torch.arange(rot, device="cuda")
    if case["pairs"]:
        mate, freq, sign = j ^ 1, j // 2, torch.where(j % 2 == 0, -1.0, 1.0)
    else:
        mate, freq, sign = (j + rot // 2) % rot, j % (rot // 2), torch.where(j < rot // 2, -1.0, 1.0)
    tab = s["cos_sin"].double().index_select(0, s["token_pos"].long())
    c, w = tab[:, freq], tab[:, rot // 2 + freq] * sign.double()

    def turned(x):
        x = x.double()
        y = x.clone()
        y[..., :rot] = x[..., :rot] * c[:, None] + x[..., mate] * w[:, None]
        return y

    if case["block"]:
        p = s["token_pos"].tolist()
        tq = s["token_seq"].tolist()
        tab_b = s["block_table"].cpu()
        slots = torch.tensor([int(tab_b[a, x // case["block"]]) * case["block"] + x % case["block"] for a, x in zip(tq, p)])
    else:
        slots = s["slot_mapping"].cpu()
    slots = slots.cuda()
    shape = (s["k_cache"].shape[0], case["hkv"], d)
    got = {"q": turned(s["q"])}
    for x, rows in (("k", turned(s["k"])), ("v", s["v"].double())):
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


def _exact_prefix(s, case):
    d, hkv, b, P = case["d"], case["hkv"], case["block"], case["prefix"]
    g = case["hq"] // hkv

    def rows_of(x, slots):
        if case["fmt"] in ACT:
            return s[x + "_cache"][slots].double()
        if case["fmt"] == "e4m3":
            return s[x + "_cache"][slots].view(torch.float8_e4m3fn).double() * s[x + "_layer"]
        if case["fmt"] == "int8_side":
            return s[x + "_cache"][slots].double() * s[x + "_scale"].double()[slots].unsqueeze(-1)
        rec = s[x + "_cache"][slots]
        return rec[..., :d].view(torch.int8).double() * rec[..., d:].contiguous().view(torch.float32).double()

    t = torch.arange(P, device="cuda")
    shared = s["prefix_blocks"].long()[t // b] * b + t % b
    kp, vp = (rows_of(x, shared).transpose(0, 1) for x in "kv")  # [Hkv, P, D]
    outs, lses = [], []
    for r, (seq, n) in enumerate(zip(s["row_seq"].tolist(), s["row_len"].tolist())):
        q = s["q"][r].double().view(hkv, g, d)
        if n <= 0:
            outs.append(torch.zeros((hkv * g, d), dtype=torch.float64, device="cuda"))
            lses.append(torch.full((hkv * g,), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        t = torch.arange(P, n, device="cuda")
        mine = s["block_table"][seq].long()[t // b] * b + t % b
        ko, vo = (rows_of(x, mine).transpose(0, 1) for x in "kv")
        z = torch.cat([torch.einsum("hgd,hpd->hgp", q, kp), torch.einsum("hgd,hpd->hgp", q, ko)], 2) / math.sqrt(d)
        lse = torch.logsumexp(z, 2)
        w = torch.exp(z - lse[..., None])
        outs.append((w[..., :P] @ vp + w[..., P:] @ vo).reshape(hkv * g, d))
        lses.append(lse.reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s, case) if case["op"] == "append" else _exact_prefix(s, case)
