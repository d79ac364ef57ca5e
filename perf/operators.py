"""What is measured of the operators around a long prompt's cache: rotary positions with several
axes, attention of many query rows over cached states, the attention weight each cached token
received, and the eviction that keeps the tokens with the most of it.

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the calls a
user makes of this package.  Head geometry (40 query heads and 8 KV heads of 128) is that of this
repository's benchmark; the smaller ones are those of its tests.
"""
import math

import torch

own = False

D = 128
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases -------------------------------------------------------------------------------------


def _rope(n, hq, hk, qi, qo, sec, rot=128, turns=False, adjacent=False, packed=False, inverse=False, far=65536):
    return {"op": "rope", "n": n, "hq": hq, "hk": hk, "qi": qi, "qo": qo, "sec": sec, "rot": rot, "turns": turns,
            "adjacent": adjacent, "packed": packed, "inverse": inverse, "far": far}


def _attn(b, n, m, hq, hk, kind, causal=False, ragged=False, empty=False):
    return {"op": "attn", "b": b, "n": n, "m": m, "hq": hq, "hk": hk, "kind": kind, "causal": causal,
            "ragged": ragged, "empty": empty}


def _mass(b, n, m, hq, hk, kind, causal=True, ragged=False, decay=1.0):
    return {"op": "mass", "b": b, "n": n, "m": m, "hq": hq, "hk": hk, "kind": kind, "causal": causal,
            "ragged": ragged, "empty": False, "decay": decay}


def _evict(b, n, keep, hk, kind, sink, recent, ragged=False, ties=False):
    return {"op": "evict", "b": b, "n": n, "keep": keep, "hk": hk, "kind": kind, "sink": sink, "recent": recent,
            "ragged": ragged, "ties": ties}


def listed():
    return [
        # one decode step of 16 sequences: a row each, the query widened to the decode's fp32
        dict(_rope(16, 40, 8, "bf16", "f32", "16,24,24"), name="rope step of 16 sequences"),
        # a video prompt: time, height and width take turns over the channel pairs
        dict(_rope(16384, 40, 8, "bf16", "bf16", "24,20,20", turns=True), name="rope video prompt 16k"),
        # an odd number of image tokens, read out of a packed q|k|v row, part of the channels rotated
        dict(_rope(5003, 10, 2, "f32", "f32", "24,24", rot=96, adjacent=True, packed=True), name="rope packed image rows"),
        # one token of a few short sequences: the latency of a call
        dict(_attn(4, 384, 1, 10, 2, "f16", ragged=True), name="cross one token short"),
        # one token against one long encoder output (or a long 16-bit prompt): the cache is read once
        dict(_attn(1, 65536, 1, 40, 8, "bf16"), name="cross one token 64k"),
        # decoder prompts against encoder states of about 1500 positions, ragged, one request empty
        dict(_attn(8, 1500, 448, 40, 8, "bf16", ragged=True, empty=True), name="cross 448 x 1500 ragged"),
        # the same against encoder states kept in 8 bits
        dict(_attn(4, 4096, 64, 40, 8, "q8_0", ragged=True), name="cross 64 x 4096 q8_0"),
        # the prefill of a whole prompt, causal, with the log-sum-exp the weights need
        dict(_attn(1, 8192, 8192, 40, 8, "f16", causal=True), name="causal prompt 8k"),
        # the last 32 queries of a 64k prompt weigh its tokens
        dict(_mass(1, 65536, 32, 40, 8, "bf16", decay=0.0), name="weights of a window 64k"),
        # every query of a prompt does, on top of what earlier chunks gave
        dict(_mass(2, 4096, 4096, 40, 8, "f16", ragged=True, decay=0.9), name="weights of a prompt 4k"),
        # a short conversation cut to 512 tokens
        dict(_evict(1, 2048, 512, 8, "bf16", 4, 128), name="evict 2k to 512"),
        # a batch of prompts of 4k to 32k tokens, each cut to 4096 (some have no more than that)
        dict(_evict(16, 32768, 4096, 8, "bf16", 4, 512, ragged=True, ties=True), name="evict 16 prompts to 4k"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "mass", "evict"])
    hq, hk = rng.choice([(40, 8), (10, 2), (8, 8), (16, 2), (24, 8), (3, 1)])
    if op == "rope":
        rot = rng.choice([128, 128, 96, 64])
        a = rng.randint(1, rot // 2 - 2)
        b = rng.randint(1, rot // 2 - a - 1)
        sec = rng.choice(["%d" % (rot // 2), "%d,%d" % (a, rot // 2 - a), "%d,%d,%d" % (a, b, rot // 2 - a - b)])
        qi, qo = rng.choice([("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
        return _rope(_log(rng, 1, 16384), hq, hk, qi, qo, sec, rot, rng.random() < 0.5, rng.random() < 0.5,
                     rng.random() < 0.4, rng.random() < 0.3, _log(rng, 64, 1 << 24))
    kind = rng.choice(["bf16", "f16"])
    b = rng.choice([1, 1, 2, 3, 5, 8])
    if op == "evict":
        n = _log(rng, 64, 32768)
        keep = rng.randint(max(1, n // 16), n)
        sink = rng.randint(0, min(16, keep))
        return _evict(b, n, keep, hk, kind, sink, rng.randint(0, min(keep - sink, 1024)), rng.random() < 0.6,
                      rng.random() < 0.5)
    causal = rng.random() < 0.5
    n = _log(rng, 1, 16384)
    m = _log(rng, 1, min(n, 4096) if causal else 2048)
    # the padded scores of the plain form stay within those of the largest listed case
    while b * m * n * hq > 40 * 8192 * 4096:
        m = max(1, m // 2)
    if op == "attn":
        kind = rng.choice(["bf16", "f16", "q8_0"])
        return _attn(b, n, m, hq, hk, kind, causal, b > 1 and rng.random() < 0.6, not causal and b > 1 and rng.random() < 0.3)
    return _mass(b, n, m, hq, hk, kind, causal, b > 1 and rng.random() < 0.6, rng.choice([0.0, 0.5, 1.0]))


def _lens(c):
    """Tokens of each sequence: the longest first, the others down to an eighth of it; an empty one last."""
    b, n = c["b"], c["n"]
    ls = [n - (n - -(-n // 8)) * i // max(1, b - 1) for i in range(b)] if c["ragged"] else [n] * b
    if c.get("empty"):
        ls[-1] = 0
    return ls


def _rows(c):
    """Query tokens of each sequence: the longest sequence has the most; causal ones no more than their tokens."""
    b, m = c["b"], c["m"]
    ms = [max(1, m - m * i // (2 * b)) for i in range(b)] if c["ragged"] else [m] * b
    return [min(x, n) for x, n in zip(ms, _lens(c))] if c["causal"] else ms


def _pairs(c):
    """Visible (query, token) pairs of a head over all sequences."""
    return sum(m * (n - m) + m * (m + 1) // 2 if c["causal"] else m * n for m, n in zip(_rows(c), _lens(c)))


def work(c):
    if c["op"] == "rope":
        size = {"f32": 4, "bf16": 2, "f16": 2}
        n = c["n"]
        pos = 4 * n * (c["sec"].count(",") + 1)
        return {"bytes": pos + n * D * (c["hq"] * (size[c["qi"]] + size[c["qo"]]) + c["hk"] * 4),
                "flops": 3 * n * c["rot"] * (c["hq"] + c["hk"])}
    if c["op"] == "evict":
        n, keep = sum(_lens(c)), sum(min(x, c["keep"]) for x in _lens(c))
        return {"bytes": c["hk"] * (4 * n + 8 * keep + 4 * D * 2 * keep), "flops": c["hk"] * n}
    n, m = sum(_lens(c)), sum(_rows(c))
    row = {"bf16": 2 * D, "f16": 2 * D, "q8_0": D + 8}[c["kind"]]
    if c["op"] == "attn":
        return {"bytes": 2 * row * n * c["hk"] + m * c["hq"] * (4 * D + 4), "flops": 4 * D * c["hq"] * _pairs(c)}
    reads = 0 if c["decay"] == 0.0 else 4
    return {"bytes": row * n * c["hk"] + m * c["hq"] * (2 * D + 4) + n * c["hk"] * (4 + reads),
            "flops": 2 * D * c["hq"] * _pairs(c)}


# ---- inputs ------------------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _states(c, g):
    """Keys and values [b, n, hk, 128]: a few channels of the keys are larger than the others; rows past a
    sequence's end are zero."""
    kind = torch.float16 if c["kind"] == "f16" else torch.bfloat16
    n, lens = c["n"], torch.tensor(_lens(c), device="cuda")
    k = _normal(g, c["b"], n, c["hk"], D)
    k[..., 7] *= 6.0
    k[..., 63] *= 6.0
    v = _normal(g, c["b"], n, c["hk"], D)
    on = torch.arange(n, device="cuda")[None] < lens[:, None]
    # 16-bit values that BF16 and F16 both hold, as a cache takes BF16 rows
    k, v = ((x * on[:, :, None, None]).bfloat16().to(kind) for x in (k, v))
    return k, v, lens, on


def _q8(x):
    """8-bit blocks of 32 channels: an fp16 scale absmax / 127 and the rounded quotients."""
    y = x.float().unflatten(-1, (4, 32))
    d = (y.abs().amax(-1, keepdim=True) / 127.0).half()
    df = d.float()
    return torch.where(df > 0, torch.round(y / torch.where(df > 0, df, 1.0)), 0.0).clamp(-128, 127).to(torch.int8), d


def _axes(c):
    """The axis of each channel pair: the sections one after another, or the axes taking turns while they
    have pairs left."""
    sec = [int(x) for x in c["sec"].split(",")]
    if not c["turns"]:
        return [a for a, s in enumerate(sec) for _ in range(s)]
    left, out = list(sec), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def prepare(c, seed):
    g = _gen(seed)
    s = {"c": c}
    if c["op"] == "rope":
        n, hq, hk = c["n"], c["hq"], c["hk"]
        axes = _axes(c)
        # time runs slowly, height and width inside a frame quickly, all from a far first position
        t = torch.arange(n, device="cuda")
        first = int(torch.randint(0, c["far"], (1,), generator=g, device="cuda"))
        s["pos"] = torch.stack([first + t // 256, first + t % 256 // 16, first + t % 16][: max(axes) + 1]).int()
        if max(axes) == 0:
            s["pos"] = (first + t)[None].int()
        wide = (hq + 2 * hk) * D
        if c["packed"] and c["qi"] == "bf16":
            rows = _normal(g, n, wide).bfloat16()
            s["q"], s["k"] = rows[:, : hq * D].view(n, hq, D), rows[:, hq * D : (hq + hk) * D].view(n, hk, D)
        elif c["packed"]:
            s["q"] = _normal(g, n, wide).to(DT[c["qi"]])[:, : hq * D].view(n, hq, D)
            s["k"] = _normal(g, n, 2 * hk, D).bfloat16()[:, :hk]
        else:
            s["q"], s["k"] = _normal(g, n, hq, D).to(DT[c["qi"]]), _normal(g, n, hk, D).bfloat16()
        s["axis"] = torch.tensor(axes, device="cuda")
        s["freq"] = 1e6 ** (-torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) * 2 / c["rot"])
        if own:
            from bit_kv_cache_17_b200 import kvq

            s["rope"] = kvq.Rope([int(x) for x in c["sec"].split(",")], theta=1e6, rot_dim=c["rot"], turns=c["turns"],
                                 adjacent=c["adjacent"])
        return s
    k, v, lens, on = _states(c, g)
    s["lens"], s["n_list"] = lens, _lens(c)
    if c["op"] == "evict":
        s["k"], s["v"] = k, v
        # few tokens gather most of the weight; with ties, many have had none at all
        mass = torch.exp(2.0 * _normal(g, c["b"], c["hk"], c["n"]))
        if c["ties"]:
            mass = torch.where(mass < 3.0, 0.0, mass)
        s["mass"] = mass
    else:
        rows = _rows(c)
        s["m_list"] = rows
        dt = k.dtype
        s["q"] = _normal(g, sum(rows), c["hq"], D).to(dt)
        m = max(rows)
        grid = torch.arange(m, device="cuda")[None] < torch.tensor(rows, device="cuda")[:, None]
        s["at"] = grid.nonzero(as_tuple=True)  # (sequence, token of it) of each query row
        last = lens[:, None] - torch.tensor(rows, device="cuda")[:, None] + 1 + torch.arange(m, device="cuda")[None]
        s["see"] = (last if c["causal"] else lens[:, None].expand(-1, m)).contiguous()  # tokens a row sees
        s["m"] = m
        if c["kind"] == "q8_0":
            s["k"], s["v"] = _q8(k), _q8(v)
        else:
            s["k"], s["v"] = k, v
        if c["op"] == "mass":
            s["mass"] = torch.exp(_normal(g, c["b"], c["hk"], c["n"])) * on[:, None]
            s["lse"] = _scores(s).logsumexp(-1).movedim(-1, 1).flatten(2)[s["at"]]
    if own:
        from bit_kv_cache_17_b200 import kvq

        f16 = int(c["kind"] == "f16")
        cache = kvq.KVCache(n_seqs=c["b"], n_kv_heads=c["hk"], max_ctx=c["n"], tail=0, tail_f16=f16,
                            type_k="q8_0" if c["kind"] == "q8_0" else "bf16",
                            type_v="q8_0" if c["kind"] == "q8_0" else "bf16")
        s["ids"] = list(range(c["b"]))
        cache.append(0, s["ids"], s["n_list"], k.bfloat16()[on], v.bfloat16()[on])
        s["cache"] = cache
        if c["op"] == "evict":
            s["dst"] = kvq.KVCache(n_seqs=c["b"], n_kv_heads=c["hk"], max_ctx=c["keep"], tail=0, tail_f16=f16,
                                   type_k="bf16", type_v="bf16")
            s["dst"].rows16(0).zero_()
    return s


# ---- plain forms -------------------------------------------------------------------------------


def _plain_rope(s):
    c = s["c"]
    rot, half = c["rot"], c["rot"] // 2
    angle = s["pos"].double()[s["axis"]].T * s["freq"]  # [n, half]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    sin = -sin if c["inverse"] else sin

    def turn(x, to):
        y = x.float()
        r, rest = y[..., :rot], y[..., rot:]
        a, b = (r[..., 0::2], r[..., 1::2]) if c["adjacent"] else (r[..., :half], r[..., half:])
        u, w = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((u, w), -1).flatten(-2) if c["adjacent"] else torch.cat((u, w), -1)
        return torch.cat((r, rest), -1).to(to)

    return {"q": turn(s["q"], DT[c["qo"]]), "k": turn(s["k"], torch.bfloat16)}


def _wide(x):
    return (x[0].float() * x[1].float()).flatten(-2) if isinstance(x, tuple) else x.float()


def _scores(s):
    """Scaled products of padded query rows and tokens [b, hk, g, m, n], -inf where a row sees nothing."""
    c = s["c"]
    b, g = c["b"], c["hq"] // c["hk"]
    q = s["q"].new_zeros(b, s["m"], c["hq"], D, dtype=torch.float32)
    q[s["at"]] = s["q"].float()
    q = q.view(b, s["m"], c["hk"], g, D).permute(0, 2, 3, 1, 4).reshape(b, c["hk"], g * s["m"], D)
    x = (q @ _wide(s["k"]).permute(0, 2, 3, 1)).view(b, c["hk"], g, s["m"], c["n"]).mul_(1 / math.sqrt(D))
    hide = torch.arange(c["n"], device="cuda") >= s["see"][..., None]
    return x.masked_fill_(hide[:, None, None], -torch.inf)


def _plain_attn(s):
    c = s["c"]
    x = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -torch.inf, 0.0, top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ _wide(s["v"]).permute(0, 2, 1, 3)).view(*p.shape[:-1], D)
    o = o / torch.where(total > 0, total, 1.0)
    back = lambda y: y.permute(0, 3, 1, 2, 4).flatten(2, 3)[s["at"]]  # noqa: E731
    return {"out": back(o).to(s["q"].dtype), "lse": back(top + total.log())[..., 0]}


def _plain_mass(s):
    c = s["c"]
    b, g = c["b"], c["hq"] // c["hk"]
    lse = s["lse"].new_full((b, s["m"], c["hq"]), torch.inf)
    lse[s["at"]] = s["lse"]
    x = _scores(s).sub_(lse.view(b, s["m"], c["hk"], g).permute(0, 2, 3, 1)[..., None]).exp_()
    return {"mass": s["mass"] * c["decay"] + x.flatten(2, 3).sum(2)}


def _plain_evict(s):
    c = s["c"]
    b, n, hk, keep = c["b"], c["n"], c["hk"], c["keep"]
    idx, lens = torch.arange(n, device="cuda"), s["lens"][:, None]
    safe = (idx < c["sink"]) | (idx >= lens - c["recent"])
    rank = torch.where(idx < lens, 1 + safe.int(), 0)[:, None].expand(b, hk, n)
    o = s["mass"].sort(dim=-1, descending=True, stable=True).indices
    o = o.gather(-1, rank.gather(-1, o).sort(dim=-1, descending=True, stable=True).indices)[..., :keep]
    kept = o.sort(-1).values
    off = kept >= lens[..., None]
    # a sequence of fewer tokens than the budget keeps them all: the places behind them hold -1
    kept = torch.where(off, n, kept).sort(-1).values
    off = kept >= lens[..., None]
    at = torch.where(off, 0, kept)
    mass = torch.where(off, 0.0, s["mass"].gather(-1, at))
    rows = torch.stack([x.permute(0, 2, 1, 3).gather(2, at[..., None].expand(-1, -1, -1, D)) for x in (s["k"], s["v"])], 2)
    rows = torch.where(off[:, :, None, :, None], torch.zeros((), dtype=rows.dtype, device="cuda"), rows)
    return {"kept": torch.where(off, -1, kept).int(), "mass": mass, "rows": rows}


# ---- the framework's calls -----------------------------------------------------------------------


def _own_rope(s):
    c = s["c"]
    q, k = s["rope"].apply(s["pos"], s["q"], s["k"], q_dtype=DT[c["qo"]], inverse=c["inverse"])
    return {"q": q, "k": k}


def _own_attn(s):
    out, lse = s["cache"].batch_attn(0, s["ids"], s["m_list"], s["q"], causal=s["c"]["causal"], return_lse=True)
    return {"out": out, "lse": lse}


def _own_mass(s):
    c = s["c"]
    mass = torch.zeros_like(s["mass"])
    s["cache"].attn_mass(0, s["ids"], s["m_list"], s["q"], s["lse"], causal=c["causal"], decay=c["decay"],
                         mass_in=s["mass"], mass_out=mass)
    return {"mass": mass}


def _own_evict(s):
    c = s["c"]
    kept, mass = s["cache"].evict(s["dst"], 0, 0, s["ids"], s["ids"], s["mass"], c["keep"], sink=c["sink"],
                                  recent=c["recent"])
    return {"kept": kept, "mass": mass, "rows": s["dst"].rows16(0)}


def run(s):
    op = s["c"]["op"]
    if own:
        return {"rope": _own_rope, "attn": _own_attn, "mass": _own_mass, "evict": _own_evict}[op](s)
    return {"rope": _plain_rope, "attn": _plain_attn, "mass": _plain_mass, "evict": _plain_evict}[op](s)


# ---- the definitions in 64 bits --------------------------------------------------------------------


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rope":
        # each pair as a complex number times exp(i angle)
        rot = c["rot"]
        a = torch.stack([s["pos"][ax].double() * f for ax, f in zip(s["axis"].tolist(), s["freq"].tolist())], 1)
        z = torch.polar(torch.ones_like(a), -a if c["inverse"] else a)[:, None]
        out = {}
        for name in ("q", "k"):
            x = s[name].double().clone()
            first = torch.arange(0, rot, 2) if c["adjacent"] else torch.arange(rot // 2)
            second = first + (1 if c["adjacent"] else rot // 2)
            w = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * z
            x[..., first], x[..., second] = w.real, w.imag
            out[name] = x
        return out
    if c["op"] == "evict":
        import numpy as np

        n, keep = c["n"], c["keep"]
        kept = np.full((c["b"], c["hk"], keep), -1, np.int32)
        mass, m = np.zeros((c["b"], c["hk"], keep)), s["mass"].cpu().double().numpy()
        rows = torch.zeros(c["b"], c["hk"], 2, keep, D, dtype=torch.float64, device="cuda")
        for i, ln in enumerate(s["n_list"]):
            for h in range(c["hk"]):
                must = set(range(min(c["sink"], ln))) | set(range(max(0, ln - c["recent"]), ln))
                rest = [t for t in np.lexsort((np.arange(ln), -m[i, h, :ln])) if t not in must]
                got = sorted(must | set(int(t) for t in rest[: max(0, min(keep, ln) - len(must))]))
                kept[i, h, : len(got)] = got
                mass[i, h, : len(got)] = m[i, h, got]
                at = torch.tensor(got, device="cuda")
                rows[i, h, 0, : len(got)] = s["k"][i, at, h].double()
                rows[i, h, 1, : len(got)] = s["v"][i, at, h].double()
        return {"kept": kept, "mass": mass, "rows": rows}
    # one sequence and head at a time
    hq, g = c["hq"], c["hq"] // c["hk"]
    k, v = s["k"], s["v"]
    if c["kind"] == "q8_0":
        k, v = ((x[0].double() * x[1].double()).flatten(-2) for x in (k, v))
    out = torch.zeros(sum(s["m_list"]), hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(sum(s["m_list"]), hq, dtype=torch.float64, device="cuda")
    mass = s["mass"].double() * c["decay"] if c["op"] == "mass" else None
    row = 0
    for i, (n, m) in enumerate(zip(s["n_list"], s["m_list"])):
        for h in range(hq):
            if n == 0 or m == 0:
                lse[row : row + m, h] = -torch.inf
                continue
            x = torch.einsum("md,nd->mn", s["q"][row : row + m, h].double(), k[i, :n, h // g].double()) * D ** -0.5
            if c["causal"]:
                x += torch.full((m, n), -torch.inf, dtype=torch.float64, device="cuda").triu_(n - m + 1)
            if c["op"] == "mass":
                mass[i, h // g, :n] += torch.exp(x - s["lse"][row : row + m, h].double()[:, None]).sum(0)
                continue
            out[row : row + m, h] = torch.softmax(x, -1) @ v[i, :n, h // g].double()
            lse[row : row + m, h] = torch.logsumexp(x, -1)
        row += m
    return {"mass": mass} if c["op"] == "mass" else {"out": out, "lse": lse}
