"""Measured cases of the position rotation and the paged cache: rotating queries and keys (forward and
gradient), appending tokens to a paged cache, and decoding one token per sequence from it.

Every case is run in two ways.  With ``own`` false it runs the plain form below, written with elementary
torch operations in float32 (float64 for the rotation angles and the gate sums); with ``own`` true it
makes the calls of ``gated_softmax_attention_fp32_b200.fixattn``.
"""
import math
import random

import torch

own = False

# Rotation base of the synthetic models, and the gate logits' distribution (g = logsigmoid(x), x ~
# N(GATE_MEAN, 1)): slow forgetting, as in the long-context workloads of this repository.
BASE = 10000.0
GATE_MEAN = 5.0
EPS = 1e-6


# ------------------------------------------------------------------ cases
def _rotary(name, mode, lens, Hq, Hkv, D, rot, interleaved, packed, fused, positions):
    c = {"op": "rotary", "mode": mode, "lens": lens, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
         "interleaved": interleaved, "packed": packed, "fused": fused, "positions": positions}
    return {"name": name, **c} if name else c


def _append(name, B, T, lo, hi, pick, pad, Hq, Hkv, Dk, Dv, page, scalar, rot, interleaved, packed, keys):
    c = {"op": "append", "B": B, "T": T, "lo": lo, "hi": hi, "pick": pick, "pad": pad, "Hq": Hq, "Hkv": Hkv,
         "Dk": Dk, "Dv": Dv, "page": page, "scalar": scalar, "rot": rot, "interleaved": interleaved,
         "packed": packed, "keys": keys}
    return {"name": name, **c} if name else c


def _decode(name, B, lo, hi, pick, Hq, Hkv, Dk, Dv, page, scalar, norm, gate, f32):
    c = {"op": "decode", "B": B, "lo": lo, "hi": hi, "pick": pick, "Hq": Hq, "Hkv": Hkv, "Dk": Dk, "Dv": Dv,
         "page": page, "scalar": scalar, "norm": norm, "gate": gate, "f32": f32}
    return {"name": name, **c} if name else c


def listed():
    return [
        # a training step's rotation and its gradient at the quick-start shape (B2 T2048 Hq8 Hkv4 D128)
        _rotary("rotary train B2 T2048", "train", "2048,2048", 8, 4, 128, 128, False, False, False, False),
        # the same on packed sequences, q and k being views of one fused projection's output
        _rotary("rotary train packed 16384", "train", "5211,128,7013,1,4031", 16, 4, 128, 128, False, True, True,
                False),
        # a short prompt of a small model at given far positions, half of each head rotated, interleaved pairs
        _rotary("rotary small", "infer", "33", 4, 2, 64, 32, True, False, False, True),
        # one sequence's next token, far into its context
        _append("append one token", 1, 1, 32767, 32767, 1, 0, 32, 8, 128, 128, 64, False, 128, False, False, False),
        # a decode batch of a fixed (graph-shaped) size, three of its rows being padding
        _append("append batch step", 96, 1, 1, 2000, 2, 3, 32, 8, 128, 128, 64, False, 128, False, False, False),
        # the prompts of new sequences, packed; rotated keys are returned for the prompt's attention
        _append("append prompts", 5, 0, 130, 6500, 3, 0, 16, 4, 128, 128, 16, False, 128, False, True, True),
        # a few tokens per sequence with a scalar gate and no rotation, odd page size
        _append("append few, scalar gate", 7, 5, 5, 700, 4, 0, 16, 4, 64, 64, 24, True, 0, False, False, False),
        # one sequence, short: latency alone
        _decode("decode one short", 1, 257, 257, 1, 32, 8, 128, 128, 64, False, True, False, False),
        # one sequence, long context
        _decode("decode one long", 1, 131071, 131071, 1, 32, 8, 128, 128, 64, False, True, True, False),
        # a serving batch of very unequal lengths
        _decode("decode ragged batch", 64, 1, 8191, 5, 32, 8, 128, 128, 64, False, True, False, False),
        # scalar gate without the norm, output gate, float32 output, odd page size
        _decode("decode scalar f32", 24, 300, 16000, 6, 16, 2, 64, 64, 24, True, False, True, True),
        # many short sequences, 16 query heads per kv head
        _decode("decode many short", 256, 90, 900, 7, 32, 2, 128, 128, 16, False, True, False, False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "append", "append", "decode", "decode", "decode"))
    Hkv = rng.choice((1, 2, 4, 8))
    D = rng.choice((64, 128, 128))
    pick = rng.randrange(1, 1 << 20)
    if op == "rotary":
        Hq = Hkv * rng.choice((1, 2, 4))
        packed = rng.random() < 0.5
        total = _log_int(rng, 16, 20000)
        if packed:
            cuts = sorted(rng.randrange(total + 1) for _ in range(rng.randrange(1, 8)))
            lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        else:
            lens = [max(1, total // 4)] * rng.randrange(1, 5)
        return _rotary(None, rng.choice(("train", "infer")), ",".join(map(str, lens)), Hq, Hkv, D,
                       rng.choice((D, D, D // 2, 16)), rng.random() < 0.3, packed, rng.random() < 0.5,
                       rng.random() < 0.3)
    page = rng.choice((1, 16, 24, 32, 64, 100, 128))
    scalar = rng.random() < 0.3
    if op == "append":
        Hq = Hkv * rng.choice((1, 2, 4, 8))
        rot = rng.choice((D, D, D // 2, 0))
        if rng.random() < 0.4:
            hi = _log_int(rng, 200, 4000)
            return _append(None, rng.randrange(1, 9), 0, max(1, hi // 20), hi, pick, 0, Hq, Hkv, D, D, page, scalar,
                           rot, rng.random() < 0.3, True, rot > 0 and rng.random() < 0.5)
        T, B = rng.choice((1, 1, 1, 2, 7)), _log_int(rng, 1, 128)
        hi = _log_int(rng, 20, 2000)
        return _append(None, B, T, T, T + hi, pick, min(B - 1, rng.randrange(4)), Hq, Hkv, D, D, page, scalar, rot,
                       rng.random() < 0.3, False, False)
    Dv = rng.choice((D, D, 64))
    hi = _log_int(rng, 64, 100000)
    B = max(1, min(256, _log_int(rng, 1, max(2, 2000000 // (hi * Hkv)))))
    return _decode(None, B, max(1, hi // rng.choice((1, 2, 50))), hi, pick, Hkv * rng.choice((1, 2, 4, 5, 8, 16)), Hkv,
                   D, Dv, page, scalar, rng.random() < 0.7, rng.random() < 0.4, rng.random() < 0.4)


def _lengths(case):
    """The sequences' lengths in the cache, spread over [lo, hi] in their logarithm; they go by the case alone."""
    r = random.Random(case["pick"])
    lens = [_log_int(r, case["lo"], case["hi"]) for _ in range(case["B"])]
    for i in range(case.get("pad", 0)):
        lens[-1 - i] = 0
    return lens


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _bf16(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16)


def _gates(gen, *shape):
    return torch.nn.functional.logsigmoid(_randn(gen, *shape) + GATE_MEAN)


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return torch.tensor(cu, dtype=torch.int64, device="cuda")


def _inv_freq(rot):
    i = torch.arange(0, rot, 2, dtype=torch.float64, device="cuda")
    return (BASE ** (-i / rot)).float()


def _pages(gen, case, lens):
    """Pages in a random order, each sequence's taken from them; entries that no token needs are -1."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    total = sum(need) + 3
    order = torch.randperm(total, generator=gen, device="cuda").int()
    table = torch.full((len(lens), max(max(need), 1) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    Hkv, Dv = case["Hkv"], case["Dv"]
    k = _bf16(gen, total, page, Hkv, case["Dk"])
    v = _bf16(gen, total, page, Hkv, Dv)
    g = _gates(gen, total, page, Hkv) if case["scalar"] else _gates(gen, total, page, Hkv, Dv)
    return k, v, g, table


def prepare(case, seed):
    gen = _gen(seed)
    s = {"case": case}
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rotary":
        lens = [int(x) for x in case["lens"].split(",")]
        B, T = (1, sum(lens)) if case["packed"] else (len(lens), lens[0])
        D = case["D"]
        if case["fused"]:
            qkv = _bf16(gen, B, T, Hq + 2 * Hkv, D)
            s["q"], s["k"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = _bf16(gen, B, T, Hq, D), _bf16(gen, B, T, Hkv, D)
        if case["mode"] == "train":
            s["dq"], s["dk"] = _bf16(gen, B, T, Hq, D), _bf16(gen, B, T, Hkv, D)
        s["inv_freq"] = _inv_freq(case["rot"])
        s["cu"] = _cu(lens) if case["packed"] else None
        s["positions"] = (torch.randint(0, 200000, (B, T), generator=gen, device="cuda", dtype=torch.int32)
                          if case["positions"] else None)
        return s
    lens = _lengths(case)
    s["k_pages"], s["v_pages"], s["g_pages"], s["table"] = _pages(gen, case, lens)
    s["seqlens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    Dk, Dv, B = case["Dk"], case["Dv"], case["B"]
    if case["op"] == "append":
        n, T = (1, sum(lens)) if case["packed"] else (B, case["T"])
        s["cu"] = _cu(lens) if case["packed"] else None
        s["q"] = _bf16(gen, n, T, Hq, Dk) if case["rot"] else None
        s["k"], s["v"] = _bf16(gen, n, T, Hkv, Dk), _bf16(gen, n, T, Hkv, Dv)
        s["g"] = _gates(gen, n, T, Hkv) if case["scalar"] else _gates(gen, n, T, Hkv, Dv)
        s["inv_freq"] = _inv_freq(case["rot"]) if case["rot"] else None
        return s
    s["q"] = _bf16(gen, B, Hq, Dk)
    s["w"] = (1 + 0.1 * _randn(gen, Dv)).bfloat16() if case["norm"] else None
    s["z"] = _bf16(gen, B, Hq, Dv) if case["gate"] else None
    return s


# ------------------------------------------------------------------ plain forms
def _angles(positions, inv_freq):
    """cos and sin of position x frequency: the product in float64, where far positions need it."""
    a = positions.double()[..., None] * inv_freq.double()
    return a.cos().float(), a.sin().float()


def _rotate(x, cos, sin, interleaved):
    """Rotates the pairs of the first 2 * cos.shape[-1] channels of x [B,T,H,D]; bf16 in, bf16 out."""
    half = cos.shape[-1]
    f = x[..., :2 * half].float()
    a, b = (f[..., 0::2], f[..., 1::2]) if interleaved else (f[..., :half], f[..., half:])
    c, s = cos[:, :, None], sin[:, :, None]
    ra, rb = a * c - b * s, a * s + b * c
    r = torch.stack((ra, rb), -1).flatten(-2) if interleaved else torch.cat((ra, rb), -1)
    return torch.cat((r.to(x.dtype), x[..., 2 * half:]), -1)


def _new_positions(s):
    """(position, sequence) of every new token of an append or a rotation; padding has a negative position."""
    x = s["k"]
    B, T = x.shape[:2]
    if s["cu"] is not None:
        at = torch.arange(T, device=x.device)
        seq = torch.searchsorted(s["cu"][1:], at, right=True)
        return (at - s["cu"][seq])[None], seq[None]
    seq = torch.arange(B, device=x.device)[:, None].expand(B, T)
    pos = torch.arange(T, device=x.device)[None].expand(B, T)
    if "seqlens" in s:
        pos = pos + (s["seqlens"].long()[:, None] - T)
    return pos, seq


def _plain_rotary(s):
    case = s["case"]
    pos = s["positions"] if s["positions"] is not None else _new_positions(s)[0]
    cos, sin = _angles(pos, s["inv_freq"])
    out = {x: _rotate(s[x], cos, sin, case["interleaved"]) for x in ("q", "k")}
    if case["mode"] == "train":  # the gradient of a rotation is the rotation back
        out |= {x: _rotate(s[x], cos, -sin, case["interleaved"]) for x in ("dq", "dk")}
    return out


def _plain_append(s):
    case, page = s["case"], s["case"]["page"]
    pos, seq = _new_positions(s)
    k, out = s["k"], {}
    if case["rot"]:
        cos, sin = _angles(pos.clamp(min=0), s["inv_freq"])
        k = _rotate(k, cos, sin, case["interleaved"])
        out["q"] = _rotate(s["q"], cos, sin, case["interleaved"])
        if case["keys"]:
            out["k"] = k
    at = pos.clamp(min=0)
    row = s["table"][seq, at // page].long() * page + at % page
    keep = pos >= 0
    row = row[keep]
    for name, x in (("k_pages", k), ("v_pages", s["v"]), ("g_pages", s["g"])):
        s[name].view(-1, *s[name].shape[2:])[row] = x[keep]
        out[name] = s[name]
    return out


def _plain_decode(s):
    case, page = s["case"], s["case"]["page"]
    B, Hq, Hkv, Dk, Dv = (case[x] for x in ("B", "Hq", "Hkv", "Dk", "Dv"))
    lens = s["seqlens"].long()
    at = torch.arange(case["hi"], device=lens.device)
    live = at[None] < lens[:, None]                                   # [B, L]
    row = s["table"][:, (at // page).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0) * page + at % page
    k = s["k_pages"].view(-1, Hkv, Dk)[row].float()                   # [B, L, Hkv, Dk]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, Dk)
    logits = (q @ k.permute(0, 2, 3, 1)) * Dk ** -0.5                 # [B, Hkv, grp, L]
    del k
    logits = logits.masked_fill(~live[:, None, None], -math.inf)
    p = (logits - logits.amax(-1, keepdim=True)).exp()
    den = p.sum(-1, keepdim=True)
    g = s["g_pages"].view(-1, *s["g_pages"].shape[2:])[row].double()
    if case["scalar"]:
        g = g[..., None]
    g = g.masked_fill(~live[:, :, None, None], 0.0).cumsum(1)
    decay = (g[:, -1:] - g).exp().float()                             # gates after each token
    del g
    v = s["v_pages"].view(-1, Hkv, Dv)[row].float().masked_fill(~live[:, :, None, None], 0.0)
    o = p @ (decay * v).permute(0, 2, 1, 3)                           # [B, Hkv, grp, Dv]
    if case["norm"]:
        y = o * (o.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["w"].float()
    else:
        y = o / den
    y = y.reshape(B, Hq, Dv)
    if s["z"] is not None:
        z = s["z"].float()
        y = y * (z / (1 + (-z).exp()))
    return y if case["f32"] else y.bfloat16()


def _own(s):
    from gated_softmax_attention_fp32_b200 import fixattn
    case = s["case"]
    if case["op"] == "rotary":
        if case["mode"] == "train":
            q, k = s["q"].detach().requires_grad_(True), s["k"].detach().requires_grad_(True)
            qr, kr = fixattn.fix_rotary(q, k, s["inv_freq"], cu_seqlens=s["cu"], positions=s["positions"],
                                        interleaved=case["interleaved"])
            dq, dk = torch.autograd.grad((qr, kr), (q, k), (s["dq"], s["dk"]))
            return {"q": qr.detach(), "k": kr.detach(), "dq": dq, "dk": dk}
        q, k = fixattn.fix_attn_rotary(s["q"], s["k"], s["inv_freq"], cu_seqlens=s["cu"],
                                       positions=s["positions"], interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if case["op"] == "append":
        q, k = fixattn.fix_attn_append_paged(
            s["k"], s["v"], s["g"], s["k_pages"], s["v_pages"], s["g_pages"], s["table"], s["seqlens"],
            cu_seqlens=s["cu"], q=s["q"], inv_freq=s["inv_freq"], interleaved=case["interleaved"],
            return_k=case["keys"])
        out = {x: s[x] for x in ("k_pages", "v_pages", "g_pages")}
        if q is not None:
            out["q"] = q
        if k is not None:
            out["k"] = k
        return out
    return fixattn.fix_attn_decode_paged(
        s["q"], s["k_pages"], s["v_pages"], s["g_pages"], s["table"], s["seqlens"], s["w"], eps=EPS,
        y_dtype=torch.float32 if case["f32"] else torch.bfloat16, o_gate=s["z"], o_norm=case["norm"])


def run(state):
    if own:
        return _own(state)
    return {"rotary": _plain_rotary, "append": _plain_append, "decode": _plain_decode}[state["case"]["op"]](state)


# ------------------------------------------------------------------ floors
def work(case):
    Hq, Hkv = case["Hq"], case["Hkv"]
    if case["op"] == "rotary":
        lens = [int(x) for x in case["lens"].split(",")]
        passes = 2 if case["mode"] == "train" else 1
        vals = sum(lens) * (Hq + Hkv) * passes
        return {"bytes": 2 * 2 * vals * case["D"] + 4 * passes * (sum(lens) if case["positions"] else 0),
                "flops": 3 * vals * case["rot"]}
    lens = _lengths(case)
    Dk, Dv = case["Dk"], case["Dv"]
    row = Hkv * (2 * Dk + 2 * Dv + (4 if case["scalar"] else 4 * Dv))  # bytes of one cached token
    if case["op"] == "append":
        new = sum(lens) if case["packed"] else case["B"] * case["T"]
        kept = sum(min(n, case["T"]) for n in lens) if not case["packed"] else new
        rotated = new * 4 * Hq * Dk if case["rot"] else 0
        keys = new * 2 * Hkv * Dk if case["keys"] else 0
        return {"bytes": 2 * row * kept + rotated + keys, "flops": 3 * new * (Hq + Hkv) * case["rot"] + 1}
    read = row * sum(lens) + 4 * sum(-(-n // case["page"]) for n in lens) + 4 * len(lens)
    small = case["B"] * Hq * (2 * Dk + Dv * ((4 if case["f32"] else 2) + (2 if case["gate"] else 0)))
    return {"bytes": read + small, "flops": 2 * Hq * sum(lens) * (Dk + Dv)}


# ------------------------------------------------------------------ exact values
def _turned(x, pos, inv_freq, interleaved, back=False):
    """The rotation as a product of complex numbers, in float64."""
    n = 2 * inv_freq.numel()
    a = pos.double()[..., None, None] * inv_freq.double()
    if back:
        a = -a
    unit = torch.complex(a.cos(), a.sin())
    d = x.double()
    head = d[..., :n]
    if interleaved:
        c = torch.view_as_complex(head.unflatten(-1, (n // 2, 2)).contiguous()) * unit
        r = torch.view_as_real(c).flatten(-2)
    else:
        c = torch.complex(head[..., :n // 2].contiguous(), head[..., n // 2:].contiguous()) * unit
        r = torch.cat((c.real, c.imag), -1)
    return torch.cat((r, d[..., n:]), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        lens = [int(x) for x in case["lens"].split(",")]
        if s["positions"] is not None:
            pos = s["positions"].long()
        elif case["packed"]:
            pos = torch.cat([torch.arange(n, device="cuda") for n in lens])[None]
        else:
            pos = torch.arange(lens[0], device="cuda").repeat(len(lens), 1)
        f, i = s["inv_freq"], case["interleaved"]
        out = {"q": _turned(s["q"], pos, f, i), "k": _turned(s["k"], pos, f, i)}
        if case["mode"] == "train":
            out |= {"dq": _turned(s["dq"], pos, f, i, True), "dk": _turned(s["dk"], pos, f, i, True)}
        return out
    lens, page = _lengths(case), case["page"]
    Hkv = case["Hkv"]
    if case["op"] == "append":
        out = {x: s[x].double() for x in ("k_pages", "v_pages", "g_pages")}
        q, k = s["q"], s["k"].double()
        starts = []
        for n in lens:
            starts.append(0 if case["packed"] else n - case["T"])
        if case["rot"]:
            if case["packed"]:
                pos = torch.cat([torch.arange(n, device="cuda") for n in lens])[None]
            else:
                pos = torch.stack([torch.arange(a, a + case["T"], device="cuda") for a in starts])
                pos = torch.where(pos < 0, torch.zeros_like(pos), pos)
            k = _turned(s["k"], pos, s["inv_freq"], case["interleaved"])
            out["q"] = _turned(q, pos, s["inv_freq"], case["interleaved"])
            if case["keys"]:
                out["k"] = k
        first = 0
        for b, n in enumerate(lens):
            count = n if case["packed"] else case["T"]
            src = slice(first, first + count)
            first += count
            at = torch.arange(starts[b], starts[b] + count, device="cuda")
            ok = at >= 0
            at = at[ok]
            pages, slots = s["table"][b, at // page].long(), at % page
            for name, x in (("k_pages", k), ("v_pages", s["v"].double()), ("g_pages", s["g"].double())):
                out[name][pages, slots] = x.flatten(0, 1)[src][ok]
        return out
    Hq, Dk, Dv = case["Hq"], case["Dk"], case["Dv"]
    grp = Hq // Hkv
    rows = []
    for b, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        pages, slots = s["table"][b, at // page].long(), at % page
        k, v, g = (s[x][pages, slots].double() for x in ("k_pages", "v_pages", "g_pages"))
        if case["scalar"]:
            g = g[..., None]
        after = torch.zeros_like(g)                     # gates of the tokens after each one
        after[:-1] = g[1:].flip(0).cumsum(0).flip(0)
        v = v * after.exp()
        q = s["q"][b].double()
        for h in range(Hkv):
            a = q[h * grp:(h + 1) * grp] @ k[:, h].T / math.sqrt(Dk)
            e = (a - a.max(1, keepdim=True).values).exp()
            o = e @ v[:, h]
            if case["norm"]:
                o = o / torch.sqrt((o * o).mean(1, keepdim=True) + EPS) * s["w"].double()
            else:
                o = o / e.sum(1, keepdim=True)
            rows.append(o)
    y = torch.cat(rows).view(case["B"], Hq, Dv)
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z * torch.sigmoid(z)
    return y
