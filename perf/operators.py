"""Timed cases of the prompt path: rotary positions, the causal attention of packed prompts, writing a run of new
tokens into the low-bit cache, and reading that cache back as 16-bit rows.

Shapes are those of the repository's workloads: head dimension 128, 32 query heads over 8 or 32 KV heads, up to 32768
tokens, batches of up to 16, 1 and 2 bits, groups of 32 and 64, a 16-bit window of 128."""
import math

import torch

own = False

D = 128
DEV = "cuda"


def listed():
    return [
        # the two query rows and two key rows of one decode step, wavelengths scaled by bands for a long context
        {"name": "rope_step", "op": "rope", "B": 8, "T": 2, "Hq": 32, "Hkv": 8, "rot": 128, "inter": False, "kind": "bands", "start": 32700, "values": False},
        # a whole 32K prompt out of the fused projection, keys and values going to their cache rows
        {"name": "rope_prompt", "op": "rope", "B": 1, "T": 32768, "Hq": 32, "Hkv": 8, "rot": 128, "inter": False, "kind": "plain", "start": 0, "values": True},
        # follow-up prompts far into a conversation, half of each head rotated, interleaved pairs, ungrouped heads
        {"name": "rope_part", "op": "rope", "B": 3, "T": 1031, "Hq": 32, "Hkv": 32, "rot": 64, "inter": True, "kind": "ramp", "start": 131072, "values": True},
        # one new token of eight conversations over their 16-bit histories of different lengths
        {"name": "attn_token", "op": "attn", "S": 8, "Hq": 32, "Hkv": 8, "lq": 1, "lk": 32768, "form": "history"},
        # a follow-up prompt over a long history
        {"name": "attn_turn", "op": "attn", "S": 1, "Hq": 32, "Hkv": 8, "lq": 500, "lk": 32768, "form": "history"},
        # short prompts of different lengths packed behind one another, ungrouped heads
        {"name": "attn_short", "op": "attn", "S": 5, "Hq": 32, "Hkv": 32, "lq": 130, "lk": 130, "form": "packed"},
        # a prefill batch of packed prompts
        {"name": "attn_packed", "op": "attn", "S": 9, "Hq": 32, "Hkv": 8, "lq": 4096, "lk": 4096, "form": "packed"},
        # one long prompt
        {"name": "attn_prompt", "op": "attn", "S": 1, "Hq": 32, "Hkv": 8, "lq": 32768, "lk": 32768, "form": "packed"},
        # a short turn written into the caches of eight conversations
        {"name": "write_turn", "op": "write", "B": 8, "Hkv": 8, "N": 8011, "n": 77, "R": 128, "bits": 1, "group": 32},
        # four prompts written straight from the projection
        {"name": "write_prompt", "op": "write", "B": 4, "Hkv": 8, "N": 0, "n": 32768, "R": 128, "bits": 1, "group": 32},
        # two-bit caches of ungrouped heads read back, from an odd position on
        {"name": "read_part", "op": "read", "B": 2, "Hkv": 32, "N": 2048, "R": 128, "bits": 2, "group": 64, "first": 37, "n": 2003},
        # the caches of eight long conversations read back in whole for their next prompt
        {"name": "read_long", "op": "read", "B": 8, "Hkv": 8, "N": 32768, "R": 128, "bits": 1, "group": 32, "first": 0, "n": 32768},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope", "attn", "attn", "write", "read"])
    Hkv = rng.choice([1, 2, 8, 32])
    G = rng.choice([g for g in (1, 2, 4) if Hkv * g <= 32])
    if op == "rope":
        B = rng.randint(1, 8)
        T = _log(rng, 1, 32768 * 48 // (B * (G + 2) * Hkv))
        T = min(T, 32768)
        return {"op": op, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "rot": 16 * rng.randint(1, 8), "inter": rng.random() < 0.5,
                "kind": rng.choice(["plain", "linear", "bands", "ramp"]), "start": rng.randint(0, 200000), "values": rng.random() < 0.5}
    if op == "attn":
        if rng.random() < 0.5:
            lq = _log(rng, 1, 8192)
            return {"op": op, "S": rng.randint(1, 9), "Hq": Hkv * G, "Hkv": Hkv, "lq": lq, "lk": lq, "form": "packed"}
        lq = _log(rng, 1, 2048)
        return {"op": op, "S": rng.randint(1, 8), "Hq": Hkv * G, "Hkv": Hkv, "lq": lq, "lk": lq + _log(rng, 1, 32768 // max(1, Hkv // 8)), "form": "history"}
    bits, group, R = rng.choice([1, 2]), rng.choice([32, 64]), rng.choice([0, 16, 32, 128, 200])
    B = rng.randint(1, 8)
    if op == "write":
        N = rng.choice([0, _log(rng, 1, 16384)])
        n = _log(rng, 1, 32768 * 32 // (B * Hkv))
        return {"op": op, "B": B, "Hkv": Hkv, "N": N, "n": min(n, 32768), "R": R, "bits": bits, "group": group}
    N = min(32768, _log(rng, 1, 32768 * 64 // (B * Hkv)))
    first = rng.choice([0, rng.randint(0, N - 1)])
    return {"op": op, "B": B, "Hkv": Hkv, "N": N, "R": R, "bits": bits, "group": group, "first": first, "n": rng.randint(1, N - first)}


# ---------------------------------------------------------------------------------------------------- rotary positions
def _frequencies(rot, kind):
    """Radians a position of every pair, in 64 bits, and the factor of cosine and sine."""
    f = [500000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":  # positions stretched by 4
        return [x / 4.0 for x in f], 1.0
    if kind == "bands":  # long wavelengths stretched by 8, short ones kept, a straight mix of both between
        lo, hi, factor, ctx = 1.0, 4.0, 8.0, 8192.0
        got = []
        for x in f:
            turns = ctx * x / (2.0 * math.pi)  # turns within the first context
            mix = min(1.0, max(0.0, (turns - lo) / (hi - lo)))
            got.append((1.0 - mix) * x / factor + mix * x)
        return got, 1.0
    if kind == "ramp":  # a straight ramp over the pair's index between two numbers of turns, with a factor on the result
        fast, slow, factor, ctx = 32.0, 1.0, 16.0, 8192.0

        def at(turns):
            return rot * math.log(ctx / (turns * 2.0 * math.pi)) / (2.0 * math.log(500000.0))

        lo, hi = max(math.floor(at(fast)), 0), min(math.ceil(at(slow)), rot - 1)
        got = []
        for i, x in enumerate(f):
            ramp = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            got.append(x / factor * ramp + x * (1.0 - ramp))
        return got, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _prepare_rope(c, g):
    B, T, Hq, Hkv = c["B"], c["T"], c["Hq"], c["Hkv"]
    qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
    f, m = _frequencies(c["rot"], c["kind"])
    # the table of the frequencies as a program keeps it: 64-bit fractions of a turn a position
    turns = [int(x / (2.0 * math.pi) * 2.0 ** 64) for x in f]
    turns = torch.tensor([t - (1 << 64) if t >= 1 << 63 else t for t in turns], dtype=torch.int64, device=DEV)
    first = c["start"] + torch.randint(0, 64, (B, 1), generator=g, device=DEV)
    pos = (first + torch.arange(T, device=DEV)).to(torch.int32)
    empty = lambda h: torch.empty((B, h, T, D), device=DEV, dtype=torch.bfloat16)  # noqa: E731
    return {"c": c, "q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hkv], "v": qkv[:, :, Hq + Hkv:] if c["values"] else None,
            "pos": pos, "turns": turns, "freq": torch.tensor(f, dtype=torch.float64, device=DEV), "m": m,
            "q_out": torch.empty((B, T, Hq, D), device=DEV, dtype=torch.bfloat16), "k_out": empty(Hkv).transpose(1, 2),
            "v_out": empty(Hkv).transpose(1, 2) if c["values"] else None}


def _rotate(x, cos, sin, rot, inter):
    x = x.float()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([y, z], dim=-1).flatten(-2) if inter else torch.cat([y, z], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1).to(torch.bfloat16)


def _run_rope(s):
    c = s["c"]
    if own:
        import bit_kv_cache_spc_gb300 as spc
        spc.spc_rope(s["q"], s["k"], s["pos"], s["turns"], rot=c["rot"], interleaved=c["inter"], mscale=s["m"], v=s["v"],
                     q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"])
        return [s["q_out"], s["k_out"]] + ([s["v_out"]] if c["values"] else [])
    angle = s["pos"].double()[:, :, None, None] * s["freq"]
    cos, sin = (angle.cos() * s["m"]).float(), (angle.sin() * s["m"]).float()
    got = [_rotate(s["q"], cos, sin, c["rot"], c["inter"]), _rotate(s["k"], cos, sin, c["rot"], c["inter"])]
    return got + ([s["v"].transpose(1, 2).contiguous().transpose(1, 2)] if c["values"] else [])


def _exact_rope(s):
    c = s["c"]
    half = c["rot"] // 2
    first = [2 * i if c["inter"] else i for i in range(half)]
    second = [2 * i + 1 if c["inter"] else i + half for i in range(half)]
    z = torch.polar(torch.full((), s["m"], dtype=torch.float64, device=DEV), s["pos"].double().unsqueeze(-1) * s["freq"]).unsqueeze(2)
    got = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        w = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = w.real, w.imag
        got.append(y)
    return got + ([s["v"].double()] if c["values"] else [])


def _work_rope(c):
    rows = c["B"] * c["T"] * (c["Hq"] + c["Hkv"] * (2 if c["values"] else 1))
    return {"bytes": rows * 512 + 4 * c["B"] * c["T"], "flops": 3 * c["B"] * c["T"] * (c["Hq"] + c["Hkv"]) * c["rot"]}


# --------------------------------------------------------------------------------------------------- prompt attention
def _lengths(c):
    """Lengths of the case's sequences: the first the longest, one of several empty, the others between."""
    lq, lk = [c["lq"]], [c["lk"]]
    for s in range(1, c["S"]):
        part = ((s * 37) % 64 + 1) / 64.0
        if c["form"] == "packed":
            n = 0 if s == 3 else max(1, int(c["lq"] * part))
            lq.append(n)
            lk.append(n)
        else:
            lq.append(max(1, int(c["lq"] * (1.0 - part / 3))))
            lk.append(lq[-1] + int((c["lk"] - c["lq"]) * part))
    return lq, lk


def _prepare_attn(c, g):
    Hq, Hkv = c["Hq"], c["Hkv"]
    lq, lk = _lengths(c)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    if c["form"] == "packed":  # the fused projection of all prompts' tokens, one behind the other
        T = sum(lq)
        qkv = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
        begin = [sum(lq[:s]) for s in range(len(lq))]
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        o = torch.zeros((T, Hq, D), device=DEV, dtype=torch.bfloat16)
        lse = torch.zeros((T, Hq), device=DEV)
        at = {"q_begin": i32(begin), "k_begin": i32(begin)}
    else:  # queries in a padded batch, the 16-bit rows of each sequence's history and turn in a buffer of its own
        q = torch.randn((c["S"], c["lq"], Hq, D), generator=g, device=DEV, dtype=torch.bfloat16)
        kv = torch.randn((2, c["S"], Hkv, c["lk"], D), generator=g, device=DEV, dtype=torch.bfloat16)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
        begin = [None] * c["S"]
        o = torch.zeros((c["S"], c["lq"], Hq, D), device=DEV, dtype=torch.bfloat16)
        lse = torch.zeros((c["S"], c["lq"], Hq), device=DEV)
        at = {"q_begin": None, "k_begin": None}
    q = q.mul(1.5) if c["form"] == "history" else q
    return {"c": c, "q": q, "k": k, "v": v, "o": o, "lse": lse, "lq": lq, "lk": lk, "begin": begin, "q_len": i32(lq), "k_len": i32(lk), **at}


def _rows(x, s, begin, n):
    """Sequence s's n rows: of a batch, or from row `begin` on of packed ones."""
    return x[s, :n] if begin is None else x[begin:begin + n]


def _run_attn(st):
    c = st["c"]
    if own:
        import bit_kv_cache_spc_gb300 as spc
        spc.spc_prompt_attn(st["q"], st["k"], st["v"], st["o"], st["lse"], q_begin=st["q_begin"], q_len=st["q_len"],
                            k_begin=st["k_begin"], k_len=st["k_len"], q_max=c["lq"], k_max=c["lk"])
        return [st["o"], st["lse"]]
    o, lse = torch.zeros_like(st["o"]), torch.zeros_like(st["lse"])
    Hkv, G = c["Hkv"], c["Hq"] // c["Hkv"]
    for s, (n, m) in enumerate(zip(st["lq"], st["lk"])):
        b = st["begin"][s]
        if n == 0:
            continue
        k = _rows(st["k"], s, b, m).float().permute(1, 2, 0).contiguous()  # Hkv, D, m
        v = _rows(st["v"], s, b, m).float().transpose(0, 1).contiguous()  # Hkv, m, D
        step = max(1, min(n, (1 << 30) // (c["Hq"] * m)))
        for i in range(0, n, step):
            e = min(n, i + step)
            w = e + m - n  # keys that the last row of the piece sees
            q = _rows(st["q"], s, b, n)[i:e].float().reshape(e - i, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
            x = torch.matmul(q, k[:, :, :w]).mul_(1.0 / math.sqrt(D)).view(Hkv, G, e - i, w)
            hidden = torch.arange(w, device=DEV)[None, :] > torch.arange(i, e, device=DEV)[:, None] + (m - n)
            x.masked_fill_(hidden, -math.inf)
            top = x.amax(-1, keepdim=True)
            x.sub_(top).exp_()
            total = x.sum(-1, keepdim=True)
            y = torch.matmul(x.view(Hkv, -1, w), v[:, :w]).view(Hkv, G, e - i, D) / total
            _rows(o, s, b, n)[i:e] = y.permute(2, 0, 1, 3).reshape(e - i, c["Hq"], D).to(torch.bfloat16)
            _rows(lse, s, b, n)[i:e] = (top + total.log()).squeeze(-1).permute(2, 0, 1).reshape(e - i, c["Hq"])
    return [o, lse]


def _exact_attn(st):
    c = st["c"]
    if _work_attn(c)["flops"] > 3e12:
        return None
    o, lse = st["o"].double().zero_(), st["lse"].double().zero_()
    G = c["Hq"] // c["Hkv"]
    for s, (n, m) in enumerate(zip(st["lq"], st["lk"])):
        if not n:
            continue
        b = st["begin"][s]
        q, k, v = (_rows(st[x], s, b, y).double() for x, y in (("q", n), ("k", m), ("v", m)))
        seen = torch.ones((n, m), dtype=torch.bool, device=DEV).tril(m - n)
        for h in range(c["Hq"]):
            x = (q[:, h] @ k[:, h // G].T / math.sqrt(D)).where(seen, -math.inf)
            z = torch.logsumexp(x, 1)
            _rows(lse, s, b, n)[:, h] = z
            _rows(o, s, b, n)[:, h] = torch.exp(x - z[:, None]) @ v[:, h // G]
    return [o, lse]


def _work_attn(c):
    lq, lk = _lengths(c)
    pairs = sum(n * m - n * (n - 1) // 2 for n, m in zip(lq, lk))
    return {"bytes": 512 * c["Hkv"] * sum(lk) + (512 + 4) * c["Hq"] * sum(lq), "flops": 4 * D * c["Hq"] * pairs}


# ------------------------------------------------------------------------------------------------- the low-bit cache
def _split(N, R, group):
    """Tokens held in low bits and in 16 bits."""
    nq = max(N - R, 0) // group * group
    return nq, N - nq


def _tables(dev):
    """Where the bits of a 32-token tile stand: (token, channel) of bit b of word w of the key and of the value codes, and
    the channel of each word of the keys' extremes."""
    w, b = torch.arange(128, device=dev)[:, None], torch.arange(32, device=dev)[None, :]
    L, j = w // 4, w % 4
    a, t = L // 4, L % 4
    v = (b + 21) % 32
    n, q = v % 4, v // 4
    i, h = (4 - q % 4) % 4, ((q >= 1) & (q <= 4)).long()
    e = 4 * j + i
    key = (8 * n + a) * D + 16 * (e // 2) + 8 * (e % 2) + 2 * t + h
    val = (16 * (j // 2) + 8 * (j % 2) + 2 * t + b // 16) * D + 16 * ((b % 16) // 2) + 8 * (b % 2) + a
    m, x = torch.arange(128, device=dev) % 32, torch.arange(128, device=dev) // 32
    chan = 16 * (m // 4) + 2 * x + 8 * ((m // 2) % 2) + m % 2
    if_32 = (16 * (m // 16) + 8 * ((m // 8) % 2) + 2 * x + (m // 4) % 2) * 4 + m % 4  # token and channel group, g = 32
    y = torch.arange(64, device=dev)
    p = y // 2
    if_64 = (16 * ((p // 4) % 2) + 8 * ((p // 2) % 2) + 2 * (p // 8) + p % 2) * 2 + y % 2  # the same of a half, g = 64
    return key, val, chan, if_32, if_64


def _bits16(x):
    return (x.to(torch.bfloat16) + 0.0).view(torch.int16).long() & 0xFFFF


def _zs(lo, hi, bits):
    if bits == 1:
        return (3.0 * lo + hi) * 0.25, (hi - lo) * 0.5
    return lo, (hi - lo) / torch.full((), 3.0, dtype=lo.dtype, device=lo.device)  # by a tensor: a rounded quotient, no reciprocal


def _coded(x, lo, hi, bits):
    z, s = _zs(lo, hi, bits)
    q = torch.round((x - z) / s).clamp_(0, 2 ** bits - 1)
    return q.where(s != 0, 0.0).to(torch.uint8)


def _planes(code, at, bits):
    """Words [..., bits, 128] of the codes [..., 32 tokens, D]."""
    c = code.flatten(-2)[..., at.flatten()].unflatten(-1, (128, 32))
    places = torch.tensor([1 << b if b < 31 else -(1 << 31) for b in range(32)], dtype=torch.int32, device=c.device)
    return torch.stack([((c >> p) & 1).to(torch.int32).mul_(places).sum(-1, dtype=torch.int32) for p in range(bits)], dim=-2)


def _packed(k, v, bits, group):
    """Records (int32 words) of whole groups: k, v fp32 [..., groups, group, D]."""
    key, val, chan, if_32, if_64 = _tables(k.device)
    halves = group // 32
    lo, hi = k.amin(-2, keepdim=True), k.amax(-2, keepdim=True)
    kc = _planes(_coded(k, lo, hi, bits).unflatten(-2, (halves, 32)), key, bits).flatten(-3)
    kmm = (_bits16(lo) | _bits16(hi) << 16).squeeze(-2)[..., chan]
    v = v.unflatten(-1, (D // group, group))
    lo, hi = v.amin(-1, keepdim=True), v.amax(-1, keepdim=True)
    vc = _planes(_coded(v, lo, hi, bits).flatten(-2).unflatten(-2, (halves, 32)), val, bits).flatten(-3)
    vmm = (_bits16(lo) | _bits16(hi) << 16).squeeze(-1)
    vmm = vmm.flatten(-2)[..., if_32] if group == 32 else vmm.unflatten(-2, (2, 32)).flatten(-2)[..., if_64].flatten(-2)
    return torch.cat([kc, kmm.to(torch.int32), vc, vmm.to(torch.int32)], dim=-1)


def _words(bits, group):
    return 256 * (bits + 1) if group == 32 else 512 * bits + 256


def _prepare_write(c, g):
    B, Hkv, N, n, R, group = c["B"], c["Hkv"], c["N"], c["n"], c["R"], c["group"]
    nq, r = _split(N, R, group)
    nq1, r1 = _split(N + n, R, group)
    kv = torch.randn((B, n, 2 * Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
    kv[:, :, :Hkv, 5::32] *= 8  # four key channels far larger than the others
    return {"c": c, "k": kv[:, :, :Hkv], "v": kv[:, :, Hkv:], "cap": nq1 // 32, "rcap": max(r, r1),
            "records": torch.zeros((B, Hkv, nq1 // group, _words(c["bits"], group)), dtype=torch.int32, device=DEV),
            "resid": torch.randn((B, Hkv, max(r, r1), 2, D), generator=g, device=DEV, dtype=torch.bfloat16)}


def _run_write(s):
    c = s["c"]
    if own:
        import bit_kv_cache_spc_gb300 as spc
        d = spc.Dims(c["B"], c["Hkv"], c["Hkv"], c["N"], c["R"], c["bits"], q_groups_cap=s["cap"], resid_cap=s["rcap"], group=c["group"])
        spc.spc_extend_kv(d, s["k"], s["v"], s["records"], s["resid"])
        return [s["records"], s["resid"]]
    group = c["group"]
    nq, r = _split(c["N"], c["R"], group)
    nq1, r1 = _split(c["N"] + c["n"], c["R"], group)
    k, v = (torch.cat([s["resid"][:, :, :r, i], x.transpose(1, 2)], dim=2) for i, x in enumerate((s["k"], s["v"])))
    w = nq1 - nq  # tokens that leave 16 bits
    if w:
        s["records"][:, :, nq // group:] = _packed(k[:, :, :w].float().unflatten(2, (-1, group)), v[:, :, :w].float().unflatten(2, (-1, group)), c["bits"], group)
    s["resid"][:, :, :r1] = torch.stack([k[:, :, w:], v[:, :, w:]], dim=3)
    return [s["records"], s["resid"]]


def _exact_write(s):
    """The 16-bit window; the words are whole numbers."""
    c = s["c"]
    nq, r = _split(c["N"], c["R"], c["group"])
    nq1, r1 = _split(c["N"] + c["n"], c["R"], c["group"])
    new = torch.stack([s["k"], s["v"]], dim=3).transpose(1, 2).double()
    window = s["resid"].double().clone()
    every = torch.cat([window[:, :, :r], new], dim=2)
    window[:, :, :r1] = every[:, :, every.shape[2] - r1:]
    return [None, window]


def _work_write(c):
    nq, r = _split(c["N"], c["R"], c["group"])
    nq1, r1 = _split(c["N"] + c["n"], c["R"], c["group"])
    per = 4 * _words(c["bits"], c["group"])
    rows = c["n"] + r1 + (r if nq1 > nq else 0)
    return {"bytes": c["B"] * c["Hkv"] * (512 * rows + (nq1 - nq) // c["group"] * per), "flops": 4 * D * 2 * c["B"] * c["Hkv"] * (nq1 - nq)}


def _prepare_read(c, g):
    B, Hkv, bits, group = c["B"], c["Hkv"], c["bits"], c["group"]
    nq, r = _split(c["N"], c["R"], group)
    units, words = nq // group, _words(bits, group)
    records = torch.randint(-2 ** 31, 2 ** 31, (B, Hkv, units, words), generator=g, device=DEV, dtype=torch.int32)
    codes = 128 * bits * group // 32  # words of the keys' codes and of the values' codes; each extremes' words behind them
    for at in (codes, 2 * codes + 128):
        x = torch.randn((2, B, Hkv, units, 128), generator=g, device=DEV)
        records[..., at:at + 128] = (_bits16(x.amin(0) - 1) | _bits16(x.amax(0) + 1) << 16).to(torch.int32)
    out = lambda: torch.empty((B, Hkv, c["n"], D), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return {"c": c, "records": records, "resid": torch.randn((B, Hkv, r, 2, D), generator=g, device=DEV, dtype=torch.bfloat16),
            "k": out().transpose(1, 2), "v": out().transpose(1, 2)}


def _codes_of(words, at, bits):
    """Codes [..., tokens, D] of the words [..., halves, bits, 128]."""
    put = torch.empty_like(at.flatten())
    put[at.flatten()] = torch.arange(at.numel(), device=at.device)
    got = 0
    for p in range(bits):
        w = words[..., p, :][..., put // 32]
        got = got + (((w >> (put % 32).to(torch.int32)) & 1) << p)
    return got.unflatten(-1, (32, D)).flatten(-3, -2)


def _halves16(mm):
    return (mm << 16).view(torch.float32), (mm & -65536).view(torch.float32)


def _levels(s):
    """Keys and values [B][Hkv][N][D] that a cache holds, in 32 bits."""
    c = s["c"]
    bits, group = c["bits"], c["group"]
    rec, halves = s["records"], group // 32
    key, val, chan, if_32, if_64 = _tables(rec.device)
    n = 128 * bits * halves
    back = torch.empty_like(chan)
    back[chan] = torch.arange(128, device=chan.device)
    lo, hi = (x[..., back].unsqueeze(-2) for x in _halves16(rec[..., n:n + 128]))
    z, st = _zs(lo, hi, bits)
    k = z + st * _codes_of(rec[..., :n].unflatten(-1, (halves, bits, 128)), key, bits).float()
    at = if_32 if group == 32 else torch.cat([if_64, if_64 + 64])
    back = torch.empty_like(at)
    back[at] = torch.arange(128, device=at.device)
    lo, hi = (x[..., back].unflatten(-1, (group, D // group)).unsqueeze(-1) for x in _halves16(rec[..., 2 * n + 128:]))
    z, st = _zs(lo, hi, bits)
    codes = _codes_of(rec[..., n + 128:2 * n + 128].unflatten(-1, (halves, bits, 128)), val, bits).float()
    v = (z + st * codes.unflatten(-1, (D // group, group))).flatten(-2)
    return k.flatten(2, 3), v.flatten(2, 3)


def _run_read(s):
    c = s["c"]
    first, end = c["first"], c["first"] + c["n"]
    if own:
        import bit_kv_cache_spc_gb300 as spc
        nq, r = _split(c["N"], c["R"], c["group"])
        d = spc.Dims(c["B"], c["Hkv"], c["Hkv"], c["N"], c["R"], c["bits"], q_groups_cap=nq // 32, resid_cap=r, group=c["group"])
        spc.spc_dequantize_kv(d, s["records"], s["resid"], first, s["k"], s["v"])
        return [s["k"], s["v"]]
    return [torch.cat([x.to(torch.bfloat16), s["resid"][:, :, :, i]], dim=2)[:, :, first:end].contiguous().transpose(1, 2)
            for i, x in enumerate(_levels(s))]


def _exact_read(s):
    """From the definition: a 1-bit code stands for the first or the third quarter of its group's range, a 2-bit code for
    so many thirds of it.  Every bit is put where the record's rule says."""
    c = s["c"]
    bits, group = c["bits"], c["group"]
    if c["B"] * c["Hkv"] * c["N"] > 1 << 20:
        return None
    places = torch.arange(32, dtype=torch.int32, device=DEV)
    tables = _tables(DEV)
    n = 128 * bits * group // 32
    got = []
    for kind in (0, 1):
        words = s["records"][..., kind * (n + 128):kind * (n + 128) + n + 128]
        bit = (words[..., :n].unflatten(-1, (group // 32, bits, 128, 1)) >> places & 1).flatten(-2)
        code = torch.zeros(bit.shape[:-2] + (32 * D,), dtype=torch.float64, device=DEV)
        for p in range(bits):
            code[..., tables[kind].flatten()] += bit[..., p, :] * 2.0 ** p
        code = code.unflatten(-1, (32, D)).flatten(3, 4)  # B, Hkv, units, group, D
        place = (2 * code + 1) / 4 if bits == 1 else code / 3
        ends = words[..., n:].contiguous().view(torch.bfloat16).double().unflatten(-1, (128, 2))
        if kind == 0:
            of = torch.empty_like(ends)
            of[..., tables[2], :] = ends
            lo, hi = of[..., None, :, 0], of[..., None, :, 1]
        else:
            at = tables[3] if group == 32 else torch.cat([tables[4], 64 + tables[4]])
            of = torch.empty_like(ends)
            of[..., at, :] = ends
            of = of.unflatten(-2, (group, D // group)).repeat_interleave(group, -2)
            lo, hi = of[..., 0], of[..., 1]
        rows = torch.cat([(lo + (hi - lo) * place).flatten(2, 3), s["resid"][:, :, :, kind].double()], dim=2)
        got.append(rows[:, :, c["first"]:c["first"] + c["n"]].transpose(1, 2))
    return got


def _work_read(c):
    nq, r = _split(c["N"], c["R"], c["group"])
    end = c["first"] + c["n"]
    low = max(0, min(end, nq) - c["first"])
    per = 4.0 * _words(c["bits"], c["group"]) / c["group"]
    return {"bytes": c["B"] * c["Hkv"] * (512 * c["n"] + per * low + 512 * (c["n"] - low)), "flops": 2 * D * 2 * c["B"] * c["Hkv"] * low}


_KINDS = {"rope": (_prepare_rope, _run_rope, _exact_rope, _work_rope), "attn": (_prepare_attn, _run_attn, _exact_attn, _work_attn),
          "write": (_prepare_write, _run_write, _exact_write, _work_write), "read": (_prepare_read, _run_read, _exact_read, _work_read)}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return _KINDS[case["op"]][0](case, g)


def run(state):
    return _KINDS[state["c"]["op"]][1](state)


def exact(case, seed):
    return _KINDS[case["op"]][2](prepare(case, seed))


def work(case):
    return _KINDS[case["op"]][3](case)
