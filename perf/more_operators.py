"""Timed cases of three more operators of the prompt path: norms of query and key heads with the rotation in the same pass
(also by positions of several axes), attention with a sliding window and a few first tokens that stay visible, and attention
of sequences that share a long prefix.

Shapes are those of the repository's workloads: head dimension 128, 32 query heads over 8 or 32 KV heads, up to 32768
tokens, batches of single tokens, short turns and whole prompts."""
import math

import torch

own = False

D = 128
DEV = "cuda"


def listed():
    return [
        # the query and key rows of one decode step of eight sequences
        {"name": "norm_step", "op": "norm", "B": 8, "T": 2, "Hq": 32, "Hkv": 8, "rot": 128, "inter": False, "axes": 1, "start": 32700, "values": False, "normed": True},
        # a video's tokens, pairs turned by time, height and width by turns, ungrouped heads, keys and values to their cache rows
        {"name": "norm_video", "op": "norm", "B": 2, "T": 1031, "Hq": 32, "Hkv": 32, "rot": 128, "inter": False, "axes": 3, "start": 700, "values": True, "normed": True},
        # a whole 32K prompt out of the fused projection, keys and values going to their cache rows
        {"name": "norm_prompt", "op": "norm", "B": 1, "T": 32768, "Hq": 32, "Hkv": 8, "rot": 128, "inter": False, "axes": 1, "start": 0, "values": True, "normed": True},
        # one new token of eight conversations, the last 4096 tokens of their histories and the first four
        {"name": "window_token", "op": "window", "S": 8, "Hq": 32, "Hkv": 8, "lq": 1, "lk": 32768, "W": 4096, "sinks": 4, "form": "history"},
        # a follow-up prompt in a layer with a short window
        {"name": "window_turn", "op": "window", "S": 1, "Hq": 32, "Hkv": 8, "lq": 500, "lk": 32768, "W": 1024, "sinks": 4, "form": "history"},
        # a prefill batch of packed prompts of different lengths, ungrouped heads, the shortest window
        {"name": "window_packed", "op": "window", "S": 9, "Hq": 32, "Hkv": 32, "lq": 4096, "lk": 4096, "W": 128, "sinks": 0, "form": "packed"},
        # one long prompt, a window of 4096
        {"name": "window_prompt", "op": "window", "S": 1, "Hq": 32, "Hkv": 8, "lq": 32768, "lk": 32768, "W": 4096, "sinks": 4, "form": "packed"},
        # one token each of five answers to one short question
        {"name": "prefix_few", "op": "prefix", "S": 5, "Hq": 32, "Hkv": 8, "P": 2003, "lq": 1, "lk": 130, "form": "history"},
        # one token each of 64 requests behind one long document
        {"name": "prefix_token", "op": "prefix", "S": 64, "Hq": 32, "Hkv": 8, "P": 32768, "lq": 1, "lk": 1024, "form": "history"},
        # short questions of different lengths, packed, behind a system prompt, ungrouped heads
        {"name": "prefix_turn", "op": "prefix", "S": 17, "Hq": 32, "Hkv": 32, "P": 8011, "lq": 77, "lk": 77, "form": "packed"},
        # longer prompts behind a document
        {"name": "prefix_prompt", "op": "prefix", "S": 4, "Hq": 32, "Hkv": 8, "P": 16384, "lq": 2048, "lk": 2048, "form": "packed"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["norm", "window", "window", "prefix", "prefix"])
    Hkv = rng.choice([1, 2, 8, 32])
    G = rng.choice([g for g in (1, 2, 4) if Hkv * g <= 32])
    if op == "norm":
        B = rng.randint(1, 8)
        T = min(32768, _log(rng, 1, 32768 * 48 // (B * (G + 2) * Hkv)))
        return {"op": op, "B": B, "T": T, "Hq": Hkv * G, "Hkv": Hkv, "rot": 16 * rng.randint(1, 8), "inter": rng.random() < 0.5,
                "axes": rng.choice([1, 1, 2, 3]), "start": rng.randint(0, 200000), "values": rng.random() < 0.5, "normed": rng.random() < 0.8}
    form = rng.choice(["packed", "history"])
    if op == "window":
        lq = _log(rng, 1, 4096 if form == "packed" else 2048)
        lk = lq if form == "packed" else lq + _log(rng, 1, 32768 // max(1, Hkv // 8))
        return {"op": op, "S": rng.randint(1, 9), "Hq": Hkv * G, "Hkv": Hkv, "lq": lq, "lk": lk, "W": _log(rng, 1, 4096),
                "sinks": rng.choice([0, 1, 4, 16, rng.randint(1, 200)]), "form": form}
    S = _log(rng, 1, 64)
    lq = _log(rng, 1, 6000 // S)
    lk = lq if form == "packed" else lq + _log(rng, 1, 1024)
    return {"op": op, "S": S, "Hq": Hkv * G, "Hkv": Hkv, "P": _log(rng, 1, 16384), "lq": lq, "lk": lk, "form": form}


# ----------------------------------------------------------------------------------------- norms of heads and rotation
def _axis_of(rot, axes, inter):
    """The axis of every pair: sections behind one another, or (interleaved pairs) as many by turns."""
    half = rot // 2
    if axes == 1:
        return [0] * half
    small = max(1, half // (axes + 1)) if axes > 1 else 0
    sections = [half - small * (axes - 1)] + [small] * (axes - 1)
    if inter:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    return [i % axes if i < axes * sections[i % axes] else 0 for i in range(half)]


def _prepare_norm(c, g):
    B, T, Hq, Hkv, A = c["B"], c["T"], c["Hq"], c["Hkv"], c["axes"]
    qkv = torch.randn((B, T, Hq + 2 * Hkv, D), generator=g, device=DEV, dtype=torch.bfloat16)
    qkv[:, :, ::3] *= 4  # heads of different size
    f = [500000.0 ** (-2.0 * i / c["rot"]) for i in range(c["rot"] // 2)]
    # the table of the frequencies as a program keeps it: 64-bit fractions of a turn a position
    turns = [int(x / (2.0 * math.pi) * 2.0 ** 64) for x in f]
    first = c["start"] + torch.randint(0, 64, (A, B, 1), generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    steps = [t] if A == 1 else [t // 64, t // 8 % 8, t % 8][:A]  # rows of images of 8 x 8 patches
    pos = (first + torch.stack(steps)[:, None, :]).to(torch.int32)
    weight = lambda: 1.0 + 0.2 * torch.randn((D,), generator=g, device=DEV)  # noqa: E731
    empty = lambda h: torch.empty((B, h, T, D), device=DEV, dtype=torch.bfloat16)  # noqa: E731
    return {"c": c, "q": qkv[:, :, :Hq], "k": qkv[:, :, Hq:Hq + Hkv], "v": qkv[:, :, Hq + Hkv:] if c["values"] else None,
            "pos": pos.contiguous(), "turns": torch.tensor(turns, dtype=torch.int64, device=DEV), "freq": torch.tensor(f, dtype=torch.float64, device=DEV),
            "axis": _axis_of(c["rot"], A, c["inter"]), "wq": weight() if c["normed"] else None, "wk": weight() if c["normed"] else None,
            "q_out": torch.empty((B, T, Hq, D), device=DEV, dtype=torch.bfloat16), "k_out": empty(Hkv).transpose(1, 2),
            "v_out": empty(Hkv).transpose(1, 2) if c["values"] else None}


def _run_norm(s):
    c = s["c"]
    rot, inter = c["rot"], c["inter"]
    if own:
        import bit_kv_cache_spc_gb300 as spc
        spc.spc_norm_rope(s["q"], s["k"], s["pos"], s["turns"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, axis=s["axis"],
                          rot=rot, interleaved=inter, v=s["v"], q_out=s["q_out"], k_out=s["k_out"], v_out=s["v_out"])
        return [s["q_out"], s["k_out"]] + ([s["v_out"]] if c["values"] else [])
    axis = torch.tensor(s["axis"], device=DEV)
    angle = s["pos"].double()[axis].permute(1, 2, 0)[:, :, None, :] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.float()
        if w is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + 1e-6) * w
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
        y, z = a * cos - b * sin, a * sin + b * cos
        turned = torch.stack([y, z], dim=-1).flatten(-2) if inter else torch.cat([y, z], dim=-1)
        got.append(torch.cat([turned, x[..., rot:]], dim=-1).to(torch.bfloat16))
    return got + ([s["v"].transpose(1, 2).contiguous().transpose(1, 2)] if c["values"] else [])


def _exact_norm(s):
    c = s["c"]
    half = c["rot"] // 2
    first = [2 * i if c["inter"] else i for i in range(half)]
    second = [2 * i + 1 if c["inter"] else i + half for i in range(half)]
    angle = torch.stack([s["pos"][a].double() * s["freq"][i] for i, a in enumerate(s["axis"])], dim=-1)
    z = torch.polar(torch.ones_like(angle), angle).unsqueeze(2)
    got = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        y = x.double().clone()
        if w is not None:
            y *= torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
            y *= w.double()
        u = torch.complex(y[..., first], y[..., second]) * z
        y[..., first], y[..., second] = u.real, u.imag
        got.append(y)
    return got + ([s["v"].double()] if c["values"] else [])


def _work_norm(c):
    heads = c["Hq"] + c["Hkv"]
    rows = c["B"] * c["T"] * (heads + (c["Hkv"] if c["values"] else 0))
    return {"bytes": rows * 512 + 4 * c["axes"] * c["B"] * c["T"], "flops": c["B"] * c["T"] * heads * (3 * c["rot"] + (4 * D if c["normed"] else 0))}


# --------------------------------------------------------------------------------------------- both kinds of attention
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
        q = torch.randn((c["S"], c["lq"], Hq, D), generator=g, device=DEV, dtype=torch.bfloat16).mul_(1.5)
        kv = torch.randn((2, c["S"], Hkv, c["lk"], D), generator=g, device=DEV, dtype=torch.bfloat16)
        k, v = kv[0].transpose(1, 2), kv[1].transpose(1, 2)
        begin = [None] * c["S"]
        o = torch.zeros((c["S"], c["lq"], Hq, D), device=DEV, dtype=torch.bfloat16)
        lse = torch.zeros((c["S"], c["lq"], Hq), device=DEV)
        at = {"q_begin": None, "k_begin": None}
    st = {"c": c, "q": q, "k": k, "v": v, "o": o, "lse": lse, "lq": lq, "lk": lk, "begin": begin, "q_len": i32(lq), "k_len": i32(lk), **at}
    if c["op"] == "prefix":  # in the head-major rows of a cache
        p = torch.randn((2, Hkv, c["P"], D), generator=g, device=DEV, dtype=torch.bfloat16)
        st["pk"], st["pv"] = p[0].transpose(0, 1), p[1].transpose(0, 1)
    return st


def _rows(x, s, begin, n):
    """Sequence s's n rows: of a batch, or from row `begin` on of packed ones."""
    return x[s, :n] if begin is None else x[begin:begin + n]


def _attend(q, k, v, shown, o, lse):
    """q [n][Hq][D], k and v [Hkv][D][m] and [Hkv][m][D] in 32 bits; shown [n][m]; rows of o and lse."""
    n, Hq = q.shape[:2]
    Hkv, m = v.shape[:2]
    G = Hq // Hkv
    x = q.float().reshape(n, Hkv, G, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    x = torch.matmul(x, k).mul_(1.0 / math.sqrt(D)).view(Hkv, G, n, m)
    x.masked_fill_(~shown, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    y = torch.matmul(x.view(Hkv, -1, m), v).view(Hkv, G, n, D) / total
    o[:] = y.permute(2, 0, 1, 3).reshape(n, Hq, D).to(torch.bfloat16)
    lse[:] = (top + total.log()).squeeze(-1).permute(2, 0, 1).reshape(n, Hq)


def _window_plain(st, o, lse):
    c = st["c"]
    W, sinks = c["W"], c["sinks"]
    for s, (n, m) in enumerate(zip(st["lq"], st["lk"])):
        b = st["begin"][s]
        if n == 0:
            continue
        k = _rows(st["k"], s, b, m).float().permute(1, 2, 0).contiguous()  # Hkv, D, m
        v = _rows(st["v"], s, b, m).float().transpose(0, 1).contiguous()  # Hkv, m, D
        step = max(1, min(n, 1024, (1 << 29) // (c["Hq"] * min(m, W + sinks + 1024))))
        for i in range(0, n, step):
            e = min(n, i + step)
            lo, hi = max(0, i + m - n - W + 1), e + m - n  # keys that the windows of the piece's rows reach
            head = min(sinks, lo)
            at = torch.cat([torch.arange(head, device=DEV), torch.arange(lo, hi, device=DEV)])
            p = torch.arange(i, e, device=DEV)[:, None] + (m - n)
            shown = (at <= p) & ((at > p - W) | (at < sinks))
            kk = torch.cat([k[:, :, :head], k[:, :, lo:hi]], dim=2)
            vv = torch.cat([v[:, :head], v[:, lo:hi]], dim=1)
            _attend(_rows(st["q"], s, b, n)[i:e], kk, vv, shown, _rows(o, s, b, n)[i:e], _rows(lse, s, b, n)[i:e])


def _prefix_plain(st, o, lse):
    c = st["c"]
    P = c["P"]
    pk, pv = st["pk"].float().permute(1, 2, 0), st["pv"].float().transpose(0, 1)
    for s, (n, m) in enumerate(zip(st["lq"], st["lk"])):
        b = st["begin"][s]
        if n == 0:
            continue
        k = torch.cat([pk, _rows(st["k"], s, b, m).float().permute(1, 2, 0)], dim=2)
        v = torch.cat([pv, _rows(st["v"], s, b, m).float().transpose(0, 1)], dim=1)
        step = max(1, min(n, (1 << 30) // (c["Hq"] * (P + m))))
        at = torch.arange(P + m, device=DEV)
        for i in range(0, n, step):
            e = min(n, i + step)
            shown = at <= torch.arange(i, e, device=DEV)[:, None] + (P + m - n)
            _attend(_rows(st["q"], s, b, n)[i:e], k, v, shown, _rows(o, s, b, n)[i:e], _rows(lse, s, b, n)[i:e])


def _run_attn(st):
    c = st["c"]
    if own:
        import bit_kv_cache_spc_gb300 as spc
        at = dict(q_begin=st["q_begin"], q_len=st["q_len"], k_begin=st["k_begin"], k_len=st["k_len"], q_max=c["lq"], k_max=c["lk"])
        if c["op"] == "window":
            spc.spc_window_attn(st["q"], st["k"], st["v"], st["o"], c["W"], c["sinks"], lse=st["lse"], **at)
        else:
            spc.spc_prefix_attn(st["q"], st["pk"], st["pv"], st["k"], st["v"], st["o"], lse=st["lse"], **at)
        return [st["o"], st["lse"]]
    o, lse = torch.zeros_like(st["o"]), torch.zeros_like(st["lse"])
    (_window_plain if c["op"] == "window" else _prefix_plain)(st, o, lse)
    return [o, lse]


def _exact_attn(st):
    """Head by head in 64 bits, from the places that a query's rule lets it see."""
    c = st["c"]
    if _work_attn(c)["flops"] > 3e12:
        return None
    o, lse = st["o"].double().zero_(), st["lse"].double().zero_()
    G = c["Hq"] // c["Hkv"]
    P = c.get("P", 0)
    for s, (n, m) in enumerate(zip(st["lq"], st["lk"])):
        if not n:
            continue
        b = st["begin"][s]
        q, k, v = (_rows(st[x], s, b, y).double() for x, y in (("q", n), ("k", m), ("v", m)))
        if P:
            k, v = torch.cat([st["pk"].double(), k]), torch.cat([st["pv"].double(), v])
        place = torch.arange(n, device=DEV) + (P + m - n)
        for i in range(0, n, 2048):
            p = place[i:i + 2048, None]
            most = int(place[min(i + 2048, n) - 1]) + 1
            j = torch.arange(most, device=DEV)
            if c["op"] == "window":
                least = max(0, int(place[i]) - c["W"] + 1)
                j = torch.cat([j[:min(c["sinks"], least)], j[least:]])
                seen = (j <= p) & ((p - j < c["W"]) | (j < c["sinks"]))
            else:
                seen = j <= p
            for h in range(c["Hq"]):
                x = (q[i:i + 2048, h] @ k[j, h // G].T / math.sqrt(D)).where(seen, -math.inf)
                z = torch.logsumexp(x, 1)
                _rows(lse, s, b, n)[i:i + 2048, h] = z
                _rows(o, s, b, n)[i:i + 2048, h] = torch.exp(x - z[:, None]) @ v[j, h // G]
    return [o, lse]


def _pairs(c, n, m):
    """(query, key) pairs that the rule shows of n queries at the end of m keys, and the keys that some query sees."""
    if c["op"] == "prefix":
        return n * (c["P"] + m) - n * (n - 1) // 2, m
    W, sinks = c["W"], c["sinks"]
    total = sum(min(p + 1, W) + max(0, min(sinks, p + 1 - W)) for p in range(m - n, m))
    least = max(0, m - n - W + 1)
    return total, (m - least + min(sinks, least)) if n else 0


def _work_attn(c):
    lq, lk = _lengths(c)
    got = [_pairs(c, n, m) for n, m in zip(lq, lk)]
    keys = sum(x[1] for x in got) + c.get("P", 0)
    return {"bytes": 512 * c["Hkv"] * keys + (512 + 4) * c["Hq"] * sum(lq), "flops": 4 * D * c["Hq"] * sum(x[0] for x in got)}


_KINDS = {"norm": (_prepare_norm, _run_norm, _exact_norm, _work_norm), "window": (_prepare_attn, _run_attn, _exact_attn, _work_attn),
          "prefix": (_prepare_attn, _run_attn, _exact_attn, _work_attn)}


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
