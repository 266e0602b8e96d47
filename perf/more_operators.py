"""Work of rotary positions in every form, and of attention of prompt chunks over a paged cache.

Two operators, used one after the other as a prompt is served in chunks (the paged writer
between them is measured by operators.py).  "rope" turns pairs of each head vector by the
token's position: neighbouring elements or the two halves of the turned part, the whole head or
a part of it, frequencies as they are or scaled for contexts longer than the trained one;
backward is the transposed map, for training.  "prefill" attends the new tokens of many
sequences, packed, over the sequences' pages, the new tokens' own keys among them.

The cache is [pages][KV heads][tokens of a page][head size]; the table [sequences][most pages]
names each sequence's pages, -1 where it has none.
"""
import math

import torch

own = False

FLOATS = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding step of 64 conversations: query and key heads inside a fused projection's rows, scaled for a long context
        {"name": "rope_step_bf16", "op": "rope", "B": 64, "T": 1, "H": 40, "beside": 8, "hd": 128, "part": 128, "start": 0,
         "pairs": "half", "dt": "bf16", "theta": 500000.0, "scaling": "bands", "factor": 8.0, "far": 100000, "backward": False},
        # the queries of the batch that the prefill benchmark uses, neighbouring pairs
        {"name": "rope_train_bf16", "op": "rope", "B": 4, "T": 2048, "H": 32, "beside": 0, "hd": 128, "part": 128, "start": 0,
         "pairs": "interleaved", "dt": "bf16", "theta": 10000.0, "scaling": "", "factor": 1.0, "far": 0, "backward": False},
        # the gradient of the same through the half layout, stretched by a ramp over the frequencies
        {"name": "rope_backward_bf16", "op": "rope", "B": 4, "T": 2048, "H": 32, "beside": 0, "hd": 128, "part": 128, "start": 0,
         "pairs": "half", "dt": "bf16", "theta": 10000.0, "scaling": "ramp", "factor": 16.0, "far": 0, "backward": True},
        # a packed batch of ragged prompts, a part of wide heads turned, fp32 activations
        {"name": "rope_part_f32", "op": "rope", "B": 1, "T": 5003, "H": 16, "beside": 0, "hd": 256, "part": 64, "start": 0,
         "pairs": "half", "dt": "f32", "theta": 10000.0, "scaling": "linear", "factor": 4.0, "far": 30000, "backward": False},
        # one conversation's next 64 tokens over a short cache: latency
        {"name": "prefill_next_bf16", "op": "prefill", "B": 1, "new_lo": 64, "new": 64, "lo": 777, "length": 777, "H": 32, "Hkv": 8,
         "hd": 128, "page": 16, "dt": "bf16", "cache": "bf16", "causal": True, "window": 0, "softcap": 0.0},
        # four first chunks of 2048 tokens, the batch that the prefill benchmark uses, its keys in pages
        {"name": "prefill_first_bf16", "op": "prefill", "B": 4, "new_lo": 2048, "new": 2048, "lo": 2048, "length": 2048, "H": 32,
         "Hkv": 8, "hd": 128, "page": 16, "dt": "bf16", "cache": "bf16", "causal": True, "window": 0, "softcap": 0.0},
        # the last chunk of a long prompt, over 16-bit and over 8-bit pages
        {"name": "prefill_long_bf16", "op": "prefill", "B": 1, "new_lo": 2048, "new": 2048, "lo": 32768, "length": 32768, "H": 32,
         "Hkv": 8, "hd": 128, "page": 64, "dt": "bf16", "cache": "bf16", "causal": True, "window": 0, "softcap": 0.0},
        {"name": "prefill_long_e4m3", "op": "prefill", "B": 1, "new_lo": 2048, "new": 2048, "lo": 32768, "length": 32768, "H": 32,
         "Hkv": 8, "hd": 128, "page": 64, "dt": "bf16", "cache": "e4m3", "causal": True, "window": 0, "softcap": 0.0},
        # ragged chunks of many running prompts beside short follow-ups, small pages
        {"name": "prefill_ragged_e4m3", "op": "prefill", "B": 24, "new_lo": 3, "new": 1021, "lo": 1500, "length": 9973, "H": 32,
         "Hkv": 8, "hd": 128, "page": 16, "dt": "bf16", "cache": "e4m3", "causal": True, "window": 0, "softcap": 0.0},
        # a short follow-up to one long conversation: few rows, all of the cache to read
        {"name": "prefill_follow_e4m3", "op": "prefill", "B": 1, "new_lo": 29, "new": 29, "lo": 32768, "length": 32768, "H": 32,
         "Hkv": 8, "hd": 128, "page": 64, "dt": "bf16", "cache": "e4m3", "causal": True, "window": 0, "softcap": 0.0},
        # sliding-window layers with a softcap and wide heads
        {"name": "prefill_window_hd256_e5m2", "op": "prefill", "B": 8, "new_lo": 100, "new": 600, "lo": 700, "length": 6001, "H": 16,
         "Hkv": 4, "hd": 256, "page": 32, "dt": "bf16", "cache": "e5m2", "causal": True, "window": 1024, "softcap": 50.0},
        # a small fp16 model without grouping
        {"name": "prefill_heads_f16", "op": "prefill", "B": 8, "new_lo": 33, "new": 333, "lo": 333, "length": 1025, "H": 12, "Hkv": 12,
         "hd": 64, "page": 16, "dt": "f16", "cache": "f16", "causal": True, "window": 0, "softcap": 0.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    return _draw_rope(rng) if rng.random() < 0.4 else _draw_prefill(rng)


def _draw_rope(rng):
    while True:
        hd = rng.choice([32, 64, 80, 96, 128, 128, 256])
        part = rng.choice([hd, hd, hd // 2, hd // 4])
        c = {"op": "rope", "B": _log(rng, 1, 64), "T": _log(rng, 1, 8192), "H": rng.choice([1, 2, 5, 8, 12, 32, 40]),
             "beside": rng.choice([0, 0, 1, 8]), "hd": hd, "part": part, "start": rng.choice([0, 0, hd - part]),
             "pairs": rng.choice(["half", "interleaved"]), "dt": rng.choice(["f32", "f16", "bf16", "bf16"]),
             "theta": rng.choice([10000.0, 500000.0]), "scaling": rng.choice(["", "", "linear", "base", "ramp", "bands"]),
             "far": rng.choice([0, _log(rng, 1, 1000000)]), "backward": rng.random() < 0.4}
        c["factor"] = rng.choice([2.0, 8.0, 32.0]) if c["scaling"] else 1.0
        if c["B"] * c["T"] * (c["H"] + c["beside"]) * hd * BYTES[c["dt"]] <= 4 * 2048 * 32 * 128 * 4:
            return c


def _draw_prefill(rng):
    while True:
        Hkv = rng.choice([1, 2, 4, 8, 12])
        G = rng.choice([1, 2, 4, 7, 8]) if Hkv < 12 else 1
        dt = rng.choice(["bf16", "f16"])
        c = {"op": "prefill", "B": _log(rng, 1, 64), "H": G * Hkv, "Hkv": Hkv, "hd": rng.choice([64, 128, 128, 256]),
             "page": rng.choice([16, 32, 64, 128]), "dt": dt, "cache": rng.choice([dt, dt, "e4m3", "e5m2"]),
             "causal": rng.random() < 0.9, "window": rng.choice([0, 0, 0, _log(rng, 1, 8000)]),
             "softcap": rng.choice([0.0, 0.0, 0.0, 30.0])}
        length = _log(rng, 17, 33000)
        c["length"], c["lo"] = length, rng.choice([length, _log(rng, 1, length)])
        c["new"] = _log(rng, 1, min(length, 2048))
        c["new_lo"] = rng.choice([c["new"], _log(rng, 1, c["new"])])
        c["lo"] = max(c["lo"], c["new"])
        if c["B"] * (length + c["page"]) * Hkv * c["hd"] > 16 * 32768 * 8 * 128:
            continue
        # whole chunks, as the plain form computes them
        if sum(a * b for a, b in zip(*_counts(c))) * c["H"] * c["hd"] <= 2048 * 32768 * 32 * 128:
            return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread: the same for every seed, in an order of its own."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _counts(c):
    """(lengths, new tokens) of the sequences; the new tokens are the last of each length."""
    return _spread(c["lo"], c["length"], c["B"]), _spread(c["new_lo"], c["new"], c["B"])[::-1]


def _sides(c):
    """(tokens back, tokens ahead) that a row sees, None for all."""
    w = c["window"] - 1 if c["window"] else None
    return w, 0 if c["causal"] else w


def work(c):
    if c["op"] == "rope":
        rows = c["B"] * c["T"]
        return {"bytes": rows * (2 * c["H"] * c["hd"] * BYTES[c["dt"]] + 4), "flops": 3 * rows * c["H"] * c["part"]}
    kv, e, es = c["Hkv"] * c["hd"], BYTES[c["dt"]], BYTES[c["cache"]]
    back, ahead = _sides(c)
    lengths, new = _counts(c)
    pairs = keys = rows = 0
    for n, m in zip(lengths, new):
        first = n - m
        keys += n - (max(0, first - back) if back is not None else 0)
        rows += m
        for p in range(first, n):
            low = 0 if back is None else max(0, p - back)
            pairs += (n if ahead is None else min(n, p + ahead + 1)) - low
    scales = keys // c["page"] * 8 * c["Hkv"] if es == 1 else 0  # of a page: a key's and a value's
    return {"bytes": keys * 2 * kv * es + scales + rows * c["H"] * (2 * c["hd"] * e + 4), "flops": 4 * pairs * c["H"] * c["hd"]}


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
    return (_prepare_rope if case["op"] == "rope" else _prepare_prefill)(dict(case), g, h)


def _scaling(c):
    """The frequencies' options: trained for 8192 positions where the scaling asks."""
    extra = {"original_length": 8192} if c["scaling"] in ("ramp", "bands") else {}
    return dict(theta=c["theta"], **(dict(scaling=c["scaling"], factor=c["factor"], **extra) if c["scaling"] else {}))


def _prepare_rope(c, g, h):
    rows, width = c["B"] * c["T"], c["H"] * c["hd"]
    s = {"case": c}
    x = torch.randn((rows, width + c["beside"] * c["hd"]), generator=g, device="cuda", dtype=torch.float32).to(FLOATS[c["dt"]])
    s["x"] = x[:, :width]
    # each sequence's tokens from a position of its own
    first = torch.randint(0, c["far"] + 1, (c["B"], 1), generator=h)
    s["positions"] = (first + torch.arange(c["T"])).flatten().to(torch.int32).cuda()
    if own:
        import attention_attn_fwd_08_gb300 as A

        s["freqs"] = A.attn_rope_freqs(c["part"], **_scaling(c))
    return s


def _pool(g, c, pages):
    """Pages full of keys or values as earlier steps left them: (data, scales or None).  Heads and pages differ in size."""
    x = torch.randn((pages, c["Hkv"], c["page"], c["hd"]), generator=g, device="cuda", dtype=torch.float16)
    x *= torch.exp2(torch.randint(-3, 2, (pages, c["Hkv"], 1, 1), generator=g, device="cuda").half())
    if c["cache"] not in LARGEST:
        return x.to(FLOATS[c["cache"]]), None
    # powers of two, as the cache's writer chooses them
    big = x.abs().amax(dim=(2, 3)).double().clamp(min=2.0 ** -60)
    scale = torch.exp2(torch.ceil(torch.log2(big / LARGEST[c["cache"]]))).float()
    return (x.float() / scale[:, :, None, None]).to(FLOATS[c["cache"]]), scale


def _prepare_prefill(c, g, h):
    lengths, new = _counts(c)
    order = torch.randperm(c["B"], generator=h).tolist()
    lengths, new = [lengths[i] for i in order], [new[i] for i in order]
    most = (c["length"] + c["page"] - 1) // c["page"]
    used = [(n + c["page"] - 1) // c["page"] for n in lengths]
    pages = sum(used) + 3  # three pages that no sequence owns
    perm = torch.randperm(pages, generator=h, dtype=torch.int32)
    table, at = torch.full((c["B"], most), -1, dtype=torch.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = perm[at:at + n]
        at += n
    s = {"case": c, "host": (lengths, new), "table": table.cuda(), "lengths": torch.tensor(lengths, dtype=torch.int32).cuda()}
    s["k_cache"], s["k_scale"] = _pool(g, c, pages)
    s["v_cache"], s["v_scale"] = _pool(g, c, pages)
    s["cu"] = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    # the queries inside the rows of one projection, [queries | keys | values], a few rows of padding behind the last sequence
    rows, width = sum(new) + 5, c["H"] * c["hd"]
    qkv = torch.randn((rows, width + 2 * c["Hkv"] * c["hd"]), generator=g, device="cuda", dtype=torch.float32).to(FLOATS[c["dt"]])
    s["q"] = qkv[:, :width]
    s["o"] = torch.zeros((rows, width), device="cuda", dtype=FLOATS[c["dt"]])
    s["lse"] = torch.zeros((c["H"], rows), device="cuda", dtype=torch.float32)
    return s


# ------------------------------------------------------------ the operators
def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return _rope(s) if c["op"] == "rope" else _prefill(s)


def _own(s):
    import attention_attn_fwd_08_gb300 as A

    c = s["case"]
    if c["op"] == "rope":
        return A.attn_rope_ex(s["x"], s["freqs"], H=c["H"], positions=s["positions"], layout=c["pairs"], rotary_start=c["start"],
                              backward=c["backward"])
    return list(A.attn_paged_prefill(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["cu"], H=c["H"], Hkv=c["Hkv"],
                                     k_scale=s["k_scale"], v_scale=s["v_scale"], causal=c["causal"], window=c["window"],
                                     softcap=c["softcap"], o=s["o"], lse=s["lse"]))


def _frequencies(c):
    """The turn of each pair from one position to the next, in 64 bits, and the factor on the turned pairs."""
    d, theta = c["part"], c["theta"]
    if c["scaling"] == "base":
        theta = theta * c["factor"] ** (d / (d - 2))
    i = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    f = theta ** (-2.0 * i / d)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    elif c["scaling"] == "ramp":  # the pairs that turn more than 32 times in the trained length stay, those below once are stretched
        low, high = (d * math.log(8192 / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (32.0, 1.0))
        low, high = max(math.floor(low), 0), min(math.ceil(high), d - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / c["factor"] * ramp, 0.1 * math.log(c["factor"]) + 1
    elif c["scaling"] == "bands":  # the same by wavelength, from four turns down to one
        part = ((8192 * f / (2 * math.pi) - 1) / 3).clamp(0, 1)
        f = f * ((1 - part) / c["factor"] + part)
    return f, 1.0


def _rope(s):
    c, x = s["case"], s["x"]
    f, amplitude = _frequencies(c)
    angle = s["positions"].double()[:, None] * f
    cos, sin = (angle.cos() * amplitude).float()[:, None], (angle.sin() * amplitude).float()[:, None]
    if c["backward"]:
        sin = -sin
    out = x.reshape(-1, c["H"], c["hd"]).clone()
    part = out[..., c["start"]:c["start"] + c["part"]]
    if c["pairs"] == "half":
        a, b = part[..., :c["part"] // 2].float(), part[..., c["part"] // 2:].float()
        part.copy_(torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2))
    else:
        a, b = part[..., 0::2].float(), part[..., 1::2].float()
        part.copy_(torch.stack([a * cos - b * sin, b * cos + a * sin], dim=3).flatten(2))
    return out.flatten(1)


def _paged(s, b, n, cache, scale):
    """The first n tokens of sequence b in 32 bits: [heads][n][hd]."""
    page = cache.shape[2]
    ids = s["table"][b, :(n + page - 1) // page].long()
    x = cache.view(torch.uint8)[ids].view(cache.dtype).float() if cache.element_size() == 1 else cache[ids].float()
    if scale is not None:
        x = x * scale[ids][..., None, None]
    return x.transpose(0, 1).flatten(1, 2)[:, :n]


def _prefill(s):
    c = s["case"]
    Hkv, hd, G = c["Hkv"], c["hd"], c["H"] // c["Hkv"]
    back, ahead = _sides(c)
    at = 0
    for b, (n, m) in enumerate(zip(*s["host"])):
        k, v = _paged(s, b, n, s["k_cache"], s["k_scale"]), _paged(s, b, n, s["v_cache"], s["v_scale"])
        j = torch.arange(n, device="cuda")[None, :]
        step = max(1, 2 ** 28 // (c["H"] * n))  # rows whose scores fit in a gigabyte
        for i in range(0, m, step):
            r = slice(at + i, at + min(i + step, m))
            w = r.stop - r.start
            q = s["q"][r].float().view(w, Hkv, G, hd).permute(1, 2, 0, 3).flatten(1, 2)
            x = torch.matmul(q, k.transpose(1, 2)) * (1.0 / math.sqrt(hd))
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            p = n - m + i + torch.arange(w, device="cuda").repeat(G)[:, None]
            seen = torch.ones_like(p + j, dtype=torch.bool)
            if ahead is not None:
                seen = seen & (j <= p + ahead)
            if back is not None:
                seen = seen & (j >= p - back)
            x = x.masked_fill(~seen, -math.inf)
            top = x.amax(dim=2, keepdim=True)
            e = torch.exp(x - torch.where(top == -math.inf, torch.zeros_like(top), top))
            total = e.sum(dim=2, keepdim=True)
            o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))
            s["o"][r] = o.unflatten(1, (G, w)).permute(2, 0, 1, 3).reshape(w, -1).to(s["o"].dtype)
            s["lse"][:, r] = (top + torch.log(total)).reshape(c["H"], w)
        at += m
    return [s["o"], s["lse"]]


# ------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_prefill(s)


def _exact_rope(s):
    c = s["case"]
    d, L = c["part"], 8192
    theta = c["theta"] * c["factor"] ** (d / (d - 2)) if c["scaling"] == "base" else c["theta"]
    f, grow = [theta ** (-2.0 * i / d) for i in range(d // 2)], 1.0
    if c["scaling"] == "linear":
        f = [y / c["factor"] for y in f]
    if c["scaling"] == "ramp":
        grow = 1 + math.log(c["factor"]) / 10
        a = max(math.floor(d / 2 * math.log(L / (64 * math.pi), theta)), 0)
        b = min(math.ceil(d / 2 * math.log(L / (2 * math.pi), theta)), d - 1)
        share = [min(max((i - a) / max(b - a, 0.001), 0.0), 1.0) for i in range(d // 2)]
        f = [y * (1 - t) + y * t / c["factor"] for y, t in zip(f, share)]
    if c["scaling"] == "bands":
        f = [y if 2 * math.pi / y <= L / 4 else y / c["factor"] if 2 * math.pi / y >= L else
             y / c["factor"] + (y - y / c["factor"]) * (L * y / (2 * math.pi) - 1) / 3 for y in f]
    angle = s["positions"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    turn = torch.polar(torch.full_like(angle, grow), -angle if c["backward"] else angle)[:, None]
    out = s["x"].double().reshape(-1, c["H"], c["hd"])
    part = out[..., c["start"]:c["start"] + d].clone()
    if c["pairs"] == "half":
        z = torch.complex(*part.unflatten(2, (2, d // 2)).unbind(2)) * turn
        part = torch.cat([z.real, z.imag], dim=2)
    else:
        part = torch.view_as_real(torch.view_as_complex(part.unflatten(2, (d // 2, 2))) * turn).flatten(2)
    return torch.cat([out[..., :c["start"]], part, out[..., c["start"] + d:]], dim=2).flatten(1)


def _exact_prefill(s):
    c = s["case"]
    H, Hkv, hd = c["H"], c["Hkv"], c["hd"]
    lengths, new = s["host"]
    if sum(n * m for n, m in zip(lengths, new)) * H * hd > 2048 * 32768 * 32 * 128:
        return None
    cu = s["cu"].tolist()
    out = s["o"].double()
    lse = s["lse"].double()
    back, ahead = _sides(c)
    for b, n in enumerate(lengths):
        m = cu[b + 1] - cu[b]
        ids = [i for i in s["table"][b].tolist() if i >= 0]
        for g in range(Hkv):
            k, v = ([cache[i, g].double() * (1.0 if scale is None else scale[i, g].double()) for i in ids]
                    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            k, v = torch.cat(k)[:n], torch.cat(v)[:n]
            for hq in range(g * H // Hkv, (g + 1) * H // Hkv):
                z = s["q"][cu[b]:cu[b + 1], hq * hd:(hq + 1) * hd].double() @ k.t() / math.sqrt(hd)
                z = c["softcap"] * torch.tanh(z / c["softcap"]) if c["softcap"] else z
                hidden = torch.zeros((m, n), dtype=torch.bool, device="cuda")
                if ahead is not None:
                    hidden |= torch.ones_like(hidden).triu(n - m + ahead + 1)
                if back is not None:
                    hidden |= torch.ones_like(hidden).tril(n - m - back - 1)
                z.masked_fill_(hidden, -math.inf)
                total = torch.logsumexp(z, dim=1)
                out[cu[b]:cu[b + 1], hq * hd:(hq + 1) * hd] = torch.exp(z - total[:, None]) @ v
                lse[hq, cu[b]:cu[b + 1]] = total
    return [out, lse]
