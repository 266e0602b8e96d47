"""Work of the paged key/value cache, as a serving program does it.

Three operators.  "append" turns the new tokens' keys (and queries) by their
position and stores keys and values in the pages of their sequences, in 16 bits or
in 8 bits with one scale for each page and head.  "decode" attends a few query rows
of each sequence over its pages.  "gather" reads sequences' pages back into packed
16-bit rows, for attention of a long prompt over a cached prefix.

The cache is [pages][KV heads][tokens of a page][head size]; the table
[sequences][most pages] names each sequence's pages, -1 where it has none.
"""
import math

import torch

own = False

FLOATS = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
BYTES = {"f16": 2, "bf16": 2, "e4m3": 1, "e5m2": 1}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 64 conversations of a GQA model: each has one new token
        {"name": "append_step_e4m3", "op": "append", "B": 64, "new_lo": 1, "new": 1, "lo": 200, "length": 8000, "H": 32, "Hkv": 8,
         "hd": 128, "page": 64, "dt": "bf16", "cache": "e4m3", "theta": 500000.0, "turn_q": True},
        # four prompts of 2048 tokens, the batch that the prefill benchmark uses, into a 16-bit cache
        {"name": "append_prompt_bf16", "op": "append", "B": 4, "new_lo": 2048, "new": 2048, "lo": 2048, "length": 2048, "H": 32,
         "Hkv": 8, "hd": 128, "page": 16, "dt": "bf16", "cache": "bf16", "theta": 10000.0, "turn_q": True},
        # ragged chunks of running prompts, far into long sequences, into an 8-bit cache
        {"name": "append_chunks_e4m3", "op": "append", "B": 24, "new_lo": 3, "new": 1021, "lo": 1500, "length": 40000, "H": 32, "Hkv": 8,
         "hd": 128, "page": 64, "dt": "bf16", "cache": "e4m3", "theta": 1000000.0, "turn_q": True},
        # the same for a small model with one KV head per query head, no rotation, the wider 8-bit type
        {"name": "append_small_e5m2", "op": "append", "B": 9, "new_lo": 1, "new": 333, "lo": 333, "length": 1000, "H": 12, "Hkv": 12,
         "hd": 64, "page": 32, "dt": "f16", "cache": "e5m2", "theta": 0.0, "turn_q": False},
        # one conversation, one token, a short cache: latency
        {"name": "decode_one_bf16", "op": "decode", "B": 1, "Lq": 1, "lo": 777, "length": 777, "H": 32, "Hkv": 8, "hd": 128, "page": 16,
         "dt": "bf16", "cache": "bf16", "window": 0, "softcap": 0.0},
        # the long-cache decode benchmark's shape, its cache in pages: 16 bits with four draft tokens, 8 bits with one token
        {"name": "decode_long_lq4_bf16", "op": "decode", "B": 16, "Lq": 4, "lo": 32768, "length": 32768, "H": 32, "Hkv": 8, "hd": 128,
         "page": 64, "dt": "bf16", "cache": "bf16", "window": 0, "softcap": 0.0},
        {"name": "decode_long_e4m3", "op": "decode", "B": 16, "Lq": 1, "lo": 32768, "length": 32768, "H": 32, "Hkv": 8, "hd": 128,
         "page": 64, "dt": "bf16", "cache": "e4m3", "window": 0, "softcap": 0.0},
        # a serving batch of very unlike lengths, small pages
        {"name": "decode_ragged_e4m3", "op": "decode", "B": 61, "Lq": 1, "lo": 5, "length": 9973, "H": 32, "Hkv": 8, "hd": 128,
         "page": 16, "dt": "bf16", "cache": "e4m3", "window": 0, "softcap": 0.0},
        # sliding-window layers with a softcap and wide heads, draft tokens
        {"name": "decode_window_hd256_e5m2", "op": "decode", "B": 32, "Lq": 3, "lo": 700, "length": 6001, "H": 16, "Hkv": 4, "hd": 256,
         "page": 32, "dt": "bf16", "cache": "e5m2", "window": 1024, "softcap": 50.0},
        # a small fp16 model without grouping
        {"name": "decode_heads_f16", "op": "decode", "B": 8, "Lq": 1, "lo": 100, "length": 1025, "H": 12, "Hkv": 12, "hd": 64,
         "page": 16, "dt": "f16", "cache": "f16", "window": 0, "softcap": 0.0},
        # a long cached prefix read back for the next chunk of its prompt
        {"name": "gather_prefix_e4m3", "op": "gather", "B": 1, "lo": 32768, "length": 32768, "Hkv": 8, "hd": 128, "page": 64,
         "dt": "bf16", "cache": "e4m3"},
        # many short prefixes of odd lengths
        {"name": "gather_ragged_f16", "op": "gather", "B": 17, "lo": 1, "length": 1999, "Hkv": 4, "hd": 64, "page": 16, "dt": "f16",
         "cache": "f16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        op = rng.choice(["append", "append", "decode", "decode", "decode", "gather"])
        Hkv = rng.choice([1, 2, 4, 8, 12])
        G = rng.choice([1, 2, 4, 7, 8]) if Hkv < 12 else 1
        hd = rng.choice([64, 128, 128, 256])
        dt = rng.choice(["bf16", "f16"])
        c = {"op": op, "B": _log(rng, 1, 128), "Hkv": Hkv, "hd": hd, "page": rng.choice([16, 32, 64, 128]), "dt": dt,
             "cache": rng.choice([dt, "e4m3", "e4m3", "e5m2"])}
        length = _log(rng, 17, 33000)
        c["length"], c["lo"] = length, rng.choice([length, _log(rng, 1, length)])
        if op == "append":
            c["H"] = G * Hkv
            c["new"] = 1 if rng.random() < 0.4 else _log(rng, 1, min(length, 2048))
            c["new_lo"] = rng.choice([c["new"], _log(rng, 1, c["new"])])
            c["lo"] = max(c["lo"], c["new"])
            c["theta"] = rng.choice([10000.0, 500000.0, 0.0])
            c["turn_q"] = c["theta"] > 0 and rng.random() < 0.7
            pool = c["B"] * (length + c["page"]) * Hkv * hd
            if c["B"] * c["new"] * (c["H"] + Hkv) * hd > 4 * 2048 * 40 * 128 or pool > 24 * 20800 * 8 * 128:
                continue
        elif op == "decode":
            c["H"] = G * Hkv
            c["Lq"] = rng.choice([1, 1, rng.randint(1, min(16, 64 // G))])
            c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 8000)])
            c["softcap"] = rng.choice([0.0, 0.0, 0.0, 30.0])
        if op != "append" and c["B"] * (length + c["page"]) * Hkv * hd > 16 * 32768 * 8 * 128:
            continue
        if op == "gather" and c["B"] * length > 65536:
            continue
        return c


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly spread: the same for every seed, in an order of its own."""
    return [hi if n == 1 else lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _counts(c):
    """(lengths, new tokens) of the sequences; the new tokens are the last of each length."""
    lengths = _spread(c["lo"], c["length"], c["B"])
    return lengths, _spread(c["new_lo"], c["new"], c["B"])[::-1] if c["op"] == "append" else [0] * c["B"]


def work(c):
    lengths, new = _counts(c)
    kv, e, es = c["Hkv"] * c["hd"], BYTES[c["dt"]], BYTES[c["cache"]]
    scales = 8 * c["Hkv"] if es == 1 else 0  # of a page: a key's and a value's
    if c["op"] == "append":
        q = c["H"] * c["hd"] if c["turn_q"] else 0
        pages = sum((n + c["page"] - 1) // c["page"] for n in new)
        flops = sum(new) * (3 * (kv + q) if c["theta"] else 0) + (sum(new) * 4 * kv if es == 1 else 0)
        return {"bytes": sum(new) * (2 * kv * (e + es) + 2 * q * e) + pages * scales, "flops": flops}
    if c["op"] == "gather":
        pages = sum((n + c["page"] - 1) // c["page"] for n in lengths)
        return {"bytes": sum(lengths) * 2 * kv * (e + es) + pages * scales, "flops": sum(lengths) * 2 * kv}
    pairs = keys = 0
    for n in lengths:
        first = max(0, n - c["Lq"])
        keys += n - (max(0, first - c["window"] + 1) if c["window"] else 0)
        for i in range(c["Lq"]):
            p = n - c["Lq"] + i
            if p >= 0:
                pairs += min(p + 1, c["window"]) if c["window"] else p + 1
    rows = c["B"] * c["Lq"] * c["H"]
    return {"bytes": keys * 2 * kv * es + keys // c["page"] * scales + rows * (2 * c["hd"] * e + 4), "flops": 4 * pairs * c["H"] * c["hd"]}


# ----------------------------------------------------------------- inputs
def _amax_scale(x, cache):
    """A power of two for each page and head that brings its largest value into the 8-bit type's range."""
    big = x.abs().amax(dim=(2, 3)).double().clamp(min=2.0 ** -60)
    return torch.exp2(torch.ceil(torch.log2(big / LARGEST[cache]))).float()


def _pool(g, c, pages):
    """Pages full of keys or values as an earlier step left them: (data, scales or None).  Heads and pages differ in size."""
    x = torch.randn((pages, c["Hkv"], c["page"], c["hd"]), generator=g, device="cuda", dtype=torch.float16)
    x *= torch.exp2(torch.randint(-3, 2, (pages, c["Hkv"], 1, 1), generator=g, device="cuda").half())
    if c["cache"] not in LARGEST:
        return x.to(FLOATS[c["cache"]]), None
    scale = _amax_scale(x, c["cache"])
    if c["op"] != "append":  # scales that a calibration chose are no powers of two
        scale = x.abs().amax(dim=(2, 3)).float() / LARGEST[c["cache"]]
    return (x.float() / scale[:, :, None, None]).to(FLOATS[c["cache"]]), scale


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    h = torch.Generator().manual_seed(seed)
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
    s = {"case": c, "table": table.cuda(), "lengths": torch.tensor(lengths, dtype=torch.int32).cuda()}
    s["k_cache"], s["k_scale"] = _pool(g, c, pages)
    s["v_cache"], s["v_scale"] = _pool(g, c, pages)
    dt, kv = FLOATS[c["dt"]], c["Hkv"] * c["hd"]

    def rows(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)

    if c["op"] == "append":
        cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0)
        s["rows"] = int(cu[-1])
        s["cu"] = cu.to(torch.int32).cuda()
        # the rows of one projection, [queries | keys | values], with a few rows of padding behind the last sequence
        qkv = rows(s["rows"] + 5, c["H"] * c["hd"] + 2 * kv)
        s["q"], s["k"], s["v"] = qkv[:, :c["H"] * c["hd"]], qkv[:, -2 * kv:-kv], qkv[:, -kv:]
        s["q_out"] = torch.zeros((s["rows"] + 5, c["H"] * c["hd"]), device="cuda", dtype=dt) if c["turn_q"] else None
    elif c["op"] == "decode":
        s["q"] = rows(c["B"], c["Lq"], c["H"] * c["hd"])
    else:
        cu = torch.tensor([0] + lengths, dtype=torch.int64).cumsum(0)
        s["rows"] = int(cu[-1])
        s["cu"] = cu.to(torch.int32).cuda()
    return s


# ------------------------------------------------------------ the operators
def run(s):
    c = s["case"]
    if own:
        return _own(s)
    return {"append": _append, "decode": _decode, "gather": _gather}[c["op"]](s)


def _own(s):
    import attention_attn_fwd_08_gb300 as A

    c = s["case"]
    if c["op"] == "append":
        A.attn_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["cu"], H=c["H"], Hkv=c["Hkv"],
                            k_scale=s["k_scale"], v_scale=s["v_scale"], q=s["q"] if c["turn_q"] else None, q_out=s["q_out"],
                            rope_theta=c["theta"] or None)
        return [x for x in (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_out"]) if x is not None]
    if c["op"] == "decode":
        return list(A.attn_paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], H=c["H"], Hkv=c["Hkv"],
                                        k_scale=s["k_scale"], v_scale=s["v_scale"], causal=True, window=c["window"],
                                        softcap=c["softcap"]))
    return list(A.attn_paged_gather(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["rows"], Hkv=c["Hkv"], dtype=FLOATS[c["dt"]],
                                    k_scale=s["k_scale"], v_scale=s["v_scale"]))


def _bits(x):
    """A view that every torch can index: 8-bit floats as bytes."""
    return x.view(torch.uint8) if x.element_size() == 1 else x


def _places(s, page, first):
    """Of each packed row: its sequence and position, and the page and row in it that hold the position."""
    r = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(s["cu"][1:].long(), r, right=True)
    pos = first[b] + r - s["cu"][b]
    return pos, s["table"][b, pos // page].long(), pos % page


def _turned(x, heads, pos, theta):
    """Rows [n][heads * hd] in 32 bits, turned by their positions (angles in 64 bits)."""
    x = x.float().unflatten(1, (heads, -1))
    if not theta:
        return x
    hd = x.shape[2]
    angle = pos.double()[:, None, None] * theta ** (-2.0 * torch.arange(hd // 2, device="cuda", dtype=torch.float64) / hd)
    cos, sin = angle.cos().float(), angle.sin().float()
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=2)


def _store(cache, scale, x, slot, off, first_slot, kept):
    """Rows x [n][heads][hd] into their places of the cache."""
    if scale is None:
        cache[slot, :, off] = x.to(cache.dtype)
        return
    top = LARGEST["e4m3" if cache.dtype == torch.float8_e4m3fn else "e5m2"]
    amax = x.abs().amax(dim=2)
    need = torch.zeros_like(scale).scatter_reduce_(0, slot[:, None].expand_as(amax), amax, "amax")
    need = torch.exp2(torch.ceil(torch.log2((need.double() / top).clamp(min=2.0 ** -64)))).float()
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device="cuda")
    touched[slot] = True
    count = torch.zeros(scale.shape[0], dtype=torch.int64, device="cuda")
    count[first_slot] = kept  # rows of a page that an earlier step stored
    new = torch.where(touched[:, None], torch.where(count[:, None] > 0, torch.maximum(need, scale), need), scale)
    # rows that were there, in units of the new scale
    old = _bits(cache)[first_slot]
    again = (old.view(cache.dtype).float() * (scale / new)[first_slot][:, :, None, None]).to(cache.dtype).view(torch.uint8)
    there = torch.arange(cache.shape[2], device="cuda")[None, :] < kept[:, None]
    _bits(cache)[first_slot] = torch.where(there[:, None, :, None], again, old)
    _bits(cache)[slot, :, off] = (x / new[slot][:, :, None]).clamp(-top, top).to(cache.dtype).view(torch.uint8)
    scale.copy_(new)


def _append(s):
    c, n = s["case"], s["rows"]
    first = s["lengths"].long() - (s["cu"][1:] - s["cu"][:-1])
    pos, slot, off = _places(s, c["page"], first)
    first_slot = s["table"].long().gather(1, (first // c["page"])[:, None])[:, 0]
    kept = first % c["page"]
    _store(s["k_cache"], s["k_scale"], _turned(s["k"][:n], c["Hkv"], pos, c["theta"]), slot, off, first_slot, kept)
    _store(s["v_cache"], s["v_scale"], _turned(s["v"][:n], c["Hkv"], pos, 0.0), slot, off, first_slot, kept)
    if c["turn_q"]:
        s["q_out"][:n] = _turned(s["q"][:n], c["H"], pos, c["theta"]).flatten(1).to(s["q_out"].dtype)
    return [x for x in (s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["q_out"]) if x is not None]


def _paged(s, cache, scale):
    """Every sequence's pages in order, in 32 bits: [sequences][heads][tokens][hd]."""
    t = s["table"].clamp(min=0).long()
    x = _bits(cache)[t].view(cache.dtype).float()
    if scale is not None:
        x = x * scale[t][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _decode(s):
    c = s["case"]
    G, Lq, hd = c["H"] // c["Hkv"], c["Lq"], c["hd"]
    q = s["q"].float().view(c["B"], Lq, c["Hkv"], G, hd).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = torch.matmul(q, _paged(s, s["k_cache"], s["k_scale"]).transpose(2, 3)) * (1.0 / math.sqrt(hd))
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    j = torch.arange(x.shape[3], device="cuda")[None, None, :]
    p = (s["lengths"].long()[:, None] - Lq + torch.arange(Lq, device="cuda")).repeat(1, G)[:, :, None]
    seen = (j <= p) & (j < s["lengths"].long()[:, None, None])
    if c["window"]:
        seen = seen & (j > p - c["window"])
    seen = seen[:, None]
    x = x.masked_fill(~seen, -math.inf)
    m = x.amax(dim=3, keepdim=True)
    e = torch.where(seen, torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m)), torch.zeros_like(x))
    l = e.sum(dim=3, keepdim=True)
    o = torch.matmul(e, _paged(s, s["v_cache"], s["v_scale"])) / torch.where(l > 0, l, torch.ones_like(l))
    o = o.unflatten(2, (G, Lq)).permute(0, 3, 1, 2, 4).reshape(c["B"], Lq, c["H"] * hd)
    lse = (m + torch.log(l)).reshape(c["B"], c["H"], Lq)
    return [o.to(FLOATS[c["dt"]]), lse]


def _gather(s):
    c = s["case"]
    _, slot, off = _places(s, c["page"], torch.zeros_like(s["lengths"].long()))

    def read(cache, scale):
        x = _bits(cache)[slot, :, off].view(cache.dtype).float()
        x = x if scale is None else x * scale[slot][:, :, None]
        return x.flatten(1).to(FLOATS[c["dt"]])

    return [read(s["k_cache"], s["k_scale"]), read(s["v_cache"], s["v_scale"])]


# ------------------------------------------------------- in 64 bits, apart
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "decode": _exact_decode, "gather": _exact_gather}[case["op"]](s)


def _tokens(s, b, n, cache, scale):
    """The first n tokens of sequence b in 64 bits: [heads][n][hd]."""
    page = cache.shape[2]
    ids = s["table"][b, :(n + page - 1) // page].tolist()
    got = [cache[i].double() * (scale[i].double()[:, None, None] if scale is not None else 1.0) for i in ids]
    return torch.cat(got, dim=1)[:, :n]


def _exact_decode(s):
    c = s["case"]
    H, Hkv, Lq, hd = c["H"], c["Hkv"], c["Lq"], c["hd"]
    o = torch.zeros((c["B"], Lq, H, hd), dtype=torch.float64, device="cuda")
    lse = torch.full((c["B"], H, Lq), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lengths"].tolist()):
        k, v = _tokens(s, b, n, s["k_cache"], s["k_scale"]), _tokens(s, b, n, s["v_cache"], s["v_scale"])
        for i in range(Lq):
            at = n - Lq + i
            if at < 0:
                continue
            low = max(0, at + 1 - c["window"]) if c["window"] else 0
            q = s["q"][b, i].double().view(Hkv, H // Hkv, hd)
            z = torch.einsum("ghd,gnd->ghn", q, k[:, low:at + 1]) / math.sqrt(hd)
            z = c["softcap"] * torch.tanh(z / c["softcap"]) if c["softcap"] else z
            total = torch.logsumexp(z, dim=2)
            o[b, i] = torch.einsum("ghn,gnd->ghd", torch.exp(z - total[..., None]), v[:, low:at + 1]).reshape(H, hd)
            lse[b, :, i] = total.reshape(H)
    return [o.reshape(c["B"], Lq, H * hd), lse]


def _exact_gather(s):
    found = []
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        rows = [_tokens(s, b, n, cache, scale).transpose(0, 1).flatten(1) for b, n in enumerate(s["lengths"].tolist())]
        found.append(torch.cat(rows))
    return found


def _exact_append(s):
    c = s["case"]
    page, hd, cu, lengths, table = c["page"], c["hd"], s["cu"].tolist(), s["lengths"].tolist(), s["table"].tolist()

    def turn(x, heads, pos):
        z = torch.complex(*x.double().view(len(pos), heads, 2, hd // 2).unbind(2))
        freq = torch.tensor([c["theta"] ** (-2.0 * i / hd) for i in range(hd // 2)], dtype=torch.float64, device="cuda")
        z = z * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), pos.double()[:, None] * freq)[:, None]
        return torch.cat([z.real, z.imag], dim=2)

    def stored(x, cache, scale, turning):
        out, sc = cache.double(), None if scale is None else scale.double().clone()
        for b, n in enumerate(lengths):
            new = x[cu[b]:cu[b + 1]]
            first = n - len(new)
            pos = torch.arange(first, n, device="cuda")
            new = turn(new, c["Hkv"], pos) if turning else new.double().view(len(new), c["Hkv"], hd)
            for j in range(first // page, (n - 1) // page + 1):
                lo, hi, i = max(first, j * page), min(n, (j + 1) * page), table[b][j]
                part, at = new[lo - first:hi - first].transpose(0, 1), lo - j * page
                if sc is None:
                    out[i, :, at:at + hi - lo] = part
                    continue
                need = part.abs().amax(dim=(1, 2)) / LARGEST[c["cache"]]
                step = torch.exp2(torch.ceil(torch.log2(need.clamp(min=2.0 ** -64))))
                if at:
                    step = torch.maximum(step, sc[i])
                    out[i, :, :at] *= (sc[i] / step)[:, None, None]
                sc[i] = step
                out[i, :, at:at + hi - lo] = part / step[:, None, None]
        return out, sc

    k, ks = stored(s["k"][:s["rows"]], s["k_cache"], s["k_scale"], c["theta"] > 0)
    v, vs = stored(s["v"][:s["rows"]], s["v_cache"], s["v_scale"], False)
    found = [k, v] + ([ks, vs] if ks is not None else [])
    if c["turn_q"]:
        q = s["q_out"].double()
        for b, n in enumerate(lengths):
            pos = torch.arange(n - (cu[b + 1] - cu[b]), n, device="cuda")
            q[cu[b]:cu[b + 1]] = turn(s["q"][cu[b]:cu[b + 1]], c["H"], pos).flatten(1)
        found.append(q)
    return found
