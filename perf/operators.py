"""Cases for measuring the paged key-value cache operators: the per-head norm with rotation, the cache's
write and read, and the attention of one new token over it.

The cache is a pool of pages.  A page holds page_size positions of every KV head; for one page and head the
codes of all positions come first (fp16 values, Q8_0 bytes, or Q4_0 nibble pairs), then one fp16 scale for
each position and 32 values.  A table gives each sequence's pages in order."""
import math
import random

import torch

own = False

F16, Q4_0, Q8_0 = 1, 2, 8
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token of an 8B-shaped model (32 query heads, 8 KV heads): latency
        {"name": "rope one token", "op": "rope", "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "halves": False,
         "far": 2048, "pad": 0},
        # a batch of decoded tokens, small heads, part of each head rotated, some rows of the batch unused
        {"name": "rope ragged batch", "op": "rope", "tokens": 173, "hq": 20, "hkv": 5, "d": 64, "rot": 48,
         "halves": True, "far": 8192, "pad": 13},
        # a long prompt of a 70B-shaped model (64 query heads), positions far out
        {"name": "rope long prompt", "op": "rope", "tokens": 8192, "hq": 64, "hkv": 8, "d": 128, "rot": 128,
         "halves": True, "far": 131072, "pad": 0},
        # one new token written and read back: latency
        {"name": "cache one token", "op": "cache", "type": Q8_0, "tokens": 1, "hkv": 8, "d": 128, "page": 64,
         "seqs": 1, "pad": 0, "write": True},
        # tokens of several sequences (prompts being filled next to decoding ones), fp16 cache, odd count
        {"name": "cache ragged batch", "op": "cache", "type": F16, "tokens": 1531, "hkv": 4, "d": 256, "page": 16,
         "seqs": 37, "pad": 21, "write": True},
        # a prompt of one sequence written in 4 bits and read back
        {"name": "cache long prompt", "op": "cache", "type": Q4_0, "tokens": 16384, "hkv": 8, "d": 128, "page": 64,
         "seqs": 1, "pad": 0, "write": True},
        # a shared prefix read back from the cache
        {"name": "cache prefix read", "op": "cache", "type": Q8_0, "tokens": 24001, "hkv": 8, "d": 128, "page": 32,
         "seqs": 3, "pad": 0, "write": False},
        # the first tokens after a short prompt, one sequence: latency
        {"name": "attend short", "op": "attend", "type": F16, "hq": 32, "hkv": 8, "d": 128, "page": 16, "seqs": 1,
         "longest": 145, "even": True, "lens": 1},
        # one sequence of a 70B-shaped model at the context of this repository's 70B workload
        {"name": "attend one sequence", "op": "attend", "type": Q8_0, "hq": 64, "hkv": 8, "d": 128, "page": 64,
         "seqs": 1, "longest": 2049, "even": True, "lens": 1},
        # a serving batch: sequences of very different lengths, some just admitted (length 0)
        {"name": "attend ragged batch", "op": "attend", "type": Q8_0, "hq": 32, "hkv": 8, "d": 128, "page": 32,
         "seqs": 64, "longest": 8191, "even": False, "lens": 5},
        # a long document, one sequence, fp16 cache
        {"name": "attend long", "op": "attend", "type": F16, "hq": 32, "hkv": 8, "d": 128, "page": 64, "seqs": 1,
         "longest": 131071, "even": True, "lens": 1},
        # wide heads that share one KV head sixteenfold, 4-bit cache
        {"name": "attend wide heads", "op": "attend", "type": Q4_0, "hq": 32, "hkv": 2, "d": 256, "page": 48,
         "seqs": 24, "longest": 12000, "even": False, "lens": 9},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(("rope", "cache", "attend", "attend"))
    d = rng.choice((64, 128, 128, 256))
    hkv = rng.randint(1, 8)
    if op == "rope":
        group = rng.choice((1, 2, 4, 5, 8))
        tokens = _log(rng, 1, 8192 * 72 * 128 // ((group + 1) * hkv * d) // 2)
        rot = d if rng.random() < 0.6 else 2 * rng.randint(1, d // 2)
        return {"op": op, "tokens": min(tokens, 16384), "hq": group * hkv, "hkv": hkv, "d": d, "rot": rot,
                "halves": rng.random() < 0.5, "far": _log(rng, 16, 131072), "pad": rng.choice((0, 0, 1, 7))}
    kind = rng.choice((F16, Q8_0, Q4_0))
    page = 16 * rng.choice((1, 2, 3, 4, 8, 16))
    if op == "cache":
        tokens = _log(rng, 1, min(24000, 24000 * 8 * 128 // (hkv * d)))
        return {"op": op, "type": kind, "tokens": tokens, "hkv": hkv, "d": d, "page": page,
                "seqs": rng.randint(1, max(1, min(40, tokens // 4))), "pad": rng.choice((0, 0, 1, 9)),
                "write": rng.random() < 0.7}
    seqs = _log(rng, 1, 96)
    longest = _log(rng, 1, min(131071, 131071 * 8 * 128 // (hkv * d * seqs) // 2))
    return {"op": op, "type": kind, "hq": hkv * rng.choice((1, 2, 3, 4, 8, 12)), "hkv": hkv, "d": d, "page": page,
            "seqs": seqs, "longest": longest, "even": rng.random() < 0.3, "lens": rng.randint(1, 10 ** 6)}


def _lens(case):
    """Lengths of the sequences of an attention case: the longest, and others spread over the logarithm, an
    empty one among them where there are many."""
    n, longest = case["seqs"], case["longest"]
    if case["even"]:
        return [longest] * n
    r = random.Random(case["lens"])
    lens = [_log(r, 1, longest) for _ in range(n)]
    lens[r.randrange(n)] = longest
    if n >= 8:
        lens[r.randrange(n)] = 0
    return lens


def _row_bytes(kind, d):
    return {F16: 2 * d, Q8_0: d + d // 16, Q4_0: d // 2 + d // 16}[kind]


def _token_slots(case):
    """(sequence, position) of each token of a cache case, unused rows last: the tokens of a sequence follow on
    its earlier ones."""
    n, seqs = case["tokens"], case["seqs"]
    share = [n // seqs + (i < n % seqs) for i in range(seqs)]
    seq = [i for i in range(seqs) for _ in range(share[i])]
    pos = [(7 * i) % 41 + p for i in range(seqs) for p in range(share[i])]
    return seq + [0] * case["pad"], pos + [-1] * case["pad"]


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["hq"] + case["hkv"]) * case["d"]
        return {"bytes": 8 * n + 4 * case["tokens"] + 8 * case["d"], "flops": 7 * n}
    if case["op"] == "cache":
        rows = 2 * case["tokens"] * case["hkv"]
        row = _row_bytes(case["type"], case["d"]) + 4 * case["d"]
        return {"bytes": rows * row * (2 if case["write"] else 1) + 8 * case["tokens"],
                "flops": rows * case["d"] * (5 if case["write"] else 1)}
    total = sum(_lens(case))
    return {"bytes": 2 * total * case["hkv"] * _row_bytes(case["type"], case["d"])
            + 8 * case["seqs"] * case["hq"] * case["d"] + 4 * total // case["page"],
            "flops": 4 * total * case["hq"] * case["d"]}


# ------------------------------------------------------------------ the cache's values
def _quantise(w, kind):
    """Codes (uint8, [..., D or D/2]) and fp16 scales ([..., D/32]) of rows w [..., D]."""
    b = w.reshape(*w.shape[:-1], w.shape[-1] // 32, 32)
    a = b.abs()
    top = a.amax(-1, keepdim=True)
    if kind == Q8_0:
        d = top / torch.full((), 127.0, device=w.device)
    else:
        first = torch.where(a == top, torch.arange(32, device=w.device), 32).amin(-1, keepdim=True)
        d = torch.gather(b, -1, first) * -0.125
    x = torch.where(top > 0, b / d, 0.0)
    low = x.abs().floor()
    q = torch.where(x.abs() - low >= 0.5, low + 1, low) * torch.sign(x)
    if kind == Q8_0:
        codes = q.clamp(-127, 127).to(torch.int8).view(torch.uint8).reshape(*w.shape)
    else:
        q = (q + 8).clamp(0, 15).to(torch.uint8)
        codes = (q[..., :16] | (q[..., 16:] << 4)).reshape(*w.shape[:-1], w.shape[-1] // 2)
    return codes, d[..., 0].half()


def _values(codes, scales, kind, dtype=torch.float32):
    if kind == Q8_0:
        q = codes.view(torch.int8).to(dtype)
    else:
        c = codes.reshape(*scales.shape, 16)
        q = torch.cat([c & 15, c >> 4], -1).to(dtype).reshape(*scales.shape[:-1], scales.shape[-1] * 32) - 8
    return (q.reshape(*scales.shape, 32) * scales.to(dtype)[..., None]).reshape(q.shape)


def _parts(pool, s):
    """Codes [pages, heads, page, ...] and scales [pages, heads, page, D/32] of a pool, as views of it."""
    n, h, ps, d, kind = s["n_pages"], s["hkv"], s["page"], s["d"], s["type"]
    if kind == F16:
        return pool.view(torch.float16).view(n, h, ps, d), None
    p = pool.view(n, h, ps * _row_bytes(kind, d))
    c = d if kind == Q8_0 else d // 2
    return (p[:, :, :ps * c].unflatten(2, (ps, c)), p[:, :, ps * c:].view(torch.float16).unflatten(2, (ps, d // 32)))


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = dict(case)
    if case["op"] == "rope":
        n = case["tokens"] + case["pad"]
        wide = (case["hq"] + 2 * case["hkv"]) * case["d"]  # q, k and v of a token side by side, as a projection leaves them
        x = torch.randn(n, wide, generator=g, device=DEV) * torch.exp(
            torch.randn(n, 1, generator=g, device=DEV))
        pos = torch.randint(0, case["far"], (n,), generator=g, device=DEV, dtype=torch.int32)
        pos[case["tokens"]:] = -1
        nq, nk = case["hq"] * case["d"], case["hkv"] * case["d"]
        s |= {"x": x, "q": x[:, :nq], "k": x[:, nq:nq + nk], "pos": pos, "stride": wide,
              "wq": 1 + 0.1 * torch.randn(case["d"], generator=g, device=DEV),
              "wk": 1 + 0.1 * torch.randn(case["d"], generator=g, device=DEV)}
        y = torch.zeros(n, wide, device=DEV)
        s |= {"y": y, "q_out": y[:, :nq], "k_out": y[:, nq:nq + nk]}
        return s
    ps, d, hkv, kind = case["page"], case["d"], case["hkv"], case["type"]
    if case["op"] == "cache":
        seq, pos = _token_slots(case)
        lens = [0] * case["seqs"]
        for a, b in zip(seq, pos):
            lens[a] = max(lens[a], b + 1)
    else:
        lens = _lens(case)
    used = [-(-n // ps) for n in lens]
    s["n_pages"] = sum(used) + 3
    s["max_pages"] = max(1, max(used)) + 1
    order = torch.randperm(s["n_pages"], generator=g, device=DEV).to(torch.int32)
    width = torch.tensor(used, device=DEV)
    taken = torch.arange(s["max_pages"], device=DEV)[None] < width[:, None]
    table = torch.full((case["seqs"], s["max_pages"]), -1, dtype=torch.int32, device=DEV)
    table[taken] = order[:sum(used)]
    s["table"] = table
    size = s["n_pages"] * hkv * ps * _row_bytes(kind, d)
    for name in ("k_pages", "v_pages"):
        pool = torch.zeros(size, dtype=torch.uint8, device=DEV)
        codes, scales = _parts(pool, s)
        if case["op"] == "attend" or not case["write"]:
            piece = max(1, (1 << 26) // (hkv * ps * d))
            for i in range(0, s["n_pages"], piece):
                w = torch.randn(min(piece, s["n_pages"] - i), hkv, ps, d, generator=g, device=DEV)
                if kind == F16:
                    codes[i:i + piece] = w.half()
                else:
                    c, e = _quantise(w, kind)
                    codes[i:i + piece], scales[i:i + piece] = c, e
        s[name] = pool
    if case["op"] == "cache":
        n = len(seq)
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device=DEV)
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device=DEV)
        s["k"] = torch.randn(n, hkv * d, generator=g, device=DEV)
        s["v"] = torch.randn(n, hkv * d, generator=g, device=DEV)
        s["k_out"], s["v_out"] = torch.zeros(n, hkv * d, device=DEV), torch.zeros(n, hkv * d, device=DEV)
    else:
        s["len"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = torch.randn(case["seqs"], case["hq"] * d, generator=g, device=DEV) * 1.5
        s["out"] = torch.zeros(case["seqs"], case["hq"] * d, device=DEV)
        s["scale"] = 1 / math.sqrt(d)
    if own:
        import quantized_weight_gemv_dequant_b200 as ntx

        s["kv"] = ntx.make_paged_kv(kind, hkv, d, ps, s["n_pages"], s["k_pages"], s["v_pages"], table, case["seqs"],
                                    s["max_pages"])
        if case["op"] == "attend":
            s["ws_bytes"] = ntx.ntx_attn_paged_workspace_bytes(s["kv"], case["hq"])
            s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def _plain_rope(s):
    d, rot, n = s["d"], s["rot"], s["pos"].shape[0]
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    angle = s["pos"].double()[:, None] * torch.pow(500000.0, -2 * i / rot)
    c, z = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    keep = (s["pos"] >= 0)[:, None]
    for x, w, out in ((s["q"], s["wq"], s["q_out"]), (s["k"], s["wk"], s["k_out"])):
        x = x.unflatten(1, (-1, d))
        y = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        if s["halves"]:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            y = torch.cat([a * c - b * z, a * z + b * c, y[..., rot:]], -1)
        else:
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            y = torch.cat([torch.stack([a * c - b * z, a * z + b * c], -1).flatten(-2), y[..., rot:]], -1)
        out.copy_(torch.where(keep, y.flatten(1), out))
    return {"q": s["q_out"], "k": s["k_out"]}


def _plain_cache(s):
    kind, d = s["type"], s["d"]
    n, live = s["pos"].shape[0], s["pos"] >= 0
    pos = s["pos"].clamp(min=0).long()
    page = s["table"][s["seq"].long(), pos // s["page"]].long()
    at = pos % s["page"]
    out = {}
    for name in ("k", "v"):
        codes, scales = _parts(s[name + "_pages"], s)
        if s["write"]:
            w = s[name].view(n, -1, d)
            p, r = page[live], at[live]
            if kind == F16:
                codes[p, :, r] = w[live].half()
            else:
                codes[p, :, r], scales[p, :, r] = _quantise(w[live], kind)
        got = codes[page, :, at]
        got = got.float() if kind == F16 else _values(got, scales[page, :, at], kind)
        s[name + "_out"].copy_(torch.where(live[:, None], got.flatten(1), s[name + "_out"]))
        out[name] = s[name + "_out"]
    return out


def _plain_attend(s):
    kind, d, ps, n, hkv = s["type"], s["d"], s["page"], s["seqs"], s["hkv"]
    table = s["table"].clamp(min=0).long()
    live = torch.arange(s["max_pages"] * ps, device=DEV)[None] < s["len"][:, None]
    q = (s["q"] * s["scale"]).view(n, hkv, -1, d)
    rows = []
    for name in ("k_pages", "v_pages"):
        codes, scales = _parts(s[name], s)
        x = codes[table].float() if kind == F16 else _values(codes[table], scales[table], kind)
        rows.append(x.transpose(1, 2).flatten(2, 3))  # [sequence, head, position, D]
    score = torch.matmul(q, rows[0].transpose(2, 3)).masked_fill(~live[:, None, None], -torch.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isfinite(top), top, 0.0))
    total = p.sum(-1, keepdim=True)
    s["out"].copy_((torch.matmul(p, rows[1]) / torch.where(total > 0, total, 1.0)).reshape(n, -1))
    return s["out"]


def run(s):
    if not own:
        return {"rope": _plain_rope, "cache": _plain_cache, "attend": _plain_attend}[s["op"]](s)
    import quantized_weight_gemv_dequant_b200 as ntx

    if s["op"] == "rope":
        ntx.ntx_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["stride"], s["stride"], s["wq"], s["wk"],
                             s["pos"], s["pos"].shape[0], s["hq"], s["hkv"], s["d"], s["rot"],
                             ntx.NTX_ROPE_HALVES if s["halves"] else ntx.NTX_ROPE_ADJACENT, 500000.0, 1e-6)
        return {"q": s["q_out"], "k": s["k_out"]}
    if s["op"] == "cache":
        n, stride = s["pos"].shape[0], s["hkv"] * s["d"]
        if s["write"]:
            ntx.ntx_kv_append(s["kv"], s["k"], s["v"], stride, stride, s["seq"], s["pos"], n)
        ntx.ntx_kv_read(s["kv"], s["k_out"], s["v_out"], stride, stride, s["seq"], s["pos"], n)
        return {"k": s["k_out"], "v": s["v_out"]}
    ntx.ntx_attn_decode_paged(s["kv"], s["q"], s["hq"] * s["d"], s["out"], s["hq"], s["len"], s["scale"], s["ws"],
                              s["ws_bytes"])
    return s["out"]


# ------------------------------------------------------------------ in 64 bits
def _exact_rope(s):
    d, rot = s["d"], s["rot"]
    out = {}
    for name, h in (("q", s["hq"]), ("k", s["hkv"])):
        y = torch.zeros(s["pos"].shape[0], h, d, dtype=torch.float64, device=DEV)
        for lo in range(0, y.shape[0], 1024):
            x = s[name][lo:lo + 1024].double().reshape(-1, h, d)
            pos = s["pos"][lo:lo + 1024].double()
            x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / d + 1e-6) * s["w" + name].double()
            e = torch.arange(rot // 2, device=DEV)
            first, second = (e, e + rot // 2) if s["halves"] else (2 * e, 2 * e + 1)
            turn = torch.polar(torch.ones_like(pos)[:, None].expand(-1, rot // 2),
                               pos[:, None] * torch.exp(-2 * e.double() / rot * math.log(500000.0)))[:, None]
            z = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = z.real, z.imag
            y[lo:lo + 1024] = torch.where((pos >= 0)[:, None, None], x, 0.0)
        out[name] = y.flatten(1)
    return out


def _exact_block(w, kind):
    """The values that rows of 32 stand for in the cache.  The fp32 and fp16 roundings here are the format's."""
    w = w.double()
    big = w.abs().max(-1, keepdim=True).values
    if kind == Q8_0:
        d, lo, hi = (big / torch.full_like(big, 127)).float().double(), -127, 127
    else:
        top = torch.where((w == big).int().cumsum(-1).gt(0).sum(-1, keepdim=True)
                          > (w == -big).int().cumsum(-1).gt(0).sum(-1, keepdim=True), big, -big)
        d, lo, hi = top / -8, -8, 7
    x = (w / torch.where(d == 0, 1.0, d)).float().double()
    q = torch.copysign(torch.floor(x.abs() + 0.5), x).clamp(lo, hi)
    return q * d.float().half().double()


def _exact_cache(s):
    kind, d, ps, n = s["type"], s["d"], s["page"], s["pos"].shape[0]
    out = {}
    live = s["pos"] >= 0
    for name in ("k", "v"):
        if s["write"]:
            w = s[name]
            y = w.half().double() if kind == F16 else _exact_block(w.view(n, -1, 32), kind).view(n, -1)
        else:
            where = s["table"][s["seq"].long(), s["pos"].clamp(min=0).long() // ps].long()
            y = _exact_rows(s[name + "_pages"], s, where, s["pos"].clamp(min=0).long() % ps)
        out[name] = torch.where(live[:, None], y, 0.0)
    return out


def _exact_rows(pool, s, page, at):
    """Rows [n, heads * D] of (page, place in the page), decoded byte by byte from the pool."""
    kind, d, ps, h = s["type"], s["d"], s["page"], s["hkv"]
    rb = _row_bytes(kind, d)
    base = (page[:, None] * h + torch.arange(h, device=DEV)) * (ps * rb)
    e = torch.arange(d, device=DEV)

    def half_at(where):
        raw = pool[where].to(torch.int16) | (pool[where + 1].to(torch.int16) << 8)
        return raw.view(torch.float16).double()

    if kind == F16:
        return half_at(base[..., None] + at[:, None, None] * rb + 2 * e).flatten(1)
    wide = d if kind == Q8_0 else d // 2
    scale = half_at(base[..., None] + ps * wide + at[:, None, None] * (d // 16) + 2 * (e // 32))
    if kind == Q8_0:
        q = pool[base[..., None] + at[:, None, None] * wide + e].double()
        q = torch.where(q > 127, q - 256, q)
    else:
        byte = pool[base[..., None] + at[:, None, None] * wide + 16 * (e // 32) + e % 16]
        q = torch.where(e % 32 < 16, byte % 16, byte // 16).double() - 8
    return (q * scale).flatten(1)


def _exact_attend(s):
    d, ps, hkv = s["d"], s["page"], s["hkv"]
    out = torch.zeros(s["seqs"], s["hq"], d, dtype=torch.float64, device=DEV)
    for i, n in enumerate(s["len"].tolist()):
        if n == 0:
            continue
        q = s["q"][i].double().view(hkv, -1, d) * s["scale"]
        best, weight, sum_v = None, None, None
        for lo in range(0, n, 8192):
            p = torch.arange(lo, min(n, lo + 8192), device=DEV)
            page = s["table"][i, p // ps].long()
            k, v = (_exact_rows(s[name], s, page, p % ps).view(-1, hkv, d).transpose(0, 1)
                    for name in ("k_pages", "v_pages"))
            score = torch.einsum("hgd,hpd->hgp", q, k)
            lse = torch.logsumexp(score, -1, keepdim=True)
            part = torch.einsum("hgp,hpd->hgd", torch.exp(score - lse), v)
            if best is None:
                best, sum_v = lse, part
            else:
                both = torch.logaddexp(best, lse)
                sum_v = sum_v * torch.exp(best - both) + part * torch.exp(lse - both)
                best = both
        out[i] = sum_v.reshape(-1, d)
    return out.flatten(1)


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "cache": _exact_cache, "attend": _exact_attend}[case["op"]](s)
