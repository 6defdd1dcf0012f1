"""Cases of the attention-side operators and of the adapter product, in plain torch and as calls of the library.

A serving step of one decoder layer: the q/k/v product with the requests' low-rank
adapters, norm and rotation of q and k with the INT4 append into the paged cache,
attention of the new tokens over the cache, and the adapter product again. Head
layouts and matrices are those of the Llama-3-70B (64 query and 8 KV heads of 128
channels, 8192 channels) and Llama-3-8B (32 and 8 heads, 4096 channels) shapes.
"""

from __future__ import annotations

import math
import random

import torch

own = False


def _lib():
    import w4a16_decode_amd as q4

    return q4


# ---- cases ---------------------------------------------------------------------


def listed():
    return [
        # one decoded token of the 8B shape, q and k norms: pure launch latency
        {"name": "rope_decode_8b", "op": "rope", "tokens": 1, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "norm": True},
        # a long prompt chunk of the 70B shape, an odd token count: bandwidth
        {"name": "rope_prefill_70b", "op": "rope", "tokens": 8191, "hq": 64, "hkv": 8, "d": 128, "rot": 128,
         "interleaved": False, "norm": True},
        # 16 sequences decode one token each (70B shape, no norms): latency, scattered pages
        {"name": "append_decode_b16", "op": "append", "tokens": 16, "hq": 64, "hkv": 8, "d": 128, "group": 128,
         "page": 16, "rot": 128, "interleaved": False, "norm": False},
        # a prompt chunk of the 8B shape with norms, partial interleaved rotation, finer groups
        {"name": "append_prefill_8b", "op": "append", "tokens": 4097, "hq": 32, "hkv": 8, "d": 128, "group": 64,
         "page": 64, "rot": 64, "interleaved": True, "norm": True},
        # one request decodes early in its answer (8B shape): latency
        {"name": "attn_decode_short", "op": "attn", "seqs": 1, "new": 1, "max_kv": 129, "hq": 32, "hkv": 8, "d": 128,
         "group": 128, "page": 16, "window": 0},
        # a full decode batch with ragged contexts (70B shape): the cache's bytes
        {"name": "attn_decode_b48_70b", "op": "attn", "seqs": 48, "new": 1, "max_kv": 8191, "hq": 64, "hkv": 8,
         "d": 128, "group": 128, "page": 32, "window": 0},
        # few requests with long contexts (8B shape): the context has to be split
        {"name": "attn_decode_long", "op": "attn", "seqs": 3, "new": 1, "max_kv": 100003, "hq": 32, "hkv": 8,
         "d": 128, "group": 64, "page": 64, "window": 0},
        # chunked prefill of four requests over longer contexts (70B shape): matrix work
        {"name": "attn_chunk_70b", "op": "attn", "seqs": 4, "new": 509, "max_kv": 8190, "hq": 64, "hkv": 8, "d": 128,
         "group": 128, "page": 32, "window": 0},
        # a sliding window over 64-channel heads, groups of 32
        {"name": "attn_chunk_window", "op": "attn", "seqs": 2, "new": 1025, "max_kv": 6001, "hq": 32, "hkv": 8,
         "d": 64, "group": 32, "page": 48, "window": 2048},
        # one token, one adapter, the 8B attention output projection: latency
        {"name": "lora_b1_8b", "op": "lora", "rows": 1, "out": 4096, "in": 4096, "group": 128, "rank": 16,
         "adapters": 4},
        # a decode batch of mixed adapters on the 70B q/k/v product: the weights' bytes
        {"name": "lora_b13_qkv_70b", "op": "lora", "rows": 13, "out": 10240, "in": 8192, "group": 128, "rank": 16,
         "adapters": 8},
        # a mixed batch of prompt chunks on a 70B up projection
        {"name": "lora_b192_70b", "op": "lora", "rows": 192, "out": 28672, "in": 8192, "group": 128, "rank": 32,
         "adapters": 6},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "lora"])
    hkv = rng.choice([4, 8])
    d = rng.choice([64, 128, 128, 256])
    hq = hkv * rng.choice([1, 4, 7, 8])
    if op == "rope":
        return {"op": op, "tokens": _log(rng, 1, 4096), "hq": hq, "hkv": hkv, "d": d,
                "rot": d // rng.choice([1, 1, 2]), "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.6}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 4096), "hq": hq, "hkv": hkv, "d": d,
                "group": rng.choice([g for g in (32, 64, 128) if g <= d]), "page": 16 * rng.choice([1, 2, 3, 8]),
                "rot": d // rng.choice([1, 1, 2]), "interleaved": rng.random() < 0.4, "norm": rng.random() < 0.6}
    if op == "attn":
        kind = rng.choice(["decode", "decode", "few", "chunk"])
        seqs = _log(rng, 1, 32) if kind == "decode" else rng.randint(1, 3)
        new = 1 if kind == "decode" else rng.randint(2, 9) if kind == "few" else _log(rng, 10, 500)
        max_kv = new + _log(rng, 1, 6000)
        return {"op": op, "seqs": seqs, "new": new, "max_kv": max_kv, "hq": hq, "hkv": hkv, "d": d,
                "group": rng.choice([g for g in (32, 64, 128) if g <= d]), "page": 16 * rng.choice([1, 2, 3, 8]),
                "window": rng.choice([0, 0, 0, _log(rng, 16, 2000)])}
    return {"op": op, "rows": _log(rng, 1, 128), "out": 16 * _log(rng, 16, 700) - rng.choice([0, 0, 5]),
            "in": 128 * _log(rng, 8, 64), "group": rng.choice([32, 64, 128, 128]), "rank": rng.choice([8, 16, 32, 64]),
            "adapters": _log(rng, 1, 12)}


def _lens(case):
    """Context lengths of the sequences: ragged, the first at the maximum."""
    rng = random.Random("%(seqs)d %(max_kv)d" % case)
    lo = max(case["new"], case["max_kv"] // 4)
    return [case["max_kv"]] + [rng.randint(lo, case["max_kv"]) for _ in range(case["seqs"] - 1)]


def _ids(case):
    """Adapter of each row: runs of rows of one request, some without an adapter."""
    rng = random.Random("%(rows)d %(adapters)d" % case)
    ids = []
    while len(ids) < case["rows"]:
        a = rng.randint(-1, case["adapters"] - 1) if ids else 0
        ids += [a] * (1 if case["rows"] <= 16 else rng.randint(1, 40))
    return ids[:case["rows"]]


def work(case):
    op = case["op"]
    if op in ("rope", "append"):
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        n = t * (hq + hkv) * d
        nbytes, flops = 4 * n + 4 * t * case["rot"] + 4 * t, 8 * n
        if op == "append":
            codes = d // 2 + 2 * (d // case["group"])
            # v is read too and k's rows are not written; codes and scales of k and v, and the values they stand for
            nbytes += t * hkv * (2 * codes + 4 * d) + 4 * t
            flops += 8 * 2 * t * hkv * d
        return {"bytes": nbytes, "flops": flops}
    if op == "attn":
        lens, new, w = _lens(case), case["new"], case["window"]
        pairs = sum(min(p + 1, w) if w else p + 1 for n in lens for p in range(n - new, n))
        keys = sum(min(n, w + new - 1) if w else n for n in lens)
        per_key = case["hkv"] * 2 * (case["d"] // 2 + 2 * (case["d"] // case["group"]))
        return {"bytes": keys * per_key + 4 * len(lens) * new * case["hq"] * case["d"] + 4 * keys // case["page"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    rows, n, k, r = case["rows"], case["out"], case["in"], case["rank"]
    ids = [a for a in _ids(case) if a >= 0]
    return {"bytes": n * k // 2 + 2 * n * (k // case["group"]) + 2 * rows * (n + k) + 2 * len(set(ids)) * r * (n + k),
            "flops": 2 * rows * n * k + 2 * len(ids) * r * (n + k)}


# ---- inputs ----------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _table(positions, rot):
    """cos and sin of position * 10000^(-2 i / rot), angles in 64 bits: [positions, rot / 2, 2]."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.stack((a.cos(), a.sin()), -1).float()


def _projected(g, tokens, heads, d):
    """Rows as a projection leaves them: a few channels much larger than the others."""
    return (_normal(g, tokens, heads, d) * torch.exp(0.5 * _normal(g, 1, heads, d))).half()


def _rope_inputs(case, seed):
    g = _gen(seed)
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    # the rows of one fused q/k/v product
    qkv = torch.cat((_projected(g, t, hq, d), _projected(g, t, hkv, d), _projected(g, t, hkv, d)), 1)
    first = 0 if t > 16 else 997 * (seed % 3)
    pos = first + torch.arange(t, device="cuda", dtype=torch.int32)
    norm = [(1 + 0.2 * _normal(g, d)).half() if case["norm"] else None for _ in range(2)]
    return {"qkv": qkv, "q": qkv[:, :hq], "k": qkv[:, hq:hq + hkv], "v": qkv[:, hq + hkv:], "positions": pos,
            "table": _table(first + t, case["rot"]), "q_weight": norm[0], "k_weight": norm[1], "eps": 1e-6}


def _slots(case, seed):
    """Cache slots of the new tokens: a chunk fills pages taken from all over the pool, decoded tokens sit anywhere."""
    g, t, page = _gen(seed + 1), case["tokens"], case["page"]
    if t <= 16:
        pages = 4 * t
        at = torch.randperm(pages, generator=g, device="cuda")[:t] * page
        return pages, (at + torch.randint(0, page, (t,), generator=g, device="cuda")).int()
    pages = -(-t // page) + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(t, device="cuda")
    return pages, (order[i // page] * page + i % page).int()


def _attn_inputs(case, seed):
    g, lens = _gen(seed), _lens(case)
    hkv, d, page = case["hkv"], case["d"], case["page"]
    blocks = -(-max(lens) // page)
    pages = len(lens) * blocks + 2
    table = torch.randperm(pages, generator=g, device="cuda")[:len(lens) * blocks].view(len(lens), blocks)
    rows = len(lens) * case["new"]
    channel = torch.exp(0.4 * _normal(g, 1, hkv, d))
    # every slot of the pool holds a token, as in a cache in use: what lies behind a length is another request's
    k = (_normal(g, pages * page, hkv, d) * channel).half()
    v = _normal(g, pages * page, hkv, d).half()
    return {"q": _normal(g, rows, case["hq"], d).half(), "k": k, "v": v, "pages": pages, "block_table": table.int(),
            "q_offsets": torch.arange(0, rows + 1, case["new"], device="cuda", dtype=torch.int32),
            "kv_lens": torch.tensor(lens, device="cuda", dtype=torch.int32), "new": case["new"], "max_kv": max(lens)}


def _lora_inputs(case, seed):
    g = _gen(seed)
    rows, n, k, r, a = case["rows"], case["out"], case["in"], case["rank"], case["adapters"]
    w = (_normal(g, n, k) / math.sqrt(k)).half()
    return {"w": w, "x": _normal(g, rows, k).half(), "ids": torch.tensor(_ids(case), device="cuda", dtype=torch.int32),
            "a": (_normal(g, a, r, k) / math.sqrt(k)).half(), "b": (0.1 * _normal(g, a, n, r)).half(),
            "scaling": torch.rand(a, generator=g, device="cuda") + 0.5}


def _rtn4(x, group):
    """Group-wise INT4 of the last axis: codes and float16 scales, decided in 64 bits."""
    y = x.view(*x.shape[:-1], -1, group)
    s = (y.abs().amax(-1).double() / 7).half()
    z = s.double()[..., None]
    codes = torch.where(z == 0, 0.0, (y.double() / z.where(z != 0, 1.0)).round().clamp(-8, 7))
    return codes.to(torch.int8).view(x.shape), s


def prepare(case, seed):
    op = case["op"]
    if op in ("rope", "append"):
        s = _rope_inputs(case, seed)
        if op == "append":
            pages, s["slots"] = _slots(case, seed)
            if own:
                s["cache"] = _lib().paged_kv_alloc(pages, case["page"], case["hkv"], case["d"], case["group"])
    elif op == "attn":
        s = _attn_inputs(case, seed)
        k, v = s.pop("k"), s.pop("v")
        if own:
            s["cache"] = _lib().paged_kv_alloc(s["pages"], case["page"], case["hkv"], case["d"], case["group"])
            _lib().paged_kv_append(k, v, s["cache"], torch.arange(len(k), device="cuda", dtype=torch.int32))
        else:
            s["k"], s["v"] = _rtn4(k, case["group"]), _rtn4(v, case["group"])
    else:
        s = _lora_inputs(case, seed)
        w = s.pop("w")
        if own:
            s["weight"] = _lib().quantize_pack(w, case["group"])
            s["adapters"] = _lib().LoraAdapters(s.pop("a"), s.pop("b"), s.pop("scaling"))
        else:
            s["codes"], s["scales"] = _rtn4(w, case["group"])
    return {"case": case, **s}


# ---- one pass -----------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        return _run_own(case, s)
    return {"rope": _rope, "append": _append, "attn": _attn, "lora": _lora}[case["op"]](case, s)


def _run_own(case, s):
    q4, op = _lib(), case["op"]
    if op == "rope":
        return q4.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["q_weight"], s["k_weight"], eps=s["eps"],
                               interleaved=case["interleaved"])
    if op == "append":
        q = q4.qk_norm_rope_append(s["q"], s["k"], s["v"], s["positions"], s["table"], s["cache"], s["slots"],
                                   s["q_weight"], s["k_weight"], eps=s["eps"], interleaved=case["interleaved"])
        return (q, *q4.paged_kv_dequant(s["cache"], s["slots"]))
    if op == "attn":
        return q4.paged_attention(s["q"], s["cache"], s["block_table"], s["q_offsets"], s["kv_lens"], s["new"],
                                  s["max_kv"], window=case["window"])
    return q4.gemm_lora(s["x"], s["weight"], s["adapters"], s["ids"])


def _norm_rope(x, weight, s, case, dtype):
    """RMS norm of each head and rotation of its first channels, unrounded."""
    h, rot = x.to(dtype), case["rot"]
    if weight is not None:
        h = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + s["eps"]) * weight.to(dtype)
    cs = s["table"][s["positions"].long()].to(dtype)[:, None]
    c, sn = cs[..., 0], cs[..., 1]
    if case["interleaved"]:
        a, b = h[..., 0:rot:2], h[..., 1:rot:2]
        turned = torch.stack((a * c - b * sn, b * c + a * sn), -1).flatten(-2)
    else:
        a, b = h[..., :rot // 2], h[..., rot // 2:rot]
        turned = torch.cat((a * c - b * sn, b * c + a * sn), -1)
    return torch.cat((turned, h[..., rot:]), -1)


def _rope(case, s):
    return (_norm_rope(s["q"], s["q_weight"], s, case, torch.float32).half(),
            _norm_rope(s["k"], s["k_weight"], s, case, torch.float32).half())


def _append(case, s):
    # k in 64 bits: it lies next to the borders of the 4-bit codes
    q = _norm_rope(s["q"], s["q_weight"], s, case, torch.float32).half()
    k = _norm_rope(s["k"], s["k_weight"], s, case, torch.float64).half()
    kv, scales = _rtn4(torch.cat((k, s["v"]), 1), case["group"])
    kv = (_spread(kv, scales)).half()
    return q, kv[:, :case["hkv"]].contiguous(), kv[:, case["hkv"]:].contiguous()


def _spread(codes, scales):
    """The float32 values that codes and their groups' scales stand for."""
    y = codes.float().view(*scales.shape, -1)
    return (y * scales.float()[..., None]).view(codes.shape)


def _attn(case, s):
    n, new, hkv, d, page = case["seqs"], case["new"], case["hkv"], case["d"], case["page"]
    ctx = s["block_table"].shape[1] * page

    def cached(codes, scales):
        pick = s["block_table"].long()
        x = _spread(codes.view(-1, page, hkv, d)[pick], scales.view(s["pages"], page, hkv, -1)[pick])
        return x.view(n, ctx, hkv, d).transpose(1, 2).contiguous()

    k, v = cached(*s["k"]), cached(*s["v"])
    q = s["q"].float().view(n, new, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)  # rows (head, token)
    p = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(d)
    key = torch.arange(ctx, device="cuda")
    at = (s["kv_lens"][:, None] - new + torch.arange(new, device="cuda"))[..., None]
    seen = (key <= at) & (key > at - (case["window"] or ctx + 1))
    p = p.view(n, hkv, -1, new, ctx).masked_fill_(~seen[:, None, None], -math.inf)
    p = (p - p.amax(-1, keepdim=True)).exp_()
    p = (p / p.sum(-1, keepdim=True)).view(n, hkv, -1, ctx)
    o = torch.matmul(p, v).view(n, hkv, -1, new, d)
    return o.permute(0, 3, 1, 2, 4).reshape(n * new, case["hq"], d).half()


def _lora(case, s):
    x = s["x"].float()
    y = x @ _spread(s["codes"], s["scales"]).t()
    at = s["ids"].long().clamp(min=0)
    t = torch.bmm(s["a"].float()[at], x[..., None])
    t = t * torch.where(s["ids"] >= 0, s["scaling"][at], 0.0)[:, None, None]
    return (y + torch.bmm(s["b"].float()[at], t).squeeze(-1)).half()


# ---- in 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    return {"rope": _exact_rope, "append": _exact_append, "attn": _exact_attn, "lora": _exact_lora}[case["op"]](case, seed)


def _exact_heads(x, weight, s, case):
    """One rotation matrix a pair: the pair as a complex number times exp(i angle)."""
    rot, y = case["rot"], x.double()
    if weight is not None:
        y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + s["eps"]) * weight.double()
    turn = torch.view_as_complex(s["table"].double().contiguous())[s["positions"].long()].unsqueeze(1)
    out = y.clone()
    if case["interleaved"]:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    else:
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    z = torch.complex(y[..., first], y[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


def _exact_rope(case, seed):
    s = _rope_inputs(case, seed)
    return tuple(_exact_heads(s[n], s[n + "_weight"], s, case) for n in "qk")


def _exact_append(case, seed):
    s, g = _rope_inputs(case, seed), case["group"]
    out = [_exact_heads(s["q"], s["q_weight"], s, case)]
    for x in (_exact_heads(s["k"], s["k_weight"], s, case).half().double(), s["v"].double()):
        parts = []
        for j in range(0, case["d"], g):  # the stored values, group by group
            y = x[..., j:j + g]
            step = (y.abs().max(-1, keepdim=True).values / 7).half().double()
            codes = torch.nan_to_num(torch.round(y / step)).clamp(-8, 7)
            parts.append(codes * step)
        out.append(torch.cat(parts, -1))
    return tuple(out)


def _exact_attn(case, seed):
    s, g, d = _attn_inputs(case, seed), case["group"], case["d"]
    lens, new, hkv = _lens(case), case["new"], case["hkv"]
    share = case["hq"] // hkv
    out = torch.zeros(len(lens) * new, case["hq"], d, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lens):
        t = torch.arange(n, device="cuda")
        at = s["block_table"][i].long()[t // case["page"]] * case["page"] + t % case["page"]
        kv = []
        for x in (s["k"][at], s["v"][at]):
            codes, scales = _rtn4(x, g)
            kv.append(codes.double() * scales.double().repeat_interleave(g, -1))
        pos = torch.arange(n - new, n, device="cuda")[:, None]
        hidden = (t > pos) | ((t <= pos - case["window"]) if case["window"] else t < 0)
        for h in range(hkv):
            kh, vh = kv[0][:, h].t().contiguous(), kv[1][:, h].contiguous()
            for j in range(h * share, (h + 1) * share):
                z = s["q"][i * new:(i + 1) * new, j].double() @ kh * d ** -0.5
                z[hidden] = -math.inf
                out[i * new:(i + 1) * new, j] = torch.softmax(z, -1) @ vh
    return out


def _exact_lora(case, seed):
    s, g = _lora_inputs(case, seed), case["group"]
    codes, scales = _rtn4(s["w"], g)
    w = codes.double() * scales.double().repeat_interleave(g, -1)
    y = s["x"].double() @ w.t().contiguous()
    for i, a in enumerate(_ids(case)):
        if a >= 0:
            y[i] += s["scaling"][a].double() * (s["b"][a].double() @ (s["a"][a].double() @ s["x"][i].double()))
    return y
