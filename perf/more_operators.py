"""Cases of the operators between and around a decoder's layers, in plain torch and as calls of the library.

One turn of a serving loop: the batch plan (slots, pages and offsets of the new tokens from
the requests' lengths), attention for requests that share a long prompt over the paged INT4
cache, and the choice of the next tokens from the logits. Head layouts are those of the
Llama-3-70B (64 query and 8 KV heads of 128 channels) and Llama-3-8B (32 and 8 heads) shapes.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False


def _lib():
    import w4a16_decode_amd as q4

    return q4


# ---- cases ---------------------------------------------------------------------


def listed():
    return [
        # a decode batch, one token each: latency of the step's bookkeeping
        {"name": "plan_decode_b48", "op": "plan", "seqs": 48, "new": 1, "max_kv": 8191, "page": 32, "reset": 0.0},
        # a scheduler that packs many prompts into one call, requests that ended give back their pages
        {"name": "plan_prefill_mixed", "op": "plan", "seqs": 61, "new": 4001, "max_kv": 2049, "page": 16,
         "reset": 0.2},
        # a few requests behind one system prompt (8B shape): latency
        {"name": "shared_decode_b8_8b", "op": "attn", "seqs": 8, "shared": 1, "new": 1, "max_prefix": 1003,
         "max_own": 130, "hq": 32, "hkv": 8, "d": 128, "group": 128, "page": 16},
        # a full decode batch over one long document (70B shape)
        {"name": "shared_decode_b64_70b", "op": "attn", "seqs": 64, "shared": 1, "new": 1, "max_prefix": 8190,
         "max_own": 513, "hq": 64, "hkv": 8, "d": 128, "group": 128, "page": 32},
        # several documents, a ragged number of requests each, finer scale groups and longer answers
        {"name": "shared_decode_groups", "op": "attn", "seqs": 41, "shared": 5, "new": 1, "max_prefix": 6001,
         "max_own": 1025, "hq": 32, "hkv": 8, "d": 128, "group": 64, "page": 64},
        # questions of several tokens behind a shared document (70B shape): matrix work
        {"name": "shared_chunk_70b", "op": "attn", "seqs": 9, "shared": 2, "new": 251, "max_prefix": 6001,
         "max_own": 700, "hq": 64, "hkv": 8, "d": 128, "group": 128, "page": 48},
        # one request, the usual filters: latency over one long row
        {"name": "sample_b1", "op": "sample", "rows": 1, "vocab": 128256, "type": "float16", "temperature": True,
         "top_k": 50, "top_p": True, "min_p": False, "masked": 0.0},
        # a decode batch of requests with settings of their own, greedy ones among them
        {"name": "sample_b64_mixed", "op": "sample", "rows": 64, "vocab": 128256, "type": "float32",
         "temperature": True, "top_k": 200, "top_p": True, "min_p": True, "masked": 0.0},
        # many rows, the plain softmax draw: the whole distribution counts
        {"name": "sample_b256_softmax", "op": "sample", "rows": 256, "vocab": 32000, "type": "float16",
         "temperature": True, "top_k": 0, "top_p": False, "min_p": False, "masked": 0.0},
        # an odd vocabulary, half of it forbidden by a grammar
        {"name": "sample_b17_masked", "op": "sample", "rows": 17, "vocab": 50257, "type": "bfloat16",
         "temperature": True, "top_k": 0, "top_p": True, "min_p": False, "masked": 0.5},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "attn", "attn", "sample", "sample"])
    if op == "plan":
        new = rng.choice([1, 1, _log(rng, 2, 2000)])
        return {"op": op, "seqs": _log(rng, 1, 512 if new == 1 else 61), "new": new, "max_kv": _log(rng, 1, 8000),
                "page": 16 * rng.choice([1, 2, 3, 8]), "reset": rng.choice([0.0, 0.0, 0.3])}
    if op == "attn":
        hkv, d = rng.choice([4, 8]), rng.choice([64, 128, 128, 256])
        kind = rng.choice(["decode", "decode", "few", "chunk"])
        seqs = _log(rng, 1, 64 if kind == "decode" else 10 if kind == "few" else 5)
        new = 1 if kind == "decode" else rng.randint(2, 9) if kind == "few" else _log(rng, 10, 150)
        return {"op": op, "seqs": seqs, "shared": rng.randint(1, min(seqs, 4)), "new": new,
                "max_prefix": _log(rng, 1, 4000), "max_own": new + _log(rng, 1, 600),
                "hq": hkv * rng.choice([1, 4, 7, 8]), "hkv": hkv, "d": d,
                "group": rng.choice([g for g in (32, 64, 128) if g <= d]), "page": 16 * rng.choice([1, 2, 3, 8])}
    return {"op": op, "rows": _log(rng, 1, 200), "vocab": _log(rng, 1000, 64000),
            "type": rng.choice(["float16", "bfloat16", "float32"]), "temperature": rng.random() < 0.8,
            "top_k": rng.choice([0, _log(rng, 1, 2000)]), "top_p": rng.random() < 0.5, "min_p": rng.random() < 0.3,
            "masked": rng.choice([0.0, 0.0, 0.7])}


def _ragged(rng, count, lo, hi):
    """Whole numbers in [lo, hi], the first at hi."""
    return [hi] + [rng.randint(lo, hi) for _ in range(count - 1)]


def _plan_lens(case):
    """Per sequence: tokens in the cache, new tokens, whether its request has ended."""
    rng = random.Random("%(seqs)d %(new)d %(max_kv)d" % case)
    n = case["seqs"]
    lens = _ragged(rng, n, case["max_kv"] // 4, case["max_kv"])
    reset = [i > 0 and rng.random() < case["reset"] for i in range(n)]
    new = _ragged(rng, n, (case["new"] + 3) // 4, case["new"])
    return lens, [0 if r else k for r, k in zip(reset, new)], [int(r) for r in reset]


def _attn_lens(case):
    """New tokens and own lengths of the sequences, their number in each group, the prefixes' lengths."""
    rng = random.Random("%(seqs)d %(shared)d %(new)d %(max_own)d" % case)
    new = _ragged(rng, case["seqs"], (case["new"] + 3) // 4, case["new"])
    lens = [max(k, m) for k, m in zip(new, _ragged(rng, case["seqs"], case["max_own"] // 4, case["max_own"]))]
    cuts = sorted(rng.sample(range(1, case["seqs"]), case["shared"] - 1))
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [case["seqs"]])]
    return new, lens, sizes, _ragged(rng, case["shared"], case["max_prefix"] // 4, case["max_prefix"])


def work(case):
    op = case["op"]
    if op == "plan":
        lens, new, reset = _plan_lens(case)
        page = case["page"]
        pages = [-(-(0 if r else n) // page) for n, r in zip(lens, reset)]
        fresh = sum(-(-((0 if r else n) + k) // page) - p for n, k, r, p in zip(lens, new, reset, pages))
        freed = sum(-(-n // page) for n, r in zip(lens, reset) if r)
        # lengths in and out, flags, offsets, starts; pages moved; position, slot and page of the rows
        return {"bytes": 24 * case["seqs"] + 8 * (fresh + freed) + 12 * sum(new), "flops": 10 * sum(new)}
    if op == "attn":
        new, lens, sizes, prefix = _attn_lens(case)
        shared = [p for p, k in zip(prefix, sizes) for _ in range(k)]
        pairs = sum(k * p + k * n - k * (k - 1) // 2 for k, n, p in zip(new, lens, shared))
        keys = sum(prefix) + sum(lens)
        per_key = case["hkv"] * 2 * (case["d"] // 2 + 2 * (case["d"] // case["group"]))
        return {"bytes": keys * per_key + 4 * sum(new) * case["hq"] * case["d"] + 4 * keys // case["page"],
                "flops": 4 * pairs * case["hq"] * case["d"]}
    n = case["rows"] * case["vocab"]
    # a difference, a product, an exponential and a sum a logit
    return {"bytes": n * (4 if case["type"] == "float32" else 2) + 28 * case["rows"], "flops": 4 * n}


# ---- inputs ----------------------------------------------------------------------


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(x):
    return torch.tensor(x, device="cuda", dtype=torch.int32)


def _sums(x):
    return _ints([0] + list(np.cumsum(x)))


def _plan_inputs(case, seed):
    lens, new, reset = _plan_lens(case)
    g, page, n = _gen(seed), case["page"], case["seqs"]
    blocks = -(-max(a + b for a, b in zip(lens, new)) // page) + 2
    pages = n * blocks + 5
    order = torch.randperm(pages, generator=g, device="cuda").int()
    held = torch.arange(blocks, device="cuda") < _ints([-(-a // page) for a in lens])[:, None]
    at = held.flatten().cumsum(0).view(n, blocks) - 1
    used = sum(-(-a // page) for a in lens)
    free = torch.zeros(pages, device="cuda", dtype=torch.int32)
    free[:pages - used] = order[used:]
    return {"kv_lens": _ints(lens), "new_lens": _ints(new), "reset": _ints(reset) if case["reset"] else None,
            "starts": torch.randint(0, 4000, (n,), generator=g, device="cuda", dtype=torch.int32),
            "table": torch.where(held, order[at.clamp(min=0)], -1), "free": free, "count": _ints([pages - used]),
            "pages": pages, "tokens": sum(new)}


def _attn_inputs(case, seed):
    new, lens, sizes, prefix = _attn_lens(case)
    g, hkv, d, page = _gen(seed), case["hkv"], case["d"], case["page"]
    wide, narrow = -(-max(prefix) // page), -(-max(lens) // page)
    pages = len(prefix) * wide + len(lens) * narrow + 2
    order = torch.randperm(pages, generator=g, device="cuda").int()
    channel = torch.exp(0.4 * _normal(g, 1, hkv, d))
    # every slot of the pool holds a token, as in a cache in use: what lies behind a length is another request's
    k = (_normal(g, pages * page, hkv, d) * channel).half()
    v = _normal(g, pages * page, hkv, d).half()
    rows = np.cumsum([0] + new)
    return {"q": _normal(g, int(rows[-1]), case["hq"], d).half(), "k": k, "v": v, "pages": pages,
            "prefix_table": order[:len(prefix) * wide].view(len(prefix), wide).contiguous(),
            "block_table": order[len(prefix) * wide:pages - 2].view(len(lens), narrow).contiguous(),
            "prefix_lens": _ints(prefix), "group_offsets": _sums(sizes), "q_offsets": _sums(new),
            "kv_lens": _ints(lens), "max_q": max(new), "max_kv": max(lens), "max_prefix": max(prefix),
            "max_group_q": int(max(np.diff(rows[np.cumsum([0] + sizes)])))}


def _sample_inputs(case, seed):
    g, n, v = _gen(seed), case["rows"], case["vocab"]
    # a few tokens far ahead of a long tail, more or less of them from row to row
    logits = _normal(g, n, v) * (1.5 + 1.5 * torch.rand(n, 1, generator=g, device="cuda"))
    if case["masked"]:
        logits.masked_fill_(torch.rand(n, v, generator=g, device="cuda") < case["masked"], -math.inf)

    def some(x, off):
        return torch.where(torch.rand(n, generator=g, device="cuda") < 0.75, x, torch.full_like(x, off))

    def rand(lo, hi):
        return lo + (hi - lo) * torch.rand(n, generator=g, device="cuda")

    return {"logits": logits.to(getattr(torch, case["type"])), "uniforms": rand(0.0, 1.0),
            "temperature": some(rand(0.5, 1.4), 0.0) if case["temperature"] else None,
            "top_k": some(torch.randint(1, case["top_k"] + 1, (n,), generator=g, device="cuda"), 0).int()
            if case["top_k"] else None,
            "top_p": some(rand(0.7, 0.99), 1.0) if case["top_p"] else None,
            "min_p": some(rand(0.01, 0.2), 0.0) if case["min_p"] else None}


def _rtn4(x, group):
    """Group-wise INT4 of the last axis: codes and float16 scales, decided in 64 bits."""
    y = x.view(*x.shape[:-1], -1, group)
    s = (y.abs().amax(-1).double() / 7).half()
    z = s.double()[..., None]
    codes = torch.where(z == 0, 0.0, (y.double() / z.where(z != 0, 1.0)).round().clamp(-8, 7))
    return codes.to(torch.int8).view(x.shape), s


def prepare(case, seed):
    s = {"plan": _plan_inputs, "attn": _attn_inputs, "sample": _sample_inputs}[case["op"]](case, seed)
    if case["op"] == "plan" and own:
        s["pool"] = _lib().PagePool(s["free"], s["count"])
    if case["op"] == "attn":
        k, v = s.pop("k"), s.pop("v")
        if own:
            s["cache"] = _lib().paged_kv_alloc(s["pages"], case["page"], case["hkv"], case["d"], case["group"])
            _lib().paged_kv_append(k, v, s["cache"], torch.arange(len(k), device="cuda", dtype=torch.int32))
        else:
            s["k"], s["v"] = _rtn4(k, case["group"]), _rtn4(v, case["group"])
    return {"case": case, **s}


# ---- one pass -----------------------------------------------------------------------


def run(s):
    case = s["case"]
    if own:
        return _run_own(case, s)
    return {"plan": _plan, "attn": _attn, "sample": _sample}[case["op"]](case, s)


def _run_own(case, s):
    q4, op = _lib(), case["op"]
    if op == "plan":
        p = q4.paged_plan(s["kv_lens"], s["new_lens"], s["table"], case["page"], s["tokens"], s["pool"],
                          starts=s["starts"], reset=s["reset"])
        return (p.q_offsets, p.positions, p.slots, p.kv_lens, s["table"], s["pool"].pages, p.free_count, p.lacking)
    if op == "attn":
        return q4.paged_attention_shared(s["q"], s["cache"], s["prefix_table"], s["prefix_lens"], s["group_offsets"],
                                         s["block_table"], s["q_offsets"], s["kv_lens"], s["max_q"], s["max_kv"],
                                         s["max_group_q"], s["max_prefix"])
    return q4.sample(s["logits"], s["uniforms"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])


def _plan(case, s):
    page, table, free = case["page"], s["table"].clone(), s["free"].clone()
    blocks = torch.arange(table.shape[1], device="cuda")
    lens, new = s["kv_lens"].long(), s["new_lens"].long()
    count = s["count"].long()
    if s["reset"] is not None:
        # pages of the requests that ended, pushed in order
        given = (s["reset"][:, None] != 0) & (blocks < -(-lens // page)[:, None])
        at = (count + given.flatten().cumsum(0) - 1).view(table.shape)
        free[at[given]] = table[given]
        count = count + given.sum()
        lens = torch.where(s["reset"] != 0, 0, lens)
    have, want = -(-lens // page), -(-(lens + new) // page)
    fresh = (blocks >= have[:, None]) & (blocks < want[:, None])
    at = (count - fresh.flatten().cumsum(0)).view(table.shape)
    table[fresh] = free[at[fresh]]
    offsets = torch.cat((torch.zeros(1, dtype=torch.long, device="cuda"), new.cumsum(0)))
    seq = torch.repeat_interleave(torch.arange(len(new), device="cuda"), new, output_size=s["tokens"])
    at = lens[seq] + torch.arange(s["tokens"], device="cuda") - offsets[seq]
    slots = table[seq, at // page] * page + at % page
    return (offsets.int(), (s["starts"][seq] + at).int(), slots.int(), (lens + new).int(), table, free,
            (count - fresh.sum()).int(), torch.zeros(1, dtype=torch.int32, device="cuda"))


def _spread(codes, scales):
    """The float32 values that codes and their groups' scales stand for."""
    y = codes.float().view(*scales.shape, -1)
    return (y * scales.float()[..., None]).view(codes.shape)


def _attn(case, s):
    hkv, d, page = case["hkv"], case["d"], case["page"]
    share = case["hq"] // hkv
    tokens = len(s["q"])

    def cached(name, table):
        codes, scales = s[name]
        pick = table.long()
        x = _spread(codes.view(-1, page, hkv, d)[pick], scales.view(s["pages"], page, hkv, -1)[pick])
        return x.view(len(table), -1, hkv, d).transpose(1, 2).contiguous()  # [tables, heads, keys, d]

    def part(table, first, rows_max, seen):
        """Maximum, sum and output, before the division, of the rows over the keys of their table."""
        k, v = cached("k", table), cached("v", table)
        n, keys = len(table), k.shape[2]
        row = first[:-1, None].long() + torch.arange(rows_max, device="cuda")  # [tables, rows]
        there = row < first[1:, None]
        q = s["q"].float()[row.clamp(max=tokens - 1)].view(n, rows_max, hkv, share, d)
        q = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, -1, d)  # rows (head, token)
        p = torch.matmul(q, k.transpose(-1, -2).contiguous()) / math.sqrt(d)
        p = p.view(n, hkv, share, rows_max, keys).masked_fill_(~seen(row, keys)[:, None, None], -math.inf)
        top = p.amax(-1, keepdim=True).clamp(min=-1e30)
        p = (p - top).exp_()
        o = torch.matmul(p.view(n, hkv, -1, keys), v).view(n, hkv, share, rows_max, d)

        def rows(x):  # [tokens, heads, channels]
            return x.permute(0, 3, 1, 2, 4)[there].reshape(tokens, case["hq"], -1)

        return rows(top), rows(p.sum(-1, keepdim=True)), rows(o)

    def seen_prefix(row, keys):
        return (torch.arange(keys, device="cuda") < s["prefix_lens"][:, None])[:, None].expand(*row.shape, keys)

    def seen_own(row, keys):
        at = row + (s["kv_lens"] - s["q_offsets"][1:])[:, None]  # a row's own position
        return torch.arange(keys, device="cuda") <= at[..., None]

    group_rows = s["q_offsets"][s["group_offsets"].long()]
    m1, l1, o1 = part(s["prefix_table"], group_rows, s["max_group_q"], seen_prefix)
    m2, l2, o2 = part(s["block_table"], s["q_offsets"], s["max_q"], seen_own)
    m = torch.maximum(m1, m2)
    a1, a2 = (m1 - m).exp(), (m2 - m).exp()
    return ((o1 * a1 + o2 * a2) / (l1 * a1 + l2 * a2)).half()


def _sample(case, s):
    n, v = s["logits"].shape

    def setting(name, off):
        return torch.full((n, 1), off, dtype=torch.float64, device="cuda") if s[name] is None else \
            s[name].double()[:, None]

    # 64 bits: sums over the vocabulary and values next to a border decide whole numbers
    x = s["logits"].double()
    t, k = setting("temperature", 1.0), setting("top_k", 0.0)
    greedy = t <= 0
    k = torch.where(greedy, 1.0, torch.where(k > 0, k, float(v)))
    w = ((x - x.amax(-1, keepdim=True)) / torch.where(greedy, 1.0, t)).exp()
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    y = w.gather(-1, order) * (torch.arange(v, device="cuda") < k)
    total = y.cumsum(-1)
    keep = (total - y < setting("top_p", 1.0) * total[:, -1:]) & (y >= setting("min_p", 0.0)) & (y > 0)
    w = w * torch.zeros_like(w).scatter_(-1, order, keep.double())
    total = w.cumsum(-1)
    at = (total <= s["uniforms"].double()[:, None] * total[:, -1:]).sum(-1, keepdim=True).clamp(max=v - 1)
    return at[:, 0].int(), (w.gather(-1, at) / total[:, -1:])[:, 0].float()


# ---- in 64 bits ----------------------------------------------------------------------


def exact(case, seed):
    return {"plan": _exact_plan, "attn": _exact_attn, "sample": _exact_sample}[case["op"]](case, seed)


def _exact_plan(case, seed):
    """A list of free pages, sequence after sequence."""
    s, page = _plan_inputs(case, seed), case["page"]
    lens, new, reset = _plan_lens(case)
    table, free, starts = (s[n].cpu().numpy().copy() for n in ("table", "free", "starts"))
    count = int(s["count"][0])
    for i in [i for i, r in enumerate(reset) if r]:
        given = table[i, :-(-lens[i] // page)]
        free[count:count + len(given)] = given
        count, lens[i] = count + len(given), 0
    positions, slots = [], []
    for i, (n, k) in enumerate(zip(lens, new)):
        for b in range(-(-n // page), -(-(n + k) // page)):
            count -= 1
            table[i, b] = free[count]
        p = np.arange(n, n + k)
        positions.append(starts[i] + p)
        slots.append(table[i, p // page].astype(np.int64) * page + p % page)
    return (_sums(new), _ints(np.concatenate(positions)), _ints(np.concatenate(slots)),
            _ints([n + k for n, k in zip(lens, new)]), _ints(table), _ints(free), _ints([count]), _ints([0]))


def _exact_attn(case, seed):
    s, g, d, page = _attn_inputs(case, seed), case["group"], case["d"], case["page"]
    new, lens, sizes, prefix = _attn_lens(case)
    share = case["hq"] // case["hkv"]
    out = torch.zeros(sum(new), case["hq"], d, dtype=torch.float64, device="cuda")
    first, groups = 0, [i for i, k in enumerate(sizes) for _ in range(k)]
    for i, (k, n) in enumerate(zip(new, lens)):
        p = prefix[groups[i]]
        t, u = torch.arange(p, device="cuda"), torch.arange(n, device="cuda")
        at = torch.cat((s["prefix_table"][groups[i]].long()[t // page] * page + t % page,
                        s["block_table"][i].long()[u // page] * page + u % page))
        kv = []
        for x in (s["k"][at], s["v"][at]):
            codes, scales = _rtn4(x, g)
            kv.append(codes.double() * scales.double().repeat_interleave(g, -1))
        hidden = torch.arange(p + n, device="cuda") > torch.arange(p + n - k, p + n, device="cuda")[:, None]
        for h in range(case["hkv"]):
            heads = slice(h * share, (h + 1) * share)
            q = s["q"][first:first + k, heads].double().transpose(0, 1).reshape(share * k, d)
            z = (q @ kv[0][:, h].t().contiguous() * d ** -0.5).view(share, k, -1)
            z[:, hidden] = -math.inf
            o = torch.softmax(z, -1).view(share * k, -1) @ kv[1][:, h].contiguous()
            out[first:first + k, heads] = o.view(share, k, d).transpose(0, 1)
        first += k
    return out


def _exact_sample(case, seed):
    """Row by row on the host: the order, the cuts one after the other, the draw."""
    s = {n: None if x is None else x.double().cpu().numpy() for n, x in _sample_inputs(case, seed).items()}
    tokens, probs = [], []
    for r, x in enumerate(s["logits"]):
        def of(name, off):
            return off if s[name] is None else s[name][r]

        t = of("temperature", 1.0)
        order = np.argsort(-x, kind="stable")
        order = order[:1 if t <= 0 else int(of("top_k", 0)) or None]
        w = np.exp((x[order] - x[order[0]]) / (t if t > 0 else 1.0))
        if of("top_p", 1.0) < 1.0:
            cut = int(np.searchsorted(np.cumsum(w), of("top_p", 1.0) * w.sum(), side="left")) + 1
            order, w = order[:cut], w[:cut]
        order, w = order[w >= of("min_p", 0.0)], w[w >= of("min_p", 0.0)]
        by_index = np.argsort(order)
        order, w = order[by_index], w[by_index]
        i = min(int(np.searchsorted(np.cumsum(w), s["uniforms"][r] * w.sum(), side="right")), len(w) - 1)
        tokens.append(int(order[i]))
        probs.append(w[i] / w.sum())
    return _ints(tokens), torch.tensor(probs, dtype=torch.float64, device="cuda")
