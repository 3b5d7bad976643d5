"""The serving operators around the prefill path, as they are measured.

Three operators that belong together: rotary positions of packed queries and
keys, appending keys and values to a paged cache with the rotation applied on
the way, and attention over that cache for batches whose sequences share a long
prefix.  ``run`` computes each in its plain form (elementary torch operations),
or, where ``own`` is true, calls the framework's operator.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # rotary positions: a decode step of eight sequences (latency)
        {"name": "rope_step_8", "op": "rope", "dtype": "bf16", "tokens": 8, "hq": 32, "hkv": 8, "d": 128,
         "rotary": 128, "interleaved": False, "scaling": "llama3", "base": 500000.0, "far": 131072},
        # ... a ragged fp32 batch with a quarter of each head rotated, interleaved pairs
        {"name": "rope_f32_partial", "op": "rope", "dtype": "f32", "tokens": 8191, "hq": 8, "hkv": 4, "d": 256,
         "rotary": 64, "interleaved": True, "scaling": "yarn", "base": 10000.0, "far": 65536},
        # ... a whole 128K prompt before planning
        {"name": "rope_prompt_128k", "op": "rope", "dtype": "bf16", "tokens": 131072, "hq": 32, "hkv": 8, "d": 128,
         "rotary": 128, "interleaved": False, "scaling": "llama3", "base": 500000.0, "far": 131072},
        # paged append: one new token for each of 64 running sequences
        {"name": "append_step_64", "op": "append", "dtype": "bf16", "seqs": 64, "new_lo": 1, "new_hi": 1,
         "old_lo": 0, "old_hi": 8000, "lens": 1, "hq": 32, "hkv": 8, "d": 128, "page": 16, "rotary": 128,
         "interleaved": False, "scaling": "none", "base": 10000.0},
        # ... a ragged fp32 batch of prompts and continuations, odd sizes
        {"name": "append_f32_ragged", "op": "append", "dtype": "f32", "seqs": 7, "new_lo": 1, "new_hi": 701,
         "old_lo": 0, "old_hi": 999, "lens": 2, "hq": 6, "hkv": 2, "d": 64, "page": 32, "rotary": 32,
         "interleaved": True, "scaling": "linear", "base": 10000.0},
        # ... four prompts of 4K to 16K tokens, on the way into prefill
        {"name": "append_prompts_16k", "op": "append", "dtype": "bf16", "seqs": 4, "new_lo": 4096, "new_hi": 16384,
         "old_lo": 0, "old_hi": 0, "lens": 3, "hq": 32, "hkv": 8, "d": 128, "page": 64, "rotary": 128,
         "interleaved": False, "scaling": "llama3", "base": 500000.0},
        # attention: four answers to one short prompt (latency)
        {"name": "attend_4_short", "op": "attend", "dtype": "bf16", "groups": 1, "seqs": 4, "new": 1, "prefix": 1001,
         "own_lo": 1, "own_hi": 200, "lens": 4, "hq": 32, "hkv": 8, "d": 128, "page": 16},
        # ... ordinary decode, nothing shared, ragged lengths
        {"name": "attend_48_unshared", "op": "attend", "dtype": "bf16", "groups": 0, "seqs": 48, "new": 1, "prefix": 0,
         "own_lo": 100, "own_hi": 8192, "lens": 5, "hq": 32, "hkv": 8, "d": 128, "page": 64},
        # ... two prompts, five drafted tokens to verify for each of twelve answers, wide heads
        {"name": "attend_draft5_d256", "op": "attend", "dtype": "bf16", "groups": 2, "seqs": 12, "new": 5,
         "prefix": 4097, "own_lo": 5, "own_hi": 600, "lens": 6, "hq": 8, "hkv": 4, "d": 256, "page": 16},
        # ... fp32, small heads
        {"name": "attend_f32_d64", "op": "attend", "dtype": "f32", "groups": 3, "seqs": 5, "new": 1, "prefix": 2050,
         "own_lo": 1, "own_hi": 500, "lens": 7, "hq": 8, "hkv": 2, "d": 64, "page": 32},
        # ... 32 answers to a 32K prompt
        {"name": "attend_32_of_32k", "op": "attend", "dtype": "bf16", "groups": 1, "seqs": 32, "new": 1,
         "prefix": 32768, "own_lo": 1, "own_hi": 1024, "lens": 8, "hq": 32, "hkv": 8, "d": 128, "page": 16},
        # ... 64 answers to a 128K prompt
        {"name": "attend_64_of_128k", "op": "attend", "dtype": "bf16", "groups": 1, "seqs": 64, "new": 1,
         "prefix": 131072, "own_lo": 1, "own_hi": 2048, "lens": 9, "hq": 32, "hkv": 8, "d": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = _any(rng)
    # no more than the largest listed case, and fp32, which stands for checks
    # and small models, a sixteenth of its products
    flops = 1.3e11 / (16 if case["dtype"] == "f32" else 1)
    while True:
        w = work(case)
        if w["bytes"] <= 2.6e9 and (w["flops"] <= flops or case["op"] != "attend"):
            return case
        if case["op"] == "rope":
            case["tokens"] = 2 * case["tokens"] // 3
        elif case["seqs"] > 1:
            case["seqs"] = 2 * case["seqs"] // 3
        elif case["op"] == "append":
            case["new_lo"] = case["new_hi"] = 2 * case["new_hi"] // 3
        else:
            case["prefix"] = 2 * case["prefix"] // 3


def _any(rng):
    d = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 8] if hkv <= 4 else [1, 2, 4])
    case = {"op": rng.choice(["rope", "append", "attend", "attend"]), "dtype": rng.choice(["bf16", "bf16", "bf16", "f32"]),
            "hq": hq, "hkv": hkv, "d": d}
    if case["op"] != "attend":
        case.update(rotary=rng.choice([d, d, d // 2, d // 4, 2 * rng.randint(1, d // 2)]), interleaved=rng.random() < 0.4,
                    scaling=rng.choice(["none", "linear", "llama3", "yarn"]), base=rng.choice([10000.0, 500000.0]))
    if case["op"] == "rope":
        case.update(tokens=_log(rng, 1, 65536), far=rng.choice([4096, 131072, 1000000]))
        return case
    case.update(page=rng.choice([16, 32, 64, 128]), lens=rng.randint(100, 10 ** 6))
    if case["op"] == "append":
        hi = _log(rng, 1, 4096)
        case.update(seqs=_log(rng, 1, 128 if hi > 64 else 400), new_lo=rng.randint(1, hi), new_hi=hi, old_lo=0,
                    old_hi=_log(rng, 1, 4000))
        case["seqs"] = max(1, min(case["seqs"], 40000 // hi))
        return case
    groups = rng.choice([0, 1, 1, 2, 3])
    prefix = 0 if groups == 0 else _log(rng, 64, 65536)
    new = rng.choice([1, 1, 1, 2, 4, 7])
    seqs = _log(rng, 1, 64)
    if groups:
        seqs = max(1, min(seqs, 48 * 65536 // (prefix * groups), 64 // groups))
    own_hi = _log(rng, new, 4096)
    case.update(groups=groups, seqs=seqs, new=new, prefix=prefix, own_lo=rng.randint(new, own_hi), own_hi=own_hi)
    return case


# --------------------------------------------------------------- sizes


def _sequences(case):
    """(new tokens, tokens held after them) of each sequence: from the case alone."""
    r = random.Random(case["lens"])
    if case["op"] == "append":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["seqs"])]
        return new, [n + r.randint(case["old_lo"], case["old_hi"]) for n in new]
    count = case["seqs"] * max(1, case["groups"])
    return [case["new"]] * count, [case["prefix"] + r.randint(case["own_lo"], case["own_hi"]) for _ in range(count)]


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        elems = case["tokens"] * (hq + hkv) * d
        return {"bytes": 2 * elems * size + 4 * case["tokens"],
                "flops": 3 * case["tokens"] * (hq + hkv) * case["rotary"]}
    new, held = _sequences(case)
    tokens = sum(new)
    if case["op"] == "append":
        # q, k, v read; q, the packed k and the two pages written
        return {"bytes": tokens * d * size * (2 * hq + 5 * hkv) + 8 * len(new),
                "flops": 3 * tokens * (hq + hkv) * case["rotary"]}
    kv = case["groups"] * case["prefix"] + sum(h - case["prefix"] for h in held)
    pairs = sum(n * h - n * (n - 1) // 2 for n, h in zip(new, held))
    return {"bytes": 2 * kv * hkv * d * size + 2 * tokens * hq * d * size + 4 * (kv // case["page"] + 2 * len(new)) + 4 * tokens * hq,
            "flops": 4 * pairs * hq * d}


# -------------------------------------------------------------- inputs


def _scaling(case):
    kind = case["scaling"]
    return {"none": None,
            "linear": {"kind": "linear", "factor": 4.0},
            "llama3": {"kind": "llama3", "factor": 8.0, "original_len": 8192, "low_freq_factor": 1.0,
                       "high_freq_factor": 4.0},
            "yarn": {"kind": "yarn", "factor": 16.0, "original_len": 4096, "beta_fast": 32.0, "beta_slow": 1.0}}[kind]


def _rope_handle(case):
    from dynamic_hierarchical_sparse_b200 import api, workloads

    s = _scaling(case)
    return api.Rope(case["rotary"], base=case["base"], interleaved=case["interleaved"],
                    scaling=None if s is None else workloads.RopeScaling(**s))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    st = {"case": case}
    if case["op"] == "rope":
        n = case["tokens"]
        # q and k as the two parts of one projection's output
        qk = randn(n, hq + hkv, d).to(dt)
        st["q"], st["k"] = qk[:, :hq], qk[:, hq:]
        st["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=dev, dtype=torch.int32)
        st["q_out"] = torch.empty(n, hq, d, dtype=dt, device=dev)
        st["k_out"] = torch.empty(n, hkv, d, dtype=dt, device=dev)
        if own:  # the handle a program keeps: frequencies only
            st["rope"] = _rope_handle(case)
        return st

    new, held = _sequences(case)
    page, prefix, count = case["page"], case.get("prefix", 0), len(new)
    # pages in a random order, as a running allocator leaves them; the whole
    # pages of a shared prefix are the same ones for every sequence of a group
    shared = prefix // page
    groups = case.get("groups", 0)
    per_group = case["seqs"] if groups else 1
    width = max(-(-h // page) for h in held)
    free = torch.randperm(groups * shared + count * (width - shared) + 3, generator=gen, device=dev).to(torch.int32)
    pages = free.numel()
    table = torch.zeros(count, width, dtype=torch.int32, device=dev)
    if groups and shared:
        table[:, :shared] = free[:groups * shared].view(groups, 1, shared).expand(-1, per_group, -1).reshape(count, -1)
    if width > shared:
        table[:, shared:] = free[groups * shared:groups * shared + count * (width - shared)].view(count, -1)
    st["table"] = table
    st["kv_lens"] = torch.tensor(held, dtype=torch.int32, device=dev)
    st["cu_q"] = [0]
    for n in new:
        st["cu_q"].append(st["cu_q"][-1] + n)
    tokens = st["cu_q"][-1]
    v_dt = torch.float16 if dt == torch.bfloat16 else dt
    if case["op"] == "append":
        qkv = randn(tokens, hq + 2 * hkv, d).to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        st["k_pages"] = randn(pages, hkv, page, d).to(dt)
        st["v_pages"] = randn(pages, hkv, page, d).to(v_dt)
        st["q_out"] = torch.empty(tokens, hq, d, dtype=dt, device=dev)
        st["k_out"] = torch.empty(tokens, hkv, d, dtype=dt, device=dev)
        # the owners of the new tokens, which the plain form goes by
        st["seq_of"] = torch.repeat_interleave(torch.arange(count, device=dev), torch.tensor(new, device=dev))
        st["cu"] = torch.tensor(st["cu_q"], device=dev)
        if own:
            from dynamic_hierarchical_sparse_b200 import api

            cache = api.PagedCache(st["k_pages"], st["v_pages"])
            batch = api.PagedBatch(st["cu_q"], st["kv_lens"], table)
            st["append"] = api.KvAppender(cache, batch, _rope_handle(case))
        return st

    # some of the variance of queries and keys lies in four directions a KV
    # head, so attention has peaks as a model's does
    mix = randn(hkv, 4, d)
    q = randn(tokens, hkv, hq // hkv, d) + 0.5 * torch.einsum("tgrc,gcd->tgrd", randn(tokens, hkv, hq // hkv, 4), mix)
    st["q"] = q.reshape(tokens, hq, d).to(dt)
    k = randn(pages, hkv, page, d)
    k += 0.5 * torch.einsum("pgsc,gcd->pgsd", randn(pages, hkv, page, 4), mix)
    st["k_pages"] = k.to(dt)
    del k
    st["v_pages"] = randn(pages, hkv, page, d).to(v_dt)
    if groups and prefix % page:
        # a prefix that ends inside a page: every sequence got a copy of that page's part to write behind
        for x in (st["k_pages"], st["v_pages"]):
            part = x[table[::per_group, shared].long(), :, :prefix % page]
            x[table[:, shared].long(), :, :prefix % page] = part.repeat_interleave(per_group, 0)
    st["out"] = torch.empty(tokens, hq, d, dtype=dt, device=dev)
    st["lse"] = torch.empty(tokens, hq, dtype=torch.float32, device=dev)
    if own:
        from dynamic_hierarchical_sparse_b200 import api

        cache = api.PagedCache(st["k_pages"], st["v_pages"])
        group_ptr, prefix_lens = None, None
        if groups:
            group_ptr = [g * per_group for g in range(groups + 1)]
            prefix_lens = torch.full((groups,), prefix, dtype=torch.int32, device=dev)
        batch = api.PagedBatch(st["cu_q"], st["kv_lens"], table, group_ptr, prefix_lens)
        st["attend"] = api.PagedAttention(cache, batch, hq)
    return st


# --------------------------------------------------------- plain forms


def _frequencies(case, dev):
    """The rotation's frequencies in 64 bits, and the factor on cos and sin."""
    rd, base, s = case["rotary"], case["base"], _scaling(case)
    i = torch.arange(rd // 2, dtype=torch.float64, device=dev)
    f = base ** (-2.0 * i / rd)
    if s is None:
        return f, 1.0
    if s["kind"] == "linear":
        return f / s["factor"], 1.0
    if s["kind"] == "llama3":
        turns = s["original_len"] * f / (2 * math.pi)  # turns within the original length
        lo, hi = s["low_freq_factor"], s["high_freq_factor"]
        keep = ((turns - lo) / (hi - lo)).clamp(0.0, 1.0)
        return f * keep + f / s["factor"] * (1 - keep), 1.0
    low = math.floor(rd * math.log(s["original_len"] / (s["beta_fast"] * 2 * math.pi)) / (2 * math.log(base)))
    high = math.ceil(rd * math.log(s["original_len"] / (s["beta_slow"] * 2 * math.pi)) / (2 * math.log(base)))
    low, high = max(low, 0), min(high, rd - 1)
    ramp = ((i - low) / (high - low if high != low else 0.001)).clamp(0.0, 1.0)
    return f / s["factor"] * ramp + f * (1 - ramp), 0.1 * math.log(s["factor"]) + 1.0


def _rotate(x, positions, case):
    f, m = _frequencies(case, x.device)
    angle = positions.double()[:, None] * f
    cos, sin = (m * angle.cos()).float()[:, None], (m * angle.sin()).float()[:, None]
    rd = case["rotary"]
    x32 = x.float()
    if case["interleaved"]:
        x1, x2 = x32[..., 0:rd:2], x32[..., 1:rd:2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = x32[..., :rd // 2], x32[..., rd // 2:rd]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([y, x32[..., rd:]], -1).to(x.dtype)


def _plain_append(st):
    case, page = st["case"], st["case"]["page"]
    seq = st["seq_of"]
    at = torch.arange(seq.numel(), device=seq.device) - st["cu"][seq + 1] + st["kv_lens"].long()[seq]
    slot_page, slot = st["table"].long()[seq, at // page], at % page
    q, k = _rotate(st["q"], at, case), _rotate(st["k"], at, case)
    st["k_pages"][slot_page, :, slot] = k
    st["v_pages"][slot_page, :, slot] = st["v"].to(st["v_pages"].dtype)
    return {"q": q, "k": k, "k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _plain_attend(st):
    case = st["case"]
    hq, hkv, d, page, prefix, new = (case[x] for x in ("hq", "hkv", "d", "page", "prefix", "new"))
    table, lens = st["table"].long(), st["kv_lens"].long()
    count, r, dev = table.shape[0], hq // hkv, table.device
    q = st["q"].float().view(count, new, hkv, r, d) * (1 / math.sqrt(d))
    limit = lens[:, None] - new + 1 + torch.arange(new, device=dev)  # keys that each query sees
    # each sequence's own part
    at = prefix + torch.arange(int(case["own_hi"]), device=dev)
    where = table[:, (at // page).clamp(max=table.shape[1] - 1)]
    k = st["k_pages"][where, :, at % page].float()
    v = st["v_pages"][where, :, at % page].float()
    s = torch.einsum("bnhrd,blhd->bnhrl", q, k)
    s = s.masked_fill((at >= limit[..., None])[:, :, None, None], -math.inf)
    if case["groups"]:
        # the shared part, once for a group
        g, n = case["groups"], case["seqs"]
        first = torch.arange(prefix, device=dev)
        where = table[::n, first // page]
        pk = st["k_pages"][where, :, first % page].float()
        pv = st["v_pages"][where, :, first % page].float()
        sp = torch.einsum("gbnhrd,glhd->gbnhrl", q.view(g, n, new, hkv, r, d), pk).reshape(count, new, hkv, r, prefix)
        top = torch.maximum(s.amax(-1, keepdim=True), sp.amax(-1, keepdim=True))
        s, sp = (s - top).exp(), (sp - top).exp()
        total = s.sum(-1) + sp.sum(-1)
        o = torch.einsum("gbnhrl,glhd->gbnhrd", sp.view(g, n, new, hkv, r, prefix), pv).reshape(q.shape)
    else:
        top = s.amax(-1, keepdim=True)
        s = (s - top).exp()
        total, o = s.sum(-1), 0.0
    v = v.masked_fill((at >= lens[:, None])[..., None, None], 0.0)
    o = o + torch.einsum("bnhrl,blhd->bnhrd", s, v)
    lse = (top[..., 0] + total.log()).reshape(count * new, hq)
    return {"out": (o / total[..., None]).reshape(count * new, hq, d).to(st["q"].dtype), "lse": lse}


def run(state):
    op = state["case"]["op"]
    if op == "rope":
        if own:
            from dynamic_hierarchical_sparse_b200 import api

            q, k = api.rope(state["q"], state["k"], state["positions"], state["rope"], state["q_out"], state["k_out"])
        else:
            q, k = (_rotate(state[x], state["positions"], state["case"]) for x in ("q", "k"))
        return {"q": q, "k": k}
    if op == "append":
        if own:
            q, k = state["append"](state["k"], state["v"], state["q"], state["q_out"], state["k_out"])
            return {"q": q, "k": k, "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
        return _plain_append(state)
    if own:
        return {"out": state["attend"](state["q"], state["out"], lse=state["lse"]), "lse": state["lse"]}
    return _plain_attend(state)


# ------------------------------------------------- the definition in 64 bits


def _exact_rotate(x, positions, case):
    """Each pair of numbers as a complex one, turned by its angle."""
    rd, base, s = case["rotary"], case["base"], _scaling(case) or {"kind": "none"}
    freqs, factor = [], 1.0
    for i in range(rd // 2):
        f = math.pow(base, -2.0 * i / rd)
        if s["kind"] == "linear":
            f /= s["factor"]
        elif s["kind"] == "llama3":
            length = 2 * math.pi / f
            if length > s["original_len"] / s["low_freq_factor"]:
                f /= s["factor"]
            elif length >= s["original_len"] / s["high_freq_factor"]:
                mid = (s["original_len"] / length - s["low_freq_factor"]) / (s["high_freq_factor"] - s["low_freq_factor"])
                f = (1 - mid) * f / s["factor"] + mid * f
        elif s["kind"] == "yarn":
            def place(turns):
                return rd * math.log(s["original_len"] / (turns * 2 * math.pi)) / (2 * math.log(base))
            low, high = max(math.floor(place(s["beta_fast"])), 0), min(math.ceil(place(s["beta_slow"])), rd - 1)
            if low == high:
                high += 0.001
            share = min(max((i - low) / (high - low), 0.0), 1.0)
            f = share * f / s["factor"] + (1 - share) * f
            factor = 0.1 * math.log(s["factor"]) + 1.0
        freqs.append(f)
    angle = positions.double()[:, None, None] * torch.tensor(freqs, dtype=torch.float64, device=x.device)
    y = x.double().clone()
    if case["interleaved"]:
        pairs = torch.view_as_complex(y[..., :rd].reshape(*y.shape[:-1], rd // 2, 2).contiguous())
    else:
        pairs = torch.complex(y[..., :rd // 2].contiguous(), y[..., rd // 2:rd].contiguous())
    turned = pairs * torch.polar(torch.full_like(angle, factor), angle)
    if case["interleaved"]:
        y[..., 0:rd:2], y[..., 1:rd:2] = turned.real, turned.imag
    else:
        y[..., :rd // 2], y[..., rd // 2:rd] = turned.real, turned.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return {x: _exact_rotate(st[x], st["positions"], case) for x in ("q", "k")}
    new, held = _sequences(case)
    page, dev = case["page"], st["table"].device
    if case["op"] == "append":
        at = torch.cat([torch.arange(h - n, h) for n, h in zip(new, held)]).to(dev)
        q, k = _exact_rotate(st["q"], at, case), _exact_rotate(st["k"], at, case)
        k_pages, v_pages = st["k_pages"].double(), st["v_pages"].double()
        begin = 0
        for b, (n, h) in enumerate(zip(new, held)):
            for p in range((h - n) // page, -(-h // page)):  # page by page
                lo, hi = max(p * page, h - n), min((p + 1) * page, h)
                rows = slice(begin + lo - (h - n), begin + hi - (h - n))
                where = int(st["table"][b, p])
                k_pages[where, :, lo - p * page:hi - p * page] = k[rows].transpose(0, 1)
                v_pages[where, :, lo - p * page:hi - p * page] = st["v"][rows].double().transpose(0, 1)
            begin += n
        return {"q": q, "k": k, "k_pages": k_pages, "v_pages": v_pages}
    r, out, lse = case["hq"] // case["hkv"], [], []
    for b, (n, h) in enumerate(zip(new, held)):  # each sequence alone, over all its keys
        rows = st["table"][b, :-(-h // page)].long()
        k = st["k_pages"][rows].transpose(0, 1).flatten(1, 2)[:, :h].double()
        v = st["v_pages"][rows].transpose(0, 1).flatten(1, 2)[:, :h].double()
        q = st["q"][b * n:(b + 1) * n].double().transpose(0, 1).reshape(case["hkv"], r * n, case["d"])
        s = q @ k.transpose(1, 2) / math.sqrt(case["d"])
        hidden = torch.arange(h, device=dev) > h - n + torch.arange(n, device=dev)[:, None]
        s = s.view(case["hkv"], r, n, h).masked_fill(hidden, -math.inf)
        lse.append(s.logsumexp(-1).view(case["hq"], n).transpose(0, 1))
        out.append((s.softmax(-1).view(case["hkv"], r * n, h) @ v).view(case["hq"], n, case["d"]).transpose(0, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
