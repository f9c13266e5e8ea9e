"""The grouped-head attention (GQA) operators, as workloads: plain torch forms and the library's calls on the same inputs.

Five operators of one decoder layer's attention whose query heads share key and value heads: attention of whole prompts
(gqa_prefill), the write of keys and values into a paged cache held in 4 bits (gqa_append) and their way back (gqa_read),
attention of the newest tokens over that cache, which can add up the weight that each cached token got (gqa_attend), and the
choice of the tokens that stay by that weight (gqa_evict).  What is held in 4 bits is seen through gqa_read: the cases that write
or move it end with that call.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one long prompt
        {"name": "prompt, 1x8192", "op": "prompt", "seqs": 1, "len": 8192, "prefix": 0, "heads": 32, "kv": 8, "dim": 128, "f32": False},
        # short ragged prompts behind a cached prefix, groups of 7 heads
        {"name": "prompt, 6 ragged, prefix", "op": "prompt", "seqs": 6, "len": 700, "prefix": 333, "heads": 28, "kv": 4, "dim": 128, "f32": False},
        # many short ones of a small model, f32 as the library's own products write them
        {"name": "prompt, 24 short f32", "op": "prompt", "seqs": 24, "len": 301, "prefix": 0, "heads": 16, "kv": 2, "dim": 64, "f32": True},
        # one new token of each of 8 running sequences, written and read back: latency
        {"name": "write, 8 tokens", "op": "write", "tokens": 8, "kv": 8, "dim": 128, "gs": 32, "page": 64, "f32": True},
        # a prefill chunk written, and read back as the prefix of the next chunk
        {"name": "write, 16384 tokens", "op": "write", "tokens": 16384, "kv": 8, "dim": 128, "gs": 32, "page": 64, "f32": False},
        # a decode step of one short sequence: latency
        {"name": "step, 1x1000", "op": "step", "seqs": 1, "n_q": 1, "len": 1000, "heads": 32, "kv": 8, "dim": 128, "gs": 32, "page": 64, "weigh": False},
        # speculative tokens of a few sequences
        {"name": "step, 4x9000 of 3", "op": "step", "seqs": 4, "n_q": 3, "len": 9000, "heads": 28, "kv": 4, "dim": 128, "gs": 64, "page": 16, "weigh": False},
        # a serving batch with long contexts
        {"name": "step, 48x12000", "op": "step", "seqs": 48, "n_q": 1, "len": 12000, "heads": 64, "kv": 8, "dim": 128, "gs": 32, "page": 64, "weigh": False},
        # one very long context
        {"name": "step, 1x100000", "op": "step", "seqs": 1, "n_q": 1, "len": 100000, "heads": 32, "kv": 8, "dim": 128, "gs": 128, "page": 64, "weigh": False},
        # a batch whose cached tokens' weights are added up, for an eviction later
        {"name": "step, 16x8000 weighed", "op": "step", "seqs": 16, "n_q": 1, "len": 8000, "heads": 32, "kv": 8, "dim": 128, "gs": 32, "page": 64, "weigh": True},
        # one sequence cut to a quarter, and read back
        {"name": "evict, 1x4096", "op": "evict", "seqs": 1, "len": 4096, "keep": 1024, "recent": 128, "kv": 8, "dim": 128, "gs": 32, "page": 64},
        # a batch of long ones
        {"name": "evict, 12x16000", "op": "evict", "seqs": 12, "len": 16000, "keep": 4001, "recent": 64, "kv": 8, "dim": 128, "gs": 32, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cache_kind(rng):
    """A head layout and a cache layout."""
    dim = rng.choice([64, 128, 128])
    return {"kv": rng.choice([1, 2, 4, 8]), "dim": dim, "gs": rng.choice([32, 32, 64, dim]), "page": rng.choice([16, 32, 48, 64, 128])}


def draw(rng):
    op = rng.choice(["prompt", "prompt", "write", "step", "step", "step", "evict"])
    if op == "prompt":
        seqs, kv = _log(rng, 1, 24), rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 3, 4, 7, 8])
        most = int(8192 / math.sqrt(seqs * max(1.0, heads / 32)) / 1.5)
        n = _log(rng, 1, most)
        return {"op": op, "seqs": seqs, "len": n, "prefix": rng.choice([0, 0, _log(rng, 1, most // 2)]), "heads": heads, "kv": kv,
                "dim": rng.choice([64, 128, 128]), "f32": rng.random() < 0.3}
    c = {"op": op, **_cache_kind(rng)}
    if op == "write":
        return {**c, "tokens": _log(rng, 1, 16384), "f32": rng.random() < 0.5}
    if op == "evict":
        seqs = _log(rng, 1, 12)
        n = _log(rng, 16, 16000)
        keep = rng.randint(max(1, n // 8), max(1, n // 3))
        return {**c, "seqs": seqs, "len": n, "keep": keep, "recent": rng.randint(0, min(keep, 256))}
    n_q, group = rng.choice([1, 1, 1, 2, 5]), rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    seqs = _log(rng, 1, 48)
    rows = -(-n_q * group // 16)
    most = min(100000, 48 * 12000 // (seqs * rows))
    return {**c, "seqs": seqs, "n_q": n_q, "len": _log(rng, 4, most), "heads": c["kv"] * group, "weigh": rng.random() < 0.3}


def _lengths(case):
    """The sequences' lengths: the first has `len`, the others between a quarter of it and all of it."""
    r = random.Random("%d %d" % (case["seqs"], case["len"]))
    return [case["len"]] + [r.randint(max(1, case["len"] // 4), case["len"]) for _ in range(case["seqs"] - 1)]


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


# ------------------------------------------------------------------ inputs
def _tables(lens, page, more, g):
    """Page tables of sequences of the given lengths, their pages in no order, and the number of pages; `more` spare ones."""
    per = [-(-n // page) for n in lens]
    total = sum(per) + more
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return table, order[at:], total


def _fill(s, case, pages, g):
    """A cache of that many pages: random codes, scales of values around 1."""
    kv, page, dim, gs = case["kv"], case["page"], case["dim"], case["gs"]
    for name in ("k", "v"):
        s[name] = torch.randint(0, 256, (pages, kv, page, dim // 2), device=DEV, dtype=torch.uint8, generator=g)
        s[name + "_scales"] = (torch.rand(pages, kv, page, dim // gs, device=DEV, generator=g) * 0.3 + 0.05).to(torch.bfloat16)
    s["weights"] = None


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case), "scale": 1.0 / math.sqrt(case["dim"])}
    rnd = lambda *shape: torch.randn(*shape, device=DEV, generator=g)  # noqa: E731
    i32 = lambda v: torch.tensor(v, device=DEV, dtype=torch.int32)  # noqa: E731
    if op == "prompt":
        lens, h, kv, d = _lengths(case), case["heads"], case["kv"], case["dim"]
        cu_q, cu_k = _offsets(lens), _offsets([n + case["prefix"] for n in lens])
        kind = torch.float32 if case["f32"] else torch.bfloat16
        kv_rows = rnd(cu_k[-1], 2 * kv, d).to(kind)  # keys and values of a token in one row, as one product writes them
        s.update(cu_q=i32(cu_q), cu_k=i32(cu_k), max_q=max(lens), max_k=max(lens) + case["prefix"], q=rnd(cu_q[-1], h, d).to(kind),
                 k=kv_rows[:, :kv], v=kv_rows[:, kv:], out=torch.empty(cu_q[-1], h, d, device=DEV, dtype=torch.bfloat16))
        return s
    kv, page, d, gs = case["kv"], case["page"], case["dim"], case["gs"]
    if op == "write":
        t = case["tokens"]
        s["pages"], _, total = _tables([t], page, 2, g)
        i = torch.arange(t, device=DEV)
        new = rnd(t, 2 * kv, d) * (torch.rand(t, 2 * kv, 1, device=DEV, generator=g) * 3 + 0.1)
        new = new if case["f32"] else new.to(torch.bfloat16)
        for name in ("k", "v"):
            s[name] = torch.zeros(total, kv, page, d // 2, device=DEV, dtype=torch.uint8)
            s[name + "_scales"] = torch.zeros(total, kv, page, d // gs, device=DEV, dtype=torch.bfloat16)
        s.update(weights=None, new_k=new[:, :kv], new_v=new[:, kv:], slots=s["pages"].long()[0, i // page] * page + i % page, cu=i32([0, t]),
                 out_k=torch.empty(t, kv, d, device=DEV, dtype=torch.bfloat16), out_v=torch.empty(t, kv, d, device=DEV, dtype=torch.bfloat16))
    elif op == "step":
        lens, b, nq, h = _lengths(case), case["seqs"], case["n_q"], case["heads"]
        s["pages"], _, total = _tables(lens, page, 3, g)
        _fill(s, case, total, g)
        if case["weigh"]:
            s["weights"] = torch.zeros(total, kv, page, device=DEV)
        s.update(lens=i32(lens), q=rnd(b, nq, h, d).to(torch.bfloat16), out=torch.empty(b, nq, h, d, device=DEV, dtype=torch.bfloat16))
    else:
        lens, keep = _lengths(case), case["keep"]
        per = -(-keep // page)
        s["pages"], spare, total = _tables(lens, page, per * len(lens), g)
        _fill(s, case, total, g)
        # a few tokens get most of the weight, and many of them nearly nothing
        s["weights"] = torch.exp(rnd(total, kv, page) * 2.0 - 4.0) * (torch.rand(total, kv, page, device=DEV, generator=g) > 0.02)
        n = _offsets([min(keep, m) for m in lens])
        s.update(lens=i32(lens), dst=spare.view(len(lens), per).contiguous(), kept=torch.empty(len(lens), kv, keep, device=DEV, dtype=torch.int32),
                 new_lens=torch.empty(len(lens), device=DEV, dtype=torch.int32), cu=i32(n),
                 out_k=torch.empty(n[-1], kv, d, device=DEV, dtype=torch.bfloat16), out_v=torch.empty(n[-1], kv, d, device=DEV, dtype=torch.bfloat16))
    if own:
        import bit_weight_gemv_fmt1_gb300 as coli
        s["cache"] = coli.GqaCache(s["k"], s["v"], s["k_scales"], s["v_scales"], weights=s["weights"])
    return s


# ------------------------------------------------------------------ plain forms
def _values(codes, scales, page, head, at):
    """Cached rows [..., dim] in f32 at (page, head, place in the page), index tensors of one shape."""
    c = codes[page, head, at]
    x = torch.stack([c & 15, c >> 4], -1).flatten(-2).float() - 8.0
    sc = scales[page, head, at].float()
    return (x.view(*sc.shape, -1) * sc[..., None]).view(x.shape)


def _plain_prompt(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    h, kv, d = s["q"].shape[1], s["k"].shape[1], s["q"].shape[2]
    group, b = h // kv, cu_q.shape[0] - 1
    n_q, n_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    at_q = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    q = s["q"][at_q].float().view(b, -1, kv, group, d).permute(0, 2, 3, 1, 4).reshape(b, kv, -1, d)   # [b][kv][group * max_q][d]
    k, v = s["k"][at_k].float().transpose(1, 2), s["v"][at_k].float().transpose(1, 2)                 # [b][kv][max_k][d]
    seen = (j[None, None, :] < n_k[:, None, None]) & (j[None, None, :] <= i[None, :, None] + (n_k - n_q)[:, None, None])
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"]).view(b, kv, group, s["max_q"], s["max_k"])
    score = score.masked_fill_(~seen[:, None, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == float("-inf"), 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(b, kv, -1, s["max_k"]), v).view(b, kv, group, s["max_q"], d) / torch.where(z > 0, z, torch.ones_like(z))
    o = o.permute(0, 3, 1, 2, 4).reshape(b, s["max_q"], h, d)
    valid = i[None, :] < n_q[:, None]
    s["out"][at_q[valid]] = o[valid].to(torch.bfloat16)
    return s["out"]


def _plain_quantise(new, gs):
    """Packed codes and scales of new [T, kv, dim]."""
    x = new.float()
    x = x.view(*x.shape[:2], -1, gs)
    scale = (x.abs().amax(-1) / 7.0).to(torch.bfloat16)
    d = scale.float()[..., None]
    code = (x / torch.where(d > 0, d, torch.ones_like(d))).round().clamp(-8, 7).add(8).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale


def _plain_read(s, cu, pages):
    """The first tokens of the sequences, one after another, all heads."""
    page, kv = s["case"]["page"], s["case"]["kv"]
    i = torch.arange(s["out_k"].shape[0], device=DEV)
    b = torch.searchsorted(cu.long(), i, right=True) - 1
    t = i - cu.long()[b]
    head = torch.arange(kv, device=DEV)[None, :].expand(i.shape[0], kv)
    p, at = pages.long()[b, t // page][:, None].expand_as(head), (t % page)[:, None].expand_as(head)
    s["out_k"].copy_(_values(s["k"], s["k_scales"], p, head, at))
    s["out_v"].copy_(_values(s["v"], s["v_scales"], p, head, at))
    return s["out_k"], s["out_v"]


def _plain_write(s):
    page, gs = s["case"]["page"], s["case"]["gs"]
    p, at = s["slots"] // page, s["slots"] % page
    s["k"][p, :, at], s["k_scales"][p, :, at] = _plain_quantise(s["new_k"], gs)
    s["v"][p, :, at], s["v_scales"][p, :, at] = _plain_quantise(s["new_v"], gs)
    return _plain_read(s, s["cu"], s["pages"])


def _plain_step(s):
    page, kv = s["case"]["page"], s["case"]["kv"]
    b, nq, h, d = s["q"].shape
    group = h // kv
    most = s["pages"].shape[1] * page
    t = torch.arange(most, device=DEV)
    ids = s["pages"].long().clamp(min=0)[:, t // page]                                            # [b][most]
    head = torch.arange(kv, device=DEV)[None, :, None].expand(b, kv, most)
    p_at, at = ids[:, None, :].expand_as(head), (t % page).expand_as(head)
    k, v = _values(s["k"], s["k_scales"], p_at, head, at), _values(s["v"], s["v_scales"], p_at, head, at)   # [b][kv][most][d]
    q = s["q"].float().view(b, nq, kv, group, d).transpose(1, 2).reshape(b, kv, nq * group, d)
    limit = s["lens"].long()[:, None] - (nq - 1 - torch.arange(nq, device=DEV))                   # [b][nq]
    seen = (t < limit[..., None])[:, None, :, None, :].expand(b, kv, nq, group, most).reshape(b, kv, nq * group, most)
    score = (torch.matmul(q, k.transpose(-1, -2)) * s["scale"]).masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == float("-inf"), 0.0))
    z = p.sum(-1, keepdim=True)
    p = p / torch.where(z > 0, z, torch.ones_like(z))
    s["out"].copy_(torch.matmul(p, v).view(b, kv, nq, group, d).transpose(1, 2).reshape(b, nq, h, d))
    if s["weights"] is None:
        return s["out"]
    valid = (t < s["lens"].long()[:, None])[:, None, :].expand_as(head)
    s["weights"][p_at[valid], head[valid], at[valid]] += p.sum(2)[valid]
    return s["out"], s["weights"]


def _plain_evict(s):
    page, kv, keep, recent = s["case"]["page"], s["case"]["kv"], s["case"]["keep"], s["case"]["recent"]
    lens, b = s["lens"].long(), s["lens"].shape[0]
    most = s["pages"].shape[1] * page
    t = torch.arange(most, device=DEV)
    head = torch.arange(kv, device=DEV)[None, :, None]
    p_at, at = s["pages"].long().clamp(min=0)[:, None, t // page].expand(b, kv, most), (t % page).expand(b, kv, most)
    w = s["weights"][p_at, head.expand(b, kv, most), at]
    n = lens[:, None, None]
    w = torch.where(t < n - recent, w, torch.where(t < n, float("inf"), float("-inf")))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :keep]
    new = lens.clamp(max=keep)
    i = torch.arange(keep, device=DEV)
    live = (i < new[:, None, None])[..., :order.shape[-1]].expand_as(order)
    order = torch.where(live, order, most).sort(-1).values
    s["kept"].fill_(-1)
    s["kept"][..., :order.shape[-1]] = torch.where(live, order, -1)
    s["new_lens"].copy_(new)
    bi, hi, ri = live.nonzero(as_tuple=True)
    src = order[bi, hi, ri]
    sp, sa = s["pages"].long()[bi, src // page], src % page
    dp, da = s["dst"].long()[bi, ri // page], ri % page
    for name in ("k", "v", "k_scales", "v_scales", "weights"):
        s[name][dp, hi, da] = s[name][sp, hi, sa]
    return s["kept"], s["new_lens"], s["weights"], _plain_read(s, s["cu"], s["dst"])


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"prompt": _plain_prompt, "write": _plain_write, "step": _plain_step, "evict": _plain_evict}[op](s)
    import bit_weight_gemv_fmt1_gb300 as coli
    if op == "prompt":
        return coli.gqa_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], s["scale"], s["out"])
    if op == "write":
        coli.gqa_append(s["cache"], s["new_k"], s["new_v"], s["slots"])
        return coli.gqa_read(s["cache"], s["pages"], s["cu"], s["out_k"], s["out_v"])
    if op == "step":
        out = coli.gqa_attend(s["cache"], s["q"], s["pages"], s["lens"], s["scale"], s["out"], weigh=case["weigh"])
        return (out, s["weights"]) if case["weigh"] else out
    coli.gqa_evict(s["cache"], s["pages"], s["lens"], case["keep"], case["recent"], s["dst"], s["kept"], s["new_lens"])
    return s["kept"], s["new_lens"], s["weights"], coli.gqa_read(s["cache"], s["dst"], s["cu"], s["out_k"], s["out_v"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, kv, d = case["op"], case["kv"], case["dim"]
    if op == "prompt":
        lens, h = _lengths(case), case["heads"]
        tq, tk = sum(lens), sum(lens) + case["prefix"] * case["seqs"]
        pairs = sum(n * case["prefix"] + n * (n + 1) // 2 for n in lens)
        size = 4 if case["f32"] else 2
        return {"bytes": size * (tq * h * d + 2 * tk * kv * d) + 2 * tq * h * d, "flops": 4.0 * h * d * pairs}
    row = 2 * kv * (d // 2 + 2 * (d // case["gs"]))       # a token's codes and scales
    if op == "write":
        t = case["tokens"]
        return {"bytes": t * (2 * kv * d * (4 if case["f32"] else 2) + 8 + 2 * row + 2 * kv * d * 2), "flops": 4.0 * t * kv * d}
    lens = _lengths(case)
    if op == "step":
        nq, h = case["n_q"], case["heads"]
        pairs = sum(max(0, n - (nq - 1 - j)) for n in lens for j in range(nq))
        more = 8 * kv * sum(lens) if case["weigh"] else 0
        return {"bytes": sum(lens) * row + more + case["seqs"] * nq * h * d * 4 + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 4.0 * h * d * pairs}
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": sum(lens) * kv * 4 + kept * (3 * row + 2 * kv * d * 2 + 4 * kv) + case["seqs"] * kv * case["keep"] * 4,
            "flops": float(sum(lens) * kv)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rows(s, which, ids, n):
    """The first n rows of the pages `ids`, all heads, [kv][n][dim]."""
    byte = s[which][ids.long()].int()                                            # [pages][kv][page][dim / 2]
    value = torch.empty(*byte.shape[:3], byte.shape[3] * 2, device=DEV, dtype=torch.float64)
    value[..., 0::2], value[..., 1::2] = (byte % 16 - 8).double(), (byte // 16 - 8).double()
    sc = s[which + "_scales"][ids.long()].double()
    value *= sc.repeat_interleave(value.shape[-1] // sc.shape[-1], -1)
    return value.transpose(0, 1).flatten(1, 2)[:, :n]


def _exact_held(x, gs):
    """What 4 bits hold of x [T, kv, dim]."""
    x = x.double()
    parts = []
    for part in x.split(gs, -1):
        step = (part.abs().max(-1, keepdim=True).values / 7).to(torch.bfloat16).double()
        parts.append(torch.where(step > 0, torch.clamp(torch.round(part / step), -8, 7) * step, 0.0))
    return torch.cat(parts, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        out = torch.zeros(s["out"].shape, device=DEV, dtype=torch.float64)
        cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
        group = case["heads"] // case["kv"]
        for b in range(case["seqs"]):
            q, k, v = s["q"][cu_q[b]:cu_q[b + 1]], s["k"][cu_k[b]:cu_k[b + 1]], s["v"][cu_k[b]:cu_k[b + 1]]
            n, m = q.shape[0], k.shape[0]
            later = torch.ones(n, m, device=DEV, dtype=torch.bool).triu(m - n + 1)
            for head in range(case["heads"]):
                a = (q[:, head].double() @ k[:, head // group].double().T * s["scale"]).masked_fill_(later, float("-inf"))
                out[cu_q[b]:cu_q[b + 1], head] = torch.softmax(a, -1) @ v[:, head // group].double()
        return out
    if op == "write":
        return _exact_held(s["new_k"], case["gs"]), _exact_held(s["new_v"], case["gs"])
    if op == "step":
        nq, group = case["n_q"], case["heads"] // case["kv"]
        out = torch.zeros(s["out"].shape, device=DEV, dtype=torch.float64)
        weights = torch.zeros(s["k"].shape[:3], device=DEV, dtype=torch.float64)
        for b, n in enumerate(_lengths(case)):
            ids = s["pages"][b, : -(-n // case["page"])]
            k, v = _exact_rows(s, "k", ids, n), _exact_rows(s, "v", ids, n)
            got = torch.zeros(case["kv"], ids.shape[0] * case["page"], device=DEV, dtype=torch.float64)
            for j in range(nq):
                m = n - (nq - 1 - j)
                if m <= 0:
                    continue
                q = s["q"][b, j].double().view(case["kv"], group, -1)
                p = torch.softmax(torch.einsum("hgd,htd->hgt", q, k[:, :m]) * s["scale"], -1)
                out[b, j] = torch.einsum("hgt,htd->hgd", p, v[:, :m]).flatten(0, 1)
                got[:, :m] += p.sum(1)
            weights[ids.long()] = got.view(case["kv"], -1, case["page"]).transpose(0, 1)
        return (out, weights) if case["weigh"] else out
    ks, vs = [], []
    weights = s["weights"].double()
    for b, n in enumerate(_lengths(case)):
        ids = s["pages"][b, : -(-n // case["page"])]
        k, v = _exact_rows(s, "k", ids, n), _exact_rows(s, "v", ids, n)
        w = s["weights"][ids.long()].transpose(0, 1).flatten(1, 2)[:, :n].cpu().tolist()
        old = max(0, n - case["recent"])
        k_rows, v_rows = [], []
        for head in range(case["kv"]):
            best = sorted(range(old), key=lambda t: (-w[head][t], t))[: max(0, min(n, case["keep"]) - (n - old))]
            stay = torch.tensor(sorted(best) + list(range(old, n)), device=DEV)
            k_rows.append(k[head, stay])
            v_rows.append(v[head, stay])
            to = torch.arange(stay.shape[0], device=DEV)
            page_of = s["dst"][b].long()[to // case["page"]]
            weights[page_of, head, to % case["page"]] = torch.tensor(w[head], device=DEV, dtype=torch.float64)[stay]
        ks.append(torch.stack(k_rows, 1))
        vs.append(torch.stack(v_rows, 1))
    return None, None, weights, (torch.cat(ks), torch.cat(vs))
