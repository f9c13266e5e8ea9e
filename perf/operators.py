"""The latent-attention (MLA) operators, as workloads: plain torch forms and the library's calls on the same inputs.

Five operators of one decoder layer's attention, in the order a layer runs them: the queries' split and rotation
(mla_query), the write of new tokens into the paged latent cache with norm, rotation and quantisation (mla_append),
reading cached rows back (mla_read), attention of the newest tokens over the cache in the absorbed form (mla_attend)
and attention of whole prompts in the expanded form (mla_prefill).
"""
import math
import random

import torch

own = False

L, R = 512, 64      # latent and rotary dims of a cached row
N, V = 128, 128     # no-position key dims and value dims of a head
EPS = 1e-6
E4M3_MAX = 448.0
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the queries of one decode step of one sequence: latency
        {"name": "query, one token", "op": "query", "tokens": 1, "heads": 128, "bf16": False, "interleaved": False},
        # the queries of a prompt, 64 heads, on their way to the expanded form
        {"name": "query, prompt of 6001", "op": "query", "tokens": 6001, "heads": 64, "bf16": True, "interleaved": True},
        # one new token of each of 8 running sequences
        {"name": "append, 8 tokens e4m3", "op": "append", "tokens": 8, "e4m3": True, "page": 64, "interleaved": False},
        # a prefill chunk of 16k tokens written at once
        {"name": "append, 16384 tokens e4m3", "op": "append", "tokens": 16384, "e4m3": True, "page": 64, "interleaved": True},
        # a short cached prefix read back
        {"name": "read, 2 short e4m3", "op": "read", "seqs": 2, "len": 300, "e4m3": True, "page": 16, "bf16": False},
        # the prefixes of 7 sequences read back to be expanded again
        {"name": "read, 7 long bf16", "op": "read", "seqs": 7, "len": 20000, "e4m3": False, "page": 64, "bf16": True},
        # a decode step of one short sequence: latency
        {"name": "attend, 1x1000 e4m3", "op": "attend", "seqs": 1, "n_q": 1, "heads": 128, "len": 1000, "e4m3": True, "page": 64},
        # speculative tokens of a few sequences on one of several tensor-parallel ranks
        {"name": "attend, 4x9000 16 heads bf16", "op": "attend", "seqs": 4, "n_q": 3, "heads": 16, "len": 9000, "e4m3": False, "page": 32},
        # a serving batch with long contexts, 8-bit cache
        {"name": "attend, 48x12000 e4m3", "op": "attend", "seqs": 48, "n_q": 1, "heads": 128, "len": 12000, "e4m3": True, "page": 64},
        # one very long context in bf16
        {"name": "attend, 1x100000 bf16", "op": "attend", "seqs": 1, "n_q": 1, "heads": 128, "len": 100000, "e4m3": False, "page": 64},
        # short ragged prompts behind a cached prefix
        {"name": "prefill, 5 ragged, prefix", "op": "prefill", "seqs": 5, "len": 700, "prefix": 333, "heads": 16},
        # one long prompt
        {"name": "prefill, 1x8192", "op": "prefill", "seqs": 1, "len": 8192, "prefix": 0, "heads": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["query", "append", "read", "attend", "attend", "prefill"])
    if op == "query":
        heads = rng.choice([8, 16, 24, 64, 128])
        return {"op": op, "tokens": _log(rng, 1, 6001 * 64 // heads), "heads": heads, "bf16": rng.random() < 0.5,
                "interleaved": rng.random() < 0.5}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 16384), "e4m3": rng.random() < 0.7, "page": rng.choice([16, 32, 64, 128]),
                "interleaved": rng.random() < 0.5}
    if op == "read":
        seqs = _log(rng, 1, 16)
        return {"op": op, "seqs": seqs, "len": _log(rng, 1, 100000 // seqs), "e4m3": rng.random() < 0.6,
                "page": rng.choice([16, 32, 64, 128]), "bf16": rng.random() < 0.5}
    if op == "attend":
        heads, n_q = rng.choice([8, 16, 20, 32, 64, 128]), rng.choice([1, 1, 1, 2, 4])
        seqs = _log(rng, 1, 48)
        most = min(100000, 48 * 12000 // seqs, 48 * 12000 * 128 // (seqs * heads * n_q))
        return {"op": op, "seqs": seqs, "n_q": n_q, "heads": heads, "len": _log(rng, 4, most), "e4m3": rng.random() < 0.6,
                "page": rng.choice([16, 32, 64, 128])}
    heads, seqs = rng.choice([4, 16, 32]), _log(rng, 1, 8)
    most = int(8192 / math.sqrt(seqs) / 1.5)
    n = _log(rng, 1, most)
    return {"op": op, "seqs": seqs, "len": n, "prefix": rng.choice([0, 0, _log(rng, 1, most // 2)]), "heads": heads}


def _lengths(case):
    """The sequences' lengths: the first has `len`, the others between a quarter of it and all of it."""
    r = random.Random("%d %d" % (case["seqs"], case["len"]))
    return [case["len"]] + [r.randint(max(1, case["len"] // 4), case["len"]) for _ in range(case["seqs"] - 1)]


# ------------------------------------------------------------------ inputs
def _rotation(n_pos):
    """cos | sin of the positions' angles, [n_pos][R]."""
    f = 10000.0 ** (-torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
    a = torch.arange(n_pos, device=DEV, dtype=torch.float64)[:, None] * f[None, :]
    return torch.cat([a.cos(), a.sin()], 1).float()


def _cache(case, lens, g):
    """A paged cache holding sequences of the given lengths, its page table and its rows' values."""
    page = case["page"]
    per = [-(-n // page) for n in lens]
    total = sum(per) + 3
    rows = torch.randn(total, page, L + R, device=DEV, generator=g)
    scales = None
    if case["e4m3"]:
        rows *= torch.rand(total, page, 1, device=DEV, generator=g) + 0.5
        scales = rows.abs().amax(-1) / E4M3_MAX
        rows = (rows / scales[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    else:
        rows = rows.to(torch.bfloat16)
    order = torch.randperm(total, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(per)), -1, device=DEV, dtype=torch.int32)
    at = 0
    for b, n in enumerate(per):
        table[b, :n] = order[at:at + n]
        at += n
    return rows, scales, table


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    s = {"case": dict(case)}
    rnd = lambda *shape: torch.randn(*shape, device=DEV, generator=g)  # noqa: E731
    if op == "query":
        t, h = case["tokens"], case["heads"]
        out = torch.bfloat16 if case["bf16"] else torch.float32
        s.update(q=rnd(t, h, N + R), pos=torch.arange(37, 37 + t, device=DEV, dtype=torch.int32), rot=_rotation(t + 64))
        if case["bf16"]:  # one row a head, as the expanded form reads it
            s["row"] = torch.empty(t, h, N + R, device=DEV, dtype=out)
            s["nope"], s["rope"] = s["row"][..., :N], s["row"][..., N:]
        else:
            s["nope"], s["rope"] = torch.empty(t, h, N, device=DEV, dtype=out), torch.empty(t, h, R, device=DEV, dtype=out)
    elif op == "append":
        t, page = case["tokens"], case["page"]
        pages = -(-t // page) + 2
        s.update(kv=rnd(t, L + R) * (torch.rand(t, 1, device=DEV, generator=g) * 3 + 0.1), norm=torch.rand(L, device=DEV, generator=g) + 0.5,
                 pos=torch.arange(11, 11 + t, device=DEV, dtype=torch.int32), rot=_rotation(t + 16),
                 slots=torch.randperm(pages * page, device=DEV, generator=g)[:t].contiguous(),
                 rows=torch.zeros(pages, page, L + R, device=DEV, dtype=torch.float8_e4m3fn if case["e4m3"] else torch.bfloat16),
                 scales=torch.zeros(pages, page, device=DEV) if case["e4m3"] else None)
    elif op == "read":
        lens = _lengths(case)
        s["rows"], s["scales"], s["pages"] = _cache(case, lens, g)
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        s["cu"] = torch.tensor(cu, device=DEV, dtype=torch.int32)
        s["out"] = torch.empty(cu[-1], L + R, device=DEV, dtype=torch.bfloat16 if case["bf16"] else torch.float32)
    elif op == "attend":
        lens = _lengths(case)
        b, nq, h = case["seqs"], case["n_q"], case["heads"]
        s["rows"], s["scales"], s["pages"] = _cache(case, lens, g)
        s.update(lens=torch.tensor(lens, device=DEV, dtype=torch.int32), q_latent=rnd(b, nq, h, L).to(torch.bfloat16),
                 q_rope=rnd(b, nq, h, R).to(torch.bfloat16), scale=1.0 / math.sqrt(N + R),
                 out=torch.empty(b, nq, h, L, device=DEV, dtype=torch.bfloat16))
    else:
        lens, h = _lengths(case), case["heads"]
        cu_q, cu_k = [0], [0]
        for n in lens:
            cu_q.append(cu_q[-1] + n)
            cu_k.append(cu_k[-1] + n + case["prefix"])
        s.update(cu_q=torch.tensor(cu_q, device=DEV, dtype=torch.int32), cu_k=torch.tensor(cu_k, device=DEV, dtype=torch.int32),
                 max_q=max(lens), max_k=max(lens) + case["prefix"], scale=1.0 / math.sqrt(N + R),
                 q=rnd(cu_q[-1], h, N + R).to(torch.bfloat16), kv=rnd(cu_k[-1], h, N + V).to(torch.bfloat16),
                 k_rope=rnd(cu_k[-1], R).to(torch.bfloat16), out=torch.empty(cu_q[-1], h, V, device=DEV, dtype=torch.bfloat16))
    if own and "rows" in s:
        import bit_weight_gemv_fmt1_gb300 as coli
        s["cache"] = coli.MlaCache(s["rows"], latent=L, rope=R, scales=s["scales"])
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, rot, interleaved):
    """x [..., R] turned by rot [..., R] = cos | sin."""
    c, s = rot[..., :R // 2], rot[..., R // 2:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x[..., :R // 2], x[..., R // 2:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _plain_query(s):
    rot = s["rot"][s["pos"].long()][:, None, :]
    s["nope"].copy_(s["q"][..., :N])
    s["rope"].copy_(_rotate(s["q"][..., N:], rot, s["case"]["interleaved"]))
    return s["nope"], s["rope"]


def _plain_append(s):
    c = s["kv"][:, :L]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["norm"]
    k = _rotate(s["kv"][:, L:], s["rot"][s["pos"].long()], s["case"]["interleaved"])
    row = torch.cat([c, k], -1)
    flat = s["rows"].view(-1, L + R)
    if s["scales"] is None:
        flat[s["slots"]] = row.to(torch.bfloat16)
        return s["rows"]
    scale = row.abs().amax(-1) / E4M3_MAX
    code = (row / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    flat.view(torch.uint8)[s["slots"]] = code.view(torch.uint8)
    s["scales"].view(-1)[s["slots"]] = scale
    return s["rows"], s["scales"]


def _rows_at(s, slot):
    """The cached rows at the slots, in f32."""
    r = s["rows"].view(-1, L + R)
    if s["scales"] is None:
        return r[slot].float()
    r = r.view(torch.uint8)[slot].view(torch.float8_e4m3fn).float()
    return r * s["scales"].view(-1)[slot][..., None]


def _plain_read(s):
    page = s["case"]["page"]
    i = torch.arange(s["out"].shape[0], device=DEV)
    b = torch.searchsorted(s["cu"].long(), i, right=True) - 1
    t = i - s["cu"].long()[b]
    s["out"].copy_(_rows_at(s, s["pages"].long()[b, t // page] * page + t % page))
    return s["out"]


def _plain_attend(s):
    page = s["case"]["page"]
    b, nq, h, _ = s["q_latent"].shape
    most = s["pages"].shape[1] * page
    t = torch.arange(most, device=DEV)
    slot = s["pages"].long().clamp(min=0)[:, t // page] * page + t % page
    rows = _rows_at(s, slot)                                                     # [b][most][L+R]
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float().view(b, nq * h, L + R)
    limit = s["lens"].long()[:, None] - (nq - 1 - torch.arange(nq, device=DEV))  # [b][nq]
    seen = (t < limit[..., None])[:, :, None, :].expand(b, nq, h, most).reshape(b, nq * h, most)
    score = (torch.matmul(q, rows.transpose(1, 2)) * s["scale"]).masked_fill(~seen, float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top.masked_fill(top == float("-inf"), 0.0))
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, rows[..., :L]) / torch.where(z > 0, z, torch.ones_like(z))
    s["out"].copy_(o.view(b, nq, h, L))
    return s["out"]


def _plain_prefill(s):
    cu_q, cu_k = s["cu_q"].long(), s["cu_k"].long()
    h = s["q"].shape[1]
    n_q, n_k = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    i, j = torch.arange(s["max_q"], device=DEV), torch.arange(s["max_k"], device=DEV)
    at_q = (cu_q[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp(max=s["kv"].shape[0] - 1)
    q = s["q"][at_q].float().transpose(1, 2)                                     # [b][h][max_q][N+R]
    kv = s["kv"][at_k].float().transpose(1, 2)                                   # [b][h][max_k][N+V]
    k_rope = s["k_rope"][at_k].float()[:, None].expand(-1, h, -1, -1)
    seen = (j[None, None, :] < n_k[:, None, None]) & (j[None, None, :] <= i[None, :, None] + (n_k - n_q)[:, None, None])
    score = torch.matmul(q, torch.cat([kv[..., :N], k_rope], -1).transpose(-1, -2)) * s["scale"]
    score = score.masked_fill_(~seen[:, None], float("-inf"))
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == float("-inf"), 0.0)).exp_()
    z = p.sum(-1, keepdim=True)
    o = (torch.matmul(p, kv[..., N:]) / torch.where(z > 0, z, torch.ones_like(z))).transpose(1, 2)
    valid = i[None, :] < n_q[:, None]
    s["out"][at_q[valid]] = o[valid].to(torch.bfloat16)
    return s["out"]


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"query": _plain_query, "append": _plain_append, "read": _plain_read, "attend": _plain_attend,
                "prefill": _plain_prefill}[op](s)
    import bit_weight_gemv_fmt1_gb300 as coli
    if op == "query":
        coli.mla_query(s["q"], s["pos"], s["rot"], s["nope"], s["rope"], interleaved=case["interleaved"])
        return s["nope"], s["rope"]
    if op == "append":
        coli.mla_append(s["cache"], s["kv"], s["norm"], EPS, s["pos"], s["rot"], s["slots"], interleaved=case["interleaved"])
        return s["rows"] if s["scales"] is None else (s["rows"], s["scales"])
    if op == "read":
        return coli.mla_read(s["cache"], s["pages"], s["cu"], s["out"])
    if op == "attend":
        return coli.mla_attend(s["cache"], s["q_latent"], s["q_rope"], s["pages"], s["lens"], s["scale"], s["out"])
    return coli.mla_prefill(s["q"], s["kv"], s["k_rope"], s["cu_q"], s["cu_k"], s["scale"], s["out"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "query":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * (N + R) * (4 + (2 if case["bf16"] else 4)) + case["tokens"] * (4 + 4 * R), "flops": 3.0 * n * R}
    if op == "append":
        t = case["tokens"]
        stored = L + R + 4 if case["e4m3"] else 2 * (L + R)
        return {"bytes": t * (4 * (L + R) + stored + 4 * R + 12) + 4 * L, "flops": t * (4.0 * L + 3.0 * R)}
    if op == "read":
        t = sum(_lengths(case))
        return {"bytes": t * ((L + R + 4 if case["e4m3"] else 2 * (L + R)) + (L + R) * (2 if case["bf16"] else 4)), "flops": float(t * (L + R))}
    if op == "attend":
        lens, nq, h = _lengths(case), case["n_q"], case["heads"]
        rows = sum(lens) * (L + R + 4 if case["e4m3"] else 2 * (L + R))
        pairs = sum(max(0, n - (nq - 1 - j)) for n in lens for j in range(nq))
        return {"bytes": rows + case["seqs"] * nq * h * 2 * (2 * L + R) + 4 * sum(-(-n // case["page"]) for n in lens),
                "flops": 2.0 * h * pairs * (2 * L + R)}
    lens, h = _lengths(case), case["heads"]
    tq, tk = sum(lens), sum(lens) + case["prefix"] * case["seqs"]
    pairs = sum(n * case["prefix"] + n * (n + 1) // 2 for n in lens)
    return {"bytes": 2 * (tq * h * (N + R + V) + tk * (h * (N + V) + R)), "flops": 2.0 * h * pairs * (N + R + V)}


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rotate(x, cos, sin, interleaved):
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :R // 2], x[..., R // 2:])
    z = z * torch.complex(cos, sin)
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def _exact_sequence(s, b, n):
    """The first n cached rows of sequence b."""
    page = s["rows"].shape[1]
    ids = s["pages"][b, : -(-n // page)].long()
    rows = s["rows"].view(torch.uint8)[ids].view(s["rows"].dtype).double()
    if s["scales"] is not None:
        rows = rows * s["scales"][ids].double()[..., None]
    return rows.reshape(-1, L + R)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "query":
        rot = s["rot"].double()[s["pos"].long()][:, None, :]
        q = s["q"].double()
        return q[..., :N].contiguous(), _exact_rotate(q[..., N:], rot[..., :R // 2], rot[..., R // 2:], case["interleaved"])
    if op == "append":
        kv = s["kv"].double()
        ms = kv[:, :L].square().sum(-1, keepdim=True) / L
        rot = s["rot"].double()[s["pos"].long()]
        row = torch.cat([kv[:, :L] / (ms + EPS).sqrt() * s["norm"].double(),
                         _exact_rotate(kv[:, L:], rot[:, :R // 2], rot[:, R // 2:], case["interleaved"])], -1)
        rows = torch.zeros(s["rows"].shape, device=DEV, dtype=torch.float64)
        if s["scales"] is None:
            rows.view(-1, L + R)[s["slots"]] = row
            return rows
        scales = torch.zeros(s["scales"].shape, device=DEV, dtype=torch.float64)
        amax = row.abs().max(-1).values / E4M3_MAX
        rows.view(-1, L + R)[s["slots"]] = row / amax[:, None]
        scales.view(-1)[s["slots"]] = amax
        return rows, scales
    if op == "read":
        return torch.cat([_exact_sequence(s, b, n) for b, n in enumerate(_lengths(case))])
    if op == "attend":
        nq, h = case["n_q"], case["heads"]
        out = torch.zeros(s["out"].shape, device=DEV, dtype=torch.float64)
        for b, n in enumerate(_lengths(case)):
            rows = _exact_sequence(s, b, n)
            for j in range(nq):
                m = n - (nq - 1 - j)
                if m > 0:
                    a = s["q_latent"][b, j].double() @ rows[:m, :L].T + s["q_rope"][b, j].double() @ rows[:m, L:].T
                    out[b, j] = torch.softmax(a * s["scale"], -1) @ rows[:m, :L]
        return out
    out = torch.zeros(s["out"].shape, device=DEV, dtype=torch.float64)
    cu_q, cu_k = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(case["seqs"]):
        q, kv = s["q"][cu_q[b]:cu_q[b + 1]], s["kv"][cu_k[b]:cu_k[b + 1]]
        kr = s["k_rope"][cu_k[b]:cu_k[b + 1]].double()
        n, m = q.shape[0], kv.shape[0]
        later = torch.ones(n, m, device=DEV, dtype=torch.bool).triu(m - n + 1)
        for head in range(case["heads"]):
            a = q[:, head, :N].double() @ kv[:, head, :N].double().T + q[:, head, N:].double() @ kr.T
            a = (a * s["scale"]).masked_fill_(later, float("-inf"))
            out[cu_q[b]:cu_q[b + 1], head] = torch.softmax(a, -1) @ kv[:, head, N:].double()
    return out
