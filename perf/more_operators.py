"""What a serving step with chunked prompts does around its products, as cases that can be timed and checked.

Three operators over the paged cache: norms and rotary positions of packed queries and keys, the same on the way of new
keys and values into the cache's pages, and attention of chunks of new tokens (of one token, of drafts, of pieces of a
prompt, mixed) over what the cache holds, with scores as they are, capped by a tanh, or with a bias by distance.

`run` computes a case in its plain form with torch where `own` is false, and through activation_sparse_predict_amd where
it is true.  `exact` computes the same outputs from the definitions in 64 bits.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # queries and keys of a question of one line, LLaMA-2-7B's heads: all latency
        dict(name="rope short", op="rope", dtype="f16", heads=32, kv_heads=32, dim=128, seqs=1, tokens=7, start=0, rotary=128,
             layout="half", scaling="none", norm=False),
        # a server's batch of prompts behind long cached texts, grouped heads with their own norms, frequencies in bands
        dict(name="rope packed", op="rope", dtype="bf16", heads=64, kv_heads=8, dim=128, seqs=13, tokens=6151, start=100000,
             rotary=128, layout="half", scaling="bands", norm=True),
        # neighbouring dimensions of half a head turn, Falcon-40B's heads
        dict(name="rope part", op="rope", dtype="f16", heads=128, kv_heads=8, dim=64, seqs=1, tokens=1501, start=0, rotary=32,
             layout="pairs", scaling="linear", norm=False),
        # a decoding step of a batch: one token for each sequence into its page
        dict(name="append step", op="append", dtype="bf16", heads=64, kv_heads=8, dim=128, page=16, seqs=32, tokens=32,
             past=4000, rotary=128, layout="half", scaling="bands", norm=True),
        # a server's batch of prompts into the cache
        dict(name="append prompts", op="append", dtype="f16", heads=32, kv_heads=8, dim=128, page=16, seqs=13, tokens=6151,
             past=900, rotary=128, layout="pairs", scaling="none", norm=False),
        # the next token of one conversation, LLaMA-2-7B's heads: all latency
        dict(name="chunk one", op="chunk", dtype="f16", heads=32, kv_heads=32, dim=128, page=16, seqs=1, tokens=1, past=1500,
             cap=0.0, slopes=False, window=0),
        # five drafted tokens of each of sixteen sequences are checked at once
        dict(name="chunk drafts", op="chunk", dtype="bf16", heads=64, kv_heads=8, dim=128, page=16, seqs=16, tokens=80,
             past=4000, cap=0.0, slopes=False, window=0),
        # a piece of a long document's prompt behind what the cache has of it
        dict(name="chunk long", op="chunk", dtype="bf16", heads=32, kv_heads=8, dim=128, page=16, seqs=1, tokens=512,
             past=32768, cap=0.0, slopes=False, window=0),
        # decoding steps and pieces of prompts in one batch, Falcon-40B's heads, large pages
        dict(name="chunk mixed", op="chunk", dtype="f16", heads=128, kv_heads=8, dim=64, page=64, seqs=24, tokens=1201,
             past=2050, cap=0.0, slopes=False, window=0),
        # a whole prompt through the cache, OPT-30B's heads
        dict(name="chunk whole", op="chunk", dtype="bf16", heads=56, kv_heads=56, dim=128, page=16, seqs=1, tokens=4096, past=0,
             cap=0.0, slopes=False, window=0),
        # capped scores in a window, wide heads: a piece of a prompt
        dict(name="chunk capped", op="chunk", dtype="bf16", heads=16, kv_heads=8, dim=256, page=16, seqs=3, tokens=2050,
             past=5000, cap=30.0, slopes=False, window=4096),
        # a bias by distance, a decoding step of a small batch
        dict(name="chunk distance", op="chunk", dtype="f16", heads=32, kv_heads=32, dim=128, page=32, seqs=8, tokens=8,
             past=2900, cap=0.0, slopes=True, window=0),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "chunk", "chunk", "chunk"])
    heads, kv_heads, dim = rng.choice([(32, 32, 128), (56, 56, 128), (128, 8, 64), (32, 8, 128), (64, 8, 128), (40, 8, 80),
                                       (16, 1, 64), (24, 24, 96), (16, 8, 256), (28, 4, 128), (71, 1, 64)])
    case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), heads=heads, kv_heads=kv_heads, dim=dim)
    if op != "chunk":
        seqs = _spread(rng, 1, 32)
        turn = dict(rotary=rng.choice([dim, dim, dim // 2, dim // 4 * 2 - 2]), layout=rng.choice(["half", "pairs"]),
                    scaling=rng.choice(["none", "linear", "bands", "ramp"]), norm=rng.random() < 0.5)
        tokens = max(seqs, _spread(rng, 1, 6000))
        if op == "rope":
            return dict(case, seqs=seqs, tokens=tokens, start=rng.choice([0, _spread(rng, 1, 1000000)]), **turn)
        return dict(case, page=rng.choice([16, 32, 64]), seqs=seqs, tokens=tokens, past=rng.choice([0, _spread(rng, 1, 4000)]),
                    **turn)
    seqs, past = _spread(rng, 1, 32), rng.choice([0, _spread(rng, 1, 30000), _spread(rng, 1, 4000)])
    # a batch of decoding steps, of drafts, or of anything up to a whole prompt, no more of it than a long case has to do
    tokens = rng.choice([seqs, seqs * _spread(rng, 2, 16), max(seqs, _spread(rng, 1, 4000))])
    while heads * dim * tokens * (past + tokens) > 4e10:
        past, tokens = past * 2 // 3, max(seqs, tokens * 2 // 3)
    return dict(case, page=rng.choice([16, 32, 64]), seqs=seqs, tokens=tokens, past=min(past, 55000000 // (kv_heads * dim * seqs)),
                cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3,
                window=rng.choice([0, 0, 0, _spread(rng, 1, 5000)]))


def _counts(case):
    """New tokens of each sequence, by the case alone: ragged unless they divide evenly, one at least, `tokens` in all."""
    n, total = case["seqs"], case["tokens"]
    if total % n == 0 and total // n <= 16:
        return [total // n] * n
    cuts = sorted(random.Random(1000 * total + n).sample(range(1, total), n - 1)) if n > 1 else []
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def _pasts(case):
    """Tokens that each sequence has in the cache before the new ones: up to `past`, one of that many."""
    r = random.Random(7 * case["past"] + case["seqs"])
    return [case["past"]] + [r.randint(0, case["past"]) for _ in range(case["seqs"] - 1)]


def _cdiv(a, b):
    return -(-a // b)


# ----------------------------------------------------------------- the inputs
def _normal(gen, *shape, dtype=torch.float32, scale=1.0):
    t = torch.randn(*shape, device=DEV, generator=gen, dtype=torch.float32 if math.prod(shape) < 1 << 26 else dtype)
    return (t * scale if scale != 1.0 else t).to(dtype)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _offsets(counts):
    at = [0]
    for n in counts:
        at.append(at[-1] + n)
    return at


# Frequencies are the definition's; factor, trained length and bounds are one set for each rule.
SCALING = {"none": {}, "linear": dict(factor=4.0), "bands": dict(factor=8.0, trained=8192, low=1.0, high=4.0),
           "ramp": dict(factor=16.0, trained=4096, low=1.0, high=32.0)}
BASE = {"none": 10000.0, "linear": 10000.0, "bands": 500000.0, "ramp": 10000.0}


def _frequencies(case):
    """Radians that each pair of dimensions turns by at every token, and what the turned values are multiplied by."""
    r, rule = case["rotary"], case["scaling"]
    p, base = SCALING[rule], BASE[rule]
    i = torch.arange(r // 2, dtype=torch.float64, device=DEV)
    f = base ** (-2 * i / r)
    if rule == "linear":
        return f / p["factor"], 1.0
    if rule == "bands":                                    # by how often a pair turns within the trained length
        share = ((p["trained"] * f / (2 * math.pi) - p["low"]) / (p["high"] - p["low"])).clamp(0, 1)
        return f * share + f / p["factor"] * (1 - share), 1.0
    if rule == "ramp":                                     # by the pair's number, between those of two such counts
        low, high = (r * math.log(p["trained"] / (2 * math.pi * n)) / (2 * math.log(base)) for n in (p["high"], p["low"]))
        low, high = max(math.floor(low), 0), min(math.ceil(high), r - 1)
        share = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - share) + f / p["factor"] * share, 0.1 * math.log(p["factor"]) + 1
    return f, 1.0


def _keep_turn(s, case, gen):
    """The frequencies and the norms' weights, as a program has them for a model."""
    d = case["dim"]
    s["freqs"], s["magnitude"] = _frequencies(case)
    s["q_norm"], s["k_norm"] = ((1 + _normal(gen, d, scale=0.2) for _ in range(2)) if case["norm"] else (None, None))
    if own:
        import activation_sparse_predict_amd as pi
        rule = case["scaling"]
        s["rope"] = pi.Rope(case["rotary"], base=BASE[rule], layout=case["layout"],
                            scaling=None if rule == "none" else rule, device=DEV, **SCALING[rule])


def _keep_cache(s, case, gen, layers, counts, pasts):
    """A pool whose pages lie anywhere, and the tables of sequences that hold their past and the new tokens."""
    page, seed = case["page"], int(s["seed"])
    lens = [a + b for a, b in zip(counts, pasts)]
    held = [_cdiv(n, page) for n in lens]
    pages, wide = sum(held) + 5, max(held) + 1
    ids = random.Random(seed).sample(range(pages), sum(held))
    table, ref, at = torch.zeros(len(lens), wide, dtype=torch.int32), [0] * pages, 0
    for i, n in enumerate(held):
        table[i, :n] = torch.tensor(ids[at:at + n], dtype=torch.int32)
        at += n
    for p in ids:
        ref[p] = 1
    free = [p for p in range(pages) if not ref[p]]
    meta = torch.cat([table.reshape(-1), torch.tensor(lens + ref + free + [0] * (pages - len(free)) + [len(free), 0, 0, 0],
                                                      dtype=torch.int32)]).to(DEV)
    shape = (layers, pages, case["kv_heads"], page, case["dim"])
    s["k_pool"], s["v_pool"] = _normal(gen, *shape, dtype=s["type"]), _normal(gen, *shape, dtype=s["type"])
    s["table"], s["lens"], s["cu"], s["seqs"] = table.to(DEV), lens, _ints(_offsets(counts)), _ints(list(range(len(lens))))
    s["counts"] = counts
    if own:                                                # the handle that a program keeps for its cache
        import activation_sparse_predict_amd as pi
        s["cache"] = pi.Cache(s["k_pool"], s["v_pool"], meta, len(lens), wide)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, counts = case["op"], _counts(case)
    t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    s = dict(case=case, seed=seed, type=TYPES[case["dtype"]])
    if op == "chunk":
        # scores that a cap reaches come from larger queries
        s["q"] = _normal(gen, t, h, d, dtype=s["type"], scale=4.0 if case["cap"] else 1.0)
        s["out"] = torch.empty_like(s["q"])
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, h + 1, device=DEV) / h) if case["slopes"] else None
        _keep_cache(s, case, gen, 1, counts, _pasts(case))
        return s
    # query, key and value are slices of one projection's output; some dimensions are larger than others
    qkv = _normal(gen, t, h + 2 * g, d) * torch.exp(0.5 * _normal(gen, h + 2 * g, d))
    qkv = qkv.to(s["type"])
    s["q"], s["k"], s["v"] = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    s["q_out"] = torch.empty(t, h, d, device=DEV, dtype=s["type"])
    _keep_turn(s, case, gen)
    if op == "rope":
        s["k_out"] = torch.empty(t, g, d, device=DEV, dtype=s["type"])
        s["pos"] = torch.cat([torch.arange(n, dtype=torch.int32) for n in counts]).add_(case["start"]).to(DEV)
    else:
        _keep_cache(s, case, gen, 2, counts, _pasts(case))
    return s


# ------------------------------------------------------------- the plain forms
def _plain_turn(s, x, weight, pos):
    """Norm and rotation of heads x [tokens, heads, dim] at positions pos."""
    r, y = s["case"]["rotary"], x.float()
    if weight is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight
    angle = (pos.double().unsqueeze(1) * s["freqs"]).unsqueeze(1)     # [tokens, 1, pairs]
    cos, sin = (torch.cos(angle) * s["magnitude"]).float(), (torch.sin(angle) * s["magnitude"]).float()
    if s["case"]["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin, y[..., r:]], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), y[..., r:]], -1)
    return turned.to(x.dtype)


def _plain_append(s):
    page, cu = s["case"]["page"], s["cu"].long()
    token = torch.arange(s["case"]["tokens"], device=DEV)
    seq = torch.searchsorted(cu, token, right=True) - 1
    lens = torch.tensor(s["lens"], device=DEV)
    pos = lens[seq] - cu[seq + 1] + token
    where = s["table"][seq, pos // page].long()
    s["k_pool"][1][where, :, pos % page] = _plain_turn(s, s["k"], s["k_norm"], pos)
    s["v_pool"][1][where, :, pos % page] = s["v"]
    return dict(q=_plain_turn(s, s["q"], s["q_norm"], pos), k=s["k_pool"], v=s["v_pool"])


def _plain_attend(s, q, tables, lens, counts):
    """Rows q [n, c, heads, dim] in 32 bits of n sequences over their pages; a sequence's first counts[i] rows exist."""
    case = s["case"]
    n, c, h, d = q.shape
    g, page = case["kv_heads"], case["page"]
    places = _cdiv(max(lens), page)
    ids, m = tables[:, :places].long(), places * page
    k = s["k_pool"][0][ids].float().permute(0, 2, 4, 1, 3).reshape(n, g, 1, d, m)
    v = s["v_pool"][0][ids].float().permute(0, 2, 1, 3, 4).reshape(n, g, 1, m, d)
    x = (q.permute(0, 2, 1, 3).reshape(n, g, h // g, c, d) * d ** -0.5) @ k
    if case["cap"]:
        x = torch.tanh(x.div_(case["cap"])).mul_(case["cap"])
    first = torch.tensor([a - b for a, b in zip(lens, counts)], device=DEV)
    pos = first.view(n, 1, 1) + torch.arange(c, device=DEV).view(1, c, 1)
    far = torch.arange(m, device=DEV) - pos                # [n, c, m]
    if s["slopes"] is not None:
        x.add_(s["slopes"].view(1, g, h // g, 1, 1) * far.view(n, 1, 1, c, m))
    unseen = (far > 0) | (far <= -case["window"]) if case["window"] else far > 0
    x.masked_fill_(unseen.view(n, 1, 1, c, m), -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    return ((p @ v) / p.sum(-1, keepdim=True)).reshape(n, h, c, d).permute(0, 2, 1, 3)


def _plain_chunk(s):
    """Sequences as one batch where they are much alike, one after the other where they are not."""
    q, lens, counts = s["q"].float(), s["lens"], s["counts"]
    n, c = len(lens), max(counts)
    if n * c * max(lens) <= 2 * sum(a * b for a, b in zip(lens, counts)) and min(counts) == c:
        return _plain_attend(s, q.view(n, c, *q.shape[1:]), s["table"], lens, counts).reshape(q.shape).to(s["type"])
    out, at = torch.empty_like(s["q"]), _offsets(counts)
    for i in range(n):
        rows = slice(at[i], at[i + 1])
        out[rows] = _plain_attend(s, q[rows].unsqueeze(0), s["table"][i:i + 1], lens[i:i + 1], counts[i:i + 1])[0]
    return out


def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    if op == "rope":
        return dict(q=_plain_turn(s, s["q"], s["q_norm"], s["pos"]), k=_plain_turn(s, s["k"], s["k_norm"], s["pos"]))
    return _plain_append(s) if op == "append" else _plain_chunk(s)


def _run_own(s, op):
    import activation_sparse_predict_amd as pi
    case = s["case"]
    if op == "rope":
        pi.rope_heads(s["rope"], s["pos"], s["q"], s["q_out"], s["k"], s["k_out"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        return dict(q=s["q_out"], k=s["k_out"])
    if op == "append":
        s["cache"].append_rope(1, s["rope"], s["q"], s["q_out"], s["k"], s["v"], s["cu"], s["seqs"], q_norm=s["q_norm"],
                               k_norm=s["k_norm"], eps=EPS)
        return dict(q=s["q_out"], k=s["k_pool"], v=s["v_pool"])
    pi.attn_chunk(s["cache"], 0, s["q"], s["out"], s["cu"], s["seqs"], cap=case["cap"], slopes=s["slopes"],
                  window=case["window"])
    return s["out"]


# ------------------------------------------------------- the work, and 64 bits
def work(case):
    t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] != "chunk":
        rows = h + g if case["op"] == "rope" else h + 2 * g
        return dict(bytes=4 * t * rows * d + 4 * t, flops=t * (h + g) * (3 * case["rotary"] + 4 * d * case["norm"]))
    keys = pairs = 0
    for c, past in zip(_counts(case), _pasts(case)):
        w = case["window"] or past + c
        keys += min(past + c, c - 1 + w)                   # those that any row sees
        low = max(0, min(c, w - past))                     # rows that see all before them: past + 1, past + 2, ...
        pairs += low * past + low * (low + 1) // 2 + (c - low) * w
    return dict(bytes=4 * g * d * keys + 4 * t * h * d, flops=4 * h * d * pairs)


def _exact_turn(case, x, weight, pos):
    """Norm and rotation in 64 bits: a pair of dimensions as a complex number times m e^(i p f)."""
    r, rule, x = case["rotary"], case["scaling"], x.double()
    if weight is not None:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["dim"] + EPS) * weight.double()
    p, base, freqs, m = SCALING[rule], BASE[rule], [], 1.0
    for i in range(r // 2):
        f = math.exp(-2 * i / r * math.log(base))
        keep = 1.0                                         # how much of the pair's own frequency stays
        if rule == "linear":
            keep = 0.0
        elif rule == "bands":
            turns = p["trained"] * f / (2 * math.pi)
            keep = 0.0 if turns < p["low"] else 1.0 if turns > p["high"] else (turns - p["low"]) / (p["high"] - p["low"])
        elif rule == "ramp":
            def pair_of(turns):                            # the pair that turns so often within the trained length
                return r / 2 * math.log(p["trained"] / turns / (2 * math.pi), base)
            a, b = max(0, math.floor(pair_of(p["high"]))), min(r - 1, math.ceil(pair_of(p["low"])))
            keep = 1.0 - min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            m = 1.0 + 0.1 * math.log(p["factor"])
        freqs.append(f * keep + f * (1.0 - keep) / p.get("factor", 1.0))
    angle = torch.outer(pos.double(), torch.tensor(freqs, dtype=torch.float64, device=DEV))
    turn = torch.polar(torch.full_like(angle, m), angle)[:, None, :]
    out = x.clone()
    if case["layout"] == "half":
        z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn
        out[..., :r // 2], out[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * turn
        out[..., 0:r:2], out[..., 1:r:2] = z.real, z.imag
    return out


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "rope":
        return dict(q=_exact_turn(case, s["q"], s["q_norm"], s["pos"]), k=_exact_turn(case, s["k"], s["k_norm"], s["pos"]))
    group, page = case["heads"] // case["kv_heads"], case["page"]
    tables, at = s["table"].tolist(), _offsets(s["counts"])
    if case["op"] == "append":                             # values are moved as they are
        pos = torch.cat([torch.arange(n - c, n) for n, c in zip(s["lens"], s["counts"])])
        q, k = (_exact_turn(case, x, w, pos.to(DEV)) for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])))
        pool = s["k_pool"].double()
        page_of = [tables[i][n // page] for i in range(case["seqs"]) for n in range(s["lens"][i] - s["counts"][i], s["lens"][i])]
        pool[1].index_put_((torch.tensor(page_of, device=DEV)[:, None], torch.arange(case["kv_heads"], device=DEV)[None, :],
                            (pos % page).to(DEV)[:, None]), k)
        return dict(q=q, k=pool, v=None)
    out = torch.empty(case["tokens"], case["heads"], case["dim"], dtype=torch.float64, device=DEV)
    for i, (n, c) in enumerate(zip(s["lens"], s["counts"])):
        ids = torch.tensor(tables[i][:_cdiv(n, page)], device=DEV)
        k, v = (pool[0].index_select(0, ids).transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[:n].double()
                for pool in (s["k_pool"], s["v_pool"]))
        back = torch.arange(n - c, n, device=DEV)[:, None] - torch.arange(n, device=DEV)[None, :]
        sees = back >= 0
        if case["window"]:
            sees &= back < case["window"]
        for j in range(case["heads"]):
            x = torch.mm(s["q"][at[i]:at[i + 1], j].double(), k[:, j // group].T.contiguous()) / math.sqrt(case["dim"])
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if s["slopes"] is not None:
                x = x - float(s["slopes"][j]) * back
            x = torch.where(sees, x, torch.full_like(x, -math.inf))
            out[at[i]:at[i + 1], j] = torch.mm(torch.softmax(x, 1), v[:, j // group].contiguous())
    return out
