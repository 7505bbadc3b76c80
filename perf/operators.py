"""The cases on which the library's operators beside the weight products are measured.

Three operators, each in its plain form (elementary torch operations in 32
bits) and, where ``own`` is true, through the library's entry points:

* ``attention``: new tokens of several sequences over a paged key/value cache;
* ``heads``: per-head norms of queries and keys with the position rotation,
  and the append of keys and values to the paged cache;
* ``adapters``: low-rank adapters of many requests added to a projection's
  output.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user's next token on a short chat, heads of a 4096-wide model: all latency
        dict(name="attention_1x512", op="attention", type="fp16", seqs=1, heads=32, kv_heads=32,
             dim=128, new=1, ones=0, longest=512, spread=0.0, page=16, window=0),
        # a decode step of 48 requests of very different lengths, 8 query heads to a key head
        dict(name="attention_48x8000", op="attention", type="bf16", seqs=48, heads=64, kv_heads=8,
             dim=128, new=1, ones=0, longest=8000, spread=0.9, page=32, window=0),
        # a decode step of four requests on whole documents: 2 GB of cache to read
        dict(name="attention_4x131072", op="attention", type="fp16", seqs=4, heads=64, kv_heads=8,
             dim=128, new=1, ones=0, longest=131072, spread=0.1, page=64, window=0),
        # a chunk of a long prompt, all its keys visible: the matrix products bound it
        dict(name="attention_chunk_2048", op="attention", type="bf16", seqs=1, heads=32,
             kv_heads=8, dim=128, new=2048, ones=0, longest=16384, spread=0.0, page=64, window=0),
        # a mixed batch: prompt chunks of odd lengths beside single tokens, small heads
        dict(name="attention_mixed", op="attention", type="fp16", seqs=16, heads=32, kv_heads=32,
             dim=64, new=253, ones=6, longest=4099, spread=0.8, page=16, window=0),
        # a decode step of 8 requests between the QKV product and the attention
        dict(name="heads_8", op="heads", type="fp16", tokens=8, heads=32, kv_heads=32, dim=128,
             rotary=128, pairs="halves", norm=True, page=16),
        # a prompt chunk of an odd length, rotation of half of each small head, no norms
        dict(name="heads_1013", op="heads", type="fp16", tokens=1013, heads=32, kv_heads=4, dim=64,
             rotary=32, pairs="neighbours", norm=False, page=16),
        # a long prompt with grouped heads, norms and rotation
        dict(name="heads_8192", op="heads", type="bf16", tokens=8192, heads=64, kv_heads=8,
             dim=128, rotary=128, pairs="halves", norm=True, page=64),
        # one request with its adapter on a square projection: all latency
        dict(name="adapters_1", op="adapters", type="fp16", rows=1, K=4096, N=4096, rank=16,
             adapters=1, without=0, order="runs"),
        # a decode step of 32 requests with 16 adapters on a fused QKV projection
        dict(name="adapters_32", op="adapters", type="fp16", rows=32, K=4096, N=12288, rank=16,
             adapters=16, without=3, order="mixed"),
        # an odd batch with wide adapters on a down projection
        dict(name="adapters_61", op="adapters", type="bf16", rows=61, K=11008, N=4096, rank=64,
             adapters=24, without=5, order="mixed"),
        # prompts of eight requests in one pass
        dict(name="adapters_4096", op="adapters", type="fp16", rows=4096, K=8192, N=8192, rank=32,
             adapters=8, without=0, order="runs"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (query heads, key heads, head size)
_HEADS = [(32, 32, 128), (64, 8, 128), (32, 8, 128), (8, 1, 128), (20, 4, 128), (40, 10, 128),
          (12, 12, 64), (32, 4, 64), (24, 1, 64), (14, 2, 64)]


def draw(rng):
    op = rng.choice(["attention", "attention", "heads", "adapters"])
    kind = rng.choice(["fp16", "bf16"])
    if op == "attention":
        while True:
            heads, kv, dim = rng.choice(_HEADS)
            seqs, longest = _log(rng, 1, 64), _log(rng, 33, 65536)
            new = 1 if rng.random() < 0.5 else min(_log(rng, 2, 1024), longest)
            c = dict(op=op, type=kind, seqs=seqs, heads=heads, kv_heads=kv, dim=dim, new=new,
                     ones=rng.randrange(seqs) if new > 1 else 0, longest=longest,
                     spread=round(rng.uniform(0.0, 0.95), 2), page=rng.choice([16, 32, 64, 128]),
                     window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
            if seqs * heads * new * longest <= 1 << 29 and seqs * longest * kv * dim <= 1 << 28:
                return c
    if op == "heads":
        heads, kv, dim = rng.choice(_HEADS)
        return dict(op=op, type=kind, tokens=_log(rng, 1, 4096), heads=heads, kv_heads=kv, dim=dim,
                    rotary=rng.choice([dim, dim // 2]), pairs=rng.choice(["halves", "neighbours"]),
                    norm=rng.random() < 0.5, page=rng.choice([16, 64]))
    rows, adapters = _log(rng, 1, 2048), _log(rng, 1, 64)
    return dict(op=op, type=kind, rows=rows, K=8 * _log(rng, 64, 1376), N=4 * _log(rng, 100, 2752) + 1,
                rank=rng.choice([8, 16, 32, 64]), adapters=adapters, without=rng.randrange(1 + rows // 4),
                order=rng.choice(["runs", "mixed"]))


# ------------------------------------------------- lengths, from the case alone

def _fraction(i):
    """The i-th of a sequence of fractions that fill [0, 1) evenly."""
    return (0.6180339887498949 * i) % 1.0


def _lengths(c):
    """(new tokens, keys in all) of each sequence."""
    got = []
    for i in range(c["seqs"]):
        f = 1.0 - c["spread"] * _fraction(i)
        new = 1 if i < c["ones"] else max(1, int(c["new"] * (1.0 - 0.5 * _fraction(3 * i))))
        got.append((new, max(new, int(c["longest"] * f))))
    return got


def _visible(c):
    """(pairs of a row and a key that it sees, keys that any row sees), over all sequences."""
    pairs = keys = 0
    for new, n in _lengths(c):
        first, w = n - new, c["window"] or n
        full = max(0, min(new, w - 1 - first))  # rows that see every key before them
        pairs += full * (first + 1) + full * (full - 1) // 2 + (new - full) * min(w, n)
        keys += min(n, new + w - 1)
    return pairs, keys


def work(case):
    c = case
    if c["op"] == "attention":
        pairs, keys = _visible(c)
        rows = sum(new for new, _ in _lengths(c))
        return {"bytes": 4 * keys * c["kv_heads"] * c["dim"] + 4 * rows * c["heads"] * c["dim"],
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "heads":
        wide = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
        turned = (c["heads"] + c["kv_heads"]) * (3 * c["rotary"] + (4 * c["dim"] if c["norm"] else 0))
        return {"bytes": c["tokens"] * (4 * wide + 4 * c["rotary"] + 16),
                "flops": c["tokens"] * max(1, turned)}
    with_one = c["rows"] - c["without"]
    used = min(c["adapters"], with_one)
    return {"bytes": 2 * (with_one * c["K"] + 2 * c["rows"] * c["N"] + used * c["rank"] * (c["K"] + c["N"])),
            "flops": 2 * with_one * c["rank"] * (c["K"] + c["N"])}


# ------------------------------------------------------------------ the inputs

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"attention": _prepare_attention, "heads": _prepare_heads,
            "adapters": _prepare_adapters}[case["op"]](case, gen)


def _prepare_attention(c, gen):
    dtype, page = TYPES[c["type"]], c["page"]
    lengths = _lengths(c)
    width = max(-(-n // page) for _, n in lengths)
    need = [-(-n // page) for _, n in lengths]
    pages = sum(need) + 3
    # every sequence's pages lie anywhere in the cache, as after long use
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    table, at = torch.zeros((c["seqs"], width), dtype=torch.int32), 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    starts = [0]
    for new, _ in lengths:
        starts.append(starts[-1] + new)
    shape = (pages, page, c["kv_heads"], c["dim"])
    return dict(c=c, q=_normal(gen, (starts[-1], c["heads"], c["dim"]), dtype),
                k_pages=_normal(gen, shape, dtype), v_pages=_normal(gen, shape, dtype),
                page_table=table.to(DEV),
                kv_lens=torch.tensor([n for _, n in lengths], dtype=torch.int32, device=DEV),
                q_starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                max_q=max(new for new, _ in lengths), max_kv=max(n for _, n in lengths),
                scale=c["dim"] ** -0.5)


def _prepare_heads(c, gen):
    dtype, tokens, page = TYPES[c["type"]], c["tokens"], c["page"]
    wide = (c["heads"] + 2 * c["kv_heads"]) * c["dim"]
    limit = 16384
    angle = (torch.arange(limit, device=DEV, dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(0, c["rotary"], 2, device=DEV, dtype=torch.float64) / c["rotary"]))
    # a chunk's tokens follow each other; decode tokens stand anywhere
    if tokens <= 64:
        positions = torch.randint(limit, (tokens,), generator=gen, device=DEV)
    else:
        positions = torch.arange(tokens, device=DEV) + int(
            torch.randint(limit - tokens, (1,), generator=gen, device=DEV))
    pages = -(-tokens // page) + 2
    shape = (pages, page, c["kv_heads"], c["dim"])
    slots = torch.randperm(pages * page, generator=gen, device=DEV)[:tokens]
    if tokens > 64:  # whole pages in any order, filled one after the other
        order = torch.randperm(pages, generator=gen, device=DEV)
        slots = (order[:, None] * page + torch.arange(page, device=DEV)).reshape(-1)[:tokens].contiguous()
    weight = [(1.0 + _normal(gen, (c["dim"],), torch.float32, 0.2)).to(dtype) if c["norm"] else None
              for _ in range(2)]
    return dict(c=c, qkv=_normal(gen, (tokens, wide), dtype), positions=positions,
                table=torch.cat([angle.cos(), angle.sin()], 1).float(), slots=slots,
                q_weight=weight[0], k_weight=weight[1], eps=1e-6,
                k_pages=_normal(gen, shape, dtype), v_pages=_normal(gen, shape, dtype))


def _prepare_adapters(c, gen):
    dtype, rows = TYPES[c["type"]], c["rows"]
    with_one = rows - c["without"]
    ids = torch.arange(with_one, device=DEV) * c["adapters"] // max(1, with_one)
    ids = torch.cat([ids, torch.full((c["without"],), -1, device=DEV)]).to(torch.int32)
    if c["order"] == "mixed":
        spread = torch.arange(with_one, device=DEV) % c["adapters"]
        ids[:with_one] = spread.to(torch.int32)
        ids = ids[torch.randperm(rows, generator=gen, device=DEV)].contiguous()
    return dict(c=c, x=_normal(gen, (rows, c["K"]), dtype), y=_normal(gen, (rows, c["N"]), dtype),
                a=_normal(gen, (c["adapters"], c["rank"], c["K"]), dtype, c["K"] ** -0.5),
                b=_normal(gen, (c["adapters"], c["N"], c["rank"]), dtype, c["rank"] ** -0.5),
                scales=0.5 + torch.rand((c["adapters"],), generator=gen, device=DEV), ids=ids)


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        import lut_gemv_amd as lg
        if op == "attention":
            return lg.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["kv_lens"],
                                      s["q_starts"], max_q=s["max_q"], max_kv=s["max_kv"],
                                      scale=s["scale"], window=s["c"]["window"])
        if op == "heads":
            q = lg.qk_norm_rotate(s["qkv"], s["c"]["heads"], s["c"]["kv_heads"], s["positions"], s["table"],
                                  q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"],
                                  interleaved=s["c"]["pairs"] == "neighbours",
                                  k_pages=s["k_pages"], v_pages=s["v_pages"], slots=s["slots"])
            return q, s["k_pages"], s["v_pages"]
        return lg.adapters_add(s["y"], s["x"], s["a"], s["b"], s["ids"], s["scales"])
    return {"attention": _attention, "heads": _heads, "adapters": _adapters}[op](s)


def _attention(s):
    q, table, lens, starts = s["q"], s["page_table"].long(), s["kv_lens"].long(), s["q_starts"].long()
    tokens, heads, dim = q.shape
    pages, page, kv, _ = s["k_pages"].shape
    seqs, keys, most, group = table.shape[0], table.shape[1] * page, s["max_q"], heads // kv
    # keys and values of each sequence side by side, [seq][head][key][dim]
    k = s["k_pages"][table].reshape(seqs, keys, kv, dim).transpose(1, 2).float()
    v = s["v_pages"][table].reshape(seqs, keys, kv, dim).transpose(1, 2).float()
    key = torch.arange(keys, device=q.device)
    v = torch.where((key < lens[:, None])[:, None, :, None], v, 0.0)
    row = torch.arange(most, device=q.device)
    at = (starts[:-1, None] + row).clamp(max=tokens - 1)
    qs = q[at].float().reshape(seqs, most, kv, group, dim).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(qs.reshape(seqs, kv, group * most, dim), k.transpose(2, 3)) * s["scale"]
    last = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + row  # the last key that a row sees
    seen = (key <= last[..., None]) & (key < lens[:, None, None])
    if s["c"]["window"]:
        seen &= key > last[..., None] - s["c"]["window"]
    scores = scores.reshape(seqs, kv, group, most, keys)
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top.masked_fill_(top == -math.inf, 0.0)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(seqs, kv, group * most, keys), v).reshape(seqs, kv, group, most, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(seqs, most, heads, dim)
    token = torch.arange(tokens, device=q.device)
    seq = torch.bucketize(token, starts[1:], right=True)
    return o[seq, token - starts[seq]].to(q.dtype)


def _turned(x, cos, sin, rotary, pairs):
    """x [token][head][dim] with its first `rotary` entries turned by their pairs' angles."""
    turn = x[..., :rotary]
    a, b = (turn[..., 0::2], turn[..., 1::2]) if pairs == "neighbours" else turn.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    turn = torch.stack([a, b], -1).flatten(-2) if pairs == "neighbours" else torch.cat([a, b], -1)
    return torch.cat([turn, x[..., rotary:]], -1)


def _heads(s):
    c, qkv = s["c"], s["qkv"]
    heads, kv, dim, rotary = c["heads"], c["kv_heads"], c["dim"], c["rotary"]
    q, k, v = qkv.view(-1, heads + 2 * kv, dim).split([heads, kv, kv], 1)
    cos, sin = s["table"][s["positions"]][:, None].chunk(2, -1)
    q, k = q.float(), k.float()
    if s["q_weight"] is not None:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + s["eps"]) * s["q_weight"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + s["eps"]) * s["k_weight"].float()
    q = _turned(q, cos, sin, rotary, c["pairs"]).to(qkv.dtype)
    k = _turned(k, cos, sin, rotary, c["pairs"]).to(qkv.dtype)
    s["k_pages"].view(-1, kv, dim)[s["slots"]] = k
    s["v_pages"].view(-1, kv, dim)[s["slots"]] = v
    return q, s["k_pages"], s["v_pages"]


def _adapters(s):
    x, y, a, b, ids = s["x"], s["y"], s["a"], s["b"], s["ids"]
    count, rank, _ = a.shape
    # every row through every adapter's first matrix, the others' results dropped
    t = torch.matmul(x.float(), a.float().reshape(count * rank, -1).t()).reshape(-1, count, rank)
    mine = ids[:, None] == torch.arange(count, device=x.device)
    t = torch.where(mine[..., None], t * s["scales"][:, None], 0.0).reshape(-1, count * rank)
    out = y.float() + torch.matmul(t, b.float().transpose(1, 2).reshape(count * rank, -1))
    return out.to(y.dtype)


# ------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "heads": _exact_heads,
            "adapters": _exact_adapters}[case["op"]](s)


def _exact_attention(s):
    c, q = s["c"], s["q"].double()
    group, page = c["heads"] // c["kv_heads"], c["page"]
    out, begin = torch.zeros_like(q), 0
    for i, (new, n) in enumerate(_lengths(c)):
        own_pages = s["page_table"][i, :-(-n // page)].long()
        k = s["k_pages"][own_pages].flatten(0, 1)[:n]
        v = s["v_pages"][own_pages].flatten(0, 1)[:n]
        last = torch.arange(n - new, n, device=q.device)[:, None]
        key = torch.arange(n, device=q.device)[None]
        hidden = key > last
        if c["window"]:
            hidden |= key <= last - c["window"]
        for h in range(c["kv_heads"]):
            mine = slice(h * group, (h + 1) * group)
            qh = q[begin:begin + new, mine].transpose(0, 1)
            kh, vh = k[:, h].double(), v[:, h].double()
            weight = torch.matmul(qh.reshape(-1, c["dim"]), kh.t()).view(group, new, n) * s["scale"]
            weight = torch.softmax(weight.masked_fill(hidden, -math.inf), -1)
            oh = torch.matmul(weight.view(-1, n), vh).view(group, new, -1)
            out[begin:begin + new, mine] = oh.transpose(0, 1)
        begin += new
    return out


def _exact_heads(s):
    c = s["c"]
    heads, kv, dim, half = c["heads"], c["kv_heads"], c["dim"], c["rotary"] // 2
    x = s["qkv"].double().view(c["tokens"], heads + 2 * kv, dim)
    angles = s["table"].double()[s["positions"]]
    first = torch.arange(half, device=x.device) * (2 if c["pairs"] == "neighbours" else 1)
    second = first + (1 if c["pairs"] == "neighbours" else half)
    done = []
    for part, weight in ((x[:, :heads], s["q_weight"]), (x[:, heads:heads + kv], s["k_weight"])):
        if weight is not None:
            part = part / (part.pow(2).mean(2, keepdim=True) + s["eps"]).sqrt() * weight.double()
        turn = torch.complex(part[..., first], part[..., second])
        turn = turn * torch.complex(angles[:, None, :half], angles[:, None, half:])
        part = part.clone()
        part[..., first], part[..., second] = turn.real, turn.imag
        done.append(part)
    pages = [s["k_pages"].double(), s["v_pages"].double()]
    for cache, new in zip(pages, (done[1], x[:, heads + kv:])):
        cache.view(-1, kv, dim).index_copy_(0, s["slots"], new)
    return done[0], pages[0], pages[1]


def _exact_adapters(s):
    x, out = s["x"].double(), s["y"].double()
    for i in range(s["c"]["adapters"]):
        rows = (s["ids"] == i).nonzero()[:, 0]
        inner = torch.mm(x[rows], s["a"][i].double().t())
        out[rows] += torch.mm(inner, s["b"][i].double().t()) * s["scales"][i].double()
    return out
