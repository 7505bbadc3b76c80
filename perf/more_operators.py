"""The cases on which the operators around a serving step's layers are measured.

Three operators, each in its plain form (elementary torch operations) and, where
``own`` is true, through the library's entry points:

* ``tables``: a step's page tables, slots, positions and row ranges from the
  requests' lengths, pages taken from and given back to a ring of free ones;
* ``shared``: attention of a batch whose sequences share long prefixes;
* ``sample``: next tokens drawn from logits with temperature, top-k, top-p and
  min-p, by one given random number a row.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one request's next token: all latency
        dict(name="tables_1", op="tables", seqs=1, new=1, chunks=0, longest=512, page=16, done=0,
             back=0, room=0),
        # a decode step of 400 requests, some finished, some with rejected drafts taken back
        dict(name="tables_400", op="tables", seqs=400, new=1, chunks=0, longest=8000, page=16, done=9,
             back=31, room=23),
        # prompts of odd lengths admitted beside running requests
        dict(name="tables_prompts", op="tables", seqs=160, new=4099, chunks=64, longest=16384, page=64,
             done=5, back=0, room=0),
        # two requests on one short system prompt: all latency
        dict(name="shared_2x512", op="shared", type="fp16", seqs=2, groups=1, heads=32, kv_heads=32,
             dim=128, prefix=512, spread=0.0, new=1, longest=61, page=16),
        # a decode step of 64 requests on one long document, 8 query heads to a key head
        dict(name="shared_64x32768", op="shared", type="bf16", seqs=64, groups=1, heads=64, kv_heads=8,
             dim=128, prefix=32768, spread=0.0, new=1, longest=900, page=64),
        # five system prompts of odd lengths, one key head to a query head, small heads
        dict(name="shared_40_in_5", op="shared", type="fp16", seqs=40, groups=5, heads=32, kv_heads=32,
             dim=64, prefix=4099, spread=0.7, new=1, longest=2000, page=16),
        # drafts and prompt chunks behind one long prefix: the matrix products bound it
        dict(name="shared_chunks", op="shared", type="bf16", seqs=8, groups=1, heads=32, kv_heads=8,
             dim=128, prefix=16384, spread=0.0, new=253, longest=700, page=64),
        # one request, nucleus sampling: all latency
        dict(name="sample_1", op="sample", type="fp16", rows=1, vocab=50272, how="top_p", masked=0),
        # a batch in which every request has settings of its own, some greedy
        dict(name="sample_48", op="sample", type="fp16", rows=48, vocab=32000, how="mixed", masked=100),
        # logits in 32 bits, temperature alone
        dict(name="sample_61", op="sample", type="fp32", rows=61, vocab=128001, how="plain", masked=0),
        # a full machine's batch on a large vocabulary of an odd size
        dict(name="sample_256", op="sample", type="bf16", rows=256, vocab=131073, how="top_p", masked=1000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


# (query heads, key heads, head size)
_HEADS = [(32, 32, 128), (64, 8, 128), (32, 8, 128), (8, 1, 128), (20, 4, 128), (40, 10, 128),
          (12, 12, 64), (32, 4, 64), (24, 1, 64), (14, 2, 64)]


def draw(rng):
    op = rng.choice(["tables", "shared", "shared", "sample", "sample"])
    if op == "tables":
        seqs = _log(rng, 1, 2048)
        chunks = rng.choice([0, rng.randrange(1 + min(seqs, 64))])
        rest = seqs - chunks
        return dict(op=op, seqs=seqs, new=_log(rng, 2, 4099), chunks=chunks, longest=_log(rng, 64, 16384),
                    page=rng.choice([16, 32, 64, 128]), done=rng.randrange(1 + rest // 8),
                    back=rng.randrange(1 + rest // 8), room=rng.choice([0, rng.randrange(1, 200)]))
    if op == "shared":
        while True:
            heads, kv, dim = rng.choice(_HEADS)
            seqs, prefix = _log(rng, 1, 96), _log(rng, 17, 32768)
            new = 1 if rng.random() < 0.7 else _log(rng, 2, 300)
            c = dict(op=op, type=rng.choice(["fp16", "bf16"]), seqs=seqs,
                     groups=rng.choice([1, 1, rng.randrange(1, 1 + min(seqs, 12))]), heads=heads,
                     kv_heads=kv, dim=dim, prefix=prefix, spread=round(rng.uniform(0.0, 0.9), 2),
                     new=new, longest=_log(rng, max(new, 8), max(new, 8) + 4000),
                     page=rng.choice([16, 32, 64, 128]))
            if (seqs * heads * new * dim * (prefix + c["longest"]) <= 1 << 34
                    and (c["groups"] * prefix + seqs * c["longest"]) * kv * dim <= 1 << 26):
                return c
    rows, vocab = _log(rng, 1, 256), _log(rng, 1000, 131073)
    return dict(op=op, type=rng.choice(["fp16", "bf16", "fp32"]), rows=rows, vocab=vocab,
                how=rng.choice(["plain", "top_p", "top_k", "min_p", "mixed"]),
                masked=rng.choice([0, rng.randrange(vocab // 2)]))


# ------------------------------------------------- lengths, from the case alone

def _fraction(i):
    """The i-th of a sequence of fractions that fill [0, 1) evenly."""
    return (0.6180339887498949 * i) % 1.0


def _changes(c):
    """(keys in the cache, new tokens or minus the keys taken back) of each request: chunks of
    prompts first, then finished requests, taken-back drafts and single tokens."""
    got = []
    for i in range(c["seqs"]):
        n = max(1, int(c["longest"] * (1.0 - 0.9 * _fraction(i))))
        j = i - c["chunks"]
        if j < 0:
            got.append((n if i % 3 == 0 else 0, max(1, int(c["new"] * (1.0 - 0.5 * _fraction(3 * i))))))
        elif j < c["done"]:
            got.append((n, -n))
        elif j < c["done"] + c["back"]:
            got.append((n, -min(n, 1 + j % 5)))
        else:
            got.append((n, 1))
    # requests of all kinds stand in any order
    return [got[(i * 7919) % c["seqs"]] for i in range(c["seqs"])] if c["seqs"] % 7919 else got


def _own(c):
    """(new tokens, keys behind the prefix) of each sequence."""
    got = []
    for i in range(c["seqs"]):
        new = max(1, int(c["new"] * (1.0 - 0.5 * _fraction(3 * i))))
        got.append((new, max(new, int(c["longest"] * (1.0 - 0.9 * _fraction(i))))))
    return got


def _groups(c):
    """(first sequence, end, keys of the prefix) of each group."""
    g, s = c["groups"], c["seqs"]
    return [(i * s // g, (i + 1) * s // g, max(1, int(c["prefix"] * (1.0 - c["spread"] * _fraction(i)))))
            for i in range(g)]


def work(case):
    c = case
    if c["op"] == "tables":
        rows = sum(max(0, d) for _, d in _changes(c)) + c["room"]
        moved = sum(abs(-(-(n + d) // c["page"]) + (-n // c["page"])) for n, d in _changes(c))
        return {"bytes": 16 * rows + 8 * moved + 16 * c["seqs"], "flops": rows}
    if c["op"] == "shared":
        own = _own(c)
        rows = sum(new for new, _ in own)
        pairs = sum(new * (n - new) + new * (new + 1) // 2 for new, n in own)
        keys = sum(n for _, n in own)
        for first, end, n in _groups(c):
            if end > first:
                keys += n
                pairs += n * sum(new for new, _ in own[first:end])
        return {"bytes": 4 * keys * c["kv_heads"] * c["dim"] + 4 * rows * c["heads"] * c["dim"],
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    size = 4 if c["type"] == "fp32" else 2
    return {"bytes": c["rows"] * (size * c["vocab"] + 32), "flops": 4 * c["rows"] * c["vocab"]}


# ------------------------------------------------------------------ the inputs

def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _int(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return {"tables": _prepare_tables, "shared": _prepare_shared,
            "sample": _prepare_sample}[case["op"]](case, gen)


def _prepare_tables(c, gen):
    changes, page = _changes(c), c["page"]
    held = [-(-n // page) for n, _ in changes]
    width = max(-(-(n + max(d, 0)) // page) for n, d in changes) + 1
    need = sum(max(0, -(-(n + d) // page) - h) for (n, d), h in zip(changes, held))
    pages = sum(held) + need + need // 8 + 5
    # the requests' pages and the free ones lie anywhere, as after long use
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    table = torch.full((c["seqs"], width), -1, dtype=torch.int32)
    at = 0
    for i, k in enumerate(held):
        table[i, :k] = order[at:at + k]
        at += k
    # the ring of free pages begins anywhere
    first = int(torch.randint(pages, (1,), generator=gen, device=DEV))
    ring = torch.full((pages,), -1, dtype=torch.int32)
    ring[(first + torch.arange(pages - at)) % pages] = order[at:]
    return dict(c=c, new=_int([d for _, d in changes]), kv_lens=_int([n for n, _ in changes]),
                page_table=table.to(DEV), free_pages=ring.to(DEV), free_range=_int([first, pages - at]),
                tokens=sum(max(0, d) for _, d in changes) + c["room"], page=page)


def _prepare_shared(c, gen):
    dtype, page = TYPES[c["type"]], c["page"]
    own, groups = _own(c), _groups(c)
    need = [-(-n // page) for _, _, n in groups] + [-(-n // page) for _, n in own]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32).cpu()
    tables = [torch.zeros((len(groups), max(need[:len(groups)])), dtype=torch.int32),
              torch.zeros((len(own), max(need[len(groups):])), dtype=torch.int32)]
    at = 0
    for i, k in enumerate(need):
        t, j = (tables[0], i) if i < len(groups) else (tables[1], i - len(groups))
        t[j, :k] = order[at:at + k]
        at += k
    starts = [0]
    for new, _ in own:
        starts.append(starts[-1] + new)
    shape = (pages, page, c["kv_heads"], c["dim"])
    return dict(c=c, q=_normal(gen, (starts[-1], c["heads"], c["dim"]), dtype),
                k_pages=_normal(gen, shape, dtype), v_pages=_normal(gen, shape, dtype),
                prefix_table=tables[0].to(DEV), prefix_lens=_int([n for _, _, n in groups]),
                page_table=tables[1].to(DEV), kv_lens=_int([n for _, n in own]), q_starts=_int(starts),
                group_starts=_int([first for first, _, _ in groups] + [c["seqs"]]),
                max_q=max(new for new, _ in own), max_kv=max(n for _, n in own),
                max_prefix=max(n for _, _, n in groups), scale=c["dim"] ** -0.5)


def _prepare_sample(c, gen):
    rows, vocab, how = c["rows"], c["vocab"], c["how"]
    # a language model's logits: a broad bulk, and some tokens that the context suggests
    x = torch.randn((rows, vocab), generator=gen, device=DEV) * 2.2
    some = min(64, vocab)
    at = torch.randint(vocab, (rows, some), generator=gen, device=DEV)
    x.scatter_add_(1, at, 5.0 + 2.5 * torch.randn((rows, some), generator=gen, device=DEV))
    if c["masked"]:  # tokens that a grammar forbids
        gone = torch.randperm(vocab, generator=gen, device=DEV)[:c["masked"]]
        x[:, gone] = -math.inf

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand((rows,), generator=gen, device=DEV)

    one = torch.ones((rows,), device=DEV)
    temperature, k, p, m = uniform(0.6, 1.2), None, None, None
    if how in ("top_p", "mixed"):
        p = uniform(0.8, 0.99)
    if how in ("top_k", "mixed"):
        k = torch.randint(1, 200, (rows,), generator=gen, device=DEV, dtype=torch.int32)
    if how in ("min_p", "mixed"):
        m = uniform(0.01, 0.2)
    if how == "mixed":  # each row has some of the filters, every eighth none but the lowest temperature
        row = torch.arange(rows, device=DEV)
        temperature = torch.where(row % 8 == 5, 0.0 * one, temperature)
        p = torch.where(row % 2 == 0, p, one)
        k = torch.where(row % 3 == 0, k, 0)
        m = torch.where(row % 5 == 0, m, 0.0 * one)
    return dict(c=c, logits=x.to(TYPES[c["type"]]), u=uniform(0.0, 1.0).clamp_(max=1.0 - 2.0 ** -24),
                temperature=temperature, top_k=k, top_p=p, min_p=m)


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    op = s["c"]["op"]
    if own:
        import lut_gemv_amd as lg
        if op == "tables":
            got = lg.batch_tables(s["new"], s["kv_lens"], s["page_table"], s["page"], s["tokens"],
                                  s["free_pages"], s["free_range"])
            return (*got, s["page_table"], s["free_pages"])
        if op == "shared":
            return lg.shared_prefix_attention(
                s["q"], s["k_pages"], s["v_pages"], s["prefix_table"], s["prefix_lens"], s["page_table"],
                s["kv_lens"], s["q_starts"], s["group_starts"], max_q=s["max_q"], max_kv=s["max_kv"],
                max_prefix=s["max_prefix"], scale=s["scale"])
        return lg.sample_tokens(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"])
    return {"tables": _tables, "shared": _shared, "sample": _sample}[op](s)


def _tables(s):
    new, lens, table, page = s["new"].long(), s["kv_lens"].long(), s["page_table"], s["page"]
    ring, tokens = s["free_pages"], s["tokens"]
    capacity, width = ring.numel(), table.shape[1]
    first, count = s["free_range"].long().unbind()
    lens = lens.clamp(0, width * page)
    grow = new.clamp(min=0)
    grow = torch.where(lens + grow <= width * page, grow, 0)
    held = (lens + page - 1) // page
    need = (lens + grow + page - 1) // page - held
    ends, page_ends = grow.cumsum(0), need.cumsum(0)
    served = (ends <= tokens) & (page_ends <= count)
    grow, need = torch.where(served, grow, 0), torch.where(served, need, 0)
    after = torch.where(new < 0, (lens + new).clamp(min=0), lens + grow)
    back = torch.where(new < 0, held - (after + page - 1) // page, 0)
    # pages given back go behind the ring's last, pages taken come from its first
    column = torch.arange(width, device=new.device)
    gone = (column >= (held - back)[:, None]) & (column < held[:, None])
    nth = gone.reshape(-1).cumsum(0).reshape(gone.shape) - 1
    to = (first + count + nth) % capacity
    fresh = (column >= held[:, None]) & (column < (held + need)[:, None])
    mine = (first + (need.cumsum(0) - need)[:, None] + column - held[:, None]) % capacity
    taken = ring[torch.where(fresh, mine, 0)]
    keep = torch.where(gone, table, 0)
    old = torch.cat([ring, ring.new_zeros(1)])
    old[torch.where(gone, to, capacity)] = keep
    ring.copy_(old[:capacity])
    table.copy_(torch.where(fresh, taken, table))
    starts = torch.cat([grow.new_zeros(1), grow.cumsum(0)])
    row = torch.arange(tokens, device=new.device)
    seq = torch.bucketize(row, starts[1:], right=True)
    inside = seq < new.numel()
    seq = seq.clamp(max=new.numel() - 1)
    position = lens[seq] + row - starts[seq]
    slot = table[seq, (position // page).clamp(max=width - 1)].long() * page + position % page
    free = torch.stack([(first + need.sum()) % capacity, count - need.sum() + back.sum()])
    return (torch.where(inside, position, 0), torch.where(inside, slot, -1), after.int(), starts.int(),
            free.int(), table, ring)


def _weigh(q, k, v, seen, scale):
    """(weighted values, weights' sum, maximum) of q [head][row][dim], k and v [head][key][dim]."""
    x = torch.matmul(q, k.transpose(1, 2)) * scale
    if seen is not None:
        x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    return torch.matmul(x, v), x.sum(-1, keepdim=True), top


def _gather(pages, table, n):
    """The first n keys of a table's row, [head][key][dim] in 32 bits."""
    page = pages.shape[1]
    got = pages[table[:-(-n // page)].long()]
    return got.flatten(0, 1)[:n].transpose(0, 1).float()


def _shared(s):
    c, q = s["c"], s["q"]
    tokens, heads, dim = q.shape
    kv, group = c["kv_heads"], c["heads"] // c["kv_heads"]
    own = _own(c)
    starts = [0]
    for new, _ in own:
        starts.append(starts[-1] + new)
    # rows [key head][token, query head of the group][dim]
    rows = q.float().view(tokens, kv, group, dim).transpose(0, 1).reshape(kv, tokens * group, dim)
    out = torch.empty_like(rows)
    for g, (first, end, n) in enumerate(_groups(c)):
        if end == first:
            continue
        mine = slice(starts[first] * group, starts[end] * group)
        k, v = (_gather(s[x], s["prefix_table"][g], n) for x in ("k_pages", "v_pages"))
        o, total, top = _weigh(rows[:, mine], k, v, None, s["scale"])
        for i in range(first, end):
            new, n = own[i]
            part = slice((starts[i] - starts[first]) * group, (starts[i + 1] - starts[first]) * group)
            k, v = (_gather(s[x], s["page_table"][i], n) for x in ("k_pages", "v_pages"))
            last = n - new + torch.arange(new * group, device=q.device) // group
            seen = torch.arange(n, device=q.device) <= last[:, None]
            o2, total2, top2 = _weigh(rows[:, starts[i] * group:starts[i + 1] * group], k, v, seen,
                                      s["scale"])
            most = torch.maximum(top[:, part], top2)
            f, f2 = torch.exp(top[:, part] - most), torch.exp(top2 - most)
            out[:, starts[i] * group:starts[i + 1] * group] = (
                (o[:, part] * f + o2 * f2) / (total[:, part] * f + total2 * f2))
    return out.view(kv, tokens, group, dim).transpose(0, 1).reshape(tokens, heads, dim).to(q.dtype)


def _sample(s):
    # in 64 bits: the sums' order must not move a token's border past the random number
    x, rows = s["logits"].double(), s["logits"].shape[0]
    vocab = x.shape[1]
    t = s["temperature"].double()[:, None]
    greedy = t == 0.0
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    weight = torch.exp((x - x[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(vocab, device=x.device)
    keep = (rank == 0) | ~greedy
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep = keep & ((rank < k) | (k <= 0))
    weight = torch.where(keep, weight, 0.0)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        upto = weight.cumsum(1)
        before = torch.cat([torch.zeros_like(upto[:, :1]), upto[:, :-1]], 1)
        weight = torch.where((before < p * upto[:, -1:]) | (p >= 1.0) | (rank == 0), weight, 0.0)
    if s["min_p"] is not None:
        weight = torch.where(weight >= s["min_p"].double()[:, None], weight, 0.0)
    weight = torch.zeros_like(weight).scatter_(1, order, weight)
    upto = weight.cumsum(1)
    token = (upto <= s["u"].double()[:, None] * upto[:, -1:]).sum(1).clamp(max=vocab - 1)
    logprob = torch.log(weight.gather(1, token[:, None])[:, 0] / upto[:, -1])
    return token, logprob.float()


# ------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "shared": _exact_shared,
            "sample": _exact_sample}[case["op"]](s)


def _exact_tables(s):
    page, tokens = s["page"], s["tokens"]
    table, ring = s["page_table"].cpu(), s["free_pages"].cpu()
    first, count = s["free_range"].tolist()
    capacity, (seqs, width) = ring.numel(), table.shape
    row, taken, given = 0, 0, []
    positions, slots = [], []
    after, starts = [], [0]
    for i, (d, n) in enumerate(zip(s["new"].tolist(), s["kv_lens"].tolist())):
        pages = -(-n // page)
        if d < 0:
            n = max(0, n + d)
            given += table[i, -(-n // page):pages].tolist()
        else:
            more = -(-(n + d) // page) - pages
            assert n + d <= width * page and row + d <= tokens and taken + more <= count
            for j in range(more):
                table[i, pages + j] = ring[(first + taken + j) % capacity]
            taken += more
            at = torch.arange(n, n + d)
            positions.append(at)
            slots.append(table[i, at // page].long() * page + at % page)
            n += d
            row += d
        after.append(n)
        starts.append(row)
    for j, x in enumerate(given):
        ring[(first + count + j) % capacity] = x
    rest = torch.zeros(tokens - row, dtype=torch.int64)
    free = [(first + taken) % capacity, count - taken + len(given)]
    return (torch.cat(positions + [rest]).to(DEV), torch.cat(slots + [rest - 1]).to(DEV), _int(after),
            _int(starts), _int(free), table.to(DEV), ring.to(DEV))


def _exact_shared(s):
    c, q = s["c"], s["q"].double()
    group, page, begin = c["heads"] // c["kv_heads"], c["page"], 0
    out = torch.zeros_like(q)
    own, groups = _own(c), _groups(c)
    for i, (new, n) in enumerate(own):
        g = next(j for j, (first, end, _) in enumerate(groups) if first <= i < end)
        shared = groups[g][2]
        ids = [s["prefix_table"][g, :-(-shared // page)].long(), s["page_table"][i, :-(-n // page)].long()]
        key = torch.arange(shared + n, device=q.device)
        hidden = key > torch.arange(shared + n - new, shared + n, device=q.device)[:, None]
        for h in range(c["kv_heads"]):
            k, v = (torch.cat([cache[ids[0], :, h].flatten(0, 1)[:shared],
                               cache[ids[1], :, h].flatten(0, 1)[:n]]).double()
                    for cache in (s["k_pages"], s["v_pages"]))
            mine = slice(h * group, (h + 1) * group)
            qh = q[begin:begin + new, mine].transpose(0, 1).reshape(-1, c["dim"])
            x = torch.mm(qh, k.t()).view(group, new, -1) * s["scale"]
            x = torch.softmax(x.masked_fill(hidden, -math.inf), -1)
            out[begin:begin + new, mine] = torch.mm(x.view(group * new, -1), v).view(group, new, -1).transpose(0, 1)
        begin += new
    return out


def _exact_sample(s):
    import numpy as np
    x = s["logits"].double().cpu().numpy()
    settings = [None if s[k] is None else s[k].double().cpu().numpy()
                for k in ("u", "temperature", "top_k", "top_p", "min_p")]
    tokens, logprobs = [], []
    for r in range(x.shape[0]):
        u, t, k, p, m = (None if a is None else a[r] for a in settings)
        if t == 0.0:
            tokens.append(int(np.argmax(x[r])))
            logprobs.append(0.0)
            continue
        order = np.argsort(-x[r], kind="stable")
        w = np.exp((x[r][order] - x[r][order[0]]) / t)
        if k is not None and k > 0:
            w[int(k):] = 0.0
        if p is not None and p < 1.0:
            end = np.searchsorted(np.cumsum(w), p * np.sum(w), side="left")
            w[max(1, end + 1):] = 0.0
        if m is not None:
            w[w < m] = 0.0
        back = np.zeros_like(w)
        back[order] = w
        upto = np.cumsum(back)
        i = int(np.searchsorted(upto, u * upto[-1], side="right"))
        tokens.append(i)
        logprobs.append(float(np.log(back[i]) - np.log(upto[-1])))
    return _int(tokens, torch.int64), _int(logprobs, torch.float64)
