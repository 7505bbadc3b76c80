"""The operators around a serving step on the GPU, against their plain forms
(oracle/serving.py): attention over shared prefixes with the bounds counted there, batch tables in
whole numbers, sampling against 64 bits; then a run of them together."""
import sys

import numpy as np
import pytest

from oracle import serving as plain

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import lut_gemv_amd as lg  # noqa: E402

DEV = "cuda:0"
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
NAN, INF = float("nan"), float("inf")


def _say(msg):
    print(f"[steps] {msg}", flush=True)
    sys.stdout.flush()


def _np(t):
    return t.detach().cpu().double().numpy()


def _int(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


# ---------------------------------------------------- attention over shared prefixes

class Shared:
    """Sequences behind shared prefixes in a paged cache whose unused slots and pages hold NaN."""

    def __init__(self, dtype, heads, kv_heads, dim, page, prefixes, starts, lens, news, seed=0, scale=1.0,
                 lead=0, tail=0):
        self.dtype, self.page, self.heads, self.kv_heads, self.dim = dtype, page, heads, kv_heads, dim
        self.prefixes, self.starts, self.lens, self.news, self.lead = prefixes, starts, lens, news, lead
        all_lens = list(prefixes) + list(lens)
        need = [-(-n // page) for n in all_lens]
        pages = sum(need) + 2
        ids = np.random.default_rng(seed).permutation(pages)
        k, v = (torch.full((pages, page, kv_heads, dim), NAN, dtype=dtype) for _ in range(2))
        tables = [torch.full((n, max(c + [1]) + 1), -7, dtype=torch.int32)
                  for n, c in ((len(prefixes), need[:len(prefixes)]), (len(lens), need[len(prefixes):]))]
        g = torch.Generator().manual_seed(seed)
        self.kv, at = [], 0
        for i, n in enumerate(all_lens):
            kn = (torch.randn((n, kv_heads, dim), generator=g) * scale).to(dtype)
            vn = torch.randn((n, kv_heads, dim), generator=g).to(dtype)
            t, row = (tables[0], i) if i < len(prefixes) else (tables[1], i - len(prefixes))
            for j in range(need[i]):
                page_id = int(ids[at])
                at += 1
                t[row, j] = page_id
                part = slice(j * page, min(n, (j + 1) * page))
                k[page_id, :part.stop - part.start] = kn[part]
                v[page_id, :part.stop - part.start] = vn[part]
            self.kv.append((kn, vn))
        tokens = lead + sum(news) + tail
        self.q = (torch.randn((tokens, heads, dim), generator=g) * scale).to(dtype).to(DEV)
        self.k_pages, self.v_pages = k.to(DEV), v.to(DEV)
        self.prefix_table, self.page_table = tables[0].to(DEV), tables[1].to(DEV)
        self.prefix_lens, self.kv_lens = _int(list(prefixes)), _int(list(lens))
        self.q_starts = _int([lead + sum(news[:i]) for i in range(len(news) + 1)])
        self.group_starts = _int(list(starts))

    def run(self, **kw):
        a = dict(q_starts=self.q_starts, group_starts=self.group_starts)
        a.update(kw)
        return lg.shared_prefix_attention(self.q, self.k_pages, self.v_pages, self.prefix_table,
                                          self.prefix_lens, self.page_table, self.kv_lens, **a)

    def group(self, s):
        for g in range(len(self.prefixes)):
            if self.starts[g] <= s < self.starts[g + 1]:
                return g
        return -1

    def want(self, s):
        """Result and bound of sequence s (all of its own keys precede or are its new tokens')."""
        g, at = self.group(s), self.lead + sum(self.news[:s])
        k, v = (_np(t) for t in self.kv[len(self.prefixes) + s])
        n = self.lens[s]
        if g >= 0:
            pk, pv = (_np(t) for t in self.kv[g])
            k, v, n = np.concatenate([pk, k]), np.concatenate([pv, v]), n + self.prefixes[g]
        q = _np(self.q[at:at + self.news[s]])
        return plain.attention(q, k, v, self.news[s], n, self.dim ** -0.5, 0, U[self.dtype])

    def check(self, out, what):
        got, worst = _np(out), 0.0
        for s in range(len(self.lens)):
            want, bound = self.want(s)
            at = self.lead + sum(self.news[:s])
            mine = got[at:at + self.news[s]]
            assert np.isfinite(mine).all(), f"{what}: sequence {s} is not finite"
            if mine.size:
                worst = max(worst, float((np.abs(mine - want) / bound).max()))
        _say(f"{what}: worst err/bound {worst:.3f}")
        assert worst <= 1.0, what


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 8, 128), (16, 2, 128), (12, 4, 64), (14, 2, 64), (6, 1, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_shared_single_tokens(dtype, heads, kv_heads, dim):
    prefixes, starts = [65, 1, 0, 300, 64], [0, 3, 5, 6, 6, 9]
    b = Shared(dtype, heads, kv_heads, dim, 16, prefixes, starts, [1, 40, 16, 17, 200, 33, 1, 2, 130], [1] * 9)
    b.check(b.run(), f"{dtype} {heads}/{kv_heads}x{dim}")
    b.check(b.run(q_starts=None, max_q=1, max_kv=200, max_prefix=300), "hints")


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_shared_chunks_and_single_tokens(dtype, heads, kv_heads, dim, page):
    b = Shared(dtype, heads, kv_heads, dim, page, [130, 77], [1, 4, 6], [50, 5, 1, 200, 9, 131, 3],
               [7, 5, 1, 140, 1, 131, 1], seed=3)
    b.check(b.run(), f"{dtype} chunks, page {page}")
    b.check(b.run(max_q=140, max_kv=200, max_prefix=130), "with hints")
    b.check(b.run(max_q=1, max_kv=1, max_prefix=1), "hints far too small")
    b.check(b.run(max_q=0, max_kv=0, max_prefix=0), "hints of zero")


@pytest.mark.parametrize("seqs,heads,kv_heads", [(24, 8, 1), (5, 4, 4)])
def test_shared_long_prefix_in_parts(seqs, heads, kv_heads):
    b = Shared(BF16, heads, kv_heads, 128, 64, [4999], [0, seqs], [11 + 37 * i for i in range(seqs)], [1] * seqs,
               seed=5)
    b.check(b.run(), f"{seqs} sequences on 4999 keys")
    b.check(b.run(group_starts=None), "one group by default")


def test_shared_more_groups_and_sequences_than_lanes():
    n = 150
    starts = [0] + [2 * i + (i % 3 == 0) for i in range(1, 71)]
    b = Shared(F16, 4, 2, 64, 16, [1 + (5 * i) % 40 for i in range(70)], starts, [1 + (7 * i) % 50 for i in range(n)],
               [1 + (i % 7 == 0) * min(3, (7 * i) % 50) for i in range(n)], seed=7)
    b.check(b.run(), "70 groups of 150 sequences")
    b.check(b.run(max_q=4, max_kv=50, max_prefix=41), "with hints")


def test_shared_equals_attention_on_joined_tables():
    """Prefixes of whole pages: paged_attention on the tables put together says the same."""
    b = Shared(BF16, 16, 4, 128, 32, [96, 160], [0, 3, 7], [5, 40, 1, 77, 32, 64, 100], [1, 3, 1, 70, 1, 2, 1], seed=9)
    joined, lens = [], []
    for s in range(7):
        g = b.group(s)
        row = b.prefix_table[g, :b.prefixes[g] // 32].tolist() + b.page_table[s].tolist()
        joined.append(row)
        lens.append(b.lens[s] + b.prefixes[g])
    width = max(map(len, joined))
    table = _int([r + [-1] * (width - len(r)) for r in joined])
    other = lg.paged_attention(b.q, b.k_pages, b.v_pages, table, _int(lens), b.q_starts)
    out = b.run()
    b.check(out, "shared")
    b.check(other, "joined")


def test_shared_rows_left_alone_and_strides():
    b = Shared(F16, 8, 2, 128, 16, [40], [0, 4], [9, 20, 3, 64], [1, 20, 1, 1], seed=11, lead=3, tail=5)
    out = torch.full((b.q.shape[0], 8, 256), 7.0, dtype=F16, device=DEV)[:, :, 64:192]
    got = b.run(out=out)
    assert got.data_ptr() == out.data_ptr()
    b.check(got, "strided output")
    assert (got[:3] == 7).all() and (got[-5:] == 7).all()
    whole = torch.full((b.q.shape[0], 8, 256), 0.0, dtype=F16, device=DEV)
    whole[:, :, 64:192] = got
    # queries in rows of a fused buffer, pages with heads outside slots
    wide = torch.zeros((b.q.shape[0], 12, 128), dtype=F16, device=DEV)
    wide[:, 2:10] = b.q
    b.q = wide[:, 2:10]
    b.k_pages, b.v_pages = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (b.k_pages, b.v_pages))
    b.check(b.run(), "strided inputs")


def test_shared_output_over_the_queries():
    b = Shared(BF16, 8, 2, 64, 16, [70], [0, 5], [9, 20, 3, 64, 18], [1, 17, 1, 30, 1], seed=13)
    first = b.run().clone()
    got = b.run(out=b.q)
    assert got.data_ptr() == b.q.data_ptr() and torch.equal(got, first)


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [1, 30, 20, 1]])
def test_shared_bad_pages_and_lengths(news):
    lens = [40, 30, 33, 1]
    b = Shared(F16, 4, 2, 64, 16, [50, 33], [0, 2, 4], lens, news, seed=15)
    good = b.run()
    b.check(good, "good")
    starts = [0, *np.cumsum(news)]

    def rows(s):
        return slice(starts[s], starts[s + 1])

    table = b.prefix_table.clone()
    b.prefix_table[0, 1] = 1 << 30
    out = b.run()
    for s in range(4):
        assert out[rows(s)].isnan().all() if s < 2 else torch.equal(out[rows(s)], good[rows(s)])
    b.prefix_table = table.clone()
    b.prefix_table[1, 2] = -1
    out = b.run()
    assert not out[rows(0)].isnan().any() and out[rows(2)].isnan().all() and out[rows(3)].isnan().all()
    b.prefix_table = table
    b.prefix_lens = _int([1 << 20, 33])
    out = b.run()
    assert out[:starts[2]].isnan().all() and torch.equal(out[starts[2]:], good[starts[2]:])
    b.prefix_lens = _int([-5, 33])  # counts as 0
    out = b.run()
    assert out.isfinite().all() and torch.equal(out[starts[2]:], good[starts[2]:])
    b.prefix_lens = _int([50, 33])
    b.kv_lens = _int([40, 1 << 25, 33, 1])
    out = b.run()
    assert out[rows(1)].isnan().all() and torch.equal(out[rows(0)], good[rows(0)])
    b.kv_lens = _int(lens)
    b.page_table[2, 0] = 1 << 20
    out = b.run()
    assert out[rows(2)].isnan().all() and torch.equal(out[rows(3)], good[rows(3)])


def test_shared_rows_that_see_nothing():
    """No keys at all: zero. None of their own before the prefix's: the prefix alone."""
    b = Shared(F16, 4, 2, 64, 16, [0, 20], [0, 2, 4], [3, 0, 0, 2], [3, 1, 1, 2], seed=17)
    b.kv_lens = _int([2, 0, 0, 2])  # the first sequence holds fewer keys than it has new tokens
    out = b.run()
    assert (out[0] == 0).all() and (out[3] == 0).all() and out[1:3].abs().sum() > 0
    k, v = (_np(t) for t in b.kv[1])
    want, bound = plain.attention(_np(b.q[4:5]), k, v, 1, 20, 64 ** -0.5, 0, U[F16])
    assert (np.abs(_np(out[4:5]) - want) <= bound).all()


def test_shared_non_finite_values():
    """Among a prefix's values they reach its group's rows alone, among a sequence's own those that
    see them; keys without weight too."""
    b = Shared(BF16, 4, 2, 64, 16, [40, 20], [0, 2, 4], [10, 33, 20, 2], [1, 33, 1, 2], seed=19)
    good = b.run()
    page = int(b.prefix_table[0, 2])
    b.v_pages[page, 7, 1, 5] = INF           # key 39 of the first prefix, key head 1
    page = int(b.page_table[1, 1])
    b.v_pages[page, 4, 0, 9] = NAN           # key 20 of sequence 1, key head 0
    out = b.run()
    assert (out[:34, 2:, 5] == INF).all()
    seen = 1 + 20                            # rows of sequence 1 from position 20 on
    assert out[seen:34, :2, 9].isnan().all() and not out[:seen, :2, 9].isnan().any()
    mask = torch.ones_like(good, dtype=torch.bool)
    mask[:34, 2:, 5] = False
    mask[seen:34, :2, 9] = False
    assert torch.equal(out[mask], good[mask])


@pytest.mark.parametrize("news", [[1, 1], [40, 1]])
def test_shared_scores_of_minus_infinity(news):
    """Rows whose scores are all minus infinity have no softmax, also in parts; a part of such
    scores beside finite ones has no weight."""
    b = Shared(BF16, 2, 2, 64, 16, [600], [0, 2], [40, 3], news, seed=21)
    good = _np(b.run())
    b.q[0] = 3e38
    used = b.prefix_table[0, :38].long()
    b.k_pages[used] = -3e38
    out = b.run()
    b.kv_lens = _int([0, 3])
    alone = b.run(q_starts=_int([0, 1, 1 + news[1]]))
    assert alone[0].isnan().all()
    assert good.shape == out.shape


def test_shared_repeats_graphs_and_streams():
    b = Shared(BF16, 16, 2, 128, 32, [900], [0, 6], [20, 300, 7, 64, 65, 1], [1, 40, 1, 3, 1, 1], seed=23)
    hints = dict(max_q=40, max_kv=512, max_prefix=1024)
    first = b.run(**hints)
    b.check(first, "eager")
    for _ in range(3):
        assert torch.equal(b.run(**hints), first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.run(**hints)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = b.run(**hints)
    for i in range(4):
        b.prefix_lens.fill_(900 if i % 2 == 0 else 333)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b.run(**hints))
    with torch.cuda.stream(side):
        other = b.run(**hints)
    here = b.run(**hints)
    torch.cuda.synchronize()
    assert torch.equal(here, other)


def test_shared_group_starts_outside_and_sequences_without_rows():
    """Starts are brought into [0, seqs]; sequences and groups without new tokens take no rows."""
    b = Shared(F16, 8, 2, 64, 16, [33, 40, 17], [-3, 2, 4, 1 << 30], [9, 20, 33, 4, 50, 7], [1, 0, 0, 0, 30, 1], seed=27)
    b.starts = [0, 2, 4, 6]
    b.check(b.run(), "starts outside")
    b.check(b.run(max_q=1), "starts outside, all said to be single tokens")


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 1, 128), (2, 2, 64)])
def test_shared_uneven_groups(heads, kv_heads, dim):
    """Groups of a few rows beside one of many: the rows a group are an average."""
    news = [1] * 9 + [2] + [1] * 40
    starts = [0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 50]
    b = Shared(BF16, heads, kv_heads, dim, 16, [20 + 31 * i for i in range(10)], starts, [3 + (11 * i) % 70 for i in range(50)],
               news, seed=29)
    b.check(b.run(), f"{heads}/{kv_heads}x{dim}")


@pytest.mark.parametrize("news", [[1, 1, 1], [30, 1, 140]])
def test_shared_far_pages(news):
    """Pages more than 2^32 bytes, and 2^31 elements, into the cache, prefixes' and own."""
    pages = (1 << 31) // (64 * 2 * 128) + 40
    k, v = (torch.zeros((pages, 64, 2, 128), dtype=F16, device=DEV) for _ in range(2))
    assert k.numel() > 1 << 31
    b = Shared(F16, 8, 2, 128, 64, [200], [0, 3], [30, 65, 150], news, seed=31)
    for table in (b.prefix_table, b.page_table):
        for at in (table >= 0).nonzero().tolist():
            near = int(table[tuple(at)])
            table[tuple(at)] = pages - 1 - near
            k[pages - 1 - near], v[pages - 1 - near] = b.k_pages[near], b.v_pages[near]
    b.k_pages, b.v_pages = k, v
    b.check(b.run(), "far pages")


def test_shared_nothing_to_do():
    b = Shared(F16, 4, 2, 64, 16, [20], [0, 3], [3, 2, 5], [1, 1, 1], seed=25)
    b.q = b.q[:0]
    assert b.run(q_starts=_int([0, 0, 0, 0])).shape == (0, 4, 64)
    b = Shared(F16, 4, 2, 64, 16, [], [0], [3, 2, 5], [1, 1, 1], seed=25)
    b.check(b.run(), "no groups")


# ---------------------------------------------------------------- batch tables

def _tables_case(seqs, page, longest, seed, grow=9, ring=True):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, seqs)
    change = rng.integers(-3, grow + 1, seqs)
    change[rng.random(seqs) < 0.1] = -10 ** 9
    width = -(-(longest + grow) // page) + 1
    held = -(-lens // page)
    pages = int(held.sum()) + seqs * (grow // page + 2) + 7
    ids = rng.permutation(pages)
    table = np.full((seqs, width), -1, np.int32)
    at = 0
    for s in range(seqs):
        table[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    first = int(rng.integers(pages))
    free = np.full(pages, -1, np.int32)
    free[(first + np.arange(pages - at)) % pages] = ids[at:]
    return change, lens, table, free, [first, pages - at]


def _tables_check(change, lens, table, page, tokens, ring, free, offsets=None, **kw):
    wt, wr = table.tolist(), None if ring is None else ring.tolist()
    want = plain.tables(change.tolist(), lens.tolist(), wt, page, tokens, wr, free, offsets)
    dt = _int(table.tolist()) if table.size else torch.empty(table.shape, dtype=torch.int32, device=DEV)
    dr = None if ring is None else _int(ring.tolist())
    dc, dl = (_int(a.tolist()) for a in (change, lens))
    got = lg.batch_tables(dc, dl, dt, page, tokens, dr, None if ring is None else _int(free),
                          None if offsets is None else _int(offsets), **kw)
    for g, w, what in zip(got, want, ("positions", "slots", "kv_lens", "q_starts", "free_range")):
        assert (g is None and w is None) or g.tolist() == w, what
    assert dt.tolist() == wt, "page_table"
    assert ring is None or dr.tolist() == wr, "free_pages"
    return got


@pytest.mark.parametrize("seqs,page,longest", [(1, 16, 100), (7, 1, 9), (63, 16, 300), (64, 32, 31), (65, 48, 1000),
                                               (1023, 16, 100), (1024, 64, 70), (1025, 16, 40), (3001, 128, 500)])
def test_tables(seqs, page, longest):
    for seed in range(3):
        change, lens, table, ring, free = _tables_case(seqs, page, longest, 100 * seqs + seed)
        tokens = int(change.clip(0).sum()) + 5 * seed
        offsets = None if seed == 0 else np.random.default_rng(seed).integers(0, 9999, seqs).tolist()
        got = _tables_check(change, lens, table, page, tokens, ring, free, offsets)
        assert int(got[3][-1]) == change.clip(0).sum()


@pytest.mark.parametrize("seqs", [5, 300, 2500])
def test_tables_without_room(seqs):
    change, lens, table, ring, free = _tables_case(seqs, 16, 90, seqs)
    rows = int(change.clip(0).sum())
    for tokens in (0, 1, rows // 2, rows - 1):
        _tables_check(change, lens, table, 16, tokens, ring, free)
    for count in (0, 1, seqs // 3):
        _tables_check(change, lens, table, 16, rows, ring, [free[0], count])
    # table rows that are full
    _tables_check(change, lens, np.ascontiguousarray(table[:, :4]), 16, rows, ring, free)
    assert (lens + change.clip(0)).max() > 4 * 16


def test_tables_long_prompts():
    change = np.array([40000, 0, 1, 70001, -5])
    lens = np.array([0, 17, 15, 1000, 33])
    rng = np.random.default_rng(1)
    ids = rng.permutation(4000)
    table = np.full((5, 2300), -1, np.int32)
    at = 0
    for s, n in enumerate(lens):
        k = -(-int(n) // 32)
        table[s, :k] = ids[at:at + k]
        at += k
    ring = np.concatenate([ids[at:], np.full(at, -1)]).astype(np.int32)
    _tables_check(change, lens, table, 32, 110100, ring, [0, 4000 - at])


@pytest.mark.parametrize("tokens", [4096, 4097])
def test_tables_prompts_beside_single_tokens(tokens):
    """Rows of every kind of sequence in one launch and in two."""
    rng = np.random.default_rng(tokens)
    for seqs, big in ((1, 4000), (7, 500), (256, 40), (257, 30), (1500, 9)):
        change = np.where(rng.random(seqs) < 0.3, big, rng.integers(-2, 6, seqs))
        change[np.cumsum(change.clip(0)) > 4000] = -1
        change[0] = min(big, 90)
        lens = rng.integers(0, 200, seqs)
        held = -(-lens // 16)
        pages = int(held.sum()) + 4000
        ids = rng.permutation(pages)
        table = np.full((seqs, 280), -1, np.int32)
        at = 0
        for s in range(seqs):
            table[s, :held[s]] = ids[at:at + held[s]]
            at += held[s]
        ring = np.concatenate([ids[at:], np.full(at, -1)]).astype(np.int32)
        _tables_check(change, lens, table, 16, tokens, ring, [0, pages - at], rng.integers(0, 99, seqs).tolist())


def test_tables_without_a_ring():
    change, lens, table, _, _ = _tables_case(40, 16, 200, 3)
    table = np.random.default_rng(3).permutation(table.size).astype(np.int32).reshape(table.shape)
    got = _tables_check(change, lens, table, 16, int(change.clip(0).sum()) + 3, None, [0, 0])
    assert got[4] is None


def test_tables_lengths_and_ranges_outside():
    """They are brought inside; a ring that would overflow drops what is given back."""
    change = np.array([3, -2, 5, -(1 << 31), (1 << 31) - 1, 2])
    lens = np.array([-7, 1 << 30, 20, 31, 4, -(1 << 31)])
    table = np.arange(6 * 4, dtype=np.int32).reshape(6, 4)
    ring = np.arange(100, 130, dtype=np.int32)
    for free in ([-3, 20], [1 << 30, 29], [-(1 << 31), -1], [7, 1 << 30], [29, 30]):
        _tables_check(change, lens, table, 16, 20, ring, free)


def test_tables_no_sequences_no_rows():
    got = _tables_check(np.zeros(0, int), np.zeros(0, int), np.zeros((0, 4), np.int32), 16, 3, np.arange(5), [2, 3])
    assert got[3].tolist() == [0]
    _tables_check(np.array([-3]), np.array([20]), np.arange(4, dtype=np.int32)[None], 16, 0, np.arange(5), [2, 3])


def test_tables_strided_table():
    change, lens, table, ring, free = _tables_case(9, 16, 100, 5)
    wide = torch.full((9, table.shape[1] + 7), -5, dtype=torch.int32, device=DEV)
    wide[:, 2:-5] = _int(table.tolist())
    wt, wr = table.tolist(), ring.tolist()
    want = plain.tables(change.tolist(), lens.tolist(), wt, 16, 80, wr, free)
    got = lg.batch_tables(_int(change.tolist()), _int(lens.tolist()), wide[:, 2:-5], 16, 80, _int(ring.tolist()),
                          _int(free))
    assert all(g.tolist() == w for g, w in zip(got, want))
    assert wide[:, 2:-5].tolist() == wt and (wide[:, :2] == -5).all() and (wide[:, -5:] == -5).all()


def test_tables_in_place_and_replayed():
    """A captured step goes on from where it ended: 40 steps of 6 sequences, some of which end."""
    page, seqs = 4, 6
    table, ring, free = np.full((seqs, 12), -1, np.int32), np.arange(30)[::-1].copy(), [11, 30]
    lens = np.zeros(seqs, int)
    dt, dr, df, dl = _int(table.tolist()), _int(ring.tolist()), _int(free), _int(lens.tolist())
    dc = _int([1] * seqs)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = lg.batch_tables(dc, dl, dt, page, seqs, dr, df, in_place=True)
    assert got[2].data_ptr() == dl.data_ptr() and got[4].data_ptr() == df.data_ptr()
    wt, wr, wl, wf = table.tolist(), ring.tolist(), lens.tolist(), free
    rng = np.random.default_rng(0)
    for _ in range(40):
        change = [int(-wl[s]) if rng.random() < 0.1 else int(rng.integers(-1, 3)) for s in range(seqs)]
        dc.copy_(_int(change))
        want = plain.tables(change, wl, wt, page, seqs, wr, wf)
        graph.replay()
        torch.cuda.synchronize()
        assert [g.tolist() for g in got] == list(want)
        assert dt.tolist() == wt and dr.tolist() == wr
        wl, wf = want[2], want[4]


@pytest.mark.parametrize("tokens", [4000, 9000])
def test_tables_of_prompts_replayed(tokens):
    """Both ways of writing rows, captured: replays read the lengths and the ring anew."""
    page, seqs = 16, 12
    dl, dc, df = _int([0] * seqs), _int([0] * seqs), _int([0, 700])
    dt, dr = torch.full((seqs, 100), -1, dtype=torch.int32, device=DEV), _int(list(range(700)))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = lg.batch_tables(dc, dl, dt, page, tokens, dr, df, in_place=True)
    wt, wr, wl, wf = dt.tolist(), dr.tolist(), [0] * seqs, [0, 700]
    rng = np.random.default_rng(3)
    for step in range(8):
        change = [-wl[s] if (s + step) % 3 == 0 else int(rng.integers(1, 900)) for s in range(seqs)]
        dc.copy_(_int(change))
        want = plain.tables(change, wl, wt, page, tokens, wr, wf)
        graph.replay()
        torch.cuda.synchronize()
        assert [g.tolist() for g in got] == list(want)
        assert dt.tolist() == wt and dr.tolist() == wr
        wl, wf = want[2], want[4]


# -------------------------------------------------------------------- sampling

def _margin(vocab):
    """How far, of the total, a border has to be from moving so that it does not; a total's
    logarithm is off by no more. A weight m 2^e, m in [1, 2], is off by at most 2^(e - 41) (rounded
    to 41 bits) and 2^-43 of itself (its polynomial). Sums in units of 2^-S of the largest weight,
    S = min(50, 62 - log2(vocab)), lose up to a unit for each of 1024 bins and each 256 tokens;
    tokens below 2^-63 are left out. Twice all that, for a sum and what it is compared with."""
    unit = 2.0 ** -min(50, 62 - (vocab - 1).bit_length())
    return 2 * ((1024 + vocab / 256) * unit + 2.0 ** -41 + 2.0 ** -43 + vocab * 2.0 ** -63)


def _logits(rows, vocab, seed, spread=2.5):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, spread, (rows, vocab))
    for r in range(rows):
        at = rng.integers(0, vocab, min(20, vocab))
        x[r, at] += rng.normal(5, 2.5, len(at))
    return x


def _sample_check(x, u, temperature=None, top_k=None, top_p=None, min_p=None, logits=None):
    """x: a CPU tensor of logits; the settings lists or None."""
    d = x.to(DEV) if logits is None else logits
    dev = [None if a is None else _int(a, t) for a, t in ((temperature, F32), (top_k, torch.int32), (top_p, F32),
                                                         (min_p, F32))]
    tokens, logprobs = lg.sample_tokens(d, _int(u, F32), *dev)
    assert tokens.dtype == torch.int64 and logprobs.dtype == F32
    tokens, logprobs = tokens.tolist(), logprobs.tolist()
    near = 0
    rows = x.double().numpy()

    def setting(a, r, default):
        return default if a is None else float(np.float32(a[r]))

    for r in range(x.shape[0]):
        want, logprob, margin = plain.sample(rows[r], float(np.float32(u[r])), setting(temperature, r, 1.0),
                                             0 if top_k is None else top_k[r], setting(top_p, r, 1.0),
                                             setting(min_p, r, 0.0))
        if margin < _margin(x.shape[1]):
            near += 1
            continue
        assert tokens[r] == want, (r, tokens[r], want, margin)
        if want < 0:
            assert logprobs[r] != logprobs[r]
        else:  # rounded once from 64 bits
            assert abs(logprobs[r] - logprob) <= 2.0 ** -24 * abs(logprob) + _margin(x.shape[1]), (r, logprobs[r], logprob)
    assert near <= x.shape[0] // 20, f"{near} rows too close to a border"
    return tokens


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 64, 1000, 4097, 8191, 8192, 32000, 50272, 131073])
def test_sample(dtype, vocab):
    rows = 24
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(_logits(rows, vocab, vocab)).to(dtype)
    u = rng.random(rows).astype(np.float32).clip(0, 1 - 2.0 ** -24).tolist()
    t, p, m = rng.uniform(0.5, 1.5, rows).tolist(), rng.uniform(0.3, 0.99, rows).tolist(), rng.uniform(0, 0.2, rows).tolist()
    k = rng.integers(1, 300, rows).tolist()
    _sample_check(x, u)
    _sample_check(x, u, t)
    _sample_check(x, u, t, top_k=k)
    _sample_check(x, u, t, top_p=p)
    _sample_check(x, u, t, min_p=m)
    _sample_check(x, u, t, k, p, m)
    mixed = [[v if i % 3 == j else off for i, v in enumerate(a)] for j, (a, off) in
             enumerate(((k, 0), (p, 1.0), (m, 0.0)))]
    t[4] = t[9] = 0.0
    _sample_check(x, u, t, *mixed)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_sample_equal_logits(dtype):
    """Equal logits are taken by their index; sums of equal weights are exact."""
    rows, vocab = 16, 4096
    x = torch.zeros((rows, vocab), dtype=dtype)
    x[1] = -0.0
    x[2, ::2] = -0.0
    x[3, 100:] = -5.0
    x[4] = torch.arange(vocab).remainder(3).to(dtype)
    x[5, 7] = x[5, 4000] = 4.0
    u = [i / rows for i in range(rows)]
    one = [1.0] * rows
    assert _sample_check(x, u)[:2] == [0, 256]
    # k of the equal ones: the first k
    got = _sample_check(x, [1 - 2.0 ** -24] * rows, top_k=[5] * rows)
    assert got[0] == 4 and got[1] == 4 and got[2] == 4 and got[3] == 4 and got[4] == 14
    got = _sample_check(x, [1 - 2.0 ** -24] * rows, top_p=[0.25] * rows)
    assert got[0] == 1023 and got[1] == 1023 and got[2] == 1023
    got = _sample_check(x, [1 - 2.0 ** -24] * rows, top_p=[0.5] * rows, top_k=[8] * rows)
    assert got[0] == 3
    got = _sample_check(x, [1 - 2.0 ** -24] * rows, min_p=one)
    assert got[0] == vocab - 1 and got[5] == 4000
    got = _sample_check(x, u, temperature=[0.0] * rows)
    assert got[0] == 0 and got[4] == 2 and got[5] == 7


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_sample_masked_and_extreme_logits(dtype):
    rows, vocab = 12, 9001
    x = torch.from_numpy(_logits(rows, vocab, 5)).to(dtype)
    x[0, 1:] = -INF
    x[1, :-1] = -INF
    x[2, ::2] = -INF
    x[3] = -INF
    x[3, 4000:4003] = 2.0
    big = torch.finfo(dtype).max
    x[4] = -big
    x[4, 77] = big
    x[5] = big
    x[6] = torch.finfo(dtype).tiny * torch.arange(vocab).remainder(5).to(dtype)
    x[7] *= 0
    x[7, 5] = -big
    x[8] *= 100
    u = np.random.default_rng(2).random(rows).astype(np.float32).tolist()
    u[0] = 0.0
    u[1] = 1 - 2.0 ** -24
    for t in (1.0, 0.01, 1e-30, 1e30, 3e38, 1e-45):
        for more in (dict(), dict(top_k=[3] * rows), dict(top_p=[0.6] * rows), dict(top_k=[2000] * rows, top_p=[0.9] * rows),
                     dict(min_p=[0.05] * rows)):
            _sample_check(x, u, [t] * rows, **more)


def test_sample_rows_without_a_distribution():
    rows, vocab = 14, 1003
    x = torch.from_numpy(_logits(rows, vocab, 6)).to(F16)
    x[0, 7] = NAN
    x[1, 1002] = INF
    x[2] = -INF
    u, t, p, m = [0.5] * rows, [1.0] * rows, [0.9] * rows, [0.0] * rows
    u[3], u[4], u[5], u[6] = 1.0, -0.1, NAN, INF
    t[7], t[8], t[9] = -1.0, NAN, INF
    p[10], m[11] = NAN, NAN
    p[12], m[13] = -1.0, 5.0
    for more in (dict(), dict(top_k=[9] * rows)):
        got = _sample_check(x, u, t, top_p=p, min_p=m, **more)
        assert got[:12] == [-1] * 12 and min(got[12:]) >= 0
        assert got[12] == int(x[12].float().argmax()) and got[13] == int(x[13].float().argmax())


def test_sample_settings_that_filter_nothing():
    x = torch.from_numpy(_logits(5, 3001, 7)).to(BF16)
    u = [0.1, 0.3, 0.5, 0.7, 0.9]
    want = _sample_check(x, u)
    assert _sample_check(x, u, [1.0] * 5, [0, -1, 3001, 1 << 30, -(1 << 31)], [1.0, 1.5, INF, 1.0, 2.0],
                         [0.0, -1.0, -INF, 0.0, -0.5]) == want


@pytest.mark.parametrize("dtype", [F16, F32])
@pytest.mark.parametrize("top_p", [0.999999, 0.5, 1e-30, 0.0])
def test_sample_flat_and_steep(dtype, top_p):
    """Borders among many tokens of one value, and none but the first."""
    rows, vocab = 6, 70001
    x = torch.zeros((rows, vocab), dtype=dtype)
    x[1] = torch.linspace(-1, 1, vocab).to(dtype)
    x[2] = torch.linspace(0, 50, vocab).to(dtype)
    x[3, 50000:] = 0.25
    x[4] = torch.arange(vocab).remainder(256).to(dtype) / 16
    x[5, 69999] = 12.0
    u = [0.999999, 0.2, 0.4, 0.6, 0.8, 0.3]
    _sample_check(x, u, top_p=[top_p] * rows)
    _sample_check(x, u, top_p=[top_p] * rows, top_k=[40000] * rows)
    _sample_check(x, u, [0.7] * rows, top_p=[top_p] * rows, min_p=[0.01] * rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("k", [2047, 2048, 2049, 4096, 4097, 20000])
def test_sample_large_top_k(dtype, k):
    """About where a list ends, with borders among equal values and all filters together."""
    rows, vocab = 8, 30001
    x = torch.from_numpy(_logits(rows, vocab, k)).to(dtype)
    x[5] = torch.arange(vocab).remainder(9).to(dtype) / 8
    x[6, 2100:] = -INF
    x[7] = 1.5
    u = [(i + 0.5) / rows for i in range(rows)]
    _sample_check(x, u, top_k=[k] * rows)
    _sample_check(x, u, [1.4] * rows, [k] * rows, [0.95] * rows)
    _sample_check(x, u, [0.8] * rows, [k] * rows, None, [0.003] * rows)
    _sample_check(x, u, [1.1] * rows, [k] * rows, [0.9] * rows, [0.001] * rows)


def test_sample_more_rows_than_a_launch_takes():
    """Rows beyond what the workspace holds at a time: the same inputs give the same results."""
    rows, period, vocab = 3000, 100, 50272
    base = torch.from_numpy(_logits(period, vocab, 13)).to(BF16)
    x = base.to(DEV).repeat(rows // period, 1)
    rng = np.random.default_rng(13)
    u = np.tile(rng.random(period).astype(np.float32).clip(0, 1 - 2.0 ** -24), rows // period).tolist()
    p = [1.0 if r % period < 50 else 0.9 for r in range(rows)]
    k = [40 if r % period % 7 == 0 else 0 for r in range(rows)]
    t = [0.0 if r % period == 3 else 0.9 for r in range(rows)]
    got = lg.sample_tokens(x, _int(u, F32), _int(t, F32), _int(k), _int(p, F32))
    for g in got:
        assert torch.equal(g, g[:period].repeat(rows // period))
    want = _sample_check(base, u[:period], t[:period], k[:period], p[:period])
    assert got[0][:period].tolist() == want


def test_sample_strided_and_unaligned_rows():
    wide = torch.from_numpy(_logits(9, 5011, 8)).to(F16)
    dev = wide.to(DEV)
    u = [i / 9 for i in range(9)]
    for lo, hi in ((1, 5010), (3, 4099), (8, 5000), (0, 5011)):
        _sample_check(wide[:, lo:hi].contiguous(), u, top_p=[0.9] * 9, logits=dev[:, lo:hi])
    _sample_check(wide[::2].contiguous(), u[:5], top_k=[50] * 5, logits=dev[::2])


def test_sample_largest_vocabulary():
    x = torch.from_numpy(_logits(2, 1 << 20, 9, 1.0)).to(F32)
    _sample_check(x, [0.3, 0.9], top_p=[0.7, 0.9])
    _sample_check(x, [0.3, 0.9])
    _sample_check(x.to(BF16), [0.3, 0.9], top_p=[0.7, 0.9])


def test_sample_repeats_graphs_and_streams():
    rows, vocab = 40, 32000
    x = torch.from_numpy(_logits(rows, vocab, 10)).to(F16).to(DEV)
    u = torch.rand(rows, device=DEV)
    t, p = torch.full((rows,), 0.8, device=DEV), torch.full((rows,), 0.9, device=DEV)
    first = lg.sample_tokens(x, u, t, top_p=p)
    for _ in range(3):
        again = lg.sample_tokens(x, u, t, top_p=p)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = lg.sample_tokens(x, u, t, top_p=p)
    for _ in range(4):
        u.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, lg.sample_tokens(x, u, t, top_p=p)))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = lg.sample_tokens(x, u, t, top_p=p)
    here = lg.sample_tokens(x, u, t, top_p=p)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(here, other))


def test_sample_rows_far_apart():
    """Rows that begin more than 2^32 bytes, and 2^31 elements, into the logits."""
    vocab = 131073
    x = torch.from_numpy(_logits(5, vocab, 14)).to(BF16)
    dev = torch.zeros((4 * 4100 + 1, vocab), dtype=BF16, device=DEV)
    assert dev.numel() > 1 << 31
    far = dev[::4100]
    far.copy_(x)
    u = [0.1, 0.3, 0.5, 0.7, 0.9]
    _sample_check(x, u, top_p=[0.9, 0.8, 0.7, 1.0, 0.95], logits=far)
    _sample_check(x, u, [0.0, 1.0, 0.0, 1.0, 0.0], logits=far)


def test_two_graphs_replayed_at_once():
    """Graphs of all three operators on two streams at a time share nothing."""
    b = Shared(BF16, 16, 2, 128, 32, [900], [0, 6], [20, 300, 7, 64, 65, 1], [1, 40, 1, 3, 1, 1], seed=33)
    x = torch.from_numpy(_logits(50, 32000, 15)).to(F16).to(DEV)
    change, lens = _int([3] * 2000), _int([17] * 2000)
    ring, free = _int(list(range(6000))), _int([5, 4000])

    def work(i):
        table = torch.arange(8000, dtype=torch.int32, device=DEV).view(2000, 4)
        u = torch.linspace(0.1 * i, 0.5 + 0.1 * i, 50, device=DEV)
        got = lg.sample_tokens(x, u, top_p=torch.full((50,), 0.9, device=DEV))
        return (b.run(), *got, *lg.batch_tables(change, lens, table, 16, 6000 + i, ring, free), table)

    want = [work(i) for i in range(2)]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[i]):
            out = work(i)
        graphs.append((g, out))
    for _ in range(3):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i][0].replay()
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))


def test_results_under_inference_mode():
    x = torch.from_numpy(_logits(3, 100, 16)).to(F16).to(DEV)
    u = _int([0.2, 0.5, 0.8], F32)
    want = lg.sample_tokens(x, u)
    table = _int([[0, 1], [2, 3]])
    with torch.inference_mode():
        tokens, logprobs = lg.sample_tokens(x, u)
        got = lg.batch_tables(_int([1, 2]), _int([3, 4]), table, 4, 3)
        assert torch.equal(tokens + 1, want[0] + 1) and torch.equal(logprobs * 2, want[1] * 2)
        assert got[0].tolist() == [3, 4, 5] and got[1].tolist() == [3, 12, 13]
        got[0].add_(1)
    assert tokens.is_inference() and got[3].tolist() == [0, 1, 3] and got[0].tolist() == [4, 5, 6]


def test_sample_follows_the_distribution():
    """Evenly spaced numbers draw each token as often as its probability says, to one draw."""
    vocab, rows = 50, 4096
    x = torch.from_numpy(_logits(1, vocab, 11, 1.5)).to(F32)
    u = (np.arange(rows) + 0.5) / rows
    tokens, _ = lg.sample_tokens(x.expand(rows, vocab).to(DEV), _int(u.tolist(), F32))
    count = np.bincount(tokens.cpu().numpy(), minlength=vocab)
    p = torch.softmax(x[0].double(), 0).numpy()
    assert np.abs(count - p * rows).max() <= 1.0 + 1e-3


def test_sample_nothing_to_do_and_out():
    tokens, logprobs = lg.sample_tokens(torch.empty((0, 100), dtype=F16, device=DEV), _int([], F32))
    assert tokens.shape == (0,) and logprobs.shape == (0,)
    out = torch.full((3,), -9, dtype=torch.int64, device=DEV)
    before = out._version
    tokens, _ = lg.sample_tokens(torch.zeros((3, 10), dtype=F32, device=DEV), _int([0.0, 0.5, 0.9], F32), out=out)
    assert tokens.data_ptr() == out.data_ptr() and out._version > before
    assert out.tolist() == [0, 5, 8]  # 0.9 in 32 bits is less than 9 of 10


def test_sample_filters_together_on_few_tokens():
    """top_k above the number of tokens with weight, with top_p before min_p."""
    x = torch.full((4, 5000), -INF)
    x[:, 100:140] = torch.from_numpy(_logits(4, 40, 12, 1.5)).float()
    u = [0.2, 0.5, 0.8, 0.99]
    for dtype in (F16, BF16, F32):
        for k in (39, 40, 41, 1000, 4000):
            for p, m in ((0.7, 0.0), (0.9, 0.3), (0.5, 0.6), (1.0, 0.2)):
                _sample_check(x.to(dtype), u, [1.3] * 4, [k] * 4, [p] * 4, [m] * 4)


def test_sample_largest_value_late_and_at_ends():
    """A piece whose first tokens say little of its largest, rows of every alignment and end."""
    for vocab in (8193, 40000, 70001, 131073):
        base = _logits(6, vocab + 16, vocab, 1.0)
        base[0, -vocab // 2] = 60.0
        base[1, vocab - 1] = 30.0
        base[2, 0] = 25.0
        base[3, : vocab // 2] = -INF
        base[4] = np.sort(base[4]) * 4
        x = torch.from_numpy(base)
        for dtype in (F16, F32):
            dev = x.to(dtype).to(DEV)
            for lo in (0, 1, 3):
                part = x.to(dtype)[:, lo:lo + vocab].contiguous()
                for more in (dict(), dict(top_p=[0.8] * 6), dict(top_k=[40] * 6), dict(min_p=[0.02] * 6)):
                    _sample_check(part, [0.1, 0.3, 0.5, 0.7, 0.9, 0.97], [0.9] * 6, logits=dev[:, lo:lo + vocab], **more)


# ------------------------------------------------------------------- together

def test_requests_on_a_shared_prefix_from_tables_to_tokens():
    """Requests that share a system prompt: its keys once, then chunks of their own prompts and
    single tokens, finished ones giving their pages back: tables, rotation and append, attention,
    head product and draw against the plain forms on the keys appended so far."""
    heads, kv, dim, page, vocab = 8, 2, 64, 16, 500
    g = torch.Generator().manual_seed(0)
    rope = lg.rotary_table(400, dim, device=DEV)
    pages, width = 60, 9
    k_pages, v_pages = (torch.full((pages, page, kv, dim), NAN, dtype=F16, device=DEV) for _ in range(2))
    head = (torch.randn((heads * dim, vocab), generator=g) * 0.2).to(F16).to(DEV)
    prefix = 37
    # the prefix by one step of its own
    ring, free = _int(np.random.default_rng(0).permutation(pages).tolist()), _int([50, pages])
    ptable, plen = _int([[-1] * 5]), _int([0])
    pos, slots, plen, starts, free = lg.batch_tables(_int([prefix]), plen, ptable, page, prefix, ring, free)
    assert plen.tolist() == [prefix] and pos.tolist() == list(range(prefix))
    qkv = torch.randn((prefix, (heads + 2 * kv) * dim), generator=g).to(F16).to(DEV)
    q = lg.qk_norm_rotate(qkv, heads, kv, pos, rope, k_pages=k_pages, v_pages=v_pages, slots=slots)
    lg.paged_attention(q, k_pages, v_pages, ptable, plen, starts)

    def keys(table, n):
        rows = table[:-(-n // page)].long()
        return [_np(t[rows].flatten(0, 1)[:n]) for t in (k_pages, v_pages)]

    want_prefix = keys(ptable[0], prefix)
    assert all(np.isfinite(t).all() for t in want_prefix)
    table = torch.full((3, width), -1, dtype=torch.int32, device=DEV)
    lens, offsets = _int([0, 0, 0]), _int([prefix] * 3)
    host = [0, 0, 0]
    for step, change in enumerate([[30, 1, 7], [1, 1, 1], [1, -2, 20], [2, 3, 1], [-33, 1, 1], [5, 1, -10]]):
        tokens = 40
        pos, slots, lens, starts, free = lg.batch_tables(_int(change), lens, table, page, tokens, ring, free, offsets)
        at = starts.tolist()
        for r, c in enumerate(change):
            assert pos[at[r]:at[r + 1]].tolist() == list(range(prefix + host[r], prefix + host[r] + max(c, 0)))
            host[r] = max(0, host[r] + c)
        assert lens.tolist() == host
        qkv = torch.randn((tokens, (heads + 2 * kv) * dim), generator=g).to(F16).to(DEV)
        q = lg.qk_norm_rotate(qkv, heads, kv, pos, rope, k_pages=k_pages, v_pages=v_pages, slots=slots)
        o = lg.shared_prefix_attention(q, k_pages, v_pages, ptable, plen, table, lens, starts)
        x = _np(qkv).reshape(tokens, heads + 2 * kv, dim)
        for r, c in enumerate(change):
            if c <= 0:
                continue
            rows = slice(at[r], at[r + 1])
            ks, vs = keys(table[r], host[r])
            assert np.array_equal(vs[-c:], x[rows, heads + kv:])
            ks, vs = np.concatenate([want_prefix[0], ks]), np.concatenate([want_prefix[1], vs])
            want, bound = plain.attention(_np(q[rows]), ks, vs, c, prefix + host[r], dim ** -0.5, 0, U[F16])
            assert (np.abs(_np(o[rows]) - want) <= bound).all(), (step, r)
        live = [r for r, c in enumerate(change) if c > 0]
        last = torch.tensor([at[r + 1] - 1 for r in live], device=DEV)
        logits = o[last].reshape(len(live), -1) @ head
        u = [(0.37 * (step + 1) + 0.21 * r) % 1 for r in live]
        _sample_check(logits.cpu(), u, [0.7] * len(live), top_p=[0.9] * len(live))
    # what the requests hold and what is free are all pages, once each
    used = ptable[0, :3].tolist() + [p for r in range(3) for p in table[r, :-(-host[r] // page)].tolist()]
    first, count = free.tolist()
    assert sorted(used + [ring[(first + i) % pages].item() for i in range(count)]) == list(range(pages))


@pytest.mark.parametrize("model,prefix", [("llama7b", 70), ("llama7b", 0), ("opt175b", 64)])
def test_decode_stack_steps_forward(model, prefix):
    """Captured steps on a cache with room: each appends the next token of every sequence, attends
    over prefix and own keys, and draws a token; when the room is full nothing moves any more."""
    from lut_gemv_amd import decode
    layers = 2 if model == "llama7b" else 1
    st = decode.DecodeStack(model, layers=layers, q=2, g=128, m=3, device=DEV, context=100, page_size=16,
                            prefix=prefix, room=6, sample=True)
    heads, own = st.heads, 100 - prefix
    room = -(-(own + 6) // 16) * 16      # whole pages
    graph = st.capture()                 # an eager step: the first
    held = st.page_table.clone()
    for step in range(1, room - own + 2):
        st.u.copy_(_int([0.1 * step % 1, 0.5, 0.9], F32))
        before = st.attended.clone()
        graph.replay()
        torch.cuda.synchronize()
        n = min(own + step + 1, room)
        assert st.kv_lens.tolist() == [n] * 3
        if own + step >= room:
            assert torch.equal(st.attended, before) and st.slots.tolist() == [-1] * 3
            continue
        assert st.positions.tolist() == [100 + step] * 3
        k_pages, v_pages = st.caches[-1]
        pk, pv = ([], []) if not prefix else ([t[st.prefix_table[0].long()].flatten(0, 1)[:prefix]] for t in
                                             (k_pages, v_pages))
        for i in range(3):
            rows = st.page_table[i, :-(-n // 16)].long()
            ks, vs = (torch.cat(a + [t[rows].flatten(0, 1)[:n]]) for a, t in ((pk, k_pages), (pv, v_pages)))
            want, bound = plain.attention(_np(st.queries[i:i + 1]), _np(ks), _np(vs), 1, prefix + n, 128 ** -0.5, 0,
                                          U[F16])
            got = _np(st.attended.view(3, heads, 128)[i:i + 1])
            assert (np.abs(got - want) <= bound).all(), (step, i)
            qkv = _np(st.outs["qkv"][i]).reshape(3 * heads, 128)
            assert np.array_equal(_np(vs[-1]), qkv[2 * heads:])
        logits = st.head(st.outs[st.out_name])
        assert torch.equal(logits, st.logits)
        for i in range(3):
            token, logprob, margin = plain.sample(_np(logits[i]), float(st.u[i]), float(st.temperature[i]), 0,
                                                  float(st.top_p[i]))
            if margin >= _margin(logits.shape[1]):
                assert int(st.tokens[i]) == token
                assert abs(float(st.logprobs[i]) - logprob) <= 2.0 ** -24 * abs(logprob) + _margin(logits.shape[1])
    assert (st.page_table >= 0).sum() >= (held >= 0).sum()


def test_decode_rate_counts_prefix_and_head():
    from lut_gemv_amd import decode
    st = decode.DecodeStack("llama7b", layers=1, q=2, g=128, m=3, device=DEV, page_size=16, context=100, prefix=60,
                            sample=True)
    nb, na, _ = lg.packed_sizes(32000, 4096, 2, 128, False)
    read = st.bytes_per_step() + (60 + 3 * 41) * 2 * 4096 * 2 + nb + 2 * na + 2 * 3 * 32000
    r = st.time_tokens(tokens=2, warmup=1)
    assert r["GBps"] == pytest.approx(read / (r["ms_per_step"] * 1e-3) / 1e9, rel=1e-9)


def _sample_rows(x, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """Every row's draw by the definition, also next to a border: a token that the filters keep, up to
    which the kept weights sum to more than u times their total, but for _margin of it. What the
    last call's results held is no answer: the memory is filled before."""
    rows, vocab = x.shape
    near = _margin(vocab)
    dev = [None if a is None else _int(a, t) for a, t in ((temperature, F32), (top_k, torch.int32), (top_p, F32),
                                                         (min_p, F32))]
    d, du, out = x.to(DEV), _int(u, F32), _int([-7] * rows, torch.int64)
    last = torch.full((12 * rows,), 0xFF, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    del last
    tokens, logprobs = lg.sample_tokens(d, du, *dev, out=out)
    tokens, logprobs, rounded = tokens.tolist(), logprobs.tolist(), x.double().numpy()
    for r in range(rows):
        t = 1.0 if temperature is None else float(np.float32(temperature[r]))
        order = np.argsort(-rounded[r], kind="stable")
        w = np.exp((rounded[r][order] - rounded[r][order[0]]) / t)
        sure = np.ones(vocab, bool)      # kept wherever the borders lie within the margin
        if top_k is not None and top_k[r] > 0:
            w[top_k[r]:] = 0
        maybe = w > 0
        if top_p is not None and top_p[r] < 1:
            before = (np.cumsum(w) - w) / w.sum()
            p = float(np.float32(top_p[r]))
            sure &= before < p - near
            maybe &= before < p + near
        if min_p is not None and min_p[r] > 0:
            least = min(float(np.float32(min_p[r])), 1.0)
            sure &= w >= least * (1 + 2.0 ** -40)
            maybe &= w >= least * (1 - 2.0 ** -40)
        sure[0] = maybe[0] = True
        sure &= maybe
        kept, most = np.zeros(vocab), np.zeros(vocab)
        kept[order], most[order] = w * sure, w * maybe
        loose = (most.sum() - kept.sum()) / kept.sum() + near
        token = tokens[r]
        assert 0 <= token < vocab and most[token] > 0, (r, token)
        upto = np.cumsum(most) / most.sum()
        below = upto[token] - most[token] / most.sum()
        assert below - loose <= u[r] <= upto[token] + loose, (r, token, below, upto[token], u[r])
        logprob = np.log(most[token] / most.sum())
        assert abs(logprobs[r] - logprob) <= 2.0 ** -24 * abs(logprob) + 2 * loose, (r, logprobs[r], logprob)
    return tokens


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 11])
def test_sample_small_parts_of_a_large_top_k(dtype, rows):
    """One token has nearly all weight, and u is among the last places of the total: the first
    pieces' tokens have a sum together, but none that their parts, 64 words of 16 bytes each, would
    be rounded to. A row is answered whatever the sums of its pieces and its parts are."""
    vocab = 131072                       # sums in units of 2^-45 of the largest weight
    part = 64 * (4 if dtype == F32 else 8)
    x = torch.full((rows, vocab), -INF, dtype=dtype)
    for r in range(rows):
        x[r, vocab - 1] = r / 8
        light = np.log((0.1 + 0.03 * r) * 2.0 ** -45) + r / 8
        x[r, part + r:16384:part] = light                # no part of these has half a unit
        x[r, 65536 + 20 * np.arange(3000)] = light       # many in each part
    for u in (0.0, 2.0 ** -45, 2.0 ** -40, 0.5):
        for k in (2049, 2500, 100000):
            _sample_rows(x, [u] * rows, top_k=[k] * rows)
            _sample_rows(x, [u] * rows, top_k=[k] * rows, top_p=[1 - 2.0 ** -24] * rows)
            _sample_rows(x, [u] * rows, top_p=[1 - 2.0 ** -24] * rows)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("vocab", [50272, 131073])
def test_sample_peaked_rows_at_the_ends(dtype, vocab):
    """u at and next to 0 and 1 on rows whose weights span all that is counted."""
    rows = 6
    rng = np.random.default_rng(vocab)
    x = -rng.exponential(1, (rows, vocab)) * 2.0 ** np.arange(rows)[:, None] - 5.0 * np.arange(rows)[::-1, None]
    x[rng.random((rows, vocab)) < 0.3] = -INF
    x[np.arange(rows), rng.integers(0, vocab, rows)] = 1.0
    x = torch.from_numpy(x).to(dtype)
    for u in (0.0, 1e-45, 2.0 ** -50, 2.0 ** -44, 2.0 ** -30, 1 - 2.0 ** -24):
        for more in (dict(), dict(top_k=[7] * rows), dict(top_k=[2048] * rows), dict(top_k=[2500] * rows),
                     dict(top_k=[20000] * rows, top_p=[0.9999] * rows), dict(top_p=[0.97] * rows),
                     dict(top_p=[1 - 2.0 ** -24] * rows)):
            _sample_rows(x, [u] * rows, **more)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_sample_u_of_minus_zero(dtype):
    """-0 is 0: the first kept token."""
    rows, vocab = 3, 9001
    x = torch.from_numpy(_logits(rows, vocab, 11)).to(dtype)
    x[0, 4000:] = -INF       # the last parts are empty
    x[1, :5000] = -INF
    for more in (dict(), dict(top_k=[9] * rows), dict(top_k=[3000] * rows), dict(top_p=[0.9] * rows),
                 dict(temperature=[0.0] * rows),
                 dict(top_k=[2500] * rows, top_p=[0.99] * rows, min_p=[0.001] * rows)):
        got = _sample_check(x, [-0.0] * rows, **more)
        assert got == _sample_check(x, [0.0] * rows, **more)
        assert min(got) >= 0 and got[1] >= 5000


@pytest.mark.parametrize("dtype", [F16, F32])
def test_sample_min_p_alone_after_other_kernels(dtype):
    """The table of steps is written before any wave reads it, whatever the call before has left in
    the compute units' LDS."""
    rows, vocab = 600, 4001
    x = torch.from_numpy(_logits(rows, vocab, 12)).to(dtype)
    u = np.random.default_rng(4).random(rows).astype(np.float32).clip(0, 1 - 2.0 ** -24).tolist()
    m = np.random.default_rng(5).uniform(0.0005, 0.3, rows).tolist()
    b = Shared(F16, 32, 4, 128, 64, [2000], [0, 64], [70] * 64, [1] * 64, seed=31)
    b.run()
    first = _sample_check(x, u, min_p=m)
    for _ in range(3):
        b.run()
        assert _sample_check(x, u, min_p=m) == first
    assert _sample_check(x, [-0.0] * rows, min_p=m) == _sample_check(x, [0.0] * rows, min_p=m)


@pytest.mark.parametrize("low", ["prefix", "own"])
@pytest.mark.parametrize("news", [[1, 1], [40, 1]])
def test_shared_part_of_minus_infinity_beside_finite_scores(news, low):
    """A part all of whose scores are minus infinity has no weight beside a finite one: the row is
    that of the other keys alone. The other rows see finite scores in all parts."""
    b = Shared(BF16, 2, 2, 64, 16, [600], [0, 2], [40, 3], news, seed=21)
    b.q[:, :, 0] = 0
    low_key = -1e30
    b.q[0, :, 0] = 1e20
    own = b.page_table[:, :3][b.page_table[:, :3] >= 0].long()
    for which, pages, held in (("prefix", b.prefix_table[0, :38].long(), b.kv[:1]), ("own", own, b.kv[1:])):
        b.k_pages[pages, :, :, 0] = low_key if which == low else 0
        for k, _ in held:
            k[:, :, 0] = low_key if which == low else 0
    out = b.run()                         # the product is -1e50: minus infinity in fp32
    n = 40 - news[0] + 1                  # keys that the first row sees
    k, v = (_np(t) for t in (b.kv[1] if low == "prefix" else b.kv[0]))
    if low == "prefix":
        k, v = k[:n], v[:n]
    want, bound = plain.attention(_np(b.q[:1]), k, v, 1, len(k), 64 ** -0.5, 0, U[BF16])
    got = _np(out[:1])
    assert np.isfinite(got).all() and (np.abs(got - want) <= bound).all()
    for s in range(2):
        at = sum(news[:s])
        want, bound = b.want(s)
        skip = 1 if s == 0 else 0
        got = _np(out[at:at + news[s]])
        assert (np.abs(got - want) <= bound)[skip:].all(), s


def test_tables_of_more_pages_back_than_are_counted():
    """Two sequences give back 2^30 pages each, the second far behind what the ring takes: the ring
    gets the first pages of the first alone. (Their rows of the table are 8 GB.)"""
    width, capacity = 1 << 30, 1000
    table = torch.empty((2, width), dtype=torch.int32, device=DEV)
    table[:, :2000] = torch.arange(4000, dtype=torch.int32, device=DEV).view(2, 2000)
    ring = torch.full((capacity,), -1, dtype=torch.int32, device=DEV)
    lens = _int([width, width])
    got = lg.batch_tables(_int([-width, -width]), lens, table, 1, 0, ring, _int([300, 10]))
    assert got[2].tolist() == [0, 0] and got[4].tolist() == [300, capacity]
    want = [-1] * capacity
    for i in range(capacity - 10):
        want[(310 + i) % capacity] = i
    assert ring.tolist() == want
    # the second keeps its first pages, the first ends: the ring takes what there is room for
    ring.fill_(-1)
    got = lg.batch_tables(_int([-5, -width + 7]), _int([12, width]), table, 1, 0, ring, _int([0, 0]))
    assert got[2].tolist() == [7, 7] and got[4].tolist() == [0, capacity]
    assert ring.tolist() == list(range(7, 12)) + list(range(2007, 2007 + capacity - 5))


def test_decode_times_steps_from_the_context_on():
    """With room each kernel's timed steps begin at the context, none is behind the room's end, and
    the rate counts the keys that they read."""
    from lut_gemv_amd import decode
    st = decode.DecodeStack("llama7b", layers=1, q=2, g=128, m=3, device=DEV, page_size=16, context=100, prefix=60,
                            room=9)
    assert st.steps == 24                    # 40 own keys and 24 more in four pages
    tables = []
    for kernel in ("lut", "dequant", "lut"):
        for tokens, warmup in ((20, 4), (3, 0)):
            r = st.time_tokens(kernel, tokens, warmup)
            assert st.kv_lens.tolist() == [40 + warmup + tokens] * 3
            assert st.positions.tolist() == [99 + warmup + tokens] * 3
            keys = 60 + 3 * (41 + warmup + (tokens - 1) / 2)
            read = st.bytes_per_step() + keys * 2 * 4096 * 2
            assert r["GBps"] == pytest.approx(read / (r["ms_per_step"] * 1e-3) / 1e9, rel=1e-9)
        tables.append(st.page_table.tolist())
    assert tables[0] == tables[1] == tables[2]
    with pytest.raises(ValueError, match="room for 24 steps"):
        st.time_tokens("lut", 20, 5)


def test_readme_step_behind_a_prefix():
    """The step of the use example: rotated by positions behind the prefix, a request on a shared prefix
    has the results of one whose table holds the prefix itself."""
    rng = torch.Generator().manual_seed(8)
    heads, kv_heads, dim, page, prefix, own, pages = 8, 2, 128, 64, 150, 21, 12
    rope = lg.rotary_table(positions=512, rotary=dim, device=DEV)
    k, v = (torch.randn((pages, page, kv_heads, dim), generator=rng).to(F16).to(DEV) for _ in range(2))
    qkv = torch.randn((1, (heads + 2 * kv_heads) * dim), generator=rng).to(F16).to(DEV)
    ring = torch.arange(6, pages, dtype=torch.int32, device=DEV)
    # its own keys behind a prefix of whole pages: 128 keys in pages 0 and 1, 22 + 21 in page 2
    shared, table = 2 * page, _int([[2, -1, -1]])
    at = prefix - shared + own
    positions, slots, kv_lens, q_starts, _ = lg.batch_tables(
        _int([1]), _int([at]), table, page_size=page, tokens=1, free_pages=ring, free_range=_int([0, 6]),
        offsets=_int([shared]))
    assert positions.tolist() == [prefix + own] and slots.tolist() == [2 * page + at]
    q = lg.qk_norm_rotate(qkv, heads, kv_heads, positions, rope, k_pages=k, v_pages=v, slots=slots)
    o = lg.shared_prefix_attention(q, k, v, _int([[0, 1]]), _int([shared]), table, kv_lens, q_starts)
    whole = _int([[0, 1, 2, -1]])
    k2, v2 = k.clone(), v.clone()
    k2[2, at], v2[2, at] = 0, 0
    positions, slots, kv_lens, q_starts, _ = lg.batch_tables(
        _int([1]), _int([prefix + own]), whole, page_size=page, tokens=1, free_pages=ring.clone(),
        free_range=_int([0, 6]))
    q2 = lg.qk_norm_rotate(qkv, heads, kv_heads, positions, rope, k_pages=k2, v_pages=v2, slots=slots)
    assert torch.equal(q, q2) and torch.equal(k, k2) and torch.equal(v, v2)
    n = prefix + own + 1
    ks, vs = (_np(t[:3]).reshape(-1, kv_heads, dim)[:n] for t in (k, v))
    want, bound = plain.attention(_np(q), ks, vs, 1, n, dim ** -0.5, 0, U[F16])
    for got in (o, lg.paged_attention(q2, k2, v2, whole, kv_lens, q_starts)):
        assert (np.abs(_np(got) - want) <= bound).all()


@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(BF16, 16, 2, 128), (F16, 4, 4, 64)])
@pytest.mark.parametrize("small", [9, 63, 64, 90])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_shared_large_group_among_small_ones(small, at, dtype, heads, kv_heads, dim):
    """A group of many rows beside groups of one token, and chunks among them: each group by its
    own rows, however many there are on average."""
    large = 5 * small // (heads // kv_heads) + 20 // (heads // kv_heads)
    sizes = [1] * small
    sizes.insert(dict(first=0, middle=small // 2, last=small)[at], large)
    starts = [0, *np.cumsum(sizes).tolist()]
    seqs = starts[-1]
    rng = np.random.default_rng(small)
    for chunks in (False, True):
        news = [23 if chunks and s == seqs // 2 else 1 for s in range(seqs)]
        lens = [n + int(x) for n, x in zip(news, rng.integers(0, 40, seqs))]
        b = Shared(dtype, heads, kv_heads, dim, 16, [int(x) for x in rng.integers(0, 200, len(sizes))], starts, lens, news,
                   seed=small)
        b.check(b.run(), f"{large} among {small}, chunks {chunks}")
        b.check(b.run(max_q=max(news), max_kv=70, max_prefix=200), "with hints")


def test_shared_time_of_a_large_group_among_small_ones():
    """One call takes about as long as one of the large group and one of the small ones: were the
    large group read as single tokens are, 16 rows at a time, it would take ten times that."""
    gen = torch.Generator(device=DEV).manual_seed(0)

    def call(sizes):
        groups, seqs, pages = len(sizes), sum(sizes), 64
        total = groups * pages + 2 * seqs
        k, v = (torch.empty((total, 64, 4, 128), dtype=BF16, device=DEV).normal_(generator=gen) for _ in range(2))
        ids = torch.arange(total, dtype=torch.int32, device=DEV)
        q = torch.empty((seqs, 32, 128), dtype=BF16, device=DEV).normal_(generator=gen)
        a = (q, k, v, ids[:groups * pages].view(groups, pages), _int([4096] * groups),
             ids[groups * pages:].view(seqs, 2), _int([100] * seqs), None, _int([0, *np.cumsum(sizes).tolist()]))
        return lambda: lg.shared_prefix_attention(*a, max_q=1, max_kv=100, max_prefix=4096)

    def least(f):
        times = []
        for _ in range(12):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(5):
                f()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b) / 5)
        return min(times)

    apart = least(call([64])) + least(call([1] * 63))
    together = least(call([64] + [1] * 63))
    _say(f"apart {apart * 1e3:.0f} us, together {together * 1e3:.0f} us")
    assert together < 3 * apart
