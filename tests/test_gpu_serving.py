"""The operators beside the weight products on the GPU, against their plain fp64
forms (oracle/serving.py) with bounds counted there: paged attention, head norms
with rotation and cache append, low-rank adapters; then a run of them together
as a decoder layer uses them."""
import sys

import numpy as np
import pytest

from oracle import serving as plain

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import lut_gemv_amd as lg  # noqa: E402

DEV = "cuda:0"
F16, BF16 = torch.float16, torch.bfloat16
U = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
NAN = float("nan")


def _say(msg):
    print(f"[serving] {msg}", flush=True)
    sys.stdout.flush()


def _np(t):
    return t.detach().cpu().double().numpy()


def _inside(got, want, bound, what):
    got = _np(got)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float((np.abs(got - want) / np.maximum(bound, 1e-300)).max()) if got.size else 0.0
    _say(f"{what}: worst err/bound {worst:.3f}")
    assert worst <= 1.0, what


def _normal(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).to(DEV)


# ---------------------------------------------------------------- paged attention

class Batch:
    """Sequences in a paged cache whose unused slots and pages hold NaN."""

    def __init__(self, dtype, heads, kv_heads, dim, page, lens, news, seed=0, order="nhd",
                 scale=1.0, lead=0, tail=0):
        self.dtype, self.lens, self.news = dtype, lens, news
        self.page, self.heads, self.kv_heads, self.dim = page, heads, kv_heads, dim
        self.lead = lead
        need = [-(-n // page) for n in lens]
        pages, width = sum(need) + 2, max(max(need), 1) + 1
        rng = np.random.default_rng(seed)
        ids = rng.permutation(pages)
        shape = (pages, page, kv_heads, dim)
        k, v = (torch.full(shape, NAN, dtype=dtype) for _ in range(2))
        table = torch.full((len(lens), width), -7, dtype=torch.int32)
        g = torch.Generator().manual_seed(seed)
        self.k, self.v, at = [], [], 0
        for i, n in enumerate(lens):
            kn = (torch.randn((n, kv_heads, dim), generator=g) * scale).to(dtype)
            vn = torch.randn((n, kv_heads, dim), generator=g).to(dtype)
            for j in range(need[i]):
                page_id = int(ids[at])
                at += 1
                table[i, j] = page_id
                part = slice(j * page, min(n, (j + 1) * page))
                k[page_id, :part.stop - part.start] = kn[part]
                v[page_id, :part.stop - part.start] = vn[part]
            self.k.append(kn)
            self.v.append(vn)
        tokens = lead + sum(news) + tail
        self.q = _normal((tokens, heads, dim), dtype, seed + 1, scale)
        if order == "hnd":   # heads outside slots
            k, v = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (k, v))
            self.k_pages = k.to(DEV).transpose(1, 2).contiguous().transpose(1, 2)
            self.v_pages = v.to(DEV).transpose(1, 2).contiguous().transpose(1, 2)
        else:
            self.k_pages, self.v_pages = k.to(DEV), v.to(DEV)
        self.table = table.to(DEV)
        self.kv_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        starts = np.concatenate([[0], np.cumsum(news)]) + lead
        self.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)

    def call(self, **kw):
        return lg.paged_attention(self.q, self.k_pages, self.v_pages, self.table, self.kv_lens,
                                  kw.pop("q_starts", self.starts), **kw)

    def check(self, got, what, scale=None, window=0, only=None):
        scale = self.dim ** -0.5 if scale is None else scale
        q = _np(self.q)
        at = self.lead
        for i, (n, new) in enumerate(zip(self.lens, self.news)):
            rows = slice(at, at + new)
            at += new
            if only is not None and i not in only:
                continue
            want, bound = plain.attention(q[rows], _np(self.k[i]), _np(self.v[i]), new, n, scale,
                                          window, U[self.dtype])
            _inside(got[rows], want, bound, f"{what} seq {i} ({new} of {n})")


DECODE_LENS = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 300]


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 128), (16, 2, 128), (14, 2, 64), (3, 1, 64),
                                                (32, 2, 64), (24, 1, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_single_tokens(dtype, heads, kv_heads, dim):
    """One new token a sequence, keys from none to a few tiles, with and without starts."""
    b = Batch(dtype, heads, kv_heads, dim, 16, DECODE_LENS, [1] * len(DECODE_LENS), seed=heads)
    got = b.call(q_starts=None)
    b.check(got, f"decode {heads}/{kv_heads}x{dim}")
    assert torch.equal(got[0], torch.zeros_like(got[0]))
    same = b.call(max_q=1)
    b.check(same, "decode with starts")


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("window", [0, 1, 40, 700])
def test_attention_split_long_and_windows(page, window):
    """Keys split over workgroups, pages that end inside a tile, and windows."""
    lens = [2111, 1, 777, 1536, 0, 4097]
    b = Batch(F16, 8, 2, 128, page, lens, [1] * 6, seed=page + window)
    b.check(b.call(q_starts=None, window=window), f"page {page} window {window}", window=window)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 4, 128), (8, 2, 64), (5, 1, 128)])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("window", [0, 33])
def test_attention_chunks(dtype, heads, kv_heads, dim, window):
    """Chunks of one to a few tiles beside single tokens and sequences with no new
    token; one whose rows stand before its first key."""
    lens = [300, 5, 64, 129, 700, 1, 40, 513, 20]
    news = [130, 5, 64, 1, 3, 1, 0, 257, 33]
    b = Batch(dtype, heads, kv_heads, dim, 16, lens, news, seed=3 * heads + window)
    got = b.call(window=window)
    b.check(got, f"chunks {heads}/{kv_heads}x{dim} window {window}", window=window)
    b.check(b.call(window=window, max_q=1, max_kv=64), "with wrong hints", window=window)
    b.check(b.call(window=window, max_q=257, max_kv=700), "with right hints", window=window)


def test_attention_one_long_chunk_split():
    """Few row tiles on a long key axis: the 128-row kernel's parts are joined."""
    b = Batch(BF16, 4, 1, 128, 64, [5000], [40], seed=5)
    b.check(b.call(), "40 of 5000")
    b = Batch(F16, 8, 8, 64, 32, [3000, 2500, 90], [17, 1, 90], seed=6)
    b.check(b.call(), "17 of 3000 beside one of 2500")


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (8, 1, 128)])
def test_attention_more_sequences_than_lanes(heads, kv_heads, dim):
    """Row tiles are found otherwise from 65 sequences on; long ones among them are split."""
    rng = np.random.default_rng(3)
    news = [int(rng.choice([0, 1, 1, 3, 20, 70])) for _ in range(131)]
    lens = [n + int(rng.integers(0, 90)) for n in news]
    lens[5], news[5], lens[100], news[100] = 1700, 150, 2600, 1
    lens[64], news[64], lens[130], news[130] = 1300, 33, 1100, 129
    b = Batch(F16, heads, kv_heads, dim, 16, lens, news, seed=24)
    b.check(b.call(), "131 sequences")


@pytest.mark.parametrize("window", [0, 8500])
@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(F16, 8, 2, 64), (BF16, 4, 1, 128)])
def test_attention_chunks_on_long_unsplit_keys(dtype, heads, kv_heads, dim, window):
    """A launch made for short sequences takes a long key axis in one part: the pages'
    numbers are read 64 tiles at a time."""
    b = Batch(dtype, heads, kv_heads, dim, 16, [9000, 8300, 4200], [20, 17, 9], seed=44)
    b.check(b.call(max_kv=1, window=window), f"one part, window {window}", window=window)


def test_attention_large_and_small_scores():
    """Scores of some hundreds, where one key takes all the weight, and a small scale."""
    b = Batch(F16, 8, 2, 128, 16, [900, 33], [20, 1], seed=7, scale=4.0)
    b.check(b.call(), "scores near +-180", scale=None)
    b.check(b.call(scale=1e-4), "scale 1e-4", scale=1e-4)


@pytest.mark.parametrize("lens,news,hints", [
    ([40000, 30000], [1, 1], dict(max_q=1, max_kv=1)), ([40000, 30000], [1, 1], dict(max_q=1)),
    ([40000, 30000], [3, 4], dict(max_kv=1)), ([40000], [3], {}), ([40000, 50, 30000], [3, 1, 1], {}),
])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_many_small_weights_beside_a_large_one(dtype, lens, news, hints):
    """One key takes nearly all the weight and its value is zero: the output is what
    thousands of keys add whose weights are each about 2^-25.4 of it."""
    b = Batch(dtype, 8, 1, 64, 64, lens, news, seed=41)
    for i, n in enumerate(lens):
        b.k[i].zero_()
        b.k[i][0] = 2.2        # 64 x 2.2 / 8: 17.6, in base 2 25.4
        b.v[i][:] = 1.0 + (torch.arange(n) % 5)[:, None, None].to(dtype) / 8
        b.v[i][0] = 0
        for j in range(-(-n // 64)):
            part = slice(64 * j, min(n, 64 * j + 64))
            b.k_pages[int(b.table[i, j]), :part.stop - part.start] = b.k[i][part].to(DEV)
            b.v_pages[int(b.table[i, j]), :part.stop - part.start] = b.v[i][part].to(DEV)
    b.q.fill_(1.0)
    b.check(b.call(**hints), f"small weights {hints}")


def test_attention_rising_scores():
    """Every key scores higher than the one before: the running maximum moves all along."""
    b = Batch(F16, 4, 4, 64, 16, [640, 640], [1, 64], seed=8)
    for i in range(2):
        ramp = torch.linspace(-2, 2, 640)[:, None, None] * torch.ones((640, 4, 64))
        b.k[i] = ramp.to(F16)
        for j in range(40):
            b.k_pages[int(b.table[i, j])] = b.k[i][16 * j:16 * j + 16].to(DEV)
    b.q.fill_(1.0)
    b.check(b.call(scale=0.5), "rising", scale=0.5)


def test_attention_strides_and_rows_left_alone():
    """Heads outside slots in the cache, queries inside a fused product's rows, an output
    with gaps, rows before the first and after the last sequence left as they were."""
    b = Batch(F16, 6, 2, 64, 32, [100, 50, 333], [20, 1, 40], seed=9, order="hnd", lead=3, tail=4)
    assert b.k_pages.stride(2) > b.k_pages.stride(1)
    fused = _normal((b.q.shape[0], 10, 64), F16, 10)
    fused[:, :6] = b.q
    b.q = fused[:, :6]
    wide = torch.full((b.q.shape[0], 7, 72), 5.0, dtype=F16, device=DEV)
    out = wide[:, :6, :64]
    assert b.call(out=out) is out
    b.check(out, "strided")
    assert (wide[:3] == 5).all() and (wide[-4:] == 5).all()
    assert (wide[:, 6:] == 5).all() and (wide[:, :, 64:] == 5).all()


@pytest.mark.parametrize("news", [[1, 1, 1, 1], [20, 1, 30, 9]])
def test_attention_bad_pages_and_lengths(news):
    """A page number outside the cache or more keys than the table holds make that
    sequence's rows NaN and no others; negative lengths count as none."""
    b = Batch(F16, 4, 2, 128, 16, [70, 80, 90, 60], news, seed=11)
    b.table[0, 2] = 10 ** 6
    b.kv_lens[2] = 100000
    b.table[2] = 0
    got = b.call()
    at = np.concatenate([[0], np.cumsum(news)])
    # rows of sequence 0 that see a key of its third page
    assert torch.isnan(got[at[0 + 1] - 1]).all()
    assert torch.isnan(got[at[2]:at[3]]).all()
    b.check(got, "the others", only=[1, 3])
    b.table[0, 2] = -1
    b.kv_lens[3] = -5
    got = b.call()
    assert torch.isnan(got[at[1] - 1]).all()
    assert (got[at[3]:] == 0).all()


@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("lens,news,window", [
    ([127, 700, 64, 33], [1, 1, 1, 1], 64), ([127, 700, 90], [40, 1, 90], 40),
    ([5000, 4800], [1, 1], 700), ([3000, 2500], [20, 30], 600), ([300, 290], [1, 3], 1),
])
def test_attention_pages_released_behind_the_window(page, lens, news, window):
    """Table entries whose keys all lie before the window of a sequence's first new token
    may hold anything."""
    b = Batch(F16, 8, 2, 128, page, lens, news, seed=page + window)
    want = b.call(window=window, max_q=max(news))
    for i, (n, new) in enumerate(zip(lens, news)):
        gone = max(n - new - window + 1, 0) // page
        b.table[i, :gone] = torch.tensor([-1, 2 ** 31 - 1, len(b.k_pages)] * gone)[:gone]
    got = b.call(window=window, max_q=max(news))
    b.check(got, "released pages", window=window)
    assert torch.equal(got, want)


def test_attention_non_finite_keys_stay_behind_the_mask():
    """NaN and infinity among the keys reach exactly the rows that see them."""
    b = Batch(F16, 2, 1, 64, 16, [200], [100], seed=12)
    bad = 150
    b.k_pages[int(b.table[0, bad // 16]), bad % 16, 0, 5] = float("nan")
    got = b.call()
    row = bad - 100
    assert torch.isfinite(got[:row]).all() and torch.isnan(got[row:]).all()


@pytest.mark.parametrize("lens,news", [
    ([1, 40], [1, 1]), ([40, 129], [40, 129]), ([3000, 2000], [1, 1]), ([3000], [20]),
    ([700, 30], [130, 1]),
])
def test_attention_rows_whose_scores_are_all_minus_infinity(lens, news):
    """The softmax of such a row is not defined: it is NaN, and not the zero of a row that
    sees no key. Among finite scores minus infinity is a weight of zero."""
    b = Batch(F16, 8, 2, 64, 16, lens, news, seed=43)
    b.q[:, :, 3] = 1.0
    keep = b.k_pages.clone()
    b.k_pages[..., 3] = float("-inf")
    assert torch.isnan(b.call()).all()
    b.k_pages.copy_(keep)
    for i in range(len(lens)):   # one key of many
        if lens[i] > 5 and lens[i] - news[i] > 5:
            b.k_pages[int(b.table[i, 0]), 4, :, 3] = float("-inf")
            b.v[i] = torch.cat([b.v[i][:4], b.v[i][5:]])
            b.k[i] = torch.cat([b.k[i][:4], b.k[i][5:]])
            b.lens = b.lens[:i] + [lens[i] - 1] + b.lens[i + 1:]
    b.check(b.call(), "one score of minus infinity")


@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(F16, 4, 2, 128), (BF16, 3, 1, 64)])
@pytest.mark.parametrize("lens,news,window", [
    ([200], [100], 0), ([200, 90], [5, 4], 0), ([200, 190], [1, 1], 40), ([4000], [40], 0),
    ([300, 280, 150], [130, 1, 3], 50), ([2200, 700], [3, 1], 90),
])
def test_attention_non_finite_values_stay_behind_the_mask(dtype, heads, kv_heads, dim, lens, news,
                                                          window):
    """NaN and infinities among the values reach the rows that see them, in their own
    columns, and no others. The first two lie at the first new token and one before it
    (rows see the last keys, windows only some), the third before the window."""
    b = Batch(dtype, heads, kv_heads, dim, 16, lens, news, seed=21)
    marks = []
    for i, (n, new) in enumerate(zip(lens, news)):
        first = n - new
        for key, col, value in ((first + new // 2, 5, NAN), (first, 18, float("inf")),
                                (max(first - window - 1, 0), dim - 1, float("-inf"))):
            b.v_pages[int(b.table[i, key // 16]), key % 16, :, col] = value
            b.v[i][key, :, col] = 0
            marks.append((i, key, col, value))
    got = b.call(window=window)
    at = np.concatenate([[0], np.cumsum(news)])
    seen = torch.zeros(got.shape, dtype=torch.bool, device=DEV)
    for i, key, col, value in marks:
        for t in range(news[i]):
            pos = lens[i] - news[i] + t
            if key <= pos and (not window or key > pos - window):
                seen[at[i] + t, :, col] = True
                mine = got[at[i] + t, :, col]
                assert (torch.isnan(mine) if value != value else mine == value).all(), (i, t, col)
    assert seen.any() and not seen.all()
    assert torch.isfinite(got[~seen]).all()
    b.check(_patched(b, got, seen, window), "the rest", window=window)


@pytest.mark.parametrize("lens,news,window", [
    ([130, 64], [130, 64], 0), ([100, 300, 40], [100, 1, 40], 0), ([900, 800], [200, 150], 30),
])
@pytest.mark.parametrize("dtype,heads,kv_heads,dim", [(F16, 16, 8, 128), (BF16, 32, 8, 64)])
def test_attention_non_finite_values_of_a_chunks_first_tile(dtype, heads, kv_heads, dim, lens, news,
                                                            window):
    """Infinities among the very first values that a workgroup brings, in each wave's share
    of them, in chunks and in a batch with single tokens."""
    b = Batch(dtype, heads, kv_heads, dim, 16, lens, news, seed=31)
    got_at = np.concatenate([[0], np.cumsum(news)])
    seen = torch.zeros((sum(news), heads, dim), dtype=torch.bool, device=DEV)
    for i, (n, new) in enumerate(zip(lens, news)):
        low = max(n - new - window + 1, 0) if window else 0   # the first row's first key
        for j, key in enumerate(range(low + 1, min(low + 64, n), 17)):
            b.v_pages[int(b.table[i, key // 16]), key % 16, :, 7 + j] = float("inf")
            b.v[i][key, :, 7 + j] = 0
            for t in range(new):
                pos = n - new + t
                if key <= pos and (not window or key > pos - window):
                    seen[got_at[i] + t, :, 7 + j] = True
    got = b.call(window=window)
    assert seen.any() and not seen.all()
    assert (got[seen] == float("inf")).all()
    assert torch.isfinite(got[~seen]).all()
    b.check(_patched(b, got, seen, window), "the rest", window=window)


def _patched(b, got, seen, window):
    """`got` with the exact values in the marked places."""
    got, at = got.clone(), 0
    for i, (n, new) in enumerate(zip(b.lens, b.news)):
        want, _ = plain.attention(_np(b.q[at:at + new]), _np(b.k[i]), _np(b.v[i]), new, n,
                                  b.dim ** -0.5, window, U[b.dtype])
        want = torch.from_numpy(want).to(got)
        got[at:at + new] = torch.where(seen[at:at + new], want, got[at:at + new])
        at += new
    return got


def test_operators_refuse_tensors_that_need_gradients():
    """The operators have no backward pass: a graph is not cut without a word."""
    b = Batch(F16, 4, 2, 64, 16, [20], [1], seed=22)
    b.q.requires_grad_()
    with pytest.raises(ValueError, match="no gradient"):
        b.call()
    with torch.no_grad():
        b.check(b.call(), "without gradients")
    qkv, table, positions, _ = _heads_case(F16, 3, 2, 1, 64, 64, False, False)
    with pytest.raises(ValueError, match="no gradient"):
        lg.qk_norm_rotate(qkv.requires_grad_(), 2, 1, positions, table)
    y, x, a, w, ids, scales = _adapters_case(F16, 2, 64, 40, 8, 2, [0, 1])
    with pytest.raises(ValueError, match="no gradient"):
        lg.adapters_add(y, x, a.requires_grad_(), w, ids, scales)


@pytest.mark.parametrize("which", ["q_weight", "out", "scales", "k_pages"])
def test_operators_refuse_any_tensor_that_needs_gradients(which):
    b = Batch(F16, 4, 2, 64, 16, [20], [1], seed=25)
    qkv, table, positions, w = _heads_case(F16, 3, 2, 1, 64, 64, False, True)
    y, x, a, up, ids, scales = _adapters_case(F16, 2, 64, 40, 8, 2, [0, 1])
    with pytest.raises(ValueError, match="no gradient"):
        if which == "q_weight":
            lg.qk_norm_rotate(qkv, 2, 1, positions, table, w[0].requires_grad_(), w[1])
        elif which == "out":
            b.call(out=torch.zeros_like(b.q).requires_grad_())
        elif which == "scales":
            lg.adapters_add(y, x, a, up, ids, scales.requires_grad_())
        else:
            b.k_pages.requires_grad_()
            b.call()


def test_tensors_that_are_written_count_it():
    """Autograd tells by a tensor's version that a saved one was written over."""
    b = Batch(F16, 4, 2, 64, 16, [20], [1], seed=49)
    qkv, table, positions, _ = _heads_case(F16, 1, 4, 2, 64, 64, False, False)
    y, x, a, up, ids, s = _adapters_case(F16, 2, 64, 40, 8, 2, [0, 1])
    slots = torch.zeros(1, dtype=torch.int64, device=DEV)
    out = torch.zeros_like(b.q)
    w = torch.ones_like(out, requires_grad=True)
    saved = (w * out).sum()
    calls = [
        ((out,), lambda: b.call(out=out)),
        ((out, b.k_pages, b.v_pages),
         lambda: lg.qk_norm_rotate(qkv, 4, 2, positions, table, k_pages=b.k_pages, v_pages=b.v_pages,
                                   slots=slots, out=out)),
        ((y,), lambda: lg.adapters_add(y, x, a, up, ids, s, out=y)),
    ]
    for written, call in calls:
        before = [t._version for t in written]
        call()
        assert [t._version for t in written] == [v + 1 for v in before]
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        saved.backward()
    with torch.inference_mode():
        hidden = torch.zeros_like(out)
    lg.paged_attention(b.q, b.k_pages, b.v_pages, b.table, b.kv_lens, out=hidden)
    assert torch.equal(hidden, b.call())


def test_attention_padded_batch():
    """Rows behind the last sequence, in a batch much larger than its tokens, with the hints of
    a decode step, split and not."""
    for lens in ([3000, 40, 900], [50, 60, 20]):
        b = Batch(F16, 8, 2, 128, 16, lens, [1, 1, 1], seed=26, lead=5, tail=200)
        out = torch.full_like(b.q, 3.0)
        b.check(b.call(max_q=1, max_kv=3000, out=out), "padded")
        assert (out[:5] == 3).all() and (out[8:] == 3).all()


def test_outputs_that_overlap_are_refused():
    b = Batch(F16, 4, 2, 64, 16, [20, 20], [1, 1], seed=23)
    with pytest.raises(lg.LutGemmError):
        b.call(out=torch.zeros((1, 4, 64), dtype=F16, device=DEV).expand(2, 4, 64))
    with pytest.raises(lg.LutGemmError):
        b.call(out=torch.zeros((2, 1, 64), dtype=F16, device=DEV).expand(2, 4, 64))
    turned = torch.zeros((4, 2, 64), dtype=F16, device=DEV).transpose(0, 1)
    b.check(b.call(out=turned), "heads outside tokens")


def test_attention_output_in_place_of_the_queries():
    """`out` may be `q` itself, for single tokens, chunks, parts; it may not overlap it
    otherwise."""
    for lens, news in (([40, 3000], [1, 1]), ([300, 70], [130, 70]), ([3000], [20])):
        b = Batch(F16, 8, 2, 64, 16, lens, news, seed=47)
        want = b.call()
        fused = torch.zeros((len(b.q), 24, 64), dtype=F16, device=DEV)
        fused[:, 4:12] = b.q
        b.q = fused[:, 4:12]
        for out in (fused[:, 3:11], fused[:, 8:16], fused.view(-1)[256:256 + want.numel()].view_as(want)):
            with pytest.raises(lg.LutGemmError, match="SHAPE"):
                b.call(out=out)
        assert torch.equal(b.call(out=fused[:, 12:20]), want)
        assert torch.equal(b.call(out=b.q), want)
        assert (fused[:, :4] == 0).all() and (fused[:, 20:] == 0).all()


def test_attention_far_pages():
    """Pages more than 2^32 bytes, and 2^31 elements, into the cache."""
    pages = (1 << 31) // (64 * 8 * 128) + 40
    k = torch.zeros((pages, 64, 8, 128), dtype=F16, device=DEV)
    v = torch.zeros((pages, 64, 8, 128), dtype=F16, device=DEV)
    assert k.numel() > 1 << 31
    b = Batch(F16, 16, 8, 128, 64, [200, 130], [1, 30], seed=13)
    far = {}
    for i in range(2):
        for j in range(-(-b.lens[i] // 64)):
            near = int(b.table[i, j])
            far[near] = pages - 1 - near
            k[far[near]], v[far[near]] = b.k_pages[near], b.v_pages[near]
            b.table[i, j] = far[near]
    b.k_pages, b.v_pages = k, v
    b.check(b.call(), "far pages")


def test_attention_repeats_and_graphs():
    """The same bits from every call, from two captured graphs replayed in turn and at
    once on two streams, with eager work between."""
    b = Batch(F16, 16, 2, 128, 16, [2000, 30, 900], [1, 1, 1], seed=14)
    c = Batch(BF16, 8, 2, 128, 32, [1500, 700], [33, 2], seed=15)
    want_b, want_c = b.call(max_q=1), c.call()
    assert torch.equal(want_b, b.call(max_q=1)) and torch.equal(want_c, c.call())
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for batch, kw in ((b, dict(max_q=1)), (c, {})):
        out = torch.zeros_like(batch.q)
        with torch.cuda.stream(side):
            batch.call(out=out, **kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            batch.call(out=out, **kw)
        graphs.append((g, out))
    other = torch.cuda.Stream()
    for r in range(4):
        for _, out in graphs:
            out.fill_(3)
        junk = torch.randn(1 << 16, device=DEV).sum()
        torch.cuda.synchronize()
        if r % 2:
            graphs[0][0].replay()
            with torch.cuda.stream(other):
                graphs[1][0].replay()
        else:
            graphs[1][0].replay()
            graphs[0][0].replay()
        torch.cuda.synchronize()
        assert torch.equal(graphs[0][1], want_b) and torch.equal(graphs[1][1], want_c), r
        assert torch.isfinite(junk)


def test_attention_nothing_to_do():
    b = Batch(F16, 4, 2, 64, 16, [10], [1], seed=16)
    empty = lg.paged_attention(b.q[:0], b.k_pages, b.v_pages, b.table[:0], b.kv_lens[:0])
    assert empty.shape == (0, 4, 64)
    none = torch.zeros(2, dtype=torch.int32, device=DEV)
    out = torch.full_like(b.q, 9.0)
    lg.paged_attention(b.q, b.k_pages, b.v_pages, b.table, b.kv_lens, none, out=out)
    torch.cuda.synchronize()
    assert (out == 9).all()


# ------------------------------------------------- norms, rotation, cache append

def _heads_case(dtype, tokens, heads, kv, dim, rotary, interleaved, norm, seed=0, limit=1000):
    qkv = _normal((tokens, (heads + 2 * kv) * dim), dtype, seed)
    table = lg.rotary_table(limit, rotary, device=DEV) if rotary else None
    g = torch.Generator().manual_seed(seed + 1)
    positions = torch.randint(limit, (tokens,), generator=g).to(DEV)
    w = [_normal((dim,), dtype, seed + 2 + i) for i in range(2)] if norm else [None, None]
    return qkv, table, positions, w


def _heads_want(qkv, table, positions, w, heads, kv, dim, interleaved, eps, u):
    x = _np(qkv).reshape(qkv.shape[0], heads + 2 * kv, dim)
    t = _np(table)[positions.cpu().numpy()] if table is not None else np.zeros((len(x), 0))
    c, s = t[:, :t.shape[1] // 2], t[:, t.shape[1] // 2:]
    return [plain.heads(part, None if wt is None else _np(wt), eps, c, s, interleaved, u)
            for part, wt in ((x[:, :heads], w[0]), (x[:, heads:heads + kv], w[1]))] \
        + [x[:, heads + kv:]]


@pytest.mark.parametrize("heads,kv,dim,rotary", [(4, 2, 128, 128), (3, 1, 64, 32), (5, 5, 96, 96),
                                                 (1, 1, 16, 16), (2, 2, 256, 64), (7, 1, 80, 0),
                                                 (40, 8, 128, 64)])
@pytest.mark.parametrize("dtype,interleaved,norm", [(F16, False, True), (BF16, True, True),
                                                    (F16, True, False), (BF16, False, False)])
@pytest.mark.parametrize("tokens", [1, 37])
def test_heads_into_the_cache(dtype, interleaved, norm, heads, kv, dim, rotary, tokens):
    qkv, table, positions, w = _heads_case(dtype, tokens, heads, kv, dim, rotary, interleaved, norm,
                                           seed=heads + dim)
    pages, page = 6, 8
    k_pages = torch.full((pages, page, kv, dim), 7.0, dtype=dtype, device=DEV)
    v_pages = torch.full((pages, kv, page, dim), 7.0, dtype=dtype, device=DEV).transpose(1, 2)
    slots = torch.from_numpy(np.random.default_rng(1).permutation(pages * page)[:tokens].copy()).to(DEV)
    if tokens > 4:
        slots[3], slots[4] = -1, pages * page
    q = lg.qk_norm_rotate(qkv, heads, kv, positions, table, *w, eps=1e-5, interleaved=interleaved,
                          k_pages=k_pages, v_pages=v_pages, slots=slots)
    (qw, qb), (kw, kb), vw = _heads_want(qkv, table, positions, w, heads, kv, dim, interleaved,
                                         1e-5, U[dtype])
    _inside(q, qw, qb, "queries")
    used = np.zeros(pages * page, bool)
    for t, slot in enumerate(slots.tolist()):
        if 0 <= slot < pages * page:
            used[slot] = True
            _inside(k_pages[slot // page, slot % page], kw[t], kb[t], f"key {t}") if t < 3 else None
            assert np.abs(_np(k_pages[slot // page, slot % page]) - kw[t]).max() <= kb[t].max()
            assert np.array_equal(_np(v_pages[slot // page, slot % page]), vw[t])
    for slot in np.flatnonzero(~used):
        assert (k_pages[slot // page, slot % page] == 7).all()
        assert (v_pages[slot // page, slot % page] == 7).all()


def test_heads_without_a_cache_and_in_place():
    qkv, table, positions, w = _heads_case(F16, 50, 6, 2, 128, 128, False, True, seed=20)
    (qw, qb), (kw, kb), _ = _heads_want(qkv, table, positions, w, 6, 2, 128, False, 1e-6, U[F16])
    q, k = lg.qk_norm_rotate(qkv, 6, 2, positions, table, *w)
    _inside(q, qw, qb, "queries")
    _inside(k, kw, kb, "keys")
    # a fused row with room on both sides, the queries written over themselves
    wide = torch.full((50, 10 * 128 + 64), 3.0, dtype=F16, device=DEV)
    inner = wide[:, 32:32 + 10 * 128]
    inner.copy_(qkv)
    out = inner[:, :6 * 128].unflatten(1, (6, 128))
    q2, k2 = lg.qk_norm_rotate(inner, 6, 2, positions, table, *w, out=out)
    assert torch.equal(q2, q) and torch.equal(k2, k) and q2.data_ptr() == inner.data_ptr()
    assert torch.equal(inner[:, 6 * 128:], qkv[:, 6 * 128:])
    assert (wide[:, :32] == 3).all() and (wide[:, -32:] == 3).all()


def test_heads_positions_outside_the_table():
    qkv, table, positions, _ = _heads_case(F16, 6, 2, 1, 64, 32, False, False, seed=21)
    positions[1], positions[4] = -1, 1000
    q, k = lg.qk_norm_rotate(qkv, 2, 1, positions, table)
    for t in range(6):
        assert torch.isnan(q[t, :, :32]).all() == (t in (1, 4))
        assert torch.isfinite(q[t, :, 32:]).all()
        assert torch.isnan(k[t, :, :32]).all() == (t in (1, 4))


def test_heads_many_tokens_and_tiny_values():
    """A workgroup that walks all heads, and rows of zeros and of the smallest numbers."""
    qkv, table, positions, w = _heads_case(BF16, 3000, 20, 4, 64, 64, True, True, seed=22)
    qkv[7] = 0
    qkv[8] = 1e-30
    q, k = lg.qk_norm_rotate(qkv, 20, 4, positions, table, *w, interleaved=True)
    (qw, qb), (kw, kb), _ = _heads_want(qkv, table, positions, w, 20, 4, 64, True, 1e-6, U[BF16])
    _inside(q, qw, qb, "queries")
    _inside(k, kw, kb, "keys")


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_heads_larger_than_the_caches(dtype):
    """More than 32 MB of heads, in place and into the cache."""
    heads, kv, dim, tokens = 64, 8, 128, 1700
    qkv, table, positions, w = _heads_case(dtype, tokens, heads, kv, dim, dim, False, True, seed=41)
    k_pages = torch.zeros((107, 16, kv, dim), dtype=dtype, device=DEV)
    v_pages = torch.zeros_like(k_pages)
    slots = torch.arange(tokens, device=DEV).flip(0).contiguous()
    some = torch.tensor([0, 1, 255, 256, 1024, tokens - 1], device=DEV)
    (qw, qb), (kw, kb), vw = _heads_want(qkv[some], table, positions[some], w, heads, kv, dim, False,
                                         1e-6, U[dtype])
    out = qkv[:, :heads * dim].unflatten(1, (heads, dim))
    q = lg.qk_norm_rotate(qkv, heads, kv, positions, table, *w, k_pages=k_pages, v_pages=v_pages,
                          slots=slots, out=out)
    _inside(q[some], qw, qb, "queries")
    _inside(k_pages.reshape(-1, kv, dim)[slots[some]], kw, kb, "keys")
    assert np.array_equal(_np(v_pages.reshape(-1, kv, dim)[slots[some]]), vw)


@pytest.mark.parametrize("eps", [0.0, 1e-40])
def test_heads_mean_squares_below_the_normal_numbers(eps):
    """Squares of about 1e-39, and heads of zeros beside an epsilon below 2^-126."""
    qkv, table, positions, w = _heads_case(BF16, 9, 4, 2, 128, 64, False, True, seed=45)
    qkv = (qkv.float() * 3e-20).to(BF16)
    if eps:
        qkv[4] = 0
    q, k = lg.qk_norm_rotate(qkv, 4, 2, positions, table, *w, eps=eps)
    eps = float(np.float32(eps))
    (qw, qb), (kw, kb), _ = _heads_want(qkv, table, positions, w, 4, 2, 128, False, eps, U[BF16])
    _inside(q, qw, qb, "queries")
    _inside(k, kw, kb, "keys")


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("tokens", [3, 1700])
def test_heads_of_zeros_with_a_tiny_epsilon(dtype, tokens):
    """0 / sqrt(1e-40) is zero, in launches of both sizes; other heads have their norm."""
    qkv, table, positions, w = _heads_case(dtype, tokens, 64, 8, 128, 128, True, True, seed=47)
    qkv[1] = 0
    q, k = lg.qk_norm_rotate(qkv, 64, 8, positions, table, *w, eps=1e-40, interleaved=True)
    assert (q[1] == 0).all() and (k[1] == 0).all()
    (qw, qb), (kw, kb), _ = _heads_want(qkv[:3], table, positions[:3], w, 64, 8, 128, True,
                                        float(np.float32(1e-40)), U[dtype])
    _inside(q[:3], qw, qb, "queries")
    _inside(k[:3], kw, kb, "keys")


def test_heads_outputs_over_other_parts_of_qkv_are_refused():
    qkv, table, positions, _ = _heads_case(F16, 6, 2, 1, 64, 64, False, False, seed=46)
    before = qkv.clone()
    heads = qkv.view(6, 4, 64)
    for out in (heads[:, 1:3], heads[:, 2:4], qkv.view(-1)[:6 * 128].view(6, 2, 64)):
        with pytest.raises(lg.LutGemmError, match="SHAPE"):
            lg.qk_norm_rotate(qkv, 2, 1, positions, table, out=out)
    assert torch.equal(qkv, before)
    want, _ = lg.qk_norm_rotate(qkv, 2, 1, positions, table)
    wide = torch.zeros((6, 6, 64), dtype=F16, device=DEV)   # the queries beside qkv's own rows
    wide[:, 2:] = heads
    inner = wide.view(6, -1)[:, 128:]
    got, _ = lg.qk_norm_rotate(inner, 2, 1, positions, table, out=wide[:, :2])
    assert torch.equal(got, want) and torch.equal(wide[:, 2:], heads)


def test_rotary_table_is_rounded_from_64_bits():
    t = lg.rotary_table(70000, 64, 10000.0, device="cpu").double().numpy()
    p = np.arange(70000)[:, None] * 10000.0 ** (-np.arange(0, 64, 2) / 64)
    assert np.abs(t - np.concatenate([np.cos(p), np.sin(p)], 1)).max() <= 2.0 ** -24


# ------------------------------------------------------------- low-rank adapters

def _adapters_case(dtype, rows, K, N, rank, count, ids, seed=0):
    x, y = _normal((rows, K), dtype, seed), _normal((rows, N), dtype, seed + 1)
    a = _normal((count, rank, K), dtype, seed + 2, max(K, 1) ** -0.5)
    b = _normal((count, N, rank), dtype, seed + 3, rank ** -0.5)
    scales = torch.linspace(0.5, 2.0, max(count, 1))[:count].to(DEV)
    return y, x, a, b, torch.tensor(ids, dtype=torch.int32, device=DEV), scales


def _adapters_check(got, y, x, a, b, ids, scales, what):
    pair = {F16: 2.0 ** -21, BF16: 2.0 ** -16}[x.dtype]
    want, bound = plain.adapters(_np(y), _np(x), _np(a), _np(b), ids.tolist(),
                                 None if scales is None else _np(scales), U[x.dtype], pair)
    _inside(got, want, bound, what)
    for i, l in enumerate(ids.tolist()):
        if not 0 <= l < a.shape[0]:
            assert torch.equal(got[i], y[i])


def _ids(rows, count, seed, none=0.2):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, max(count, 1), rows)
    ids[rng.random(rows) < none] = rng.choice([-1, count, -2 ** 31, 2 ** 31 - 1])
    return ids.tolist()


@pytest.mark.parametrize("rows,count", [(1, 1), (1, 3), (16, 1), (17, 1), (17, 5), (64, 3), (64, 64),
                                        (65, 1), (65, 70), (200, 4)])
@pytest.mark.parametrize("dtype,K,N,rank", [(F16, 520, 260, 16), (BF16, 1032, 129, 8),
                                            (F16, 8, 5, 40), (BF16, 2056, 640, 128)])
def test_adapters(dtype, K, N, rank, rows, count):
    """Every grouping (one row to a lane, sorted above 64 rows), odd and narrow sizes."""
    case = _adapters_case(dtype, rows, K, N, rank, count, _ids(rows, count, rows + count), seed=rows)
    got = lg.adapters_add(*case)
    _adapters_check(got, *case, f"{rows} rows, {count} adapters, {K}->{N}, rank {rank}")
    assert torch.equal(got, lg.adapters_add(*case))   # the same bits again


@pytest.mark.parametrize("rows,count", [(65, 255), (65, 256), (300, 255), (300, 256), (257, 1),
                                        (1025, 40), (4095, 7), (4096, 255), (4097, 7)])
@pytest.mark.parametrize("order", ["mixed", "runs", "one", "none"])
def test_adapters_of_many_rows(rows, count, order):
    """Rows grouped by each workgroup and by a launch of its own: numbers of rows and adapters
    on both sides of the limits, ids in any order, all alike and all outside."""
    ids = _ids(rows, count, rows + count)
    ids = {"mixed": ids, "runs": sorted(ids), "one": [count - 1] * rows, "none": [-1] * rows}[order]
    case = _adapters_case(F16, rows, 64, 40, 8, count, ids, seed=rows)
    got = lg.adapters_add(*case)
    _adapters_check(got, *case, f"{rows} rows, {count} adapters, {order}")
    assert torch.equal(got, lg.adapters_add(*case))


def test_adapters_rows_do_not_depend_on_others():
    """A row alone, in a full batch and in a sorted batch gives the same bits when the
    work is split alike, and the same value in any case."""
    ids = _ids(130, 7, 1)
    y, x, a, b, d_ids, s = _adapters_case(F16, 130, 512, 200, 16, 7, ids, seed=30)
    whole = lg.adapters_add(y, x, a, b, d_ids, s)
    for i in (0, 5, 129):
        one = lg.adapters_add(y[i:i + 1], x[i:i + 1], a, b, d_ids[i:i + 1].contiguous(), s)
        assert torch.equal(one[0], whole[i])


def test_adapters_in_place_strided_and_plain_scales():
    ids = _ids(40, 3, 2)
    y, x, a, b, d_ids, s = _adapters_case(F16, 40, 256, 136, 24, 3, ids, seed=31)
    wide_x = _normal((40, 300 + 4), F16, 32)
    wide_x[:, 16:272] = x
    wide_y = torch.full((40, 150), 2.0, dtype=F16, device=DEV)
    wide_y[:, 3:139] = y
    part = wide_y[:, 3:139]
    got = lg.adapters_add(part, wide_x[:, 16:272], a, b, d_ids, None, out=part)
    assert got is part
    _adapters_check(got, y, x, a, b, d_ids, None, "in place, odd offsets")
    assert (wide_y[:, :3] == 2).all() and (wide_y[:, 139:] == 2).all()
    y2 = y.clone()
    lg.adapters_add(y2, x, a, b, d_ids, s, out=y2)
    assert torch.equal(y2, lg.adapters_add(y, x, a, b, d_ids, s))


def test_adapters_large_and_tiny_inner_values():
    """Inner values past fp16's range and below its normal numbers."""
    for scale, back in ((300.0, 1e-4), (1e-4, 100.0)):
        y, x, a, b, ids, s = _adapters_case(F16, 9, 1024, 64, 16, 2, [0, 1] * 4 + [0], seed=33)
        x = (x.float() * scale).to(F16)
        a = (a.float() * min(scale, 30.0)).to(F16)
        s = s * (back / scale / 30)
        got = lg.adapters_add(y, x, a, b, ids, s)
        _adapters_check(got, y, x, a, b, ids, s, f"inner values scaled by {scale}")


def test_adapters_nothing_to_add():
    y, x, a, b, ids, s = _adapters_case(F16, 70, 64, 32, 8, 2, [-1] * 70, seed=34)
    assert torch.equal(lg.adapters_add(y, x, a, b, ids, s), y)
    none = lg.adapters_add(y, x, a[:0], b[:0], ids, s[:0])
    assert torch.equal(none, y)
    assert lg.adapters_add(y[:0], x[:0], a, b, ids[:0], s).shape == (0, 32)
    flat = lg.adapters_add(y, x[:, :0], a[:, :, :0].contiguous(), b, torch.zeros_like(ids), s)
    assert torch.equal(flat, y)


def test_adapters_of_no_inputs():
    """K = 0, of a tensor of its own: its rows have a stride of one."""
    y, x, a, b, ids, s = _adapters_case(F16, 33, 0, 40, 8, 2, [0] * 33, seed=36)
    assert x.stride(0) == 1
    assert torch.equal(lg.adapters_add(y, x, a, b, ids, s), y)


@pytest.mark.parametrize("rows", [5, 40, 200])
def test_adapters_outputs_over_their_inputs_are_refused(rows):
    """K = N: `out` may be y, not x, and no other rows of either."""
    y, x, a, b, ids, s = _adapters_case(F16, rows, 512, 512, 16, 3, _ids(rows, 3, 5), seed=48)
    want = lg.adapters_add(y, x, a, b, ids, s)
    wide = torch.zeros((rows + 1, 3 * 512), dtype=F16, device=DEV)
    wide[:rows, :512], wide[:rows, 512:1024] = x, y
    x, y = wide[:rows, :512], wide[:rows, 512:1024]
    for out in (x, wide[:rows, 8:520], wide[:rows, 600:1112], wide[1:, 512:1024], wide[1:, :512],
                wide.view(-1)[64:64 + rows * 512].view(rows, 512)):
        with pytest.raises(lg.LutGemmError, match="SHAPE"):
            lg.adapters_add(y, x, a, b, ids, s, out=out)
    assert torch.equal(lg.adapters_add(y, x, a, b, ids, s, out=wide[:rows, 1024:]), want)
    assert torch.equal(lg.adapters_add(y, x, a, b, ids, s, out=y), want)


@pytest.mark.parametrize("rows,count", [(1100, 5), (1500, 300), (130, 260)])
@pytest.mark.parametrize("dtype,K,N,rank", [(BF16, 2056, 129, 128), (F16, 1544, 333, 40),
                                            (BF16, 4104, 256, 64), (F16, 520, 72, 24)])
def test_adapters_of_sorted_rows(dtype, K, N, rank, rows, count):
    """Rows sorted by a launch of its own, with wide ranks, K in several parts and odd N."""
    case = _adapters_case(dtype, rows, K, N, rank, count, _ids(rows, count, rows + count), seed=rows)
    got = lg.adapters_add(*case)
    _adapters_check(got, *case, f"{rows} rows, {count} adapters, {K}->{N}, rank {rank}")
    assert torch.equal(got, lg.adapters_add(*case))


def test_adapters_graph_and_streams():
    case = _adapters_case(BF16, 100, 1024, 512, 32, 9, _ids(100, 9, 3), seed=35)
    want = lg.adapters_add(*case)
    outs = [torch.zeros_like(want) for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for out in outs:
        with torch.cuda.stream(side):
            lg.adapters_add(*case, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lg.adapters_add(*case, out=out)
        graphs.append(g)
    other = torch.cuda.Stream()
    for r in range(3):
        for out in outs:
            out.fill_(0)
        torch.randn(1 << 16, device=DEV).sum()
        torch.cuda.synchronize()
        graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want), r


# ------------------------------------------------------------------ used together

def test_packed_product_with_adapters():
    """PackedBCQ's product with its rows' adapters is the product, then the adapters."""
    import workloads
    w = workloads.random_bcq(528, 1024, 3, 128, m=5, seed=40, sigma=0.02)
    pw = lg.PackedBCQ.from_bcq(w.bits, w.alpha, None, w.g, device=DEV)
    x = torch.from_numpy(w.x).to(DEV)
    _, _, a, b, ids, s = _adapters_case(F16, 5, 1024, 528, 16, 3, [2, -1, 0, 2, 1], seed=41)
    y = pw(x)
    got = pw(x, adapters=(a, b, s), ids=ids)
    assert torch.equal(got, lg.adapters_add(y, x, a, b, ids, s))
    assert torch.equal(got[1], y[1]) and not torch.equal(got[0], y[0])


@pytest.mark.parametrize("norm", [False, True])
def test_a_prompt_in_chunks_then_tokens(norm):
    """Two requests through projection, adapters, norms, rotation, cache and attention,
    their prompts in chunks and then token by token: each step's attention is that of
    the fp64 form on the cache as it stands."""
    import workloads
    heads, kv, dim, page, K = 4, 2, 64, 16, 256
    N = (heads + 2 * kv) * dim
    w = workloads.random_bcq(N, K, 3, 128, seed=50, sigma=0.06)
    pw = lg.PackedBCQ.from_bcq(w.bits, w.alpha, None, w.g, device=DEV)
    _, _, a, b, _, s = _adapters_case(F16, 1, K, N, 16, 2, [0], seed=51)
    weights = [_normal((dim,), F16, 52), _normal((dim,), F16, 53)] if norm else [None, None]
    rope = lg.rotary_table(256, dim, device=DEV)
    k_pages = torch.full((12, page, kv, dim), NAN, dtype=F16, device=DEV)
    v_pages = torch.full((12, page, kv, dim), NAN, dtype=F16, device=DEV)
    table = torch.tensor([[3, 9, 1, 7, 0], [2, 11, 5, 8, 10]], dtype=torch.int32, device=DEV)
    have = [0, 0]
    for step, news in enumerate([(40, 19), (11, 1), (1, 1), (1, 1)]):
        req = np.repeat([0, 1], news)
        pos = np.concatenate([np.arange(h, h + n) for h, n in zip(have, news)])
        have = [h + n for h, n in zip(have, news)]
        x = _normal((len(req), K), F16, 60 + step)
        ids = torch.tensor(np.where(req == 0, 1, -1), dtype=torch.int32, device=DEV)
        qkv = pw(x, adapters=(a, b, s), ids=ids)
        d_req, d_pos = torch.from_numpy(req).to(DEV), torch.from_numpy(pos).to(DEV)
        slots = table[d_req, d_pos // page].long() * page + d_pos % page
        q = lg.qk_norm_rotate(qkv, heads, kv, d_pos, rope, *weights, k_pages=k_pages,
                              v_pages=v_pages, slots=slots)
        starts = torch.tensor([0, news[0], sum(news)], dtype=torch.int32, device=DEV)
        lens = torch.tensor(have, dtype=torch.int32, device=DEV)
        o = lg.paged_attention(q, k_pages, v_pages, table, lens, starts, max_q=max(news))
        for r in range(2):
            rows = slice(int(starts[r]), int(starts[r + 1]))
            ks, vs = (t[table[r].long()].flatten(0, 1)[:have[r]] for t in (k_pages, v_pages))
            want, bound = plain.attention(_np(q[rows]), _np(ks), _np(vs), news[r], have[r],
                                          dim ** -0.5, 0, U[F16])
            _inside(o[rows], want, bound, f"step {step} request {r}")


@pytest.mark.parametrize("model,adapters", [("llama7b", 0), ("llama7b", 2)])
def test_decode_stack_with_a_cache(model, adapters):
    """A decode step with attention (and adapters): each layer's attention is that of the
    fp64 form on its cache as the step left it, every captured replay equals the
    eager step, and the products without them are the driver's own as before."""
    from lut_gemv_amd import decode
    st = decode.DecodeStack(model, layers=2, q=2, g=128, m=3, device=DEV, context=150, page_size=32,
                            adapters=adapters)
    eager = st.token().clone()
    torch.cuda.synchronize()
    assert torch.isfinite(eager).all()
    heads = st.heads
    for layer in (0, 1):
        st.token()
        k_pages, v_pages = st.caches[layer]
        if layer == 1:   # the last layer's queries and output are the ones that are left
            for i in range(st.m):
                rows = st.page_table[i].long()
                ks, vs = (t[rows].flatten(0, 1)[:151] for t in (k_pages, v_pages))
                want, bound = plain.attention(_np(st.queries[i:i + 1]), _np(ks), _np(vs), 1, 151,
                                              128 ** -0.5, 0, U[F16])
                _inside(st.attended.view(3, heads, 128)[i:i + 1], want, bound, f"sequence {i}")
                qkv = _np(st.outs["qkv"][i]).reshape(3 * heads, 128)
                assert np.array_equal(_np(vs[150]), qkv[2 * heads:])
                angle = _np(st.rotary[150])
                want, bound = plain.heads(qkv[None, heads:2 * heads], None, 0.0, angle[None, :64],
                                          angle[None, 64:], False, U[F16])
                _inside(ks[150:151], want, bound, f"key of sequence {i}")
    g = st.capture()
    for r in range(3):
        st.outs[st.out_name].fill_(0)
        torch.randn(1 << 16, device=DEV).sum()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(st.outs[st.out_name], eager), f"replay {r}"


def test_decode_stack_adds_the_adapters_of_every_projection():
    """Each projection's output in a step is its product and then its adapters, those of
    sequence i being adapter i modulo their number."""
    from lut_gemv_amd import decode
    st = decode.DecodeStack("llama7b", layers=1, q=2, g=128, m=3, device=DEV, context=70, page_size=16,
                            adapters=2, rank=8)
    st.token()
    torch.cuda.synchronize()
    for p in st.projs:
        src = st._src(p, st.x).contiguous()
        product = st.weights[0][p.name](src)
        a, b = st.lora[0][p.name]
        assert not torch.equal(st.outs[p.name], product)
        cols = torch.arange(0, p.N, 37, device=DEV)
        want, bound = plain.adapters(_np(product[:, cols]), _np(src), _np(a), _np(b[:, cols]), [0, 1, 0],
                                     None, U[F16], 2.0 ** -21)
        _inside(st.outs[p.name][:, cols], want, bound, p.name)


def test_decode_stack_attends_in_every_layer(monkeypatch):
    """Each layer's queries, keys and attention are those of its own QKV output and cache."""
    from lut_gemv_amd import decode
    st = decode.DecodeStack("llama7b", layers=2, q=2, g=128, m=2, device=DEV, context=90, page_size=16)
    left, attend = [], st._attend

    def noted(layer):
        attend(layer)
        left.append([st.outs["qkv"].clone(), st.queries.clone(), st.attended.clone()])

    monkeypatch.setattr(st, "_attend", noted)
    st.token()
    assert len(left) == 2 and not torch.equal(left[0][2], left[1][2])
    angle = _np(st.rotary[90])[None].repeat(2, 0)
    for layer, (qkv, queries, attended) in enumerate(left):
        x = _np(qkv).reshape(2, 3 * st.heads, 128)
        want, bound = plain.heads(x[:, :st.heads], None, 0.0, angle[:, :64], angle[:, 64:], False, U[F16])
        _inside(queries, want, bound, f"queries of layer {layer}")
        k_pages, v_pages = st.caches[layer]
        for i in range(2):
            ks, vs = (t[st.page_table[i].long()].flatten(0, 1)[:91] for t in (k_pages, v_pages))
            assert np.array_equal(_np(vs[90]), x[i, 2 * st.heads:])
            want, bound = plain.attention(_np(queries[i:i + 1]), _np(ks), _np(vs), 1, 91, 128 ** -0.5, 0,
                                          U[F16])
            _inside(attended.view(2, st.heads, 128)[i:i + 1], want, bound, f"layer {layer} sequence {i}")


@pytest.mark.parametrize("extra", [{}, dict(context=100, adapters=3, rank=8)])
def test_decode_rate_counts_all_that_a_step_reads(extra):
    from lut_gemv_amd import decode
    st = decode.DecodeStack("llama7b", layers=1, q=2, g=128, m=2, device=DEV, page_size=16, **extra)
    read = st.bytes_per_step()
    if extra:
        entries = sum(p.K + p.N for p in st.projs)
        read += 2 * 101 * 2 * 4096 * 2 + 2 * 2 * 8 * entries   # two sequences, two of three adapters
    r = st.time_tokens(tokens=2, warmup=1)
    assert r["GBps"] == pytest.approx(read / (r["ms_per_step"] * 1e-3) / 1e9, rel=1e-9)
