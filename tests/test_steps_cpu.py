"""The operators around a serving step, host side: every argument error is reported before
any HIP call, the descriptors' layout is the header's, and the plain forms agree with
torch. No GPU."""
import ctypes
import os
import shutil
import struct
import subprocess

import numpy as np
import pytest

import lut_gemv_amd as lg
from oracle import serving as plain

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000     # a fake, aligned device address: never dereferenced
FAR = 1 << 32    # between arrays that must lie apart
NULL, SHAPE, VALUE, BUFFER, ALIGN = 1, 2, 3, 4, 5
# the header's descriptors
_SHARED = struct.Struct("@8ifi15q2i2q")
_TABLES = struct.Struct("@4i2q")
_SAMPLE = struct.Struct("@4iq")

SHARED = dict(type=0, heads=8, kv_heads=2, head_dim=128, page_size=16, seqs=3, table_width=10, window=0,
              scale=0.1, reserved=0, tokens=30, pages=20, table_stride=10, max_q=10, max_kv=160,
              q_token=1024, q_head=128, o_token=1024, o_head=128, k_page=4096, k_slot=256, k_head=128,
              v_page=4096, v_slot=256, v_head=128, groups=2, prefix_width=8, prefix_stride=8, max_prefix=128)


def _shared(ws=A, wsb=1 << 40, q=A, k=A, v=A, ptable=A, plens=A, gstarts=A, table=A, lens=A, starts=A, out=A,
            **change):
    d = _SHARED.pack(*{**SHARED, **change}.values())
    return lg.lib().lutgemm_shared_attention(d, q, k, v, ptable, plens, gstarts, table, lens, starts, out, ws,
                                             wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(type=2), SHAPE), (dict(head_dim=96), SHAPE), (dict(heads=7), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(seqs=-1), SHAPE), (dict(seqs=1 << 20), SHAPE),
    (dict(tokens=-1), SHAPE), (dict(table_width=0), SHAPE), (dict(pages=0), SHAPE), (dict(window=5), SHAPE),
    (dict(window=-1), SHAPE), (dict(scale=0.0), VALUE), (dict(scale=float("nan")), VALUE),
    (dict(q_token=1020), SHAPE), (dict(o_head=64), SHAPE), (dict(k_slot=1 << 24), SHAPE),
    (dict(groups=-1), SHAPE), (dict(groups=1 << 20), SHAPE), (dict(prefix_width=0), SHAPE),
    (dict(prefix_width=1 << 27), SHAPE), (dict(prefix_stride=-1), SHAPE), (dict(prefix_stride=1 << 40), SHAPE),
    (dict(max_prefix=-1), SHAPE), (dict(max_q=-1), SHAPE), (dict(max_kv=-1), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(ptable=None), NULL), (dict(plens=None), NULL),
    (dict(ws=None), NULL), (dict(wsb=100), BUFFER), (dict(ws=A + 8), ALIGN), (dict(q=A + 8), ALIGN),
    (dict(k=A + 2), ALIGN), (dict(out=A + 8), ALIGN), (dict(ptable=A + 2), ALIGN), (dict(plens=A + 1), ALIGN),
    (dict(gstarts=A + 2), ALIGN), (dict(table=A + 2), ALIGN), (dict(lens=A + 1), ALIGN),
    (dict(starts=A + 2), ALIGN), (dict(starts=None), SHAPE), (dict(gstarts=None), SHAPE),
    (dict(tokens=1 << 23, heads=1024, kv_heads=1024), SHAPE),
])
def test_shared_refusals(change, status):
    assert _shared(**change) == status


def _shared_workspace(**change):
    n = ctypes.c_size_t(7)
    d = _SHARED.pack(*{**SHARED, **change}.values())
    st = lg.lib().lutgemm_shared_attention_workspace(d, ctypes.byref(n))
    return st, n.value


def test_shared_workspace_and_empty_calls():
    assert _shared_workspace(type=3)[0] == SHAPE
    assert lg.lib().lutgemm_shared_attention_workspace(_SHARED.pack(*SHARED.values()), None) == NULL
    assert lg.lib().lutgemm_shared_attention_workspace(None, None) == NULL
    assert _shared_workspace(tokens=0) == (0, 0) and _shared_workspace(seqs=0) == (0, 0)
    assert _shared(tokens=0, q=None) == 0 and _shared(seqs=0, tokens=0, starts=None) == 0
    # a part of the prefix and one of the own keys for each row, of 128 sums and two numbers more
    for change in (dict(), dict(groups=0), dict(max_kv=1, max_q=1, max_prefix=1)):
        st, n = _shared_workspace(**change)
        assert st == 0 and n >= 30 * 8 * 130 * 4 and n % (30 * 8 * 130 * 4) == 0
    # parts of a long prefix are no more than the launch has use for
    st, n = _shared_workspace(seqs=64, tokens=64, max_prefix=1 << 20, prefix_width=1 << 16, max_q=1)
    assert st == 0 and n <= 300 * 64 * 8 * 130 * 4


TABLES = dict(seqs=3, page_size=16, table_width=10, capacity=50, tokens=20, table_stride=10)


def _tables(wsb=1 << 30, **change):
    at = dict(change=A, lens=A + FAR, offsets=A + 2 * FAR, table=A + 3 * FAR, ring=A + 4 * FAR, range=A + 5 * FAR,
              positions=A + 6 * FAR, slots=A + 7 * FAR, lens_out=A + 8 * FAR, starts=A + 9 * FAR,
              range_out=A + 10 * FAR, ws=A + 11 * FAR)
    d = _TABLES.pack(*[change.get(k, v) for k, v in TABLES.items()])
    at.update({k: v for k, v in change.items() if k in at})
    return lg.lib().lutgemm_batch_tables(d, *at.values(), wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(seqs=-1), SHAPE), (dict(seqs=1 << 20), SHAPE), (dict(page_size=0), SHAPE), (dict(page_size=65537), SHAPE),
    (dict(table_width=0), SHAPE), (dict(table_width=1 << 27, table_stride=1 << 27), SHAPE), (dict(capacity=-1), SHAPE),
    (dict(capacity=1 << 29), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 24), SHAPE),
    (dict(table_stride=9), SHAPE), (dict(table_stride=1 << 40), SHAPE),
    (dict(change=None), NULL), (dict(lens=None), NULL), (dict(table=None), NULL), (dict(ring=None), NULL),
    (dict(range=None), NULL), (dict(range_out=None), NULL), (dict(positions=None), NULL), (dict(slots=None), NULL),
    (dict(lens_out=None), NULL), (dict(starts=None), NULL), (dict(tokens=9999, ws=None), NULL),
    (dict(tokens=9999, wsb=23), BUFFER),
    (dict(change=A + 2), ALIGN), (dict(positions=A + 6 * FAR + 4), ALIGN), (dict(slots=A + 7 * FAR + 4), ALIGN),
    (dict(ring=A + 4 * FAR + 1), ALIGN), (dict(offsets=A + 2), ALIGN), (dict(ws=A + 2), ALIGN),
    (dict(slots=A + 6 * FAR + 152), SHAPE), (dict(lens_out=A + FAR + 4), SHAPE), (dict(starts=A + 4), SHAPE),
    (dict(range_out=A + 5 * FAR + 4), SHAPE), (dict(ring=A + 2 * FAR - 196), SHAPE), (dict(tokens=9999, ws=A + 8), SHAPE),
])
def test_tables_refusals(change, status):
    assert _tables(**change) == status


def test_tables_workspace():
    n = ctypes.c_size_t(7)
    for tokens, need in ((20, 0), (100000, 24)):  # few rows are written by the launch that counts them
        d = _TABLES.pack(*{**TABLES, "tokens": tokens}.values())
        assert lg.lib().lutgemm_batch_tables_workspace(d, ctypes.byref(n)) == 0 and n.value == need
    assert lg.lib().lutgemm_batch_tables_workspace(_TABLES.pack(*TABLES.values()), None) == NULL
    assert lg.lib().lutgemm_batch_tables_workspace(None, ctypes.byref(n)) == NULL


SAMPLE = dict(type=0, rows=4, vocab=1000, reserved=0, row_step=1000)


def _sample(wsb=1 << 30, **change):
    at = dict(logits=A, u=A + FAR, temperature=A + 2 * FAR, top_k=A + 3 * FAR, top_p=A + 4 * FAR,
              min_p=A + 5 * FAR, tokens=A + 6 * FAR, logprobs=A + 7 * FAR, ws=A + 8 * FAR)
    d = _SAMPLE.pack(*[change.get(k, v) for k, v in SAMPLE.items()])
    at.update({k: v for k, v in change.items() if k in at})
    return lg.lib().lutgemm_sample_tokens(d, *at.values(), wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(type=3), SHAPE), (dict(type=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 22), SHAPE),
    (dict(vocab=0), SHAPE), (dict(vocab=(1 << 20) + 1), SHAPE), (dict(row_step=-1), SHAPE),
    (dict(row_step=1 << 40), SHAPE), (dict(logits=None), NULL), (dict(u=None), NULL), (dict(tokens=None), NULL),
    (dict(logits=A + 1), ALIGN), (dict(type=2, logits=A + 2), ALIGN), (dict(u=A + 2), ALIGN),
    (dict(temperature=A + 2), ALIGN), (dict(top_k=A + 1), ALIGN), (dict(top_p=A + 2), ALIGN),
    (dict(min_p=A + 2), ALIGN), (dict(tokens=A + 6 * FAR + 4), ALIGN), (dict(logprobs=A + 2), ALIGN),
    (dict(tokens=A + 7992), SHAPE), (dict(tokens=A + FAR + 8), SHAPE), (dict(logprobs=A + 6 * FAR + 28), SHAPE),
    (dict(logprobs=A + 3 * FAR), SHAPE), (dict(ws=None), NULL), (dict(ws=A + 8 * FAR + 8), ALIGN),
    (dict(wsb=100), BUFFER), (dict(ws=A), SHAPE), (dict(ws=A + 5 * FAR), SHAPE),
])
def test_sample_refusals(change, status):
    assert _sample(**change) == status


def test_sample_empty_call():
    assert _sample(rows=0, logits=None, u=None, tokens=None) == 0
    assert lg.lib().lutgemm_sample_tokens(None, *[A] * 9, 1 << 30, None) == NULL


def test_sample_workspace():
    n = ctypes.c_size_t(7)
    for rows, vocab in ((0, 5), (1, 1), (1, 1 << 20), (256, 131073), ((1 << 22) - 1, 1 << 20), (5000, 32000)):
        d = _SAMPLE.pack(0, rows, vocab, 0, vocab)
        assert lg.lib().lutgemm_sample_tokens_workspace(d, ctypes.byref(n)) == 0
        assert (n.value > 0) == (rows > 0) and n.value <= 52 << 20
    assert lg.lib().lutgemm_sample_tokens_workspace(d, None) == NULL


def test_descriptors_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('''
#include <stdio.h>
#include "lutgemm.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(lutgemm_shared), offsetof(lutgemm_shared, max_prefix),
         sizeof(lutgemm_tables), offsetof(lutgemm_tables, table_stride), sizeof(lutgemm_sample),
         offsetof(lutgemm_sample, row_step));
  return 0;
}
''')
    exe = tmp_path / "sizes"
    subprocess.run([cc, "-std=c99", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)], check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = []
    for s in (_SHARED, _TABLES, _SAMPLE):
        want += [s.size, s.size - 8]
    assert got == want


# ------------------------------------------------------------- the binding's checks

def test_binding_refuses_cpu_tensors_and_types():
    h, i = torch.zeros((2, 256), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    q = h.view(2, 2, 128)
    with pytest.raises(ValueError, match="GPU"):
        lg.shared_prefix_attention(q, h, h, h, i, h, i)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        lg.shared_prefix_attention(q.float(), h, h, h, i, h, i)
    with pytest.raises(ValueError, match="GPU"):
        lg.batch_tables(i, i, h, 16, 2)
    with pytest.raises(ValueError, match="tensor"):
        lg.batch_tables([1], i, h, 16, 2)
    with pytest.raises(ValueError, match="GPU"):
        lg.sample_tokens(h, torch.zeros(2))
    with pytest.raises(ValueError, match="fp16, bf16 or fp32"):
        lg.sample_tokens(h.double(), torch.zeros(2))


@pytest.mark.parametrize("which", ["q", "v_pages", "logits", "min_p"])
def test_binding_refuses_tensors_with_gradients(which):
    from torch.autograd import forward_ad
    h, i, flat = torch.zeros((2, 256), dtype=torch.float16), torch.zeros(2, dtype=torch.int32), torch.zeros(2)
    calls = {"q": (lambda t: lg.shared_prefix_attention(t.view(2, 2, 128), h, h, h, i, h, i), h),
             "v_pages": (lambda t: lg.shared_prefix_attention(h.view(2, 2, 128), h, t, h, i, h, i), h),
             "logits": (lambda t: lg.sample_tokens(t, flat), h),
             "min_p": (lambda t: lg.sample_tokens(h, flat, None, None, None, t), flat)}
    call, t = calls[which]
    with pytest.raises(ValueError, match="no gradient"):
        call(t.clone().requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        call(t.clone().requires_grad_())
    with forward_ad.dual_level(), torch.no_grad(), pytest.raises(ValueError, match="no gradient"):
        call(forward_ad.make_dual(t, torch.ones_like(t)))


# ----------------------------------------------------------------- the plain forms

def test_plain_sample_follows_torch():
    """Each kept token's share of evenly spaced random numbers is its probability."""
    rng = np.random.default_rng(0)
    x = rng.normal(0, 2, 40).astype(np.float32)
    p = torch.softmax(torch.from_numpy(x).double() / 0.7, 0).numpy()
    order = np.argsort(-p, kind="stable")
    k = 9
    keep = np.zeros(40, bool)
    keep[order[:k]] = True
    cut = p * keep / (p * keep).sum()
    upto = np.cumsum(cut[order])
    keep[order[int(np.searchsorted(upto, 0.8)) + 1:]] = False
    keep &= p >= 0.05 * p.max()
    want = p * keep / (p * keep).sum()
    n = 20000
    got = np.bincount([plain.sample(x, (i + 0.5) / n, 0.7, k, 0.8, 0.05)[0] for i in range(n)], minlength=40)
    assert np.abs(got / n - want).max() <= 1.0 / n + 1e-12
    token, logprob, _ = plain.sample(x, 0.3, 0.7, k, 0.8, 0.05)
    assert abs(logprob - np.log(want[token])) < 1e-12


def test_plain_tables_keep_every_page_once():
    """Over many steps each page is in one table row or in the ring's free part."""
    rng = np.random.default_rng(1)
    page, pages, seqs, width = 4, 37, 5, 9
    table, ring, free = [[-1] * width for _ in range(seqs)], list(range(pages)), [13, pages]
    lens = [0] * seqs
    for _ in range(300):
        change = [-lens[s] if rng.random() < 0.1 else int(rng.integers(-3, 8)) for s in range(seqs)]
        positions, slots, after, starts, free = plain.tables(change, lens, table, page, 16, ring, free)
        for s in range(seqs):
            rows = range(starts[s], starts[s + 1])
            assert [positions[r] for r in rows] == list(range(lens[s], lens[s] + len(rows)))
            assert after[s] == max(0, lens[s] + (change[s] if change[s] < 0 else len(rows)))
            assert [slots[r] for r in rows] == [table[s][positions[r] // page] * page + positions[r] % page for r in rows]
        lens = after
        used = [p for s in range(seqs) for p in table[s][:-(-lens[s] // page)]]
        rest = [ring[(free[0] + i) % pages] for i in range(free[1])]
        assert sorted(used + rest) == list(range(pages))


def test_decode_stack_arguments():
    from lut_gemv_amd import decode
    for kw in (dict(prefix=1), dict(context=10, prefix=11), dict(context=10, prefix=-1), dict(room=3),
               dict(context=10, room=-1)):
        with pytest.raises(ValueError, match="prefix must be"):
            decode.DecodeStack("llama7b", layers=1, device="cpu", **kw)


@pytest.mark.parametrize("context,prefix,room,page,steps", [(100, 70, 6, 16, 18), (100, 100, 1, 16, 16), (64, 0, 64, 64, 64),
                                                            (1024, 0, 8, 16, 16)])
def test_decode_times_only_steps_that_have_room(context, prefix, room, page, steps):
    """A step without room attends over nothing and would be timed as a fast one."""
    from lut_gemv_amd import decode
    assert decode.room_steps(context, prefix, room, page) == steps
    st = object.__new__(decode.DecodeStack)
    st.room, st.steps = room, steps
    with pytest.raises(ValueError, match=f"room for {steps} steps"):
        st.time_tokens(tokens=steps, warmup=1)
    args = [f"--context={context}", f"--prefix={prefix}", f"--room={room}", f"--page-size={page}", "--model=llama7b"]
    with pytest.raises(SystemExit):
        decode.main([*args, f"--tokens={steps - 4}", "--warmup=5"])


@pytest.mark.parametrize("count", [700000, (1 << 20) - 1])
def test_shared_many_groups_fit_a_launch(count):
    """Groups of one token: workgroups for larger ones among them are left out where they would make
    the launch too large (the missing workspace is found behind that)."""
    assert _shared(type=1, seqs=count, tokens=count, groups=count, heads=4, kv_heads=4, max_q=1, max_kv=16, max_prefix=16,
                   ws=None) == NULL
    assert _shared(type=1, seqs=count, tokens=count, groups=count, heads=8, kv_heads=8, max_q=1, max_kv=16, max_prefix=16,
                   ws=None) == SHAPE
