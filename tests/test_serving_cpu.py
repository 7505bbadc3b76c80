"""The operators beside the weight products, host side: every argument error is
reported before any HIP call, the descriptors' layout is the header's, and the
plain forms agree with torch's own attention. No GPU."""
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
NULL, SHAPE, VALUE, BUFFER, ALIGN = 1, 2, 3, 4, 5
# the header's descriptors
_HEADS = struct.Struct("@7if11q")
_ATTENTION = struct.Struct("@8ifi15q")
_ADAPTERS = struct.Struct("@6i3q")


# ------------------------------------------------------------- attention refusals

ATT = dict(type=0, heads=8, kv_heads=2, head_dim=128, page_size=16, seqs=3, table_width=10, window=0,
           scale=0.1, reserved=0, tokens=30, pages=20, table_stride=10, max_q=10, max_kv=160,
           q_token=1024, q_head=128, o_token=1024, o_head=128, k_page=4096, k_slot=256, k_head=128,
           v_page=4096, v_slot=256, v_head=128)


def _attention(ws=None, wsb=0, q=A, k=A, v=A, table=A, lens=A, starts=A, out=A, **change):
    d = _ATTENTION.pack(*{**ATT, **change}.values())
    return lg.lib().lutgemm_paged_attention(d, q, k, v, table, lens, starts, out, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(type=2), SHAPE), (dict(type=-1), SHAPE), (dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE),
    (dict(heads=0), SHAPE), (dict(heads=7), SHAPE), (dict(heads=2048), SHAPE), (dict(kv_heads=0), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=48), SHAPE), (dict(page_size=1 << 17), SHAPE),
    (dict(seqs=-1), SHAPE), (dict(seqs=1 << 20), SHAPE), (dict(tokens=-1), SHAPE),
    (dict(tokens=1 << 24), SHAPE), (dict(table_width=0), SHAPE), (dict(table_width=1 << 27), SHAPE),
    (dict(table_stride=-1), SHAPE), (dict(pages=0), SHAPE), (dict(pages=1 << 31), SHAPE),
    (dict(window=-1), SHAPE), (dict(max_q=-1), SHAPE), (dict(max_kv=-1), SHAPE),
    (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=float("nan")), VALUE),
    (dict(scale=float("inf")), VALUE), (dict(q_token=1020), SHAPE), (dict(q_head=-8), SHAPE),
    (dict(o_head=4), SHAPE), (dict(k_slot=1 << 24), SHAPE), (dict(v_page=12), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(q=A + 8), ALIGN), (dict(k=A + 2), ALIGN),
    (dict(v=A + 8), ALIGN), (dict(out=A + 8), ALIGN), (dict(table=A + 2), ALIGN),
    (dict(lens=A + 1), ALIGN), (dict(starts=A + 2), ALIGN), (dict(starts=None), SHAPE),
])
def test_attention_refusals(change, status):
    assert _attention(**change) == status


@pytest.mark.parametrize("call,change", [
    ("attention", dict(o_token=0)), ("attention", dict(o_head=0)), ("attention", dict(o_head=120)),
    ("attention", dict(o_token=128)), ("attention", dict(o_token=1016)),
    ("heads", dict(q_token=0)), ("heads", dict(q_token=248)), ("heads", dict(k_head=0)),
    ("heads", dict(k_slot=64)), ("heads", dict(v_page=0)), ("heads", dict(v_slot=120)),
    ("adapters", dict(out_row=0)), ("adapters", dict(out_row=39)),
])
def test_outputs_that_overlap_are_refused(call, change):
    assert {"attention": _attention, "heads": _heads, "adapters": _adapters}[call](**change) == SHAPE


def test_attention_positions_stay_in_32_bits():
    """Tables of up to 2^30 keys: a position, a window and a tile past them add up."""
    assert _attention(q=None, table_width=1 << 26) == NULL
    assert _attention(q=None, table_width=(1 << 26) + 1) == SHAPE


@pytest.mark.parametrize("change", [
    dict(seqs=16, tokens=8192, heads=64, kv_heads=8, max_q=8000),   # chunks beside single tokens
    dict(seqs=16, tokens=8192, heads=64, kv_heads=8, max_q=1),      # a padded batch, or a wrong bound
    dict(seqs=1, tokens=1, heads=128, kv_heads=1, max_q=1),
    dict(seqs=1, tokens=300, heads=8, kv_heads=1, max_q=300),
])
def test_attention_workspace_stays_small(change):
    """Room for the parts of the rows that can be split, not for every row of the batch."""
    n = ctypes.c_size_t()
    d = _ATTENTION.pack(*{**ATT, "max_kv": 1 << 20, "table_width": 1 << 16, "o_token": 1 << 14, **change}.values())
    assert lg.lib().lutgemm_paged_attention_workspace(d, ctypes.byref(n)) == 0
    assert 0 < n.value < 80 << 20


@pytest.mark.parametrize("change", [
    dict(out=A + 16), dict(out=A - 16), dict(out=A + 256), dict(out=A - 256),
    dict(q_token=2048, o_token=2048, out=A + 1920), dict(q_token=2048, o_token=2048, out=A - 1920),
    dict(q_token=2048, out=A), dict(q_head=256, q_token=2048, o_token=2048, out=A),
    dict(q_token=2048, out=A + 29 * 4096),
    dict(q_token=128, q_head=3840, o_token=128, o_head=3840, out=A + 256),  # heads outside tokens
])
def test_attention_outputs_over_the_queries_are_refused(change):
    assert _attention(**change) == SHAPE


@pytest.mark.parametrize("change", [
    dict(), dict(q=2 * A), dict(q_token=2048, o_token=2048, out=A + 2048),
    dict(q_token=2048, o_token=2048, out=A - 2048), dict(out=A + 30 * 2048), dict(out=A - 30 * 2048),
    dict(q_token=128, q_head=3840, o_token=128, o_head=3840),
    dict(q_token=128, q_head=7680, o_token=128, o_head=7680, out=A + 2 * 3840),  # heads outside tokens
])
def test_attention_outputs_in_place_or_beside_the_queries_are_not(change):
    """Another error is the first to be found (no workspace): nothing is launched."""
    long = dict(seqs=1, max_kv=65536, table_width=4096)
    assert _attention(**{**long, **change}) == NULL


def test_attention_empty_calls_and_workspace():
    assert _attention(tokens=0) == 0 and _attention(tokens=0, seqs=0, starts=None) == 0
    L = lg.lib()
    assert L.lutgemm_paged_attention(None, A, A, A, A, A, A, A, None, 0, None) == NULL
    n = ctypes.c_size_t()
    long = dict(seqs=1, tokens=1, max_q=1, max_kv=65536, table_width=4096)
    d = _ATTENTION.pack(*{**ATT, **long}.values())
    assert L.lutgemm_paged_attention_workspace(d, ctypes.byref(n)) == 0 and n.value > 0
    assert L.lutgemm_paged_attention_workspace(d, None) == NULL
    assert _attention(**long) == NULL
    assert _attention(ws=A, wsb=n.value - 1, **long) == BUFFER
    assert _attention(ws=A + 4, wsb=n.value, **long) == ALIGN


# ----------------------------------------------------------------- heads refusals

HEADS = dict(type=1, heads=4, kv_heads=2, head_dim=64, rotary=64, interleaved=0, page_size=16, eps=1e-6,
             tokens=5, positions=100, pages=9, qkv_token=512, q_token=256, k_page=2048, k_slot=128,
             k_head=64, v_page=2048, v_slot=128, v_head=64)


def _heads(qkv=A, at=A, table=A, qw=A, kw=A, q=A, k=A, v=A, slots=A, **change):
    d = _HEADS.pack(*{**HEADS, **change}.values())
    return lg.lib().lutgemm_qk_norm_rotate(d, qkv, at, table, qw, kw, q, k, v, slots, None)


@pytest.mark.parametrize("change,status", [
    (dict(type=3), SHAPE), (dict(heads=0), SHAPE), (dict(kv_heads=0), SHAPE), (dict(heads=70000), SHAPE),
    (dict(head_dim=8), SHAPE), (dict(head_dim=72), SHAPE), (dict(head_dim=272), SHAPE),
    (dict(rotary=80), SHAPE), (dict(rotary=8), SHAPE), (dict(rotary=-16), SHAPE),
    (dict(interleaved=2), SHAPE), (dict(page_size=0), SHAPE), (dict(eps=-1.0), VALUE),
    (dict(eps=float("nan")), VALUE), (dict(eps=float("inf")), VALUE), (dict(tokens=-1), SHAPE),
    (dict(tokens=1 << 24), SHAPE), (dict(positions=0), SHAPE), (dict(pages=-1), SHAPE),
    (dict(qkv_token=4), SHAPE), (dict(q_token=-8), SHAPE), (dict(k_slot=1), SHAPE),
    (dict(v_head=12), SHAPE), (dict(qkv=None), NULL), (dict(q=None), NULL), (dict(k=None), NULL),
    (dict(v=None), NULL), (dict(at=None), NULL), (dict(table=None), NULL), (dict(qw=None), NULL),
    (dict(kw=None), NULL), (dict(qkv=A + 2), ALIGN), (dict(q=A + 8), ALIGN), (dict(k=A + 8), ALIGN),
    (dict(v=A + 8), ALIGN), (dict(table=A + 4), ALIGN), (dict(qw=A + 2), ALIGN), (dict(at=A + 4), ALIGN),
    (dict(slots=A + 4), ALIGN),
])
def test_heads_refusals(change, status):
    assert _heads(**change) == status


@pytest.mark.parametrize("change", [
    dict(q=A), dict(q=A + 16, q_token=512), dict(q=A + 512, q_token=512), dict(q=A + 1008, q_token=512),
    dict(q=A - 16, q_token=512), dict(q=A + 4 * 1024 + 1008), dict(tokens=1, q=A + 128),
])
def test_heads_outputs_over_other_parts_of_qkv_are_refused(change):
    assert _heads(**{**dict(k=2 * A, v=3 * A), **change}) == SHAPE


def test_heads_empty_call():
    assert _heads(tokens=0) == 0
    assert lg.lib().lutgemm_qk_norm_rotate(None, A, A, A, A, A, A, A, A, A, None) == NULL


# -------------------------------------------------------------- adapters refusals

ADD = dict(type=0, rows=80, K=64, N=40, rank=16, adapters=3, x_row=64, y_row=40, out_row=40)


def _adapters(x=A, y=A, a=A, b=A, s=A, ids=A, out=2 * A, ws=A, wsb=1 << 20, **change):
    d = _ADAPTERS.pack(*{**ADD, **change}.values())
    return lg.lib().lutgemm_adapters_add(d, x, y, a, b, s, ids, out, ws, wsb, None)


@pytest.mark.parametrize("change,status", [
    (dict(type=2), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=65536), SHAPE), (dict(K=12), SHAPE),
    (dict(K=-8), SHAPE), (dict(K=1 << 23), SHAPE), (dict(N=-1), SHAPE), (dict(N=1 << 23), SHAPE),
    (dict(rank=0), SHAPE), (dict(rank=12), SHAPE), (dict(rank=136), SHAPE), (dict(adapters=-1), SHAPE),
    (dict(adapters=4097), SHAPE), (dict(x_row=60), SHAPE), (dict(y_row=-1), SHAPE),
    (dict(out_row=-1), SHAPE), (dict(x_row=1 << 26), SHAPE), (dict(y_row=1 << 40), SHAPE),
    (dict(out_row=57 << 20), SHAPE), (dict(x=None), NULL), (dict(y=None), NULL), (dict(a=None), NULL),
    (dict(b=None), NULL), (dict(ids=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(wsb=16), BUFFER), (dict(ws=A + 8), ALIGN), (dict(x=A + 8), ALIGN), (dict(a=A + 2), ALIGN),
    (dict(b=A + 4), ALIGN), (dict(s=A + 2), ALIGN), (dict(ids=A + 2), ALIGN), (dict(y=A + 1), ALIGN),
    (dict(out=A + 1), ALIGN), (dict(out=A, out_row=48), SHAPE),
])
def test_adapters_refusals(change, status):
    assert _adapters(**change) == status


@pytest.mark.parametrize("change", [
    dict(x=2 * A, K=40, x_row=40),                                   # x itself
    dict(x=2 * A + 16, x_row=64), dict(x=2 * A - 16, x_row=64),      # x, other rows' steps
    dict(x=2 * A + 80 * 80 - 16, x_row=64), dict(x=2 * A - 2 * (79 * 64 + 64) + 16),
    dict(y=2 * A + 2), dict(y=2 * A - 2), dict(y=2 * A + 80), dict(y=2 * A, y_row=48, out_row=40),
    dict(x=2 * A + 64, x_row=104, out_row=104), dict(y=2 * A + 78, y_row=200, out_row=200),
    dict(x=2 * A + 80, x_row=96, out_row=96), dict(y=2 * A + 80 * 99, y_row=80, out_row=79),
    dict(rows=1, x=2 * A + 64), dict(rows=1, y=2 * A - 78, y_row=0, out_row=0),
])
def test_adapters_outputs_over_their_inputs_are_refused(change):
    assert _adapters(**{**dict(x=4 * A, y=6 * A), **change}) == SHAPE


@pytest.mark.parametrize("change", [
    dict(y=2 * A), dict(x=2 * A + 80 * 80), dict(x=2 * A - 2 * (79 * 64 + 64)),
    dict(x=2 * A + 80, x_row=104, out_row=104), dict(x=2 * A - 128, x_row=104, out_row=104),
    dict(y=2 * A + 80, y_row=80, out_row=80), dict(y=2 * A - 80, y_row=80, out_row=80),
    dict(rows=1, x=2 * A + 80), dict(rows=1, y=2 * A - 80), dict(adapters=0, x=2 * A, K=40, x_row=40),
])
def test_adapters_outputs_beside_their_inputs_are_not(change):
    """Another error is the first to be found (no workspace): nothing is launched."""
    assert _adapters(**{**dict(x=4 * A, y=6 * A, ws=None, rank=128), **change}) == NULL


def test_adapters_empty_calls():
    assert _adapters(rows=0) == 0 and _adapters(N=0) == 0
    assert lg.lib().lutgemm_adapters_add(None, A, A, A, A, A, A, A, A, 0, None) == NULL
    assert lg.lib().lutgemm_adapters_workspace(_ADAPTERS.pack(*ADD.values()), None) == NULL


# ------------------------------------------------------------- the binding's checks

def test_binding_refuses_cpu_tensors_and_types():
    h = torch.zeros((2, 256), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        lg.qk_norm_rotate(h, 2, 1)
    with pytest.raises(ValueError, match="fp16 or bf16"):
        lg.qk_norm_rotate(h.float(), 2, 1)
    with pytest.raises(ValueError, match="GPU"):
        lg.paged_attention(h.view(2, 2, 128), h, h, h, h)
    with pytest.raises(ValueError, match="GPU"):
        lg.adapters_add(h, h, h, h, h)
    with pytest.raises(ValueError):
        lg.rotary_table(0, 64)
    with pytest.raises(ValueError):
        lg.rotary_table(8, 7)


@pytest.mark.parametrize("which", ["qkv", "k_weight", "k_pages", "scales"])
def test_binding_refuses_forward_mode_tangents(which):
    """A dual tensor's tangent is not dropped without a word, under no_grad neither."""
    from torch.autograd import forward_ad
    h, flat = torch.zeros((2, 256), dtype=torch.float16), torch.zeros(2)
    calls = {"qkv": (lambda t: lg.qk_norm_rotate(t, 2, 1), h),
             "k_weight": (lambda t: lg.qk_norm_rotate(h, 2, 1, None, None, h, t), h),
             "k_pages": (lambda t: lg.paged_attention(h.view(2, 2, 128), t, h, h, h), h),
             "scales": (lambda t: lg.adapters_add(h, h, h, h, h, t), flat)}
    call, t = calls[which]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(t, torch.ones_like(t))
        with pytest.raises(ValueError, match="no gradient"):
            call(dual)
        with torch.no_grad(), pytest.raises(ValueError, match="no gradient"):
            call(dual)
        with pytest.raises(ValueError, match="GPU"):
            call(forward_ad.unpack_dual(dual).primal)


def test_packed_call_needs_adapters_and_ids_together():
    import workloads
    w = workloads.random_bcq(32, 512, 2, 128, seed=1)
    pw = lg.PackedBCQ.from_bcq(w.bits, w.alpha, None, w.g, device="cpu")
    x = torch.zeros((2, 512), dtype=torch.float16)
    for kw in (dict(adapters=(x, x, None)), dict(ids=x)):
        with pytest.raises(ValueError, match="together"):
            pw(x, **kw)


def test_decode_stack_arguments():
    from lut_gemv_amd import decode
    for kw in (dict(context=-1), dict(adapters=-1)):
        with pytest.raises(ValueError):
            decode.DecodeStack("llama7b", layers=1, device="cpu", **kw)


@pytest.mark.parametrize("torch_found", [True, False])
def test_the_library_builds_without_torch(torch_found, tmp_path, monkeypatch):
    """Where torch is not installed the C library is built, and only the binding is not."""
    from lut_gemv_amd import build
    calls = []

    def run(cmd, verbose):
        calls.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    monkeypatch.setattr(build, "_run", run)
    for name in ("LIB_PATH", "TRACE_LIB_PATH", "BINDING_PATH"):
        monkeypatch.setattr(build, name, str(tmp_path / name))
    if not torch_found:
        find = build.importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec",
                            lambda name, *a: None if name == "torch" else find(name, *a))
        monkeypatch.setattr(build, "_binding_job", None)
    assert build.build() == str(tmp_path / "LIB_PATH")
    built = sorted(f.name for f in tmp_path.iterdir())
    assert built == ["BINDING_PATH"] * torch_found + ["LIB_PATH", "TRACE_LIB_PATH"]
    assert any(cmd[-1] == str(tmp_path / "LIB_PATH.tmp") for cmd in calls)


def test_descriptors_match_the_header(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('''
#include <stdio.h>
#include "lutgemm.h"
int main(void) {
  printf("%zu %zu %zu %zu %zu %zu\\n", sizeof(lutgemm_heads), offsetof(lutgemm_heads, v_head),
         sizeof(lutgemm_attention), offsetof(lutgemm_attention, v_head), sizeof(lutgemm_adapters),
         offsetof(lutgemm_adapters, out_row));
  return 0;
}
''')
    exe = tmp_path / "sizes"
    subprocess.run([cc, "-std=c99", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", str(exe)],
                   check=True)
    got = [int(v) for v in subprocess.run([str(exe)], capture_output=True, text=True).stdout.split()]
    want = []
    for s in (_HEADS, _ATTENTION, _ADAPTERS):
        want += [s.size, s.size - 8]
    assert got == want and struct.calcsize("@i") == 4


# ----------------------------------------------------------------- the plain forms

def test_plain_attention_is_softmax_attention():
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((3, 4, 8), (7, 2, 8), (7, 2, 8)))
    out, _ = plain.attention(q, k, v, 3, 7, 0.3, 0, 2.0 ** -11)
    tq, tk, tv = (torch.from_numpy(t).transpose(0, 1) for t in (q, k, v))
    tk, tv = (t.repeat_interleave(2, 0) for t in (tk, tv))
    mask = torch.tril(torch.ones(7, 7, dtype=torch.bool))[-3:]
    ref = torch.nn.functional.scaled_dot_product_attention(tq, tk, tv, attn_mask=mask, scale=0.3)
    assert np.allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12)
    early, _ = plain.attention(q, k[:1], v[:1], 3, 1, 0.3, 0, 2.0 ** -11)
    assert (early[:2] == 0).all() and np.allclose(early[2], v[0].repeat(2, 0))


def test_plain_heads_turn_pairs():
    x = np.random.default_rng(1).standard_normal((2, 3, 6))
    th = np.array([[0.5, 1.0], [0.1, -0.4]])
    for interleaved in (False, True):
        out, _ = plain.heads(x, None, 0.0, np.cos(th), np.sin(th), interleaved, 2.0 ** -11)
        a, b = (x[..., [0, 2]], x[..., [1, 3]]) if interleaved else (x[..., :2], x[..., 2:4])
        z = (a + 1j * b) * np.exp(1j * th)[:, None]
        got = (out[..., [0, 2]] + 1j * out[..., [1, 3]]) if interleaved \
            else out[..., :2] + 1j * out[..., 2:4]
        assert np.allclose(got, z) and np.array_equal(out[..., 4:], x[..., 4:])


def test_plain_adapters():
    rng = np.random.default_rng(2)
    y, x, a, b = (rng.standard_normal(s) for s in ((3, 5), (3, 8), (2, 4, 8), (2, 5, 4)))
    out, _ = plain.adapters(y, x, a, b, [1, -1, 0], [2.0, 3.0], 2.0 ** -11, 2.0 ** -21)
    assert np.allclose(out[0], y[0] + 3 * b[1] @ a[1] @ x[0]) and np.array_equal(out[1], y[1])
    assert np.allclose(out[2], y[2] + 2 * b[0] @ a[0] @ x[2])
