"""Argument checks of the operators around the layer (moe_linear_q,
moe_beam_select, moe_beam_reorder) and of their binding: CPU only, every call
here is answered before any kernel launch."""
import ctypes
import os

import pytest
import torch

from sparse_moe_router_amd import api

pytestmark = pytest.mark.skipif(not os.path.exists(api.LIB_PATH), reason="libmoe.so not built")

FAKE = 0x10000  # a non-null, aligned address that is never dereferenced here


# ----------------------------------------------------------------------------- moe_linear_q

def linear(**kw):
    d = dict(rows=64, cols=96, qfmt=api.MOE_Q4_SYM_G32, act=api.MOE_ACT_BF16, out=api.MOE_ACT_F32, codes=FAKE,
             scales=FAKE, mins=None, bias=None)
    d.update(kw)
    return api.c_linear(d["rows"], d["cols"], d["qfmt"], d["act"], d["out"],
                        api.c_qmat(d["codes"], d["scales"], d["mins"]), d["bias"])


def run_linear(L, x=FAKE, xs=96, T=4, y=FAKE, ys=64):
    return api.lib().moe_linear_q(ctypes.byref(L) if L is not None else None, x, xs, T, y, ys, None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), api.MOE_E_ARG),
    (dict(cols=0), api.MOE_E_ARG),
    (dict(cols=100), api.MOE_E_ARG),
    (dict(cols=65536 + 32), api.MOE_E_UNSUPPORTED),
    (dict(rows=(1 << 24) + 1), api.MOE_E_UNSUPPORTED),
    (dict(qfmt=9), api.MOE_E_UNSUPPORTED),
    (dict(act=2), api.MOE_E_UNSUPPORTED),
    (dict(out=-1), api.MOE_E_UNSUPPORTED),
    (dict(codes=None), api.MOE_E_ARG),
    (dict(codes=FAKE + 8), api.MOE_E_ARG),
    (dict(scales=None), api.MOE_E_ARG),
    (dict(scales=FAKE + 1), api.MOE_E_ARG),
    (dict(qfmt=api.MOE_Q2_ASYM_G32), api.MOE_E_ARG),
    (dict(bias=FAKE + 2), api.MOE_E_ARG),
])
def test_linear_descriptor(kw, status):
    assert run_linear(linear(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), api.MOE_E_ARG),
    (dict(T=(1 << 20) + 1), api.MOE_E_UNSUPPORTED),
    (dict(x=None), api.MOE_E_ARG),
    (dict(y=None), api.MOE_E_ARG),
    (dict(x=FAKE + 8), api.MOE_E_ARG),
    (dict(y=FAKE + 2), api.MOE_E_ARG),
    (dict(xs=95), api.MOE_E_ARG),
    (dict(xs=100), api.MOE_E_ARG),      # rows not at multiples of 16 bytes
    (dict(ys=63), api.MOE_E_ARG),
    (dict(ys=-64), api.MOE_E_ARG),
    (dict(xs=1 << 41), api.MOE_E_ARG),
])
def test_linear_call(kw, status):
    assert run_linear(linear(), **kw) == status


def test_linear_no_tokens_and_no_descriptor():
    assert run_linear(None) == api.MOE_E_ARG
    assert run_linear(linear(), x=None, y=None, T=0) == api.MOE_OK


def test_linear_binding_checks():
    codes, scales = torch.zeros(64, 48, dtype=torch.uint8), torch.zeros(64, 3, dtype=torch.int16)
    ok = dict(rows=64, cols=96, qfmt="q4_sym_g32", act="bf16", codes=codes, scales=scales)
    for kw, match in ((dict(qfmt="q5"), "unknown format"), (dict(act="f16"), "act must be"), (dict(out=7), "out must be"),
                      (dict(codes=codes[:, :-1]), "codes must be"), (dict(scales=scales[:-1]), "scales must be"),
                      (dict(mins=scales), "2-bit format only"), (dict(qfmt="q3_sym_g32"), "codes must be"),
                      (dict(bias=torch.zeros(63)), "bias must be"), (dict(), "device memory")):
        with pytest.raises(ValueError, match=match):
            api.Linear(**{**ok, **kw})
    L = object.__new__(api.Linear)
    L.rows, L.cols, L.act_dtype, L.out_dtype, L.device = 64, 96, torch.bfloat16, torch.float32, torch.device("cuda", 0)
    L.c = linear()
    x, y = torch.zeros(4, 96, dtype=torch.bfloat16), torch.zeros(4, 64)
    with pytest.raises(TypeError, match="x: expected"):
        api.moe_linear_q(L, x.float(), 4, y)
    for a, b, match in ((x[:3], y, r"x must be \[>=4\]\[96\]"), (x[:, :64], y, "x must be"), (x, y[:3], "y must be"),
                        (x.t().contiguous().t(), y, "contiguous"), (x[:1].expand(4, 96), y, "rows overlap"),
                        (x, y, "device memory")):
        with pytest.raises(ValueError, match=match):
            api.moe_linear_q(L, a, 4, b)


# ----------------------------------------------------------------------------- moe_beam_select

def beam(**kw):
    d = dict(batch=2, beams=3, vocab=1000, n_out=6, act=api.MOE_ACT_F32, eos=5)
    d.update(kw)
    return api.c_beam(d["batch"], d["beams"], d["vocab"], d["n_out"], d["act"], d["eos"])


def run_select(b, logits=FAKE, ld=1000, scores=FAKE, finished=None, allowed=None, lda=0, out=(FAKE, FAKE, FAKE), ws=FAKE,
               ws_bytes=1 << 40):
    return api.lib().moe_beam_select(ctypes.byref(b) if b is not None else None, logits, ld, scores, finished, allowed,
                                     lda, *out, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), api.MOE_E_ARG),
    (dict(beams=0), api.MOE_E_ARG),
    (dict(vocab=0), api.MOE_E_ARG),
    (dict(n_out=0), api.MOE_E_ARG),
    (dict(eos=-2), api.MOE_E_ARG),
    (dict(eos=1000), api.MOE_E_ARG),
    (dict(beams=65), api.MOE_E_UNSUPPORTED),
    (dict(n_out=129), api.MOE_E_UNSUPPORTED),
    (dict(vocab=(1 << 24) + 1), api.MOE_E_UNSUPPORTED),
    (dict(batch=(1 << 20)), api.MOE_E_UNSUPPORTED),
    (dict(act=3), api.MOE_E_UNSUPPORTED),
])
def test_beam_descriptor(kw, status):
    b = beam(**kw)
    assert run_select(b, ld=1 << 30) == status
    assert api.lib().moe_beam_workspace_bytes(ctypes.byref(b)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), api.MOE_E_ARG),
    (dict(logits=FAKE + 2), api.MOE_E_ARG),
    (dict(scores=None), api.MOE_E_ARG),
    (dict(ld=999), api.MOE_E_ARG),
    (dict(out=(None, FAKE, FAKE)), api.MOE_E_ARG),
    (dict(out=(FAKE, FAKE + 1, FAKE)), api.MOE_E_ARG),
    (dict(allowed=FAKE, lda=31), api.MOE_E_ARG),   # 32 words hold 1000 bits
    (dict(allowed=FAKE, lda=-32), api.MOE_E_ARG),
    (dict(allowed=FAKE + 2), api.MOE_E_ARG),
    (dict(ws=None), api.MOE_E_WORKSPACE),
    (dict(ws=FAKE + 64), api.MOE_E_ARG),
])
def test_beam_call(kw, status):
    assert run_select(beam(), **kw) == status


def test_beam_workspace_and_empty_batch():
    b = beam()
    need = api.lib().moe_beam_workspace_bytes(ctypes.byref(b))
    assert need > 0 and run_select(b, ws_bytes=need - 1) == api.MOE_E_WORKSPACE
    assert run_select(None) == api.MOE_E_ARG
    assert run_select(beam(eos=-1), finished=FAKE) == api.MOE_E_ARG  # finished beams need a token to go on with
    assert run_select(beam(batch=0), None, 0, None, out=(None, None, None), ws=None, ws_bytes=0) == api.MOE_OK
    assert api.lib().moe_beam_workspace_bytes(ctypes.byref(beam(batch=0))) == 256


def test_beam_binding_checks():
    b = api.Beam(batch=2, beams=3, vocab=100, n_out=6, eos=1)
    i32 = torch.int32
    a = dict(logits=torch.zeros(6, 100), scores=torch.zeros(2, 3), out_score=torch.zeros(2, 6),
             out_parent=torch.zeros(2, 6, dtype=i32), out_token=torch.zeros(2, 6, dtype=i32),
             finished=torch.zeros(2, 3, dtype=torch.uint8), allowed=torch.zeros(6, 4, dtype=i32))
    for key in ("scores", "out_score", "out_parent", "out_token", "finished"):
        with pytest.raises(ValueError, match=f"{key}: .* at least"):
            api.moe_beam_select(b, **{**a, key: a[key].flatten()[:-1]})
    for kw, match in ((dict(logits=a["logits"][:5]), "logits must be"), (dict(logits=a["logits"][:, :99]), "logits must be"),
                      (dict(allowed=a["allowed"][:5]), "allowed must be"), (dict(allowed=a["allowed"][:, :3]), "allowed must"),
                      (dict(), "device memory")):
        with pytest.raises(ValueError, match=match):
            api.moe_beam_select(b, **{**a, **kw})
    with pytest.raises(TypeError, match="logits"):
        api.moe_beam_select(b, **{**a, "logits": a["logits"].bfloat16()})
    with pytest.raises(TypeError, match="finished"):
        api.moe_beam_select(b, **{**a, "finished": a["finished"].bool()})
    with pytest.raises(api.MoeError):
        api.beam_workspace(api.Beam(batch=2, beams=3, vocab=100, n_out=0), "cpu")


# ----------------------------------------------------------------------------- moe_beam_reorder

def state(**kw):
    d = dict(src=FAKE, dst=FAKE << 8, chunk_bytes=64, chunks=2, src_row_stride=256, src_chunk_stride=128, dst_row_stride=128,
             dst_chunk_stride=64)
    d.update(kw)
    return api.c_state(d["src"], d["dst"], d["chunk_bytes"], d["chunks"], d["src_row_stride"], d["src_chunk_stride"],
                       d["dst_row_stride"], d["dst_chunk_stride"])


def run_reorder(states, n=None, parent=FAKE, ldp=4, batch=2, beams=4):
    arr = (api.c_state * max(len(states), 1))(*states)
    return api.lib().moe_beam_reorder(arr, len(states) if n is None else n, parent, ldp, batch, beams, None)


SAME = dict(dst=FAKE, dst_row_stride=256, dst_chunk_stride=128)


@pytest.mark.parametrize("kw", [
    dict(chunk_bytes=-1), dict(chunks=-1), dict(src=None), dict(dst=None), dict(src_row_stride=-256),
    dict(dst_chunk_stride=-64),
    dict(dst_chunk_stride=63),                        # pieces overlap
    dict(dst_row_stride=127),                         # rows overlap
    dict(dst_row_stride=64, dst_chunk_stride=256),    # 8 rows of 64 bytes reach past the next piece
    dict(dst=FAKE + 512),                             # inside src's range
    dict(dst=FAKE - 512),                             # ends inside src's range
    {**SAME, "dst_row_stride": 512},                  # in place with other strides
    {**SAME, "dst_chunk_stride": 64},
    dict(src_row_stride=1 << 41),
])
def test_reorder_state(kw):
    assert run_reorder([state(**kw)]) == api.MOE_E_ARG
    assert run_reorder([state(chunks=0, **{k: v for k, v in kw.items() if k != "chunks"}), state(**kw)]) == api.MOE_E_ARG


def test_reorder_call():
    assert run_reorder([state()], parent=None) == api.MOE_E_ARG
    assert run_reorder([state()], parent=FAKE + 2) == api.MOE_E_ARG
    assert run_reorder([state()], ldp=3) == api.MOE_E_ARG
    assert run_reorder([state()], n=-1) == api.MOE_E_ARG
    assert run_reorder([state()], batch=-1) == api.MOE_E_ARG
    assert run_reorder([state()], beams=0) == api.MOE_E_ARG
    assert run_reorder([state()], beams=65) == api.MOE_E_UNSUPPORTED
    assert run_reorder([state(chunks=(1 << 22) + 1)]) == api.MOE_E_UNSUPPORTED
    assert run_reorder([state()], batch=0, parent=None) == api.MOE_OK
    assert run_reorder([], parent=None) == api.MOE_OK


def test_reorder_binding_checks():
    parent = torch.zeros(2, 4, dtype=torch.int32)
    s = torch.zeros(8, 3, 10)
    for states, par, dst, match in (
            ([s[:7]], parent, None, "must have 8 rows"), ([s], parent[:1], None, "parent must be"),
            ([s], parent.long(), None, "parent must be"), ([s], parent, [], "1 states, 0 destinations"),
            ([s], parent, [s[:, :2]], "same shape"), ([s], parent, [s.half()], "same shape and type"),
            ([torch.zeros(8, 4, 5, 6)[:, :3, :, ::2]], parent, None, "device memory"),  # equally spaced single elements
            ([torch.zeros(8, 4, 5, 6)[:, :3, :4, :5]], parent, None, "equally spaced"),
            ([s[:, :, :4]], parent, [torch.zeros(8, 6, 10)[:, ::2, :4].flip(0)], "device memory"),
            ([s], parent, None, "device memory")):
        with pytest.raises(ValueError, match=match):
            api.moe_beam_reorder(states, par, 2, 4, dst=dst)
    assert api._pieces(torch.zeros(8, 4, 100, 16)[:, :, :7]) == (112, 4, 1600)
    assert api._pieces(torch.zeros(8, 4, 100, 16)) == (6400, 1, 0)
    assert api._pieces(torch.zeros(8)) == (1, 1, 0)
    assert api._pieces(torch.zeros(8, 2, 3, 100, 16)[:, :, :, 50:]) == (800, 6, 1600)
