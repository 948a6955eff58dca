"""moe_beam_select and moe_beam_reorder against their definitions in 64 bits on
the CPU, and a beam search of several steps through the head's projection, the
selection and the reordering."""
import numpy as np
import pytest
import torch

import synth
from oracle import moe_oracle as mo
from sparse_moe_router_amd import api
from tests import gpu_util as gu

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    api.lib()


def select_ref(logits, scores, n_out, finished=None, eos=-1, allowed=None):
    """(totals, parents, tokens): the definition, logits [B*W][V] float64 (exact values of the stored type),
    allowed bool [B*W][V]."""
    B, W = scores.shape
    V = logits.shape[1]
    out = (np.full((B, n_out), -np.inf), np.full((B, n_out), -1, np.int64), np.full((B, n_out), -1, np.int64))
    for b in range(B):
        totals, flats = [], []
        for w in range(W):
            s = float(scores[b, w])
            if not np.isfinite(s):
                continue
            if finished is not None and finished[b, w]:
                totals.append(np.array([s]))
                flats.append(np.array([w * V + eos]))
                continue
            row = logits[b * W + w]
            ids = np.arange(V) if allowed is None else np.nonzero(allowed[b * W + w])[0]
            v = row[ids]
            if v.size == 0 or np.isnan(v).any() or v.max() in (np.inf, -np.inf):
                continue
            top = v.max()
            with np.errstate(under="ignore"):
                total = np.log(np.sum(np.exp(v - top)))
            keep = v > -np.inf
            totals.append(s + ((v[keep] - top) - total))
            flats.append(w * V + ids[keep])
        if not totals:
            continue
        t, f = np.concatenate(totals), np.concatenate(flats)
        order = np.lexsort((f, -t))[:n_out]
        k = order.size
        out[0][b, :k], out[1][b, :k], out[2][b, :k] = t[order], f[order] // V, f[order] % V
    return out


def pack_allowed(mask):
    rows, V = mask.shape
    words = (V + 31) // 32
    bits = np.zeros((rows, words * 32), np.uint8)
    bits[:, :V] = mask
    return np.packbits(bits, axis=1, bitorder="little").view(np.uint32)


def run_select(logits, scores, n_out, finished=None, eos=-1, allowed=None, act="f32", dev_logits=None, stream=None):
    B, W = scores.shape
    V = logits.shape[1]
    lg = torch.from_numpy(logits.astype(np.float32)).to(gu.DEV).to(DT[act]) if dev_logits is None else dev_logits
    beam = api.Beam(batch=B, beams=W, vocab=V, n_out=n_out, act=act, eos=eos)
    outs = (torch.full((B, n_out), 9.0, device=gu.DEV), torch.full((B, n_out), 9, dtype=torch.int32, device=gu.DEV),
            torch.full((B, n_out), 9, dtype=torch.int32, device=gu.DEV))
    ws = api.beam_workspace(beam, gu.DEV)
    ws.fill_(0xAB)  # nothing may depend on what the workspace held
    api.moe_beam_select(
        beam, lg, torch.from_numpy(scores.astype(np.float32)).to(gu.DEV), *outs,
        finished=None if finished is None else torch.from_numpy(finished.astype(np.uint8)).to(gu.DEV),
        allowed=None if allowed is None else torch.from_numpy(pack_allowed(allowed).view(np.int32)).to(gu.DEV), ws=ws,
        stream=stream)
    torch.cuda.synchronize()
    return tuple(o.cpu().numpy() for o in outs)


def check(logits, scores, n_out, finished=None, eos=-1, allowed=None, act="f32", **kw):
    """Parents and tokens equal; scores off by the rounding to fp32 (2^-24) and an L good to 2^-30 of its size + 1
    (the totals themselves are held in 64 bits)."""
    got = run_select(logits, scores, n_out, finished, eos, allowed, act, **kw)
    full = None if allowed is None else np.broadcast_to(allowed, (logits.shape[0], logits.shape[1]))
    want = select_ref(logits, scores.astype(np.float32).astype(np.float64), n_out, finished, eos, full)
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[2], want[2]), (got[2], want[2])
    live = want[1] >= 0
    assert np.all(got[0][~live] == -np.inf)
    lim = 2.0 ** -24 * np.abs(want[0][live]) + 2.0 ** -30 * (1 + np.abs(want[0][live]))
    assert np.all(np.abs(got[0][live] - want[0][live]) <= lim)
    return got


def gen(r, B, W, V, act, spread=2.2):
    lg = spread * r.standard_normal((B * W, V))
    lg[np.arange(B * W)[:, None], r.integers(0, V, (B * W, 8))] += 3 + 6 * r.random((B * W, 8))
    sc = -np.sort(5 + 10 * r.random((B, W)), axis=1)
    return mo.round_act(lg, act), sc


SELECT = [  # batch, beams, vocab, n_out
    (1, 1, 1, 1), (1, 1, 7, 3), (2, 3, 5, 20), (1, 4, 33, 8), (3, 2, 255, 4), (1, 5, 1000, 10), (2, 8, 4097, 16),
    (1, 64, 301, 128), (4, 1, 50021, 1), (1, 3, 70001, 128), (5, 16, 2048, 32), (1, 2, 262144, 5), (70, 3, 600, 6), (4, 11, 520, 18),
    (3, 24, 6035, 42), (2, 2, 256, 4), (2, 3, 257, 4), (1, 6, 769, 30)]


@pytest.mark.parametrize("act", ("f32", "bf16"))
@pytest.mark.parametrize("B,W,V,n", SELECT)
def test_select(B, W, V, n, act):
    r = np.random.default_rng(B * 1000 + W * 100 + n)
    lg, sc = gen(r, B, W, V, act)
    gu.say(f"select B={B} W={W} V={V} n={n} {act}")
    check(lg, sc, n, act=act)
    fin = (r.random((B, W)) < 0.4)
    mask = r.random((B * W, V)) < 0.5
    mask[r.integers(0, B * W)] = False
    noisy = lg.copy()
    noisy[~mask & (r.random((B * W, V)) < 0.2)] = np.nan
    noisy[~mask & (r.random((B * W, V)) < 0.1)] = np.inf
    check(noisy, sc, n, fin, V // 2, mask, act)
    check(lg, sc, n, fin, V - 1, mask[:1], act)
    check(lg, sc, n, np.ones((B, W), bool), 0, None, act)


@pytest.mark.parametrize("act", ("f32", "bf16"))
@pytest.mark.parametrize("V", (40, 3000, 40007))
def test_select_ties(V, act):
    """Equal totals: lowest beam, then lowest token.  Rows of one value, of two values, of few values, equal beams."""
    sc = np.array([[-1.0, -1.0, -1.0], [0.0, -np.inf, 0.0]])
    r = np.random.default_rng(V)
    one = np.zeros((6, V))
    two = np.where(r.random((6, V)) < 0.3, 1.0, -1.0)
    few = r.integers(0, 4, (1, V)).repeat(6, axis=0).astype(np.float64)
    zeros = np.where(r.random((6, V)) < 0.5, 0.0, -0.0)
    for lg in (one, two, few, zeros, np.sort(r.standard_normal((6, V)).round(1), axis=1),
               -np.sort(r.standard_normal((6, V)).round(1), axis=1)):
        lg = mo.round_act(lg, act)
        for n in (1, 6, 64, 128):
            check(lg, sc, n, act=act)
        check(lg, sc, 20, act=act, allowed=r.random((6, V)) < 0.1)


def test_select_rows_without_candidates():
    """Empty masks, -inf everywhere, a NaN or +inf among the allowed, scores that are not finite: those beams offer
    nothing and the others are served."""
    r = np.random.default_rng(3)
    for V in (50, 9000):
        lg, sc = gen(r, 3, 6, V, "f32")
        lg[0], lg[1, 1:], lg[2, V // 3], lg[3, V - 1] = -np.inf, -np.inf, np.nan, np.inf
        lg[4, ::2] = -np.inf
        lg[6:12] = -np.inf
        lg[12] = np.finfo(np.float32).min
        lg[13, :3] = [np.finfo(np.float32).max, 0, np.finfo(np.float32).min]
        lg[14] = -1e30
        sc[2] = [-3, -4, np.inf, np.nan, -np.inf, -1e30]
        for n in (3, 12, 100):
            check(lg, sc, n)
        mask = np.zeros((18, V), bool)
        mask[0, 5] = mask[17, V - 1] = True
        check(lg, sc, 12, allowed=mask)
        check(lg, sc, 12, allowed=np.zeros((1, V), bool))


@pytest.mark.parametrize("act", ("f32", "bf16"))
@pytest.mark.parametrize("size", (1e4, 1e11, 1.5e38))
def test_select_large_logits(size, act):
    """Logits far apart: every exp but the largest's is zero or nearly so, the differences reach 3e38, and the sum of
    a row of equal large logits is still ln V."""
    r = np.random.default_rng(8)
    lg = mo.round_act(np.clip(size * r.standard_normal((6, 5003)), -2 * size, 2 * size), act)
    lg[5] = mo.round_act(np.full(1, size), act)[0]
    sc = -np.sort(5 + 10 * r.random((2, 3)), axis=1)
    check(lg, sc, 7, act=act)
    got = check(lg[5:], sc[1:, 2:], 7, act=act)
    assert np.array_equal(got[2][0], np.arange(7))
    assert np.all(np.abs(got[0][0] - (float(np.float32(sc[1, 2])) - np.log(5003))) <= 2.0 ** -23 * 40)


def test_select_long_rows_of_small_terms():
    """A row whose sum is many small terms under one peak, and a nearly flat one: L keeps its digits, so beams whose
    totals lie 1e-6 apart come in the right order."""
    r = np.random.default_rng(8)
    V = 200_001
    lg = mo.round_f32(r.standard_normal((4, V)) * 0.01)
    lg[1, 77] = 12.0
    lg[2] = mo.round_f32(lg[0] + 0.0)
    lg[3, 5] = 14.0
    ref = select_ref(lg, np.zeros((4, 1)), 1)[0]
    sc = -ref.reshape(1, 4).astype(np.float32).astype(np.float64) + np.array([[0.0, 1e-6, -1e-6, 2e-6]])
    check(lg, sc.astype(np.float32).astype(np.float64), 8)


def test_select_strided_and_unaligned_logits():
    for act in ("f32", "bf16"):
        lg, sc = gen(np.random.default_rng(4), 2, 3, 5003, act)
        want = run_select(lg, sc, 9, act=act)
        wide = torch.full((6, 5003 + 10), float("nan"), dtype=DT[act], device=gu.DEV)
        for off in (1, 2, 3, 5):
            wide.fill_(float("nan"))
            view = wide[:, off:off + 5003]
            view.copy_(torch.from_numpy(lg.astype(np.float32)).to(gu.DEV).to(DT[act]))
            got = run_select(lg, sc, 9, act=act, dev_logits=view)
            for a, b in zip(got, want):
                assert np.array_equal(a, b)


def test_select_past_32_bit_offsets():
    """Rows whose elements lie past 2^31 elements from the first: the last row's peak is found."""
    V, W = 1 << 24, 40  # 40 rows of 2^24 bf16 logits spaced 2^26 elements apart would be 5 GB; stride 2^26
    ld = 1 << 26
    lg = torch.zeros(((W - 1) * ld + V,), dtype=torch.bfloat16, device=gu.DEV).as_strided((W, V), (ld, 1))
    lg[W - 1, V - 3] = 8.0
    lg[W - 2, 11] = 7.0
    sc = np.zeros((1, W))
    beam = api.Beam(batch=1, beams=W, vocab=V, n_out=4, act="bf16")
    outs = (torch.zeros((1, 4), device=gu.DEV), torch.zeros((1, 4), dtype=torch.int32, device=gu.DEV),
            torch.zeros((1, 4), dtype=torch.int32, device=gu.DEV))
    api.moe_beam_select(beam, lg, torch.zeros((1, W), device=gu.DEV), *outs, ws=api.beam_workspace(beam, gu.DEV))
    torch.cuda.synchronize()
    assert outs[1].tolist() == [[W - 1, W - 2, 0, 0]] and outs[2].tolist() == [[V - 3, 11, 0, 1]]
    L = np.log(V - 1 + np.exp(8.0))
    assert abs(outs[0][0, 0].item() - (8.0 - L)) <= 2.0 ** -24 * 10 + 2.0 ** -28


# ----------------------------------------------------------------------------- reordering

def reorder_ref(src, dst, parent, B, W):
    out = dst.clone()
    for b in range(B):
        for i in range(W):
            p = int(parent[b, i])
            if 0 <= p < W:
                out[b * W + i] = src[b * W + p]
    return out


def rand_state(r, shape, dtype):
    return torch.from_numpy(r.integers(0, 120, shape)).to(dtype).to(gu.DEV)


@pytest.mark.parametrize("B,W", [(1, 1), (1, 2), (3, 4), (2, 8), (1, 17), (2, 33), (1, 64), (300, 2)])
def test_reorder(B, W):
    r = np.random.default_rng(B * 100 + W)
    rows = B * W
    for trial in range(3):
        parent = torch.from_numpy(r.integers(0, W, (B, W + 2)).astype(np.int32)).to(gu.DEV)
        if trial == 1:
            parent[r.integers(0, B), r.integers(0, W)] = -1
            parent[r.integers(0, B), r.integers(0, W)] = W
        if trial == 2:
            parent[:, :W] = torch.arange(W, device=gu.DEV).roll(1)  # a cycle: every row is read after its place is taken
        for dtype in (torch.uint8, torch.bfloat16, torch.float32):
            base = rand_state(r, (rows, 3, 40, 7), dtype)
            shapes = [base[:, :, :23], base[:, 1], base[:, :, 3:4], base[:, :2, :, 2:3], base[:, 0, 0, 0], base]
            for s in shapes:
                want = reorder_ref(s, s, parent, B, W)
                # out of place, into a dense tensor and into a part of a wider one
                d = torch.full(s.shape, 9, dtype=dtype, device=gu.DEV)
                wide = torch.full(base.shape, 9, dtype=dtype, device=gu.DEV)
                for dst in (d, wide[:, :, :23] if s.shape == shapes[0].shape else d):
                    before = reorder_ref(s, dst, parent, B, W)
                    api.moe_beam_reorder([s], parent, B, W, dst=[dst])
                    torch.cuda.synchronize()
                    assert torch.equal(dst, before)
                assert torch.all(wide[:, :, 23:] == 9)
                keep = base.clone()
                t = keep.as_strided(s.shape, s.stride(), s.storage_offset())
                other = keep.clone()
                other.as_strided(s.shape, s.stride(), s.storage_offset()).copy_(want)
                api.moe_beam_reorder([t], parent, B, W)
                torch.cuda.synchronize()
                assert torch.equal(keep, other)


def test_reorder_many_states_of_all_sizes():
    r = np.random.default_rng(5)
    B, W = 3, 5
    parent = torch.from_numpy(r.integers(0, W, (B, W)).astype(np.int32)).to(gu.DEV)
    states, wants = [], []
    for i in range(75):
        s = rand_state(r, (B * W, int(r.integers(0, 3)) if i % 9 == 0 else 1 + i % 4, int(r.choice([1, 5, 64, 1000, 4096]))),
                       (torch.uint8, torch.int16, torch.float32, torch.int64)[i % 4])
        states.append(s)
        wants.append(reorder_ref(s, s, parent, B, W))
    api.moe_beam_reorder(states, parent, B, W)
    torch.cuda.synchronize()
    for s, w in zip(states, wants):
        assert torch.equal(s, w)
    api.moe_beam_reorder([], parent, B, W)


@pytest.mark.parametrize("W", (3, 40))
def test_reorder_large_rows_at_odd_addresses(W):
    """Rows above 8 KiB whose pieces are no multiple of 16 bytes and start anywhere: in place, and into another buffer
    of another alignment; nothing beside the pieces is written."""
    r = np.random.default_rng(W)
    B = 2
    parent = torch.from_numpy(r.integers(0, W, (B, W)).astype(np.int32)).to(gu.DEV)
    for dtype, shape, part in ((torch.uint8, (4, 4099), (1, 4098)), (torch.uint8, (1, 9001), (3, 9000)),
                               (torch.bfloat16, (213, 37), (2, 35)), (torch.float32, (5, 1003), (1, 1002)),
                               (torch.uint8, (700, 31), (1, 16)), (torch.uint8, (700, 31), (0, 15))):
        base = rand_state(r, (B * W, *shape), dtype)
        s = base[:, :, part[0]:part[1]]
        want = reorder_ref(s, s, parent, B, W)
        dst = torch.full((B * W, shape[0], shape[1] + 2), 5, dtype=dtype, device=gu.DEV)
        d = dst[:, :, 1:1 + part[1] - part[0]]
        api.moe_beam_reorder([s], parent, B, W, dst=[d])
        torch.cuda.synchronize()
        assert torch.equal(d, want)
        d.fill_(5)
        assert torch.all(dst == 5)
        other = base.clone()
        other[:, :, part[0]:part[1]] = want
        api.moe_beam_reorder([s], parent, B, W)
        torch.cuda.synchronize()
        assert torch.equal(base, other)


def test_reorder_past_32_bit_offsets():
    """Rows of 1.5 GB: bytes past 2^32 of a state move."""
    rows, n = 4, 3 << 29
    s = torch.zeros((rows, n), dtype=torch.uint8, device=gu.DEV)
    for i in range(rows):
        s[i, 0], s[i, n - 1], s[i, n // 2 + 1] = 10 + i, 20 + i, 30 + i
    parent = torch.tensor([[3, 0, 0, 1]], dtype=torch.int32, device=gu.DEV)
    d = torch.full_like(s, 1)
    api.moe_beam_reorder([s], parent, 1, 4, dst=[d])
    api.moe_beam_reorder([s], parent, 1, 4)
    torch.cuda.synchronize()
    for t in (s, d):
        assert t[:, 0].tolist() == [13, 10, 10, 11]
        assert t[:, n - 1].tolist() == [23, 20, 20, 21]
        assert t[:, n // 2 + 1].tolist() == [33, 30, 30, 31]
        assert [int(t[i].sum(dtype=torch.int64)) for i in range(4)] == [69, 60, 60, 63]


# ----------------------------------------------------------------------------- together

def test_beam_search_steps():
    """Six steps of a toy model: hidden states -> packed head -> selection -> reordered states and finished flags, eager
    and from a captured step, against the same search in 64 bits on the CPU.  The CPU search takes the device's logits
    (held to the projection's bound on the way), so every parent and token has to match."""
    r = np.random.default_rng(12)
    B, W, H, V, n, eos = 3, 4, 128, 1501, 8, 7
    u = r.integers(0, 16, (V, H)).astype(np.uint8)
    s16 = (0.05 * (0.5 + r.random((V, H // 32)))).astype(np.float16)
    w = mo.dequant(synth.pack_q4(u), s16.view(np.uint16), None, "q4_sym_g32")
    emb = mo.round_bf16(r.standard_normal((V, H)))
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(gu.DEV)
    lin = api.Linear(rows=V, cols=H, qfmt="q4_sym_g32", act="bf16", codes=dev(synth.pack_q4(u)), scales=dev(s16.view(np.int16)))
    beam = api.Beam(batch=B, beams=W, vocab=V, n_out=n, eos=eos)
    ws = api.beam_workspace(beam, gu.DEV)
    rows = B * W
    for captured in (False, True):
        x = torch.zeros((rows, H), dtype=torch.bfloat16, device=gu.DEV)
        cache = torch.zeros((rows, 2, 16, 3), dtype=torch.bfloat16, device=gu.DEV)
        tokens = torch.full((rows, 8), -1, dtype=torch.int32, device=gu.DEV)
        scores = torch.full((B, W), float("-inf"), device=gu.DEV)
        fin = torch.zeros((B, W), dtype=torch.uint8, device=gu.DEV)
        logits = torch.zeros((rows, V), device=gu.DEV)
        outs = (torch.zeros((B, n), device=gu.DEV), torch.zeros((B, n), dtype=torch.int32, device=gu.DEV),
                torch.zeros((B, n), dtype=torch.int32, device=gu.DEV))
        emb_d = dev(emb.astype(np.float32)).bfloat16()

        def step():
            api.moe_linear_q(lin, x, rows, logits)
            api.moe_beam_select(beam, logits, scores, *outs, finished=fin, ws=ws)
            api.moe_beam_reorder([x, cache, tokens, fin.view(rows, 1)], outs[1], B, W)
            scores.copy_(outs[0][:, :W])

        x0 = mo.round_bf16(r.standard_normal((B, 1, H)).repeat(W, axis=1).reshape(rows, H))

        def reset():
            x.copy_(dev(x0.astype(np.float32)).bfloat16())
            cache.copy_(torch.arange(rows, device=gu.DEV).view(rows, 1, 1, 1).expand_as(cache))
            tokens.fill_(-1)
            scores.fill_(float("-inf"))
            scores[:, 0] = 0.0
            fin.zero_()

        reset()
        step()
        torch.cuda.synchronize()
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=torch.cuda.Stream()):
                step()
        reset()
        cx, ctok = x0.copy(), [[] for _ in range(rows)]
        cid = np.arange(rows)
        csc = np.full((B, W), -np.inf)
        csc[:, 0] = 0.0
        cfin = np.zeros((B, W), bool)
        for i in range(6):
            g.replay() if captured else step()
            torch.cuda.synchronize()
            lg = logits.cpu().numpy().astype(np.float64)
            ref = cx @ w.T
            assert np.abs(lg - ref).max() <= 1e-4 * np.sqrt(np.mean(ref ** 2))
            t, p, k = select_ref(lg, csc, n, cfin, eos)
            assert np.array_equal(outs[1].cpu().numpy(), p) and np.array_equal(outs[2].cpu().numpy(), k), (captured, i)
            flat = (np.arange(B)[:, None] * W + p[:, :W]).reshape(-1)
            cx, cid = cx[flat], cid[flat]
            ctok = [ctok[f] + [int(v)] for f, v in zip(flat, k[:, :W].reshape(-1))]
            cfin = np.take_along_axis(cfin, p[:, :W], 1) | (k[:, :W] == eos)
            csc = outs[0][:, :W].cpu().numpy().astype(np.float64)
            # the host's part of a step: the new token enters its beam
            last = outs[2][:, :W].reshape(-1)
            assert torch.equal(x.float().cpu(), torch.from_numpy(cx.astype(np.float32)))
            assert torch.equal(cache[:, 0, 0, 0].cpu().long(), torch.from_numpy(cid))
            tokens[:, i] = last
            fin |= (outs[2][:, :W] == eos).to(torch.uint8)
            x.copy_((x.float() * 0.5 + emb_d[last.long()].float()).bfloat16())
            cx = mo.round_bf16(cx * 0.5 + emb[k[:, :W].reshape(-1)])
            assert tokens[:, :i + 1].tolist() == ctok
            assert np.array_equal(fin.cpu().numpy().astype(bool), cfin)


def test_scores_updated_in_place():
    """out_score may be scores (n_out == beams), with more sequences than fit the chip at once."""
    r = np.random.default_rng(12)
    B, W, V = 600, 4, 700
    lg, sc = gen(r, B, W, V, "f32")
    want = run_select(lg, sc, W)
    beam = api.Beam(batch=B, beams=W, vocab=V, n_out=W)
    s = torch.from_numpy(sc.astype(np.float32)).to(gu.DEV)
    outs = (torch.zeros((B, W), dtype=torch.int32, device=gu.DEV), torch.zeros((B, W), dtype=torch.int32, device=gu.DEV))
    api.moe_beam_select(beam, torch.from_numpy(lg.astype(np.float32)).to(gu.DEV), s, s, *outs,
                        ws=api.beam_workspace(beam, gu.DEV))
    torch.cuda.synchronize()
    for got, w in zip((s, *outs), want):
        assert np.array_equal(got.cpu().numpy(), w)


def test_captured_selections_do_not_share_a_workspace():
    """Two captured selections with a workspace each, replayed on two streams at once, keep their eager results."""
    r = np.random.default_rng(31)
    made = []
    for i, (B, W, V, n) in enumerate(((2, 4, 30011, 8), (4, 2, 20001, 4))):
        lg, sc = gen(r, B, W, V, "f32")
        want = run_select(lg, sc, n)
        beam = api.Beam(batch=B, beams=W, vocab=V, n_out=n)
        ws = api.beam_workspace(beam, gu.DEV)
        ld, sd = torch.from_numpy(lg.astype(np.float32)).to(gu.DEV), torch.from_numpy(sc.astype(np.float32)).to(gu.DEV)
        outs = (torch.zeros((B, n), device=gu.DEV), torch.zeros((B, n), dtype=torch.int32, device=gu.DEV),
                torch.zeros((B, n), dtype=torch.int32, device=gu.DEV))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=torch.cuda.Stream()):
            api.moe_beam_select(beam, ld, sd, *outs, ws=ws)
        made.append((g, torch.cuda.Stream(), outs, want, (ld, sd, ws)))
    for rep in range(4):
        for g, st, outs, _, _ in made:
            for o in outs:
                o.fill_(5)
        torch.cuda.synchronize()
        for g, st, _, _, _ in made:
            with torch.cuda.stream(st):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for _, _, outs, want, _ in made:
            for o, w in zip(outs, want):
                assert np.array_equal(o.cpu().numpy(), w)
