"""What the dense and decoding operators are measured on.

Three operators that a serving program calls next to the routed layer: a dense
projection with packed weights (``linear_q``), the selection of a beam search's
next tokens (``beam_select``) and the move of the beams' states to follow their
parents (``beam_reorder``).  ``run`` computes them in elementary torch
operations, or, where ``own`` is true, through the library's entry points.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
GROUP = 32
BITS = {"q4_sym_g32": 4, "q3_sym_g32": 3, "q2_asym_g32": 2}
ZERO = {"q4_sym_g32": 8, "q3_sym_g32": 4}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _linear(name, tokens, cols, rows, qfmt, act="bf16", out="f32", bias=False):
    return dict(name=name, op="linear_q", tokens=tokens, cols=cols, rows=rows, qfmt=qfmt, act=act, out=out, bias=bias)


def _select(name, batch, beams, vocab, n_out, act="f32", finished=0, mask="none"):
    return dict(name=name, op="beam_select", batch=batch, beams=beams, vocab=vocab, n_out=n_out, act=act,
                finished=finished, mask=mask)


def _reorder(name, batch, beams, states, heads, room, used, dim, in_place=False):
    return dict(name=name, op="beam_reorder", batch=batch, beams=beams, states=states, heads=heads, room=room,
                used=used, dim=dim, in_place=in_place)


def listed():
    return [
        # a projection of one decoded token: the smallest call, where the launch and one trip to memory count
        _linear("linear_q4_T1_square", 1, 2048, 2048, "q4_sym_g32", out="bf16"),
        # the output head for one token: streams the largest matrix of a model
        _linear("linear_q4_T1_head", 1, 2048, 131072, "q4_sym_g32"),
        # three rows of fp32 activations through a small projection with a bias
        _linear("linear_q4_T3_f32", 3, 768, 2048, "q4_sym_g32", act="f32", bias=True),
        # the output head for a verify batch (1 + 4 drafted tokens), 2-bit weights
        _linear("linear_q2_T5_head", 5, 2048, 65536, "q2_asym_g32"),
        # a batch of 13 sequences, an odd vocabulary and an odd number of groups, 3-bit weights
        _linear("linear_q3_T13_odd", 13, 2016, 50021, "q3_sym_g32", bias=True),
        # a batch of 64 sequences through a wide projection
        _linear("linear_q4_T64_wide", 64, 4096, 16384, "q4_sym_g32", out="bf16"),
        # a prompt of 1000 tokens through the same kind of projection
        _linear("linear_q4_T1000_prompt", 1000, 2048, 8192, "q4_sym_g32", out="bf16"),
        # one sequence with four beams: the smallest selection
        _select("select_b1_w4", 1, 4, 32768, 8),
        # 32 sequences with 8 beams over a large vocabulary, twice as many candidates as beams
        _select("select_b32_w8", 32, 8, 131072, 16),
        # a ragged batch: bf16 logits (many equal values), finished beams, a mask of allowed tokens for each row
        _select("select_b3_w5_masked", 3, 5, 50021, 10, act="bf16", finished=1, mask="rows"),
        # the states of a few layers, moved in place: beams that stay keep their slot
        _reorder("reorder_in_place", 2, 4, 8, 1, 2048, 2048, 1, in_place=True),
        # caches of 8 sequences with 8 beams, two thirds full, copied into the other half of a double buffer
        _reorder("reorder_cache", 8, 8, 12, 4, 768, 517, 128),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    caps = {}
    for c in listed():
        w = work(c)
        cap = caps.setdefault(c["op"], [0, 0])
        cap[0], cap[1] = max(cap[0], w["bytes"]), max(cap[1], w["flops"])
    op = rng.choice(["linear_q", "linear_q", "linear_q", "beam_select", "beam_select", "beam_reorder"])
    while True:
        if op == "linear_q":
            c = _linear("", _log_int(rng, 1, 1000), GROUP * _log_int(rng, 1, 256), _log_int(rng, 1, 131072),
                        rng.choice(list(BITS)), rng.choice(["bf16", "bf16", "f32"]), rng.choice(["f32", "bf16"]),
                        rng.random() < 0.3)
        elif op == "beam_select":
            beams = _log_int(rng, 1, 32)
            vocab = _log_int(rng, 100, 200000)
            c = _select("", _log_int(rng, 1, 32), beams, vocab, min(vocab, rng.randint(beams, 2 * beams)),
                        rng.choice(["f32", "bf16"]), rng.randint(0, beams // 2), rng.choice(["none", "one", "rows"]))
        else:
            room = _log_int(rng, 1, 2048)
            c = _reorder("", _log_int(rng, 1, 16), _log_int(rng, 1, 32), rng.randint(1, 40), rng.choice([1, 2, 3, 8]),
                         room, rng.randint(1, room), rng.choice([1, 33, 64, 96, 128]), rng.random() < 0.3)
        w = work(c)
        # an fp32 activation is three bf16 parts of work
        if w["bytes"] <= caps[op][0] and w["flops"] * (3 if c.get("act") == "f32" and op == "linear_q" else 1) <= caps[op][1]:
            del c["name"]
            return c


def work(case):
    c = case
    if c["op"] == "linear_q":
        t, k, n = c["tokens"], c["cols"], c["rows"]
        planes = 2 if c["qfmt"] == "q2_asym_g32" else 1
        weights = n * k * BITS[c["qfmt"]] // 8 + planes * 2 * n * (k // GROUP)
        size = lambda a: 2 if a == "bf16" else 4
        return {"bytes": weights + t * k * size(c["act"]) + t * n * size(c["out"]) + (4 * n if c["bias"] else 0),
                "flops": 2 * t * n * k}
    if c["op"] == "beam_select":
        rows = c["batch"] * (c["beams"] - c["finished"])
        masks = {"none": 0, "one": 1, "rows": rows}[c["mask"]] * ((c["vocab"] + 31) // 32) * 4
        return {"bytes": rows * c["vocab"] * (2 if c["act"] == "bf16" else 4) + masks + c["batch"] * c["n_out"] * 12,
                "flops": 3 * rows * c["vocab"]}
    row = c["heads"] * c["used"] * c["dim"] * 2
    stay = _survivors(c["beams"])  # distinct parents of each sequence
    written = c["beams"] - stay if c["in_place"] else c["beams"]
    read = min(stay, written) if c["in_place"] else stay
    return {"bytes": c["batch"] * c["states"] * (read + written) * row, "flops": 0}


def _survivors(beams):
    return (beams + 1) // 2


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed & 0x7FFFFFFFFFFF)
    return g


def _pack(u, qfmt):
    """Codes [rows][cols] (uint8 values) to the packed bytes of a format."""
    n, k = u.shape
    if qfmt == "q4_sym_g32":
        return u[:, 0::2] | (u[:, 1::2] << 4)
    low = u & 3
    two = low[:, 0::4] | (low[:, 1::4] << 2) | (low[:, 2::4] << 4) | (low[:, 3::4] << 6)
    if qfmt == "q2_asym_g32":
        return two
    h = (u >> 2).view(n, k // 8, 8)
    top = h[..., 0].clone()
    for i in range(1, 8):
        top |= h[..., i] << i
    g = k // GROUP
    return torch.cat([two.view(n, g, 8), top.view(n, g, 4)], dim=2).reshape(n, g * 12)


def _prepare_linear(c, seed):
    g = _gen(seed)
    n, k, t, qfmt = c["rows"], c["cols"], c["tokens"], c["qfmt"]
    top = (1 << BITS[qfmt]) - 1
    mid = ZERO.get(qfmt, 1.5)
    codes = torch.empty((n, k * BITS[qfmt] // 8), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // k)
    for r in range(0, n, step):  # codes of normally distributed weights
        m = min(step, n - r)
        u = torch.randn((m, k), device=DEV, generator=g).mul_(top / 5.0).add_(mid).round_().clamp_(0, top)
        codes[r:r + m] = _pack(u.to(torch.uint8), qfmt)
    scales = (0.1 / (top + 1) * (0.6 + 0.8 * torch.rand((n, k // GROUP), device=DEV, generator=g))).half()
    mins = (-1.5 * scales.float() * (0.9 + 0.2 * torch.rand(scales.shape, device=DEV, generator=g))).half() \
        if qfmt == "q2_asym_g32" else None
    x = torch.randn((t, k), device=DEV, generator=g)
    x *= torch.where(torch.rand(k, device=DEV, generator=g) < 0.01, 12.0, 1.0)  # a few channels are large in earnest
    x = x.to(TYPES[c["act"]])
    bias = torch.randn(n, device=DEV, generator=g) if c["bias"] else None
    st = dict(case=c, codes=codes, scales=scales, mins=mins, x=x, bias=bias)
    if own:
        from sparse_moe_router_amd import api
        y = torch.empty((t, n), dtype=TYPES[c["out"]], device=DEV)
        lin = api.Linear(rows=n, cols=k, qfmt=qfmt, act=c["act"], out=c["out"], codes=codes,
                         scales=scales.view(torch.int16), mins=None if mins is None else mins.view(torch.int16),
                         bias=bias)
        st.update(y=y, call=api.bind_linear_q(lin, x, t, y))
    return st


def _prepare_select(c, seed):
    g = _gen(seed)
    b, w, v = c["batch"], c["beams"], c["vocab"]
    rows = b * w
    logits = torch.randn((rows, v), device=DEV, generator=g).mul_(2.2)
    peaks = torch.randint(0, v, (rows, 24), device=DEV, generator=g)  # the tokens a model finds likely
    logits.scatter_add_(1, peaks, 3.0 + 9.0 * torch.rand((rows, 24), device=DEV, generator=g))
    logits = logits.to(TYPES[c["act"]])
    scores = -5.0 - 10.0 * torch.rand((b, 1), device=DEV, generator=g) - 3.0 * torch.rand((b, w), device=DEV, generator=g)
    scores = torch.sort(scores, dim=1, descending=True).values.contiguous()
    finished = torch.zeros((b, w), dtype=torch.uint8, device=DEV)
    if c["finished"]:
        pick = torch.rand((b, w), device=DEV, generator=g).argsort(dim=1)[:, :c["finished"]]
        finished.scatter_(1, pick, 1)
    eos = int(torch.randint(0, v, (1,), device=DEV, generator=g))
    allowed = None
    if c["mask"] != "none":  # a grammar allows a part of the vocabulary
        r = rows if c["mask"] == "rows" else 1
        words = (v + 31) // 32
        bits = torch.randint(0, 1 << 32, (r, words), device=DEV, generator=g, dtype=torch.int64)
        bits &= torch.randint(0, 1 << 32, (r, words), device=DEV, generator=g, dtype=torch.int64)
        if c["mask"] == "rows" and rows > 2:
            bits[rows - 1] = 0  # a beam that the grammar leaves nothing
        allowed = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
        # what stands in masked places is never looked at
        bad = ~_allowed_mask(allowed, v).expand(rows, v) & (torch.rand((rows, v), device=DEV, generator=g) < 0.01)
        logits.masked_fill_(bad, float("nan"))
    st = dict(case=c, logits=logits, scores=scores, finished=finished, eos=eos, allowed=allowed)
    if own:
        from sparse_moe_router_amd import api
        n = c["n_out"]
        outs = (torch.empty((b, n), dtype=torch.float32, device=DEV), torch.empty((b, n), dtype=torch.int32, device=DEV),
                torch.empty((b, n), dtype=torch.int32, device=DEV))
        beam = api.Beam(batch=b, beams=w, vocab=v, n_out=n, act=c["act"], eos=eos)
        ws = api.beam_workspace(beam, DEV)
        st.update(outs=outs, call=api.bind_beam_select(beam, logits, scores, *outs, finished=finished, allowed=allowed,
                                                       ws=ws))
    return st


def _prepare_reorder(c, seed):
    g = _gen(seed)
    b, w = c["batch"], c["beams"]
    shape = (b * w, c["heads"], c["room"], c["dim"])
    full = [torch.randn(shape, device=DEV, generator=g).to(torch.bfloat16) for _ in range(c["states"])]
    src = [t[:, :, :c["used"]] for t in full]
    # half of the beams go on; each keeps its slot, the others' slots are taken by copies of them
    order = torch.rand((b, w), device=DEV, generator=g).argsort(dim=1)[:, :_survivors(w)]
    parent = torch.gather(order, 1, torch.randint(0, order.shape[1], (b, w), device=DEV, generator=g))
    parent.scatter_(1, order, order)
    parent = parent.to(torch.int32).contiguous()
    dst = src if c["in_place"] else [torch.zeros_like(t)[:, :, :c["used"]] for t in full]
    st = dict(case=c, src=src, dst=dst, parent=parent)
    if own:
        from sparse_moe_router_amd import api
        st["call"] = api.bind_beam_reorder(src, parent, b, w, dst=None if c["in_place"] else dst)
    return st


def prepare(case, seed):
    return {"linear_q": _prepare_linear, "beam_select": _prepare_select, "beam_reorder": _prepare_reorder}[case["op"]](
        case, seed)


# ------------------------------------------------------------------ plain forms

def _codes(codes, qfmt, dtype):
    """The codes u of packed rows as numbers [rows][cols]."""
    if qfmt == "q4_sym_g32":
        return torch.stack([codes & 15, codes >> 4], dim=2).flatten(1).to(dtype)
    if qfmt == "q2_asym_g32":
        return torch.stack([(codes >> s) & 3 for s in (0, 2, 4, 6)], dim=2).flatten(1).to(dtype)
    rows = codes.shape[0]
    grp = codes.view(rows, -1, 12)
    low = torch.stack([(grp[..., :8] >> s) & 3 for s in (0, 2, 4, 6)], dim=3).flatten(2)
    top = torch.stack([(grp[..., 8:] >> s) & 1 for s in range(8)], dim=3).flatten(2)
    return (low + 4 * top).flatten(1).to(dtype)


def _plain_linear(st):
    c = st["case"]
    n, k = c["rows"], c["cols"]
    u = _codes(st["codes"], c["qfmt"], torch.float32).view(n, k // GROUP, GROUP)
    s = st["scales"].float().unsqueeze(2)
    w = u * s + st["mins"].float().unsqueeze(2) if st["mins"] is not None else (u - ZERO[c["qfmt"]]) * s
    y = st["x"].float() @ w.view(n, k).t()
    if st["bias"] is not None:
        y = y + st["bias"]
    return y.to(TYPES[c["out"]])


def _allowed_mask(allowed, vocab):
    bit = torch.arange(32, device=allowed.device, dtype=torch.int32)
    return (((allowed.unsqueeze(2) >> bit) & 1) != 0).flatten(1)[:, :vocab]


def _plain_select(st):
    """In 64 bits: totals of different beams lie next to each other."""
    c = st["case"]
    b, w, v, n = c["batch"], c["beams"], c["vocab"], c["n_out"]
    none = float("-inf")
    lg = st["logits"].double()
    if st["allowed"] is not None:
        lg = torch.where(_allowed_mask(st["allowed"], v).expand(b * w, v), lg, none)
    top = lg.amax(dim=1, keepdim=True)
    lse = top + torch.log(torch.exp(lg - top).sum(dim=1, keepdim=True))
    score = st["scores"].double().view(b * w, 1)
    total = score + (lg - lse)
    total = torch.where(torch.isfinite(lse) & torch.isfinite(score), total, none)
    done = st["finished"].view(b * w, 1) != 0
    token = torch.arange(v, device=lg.device)
    total = torch.where(done, torch.where(token == st["eos"], score, none), total).view(b, w * v)
    best, index = torch.sort(total, dim=1, descending=True, stable=True)
    best, index = best[:, :n], index[:, :n]
    empty = best == none
    parent = torch.where(empty, -1, index // v).to(torch.int32)
    tok = torch.where(empty, -1, index % v).to(torch.int32)
    return best.float(), parent, tok


def _plain_reorder(st):
    c = st["case"]
    b, w = c["batch"], c["beams"]
    rows = (torch.arange(b, device=DEV).unsqueeze(1) * w + st["parent"]).view(-1)
    for s, d in zip(st["src"], st["dst"]):
        d.copy_(s[rows])
    return st["dst"]


def run(state):
    op = state["case"]["op"]
    if own:
        state["call"]()
        return {"linear_q": lambda: state["y"], "beam_select": lambda: state["outs"],
                "beam_reorder": lambda: state["dst"]}[op]()
    return {"linear_q": _plain_linear, "beam_select": _plain_select, "beam_reorder": _plain_reorder}[op](state)


# ------------------------------------------------------------------ 64 bits

def _exact_linear(st):
    c = st["case"]
    n, k = c["rows"], c["cols"]
    x = st["x"].double()
    y = torch.empty((c["tokens"], n), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 25) // k)
    for r in range(0, n, step):
        sl = slice(r, min(n, r + step))
        u = _codes(st["codes"][sl], c["qfmt"], torch.float64)
        s = st["scales"][sl].double().repeat_interleave(GROUP, dim=1)
        if st["mins"] is None:
            w = s * (u - ZERO[c["qfmt"]])
        else:  # the format rounds a 2-bit weight once to fp32
            w = (s * u + st["mins"][sl].double().repeat_interleave(GROUP, dim=1)).float().double()
        y[:, sl] = x @ w.t()
    return y if st["bias"] is None else y + st["bias"].double()


def _exact_select(st):
    c = st["case"]
    b, w, v, n = c["batch"], c["beams"], c["vocab"], c["n_out"]
    out_s = torch.full((b, n), float("-inf"), dtype=torch.float64)
    out_p = torch.full((b, n), -1, dtype=torch.int32)
    out_t = torch.full((b, n), -1, dtype=torch.int32)
    scores, finished = st["scores"].double().cpu(), st["finished"].cpu()
    for i in range(b):
        found = []  # (total, flat index) of each beam's best
        for j in range(w):
            s = float(scores[i, j])
            if finished[i, j]:
                found.append((s, j * v + st["eos"]))
                continue
            row = st["logits"][i * w + j].double()
            ids = torch.arange(v, device=DEV)
            if st["allowed"] is not None:
                words = st["allowed"][i * w + j if st["allowed"].shape[0] > 1 else 0].long()
                ids = ids[((words[ids // 32] >> (ids % 32)) & 1) == 1]
                row = row[ids]
            if row.numel() == 0:
                continue
            total = s + (row - torch.logsumexp(row, 0))
            edge = torch.topk(total, min(n, total.numel())).values[-1]
            near = total >= edge  # every value equal to the last one too
            found += list(zip(total[near].tolist(), (j * v + ids[near]).tolist()))
        found.sort(key=lambda e: (-e[0], e[1]))
        for q, (s, flat) in enumerate(found[:n]):
            out_s[i, q], out_p[i, q], out_t[i, q] = s, flat // v, flat % v
    return out_s.to(DEV), out_p.to(DEV), out_t.to(DEV)


def _exact_reorder(st):
    c = st["case"]
    parent = st["parent"].cpu().tolist()
    outs = []
    for s in st["src"]:
        d = torch.empty(s.shape, dtype=torch.float64, device=DEV)
        for i in range(c["batch"]):
            for j, p in enumerate(parent[i]):
                d[i * c["beams"] + j] = s[i * c["beams"] + p].double()
        outs.append(d)
    return outs


def exact(case, seed):
    st = prepare(case, seed)
    return {"linear_q": _exact_linear, "beam_select": _exact_select, "beam_reorder": _exact_reorder}[case["op"]](st)
