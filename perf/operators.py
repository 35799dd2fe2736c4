"""Workloads of the 8-bit activation checkpoints and of the preference loss:
the calls a preference-tuning step over QLoRA adapters makes around the
linear layer, each beside its plain form in elementary torch operations.

Kinds of cases:

* ``act8``: an activation goes into an 8-bit checkpoint (one signed code per
  element, one fp32 scale per 64 columns of a row) and comes back, as between
  a layer's forward and its backward; returns the restored activation and the
  scales.
* ``bwd``: the backward of a QLoRA linear layer whose input was kept as such
  a checkpoint: dX (left out for a first layer, whose input needs no
  gradient), dA and dB.
* ``logprob``: log-probabilities of packed sequences of different lengths
  under given logits, as the reference pass of preference tuning needs them.
* ``pref``: the paired log-ratio loss, forward and backward: one loss per
  pair and the gradient of the mean loss with respect to the logits.
"""

import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decoded token of a 4096-wide model: latency alone
        dict(name="act8_1x4096", kind="act8", rows=1, cols=4096, x="bf16", y="bf16"),
        # the 4096-token input of a 7B-class gate projection
        dict(name="act8_4096x4096", kind="act8", rows=4096, cols=4096, x="bf16", y="bf16"),
        # the input of a 70B-class down projection, kept in fp32 by its producer
        dict(name="act8_2048x28672_f32", kind="act8", rows=2048, cols=28672, x="f32", y="bf16"),
        # a few tokens through a 7B-class attention projection
        dict(name="bwd_q7b_16", kind="bwd", m=16, n=4096, k=4096, r=16, dx="bf16"),
        # the 7B-class gate projection, 4096 tokens
        dict(name="bwd_gate7b", kind="bwd", m=4096, n=11008, k=4096, r=16, dx="bf16"),
        # a 70B-class first layer: only the adapters get gradients
        dict(name="bwd_q70b_adapters", kind="bwd", m=2048, n=8192, k=8192, r=64, dx="none"),
        # a ragged batch through a 70B-class k / v projection, fp32 dX
        dict(name="bwd_k70b_1003", kind="bwd", m=1003, n=1024, k=8192, r=24, dx="f32"),
        # two short answers under a 32000-word vocabulary: latency
        dict(name="logprob_2x12", kind="logprob", seqs=2, length=12, vocab=32000, pad=0, x="bf16"),
        # the reference pass of a batch of 8 pairs
        dict(name="logprob_16x256", kind="logprob", seqs=16, length=256, vocab=32000, pad=0, x="bf16"),
        # one pair of short answers, odd vocabulary padded to the head's rows
        dict(name="pref_1x40_odd", kind="pref", seqs=2, length=40, vocab=50257, pad=7, x="bf16", d="bf16"),
        # a training batch of 8 pairs
        dict(name="pref_8x256", kind="pref", seqs=16, length=256, vocab=32000, pad=0, x="bf16", d="bf16"),
        # long answers under a large vocabulary, fp32 logits, bf16 gradient
        dict(name="pref_2x600_large", kind="pref", seqs=4, length=600, vocab=128256, pad=0, x="f32", d="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["act8", "bwd", "bwd", "logprob", "pref", "pref"])
    if kind == "act8":
        cols = _log(rng, 64, 28672)
        rows = _log(rng, 1, min(16384, 2048 * 28672 // cols))
        x = rng.choice(["bf16", "bf16", "f32"])
        # an fp32 input rounds 127 x once before its quotient, so a code next
        # to a half step may be one off its definition in 64 bits: below what
        # bf16 resolves, but not below fp32
        return dict(kind=kind, rows=rows, cols=cols, x=x,
                    y="bf16" if x == "f32" else rng.choice(["bf16", "f32"]))
    if kind == "bwd":
        n, k = 8 * _log(rng, 8, 1376), 64 * _log(rng, 1, 128)
        m = _log(rng, 1, min(4096, 4096 * 11008 * 4096 // (n * k)))
        return dict(kind=kind, m=m, n=n, k=k, r=rng.choice([4, 8, 16, 24, 32, 64]),
                    dx=rng.choice(["bf16", "bf16", "f32", "none"]))
    vocab = _log(rng, 1000, 128256)
    seqs = 2 * _log(rng, 1, 16)
    length = _log(rng, 1, max(1, min(2048, 2400 * 128256 // (2 * vocab * seqs))))
    case = dict(kind=kind, seqs=seqs, length=length, vocab=vocab, pad=-vocab % 8,
                x=rng.choice(["bf16", "bf16", "f32"]))
    if kind == "pref":
        case["d"] = "bf16" if case["x"] == "bf16" else rng.choice(["bf16", "f32"])
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

BETA, SMOOTH = 0.1, 0.05


def _levels():
    """The 16 NF4 levels: normal quantiles, 8 above zero, 7 below, and 0."""
    delta = 1 - 0.5 * (1 / 32 + 1 / 30)
    pos = torch.tensor([delta - i * (delta - 0.5) / 8 for i in range(8)], dtype=torch.float64)
    neg = torch.tensor([delta - i * (delta - 0.5) / 7 for i in range(7)], dtype=torch.float64)
    q = torch.cat([-torch.special.ndtri(neg), torch.zeros(1, dtype=torch.float64),
                   torch.special.ndtri(pos).flip(0)])
    return (q / q[-1]).to(torch.float32)


def _nf4(n, k, g):
    """A normal weight as NF4 codes (two per byte), 8-bit block constants and
    one fp32 scale per 256 blocks."""
    w = torch.randn(n * k // 64, 64, device=DEV, generator=g) * 0.02
    c = w.abs().amax(1, keepdim=True)
    lv = _levels().to(DEV)
    mid = ((lv[1:].double() + lv[:-1].double()) / 2).float()
    code = torch.bucketize(w / c, mid).to(torch.uint8).view(-1, 2)
    packed = code[:, 0] | (code[:, 1] << 4)
    blocks = c.numel()
    cg = torch.nn.functional.pad(c.view(-1), (0, -blocks % 256)).view(-1, 256)
    d = cg.amax(1) / 255
    q = torch.round(cg / d[:, None]).clamp_(max=255).to(torch.uint8).view(-1)[:blocks]
    return packed.contiguous(), q.contiguous(), d.contiguous()


def _activation(rows, cols, dtype, g):
    """Normal values with a per-column gain and a few outlier columns, as
    after a norm layer."""
    gain = 0.5 + torch.rand(cols, device=DEV, generator=g)
    gain[torch.randint(0, cols, (max(1, cols // 512),), device=DEV, generator=g)] *= 20
    return (torch.randn(rows, cols, device=DEV, generator=g) * gain).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    s = dict(case)
    if case["kind"] == "act8":
        s["xt"] = _activation(case["rows"], case["cols"], DTYPES[case["x"]], g)
    elif case["kind"] == "bwd":
        m, n, k, r = case["m"], case["n"], case["k"], case["r"]
        s["packed"], s["qabs"], s["gscale"] = _nf4(n, k, g)
        x = _activation(m, k, torch.bfloat16, g)
        blocks = x.float().view(m, k // 64, 64)
        s["scale"] = (blocks.abs().amax(2) / 127).contiguous()
        s["codes"] = torch.round(blocks / s["scale"][:, :, None]).to(torch.int8).view(m, k)
        s["A"] = (torch.randn(r, k, device=DEV, generator=g) / math.sqrt(k)).bfloat16()
        s["B"] = (torch.randn(n, r, device=DEV, generator=g) * 0.05).bfloat16()
        s["dy"] = torch.randn(m, n, device=DEV, generator=g).bfloat16()
        s["T"] = x.float() @ s["A"].float().t()
    else:
        S, V, ld = case["seqs"], case["vocab"], case["vocab"] + case["pad"]
        # ragged lengths from half to one and a half of the case's (its own,
        # so that every seed has the same shapes), and a prompt of a third of
        # every sequence whose tokens do not count (label -100)
        span = (torch.arange(1, S + 1, device=DEV, dtype=torch.float64) * 0.6180339887) % 1.0
        lens = (case["length"] * (0.5 + span)).round().long().clamp_(min=1)
        off = torch.nn.functional.pad(lens.cumsum(0), (1, 0))
        T = int(off[-1])
        seg = torch.searchsorted(off, torch.arange(T, device=DEV), right=True) - 1
        label = torch.randint(0, V, (T,), device=DEV, generator=g)
        prompt = torch.arange(T, device=DEV) - off[seg] < lens[seg] // 3
        s["labels"] = torch.where(prompt, -100, label)
        s["offsets"] = off
        # peaked rows: a trained head gives the next word a few nats more
        logits = torch.randn(T, ld, device=DEV, generator=g) * 2
        logits.scatter_add_(1, label[:, None], 6 + 2 * torch.randn(T, 1, device=DEV, generator=g))
        s["logits"] = logits.to(DTYPES[case["x"]])
        if case["kind"] == "pref":
            # reference log-probabilities a few nats from the policy's
            logp = _logprob_plain(s)[0]
            s["ref"] = (logp + 3 * torch.randn(S, device=DEV, generator=g)).contiguous()
            s["dlogits"] = torch.zeros(T, ld, device=DEV, dtype=DTYPES[case["d"]])
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _act8_plain(s):
    rows, cols = s["rows"], s["cols"]
    pad = -cols % 64
    x = torch.nn.functional.pad(s["xt"].float(), (0, pad)).view(rows, -1, 64)
    a = x.abs().amax(2, keepdim=True)
    # 127 x / a, both divided by 256 so that no product overflows
    code = torch.round((x * (127 / 256)) / (a / 256))
    code = torch.where(a < 2.0 ** -100, torch.zeros_like(code), code).to(torch.int8)
    scale = torch.where(a < 2.0 ** -100, torch.zeros_like(a), a / 127)
    y = (code.float() * scale).view(rows, -1)[:, :cols].to(DTYPES[s["y"]])
    return y, scale.squeeze(2)


def _weight_plain(s):
    n, k = s["n"], s["k"]
    code = torch.stack([s["packed"] & 15, s["packed"] >> 4], 1).view(-1, 64).long()
    cp = s["qabs"].float() * s["gscale"].repeat_interleave(256)[:s["qabs"].numel()]
    return (_levels().to(DEV)[code] * cp[:, None]).bfloat16().float().view(n, k)


def _bwd_plain(s):
    m, k = s["m"], s["k"]
    sc = 32.0 / s["r"]
    x = (s["codes"].float().view(m, -1, 64) * s["scale"][:, :, None]).bfloat16().float().view(m, k)
    dy, A, B = s["dy"].float(), s["A"].float(), s["B"].float()
    G = dy @ B
    dA = sc * (G.t() @ x)
    dB = sc * (dy.t() @ s["T"])
    if s["dx"] == "none":
        return dA, dB
    dx = dy @ _weight_plain(s) + sc * (G @ A)
    return dx.to(DTYPES[s["dx"]]), dA, dB


def _logprob_plain(s):
    """(logp of each sequence, lse of each row, log-softmax shift of rows)."""
    x = s["logits"][:, :s["vocab"]].float()
    mx = x.amax(1, keepdim=True)
    total = torch.exp(x - mx).sum(1)
    on = s["labels"] >= 0
    lab = torch.where(on, s["labels"], torch.zeros_like(s["labels"]))
    hit = x.gather(1, lab[:, None]).squeeze(1).double()
    lse = mx.squeeze(1).double() + torch.log(total.double())
    tok = torch.where(on, hit - lse, torch.zeros_like(lse))
    T = lab.numel()
    seg = torch.searchsorted(s["offsets"], torch.arange(T, device=DEV), right=True) - 1
    logp = torch.zeros(s["seqs"], dtype=torch.float64, device=DEV).index_add_(0, seg, tok)
    return logp.float(), torch.where(on, lse, torch.zeros_like(lse)).float(), logp, lab, on, seg


def _pref_plain(s):
    out, lse, logp, lab, on, seg = _logprob_plain(s)
    P, V = s["seqs"] // 2, s["vocab"]
    ratio = logp - s["ref"].double()
    h = BETA * (ratio[:P] - ratio[P:])
    soft = lambda v: torch.log1p(torch.exp(-v.abs())) + (-v).clamp(min=0)  # noqa: E731
    loss = (1 - SMOOTH) * soft(h) + SMOOTH * soft(-h)
    dh = -(1 - SMOOTH) / (1 + torch.exp(h)) + SMOOTH / (1 + torch.exp(-h))
    d = torch.cat([BETA * dh, -BETA * dh]).float() / P
    coef = torch.where(on, d[seg], torch.zeros_like(d[seg]))[:, None]
    g = -coef * torch.exp(s["logits"][:, :V].float() - lse[:, None])
    g.scatter_add_(1, lab[:, None], coef)
    g = torch.where(on[:, None], g, torch.zeros_like(g))
    dl = torch.nn.functional.pad(g, (0, s["pad"])).to(DTYPES[s["d"]])
    return loss.float(), out, dl


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    kind = s["kind"]
    if not own:
        if kind == "act8":
            return _act8_plain(s)
        if kind == "bwd":
            return _bwd_plain(s)
        if kind == "logprob":
            return _logprob_plain(s)[:2]
        return _pref_plain(s)
    from bit_nf4_quantized_14_amd import capi
    code = {"bf16": capi.QN_BF16, "f32": capi.QN_F32, "none": capi.QN_BF16}
    if kind == "act8":
        t = capi.qn_act8_encode(s["xt"])
        return capi.qn_act8_decode(t, dtype=code[s["y"]]), t.scale
    if kind == "bwd":
        w = capi.NF4Tensor(s["packed"], s["qabs"], s["gscale"], s["n"], s["k"])
        x8 = capi.Act8Tensor(s["codes"], s["scale"], s["m"], s["k"])
        dx, dA, dB = capi.qlora_linear_bwd_act8(
            s["dy"], x8, w, s["A"], s["B"], s["r"], 32.0, s["T"],
            dx_dtype=code[s["dx"]], need_dx=s["dx"] != "none")
        return (dA, dB) if dx is None else (dx, dA, dB)
    logits = s["logits"][:, :s["vocab"]]
    if kind == "logprob":
        return capi.qn_seq_logprob(logits, s["labels"], s["offsets"])
    f = capi.qn_pref_loss_fwd(logits, s["labels"], s["offsets"], s["ref"], BETA,
                              label_smoothing=SMOOTH)
    dl = capi.qn_pref_loss_bwd(logits, s["labels"], s["offsets"], f, dlogits=s["dlogits"])
    return f.loss, f.logp, dl


def work(case):
    es = {"bf16": 2, "f32": 4, "none": 0}
    if case["kind"] == "act8":
        n = case["rows"] * case["cols"]
        ck = n + 4 * case["rows"] * -(-case["cols"] // 64)
        # x in, the checkpoint out and in again, the restored x out
        return dict(bytes=n * (es[case["x"]] + es[case["y"]]) + 2 * ck, flops=8 * n)
    if case["kind"] == "bwd":
        m, n, k, r = case["m"], case["n"], case["k"], case["r"]
        by = 2 * m * n + m * k + m * k // 16 + 2 * r * (n + k) + 4 * m * r + 4 * r * (n + k)
        fl = 4 * m * n * r + 2 * m * k * r
        if case["dx"] != "none":
            by += n * k // 2 + n * k // 64 + es[case["dx"]] * m * k
            fl += 2 * m * n * k + 2 * m * k * r
        return dict(bytes=by, flops=fl)
    # a counted row is read whole; about a third of the rows is prompt
    rows = case["seqs"] * case["length"]
    n = rows * case["vocab"]
    by, fl = n * es[case["x"]] * 2 // 3, 4 * n * 2 // 3
    if case["kind"] == "pref":
        by += rows * (case["vocab"] + case["pad"]) * es[case["d"]]
        fl += 4 * n * 2 // 3
    return dict(bytes=by + 20 * rows, flops=fl)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["kind"] == "act8":
        x = s["xt"].to(f64)
        y, scales = torch.empty_like(x), []
        for c0 in range(0, case["cols"], 64):
            b = x[:, c0:c0 + 64]
            top = b.abs().max(1, keepdim=True).values
            live = top >= 2.0 ** -100
            safe = torch.where(live, top, torch.ones_like(top))
            y[:, c0:c0 + 64] = torch.where(live, torch.round(127 * b / safe) * (safe / 127), 0)
            scales.append(torch.where(live, top / 127, 0))
        return y, torch.cat(scales, 1)
    if case["kind"] == "bwd":
        sc = 32.0 / case["r"]
        x = (s["codes"].to(f64) * s["scale"].to(f64).repeat_interleave(64, 1)).float()
        x = x.bfloat16().to(f64)
        dy, A, B, T = (s[v].to(f64) for v in ("dy", "A", "B", "T"))
        G = torch.mm(dy, B)
        dA, dB = torch.mm(G.t().contiguous(), x) * sc, torch.mm(dy.t().contiguous(), T) * sc
        if case["dx"] == "none":
            return dA, dB
        pk = s["packed"].to(torch.int64)
        e = torch.arange(case["n"] * case["k"], device=DEV)
        code = (pk[e // 2] >> (4 * (e % 2))) & 15
        const = s["qabs"].float() * s["gscale"][torch.arange(s["qabs"].numel(), device=DEV) // 256]
        w = (_levels().to(DEV)[code] * const[e // 64]).bfloat16().to(f64).view(case["n"], case["k"])
        return torch.mm(dy, w) + sc * torch.mm(G, A), dA, dB
    V, S, off = case["vocab"], case["seqs"], s["offsets"].tolist()
    logp, lses, probs = torch.zeros(S, dtype=f64, device=DEV), [], []
    for i in range(S):
        x = s["logits"][off[i]:off[i + 1], :V].to(f64)
        y = s["labels"][off[i]:off[i + 1]]
        lse = torch.logsumexp(x, 1)
        on = y >= 0
        at = x[on].gather(1, y[on][:, None])[:, 0]
        logp[i] = (at - lse[on]).sum()
        lses.append(torch.where(on, lse, 0))
        if case["kind"] == "pref":
            p = -torch.softmax(x, 1)
            p[on, y[on]] += 1
            p[~on] = 0
            probs.append(p)
    if case["kind"] == "logprob":
        return logp, torch.cat(lses)
    P = S // 2
    ref = s["ref"].to(f64)
    h = BETA * ((logp[:P] - ref[:P]) - (logp[P:] - ref[P:]))
    ls = torch.nn.functional.logsigmoid
    loss = -(1 - SMOOTH) * ls(h) - SMOOTH * ls(-h)
    dh = (-(1 - SMOOTH) * torch.sigmoid(-h) + SMOOTH * torch.sigmoid(h)) * BETA / P
    dl = torch.zeros(off[-1], V + case["pad"], dtype=f64, device=DEV)
    for i in range(S):
        dl[off[i]:off[i + 1], :V] = probs[i] * (dh[i] if i < P else -dh[i - P])
    return loss, logp, dl
