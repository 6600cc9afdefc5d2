"""The attention half of a transformer block around the quantised projections, measured.

Three operators and their directions, each in a plain form (elementary torch
operations in 32 bits) and as the library's calls:

- "norm":      RMS norm of every query and key head with the rotary position
               rotation (one or several position axes) in the same pass;
- "norm_bwd":  its gradients (both inputs and both norm weights);
- "attn":      softmax attention over packed sequences, causal or not, with
               grouped heads: the output and the row log-sum-exps;
- "attn_bwd":  its gradients;
- "decode":    attention of one new token per sequence over a key/value cache.

The widths are those of the linear layers of this repository: 24 heads of 128
(hidden 3072, 4608 image tokens) and 40 heads of 128 (hidden 5120, the small
batches of decoding), with 8 key/value heads where heads are grouped.
"""
import math
import random

import torch

own = False

EPS = 1e-6


# ---------------------------------------------------------------- the cases

def _ints(text):
    return [int(v) for v in text.split(",")]


def _decode_lengths(case):
    """Filled cache slots of every sequence: between lo and hi, spread evenly over their logarithm."""
    rng = random.Random(case["spread"])
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    n = [int(round(math.exp(rng.uniform(lo, hi)))) for _ in range(case["batch"])]
    n[0] = case["hi"]
    return n


def listed():
    return [
        # one new token of a decoding model, grouped heads, plain sequence positions: all latency
        {"name": "norm_token", "op": "norm", "tokens": 1, "hq": 40, "hk": 8, "d": 128, "rot": 128, "sections": "64",
         "interleaved": False, "fused": True},
        # an image transformer's block at 4608 tokens, time / height / width positions
        {"name": "norm_image", "op": "norm", "tokens": 4608, "hq": 24, "hk": 24, "d": 128, "rot": 128,
         "sections": "8,28,28", "interleaved": True, "fused": False},
        # the same block's gradients when an adapter is trained
        {"name": "norm_image_bwd", "op": "norm_bwd", "tokens": 4608, "hq": 24, "hk": 24, "d": 128, "rot": 128,
         "sections": "8,28,28", "interleaved": True, "fused": False},
        # fine-tuning on a text: one position axis, positions in the thousands; an odd number of tokens, narrow heads rotated
        # in part, read out of one fused q/k/v row
        {"name": "norm_odd_bwd", "op": "norm_bwd", "tokens": 1217, "hq": 10, "hk": 2, "d": 72, "rot": 64,
         "sections": "32", "interleaved": False, "fused": True},
        # a few short prompts (text encoder), odd lengths, narrow heads: latency
        {"name": "attn_short", "op": "attn", "lens_q": "1,77,130", "lens_k": "1,77,130", "hq": 12, "hk": 12, "d": 64,
         "causal": True},
        # an image transformer's block: every token sees every token
        {"name": "attn_image", "op": "attn", "lens_q": "4608", "lens_k": "4608", "hq": 24, "hk": 24, "d": 128,
         "causal": False},
        # a batch of prompts of a language model, packed, grouped heads, one of them going on from a cached prefix
        {"name": "attn_packed", "op": "attn", "lens_q": "4001,37,1999,512,1,1023,129,300",
         "lens_k": "4001,37,1999,512,1,1023,129,1500", "hq": 40, "hk": 8, "d": 128, "causal": True},
        # a short video: four times the image's tokens, the largest case
        {"name": "attn_video", "op": "attn", "lens_q": "18432", "lens_k": "18432", "hq": 24, "hk": 24, "d": 128,
         "causal": False},
        # the image block's gradients
        {"name": "attn_image_bwd", "op": "attn_bwd", "lens_q": "4608", "lens_k": "4608", "hq": 24, "hk": 24, "d": 128,
         "causal": False},
        # fine-tuning on packed texts of odd lengths, grouped heads
        {"name": "attn_packed_bwd", "op": "attn_bwd", "lens_q": "1501,333,64,2047,15", "lens_k": "1501,333,64,2047,15",
         "hq": 40, "hk": 8, "d": 128, "causal": True},
        # one chat: a single sequence's next token, latency and work split along the cache
        {"name": "decode_chat", "op": "decode", "batch": 1, "slots": 8192, "lo": 5003, "hi": 5003, "spread": 0, "hq": 40,
         "hk": 8, "d": 128},
        # a serving batch with lengths of every size in one cache
        {"name": "decode_batch", "op": "decode", "batch": 64, "slots": 16384, "lo": 300, "hi": 16001, "spread": 3,
         "hq": 40, "hk": 8, "d": 128},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    hk = rng.choice([1, 2, 3, 4, 8])
    return hk * rng.choice([1, 1, 2, 3, 4, 5]), hk


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "attn", "attn", "attn_bwd", "decode"])
    if op in ("norm", "norm_bwd"):
        hq, hk = _heads(rng)
        d = rng.choice([64, 128, 128, 8 * rng.randint(4, 16)])
        rot = d if rng.random() < 0.6 else 4 * rng.randint(4, d // 4)
        half, axes = rot // 2, rng.choice([1, 2, 3])
        first = [half // (axes + 1)] * (axes - 1)
        sections = ",".join(str(n) for n in first + [half - sum(first)])
        return {"op": op, "tokens": _log_int(rng, 1, 16384), "hq": hq, "hk": hk, "d": d, "rot": rot,
                "sections": sections, "interleaved": rng.random() < 0.5, "fused": rng.random() < 0.5}
    if op in ("attn", "attn_bwd"):
        hq, hk = _heads(rng)
        d = rng.choice([64, 128, 128, 8 * rng.randint(4, 16)])
        causal = rng.random() < 0.5
        n = rng.choice([1, 1, 2, 3, 5, 8])
        most = _log_int(rng, 16, 12000 if op == "attn" else 6000)
        while n * hq * most * most > (4 << 30 if op == "attn" else 1 << 30):
            most = most * 3 // 4
        lens_q = [most] + [_log_int(rng, 1, most) for _ in range(n - 1)]
        # some sequences have more keys than queries (a prefix before them), a few have fewer
        lens_k = [max(1, m + rng.choice([0, 0, 0, 7, 64, 250, -3])) for m in lens_q]
        return {"op": op, "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)), "hq": hq,
                "hk": hk, "d": d, "causal": causal}
    hq, hk = _heads(rng)
    hi = _log_int(rng, 16, 16384)
    return {"op": op, "batch": _log_int(rng, 1, 64), "slots": hi + rng.choice([0, 1, 100]), "lo": max(1, hi // 20),
            "hi": hi, "spread": rng.randint(0, 1 << 20), "hq": hq, "hk": hk, "d": rng.choice([64, 128, 128, 96])}


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _unit_heads(g, tokens, heads, d, gain):
    """What a head norm leaves: heads of unit mean square, times channel weights around `gain`."""
    x = _randn(g, tokens, heads, d)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
    return (x * (gain + 0.2 * _randn(g, d))).to(torch.bfloat16)


def _starts(lens):
    return torch.tensor([0] + lens).cumsum(0).to(torch.int32).to("cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * (seed % 100000) + 17)
    op, hq, hk, d = case["op"], case["hq"], case["hk"], case["d"]
    s = {"case": case}
    if op in ("norm", "norm_bwd"):
        t, rot = case["tokens"], case["rot"]
        sections = tuple(_ints(case["sections"]))
        channel = torch.ones(d, device="cuda")
        channel[torch.randint(0, d, (2,), generator=g, device="cuda")] = 6.0  # the outlier channels of a projection
        if case["fused"]:
            row = (_randn(g, t, hq + 2 * hk, d) * channel).to(torch.bfloat16)
            s["q"], s["k"] = row[:, :hq], row[:, hq:hq + hk]
        else:
            s["q"] = (_randn(g, t, hq, d) * channel).to(torch.bfloat16)
            s["k"] = (_randn(g, t, hk, d) * channel).to(torch.bfloat16)
        s["q_weight"] = 1.0 + 0.2 * _randn(g, d)
        s["k_weight"] = 1.0 + 0.2 * _randn(g, d)
        # positions: of a sequence (some offset into it), or of the points of a grid in row order
        n = torch.arange(t, device="cuda")
        first = int(torch.randint(0, 4096, (1,), generator=g, device="cuda"))
        width = max(1, int(math.sqrt(t / max(1, len(sections) - 1))))
        axes = {1: [n + first], 2: [n // width, n % width],
                3: [n // (width * width), n // width % width, n % width]}[len(sections)]
        s["positions"] = torch.stack(axes, 1).to(torch.int32).contiguous()
        freqs = [torch.pow(10000.0, -torch.arange(m, dtype=torch.float64) / m) for m in sections]
        s["freqs"] = torch.cat(freqs).to(torch.float32).to("cuda")
        s["axis"] = torch.cat([torch.full((m,), i) for i, m in enumerate(sections)]).to("cuda")  # of every pair
        s["sections"], s["rot"] = sections, rot
        if op == "norm_bwd":
            s["dq"], s["dk"] = _randn(g, t, hq, d).to(torch.bfloat16), _randn(g, t, hk, d).to(torch.bfloat16)
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    if op in ("attn", "attn_bwd"):
        lens_q, lens_k = _ints(case["lens_q"]), _ints(case["lens_k"])
        s["q"] = _unit_heads(g, sum(lens_q), hq, d, 1.6)
        s["k"] = _unit_heads(g, sum(lens_k), hk, d, 1.0)
        s["v"] = _randn(g, sum(lens_k), hk, d).to(torch.bfloat16)
        s["cu_q"], s["cu_k"] = _starts(lens_q), _starts(lens_k)
        s["most_q"], s["most_k"] = max(lens_q), max(lens_k)
        if op == "attn_bwd":
            s["dout"] = _randn(g, sum(lens_q), hq, d).to(torch.bfloat16)
            s["out"], s["lse"] = _attn_plain(s)  # what the forward pass left
        return s
    b = case["batch"]
    s["q"] = _unit_heads(g, b, hq, d, 1.6)
    # slots past a sequence's length hold what was there before
    s["k"] = _unit_heads(g, b * case["slots"], hk, d, 1.0).view(b, case["slots"], hk, d)
    s["v"] = _randn(g, b, case["slots"], hk, d).to(torch.bfloat16)
    s["lengths"] = torch.tensor(_decode_lengths(case), dtype=torch.int32, device="cuda")
    return s


# ---------------------------------------------------------------- the plain forms

def _angles(s):
    # formed in 64 bits: in 32, a position of some 10^4 times a frequency is off by up to 1e-3 rad
    a = s["positions"].double()[:, s["axis"]] * s["freqs"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _split(x, s):
    """The pairs of the rotated part of a head, and the rest of it."""
    rot = s["rot"]
    if s["case"]["interleaved"]:
        return x[..., 0:rot:2], x[..., 1:rot:2], x[..., rot:]
    return x[..., :rot // 2], x[..., rot // 2:rot], x[..., rot:]


def _join(a, b, rest, s):
    turned = torch.stack((a, b), -1).flatten(-2) if s["case"]["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((turned, rest), -1)


def _norm_plain(x, weight, cos, sin, s):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    a, b, rest = _split(y, s)
    return _join(a * cos - b * sin, b * cos + a * sin, rest, s).to(torch.bfloat16)


def _norm_bwd_plain(dy, x, weight, cos, sin, s):
    x, dy = x.float(), dy.float()
    a, b, rest = _split(dy, s)
    dz = _join(a * cos + b * sin, b * cos - a * sin, rest, s)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xn = x * r
    dweight = (dz * xn).sum((0, 1))
    dxn = dz * weight
    dx = r * (dxn - xn * (dxn * xn).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), dweight


def _pad(x, cu, most):
    """Packed rows [tokens, heads, d] -> [sequences, heads, most, d] in 32 bits, and which rows are real."""
    at = torch.arange(most, device=x.device)
    rows = (cu[:-1, None] + at).clamp(max=x.shape[0] - 1)
    return x[rows].float().transpose(1, 2), at < (cu[1:] - cu[:-1])[:, None]


def _pack(x, cu, tokens):
    """[sequences, heads, most, ...] -> [tokens, heads, ...]"""
    at = torch.arange(tokens, device=x.device)
    seq = torch.searchsorted(cu[1:].contiguous(), at, right=True)
    return x[seq, :, at - cu[seq]]


def _scores(q, k, real_k, s):
    """Scores of padded operands, grouped heads folded into rows [sequences, hk, group * most_q, most_k]; -inf where masked."""
    n, hq, lq, d = q.shape
    hk, lk = k.shape[1], k.shape[2]
    z = torch.matmul(q.reshape(n, hk, hq // hk * lq, d), k.transpose(2, 3).contiguous()).mul_(s["scale"])
    seen = real_k[:, None, :]
    if s["case"]["causal"]:
        len_q, len_k = (c[1:] - c[:-1] for c in (s["cu_q"], s["cu_k"]))
        last = torch.arange(lq, device=q.device) + (len_k - len_q)[:, None]
        seen = seen & (torch.arange(lk, device=q.device) <= last[:, :, None])
    else:
        seen = seen.expand(n, lq, lk)
    z.view(n, hk, hq // hk, lq, lk).masked_fill_(~seen[:, None, None], -math.inf)
    return z


def _softmax_(z):
    """In place; rows that see nothing give zeros and a log-sum-exp of -inf."""
    top = z.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    z.sub_(top).exp_()
    total = z.sum(-1, keepdim=True)
    z.div_(torch.where(total == 0, 1.0, total))
    return z, (top + total.log()).squeeze(-1)


def _attn_plain(s):
    q, k, v = s["q"], s["k"], s["v"]
    tokens, hq, d = q.shape
    n = s["cu_q"].numel() - 1
    qp, _ = _pad(q, s["cu_q"], s["most_q"])
    kp, real_k = _pad(k, s["cu_k"], s["most_k"])
    vp, _ = _pad(v, s["cu_k"], s["most_k"])
    p, lse = _softmax_(_scores(qp, kp, real_k, s))
    out = torch.matmul(p, vp.contiguous()).reshape(n, hq, -1, d)
    out = _pack(out, s["cu_q"], tokens).to(torch.bfloat16)
    return out, _pack(lse.reshape(n, hq, -1), s["cu_q"], tokens).t().contiguous()


def _attn_bwd_plain(s):
    q, k, v = s["q"], s["k"], s["v"]
    tokens, hq, d = q.shape
    hk, n, lq = k.shape[1], s["cu_q"].numel() - 1, s["most_q"]
    qp, real_q = _pad(q, s["cu_q"], lq)
    dop, _ = _pad(s["dout"], s["cu_q"], lq)
    op, _ = _pad(s["out"], s["cu_q"], lq)
    lp, _ = _pad(s["lse"].t()[:, :, None], s["cu_q"], lq)
    kp, real_k = _pad(k, s["cu_k"], s["most_k"])
    vp, _ = _pad(v, s["cu_k"], s["most_k"])
    rows = (n, hk, hq // hk * lq)
    dop = (dop * real_q[:, None, :, None]).reshape(*rows, d)
    qp, op, lp = qp.reshape(*rows, d), op.reshape(*rows, d), lp.reshape(*rows, 1)
    p = _scores(qp.view(n, hq, lq, d), kp, real_k, s)
    p.sub_(torch.where(lp == -math.inf, 0.0, lp)).exp_()
    dv = torch.matmul(p.transpose(2, 3).contiguous(), dop)
    ds = torch.matmul(dop, vp.transpose(2, 3).contiguous())
    ds.sub_((dop * op).sum(-1, keepdim=True)).mul_(p).mul_(s["scale"])
    del p
    dq = torch.matmul(ds, kp.contiguous()).reshape(n, hq, lq, d)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), qp.contiguous())
    return (_pack(dq, s["cu_q"], tokens).to(torch.bfloat16), _pack(dk, s["cu_k"], k.shape[0]).to(torch.bfloat16),
            _pack(dv, s["cu_k"], k.shape[0]).to(torch.bfloat16))


def _decode_plain(s):
    b, hq, d = s["q"].shape
    slots, hk = s["k"].shape[1:3]
    z = torch.matmul(s["q"].float().view(b, hk, hq // hk, d), s["k"].float().permute(0, 2, 3, 1).contiguous())
    unseen = torch.arange(slots, device=z.device) >= s["lengths"][:, None]
    z.mul_(s["scale"]).masked_fill_(unseen[:, None, None], -math.inf)
    p, lse = _softmax_(z)
    out = torch.matmul(p, s["v"].float().transpose(1, 2).contiguous())
    return out.reshape(b, hq, d).to(torch.bfloat16), lse.reshape(b, hq).t().contiguous()


# ---------------------------------------------------------------- one pass

def _run_own(op, s):
    import int4_w4a4_quantized_amd as ck
    if op == "norm":
        return ck.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"], s["freqs"], s["sections"],
                               interleaved=s["case"]["interleaved"], eps=EPS)
    if op == "norm_bwd":
        return ck.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"],
                                        s["freqs"], s["sections"], interleaved=s["case"]["interleaved"], eps=EPS)
    if op == "attn":
        return ck.attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["case"]["causal"], scale=s["scale"])
    if op == "attn_bwd":
        return ck.attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["cu_q"], s["cu_k"],
                                     causal=s["case"]["causal"], scale=s["scale"])
    return ck.attention_decode(s["q"], s["k"], s["v"], s["lengths"], scale=s["scale"])


def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(op, state)
    if op == "norm":
        cos, sin = _angles(state)
        return (_norm_plain(state["q"], state["q_weight"], cos, sin, state),
                _norm_plain(state["k"], state["k_weight"], cos, sin, state))
    if op == "norm_bwd":
        cos, sin = _angles(state)
        dq, dq_weight = _norm_bwd_plain(state["dq"], state["q"], state["q_weight"], cos, sin, state)
        dk, dk_weight = _norm_bwd_plain(state["dk"], state["k"], state["k_weight"], cos, sin, state)
        return dq, dk, dq_weight, dk_weight
    if op == "attn":
        return _attn_plain(state)
    if op == "attn_bwd":
        return _attn_bwd_plain(state)
    return _decode_plain(state)


# ---------------------------------------------------------------- the same in 64 bits

def _exact_norm(x, weight, s):
    """Norm and rotation from their definition: each pair of a head, as a complex number, times exp(i position freq)."""
    rot, half = s["rot"], s["rot"] // 2
    y = weight * x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    angle = torch.gather(s["positions"].double(), 1, s["axis"].expand(x.shape[0], half)) * s["freqs"].double()
    spin = torch.polar(torch.ones_like(angle), angle)[:, None, :]
    head = y[..., :rot]
    pairs = head.unflatten(-1, (half, 2)) if s["case"]["interleaved"] else head.unflatten(-1, (2, half)).mT
    turned = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * spin)
    turned = turned.flatten(-2) if s["case"]["interleaved"] else turned.mT.flatten(-2)
    return torch.cat((turned, y[..., rot:]), -1)


def _exact_rows(q, k, v, causal, scale):
    """One head of one sequence, in 64 bits: output and log-sum-exps; rows that see nothing give zeros and -inf."""
    z = torch.mm(q, k.t().contiguous()) * scale
    if causal:
        z = z + torch.full_like(z, -math.inf).triu(1 + k.shape[0] - q.shape[0])
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[:, None])
    return torch.mm(p, v), lse


def exact(case, seed):
    if work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        return tuple(_exact_norm(s[n].double(), s[n + "_weight"].double(), s) for n in ("q", "k"))
    if op == "norm_bwd":
        with torch.enable_grad():
            got = []
            for n in ("q", "k"):
                x, w = s[n].double().requires_grad_(), s[n + "_weight"].double().requires_grad_()
                got.append(torch.autograd.grad(_exact_norm(x, w, s), (x, w), s["d" + n].double()))
        return got[0][0], got[1][0], got[0][1], got[1][1]
    hq, hk = case["hq"], case["hk"]
    if op == "decode":
        out, lse = torch.zeros(s["q"].shape, dtype=torch.float64), torch.zeros(hq, case["batch"], dtype=torch.float64)
        for i, n in enumerate(_decode_lengths(case)):
            q, k, v = s["q"][i].double(), s["k"][i, :n].double(), s["v"][i, :n].double()
            k, v = (x.repeat_interleave(hq // hk, 1) for x in (k, v))
            z = (q * k).sum(-1) * s["scale"]
            out[i] = (torch.softmax(z, 0)[..., None] * v).sum(0)
            lse[:, i] = torch.logsumexp(z, 0)
        return out, lse
    lens_q, lens_k = _ints(case["lens_q"]), _ints(case["lens_k"])
    starts = [(sum(lens_q[:i]), sum(lens_k[:i])) for i in range(len(lens_q))]
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    lse = torch.zeros(hq, s["q"].shape[0], dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros_like(s["k"], dtype=torch.float64) for _ in range(2))
    for (a, c), nq, nk in zip(starts, lens_q, lens_k):
        for h in range(hq):
            u = h // (hq // hk)
            q, k, v = s["q"][a:a + nq, h].double(), s["k"][c:c + nk, u].double(), s["v"][c:c + nk, u].double()
            if op == "attn":
                out[a:a + nq, h], lse[h, a:a + nq] = _exact_rows(q, k, v, case["causal"], s["scale"])
                continue
            with torch.enable_grad():
                q, k, v = (x.requires_grad_() for x in (q, k, v))
                o, _ = _exact_rows_grad(q, k, v, case["causal"], s["scale"])
                gq, gk, gv = torch.autograd.grad(o, (q, k, v), s["dout"][a:a + nq, h].double())
            out[a:a + nq, h] = gq
            dk[c:c + nk, u] += gk
            dv[c:c + nk, u] += gv
    return (out, lse) if op == "attn" else (out, dk, dv)


def _exact_rows_grad(q, k, v, causal, scale):
    """_exact_rows for differentiation: rows that see nothing stay out of the graph."""
    first = max(0, q.shape[0] - k.shape[0]) if causal else 0
    o, lse = _exact_rows(q[first:], k, v, causal, scale)
    return torch.cat((torch.zeros_like(q[:first]), o)), lse


# ---------------------------------------------------------------- the work

def _pairs(case):
    """Query/key pairs of one head that the mask leaves."""
    total = 0
    for nq, nk in zip(_ints(case["lens_q"]), _ints(case["lens_k"])):
        # row i of a causal sequence sees nk - nq + i + 1 keys, none where that is negative
        total += sum(range(max(0, nk - nq + 1), nk + 1)) if case["causal"] else nq * nk
    return total


def work(case):
    op, hq, hk, d = case["op"], case["hq"], case["hk"], case["d"]
    if op in ("norm", "norm_bwd"):
        values = case["tokens"] * (hq + hk) * d
        small = case["tokens"] * 4 * len(_ints(case["sections"])) + case["rot"] * 2 + 8 * d
        if op == "norm":
            return {"bytes": 4 * values + small, "flops": 7 * values}
        return {"bytes": 6 * values + small + 8 * d, "flops": 15 * values}
    if op == "decode":
        seen, b = sum(_decode_lengths(case)), case["batch"]
        return {"bytes": 4 * seen * hk * d + b * hq * (4 * d + 4) + 4 * b, "flops": 4 * seen * hq * d}
    nq, nk = sum(_ints(case["lens_q"])), sum(_ints(case["lens_k"]))
    if op == "attn":
        return {"bytes": 4 * nq * hq * d + 4 * nk * hk * d + 4 * nq * hq, "flops": 4 * d * hq * _pairs(case)}
    return {"bytes": 8 * nq * hq * d + 8 * nk * hk * d + 4 * nq * hq, "flops": 10 * d * hq * _pairs(case)}
