"""Head norm with rotary positions, attention, their gradients and decoding
over a cache, on the GPU, against the 64-bit oracle. The bounds are the
oracle's: they follow from the formulas' roundings."""
import math

import pytest
import torch

import attention_oracle as ao

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ck():
    import int4_w4a4_quantized_amd as ck
    assert torch.cuda.get_device_properties(0).gcnArchName.startswith("gfx950")
    return ck


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rand(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(BF16)


def _near(got, want, tol, what):
    got = got.double().cpu()
    assert got.shape == want.shape
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine], want[~fine]), what
    off = (got - want).abs()
    bad = fine & ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} values are off, at most {float(off[bad].max())}"


def _bits(*ts):
    torch.cuda.synchronize()
    return [t.contiguous().view(torch.int16 if t.dtype == BF16 else torch.int32).cpu() for t in ts]


# ------------------------------------------------------------ norm and rotation

# tokens, hq, hk, d, sections, interleaved, fp32 positions
NORMS = [
    (1, 1, 1, 8, (4,), True, False),          # one token, one head, the narrowest head
    (1, 40, 8, 128, (64,), False, False),
    (3, 5, 2, 128, (8, 28, 28), True, False),
    (37, 24, 24, 128, (8, 28, 28), False, True),
    (65, 3, 1, 72, (16, 16), False, False),   # rotated in part
    (9, 2, 2, 72, (10, 8), False, True),      # half-split pairs that end inside a 16-byte chunk
    (9, 2, 2, 72, (9, 8), True, False),
    (257, 4, 1, 64, (32,), True, False),
    (130, 7, 3, 104, (13, 13, 26), False, False),
    (50, 2, 1, 256, (100, 20, 5, 3), True, True),
    (33, 2, 1, 136, (68,), False, False),
    (1300, 6, 2, 32, (2, 0, 9), True, False),  # an axis without pairs
    (2048, 1, 1, 40, (20,), False, False),
]


def _norm_inputs(t, hq, hk, d, sections, pos_f32, seed):
    g = _gen(seed)
    q, k = _rand(g, t, hq, d), _rand(g, t, hk, d)
    q[t // 2, 0] = 0  # a head of zeros
    k[:, :, d // 3] *= 20
    pairs = sum(sections)
    pos = torch.randint(-50, 9000, (t, len(sections)), generator=g).int()
    if pos_f32:
        pos = pos.float() + 0.25
    freqs = (10000.0 ** -(torch.arange(pairs) / pairs)).float()
    return q, k, 1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g), pos, freqs


def _norm_tol(y):
    # one rounding to bf16, and fp32 terms of the head's size
    return ao.EPS * y.abs() + 2.0 ** -20 * y.abs().amax(-1, keepdim=True)


@pytest.mark.parametrize("t,hq,hk,d,sections,interleaved,pos_f32", NORMS)
def test_norm_rope(ck, t, hq, hk, d, sections, interleaved, pos_f32):
    q, k, wq, wk, pos, freqs = _norm_inputs(t, hq, hk, d, sections, pos_f32, 100 + t + d)
    got = ck.qk_norm_rope(q.cuda(), k.cuda(), wq.cuda(), None, pos.cuda(), freqs.cuda(), sections, interleaved)
    for x, w, y, name in ((q, wq, got[0], "q"), (k, None, got[1], "k")):
        want = ao.norm_rope(x.double(), None if w is None else w.double(), pos.double(), freqs.double(), sections,
                            interleaved)
        _near(y, want, _norm_tol(want), name)


@pytest.mark.parametrize("t,hq,hk,d,sections,interleaved,pos_f32", NORMS)
def test_norm_rope_backward(ck, t, hq, hk, d, sections, interleaved, pos_f32):
    q, k, wq, wk, pos, freqs = _norm_inputs(t, hq, hk, d, sections, pos_f32, 300 + t + d)
    q[t // 2, 0, 0] = 0.5  # the gradient at a head of zeros is 1 / sqrt(eps) large: not this test's
    g = _gen(t)
    dyq, dyk = _rand(g, t, hq, d), _rand(g, t, hk, d)
    dq, dk, dwq, dwk = ck.qk_norm_rope_backward(dyq.cuda(), dyk.cuda(), q.cuda(), k.cuda(), wq.cuda(), wk.cuda(),
                                                pos.cuda(), freqs.cuda(), sections, interleaved)
    for x, w, dy, dx, dw, name in ((q, wq, dyq, dq, dwq, "q"), (k, wk, dyk, dk, dwk, "k")):
        want, want_w, size_w = ao.norm_rope_backward(dy.double(), x.double(), w.double(), pos.double(), freqs.double(),
                                                     sections, interleaved)
        r = 1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)
        size = (dy.double() * r).abs().amax(-1, keepdim=True) * w.double().abs().max()
        _near(dx, want, ao.EPS * want.abs() + 2.0 ** -18 * size, "d" + name)
        _near(dw, want_w, 2.0 ** -18 * size_w, f"d{name}_weight")


# more steps than the launches have wavefronts (8192, and 4096 backward), in uneven shares that cross tokens
NORMS_LONG = [
    (1531, 24, 5, 128, (64,), False, False),       # 8 steps a token
    (1531, 24, 5, 128, (8, 28, 28), True, False),
    (1531, 24, 5, 128, (30, 31), False, True),     # half-split pairs that end inside a 16-byte chunk
    (5003, 3, 2, 136, (68,), True, False),         # 2 heads a step: 3 steps a token, the last half full
    (2311, 29, 12, 72, (32,), False, False),       # rotated in part, 4 heads a step, the last step a quarter full
]


@pytest.mark.parametrize("t,hq,hk,d,sections,interleaved,pos_f32", NORMS_LONG)
def test_norm_rope_many_steps_a_wavefront(ck, t, hq, hk, d, sections, interleaved, pos_f32):
    test_norm_rope(ck, t, hq, hk, d, sections, interleaved, pos_f32)
    test_norm_rope_backward(ck, t, hq, hk, d, sections, interleaved, pos_f32)


@pytest.mark.parametrize("t,hq,hk,d,sections,interleaved,pos_f32", NORMS_LONG)
def test_norm_rope_many_steps_in_place(ck, t, hq, hk, d, sections, interleaved, pos_f32):
    """Outputs that are the inputs, with the next heads loaded ahead of a store: the same bits; and twice the same."""
    q, k, wq, wk, pos, freqs = (x.cuda() for x in _norm_inputs(t, hq, hk, d, sections, pos_f32, 500 + t + d))
    g = _gen(t)
    dyq, dyk = _rand(g, t, hq, d).cuda(), _rand(g, t, hk, d).cuda()
    rest = (wq, wk, pos, freqs, sections, interleaved)
    want, want_g = ck.qk_norm_rope(q, k, *rest), ck.qk_norm_rope_backward(dyq, dyk, q, k, *rest)
    over = [x.clone() for x in (dyq, dyk)]
    got_g = ck.qk_norm_rope_backward(*over, q, k, *rest, dq=over[0], dk=over[1])
    assert got_g[0] is over[0] and all(torch.equal(a, b) for a, b in zip(_bits(*got_g), _bits(*want_g)))
    over = [x.clone() for x in (q, k)]
    got_g = ck.qk_norm_rope_backward(dyq, dyk, *over, *rest, dq=over[0], dk=over[1])
    assert all(torch.equal(a, b) for a, b in zip(_bits(*got_g), _bits(*want_g)))
    got = ck.qk_norm_rope(q, k, *rest, q_out=q, k_out=k)
    assert got[0] is q and all(torch.equal(a, b) for a, b in zip(_bits(*got), _bits(*want)))


def test_norm_rope_against_differences(ck):
    """The kernel's gradients along random directions against differences of the 64-bit forward pass."""
    t, h, d, sections = 6, 2, 64, (8, 12, 12)
    q, k, wq, wk, pos, freqs = _norm_inputs(t, h, h, d, sections, False, 7)
    q[t // 2, 0] = 1
    dy = _rand(_gen(8), t, h, d)
    zeros = torch.zeros_like(dy)
    dq, _, dwq, _ = ck.qk_norm_rope_backward(dy.cuda(), zeros.cuda(), q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), pos.cuda(),
                                             freqs.cuda(), sections, True)

    def loss(x, w):
        return (ao.norm_rope(x, w, pos.double(), freqs.double(), sections, True) * dy.double()).sum().item()

    g = _gen(9)
    ux, uw = torch.randn(t, h, d, generator=g).double(), torch.randn(d, generator=g).double()
    x, w, e = q.double(), wq.double(), 1e-6
    dq, dwq = dq.double().cpu(), dwq.double().cpu()
    diff = (loss(x + e * ux, w) - loss(x - e * ux, w)) / (2 * e)
    assert abs((dq * ux).sum().item() - diff) <= 2 * ao.EPS * (dq * ux).abs().sum().item()
    diff = (loss(x, w + e * uw) - loss(x, w - e * uw)) / (2 * e)
    assert abs((dwq * uw).sum().item() - diff) <= 1e-4 * (dwq * uw).abs().sum().item()


@pytest.mark.parametrize("sections", [(0,), (0, 0, 0)])
@pytest.mark.parametrize("interleaved", [True, False])
def test_norm_without_rotation(ck, sections, interleaved):
    """No pair is turned: the norm and its gradients alone."""
    shape = 37, 5, 2, 72, sections, interleaved, False
    test_norm_rope(ck, *shape)
    test_norm_rope_backward(ck, *shape)


def test_norm_rope_views_and_in_place(ck):
    """A fused projection's rows as inputs, a joint buffer and the inputs themselves as outputs: the same bits."""
    t, hq, hk, d = 70, 6, 2, 96
    g = _gen(11)
    row = _rand(g, t, hq + 2 * hk, d).cuda()
    wq, wk = torch.rand(d, generator=g).cuda(), torch.rand(d, generator=g).cuda()
    pos, freqs = torch.arange(t).int().cuda(), torch.rand(48, generator=g).cuda()
    q, k = row[:, :hq], row[:, hq:hq + hk]
    want = ck.qk_norm_rope(q.contiguous(), k.contiguous(), wq, wk, pos, freqs)
    joint = torch.full((t + 10, hq + hk, d), 7.0, dtype=BF16, device="cuda")
    ck.qk_norm_rope(q, k, wq, wk, pos, freqs, q_out=joint[5:5 + t, :hq], k_out=joint[5:5 + t, hq:])
    heads_first = torch.empty(hq, t, d, dtype=BF16, device="cuda").transpose(0, 1)
    ck.qk_norm_rope(q, k, wq, wk, pos, freqs, q_out=heads_first)
    rest = row[:, hq + hk:].clone()
    dy = _rand(g, t, hq, d).cuda(), _rand(g, t, hk, d).cuda()
    want_g = ck.qk_norm_rope_backward(*dy, q, k, wq, wk, pos, freqs)
    row2 = row.clone()
    got_g = ck.qk_norm_rope_backward(*dy, row2[:, :hq], row2[:, hq:hq + hk], wq, wk, pos, freqs, dq=row2[:, :hq],
                                     dk=row2[:, hq:hq + hk])
    ck.qk_norm_rope(q, k, wq, wk, pos, freqs, q_out=q, k_out=k)
    for got in ((joint[5:5 + t, :hq], joint[5:5 + t, hq:]), (heads_first, want[1]), (q, k)):
        assert all(torch.equal(a, b) for a, b in zip(_bits(*got), _bits(*want)))
    assert (joint[:5] == 7).all() and (joint[5 + t:] == 7).all() and torch.equal(row[:, hq + hk:], rest)
    assert all(torch.equal(a, b) for a, b in zip(_bits(*got_g), _bits(*want_g)))


# ------------------------------------------------------------ attention

# lengths of q, of k, hq, hk, d, causal
SHAPES = [
    ([1], [1], 1, 1, 64, False),
    ([1], [300], 4, 1, 128, True),               # one row, many keys
    ([130], [1], 2, 2, 128, False),              # many rows, one key
    ([64], [64], 2, 1, 64, True),
    ([63, 65], [63, 65], 3, 3, 64, True),
    ([129], [257], 2, 1, 128, True),             # a prefix before the rows
    ([257], [129], 2, 1, 128, True),             # more rows than keys: the first see nothing
    ([5, 0, 70, 0], [9, 40, 0, 0], 2, 2, 128, False),  # sequences without rows, without keys, without both
    ([5, 0, 70, 1], [9, 40, 0, 3], 2, 2, 64, True),
    ([300], [300], 5, 1, 128, True),
    ([256], [256], 4, 2, 128, False),
    ([40, 1, 513], [40, 77, 513], 8, 2, 128, True),
    ([200, 33], [150, 90], 3, 1, 72, False),     # heads narrower than the tile
    ([200, 33], [150, 90], 3, 1, 40, True),
    ([90], [90], 2, 2, 8, True),
    ([100], [130], 2, 2, 96, False),
    ([100], [130], 2, 2, 120, True),
    ([1] * 70, [1 + i % 9 for i in range(70)], 2, 1, 64, True),  # more sequences than lanes
    # few tiles of rows and many keys: tiles cut along the keys
    ([1], [2500], 2, 1, 128, True),
    ([300], [3000], 1, 1, 64, False),
    ([1100], [1100], 2, 1, 128, True),
    ([700], [1500], 3, 3, 72, True),
    ([900], [700], 1, 1, 128, True),             # rows that see nothing, in tiles of their own
    ([2000, 3, 600, 0, 1], [2000, 30, 900, 5, 0], 1, 1, 64, True),
    ([3] * 66 + [1500], [5] * 66 + [1500], 1, 1, 64, False),  # the long one behind more sequences than lanes
    ([1300], [40], 4, 1, 64, False),             # one tile of keys, many rows of several heads
    ([10] * 60, [10] * 59 + [1300], 5, 1, 64, True),  # room for cutting, but short tiles: more of them than pieces
]


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _attn_inputs(lens_q, lens_k, hq, hk, d, seed, std=1.0):
    g = _gen(seed)
    return (_rand(g, sum(lens_q), hq, d, std=std), _rand(g, sum(lens_k), hk, d, std=std), _rand(g, sum(lens_k), hk, d),
            _rand(g, sum(lens_q), hq, d))


def _dev_cu(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("std", [1.0, 3.0])  # 3: scores of up to some 100, near one-hot rows
@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d,causal", SHAPES)
def test_attention(ck, lens_q, lens_k, hq, hk, d, causal, std):
    q, k, v, _ = _attn_inputs(lens_q, lens_k, hq, hk, d, sum(lens_q) + d, std)
    cu_q, cu_k, scale = _cu(lens_q), _cu(lens_k), d ** -0.5
    out, lse = ck.attention(q.cuda(), k.cuda(), v.cuda(), _dev_cu(cu_q), _dev_cu(cu_k), causal=causal)
    want, want_lse, tol, lse_tol = ao.attention(q.double(), k.double(), v.double(), cu_q, cu_k, causal, scale)
    _near(out, want, tol, "out")
    _near(lse, want_lse, lse_tol, "lse")
    if len(lens_q) == 1:
        out1, lse1 = ck.attention(q.cuda(), k.cuda(), v.cuda(), causal=causal)
        assert all(torch.equal(a, b) for a, b in zip(_bits(out, lse), _bits(out1, lse1)))


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d,causal", SHAPES)
def test_attention_backward(ck, lens_q, lens_k, hq, hk, d, causal):
    q, k, v, do = _attn_inputs(lens_q, lens_k, hq, hk, d, sum(lens_q) + d + 1)
    cu_q, cu_k, scale = _cu(lens_q), _cu(lens_k), 1.3 * d ** -0.5
    x = [t.double() for t in (q, k, v)]
    out, lse, _, _ = ao.attention(*x, cu_q, cu_k, causal, scale)
    out, lse = out.to(BF16), lse.float()
    want, tols = ao.attention_backward(do.double(), *x, out.double(), cu_q, cu_k, causal, scale)
    args = [t.cuda() for t in (do, q, k, v, out, lse)] + [_dev_cu(cu_q), _dev_cu(cu_k)]
    got = ck.attention_backward(*args, causal=causal, scale=scale)
    for y, w, t, name in zip(got, want, tols, ("dq", "dk", "dv")):
        _near(y, w, t, name)
    again = ck.attention_backward(*args, causal=causal, scale=scale)
    assert all(torch.equal(a, b) for a, b in zip(_bits(*got), _bits(*again)))


# more than 256 whole tiles of keys and of queries, none cut: a launch each for their gradients; numbers of heads of which
# an XCD has several
WHOLE = [
    ([20] * 40, [20] * 40, 40, 8, 128, True),
    ([300, 1, 0, 77] * 12, [310, 1, 5, 40] * 12, 16, 8, 64, True),
    ([20] * 40, [33] * 40, 40, 8, 128, False),
    ([5, 260] * 12, [260, 5] * 12, 24, 8, 72, False),
    ([300, 20, 600] * 5, [300, 50, 600] * 5, 24, 24, 128, True),
    ([300, 20, 600] * 5, [300, 50, 600] * 5, 24, 24, 40, True),
]


@pytest.mark.parametrize("lens_q,lens_k,hq,hk,d,causal", WHOLE)
def test_attention_many_whole_tiles(ck, lens_q, lens_k, hq, hk, d, causal):
    sizes = len(lens_q), sum(lens_q), sum(lens_k), hq, hk, d
    assert ck.lib().ck4_attention_workspace_bytes(*sizes) == 0
    assert ck.lib().ck4_attention_backward_workspace_bytes(*sizes) == 8 * sum(lens_q) * hq  # the rows' statistics alone
    test_attention(ck, lens_q, lens_k, hq, hk, d, causal, 1.0)
    test_attention_backward(ck, lens_q, lens_k, hq, hk, d, causal)


def test_attention_against_differences(ck):
    """Forward and backward kernels together: gradients along random directions against differences in 64 bits."""
    lens_q, lens_k, hq, hk, d = [70, 9], [81, 5], 4, 2, 64
    q, k, v, do = _attn_inputs(lens_q, lens_k, hq, hk, d, 21)
    cu_q, cu_k = _cu(lens_q), _cu(lens_k)
    dev = [t.cuda() for t in (q, k, v)] + [_dev_cu(cu_q), _dev_cu(cu_k)]
    out, lse = ck.attention(*dev, causal=True)
    got = ck.attention_backward(do.cuda(), *dev[:3], out, lse, *dev[3:], causal=True)
    x = [t.double() for t in (q, k, v)]
    _, tols = ao.attention_backward(do.double(), *x, out.double().cpu(), cu_q, cu_k, True, d ** -0.5)

    def loss(x):
        return (ao.attention(*x, cu_q, cu_k, True, d ** -0.5)[0] * do.double()).sum().item()

    g = _gen(22)
    for i in range(3):
        u, e = torch.randn(x[i].shape, generator=g).double(), 1e-5
        diff = (loss([t + e * u if n == i else t for n, t in enumerate(x)]) -
                loss([t - e * u if n == i else t for n, t in enumerate(x)])) / (2 * e)
        assert abs((got[i].double().cpu() * u).sum().item() - diff) <= (tols[i] * u.abs()).sum().item()


def test_attention_views(ck):
    """Views of a fused projection, heads-first and joint buffers: the same bits as contiguous tensors."""
    t, hq, hk, d = 200, 4, 2, 128
    g = _gen(31)
    row = _rand(g, t, hq + 2 * hk, d).cuda()
    q, k, v = row[:, :hq], row[:, hq:hq + hk], row[:, hq + hk:]
    want, lse = ck.attention(q.contiguous(), k.contiguous(), v.contiguous(), causal=True)
    do = _rand(g, hq, t, d).cuda().transpose(0, 1)
    grads = ck.attention_backward(do.contiguous(), q.contiguous(), k.contiguous(), v.contiguous(), want, lse, causal=True)
    out = torch.full((t, hq + 1, d), 5.0, dtype=BF16, device="cuda")
    got, lse2 = ck.attention(q, k, v, causal=True, out=out[:, 1:])
    drow = torch.full_like(row, 5.0)
    got_g = ck.attention_backward(do, q, k, v, out[:, 1:], lse2, causal=True, dq=drow[:, :hq], dk=drow[:, hq:hq + hk],
                                  dv=drow[:, hq + hk:])
    assert all(torch.equal(a, b) for a, b in zip(_bits(got, lse2, *got_g), _bits(want, lse, *grads)))
    assert (out[:, 0] == 5).all()


def test_attention_other_sequences_never_reach_a_row(ck):
    """NaN and infinities in a neighbour's keys and values, in tiles that both sequences share."""
    lens, hq, d = [70, 33, 90], 2, 64
    cu = _dev_cu(_cu(lens))
    q, k, v, do = (t.cuda() for t in _attn_inputs(lens, lens, hq, hq, d, 41))
    for causal in (False, True):
        want = ck.attention(q, k, v, cu, cu, causal=causal)
        k2, v2 = k.clone(), v.clone()
        k2[70:103], v2[70:103] = math.nan, math.inf
        got = ck.attention(q, k2, v2, cu, cu, causal=causal)
        g1 = ck.attention_backward(do, q, k, v, *want, cu, cu, causal=causal)
        g2 = ck.attention_backward(do, q, k2, v2, *want, cu, cu, causal=causal)
        rows = torch.cat((torch.arange(70), torch.arange(103, 193))).cuda()
        assert all(torch.equal(a, b) for a, b in zip(_bits(got[0][rows], got[1][:, rows]),
                                                     _bits(want[0][rows], want[1][:, rows])))
        assert all(torch.equal(a[rows], b[rows]) for a, b in zip(g1, g2))


def test_attention_extreme_scores(ck):
    """Scores of thousands, all of one sign, and one key far above the rest: no overflow, the oracle's results."""
    g = _gen(51)
    for mean in (0.0, 30.0, -30.0):
        q, k, v = _rand(g, 150, 1, 64, std=0.2), _rand(g, 200, 1, 64, std=0.2), _rand(g, 200, 1, 64)
        q = (q + 30).to(BF16)
        k = (k + mean / 30).to(BF16)
        k[137] = 20
        out, lse = ck.attention(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
        want, want_lse, tol, lse_tol = ao.attention(q.double(), k.double(), v.double(), [0, 150], [0, 200], False, 1.0)
        # scores of this size are off by their own fp32 roundings: so is every weight
        s = 2.0 ** -20 * (q.double()[:, 0].abs() @ k.double()[:, 0].abs().t()).amax(-1)[:, None, None]
        _near(out, want, tol + s * v.double().abs().max(), "out")
        _near(lse, want_lse, lse_tol, "lse")


def test_attention_starts_out_of_range(ck):
    """Starts past the tensors or out of order: nothing outside the tensors is written (which of the sequences that
    claim a row writes it last is open), and keys outside them are not read."""
    q, k, v, do = (t.cuda() for t in _attn_inputs([100], [100], 1, 1, 64, 61))
    cu = _dev_cu([0, 60, 1 << 30, -5, 1 << 30])
    bufs = [torch.full((300, 1, 64), 3.0, dtype=BF16, device="cuda") for _ in range(4)]
    views = [b[100:200] for b in bufs]
    pad_k, pad_v = (torch.full((300, 1, 64), math.nan, dtype=BF16, device="cuda") for _ in range(2))
    pad_k[100:200], pad_v[100:200] = k, v
    out, lse = ck.attention(q, pad_k[100:200], pad_v[100:200], cu, cu, out=views[0])
    ck.attention_backward(do, q, pad_k[100:200], pad_v[100:200], out, lse, cu, cu, dq=views[1], dk=views[2], dv=views[3])
    for b in bufs:
        assert torch.isfinite(b.float()).all() and (b[:100] == 3).all() and (b[200:] == 3).all()


@pytest.mark.parametrize("tq,tk,seqs,hq,hk,d", [
    (1024, 1344, 3, 1, 1, 128), (2560, 1280, 10, 1, 1, 64), (2560, 1280, 9, 2, 1, 128), (700, 4000, 30, 4, 2, 72),
])
@pytest.mark.parametrize("causal", [False, True])
def test_attention_starts_out_of_order_and_cut_tiles(ck, tq, tk, seqs, hq, hk, d, causal):
    """Every other sequence claims all rows, at sizes whose tiles are cut: nothing outside the workspace and the tensors
    is written."""
    q, k, v, do = (t.cuda() for t in _attn_inputs([tq], [tk], hq, hk, d, tq + tk))
    cu_q, cu_k = (_dev_cu([n if i % 2 else 0 for i in range(seqs + 1)]) for n in (tq, tk))
    lib, guard = ck.lib(), 1 << 20
    sizes = [f(seqs, tq, tk, hq, hk, d) for f in (lib.ck4_attention_workspace_bytes, lib.ck4_attention_backward_workspace_bytes)]
    assert sizes[0] > 0
    room = [torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda") for n in sizes]
    ws = [r[guard:guard + n] for r, n in zip(room, sizes)]
    bufs = [torch.full((x.shape[0] + 200, *x.shape[1:]), 3.0, dtype=BF16, device="cuda") for x in (q, q, k, k)]
    views = [b[100:-100] for b in bufs]
    out, lse = ck.attention(q, k, v, cu_q, cu_k, causal=causal, out=views[0], workspace=ws[0])
    ck.attention_backward(do, q, k, v, out, lse, cu_q, cu_k, causal=causal, dq=views[1], dk=views[2], dv=views[3],
                          workspace=ws[1])
    for r, n in zip(room, sizes):
        assert (r[:guard] == 0xA5).all() and (r[guard + n:] == 0xA5).all()
    for b in bufs:
        assert (b[:100] == 3).all() and (b[-100:] == 3).all()


def test_attention_streams_and_graph(ck):
    """On a stream that is not the default one, and captured into a graph and replayed on new data."""
    t, hq, hk, d = 190, 4, 2, 64
    data = [_attn_inputs([t], [t], hq, hk, d, s) for s in (71, 72, 73)]
    w, pos = torch.ones(d, device="cuda"), torch.arange(t, device="cuda", dtype=torch.int32)
    freqs = torch.rand(32, generator=_gen(74)).cuda()
    cache = [torch.zeros(2, t, hk, d, dtype=BF16, device="cuda") for _ in range(2)]
    lengths = torch.tensor([t, 33], dtype=torch.int32, device="cuda")

    def block(q, k, v, do):
        qn, kn = ck.qk_norm_rope(q, k, w, w, pos, freqs)
        out, lse = ck.attention(qn, kn, v, causal=True)
        dqn, dkn, dv = ck.attention_backward(do, qn, kn, v, out, lse, causal=True)
        grads = ck.qk_norm_rope_backward(dqn, dkn, q, k, w, w, pos, freqs)
        cache[0][:] = kn
        cache[1][:] = v
        return [out, lse, dv, *grads, *ck.attention_decode(qn[-2:], *cache, lengths)]

    want = [_bits(*block(*(x.cuda() for x in xs))) for xs in data]
    static = [x.cuda() for x in data[0]]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = block(*static)
    assert all(torch.equal(a, b) for a, b in zip(_bits(*got), want[0]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(*static)
    for i in (0, 1, 2, 1, 0):
        for x, y in zip(static, data[i]):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(_bits(*got), want[i])), i


@pytest.mark.parametrize("which,reach", [("k", 0), ("v", 95)])
@pytest.mark.parametrize("at", [63, 64, 300])
def test_attention_causal_nonfinite(ck, which, reach, at):
    """NaN in one key or value of a causal sequence: all rows that see it, and of the earlier ones none or the nearest."""
    g = _gen(at)
    q, k, v = _rand(g, 400, 4, 128), _rand(g, 400, 2, 128), _rand(g, 400, 2, 128)
    bad_k, bad_v = k.clone(), v.clone()
    (bad_k if which == "k" else bad_v)[at] = math.nan
    out, lse = ck.attention(q.cuda(), bad_k.cuda(), bad_v.cuda(), causal=True)
    want, want_lse, tol, lse_tol = ao.attention(q.double(), k.double(), v.double(), [0, 400], [0, 400], True, 128 ** -0.5)
    free = max(0, at - reach)
    _near(out[:free], want[:free], tol[:free], "out")
    _near(lse[:, :free], want_lse[:, :free], lse_tol[:, :free], "lse")
    assert out[at:].isnan().all()


@pytest.mark.parametrize("n,hq,hk,d", [(700, 4, 2, 128), (1500, 4, 2, 64), (700, 24, 24, 72)])
@pytest.mark.parametrize("at", [63, 64, 300])
def test_attention_backward_causal_nonfinite(ck, n, hq, hk, d, at):
    """NaN in one row of q, k, v or dout of a causal sequence: gradients that do not depend on it, and are further than
    320 from it, are the same bits as without it."""
    q, k, v, do = (x.cuda() for x in _attn_inputs([n], [n], hq, hk, d, at + n))
    out, lse = ck.attention(q, k, v, causal=True)
    want = ck.attention_backward(do, q, k, v, out, lse, causal=True)
    for which in range(4):
        x = [do, q, k, v]
        x[which] = x[which].clone()
        x[which][at] = math.inf if which % 2 else math.nan
        got = ck.attention_backward(*x, *ck.attention(*x[1:], causal=True), causal=True)
        if which < 2:  # a row: the other rows' dq, and the keys after it
            free_q = torch.arange(n) != at
            assert got[0][at].isnan().all()
            after = slice(min(n, at + 321), None)
            assert all(torch.equal(a[after], b[after]) for a, b in zip(_bits(*got[1:]), _bits(*want[1:])))
        else:  # a key: the rows before it
            free_q = torch.arange(n) < at - 320
        assert torch.equal(_bits(got[0])[0][free_q], _bits(want[0])[0][free_q])


# ------------------------------------------------------------ decoding

# lengths, slots, hq, hk, d
DECODES = [
    ([1], 1, 1, 1, 64),
    ([0], 5, 2, 1, 64),
    ([0, 3, 0, 0, 100, 0], 100, 4, 2, 128),       # empty sequences between others
    ([31, 32, 33, 64, 65], 70, 8, 8, 128),
    ([500], 500, 40, 8, 128),
    ([3000], 3001, 5, 1, 128),                    # one unit over many workgroups
    ([700, 1, 1300], 1300, 34, 1, 64),            # more query heads than a column block
    ([256, 77], 300, 48, 3, 96),
    ([100 + 13 * i for i in range(70)], 1100, 3, 1, 40),  # more sequences than lanes
    ([5, 9], 16, 2, 2, 8),
]
# either side of the lengths at which the work is dealt otherwise
DECODES += [
    ([512, 300, 0], 512, 4, 2, 128), ([513, 1, 0, 257], 513, 4, 2, 128), ([2048, 2047, 33], 2048, 6, 2, 64),
    ([2049, 0, 31], 2049, 6, 2, 64), ([0, 3, 0, 0, 100, 0], 2100, 4, 2, 128), ([700, 1, 1300], 2200, 34, 1, 64),
    ([1900, 5], 2000, 20, 1, 128), ([50 + 29 * i for i in range(70)], 2064, 3, 1, 40), ([4096], 5000, 17, 1, 128),
]

# so many units that one group of threads joins each
DECODES += [
    ([2100, 0, 1, 700, 33] * 4, 2100, 40, 8, 128), ([100 + 97 * i for i in range(21)], 2065, 40, 8, 64),
    ([2500 - 700 * (i % 4) for i in range(33)], 2500, 20, 4, 72),
]


@pytest.mark.parametrize("layout", ["slots_first", "heads_first"])
@pytest.mark.parametrize("lengths,slots,hq,hk,d", DECODES)
def test_decode(ck, lengths, slots, hq, hk, d, layout):
    b, g = len(lengths), _gen(sum(lengths) + d)
    q = _rand(g, b, hq, d, std=1.5)
    kv = [_rand(g, b, slots, hk, d) for _ in range(2)]
    for c in kv:
        for i, n in enumerate(lengths):
            c[i, n:] = math.nan  # what a slot past the length holds does not matter
    dev = [c.cuda() for c in kv]
    if layout == "heads_first":
        dev = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in dev]
    out, lse = ck.attention_decode(q.cuda(), *dev, torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for i, n in enumerate(lengths):
        want, want_lse, tol, lse_tol = ao.attention(q[i:i + 1].double(), kv[0][i, :n].double(), kv[1][i, :n].double(),
                                                    [0, 1], [0, n], False, d ** -0.5)
        _near(out[i:i + 1], want, tol, f"out {i}")
        _near(lse[:, i:i + 1], want_lse, lse_tol, f"lse {i}")


def test_decode_lengths_out_of_range(ck):
    g = _gen(81)
    q, k, v = (_rand(g, 2, 2, 64).cuda(), _rand(g, 2, 50, 1, 64).cuda(), _rand(g, 2, 50, 1, 64).cuda())
    want, _ = ck.attention_decode(q, k, v, torch.tensor([50, 0], dtype=torch.int32, device="cuda"))
    got, _ = ck.attention_decode(q, k, v, torch.tensor([1 << 30, -7], dtype=torch.int32, device="cuda"))
    assert torch.equal(*_bits(got, want))


def test_decode_agrees_with_attention(ck):
    """One new token: the last row of the causal call over the same keys, within both bounds."""
    g = _gen(91)
    q, k, v = _rand(g, 400, 10, 128), _rand(g, 400, 2, 128), _rand(g, 400, 2, 128)
    full, lse = ck.attention(q.cuda(), k.cuda(), v.cuda(), causal=True)
    out, lse1 = ck.attention_decode(q[-1:].cuda(), k.cuda()[None], v.cuda()[None],
                                    torch.tensor([400], dtype=torch.int32, device="cuda"))
    _, _, tol, lse_tol = ao.attention(q[-1:].double(), k.double(), v.double(), [0, 1], [0, 400], False, 128 ** -0.5)
    _near(out, full[-1:].double().cpu(), 2 * tol, "out")
    _near(lse1, lse[:, -1:].double().cpu(), 2 * lse_tol, "lse")


def test_long_cache_offsets(ck):
    """Element offsets past 2^31 and byte offsets past 2^32: the last sequence of a 9 GB cache, and a far slot."""
    slots, hk, d = 1 << 20, 8, 128
    base = torch.zeros(slots * 4 + 64, hk, d, dtype=BF16, device="cuda")
    g = _gen(95)
    q, new = _rand(g, 1, hk, d), _rand(g, 100, hk, d)
    base[-100:] = new.cuda()
    far = base[-100:][None]
    want, _ = ck.attention_decode(q.cuda(), new.cuda()[None], new.cuda()[None],
                                  torch.tensor([100], dtype=torch.int32, device="cuda"))
    # a batch of two whose second sequence lies 4 * 2^20 - 36 rows into the buffer
    two = base.as_strided((2, 100, hk, d), ((base.shape[0] - 100) * hk * d, hk * d, d, 1))
    got, _ = ck.attention_decode(q.repeat(2, 1, 1).cuda(), two, two, torch.tensor([0, 100], dtype=torch.int32, device="cuda"))
    assert torch.equal(*_bits(got[1:], want)) and (got[0] == 0).all()
    # the same rows as the last sequence of a packed call
    cu = torch.tensor([0, 0, 1], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, base.shape[0] - 100, base.shape[0]], dtype=torch.int32, device="cuda")
    o1, _ = ck.attention(q.cuda(), base, base, cu, cu_k)
    o2, _ = ck.attention(q.cuda(), far[0], far[0])
    assert torch.equal(*_bits(o1, o2))


def test_example_block(ck):
    """The example's new token gives what the prompt pass gives for the same token at a sequence's end."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "attention_block.py")
    spec = importlib.util.spec_from_file_location("attention_block", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    r = ex.run(tokens=200, hidden=512, heads=8, kv_heads=2)
    assert all(torch.isfinite(t.float()).all() for t in [r["prompt"], r["token"], *r["grads"].values()])
    xs, pos, lens = [], [], [n + 1 for n in r["lens"]]
    for i, n in enumerate(r["lens"]):
        a = int(r["cu"][i])
        xs += [r["x"][a:a + n], r["new"][i:i + 1]]
        pos.append(torch.arange(n + 1))
    cu = _dev_cu(_cu(lens))
    block = r["block"]
    q, k, v = block.project(torch.cat(xs))
    q, k = block.norm(q, k, torch.cat(pos).int().cuda())
    heads, _ = ck.attention(q, k, v, cu, cu, causal=True)
    rows = (cu[1:] - 1).long()
    # the same token's attention through the cache, before the output projection quantises it
    caches = [torch.zeros(len(lens), max(lens), 2, 64, dtype=BF16, device="cuda") for _ in range(2)]
    for i, n in enumerate(lens):
        a = int(cu[i])
        caches[0][i, :n], caches[1][i, :n] = k[a:a + n], v[a:a + n]
    out, _ = ck.attention_decode(q[rows], *caches, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    _, _, tol, _ = ao.attention(q.double().cpu(), k.double().cpu(), v.double().cpu(), _cu(lens), _cu(lens), True, 64 ** -0.5)
    _near(out, heads[rows].double().cpu(), 2 * tol[rows.cpu()], "token")
    torch.testing.assert_close(r["token"], block.output(out), rtol=0, atol=0)
