"""The plain forms of perf/operators.py against the 64-bit oracle (CPU)."""
import importlib.util
import os

import pytest
import torch

import attention_oracle as ao

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


@pytest.fixture(scope="module")
def ops():
    spec = importlib.util.spec_from_file_location("perf_operators", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _norm_state(sections, interleaved, positions, d=72, hq=2, hk=1):
    g = torch.Generator().manual_seed(sum(positions))
    t, pairs = len(positions), sum(sections)
    freqs = torch.cat([torch.pow(10000.0, -torch.arange(m, dtype=torch.float64) / m) for m in sections]).float()
    bf = lambda h: torch.randn(t, h, d, generator=g).to(torch.bfloat16)  # noqa: E731
    return {"case": {"op": "norm_bwd", "interleaved": interleaved}, "q": bf(hq), "k": bf(hk), "dq": bf(hq), "dk": bf(hk),
            "q_weight": 1 + 0.2 * torch.randn(d, generator=g), "k_weight": 1 + 0.2 * torch.randn(d, generator=g),
            "positions": torch.tensor(positions, dtype=torch.int32)[:, None].repeat(1, len(sections)), "freqs": freqs,
            "axis": torch.cat([torch.full((m,), i) for i, m in enumerate(sections)]), "sections": sections, "rot": 2 * pairs}


POSITIONS = [0, 1, 777, 4095, 12289, 19997, 20479]  # of one sequence: some offset and up to 16384 tokens


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("sections", [(32,), (16, 16), (4, 14, 14)])
def test_plain_norm_gradients_at_large_positions(ops, sections, interleaved):
    s = _norm_state(sections, interleaved, POSITIONS)
    angle = s["positions"].double()[:, s["axis"]] * s["freqs"].double()
    cos, sin = ops._angles(s)
    for got, want in ((cos, angle.cos()), (sin, angle.sin())):
        # one rounding to fp32 of a value of at most 1, and the 64-bit function's own last place
        assert (got[:, 0].double() - want).abs().max() <= 2.0 ** -24
    dq, dk, dwq, dwk = ops.run(s)
    for x, w, dy, dx, dw in ((s["q"], s["q_weight"], s["dq"], dq, dwq), (s["k"], s["k_weight"], s["dk"], dk, dwk)):
        x, w, dy = x.double(), w.double(), dy.double()
        want, want_w, _ = ao.norm_rope_backward(dy, x, w, s["positions"].double(), s["freqs"].double(), sections,
                                                interleaved)
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        # at most 14 terms z n of at most |g|_a + |g|_b times |n|: some 10 roundings each and 13 of the sum, 2^-24 of them
        size = (2 * dy.abs().amax(-1, keepdim=True) * n.abs()).sum((0, 1))
        assert ((dw.double() - want_w).abs() <= 2.0 ** -19 * size).all()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
        size = (2 * dy.abs() * r).amax(-1, keepdim=True) * w.abs().max()
        assert ((dx.double() - want).abs() <= ao.EPS * want.abs() + 2.0 ** -18 * size).all()
