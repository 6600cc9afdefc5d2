"""Refusals of the attention-block operators (no GPU needed, nothing is
launched): the binding's checks of tensors, and the C ABI's of raw arguments."""
import ctypes

import pytest
import torch

import int4_w4a4_quantized_amd as ck

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def _h(t, heads, d, dtype=BF16):
    return torch.zeros(t, heads, d, dtype=dtype)


def _norm(**kw):
    a = dict(q=_h(4, 3, 64), k=_h(4, 2, 64), q_weight=torch.ones(64), k_weight=torch.ones(64),
             positions=torch.zeros(4, 2, dtype=I32), freqs=torch.ones(32), sections=(20, 12))
    a.update(kw)
    return ck.qk_norm_rope(**a)


def _norm_bwd(**kw):
    a = dict(dq_out=_h(4, 3, 64), dk_out=_h(4, 2, 64), q=_h(4, 3, 64), k=_h(4, 2, 64), q_weight=torch.ones(64),
             k_weight=None, positions=torch.zeros(4, 2, dtype=I32), freqs=torch.ones(32), sections=(20, 12))
    a.update(kw)
    return ck.qk_norm_rope_backward(**a)


def _attn(**kw):
    a = dict(q=_h(6, 4, 64), k=_h(8, 2, 64), v=_h(8, 2, 64), cu_q=torch.tensor([0, 6], dtype=I32),
             cu_k=torch.tensor([0, 8], dtype=I32))
    a.update(kw)
    return ck.attention(**a)


def _attn_bwd(**kw):
    a = dict(dout=_h(6, 4, 64), q=_h(6, 4, 64), k=_h(8, 2, 64), v=_h(8, 2, 64), out=_h(6, 4, 64), lse=torch.zeros(4, 6))
    a.update(kw)
    return ck.attention_backward(**a)


def _decode(**kw):
    a = dict(q=_h(2, 4, 64), k_cache=torch.zeros(2, 9, 2, 64, dtype=BF16), v_cache=torch.zeros(2, 9, 2, 64, dtype=BF16),
             lengths=torch.ones(2, dtype=I32))
    a.update(kw)
    return ck.attention_decode(**a)


BAD = [
    (_norm, dict(q=_h(4, 3, 64, F32)), "bfloat16"),
    (_norm, dict(q=_h(4, 3, 64)[0]), "tokens, heads, d"),
    (_norm, dict(k=_h(5, 2, 64)), "shape"),
    (_norm, dict(k=_h(4, 2, 72)), "heads of"),
    (_norm, dict(q=_h(4, 64, 3).transpose(1, 2)), "unit stride"),
    (_norm, dict(q_weight=torch.ones(32)), "q_weight"),
    (_norm, dict(k_weight=torch.ones(64, dtype=BF16)), "k_weight"),
    (_norm, dict(positions=torch.zeros(4, 2, dtype=torch.int64)), "positions"),
    (_norm, dict(positions=torch.zeros(4, 3, dtype=I32)), "positions"),
    (_norm, dict(positions=torch.zeros(3, 2, dtype=I32)), "positions"),
    (_norm, dict(freqs=torch.ones(31)), "sections hold"),
    (_norm, dict(freqs=torch.ones(33), sections=(20, 13)), "do not fit"),
    (_norm, dict(q_out=_h(4, 2, 64)), "q_out"),
    (_norm, dict(), "CUDA"),
    (_norm_bwd, dict(dq_out=_h(4, 2, 64)), "dq_out"),
    (_norm_bwd, dict(dk=_h(4, 2, 72)), "dk"),
    (_norm_bwd, dict(workspace=torch.zeros(8)), "workspace"),
    (_norm_bwd, dict(), "CUDA"),
    (_attn, dict(v=_h(8, 1, 64)), "v must"),
    (_attn, dict(k=_h(8, 2, 72), v=_h(8, 2, 72)), "heads of"),
    (_attn, dict(cu_q=None), "cu_q"),
    (_attn, dict(cu_k=torch.tensor([0, 4, 8], dtype=I32)), "one start more"),
    (_attn, dict(cu_q=torch.tensor([0, 6]), cu_k=torch.tensor([0, 8])), "cu_q"),
    (_attn, dict(out=_h(6, 2, 64)), "out"),
    (_attn, dict(lse=torch.zeros(6, 4)), "lse"),
    (_attn, dict(), "CUDA"),
    (_attn_bwd, dict(dout=_h(5, 4, 64)), "dout"),
    (_attn_bwd, dict(lse=torch.zeros(4, 6, dtype=torch.float64)), "lse"),
    (_attn_bwd, dict(dv=_h(8, 4, 64)), "dv"),
    (_attn_bwd, dict(), "CUDA"),
    (_decode, dict(k_cache=torch.zeros(3, 9, 2, 64, dtype=BF16)), "k_cache"),
    (_decode, dict(v_cache=torch.zeros(2, 8, 2, 64, dtype=BF16)), "v_cache"),
    (_decode, dict(lengths=torch.ones(3, dtype=I32)), "lengths"),
    (_decode, dict(lengths=torch.ones(2, dtype=torch.int64)), "lengths"),
    (_decode, dict(), "CUDA"),
]


@pytest.mark.parametrize("call,args,said", BAD)
def test_binding_refuses(call, args, said):
    with pytest.raises(ValueError, match=said):
        call(**args)


# The C ABI. Pointers are never followed: every call here is refused.
P, ODD = 1 << 20, (1 << 20) + 4
INV, UNS = ck.CK4_ERR_INVALID, ck.CK4_ERR_UNSUPPORTED
SECS = (ctypes.c_int * 4)(8, 8, 8, 8)

NORM = dict(q=P, q_st=192, q_sh=64, k=P, k_st=128, k_sh=64, tokens=4, hq=3, hk=2, d=64, qw=P, kw=P, pos=P, f32=0, axes=4,
            secs=SECS, freqs=P, inter=1, eps=1e-6, qo=P, qo_st=192, qo_sh=64, ko=P, ko_st=128, ko_sh=64, stream=None)
ATTN = dict(q=P, q_st=256, q_sh=64, k=P, k_st=128, k_sh=64, v=P, v_st=128, v_sh=64, cu_q=P, cu_k=P, seqs=3, tq=6, tk=8,
            hq=4, hk=2, d=64, causal=1, scale=0.125, o=P, o_st=256, o_sh=64, lse=P, ws=None, ws_bytes=0, stream=None)
DEC = dict(q=P, q_st=256, q_sh=64, k=P, k_sb=1280, k_st=128, k_sh=64, v=P, v_sb=1280, v_st=128, v_sh=64, lengths=P,
           batch=2, slots=1000, hq=4, hk=2, d=64, scale=0.125, o=P, o_st=256, o_sh=64, lse=P, ws=P, ws_bytes=1 << 40,
           stream=None)
ABI = [
    ("ck4_qk_norm_rope", NORM, [
        (dict(q=None), INV), (dict(pos=None), INV), (dict(secs=None), INV), (dict(ko=None), INV), (dict(tokens=0), INV),
        (dict(hk=-1), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(d=60), UNS), (dict(d=264), UNS),
        (dict(axes=0), UNS), (dict(axes=5), UNS), (dict(secs=(ctypes.c_int * 4)(8, 8, 8, 9)), INV),
        (dict(secs=(ctypes.c_int * 4)(8, -1, 8, 8)), INV), (dict(q=ODD), INV), (dict(ko=ODD), INV), (dict(q_st=196), INV),
        (dict(k_sh=56), INV), (dict(q_st=-192), INV), (dict(q_st=1 << 25), UNS), (dict(qo_st=64), INV),
        (dict(qo_sh=128, qo_st=192), INV), (dict(freqs=P + 2), INV), (dict(tokens=1 << 40), UNS), (dict(hq=5000), UNS),
    ]),
    ("ck4_attention", ATTN, [
        (dict(v=None), INV), (dict(o=None), INV), (dict(cu_q=None), INV), (dict(cu_q=None, cu_k=None), INV),
        (dict(cu_k=P + 1), INV), (dict(tq=0), INV), (dict(tk=-1), INV), (dict(seqs=0), INV), (dict(hq=3), INV),
        (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=float("inf")), INV), (dict(scale=2e6), UNS), (dict(d=68), UNS),
        (dict(d=136), UNS), (dict(k=ODD), INV), (dict(v_st=56), INV), (dict(k_st=1 << 25), UNS), (dict(o_sh=32), INV),
        (dict(o_st=64), INV), (dict(lse=P + 2), INV), (dict(seqs=1 << 30), UNS), (dict(tq=1 << 31), UNS),
        (dict(hq=1 << 20, hk=1 << 20), UNS), (dict(tq=1 << 30, hq=4096), UNS), (dict(ws=P + 8), INV),
        (dict(tk=5000), INV), (dict(tk=5000, ws=P, ws_bytes=100), INV),  # few rows, many keys: a workspace is needed
    ]),
    ("ck4_attention_decode", DEC, [
        (dict(lengths=None), INV), (dict(slots=5000, ws=None), INV), (dict(batch=0), INV), (dict(slots=0), INV), (dict(hk=3), INV),
        (dict(scale=float("nan")), INV), (dict(d=132), UNS), (dict(k_sb=1284), INV), (dict(v_sb=-8), INV),
        (dict(k_st=32), INV), (dict(v_st=1 << 25), UNS), (dict(slots=5000, ws_bytes=100), INV), (dict(ws=P + 8), INV),
        (dict(batch=1 << 21), UNS), (dict(slots=1 << 31), UNS), (dict(o_st=8), INV), (dict(k_sb=1 << 41), UNS),
    ]),
]


@pytest.mark.parametrize("fn,good,bad", ABI, ids=[a[0] for a in ABI])
def test_abi_refuses(fn, good, bad):
    f = getattr(ck.lib(), fn)
    for change, want in bad:
        assert f(*{**good, **change}.values()) == want, (change, ck.lib().ck4_last_error())
        assert ck.lib().ck4_last_error().decode().startswith(fn + ":")


def test_abi_refuses_backward():
    L = ck.lib()
    heads = dict(dout=P, a=256, b=64, q=P, q_st=256, q_sh=64, k=P, k_st=128, k_sh=64, v=P, v_st=128, v_sh=64, o=P,
                 o_st=256, o_sh=64)
    good = dict(heads, lse=P, cu_q=P, cu_k=P, seqs=3, tq=6, tk=8, hq=4, hk=2, d=64, causal=1, scale=0.125, dq=P, dq_st=256,
                dq_sh=64, dk=P, dk_st=128, dk_sh=64, dv=P, dv_st=128, dv_sh=64, ws=P, ws_bytes=1 << 40, stream=None)
    for change, want in [(dict(lse=None), INV), (dict(dk=None), INV), (dict(ws=None), INV), (dict(ws_bytes=10), INV),
                         (dict(dv_st=64), INV), (dict(dq=ODD), INV), (dict(b=60), INV), (dict(ws=P + 8), INV),
                         (dict(d=256), UNS), (dict(scale=0.0), INV)]:
        assert L.ck4_attention_backward(*{**good, **change}.values()) == want, change
    norm = dict(dqo=P, x=192, y=64, dko=P, z=128, w=64, q=P, q_st=192, q_sh=64, k=P, k_st=128, k_sh=64, tokens=4, hq=3,
                hk=2, d=64, qw=P, kw=P, pos=P, f32=0, axes=4, secs=SECS, freqs=P, inter=1, eps=1e-6, dq=P, dq_st=192,
                dq_sh=64, dk=P, dk_st=128, dk_sh=64, dqw=P, dkw=P, ws=P, ws_bytes=1 << 40, stream=None)
    for change, want in [(dict(dqo=None), INV), (dict(ws=None), INV), (dict(ws_bytes=10), INV), (dict(dq_st=64), INV),
                         (dict(dk_sh=60), INV), (dict(dqw=P + 1), INV), (dict(d=264), UNS), (dict(eps=-1e-6), INV)]:
        assert L.ck4_qk_norm_rope_backward(*{**norm, **change}.values()) == want, change


def test_workspace_sizes():
    L = ck.lib()
    assert L.ck4_qk_norm_rope_workspace_bytes(0, 64) == 0 and L.ck4_qk_norm_rope_workspace_bytes(5, 64) >= 5 * 2 * 64 * 4
    assert L.ck4_attention_backward_workspace_bytes(1, 7, 7, 0, 1, 64) == 0
    assert L.ck4_attention_backward_workspace_bytes(1, 7, 7, 3, 1, 64) >= 2 * 7 * 3 * 4
    assert L.ck4_attention_workspace_bytes(1, 7, 7, 3, 2, 64) == 0  # heads do not divide
    assert L.ck4_attention_workspace_bytes(1, 7, 7, 4, 2, 64) == 0  # short: not cut
    assert L.ck4_attention_workspace_bytes(1, 7, 7000, 4, 2, 64) > 0
    assert L.ck4_attention_workspace_bytes(1, 70000, 70000, 4, 2, 64) == 0  # enough tiles
    assert L.ck4_attention_decode_workspace_bytes(2, 5000, 5, 2, 64) == 0  # heads do not divide
    assert L.ck4_attention_decode_workspace_bytes(2, 100, 4, 2, 64) == 0  # short: units are not cut
    assert L.ck4_attention_decode_workspace_bytes(2, 5000, 4, 2, 64) > 0


@pytest.mark.parametrize("t,d", [(4, 264), (4, 60), (0, 64)])
def test_norm_gradients_refuse_sizes_without_a_workspace(monkeypatch, t, d):
    """Sizes that no workspace is given for end in the library's error, as in the forward call (host tensors: nothing is
    launched)."""
    monkeypatch.setattr(ck, "_gpu_stream", lambda *a: None)
    q, k, pos, freqs = _h(t, 3, d), _h(t, 2, d), torch.zeros(t, 1, dtype=I32), torch.ones(4)
    with pytest.raises(ck.Ck4Error) as fwd:
        ck.qk_norm_rope(q, k, None, None, pos, freqs)
    with pytest.raises(ck.Ck4Error) as bwd:
        ck.qk_norm_rope_backward(q, k, q, k, None, None, pos, freqs)
    assert bwd.value.status == fwd.value.status


@pytest.mark.parametrize("tq,tk,hk,d", [(6, 8, 2, 136), (6, 8, 2, 60), (6, 8, 3, 64), (0, 8, 2, 64), (6, 0, 2, 64)])
def test_attention_gradients_refuse_sizes_without_a_workspace(monkeypatch, tq, tk, hk, d):
    monkeypatch.setattr(ck, "_gpu_stream", lambda *a: None)
    q, k, lse = _h(tq, 4, d), _h(tk, hk, d), torch.zeros(4, tq)
    with pytest.raises(ck.Ck4Error) as fwd:
        ck.attention(q, k, k)
    with pytest.raises(ck.Ck4Error) as bwd:
        ck.attention_backward(q, q, k, k, q, lse)
    assert bwd.value.status == fwd.value.status


def test_no_workspace_size_for_refused_sizes():
    """The sizes are 0 where the calls refuse them: heads that are no multiple of 8, and more tiles than a launch takes."""
    L = ck.lib()
    big = 1 << 60
    norm = dict(dqo=P, x=192, y=64, dko=P, z=128, w=64, q=P, q_st=192, q_sh=64, k=P, k_st=128, k_sh=64, tokens=4, hq=3,
                hk=2, d=60, qw=None, kw=None, pos=P, f32=0, axes=1, secs=SECS, freqs=P, inter=1, eps=1e-6, dq=P, dq_st=192,
                dq_sh=64, dk=P, dk_st=128, dk_sh=64, dqw=P, dkw=P, ws=P, ws_bytes=big, stream=None)
    assert L.ck4_qk_norm_rope_backward(*norm.values()) == UNS
    assert L.ck4_qk_norm_rope_workspace_bytes(4, 60) == 0
    for seqs, tq, tk, hq, hk, d in [(3, 2000, 2000, 4, 2, 60), (1, 1 << 30, 8, 4096, 4096, 8), (1 << 20, 8, 8, 4096, 8, 64),
                                    (1, 8, 1 << 30, 4096, 4096, 8)]:
        q, k = (max(st, 8) for st in (hq * d, hk * d))
        good = {**ATTN, "seqs": seqs, "tq": tq, "tk": tk, "hq": hq, "hk": hk, "d": d, "q_st": q, "k_st": k, "v_st": k,
                "o_st": q, "q_sh": d, "k_sh": d, "v_sh": d, "o_sh": d, "ws": P, "ws_bytes": big}
        assert L.ck4_attention(*good.values()) == UNS
        assert L.ck4_attention_workspace_bytes(seqs, tq, tk, hq, hk, d) == 0
        assert L.ck4_attention_backward_workspace_bytes(seqs, tq, tk, hq, hk, d) == 0
    for batch, slots, hq, hk, d in [(2, 5000, 4, 2, 60), (1 << 20, 5000, 4096, 8, 64), (1 << 20, 1 << 30, 1, 1, 64)]:
        good = {**DEC, "batch": batch, "slots": slots, "hq": hq, "hk": hk, "d": d, "q_st": hq * d, "q_sh": d,
                "k_st": hk * d, "k_sh": d, "v_st": hk * d, "v_sh": d, "o_st": hq * d, "o_sh": d, "ws_bytes": big}
        assert L.ck4_attention_decode(*good.values()) == UNS
        assert L.ck4_attention_decode_workspace_bytes(batch, slots, hq, hk, d) == 0


@pytest.mark.parametrize("sections", [(64.0,), (20.5, 43.5), ("64",), (None,), 64, (1 << 32, 64 - (1 << 32))])
def test_sections_are_whole_numbers(monkeypatch, sections):
    """Whatever sections an earlier call had: a float that equals a whole number is refused too."""
    monkeypatch.setattr(ck, "_gpu_stream", lambda *a: None)
    monkeypatch.setattr(ck, "lib", lambda: pytest.fail("the library was called"))
    ck._host_ints((64,))
    q, pos = _h(4, 1, 128), torch.zeros(4, 2 if isinstance(sections, tuple) and len(sections) == 2 else 1, dtype=I32)
    with pytest.raises(ValueError, match="sections"):
        ck.qk_norm_rope(q, q, None, None, pos, torch.ones(64), sections)
