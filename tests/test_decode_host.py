"""Refusals of the decode calls (tr_prefix_attention, tr_beam_select, tr_beam_reorder) on the
host: each invalid argument is named and nothing is launched, so no GPU is needed."""
import ctypes as C

import pytest
import torch

P = 1 << 20    # a 16-byte aligned address that no refused call touches


@pytest.fixture(scope="module")
def lib():
    from transformer_candidate_scoring_b200 import _lib, build
    build.build()
    return _lib.load()


def _L():
    from transformer_candidate_scoring_b200 import _lib
    return _lib


def off(*v):
    return (C.c_int64 * len(v))(*v)


def desc(**over):
    d = dict(n_head=8, n_kv_head=2, d_head=64, L_t=1, causal=0, suffix_cap=4, scale=0.125, dtype=1, q_token=512,
             prefix_token=128, prefix_head=64, suffix_seq=512, suffix_token=128, suffix_head=64)
    d.update(over)
    return _L().AttnDesc(*[d[n] for n, _ in _L().AttnDesc._fields_])


def attn(lib, d=None, seq=(0, 2, 3), pre=(0, 5, 9), R=2, q=P, kp=P, vp=P, ks=P, vs=P, sl=P, out=P, lse=P, ws=P, wb=1 << 40):
    return lib.tr_prefix_attention(C.byref(d) if d is not None else None, q, off(*seq) if seq else None, kp, vp,
                                   off(*pre) if pre else None, ks, vs, sl, R, out, lse, ws, wb, None)


BAD_DESC = [dict(n_head=7), dict(n_kv_head=0), dict(n_head=0), dict(n_head=1026, n_kv_head=2), dict(d_head=60), dict(d_head=0),
            dict(d_head=136), dict(L_t=0), dict(L_t=17), dict(causal=2), dict(suffix_cap=-1), dict(scale=float("nan")),
            dict(scale=float("inf")), dict(scale=0.0), dict(scale=-1.0), dict(prefix_token=0), dict(dtype=5), dict(q_token=516), dict(prefix_token=-128), dict(prefix_head=4),
            dict(suffix_seq=1), dict(suffix_token=2), dict(suffix_head=12), dict(q_token=1 << 40)]


@pytest.mark.parametrize("over", BAD_DESC, ids=str)
def test_attention_refuses_descriptions(lib, over):
    L = _L()
    assert attn(lib, desc(**over)) in (L.TR_ERR_INVALID_ARG, L.TR_ERR_UNSUPPORTED)
    assert lib.tr_last_error()
    assert lib.tr_prefix_attention_workspace(C.byref(desc(**over)), off(0, 2, 3), off(0, 5, 9), 2) == C.c_size_t(-1).value


def test_attention_refuses_offsets_and_pointers(lib):
    L = _L()
    bad = L.TR_ERR_INVALID_ARG
    assert attn(lib, None) == bad
    assert attn(lib, desc(), R=0) == bad
    assert attn(lib, desc(), R=L.TR_MAX_REQUESTS + 1) == bad
    assert attn(lib, desc(), seq=None) == bad
    assert attn(lib, desc(), pre=None) == bad
    assert attn(lib, desc(), seq=(1, 2, 3)) == bad
    assert attn(lib, desc(), seq=(0, 3, 2)) == bad
    assert attn(lib, desc(), pre=(-1, 5, 9)) == bad
    assert attn(lib, desc(), pre=(0, 5, 4)) == bad
    assert attn(lib, desc(), pre=(0, 5, 1 << 31)) == L.TR_ERR_UNSUPPORTED
    assert attn(lib, desc(), seq=(0, 5, 1 << 28)) == L.TR_ERR_UNSUPPORTED       # 2^31 query rows
    for name in ("q", "kp", "vp", "ks", "vs", "sl", "out"):
        assert attn(lib, desc(), **{name: None}) == bad, name
        assert b"null" in lib.tr_last_error()
    for name in ("q", "kp", "vp", "ks", "vs", "out"):
        assert attn(lib, desc(), **{name: P + 8}) == bad, name
        assert b"16-byte" in lib.tr_last_error()
    assert attn(lib, desc(), sl=P + 2) == bad
    assert attn(lib, desc(), lse=P + 2) == bad
    # no sequences: nothing to do, whatever the pointers are
    assert attn(lib, desc(), seq=(0, 0, 0), q=None, out=None) == L.TR_OK


def select(lib, logits=P, dt=0, ld=100, cum=P, fin=None, al=None, ald=0, R=2, W=3, V=100, k=4, pad=0, par=P, tok=P, sc=P, ws=P,
           wb=1 << 40):
    return lib.tr_beam_select(logits, dt, ld, cum, fin, al, ald, R, W, V, k, pad, par, tok, sc, ws, wb, None)


@pytest.mark.parametrize("kw", [dict(W=0), dict(W=257), dict(R=0), dict(R=1 << 19), dict(V=0), dict(V=(1 << 24) + 1, ld=1 << 25),
                                dict(k=0), dict(k=257), dict(dt=3), dict(ld=99), dict(al=P, ald=3), dict(pad=-1),
                                dict(pad=1 << 24), dict(logits=None), dict(cum=None), dict(par=None), dict(tok=None),
                                dict(sc=None), dict(logits=P + 2), dict(cum=P + 1), dict(al=P + 2, ald=4), dict(par=P + 2),
                                dict(ws=None), dict(ws=P + 4), dict(wb=16)], ids=str)
def test_select_refuses(lib, kw):
    assert select(lib, **kw) == _L().TR_ERR_INVALID_ARG
    assert lib.tr_last_error()


def test_select_workspace_refuses_bad_sizes(lib):
    assert lib.tr_beam_select_workspace(2, 0, 10, 3) == C.c_size_t(-1).value
    assert lib.tr_beam_select_workspace(2, 4, 10, 300) == C.c_size_t(-1).value
    assert 0 < lib.tr_beam_select_workspace(2, 4, 10, 3) < 1 << 20


def move(lib, states, R=2, W_in=4, W_out=4, parent=P, n=None):
    L = _L()
    arr = (L.BeamState * max(len(states), 1))(*[L.BeamState(*s) for s in states])
    return lib.tr_beam_reorder(arr, len(states) if n is None else n, parent, R, W_in, W_out, None)


def test_reorder_refuses(lib):
    L = _L()
    bad = L.TR_ERR_INVALID_ARG
    a, b = P, 2 * P
    ok = (a, b, 64, 64, 64)
    assert move(lib, [ok], R=0) == bad
    assert move(lib, [ok], W_in=0) == bad
    assert move(lib, [ok], W_out=257) == bad
    assert move(lib, [ok], R=1 << 19) == bad
    assert move(lib, [ok], parent=None) == bad
    assert move(lib, [ok], parent=P + 2) == bad
    assert move(lib, [ok], n=65) == bad
    assert move(lib, [ok], n=-1) == bad
    assert move(lib, [(None, b, 64, 64, 64)]) == bad
    assert move(lib, [(a, None, 64, 64, 64)]) == bad
    assert move(lib, [(a, b, 63, 64, 64)]) == bad                       # stride below the row
    assert move(lib, [(a, b, 64, 63, 64)]) == bad
    assert move(lib, [(a, b, 64, 64, -1)]) == bad
    assert move(lib, [(a, a, 64, 64, 64)], W_out=3) == bad              # in place with another width
    assert move(lib, [(a, a, 64, 128, 64)]) == bad
    assert move(lib, [(a, a + 64, 64, 64, 64)]) == bad                  # overlaps, but not in place
    assert move(lib, [(a, a + 32, 128, 128, 64)]) == bad                # interleaved too tightly
    assert move(lib, [(a, b, 64, 64, 64), (b, a + 4 * P, 64, 64, 64)]) == bad    # one's dst is another's src
    assert move(lib, [(a, b, 64, 64, 64), (a, b + 4 * P, 64, 64, 64)]) == bad    # the same dst twice
    assert move(lib, [], n=0) == L.TR_OK


def test_binding_refuses_host_tensors_and_shapes():
    from transformer_candidate_scoring_b200 import api
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    k = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.prefix_attention(q, k, k, [0, 5], [0, 2])
    with pytest.raises(ValueError, match="CUDA"):
        api.beam_select(torch.zeros(4, 10), torch.zeros(2, 2), 3)
    with pytest.raises(ValueError, match="CUDA"):
        api.beam_reorder([torch.zeros(4, 8)], torch.zeros(2, 2, dtype=torch.int32))
