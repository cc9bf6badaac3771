"""Refusals of tr_beam_reorder_check, on the host, over more states than one call takes, and of a parent that
would move too."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from transformer_candidate_scoring_b200 import _lib, build
    build.build()
    return _lib.load()


def check(lib, states, R=2, W_in=4, W_out=4, n=None, parent=1 << 40):
    from transformer_candidate_scoring_b200 import _lib as L
    arr = (L.BeamState * max(len(states), 1))(*[L.BeamState(*s) for s in states])
    return lib.tr_beam_reorder_check(arr, len(states) if n is None else n, parent, R, W_in, W_out)


def test_reorder_check_sees_all_states(lib):
    from transformer_candidate_scoring_b200 import _lib as L
    bad, n = L.TR_ERR_INVALID_ARG, 150
    src, dst = [(i + 1) << 16 for i in range(n)], [(i + 1000) << 16 for i in range(n)]

    def rows(dst, src):
        return [(d, s, 64, 64, 64) for d, s in zip(dst, src)]
    assert check(lib, rows(dst, src)) == L.TR_OK
    assert check(lib, rows(src, src)) == L.TR_OK                       # all in place
    assert check(lib, rows(dst, [src[0]] * n)) == L.TR_OK              # all from one
    assert check(lib, rows([dst[0] + 64 * i for i in range(n)], src)) == bad
    joint = [(dst[0] + 64 * i, src[0] + 64 * i, 64 * n, 64 * n, 64) for i in range(n)]
    assert check(lib, joint) == L.TR_OK                                # rows interleaved at one stride
    for i, j in ((0, 64), (63, 64), (2, 149), (149, 5)):
        for with_dst, with_src in ((dst[:i] + [dst[j]] + dst[i + 1:], src), (dst[:i] + [src[j]] + dst[i + 1:], src),
                                   (dst[:i] + [src[j] + 64 * 7] + dst[i + 1:], src), (src, src[:i] + [src[j]] + src[i + 1:])):
            assert check(lib, rows(with_dst, with_src)) == bad, (i, j)
            assert b"overlaps" in lib.tr_last_error()
        assert check(lib, rows(dst[:i] + [src[j] + 64 * 8] + dst[i + 1:], src)) == L.TR_OK     # just behind its rows


def test_reorder_check_refuses_what_the_call_refuses(lib):
    from transformer_candidate_scoring_b200 import _lib as L
    bad, a, b = L.TR_ERR_INVALID_ARG, 1 << 20, 2 << 20
    one = [(a, b, 64, 64, 64)]
    assert check(lib, one) == L.TR_OK and check(lib, []) == L.TR_OK
    assert check(lib, one, R=0) == bad and check(lib, one, W_in=0) == bad and check(lib, one, W_out=257) == bad
    assert check(lib, one, R=1 << 19) == bad and check(lib, one, n=-1) == bad
    assert lib.tr_beam_reorder_check(None, 1, 1 << 40, 2, 4, 4) == bad
    assert check(lib, one, parent=None) == bad and check(lib, one, parent=a + 64 * 7) == bad and check(lib, one, parent=b) == L.TR_OK
    assert check(lib, [(None, b, 64, 64, 64)]) == bad and check(lib, [(a, b, 63, 64, 64)]) == bad
    assert check(lib, [(a, a, 64, 64, 64)], W_out=3) == bad and check(lib, [(a, b, 64, 64, -1)]) == bad


def test_reorder_refuses_a_dst_over_parent(lib):
    from transformer_candidate_scoring_b200 import _lib as L
    a, b, par = 1 << 20, 2 << 20, 3 << 20                                # parent: 16 x 4 int32, 256 bytes
    # rows too long for one grid: a call that passes the check of parent is refused for them, nothing is launched
    huge = (1 << 50, 1 << 51, 1 << 40, 1 << 40, 1 << 40)

    def call(*states):
        arr = (L.BeamState * (len(states) + 1))(*[L.BeamState(*s) for s in states], L.BeamState(*huge))
        return lib.tr_beam_reorder(arr, len(states) + 1, par, 16, 4, 4, None)
    for dst in (par, par - 63 * 64, par + 252):
        assert call((a, b, 64, 64, 64), (dst, b, 64, 64, 64)) == L.TR_ERR_INVALID_ARG, dst - par
        assert b"parent" in lib.tr_last_error()
    assert call((par, par, 4, 4, 4)) == L.TR_ERR_INVALID_ARG             # parent itself, in place
    assert b"parent" in lib.tr_last_error()
    for dst in (par - 64 * 64, par + 256):                               # beside it
        assert call((dst, b, 64, 64, 64)) not in (L.TR_OK, L.TR_ERR_INVALID_ARG)
        assert b"parent" not in lib.tr_last_error()
