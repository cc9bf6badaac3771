"""The decode calls on the GPU where their arithmetic, their sizes or their buffers come to an edge:
logits of large size, the longest rows, buffers of calls on other streams, states that overlap."""
import math

import pytest
import torch

from test_gpu_decode import DT, api, attn_inputs, bits, call, check_select, dev, ok, select_reference  # noqa: F401  (api: a fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ selection
# Tolerances are check_select's: beside the errors named there, the exponent of a term, a difference of
# two numbers that are each rounded to 24 bits, is up to 64 in size where logits are near 1e9, so it is off by
# 2^-18 at most, and a total by ln 2 times that; 64-bit totals near 1e9 are off by 2^-22.
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1000, 20001])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("size", [1e4, 1e5, 1e6, 1e7, 7e7, 8e7, 1e8, 9e8, 1e9, 1.1e9, 1e12])
def test_select_logits_of_large_size(api, size, sign, V, dtype):
    """Rows whose largest logits are far from zero: all tokens equal, a spread of a few units around the
    value, a few representable steps around it, and tokens of ordinary size beside it (the value as a
    mask, or as the only token that counts)."""
    g = torch.Generator().manual_seed(V)
    m = sign * size
    x = torch.full((6, V), m)
    x[1] += 3 * torch.randn(V, generator=g)
    x[2] *= 1 + torch.randint(-3, 4, (V,), generator=g) * torch.finfo(DT[dtype]).eps
    x[3] = torch.where(torch.rand(V, generator=g) < 0.5, torch.randn(V, generator=g), x[3])
    x[4, 1:] = torch.randn(V - 1, generator=g)
    x[5] = 2 * torch.randn(V, generator=g)
    x = x.to(DT[dtype])
    # a request per row: each row's totals; then all rows as beams of one request, nearly level
    cum = -torch.rand(6, 1, generator=g)
    got = api.beam_select(x.cuda(), cum.cuda(), 20)
    ok(api)
    check_select(got, select_reference(x, cum, 20), 20)
    assert (got[0] == 0).all()
    got = api.beam_select(x.cuda(), cum.view(1, 6).cuda(), 200)
    ok(api)
    check_select(got, select_reference(x, cum.view(1, 6), 200), 200)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fill", [-1e8, -1e9])
def test_select_row_filled_with_a_mask_value(api, fill, dtype):
    """A beam whose tokens were all filled with the usual mask value offers them as equals."""
    V, k = 300, 256
    x = torch.full((1, V), fill).to(DT[dtype])
    par, tok, sc = api.beam_select(x.cuda(), torch.tensor([[-1.5]]).cuda(), k)
    ok(api)
    assert par[0].tolist() == [0] * k and tok[0].tolist() == list(range(k))
    assert (sc.double().cpu() - (-1.5 - math.log(V))).abs().max() <= 2.0 ** -16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(50, 8), (50, 70), (9000, 256), (40000, 100)])
def test_select_totals_outside_fp32(api, V, k, dtype):
    """Totals below fp32's range are finite in 64 bits: such a token is still a candidate, in its place,
    and its score is -inf, the total rounded to fp32.  -inf itself offers nothing."""
    g = torch.Generator().manual_seed(V)
    low = -3.3e38 * torch.rand(2, V, generator=g)
    x = low.clone()
    x[0, 3], x[1, V // 2] = 3e38, math.inf                  # the second row: +inf leaves the others a total of -inf
    x[0, 5] = -math.inf
    x = x.to(DT[dtype])
    y = torch.stack([torch.zeros(V), low[1]]).to(DT[dtype])
    for logits, cum in ((x, torch.tensor([[-1.0, -0.5]])), (y, torch.tensor([[-3.4e38, -2e38]]))):
        got = api.beam_select(logits.cuda(), cum.cuda(), k)
        ok(api)
        want = select_reference(logits, cum, k)[0][:k]
        n = len(want)
        assert got[0][0].tolist() == [w[1] for w in want] + [-1] * (k - n)
        assert got[1][0].tolist() == [w[3] for w in want] + [-1] * (k - n)
        total = torch.tensor([w[0] for w in want] + [-math.inf] * (k - n), dtype=torch.float64)
        assert (total[:n] > -math.inf).all()
        score, rounded = got[2][0].cpu(), total.float()
        assert torch.equal(score == -math.inf, rounded == -math.inf)
        at = rounded > -math.inf
        assert ((score[at].double() - total[at]).abs() <= 2.0 ** -16 + 2.0 ** -23 * total[at].abs()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,V,k", [(2, 1 << 24, 256), (256, 1 << 17, 256), (256, 160001, 100), (1, (1 << 24) - 5, 7)])
def test_select_largest_sizes(api, W, V, k, dtype):
    """The reference is check_select's, formed on the GPU: the k + 50 best totals of each call in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(V + W)
    x = (torch.randn(W, V, generator=g, device="cuda") * 2).to(DT[dtype])
    x[:, V - 1] = 9.0                                        # the last token is among the best
    cum = -2 * torch.rand(1, W, generator=g, device="cuda")
    got = api.beam_select(x, cum, k)
    ok(api)
    found = []
    for b in range(W):
        y = x[b].double()
        lse = torch.logsumexp(y, 0)
        top = torch.topk(y, k).values[-1]
        at = torch.nonzero(y >= top).view(-1)
        found += [(float(cum[0, b]) + float(y[v] - lse), b, float(y[v]), int(v)) for v in at[torch.argsort(-y[at], stable=True)[:k + 50]]]
    found.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
    check_select(got, [found], k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W,V,k", [(32, 8192, 32), (32, 131072, 256), (1, 100003, 7), (256, 2500, 256)])
@pytest.mark.parametrize("fill", [0.0, -1e9])
def test_select_level_rows(api, fill, W, V, k, dtype):
    """Beams of equal logits: the lowest tokens of the first of the best beams, in each of two requests."""
    x = torch.full((2 * W, V), fill, device="cuda").to(DT[dtype])
    cum = torch.full((2, W), -1.0)
    cum[1, :W // 2] = -1.5
    got = api.beam_select(x, cum.cuda(), k)
    ok(api)
    for r, b in ((0, 0), (1, W // 2)):
        assert got[0][r].tolist() == [b] * k and got[1][r].tolist() == list(range(k))
    assert (got[2].double().cpu() - (-1.0 - math.log(V))).abs().max() <= 2.0 ** -16


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5000, 60000])
@pytest.mark.parametrize("n1,n3,n4", [(100, 50, 1600), (256, 0, 1600), (0, 300, 1600), (255, 1, 1600), (7, 2, 1700)])
def test_select_ties_across_beams(api, n1, n3, n4, V, dtype):
    """Beams with copies of one row of three values, three of them with equal totals, whose masks allow few of
    its best tokens: more tokens tie at the last place than are sorted, and the ties go on from beam to beam."""
    W, k, best = 6, 256, [1, 3, 4]
    g = torch.Generator().manual_seed(V + n1)
    row = torch.randint(0, 3, (V,), generator=g).float()
    row[torch.randperm(V, generator=g)[:1800]] = 2.0
    top = torch.nonzero(row == 2).view(-1)
    allowed = torch.zeros(W, V, dtype=torch.bool)
    want = []
    for b, n in zip(best, (n1, n3, n4)):
        at = top[torch.randperm(len(top), generator=g)[:n]].sort().values
        allowed[b, at] = True
        allowed[b, torch.nonzero(row == 0).view(-1)] = True
        want += [(b, int(v)) for v in at]
    allowed[[0, 2, 5]] = True
    cum = torch.tensor([[-9.0, -1.0, -9.0, -1.0, -1.0, -9.0]])
    x = row.expand(W, V).contiguous().to(DT[dtype])
    got = api.beam_select(x.cuda(), cum.cuda(), k, allowed=bits(allowed).cuda())
    ok(api)
    assert list(zip(got[0][0].tolist(), got[1][0].tolist())) == want[:k]
    assert (got[2][0] == got[2][0, 0]).all()


def test_select_nothing_to_offer(api):
    """Requests whose beams are all dead, or whose masks allow nothing, beside one that offers."""
    R, W, V, k = 4, 3, 9000, 5
    x = torch.randn(R * W, V, generator=torch.Generator().manual_seed(2))
    cum = torch.full((R, W), -math.inf)
    cum[1], cum[3] = -1.0, -2.0
    words = torch.full((R * W, -(-V // 32)), -1, dtype=torch.int32)
    words[9:] = 0
    got = api.beam_select(x.cuda(), cum.cuda(), k, allowed=words.cuda())
    ok(api)
    check_select(got, select_reference(x, cum, k, None, (words != 0).repeat_interleave(32, 1)[:, :V]), k)
    for r in (0, 2, 3):
        assert got[0][r].tolist() == got[1][r].tolist() == [-1] * k and torch.isneginf(got[2][r]).all()


def test_select_score_over_cum(api):
    """With k == W the score may be cum itself."""
    R, W, V = 6, 5, 3000
    x = torch.randn(R * W, V, generator=torch.Generator().manual_seed(4)).cuda()
    cum = -torch.rand(R, W, generator=torch.Generator().manual_seed(5)).cuda()
    want = api.beam_select(x, cum, W)
    got = api.beam_select(x, cum, W, score=cum)
    ok(api)
    assert got[2].data_ptr() == cum.data_ptr() and all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ streams
def _choose(api, x, **kw):
    return api.beam_select(x["logits"], x["cum"], 20, **kw)


def _stream_inputs(what, seed):
    if what == "attention":
        return dev(attn_inputs(seed, [33, 20], [1500, 900], 8, 2, 128, 7))
    g = torch.Generator().manual_seed(seed)
    return {"logits": torch.randn(32, 30000, generator=g).cuda(), "cum": -torch.rand(4, 8, generator=g).cuda()}


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("what,run", [("attention", call), ("selection", _choose)])
def test_buffers_of_a_call_on_another_stream(api, what, run, handle):
    """Results and workspace of a call on a side stream share no memory with blocks that the current stream
    still works on, whether freed before the call or after its results were used."""
    x, y = _stream_inputs(what, 1), _stream_inputs(what, 2)
    want, other = run(api, x), run(api, y)
    ok(api)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    torch.cuda.empty_cache()
    # blocks of every size that the call may ask for, freed while the current stream has yet to fill them
    sizes = [t.numel() * t.element_size() for t in want] + [1 << n for n in range(8, 25)]
    torch.cuda._sleep(100_000_000)
    held = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    spans = [(t.data_ptr(), t.data_ptr() + t.numel()) for t in held]
    for t in held:
        t.fill_(255)
    del held, t
    got = run(api, x, stream=stream)
    assert not any(a <= t.data_ptr() < b for t in got for a, b in spans)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # results that the current stream has yet to read, freed, and a second call
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    kept = [t.clone() for t in got]
    del got
    again = run(api, y, stream=stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))
    assert all(torch.equal(a, b) for a, b in zip(again, other))
    ok(api)


@pytest.mark.parametrize("what,run", [("attention", call), ("selection", _choose)])
def test_buffers_come_from_the_stream_given(api, what, run):
    """A stream, its handle, the default stream's handle 0 and none at all, called while another stream is current:
    each result is in memory that torch's allocator holds for the call's own stream."""
    x = _stream_inputs(what, 3)
    want = run(api, x)
    ok(api)
    side, here = torch.cuda.Stream(), torch.cuda.Stream()

    def owner(t):
        seg, = [s for s in torch.cuda.memory_snapshot() if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        return seg["stream"]
    for stream, handle in ((side, side.cuda_stream), (side.cuda_stream, side.cuda_stream), (0, 0), (torch.cuda.default_stream(), 0),
                           (None, here.cuda_stream)):
        with torch.cuda.stream(here):
            got = run(api, x, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert [owner(t) for t in got] == [handle] * len(got), stream
    ok(api)


# ------------------------------------------------------------------ reordering
def test_reorder_refuses_conflicts_among_many_states(api):
    """Over 64 states: one listed twice, an out that is another's state, two equal outs, wherever they stand,
    are refused before anything moves; K and V of joint caches, and states read twice, are not."""
    R, W, n = 2, 3, 150
    par = torch.tensor([[1, 2, 0], [2, 2, 1]], dtype=torch.int32).cuda()
    rows = torch.tensor([1, 2, 0, 5, 5, 4])
    init = torch.arange(n * R * W * 5, dtype=torch.float32).view(n, R * W, 5)

    def fresh():
        return list(init.cuda().unbind(0)), list(torch.zeros(n, R * W, 5, device="cuda").unbind(0))
    for i, j in ((0, 1), (0, 64), (63, 64), (2, 149), (70, 140), (149, 5)):
        st, out = fresh()
        twice = list(st)
        twice[j] = st[i]
        with pytest.raises(api.TrError):
            api.beam_reorder(twice, par)
        into = list(out)
        into[i] = st[j]
        with pytest.raises(api.TrError):
            api.beam_reorder(st, par, outs=into)
        same = list(out)
        same[i] = out[j]
        with pytest.raises(api.TrError):
            api.beam_reorder(st, par, outs=same)
        ok(api)
        assert torch.equal(torch.stack(st).cpu(), init) and not torch.stack(out).any()
        got = api.beam_reorder(twice, par, outs=out)             # read twice
        ok(api)
        assert torch.equal(got[j].cpu(), init[i][rows]) and torch.equal(got[i].cpu(), init[i][rows])
    joint = torch.arange(40 * R * W * 2 * 5, dtype=torch.float32).view(40, R * W, 2, 5)
    d = joint.cuda()
    api.beam_reorder([d[i, :, kv] for i in range(40) for kv in range(2)], par)
    ok(api)
    assert torch.equal(d.cpu(), joint[:, rows])


def test_reorder_refuses_its_own_parent(api):
    par = torch.tensor([[1, 2, 0], [2, 2, 1]], dtype=torch.int32).cuda()
    with pytest.raises(api.TrError):
        api.beam_reorder([par.view(6)], par)
    ok(api)
    assert par.tolist() == [[1, 2, 0], [2, 2, 1]]


@pytest.mark.parametrize("row", [(1 << 30) + 48, (1 << 28) + 4])
def test_reorder_rows_and_states_beyond_32_bits(api, row):
    """Rows of a gigabyte and a state of several, in place; then rows of another state 2^32 bytes apart."""
    R, W = 2, 3
    x = torch.randint(-2**31, 2**31, (R * W, row // 4), dtype=torch.int32, device="cuda")
    ends = [0, row // 8, row // 4 - 1]
    before, sums = x[:, ends].clone(), x.sum(1)
    par = torch.tensor([[1, 2, 0], [2, 2, 1]], dtype=torch.int32).cuda()
    rows = torch.tensor([1, 2, 0, 5, 5, 4]).cuda()
    api.beam_reorder([x], par)
    ok(api)
    assert torch.equal(x[:, ends], before[rows]) and torch.equal(x.sum(1), sums[rows])
    del x
    far = torch.empty(5 * (1 << 30) + 64, dtype=torch.int32, device="cuda").as_strided((R * W, 16), (1 << 30, 1))
    far.copy_(torch.arange(96, dtype=torch.int32).view(6, 16))
    api.beam_reorder([far], par)
    ok(api)
    assert torch.equal(far.cpu(), torch.arange(96, dtype=torch.int32).view(6, 16)[rows.cpu()])
