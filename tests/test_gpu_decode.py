"""The decode calls on the GPU against plain 64-bit implementations: shared-prefix attention,
beam selection, reordering of beam states, and a decode loop of the three.

Attention tolerances, element by element, from the arithmetic: with e = 2^-24 and A the largest
scale * sum_i |q_i k_i| of a row, a score is off by at most (d + 3) e A (products, sums, scale), a
softmax weight by that twice (numerator and sum) plus 2^-20 (exponential, division), so
    |out error| <= (2 (d + 3) e A + 2^-20 + n e) sum_j p_j |v_j|
over n keys.  bf16 adds its two roundings, half a step each: 2^-8 of sum_j p_j |v_j| for the
numerators of a value product and 2^-8 |out| for the result; and an output that is rounded to
bf16 from below its smallest normal number is off by less than 2^-133.
"""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def api():
    from transformer_candidate_scoring_b200 import api as a, build
    build.build()
    assert torch.cuda.is_available()
    return a


def ok(api):
    torch.cuda.synchronize()
    assert api.sync_status() == 0


# ------------------------------------------------------------------ attention
def attn_inputs(seed, counts, prefix, H, H_kv, d, S, L_t=1, dtype="bf16", lens=None, q_scale=2.0, lead=0):
    g = torch.Generator().manual_seed(seed)
    n, T = sum(counts), sum(prefix) + lead

    def rnd(*shape, s=1.0):
        return (torch.randn(*shape, generator=g) * s).to(DT[dtype])
    x = {"q": rnd(n, L_t, H, d, s=q_scale), "k": rnd(max(T, 1), H_kv, d), "v": rnd(max(T, 1), H_kv, d), "ks": None, "vs": None,
         "sl": None, "so": np.concatenate([[0], np.cumsum(counts)]).tolist(),
         "po": (lead + np.concatenate([[0], np.cumsum(prefix)])).tolist()}
    if S:
        x["ks"], x["vs"] = rnd(n, S, H_kv, d), rnd(n, S, H_kv, d)
        sl = torch.randint(0, S + 1, (n,), generator=g) if lens is None else torch.tensor([lens[i % len(lens)] for i in range(n)])
        x["sl"] = sl.to(torch.int32)
    return x


def attn_reference(x, scale, causal):
    """(out, lse, tolerance of out, tolerance of lse), in 64 bits."""
    q, k, v = x["q"].double(), x["k"].double(), x["v"].double()
    n, L_t, H, d = q.shape
    G = H // k.shape[1]
    bf = x["q"].dtype == torch.bfloat16
    out, lse = torch.zeros(n, L_t, H, d, dtype=torch.float64), torch.full((n, L_t, H), -math.inf, dtype=torch.float64)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(x["so"]) - 1):
        for s in range(x["so"][r], x["so"][r + 1]):
            for t in range(L_t):
                kk, vv = k[x["po"][r]:x["po"][r + 1]], v[x["po"][r]:x["po"][r + 1]]
                if x["ks"] is not None:
                    c = min(max(int(x["sl"][s]), 0), x["ks"].shape[1])
                    c = max(0, c - (L_t - 1 - t)) if causal else c
                    kk, vv = torch.cat([kk, x["ks"][s, :c].double()]), torch.cat([vv, x["vs"][s, :c].double()])
                if len(kk) == 0:
                    continue
                kk, vv = (z.repeat_interleave(G, 1) for z in (kk, vv))                 # [keys, H, d]
                a = torch.einsum("hd,jhd->hj", q[s, t], kk) * scale
                lse[s, t] = torch.logsumexp(a, -1)
                p = torch.exp(a - lse[s, t][:, None])
                out[s, t] = torch.einsum("hj,jhd->hd", p, vv)
                A = (torch.einsum("hd,jhd->hj", q[s, t].abs(), kk.abs()) * abs(scale)).amax(-1)
                pv = torch.einsum("hj,jhd->hd", p, vv.abs())
                rel = 2 * (d + 3) * EPS * A + 2.0 ** -20 + len(kk) * EPS
                tol[s, t] = rel[:, None] * pv
                if bf:
                    tol[s, t] += 2.0 ** -8 * pv + 2.0 ** -8 * out[s, t].abs() + 2.0 ** -133
                tol_l[s, t] = rel + EPS * lse[s, t].abs()
    return out, lse, tol, tol_l


def dev(x):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in x.items()}


def call(api, x, **kw):
    return api.prefix_attention(x["q"], x["k"], x["v"], x["po"], x["so"], x["ks"], x["vs"], x["sl"], **kw)


def agrees(got, x, scale, causal):
    out, lse, tol, tol_l = attn_reference(x, scale, causal)
    o, z = (t.double().cpu().view(r.shape) for t, r in zip(got, (out, lse)))
    empty = lse == -math.inf
    assert torch.equal(z == -math.inf, empty)
    assert bool((o[empty] == 0).all())
    bad = (o - out).abs() > tol
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), ((o - out).abs() / tol.clamp(min=1e-300)).max().item())
    bad = (z[~empty] - lse[~empty]).abs() > tol_l[~empty]
    assert not bad.any(), ((z[~empty] - lse[~empty]).abs() / tol_l[~empty]).max().item()


ATTN = [
    # counts, prefix, H, H_kv, d, S, L_t, causal
    ([1], [1], 1, 1, 64, 0, 1, False),
    ([3], [0], 4, 2, 64, 3, 1, False),                       # no prefix at all
    ([4, 2], [200, 7], 8, 8, 64, 4, 1, False),
    ([5, 0, 3], [33, 10, 0], 6, 2, 128, 5, 1, False),        # a request without sequences, one without prefix
    ([7], [129], 8, 1, 128, 17, 1, False),                   # eight heads share one key head
    ([2, 3], [127, 128], 5, 5, 16, 1, 1, False),
    ([9], [300], 6, 2, 80, 9, 3, True),
    ([9], [65], 6, 2, 96, 9, 3, False),
    ([3], [64], 3, 1, 8, 2, 16, True),                       # more query tokens than suffix keys: empty rows
    ([3], [0], 3, 3, 40, 20, 16, True),
    ([130], [130], 3, 1, 72, 3, 1, False),                   # rows that end inside a tile
    ([40, 1, 86], [257, 513, 1], 4, 2, 128, 33, 2, True),
    ([2], [5000], 4, 4, 32, 130, 1, False),                  # a long prefix for few rows
    ([300, 2], [1100, 700], 8, 4, 64, 2, 1, False),
    ([1], [2], 64, 1, 128, 300, 1, False),
    ([3, 2, 4], [0, 50, 0], 4, 2, 64, 1, 1, False),          # one own key, requests without a prefix
    ([3, 2, 140], [0, 50, 0], 4, 2, 128, 0, 1, False),
    ([5, 66], [0, 3], 8, 2, 32, 1, 2, True),
    ([150, 9], [260, 0], 4, 1, 96, 1, 1, False),
    ([130, 7], [300, 0], 2, 1, 104, 4, 4, True),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("case", ATTN, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}x{c[3]}x{c[4]}-s{c[5]}-t{c[6]}{'c' if c[7] else ''}".replace(" ", ""))
def test_attention(api, case, dtype):
    counts, prefix, H, H_kv, d, S, L_t, causal = case
    x = attn_inputs(sum(prefix) + d + S, counts, prefix, H, H_kv, d, S, L_t, dtype)
    got = call(api, dev(x), causal=causal)
    ok(api)
    assert got[0].dtype == DT[dtype] and got[0].shape == x["q"].shape and got[1].shape == x["q"].shape[:-1]
    agrees(got, x, d ** -0.5, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_strides_scale_and_single_token_form(api, dtype):
    """q out of a fused projection, K and V joint in one buffer with heads outermost, a suffix
    buffer with its own strides, tokens before the first request, another scale, [n, H, d]."""
    counts, prefix, H, H_kv, d, S = [4, 9], [70, 150], 4, 2, 64, 6
    x = attn_inputs(5, counts, prefix, H, H_kv, d, S, 1, dtype, lead=11)
    n, T = sum(counts), x["k"].shape[0]
    y = dev(x)
    fused = torch.full((n, (H + 2 * H_kv) * d), float("nan"), dtype=DT[dtype], device="cuda")
    fused[:, :H * d] = y["q"].view(n, H * d)
    joint = torch.full((2, H_kv, T + 3, d), float("nan"), dtype=DT[dtype], device="cuda")
    joint[0, :, :T], joint[1, :, :T] = y["k"].transpose(0, 1), y["v"].transpose(0, 1)
    suffix = torch.full((n, 2, S + 2, H_kv, d), float("nan"), dtype=DT[dtype], device="cuda")
    suffix[:, 0, :S], suffix[:, 1, :S] = y["ks"], y["vs"]
    got = api.prefix_attention(fused[:, :H * d].view(n, H, d), joint[0].transpose(0, 1)[:T], joint[1].transpose(0, 1)[:T],
                               x["po"], x["so"], suffix[:, 0, :S], suffix[:, 1, :S], y["sl"], scale=0.31)
    ok(api)
    assert got[0].shape == (n, H, d) and got[1].shape == (n, H)
    agrees(got, x, 0.31, False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_attention_ignores_values_behind_prefix_and_suffix(api, dtype, bad):
    """Rows behind a prefix, between requests and behind a suffix hold NaN or infinities."""
    counts, H, H_kv, d, S = [3, 140], 4, 2, 128, 40
    x = attn_inputs(6, counts, [37, 141], H, H_kv, d, S, 1, dtype, lens=[0, 1, 17, 39])
    gap, dirty = 9, {}
    po = [4, 4 + 37, 4 + 37 + gap, 4 + 37 + gap + 141]
    for name in ("k", "v"):
        z = torch.full((po[-1] + 200, H_kv, d), bad, dtype=DT[dtype])
        z[po[0]:po[1]], z[po[2]:po[3]] = x[name][:37], x[name][37:178]
        dirty[name] = z
    y = dict(x)
    for name in ("ks", "vs"):
        z = x[name].clone()
        for s in range(sum(counts)):
            z[s, int(x["sl"][s]):] = bad
        y[name] = z
    y = dev(y)
    # one call per request, as the requests' prefixes are not adjacent here
    for r, (p0, p1) in enumerate(((po[0], po[1]), (po[2], po[3]))):
        s0, s1 = x["so"][r], x["so"][r + 1]
        got = api.prefix_attention(y["q"][s0:s1], dirty["k"].cuda(), dirty["v"].cuda(), [p0, p1], [0, s1 - s0], y["ks"][s0:s1],
                                   y["vs"][s0:s1], y["sl"][s0:s1])
        ok(api)
        part = dict(x, q=x["q"][s0:s1], ks=x["ks"][s0:s1], vs=x["vs"][s0:s1], sl=x["sl"][s0:s1], so=[0, s1 - s0],
                    po=[x["po"][r], x["po"][r + 1]])
        agrees(got, part, d ** -0.5, False)


@pytest.mark.parametrize("d", [64, 104])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_attention_causal_rows_ignore_later_values(api, dtype, bad, d):
    """The values of a sequence's last two tokens hold NaN or infinities: the query tokens before
    them get what they get without, the others what the formula gives."""
    x = attn_inputs(16, [2, 3], [20, 0], 6, 2, d, 40, 5, dtype, lens=[40, 33, 9, 2, 17])
    y = dict(x, vs=x["vs"].clone())
    for s in range(5):
        y["vs"][s, max(0, int(x["sl"][s]) - 2):int(x["sl"][s])] = bad
    clean, got = (call(api, dev(z), causal=True) for z in (x, y))
    ok(api)
    agrees(clean, x, d ** -0.5, True)
    agrees((got[0][:, :3], got[1][:, :3]), dict(x, q=x["q"][:, :3], sl=(x["sl"] - 2).clamp(min=0)), d ** -0.5, True)
    late = got[0][:, 3:].float()
    assert bool((torch.isnan(late) if bad != bad else late == bad).all())
    assert torch.equal(got[1], clean[1])                    # scores do not read values


# More units of rows than SMs, the last wave of them less than half full, the last unit of a key head shorter than a tile.
WAVES = [([2400], [130], 16, 16, 16, 1, 1, False), ([2300, 7], [129, 0], 20, 20, 128, 0, 1, False),
         ([2400], [70], 16, 16, 104, 2, 1, False), ([1203], [300], 16, 16, 64, 4, 2, True)]


@pytest.mark.parametrize("case", WAVES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}x{c[4]}-s{c[5]}".replace(" ", ""))
def test_attention_partial_last_wave(api, case):
    counts, prefix, H, H_kv, d, S, L_t, causal = case
    x = attn_inputs(18, counts, prefix, H, H_kv, d, S, L_t)
    got = call(api, dev(x), causal=causal)
    ok(api)
    agrees(got, x, d ** -0.5, causal)


# Several short units per SM, some without any key of the prefix.
SHORT = [(64, 1), (128, 1), (128, 0), (40, 1), (128, 5), (64, 12)]


@pytest.mark.parametrize("d,S", SHORT)
def test_attention_many_short_prefixes(api, d, S):
    R, H = 60, 10
    counts = [(3 * i + 1) % 7 for i in range(R)]
    prefix = [0 if i % 4 == 1 else (37 * i) % 300 for i in range(R)]
    L_t = 2 if S else 1
    x = attn_inputs(19, counts, prefix, H, H, d, S, L_t)
    got = call(api, dev(x), causal=S > 0)
    ok(api)
    agrees(got, x, d ** -0.5, S > 0)


@pytest.mark.parametrize("d,S", [(64, 1), (128, 1), (128, 0), (40, 0), (128, 9), (64, 3)])
def test_attention_many_units_of_one_tile(api, d, S):
    """The same with more rows each, up to 60 per key head."""
    R, H = 60, 10
    counts = [(13 * i) % 60 + 1 for i in range(R)]
    prefix = [0 if i % 4 == 1 else (37 * i) % 300 + 100 for i in range(R)]
    x = attn_inputs(20, counts, prefix, H, H, d, S)
    got = call(api, dev(x))
    ok(api)
    agrees(got, x, d ** -0.5, False)


RAGGED = [5003, 1, 700, 2049, 4100, 128, 127, 5990, 3333, 129, 64, 2500, 1111, 5500, 900, 0, 4999, 2222]
RUNS = [
    # counts, prefix, H, H_kv, d, S, L_t, causal
    ([1 + i % 2 for i in range(18)], RAGGED, 8, 8, 64, 3, 1, False),
    ([1 + i % 2 for i in range(17)] + [0], RAGGED, 16, 8, 128, 9, 1, False),
    ([1 + i % 2 for i in range(18)], RAGGED, 10, 10, 32, 0, 1, False),
    ([1 + i % 2 for i in range(17)] + [35], RAGGED, 16, 8, 96, 1, 2, True),      # of the last, two tiles of rows
]


@pytest.mark.parametrize("case", RUNS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}x{c[3]}x{c[4]}".replace(" ", ""))
def test_attention_ragged_long_prefixes(api, case):
    """Prefixes of very different lengths for few rows each: their keys are shared out by equal runs."""
    counts, prefix, H, H_kv, d, S, L_t, causal = case
    x = attn_inputs(17, counts, prefix, H, H_kv, d, S, L_t)
    got = call(api, dev(x), causal=causal)
    again = call(api, dev(x), causal=causal)
    ok(api)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    agrees(got, x, d ** -0.5, causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_neighbouring_prefixes_do_not_leak(api, dtype):
    """A request whose prefix holds NaN leaves the requests before and after it untouched."""
    x = attn_inputs(7, [5, 2, 6], [50, 30, 77], 4, 2, 64, 3, 1, dtype)
    clean = call(api, dev(x))
    y = dict(x, k=x["k"].clone(), v=x["v"].clone())
    y["k"][50:80] = float("nan")
    y["v"][50:80] = float("nan")
    got = call(api, dev(y))
    ok(api)
    for a, b in zip(got, clean):
        assert torch.equal(a[:5], b[:5]) and torch.equal(a[7:], b[7:])
        assert torch.isnan(a[5:7].float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_large_scores(api, dtype):
    """Scores of several hundred, all of one sign in each half of the rows, rising key by key so
    that the running maximum keeps growing; and a single-key row, whose result is its value."""
    x = attn_inputs(8, [6], [400], 2, 1, 64, 0, 1, dtype)
    ramp = torch.linspace(0.01, 1.0, 400)
    x["k"] = (torch.ones(400, 1, 64) * ramp[:, None, None]).to(DT[dtype])
    x["q"] = torch.full((6, 1, 2, 64), 40.0).to(DT[dtype])
    x["q"][:, :, 1] *= -1
    got = call(api, dev(x))
    ok(api)
    agrees(got, x, 0.125, False)
    one = attn_inputs(9, [5], [1], 4, 2, 64, 0, 1, dtype, q_scale=30.0)
    out, _ = call(api, dev(one))
    ok(api)
    assert torch.equal(out.cpu(), one["v"][0].repeat_interleave(2, 0).expand(5, 1, 4, 64))


def test_attention_bad_suffix_length_is_clamped_and_reported(api):
    x = attn_inputs(10, [4], [20], 4, 2, 64, 5, lens=[0, 5, -3, 900])
    got = call(api, dev(x))
    torch.cuda.synchronize()
    from transformer_candidate_scoring_b200 import _lib as L
    assert api.sync_status() == L.TR_ERR_KEY_RANGE
    assert api.sync_status() == 0
    agrees(got, x, 0.125, False)


def test_attention_empty_batches(api):
    x = attn_inputs(11, [0, 0], [5, 6], 4, 2, 64, 0)
    out, lse = call(api, dev(x))
    ok(api)
    assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 1, 4)
    x = attn_inputs(12, [3], [0], 4, 2, 64, 0)
    out, lse = call(api, dev(x))
    ok(api)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_attention_buffers_streams_and_repeats(api):
    """Caller's out, lse and workspace on a side stream; nothing behind them is written; the same
    inputs give the same bits each time."""
    x = attn_inputs(13, [33, 20], [1500, 900], 8, 2, 128, 7)
    y = dev(x)
    first = call(api, y)
    ok(api)
    o = torch.full((53 * 8 * 128 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((53 * 8 + 64,), 7.0, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        call(api, y, out=o[:53 * 8 * 128].view(53, 1, 8, 128), lse=z[:53 * 8].view(53, 1, 8), stream=side)
    side.synchronize()
    assert torch.equal(o[:53 * 8 * 128].view(53, 1, 8, 128), first[0]) and torch.equal(z[:53 * 8].view(53, 1, 8), first[1])
    assert bool((o[53 * 8 * 128:] == 7).all()) and bool((z[53 * 8:] == 7).all())
    with pytest.raises(ValueError):
        call(api, y, out=o[:10])


def test_attention_binding_refusals(api):
    x = dev(attn_inputs(14, [3], [5], 4, 2, 64, 2))
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"], x["k"], x["v"][:4], x["po"], x["so"])
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"].float(), x["k"], x["v"], x["po"], x["so"])
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"], x["k"], x["v"], [0, 6], x["so"])
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"], x["k"], x["v"], x["po"], [0, 2])
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"], x["k"], x["v"], x["po"], x["so"], x["ks"], x["vs"])
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"], x["k"], x["v"], x["po"], x["so"], x["ks"], x["vs"], x["sl"].long())
    with pytest.raises(ValueError):
        api.prefix_attention(x["q"].transpose(2, 3).contiguous().transpose(2, 3), x["k"], x["v"], x["po"], x["so"])
    with pytest.raises(api.TrError):                       # heads of 4
        api.prefix_attention(*(x[n][..., :4].contiguous() for n in ("q", "k", "v")), x["po"], x["so"])


# ------------------------------------------------------------------ selection
# A total's error: the exponentials (2^-21 relative each), their sums in fp32 within a thread (at
# most 64 terms, 2^-18) -- the log of a sum that near 1 + 2^-17 -- so totals nearer than 2^-16
# may change places; the score is the total rounded to fp32.
TOL = 2.0 ** -16


def select_reference(x, cum, k, finished=None, allowed=None, pad=0):
    """Per request the (total, beam, token) triples in order, in 64 bits."""
    R, W = cum.shape
    V = x.shape[-1]
    x, cum = x.double().view(R, W, V), cum.double()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    res = []
    for r in range(R):
        tot = []
        for b in range(W):
            if not torch.isfinite(cum[r, b]):
                continue
            if finished is not None and finished[r, b]:
                tot.append((float(cum[r, b]), b, 0.0, pad))
                continue
            row = x[r, b]
            m = row.max()
            if m == -math.inf:
                continue
            d = torch.where(row == m, torch.zeros_like(row), row - m)
            lp = d - torch.log(torch.exp(d).sum())
            if allowed is not None:
                lp = torch.where(allowed[r * W + b], lp, torch.full_like(lp, -math.inf))
            n = min(k, V)
            kth = torch.topk(lp, n).values[-1]
            for v in torch.nonzero((lp >= kth) & (lp > -math.inf)).view(-1).tolist():
                tot.append((float(cum[r, b] + lp[v]), b, float(row[v]), v))
        tot.sort(key=lambda c: (-c[0], c[1], -c[2], c[3]))
        res.append(tot)
    return res


def check_select(got, ref, k):
    par, tok, sc = (t.cpu().numpy() for t in got)
    for r, want in enumerate(ref):
        m = min(k, len(want))
        assert (par[r, m:] == -1).all() and (tok[r, m:] == -1).all() and np.isneginf(sc[r, m:]).all()
        total = {(b, v): t for t, b, _, v in want}
        mine = [(int(par[r, j]), int(tok[r, j])) for j in range(m)]
        assert len(set(mine)) == m
        for j in range(m):
            t = want[j][0]
            assert abs(float(sc[r, j]) - t) <= TOL + 2.0 ** -23 * abs(t), (r, j)
            near = [i for i in (j - 1, j + 1) if 0 <= i < len(want) and abs(want[i][0] - t) <= TOL and want[i][1] != want[j][1]]
            if not near:
                assert mine[j] == (want[j][1], want[j][3]), (r, j, mine[j], want[j])
            else:
                assert abs(total[mine[j]] - t) <= TOL


def bits(allowed):
    """bool [rows, V] -> int32 words"""
    rows, V = allowed.shape
    w = -(-V // 32)
    a = np.zeros((rows, w * 32), np.uint8)
    a[:, :V] = allowed.numpy()
    return torch.from_numpy(np.packbits(a, axis=1, bitorder="little").view(np.int32).copy())


SELECT = [(1, 1, 1, 1), (1, 1, 1, 5), (2, 4, 7, 4), (1, 4, 256, 4), (3, 5, 1000, 10), (2, 3, 8192, 256), (2, 8, 8193, 16),
          (1, 2, 16384, 33), (2, 2, 16391, 8), (1, 256, 100, 256), (5, 7, 50257, 20), (1, 16, 131072, 32), (2, 33, 3, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,W,V,k", SELECT)
def test_select(api, R, W, V, k, dtype):
    g = torch.Generator().manual_seed(V + k)
    x = (torch.randn(R * W, V, generator=g) * 2.5).to(DT[dtype])
    cum = -5 * torch.rand(R, W, generator=g)
    got = api.beam_select(x.cuda(), cum.cuda(), k)
    ok(api)
    check_select(got, select_reference(x, cum, k), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [50, 9000, 20001])
def test_select_finished_dead_masked(api, V, dtype):
    """Finished beams (one with NaN logits), dead beams of each kind, a trie that leaves one beam
    nothing and another a single token, rows of a wider buffer at odd addresses."""
    R, W, k = 3, 6, 12
    g = torch.Generator().manual_seed(V)
    wide = torch.randn(R * W, V + 13, generator=g).to(DT[dtype])
    x = wide[:, 5:5 + V]
    cum = -3 * torch.rand(R, W, generator=g)
    cum[0, 1], cum[1, 0], cum[2, 5] = -math.inf, math.nan, math.inf
    fin = torch.zeros(R, W, dtype=torch.bool)
    fin[0, 2] = fin[1, 4] = fin[0, 1] = True
    x[2] = math.nan
    al = torch.rand(R * W, V, generator=g) < 0.3
    al[3] = False
    al[4] = False
    al[4, V - 1] = True
    words = bits(al)
    pad_words = torch.full((R * W, words.shape[1] + 2), -1, dtype=torch.int32)
    pad_words[:, :words.shape[1]] = words
    got = api.beam_select(wide.cuda()[:, 5:5 + V], cum.cuda(), k, finished=fin.cuda(), allowed=pad_words.cuda(), pad_token=V + 3)
    ok(api)
    check_select(got, select_reference(x, cum, k, fin, al, V + 3), k)
    got = api.beam_select(wide.cuda()[:, 5:5 + V], cum.cuda(), k, finished=fin.to(torch.uint8).cuda())
    ok(api)
    check_select(got, select_reference(x, cum, k, fin), k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,k", [(10, 4), (300, 256), (8192, 200), (40000, 64), (40000, 256), (20001, 256)])
def test_select_ties(api, V, k, dtype):
    """Equal logits everywhere (the lowest tokens of the lowest beam win), beams that are copies
    of one another (equal totals: the lower beam), few distinct values, rising and falling rows."""
    x = torch.full((4, V), 1.5).to(DT[dtype])
    cum = torch.zeros(1, 4)
    got = api.beam_select(x.cuda(), cum.cuda(), k)
    ok(api)
    m = min(k, 4 * V)
    assert got[0][0, :m].tolist() == [j // V for j in range(m)] and got[1][0, :m].tolist() == [j % V for j in range(m)]
    g = torch.Generator().manual_seed(V)
    row = torch.randn(V, generator=g)
    x = row.expand(5, V).contiguous().to(DT[dtype])
    got = api.beam_select(x.cuda(), torch.full((1, 5), -2.0).cuda(), k)
    ok(api)
    p, t = got[0][0].tolist(), got[1][0].tolist()
    val = x[0].double()
    want = sorted(((-float(val[v]), b, v) for b in range(5) for v in torch.topk(val, min(k, V)).indices.tolist()))[:k]
    # copies: sorted by value, then beam, then token; equal values within one beam by token
    seq = [(-float(val[tt]), pp, tt) for pp, tt in zip(p, t)]
    assert seq == sorted(seq) and [s[:2] for s in seq] == [w[:2] for w in want]
    for gen in (torch.randint(0, 3, (4, V), generator=g).float(), torch.linspace(-4, 4, V).expand(4, V).contiguous(),
                torch.linspace(4, -4, V).expand(4, V).contiguous()):
        y = gen.to(DT[dtype])
        c = torch.tensor([[-1.0, -0.5, -2.0, -0.25]])
        got = api.beam_select(y.cuda(), c.cuda(), k)
        ok(api)
        check_select(got, select_reference(y, c, k), k)


def test_select_infinite_and_nan_logits(api):
    x = torch.randn(6, 500, generator=torch.Generator().manual_seed(3))
    x[0] = -math.inf                                    # offers nothing
    x[1, :] = math.nan
    x[1, 7] = 0.5                                       # one token with all of the probability
    x[2, [5, 9]] = math.inf                             # two tokens share it
    x[3, ::2] = -math.inf
    x[4] = -3e38
    cum = torch.tensor([[-0.1, -0.2, -0.3, -1.0, -2.0, -3.0]])
    for dtype in (torch.float32, torch.bfloat16):
        y = x.to(dtype)
        got = api.beam_select(y.cuda(), cum.cuda(), 20)
        ok(api)
        check_select(got, select_reference(y, cum, 20), 20)
        assert (got[0] == 0).sum() == 0
    got = api.beam_select(x[:1].cuda(), cum[:, :1].cuda(), 3)
    ok(api)
    assert got[0].tolist() == [[-1] * 3] and torch.isneginf(got[2]).all()


def test_select_buffers_streams_and_3d(api):
    R, W, V, k = 4, 3, 30000, 6
    x = torch.randn(R, W, V, generator=torch.Generator().manual_seed(1))
    cum = -torch.rand(R, W)
    first = api.beam_select(x.cuda(), cum.cuda(), k)
    ok(api)
    side = torch.cuda.Stream()
    d, c = x.cuda(), cum.cuda()
    side.wait_stream(torch.cuda.current_stream())
    bufs = [torch.full((R + 1, k), 9, dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
    side.wait_stream(torch.cuda.current_stream())
    api.beam_select(d, c, k, parent=bufs[0][:R], token=bufs[1][:R], score=bufs[2][:R], stream=side)
    side.synchronize()
    for b, f in zip(bufs, first):
        assert torch.equal(b[:R], f) and bool((b[R] == 9).all())
    with pytest.raises(ValueError):
        api.beam_select(d, c, k, parent=bufs[0])
    with pytest.raises(ValueError):
        api.beam_select(d, c, k, workspace=torch.empty(8, device="cuda"))
    with pytest.raises(api.TrError):
        api.beam_select(d, c, 0)


# ------------------------------------------------------------------ reordering
@pytest.mark.parametrize("shape,dtype", [((3, 2, 16), torch.bfloat16), ((1,), torch.uint8), ((5, 3), torch.int32),
                                         ((7,), torch.float16), ((48, 8, 128), torch.bfloat16), ((1000,), torch.float64)], ids=str)
@pytest.mark.parametrize("R,W_in,W_out", [(1, 1, 1), (3, 4, 4), (2, 5, 8), (4, 16, 3), (1, 256, 256), (2, 33, 33)])
def test_reorder(api, R, W_in, W_out, shape, dtype):
    g = torch.Generator().manual_seed(R * W_in + W_out)

    def rnd(n):
        return (torch.randint(0, 250, (n, *shape), generator=g)).to(dtype)
    src = [rnd(R * W_in) for _ in range(3)]
    dst = [rnd(R * W_out) for _ in range(3)]
    par = torch.randint(-1, W_in, (R, W_out), generator=g).to(torch.int32)
    rows = (par + W_in * torch.arange(R)[:, None]).view(-1)
    keep = (par < 0).view(-1)
    want = []
    for s, d in zip(src, dst):
        w = s[rows.clamp(min=0)].clone()
        w[keep] = d[keep]
        want.append(w)
    got = api.beam_reorder([s.cuda() for s in src], par.cuda(), outs=[d.cuda() for d in dst])
    ok(api)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(got, want))
    if W_in == W_out:
        inplace = [s.cuda() for s in src]
        got = api.beam_reorder(inplace, par.cuda())
        ok(api)
        for a, s in zip(got, src):
            w = s[rows.clamp(min=0)].clone()
            w[keep] = s[keep]
            assert torch.equal(a.cpu(), w)


def test_reorder_partial_rows_joint_cache_and_many_states(api):
    """The filled part of caches moves and the rest stays; K and V of one joint buffer are two
    states; over 64 states go in several launches; cycles and copies in place."""
    R, W, S = 2, 6, 10
    par = torch.tensor([[1, 2, 0, 0, 5, 4], [5, 4, 3, 2, 1, 0]], dtype=torch.int32)
    rows = (par + W * torch.arange(R)[:, None]).view(-1)
    joint = torch.arange(R * W * 2 * S * 8, dtype=torch.float32).view(R * W, 2, S, 8)
    d = joint.cuda()
    api.beam_reorder([d[:, 0, :7], d[:, 1, :7]], par.cuda())
    ok(api)
    want = joint.clone()
    want[:, :, :7] = joint[rows][:, :, :7]
    assert torch.equal(d.cpu(), want)
    many = [torch.randn(R * W, 5) for _ in range(130)]
    got = api.beam_reorder([m.cuda() for m in many], par.cuda())
    ok(api)
    assert all(torch.equal(a.cpu(), m[rows]) for a, m in zip(got, many))


def test_reorder_bad_parent_leaves_the_row_and_is_reported(api):
    from transformer_candidate_scoring_b200 import _lib as L
    x = torch.arange(24, dtype=torch.float32).view(4, 6).cuda()
    api.beam_reorder([x], torch.tensor([[1, 7, 4, 3]], dtype=torch.int32).cuda())
    torch.cuda.synchronize()
    assert api.sync_status() == L.TR_ERR_KEY_RANGE
    w = torch.arange(24, dtype=torch.float32).view(4, 6)
    w[0] = w[1].clone()
    assert torch.equal(x.cpu(), w)
    buf = torch.zeros(5, 6, device="cuda")
    with pytest.raises(api.TrError):                       # shifted by one row: neither in place nor apart
        api.beam_reorder([buf[:4]], torch.zeros(1, 4, dtype=torch.int32).cuda(), outs=[buf[1:]])


# ------------------------------------------------------------------ together
class Decoder:
    """A one-layer decoder over a shared prefix: token embedding -> attention -> logits."""

    def __init__(self, api, R, W, P, V, steps, dtype, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.api, self.R, self.W, self.V, self.H, self.d = api, R, W, V, 4, 64
        self.n, E = R * W, self.H * self.d
        dt = DT[dtype]

        def rnd(*s, scale=1.0):
            return (torch.randn(*s, generator=g) * scale).to(dt).cuda()
        self.emb, self.wq, self.wk, self.wv, self.wo = rnd(V, E), rnd(E, E, scale=0.1), rnd(E, E, scale=0.1), rnd(E, E, scale=0.1), rnd(E, V, scale=0.2)
        self.pk, self.pv = rnd(R * P, self.H, self.d), rnd(R * P, self.H, self.d)
        self.po, self.so = [P * r for r in range(R + 1)], [W * r for r in range(R + 1)]
        self.sk = torch.zeros(self.n, steps, self.H, self.d, dtype=dt, device="cuda")
        self.sv = torch.zeros_like(self.sk)
        self.len = torch.zeros(self.n, dtype=torch.int32, device="cuda")
        self.cum = torch.full((R, W), -math.inf, device="cuda")
        self.cum[:, 0] = 0.0                               # one live beam per request at first
        self.tok = torch.zeros(self.n, dtype=torch.int64, device="cuda")
        self.hist = torch.zeros(self.n, steps, dtype=torch.int64, device="cuda")

    def append(self):
        x = self.emb[self.tok]
        at = self.len.long()[:, None, None, None].expand(-1, 1, self.H, self.d)
        self.sk.scatter_(1, at, (x @ self.wk).view(self.n, 1, self.H, self.d))
        self.sv.scatter_(1, at, (x @ self.wv).view(self.n, 1, self.H, self.d))
        self.len += 1
        return (x @ self.wq).view(self.n, self.H, self.d)

    def step(self):
        q = self.append()
        o, _ = self.api.prefix_attention(q, self.pk, self.pv, self.po, self.so, self.sk, self.sv, self.len)
        logits = o.view(self.n, -1) @ self.wo
        par, tok, score = self.api.beam_select(logits, self.cum, self.W)
        self.api.beam_reorder([self.sk, self.sv, self.hist, self.len], par)
        self.cum.copy_(score)
        self.tok.copy_(tok.view(-1).clamp(min=0))
        self.hist.scatter_(1, (self.len.long() - 1)[:, None], self.tok[:, None])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decode_loop_matches_full_recomputation(api, dtype):
    """Five decode steps; then every surviving beam's score, recomputed in 64 bits from its token
    history alone (each token attending to the prefix and to the tokens before it), agrees."""
    R, W, P, V, steps = 3, 5, 150, 97, 5
    m = Decoder(api, R, W, P, V, steps, dtype)
    for _ in range(steps):
        m.step()
    ok(api)
    f = {k: getattr(m, k).double().cpu() for k in ("emb", "wq", "wk", "wv", "wo", "pk", "pv")}
    hist, cum = m.hist.cpu(), m.cum.cpu()
    assert torch.isfinite(cum).all()
    for i in range(R * W):
        toks = [0] + hist[i].tolist()
        r, total = i // W, 0.0
        ks, vs = [], []
        for t in range(steps):
            x = f["emb"][toks[t]]
            ks.append((x @ f["wk"]).view(m.H, m.d))
            vs.append((x @ f["wv"]).view(m.H, m.d))
            k = torch.cat([f["pk"][r * P:(r + 1) * P], torch.stack(ks)])
            v = torch.cat([f["pv"][r * P:(r + 1) * P], torch.stack(vs)])
            a = torch.einsum("hd,jhd->hj", (x @ f["wq"]).view(m.H, m.d), k) / 8.0
            o = torch.einsum("hj,jhd->hd", torch.softmax(a, -1), v).reshape(-1)
            total += float(torch.log_softmax(o @ f["wo"], -1)[toks[t + 1]])
        # bf16: the projections, attention output and logits are each rounded (2^-8 of values of
        # a few units) in every step; fp32: products over 256 terms
        assert abs(float(cum[i // W, i % W]) - total) < steps * (0.1 if dtype == "bf16" else 1e-3)
    # beams of a request are distinct histories, best first
    for r in range(R):
        assert len({tuple(hist[r * W + b].tolist()) for b in range(W)}) == W
        assert (cum[r, :-1] >= cum[r, 1:]).all()


def test_decode_step_captured_and_replayed(api):
    """A captured step, replayed, gives what eager steps give, with the workspaces in the graph's
    own pool; two captured graphs replayed on two streams at once do not disturb each other."""
    def make(seed):
        return Decoder(api, 4, 8, 700, 3000, 6, "bf16", seed)
    want = []
    for seed in (1, 2):
        m = make(seed)
        for _ in range(4):
            m.step()
        want.append((m.hist.clone(), m.cum.clone(), m.sk.clone()))
    ok(api)
    models, graphs, streams = [make(1), make(2)], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for m, s in zip(models, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m.step()                                    # warm-up on the stream, also the first step
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            m.step()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    ok(api)
    for m, w in zip(models, want):
        assert torch.equal(m.hist, w[0]) and torch.equal(m.cum, w[1]) and torch.equal(m.sk, w[2])
