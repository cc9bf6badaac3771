"""tr_prefix_attention in each of the forms that its plan chooses between, told apart by the workspace it asks for:
    merge    a prefix kernel (tensor cores in bf16, tiled in fp32) leaves partial results, which the kernel of the own
             keys merges: a workspace
    direct   the tensor-core kernel writes the results itself (at most one own key): none, but the same call with
             room for two own keys has one (over a few dozen keys that call may have none either: not told from the next)
    own      the kernel of the own keys reads the prefixes as well: none
Tolerances are those of test_gpu_decode.py, from the same arithmetic; the reference runs in 64 bits on the GPU.
"""
import math

import pytest
import torch

from test_gpu_decode import DT, EPS, api, attn_inputs, dev, ok  # noqa: F401  (api: a fixture)

pytestmark = pytest.mark.gpu


def formula(x, scale, causal):
    """(out, lse, tolerance of out, tolerance of lse) of inputs on the GPU, in 64 bits, a request at a time."""
    n, L_t, H, d = x["q"].shape
    G = H // x["k"].shape[1]
    opts = {"dtype": torch.float64, "device": "cuda"}
    out, lse = torch.zeros(n, L_t, H, d, **opts), torch.full((n, L_t, H), -math.inf, **opts)
    tol, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for r in range(len(x["so"]) - 1):
        s, p = slice(x["so"][r], x["so"][r + 1]), slice(x["po"][r], x["po"][r + 1])
        if s.start == s.stop:
            continue
        q = x["q"][s].double()
        k, v = (x[z][p].double().repeat_interleave(G, 1) for z in ("k", "v"))               # [P, H, d]
        a, A = (torch.einsum("nthd,jhd->nthj", f(q), f(k)) for f in (lambda z: z, torch.abs))
        P = a.shape[-1]
        if x["ks"] is not None:
            S = x["ks"].shape[1]
            ks, vs = (x[z][s].double().repeat_interleave(G, 2) for z in ("ks", "vs"))       # [n, S, H, d]
            end = x["sl"][s].long().clamp(0, S)[:, None].expand(-1, L_t)
            if causal:
                end = (end - (L_t - 1 - torch.arange(L_t, device="cuda"))).clamp(min=0)
            seen = torch.arange(S, device="cuda") < end[:, :, None]                         # [n, L_t, S]
            ks, vs = (z.masked_fill(~seen.any(1)[:, :, None, None], 0.0) for z in (ks, vs))
            b, B = (torch.einsum("nthd,njhd->nthj", f(q), f(ks)) for f in (lambda z: z, torch.abs))
            a = torch.cat([a, b.masked_fill(~seen[:, :, None], -math.inf)], -1)
            A = torch.cat([A, B.masked_fill(~seen[:, :, None], 0.0)], -1)
        if a.shape[-1] == 0:
            continue
        z = torch.logsumexp(a * scale, -1)
        w = torch.where(z[..., None] == -math.inf, 0.0, torch.exp(a * scale - z[..., None]))
        o, pv = (torch.einsum("nthj,jhd->nthd", w[..., :P], f(v)) for f in (lambda z: z, torch.abs))
        if x["ks"] is not None:
            o += torch.einsum("nthj,njhd->nthd", w[..., P:], vs)
            pv += torch.einsum("nthj,njhd->nthd", w[..., P:], vs.abs())
        rel = 2 * (d + 3) * EPS * A.amax(-1) * scale + 2.0 ** -20 + a.shape[-1] * EPS
        out[s], lse[s], tol[s], tol_l[s] = o, z, rel[..., None] * pv, rel + EPS * z.abs().nan_to_num(posinf=0.0)
        if x["q"].dtype == torch.bfloat16:
            tol[s] += 2.0 ** -8 * pv + 2.0 ** -8 * o.abs() + 2.0 ** -133
    return out, lse, tol, tol_l


def agrees(got, want):
    out, lse, tol, tol_l = want
    o, z = (t.double().view(r.shape) for t, r in zip(got, (out, lse)))
    empty = lse == -math.inf
    assert torch.equal(z == -math.inf, empty) and bool((o[empty] == 0).all())
    assert bool(((o - out).abs() <= tol).all()), ((o - out).abs() / tol.clamp(min=1e-300)).max().item()
    assert bool(((z - lse).abs() <= tol_l)[~empty].all())


def form_of(api, x, causal):
    """Which form the call takes, from the workspace that its plan asks for."""
    def need(cap):
        q, kp = x["q"], x["k"]
        n, L_t, H, d = q.shape
        K = kp.shape[1]
        kv = K * d
        L = api.L
        desc = L.AttnDesc(H, K, d, L_t, int(causal), cap, d ** -0.5, api.dtype_code(q.dtype), H * d, kv, d, max(cap, 1) * kv, kv, d)
        R = len(x["so"]) - 1
        arr = [(api.C.c_int64 * (R + 1))(*z) for z in (x["so"], x["po"])]
        got = L.load().tr_prefix_attention_workspace(api.C.byref(desc), *arr, R)
        assert got != api.C.c_size_t(-1).value
        return got
    S = 0 if x["ks"] is None else x["ks"].shape[1]
    return "merge" if need(S) else "direct" if S <= 1 and x["q"].dtype == torch.bfloat16 and need(2) else "own"


def call(api, x, causal=False, **kw):
    return api.prefix_attention(x["q"], x["k"], x["v"], x["po"], x["so"], x["ks"], x["vs"], x["sl"], causal=causal, **kw)


# form, counts, prefix, H, H_kv, d, S, L_t, causal
LONG, MANY, FEW = ([150, 40], [1037, 1301]), ([900, 700], [1037, 1301]), ([3, 5, 2], [3001, 5005, 130])
RUNS = ([1 + i % 2 for i in range(18)],
        [5003, 1, 700, 2049, 4100, 128, 127, 5990, 3333, 129, 64, 2500, 1111, 5500, 900, 0, 4999, 2222])
BF16 = [
    ("merge", *LONG, 4, 2, 64, 3, 1, False), ("merge", *LONG, 4, 2, 128, 40, 1, False), ("merge", *LONG, 4, 2, 72, 0, 1, False),
    ("merge", *LONG, 4, 2, 8, 9, 1, False), ("merge", *LONG, 4, 2, 104, 1, 1, False), ("merge", *LONG, 4, 1, 16, 7, 1, False),
    ("merge", [60, 90], [1037, 1301], 6, 2, 64, 40, 5, True), ("merge", [60, 90], [1037, 1301], 6, 2, 104, 5, 5, True),
    ("merge", [20, 9], [1037, 1301], 4, 2, 64, 20, 16, True), ("merge", [20, 9], [1037, 1301], 4, 2, 128, 3, 16, True),
    ("merge", *FEW, 4, 2, 96, 3, 1, False), ("merge", *FEW, 4, 2, 128, 17, 1, False), ("merge", *FEW, 8, 8, 40, 0, 1, False),
    ("direct", *MANY, 16, 8, 64, 1, 1, False), ("direct", *MANY, 16, 8, 128, 0, 1, False), ("direct", *MANY, 16, 8, 8, 1, 1, False),
    ("direct", *MANY, 16, 8, 72, 1, 1, False), ("direct", [450, 350], [1037, 1301], 16, 8, 40, 1, 2, True),
    ("direct", [100] * 30, [133] * 30, 8, 8, 128, 1, 1, False),                   # tiles of one request each
    ("direct", [2400], [130], 16, 16, 16, 1, 1, False), ("direct", [2300, 7], [129, 0], 20, 20, 128, 0, 1, False),  # halved units
    ("merge", *RUNS, 8, 8, 64, 3, 1, False), ("merge", *RUNS, 16, 8, 128, 9, 1, False),                             # equal runs of keys
    ("own", [5, 3], [37, 141], 4, 2, 128, 40, 1, False), ("own", [5, 3], [37, 141], 4, 2, 8, 1, 1, False),
    ("own", [5, 3], [37, 141], 6, 2, 64, 12, 5, True), ("own", [2, 3], [9, 60], 4, 2, 104, 5, 16, True),
]
F32 = [
    ("merge", *LONG, 4, 2, 64, 3, 1, False), ("merge", *LONG, 4, 2, 128, 40, 1, False), ("merge", *LONG, 4, 2, 72, 1, 1, False),
    ("merge", *LONG, 4, 2, 8, 0, 1, False), ("merge", [60, 90], [1037, 1301], 6, 2, 96, 40, 5, True),
    ("merge", *FEW, 4, 2, 64, 3, 1, False), ("merge", *FEW, 4, 2, 96, 3, 1, False), ("merge", *FEW, 4, 2, 128, 3, 1, False),
    ("merge", [2, 1], [1037, 1301], 4, 2, 128, 20, 8, True),
    ("own", [5, 3], [37, 141], 4, 2, 128, 40, 1, False), ("own", [5, 3], [37, 141], 6, 2, 64, 12, 5, True),
]
CASES = [("bf16", *c) for c in BF16] + [("f32", *c) for c in F32]


def _id(c):
    return f"{c[0]}-{c[1]}-{c[2][0]}x{len(c[2])}-{c[3][0]}-{c[4]}x{c[5]}x{c[6]}-s{c[7]}-t{c[8]}{'c' if c[9] else ''}"


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("case", CASES, ids=_id)
def test_form_ignores_what_no_row_sees(api, case, bad):
    """Each request's prefix has, before and behind it, tokens of a request without sequences that hold NaN or an
    infinity, and so has each suffix behind its length."""
    dtype, form, counts, prefix, H, H_kv, d, S, L_t, causal = case
    gap = 131
    cc = [z for c in counts for z in (0, c)] + [0]
    pp = [z for p in prefix for z in (gap, p)] + [gap]
    x = dev(attn_inputs(sum(prefix) + d + S, cc, pp, H, H_kv, d, S, L_t, dtype))
    want = formula(x, d ** -0.5, causal)
    y = dict(x)
    hidden = torch.ones(x["k"].shape[0], dtype=torch.bool, device="cuda")
    for r, c in enumerate(cc):
        if c:
            hidden[x["po"][r]:x["po"][r + 1]] = False
    for z in ("k", "v"):
        y[z] = x[z].masked_fill(hidden[:, None, None], bad)
    if S:
        behind = torch.arange(S, device="cuda") >= x["sl"][:, None]
        for z in ("ks", "vs"):
            y[z] = x[z].masked_fill(behind[:, :, None, None], bad)
    assert form_of(api, y, causal) == form
    launches = api.kernel_launches()
    got = call(api, y, causal)
    assert api.kernel_launches() - launches == (2 if form == "merge" else 1)
    ok(api)
    agrees(got, want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("case", [c for c in CASES if c[9] and c[7] > 1], ids=_id)
def test_form_causal_rows_ignore_later_values(api, case, bad):
    """The values of a sequence's last two tokens hold NaN or infinities: the query tokens before them
    get what the formula gives without, the others what it gives with them."""
    dtype, form, counts, prefix, H, H_kv, d, S, L_t, causal = case
    n = sum(counts)
    x = attn_inputs(d + S, counts, prefix, H, H_kv, d, S, L_t, dtype, lens=[S, max(2, S // 2), 2])
    x = dev(x)
    y = dict(x, vs=x["vs"].clone())
    for s in range(n):
        y["vs"][s, int(x["sl"][s]) - 2:int(x["sl"][s])] = bad
    assert form_of(api, y, causal) == form
    got, want = call(api, y, causal), formula(x, d ** -0.5, causal)
    ok(api)
    agrees((got[0][:, :L_t - 2], got[1][:, :L_t - 2]), [z[:, :L_t - 2] for z in want])
    late = got[0][:, L_t - 2:].float()
    assert bool((torch.isnan(late) if bad != bad else late == bad).all())
    assert bool(((got[1].double() - want[1]).abs() <= want[3])[want[1] > -math.inf].all())   # scores do not read values


STRIDED = [("bf16", "merge", *LONG, 4, 2, 64, 6, 1, False), ("bf16", "merge", *LONG, 4, 2, 128, 12, 1, False),
           ("bf16", "direct", *MANY, 16, 8, 64, 1, 1, False), ("bf16", "direct", *MANY, 16, 8, 96, 0, 1, False),
           ("bf16", "merge", *FEW, 4, 2, 96, 3, 1, False), ("f32", "merge", *LONG, 4, 2, 64, 6, 1, False),
           ("f32", "merge", *FEW, 4, 2, 128, 3, 1, False), ("bf16", "merge", [60, 90], [1037, 1301], 6, 2, 64, 40, 5, True)]


@pytest.mark.parametrize("case", STRIDED, ids=_id)
def test_form_strides(api, case):
    """q out of a fused projection, K and V joint in one buffer with heads outermost or tokens outermost, suffix buffers
    with strides of their own, tokens before the first request, another scale; the gaps hold NaN."""
    dtype, form, counts, prefix, H, H_kv, d, S, L_t, causal = case
    x = dev(attn_inputs(d + H, counts, prefix, H, H_kv, d, S, L_t, dtype, lead=11))
    n, T, nan = sum(counts), x["k"].shape[0], float("nan")
    fused = torch.full((n, L_t, (H + 2 * H_kv) * d), nan, dtype=DT[dtype], device="cuda")
    fused[..., :H * d] = x["q"].reshape(n, L_t, H * d)
    y = dict(x, q=fused[..., :H * d].view(n, L_t, H, d))
    if S:
        room = torch.full((n, 2, S + 2, H_kv, d), nan, dtype=DT[dtype], device="cuda")
        room[:, 0, :S], room[:, 1, :S] = x["ks"], x["vs"]
        y["ks"], y["vs"] = room[:, 0, :S], room[:, 1, :S]
    want = formula(x, 0.31, causal)
    for outer in (True, False):
        if outer:
            joint = torch.full((2, H_kv, T + 3, d), nan, dtype=DT[dtype], device="cuda")
            joint[0, :, 11:T], joint[1, :, 11:T] = x["k"][11:].transpose(0, 1), x["v"][11:].transpose(0, 1)
            y["k"], y["v"] = joint[0].transpose(0, 1)[:T], joint[1].transpose(0, 1)[:T]
        else:
            joint = torch.full((T + 3, H_kv, 2, d), nan, dtype=DT[dtype], device="cuda")
            joint[11:T, :, 0], joint[11:T, :, 1] = x["k"][11:], x["v"][11:]
            y["k"], y["v"] = joint[:T, :, 0], joint[:T, :, 1]
        assert form_of(api, x, causal) == form
        got = call(api, y, causal, scale=0.31)
        ok(api)
        agrees(got, want)


# Keys whose offsets from the buffer's start pass 2^32 elements; sequences' own keys and queries too.
@pytest.mark.parametrize("dtype,form,counts,prefix,S", [("bf16", "merge", [3], [5005], 9), ("bf16", "own", [3], [77], 9),
                                                        ("bf16", "own", [3], [77], 3), ("bf16", "direct", [1700], [1300], 1),
                                                        ("f32", "merge", [3], [3001], 3), ("f32", "own", [3], [77], 3)])
def test_form_offsets_beyond_32_bits(api, dtype, form, counts, prefix, S):
    H, H_kv, d = (16, 8, 128) if form == "direct" else (4, 2, 128)
    n, P = sum(counts), sum(prefix)
    x = dev(attn_inputs(P, counts, prefix, H, H_kv, d, S, 1, dtype))
    pairs = 2 * H_kv * d
    lead = (1 << 32) // pairs
    kv = torch.empty(lead + P, 2, H_kv, d, dtype=DT[dtype], device="cuda")
    kv[lead:, 0], kv[lead:, 1] = x["k"], x["v"]
    y = dict(x, k=kv[:, 0], v=kv[:, 1], po=[lead, lead + P])
    # sequences as far apart as the buffer holds them (in another one)
    far = ((1 << 32) + (1 << 20)) // (n - 1) // 64 * 64
    room = torch.empty((n - 1) * far + (1 << 20), dtype=DT[dtype], device="cuda")
    for z, at in (("q", 0), ("ks", 1 << 12), ("vs", 1 << 15)):
        shape = x[z].shape
        inner = [H * d, H * d, d, 1] if z == "q" else [S * H_kv * d, H_kv * d, d, 1]
        y[z] = room[at:].as_strided(shape, [far] + inner[1:])
        y[z].copy_(x[z])
    assert far > (1 << 15) + 16 * H_kv * d
    assert form_of(api, x, False) == form
    got = call(api, y)
    ok(api)
    agrees(got, formula(x, d ** -0.5, False))


# The first request alone and beside others, which take it to another form or cut its keys in other places.  Each result is
# within its tolerance of the formula, so the two are within twice that of one another: twice the fp32 terms and, in
# bf16, 2^-7 sum_j p_j |v_j| for the numerators and 2^-7 |out| for the results.
BESIDE = [("bf16", "own", "merge", 32, 64, [32] * 15, [64] * 15, 8, 8, 64, 4), ("bf16", "own", "merge", 32, 64, [1], [8000], 8, 8, 64, 4),
          ("bf16", "own", "merge", 32, 64, [1], [8000], 8, 8, 128, 20), ("bf16", "merge", "merge", 40, 4001, [40] * 20, [2222] * 20, 8, 4, 128, 9),
          ("bf16", "merge", "direct", 300, 2000, [2000] * 3, [2000] * 3, 16, 8, 64, 1), ("f32", "own", "merge", 32, 64, [1], [8000], 8, 8, 64, 4),
          ("f32", "merge", "merge", 40, 4001, [40] * 20, [2222] * 20, 8, 4, 80, 9)]


@pytest.mark.parametrize("case", BESIDE, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}x{c[4]}-{c[7]}x{c[8]}x{c[9]}")
def test_form_request_alone_and_beside_others(api, case):
    dtype, alone, beside, count, prefix, counts, prefixes, H, H_kv, d, S = case
    x = dev(attn_inputs(3, [count, *counts], [prefix, *prefixes], H, H_kv, d, S, 1, dtype))
    y = {z: x[z][:n] for z, n in (("q", count), ("k", prefix), ("v", prefix), ("ks", count), ("vs", count), ("sl", count))}
    y.update(so=x["so"][:2], po=x["po"][:2])
    assert form_of(api, y, False) == alone and form_of(api, x, False) == beside
    one, all_, again = call(api, y), call(api, x), call(api, x)
    ok(api)
    assert all(torch.equal(a, b) for a, b in zip(all_, again))
    want = formula(y, d ** -0.5, False)
    part = [z[:count] for z in all_]
    agrees(one, want)
    agrees(part, want)
    for a, b, tol in zip(one, part, want[2:]):
        assert bool(((a.double() - b.double()).abs() <= 2 * tol).all())


# Shapes on both sides of the choice between the prefix kernel and the one launch of the own keys' kernel.
CHOICE = [([300] * 16, 16, 8, 128, 23, "bf16", {2: "own", 16: "own", 64: "merge"}), ([4] * 4, 8, 8, 128, 40, "bf16", {2: "own", 128: "own", 4096: "merge"}),
          ([459] * 5, 16, 2, 96, 2, "bf16", {2: "own", 8: "own", 64: "merge"}), ([77] * 24, 32, 8, 128, 0, "f32", {2: "own", 16: "own", 256: "merge"}),
          ([4], 8, 8, 64, 4, "bf16", {2: "own", 200: "own", 4096: "merge"}), ([4096] * 16, 8, 8, 16, 1, "bf16", {128: "direct"})]


@pytest.mark.parametrize("case", CHOICE, ids=lambda c: f"{c[5]}-{c[0][0]}x{len(c[0])}-{c[1]}x{c[2]}x{c[3]}-s{c[4]}")
def test_form_chosen(api, case):
    counts, H, H_kv, d, S, dtype, want = case
    n, so = sum(counts), [sum(counts[:r]) for r in range(len(counts) + 1)]
    for prefix, form in want.items():
        x = {"q": torch.empty(n, 1, H, d, dtype=DT[dtype], device="meta"), "k": torch.empty(1, H_kv, d, dtype=DT[dtype], device="meta"),
             "ks": torch.empty(n, S, H_kv, d, device="meta") if S else None, "so": so, "po": [prefix * r for r in range(len(so))]}
        assert form_of(api, x, False) == form, prefix
