"""Cases and plain forms of the beam-decoding operators: shared-prefix attention, beam selection
and the reordering of beam states.

A decode step of generative recall runs them in this order: every beam of a request attends to
the request's long shared prefix (computed once, stored once) and to the few tokens of its own;
the next tokens are selected over beams and vocabulary; the beams' own states follow their
parents.  ``own`` chooses between the plain forms below and the package's kernels.
"""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
NEG = float("-inf")


# ------------------------------------------------------------------ cases
def _attn(name, R, W, H, Hkv, d, lo, hi, S, Lt=1, dtype="bf16", causal=False, joint=False):
    """R requests of W sequences (ragged: some have fewer), prefixes of lo..hi tokens, suffix
    buffers of S tokens, Lt query tokens per sequence; joint: K and V interleaved in one buffer."""
    return {"name": name, "op": "attention", "R": R, "W": W, "H": H, "Hkv": Hkv, "d": d, "lo": lo, "hi": hi, "S": S,
            "Lt": Lt, "dtype": dtype, "causal": causal, "joint": joint}


def _select(name, R, W, V, k, dtype="bf16", done=0, masked=False):
    """R requests of W beams over V tokens, the best k; every done-th beam finished (0: none);
    masked: a trie allows some of the tokens of each beam."""
    return {"name": name, "op": "select", "R": R, "W": W, "V": V, "k": k, "dtype": dtype, "done": done, "masked": masked}


def _reorder(name, R, W, states, S, Hkv, d, dtype="bf16"):
    """``states`` K or V caches [R*W, S, Hkv, d] that follow the surviving beams."""
    return {"name": name, "op": "reorder", "R": R, "W": W, "states": states, "S": S, "Hkv": Hkv, "d": d, "dtype": dtype}


def listed():
    return [
        # one user, four beams, a short history: latency alone
        _attn("attn-1x4-p200", 1, 4, 8, 8, 64, 200, 200, 4),
        # candidates of 16 packed requests, 8 heads of 16, 16..128 user tokens, one own token each
        _attn("attn-16x4096-p128-d16", 16, 4096, 8, 8, 16, 16, 128, 1),
        # beams of 16 users over long ragged histories, grouped heads, a growing suffix
        _attn("attn-16x32-p8192-d128", 16, 32, 32, 8, 128, 2048, 8192, 64),
        # one user with a very long history: the read of its K/V bounds the step
        _attn("attn-1x16-p131072-d128", 1, 16, 16, 4, 128, 131072, 131072, 32, joint=True),
        # thousands of candidates against long histories: the products bound the step
        _attn("attn-2x4096-p4096-d128", 2, 4096, 16, 4, 128, 4096, 4096, 1),
        # fp32, odd head width, several query tokens per sequence, causal among themselves, ragged
        _attn("attn-3x37-p1501-d80-f32", 3, 37, 6, 2, 80, 0, 1501, 9, Lt=3, dtype="f32", causal=True),
        # one user, four beams, one codebook of semantic ids: latency alone
        _select("select-1x4-v256", 1, 4, 256, 4, dtype="f32"),
        # codebook-sized vocabularies with a trie, many users
        _select("select-64x32-v8192-trie", 64, 32, 8192, 32, masked=True),
        # a language model's vocabulary
        _select("select-64x16-v131072", 64, 16, 131072, 32),
        # fp32, odd sizes, every third beam finished
        _select("select-7x50-v50257-f32", 7, 50, 50257, 100, dtype="f32", done=3),
        # the states of one user's four beams: latency alone
        _reorder("reorder-1x4", 1, 4, 10, 4, 8, 16),
        # K and V of eight layers, 32 users
        _reorder("reorder-32x32", 32, 32, 16, 48, 8, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: the three operators with sizes spread over the listed ranges, none costlier
    than the largest listed case of its operator."""
    op = rng.choice(["attention", "attention", "attention", "select", "select", "reorder"])
    while True:
        if op == "attention":
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 2, 3, 4, 5, 8])
            R, W = _log(rng, 1, 64), _log(rng, 1, 4096)
            hi = _log(rng, 1, 131072)
            lo = rng.choice([0, hi // 4, hi])
            c = _attn("", R, W, Hkv * G, Hkv, rng.choice([16, 32, 64, 64, 80, 96, 128, 128, 8 * rng.randint(1, 16)]), lo, hi,
                      rng.choice([0, 1, _log(rng, 1, 128)]), Lt=rng.choice([1, 1, 1, rng.randint(2, 8)]), dtype=dtype,
                      causal=rng.choice([False, True]), joint=rng.choice([False, True]))
            fl, by = (32e9, 2e9) if dtype == "f32" else (275e9, 2e9)
            w = work(c)
            rows = R * W * c["Lt"] * c["H"]
            if w["flops"] > fl or w["bytes"] > by or rows * max(hi, 1) > 5.4e8 or rows * c["S"] * c["d"] > 1e9 or R * hi * Hkv * c["d"] > 1e9:
                continue
        elif op == "select":
            W = _log(rng, 1, 256)
            c = _select("", _log(rng, 1, 64), W, _log(rng, 2, 160000), rng.choice([W, 2 * W, rng.randint(1, 256)]),
                        dtype=rng.choice(["bf16", "f32"]), done=rng.choice([0, 0, 2, 3, 5]), masked=rng.choice([False, False, True]))
            if c["R"] * W * c["V"] > (1 << 27) or c["k"] > 256:
                continue
        else:
            c = _reorder("", _log(rng, 1, 64), _log(rng, 1, 256), rng.randint(1, 24), _log(rng, 1, 128), rng.choice([1, 2, 4, 8]),
                         8 * rng.randint(1, 16), dtype=rng.choice(["bf16", "f32"]))
            if work(c)["bytes"] > 3.3e9:
                continue
        del c["name"]
        return c


def _prefix_lens(c):
    """Deterministic ragged prefix lengths in lo..hi; request 0 has hi tokens, request 1 lo."""
    R, lo, hi = c["R"], c["lo"], c["hi"]
    return [hi if r == 0 else lo if r == 1 else lo + int((hi - lo) * ((r * 0.6180339887) % 1.0)) for r in range(R)]


def _seq_counts(c):
    """Sequences of each request: W, the last requests of a ragged batch a few less."""
    return [max(1, c["W"] - (r % 3)) if c["lo"] != c["hi"] else c["W"] for r in range(c["R"])]


def _suffix_lens(c):
    """Filled tokens of each sequence's suffix buffer: full, or up to three short."""
    n = sum(_seq_counts(c))
    return [max(0, c["S"] - (s % 4 if c["S"] > 4 else 0)) for s in range(n)]


def _seen(c, length):
    """Suffix tokens that the query tokens of a sequence see, summed over its query tokens."""
    return sum(max(0, length - (c["Lt"] - 1 - t)) if c["causal"] else length for t in range(c["Lt"]))


def work(case):
    c = case
    if c["op"] == "attention":
        e = 2 if c["dtype"] == "bf16" else 4
        counts, pre, suf = _seq_counts(c), _prefix_lens(c), _suffix_lens(c)
        n = sum(counts)
        rows = n * c["Lt"] * c["H"]
        pairs = sum(a * b for a, b in zip(counts, pre)) * c["Lt"] + sum(_seen(c, x) for x in suf)
        return {"bytes": rows * (2 * c["d"] * e + 4) + (sum(pre) + sum(suf)) * 2 * c["Hkv"] * c["d"] * e,
                "flops": 4 * c["H"] * c["d"] * pairs}
    if c["op"] == "select":
        rows = c["R"] * c["W"]
        live = rows - (len(range(0, rows, c["done"])) if c["done"] else 0)
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": live * c["V"] * (e + (0.125 if c["masked"] else 0)) + rows * 5 + c["R"] * c["k"] * 12,
                "flops": 4 * live * c["V"]}
    row = c["S"] * c["Hkv"] * c["d"] * (2 if c["dtype"] == "bf16" else 4)
    return {"bytes": 2 * c["states"] * c["R"] * c["W"] * row + c["R"] * c["W"] * 4, "flops": 0}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _offsets(counts):
    off = [0]
    for x in counts:
        off.append(off[-1] + x)
    return off


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "attention":
        dt, d, Hkv, S = DT[c["dtype"]], c["d"], c["Hkv"], c["S"]
        st["seq_offsets"], st["prefix_offsets"] = _offsets(_seq_counts(c)), _offsets(_prefix_lens(c))
        n, T = st["seq_offsets"][-1], max(1, st["prefix_offsets"][-1])
        # queries and keys whose scores spread as a trained model's do: a few keys carry most of a row
        st["q"] = _randn(g, n, c["Lt"], c["H"], d, dtype=dt, scale=2.0)
        if c["joint"]:
            kv = _randn(g, T, 2, Hkv, d, dtype=dt)
            st["k"], st["v"] = kv[:, 0], kv[:, 1]
        else:
            st["k"], st["v"] = _randn(g, T, Hkv, d, dtype=dt), _randn(g, T, Hkv, d, dtype=dt)
        st["sk"] = _randn(g, n, S, Hkv, d, dtype=dt) if S else None
        st["sv"] = _randn(g, n, S, Hkv, d, dtype=dt) if S else None
        st["slen"] = torch.tensor(_suffix_lens(c), dtype=torch.int32, device=DEV) if S else None
        st["seq_dev"] = torch.tensor(st["seq_offsets"], device=DEV)
        st["prefix_dev"] = torch.tensor(st["prefix_offsets"], device=DEV)
    elif c["op"] == "select":
        rows, V = c["R"] * c["W"], c["V"]
        x = _randn(g, rows, V, scale=2.0)
        x += 3.0 * torch.rand(rows, V, generator=g, device=DEV).lt(0.01) * _randn(g, rows, V).abs()  # a head of likely tokens
        st["logits"] = x.to(DT[c["dtype"]])
        st["cum"] = -8.0 * torch.rand(c["R"], c["W"], generator=g, device=DEV)
        st["finished"] = None
        if c["done"]:
            st["finished"] = (torch.arange(rows, device=DEV) % c["done"] == 0).view(c["R"], c["W"])
        st["allowed"] = None
        if c["masked"]:  # bit v % 32 of word v / 32: token v continues an item of the trie
            keep = torch.randint(-2**31, 2**31, (rows, -(-V // 32)), generator=g, device=DEV)
            st["allowed"] = (keep & torch.randint(-2**31, 2**31, keep.shape, generator=g, device=DEV)).to(torch.int32)
    else:
        n = c["R"] * c["W"]
        st["states"] = [_randn(g, n, c["S"], c["Hkv"], c["d"], dtype=DT[c["dtype"]]) for _ in range(c["states"])]
        st["outs"] = [torch.empty_like(x) for x in st["states"]]   # the caches of a decoder are held twice
        st["parent"] = torch.randint(0, c["W"], (c["R"], c["W"]), generator=g, device=DEV, dtype=torch.int32)
    return st


# ------------------------------------------------------------------ plain forms
def _plain_attention(s):
    c = s["case"]
    R, Lt, H, Hkv, d = c["R"], c["Lt"], c["H"], c["Hkv"], c["d"]
    G, scale = H // Hkv, 1.0 / math.sqrt(d)
    n = s["q"].shape[0]
    so, po = s["seq_dev"], s["prefix_dev"]
    W, L = max(_seq_counts(c)), max(1, max(_prefix_lens(c)))
    # sequences and prefixes padded to [R, W] and [R, L]
    at = torch.arange(L, device=DEV)
    idx = po[:-1, None] + at
    live = idx < po[1:, None]
    idx = idx.clamp(max=s["k"].shape[0] - 1)
    k, v = (x[idx].float().permute(0, 2, 1, 3) for x in (s["k"], s["v"]))            # [R, Hkv, L, d]
    row = torch.arange(n, device=DEV)
    req = torch.searchsorted(so[1:].contiguous(), row, right=True)
    rel = row - so[req]
    q = s["q"].float().view(n, Lt, Hkv, G, d)
    pad = (so[:-1, None] + torch.arange(W, device=DEV)).clamp(max=n - 1)
    qp = q[pad].permute(0, 3, 1, 2, 4, 5).reshape(R, Hkv, W * Lt * G, d)
    a = (qp @ k.transpose(-1, -2)).mul_(scale)
    a.masked_fill_(~live[:, None, None, :], NEG)
    m1 = a.amax(-1)
    a.sub_(m1.masked_fill(m1 == NEG, 0.0)[..., None]).exp_()
    l1, o1 = a.sum(-1), a @ v
    del a

    def rows_of(x):                                                                  # [R, Hkv, W*Lt*G, *] -> [n, Lt, Hkv, G, *]
        x = x.reshape(R, Hkv, W, Lt, G, -1)
        return x[req, :, rel].permute(0, 2, 1, 3, 4)
    m1, l1, o1 = rows_of(m1[..., None]), rows_of(l1[..., None]), rows_of(o1)
    if s["sk"] is not None:
        S = s["sk"].shape[1]
        ks, vs = (x.float().permute(0, 2, 1, 3) for x in (s["sk"], s["sv"]))         # [n, Hkv, S, d]
        qs = q.permute(0, 2, 1, 3, 4).reshape(n, Hkv, Lt * G, d)
        b = (qs @ ks.transpose(-1, -2)).mul_(scale).view(n, Hkv, Lt, G, S)
        end = s["slen"][:, None].expand(n, Lt)
        if c["causal"]:
            end = end - (Lt - 1 - torch.arange(Lt, device=DEV))
        b.masked_fill_(torch.arange(S, device=DEV) >= end[:, None, :, None, None], NEG)
        m2 = b.amax(-1, keepdim=True)
        b = (b - m2.masked_fill(m2 == NEG, 0.0)).exp()
        l2 = b.sum(-1, keepdim=True)
        o2 = (b.reshape(n, Hkv, Lt * G, S) @ vs).view(n, Hkv, Lt, G, d)
        m2, l2, o2 = (x.permute(0, 2, 1, 3, 4) for x in (m2, l2, o2))
        m = torch.maximum(m1, m2)
        z = m.masked_fill(m == NEG, 0.0)
        f1, f2 = (m1 - z).exp(), (m2 - z).exp()
        m1, l1, o1 = m, l1 * f1 + l2 * f2, o1 * f1 + o2 * f2
    o = torch.where(l1 > 0, o1 / l1, torch.zeros_like(o1))
    return o.reshape(n, Lt, H, d).to(DT[c["dtype"]]), (m1 + l1.log()).reshape(n, Lt, H)


def _plain_select(s):
    c = s["case"]
    R, W, V, k = c["R"], c["W"], c["V"], c["k"]
    x = s["logits"].double()       # 64 bits: the order of two totals that nearly agree is part of the result
    m = x.amax(-1, keepdim=True)
    lse = m + (x - m).exp().sum(-1, keepdim=True).log()
    total = s["cum"].double().view(R * W, 1) + (x - lse)
    if s["allowed"] is not None:
        at = torch.arange(V, device=DEV)
        total.masked_fill_((s["allowed"][:, at // 32] >> (at % 32)) & 1 == 0, NEG)
    if s["finished"] is not None:  # a finished beam stands for itself, with token 0
        f = s["finished"].view(R * W)
        total.masked_fill_(f[:, None], NEG)
        total[:, 0] = torch.where(f, s["cum"].double().view(-1), total[:, 0])
    total = total.view(R, W * V)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    if W * V < k:
        best = torch.nn.functional.pad(best, (0, k - W * V), value=NEG)
        at = torch.nn.functional.pad(at, (0, k - W * V))
    best, at = best[:, :k], at[:, :k]
    none = best == NEG
    parent, token = (y.masked_fill(none, -1).int() for y in (at // V, at % V))
    return parent, token, best.float()


def _plain_reorder(s):
    W = s["case"]["W"]
    p = s["parent"]
    rows = (p + W * torch.arange(p.shape[0], device=DEV)[:, None]).view(-1)
    return [x[rows] for x in s["states"]]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from transformer_candidate_scoring_b200 import api
        if op == "attention":
            return api.prefix_attention(s["q"], s["k"], s["v"], s["prefix_offsets"], s["seq_offsets"], s["sk"], s["sv"],
                                        s["slen"], causal=s["case"]["causal"])
        if op == "select":
            return api.beam_select(s["logits"], s["cum"], s["case"]["k"], finished=s["finished"], allowed=s["allowed"])
        return api.beam_reorder(s["states"], s["parent"], outs=s["outs"])
    return {"attention": _plain_attention, "select": _plain_select, "reorder": _plain_reorder}[op](s)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "attention":
        n, Lt, H, d = s["q"].shape
        G = H // c["Hkv"]
        out = torch.zeros(n, Lt, H, d, dtype=torch.float64, device=DEV)
        lse = torch.full((n, Lt, H), NEG, dtype=torch.float64, device=DEV)
        slen = s["slen"].tolist() if s["slen"] is not None else [0] * n
        kk = torch.arange(c["S"], device=DEV)
        for r in range(c["R"]):
            s0, s1 = s["seq_offsets"][r:r + 2]
            p0, p1 = s["prefix_offsets"][r:r + 2]
            step = max(1, int(1e8) // max(1, (p1 - p0 + c["S"]) * Lt * G))
            for b0 in range(s0, s1, step):
                b1 = min(s1, b0 + step)
                for h in range(c["Hkv"]):
                    q = s["q"][b0:b1, :, h * G:(h + 1) * G].double() * d ** -0.5           # [b, Lt, G, d]
                    kp, vp = s["k"][p0:p1, h].double(), s["v"][p0:p1, h].double()
                    a = torch.einsum("btgd,jd->btgj", q, kp)
                    if s["sk"] is not None:
                        ks, vs = s["sk"][b0:b1, :, h].double(), s["sv"][b0:b1, :, h].double()
                        e = torch.einsum("btgd,bjd->btgj", q, ks)
                        for t in range(Lt):
                            end = torch.tensor([x - (Lt - 1 - t) if c["causal"] else x for x in slen[b0:b1]], device=DEV)
                            e[:, t][(kk >= end[:, None])[:, None].expand(-1, G, -1)] = NEG
                        a = torch.cat([a, e], -1)
                    if a.shape[-1] == 0:
                        continue
                    z = torch.logsumexp(a, -1)
                    p = torch.where(z[..., None] == NEG, 0.0, torch.exp(a - z[..., None]))
                    o = torch.einsum("btgj,jd->btgd", p[..., :p1 - p0], vp)
                    if s["sk"] is not None:
                        o += torch.einsum("btgj,bjd->btgd", p[..., p1 - p0:], vs)
                    out[b0:b1, :, h * G:(h + 1) * G], lse[b0:b1, :, h * G:(h + 1) * G] = o, z
        return out, lse
    if c["op"] == "select":
        R, W, V, k = c["R"], c["W"], c["V"], c["k"]
        parent = torch.full((R, k), -1, dtype=torch.int32, device=DEV)
        token = torch.full((R, k), -1, dtype=torch.int32, device=DEV)
        score = torch.full((R, k), NEG, dtype=torch.float64, device=DEV)
        bit = torch.arange(32, device=DEV)
        for r in range(R):
            t = torch.log_softmax(s["logits"][r * W:(r + 1) * W].double(), -1) + s["cum"][r].double()[:, None]
            if s["allowed"] is not None:
                bits = (s["allowed"][r * W:(r + 1) * W, :, None] >> bit & 1).view(W, -1)[:, :V]
                t[bits == 0] = NEG
            if s["finished"] is not None:
                f = s["finished"][r]
                t[f] = NEG
                t[f, 0] = s["cum"][r][f].double()
            t = t.view(-1)
            last = torch.topk(t, min(k, t.numel())).values[-1]
            at = torch.nonzero((t >= last) & (t > NEG)).view(-1)                           # ascending
            at = at[torch.argsort(-t[at], stable=True)][:k]
            parent[r, :len(at)], token[r, :len(at)], score[r, :len(at)] = at // V, at % V, t[at]
        return parent, token, score
    W = c["W"]
    p = s["parent"].long()
    return [torch.stack([x.view(c["R"], W, -1)[r][p[r]] for r in range(c["R"])]).view_as(x).double() for x in s["states"]]
