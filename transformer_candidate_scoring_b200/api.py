"""Python binding of libtr: the C ABI's calls under the same names.

Argument marshalling only: torch tensors are passed by device pointer on the current
CUDA stream; every step of the computation runs in libtr's kernels.
"""
from __future__ import annotations

import ctypes as C
from typing import Dict, Sequence

import numpy as np
import torch

from . import _lib as L


class TrError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"libtr status {status}: {msg}")
        self.status = status


def _check(status: int) -> None:
    if status != L.TR_OK:
        raise TrError(status, L.load().tr_last_error().decode())


def _stream(stream) -> C.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _ptr(t: torch.Tensor | None) -> C.c_void_p:
    if t is None:
        return C.c_void_p(0)
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return C.c_void_p(t.data_ptr())


def dtype_code(dt) -> int:
    if dt in (torch.float32, "f32"):
        return L.TR_F32
    if dt in (torch.bfloat16, "bf16"):
        return L.TR_BF16
    raise ValueError(f"unsupported dtype {dt}")


def torch_dtype(code_or_name) -> torch.dtype:
    return torch.bfloat16 if code_or_name in (L.TR_BF16, "bf16") else torch.float32


def kernel_launches() -> int:
    """Kernels libtr has launched so far in this process."""
    return int(L.load().tr_kernel_launches())


def version() -> str:
    return L.load().tr_version().decode()


class Model:
    """A model handle (tr_model_create / tr_model_destroy) built from named fp32 arrays.

    ``params`` uses the names of ``datagen.params``: domain_emb, l{i}.{ln1_g, ..., b2},
    lnf_g, lnf_b, w_head, b_head, c{i}.{W, b, prelu, ln_g, ln_b}.
    """

    def __init__(self, dims, params: Dict[str, np.ndarray]):
        lib = L.load()
        self.dims = dims
        keep = []

        def fp(name):
            a = np.ascontiguousarray(params[name], dtype=np.float32)
            keep.append(a)
            return a.ctypes.data_as(L._fp)

        desc = L.ModelDesc(dims.D, dims.n_layer, dims.n_head, dims.ffn_hidden, dims.n_target_fields,
                           (C.c_int * 4)(*dims.comp_dims), dims.n_domains, dtype_code(dims.dtype))
        layers = (L.LayerWeights * dims.n_layer)()
        for l in range(dims.n_layer):
            for f, _ in L.LayerWeights._fields_:
                setattr(layers[l], f, fp(f"l{l}.{f}"))
        w = L.ModelWeights()
        w.domain_emb = fp("domain_emb")
        w.layers = layers
        w.lnf_g, w.lnf_b, w.w_head = fp("lnf_g"), fp("lnf_b"), fp("w_head")
        w.b_head = float(np.asarray(params["b_head"]).reshape(-1)[0])
        for i in range(3):
            w.comp_W[i] = fp(f"c{i}.W")
            w.comp_b[i] = fp(f"c{i}.b")
        for i in range(2):
            w.comp_prelu[i] = fp(f"c{i}.prelu")
            w.comp_ln_g[i] = fp(f"c{i}.ln_g")
            w.comp_ln_b[i] = fp(f"c{i}.ln_b")
        h = C.c_void_p()
        _check(lib.tr_model_create(C.byref(desc), C.byref(w), C.byref(h)))
        self._h = h

    @property
    def handle(self) -> C.c_void_p:
        return self._h

    def close(self) -> None:
        if getattr(self, "_h", None) and self._h.value:
            L.load().tr_model_destroy(self._h)
            self._h = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


AGG_MODES = {"mean": 0, "sum": 1, "max": 2}
AGG_POST_LN = 0x100


def aggregate(tables: Sequence[torch.Tensor], bag_table: torch.Tensor, offsets: torch.Tensor,
              keys: torch.Tensor, weights: torch.Tensor, out: torch.Tensor, stream=None, mode: str = "mean",
              post_ln: bool = False) -> torch.Tensor:
    """tr_aggregate (mode "mean", no LayerNorm) or tr_aggregate_ex: one token per bag into
    out [n_bags, D]."""
    n = len(tables)
    arr = (L.Table * max(n, 1))()
    for i, t in enumerate(tables):
        arr[i] = L.Table(t.data_ptr(), t.shape[0], dtype_code(t.dtype))
    D = out.shape[-1]
    n_bags = offsets.numel() - 1
    if mode == "mean" and not post_ln:
        _check(L.load().tr_aggregate(arr, n, _ptr(bag_table), _ptr(offsets), _ptr(keys), _ptr(weights),
                                     n_bags, D, dtype_code(out.dtype), _ptr(out), _stream(stream)))
    else:
        code = AGG_MODES[mode] | (AGG_POST_LN if post_ln else 0)
        _check(L.load().tr_aggregate_ex(arr, n, _ptr(bag_table), _ptr(offsets), _ptr(keys), _ptr(weights),
                                        n_bags, D, dtype_code(out.dtype), code, _ptr(out), _stream(stream)))
    return out


def kv_cache_bytes(model: Model, L_u: int) -> int:
    return int(L.load().tr_kv_cache_bytes(model.handle, L_u))


def prefill_user(model: Model, user_tokens: torch.Tensor, L_u: int, domain: int, kv: torch.Tensor,
                 stream=None) -> torch.Tensor:
    """tr_prefill_user: fp32 user tokens [L_u, D] -> this request's K/V cache."""
    _check(L.load().tr_prefill_user(model.handle, _ptr(user_tokens), L_u, domain, _ptr(kv), _stream(stream)))
    return kv


def prefill_users(model: Model, user_tokens: Sequence[torch.Tensor], L_u: Sequence[int], domain: Sequence[int],
                  kv: Sequence[torch.Tensor], stream=None) -> None:
    """tr_prefill_users: the user sides of R requests in one call (fp32 user tokens [L_u, D]
    of each request -> its K/V cache)."""
    R = len(L_u)
    ut = (C.c_void_p * R)(*[(t.data_ptr() if int(l) else 0) for t, l in zip(user_tokens, L_u)])
    kvp = (C.c_void_p * R)(*[(k.data_ptr() if int(l) else 0) for k, l in zip(kv, L_u)])
    lu = (C.c_int32 * R)(*[int(x) for x in L_u])
    dm = (C.c_int32 * R)(*[int(x) for x in domain])
    for t in list(user_tokens) + list(kv):
        if not t.is_cuda:
            raise ValueError("expected CUDA tensors")
    _check(L.load().tr_prefill_users(model.handle, ut, lu, dm, kvp, R, _stream(stream)))


def prefill_user_noalloc(model: Model, user_tokens: torch.Tensor, L_u: int, domain: int, kv: torch.Tensor,
                         stream=None) -> torch.Tensor:
    """tr_prefill_user_noalloc: the user side with no device allocation, for callers that
    cannot allocate (open stream capture, an engine that owns all device memory)."""
    _check(L.load().tr_prefill_user_noalloc(model.handle, _ptr(user_tokens), L_u, domain, _ptr(kv),
                                            _stream(stream)))
    return kv


def compress_targets(model: Model, x: torch.Tensor, tokens: torch.Tensor, stream=None) -> torch.Tensor:
    """tr_compress_targets: x [n, F*D] (model dtype) -> tokens [n, D] fp32."""
    if tokens.dtype != torch.float32:
        raise ValueError("compressed tokens are fp32")
    _check(L.load().tr_compress_targets(model.handle, _ptr(x), x.shape[0], _ptr(tokens), _stream(stream)))
    return tokens


def compress_target_bags(model: Model, tables: Sequence[torch.Tensor], bag_table: torch.Tensor,
                         offsets: torch.Tensor, keys: torch.Tensor, weights: torch.Tensor, tokens: torch.Tensor,
                         stream=None) -> torch.Tensor:
    """tr_compress_target_bags: the target side in one launch, n = tokens.shape[0]
    candidates whose F field bags are c*F .. c*F+F-1 -> tokens [n, D] fp32."""
    if tokens.dtype != torch.float32:
        raise ValueError("compressed tokens are fp32")
    n = len(tables)
    arr = (L.Table * max(n, 1))()
    for i, t in enumerate(tables):
        arr[i] = L.Table(t.data_ptr(), t.shape[0], dtype_code(t.dtype))
    _check(L.load().tr_compress_target_bags(model.handle, arr, n, _ptr(bag_table), _ptr(offsets), _ptr(keys),
                                            _ptr(weights), tokens.shape[0], _ptr(tokens), _stream(stream)))
    return tokens


def score_candidates(model: Model, tokens: torch.Tensor, req_offsets: Sequence[int], kv: Sequence[torch.Tensor],
                     L_u: Sequence[int], domain: Sequence[int], scores: torch.Tensor, stream=None) -> torch.Tensor:
    """tr_score_candidates over packed requests: tokens [n, D] fp32; scores [n] fp32."""
    if tokens.dtype != torch.float32:
        raise ValueError("candidate tokens are fp32")
    R = len(L_u)
    off = (C.c_int64 * (R + 1))(*[int(x) for x in req_offsets])
    kvp = (C.c_void_p * R)(*[(k.data_ptr() if k is not None and k.numel() else 0) for k in kv])
    lu = (C.c_int32 * R)(*[int(x) for x in L_u])
    dm = (C.c_int32 * R)(*[int(x) for x in domain])
    _check(L.load().tr_score_candidates(model.handle, _ptr(tokens), int(req_offsets[-1]), off, kvp, lu, dm, R,
                                        _ptr(scores), _stream(stream)))
    return scores


def score_candidates_uncompressed(model: Model, tokens: torch.Tensor, L_t: int, req_offsets: Sequence[int],
                                  kv: Sequence[torch.Tensor], L_u: Sequence[int], domain: Sequence[int],
                                  scores: torch.Tensor, stream=None) -> torch.Tensor:
    """tr_score_candidates_uncompressed: candidates of L_t target tokens each (tokens
    [n, L_t, D] or [n*L_t, D]); scores [n] fp32."""
    R = len(L_u)
    off = (C.c_int64 * (R + 1))(*[int(x) for x in req_offsets])
    kvp = (C.c_void_p * R)(*[(k.data_ptr() if k is not None and k.numel() else 0) for k in kv])
    lu = (C.c_int32 * R)(*[int(x) for x in L_u])
    dm = (C.c_int32 * R)(*[int(x) for x in domain])
    _check(L.load().tr_score_candidates_uncompressed(model.handle, _ptr(tokens), int(req_offsets[-1]), int(L_t), off,
                                                     kvp, lu, dm, R, _ptr(scores), _stream(stream)))
    return scores


def topk(scores: torch.Tensor, req_offsets: Sequence[int], k: int, out_idx: torch.Tensor = None,
         out_score: torch.Tensor = None, stream=None):
    """tr_topk: per-request top-k; returns (out_idx int64 [R, k], out_score fp32 [R, k])."""
    R = len(req_offsets) - 1
    off = (C.c_int64 * (R + 1))(*[int(x) for x in req_offsets])
    if out_idx is None:
        out_idx = torch.empty(R, k, dtype=torch.int64, device=scores.device)
    if out_score is None:
        out_score = torch.empty(R, k, dtype=torch.float32, device=scores.device)
    _check(L.load().tr_topk(_ptr(scores), int(req_offsets[-1]), off, R, int(k), _ptr(out_idx), _ptr(out_score),
                            _stream(stream)))
    return out_idx, out_score


def _on(stream, *tensors):
    """The device all of ``tensors`` (None aside) are on, and the stream to launch on: ``stream``,
    or that device's current one."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("expected CUDA tensors")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {t.device}")
    return dev, _stream(torch.cuda.current_stream(dev) if stream is None else stream)


def _new(shape, dtype, dev, stream) -> torch.Tensor:
    """A buffer from torch's allocator for work on ``stream`` (None: the current one), kept from
    reuse until that work is done."""
    t = torch.empty(shape, dtype=dtype, device=dev)
    if stream is not None:
        t.record_stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), dev))
    return t


def _workspace(workspace, need: int, dev, stream):
    """``workspace`` if it is large enough, or a new buffer of ``need`` bytes."""
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.device != dev:
            raise ValueError("workspace: expected a contiguous tensor on the inputs' device")
        size = workspace.numel() * workspace.element_size()
        if size < need:
            raise ValueError(f"workspace of {size} bytes: need {need}")
        return workspace, size
    return _new((max(need, 16),), torch.uint8, dev, stream), need


def _host_offsets(x, what: str):
    a = [int(v) for v in x]
    if len(a) < 2:
        raise ValueError(f"{what}: expected R + 1 offsets")
    return (C.c_int64 * len(a))(*a), a


def _kv_strides(k, v, what: str):
    """The strides of a key and a value tensor whose rows of d_head are contiguous."""
    if k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError(f"{what}: keys and values differ in shape or type")
    if k.stride() != v.stride() and k.numel() > 0:
        raise ValueError(f"{what}: keys and values differ in strides")
    if k.numel() > 0 and k.shape[-1] > 1 and k.stride(-1) != 1:
        raise ValueError(f"{what}: the head dimension must be contiguous")
    # a dimension of one entry may come with any stride; it is never multiplied
    inner, strides = k.shape[-1], []
    for size, stride in zip(reversed(k.shape[:-1]), reversed(k.stride()[:-1])):
        strides.insert(0, stride if size > 1 else max(inner, 1))
    return strides


def prefix_attention(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, prefix_offsets: Sequence[int],
                     seq_offsets: Sequence[int], k_suffix: torch.Tensor = None, v_suffix: torch.Tensor = None,
                     suffix_len: torch.Tensor = None, *, scale: float = None, causal: bool = False,
                     out: torch.Tensor = None, lse: torch.Tensor = None, workspace: torch.Tensor = None, stream=None):
    """tr_prefix_attention: attention of sequences that share their request's prefix.

    q [n, L_t, H, d] (or [n, H, d] for one query token; heads contiguous) -> (out, lse), out
    contiguous of q's shape and type, lse fp32 without the last dimension.  Sequences
    seq_offsets[r] .. seq_offsets[r+1]-1 attend to tokens prefix_offsets[r] ..
    prefix_offsets[r+1]-1 of k_prefix, v_prefix [T, H_kv, d] (any token and head strides) and to
    the first suffix_len[s] (int32) tokens of their own k_suffix, v_suffix [n, S, H_kv, d];
    with ``causal``, query token t to L_t - 1 - t fewer of those.  ``scale`` defaults to
    1 / sqrt(d).  bf16 or fp32.  Buffers that are not given are allocated."""
    dev, st = _on(stream, q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_len, out, lse)
    if q.dim() not in (3, 4) or k_prefix.dim() != 3:
        raise ValueError("expected q [n, L_t, H, d] or [n, H, d] and k_prefix, v_prefix [T, H_kv, d]")
    n, H, d = q.shape[0], q.shape[-2], q.shape[-1]
    L_t = q.shape[1] if q.dim() == 4 else 1
    H_kv = k_prefix.shape[1]
    if q.numel() and ((d > 1 and q.stride(-1) != 1) or (H > 1 and q.stride(-2) != d)):
        raise ValueError("q: the heads of a token must be contiguous")
    q_token = q.stride(-3)
    if q.dim() == 4:
        if L_t == 1:
            q_token = q.stride(0)
        elif n > 1 and q.stride(0) != L_t * q.stride(1):
            raise ValueError("q: the tokens must follow one another at one stride")
    if n <= 1 and L_t == 1:
        q_token = H * d
    pk = _kv_strides(k_prefix, v_prefix, "prefix")
    if k_prefix.shape[2] != d or k_prefix.dtype != q.dtype:
        raise ValueError("prefix: head width or type differs from q's")
    po, po_list = _host_offsets(prefix_offsets, "prefix_offsets")
    so, so_list = _host_offsets(seq_offsets, "seq_offsets")
    if len(po_list) != len(so_list):
        raise ValueError("prefix_offsets and seq_offsets differ in length")
    if so_list[-1] != n or po_list[-1] > k_prefix.shape[0]:
        raise ValueError("seq_offsets must end at n, prefix_offsets within k_prefix")
    S, sk = 0, (0, 0, 0)
    if k_suffix is not None:
        if v_suffix is None or suffix_len is None:
            raise ValueError("k_suffix, v_suffix and suffix_len come together")
        if k_suffix.dim() != 4 or k_suffix.shape[0] != n or k_suffix.shape[2:] != (H_kv, d) or k_suffix.dtype != q.dtype:
            raise ValueError("expected k_suffix, v_suffix [n, S, H_kv, d] of q's type")
        if suffix_len.dtype != torch.int32 or suffix_len.shape != (n,) or not suffix_len.is_contiguous():
            raise ValueError("suffix_len: expected contiguous int32 [n]")
        S, sk = k_suffix.shape[1], _kv_strides(k_suffix, v_suffix, "suffix")
    elif v_suffix is not None or suffix_len is not None:
        raise ValueError("k_suffix, v_suffix and suffix_len come together")
    if out is None:
        out = _new(q.shape, q.dtype, dev, stream)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out: expected q's shape and type")
    if lse is None:
        lse = _new(q.shape[:-1], torch.float32, dev, stream)
    elif lse.shape != q.shape[:-1] or lse.dtype != torch.float32:
        raise ValueError("lse: expected fp32 of q's shape without the last dimension")
    desc = L.AttnDesc(H, H_kv, d, L_t, int(bool(causal)), S, d ** -0.5 if scale is None else float(scale),
                      dtype_code(q.dtype), q_token, pk[0], pk[1], sk[0], sk[1], sk[2])
    lib, R = L.load(), len(so_list) - 1
    with torch.cuda.device(dev):
        need = lib.tr_prefix_attention_workspace(C.byref(desc), so, po, R)
        if need == C.c_size_t(-1).value:
            _check(L.TR_ERR_INVALID_ARG)
        ws, size = _workspace(workspace, need, dev, stream)
        _check(lib.tr_prefix_attention(
            C.byref(desc), q.data_ptr(), so, k_prefix.data_ptr(), v_prefix.data_ptr(), po,
            k_suffix.data_ptr() if S else None, v_suffix.data_ptr() if S else None,
            suffix_len.data_ptr() if S else None, R, _ptr(out), _ptr(lse), ws.data_ptr(), size, st))
    return out, lse


def beam_select(logits: torch.Tensor, cum: torch.Tensor, k: int, *, finished: torch.Tensor = None,
                allowed: torch.Tensor = None, pad_token: int = 0, parent: torch.Tensor = None,
                token: torch.Tensor = None, score: torch.Tensor = None, workspace: torch.Tensor = None, stream=None):
    """tr_beam_select: the k best continuations of every request over its beams and the vocabulary.

    logits [R*W, V] or [R, W, V] (bf16 or fp32, contiguous along V), cum fp32 [R, W] -> (parent
    int32 [R, k], token int32 [R, k], score fp32 [R, k]), best first.  ``finished`` bool or uint8
    [R, W]; ``allowed`` int32 [R*W, ceil(V/32)] or more words: bit v % 32 of word v // 32 allows
    token v."""
    dev, st = _on(stream, logits, cum, finished, allowed, parent, token, score)
    if cum.dim() != 2 or cum.dtype != torch.float32:
        raise ValueError("cum: expected fp32 [R, W]")
    R, W = cum.shape
    V = logits.shape[-1]
    rows = logits.view(R * W, V) if logits.dim() == 3 else logits
    if rows.dim() != 2 or rows.shape[0] != R * W or (V > 1 and rows.stride(1) != 1):
        raise ValueError("logits: expected [R*W, V] or [R, W, V], contiguous along V")
    if finished is not None and (finished.dtype not in (torch.bool, torch.uint8) or finished.numel() != R * W):
        raise ValueError("finished: expected bool or uint8 [R, W]")
    if allowed is not None and (allowed.dtype != torch.int32 or allowed.dim() != 2 or allowed.shape[0] != R * W
                                or (allowed.shape[1] > 1 and allowed.stride(1) != 1) or allowed.shape[1] * 32 < V):
        raise ValueError("allowed: expected int32 [R*W, ceil(V/32)], contiguous along the words")
    for name, t, dt in (("parent", parent, torch.int32), ("token", token, torch.int32), ("score", score, torch.float32)):
        if t is not None and (t.shape != (R, k) or t.dtype != dt):
            raise ValueError(f"{name}: expected {dt} [R, k]")
    lib = L.load()
    need = lib.tr_beam_select_workspace(R, W, V, int(k))
    if need == C.c_size_t(-1).value:
        _check(L.TR_ERR_INVALID_ARG)
    if parent is None:
        parent = _new((R, k), torch.int32, dev, stream)
    if token is None:
        token = _new((R, k), torch.int32, dev, stream)
    if score is None:
        score = _new((R, k), torch.float32, dev, stream)
    with torch.cuda.device(dev):
        ws, size = _workspace(workspace, need, dev, stream)
        _check(lib.tr_beam_select(
            rows.data_ptr(), dtype_code(rows.dtype), rows.stride(0) if R * W > 1 else V, _ptr(cum), _ptr(finished),
            None if allowed is None else allowed.data_ptr(),
            0 if allowed is None else allowed.stride(0) if R * W > 1 else allowed.shape[1],
            R, W, V, int(k), int(pad_token), _ptr(parent), _ptr(token), _ptr(score), ws.data_ptr(), size, st))
    return parent, token, score


def _row_bytes(t: torch.Tensor) -> int:
    """Bytes of one row of t, whose elements must be contiguous within the row."""
    if t.dim() < 1 or (t.numel() and not t[0].is_contiguous()):
        raise ValueError("states: the elements of a row must be contiguous")
    return t[0].numel() * t.element_size() if t.shape[0] else 0


def beam_reorder(states: Sequence[torch.Tensor], parent: torch.Tensor, outs: Sequence[torch.Tensor] = None,
                 stream=None) -> Sequence[torch.Tensor]:
    """tr_beam_reorder: row r*W_out + i of every state becomes row r*W_in + parent[r, i] (int32
    [R, W_out]); a negative parent leaves the row as it was.  states: tensors [R*W_in, ...] of any
    type, each row contiguous (cache[:, :len] moves the filled part).  In place without ``outs``;
    else into outs [R*W_out, ...].  Any number of states."""
    states = list(states)
    dsts = states if outs is None else list(outs)
    dev, st = _on(stream, parent, *states, *dsts)
    if parent.dim() != 2 or parent.dtype != torch.int32:
        raise ValueError("parent: expected int32 [R, W_out]")
    R, W_out = parent.shape
    if len(dsts) != len(states):
        raise ValueError("outs: expected one per state")
    if not states or not R:
        return dsts
    W_in = states[0].shape[0] // R
    arr = (L.BeamState * len(states))()
    for i, (s, o) in enumerate(zip(states, dsts)):
        if s.shape[0] != R * W_in or o.shape != (R * W_out, *s.shape[1:]) or o.dtype != s.dtype:
            raise ValueError(f"state {i}: expected rows [R*W_in, ...] and an out [R*W_out, ...] of the same type")
        nb = _row_bytes(s)
        _row_bytes(o)
        e = s.element_size()
        arr[i] = L.BeamState(o.data_ptr(), s.data_ptr(), o.stride(0) * e if R * W_out > 1 else nb,
                             s.stride(0) * e if R * W_in > 1 else nb, nb)
    lib = L.load()
    with torch.cuda.device(dev):
        for i in range(0, len(states), L.TR_MAX_STATES):
            m = min(L.TR_MAX_STATES, len(states) - i)
            _check(lib.tr_beam_reorder(C.pointer(arr[i]), m, _ptr(parent), R, W_in, W_out, st))
    return dsts


def sync_status(stream=None, timeout_ms: int = 10_000) -> int:
    """tr_sync_status; returns the status code (does not raise)."""
    return int(L.load().tr_sync_status(_stream(stream), timeout_ms))


def last_error() -> str:
    return L.load().tr_last_error().decode()
