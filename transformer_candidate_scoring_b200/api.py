"""Python binding of libtr: the C ABI's calls under the same names.

Argument marshalling only: torch tensors are passed by device pointer on the current
CUDA stream; every step of the computation runs in libtr's kernels.
"""
from __future__ import annotations

import ctypes as C
import functools
import math
import struct
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


def _on(*tensors) -> int:
    """The device ordinal that all of ``tensors`` (None aside) are on."""
    dev = -2
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("expected CUDA tensors")
                if dev >= 0:
                    raise ValueError(f"tensors on different devices: cuda:{dev} and cuda:{d}")
                dev = d
    return dev


def _run(dev: int, stream, call, *args) -> None:
    """call(*args, stream) with ``dev`` current, on ``stream`` or that device's current one."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(dev)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch._C._cuda_getDevice() == dev:
        status = call(*args, raw)
        if status:
            _check(status)
    else:
        with torch.cuda.device(dev):
            _check(call(*args, raw))


def _new(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """A buffer on the device of ``like`` for work on ``stream`` (None: the current one), out of that stream's
    share of torch's allocator: what the block held before was freed behind work of the same stream."""
    if stream is None:
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):
        raw, dev = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), like.get_device()
        # (torch takes an external handle of 0 for a stream yet to be made)
        stream = torch.cuda.ExternalStream(raw, dev) if raw else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return like.new_empty(shape, dtype=dtype)


def _result(like: torch.Tensor, shape, dtype, stream) -> torch.Tensor:
    """The same for a result: kept from reuse until the caller's current stream has run what uses it, too."""
    t = _new(like, shape, dtype, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _workspace(workspace, need: int, like: torch.Tensor, stream):
    """``workspace`` if it is large enough, or a new buffer of ``need`` bytes on the device of ``like``; and its size."""
    if workspace is None:
        return _new(like, (max(need, 16),), torch.uint8, stream), need
    if not workspace.is_contiguous() or workspace.get_device() != like.get_device():
        raise ValueError("workspace: expected a contiguous tensor on the inputs' device")
    size = workspace.numel() * workspace.element_size()
    if size < need:
        raise ValueError(f"workspace of {size} bytes: need {need}")
    return workspace, size


def _layout(t):
    """What a call's checks and strides depend on; None for no tensor."""
    return None if t is None else (t.shape, t.stride(), t.dtype)


def _kv_strides(k, v, what: str):
    """The strides of keys and values (layouts) whose rows of d_head are contiguous."""
    (shape, stride, dtype), empty = k, 0 in k[0]
    if v[0] != shape or v[2] != dtype:
        raise ValueError(f"{what}: keys and values differ in shape or type")
    if not empty and v[1] != stride:
        raise ValueError(f"{what}: keys and values differ in strides")
    if not empty and shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{what}: the head dimension must be contiguous")
    # a dimension of one entry may come with any stride; it is never multiplied
    return [st if n > 1 else max(shape[-1], 1) for n, st in zip(shape[:-1], stride[:-1])]


@functools.lru_cache(maxsize=1024)
def _attention_plan(q, kp, vp, ks, vs, sl, po, so, scale, causal, dev):
    """The checked arguments of a prefix_attention call that follow from its layouts and offsets, and the
    bytes of its workspace."""
    shape, stride, dtype = q
    if len(shape) not in (3, 4) or len(kp[0]) != 3:
        raise ValueError("expected q [n, L_t, H, d] or [n, H, d] and k_prefix, v_prefix [T, H_kv, d]")
    n, H, d = shape[0], shape[-2], shape[-1]
    L_t = shape[1] if len(shape) == 4 else 1
    H_kv = kp[0][1]
    if 0 not in shape and ((d > 1 and stride[-1] != 1) or (H > 1 and stride[-2] != d)):
        raise ValueError("q: the heads of a token must be contiguous")
    q_token = H * d if n <= 1 and L_t == 1 else stride[0] if L_t == 1 else stride[1]
    if L_t > 1 and n > 1 and stride[0] != L_t * stride[1]:
        raise ValueError("q: the tokens must follow one another at one stride")
    pk = _kv_strides(kp, vp, "prefix")
    if kp[0][2] != d or kp[2] != dtype:
        raise ValueError("prefix: head width or type differs from q's")
    if len(po) < 2 or len(po) != len(so):
        raise ValueError("expected R + 1 prefix_offsets and as many seq_offsets")
    if so[-1] != n or po[-1] > kp[0][0]:
        raise ValueError("seq_offsets must end at n, prefix_offsets within k_prefix")
    S, sk = 0, (0, 0, 0)
    if (ks is None) != (vs is None) or (ks is None) != (sl is None):
        raise ValueError("k_suffix, v_suffix and suffix_len come together")
    if ks is not None:
        if len(ks[0]) != 4 or ks[0][0] != n or ks[0][2:] != (H_kv, d) or ks[2] != dtype:
            raise ValueError("expected k_suffix, v_suffix [n, S, H_kv, d] of q's type")
        if sl[2] != torch.int32 or sl[0] != (n,) or (n > 1 and sl[1] != (1,)):
            raise ValueError("suffix_len: expected contiguous int32 [n]")
        S, sk = ks[0][1], _kv_strides(ks, vs, "suffix")
    desc = L.AttnDesc(H, H_kv, d, L_t, int(causal), S, d ** -0.5 if scale is None else scale, dtype_code(dtype), q_token,
                      pk[0], pk[1], sk[0], sk[1], sk[2])
    R = len(so) - 1
    so_c, po_c = (C.c_int64 * (R + 1))(*so), (C.c_int64 * (R + 1))(*po)
    with torch.cuda.device(dev):
        need = L.load().tr_prefix_attention_workspace(C.byref(desc), so_c, po_c, R)
    if need == C.c_size_t(-1).value:
        _check(L.TR_ERR_INVALID_ARG)
    return C.pointer(desc), so_c, po_c, R, S, need


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
    1 / sqrt(d).  bf16 or fp32.  Buffers that are not given are allocated.  A request's result may
    change with the requests beside it, by rounding (in bf16 of the softmax numerators too)."""
    dev = _on(q, k_prefix, v_prefix, k_suffix, v_suffix, suffix_len, out, lse)
    desc, so, po, R, S, need = _attention_plan(
        _layout(q), _layout(k_prefix), _layout(v_prefix), _layout(k_suffix), _layout(v_suffix), _layout(suffix_len),
        tuple(map(int, prefix_offsets)), tuple(map(int, seq_offsets)), None if scale is None else float(scale), bool(causal), dev)
    if out is None:
        out = torch.empty_like(q) if stream is None and q.is_contiguous() else _result(q, q.shape, q.dtype, stream)
    elif out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError("out: expected q's shape and type")
    else:
        _ptr(out)
    if lse is None:
        lse = _result(q, q.shape[:-1], torch.float32, stream)
    elif lse.shape != q.shape[:-1] or lse.dtype != torch.float32:
        raise ValueError("lse: expected fp32 of q's shape without the last dimension")
    else:
        _ptr(lse)
    ws, size = _workspace(workspace, need, q, stream) if need else (None, 0)
    _run(dev, stream, L.load().tr_prefix_attention, desc, q.data_ptr(), so, k_prefix.data_ptr(), v_prefix.data_ptr(), po,
         k_suffix.data_ptr() if S else None, v_suffix.data_ptr() if S else None, suffix_len.data_ptr() if S else None, R,
         out.data_ptr(), lse.data_ptr(), ws.data_ptr() if need else None, size)
    return out, lse


@functools.lru_cache(maxsize=1024)
def _select_plan(logits, cum, finished, allowed, k):
    """The checked arguments of a beam_select call that follow from its layouts, and the bytes of
    its workspace."""
    if len(cum[0]) != 2 or cum[2] != torch.float32:
        raise ValueError("cum: expected fp32 [R, W]")
    R, W = cum[0]
    shape, stride, dtype = logits
    V = shape[-1]
    if len(shape) == 3 and shape[:2] == (R, W) and (R <= 1 or W <= 1 or stride[0] == W * stride[1]):
        shape, stride = (R * W, V), (stride[1] if W > 1 else stride[0], stride[2])
    if len(shape) != 2 or shape[0] != R * W or (V > 1 and stride[1] != 1):
        raise ValueError("logits: expected [R*W, V] or [R, W, V], contiguous along V, rows at one stride")
    if finished is not None and (finished[2] not in (torch.bool, torch.uint8) or math.prod(finished[0]) != R * W):
        raise ValueError("finished: expected bool or uint8 [R, W]")
    if allowed is not None:
        (ash, ast, adt), words = allowed, -(-V // 32)
        if adt != torch.int32 or len(ash) != 2 or ash[0] != R * W or (ash[1] > 1 and ast[1] != 1) or ash[1] < words:
            raise ValueError("allowed: expected int32 [R*W, ceil(V/32)], contiguous along the words")
    need = L.load().tr_beam_select_workspace(R, W, V, k)
    if need == C.c_size_t(-1).value:
        _check(L.TR_ERR_INVALID_ARG)
    one = R * W <= 1
    return (dtype_code(dtype), V if one else stride[0], 0 if allowed is None else allowed[0][1] if one else allowed[1][0], R, W, V,
            need)


def beam_select(logits: torch.Tensor, cum: torch.Tensor, k: int, *, finished: torch.Tensor = None,
                allowed: torch.Tensor = None, pad_token: int = 0, parent: torch.Tensor = None,
                token: torch.Tensor = None, score: torch.Tensor = None, workspace: torch.Tensor = None, stream=None):
    """tr_beam_select: the k best continuations of every request over its beams and the vocabulary.

    logits [R*W, V] or [R, W, V] (bf16 or fp32, contiguous along V), cum fp32 [R, W] -> (parent
    int32 [R, k], token int32 [R, k], score fp32 [R, k]), best first.  ``finished`` bool or uint8
    [R, W]; ``allowed`` int32 [R*W, ceil(V/32)] or more words: bit v % 32 of word v // 32 allows
    token v."""
    dev = _on(logits, cum, finished, allowed, parent, token, score)
    k = int(k)
    code, ld, allowed_ld, R, W, V, need = _select_plan(_layout(logits), _layout(cum), _layout(finished), _layout(allowed), k)
    for name, t, dt in (("parent", parent, torch.int32), ("token", token, torch.int32), ("score", score, torch.float32)):
        if t is not None:
            if t.shape != (R, k) or t.dtype != dt:
                raise ValueError(f"{name}: expected {dt} [R, k]")
            _ptr(t)
    if parent is None:
        parent = _result(logits, (R, k), torch.int32, stream)
    if token is None:
        token = _result(logits, (R, k), torch.int32, stream)
    if score is None:
        score = _result(logits, (R, k), torch.float32, stream)
    ws, size = _workspace(workspace, need, logits, stream)
    _run(dev, stream, L.load().tr_beam_select, logits.data_ptr(), code, ld, _ptr(cum), _ptr(finished),
         None if allowed is None else allowed.data_ptr(), allowed_ld, R, W, V, k, int(pad_token), parent.data_ptr(), token.data_ptr(),
         score.data_ptr(), ws.data_ptr(), size)
    return parent, token, score


@functools.lru_cache(maxsize=1024)
def _row_layout(shape, stride, size: int):
    """(rows, bytes from row to row, bytes of a row) of a tensor whose rows are contiguous."""
    if len(shape) < 1:
        raise ValueError("states: expected rows")
    inner = 1
    for n, st in zip(reversed(shape[1:]), reversed(stride[1:])):
        if n > 1 and st != inner and 0 not in shape:
            raise ValueError("states: the elements of a row must be contiguous")
        inner *= n
    return shape[0], (stride[0] if shape[0] > 1 else inner) * size, inner * size


def beam_reorder(states: Sequence[torch.Tensor], parent: torch.Tensor, outs: Sequence[torch.Tensor] = None,
                 stream=None) -> Sequence[torch.Tensor]:
    """tr_beam_reorder: row r*W_out + i of every state becomes row r*W_in + parent[r, i] (int32
    [R, W_out]); a negative parent leaves the row as it was.  states: tensors [R*W_in, ...] of any
    type, each row contiguous (cache[:, :len] moves the filled part).  In place without ``outs``;
    else into outs [R*W_out, ...].  Any number of states, none of whose rows another's may overlap
    but where both are only read."""
    states = list(states)
    dsts = states if outs is None else list(outs)
    if parent.dim() != 2 or parent.dtype != torch.int32:
        raise ValueError("parent: expected int32 [R, W_out]")
    R, W_out = parent.shape
    if len(dsts) != len(states):
        raise ValueError("outs: expected one per state")
    dev = _on(parent, *states) if outs is None else _on(parent, *states, *dsts)
    if not states or not R:
        return dsts
    W_in = states[0].shape[0] // R
    flat, last = [], None
    for i, (s, o) in enumerate(zip(states, dsts)):
        layout = (s.shape, s.stride(), s.dtype, o.shape, o.stride(), o.dtype)
        if layout != last:                # (the states of a decoder's layers are alike)
            size = s.element_size()
            rows, stride, row_bytes = _row_layout(layout[0], layout[1], size)
            o_rows, o_stride, _ = _row_layout(layout[3], layout[4], size)
            if o.dtype != s.dtype or o.shape[1:] != s.shape[1:]:
                raise ValueError(f"state {i}: its out differs in row shape or type")
            if rows != R * W_in or o_rows != R * W_out:
                raise ValueError(f"state {i}: expected rows [R*W_in, ...] and an out [R*W_out, ...]")
            last = layout
        flat += (o.data_ptr(), s.data_ptr(), o_stride, stride, row_bytes)
    lib, par, n = L.load(), _ptr(parent), len(states)
    packed = struct.pack("=" + "QQqqq" * n, *flat)
    if n > L.TR_MAX_STATES:               # (several calls: what one moves, another must not read)
        _check(lib.tr_beam_reorder_check(packed, n, par, R, W_in, W_out))
    for i in range(0, n, L.TR_MAX_STATES):
        m, size = min(L.TR_MAX_STATES, n - i), C.sizeof(L.BeamState)
        _run(dev, stream, lib.tr_beam_reorder, packed[i * size:(i + m) * size] if m < n else packed, m, par, R, W_in, W_out)
    return dsts


def sync_status(stream=None, timeout_ms: int = 10_000) -> int:
    """tr_sync_status; returns the status code (does not raise)."""
    return int(L.load().tr_sync_status(_stream(stream), timeout_ms))


def last_error() -> str:
    return L.load().tr_last_error().decode()
