"""Python binding of the jenga C ABI: same names, torch tensors in, argument
marshalling only.  Every step of the path runs in libjenga.so kernels; PyTorch
supplies device memory (outputs, workspaces) and the current CUDA stream.
"""
import ctypes

import torch

from . import _lib
from ._lib import BF16, F32, LayerWeights, Lora, LoraGrads, check, load

SCORE_MODES = {"softmax_mass": _lib.SCORE_SOFTMAX_MASS, "paper_blockmax": _lib.SCORE_PAPER_BLOCKMAX}
SELECT_MODES = {"mean_ge": _lib.SELECT_MEAN_GE, "topk_frac": _lib.SELECT_TOPK_FRAC, "abs_ge": _lib.SELECT_ABS_GE,
                "topk": _lib.SELECT_TOPK}

ACTIVATIONS = {"none": _lib.ACT_NONE, "relu": _lib.ACT_RELU, "gelu": _lib.ACT_GELU, "silu": _lib.ACT_SILU}


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _dt(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _p(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _ws(nbytes, device):
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("jenga: tensors must be CUDA tensors (the library has no CPU path)")


# ------------------------------------------------------------------ status
def jenga_check_device_status(stream=None):
    lib = load()
    det = (ctypes.c_uint32 * 2)()
    st = lib.jenga_check_device_status(_stream(stream), det)
    if st != 0:
        raise _lib.JengaError(st, _lib.last_error())


def jenga_set_wait_budget_ns(ns):
    check(load().jenga_set_wait_budget_ns(int(ns)))


def jenga_version():
    return load().jenga_version().decode()


def jenga_profile_enable(on=True):
    check(load().jenga_profile_enable(1 if on else 0))


def jenga_profile_report():
    """Per-kernel launch counts and milliseconds recorded since jenga_profile_enable."""
    import json
    lib = load()
    buf = ctypes.create_string_buffer(1 << 16)
    lib.jenga_profile_report(buf, 1 << 16)
    return json.loads(buf.value.decode())


# ------------------------------------------------------------------ scoring / selection / movement
def jenga_score_blocks(q, k, heads, head_dim, blk, causal=True, mode="softmax_mass", out=None, ws=None,
                       stream=None):
    """q, k: [B, S, >= heads*head_dim] (or [S, ...]) fp32/bf16 CUDA tensors, last dim contiguous."""
    _need_cuda(q, k)
    q3 = q if q.dim() == 3 else q.unsqueeze(0)
    k3 = k if k.dim() == 3 else k.unsqueeze(0)
    B, S = q3.shape[0], q3.shape[1]
    assert q3.stride(-1) == 1 and k3.stride(-1) == 1 and q3.stride(0) == S * q3.stride(1)
    nb = S // blk
    lib = load()
    need = lib.jenga_score_workspace_bytes(B, S, heads, head_dim, blk)
    if ws is None:
        ws = _ws(need, q.device)
    if out is None:
        out = torch.empty(B, nb, dtype=torch.float32, device=q.device)
    check(lib.jenga_score_blocks(_p(q3), q3.stride(1), _p(k3), k3.stride(1), B, S, heads, head_dim, blk,
                                 1 if causal else 0, _dt(q3), SCORE_MODES[mode], _p(out), _p(ws), ws.numel(),
                                 _stream(stream)))
    return out if q.dim() == 3 else out[0]


def jenga_select(scores, mode, param=0.0, out=None, ws=None, stream=None):
    """scores [B, nb] fp32 -> (idx int32 [B, nb], n_kept int32 [B], mask uint8 [B, nb]).
    out: optional preallocated (idx, n_kept, mask)."""
    _need_cuda(scores)
    s2 = scores if scores.dim() == 2 else scores.unsqueeze(0)
    s2 = s2.contiguous()
    B, nb = s2.shape
    lib = load()
    if out is not None:
        idx, nk, mask = out
    else:
        idx = torch.empty(B, nb, dtype=torch.int32, device=scores.device)
        nk = torch.empty(B, dtype=torch.int32, device=scores.device)
        mask = torch.empty(B, nb, dtype=torch.uint8, device=scores.device)
    need = lib.jenga_select_workspace_bytes(B, nb)
    if ws is None or ws.numel() < need:
        ws = _ws(need, scores.device)
    check(lib.jenga_select(_p(s2), B, nb, SELECT_MODES[mode], float(param), _p(idx), _p(nk), _p(mask), _p(ws),
                           ws.numel(), _stream(stream)))
    if scores.dim() == 1:
        return idx[0], nk, mask[0]
    return idx, nk, mask


def jenga_gather(x, idx, n_kept, blk, n_cap, out=None, stream=None):
    """x [B, S, h] or [S, h]; returns out [B, n_cap, h] (rows past n_kept*blk untouched)."""
    _need_cuda(x, idx, n_kept)
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    B, S, h = x3.shape
    if out is None:
        out = torch.empty(B, n_cap, h, dtype=x.dtype, device=x.device)
    o3 = out if out.dim() == 3 else out.unsqueeze(0)
    check(load().jenga_gather(_p(x3), x3.stride(1), B, S, h, blk, _p(idx), _p(n_kept), _dt(x3), _p(o3), o3.stride(1),
                              n_cap, _stream(stream)))
    return out if x.dim() == 3 else o3[0]


def jenga_scatter_add(x, y, idx, n_kept, blk, alpha=1.0, stream=None):
    """In place: x[row(i)] = round(x + alpha * y[i]) on retained rows."""
    _need_cuda(x, y, idx, n_kept)
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    y3 = y if y.dim() == 3 else y.unsqueeze(0)
    B, S, h = x3.shape
    check(load().jenga_scatter_add(_p(x3), x3.stride(1), _p(y3), y3.stride(1), B, S, h, blk, _p(idx), _p(n_kept),
                                   float(alpha), _dt(x3), y3.shape[1], _stream(stream)))
    return x


def jenga_scale_rows(x, rows, factor, stream=None):
    _need_cuda(x, rows)
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    B, S, h = x3.shape
    r2 = rows if rows.dim() == 2 else rows.unsqueeze(0)
    check(load().jenga_scale_rows(_p(x3), x3.stride(1), B, S, h, _p(r2), r2.shape[1], float(factor), _dt(x3),
                                  _stream(stream)))
    return x


# ------------------------------------------------------------------ layer
class LayerHandle:
    """Device tensors of one layer (frozen bf16 weights, LoRA, packed re-layout) and the
    ctypes structs that point at them."""

    def __init__(self, wq, wk, wv, wo, wg, wu, wd, attn_norm, mlp_norm, aq, bq, av, bv, heads, head_dim,
                 rms_eps=1e-5, rope_theta=10000.0, lora_scale=1.0, stream=None):
        ts = dict(wq=wq, wk=wk, wv=wv, wo=wo, wg=wg, wu=wu, wd=wd, attn_norm=attn_norm, mlp_norm=mlp_norm,
                  aq=aq, bq=bq, av=av, bv=bv)
        for k, t in ts.items():
            if not (t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
                raise ValueError(f"{k}: contiguous bf16 CUDA tensor required")
        self.t = ts
        self.hidden = wq.shape[1]
        self.heads, self.head_dim, self.ffn = heads, head_dim, wg.shape[0]
        self.w = LayerWeights(self.hidden, heads, head_dim, self.ffn, rms_eps, rope_theta,
                              _p(attn_norm), _p(mlp_norm), _p(wq), _p(wk), _p(wv), _p(wo), _p(wg), _p(wu), _p(wd))
        self.lora = Lora(aq.shape[0], lora_scale, _p(aq), _p(bq), _p(av), _p(bv))
        lib = load()
        n = lib.jenga_layer_pack_bytes(ctypes.byref(self.w), ctypes.byref(self.lora))
        if n == 0:
            raise ValueError("jenga_layer_pack_bytes rejected the layer shape: " + _lib.last_error())
        self.packed = _ws(n, wq.device)
        check(lib.jenga_layer_pack(ctypes.byref(self.w), ctypes.byref(self.lora), _p(self.packed),
                                   self.packed.numel(), _stream(stream)))

    def saved_bytes(self, blk, n_kept_max, B=1):
        return load().jenga_layer_saved_bytes(ctypes.byref(self.w), B, blk, n_kept_max)

    def fwd_ws_bytes(self, blk, n_kept_max, B=1):
        return load().jenga_layer_fwd_workspace_bytes(ctypes.byref(self.w), B, blk, n_kept_max)

    def bwd_ws_bytes(self, blk, n_kept_max, segment_tokens, B=1):
        return load().jenga_layer_bwd_workspace_bytes(ctypes.byref(self.w), B, blk, n_kept_max, segment_tokens)

    def qk_ws_bytes(self, S, B=1):
        return load().jenga_layer_score_qk_workspace_bytes(ctypes.byref(self.w), B, S)


def jenga_layer_score_qk(layer: LayerHandle, x, out=None, ws=None, stream=None):
    """q and k of all S tokens for scoring: x [S, h] bf16 -> [S, 2*H*D] bf16 (q | k)."""
    _need_cuda(x)
    S = x.shape[-2]
    HD = layer.heads * layer.head_dim
    if out is None:
        out = torch.empty(S, 2 * HD, dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = _ws(layer.qk_ws_bytes(S), x.device)
    check(load().jenga_layer_score_qk(ctypes.byref(layer.w), ctypes.byref(layer.lora), _p(layer.packed), _p(x), 1, S,
                                      _p(out), _p(ws), ws.numel(), _stream(stream)))
    return out


def jenga_sparse_layer_fwd(layer: LayerHandle, x, idx, n_kept, blk, n_kept_max, saved=None, ws=None, stream=None,
                           qk=None):
    """In place on x [S, h] bf16.  Returns the saved-context buffer for the backward.

    qk: optional [S, 2 H D] bf16 q | k of all rows from jenga_layer_score_qk on the same x;
    the retained rows' q and k are then taken from it (bit-identical) instead of projected.
    qk must have been computed from this x, after any change to x (e.g. jenga_scale_rows),
    and with this layer's weights and LoRA: a stale qk silently gives wrong q and k."""
    _need_cuda(x, idx, n_kept)
    S = x.shape[-2]
    if saved is None:
        saved = _ws(layer.saved_bytes(blk, n_kept_max), x.device)
    if ws is None:
        ws = _ws(layer.fwd_ws_bytes(blk, n_kept_max), x.device)
    if qk is None:
        check(load().jenga_sparse_layer_fwd(ctypes.byref(layer.w), ctypes.byref(layer.lora), _p(layer.packed), _p(x), 1,
                                            S, blk, _p(idx), _p(n_kept), int(n_kept_max), _p(saved), saved.numel(),
                                            _p(ws), ws.numel(), _stream(stream)))
    else:
        _need_cuda(qk)
        HD = layer.heads * layer.head_dim
        if qk.dtype != torch.bfloat16 or qk.device != x.device:
            raise ValueError("qk must be a bf16 tensor on x's device")
        if qk.dim() != 2 or qk.shape[0] < S or qk.shape[1] < 2 * HD or qk.stride(1) != 1:
            raise ValueError(f"qk must be [>= {S}, >= {2 * HD}] with a contiguous last dimension, got "
                             f"{tuple(qk.shape)} strides {qk.stride()}")
        check(load().jenga_sparse_layer_fwd_qk(ctypes.byref(layer.w), ctypes.byref(layer.lora), _p(layer.packed), _p(x),
                                               1, S, blk, _p(idx), _p(n_kept), int(n_kept_max), _p(qk), qk.stride(0),
                                               _p(saved), saved.numel(), _p(ws), ws.numel(), _stream(stream)))
    return saved


def jenga_sparse_layer_fwd_mlp(layer: LayerHandle, x, idx, n_kept, blk, n_kept_max, mlp_mode, mlp_param, saved=None,
                               ws=None, stream=None, qk=None, mlp_pos=None, n_mlp=None, mlp_scores=None):
    """jenga_sparse_layer_fwd with MLP-block elimination: the MLP sub-block keeps the retained
    blocks that jenga_select(mlp_mode, mlp_param) picks on their SiLU(gate) * up mass.
    Returns (saved, mlp_scores fp32 [n_kept_max], mlp_pos int32 [n_kept_max], n_mlp int32 [1])."""
    _need_cuda(x, idx, n_kept)
    S = x.shape[-2]
    if saved is None:
        saved = _ws(layer.saved_bytes(blk, n_kept_max), x.device)
    if ws is None:
        ws = _ws(layer.fwd_ws_bytes(blk, n_kept_max), x.device)
    if mlp_pos is None:
        mlp_pos = torch.empty(max(int(n_kept_max), 1), dtype=torch.int32, device=x.device)
    if n_mlp is None:
        n_mlp = torch.empty(1, dtype=torch.int32, device=x.device)
    if mlp_scores is None:
        mlp_scores = torch.empty(max(int(n_kept_max), 1), dtype=torch.float32, device=x.device)
    ld_qk = 0
    if qk is not None:
        _need_cuda(qk)
        HD = layer.heads * layer.head_dim
        if qk.dtype != torch.bfloat16 or qk.device != x.device or qk.dim() != 2 or qk.shape[0] < S \
                or qk.shape[1] < 2 * HD or qk.stride(1) != 1:
            raise ValueError("qk must be a bf16 [>= S, >= 2 H D] tensor on x's device, last dimension contiguous")
        ld_qk = qk.stride(0)
    check(load().jenga_sparse_layer_fwd_mlp(ctypes.byref(layer.w), ctypes.byref(layer.lora), _p(layer.packed), _p(x), 1,
                                            S, blk, _p(idx), _p(n_kept), int(n_kept_max), _p(qk), ld_qk,
                                            SELECT_MODES[mlp_mode], float(mlp_param), _p(mlp_scores), _p(mlp_pos),
                                            _p(n_mlp), _p(saved), saved.numel(), _p(ws), ws.numel(), _stream(stream)))
    return saved, mlp_scores, mlp_pos, n_mlp


def new_lora_grads(layer: LayerHandle):
    dev = layer.t["aq"].device
    return {k: torch.zeros(layer.t[k[1:]].shape, dtype=torch.float32, device=dev) for k in ("daq", "dbq", "dav", "dbv")}


def jenga_sparse_layer_bwd(layer: LayerHandle, dx, idx, n_kept, blk, n_kept_max, saved, grads, segment_tokens=4096,
                           ws=None, stream=None):
    """dx [S, h] bf16 holds G on entry and dL/dx on return; grads (dict of fp32) accumulate."""
    _need_cuda(dx, idx, n_kept, saved)
    S = dx.shape[-2]
    if ws is None:
        ws = _ws(layer.bwd_ws_bytes(blk, n_kept_max, segment_tokens), dx.device)
    g = LoraGrads(_p(grads["daq"]), _p(grads["dbq"]), _p(grads["dav"]), _p(grads["dbv"]))
    check(load().jenga_sparse_layer_bwd(ctypes.byref(layer.w), ctypes.byref(layer.lora), _p(layer.packed), _p(dx), 1, S,
                                        blk, _p(idx), _p(n_kept), int(n_kept_max), _p(saved), saved.numel(),
                                        ctypes.byref(g), int(segment_tokens), _p(ws), ws.numel(), _stream(stream)))
    return dx


# ------------------------------------------------------------------ predictor
def jenga_predict_blocks(x, blk, w1, b1, w2, b2, out=None, ws=None, stream=None):
    """x [S, h] bf16; w1 [m, h] bf16, b1 [m] fp32, w2 [m] bf16, b2 [1] fp32 -> scores [nb] fp32."""
    _need_cuda(x, w1, b1, w2, b2)
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    B, S, h = x3.shape
    nb = S // blk
    lib = load()
    if ws is None:
        ws = _ws(lib.jenga_predict_workspace_bytes(B, S, h, blk), x.device)
    if out is None:
        out = torch.empty(B, nb, dtype=torch.float32, device=x.device)
    check(lib.jenga_predict_blocks(_p(x3), B, S, h, blk, _p(w1), _p(b1), _p(w2), _p(b2), w1.shape[0], _p(out), _p(ws),
                                   ws.numel(), _stream(stream)))
    return out if x.dim() == 3 else out[0]


def jenga_mlp_block_scores(a, blk, n_kept=None, out=None, stream=None):
    """a [n_cap * blk, F] bf16 (compact retained rows) -> scores [n_cap] fp32 (-inf past n_kept)."""
    _need_cuda(a)
    n_cap = a.shape[0] // blk
    if out is None:
        out = torch.empty(n_cap, dtype=torch.float32, device=a.device)
    check(load().jenga_mlp_block_scores(_p(a), a.stride(0), a.shape[1], blk, _p(n_kept) if n_kept is not None else None,
                                        n_cap, _p(out), _stream(stream)))
    return out


def jenga_compose_block_indices(outer, pos, n_pos, out=None, stream=None):
    """out[i] = outer[pos[i]] for i < n_pos, -1 after (int32 device tensors)."""
    _need_cuda(outer, pos, n_pos)
    if out is None:
        out = torch.empty(pos.numel(), dtype=torch.int32, device=pos.device)
    check(load().jenga_compose_block_indices(_p(outer), outer.numel(), _p(pos), _p(n_pos), pos.numel(), _p(out),
                                             _stream(stream)))
    return out


def jenga_predict_blocks_qk(x, blk, q_w, k_w, causal=True, out=None, ws=None, stream=None):
    """x [S, h] or [B, S, h] bf16; q_w, k_w: (W1 [r1, h], W2 [r2, r1], W3 [d, r2]) bf16 ->
    scores [nb] (or [B, nb]) fp32: column sums of the query-key score-block products."""
    _need_cuda(x, *q_w, *k_w)
    x3 = x if x.dim() == 3 else x.unsqueeze(0)
    B, S, h = x3.shape
    r1, r2, d = q_w[0].shape[0], q_w[1].shape[0], q_w[2].shape[0]
    lib = load()
    if ws is None:
        ws = _ws(lib.jenga_predict_qk_workspace_bytes(B, S, h, blk, d), x.device)
    if out is None:
        out = torch.empty(B, S // blk, dtype=torch.float32, device=x.device)
    check(lib.jenga_predict_blocks_qk(_p(x3), B, S, h, blk, *[_p(t) for t in q_w], *[_p(t) for t in k_w], r1, r2, d,
                                      1 if causal else 0, _p(out), _p(ws), ws.numel(), _stream(stream)))
    return out if x.dim() == 3 else out[0]


def jenga_lm_loss_segmented(hidden, w, labels, segment_tokens=4096, dhidden=None, loss=None, ws=None, stream=None):
    """hidden [S, h] bf16, w [V, h] bf16, labels [S] int32 -> (loss fp32 [1], dhidden [S, h] bf16).

    Mean causal-LM cross-entropy over the tokens whose label is in [0, V) and its gradient
    with respect to hidden, computed segment_tokens rows at a time."""
    _need_cuda(hidden, w, labels)
    S, h = hidden.shape
    V = w.shape[0]
    lib = load()
    if ws is None:
        ws = _ws(lib.jenga_lm_loss_workspace_bytes(S, h, V, segment_tokens), hidden.device)
    if dhidden is None:
        dhidden = torch.empty(S, h, dtype=torch.bfloat16, device=hidden.device)
    if loss is None:
        loss = torch.empty(1, dtype=torch.float32, device=hidden.device)
    check(lib.jenga_lm_loss_segmented(_p(hidden), _p(w), _p(labels), S, h, V, segment_tokens, _p(loss), _p(dhidden),
                                      _p(ws), ws.numel(), _stream(stream)))
    return loss, dhidden


# ------------------------------------------------------------------ dense sub-block operators
# These calls are short (a few microseconds of kernel for small inputs), so the binding passes
# plain integers and touches each tensor attribute once.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _begin(stream, x, *ts):
    """The call's device guard and stream.  All tensors are on one CUDA device; outputs and
    workspaces are allocated under the call's stream, so the caching allocator reuses them in
    that stream's order.  Returns (guard to leave or None, raw stream)."""
    dev = x.get_device()
    for t in (x, *ts):
        if t is not None and t.get_device() != dev:
            if not t.is_cuda or dev < 0:
                raise ValueError("jenga: tensors must be CUDA tensors (the library has no CPU path)")
            raise ValueError(f"jenga: tensors on {t.device} and {x.device}")
    if dev < 0:
        raise ValueError("jenga: tensors must be CUDA tensors (the library has no CPU path)")
    if stream is not None:
        if stream.device_index != dev:
            raise ValueError(f"jenga: stream of device {stream.device_index}, tensors on {x.device}")
        guard = torch.cuda.stream(stream)
        guard.__enter__()
        return guard, stream.cuda_stream
    guard = None
    if torch.cuda.current_device() != dev:
        guard = torch.cuda.device(dev)
        guard.__enter__()
    return guard, _raw_stream(dev)


def _end(guard):
    if guard is not None:
        guard.__exit__(None, None, None)


def _ptr(t):
    return t.data_ptr() if t is not None else None


_INT_MAX = 2 ** 31 - 1


def _mat(t, name, cols=None, rows=None, dtype=None):
    """A 2-d tensor with contiguous rows; its pitch."""
    shape, st = t.shape, t.stride()
    if len(shape) != 2 or (st[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: a matrix with contiguous rows required, got {tuple(shape)} strides {st}")
    if (cols is not None and shape[1] != cols) or (rows is not None and shape[0] < rows):
        raise ValueError(f"{name}: [{'>= ' + str(rows) if rows is not None else '*'}, {cols}] required, got {tuple(shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name}: {dtype} required, got {t.dtype}")
    if shape[0] > _INT_MAX or shape[1] > _INT_MAX:  # ctypes would pass the low 32 bits
        raise ValueError(f"{name}: {tuple(shape)}: at most 2^31 - 1 rows and columns")
    if shape[0] > 1:
        if st[0] < shape[1]:
            raise ValueError(f"{name}: rows overlap (strides {st})")
        return st[0]
    return max(st[0], shape[1])


def _vec(t, name, n, dtype=None):
    if t is not None and (t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1)
                          or (dtype is not None and t.dtype != dtype)):
        raise ValueError(f"{name}: contiguous {dtype if dtype is not None else ''} [{n}] required, got {t.dtype} "
                         f"{tuple(t.shape)}")


def _rows_arg(idx, n_kept, blk, n_kept_max, rows):
    """Rows of a call: n_kept_max blocks with a block list, else `rows`."""
    if not 1 <= blk <= _INT_MAX:
        raise ValueError(f"blk: {blk} rows a block")
    for t, name in ((idx, "idx"), (n_kept, "n_kept")):
        if t is not None and (t.dtype != torch.int32 or not t.is_contiguous()):
            raise ValueError(f"{name}: contiguous int32 required")
    if n_kept is not None and n_kept.numel() != 1:
        raise ValueError(f"n_kept: one count required, got {tuple(n_kept.shape)}")
    if idx is None:
        return rows
    n = idx.numel() if n_kept_max is None else int(n_kept_max)
    if n < 0 or n > idx.numel():
        raise ValueError(f"n_kept_max {n} of a list of {idx.numel()}")
    if n * blk > _INT_MAX:
        raise ValueError(f"{n} blocks of {blk} rows: at most 2^31 - 1 rows")
    return n * int(blk)


def jenga_layernorm_fwd(x, gamma=None, beta=None, eps=1e-5, idx=None, n_kept=None, blk=1, n_kept_max=None, out=None,
                        mean=None, rstd=None, stream=None):
    """Layer norm of the rows of x [S, h] (fp32 / bf16), or of the kept blocks' rows with idx
    (n_kept_max blocks of blk rows, default all of idx) -> (y [rows, h], mean, rstd fp32 [rows]).

    gamma, beta: [h] fp32 or bf16 (both alike), optional.  n_kept: device int32 count of valid
    blocks; rows past it stay as they are in the outputs.  out may be x itself without idx."""
    guard, s = _begin(stream, x, gamma, beta, idx, n_kept, out, mean, rstd)
    try:
        ldx = _mat(x, "x")
        S, h = x.shape
        rows = S if idx is None and n_kept is None else _rows_arg(idx, n_kept, blk, n_kept_max, S)
        w = gamma if gamma is not None else beta
        if gamma is not None:
            _vec(gamma, "gamma", h)
        if beta is not None:
            _vec(beta, "beta", h, w.dtype)
        dt = _dt(x)
        if out is None:
            y, ldy = x.new_empty((rows, h)), h
        else:
            y, ldy = out, _mat(out, "out", h, rows, x.dtype)
        if mean is None:
            mean = x.new_empty(rows, dtype=torch.float32)
        else:
            _vec(mean, "mean", rows, torch.float32)
        if rstd is None:
            rstd = x.new_empty(rows, dtype=torch.float32)
        else:
            _vec(rstd, "rstd", rows, torch.float32)
        check(load().jenga_layernorm_fwd(x.data_ptr(), ldx, S, h, _ptr(idx), _ptr(n_kept), int(blk), rows, _ptr(gamma),
                                         _ptr(beta), _dt(w) if w is not None else F32, float(eps), dt, y.data_ptr(), ldy,
                                         mean.data_ptr(), rstd.data_ptr(), s))
    finally:
        _end(guard)
    return y, mean, rstd


def jenga_layernorm_bwd(dy, x, mean, rstd, gamma=None, idx=None, n_kept=None, blk=1, n_kept_max=None, dres=None,
                        dx=None, dgamma=None, dbeta=None, accumulate=False, weight_grads=True, ws=None, stream=None):
    """Gradients of jenga_layernorm_fwd: dy [rows, h] compact; x, dres and dx like the forward's x
    -> (dx, dgamma fp32 [h], dbeta fp32 [h]).

    dres: gradient of the residual branch, added into dx (dx may be dres: in place).  With idx or
    n_kept and no dx given, rows outside the list are zero.  accumulate: add into the given dgamma and
    dbeta.  weight_grads=False skips both (None unless given)."""
    guard, s = _begin(stream, x, dy, mean, rstd, gamma, idx, n_kept, dres, dx, dgamma, dbeta, ws)
    try:
        ldx = _mat(x, "x")
        S, h = x.shape
        rows = S if idx is None and n_kept is None else _rows_arg(idx, n_kept, blk, n_kept_max, S)
        ldy = _mat(dy, "dy", h, rows, x.dtype)
        if gamma is not None:
            _vec(gamma, "gamma", h)
        _vec(mean, "mean", rows, torch.float32)
        _vec(rstd, "rstd", rows, torch.float32)
        dt = _dt(x)
        if dx is None:
            dx, ldd = x.new_empty((S, h)) if idx is None and n_kept is None else x.new_zeros((S, h)), h
        else:
            ldd = _mat(dx, "dx", h, S, x.dtype)
        ldr = _mat(dres, "dres", h, S, x.dtype) if dres is not None else 0
        if weight_grads and accumulate and (dgamma is None or dbeta is None):
            raise ValueError("accumulate needs dgamma and dbeta")
        if dgamma is not None:
            _vec(dgamma, "dgamma", h, torch.float32)
        elif weight_grads:
            dgamma = mean.new_empty(h)
        if dbeta is not None:
            _vec(dbeta, "dbeta", h, torch.float32)
        elif weight_grads:
            dbeta = mean.new_empty(h)
        lib = load()
        if ws is None and (dgamma is not None or dbeta is not None):
            ws = x.new_empty(lib.jenga_layernorm_bwd_workspace_bytes(rows, h), dtype=torch.uint8)
        check(lib.jenga_layernorm_bwd(dy.data_ptr(), ldy, x.data_ptr(), ldx, S, h, _ptr(idx), _ptr(n_kept), int(blk), rows,
                                      mean.data_ptr(), rstd.data_ptr(), _ptr(gamma),
                                      _dt(gamma) if gamma is not None else F32, _ptr(dres), ldr, dt, dx.data_ptr(),
                                      ldd, _ptr(dgamma), _ptr(dbeta), 1 if accumulate else 0, _ptr(ws),
                                      ws.numel() if ws is not None else 0, s))
    finally:
        _end(guard)
    return dx, dgamma, dbeta


def jenga_linear_fwd(x, w, bias=None, act="none", residual=None, n_kept=None, blk=1, out=None, pre=None,
                     save_pre=False, ws=None, stream=None):
    """y = act(x w^T + bias) + residual: x [M, K], w [N, K], residual [M, N] bf16, bias [N] fp32 or
    bf16 -> (y [M, N] bf16, pre [M, N] bf16 or None).

    act: "none", "relu", "gelu" (erf) or "silu".  save_pre (or a given pre) keeps x w^T + bias for
    the backward.  n_kept: device int32 count of valid blocks of blk rows; later rows of the
    outputs stay as they are.  out may be residual itself."""
    bf = torch.bfloat16
    guard, s = _begin(stream, x, w, bias, residual, n_kept, out, pre, ws)
    try:
        ldx = _mat(x, "x", dtype=bf)
        M, K = x.shape
        ldw = _mat(w, "w", K, dtype=bf)
        N = w.shape[0]
        if n_kept is not None:
            _rows_arg(None, n_kept, blk, None, M)
        if bias is not None:
            _vec(bias, "bias", N)
        ldr = _mat(residual, "residual", N, M, bf) if residual is not None else 0
        y = x.new_empty((M, N)) if out is None else out
        ldy = N if out is None else _mat(y, "out", N, M, bf)
        if pre is None and save_pre:
            pre = x.new_empty((M, N))
        ldp = _mat(pre, "pre", N, M, bf) if pre is not None else 0
        lib = load()
        nws = lib.jenga_linear_fwd_workspace_bytes(M, N, K)
        if ws is None and nws:
            ws = x.new_empty(nws, dtype=torch.uint8)
        check(lib.jenga_linear_fwd(x.data_ptr(), ldx, w.data_ptr(), ldw, _ptr(bias),
                                   _dt(bias) if bias is not None else F32, ACTIVATIONS[act], _ptr(residual), ldr, M, N,
                                   K, _ptr(n_kept), int(blk), y.data_ptr(), ldy, _ptr(pre), ldp, _ptr(ws),
                                   ws.numel() if ws is not None else 0, s))
    finally:
        _end(guard)
    return y, pre


def jenga_linear_bwd(dy, x, w, act="none", pre=None, n_kept=None, blk=1, need=("dx", "dw", "db"), dx=None, dw=None,
                     db=None, accumulate=False, ws=None, stream=None):
    """Gradients of jenga_linear_fwd: dy [M, N], x [M, K], w [N, K], pre [M, N] bf16 ->
    (dx [M, K] bf16, dw [N, K] fp32, db [N] fp32), None for what `need` leaves out.

    accumulate: add into the given dw and db.  The residual's gradient is dy itself."""
    bf, f32 = torch.bfloat16, torch.float32
    guard, s = _begin(stream, x, dy, w, pre, n_kept, dx, dw, db, ws)
    try:
        ldx = _mat(x, "x", dtype=bf)
        M, K = x.shape
        ldw = _mat(w, "w", K, dtype=bf)
        N = w.shape[0]
        ldy = _mat(dy, "dy", N, M, bf)
        if n_kept is not None:
            _rows_arg(None, n_kept, blk, None, M)
        if act != "none" and pre is None:
            raise ValueError(f"the gradient of {act} needs pre")
        ldp = _mat(pre, "pre", N, M, bf) if pre is not None else 0
        want_w, want_b = "dw" in need, "db" in need
        if accumulate and ((want_w and dw is None) or (want_b and db is None)):
            raise ValueError("accumulate needs dw and db")
        ldd, lddw = K, K
        if "dx" not in need:
            dx = None
        elif dx is None:
            dx = x.new_empty((M, K))
        else:
            ldd = _mat(dx, "dx", K, M, bf)
        if not want_w:
            dw = None
        elif dw is None:
            dw = x.new_empty((N, K), dtype=f32)
        else:
            lddw = _mat(dw, "dw", K, N, f32)
        if not want_b:
            db = None
        elif db is None:
            db = x.new_empty(N, dtype=f32)
        else:
            _vec(db, "db", N, f32)
        lib, a = load(), ACTIVATIONS[act]
        if ws is None:
            wa = a if want_w else min(a, _lib.ACT_RELU)  # dz's further parts are dw's
            ws = x.new_empty(lib.jenga_linear_bwd_workspace_bytes(M, N, K, wa), dtype=torch.uint8)
        check(lib.jenga_linear_bwd(dy.data_ptr(), ldy, x.data_ptr(), ldx, w.data_ptr(), ldw, a, _ptr(pre), ldp, M, N, K,
                                   _ptr(n_kept), int(blk), _ptr(dx), ldd, _ptr(dw), lddw, _ptr(db), 1 if accumulate else 0,
                                   ws.data_ptr(), ws.numel(), s))
    finally:
        _end(guard)
    return dx, dw, db


def jenga_dropout(x, p, seed, offset=0, residual=None, idx=None, n_kept=None, blk=1, row0=0, out=None, stream=None):
    """y = keep ? x / (1 - p) : 0, plus residual, for x [rows, cols] fp32 / bf16 (compact rows).

    The mask is a function of (seed, offset, sequence position, column) -- recomputed, never
    stored -- with positions row0 + r, or the block list's rows with idx.  The backward is the
    same call on the gradient, without the residual.  out may be x or residual (in place)."""
    guard, s = _begin(stream, x, residual, idx, n_kept, out)
    try:
        ldx = _mat(x, "x")
        rows, cols = x.shape
        if idx is not None or n_kept is not None:
            _rows_arg(idx, n_kept, blk, None, rows)
            if idx is not None and idx.numel() * blk < rows:
                raise ValueError("idx: a list of every row's block required")
        dt = _dt(x)
        ldr = _mat(residual, "residual", cols, rows, x.dtype) if residual is not None else 0
        y = x.new_empty((rows, cols)) if out is None else out
        ldy = cols if out is None else _mat(y, "out", cols, rows, x.dtype)
        m64 = (1 << 64) - 1
        check(load().jenga_dropout(x.data_ptr(), ldx, _ptr(residual), ldr, rows, cols, _ptr(idx), _ptr(n_kept), int(blk),
                                   int(row0), float(p), int(seed) & m64, int(offset) & m64, dt, y.data_ptr(), ldy, s))
    finally:
        _end(guard)
    return y


def jenga_test_gemm(a, b, out_f32=True, bn=256, stream=None):
    """C = A B^T through the tcgen05 GEMM (test hook)."""
    M, K = a.shape
    N = b.shape[0]
    c = torch.empty(M, N, dtype=torch.float32 if out_f32 else torch.bfloat16, device=a.device)
    check(load().jenga_test_gemm(_p(a), a.stride(0), _p(b), b.stride(0), M, N, K, _p(c), c.stride(0),
                                 1 if out_f32 else 0, bn, _stream(stream)))
    return c


def jenga_test_wait_timeout(stream=None):
    """Launch the wait-bound test hook (see include/jenga.h); read the result with
    jenga_check_device_status."""
    check(load().jenga_test_wait_timeout(_stream(stream)))


def jenga_test_exp2(x, stream=None):
    """(2^x by the FMA-pipe exponential, 2^x by ex2.approx) for fp32 device x (test hook)."""
    x = x.contiguous()
    y_fma = torch.empty_like(x)
    y_mufu = torch.empty_like(x)
    check(load().jenga_test_exp2(_p(x), _p(y_fma), _p(y_mufu), x.numel(), _stream(stream)))
    return y_fma, y_mufu
