"""Thin torch-facing binding of the training-step calls around the layer: token embedding,
layer norm, choice of experts from scores, policy loss, AdamW and Muon (the C calls of the same names).
The functions check what a tensor's type,
shape and device say, and marshal pointers; nothing is computed here.
"""
import ctypes
import math

import torch

from . import _lib as L
from .layer import MOE_DTYPE, TORCH_DTYPE


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, gpu):
    """The stream's handle. The current one is asked for as a number: a torch.cuda.Stream object for
    each call would take longer (3 us) than the call itself."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(gpu)


def _one_gpu(first, *rest):
    """The GPU that the tensors are on. Refuses others: the kernels would follow a host address."""
    gpu = first.get_device()
    if gpu >= 0:
        for t in rest:
            if t is not None and t.get_device() != gpu:
                break
        else:
            return gpu
    on = sorted({t.get_device() for t in (first, *rest) if t is not None})
    raise ValueError(f"tensors on devices {on} (-1: the host): all have to be on one GPU")


def _arg(what, t, dtype, shape, gpu):
    """The address of a contiguous tensor of this type and shape on GPU `gpu`; others are refused, as the C
    call sees only the address. One pass over what the tensor says: small calls are as long as their checks."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == gpu:
        return t.data_ptr()
    _want(what, t, dtype, shape)
    raise ValueError(f"{what} is on device {t.get_device()}, another tensor on {gpu} (-1: the host): all have to be "
                     "on one GPU")


def _opt(what, t, dtype, shape, gpu):
    return None if t is None else _arg(what, t, dtype, shape, gpu)


def _bytes(what, cfg, gpu, *fields):
    """The C call's answer for this configuration on GPU `gpu` (it depends on its number of SMs), asked for once while
    the fields that it depends on stay."""
    got, key = cfg.__dict__.get("_bytes"), (what, gpu, *fields)
    if got is None or got[0] != key:
        if gpu < 0 or torch._C._cuda_getDevice() == gpu:
            need = getattr(L.load(), what)(ctypes.byref(cfg))
        else:
            with torch.cuda.device(gpu):
                need = getattr(L.load(), what)(ctypes.byref(cfg))
        got = key, int(need)
        if got[1]:                      # 0: the configuration is refused, as the call will be
            cfg._bytes = got
    return got[1]


def _work(ws, need, gpu):
    """The address of a workspace of `need` bytes on GPU `gpu`."""
    if ws is None or ws.nbytes < need or not ws.is_contiguous():
        raise ValueError(f"ws: {need} contiguous bytes are needed")
    if ws.get_device() != gpu:
        raise ValueError(f"ws is on device {ws.get_device()}, other tensors on {gpu}: all have to be on one GPU")
    return ws.data_ptr()


_CALLS = {}


def _launch(what, gpu, stream, *args):
    """One C call on tensors of GPU `gpu`, which need not be the current one."""
    if gpu < 0:
        raise ValueError("tensors on the host: all have to be on one GPU")
    fn = _CALLS.get(what)
    if fn is None:
        fn = _CALLS[what] = getattr(L.load(), what)
    if torch._C._cuda_getDevice() == gpu:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(gpu) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(gpu):
            status = fn(*args, _stream(stream, gpu))
    if status:
        raise L.MoeError(what, status)


def _want(what, t, dtype, shape, optional=False):
    """Refuse a tensor that the call would misread: the C call sees only its address."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{what} is missing")
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: want contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}"
                         f" strides {t.stride()}")


def _room(what, ws, need):
    if ws is None or ws.numel() * ws.element_size() < need or not ws.is_contiguous():
        raise ValueError(f"{what}: {need} contiguous bytes are needed")


_TORCH = {MOE_DTYPE[k]: v for k, v in TORCH_DTYPE.items()}


# ---------------------------------------------------------------- embedding

def make_embed_config(T, V, d, scale=1.0, dtype="bf16", grad_dtype=None, accumulate=False, padding_id=-1):
    """A moe_embed_config_t (the calls check it and raise MoeError). grad_dtype: the type of dW
    (default: the table's)."""
    return L.MoeEmbedConfig(T=T, V=V, d=d, scale=float(scale), padding_id=int(padding_id), dtype=MOE_DTYPE[dtype],
                            grad_dtype=MOE_DTYPE[grad_dtype or dtype], accumulate=int(bool(accumulate)))


def embed(cfg, ids, W, y, stream=None):
    """y [T, d] = scale * W [V, d][ids [T] int32]."""
    dt = _TORCH[cfg.dtype]
    _want("ids", ids, torch.int32, (cfg.T,))
    _want("W", W, dt, (cfg.V, cfg.d))
    _want("y", y, dt, (cfg.T, cfg.d))
    gpu = _one_gpu(W, ids, y)
    L.check("moe_embed", L.load().moe_embed(ctypes.byref(cfg), _ptr(ids), _ptr(W), _ptr(y), _stream(stream, gpu)))


def embed_workspace_bytes(cfg):
    return int(L.load().moe_embed_workspace_bytes(ctypes.byref(cfg)))


def embed_backward(cfg, ids, dy, dW, ws, stream=None):
    """dW [V, d] = (or +=, with cfg.accumulate) scale * the sum of dy [T, d] over the tokens of each id."""
    _want("ids", ids, torch.int32, (cfg.T,))
    _want("dy", dy, _TORCH[cfg.dtype], (cfg.T, cfg.d))
    _want("dW", dW, _TORCH[cfg.grad_dtype], (cfg.V, cfg.d))
    _room("ws", ws, embed_workspace_bytes(cfg))
    gpu = _one_gpu(dW, ids, dy, ws)
    L.check("moe_embed_backward", L.load().moe_embed_backward(
        ctypes.byref(cfg), _ptr(ids), _ptr(dy), _ptr(dW), _ptr(ws), _stream(stream, gpu)))


# ---------------------------------------------------------------- policy loss

def make_policy_config(T, V, dtype="bf16", temperature=1.0, clip_low=0.2, clip_high=0.2, kl_weight=0.0, ld=None,
                       ld_grad=None):
    """A moe_policy_config_t (the calls check it and raise MoeError). ld, ld_grad: elements between
    the rows of logits and dlogits (default: V)."""
    return L.MoePolicyConfig(T=T, V=V, ld=V if ld is None else int(ld), ld_grad=V if ld_grad is None else int(ld_grad),
                             dtype=MOE_DTYPE[dtype], temperature=float(temperature), clip_low=float(clip_low),
                             clip_high=float(clip_high), kl_weight=float(kl_weight))


def policy_workspace_bytes(cfg):
    return int(L.load().moe_policy_workspace_bytes(ctypes.byref(cfg)))


def _rows(what, t, cfg, ld):
    if t.dtype != _TORCH[cfg.dtype] or t.shape != (cfg.T, cfg.V) or \
            (cfg.T > 1 and t.stride(0) != ld) or (cfg.V > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: want {_TORCH[cfg.dtype]} {(cfg.T, cfg.V)} with rows {ld} apart, got {t.dtype} "
                         f"{tuple(t.shape)} strides {t.stride()}")


def policy_loss(cfg, logits, target, advantage, old_logp, ref_logp, weight, logp, loss, dlogits, ws, stream=None):
    """Clipped policy loss with a KL term: logp [T], loss [1] and dlogits [T, V] (each may be None)
    from logits [T, V], target [T] int32 and advantage, old_logp, ref_logp, weight [T] fp32
    (old_logp None: on-policy; ref_logp None without a KL term; weight None: 1). dlogits may be
    logits."""
    _rows("logits", logits, cfg, cfg.ld)
    if dlogits is not None:
        _rows("dlogits", dlogits, cfg, cfg.ld_grad)
    f32, shape = torch.float32, (cfg.T,)
    _want("target", target, torch.int32, shape)
    _want("advantage", advantage, f32, shape)
    _want("old_logp", old_logp, f32, shape, True)
    _want("ref_logp", ref_logp, f32, shape, True)
    _want("weight", weight, f32, shape, True)
    _want("logp", logp, f32, shape, True)
    _want("loss", loss, f32, (1,), True)
    if loss is not None:
        _room("ws", ws, policy_workspace_bytes(cfg))
    gpu = _one_gpu(logits, target, advantage, old_logp, ref_logp, weight, logp, loss, dlogits, ws)
    L.check("moe_policy_loss", L.load().moe_policy_loss(
        ctypes.byref(cfg), _ptr(logits), _ptr(target), _ptr(advantage), _ptr(old_logp), _ptr(ref_logp), _ptr(weight), _ptr(logp),
        _ptr(loss), _ptr(dlogits), _ptr(ws), _stream(stream, gpu)))


def token_logp(cfg, logits, target, logp, stream=None):
    """logp [T] = log softmax(logits [T, V] / temperature)[target [T] int32]."""
    _rows("logits", logits, cfg, cfg.ld)
    _want("target", target, torch.int32, (cfg.T,))
    _want("logp", logp, torch.float32, (cfg.T,))
    gpu = _one_gpu(logits, target, logp)
    L.check("moe_token_logp", L.load().moe_token_logp(ctypes.byref(cfg), _ptr(logits), _ptr(target), _ptr(logp),
                                                           _stream(stream, gpu)))


# ---------------------------------------------------------------- AdamW

_ARRAYS = ("p", "g", "master", "m", "v", "m_scale", "v_scale")
_KIND = {torch.float32: L.MOE_F32, torch.bfloat16: L.MOE_BF16}


class AdamW:
    """moe_adamw over a fixed list of weights. `tensors` is a list of dicts:

      p, g           weights and their gradient (bf16 or fp32, contiguous, the same number of elements)
      master         fp32 copy that the step is taken on, or None
      m, v           states: fp32, or float8_e4m3fn with m_scale and v_scale (fp32, one value to
                     MOE_ADAMW_BLOCK elements); left out, they are made, zeroed, by `bits`
      weight_decay   default: the class's

    rounding: how 8-bit states are rounded, "even" (m and v right on average) or "weyl" (fewer
    instructions, v some per cent high); see MOE_ADAMW_ROUND_*.

    step() takes one step on the current gradients; it may be captured into a CUDA graph, which
    then counts its own steps. The tensors are bound here: refill the gradients in place.
    `step` is the number of steps that the given states have seen."""

    def __init__(self, tensors, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, bits=32, step=0,
                 rounding="even"):
        if bits not in (8, 32):
            raise ValueError("bits: 8 or 32")
        if rounding not in L.MOE_ADAMW_ROUND:
            raise ValueError(f"rounding: one of {sorted(L.MOE_ADAMW_ROUND)}")
        self.cfg = L.MoeAdamwConfig(lr=lr, beta1=beta1, beta2=beta2, eps=eps, rounding=L.MOE_ADAMW_ROUND[rounding])
        self.tensors = [self._bind(dict(t), weight_decay, bits) for t in tensors]
        self.table = (L.MoeAdamwTensor * max(1, len(self.tensors)))()
        for e, t in zip(self.table, self.tensors):
            for k in _ARRAYS:
                setattr(e, k, None if t[k] is None else t[k].data_ptr())
            e.n, e.dtype, e.grad_dtype = t["p"].numel(), _KIND[t["p"].dtype], _KIND[t["g"].dtype]
            e.weight_decay = t["weight_decay"]
        device = self.tensors[0]["p"].device if self.tensors else "cuda"
        at = torch.zeros(L.MOE_ADAMW_STATE_BYTES // 8, dtype=torch.float64)
        if step:
            at[0], at[1] = (-math.expm1(step * math.log(b)) if b else 1.0 for b in (beta1, beta2))
            at.view(torch.int64)[2] = int(step)
        self.state = at.to(device)
        self.placed = False             # whether the bound arrays have been seen to be on one GPU

    @staticmethod
    def _bind(t, weight_decay, bits):
        p, g, n = t["p"], t["g"], t["p"].numel()
        blocks = -(-n // L.MOE_ADAMW_BLOCK)
        for k in ("p", "g"):
            if t[k].dtype not in _KIND:
                raise ValueError(f"{k}: bf16 or fp32, got {t[k].dtype}")
        if g.numel() != n or not p.is_contiguous() or not g.is_contiguous():
            raise ValueError("p and g: contiguous, with as many elements")
        for k in ("master", "m", "v", "m_scale", "v_scale"):
            t.setdefault(k, None)
        if t["m"] is None and t["v"] is None:
            dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
            t["m"], t["v"] = (torch.zeros(n, dtype=dt, device=p.device) for _ in "mv")
            if bits == 8:
                t["m_scale"], t["v_scale"] = (torch.zeros(blocks, dtype=torch.float32, device=p.device) for _ in "mv")
        narrow = t["m_scale"] is not None or t["v_scale"] is not None
        held = torch.float8_e4m3fn if narrow else torch.float32
        for k, dt, size in (("master", torch.float32, n), ("m", held, n), ("v", held, n),
                            ("m_scale", torch.float32, blocks), ("v_scale", torch.float32, blocks)):
            if t[k] is None:
                if k in ("m", "v") or (narrow and k != "master"):
                    raise ValueError(f"{k} is missing")
            elif t[k].dtype != dt or t[k].numel() != size or not t[k].is_contiguous():
                raise ValueError(f"{k}: want {size} contiguous {dt}")
        t["weight_decay"] = float(t.get("weight_decay", weight_decay))
        return t

    def step(self, lr=None, grad_scale=None, stream=None):
        """One step. lr, grad_scale: fp32 device tensors of one element, read when the step runs
        (they replace the class's lr; multiply every gradient)."""
        for what, t in (("lr", lr), ("grad_scale", grad_scale)):
            if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
                raise ValueError(f"{what}: one fp32 element")
        if not self.placed:
            _one_gpu(self.state, *(t[k] for t in self.tensors for k in _ARRAYS))
            self.placed = True
        gpu = _one_gpu(self.state, lr, grad_scale)
        L.check("moe_adamw", L.load().moe_adamw(ctypes.byref(self.cfg), self.table, len(self.tensors), _ptr(lr),
                                                _ptr(grad_scale), _ptr(self.state), _stream(stream, gpu)))

    def steps_done(self):
        """Steps that the device has counted (synchronises)."""
        return int(self.state.view(torch.int64)[2])


# ---------------------------------------------------------------- choice of experts from scores

def make_score_config(T, E, k, score="softmax", groups=1, groups_kept=None, group_top=1, renormalise=True,
                      temperature=1.0, scale=1.0):
    """A moe_score_config_t (the calls check it and raise MoeError). groups_kept: default, all."""
    if score not in L.MOE_SCORE:
        raise ValueError(f"score: one of {sorted(L.MOE_SCORE)}")
    return L.MoeScoreConfig(T=T, E=E, k=k, score=L.MOE_SCORE[score], groups=groups,
                            groups_kept=groups if groups_kept is None else groups_kept, group_top=group_top,
                            renormalise=int(bool(renormalise)), temperature=float(temperature), scale=float(scale))


def route_scores_workspace_bytes(cfg):
    return int(L.load().moe_route_scores_workspace_bytes(ctypes.byref(cfg)))


def route_scores(cfg, logits, bias, idx, w, counts=None, balance_loss=None, ws=None, stream=None):
    """idx [T, k] int32 and w [T, k] fp32 from logits [T, E] fp32 (moe_route's `logits`) and bias [E] fp32
    (or None) by scores, groups and top-k; counts [E] int32 and balance_loss [1] fp32 (each may be None;
    ws is needed for them)."""
    T, E, k, f32, i32, gpu = cfg.T, cfg.E, cfg.k, torch.float32, torch.int32, logits.get_device()
    args = (_arg("logits", logits, f32, (T, E), gpu), _opt("bias", bias, f32, (E,), gpu),
            _arg("idx", idx, i32, (T, k), gpu), _arg("w", w, f32, (T, k), gpu), _opt("counts", counts, i32, (E,), gpu),
            _opt("balance_loss", balance_loss, f32, (1,), gpu))
    tally = counts is not None or balance_loss is not None
    at = _work(ws, _bytes("moe_route_scores_workspace_bytes", cfg, gpu, T, E), gpu) if tally else None
    _launch("moe_route_scores", gpu, stream, ctypes.byref(cfg), *args, at)


def route_scores_backward(cfg, logits, idx, dw, dlogits, stream=None):
    """dlogits [T, E] = the gradient of sum(w * dw) in the logits."""
    T, E, k, f32, gpu = cfg.T, cfg.E, cfg.k, torch.float32, logits.get_device()
    _launch("moe_route_scores_backward", gpu, stream, ctypes.byref(cfg), _arg("logits", logits, f32, (T, E), gpu),
            _arg("idx", idx, torch.int32, (T, k), gpu), _arg("dw", dw, f32, (T, k), gpu),
            _arg("dlogits", dlogits, f32, (T, E), gpu))


# ---------------------------------------------------------------- layer norm

def make_norm_config(T, d, eps=1e-5, dtype="bf16", param_dtype="f32", accumulate=False):
    """A moe_norm_config_t (the calls check it and raise MoeError)."""
    return L.MoeNormConfig(T=T, d=d, eps=float(eps), dtype=MOE_DTYPE[dtype], param_dtype=MOE_DTYPE[param_dtype],
                           accumulate=int(bool(accumulate)))


def norm_workspace_bytes(cfg):
    return int(L.load().moe_norm_workspace_bytes(ctypes.byref(cfg)))


def layer_norm(cfg, x, gain, bias, y, residual=None, total=None, mean=None, rstd=None, stream=None):
    """y [T, d] = the norm of x + residual, total [T, d] = that sum (both or neither of residual and
    total); mean, rstd [T] fp32 for the backward pass; gain, bias [d] may be None."""
    T, d, dt, pt, f32, gpu = cfg.T, cfg.d, _TORCH[cfg.dtype], _TORCH[cfg.param_dtype], torch.float32, x.get_device()
    shape, row, col = (T, d), (d,), (T,)
    both = residual is not None or total is not None
    _launch("moe_layer_norm", gpu, stream, ctypes.byref(cfg), _arg("x", x, dt, shape, gpu),
            _arg("residual", residual, dt, shape, gpu) if both else None, _opt("gain", gain, pt, row, gpu),
            _opt("bias", bias, pt, row, gpu), _arg("total", total, dt, shape, gpu) if both else None,
            _arg("y", y, dt, shape, gpu), _opt("mean", mean, f32, col, gpu), _opt("rstd", rstd, f32, col, gpu))


def layer_norm_backward(cfg, dy, s, gain, mean, rstd, dx, dgain, dbias, ws, dtotal=None, stream=None):
    """dx [T, d] (+ dtotal, the gradient that reaches the sum itself) and dgain, dbias [d] fp32 from dy and
    the forward's s (its total, or x), mean and rstd. dx, dgain and dbias may each be None."""
    T, d, dt, f32, gpu = cfg.T, cfg.d, _TORCH[cfg.dtype], torch.float32, dy.get_device()
    shape, row, col = (T, d), (d,), (T,)
    args = (_arg("dy", dy, dt, shape, gpu), _arg("s", s, dt, shape, gpu),
            _opt("gain", gain, _TORCH[cfg.param_dtype], row, gpu), _arg("mean", mean, f32, col, gpu),
            _arg("rstd", rstd, f32, col, gpu), _opt("dtotal", dtotal, dt, shape, gpu), _opt("dx", dx, dt, shape, gpu),
            _opt("dgain", dgain, f32, row, gpu), _opt("dbias", dbias, f32, row, gpu))
    sums = dgain is not None or dbias is not None
    _launch("moe_layer_norm_backward", gpu, stream, ctypes.byref(cfg), *args,
            _work(ws, _bytes("moe_norm_workspace_bytes", cfg, gpu, T, d, dt), gpu) if sums else None)


# ---------------------------------------------------------------- orthogonalised updates (Muon)

MUON_COEF = (3.4445, -4.7750, 2.0315)


def make_muon_config(count, rows, cols, dtype="bf16", grad_dtype=None, precision=None, steps=5, coef=MUON_COEF,
                     lr=0.02, momentum=0.95, weight_decay=0.0, scale=None, eps=1e-7, nesterov=True):
    """A moe_muon_config_t (the calls check it and raise MoeError) for `count` matrices [rows, cols].
    grad_dtype, precision: default, dtype. scale: default 0.2 sqrt(max(rows, cols)), which makes the
    update's elements 0.2 lr in size."""
    a, b, c = coef
    return L.MoeMuonConfig(count=count, rows=rows, cols=cols, steps=steps, a=a, b=b, c=c, lr=lr, momentum=momentum,
                           weight_decay=weight_decay,
                           scale=0.2 * math.sqrt(max(rows, cols)) if scale is None else scale, eps=eps,
                           nesterov=int(bool(nesterov)), dtype=MOE_DTYPE[dtype], grad_dtype=MOE_DTYPE[grad_dtype or dtype],
                           precision=MOE_DTYPE[precision or dtype])


def muon_workspace_bytes(cfg):
    return int(L.load().moe_muon_workspace_bytes(ctypes.byref(cfg)))


def orthogonalize(cfg, g, o, ws, stream=None):
    """o [count, rows, cols] = g with the singular values of each matrix brought near 1. o may be g."""
    shape, gpu = (cfg.count, cfg.rows, cfg.cols), g.get_device()
    _launch("moe_orthogonalize", gpu, stream, ctypes.byref(cfg), _arg("g", g, _TORCH[cfg.grad_dtype], shape, gpu),
            _arg("o", o, _TORCH[cfg.dtype], shape, gpu), _work(ws, muon_workspace_bytes(cfg), gpu))


class Muon:
    """moe_muon over a list of weight matrices. `tensors` is a list of dicts:

      p, g           weights and their gradient (bf16 or fp32, contiguous): a matrix [rows, cols], or a
                     stack of them [count, rows, cols] (an expert layer's W1 or W2), each on its own
      master         fp32 copy that the step is taken on, or None
      m              momentum, fp32 (left out: made, zeroed)
      weight_decay, scale, precision   default: the class's; scale's is 0.2 sqrt(max(rows, cols)),
                     precision's the weights' own type

    step() takes one step on the current gradients and may be captured into a CUDA graph. The tensors are
    bound here: refill the gradients in place. One workspace serves all of the tensors, one after another,
    so two steps of one Muon must not run at once; two Muons have a workspace each."""

    def __init__(self, tensors, lr=0.02, momentum=0.95, weight_decay=0.0, nesterov=True, steps=5, coef=MUON_COEF,
                 eps=1e-7, scale=None, precision=None):
        self.tensors = []
        need, device = 0, "cpu"
        for t in tensors:
            t = dict(t)
            p, g = t["p"], t["g"]
            for k in ("p", "g"):
                if t[k].dtype not in _KIND:
                    raise ValueError(f"{k}: bf16 or fp32, got {t[k].dtype}")
            if p.dim() not in (2, 3) or g.shape != p.shape or not p.is_contiguous() or not g.is_contiguous():
                raise ValueError("p and g: contiguous, of one shape [rows, cols] or [count, rows, cols]")
            if t.get("m") is None:
                t["m"] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
            for k in ("m", "master"):
                t.setdefault(k, None)
                if t[k] is not None and (t[k].dtype != torch.float32 or t[k].shape != p.shape or
                                         not t[k].is_contiguous()):
                    raise ValueError(f"{k}: want contiguous torch.float32 {tuple(p.shape)}")
            rows, cols = p.shape[-2:]
            count = p.shape[0] if p.dim() == 3 else 1
            cfg = make_muon_config(count, rows, cols, steps=steps, coef=coef, lr=lr, momentum=momentum, eps=eps,
                                   nesterov=nesterov, weight_decay=float(t.get("weight_decay", weight_decay)),
                                   scale=t.get("scale", scale))
            cfg.dtype, cfg.grad_dtype = _KIND[p.dtype], _KIND[g.dtype]
            own = t.get("precision", precision)
            cfg.precision = cfg.dtype if own is None else MOE_DTYPE[own]
            t["cfg"] = cfg
            if count > 0:
                size = muon_workspace_bytes(cfg)
                if size == 0:               # refused: the call says why
                    L.check("moe_muon", L.load().moe_muon(ctypes.byref(cfg), *[None] * 8))
                need, device = max(need, size), p.device
            self.tensors.append(t)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device)
        self.placed = None              # the GPU that the bound arrays have been seen to be on

    def step(self, lr=None, grad_scale=None, stream=None):
        """One step. lr, grad_scale: fp32 device tensors of one element, read when the step runs (they
        replace the class's lr; multiply every gradient)."""
        for what, t in (("lr", lr), ("grad_scale", grad_scale)):
            if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
                raise ValueError(f"{what}: one fp32 element")
        if not self.ws.numel():
            return                      # nothing but empty stacks
        if self.placed is None:
            bound = [t[k] for t in self.tensors for k in ("p", "g", "m", "master")]
            gpu = _one_gpu(self.ws, *bound)
            if any(t is not None and t.data_ptr() % 16 for t in bound):      # (before the first tensor is stepped)
                raise ValueError("p, g, m and master start on 16-byte boundaries")
            self.placed = gpu
        gpu = _one_gpu(self.ws, lr, grad_scale)
        for t in self.tensors:
            _launch("moe_muon", gpu, stream, ctypes.byref(t["cfg"]), _ptr(t["p"]), _ptr(t["g"]),
                    _ptr(t["master"]), _ptr(t["m"]), _ptr(lr), _ptr(grad_scale), _ptr(self.ws))
