"""Thin torch-facing binding of the training-step calls around the layer: token embedding,
policy loss and AdamW (the C calls of the same names). The functions check what a tensor's type,
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
