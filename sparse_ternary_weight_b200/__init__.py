"""Sherry 3:4-sparse ternary (1.25-bit) weights on B200: quantise+pack, packed
linear and unpack, every step in the CUDA library ``libsherry.so``.

This module only marshals arguments: torch supplies device memory and the
current stream, and each call goes straight to one C-ABI entry point
(include/sherry.h).  There is no CPU or PyTorch fallback: if the library is
missing or the tensors are not on a CUDA device, the calls raise.
"""
from __future__ import annotations

import ctypes
from contextlib import nullcontext
from dataclasses import dataclass

from . import _abi
from ._abi import (BF16, F32, PER_CHANNEL, PER_GROUP, PER_TENSOR, SherryError,  # noqa: F401
                   check, lib)

GRANULARITY = {"per_tensor": PER_TENSOR, "per_channel": PER_CHANNEL, "per_group": PER_GROUP}


def _gran(g) -> int:
    if isinstance(g, str):
        if g not in GRANULARITY:
            raise ValueError(f"unsupported granularity {g!r}")
        return GRANULARITY[g]
    return int(g)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device=None) -> int:
    """Handle of the current stream of ``device`` (as torch.cuda.current_stream, without
    the object around it, which costs more than a launch's arguments)."""
    import torch
    index = None if device is None else device.index
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


_NO_GUARD = nullcontext()


def _on(device):
    """A guard that makes ``device`` current; nothing where it is."""
    import torch
    return _NO_GUARD if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on a CUDA device (no CPU fallback)")


@dataclass
class PackedWeight:
    """Packed planes of one [N,K] weight: idx uint32 [N,K/32] (stored as int32),
    sgn uint8 [N,K/32], scales float32, plus the scale granularity."""
    idx: "object"
    sgn: "object"
    scales: "object"
    N: int
    K: int
    granularity: int
    group: int

    def nbytes(self) -> int:
        return self.idx.numel() * 4 + self.sgn.numel() + self.scales.numel() * 4


_ws_cache: dict = {}
_ws_timeouts = [0]  # the library's timeout count when the cached buffers were last known clean


def workspace(nbytes: int, device, kind: str = "linear") -> "object":
    """A device scratch buffer of at least ``nbytes``, cached per (device, kind).
    ``kind="linear"`` buffers are zero-filled when allocated and used by the
    linear calls only: their split-K ticket counters must start at zero, and
    every successful call leaves them at zero.  Other kinds hold scratch that
    the next call overwrites.  Once any bounded device wait has been reported
    as given up (sherry_device_status, by whichever caller), every cached
    buffer is dropped: a timed-out kernel may have left tickets nonzero."""
    import torch
    if nbytes <= 0:
        return None
    seen = lib().sherry_timeout_count()
    if seen != _ws_timeouts[0]:
        _ws_cache.clear()
        _ws_timeouts[0] = seen
    key = (str(device), kind)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 1 << 16), dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


def device_status(device=None) -> int:
    """Synchronise the current stream of ``device`` and return the library's
    device status (0, or ERR_TIMEOUT when a bounded wait of a kernel gave up
    since the last query).  After a timeout the cached workspaces may hold
    nonzero split-K tickets; the next workspace request drops them (the
    library counts every nonzero status it reports)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return lib().sherry_device_status(_stream(dev))


def quantize_pack(W, granularity="per_group", group: int = 128, out: PackedWeight | None = None) -> PackedWeight:
    """Greedy Sparse-AbsMean 3:4 quantise + 5-bit pack of W [N,K] (fp32 or bf16)."""
    import torch
    _require_cuda(W)
    if W.dim() != 2:
        raise ValueError("expects a 2D weight")
    W = W.contiguous()
    N, K = W.shape
    g = _gran(granularity)
    L = lib()
    ns = L.sherry_num_scales(N, K, g, group)
    if ns < 0:
        raise SherryError(_abi.ERR_SHAPE if K % 32 or K < 32 else _abi.ERR_GROUP, "quantize_pack")
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(W.dtype)
    if dt is None:
        raise SherryError(_abi.ERR_DTYPE, "quantize_pack")
    if out is None:
        out = _new_packed(N, K, g, group, ns, W.device)
    wsb = L.sherry_workspace_bytes(_abi.OP_QUANTIZE_PACK, 0, N, K, g, group)
    ws = workspace(wsb, W.device, "quantize")
    check(L.sherry_quantize_pack(_ptr(W), dt, N, K, g, group, _ptr(out.idx), _ptr(out.sgn), _ptr(out.scales),
                                 _ptr(ws), wsb, _stream(W.device)), "quantize_pack")
    return out


def _new_packed(N, K, g, group, ns, dev) -> PackedWeight:
    import torch
    return PackedWeight(torch.empty((N, K // 32), dtype=torch.int32, device=dev),
                        torch.empty((N, K // 32), dtype=torch.uint8, device=dev),
                        torch.empty((max(ns, 1),), dtype=torch.float32, device=dev), N, K, g, group)


def fake_quant(W, granularity="per_group", group: int = 128, out_dtype=None, out=None,
               packed: PackedWeight | None = None):
    """The quantiser's forward output W_q = t * alpha [N,K] (fp32 or bf16, default
    W's dtype) in one pass over W, plus the packed weight.  Returns (W_q, packed)."""
    import torch
    _require_cuda(W)
    if W.dim() != 2:
        raise ValueError("expects a 2D weight")
    W = W.contiguous()
    N, K = W.shape
    g = _gran(granularity)
    L = lib()
    ns = L.sherry_num_scales(N, K, g, group)
    if ns < 0:
        raise SherryError(_abi.ERR_SHAPE if K % 32 or K < 32 else _abi.ERR_GROUP, "fake_quant")
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(W.dtype)
    if dt is None:
        raise SherryError(_abi.ERR_DTYPE, "fake_quant")
    out_dtype = out_dtype or W.dtype
    qd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        out = torch.empty((N, K), dtype=out_dtype, device=W.device)
    if packed is None:
        packed = _new_packed(N, K, g, group, ns, W.device)
    wsb = L.sherry_workspace_bytes(_abi.OP_QUANTIZE_PACK, 0, N, K, g, group)
    ws = workspace(wsb, W.device, "quantize")
    check(L.sherry_fake_quant(_ptr(W), dt, N, K, g, group, _ptr(out), qd, _ptr(packed.idx), _ptr(packed.sgn),
                              _ptr(packed.scales), _ptr(ws), wsb, _stream(W.device)), "fake_quant")
    return out, packed


def _ste_function():
    import torch

    class SherryFakeQuant(torch.autograd.Function):
        """Fake quantisation with the straight-through estimator: the forward is
        :func:`fake_quant` (one kernel), the backward passes the incoming gradient
        to W unchanged ("Sherry, Tequila and Fairies in Python", section 1.1:
        SherryNMQuant.backward returns grad_output) -- no kernel and no copy."""

        @staticmethod
        def forward(ctx, W, granularity, group):
            return fake_quant(W, granularity, group)[0]

        @staticmethod
        def backward(ctx, grad):
            return grad, None, None

    return SherryFakeQuant


_STE = None


def fake_quant_ste(W, granularity="per_group", group: int = 128):
    """Differentiable fake quantisation for QAT: W_q from the CUDA kernel, identity gradient."""
    global _STE
    if _STE is None:
        _STE = _ste_function()
    return _STE.apply(W, granularity, group)


def quantize_pack_batched(weights, granularity="per_group", group: int = 128, outs=None, wq_outs=None):
    """Quantise + pack several weights in one launch (plus one scale-finalise launch
    when any scale is per-tensor).  ``weights`` is a list of 2D fp32/bf16 tensors;
    ``wq_outs`` (optional) a list of fake-quantised outputs (or None entries)."""
    import torch
    if not weights:
        return []
    g = _gran(granularity)
    L = lib()
    dev = weights[0].device
    arr = (_abi.QuantizeDesc * len(weights))()
    packs = []
    for i, W in enumerate(weights):
        _require_cuda(W)
        if W.dim() != 2 or not W.is_contiguous():
            raise ValueError("each weight must be a contiguous 2D tensor")
        N, K = W.shape
        ns = L.sherry_num_scales(N, K, g, group)
        if ns < 0:
            raise SherryError(_abi.ERR_SHAPE if K % 32 or K < 32 else _abi.ERR_GROUP, "quantize_pack_batched")
        P = outs[i] if outs is not None else _new_packed(N, K, g, group, ns, W.device)
        packs.append(P)
        wq = wq_outs[i] if wq_outs is not None else None
        arr[i] = _abi.QuantizeDesc(_ptr(W), _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), _ptr(wq), N, K,
                                   {torch.float32: F32, torch.bfloat16: BF16}[W.dtype], g, group,
                                   BF16 if (wq is not None and wq.dtype == torch.bfloat16) else F32)
    wsb = L.sherry_quantize_pack_batched_workspace_bytes(arr, len(weights))
    ws = workspace(wsb, dev, "quantize")
    check(L.sherry_quantize_pack_batched(arr, len(weights), _ptr(ws), wsb, _stream(dev)), "quantize_pack_batched")
    return packs


def linear(X, P: PackedWeight, out_dtype=None, out=None):
    """Y [M,N] = X [M,K] (bf16) times the packed weight transposed; fp32 or bf16 Y."""
    import torch
    _require_cuda(X)
    if X.dtype != torch.bfloat16 or X.dim() != 2:
        raise ValueError("X must be a 2D bf16 tensor")
    X = X.contiguous()
    M, K = X.shape
    if K != P.K:
        raise ValueError("inner dimensions differ")
    out_dtype = out_dtype or torch.float32
    yd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        out = torch.empty((M, P.N), dtype=out_dtype, device=X.device)
    L = lib()
    wsb = L.sherry_workspace_bytes(_abi.OP_LINEAR, M, P.N, K, P.granularity, P.group)
    ws = workspace(wsb, X.device)
    check(L.sherry_linear(_ptr(X), M, P.N, K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.granularity, P.group,
                          _ptr(out), yd, _ptr(ws), wsb, _stream(X.device)), "linear")
    return out


def make_batch(pairs, outs) -> "ctypes.Array":
    """Descriptor array for :func:`linear_batched` from (X, PackedWeight) pairs."""
    arr = (_abi.LinearDesc * len(pairs))()
    for i, ((X, P), Y) in enumerate(zip(pairs, outs)):
        arr[i] = _abi.LinearDesc(_ptr(X), _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), _ptr(Y), P.N, P.K,
                                 P.granularity, P.group)
    return arr


def linear_batched(pairs, out_dtype=None, outs=None, descs=None):
    """Independent linears with the same M in one call (one launch per kernel used)."""
    import torch
    out_dtype = out_dtype or torch.float32
    yd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if not pairs:
        return []
    M = pairs[0][0].shape[0]
    for X, P in pairs:
        _require_cuda(X)
        if X.dtype != torch.bfloat16 or X.shape[0] != M or X.shape[1] != P.K or not X.is_contiguous():
            raise ValueError("each X must be contiguous bf16 [M,K] with the same M")
    if outs is None:
        outs = [torch.empty((M, P.N), dtype=out_dtype, device=X.device) for X, P in pairs]
    if descs is None:
        descs = make_batch(pairs, outs)
    L = lib()
    wsb = L.sherry_linear_batched_workspace_bytes(descs, len(pairs), M)
    ws = workspace(wsb, pairs[0][0].device)
    check(L.sherry_linear_batched(descs, len(pairs), M, yd, _ptr(ws), wsb, _stream(pairs[0][0].device)),
          "linear_batched")
    return outs


def quantize_pack_tequila(W, granularity="per_group", group: int = 128, eps: float = 1e-5):
    """Quantise + pack as :func:`quantize_pack` and, in the same pass over W, the
    Tequila-style dead-weight plane D (bf16 [N, K/4]: eps * the zeroed weight of
    each block) and its row sums (fp32 [N]).  Returns (packed, D, bias)."""
    import torch
    _require_cuda(W)
    if W.dim() != 2:
        raise ValueError("expects a 2D weight")
    W = W.contiguous()
    N, K = W.shape
    g = _gran(granularity)
    L = lib()
    ns = L.sherry_num_scales(N, K, g, group)
    if ns < 0:
        raise SherryError(_abi.ERR_SHAPE if K % 32 or K < 32 else _abi.ERR_GROUP, "quantize_pack_tequila")
    dt = {torch.float32: F32, torch.bfloat16: BF16}.get(W.dtype)
    if dt is None:
        raise SherryError(_abi.ERR_DTYPE, "quantize_pack_tequila")
    P = _new_packed(N, K, g, group, ns, W.device)
    D = torch.empty((N, K // 4), dtype=torch.bfloat16, device=W.device)
    bias = torch.empty((N,), dtype=torch.float32, device=W.device)
    wsb = L.sherry_workspace_bytes(_abi.OP_QUANTIZE_PACK, 0, N, K, g, group)
    ws = workspace(wsb, W.device, "quantize")
    check(L.sherry_quantize_pack_tequila(_ptr(W), dt, N, K, g, group, float(eps), _ptr(P.idx), _ptr(P.sgn),
                                         _ptr(P.scales), _ptr(D), _ptr(bias), _ptr(ws), wsb, _stream(W.device)),
          "quantize_pack_tequila")
    return P, D, bias


def linear_tequila(X, P: PackedWeight, D, bias, mode="sign", out_dtype=None, out=None):
    """Y = X (T alpha)^T + the dead-weight term: ``mode="ones"`` adds bias[n],
    ``mode="sign"`` adds sign(X) D^T."""
    import torch
    _require_cuda(X)
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != P.K:
        raise ValueError("X must be a 2D bf16 tensor [M, K]")
    X = X.contiguous()
    M, K = X.shape
    md = {"ones": _abi.TEQUILA_ONES, "sign": _abi.TEQUILA_SIGN}[mode]
    out_dtype = out_dtype or torch.float32
    yd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        out = torch.empty((M, P.N), dtype=out_dtype, device=X.device)
    L = lib()
    wsb = L.sherry_linear_tequila_workspace_bytes(M, P.N, K, P.granularity, P.group, yd)
    ws = workspace(wsb, X.device)
    check(L.sherry_linear_tequila(_ptr(X), M, P.N, K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.granularity,
                                  P.group, _ptr(D), _ptr(bias), md, _ptr(out), yd, _ptr(ws), wsb, _stream(X.device)),
          "linear_tequila")
    return out


def arenas_lambda(step: int, total: int, lambda0: float) -> float:
    """Cosine-decayed weight of the Arenas residual: lambda0 (1 + cos(pi t / T)) / 2."""
    return float(lib().sherry_arenas_lambda(int(step), int(total), float(lambda0)))


def arenas_linear(X, P: PackedWeight, Wd, lam: float, out_dtype=None, out=None):
    """Arenas training linear Y = X (T alpha)^T + lam X Wd^T in one tensor-core
    kernel (Wd: the latent weight, bf16 [N, K])."""
    import torch
    _require_cuda(X, Wd)
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != P.K:
        raise ValueError("X must be a 2D bf16 tensor [M, K]")
    if Wd.dtype != torch.bfloat16 or tuple(Wd.shape) != (P.N, P.K):
        raise ValueError("Wd must be bf16 [N, K]")
    X = X.contiguous()
    Wd = Wd.contiguous()
    M = X.shape[0]
    out_dtype = out_dtype or torch.float32
    yd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        out = torch.empty((M, P.N), dtype=out_dtype, device=X.device)
    check(lib().sherry_arenas_linear(_ptr(X), M, P.N, P.K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.granularity,
                                     P.group, _ptr(Wd), float(lam), _ptr(out), yd, _stream(X.device)), "arenas_linear")
    return out


def linear_chain(phases, out_dtype=None, descs=None):
    """Chained linears: ``phases`` is a list of phases, each a list of (X, P, Y)
    triples (X bf16 [M,K], Y [M,N] preallocated).  Every linear of a phase starts
    after every linear of the previous phase has written its Y, so an X may be
    (a view of) an earlier phase's Y.  Returns the list of Y per phase."""
    import torch
    out_dtype = out_dtype or torch.float32
    yd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    flat = [t for ph in phases for t in ph]
    if not flat:
        return []
    M = flat[0][0].shape[0]
    for X, P, Y in flat:
        _require_cuda(X, Y)
        if X.dtype != torch.bfloat16 or X.shape != (M, P.K) or not X.is_contiguous():
            raise ValueError("each X must be contiguous bf16 [M,K] with the same M")
        if Y.dtype != out_dtype or Y.shape != (M, P.N) or not Y.is_contiguous():
            raise ValueError("each Y must be contiguous [M,N] of out_dtype")
    if descs is None:
        descs = make_batch([(X, P) for X, P, _ in flat], [Y for _, _, Y in flat])
    begin = [0]
    for ph in phases:
        begin.append(begin[-1] + len(ph))
    pb = (ctypes.c_int * len(begin))(*begin)
    L = lib()
    wsb = L.sherry_linear_chain_workspace_bytes(descs, len(flat), pb, len(phases), M)
    ws = workspace(wsb, flat[0][0].device)
    check(L.sherry_linear_chain(descs, len(flat), pb, len(phases), M, yd, _ptr(ws), wsb, _stream(flat[0][0].device)),
          "linear_chain")
    return [[Y for _, _, Y in ph] for ph in phases]


def quantize_pack_fused(weights, granularity="per_group", group: int = 128) -> PackedWeight:
    """One packed weight whose rows are the rows of ``weights`` in order (e.g. the
    q, k and v projections, or gate and up, of a decoder layer), so that one
    linear call computes all of them.  The planes and the group or row scales of
    each part are exactly those of packing it alone (they depend on its own rows
    only); per-tensor scales are per part and cannot share one packed weight."""
    import torch
    g = _gran(granularity)
    if g == PER_TENSOR:
        raise ValueError("per-tensor scales are one per weight: pack the parts separately")
    K = weights[0].shape[1]
    if any(W.dim() != 2 or W.shape[1] != K for W in weights):
        raise ValueError("every part must be 2D with the same K")
    N = sum(W.shape[0] for W in weights)
    L = lib()
    ns = L.sherry_num_scales(N, K, g, group)
    if ns < 0:
        raise SherryError(_abi.ERR_SHAPE if K % 32 or K < 32 else _abi.ERR_GROUP, "quantize_pack_fused")
    fused = _new_packed(N, K, g, group, ns, weights[0].device)
    spr = ns // N  # scales per row
    r0 = 0
    parts = []
    for W in weights:
        n = W.shape[0]
        parts.append(PackedWeight(fused.idx[r0:r0 + n], fused.sgn[r0:r0 + n], fused.scales[r0 * spr:(r0 + n) * spr],
                                  n, K, g, group))
        r0 += n
    quantize_pack_batched([W.contiguous() for W in weights], g, group, outs=parts)
    return fused


def unpack_batched(packs, outs=None):
    """Dense bf16 of several packed weights in one launch (each as by :func:`unpack`)."""
    import torch
    if not packs:
        return []
    if outs is None:
        outs = [torch.empty((P.N, P.K), dtype=torch.bfloat16, device=P.idx.device) for P in packs]
    arr = (_abi.UnpackDesc * len(packs))()
    for i, (P, o) in enumerate(zip(packs, outs)):
        _require_cuda(P.idx, o)
        arr[i] = _abi.UnpackDesc(_ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.N, P.K, P.granularity, P.group,
                                 _ptr(o))
    check(lib().sherry_unpack_batched(arr, len(packs), _stream(packs[0].idx.device)), "unpack_batched")
    return outs


def unpack(P: PackedWeight, out=None):
    """Dense bf16 [N,K] = RNE(t * alpha)."""
    import torch
    if out is None:
        out = torch.empty((P.N, P.K), dtype=torch.bfloat16, device=P.idx.device)
    check(lib().sherry_unpack(_ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.N, P.K, P.granularity, P.group,
                              _ptr(out), _stream(P.idx.device)), "unpack")
    return out


# ---- adapters and the input gradient -------------------------------------------------------------------

_KEPT_BYTES = 4 << 20


def _stream_workspace(nbytes: int, device) -> "object":
    """A linear workspace (tickets zero) for a call on the current stream of ``device``.
    Calls on different streams may overlap, so each stream keeps its own of up to 4 MB, which
    saves a decode step the zeroing.  A larger one, mostly a chunk's logits or an fp32 Y, is the
    call's own and goes back to the allocator; so is one under graph capture, since a graph may
    be replayed beside other graphs and eager calls."""
    import torch
    if nbytes > _KEPT_BYTES or torch.cuda.is_current_stream_capturing():
        buf = torch.empty(nbytes, dtype=torch.uint8, device=device)
        buf[:_abi.TICKET_BYTES].zero_()
        return buf
    key = (device, "linear", _stream(device))
    seen = lib().sherry_timeout_count()
    if seen != _ws_timeouts[0]:
        _ws_cache.clear()
        _ws_timeouts[0] = seen
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(nbytes, dtype=torch.uint8, device=device)
        _ws_cache[key] = buf
    return buf


_native = [None]


def _calls():
    """The compiled form of the ordinary calls (csrc/binding.cpp): contiguous tensors of the
    right types on the current device.  Its functions return None for any other call,
    which the wrappers then convert or refuse themselves, and an int for a status."""
    if _native[0] is None:
        lib()  # a missing library is reported in its own words
        try:
            from . import _binding as module
        except ImportError as e:
            raise RuntimeError("_binding.so is missing or was built for another torch; build it with "
                               "`python -m sparse_ternary_weight_b200.build`") from e
        _native[0] = module
    return _native[0]


def _done(r, what):
    """What the binding returned, unless that is the status of a refused call."""
    if type(r) is int:
        check(r, what)
    return r


def _scratch(nbytes: int, device) -> "object":
    """Uninitialised scratch of one call, from torch's stream-ordered allocator."""
    import torch
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None


def _same_device(device, *ts):
    for t in ts:
        if t is not None and t.device != device:
            raise ValueError("tensors must be on one CUDA device")


def _planes(P, device):
    """Refuses planes that are not what P's shape and granularity say: the kernels index them by those."""
    import torch
    words = P.N * (P.K // 32)
    scales = lib().sherry_num_scales(P.N, P.K, P.granularity, P.group) if P.N else 0  # (below 0: the call reports why)
    for t, dtypes, count, name in ((P.idx, (torch.int32, torch.uint32), words, "idx"), (P.sgn, (torch.uint8,), words, "sgn"),
                                   (P.scales, (torch.float32,), scales, "scales")):
        if t.device != device:
            raise ValueError("tensors must be on one CUDA device")
        if t.dtype not in dtypes or not t.is_contiguous() or t.numel() < count or (name != "scales" and t.numel() != count):
            raise ValueError(f"{name} of a packed [{P.N}, {P.K}] weight must be {count} contiguous elements of "
                             f"{' or '.join(str(d) for d in dtypes)}")


def _activations(X, K, what="X"):
    import torch
    _require_cuda(X)
    if X.dtype != torch.bfloat16 or X.dim() != 2 or X.shape[1] != K:
        raise ValueError(f"{what} must be a 2D bf16 tensor with {K} columns")
    return X.contiguous()


def _output_gradient(dY, N):
    """dY as the kernels take it: rows of a batch whose rows are not a multiple of 16 bytes may start
    anywhere (a slice, a split's share of a gradient), and are then copied."""
    dY = _activations(dY, N, "dY")
    return dY.clone() if dY.data_ptr() % 16 else dY


def _adapters(X, P, A, B, ids, scaling):
    """Checked and contiguous (A, B, ids, scaling, n_adapters, rank)."""
    import torch
    _require_cuda(A, B, ids, scaling)
    _planes(P, X.device)
    _same_device(X.device, A, B, ids, scaling)
    if A.dtype != torch.bfloat16 or A.dim() != 3 or A.shape[2] != P.K:
        raise ValueError("A must be bf16 [n_adapters, rank, K]")
    n, R = A.shape[0], A.shape[1]
    if B.dtype != torch.bfloat16 or tuple(B.shape) != (n, P.N, R):
        raise ValueError("B must be bf16 [n_adapters, N, rank]")
    if not 1 <= n <= _abi.MAX_ADAPTERS:
        raise ValueError(f"1 to {_abi.MAX_ADAPTERS} adapters per call")
    if R % 8 or not 8 <= R <= _abi.MAX_RANK:
        raise ValueError(f"the rank must be a multiple of 8 up to {_abi.MAX_RANK} (pad with zeros)")
    if ids.dtype not in (torch.int32, torch.int64) or tuple(ids.shape) != (X.shape[0],):
        raise ValueError("ids must be int32 or int64 [M]")
    if scaling is not None and (scaling.dtype != torch.float32 or tuple(scaling.shape) != (n,)):
        raise ValueError("scaling must be fp32 [n_adapters]")
    if ids.dtype == torch.int64:  # a value int32 cannot hold names no adapter
        ids = ids.clamp(-1, n).to(torch.int32)
    return (A.contiguous(), B.contiguous(), ids.contiguous(), None if scaling is None else scaling.contiguous(), n, R)


def _result(out, shape, dtype, device, *inputs):
    """``out`` checked, or a new tensor; the kernels read ``inputs`` while they write it."""
    import torch
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if out.dtype != dtype or tuple(out.shape) != tuple(shape) or not out.is_contiguous() or out.device != device:
        raise ValueError(f"out must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    for t in inputs:
        if t is not None and out.numel() and t.numel() and _spans_overlap(out.view(1, -1), t.view(1, -1)):
            raise ValueError("out must not overlap what the call reads")
    return out


def linear_lora(X, P: PackedWeight, A, B, ids, scaling=None, out_dtype=None, out=None, return_u: bool = False):
    """The packed linear with a low-rank adapter per token: Y[m] = X[m] (T alpha)^T +
    U[m] B_a^T with U[m] = scaling[a] X[m] A_a^T and a = ids[m].  A is bf16
    [n_adapters, rank, K], B bf16 [n_adapters, N, rank] (rank a multiple of 8), ids
    int32 or int64 [M] in any order (a value outside [0, n_adapters): no adapter),
    scaling fp32 [n_adapters] or None for 1.  With ``return_u`` returns (Y, U), U fp32
    [M, rank], which :func:`linear_lora_backward` takes."""
    import torch
    out_dtype = out_dtype or torch.float32
    yd = {torch.float32: F32, torch.bfloat16: BF16}[out_dtype]
    if out is None:
        r = _done(_calls().linear_lora(X, P.idx, P.sgn, P.scales, P.N, P.K, P.granularity, P.group, A, B, ids, scaling,
                                         yd, return_u), "linear_lora")
        if r is not None:
            return r if return_u else r[0]
    X = _activations(X, P.K)
    A, B, ids, scaling, n, R = _adapters(X, P, A, B, ids, scaling)
    M = X.shape[0]
    out = _result(out, (M, P.N), out_dtype, X.device, X, A, B, ids, scaling, P.idx, P.sgn, P.scales)
    U = torch.empty((M, R), dtype=torch.float32, device=X.device) if return_u else None
    with _on(X.device):
        L = lib()
        wsb = L.sherry_linear_lora_workspace_bytes(M, P.N, P.K, P.granularity, P.group, n, R, yd)
        tickets = wsb and L.sherry_linear_lora_needs_tickets(M, P.N, P.K, P.granularity, P.group)
        ws = _stream_workspace(wsb, X.device) if tickets else _scratch(wsb, X.device)
        check(L.sherry_linear_lora(_ptr(X), M, P.N, P.K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.granularity,
                                   P.group, _ptr(A), _ptr(B), _ptr(ids), _ptr(scaling), n, R, _ptr(U), _ptr(out), yd,
                                   _ptr(ws), wsb, _stream(X.device)), "linear_lora")
    return (out, U) if return_u else out


def linear_backward(dY, P: PackedWeight, out=None):
    """Input gradient of the packed linear: dX [M,K] = dY [M,N] (T alpha), bf16."""
    import torch
    dY = _output_gradient(dY, P.N)
    _planes(P, dY.device)
    M = dY.shape[0]
    out = _result(out, (M, P.K), torch.bfloat16, dY.device, dY, P.idx, P.sgn, P.scales)
    with _on(dY.device):
        L = lib()
        wsb = L.sherry_linear_backward_workspace_bytes(M, P.N, P.K)
        ws = _scratch(wsb, dY.device)
        check(L.sherry_linear_backward(_ptr(dY), M, P.N, P.K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.granularity,
                                       P.group, _ptr(out), _ptr(ws), wsb, _stream(dY.device)), "linear_backward")
    return out


def linear_lora_backward(dY, X, P: PackedWeight, A, B, ids, U, scaling=None, grad_dtype=None,
                         need=(True, True, True)):
    """Gradients of :func:`linear_lora`: (dX bf16 [M,K], dA, dB) from dY (bf16 [M,N]) and
    the U that the forward call returned; dA and dB are sums over each adapter's
    tokens in ``grad_dtype`` (bf16, the default, or fp32).  ``need`` leaves out the
    gradients that are not wanted (None in their place)."""
    import torch
    grad_dtype = grad_dtype or torch.bfloat16
    gd = {torch.float32: F32, torch.bfloat16: BF16}[grad_dtype]
    r = _done(_calls().linear_lora_backward(dY, X, P.idx, P.sgn, P.scales, P.N, P.K, P.granularity, P.group, A, B, ids,
                                              scaling, U, gd, bool(need[0]) + 2 * bool(need[1]) + 4 * bool(need[2])),
              "linear_lora_backward")
    if r is not None:
        return r
    dY = _output_gradient(dY, P.N)
    X = _activations(X, P.K)
    M = X.shape[0]
    if dY.shape[0] != M:
        raise ValueError("dY and X must have the same number of rows")
    A, B, ids, scaling, n, R = _adapters(X, P, A, B, ids, scaling)
    _same_device(X.device, dY, U)
    if U is not None and (U.dtype != torch.float32 or tuple(U.shape) != (M, R)):
        raise ValueError("U must be fp32 [M, rank]")
    if need[2] and U is None:
        raise ValueError("dB needs U of the forward pass")
    U = None if U is None else U.contiguous()
    dX = torch.empty_like(X) if need[0] else None
    dA = torch.empty_like(A, dtype=grad_dtype) if need[1] else None
    dB = torch.empty_like(B, dtype=grad_dtype) if need[2] else None
    with _on(X.device):
        L = lib()
        wsb = L.sherry_linear_lora_backward_workspace_bytes(M, P.N, P.K, n, R)
        ws = _scratch(wsb, X.device)
        check(L.sherry_linear_lora_backward(_ptr(dY), _ptr(X), M, P.N, P.K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales),
                                            P.granularity, P.group, _ptr(A), _ptr(B), _ptr(ids), _ptr(scaling), n, R,
                                            _ptr(U), _ptr(dX), _ptr(dA), _ptr(dB), gd, _ptr(ws), wsb,
                                            _stream(X.device)), "linear_lora_backward")
    return dX, dA, dB


def _refuse_capture(what, explicit):
    """Autograd's accumulation of a leaf's gradient runs on the stream where an earlier
    graph of the same leaf was built; under capture that ends the capture, and the
    process with it.  So the differentiable forms are not captured, neither forward nor
    the backward pass of an eager call."""
    import torch
    if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
        raise RuntimeError(f"{what} cannot be captured into a CUDA graph: capture {explicit}")


def _lora_function():
    import torch

    class SherryLinearLora(torch.autograd.Function):
        """:func:`linear_lora` with :func:`linear_lora_backward`; the packed weight and
        the scaling are constants."""

        @staticmethod
        def forward(ctx, X, A, B, P, ids, scaling, out_dtype):
            Y, U = linear_lora(X, P, A, B, ids, scaling, out_dtype, return_u=True)
            ctx.save_for_backward(X, A, B, ids, scaling, U)
            ctx.packed = P
            return Y

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dY):
            _refuse_capture("the backward pass of linear_lora_train", "linear_lora_backward")
            X, A, B, ids, scaling, U = ctx.saved_tensors
            need = ctx.needs_input_grad[:3]
            dX, dA, dB = linear_lora_backward(dY.to(torch.bfloat16), X, ctx.packed, A, B, ids, U, scaling, need=need)
            return dX, dA, dB, None, None, None, None

    return SherryLinearLora


_LORA = None


def linear_lora_train(X, P: PackedWeight, A, B, ids, scaling=None, out_dtype=None):
    """Differentiable :func:`linear_lora`: gradients reach X, A and B (bf16, as the
    tensors); the packed weight is frozen and ``scaling`` a constant.  An fp32 gradient
    of Y is rounded to the bf16 that the tensor cores multiply."""
    global _LORA
    import torch
    if torch.is_grad_enabled():
        _refuse_capture("linear_lora_train", "linear_lora and linear_lora_backward")
    if _LORA is None:
        _LORA = _lora_function()
    return _LORA.apply(X, A, B, P, ids, scaling, out_dtype)


# ---- log probabilities of tokens -------------------------------------------------------------------------

@dataclass
class TokenLogprobs:
    """Of every row: log p(target) [M] (None without targets), entropy [M], stats [M,2]
    (the largest logit, log of the sum of exp(z - largest)), and the likeliest
    tokens' log probabilities and ids [M,top] (None for top = 0)."""
    logp: "object"
    entropy: "object"
    stats: "object"
    top_logp: "object"
    top_ids: "object"

    @property
    def lse(self):
        """log sum exp of the row's logits."""
        return self.stats[:, 0] + self.stats[:, 1]


def _logits(z):
    import torch
    _require_cuda(z)
    if z.dim() != 2 or z.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be a 2D fp32 or bf16 tensor")
    M, V = z.shape
    if not 1 <= V <= _abi.MAX_VOCAB:
        raise ValueError(f"1 to {_abi.MAX_VOCAB} logits per row")
    if (V > 1 and z.stride(1) != 1) or (M > 1 and z.stride(0) < V):
        z = z.contiguous()
    return z, BF16 if z.dtype == torch.bfloat16 else F32, (z.stride(0) if M > 1 else V)


def _targets(t, M, V, device):
    import torch
    if t is None:
        return None
    _require_cuda(t)
    _same_device(device, t)
    if t.dtype not in (torch.int32, torch.int64) or tuple(t.shape) != (M,):
        raise ValueError("targets must be int32 or int64 [M]")
    if t.dtype == torch.int64:  # a value int32 cannot hold is outside [0, V) all the same
        t = t.clamp(-1, V).to(torch.int32)
    return t.contiguous()


def _scores(M, V, targets, top, device):
    import torch
    if not 0 <= top <= min(V, _abi.MAX_TOP):
        raise ValueError(f"top must be 0 to min(V, {_abi.MAX_TOP})")
    entropy = torch.empty(M, dtype=torch.float32, device=device)  # the others from it: cheaper than anew
    top_logp = entropy.new_empty((M, top)) if top else None
    return TokenLogprobs(torch.empty_like(entropy) if targets is not None else None, entropy, entropy.new_empty((M, 2)),
                         top_logp, torch.empty_like(top_logp, dtype=torch.int32) if top else None)


def token_logprobs(logits, targets=None, top: int = 0) -> TokenLogprobs:
    """Log probabilities of one given token per row, the entropy, and the ``top`` likeliest
    tokens (ties to the lowest id) of logits [M,V] (fp32 or bf16; rows may be slices of
    a padded buffer), in one pass.  targets is int32 or int64 [M]; a value outside
    [0, V) is left out (log p 0, and no gradient even where the row holds NaN).  -inf logits have p = 0; a row of -inf
    only gives -inf and entropy 0, one with NaN or +inf gives NaN and ids -1."""
    r = _done(_calls().token_logprobs(logits, targets, top), "token_logprobs")
    if r is not None:
        return TokenLogprobs(*r)
    z, dt, ld = _logits(logits)
    M, V = z.shape
    targets = _targets(targets, M, V, z.device)
    r = _scores(M, V, targets, top, z.device)
    with _on(z.device):
        check(lib().sherry_token_logprobs(_ptr(z), dt, M, V, ld, _ptr(targets), top, _ptr(r.logp), _ptr(r.entropy),
                                          _ptr(r.stats), _ptr(r.top_logp), _ptr(r.top_ids), _stream(z.device)),
              "token_logprobs")
    return r


def token_logprobs_backward(logits, targets, stats, entropy, dlogp=None, dentropy=None, out=None):
    """Gradient of :func:`token_logprobs` in the logits, [M,V] in their type:
    dlogp (onehot(target) - p) - dentropy p (log p + entropy).  ``out`` may be the logits
    themselves (rows in place) or a tensor that does not overlap them."""
    import torch
    if out is None:
        r = _done(_calls().token_logprobs_backward(logits, targets, stats, entropy, dlogp, dentropy),
                  "token_logprobs_backward")
        if r is not None:
            return r
    z, dt, ld = _logits(logits)
    M, V = z.shape
    targets = _targets(targets, M, V, z.device)
    _require_cuda(stats, entropy, dlogp, dentropy, out)
    _same_device(z.device, stats, entropy, dlogp, dentropy, out)
    vec = []
    for t, shape, name in ((stats, (M, 2), "stats"), (entropy, (M,), "entropy"), (dlogp, (M,), "dlogp"),
                           (dentropy, (M,), "dentropy")):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != shape):
            raise ValueError(f"{name} must be fp32 {list(shape)}")
        vec.append(None if t is None else t.contiguous())
    stats, entropy, dlogp, dentropy = vec
    if stats is None or (dentropy is not None and entropy is None) or (dlogp is not None and targets is None):
        raise ValueError("needs stats, targets with dlogp, and entropy with dentropy")
    if out is None:
        out = z.new_empty((M, V))
    elif (out.dtype != z.dtype or tuple(out.shape) != (M, V) or (V > 1 and out.stride(1) != 1)
          or (M > 1 and out.stride(0) < V)):
        raise ValueError("out must be [M, V] of the logits' type with rows of unit stride")
    elif M > 0 and _spans_overlap(z, out) and not (out.data_ptr() == z.data_ptr() and (M == 1 or out.stride(0) == ld)):
        raise ValueError("out must be the logits themselves or not overlap them")
    ldd = out.stride(0) if M > 1 else V
    with _on(z.device):
        check(lib().sherry_token_logprobs_backward(_ptr(z), dt, M, V, ld, _ptr(targets), _ptr(stats), _ptr(entropy),
                                                   _ptr(dlogp), _ptr(dentropy), _ptr(out), ldd, _stream(z.device)),
              "token_logprobs_backward")
    return out


def _spans_overlap(a, b) -> bool:
    """Whether the address ranges of two row-strided matrices meet."""
    def span(t):
        return t.data_ptr(), t.data_ptr() + ((t.shape[0] - 1) * t.stride(0) + t.shape[1]) * t.element_size()
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def _logprobs_function():
    import torch

    class SherryTokenLogprobs(torch.autograd.Function):
        """log p(target) and entropy with :func:`token_logprobs_backward`."""

        @staticmethod
        def forward(ctx, logits, targets):
            r = token_logprobs(logits, targets)
            ctx.save_for_backward(logits, targets, r.stats, r.entropy)
            ctx.set_materialize_grads(False)
            return r.logp, r.entropy

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, dlogp, dentropy):
            _refuse_capture("the backward pass of token_logprobs_train", "token_logprobs_backward")
            if dlogp is None and dentropy is None:
                return None, None
            logits, targets, stats, entropy = ctx.saved_tensors
            return token_logprobs_backward(logits, targets, stats, entropy, dlogp, dentropy), None

    return SherryTokenLogprobs


_LOGPROBS = None


def token_logprobs_train(logits, targets):
    """Differentiable (log p(target), entropy) of every row; the loss of a model is, say,
    ``-logp.mean()``."""
    global _LOGPROBS
    import torch
    if torch.is_grad_enabled():
        _refuse_capture("token_logprobs_train", "token_logprobs and token_logprobs_backward")
    if _LOGPROBS is None:
        _LOGPROBS = _logprobs_function()
    return _LOGPROBS.apply(logits, targets)


def linear_logprobs(X, P: PackedWeight, targets=None, top: int = 0) -> TokenLogprobs:
    """:func:`token_logprobs` of a packed head's logits X (T alpha)^T (P.N is the
    vocabulary), a chunk of tokens at a time, so that only a chunk's logits exist."""
    import torch
    X = _activations(X, P.K)
    _planes(P, X.device)
    M = X.shape[0]
    if not 1 <= P.N <= _abi.MAX_VOCAB:
        raise ValueError(f"a head has 1 to {_abi.MAX_VOCAB} rows")
    targets = _targets(targets, M, P.N, X.device)
    r = _scores(M, P.N, targets, top, X.device)
    with _on(X.device):
        L = lib()
        wsb = L.sherry_linear_logprobs_workspace_bytes(M, P.N, P.K, P.granularity, P.group)
        ws = _stream_workspace(wsb, X.device) if wsb else None
        check(L.sherry_linear_logprobs(_ptr(X), M, P.N, P.K, _ptr(P.idx), _ptr(P.sgn), _ptr(P.scales), P.granularity,
                                       P.group, _ptr(targets), top, _ptr(r.logp), _ptr(r.entropy), _ptr(r.stats),
                                       _ptr(r.top_logp), _ptr(r.top_ids), _ptr(ws), wsb, _stream(X.device)),
              "linear_logprobs")
    return r
