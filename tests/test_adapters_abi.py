"""Host-side checks of the adapters' and the token log probabilities' entry points:
documented statuses, nothing launched (no GPU needed)."""
import pytest

from sparse_ternary_weight_b200 import _abi
from sparse_ternary_weight_b200.build import build

FAKE = 0x10000  # aligned, never dereferenced: every call below fails validation first, or has nothing to do


@pytest.fixture(scope="module")
def L():
    build()
    return _abi.lib()


def lora_args(**kw):
    d = dict(X=FAKE, M=4, N=8, K=64, idx=FAKE, sgn=FAKE, sc=FAKE, g=_abi.PER_GROUP, group=32, A=FAKE, B=FAKE, ids=FAKE,
             s=None, n=2, R=8, U=None, Y=FAKE, yd=_abi.F32, ws=None, wsb=0)
    d.update(kw)
    return [d[k] for k in ("X", "M", "N", "K", "idx", "sgn", "sc", "g", "group", "A", "B", "ids", "s", "n", "R", "U", "Y",
                           "yd", "ws", "wsb")] + [None]


def test_linear_lora_validation(L):
    f = lambda **kw: L.sherry_linear_lora(*lora_args(**kw))  # noqa: E731
    for kw in (dict(M=-1), dict(M=1 << 31), dict(K=40), dict(n=0), dict(n=_abi.MAX_ADAPTERS + 1), dict(R=0), dict(R=12),
               dict(R=_abi.MAX_RANK + 8), dict(N=-1)):
        assert f(**kw) == _abi.ERR_SHAPE, kw
    assert f(group=48) == _abi.ERR_GROUP and f(g=7) == _abi.ERR_GRANULARITY and f(yd=5) == _abi.ERR_DTYPE
    for k in ("X", "idx", "A", "B", "ids", "Y"):
        assert f(**{k: None}) == _abi.ERR_NULL, k
    for kw in (dict(A=FAKE + 8), dict(B=FAKE + 2), dict(ids=FAKE + 2), dict(s=FAKE + 1), dict(U=FAKE + 4), dict(Y=FAKE + 4)):
        assert f(**kw) == _abi.ERR_ALIGN, kw
    assert f() == _abi.ERR_WORKSPACE
    need = L.sherry_linear_lora_workspace_bytes(4, 8, 64, _abi.PER_GROUP, 32, 2, 8, _abi.F32)
    assert need > 256 * 1024
    assert f(ws=FAKE, wsb=need - 1) == _abi.ERR_WORKSPACE
    assert f(ws=FAKE + 16, wsb=need) == _abi.ERR_ALIGN
    assert f(M=0, X=None) == _abi.OK and f(N=0, idx=None, sgn=None, sc=None, B=None, Y=None) == _abi.OK


def test_backward_validation(L):
    def f(**kw):
        d = dict(dY=FAKE, X=FAKE, M=4, N=8, K=64, idx=FAKE, sgn=FAKE, sc=FAKE, g=_abi.PER_GROUP, group=32, A=FAKE, B=FAKE,
                 ids=FAKE, s=None, n=2, R=8, U=FAKE, dX=FAKE, dA=FAKE, dB=FAKE, gd=_abi.F32, ws=None, wsb=0)
        d.update(kw)
        return L.sherry_linear_lora_backward(*d.values(), None)
    for kw in (dict(M=-1), dict(K=8), dict(n=0), dict(R=20)):
        assert f(**kw) == _abi.ERR_SHAPE, kw
    for kw in (dict(dY=None), dict(A=None), dict(ids=None), dict(U=None), dict(X=None), dict(sc=None)):
        assert f(**kw) == _abi.ERR_NULL, kw
    for kw in (dict(dY=FAKE + 2), dict(U=FAKE + 4), dict(dA=FAKE + 4), dict(dB=FAKE + 4), dict(dX=FAKE + 8)):
        assert f(**kw) == _abi.ERR_ALIGN, kw
    assert f(gd=9) == _abi.ERR_DTYPE
    assert f() == _abi.ERR_WORKSPACE
    assert f(dX=None, dA=None, dB=None) == _abi.OK and f(dX=None, dA=None, X=None) == _abi.ERR_WORKSPACE
    g = L.sherry_linear_backward
    args = lambda **kw: [*{**dict(dY=FAKE, M=4, N=8, K=64, idx=FAKE, sgn=FAKE, sc=FAKE, g=_abi.PER_CHANNEL, group=0,  # noqa: E731
                                  dX=FAKE, ws=None, wsb=0), **kw}.values(), None]
    assert g(*args(M=-2)) == _abi.ERR_SHAPE and g(*args(dX=None)) == _abi.ERR_NULL and g(*args(dX=FAKE + 2)) == _abi.ERR_ALIGN
    assert g(*args(M=0)) == _abi.OK
    assert L.sherry_linear_backward_workspace_bytes(4, 7, 64) > 0  # odd rows are padded
    assert g(*args(N=7)) == _abi.ERR_WORKSPACE


def test_logprobs_validation(L):
    def f(**kw):
        d = dict(z=FAKE, dt=_abi.F32, M=2, V=10, ld=10, t=FAKE, top=0, logp=FAKE, ent=FAKE, st=FAKE, tl=None, ti=None)
        d.update(kw)
        return L.sherry_token_logprobs(*d.values(), None)
    assert f(dt=3) == _abi.ERR_DTYPE
    for kw in (dict(M=-1), dict(V=0), dict(ld=9), dict(V=_abi.MAX_VOCAB + 1, ld=1 << 30), dict(top=-1), dict(top=11),
               dict(V=100, ld=100, top=33)):
        assert f(**kw) == _abi.ERR_SHAPE, kw
    for kw in (dict(z=None), dict(st=None), dict(t=None), dict(top=2), dict(top=2, tl=FAKE)):
        assert f(**kw) == _abi.ERR_NULL, kw
    assert f(z=FAKE + 2) == _abi.ERR_ALIGN and f(st=FAKE + 1) == _abi.ERR_ALIGN
    assert f(M=0, z=None) == _abi.OK

    def b(**kw):
        d = dict(z=FAKE, dt=_abi.BF16, M=2, V=10, ld=10, t=FAKE, st=FAKE, ent=FAKE, g=FAKE, h=FAKE, out=2 * FAKE, ldd=10)
        d.update(kw)
        return L.sherry_token_logprobs_backward(*d.values(), None)
    for kw in (dict(ldd=9), dict(out=FAKE, ldd=11)):
        assert b(**kw) == _abi.ERR_SHAPE, kw
    for kw in (dict(out=None), dict(st=None), dict(ent=None), dict(t=None)):
        assert b(**kw) == _abi.ERR_NULL, kw
    assert b(out=2 * FAKE + 1) == _abi.ERR_ALIGN and b(M=0, z=None, out=None) == _abi.OK


def test_linear_logprobs_validation(L):
    def f(**kw):
        d = dict(X=FAKE, M=2, N=100, K=64, idx=FAKE, sgn=FAKE, sc=FAKE, g=_abi.PER_CHANNEL, group=0, t=FAKE, top=0, logp=FAKE,
                 ent=FAKE, st=FAKE, tl=None, ti=None, ws=None, wsb=0)
        d.update(kw)
        return L.sherry_linear_logprobs(*d.values(), None)
    assert f(N=0) == _abi.ERR_SHAPE and f(K=8) == _abi.ERR_SHAPE and f(top=33) == _abi.ERR_SHAPE
    assert f(X=None) == _abi.ERR_NULL and f(st=None) == _abi.ERR_NULL and f(X=FAKE + 2) == _abi.ERR_ALIGN
    assert f() == _abi.ERR_WORKSPACE and f(M=0, X=None) == _abi.OK
    need = L.sherry_linear_logprobs_workspace_bytes(2, 100, 64, _abi.PER_CHANNEL, 0)
    assert need >= 256 * 1024 + 2 * 100 * 4
    assert f(ws=FAKE, wsb=need - 1) == _abi.ERR_WORKSPACE


def test_binding_rejects_cpu_tensors():
    import torch
    import sparse_ternary_weight_b200 as sw
    z = torch.zeros(2, 8)
    x = torch.zeros(2, 32, dtype=torch.bfloat16)
    P = sw.PackedWeight(torch.zeros(8, 1, dtype=torch.int32), torch.zeros(8, 1, dtype=torch.uint8), torch.zeros(8), 8, 32,
                        _abi.PER_CHANNEL, 0)
    a, b = torch.zeros(1, 8, 32, dtype=torch.bfloat16), torch.zeros(1, 8, 8, dtype=torch.bfloat16)
    ids = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: sw.token_logprobs(z), lambda: sw.linear_logprobs(x, P), lambda: sw.linear_backward(x[:, :8], P),
                 lambda: sw.linear_lora(x, P, a, b, ids)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_scratch_goes_by_the_tokens(L):
    """A bank of many adapters costs a few tokens no more than the slots (tile, adapter) that they can make."""
    fwd = lambda M, n, R=128: L.sherry_linear_lora_workspace_bytes(M, 8192, 4096, _abi.PER_GROUP, 128, n, R, _abi.BF16)  # noqa: E731
    bwd = lambda M, n, R=128: L.sherry_linear_lora_backward_workspace_bytes(M, 8192, 4096, n, R)  # noqa: E731
    # 100 tokens: at most 100 slots of 128 rows, two terms of U (bf16 Y), three of P and of U
    slots = 100 * 128 * 128 * 2
    base = fwd(100, 1) + 256 * 1024
    assert fwd(100, 1024) <= base + 2 * slots + 64 * 1024
    assert bwd(100, 1024) <= bwd(100, 1) + 2 * 3 * slots + 64 * 1024
    assert fwd(100, 1024) - fwd(100, 512) <= 8 * 1024  # the plan's counts alone


def test_planes_are_what_the_weight_says():
    """A packed weight whose planes are of another type, length or layout is refused, not read as it lies."""
    import dataclasses

    import torch
    import sparse_ternary_weight_b200 as sw
    cpu = torch.device("cpu")
    P = sw.PackedWeight(torch.zeros(8, 2, dtype=torch.int32), torch.zeros(8, 2, dtype=torch.uint8), torch.zeros(16), 8, 64,
                        _abi.PER_GROUP, 32)
    sw._planes(P, cpu)
    sw._planes(dataclasses.replace(P, granularity=_abi.PER_TENSOR), cpu)  # more scales than are read
    sw._planes(dataclasses.replace(P, idx=P.idx.view(torch.uint32)), cpu)
    for kw in bad_planes(P):
        with pytest.raises(ValueError):
            sw._planes(dataclasses.replace(P, **kw), cpu)
    with pytest.raises(ValueError):
        sw._planes(P, torch.device("meta"))


def bad_planes(P):
    """What is wrong with a plane of P, one thing at a time."""
    import torch
    two = lambda t: torch.stack([t, t], -1)[..., 0]  # noqa: E731  (every other element)
    return [dict(idx=P.idx[:-1]), dict(idx=P.idx.long()), dict(idx=two(P.idx)), dict(idx=P.idx.t()), dict(sgn=P.sgn[:, :1]),
            dict(sgn=P.sgn.int()), dict(sgn=two(P.sgn)), dict(scales=P.scales[:-1]), dict(scales=P.scales.double()),
            dict(scales=P.scales.to(torch.bfloat16)), dict(scales=two(P.scales)), dict(N=P.N + 1), dict(N=P.N - 1)]


def test_u_without_outputs_needs_its_inputs(L):
    f = lambda **kw: L.sherry_linear_lora(*lora_args(**{**dict(N=0, U=FAKE, idx=None, sgn=None, sc=None, B=None, Y=None), **kw}))  # noqa: E731
    for k in ("X", "A", "ids"):
        assert f(**{k: None}) == _abi.ERR_NULL, k
    assert f(U=FAKE + 4) == _abi.ERR_ALIGN and f(M=0, X=None, A=None, ids=None) == _abi.OK


def test_a_missing_binding_is_reported(monkeypatch):
    """In its own words, as a missing library is: there is no other form of the calls to fall back to."""
    import sys

    import torch
    import sparse_ternary_weight_b200 as sw
    monkeypatch.setattr(sw, "_native", [None])
    monkeypatch.setitem(sys.modules, "sparse_ternary_weight_b200._binding", None)
    monkeypatch.delattr(sw, "_binding", raising=False)
    with pytest.raises(RuntimeError, match="sparse_ternary_weight_b200.build"):
        sw.token_logprobs(torch.zeros(2, 8))
