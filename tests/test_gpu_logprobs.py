"""Token log probabilities, entropy, likeliest tokens and their gradient against
64-bit formulas (needs a B200).

Tolerances: a sum of V positive fp32 terms, V / 256 of them in a chain, is off by at
most (V / 256 + 64) 2^-24 of itself; each term's exponential adds 2^-21 and its
argument's rounding |y| 2^-23, y = log2 of the term.  bf16 results add half a step."""
from __future__ import annotations

import math

import numpy as np
import pytest

from sparse_ternary_weight_b200 import synth
from tests.gpu_common import GRAN, packed_to_host, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sw():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_ternary_weight_b200.build import build
    build()
    import sparse_ternary_weight_b200 as sw
    return sw


def reference(z, t):
    """(logp, entropy, max, lsum) in float64 from host logits (float64) and targets."""
    m = z.max(1)
    with np.errstate(invalid="ignore", divide="ignore"):
        d = z - m[:, None]
        e = np.exp(d)
        s = e.sum(1)
        lsum = np.log(s)
        ent = lsum - np.where(e > 0, e * np.where(e > 0, d, 0), 0).sum(1) / s
    valid = (t >= 0) & (t < z.shape[1])
    logp = np.where(valid, d[np.arange(len(t)), np.where(valid, t, 0)] - lsum, 0.0)
    dead = np.isneginf(m)
    ent[dead], lsum[dead] = 0.0, 0.0
    logp[dead & valid] = -np.inf
    return logp, ent, m, lsum


def top_reference(z, k):
    return np.argsort(-(z + 0.0), axis=1, kind="stable")[:, :k]


def eps_sum(V):
    return (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -21


def make(M, V, dt, pad=0, off=0, spread=3.0, seed=0, coarse=False):
    """Logits as rows of a padded buffer that starts `off` elements into an allocation."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + M + V)
    ld = V + pad
    buf = torch.full((off + M * ld + 16,), float("nan"), dtype=dt, device="cuda")
    z = buf[off:off + M * ld].view(M, ld)[:, :V]
    x = spread * torch.randn((M, V), generator=g, device="cuda")
    z.copy_(torch.round(x) if coarse else x)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[::7] = -1
    if M > 3:
        t[3] = V  # outside: left out
    return buf, z, t.to(torch.int32)


def check(sw, z, t, top):
    import torch
    r = sw.token_logprobs(z, t, top=top)
    zh, th = z.double().cpu().numpy(), t.cpu().numpy().astype(np.int64)
    V = zh.shape[1]
    logp, ent, m, lsum = reference(zh, th)
    e = eps_sum(V)
    got = r.logp.double().cpu().numpy()
    fin = np.isfinite(logp)
    assert np.array_equal(np.isneginf(logp), np.isneginf(got))
    assert np.all(np.abs(got[fin] - logp[fin]) <= e + 2.0 ** -23 * np.abs(logp[fin]) + 2.0 ** -23), np.abs(got[fin] - logp[fin]).max()
    assert np.array_equal(got[(th < 0) | (th >= V)], np.zeros(((th < 0) | (th >= V)).sum()))
    scale = 2.0 + 2.0 * math.log(V + 1)
    assert np.all(np.abs(r.entropy.double().cpu().numpy() - ent) <= scale * e), np.abs(r.entropy.double().cpu().numpy() - ent).max()
    st = r.stats.double().cpu().numpy()
    assert np.array_equal(st[:, 0], m)
    assert np.all(np.abs(st[:, 1] - lsum) <= e + 2.0 ** -23 * np.abs(lsum))
    if top:
        ids = r.top_ids.cpu().numpy()
        want = top_reference(zh, top)
        assert np.array_equal(ids, want)
        dead = np.isneginf(m)
        with np.errstate(invalid="ignore"):
            lp = np.take_along_axis(zh, want, 1) - m[:, None] - lsum[:, None]
        lp[dead] = -np.inf
        tl = r.top_logp.double().cpu().numpy()
        f = np.isfinite(lp)
        assert np.array_equal(f, np.isfinite(tl))
        assert np.all(np.abs(tl[f] - lp[f]) <= e + 2.0 ** -23 * np.abs(lp[f]) + 2.0 ** -23)
    again = sw.token_logprobs(z, t, top=top)
    for a, b in zip((r.logp, r.entropy, r.stats), (again.logp, again.entropy, again.stats)):
        assert torch.equal(a, b)
    return r


SHAPES = [(1, 1, 1), (3, 2, 2), (5, 7, 5), (4, 8, 8), (2, 9, 0), (300, 37, 3), (1, 1000, 20), (7, 4097, 32),
          (1, 32000, 32), (3, 50257, 5), (2, 128256, 20), (700, 1031, 8), (1, 300000, 1)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}x{s[1]}-top{s[2]}")
def test_forward(sw, shape, dt):
    import torch
    M, V, top = shape
    T = torch.float32 if dt == "f32" else torch.bfloat16
    for pad, off in ((0, 0), (0, 1), (5, 3)):
        buf, z, t = make(M, V, T, pad, off, seed=pad)
        check(sw, z, t, top)
        check(sw, z, t, 0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2100, 701, 8), (2050, 4003, 20), (2048, 33, 32), (600, 9001, 20), (1100, 31, 5)],
                         ids=lambda s: f"{s[0]}x{s[1]}-top{s[2]}")
def test_forward_of_many_short_rows(sw, shape, dt):
    """The forms with fewer threads per row, odd lengths and alignments."""
    import torch
    M, V, top = shape
    T = torch.float32 if dt == "f32" else torch.bfloat16
    for pad, off, coarse in ((0, 0, False), (3, 1, True)):
        buf, z, t = make(M, V, T, pad, off, seed=pad, coarse=coarse)
        check(sw, z, t, top)
        check(sw, z, t, 0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_extremes_in_many_short_rows(sw, dt):
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    V = 1003
    low, high = torch.finfo(T).min, torch.finfo(T).max
    z = (2 * torch.randn((8, V), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")).to(T)
    z[0] = -math.inf
    z[1] = low
    z[2, 1:] = low
    z[3, ::2] = -math.inf
    z[4] = high
    z[5] = -1.05e38          # between the rows' edge and the floor of their elements
    z[5, 7] = -1.0e38
    z[6] = -1.2e38
    z[6, :3] = 0.0
    z[7] = 0.0
    t = torch.tensor([3, 3, 0, 1, 9, 7, 500, V - 1], dtype=torch.int32, device="cuda")
    check(sw, z, t, 20)
    far = torch.stack([x + z[7] * 0 + s for s in (-1e10, 1e10, -1e9, 1e9, -0.99e8, 1.01e8, -2.1e8, -1e30)
                       for x in [torch.zeros(V, device="cuda", dtype=T)]])
    far[:, ::5] *= 2          # a whole row far away, its elements further still
    check(sw, far, t, 20)
    z = torch.cat([z, far])
    t = t.repeat(2)
    for n in (50, 150):
        check(sw, z.repeat(n, 1), t.repeat(n), 20)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_ties_and_orders(sw, dt):
    """All equal, few distinct values, ascending and descending rows: every element or none
    passes the running threshold; ties go to the lowest index."""
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    V = 40003
    ramp = torch.arange(V, device="cuda", dtype=torch.float32)
    rows = [torch.zeros(V, device="cuda"), torch.full((V,), -2.5, device="cuda"), ramp / 4096, -ramp / 4096,
            (ramp % 3) - 1, -0.0 * ramp, torch.where(ramp % 2 == 0, 0.0, -0.0), (ramp // 1000) % 7]
    z = torch.stack(rows).to(T)
    t = torch.tensor([0, V - 1, V - 1, V - 1, 5, 6, 7, 8], dtype=torch.int32, device="cuda")
    for top in (1, 20, 32):
        check(sw, z, t, top)
    big = z.repeat(200, 1)  # one CTA per row
    check(sw, big, t.repeat(200), 20)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_masks_and_extremes(sw, dt):
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    V = 9001
    low = torch.finfo(T).min
    g = torch.Generator(device="cuda").manual_seed(3)
    x = 2 * torch.randn((12, V), generator=g, device="cuda")
    keep = torch.rand((12, V), generator=g, device="cuda") < 0.01
    z = x.to(T)
    z[0] = -math.inf                                        # nothing left
    z[1] = low                                              # masked by the lowest value only
    z[2] = torch.where(keep[2], z[2], torch.tensor(low, dtype=T, device="cuda"))
    z[3] = torch.where(keep[3], z[3], torch.tensor(-math.inf, dtype=T, device="cuda"))
    z[4] = -math.inf
    z[4, 8999] = 1.5                                        # one token left
    z[5] = z[5] + 10000                                     # far offsets
    z[6] = z[6] - 10000
    z[7, :] = -math.inf
    z[7, 17] = low                                          # the lowest value alone
    z[8, 4000] = torch.finfo(T).max                         # one huge logit
    z[9, :5000] = low
    z[10, 5000:] = -math.inf
    t = torch.tensor([5, 5, 5, 5, 8999, 1, 2, 17, 4000, 8000, 10, -1], dtype=torch.int32, device="cuda")
    check(sw, z, t, 20)
    check(sw, z.repeat(60, 1), t.repeat(60), 20)
    # the gradient of those rows is finite, and nothing where p is nothing
    r = sw.token_logprobs(z, t)
    dz = sw.token_logprobs_backward(z, t, r.stats, r.entropy, torch.ones(12, device="cuda"), torch.ones(12, device="cuda"))
    assert bool(torch.isfinite(dz).all())
    assert not dz[0].any()
    gone = torch.isinf(z[3]) & (torch.arange(V, device="cuda") != 5)
    assert not dz[3][gone].any()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_and_infinity(sw, dt, bad):
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    _, z, t = make(6, 20000, T)
    t[:] = 3
    want = sw.token_logprobs(z, t, top=4)
    z[2, 11111] = bad
    r = sw.token_logprobs(z, t, top=4)
    others = [0, 1, 3, 4, 5]
    for a, b in ((r.logp, want.logp), (r.entropy, want.entropy), (r.stats, want.stats), (r.top_logp, want.top_logp)):
        assert bool(torch.isnan(a[2]).all()) and torch.equal(a[others], b[others])
    assert bool((r.top_ids[2] == -1).all()) and torch.equal(r.top_ids[others], want.top_ids[others])


def grad_reference(z, t, g, h):
    logp, ent, m, lsum = reference(z, t)
    with np.errstate(invalid="ignore"):
        lp = z - m[:, None] - lsum[:, None]
    p = np.where(np.isneginf(m)[:, None], 0.0, np.exp(lp))
    lps = np.where(p > 0, lp, 0.0)
    valid = (t >= 0) & (t < z.shape[1]) & ~np.isneginf(m)
    g = np.where(valid, g, 0.0)
    out = -p * (g[:, None] + h[:, None] * (lps + ent[:, None]))
    out[np.arange(len(t))[valid], t[valid]] += g[valid]
    mag = p * (np.abs(g)[:, None] + np.abs(h)[:, None] * (np.abs(lps) + ent[:, None]))
    return out, mag, np.abs(lps)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (3, 2), (5, 9), (300, 37), (7, 4097), (3, 50257), (2, 128256)],
                         ids=lambda s: f"{s[0]}x{s[1]}")
def test_backward(sw, shape, dt):
    import torch
    M, V = shape
    T = torch.float32 if dt == "f32" else torch.bfloat16
    for pad, off in ((0, 0), (0, 1), (5, 3), (8, 2)):
        buf, z, t = make(M, V, T, pad, off, seed=pad)
        r = sw.token_logprobs(z, t)
        gen = torch.Generator(device="cuda").manual_seed(M)
        g, h = (torch.randn(M, generator=gen, device="cuda") for _ in range(2))
        out = sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, h)
        zh, th = z.double().cpu().numpy(), t.cpu().numpy().astype(np.int64)
        ref, mag, lp = grad_reference(zh, th, g.double().cpu().numpy(), h.double().cpu().numpy())
        e = eps_sum(V) * (4 + 2 * math.log(V + 1))
        gmag = np.abs(g.double().cpu().numpy())[:, None]
        hmag = np.abs(h.double().cpu().numpy())[:, None]
        p = np.exp(-lp)
        bound = (e + 2.0 ** -22 * (1 + lp)) * (mag + hmag * p) + 2.0 ** -23 * (np.abs(ref) + gmag * (np.abs(ref) > 0) * p) + 1e-36
        if dt == "bf16":
            bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
        err = np.abs(out.double().cpu().numpy() - ref)
        assert np.all(err <= bound), float((err / bound).max())
        # one of the two, and neither
        only = sw.token_logprobs_backward(z, t, r.stats, None, g)
        assert torch.equal(only, sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, torch.zeros_like(h)))
        ent = sw.token_logprobs_backward(z, None, r.stats, r.entropy, None, h)
        assert torch.equal(ent, sw.token_logprobs_backward(z, t, r.stats, r.entropy, torch.zeros_like(g), h))
        # into rows of another alignment, and in place; the padding stays as it was
        ob, o2, _ = make(M, V, T, pad + 1, 2, seed=9)
        edge = ob.clone()
        o2_ = sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, h, out=o2)
        assert torch.equal(o2_, out)
        view = edge[2:2 + M * (V + pad + 1)].view(M, V + pad + 1)[:, :V]
        view.copy_(out)
        assert torch.equal(ob.view(torch.uint8), edge.view(torch.uint8))
        before = buf.clone()
        sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, h, out=z)
        assert torch.equal(z, out)
        before[off:off + M * (V + pad)].view(M, V + pad)[:, :V].copy_(out)
        assert torch.equal(buf.view(torch.uint8), before.view(torch.uint8))


def test_other_forms_of_the_arguments(sw):
    """int64 targets, columns that are not next to each other: converted, with the same bits."""
    import torch
    _, z, t = make(9, 701, torch.bfloat16)
    z = z.contiguous()
    want = sw.token_logprobs(z, t, top=4)
    wide = torch.zeros((9, 1402), dtype=z.dtype, device="cuda")
    wide[:, ::2] = z
    got = sw.token_logprobs(wide[:, ::2], t.long() - 2 ** 40 * (t < 0), top=4)
    for a, b in ((got.logp, want.logp), (got.entropy, want.entropy), (got.stats, want.stats), (got.top_ids, want.top_ids),
                 (got.top_logp, want.top_logp)):
        assert torch.equal(a, b)
    g = torch.rand(9, device="cuda")
    dz = sw.token_logprobs_backward(z, t, want.stats, want.entropy, g, g)
    two = torch.stack([want.stats, want.stats], 2)[:, :, 0]
    assert not two.is_contiguous()
    assert torch.equal(sw.token_logprobs_backward(wide[:, ::2], t.long(), two, want.entropy, g, g), dz)


def test_differences(sw):
    """sum(g logp + h H) at z +- a step against the gradient along it."""
    import torch
    M, V = 6, 513
    _, z, t = make(M, V, torch.float32)
    gen = torch.Generator(device="cuda").manual_seed(1)
    g, h = (torch.rand(M, generator=gen, device="cuda") for _ in range(2))
    r = sw.token_logprobs(z, t)
    dz = sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, h)
    d = torch.randn((M, V), generator=gen, device="cuda")
    step = 2.0 ** -6

    def f(x):
        q = sw.token_logprobs(x.contiguous(), t)
        return float((g.double() * q.logp.double() + h.double() * q.entropy.double()).sum())

    want = (f(z + step * d) - f(z - step * d)) / (2 * step)
    got = float((dz.double() * d.double()).sum())
    # third derivatives of log-sum-exp along d are below 8 |d|_inf^3 per row (a third cumulant), and of
    # the entropy below that times |z - max|; rounding of f: eps_sum over the step
    far = float(d.abs().max()) ** 3 * 8 * (2 + float((z.max(1).values - z.min(1).values).max()))
    tol = M * (far * step ** 2 / 6 + 2 * eps_sum(V) * (2 + 2 * math.log(V)) / step)
    assert abs(want - got) <= tol, (want, got, tol)
    assert abs(want - got) <= 0.05 * max(1.0, abs(want))


def test_autograd_and_capture(sw):
    import torch
    _, z, t = make(5, 3001, torch.bfloat16)
    z = z.contiguous()
    x = z.clone().requires_grad_()
    logp, ent = sw.token_logprobs_train(x, t)
    (-logp.sum() + 0.5 * ent.sum()).backward()
    r = sw.token_logprobs(z, t)
    one = torch.ones(5, device="cuda")
    assert torch.equal(x.grad, sw.token_logprobs_backward(z, t, r.stats, r.entropy, -one, 0.5 * one))
    y = z.clone().requires_grad_()
    sw.token_logprobs_train(y, t)[0].sum().backward()  # the entropy unused
    assert torch.equal(y.grad, sw.token_logprobs_backward(z, t, r.stats, r.entropy, one))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q = sw.token_logprobs(z, t, top=3)
        dz = sw.token_logprobs_backward(z, t, q.stats, q.entropy, one)
    z.copy_(torch.flip(z, [1]))
    graph.replay()
    torch.cuda.synchronize()
    want = sw.token_logprobs(z, t, top=3)
    assert torch.equal(q.logp, want.logp) and torch.equal(q.top_ids, want.top_ids)
    assert torch.equal(dz, sw.token_logprobs_backward(z, t, want.stats, want.entropy, one))


@pytest.mark.parametrize("case", [(1, 1000, 512, "group", 128), (5, 513, 1024, "channel", 0), (300, 2001, 256, "group", 64),
                                  (40, 130, 96, "tensor", 0)], ids=lambda c: f"M{c[0]}-{c[1]}x{c[2]}-{c[3]}")
def test_linear_logprobs(sw, orc, case):
    import torch
    M, N, K, gname, group = case
    P = sw.quantize_pack(to_dev(synth.weights_normal(N, K, N + K, 0.05)), GRAN[gname], group or 128)
    X = to_dev(synth.activations_bf16(M, K, 77 + M).view(np.int16)).view(torch.bfloat16)
    t = torch.randint(0, N, (M,), device="cuda")
    r = sw.linear_logprobs(X, P, t, top=4)
    z = sw.linear(X, P, torch.float32)
    q = sw.token_logprobs(z, t, top=4)
    assert sw.device_status() == 0
    for a, b in ((r.logp, q.logp), (r.entropy, q.entropy), (r.stats, q.stats), (r.top_logp, q.top_logp)):
        assert torch.equal(a, b)
    assert torch.equal(r.top_ids, q.top_ids)
    check(sw, z, t.to(torch.int32), 4)


def test_head_in_chunks(sw):
    """A vocabulary large enough that the tokens go in several chunks, the last one short."""
    import torch
    M, N, K = 300, 140000, 128
    g = torch.Generator(device="cuda").manual_seed(2)
    P = sw.quantize_pack(0.05 * torch.randn((N, K), generator=g, device="cuda"))
    X = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    t = torch.randint(0, N, (M,), generator=g, device="cuda")
    r = sw.linear_logprobs(X, P, t, top=3)
    # chunks of 128 tokens; each may run by another kernel than the whole, so compare with theirs
    for a, b in ((0, 128), (128, 256), (256, 300)):
        q = sw.token_logprobs(sw.linear(X[a:b], P), t[a:b], top=3)
        assert torch.equal(r.logp[a:b], q.logp) and torch.equal(r.top_ids[a:b], q.top_ids)
    assert sw.device_status() == 0


def test_training_step_together(sw, orc):
    """Adapters under a packed projection, a packed head, the loss and its gradient back to the
    adapters, as a training step runs them, against the same step in 64 bits."""
    import torch
    M, K, H, V, R, n = 150, 256, 192, 1003, 8, 3
    rng = np.random.default_rng(4)
    P1 = sw.quantize_pack(to_dev(synth.weights_normal(H, K, 1, 0.05)), "per_group", 64)
    P2 = sw.quantize_pack(to_dev(synth.weights_normal(V, H, 2, 0.1)), "per_channel")
    W1 = orc.unpack_f32(*packed_to_host(P1), H, K, GRAN["group"], 64).astype(np.float64)
    W2 = orc.unpack_f32(*packed_to_host(P2), V, H, GRAN["channel"], 128).astype(np.float64)
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    X, A, B = bf(rng.standard_normal((M, K))), bf(rng.standard_normal((n, R, K)) / 16), bf(0.2 * rng.standard_normal((n, H, R)))
    ids = torch.from_numpy(rng.integers(-1, n, M)).cuda()
    t = torch.from_numpy(rng.integers(0, V, M)).cuda()
    Y, U = sw.linear_lora(X, P1, A, B, ids, None, torch.bfloat16, return_u=True)
    z = sw.linear(Y, P2, torch.bfloat16)
    r = sw.token_logprobs(z, t)
    dz = sw.token_logprobs_backward(z, t, r.stats, r.entropy, torch.full((M,), -1.0 / M, device="cuda"))
    dY = sw.linear_backward(dz, P2)
    dX, dA, dB = sw.linear_lora_backward(dY, X, P1, A, B, ids, U, None, torch.float32)
    assert sw.device_status() == 0
    # 64 bits, rounding to bf16 where the step does (so that only the operators' own errors remain)
    rnd = lambda a: torch.from_numpy(a).to(torch.bfloat16).double().numpy()  # noqa: E731
    Xh, Ah, Bh, idh = (q.double().cpu().numpy() for q in (X, A, B, ids))
    th = t.cpu().numpy()
    Uh, Yh = np.zeros((M, R)), Xh @ W1.T
    for a in range(n):
        at = idh == a
        Uh[at] = Xh[at] @ Ah[a].T
        Yh[at] += Uh[at] @ Bh[a].T
    zh = rnd(rnd(Yh) @ W2.T)
    logp, ent, m, ls = reference(zh, th)
    p = np.exp(zh - (m + ls)[:, None])
    p[np.arange(M), th] -= 1
    dYh = rnd(rnd(p / M) @ W2)
    rel = lambda got, ref: np.linalg.norm(got.double().cpu().numpy() - ref) / np.linalg.norm(ref)  # noqa: E731
    assert abs(float(r.logp.double().sum()) - logp.sum()) <= 2.0 ** -8 * np.abs(logp).sum()
    # one bf16 step in an intermediate moves what follows by at most 2^-7 of its own size on average;
    # three of them lie before dY, four before the adapters' gradients
    assert rel(dY, dYh) <= 3 * 2.0 ** -7
    for a in range(n):
        at = idh == a
        assert rel(dB[a], dYh[at].T @ Uh[at]) <= 4 * 2.0 ** -7
        assert rel(dA[a], (dYh[at] @ Bh[a]).T @ Xh[at]) <= 4 * 2.0 ** -7
    dXh = dYh @ W1
    for a in range(n):
        at = idh == a
        dXh[at] += (dYh[at] @ Bh[a]) @ Ah[a]
    assert rel(dX, dXh) <= 4 * 2.0 ** -7


def test_refusals(sw):
    import torch
    z = torch.zeros(3, 10, device="cuda")
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    for bad in (dict(logits=z.half()), dict(logits=z[0]), dict(logits=z.cpu()), dict(targets=t[:2]), dict(targets=t.float()),
                dict(top=-1), dict(top=11), dict(top=33), dict(logits=z[:, :0])):
        with pytest.raises(ValueError):
            sw.token_logprobs(**{**dict(logits=z, targets=t, top=0), **bad})
    r = sw.token_logprobs(z, t)
    g = torch.ones(3, device="cuda")
    ok = dict(logits=z, targets=t, stats=r.stats, entropy=r.entropy, dlogp=g, dentropy=g)
    for bad in (dict(stats=None), dict(entropy=None), dict(targets=None), dict(stats=r.stats[:, 0]), dict(dlogp=g.double()),
                dict(out=z[:, :9]), dict(out=z.to(torch.bfloat16)), dict(out=z.t()),
                dict(logits=z[:2, :4], targets=t[:2], stats=r.stats[:2], entropy=r.entropy[:2], dlogp=g[:2], dentropy=g[:2],
                     out=z[1:, 2:6])):
        with pytest.raises(ValueError):
            sw.token_logprobs_backward(**{**ok, **bad})
    # no tokens; columns of another order are copied first
    assert sw.token_logprobs(z[:0], t[:0], top=2).top_ids.shape == (0, 2)
    w = torch.randn(10, 3, device="cuda").t()
    a, b = sw.token_logprobs(w, t, top=2), sw.token_logprobs(w.contiguous(), t, top=2)
    assert torch.equal(a.logp, b.logp) and torch.equal(a.top_ids, b.top_ids)
