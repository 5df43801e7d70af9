"""Low-rank adapters beside a packed linear, their gradients and the packed linear's
input gradient, against 64-bit restatements of the formulas (needs a B200).

Tolerances: fp32 sums are bounded as the linear's are (2^-16 of the sum of the
terms' magnitudes, once for the product into rank space and once for the sum it
enters, hence 2^-15 with the split terms of U or P, which drop at most 2^-16);
a bf16 result adds half a step, 2^-8 of itself; the input gradient multiplies
alpha rounded to bf16, at most 2^-8 of each term, or exactly for a per-tensor scale."""
from __future__ import annotations

import numpy as np
import pytest

from sparse_ternary_weight_b200 import synth
from tests.gpu_common import GRAN, canaried, canaries_intact, packed_to_host, to_dev

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


class Problem:
    """Inputs on the device and everything in float64 on the host."""

    def __init__(self, sw, orc, M, N, K, gname, group, R, n, ids="mixed", scaled=True, seed=0):
        import torch
        rng = np.random.default_rng(seed + 7 * M + 11 * N + 13 * K + R)
        g = GRAN[gname]
        self.shape = (M, N, K)
        W = synth.weights_normal(N, K, seed + N + K, 0.02)
        self.P = sw.quantize_pack(to_dev(W), g, group if gname == "group" else 128)
        idx, sgn, sc = packed_to_host(self.P)
        self.W = orc.unpack_f32(idx, sgn, sc, N, K, g, group if gname == "group" else 128).astype(np.float64)
        self.gname = gname

        def bf16(a):
            t = torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)
            return t.cuda(), t.double().numpy()

        self.X, self.Xh = bf16(rng.standard_normal((M, K)))
        self.A, self.Ah = bf16(rng.standard_normal((n, R, K)) / np.sqrt(K))
        self.B, self.Bh = bf16(0.1 * rng.standard_normal((n, N, R)))
        self.G, self.Gh = bf16(rng.standard_normal((M, N)) / max(N, 1))
        if ids == "mixed":
            i = rng.integers(-1, n, M)
        elif ids == "sorted":
            i = np.sort(rng.integers(0, n, M))
        elif ids == "none":
            i = np.full(M, -1)
        elif ids == "wild":  # everything outside [0, n) is no adapter
            i = rng.choice([-1, n, 2 ** 31 - 1, -2 ** 31, 0, n - 1], M)
        else:
            i = np.full(M, n - 1)
        self.idsh = np.where((i >= 0) & (i < n), i, -1)
        self.ids = torch.from_numpy(i.astype(np.int32)).cuda()
        sch = (0.5 + rng.random(n)).astype(np.float32)
        self.scaling = torch.from_numpy(sch).cuda() if scaled else None
        self.s = sch.astype(np.float64) if scaled else np.ones(n)
        self.n, self.R = n, R

    def forward(self, mag=False):
        f = np.abs if mag else (lambda a: a)
        X, W, A, B = f(self.Xh), f(self.W), f(self.Ah), f(self.Bh)
        Y = X @ W.T
        U = np.zeros((self.shape[0], self.R))
        for a in range(self.n):
            at = self.idsh == a
            U[at] = self.s[a] * (X[at] @ A[a].T)
            Y[at] += U[at] @ B[a].T
        return Y, U

    def backward(self, mag=False):
        f = np.abs if mag else (lambda a: a)
        X, W, A, B, G = f(self.Xh), f(self.W), f(self.Ah), f(self.Bh), f(self.Gh)
        U = self.forward(mag)[1]
        base = G @ W
        extra = np.zeros_like(base)
        dA, dB = np.zeros_like(A), np.zeros_like(B)
        for a in range(self.n):
            at = self.idsh == a
            Pm = self.s[a] * (G[at] @ B[a])
            extra[at] = Pm @ A[a]
            dA[a] = Pm.T @ X[at]
            dB[a] = G[at].T @ U[at]
        return base, extra, dA, dB


def host(t):
    return t.double().cpu().numpy()


def check_sum(got, ref, mag, what, bf16=False):
    err = np.abs(host(got) - ref)
    bound = 2.0 ** -15 * mag + 1e-30
    if bf16:
        bound = bound + 2.0 ** -8 * (np.abs(ref) + bound)
    assert np.all(np.isfinite(host(got))), what
    assert np.all(err <= bound), (what, float((err / bound).max()))


def check_dx(pr, dX, extra=True):
    base, ext, _, _ = pr.backward()
    mb, me, _, _ = pr.backward(True)
    ref = base + (ext if extra else 0)
    bound = (2.0 ** -15 + (0 if pr.gname == "tensor" else 2.0 ** -8)) * mb + (2.0 ** -15 * me if extra else 0)
    bound = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 1e-30
    err = np.abs(host(dX) - ref)
    assert np.all(np.isfinite(host(dX)))
    assert np.all(err <= bound), float((err / bound).max())


# (M, N, K, gran, group, R, n, ids): one token and few, each linear kernel, prefill tiles that end
# inside, ranks that end inside 16, more adapters than tokens of a tile, odd N, K that only the
# general kernel takes
CASES = [
    (1, 64, 256, "group", 128, 16, 4, "mixed"),
    (1, 1, 32, "group", 32, 8, 1, "last"),
    (2, 513, 1024, "channel", 0, 24, 3, "mixed"),
    (5, 130, 96, "group", 32, 8, 2, "wild"),
    (16, 300, 512, "group", 128, 64, 20, "mixed"),
    (17, 130, 256, "tensor", 0, 40, 5, "mixed"),
    (20, 100, 192, "group", 64, 16, 5, "mixed"),
    (32, 96, 1024, "group", 256, 128, 3, "sorted"),
    (33, 257, 512, "group", 128, 8, 4, "sorted"),
    (128, 128, 64, "group", 64, 16, 1, "last"),
    (129, 200, 320, "channel", 0, 128, 2, "mixed"),
    (200, 129, 2048, "group", 128, 32, 150, "mixed"),
    (300, 384, 1024, "group", 128, 72, 7, "sorted"),
    (300, 70, 160, "group", 32, 16, 3, "mixed"),
    (257, 512, 512, "tensor", 0, 16, 3, "none"),
    (700, 1000, 768, "group", 64, 16, 9, "mixed"),
]
IDS = [f"M{c[0]}-{c[1]}x{c[2]}-{c[3]}{c[4]}-r{c[5]}x{c[6]}-{c[7]}" for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_linear_lora(sw, orc, case):
    import torch
    M, N, K, gname, group, R, n, ids = case
    pr = Problem(sw, orc, M, N, K, gname, group, R, n, ids, scaled=M % 2 == 0)
    ref, U = pr.forward()
    mag, Um = pr.forward(True)
    y32, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, torch.float32, return_u=True)
    assert sw.device_status() == 0
    check_sum(y32, ref, mag, "Y fp32")
    check_sum(u, U, Um, "U")
    assert bool((u[pr.ids.lt(0) | pr.ids.ge(n)] == 0).all())
    full, out = canaried((M, N), torch.bfloat16)
    yb = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, torch.bfloat16, out=out)
    assert yb is out and canaries_intact(full)
    check_sum(yb, ref, mag, "Y bf16", bf16=True)
    # the same call gives the same bits
    assert torch.equal(y32, sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, torch.float32))


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_linear_backward(sw, orc, case):
    import torch
    M, N, K, gname, group, R, n, ids = case
    pr = Problem(sw, orc, M, N, K, gname, group, R, n, ids)
    full, out = canaried((M, K), torch.bfloat16)
    dX = sw.linear_backward(pr.G, pr.P, out=out)
    assert sw.device_status() == 0
    assert canaries_intact(full)
    check_dx(pr, dX, extra=False)
    assert torch.equal(dX, sw.linear_backward(pr.G, pr.P))


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_linear_lora_backward(sw, orc, case, gdt):
    import torch
    M, N, K, gname, group, R, n, ids = case
    pr = Problem(sw, orc, M, N, K, gname, group, R, n, ids, scaled=M % 2 == 0)
    dt = torch.float32 if gdt == "f32" else torch.bfloat16
    U = torch.from_numpy(pr.forward()[1].astype(np.float32)).cuda()
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, dt)
    assert sw.device_status() == 0
    check_dx(pr, dX)
    _, _, refA, refB = pr.backward()
    _, _, magA, magB = pr.backward(True)
    check_sum(dA, refA, magA, "dA", gdt == "bf16")
    check_sum(dB, refB, magB, "dB", gdt == "bf16")
    for a in range(n):  # adapters without tokens: exact zeros
        if not (pr.idsh == a).any():
            assert not dA[a].any() and not dB[a].any()
    again = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, dt)
    assert all(torch.equal(p, q) for p, q in zip((dX, dA, dB), again))


# what the cases above leave out: prefill tiles with ranks of one and two blocks in two and three terms,
# K split over a cluster, tokens taken adapter by adapter (odd N besides), more slots than clusters,
# one adapter with many tiles beside many without, one and two tokens of a large weight
MORE = [
    (257, 130, 512, "group", 128, 128, 2, "sorted"),
    (300, 257, 1024, "channel", 0, 128, 3, "mixed"),
    (520, 129, 8192, "group", 128, 16, 4, "sorted"),
    (390, 70, 4096, "tensor", 0, 24, 2, "wild"),
    (1000, 201, 640, "group", 64, 40, 30, "mixed"),
    (256, 130, 256, "group", 128, 16, 4, "mixed"),
    (9000, 64, 256, "group", 128, 8, 64, "last"),
    (1, 1056, 32768, "group", 128, 16, 2, "last"),
    (2, 1057, 32768, "channel", 0, 8, 3, "sorted"),
]
MORE_IDS = [f"M{c[0]}-{c[1]}x{c[2]}-{c[3]}{c[4]}-r{c[5]}x{c[6]}-{c[7]}" for c in MORE]


@pytest.mark.parametrize("case", MORE, ids=MORE_IDS)
def test_linear_lora_more(sw, orc, case):
    test_linear_lora(sw, orc, case)


@pytest.mark.parametrize("gdt", ["f32", "bf16"])
@pytest.mark.parametrize("case", MORE[:7], ids=MORE_IDS[:7])
def test_linear_lora_backward_more(sw, orc, case, gdt):
    test_linear_lora_backward(sw, orc, case, gdt)


@pytest.mark.parametrize("M,n", [(20, 3), (300, 3), (1000, 20)])
def test_tokens_of_none_may_hold_anything(sw, orc, M, n):
    """Rows of padding (id -1) full of NaN and infinities reach no other token and no gradient."""
    import torch
    pr = Problem(sw, orc, M, 130, 512, "group", 128, 16, n, "mixed")
    none = torch.from_numpy(pr.idsh < 0).cuda()
    assert bool(none.any()) and not bool(none.all())
    y, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    want = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, torch.float32)
    X, G = pr.X.clone(), pr.G.clone()
    for t in (X, G):
        rows = torch.full_like(t, float("nan"))
        rows[:, ::2] = float("inf")
        t.copy_(torch.where(none[:, None], rows, t))
    y2, U2 = sw.linear_lora(X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    assert torch.equal(y2[~none], y[~none]) and torch.equal(U2, U)
    dX, dA, dB = sw.linear_lora_backward(G, X, pr.P, pr.A, pr.B, pr.ids, U2, pr.scaling, torch.float32)
    assert torch.equal(dX[~none], want[0][~none])
    assert torch.equal(dA, want[1]) and torch.equal(dB, want[2])


@pytest.mark.parametrize("M,ids", [(20, "mixed"), (300, "sorted"), (300, "mixed"), (1000, "mixed")])
def test_an_adapter_that_is_not_finite_stays_alone(sw, orc, M, ids):
    """NaN and infinities in one adapter's weights reach its own tokens only."""
    import torch
    pr = Problem(sw, orc, M, 130, 512, "group", 128, 16, 4, ids)
    y = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling)
    A, B = pr.A.clone(), pr.B.clone()
    A[1] = float("nan")
    B[1, ::2] = float("inf")
    y2 = sw.linear_lora(pr.X, pr.P, A, B, pr.ids, pr.scaling)
    own = pr.ids == 1
    assert torch.equal(y2[~own], y[~own])
    assert not bool(torch.isfinite(y2[own]).any())


@pytest.mark.parametrize("M,N,K,ids", [(20, 130, 512, "mixed"), (300, 130, 512, "sorted"), (1000, 130, 512, "mixed"),
                                       (1500, 328, 6688, "mixed")])
def test_gradients_beside_an_adapter_that_is_not_finite(sw, orc, M, N, K, ids):
    """Its own tokens' dX is what the formula gives, every other token's is what it was."""
    import torch
    pr = Problem(sw, orc, M, N, K, "tensor", 0, 16, 4, ids)
    _, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    want = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, torch.float32)
    A = pr.A.clone()
    A[1, 3, 5] = float("nan")
    A[1, 2, 7] = float("inf")
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, A, pr.B, pr.ids, U, pr.scaling, torch.float32)
    own = pr.ids == 1
    assert bool(own.any())
    assert torch.equal(dX[~own], want[0][~own]) and torch.equal(dA, want[1]) and torch.equal(dB, want[2])
    assert bool(torch.isnan(dX[own][:, 5]).all()) and bool(torch.isinf(dX[own][:, 7]).all())
    rest = torch.ones(K, dtype=torch.bool, device="cuda")
    rest[5] = rest[7] = False
    # the same product summed elsewhere: 2^-15 of its terms, and two roundings to bf16 of half a step each
    base, ext, _, _ = pr.backward(True)
    tol = torch.from_numpy(2.0 ** -15 * (base + ext)).cuda()[own] + 2.0 ** -7 * want[0][own].double().abs()
    assert bool(((dX[own].double() - want[0][own].double()).abs() <= tol)[:, rest].all())
    # infinities in B reach P, and through it that adapter's rows and gradient alone
    B = pr.B.clone()
    B[1, 0, 0] = float("inf")
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, B, pr.ids, U, pr.scaling, torch.float32)
    others = [0, 2, 3]
    assert torch.equal(dX[~own], want[0][~own]) and torch.equal(dA[others], want[1][others])
    assert not bool(torch.isfinite(dX[own]).any()) and not bool(torch.isfinite(dA[1, 0]).any())


def test_large_backward_tiles(sw, orc):
    """Enough tiles for the 256-token form of the input gradient, ragged in every direction."""
    import torch
    pr = Problem(sw, orc, 1500, 328, 6688, "group", 32, 16, 5, "mixed")
    U = torch.from_numpy(pr.forward()[1].astype(np.float32)).cuda()
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, torch.float32)
    assert sw.device_status() == 0
    check_dx(pr, dX)
    _, _, refA, refB = pr.backward()
    _, _, magA, magB = pr.backward(True)
    check_sum(dA, refA, magA, "dA")
    check_sum(dB, refB, magB, "dB")


def test_need_leaves_out(sw, orc):
    import torch
    pr = Problem(sw, orc, 40, 100, 256, "group", 128, 16, 3)
    U = torch.from_numpy(pr.forward()[1].astype(np.float32)).cuda()
    whole = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False, False, False)):
        part = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U if need[2] else None, pr.scaling,
                                       need=need)
        for want, p, q in zip(need, part, whole):
            assert (p is None) if not want else torch.equal(p, q)


def test_no_tokens_and_no_outputs(sw, orc):
    import torch
    pr = Problem(sw, orc, 3, 64, 64, "group", 32, 8, 2)
    e = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ids = torch.empty(0, dtype=torch.int32, device="cuda")
    y, u = sw.linear_lora(e(0, 64), pr.P, pr.A, pr.B, ids, pr.scaling, return_u=True)
    assert y.shape == (0, 64) and u.shape == (0, 8)
    dX, dA, dB = sw.linear_lora_backward(e(0, 64), e(0, 64), pr.P, pr.A, pr.B, ids, u, pr.scaling)
    assert dX.shape == (0, 64) and not dA.any() and not dB.any()
    assert sw.linear_backward(e(0, 64), pr.P).shape == (0, 64)
    none = sw.PackedWeight(pr.P.idx[:0], pr.P.sgn[:0], pr.P.scales[:0], 0, 64, pr.P.granularity, 32)
    assert not sw.linear_backward(e(3, 0), none).any()
    dX, dA, dB = sw.linear_lora_backward(e(3, 0), pr.X, none, pr.A, e(2, 0, 8), pr.ids, u.new_zeros(3, 8), pr.scaling)
    assert not dX.any() and not dA.any() and dB.numel() == 0


def test_order_of_tokens_does_not_matter(sw, orc):
    """Each token's row depends on its own adapter only, whoever stands beside it."""
    import torch
    pr = Problem(sw, orc, 260, 200, 512, "group", 128, 16, 6, "mixed")
    y = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling)
    perm = torch.randperm(260, device="cuda")
    z = sw.linear_lora(pr.X[perm], pr.P, pr.A, pr.B, pr.ids[perm].long(), pr.scaling)
    bound = 2.0 ** -15 * pr.forward(True)[0].max()
    assert float((z - y[perm]).abs().max()) <= bound


def test_differences(sw, orc):
    """Y is linear in X, in A and in B: with f = sum(Y G), (f(B + E) - f(B - E)) / 2 is <dB, E>
    up to the outputs' rounding (E of B's size, so nothing cancels that rounding could hide in)."""
    import torch
    pr = Problem(sw, orc, 96, 160, 256, "tensor", 0, 16, 3, "mixed")
    _, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    grads = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, torch.float32)

    def f(X, A, B):
        y = sw.linear_lora(X.to(torch.bfloat16), pr.P, A.to(torch.bfloat16), B.to(torch.bfloat16), pr.ids, pr.scaling)
        return float((y.double() * pr.G.double()).sum())

    base = [pr.X, pr.A, pr.B]
    gen = torch.Generator(device="cuda").manual_seed(5)
    for i in range(3):
        sign = torch.where(torch.rand(base[i].shape, generator=gen, device="cuda") < 0.5, 1.0, -1.0)
        E = 2.0 ** -2 * float(base[i].float().abs().mean()) * sign
        plus, minus = [b.float() for b in base], [b.float() for b in base]
        plus[i], minus[i] = (plus[i] + E).to(torch.bfloat16).float(), (minus[i] - E).to(torch.bfloat16).float()
        step = (plus[i] - minus[i]).double() / 2  # the step that bf16 really took
        want = (f(*plus) - f(*minus)) / 2
        got = float((grads[i].double() * step).sum())
        # f's own error: 2^-15 of the magnitudes of its terms; dX is bf16 (2^-8 of each element)
        tol = 2.0 ** -15 * float((np.abs(pr.Gh) * pr.forward(True)[0]).sum())
        tol += 2.0 ** -8 * float((grads[i].double().abs() * step.abs()).sum()) if i == 0 else 0.0
        assert abs(want - got) <= tol, (i, want, got, tol)


def test_autograd(sw, orc):
    import torch
    pr = Problem(sw, orc, 70, 130, 256, "group", 128, 8, 3, "mixed")
    X, A, B = (t.clone().requires_grad_() for t in (pr.X, pr.A, pr.B))
    y = sw.linear_lora_train(X, pr.P, A, B, pr.ids, pr.scaling, torch.bfloat16)
    assert torch.equal(y, sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, torch.bfloat16))
    y.backward(pr.G)
    _, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling)
    assert torch.equal(X.grad, dX) and torch.equal(A.grad, dA) and torch.equal(B.grad, dB)
    # a broadcast (expanded) gradient, and only one leaf
    B2 = pr.B.clone().requires_grad_()
    sw.linear_lora_train(pr.X, pr.P, pr.A, B2, pr.ids, pr.scaling).sum().backward()
    ones = torch.ones_like(pr.G)
    want = sw.linear_lora_backward(ones, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling, need=(False, False, True))[2]
    assert torch.equal(B2.grad, want)


@pytest.mark.parametrize("M", [5, 300])
def test_other_forms_of_the_arguments(sw, orc, M):
    """Strided tensors, int64 ids, results into given tensors: converted, with the same bits."""
    import torch
    pr = Problem(sw, orc, M, 136, 512, "group", 128, 16, 3, "mixed")
    y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    grads = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling)

    def strided(t):
        wide = torch.full((*t.shape[:-1], 2 * t.shape[-1]), 7, dtype=t.dtype, device="cuda")
        wide[..., ::2] = t
        return wide[..., ::2]

    out = torch.empty_like(y)
    X, A, B, G, U, s, ids = (strided(t) for t in (pr.X, pr.A, pr.B, pr.G, u, pr.scaling, pr.ids.long()))
    far = torch.where(ids < 0, ids - 2 ** 40, ids)  # no adapter, beyond int32
    assert not X.is_contiguous() and not ids.is_contiguous()
    assert torch.equal(sw.linear_lora(X, pr.P, A, B, far, s, out=out), y) and torch.equal(out, y)
    y2, u2 = sw.linear_lora(X, pr.P, A, B, ids, s, return_u=True)
    assert torch.equal(y2, y) and torch.equal(u2, u)
    assert all(torch.equal(p, q) for p, q in zip(sw.linear_lora_backward(G, X, pr.P, A, B, ids, U, s), grads))
    dX = torch.empty_like(pr.X)
    assert torch.equal(sw.linear_backward(G, pr.P, out=dX), sw.linear_backward(pr.G, pr.P))


@pytest.mark.parametrize("M", [1, 4, 40, 300])
def test_calls_that_feed_one_another(sw, orc, M):
    """Layer after layer without a wait between them, each reading what the one before wrote: kernels
    start beside the end of others, and must not read ahead of them."""
    import torch
    pr = Problem(sw, orc, M, 1024, 1024, "group", 128, 16, 3, "mixed")
    bf = torch.bfloat16

    def chain(sync):
        x, us, out = pr.X, [], []
        for _ in range(6):
            y, u = sw.linear_lora(x, pr.P, pr.A, pr.B, pr.ids, pr.scaling, bf, return_u=True)
            if sync:
                torch.cuda.synchronize()
            us.append((x, u))
            x = y
            out.append(y)
        g = x
        for x, u in reversed(us):
            g, dA, dB = sw.linear_lora_backward(g, x, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling)
            if sync:
                torch.cuda.synchronize()
            out += [g, dA, dB]
        return out

    want = chain(True)
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(chain(False), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = chain(False)
    for _ in range(5):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_capture_of_a_permuted_call(sw, orc):
    """A replay whose ids make other slots, another order of tokens or none takes them as they then are."""
    import torch
    pr = Problem(sw, orc, 700, 130, 512, "group", 128, 16, 12, "mixed")
    g = torch.cuda.CUDAGraph()
    sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling)
    with torch.cuda.graph(g):
        y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
        grads = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling)
    for ids in (pr.ids.clone(), pr.ids.sort().values, torch.full_like(pr.ids, -1), torch.flip(pr.ids, [0])):
        pr.ids.copy_(ids)
        g.replay()
        torch.cuda.synchronize()
        want, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
        assert torch.equal(y, want) and torch.equal(u, U)
        again = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling)
        assert all(torch.equal(p, q) for p, q in zip(grads, again))


@pytest.mark.parametrize("M", [4, 40])
def test_capture_and_streams(sw, orc, M):
    """Two graphs of the call and eager calls on another stream share nothing; a replay sees new inputs."""
    import torch
    pr = Problem(sw, orc, M, 200, 512, "group", 128, 16, 3)
    want, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    wb = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
            grads = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling)
        graphs.append(g)
        outs.append((y, *grads))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s, g in zip((s1, s2), graphs):
        with torch.cuda.stream(s):
            for _ in range(3):
                g.replay()
    s3 = torch.cuda.Stream()
    with torch.cuda.stream(s3):
        eager = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling)
    torch.cuda.synchronize()
    assert torch.equal(eager, want)
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, (want, *wb)))
    pr.ids.copy_(torch.flip(pr.ids, [0]))
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling))
    with pytest.raises(RuntimeError, match="captured"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sw.linear_lora_train(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling)


def test_refusals(sw, orc):
    import torch
    pr = Problem(sw, orc, 4, 64, 256, "group", 128, 16, 3)
    ok = dict(X=pr.X, P=pr.P, A=pr.A, B=pr.B, ids=pr.ids, scaling=pr.scaling)
    bad = [dict(A=pr.A.float()), dict(A=pr.A[:, :, :128]), dict(B=pr.B[:, :32]), dict(B=pr.B[:2]), dict(ids=pr.ids[:3]),
           dict(ids=pr.ids.float()), dict(scaling=pr.scaling[:2]), dict(scaling=pr.scaling.double()),
           dict(A=pr.A[:, :12], B=pr.B[:, :, :12]), dict(X=pr.X.float()), dict(X=pr.X[:, :128]),
           dict(A=pr.A.cpu()), dict(out=torch.empty(4, 64, device="cuda", dtype=torch.bfloat16)),
           dict(out=torch.empty(4, 65, device="cuda")), dict(A=pr.A[:0], B=pr.B[:0], scaling=pr.scaling[:0])]
    for b in bad:
        with pytest.raises(ValueError):
            sw.linear_lora(**{**ok, **b})
    with pytest.raises(sw.SherryError):  # an adapter that starts off a 16-byte boundary
        flat = torch.zeros(pr.A.numel() + 1, dtype=torch.bfloat16, device="cuda")
        sw.linear_lora(**{**ok, "A": flat[1:].view(pr.A.shape)})
    U = torch.zeros(4, 16, device="cuda")
    for kw in (dict(U=U[:, :8]), dict(U=None), dict(U=U.double()), dict(dY=pr.G[:2]), dict(dY=pr.G.float())):
        with pytest.raises(ValueError):
            sw.linear_lora_backward(**{**dict(dY=pr.G, X=pr.X, P=pr.P, A=pr.A, B=pr.B, ids=pr.ids, U=U), **kw})
    with pytest.raises(ValueError):
        sw.linear_backward(pr.G[:, :32], pr.P)
