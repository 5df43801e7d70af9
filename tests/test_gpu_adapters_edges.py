"""Adapters, the input gradient and token log probabilities where they went wrong once:
each test names the fault that it keeps out (needs a B200)."""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_lora import Problem, check_dx, check_sum, host

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


# one and two 128-token halves per tile, rows split over CTAs or not, N that ends inside a stage
ROUNDED = [
    (1, 33, 256, "group", 128),
    (64, 512, 2048, "group", 128),
    (130, 100, 512, "channel", 0),
    (200, 1000, 320, "group", 32),
    (300, 65, 1024, "tensor", 0),
    (1500, 97, 6688, "group", 32),
    (1500, 160, 6656, "channel", 0),
]


@pytest.mark.parametrize("adapters", [False, True], ids=["plain", "adapters"])
@pytest.mark.parametrize("case", ROUNDED, ids=lambda c: f"M{c[0]}-{c[1]}x{c[2]}-{c[3]}{c[4]}")
def test_the_input_gradient_is_rounded_once(sw, orc, case, adapters):
    """The scales enter dX with (more than) fp32 sums' own error: what is left is one rounding to bf16, 2^-8
    of the value, beside 2^-15 of the terms' magnitudes for the fp32 sums and the split terms.  A scale rounded
    to bf16 would be off by up to 2^-8 of every term."""
    import torch
    M, N, K, gname, group = case
    pr = Problem(sw, orc, M, N, K, gname, group, 16, 3, "mixed")
    if adapters:
        dX = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, None, pr.scaling, torch.float32,
                                     need=(True, False, False))[0]
    else:
        dX = sw.linear_backward(pr.G, pr.P)
    assert sw.device_status() == 0
    base, extra, _, _ = pr.backward()
    mb, me, _, _ = pr.backward(True)
    ref = base + (extra if adapters else 0)
    sums = 2.0 ** -15 * (mb + (me if adapters else 0))
    err = np.abs(host(dX) - ref)
    assert np.all(err <= sums + 2.0 ** -8 * (np.abs(ref) + sums) + 1e-30), float((err / (sums + 2.0 ** -8 * np.abs(ref))).max())


def test_scales_far_apart_keep_their_own_precision(sw, orc):
    """Scales over 40 binades, zeros among them: each is kept to its own size, not to the largest's."""
    import torch
    pr = Problem(sw, orc, 40, 96, 512, "group", 128, 8, 2, "mixed")
    rng = np.random.default_rng(8)
    factor = 2.0 ** rng.integers(-30, 10, pr.P.scales.numel()).astype(np.float32)
    factor[::13] = 0.0
    pr.P.scales.mul_(torch.from_numpy(factor.astype(np.float32)).cuda())
    pr.W = pr.W * np.repeat(factor, 128).reshape(96, 512)
    dX = sw.linear_backward(pr.G, pr.P)
    base = pr.backward()[0]
    sums = 2.0 ** -15 * pr.backward(True)[0]
    err = np.abs(host(dX) - base)
    assert np.all(err <= sums + 2.0 ** -8 * (np.abs(base) + sums) + 1e-30)


def litter(value):
    """Freed memory full of `value`, where the next calls' scratch lies."""
    import torch
    junk = [torch.full((n,), value, dtype=torch.uint8, device="cuda") for n in (1 << 18, 1 << 20, 4 << 20, 32 << 20)]
    torch.cuda.synchronize()
    del junk


# more 128 x 128 tiles than SMs: several tiles per CTA, and phases that run on past adapters' chunks
MANY = [
    ("lead", 700, 4200, 256, "group", 128, 16, 3),
    ("lead", 700, 4200, 256, "channel", 0, 128, 3),
    ("lead", 900, 2700, 320, "group", 64, 72, 2),
    ("lead", 640, 4300, 4352, "group", 128, 24, 2),
    ("mixed", 700, 4200, 256, "group", 128, 16, 20),
    ("gaps", 1100, 2690, 512, "tensor", 0, 40, 4),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{c[0]}-M{c[1]}-{c[2]}x{c[3]}-{c[4]}{c[5]}-r{c[6]}x{c[7]}")
def test_more_tiles_than_sms(sw, orc, case, dt):
    """CTAs that begin with a tile of tokens without an adapter and go on to tiles that have one: the slots' masks
    are another kernel's results and are waited for all the same."""
    import torch
    kind, M, N, K, gname, group, R, n = case
    pr = Problem(sw, orc, M, N, K, gname, group, R, n, "mixed" if kind == "mixed" else "sorted")
    if kind != "mixed":
        pr.ids[:256] = -1
        pr.idsh[:256] = -1
        if kind == "gaps":
            pr.ids[512:768] = -1
            pr.idsh[512:768] = -1
    T = torch.float32 if dt == "f32" else torch.bfloat16
    ref, U = pr.forward()
    mag, Um = pr.forward(True)
    first = None
    for value in (0, 255, 85, 255):
        litter(value)
        y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, T, return_u=True)
        if first is None:
            first = (y, u)
            assert sw.device_status() == 0
            check_sum(y, ref, mag, "Y", bf16=dt == "bf16")
            check_sum(u, U, Um, "U")
        assert torch.equal(y, first[0]) and torch.equal(u, first[1])


@pytest.mark.parametrize("M", [90, 300])
def test_a_large_bank_for_few_tokens(sw, orc, M):
    """About as many slots as tokens: the scratch holds no more, and no token is lost."""
    import torch
    pr = Problem(sw, orc, M, 130, 256, "group", 128, 16, 1024, "mixed")
    ref, U = pr.forward()
    mag, Um = pr.forward(True)
    y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    assert sw.device_status() == 0
    check_sum(y, ref, mag, "Y")
    check_sum(u, U, Um, "U")
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling, torch.float32)
    assert sw.device_status() == 0
    check_dx(pr, dX)
    for got, want, size in zip((dA, dB), pr.backward()[2:], pr.backward(True)[2:]):
        check_sum(got, want, size, "gradient")


@pytest.mark.parametrize("M,n", [(384000, 2), (270000, 1), (150000, 700)])
def test_slots_by_the_thousand(sw, orc, M, n):
    """More slots than the plan holds in shared memory, in place and adapter by adapter; the plan's work is linear
    in them."""
    import torch
    pr = Problem(sw, orc, M, 8, 64, "group", 32, 8, n, "mixed")
    ref, U = pr.forward()
    mag, Um = pr.forward(True)
    y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    assert sw.device_status() == 0
    check_sum(y, ref, mag, "Y")
    check_sum(u, U, Um, "U")
    dX, dA, dB = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling, torch.float32)
    assert sw.device_status() == 0
    check_dx(pr, dX)
    for got, want, size in zip((dA, dB), pr.backward()[2:], pr.backward(True)[2:]):
        check_sum(got, want, size, "gradient")


def test_planes_of_another_form_are_refused(sw, orc):
    """By every call that takes a packed weight here, and before anything is launched."""
    import dataclasses

    import torch
    from tests.test_adapters_abi import bad_planes
    pr = Problem(sw, orc, 4, 64, 256, "group", 32, 16, 3)
    _, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    for kw in [*bad_planes(pr.P), dict(idx=pr.P.idx.cpu()), dict(sgn=pr.P.sgn.cpu()), dict(scales=pr.P.scales.cpu())]:
        P = dataclasses.replace(pr.P, **kw)
        G, B = (pr.G, pr.B) if P.N == 64 else (torch.zeros(4, P.N, dtype=torch.bfloat16, device="cuda"),
                                               torch.zeros(3, P.N, 16, dtype=torch.bfloat16, device="cuda"))
        for call in (lambda: sw.linear_lora(pr.X, P, pr.A, B, pr.ids, pr.scaling), lambda: sw.linear_backward(G, P),
                     lambda: sw.linear_lora_backward(G, pr.X, P, pr.A, B, pr.ids, U, pr.scaling),
                     lambda: sw.linear_logprobs(pr.X, P)):
            with pytest.raises(ValueError):
                call()


@pytest.mark.parametrize("what", ["head", "plain route"])
def test_large_scratch_is_given_back(sw, what):
    """A chunk's logits, and the fp32 Y under a bf16 one, do not outlive the call; their tickets are zeroed in
    memory that held anything before, in eager calls and in replayed ones."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(6)
    N, K = (140000, 128) if what == "head" else (20000, 96)
    P = sw.quantize_pack(0.05 * torch.randn((N, K), generator=gen, device="cuda"), "per_group", 32)
    X = torch.randn((300, K), generator=gen, device="cuda").to(torch.bfloat16)
    A = torch.randn((2, 8, K), generator=gen, device="cuda").to(torch.bfloat16)
    B = torch.randn((2, N, 8), generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, 2, (300,), generator=gen, device="cuda", dtype=torch.int32)

    def call():
        if what == "head":
            r = sw.linear_logprobs(X, P, ids, top=2)
            return [r.logp, r.entropy, r.top_ids]
        return [sw.linear_lora(X, P, A, B, ids, None, torch.bfloat16)]

    with torch.cuda.stream(torch.cuda.Stream()):
        before = torch.cuda.memory_allocated()
        want = call()
        kept = torch.cuda.memory_allocated() - before - sum(t.numel() * t.element_size() for t in want)
        assert kept <= 5 << 20, kept
        for value in (255, 1):
            litter(value)
            assert all(torch.equal(p, q) for p, q in zip(call(), want))
        torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert sw.device_status() == 0


@pytest.mark.parametrize("V,pad", [(1003, 0), (4097, 3), (50257, 64)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_rows_left_out_pass_nothing_on(sw, V, pad, dt):
    """Padding rows (target -1) may hold NaN and infinities: log p 0, and a gradient of exact zeros, not NaN."""
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((6, V + pad), generator=gen, device="cuda").to(T)[:, :V]
    t = torch.tensor([1, -1, 2, -1, V, 5], dtype=torch.int32, device="cuda")
    left = torch.tensor([1, 3, 4], device="cuda")
    g = torch.rand(6, generator=gen, device="cuda") + 0.5
    r = sw.token_logprobs(z, t)
    want = sw.token_logprobs_backward(z, t, r.stats, r.entropy, g)
    assert not want[left].any()
    z[1] = float("nan")
    z[3, ::3] = float("inf")
    z[4, 17] = float("nan")
    r = sw.token_logprobs(z, t)
    assert not r.logp[left].any() and bool(torch.isnan(r.entropy[left]).all())
    zero = torch.zeros(6, device="cuda")
    for got in (sw.token_logprobs_backward(z, t, r.stats, r.entropy, g), sw.token_logprobs_backward(z, t, r.stats, None, g),
                sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, zero),
                sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, out=torch.full_like(z, 7.0))):
        assert torch.equal(got, want)
    x = z.clone().requires_grad_()
    (sw.token_logprobs_train(x, t)[0] * g).sum().backward()
    # (a copy without the padding: its rows are aligned otherwise, so their sums have another order; the same bits
    # as the explicit calls on that copy)
    rx = sw.token_logprobs(x.detach(), t)
    assert torch.equal(x.grad, sw.token_logprobs_backward(x.detach(), t, rx.stats, None, g)) and not x.grad[left].any()
    # with an entropy gradient of its own the row counts, and shows its NaN
    h = zero.clone()
    h[1] = 1.0
    assert bool(torch.isnan(sw.token_logprobs_backward(z, t, r.stats, r.entropy, g, h)[1]).all())


@pytest.mark.parametrize("what", ["adapters", "log probabilities"])
def test_the_backward_pass_of_an_eager_call_is_not_captured(sw, orc, what):
    """Refused as the capture of the whole step is; the graph that was built stays usable."""
    import torch
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        pr = Problem(sw, orc, 6, 64, 256, "group", 128, 8, 2)
        leaf = (pr.A if what == "adapters" else pr.G).clone().requires_grad_()
        if what == "adapters":
            y = sw.linear_lora_train(pr.X, pr.P, leaf, pr.B, pr.ids, pr.scaling)
        else:
            y = sw.token_logprobs_train(leaf, pr.ids)[0]
        dy = torch.ones_like(y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="captured"):
            with torch.cuda.graph(graph, stream=s):
                y.backward(dy, retain_graph=True)
        assert leaf.grad is None
        y.backward(dy)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(leaf.grad).all()) and bool(leaf.grad.any())


@pytest.mark.parametrize("M", [1, 5, 33000])
def test_u_of_a_weight_without_rows(sw, orc, M):
    """U = s_a X A_a^T does not depend on the weight's rows: it is the same beside none."""
    import torch
    pr = Problem(sw, orc, M, 8, 64, "group", 32, 8, 3, "mixed")
    none = sw.PackedWeight(pr.P.idx[:0], pr.P.sgn[:0], pr.P.scales[:0], 0, 64, pr.P.granularity, 32)
    litter(255)
    y, u = sw.linear_lora(pr.X, none, pr.A, pr.B[:, :0], pr.ids, pr.scaling, return_u=True)
    assert sw.device_status() == 0 and y.shape == (M, 0)
    check_sum(u, pr.forward()[1], pr.forward(True)[1], "U")


@pytest.mark.parametrize("N", [129, 130, 132, 136])
def test_gradients_of_a_slice_of_a_batch(sw, orc, N):
    """Rows of dY that start off a 16-byte boundary, as any row of an odd length does."""
    import torch
    pr = Problem(sw, orc, 40, N, 256, "group", 128, 16, 3, "mixed")
    _, U = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, return_u=True)
    want = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling)
    plain = sw.linear_backward(pr.G, pr.P)
    for first in (1, 2, 3):
        rows = torch.full((first + 40, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        rows[first:] = pr.G
        G = rows[first:]
        assert G.is_contiguous()
        got = sw.linear_lora_backward(G, pr.X, pr.P, pr.A, pr.B, pr.ids, U, pr.scaling)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
        assert torch.equal(sw.linear_backward(G, pr.P), plain)
    # under autograd: two calls' outputs put together
    A = pr.A.clone().requires_grad_()
    part = lambda a, b: sw.linear_lora_train(pr.X[a:b], pr.P, A, pr.B, pr.ids[a:b], pr.scaling, torch.bfloat16)  # noqa: E731
    torch.cat([part(0, 3), part(3, 40)]).backward(pr.G)
    both = [sw.linear_lora_backward(pr.G[a:b], pr.X[a:b], pr.P, pr.A, pr.B, pr.ids[a:b], U[a:b], pr.scaling)[1]
            for a, b in ((0, 3), (3, 40))]
    # (the order of the two is autograd's: a sum of two bf16 numbers does not depend on it)
    assert torch.equal(A.grad, both[0] + both[1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_no_probability_above_one(sw, dt):
    """Rows that leave one token, or one far above the rest: log S >= 0 and log p <= 0, near 0 for
    maxima of every size.  Up to 1e8 the rounding of m log2(e) is at most 4 (half a step at 2^27), so S = 2^y with
    |y| <= 4: the exponential is off by 2^-22 of itself, its logarithm (up to 2.8) by one step, 2^-22, and the
    product that takes y ln 2 back out by two half steps of 2.8 and ln 2's own, 3 x 2^-23: 2^-20 in all."""
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(3)
    size = 10.0 ** torch.linspace(-6, 7.9, 3000, device="cuda")
    z = torch.full((3000, 40), float("-inf"), dtype=T, device="cuda")
    lead = torch.where(torch.rand(3000, generator=gen, device="cuda") < 0.5, -size, size).to(T)
    t = torch.randint(0, 40, (3000,), generator=gen, device="cuda", dtype=torch.int32)
    z.scatter_(1, t.long()[:, None], lead[:, None])
    z[::3] = torch.where(torch.isinf(z[::3]), (lead[::3, None].float() - 200 - 2 * lead[::3, None].float().abs()).to(T), z[::3])
    for x, y in ((z, t), (z[:1], t[:1]), (lead[:, None].contiguous(), torch.zeros_like(t))):
        r = sw.token_logprobs(x, y, top=1)
        assert bool((r.stats[:, 1] >= 0).all()) and bool((r.logp <= 0).all()) and bool((r.top_logp <= 0).all())
        assert float(r.logp.min()) >= -2.0 ** -20 and float(r.entropy.max()) <= 2.0 ** -20 and float(r.entropy.min()) >= 0


def test_results_into_what_is_read_are_refused(sw, orc):
    """A square layer's input has its output's shape: writing over it would feed other tiles half of it."""
    import torch
    pr = Problem(sw, orc, 300, 256, 256, "group", 128, 16, 3, "mixed")
    bf = torch.bfloat16
    buf = torch.zeros(310, 256, dtype=bf, device="cuda")
    buf[:300] = pr.X
    X = buf[:300]
    for out in (X, buf[10:], buf[5:305]):
        with pytest.raises(ValueError, match="overlap"):
            sw.linear_lora(X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, bf, out=out)
        with pytest.raises(ValueError, match="overlap"):
            sw.linear_backward(X, pr.P, out=out)
    two = torch.zeros(600, 256, dtype=bf, device="cuda")
    two[:300] = pr.X
    want = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, bf)
    assert torch.equal(sw.linear_lora(two[:300], pr.P, pr.A, pr.B, pr.ids, pr.scaling, bf, out=two[300:]), want)
    empty = torch.empty(0, 256, dtype=bf, device="cuda")
    assert sw.linear_backward(empty, pr.P, out=empty) is empty


@pytest.mark.parametrize("R,dt", [(128, "f32"), (64, "f32"), (16, "bf16")])
def test_calls_at_once_on_two_streams(sw, orc, R, dt):
    """Forward and backward of two problems side by side, with and without dX, again and again: kernels of both
    share SMs, and each stream's results are those of the calls alone."""
    import torch
    T = torch.float32 if dt == "f32" else torch.bfloat16
    prs = [Problem(sw, orc, 300, 384, 1024, "group", 128, R, 3, "mixed"), Problem(sw, orc, 900, 640, 512, "channel", 0, R, 9, "mixed")]

    def step(pr):
        y, u = sw.linear_lora(pr.X, pr.P, pr.A, pr.B, pr.ids, pr.scaling, T, return_u=True)
        a = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling, T, need=(False, True, True))
        b = sw.linear_lora_backward(pr.G, pr.X, pr.P, pr.A, pr.B, pr.ids, u, pr.scaling, T)
        return [y, u, *a[1:], *b]

    want = [step(pr) for pr in prs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(prs[i]))
    torch.cuda.synchronize()
    assert sw.device_status() == 0
    for i in range(2):
        for outs in got[i]:
            assert all(torch.equal(p, q) for p, q in zip(outs, want[i]))
