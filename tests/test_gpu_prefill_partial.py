"""Prefill with a last K-chunk that ends before the second decode group's steps, over many
tiles per CTA: that group must not run ahead of the other (needs a B200)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(128, 60000, 128), (128, 60000, 64), (256, 20000, 320), (200, 20000, 640)])
def test_partial_last_chunk_over_many_tiles(M, N, K):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_ternary_weight_b200.build import build
    build()
    import sparse_ternary_weight_b200 as sw
    g = torch.Generator(device="cuda").manual_seed(N + K)
    W = 0.05 * torch.randn((N, K), generator=g, device="cuda")
    X = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    P = sw.quantize_pack(W, "per_group", 64)
    Wq = sw.fake_quant(W, "per_group", 64)[0].double()
    ref = X.double() @ Wq.T
    bound = 2.0 ** -16 * (X.double().abs() @ Wq.abs().T)
    for _ in range(3):
        Y = sw.linear(X, P)
        assert sw.device_status() == 0
        assert bool(((Y.double() - ref).abs() <= bound).all())
