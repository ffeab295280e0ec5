"""qmm_moe_experts and its workspace size agree on the sizes they take."""
import pytest
import torch

from quantized_matmul_03_b200 import binding as qb
from test_moe_abi import L, UNSUPPORTED, WORKSPACE, experts  # noqa: F401  (L: fixture)


@pytest.mark.parametrize("T,K,k,E,I,N", [
    (1, 64, 1, 1, 64, 2 ** 24), (1, 64, 1, 1, 64, 2 ** 24 + 64), (1, 64, 1, 1, 64, 2 ** 30), (1, 64, 2, 4, 64, 2 ** 28),
    (1, 2 ** 24, 1, 1, 2 ** 24, 64), (2 ** 25, 64, 32, 1, 64, 64), (1, 64, 1, 1024, 2 ** 20, 2 ** 20)])
def test_a_size_for_every_call_that_is_taken(L, T, K, k, E, I, N):
    need = L.qmm_moe_experts_workspace_size(T, K, k, E, I, N, 1)
    assert need > 0
    assert experts(L, T=T, K=K, k=k, E=E, I=I, N=N, wsb=need - 1) == WORKSPACE


@pytest.mark.parametrize("T,K,k,E,I,N", [
    (1, 64, 1, 1, 64, 2 ** 30 + 1), (1, 64, 1, 4, 64, 2 ** 28 + 1), (1, 2 ** 24 + 64, 1, 1, 64, 64),
    (1, 64, 1, 1, 2 ** 24 + 64, 64), (2 ** 25 + 1, 64, 32, 1, 64, 64), (1, 64, 1, 1024, 2 ** 20 + 64, 64),
    (1, 64, 1, 3, 64, 2 ** 62), (1, 64, 1, 1024, 2 ** 62, 64)])
def test_none_for_a_call_that_is_refused(L, T, K, k, E, I, N):
    assert L.qmm_moe_experts_workspace_size(T, K, k, E, I, N, 1) == 0
    assert experts(L, T=T, K=K, k=k, E=E, I=I, N=N) == UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("path", ["gemv", "gemm"])
def test_more_than_2_24_output_columns(path):
    """A stack with more rows than 2^24 gives the columns that its last rows alone give."""
    N, K = 2 ** 24 + 1000, 64
    g = torch.Generator(device="cuda").manual_seed(1)

    def w(rows):
        wq = torch.randint(-2 ** 31, 2 ** 31, (1, rows, K // 8), generator=g, device="cuda", dtype=torch.int64)
        s = torch.randint(120, 124, (1, rows, K // 32), generator=g, device="cuda", dtype=torch.int32)
        return wq.to(torch.int32), s.to(torch.uint8), None

    gate, up, down = w(64), w(64), w(N)
    x = torch.randn((2, K), generator=g, device="cuda").bfloat16()
    idx, wt = torch.zeros((2, 1), dtype=torch.int32, device="cuda"), torch.ones((2, 1), device="cuda")
    qb.qmm_set_path(path)
    try:
        y = qb.qmm_moe_experts(x, idx, wt, gate, up, down, group_size=32, mode="mxfp4")
        tail = tuple(None if t is None else t[:, N - 2048:].contiguous() for t in down)
        want = qb.qmm_moe_experts(x, idx, wt, gate, up, tail, group_size=32, mode="mxfp4")
        qb.qmm_device_status()
    finally:
        qb.qmm_set_path("auto")
    assert torch.equal(y[:, N - 2048:], want) and bool((want != 0).any())
