"""GPU parity: the experts' layer over every finite scale byte of the microscaled
modes, and NaN scales, against the float64 definition.

One expert per byte, one token per expert.  In mxfp4 the activations run against
the gate's and up's scales so that the products stay in range, and the routing
weights against down's.  On the tensor cores a weight is the nearest value of the
dtype, which the reference's weights are rounded to there."""
import pytest
import torch

import moe_ref
from quantized_matmul_03_b200 import binding as qb

pytestmark = pytest.mark.gpu
PATHS = ["gemv", "gemm"]


def codes(g, E, rows, cols):
    return torch.randint(-2 ** 31, 2 ** 31, (E, rows, cols // 8), generator=g, device="cuda",
                         dtype=torch.int64).to(torch.int32)


def stack(g, rows, cols, gs, byte):
    """One expert per entry of `byte`, all of its scales that byte."""
    s = byte.to(torch.uint8).view(-1, 1, 1).expand(-1, rows, cols // gs).contiguous()
    return codes(g, len(byte), rows, cols), s, None


def compare(monkeypatch, path, x, w, ws3, mode, gs):
    T = x.shape[0]
    idx = torch.arange(T, dtype=torch.int32, device="cuda").view(T, 1)
    qb.qmm_set_path(path)
    try:
        y = qb.qmm_moe_experts(x, idx, w, *ws3, group_size=gs, mode=mode)
        qb.qmm_device_status()
    finally:
        qb.qmm_set_path("auto")
    if path == "gemm":
        exact = moe_ref.dense
        monkeypatch.setattr(moe_ref, "dense", lambda *a: exact(*a).to(x.dtype).double())
    with torch.device("cuda"):
        ref, bound = moe_ref.experts(x, idx, w, *ws3, mode, gs, "silu", few_rows=path == "gemv")
    assert bool(torch.isfinite(ref).all()) and float(ref.abs().max()) < torch.finfo(x.dtype).max / 4
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), (f"worst {float((err / bound).nan_to_num(9e9).max())} of the bound, tokens "
                                        f"{torch.nonzero(~(err <= bound).all(-1)).view(-1).tolist()}")
    return ref


def bytes_of(lo, hi):
    return torch.arange(lo, hi + 1, device="cuda")


def pow2(e):
    return torch.exp2(e.double()).float()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,I", [(512, 512), (192, 64)])   # streamed by the few-row path, and not
def test_e8m0_of_gate_and_up(monkeypatch, path, dtype, K, I):
    """bf16: all bytes, but for 253 and 254 on the tensor cores, whose larger weights
    are past bf16's largest value.  f16: bytes whose weights are f16 values or below
    its smallest (there the products are next to nothing and must be so)."""
    g = torch.Generator(device="cuda").manual_seed(K)
    if dtype == torch.bfloat16:
        b = bytes_of(0, 252 if path == "gemm" else 254)
        x_exp = (127 - b).clamp(-110, 126)
    else:
        b = bytes_of(0, 140)
        x_exp = (127 - b).clamp(-14, 14)
    x = ((torch.rand((len(b), K), generator=g, device="cuda") * 2 - 1) * pow2(x_exp)[:, None]).to(dtype)
    ws3 = (stack(g, I, K, 32, b), stack(g, I, K, 32, b), stack(g, 64, I, 32, torch.full_like(b, 115)))
    w = torch.full((len(b), 1), 2.0 ** -8, device="cuda")
    ref = compare(monkeypatch, path, x, w, ws3, "mxfp4", 32)
    small = 0 if dtype == torch.bfloat16 else 110
    assert bool((ref.abs().amax(-1)[small:] > 1e-4).all())


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("I", [512, 64])
def test_e8m0_of_down(monkeypatch, path, dtype, I):
    """Bytes up to 230 (f16 on the tensor cores 140): beyond, fp32 sums of a slot overflow."""
    g = torch.Generator(device="cuda").manual_seed(I)
    b = bytes_of(0, 140 if dtype == torch.float16 and path == "gemm" else 230)
    K = 256
    x = torch.randn((len(b), K), generator=g, device="cuda").to(dtype)
    n = torch.full_like(b, 121)
    ws3 = (stack(g, I, K, 32, n), stack(g, I, K, 32, n), stack(g, 72, I, 32, b))
    w = pow2((127 - b).clamp(-126, 126)).view(-1, 1)
    compare(monkeypatch, path, x, w, ws3, "mxfp4", 32)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("K,I", [(512, 512), (192, 64)])
def test_e4m3_of_both_signs(monkeypatch, path, dtype, K, I):
    """Every byte but the two NaN, subnormals, both zeros and the sign bit included,
    each beside others in gate, up and down."""
    g = torch.Generator(device="cuda").manual_seed(K + 1)
    b = bytes_of(0, 255)
    b = b[(b & 127) != 127]
    perm = [b[torch.randperm(len(b), generator=g, device="cuda")] for _ in range(2)]
    x = (torch.randn((len(b), K), generator=g, device="cuda") * 2.0 ** -9).to(dtype)
    ws3 = (stack(g, I, K, 16, b), stack(g, I, K, 16, perm[0]), stack(g, 72, I, 16, perm[1]))
    w = torch.full((len(b), 1), 2.0 ** -14, device="cuda")
    compare(monkeypatch, path, x, w, ws3, "nvfp4", 16)
    mixed = []                                             # and all of them within one expert
    for rows, cols in ((I, K), (I, K), (72, I)):
        s = b[torch.randint(0, len(b), (4, rows, cols // 16), generator=g, device="cuda")]
        mixed.append((codes(g, 4, rows, cols), s.to(torch.uint8), None))
    compare(monkeypatch, path, x[:4], w[:4], mixed, "nvfp4", 16)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mode,gs,byte", [("nvfp4", 16, 0x7F), ("nvfp4", 16, 0xFF), ("mxfp4", 32, 0xFF)])
@pytest.mark.parametrize("K,I", [(512, 512), (192, 64)])
def test_one_nan_scale(path, dtype, mode, gs, byte, K, I):
    """One group of one up row of expert 1 and of one down row of expert 2: their
    tokens' outputs, or that output, are NaN; the other experts' are what they were."""
    g = torch.Generator(device="cuda").manual_seed(byte)
    ordinary = torch.full((4,), 10 if mode == "nvfp4" else 121, device="cuda")
    ws3 = (stack(g, I, K, gs, ordinary), stack(g, I, K, gs, ordinary), stack(g, 72, I, gs, ordinary))
    x = torch.randn((8, K), generator=g, device="cuda").to(dtype)
    idx = torch.arange(8, dtype=torch.int32, device="cuda").view(8, 1) % 4
    w = torch.ones((8, 1), device="cuda")
    qb.qmm_set_path(path)
    try:
        clean = qb.qmm_moe_experts(x, idx, w, *ws3, group_size=gs, mode=mode)
        ws3[1][1][1, I - 1, K // gs - 1] = byte
        ws3[2][1][2, 70, 0] = byte
        y = qb.qmm_moe_experts(x, idx, w, *ws3, group_size=gs, mode=mode)
        qb.qmm_device_status()
    finally:
        qb.qmm_set_path("auto")
    assert bool(torch.isfinite(clean).all())
    nan = torch.isnan(y)
    want = torch.zeros_like(nan)
    want[1::4] = True
    want[2::4, 70] = True
    assert torch.equal(nan, want)
    assert torch.equal(y[~want], clean[~want])
