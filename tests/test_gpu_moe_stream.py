"""GPU parity: the streamed form of the few-row experts' kernels against the
float64 definition, at sizes whose weights take more stages than the ring has
slots, several rounds of slots, several segments of the contraction, a last stage
and a last block with fewer rows, and slots left out.  Each case states what its
plan has to be, so that a change of the shape rule cannot empty it."""
import pytest
import torch

import moe_plan
import moe_ref
from quantized_matmul_03_b200 import binding as qb

MODES = [("mxfp4", 32), ("nvfp4", 16), ("affine", 32), ("affine", 64), ("affine", 128)]
# T, k, K, I, N
SHAPES = [(1, 2, 4096, 4096, 8168), (3, 4, 4096, 4096, 3990), (5, 4, 2048, 2048, 2048), (1, 1, 1024, 5120, 1024)]


def wraps(p):
    return p is not None and p["rounds"] * p["nst"] > p["stages"]


@pytest.mark.parametrize("mode,gs", MODES)
def test_plans_of_these_shapes(mode, gs):
    seen = []
    for T, k, K, I, N in SHAPES:
        for C, R, glu in ((K, I, True), (I, N, False)):
            p = moe_plan.stream(C, R, T * k, mode, gs, glu)
            assert p is not None, "the kernel without a ring would take it"
            seen.append((glu, p))
    for glu in (True, False):
        some = [p for g, p in seen if g == glu]
        assert any(wraps(p) and p["S"] > 1 and p["rounds"] == 1 for p in some)
        assert any(wraps(p) and p["S"] > 1 and p["rounds"] > 1 for p in some)
        assert any(p["splits"] > 1 for p in some) and any(p["last"] for p in some)
        assert any(p["rows"] % p["rows_stage"] for p in some)


def test_the_rule_is_the_kernels():
    text = moe_plan.SRC.read_text()
    body = text[text.index("bool plan_stream"):text.index("cudaError_t launch_half")]
    for line in ("if (p.S > kMaxWarps || sb % 16 != 0) return false;",
                 "sp.slots_round = std::min(p.P, kMaxWarps / p.S);",
                 "p.row_splits = kMaxWarps / (sp.slots_round * p.S);",
                 "kPart = 32 * 1024, kRing = 220 * 1024 - kPart - 128;",
                 "rows = std::min<int64_t>(rows, kPart / ((int64_t)p.units * NM * 4));",
                 "std::min<int64_t>(rows, (int64_t)(kLoads / NM) * p.row_splits);",
                 "rs = std::min(rs, rows <= kRing / row_all ? rows : kRing / 3 / row_all);",
                 "sp.stages = (int)std::min<int64_t>(8, kRing / sp.stage_bytes);"):
        assert line in body


def packed(g, E, rows, cols, mode, gs, dtype):
    """A stack of random codes and scales, its weights of about 0.05."""
    wq = torch.randint(-2 ** 31, 2 ** 31, (E, rows, cols // 8), generator=g, device="cuda",
                       dtype=torch.int64).to(torch.int32)
    shape = (E, rows, cols // gs)
    if mode == "affine":
        s = ((0.5 + torch.rand(shape, generator=g, device="cuda")) * 0.01).to(dtype)
        return wq, s, (-7.5 * s.float()).to(dtype)
    lo, hi = (120, 123) if mode == "mxfp4" else (4, 15)
    s = torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    return wq, s, None


@pytest.mark.gpu
@pytest.mark.parametrize("path", ["gemv", "auto"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mode,gs", MODES)
@pytest.mark.parametrize("T,k,K,I,N", SHAPES)
def test_rings_that_wrap(path, dtype, mode, gs, T, k, K, I, N):
    E = 3
    g = torch.Generator(device="cuda").manual_seed(K + T)
    ws3 = [packed(g, E, r, c, mode, gs, dtype) for r, c in ((I, K), (I, K), (N, I))]
    x = torch.randn((T, K), generator=g, device="cuda").to(dtype)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    if T > 1:
        idx[1, k - 1] = -1
        idx[T - 1, 0] = -1
    w = torch.rand((T, k), generator=g, device="cuda") + 0.1
    out = torch.full((T + 1, N), 3.0, dtype=dtype, device="cuda")
    before = qb.qmm_launch_count()
    qb.qmm_set_path(path)
    try:
        y = qb.qmm_moe_experts(x, idx, w, *ws3, group_size=gs, mode=mode, out=out[:T])
        qb.qmm_device_status()
    finally:
        qb.qmm_set_path("auto")
    few = path == "gemv" or qb.qmm_launch_count() - before == 2  # the other path launches four kernels
    assert few or T > 1
    with torch.device("cuda"):
        ref, bound = moe_ref.experts(x, idx, w, *ws3, mode, gs, "silu", few_rows=few)
    err = (y.double() - ref).abs()
    assert bool((err <= bound).all()), f"worst {float((err / bound).max())} of the bound"
    # The bound adds up magnitudes, so at these lengths it is of the size of y.  Weights that are independent of
    # the activations' errors pass them on as they pass on the activations: in the norm, with the largest of 32
    # below 4 (x) and 8 (h) times the root mean square, g and u are off by 2^-12, h by 2.26 times that and its own
    # integers' 2^-11, and y is rounded; the tensor cores' operands (h, affine weights in three products) each
    # within half a step.  One row of a stage gone wrong is sqrt(2 / 8168) = 0.016 of y.
    half = torch.finfo(dtype).eps / 2
    tol = half * (1 if few else 5) + 2.0 ** -9
    assert bool((err.norm(dim=-1) <= tol * ref.norm(dim=-1)).all())
    assert bool((out[T] == 3).all())
