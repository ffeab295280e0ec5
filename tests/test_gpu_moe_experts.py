"""GPU parity: qmm_moe_experts against the float64 definition, within the sum of
the roundings the header names (tests/moe_ref.py derives the bound)."""
import math

import pytest
import torch

import moe_ref
from quantized_matmul_03_b200 import binding as qb

pytestmark = pytest.mark.gpu

MODES = [("mxfp4", 32), ("nvfp4", 16), ("affine", 32), ("affine", 64), ("affine", 128)]
PATHS = ["gemv", "gemm"]
FEW = ["gemv"]


@pytest.fixture(autouse=True)
def _auto_path():
    yield
    qb.qmm_set_path("auto")


def layer(E, K, I, N, mode, gs, dtype, seed):
    g = torch.Generator().manual_seed(seed)

    def w(rows, cols):
        v = torch.randn((E, rows, cols), generator=g) * cols ** -0.5
        if mode == "nvfp4":
            v = v * 64          # group scales in E4M3's normal range
        return moe_ref.quantize(v.to(dtype), gs, mode)

    return w(I, K), w(I, K), w(N, I)


def slots(T, k, E, seed, dropped=0.0):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] if k <= E else torch.randint(0, E, (k,), generator=g)
                       for _ in range(T)]).to(torch.int32) if T else torch.empty((0, k), dtype=torch.int32)
    idx[torch.rand((T, k), generator=g) < dropped] = -1
    return idx, torch.rand((T, k), generator=g) + 0.1


def cu(packed):
    return tuple(None if t is None else t.cuda() for t in packed)


def run(x, idx, w, ws3, mode, gs, act="silu", path="auto", **kw):
    qb.qmm_set_path(path)
    y = qb.qmm_moe_experts(x.cuda(), idx.cuda(), w.cuda(), *map(cu, ws3), group_size=gs, bits=4, mode=mode,
                           activation=act, **kw)
    qb.qmm_device_status()
    return y


def check(x, idx, w, ws3, mode, gs, act="silu", path="gemv"):
    y = run(x, idx, w, ws3, mode, gs, act, path)
    ref, bound = moe_ref.experts(x, idx, w, *ws3, mode, gs, act, few_rows=path in FEW)
    assert y.dtype == x.dtype
    yd = y.cpu().double()
    # A value past the type's largest rounds to infinity of its sign.
    past = ref.abs() + bound > torch.finfo(x.dtype).max
    err = torch.where(past & torch.isinf(yd) & (yd.sign() == ref.sign()), 0.0, (yd - ref).abs())
    assert bool((err <= bound).all()), f"worst {float((err / bound).max())} of the bound"
    return y


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mode,gs", MODES)
@pytest.mark.parametrize("T,k,E,K,I,N", [(1, 2, 4, 128, 128, 128), (3, 3, 5, 1152, 384, 200), (7, 1, 3, 256, 1280, 77)])
def test_small_layers(path, dtype, mode, gs, T, k, E, K, I, N):
    ws3 = layer(E, K, I, N, mode, gs, dtype, T + K)
    idx, w = slots(T, k, E, T)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(1)).to(dtype)
    check(x, idx, w, ws3, mode, gs, "silu" if T != 3 else "gelu_tanh", path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("mode,gs", [("mxfp4", 32), ("nvfp4", 16), ("affine", 64)])
def test_odd_blocks_of_64(path, mode, gs):
    """Contractions that end inside a 128-element stage and a 1024-element unit."""
    for K, I in ((64, 64), (192, 320), (1088, 704)):
        ws3 = layer(3, K, I, 40, mode, gs, torch.bfloat16, K)
        idx, w = slots(9, 2, 3, K)
        x = torch.randn((9, K), generator=torch.Generator().manual_seed(2)).bfloat16()
        check(x, idx, w, ws3, mode, gs, "silu", path)


@pytest.mark.parametrize("mode,gs", MODES)
@pytest.mark.parametrize("T,E,K,I,N", [(40, 3, 1024, 512, 96), (700, 3, 512, 1024, 130), (650, 2, 320, 192, 200),
                                       (395, 2, 64, 1088, 64)])
def test_low_and_tall_chunks(mode, gs, T, E, K, I, N):
    """Many rows per expert: chunks of every height, rows of scales in whole and in
    broken windows, contractions of 1 to 17 blocks of 64."""
    dtype = torch.float16 if mode == "mxfp4" else torch.bfloat16
    if K % gs or I % gs:
        pytest.skip("groups do not divide the contraction")
    ws3 = layer(E, K, I, N, mode, gs, dtype, T)
    idx, w = slots(T, 2, E, T + 1, dropped=0.2)
    idx[: T // 3, 0] = 0                          # unequal experts
    idx[: T // 3, 1] = -1
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T + 2)).to(dtype)
    check(x, idx, w, ws3, mode, gs, "silu", "gemm")


@pytest.mark.parametrize("mode,gs,E,k,T,K,I", [("mxfp4", 32, 32, 2, 2048, 1024, 2048), ("nvfp4", 16, 8, 2, 1024, 512, 4096),
                                               ("affine", 64, 24, 4, 200, 1024, 1024)])
def test_many_tiles_per_block(mode, gs, E, k, T, K, I):
    """Every thread block works through many tiles, its epilogue behind its MMAs."""
    ws3 = layer(E, K, I, K, mode, gs, torch.bfloat16, E)
    idx, w = slots(T, k, E, T)
    x = torch.randn((T, K), generator=torch.Generator().manual_seed(T)).bfloat16()
    dev = tuple(map(cu, ws3))
    ref, bound = moe_ref.experts(x.cuda(), idx.cuda(), w.cuda(), *ws3, mode, gs, "silu", few_rows=False)
    first = None
    for _ in range(3):
        y = run(x, idx, w, dev, mode, gs, path="gemm")
        assert bool(((y.double() - ref).abs() <= bound).all())
        first = y if first is None else first
        assert torch.equal(first, y)


@pytest.mark.parametrize("mode,gs", [("mxfp4", 32), ("affine", 128)])
@pytest.mark.parametrize("K,I", [(17408, 64), (128, 17408), (20544, 128)])
def test_long_contractions_of_the_few_row_path(mode, gs, K, I):
    """More segments than the streamed kernel holds results for."""
    if K % gs or I % gs:
        pytest.skip("groups do not divide the contraction")
    ws3 = layer(2, K, I, 70, mode, gs, torch.bfloat16, K)
    idx, w = slots(3, 2, 2, I)
    x = torch.randn((3, K), generator=torch.Generator().manual_seed(I)).bfloat16()
    check(x, idx, w, ws3, mode, gs, "silu", "gemv")


def test_contraction_past_the_few_row_path():
    """32 slots of one token over a contraction whose partial sums the few-row
    kernels have no room for: refused there, taken by the automatic path."""
    K, k = 393216 + 1024, 32
    g = torch.Generator().manual_seed(26)
    wq = [torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=g, dtype=torch.int64).to(torch.int32)
          for s in ((1, 64, K // 8), (1, 64, K // 8), (1, 64, 8))]
    ws3 = tuple((q, torch.full((1, 64, q.shape[2] // 4), 118, dtype=torch.uint8), None) for q in wq)
    idx, w = torch.zeros((1, k), dtype=torch.int32), torch.rand((1, k), generator=g) + 0.1
    x = (torch.randn((1, K), generator=g) * 2.0 ** -6).bfloat16()
    with pytest.raises(qb.QmmError) as e:
        run(x, idx, w, ws3, "mxfp4", 32, path="gemv")
    assert e.value.status == 2
    check(x, idx, w, ws3, "mxfp4", 32, "silu", "auto")


@pytest.mark.parametrize("path", PATHS)
def test_most_experts(path):
    E, k = 1024, 8
    ws3 = layer(E, 64, 64, 40, "mxfp4", 32, torch.bfloat16, 22)
    idx, w = slots(60, k, E, 23)
    x = torch.randn((60, 64), generator=torch.Generator().manual_seed(24)).bfloat16()
    check(x, idx, w, ws3, "mxfp4", 32, "silu", path)


def test_automatic_path_is_one_of_the_two():
    ws3 = layer(8, 512, 512, 256, "mxfp4", 32, torch.bfloat16, 25)
    for T, path in ((1, "gemv"), (200, "gemm")):
        idx, w = slots(T, 2, 8, T)
        x = torch.randn((T, 512), generator=torch.Generator().manual_seed(T)).bfloat16()
        assert torch.equal(run(x, idx, w, ws3, "mxfp4", 32), run(x, idx, w, ws3, "mxfp4", 32, path=path))


@pytest.mark.parametrize("path", PATHS)
def test_slots_left_out(path):
    ws3 = layer(4, 128, 128, 64, "mxfp4", 32, torch.bfloat16, 3)
    idx, w = slots(40, 3, 4, 4, dropped=0.3)
    idx[5] = -1                                   # nothing is left of this token
    idx[6] = torch.tensor([2, 2, 2])              # one expert three times
    w[7] = torch.tensor([math.nan, 1.0, 1.0])     # the weight of a slot left out is not looked at
    idx[7] = torch.tensor([-1, 0, 1])
    x = torch.randn((40, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    y = check(x, idx, w, ws3, "mxfp4", 32, "silu", path)
    assert bool((y[5] == 0).all())
    none = torch.full_like(idx, -1)
    assert bool((run(x, none, w, ws3, "mxfp4", 32, path=path) == 0).all())


@pytest.mark.parametrize("path", PATHS)
def test_index_out_of_range_is_reported(path):
    ws3 = layer(4, 128, 128, 64, "mxfp4", 32, torch.bfloat16, 3)
    idx, w = slots(40, 2, 4, 4)
    bad = idx.clone()
    bad[3, 1] = 4
    bad[9, 0] = -2
    bad[11, 0] = 2 ** 31 - 1
    x = torch.randn((40, 128), generator=torch.Generator().manual_seed(5)).bfloat16()
    with pytest.raises(qb.QmmError) as e:
        run(x, bad, w, ws3, "mxfp4", 32, path=path)
    assert e.value.status == 5
    qb.qmm_device_status()                        # cleared
    want = idx.clone()
    want[3, 1] = want[9, 0] = want[11, 0] = -1
    y = qb.qmm_moe_experts(x.cuda(), bad.cuda(), w.cuda(), *map(cu, ws3), group_size=32, mode="mxfp4")
    with pytest.raises(qb.QmmError):
        qb.qmm_device_status()
    assert torch.equal(y, run(x, want, w, ws3, "mxfp4", 32, path=path))


@pytest.mark.parametrize("path", PATHS)
def test_nan_stays_where_it_is(path):
    """A NaN in one token, and NaN weights of an expert that nobody chose, reach no
    other token."""
    gate, up, down = layer(3, 128, 128, 64, "mxfp4", 32, torch.bfloat16, 6)
    for w_ in (gate, up, down):
        w_[1][1] = 255                            # E8M0's NaN over all of expert 1
    idx = torch.tensor([[0, 2]] * 20, dtype=torch.int32)
    w = torch.rand((20, 2), generator=torch.Generator().manual_seed(7)) + 0.1
    x = torch.randn((20, 128), generator=torch.Generator().manual_seed(8)).bfloat16()
    clean = run(x, idx, w, (gate, up, down), "mxfp4", 32, path=path)
    assert bool(torch.isfinite(clean).all())
    x[4, 9] = math.nan
    x[12, 100] = math.inf
    y = run(x, idx, w, (gate, up, down), "mxfp4", 32, path=path)
    rest = [t for t in range(20) if t not in (4, 12)]
    assert torch.equal(y[rest], clean[rest])
    assert not bool(torch.isfinite(y[4]).any()) and not bool(torch.isfinite(y[12]).any())
    idx[3, 0] = 1
    y = run(x, idx, w, (gate, up, down), "mxfp4", 32, path=path)
    assert bool(torch.isnan(y[3]).all())
    rest = [t for t in rest if t != 3]
    assert torch.equal(y[rest], clean[rest])


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("mode,gs", [("mxfp4", 32), ("nvfp4", 16)])
def test_scales_far_from_one(path, dtype, mode, gs):
    """Group scales over their range: E8M0 above 2, tiny ones, zero codes; E4M3
    scales of 4 and more, subnormal and zero ones."""
    E, K, I, N = 2, 256, 128, 48
    g = torch.Generator().manual_seed(9)

    def w(rows, cols, lo, hi):
        wq = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, rows, cols // 8), generator=g, dtype=torch.int64).to(torch.int32)
        s = torch.randint(lo, hi, (E, rows, cols // gs), generator=g, dtype=torch.int32).to(torch.uint8)
        return wq, s, None

    if mode == "mxfp4":
        ws3 = (w(I, K, 100, 136), w(I, K, 118, 130), w(N, I, 90, 128))
    else:
        ws3 = (w(I, K, 0, 90), w(I, K, 0, 70), w(N, I, 0, 30))
    x = (torch.randn((6, K), generator=g) * 2.0 ** -9).to(dtype)
    idx, wt = slots(6, 2, 2, 10)
    wt *= 2.0 ** -6
    ref, _ = moe_ref.experts(x, idx, wt, *ws3, mode, gs, "silu", few_rows=True)
    assert float(ref.abs().max()) < torch.finfo(dtype).max / 4
    check(x, idx, wt, ws3, mode, gs, "silu", path)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("gs", [32, 128])
def test_affine_scales_of_every_size(path, dtype, gs):
    """Scales of both signs from 2^-12 to 2^2, and zero, beside each other in a row.
    (Biases keep the weights among the normal f16 values, where a rounding is
    relative to the weight.)"""
    E, K, I, N = 2, 256, 128, 48
    g = torch.Generator().manual_seed(27)

    def w(rows, cols):
        wq = torch.randint(-2 ** 31, 2 ** 31 - 1, (E, rows, cols // 8), generator=g, dtype=torch.int64).to(torch.int32)
        s = torch.exp2(torch.randint(-12, 3, (E, rows, cols // gs), generator=g).float()) * (1 + torch.rand((E, rows, cols // gs), generator=g))
        s = torch.where(torch.rand(s.shape, generator=g) < 0.5, -s, s)
        s[torch.rand(s.shape, generator=g) < 0.05] = 0.0
        b = torch.where(s < 0, -1.0, 1.0) * (2.0 ** -9 + torch.rand(s.shape, generator=g) * 2.0 ** -3)
        return wq, s.to(dtype), b.to(dtype)

    ws3 = (w(I, K), w(I, K), w(N, I))
    x = (torch.randn((6, K), generator=g) * 2.0 ** -9).to(dtype)
    idx, wt = slots(6, 2, 2, 28)
    ref, _ = moe_ref.experts(x, idx, wt, *ws3, "affine", gs, "silu", few_rows=False)
    assert float(ref.abs().max()) < torch.finfo(dtype).max / 4
    check(x, idx, wt, ws3, "affine", gs, "silu", path)


def test_token_block_of_the_few_row_path():
    """More slots than one pass of the few-row kernels takes."""
    ws3 = layer(5, 128, 192, 33, "nvfp4", 16, torch.float16, 11)
    idx, w = slots(90, 4, 5, 12, dropped=0.1)
    x = torch.randn((90, 128), generator=torch.Generator().manual_seed(13)).half()
    check(x, idx, w, ws3, "nvfp4", 16, "silu", "gemv")


@pytest.mark.parametrize("path", PATHS)
def test_repeats_bit_for_bit_and_needs_no_clean_workspace(path):
    ws3 = tuple(map(cu, layer(8, 512, 256, 512, "mxfp4", 32, torch.bfloat16, 14)))
    idx, w = slots(50, 4, 8, 15, dropped=0.1)
    x = torch.randn((50, 512), generator=torch.Generator().manual_seed(16)).bfloat16().cuda()
    idx, w = idx.cuda(), w.cuda()
    qb.qmm_set_path(path)
    n = qb.qmm_moe_experts_workspace_size(50, 512, 4, 8, 256, 512)
    first = None
    for fill in (0, 255, 127):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        y = torch.full((51, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        qb.qmm_moe_experts(x, idx, w, *ws3, group_size=32, mode="mxfp4", workspace=ws[:n], out=y[:50])
        qb.qmm_device_status()
        assert bool((y[50] == 3).all()) and bool((ws[n:] == fill).all())
        first = y if first is None else first
        assert torch.equal(first, y)


@pytest.mark.parametrize("path", PATHS)
def test_captured_and_on_another_stream(path):
    ws3 = tuple(map(cu, layer(8, 256, 256, 256, "affine", 64, torch.bfloat16, 17)))
    g = torch.Generator().manual_seed(18)
    x = torch.randn((24, 256), generator=g).bfloat16().cuda()
    lg = torch.randn((24, 8), generator=g).cuda()
    qb.qmm_set_path(path)
    n = qb.qmm_moe_experts_workspace_size(24, 256, 2, 8, 256, 256)

    def step(xi, li, ws, out):
        i, w = qb.qmm_moe_route(li, 2, score="sigmoid")
        return qb.qmm_moe_experts(xi, i, w, *ws3, group_size=64, workspace=ws, out=out)

    def fresh():
        return torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(x)

    graphs = []
    for scale in (1.0, -0.5):                      # two graphs, a workspace each, replayed at the same time
        xs, ls, (ws, out) = x * scale, lg * scale, fresh()
        step(xs, ls, ws, out)
        torch.cuda.synchronize()
        gr, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(gr, stream=st):
            step(xs, ls, ws, out)
        graphs.append((gr, st, xs, ls, ws, out, step(xs, ls, *fresh()).clone()))
    torch.cuda.synchronize()
    for _ in range(3):
        for gr, st, _, _, _, out, _ in graphs:
            with torch.cuda.stream(st):
                out.zero_()
                gr.replay()
    torch.cuda.synchronize()
    for _, _, _, _, _, out, want in graphs:
        assert torch.equal(out, want)
    qb.qmm_device_status()


@pytest.mark.parametrize("T", [1, 5, 70])
def test_router_then_experts(T):
    """The two calls as a model makes them, on the automatic path."""
    E, k, K, I = 16, 4, 256, 192
    ws3 = layer(E, K, I, K, "mxfp4", 32, torch.bfloat16, 19)
    g = torch.Generator().manual_seed(20)
    x = torch.randn((T, K), generator=g).bfloat16()
    lg = torch.randn((T, E), generator=g)
    b = torch.randn((E,), generator=g) * 0.1
    kw = dict(score="sigmoid", n_groups=4, topk_groups=2, group_top=2, scale=2.5)
    ri, rw = moe_ref.route(lg, k, bias=b, **kw)
    i, w = qb.qmm_moe_route(lg.cuda(), k, bias=b.cuda(), **kw)
    y = qb.qmm_moe_experts(x.cuda(), i, w, *map(cu, ws3), group_size=32, mode="mxfp4")
    qb.qmm_device_status()
    assert torch.equal(i.cpu(), ri)
    few, bf = moe_ref.experts(x, ri, rw, *ws3, "mxfp4", 32, "silu", few_rows=True)
    _, bm = moe_ref.experts(x, ri, rw, *ws3, "mxfp4", 32, "silu", few_rows=False)
    bound = torch.maximum(bf, bm) + 2.0 ** -21 * few.abs()      # fp32 weights against the 64-bit ones
    assert bool(((y.cpu().double() - few).abs() <= bound).all())


def test_empty():
    ws3 = tuple(map(cu, layer(2, 64, 64, 64, "mxfp4", 32, torch.bfloat16, 21)))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    y = qb.qmm_moe_experts(x, torch.empty((0, 2), dtype=torch.int32, device="cuda"),
                           torch.empty((0, 2), device="cuda"), *ws3, group_size=32, mode="mxfp4")
    assert y.shape == (0, 64)
