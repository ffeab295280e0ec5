"""The shape rule of the streamed few-row kernel (plan_stream), restated so that
tests can tell which form of the kernels their sizes reach."""
import re
from pathlib import Path

SRC = Path(__file__).resolve().parent.parent / "quantized_matmul_03_b200" / "csrc" / "moe_gemv.cu"


def _constant(name, text=None):
    return int(re.search(rf"constexpr int {name} = (\d+);", text or SRC.read_text()).group(1))


def stream(C, R, P, mode, gs, glu, sms=148):
    """None where the kernel without a ring takes the product, else a dict of its
    rounds, segments, stages of a round, ring slots and rows."""
    seg, warps, loads = (_constant(n) for n in ("kSeg", "kMaxWarps", "kLoads"))
    nm, na, es = (2 if glu else 1), (3 if mode == "affine" else 2), (2 if mode == "affine" else 1)
    S = -(-C // seg)
    sb = C // gs * es
    if S > warps or sb % 16:
        return None
    slots_round = min(P, warps // S)
    splits = warps // (slots_round * S)
    part = 32 * 1024
    ring = 220 * 1024 - part - 128
    rows = min(-(-R // sms), part // (P * S * nm * 4))
    if rows < 1:
        return None
    row_all = slots_round * nm * (C // 2 + (na - 1) * sb)
    rs = min(rows, loads // nm * splits)
    rs = min(rs, rows if rows <= ring // row_all else ring // 3 // row_all)
    if rs < 1:
        return None
    return dict(S=S, rounds=-(-P // slots_round), nst=-(-rows // rs), stages=min(8, ring // (rs * row_all)),
                rows=rows, rows_stage=rs, splits=splits, last=R % rows)
