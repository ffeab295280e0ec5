"""Bit-level steps of the experts' kernels, restated in numpy on every input they
can meet (CPU only; the constants are read from the kernel sources)."""
import re
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parent.parent / "quantized_matmul_03_b200" / "csrc"
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])


def prmt(a, b, sel):
    """Byte permutation: selector nibbles 0..7 pick a byte, bit 3 its sign."""
    src = [(a >> (8 * i)) & 255 for i in range(4)] + [(b >> (8 * i)) & 255 for i in range(4)]
    out = 0
    for i in range(4):
        n = (sel >> (4 * i)) & 15
        v = src[n & 7]
        out |= ((0xFF if v & 0x80 else 0) if n & 8 else v) << (8 * i)
    return out


def test_e2m1_bytes_of_the_few_row_kernels():
    text = (CSRC / "moe_gemv.cu").read_text()
    t = {k: int(v, 16) for v, k in re.findall(r'mov\.u32 %0, (0x[0-9A-Fa-f]+);" : "=r"\((\w+)\)', text)}
    for c0 in range(16):
        for c1 in range(16):
            w = (c0 | c1 << 4 | c0 << 8 | c1 << 12 | c1 << 16 | c0 << 20 | c0 << 24 | c1 << 28) & 0xFFFFFFFF
            n = w ^ 0x88888888
            for half in (0, 16):
                got = (prmt(t["pa"], t["pb"], (w >> half) & 0xFFFF) + prmt(t["na"], t["nb"], (n >> half) & 0xFFFF))
                codes = [(w >> (half + 4 * i)) & 15 for i in range(4)]
                assert [(got >> (8 * i)) & 255 for i in range(4)] == [int(64 + 2 * E2M1[c]) for c in codes]


def test_e8m0_without_branches():
    s = np.arange(256, dtype=np.uint64)
    bits = np.maximum(((s << np.uint64(23)) & np.uint64(0xFFFFFFFF)) | (((s + np.uint64(1)) << np.uint64(14)) & np.uint64(0x400000)),
                      np.uint64(0x400000)).astype(np.uint32)
    v = bits.view(np.float32).astype(np.float64)
    assert np.isnan(v[255])
    assert (v[:255] == 2.0 ** (np.arange(255) - 127.0)).all()


def halves_bf16(r):
    return [np.array([(int(r) >> sh & 0xFFFF) << 16], np.uint32).view(np.float32)[0].astype(np.float64) for sh in (0, 16)]


def halves_f16(r):
    return [np.array([int(r) >> sh & 0xFFFF], np.uint16).view(np.float16)[0].astype(np.float64) for sh in (0, 16)]


@pytest.mark.parametrize("f16", [False, True])
def test_e2m1_placed_in_halves(f16):
    """Codes e and e + 4 as 2^-126 (bf16) or 2^-14 (f16) times their values."""
    for c0 in range(16):
        for c1 in range(16):
            w = sum(c << (4 * i) for i, c in enumerate([c0, c1, c1, c0, c1, c0, c0, c1]))
            u = w >> 8
            if f16:
                r = [((w & 0x00070007) * 512 + (w & 0x00080008) * 4096),
                     ((w & 0x00700070) * 32 + (w & 0x00800080) * 256),
                     ((u & 0x00070007) * 512 + (u & 0x00080008) * 4096),
                     ((u & 0x00700070) * 32 + (u & 0x00800080) * 256)]
            else:
                r = [((w & 0x000F000F) * 4160) & 0x81C081C0, ((w & 0x00F000F0) * 260) & 0x81C081C0,
                     ((u & 0x000F000F) * 4160) & 0x81C081C0, ((u & 0x00F000F0) * 260) & 0x81C081C0]
            for e in range(4):
                lo, hi = (halves_f16 if f16 else halves_bf16)(r[e] & 0xFFFFFFFF)
                scale = 2.0 ** (14 if f16 else 126)
                assert lo * scale == E2M1[(w >> (4 * e)) & 15]
                assert hi * scale == E2M1[(w >> (4 * e + 16)) & 15]


def test_constants_of_the_placement_are_the_kernels():
    text = (CSRC / "moe_tc.cu").read_text()
    body = text[text.index("void e2m1_place"):text.index("bool scale_in_range")]
    for c in ("0x00070007u, 512u, (w & 0x00080008u) * 4096u", "0x00700070u, 32u, (w & 0x00800080u) * 256u",
              "0x000F000Fu, 4160u", "0x00F000F0u, 260u", "0x81C081C0u"):
        assert c in body


def test_mxfp4_factors_in_range():
    """X 2^126 in bf16 and X 2^14 in f16, for the scale bytes the fast path takes (X <= 2)."""
    for s in range(129):
        b = ((s + 126) * 0x00800080) & 0xFFFFFFFF
        assert halves_bf16(b) == [2.0 ** (s - 127 + 126)] * 2
        h = (s - 98) << 10 if s >= 99 else (1 << (s - 89) if s >= 89 else 0)
        want = 2.0 ** (s - 127 + 14)
        got = halves_f16(h * 0x00010001)
        # below f16's smallest value the element 6 X is under half of it too
        assert got == [want if s >= 89 else 0.0] * 2
        if s < 89:
            assert 6 * 2.0 ** (s - 127) < 2.0 ** -25
