"""The bit-level formulas of the experts' kernels, taken from the kernel sources and
evaluated on every byte they can meet (CPU only)."""
import re
from pathlib import Path

import numpy as np

CSRC = Path(__file__).resolve().parent.parent / "quantized_matmul_03_b200" / "csrc"


def body(name, signature):
    text = (CSRC / name).read_text()
    at = text.index(signature)
    return text[at:text.index("\n}\n", at)]


def py(expr):
    """A C expression over unsigned integers without its suffixes."""
    return re.sub(r"(?<=[0-9A-Fa-f])u\b", "", expr.strip())


def f32(bits):
    return float(np.array([bits & 0xFFFFFFFF], np.uint32).view(np.float32)[0])


def test_e8m0_of_the_few_row_kernels():
    expr = re.search(r"return __uint_as_float\((.*)\);", body("moe_gemv.cu", "float e8m0(uint32_t s)")).group(1)
    for s in range(255):
        # the shifted byte leaves the word's top bit alone: s << 23 < 2^31
        assert f32(eval(py(expr), {"s": s, "max": max})) == 2.0 ** (s - 127)
    assert np.isnan(f32(eval(py(expr), {"s": 255, "max": max})))


def factor_formulas():
    text = body("moe_tc.cu", "uint32_t scale_factor(uint32_t s)")
    f16 = re.search(r"const uint32_t b = s >= 99u \? (.*) : \(s >= 89u \? (.*) : 0u\);", text)
    bf16 = re.search(r"return (\(s \+ \d+u\) \* 0x00800080u);", text)
    assert "return b * 0x00010001u;" in text
    return py(f16.group(1)), py(f16.group(2)), py(bf16.group(1))


def test_mxfp4_factors_of_the_tensor_core_kernel():
    limit = int(re.search(r"else return s <= (\d+)u;", body("moe_tc.cu", "bool scale_in_range(uint32_t s)")).group(1))
    assert limit == 128
    high, low, bf = factor_formulas()
    for s in range(limit + 1):
        w = eval(bf, {"s": s}) & 0xFFFFFFFF
        assert w >> 16 == w & 0xFFFF and f32((w & 0xFFFF) << 16) == 2.0 ** (s - 1)             # X 2^126
        h = eval(high, {"s": s}) if s >= 99 else eval(low, {"s": s}) if s >= 89 else 0
        got = float(np.array([h], np.uint16).view(np.float16)[0])
        assert got == (2.0 ** (s - 113) if s >= 89 else 0.0)                                    # X 2^14
        assert s >= 89 or 6 * 2.0 ** (s - 127) < 2.0 ** -25       # under half of f16's smallest value


def test_nvfp4_factors_stay_in_range():
    """|X| below 4 by its byte, so that X 2^126 (bf16) and X 2^14 (f16) are finite and,
    with at most four significant bits, exact."""
    text = body("moe_tc.cu", "bool scale_in_range(uint32_t s)")
    limit = int(re.search(r"\(s & 0x7Fu\) < (0x[0-9A-Fa-f]+)u", text).group(1), 16)
    value = [(i & 7) / 8 * 2.0 ** -6 if i >> 3 == 0 else (1 + (i & 7) / 8) * 2.0 ** ((i >> 3) - 7) for i in range(127)]
    assert max(value[:limit]) < 4 <= value[limit]
    for x in value[:limit]:
        assert x * 2.0 ** 126 < 2.0 ** 128 * (1 - 2.0 ** -8)
        h = np.float64(x * 2.0 ** 14).astype(np.float16)
        assert np.isfinite(h) and float(h) == x * 2.0 ** 14
