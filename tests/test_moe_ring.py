"""The packed ring of the experts' tensor-core kernel is long enough in every build
(CPU only; the sizes are read from the kernel's source).

A dequantize group that visits every BPG-th stage waits for a parity in a slot whose
last stage another group took.  Its stage before, s - BPG, is known to have waited
until stage s - BPG - NU was used up; the slot's last stage, s - SP, has to be no
later than that, or the wait can pass on an older phase."""
import re
from pathlib import Path

import pytest

TEXT = (Path(__file__).resolve().parent.parent / "quantized_matmul_03_b200" / "csrc" / "moe_tc.cu").read_text()


def ternary(name, cap):
    yes, no = re.search(rf"static constexpr int {name} = CAP <= 64 \? (\d+) : (\d+);", TEXT).groups()
    return int(yes) if cap <= 64 else int(no)


def builds():
    assert "static constexpr int NU = (512 - 2 * CAP) / (32 * U);" in TEXT
    assert "static constexpr int BBytes = CAP * 128 * U;" in TEXT
    sb = int(re.search(r"static constexpr int SB = (\d+);", TEXT).group(1))
    bar = int(re.search(r"constexpr int kBarBytes = (\d+);", TEXT).group(1))
    for cap in (64, 192):
        U, BPG = ternary("U", cap), ternary("BPG", cap)
        for nw in (1, 2):
            for win in (16, 32):
                left = 227 * 1024 - 1024 - bar - sb * cap * 128 * U
                yield cap, BPG, (512 - 2 * cap) // (32 * U), min(8, left // (128 * 256 // 2 + nw * 128 * win))


@pytest.mark.parametrize("cap,bpg,nu,sp", list(builds()))
def test_ring_is_long_enough(cap, bpg, nu, sp):
    assert sp >= 2
    assert bpg == 1 or sp >= nu + bpg


def test_the_build_checks_it_too():
    assert "SP >= Cfg::NU + Cfg::BPG" in TEXT and "static_assert(SP >= 2" in TEXT
