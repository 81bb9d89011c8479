"""The build fails when a kernel that moves registers between its warps is not compiled to the number its
source counts on (such a kernel refuses to run)."""
import pathlib
import re

import pytest

from expert_cached_sparse_b200 import build as B

CSRC = pathlib.Path(B.CSRC)
FP8 = "_ZN3moe45_GLOBAL__N__0123_19_grouped_gemm_fp8_cu_1b16gg8_kernelINS0_3CfgILb%dEEEEEvNS_2tc7RowMapsE"


def ptxas(*kernels):
    return "".join(f"ptxas info    : Compiling entry function '{name}' for 'sm_100a'\n"
                   f"ptxas info    : Function properties for {name}\n    0 bytes stack frame, 0 bytes spill stores\n"
                   f"ptxas info    : Used {n} registers, used 3 barriers, 1024 bytes smem\n" for name, n in kernels)


def test_the_count_is_checked():
    src = "constexpr int kRegs = 168, kControlRegs = 72;"
    B.check_registers("grouped_gemm_fp8.cu", src, ptxas((FP8 % 1, 131), (FP8 % 0, 168)))
    B.check_registers("router.cu", "", ptxas(("_Z1k", 20)))
    for bad in (ptxas((FP8 % 1, 168), (FP8 % 0, 160)), ptxas((FP8 % 1, 168)), ""):
        with pytest.raises(RuntimeError, match="168 registers"):
            B.check_registers("grouped_gemm_fp8.cu", src, bad)


def test_every_source_that_moves_registers_is_checked():
    assert {p.name for p in CSRC.iterdir() if "setmaxnreg" in p.read_text()} == set(B.MOVE_REGISTERS)
    for name in B.MOVE_REGISTERS:
        assert re.search(r"\bkRegs = \d+", (CSRC / name).read_text())


def test_the_splits_fit_what_the_blocks_are_launched_with():
    """setmaxnreg draws on the registers that a block was launched with: a larger split would wait for ever."""
    for name in B.MOVE_REGISTERS:
        regs, control, sums = (int(re.search(rf"\b{k} = (\d+)", (CSRC / name).read_text())[1])
                               for k in ("kRegs", "kControlRegs", "kSumRegs"))
        assert control % 8 == 0 and sums % 8 == 0 and 128 * control + 256 * sums <= 384 * regs <= 65536
