"""The attention kernels on CTA pairs divide exactly the registers that they are launched with, so the
compiler has to give each thread that many: read from its report of the library in place."""

import glob
import os

from conftest import load_builder

REPORT = """ptxas info    : Compiling entry function '_Z16attn_pair_kernelI1P' for 'sm_103a'
ptxas info    : Function properties for _Z16attn_pair_kernelI1P
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used {} registers, used 1 barriers
ptxas info    : Compiling entry function '_Z5other' for 'sm_103a'
ptxas info    : Used 40 registers, used 1 barriers
"""


def test_pair_kernels_have_their_registers():
    b = load_builder()
    b.build()
    seen = {}
    for path in glob.glob(os.path.join(b.OBJDIR, "*.ptxas")):
        with open(path) as f:
            seen.update({n: r for n, r in b.registers(f.read()).items() if "attn_pair_kernel" in n})
    if not seen:                         # a library that was built before reports were kept
        b.build(force=True)
        return test_pair_kernels_have_their_registers()
    # causal prefill; windowed prefill and prefix states in both types
    assert len(seen) == 5 and set(seen.values()) == {b.pair_registers()}, seen


def test_other_registers_are_told(capfd):
    b = load_builder()
    assert b.registers(REPORT.format(126)) == {"_Z16attn_pair_kernelI1P": 126, "_Z5other": 40}
    b._report_pairs(REPORT.format(126))
    assert "RF_ERR_UNSUPPORTED" in capfd.readouterr().err
    b._report_pairs(REPORT.format(b.pair_registers()))
    assert capfd.readouterr().err == ""
