"""The build refuses a kernel whose registers are not what its split between warps counts on."""
import os

import pytest

from sparse_compressed_attention_gb300 import build as B

LOG = """ptxas info    : Compiling entry function '_ZN2v44_GLOBAL14tree_tc_kernelILb0EEEv' for 'sm_103a'
ptxas info    : Used 128 registers, used 5 barriers
ptxas info    : Compiling entry function '_ZN2v44_GLOBAL14tree_tc_kernelILb1EEEv' for 'sm_103a'
ptxas info    : Function properties
    0 bytes stack frame
ptxas info    : Used %d registers, used 5 barriers
ptxas info    : Compiling entry function '_ZN2v44_GLOBAL16tree_join_kernelE' for 'sm_103a'
ptxas info    : Used 96 registers
"""
SRC = os.path.join(B.CSRC, "tree_tc.cu")


def test_the_right_number_passes():
    B.check_registers(SRC, LOG % 96)
    B.check_registers(os.path.join(B.CSRC, "pages.cu"), "")


@pytest.mark.parametrize("log", [LOG % 88, LOG % 104, "", LOG.split("ptxas info    : Function")[0]])
def test_others_are_refused(log):
    with pytest.raises(RuntimeError, match="tree_tc.cu.*split needs 96"):
        B.check_registers(SRC, log)


def test_a_build_is_checked():
    """The library that the tests load was built through this check."""
    assert os.path.exists(B.build()) and B.up_to_date()
