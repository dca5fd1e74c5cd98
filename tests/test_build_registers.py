"""The build's check that kernels which redistribute their registers got the number they count on."""
import pytest

from video_diffusion_attention_b200 import build as libbuild

LOG = """ptxas info    : 11 bytes gmem
ptxas info    : Compiling entry function '_ZN4tara16norm_rope_kernelIfLi8ELb0EEEvNS_12NormRopeArgsE' for 'sm_100a'
ptxas info    : Function properties for _ZN4tara16norm_rope_kernelIfLi8ELb0EEEvNS_12NormRopeArgsE
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 62 registers, used 0 barriers
ptxas info    : Compiling entry function '_ZN4tara18linear_pair_kernelILb0ELi128ELi1ELi0EEEvNS_11PairLinMapsENS_11PairLinArgsE' for 'sm_100a'
ptxas info    : Function properties for _ZN4tara18linear_pair_kernelILb0ELi128ELi1ELi0EEEvNS_11PairLinMapsENS_11PairLinArgsE
    8 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers, 8 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN4tara16attn_pair_kernelILb1EEEv14CUtensorMap_stS1_S1_NS_6TcArgsE' for 'sm_100a'
ptxas info    : Used %d registers, used 1 barriers
"""


def test_the_sources_state_their_registers():
    want = libbuild.split_registers()
    assert set(want) == set(libbuild.SPLIT_KERNELS) and all(v % 8 == 0 for v in want.values())


def test_expected_registers_pass():
    want = libbuild.split_registers()
    log = LOG % (want["linear_pair_kernel"], want["attn_pair_kernel"])
    assert libbuild.check_registers(log, want) == 2
    assert libbuild.check_registers("", want) == 0


@pytest.mark.parametrize("linear,attn,name", [(-8, 0, "linear_pair_kernel"), (0, 8, "attn_pair_kernel")])
def test_other_registers_stop_the_build(linear, attn, name):
    want = libbuild.split_registers()
    with pytest.raises(RuntimeError, match=name):
        libbuild.check_registers(LOG % (want["linear_pair_kernel"] + linear,
                                        want["attn_pair_kernel"] + attn), want)
