"""The build's check of kernels whose registers have to be an exact number."""

import pytest

from decode_qwen3_decoder_gb300 import _build

LOG = """ptxas info    : Compiling entry function '_ZN12_GLOBAL__N_119k_kv8_chunk_combineILi64ELi1EEEvNS_9Kv8ChunkPE' for 'sm_103a'
ptxas info    : Function properties for x
    0 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used 32 registers, used 0 barriers
ptxas info    : Compiling entry function '_ZN12_GLOBAL__N_111k_kv8_chunkILi64ELi1EEEvNS_9Kv8ChunkPE' for 'sm_103a'
ptxas info    : Used 128 registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN12_GLOBAL__N_111k_kv8_chunkILi128ELi0EEEvNS_9Kv8ChunkPE' for 'sm_103a'
ptxas info    : Used %d registers, used 1 barriers
"""


def test_registers_of_every_instance():
    wanted = _build.REGISTERS["k_kv8_attn.cu"]
    _build.check_registers(wanted, LOG % 128)
    _build.check_registers({}, "")
    for log in (LOG % 126, LOG % 136, LOG.split("ptxas info    : Compiling entry function '_ZN12_GLOBAL__N_111")[0], ""):
        with pytest.raises(RuntimeError, match="k_kv8_chunk"):
            _build.check_registers(wanted, log)


def test_registers_of_the_library_as_built():
    _build.build()
    for src, wanted in _build.REGISTERS.items():
        with open(_build.ptxas_log(src)) as fh:
            _build.check_registers(wanted, fh.read())
