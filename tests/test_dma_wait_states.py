"""Wait states of the LDS DMA loads written as inline assembly, in the compiled
device code (CPU only). A vector-memory instruction must come at least five wait
states after a vector instruction wrote a scalar register that it reads (its
buffer descriptor), and the compiler's hazard pass does not look into inline
assembly: the assembly brings them itself."""
import os
import re
import subprocess

import pytest

from combine_ep_layout_10_amd import build as B


def test_dma_loads_bring_their_wait_states(tmp_path):
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc not installed")
    out = tmp_path / "gemm.s"
    flags = [f for f in B.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([B.HIPCC] + flags + ["--cuda-device-only", "-S", "-o", str(out),
                                        os.path.join(B.CSRC, "ep_gemm_bf16.hip")], check=True, capture_output=True)
    lines = [l.split(";")[0].strip() for l in out.read_text().splitlines()]
    lines = [l for l in lines if l and not l.startswith(".")]
    loads = [i for i, l in enumerate(lines) if l.startswith("buffer_load_dwordx4") and l.endswith(" lds")]
    assert len(loads) > 50
    for i in loads:
        m = re.fullmatch(r"s_nop (\d+)", lines[i - 1])
        assert m and int(m.group(1)) >= 4, lines[i - 3:i + 1]
