"""CPU check of the transform's kernels in the built library: none keeps anything in scratch
memory. The 256 x 256 tiles hold 256 accumulators a lane; an epilogue that is not unrolled
whole indexes them at run time, and the compiler moves them to scratch (the exact gelu in
float32 took 482 us so for 4104 x 2056 -> 4104, in registers 203)."""
import pytest

from tests.test_norm_registers import notes, pytestmark  # noqa: F401


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    return {n: v for n, v in notes("k_linear_dz", tmp_path_factory.mktemp("co")).items()
            if "k_linear" in n or "k_gemm" in n}


def test_no_scratch(kernels):
    assert sum("EpiLinear" in n for n in kernels) == 10 and sum("EpiGrad" in n for n in kernels) == 2
    assert len(kernels) > 60
    for name, v in kernels.items():
        assert v["private_segment_fixed_size"] == 0 and v["vgpr_spill_count"] == 0, name.split("(")[0]
