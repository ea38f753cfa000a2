"""What the training entries' launches refuse, on the CPU (test build; nothing is launched)."""
import pytest

import fp32_accumulate_lm_b200 as lm
from fp32_accumulate_lm_b200 import _build

LONE, PAIR, BIG = range(3)
STATS, DLOGITS, DWEIGHT, DHIDDEN = range(4)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return lm.load_test_library()


@pytest.mark.parametrize("shape", [LONE, PAIR, BIG])
@pytest.mark.parametrize("kind", [STATS, DLOGITS, DWEIGHT, DHIDDEN])
def test_big_tiles_are_refused_for_the_loss(lib, shape, kind):
    """Their kernel has no epilogue for the statistics: the launch is an error, not a wrong result."""
    served = lib.lmhead_debug_xent_shape_serves(shape, kind)
    assert served == (0 if (shape, kind) == (BIG, STATS) else 1)
