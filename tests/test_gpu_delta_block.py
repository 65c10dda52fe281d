"""The example block: decoding from a packed prefill's states continues it, and the mixer's gradients come out."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_block_decodes_as_it_prefills():
    """Both ways round to bf16 after every operator, and the library's projections of 4 and of 300 rows may round
    an entry to the other neighbour: a few units of 2^-8 at values up to 4 or 5."""
    import delta_block

    worst, names = delta_block.main()
    assert worst <= 4 * 5 * 2 ** -8
    assert names == ["beta", "g", "head_norm", "k", "q", "v", "z"]
