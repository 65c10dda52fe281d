"""The window attention's matrix instructions and the first use of their results, read from the compiler's assembly
along every path, as for the delta rule's kernels (no GPU needed)."""
import pytest

from test_mfma_wait_states import _assembly, violations


@pytest.mark.parametrize("src", ["attn_fwd.hip", "attn_fwd_f32.hip", "attn_bwd.hip", "attn_bwd_f32.hip", "attn_decode.hip"])
def test_results_are_waited_for_on_every_path(src):
    n, bad = violations(_assembly(src))
    assert n > 100
    assert not bad, bad[:5]
