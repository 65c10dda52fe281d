"""The window attention's matrix instructions and the first use of their results, read from the compiler's assembly
along every path, as for the delta rule's kernels (no GPU needed)."""
import pytest

import test_mfma_wait_states as reader

# 32 x 32 x 16 takes twice the passes of 16 x 16 x 32, eight: 11 wait states
WAIT = {**reader.WAIT, "v_mfma_f32_32x32x16_bf16": 11}


@pytest.mark.parametrize("src", ["attn_fwd.hip", "attn_fwd_f32.hip", "attn_bwd.hip", "attn_bwd_f32.hip", "attn_decode.hip"])
def test_results_are_waited_for_on_every_path(src, monkeypatch):
    monkeypatch.setattr(reader, "WAIT", WAIT)
    n, bad = reader.violations(reader._assembly(src))
    assert n > 100
    assert not bad, bad[:5]
