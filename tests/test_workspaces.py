"""The sizes of the operators' workspaces (CPU)."""
import pytest

import block_scaled_fp4_03_amd as fp4


@pytest.fixture(scope="module", autouse=True)
def library():
    import os
    if not os.path.exists(fp4.LIB_PATH):
        import block_scaled_fp4_03_amd.build as b
        b.build()
    fp4.lib()


def test_empty_calls_need_none():
    assert fp4.fp4_verify_drafts_workspace(0, 4, 1000) == 0
    assert fp4.fp4_verify_drafts_workspace(0, 0, 1) == 0
    assert fp4.fp4_moe_sort_workspace(0, 4, 8) == 0 and fp4.fp4_moe_sort_workspace(4, 0, 8) == 0
    assert fp4.fp4_qk_norm_rope_workspace(0, 4, 2, 64) == 0 and fp4.fp4_qk_norm_rope_workspace(4, 0, 0, 64) == 0
