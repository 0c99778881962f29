"""Sizes that no C int holds: refused, not cut to their low 32 bits."""
import pytest
import torch


@pytest.fixture(scope="module")
def fr():
    from gqa_kv_head_gb300 import build
    build.build()
    import gqa_kv_head_gb300
    return gqa_kv_head_gb300


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 16, 2 ** 40 + 64, 2 ** 64 + 16])
def test_workspace_size(fr, big):
    assert fr.pages_workspace_size(16, 4) > 0
    for n in (big, -big):
        assert fr.pages_workspace_size(n, 4) == 0 and fr.pages_workspace_size(16, n) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("page_size", [2 ** 32 + 16, -2 ** 32 + 64, 2 ** 64 + 128, 2 ** 31 + 16])
def test_page_size(fr, page_size):
    refs, lens = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (8, 3))
    table = torch.full((3, 4), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(fr.FrError):
        fr.PagePool(refs, lens, table, page_size)
    fr.PagePool(refs, lens, table, 16)
