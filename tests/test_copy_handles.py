"""The copies' Python call takes any number of moves with one prepared call a shape; without a GPU."""
import pytest

from test_chunks import GOOD, api  # noqa: F401


def test_no_call_is_kept_for_a_number_of_moves(api):  # noqa: F811
    import torch
    sh = api.PagedShape(**GOOD)
    ws, k_idx = torch.zeros(4096, dtype=torch.uint8), torch.zeros(64, 128, 64, dtype=torch.bfloat16)
    kept = set()
    for n in (1, 2, 7, 1000, 0):
        with pytest.raises(ValueError, match="CUDA"):
            api.paged_copy(sh, torch.zeros(n, 3, dtype=torch.int32), None, None, None, None, k_idx, workspace=ws)
        kept.add(len(sh._more_calls))
    assert len(kept) == 1


@pytest.mark.parametrize("bad", [(3,), (2, 4), (2, 3, 1), (0,)])
def test_moves_of_another_shape_are_refused(api, bad):  # noqa: F811
    import torch
    sh = api.PagedShape(**GOOD)
    with pytest.raises(ValueError, match="moves"):
        api.paged_copy(sh, torch.zeros(bad, dtype=torch.int32), None, None, None, None, torch.zeros(64, 128, 64, dtype=torch.bfloat16),
                       workspace=torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="moves"):
        api.paged_copy(sh, torch.zeros(6, 3, dtype=torch.int32)[::2], None, None, None, None, torch.zeros(64, 128, 64, dtype=torch.bfloat16),
                       workspace=torch.zeros(4096, dtype=torch.uint8))
    with pytest.raises(ValueError, match="moves"):
        api.paged_copy(sh, None, None, None, None, None, torch.zeros(64, 128, 64, dtype=torch.bfloat16), workspace=torch.zeros(4096, dtype=torch.uint8))
