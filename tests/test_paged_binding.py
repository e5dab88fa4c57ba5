"""The paged calls' binding, host side: memory it must refuse (no call reaches a GPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def ts():
    import self_speculative_ultra_gb300 as ts
    ts.build()
    return ts


def test_a_workspace_counts_the_bytes_it_has(ts):
    given = ts._given_workspace
    whole = torch.empty(4096, dtype=torch.uint8)
    assert given(whole, 4096, -1) == (whole.data_ptr(), 4096)
    assert given(torch.empty(64, 16), 4096, -1)[1] == 4096
    with pytest.raises(ValueError):
        given(whole, 4097, -1)
    # one byte, or every second one, in the shape of more
    for x in (torch.empty(1, dtype=torch.uint8).expand(4096), whole.view(64, 64)[:, ::2],
              torch.empty(1, 64).expand(64, 64)):
        with pytest.raises(ValueError):
            given(x, 1024, -1)
