"""Caches whose block table is no table are refused before anything is written."""
import pytest
import torch

from decode_megakernel_03_gb300 import mk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2, 0), (0, 3), (0, 0), (3,), (1, 2, 3)])
def test_tables_without_entries_are_refused(shape):
    """A table without entries is not a contiguous cache."""
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mk.MkError) as e:
        mk.Cache([k], [k.clone()], torch.zeros(shape, dtype=torch.int32, device="cuda"))
    assert e.value.code == mk.MK_ERR_INVALID
