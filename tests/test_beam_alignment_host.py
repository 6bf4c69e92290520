"""Logits that do not start on 16 bytes: refused by name (no GPU needed)."""
import pytest
import torch

import rank_compressed_paged_gb300 as rcp


@pytest.mark.parametrize("dtype,V", [(torch.float16, 1001), (torch.bfloat16, 7), (torch.float32, 5)])
def test_a_slice_that_starts_inside_16_bytes_is_refused_by_name(dtype, V):
    logits, scores = torch.zeros((4, 1, V), dtype=dtype), torch.zeros((3, 1))
    part = logits[1:]
    assert part.is_contiguous() and part.data_ptr() % 16
    with pytest.raises(ValueError, match="16-byte boundary"):
        rcp._validate_beams(part, scores, None)
    with pytest.raises(ValueError, match="16-byte boundary"):
        rcp.beam_select(part, scores)
    assert rcp._validate_beams(part.clone(), scores, None)[:3] == (3, 1, V)
