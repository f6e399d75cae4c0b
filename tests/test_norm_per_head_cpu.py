"""Layer norm backward per head needs an axis of heads (CPU)."""
import pytest
import torch

import chunked_gated_delta_07_gb300 as gdr


def test_a_lone_row_has_no_heads():
    x, s = torch.zeros(8), torch.zeros(())
    with pytest.raises(ValueError, match="per_head"):
        gdr.layer_norm_bwd(x, x, s, s, per_head=True)
