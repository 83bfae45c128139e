"""What the binding of the calls between the linears does with arguments of a
wrong kind.  No GPU."""
import pytest

import w4a4_rank_corrected_quantize_amd as svdq

torch = pytest.importorskip("torch")


def test_a_plan_that_is_none_is_refused():
    index = torch.zeros(4, dtype=torch.int32)
    for bad in (torch.zeros(4096, dtype=torch.uint8), 7, "plan"):
        with pytest.raises(TypeError, match="LoraPlan"):
            svdq.lora_plan(index, 2, plan=bad)
