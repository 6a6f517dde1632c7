"""What the wrappers of the calls over packed batches refuse by themselves."""
import inspect

import pytest
import torch

from block_diffusion_speculative_injection_gb300 import capi


def test_attention_names_a_missing_status():
    t = torch.zeros(4, 3, 128, dtype=torch.bfloat16)
    off, status = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    args = (1, True, off, t[:, :1], t[:, 1:2], t[:, 2:], torch.zeros(4, 1, 128, dtype=torch.bfloat16))
    for missing in (args, (*args, torch.zeros(4, 1)), (*args, None, None)):
        with pytest.raises(capi.DFlashError, match="status: need int32"):
            capi.dflash_prompt_attention(*missing)
    with pytest.raises(capi.DFlashError, match="status"):
        capi.dflash_prompt_attention(*args, status=status.long())
    # lse may be left out (the memory is the host's, so the library itself refuses)
    names = list(inspect.signature(capi.dflash_prompt_attention).parameters)
    assert names[-3:] == ["lse", "status", "stream"]
