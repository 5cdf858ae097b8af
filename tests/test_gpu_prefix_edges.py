"""Attention over shared prefixes beside what is refused."""
import numpy as np
import pytest
import torch

from tree_testlib import DEV, i32, status


@pytest.mark.gpu
def test_a_refused_call_launches_nothing():
    """1024 rows of 32 heads over an arena of a million columns are more tiles than 32 bits number, which
    the rows' own pass refuses: the pass over the prefix must not have run then, nor told of its bounds."""
    import speculative_decoding_specdec_gb300.specdec as sd
    B, H, hd, cap = 1024, 32, 8, (1 << 20) + 64
    dtype = torch.bfloat16
    arena = torch.zeros(1, 2, 1, 1, cap, hd, dtype=dtype, device=DEV).expand(-1, -1, -1, H, -1, -1)
    prefix = torch.zeros(1, 2, 1, H, 64, hd, dtype=dtype, device=DEV)
    q = torch.zeros(B, 1, H, hd, dtype=dtype, device=DEV)
    ws, st = torch.zeros(sd.prefix_attention_workspace_bytes(q, arena, 1), dtype=torch.uint8, device=DEV), status()
    out = torch.full_like(q, 7.0)
    for groups in ([0, 5], [3, 2]):
        with pytest.raises(sd.SpecdecError):
            sd.prefix_attention(q, arena, 0, out, i32(np.full(B, 3)), None, None, st, ws, prefix, i32([40]), i32(groups),
                                first_col=i32(np.arange(B)))
        torch.cuda.synchronize()
        assert int(st) == 0 and not ws.any() and (out == 7).all()
