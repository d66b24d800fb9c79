"""What the binding of the attention over the FP8 and bf16 caches refuses before the library is called."""
import pytest

import kv_norm_rope_gb300 as k

torch = pytest.importorskip("torch")


def _call(q, out, batch=1):
    """On the host, where a call that passes the other checks is refused for that."""
    table, lens = torch.zeros(batch, 1, dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
    cache = torch.zeros(16 * 512, dtype=torch.bfloat16)
    workspace = torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8)
    k.latent_attention(k.STORE_BF16, q, cache, 1, 16, table, lens, 1.0, out, workspace=workspace)


def test_out_may_not_overlap_q():
    room = torch.zeros(6, 1, 2, 512, dtype=torch.bfloat16)
    for q, out in ((room[:2], room[:2]), (room[:2], room[1:3]), (room[2:4], room[1:3]),
                   (room[:2], room.view(-1)[2040:4088].view(2, 1, 2, 512))):
        with pytest.raises(ValueError, match="overlaps"):
            _call(q, out, 2)
    for q, out in ((room[:2], room[2:4]), (room[4:], room[2:4]), (room[:2], room.view(-1)[2048:4096].view(2, 1, 2, 512))):
        with pytest.raises(ValueError, match="CUDA"):
            _call(q, out, 2)
    with pytest.raises(ValueError, match="CUDA"):
        _call(room[:0], room[:0], 0)
