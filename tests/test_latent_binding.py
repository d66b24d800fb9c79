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


@pytest.fixture
def statuses(monkeypatch):
    """What the library says to calls with tensors of the host: all of them are refused, or end for want of a GPU."""
    if torch.cuda.is_available():
        pytest.skip("would launch on pointers of the host")
    said = []
    monkeypatch.setattr(k, "_launch", lambda what, where, stream, entry, *args: said.append(entry(*args, None)))
    return said


@pytest.mark.parametrize("first,status", [(0, k.ERR_CUDA), (2 ** 32 - 3, k.ERR_CUDA), (2 ** 32 - 2, k.ERR_SHAPE),
                                          (2 ** 64, k.ERR_SHAPE), (2 ** 64 + 5, k.ERR_SHAPE), (2 ** 63, k.ERR_SHAPE),
                                          (-1, k.ERR_SHAPE), (-2 ** 40, k.ERR_SHAPE)])
def test_first_position_is_not_cut_to_its_low_bits(statuses, first, status):
    k.rope_table((1.0, 0.5), torch.zeros(3, 4), first=first)
    assert statuses == [status]


@pytest.mark.parametrize("high", [2 ** 32, 2 ** 33, -2 ** 32, 2 ** 64])
def test_choices_are_not_cut_to_their_low_bits(statuses, high):
    x, positions, cos_sin = torch.zeros(3, 2, 16), torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    k.rope_rows(x, positions, cos_sin, layout=high)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, path = torch.zeros(16 * 1024, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    k.tree_keep(high, cache, 1, 16, table, lens, path, lens, lens)
    q = torch.zeros(2, 1, 2, 512, dtype=torch.bfloat16)
    workspace = torch.empty(k.latent_attention_workspace_bytes(), dtype=torch.uint8)
    k.latent_attention(high + 1, q, cache, 1, 16, table, lens, 1.0, torch.empty_like(q), workspace=workspace)
    assert statuses == [k.ERR_VALUE] * 3
    with pytest.raises(k.Dsv4Error) as e:
        k.rope_frequencies(64, scaling=high)
    assert e.value.status == k.ERR_VALUE
    # a cache given by its address, whose size nothing bounds
    k.tree_keep(k.STORE_BF16, 1 << 20, 1, high + 16, table, lens, path, lens, lens)
    assert statuses[3] == k.ERR_SHAPE


def test_the_choices_there_are_reach_the_library(statuses):
    x, positions, cos_sin = torch.zeros(3, 2, 16), torch.zeros(3, dtype=torch.int64), torch.zeros(5, 8)
    for layout in (k.ROPE_PAIRS, k.ROPE_HALF):
        k.rope_rows(x, positions, cos_sin, layout=layout)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    cache, path = torch.zeros(16 * 1024, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    for store in (k.STORE_FP8, k.STORE_BF16, k.STORE_FP4, k.STORE_INDEXER):
        k.tree_keep(store, cache, 1, 16, table, lens, path, lens, lens)
    assert statuses == [k.ERR_CUDA] * 6
