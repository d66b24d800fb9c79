"""The Python binding of the 4-bit cache's operators, without a GPU."""
import pytest

import kv_norm_rope_gb300 as k


def test_workspace_by_its_address(monkeypatch):
    """A workspace may be a raw address, as the other buffers may: the caller vouches for its size."""
    torch = pytest.importorskip("torch")
    calls = []

    class Library:
        def dsv4_fp4_attention_workspace_bytes(self):
            return 4096

        def dsv4_fp4_attention(self, *args):
            calls.append(args)
            return k.OK

    monkeypatch.setattr(k, "lib", lambda: Library())
    monkeypatch.setattr(k, "_on_cuda", lambda **tensors: None)
    monkeypatch.setattr(k, "_workspace_bytes", 0)
    q = torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16)
    args = (q, 1 << 20, 3, 16, torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 0.1,
            torch.empty_like(q))
    k.fp4_attention(*args, workspace=1 << 21, stream=7)
    assert calls[0][16:18] == (1 << 21, 4096)
    small = torch.empty(100, dtype=torch.uint8)
    k.fp4_attention(*args, workspace=small, stream=7)
    assert calls[1][16:18] == (small.data_ptr(), 100)


def test_windows_past_32_bits_are_all_keys(monkeypatch):
    """A number that 32 bits do not hold is not cut to its low ones."""
    torch = pytest.importorskip("torch")
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append((name, args)) or k.OK

    monkeypatch.setattr(k, "lib", lambda: Library())
    monkeypatch.setattr(k, "_on_cuda", lambda **tensors: None)
    monkeypatch.setattr(k, "_workspace_bytes", 4096)
    q, table = torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    lens, lse, w = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 1, 4), torch.zeros(2, 32)
    for window, taken in ((5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 31 - 1), (2 ** 63, 2 ** 31 - 1),
                          (-1, -1), (5 - 2 ** 32, -1)):
        calls.clear()
        k.fp4_attention(q, 1 << 20, 3, 16, table, lens, 0.1, torch.empty_like(q), window=window,
                        workspace=1 << 21, stream=7)
        k.fp4_attention_weights(q, 1 << 20, 3, 16, table, lens, 0.1, lse, w, window=window, stream=7)
        assert [args[12] for _, args in calls] == [taken, taken]
    calls.clear()
    k.fp4_evict(1 << 20, 3, 16, table, lens, w, 8, 2 ** 32 + 1, table, torch.zeros(2, 8, dtype=torch.int32), lens,
                torch.zeros(2, 8), stream=7)
    assert calls[0][1][12] == 2 ** 31 - 1  # more than the budget: refused
