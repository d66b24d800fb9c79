"""The 4-bit attention over many thousands of requests at once."""
import numpy as np
import pytest

from tests.test_fp4_gpu import DEV, Batch, dev, k, torch

pytestmark = pytest.mark.gpu


def _shared_pages(N, H, W, seed):
    """N requests over the same few pages of 16 rows: (the pages' batch, table, q, q in fp64)."""
    pages = Batch([96], 1, 1, 16, seed=seed, spare=0)
    rng = np.random.default_rng(seed)
    table = rng.integers(0, pages.nb, (N, W)).astype(np.int32)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(N, 1, H, 512, generator=gen, device=DEV).to(torch.bfloat16)
    return pages, table, q


def _expected(pages, table, q, lens, scale):
    """fp64 on the GPU: (out, lse, |p| . |rows|, scale * the largest sum |q||k|)."""
    order = pages.table_np[0]  # page -> its place in the sequence of rows
    rows = torch.zeros(pages.nb * 16, 512, dtype=torch.float64, device=DEV)
    for i, page in enumerate(order):
        rows[page * 16:page * 16 + 16] = dev(pages.rows[0][16 * i:16 * i + 16], np.float64)
    i = torch.arange(table.shape[1] * 16, device=DEV)
    at = dev(table, np.int64)[:, i // 16] * 16 + i % 16            # [N, L]
    seen = i < lens[:, None]
    q64 = q[:, 0].double()
    s = torch.einsum("nhd,rd->nhr", q64, rows) * scale             # over all rows
    reach = torch.einsum("nhd,rd->nhr", q64.abs(), rows.abs()).amax(-1) * scale
    x = s.gather(2, at[:, None].expand(-1, s.shape[1], -1)).masked_fill(~seen[:, None], -float("inf"))
    lse = torch.logsumexp(x, -1)
    p = torch.where(seen[:, None], torch.exp(x - lse[..., None]), 0.0)
    share = torch.zeros_like(s).scatter_add_(2, at[:, None].expand(-1, s.shape[1], -1), p)
    return share @ rows, lse, share @ rows.abs(), reach


@pytest.mark.parametrize("N,H,W", [(20011, 2, 40), (12000, 70, 3)])
def test_many_thousand_row_tiles(N, H, W):
    """Requests of no keys, a few, and hundreds, in one call: single tiles of rows, and two a request."""
    pages, table, q = _shared_pages(N, H, W, seed=N)
    rng = np.random.default_rng(7)
    most = W * 16
    lens_np = np.where(rng.random(N) < 0.3, 0, rng.integers(1, 40, N))
    long = rng.random(N) < 0.05
    lens_np = np.where(long, rng.integers(1, most + 1, N), lens_np)
    lens_np[[0, -1]] = most, 0
    lens = dev(lens_np, np.int32)
    scale = 512.0 ** -0.5
    out = torch.full_like(q, 9.0)
    lse = torch.full((N, 1, H), 9.0, device=DEV)
    k.fp4_attention(q, pages.cache, pages.nb, 16, dev(table), lens, scale, out, lse=lse)
    for a in range(0, N, 2000):
        part = slice(a, a + 2000)
        want, wlse, size, reach = _expected(pages, table[part], q[part], lens[part], scale)
        ds = reach * 2.0 ** -15 + 2.0 ** -18
        tol = want.abs() * 2.0 ** -8 + size * (2.0 ** -8 + 2 * ds[..., None])
        assert bool(((out[part, 0].double() - want).abs() <= tol + 1e-30).all())
        got, empty = lse[part, 0].double(), torch.isneginf(wlse)
        assert torch.equal(torch.isneginf(got), empty)
        off = torch.where(empty, 0.0, (got - wlse).abs())
        assert bool((off <= ds + torch.where(empty, 0.0, wlse.abs()) * 2.0 ** -22).all())
    again = torch.empty_like(out)
    k.fp4_attention(q, pages.cache, pages.nb, 16, dev(table), lens, scale, again)
    assert torch.equal(out, again)


def test_sinks_of_requests_without_keys():
    """Thousands of idle requests: zeros, and each head's sink as its lse."""
    N, H = 9001, 3
    pages, table, q = _shared_pages(N, H, 2, seed=5)
    lens_np = np.zeros(N, np.int32)
    lens_np[4000] = 20
    sinks = torch.tensor([0.5, -2.0, -float("inf")], device=DEV)
    out, lse = torch.full_like(q, 9.0), torch.full((N, 1, H), 9.0, device=DEV)
    k.fp4_attention(q, pages.cache, pages.nb, 16, dev(table), dev(lens_np), 0.05, out, lse=lse, sinks=sinks)
    idle = torch.arange(N, device=DEV) != 4000
    assert bool((out[idle] == 0).all()) and bool(torch.isfinite(out).all()) and bool((out[4000] != 9).all())
    assert torch.allclose(lse[idle][:, 0, :2], sinks[:2].expand(N - 1, -1), rtol=2.0 ** -21, atol=0)
    assert bool(torch.isneginf(lse[idle][:, 0, 2]).all())


def test_time_grows_no_faster_than_the_requests():
    """Idle requests cost a look at their length and their zeros: eight times as many, about eight
    times the time at most (20 allowed: a cost that grows with the square would be 64 times)."""
    pages, table, q = _shared_pages(64000, 1, 1, seed=6)
    out = torch.empty_like(q)
    table_t, lens = dev(table), torch.zeros(64000, dtype=torch.int32, device=DEV)
    workspace = torch.empty(k.fp4_attention_workspace_bytes(), dtype=torch.uint8, device=DEV)

    def best(n):
        times = []
        for _ in range(8):
            begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            begin.record()
            for _ in range(10):
                k.fp4_attention(q[:n], pages.cache, pages.nb, 16, table_t[:n], lens[:n], 0.05, out[:n],
                                workspace=workspace)
            end.record()
            torch.cuda.synchronize()
            times.append(begin.elapsed_time(end))
        return min(times)

    few, many = best(8000), best(64000)
    print(f"8000 idle requests {few * 100:.0f} us, 64000 {many * 100:.0f} us")
    assert many < 20 * few
