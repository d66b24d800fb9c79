"""The 4-bit cache's eviction at the ends of its ranges."""
import pytest

from tests.test_fp4_gpu import DEV, dev, error_word, fp4, k, np, torch

pytestmark = pytest.mark.gpu


def test_budget_a_step_below_two_to_the_31():
    """A budget far past any length: the rows there are, -1 and 0 after them to the end."""
    budget, block, n = 2 ** 31 - 1, 2 ** 20, 5
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 20 GB for kept and the new weights")
    image = np.random.default_rng(1).integers(0, 256, n * 352).astype(np.uint8)
    cache = torch.zeros(k.fp4_cache_bytes(2, block), dtype=torch.uint8, device=DEV)
    cache[:n * 352] = dev(image)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    new = torch.full((1, 2 ** 11), -1, dtype=torch.int32, device=DEV)
    new[0, 0] = 1
    w = torch.tensor([[3.0, 1.0, 2.0, 5.0, 4.0]], device=DEV)
    kept = torch.full((1, budget), -9, dtype=torch.int32, device=DEV)
    weights = torch.full((1, budget), 7.0, device=DEV)
    lens, err = torch.tensor([n], dtype=torch.int32, device=DEV), error_word()
    k.fp4_evict(cache, 2, block, table, lens, w, budget, 2, new, kept, lens, weights, device_error=err)
    assert int(err.item()) == 0 and int(lens.item()) == n
    assert kept[0, :n].tolist() == fp4.evict(w[0].cpu().numpy(), n, budget, 2)
    assert torch.equal(weights[0, :n], w[0])
    for a in range(n, budget, 1 << 28):
        assert bool((kept[0, a:a + (1 << 28)] == -1).all()) and bool((weights[0, a:a + (1 << 28)] == 0).all())
    page = block * 368
    assert torch.equal(cache[page:page + n * 352], dev(image))
    assert not bool(cache[page + n * 352:2 * page].any())
