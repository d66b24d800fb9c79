"""The rotation of many rows with an even number of heads: two rows of one token at once.  Against the
definition, with test_rope_gpu's bounds."""
import pytest

from tests.test_latent_gpu import DEV, error_word, k, torch
from tests.test_rope_gpu import TYPES, check_rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("inverse,in_place", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("T,H,width,offset,dim", [(8191, 12, 64, 0, 32), (40001, 4, 16, 0, 16), (1023, 128, 96, 32, 64)])
def test_two_rows_of_a_token_at_once(kind, half, inverse, in_place, T, H, width, offset, dim):
    check_rows(kind, T, H, width, offset, dim, half, inverse, in_place, seed=H)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("H", [11, 12])
def test_many_rows_with_positions_out_of_range(kind, half, in_place, H):
    """Tokens without a row of the table are left as they are, the others turn as they would alone."""
    dtype, _ = TYPES[kind]
    T, width, dim, layout = 8190, 64, 32, k.ROPE_HALF if half else k.ROPE_PAIRS
    gen = torch.Generator(device=DEV).manual_seed(7)
    cos_sin = torch.empty(40, dim, device=DEV)
    k.rope_table(k.rope_frequencies(dim, 100.0), cos_sin)
    x = torch.randn(T, H, width, generator=gen, device=DEV).to(dtype)
    at = torch.randint(0, 40, (T,), generator=gen, device=DEV)
    want = x.clone() if in_place else torch.empty_like(x)
    k.rope_rows(x.clone() if not in_place else want, at, cos_sin, out=want, offset=0, layout=layout)
    bad = torch.randint(0, 5, (T,), generator=gen, device=DEV) == 0
    bad[[0, T - 1]] = True
    at[bad] = torch.where(torch.arange(int(bad.sum()), device=DEV) % 2 == 0, -1, 40)
    err = error_word()
    got = x.clone() if in_place else torch.full_like(x, 9.0)
    k.rope_rows(got if in_place else x, at, cos_sin, out=got, offset=0, layout=layout, device_error=err)
    assert int(err.item()) == k.DEVERR_POS_RANGE
    assert torch.equal(got[~bad], want[~bad])
    assert torch.equal(got[bad], x[bad] if in_place else torch.full_like(x[bad], 9.0))
