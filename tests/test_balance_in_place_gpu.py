"""The balance loss's gradient added in place, d_logits being the output: bit for bit what it is with an output of its own, for every
row length's kernel, in vectors and at odd addresses (where a row's sum has another order than in vectors)."""
import pytest

torch = pytest.importorskip("torch")
from test_balance_gpu import DEV, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import unpermute_combine_amd as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("T,E", [(1, 4), (777, 8), (33, 61), (500, 64), (129, 100), (3000, 128), (401, 255), (70000, 256), (130, 260),
                                 (999, 512), (65, 1000), (5000, 1024)])
@pytest.mark.parametrize("shift", [0, 1])
def test_added_in_place(m, T, E, shift):
    K = 2
    z, idx = inputs(T + E, T, E, K)
    keep = (torch.rand(T, generator=torch.Generator().manual_seed(E)) < 0.8).to(DEV)
    _, counts, _, tokens = m.balance_loss(z, idx, token_mask=keep)
    def at_shift(value):
        room = torch.full((T * E + 8,), 7.0, device=DEV)
        rows = room[4 + shift:4 + shift + T * E].view(T, E)
        rows.copy_(value)
        return room, rows

    given = torch.randn(T, E, generator=torch.Generator().manual_seed(T)) / T
    call = lambda **kw: m.balance_loss_backward(z, counts, tokens, K, token_mask=keep, **kw)  # noqa: E731
    add, (room, place) = at_shift(given)[1], at_shift(given)
    want = call(d_logits=add, out=at_shift(0.0)[1])
    assert torch.equal(want, call(out=at_shift(0.0)[1]) + add)
    assert call(d_logits=place, out=place) is place
    assert torch.equal(place, want) and bool((room[:4 + shift] == 7).all()) and bool((room[4 + shift + T * E:] == 7).all())
