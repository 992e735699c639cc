"""What the balance loss refuses, before any launch (no GPU needed), and its gradient's formula against differences."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(4096)  # never dereferenced on the host


@pytest.fixture(scope="module")
def capi():
    from unpermute_combine_amd import _capi
    return _capi


def test_workspace_size(capi):
    lib, n = capi.lib(), ctypes.c_size_t(0)
    size = lambda T, E: (lib.moe_balance_loss_workspace_size(T, E, ctypes.byref(n)), n.value)  # noqa: E731
    assert size(0, 8) == size(1, 8) == (capi.MOE_OK, 0)  # one workgroup: nothing to put together
    st, big = size(1 << 20, 256)
    assert st == capi.MOE_OK and 0 < big <= 512 * (8 * 257) + 1024
    assert size(-1, 8)[0] == size(4, 0)[0] == lib.moe_balance_loss_workspace_size(4, 8, None) == capi.MOE_ERR_INVALID
    assert size(4, 1025)[0] == size(1 << 31, 8)[0] == capi.MOE_ERR_UNSUPPORTED


def test_forward_refusals(capi):
    lib, n = capi.lib(), ctypes.c_size_t(0)
    assert lib.moe_balance_loss_workspace_size(20000, 64, ctypes.byref(n)) == capi.MOE_OK
    need = n.value
    call = lambda lg=P, ix=P, mk=None, T=20000, E=64, K=2, coef=0.01, ls=P, ct=P, ps=P, tk=P, ws=P, wb=need: (  # noqa: E731
        lib.moe_balance_loss(lg, ix, mk, T, E, K, coef, ls, ct, ps, tk, ws, wb, None))
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=65), dict(coef=float("nan")), dict(coef=float("inf")), dict(lg=None),
                dict(ix=None), dict(ls=None), dict(ct=None), dict(ps=None), dict(tk=None), dict(ws=None), dict(wb=need - 1),
                dict(ws=ctypes.c_void_p(4100))):
        assert call(**bad) == capi.MOE_ERR_INVALID, bad
    for bad in (dict(E=1025), dict(K=33), dict(T=1 << 30, wb=1 << 30), dict(T=1 << 31, wb=1 << 30)):
        assert call(**bad) == capi.MOE_ERR_UNSUPPORTED, bad


def test_backward_refusals(capi):
    lib = capi.lib()
    call = lambda lg=P, mk=None, ct=P, tk=P, dl=None, T=4, E=64, K=2, coef=0.01, di=None, d=P: (  # noqa: E731
        lib.moe_balance_loss_backward(lg, mk, ct, tk, dl, T, E, K, coef, di, d, None))
    assert call(T=0) == call(T=0, lg=None, ct=None, tk=None, d=None) == capi.MOE_OK
    for bad in (dict(T=-1), dict(E=0), dict(K=0), dict(K=65), dict(coef=float("inf")), dict(lg=None), dict(ct=None), dict(tk=None),
                dict(d=None)):
        assert call(**bad) == capi.MOE_ERR_INVALID, bad
    for bad in (dict(E=1025), dict(K=33), dict(T=1 << 30)):
        assert call(**bad) == capi.MOE_ERR_UNSUPPORTED, bad


def test_binding_refuses_host_tensors():
    import unpermute_combine_amd as m
    lg, ix = torch.ones(2, 8), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.balance_loss(lg, ix)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.balance_loss_backward(lg, ix[0], ix[0, :1], 2)
    with pytest.raises(TypeError):
        m.balance_loss(None, ix)


def test_gradient_formula_against_differences():
    """d_logits as the header writes it, against torch's finite differences of the loss, in 64 bits."""
    g = torch.Generator().manual_seed(5)
    T, E, K, coef = 6, 5, 2, 0.3
    keep = torch.tensor([1, 1, 0, 1, 1, 1], dtype=torch.bool)
    counts = torch.tensor([4.0, 1.0, 0.0, 3.0, 2.0], dtype=torch.float64)
    n = int(keep.sum())
    f = counts / (n * K)

    class Loss(torch.autograd.Function):
        @staticmethod
        def forward(ctx, z):
            p = torch.softmax(z, 1)
            ctx.save_for_backward(p)
            return coef * E * (f * p[keep].sum(0) / n).sum()

        @staticmethod
        def backward(ctx, d):
            p, = ctx.saved_tensors
            return torch.where(keep[:, None], d * coef * E / n * p * (f - (p * f).sum(1, keepdim=True)), 0.0)

    z = torch.randn(T, E, generator=g, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(Loss.apply, (z,))
