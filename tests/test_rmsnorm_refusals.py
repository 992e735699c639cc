"""What the residual RMS norm refuses, before any launch (no GPU needed), and its formulas against differences."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(4096)  # never dereferenced on the host


@pytest.fixture(scope="module")
def capi():
    from unpermute_combine_amd import _capi
    return _capi


def test_forward_refusals(capi):
    f = capi.lib().moe_add_rmsnorm
    F, B, Q, INV, UNS = capi.MOE_F32, capi.MOE_BF16, capi.MOE_FP8_E4M3, capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED
    call = lambda x=P, xd=B, r=P, sd=B, w=P, wd=F, T=4, H=64, eps=1e-6, so=P, o=P, od=B, rs=P: f(  # noqa: E731
        x, xd, r, sd, w, wd, T, H, eps, so, o, od, rs, None)
    assert call(T=0) == capi.MOE_OK
    assert call(T=0, x=None, w=None, o=None) == capi.MOE_OK
    for bad in (dict(T=-1), dict(H=0), dict(eps=-1e-6), dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None),
                dict(w=None), dict(o=None), dict(xd=7), dict(sd=7), dict(wd=7), dict(od=7)):
        assert call(**bad) == INV, bad
    for bad in (dict(xd=Q), dict(sd=Q), dict(wd=Q), dict(od=Q), dict(H=1 << 30), dict(T=1 << 31)):
        assert call(**bad) == UNS, bad


def test_fp8_refusals(capi):
    f = capi.lib().moe_add_rmsnorm_fp8
    F, B, Q, INV, UNS = capi.MOE_F32, capi.MOE_BF16, capi.MOE_FP8_E4M3, capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED
    call = lambda x=P, xd=B, r=P, sd=B, w=P, wd=F, T=4, H=64, eps=1e-6, block=32, so=P, o=P, od=B, q=P, sc=P, rs=P: f(  # noqa: E731
        x, xd, r, sd, w, wd, T, H, eps, block, so, o, od, q, sc, rs, None)
    assert call(T=0) == capi.MOE_OK
    for bad in (dict(block=0), dict(block=-8), dict(block=48), dict(block=128), dict(q=None), dict(sc=None), dict(x=None),
                dict(w=None), dict(T=-1), dict(H=0), dict(eps=-1.0), dict(od=9)):
        assert call(**bad) == INV, bad
    for bad in (dict(xd=Q), dict(sd=Q), dict(od=Q), dict(T=1 << 31)):
        assert call(**bad) == UNS, bad


def test_backward_refusals_and_workspace(capi):
    lib = capi.lib()
    n = ctypes.c_size_t(0)
    size = lambda T, H: (lib.moe_add_rmsnorm_backward_workspace_size(T, H, ctypes.byref(n)), n.value)  # noqa: E731
    assert size(0, 64) == (capi.MOE_OK, 0)
    assert size(-1, 64)[0] == size(4, 0)[0] == capi.MOE_ERR_INVALID
    assert lib.moe_add_rmsnorm_backward_workspace_size(4, 64, None) == capi.MOE_ERR_INVALID
    assert size(4, 1 << 30)[0] == capi.MOE_ERR_UNSUPPORTED
    st, need = size(16384, 7168)
    assert st == capi.MOE_OK and 4 * 7168 <= need <= 4 * 7168 * 1024  # the ranges' sums
    F, B, Q, INV, UNS = capi.MOE_F32, capi.MOE_BF16, capi.MOE_FP8_E4M3, capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED
    need = size(4, 64)[1]
    call = lambda g=P, gd=B, h=P, hd=B, w=P, wd=F, rs=P, d=P, T=4, H=64, dx=P, dd=B, dw=P, ws=P, wb=need: (  # noqa: E731
        lib.moe_add_rmsnorm_backward(g, gd, h, hd, w, wd, rs, d, T, H, dx, dd, dw, ws, wb, None))
    assert call(T=0, dw=None) == capi.MOE_OK
    for bad in (dict(T=-1), dict(H=0), dict(g=None), dict(h=None), dict(w=None), dict(rs=None), dict(dx=None), dict(ws=None),
                dict(wb=need - 1), dict(ws=ctypes.c_void_p(4097)), dict(gd=9), dict(hd=9), dict(dd=9)):
        assert call(**bad) == INV, bad
    for bad in (dict(gd=Q), dict(hd=Q), dict(wd=Q), dict(dd=Q), dict(T=1 << 31)):
        assert call(**bad) == UNS, bad


def test_rows_longer_than_the_grids_take_are_refused(capi):
    lib, n = capi.lib(), ctypes.c_size_t(0)
    F, UNS, H = capi.MOE_F32, capi.MOE_ERR_UNSUPPORTED, (1 << 26) + 8
    assert lib.moe_add_rmsnorm_backward_workspace_size(1, 1 << 26, ctypes.byref(n)) == capi.MOE_OK and n.value == 4 << 26
    assert lib.moe_add_rmsnorm_backward_workspace_size(1, H, ctypes.byref(n)) == UNS
    assert lib.moe_add_rmsnorm_backward(P, F, P, F, P, F, P, None, 1, H, P, F, P, P, 4 * H, None) == UNS
    assert lib.moe_add_rmsnorm(P, F, None, F, P, F, 1, H, 1e-6, None, P, F, None, None) == UNS
    assert lib.moe_add_rmsnorm_fp8(P, F, None, F, P, F, 1, H, 1e-6, 8, None, None, F, P, P, None, None) == UNS


def test_binding_refuses_host_tensors():
    import unpermute_combine_amd as m
    x, w = torch.ones(2, 64), torch.ones(64)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.add_rmsnorm(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.add_rmsnorm_fp8(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.add_rmsnorm_backward(x, x, w, torch.ones(2))
    with pytest.raises(TypeError):
        m.add_rmsnorm(None, w)


def test_backward_formula_against_differences():
    """dx and dweight as the header writes them, against torch's finite differences of the forward, in 64 bits."""
    g = torch.Generator().manual_seed(3)
    eps = 1e-3

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, h, w):
            s = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
            ctx.save_for_backward(h, w, s)
            return h * s * w

        @staticmethod
        def backward(ctx, dout):
            h, w, s = ctx.saved_tensors
            a = dout * w
            m = s * s * (a * h).mean(1, keepdim=True)
            return s * (a - h * m), (dout * h * s).sum(0)

    h = torch.randn(5, 7, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(7, generator=g, dtype=torch.float64, requires_grad=True)
    assert torch.autograd.gradcheck(Norm.apply, (h, w))
