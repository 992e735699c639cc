"""What the few-token layer refuses, before any launch (no GPU needed)."""
import ctypes

import pytest

P = ctypes.c_void_p(4096)  # never dereferenced on the host


@pytest.fixture(scope="module")
def capi():
    from unpermute_combine_amd import _capi
    return _capi


def need(capi, T, H, I, E, K):
    n = ctypes.c_size_t(0)
    return capi.lib().moe_few_token_workspace_size(T, H, I, E, K, ctypes.byref(n)), n.value


def test_workspace_size(capi):
    assert need(capi, 0, 64, 64, 4, 2) == (capi.MOE_OK, 0)
    st, n = need(capi, 64, 7168, 1024, 256, 8)
    assert st == capi.MOE_OK and 64 * 8 * (1024 + 7168) * 4 <= n <= 64 * 8 * (1024 + 7168) * 5  # h and the products, and the little else
    assert capi.lib().moe_few_token_workspace_size(1, 64, 64, 4, 2, None) == capi.MOE_ERR_INVALID
    for bad in ((-1, 64, 64, 4, 2), (1, 0, 64, 4, 2), (1, 64, 0, 4, 2), (1, 64, 64, 0, 1), (1, 64, 64, 4, 0), (1, 64, 64, 4, 5)):
        assert need(capi, *bad)[0] == capi.MOE_ERR_INVALID, bad
    for bad in ((257, 64, 64, 4, 2), (1, 64, 64, 1025, 2), (1, 64, 64, 64, 33), (1, (1 << 24) + 1, 64, 4, 2), (1, 64, 1 << 25, 4, 2)):
        assert need(capi, *bad)[0] == capi.MOE_ERR_UNSUPPORTED, bad


def test_argument_errors(capi):
    lib = capi.lib()
    F, B, Q, INV, UNS = capi.MOE_F32, capi.MOE_BF16, capi.MOE_FP8_E4M3, capi.MOE_ERR_INVALID, capi.MOE_ERR_UNSUPPORTED
    ws = need(capi, 4, 256, 128, 8, 2)[1]

    def layer(x=P, dt=B, r=P, T=4, H=256, I=128, E=8, K=2, gs=0, M=0, a=P, b=P, wd=B, sa=None, sb=None, block=0, bias=None, o=P,
              od=B, idx=P, w=P, wsp=P, wb=ws):
        return lib.moe_few_token_layer(x, dt, r, T, H, I, E, K, gs, M, a, b, wd, sa, sb, block, bias, o, od, idx, w, wsp, wb, None)

    def experts(x=P, dt=B, T=4, H=256, I=128, E=8, K=2, idx=P, w=P, a=P, b=P, wd=B, sa=None, sb=None, block=0, bias=None, o=P,
                od=B, wsp=P, wb=ws):
        return lib.moe_few_token_experts(x, dt, T, H, I, E, K, idx, w, a, b, wd, sa, sb, block, bias, o, od, wsp, wb, None)

    fp8 = dict(wd=Q, sa=P, sb=P, block=128)
    for f in (layer, experts):
        assert f(T=0) == f(T=0, wsp=None, wb=0, x=None) == f(T=0, **fp8) == capi.MOE_OK
        for bad in (dict(T=-1), dict(H=0), dict(I=0), dict(E=0), dict(K=0), dict(K=9), dict(x=None), dict(a=None), dict(b=None),
                    dict(o=None), dict(idx=None), dict(dt=5), dict(wd=5), dict(od=5), dict(wsp=None), dict(wb=ws - 1),
                    dict(wsp=ctypes.c_void_p(4104)), dict(fp8, sa=None), dict(fp8, sb=None), dict(fp8, block=0),
                    dict(fp8, block=48), dict(fp8, block=256), dict(fp8, block=-128)):
            assert f(**bad) == INV, bad
        for bad in (dict(dt=Q), dict(od=Q), dict(dt=F), dict(wd=F), dict(fp8, dt=F), dict(fp8, block=64), dict(T=257),
                    dict(E=2000), dict(E=64, K=40)):
            assert f(**bad) == UNS, bad
    for bad in (dict(r=None), dict(w=None), dict(gs=3, M=1), dict(gs=4, M=0), dict(gs=4, M=3), dict(gs=1, M=1)):
        assert layer(**bad) == INV, bad
    big = need(capi, 1, 256, 128, 1024, 2)[1]
    assert layer(T=1, E=1024, gs=2, M=4, wb=big) == UNS  # more than 256 groups


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    import unpermute_combine_amd as m
    x, r, a, b = torch.ones(2, 64), torch.ones(4, 64), torch.ones(4, 64, 64), torch.ones(4, 64, 32)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.few_token_layer(x, r, a, b, 2)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.few_token_experts(x, torch.zeros(2, 2, dtype=torch.int32), None, a, b)


def test_a_rank_may_hold_fewer_experts_than_slots_a_token(capi):
    """moe_few_token_experts takes a routing whose ids repeat or name experts held elsewhere, so K may exceed E; the layer, which
    routes by itself, needs K different experts."""
    lib, n = capi.lib(), ctypes.c_size_t(0)
    size = lambda f, *a: (f(*a, ctypes.byref(n)), n.value)  # noqa: E731
    experts, layer = lib.moe_few_token_experts_workspace_size, lib.moe_few_token_workspace_size
    for sizes in ((1, 64, 64, 4, 2), (16, 512, 256, 8, 8), (256, 4096, 2048, 64, 8)):
        assert size(experts, *sizes) == size(layer, *sizes) and n.value > 0
    for E, K in ((1, 32), (3, 8), (7, 8)):
        st, need = size(experts, 256, 512, 128, E, K)
        assert st == capi.MOE_OK and need >= 4 * 256 * K * (512 + 128)  # h and the products of every slot
        assert size(layer, 256, 512, 128, E, K)[0] == capi.MOE_ERR_INVALID
    assert size(experts, 0, 64, 64, 4, 5) == (capi.MOE_OK, 0)
    assert experts(1, 64, 64, 4, 2, None) == capi.MOE_ERR_INVALID
    for bad in ((-1, 64, 64, 4, 2), (1, 0, 64, 4, 2), (1, 64, 0, 4, 2), (1, 64, 64, 0, 1), (1, 64, 64, 4, 0)):
        assert size(experts, *bad)[0] == capi.MOE_ERR_INVALID, bad
    for bad in ((257, 64, 64, 4, 5), (1, 64, 64, 1025, 2), (1, 64, 64, 4, 33), (1, (1 << 20) + 1, 64, 4, 5)):
        assert size(experts, *bad)[0] == capi.MOE_ERR_UNSUPPORTED, bad
    B = capi.MOE_BF16
    assert lib.moe_few_token_experts(P, B, 0, 256, 128, 3, 8, P, P, P, P, B, None, None, 0, None, P, B, None, 0, None) == capi.MOE_OK
    need = size(experts, 4, 256, 128, 3, 8)[1]
    assert lib.moe_few_token_experts(P, B, 4, 256, 128, 3, 8, P, P, P, P, B, None, None, 0, None, P, B, P, need - 1,
                                     None) == capi.MOE_ERR_INVALID
    assert lib.moe_few_token_layer(P, B, P, 0, 256, 128, 3, 8, 0, 0, P, P, B, None, None, 0, None, P, B, P, P, P, need,
                                   None) == capi.MOE_ERR_INVALID
