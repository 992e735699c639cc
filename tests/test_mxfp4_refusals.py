"""What the 4-bit quantisation and the grouped product refuse, before any launch (no GPU needed)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(4096)  # never dereferenced on the host


@pytest.fixture(scope="module")
def capi():
    from unpermute_combine_amd import _capi
    return _capi


def test_quantize_refusals(capi):
    f, B, Q = capi.lib().moe_quantize_mxfp4, capi.MOE_BF16, capi.MOE_FP8_E4M3
    call = lambda x=P, dt=B, T=4, H=64, q=P, s=P: f(x, dt, T, H, q, s, None)  # noqa: E731
    assert call(T=0) == call(T=0, x=None, q=None, s=None) == capi.MOE_OK
    for bad in (dict(T=-1), dict(H=0), dict(H=-32), dict(H=33), dict(H=16), dict(x=None), dict(q=None), dict(s=None), dict(dt=7)):
        assert call(**bad) == capi.MOE_ERR_INVALID, bad
    for bad in (dict(dt=Q), dict(T=1 << 31), dict(H=1 << 27), dict(dt=capi.MOE_F32, T=1 << 30, H=32), dict(T=1 << 30, H=128)):
        assert call(**bad) == capi.MOE_ERR_UNSUPPORTED, bad


def test_product_refusals(capi):
    f, F, B, Q = capi.lib().moe_grouped_product_mxfp4, capi.MOE_F32, capi.MOE_BF16, capi.MOE_FP8_E4M3
    call = lambda x=P, xs=P, xr=8, sr=None, R=8, H=64, w=P, ws=P, E=4, N=48, gated=0, gl=P, ct=None, cap=0, o=P, od=B: f(  # noqa: E731
        x, xs, xr, sr, R, H, w, ws, E, N, gated, gl, ct, cap, o, od, None)
    assert call(R=0, xr=0) == call(R=0, xr=0, x=None, xs=None, w=None, ws=None, gl=None, o=None) == capi.MOE_OK
    for bad in (dict(R=-1), dict(xr=-1), dict(H=0), dict(H=48), dict(N=0), dict(E=0), dict(cap=-1), dict(od=9), dict(x=None),
                dict(xs=None), dict(w=None), dict(ws=None), dict(gl=None), dict(o=None),
                dict(xr=7),  # fewer rows than R, and no map
                dict(cap=2, ct=None), dict(cap=3, ct=P)):  # no counts; 4 experts of 3 rows do not fit into 8
        assert call(**bad) == capi.MOE_ERR_INVALID, bad
    for bad in (dict(od=Q), dict(E=1025), dict(R=1 << 31, xr=1 << 31), dict(H=(1 << 20) + 32), dict(N=(1 << 20) + 1),
                dict(x=ctypes.c_void_p(4104)), dict(w=ctypes.c_void_p(4097)), dict(R=1 << 30, sr=P, N=1 << 20),
                dict(R=8192, xr=8192, E=1024, N=1 << 20, H=32, gated=1)):  # rows of 16 by 64 columns: 1536 * 2^14 workgroups
        assert call(**bad) == capi.MOE_ERR_UNSUPPORTED, bad


def test_binding_refuses_host_tensors():
    import unpermute_combine_amd as m
    q, s = torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.quantize_mxfp4(torch.ones(2, 64))
    with pytest.raises(ValueError, match="GPU tensor"):
        m.grouped_product_mxfp4(q, s, q[None], s[None], torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        m.quantize_mxfp4(None)
