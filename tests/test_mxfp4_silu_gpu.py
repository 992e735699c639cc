"""The gate of the experts' 4-bit products, silu(g) = g / (1 + exp(-g)), for values of g given bit by bit.

A float32 g is a sum of 24 powers of two or less; each is a block of a row of x (code +-1, the power its scale) against a code 1 of
the weights, so that the sum is g whatever its order, and a block of its own gives the up. With u = 2^-24, -log2(e) g rounds once
(the constant in two parts), u |g| in e^-g; the instructions for 2^x and 1 / x are right to 2 u each, the sum and the product round
once: (|g| + 6) u of silu. Where 1 / (1 + e^-g) is below the normal float32 (g < -87.3) it has 21 bits or more, 4 u besides; past
g = -88.72 e^-g passes float32 and silu is 0."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
U8, I32, F32 = torch.uint8, torch.int32, torch.float32
H, N = 1024, 16
ONE = 2  # the code of 1


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import unpermute_combine_amd as mod
    mod.lib()
    return mod


def pack(codes):
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).to(U8).to(DEV)


def gates(m, g, up, experts):
    """silu(g) * up as the kernels give it; up a power of two. One expert takes tiles, eight rows of each the few-row kernel."""
    R = g.numel()
    assert R % experts == 0 and torch.isfinite(g).all()
    mantissa, exponent = torch.frexp(g.abs().double())
    bits = (mantissa * 2 ** 24).long()
    codes, scales = torch.zeros(R, H // 32, 32, dtype=torch.int64), torch.full((R, H // 32), 127, dtype=torch.int64)
    for b in range(24):
        codes[:, b, 0] = (bits >> b & 1) * (ONE + 8 * (g < 0))
        scales[:, b] = (127 + exponent - 24 + b).clamp(0, 254)
    codes[:, 24, 0] = ONE
    w, ws = torch.zeros(2 * N, H // 32, 32, dtype=torch.int64), torch.full((2 * N, H // 32), 127, dtype=torch.int64)
    w[:N, :24, 0] = ONE
    w[N:, 24, 0] = ONE
    ws[N:, 24] = 127 + up
    x, xs = pack(codes.view(R, H)), scales.to(U8).to(DEV)
    w = pack(w.view(2 * N, H)).expand(experts, -1, -1).contiguous()
    ws = ws.to(U8).to(DEV).expand(experts, -1, -1).contiguous()
    ends = (torch.arange(1, experts + 1, dtype=I32) * (R // experts)).to(DEV)
    y = m.grouped_product_mxfp4(x, xs, w, ws, ends, out_dtype=F32)
    assert torch.equal(y[:, :N], g.to(DEV)[:, None].expand(R, N)) and bool((y[:, N:] == 2.0 ** up).all())
    out = m.grouped_product_mxfp4(x, xs, w, ws, ends, gated=True, out_dtype=F32)
    assert torch.equal(out, out[:, :1].expand(R, N))
    return out[:, 0].double().cpu()


@pytest.mark.parametrize("experts", [1, 512])
def test_silu_to_its_bound(m, experts):
    g = torch.empty(8 * 512).uniform_(-87.3, 87.3, generator=torch.Generator().manual_seed(1))
    g[:2048] = torch.linspace(-46, -20, 2048)
    g[2048], g[2049] = -44.37, -22.24
    got, want = gates(m, g, 0, experts), g.double() * torch.sigmoid(g.double())
    off = (got - want).abs() / (want.abs() * (g.double().abs() + 6) * U)
    assert float(off.max()) <= 1, f"g = {float(g[off.argmax()])}: {float(off.max()):.3g} of the bound"


@pytest.mark.parametrize("experts", [1, 512])
def test_silu_before_its_exponential_overflows(m, experts):
    """g in (-88.72, -87.3) beside an up of 2^60: outputs that float32 holds well."""
    g = torch.linspace(-88.72, -87.3, 8 * 512)
    got, want = gates(m, g, 60, experts), g.double() * torch.sigmoid(g.double()) * 2.0 ** 60
    off = (got - want).abs() / (want.abs() * (g.double().abs() + 10) * U)
    assert float(off.max()) <= 1, f"g = {float(g[off.argmax()])}: {float(off.max()):.3g} of the bound"


@pytest.mark.parametrize("experts", [1, 512])
def test_silu_at_its_ends(m, experts):
    g = torch.zeros(8 * 512)
    g[:8] = torch.tensor([0.0, -88.75, -100.0, -2.0 ** 30, 2.0 ** 30, 100.0, 2.0 ** -40, -2.0 ** -40])
    got = gates(m, g, 0, experts)
    assert not got[:4].any() and not got[8:].any()
    assert got[4] == 2.0 ** 30 and got[5] == 100 and got[6] == 2.0 ** -41 and got[7] == -(2.0 ** -41)
