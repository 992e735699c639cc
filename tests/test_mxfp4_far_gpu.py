"""The experts' 4-bit products of rows that a map takes from more than 4 GiB of codes, in tiles; against the definition in 64 bits with
the bounds of test_mxfp4_gpu."""
import pytest

torch = pytest.importorskip("torch")
from test_mxfp4_gpu import BF16, DEV, F32, I32, U8, expected, half, rows4, standard, values  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import unpermute_combine_amd as mod
    mod.lib()
    return mod


def far_rows(seed, H):
    """(codes, scales) of just over 4 GiB of codes, and the places of the 450 rows that hold anything: the first, those around 4 GiB
    and the last. All others have NaN scales."""
    n = (1 << 32) // (H // 2) + 1000
    at = torch.cat([torch.arange(150) + a for a in (0, (1 << 32) // (H // 2) - 75, n - 150)]).to(DEV)
    x = torch.zeros(n, H // 2, dtype=U8, device=DEV), torch.full((n, H // 32), 255, dtype=U8, device=DEV)
    x[0][at], x[1][at] = rows4(seed, len(at), H)
    assert x[0].numel() > 0xfffffff0
    return x, at


def mapped(seed, at, n, R):
    """A map [R] onto the places `at` of n rows, some outside, and each row's number in `at` (-1: a row of zeros)."""
    pick = torch.randint(-20, len(at), (R,), generator=torch.Generator().manual_seed(seed)).to(DEV)
    pick[:4] = torch.tensor([0, len(at) - 1, 225, -1])
    outside = torch.tensor([-1, n, (1 << 31) - 1, -(1 << 31)], device=DEV)[pick.clamp_max(0) % 4]
    return torch.where(pick >= 0, at[pick.clamp_min(0)], outside).to(I32), pick


def assert_product(out, x, at, pick, wv, segments, gated):
    """Rows of out against the definition; wv the weights' values, as many as out has columns."""
    xv = torch.where((pick >= 0)[:, None], values(x[0][at], x[1][at])[pick.clamp_min(0)], 0.0)
    want, bound, written = expected(xv, wv, segments, len(pick), gated)
    h = half(out.dtype)
    off = ((out.double() - want).abs() / (bound * (1 + h) + h * want.abs() + 1e-37))[written]
    assert float(off.max()) <= 1, f"{int((off > 1).sum())} values off, worst {float(off.max()):.3g} of the bound"


# (N: tiles fewer than CUs, and as many: the two sizes of tiles, at each of their heights; H: whole and ragged stages)
@pytest.mark.parametrize("lengths,H,N", [([300, 7, 0, 255], 4096, 130), ([300, 7, 0, 40, 600], 4128, 17000), ([100, 170, 300], 4096, 25000)])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_rows_through_a_map_past_4_gib(m, lengths, H, N, gated, out_dtype):
    print(f"far {lengths} H{H} N{N} gated {gated} {out_dtype}", flush=True)
    R, E = sum(lengths), len(lengths)
    x, at = far_rows(R, H)
    w = rows4(N, E, N * (2 if gated else 1), H)
    src, pick = mapped(R, at, x[0].shape[0], R)
    segments, gl = standard(lengths)
    room = torch.full((R + 2, N), 7.0, dtype=out_dtype, device=DEV)
    m.grouped_product_mxfp4(*x, *w, gl, src_row=src, gated=gated, out=room[1:-1])
    assert bool((room[0] == 7).all()) and bool((room[-1] == 7).all())
    assert_product(room[1:-1], x, at, pick, values(*w), segments, gated)


def test_many_rows_and_columns_through_a_map_past_4_gib(m):
    """Sizes that 16 rows a workgroup would pass a launch's limit with: 16400 rows of one expert by 2^20 columns, gated."""
    H, N, R, step = 4096, 1 << 20, 16400, 8192
    x, at = far_rows(1, H)
    w = torch.zeros(1, 2 * N, H // 2, dtype=U8, device=DEV), torch.full((1, 2 * N, H // 32), 127, dtype=U8, device=DEV)
    some = rows4(2, 1, 2 * N // step, H)
    w[0][:, ::step], w[1][:, ::step] = some
    src, pick = mapped(3, at, x[0].shape[0], R)
    out = m.grouped_product_mxfp4(*x, *w, torch.tensor([R], dtype=I32, device=DEV), src_row=src, gated=True)
    assert_product(out[:, ::step], x, at, pick, values(*some), [(0, R)], True)
    assert not out[:, 1::step].any() and not out[:, step - 1::step].any()
