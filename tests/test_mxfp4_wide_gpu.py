"""The experts' 4-bit products in the widest tiles with rows of a multiple of 512, whose scales come by whole lines (in other calls 16
bytes at a time): every height of a tile, rows dealt out over several, plain and gated, direct and through a map; and weights past 4 GiB,
gated. Bounds are those of test_mxfp4_gpu."""
import pytest

torch = pytest.importorskip("torch")
from test_mxfp4_gpu import BF16, DEV, F32, I32, U8, check, expected, half, rows4, standard, values  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import unpermute_combine_amd as mod
    mod.lib()
    return mod


# (experts with rows) * ceil(N / 256) >= 256, plain and gated, is what the widest tiles are taken for
SIZES = [
    # one line a row: its second half is the next row's. Heights 256, 44, 7 and 255
    ([300, 7, 0, 255], 512, 22000),
    # heights 130, 256, 4, 40, 70 and 1
    ([130, 260, 40, 70, 1], 1536, 14001),
    # long rows, dealt out evenly: 33, 64, 100, 192 192 136, 180, 256 194, 32
    ([33, 64, 100, 520, 180, 450, 32], 2560, 11000),
    # one after the other of four tiles
    ([1000, 0, 16], 2048, 33000),
]


@pytest.mark.parametrize("lengths,H,N", SIZES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_product(m, lengths, H, N, gated, out_dtype):
    print(f"wide {lengths} H{H} N{N} gated {gated} {out_dtype}", flush=True)
    R, E = sum(lengths), len(lengths)
    assert min(R, E) * (N // 256) >= 256 or (R // 256) * (N // 256) >= 256
    x, w = rows4(R + H, R, H), rows4(N, E, N * (2 if gated else 1), H)
    segments, gl = standard(lengths)
    check(m, x, w, segments, gl, out_dtype, gated)


@pytest.mark.parametrize("lengths,H,N", SIZES)
@pytest.mark.parametrize("gated", [False, True])
def test_rows_through_a_map(m, lengths, H, N, gated):
    print(f"wide map {lengths} H{H} N{N} gated {gated}", flush=True)
    R, E, rows = sum(lengths), len(lengths), sum(lengths) // 3
    x, w = rows4(R, rows, H), rows4(N, E, N * (2 if gated else 1), H)
    src = torch.randint(-2, rows + 2, (R,), generator=torch.Generator().manual_seed(R), dtype=I32).to(DEV)
    src[0] = -(1 << 31)
    src[-1] = (1 << 31) - 1
    segments, gl = standard(lengths)
    check(m, x, w, segments, gl, BF16, gated, src_row=src)


@pytest.mark.parametrize("gated", [False, True])
def test_scales_that_are_nan_stay_with_their_rows(m, gated):
    lengths, H, N = [200, 3, 40], 1536, 30000
    R = sum(lengths)
    x, w = rows4(10, R, H), rows4(11, 3, N * (2 if gated else 1), H)
    x[1][5, 0] = x[1][150, 47] = x[1][201, 16] = 255
    w[1][0, 17, 3] = w[1][2, -1, 47] = 255
    segments, gl = standard(lengths)
    check(m, x, w, segments, gl, F32, gated)
    # rows that are not there, beside weights whose scales are NaN: those columns alone
    src = torch.arange(R, dtype=I32, device=DEV)
    src[::3] = -1
    check(m, x, w, segments, gl, BF16, gated, src_row=src)


@pytest.mark.parametrize("gated,N", [(True, 17000), (False, 33000)])
@pytest.mark.parametrize("mapped", [False, True])
def test_lines_and_pieces_of_scales_agree(m, gated, N, mapped):
    """Scales at odd addresses come 16 bytes at a time: the same products, bit for bit."""
    lengths, H = [30, 300, 90], 1024
    R = sum(lengths)
    x, w = rows4(14, R, H), rows4(15, 3, N * (2 if gated else 1), H)
    segments, gl = standard(lengths)
    src = torch.randperm(R, generator=torch.Generator().manual_seed(3)).to(I32).to(DEV) if mapped else None
    want = check(m, x, w, segments, gl, F32, gated, src_row=src)
    for shift in (1, 3):
        sx, sw = (torch.empty(t.numel() + 8, dtype=U8, device=DEV)[shift:shift + t.numel()].view(t.shape).copy_(t) for t in (x[1], w[1]))
        assert torch.equal(m.grouped_product_mxfp4(x[0], sx, w[0], w[1], gl, src_row=src, gated=gated, out_dtype=F32), want)
        assert torch.equal(m.grouped_product_mxfp4(x[0], x[1], w[0], sw, gl, src_row=src, gated=gated, out_dtype=F32), want)


@pytest.mark.parametrize("capacity", [300, 40])
def test_segments_with_counts(m, capacity):
    """Drop-and-pad and aligned segments in the widest tiles."""
    E, H, N = 6, 1024, 12000
    kept = torch.tensor([capacity, 0, 17, capacity - 1, 1, capacity // 2], dtype=I32)
    x, w = rows4(20, E * capacity, H), rows4(21, E, N, H)
    segments = [(e * capacity, e * capacity + int(c)) for e, c in enumerate(kept)]
    check(m, x, w, segments, None, BF16, counts=kept.to(DEV), capacity=capacity)
    ends = (torch.arange(1, E + 1, dtype=I32) * capacity).to(DEV)
    check(m, x, w, segments, ends, BF16, counts=kept.to(DEV))


@pytest.mark.parametrize("rows", [30, 90])
def test_gated_weights_past_4_gib(m, rows):
    """Gates and ups of 2^18 columns of five experts, 5.4 GB of codes; the last expert's are used, by the few-row kernel and by tiles."""
    E, N, H, step = 5, 1 << 19, 4096, 8192
    w = torch.zeros(E, N, H // 2, dtype=U8, device=DEV), torch.full((E, N, H // 32), 127, dtype=U8, device=DEV)
    some = rows4(16, 1, N // step, H)
    w[0][-1, ::step], w[1][-1, ::step] = some[0][0], some[1][0]
    x = rows4(17, rows, H)
    a = rows // 3
    out = m.grouped_product_mxfp4(*x, *w, torch.tensor([0, 0, 0, a, rows], dtype=I32, device=DEV), gated=True, out_dtype=F32)
    want, bound, _ = expected(values(*x)[a:], values(*some), [(0, rows - a)], rows - a, True)
    lim = bound * (1 + half(F32)) + half(F32) * want.abs() + 1e-37
    off = (out[a:, ::step].double() - want).abs() / lim
    assert float(off.max()) <= 1, f"worst {float(off.max()):.3g} of the bound"
    assert not out[:a].any() and not out[a:, 1::step].any() and not out[a:, step - 1::step].any()
