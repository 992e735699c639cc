"""Rows in 4 bits (MXFP4) and the experts' products on the GPU against their definitions in 64 bits.

Codes and scales are equal bit for bit. Products of two codes and their scales are exact in float32; a sum of H of them has fewer
than H + 48 roundings of u = 2^-24 on any term's way, counting the matrix instructions' own as one for each term (they sum 128
terms at a time, to about 3 u of the sum of the magnitudes)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import unpermute_combine_amd as mod
    mod.lib()
    return mod


def half(dtype):
    return torch.finfo(dtype).eps / 2


def draw(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def pow2(e):
    """2^e in 64 bits, by the exponent's field (torch.ldexp goes through a float32 power, which is not exact)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


# ---------------------------------------------------------------- quantisation


def quantized(x):
    """(q, scales) by the definition, in 64 bits."""
    v = x.double().view(x.shape[0], -1, 32)
    top = v.abs().amax(2)
    finite = torch.isfinite(top)
    exponent = torch.frexp(torch.where(finite & (top > 0), top, 4.0)).exponent - 1  # floor(log2 top)
    e = (exponent - 2).clamp_min(-127)
    r = torch.where(finite[:, :, None], v * pow2(-e)[:, :, None], 0.0)
    a = r.abs()
    ties_up = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    code = torch.where(finite[:, :, None], ties_up + 8 * torch.signbit(v), 0).view(x.shape)
    scales = torch.where(finite, torch.where(top > 0, e, 0) + 127, 255)
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(U8), scales.to(U8)


def assert_quantized(m, x):
    q, s = m.quantize_mxfp4(x)
    want_q, want_s = quantized(x)
    assert q.dtype == s.dtype == U8
    assert torch.equal(s, want_s), f"{int((s != want_s).sum())} scales differ"
    assert torch.equal(q, want_q), f"{int((q != want_q).sum())} bytes of codes differ"


@pytest.mark.parametrize("T,H", [(1, 32), (1, 7168), (3, 64), (5, 96), (33, 1056), (64, 4096), (257, 7168), (1000, 160), (9, 32 * 1023)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_quantize(m, T, H, dt):
    x = draw(T + H, T, H) * torch.exp(2 * draw(1, T, H))
    x[T // 2, :32] = 0
    assert_quantized(m, x.to(dt))


def test_quantize_every_bf16_in_blocks_of_every_exponent(m):
    """Each finite bf16 value beside a largest element of 2^k and of just under 2^(k+1), for k over bf16's whole range."""
    bits = torch.arange(65536, dtype=I32)
    v = (bits << 16).view(F32)
    v = v[torch.isfinite(v)].to(DEV)
    for k in list(range(-132, -120)) + list(range(-6, 7)) + [100, 126, 127]:
        for lead in (2.0 ** k, 2.0 ** k * 1.9921875):
            w = torch.where(v.abs() <= lead, v, 0.0)
            rows = torch.zeros(-(-len(w) // 31), 32, device=DEV)
            rows[:, 1:] = torch.nn.functional.pad(w, (0, rows.shape[0] * 31 - len(w))).view(-1, 31)
            rows[:, 0] = lead
            assert_quantized(m, rows.bfloat16())
            assert_quantized(m, rows)


def test_quantize_beside_ties(m):
    """float32 values one step to each side of every boundary between codes, at small, ordinary and large scales."""
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0])
    near = torch.cat([(ties.view(I32) + d).view(F32) for d in (-2, -1, 0, 1, 2)])
    near = torch.cat([near, -near])
    for e in (-124, -20, 0, 3, 90, 124):
        rows = torch.zeros(len(near), 32)
        rows[:, 0] = 4.0
        rows[:, 17] = near
        assert_quantized(m, (rows * 2.0 ** e).to(DEV))


def test_quantize_small_and_not_finite_blocks(m):
    x = draw(1, 8, 128)
    x[0] *= 2.0 ** -140  # float32 subnormals, under the smallest scale
    x[1] *= 2.0 ** -126
    x[2, 40] = float("nan")
    x[3, 5] = float("inf")
    x[4, 127] = -float("inf")
    x[5] = -0.0
    x[6] = 3.0e38
    for dt in (F32, BF16):
        assert_quantized(m, x.to(dt))
    s = m.quantize_mxfp4(x)[1]
    assert s[2].tolist()[1] == 255 and s[3].tolist()[0] == 255 and s[4].tolist()[3] == 255 and s[5].tolist() == [127] * 4


@pytest.mark.parametrize("dt", [F32, BF16])
def test_quantize_at_odd_addresses(m, dt):
    T, H = 37, 96
    x = draw(2, T, H, dtype=dt)
    want = m.quantize_mxfp4(x)
    for shift in (1, 2, 3, 5):
        xs = torch.empty(T * H + 8, dtype=dt, device=DEV)[shift:shift + T * H].view(T, H)
        xs.copy_(x)
        q = torch.full((T * H // 2 + 8,), 77, dtype=U8, device=DEV)
        s = torch.full((T * H // 32 + 8,), 77, dtype=U8, device=DEV)
        out = (q[shift:shift + T * H // 2].view(T, H // 2), s[shift:shift + T * H // 32].view(T, H // 32))
        m.quantize_mxfp4(xs, out=out)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
        for room, n in ((q, T * H // 2), (s, T * H // 32)):
            assert bool((room[:shift] == 77).all()) and bool((room[shift + n:] == 77).all())


def test_quantize_no_rows_and_a_long_tensor(m):
    q, s = m.quantize_mxfp4(torch.empty(0, 64, device=DEV))
    assert q.shape == (0, 32) and s.shape == (0, 2)
    x = torch.zeros(70000, 65536, dtype=BF16, device=DEV)  # more than 2^32 elements
    x[-1] = draw(3, 65536, dtype=BF16)
    q, s = m.quantize_mxfp4(x)
    want = quantized(x[-1:])
    assert torch.equal(q[-1:], want[0]) and torch.equal(s[-1:], want[1]) and not q[:-1].any()


# ---------------------------------------------------------------- the product


def values(q, s):
    """The values that codes and scales stand for, in 64 bits."""
    table = torch.tensor(VALUES + [-v for v in VALUES], dtype=torch.float64, device=q.device)
    v = torch.stack((table[(q & 15).long()], table[(q >> 4).long()]), -1).view(*s.shape, 32)
    scale = pow2(s.int() - 127)
    return (v * torch.where(s == 255, float("nan"), scale)[..., None]).view(*q.shape[:-1], -1)


def rows4(seed, *shape):
    """Random rows of `shape` and their codes and scales, some blocks far larger or smaller than others."""
    x = draw(seed, *shape)
    x = x.view(-1, shape[-1] // 32, 32) * torch.exp2(2 * draw(seed + 1, x.numel() // shape[-1], shape[-1] // 32))[:, :, None]
    q, s = quantized(x.view(-1, shape[-1]))
    return q.view(*shape[:-1], -1), s.view(*shape[:-1], -1)


def expected(xv, wv, segments, R, gated):
    """(out, bound before the output's rounding, rows written) in 64 bits; xv the rows' values, wv [E, N', H]."""
    E, wrows, H = wv.shape
    N = wrows // 2 if gated else wrows
    out = torch.zeros(R, N, dtype=torch.float64, device=DEV)
    bound, written = torch.zeros_like(out), torch.zeros(R, dtype=torch.bool, device=DEV)
    for e, (a, b) in enumerate(segments):
        if b <= a:
            continue
        y = xv[a:b] @ wv[e].t()
        err = (H + 48) * U * (xv[a:b].abs() @ wv[e].abs().t())
        if gated:
            g, u = y[:, :N], y[:, N:]
            act = g * torch.sigmoid(g)
            # silu' lies in (-0.1, 1.1); exp, sum, quotient and product round: exp's argument to u |g|, its result to 2 u
            out[a:b] = act * u
            bound[a:b] = (1.1 * err[:, :N] + (g.abs().clamp_max(110) + 6) * U * act.abs()) * (u.abs() + err[:, N:]) + act.abs() * err[:, N:]
        else:
            out[a:b], bound[a:b] = y, err
        written[a:b] = True
    return out, bound, written


def check(m, x, w, segments, group_list, out_dtype=BF16, gated=False, src_row=None, **kw):
    xq, xs = x
    R = xq.shape[0] if src_row is None else src_row.shape[0]
    xv = values(xq, xs)
    if src_row is not None:
        ok = (src_row >= 0) & (src_row < xq.shape[0])
        xv = torch.where(ok[:, None], xv[src_row.clamp(0, xq.shape[0] - 1).long()], 0.0)
    want, bound, written = expected(xv, values(*w), segments, R, gated)
    out = torch.full((R, want.shape[1]), 7.0, dtype=out_dtype, device=DEV)
    got = m.grouped_product_mxfp4(xq, xs, w[0], w[1], group_list, src_row=src_row, gated=gated, out=out, **kw)
    assert got is out
    assert bool((out[~written] == 7.0).all()), "rows of no segment were written"
    err = (out.double() - want)[written].abs()
    lim = (bound * (1 + half(out_dtype)) + half(out_dtype) * want.abs())[written] + 1e-37
    nan = torch.isnan(want[written])
    assert torch.equal(torch.isnan(out[written]), nan)
    bad = (err > lim) & ~nan
    assert not bool(bad.any()), f"{int(bad.sum())} values off, worst {float((err / lim)[~nan].max()):.3g} of the bound"
    return out


def standard(lengths):
    ends = torch.tensor(lengths).cumsum(0).tolist()
    return list(zip([0] + ends[:-1], ends)), torch.tensor(ends, dtype=I32, device=DEV)


SIZES = [  # lengths of the segments, H, N
    ([1], 32, 1), ([1], 7168, 48), ([2, 0, 1], 64, 17), ([0, 0, 5], 96, 16), ([16, 17, 1, 0, 33], 160, 33), ([3] * 20, 512, 100),
    ([40, 64, 65], 544, 130), ([127, 128, 129, 1], 1056, 257), ([300, 7, 0, 255], 2080, 1399), ([513], 256, 512), ([1] * 70, 1024, 64),
    ([0, 700, 2], 4096, 300), ([64, 32, 16, 8], 288, 256), ([260, 511], 480, 768),
    # many columns: the largest tiles, all of their heights
    ([300, 7, 0, 255], 96, 22000), ([130, 260, 40, 70, 1], 1056, 14001), ([33, 64, 100, 520], 2080, 17000), ([600], 544, 66000),
    # few rows each of many columns: whole sums, and parts of them
    ([1] * 70, 2080, 2048), ([17, 1, 0, 3], 4128, 96),
]


@pytest.mark.parametrize("lengths,H,N", SIZES)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_dtype", [F32, BF16])
def test_product(m, lengths, H, N, gated, out_dtype):
    print(f"product {lengths} H{H} N{N} gated {gated} {out_dtype}", flush=True)
    R, E = sum(lengths), len(lengths)
    x, w = rows4(R + H, R, H), rows4(N, E, N * (2 if gated else 1), H)
    segments, gl = standard(lengths)
    check(m, x, w, segments, gl, out_dtype, gated)


@pytest.mark.parametrize("lengths,H,N", SIZES[2:])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_through_a_map(m, lengths, H, N, gated):
    """Rows named by a map: some repeated, some outside (rows of zeros), more or fewer than there are rows of x."""
    R, E, rows = sum(lengths), len(lengths), max(1, sum(lengths) // 3)
    x, w = rows4(R, rows, H), rows4(N, E, N * (2 if gated else 1), H)
    src = torch.randint(-2, rows + 2, (R,), generator=torch.Generator().manual_seed(R), dtype=I32).to(DEV)
    src[0] = -(1 << 31)
    src[-1] = (1 << 31) - 1
    segments, gl = standard(lengths)
    check(m, x, w, segments, gl, BF16, gated, src_row=src)


@pytest.mark.parametrize("gated", [False, True])
def test_no_rows_at_all(m, gated):
    w = rows4(1, 3, 64, 64)
    e = torch.empty(0, 32, dtype=U8, device=DEV), torch.empty(0, 2, dtype=U8, device=DEV)
    gl = torch.zeros(3, dtype=I32, device=DEV)
    assert m.grouped_product_mxfp4(*e, *w, gl, gated=gated).shape == (0, 32 if gated else 64)
    # a map onto no rows: rows of zeros
    src = torch.zeros(40, dtype=I32, device=DEV)
    out = m.grouped_product_mxfp4(*e, *w, torch.tensor([2, 2, 40], dtype=I32, device=DEV), src_row=src, gated=gated)
    assert out.shape[0] == 40 and not out.any()
    # segments of no rows: nothing is written
    check(m, rows4(2, 50, 64), w, [], gl, BF16, gated)


@pytest.mark.parametrize("alignment", [16, 128])
def test_aligned_segments(m, alignment):
    T, E, K, H, N = 150, 12, 3, 256, 80
    z = draw(5, T, E) - torch.log(torch.arange(1, E + 1.0, device=DEV))
    idx, w8, ix = m.route_topk_index(z, K, alignment=alignment)
    x, w = rows4(6, T, H), rows4(7, E, N, H)
    ends = ix.group_list.tolist()
    segments = [(a, a + c) for a, c in zip([0] + ends[:-1], ix.counts.tolist())]
    check(m, x, w, segments, ix.group_list, BF16, False, src_row=ix.sorted_indices, counts=ix.counts)
    # without counts the padding rows are products of rows of zeros, and the rows after the last segment are left
    check(m, x, w, list(zip([0] + ends[:-1], ends)), ix.group_list, BF16, False, src_row=ix.sorted_indices)


@pytest.mark.parametrize("capacity", [5, 37, 200])
def test_drop_and_pad_segments(m, capacity):
    T, E, K, H, N = 150, 12, 3, 256, 80
    z = draw(5, T, E) - torch.log(torch.arange(1, E + 1.0, device=DEV))
    idx, w8, ix = m.route_topk_index(z, K, capacity=capacity)
    x, w = rows4(6, T, H), rows4(7, E, 2 * N, H)
    segments = [(e * capacity, e * capacity + c) for e, c in enumerate(ix.kept_counts.tolist())]
    check(m, x, w, segments, None, BF16, True, src_row=ix.sorted_indices, counts=ix.kept_counts, capacity=capacity)


def test_bad_segments_stay_inside(m):
    """Lists that no index holds: what lies in [0, R) and does not overlap is computed, nothing else is touched."""
    H, N, R = 64, 40, 100
    x, w = rows4(8, R, H), rows4(9, 4, N, H)
    for ends in ([50, 20, 90, 200], [-5, 30, 30, 1 << 30], [1 << 30, -(1 << 31), 10, 20], [(1 << 31) - 1] * 4, [-(1 << 31)] * 4):
        guard = torch.full((R + 64, N), 7.0, dtype=BF16, device=DEV)
        out = guard[32:32 + R]
        m.grouped_product_mxfp4(*x, *w, torch.tensor(ends, dtype=I32, device=DEV), out=out)
        torch.cuda.synchronize()
        assert bool((guard[:32] == 7).all()) and bool((guard[32 + R:] == 7).all()), ends
    # as many overlapping experts as there may be, whose tiles together are more than 32 bits count
    E, R2, N2 = 1024, 8192, 1 << 16
    xq, wq = rows4(60, R2, 32), (torch.zeros(E, N2, 16, dtype=U8, device=DEV), torch.full((E, N2, 1), 127, dtype=U8, device=DEV))
    guard = torch.full((R2 + 64, N2), 7.0, dtype=BF16, device=DEV)
    ends = torch.tensor([0, R2], dtype=I32, device=DEV).repeat(E // 2)
    m.grouped_product_mxfp4(*xq, *wq, ends, out=guard[32:32 + R2])
    torch.cuda.synchronize()
    assert bool((guard[:32] == 7).all()) and bool((guard[32 + R2:] == 7).all())
    del wq, guard
    # ends past R, cut
    check(m, x, w, [(0, 0), (0, 30), (30, 30), (30, R)], torch.tensor([-5, 30, 30, 1 << 30], dtype=I32, device=DEV))
    # counts longer than their segments, or negative
    gl = torch.tensor([10, 30, 60, 100], dtype=I32, device=DEV)
    check(m, x, w, [(0, 10), (10, 15), (30, 30), (60, 100)], gl, counts=torch.tensor([99, 5, -3, 40], dtype=I32, device=DEV))
    check(m, x, w, [(0, 25), (25, 25), (50, 51), (75, 100)], None, counts=torch.tensor([99, -1, 1, 25], dtype=I32, device=DEV), capacity=25)


@pytest.mark.parametrize("H,N", [(1056, 150), (1536, 30000), (1056, 30000)])
def test_scales_that_are_nan_stay_with_their_rows(m, H, N):
    lengths, last = [70, 3, 40], H // 32 - 1
    R = sum(lengths)
    x, w = rows4(10, R, H), rows4(11, 3, N, H)
    x[1][5, 0] = x[1][71, last] = 255
    w[1][0, 17, 3] = w[1][2, N - 1, last] = 255
    segments, gl = standard(lengths)
    out = check(m, x, w, segments, gl, F32)
    assert bool(torch.isnan(out[5]).all()) and bool(torch.isnan(out[:70, 17]).all()) and int(torch.isnan(out).sum()) == 2 * N + 69 + 40


def test_scales_at_their_ends(m):
    """2^-127 against 2^127 and products that float32 holds: each is exact."""
    H, N = 128, 20
    x, w = rows4(12, 30, H), rows4(13, 1, N, H)
    for sx, sw in ((0, 254), (254, 0), (0, 200), (200, 10), (127, 127), (3, 250)):
        x[1].fill_(sx)
        w[1].fill_(sw)
        check(m, x, w, [(0, 30)], torch.tensor([30], dtype=I32, device=DEV), F32)


def test_every_pair_of_codes(m):
    """A row for each code against a column for each: all 256 products, in every position of a block's 32."""
    for at in range(32):
        xq, wq = torch.zeros(16, 32, dtype=torch.int64), torch.zeros(16, 32, dtype=torch.int64)
        xq[:, at] = wq[:, at] = torch.arange(16)
        pack = lambda c: (c[:, 0::2] + 16 * c[:, 1::2]).to(U8).to(DEV)  # noqa: E731
        s = torch.full((16, 1), 127, dtype=U8, device=DEV)
        out = check(m, (pack(xq), s), (pack(wq)[None], s[None]), [(0, 16)], torch.tensor([16], dtype=I32, device=DEV), F32)
        v = torch.tensor(VALUES + [-t for t in VALUES], device=DEV)
        assert torch.equal(out, v[:, None] * v[None, :])


@pytest.mark.parametrize("lengths,H,N", [([20, 33], 96, 37), ([30, 300], 512, 9001), ([3, 8], 2560, 100)])
def test_outputs_and_scales_at_odd_addresses(m, lengths, H, N):
    R = sum(lengths)
    x, w = rows4(14, R, H), rows4(15, 2, 2 * N, H)
    segments, gl = standard(lengths)
    for dt in (F32, BF16):
        want = m.grouped_product_mxfp4(*x, *w, gl, gated=True, out_dtype=dt)
        for shift in (1, 2, 3):
            sx = torch.empty(R * H // 32 + 8, dtype=U8, device=DEV)[shift:shift + R * H // 32].view(R, H // 32).copy_(x[1])
            sw = torch.empty(w[1].numel() + 8, dtype=U8, device=DEV)[shift:shift + w[1].numel()].view(w[1].shape).copy_(w[1])
            room = torch.full((R * N + 8,), 7.0, dtype=dt, device=DEV)
            out = room[shift:shift + R * N].view(R, N)
            m.grouped_product_mxfp4(x[0], sx, w[0], sw, gl, gated=True, out=out)
            assert torch.equal(out, want) and bool((room[:shift] == 7).all()) and bool((room[shift + R * N:] == 7).all())


@pytest.mark.parametrize("gated", [False, True])
def test_offsets_beyond_32_bits(m, gated):
    """Weights, rows and outputs each past 2^32 bytes; the far ends are used."""
    E, N, H = 5, 1 << 19, 4096
    w = torch.zeros(E, N, H // 2, dtype=U8, device=DEV), torch.full((E, N, H // 32), 127, dtype=U8, device=DEV)
    tail = rows4(16, N // 8192, H)
    w[0][-1, ::8192], w[1][-1, ::8192] = tail
    rows = (1 << 21) + 100
    x = torch.zeros(rows, H // 2, dtype=U8, device=DEV), torch.full((rows, H // 32), 127, dtype=U8, device=DEV)
    last = rows4(17, 90, H)
    x[0][-90:], x[1][-90:] = last
    src = torch.arange(rows - 90, rows, dtype=I32, device=DEV)
    gl = torch.tensor([0, 0, 0, 40, 90], dtype=I32, device=DEV)
    got = m.grouped_product_mxfp4(*x, *w, gl, src_row=src, gated=gated, out_dtype=F32)
    y = values(*last)[40:] @ values(*tail).t()
    n = got.shape[1]
    if gated:
        k = N // 2 // 8192
        g, u = y[:, :k], y[:, k:]
        y = g * torch.sigmoid(g) * u
    assert not got[:40].any()
    part = got[40:, ::8192].double()
    mag = values(*last)[40:].abs() @ values(*tail).abs().t()
    assert part.shape == y.shape and n == (N // 2 if gated else N)
    if gated:
        assert bool(((part - y).abs() <= 1e-3 * mag.amax(1, keepdim=True) ** 2).all())
    else:
        assert bool(((part - y).abs() <= (H + 48) * U * mag).all())
    del x, w
    R, N = 70000, 65552  # the output alone is past 2^32 elements
    xq, wq = rows4(18, R, 32), rows4(19, 2, N, 32)
    out = m.grouped_product_mxfp4(*xq, *wq, torch.tensor([R - 3, R], dtype=I32, device=DEV))
    for rows_, e in ((slice(R - 6, R - 3), 0), (slice(R - 3, R), 1)):
        want = values(xq[0][rows_], xq[1][rows_]) @ values(wq[0][e], wq[1][e]).t()
        mag = values(xq[0][rows_], xq[1][rows_]).abs() @ values(wq[0][e], wq[1][e]).abs().t()
        assert bool(((out[rows_].double() - want).abs() <= 80 * U * mag + half(BF16) * (want.abs() + 80 * U * mag)).all())


def test_refusals_of_the_binding(m):
    x, w = rows4(20, 8, 64), rows4(21, 2, 6, 64)
    gl = torch.tensor([4, 8], dtype=I32, device=DEV)
    call = lambda x=x[0], xs=x[1], w_=w[0], ws=w[1], gl=gl, **kw: m.grouped_product_mxfp4(x, xs, w_, ws, gl, **kw)  # noqa: E731
    assert call().shape == (8, 6)
    for bad in (dict(xs=x[1][:4]), dict(ws=w[1][:, :4].contiguous()), dict(w_=w[0][:, :, :16].contiguous()), dict(gl=gl[:1]),
                dict(counts=gl[:1]), dict(gl=None), dict(capacity=4), dict(w_=w[0][:, :5].contiguous(), ws=w[1][:, :5].contiguous(), gated=True),
                dict(out=torch.empty(7, 6, dtype=BF16, device=DEV)), dict(x=x[0].t().contiguous().t())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(x=x[0].int()), dict(gl=gl.long()), dict(src_row=gl.long()), dict(out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(m.MoeError):
        call(capacity=5, counts=gl)  # 2 experts of 5 rows, 8 rows
    odd = torch.empty(8 * 32 + 16, dtype=U8, device=DEV)[8:8 + 256].view(8, 32)
    with pytest.raises(m.MoeError):
        call(x=odd)
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(4, 48, device=DEV))
    with pytest.raises(TypeError):
        m.quantize_mxfp4(torch.zeros(4, 64, dtype=torch.float16, device=DEV))
    with pytest.raises(ValueError):
        m.quantize_mxfp4(torch.zeros(4, 64, device=DEV), out=(torch.empty(4, 32, dtype=U8, device=DEV), torch.empty(4, 1, dtype=U8, device=DEV)))


@pytest.mark.parametrize("T", [1, 200])
def test_replayed_from_a_graph_and_on_two_streams(m, T):
    """The whole chain captured, replayed with other inputs and eager work between; then twice at once."""
    E, K, H, I = 16, 4, 512, 96
    w13, w2 = rows4(22, E, 2 * I, H), rows4(23, E, H, I)

    def chain(x, z):
        idx, w, ix = m.route_topk_index(z, K)
        q, s = m.quantize_mxfp4(x)
        h = m.grouped_product_mxfp4(q, s, *w13, ix.group_list, src_row=ix.sorted_indices, gated=True)
        hq, hs = m.quantize_mxfp4(h)
        return m.unpermute_combine(m.grouped_product_mxfp4(hq, hs, *w2, ix.group_list), ix.row_of, w)

    ins = [(draw(30 + i, T, H, dtype=BF16), draw(40 + i, T, E)) for i in range(3)]
    want = [chain(*i) for i in ins]
    sx, sz = ins[0][0].clone(), ins[0][1].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            out = chain(sx, sz)
    torch.cuda.current_stream().wait_stream(s)
    for i in (0, 1, 2, 0):
        sx.copy_(ins[i][0])
        sz.copy_(ins[i][1])
        out.fill_(-1)
        assert torch.equal(chain(*ins[(i + 1) % 3]), want[(i + 1) % 3])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i]), i
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st, i in zip(streams, ins):
        with torch.cuda.stream(st):
            got.append(chain(*i))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    del g


@pytest.mark.parametrize("T,mode", [(1, "map"), (37, "dispatch"), (500, "map"), (500, "capacity"), (130, "aligned")])
def test_routing_loss_and_experts_together(m, T, mode):
    """A layer in 4 bits as it would be used: routing with the index, the balance loss on its slots, rows to 4 bits, dispatched or
    through the map, gate and up, 4 bits again, down, combine; each step against its definition on what it was given."""
    E, K, H, I = 24, 4, 416, 160
    x, z = draw(50, T, H, dtype=BF16), draw(51, T, E)
    w13, w2 = rows4(52, E, 2 * I, H), rows4(53, E, H, I)
    cap, align = (40 if mode == "capacity" else 0), (16 if mode == "aligned" else 0)
    idx, w, ix = m.route_topk_index(z, K, capacity=cap, alignment=align)
    loss, counts, total, tokens = m.balance_loss(z, idx)
    p = torch.softmax(z.double(), 1)
    assert torch.equal(counts, ix.counts) and int(tokens) == T
    want = E * (counts.double() / (T * K) * p.mean(0)).sum()
    assert abs(float(loss) - float(want)) <= 200 * U * float(want)
    q, s = m.quantize_mxfp4(x)
    kept = ix.kept_counts.tolist()
    ends = ix.group_list.tolist()
    starts = [e * cap for e in range(E)] if cap else [0] + ends[:-1]
    segments = [(a, a + n) for a, n in zip(starts, kept)]
    kw = dict(counts=ix.kept_counts, capacity=cap) if cap or align else {}
    gl = None if cap else ix.group_list
    if mode == "dispatch":  # the dispatch moves the codes and the scales as byte rows
        q, s = (m.permute_scatter(t, ix.row_of, ix.rows, src_row=ix.sorted_indices) for t in (q, s))
        h = check(m, (q, s), w13, segments, gl, BF16, True)
    else:
        h = check(m, (q, s), w13, segments, gl, BF16, True, src_row=ix.sorted_indices, **kw)
    h4 = m.quantize_mxfp4(h)
    y = check(m, h4, w2, segments, gl, BF16, False, **kw)
    out = m.unpermute_combine(y, ix.row_of, w)
    r = ix.row_of.long()
    terms = torch.where((r >= 0)[:, :, None], y.double()[r.clamp_min(0)] * w.double()[:, :, None], 0.0)
    bound = (K + 1) * U * terms.abs().sum(1)
    assert bool(((out.double() - terms.sum(1)).abs() <= bound + half(BF16) * (terms.sum(1).abs() + bound)).all())
