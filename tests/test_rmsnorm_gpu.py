"""The residual RMS norm on the GPU (rows, FP8 rows, backward) against its definition in 64 bits.

Tolerances count roundings. u = 2^-24 is half a float32 step, `half(dtype)` half a step of an output's
type. A sum over n terms that is split over at least 64 threads has at most n/64 + 16 roundings on any
term's way (each thread's own chain, then trees and short chains over threads and wavefronts)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


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


def reference(x, w, residual, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    s = 1 / torch.sqrt(h.square().mean(1) + eps)
    return h, s, h * s[:, None] * w.double()


def row_bound(H):
    """Relative error of a float32 norm output: the addition, the mean's sum (halved by the root, counted
    whole), and the mean, eps, root, reciprocal and the two products."""
    return (H / 64 + 16 + 8) * U


def assert_within(got, want, bound, what):
    err = (got.double() - want).abs()
    ok = err <= bound + 1e-37
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} values off, worst {float((err / (bound + 1e-37)).max()):.3g} of the bound"


SHAPES = [(1, 1), (1, 7168), (3, 2), (2, 7), (5, 8), (64, 63), (33, 65), (7, 512), (130, 1003), (1024, 513), (3, 4099),
          (64, 4096), (257, 7168), (5, 7176), (9, 8192), (3, 8200), (2, 16384), (2, 20001), (3, 32768), (2, 40000)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("x_dt,s_dt,o_dt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, F32), (F32, BF16, BF16)])
@pytest.mark.parametrize("with_residual", [True, False])
def test_forward(m, T, H, x_dt, s_dt, o_dt, with_residual):
    x, w = draw(1, T, H, dtype=x_dt), draw(2, H) + 1
    r = draw(3, T, H, dtype=s_dt) if with_residual else None
    h, s, n = reference(x, w, r, 1e-6)
    out, total, rstd = m.add_rmsnorm(x, w, residual=r, out_dtype=o_dt, want_rstd=True)
    b = row_bound(H)
    assert out.dtype == o_dt and rstd.dtype == F32
    assert_within(rstd, s, b * s, "rstd")
    assert_within(out, n, (b + half(o_dt)) * n.abs(), "out")
    if r is None:
        assert total is None
    else:
        assert total.dtype == s_dt
        # one float32 addition, then the rounding to the sum's type
        assert_within(total, h, (U + half(s_dt)) * h.abs(), "sum")
        assert torch.equal(total, (x.float() + r.float()).to(s_dt))


def test_weight_types_and_eps(m):
    x = draw(1, 19, 1000, dtype=BF16)
    for eps in (0.0, 1e-6, 1e-2, 3.0):
        for wd in (F32, BF16):
            w = (draw(2, 1000) + 1).to(wd)
            out = m.add_rmsnorm(x, w, eps=eps, out_dtype=F32)[0]
            n = reference(x, w, None, float(torch.tensor(eps, dtype=F32)))[2]
            assert_within(out, n, (row_bound(1000) + U) * n.abs(), f"eps {eps} {wd}")


@pytest.mark.parametrize("H", [7168, 1003])
def test_zero_rows_and_non_finite_rows_stay_apart(m, H):
    x = draw(1, 6, H, dtype=BF16)
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, H - 1] = float("nan")
    w = draw(2, H) + 1
    out, _, rstd = m.add_rmsnorm(x, w, want_rstd=True)
    n = reference(x, w, None, 1e-6)[2]
    for t in (0, 4, 5):
        assert_within(out[t], n[t], (row_bound(H) + half(BF16)) * n[t].abs(), f"row {t}")
    assert not out[1].any() and torch.isfinite(rstd[1])
    assert bool(torch.isnan(out[2, 5])) and not out[2, 6:].any() and float(rstd[2]) == 0
    assert bool(torch.isnan(out[3]).all())


@pytest.mark.parametrize("T,H", [(65, 4096), (9, 1001)])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_in_place(m, T, H, dt):
    x, r, w = draw(1, T, H, dtype=dt), draw(2, T, H, dtype=dt), draw(3, H)
    out, total, _ = m.add_rmsnorm(x, w, residual=r)
    x2, r2 = x.clone(), r.clone()
    a, b, _ = m.add_rmsnorm(x2, w, residual=r2, out=x2, sum_out=r2)
    assert a is x2 and b is r2
    assert torch.equal(x2, out) and torch.equal(r2, total)
    x3 = x.clone()
    a, b, _ = m.add_rmsnorm(x3, w, residual=r, sum_out=x3)
    assert torch.equal(a, out) and torch.equal(x3, total)
    # sum_out without a residual: the rows in the sum's type
    wide = torch.empty(T, H, dtype=F32, device=DEV)
    m.add_rmsnorm(x, w, sum_out=wide)
    assert torch.equal(wide, x.float())


def test_no_rows(m):
    w = draw(1, 256)
    e = torch.empty((0, 256), dtype=BF16, device=DEV)
    out, total, rstd = m.add_rmsnorm(e, w, residual=e, want_rstd=True)
    assert out.shape == total.shape == (0, 256) and rstd.shape == (0,)
    q, sc = m.add_rmsnorm_fp8(e, w)[:2]
    assert q.shape == (0, 256) and sc.shape == (0, 2)
    dx, dw = m.add_rmsnorm_backward(e, e, w, rstd)
    assert dx.shape == (0, 256) and not dw.any()


# ------------------------------------------------------------------ FP8 rows


def e4m3(q):
    return q.view(torch.float8_e4m3fn).double()


def codes_of(m, h, w, rows, sc, block):
    """The codes by the definition: of 448 h w / max |h w| over the block, h the float32 sum, in 64 bits up to one rounding
    to float32; blocks of zeros and those whose scale is under 2^-100 as quantize_fp8 of the float32 rows."""
    T, H = rows.shape
    p = (h.double() * w.double()).view(T, -1, block)
    top = p.abs().amax(2, keepdim=True)
    codes = (p * (448 / top)).float().to(torch.float8_e4m3fn).view(torch.uint8).view(T, H)
    by_ratio = ((rows.view(T, -1, block).abs().amax(2) > 0) & (sc >= 2.0 ** -100)).repeat_interleave(block, 1)
    return torch.where(by_ratio, codes, m.quantize_fp8(rows, block)[0])


@pytest.mark.parametrize("T,H,block", [(1, 128, 128), (64, 4096, 128), (33, 7168, 128), (7, 1024, 1024), (5, 2048, 8),
                                       (4, 1000, 8), (3, 1000, 40), (6, 999, 27), (3, 77, 77), (2, 20480, 128),
                                       (9, 4096, 256), (5, 4096, 512), (5, 4096, 4096), (3, 65, 1), (3, 40960, 64),
                                       (8, 96, 32), (8, 48, 16), (2, 8192, 64)])
@pytest.mark.parametrize("dt,s_dt", [(BF16, BF16), (F32, F32), (BF16, F32)])
def test_fp8(m, T, H, block, dt, s_dt):
    x, r, w = draw(1, T, H, dtype=dt), draw(2, T, H, dtype=s_dt), draw(3, H) + 1
    x[0, : min(block, H)] = 0
    r[0, : min(block, H)] = 0  # a block of zeros: scale 1
    h, s, n = reference(x, w, r, 1e-6)
    q, sc, total, rows, rstd = m.add_rmsnorm_fp8(x, w, residual=r, block=block, want_rows=True, out_dtype=F32, want_rstd=True)
    b = row_bound(H)
    amax = n.view(T, -1, block).abs().amax(2)
    want = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
    assert_within(sc, want, (b + U) * want, "scales")
    assert float(sc[0, 0]) == 1.0
    scale = sc.double().repeat_interleave(block, 1)
    # the code of n / scale: half an E4M3 step of the value (2^-4) or of the subnormals (2^-10), after n's own
    # error and the division's
    d = e4m3(q) * scale
    assert_within(d, n, torch.maximum((2.0 ** -4 + b + 2 * U) * n.abs(), 2.0 ** -10 * scale) + (b + 2 * U) * n.abs(), "codes")
    assert_within(rows, n, b * n.abs(), "rows")
    assert_within(rstd, s, b * s, "rstd")
    assert torch.equal(total, (x.float() + r.float()).to(s_dt))
    # bit for bit the definition's codes, and the scales of the float32 rows
    assert torch.equal(sc, m.quantize_fp8(rows, block)[1])
    assert torch.equal(q, codes_of(m, x.float() + r.float(), w, rows, sc, block))
    # and without the rows, in place, the same
    r2 = r.clone()
    q3, sc3, total3, none, none2 = m.add_rmsnorm_fp8(x, w, residual=r2, block=block, sum_out=r2)
    assert none is None and none2 is None and total3 is r2
    assert torch.equal(q, q3) and torch.equal(sc, sc3) and torch.equal(total, r2)


# ------------------------------------------------------------------ backward


def backward_reference(g, h, w, s, d):
    g, h, w, s = g.double(), h.double(), w.double(), s.double()[:, None]
    a = g * w
    mean = (a * h).mean(1, keepdim=True)
    dx = s * (a - h * s * s * mean)
    H = h.shape[1]
    # roundings: a's product, the fused difference and its product with s (3 of |a|, |h m|), m's own (the sum over the
    # row, the mean, two products)
    hm, habs = (h * s * s * mean).abs(), h.abs() * s * s * (a * h).abs().mean(1, keepdim=True)
    bound = s * (4 * U * (a.abs() + hm) + 6 * U * hm + (H / 64 + 16 + 1) * U * habs)
    if d is not None:
        dx = dx + d.double()
        bound = bound + U * dx.abs()
    return dx, bound, (g * h * s).sum(0), (g * h * s).abs().sum(0)


def dw_roundings(T):
    """At most 512 ranges of rows, each a chain over its rows (cut into at most 64 parts), then a chain over the
    ranges and parts: and two for a term's products."""
    return min(T, T / 64 + 512) + 16


@pytest.mark.parametrize("T,H", SHAPES + [(5000, 64), (2500, 1024), (20000, 40), (1100, 7168)])
@pytest.mark.parametrize("g_dt,h_dt,d_dt", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16), (F32, BF16, F32)])
@pytest.mark.parametrize("with_d", [True, False])
def test_backward(m, T, H, g_dt, h_dt, d_dt, with_d):
    g, h, w = draw(1, T, H, dtype=g_dt), draw(2, T, H, dtype=h_dt), draw(3, H) + 1
    d = draw(4, T, H, dtype=d_dt) if with_d else None
    s = reference(h, w, None, 1e-6)[1].float()
    dx_want, bound, dw_want, dw_abs = backward_reference(g, h, w, s, d)
    dx, dw = m.add_rmsnorm_backward(g, h, w, s, d_sum=d, dx_dtype=d_dt)
    assert dx.dtype == d_dt and dw.dtype == F32
    assert_within(dx, dx_want, bound * (1 + half(d_dt)) + half(d_dt) * dx_want.abs(), "dx")
    assert_within(dw, dw_want, dw_roundings(T) * U * dw_abs, "dweight")
    dx2, none = m.add_rmsnorm_backward(g, h, w, s, d_sum=d, dx_dtype=d_dt, want_dw=False)
    assert none is None and torch.equal(dx, dx2)
    if with_d:
        d2 = d.clone()
        dx3, dw3 = m.add_rmsnorm_backward(g, h, w, s, d_sum=d2, out=(d2, None))
        assert dx3 is d2 and torch.equal(dx, d2) and torch.equal(dw, dw3)


def test_gradients_agree_with_differences_of_the_forward(m):
    """The directional derivative of sum(c * out) along v from the kernel's gradients against a central
    difference of the definition in 64 bits (its error is of the order of the step squared)."""
    T, H, eps, step = 6, 96, 1e-2, 1e-4
    x, r, w, c = draw(1, T, H), draw(2, T, H), draw(3, H) + 1, draw(4, T, H)
    vx, vw = draw(5, T, H).double(), draw(6, H).double()
    _, total, rstd = m.add_rmsnorm(x, w, residual=r, eps=eps, want_rstd=True)
    dx, dw = m.add_rmsnorm_backward(c, total, w, rstd)
    loss = lambda k: float((c.double() * reference(x.double() + k * vx, w.double() + k * vw, r, eps)[2]).sum())  # noqa: E731
    want = (loss(step) - loss(-step)) / (2 * step)
    got = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
    size = float((dx.double() * vx).abs().sum() + (dw.double() * vw).abs().sum())
    # third derivatives are of the order of size * |v|^2 <= 20 * size: step^2 / 6 of that, and float32's error
    assert abs(got - want) <= size * (20 * step ** 2 / 6 + 64 * U)


# ------------------------------------------------------------------ streams, graphs, the run of them together


def test_on_another_stream_and_replayed_from_a_graph(m):
    T, H = 48, 4096
    w = draw(1, H) + 1
    bufs = [draw(k, T, H, dtype=BF16) for k in (2, 3, 4)]
    x, r, g = (b.clone() for b in bufs)
    ws = torch.empty(m.rmsnorm_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)

    def step():
        out, total, rstd = m.add_rmsnorm(x, w, residual=r, want_rstd=True)
        q, sc = m.add_rmsnorm_fp8(x, w, residual=r)[:2]
        dx, dw = m.add_rmsnorm_backward(g, total, w, rstd, d_sum=r, workspace=ws)
        return out, total, rstd, q, sc, dx, dw

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (10, 20, 30):
        for b, k in zip((x, r, g), range(3)):
            b.copy_(draw(seed + k, T, H, dtype=BF16))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))


def test_norm_to_fp8_dispatch_and_back(m):
    """The norm's FP8 rows through the dispatch, and its gradient from the combine's backward: as in a layer."""
    T, H, E, K, block = 96, 1024, 16, 4, 128
    x, r, w = draw(1, T, H, dtype=BF16), draw(2, T, H, dtype=BF16), draw(3, H) + 1
    q, sc, total, rows, rstd = m.add_rmsnorm_fp8(x, w, residual=r, block=block, want_rows=True, want_rstd=True)
    logits = (rows.float() @ draw(4, E, H).t()) * H ** -0.5
    idx, tw, ix = m.route_topk_index(logits.contiguous(), K)
    xq = m.permute_scatter(q, ix.row_of, T * K, src_row=ix.sorted_indices)
    xs = m.permute_scatter(sc, ix.row_of, T * K, src_row=ix.sorted_indices)
    src = ix.sorted_indices.long()
    assert torch.equal(xq, q[src]) and torch.equal(xs, sc[src])
    y = (e4m3(xq) * xs.double().repeat_interleave(block, 1)).to(BF16)
    out = m.unpermute_combine(y, ix.row_of, tw, bias=total)
    n = reference(x, w, r, 1e-6)[2]
    # identity experts: the weights sum to one, so the layer adds the row's own values: E4M3's half step, the rows'
    # bf16 rounding and the output's
    want = total.double() + n
    err = (out.double() - want).abs()
    scale = sc.double().repeat_interleave(block, 1)
    assert bool((err <= torch.maximum(2.0 ** -4 * n.abs(), 2.0 ** -10 * scale) * 1.01 + 2.0 ** -8 * n.abs() * 1.1
                 + 2.0 ** -8 * want.abs() * 1.01).all())
    dout = draw(5, T, H, dtype=BF16)
    dy, dtw = m.unpermute_combine_backward(dout, y, ix.row_of, tw, src_row=ix.sorted_indices)
    dn = m.unpermute_combine(dy, ix.row_of)
    dx, dw = m.add_rmsnorm_backward(dn, total, w, rstd, d_sum=dout)
    want_dx, bound, want_dw, dw_abs = backward_reference(dn, total, w, rstd, dout)
    assert_within(dx, want_dx, bound * 1.01 + half(BF16) * want_dx.abs(), "dx")
    assert_within(dw, want_dw, dw_roundings(T) * U * dw_abs, "dweight")


@pytest.mark.parametrize("block", [8, 128, 40, 640])
def test_fp8_blocks_of_any_size_of_values(m, block):
    """Scales from float32's subnormals to its largest values, and zeros of both signs."""
    T, H = 64, 640
    x = draw(1, T, H)
    x[:, 3::16], x[:, 5::16] = 0.0, -0.0
    size = torch.arange(-148, 128, 276 / H, device=DEV)[:H]
    for w in (torch.exp2(size), torch.exp2(size.flip(0)), torch.full((H,), 2.0 ** -149, device=DEV), torch.full((H,), 1e-44, device=DEV),
              torch.full((H,), 3e38 / 8, device=DEV)):
        w = w.clamp(max=3e38 / 8)  # |x| sqrt(mean x^2) stays under 8: no infinities
        q, sc, _, rows, _ = m.add_rmsnorm_fp8(x, w, block=block, want_rows=True, out_dtype=F32)
        assert bool(torch.isfinite(rows).all())
        assert torch.equal(sc, m.quantize_fp8(rows, block)[1])
        assert torch.equal(q, codes_of(m, x, w, rows, sc, block))


@pytest.mark.parametrize("T,H,block", [(4096, 4096, 128), (2100, 2048, 512), (512, 7168, 7168), (300, 4800, 96)])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_fp8_codes_beside_rounding_boundaries(m, T, H, block, dt):
    """Enough values that hundreds of them lie within float32's roundings of a boundary between two codes."""
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    x, r = torch.randn(T, H, generator=g, device=DEV).to(dt), torch.randn(T, H, generator=g, device=DEV).to(dt)
    w = draw(3, H) + 1
    q, sc, _, rows, _ = m.add_rmsnorm_fp8(x, w, residual=r, block=block, want_rows=True, out_dtype=F32)
    assert torch.equal(q, codes_of(m, x.float() + r.float(), w, rows, sc, block))
    assert int((q != m.quantize_fp8(rows, block)[0]).sum()) < T * H / 1e5


def test_more_rows_than_a_grid_has_workgroups(m):
    T, H = (1 << 20) + 77, 6
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    x, r = torch.randn(T, H, generator=g, device=DEV), torch.randn(T, H, generator=g, device=DEV)
    w = draw(3, H) + 1
    out, total, rstd = m.add_rmsnorm(x, w, residual=r, want_rstd=True)
    h, s, n = reference(x, w, r, 1e-6)
    b = row_bound(H)
    assert_within(out, n, b * n.abs(), "out")
    assert_within(rstd, s, b * s, "rstd")
    dx, dw = m.add_rmsnorm_backward(x, total, w, rstd)
    want, bound, want_dw, mag = backward_reference(x, total, w, rstd, None)
    assert_within(dx, want, bound * (1 + U) + U * want.abs(), "dx")
    assert_within(dw, want_dw, dw_roundings(T) * U * mag, "dweight")
    q, sc = m.add_rmsnorm_fp8(x, w, residual=r, block=6)[:2]
    assert torch.equal(sc, m.quantize_fp8(out, 6)[1]) and torch.equal(q, codes_of(m, total, w, out, sc, 6))


@pytest.mark.parametrize("H,block", [(256, 128), (4096, 512), (640, 40), (256, 256), (999, 999)])
def test_fp8_codes_of_products_below_float32s_normal_range(m, H, block):
    """Elements whose h s is a float32 subnormal, under weights that bring them back: h s has lost bits there, the ratio of
    h w has not."""
    x, w = draw(1, 16, H), draw(2, H)
    small = torch.arange(H, device=DEV) < max(block, H // 2) // (2 if block == H else 1)
    x, w = x * torch.where(small, 1e-25, 1e17), w * torch.where(small, 1e20, 1e-22)
    q, sc, _, rows, _ = m.add_rmsnorm_fp8(x, w, block=block, want_rows=True, out_dtype=F32)
    assert bool((sc >= 2.0 ** -100).all())
    assert torch.equal(sc, m.quantize_fp8(rows, block)[1])
    assert torch.equal(q, codes_of(m, x, w, rows, sc, block))


@pytest.mark.parametrize("T,H", [(4096, 2), (4096, 8), (4096, 64), (2048, 1024), (64, 65536)])
def test_rstd_is_rounded_once(m, T, H):
    """Rows of small integers, whose mean of squares float32 holds: what is left is the reciprocal root's one rounding."""
    x = torch.randint(1, 12, (T, H), generator=torch.Generator().manual_seed(H)).float().to(DEV)
    rstd = m.add_rmsnorm(x, torch.ones(H, device=DEV), eps=0.0, want_rstd=True)[2]
    assert torch.equal(rstd, (1 / x.double().square().mean(1).sqrt()).float())


def test_rstd_of_the_smallest_and_the_largest_rows(m):
    """Means of squares from float32's subnormals to its largest values, zeros and what passes its range."""
    size = torch.tensor([2.0 ** -74, 2.0 ** -70, 2.0 ** -63, 2.0 ** -62, 2.0 ** -30, 1.0, 2.0 ** 40, 2.0 ** 60, 0.0, 2.0 ** 70])
    x = size[:, None].expand(-1, 64).contiguous().to(DEV)
    out, _, rstd = m.add_rmsnorm(x, torch.ones(64, device=DEV), eps=0.0, want_rstd=True)
    assert torch.equal(rstd[:8], 1 / x[:8, 0]) and torch.equal(out[:8], torch.ones_like(out[:8]))
    assert bool(torch.isinf(rstd[8])) and bool(torch.isnan(out[8]).all())
    assert float(rstd[9]) == 0 and not out[9].any()


@pytest.mark.parametrize("H", [1 << 20, (1 << 24) + 3])
def test_long_rows_of_like_values(m, H):
    """Adding like values one after the other rounds the same way each time: a float32 chain of 65536 of them is up to 0.1% off.
    The threads' chains over rows that do not fit in registers are in double, so what is left are their rounding to float32, six
    of the wavefront's tree and four of the wavefronts': 11."""
    c = torch.tensor([0.1, 0.7, 1.3, 3.1], device=DEV)
    x, w = c[:, None].expand(-1, H).contiguous(), torch.full((H,), 1.5, device=DEV)
    out, _, rstd = m.add_rmsnorm(x, w, want_rstd=True)
    s = 1 / torch.sqrt(c.double().square() + 1e-6)
    # the sum, the length as float32, the mean and eps, halved by the root, and the reciprocal root
    assert bool(((rstd.double() - s).abs() <= ((11 + 3) / 2 + 1) * U * s).all())
    # and the two products
    want = (c.double() * s * 1.5)[:, None]
    assert bool(((out.double() - want).abs() <= ((11 + 3) / 2 + 3) * U * want).all())
    g = torch.full_like(x, 0.3)
    dx, _ = m.add_rmsnorm_backward(g, x, w, rstd, want_dw=False)
    a, hd, s = g[:, :1].double() * 1.5, c.double()[:, None], rstd.double()[:, None]
    hm = hd * s * s * (a * hd)
    # a's product, m's (that, the sum, the length, the mean, two products), the fused difference and its product with s
    assert bool(((dx.double() - s * (a - hm)).abs() <= s * (3 * U * a.abs() + (1 + 11 + 4 + 2) * U * hm.abs())).all())


@pytest.mark.parametrize("H", [6, 8])
def test_weight_gradient_of_very_many_like_rows(m, H):
    """No chain of float32 additions is longer than 1024 rows (32768 like ones after the other: up to 0.05% off)."""
    T = 1 << 24
    g, h = torch.linspace(0.3, 1.7, H, device=DEV).expand(T, H).contiguous(), torch.linspace(1.9, 0.4, H, device=DEV).expand(T, H).contiguous()
    dw = m.add_rmsnorm_backward(g, h, torch.ones(H, device=DEV), torch.ones(T, device=DEV))[1]
    want = T * g[0].double() * h[0].double()
    # a term's product, the chain, the sum's rounding
    assert bool(((dw.double() - want).abs() <= (1 + 1024 + 1) * U * want).all())


def test_backward_workspace_of_very_many_rows(m):
    """A range of rows is at most 1024 of them; there are 512 as long as that holds."""
    assert m.rmsnorm_workspace_bytes(512 * 1024, 8) == 512 * 8 * 4
    assert m.rmsnorm_workspace_bytes((1 << 31) - 1, 8) == (1 << 21) * 8 * 4


@pytest.mark.parametrize("H,block", [(8, 8), (9, 9), (8, 0), (9, 0), (520, 520), (1032, 8), (1033, 0)])
def test_more_rows_than_a_grid_has_workgroups_with_rows_in_registers(m, H, block):
    """A workgroup takes several rows one after the other: of one wavefront and of several, with whole and partial vectors, as rows
    and as FP8 with one scale a block or a row, in place too. bf16 rows, looked at in the places that the first, the second and
    the last workgroups have written."""
    T = (1 << 20) + 77
    g = torch.Generator(device=DEV)
    g.manual_seed(H)
    x = torch.randn(T, H, generator=g, device=DEV, dtype=BF16)
    r = torch.randn(T, H, generator=g, device=DEV, dtype=BF16)
    w = draw(3, H) + 1
    at = torch.cat([torch.arange(0, 300), torch.arange((1 << 20) - 200, T)]).to(DEV)
    h, s, n = reference(x[at], w, r[at], 1e-6)
    b = row_bound(H)
    if block:
        q, sc, total, rows, rstd = m.add_rmsnorm_fp8(x, w, residual=r, block=block, want_rows=True, want_rstd=True, out_dtype=F32)
        assert torch.equal(sc[at], m.quantize_fp8(rows[at], block)[1])
        assert torch.equal(q[at], codes_of(m, x[at].float() + r[at].float(), w, rows[at], sc[at], block))
    else:
        rows, total, rstd = m.add_rmsnorm(x, w, residual=r, want_rstd=True, out_dtype=F32)
    assert_within(rows[at], n, b * n.abs(), "out")
    assert_within(rstd[at], s, b * s, "rstd")
    assert torch.equal(total[at], (x[at].float() + r[at].float()).to(BF16))
    del rows
    if not block:
        want = m.add_rmsnorm(x[at], w, residual=r[at])[0]
        m.add_rmsnorm(x, w, residual=r, out=x, sum_out=r)
        assert torch.equal(x[at], want) and torch.equal(r, total)
