"""The router's balance loss, counts and gradient on the GPU against the definition in 64 bits.

Tolerances count roundings of u = 2^-24. The exponent x - top is rounded once, an error of at most u (top - x) in the exponential's
logarithm, on which exp, the sum over at most 1024 experts (16 a lane, then trees), the reciprocal and the product add less than
32; the sum's own terms carry as much again. Sums over tokens are double. So p is right to B = (2 spread + 64) u, spread the
row's largest top - x (past 104 p is 0 in float32)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
I32 = torch.int32
TINY = 1e-37  # float32's subnormals begin here


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import unpermute_combine_amd as mod
    mod.lib()
    return mod


def inputs(seed, T, E, K, scale=1.0, skew=1.0, missing=0.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) * scale - skew * torch.log(torch.arange(1, E + 1.0))
    idx = torch.topk(z, K, dim=1).indices.to(I32)
    if missing:
        idx[torch.rand(T, K, generator=g) < missing] = -1
    return z.to(DEV), idx.to(DEV)


def reference(z, idx, coef, keep):
    """(loss, counts, prob_sum, n, p, B of each row) in 64 bits."""
    T, E = z.shape
    K = idx.shape[1]
    keep = torch.ones(T, dtype=torch.bool, device=z.device) if keep is None else keep.bool()
    p = torch.where(keep[:, None], torch.softmax(z.double(), 1), 0.0)
    p = torch.where((z == -float("inf")).all(1, keepdim=True), 0.0, p)
    spread = torch.where(torch.isfinite(z), z.amax(1, keepdim=True).double() - z.double(), 0.0).amax(1).clamp(0, 110)
    ids = idx[keep].long().flatten()
    ids = ids[(ids >= 0) & (ids < E)]
    counts, n = torch.bincount(ids, minlength=E), int(keep.sum())
    loss = coef * E * (counts.double() / (n * K) * p.sum(0) / n).sum() if n else torch.zeros((), dtype=torch.float64, device=z.device)
    return loss, counts, p.sum(0), n, p, (2 * spread + 64) * U


def assert_within(got, want, bound, what):
    err = (got.double() - want).abs()
    ok = err <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} values off, worst {float((err / bound).max()):.3g} of the bound"


def check_forward(got, want):
    loss, counts, total, n = got
    w_loss, w_counts, w_total, w_n, p, B = want
    assert loss.shape == () and torch.equal(counts.long(), w_counts) and int(tokens_of(n)) == w_n
    bound = (p * B[:, None]).sum(0) + U * w_total + TINY
    assert_within(total, w_total, bound, "prob_sum")
    rel = float((bound / w_total.clamp_min(1e-30)).max()) if bool((w_total > 0).any()) else 0.0
    assert_within(loss, w_loss, (rel + 4 * U) * w_loss.abs() + TINY, "loss")


def tokens_of(n):
    assert n.shape == (1,) and n.dtype == I32
    return n[0]


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 7, 7), (64, 8, 2), (65, 16, 3), (63, 60, 4), (130, 61, 4), (1000, 64, 8), (257, 100, 6),
          (500, 128, 1), (333, 130, 8), (2049, 256, 8), (3000, 255, 32), (700, 260, 5), (401, 384, 8), (515, 513, 2), (290, 1000, 32),
          (1025, 1024, 8), (16384, 256, 8), (20001, 33, 2), (256, 256, 32), (255, 12, 3), (64, 600, 3), (65, 512, 4), (257, 8, 2)]


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("masked", [False, True])
def test_forward(m, T, E, K, masked):
    z, idx = inputs(T + E, T, E, K, missing=0.1)
    keep = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7).to(DEV) if masked else None
    check_forward(m.balance_loss(z, idx, coef=0.01, token_mask=keep), reference(z, idx, 0.01, keep))


def check_backward(m, z, idx, coef, keep, add, d_loss, out=None):
    _, counts, _, n, p, B = reference(z, idx, coef, keep)
    E, K = z.shape[1], idx.shape[1]
    tokens = torch.tensor([n], dtype=I32, device=DEV)
    dl = torch.tensor(d_loss, device=DEV)
    got = m.balance_loss_backward(z, counts.to(I32), tokens, K, d_loss=dl, coef=coef, token_mask=keep, d_logits=add, out=out)
    f = counts.double() / (max(n, 1) * K)
    s = (p * f).sum(1, keepdim=True)
    scale = float(torch.tensor(d_loss)) * float(torch.tensor(coef)) * E / max(n, 1)
    want = scale * p * (f - s)
    # p's relative error in the factor, and through s; four roundings of scale, difference and products
    bound = abs(scale) * p * ((B[:, None] + 4 * U) * (f - s).abs() + B[:, None] * s) + TINY
    if add is not None:
        want = want + add.double()
        bound = bound + U * want.abs()
    assert_within(got, want, bound, "d_logits")
    return got


@pytest.mark.parametrize("T,E,K", SHAPES)
@pytest.mark.parametrize("masked,added", [(False, False), (True, True)])
def test_backward(m, T, E, K, masked, added):
    z, idx = inputs(T + E, T, E, K, missing=0.1)
    keep = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.7).to(DEV) if masked else None
    add = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(DEV) / T if added else None
    got = check_backward(m, z, idx, 0.01, keep, add, 0.75)
    if masked:
        assert torch.equal(got[~keep], add[~keep])


def test_gradient_agrees_with_differences_of_the_loss(m):
    """(loss(z + h v) - loss(z - h v)) / 2h of the kernels' own loss along directions v of -1 and 1 that the gradient leans to.
    The loss is right to B + 4u of at most coef E max f; its third derivative along v, a fourth joint cumulant of f and three
    times v under p, is at most 8 coef E max f."""
    T, E, K, coef = 200, 24, 3, 4.0
    z, idx = inputs(9, T, E, K)
    loss, counts, _, tokens = m.balance_loss(z, idx, coef=coef)
    d = m.balance_loss_backward(z, counts, tokens, K, coef=coef)
    B = float(reference(z, idx, coef, None)[5].max())
    most = coef * E * float(counts.max()) / (T * K)
    for seed in range(3):
        v = torch.sign(d)
        v[torch.rand(T, E, generator=torch.Generator().manual_seed(seed)).to(DEV) < 0.1 * seed] *= -1
        h = 1.0 / 64
        a, b = m.balance_loss(z + h * v, idx, coef=coef)[0], m.balance_loss(z - h * v, idx, coef=coef)[0]
        want = (float(a) - float(b)) / (2 * h)
        got = float((d.double() * v.double()).sum())
        # z +- h v is rounded: u |z| in each logit moves the loss by at most that, too
        bound = most * (8 * h * h / 6 + (B + 4 * U + 2 * float(z.abs().max() + 1) * U) / h)
        assert abs(want) > 4 * bound and abs(got - want) <= bound, (got, want, bound)


def test_masked_tokens_hold_anything(m):
    T, E, K = 300, 96, 4
    z, idx = inputs(3, T, E, K)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[::7] = False
    clean = m.balance_loss(z, idx, token_mask=keep)
    grad = m.balance_loss_backward(z, clean[1], clean[3], K, token_mask=keep)
    for bad in (float("nan"), float("inf"), -float("inf")):
        zb, ib = z.clone(), idx.clone()
        zb[~keep] = bad
        ib[~keep] = 1 << 30
        got = m.balance_loss(zb, ib, token_mask=keep)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))
        assert torch.equal(m.balance_loss_backward(zb, clean[1], clean[3], K, token_mask=keep.to(torch.uint8)), grad)
    assert not grad[~keep].any()


def test_no_token_counts(m):
    z, idx = inputs(4, 70, 40, 2)
    none = torch.zeros(70, dtype=torch.bool, device=DEV)
    add = torch.randn(70, 40, device=DEV)
    loss, counts, total, tokens = m.balance_loss(z, idx, token_mask=none)
    assert float(loss) == 0 and not counts.any() and not total.any() and int(tokens) == 0
    assert torch.equal(m.balance_loss_backward(z, counts, tokens, 2, token_mask=none, d_logits=add), add)
    assert not m.balance_loss_backward(z, counts, tokens, 2).any()  # n = 0 without a mask: no gradient either
    e = torch.empty(0, 40, device=DEV)
    loss, counts, total, tokens = m.balance_loss(e, torch.empty(0, 2, dtype=I32, device=DEV))
    assert float(loss) == 0 and not counts.any() and not total.any() and int(tokens) == 0
    assert m.balance_loss_backward(e, counts, tokens, 2).shape == (0, 40)


@pytest.mark.parametrize("E", [40, 61, 600])
def test_infinite_and_wide_logits(m, E):
    """-inf for experts that a token may not use, a row of nothing else, logits hundreds apart, and a NaN that stays a NaN."""
    T, K = 150, 3
    z, idx = inputs(6, T, E, K, scale=40.0)
    z[3::5, E // 2:] = -float("inf")
    z[11] = -float("inf")
    check_forward(m.balance_loss(z, idx), reference(z, idx, 1.0, None))
    got = check_backward(m, z, idx, 1.0, None, None, 1.0)
    assert not got[11].any()
    z[5, 1] = float("nan")
    loss, counts, total, tokens = m.balance_loss(z, idx)
    assert bool(torch.isnan(loss)) and bool(torch.isnan(total).all())
    got2 = m.balance_loss_backward(z, counts, tokens, K)
    assert bool(torch.isnan(got2[5]).all()) and torch.equal(got2[6:], got[6:]) and torch.equal(got2[:5], got[:5])


def test_ids_outside_and_repeated(m):
    T, E = 500, 16
    z, _ = inputs(8, T, E, 2)
    idx = torch.randint(-3, E + 3, (T, 4), generator=torch.Generator().manual_seed(2), dtype=I32).to(DEV)
    idx[:50] = 7
    check_forward(m.balance_loss(z, idx), reference(z, idx, 1.0, None))


@pytest.mark.parametrize("E", [64, 8])
def test_rows_at_odd_addresses(m, E):
    T, K = 300, 2
    z, idx = inputs(10, T, E, K)
    room = torch.empty(T * E + 3, device=DEV)
    for shift in (1, 2, 3):
        zs = room[shift:shift + T * E].view(T, E)
        zs.copy_(z)
        check_forward(m.balance_loss(zs, idx), reference(z, idx, 1.0, None))
        check_backward(m, zs, idx, 1.0, None, None, 1.0)
        out = torch.empty(T * E + 3, device=DEV)[shift:shift + T * E].view(T, E)
        assert check_backward(m, z, idx, 1.0, None, zs, 1.0, out=out) is out


def test_added_in_place(m):
    T, E, K = 777, 128, 4
    z, idx = inputs(11, T, E, K)
    _, counts, _, tokens = m.balance_loss(z, idx)
    add = torch.randn(T, E, device=DEV)
    want = m.balance_loss_backward(z, counts, tokens, K, d_logits=add)
    got = m.balance_loss_backward(z, counts, tokens, K, d_logits=add, out=add)
    assert got is add and torch.equal(add, want)


def test_very_many_tokens(m):
    """More tokens than the workgroups take in a pass: like rows, whose sums are known."""
    T, E, K = 1 << 20, 32, 2
    z, idx = inputs(12, 1, E, K)
    z, idx = z.expand(T, E).contiguous(), idx.expand(T, K).contiguous()
    loss, counts, total, tokens = m.balance_loss(z, idx)
    p1 = reference(z[:1], idx[:1], 1.0, None)
    assert int(tokens) == T and torch.equal(counts.long(), p1[1] * T)
    assert_within(total, p1[2] * T, (float(p1[5]) + U) * p1[2] * T, "prob_sum")
    assert_within(loss, p1[0], (float(p1[5]) + 4 * U) * p1[0], "loss")


def test_sums_over_ranks(m):
    """Two halves of a batch, their counts, sums and tokens added: the whole batch's gradient, and its loss."""
    T, E, K, coef = 800, 48, 4, 0.1
    z, idx = inputs(13, T, E, K)
    loss, counts, total, tokens = m.balance_loss(z, idx, coef=coef)
    halves = [m.balance_loss(z[a:a + T // 2], idx[a:a + T // 2], coef=coef) for a in (0, T // 2)]
    c, t, n = halves[0][1] + halves[1][1], halves[0][2].double() + halves[1][2].double(), halves[0][3] + halves[1][3]
    assert torch.equal(c, counts) and torch.equal(n, tokens)
    assert_within(coef * E * (c * t).sum() / (float(n) ** 2 * K), loss.double(), 8 * U * loss.abs().double(), "loss")
    whole = m.balance_loss_backward(z, counts, tokens, K, coef=coef)
    for a in (0, T // 2):
        assert torch.equal(m.balance_loss_backward(z[a:a + T // 2], c, n, K, coef=coef), whole[a:a + T // 2])


def test_with_the_routing_gradient(m):
    """As a training step has them: routing, its weights' gradient, and the balance gradient joined in place."""
    T, E, K = 1500, 64, 6
    z, _ = inputs(14, T, E, K)
    idx, w = m.route_topk(z, K)
    ix = m.build_index(idx, w, E)
    loss, counts, _, tokens = m.balance_loss(z, idx, coef=0.01)
    assert torch.equal(counts, ix.counts)  # distinct ids, all tokens: the index's own counts
    dw = torch.randn(T, K, device=DEV)
    d = m.route_topk_backward(idx, w, dw, E)
    routing = d.clone()
    m.balance_loss_backward(z, counts, tokens, K, coef=0.01, d_logits=d, out=d)
    check_backward(m, z, idx, 0.01, None, routing, 1.0)
    assert torch.equal(d, m.balance_loss_backward(z, counts, tokens, K, coef=0.01, d_logits=routing))


def test_replayed_from_a_graph_and_on_two_streams(m):
    T, E, K = 5000, 100, 6
    z, idx = inputs(15, T, E, K)
    z2, idx2 = inputs(16, T, E, K)
    ws = torch.empty(m.balance_workspace_bytes(T, E), dtype=torch.uint8, device=DEV)
    static_z, static_i = z.clone(), idx.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            out = m.balance_loss(static_z, static_i, workspace=ws)
            grad = m.balance_loss_backward(static_z, out[1], out[3], K)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in ((z, idx), (z2, idx2), (z, idx)):
        static_z.copy_(a)
        static_i.copy_(b)
        for t in out:
            t.fill_(-1)
        want = m.balance_loss(a, b)  # eager work between the replays
        dwant = m.balance_loss_backward(a, want[1], want[3], K)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(out, want)) and torch.equal(grad, dwant)
    streams = [torch.cuda.Stream() for _ in range(2)]
    want = [m.balance_loss(z, idx), m.balance_loss(z2, idx2)]
    torch.cuda.synchronize()
    got = []
    for s, a in zip(streams, ((z, idx), (z2, idx2))):
        with torch.cuda.stream(s):
            got.append(m.balance_loss(*a))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    del g


def test_refusals_of_the_binding(m):
    z, idx = inputs(1, 20, 8, 2)
    _, counts, _, tokens = m.balance_loss(z, idx)
    with pytest.raises(TypeError):
        m.balance_loss(z.bfloat16(), idx)
    with pytest.raises(TypeError):
        m.balance_loss(z, idx.long())
    with pytest.raises(ValueError):
        m.balance_loss(z, idx[:10])
    with pytest.raises(ValueError, match="contiguous"):
        m.balance_loss(z.t().contiguous().t(), idx)
    with pytest.raises(TypeError):
        m.balance_loss(z, idx, token_mask=torch.ones(20, device=DEV))
    with pytest.raises(ValueError):
        m.balance_loss(z, idx, token_mask=torch.ones(19, dtype=torch.bool, device=DEV))
    with pytest.raises(m.MoeError):
        m.balance_loss(torch.zeros(4000, 64, device=DEV), torch.zeros(4000, 2, dtype=I32, device=DEV),
                       workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        m.balance_loss_backward(z, counts[:4], tokens, 2)
    with pytest.raises(ValueError):
        m.balance_loss_backward(z, counts, counts, 2)
    with pytest.raises(ValueError):
        m.balance_loss_backward(z, counts, tokens, 2, d_logits=z[:4])
    with pytest.raises(ValueError):
        m.balance_loss_backward(z, counts, tokens, 2, d_loss=z[0])
    with pytest.raises(m.MoeError):
        m.balance_loss_backward(z, counts, tokens, 9)
    with pytest.raises(m.MoeError):
        m.balance_loss(z, idx, coef=float("nan"))
