"""The few-token MoE layer on the GPU against its definition in 64 bits.

Tolerances count roundings of u = 2^-24 along a term's way, with the sums of magnitudes from the same 64-bit
computation. A wavefront may take a whole row of n elements: float32 products are then a chain of n fused multiply-adds, a
rounding each; bf16 ones n/32 matrix instructions, which may truncate (2u) and round a few times inside, fewer than n in
all. Partial sums, scales and what follows add less than 48."""
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


def say(*args):
    print(*args, flush=True)


def draw(seed, *shape, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


class Layer:
    """Random weights of a layer, as the library takes them and as the values they stand for."""

    def __init__(self, m, H, I, E, kind, seed=1, block=128):
        self.H, self.I, self.E, self.kind = H, I, E, kind
        self.rows = F32 if kind == "f32" else BF16
        self.router = draw(seed, E, H, dtype=self.rows)
        w13, w2 = draw(seed + 1, E, 2 * I, H) * H ** -0.5, draw(seed + 2, E, H, I) * I ** -0.5
        self.scales = {}
        if kind != "fp8":
            self.w13, self.w2 = w13.to(self.rows), w2.to(self.rows)
            self.v13, self.v2 = self.w13.double(), self.w2.double()
            return
        self.w13, s13 = m.quantize_fp8(w13.view(E * 2 * I, H), block)
        self.w2, s2 = m.quantize_fp8(w2.view(E * H, I), block)
        value = lambda q, s: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(block, 1)  # noqa: E731
        self.v13, self.v2 = value(self.w13, s13).view(E, 2 * I, H), value(self.w2, s2).view(E, H, I)
        self.w13, self.w2 = self.w13.view(E, 2 * I, H), self.w2.view(E, H, I)
        self.scales = dict(gate_up_scales=s13.view(E, 2 * I, H // block), down_scales=s2.view(E, H, I // block))

    def routed(self, x, K, groups=None):
        """The routing of the definition: logits in 64 bits, rounded to 32; ties to the lower id."""
        logits = (x.double() @ self.router.double().t()).float()
        if groups:
            gs, M = groups
            best = logits.view(len(x), -1, gs).amax(2)
            keep = torch.sort(best, dim=1, descending=True, stable=True)[1][:, :M]
            ok = torch.zeros_like(best, dtype=torch.bool).scatter_(1, keep, True).repeat_interleave(gs, 1)
            logits = torch.where(ok, logits, torch.full_like(logits, -float("inf")))
        v, i = torch.sort(logits, dim=1, descending=True, stable=True)
        v = v[:, :K].double()
        e = torch.exp(v - v[:, :1])
        return i[:, :K].to(torch.int32), e / e.sum(1, keepdim=True)

    def expected(self, x, idx, w, bias=None):
        """(out, bound before the output's rounding) in 64 bits."""
        T, I = len(x), self.I
        xd = x.double()
        out, bound = torch.zeros(T, self.H, dtype=torch.float64, device=DEV), torch.zeros(T, self.H, dtype=torch.float64, device=DEV)
        n_in, n_out = self.H + 48, self.I + 48 + idx.shape[1]
        for e in sorted(set(idx.flatten().tolist())):
            if not 0 <= e < self.E:
                continue
            t, k = (idx == e).nonzero(as_tuple=True)
            gu = xd[t] @ self.v13[e].t()
            mag = xd[t].abs() @ self.v13[e].abs().t()
            g, up = gu[:, :I], gu[:, I:]
            dg, du = (U * n_in * mag).split(I, 1)
            wt = torch.ones(len(t), 1, dtype=torch.float64, device=DEV) if w is None else w[t, k].double()[:, None]
            s = g * torch.sigmoid(g)
            h = wt * s * up
            # silu's slope is at most 1.1; its own evaluation, the weight and the products: 8 roundings; h kept to 2^-17
            dh = wt.abs() * (1.1 * dg * (up.abs() + du) + s.abs() * du) + (8 * U + 2.0 ** -17) * h.abs()
            out.index_add_(0, t, h @ self.v2[e].t())
            mag = h.abs() @ self.v2[e].abs().t()
            bound.index_add_(0, t, dh @ self.v2[e].abs().t() + U * n_out * mag)
        if bias is not None:
            out = out + bias.double()
            bound = bound + U * out.abs()
        return out, bound


def assert_within(got, want, bound, what="out"):
    half = torch.finfo(got.dtype).eps / 2
    bound = bound * (1 + half) + half * want.abs() + 1e-30
    err = (got.double() - want).abs()
    ok = err <= bound
    assert bool(ok.all()), f"{what}: {int((~ok).sum())} of {ok.numel()} off, worst {float((err / bound).max()):.3g} of the bound"


def assert_weights(w, want):
    """The routing's 1e-6, and half a step of float32's subnormals: weights under 2^-126 are rounded to multiples of
    2^-149, so one of them is off by up to 2^-150 however it is computed (the routing of unscaled logits has such)."""
    assert bool(((w.double() - want).abs() <= 1e-6 * want + 2.0 ** -150).all())


SIZES = [  # T, H, I, E, K
    (1, 64, 64, 1, 1), (1, 512, 1024, 8, 2), (2, 128, 64, 8, 8), (3, 1024, 192, 16, 4), (16, 256, 128, 4, 2),
    (17, 512, 320, 4, 4), (33, 192, 64, 2, 1), (64, 1024, 256, 64, 8), (100, 384, 448, 24, 6), (128, 256, 128, 128, 8),
    (256, 320, 192, 2, 2), (256, 128, 64, 1024, 32), (255, 640, 128, 9, 3), (1, 7168, 128, 256, 8), (5, 64, 2048, 32, 5),
    (49, 448, 704, 5, 2), (65, 4096, 64, 3, 1), (8, 128, 4096, 6, 2)]
RAGGED = [(1, 1, 1, 1, 1), (2, 7, 3, 4, 2), (5, 33, 17, 3, 3), (19, 100, 36, 7, 2), (40, 257, 129, 6, 3), (7, 1003, 35, 5, 4),
          (70, 36, 1001, 2, 1), (130, 65, 50, 30, 7), (3, 520, 72, 8, 2), (12, 2056, 1399, 3, 2), (1, 4, 260, 2, 2)]


@pytest.mark.parametrize("T,H,I,E,K", SIZES + RAGGED)
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_layer(m, T, H, I, E, K, kind):
    if kind == "fp8" and (T, H, I, E, K) in RAGGED:
        pytest.skip("FP8 weights have whole blocks")
    if kind == "fp8":
        H, I = -(-H // 128) * 128, -(-I // 128) * 128
    say(f"layer T={T} H={H} I={I} E={E} K={K} {kind}")
    lay = Layer(m, H, I, E, kind)
    x, bias = draw(7, T, H, dtype=lay.rows), draw(8, T, H, dtype=lay.rows)
    out, idx, w = m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, bias=bias, **lay.scales)
    want_idx, want_w = lay.routed(x, K)
    assert torch.equal(idx, want_idx)
    assert_weights(w, want_w)
    assert out.dtype == lay.rows
    assert_within(out, *lay.expected(x, idx, w, bias))
    # with the routing given: the same experts, the same values; and a float32 output without a bias
    again = m.few_token_experts(x, idx, w, lay.w13, lay.w2, bias=bias, **lay.scales)
    assert torch.equal(out, again)
    wide = m.few_token_experts(x, idx, w, lay.w13, lay.w2, out_dtype=F32, **lay.scales)
    assert_within(wide, *lay.expected(x, idx, w))
    # in place of the bias
    b2 = bias.clone()
    assert m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, bias=b2, out=b2, **lay.scales)[0] is b2
    assert torch.equal(b2, out)


@pytest.mark.parametrize("block", [128, 256, 384, 768])
def test_fp8_blocks(m, block):
    lay = Layer(m, 1536, 768, 6, "fp8", block=block)
    x = draw(3, 21, 1536, dtype=BF16)
    out, idx, w = m.few_token_layer(x, lay.router, lay.w13, lay.w2, 3, **lay.scales)
    assert_within(out, *lay.expected(x, idx, w))


def test_every_fp8_code(m):
    """Each of the 256 codes (without the two NaNs) as a weight, against its value."""
    H = I = 256
    codes = torch.arange(256, dtype=torch.int32)
    codes[127], codes[255] = 0, 0
    q = codes.to(torch.uint8).to(DEV)
    w13 = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device=DEV)
    w13[0, :I, 0] = q  # gate_i = value(i) * x[0] (the up rows give 1 by x[1] = 1)
    w13[0, I:, 1] = 0x38
    w2 = torch.zeros(1, H, I, dtype=torch.uint8, device=DEV)
    w2[0, torch.arange(256), torch.arange(256)] = 0x38
    x = torch.zeros(1, H, dtype=BF16, device=DEV)
    x[0, 0] = x[0, 1] = 1
    one = torch.ones(1, 2 * I, H // 128, device=DEV)
    out = m.few_token_experts(x, torch.zeros(1, 1, dtype=torch.int32, device=DEV), None, w13, w2, gate_up_scales=one,
                              down_scales=torch.ones(1, H, I // 128, device=DEV), out_dtype=F32)
    v = q.view(torch.float8_e4m3fn).double()
    want = v * torch.sigmoid(v)
    # exp and the quotient (8 roundings), h kept to 2^-17
    assert bool(((out[0].double() - want).abs() <= (2.0 ** -17 + 8 * U) * want.abs() + 1e-38).all())
    # the same codes as down weights of h = silu(8) * 1
    w13.zero_()
    w13[0, 0, 0], w13[0, I, 1] = 0x50, 0x38  # 8 and 1
    w2.zero_()
    w2[0, :, 0] = q
    out = m.few_token_experts(x, torch.zeros(1, 1, dtype=torch.int32, device=DEV), None, w13, w2, gate_up_scales=one,
                              down_scales=torch.ones(1, H, I // 128, device=DEV), out_dtype=F32)
    h = torch.tensor(8.0, dtype=torch.float64, device=DEV)
    want = v * (h * torch.sigmoid(h))
    assert bool(((out[0].double() - want).abs() <= (2.0 ** -17 + 8 * U) * want.abs() + 1e-38).all())


@pytest.mark.parametrize("T,K", [(1, 2), (9, 4), (70, 3), (256, 8)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_slots_that_route_nowhere_and_repeats(m, T, K, kind):
    E = 11
    lay = Layer(m, 256, 128, E, kind, seed=4)
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(-2, E + 3, (T, K), generator=g).to(torch.int32)  # out of range on both sides, repeats
    idx[T // 2] = -1  # a token without experts
    if T > 4:
        idx[1], idx[2] = 5, -2147483648
        idx[3], idx[4, 0] = 7, 2147483647
    idx = idx.to(DEV)
    w = torch.rand(T, K, generator=g).to(DEV)
    x = draw(9, T, lay.H, dtype=lay.rows)
    for weights in (w, None):
        out = m.few_token_experts(x, idx, weights, lay.w13, lay.w2, **lay.scales)
        assert_within(out, *lay.expected(x, idx, weights))
        assert not out[T // 2].any()
        for _ in range(3):  # the same bits every time
            assert torch.equal(out, m.few_token_experts(x, idx, weights, lay.w13, lay.w2, **lay.scales))
    bias = draw(10, T, lay.H, dtype=lay.rows)
    none = torch.full_like(idx, -1)
    assert torch.equal(m.few_token_experts(x, none, w, lay.w13, lay.w2, bias=bias, **lay.scales), bias)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_what_is_not_finite_stays_with_its_users(m, kind):
    T, H, I, E = 37, 200, 104, 6
    lay = Layer(m, H, I, E, kind)
    idx = torch.stack([torch.arange(T) % 4, (torch.arange(T) + 1) % 4], 1).to(torch.int32).to(DEV)
    w = torch.rand(T, 2, device=DEV)
    x = draw(3, T, H, dtype=lay.rows)
    clean = m.few_token_experts(x, idx, w, lay.w13, lay.w2)
    lay.w13[4] = float("nan")  # experts 4 and 5 are not in use
    lay.w2[5] = float("inf")
    assert torch.equal(clean, m.few_token_experts(x, idx, w, lay.w13, lay.w2))
    x[6, 3], x[20, H - 1] = float("nan"), float("inf")
    out = m.few_token_experts(x, idx, w, lay.w13, lay.w2)
    keep = [t for t in range(T) if t not in (6, 20)]
    assert torch.equal(out[keep], clean[keep])
    assert bool(torch.isnan(out[6]).all()) and not bool(torch.isfinite(out[20]).any())


@pytest.mark.parametrize("gs,M,K", [(8, 2, 6), (4, 8, 4), (16, 1, 8)])
def test_group_limited_routing(m, gs, M, K):
    lay = Layer(m, 256, 64, 32, "bf16")
    x = draw(3, 50, 256, dtype=BF16)
    out, idx, w = m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, group_size=gs, topk_groups=M)
    want_idx, want_w = lay.routed(x, K, (gs, M))
    assert torch.equal(idx, want_idx)
    assert_weights(w, want_w)
    assert_within(out, *lay.expected(x, idx, w))


def test_router_ties_go_to_the_lower_id(m):
    lay = Layer(m, 96, 32, 16, "f32")
    lay.router[3:7] = lay.router[3].clone()
    lay.router[8:] = 0
    x = draw(3, 60, 96)
    idx = m.few_token_layer(x, lay.router, lay.w13, lay.w2, 9)[1]
    assert torch.equal(idx, lay.routed(x, 9)[0])


def test_operands_at_odd_addresses(m):
    """Contiguous views that begin one element into their storage."""
    T, H, I, E, K = 21, 136, 72, 5, 2
    for kind in ("f32", "bf16"):
        lay = Layer(m, H, I, E, kind)
        x, bias = draw(7, T, H, dtype=lay.rows), draw(8, T, H, dtype=lay.rows)
        off = lambda t: torch.cat([t.new_zeros(1), t.flatten()])[1:].view(t.shape)  # noqa: E731
        want = m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, bias=bias)
        got = m.few_token_layer(off(x), off(lay.router), off(lay.w13), off(lay.w2), K, bias=off(bias))
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refusals_of_the_binding(m):
    lay = Layer(m, 128, 64, 4, "bf16")
    q = Layer(m, 128, 128, 4, "fp8")
    x = draw(1, 3, 128, dtype=BF16)
    call = lambda x=x, r=lay.router, a=lay.w13, b=lay.w2, k=2, **kw: m.few_token_layer(x, r, a, b, k, **kw)  # noqa: E731
    for bad in (dict(x=x[:, :64].contiguous()), dict(r=lay.router[:3]), dict(a=lay.w13[:3]), dict(b=lay.w2.transpose(1, 2).contiguous()),
                dict(a=lay.w13[:, :, ::2]), dict(bias=x[:2]), dict(out=torch.empty(3, 64, dtype=BF16, device=DEV)),
                dict(a=q.w13, b=q.w2, gate_up_scales=q.scales["gate_up_scales"][:, :, :1], down_scales=q.scales["down_scales"][:2]),
                dict(gate_up_scales=q.scales["gate_up_scales"], down_scales=q.scales["down_scales"])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(x=x.float()), dict(r=lay.router.float()), dict(b=lay.w2.float()), dict(a=lay.w13.half(), b=lay.w2.half()),
                dict(a=q.w13, b=q.w2), dict(bias=x.float()), dict(out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(k=0), dict(k=5), dict(x=draw(1, 257, 128, dtype=BF16)), dict(group_size=3, topk_groups=1),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(m.MoeError):
            call(**bad)
    out, idx, w = call(x=x[:0])
    assert out.shape == (0, 128) and idx.shape == w.shape == (0, 2)


@pytest.mark.parametrize("T,kind", [(1, "bf16"), (3, "f32"), (40, "fp8"), (130, "bf16")])
def test_replayed_from_a_graph_and_on_two_streams(m, T, kind):
    H, I, E, K = 512, 256, 32, 4
    lay = Layer(m, H, I, E, kind)
    bias = draw(8, T, H, dtype=lay.rows)
    x = draw(7, T, H, dtype=lay.rows)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty(m.few_token_workspace_bytes(T, H, I, E, K), dtype=torch.uint8, device=DEV) for _ in streams]
    xs = [draw(20 + i, T, H, dtype=lay.rows) for i in range(2)]
    want = [m.few_token_layer(v, lay.router, lay.w13, lay.w2, K, bias=bias, **lay.scales) for v in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):  # both at once, each with its own workspace
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(m.few_token_layer(xs[i], lay.router, lay.w13, lay.w2, K, bias=bias, workspace=ws[i], **lay.scales))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, want[i]))
    with torch.cuda.stream(streams[0]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            out = m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, bias=bias, workspace=ws[0], **lay.scales)
    for seed in range(4):
        x.copy_(draw(30 + seed, T, H, dtype=lay.rows))
        ws[0].fill_(255)  # whatever the workspace held before
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in out]
        eager = m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, bias=bias, **lay.scales)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))


@pytest.mark.parametrize("T", [1, 24, 200])
def test_norm_and_layer_as_a_decode_step(m, T):
    """residual + branch -> norm -> layer onto the residual, against the same through dispatch and combine."""
    H, I, E, K = 512, 192, 16, 4
    lay = Layer(m, H, I, E, "bf16")
    branch, residual, nw = draw(1, T, H, dtype=BF16), draw(2, T, H, dtype=BF16), draw(3, H) * 0.1 + 1
    rows, stream, _ = m.add_rmsnorm(branch, nw, residual=residual)
    out, idx, w = m.few_token_layer(rows, lay.router, lay.w13, lay.w2, K, bias=stream)
    assert_within(out, *lay.expected(rows, idx, w, stream))
    ix = m.build_index(idx, w, E)
    xp = m.permute_scatter(rows, ix.row_of, T * K, src_row=ix.sorted_indices)
    y = torch.empty(T * K, H, dtype=F32, device=DEV)
    ends = ix.group_list.tolist()
    for e in range(E):
        lo, hi = ends[e] - int(ix.counts[e]), ends[e]
        gu = xp[lo:hi].double() @ lay.v13[e].t()
        h = gu[:, :I] * torch.sigmoid(gu[:, :I]) * gu[:, I:]
        y[lo:hi] = (h @ lay.v2[e].t()).float()
    merged = m.unpermute_combine(y, ix.row_of, w, out_dtype=F32)
    want, bound = lay.expected(rows, idx, w, stream)
    # the dispatched way is in 64 bits up to y's rounding and the merge's K
    mag = (w.abs()[:, :, None] * y[ix.row_of.long()].abs()).sum(1).double()
    assert bool(((merged.double() + stream.double() - want).abs() <= (K + 2) * U * mag + U * want.abs()).all())


@pytest.mark.parametrize("T", [1, 20, 150])
@pytest.mark.parametrize("H,I", [(257, 130), (258, 131), (1024, 77), (71, 512), (130, 1026), (9, 9), (6, 200), (200, 6)])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rows_on_odd_elements(m, T, H, I, shift):
    """bf16 rows whose addresses are no multiples of a word, at every offset of the storage."""
    E, K = 5, 3
    lay = Layer(m, H, I, E, "bf16", seed=11)
    off = lambda t: torch.cat([t.new_full((shift,), float("nan")), t.flatten(), t.new_full((3,), float("nan"))])[  # noqa: E731
        shift: shift + t.numel()].view(t.shape)
    x = draw(5, T, H, dtype=BF16)
    idx, w = lay.routed(x, K)
    w = w.float()
    out = m.few_token_experts(off(x), idx, w, off(lay.w13), off(lay.w2), out_dtype=F32)
    assert_within(out, *lay.expected(x, idx, w))


@pytest.mark.parametrize("T,H,I,kind", [(200, 2056, 1032, "f32"), (200, 2056, 1032, "bf16"), (256, 2048, 1024, "fp8"),
                                        (150, 2049, 1027, "bf16"), (131, 2176, 1152, "bf16")])
def test_many_tokens_an_expert(m, T, H, I, kind):
    """Sizes at which experts with more than one or two tiles of tokens take the products through LDS: experts with a
    handful of tokens, some tens, and all of them, side by side."""
    E, K = 32, 8
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    lay = Layer(m, 128, 128, 1, kind)  # replaced below by weights drawn on the GPU
    lay.H, lay.I, lay.E = H, I, E
    w13 = torch.randn(E, 2 * I, H, generator=g, device=DEV) * H ** -0.5
    w2 = torch.randn(E, H, I, generator=g, device=DEV) * I ** -0.5
    if kind == "fp8":
        q13, s13 = m.quantize_fp8(w13.view(E * 2 * I, H))
        q2, s2 = m.quantize_fp8(w2.view(E * H, I))
        lay.w13, lay.w2 = q13.view(E, 2 * I, H), q2.view(E, H, I)
        lay.scales = dict(gate_up_scales=s13.view(E, 2 * I, -1), down_scales=s2.view(E, H, -1))
        value = lambda q, s: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)  # noqa: E731
        lay.v13, lay.v2 = value(q13, s13).view(E, 2 * I, H), value(q2, s2).view(E, H, I)
    else:
        lay.w13, lay.w2 = w13.to(lay.rows), w2.to(lay.rows)
        lay.v13, lay.v2 = lay.w13.double(), lay.w2.double()
    x = torch.randn(T, H, generator=g, device=DEV).to(lay.rows)
    # expert 0 takes every token, experts 1..6 most, the others ever fewer
    p = torch.tensor([1e9] + [8.0] * 6 + [2.0 ** (2 - e / 4) for e in range(E - 7)], device=DEV)
    idx = torch.multinomial(p.expand(T, E), K, generator=g).to(torch.int32)
    w = torch.rand(T, K, generator=g, device=DEV)
    rows = torch.bincount(idx.flatten().long(), minlength=E)
    assert int(rows.max()) == T and int((rows <= 16).sum()) >= 3 and int(((rows > 16) & (rows <= 32)).sum()) >= 2
    out = m.few_token_experts(x, idx, w, lay.w13, lay.w2, out_dtype=F32, **lay.scales)
    assert_within(out, *lay.expected(x, idx, w))
    assert torch.equal(out, m.few_token_experts(x, idx, w, lay.w13, lay.w2, out_dtype=F32, **lay.scales))


@pytest.mark.parametrize("T,E", [(16, 3), (16, 40), (256, 40)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_all_slots_with_one_expert(m, T, E, kind):
    """32 slots a token, all of them one expert's: as many rows of it as a call can have."""
    lay = Layer(m, 256, 128, E, kind, seed=4)
    x, w = draw(9, T, 256, dtype=lay.rows), draw(10, T, 3 if E == 3 else 32).abs()
    idx = torch.full(w.shape, E - 1, dtype=torch.int32, device=DEV)
    out = m.few_token_experts(x, idx, w, lay.w13, lay.w2, out_dtype=F32, **lay.scales)
    assert_within(out, *lay.expected(x, idx, w))


@pytest.mark.parametrize("T,E,K", [(3, 8, 2), (16, 600, 32), (37, 8, 2), (100, 1000, 8)])
@pytest.mark.parametrize("limited", [False, True])
def test_layer_with_rows_that_are_not_finite(m, T, E, K, limited):
    """Their logits are not numbers: they route anywhere or nowhere, and the other rows are as before."""
    groups = (E // 4, 2) if limited else None
    lay = Layer(m, 192, 64, E, "bf16")
    x = draw(3, T, 192, dtype=BF16)
    x[1], x[2, 5] = float("nan"), -float("inf")
    x[1].view(torch.int16)[:] = -1  # a negative NaN
    limit = dict(group_size=groups[0], topk_groups=groups[1]) if limited else {}
    out, idx, w = m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, **limit)
    assert bool(((idx >= -1) & (idx < E)).all())
    keep = [t for t in range(T) if t not in (1, 2)]
    want_idx, want_w = lay.routed(x[keep], K, groups)
    assert torch.equal(idx[keep], want_idx)
    assert_weights(w[keep], want_w)
    assert_within(out[keep], *lay.expected(x[keep], idx[keep], w[keep]))


@pytest.mark.parametrize("T", [2, 40])
@pytest.mark.parametrize("shift", [1, 2, 4, 8])
def test_fp8_codes_at_odd_addresses(m, T, shift):
    lay = Layer(m, 384, 256, 7, "fp8")
    x = draw(5, T, 384, dtype=BF16)
    off = lambda t: torch.cat([t.new_zeros(shift), t.flatten()])[shift:].view(t.shape)  # noqa: E731
    want = m.few_token_layer(x, lay.router, lay.w13, lay.w2, 3, **lay.scales)
    got = m.few_token_layer(off(x), off(lay.router), off(lay.w13), off(lay.w2), 3, gate_up_scales=off(lay.scales["gate_up_scales"]),
                            down_scales=off(lay.scales["down_scales"]))
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("T", [2, 30, 200])
@pytest.mark.parametrize("H,I,block", [(5120, 2304, 256), (2432, 4096, 128), (2176, 8704, 2176)])
def test_fp8_rows_of_many_blocks(m, T, H, I, block):
    """More scales to a row than are read at a time, blocks of one load and of several, starts apart."""
    lay = Layer(m, H, I, 3, "fp8", block=block)
    x = draw(5, T, H, dtype=BF16)
    idx, w = lay.routed(x, 2)
    out = m.few_token_experts(x, idx, w.float(), lay.w13, lay.w2, out_dtype=F32, **lay.scales)
    assert_within(out, *lay.expected(x, idx, w.float()))


@pytest.mark.parametrize("T,K", [(4, 3), (14, 2), (30, 3), (90, 2)])
@pytest.mark.parametrize("kind,H,I,shifts", [("bf16", 2057, 2063, (0, 1)), ("bf16", 2056, 2062, (0, 3)), ("bf16", 2060, 2056, (0, 8)),
                                             ("bf16", 2048, 2112, (2, 5)), ("f32", 2057, 2063, (0, 1)), ("fp8", 2176, 4352, (1, 6))])
def test_long_rows_off_the_cache_lines(m, T, K, kind, H, I, shifts):
    """Enough of them that they go through the window, at several places in their storage, between elements that are not
    numbers."""
    E = 12
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    lay = Layer(m, 128, 128, 1, kind)  # replaced below by weights drawn on the GPU
    lay.H, lay.I, lay.E = H, I, E
    w13 = torch.randn(E, 2 * I, H, generator=g, device=DEV) * H ** -0.5
    w2 = torch.randn(E, H, I, generator=g, device=DEV) * I ** -0.5
    if kind == "fp8":
        q13, s13 = m.quantize_fp8(w13.view(E * 2 * I, H))
        q2, s2 = m.quantize_fp8(w2.view(E * H, I))
        lay.w13, lay.w2 = q13.view(E, 2 * I, H), q2.view(E, H, I)
        lay.scales = dict(gate_up_scales=s13.view(E, 2 * I, -1), down_scales=s2.view(E, H, -1))
        value = lambda q, s: q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)  # noqa: E731
        lay.v13, lay.v2 = value(q13, s13).view(E, 2 * I, H), value(q2, s2).view(E, H, I)
    else:
        lay.w13, lay.w2 = w13.to(lay.rows), w2.to(lay.rows)
        lay.v13, lay.v2 = lay.w13.double(), lay.w2.double()
    x = torch.randn(T, H, generator=g, device=DEV).to(lay.rows)
    idx = torch.rand(T, E, generator=g, device=DEV).topk(K, 1)[1].to(torch.int32)
    w = torch.rand(T, K, generator=g, device=DEV)
    want = lay.expected(x, idx, w)
    for shift in shifts:
        def off(t):
            fill = 255 if t.dtype == torch.uint8 else float("nan")
            return torch.cat([t.new_full((shift,), fill), t.flatten(), t.new_full((9,), fill)])[shift: shift + t.numel()].view(t.shape)
        out = m.few_token_experts(off(x), idx, w, off(lay.w13), off(lay.w2), out_dtype=F32, **lay.scales)
        assert_within(out, *want)


@pytest.mark.parametrize("T", [1, 9, 40, 256])
@pytest.mark.parametrize("E,K", [(1, 8), (3, 8), (1, 32), (3, 32), (4, 5)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "fp8"])
def test_fewer_experts_than_slots_a_token(m, T, E, K, kind):
    """A rank that holds E of the experts a token may choose: most slots name others (-1), some its own, a few the same twice."""
    lay = Layer(m, 384, 128, E, kind, seed=4)
    g = torch.Generator().manual_seed(T + K)
    ids = torch.where(torch.rand(T, K, generator=g) < 0.7, torch.full((T, K), -1), torch.randint(0, E, (T, K), generator=g))
    idx = ids.to(torch.int32).to(DEV)
    w = torch.rand(T, K, generator=g).to(DEV)
    x, bias = draw(9, T, lay.H, dtype=lay.rows), draw(10, T, lay.H, dtype=lay.rows)
    ws = torch.empty(m.few_token_workspace_bytes(T, lay.H, lay.I, E, K), dtype=torch.uint8, device=DEV)
    for i, weights in ((idx, w), (idx, None), (torch.zeros_like(idx), w), (torch.full_like(idx, -1), w)):
        out = m.few_token_experts(x, i, weights, lay.w13, lay.w2, bias=bias, out=torch.empty_like(x), workspace=ws, **lay.scales)
        assert_within(out, *lay.expected(x, i, weights, bias))
    with pytest.raises(m.MoeError):  # the layer's own routing names K different experts
        m.few_token_layer(x, lay.router, lay.w13, lay.w2, K, **lay.scales)
