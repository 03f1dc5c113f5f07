"""The expert operators at the ends of their types' ranges, against float64:
gates so low that exp(gate) is subnormal or zero in fp32 while the result is
a normal number of its type.

Each tolerance is the arithmetic's own bound, derived beside it."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_expert_ffn_b200 as fx  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CODE = {BF: fx.MOE_BF16, HF: fx.MOE_F16, F32: fx.MOE_F32}


def make_layer(E):
    router = torch.zeros(E, 128, dtype=F32, device="cuda")
    return fx.MoeLayer(128, E, 1, 1, fx.LayerWeights(*[None] * 6, router), n_shared=0)


def status_ok(layer):
    code, bits = fx.moe_get_device_status(layer)
    assert code == fx.MOE_OK, hex(bits)


def rounding(dt, want):
    """Half a step of the type at `want`, its subnormals included, plus the
    same of fp32 below its normal numbers (products on the way)."""
    info = torch.finfo(dt)
    return info.eps / 2 * want.abs() + info.smallest_normal * info.eps / 2 + 2.0 ** -147


LOW_GATES = [-1.0, -40.0, -79.5, -80.0, -80.5, -87.0, -87.5, -88.0, -90.0, -91.0, -96.0, -103.0, -104.0, -120.0, -150.0,
             -172.0, -178.0, -184.0, -300.0, 60.0, 88.0, 100.0]


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("pad", [0, 1])   # rows of 16-byte vectors, and element by element
def test_swiglu_low_gates_and_large_factors(dt, pad):
    """silu(-88) is a normal number of bf16 and fp32, and a large up or dh
    brings far lower gates back into the range. The product of dh and up may
    leave the range where the gradient does not."""
    top = {BF: 3e38, HF: 6e4, F32: 3e38}[dt]
    factors = [1.0, -1.5, top, 0.5 * top ** 0.5, -top ** 0.5, 1e-5, top ** -0.5, 0.0]
    cases = [(g, u, d) for g in LOW_GATES for u in factors for d in factors]
    f = 64
    cases += [(0.0, 0.0, 0.0)] * (-len(cases) % f)
    v = torch.tensor(cases, dtype=torch.float64, device="cuda").T.reshape(3, -1, f)
    rows, ld = v.shape[1], f + pad
    buf = torch.zeros(3, rows, ld, dtype=dt, device="cuda")
    buf[:, :, :f] = v.to(dt)
    L, t = make_layer(1), CODE[dt]
    h, dg, du, h2 = (torch.empty(rows, ld, dtype=dt, device="cuda") for _ in range(4))
    g_, u_, d_ = buf[0], buf[1], buf[2]
    fx.moe_swiglu(L, t, g_, ld, u_, ld, None, rows, f, h, ld)
    fx.moe_swiglu_backward(L, t, d_, ld, g_, ld, u_, ld, None, rows, f, dg, ld, du, ld, h2, ld)
    status_ok(L)
    g, u, d = (b[:, :f].double() for b in buf)
    s, c = torch.sigmoid(g), torch.sigmoid(-g)
    slope = s * (1 + g * c)
    # exp: (|g| + 8) 2^-23 (the argument's rounding and the function's few
    # units), at most eight roundings of 2^-24 behind it; below -174 half the
    # exponential's argument leaves fp32's normal numbers too: two units of
    # 2^-149 in each of the two factors exp(g / 2) and one in a product with
    # them. The slope's 1 + g c cancels near its root, so its bound counts
    # both terms.
    rel = (g.abs() + 16) * 2.0 ** -23 + 5 * 2.0 ** -149 / torch.exp(g.clamp(min=-205, max=0) / 2)
    for name, got, want, mag in (("h", h, g * s * u, None), ("h again", h2, g * s * u, None), ("dup", du, d * g * s, None),
                                 ("dgate", dg, d * u * slope, (d * u).abs() * s * (1 + g.abs() * c))):
        got = got[:, :f].double()
        tol = rel * (want.abs() if mag is None else mag) + rounding(dt, want)
        # results at the type's top may round to infinity
        far = want.abs() > torch.finfo(dt).max * (1 - 2.0 ** -7)
        assert not torch.isnan(got).any(), name
        bad = ((got - want).abs() > tol) & ~far
        assert not bad.any(), (name, [(g[i].item(), u[i].item(), d[i].item(), got[i].item(), want[i].item())
                                      for i in map(tuple, bad.nonzero()[:4].tolist())])
        assert (got[far].abs() >= torch.finfo(dt).max * (1 - 2.0 ** -6)).all(), name
    assert torch.equal(h.view(torch.uint8)[:, :f], h2.view(torch.uint8)[:, :f])


@pytest.mark.parametrize("dt", [BF, F32])
def test_swiglu_low_gates_in_place(dt):
    """Rows whose elements are computed one by one, outputs over the inputs."""
    rows, f = 9, 72
    gen = torch.Generator(device="cuda").manual_seed(5)
    g, u, d = (torch.randn(rows, f, generator=gen, device="cuda") * 2 for _ in range(3))
    g[::2, 5] = -88.0
    u[::2, 5] = 1e38
    u[1, 7], d[1, 7] = 3e38, 1e5
    g, u, d = g.to(dt), u.to(dt), d.to(dt)
    L, t = make_layer(1), CODE[dt]
    h, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    fx.moe_swiglu(L, t, g, f, u, f, None, rows, f, h, f)
    fx.moe_swiglu_backward(L, t, d, f, g, f, u, f, None, rows, f, dg, f, du, f)
    gi, ui, di = g.clone(), u.clone(), d.clone()
    fx.moe_swiglu_backward(L, t, di, f, gi, f, ui, f, None, rows, f, gi, f, ui, f, di, f)
    assert torch.equal(gi, dg) and torch.equal(ui, du) and torch.equal(di, h)
    for target in (0, 1):
        gi, ui = g.clone(), u.clone()
        fx.moe_swiglu(L, t, gi, f, ui, f, None, rows, f, (gi, ui)[target], f)
        assert torch.equal((gi, ui)[target], h)
    status_ok(L)


@pytest.mark.parametrize("dt,out_dt", [(BF, BF), (HF, F32), (BF, F32)])
def test_w4_gate_up_low_gates(dt, out_dt):
    """The gate/up form's activation where exp(-gate) is beyond fp32: one
    column of weights, so that both products are exact."""
    gates = [-40.0, -80.5, -87.5, -88.75, -90.0, -91.5, -96.0, -104.0, -130.0, -172.0, -400.0, 90.0]
    ups = [1.0, -3.0, 1e20, -3e38]
    n, k = len(gates) * len(ups), 32
    gate_scale = torch.tensor([abs(g) / 7 for g in gates for _ in ups], dtype=torch.float64)
    up_scale = torch.tensor([abs(u) for _ in gates for u in ups], dtype=torch.float64)
    negative = torch.tensor([g < 0 for g in gates for _ in ups])
    down = torch.tensor([u < 0 for _ in gates for u in ups])

    def weights(scale, code):
        codes = torch.zeros(1, n, 16, dtype=torch.uint8)
        codes[0, :, 0] = code
        return fx.W4Weights(codes.cuda(), scale.to(F32).view(1, n, 1).cuda(), None, fx.MOE_F32, 32)

    gate, up = weights(gate_scale, torch.where(negative, 1, 15)), weights(up_scale, torch.where(down, 7, 9))
    x = torch.zeros(1, k, dtype=dt, device="cuda")
    x[0, 0] = 1
    L = make_layer(1)
    offsets = torch.tensor([0, 1, 1], dtype=torch.int32, device="cuda")
    h = torch.empty(1, n, dtype=out_dt, device="cuda")
    fx.moe_w4_gate_up(L, CODE[dt], x, 1, k, None, gate, up, offsets, 1, n, k, CODE[out_dt], h, n)
    status_ok(L)
    sign = lambda neg: torch.where(neg, -1.0, 1.0).double()  # noqa: E731
    g = (7 * gate_scale.to(F32)).double().cuda() * sign(negative).cuda()    # one fp32 rounding each
    u = up_scale.to(F32).double().cuda() * sign(down).cuda()
    want = g * torch.sigmoid(g) * u
    # as for silu in fp32, and the rounding of g in exp(g): |g| 2^-24 once more
    rel = (2 * g.abs() + 16) * 2.0 ** -23 + 5 * 2.0 ** -149 / torch.exp(g.clamp(min=-205, max=0) / 2)
    tol = rel * want.abs() + rounding(out_dt, want)
    got, far = h[0].double(), want.abs() > torch.finfo(out_dt).max * (1 - 2.0 ** -7)
    bad = ~((got - want).abs() <= tol) & ~far
    assert not bad.any(), [(g[i].item(), u[i].item(), got[i].item(), want[i].item()) for i in bad.nonzero()[:, 0].tolist()]
    assert (got[far].abs() >= torch.finfo(out_dt).max * (1 - 2.0 ** -6)).all()


@pytest.mark.parametrize("scale_dt", [BF, HF, F32])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group,k", [(32, 33), (32, 1), (64, 65), (64, 300), (128, 129), (128, 1024 + 40)])
def test_w4_infinite_last_scale(group, k, zeros, scale_dt):
    """An infinite scale of a row's last columns makes the row infinite, not
    NaN: columns past the row's end have no scale."""
    n, T = 40, 3
    ng, ld = -(-k // group), -(-((k + 1) // 2) // 16) * 16
    codes = torch.full((1, n, ld), 0x99, dtype=torch.uint8, device="cuda")       # 1 above the zero point
    scales = torch.ones(1, n, ng, dtype=scale_dt, device="cuda")
    scales[0, ::2, -1] = float("inf")
    zp = torch.full((1, n, ng), 8, dtype=torch.uint8, device="cuda") if zeros else None
    w = fx.W4Weights(codes, scales, zp, CODE[scale_dt], group)
    ldx = (k + 7) // 8 * 8
    x = torch.full((T, ldx), float("nan"), dtype=BF, device="cuda")
    x[:, :k] = torch.tensor([1.0, -1.0, 2.0], device="cuda")[:, None]
    L = make_layer(1)
    offsets = torch.tensor([0, T, T], dtype=torch.int32, device="cuda")
    y = torch.empty(T, n, dtype=F32, device="cuda")
    fx.moe_w4_matvec(L, fx.MOE_BF16, x, T, ldx, None, w, offsets, T, n, k, fx.MOE_F32, y, n)
    status_ok(L)
    want = x[:, :1].float() * k * torch.ones(1, n, device="cuda")
    want[:, ::2] *= float("inf")
    assert torch.equal(y, want)


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("counts", [(1 << 20, 70), (300_001, 0, 200_000)])
def test_wgrad_of_16_bits_over_many_rows(counts, accumulate, dt):
    """A weight gradient's contraction is its group's rows. Terms of one sign,
    so that every truncation of the accumulator goes the same way: the sum may
    be off by a quarter of half a step of its type before it is rounded."""
    n, k, G = 72, 136, len(counts)
    ends = torch.tensor([0, *counts]).cumsum(0)
    rows = int(ends[-1])
    gen = torch.Generator(device="cuda").manual_seed(rows)
    draw = lambda c, scale: ((torch.rand(rows, c, generator=gen, device="cuda") + 1) * scale).to(dt)  # noqa: E731
    x, dy = draw(k, 0.5), draw(n, 2.0 ** -8)
    L = make_layer(G)
    offsets = torch.cat([ends, ends[-1:]]).to(torch.int32).cuda()
    old = torch.randint(0, 100, (G, n, k), generator=gen, device="cuda").to(dt)
    dw = old.clone()
    fx.moe_grouped_mm_wgrad(L, CODE[dt], dy, n, x, k, offsets, rows, n, k, CODE[dt], dw, k, accumulate)
    status_ok(L)
    half = torch.finfo(dt).eps / 2
    for g, (a, b) in enumerate(zip(ends[:-1].tolist(), ends[1:].tolist())):
        want = torch.zeros(n, k, dtype=torch.float64, device="cuda")
        for i in range(a, b, 1 << 17):
            want += dy[i:min(b, i + (1 << 17))].double().T @ x[i:min(b, i + (1 << 17))].double()
        if accumulate:
            want += old[g].double()
        err = (dw[g].double() - want).abs()
        assert (err <= 1.25 * half * want.abs()).all(), (g, (err / (half * want.abs())).max().item())


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("op", ["mm", "dgrad"])
def test_products_of_16_bits_over_the_longest_contraction(op, dt):
    """65,536 terms of one sign; the bound is the weight gradients'."""
    counts, long, short = (150, 0, 40), 1 << 16, 264
    n, k = (short, long) if op == "mm" else (long, short)
    ends = torch.tensor([0, *counts]).cumsum(0)
    rows, G = int(ends[-1]), len(counts)
    gen = torch.Generator(device="cuda").manual_seed(3)
    draw = lambda *s, scale: ((torch.rand(*s, generator=gen, device="cuda") + 1) * scale).to(dt)  # noqa: E731
    a, w = draw(rows, long, scale=0.5), draw(G, n, k, scale=2.0 ** -8)
    L = make_layer(G)
    offsets = torch.cat([ends, ends[-1:]]).to(torch.int32).cuda()
    y = torch.empty(rows, short, dtype=dt, device="cuda")
    call = fx.moe_grouped_mm if op == "mm" else fx.moe_grouped_mm_dgrad
    call(L, CODE[dt], a, long, w, k, offsets, rows, n, k, CODE[dt], y, short)
    status_ok(L)
    half = torch.finfo(dt).eps / 2
    for g, (s, e) in enumerate(zip(ends[:-1].tolist(), ends[1:].tolist())):
        want = a[s:e].double() @ (w[g].double().T if op == "mm" else w[g].double())
        assert ((y[s:e].double() - want).abs() <= 1.25 * half * want.abs()).all(), g


@pytest.mark.parametrize("dt,out_dt", [(HF, HF), (BF, F32)])
def test_wgrad_group_does_not_depend_on_the_others(dt, out_dt):
    """A group's gradient has the same bits in a launch of its own rows and in
    a longer one: where a sum is cut follows from the group's rows alone."""
    n, k = 136, 264
    gen = torch.Generator(device="cuda").manual_seed(9)
    for counts in ((300, 9000), (3000, 9000), (7001, 513, 20000)):
        ends = [0]
        for c in counts:
            ends.append(ends[-1] + c)
        x = torch.randn(ends[-1], k, generator=gen, device="cuda").to(dt)
        dy = (torch.randn(ends[-1], n, generator=gen, device="cuda") * 0.1).to(dt)
        all_ = torch.empty(len(counts), n, k, dtype=out_dt, device="cuda")
        L = make_layer(len(counts))
        off = torch.tensor(ends + ends[-1:], dtype=torch.int32, device="cuda")
        fx.moe_grouped_mm_wgrad(L, CODE[dt], dy, n, x, k, off, ends[-1], n, k, CODE[out_dt], all_, k)
        one = make_layer(1)
        for g, c in enumerate(counts):
            a, b = ends[g], ends[g + 1]
            alone = torch.empty(1, n, k, dtype=out_dt, device="cuda")
            xs, ds = x[a:b].clone(), dy[a:b].clone()
            fx.moe_grouped_mm_wgrad(one, CODE[dt], ds, n, xs, k, torch.tensor([0, c, c], dtype=torch.int32, device="cuda"),
                                    c, n, k, CODE[out_dt], alone, k)
            assert torch.equal(alone[0].view(torch.uint8), all_[g].view(torch.uint8)), (counts, g)
        status_ok(L)
        status_ok(one)


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_units_of_16_rows(group, zeros, dt):
    """More than 8 rows per group on average: integers bit for bit, for every
    kernel of the wider units, and the gate/up form against its two products."""
    counts, n, k = (16, 40, 1, 15, 0, 33), 104, 552
    G, rows, ng, ld = len(counts), sum(counts), -(-k // group), k // 2 // 16 * 16 + 16
    gen = torch.Generator(device="cuda").manual_seed(group)
    rand = lambda hi, *s: torch.randint(0, hi, s, generator=gen, device="cuda")  # noqa: E731

    def weights():
        codes, sc = rand(256, G, n, ld).to(torch.uint8), 2.0 ** (rand(3, G, n, ng) - 1).float()
        zp = rand(16, G, n, ng).to(torch.uint8) if zeros else None
        q = torch.stack((codes & 15, codes >> 4), -1).view(G, n, -1)[:, :, :k].double()
        wide = lambda v: v.double().repeat_interleave(group, -1)[:, :, :k]  # noqa: E731
        return fx.W4Weights(codes, sc.to(dt), zp, CODE[dt], group), (q - (wide(zp) if zeros else 8.0)) * wide(sc)

    (gate, g64), (up, u64) = weights(), weights()
    x = (rand(5, rows, k) - 2).to(dt)
    ends = torch.tensor([0, *counts]).cumsum(0)
    offsets = torch.cat([ends, ends[-1:]]).to(torch.int32).cuda()
    L = make_layer(G)
    y, h = torch.empty(rows, n, device="cuda"), torch.empty(rows, n, device="cuda")
    fx.moe_w4_matvec(L, CODE[dt], x, rows, k, None, gate, offsets, rows, n, k, fx.MOE_F32, y, n)
    fx.moe_w4_gate_up(L, CODE[dt], x, rows, k, None, gate, up, offsets, rows, n, k, fx.MOE_F32, h, n)
    status_ok(L)
    for g, (a, b) in enumerate(zip(ends[:-1].tolist(), ends[1:].tolist())):
        gv, uv = x[a:b].double() @ g64[g].T, x[a:b].double() @ u64[g].T
        assert torch.equal(y[a:b].double(), gv), g      # halves below 2^20: exact in fp32
        want = gv * torch.sigmoid(gv) * uv
        # exp within (|gate| + 8) 2^-23, six roundings of 2^-24, as silu's bound above
        rel = (gv.abs() + 16) * 2.0 ** -23 + 5 * 2.0 ** -149 / torch.exp(gv.clamp(min=-205, max=0) / 2)
        assert ((h[a:b].double() - want).abs() <= rel * want.abs() + rounding(F32, want)).all(), g
