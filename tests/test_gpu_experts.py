"""The expert operators beside the FP8 layer on the GPU: 16-bit products
grouped by expert with their gradients, SwiGLU with its gradient, and 4-bit
products, each against its definition in float64.

Two kinds of comparison. Integer inputs whose sums stay below 2^24 are exact
in fp32 in any order, so the output has to be the exact sum rounded once to
its type, bit for bit. Random inputs are held to the arithmetic's bound: an
fp32 sum of k products (each exact in fp32) is off by at most
k * 2^-23 * sum |a b| (every addition off by one unit in the last place of a
partial sum, truncation included), and the output's rounding by eps/2 of its
type, relative, plus half its smallest step.

Layouts are unkind on purpose: operands sit in padded rows whose padding is
NaN, rows of no group (before the first and behind the last) hold NaN, and
outputs are larger than asked for, with what lies around them checked to be
left as it was."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_expert_ffn_b200 as fx  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
CODE = {BF: fx.MOE_BF16, HF: fx.MOE_F16, F32: fx.MOE_F32}
SENTINEL = 77.0


def make_layer(E, S, topk=1):
    router = torch.zeros(E, 128, dtype=F32, device="cuda")
    none = [None] * 6
    return fx.MoeLayer(128, E, topk, 1, fx.LayerWeights(*none, router), n_shared=S)


def status_ok(layer):
    code, bits = fx.moe_get_device_status(layer)
    assert code == fx.MOE_OK, hex(bits)


class Groups:
    """Rows of each group with `lead` rows before the first and `tail` behind
    the last; the shared expert's group is empty without one."""

    def __init__(self, counts, S=0, lead=0, tail=0):
        self.E, self.S, self.G = len(counts) - S, S, len(counts)
        ends = lead + np.concatenate([[0], np.cumsum(counts)])
        self.spans = [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]
        off = ends if S else np.concatenate([ends, ends[-1:]])
        self.first, self.last = int(ends[0]), int(ends[-1])
        self.rows = int(ends[-1]) + tail
        self.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        assert len(off) == self.E + 2
        self.layer = make_layer(self.E, S)


def padded(values, ld, dtype):
    """values [..., c] in rows of ld elements whose padding is NaN."""
    buf = torch.full((*values.shape[:-1], ld), float("nan"), dtype=dtype, device="cuda")
    buf[..., :values.shape[-1]] = values.to(dtype)
    return buf


def ints(rng, shape, lim):
    return torch.from_numpy(rng.integers(-lim, lim + 1, size=shape).astype(np.float64)).cuda()


def normal(rng, shape, std=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * std).cuda()


def up8(v, extra=0):
    return (v + 7) // 8 * 8 + extra


def out_buffer(rows, cols, ld, dtype):
    """rows x ld sentinels, with a guard row behind."""
    return torch.full((rows + 1, ld), SENTINEL, dtype=dtype, device="cuda")


def no_group_rows(t, gr):
    """Rows of no group hold NaN."""
    t[:gr.first] = float("nan")
    t[gr.last:] = float("nan")
    return t


def mm_reference(op, gr, x, dy, w):
    """float64 results and the sums of |products| behind each."""
    if op == "mm":
        res = torch.zeros(gr.rows, w.shape[1], dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(res)
        for g, (a, b) in enumerate(gr.spans):
            res[a:b] = x[a:b] @ w[g].T
            mag[a:b] = x[a:b].abs() @ w[g].abs().T
    elif op == "dgrad":
        res = torch.zeros(gr.rows, w.shape[2], dtype=torch.float64, device="cuda")
        mag = torch.zeros_like(res)
        for g, (a, b) in enumerate(gr.spans):
            res[a:b] = dy[a:b] @ w[g]
            mag[a:b] = dy[a:b].abs() @ w[g].abs()
    else:
        res = torch.stack([dy[a:b].T @ x[a:b] for a, b in gr.spans])
        mag = torch.stack([dy[a:b].abs().T @ x[a:b].abs() for a, b in gr.spans])
    return res, mag


def run_mm(op, gr, dt, out_dt, n, k, x, dy, w, extra=8, ldo_extra=3, accumulate=None):
    """Calls the operator on padded operands; returns the results, having
    checked that nothing else was written."""
    ldx, lddy, ldw = up8(k, extra), up8(n, extra), up8(k, extra)
    xb = no_group_rows(padded(x, ldx, dt), gr) if x is not None else None
    db = no_group_rows(padded(dy, lddy, dt), gr) if dy is not None else None
    wb = padded(w, ldw, dt) if w is not None else None
    t, ot = CODE[dt], CODE[out_dt]
    cols = n if op == "mm" else k
    ldo = cols + ldo_extra
    if op == "wgrad":
        out = out_buffer(gr.G * n, cols, ldo, out_dt)
        if accumulate is not None:
            out[:-1].view(gr.G, n, ldo)[:, :, :cols] = accumulate.to(out_dt)
        fx.moe_grouped_mm_wgrad(gr.layer, t, db, lddy, xb, ldx, gr.offsets, gr.rows, n, k, ot, out, ldo,
                                accumulate is not None)
        res = out[:-1].view(gr.G, n, ldo)
        assert (res[:, :, cols:] == SENTINEL).all()
        res = res[:, :, :cols]
    else:
        out = out_buffer(gr.rows, cols, ldo, out_dt)
        if op == "mm":
            fx.moe_grouped_mm(gr.layer, t, xb, ldx, wb, ldw, gr.offsets, gr.rows, n, k, ot, out, ldo)
        else:
            fx.moe_grouped_mm_dgrad(gr.layer, t, db, lddy, wb, ldw, gr.offsets, gr.rows, n, k, ot, out, ldo)
        assert (out[:, cols:] == SENTINEL).all()
        assert (out[:gr.first] == SENTINEL).all() and (out[gr.last:] == SENTINEL).all()
        res = out[:gr.rows, :cols]
    assert (out[-1] == SENTINEL).all()
    status_ok(gr.layer)
    return res


OPS = ("mm", "dgrad", "wgrad")

# (rows per group, shared group, n, k)
MM_SHAPES = [
    ((1,), 0, 1, 1),
    ((5,), 0, 40, 24),
    ((0, 3, 0, 1), 0, 129, 65),
    ((31, 32, 33, 64, 65), 1, 136, 200),
    ((0, 255, 0, 256, 257), 1, 257, 120),
    ((700, 2), 0, 300, 513),
    ((0, 0, 0), 0, 64, 64),
    ((2,) * 40, 1, 512, 256),
    ((1, 0, 90, 63), 0, 1000, 70),
    ((1100, 513, 512), 0, 200, 520),
    ((40, 70, 3), 0, 1030, 1025),
]


@pytest.mark.parametrize("aligned", [False, True])   # output rows of any stride, or of 16-byte pieces
@pytest.mark.parametrize("dt,out_dt", [(BF, BF), (HF, F32), (HF, HF), (BF, F32)])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("shape", MM_SHAPES, ids=str)
def test_mm_exact_integers(shape, op, dt, out_dt, aligned):
    counts, S, n, k = shape
    rng = np.random.default_rng(n * 1000 + k)
    gr = Groups(counts, S, lead=3, tail=5)
    x = ints(rng, (gr.rows, k), 4) if op != "dgrad" else None
    dy = ints(rng, (gr.rows, n), 4) if op != "mm" else None
    w = ints(rng, (gr.G, n, k), 4) if op != "wgrad" else None
    cols = n if op == "mm" else k
    res = run_mm(op, gr, dt, out_dt, n, k, x, dy, w, ldo_extra=up8(cols, 8) - cols if aligned else 3)
    ref, _ = mm_reference(op, gr, x, dy, w)
    if op != "wgrad":
        res, ref = res[gr.first:gr.last], ref[gr.first:gr.last]
    assert torch.equal(res, ref.to(F32).to(out_dt))   # sums below 2^24: exact in fp32


def check_bound(res, ref, mag, terms, out_dt, what):
    tol = terms * 2.0 ** -23 * mag + torch.finfo(out_dt).eps / 2 * ref.abs() + torch.finfo(out_dt).smallest_normal
    err = (res.double() - ref).abs()
    assert torch.isfinite(res).all(), what
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} values beyond the bound, worst {(err / tol).max().item():.2f}x"


@pytest.mark.parametrize("dt,out_dt", [(BF, BF), (HF, F32)])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("counts,S,n,k", [
    ((300, 1, 0, 77, 640), 1, 1536, 1000),
    ((17,) * 20, 0, 250, 2112),
    ((1500, 20), 0, 700, 512),
    ((5000, 130), 0, 264, 5120),
])
def test_mm_random(counts, S, n, k, op, dt, out_dt):
    rng = np.random.default_rng(n + k)
    gr = Groups(counts, S, tail=9)
    x = normal(rng, (gr.rows, k)).to(dt).double() if op != "dgrad" else None
    dy = normal(rng, (gr.rows, n), 0.1).to(dt).double() if op != "mm" else None
    w = normal(rng, (gr.G, n, k), k ** -0.5).to(dt).double() if op != "wgrad" else None
    cols = n if op == "mm" else k
    res = run_mm(op, gr, dt, out_dt, n, k, x, dy, w, ldo_extra=up8(cols) - cols)
    ref, mag = mm_reference(op, gr, x, dy, w)
    if op != "wgrad":
        res, ref, mag = res[:gr.last], ref[:gr.last], mag[:gr.last]
    terms = {"mm": k, "dgrad": n, "wgrad": max(counts)}[op]
    if out_dt == F32:   # sums of 512 products, added with one rounding each
        terms = min(terms, 512 + terms // 512 + 1)
    check_bound(res, ref, mag, terms, out_dt, op)


@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("out_dt", [BF, F32])
def test_wgrad_accumulates(out_dt, aligned):
    rng = np.random.default_rng(5)
    gr = Groups((40, 0, 100), 0, tail=2)
    n, k = 70, 300
    x, dy = ints(rng, (gr.rows, k), 3), ints(rng, (gr.rows, n), 3)
    old = ints(rng, (gr.G, n, k), 100)
    res = run_mm("wgrad", gr, BF, out_dt, n, k, x, dy, None, ldo_extra=8 - k % 8 if aligned else 3, accumulate=old)
    ref, _ = mm_reference("wgrad", gr, x, dy, None)
    assert torch.equal(res, (ref + old).to(F32).to(out_dt))


@pytest.mark.parametrize("op", OPS)
def test_mm_offsets_past_32_bits(op):
    """Weights (or their gradient) of more than 2^31 elements: the last
    groups' addresses do not fit 32 bits."""
    G, n, k = 66, 8192, 4096
    counts = [0] * G
    counts[0], counts[-1] = 3, 5
    gr = Groups(counts, 0)
    rng = np.random.default_rng(8)
    x = ints(rng, (gr.rows, k), 2)
    dy = ints(rng, (gr.rows, n), 2)
    if op == "wgrad":
        out = torch.empty(G, n, k, dtype=BF, device="cuda")
        fx.moe_grouped_mm_wgrad(gr.layer, fx.MOE_BF16, dy.to(BF), n, x.to(BF), k, gr.offsets, gr.rows, n, k,
                                fx.MOE_BF16, out, k)
        ref = dy[3:].T @ x[3:]
        assert torch.equal(out[-1], ref.to(BF))
        assert torch.equal(out[0], (dy[:3].T @ x[:3]).to(BF))
        assert (out[1:-1].view(torch.int16) == 0).all()
    else:
        w = torch.zeros(G, n, k, dtype=BF, device="cuda")
        last = ints(rng, (n, k), 2)
        w[-1] = last.to(BF)
        if op == "mm":
            out = torch.empty(gr.rows, n, dtype=F32, device="cuda")
            fx.moe_grouped_mm(gr.layer, fx.MOE_BF16, x.to(BF), k, w, k, gr.offsets, gr.rows, n, k, fx.MOE_F32, out, n)
            ref = x[3:] @ last.T
        else:
            out = torch.empty(gr.rows, k, dtype=F32, device="cuda")
            fx.moe_grouped_mm_dgrad(gr.layer, fx.MOE_BF16, dy.to(BF), n, w, k, gr.offsets, gr.rows, n, k, fx.MOE_F32,
                                    out, k)
            ref = dy[3:] @ last
        assert torch.equal(out[3:], ref.to(F32)) and (out[:3] == 0).all()
    status_ok(gr.layer)


@pytest.mark.parametrize("op", OPS)
def test_mm_nan_stays_in_its_rows(op):
    """NaN and infinities in one row (or group) do not reach another's output."""
    rng = np.random.default_rng(6)
    gr = Groups((33, 70, 5), 0)
    n, k = 96, 160
    x, dy, w = ints(rng, (gr.rows, k), 2), ints(rng, (gr.rows, n), 2), ints(rng, (gr.G, n, k), 2)
    clean = run_mm(op, gr, BF, F32, n, k, x, dy, w)
    x[40, 3], dy[40, 3] = float("nan"), float("inf")
    res = run_mm(op, gr, BF, F32, n, k, x, dy, w)
    if op == "wgrad":
        assert torch.equal(res[0], clean[0]) and torch.equal(res[2], clean[2])
        assert torch.isnan(res[1]).any()
    else:
        keep = [r for r in range(gr.rows) if r != 40]
        assert torch.equal(res[keep], clean[keep])
        assert not torch.isfinite(res[40]).all()


def test_mm_row_does_not_depend_on_the_batch():
    """A row's output has the same bits alone and inside a large ragged batch."""
    rng = np.random.default_rng(7)
    n, k = 520, 1000
    gr = Groups((300, 7), 0)
    x = normal(rng, (gr.rows, k)).to(BF).double()
    w = normal(rng, (gr.G, n, k), 0.05).to(BF).double()
    res = run_mm("mm", gr, BF, BF, n, k, x, None, w)
    one = Groups((1, 0), 0)
    for r in (0, 131, 299):
        alone = run_mm("mm", one, BF, BF, n, k, x[r:r + 1], None, w)
        assert torch.equal(alone[0].view(torch.int16), res[r].view(torch.int16))
    again = run_mm("mm", gr, BF, BF, n, k, x, None, w)
    assert torch.equal(again.view(torch.int16), res.view(torch.int16))


def test_mm_gradients_against_differences():
    """The product is linear in each operand, so with integers the difference
    of two forward calls is the gradient's prediction exactly."""
    rng = np.random.default_rng(9)
    gr = Groups((20, 0, 45), 0)
    n, k = 88, 130
    x, dy, w = ints(rng, (gr.rows, k), 3), ints(rng, (gr.rows, n), 3), ints(rng, (gr.G, n, k), 3)
    dx_step, dw_step = ints(rng, (gr.rows, k), 1), ints(rng, (gr.G, n, k), 1)
    f = lambda xx, ww: (dy * run_mm("mm", gr, BF, F32, n, k, xx, None, ww).double()).sum()  # noqa: E731
    base = f(x, w)
    dx = run_mm("dgrad", gr, BF, F32, n, k, None, dy, w).double()
    dw = run_mm("wgrad", gr, BF, F32, n, k, x, dy, None).double()
    assert f(x + dx_step, w) - base == (dx * dx_step).sum()
    assert f(x, w + dw_step) - base == (dw * dw_step).sum()


# ------------------------------------------------------------------ SwiGLU

def swiglu_reference(g, u, dh=None):
    g, u = g.double(), u.double()
    s = torch.sigmoid(g)
    if dh is None:
        return g * s * u
    dh = dh.double()
    return dh * u * (s + g * s * torch.sigmoid(-g)), dh * g * s


@pytest.mark.parametrize("dt", [BF, HF, F32])
@pytest.mark.parametrize("counts,S,f,extra", [((1,), 0, 1, 0), ((3, 0, 8), 1, 136, 8), ((700, 33), 0, 1500, 4),
                                              ((64, 5), 0, 77, 3), ((40, 0), 0, 1536, 0)])
def test_swiglu(counts, S, f, extra, dt):
    rng = np.random.default_rng(f)
    gr = Groups(counts, S, lead=2, tail=3)
    ld = f + extra
    g = padded(normal(rng, (gr.rows, f), 4.0), ld, dt)
    u = padded(normal(rng, (gr.rows, f), 1.0), ld, dt)
    d = padded(normal(rng, (gr.rows, f), 0.3), ld, dt)
    edge = [0.0, -0.0, 1e-4, -30.0, -60000.0, 60000.0, 20.0, -17.0]
    g[gr.first, :min(f, 8)] = torch.tensor(edge[:min(f, 8)], dtype=dt, device="cuda")
    h, dg, du, h2 = (out_buffer(gr.rows, f, ld, dt) for _ in range(4))
    t = CODE[dt]
    fx.moe_swiglu(gr.layer, t, g, ld, u, ld, gr.offsets, gr.rows, f, h, ld)
    fx.moe_swiglu_backward(gr.layer, t, d, ld, g, ld, u, ld, gr.offsets, gr.rows, f, dg, ld, du, ld, h2, ld)
    status_ok(gr.layer)
    own = slice(gr.first, gr.last)
    for o in (h, dg, du, h2):
        assert (o[:gr.first] == SENTINEL).all() and (o[gr.last:] == SENTINEL).all() and (o[:, f:] == SENTINEL).all()
    assert torch.equal(h[own].view(torch.uint8), h2[own].view(torch.uint8))
    gv, uv, dv = (v[own, :f] for v in (g, u, d))
    want_h = swiglu_reference(gv, uv)
    want_g, want_u = swiglu_reference(gv, uv, dv)
    # fp32 steps: exp off by 2 ulp, then at most six roundings of 2^-24 on each
    # term; dg's two terms (s and g s (1 - s)) can cancel, so its bound counts
    # their magnitudes
    gd, sg = gv.double(), torch.sigmoid(gv.double())
    terms = dv.double().abs() * uv.double().abs() * (sg + gd.abs() * sg * (1 - sg))
    rel = 12 * 2.0 ** -23
    for got, want, mag in ((h, want_h, want_h.abs()), (du, want_u, want_u.abs()), (dg, want_g, terms)):
        got = got[own, :f].double()
        tol = rel * mag + torch.finfo(dt).eps / 2 * want.abs() + torch.finfo(dt).smallest_normal
        assert torch.isfinite(got).all()
        assert ((got - want).abs() <= tol).all(), ((got - want).abs() / tol).max().item()


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(3)
    rows, f = 6, 40
    L = make_layer(1, 0)
    g, u, d = (normal(rng, (rows, f)).to(F32) for _ in range(3))
    dg, du = torch.empty_like(g), torch.empty_like(g)
    fx.moe_swiglu_backward(L, fx.MOE_F32, d, f, g, f, u, f, None, rows, f, dg, f, du, f)
    e = 1e-5
    num_g = (swiglu_reference(g.double() + e, u) - swiglu_reference(g.double() - e, u)) / (2 * e) * d.double()
    num_u = (swiglu_reference(g, u.double() + e) - swiglu_reference(g, u.double() - e)) / (2 * e) * d.double()
    # central differences: e^2/6 |h'''| (below 1e-10) and 1e-16 / e of rounding; fp32: a few 2^-24
    assert torch.allclose(dg.double(), num_g, rtol=2e-6, atol=1e-6)
    assert torch.allclose(du.double(), num_u, rtol=2e-6, atol=1e-6)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("f", [64, 33])
def test_swiglu_in_place(f, dt):
    rng = np.random.default_rng(4)
    rows = 50
    L = make_layer(1, 0)
    g, u, d = (normal(rng, (rows, f)).to(dt) for _ in range(3))
    t = CODE[dt]
    h, dg, du = torch.empty_like(g), torch.empty_like(g), torch.empty_like(g)
    fx.moe_swiglu(L, t, g, f, u, f, None, rows, f, h, f)
    fx.moe_swiglu_backward(L, t, d, f, g, f, u, f, None, rows, f, dg, f, du, f)
    for target in ("gate", "up"):
        gi, ui = g.clone(), u.clone()
        fx.moe_swiglu(L, t, gi, f, ui, f, None, rows, f, gi if target == "gate" else ui, f)
        assert torch.equal(gi if target == "gate" else ui, h)
    gi, ui, di = g.clone(), u.clone(), d.clone()
    fx.moe_swiglu_backward(L, t, di, f, gi, f, ui, f, None, rows, f, gi, f, ui, f, di, f)
    assert torch.equal(gi, dg) and torch.equal(ui, du) and torch.equal(di, h)


# ------------------------------------------------------------ 4-bit weights

class W4:
    """Random 4-bit weights of G experts; `dense` is their float64 value."""

    def __init__(self, rng, G, n, k, group, zeros, scale_dt, exact):
        ng = -(-k // group)
        ld = -(-((k + 1) // 2) // 16) * 16 + 16
        # whole random bytes: the row padding and an odd k's last half byte are not zero
        self.codes = torch.from_numpy(rng.integers(0, 256, size=(G, n, ld), dtype=np.uint8)).cuda()
        if exact:
            sc = torch.from_numpy(2.0 ** rng.integers(-2, 2, size=(G, n, ng))).cuda()
        else:
            sc = torch.from_numpy(rng.uniform(0.01, 0.05, size=(G, n, ng))).cuda()
        self.scales = sc.to(scale_dt)
        self.zeros = torch.from_numpy(rng.integers(0, 16, size=(G, n, ng), dtype=np.uint8)).cuda() if zeros else None
        q = torch.stack((self.codes & 15, self.codes >> 4), -1).view(G, n, -1)[:, :, :k].double()
        rep = lambda v: v.double().repeat_interleave(group, -1)[:, :, :k]  # noqa: E731
        self.dense = (q - (8.0 if self.zeros is None else rep(self.zeros))) * rep(self.scales)
        self.desc = fx.W4Weights(self.codes, self.scales, self.zeros, CODE[scale_dt], group)


def w4_inputs(rng, gr, T, k, dt, exact, ldx):
    x = ints(rng, (T, k), 3) if exact else normal(rng, (T, k)).to(dt).double()
    perm = torch.from_numpy(rng.integers(0, T, size=gr.rows).astype(np.int32)).cuda()
    return x, padded(x, ldx, dt), perm


# (rows per group, shared, n, k, group, zeros)
W4_SHAPES = [
    ((1,), 0, 1, 1, 32, False),
    ((0, 2, 1), 0, 40, 33, 32, True),
    ((7, 8, 9), 1, 64, 128, 128, False),
    ((15, 16, 17, 0), 0, 130, 300, 64, True),
    ((33, 64), 0, 65, 1500, 128, True),
    ((1, 0, 3), 0, 700, 2112, 32, False),
    ((2,) * 30, 1, 256, 512, 64, False),
    ((5, 20), 0, 96, 1025, 128, False),
]


@pytest.mark.parametrize("dt,out_dt,scale_dt", [(BF, BF, BF), (HF, F32, HF), (BF, F32, F32), (HF, HF, BF)])
@pytest.mark.parametrize("shape", W4_SHAPES, ids=str)
def test_w4_matvec_exact_integers(shape, dt, out_dt, scale_dt):
    counts, S, n, k, group, zeros = shape
    rng = np.random.default_rng(n + 7 * k)
    gr = Groups(counts, S, lead=2, tail=4)
    T = 11
    w = W4(rng, gr.G, n, k, group, zeros, scale_dt, exact=True)
    x, xb, perm = w4_inputs(rng, gr, T, k, dt, True, up8(k, 8))
    perm[:gr.first] = -5   # rows of no group: not looked at
    perm[gr.last:] = 1 << 30
    ldo = n + 5
    y = out_buffer(gr.rows, n, ldo, out_dt)
    fx.moe_w4_matvec(gr.layer, CODE[dt], xb, T, xb.stride(0), perm, w.desc, gr.offsets, gr.rows, n, k, CODE[out_dt],
                     y, ldo)
    status_ok(gr.layer)
    assert (y[:gr.first] == SENTINEL).all() and (y[gr.last:] == SENTINEL).all() and (y[:, n:] == SENTINEL).all()
    # quarters of integers, sums below 2^22: exact in fp32
    for g, (a, b) in enumerate(gr.spans):
        ref = x[perm[a:b].long()] @ w.dense[g].T
        assert torch.equal(y[a:b, :n], ref.to(F32).to(out_dt)), f"group {g}"


@pytest.mark.parametrize("dt,out_dt,scale_dt", [(BF, BF, BF), (HF, F32, F32)])
@pytest.mark.parametrize("counts,n,k,group,zeros", [
    ((1, 0, 4, 21), 200, 1000, 32, True),
    ((3, 70), 96, 1536, 64, False),
    ((1,) * 9, 320, 2048, 128, True),
])
def test_w4_random(counts, n, k, group, zeros, dt, out_dt, scale_dt):
    rng = np.random.default_rng(k)
    gr = Groups(counts, 0, tail=1)
    T = 9
    gate, up = (W4(rng, gr.G, n, k, group, zeros, scale_dt, exact=False) for _ in range(2))
    x, xb, perm = w4_inputs(rng, gr, T, k, dt, False, up8(k))
    y, h = out_buffer(gr.rows, n, n, out_dt), out_buffer(gr.rows, n, n, out_dt)
    a = (CODE[dt], xb, T, xb.stride(0), perm)
    fx.moe_w4_matvec(gr.layer, *a, gate.desc, gr.offsets, gr.rows, n, k, CODE[out_dt], y, n)
    fx.moe_w4_gate_up(gr.layer, *a, gate.desc, up.desc, gr.offsets, gr.rows, n, k, CODE[out_dt], h, n)
    status_ok(gr.layer)
    for g, (s, e) in enumerate(gr.spans):
        if s == e:
            continue
        xr = x[perm[s:e].long()]
        ref, mag = xr @ gate.dense[g].T, xr.abs() @ gate.dense[g].abs().T
        check_bound(y[s:e], ref, mag, k, out_dt, "matvec")
        ru, mu = xr @ up.dense[g].T, xr.abs() @ up.dense[g].abs().T
        sg = torch.sigmoid(ref)
        want = ref * sg * ru
        # each product's bound times the other factor's slope (|silu'| <= 1.1), and eight fp32 roundings
        e1 = k * 2.0 ** -23
        tol = e1 * (1.1 * mag * ru.abs() + mu * (ref * sg).abs() + 1.1 * mag * mu * e1) + 16 * 2.0 ** -24 * want.abs()
        tol = tol + torch.finfo(out_dt).eps / 2 * want.abs() + torch.finfo(out_dt).smallest_normal
        err = (h[s:e].double() - want).abs()
        assert (err <= tol).all(), (err / tol).max().item()


def test_w4_without_perm_and_single_token():
    rng = np.random.default_rng(2)
    gr = Groups((1, 0, 1), 0)
    n, k = 384, 640
    w = W4(rng, gr.G, n, k, 128, False, BF, exact=True)
    x, xb, _ = w4_inputs(rng, gr, 2, k, BF, True, k)
    y = torch.empty(2, n, dtype=F32, device="cuda")
    fx.moe_w4_matvec(gr.layer, fx.MOE_BF16, xb, 2, k, None, w.desc, gr.offsets, 2, n, k, fx.MOE_F32, y, n)
    assert torch.equal(y, torch.stack([w.dense[0] @ x[0], w.dense[2] @ x[1]]).to(F32))


def test_w4_bad_row_reads_zero_and_is_flagged():
    rng = np.random.default_rng(12)
    gr = Groups((4, 3), 0)
    n, k, T = 64, 256, 3
    w = W4(rng, gr.G, n, k, 64, False, BF, exact=True)
    x, xb, perm = w4_inputs(rng, gr, T, k, BF, True, k)
    perm[1], perm[5] = -1, T
    y = torch.empty(gr.rows, n, dtype=F32, device="cuda")
    fx.moe_w4_matvec(gr.layer, fx.MOE_BF16, xb, T, k, perm, w.desc, gr.offsets, gr.rows, n, k, fx.MOE_F32, y, n)
    code, bits = fx.moe_get_device_status(gr.layer)
    assert code == fx.MOE_ERR_DEVICE and bits == fx.MOE_STATUS_BAD_ROW
    xr = x[perm.clamp(0, T - 1).long()]
    xr[1], xr[5] = 0, 0
    for g, (a, b) in enumerate(gr.spans):
        assert torch.equal(y[a:b], (xr[a:b] @ w.dense[g].T).to(F32))


def test_w4_nan_stays_in_its_row():
    rng = np.random.default_rng(13)
    gr = Groups((5, 12), 0)
    n, k, T = 100, 300, 17
    w = W4(rng, gr.G, n, k, 32, True, BF, exact=True)
    x, xb, _ = w4_inputs(rng, gr, T, k, BF, True, up8(k))
    xb[6, 299] = float("nan")
    y = torch.empty(gr.rows, n, dtype=F32, device="cuda")
    fx.moe_w4_matvec(gr.layer, fx.MOE_BF16, xb, T, xb.stride(0), None, w.desc, gr.offsets, gr.rows, n, k, fx.MOE_F32,
                     y, n)
    for g, (a, b) in enumerate(gr.spans):
        for r in range(a, b):
            if r == 6:
                assert torch.isnan(y[r]).all()
            else:
                assert torch.equal(y[r], (w.dense[g] @ x[r]).to(F32))


# ------------------------------------------- plans, streams, graphs, failures

def all_calls(gr, n, k, rng):
    """Every operator on one set of groups: name -> (call taking outputs, output shapes)."""
    x, dy, w = normal(rng, (gr.rows, k)).to(BF), normal(rng, (gr.rows, n)).to(BF), normal(rng, (gr.G, n, k), 0.1).to(BF)
    q, q2 = (W4(rng, gr.G, n, k, 64, False, BF, exact=False) for _ in range(2))
    L, off, R, B = gr.layer, gr.offsets, gr.rows, fx.MOE_BF16
    calls = {
        "mm": (lambda o, s=None: fx.moe_grouped_mm(L, B, x, k, w, k, off, R, n, k, B, o[0], n, stream=s), [(R, n)]),
        "dgrad": (lambda o, s=None: fx.moe_grouped_mm_dgrad(L, B, dy, n, w, k, off, R, n, k, B, o[0], k, stream=s),
                  [(R, k)]),
        "wgrad": (lambda o, s=None: fx.moe_grouped_mm_wgrad(L, B, dy, n, x, k, off, R, n, k, B, o[0], k, stream=s),
                  [(gr.G, n, k)]),
        "swiglu": (lambda o, s=None: fx.moe_swiglu(L, B, dy, n, dy, n, off, R, n, o[0], n, stream=s), [(R, n)]),
        "swiglu_backward": (lambda o, s=None: fx.moe_swiglu_backward(L, B, dy, n, dy, n, dy, n, off, R, n, o[0], n,
                                                                     o[1], n, stream=s), [(R, n), (R, n)]),
        "w4_matvec": (lambda o, s=None: fx.moe_w4_matvec(L, B, x, R, k, None, q.desc, off, R, n, k, B, o[0], n,
                                                         stream=s), [(R, n)]),
        "w4_gate_up": (lambda o, s=None: fx.moe_w4_gate_up(L, B, x, R, k, None, q.desc, q2.desc, off, R, n, k, B,
                                                           o[0], n, stream=s), [(R, n)]),
    }
    keep = (x, dy, w, q, q2)
    return calls, keep


def outputs(shapes):
    return [torch.full(s, SENTINEL, dtype=BF, device="cuda") for s in shapes]


NAMES = ("mm", "dgrad", "wgrad", "swiglu", "swiglu_backward", "w4_matvec", "w4_gate_up")


@pytest.mark.parametrize("name", NAMES)
def test_bad_plans_do_no_work(name):
    gr = Groups((20, 30, 10), 0)
    good = gr.offsets.clone()
    calls, keep = all_calls(gr, 128, 192, np.random.default_rng(1))
    call, shapes = calls[name]
    for where, value in ((1, 25), (1, 61), (0, -1), (4, 70), (3, 59)):
        bad = good.clone()
        bad[where] = value
        if (where, value) == (1, 25):
            bad[2] = 24               # decreasing
        gr.offsets.copy_(bad)
        out = outputs(shapes)
        call(out)
        code, bits = fx.moe_get_device_status(gr.layer)
        assert code == fx.MOE_ERR_DEVICE and bits == fx.MOE_STATUS_BAD_PLAN, (where, value)
        assert all((o == SENTINEL).all() for o in out), (where, value)
    gr.offsets.copy_(good)
    call(outputs(shapes))
    status_ok(gr.layer)


@pytest.mark.parametrize("name", NAMES)
def test_streams_and_graphs(name):
    """The same bits eagerly, on two streams at once, and replayed from two
    captured graphs after the inputs' groups changed."""
    gr = Groups((100, 0, 300, 7), 0)
    calls, keep = all_calls(gr, 256, 320, np.random.default_rng(2))
    call, shapes = calls[name]
    base = outputs(shapes)
    call(base)
    status_ok(gr.layer)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    oa, ob = outputs(shapes), outputs(shapes)
    torch.cuda.synchronize()
    for _ in range(5):
        call(oa, a)
        call(ob, b)
    torch.cuda.synchronize()
    graphs, outs = [], [outputs(shapes), outputs(shapes)]
    torch.cuda.synchronize()
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(o)
        graphs.append(graph)
    for graph, s in zip(graphs, (a, b)):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for o in (oa, ob, *outs):
        for got, want in zip(o, base):
            assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    gr.offsets.copy_(torch.tensor([0, 50, 50, 51, 407, 407], dtype=torch.int32))
    fresh = outputs(shapes)
    call(fresh)
    for o in outs[0]:
        o.fill_(SENTINEL)
    graphs[0].replay()
    torch.cuda.synchronize()
    for got, want in zip(outs[0], fresh):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("name", [n for n in NAMES if not n.startswith("swiglu")])
def test_timed_out_wait_is_reported_and_the_handle_recovers(name):
    """A copy that never arrives (its issue withheld by the test hook): the
    waits give up after a millisecond, the status says so, and the next call
    on the handle is whole."""
    gr = Groups((100, 300, 7), 0)
    calls, keep = all_calls(gr, 512, 640, np.random.default_rng(3))
    call, shapes = calls[name]
    base = outputs(shapes)
    call(base)
    status_ok(gr.layer)
    fx.moe_test_inject_stall(gr.layer, 1_000_000)
    call(outputs(shapes))
    code, bits = fx.moe_get_device_status(gr.layer)
    assert code == fx.MOE_ERR_DEVICE and bits == fx.MOE_STATUS_WAIT_TIMEOUT
    out = outputs(shapes)
    call(out)
    status_ok(gr.layer)
    for got, want in zip(out, base):
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_calls_go_to_the_current_stream():
    """Without a stream argument a call is ordered on torch's current stream,
    whichever that is."""
    rng = np.random.default_rng(11)
    L = make_layer(1, 0)
    rows, f = 4096, 2048
    u = normal(rng, (rows, f)).to(F32)
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side, torch.cuda.default_stream()):
        assert fx._stream(None) == torch.cuda.current_stream().cuda_stream
        with torch.cuda.stream(stream):
            assert fx._stream(None) == stream.cuda_stream
            g = torch.zeros(rows, f, device="cuda")
            for _ in range(20):
                g.add_(0.1)                      # still running when the call is made
            h = torch.empty_like(g)
            fx.moe_swiglu(L, fx.MOE_F32, g, f, u, f, None, rows, f, h, f)
        stream.synchronize()
        want = swiglu_reference(g, u)
        assert torch.allclose(h.double(), want, rtol=1e-5, atol=1e-6)


# ------------------------------------------------------------ the ends of the ranges

@pytest.mark.parametrize("op", OPS)
def test_mm_with_256_experts_and_the_shared_one(op):
    rng = np.random.default_rng(21)
    counts = rng.integers(0, 9, size=257)
    counts[[0, 100, 256]] = 0, 70, 300
    gr = Groups(counts.tolist(), 1, lead=1, tail=1)
    n, k = 72, 136
    x = ints(rng, (gr.rows, k), 3) if op != "dgrad" else None
    dy = ints(rng, (gr.rows, n), 3) if op != "mm" else None
    w = ints(rng, (gr.G, n, k), 3) if op != "wgrad" else None
    res = run_mm(op, gr, BF, BF, n, k, x, dy, w, ldo_extra=0)
    ref, _ = mm_reference(op, gr, x, dy, w)
    if op != "wgrad":
        res, ref = res[gr.first:gr.last], ref[gr.first:gr.last]
    assert torch.equal(res, ref.to(F32).to(BF))


@pytest.mark.parametrize("dual", [False, True])
def test_w4_with_256_experts_and_the_shared_one(dual):
    rng = np.random.default_rng(22)
    counts = rng.integers(0, 4, size=257)
    counts[[0, 77, 256]] = 0, 300, 33
    gr = Groups(counts.tolist(), 1, lead=1, tail=1)
    n, k, T = 72, 300, 50
    a, b = (W4(rng, gr.G, n, k, 32, True, BF, exact=True) for _ in range(2))
    x, xb, perm = w4_inputs(rng, gr, T, k, BF, True, up8(k))
    y = out_buffer(gr.rows, n, n, F32)
    args = (gr.layer, fx.MOE_BF16, xb, T, xb.stride(0), perm)
    if dual:
        fx.moe_w4_gate_up(*args, a.desc, b.desc, gr.offsets, gr.rows, n, k, fx.MOE_F32, y, n)
    else:
        fx.moe_w4_matvec(*args, a.desc, gr.offsets, gr.rows, n, k, fx.MOE_F32, y, n)
    status_ok(gr.layer)
    assert (y[:gr.first] == SENTINEL).all() and (y[gr.last:] == SENTINEL).all()
    for g, (s, e) in enumerate(gr.spans):
        xr = x[perm[s:e].long()]
        ref = xr @ a.dense[g].T
        if dual:   # both products are exact; silu in fp32: exp and the quotient off by a few 2^-24
            ref = ref * torch.sigmoid(ref) * (xr @ b.dense[g].T)
            assert ((y[s:e].double() - ref).abs() <= 16 * 2.0 ** -24 * ref.abs() + 1e-30).all()
        else:
            assert torch.equal(y[s:e], ref.to(F32))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_w4_scales_at_any_element_address(group, zeros):
    """Scales and zero points that start in the middle of a 16-byte piece."""
    rng = np.random.default_rng(23)
    gr = Groups((3, 9), 0)
    n, k, T = 80, 1024, 4
    w = W4(rng, gr.G, n, k, group, zeros, BF, exact=True)

    def moved(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.view(-1)
        return buf[1:].view(t.shape)

    desc = fx.W4Weights(w.codes, moved(w.scales), moved(w.zeros) if zeros else None, fx.MOE_BF16, group)
    x, xb, perm = w4_inputs(rng, gr, T, k, BF, True, k)
    y = torch.empty(gr.rows, n, dtype=F32, device="cuda")
    fx.moe_w4_matvec(gr.layer, fx.MOE_BF16, xb, T, k, perm, desc, gr.offsets, gr.rows, n, k, fx.MOE_F32, y, n)
    status_ok(gr.layer)
    for g, (s, e) in enumerate(gr.spans):
        assert torch.equal(y[s:e], (x[perm[s:e].long()] @ w.dense[g].T).to(F32))


@pytest.mark.parametrize("n,k", [(1024, 1536), (100, 2048)])
def test_w4_gate_up_does_not_depend_on_the_batch(n, k):
    """A row's bits alone and among others in batches whose sizes split the
    contraction the same way."""
    rng = np.random.default_rng(24)
    gr = Groups((5, 0, 6), 0)
    a, b = (W4(rng, gr.G, n, k, 128, False, BF, exact=False) for _ in range(2))
    x, xb, perm = w4_inputs(rng, gr, 11, k, BF, False, k)
    call = lambda off, out: fx.moe_w4_gate_up(gr.layer, fx.MOE_BF16, xb, 11, k, None, a.desc, b.desc, off, gr.rows,  # noqa: E731
                                              n, k, fx.MOE_BF16, out, n)
    y, again, part = (out_buffer(gr.rows, n, n, BF) for _ in range(3))
    call(gr.offsets, y)
    call(gr.offsets, again)
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))
    call(torch.tensor([0, 5, 5, 6, 6], dtype=torch.int32, device="cuda"), part)   # group 2 holds row 5 alone
    assert torch.equal(part[:6].view(torch.int16), y[:6].view(torch.int16)) and (part[6:] == SENTINEL).all()
