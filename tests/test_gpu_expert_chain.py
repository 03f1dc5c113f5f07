"""The expert operators as they are used together, from the library's routing
and permutation to its combine: the BF16 experts' forward and backward pass,
and a decode step with 4-bit experts, against float64.

The bound is on the relative Frobenius error: every bf16 rounding on the way
adds at most 2^-8 of the value it rounds, the products carry a relative error
through with a factor of about one, and the gate's slope is at most 1.1; the
comment at each comparison counts the roundings."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_expert_ffn_b200 as fx  # noqa: E402
from fp8_expert_ffn_b200 import torch_utils as tu  # noqa: E402

BF, B = torch.bfloat16, fx.MOE_BF16
STEP = 2.0 ** -8


def rel(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


class Routed:
    """A routing-only handle and one batch's route and permutation."""

    def __init__(self, H, E, K, S, T, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.rand = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).to(BF)
        self.H, self.E, self.K, self.S, self.T = H, E, K, S, T
        self.router = torch.randn(E, H, generator=g, device="cuda") * 0.05
        self.layer = fx.MoeLayer(H, E, K, 1, fx.LayerWeights(*[None] * 6, self.router), n_shared=S)
        self.x = self.rand(T, H)
        self.rows = T * (K + S)
        i32 = lambda *s: torch.empty(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.idx, self.w = i32(T, K), torch.empty(T, K, device="cuda")
        self.off, self.perm, self.inv = i32(E + 2), i32(self.rows), i32(T, K)
        self.xq = torch.empty(self.rows, H, dtype=torch.uint8, device="cuda")
        self.xs = torch.empty(H // 128, self.rows, device="cuda")
        self.ws = tu.workspace(self.layer, T)
        self.route()

    def route(self):
        n = self.ws.numel()
        fx.moe_route(self.layer, self.x, self.T, self.H, self.idx, self.w, None, self.ws, n)
        fx.moe_permute(self.layer, self.x, self.T, self.H, self.idx, self.off, self.perm, self.inv, self.xq, self.xs,
                       self.ws, n)

    def spans(self):
        o = self.off.tolist()
        return list(zip(o[:self.E + self.S], o[1:]))

    def combine64(self, y):
        out = (self.w.double()[..., None] * y[self.inv.long()]).sum(1)
        return out + y[self.T * self.K:] if self.S else out


def test_bf16_experts_forward_and_backward():
    H, F, E, K, S, T = 512, 256, 16, 4, 1, 210
    r = Routed(H, E, K, S, T, 1)
    G, R, L, off = E + S, r.rows, r.layer, r.off
    wg, wu, wd = r.rand(G, F, H, std=H ** -0.5), r.rand(G, F, H, std=H ** -0.5), r.rand(G, H, F, std=F ** -0.5)
    new = lambda *s, dt=BF: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
    xr = r.x[r.perm.long()]
    gate, up, h, y, out = new(R, F), new(R, F), new(R, F), new(R, H), new(T, H)
    fx.moe_grouped_mm(L, B, xr, H, wg, H, off, R, F, H, B, gate, F)
    fx.moe_grouped_mm(L, B, xr, H, wu, H, off, R, F, H, B, up, F)
    fx.moe_swiglu(L, B, gate, F, up, F, off, R, F, h, F)
    fx.moe_grouped_mm(L, B, h, F, wd, F, off, R, H, F, B, y, H)
    fx.moe_combine(L, y, r.inv, r.w, T, out, H)

    dout = r.rand(T, H)
    dyr = torch.empty(R, H, device="cuda")
    dyr[r.inv.view(-1).long()] = (r.w[..., None] * dout.float()[:, None]).view(-1, H)
    dyr[T * K:] = dout.float()
    dy = dyr.to(BF)
    dh, dgate, dup, h2 = new(R, F), new(R, F), new(R, F), new(R, F)
    dwg, dwu, dwd = (new(*w.shape, dt=torch.float32) for w in (wg, wu, wd))
    dxg, dxu = new(R, H, dt=torch.float32), new(R, H, dt=torch.float32)
    fx.moe_grouped_mm_dgrad(L, B, dy, H, wd, F, off, R, H, F, B, dh, F)
    fx.moe_swiglu_backward(L, B, dh, F, gate, F, up, F, off, R, F, dgate, F, dup, F, h2, F)
    fx.moe_grouped_mm_wgrad(L, B, dy, H, h2, F, off, R, H, F, fx.MOE_F32, dwd, F)
    fx.moe_grouped_mm_wgrad(L, B, dgate, F, xr, H, off, R, F, H, fx.MOE_F32, dwg, H)
    fx.moe_grouped_mm_wgrad(L, B, dup, F, xr, H, off, R, F, H, fx.MOE_F32, dwu, H)
    fx.moe_grouped_mm_dgrad(L, B, dgate, F, wg, H, off, R, F, H, fx.MOE_F32, dxg, H)
    fx.moe_grouped_mm_dgrad(L, B, dup, F, wu, H, off, R, F, H, fx.MOE_F32, dxu, H)
    code, bits = fx.moe_get_device_status(L)
    assert code == fx.MOE_OK, hex(bits)

    d = lambda t: t.double().detach().requires_grad_()  # noqa: E731
    x64, g64, u64, d64 = d(xr), d(wg), d(wu), d(wd)
    parts = []
    for g, (a, b) in enumerate(r.spans()):
        ga = x64[a:b] @ g64[g].T
        parts.append((ga * torch.sigmoid(ga) * (x64[a:b] @ u64[g].T)) @ d64[g].T)
    y64 = torch.cat(parts)
    out64 = r.combine64(y64)
    out64.backward(dout.double())
    assert rel(out, out64) <= 4 * 1.1 * STEP                 # gate and up, h, y, out
    for got, want, roundings in ((dwd, d64.grad, 3),          # dy; gate and up, h
                                 (dwg, g64.grad, 5), (dwu, u64.grad, 4),   # dy, dh, gate and up, dgate (dup)
                                 (dxg + dxu, x64.grad, 5)):
        assert rel(got, want) <= roundings * 1.1 * STEP
    assert torch.equal(h.view(torch.int16), h2.view(torch.int16))


@pytest.mark.parametrize("T", [1, 7, 40])
@pytest.mark.parametrize("group,zeros", [(128, False), (32, True)])
def test_w4_decode_step(T, group, zeros):
    H, F, E, K, S = 512, 384, 20, 4, 1
    r = Routed(H, E, K, S, T, 2)
    G, R, L = E + S, r.rows, r.layer
    q = [tu.w4_quantize(r.rand(G, n, k, std=k ** -0.5), group, zeros) for n, k in ((F, H), (F, H), (H, F))]
    h = torch.empty(R, F, dtype=BF, device="cuda")
    y = torch.empty(R, H, dtype=BF, device="cuda")
    out = torch.empty(T, H, dtype=BF, device="cuda")

    def step():
        r.route()
        fx.moe_w4_gate_up(L, B, r.x, T, H, r.perm, q[0], q[1], r.off, R, F, H, B, h, F)
        fx.moe_w4_matvec(L, B, h, R, F, None, q[2], r.off, R, H, F, B, y, H)
        fx.moe_combine(L, y, r.inv, r.w, T, out, H)

    def want():
        wg, wu, wd = (tu.w4_values(w, k).double() for w, k in zip(q, (H, H, F)))
        xr = r.x.double()[r.perm.long()]
        y64 = torch.empty(R, H, dtype=torch.float64, device="cuda")
        for g, (a, b) in enumerate(r.spans()):
            ga = xr[a:b] @ wg[g].T
            y64[a:b] = (ga * torch.sigmoid(ga) * (xr[a:b] @ wu[g].T)) @ wd[g].T
        return r.combine64(y64)

    step()
    assert rel(out, want()) <= 3 * 1.1 * STEP                # h, y, out
    # the same step captured, replayed on another batch (other experts, other group sizes)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        r.x.copy_(r.rand(T, H))
        out.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert rel(out, want()) <= 3 * 1.1 * STEP
    code, bits = fx.moe_get_device_status(L)
    assert code == fx.MOE_OK, hex(bits)


def test_peer_plan_offsets_serve_the_operators():
    """moe_ep_plan's offsets alone (no gather) are enough for the products."""
    H, F, E, K, S, T = 256, 128, 8, 2, 1, 33
    r = Routed(H, E, K, S, T, 3)
    off = torch.empty_like(r.off)
    fx.moe_ep_plan(r.layer, r.idx, T, off, r.ws, r.ws.numel())
    assert torch.equal(off, r.off)
    w = r.rand(E + S, F, H, std=H ** -0.5)
    y = torch.empty(r.rows, F, dtype=BF, device="cuda")
    fx.moe_grouped_mm(r.layer, B, r.x[r.perm.long()], H, w, H, off, r.rows, F, H, B, y, F)
    x64 = r.x.double()[r.perm.long()]
    want = torch.cat([x64[a:b] @ w[g].double().T for g, (a, b) in enumerate(r.spans())])
    assert rel(y, want) <= STEP
