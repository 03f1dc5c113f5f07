"""The grouped products' hand-over between the two CTAs of a pair: many short
tiles, each a few K blocks from operands to output, so that every stage's
copies, a weight gradient's tails and the accumulators change hands
thousands of times; and waits that give up at each of these points.

Integer inputs: every sum is exact in fp32, so one stale or early operand
shows in the bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import fp8_expert_ffn_b200 as fx  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
CODE = {BF: fx.MOE_BF16, F32: fx.MOE_F32}
B = fx.MOE_BF16


def groups(counts):
    E = len(counts)
    layer = fx.MoeLayer(128, E, 1, 1, fx.LayerWeights(*[None] * 6, torch.zeros(E, 128, device="cuda")), n_shared=0)
    ends = np.concatenate([[0], np.cumsum(counts)])
    off = torch.tensor(np.concatenate([ends, ends[-1:]]), dtype=torch.int32, device="cuda")
    return layer, off, [(int(a), int(b)) for a, b in zip(ends[:-1], ends[1:])]


def ints(gen, *shape):
    return torch.randint(-3, 4, shape, generator=gen, device="cuda").to(BF)


@pytest.mark.parametrize("out_dt", [BF, F32])
@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts,n,k", [
    (tuple(range(1, 66)), 600, 520),                  # narrow tiles; every tail length
    ((130, 63, 64, 65, 1, 0, 256, 300, 191) * 4, 520, 712),
    ((577, 640, 1100, 513) * 2, 264, 648),            # parts of 512 terms in fp32
])
def test_short_tiles_change_hands(counts, n, k, op, out_dt):
    layer, off, spans = groups(counts)
    rows, G = spans[-1][1], len(counts)
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    for _ in range(12):
        x, dy, w = ints(gen, rows, k), ints(gen, rows, n), ints(gen, G, n, k)
        outs = []
        for _ in range(3):   # back to back: a launch's set-up overlaps the one before it
            if op == "mm":
                y = torch.full((rows, n), 77.0, dtype=out_dt, device="cuda")
                fx.moe_grouped_mm(layer, B, x, k, w, k, off, rows, n, k, CODE[out_dt], y, n)
            elif op == "dgrad":
                y = torch.full((rows, k), 77.0, dtype=out_dt, device="cuda")
                fx.moe_grouped_mm_dgrad(layer, B, dy, n, w, k, off, rows, n, k, CODE[out_dt], y, k)
            else:
                y = torch.full((G, n, k), 77.0, dtype=out_dt, device="cuda")
                fx.moe_grouped_mm_wgrad(layer, B, dy, n, x, k, off, rows, n, k, CODE[out_dt], y, k)
            outs.append(y)
        code, bits = fx.moe_get_device_status(layer)
        assert code == fx.MOE_OK, hex(bits)
        for g, (a, b) in enumerate(spans):
            if op == "mm":
                got, want = [y[a:b] for y in outs], x[a:b].double() @ w[g].double().T
            elif op == "dgrad":
                got, want = [y[a:b] for y in outs], dy[a:b].double() @ w[g].double()
            else:
                got, want = [y[g] for y in outs], dy[a:b].double().T @ x[a:b].double()
            want = want.to(F32).to(out_dt)
            assert all(torch.equal(v, want) for v in got), f"group {g}"


@pytest.mark.parametrize("op", ["mm", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts", [(7, 40, 63), (64, 1), (1000, 130, 7)])
def test_withheld_stage_ends_both_ctas(counts, op):
    """The withheld first stage: a weight gradient's only block (a tail, whose
    copies the other CTA of the pair still makes), a whole block, one of many.
    All waits end, the status says so, and the next call is whole."""
    layer, off, spans = groups(counts)
    n, k, rows = 304, 328, spans[-1][1]
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, dy, w = ints(gen, rows, k), ints(gen, rows, n), ints(gen, len(counts), n, k)
    y = torch.empty({"mm": (rows, n), "dgrad": (rows, k), "wgrad": (len(counts), n, k)}[op], device="cuda")

    def call():
        if op == "mm":
            fx.moe_grouped_mm(layer, B, x, k, w, k, off, rows, n, k, fx.MOE_F32, y, n)
        elif op == "dgrad":
            fx.moe_grouped_mm_dgrad(layer, B, dy, n, w, k, off, rows, n, k, fx.MOE_F32, y, k)
        else:
            fx.moe_grouped_mm_wgrad(layer, B, dy, n, x, k, off, rows, n, k, fx.MOE_F32, y, k)

    for _ in range(3):
        fx.moe_test_inject_stall(layer, 1_000_000)
        call()
        code, bits = fx.moe_get_device_status(layer)
        assert code == fx.MOE_ERR_DEVICE and bits == fx.MOE_STATUS_WAIT_TIMEOUT
        y.fill_(77.0)
        call()
        code, bits = fx.moe_get_device_status(layer)
        assert code == fx.MOE_OK, hex(bits)
        for g, (a, b) in enumerate(spans):
            got, want = {"mm": lambda: (y[a:b], x[a:b].double() @ w[g].double().T),
                         "dgrad": lambda: (y[a:b], dy[a:b].double() @ w[g].double()),
                         "wgrad": lambda: (y[g], dy[a:b].double().T @ x[a:b].double())}[op]()
            assert torch.equal(got.double(), want)
