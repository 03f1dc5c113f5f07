"""The expert operators' refusals, without a GPU: every bad argument is
reported by the host before any CUDA call, whatever the handle holds (a
zeroed block of memory stands in for it: it is not looked at before the
arguments are in order)."""
import ctypes

import pytest

import fp8_expert_ffn_b200 as fx

KEEP = ctypes.create_string_buffer(1 << 14)
H = ctypes.addressof(KEEP)
P = 1 << 20           # an aligned address that is never read
BAD, MIS = fx.MOE_ERR_INVALID_ARG, fx.MOE_ERR_MISALIGNED
B, F, F32 = fx.MOE_BF16, fx.MOE_F16, fx.MOE_F32


def mm(fn="moe_grouped_mm", layer=H, type=B, a=P, lda=64, b=P, ldb=64, off=P, rows=5, n=64, k=64, out_type=B, out=P,
       ldo=64, acc=0):
    args = [layer, type, a, lda, b, ldb, off, rows, n, k, out_type, out, ldo]
    if fn.endswith("wgrad"):
        args.append(acc)
    return getattr(fx.lib(), fn)(*args, None)


MM = ("moe_grouped_mm", "moe_grouped_mm_dgrad", "moe_grouped_mm_wgrad")


@pytest.mark.parametrize("fn", MM)
@pytest.mark.parametrize("kw,code", [
    (dict(layer=None), BAD), (dict(rows=-1), BAD), (dict(type=F32), BAD), (dict(type=3), BAD), (dict(type=-1), BAD),
    (dict(out_type=F), BAD), (dict(out_type=7), BAD), (dict(a=None), BAD), (dict(b=None), BAD), (dict(off=None), BAD),
    (dict(out=None), BAD), (dict(n=0), BAD), (dict(k=0), BAD), (dict(n=65537), BAD), (dict(k=65537), BAD),
    (dict(lda=56), BAD), (dict(ldb=56), BAD), (dict(ldo=63), BAD), (dict(lda=(1 << 20) + 8), BAD),
    (dict(ldb=(1 << 20) + 8), BAD), (dict(ldo=(1 << 20) + 1), BAD), (dict(a=P + 8), MIS), (dict(b=P + 2), MIS),
    (dict(lda=68), MIS), (dict(ldb=66), MIS), (dict(out=P + 1), MIS), (dict(out=P + 2, out_type=F32), MIS),
])
def test_mm_refusals(fn, kw, code):
    assert mm(fn, **kw) == code


def test_mm_sizes_are_checked_against_the_right_stride():
    # n = 40, k = 64: the row operand of the forward is k wide, of dgrad n, of wgrad n and k
    assert mm(n=40, lda=40, ldo=40) == BAD
    assert mm("moe_grouped_mm_dgrad", n=40, lda=40, ldo=40) == BAD
    assert mm("moe_grouped_mm_wgrad", n=40, lda=40, ldb=40) == BAD
    assert mm("moe_grouped_mm_wgrad", n=40, lda=32) == BAD


def test_wgrad_refusals_without_rows():
    w = "moe_grouped_mm_wgrad"
    assert mm(w, acc=2) == BAD and mm(w, acc=-1) == BAD
    for kw, code in ((dict(out=None), BAD), (dict(k=0), BAD), (dict(ldo=63), BAD), (dict(type=F32), BAD),
                     (dict(out_type=F), BAD), (dict(out=P + 1), MIS)):
        assert mm(w, rows=0, a=None, b=None, **kw) == code


def test_no_rows_is_a_no_op():
    for fn in MM[:2]:
        assert mm(fn, rows=0, a=None, b=None, off=None, out=None) == fx.MOE_OK
    lib = fx.lib()
    assert lib.moe_swiglu(H, B, None, 0, None, 0, None, 0, 0, None, 0, None) == fx.MOE_OK
    assert lib.moe_swiglu_backward(H, B, None, 0, None, 0, None, 0, None, 0, 0, None, 0, None, 0, None, 0,
                                   None) == fx.MOE_OK
    assert w4(rows=0, x=None, y=None) == fx.MOE_OK and w4("moe_w4_gate_up", rows=0, x=None) == fx.MOE_OK


def act(backward, layer=H, type=B, rows=5, f=64, ptr=None, ld=None):
    names = ("dh", "gate", "up", "o0", "o1", "h") if backward else ("gate", "up", "o0")
    p = {x: P + 4096 * i for i, x in enumerate(names)}
    s = {x: 64 for x in names}
    p.update(ptr or {})
    s.update(ld or {})
    if backward:
        return fx.lib().moe_swiglu_backward(layer, type, p["dh"], s["dh"], p["gate"], s["gate"], p["up"], s["up"], None,
                                            rows, f, p["o0"], s["o0"], p["o1"], s["o1"], p["h"], s["h"], None)
    return fx.lib().moe_swiglu(layer, type, p["gate"], s["gate"], p["up"], s["up"], None, rows, f, p["o0"], s["o0"],
                               None)


@pytest.mark.parametrize("backward", [False, True])
def test_swiglu_refusals(backward):
    for kw, code in ((dict(layer=None), BAD), (dict(rows=-1), BAD), (dict(type=3), BAD), (dict(type=-1), BAD),
                     (dict(f=0), BAD), (dict(f=65537), BAD), (dict(ptr=dict(gate=None)), BAD),
                     (dict(ptr=dict(up=None)), BAD), (dict(ptr=dict(o0=None)), BAD), (dict(ld=dict(gate=63)), BAD),
                     (dict(ld=dict(o0=(1 << 20) + 1)), BAD), (dict(ptr=dict(up=P + 1)), MIS),
                     (dict(type=F32, ptr=dict(o0=P + 2)), MIS)):
        assert act(backward, **kw) == code, kw
    if backward:
        for kw in (dict(ptr=dict(o0=P, o1=P)), dict(ptr=dict(h=P, o1=P)), dict(ptr=dict(h=P, o0=P)),
                   dict(ptr=dict(o1=None)), dict(ptr=dict(dh=None)), dict(ld=dict(h=10))):
            assert act(True, **kw) == BAD, kw


def w4(fn="moe_w4_matvec", layer=H, type=B, x=P, x_rows=5, ldx=64, perm=P, codes=P, scales=P, zeros=None, scale_type=B,
       group=32, ld=32, up=None, off=P, rows=5, n=64, k=64, y_type=B, y=P, ldy=64):
    one = fx.moe_w4_weights(codes, scales, zeros, scale_type, group, ld)
    two = fx.moe_w4_weights(*({**dict(codes=P, scales=P, zeros=zeros, scale_type=scale_type, group=group, ld=ld),
                               **(up or {})}.values()))
    ws = [ctypes.byref(one)] + ([ctypes.byref(two)] if fn == "moe_w4_gate_up" else [])
    return getattr(fx.lib(), fn)(layer, type, x, x_rows, ldx, perm, *ws, off, rows, n, k, y_type, y, ldy, None)


@pytest.mark.parametrize("fn", ["moe_w4_matvec", "moe_w4_gate_up"])
@pytest.mark.parametrize("kw,code", [
    (dict(layer=None), BAD), (dict(rows=-1), BAD), (dict(type=F32), BAD), (dict(y_type=F), BAD), (dict(x=None), BAD),
    (dict(y=None), BAD), (dict(off=None), BAD), (dict(n=0), BAD), (dict(k=0), BAD), (dict(n=65537), BAD),
    (dict(ldx=56), BAD), (dict(ldy=63), BAD), (dict(x_rows=0), BAD), (dict(rows=(1 << 20) + 1), BAD), (dict(perm=None, x_rows=4), BAD),
    (dict(codes=None), BAD), (dict(scales=None), BAD), (dict(scale_type=3), BAD), (dict(group=16), BAD),
    (dict(group=256), BAD), (dict(ld=16), BAD), (dict(k=65, ldx=72, ld=32), BAD), (dict(ld=65552), BAD),
    (dict(x=P + 8), MIS), (dict(ldx=68), MIS), (dict(codes=P + 8), MIS), (dict(ld=40), MIS), (dict(scales=P + 1), MIS),
    (dict(scales=P + 2, scale_type=F32), MIS), (dict(y=P + 1), MIS),
])
def test_w4_refusals(fn, kw, code):
    assert w4(fn, **kw) == code


def test_w4_gate_up_wants_two_alike():
    for up in (dict(group=64), dict(scale_type=F), dict(ld=48), dict(zeros=P), dict(codes=None), dict(scales=None)):
        assert w4("moe_w4_gate_up", up=up) == BAD, up
    lib = fx.lib()
    one = fx.moe_w4_weights(P, P, None, B, 32, 32)
    assert lib.moe_w4_matvec(H, B, P, 5, 64, P, None, P, 5, 64, 64, B, P, 64, None) == BAD
    assert lib.moe_w4_gate_up(H, B, P, 5, 64, P, ctypes.byref(one), None, P, 5, 64, 64, B, P, 64, None) == BAD
