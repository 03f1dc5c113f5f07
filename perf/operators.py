"""The expert operators beside the FP8 layer: products grouped by expert in
bf16 / fp16 with their two gradients, SwiGLU over the grouped rows with its
gradient, and decode products with 4-bit expert weights. Sizes are those of
the layers this package is tested and benchmarked on: hidden 5120 with
experts of FFN 1536 (top-8 plus a shared one), the FFN 1500 variant, the
vision tower's hidden 1536 / FFN 2112 / 64 experts top-2, the dense FFN of
13824, and the 16-expert toy layer of hidden 512 / FFN 256."""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# "n" x "k" is one expert's weight ([n][k], y = x w^T), "E" routed experts of
# which every one of "T" tokens takes "topk", "S" shared experts that take all
# tokens; "skew" is the exponent of a Zipf law over the experts (0: balanced).
MM = ("mm", "dgrad", "wgrad")
W4 = ("w4_gate_up", "w4_matvec")
ACT = ("swiglu", "swiglu_backward")


def listed():
    return [
        # one decode step of the BF16 experts' gate projection: every touched expert's weight is streamed
        dict(name="mm decode", op="mm", dtype="bf16", out="bf16", T=64, E=64, S=1, topk=8, n=1536, k=5120, skew=0.0),
        # the same projection over a training batch / long prompt, with the usual uneven load
        dict(name="mm prefill", op="mm", dtype="bf16", out="bf16", T=4096, E=32, S=1, topk=8, n=1536, k=5120, skew=0.5),
        # the smallest backward call: the toy layer's down projection
        dict(name="dgrad toy", op="dgrad", dtype="bf16", out="bf16", T=32, E=16, S=1, topk=4, n=512, k=256, skew=0.0),
        # input gradient of the down projection over a training batch
        dict(name="dgrad train", op="dgrad", dtype="bf16", out="bf16", T=4096, E=32, S=1, topk=8, n=5120, k=1536,
             skew=0.5),
        # weight gradient of the vision tower's experts, kept in fp32 for the optimiser
        dict(name="wgrad vision", op="wgrad", dtype="f16", out="f32", T=4096, E=16, S=0, topk=2, n=2112, k=1536,
             skew=0.3),
        # weight gradient of the gate projection of the FFN 1500 variant (ragged edge tiles)
        dict(name="wgrad f1500", op="wgrad", dtype="bf16", out="bf16", T=4099, E=15, S=1, topk=8, n=1500, k=5120,
             skew=0.5),
        # one token of decode through the 4-bit gate and up projections: latency
        dict(name="w4 gate_up T1", op="w4_gate_up", dtype="bf16", out="bf16", T=1, E=256, S=1, topk=8, n=1536, k=5120,
             group=128, zeros=False, skew=0.0),
        # a decode batch over all experts: the codes are streamed once
        dict(name="w4 gate_up T64", op="w4_gate_up", dtype="bf16", out="bf16", T=64, E=256, S=1, topk=8, n=1536,
             k=5120, group=128, zeros=False, skew=0.0),
        # the down projection of a small decode batch, asymmetric codes
        dict(name="w4 down T16", op="w4_matvec", dtype="f16", out="f16", T=16, E=64, S=1, topk=8, n=5120, k=1536,
             group=64, zeros=True, skew=0.5),
        # the dense FFN's gate projection, one weight matrix and a few rows
        dict(name="w4 dense T5", op="w4_matvec", dtype="bf16", out="f32", T=5, E=1, S=0, topk=1, n=13824, k=5120,
             group=32, zeros=False, skew=0.0),
        # activation between the products of a decode batch
        dict(name="swiglu decode", op="swiglu", dtype="bf16", out="bf16", T=64, E=64, S=1, topk=8, n=1536, k=0,
             skew=0.0),
        # its gradient over a training batch
        dict(name="swiglu_backward train", op="swiglu_backward", dtype="bf16", out="bf16", T=4096, E=32, S=1, topk=8,
             n=1536, k=0, skew=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.4 else max(lo, v // 64 * 64) if v >= 128 else max(lo, v // 8 * 8)


def draw(rng):
    while True:
        op = rng.choice(MM + MM + W4 + W4 + ACT)
        E = rng.choice((1, 3, 8, 16, 31, 64, 128, 256))
        c = dict(op=op, dtype=rng.choice(("bf16", "f16")), E=E, S=rng.choice((0, 1)),
                 topk=rng.randint(1, min(8, E)), skew=rng.choice((0.0, 0.5, 1.0)))
        if op in MM:
            c.update(T=_log(rng, 1, 4500), n=_size(rng, 40, 5120), k=_size(rng, 40, 5120))
            c["out"] = rng.choice((c["dtype"], "f32"))
        elif op in W4:
            c.update(T=_log(rng, 1, 64), n=_size(rng, 40, 5120), k=_size(rng, 64, 5120),
                     group=rng.choice((32, 64, 128)), zeros=rng.random() < 0.5)
            c["out"] = rng.choice((c["dtype"], "f32"))
        else:
            c.update(T=_log(rng, 1, 4500), n=_size(rng, 40, 2112), k=0, dtype=rng.choice(("bf16", "f16", "f32")))
            c["out"] = c["dtype"]
        w = work(c)
        weights = (E + c["S"]) * c["n"] * c["k"]
        # no dearer than the dearest listed case of its kind
        if op in MM and w["flops"] <= 5.8e11 and weights <= 1.3e8 * (4 if op == "mm" else 1):
            return c
        if op in W4 and w["bytes"] <= 2.0e9 and weights <= 2.1e9:
            return c
        if op in ACT and w["bytes"] <= 5.6e8:
            return c


def _offsets(case, seed):
    """Group offsets [E+2] (the shared expert's rows last) and each row's token."""
    rng = np.random.default_rng([seed, 7])
    T, E, topk = case["T"], case["E"], case["topk"]
    score = rng.gumbel(size=(T, E)) - case["skew"] * np.log(1.0 + rng.permutation(E))[None, :]
    pick = np.argsort(-score, axis=1)[:, :topk]
    order = np.argsort(pick.ravel(), kind="stable")
    off = np.zeros(E + 2, np.int64)
    off[1:E + 1] = np.cumsum(np.bincount(pick.ravel(), minlength=E))
    off[E + 1] = off[E] + T * case["S"]
    perm = np.concatenate([order // topk] + [np.arange(T)] * case["S"])
    return off.tolist(), perm.astype(np.int32)


def work(case):
    off, _ = _offsets(case, 0)
    rows, n, k = off[-1], case["n"], case["k"]
    touched = sum(b > a for a, b in zip(off, off[1:]))
    b, o = TYPES[case["dtype"]].itemsize, TYPES[case["out"]].itemsize
    if case["op"] == "mm":
        return {"bytes": b * (rows * k + touched * n * k) + o * rows * n, "flops": 2 * rows * n * k}
    if case["op"] == "dgrad":
        return {"bytes": b * (rows * n + touched * n * k) + o * rows * k, "flops": 2 * rows * n * k}
    if case["op"] == "wgrad":
        return {"bytes": b * rows * (n + k) + o * (case["E"] + case["S"]) * n * k, "flops": 2 * rows * n * k}
    if case["op"] in W4:
        mats = 2 if case["op"] == "w4_gate_up" else 1
        groups = -(-k // case["group"])
        per = n * ((k + 1) // 2 + groups * (b + (1 if case["zeros"] else 0)))
        return {"bytes": mats * touched * per + b * case["T"] * k + 4 * rows + o * rows * n,
                "flops": 2 * mats * rows * n * k}
    streams = 3 if case["op"] == "swiglu" else 5
    return {"bytes": streams * b * rows * n, "flops": (5 if case["op"] == "swiglu" else 12) * rows * n}


def _pad8(v):
    return (v + 7) // 8 * 8


def _randn(gen, shape, dtype, std):
    """Normal values in rows padded to 8 elements; the view of the real columns."""
    t = torch.empty(*shape[:-1], _pad8(shape[-1]), dtype=dtype, device="cuda")
    if t.numel():
        part = t.view(-1, t.shape[-1])
        step = max(1, (1 << 27) // part.shape[1])
        for i in range(0, part.shape[0], step):   # in slices: the fp32 draw stays small
            p = part[i:i + step]
            p.copy_(torch.randn(p.shape, generator=gen, device="cuda").mul_(std))
    return t[..., :shape[-1]]


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 11)
    off, perm = _offsets(case, seed)
    dt, rows, n, k, G = TYPES[case["dtype"]], off[-1], case["n"], case["k"], case["E"] + case["S"]
    s = dict(off=off, perm=perm, rows=rows)
    op = case["op"]
    if op in ("mm", "dgrad"):
        s["w"] = _randn(gen, (G, n, k), dt, 1 / math.sqrt(k))
    if op in ("mm", "wgrad"):
        s["x"] = _randn(gen, (rows, k), dt, 1.0)
    if op in ("dgrad", "wgrad"):
        s["dy"] = _randn(gen, (rows, n), dt, 0.05)
    if op in W4:
        s["x"] = _randn(gen, (case["T"], k), dt, 1.0)
        ng = -(-k // case["group"])
        ld = -(-((k + 1) // 2) // 16) * 16
        for name in ("gate", "up") if op == "w4_gate_up" else ("w",):
            s[name] = dict(
                codes=torch.randint(0, 256, (G, n, ld), generator=gen, device="cuda", dtype=torch.uint8),
                # code steps of weights of spread 1/sqrt(k): uneven from group to group
                scales=(torch.rand((G, n, ng), generator=gen, device="cuda").add_(0.5) * (0.2 / math.sqrt(k))).to(dt),
                zeros=torch.randint(5, 11, (G, n, ng), generator=gen, device="cuda", dtype=torch.uint8)
                if case["zeros"] else None)
    if op in ACT:
        s["gate"] = _randn(gen, (rows, n), dt, 2.0)
        s["up"] = _randn(gen, (rows, n), dt, 1.0)
        if op == "swiglu_backward":
            s["dh"] = _randn(gen, (rows, n), dt, 0.05)
    return s


def _empty(rows, cols, dtype):
    return torch.empty(rows, _pad8(cols), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    out, rows, n, k, G = TYPES[case["out"]], s["rows"], case["n"], case["k"], case["E"] + case["S"]
    op = case["op"]
    s["offsets"] = torch.tensor(s["off"], dtype=torch.int32, device="cuda")
    s["perm"] = torch.from_numpy(s["perm"]).cuda()
    if op == "wgrad":
        s["y"] = torch.empty(G, n, k, dtype=out, device="cuda")
    elif op == "swiglu_backward":
        s["y"] = _empty(rows, n, out), _empty(rows, n, out)
    else:
        s["y"] = _empty(rows, k if op == "dgrad" else n, out)
    if own:
        import fp8_expert_ffn_b200 as fx
        s["fx"] = fx
        router = torch.zeros(case["E"], 128, dtype=torch.float32, device="cuda")
        # the handle a user of the experts' products keeps: router, groups, status word
        s["layer"] = fx.MoeLayer(128, case["E"], case["topk"], 1,
                                 fx.LayerWeights(None, None, None, None, None, None, router), n_shared=case["S"])
        s["type"] = {"bf16": fx.MOE_BF16, "f16": fx.MOE_F16, "f32": fx.MOE_F32}[case["dtype"]]
        s["out_type"] = {"bf16": fx.MOE_BF16, "f16": fx.MOE_F16, "f32": fx.MOE_F32}[case["out"]]
        for name in ("gate", "up", "w"):
            if op in W4 and name in s:
                s[name]["handle"] = fx.W4Weights(s[name]["codes"], s[name]["scales"], s[name]["zeros"], s["type"],
                                                 case["group"])
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    c, fx, L, ty, oty, off, rows, y = (s["case"], s["fx"], s["layer"], s["type"], s["out_type"], s["offsets"],
                                       s["rows"], s["y"])
    op, n, k = c["op"], c["n"], c["k"]
    if op == "mm":
        fx.moe_grouped_mm(L, ty, s["x"], s["x"].stride(0), s["w"], s["w"].stride(1), off, rows, n, k, oty, y,
                          y.stride(0))
    elif op == "dgrad":
        fx.moe_grouped_mm_dgrad(L, ty, s["dy"], s["dy"].stride(0), s["w"], s["w"].stride(1), off, rows, n, k, oty, y,
                                y.stride(0))
    elif op == "wgrad":
        fx.moe_grouped_mm_wgrad(L, ty, s["dy"], s["dy"].stride(0), s["x"], s["x"].stride(0), off, rows, n, k, oty, y,
                                y.stride(1), False)
    elif op == "w4_gate_up":
        fx.moe_w4_gate_up(L, ty, s["x"], c["T"], s["x"].stride(0), s["perm"], s["gate"]["handle"], s["up"]["handle"],
                          off, rows, n, k, oty, y, y.stride(0))
    elif op == "w4_matvec":
        fx.moe_w4_matvec(L, ty, s["x"], c["T"], s["x"].stride(0), s["perm"], s["w"]["handle"], off, rows, n, k, oty,
                         y, y.stride(0))
    elif op == "swiglu":
        fx.moe_swiglu(L, ty, s["gate"], s["gate"].stride(0), s["up"], s["up"].stride(0), off, rows, n, y, y.stride(0))
    else:
        dg, du = y
        fx.moe_swiglu_backward(L, ty, s["dh"], s["dh"].stride(0), s["gate"], s["gate"].stride(0), s["up"],
                               s["up"].stride(0), off, rows, n, dg, dg.stride(0), du, du.stride(0), None, 0)
    return y


def _spans(off):
    return [(g, a, b) for g, (a, b) in enumerate(zip(off, off[1:])) if b > a]


def _dequant32(w, g, group, k):
    codes = w["codes"][g]
    q = torch.stack((codes & 15, codes >> 4), dim=-1).view(codes.shape[0], -1)[:, :k].float()
    zero = 8.0 if w["zeros"] is None else w["zeros"][g].float().repeat_interleave(group, 1)[:, :k]
    return (q - zero) * w["scales"][g].float().repeat_interleave(group, 1)[:, :k]


def _plain(s):
    c, y, off = s["case"], s["y"], s["off"]
    op, k = c["op"], c["k"]
    if op == "mm":
        for g, a, b in _spans(off):
            y[a:b] = s["x"][a:b].float() @ s["w"][g].float().t()
    elif op == "dgrad":
        for g, a, b in _spans(off):
            y[a:b] = s["dy"][a:b].float() @ s["w"][g].float()
    elif op == "wgrad":
        for g in range(y.shape[0]):
            a, b = off[g], off[g + 1]
            y[g] = s["dy"][a:b].float().t() @ s["x"][a:b].float()
    elif op in W4:
        xr = s["x"][s["perm"].long()].float()
        for g, a, b in _spans(off):
            if op == "w4_matvec":
                y[a:b] = xr[a:b] @ _dequant32(s["w"], g, c["group"], k).t()
            else:
                gate = xr[a:b] @ _dequant32(s["gate"], g, c["group"], k).t()
                up = xr[a:b] @ _dequant32(s["up"], g, c["group"], k).t()
                y[a:b] = gate / (1 + torch.exp(-gate)) * up
    else:
        gate, up = s["gate"].float(), s["up"].float()
        sig = 1 / (1 + torch.exp(-gate))
        if op == "swiglu":
            y.copy_(gate * sig * up)
        else:
            dh = s["dh"].float()
            y[0].copy_(dh * up * sig * (1 + gate * (1 - sig)))
            y[1].copy_(dh * gate * sig)
    return y


def exact(case, seed):
    """The definitions in float64, from the inputs alone."""
    s = _inputs(case, seed)
    op, off, rows, n, k = case["op"], s["off"], s["rows"], case["n"], case["k"]
    d = torch.float64
    ends = list(zip(off[:-1], off[1:]))
    if op == "wgrad":
        res = torch.zeros(case["E"] + case["S"], n, k, dtype=d, device="cuda")
        for g in range(res.shape[0]):
            lo, hi = ends[g]
            res[g] = torch.einsum("rn,rk->nk", s["dy"][lo:hi].to(d), s["x"][lo:hi].to(d))
        return res
    if op in ("mm", "dgrad"):
        res = torch.zeros(rows, n if op == "mm" else k, dtype=d, device="cuda")
        for g, (lo, hi) in enumerate(ends):
            if hi > lo and op == "mm":
                res[lo:hi] = torch.einsum("rk,nk->rn", s["x"][lo:hi].to(d), s["w"][g].to(d))
            elif hi > lo:
                res[lo:hi] = torch.einsum("rn,nk->rk", s["dy"][lo:hi].to(d), s["w"][g].to(d))
        return res
    if op in W4:
        col = torch.arange(k, device="cuda")
        grp = col // case["group"]
        tok = torch.from_numpy(s["perm"]).cuda().long()

        def product(w, g, lo, hi):
            byte = w["codes"][g][:, col // 2].to(torch.int32)
            code = torch.where(col % 2 == 0, byte % 16, byte // 16).to(d)
            mid = w["zeros"][g][:, grp].to(d) if case["zeros"] else 8.0
            return torch.einsum("rk,nk->rn", s["x"][tok[lo:hi]].to(d), (code - mid) * w["scales"][g][:, grp].to(d))

        res = torch.zeros(rows, n, dtype=d, device="cuda")
        for g, (lo, hi) in enumerate(ends):
            if hi > lo and op == "w4_matvec":
                res[lo:hi] = product(s["w"], g, lo, hi)
            elif hi > lo:
                a = product(s["gate"], g, lo, hi)
                res[lo:hi] = a * torch.sigmoid(a) * product(s["up"], g, lo, hi)
        return res
    a, b = s["gate"].to(d), s["up"].to(d)
    p, q = torch.sigmoid(a), torch.sigmoid(-a)
    if op == "swiglu":
        return a * p * b
    e = s["dh"].to(d)
    return e * b * (p + a * p * q), e * a * p
