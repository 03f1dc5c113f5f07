"""PyTorch plumbing for the library: device copies of a layer's weights,
workspace allocation, bf16 bit-pattern conversions and the packing of 4-bit
weights. No layer arithmetic."""
from __future__ import annotations

import numpy as np
import torch

from . import MOE_BF16, MOE_F16, MOE_F32, LayerWeights, MoeLayer, W4Weights, moe_workspace_size

TYPE_CODES = {torch.bfloat16: MOE_BF16, torch.float16: MOE_F16, torch.float32: MOE_F32}   # moe_dtype


def to_device(a: np.ndarray, device="cuda") -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a)).to(device)


def bf16_tensor(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """uint16 bf16 bit patterns -> torch.bfloat16 tensor on `device`."""
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(device)


def bf16_bits(t: torch.Tensor) -> np.ndarray:
    return t.detach().contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def upload_layer(host, device="cuda", routed_scaling=None, share_experts: MoeLayer = None) -> MoeLayer:
    """host: an object with shape (H, E, K, F, ld_f) and the numpy weight arrays
    router_w, w_gate, s_gate, w_up, s_up, w_down, s_down; optional router
    settings routed_scaling, n_group, topk_group, norm_topk and router_bias
    (numpy [E]) are read from it when present. With share_experts, the expert
    tensors of that layer are reused and only the router is copied."""
    sh = host.shape
    if share_experts is not None:
        src = share_experts.weights
        w = LayerWeights(w_gate=src.w_gate, w_up=src.w_up, w_down=src.w_down, s_gate=src.s_gate,
                         s_up=src.s_up, s_down=src.s_down, router_w=to_device(host.router_w, device))
    else:
        w = LayerWeights(
            w_gate=to_device(host.w_gate, device), w_up=to_device(host.w_up, device),
            w_down=to_device(host.w_down, device), s_gate=to_device(host.s_gate, device),
            s_up=to_device(host.s_up, device), s_down=to_device(host.s_down, device),
            router_w=to_device(host.router_w, device))
    if routed_scaling is None:
        routed_scaling = getattr(host, "routed_scaling", 1.0)
    bias = getattr(host, "router_bias", None)
    bias_dev = None if bias is None else to_device(np.asarray(bias, np.float32), device)
    return MoeLayer(sh.H, sh.E, sh.K, sh.F, w, ld_h=host.w_gate.shape[2], ld_f=host.w_down.shape[2],
                    routed_scaling=routed_scaling, n_shared=getattr(sh, "S", 1),
                    n_group=getattr(host, "n_group", 1), topk_group=getattr(host, "topk_group", 1),
                    norm_topk=getattr(host, "norm_topk", True), router_bias=bias_dev)


def workspace(layer: MoeLayer, T: int, device="cuda") -> torch.Tensor:
    n = moe_workspace_size(layer, T)
    if n == 0:
        raise ValueError("moe_workspace_size returned 0")
    return torch.empty(n, dtype=torch.uint8, device=device)


def w4_quantize(w: torch.Tensor, group: int = 128, zeros: bool = False, scale_dtype=torch.bfloat16) -> W4Weights:
    """4-bit weights (round to nearest) of w [experts][n][k], for moe_w4_matvec
    and moe_w4_gate_up: one scale per `group` columns of a row, the largest
    magnitude at +-7 steps around a fixed zero point of 8, or, with `zeros`,
    the group's range spread over the 16 codes around its own zero point.
    An offline step, done once per checkpoint."""
    G, n, k = w.shape
    ng, ld = -(-k // group), -(-((k + 1) // 2) // 16) * 16
    v = torch.nn.functional.pad(w.float(), (0, ng * group - k)).view(G, n, ng, group)
    if zeros:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        scales = ((hi - lo) / 15).to(scale_dtype)
    else:
        scales = (v.abs().amax(-1) / 7).to(scale_dtype)
    step = scales.float()
    step = torch.where(step > 0, step, torch.ones_like(step))   # a group of zeros: every code is its zero point
    z = (-lo / step).round().clamp(0, 15) if zeros else torch.full_like(step, 8.0)
    q = ((v / step[..., None]).round() + z[..., None]).clamp(0, 15).to(torch.uint8).view(G, n, -1)[:, :, :k]
    codes = torch.zeros(G, n, 2 * ld, dtype=torch.uint8, device=w.device)
    codes[:, :, :k] = q
    codes = codes[:, :, 0::2] | (codes[:, :, 1::2] << 4)
    return W4Weights(codes.contiguous(), scales.contiguous(), z.to(torch.uint8).contiguous() if zeros else None,
                     TYPE_CODES[scale_dtype], group)


def w4_values(w: W4Weights, k: int) -> torch.Tensor:
    """The float32 values [experts][n][k] that 4-bit weights stand for."""
    G, n, _ = w.codes.shape
    q = torch.stack((w.codes & 15, w.codes >> 4), -1).view(G, n, -1)[:, :, :k].float()
    wide = lambda t: t.float().repeat_interleave(w.desc.group, -1)[:, :, :k]  # noqa: E731
    return (q - (8.0 if w.zeros is None else wide(w.zeros))) * wide(w.scales)
