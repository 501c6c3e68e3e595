"""4-bit weights in plain torch: the values that codes and scales stand for, and the
quantiser, in 64 bits."""

import torch


def values(q, scale, group):
    """(code - 8) * scale in 64 bits, of q [..., K/2] bytes and scale [..., ceil(K/group)]."""
    codes = torch.stack([q & 15, q >> 4], -1).flatten(-2).double() - 8.0
    s = scale.double().repeat_interleave(group, -1)[..., :codes.shape[-1]]
    return codes * s


def pack(codes):
    """Codes [..., K] in 0..15 to bytes, the even column's in the low half."""
    c = codes.to(torch.uint8)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).contiguous()


def quantize(w, group):
    """(codes [rows, K], scales in w's type) of w [rows, K] by the definition, in 64 bits."""
    rows, K = w.shape
    G = -(-K // group)
    p = torch.nn.functional.pad(w.double(), (0, G * group - K)).view(rows, G, group)
    scale = (p.abs().amax(2) / 7.0).to(w.dtype)
    s = scale.double()[:, :, None]
    fine = torch.isfinite(s) & (s > 0)
    k = torch.where(fine, torch.round(p / torch.where(fine, s, torch.ones_like(s))),
                    torch.zeros_like(p))
    return (k.clamp(-8, 7) + 8).view(rows, -1)[:, :K], scale
