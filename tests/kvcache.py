"""The int8 paged cache, modelled from its documented layout: a page and head
are page / 16 tiles of 32 D + 128 bytes, K codes [D/16][16 tokens][16], V codes
[D/64][4][64][4 tokens], K scales [16], V scales [16]."""
import torch


def unpack(cache, D):
    """Codes int8 [slots, heads, D] and scales fp32 [slots, heads] of keys and of values."""
    pages, H, size = cache.shape
    tiles = cache.reshape(pages, H, -1, 32 * D + 128)
    n = tiles.shape[2]
    assert size == n * (32 * D + 128)
    part = lambda a, b: tiles[..., a:b].contiguous()
    k = part(0, 16 * D).view(torch.int8).reshape(pages, H, n, D // 16, 16, 16).permute(0, 2, 4, 1, 3, 5)
    v = part(16 * D, 32 * D).view(torch.int8).reshape(pages, H, n, D // 64, 4, 64, 4).permute(0, 2, 4, 6, 1, 3, 5)
    ks, vs = (part(32 * D + o, 32 * D + o + 64).view(torch.float32).reshape(pages, H, n, 16).permute(0, 2, 3, 1)
              for o in (0, 64))
    S = pages * n * 16
    return (k.reshape(S, H, D), ks.reshape(S, H)), (v.reshape(S, H, D), vs.reshape(S, H))


def quantize_rows(x):
    """The row code in fp32: scale amax / 127, codes half away from zero."""
    x = x.float()
    finite = torch.isfinite(x).all(-1)
    amax = torch.where(finite, x.abs().amax(-1), torch.zeros(()))
    d = amax / torch.full_like(amax, 127.0)
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    inv = torch.where(torch.isinf(inv), torch.zeros_like(inv), inv)
    y = torch.where(finite[..., None], x, torch.zeros(())) * inv[..., None]
    t = torch.trunc(y)
    codes = (t + torch.sign(y) * ((y - t).abs() >= 0.5)).clamp(-127, 127).to(torch.int8)
    return codes, torch.where(finite, d, torch.full_like(d, float("nan")))
