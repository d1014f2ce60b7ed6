"""What the limit on chunk attention's error lets pass, on the CPU: a plain restatement of the tensor-core kernels'
roundings stays within it, and every planted mistake is outside."""
import math
from types import SimpleNamespace

import pytest
import torch

from tests.serving_helpers import check_spread, chunk_spread

TAU = 1 / math.sqrt(128)
F32 = torch.float32


class StoredCache:
    """A contiguous cache's stored arrays, made on the CPU: B rows of H heads, n tokens each, and a buffer."""

    def __init__(self, x, buf, bits, g, k, rank):
        U, n, _ = x.shape
        self.dtype, self.mem, self.n_blk, self.n_buf = torch.float16, torch.empty(0), 1, buf.shape[1]
        p = SimpleNamespace(group_size=g, bits=bits, buffer_len=20, buffer_rank=2, channel_groups=0)
        self.c = SimpleNamespace(H=2, p=p, k=k, r_max=rank, blk0_rank=rank, blk0_len=n)
        f = x.double()
        oi = f.abs().topk(k, dim=2).indices.sort(dim=2).values
        keep = torch.ones_like(f, dtype=torch.bool).scatter(2, oi, False)
        grp, kg = f.view(U, n, -1, g), keep.view(U, n, -1, g)
        zero = grp.masked_fill(~kg, math.inf).amin(3).float()
        scale = ((grp.masked_fill(~kg, -math.inf).amax(3) - zero) / (2 ** bits - 1)).float()
        code = ((grp - zero[..., None]) / scale[..., None]).round().clamp(0, 2 ** bits - 1).masked_fill(~kg, 0).long()
        res = (grp - code * scale[..., None].double() - zero[..., None].double()).masked_fill(~kg, 0).view(U, n, 128)
        u, s, vt = torch.linalg.svd(res, full_matrices=False)
        e = 2.0 ** (int(math.log2(n)) // 2)
        words = (code.view(U, n, -1, 32 // bits) << (torch.arange(32 // bits) * bits)).sum(3)
        self.a = dict(codes=words, meta=torch.stack((scale, zero), -1), oidx=oi.to(torch.uint8), oval=x.gather(2, oi),
                      lfac=(u[:, :, :rank] * e).half(), buf=buf,
                      rfac=(vt[:, :rank] * s[:, :rank, None] / e).float().transpose(1, 2)[:, None].contiguous())

    def arrays(self):
        return self.a


def half(x):
    return x.half().double()


def operands(cache, b, h, new):
    """(D, L, Rf) of a unit as the kernels have them: binary16 D with an outlier less its low-rank part, L of prompt
    tokens, Rf."""
    c, A, unit = cache.c, cache.arrays(), b * cache.c.H + h
    bits, g = c.p.bits, c.p.group_size
    ch = torch.arange(128)
    code = (A["codes"][unit][:, ch * bits // 32] >> (ch * bits % 32)) & (2 ** bits - 1)
    meta = A["meta"][unit][:, ch // g].double()
    m = 2 ** (bits - 1)
    d = half((code - m) * half(meta[..., 0]) + half(meta[..., 1] + m * meta[..., 0]))
    L, rf = A["lfac"][unit].double(), A["rfac"][unit, 0].double()
    oi = A["oidx"][unit].long()
    d.scatter_(1, oi, half(A["oval"][unit].double() - (L @ rf.T).gather(1, oi)))
    raw = torch.cat((A["buf"][unit], new)).double()
    return torch.cat((d, raw)), torch.cat((L, torch.zeros(raw.shape[0], L.shape[1], dtype=L.dtype))), rf


def restated(kc, vc, counts, q, kn, vn, mistake=None):
    out = torch.zeros(q.shape, dtype=torch.float64)
    H, at = kc.c.H, 0
    hq = q.shape[1] // H
    for b, n in enumerate(counts):
        for h in range(H):
            DK, LK, RK = operands(kc, b, h, kn[at:at + n, h])
            DV, LV, RV = operands(vc, b, h, vn[at:at + n, h])
            other = operands(kc, (b + 1) % len(counts), h, kn[:0, h])[2]
            base = DK.shape[0] - n
            qq = q[at:at + n, h * hq:(h + 1) * hq].double().reshape(n * hq, 128)
            low = half(qq @ RK) @ LK.T
            if mistake == "no low-rank part of keys":
                low = low * 0
            if mistake == "another row's Rf":
                low = half(qq @ other) @ LK.T
            if mistake == "another row's Rf in odd tiles":
                odd = (torch.arange(DK.shape[0]) // 96 % 2 == 1)[None]
                low = torch.where(odd, half(qq @ other) @ LK.T, low)
            S = (qq @ DK.T + low) * TAU
            seen = torch.arange(DK.shape[0])[None] < base + 1 + torch.arange(n).repeat_interleave(hq)[:, None]
            if mistake == "own token left out":
                seen = seen & (torch.arange(DK.shape[0])[None] < base + torch.arange(n).repeat_interleave(hq)[:, None])
            S = S.masked_fill(~seen, -math.inf)
            w = torch.exp(S - S.amax(1, keepdim=True)) * 128
            p = half(w)
            pv = p @ LV @ RV.T * (mistake != "no low-rank part of values")
            if mistake == "a tile left out":
                p[:, 96:192] = 0
            o = (p @ DV + pv) / w.sum(1, keepdim=True)
            if mistake == "nothing":
                o = o * 0
            if mistake == "the buffer's first token twice":
                o = (p @ DV + pv + p[:, base - 3:base - 2] * DV[base - 3]) / (w.sum(1, keepdim=True) + w[:, base - 3:base - 2])
            out[at:at + n, h * hq:(h + 1) * hq] = o.view(n, hq, 128)
        at += n
    return out.float()


CODECS = [dict(bits=4, g=64, k=3, rank=4), dict(bits=2, g=32, k=7, rank=8), dict(bits=8, g=128, k=3, rank=2)]
# (an eight-bit code's residual is below a rounding to binary16: its low-rank part cannot be missed)
LOW_RANK = ["no low-rank part of keys", "another row's Rf", "another row's Rf in odd tiles", "no low-rank part of values"]
MISTAKES = ["nothing", "own token left out", "a tile left out", "the buffer's first token twice"]


@pytest.mark.parametrize("n", [300, 4000])
@pytest.mark.parametrize("codec", CODECS)
def test_the_limit_passes_roundings_and_no_mistake(codec, n):
    g = torch.Generator().manual_seed(n)
    sig = torch.exp(torch.rand(128, generator=g) * math.log(4) + math.log(0.5))

    def rnd(*shape):
        return torch.randn(*shape, generator=g)

    x = lambda *shape: (rnd(*shape, 128) * sig).half()
    kc, vc = (StoredCache(x(4, n), x(4, 3), **codec) for _ in range(2))
    counts = [2, 5]
    q, kn, vn = rnd(7, 4, 128).half(), x(7, 2), x(7, 2)
    ref, sigma = chunk_spread(kc, vc, [0, 1], counts, q, kn, vn, TAU)
    check_spread(restated(kc, vc, counts, q, kn, vn), ref, sigma, F32)
    got16 = restated(kc, vc, counts, q, kn, vn).half()
    check_spread(got16, ref, sigma, torch.float16)
    assert (sigma.norm() / ref.norm() < 3e-3).all()   # the limit is a few thousandths of the result
    for m in MISTAKES + (LOW_RANK if codec["bits"] < 8 else []):
        with pytest.raises(AssertionError):
            check_spread(restated(kc, vc, counts, q, kn, vn, m), ref, sigma, F32, m)
