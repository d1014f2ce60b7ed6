"""Plain 64-bit forms of the serving-step operators, from the caches' stored arrays."""
from __future__ import annotations

import torch

HALF = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def norm_rope64(x, w, pos, table, rot, inter, eps=1e-6):
    """[T][heads][128] -> float64, one head at a time as the formula has it."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y ** 2).mean(-1, keepdim=True) + eps) * w.double()
    if table is None:
        return y
    out = y.clone()
    cs = table.double()[pos.long()]
    for p in range(rot // 2):
        i, j = (2 * p, 2 * p + 1) if inter else (p, p + rot // 2)
        c, s = cs[:, p, 0][:, None], cs[:, p, 1][:, None]
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
    return out


def state(cache, b):
    """(block-0 length, blocks, buffer fill) of row b."""
    if hasattr(cache, "counters"):
        b0, nblk, nbuf, _ = cache.counters()
        return (int(b0[b]) if nblk[b] else 0), int(nblk[b]), int(nbuf[b])
    return cache.c.blk0_len, cache.n_blk, cache.n_buf


def dense64(cache, b):
    """Reconstruction [H][tokens][128] (float64) of row b: blocks, then the buffer. Also the sum of the
    magnitudes of its parts |(code - m) scale| + |zero + m scale| + |L Rf^T| with m = 2^(bits - 1), which
    is how the kernel puts codes together (what its roundings are relative to)."""
    c, A = cache.c, cache.arrays()
    H, g, bits = c.H, c.p.group_size, c.p.bits
    b0, nblk, nbuf = state(cache, b)
    n_b = c.p.buffer_len
    m = b0 + (nblk - 1) * n_b if nblk else 0
    dev = cache.mem.device
    tok = torch.arange(m, device=dev)
    ch = torch.arange(128, device=dev)
    paged = hasattr(cache, "counters")
    if paged:
        P = c.page_tokens
        table = torch.from_numpy(cache.counters()[3][b].astype("int64")).to(dev)
        pages = table[: -(-m // P)]
        assert (pages >= 0).all() and (pages < c.num_pages).all()

    def take(name, h):
        if paged:
            return A[name][pages, h].flatten(0, 1)[:m]
        return A[name][b * H + h, :m]

    outs, mags = [], []
    blk = torch.where(tok < b0, 0, 1 + (tok - b0).clamp_min(0) // n_b)
    for h in range(H):
        code = ((take("codes", h).long()[:, ch * bits // 32] >> (ch * bits % 32)) & (2 ** bits - 1)).double()
        if c.p.channel_groups:
            slot = torch.where(tok < b0, tok // g, -(-b0 // g) + (tok - b0).clamp_min(0) // g)
            meta = (A["meta"][b, h] if paged else A["meta"][b * H + h])[slot].double()
        else:
            meta = take("meta", h).double()[:, ch // g]
        d = code * meta[..., 0] + meta[..., 1]
        rf = (A["rfac"][b, h] if paged else A["rfac"][b * H + h]).double()
        lf = take("lfac", h).double()
        lr = torch.zeros_like(d)
        for j in range(c.r_max):
            used = torch.where(blk == 0, j < (c.blk0_rank if nblk else 0), j < c.p.buffer_rank)[:, None]
            lr = lr + torch.where(used, lf[:, j:j + 1] * rf[blk, :, j], 0.0)
        mid = meta[..., 1] + 2 ** (bits - 1) * meta[..., 0]
        x, mag = d + lr, (d - mid).abs() + mid.abs() + lr.abs()
        if c.k:
            oi, ov = take("oidx", h).long(), take("oval", h).double()
            x, mag = x.scatter(1, oi, ov), mag.scatter_add(1, oi, ov.abs())
        buf = (A["buf"][b, h] if paged else A["buf"][b * H + h])[:nbuf].double()
        outs.append(torch.cat((x, buf)))
        mags.append(torch.cat((mag, buf.abs())))
    return torch.stack(outs), torch.stack(mags)


def chunk_ref(kc, vc, rows, counts, q, kn, vn, tau, plen=None):
    """(out, bound) float64 [T][Hq][128]. The bound is the sum of what rounding to binary16 can do:
    scores, from keys and the low-rank product of a row (half a step of each part, twice where a part is
    rounded in two places), are off by at most ds = tau sum_c |q_c| mag_c * 4 u; weights then by a factor
    exp(2 ds) with the maximum's own error, their rounding u and the values' 2 u: all relative to
    sum_t p_t |V_t|. With binary32 caches u is that of a 128-term binary32 sum instead."""
    f32 = kc.dtype == torch.float32
    u = 2.0 ** -24 * 130 if f32 else 2.0 ** -11
    Hq, H = q.shape[1], kc.c.H
    hq = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    at = 0
    for b, n in zip(rows, counts):
        (K0, KM), (V0, VM) = dense64(kc, b), dense64(vc, b)
        base = K0.shape[1]
        b0 = state(kc, b)[0]
        for h in range(H):
            K, V, km, vm = K0[h], V0[h], KM[h], VM[h]
            if kn is not None:
                k1, v1 = kn[at:at + n, h].double(), vn[at:at + n, h].double()
                K, km = torch.cat((K, k1)), torch.cat((km, k1.abs()))
                V, vm = torch.cat((V, v1)), torch.cat((vm, v1.abs()))
            t = torch.arange(K.shape[0], device=q.device)
            for j in range(h * hq, (h + 1) * hq):
                qq = q[at:at + n, j].double()
                seen = t[None] < base + torch.arange(1, n + 1, device=q.device)[:, None]
                if plen is not None:
                    p = min(max(int(plen[b]), 0), b0)
                    seen = seen & ~((t >= p) & (t < b0))[None]
                S = (qq @ K.T * tau).masked_fill(~seen, -torch.inf)
                if S.shape[1] == 0:
                    continue
                m = S.amax(1, keepdim=True)
                p = torch.where(seen, torch.exp(S - torch.where(m.isinf(), 0.0, m)), 0.0)
                l = p.sum(1, keepdim=True)
                p = torch.where(l > 0, p / l, 0.0)
                ds = ((qq.abs() @ km.T) * abs(tau) * 4 * u).masked_fill(~seen, 0).amax(1, keepdim=True)
                out[at:at + n, j] = p @ torch.where(seen.any(0)[:, None], V, 0.0)
                bound[at:at + n, j] = (torch.expm1(2 * ds) + 6 * u) * (p @ torch.where(seen.any(0)[:, None], vm, 0.0))
        at += n
    return out, bound


def check_chunk(got, ref, bound, dt, what=""):
    """Elementwise within the bound and the output's own half step; and, as roundings of independent terms
    do not add up all one way, within a small part of it in the mean square."""
    err = (got.double() - ref).abs()
    tol = bound + HALF[dt] * ref.abs() * (1 + 1e-6) + 1e-7 * bound.amax().clamp_min(1e-30)
    assert not torch.isnan(got).any(), f"{what}: NaN"
    bad = err > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, worst {float((err - tol).max()):.3e}, first {bad.nonzero()[0]}"
    if ref.numel() >= 4096 and ref.norm() > 0:
        rel = float(err.norm() / ref.norm())
        lim = max(1e-5, float(HALF[dt]) + 0.25 * float(bound.norm() / ref.norm()))
        assert rel <= lim, f"{what}: {rel:.2e} of the result's norm off, at most {lim:.2e}"


def chunk_spread(kc, vc, rows, counts, q, kn, vn, tau, plen=None):
    """(out, sigma), float64 [T][Hq][128] and [T][Hq]: the result, and the root mean square that the norm of a
    row's error can have when its roundings are independent. A rounding to binary16 is at most 2^-11 of the
    value off, d = 2^-11 / sqrt(3) in the root mean square. A key's or value's channel takes four of them at
    most, each of no more than the sum `mag` of its parts (the scale's and the middle value's product, their
    sum, a further one for a flushed block's low-rank part or an outlier's): its variance is below
    (2 d mag)^2; fp16 caches' values, which no power of two of their own scales, are held halved in binary16,
    whose step below 2^-14 is 2^-24: half of it, doubled again, is 2^-24 each time, with the variance 4 (2^-24)^2 / 3. So a score's is (2 d tau)^2 sum_c q_c^2 mag_c^2 =: e_t^2, which
    moves the result by p_t e_t (V_t - out); the weight's own rounding moves it by p_t d V_t. Sums over tokens
    add the squares."""
    d = 2.0 ** -11 / 3 ** 0.5
    if kc.dtype == torch.float32:
        d = 2.0 ** -24 * 128 ** 0.5   # a sum of 128 terms
    tiny = 2.0 ** -24 / 3 ** 0.5 / d if kc.dtype == torch.float16 else 0.0   # beside mag
    Hq, H = q.shape[1], kc.c.H
    hq = Hq // H
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    var = torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    at = 0
    for b, n in zip(rows, counts):
        if n == 0:
            continue
        (K, KM), (V, VM) = dense64(kc, b), dense64(vc, b)
        base, b0 = K.shape[1], state(kc, b)[0]
        if kn is not None:
            k1, v1 = kn[at:at + n].double().transpose(0, 1), vn[at:at + n].double().transpose(0, 1)
            K, KM, V, VM = (torch.cat(x, 1) for x in ((K, k1), (KM, k1.abs()), (V, v1), (VM, v1.abs())))
        t = torch.arange(K.shape[1], device=q.device)
        seen = t[None] < base + torch.arange(1, n + 1, device=q.device)[:, None]
        if plen is not None:
            p = min(max(int(plen[b]), 0), b0)
            seen = seen & ~((t >= p) & (t < b0))[None]
        live = seen.any(0)[:, None]
        if K.shape[1] == 0:
            at += n
            continue
        mask = seen.repeat_interleave(hq, 0)   # row (token, query head of the group)
        for h in range(H):
            k, km, v, vm = (torch.where(live, x[h], 0.0) for x in (K, KM, V, VM))
            qq = q[at:at + n, h * hq:(h + 1) * hq].double().reshape(n * hq, 128)
            S = (qq @ k.T * tau).masked_fill(~mask, -torch.inf)
            m = S.amax(1, keepdim=True)
            w = torch.where(mask, torch.exp(S - torch.where(m.isinf(), 0.0, m)), 0.0)
            l = w.sum(1, keepdim=True)
            w = torch.where(l > 0, w / l, 0.0)
            o = w @ v
            km2, vm2 = (torch.where(live, x.square() + tiny * tiny, 0.0) for x in (km, vm))
            e2 = (2 * d * tau) ** 2 * (qq.square() @ km2.T)
            far = (v.square().sum(1)[None] - 2 * o @ v.T + o.square().sum(1, keepdim=True)).clamp_min(0)
            s2 = (w.square() * (e2 * far + d * d * (v.square() + 4 * vm2).sum(1)[None])).sum(1)
            out[at:at + n, h * hq:(h + 1) * hq] = o.view(n, hq, 128)
            var[at:at + n, h * hq:(h + 1) * hq] = s2.view(n, hq)
        at += n
    return out, var.sqrt()


def check_spread(got, ref, sigma, dt, what=""):
    """Each row's error within 5 sigma of its norm (a row that one token dominates is nearly a single rounding,
    at most sqrt(3) times its root mean square; the others are sums of many), all rows' together within twice
    theirs, beside the output's own rounding, at most half a step of every element."""
    assert not torch.isnan(got).any(), f"{what}: NaN"
    err, size = (got.double() - ref).norm(dim=-1), HALF[dt] * ref.norm(dim=-1)
    if dt == torch.float16:
        size = size + 2.0 ** -25 * 128 ** 0.5   # results below 2^-14
    floor = 1e-6 * ref.norm(dim=-1)             # binary32 sums of the result
    bad = err > 5 * sigma + size + floor
    worst = float((err / (5 * sigma + size + floor).clamp_min(1e-300)).max()) if err.numel() else 0.0
    assert not bad.any(), f"{what}: {int(bad.sum())} rows off, {worst:.2f} times the limit, first {bad.nonzero()[0].tolist()}"
    both = float(err.norm()), float(2 * sigma.norm() + size.norm() + floor.norm())
    assert both[0] <= both[1], f"{what}: {both[0]:.3e} off in all, at most {both[1]:.3e}"
