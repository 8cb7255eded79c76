"""Plain references in 64 bits for the attention-path operators, and the error
that a right kernel may have.

The bounds count roundings: u = 2^-24 is half a step of fp32, and a result
rounded to type t is off by at most finfo(t).eps / 2 of its value (plus half
the smallest subnormal)."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def phases(table, positions):
    """Angles of [T, pairs] in fp64 from the table's 64-bit fractions, with
    exact integer arithmetic."""
    turns = [t % 2 ** 64 for t in table.turns.tolist()]
    axis = table.axis.tolist()
    pos = positions.reshape(-1, positions.shape[-1]).tolist()
    rows = [[((pos[a][t] * f + 2 ** 63) % 2 ** 64 - 2 ** 63) / 2.0 ** 63 * math.pi
             for a, f in zip(axis, turns)] for t in range(positions.shape[-1])]
    return torch.tensor(rows, dtype=torch.float64).reshape(positions.shape[-1], len(turns))


def rope(x, w, table, positions, head_dim, eps, woff, interleaved):
    """(out, bound) in fp64 for x [T, H * D] (CPU)."""
    T = x.shape[0]
    y = x.double().reshape(T, -1, head_dim)
    rel = 0.0
    if eps is not None:
        wt = torch.ones(head_dim, dtype=torch.float64) if w is None else w.double()
        y = (wt + woff) * y / torch.sqrt((y * y).sum(-1, keepdim=True) / head_dim + float(
            torch.tensor(eps, dtype=torch.float32)))
        # the sum's tree (at most head_dim / 32 terms a lane, 5 levels), the
        # mean, the root, the weight's sum and two products
        rel = (head_dim / 32 + 16) * U
    P = table.rot_dim // 2
    ang = phases(table, positions)[:, None]
    c, s = ang.cos(), ang.sin()
    i = torch.arange(P) * 2 if interleaved else torch.arange(P)
    j = i + 1 if interleaved else i + P
    out, bound = y.clone(), y.abs() * rel
    a, b = y[..., i], y[..., j]
    out[..., i], out[..., j] = a * c - b * s, b * c + a * s
    # the phase rounded to fp32 (pi 2^-25), sin and cos off by 2 ulp, three roundings
    err = torch.hypot(a, b) * (rel + 2.0 ** -22 + 4 * U) * 1.5
    bound[..., i], bound[..., j] = err, err
    dt = x.dtype
    bound = bound + HALF[dt] * (out.abs() + bound) + TINY[dt]
    return out.reshape(x.shape), bound.reshape(x.shape)


def e4m3(codes):
    return codes.view(torch.float8_e4m3fn).double()


def half_step(v):
    """Half a step of E4M3 at v: 2^(e - 4) in binade e >= -6."""
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6)))
    return torch.exp2(e - 4)


def append(cache, x, side, table, lengths, cu):
    """The quotients that the codes round, the scales, and which rows change:
    (value, scale, touched) for side "k" or "v" on the CPU.  ``cache``: the
    tensors before, ``x`` [T, H, D]."""
    codes, scale = cache[side].cpu(), cache[side + "_scale"].cpu().double().clone()
    value = e4m3(codes)
    touched = torch.zeros(codes.shape[:3], dtype=torch.bool)
    pages, _, page, _ = codes.shape
    x = x.cpu().double()
    for b, old in enumerate(lengths.tolist()):
        c0, c1 = (b, b + 1) if cu is None else (int(cu[b]), int(cu[b + 1]))
        if old < 0:
            continue
        pos, end = old, old + c1 - c0
        while pos < end:
            stop = min(end, (pos // 16 + 1) * 16)
            slot = pos // page
            pg = int(table[b][slot]) if slot < table.shape[1] else -1
            if 0 <= pg < pages:
                new = x[c0 + pos - old:c0 + stop - old].transpose(0, 1)
                a = torch.nan_to_num(new.abs(), nan=0.0, posinf=3.4028234663852886e38)
                blk, lo = pos % page // 16, pos // 16 * 16 % page
                at = a.amax((1, 2)) / 448
                before = scale[pg, :, blk] if pos % 16 else torch.zeros_like(at)
                after = torch.maximum(at, before)
                after = torch.where((after > 0) & (after < 2.0 ** -126),
                                    torch.full_like(after, 2.0 ** -126), after)
                safe = torch.where(after > 0, after, torch.ones_like(after))[:, None, None]
                k = pos % 16
                grown = (after > before)[:, None, None]
                old_rows = value[pg, :, lo:lo + k]
                value[pg, :, lo:lo + k] = torch.where(
                    grown, old_rows * (before[:, None, None] / safe), old_rows)
                touched[pg, :, lo:lo + k] |= grown[..., 0]
                value[pg, :, lo + k:lo + k + stop - pos] = new / safe
                touched[pg, :, lo + k:lo + k + stop - pos] = True
                scale[pg, :, blk] = after
            pos = stop
    return value, scale, touched


def check_append(before, after, x, side, table, lengths, cu):
    """The cache after an append against the definition: untouched codes and
    scales bit for bit, scales to an fp32 rounding, codes the nearest (to
    within three fp32 roundings of the quotient)."""
    value, scale, touched = append(before, x, side, table, lengths, cu)
    got, was = after[side].cpu(), before[side].cpu()
    assert torch.equal(got[~touched], was[~touched]), "a row that was not appended to changed"
    gs = after[side + "_scale"].cpu().double()
    same = (gs == scale) | (gs.isnan() & scale.isnan())
    assert bool((same | ((gs - scale).abs() <= 1.01 * U * scale)).all()), "scales"
    have, want = e4m3(got[touched]), value[touched]
    nan = want.isnan()
    assert torch.equal(have.isnan(), nan), "NaN codes"
    want = want.clamp(-448, 448)
    off = (have - want).abs()
    room = half_step(want) * (1 + 8 * U) + 4 * U * want.abs()
    assert bool((off <= room)[~nan].all()), f"codes: {float((off / room)[~nan].max())} of the room"


def attend(q, cache, table, lengths, scale, window, sinks):
    """(out, bound) in fp64 for q [B, n, Hq, D] on q's device."""
    B, n, Hq, D = q.shape
    kc, vc = cache["k"], cache["v"]
    pages, Hk, page, _ = kc.shape
    G = Hq // Hk
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, L in enumerate(lengths.tolist()):
        room = table.shape[1] * page
        j = torch.arange(max(0, min(L, room)), device=q.device)
        if not j.numel():
            continue
        pg = table[b].long()[j // page]
        good = (pg >= 0) & (pg < pages)
        pg = pg.clamp(0, max(0, pages - 1))
        k = e4m3(kc[pg, :, j % page].contiguous()) * cache["k_scale"][pg, :, j % page // 16].double()[..., None]
        code = e4m3(vc[pg, :, j % page].contiguous())
        vs = cache["v_scale"][pg, :, j % page // 16].double()
        v = code * vs[..., None]
        for i in range(n):
            pos = L - n + i
            seen = good & (j <= pos)
            if window:
                seen &= (j > pos - window) | (j < sinks)
            if not bool(seen.any()):
                continue
            for h in range(Hk):
                qq = q[b, i, h * G:(h + 1) * G].double()
                kk, vv = k[seen, h], v[seen, h]
                s = qq @ kk.T * scale
                p = torch.softmax(s, -1)
                o = p @ vv
                # a score: D products summed in fp32 (a tensor-core sum may
                # truncate: 2 u a term), three products and the difference
                # from the maximum; a weight: that, exp2's two ulp, the rounding
                # to fp16 (half a step: 2^-11); a sum: one rounding for every 16 tokens
                # and the joins
                ds = float((qq.abs() @ kk.abs().T).max()) * abs(scale) * (2 * D + 8) * U + float(
                    s.abs().max()) * 4 * U
                rel = 2.0 ** -11 + 2 * (ds + 4 * U) + (2 * vv.shape[0] / 16 + 64) * 2 * U
                # fp16 rounds a weight below its normal range by 2^-25 at most,
                # in units of 2^-8 of the row's reference (which is no more
                # than the largest weight, so than the weights' sum) times the
                # row's largest value scale
                lost = 2.0 ** -33 * vs[good, h].nan_to_num(0, 0, 0).max() * code[seen, h].abs().sum(0)
                out[b, i, h * G:(h + 1) * G] = o
                bound[b, i, h * G:(h + 1) * G] = rel * (p @ vv.abs()) + lost
    dt = q.dtype
    bound = bound + HALF[dt] * (out.abs() + bound) + TINY[dt]
    return out, bound


def random_cache(pages, H, page, D, seed, device, spread=True):
    """Codes and scales of full blocks of random values (scales spread over
    some binades), on the device."""
    g = torch.Generator().manual_seed(seed)
    c = {}
    for side in ("k", "v"):
        x = torch.randn((pages, H, page // 16, 16 * D), generator=g)
        if spread:
            x = x * torch.exp2(2 * torch.randn((pages, H, page // 16, 1), generator=g))
        s = x.abs().amax(-1) / 448
        codes = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        c[side] = codes.view(torch.uint8).reshape(pages, H, page, D).to(device)
        c[side + "_scale"] = s.to(device)
    return c


def tables(B, width, pages, seed, device):
    g = torch.Generator().manual_seed(seed)
    return torch.randperm(pages, generator=g)[:B * width].to(torch.int32).reshape(B, width).to(device)
