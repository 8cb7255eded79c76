"""The attention path's operators, in plain torch and as the package's kernels.

Three operators of a transformer layer between its qkv projection and its
output projection:

  rope     per-head RMS norm of the query and key heads (optional) and rotary
           positions with one to three axes (time, height, width)
  append   new keys and values into a paged cache held in E4M3 codes, with one
           fp32 scale for every block of 16 tokens and head
  attend   attention of one or a few query tokens per sequence over that
           cache, with an optional sliding window and first tokens (sinks)
           that stay visible

Definitions (x: a head of D elements):

  rope     y = (w + w_offset) x / sqrt(mean(x^2) + eps)    (or y = x)
           pair p of R / 2, at elements (p, p + R/2) or (2p, 2p + 1), is turned
           by the angle position[axis(p)] * f(p); elements from R on stay
  append   per block and head: s = max(s before, max|x| / 448) (s before is 0
           where the block's first token is among the new ones); codes
           E4M3(x / s); older codes of the block are re-encoded if s grew
  attend   softmax(scale q k) v over the tokens j <= i with j > i - window or
           j < sinks, for the query at position i; no visible token gives 0
"""
import math

import torch

own = False

BLOCK = 16  # tokens that share a scale
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FMAX = 3.4028234663852886e38
EPS = 1e-6


def listed():
    rope = {"op": "rope", "norm": True, "interleaved": False, "fused": True, "dtype": "bf16"}
    append = {"op": "append", "page": 64, "dtype": "bf16"}
    attend = {"op": "attend", "page": 64, "n": 1, "window": 0, "sinks": 0, "dtype": "bf16"}
    return [
        # a decode step of a few sequences, far into long contexts
        {**rope, "name": "rope_decode_8", "T": 8, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "axes": 1, "far": 1000000},
        # a prefill of video tokens, three axes, inside the fused qkv rows
        {**rope, "name": "rope_video_16384", "T": 16384, "Hq": 32, "Hk": 8, "D": 128, "R": 128, "axes": 3, "far": 20000},
        # image tokens: no norm, neighbouring pairs, half of each head turned, an odd count
        {**rope, "name": "rope_image_4099", "T": 4099, "Hq": 16, "Hk": 16, "D": 64, "R": 32, "axes": 2, "far": 128,
         "norm": False, "interleaved": True, "fused": False, "dtype": "f16"},
        # one decode step of a busy server: one token to each of many sequences
        {**append, "name": "append_decode_64", "B": 64, "new": 1, "old": 8000, "H": 8, "D": 128},
        # chunks of several prompts, some of them behind an earlier chunk
        {**append, "name": "append_prefill_16x2000", "B": 16, "new": 2000, "old": 1000, "H": 8, "D": 128},
        # short ragged pieces into small pages, small heads
        {**append, "name": "append_ragged_37x21", "B": 37, "new": 21, "old": 300, "H": 2, "D": 64, "page": 16, "dtype": "f16"},
        # one sequence, a short context: latency
        {**attend, "name": "attend_1x1000", "B": 1, "L": 1000, "Hq": 32, "Hk": 8, "D": 128},
        # a decode step of a busy server over long contexts
        {**attend, "name": "attend_64x8192", "B": 64, "L": 8192, "Hq": 32, "Hk": 8, "D": 128},
        # one very long context
        {**attend, "name": "attend_1x131072", "B": 1, "L": 131072, "Hq": 32, "Hk": 8, "D": 128},
        # long contexts of which a window and the first tokens are seen
        {**attend, "name": "attend_32x65536_w4096", "B": 32, "L": 65536, "Hq": 64, "Hk": 8, "D": 64, "window": 4096, "sinks": 4, "dtype": "f16"},
        # four drafted tokens a sequence are verified at once
        {**attend, "name": "attend_48x2000_n4", "B": 48, "L": 2000, "Hq": 32, "Hk": 8, "D": 128, "n": 4, "page": 16},
        # wide heads, many query heads to a key head
        {**attend, "name": "attend_9x5000_d256", "B": 9, "L": 5000, "Hq": 16, "Hk": 1, "D": 256, "page": 32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    if op == "rope":
        D = rng.choice([64, 96, 128, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        most = 16384 * 40 * 128 * 2 // ((Hq + Hk) * D * (4 if dtype == "f32" else 2))
        axes = rng.choice([1, 2, 3])
        return {"op": op, "T": _log(rng, 1, min(20000, most)), "Hq": Hq, "Hk": Hk, "D": D, "R": rng.choice([D, D, D // 2]), "axes": axes,
                "far": _log(rng, 100, 1000000), "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.4, "fused": rng.random() < 0.6, "dtype": dtype}
    if op == "append":
        H, D = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        new = rng.choice([1, 1, _log(rng, 2, 3000)])
        most = 16 * 2000 * 8 * 128 // (H * D * new)
        old = _log(rng, 1, 8000)
        return {"op": op, "B": _log(rng, 1, max(1, min(256, most, 260000 * 1024 // ((old + new) * H * D)))), "new": new, "old": old, "H": H, "D": D, "page": rng.choice([16, 32, 64, 128]),
                "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    D = rng.choice([64, 128, 128, 256])
    Hk = rng.choice([1, 2, 4, 8])
    L = _log(rng, 1, 131072)
    most = 64 * 8192 * 8 * 128 // (2 * L * Hk * D)
    window = rng.choice([0, 0, _log(rng, 16, 5000)])
    return {"op": op, "B": _log(rng, 1, max(1, min(128, most))), "L": L, "Hq": Hk * rng.choice([1, 2, 4, 7, 8]), "Hk": Hk, "D": D, "n": rng.choice([1, 1, 1, 2, 3, 5]),
            "window": window, "sinks": rng.choice([0, 4, 20]) if window else 0, "page": rng.choice([16, 32, 64, 128]), "dtype": rng.choice(["bf16", "bf16", "f16"])}


# ---------------------------------------------------------------- inputs


def _sections(pairs, axes):
    """A quarter of the pairs for time, the rest shared by height and width."""
    if axes == 1:
        return [pairs]
    if axes == 2:
        return [pairs // 2, pairs - pairs // 2]
    first = pairs // 4
    second = (pairs - first) // 2
    return [first, second, pairs - first - second]


def _frequencies(R, sections):
    """The angle a step of the position turns each pair by (fp64), and the pair's axis."""
    pairs = R // 2
    f = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    axis = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections))
    return f, axis


def _pages(g, count, dev):
    """`count` different pages in an order of no meaning, as a server hands them out."""
    return torch.randperm(count, generator=g, device=dev).to(torch.int32)


def _table(g, B, need, page, dev):
    """Block table [B, width] of random pages for `need` tokens a sequence, and the number of pages."""
    width = -(-need // page)
    return _pages(g, B * width + 1, dev)[: B * width].reshape(B, width).contiguous(), B * width + 1


def _filled(g, pages, H, page, D, dev):
    """Codes and scales of a cache of which every block holds 16 random tokens."""
    codes = torch.empty((pages, H, page, D), dtype=torch.uint8, device=dev)
    scale = torch.empty((pages, H, page // BLOCK), dtype=torch.float32, device=dev)
    step = max(1, (1 << 27) // (H * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn((n, H, page // BLOCK, BLOCK * D), generator=g, device=dev)
        s = x.abs().amax(-1) * (1.0 / 448)
        scale[p:p + n] = s
        codes[p:p + n] = (x / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, H, page, D)
    return codes, scale


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "rope":
        T, Hq, Hk, D = case["T"], case["Hq"], case["Hk"], case["D"]
        sections = _sections(case["R"] // 2, case["axes"])
        if case["fused"]:  # query, key and value heads of a token side by side
            row = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device=dev).to(dt)
            s["q"], s["k"] = row[:, :Hq * D], row[:, Hq * D:(Hq + Hk) * D]
        else:
            s["q"] = torch.randn((T, Hq * D), generator=g, device=dev).to(dt)
            s["k"] = torch.randn((T, Hk * D), generator=g, device=dev).to(dt)
        s["wq"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt) if case["norm"] else None
        s["wk"] = (1 + 0.1 * torch.randn(D, generator=g, device=dev)).to(dt) if case["norm"] else None
        s["positions"] = torch.randint(0, case["far"], (case["axes"], T), generator=g, device=dev, dtype=torch.int32)
        f, axis = _frequencies(case["R"], sections)
        s["f"], s["axis"] = f.to(dev), axis.to(dev)
        if own:
            import residual_add_rmsnorm_vec_gb300 as rn
            s["table"] = rn.rope_table(case["R"], base=10000.0, sections=sections, device=dev)
    elif case["op"] == "append":
        B, H, D, page = case["B"], case["H"], case["D"], case["page"]
        # ragged: each piece that is longer than the usual has one that is as much shorter
        half = torch.randint(0, case["new"] // 2 + 1, (B // 2,), generator=g, device=dev)
        n = case["new"] + torch.cat([half, -half, half.new_zeros(B % 2)])
        old = torch.randint(0, 2 * case["old"], (B,), generator=g, device=dev)
        T = B * case["new"]
        s["table"], pages = _table(g, B, 2 * case["old"] + case["new"] + case["new"] // 2, page, dev)
        s["lengths"] = old.to(torch.int32)
        s["cu"] = torch.cat([n.new_zeros(1), n.cumsum(0)]).to(torch.int32)
        row = torch.randn((T, 2 * H * D), generator=g, device=dev)
        row = (row * torch.exp2(torch.randn((T, 1), generator=g, device=dev))).to(dt)
        s["k"], s["v"] = row[:, :H * D].unflatten(1, (H, D)), row[:, H * D:].unflatten(1, (H, D))
        s["kc"], s["ks"] = _filled(g, pages, H, page, D, dev)
        s["vc"], s["vs"] = _filled(g, pages, H, page, D, dev)
    else:
        B, Hk, D, page, n = case["B"], case["Hk"], case["D"], case["page"], case["n"]
        low = max(n, case["L"] * 3 // 4)
        s["lengths"] = torch.randint(low, max(n, case["L"]) + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s["lengths"][0] = max(n, case["L"])
        s["table"], pages = _table(g, B, max(n, case["L"]), page, dev)
        s["q"] = torch.randn((B, n, case["Hq"], D), generator=g, device=dev).to(dt)
        s["kc"], s["ks"] = _filled(g, pages, Hk, page, D, dev)
        s["vc"], s["vs"] = _filled(g, pages, Hk, page, D, dev)
    if own and case["op"] != "rope":
        import residual_add_rmsnorm_vec_gb300 as rn
        s["cache"] = rn.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
    return s


# ---------------------------------------------------------------- plain forms


def _plain_heads(x, w, case, cos, sin):
    T, D, R = case["T"], case["D"], case["R"]
    y = x.reshape(T, -1, D).float()
    if case["norm"]:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    turned = y[..., :R].reshape(T, -1, R // 2, 2).transpose(-1, -2) if case["interleaved"] else y[..., :R].reshape(T, -1, 2, R // 2)
    a, b = turned[..., 0, :], turned[..., 1, :]
    c, s = cos[:, None], sin[:, None]
    out = torch.stack([a * c - b * s, a * s + b * c], -1 if case["interleaved"] else -2).reshape(T, -1, R)
    return torch.cat([out, y[..., R:]], -1).to(x.dtype).reshape(x.shape)


def _plain_rope(s):
    case = s["case"]
    angle = s["positions"][s["axis"]].double().T * s["f"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    return [_plain_heads(s["q"], s["wq"], case, cos, sin), _plain_heads(s["k"], s["wk"], case, cos, sin)]


def _plain_append(x, codes, scale, s):
    page = s["case"]["page"]
    T, H, D = x.shape
    token = torch.arange(T, device=x.device)
    seq = torch.bucketize(token, s["cu"][1:], right=True)
    pos = s["lengths"][seq] + (token - s["cu"][seq])
    pg, off = s["table"][seq, pos // page].long(), pos % page
    blk = off // BLOCK
    h = torch.arange(H, device=x.device)
    y = x.float()
    # scales: of the block before (0 where its first token is new), and the new tokens' own
    cell = ((pg[:, None] * H + h) * (page // BLOCK) + blk[:, None]).reshape(-1)
    first = (pos - pos % BLOCK >= s["lengths"][seq])[:, None].expand(T, H).reshape(-1)
    flat = scale.reshape(-1)
    before = flat[cell].where(~first, torch.zeros_like(flat[cell]))
    flat[cell] = torch.zeros_like(before)
    flat.scatter_reduce_(0, cell, before, "amax")
    start = flat.clone()
    flat.scatter_reduce_(0, cell, (y.abs().clamp(max=FMAX).amax(-1) / 448).reshape(-1), "amax")
    back = torch.where(flat > 0, 1 / flat, torch.zeros_like(flat))
    # the first block of each sequence may hold older tokens: their codes follow the scale
    at = s["lengths"]
    has = s["cu"][1:] > s["cu"][:-1]
    pb = s["table"][torch.arange(at.numel(), device=x.device), (at // page).clamp(max=s["table"].shape[1] - 1)].long()
    bb = at % page // BLOCK
    rows = (bb[:, None] * BLOCK + torch.arange(BLOCK, device=x.device)).long()
    cells = (pb[:, None] * H + h) * (page // BLOCK) + bb[:, None]
    ratio = (start[cells] * back[cells])[:, :, None, None]
    was = codes[pb[:, None, None], h[:, None], rows[:, None, :]]
    now = (was.view(torch.float8_e4m3fn).float() * ratio).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    keep = (has[:, None] & (torch.arange(BLOCK, device=x.device) < (at % BLOCK)[:, None]))[:, None, :, None]
    codes[pb[:, None, None], h[:, None], rows[:, None, :]] = torch.where(keep, now, was)
    # the new tokens
    code = (y * back[cell].reshape(T, H, 1)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[pg[:, None], h, off[:, None].long()] = code


def _plain_attend(s):
    case = s["case"]
    B, n, Hq, D = s["q"].shape
    Hk, page, width = case["Hk"], case["page"], s["table"].shape[1]
    L = width * page
    t = s["table"].long()

    def values(codes, scale):
        x = codes[t].view(torch.float8_e4m3fn).float()  # [B, width, Hk, page, D]
        x = x.unflatten(3, (page // BLOCK, BLOCK)) * scale[t][..., None, None]
        return x.flatten(3, 4).transpose(1, 2).reshape(B, Hk, L, D)

    q = s["q"].float().reshape(B, n, Hk, Hq // Hk, D).transpose(1, 2).reshape(B, Hk, -1, D)
    scores = q @ values(s["kc"], s["ks"]).transpose(-1, -2) * (1 / math.sqrt(D))
    j = torch.arange(L, device=q.device)
    i = s["lengths"].long()[:, None] - n + torch.arange(n, device=q.device)  # position of each query
    seen = j <= i[..., None]
    if case["window"]:
        seen &= (j > i[..., None] - case["window"]) | (j < case["sinks"])
    seen = seen[:, None, :, None].expand(B, 1, n, Hq // Hk, L).reshape(B, 1, -1, L)
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - top)
    o = (p @ values(s["vc"], s["vs"])) / p.sum(-1, keepdim=True)
    return o.reshape(B, Hk, n, Hq // Hk, D).transpose(1, 2).reshape(B, n, Hq, D).to(s["q"].dtype)


def run(s):
    case = s["case"]
    if own:
        import residual_add_rmsnorm_vec_gb300 as rn
    if case["op"] == "rope":
        if own:
            return list(rn.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], s["wq"], s["wk"], head_dim=case["D"],
                                        eps=EPS if case["norm"] else None, interleaved=case["interleaved"]))
        return _plain_rope(s)
    if case["op"] == "append":
        if own:
            rn.kv_cache_append_(s["cache"], s["k"], s["v"], s["table"], s["lengths"], s["cu"])
        else:
            _plain_append(s["k"], s["kc"], s["ks"], s)
            _plain_append(s["v"], s["vc"], s["vs"], s)
        return {"k": s["kc"].view(torch.float8_e4m3fn), "v": s["vc"].view(torch.float8_e4m3fn), "k_scale": s["ks"], "v_scale": s["vs"]}
    if own:
        return rn.kv_cache_attention(s["q"], s["cache"], s["table"], s["lengths"], window=case["window"], sinks=case["sinks"])
    return _plain_attend(s)


# ---------------------------------------------------------------- cost and the definition in 64 bits


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "rope":
        heads = case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * heads * size + case["T"] * case["axes"] * 4, "flops": heads * 8}
    if case["op"] == "append":
        values = 2 * case["B"] * case["new"] * case["H"] * case["D"]
        return {"bytes": values * (size + 1) + values // (BLOCK * case["D"]) * 4, "flops": values * 3}
    n, B, L = case["n"], case["B"], max(case["n"], case["L"])
    mean = (max(n, case["L"] * 3 // 4) + L) / 2  # tokens of a sequence but the first, which has L
    first = L
    if case["window"]:
        most = case["window"] + case["sinks"] + n - 1
        first, mean = min(first, most), min(mean, most)
    seen = first + (B - 1) * mean
    return {"bytes": int(seen * case["Hk"] * 2 * (case["D"] + 4 / BLOCK) + 2 * B * n * case["Hq"] * case["D"] * size), "flops": int(4 * seen * n * case["Hq"] * case["D"])}


def _exact_heads(x, w, case, positions, axis):
    D, R = case["D"], case["R"]
    y = x.double().reshape(case["T"], -1, D)
    if case["norm"]:
        y = w.double() * y / torch.sqrt(y.square().sum(-1, keepdim=True) / D + EPS)
    out = y.clone()
    for p in range(R // 2):
        angle = positions[int(axis[p])].double() * math.pow(10000.0, -2.0 * p / R)
        i, j = (2 * p, 2 * p + 1) if case["interleaved"] else (p, p + R // 2)
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        out[..., i] = y[..., i] * c - y[..., j] * s
        out[..., j] = y[..., j] * c + y[..., i] * s
    return out.reshape(x.shape)


def _exact_append(x, codes, scale, s):
    """The cache after the append: codes as the quotients that they round."""
    page = s["case"]["page"]
    value = codes.view(torch.float8_e4m3fn).double()
    scale = scale.double().clone()
    lengths, cu, table = s["lengths"].tolist(), s["cu"].tolist(), s["table"].tolist()
    for b, old in enumerate(lengths):
        pos, end = old, old + cu[b + 1] - cu[b]
        while pos < end:  # block by block
            stop = min(end, (pos // BLOCK + 1) * BLOCK)
            new = x[cu[b] + pos - old:cu[b] + stop - old].double().transpose(0, 1)
            pg, blk, lo = table[b][pos // page], pos % page // BLOCK, pos // BLOCK * BLOCK % page
            at = new.abs().amax((1, 2)) / 448
            before = scale[pg, :, blk] if pos % BLOCK else torch.zeros_like(at)
            after = torch.maximum(at, before)
            value[pg, :, lo:lo + pos % BLOCK] *= (before / after)[:, None, None]
            value[pg, :, lo + pos % BLOCK:lo + pos % BLOCK + stop - pos] = new / after[:, None, None]
            scale[pg, :, blk] = after
            pos = stop
    return value, scale


def _exact_attend(s):
    case = s["case"]
    B, n, Hq, D = s["q"].shape
    page, group = case["page"], Hq // case["Hk"]
    out = torch.zeros((B, n, Hq, D), dtype=torch.float64, device=s["q"].device)
    for b, L in enumerate(s["lengths"].tolist()):
        t = s["table"][b, :-(-L // page)].long()
        for h in range(case["Hk"]):
            kv = []
            for codes, scale in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
                each = scale[t, h].double().reshape(-1).repeat_interleave(BLOCK)[:L, None]
                kv.append(codes[t, h].view(torch.float8_e4m3fn).double().reshape(-1, D)[:L] * each)
            for k in range(n):
                i = L - n + k
                seen = torch.arange(i + 1, device=t.device)
                if case["window"]:
                    seen = seen[(seen > i - case["window"]) | (seen < case["sinks"])]
                q = s["q"][b, k, h * group:(h + 1) * group].double()
                out[b, k, h * group:(h + 1) * group] = torch.softmax(q @ kv[0][seen].T / math.sqrt(D), -1) @ kv[1][seen]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return [_exact_heads(s["q"], s["wq"], case, s["positions"], s["axis"]), _exact_heads(s["k"], s["wk"], case, s["positions"], s["axis"])]
    if case["op"] == "append":
        if case["B"] * (case["new"] // BLOCK + 2) > 20000:
            return None
        k, ks = _exact_append(s["k"], s["kc"], s["ks"], s)
        v, vs = _exact_append(s["v"], s["vc"], s["vs"], s)
        return {"k": k, "v": v, "k_scale": ks, "v_scale": vs}
    return _exact_attend(s)
