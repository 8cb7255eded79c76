"""Operators of a serving step around the attention path, in plain torch and as the package's kernels.

  pages    the step's plan, made on the GPU from the requests' lengths: finished
           sequences give their pages back, growing ones get new pages from the
           list of free ones (block table), and every row of the step's batch
           its position, its place in the cache (slot) and its sequence
  prefix   attention of one or a few query tokens per sequence over the paged
           E4M3 cache, where groups of sequences share a long first part
           (a system prompt, a document): the shared tokens once for the group
  norms    the end of one block and the begin of the next: RMS norm of the
           block's output, its gate, the residual update and the RMS norm of
           the updated residual

Definitions:

  pages    sequence s holds L tokens and gets a more (a < 0: it is finished).
           In the sequences' order a finished one returns the pages
           [shared, ceil(L / page)) of its row, behind the free ones; with F
           free pages then, the k-th page that is taken is free[F - 1 - k].
           A sequence takes ceil((L + a) / page) - ceil(L / page) pages; it is
           left out if they outrun F, the table's width or the batch's rows.
  prefix   softmax(scale q k) v over the tokens j <= i of the query's own
           sequence, i its position; no visible token gives 0
  norms    h = residual_scale residual + gate (post_w + offset) x / rms(x)
           y = (w + offset) h / rms(h),  rms(v) = sqrt(mean(v^2) + eps), of the
           h that is stored; y in the type of x, or E4M3 codes with the row's
           scale max|y| / 448
"""
import math

import torch

own = False

BLOCK = 16  # tokens that share a scale of the cache
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


def listed():
    pages = {"op": "pages", "page": 64, "done": 0.0, "shared": 0, "poor": False}
    prefix = {"op": "prefix", "page": 64, "n": 1, "groups": 1, "dtype": "bf16"}
    norms = {"op": "norms", "gate": "none", "dtype": "bf16", "stream": "same", "fp8": False, "offset": 0.0}
    return [
        # a decode step of a few sequences: latency
        {**pages, "name": "pages_decode_8", "B": 8, "new": 1, "old": 2000},
        # a decode step of a busy server: some sequences have ended, all share a system prompt
        {**pages, "name": "pages_decode_1024", "B": 1024, "new": 1, "old": 4000, "done": 0.05, "shared": 512, "page": 16},
        # a batch of ragged prompts and of chunks behind earlier ones
        {**pages, "name": "pages_prefill_64x2000", "B": 64, "new": 2000, "old": 1000, "done": 0.05},
        # a few sequences behind a short system prompt: latency
        {**prefix, "name": "prefix_8x2048", "B": 8, "P": 2048, "own": 100, "Hq": 32, "Hk": 8, "D": 128},
        # a decode step of a busy server behind one long document
        {**prefix, "name": "prefix_64x8192", "B": 64, "P": 8192, "own": 500, "Hq": 32, "Hk": 8, "D": 128},
        # the largest batch, the shared part far above the sequences' own
        {**prefix, "name": "prefix_256x16384", "B": 256, "P": 16384, "own": 500, "Hq": 32, "Hk": 8, "D": 128},
        # several system prompts, two drafted tokens a sequence, small heads and pages
        {**prefix, "name": "prefix_96_groups_d64", "B": 96, "P": 3000, "own": 301, "groups": 6, "n": 2, "Hq": 64, "Hk": 8, "D": 64, "page": 16, "dtype": "f16"},
        # wide heads, an odd batch
        {**prefix, "name": "prefix_37x5000_d256", "B": 37, "P": 5000, "own": 333, "Hq": 16, "Hk": 2, "D": 256, "page": 32},
        # a decode step: latency
        {**norms, "name": "norms_decode_8", "T": 8, "H": 4096},
        # a prefill, the gate one learned vector of the layer
        {**norms, "name": "norms_prefill_16384x8192", "T": 16384, "H": 8192, "gate": "layer"},
        # image and video tokens, a gate row for each sequence of the batch, codes for the next product
        {**norms, "name": "norms_gated_fp8_4096x5120", "T": 4096, "H": 5120, "gate": "sequence", "fp8": True},
        # rows off the vectors' grid, gates of every token, an fp32 residual stream
        {**norms, "name": "norms_odd_4099x2045", "T": 4099, "H": 2045, "gate": "token", "stream": "f32", "dtype": "f16", "offset": 1.0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "prefix", "prefix", "norms"])
    if op == "pages":
        B = _log(rng, 1, 4096)
        new = rng.choice([1, 1, _log(rng, 2, 3000)])
        return {"op": op, "B": B, "new": min(new, max(1, 128000 // B)), "old": _log(rng, 1, min(16000, 4000000 // B)), "page": rng.choice([16, 32, 64, 128]),
                "done": rng.choice([0.0, 0.1, 0.4]), "shared": rng.choice([0, 0, 512]), "poor": rng.random() < 0.15}
    if op == "prefix":
        D = rng.choice([64, 128, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 7, 8])
        n = rng.choice([1, 1, 1, 2, 3, 5])
        page = rng.choice([16, 32, 64, 128])
        B = _log(rng, 1, min(300, 256 * 32 * 128 // (Hk * G * n * D)))
        return {"op": op, "B": B, "P": _log(rng, 16, min(65536, max(32, 256 * 16384 * 32 * 128 // (B * Hk * G * n * D)))),
                "own": _log(rng, n, max(n + 1, min(3000, 256 * 500 * 8 * 128 // (B * Hk * D)))), "groups": rng.choice([1, 1, _log(rng, 1, B)]), "n": n,
                "Hq": Hk * G, "Hk": Hk, "D": D, "page": page, "dtype": rng.choice(["bf16", "bf16", "f16"])}
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    gate = rng.choice(["none", "layer", "sequence", "token"])
    H = _log(rng, 64, 16384)
    if rng.random() < 0.6:
        H = max(64, H // 64 * 64)
    size = (4 if dtype == "f32" else 2) * (5 if gate == "token" else 4)
    return {"op": op, "T": _log(rng, 1, min(20000, 16384 * 8192 * 8 // (H * size))), "H": H, "gate": gate, "dtype": dtype,
            "stream": rng.choice(["same", "same", "f32"]) if dtype != "f32" else "same", "fp8": rng.random() < 0.3, "offset": rng.choice([0.0, 0.0, 1.0])}


# ---------------------------------------------------------------- inputs


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


def _host(seed):
    """Random whole numbers that shape a case (group borders), on the host."""
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "pages":
        B, page = case["B"], case["page"]
        # ragged: each piece that is longer than the usual has one that is as much shorter
        half = torch.randint(0, case["new"] // 2 + 1, (B // 2,), generator=g, device=dev)
        new = case["new"] + torch.cat([half, -half, half.new_zeros(B % 2)])
        old = torch.randint(0, 2 * case["old"], (B,), generator=g, device=dev)
        old[0] = 2 * case["old"]
        first = case["shared"] // page  # pages of the prompt that all of them begin with
        old = torch.where(old < first * page, old + first * page, old)
        done = torch.rand(B, generator=g, device=dev) < case["done"]
        rows = int(new.sum())  # a batch of fixed size; the finished sequences' rows stay empty
        width = -(-(2 * case["old"] + first * page + case["new"] + case["new"] // 2) // page)
        pages = B * width + first
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = order[first:].reshape(B, width).clone()
        table[:, :first] = order[:first]
        has = (old + page - 1) // page
        held = torch.arange(width, device=dev) < has[:, None]
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        left = order[first:].reshape(B, width)[~held]
        if case["poor"]:  # the free pages may run out
            left = left[: B // 2 + 1]
        s["free"][: left.numel()] = left
        s["n_free"] = torch.tensor([left.numel()], dtype=torch.int32, device=dev)
        s["table"] = torch.where(held, table, -1)
        s["lengths"] = old.to(torch.int32)
        s["new"] = torch.where(done, -1, new).to(torch.int32)
        s["shared"] = torch.full((B,), first, dtype=torch.int32, device=dev)
        s["rows"] = rows
        return s
    dt = DTYPES[case["dtype"]]
    if case["op"] == "prefix":
        B, Hk, D, page, n, G = case["B"], case["Hk"], case["D"], case["page"], case["n"], case["groups"]
        h = _host(seed)
        cuts = sorted(torch.randperm(B - 1, generator=h)[: G - 1].add(1).tolist()) if B > 1 else []
        cu = [0] + cuts + [B]
        # the first group shares all of P, the others a part; whole pages
        P = [max(1, int(case["P"] * (1.0 if i == 0 else float(torch.rand(1, generator=h))))) // page * page for i in range(len(cu) - 1)]
        mine = torch.randint(max(n, case["own"] // 2), 2 * max(n, case["own"]) - max(n, case["own"] // 2) + 1, (B,), generator=g, device=dev)
        start = torch.repeat_interleave(torch.tensor(P), torch.tensor([b - a for a, b in zip(cu, cu[1:])])).to(dev)
        wide = -(-(2 * max(n, case["own"])) // page)  # pages of a sequence's own tokens
        width = max(P) // page + wide
        total = sum(P) // page + B * wide
        order = torch.randperm(total, generator=g, device=dev).to(torch.int32)
        table = torch.zeros((B, width), dtype=torch.int32, device=dev)
        at = 0
        for i, p in enumerate(P):
            a, b, k = cu[i], cu[i + 1], p // page
            table[a:b, :k] = order[at:at + k]
            at += k
            table[a:b, k:k + wide] = order[at:at + (b - a) * wide].reshape(b - a, wide)
            at += (b - a) * wide
        s["table"], s["lengths"] = table, (start + mine).to(torch.int32)
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev)
        s["P"] = torch.tensor(P, dtype=torch.int32, device=dev)
        s["plan"] = list(zip(cu, cu[1:], P))
        s["wide"] = wide
        s["q"] = torch.randn((B, n, case["Hq"], D), generator=g, device=dev).to(dt)
        s["kc"], s["ks"] = _filled(g, total, Hk, page, D, dev)
        s["vc"], s["vs"] = _filled(g, total, Hk, page, D, dev)
        if own:
            import residual_add_rmsnorm_vec_gb300 as rn
            s["cache"] = rn.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        return s
    T, H = case["T"], case["H"]
    stream = torch.float32 if case["stream"] == "f32" else dt
    s["x"] = (3 * torch.randn((T, H), generator=g, device=dev)).to(dt)
    s["residual"] = (2 * torch.randn((T, H), generator=g, device=dev)).to(stream)
    for name in ("post_w", "w"):
        s[name] = (1 - case["offset"] + 0.1 * torch.randn(H, generator=g, device=dev)).to(dt)
    s["index"] = s["gate"] = None
    if case["gate"] == "layer":
        s["gate"] = (0.5 + 0.2 * torch.randn(H, generator=g, device=dev)).to(dt)
    elif case["gate"] == "token":
        s["gate"] = torch.sigmoid(torch.randn((T, H), generator=g, device=dev)).to(dt)
    elif case["gate"] == "sequence":
        n = max(1, min(16, T // 3))
        s["gate"] = torch.randn((n, H), generator=g, device=dev).to(dt)
        s["index"] = torch.randint(0, n, (T,), generator=g, device=dev).sort().values.to(torch.int32)
    s["alpha"] = 0.75
    return s


# ---------------------------------------------------------------- plain forms


def _plain_pages(s):
    page, T = s["case"]["page"], s["rows"]
    free, table = s["free"], s["table"]
    dev, n, (B, width) = free.device, free.numel(), table.shape
    L, a = s["lengths"].long(), s["new"].long()
    live = L >= 0
    done = live & (a < 0)
    more = torch.where(live & (a > 0), a, 0)
    has = (L.clamp(min=0) + page - 1) // page
    need = (L.clamp(min=0) + more + page - 1) // page
    end = more.cumsum(0)
    begin = end - more
    fits = (need <= width) & (end <= T) & (L + more < 2**31)
    take = torch.where(live & ~done & fits, need - has, 0)
    shared = torch.minimum(s["shared"].long().clamp(min=0), has)
    freed = torch.where(done, has - shared, 0)
    freed_end = freed.cumsum(0)
    count = s["n_free"].long().clamp(0, n)
    top = (count + freed_end[-1]).clamp(max=n)
    taken_end = take.cumsum(0)
    ok = live & ~done & fits & ((take == 0) | (taken_end <= top))
    left = top - torch.where(ok, taken_end, 0).amax()
    # the free pages and behind them the returned ones
    i = torch.arange(n, device=dev)
    f = i - count
    of = torch.searchsorted(freed_end, f.clamp(min=0), right=True).clamp(max=B - 1)
    col = (shared[of] + f - (freed_end - freed)[of]).clamp(0, width - 1)
    stack = torch.where(f < 0, free, table[of, col])
    # new pages
    j = torch.arange(width, device=dev)
    fresh = ok[:, None] & (j >= has[:, None]) & (j < need[:, None])
    place = top - 1 - ((taken_end - take)[:, None] + j - has[:, None])
    table.copy_(torch.where(fresh, stack[place.clamp(0, n - 1)], table))
    free.copy_(torch.where(i < left, stack, free))
    # rows
    t = torch.arange(T, device=dev)
    row = torch.searchsorted(end, t, right=True)
    on = row < B
    row = row.clamp(max=B - 1)
    pos = L[row] + t - begin[row]
    pg = table[row, (pos // page).clamp(0, width - 1)].long()
    cu = torch.cat([end.new_zeros(1), end]).clamp(max=T).to(torch.int32)
    return [cu, torch.where(on, pos, 0).to(torch.int32), torch.where(on & ok[row] & (pg >= 0) & (pg < n), pg * page + pos % page, -1),
            torch.where(on, row, -1).to(torch.int32), torch.where(ok, L, -1).to(torch.int32),
            torch.where(done, 0, torch.where(ok, L + more, L)).to(torch.int32), left.to(torch.int32).reshape(1), table, free]


def _values(codes, scale, t):
    """Values of the tokens of tables t [..., pages]: [..., heads, tokens, D]."""
    x = codes[t].view(torch.float8_e4m3fn).float()
    x = x.unflatten(-2, (x.shape[-2] // BLOCK, BLOCK)) * scale[t][..., None, None]
    return x.flatten(-3, -2).transpose(-4, -3).flatten(-3, -2)


def _plain_prefix(s):
    case = s["case"]
    B, n, Hq, D = s["q"].shape
    Hk, page, wide = case["Hk"], case["page"], s["wide"]
    out = torch.empty_like(s["q"])
    for a, b, P in s["plan"]:
        table = s["table"][a:b].long()
        q = s["q"][a:b].float().reshape(b - a, n, Hk, Hq // Hk, D).permute(2, 0, 1, 3, 4).reshape(Hk, b - a, -1, D)
        shared = q.flatten(1, 2) @ _values(s["kc"], s["ks"], table[0, :P // page]).transpose(-1, -2)  # [Hk, columns, P]
        mine = table[:, P // page:P // page + wide]
        k, v = (_values(c, x, mine).transpose(0, 1) for c, x in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        last = s["lengths"][a:b].long()[:, None] - n + torch.arange(n, device=q.device)
        seen = (P + torch.arange(wide * page, device=q.device) <= last[..., None]).repeat_interleave(Hq // Hk, 1)
        scores = (q @ k.transpose(-1, -2)).masked_fill(~seen, -math.inf).flatten(1, 2)
        scale = 1 / math.sqrt(D)
        top = scores.amax(-1, keepdim=True)
        if P:
            top = torch.maximum(top, shared.amax(-1, keepdim=True))
        p = torch.exp((scores - top) * scale)
        total = p.sum(-1, keepdim=True)
        o = (p.unflatten(1, (b - a, -1)) @ v).flatten(1, 2)
        if P:
            p = torch.exp((shared - top) * scale)
            total = total + p.sum(-1, keepdim=True)
            o = o + p @ _values(s["vc"], s["vs"], table[0, :P // page])
        out[a:b] = (o / total).reshape(Hk, b - a, n, Hq // Hk, D).permute(1, 2, 0, 3, 4).reshape(b - a, n, Hq, D).to(out.dtype)
    return out


def _plain_norms(s):
    off = s["case"]["offset"]
    x = s["x"].float()
    p = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s["post_w"].float() + off)
    if s["gate"] is not None:
        gate = s["gate"] if s["index"] is None else s["gate"][s["index"].long()]
        p = p * gate.float()
    h = (s["alpha"] * s["residual"].float() + p).to(s["residual"].dtype)
    y = h.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (s["w"].float() + off)
    if not s["case"]["fp8"]:
        return [y.to(s["x"].dtype), h]
    top = y.abs().amax(-1, keepdim=True)
    back = torch.where(top > 0, 448 / top, torch.zeros_like(top))
    return [(y * back).clamp(-448, 448).to(torch.float8_e4m3fn), h, (top / 448)[:, 0]]


def run(s):
    case = s["case"]
    if not own:
        return {"pages": _plain_pages, "prefix": _plain_prefix, "norms": _plain_norms}[case["op"]](s)
    import residual_add_rmsnorm_vec_gb300 as rn
    if case["op"] == "pages":
        step = rn.kv_pages_step_(s["free"], s["n_free"], s["table"], s["lengths"], s["new"], s["shared"], page_size=case["page"], n_rows=s["rows"])
        return [*step, s["table"], s["free"]]
    if case["op"] == "prefix":
        return rn.kv_cache_prefix_attention(s["q"], s["cache"], s["table"], s["lengths"], s["P"], s["cu"])
    y, h, scale = rn.fused_block_norms(s["x"], s["residual"], s["post_w"], s["w"], eps=EPS, gate=s["gate"], gate_index=s["index"], residual_scale=s["alpha"],
                                       weight_offset=case["offset"], out_dtype="fp8" if case["fp8"] else None)
    return [y.view(torch.float8_e4m3fn), h, scale] if case["fp8"] else [y, h]


# ---------------------------------------------------------------- cost and the definition in 64 bits


def work(case):
    if case["op"] == "pages":
        B, T, page = case["B"], case["B"] * case["new"], case["page"]
        moved = T // page + int(B * case["done"] * case["old"] / page)  # pages taken and returned
        return {"bytes": 24 * B + 16 * T + 8 * moved, "flops": T}
    if case["op"] == "prefix":
        B, n, Hk, D = case["B"], case["n"], case["Hk"], case["D"]
        shared = case["P"] * (1 + (case["groups"] - 1) / 2)  # tokens that are read once for their group
        seen = B * (case["P"] * (1 + (case["groups"] - 1) / 2) / case["groups"] + max(n, case["own"]))
        return {"bytes": int((shared + B * max(n, case["own"])) * Hk * 2 * (D + 4 / BLOCK) + 4 * B * n * case["Hq"] * D), "flops": int(4 * seen * n * case["Hq"] * D)}
    T, H, size = case["T"], case["H"], 4 if case["dtype"] == "f32" else 2
    stream = 4 if case["stream"] == "f32" else size
    rows = size + 2 * stream + (1 if case["fp8"] else size) + (size if case["gate"] == "token" else 0)
    return {"bytes": T * H * rows + 2 * H * size + (4 * T if case["fp8"] else 0) + (H * size if case["gate"] == "layer" else 0), "flops": 11 * T * H}


def _exact_pages(s):
    """The step sequence by sequence, in whole numbers on the host."""
    page, T = s["case"]["page"], s["rows"]
    L, new, shared = s["lengths"].tolist(), s["new"].tolist(), s["shared"].tolist()
    table, free = s["table"].cpu().clone(), s["free"].tolist()
    n, width = len(free), table.shape[1]
    stack = free[:min(max(int(s["n_free"]), 0), n)]
    for b, (have, a) in enumerate(zip(L, new)):
        if have >= 0 and a < 0:
            stack += table[b, min(max(shared[b], 0), -(-have // page)):-(-have // page)].tolist()
    stack = stack[:n]
    given, wanted = 0, 0  # pages that went out, and that were asked for so far
    cu, before, after = [0], [], []
    pos = torch.zeros(T, dtype=torch.int64)
    slot, row = torch.full((T,), -1, dtype=torch.int64), torch.full((T,), -1, dtype=torch.int64)
    for b, (have, a) in enumerate(zip(L, new)):
        begin, count = cu[-1], max(a, 0) if have >= 0 else 0
        cu.append(begin + count)
        if have < 0 or a < 0:
            before.append(-1)
            after.append(have if have < 0 else 0)
            continue
        old, need = -(-have // page), -(-(have + count) // page)
        ok = need <= width and begin + count <= T and have + count < 2**31
        if ok:
            wanted += need - old
            ok = need == old or wanted <= len(stack)
        if ok and need > old:
            for j in range(old, need):
                table[b, j] = stack[len(stack) - 1 - given]
                given += 1
        p = have + torch.arange(max(0, min(count, T - begin)))
        pos[begin:begin + count], row[begin:begin + count] = p, b
        if ok:
            pg = table[b, p // page].long()
            slot[begin:begin + count] = torch.where((pg >= 0) & (pg < n), pg * page + p % page, -1)
        before.append(have if ok else -1)
        after.append(have + count if ok else have)
    left = len(stack) - given
    free[:left] = stack[:left]
    return [torch.tensor(v) for v in ([min(c, T) for c in cu], pos.tolist(), slot.tolist(), row.tolist(), before, after, [left], table.tolist(), free)]


def _exact_prefix(s):
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
                see = L - n + k + 1
                q = s["q"][b, k, h * group:(h + 1) * group].double()
                out[b, k, h * group:(h + 1) * group] = torch.softmax(q @ kv[0][:see].T / math.sqrt(D), -1) @ kv[1][:see]
    return out


def _exact_norms(s):
    off = s["case"]["offset"]
    x, r = s["x"].double(), s["residual"].double()
    gate = torch.ones((), dtype=torch.float64, device=x.device)
    if s["gate"] is not None:
        gate = s["gate"].double() if s["index"] is None else s["gate"].double().index_select(0, s["index"])
    h = s["alpha"] * r + gate * ((s["post_w"].double() + off) * x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[1] + EPS))
    kept = h.to(s["residual"].dtype).double()  # the norm is of what is stored
    y = (s["w"].double() + off) * kept / torch.sqrt(kept.square().sum(-1, keepdim=True) / x.shape[1] + EPS)
    if not s["case"]["fp8"]:
        return [y, h]
    scale = y.abs().amax(-1) / 448
    return [torch.where(scale[:, None] > 0, y / scale[:, None], 0.0), h, scale]


def exact(case, seed):
    s = prepare(case, seed)
    return {"pages": _exact_pages, "prefix": _exact_prefix, "norms": _exact_norms}[case["op"]](s)
