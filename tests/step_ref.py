"""Plain references for the operators around the attention in a serving step, and
the error that a right kernel may have (tests/attn_ref.py has the attention's)."""
import torch

from attn_ref import HALF, TINY, U, half_step


def pages_step(free, n_free, table, lengths, new, shared, page, T):
    """The step sequence by sequence, in whole numbers: the seven results, the
    table and the free list."""
    n, width = len(free), len(table[0]) if table else 0
    free, table = list(free), [list(r) for r in table]
    stack = free[:min(max(n_free, 0), n)]
    for s, L in enumerate(lengths):
        if L >= 0 and new[s] < 0:
            stack += table[s][max(shared[s], 0) if shared else 0:min(-(-L // page), width)]
    stack = stack[:n]
    wanted = given = 0
    cu, before, after = [0], [], []
    pos, slots, rows = [0] * T, [-1] * T, [-1] * T
    for s, L in enumerate(lengths):
        a = max(new[s], 0) if L >= 0 else 0
        begin = cu[-1]
        cu.append(begin + a)
        if L < 0 or new[s] < 0:
            before.append(-1)
            after.append(min(L, 0))
            continue
        own, need = -(-L // page), -(-(L + a) // page)
        ok = need <= width and begin + a <= T and L + a < 2 ** 31
        if ok:
            wanted += need - own
            ok = need == own or wanted <= len(stack)
            if ok:
                for j in range(own, need):
                    table[s][j] = stack[len(stack) - 1 - given]
                    given += 1
        for t in range(begin, min(begin + a, T)):
            p = L + t - begin
            pos[t], rows[t] = (p + 2 ** 31) % 2 ** 32 - 2 ** 31, s
            if ok and 0 <= table[s][p // page] < n:
                slots[t] = table[s][p // page] * page + p % page
        before.append(L if ok else -1)
        after.append(L + a if ok else L)
    left = len(stack) - given
    free[:left] = stack[:left]
    return [[min(c, T) for c in cu], pos, slots, rows, before, after, [left]], table, free


def norms(x, residual, post_w, w, gate, index, eps, alpha, offset):
    """(y, bound of y, h, bound of h) of ``fused_block_norms`` on the CPU, in fp64;
    y is taken of h as the kernel stored it (``h_of``)."""
    H = x.shape[1]
    eps = float(torch.tensor(eps, dtype=torch.float32))
    alpha, offset = (float(torch.tensor(v, dtype=torch.float32)) for v in (alpha, offset))
    one = torch.ones(H, dtype=torch.float64)
    # a row's sum of squares (a lane's terms one by one, five levels in a warp,
    # up to 32 warps), the mean, eps, the root; two products and the weight's sum
    rel = (max(32, H / 256) + 64) * U / 2 + 8 * U

    def norm(v, weight):
        f = one if weight is None else weight.double() + offset
        return f * v / torch.sqrt(v.square().mean(-1, keepdim=True) + eps)

    p = norm(x.double(), post_w)
    if gate is not None:
        p = p * (gate.double() if index is None else gate.double()[index.long().clamp(min=0)])
    h = alpha * residual.double() + p
    dt = residual.dtype
    err = p.abs() * (rel + 2 * U) + h.abs() * U
    h_bound = err + HALF[dt] * (h.abs() + err) + TINY[dt]

    def of(stored):
        y = norm(stored.double(), w)
        e = y.abs() * rel
        return y, e + HALF[x.dtype] * (y.abs() + e) + TINY[x.dtype], e

    return h, h_bound, of


def check_codes(codes, scale, y, err, what=""):
    """E4M3 codes and row scales of y: the scale to fp32's roundings, each code the
    nearest to within the error of its quotient."""
    top = y.abs().amax(-1)
    off = err.amax(-1) + top * 3 * U
    assert bool(((scale.double() - top / 448).abs() <= off / 448).all()), f"{what}: scales"
    safe = torch.where(top > 0, top, torch.ones_like(top))[:, None]
    q = y * 448 / safe
    have = codes.view(torch.float8_e4m3fn).double()
    room = half_step(q) * (1 + 8 * U) + (err + y.abs() * 4 * U) * 448 / safe + q.abs() * off[:, None] / safe
    assert bool(((have - q.clamp(-448, 448)).abs() <= room).all()), f"{what}: codes"
