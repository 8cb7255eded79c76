"""CPU checks of the serving step's operators at their edges: empty batches and
arguments that only look wrong.  No call here reaches a kernel."""
import pytest

from test_attn_binding import BF16, F32, rn  # noqa: F401  (rn: a fixture)

R32, FP8 = 0x200, 0x8000
OK, EINVAL = 0, -1


def norms(rn, **kw):
    a = dict(x=None, residual=None, post=16, w=16, gate=None, gs=0, index=None, n_gates=0, out=None, ro=None, scale=None,
             T=0, H=64, eps=1e-6, alpha=1.0, off=0.0, flags=BF16)
    a.update(kw)
    return rn.load_attn().rmsattn_block_norms(*a.values(), None)


@pytest.mark.parametrize("flags", [BF16, F32, BF16 | R32, BF16 | FP8])
@pytest.mark.parametrize("gate", [
    dict(), dict(gate=16, n_gates=1),          # none, one row for all
    dict(gs=64), dict(gate=16, gs=64),         # a row for each of no tokens (an empty tensor's address may be NULL)
    dict(gate=16, gs=64, n_gates=3),           # rows with an index of no tokens, whose address is NULL
    dict(gate=16, gs=64, n_gates=3, index=16), dict(gs=64, index=16),
])
def test_norms_of_no_tokens(rn, flags, gate):  # noqa: F811
    assert norms(rn, flags=flags, **gate) == OK


@pytest.mark.parametrize("kw", [
    dict(gate=16, gs=63, n_gates=3), dict(gate=16, gs=-64, n_gates=3), dict(gate=16, gs=64, n_gates=-1),
    dict(gs=-64), dict(gs=63), dict(n_gates=-1), dict(gate=16, gs=64, n_gates=1 << 60), dict(scale=16), dict(H=0),
    dict(eps=-1.0), dict(flags=3),
])
def test_norms_of_no_tokens_still_refuse(rn, kw):  # noqa: F811
    assert norms(rn, **kw) == EINVAL


@pytest.mark.parametrize("flags,status", [(0x70000 | FP8, OK), (0x30000, OK), (0x40000, EINVAL), (0x80000, EINVAL)])
def test_norms_flags_of_rows_left_out(rn, flags, status):  # noqa: F811
    assert norms(rn, flags=BF16 | flags) == status


# ---------------------------------------------------------------- pages

WRITTEN = dict(cu=16, pos=16, slots=32, rows=16, before=12, after=12, out=4, free=32, ws=0)  # bytes, of 3 sequences, 4 rows, 8 pages
READ = dict(table=40, n_free=4, lengths=12, new=12, shared=12)  # rows of 2, 4 apart


def pages(rn, **kw):
    a = dict(free=0x1000, pages=8, n_free=0x2000, table=0x3000, ts=4, width=2, lengths=0x4000, new=0x5000, shared=0x6000,
             B=3, page=16, T=4, cu=0x7000, pos=0x8000, slots=0x9000, rows=0xA000, before=0xB000, after=0xC000, out=0xD000,
             ws=None, wsb=0, flags=0)
    a.update(kw)
    return rn.load_attn().rmsattn_pages_step(*a.values(), None), a


def pairs():
    names = list(WRITTEN)[:-1] + list(READ)
    for i, w in enumerate(list(WRITTEN)[:-1]):
        for r in names[i + 1:]:
            yield w, r
    for r in list(READ)[1:]:
        yield "table", r


@pytest.mark.parametrize("one,other", list(pairs()))
def test_pages_that_share_memory_are_refused(rn, one, other):  # noqa: F811
    size = {**WRITTEN, **READ}
    wide = [n for n in (one, other) if n in ("pos", "slots", "rows")]  # (16-byte aligned)
    _, a = pages(rn, flags=1)  # (refused: for the addresses alone)
    assert pages(rn, **{one: a[other]})[0] == EINVAL
    # the last bytes of one on the first of the other, where alignment lets them
    for x, y in ((one, other), (other, one)):
        if x not in wide:
            assert pages(rn, **{x: a[y] - size[x] + 4})[0] == EINVAL


@pytest.mark.parametrize("name,at", [("lengths", 0x3000), ("lengths", 0x2FF8), ("lengths", 0x3004), ("lengths", 0x3008),
                                     ("lengths", 0x300C), ("lengths", 0x3020), ("lengths", 0x3024), ("after", 0x3010),
                                     ("before", 0x301C), ("out", 0x3014), ("out", 0x3024), ("n_free", 0x3020)])
def test_pages_within_the_tables_rows_are_refused(rn, name, at):  # noqa: F811
    assert pages(rn, **{name: at})[0] == EINVAL  # rows of 8 bytes, 16 apart, from 0x3000 on


def test_pages_workspace_apart(rn):  # noqa: F811
    big = dict(B=3000, table=0x100000, lengths=0x200000, new=0x300000, shared=None, cu=0x400000, before=0x500000,
               after=0x600000, ws=0x700000, wsb=1 << 20)
    for name in ("free", "n_free", "lengths", "new", "cu", "pos", "slots", "rows", "before", "after", "out", "table"):
        assert pages(rn, **{**big, name: 0x700000})[0] == EINVAL


@pytest.mark.parametrize("kw", [
    dict(flags=BF16 | FP8, scale=0xF000, out=0x1000), dict(flags=BF16 | FP8, scale=0xF000, out=0x11C0),  # bytes on x's rows
    dict(flags=BF16 | R32, out=0x2000), dict(flags=BF16 | R32, ro=0x1000),  # rows of other sizes
    dict(out=0x1010), dict(ro=0x2010), dict(out=0x0FF0), dict(ro=0x1E10),   # rows shifted
    dict(out=0x3000), dict(ro=0x4040), dict(out=0x4070),                    # weights
    dict(gate=0x5000, n_gates=1, out=0x5000), dict(gate=0x5000, gs=72, n_gates=4, out=0x5000),
    dict(gate=0x5000, gs=64, n_gates=4, ro=0x5080), dict(gate=0x5000, gs=64, n_gates=9, index=0x6000, out=0x5000),
    dict(gate=0x5000, gs=64, n_gates=9, index=0x6000, ro=0x6000), dict(gate=0x5000, gs=64, n_gates=9, index=0x81F0),
    dict(flags=BF16 | FP8, scale=0x1000), dict(flags=BF16 | FP8, scale=0x8000), dict(flags=BF16 | FP8, scale=0x91FC),
    dict(out=0x9000), dict(out=0x9100),
])
def test_norms_that_share_memory_are_refused(rn, kw):  # noqa: F811
    a = dict(T=4, x=0x1000, residual=0x2000, post=0x3000, w=0x4000, out=0x8000, ro=0x9000)
    assert norms(rn, **{**a, **kw}) == EINVAL
