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
