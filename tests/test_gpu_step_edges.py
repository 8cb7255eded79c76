"""GPU tests of the serving step's operators at their edges: empty batches, rows and
sequences that are left out, shared memory between arguments, many small groups."""
import pytest
import torch

from test_gpu_step import i32, norms_inputs, rn  # noqa: F401  (rn: a fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norms


@pytest.mark.parametrize("eps", [1e-6, 1])  # (a whole number: the way that is not marshalled natively)
@pytest.mark.parametrize("out_dtype", [None, "fp8"])
@pytest.mark.parametrize("gate", ["none", "layer", "token", "sequence"])
def test_norms_of_no_tokens(rn, eps, out_dtype, gate):  # noqa: F811
    H = 64
    x, r, pw, w, _, _ = norms_inputs(0, H, "bf16", "same", "none", 0.0)
    g = {"none": None, "layer": torch.ones(H), "token": torch.ones(0, H), "sequence": torch.ones(3, H)}[gate]
    out, ro, scale = rn.fused_block_norms(x, r, pw, w, eps=eps, gate=None if g is None else g.bfloat16().cuda(),
                                          gate_index=i32([]) if gate == "sequence" else None, out_dtype=out_dtype)
    assert out.shape == (0, H) and ro.shape == (0, H) and (scale is None if out_dtype is None else scale.shape == (0,))


@pytest.mark.parametrize("eps", [1e-6, 1])
def test_norms_of_no_gates(rn, eps):  # noqa: F811
    # no sequence has a gate row: every token is left out, and one that names a row is told
    x, r, pw, w, _, _ = norms_inputs(5, 64, "bf16", "same", "none", 0.0)
    none = torch.ones(0, 64, dtype=torch.bfloat16, device="cuda")
    out, ro = torch.full_like(x, 7.0), torch.full_like(r, 5.0)
    for index, status in (([-1] * 5, 0), ([-1, -3, 0, -1, -1], rn.RMSATTN_BAD_PAGE)):
        rn.fused_block_norms(x, r, pw, w, eps=eps, gate=none, gate_index=i32(index), out=out, residual_out=ro)
        torch.cuda.synchronize()
        assert rn.rmsattn_read_status(clear=True) == status
        assert (out == 7).all() and (ro == 5).all()
