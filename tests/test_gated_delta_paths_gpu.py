"""The gated delta rule's rarer paths on the GPU: waits that run out, packs of
every walk width, what a call must leave alone."""
import numpy as np
import pytest
import torch

import selective_ssm_packed_gb300 as vs
from selective_ssm_packed_gb300 import binding
from test_gated_delta_gpu import inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from selective_ssm_packed_gb300 import build
    build.build()
    binding.lib()


def buffers(x, dtype):
    """(saved, workspace) large enough for both directions."""
    T, Hk, K = x["q"].shape
    Hv, V = x["v"].shape[1:]
    sizes = (T, x["cu"].numel() - 1, Hk, Hv, K, V, 0 if dtype == "f32" else 1)
    size = max(binding.gated_delta_fwd_workspace_size(*sizes), binding.gated_delta_bwd_workspace_size(*sizes))
    return [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in (binding.gated_delta_saved_size(*sizes), size)]


@pytest.mark.parametrize("dtype,lens,Hk,Hv,K,V", [
    ("f32", [5, 300, 0, 77], 2, 4, 96, 80), ("bf16", [700], 1, 2, 128, 128),
    ("bf16", [40, 130, 10, 60] * 10, 4, 12, 64, 72), ("bf16", [64, 200, 30, 90, 16] * 5, 8, 32, 128, 136)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(dtype, lens, Hk, Hv, K, V):
    # the knob has one CTA of each kernel treat its first wait as run out once it is over: nothing is withheld
    x = inputs(lens, Hk, Hv, K, V, dtype, 40, states=True)
    a = [x[n] for n in ("q", "k", "v", "g", "beta")]
    ref = run(x, states=True)
    saved, ws = buffers(x, dtype)
    for cta in (0, 3):
        try:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, cta)
            vs.varlen_gated_delta_fwd(*a, x["cu"], saved=False, workspace=ws, initial_states=x["init"], final_states=True)
            assert binding.read_status(ws) == -17
            vs.varlen_gated_delta_fwd(*a, x["cu"], saved=saved, workspace=ws, initial_states=x["init"])
            assert binding.read_status(ws) == -17
        finally:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
        out, _, final = vs.varlen_gated_delta_fwd(*a, x["cu"], saved=saved, workspace=ws, initial_states=x["init"],
                                                  final_states=True)
        assert binding.read_status(ws) == 0
        assert torch.equal(out, ref["out"]) and torch.equal(final, ref["final"])
        try:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, cta)
            vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, workspace=ws, d_final_states=x["dfinal"],
                                      d_initial_states=True)
            assert binding.read_status(ws) == -17
        finally:
            binding.debug_set(binding.VSSM_DBG_FORCE_COPY_TIMEOUT, -1)
        g = vs.varlen_gated_delta_bwd(*a, x["dout"], x["cu"], saved, workspace=ws, d_final_states=x["dfinal"],
                                      d_initial_states=True)
        assert binding.read_status(ws) == 0
        for n in ("dq", "dk", "dv", "dg", "dbeta", "d_initial_states"):
            assert torch.equal(g[n], ref[n]), n
