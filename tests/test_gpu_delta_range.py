"""The gated delta rule outside the decays that training starts from: states that grow, and
gradients of decays so strong that little of a state outlives a token.  Shapes select every
walk; tolerances as in test_gpu_delta unless a test states its own."""
import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_03_amd as ssd
from test_gpu_delta import F32, backward, check_backward, check_forward, up

pytestmark = pytest.mark.gpu

# b, T, H, P, N, G, dtype: teams of one and two column tiles, dstate 256, the walks of narrow
# states and of float32
SHAPES = [(2, 130, 4, 64, 64, 2, "bf16"), (1, 130, 80, 64, 128, 8, "bf16"), (1, 100, 2, 128, 256, 1, "bf16"),
          (1, 130, 4, 32, 32, 2, "bf16"), (2, 100, 2, 16, 16, 1, "bf16"), (2, 130, 4, 64, 64, 2, "f32"),
          (1, 100, 2, 32, 256, 1, "f32"), (1, 77, 3, 16, 16, 1, "f32")]
NAME = "b{}T{}H{}P{}N{}G{}{}"


@pytest.mark.parametrize("case", SHAPES, ids=lambda c: NAME.format(*c))
def test_growing_states(case):
    """A > 0: a_t = exp(dt A) up to 1.03, the state grows by e^2 over the tokens."""
    b, T, H, P, N, G, dtype = case
    d = ref.make(b, T, H, P, N, G, 51, dtype, dt_hi=0.002)
    d["A"] = d["A"].abs()
    check_forward(d, dtype, case)
    check_backward(d, ref.make_grads(b, T, H, P, N, 51, dtype), dtype, case)
