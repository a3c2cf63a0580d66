"""GPU tests of the gated backward pass at the ends of bf16's range."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import packed_ops_ref as R  # noqa: E402
from test_gpu_packed_ops import BF, weight  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import post_weight_quantization_29_amd as P
    P.lib()
    return P


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_of_far_gates(P, act):
    """Far from 0 the activations go to x or 0, their slopes to 1 or 0: also where x^2 is beyond fp32.  fp32's part of
    the error, 32 units of terms of up to |x| e^x, is far below the output's half step at |x| >= 30."""
    Lg, Lu = R.layer(32, 64, 32, 1, "cuda"), R.layer(32, 64, 32, 2, "cuda")
    far = torch.tensor([30.0, 200.0, 1e6, 1e13, 1.9e19, 1e25, 1e32, 3e38], device="cuda")
    G = torch.cat([far, -far]).to(BF).repeat(3, 2)
    U = torch.linspace(-2, 2, 96, device="cuda").to(BF).view(3, 32)
    dM = torch.full_like(G, 0.5)
    dG, dU, dX = torch.empty_like(G), torch.empty_like(G), torch.empty((3, 64), dtype=BF, device="cuda")
    P.gptq_w4_gated_backward(dM, G, U, weight(P, Lg), weight(P, Lu), dX, dG=dG, dU=dU, act=act)
    a, slope = R.act64(G.double(), act)
    for got, ref in ((dG, 0.5 * U.double() * slope), (dU, 0.5 * a)):
        worst = float(((got.double() - ref).abs() / (R.EPS[BF] * (1 + R.EPS[BF]) * ref.abs() + 1e-38)).nan_to_num(nan=9e9).max())
        assert worst <= 1.0
