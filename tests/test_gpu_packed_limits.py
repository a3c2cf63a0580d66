"""GPU tests of the packed layer's operators and the 4-bit cache at the ends of
their ranges of sizes: as many rows, workgroups or sequences as a call takes."""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")
import packed_ops_ref as R  # noqa: E402
from test_gpu_kv4 import BF, i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def P():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import post_weight_quantization_29_amd as P
    P.lib()
    return P


@pytest.mark.parametrize("m,d_in,group", [(1, 8, 8), (2, 32, 32)])
def test_linear_of_the_most_rows(P, m, d_in, group):
    """2^27 - 32 weight rows; weights of small whole numbers, so every sum is exact."""
    d_out = (1 << 27) - 32
    words = torch.randint(-2 ** 31, 2 ** 31, (d_out, d_in // 8), dtype=torch.int64, device="cuda").to(torch.int32)
    w = P.W4Weight(words, torch.ones((d_out, 1), device="cuda"), torch.full((d_out, 1), 7, dtype=torch.int32, device="cuda"), group)
    X = torch.ones((m, d_in), dtype=BF, device="cuda")
    Y = torch.zeros((m, d_out), dtype=torch.float32, device="cuda")
    P.gptq_w4_linear(X, w, Y)
    want = torch.full((d_out,), -7.0 * d_in, device="cuda")
    for k in range(8):
        want += ((words >> (4 * k)) & 15).sum(1).float()
    assert bool((Y == want).all())
