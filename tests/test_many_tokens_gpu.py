"""The weight's gradient over as many tokens as an int holds."""
import pytest
import torch

import latency_skinny_bf16_gb300 as sk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [2147483584, 2147483600, 2147483647])
def test_weight_gradient_of_the_most_tokens(M):
    """All but a few rows are zeros; the others' products, whole numbers below 2^8, are exact in any order."""
    N = K = 8
    if torch.cuda.mem_get_info()[0] < 4 * M * N + (8 << 30):
        pytest.skip("room for two matrices of this many rows")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    want = torch.zeros((N, K), dtype=torch.float64)
    g = torch.Generator().manual_seed(M % 1000)
    for at in (0, 63, M // 8 - 1, M // 2, M - 65, M - 64, M - 17, M - 1):
        a, b = (torch.randint(-3, 4, (8,), generator=g).double() for _ in range(2))
        dy[at], x[at] = a.bfloat16().cuda(), b.bfloat16().cuda()
        want += a[:, None] * b[None, :]
    w = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    dw = torch.full((N, K), 77.0, dtype=torch.bfloat16, device="cuda")
    sk.linear_grad(dy, x, w, dw=dw, input_grad=False)
    assert torch.equal(dw.double().cpu(), want)
    assert sk.skinny_get_device_status() == 0
