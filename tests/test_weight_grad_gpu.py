"""The gradient of combine without the weights' part, through the tensor function."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import latency_skinny_bf16_gb300 as sk
from test_expert_rows_gpu import host, matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,H,dtype", [(1, 8, 7168, "bf16"), (40, 4, 1001, "bf16"), (700, 6, 509, "fp32"), (33, 2, 264, "fp32"), (3, 2, 0, "fp32")])
def test_rows_alone(T, k, H, dtype, weighted):
    ids, w = ref.routing(T, k, 16, seed=H, drop=0.2)
    pos, _, off = ref.dispatch(ids, 16)
    n = int(off[-1])
    dy, ys = matrix(T, H, dtype, 1), matrix(T * k, H, dtype, 2)
    ys.fill_(float("nan"))                     # not read
    pt, wt = torch.from_numpy(pos).cuda(), torch.from_numpy(w).cuda() if weighted else None
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for stream in (None, s):
        dys = torch.full_like(ys, -5.0)
        s.wait_stream(torch.cuda.current_stream())
        got, dw = sk.expert_combine_grad(dy, ys, pt, wt, dys=dys, stream=stream, weight_grad=False)
        torch.cuda.synchronize()
        assert dw is None and got is dys
        want, _, _ = ref.combine_grad(host(dy), host(ys), pos, w if weighted else None)
        g = host(dys)
        assert (g[n:] == -5.0).all()
        assert (np.abs(g[:n] - want[:n]) <= ref.rounded(want[:n], ref.U32 * np.abs(want[:n]), dtype)).all()


def test_refusal():
    dy, pos = matrix(2, 8, "fp32", 1), torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        sk.expert_combine_grad(dy, dy, pos, dweights=torch.empty((2, 1), device="cuda"), weight_grad=False)
