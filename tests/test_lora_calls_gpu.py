"""The three kernels of a projection with adapters as one call: what follows a
projection that gave up, and calls one behind the other."""
import numpy as np
import pytest
import torch

import experts_ref as ref
import latency_skinny_bf16_gb300 as sk
from test_experts_gemm_gpu import DT, host
from test_lora_gpu import check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _init():
    assert sk.skinny_init(0) == sk.SKINNY_OK
    yield
    assert sk.skinny_get_device_status() == 0


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M", [1, 16, 40])
@pytest.mark.parametrize("backend", [sk.SKINNY_BACKEND_TCGEN05, sk.SKINNY_BACKEND_AUTO])
def test_projection_that_gives_up(M, out, backend):
    """Without any budget the projection's waits give up, and the two kernels behind it run all the same: the status
    says so, only Y is written, and the calls after it, eager and captured, are right."""
    N = 640
    x, w, a, b, ranks, scales = inputs(M, N, 1024, 6, 32, seed=M)
    ids = np.random.default_rng(M).integers(-1, 6, M).astype(np.int32)
    dev = [torch.from_numpy(v).cuda() for v in (ids, ranks, scales)]
    nbytes = sk.lora_workspace(M, N, 32, DT[out])
    ws = torch.full((nbytes + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    with sk.options(backend=backend):
        want = check(x, w, a, b, ids, ranks, scales, out)
        y = torch.full((M, N + 5), -7.0, dtype=DT[out], device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())

        def call():
            sk.lora_gemm(x, w, a, b, *dev, out=y[:, :N], workspace=ws[:nbytes])

        def captured():
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                call()
            return g

        good = captured()
        for pdl in (0, 1):
            with sk.options(wait_timeout_us=0, pdl=pdl):
                bad = captured()
                for run in (call, bad.replay, bad.replay):
                    run()
                    torch.cuda.synchronize()
                    assert sk.skinny_get_device_status() & 0xFF == sk.SKINNY_ERR_DEVICE_TIMEOUT
                    assert (y[:, N:] == -7.0).all() and (ws[nbytes:] == 0x5A).all()
                    with sk.options(wait_timeout_us=500000):
                        for again in (call, good.replay):
                            y[:, :N] = float("nan")
                            again()
                            assert torch.equal(y[:, :N], want)
                    assert sk.skinny_get_device_status() == 0
                del bad
        del good


@pytest.mark.parametrize("pdl", [0, 1, 2])
@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(16, 640, 1024), (3, 200, 777), (64, 2048, 512), (1, 2112, 7168)])
def test_calls_one_behind_the_other(M, N, K, out, pdl):
    """Calls with inputs, ids and outputs of their own share one workspace: what a call writes there must not reach the
    one before it, nor what that left the call itself. Buffers are filled before every replay."""
    calls = []
    for s in range(4):
        x, w, a, b, ranks, scales = inputs(M, N, K, 5, 48, seed=10 * s + M)
        ids = np.random.default_rng(s).integers(-1, 5, M).astype(np.int32)
        want = check(x, w, a, b, ids, ranks, scales, out)
        calls.append((x, w, a, b, *[torch.from_numpy(v).cuda() for v in (ids, ranks, scales)], torch.empty_like(want), want))
    ws = torch.empty(sk.lora_workspace(M, N, 48, DT[out]), dtype=torch.uint8, device="cuda")

    def all_calls():
        for _ in range(2):
            for c in calls:
                sk.lora_gemm(*c[:7], out=c[7], workspace=ws)

    with sk.options(pdl=pdl):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            all_calls()
        for run in (all_calls, g.replay, g.replay):
            ws.fill_(0xFF)
            for c in calls:
                c[7].fill_(float("nan"))
            run()
            torch.cuda.synchronize()
            for c in calls:
                assert torch.equal(c[7], c[8])
        del g


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("M", [17, 33, 64])
@pytest.mark.parametrize("K,pad,offset", [(777, 0, 0), (520, 0, 1), (520, 3, 5), (130, 2, 2), (1001, 7, 4)])
def test_many_tokens_unaligned(M, K, pad, offset, out):
    """Rows off 16 bytes are served at every number of tokens, several of them to an adapter."""
    x, w, a, b, ranks, scales = inputs(M, 333, K, 7, 40, seed=M + K, pad=pad, offset=offset)
    ids = np.random.default_rng(M).integers(-1, 7, M).astype(np.int32)
    check(x, w, a, b, ids, ranks, scales, out, ypad=1)


@pytest.mark.parametrize("out", ["fp32", "bf16"])
@pytest.mark.parametrize("L,R", [(0, 8), (4, 0)])
@pytest.mark.parametrize("M,K,pad,offset", [(17, 777, 0, 0), (64, 520, 0, 1), (40, 520, 3, 5), (16, 777, 0, 0), (40, 520, 0, 0)])
def test_no_adapters_at_any_alignment(M, K, pad, offset, L, R, out):
    """The projection alone takes what the call with adapters takes."""
    x, w, *_ = inputs(M, 333, K, 1, 8, seed=M + K, pad=pad, offset=offset)
    a, b = torch.zeros((L, R, K), dtype=torch.bfloat16, device="cuda"), torch.zeros((L, 333, R), dtype=torch.bfloat16, device="cuda")
    y = sk.lora_gemm(x, w, a, b, torch.zeros(M, dtype=torch.int32, device="cuda"),
                     out=torch.full((M, 334), -7.0, dtype=DT[out], device="cuda")[:, :333])
    want = host(x) @ host(w).T
    err = 1e-5 * (np.abs(host(x)) @ np.abs(host(w)).T)
    assert (np.abs(host(y) - want) <= ref.rounded(want, err, out) + 1e-6).all()
