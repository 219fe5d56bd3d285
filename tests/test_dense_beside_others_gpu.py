"""Products that follow one another on two streams while chunked prefills, which hold tensor memory too, run on a third:
each gives the bits that it gives alone."""
import pytest
import torch

import linear_attention_recurrence_chunk_gb300 as kda
from test_dense_chain_gpu import Layer

pytestmark = pytest.mark.gpu


def _products(seed, sizes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ops = [(*kda.kda_fp8_quant(torch.randn(M, K, device="cuda", generator=g)), *kda.kda_fp8_quant(torch.randn(N, K, device="cuda", generator=g), 128))
           for M, N, K in sizes]
    return lambda: [kda.kda_fp8_matmul(*o) for o in ops]


def _prefill(seed, T, H):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v, gate = (torch.randn(2, T, H, 128, device="cuda", generator=g) for _ in range(4))
    q, k = (torch.nn.functional.normalize(x, dim=-1) for x in (q, k))
    args = [x.bfloat16() for x in (q, k, v, gate)] + [torch.rand(2, T, H, device="cuda", generator=g)]
    return lambda: list(kda.kda_chunk_fwd(*args))


def test_products_beside_prefills():
    jobs = [_products(1, [(100, 2052, 512), (128, 16416, 1024), (700, 1000, 2048), (60, 4096, 4096)]),
            _products(2, [(128, 4096, 2048), (300, 2048, 512), (2000, 4096, 1024), (1, 2052, 512)]),
            _prefill(3, 700, 8), Layer(90, 4)]
    jobs[3] = (lambda layer: lambda: list(layer()))(jobs[3])
    want = [job() for job in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = []
    for _ in range(20):
        for i, (job, s) in enumerate(zip(jobs, streams)):
            with torch.cuda.stream(s):
                got.append((i, job()))
    torch.cuda.synchronize()
    for i, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i])), i
    assert kda.kda_device_error() == (0, 0)
