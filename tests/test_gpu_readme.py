"""The README's mixture-of-experts example as it stands there: its first part
once, its second part captured into a CUDA graph and replayed with new inputs."""
import os
import re

import pytest
import torch

import bit_gemm_quantize_b200 as bgq

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_expert_example_in_a_graph(cuda_device):
    with open(README) as f:
        block = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "moe_route_sort" in b)
    once, step = block.split("\n\n")
    T, E, K, N = 6, 4, 256, 136
    g = torch.Generator().manual_seed(1)
    ns = dict(torch=torch, bgq=bgq, E=E, N=N, x=torch.zeros(T, K, dtype=torch.bfloat16, device=cuda_device),
              logits=torch.zeros(T, E, device=cuda_device),
              expert_weights=[(torch.randn(K, N, generator=g) * 0.02).to(cuda_device) for _ in range(E)])
    exec(once, ns)
    exec(step, ns)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        exec(step, ns)
    ns["x"].copy_(torch.randn(T, K, generator=g).to(torch.bfloat16))
    ns["logits"].copy_(torch.randn(T, E, generator=g))
    graph.replay()
    torch.cuda.synchronize()
    out = ns["out"].double().cpu()
    top = torch.softmax(ns["logits"], 1).topk(2, dim=1)
    x = ns["x"].double().cpu()
    for t in range(T):
        ref, mag = torch.zeros(N, dtype=torch.float64), torch.zeros(N, dtype=torch.float64)
        for w, e in zip(top.values[t].double().cpu(), top.indices[t].tolist()):
            eye = torch.eye(K, device=cuda_device)
            wd = torch.cat([bgq.w4a16_gemv(eye[i:i + 8], ns["pk"]["packed"][e], S=ns["pk"]["S"][e],
                                           alpha=ns["pk"]["alpha"], out="f32") for i in range(0, K, 8)]).double().cpu()
            ref += w * (x[t] @ wd)
            mag += w * (x[t].abs() @ wd.abs())
        # the experts' outputs rounded to fp16, the sum to bf16 (half a step each), and fp32 sums
        assert torch.all((out[t] - ref).abs() <= (2.0 ** -11 + 2.0 ** -8) * (1 + 2.0 ** -8) * mag + 2.0 ** -24)
    assert bgq.device_status() == 0
