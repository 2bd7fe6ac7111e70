"""The few-token product's ring of stages: nothing is loaded over values that are still to be read,
however busy the SMs are with work of other streams."""

import threading

import pytest
import torch

from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


def test_many_products_beside_other_streams():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x = torch.randn(200, 4096, generator=g, device="cuda").to(torch.bfloat16)
    w = (torch.randn(4096, 8192, generator=g, device="cuda") * 0.02).to(torch.bfloat16)
    narrow = w[:, :640].contiguous()
    rows = (1, 3, 20, 32)
    want = [pb.linear(x[:t], w, activation="gelu") for t in rows]
    torch.cuda.synchronize()
    wrong, done = [], []

    def work():
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(600):
                got, others = [], []
                for t in rows:
                    got.append(pb.linear(x[:t], w, activation="gelu"))
                    others.append(pb.linear(x[:t], narrow, out_dtype=torch.float32))
                others.append(pb.linear(x, narrow))
                others += pb.linear_backward(others[-1], x, narrow, bias=True)
                torch.cuda.current_stream().synchronize()
                wrong.extend(t for t, a, b in zip(rows, got, want) if not torch.equal(a, b))
            done.append(True)

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and len(done) == 4
