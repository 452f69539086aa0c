"""Sequence parallelism on packed documents: SPAttention with the masked local steps, through NCCL
in a one-rank group, against the direct calls (the ranks' local steps of larger groups are run one
after the other in test_masked_gpu.py)."""
import os
import socket

import pytest
import torch
import torch.distributed as dist

from mla_attention_sequence_gb300 import laga
from mla_attention_sequence_gb300.sp import Layout, SPAttention, packed_document_ops

from test_masked_gpu import DSV3, GRADS, built, dev, inputs, slopes, step  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nccl_group():
    with socket.socket(socket.AF_INET, socket.SOCK_STREAM) as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    torch.cuda.set_device(0)
    dist.init_process_group("nccl", rank=0, world_size=1)
    yield
    dist.destroy_process_group()


@pytest.mark.parametrize("prefix", [False, True])
def test_packed_documents_through_the_exchange(nccl_group, prefix):
    x, dout = inputs(1, 384, 384, 2, DSV3, torch.bfloat16, 31)
    st = torch.tensor([[0, 100, 350]], dtype=torch.int32, device=dev())
    pre = torch.tensor([[30, 0]], dtype=torch.int32, device=dev()) if prefix else None
    kw = dict(softcap=20.0, slopes=slopes(2))
    fwd, bwd = packed_document_ops(st, prefix=pre, **kw)
    block = SPAttention(Layout(384, 1), local_fwd=fwd, local_bwd=bwd)
    out, _ = block.forward(*x.values())
    got = {"out": out, **block.backward(dout)}
    lo, hi = laga.key_bounds(st, 384, prefix=pre)
    want = step(x, dout, key_lo=lo, key_hi=hi, causal=not prefix, **kw)
    for k in ("out", *GRADS):
        assert torch.equal(got[k], want[k]), k
    laga.check(dev())
