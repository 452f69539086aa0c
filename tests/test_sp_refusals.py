"""What SPAttention and the packed documents' local steps refuse, before any collective or launch."""
import os
import socket

import pytest
import torch
import torch.distributed as dist

from mla_attention_sequence_gb300.sp import LibraryOps, Layout, SPAttention, packed_document_ops


@pytest.fixture(scope="module")
def group():
    with socket.socket(socket.AF_INET, socket.SOCK_STREAM) as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=0, world_size=1)
    yield
    dist.destroy_process_group()


STARTS = torch.tensor([[0, 3, 8]], dtype=torch.int32)


def test_overlap_refuses_local_steps_that_it_would_not_call(group):
    fwd, bwd = packed_document_ops(STARTS)
    for kw in (dict(local_fwd=fwd, local_bwd=bwd), dict(local_fwd=fwd), dict(local_bwd=bwd),
               dict(local_fwd=fwd, local_bwd=bwd, ops=LibraryOps())):
        with pytest.raises(ValueError, match="overlap"):
            SPAttention(Layout(8, 1), overlap=True, **kw)
    SPAttention(Layout(8, 1), overlap=True)
    SPAttention(Layout(8, 1), overlap=True, ops=LibraryOps())
    SPAttention(Layout(8, 1), local_fwd=fwd, local_bwd=bwd)


def test_documents_refuse_attention_that_is_not_causal():
    fwd, bwd = packed_document_ops(STARTS, window=2)
    x = [torch.zeros(1, 8, 1, 4), torch.zeros(1, 8, 4), torch.zeros(1, 8, 2), torch.zeros(4, 2), torch.zeros(4, 2)]
    out, lse = torch.zeros(1, 8, 1, 2), torch.zeros(1, 1, 8)
    with pytest.raises(ValueError, match="causal"):
        fwd(*x, 0, False, 0, 0)
    with pytest.raises(ValueError, match="causal"):
        bwd(*x, out, lse, out, 0, False, 0, 0)
    # with prefixes the rows see ahead as far as those reach, whatever `causal` says; CPU tensors are refused later
    fwd, _ = packed_document_ops(STARTS, prefix=torch.tensor([[3, 5]], dtype=torch.int32))
    with pytest.raises(RuntimeError, match="CUDA"):
        fwd(*x, 0, False, 0, 0)


def test_backward_refuses_another_mask_than_the_forwards(group):
    (fwd, bwd), (other, _) = packed_document_ops(STARTS), packed_document_ops(STARTS, window=2)
    saved = (None,) * 7
    for kw in (dict(local_fwd=fwd), dict(local_bwd=bwd), dict(local_fwd=other, local_bwd=bwd)):
        block = SPAttention(Layout(8, 1), **kw)
        block._saved = saved  # as a forward leaves it
        with pytest.raises(ValueError, match="mask"):
            block.backward(None)
    calls = []

    def plain_fwd(*a):
        calls.append("fwd")

    def plain_bwd(*a):
        calls.append("bwd")
        raise KeyError("reached")
    for kw in (dict(local_bwd=plain_bwd), dict(local_fwd=plain_fwd, local_bwd=plain_bwd)):
        block = SPAttention(Layout(8, 1), **kw)
        block._saved = saved
        with pytest.raises(KeyError):
            block.backward(None)
    assert calls == ["bwd", "bwd"]
