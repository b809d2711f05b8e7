"""What the wrappers allocate belongs to the stream they are given.  Owned by another stream, a
workspace, which is freed when the call returns, could be handed to that stream's work while the
kernels still use it."""
import os

import pytest
import torch

os.environ.setdefault("RA_WAIT_TIMEOUT_MS", "3000")

pytestmark = pytest.mark.gpu


def test_attention_and_feed_forward_allocate_on_the_stream_they_are_given(monkeypatch):
    import blockwise_exact_attention_ra_gb300 as ra
    from blockwise_exact_attention_ra_gb300.inputs import make_ffn
    q, k, v, do = (torch.randn(1, 512, 2, 64, device="cuda").bfloat16() for _ in range(4))
    x, w1, w2, dy = make_ffn(256, 256, 512, torch.bfloat16, "cuda", 3)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    workspaces = []
    allocate = ra._workspace
    monkeypatch.setattr(ra, "_workspace", lambda n, device: workspaces.append(allocate(n, device)) or workspaces[-1])
    o, lse = ra.ring_attention_fwd(q, k, v, P=2, stream=stream)
    grads = ra.ring_attention_bwd(q, k, v, o, lse, do, P=2, stream=stream)
    y = ra.ffn_fwd(x, w1, w2, 128, stream=stream)
    ffn = ra.ffn_bwd(x, w1, w2, dy, 128, stream=stream)
    stream.synchronize()
    ra.ra_sync_status()
    owner = {b["address"]: s["stream"] for s in torch.cuda.memory_snapshot() for b in s["blocks"] if "address" in b}
    assert len(workspaces) == 4
    for t in (o, lse, *grads, y, *ffn, *workspaces):
        assert owner[t.data_ptr()] == stream.cuda_stream
    # and the values are those of the calls on the current stream
    o2, lse2 = ra.ring_attention_fwd(q, k, v, P=2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(y, ra.ffn_fwd(x, w1, w2, 128))
    for a, b in zip(ffn, ra.ffn_bwd(x, w1, w2, dy, 128)):
        assert torch.equal(a, b)
