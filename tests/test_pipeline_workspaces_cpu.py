"""Workspaces of the pipeline objects across streams, with the library's calls
replaced by recorders (no GPU): no buffer may go back to the allocator while
another stream's kernels are still to use it."""
import torch

from post_weight_quantization_syrk_b200 import _lib as K
from post_weight_quantization_syrk_b200 import pipeline


def test_gated_calibration_takes_a_workspace_per_batch(monkeypatch):
    d, f = 256, 512
    used = []

    def backward(X, Wg, Wu, dH, act, H=None, **kw):
        return torch.empty_like(H), torch.empty_like(H), torch.empty_like(X), None, None

    monkeypatch.setattr(K, "kq_gated_ffn_backward", backward)
    monkeypatch.setattr(K, "kq_accum_cov", lambda A, C, alpha, accumulate, ws, info: used.append((A.shape, ws)))
    cal = pipeline.GatedCalibration(d, f, device="cpu")
    W = torch.zeros((f, d), dtype=torch.bfloat16)
    for t in (4096, 4096, 100):
        cal.add(torch.zeros((t, d), dtype=torch.bfloat16), W, W, torch.zeros((t, f), dtype=torch.bfloat16), 9000)
    batches = [used[i:i + 4] for i in (0, 4, 8)]
    for calls in batches:
        assert all(ws is calls[0][1] for _, ws in calls)
        assert all(ws.numel() >= K.kq_accum_cov_workspace_size(*shape) for shape, ws in calls)
    assert len({id(calls[0][1]) for calls in batches}) == 3
    assert not any(ws is v for _, ws in used for v in vars(cal).values())      # none is kept for the next call
