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


class Buffer:
    """A workspace that notes the streams it is recorded on."""

    def __init__(self, nbytes, device):
        self.nbytes, self.streams = nbytes, []

    def record_stream(self, stream):
        self.streams.append(stream)


def test_layer_workspace_is_recorded_on_every_stream_that_uses_it(monkeypatch):
    d_out, d_in = 256, 512
    current = ["default"]

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            current.append(self.stream)

        def __exit__(self, *exc):
            current.pop()

    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(K, "workspace", Buffer)
    seen = []                                       # (call, its workspace, the stream it runs on)

    def spy(name, ws_at, stream_at):
        def call(*args):
            seen.append((name, args[ws_at], current[-1] if args[stream_at] is None else args[stream_at]))
        monkeypatch.setattr(K, name, call)

    spy("kq_accum_cov", 4, 6)
    spy("kq_chol_inv", 4, 6)
    spy("kq_quantize_layer", 11, 13)
    spy("kq_quantize_layer_multi", 10, 12)
    spy("kq_kron_loss", 5, 6)
    spy("kq_kron_loss_multi", 5, 6)
    monkeypatch.setattr(K, "kq_fp4_quantize", lambda *a, **kw: None)
    lq = pipeline.LayerQuantizer(d_out, d_in, device="cpu")
    X, G = (torch.zeros((4096, d), dtype=torch.bfloat16) for d in (d_in, d_out))
    lq.statistics(X, G, stream="s1")
    lq.factor(stream="s2")
    lq.factor()
    res = lq.alloc_results([(4, 0), (3, 0)])
    lq.quantize(res[0], stream="s1")
    lq.quantize_all(res, stream="s3")
    lq.loss_all(res, stream="s2")
    lq.loss(res[0])
    lq.quantize_fp4(K.KQ_FP4_MX, stream="s4")
    assert [n for n, _, _ in seen] == ["kq_accum_cov"] * 2 + ["kq_chol_inv"] * 2 + [
        "kq_quantize_layer", "kq_quantize_layer_multi", "kq_kron_loss_multi", "kq_kron_loss", "kq_kron_loss"]
    assert {s for _, _, s in seen} == {"default", "s1", "s2", "s3", "s4"}
    for name, ws, stream in seen:
        assert stream in ws.streams, (name, stream)
