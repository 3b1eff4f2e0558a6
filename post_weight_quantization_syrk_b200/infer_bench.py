"""Latency of the inference-side matvec with U and V reverted online against
the same packed matvec without rotations.

    python -m post_weight_quantization_syrk_b200.infer_bench    (from the repository root:
                                                                it draws the rotations with synth/)

For each layer shape of the 7B model (4-bit, per-channel grid) and batch 1
and 8, it cycles through 24 distinct packed layers (more bytes than L2, so
the weights stream from HBM as in decode) and reports the CUDA-event time per
kq_reverted_matvec call, issued back to back from Python (at batch 1 the
plain call is bound by the host's launch rate, so its time is an upper bound
of the device time), and the device time per call with the 24 calls captured
in one CUDA graph and replayed.  The rotation parameters are seeded synthetic
draws.

The same layers in 4-bit floating point follow, per format: the matvec of
kq_fp4_matvec on bf16 vectors (batch 1 and 8) and, for 16 and 512 tokens, the
product kq_fp4_gemm with the tokens' quantization (kq_fp4_quantize) in the
time, both as device times of a replayed graph.
"""
import torch

import post_weight_quantization_syrk_b200 as P
from post_weight_quantization_syrk_b200.pipeline import global_scale


def _rht(n, seed, dev):
    import synth
    p = synth.rht_params(n, seed)
    return P.RHT(p.n, p.log2_p, p.m, p.signs.to(dev), None if p.Qm is None else p.Qm.to(dev))


def _graph_us(calls, replays=10):
    """Device time per call of `calls`, captured in order in one graph and replayed."""
    for call in calls:
        call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            for call in calls:
                call()
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    torch.cuda.synchronize()
    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    e0.record()
    for _ in range(replays):
        graph.replay()
    e1.record()
    torch.cuda.synchronize()
    return e0.elapsed_time(e1) / (replays * len(calls)) * 1e3


def fp4(shapes=((4096, 4096), (11008, 4096), (4096, 11008)), batches=(1, 8), tokens=(16, 512), n_layers=24):
    dev = torch.device("cuda")
    info = P.new_info(dev)
    for d_out, d_in in shapes:
        W = torch.randn((d_out, d_in), device=dev) * 0.02
        for name, fmt in (("mx", P.KQ_FP4_MX), ("nv", P.KQ_FP4_NV)):
            def gscale(M):
                return global_scale(M) if fmt == P.KQ_FP4_NV else None
            layers = [P.kq_fp4_quantize(W, fmt, gscale(W), info=info) for _ in range(n_layers)]
            mb = (layers[0].codes.nbytes + layers[0].scales.nbytes) / 1e6
            out = []
            for batch in batches:
                X = torch.randn((batch, d_in), device=dev).bfloat16()
                Y = torch.empty((batch, d_out), dtype=torch.bfloat16, device=dev)
                us = _graph_us([lambda L=L: P.kq_fp4_matvec(L, X, Y) for L in layers])
                out.append(f"batch {batch} {us:.2f} us ({mb / us * 1e3:.0f} GB/s of weights)")
            for T in tokens:
                X = torch.randn((T, d_in), device=dev).bfloat16()
                Y = torch.empty((T, d_out), dtype=torch.bfloat16, device=dev)
                g = gscale(X)
                us = _graph_us([lambda L=L: P.kq_fp4_gemm(P.kq_fp4_quantize(X, fmt, g, info=info), L, Y, info=info)
                                for L in layers])
                out.append(f"{T} tokens {us:.2f} us ({2e-6 * T * d_out * d_in / us:.0f} TFLOP/s)")
            print(f"{d_out}x{d_in} fp4 {name}: " + ", ".join(out) + f", weights {mb:.1f} MB", flush=True)
            del layers
        torch.cuda.empty_cache()
    P.check_info(info)


def main(shapes=((4096, 4096), (11008, 4096), (4096, 11008)), batches=(1, 8), n_layers=24, bits=4):
    dev = torch.device("cuda")
    for d_out, d_in in shapes:
        g = torch.Generator(device=dev)
        g.manual_seed(1)
        layers = []
        for _ in range(n_layers):
            codes = torch.randint(0, 1 << bits, (d_out, d_in), dtype=torch.uint8, device=dev, generator=g)
            layers.append(P.kq_pack_codes(codes, bits))
        del codes
        scales = torch.rand((d_out, 1), device=dev) * 0.01 + 0.001
        zeros = torch.full((d_out, 1), float(1 << (bits - 1)), device=dev)
        T_in, T_out = _rht(d_in, 3, dev), _rht(d_out, 4, dev)
        for batch in batches:
            X = torch.randn((batch, d_in), device=dev)
            Y = torch.empty((batch, d_out), device=dev)
            ws = P.workspace(P.kq_reverted_matvec_workspace_size(d_in, batch), dev)
            us = {}
            for name, a, b in (("reverted", T_in, T_out), ("plain", None, None)):
                for i in range(3 * n_layers):
                    P.kq_reverted_matvec(layers[i % n_layers], bits, scales, zeros, 0, a, b, X, Y, ws)
                torch.cuda.synchronize()
                e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                n = 10 * n_layers
                e0.record()
                for i in range(n):
                    P.kq_reverted_matvec(layers[i % n_layers], bits, scales, zeros, 0, a, b, X, Y, ws)
                e1.record()
                torch.cuda.synchronize()
                us[name] = e0.elapsed_time(e1) / n * 1e3
                # device time: the calls of one pass over the layers as a CUDA graph
                side = torch.cuda.Stream()
                side.wait_stream(torch.cuda.current_stream())
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.stream(side):
                    with torch.cuda.graph(graph, stream=side):
                        for i in range(n_layers):
                            P.kq_reverted_matvec(layers[i], bits, scales, zeros, 0, a, b, X, Y, ws)
                torch.cuda.current_stream().wait_stream(side)
                graph.replay()
                torch.cuda.synchronize()
                e0.record()
                for _ in range(10):
                    graph.replay()
                e1.record()
                torch.cuda.synchronize()
                us[name + "_dev"] = e0.elapsed_time(e1) / (10 * n_layers) * 1e3
                del graph
            gb = d_out * d_in * bits / 8 / 1e9
            print(f"{d_out}x{d_in} {bits}-bit batch {batch}: reverted {us['reverted']:.2f} us "
                  f"(device {us['reverted_dev']:.2f}), plain {us['plain']:.2f} us (device {us['plain_dev']:.2f}, "
                  f"{gb / (us['plain_dev'] * 1e-6):.0f} GB/s of packed weights), weights {gb * 1e3:.1f} MB, "
                  f"rotation overhead on the device {us['reverted_dev'] - us['plain_dev']:.2f} us", flush=True)
        del layers
        torch.cuda.empty_cache()


if __name__ == "__main__":
    main()
    fp4()
