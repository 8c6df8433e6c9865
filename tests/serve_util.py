"""Inputs shared by the tests of the calls that run a quantized layer (no step of the
method here): packed 4-bit weights made with the oracle's packing, and device views."""
from __future__ import annotations

import numpy as np
import torch

import oracle

DEV = "cuda:0"
U32 = 2.0 ** -24   # half a step of float32
U16 = 2.0 ** -8    # half a step of bf16


def packed_weights(d_in, d_out, g, seed):
    """codes, and (qweight uint32, scales bits, zeros bits) as gptq_pack lays them out."""
    rng = np.random.default_rng(seed)
    G = d_in if g == -1 else g
    ng = d_in // G
    codes = rng.integers(0, 16, size=(d_out, d_in), dtype=np.uint8)
    scales = oracle.fp16_rne(np.exp(rng.uniform(-6.0, -2.0, size=(d_out, ng))))
    zeros = rng.integers(0, 16, size=(d_out, ng)).astype(np.float64)
    return codes, oracle.pack_rows(codes, 4), oracle.fp16_bits(scales), oracle.fp16_bits(zeros)


def dev_weights(qw, s16, z16):
    Q = torch.from_numpy(qw.astype(np.uint32).view(np.int32)).to(DEV)
    S = torch.from_numpy(s16.view(np.int16)).to(DEV)
    Z = None if z16 is None else torch.from_numpy(z16.view(np.int16)).to(DEV)
    return Q, S, Z


def abs_terms(qw, s16, z16, sym, g, d_in):
    """s (q + z) per weight, float64: what the bound of sum x q - z sum x is made of."""
    q = oracle.unpack_rows(qw, 4, d_in).astype(np.float64)
    G = d_in if g == -1 else g
    k = np.arange(d_in) // G
    s = s16.view(np.float16).astype(np.float64)[:, k]
    z = 8.0 if sym else z16.view(np.float16).astype(np.float64)[:, k]
    return s * (q + z)


def replayed(call, outputs, times=3):
    """Captures call() into a graph and replays it `times` times with other work between the
    replays; the outputs (tensors that call() writes) after each replay, on the host."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    got = []
    for _ in range(times):
        for t in outputs:
            t.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got.append([t.clone().cpu() for t in outputs])
    return got
