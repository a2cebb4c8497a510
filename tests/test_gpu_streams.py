"""Reentrancy: the library keeps no per-call state, so calls of different entry points
running at the same time on different streams give, bit for bit, what each gives alone
on the default stream."""

import numpy as np
import pytest
import torch

from expert_ffn_ragged_amd import rd, workloads
from expert_ffn_ragged_amd.workloads import bf16_normal
from tests.gpu_util import say

pytestmark = pytest.mark.gpu

DEV = "cuda"


def dev_i32(v):
    return torch.tensor([int(v)], dtype=torch.int32, device=DEV)


def test_concurrent_calls_on_four_streams_match_calls_alone():
    say("concurrent forward / trans with row split / fp8 trans_rhs / GLU on four streams")
    G, m, k, n = 8, 6144, 512, 768
    gs = torch.from_numpy(workloads.random_sizes(G, m - 100, seed=120, empty=(5,))).to(DEV)
    hot = torch.tensor([4500, 300, 0, 400, 344, 200, 300, 100], dtype=torch.int32, device=DEV)  # split in dW
    x = bf16_normal((m, k), 1.0, 121, DEV)
    w = bf16_normal((G, k, n), 0.05, 122, DEV)
    dy = bf16_normal((m, n), 1.0, 123, DEV)
    g8 = torch.Generator(device=DEV).manual_seed(124)
    x8 = torch.randn((m, k), generator=g8, device=DEV).to(torch.float8_e4m3fn)
    w8 = (torch.randn((G, n, k), generator=g8, device=DEV) * 0.05).to(torch.float8_e4m3fn)
    fused = bf16_normal((m, 2 * n), 2.0, 125, DEV)
    lim = dev_i32(m - 700)
    off = dev_i32(2)
    ws = torch.zeros(rd.trans_workspace_size(m, k, n, G), dtype=torch.uint8, device=DEV)

    def run(outs, streams, wsp):
        rd.ragged_dot(x, w[:4], gs, off, lim, out=outs[0], stream=streams[0])
        rd.trans_ragged_dot(x, dy, hot, out=outs[1], workspace=wsp, stream=streams[1])
        rd.ragged_dot_fp8(x8, w8, gs, trans_rhs=True, out=outs[2], stream=streams[2])
        rd.glu_fwd(fused, lim, out=outs[3], stream=streams[3])

    def fresh():
        return [torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV),
                torch.full((G, k, n), float("nan"), dtype=torch.float32, device=DEV),
                torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV),
                torch.full((m, n), float("nan"), dtype=torch.bfloat16, device=DEV)]

    alone = fresh()
    torch.cuda.synchronize()
    run(alone, [None] * 4, ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32).item()) > 0, "the hot group was not split"
    streams = [torch.cuda.Stream() for _ in range(4)]
    for rep in range(3):
        outs = fresh()
        ws2 = torch.zeros_like(ws)
        torch.cuda.synchronize()
        run(outs, streams, ws2)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, alone)):
            assert torch.equal(a.view(torch.int16 if a.dtype != torch.float32 else torch.int32),
                               b.view(torch.int16 if b.dtype != torch.float32 else torch.int32)), f"rep {rep}: op {i} differs"


def stream_cases():
    """name -> (call(stream) -> outputs, bytes of the workspace it allocates)"""
    bf16 = lambda s, seed, std=1.0: bf16_normal(s, std, seed, DEV)  # noqa: E731
    x, w, dy = bf16((512, 512), 130), bf16((4, 512, 768), 131, 0.05), bf16((512, 768), 132)
    gs = torch.tensor([200, 0, 12, 300], dtype=torch.int32, device=DEV)
    xd, wd, gd = bf16((16, 1024), 133), bf16((2, 1024, 512), 134, 0.05), torch.tensor([9, 7], dtype=torch.int32, device=DEV)
    logits, slots = bf16((600, 32), 135), torch.arange(1200, dtype=torch.int32, device=DEV).view(600, 2)
    ids = torch.randint(0, 100, (9000,), generator=torch.Generator(device=DEV).manual_seed(1), device=DEV, dtype=torch.int32)
    y, g, weights = bf16((1200, 256), 136), bf16((600, 256), 137), torch.rand((600, 2), device=DEV)
    xq, wq = rd.quantize_mx(x, bits=8), rd.quantize_mx(w.transpose(1, 2).contiguous())
    kept = rd.glu_fwd_mx8(dy)[1:]
    d_act = bf16((512, 384), 138)
    return dict(
        ragged_dot=(lambda s: rd.ragged_dot(x, w, gs, stream=s), 0),
        ragged_dot_decode=(lambda s: rd.ragged_dot(xd, wd, gd, stream=s),
                           rd.library().rd_forward_workspace_size(16, 1024, 512, 2, 0)),
        trans_ragged_dot=(lambda s: rd.trans_ragged_dot(x, dy, gs, stream=s), rd.trans_workspace_size(512, 512, 768, 4)),
        glu_fwd=(lambda s: rd.glu_fwd(dy, stream=s), 0),
        unsort_bwd_rows=(lambda s: rd.unsort_bwd_rows(y, y, weights.view(-1), stream=s), 0),
        route=(lambda s: rd.route(logits, 2, stream=s), 0),
        group_rows=(lambda s: rd.group_rows(ids, 100, stream=s), rd.group_rows_workspace_size(9000, 100)),
        dispatch_rows=(lambda s: rd.dispatch_rows(g, slots, stream=s), 0),
        combine_rows_bwd=(lambda s: rd.combine_rows_bwd(g, y, slots, weights, stream=s), 0),
        quantize_mx=(lambda s: rd.quantize_mx(x, stream=s), 0),
        dequantize_mx=(lambda s: rd.dequantize_mx(*xq, stream=s), 0),
        ragged_dot_mx=(lambda s: rd.ragged_dot_mx(*xq, *wq, gs, stream=s), 0),
        glu_fwd_mx8=(lambda s: rd.glu_fwd_mx8(dy, stream=s), 0),
        glu_bwd_mx8=(lambda s: rd.glu_bwd_mx8(*kept, d_act, stream=s), 0),
    )


def as_bytes(t):
    return t.contiguous().view(torch.uint8).view(-1)


def test_outputs_for_another_stream_keep_clear_of_queued_work():
    """Work waits on the current stream, its temporaries already freed on the host, when a call on another stream
    allocates outputs and workspace of the same sizes: neither may see the other's values."""
    a = bf16_normal((4096, 4096), 1.0, 139, DEV)
    b = torch.empty_like(a)
    side = torch.cuda.Stream()
    for name, (call, workspace) in stream_cases().items():
        say(f"outputs of {name} on another stream")
        want = call(None)
        want = want if isinstance(want, tuple) else (want,)
        torch.cuda.synchronize()
        for _ in range(20):
            torch.mm(a, a, out=b)  # the current stream is busy
        temps = [torch.empty_like(t) for t in want]
        if workspace:
            temps.append(torch.empty(workspace, dtype=torch.uint8, device=DEV))
        kept = []
        for t in temps:
            as_bytes(t).fill_(0x5A)
            kept.append(as_bytes(t).clone())
        freed = {t.data_ptr() for t in temps}
        del temps, t
        got = call(side)
        got = got if isinstance(got, tuple) else (got,)
        assert not freed & {t.data_ptr() for t in got}, name
        side.synchronize()
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(as_bytes(g), as_bytes(w)), name
        for k in kept:
            assert bool((k == 0x5A).all()), name
