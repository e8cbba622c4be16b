"""GPU tests of the binding's default workspaces: captured calls beside eager ones of other sizes. Every result is
compared bit for bit with an eager call on the same inputs."""

import threading

import pytest
import torch

import block_scaled_fp8_bfp8_amd as bfp8
import workloads
from tests.gpu_util import announce
from tests.test_gpu_latent_attention import attend, make

pytestmark = pytest.mark.gpu


def decode(gpu, lens, heads, seed, new=None):
    """(inputs, an output, bytes of workspace) of an attention whose blocks may be cut."""
    c, _ = make(gpu, lens, new or [1] * len(lens), heads, 64, seed=seed)
    out = torch.empty(c["q"].shape[0], heads, 512, dtype=torch.bfloat16, device=gpu)
    need = bfp8.latent_attention_workspace_bytes(c["q"].shape[0], len(lens), heads, c["table"].shape[1] * 64)
    assert need > 0
    return c, out, need


def captured(call, side):
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()  # as a user warms up
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            call()
    torch.cuda.synchronize()
    return graph


def other_tensors(gpu):
    """Tensors of many sizes, as a program makes them later on, 600 MB in all."""
    return [torch.full((n,), 7, dtype=torch.uint8, device=gpu) for n in [1 << 20, 2 << 20, 5 << 20, 17 << 20, 34 << 20] * 10]


def test_replay_after_a_larger_call_on_the_stream(gpu):
    """A captured decode, then a call on the same stream that needs more, then other tensors, then the replay."""
    side = torch.cuda.Stream(gpu)
    c, out, need = decode(gpu, [2000], 16, seed=51)
    c2, out2, need2 = decode(gpu, [3000] * 5, 128, seed=52, new=[3] * 5)
    assert need2 > max(need, 1 << 20)
    want, want2 = attend(c), attend(c2)
    announce("workspace growth behind a graph")
    graph = captured(lambda: attend(c, out=out), side)
    with torch.cuda.stream(side):
        attend(c2, out=out2)
        others = other_tensors(gpu)
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(bool((t == 7).all()) for t in others)
        with torch.cuda.stream(side):
            attend(c2, out=out2)
        torch.cuda.synchronize()
        assert torch.equal(out2, want2)


def test_linear_after_a_larger_call_on_the_stream(gpu):
    side = torch.cuda.Stream(gpu)
    w = workloads.weight(1280, 2048, seed=53)
    wq, ws = w.q.to(gpu), w.s.to(gpu)
    x = workloads.act_normal_bf16(600, 2048, seed=54).to(gpu)
    big = workloads.act_normal_bf16(9000, 2048, seed=55).to(gpu)
    out = torch.empty(600, 1280, dtype=torch.bfloat16, device=gpu)
    want = bfp8.linear(x, wq, ws)
    announce("linear workspace growth behind a graph")
    graph = captured(lambda: bfp8.linear(x, wq, ws, out=out), side)
    with torch.cuda.stream(side):
        bfp8.linear(big, wq, ws)
        others = other_tensors(gpu)
    torch.cuda.synchronize()
    for _ in range(3):
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert all(bool((t == 7).all()) for t in others)


def test_two_graphs_of_one_stream_replayed_on_two(gpu):
    side, other = torch.cuda.Stream(gpu), torch.cuda.Stream(gpu)
    cases = [decode(gpu, [5000], 64, seed=56), decode(gpu, [4000, 4500], 64, seed=57)]
    wants = [attend(c) for c, _, _ in cases]
    announce("two graphs, two streams")
    graphs = [captured(lambda c=c, out=out: attend(c, out=out), side) for c, out, _ in cases]
    for _ in range(20):
        for _, out, _ in cases:
            out.fill_(3.0)
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, (side, other)):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for (_, out, _), want in zip(cases, wants):
            assert torch.equal(out, want)


def test_two_host_threads_on_one_stream(gpu):
    """Calls of two launches each, made by two threads on the same stream."""
    side = torch.cuda.Stream(gpu)
    cases = [decode(gpu, [5000], 64, seed=58), decode(gpu, [4000, 4500], 64, seed=59)]
    wants = [attend(c) for c, _, _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    announce("two host threads, one stream")

    def work(i):
        with torch.cuda.stream(side):
            outs[i].extend(attend(cases[i][0]) for _ in range(100))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for got, want in zip(outs, wants):
        assert len(got) == 100 and all(torch.equal(o, want) for o in got)
