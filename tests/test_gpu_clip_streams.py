"""LoRAGradients and lora_clip_gradients on other streams than the one the
object was made on, at once, and in graphs that outlive it (GPU)."""
import pytest
import torch

import expand_gemm_gb300 as eg

pytestmark = pytest.mark.gpu


def gradients(seed, groups=1):
    """Enough of them that a call's partial sums are many, in stacks of `groups`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(groups, 700001, generator=g, device="cuda"),
            torch.randn(groups, 300000, generator=g, device="cuda").bfloat16()]


def expected(grads, groups, max_norm):
    norms = sum(v.double().reshape(groups, -1).square().sum(1) for v in grads).sqrt()
    f = (max_norm / (norms + 1e-6)).clamp(max=1.0)
    return norms, [v.double() * f[:, None] for v in grads]


def check(grads, norms, out, groups, max_norm):
    want_norms, want = expected(grads, groups, max_norm)
    assert bool(((norms.double() - want_norms).abs() <= 20 * 2.0 ** -24 * want_norms).all())
    for o, w in zip(out, want):
        step = 2.0 ** -8 if o.dtype is torch.bfloat16 else 2.0 ** -24
        assert bool(((o.double() - w).abs() <= w.abs() * (step + 22 * 2.0 ** -24) + 2.0 ** -133).all())


def spoil(groups):
    """Memory of every size near the workspace's, taken and filled on the current stream."""
    need = eg.LoRAGradients.make(torch.zeros(groups, 4, device="cuda"), groups).workspace_bytes
    held = [torch.full((max(256, need + d),), 255, dtype=torch.uint8, device="cuda") for d in (0, -256, 256, 0, 0, 0)]
    return held


@pytest.mark.parametrize("groups", [1, 5])
def test_made_on_one_stream_used_on_another_and_dropped(groups):
    made, used = torch.cuda.Stream(), torch.cuda.Stream()
    grads = gradients(1, groups)
    out = [torch.empty_like(v) for v in grads]
    norms = torch.empty(groups, device="cuda")
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(made):
            handle = eg.LoRAGradients.make(grads, groups, out=out)
        with torch.cuda.stream(used):
            torch.cuda._sleep(20_000_000)                   # the call waits in its stream
            eg.lora_clip_gradients(handle, 10.0, norms)
        del handle
        with torch.cuda.stream(made):
            for _ in range(20):
                held = spoil(groups)
                del held
        torch.cuda.synchronize()
        check(grads, norms, out, groups, 10.0)


def test_norms_by_one_object_on_two_streams_at_once():
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    grads = gradients(2, 3)
    handle, norms = eg.LoRAGradients.make(grads, 3), [torch.empty(3, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, n in zip(streams, norms):
            with torch.cuda.stream(s):
                eg.lora_clip_gradients(handle, None, n)
    torch.cuda.synchronize()
    want = expected(grads, 3, 1.0)[0]
    for n in norms:
        assert bool(((n.double() - want).abs() <= 20 * 2.0 ** -24 * want).all())


def test_graphs_outlive_the_object_and_share_nothing():
    sets = []
    for seed in (3, 4):
        grads = gradients(seed, 2)
        out = [torch.empty_like(v) for v in grads]
        norms = torch.empty(2, device="cuda")
        handle = eg.LoRAGradients.make(grads, 2, out=out)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            eg.lora_clip_gradients(handle, 10.0, norms)
        again = torch.cuda.CUDAGraph()
        with torch.cuda.graph(again):
            eg.lora_clip_gradients(handle, 30.0, norms)
        del handle
        sets.append((grads, out, norms, graph, again))
    held = [spoil(2) for _ in range(20)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for k, limit in ((3, 10.0), (4, 30.0)):
        for _ in range(10):
            for s, case in zip(streams, sets):
                with torch.cuda.stream(s):
                    case[k].replay()
        torch.cuda.synchronize()
        for grads, out, norms, *_ in sets:
            check(grads, norms, out, 2, limit)
    assert all(bool((t == 255).all()) for h in held for t in h)


def test_calls_on_one_stream_before_between_and_after_captures():
    """A stream's kept workspace is no captured call's: eager calls run beside a replay."""
    grads, other = gradients(5, 2), gradients(6, 2)
    out, norms = [torch.empty_like(v) for v in grads], [torch.empty(2, device="cuda") for _ in range(2)]
    handle = eg.LoRAGradients.make(grads, 2, out=out)
    side, replays = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        eg.lora_clip_gradients(handle, None, norms[0])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            eg.lora_clip_gradients(handle, 10.0, norms[1])
    quiet = eg.LoRAGradients.make(other, 2)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(replays):
            graph.replay()
        with torch.cuda.stream(side):
            eg.lora_clip_gradients(quiet, None, norms[0])
    torch.cuda.synchronize()
    check(grads, norms[1], out, 2, 10.0)
    want = expected(other, 2, 1.0)[0]
    assert bool(((norms[0].double() - want).abs() <= 20 * 2.0 ** -24 * want).all())
    with torch.cuda.stream(side):
        eg.lora_clip_gradients(handle, 30.0, norms[0])
    torch.cuda.synchronize()
    check(grads, norms[0], out, 2, 30.0)
