"""The norms' backward pass of rows whose gains take more than 64 KB of LDS: captured into a graph,
and called by host threads at once with other widths."""
import threading

import pytest
import torch

from bit_microscaled_quantized_amd import blocks

pytestmark = pytest.mark.gpu


def leaves_of(rows, cols, dtype, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype).requires_grad_()  # noqa: E731
    gate = None if kind is None else rnd(cols) if kind == "channel" else rnd(rows, cols)
    return [rnd(rows, cols), rnd(rows, cols), rnd(cols), rnd(cols)] + ([] if gate is None else [gate])


def grads(leaves):
    x, r, post, pre, *gate = leaves
    h, y = blocks.block_norms(x, r, post, pre, gate[0] if gate else None, 0.5)
    return torch.autograd.grad((h, y), leaves, (torch.ones_like(h), torch.full_like(y, 0.25)))


@pytest.mark.parametrize("rows,cols,dtype,kind", [(70, 9000, torch.bfloat16, "token"), (9, 12001, torch.bfloat16, "channel"),
                                                  (30, 8191, torch.float32, "channel"), (600, 12288, torch.float32, None)])
def test_a_captured_backward_pass(rows, cols, dtype, kind):
    leaves = leaves_of(rows, cols, dtype, kind, 1)
    other = leaves_of(rows, 5 * cols // 6, dtype, kind, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        grads(leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = grads(leaves)
    for n in range(3):
        with torch.no_grad():
            for t, v in zip(leaves, leaves_of(rows, cols, dtype, kind, 10 + n)):
                t.copy_(v)
        graph.replay()
        grads(other)  # eager calls of another width between the replays
        torch.cuda.synchronize()
        for got, want in zip(out, grads(leaves)):
            assert torch.equal(got, want)


def test_host_threads_of_other_widths():
    """Each thread's results are those of the same calls one after another."""
    jobs = [leaves_of(40, cols, torch.bfloat16, "token", cols) for cols in (8200, 10000, 12000, 16000)]
    want = [grads(v) for v in jobs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(10):
                    got = grads(jobs[i])
                    torch.cuda.current_stream().synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        failed.append((i, "other results"))
        except Exception as e:  # noqa: BLE001
            failed.append((i, repr(e)))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
