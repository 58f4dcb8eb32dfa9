"""The operators called with a stream of their own while other work is pending,
and from several streams and host threads at once.

Torch's allocator hands a freed block out again at once, in the order of the
stream that it belongs to.  Memory that a call allocates for itself has to
belong to the stream it runs on: a block of the current stream's may still be
read or written by work queued there.
"""
from __future__ import annotations

import gc
import threading

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

DELAY = 20_000_000  # cycles, some 10 ms: far longer than the calls below

# B copied, B and A copied, B read in place and A copied per class of rows
UNALIGNED = [(300, 1025, 999, 0), (700, 900, 1001, 0), (17, 1301, 999, 3), (30, 1200, 1004, 0)]


def _whole(m, n, k, dtype, dev, off=0):
    """Operands of small whole numbers: every partial sum is exact in fp32."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(m * n + k)
    out = []
    for rows in (m, n):
        buf = torch.zeros(rows * k + off, device=dev).to(dtype)
        v = buf[off:].view(rows, k)
        v.copy_(torch.randint(-3, 4, (rows, k), generator=gen, device=dev).float())
        out.append(v)
    return out


@pytest.mark.parametrize("dtype", [torch.float16, torch.float8_e4m3fn])
@pytest.mark.parametrize("m,n,k,off", UNALIGNED)
def test_copies_do_not_take_pending_memory(cuda_dev, m, n, k, off, dtype):
    """A block of the workspace's size, freed while the current stream has still to
    read it, keeps its contents, and the product on another stream is exact."""
    A, B = _whole(m, n, k, dtype, cuda_dev, off)
    want = A.double() @ B.double().t()
    size = g.gemm_workspace(B, A)
    assert size > 0
    out = torch.empty((m, n), device=cuda_dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()  # the block freed next is the one of its size
    temporary = torch.full((size,), 7, dtype=torch.uint8, device=cuda_dev)
    torch.cuda._sleep(DELAY)
    kept = temporary.clone()
    del temporary
    gc.collect()
    g.gemm_fused(B, A, out, stream=side)
    side.synchronize()
    assert torch.equal(out.double(), want)
    torch.cuda.synchronize()
    assert (kept == 7).all()


@pytest.mark.parametrize("m,n,k,off", UNALIGNED)
def test_a_given_workspace(cuda_dev, m, n, k, off):
    A, B = _whole(m, n, k, torch.bfloat16, cuda_dev, off)
    want = A.double() @ B.double().t()
    size = g.gemm_workspace(B, A)
    room = torch.full((size + 512,), 9, dtype=torch.uint8, device=cuda_dev)
    c = g.gemm_fused(B, A, out_dtype=torch.float32, workspace=room[256:256 + size])
    assert torch.equal(c.double(), want)
    assert (room[:256] == 9).all() and (room[256 + size:] == 9).all() and (room[256:256 + size] != 9).any()
    with pytest.raises(g.GemvError) as e:
        g.gemm_fused(B, A, workspace=room[:size - 1])
    assert e.value.status == g.GEMV_ERR_SCRATCH
    with pytest.raises(g.GemvError) as e:
        g.gemm_fused(B, A, workspace=room[8:])
    assert e.value.status == g.GEMV_ERR_ALIGN
    with pytest.raises(ValueError):
        g.gemm_fused(B, A, workspace=room[::2])


@pytest.mark.parametrize("m,n,k,off", UNALIGNED)
def test_copies_in_a_graph(cuda_dev, m, n, k, off):
    A, B = _whole(m, n, k, torch.bfloat16, cuda_dev, off)
    out = torch.empty((m, n), device=cuda_dev)
    g.gemm_fused(B, A, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gemm_fused(B, A, out)
    for scale in (1, -1, 2):
        A.copy_(A.float() * scale)
        want = A.double() @ B.double().t()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.double(), want)


@pytest.mark.parametrize("m,n,k,off", UNALIGNED)
def test_copies_read_what_the_kernel_before_wrote(cuda_dev, m, n, k, off):
    """A product over unaligned vectors that the call just before it, a norm, writes:
    the copy kernel starts early and must not read them before they are there."""
    _, B = _whole(m, n, k, torch.bfloat16, cuda_dev, off)
    signs = torch.randint(0, 2, (m, k), device=cuda_dev).to(torch.bfloat16) * 2 - 1
    weight = torch.ones(k, device=cuda_dev)
    y, out = torch.zeros((m, k), dtype=torch.bfloat16, device=cuda_dev), torch.empty((m, n), device=cuda_dev)
    inputs = [signs, -signs] * 4
    wants = [s.double() @ B.double().t() for s in inputs[:2]]
    outs = [torch.empty_like(out) for _ in inputs]
    torch.cuda.synchronize()
    for s, c in zip(inputs, outs):  # rows of +-1: the norm gives them back
        g.rms_norm_fused(s, weight, eps=0.0, y=y)
        g.gemm_fused(B, y, c)
    torch.cuda.synchronize()
    for i, c in enumerate(outs):
        assert torch.equal(c.double(), wants[i % 2])


def _calls(dev):
    """name -> (call(stream) -> outputs that the call allocates, the value that each
    holds throughout); the inputs are made here."""
    ones = torch.ones((64, 512), device=dev)
    weight, zeros = ones[0], torch.zeros((64, 512), device=dev)
    eye = torch.eye(256, device=dev).to(torch.bfloat16)
    others = 1 - eye
    steps, reset = torch.ones((2, 64, 256), device=dev), torch.full((2, 64, 256), float("-inf"), device=dev)
    return {
        "norm": (lambda s: g.rms_norm_fused(ones, weight, residual=zeros, eps=0.0, stream=s)[::2], (1, 1)),
        "norm_8": (lambda s: g.rms_norm_fused(ones, weight, eps=0.0, eight_bit=True, stream=s)[:2], (448, 1 / 448)),
        "gemm": (lambda s: (g.gemm_fused(eye, eye, residual=others, stream=s),), (1,)),
        "scan": (lambda s: g.gated_scan(steps, reset, stream=s), (1, 1)),
        "grad": (lambda s: g.gated_scan_backward(steps, reset, steps, stream=s), (1, 0, 0)),
    }


@pytest.mark.parametrize("name", ["norm", "norm_8", "gemm", "scan", "grad"])
def test_outputs_do_not_take_pending_memory(cuda_dev, name):
    """Blocks of the outputs' sizes, freed while the current stream has still to read
    them, keep their contents when a call on another stream allocates its outputs."""
    call, want = _calls(cuda_dev)[name]
    side = torch.cuda.Stream()
    sizes = [t.numel() * t.element_size() for t in call(None)]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    temporary = [torch.full((size,), 7, dtype=torch.uint8, device=cuda_dev) for size in sizes]
    torch.cuda._sleep(DELAY)
    kept = [t.clone() for t in temporary]
    del temporary
    gc.collect()
    out = call(side)
    torch.cuda.synchronize()
    assert all((t == 7).all() for t in kept)
    for t, v in zip(out, want):
        assert ((t.double() - v).abs() <= 1e-6 * v).all(), name


def test_outputs_outlive_their_readers(cuda_dev):
    """An output freed while the current stream has still to read it is not handed
    out again on the call's stream."""
    call, _ = _calls(cuda_dev)["gemm"]
    side = torch.cuda.Stream()
    call(side)
    torch.cuda.synchronize()
    (out,) = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(DELAY)
    kept = out.clone()
    del out
    with torch.cuda.stream(side):
        overwritten = torch.full((256, 256), 5, dtype=torch.bfloat16, device=cuda_dev)
    torch.cuda.synchronize()
    assert (kept == 1).all() and (overwritten == 5).all()


def _work(dev, seed):
    """(call -> outputs) of every operator and kernel, on inputs of their own."""
    bf16, e4m3 = torch.bfloat16, torch.float8_e4m3fn

    def rand(i, *shape, dtype=bf16, lo=-1.0, hi=1.0):
        return ref.uniform(shape, dtype, 100 * seed + i, dev, lo, hi)

    def product(i, m, n, k, dtype):
        B, A = rand(i, n, k, dtype=dtype), rand(i + 1, m, k, dtype=dtype)
        return lambda: (g.gemm_fused(B, A, activation="silu"),)

    def norm(i, rows, d, eight):
        x, r, w = rand(i, rows, d), rand(i + 1, rows, d), rand(i + 2, d)
        return lambda: tuple(t for t in g.rms_norm_fused(x, w, residual=r, eight_bit=eight) if t is not None)

    def scan(i, b, t, d):
        x, gate, h0 = rand(i, b, t, d), rand(i + 1, b, t, d, lo=-1.5, hi=0.0), rand(i + 2, b, d, dtype=torch.float32)

        def call():
            h, state = g.gated_scan(x, gate, h0=h0)
            return (h, state, *g.gated_scan_backward(x, gate, h, h0=h0, dstate=state))
        return call

    return [product(1, 1, 2048, 2048, bf16), product(3, 20, 1000, 1024, e4m3), product(5, 600, 2048, 512, bf16),
            product(7, 17, 1301, 999, bf16), product(9, 300, 700, 1001, e4m3), norm(11, 200, 4096, True),
            norm(14, 100, 1001, False), norm(17, 900, 64, True), norm(20, 3, 40000, False), scan(23, 2, 1, 512),
            scan(26, 1, 3000, 256), scan(29, 2, 700, 65), scan(32, 40, 300, 512)]


def _same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(a, b))


def test_several_streams_at_once(cuda_dev):
    """All operators on four streams, nothing waited for between the calls: each
    gives, to the bit, what it gives alone."""
    work = _work(cuda_dev, 1)
    alone = []
    for call in work:
        alone.append(call())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    results = []
    for turn in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                for j in range(len(work)):
                    k = (j * (2 * i + 1) + turn) % len(work)
                    results.append((k, work[k]()))
    torch.cuda.synchronize()
    assert all(_same(out, alone[k]) for k, out in results)
    assert g.gemv_wait_timeouts() == 0


def test_several_host_threads(cuda_dev):
    """Six threads, each on a stream of its own, in different orders."""
    work = _work(cuda_dev, 2)
    alone = []
    for call in work:
        alone.append(call())
        torch.cuda.synchronize()
    wrong = []

    def body(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for turn in range(8):
                kept = []
                for j in range(len(work)):
                    k = (j * (2 * i + 1) + turn * 5 + i) % len(work)
                    kept.append((k, work[k]()))
                s.synchronize()
                wrong.extend((i, turn, k) for k, out in kept if not _same(out, alone[k]))

    threads = [threading.Thread(target=body, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong and g.gemv_wait_timeouts() == 0


def test_forms_of_a_stream(cuda_dev):
    """A stream as torch's object, as a handle, and the default stream as 0."""
    side = torch.cuda.Stream()
    for name, (call, want) in _calls(cuda_dev).items():
        torch.cuda.synchronize()
        for stream in (None, 0, torch.cuda.default_stream(), side, side.cuda_stream):
            out = call(stream)
            torch.cuda.synchronize()
            for t, v in zip(out, want):
                assert ((t.double() - v).abs() <= 1e-6 * v).all(), (name, stream)
