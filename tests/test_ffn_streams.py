"""The stream argument of the feed-forward operators."""
import contextlib

import pytest
import torch

import dense_tiled_gemm_relu_amd as gr
from dense_tiled_gemm_relu_amd import ffn


class Stream:
    """A torch stream's handle; torch gives out a pool stream where ExternalStream gets 0."""
    def __init__(self, handle, device=None):
        self.cuda_stream = handle or 0x9999


def test_a_handle_of_zero_is_the_default_stream(monkeypatch):
    default, handles = Stream(1), []
    default.cuda_stream = 0

    class FrontEnd:
        @staticmethod
        def quantize_rows(x, handle):
            handles.append((handle, current[-1]))

    class X:
        def get_device(self):
            return 3
    current = [None]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()
    monkeypatch.setattr(ffn, "_ops", FrontEnd)
    monkeypatch.setattr(torch.cuda, "device", lambda index: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: default if device == 3 else None)
    other = Stream(4096)
    for stream in (0, 4096, other, default):
        gr.quantize_rows(X(), stream=stream)
    assert [h for h, _ in handles] == [0, 4096, 4096, 0]
    # the results are allocated for the stream that the kernel runs on
    assert all(made.cuda_stream == h for h, made in handles)


def operators():
    """Each operator as (name, function of a stream); its inputs are built here."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")
    x, w, b, dy = randn(40, 264).half(), randn(264).half(), randn(264).half(), randn(40, 264).half()
    wg, dh = (randn(2 * 72, 264) * 0.1).half(), randn(40, 72).half()
    _, mean, rstd = gr.layer_norm(x, w, b, stats=True)
    _, gu = gr.matmul_gated(x, wg, save=True)
    q, s = gr.quantize_rows(x)
    wi, ws = gr.quantize_rows(wg)
    return [("layer_norm", lambda st: gr.layer_norm(x, w, b, stats=True, stream=st)),
            ("layer_norm_backward", lambda st: gr.layer_norm_backward(dy, x, w, mean, rstd, stream=st)),
            ("matmul_gated", lambda st: gr.matmul_gated(x, wg, save=True, stream=st)),
            ("matmul_gated_backward", lambda st: gr.matmul_gated_backward(dh, gu, x, wg, stream=st)),
            ("quantize_rows", lambda st: gr.quantize_rows(x, stream=st)),
            ("matmul_i8", lambda st: (gr.matmul_i8(q, s, wi, ws, stream=st),))]


@pytest.mark.gpu
def test_the_kernels_get_the_handle_that_was_given(monkeypatch):
    own = torch.cuda.Stream()
    cases = operators()
    want = {name: fn(None) for name, fn in cases}
    torch.cuda.synchronize()
    handles = []

    class Recorder:
        def __getattr__(self, name):
            fn = getattr(front_end, name)

            def call(*args):
                handles.append(args[-1])
                return fn(*args)
            return call
    front_end = ffn._ops
    monkeypatch.setattr(ffn, "_ops", Recorder())
    default = torch.cuda.default_stream().cuda_stream
    assert default == 0
    for name, fn in cases:
        for stream, handle in ((0, 0), (default, 0), (torch.cuda.default_stream(), 0), (None, 0),
                               (own, own.cuda_stream), (own.cuda_stream, own.cuda_stream)):
            handles.clear()
            got = fn(stream)
            torch.cuda.synchronize()
            assert handles == [handle], (name, stream)
            assert all(torch.equal(p, q) for p, q in zip(got, want[name]))
        with torch.cuda.stream(own):
            handles.clear()
            got = fn(0)
            torch.cuda.synchronize()
            assert handles == [0], name


@pytest.mark.gpu
def test_a_handle_of_zero_waits_for_the_producer():
    # the producer's products take some milliseconds; the call has to come after them,
    # and what reads its result after it
    x = torch.zeros(512, 1024, device="cuda")
    w = torch.ones(1024, device="cuda")
    final = torch.randn(512, 1024, device="cuda")
    want = gr.layer_norm(final, w)
    busy = torch.randn(8192, 8192, device="cuda")
    torch.cuda.synchronize()
    for _ in range(4):
        busy @ busy
    x.copy_(final)
    got = gr.layer_norm(x, w, stream=0) + 0.0
    x.zero_()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
