"""Memory of calls that are given a stream other than the current one."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _calls(kq):
    """name -> a call that allocates its outputs (and workspaces) itself, on the given stream."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(9, 512, device="cuda", generator=g)
    xh, xb = x.to(torch.float16), x.to(torch.bfloat16)
    w = torch.randn(256, 512, device="cuda", generator=g).to(torch.float16)
    wt = w.t().contiguous()
    L1 = torch.randn(32, 512, device="cuda", generator=g).to(torch.float16)
    L2 = torch.randn(256, 32, device="cuda", generator=g).to(torch.float16)
    omega = torch.randn(512, 48, device="cuda", generator=g)
    xf = kq.Xform.none(512)
    xc, xs, _ = kq.transform_quantize(xh, xf)
    wc, ws, _ = kq.fold_inverse_into_weights_nk(w, xf)
    x8, w8 = kq.quantize_fp8(xb), kq.quantize_fp8(w)
    T = kq.lowrank_down(xh, L1)
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    return {
        "transform_quantize": lambda s: kq.transform_quantize(xh, xf, stream=s),
        "transform_quantize_lowrank": lambda s: kq.transform_quantize_lowrank(xh, xf, L1, stream=s),
        "fold_kn": lambda s: kq.fold_inverse_into_weights(wt, xf, stream=s),
        "fold_nk": lambda s: kq.fold_inverse_into_weights_nk(w, xf, stream=s),
        "lowrank_down": lambda s: kq.lowrank_down(xh, L1, stream=s),
        "svd_lowrank": lambda s: kq.svd_lowrank(w, 32, omega, stream=s),
        "w4a4_linear": lambda s: kq.w4a4_linear(xc, xs, wc, ws, X=xh, L1=L1, L2=L2, stream=s),
        "w4a4_linear_t": lambda s: kq.w4a4_linear_t(xc, xs, wc, ws, T=T, L2=L2, stream=s),
        "quantize_fp8": lambda s: kq.quantize_fp8(xb, stream=s),
        "rmsnorm_quantize_fp8": lambda s: kq.rmsnorm_quantize_fp8(xb, gamma, residual=xb, stream=s),
        "fp8_linear": lambda s: kq.fp8_linear(*x8, *w8, stream=s),
        "fp8_gated_linear": lambda s: kq.fp8_gated_linear(*x8, *w8, stream=s),
    }


NAMES = ["transform_quantize", "transform_quantize_lowrank", "fold_kn", "fold_nk", "lowrank_down", "svd_lowrank", "w4a4_linear",
         "w4a4_linear_t", "quantize_fp8", "rmsnorm_quantize_fp8", "fp8_linear", "fp8_gated_linear"]


def _tensors(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_and_workspaces_are_the_streams_own(kq, name):
    """Outputs, and whatever else the call takes from the allocator, come from memory of the stream that the
    kernels run on: a block of the current stream's could still be written by work pending there."""
    call = _calls(kq)[name]
    expect = _tensors(call(None))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    before = {s["address"] for s in torch.cuda.memory_snapshot()}
    out = call(side)
    segments = torch.cuda.memory_snapshot()
    for t in _tensors(out):
        home = [s for s in segments if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
        assert len(home) == 1 and home[0]["stream"] == side.cuda_stream
    assert all(s["stream"] == side.cuda_stream for s in segments if s["address"] not in before)
    torch.cuda.synchronize()
    for a, b in zip(expect, _tensors(out)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_dropped_output_is_not_reused_under_the_callers_work(kq):
    """An output made on another stream, used on the current one and dropped while that use is pending, is not
    handed to the other stream's next call."""
    call = _calls(kq)["fp8_linear"]
    a = torch.randn(8192, 8192, device="cuda", dtype=torch.bfloat16)
    a @ a, call(None) + 1                                    # kernels loaded
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    here = torch.cuda.current_stream()
    y = call(side)
    here.wait_stream(side)
    for _ in range(200):                                     # a tenth of a second
        a @ a
    z = y + 1
    done = torch.cuda.Event()
    done.record()
    at = y.data_ptr()
    del y
    again = [call(side) for _ in range(3)]
    assert not done.query()
    assert all(t.data_ptr() != at for t in again)
    torch.cuda.synchronize()
    assert all(torch.equal(z, t + 1) for t in again)


def test_given_tensors_come_back(kq):
    """Given outputs are returned themselves, on whatever stream."""
    x = torch.randn(5, 512, device="cuda").to(torch.bfloat16)
    codes, scales = kq.quantize_fp8(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c, s = kq.quantize_fp8(x, codes=codes, stream=side)
    assert c is codes and s is not scales
    torch.cuda.synchronize()
    assert torch.equal(s, scales)
    c, s = kq.quantize_fp8(x, None, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(s, scales)


def test_current_stream_stays(kq):
    """The current stream after a call on another one is the one before it, also when the call is refused."""
    x = torch.randn(5, 512, device="cuda").to(torch.bfloat16)
    side, mine = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(mine):
        kq.quantize_fp8(x, stream=side)
        assert torch.cuda.current_stream() == mine
        with pytest.raises(ValueError):
            kq.quantize_fp8(x.float(), stream=side)
        with pytest.raises(kq.KQError):
            kq.quantize_fp8(x[:, :40].contiguous(), stream=side)
        assert torch.cuda.current_stream() == mine
    torch.cuda.synchronize()


def test_captured_on_a_forked_stream(kq):
    """A graph whose capture forks to another stream for a gated pair (a workspace and two launches) and a
    linear, replayed on new inputs with eager work and waits between."""
    g = torch.Generator(device="cuda").manual_seed(3)
    gu = kq.quantize_fp8(torch.randn(512, 512, device="cuda", generator=g).to(torch.bfloat16))
    dn = kq.quantize_fp8(torch.randn(512, 256, device="cuda", generator=g).to(torch.bfloat16))
    x = torch.randn(9, 512, device="cuda", generator=g).to(torch.bfloat16)

    def block(stream):
        codes, scales = kq.quantize_fp8(x)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        codes, scales = kq.fp8_gated_linear(codes, scales, *gu, stream=stream)
        y = kq.fp8_linear(codes, scales, *dn, dtype=torch.bfloat16, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return y + 1
    side = torch.cuda.Stream()
    block(None), block(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block(side)
    for k in range(3):
        x.copy_(torch.randn(9, 512, device="cuda", generator=g))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, block(None)), k
        assert torch.equal(y, block(side)), k
        torch.cuda.synchronize()
