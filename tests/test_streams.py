"""A helper that launches on `stream` allocates there, and keeps its tensors until both streams are past them.  On the
CPU, with the launches, the streams and record_stream replaced; on the GPU against the allocator itself."""
import contextlib

import pytest
import torch

from nvfp4_bit_block_amax_b200 import build as B
from nvfp4_bit_block_amax_b200 import nvfp4 as N

BF, U8, I32 = torch.bfloat16, torch.uint8, torch.int32


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def z(*shape, dtype=BF, device="cpu"):
    return torch.zeros(*shape, dtype=dtype, device=device)


def calls(device="cpu"):
    """name -> (tensors given, call) for every helper that takes a stream."""
    n = lambda *s, dtype=BF: z(*s, dtype=dtype, device=device)
    plan = N.MoePlan(n(3, dtype=I32), n(2, dtype=I32), n(256, dtype=I32), n(8, 2, dtype=I32))
    op = lambda rows, k, e=1: (n(e, rows, k // 2, dtype=U8), n(e * 16384, dtype=U8), n(e, dtype=torch.float32))
    q = N.Quantized(n(128, 32, dtype=U8), n(128, 4, dtype=U8), n(16384, dtype=U8), n(1, dtype=torch.float32), 128, 64)
    x, y, w = n(8, 64), n(256, 64), n(8, 2, dtype=torch.float32)
    a, b, be = op(256, 64), op(128, 64), op(128, 64, 2)
    t1, t2 = op(64, 256), op(128, 256)
    big, ids, ew = n(256, 128), n(8, 2, dtype=I32), n(2, 64, 64)
    return {
        "quantize_1d": ([y], lambda **k: N.quantize_1d(y, **k)),
        "quantize_2d": ([y], lambda **k: N.quantize_2d(y, **k)),
        "quantize_dual": ([y], lambda **k: N.quantize_dual(y, **k)),
        "mxfp4_quantize": ([y], lambda **k: N.mxfp4_quantize(y, **k)),
        "dequantize": ([q.codes, q.scales, q.global_scale], lambda **k: N.dequantize(q, **k)),
        "gemm": ([*a, *b], lambda **k: N.gemm(*a, *b, 256, 128, 64, **k)),
        "mxfp4_gemm": ([q.codes, q.scales_mma], lambda **k: N.mxfp4_gemm(q, q, **k)),
        "gemm_epilogue": ([*a, *b], lambda **k: N.gemm_epilogue(*a, *b, 256, 128, 64, **k)),
        "act_grad": ([y, plan.counts], lambda **k: N.act_grad(y, y, N.NVFP4_ACT_SILU, plan=plan, **k)),
        "moe_sort": ([ids], lambda **k: N.moe_sort(ids, 2, **k)),
        "moe_gather": ([x, plan.copy_row], lambda **k: N.moe_gather(x, plan, **k)),
        "moe_combine": ([y, w], lambda **k: N.moe_combine(y, plan, w, **k)),
        "moe_combine_grad": ([x, y, w], lambda **k: N.moe_combine_grad(x, y, plan, w, **k)),
        "gemm_grouped": ([*a, *be], lambda **k: N.gemm_grouped(*a, *be, plan, 256, 128, 64, **k)),
        "gemm_grouped_wgrad": ([*t1, *t2], lambda **k: N.gemm_grouped_wgrad(*t1, *t2, plan, 64, 128, 256, **k)),
        "quantize_2d_experts": ([ew], lambda **k: N.quantize_2d_experts(ew, **k)),
    }


NAMES = sorted(calls())


@pytest.fixture
def fake(monkeypatch):
    """Streams 10 (the caller's) and 20; the order of what happens on which."""
    B.build()
    log = {"now": [10], "launched": [], "recorded": {}}

    @contextlib.contextmanager
    def stream(s):
        log["now"].append(s.cuda_stream)
        yield
        log["now"].pop()

    class Lib:
        def __getattr__(self, name):
            f = getattr(real, name)
            if "size" in name or "rows" in name or "bytes" in name:
                return f
            return lambda *a: log["launched"].append((log["now"][-1], a[-1])) or 0

    real = N.lib()
    monkeypatch.setattr(N, "lib", Lib)
    monkeypatch.setattr(N, "_here", lambda *t: None)
    monkeypatch.setattr(N, "workspace", lambda dev=None: z(16384, dtype=U8))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(log["now"][-1]))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a, **k: Stream(h))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: Stream(0))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: log["now"][-1])
    monkeypatch.setattr(N, "_current_device", lambda: 0)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log["recorded"].setdefault(
        t.untyped_storage().data_ptr(), set()).add(s.cuda_stream))
    return log


def results(value):
    if isinstance(value, torch.Tensor):
        return [value]
    if isinstance(value, (tuple, list)):
        return [t for v in value for t in results(v)]
    return [t for t in vars(value).values() if isinstance(t, torch.Tensor)] if hasattr(value, "__dict__") else []


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("stream", [Stream(20), 20])
def test_allocated_launched_and_kept(fake, name, stream):
    given, call = calls()[name]
    out = results(call(stream=stream))
    assert out and fake["launched"] and all(l == (20, 20) for l in fake["launched"])
    at = lambda t: fake["recorded"].get(t.untyped_storage().data_ptr(), set())
    assert all(20 in at(t) for t in given), "an argument may be dropped while `stream` still reads it"
    assert all(10 in at(t) for t in out), "a result may be dropped while the caller's stream still reads it"


@pytest.mark.parametrize("name", NAMES)
def test_nothing_to_keep_on_the_callers_own_stream(fake, name):
    for stream in (None, 10):
        calls()[name][1](stream=stream)
    assert fake["launched"] and all(l == (10, 10) for l in fake["launched"]) and not fake["recorded"]


def test_the_default_streams_handles(fake):
    """0 and 1 stand for the default stream; neither is a stream object's address."""
    for handle in (0, 1):
        x = z(256, 64)
        N.mxfp4_quantize(x, stream=handle)
        assert fake["recorded"].pop(x.untyped_storage().data_ptr()) == {0}
        fake["recorded"].clear()


def test_scratch_is_not_shared_between_calls(fake, monkeypatch):
    """Two calls on two streams, or two captured graphs, may run at once."""
    monkeypatch.setattr(N, "workspace", lambda dev=None: pytest.fail("one workspace for every stream"))
    for name in NAMES:
        calls()[name][1](stream=None)


@pytest.mark.gpu
def test_quantizers_on_two_streams_at_once():
    """Maxima that differ by call: with shared scratch one call's would show in the other's scale."""
    xs = [torch.randn(4096, 2048, device="cuda").bfloat16() * 10.0 ** i for i in range(2)]
    makes = (lambda x, s: N.quantize_1d(x, stream=s), lambda x, s: N.quantize_2d(x, stream=s))
    want = [[m(x, None) for x in xs] for m in makes]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for m, ws in zip(makes, want):
        for _ in range(20):
            got = [m(x, s) for x, s in zip(xs, streams)]
            torch.cuda.synchronize()
            for g, w in zip(got, ws):
                assert torch.equal(g.global_scale, w.global_scale) and torch.equal(g.codes, w.codes)


@pytest.mark.gpu
def test_dropped_results_are_not_handed_out_while_the_other_stream_writes_them():
    side = torch.cuda.Stream()
    dy, zz = (torch.randn(256, 512, device="cuda").bfloat16() for _ in range(2))
    N.act_grad(dy, zz, N.NVFP4_ACT_SILU)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                     # about 10 ms
        N.act_grad(dy, zz, N.NVFP4_ACT_SILU, stream=stream)   # dz and dbias dropped at once
        mine = [torch.full((512,), 7.0, device="cuda") for _ in range(8)]
        mine += [torch.full((256, 512), 7.0, device="cuda", dtype=BF) for _ in range(8)]
        torch.cuda.synchronize()
        assert all((m == 7.0).all() for m in mine)


@pytest.mark.gpu
def test_temporaries_on_another_stream():
    """x sorted, quantized and multiplied on a stream of its own, every intermediate dropped while it is in use."""
    side, E, K, n = torch.cuda.Stream(), 4, 256, 128
    x = torch.randn(300, K, device="cuda").bfloat16()
    ids = (torch.arange(600, device="cuda", dtype=I32) * 7 % E).reshape(300, 2).contiguous()
    w = N.quantize_2d_experts(torch.randn(E, n, K, device="cuda").bfloat16(), columnwise=False)[0]

    def step(s):
        plan = N.moe_sort(ids, E, stream=s)
        q = N.quantize_1d(N.moe_gather(x, plan, stream=s), stream=s)
        c = N.gemm_grouped(q.codes, q.scales_mma, q.global_scale, w.codes, w.scales_mma, w.global_scale, plan,
                           plan.rows, n, K, activation=N.NVFP4_ACT_SILU, stream=s)
        return N.moe_combine(c, plan, residual=None, stream=s)

    want = step(None)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(5):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
        got.append(step(side))
        junk = [torch.full((300, K), float("nan"), device="cuda", dtype=BF) for _ in range(6)]
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.gpu
def test_captured_on_a_forked_stream_and_on_the_default_streams_handle():
    plan_ids = (torch.arange(120, device="cuda", dtype=I32) * 7 % 4).reshape(60, 2).contiguous()
    x, side = torch.randn(60, 128, device="cuda").bfloat16(), torch.cuda.Stream()

    def step(s):
        plan = N.moe_sort(plan_ids, 4, stream=s)
        return N.moe_combine(N.moe_gather(x, plan, stream=s), plan, stream=s)

    want = step(None)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                                        # two graphs, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            out = step(side)
            torch.cuda.current_stream().wait_stream(side)
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            out.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out, want) for _, out in graphs)
    with torch.cuda.stream(side):
        got = [step(handle) for handle in (0, 1)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
