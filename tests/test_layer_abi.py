"""The linear layer's and the expert layer's entry points refuse bad arguments on the host, before any launch, and
their host-side sizes are what the header says (no GPU)."""
import pytest
import torch

from nvfp4_bit_block_amax_b200 import build as B
from nvfp4_bit_block_amax_b200 import nvfp4 as N

FAKE = 1 << 20          # 16-byte aligned, never dereferenced: every call below fails validation first
ARG, SHAPE, ALIGN, WORK = (N.NVFP4_ERR_INVALID_ARG, N.NVFP4_ERR_UNSUPPORTED_SHAPE, N.NVFP4_ERR_MISALIGNED,
                           N.NVFP4_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def L():
    B.build()
    return N.lib()


@pytest.fixture(autouse=True)
def nothing_launched(L):
    before = L.nvfp4_kernel_launches()
    yield
    assert L.nvfp4_kernel_launches() == before


def call(f, defaults, **kw):
    assert set(kw) <= set(defaults), kw
    return f(*{**defaults, **kw}.values(), None)


OPERANDS = dict(a=FAKE, sa=FAKE, ga=FAKE, b=FAKE, sb=FAKE, gb=FAKE)
EPILOGUE = dict(M=128, N=128, K=256, bias=FAKE, act=1, res=FAKE, ldr=128, dt=1, c=FAKE, ldc=128, pre=FAKE, ldp=128,
                amax=FAKE)


def check_epilogue(refused):
    for name in OPERANDS:
        assert refused(**{name: None}) == ARG and refused(**{name: FAKE + 2}) == ALIGN
    for name in ("a", "sa", "b", "sb", "c", "res", "pre"):
        assert refused(**{name: FAKE + 8}) == ALIGN
    assert refused(c=None) == ARG and refused(dt=2) == ARG
    for act in (-1, 6):
        assert refused(act=act) == ARG
    for size in ("N", "K"):
        for v in (0, -64, 1 << 31):
            assert refused(**{size: v}) == ARG
    assert refused(K=96) == SHAPE
    for ld in ("ldr", "ldc", "ldp"):
        assert refused(**{ld: 120}) == ARG and refused(**{ld: 132}) == ALIGN
    assert refused(bias=FAKE + 1) == ALIGN and refused(amax=FAKE + 2) == ALIGN


def test_gemm_epilogue(L):
    check_epilogue(lambda **kw: call(L.nvfp4_gemm_epilogue, {**OPERANDS, **EPILOGUE}, **kw))
    assert call(L.nvfp4_gemm_epilogue, {**OPERANDS, **EPILOGUE}, M=0) == ARG


def test_gemm_grouped(L):
    d = {**OPERANDS, "off": FAKE, "cnt": FAKE, "E": 4, **EPILOGUE}
    check_epilogue(lambda **kw: call(L.nvfp4_gemm_grouped, d, **kw))
    refused = lambda **kw: call(L.nvfp4_gemm_grouped, d, **kw)
    assert refused(off=None) == ARG and refused(cnt=None) == ARG
    assert refused(off=FAKE + 2) == ALIGN and refused(cnt=FAKE + 1) == ALIGN
    for e in (0, -1, 513):
        assert refused(E=e) == ARG
    assert refused(E=512, N=1 << 22, ldc=1 << 22, ldr=1 << 22, ldp=1 << 22) == ARG      # E N past 31 bits
    assert refused(M=192) == SHAPE and refused(M=0) == ARG and refused(M=(1 << 23) + 128) == SHAPE


def test_gemm_grouped_wgrad(L):
    d = {**OPERANDS, "off": FAKE, "cnt": FAKE, "E": 4, "M": 128, "N": 128, "K": 256, "dt": 0, "c": FAKE, "ldc": 128}
    refused = lambda **kw: call(L.nvfp4_gemm_grouped_wgrad, d, **kw)
    for name in OPERANDS:
        assert refused(**{name: None}) == ARG and refused(**{name: FAKE + 2}) == ALIGN
    assert refused(K=192) == SHAPE and refused(K=100) == SHAPE           # segments start at multiples of 128
    assert refused(E=0) == ARG and refused(E=513) == ARG and refused(off=None) == ARG and refused(cnt=None) == ARG
    assert refused(ldc=120) == ARG and refused(ldc=132) == ALIGN and refused(c=FAKE + 4) == ALIGN
    assert refused(dt=5) == ARG and refused(M=0) == ARG and refused(N=0) == ARG
    assert refused(E=512, M=1 << 22) == ARG                              # rows of C past 31 bits


def test_act_grad(L):
    need = N.nvfp4_act_grad_workspace_size(300, 128)
    assert need >= 3 * 128 * 4 and N.nvfp4_act_grad_workspace_size(0, 8) == 0
    d = dict(dy=FAKE, ldy=128, z=FAKE, ldz=128, M=300, N=128, act=3, off=None, cnt=None, E=0, dz=FAKE, lddz=128,
             db=FAKE, amax=FAKE, ws=FAKE, wsb=need)
    refused = lambda **kw: call(L.nvfp4_act_grad, d, **kw)
    for m, ld in (("dy", "ldy"), ("z", "ldz"), ("dz", "lddz")):
        assert refused(**{m: None}) == ARG and refused(**{m: FAKE + 8}) == ALIGN
        assert refused(**{ld: 120}) == ARG and refused(**{ld: 132}) == ALIGN
    assert refused(M=0) == ARG and refused(N=0) == ARG and refused(M=1 << 31) == ARG and refused(act=6) == ARG
    assert refused(E=-1) == ARG and refused(E=2) == ARG and refused(E=513, off=FAKE, cnt=FAKE) == ARG
    assert refused(E=2, off=FAKE, cnt=FAKE) == SHAPE                     # 300 rows
    assert refused(db=FAKE + 2) == ALIGN and refused(amax=FAKE + 2) == ALIGN
    assert refused(ws=None) == WORK and refused(wsb=need - 1) == WORK and refused(ws=FAKE + 4) == WORK


def test_moe_sort(L):
    assert N.nvfp4_moe_rows(1, 1) == 128 and N.nvfp4_moe_rows(1, 500) == 128
    assert N.nvfp4_moe_rows(128, 1) == 256               # 128 copies of one expert fit in 128, but 128 + 127 bounds
    assert N.nvfp4_moe_rows(74, 8) == 1152 and N.nvfp4_moe_rows(0, 4) == 0 and N.nvfp4_moe_rows(4, 513) == 0
    need = N.nvfp4_moe_workspace_size(5000, 64)
    assert need >= 64 * 4 and N.nvfp4_moe_workspace_size(0, 1) == 0
    d = dict(ids=FAKE, n=5000, E=64, rows=N.nvfp4_moe_rows(5000, 64), off=FAKE, cnt=FAKE, rc=FAKE, cr=FAKE, ws=FAKE,
             wsb=need)
    refused = lambda **kw: call(L.nvfp4_moe_sort, d, **kw)
    for name in ("ids", "off", "cnt", "rc", "cr"):
        assert refused(**{name: None}) == ARG and refused(**{name: FAKE + 2}) == ALIGN
    for n in (0, -1, 1 << 31, (1 << 31) - 1):            # the last one's rows pass 31 bits
        assert refused(n=n) == ARG
    assert refused(E=0) == ARG and refused(E=513) == ARG and refused(rows=0) == ARG and refused(rows=200) == SHAPE
    assert refused(ws=None) == WORK and refused(wsb=need - 4) == WORK and refused(ws=FAKE + 4) == WORK


def test_every_routing_fits_the_row_capacity():
    for copies, experts in ((1, 1), (129, 2), (300, 3), (64, 64), (1000, 16)):
        rows = N.nvfp4_moe_rows(copies, experts)
        spread = [1] * min(experts - 1, copies - 1)      # as many segments of one copy as there can be
        worst = sum((c + 127) // 128 * 128 for c in spread + [copies - len(spread)])
        assert worst <= rows and rows % 128 == 0


def test_row_movements(L):
    g = dict(x=FAKE, ldx=64, T=8, k=2, cols=64, cr=FAKE, rc=FAKE, rows=256, y=FAKE, ldy=64, amax=FAKE)
    c = dict(y=FAKE, ldy=64, rows=256, cols=64, cr=FAKE, w=FAKE, res=FAKE, ldr=64, T=8, k=2, out=FAKE, ldo=64)
    d = dict(dout=FAKE, ldo=64, y=FAKE, ldy=64, T=8, k=2, cols=64, cr=FAKE, rc=FAKE, rows=256, w=FAKE, dy=FAKE,
             lddy=64, dw=FAKE, amax=FAKE)
    for f, args, mats, words in ((L.nvfp4_moe_gather, g, ("x", "y"), ("cr", "rc", "amax")),
                                 (L.nvfp4_moe_combine, c, ("y", "out", "res"), ("cr", "w")),
                                 (L.nvfp4_moe_combine_grad, d, ("dout", "y", "dy"), ("cr", "rc", "w", "dw", "amax"))):
        refused = lambda **kw: call(f, args, **kw)
        for m in mats:
            assert refused(**{m: FAKE + 8}) == ALIGN
            if m != "res":
                assert refused(**{m: None}) == ARG
        for w in words:
            assert refused(**{w: FAKE + 2}) == ALIGN
        assert refused(cr=None) == ARG
        if "rc" in args:
            assert refused(rc=None) == ARG
        for size in ("T", "k", "rows", "cols"):
            for v in (0, -8, 1 << 31):
                assert refused(**{size: v}) == ARG
        assert refused(T=1 << 20, k=1 << 12) == ARG      # copies past 31 bits
        assert refused(cols=60) == SHAPE
        for ld in [k for k in args if k.startswith("ld")]:
            assert refused(**{ld: 56}) == ARG and refused(**{ld: 68}) == ALIGN


def test_helpers_refuse_mismatched_tensors(monkeypatch):
    """The torch helpers check shapes and types before they hand out pointers (CPU tensors stand in)."""
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    monkeypatch.setattr(N, "_here", lambda *t: None)     # the device check has a test of its own
    f = torch.zeros(1)
    plan = N.MoePlan(*(torch.zeros(s, dtype=torch.int32) for s in (3, 2, 256, (8, 2))))
    assert (plan.experts, plan.rows, plan.tokens, plan.topk) == (2, 256, 8, 2)
    op = (u8(128, 32), u8(512), f)
    with pytest.raises(AssertionError):
        N.gemm_epilogue(u8(128, 16), u8(512), f, *op, 128, 128, 64)             # K mismatch
    with pytest.raises(AssertionError):
        N.gemm_epilogue(u8(128, 32), u8(511), f, *op, 128, 128, 64)             # short scales
    with pytest.raises(AssertionError):
        N.gemm_epilogue(*op, *op, 128, 128, 64, bias=torch.zeros(127, dtype=torch.bfloat16))
    with pytest.raises(AssertionError):
        N.gemm_epilogue(*op, *op, 128, 128, 64, residual=torch.zeros(128, 128))  # not bf16
    with pytest.raises(AssertionError):
        N.gemm_grouped(*op, *op, plan, 256, 128, 64)
    with pytest.raises(AssertionError):
        N.moe_gather(torch.zeros(9, 64, dtype=torch.bfloat16), plan)            # 8 tokens
    with pytest.raises(AssertionError):
        N.moe_combine(torch.zeros(256, 64, dtype=torch.bfloat16), plan, torch.zeros(8, 3))
    with pytest.raises(AssertionError):
        N.moe_sort(torch.zeros(8, 2, dtype=torch.int64), 4)
    with pytest.raises(AssertionError):
        N.act_grad(torch.zeros(8, 64, dtype=torch.bfloat16), torch.zeros(8, 63, dtype=torch.bfloat16), N.NVFP4_ACT_SILU)
    with pytest.raises(AssertionError):
        N.MoePlan(*(torch.zeros(s, dtype=torch.int32) for s in (3, 3, 256, (8, 2))))


def test_helpers_refuse_tensors_that_are_not_on_the_current_device(monkeypatch):
    """Host tensors stand for those of another device: either would hand the kernels addresses they cannot read."""
    monkeypatch.setattr(N, "_current_device", lambda: 0)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    plan = N.MoePlan(*(torch.zeros(s, dtype=torch.int32) for s in (3, 2, 256, (8, 2))))
    op = (u8(128, 32), u8(512), torch.zeros(1))
    for call_ in (lambda: N.gemm_epilogue(*op, *op, 128, 128, 64),
                  lambda: N.act_grad(bf(8, 64), bf(8, 64), N.NVFP4_ACT_SILU),
                  lambda: N.moe_sort(torch.zeros(8, 2, dtype=torch.int32), 4),
                  lambda: N.moe_gather(bf(8, 64), plan),
                  lambda: N.moe_combine(bf(256, 64), plan),
                  lambda: N.moe_combine_grad(bf(8, 64), bf(256, 64), plan),
                  lambda: N.gemm_grouped(u8(256, 32), u8(1024), torch.zeros(1), u8(2, 128, 32), u8(2, 512),
                                         torch.zeros(2), plan, 256, 128, 64),
                  lambda: N.gemm_grouped_wgrad(u8(64, 128), u8(2048), torch.zeros(1), u8(64, 128), u8(2048),
                                               torch.zeros(1), plan, 64, 64, 256),
                  lambda: N.quantize_2d_experts(bf(2, 64, 64))):
        with pytest.raises(AssertionError, match="current CUDA device"):
            call_()


def test_act_grad_refuses_a_plan_that_is_not_on_the_current_device(monkeypatch):
    """Its matrices may all be where they should: the plan's offsets and counts are device pointers too."""
    monkeypatch.setattr(N, "_current_device", lambda: 0)
    matrices = []
    here = N._here
    monkeypatch.setattr(N, "_here", lambda *t: here(*(x for x in t if x.dtype is torch.int32)) if any(
        x.dtype is torch.int32 for x in t) else matrices.append(t))
    monkeypatch.setattr(N, "nvfp4_act_grad", lambda *a, **k: pytest.fail("launched with a plan elsewhere"))
    monkeypatch.setattr(N, "_scratch", lambda n, *where: torch.empty(max(n, 16), dtype=torch.uint8))
    plan = N.MoePlan(*(torch.zeros(s, dtype=torch.int32) for s in (3, 2, 256, (8, 2))))
    dy = torch.zeros(256, 64, dtype=torch.bfloat16)
    with pytest.raises(AssertionError, match="current CUDA device"):
        N.act_grad(dy, dy, N.NVFP4_ACT_SILU, plan=plan)


def test_operands_scales_are_bytes(monkeypatch):
    """A scale to an element: a wider type of as many elements is another array."""
    monkeypatch.setattr(N, "_here", lambda *t: None)
    monkeypatch.setattr(N, "nvfp4_gemm_epilogue", lambda *a, **k: None)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    op = lambda t: (u8(128, 32), torch.zeros(512, dtype=t), torch.zeros(1))
    for wide in (torch.int32, torch.float32, torch.int16):
        for a, b in ((wide, torch.uint8), (torch.uint8, wide)):
            with pytest.raises(AssertionError):
                N.gemm_epilogue(*op(a), *op(b), 128, 128, 64)
    for byte in (torch.uint8, torch.float8_e4m3fn):
        N.gemm_epilogue(*op(byte), *op(byte), 128, 128, 64)
