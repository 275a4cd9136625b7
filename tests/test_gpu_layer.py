"""The linear layer's epilogue and its gradient, and the layer of experts,
against plain 64-bit implementations.

Tolerances, counted from the arithmetic:
- the product: the operands' values are exact in 64 bits here; the tensor core
  adds K/16 groups of exact products in binary32, each addition off by at most
  2^-22 of S = sum |a b| (its alignment may truncate), and alpha and its
  multiply are rounded: |z - z64| <= (K/16 + 4) 2^-22 S + |bias| 2^-23;
- the activation: slope at most L (1.13 for the gelus, 1.1 for silu, 1 for
  relu, 2|z| for relu2) times that, and its own evaluation, a few binary32
  steps and the fast exponential's 2^-21: 2^-19 (|z| + |z|^2 for relu2);
- the stored value: half a step of its type, plus one binary32 step of the
  residual's addition.
"""
import math

import numpy as np
import pytest
import torch

from nvfp4_bit_block_amax_b200 import inputs as G
from nvfp4_bit_block_amax_b200 import nvfp4 as N
from tests.helpers import to_device_bf16

pytestmark = pytest.mark.gpu
F64 = torch.float64
ACTS = [N.NVFP4_ACT_NONE, N.NVFP4_ACT_RELU, N.NVFP4_ACT_RELU2, N.NVFP4_ACT_GELU, N.NVFP4_ACT_GELU_TANH,
        N.NVFP4_ACT_SILU]
GRID = [0, .5, 1, 1.5, 2, 3, 4, 6]


def act64(act, z):
    return {N.NVFP4_ACT_NONE: lambda: z, N.NVFP4_ACT_RELU: lambda: z.clamp_min(0),
            N.NVFP4_ACT_RELU2: lambda: z.clamp_min(0) ** 2, N.NVFP4_ACT_GELU: lambda: z * torch.special.ndtr(z),
            N.NVFP4_ACT_GELU_TANH: lambda: 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
            N.NVFP4_ACT_SILU: lambda: z * torch.sigmoid(z)}[act]()


def slope64(act, z):
    """The derivatives by hand."""
    if act == N.NVFP4_ACT_NONE:
        return torch.ones_like(z)
    if act == N.NVFP4_ACT_RELU:
        return (z > 0).to(F64)
    if act == N.NVFP4_ACT_RELU2:
        return 2 * z.clamp_min(0)
    if act == N.NVFP4_ACT_GELU:
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == N.NVFP4_ACT_GELU_TANH:
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return s + z * s * (1 - s)


def values64(codes, scales, gs):
    """Exact values of 1D-quantized codes (plain scales)."""
    grid = torch.tensor(GRID + [-g for g in GRID], dtype=F64, device=codes.device)
    v = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], -1).reshape(codes.shape[0], -1, 16)
    s = scales.reshape(codes.shape[0], -1).view(torch.float8_e4m3fn).to(F64)
    return (v * s[:, :, None]).reshape(codes.shape[0], -1) * gs.to(F64)


def bf16(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def step(t):
    """Half a step of a type, relative."""
    return torch.finfo(t).eps / 2


def z_bound(K, S, bias=None):
    b = (K / 16 + 4) * 2.0 ** -22 * S
    return b if bias is None else b + bias.abs().to(F64) * 2.0 ** -23 + S * 2.0 ** -23


def c_bound(act, z, dz, c, dtype):
    slope = 2 * z.abs() + 1 if act == N.NVFP4_ACT_RELU2 else 1.13
    own = 2.0 ** -19 * (z.abs() + (z * z if act == N.NVFP4_ACT_RELU2 else 0))
    e = slope * dz + own
    return e + (c.abs() + e) * (step(dtype) + 2.0 ** -23) + 1e-38


def within(got, want, bound, what=""):
    got = got.to(F64)
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: off by {over.max().item():.3e} over the bound at {over.argmax().item()}"


def operands(M, Nn, K, seed):
    a = N.quantize_1d(bf16(M, K, seed=seed))
    b = N.quantize_1d(bf16(Nn, K, seed=seed + 1, scale=K ** -0.5))
    return a, b, values64(a.codes, a.scales, a.global_scale), values64(b.codes, b.scales, b.global_scale)


def quant_args(q):
    return q.codes, q.scales_mma, q.global_scale


def ok():
    torch.cuda.synchronize()
    assert N.nvfp4_get_error() == 0


# ---------------------------------------------------------------- epilogue --
SHAPES = [(1, 64, 64), (1, 4100, 1024), (3, 130, 192), (8, 8, 64), (17, 1000, 4160), (33, 520, 320), (64, 264, 8192),
          (65, 129, 128), (128, 256, 256), (129, 1024, 1088), (300, 200, 832), (513, 1, 64),
          (5, 40000, 320), (20, 40008, 64), (100, 20000, 256)]     # more tiles than there are CTAs


@pytest.mark.parametrize("M,Nn,K", SHAPES)
@pytest.mark.parametrize("act,dtype", [(N.NVFP4_ACT_SILU, torch.bfloat16), (N.NVFP4_ACT_GELU, torch.float32)])
def test_epilogue_shapes(M, Nn, K, act, dtype):
    a, b, av, bv = operands(M, Nn, K, seed=7 * M + Nn + K)
    bias, ld = bf16(Nn, seed=3, scale=0.3), (Nn + 7) // 8 * 8 + 8
    res = bf16(M, ld, seed=4)[:, :Nn]
    # guards around C and pre: nothing outside [M x N] is written
    cbuf = torch.full((M + 2, ld), 7.0, dtype=dtype, device="cuda")
    pbuf = torch.full((M + 2, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    amax = torch.full((1,), -1.0, device="cuda")
    c = N.gemm_epilogue(*quant_args(a), *quant_args(b), M, Nn, K, bias=bias, activation=act, residual=res,
                        out_dtype=N.NVFP4_OUT_F32 if dtype == torch.float32 else N.NVFP4_OUT_BF16,
                        out=cbuf[1:M + 1, :Nn], pre=pbuf[1:M + 1, :Nn], amax_out=amax)
    ok()
    z = av @ bv.t() + bias.to(F64)
    dz = z_bound(K, av.abs() @ bv.abs().t(), bias)
    want = act64(act, z) + res.to(F64)
    within(c, want, c_bound(act, z, dz, want, dtype) + res.to(F64).abs() * 2.0 ** -23, "C")
    within(pbuf[1:M + 1, :Nn], z, dz + (z.abs() + dz) * step(torch.bfloat16), "pre")
    assert amax.item() == c.float().abs().max().item()
    for buf in (cbuf, pbuf):
        keep = buf.clone()
        keep[1:M + 1, :Nn] = 7.0
        assert (keep == 7.0).all()


@pytest.mark.parametrize("M", [2, 200])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual,pre", [(0, 0, 0), (1, 0, 1), (0, 1, 0)])
def test_epilogue_parts(M, act, bias, residual, pre):
    Nn, K = 264, 448
    a, b, av, bv = operands(M, Nn, K, seed=act)
    bv_bias = bf16(Nn, seed=8) if bias else None
    res = bf16(M, Nn, seed=9) if residual else None
    p = torch.empty(M, Nn, dtype=torch.bfloat16, device="cuda") if pre else None
    c = N.gemm_epilogue(*quant_args(a), *quant_args(b), M, Nn, K, bias=bv_bias, activation=act, residual=res, pre=p)
    ok()
    z = av @ bv.t() + (bv_bias.to(F64) if bias else 0)
    dz = z_bound(K, av.abs() @ bv.abs().t(), bv_bias)
    want = act64(act, z) + (res.to(F64) if residual else 0)
    within(c, want, c_bound(act, z, dz, want, torch.bfloat16) + (res.to(F64).abs() * 2.0 ** -23 if residual else 0))
    if pre:
        within(p, z, dz + (z.abs() + dz) * step(torch.bfloat16))


@pytest.mark.parametrize("M", [4, 300])
def test_epilogue_without_parts_is_the_gemm(M):
    a, b, av, bv = operands(M, 512, 512, seed=21)
    c = N.gemm_epilogue(*quant_args(a), *quant_args(b), M, 512, 512, out_dtype=N.NVFP4_OUT_F32)
    want = av @ bv.t()
    ok()
    within(c, want, z_bound(512, av.abs() @ bv.abs().t()) + want.abs() * 2.0 ** -23)


@pytest.mark.parametrize("M", [5, 260])
def test_epilogue_residual_in_place(M):
    a, b, _, _ = operands(M, 328, 256, seed=31)
    res = bf16(M, 328, seed=32)
    want = N.gemm_epilogue(*quant_args(a), *quant_args(b), M, 328, 256, activation=N.NVFP4_ACT_RELU, residual=res)
    got = res.clone()
    N.gemm_epilogue(*quant_args(a), *quant_args(b), M, 328, 256, activation=N.NVFP4_ACT_RELU, residual=got, out=got)
    ok()
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [3, 200])
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_epilogue_extreme_global_scales(M, scale):
    """Tiny or huge global scales whose product alone leaves binary32: one operand's scale times the other's
    reciprocal range keeps C in range, so the factors have to be applied one after the other."""
    a, b, av, bv = operands(M, 136, 128, seed=41)
    sa, sb = torch.tensor([scale], device="cuda"), torch.tensor([1e-13 if scale < 1 else 1e12], device="cuda")
    ga, gb = a.global_scale * sa, b.global_scale * sb
    c = N.gemm_epilogue(a.codes, a.scales_mma, ga, b.codes, b.scales_mma, gb, M, 136, 128, out_dtype=N.NVFP4_OUT_F32)
    ok()
    av = values64(a.codes, a.scales, ga)
    bv = values64(b.codes, b.scales, gb)
    want = av @ bv.t()
    fits = want.abs() < 3e38
    bound = z_bound(128, av.abs() @ bv.abs().t()) + want.abs() * 2.0 ** -22 + 1.5e-45
    assert ((c.to(F64) - want).abs() <= bound)[fits].all()


def test_epilogue_repeats_bit_for_bit_and_on_another_stream():
    for M in (7, 300):
        a, b, _, _ = operands(M, 1032, 2048, seed=51)
        bias = bf16(1032, seed=52)
        run = lambda s=None: N.gemm_epilogue(*quant_args(a), *quant_args(b), M, 1032, 2048, bias=bias,
                                             activation=N.NVFP4_ACT_GELU_TANH, stream=s)
        first = run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        many = [run(side) for _ in range(4)] + [run() for _ in range(4)]   # both streams at once
        ok()
        assert all(torch.equal(first, m) for m in many)


# ---------------------------------------------------------------- act_grad --
def grad_bound(act, dy, z):
    """slope evaluated to 2^-19 (1 + |z|^2 exp(-z^2/2)-sized terms stay below 2), then dz rounded."""
    d = dy.abs()
    slope = slope64(act, z)
    e = d * 2.0 ** -19 * (1 + slope.abs())
    return e


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,Nn", [(1, 8), (1, 1), (5, 130), (128, 256), (129, 257), (1000, 100), (300, 4100)])
def test_act_grad(act, M, Nn):
    ld = (Nn + 7) // 8 * 8 + 16
    dy, z = bf16(M, ld, seed=61)[:, :Nn], bf16(M, ld, seed=62, scale=2.0)[:, :Nn]
    buf = torch.full((M + 1, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    amax = torch.full((1,), -1.0, device="cuda")
    dz, db = N.act_grad(dy, None if act == N.NVFP4_ACT_NONE else z, act, out=buf[:M, :Nn], amax_out=amax)
    ok()
    want = dy.to(F64) * slope64(act, z.to(F64))
    e = grad_bound(act, dy.to(F64), z.to(F64))
    within(dz, want, e + (want.abs() + e) * step(torch.bfloat16))
    # a thread's 16 rows, 8 warps, 4 parts of row tiles: at most M binary32 additions of |dz|
    within(db, want.sum(0), e.sum(0) + (want.abs() + e).sum(0) * min(M, 48 + M / 512) * 2.0 ** -24 + 1e-38)
    assert amax.item() == dz.float().abs().max().item()
    rest = buf.clone()
    rest[:M, :Nn] = 7.0
    assert (rest == 7.0).all()


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_are_the_activations_differences(act):
    z = torch.linspace(-9, 9, 4001, dtype=F64)
    z = z[z.abs() > 1e-3]        # relu's corner
    h = 1e-5
    diff = (act64(act, z + h) - act64(act, z - h)) / (2 * h)
    assert (diff - slope64(act, z)).abs().max() < 1e-8          # h^2 |f'''| / 6 + 2^-52 |f| / h
    zc = z.to(torch.bfloat16).cuda()[None]
    dz, _ = N.act_grad(torch.ones_like(zc), zc, act)
    want = slope64(act, zc.to(F64))
    within(dz, want, 2.0 ** -18 + want.abs() * step(torch.bfloat16))


@pytest.mark.parametrize("act", ACTS[1:])
def test_act_grad_far_out(act):
    """Large |z|: the slope is 0 or 1 (or 2 z), never NaN."""
    z = torch.tensor([[-3e38, -1e20, -1e5, -100.0, -0.0, 0.0, 100.0, 1e5, 1e15, 1e20, 3e38, 1.0]],
                     device="cuda").bfloat16()
    dz, db = N.act_grad(torch.full_like(z, 0.5), z, act)
    ok()
    want = (0.5 * slope64(act, z.to(F64))).bfloat16()
    fin = torch.isfinite(want)
    assert torch.isfinite(dz[fin]).all() and (dz[fin].float() - want[fin].float()).abs().max() <= \
        want[fin].float().abs().max() * 2 ** -7
    assert not dz.isnan().any()


def test_act_grad_in_place():
    dy, z = bf16(300, 520, seed=63), bf16(300, 520, seed=64)
    want, db = N.act_grad(dy, z, N.NVFP4_ACT_SILU)
    for target in (dy.clone(), z.clone()):
        is_dy = torch.equal(target, dy)
        got, db2 = N.act_grad(target if is_dy else dy, z if is_dy else target, N.NVFP4_ACT_SILU, out=target)
        ok()
        assert torch.equal(got, want) and torch.equal(db, db2)


# -------------------------------------------------------------------- sort --
def sort_reference(ids, experts, rows):
    ids = ids.reshape(-1)
    counts = [[] for _ in range(experts)]
    for c, e in enumerate(ids):
        if 0 <= e < experts:
            counts[e].append(c)
    off, at = [], 0
    for e in range(experts):
        off.append(min(at, rows))
        at += (len(counts[e]) + 127) // 128 * 128
    off.append(min(at, rows))
    row_copy, copy_row = np.full(rows, -1, np.int32), np.full(ids.size, -1, np.int32)
    kept = []
    for e in range(experts):
        keep = counts[e][:off[e + 1] - off[e]]
        kept.append(len(keep))
        for i, c in enumerate(keep):
            row_copy[off[e] + i] = c
            copy_row[c] = off[e] + i
    return np.array(off, np.int32), np.array(kept, np.int32), row_copy, copy_row


def routing(tokens, topk, experts, seed, skew=2.0, bad=0.0):
    rng = np.random.default_rng(seed)
    p = np.exp(skew * rng.standard_normal(experts))
    ids = rng.choice(experts, size=(tokens, topk), p=p / p.sum()).astype(np.int32)   # the same expert twice as well
    if bad:
        wrong = rng.random(ids.shape) < bad
        ids[wrong] = rng.choice([-1, experts, -2**31, 2**31 - 1], size=int(wrong.sum()))
    return torch.from_numpy(ids).cuda()


SORTS = [(1, 1, 1, 0.0), (1, 1, 512, 0.0), (3, 2, 2, 0.0), (37, 2, 8, 0.0), (300, 8, 64, 0.05), (1000, 1, 7, 0.3),
         (1025, 1, 3, 0.0), (5000, 8, 128, 0.01), (20000, 2, 500, 0.0), (64, 4, 512, 0.0), (50, 3, 5, 1.0)]


@pytest.mark.parametrize("tokens,topk,experts,bad", SORTS)
def test_sort(tokens, topk, experts, bad):
    ids = routing(tokens, topk, experts, seed=tokens + experts, bad=bad)
    plan = N.moe_sort(ids, experts)
    again = N.moe_sort(ids, experts)
    ok()
    want = sort_reference(ids.cpu().numpy(), experts, plan.rows)
    for got, twin, w in zip((plan.offsets, plan.counts, plan.row_copy, plan.copy_row.reshape(-1)),
                            (again.offsets, again.counts, again.row_copy, again.copy_row.reshape(-1)), want):
        assert np.array_equal(got.cpu().numpy(), w) and torch.equal(got, twin)


@pytest.mark.parametrize("rows", [128, 384, 1024])
def test_sort_with_too_few_rows_drops_the_last(rows):
    ids = routing(700, 2, 6, seed=rows)
    plan = N.moe_sort(ids, 6, rows=rows)
    ok()
    for got, w in zip((plan.offsets, plan.counts, plan.row_copy, plan.copy_row.reshape(-1)),
                      sort_reference(ids.cpu().numpy(), 6, rows)):
        assert np.array_equal(got.cpu().numpy(), w)


# ------------------------------------------------------ rows there and back --
MOVES = [(1, 1, 1, 8, 0.0), (5, 2, 3, 64, 0.0), (37, 2, 8, 4096, 0.2), (130, 9, 16, 1032, 0.1), (700, 4, 5, 520, 0.0),
         (64, 17, 40, 8192, 0.3), (20, 2, 4, 512, 1.0)]


@pytest.mark.parametrize("tokens,topk,experts,cols,bad", MOVES)
def test_gather(tokens, topk, experts, cols, bad):
    plan = N.moe_sort(routing(tokens, topk, experts, seed=cols, bad=bad), experts)
    x = bf16(tokens + 1, cols + 24, seed=71)[1:, 8:8 + cols]           # strided
    buf = torch.full((plan.rows, cols + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    amax = torch.full((1,), -1.0, device="cuda")
    y = N.moe_gather(x, plan, out=buf[:, :cols], amax_out=amax)
    ok()
    c = plan.row_copy.long()
    want = torch.where((c >= 0)[:, None], x[c.clamp_min(0) // topk], torch.zeros((), dtype=x.dtype, device="cuda"))
    assert torch.equal(y, want) and (buf[:, cols:] == 7.0).all()
    assert amax.item() == want.float().abs().max().item()


@pytest.mark.parametrize("tokens,topk,experts,cols,bad", MOVES)
@pytest.mark.parametrize("weighted,residual", [(True, True), (False, False)])
def test_combine_and_gradient(tokens, topk, experts, cols, bad, weighted, residual):
    plan = N.moe_sort(routing(tokens, topk, experts, seed=cols + 1, bad=bad), experts)
    y = bf16(plan.rows, cols, seed=72)
    y[plan.row_copy < 0] = float("nan")                     # padding rows are not read
    w = torch.rand(tokens, topk, device="cuda") if weighted else None
    res = bf16(tokens, cols, seed=73) if residual else None
    out = N.moe_combine(y, plan, w, residual=res)
    ok()
    r = plan.copy_row.long()
    there = (r >= 0)
    rows = torch.where(there[:, :, None], y[r.clamp_min(0)].to(F64), 0.0)
    wv = w.to(F64) if weighted else torch.ones(tokens, topk, dtype=F64, device="cuda")
    want = (wv[:, :, None] * rows).sum(1) + (res.to(F64) if residual else 0)
    size = (wv[:, :, None] * rows).abs().sum(1) + (res.to(F64).abs() if residual else 0)
    e = size * (topk + 1) * 2.0 ** -24
    within(out, want, e + (want.abs() + e) * step(torch.bfloat16))
    if residual:                                            # in place
        got = res.clone()
        N.moe_combine(y, plan, w, residual=got, out=got)
        assert torch.equal(got, out)

    dout = bf16(tokens, cols, seed=74)
    amax = torch.full((1,), -1.0, device="cuda")
    dy, dw = N.moe_combine_grad(dout, y, plan, w, amax_out=amax)
    ok()
    c = plan.row_copy.long()
    live = (c >= 0)[:, None]
    prod = wv.reshape(-1)[c.clamp_min(0)][:, None] * dout.to(F64)[c.clamp_min(0) // topk]
    want_dy = torch.where(live, prod, 0.0)
    within(dy, want_dy, want_dy.abs() * (step(torch.bfloat16) + 2.0 ** -23))
    assert (dy[~live[:, 0]] == 0).all() and amax.item() == dy.float().abs().max().item()
    want_dw = (rows * dout.to(F64)[:, None]).sum(2)
    # a thread adds cols/256 products, then 5 lane steps and 8 warps
    within(dw, want_dw, (rows * dout.to(F64)[:, None]).abs().sum(2) * (cols / 256 + 16) * 2.0 ** -24 + 1e-38)
    assert (dw[~there] == 0).all()
    none, nodw = N.moe_combine_grad(dout, None, plan, w)
    assert nodw is None and torch.equal(none, dy)


def test_gather_and_combine_are_each_others_gradient():
    """<dout, combine(y)> moves with y as combine_grad says, and <gather(x), g> = <x, combine(g)>: differences of
    functions that are linear in y are exact up to rounding, so whole directions are compared."""
    plan = N.moe_sort(routing(50, 3, 4, seed=5, bad=0.1), 4)
    x, g, w = bf16(50, 64, seed=75), bf16(plan.rows, 64, seed=76), torch.rand(50, 3, device="cuda")
    lhs = (N.moe_gather(x, plan).to(F64) * g.to(F64)).sum()
    rhs = (x.to(F64) * N.moe_combine(g, plan).to(F64)).sum()
    size = (x.to(F64) * N.moe_combine(g, plan).to(F64)).abs().sum()
    assert (lhs - rhs).abs() <= size * step(torch.bfloat16)
    dout, y, d = bf16(50, 64, seed=77), bf16(plan.rows, 64, seed=78), bf16(plan.rows, 64, seed=79)
    dy, dw = N.moe_combine_grad(dout, y, plan, w)
    f = lambda y, w: (N.moe_combine(y, plan, w).to(F64) * dout.to(F64)).sum()
    got = (dy.to(F64) * d.to(F64)).sum()
    size = (N.moe_combine(d, plan, w).to(F64) * dout.to(F64)).abs().sum() + (dy.to(F64) * d.to(F64)).abs().sum()
    assert (f(d, w) - got).abs() <= 2 * size * step(torch.bfloat16)
    dirw = torch.rand(50, 3, device="cuda")
    size = (N.moe_combine(y, plan, dirw).to(F64) * dout.to(F64)).abs().sum()
    assert (f(y, dirw) - (dw.to(F64) * dirw.to(F64)).sum()).abs() <= 2 * size * step(torch.bfloat16)


# ---------------------------------------------------------------- experts ---
EXPERTS = [(1, 1, 1, 64, 64), (16, 2, 8, 264, 128), (5, 2, 3, 1000, 320), (300, 2, 4, 520, 192), (700, 3, 5, 256, 1088),
           (100, 1, 40, 130, 64), (2000, 4, 16, 384, 512),
           (90, 2, 128, 520, 64), (40, 2, 3, 264, 1088), (90, 1, 2, 130, 2112), (60, 1, 1, 300, 4160)]


def expert_operands(tokens, topk, experts, Nn, K, seed, bad=0.0):
    plan = N.moe_sort(routing(tokens, topk, experts, seed=seed, bad=bad), experts)
    xs = N.moe_gather(bf16(tokens, K, seed=seed + 1), plan)
    a = N.quantize_1d(xs)
    qs = [N.quantize_1d(bf16(Nn, K, seed=seed + 2 + e, scale=K ** -0.5 * (1 + e))) for e in range(experts)]
    b = (torch.stack([q.codes for q in qs]), torch.stack([q.scales_mma for q in qs]),
         torch.cat([q.global_scale for q in qs]))
    return plan, a, b, values64(a.codes, a.scales, a.global_scale), \
        [values64(q.codes, q.scales, q.global_scale) for q in qs]


@pytest.mark.parametrize("tokens,topk,experts,Nn,K", EXPERTS)
@pytest.mark.parametrize("act,dtype,full", [(N.NVFP4_ACT_SILU, torch.bfloat16, True),
                                            (N.NVFP4_ACT_NONE, torch.float32, False)])
def test_grouped(tokens, topk, experts, Nn, K, act, dtype, full):
    plan, a, b, av, bvs = expert_operands(tokens, topk, experts, Nn, K, seed=tokens, bad=0.1)
    R, ld = plan.rows, (Nn + 7) // 8 * 8
    bias = bf16(experts, Nn, seed=81) if full else None
    res = bf16(R, ld, seed=82)[:, :Nn] if full else None
    pre = torch.full((R, ld), 7.0, dtype=torch.bfloat16, device="cuda")[:, :Nn] if full else None
    out = torch.full((R, ld), 7.0, dtype=dtype, device="cuda")
    amax = torch.full((1,), -1.0, device="cuda")
    c = N.gemm_grouped(*quant_args(a), *b, plan, R, Nn, K, bias=bias, activation=act, residual=res, pre=pre,
                       out=out[:, :Nn], amax_out=amax,
                       out_dtype=N.NVFP4_OUT_F32 if dtype == torch.float32 else N.NVFP4_OUT_BF16)
    ok()
    seen = torch.zeros(R, dtype=torch.bool, device="cuda")
    for e, (o, n) in enumerate(zip(plan.offsets.tolist(), plan.counts.tolist())):
        s = slice(o, o + n)
        seen[s] = True
        z = av[s] @ bvs[e].t() + (bias[e].to(F64) if full else 0)
        dz = z_bound(K, av[s].abs() @ bvs[e].abs().t(), bias[e] if full else None)
        want = act64(act, z) + (res[s].to(F64) if full else 0)
        within(c[s], want, c_bound(act, z, dz, want, dtype) + (res[s].to(F64).abs() * 2.0 ** -23 if full else 0), e)
        if full:
            within(pre[s], z, dz + (z.abs() + dz) * step(torch.bfloat16), e)
    assert (c[~seen] == 0).all() and (not full or (pre[~seen] == 0).all())
    assert amax.item() == c.float().abs().max().item()
    assert (out[:, Nn:] == 7.0).all()


@pytest.mark.parametrize("experts,tokens,share", [(40, 300, 1), (40, 700, 2), (3, 90, 1), (200, 1000, 3)])
def test_grouped_with_most_rows_at_one_expert(experts, tokens, share):
    """Every share-th token goes to one expert, the others in turn: many passes for one segment, none or one for the
    others, in the kernel for few rows."""
    K = 128
    ids = (torch.arange(tokens, device="cuda", dtype=torch.int32) * 7) % experts
    ids[::share] = experts - 1
    plan = N.moe_sort(ids[:, None].contiguous(), experts)
    a = N.quantize_1d(N.moe_gather(bf16(tokens, K, seed=51), plan))
    w = N.quantize_1d(bf16(experts * 256, K, seed=52))       # 256 rows each, so that the scales divide by expert
    gs = w.global_scale.repeat(experts)
    pre = torch.full((plan.rows, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    c = N.gemm_grouped(*quant_args(a), w.codes, w.scales_mma, gs, plan, plan.rows, 256, K, out_dtype=N.NVFP4_OUT_F32,
                       pre=pre)
    ok()
    av, wv = values64(a.codes, a.scales, a.global_scale), values64(w.codes, w.scales, w.global_scale)
    copy = plan.row_copy.long()
    e = ids.long()[copy.clamp_min(0)]
    want = torch.einsum("rk,rnk->rn", av, wv.reshape(experts, 256, K)[e])
    S = torch.einsum("rk,rnk->rn", av.abs(), wv.abs().reshape(experts, 256, K)[e])
    live = (copy >= 0)[:, None]
    want, S = torch.where(live, want, 0.0), torch.where(live, S, 0.0)
    within(c, want, z_bound(K, S) + want.abs() * 2.0 ** -23)
    within(pre, want, z_bound(K, S) + (want.abs() + z_bound(K, S)) * step(torch.bfloat16))
    assert (c[~live[:, 0]] == 0).all() and (pre[~live[:, 0]] == 0).all()


@pytest.mark.parametrize("tokens,topk,experts,M,Nn,dtype", [
    (1, 1, 1, 64, 64, torch.float32), (16, 2, 8, 264, 136, torch.bfloat16), (300, 2, 5, 40, 520, torch.float32),
    (700, 3, 40, 136, 64, torch.float32), (3000, 2, 4, 512, 256, torch.bfloat16)])
def test_grouped_wgrad(tokens, topk, experts, M, Nn, dtype):
    plan = N.moe_sort(routing(tokens, topk, experts, seed=M, bad=0.1), experts)
    dys, xs = N.moe_gather(bf16(tokens, M, seed=83), plan), N.moe_gather(bf16(tokens, Nn, seed=84), plan)
    a, b = N.quantize_1d(dys, transpose=True), N.quantize_1d(xs, transpose=True)
    got = N.gemm_grouped_wgrad(*quant_args(a), *quant_args(b), plan, M, Nn, plan.rows,
                               out_dtype=N.NVFP4_OUT_F32 if dtype == torch.float32 else N.NVFP4_OUT_BF16)
    ok()
    av, bv = values64(a.codes, a.scales, a.global_scale), values64(b.codes, b.scales, b.global_scale)
    for e in range(experts):
        s = slice(int(plan.offsets[e]), int(plan.offsets[e]) + int(plan.counts[e]))
        want = av[:, s] @ bv[:, s].t()
        dz = z_bound((s.stop - s.start + 63) // 64 * 64, av[:, s].abs() @ bv[:, s].abs().t())
        within(got[e], want, dz + (want.abs() + dz) * step(dtype), e)
        if s.stop == s.start:
            assert (got[e] == 0).all()


@pytest.mark.parametrize("rows", [None, 4096])     # the kernel for few rows, and the large one
def test_products_with_nothing_routed(rows):
    """Every copy dropped: C, pre, the weight gradients and the bias gradients are zeros, whatever was there."""
    E, Nn, K = 4, 264, 128
    plan = N.moe_sort(torch.full((9, 2), E, dtype=torch.int32, device="cuda"), E, rows=rows)
    R = plan.rows
    a, b = N.quantize_1d(bf16(R, K, seed=1)), N.quantize_1d(bf16(E * Nn, K, seed=2))
    b_scales = torch.stack([N.quantize_1d(bf16(Nn, K, seed=3)).scales_mma] * E)
    out, pre = (torch.full((R, Nn), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    amax = torch.full((1,), -1.0, device="cuda")
    N.gemm_grouped(*quant_args(a), b.codes, b_scales, torch.ones(E, device="cuda"), plan, R, Nn, K,
                   bias=bf16(E, Nn, seed=4), activation=N.NVFP4_ACT_SILU, out=out, pre=pre, amax_out=amax)
    t = N.quantize_1d(bf16(R, 64, seed=5), transpose=True)
    dw = N.gemm_grouped_wgrad(*quant_args(t), *quant_args(t), plan, 64, 64, R,
                              out=torch.full((E, 64, 64), 7.0, device="cuda"))
    dz, db = N.act_grad(bf16(R, Nn, seed=6), bf16(R, Nn, seed=7), N.NVFP4_ACT_GELU, plan=plan)
    ok()
    assert all((x == 0).all() for x in (out, pre, dw, dz, db)) and amax.item() == 0


@pytest.mark.parametrize("experts,count", [(1, 40), (2, 100), (3, 129), (16, 33), (70, 5)])
def test_grouped_kernels_agree_where_the_choice_changes(experts, count):
    """The same rows with a row capacity just below and above the one that decides between the two kernels."""
    Nn, K = 264, 320
    ids = torch.arange(experts * count, device="cuda", dtype=torch.int32)[:, None] % experts
    x = bf16(experts * count, K, seed=41)
    q = [N.quantize_1d(bf16(Nn, K, seed=42 + e)) for e in range(experts)]
    b = (torch.stack([w.codes for w in q]), torch.stack([w.scales_mma for w in q]), torch.cat([w.global_scale for w in q]))
    got = []
    need = experts * ((count + 127) // 128 * 128)
    for rows in (need, 160 * experts + 255 + need):
        plan = N.moe_sort(ids.contiguous(), experts, rows=rows // 128 * 128)
        a = N.quantize_1d(N.moe_gather(x, plan))
        c = N.gemm_grouped(*quant_args(a), *b, plan, plan.rows, Nn, K, bias=bf16(experts, Nn, seed=43),
                           activation=N.NVFP4_ACT_GELU_TANH, out_dtype=N.NVFP4_OUT_F32)
        ok()
        got.append(c[:need].to(F64))
        av = values64(a.codes, a.scales, a.global_scale)[:need]
        S = torch.cat([av[e * need // experts:(e + 1) * need // experts].abs()
                       @ values64(w.codes, w.scales, w.global_scale).abs().t() for e, w in enumerate(q)])
    # two kernels, each within the product's bound of the exact sums and two evaluations of the activation
    assert ((got[0] - got[1]).abs() <= 2 * (1.13 * z_bound(K, S) + 2.0 ** -18 * (S + 1))).all()


def test_act_grad_by_expert():
    plan = N.moe_sort(routing(500, 3, 9, seed=3, skew=3.0), 9)
    R, Nn = plan.rows, 260
    dy, z = bf16(R, 264, seed=85)[:, :Nn], bf16(R, 264, seed=86)[:, :Nn]
    empty = plan.row_copy < 0
    dy[empty] = float("nan")                                # padding rows are not read
    amax = torch.full((1,), -1.0, device="cuda")
    dz, db = N.act_grad(dy, z, N.NVFP4_ACT_GELU, plan=plan, amax_out=amax)
    ok()
    assert (dz[empty] == 0).all() and amax.item() == dz.float().abs().max().item()
    want = dy.to(F64) * slope64(N.NVFP4_ACT_GELU, z.to(F64))
    want[empty] = 0
    e = torch.where(empty[:, None], 0.0, grad_bound(N.NVFP4_ACT_GELU, dy.to(F64), z.to(F64)))
    within(dz, want, e + (want.abs() + e) * step(torch.bfloat16))
    for i in range(9):
        s = slice(int(plan.offsets[i]), int(plan.offsets[i + 1]))
        within(db[i], want[s].sum(0), e[s].sum(0) + (want[s].abs() + e[s]).sum(0) * 64 * 2.0 ** -24 + 1e-38)


@pytest.mark.parametrize("offsets,counts", [([0, 128, 64, 10 ** 9], [5, 10 ** 9, -4]), ([-5, -5, -5, -5], [1, 1, 1]),
                                            ([77, 200, 300, 400], [128, 128, 128]), ([512, 384, 128, 0], [9, 9, 9])])
def test_offsets_that_no_sort_gives_stay_in_bounds(offsets, counts):
    """The products clamp unchecked device data: guards around the outputs stay, everything ends, and real segments
    keep their meaning afterwards.  (Every address is formed from clamped values; see fill_groups.)"""
    R, Nn, K = 512, 128, 128
    plan = N.MoePlan(torch.tensor(offsets, dtype=torch.int32, device="cuda"),
                     torch.tensor(counts, dtype=torch.int32, device="cuda"),
                     torch.full((R,), 10 ** 9, dtype=torch.int32, device="cuda"),
                     torch.tensor([[10 ** 9, -7], [5, 2 ** 31 - 1]], dtype=torch.int32, device="cuda"))
    a = N.quantize_1d(bf16(R, K, seed=91))
    b = N.quantize_1d(bf16(3 * Nn, K, seed=92))
    buf = torch.full((R + 2, Nn), 7.0, dtype=torch.bfloat16, device="cuda")
    N.gemm_grouped(*quant_args(a), b.codes, b.scales_mma, torch.ones(3, device="cuda"), plan, R, Nn, K,
                   out=buf[1:R + 1])
    N.gemm_grouped_wgrad(*quant_args(N.quantize_1d(bf16(64, R, seed=93))), *quant_args(N.quantize_1d(bf16(64, R, seed=94))),
                         plan, 64, 64, R)
    N.act_grad(bf16(R, Nn, seed=95), None, N.NVFP4_ACT_NONE, plan=plan)
    N.moe_gather(bf16(2, 64, seed=96), plan)
    y = bf16(R, 64, seed=97)
    out = N.moe_combine(y, plan)
    N.moe_combine_grad(bf16(2, 64, seed=98), y, plan)
    ok()
    assert (buf[0] == 7.0).all() and (buf[R + 1] == 7.0).all()
    assert (out[0] == 0).all() and torch.equal(out[1], y[5])


# ----------------------------------------------------------- run together ---
def experts_step(x, ids, weights, w1, b1, w2, dout, sr_seed=7, rht_seed=11):
    """One forward and backward pass of a layer of experts in the library's own path."""
    experts, ffn, hidden = w1[0].codes.shape[0], w1[0].rows, w1[0].cols
    plan = N.moe_sort(ids, experts)
    R = plan.rows
    amax = [torch.empty(1, device="cuda") for _ in range(5)]
    xs = N.moe_gather(x, plan, amax_out=amax[0])
    qx = N.quantize_1d(xs, amax=amax[0])
    pre = torch.empty(R, ffn, dtype=torch.bfloat16, device="cuda")
    h = N.gemm_grouped(*quant_args(qx), *quant_args(w1[0]), plan, R, ffn, hidden, bias=b1,
                       activation=N.NVFP4_ACT_SILU, pre=pre, amax_out=amax[1])
    qh = N.quantize_1d(h, amax=amax[1])
    y = N.gemm_grouped(*quant_args(qh), *quant_args(w2[0]), plan, R, hidden, ffn)
    out = N.moe_combine(y, plan, weights, residual=x)
    dy, dw = N.moe_combine_grad(dout, y, plan, weights, amax_out=amax[2])
    qdy = N.quantize_1d(dy, rounding=N.NVFP4_SR, sr_seed=sr_seed, amax=amax[2])
    dh = N.gemm_grouped(*quant_args(qdy), *quant_args(w2[1]), plan, R, ffn, hidden)
    dz, db1 = N.act_grad(dh, pre, N.NVFP4_ACT_SILU, plan=plan, amax_out=amax[3])
    qdz = N.quantize_1d(dz, rounding=N.NVFP4_SR, sr_seed=sr_seed + 1, amax=amax[3])
    dxs = N.gemm_grouped(*quant_args(qdz), *quant_args(w1[1]), plan, R, hidden, ffn)
    dx = N.moe_combine(dxs, plan, residual=dout)
    t = lambda m, s: N.quantize_1d(m, transpose=True, rht=True, rht_seed=rht_seed, rounding=s, sr_seed=sr_seed + 2)
    dw1 = N.gemm_grouped_wgrad(*quant_args(t(dz, N.NVFP4_SR)), *quant_args(t(xs, N.NVFP4_RNE)), plan, ffn, hidden, R)
    dw2 = N.gemm_grouped_wgrad(*quant_args(t(dy, N.NVFP4_SR)), *quant_args(t(h, N.NVFP4_RNE)), plan, hidden, ffn, R)
    return out, dx, dw, dw1, db1, dw2


def experts_problem(tokens=200, experts=4, hidden=256, ffn=512):
    x, dout = bf16(tokens, hidden, seed=101), bf16(tokens, hidden, seed=102)
    ids = routing(tokens, 2, experts, seed=103, skew=0.5)
    weights = torch.softmax(torch.randn(tokens, 2, device="cuda", generator=torch.Generator("cuda").manual_seed(5)), 1)
    w1 = N.quantize_2d_experts(bf16(experts, ffn, hidden, seed=104, scale=hidden ** -0.5))
    w2 = N.quantize_2d_experts(bf16(experts, hidden, ffn, seed=105, scale=ffn ** -0.5))
    return x, ids, weights, w1, bf16(experts, ffn, seed=106, scale=0.2), w2, dout


def unswizzle(q, e):
    """Plain scales of expert e's stacked operand, from the layout's formula."""
    r, b = torch.arange(q.rows, device="cuda")[:, None], torch.arange(q.cols // 16, device="cuda")[None]
    chunks = (q.cols // 16 + 3) // 4
    return q.scales_mma[e][((r // 128) * chunks + b // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + b % 4]


def test_layer_of_experts_forward_and_backward():
    """Against the same layer in 64 bits on the dequantized weights.  What remains is the 4-bit rounding of x, h,
    dy, dz: an E2M1 step is at most a third of a value (2 -> 3), so half a step is a sixth, RMS well below; sums over
    hundreds of terms average it out.  A wrong row, expert, scale or missing term is off by the result itself, so
    one part in three of the norm tells them apart."""
    x, ids, weights, w1, b1, w2, dout = experts_problem()
    out, dx, dw, dw1, db1, dw2 = experts_step(x, ids, weights, w1, b1, w2, dout)
    ok()
    E = w1[0].codes.shape[0]
    v1 = torch.stack([values64(w1[0].codes[e], unswizzle(w1[0], e).contiguous(), w1[0].global_scale[e]) for e in range(E)])
    v2 = torch.stack([values64(w2[0].codes[e], unswizzle(w2[0], e).contiguous(), w2[0].global_scale[e]) for e in range(E)])
    leaves = [t.detach().to(F64).requires_grad_() for t in (x, weights, v1, b1, v2)]
    x64, wt64, v1, b64, v2 = leaves
    ref = x64
    for j in range(2):
        e = ids[:, j].long()
        z = torch.einsum("tk,tnk->tn", x64, v1[e]) + b64[e]
        ref = ref + wt64[:, j:j + 1] * torch.einsum("tk,tnk->tn", z * torch.sigmoid(z), v2[e])
    grads = torch.autograd.grad(ref, leaves, dout.to(F64))
    for name, got, want in (("out", out, ref.detach()), ("dx", dx, grads[0]), ("dweights", dw, grads[1]),
                            ("dw1", dw1, grads[2]), ("db1", db1, grads[3]), ("dw2", dw2, grads[4])):
        rel = (got.to(F64) - want).norm() / want.norm()
        assert rel < 1 / 3, (name, rel.item())


def test_layer_of_experts_repeats_and_is_captured():
    args = experts_problem(tokens=70)
    want = experts_step(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        experts_step(*args)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for _ in range(2):                                       # two graphs of the same work, replayed in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(experts_step(*args))
        graphs.append(g)
    for _ in range(2):
        for g in graphs:
            g.replay()
    ok()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, want))
    ids = routing(70, 2, 4, seed=999, skew=3.0)             # new routing through the captured work
    args[1].copy_(ids)
    graphs[1].replay()
    fresh = experts_step(*args)
    ok()
    assert all(torch.equal(a, b) for a, b in zip(outs[1], fresh))


def test_dense_layer_forward_and_backward():
    """x -> act(x w^T + b) + x with gradients, few and many rows, on the dequantized operands in 64 bits."""
    for M in (24, 272):
        K = Nn = 512
        x, dout = bf16(M, K, seed=111), bf16(M, Nn, seed=112)
        qw = N.quantize_2d(bf16(Nn, K, seed=113, scale=K ** -0.5))
        bias = bf16(Nn, seed=114, scale=0.2)
        qx = N.quantize_1d(x)
        pre = torch.empty(M, Nn, dtype=torch.bfloat16, device="cuda")
        out = N.gemm_epilogue(*quant_args(qx), *quant_args(qw), M, Nn, K, bias=bias, activation=N.NVFP4_ACT_GELU_TANH,
                              residual=x, pre=pre)
        amax = torch.empty(1, device="cuda")
        dz, db = N.act_grad(dout, pre, N.NVFP4_ACT_GELU_TANH, amax_out=amax)
        qdz = N.quantize_1d(dz, amax=amax)
        dx = N.gemm_epilogue(*quant_args(qdz), qw.codes_col, qw.scales_mma_col, qw.global_scale, M, K, Nn,
                             residual=dout)
        ok()
        w = values64(qw.codes, qw.scales.repeat_interleave(16, 0), qw.global_scale)
        leaves = [t.detach().to(F64).requires_grad_() for t in (x, bias)]
        ref = act64(N.NVFP4_ACT_GELU_TANH, leaves[0] @ w.t() + leaves[1]) + leaves[0]
        grads = torch.autograd.grad(ref, leaves, dout.to(F64))
        for name, got, want in (("out", out, ref.detach()), ("dx", dx, grads[0]), ("dbias", db, grads[1])):
            rel = (got.to(F64) - want).norm() / want.norm()
            assert rel < 1 / 6, (name, M, rel.item())
