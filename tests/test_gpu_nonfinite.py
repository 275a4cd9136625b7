"""What the linear layer does with NaN and infinities of its own making: pre-activations that overflow binary32, a bias
or a stored pre-activation that is not finite.  The many-row and the few-row kernel, whole and ragged columns, have to
give the same, and a NaN has to stay one."""
import pytest
import torch

from nvfp4_bit_block_amax_b200 import nvfp4 as N
from tests.test_gpu_layer import ACTS, bf16, ok, quant_args

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
ROWS = [4, 20, 100, 200]          # few-row kernels with 16, 32 and 128 tokens a pass, and the large one


def layer(M, Nn, bias, act, dtype=torch.float32, **kw):
    """act(0 + bias): the weight is zero, so that the bias is the pre-activation."""
    a = N.quantize_1d(bf16(M, 128, seed=1))
    b = N.quantize_1d(torch.zeros(Nn, 128, device="cuda", dtype=torch.bfloat16))
    c = N.gemm_epilogue(*quant_args(a), *quant_args(b), M, Nn, 128, bias=bias, activation=act,
                        out_dtype=N.NVFP4_OUT_F32 if dtype == torch.float32 else N.NVFP4_OUT_BF16, **kw)
    ok()
    return c


def biases(Nn, value):
    b = torch.linspace(-3, 3, Nn, device="cuda").bfloat16()
    b[::5] = value
    return b


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("Nn", [64, 131])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_nan_stays(act, M, Nn, dtype):
    bias = biases(Nn, NAN)
    c = layer(M, Nn, bias, act, dtype)
    assert torch.equal(c.isnan(), bias.isnan().expand(M, Nn))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("cols", [8, 16, 131])
def test_nan_stays_in_the_gradient(act, cols):
    zz = bf16(200, (cols + 7) // 8 * 8, seed=2)[:, :cols]
    zz[::7, ::5] = NAN
    dy = torch.ones(200, (cols + 7) // 8 * 8, device="cuda").bfloat16()[:, :cols]     # rows on 16-byte boundaries
    if act == N.NVFP4_ACT_NONE:
        dy, zz = zz, None
    dz, db = N.act_grad(dy, zz, act)
    ok()
    nan = (dy if zz is None else zz).isnan()
    assert torch.equal(dz.isnan(), nan) and torch.equal(db.isnan(), nan.any(0))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("Nn", [64, 131])
@pytest.mark.parametrize("value,want", [(INF, INF), (3e38, None), (-INF, None)])
def test_infinities_through_the_activations(act, M, Nn, value, want):
    """act(inf) = inf for all of them; 3e38 stays itself (its square overflows); at -inf relu and relu2 are 0, and the
    products z P(z), z s(z) with a factor of 0 are NaN, as their definitions are."""
    bias = biases(Nn, value)
    c = layer(M, Nn, bias, act)[:, ::5]
    z = bias[::5].float()
    if value == -INF:
        zero = act in (N.NVFP4_ACT_RELU, N.NVFP4_ACT_RELU2)
        assert (c == 0).all() if zero else (c == -INF).all() if act == N.NVFP4_ACT_NONE else c.isnan().all()
    elif want or act == N.NVFP4_ACT_RELU2:
        assert (c == INF).all()
    else:                                            # z times a reciprocal that may be off by a step
        assert ((c - z).abs() <= z * 2.0 ** -22).all()


@pytest.mark.parametrize("act", ACTS)
def test_both_kernels_on_a_product_that_overflows(act):
    """Finite operands whose z passes binary32: the few-row and the many-row kernel say the same."""
    K, Nn = 128, 72
    x = torch.ones(200, K, device="cuda").bfloat16()
    w = torch.ones(Nn, K, device="cuda").bfloat16()
    w[::3] *= -1
    a, b = N.quantize_1d(x), N.quantize_1d(w)
    big = torch.full((1,), 1e19, device="cuda")
    run = lambda M: N.gemm_epilogue(a.codes[:M], a.scales_mma, big, b.codes, b.scales_mma, big, M, Nn, K,
                                    activation=act, out_dtype=N.NVFP4_OUT_F32)
    many, few = run(200), run(8)
    ok()
    z = torch.where(torch.arange(Nn, device="cuda") % 3 == 0, -INF, INF)
    assert torch.equal(many[:8].nan_to_num(nan=5.0, posinf=INF, neginf=-INF), few.nan_to_num(nan=5.0, posinf=INF, neginf=-INF))
    assert (many[:, z > 0] == INF).all()


@pytest.mark.parametrize("act", ACTS[1:])
def test_slopes_at_infinity_in_whole_and_ragged_columns(act):
    """The slope's limits, 0 and 1 (relu2: 0 and inf), in every column: the last ones of a ragged row go one by one."""
    z = torch.tensor([-INF, INF], device="cuda").repeat(40)[:19].repeat(3, 1)
    pad = torch.zeros(3, 24, device="cuda").bfloat16()
    pad[:, :19] = z.bfloat16()
    dz, _ = N.act_grad(torch.ones_like(pad)[:, :19], pad[:, :19], act)
    ok()
    top = INF if act == N.NVFP4_ACT_RELU2 else 1.0
    assert torch.equal(dz.float(), torch.where(z > 0, top, 0.0))


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("Nn,at", [(64, 0), (131, 129), (131, 130), (300, 255)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_products_maximum(M, Nn, at, dtype):
    for value in (NAN, INF, -INF):
        bias = torch.linspace(-3, 3, Nn, device="cuda").bfloat16()
        bias[at] = value
        amax = torch.zeros(1, device="cuda")
        layer(M, Nn, bias, N.NVFP4_ACT_NONE, dtype, amax_out=amax)
        assert amax.isnan().item() if value != value else amax.item() == INF


@pytest.mark.parametrize("rows,cols", [(5, 64), (130, 131), (4000, 256)])
@pytest.mark.parametrize("bias_grad", [True, False])
def test_the_gradients_maximum(rows, cols, bias_grad):
    for value in (NAN, INF):
        dy = bf16(rows, (cols + 7) // 8 * 8, seed=3)[:, :cols]
        dy[rows - 1, cols - 1] = value
        amax = torch.zeros(1, device="cuda")
        N.act_grad(dy, None, N.NVFP4_ACT_NONE, bias_grad=bias_grad, amax_out=amax)
        ok()
        assert amax.isnan().item() if value != value else amax.item() == INF


@pytest.mark.parametrize("tokens,cols", [(3, 64), (400, 1032), (3000, 64)])
def test_the_movements_maxima(tokens, cols):
    ids = (torch.arange(2 * tokens, device="cuda", dtype=torch.int32) * 5 % 4).reshape(tokens, 2).contiguous()
    plan = N.moe_sort(ids, 4)
    x = bf16(tokens, cols, seed=4)
    x[tokens - 1, cols - 1] = NAN
    first, second = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    N.moe_gather(x, plan, amax_out=first)
    N.moe_combine_grad(x, None, plan, amax_out=second)
    ok()
    assert first.isnan().item() and second.isnan().item()


@pytest.mark.parametrize("rows", [None, 4096])
def test_the_experts_maximum(rows):
    """By expert, few rows and many; the NaN of an expert without tokens counts nowhere."""
    E, Nn, K = 4, 136, 128
    ids = torch.tensor([[0, 1], [1, 3], [0, 3]], dtype=torch.int32, device="cuda")
    plan = N.moe_sort(ids, E, rows=rows)
    a = N.quantize_1d(N.moe_gather(bf16(3, K, seed=5), plan))
    w = N.quantize_2d_experts(torch.zeros(E, 144, K, device="cuda").bfloat16(), columnwise=False)[0]
    codes, scales = w.codes[:, :Nn].contiguous(), w.scales_mma
    for expert, dtype in ((2, torch.float32), (3, torch.float32), (3, torch.bfloat16)):
        bias = torch.ones(E, Nn, device="cuda").bfloat16()
        bias[expert, Nn - 1] = NAN
        amax = torch.zeros(1, device="cuda")
        N.gemm_grouped(*quant_args(a), codes, scales, w.global_scale, plan, plan.rows, Nn, K, bias=bias, amax_out=amax,
                       out_dtype=N.NVFP4_OUT_F32 if dtype == torch.float32 else N.NVFP4_OUT_BF16)
        ok()
        assert amax.item() == 1.0 if expert == 2 else amax.isnan().item()


@pytest.mark.parametrize("M", [16, 272])
def test_a_diverged_layer_shows_in_the_next_one(M):
    """One NaN pre-activation: the maximum is NaN, so the quantizer's scale and all of the next product are."""
    K = 256
    x, w = N.quantize_1d(bf16(M, K, seed=6)), N.quantize_1d(bf16(K, K, seed=7, scale=K ** -0.5))
    bias, amax = torch.zeros(K, device="cuda").bfloat16(), torch.zeros(1, device="cuda")
    for value in (0.0, NAN):
        bias[K - 1] = value
        h = N.gemm_epilogue(*quant_args(x), *quant_args(w), M, K, K, bias=bias, activation=N.NVFP4_ACT_RELU,
                            amax_out=amax)
        q = N.quantize_1d(h, amax=amax)
        y = N.gemm_epilogue(*quant_args(q), *quant_args(w), M, K, K)
        ok()
        assert y.isnan().all() if value != value else y.isfinite().all()
