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
    dy = torch.ones_like(zz)
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
