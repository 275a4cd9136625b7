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
