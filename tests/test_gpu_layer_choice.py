"""The experts' product around the choice between its kernels, and with routings that leave most experts without rows.
Exact products in 64 bits, with the tolerances of test_gpu_layer."""
import pytest
import torch

from nvfp4_bit_block_amax_b200 import nvfp4 as N
from tests.test_gpu_layer import F64, act64, bf16, c_bound, ok, quant_args, step, values64, within, z_bound

pytestmark = pytest.mark.gpu


def limit(experts):
    """Most rows with which the kernel for few rows is taken, as a multiple of 128."""
    return (159 * experts + 127) // 128 * 128


def weights(experts, Nn, K, seed):
    q = [N.quantize_1d(bf16(Nn, K, seed=seed + e, scale=K ** -0.5)) for e in range(experts)]
    return ((torch.stack([w.codes for w in q]), torch.stack([w.scales_mma for w in q]),
             torch.cat([w.global_scale for w in q])), [values64(w.codes, w.scales, w.global_scale) for w in q])


def check(ids, experts, rows, Nn, K, b, values, full=True):
    """gemm_grouped over the sorted tokens, every part, against the product of each expert."""
    plan = N.moe_sort(ids, experts, rows=rows)
    R, ld = plan.rows, (Nn + 7) // 8 * 8
    a = N.quantize_1d(N.moe_gather(bf16(ids.shape[0], K, seed=31), plan))
    av = values64(a.codes, a.scales, a.global_scale)
    bias = bf16(experts, Nn, seed=32, scale=0.3) if full else None
    res = bf16(R, ld, seed=33)[:, :Nn] if full else None
    pre = torch.full((R, ld), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.full((R, ld), 7.0, dtype=torch.float32, device="cuda")
    amax = torch.empty(1, device="cuda")
    act = N.NVFP4_ACT_GELU_TANH if full else N.NVFP4_ACT_NONE
    c = N.gemm_grouped(*quant_args(a), *b, plan, R, Nn, K, bias=bias, activation=act, residual=res, pre=pre[:, :Nn],
                       out=out[:, :Nn], out_dtype=N.NVFP4_OUT_F32, amax_out=amax)
    ok()
    seen = torch.zeros(R, dtype=torch.bool, device="cuda")
    for e, (o, n) in enumerate(zip(plan.offsets.tolist(), plan.counts.tolist())):
        s = slice(o, o + n)
        seen[s] = True
        z = av[s] @ values[e].t() + (bias[e].to(F64) if full else 0)
        dz = z_bound(K, av[s].abs() @ values[e].abs().t(), bias[e] if full else None)
        want = act64(act, z) + (res[s].to(F64) if full else 0)
        within(c[s], want, c_bound(act, z, dz, want, torch.float32) + (res[s].to(F64).abs() * 2.0 ** -23 if full else 0), e)
        within(pre[s, :Nn], z, dz + (z.abs() + dz) * step(torch.bfloat16), e)
    assert (c[~seen] == 0).all() and (pre[~seen, :Nn] == 0).all()
    assert (out[:, Nn:] == 7.0).all() and (pre[:, Nn:] == 7.0).all()
    assert amax.item() == c.abs().max().item()
    return plan


@pytest.mark.parametrize("K", [320, 2048])           # K as one, and split over a cluster where there are few tiles
@pytest.mark.parametrize("experts", [1, 2, 3, 7, 16, 70])
def test_on_both_sides_of_the_choice(experts, K):
    """The most rows that the one kernel takes and the next multiple of 128; the tokens fit either."""
    Nn = 264
    below = limit(experts)
    segments = below // 128
    # as many full segments as fit, a ragged one for the expert behind the last full one
    counts = [128] * min(experts, segments - 1) + [1] * (experts > segments - 1)
    counts[0] -= 27
    ids = torch.cat([torch.full((c,), e, dtype=torch.int32) for e, c in enumerate(counts)])
    ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(1))].cuda()[:, None].contiguous()
    b, values = weights(experts, Nn, K, seed=40)
    for rows in (below, below + 128):
        plan = check(ids, experts, rows, Nn, K, b, values)
        assert plan.counts.sum().item() == len(ids)


SKEWED = [(64, 256, 2048, 2048, 1), (64, 256, 2048, 2000, 3), (5, 1000, 1024, 190, 1), (3, 264, 4160, 129, 1),
          (140, 128, 1088, 900, 2), (161, 100, 1024, 700, 1), (2, 1024, 4096, 191, 1)]


@pytest.mark.parametrize("experts,Nn,K,tokens,share", SKEWED)
@pytest.mark.parametrize("full", [True, False])
def test_most_rows_at_one_expert_where_k_is_split(experts, Nn, K, tokens, share, full):
    ids = (torch.arange(tokens, device="cuda", dtype=torch.int32) * 7) % experts
    ids[::share] = experts - 1
    q = N.quantize_2d_experts(bf16(experts, (Nn + 15) // 16 * 16, K, seed=51, scale=K ** -0.5), columnwise=False)[0]
    b = (q.codes[:, :Nn].contiguous(), q.scales_mma, q.global_scale)
    r, k = torch.arange(Nn, device="cuda")[:, None], torch.arange(K // 16, device="cuda")[None]
    at = ((r // 128) * ((K // 16 + 3) // 4) + k // 4) * 512 + (r % 32) * 16 + ((r // 32) % 4) * 4 + k % 4
    values = [values64(b[0][e], q.scales_mma[e][at].contiguous(), q.global_scale[e]) for e in range(experts)]
    check(ids[:, None].contiguous(), experts, None, Nn, K, b, values, full)


def time_us(f, n=10):
    for _ in range(3):
        f()
    torch.cuda.synchronize()
    best = float("inf")
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) / n * 1e3)
    return best


def test_a_heavy_expert_does_not_leave_the_gpu_idle():
    """2048 rows over 64 experts of 256 x 2048, or all at one: the heavy expert's rows were once walked by its own four
    CTAs, 30 times as long.  Dealt to all, it stays within a small multiple; 8 leaves room for the noise of a host."""
    E, Nn, K, n = 64, 256, 2048, 2048
    x, b, times = bf16(n, K, seed=61), weights(E, Nn, K, seed=62)[0], []
    for heavy in (False, True):
        ids = torch.arange(n, device="cuda", dtype=torch.int32) % E
        if heavy:
            ids.fill_(E - 1)
        plan = N.moe_sort(ids[:, None].contiguous(), E)
        a = N.quantize_1d(N.moe_gather(x, plan))
        out = torch.empty(plan.rows, Nn, dtype=torch.bfloat16, device="cuda")
        times.append(time_us(lambda: N.gemm_grouped(*quant_args(a), *b, plan, plan.rows, Nn, K, out=out)))
    ok()
    assert times[1] < 8 * times[0], times
