"""The linear layer's and the expert layer's operators: what is computed, on what, and at what sizes.

Each case names one operator ("op"):
  linear    C = act(A . B^T + bias) + residual from NVFP4 operands; optionally the pre-activation and max |C|
  act_grad  dz = dy * act'(z), the bias gradient (column sums of dz) and max |dz|
  experts   the linear layer over rows sorted by expert, one weight per expert
  wgrad     one weight gradient per expert from the two transposed operands of the sorted rows
  route     the stable sort of token copies by expert and the gather of their rows, with max |x|
  combine   the weighted sum of a token's copies plus a residual
  combine_grad  its gradients with respect to the copies and the weights

Rows sorted by expert lie in segments that start at multiples of 128; the rows between a segment's last token and
the next segment are padding and hold zeros, here and in every output.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "relu2", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one token through an MLP's first linear layer (the 4096 x 14336 MLP): latency and weight traffic
        {"name": "linear_token", "op": "linear", "M": 1, "N": 14336, "K": 4096, "act": "silu", "bias": True,
         "residual": False, "pre": False, "amax": False, "out": "bf16"},
        # a mixed batch of ragged size through every part of the epilogue
        {"name": "linear_ragged", "op": "linear", "M": 1000, "N": 4100, "K": 4160, "act": "gelu", "bias": True,
         "residual": True, "pre": True, "amax": True, "out": "bf16"},
        # fprop of the MLP training step (16384 tokens, 8192 -> 28672), keeping what the backward pass needs
        {"name": "linear_step", "op": "linear", "M": 16384, "N": 28672, "K": 8192, "act": "gelu_tanh", "bias": True,
         "residual": False, "pre": True, "amax": True, "out": "bf16"},
        # the same two layers' activation and bias gradients
        {"name": "act_grad_ragged", "op": "act_grad", "M": 1000, "N": 4100, "act": "gelu", "amax": True},
        {"name": "act_grad_step", "op": "act_grad", "M": 16384, "N": 28672, "act": "gelu_tanh", "amax": True},
        # decoding 16 sequences through 8 experts of the 4096 x 14336 MLP: every expert's weight is read once
        {"name": "experts_few", "op": "experts", "T": 16, "k": 2, "E": 8, "N": 14336, "K": 4096, "act": "silu",
         "bias": True, "pre": False, "amax": False},
        # a training batch of 8192 tokens through the same experts
        {"name": "experts_batch", "op": "experts", "T": 8192, "k": 2, "E": 8, "N": 14336, "K": 4096, "act": "silu",
         "bias": True, "pre": True, "amax": True},
        # weight gradients of 16 smaller experts, in fp32 as an optimizer takes them
        {"name": "wgrad_batch", "op": "wgrad", "T": 8192, "k": 2, "E": 16, "N": 4096, "K": 2048, "out": "f32"},
        # routing of a few decoded tokens, and of a training batch
        {"name": "route_few", "op": "route", "T": 37, "k": 2, "E": 8, "H": 4096},
        {"name": "route_batch", "op": "route", "T": 16384, "k": 2, "E": 8, "H": 8192},
        # the way back: a training batch with the residual, and the gradient with many small experts
        {"name": "combine_batch", "op": "combine", "T": 16384, "k": 2, "E": 8, "H": 8192, "residual": True},
        {"name": "combine_grad_many", "op": "combine_grad", "T": 8192, "k": 8, "E": 64, "H": 2048, "amax": True},
    ]


def _log(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "act_grad", "experts", "experts", "wgrad", "route", "combine",
                     "combine_grad"))
    flag = lambda: rng.random() < 0.5
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "K": _log(rng, 64, 8192, 64),
                "act": rng.choice(ACTS), "bias": flag(), "residual": flag(), "pre": flag(), "amax": flag(),
                "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "act_grad":
        return {"op": op, "M": _log(rng, 1, 8192), "N": _log(rng, 64, 16384), "act": rng.choice(ACTS[1:]),
                "amax": flag()}
    e = _log(rng, 2, 64)
    case = {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, min(e, 8)), "E": e}
    if op == "experts":
        case.update(N=_log(rng, 128, 4096, 8), K=_log(rng, 128, 4096, 64), act=rng.choice(ACTS), bias=flag(),
                    pre=flag(), amax=flag())
    elif op == "wgrad":
        case.update(N=_log(rng, 128, 2048, 16), K=_log(rng, 128, 2048, 16), out=rng.choice(("bf16", "f32")))
    else:
        case.update(H=_log(rng, 64, 8192, 8))
        if op == "combine":
            case.update(residual=flag())
        elif op == "combine_grad":
            case.update(amax=flag())
    return case


# ------------------------------------------------------------------ inputs --
def _capacity(copies, experts):
    """Rows that hold `copies` rows in segments starting at multiples of 128, however they fall."""
    return (copies + 127 * min(copies, experts) + 127) // 128 * 128


def _to_layout(scales):
    """Block scales [R, K/16] in the tensor cores' layout: 128 rows x 4 blocks to a chunk of 512 bytes."""
    r, kb = scales.shape
    rc, kc = -(-r // 128), -(-kb // 4)
    full = torch.zeros(rc * 128, kc * 4, dtype=torch.uint8, device=scales.device)
    full[:r, :kb] = scales
    return full.view(rc, 4, 32, kc, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _from_layout(flat, rows, blocks):
    rc, kc = -(-rows // 128), -(-blocks // 4)
    return flat.view(rc, kc, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rc * 128, kc * 4)[:rows, :blocks]


def _quantized(x):
    """(codes, scales in the tensor cores' layout, global scale) of a matrix, as a quantizer hands them over."""
    x = x.float()
    g = (x.abs().max() / 2688).reshape(1)
    blocks = x.view(x.shape[0], -1, 16)
    s = (blocks.abs().amax(2) / (6 * g).clamp_min(1e-30)).clamp(max=448).to(torch.float8_e4m3fn)
    v = blocks / (s.float() * g).clamp_min(1e-30)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = (torch.bucketize(v.abs().view(x.shape), edges) + 8 * (v.view(x.shape) < 0)).to(torch.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), _to_layout(s.view(torch.uint8)), g


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _activations(gen, rows, cols):
    """Normal values with rare large ones, as activations have them."""
    x = _randn(gen, rows, cols)
    return torch.where(torch.rand(rows, cols, generator=gen, device="cuda") < 5e-4, x * 100, x).bfloat16()


def _ids(gen, case):
    """Expert numbers of each token's copies: distinct within a token, some experts liked better than others."""
    liking = _randn(gen, 1, case["E"]) + _randn(gen, case["T"], case["E"])
    return liking.topk(case["k"], dim=1).indices.to(torch.int32)


def _sorted_rows(ids, experts):
    """offsets [E+1], counts [E], row -> copy [R] and copy -> row [T, k] of a routing, as 32-bit numbers."""
    flat = ids.reshape(-1).long()
    n, rows = flat.numel(), _capacity(flat.numel(), experts)
    order = torch.sort(flat, stable=True).indices
    counts = (flat[None] == torch.arange(experts, device=flat.device)[:, None]).sum(1)
    ends = torch.cumsum((counts + 127) // 128 * 128, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    first = torch.cumsum(counts, 0) - counts
    by = flat[order]
    row = offsets[by] + torch.arange(n, device=flat.device) - first[by]
    row_copy = torch.full((rows,), -1, dtype=torch.int32, device=flat.device)
    row_copy[row] = order.to(torch.int32)
    copy_row = torch.empty(n, dtype=torch.int32, device=flat.device)
    copy_row[order] = row.to(torch.int32)
    return offsets.to(torch.int32), counts.to(torch.int32), row_copy, copy_row.view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    op, s = case["op"], {"case": case}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        s["a"] = _quantized(_activations(gen, M, K))
        s["b"] = _quantized(_randn(gen, N, K) * K ** -0.5)
        s["bias"] = (_randn(gen, N) * 0.1).bfloat16() if case["bias"] else None
        s["residual"] = _randn(gen, M, -(-N // 8) * 8).bfloat16()[:, :N] if case["residual"] else None
        return s
    if op == "act_grad":
        M, ld = case["M"], -(-case["N"] // 8) * 8
        s["dy"] = (_randn(gen, M, ld) * 1e-3).bfloat16()[:, :case["N"]]
        s["z"] = (_randn(gen, M, ld) * 1.5).bfloat16()[:, :case["N"]]
        return s
    ids, E = _ids(gen, case), case["E"]
    if op == "route":
        return dict(s, ids=ids, x=_activations(gen, case["T"], case["H"]))
    s["offsets"], s["counts"], s["row_copy"], s["copy_row"] = _sorted_rows(ids, E)
    R = s["row_copy"].numel()
    real = (s["row_copy"] >= 0)[:, None]
    if op == "experts":
        N, K = case["N"], case["K"]
        s["a"] = _quantized(torch.where(real, _activations(gen, R, K), 0))
        codes, scales, g = zip(*(_quantized(_randn(gen, N, K) * K ** -0.5) for _ in range(E)))
        s["b"] = torch.stack(codes), torch.stack(scales), torch.cat(g)
        s["bias"] = (_randn(gen, E, N) * 0.1).bfloat16() if case["bias"] else None
    elif op == "wgrad":
        s["a"] = _quantized(torch.where(real, _randn(gen, R, case["N"]) * 1e-3, 0).t().contiguous())
        s["b"] = _quantized(torch.where(real, _randn(gen, R, case["K"]), 0).t().contiguous())
    else:
        s["y"] = torch.where(real, _randn(gen, R, case["H"]), 0).bfloat16()
        s["weights"] = torch.softmax(_randn(gen, case["T"], case["k"]), 1)
        s["dout"] = (_randn(gen, case["T"], case["H"]) * 1e-3).bfloat16() if op == "combine_grad" else None
        s["residual"] = _randn(gen, case["T"], case["H"]).bfloat16() if case.get("residual") else None
    return s


# ------------------------------------------------------------- plain forms --
def _values(codes, scales, g, dtype=torch.float32):
    """What NVFP4 codes stand for."""
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype,
                        device=codes.device)
    v = torch.stack([grid[(codes & 15).int()], grid[(codes >> 4).int()]], 2)
    s = _from_layout(scales, codes.shape[0], codes.shape[1] // 8).contiguous().view(torch.float8_e4m3fn).to(dtype)
    return (v.view(codes.shape[0], -1, 16) * s[:, :, None]).view(codes.shape[0], -1) * g.to(dtype)


def _act(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "relu2":
        return z.clamp_min(0) * z.clamp_min(0)
    if name == "gelu":
        return z * (0.5 + 0.5 * torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z)) if name == "silu" else z


def _slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "relu2":
        return 2 * z.clamp_min(0)
    if name == "gelu":
        return 0.5 + 0.5 * torch.erf(z * 0.5 ** 0.5) + z * torch.exp(-0.5 * z * z) * (2 * math.pi) ** -0.5
    if name == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _peak(t):
    return t.abs().max().float().reshape(1)


def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "linear":
        z = _values(*s["a"]) @ _values(*s["b"]).t()
        z = z if s["bias"] is None else z + s["bias"].float()
        c = _act(case["act"], z)
        c = c if s["residual"] is None else c + s["residual"].float()
        c = c.to(torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        return {"c": c, "pre": z.bfloat16() if case["pre"] else None, "amax": _peak(c) if case["amax"] else None}
    if op == "act_grad":
        dz = s["dy"].float() * _slope(case["act"], s["z"].float())
        out = dz.bfloat16()
        return {"dz": out, "dbias": dz.sum(0), "amax": _peak(out) if case["amax"] else None}
    if op == "route":
        offsets, counts, row_copy, copy_row = _sorted_rows(s["ids"], case["E"])
        x = torch.where((row_copy >= 0)[:, None], s["x"][row_copy.clamp_min(0).long() // case["k"]], 0)
        return {"offsets": offsets, "counts": counts, "row_copy": row_copy, "copy_row": copy_row, "x": x,
                "amax": _peak(x)}
    if op == "combine":
        out = (s["y"][s["copy_row"].long()].float() * s["weights"][:, :, None]).sum(1)
        out = out if s["residual"] is None else out + s["residual"].float()
        return {"out": out.bfloat16()}
    if op == "combine_grad":
        copy, k = s["row_copy"].long(), case["k"]
        w = torch.where(copy >= 0, s["weights"].reshape(-1)[copy.clamp_min(0)], 0)
        dy = (s["dout"][copy.clamp_min(0) // k].float() * w[:, None]).bfloat16()
        dw = (s["y"][s["copy_row"].long()].float() * s["dout"][:, None].float()).sum(2)
        return {"dy": dy, "dweights": dw, "amax": _peak(dy) if case["amax"] else None}
    # one product per expert over its own rows, so the loop over experts is the plain form
    segments = list(zip(s["offsets"].tolist(), s["counts"].tolist()))
    if op == "experts":
        a = _values(*s["a"])
        c = torch.zeros(a.shape[0], case["N"], dtype=torch.bfloat16, device=a.device)
        pre = torch.zeros_like(c) if case["pre"] else None
        for e, (at, n) in enumerate(segments):
            if not n:
                continue
            z = a[at:at + n] @ _values(*(t[e] for t in s["b"])).t()
            z = z if s["bias"] is None else z + s["bias"][e].float()
            c[at:at + n] = _act(case["act"], z).bfloat16()
            if pre is not None:
                pre[at:at + n] = z.bfloat16()
        return {"c": c, "pre": pre, "amax": _peak(c) if case["amax"] else None}
    a, b = _values(*s["a"]), _values(*s["b"])
    dw = torch.stack([a[:, at:at + n] @ b[:, at:at + n].t() for at, n in segments])
    return {"dw": dw if case["out"] == "f32" else dw.bfloat16()}


# -------------------------------------------------------- the framework's --
def _own(s):
    from nvfp4_bit_block_amax_b200 import nvfp4 as N
    case, op = s["case"], s["case"]["op"]
    act = getattr(N, "NVFP4_ACT_" + case.get("act", "none").upper())
    out = N.NVFP4_OUT_F32 if case.get("out") == "f32" else N.NVFP4_OUT_BF16
    amax = torch.empty(1, dtype=torch.float32, device="cuda") if case.get("amax") or op == "route" else None
    if op == "linear":
        M, n, K = case["M"], case["N"], case["K"]
        pre = torch.empty(M, -(-n // 8) * 8, dtype=torch.bfloat16, device="cuda")[:, :n] if case["pre"] else None
        c = N.gemm_epilogue(*_operand(s["a"]), *_operand(s["b"]), M, n, K, bias=s["bias"], activation=act,
                            residual=s["residual"], out_dtype=out, pre=pre, amax_out=amax)
        return {"c": c, "pre": pre, "amax": amax}
    if op == "act_grad":
        dz, dbias = N.act_grad(s["dy"], s["z"], act, amax_out=amax)
        return {"dz": dz, "dbias": dbias, "amax": amax}
    if op == "route":
        plan = N.moe_sort(s["ids"], case["E"])
        x = N.moe_gather(s["x"], plan, amax_out=amax)
        return {"offsets": plan.offsets, "counts": plan.counts, "row_copy": plan.row_copy, "copy_row": plan.copy_row,
                "x": x, "amax": amax}
    plan = N.MoePlan(s["offsets"], s["counts"], s["row_copy"], s["copy_row"])
    if op == "combine":
        return {"out": N.moe_combine(s["y"], plan, s["weights"], residual=s["residual"])}
    if op == "combine_grad":
        dy, dw = N.moe_combine_grad(s["dout"], s["y"], plan, s["weights"], amax_out=amax)
        return {"dy": dy, "dweights": dw, "amax": amax}
    R = s["row_copy"].numel()
    if op == "experts":
        pre = torch.empty(R, case["N"], dtype=torch.bfloat16, device="cuda") if case["pre"] else None
        c = N.gemm_grouped(*_operand(s["a"]), *_operand(s["b"]), plan, R, case["N"], case["K"], bias=s["bias"],
                           activation=act, pre=pre, amax_out=amax)
        return {"c": c, "pre": pre, "amax": amax}
    return {"dw": N.gemm_grouped_wgrad(*_operand(s["a"]), *_operand(s["b"]), plan, case["N"], case["K"], R,
                                       out_dtype=out)}


def _operand(q):
    return q[0], q[1], q[2]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------ 64-bit forms --
def _act64(name, z):
    """Each activation from its definition: z times a probability for the smooth ones."""
    if name == "none":
        return z
    if name in ("relu", "relu2"):
        return torch.where(z > 0, z if name == "relu" else z ** 2, torch.zeros_like(z))
    if name == "gelu":
        return z * torch.special.ndtr(z)
    return z * torch.sigmoid(z if name == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    f64 = torch.float64
    # the largest stored value: that of the values as the output's type holds them
    peak = lambda t: t.to(torch.float32 if case.get("out") == "f32" else torch.bfloat16).to(f64).abs().max().reshape(1)
    if op == "route":
        return None
    if op == "linear":
        z = _values(*s["a"], dtype=f64).matmul(_values(*s["b"], dtype=f64).mT)
        if case["bias"]:
            z += s["bias"].to(f64)
        c = _act64(case["act"], z)
        if case["residual"]:
            c += s["residual"].to(f64)
        return {"c": c, "pre": z if case["pre"] else None, "amax": peak(c) if case["amax"] else None}
    if op == "act_grad":
        z = s["z"].to(f64).requires_grad_()
        dz, = torch.autograd.grad(_act64(case["act"], z), z, s["dy"].to(f64))
        return {"dz": dz, "dbias": dz.sum(0), "amax": peak(dz) if case["amax"] else None}
    if op in ("combine", "combine_grad"):
        T, k, H = case["T"], case["k"], case["H"]
        out = torch.zeros(T, H, dtype=f64, device="cuda")
        dw = torch.empty(T, k, dtype=f64, device="cuda")
        dy = torch.zeros(s["y"].shape, dtype=f64, device="cuda")
        for j in range(k):
            rows, w = s["copy_row"][:, j].long(), s["weights"][:, j, None].to(f64)
            y = s["y"][rows].to(f64)
            if op == "combine":
                out += w * y
            else:
                dy[rows] = w * s["dout"].to(f64)
                dw[:, j] = torch.einsum("th,th->t", y, s["dout"].to(f64))
        if op == "combine":
            return {"out": out + s["residual"].to(f64) if case["residual"] else out}
        return {"dy": dy, "dweights": dw, "amax": peak(dy) if case["amax"] else None}
    a = _values(*s["a"], dtype=f64)
    starts, counts = s["offsets"].tolist(), s["counts"].tolist()
    if op == "experts":
        z = torch.zeros(a.shape[0], case["N"], dtype=f64, device="cuda")
        c = torch.zeros_like(z)
        for e in range(case["E"]):
            rows = slice(starts[e], starts[e] + counts[e])
            z[rows] = torch.einsum("rk,nk->rn", a[rows], _values(*(t[e] for t in s["b"]), dtype=f64))
            if case["bias"]:
                z[rows] += s["bias"][e].to(f64)
            c[rows] = _act64(case["act"], z[rows])
        return {"c": c, "pre": z if case["pre"] else None, "amax": peak(c) if case["amax"] else None}
    b = _values(*s["b"], dtype=f64)
    dw = torch.zeros(case["E"], case["N"], case["K"], dtype=f64, device="cuda")
    for e in range(case["E"]):
        seg = slice(starts[e], starts[e + 1])
        dw[e] = torch.einsum("nr,kr->nk", a[:, seg], b[:, seg])
    return {"dw": dw}


# -------------------------------------------------------------------- work --
def _nvfp4_bytes(rows, cols):
    return rows * cols * (0.5 + 1 / 16) + 4


def work(case):
    """Inputs read once and outputs written once; rows of the sorted matrices that are padding count where they
    have to be written (they are zeros) and not where they need not be read."""
    op = case["op"]
    size = 4 if case.get("out") == "f32" else 2
    amax = 4 * bool(case.get("amax") or op == "route")
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        wide = size + 2 * case["residual"] + 2 * case["pre"]
        return {"bytes": _nvfp4_bytes(M, K) + _nvfp4_bytes(N, K) + M * N * wide + 2 * N * case["bias"] + amax,
                "flops": 2 * M * N * K}
    if op == "act_grad":
        return {"bytes": 6 * case["M"] * case["N"] + 4 * case["N"] + amax, "flops": 10 * case["M"] * case["N"]}
    T, n, E = case["T"], case["T"] * case["k"], case["E"]
    R, ints = _capacity(n, E), 4 * (2 * E + 1)
    used = min(E, n)   # experts that have rows, at most
    if op == "experts":
        N, K = case["N"], case["K"]
        return {"bytes": _nvfp4_bytes(n, K) + used * (_nvfp4_bytes(N, K) + 2 * N * case["bias"]) +
                R * N * 2 * (1 + case["pre"]) + ints + amax, "flops": 2 * n * N * K}
    if op == "wgrad":
        N, K = case["N"], case["K"]
        return {"bytes": _nvfp4_bytes(n, N) + _nvfp4_bytes(n, K) + E * N * K * size + ints, "flops": 2 * n * N * K}
    H = case["H"]
    if op == "route":
        return {"bytes": 4 * (2 * n + R) + ints + 2 * H * (T + R) + amax, "flops": n * max(1, math.log2(E))}
    if op == "combine":
        return {"bytes": 8 * n + 2 * H * (n + T + T * case["residual"]), "flops": 2 * n * H}
    return {"bytes": 12 * n + 4 * R + 2 * H * (T + n + R) + amax, "flops": 3 * n * H}
