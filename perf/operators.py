"""The operators on 4-bit weights with group scales: their cases, inputs and plain forms.

Two operators share the weight format codes [N, K/2] (two 4-bit codes per byte, the low nibble the
even element), scales [N, K/G] in the activations' type and, optionally, zero points [N, K/G]:
W[n, k] = (code - zero) * scale, zero = 8 where there are none.

  gemm    C = x . W^T for 1 to 64 rows of x, as a decode step's linear layers run it
  layer   a whole mixture-of-experts layer for 1 to 64 tokens: top-k of the router's scores, gate
          and up products, silu(g) * u, the down product, and the sum weighted by the normalised
          sigmoids of the selected scores, with or without an always-on shared expert

``run`` computes either in elementary torch operations in fp32, or, with ``own``, by the package.
"""
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _gemm(name, M, N, K, group, dtype, zeros):
    return dict(name=name, op="gemm", M=M, N=N, K=K, group=group, dtype=dtype, zeros=zeros)


def _layer(name, T, E, k, d, f, group, dtype, zeros, shared, skew):
    return dict(name=name, op="layer", T=T, E=E, k=k, d=d, f=f, group=group, dtype=dtype,
                zeros=zeros, shared=shared, skew=skew)


def listed():
    return [
        # one token through a square projection of the hidden size: latency counts
        _gemm("gemm m1 4096x4096 g128", 1, 4096, 4096, 128, "bf16", False),
        # a few tokens, ragged rows and a reduction that ends inside a tile, with zero points
        _gemm("gemm m3 4099x2080 g32 zp", 3, 4099, 2080, 32, "fp16", True),
        # four tokens into an output as wide as a vocabulary
        _gemm("gemm m4 65536x4096 g128", 4, 65536, 4096, 128, "bf16", False),
        # an odd batch, the expert's width back to the hidden size
        _gemm("gemm m17 4096x2048 g64 zp", 17, 4096, 2048, 64, "bf16", True),
        # the largest batch, a wide projection
        _gemm("gemm m64 8192x4096 g128", 64, 8192, 4096, 128, "fp16", False),
        # the smallest layer: one token, small experts, finest groups
        _layer("layer t1 e8 d512 g32 zp", 1, 8, 2, 512, 512, 32, "fp16", True, True, 0.0),
        # one token of the decode workload
        _layer("layer t1 e256 g128", 1, 256, 6, 4096, 2048, 128, "bf16", False, True, 0.0),
        # the tokens of a speculative step
        _layer("layer t4 e256 g64 zp", 4, 256, 6, 4096, 2048, 64, "bf16", True, True, 0.0),
        # a ragged layer: odd counts, no shared expert
        _layer("layer t7 e61 d2080 f1376 g32", 7, 61, 3, 2080, 1376, 32, "fp16", False, False, 0.0),
        # a small serving batch with popular experts
        _layer("layer t16 e256 g128 zipf", 16, 256, 6, 4096, 2048, 128, "fp16", False, True, 1.0),
        # few experts, many tokens each
        _layer("layer t32 e16 k4 d2048 f1408", 32, 16, 4, 2048, 1408, 128, "bf16", True, False, 0.0),
        # the largest decode batch
        _layer("layer t64 e256 g128 zipf", 64, 256, 6, 4096, 2048, 128, "bf16", False, True, 1.0),
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], evenly over its logarithm."""
    return min(high, int(low * (high / low) ** rng.random() * (1 + 1e-9)))


def draw(rng):
    group = rng.choice([32, 64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    zeros = rng.random() < 0.5
    if rng.random() < 0.45:
        return dict(op="gemm", M=_spread(rng, 1, 64), N=_spread(rng, 300, 16384),
                    K=group * max(1, _spread(rng, 512, 8192) // group), group=group, dtype=dtype,
                    zeros=zeros)
    T, k = _spread(rng, 1, 60), rng.randint(1, 6)
    many = T * k > 96  # a large batch has popular experts, as the largest listed one
    return dict(op="layer", T=T, E=_spread(rng, 8, 256), k=k,
                d=group * (_spread(rng, 512, 4096) // group),
                f=group * (_spread(rng, 512, 2048) // group), group=group, dtype=dtype,
                zeros=zeros and not many, shared=rng.random() < 0.6,
                skew=1.0 if many else rng.choice([0.0, 1.0]))


def _weights(gen, shape, group, dtype, zeros):
    """codes, scales and zero points of matrices [..., N, K], scaled so that products of unit rows
    come out near one."""
    *lead, N, K = shape
    dev = gen.device
    codes = torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, device=dev, generator=gen)
    u = torch.rand((*lead, N, K // group), device=dev, generator=gen)
    scales = ((0.5 + u) / (4.6 * K ** 0.5)).to(dtype)
    z = None
    if zeros:
        z = torch.randint(5, 12, (*lead, N, K // group), dtype=torch.uint8, device=dev,
                          generator=gen)
    return codes, scales, z


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    G, zp = case["group"], case["zeros"]
    if case["op"] == "gemm":
        x = torch.randn((case["M"], case["K"]), device="cuda", generator=gen).to(dtype)
        return dict(case=case, x=x, w=_weights(gen, (case["N"], case["K"]), G, dtype, zp))
    T, E, d, f = case["T"], case["E"], case["d"], case["f"]
    n = E + (1 if case["shared"] else 0)  # the shared expert is the last
    x = torch.randn((T, d), device="cuda", generator=gen).to(dtype)
    # router scores: plain, or with experts of a Zipf popularity (log p + Gumbel noise)
    if case["skew"] > 0:
        logp = -case["skew"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
        logp = logp[torch.randperm(E, device="cuda", generator=gen)]
        u = torch.rand((T, E), device="cuda", generator=gen).clamp_(1e-7, 1 - 1e-7)
        scores = logp - torch.log(-torch.log(u))
    else:
        scores = torch.randn((T, E), device="cuda", generator=gen)
    return dict(case=case, x=x, scores=scores, gate=_weights(gen, (n, f, d), G, dtype, zp),
                up=_weights(gen, (n, f, d), G, dtype, zp),
                down=_weights(gen, (n, d, f), G, dtype, zp))


def _dense(codes, scales, zeros, group):
    """The matrices in fp32."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    q = q.unflatten(-1, (-1, group)).float()
    z = 8.0 if zeros is None else zeros.unsqueeze(-1).float()
    return ((q - z) * scales.unsqueeze(-1).float()).flatten(-2)


def _rows(w, experts):
    return tuple(None if t is None else t[experts] for t in w)


def _ffn(x, state, experts, G):
    """y [pairs, d] of one row of x [pairs, d] and one expert each."""
    g = (_dense(*_rows(state["gate"], experts), G) @ x.unsqueeze(-1)).squeeze(-1)
    u = (_dense(*_rows(state["up"], experts), G) @ x.unsqueeze(-1)).squeeze(-1)
    h = g / (1.0 + torch.exp(-g)) * u
    return (_dense(*_rows(state["down"], experts), G) @ h.unsqueeze(-1)).squeeze(-1)


def _plain(state):
    case, x = state["case"], state["x"].float()
    G = case["group"]
    if case["op"] == "gemm":
        return x @ _dense(*state["w"], G).T
    T, E, k = case["T"], case["E"], case["k"]
    top, idx = torch.sort(state["scores"], dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    sig = 1.0 / (1.0 + torch.exp(-top))
    w = sig / sig.sum(1, keepdim=True)
    y = _ffn(x.repeat_interleave(k, 0), state, idx.reshape(-1), G).view(T, k, -1)
    out = (y * w.unsqueeze(-1)).sum(1)
    if case["shared"]:
        g = x @ _dense(*_rows(state["gate"], E), G).T
        u = x @ _dense(*_rows(state["up"], E), G).T
        out = out + (g / (1.0 + torch.exp(-g)) * u) @ _dense(*_rows(state["down"], E), G).T
    return out, idx.int(), w


def run(state):
    if own:
        import bit_moe_routed_b200 as bm
        case = state["case"]
        if case["op"] == "gemm":
            if "matrix" not in state:  # the weights' descriptor, kept beside them
                codes, scales, zeros = state["w"]
                state["matrix"] = bm.W4Matrix(codes, scales, zeros)
            return bm.w4_gemm(state["x"], state["matrix"])
        if "layer" not in state:  # the descriptor and the workspace a decode loop keeps
            state["layer"] = bm.W4Layer(*(bm.W4Matrix(*state[m]) for m in ("gate", "up", "down")),
                                        shared=case["shared"])
            state["ws"] = bm.alloc_workspace_w4(case["T"], case["k"], state["layer"])
        r = bm.forward_w4(state["x"], state["scores"], case["k"], state["layer"], ws=state["ws"])
        return r["out"], r["idx"], r["w"]
    return _plain(state)


def _matrix_bytes(N, K, case):
    return N * K // 2 + N * (K // case["group"]) * (3 if case["zeros"] else 2)


def work(case):
    if case["op"] == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": _matrix_bytes(N, K, case) + 2 * M * K + 4 * M * N, "flops": 2 * M * N * K}
    T, E, k, d, f = (case[n] for n in ("T", "E", "k", "d", "f"))
    # the experts that a batch selects: all distinct ones it is expected to, each read once
    if case["skew"] > 0:
        p = [1.0 / (e + 1) ** case["skew"] for e in range(E)]
        total = sum(p)
        # a token holds expert e with about the chance of one of its k draws taking it
        active = sum(1.0 - (1.0 - min(1.0, q / total)) ** (T * k) for q in p)
    else:
        active = E * (1.0 - (1.0 - k / E) ** T)
    active = max(active, float(min(k, E))) + (1 if case["shared"] else 0)
    per = 2 * _matrix_bytes(f, d, case) + _matrix_bytes(d, f, case)
    rows = T * (k + (1 if case["shared"] else 0))
    return {"bytes": active * per + T * (2 * d + 4 * E + 4 * d + 8 * k), "flops": 6 * rows * d * f}


def _exact_matrix(w, group, e=None):
    """A matrix in 64 bits, code by code from the format's definition."""
    codes, scales, zeros = (t if t is None or e is None else t[e] for t in w)
    N, K = codes.shape[0], codes.shape[1] * 2
    W = torch.empty((N, K), dtype=torch.float64, device=codes.device)
    W[:, 0::2] = torch.remainder(codes, 16).double()
    W[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    W -= 8.0 if zeros is None else torch.repeat_interleave(zeros.double(), group, dim=1)
    W *= torch.repeat_interleave(scales.double(), group, dim=1)
    return W


def exact(case, seed):
    s = prepare(case, seed)
    G, x = case["group"], s["x"].double()
    if case["op"] == "gemm":
        return torch.einsum("mk,nk->mn", x, _exact_matrix(s["w"], G))
    T, E, k = case["T"], case["E"], case["k"]
    scores = s["scores"].cpu()
    # a token's experts: by falling score, equal scores by rising index
    idx = torch.tensor([sorted(range(E), key=lambda e: (-row[e], e))[:k] for row in scores.tolist()])
    sig = torch.sigmoid(torch.gather(scores.double(), 1, idx))
    w = (sig / sig.sum(1, keepdim=True)).cuda()
    out = torch.zeros((T, case["d"]), dtype=torch.float64, device="cuda")
    groups = {e: (idx == e).nonzero().tolist() for e in sorted(set(idx.flatten().tolist()))}
    if case["shared"]:
        groups[E] = [(t, -1) for t in range(T)]
    for e, pairs in groups.items():
        rows = torch.tensor([t for t, _ in pairs], device="cuda")
        gate = torch.einsum("td,fd->tf", x[rows], _exact_matrix(s["gate"], G, e))
        up = torch.einsum("td,fd->tf", x[rows], _exact_matrix(s["up"], G, e))
        y = torch.einsum("tf,df->td", gate * torch.sigmoid(gate) * up, _exact_matrix(s["down"], G, e))
        weight = torch.stack([w[t, j] if j >= 0 else w.new_tensor(1.0) for t, j in pairs])
        out.index_add_(0, rows, y * weight.unsqueeze(1))
    return out, None, w
