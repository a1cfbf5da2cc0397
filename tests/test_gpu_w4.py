"""The 4-bit operators on the GPU (moe_w4_gemm, moe_forward_w4) against their definition in
64 bits.

Bounds, derived before the first run.  u = 2^-23 bounds the relative error of one fp32
rounding in any mode.  Two forms: few rows of x in whole numbers, more in 16-bit operands.
In the first x enters as fixed point, an element off by at most fx = 2^-30 max |x| over its 256
elements (half a step where the largest is scaled to 2^29 or more), and the sums of (q - z) x
are exact; in the second 16-bit x enters as it is and fp32 rows (h) as two fp16 terms, off by
fx = 2^-22 |x| (a rounding to fp16 is off by at most 2^-11 of the value, the second one rounds
the first one's rest) + 2^-39 max |x| (half of fp16's smallest step, 2^-25, where the largest is
scaled to 2^14 or more), and an element meets at most G roundings inside its group's sum.
GEMM: the group's sum meets one rounding to fp32, one in the scaling multiply-add of each of
the slice's 256/G groups, one where its low and high parts are joined, one for each pass that
adds a warp's slices and one for each of the at most 16 warps whose sums are added, so
  |C - C64| <= sum_k fx |W| + D u sum_k |x W|,   D = 256/G + ceil(K/4096) + 18 (+ G).
Layer: g and u as above; h = g / (1 + exp(-g)) u adds |u| |silu'(g)| dg + |silu(g)| du and
their product, and 9 u |h| for the element-wise operations; y = Wd h adds sum fh |Wd| for h as
it enters and D u sum |Wd h|; the weights are off by at most (k + 10) u of their value (expf
2 units, the sum of k, two divisions), and the combine rounds once per term:
  |out - out64| <= sum_j w_j (dy_j + (k + 10 + k + 2) u |y_j|) + dy_sh + (k + 2) u |y_sh|.
All with a factor 1.01 for the second-order terms."""
import pytest
import torch

bm = pytest.importorskip("bit_moe_routed_b200")

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(autouse=True)
def _needs_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def weights(gen, shape, G, dtype, zeros, wide=False):
    *lead, N, K = shape
    codes = torch.randint(0, 256, (*lead, N, K // 2), dtype=torch.uint8, device="cuda", generator=gen)
    u = torch.rand((*lead, N, K // G), device="cuda", generator=gen)
    scales = ((0.25 + u) / (4.6 * K ** 0.5)).to(dtype)
    z = None
    if zeros:
        z = torch.randint(0, 128 if wide else 16, (*lead, N, K // G), dtype=torch.uint8,
                          device="cuda", generator=gen)
    return codes, scales, z


def dense(codes, scales, zeros, G):
    q = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.float64, device=codes.device)
    q[..., 0::2] = (codes & 15).double()
    q[..., 1::2] = (codes >> 4).double()
    z = 8.0 if zeros is None else zeros.double().repeat_interleave(G, -1)
    return (q - z) * scales.double().repeat_interleave(G, -1)


def depth(K, G, wide=False):
    return 256 // G + -(-K // 4096) + 18 + (G if wide else 0)


def entry(x, wide=False, fp32=False):
    """How far an element of x may be off as it enters the product."""
    K = x.shape[1]
    top = torch.nn.functional.pad(x.abs(), (0, -K % 256)).unflatten(1, (-1, 256)).amax(2)
    top = top.repeat_interleave(256, 1)[:, :K]
    if not wide:
        return 2.0 ** -30 * top
    return 2.0 ** -22 * x.abs() + 2.0 ** -39 * top if fp32 else torch.zeros_like(x)


def product_bound(x, W, G, wide=False, fp32=False):
    """The bound on x . W^T for x and W in 64 bits."""
    return (entry(x, wide, fp32) + depth(x.shape[1], G, wide) * U * x.abs()) @ W.abs().T


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def check_gemm(C, x, W, G, rows=slice(None)):
    ref = x.double() @ W.T
    bound = 1.01 * product_bound(x.double(), W, G, wide=x.shape[0] > 4)
    err = (C[:, rows].double() - ref).abs()
    worst = float((err / bound.clamp_min(1e-300)).max())
    assert bool((err <= bound).all()), f"worst error is {worst:.3g} of its bound"
    return worst


GEMMS = [  # M, N, K, G, dtype, zeros
    (1, 1, 32, 32, BF, False), (1, 15, 64, 64, FP, True), (2, 17, 96, 32, BF, True),
    (3, 16, 128, 128, FP, False), (4, 33, 160, 32, FP, True), (5, 300, 288, 32, BF, False),
    (7, 64, 384, 128, BF, True), (8, 4099, 256, 64, BF, False), (9, 47, 512, 64, FP, True),
    (15, 129, 2080, 32, FP, True), (16, 2048, 4096, 128, BF, False), (17, 31, 4160, 64, BF, True),
    (24, 1000, 1408, 128, FP, True), (33, 5, 4224, 32, BF, True), (47, 2100, 8320, 64, FP, False),
    (64, 257, 16384, 128, BF, True), (64, 4096, 2048, 32, FP, True), (1, 4096, 4096, 128, BF, False),
    (1, 20000, 4096, 64, FP, True), (6, 9000, 640, 128, FP, False)]


@pytest.mark.parametrize("M,N,K,G,dtype,zeros", GEMMS)
def test_gemm(M, N, K, G, dtype, zeros):
    gen = generator(M * 1000003 + N * 101 + K)
    w = weights(gen, (N, K), G, dtype, zeros, wide=N % 2 == 1)
    x = torch.randn((M, K), device="cuda", generator=gen).to(dtype)
    C = bm.w4_gemm(x, bm.W4Matrix(*w))
    bm.sync_status()
    worst = check_gemm(C, x, dense(*w, G), G)
    print(f"W4GEMM M={M} N={N} K={K} G={G}: worst err/bound {worst:.2e}")


@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_gemm_scales_off_their_alignment(G, dtype):
    """Scales and zero points that start two bytes (one byte) into an allocation."""
    N, K, M = 96, 1024, 5
    gen = generator(G)
    c, s, z = weights(gen, (N, K), G, dtype, True)
    s2 = torch.empty(s.numel() + 1, dtype=dtype, device="cuda")[1:].view(s.shape).copy_(s)
    z2 = torch.empty(z.numel() + 1, dtype=torch.uint8, device="cuda")[1:].view(z.shape).copy_(z)
    assert s2.data_ptr() % 4 == 2 and z2.data_ptr() % 2 == 1
    x = torch.randn((M, K), device="cuda", generator=gen).to(dtype)
    a, b = bm.w4_gemm(x, bm.W4Matrix(c, s, z)), bm.w4_gemm(x, bm.W4Matrix(c, s2, z2))
    bm.sync_status()
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,lo,hi", [(BF, -22, 0), (FP, -14, 5), (BF, -126, -100), (BF, 90, 112)])
def test_gemm_exact_over_the_range_of_fixed_point(dtype, lo, hi):
    """Elements of all magnitudes that fixed point holds exactly beside the slice's largest (and
    slices of the smallest and largest numbers): the result's error is the sums' alone."""
    M, N, K, G = 4, 40, 512, 32  # whole numbers
    gen = generator(hi - lo)
    c, s, z = weights(gen, (N, K), G, dtype, True)
    s = (s.float() / 2 ** 4).to(dtype)
    e = torch.randint(lo, hi + 1, (M, K), device="cuda", generator=gen).double()
    m = 1 + torch.randint(0, 128, (M, K), device="cuda", generator=gen).double() / 128
    x = (m * 2.0 ** e * torch.sign(torch.randn((M, K), device="cuda", generator=gen))).to(dtype)
    C = bm.w4_gemm(x, bm.W4Matrix(c, s, z))
    bm.sync_status()
    W = dense(c, s, z, G)
    err = (C.double() - x.double() @ W.T).abs()
    assert bool((err <= 1.01 * depth(K, G) * U * (x.double().abs() @ W.abs().T)).all())


@pytest.mark.parametrize("M", [3, 12])
def test_gemm_rows_do_not_meet(M):
    """inf and NaN in one row of x leave the others' bits as they were and give what floating
    point gives; a zero scale's group adds nothing."""
    N, K, G = 50, 544, 32
    gen = generator(7)
    c, s, z = weights(gen, (N, K), G, BF, True)
    x = torch.randn((M, K), device="cuda", generator=gen).to(BF)
    m = bm.W4Matrix(c, s, z)
    base = bm.w4_gemm(x, m)
    y = x.clone()
    y[1, 5], y[2, 77] = float("inf"), float("nan")
    got = bm.w4_gemm(y, m)
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(got[keep], base[keep])
    ref = y.double() @ dense(c, s, z, G).T
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    fin = ~torch.isnan(ref)
    assert torch.equal(torch.isinf(got[fin]), torch.isinf(ref[fin]))
    assert torch.equal(got[1][torch.isinf(ref[1])].double(), ref[1][torch.isinf(ref[1])])
    s0 = torch.zeros_like(s)
    assert bool((bm.w4_gemm(x, bm.W4Matrix(c, s0, z)) == 0).all())


def test_gemm_writes_its_output_alone_and_takes_any_stream():
    M, N, K, G = 11, 77, 320, 64
    gen = generator(3)
    w = weights(gen, (N, K), G, FP, False)
    x = torch.randn((M, K), device="cuda", generator=gen).to(FP)
    buf = torch.full((M * N + 64,), -7.0, device="cuda")
    out = buf[32:32 + M * N].view(M, N)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    bm.w4_gemm(x, bm.W4Matrix(*w), out=out, stream=s)
    s.synchronize()
    assert bool((buf[:32] == -7).all()) and bool((buf[32 + M * N:] == -7).all())
    check_gemm(out, x, dense(*w, G), G)
    assert bm.w4_gemm(x[:0], bm.W4Matrix(*w)).shape == (0, N)


def test_gemm_past_four_gigabytes_of_codes():
    """Rows whose codes and scales start past 2^32 bytes."""
    N, K, G = (1 << 21) + 40, 4096, 32
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB of device memory")
    gen = generator(11)
    w = weights(gen, (N, K), G, BF, True)
    x = torch.randn((1, K), device="cuda", generator=gen).to(BF)
    C = bm.w4_gemm(x, bm.W4Matrix(*w))
    bm.sync_status()
    for a, b in [(0, 64), (N // 2, N // 2 + 64), (N - 90, N)]:
        check_gemm(C, x, dense(*(t[a:b] for t in w), G), G, slice(a, b))


# ------------------------------------------------------------------------------- the layer
def make_layer(seed, E, d, f, G, dtype, zeros, shared):
    gen = generator(seed)
    n = E + int(shared)
    mats = [weights(gen, s, G, dtype, zeros) for s in ((n, f, d), (n, f, d), (n, d, f))]
    return mats, bm.W4Layer(*(bm.W4Matrix(*m) for m in mats), shared=shared)


def top_k(scores, k):
    """By falling score, equal ones by rising index."""
    rows = scores.cpu().tolist()
    return torch.tensor([sorted(range(len(r)), key=lambda e: (-r[e], e))[:k] for r in rows],
                        dtype=torch.int32)


def check_layer_w4(r, x, scores, k, mats, shared, G):
    T, d = x.shape
    E = scores.shape[1]
    idx = top_k(scores, k)
    assert torch.equal(r["idx"].cpu(), idx)
    sig = torch.sigmoid(torch.gather(scores.double().cpu(), 1, idx.long()))
    w = (sig / sig.sum(1, keepdim=True)).cuda()
    assert bool(((r["w"].double() - w).abs() <= (k + 10) * U * w).all())
    xd = x.double()
    out = torch.zeros((T, d), dtype=torch.float64, device="cuda")
    bound = torch.zeros_like(out)
    wide = T > 8 and T * k >= 4 * E
    pairs = {}
    for t in range(T):
        for j in range(k):
            pairs.setdefault(int(idx[t, j]), []).append((t, j))
    if shared:
        pairs[E] = [(t, -1) for t in range(T)]
    for e, tj in pairs.items():
        tok = torch.tensor([t for t, _ in tj], device="cuda")
        Wg, Wu, Wd = (dense(*(None if q is None else q[e] for q in m), G) for m in mats)
        g, u = xd[tok] @ Wg.T, xd[tok] @ Wu.T
        dg, du = product_bound(xd[tok], Wg, G, wide), product_bound(xd[tok], Wu, G, wide)
        sg = torch.sigmoid(g)
        silu, slope = g * sg, (sg * (1 + g * (1 - sg))).abs()
        h = silu * u
        dh = u.abs() * slope * dg + silu.abs() * du + dg * du + 9 * U * h.abs()
        y = h @ Wd.T
        dy = dh @ Wd.abs().T + product_bound(h, Wd, G, wide, fp32=True)
        wt = torch.tensor([1.0 if j < 0 else float(w[t, j]) for t, j in tj], device="cuda",
                          dtype=torch.float64).unsqueeze(1)
        extra = torch.tensor([k + 2 if j < 0 else 2 * k + 12 for _, j in tj], device="cuda",
                             dtype=torch.float64).unsqueeze(1)
        out.index_add_(0, tok, wt * y)
        bound.index_add_(0, tok, wt * (dy + extra * U * y.abs()))
    bound *= 1.01
    err = (r["out"].double() - out).abs()
    worst = float((err / bound.clamp_min(1e-300)).max())
    rel = float((r["out"].double() - out).norm() / out.norm())
    assert bool((err <= bound).all()), f"worst error is {worst:.3g} of its bound, rel {rel:.3g}"
    return worst, rel


LAYERS = [  # T, E, k, d, f, G, dtype, zeros, shared
    (1, 1, 1, 32, 32, 32, BF, False, False), (1, 8, 2, 512, 512, 32, FP, True, True),
    (1, 256, 6, 4096, 2048, 128, BF, False, True), (2, 3, 3, 64, 192, 64, BF, True, True),
    (3, 8, 2, 128, 128, 128, FP, False, False), (4, 64, 6, 2048, 1024, 64, BF, True, True),
    (5, 40, 5, 672, 352, 32, FP, True, True), (7, 61, 3, 2080, 1376, 32, FP, False, False),
    (8, 300, 8, 384, 640, 128, BF, True, False), (9, 16, 16, 256, 96, 32, BF, False, True),
    (16, 4, 2, 1088, 832, 64, FP, True, True), (17, 1024, 4, 96, 64, 32, BF, True, True),
    (33, 600, 32, 128, 256, 64, FP, False, True), (64, 8, 1, 4224, 384, 128, BF, True, False),
    (64, 128, 6, 1024, 512, 128, BF, False, True), (64, 40, 32, 64, 64, 32, FP, True, True),
    (12, 6, 2, 256, 4352, 128, FP, False, True), (3, 1024, 8, 256, 256, 128, BF, True, False),
    (4, 300, 8, 1024, 512, 32, FP, False, True), (2, 600, 32, 192, 320, 64, BF, False, True),
    (1, 64, 32, 512, 2048, 64, FP, True, False), (64, 1, 1, 256, 128, 32, BF, False, False),
    (10, 2, 2, 4608, 96, 32, FP, True, True)]


@pytest.mark.parametrize("T,E,k,d,f,G,dtype,zeros,shared", LAYERS)
def test_layer(T, E, k, d, f, G, dtype, zeros, shared):
    seed = T * 7919 + E * 31 + d + f
    mats, w = make_layer(seed, E, d, f, G, dtype, zeros, shared)
    gen = generator(seed + 1)
    x = torch.randn((T, d), device="cuda", generator=gen).to(dtype)
    s = torch.randn((T, E), device="cuda", generator=gen)
    r = bm.forward_w4(x, s, k, w)
    bm.sync_status()
    worst, rel = check_layer_w4(r, x, s, k, mats, shared, G)
    print(f"W4LAYER T={T} E={E} k={k} d={d} f={f} G={G}: worst err/bound {worst:.2e}, rel {rel:.2e}")


def test_layer_without_tokens():
    _, w = make_layer(4, 4, 64, 64, 32, BF, False, True)
    r = bm.forward_w4(torch.empty((0, 64), dtype=BF, device="cuda"), torch.empty((0, 4), device="cuda"), 2, w)
    bm.sync_status()
    assert r["out"].shape == (0, 64) and r["idx"].shape == (0, 2)


def test_refusals_on_the_gpu():
    """A misaligned x, a workspace too small, too many tokens and k above E come back as errors."""
    E, d, f, G = 4, 64, 64, 32
    _, w = make_layer(4, E, d, f, G, BF, False, True)
    x, s = torch.zeros((3, d), dtype=BF, device="cuda"), torch.zeros((3, E), device="cuda")
    off = torch.zeros(3 * d + 1, dtype=BF, device="cuda")[1:].view(3, d)
    m = bm.W4Matrix(w.gate.codes[0], w.gate.scales[0])
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    for code, call in [(bm.MOE_ERR_INVALID_ARG, lambda: bm.w4_gemm(off, m)),
                       (bm.MOE_ERR_INVALID_ARG, lambda: bm.w4_gemm(x[:1].expand(65, d).contiguous(), m)),
                       (bm.MOE_ERR_INVALID_ARG, lambda: bm.forward_w4(off, s, 2, w)),
                       (bm.MOE_ERR_INVALID_ARG, lambda: bm.forward_w4(x, s, 5, w)),
                       (bm.MOE_ERR_WORKSPACE, lambda: bm.forward_w4(x, s, 2, w, ws=ws))]:
        with pytest.raises(bm.MoeError) as ei:
            call()
        assert ei.value.code == code
    for call in (lambda: bm.w4_gemm(x.t().contiguous().t(), m), lambda: bm.w4_gemm(x.half(), m),
                 lambda: bm.forward_w4(x, s.t().contiguous().t(), 2, w),
                 lambda: bm.forward_w4(x, s, 2, w, outs={"out": torch.empty((3, d + 1), device="cuda")})):
        with pytest.raises(ValueError):
            call()
    bm.sync_status()


@pytest.mark.parametrize("T", [1, 8, 9, 64])
def test_layer_every_token_on_the_same_experts(T):
    """One expert with all tokens (several slots of 8), tied scores (the lower index wins),
    scores of both signs of zero."""
    E, k, d, f, G = 16, 3, 256, 160, 32
    mats, w = make_layer(5, E, d, f, G, BF, True, True)
    x = torch.randn((T, d), device="cuda", generator=generator(6)).to(BF)
    s = torch.full((T, E), -1.0, device="cuda")
    s[:, 11] = 2.0
    s[:, 4], s[:, 9] = -0.0, 0.0  # equal: 4 before 9
    r = bm.forward_w4(x, s, k, w)
    bm.sync_status()
    assert r["idx"].cpu().tolist() == [[11, 4, 9]] * T
    check_layer_w4(r, x, s, k, mats, True, G)
    s = torch.zeros((T, E), device="cuda")  # all equal
    r = bm.forward_w4(x, s, k, w)
    bm.sync_status()
    assert r["idx"].cpu().tolist() == [[0, 1, 2]] * T
    check_layer_w4(r, x, s, k, mats, True, G)


@pytest.mark.parametrize("E,k,T", [(8, 2, 6), (4, 2, 20)])
def test_layer_tokens_do_not_meet_and_large_h_stays_finite(E, k, T):
    """A token of inf and NaN leaves the others' bits alone; an h past fp16's range passes."""
    d, f, G = 256, 128, 64
    mats, w = make_layer(8, E, d, f, G, BF, False, True)
    gen = generator(9)
    x = torch.randn((T, d), device="cuda", generator=gen).to(BF)
    s = torch.randn((T, E), device="cuda", generator=gen)
    base = bm.forward_w4(x, s, k, w)["out"]
    y = x.clone()
    y[2, 3], y[4, 9] = float("nan"), float("inf")
    got = bm.forward_w4(y, s, k, w)["out"]
    bm.sync_status()
    keep = [t for t in range(T) if t not in (2, 4)]
    assert torch.equal(got[keep], base[keep])
    assert bool(torch.isnan(got[2]).all())
    big = (x.float() * 1e15).to(BF)
    r = bm.forward_w4(big, s, k, w)
    assert float(r["out"].abs().max()) > 1e28
    check_layer_w4(r, big, s, k, mats, True, G)


@pytest.mark.parametrize("T", [1, 5, 64])
def test_layer_workspace_and_repeats(T):
    """Two calls with different garbage in a workspace of exactly the stated size give the same
    bits, and the bytes behind it stay."""
    E, k, d, f, G = 32, 4, 544, 352, 32
    _, w = make_layer(12, E, d, f, G, FP, True, True)
    gen = generator(13)
    x = torch.randn((T, d), device="cuda", generator=gen).to(FP)
    s = torch.randn((T, E), device="cuda", generator=gen)
    n = bm.workspace_size_w4(T, k, w)
    res = []
    for fill in (0xFF, 0x00, 0x5A):
        buf = torch.full((n + (1 << 20),), fill, dtype=torch.uint8, device="cuda")
        outs = {"out": torch.full((T, d), 3.0, device="cuda")}
        r = bm.forward_w4(x, s, k, w, ws=buf[:n], outs=outs)
        bm.sync_status()
        assert bool((buf[n:] == fill).all())
        assert r["out"] is outs["out"]
        res.append(r["out"].clone())
    assert torch.equal(res[0], res[1]) and torch.equal(res[0], res[2])


def test_layer_captured_replayed_and_on_two_streams():
    """A captured call follows its inputs; two calls at once with a workspace each agree with
    the same calls alone."""
    T, E, k, d, f, G = 4, 24, 3, 512, 256, 64
    _, w = make_layer(21, E, d, f, G, BF, True, True)
    gen = generator(22)
    xs = [torch.randn((T, d), device="cuda", generator=gen).to(BF) for _ in range(3)]
    ss = [torch.randn((T, E), device="cuda", generator=gen) for _ in range(3)]
    alone = [bm.forward_w4(a, b, k, w)["out"].clone() for a, b in zip(xs, ss)]
    x, s = xs[0].clone(), ss[0].clone()
    ws = bm.alloc_workspace_w4(T, k, w)
    outs = {n: t.clone() for n, t in bm.forward_w4(x, s, k, w, ws=ws).items()}
    head = weights(gen, (100, d), G, BF, False)
    hm = bm.W4Matrix(*head)
    logits = torch.empty((T, 100), device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bm.forward_w4(x, s, k, w, ws=ws, outs=outs)
        bm.w4_gemm(outs["out"].to(BF), hm, out=logits)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        s.copy_(ss[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs["out"], alone[i])
        assert torch.equal(logits, bm.w4_gemm(alone[i].to(BF), hm))
    streams = [torch.cuda.Stream() for _ in range(3)]
    works = [bm.alloc_workspace_w4(T, k, w) for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got.append(bm.forward_w4(xs[i], ss[i], k, w, ws=works[i])["out"])
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_a_decode_step_through_router_layers_and_head(dtype):
    """The operators as a decode loop uses them: router scores, two layers with residuals, a
    vocabulary projection; each against the definition on the same inputs."""
    T, E, k, d, f, G, V = 3, 16, 2, 512, 256, 128, 1003
    gen = generator(31)
    hidden = torch.randn((T, d), device="cuda", generator=gen).to(dtype)
    for layer in range(2):
        mats, w = make_layer(32 + layer, E, d, f, G, dtype, False, True)
        router = (torch.randn((E, d), device="cuda", generator=gen) / d ** 0.5).to(BF)
        scores, idx, tw = bm.router_topk(hidden.to(BF), router, k)
        r = bm.forward_w4(hidden, scores, k, w)
        bm.sync_status()
        assert torch.equal(r["idx"], idx)
        assert bool(((r["w"] - tw).abs() <= 1e-6 * tw).all())
        check_layer_w4(r, hidden, scores, k, mats, True, G)
        hidden = (hidden.float() + r["out"]).to(dtype)
    head = weights(gen, (V, d), G, dtype, True)
    logits = bm.w4_gemm(hidden, bm.W4Matrix(*head))
    bm.sync_status()
    check_gemm(logits, hidden, dense(*head, G), G)


def test_expired_waits_are_reported_and_recoverable():
    """With a limit of 1 ns the kernels' waits run out: the status reports it (or every copy was
    there in time), the calls return, and the next call is right."""
    T, E, k, d, f, G = 6, 12, 3, 1024, 512, 64
    mats, w = make_layer(41, E, d, f, G, BF, True, True)
    gen = generator(42)
    x = torch.randn((T, d), device="cuda", generator=gen).to(BF)
    s = torch.randn((T, E), device="cuda", generator=gen)
    m = weights(gen, (500, d), G, BF, True)
    bm.sync_status()
    bm.set_wait_limit_ns(1)
    try:
        for call in (lambda: bm.forward_w4(x, s, k, w), lambda: bm.forward_w4(x[:1], s[:1], k, w),
                     lambda: bm.w4_gemm(x, bm.W4Matrix(*m)), lambda: bm.w4_gemm(x[:2], bm.W4Matrix(*m))):
            call()
            try:
                bm.sync_status()
            except bm.MoeError as e:
                assert e.code == bm.MOE_ERR_TIMEOUT
    finally:
        bm.set_wait_limit_ns(0)
    bm.sync_status()
    check_layer_w4(bm.forward_w4(x, s, k, w), x, s, k, mats, True, G)
    check_gemm(bm.w4_gemm(x, bm.W4Matrix(*m)), x, dense(*m, G), G)
