"""The whole layer for a few tokens (moe_layer_few, moe_layer_few_routed) on the GPU.

  * inputs on which every step is exact in fp32 (integers; gate sums so large
    that SiLU(g) = g; power-of-two routing weights): y bit for bit, so a wrong
    row, column, scale, nibble, token or a lost slot shows;
  * random inputs against a float64 evaluation under a bound derived from the
    sums' lengths;
  * the routing against float64 logits: ids equal, ties to the lower expert;
  * masked slots, repeated ids, NaN weights and tokens next to healthy ones.
"""
import pytest
import torch

from helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda:0"
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
KINDS = ["16bit", "fp8", "mx"]


def _mr():
    import mixture_experts_routed_moe_amd as mr
    return mr


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _exact_weights(E, N, Kd, kind, dtype, g, choices):
    """(the framework's weights, their float64 values): values from `choices`
    times a power of two per row (FP8) or per 32 elements (MXFP4)."""
    mr = _mr()
    idx = torch.randint(len(choices), (E, N, Kd), generator=g, device=DEV)
    v = torch.tensor(choices, device=DEV)[idx]
    if kind == "16bit":
        return v.to(dtype), v.double()
    if kind == "fp8":
        k = torch.randint(-1, 2, (E, N), generator=g, device=DEV).float()
        return (mr.FP8Weights(v.to(torch.float8_e4m3fn).view(torch.uint8), torch.exp2(k)),
                v.double() * torch.exp2(k).double().unsqueeze(-1))
    k = torch.randint(-1, 2, (E, N, Kd // 32), generator=g, device=DEV)
    code = torch.bucketize(v.abs(), GRID.to(DEV)) + 8 * (v < 0)
    code = code.view(E, N, Kd // 2, 2).to(torch.uint8)
    packed = (code[..., 0] | (code[..., 1] << 4)).contiguous()
    value = v.double() * torch.exp2(k.double()).repeat_interleave(32, -1)
    return mr.MXWeights(packed, (k + 127).to(torch.uint8)), value


def _random_weights(E, N, Kd, kind, dtype, g):
    mr = _mr()
    w = (torch.randn(E, N, Kd, generator=g, device=DEV) * Kd ** -0.5).to(dtype)
    if kind == "16bit":
        return w, w.double()
    if kind == "fp8":
        q = mr.quantize_fp8_rows(w)
        return q, q.codes.view(torch.float8_e4m3fn).double() * q.scales.double().unsqueeze(-1)
    q = mr.quantize_mx_weights(w)
    code = torch.stack([q.packed & 15, q.packed >> 4], -1).view(E, N, Kd).long()
    grid = torch.cat([GRID, -GRID]).double().to(DEV)
    return q, grid[code] * torch.exp2(q.scales.double() - 127).repeat_interleave(32, -1)


def _layer64(x, ids, w, wg, wu, wd):
    """y in float64 and a bound on the fp32 path's error before the last rounding.

    A product of operands is exact in the matrix unit; a sum of n products is
    off by at most n U times the sum of magnitudes, with U = 2^-23 (an fp32
    addition that truncates). SiLU has slope at most 1.1 and costs 8 U with
    the products behind it; hw as two bf16 adds 2^-17 of itself."""
    U = 2.0 ** -23
    T, H = x.shape
    D = wg.shape[1]
    y = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    err = torch.zeros_like(y)
    n = ids.shape[1]
    for t in range(T):
        for k in range(n):
            e = int(ids[t, k])
            if e < 0 or e >= wg.shape[0]:
                continue
            xt = x[t].double()
            g, u = wg[e] @ xt, wu[e] @ xt
            dg, du = (H * U * (m[e].abs() @ xt.abs()) for m in (wg, wu))
            s = g * torch.sigmoid(g)
            h = s * u
            dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 8 * U * h.abs()
            y[t] += w[t, k].double() * (wd[e] @ h)
            err[t] += w[t, k].double().abs() * (wd[e].abs() @ (dh + (n * D * U + 2.0 ** -17) * h.abs()))
    return y, err


def _close(got, y, err):
    t = got.dtype
    step = torch.finfo(t).eps / 2 * y.abs() + torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    bad = (got.double() - y).abs() > err * (1 + torch.finfo(t).eps) + step
    assert not bad.any(), ((got.double() - y).abs() - err - step).max()


SHAPES = [  # T, H, D, E, K
    (1, 256, 256, 8, 2), (1, 2048, 768, 16, 8), (3, 512, 256, 4, 4), (16, 256, 256, 5, 2), (7, 1792, 512, 33, 3),
    (16, 4352, 256, 6, 2), (2, 7168, 256, 3, 1), (16, 256, 1280, 70, 8),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T, H, D, E, K", SHAPES)
def test_exact_layers_bit_for_bit(dtype, kind, T, H, D, E, K):
    mr = _mr()
    g = _gen(T * H + K)
    # x in {1, 2}: every gate sum is at least H / 4 >= 64 (weights 1 and above,
    # scales 1/2 and above), where SiLU(g) = g in fp32; |u| <= 4 H, so g * u
    # stays below 2^24 only for the short rows: the up weights are sparse
    x = torch.randint(1, 3, (T, H), generator=g, device=DEV).to(dtype)
    wg, vg = _exact_weights(E, D, H, kind, dtype, g, [1.0])
    sparse = [0.0] * 63 + [1.0]
    wu, vu = _exact_weights(E, D, H, kind, dtype, g, sparse)
    wd, vd = _exact_weights(E, H, D, kind, dtype, g, sparse + [-1.0])
    ids = torch.stack([torch.randperm(E, generator=g, device=DEV)[:K] for _ in range(T)]).to(torch.int32)
    w = torch.exp2(torch.randint(-8, -5, (T, K), generator=g, device=DEV).float())
    if T > 2:
        ids[1, 0] = -1
        ids[2] = -5                                    # a token without experts
        ids[0, -1] = ids[0, 0]                         # an expert twice
    y, _ = _layer64(x, ids, w, vg, vu, vd)
    h_top = 0.0
    for t in range(T):
        for e in ids[t].tolist():
            if e >= 0:
                h_top = max(h_top, float(((vg[e] @ x[t].double()) * (vu[e] @ x[t].double())).max()))
    # hw / 2^-10 is an integer (scales give 2^-1 each, weights 2^-8): exact as
    # two bf16 (16 bits), and so are the sums, if these hold
    exact = h_top * 2 ** 2 < 2 ** 16 or (dtype == torch.float16 and kind == "16bit")
    partial = float(_layer64(x, ids, w, vg, vu, vd.abs())[0].max())      # no partial sum is larger
    got = mr.moe_layer_few_routed(x, ids, w, wg, wu, wd)
    torch.cuda.synchronize()
    if exact and partial * 2 ** 11 < 2 ** 23:
        assert torch.equal(got, y.to(dtype))
    else:
        # beyond: hw rounds to 16 bits (2^-17 of itself); an fp16 y past 65520,
        # half a step beyond the largest value, rounds to infinity
        mag = sum(w[:, k].double().unsqueeze(1) for k in range(K))
        tol = torch.finfo(dtype).eps / 2 * y.abs() + 2.0 ** -16 * mag * h_top * vd.abs().sum(-1).max()
        over = torch.isinf(y.to(dtype)) & torch.isinf(got) & (got.sign() == y.sign())
        assert (((got.double() - y).abs() <= tol) | over).all()
    if T > 2:
        assert (got[2] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T, H, D, E, K", SHAPES)
def test_random_layers_against_float64(dtype, kind, T, H, D, E, K):
    mr = _mr()
    g = _gen(T + H)
    x = torch.randn(T, H, generator=g, device=DEV).to(dtype)
    router = torch.randn(E, H, generator=g, device=DEV) * 0.02
    (wg, vg), (wu, vu), (wd, vd) = (_random_weights(E, *s, kind, dtype, g) for s in ((D, H), (D, H), (H, D)))
    y, ids, w = mr.moe_layer_few(x, router, wg, wu, wd, K)
    torch.cuda.synchronize()
    want, err = _layer64(x, ids, w, vg, vu, vd)
    _close(y, want, err)
    again = mr.moe_layer_few_routed(x, ids, w, wg, wu, wd)
    assert torch.equal(again, y)                       # the same routing, given


def _route64(x, router, bias, K, renorm):
    logits = x.double() @ router.double().t()
    if bias is not None:
        logits = logits + bias.double()
    order = torch.sort(logits.float(), dim=-1, descending=True, stable=True).indices[:, :K]
    p = torch.softmax(logits, -1).gather(1, order)
    return order, p / p.sum(-1, keepdim=True) if renorm else p, logits


@pytest.mark.parametrize("E, K", [(1, 1), (8, 8), (64, 5), (65, 6), (128, 8), (256, 8), (257, 3), (1000, 64), (1024, 17)])
@pytest.mark.parametrize("T", [1, 2, 5, 16])
def test_routing(E, K, T):
    mr = _mr()
    H, D = 512, 128
    for renorm, with_bias, dtype in ((True, False, torch.bfloat16), (False, True, torch.float16)):
        g = _gen(E + T)
        x = torch.randn(T, H, generator=g, device=DEV).to(dtype)
        router = torch.randn(E, H, generator=g, device=DEV) * 0.05
        bias = torch.randn(E, generator=g, device=DEV) if with_bias else None
        weights = torch.zeros(E, D, H, dtype=dtype, device=DEV), torch.zeros(E, H, D, dtype=dtype, device=DEV)
        y, ids, w = mr.moe_layer_few(x, router, weights[0], weights[0], weights[1], K, renorm=renorm, bias=bias)
        want_ids, want_w, logits = _route64(x, router, bias, K, renorm)
        assert torch.equal(ids.long(), want_ids)
        # expf 4 U, its argument's rounding range * U (twice: numerator and sum), the sums' E and K terms in trees
        tol = 2.0 ** -24 * (40 + 4 * float(logits.max() - logits.min()))
        assert ((w.double() - want_w).abs() <= tol * want_w).all()
        assert (y == 0).all()


def test_ties_go_to_the_lower_expert():
    mr = _mr()
    H, D, E, K = 256, 128, 300, 7
    g = _gen(5)
    x = torch.randn(3, H, generator=g, device=DEV).to(torch.bfloat16)
    base = torch.randn(4, H, generator=g, device=DEV)
    router = base[torch.randint(4, (E,), generator=g, device=DEV)].contiguous()     # many equal rows
    router[17] = 0.0
    router[41] = -0.0                                                               # logits 0 and -0 tie
    z = torch.zeros(E, D, H, dtype=torch.bfloat16, device=DEV)
    _, ids, _ = mr.moe_layer_few(x, router, z, z, z.view(E, H, D), K)
    assert torch.equal(ids.long(), _route64(x, router, None, K, True)[0])
    _, ids, w = mr.moe_layer_few(torch.zeros_like(x), router, z, z, z.view(E, H, D), K)
    assert torch.equal(ids, torch.arange(K, device=DEV, dtype=torch.int32).expand(3, K))
    assert ((w - 1 / K).abs() <= 1e-6).all()


@pytest.mark.parametrize("kind", KINDS)
def test_nothing_leaks_between_tokens_and_experts(kind):
    mr = _mr()
    T, H, D, E, K, dtype = 6, 512, 256, 9, 2, torch.bfloat16
    g = _gen(3)
    x = torch.randn(T, H, generator=g, device=DEV).to(dtype)
    (wg, vg), (wu, vu), (wd, vd) = (_random_weights(E, *s, kind, dtype, g) for s in ((D, H), (D, H), (H, D)))
    ids = torch.tensor([[0, 1], [2, 3], [-1, 4], [5, 9], [2, 2], [7, 1]], dtype=torch.int32, device=DEV)  # 9: no expert
    w = torch.rand(T, K, generator=g, device=DEV)
    w[2, 0] = float("nan")                             # the weight of a masked slot is not used
    w[3, 1] = float("inf")
    clean = mr.moe_layer_few_routed(x, ids, w, wg, wu, wd)
    assert torch.isfinite(clean).all()
    want, err = _layer64(x, ids, w, vg, vu, vd)
    _close(clean, want, err)

    def spoil(weights, experts):
        for q in weights:
            t = q if kind == "16bit" else q.scales
            for e in experts:
                t[e] = float("nan") if kind != "mx" else 255
        return weights

    spoil((wg, wu, wd), (6, 8))                        # experts of no token
    assert torch.equal(mr.moe_layer_few_routed(x, ids, w, wg, wu, wd), clean)
    bad = x.clone()
    bad[1] = float("inf")
    got = mr.moe_layer_few_routed(bad, ids, w, wg, wu, wd)
    keep = [0, 2, 3, 4, 5]
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[1]).all()
    spoil((wg, wu, wd), (1,))                          # expert 1 serves tokens 0 and 5
    got = mr.moe_layer_few_routed(x, ids, w, wg, wu, wd)
    keep = [1, 2, 3, 4]
    assert torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T, H, D, E, K", [(16, 256, 256, 1024, 64), (1, 65792, 256, 2, 1), (16, 65792, 256, 2, 2)])
def test_every_expert_and_the_longest_rows(kind, T, H, D, E, K):
    """1024 distinct experts in one call; more column tiles than workgroups run
    at once (the down kernel then writes y itself)."""
    mr = _mr()
    g = _gen(T + E)
    x = torch.randn(T, H, generator=g, device=DEV).to(torch.bfloat16)
    (wg, vg), (wu, vu), (wd, vd) = (_random_weights(E, *s, kind, torch.bfloat16, g) for s in ((D, H), (D, H), (H, D)))
    ids = torch.randperm(T * K, generator=g, device=DEV).view(T, K).to(torch.int32) % E
    w = torch.rand(T, K, generator=g, device=DEV)
    y = mr.moe_layer_few_routed(x, ids, w, wg, wu, wd)
    torch.cuda.synchronize()
    want, err = _layer64(x, ids, w, vg, vu, vd)
    _close(y, want, err)


def test_weights_none_and_all_masked():
    mr = _mr()
    T, H, D, E, K, dtype = 4, 256, 128, 6, 3, torch.float16
    g = _gen(8)
    x = torch.randn(T, H, generator=g, device=DEV).to(dtype)
    wg, wu, wd = (_random_weights(E, *s, "16bit", dtype, g)[0] for s in ((D, H), (D, H), (H, D)))
    ids = torch.randint(0, E, (T, K), generator=g, device=DEV).to(torch.int32)
    assert torch.equal(mr.moe_layer_few_routed(x, ids, None, wg, wu, wd),
                       mr.moe_layer_few_routed(x, ids, torch.ones(T, K, device=DEV), wg, wu, wd))
    y = torch.full((T, H), 3.0, dtype=dtype, device=DEV)
    mr.moe_layer_few_routed(x, torch.full_like(ids, -1), None, wg, wu, wd, y=y)
    assert (y == 0).all()


def test_64_slots_and_rows_past_the_batch():
    mr = _mr()
    T, H, D, E, K, dtype = 16, 256, 128, 20, 64, torch.bfloat16
    g = _gen(9)
    x = torch.randn(T, H, generator=g, device=DEV).to(dtype)
    (wg, vg), (wu, vu), (wd, vd) = (_random_weights(E, *s, "16bit", dtype, g) for s in ((D, H), (D, H), (H, D)))
    ids = torch.randint(-4, E, (T, K), generator=g, device=DEV).to(torch.int32)      # every id several times
    w = torch.rand(T, K, generator=g, device=DEV) / K
    big = torch.full((T + 4, H), 7.0, dtype=dtype, device=DEV)
    mr.moe_layer_few_routed(x, ids, w, wg, wu, wd, y=big[2:T + 2])
    want, err = _layer64(x, ids, w, vg, vu, vd)
    _close(big[2:T + 2], want, err)
    assert (big[:2] == 7).all() and (big[T + 2:] == 7).all()


def _small(seed=1, T=5, dtype=torch.bfloat16):
    g = _gen(seed)
    H, D, E = 512, 256, 12
    d = dict(x=torch.randn(T, H, generator=g, device=DEV).to(dtype),
             w_router=torch.randn(E, H, generator=g, device=DEV) * 0.05)
    for n, s in (("w_gate", (D, H)), ("w_up", (D, H)), ("w_down", (H, D))):
        d[n] = _random_weights(E, *s, "16bit", dtype, g)[0]
    return d


def test_streams_graphs_and_a_shared_workspace():
    mr = _mr()
    d, e = _small(1), _small(2, T=16)
    want = [mr.moe_layer_few(**v, top_k=3) for v in (d, e)]
    ws = mr.few_workspace(16, 3, 12, 256, DEV)
    outs = [[torch.empty_like(t) for t in w] for w in want]
    graphs = []
    for v, o in zip((d, e), outs):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            mr.moe_layer_few(**v, top_k=3, y=o[0], topk_ids=o[1], topk_weights=o[2], workspace=ws)
        graphs.append(gr)
    for i in range(4):                                 # two graphs, one workspace, one after the other
        for v in (d, e):
            v["x"].copy_(torch.randn(v["x"].shape, generator=_gen(20 + i), device=DEV).to(v["x"].dtype))
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        for v, o in zip((d, e), outs):
            for a, b in zip(o, mr.moe_layer_few(**v, top_k=3)):
                assert torch.equal(a, b)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]   # two calls at once, a workspace each
    torch.cuda.synchronize()
    got = []
    for v, s in zip((d, e), side):
        with torch.cuda.stream(s):
            got.append(mr.moe_layer_few(**v, top_k=3, workspace=mr.few_workspace(16, 3, 12, 256, DEV)))
    torch.cuda.synchronize()
    for v, o in zip((d, e), got):
        for a, b in zip(o, mr.moe_layer_few(**v, top_k=3)):
            assert torch.equal(a, b)


def test_near_the_general_path():
    """The same layer by moe_gate, moe_dispatch and moe_routed_forward, which
    round h and expert_out to 16 bits on the way."""
    mr = _mr()
    d = _small(4, T=16)
    y, ids, w = mr.moe_layer_few(**d, top_k=4)
    gids, gw, _ = mr.moe_gate(d["x"], d["w_router"], 4)
    assert torch.equal(ids, gids)
    tables = mr.moe_dispatch(gids, gw, 12)
    z = mr.moe_routed_forward(d["x"], d["w_gate"], d["w_up"], d["w_down"], tables)
    assert float((y.double() - z.double()).norm() / z.double().norm()) <= 3 * torch.finfo(y.dtype).eps / 2


def test_one_block_after_another():
    """norm -> layer -> norm -> layer, as a decoder calls them, against float64."""
    mr = _mr()
    d = _small(6, T=3)
    g1, g2, gp = (1 + 0.1 * torch.randn(512, generator=_gen(i), device=DEV) for i in (1, 2, 3))
    r = torch.randn(3, 512, generator=_gen(4), device=DEV)
    layer = {k: v for k, v in d.items() if k != "x"}
    _, h = mr.moe_block_norm(None, r, gamma_pre=g1, dtype=torch.bfloat16)
    y, ids, w = mr.moe_layer_few(h, **layer, top_k=3)
    r2, h2 = mr.moe_block_norm(y, r, gamma_post=gp, gamma_pre=g2, alpha=0.5)
    y2, _, _ = mr.moe_layer_few(h2, **layer, top_k=3)
    torch.cuda.synchronize()
    norm = lambda v, g: v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-6) * g.double()  # noqa: E731
    v64 = [layer[n].double() for n in ("w_gate", "w_up", "w_down")]
    step = torch.finfo(torch.bfloat16).eps / 2
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    want_h = norm(r.double(), g1)
    assert rel(h, want_h) <= step
    want_y = _layer64(h, ids, w, *v64)[0]
    assert rel(y, want_y) <= step
    want_r = r.double() + 0.5 * norm(y.double(), gp)
    assert rel(r2, want_r) <= 2.0 ** -20
    assert rel(h2, norm(want_r, g2)) <= step
    assert torch.isfinite(y2).all()


def test_no_tokens_and_refusals_of_the_binding():
    mr = _mr()
    d = _small()
    y, ids, w = mr.moe_layer_few(**dict(d, x=d["x"][:0]), top_k=3)
    assert y.shape == (0, 512) and ids.shape == w.shape == (0, 3)
    many = torch.zeros(17, 512, dtype=torch.bfloat16, device=DEV)
    for bad in (dict(x=many), dict(x=d["x"].float()), dict(x=d["x"][:, ::2]), dict(w_router=d["w_router"].half()),
                dict(w_router=d["w_router"][:, :256]), dict(w_up=d["w_up"][:, :128]), dict(w_down=d["w_down"].half()),
                dict(top_k=13), dict(top_k=0), dict(bias=torch.zeros(3, device=DEV)),
                dict(w_up=mr.quantize_fp8_rows(d["w_up"])), dict(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
                dict(y=torch.empty(5, 512, device=DEV))):
        kw = dict(d, top_k=3)
        kw.update(bad)
        with pytest.raises(mr.MoeError):
            mr.moe_layer_few(**kw)
