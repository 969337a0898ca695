"""MXFP4 x MXFP4 experts (moe_*_mx4) on the GPU.

Stage by stage against float64, each stage on the codes that the GPU's stage
before it wrote:
  * the down product on inputs whose sums are exact in fp32, with a random
    scale in every 32-block on both sides: bit for bit;
  * hq, hs: the codes of SiLU(g) * u from float64 sums, or the neighbours that
    the fp32 sums' error allows;
  * expert_out within its rounding and the sums' error; y = the library's
    reduce of expert_out, bit for bit.
"""
import pytest
import torch

import synthetic as S
from helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda:0"
U = 2.0 ** -23            # of one fp32 addition that truncates


def _mr():
    import mixture_experts_routed_moe_amd as mr
    return mr


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def _decode(codes, scales):
    """float64 values of MXFP4 codes [..., n/2] with E8M0 scales [..., n/32]."""
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    v = torch.cat([GRID, -GRID]).to(DEV)[c]
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1)


def _encode(v, scales):
    """Values of v [rows, n] float64 rounded to E2M1 at the given scales
    (nearest, ties to the even code, saturating)."""
    X = torch.exp2(scales.double() - 127).repeat_interleave(32, -1)
    a = (v / X).abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), v) * X


def _exact_codes(shape, g):
    """Random MXFP4 codes with scales 2^-1 .. 2^1 per block: every product is a
    multiple of 2^-4 and a sum of 1024 of them stays below 2^20."""
    n = shape[-1]
    codes = torch.randint(0, 256, (*shape[:-1], n // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.randint(126, 129, (*shape[:-1], n // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def _routing(T, E, K, seed):
    """Ids with a hot expert, masked slots, an expert twice in a token."""
    g = _gen(seed)
    ids = torch.stack([torch.randperm(E, generator=g, device=DEV)[:K] for _ in range(T)]).to(torch.int32)
    ids[::3, 0] = 1
    if T > 6:
        ids[::7, -1] = -1
        ids[5] = -1
        ids[6, -1] = ids[6, 0]
    return ids, torch.rand(T, K, generator=g, device=DEV)


def _rows_of(tables):
    sizes, offs = tables.group_sizes.tolist(), tables.group_offsets.tolist()
    return [(e, slice(o, o + n)) for e, (n, o) in enumerate(zip(sizes, offs)) if n]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("block_m", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T, D", [(200, 512), (1, 256), (333, 768), (700, 1024)])
def test_down_exact(dtype, block_m, T, D):
    mr = _mr()
    H, E, K = 512, 5, 3
    ids, w = _routing(T, E, K, T)
    tables = mr.moe_dispatch(ids, w, E, block_m=block_m)
    g = _gen(D)
    P = T * K
    hq, hs = _exact_codes((P, D), g)
    wq, wsc = _exact_codes((E, H, D), g)
    eo = torch.full((P, H), float("nan"), dtype=dtype, device=DEV)
    mr.moe_expert_down_mx4(hq, hs, mr.MXWeights(wq, wsc), tables, dtype, expert_out=eo)
    h64, w64 = _decode(hq, hs), _decode(wq, wsc)
    n = int(tables.group_sizes.sum())
    for e, rows in _rows_of(tables):
        assert torch.equal(eo[rows], (h64[rows] @ w64[e].t()).to(dtype)), "expert %d" % e
    assert torch.isnan(eo[n:]).all()                       # rows behind the last are left alone


def _check_hidden(tables, xq, xs, wg, wu, hq, hs):
    x64 = _decode(xq, xs)
    got = _decode(hq, hs)
    H = x64.shape[1]
    for e, rows in _rows_of(tables):
        x = x64[tables.sorted_token[rows].long()]
        g, u = x @ wg[e].t(), x @ wu[e].t()
        dg, du = (H * U * (x.abs() @ m[e].abs().t()) for m in (wg, wu))
        s = g * torch.sigmoid(g)
        h = s * u
        err = 1.1 * dg * (u.abs() + du) + s.abs() * du + 8 * U * h.abs()
        # the scale: floor(log2 amax) - 2 of an amax within its error
        top, slack = (t.view(t.shape[0], -1, 32).amax(-1) for t in (h.abs(), err))
        lo, hi = (torch.floor(torch.log2(t.clamp(min=2.0 ** -120))) - 2 + 127 for t in (top - slack, top + slack))
        sc = hs[rows].double()
        zero = top == 0                                    # the scale of a zero block is 127
        assert (torch.where(zero, sc == 127, (sc >= lo) & (sc <= hi))).all(), "scales of expert %d" % e
        below, above = _encode(h - err, hs[rows]), _encode(h + err, hs[rows])
        assert ((got[rows] >= below) & (got[rows] <= above)).all(), "codes of expert %d" % e


def _forward(d, block_m=None, dtype=torch.bfloat16):
    """Runs the forward and checks every stage."""
    mr = _mr()
    T, H, D, E = d["T"], d["H"], d["D"], d["E"]
    w = [mr.quantize_mx_weights(d[n]) for n in ("w_gate", "w_up", "w_down")]
    tables = mr.moe_dispatch(d["topk_ids"], d["topk_weights"], E, block_m=block_m)
    ws, eo, xq, xs, hq, hs = mr.forward_mx4_workspace(tables, H, D, dtype)
    ws.fill_(0xFF)                                         # NaN rows, NaN scales
    y = torch.full((T, H), float("nan"), dtype=dtype, device=DEV)
    mr.moe_routed_forward_mx4(d["x"], *w, tables, y=y, workspace=ws)
    torch.cuda.synchronize()
    n = int(tables.group_sizes.sum())
    assert (hq[n:] == 0xFF).all() and (hs[n:] == 0xFF).all() and (eo.view(torch.uint8)[n:] == 0xFF).all()
    want_xq, want_xs = mr.quantize_mx_rows(d["x"], mr.MX_FP4)
    assert torch.equal(xq, want_xq) and torch.equal(xs, want_xs)
    wg, wu, wd = ([_decode(q.packed[e], q.scales[e]) if e in used else None for e in range(E)]
                  for used in [{e for e, _ in _rows_of(tables)}] for q in w)
    _check_hidden(tables, xq, xs, wg, wu, hq, hs)
    h64 = _decode(hq[:n], hs[:n])
    step = torch.finfo(dtype).eps / 2
    for e, rows in _rows_of(tables):
        want = h64[rows] @ wd[e].t()
        err = D * U * (h64[rows].abs() @ wd[e].abs().t())
        tiny = torch.finfo(dtype).smallest_normal * step
        assert ((eo[rows].double() - want).abs() <= err * (1 + 2 * step) + step * want.abs() + tiny).all(), e
    assert torch.equal(y, mr.moe_reduce_fused(eo, tables.token_topk_to_pos.view(T, -1), d["topk_weights"]))
    return y, w, tables


def _inputs(T, H, D, E, K, dtype, seed):
    g = _gen(seed)
    ids, w = _routing(T, E, K, seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return dict(T=T, H=H, D=D, E=E, K=K, x=r(T, H).to(dtype), topk_ids=ids, topk_weights=w,
                w_gate=(r(E, D, H) * H ** -0.5).to(dtype), w_up=(r(E, D, H) * H ** -0.5).to(dtype),
                w_down=(r(E, H, D) * D ** -0.5).to(dtype))


@pytest.mark.parametrize("block_m", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("T, H, D, E, K", [(1, 256, 256, 4, 2), (67, 512, 768, 9, 3), (300, 1792, 256, 5, 3),
                                           (700, 256, 512, 3, 2), (16, 2048, 1024, 40, 8)])
def test_forward_stages(block_m, T, H, D, E, K):
    _forward(_inputs(T, H, D, E, K, torch.bfloat16, T), block_m)


def test_forward_fp16_and_default_blocks():
    _forward(_inputs(130, 512, 512, 6, 2, torch.float16, 3), dtype=torch.float16)


def test_all_masked_and_zero_rows():
    mr = _mr()
    d = _inputs(40, 256, 256, 4, 2, torch.bfloat16, 5)
    d["x"][3] = 0
    y, w, tables = _forward(d)
    assert (y[3] == 0).all()                               # zero blocks: scale 127, codes 0
    d["topk_ids"] = torch.full_like(d["topk_ids"], -1)
    tables = mr.moe_dispatch(d["topk_ids"], d["topk_weights"], 4)
    assert (mr.moe_routed_forward_mx4(d["x"], *w, tables) == 0).all()


@pytest.mark.parametrize("ci", [1, 2])
def test_workloads(ci):
    cfg = S.CONFIGS[ci]
    _forward(S.make_moe_inputs(cfg, device=DEV, T=cfg["T"]))


def test_norm_feeds_the_experts():
    """norm (MXFP4 codes) -> gate/up -> down -> combine with the next norm."""
    mr = _mr()
    d = _inputs(50, 512, 256, 6, 2, torch.bfloat16, 9)
    w = [mr.quantize_mx_weights(d[n]) for n in ("w_gate", "w_up", "w_down")]
    g1, g2 = (1 + 0.1 * torch.randn(512, generator=_gen(i), device=DEV) for i in (1, 2))
    r = torch.randn(50, 512, generator=_gen(3), device=DEV)
    _, h, xq, xs = mr.moe_block_norm(None, r, gamma_pre=g1, quant="mxfp4", dtype=torch.bfloat16)
    tables = mr.moe_dispatch(d["topk_ids"], d["topk_weights"], 6, block_m=mr.default_block_m(50, 2, 6, "mx4"))
    hq, hs = mr.moe_expert_gate_up_mx4(xq, xs, w[0], w[1], tables)
    _check_hidden(tables, xq, xs, *([_decode(q.packed[e], q.scales[e]) for e in range(6)] for q in w[:2]), hq, hs)
    eo = mr.moe_expert_down_mx4(hq, hs, w[2], tables)
    pos = tables.token_topk_to_pos.view(50, 2)
    r2, h2 = mr.moe_reduce_norm(eo, pos, d["topk_weights"], r, gamma_pre=g2, gamma_post=g1)
    y = mr.moe_reduce_fused(eo, pos, d["topk_weights"], out_dtype=torch.float32)
    want = r.double() + y.double() / torch.sqrt(y.double().square().mean(-1, keepdim=True) + 1e-6) * g1.double()
    assert float((r2.double() - want).norm() / want.norm()) <= 2.0 ** -20
    assert torch.isfinite(h2).all()


def test_graph_replays_and_streams():
    mr = _mr()
    d = _inputs(90, 512, 256, 6, 2, torch.bfloat16, 12)
    w = [mr.quantize_mx_weights(d[n]) for n in ("w_gate", "w_up", "w_down")]
    tables = mr.moe_dispatch(d["topk_ids"], d["topk_weights"], 6)
    ws = mr.forward_mx4_workspace(tables, 512, 256, torch.bfloat16)[0]
    y = torch.empty_like(d["x"])
    want = mr.moe_routed_forward_mx4(d["x"], *w, tables)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        mr.moe_routed_forward_mx4(d["x"], *w, tables, y=y, workspace=ws)
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mr.moe_dispatch(d["topk_ids"], d["topk_weights"], 6, tables.block_m, tables)
        mr.moe_routed_forward_mx4(d["x"], *w, tables, y=y, workspace=ws)
    for i in range(4):
        d["x"].copy_(torch.randn(90, 512, generator=_gen(30 + i), device=DEV))
        d["topk_ids"].copy_(_routing(90, 6, 2, 40 + i)[0])
        graph.replay()
        torch.cuda.synchronize()
        fresh = mr.moe_dispatch(d["topk_ids"], d["topk_weights"], 6)
        assert torch.equal(y, mr.moe_routed_forward_mx4(d["x"], *w, fresh))


def test_refusals_of_the_binding():
    mr = _mr()
    d = _inputs(8, 256, 256, 4, 2, torch.bfloat16, 1)
    w = [mr.quantize_mx_weights(d[n]) for n in ("w_gate", "w_up", "w_down")]
    tables = mr.moe_dispatch(d["topk_ids"], d["topk_weights"], 4)
    xq, xs = mr.quantize_mx_rows(d["x"], mr.MX_FP4)
    bad_calls = [
        lambda: mr.moe_routed_forward_mx4(d["x"].float(), *w, tables),
        lambda: mr.moe_routed_forward_mx4(d["x"], d["w_gate"], w[1], w[2], tables),
        lambda: mr.moe_routed_forward_mx4(d["x"][:7], *w, tables),
        lambda: mr.moe_routed_forward_mx4(d["x"], *w, tables, y=torch.empty(8, 128, device=DEV)),
        lambda: mr.moe_routed_forward_mx4(d["x"], *w, tables, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)),
        lambda: mr.moe_expert_gate_up_mx4(xq, xs[:, :4].contiguous(), w[0], w[1], tables),
        lambda: mr.moe_expert_gate_up_mx4(*mr.quantize_mx_rows(d["x"], mr.MX_FP8), w[0], w[1], tables),
        lambda: mr.moe_expert_down_mx4(xq, xs, w[2], tables),
        lambda: mr.moe_expert_down_mx4(xq.repeat(2, 1), xs.repeat(2, 1), w[2], tables, torch.float32),
    ]
    for call in bad_calls:
        with pytest.raises(mr.MoeError):
            call()
