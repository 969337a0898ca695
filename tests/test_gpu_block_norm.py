"""The norms around a block (moe_block_norm, moe_reduce_norm) on the GPU.

The fp32 path is compared with a float64 evaluation of the definition under
bounds derived from it; the 16-bit paths widen exactly and run the same
arithmetic, so their outputs must be the fp32 path's outputs rounded once,
bit for bit; and the codes must be those of the library's quantisers on the
fp32 path's h (which holds the unrounded values), bit for bit.
"""
import pytest
import torch

from helpers import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs a GPU")]

DEV = "cuda:0"
U = 2.0 ** -24
EPS = 1e-6


def _mr():
    import mixture_experts_routed_moe_amd as mr
    return mr


def _inputs(T, H, gate="none", post=True, seed=0, dtype=torch.float32, K=0, mask=0.2):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(residual=(3 * r(T, H)).to(dtype), gamma_pre=1 + 0.2 * r(H),
             gamma_post=0.5 + 0.2 * r(H) if post else None, alpha=0.75,
             gate={"none": None, "channel": 1 + 0.1 * r(H), "token": torch.sigmoid(r(T, 1)),
                   "full": torch.sigmoid(r(T, H)).to(dtype)}[gate])
    if K:
        rows = T * K + 3
        d["rows"] = r(rows, H).to(dtype)
        pos = torch.randperm(rows, generator=g)[:T * K].to(torch.int32)
        pos[torch.rand(T * K, generator=g) < mask] = -1
        unread = torch.ones(rows, dtype=torch.bool)
        unread[pos[pos >= 0].long()] = False
        d["rows"][unread] = float("nan")              # rows that no slot names are never read
        d["pos"] = pos.view(T, K)
        d["pos"][0] = -1                              # a token that no expert served
        d["w"] = torch.softmax(r(T, K), -1)
    else:
        d["y"] = r(T, H).to(dtype)
    return {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in d.items()}


def _call(d, **more):
    mr = _mr()
    kw = dict(gamma_post=d["gamma_post"], gamma_pre=d["gamma_pre"], gate=d["gate"], alpha=d["alpha"], eps=EPS)
    kw.update(more)
    if "rows" in d:
        out = mr.moe_reduce_norm(d["rows"], d["pos"], d["w"], d["residual"], **kw)
    else:
        out = mr.moe_block_norm(d["y"], d["residual"], **kw)
    torch.cuda.synchronize()
    return out


def _reference(d):
    """r and n in float64 with bounds on the fp32 path's errors.

    A value of the combine is off by at most K U vabs (K fused multiply-adds,
    vabs the sum of magnitudes). A sum of squares is at most 64 additions
    deep (16 values a thread, 6 lane steps, 16 waves, the square): 64 U
    relative. So rstd is off by half that, the division's and square root's
    2 U, and what the combine's errors make of it; the products that follow
    add less than 8 U. 64 U covers the first and third."""
    K = d["w"].shape[1] if "w" in d else 0
    if K:
        p = d["pos"].long()
        x = d["rows"][p.clamp(min=0)].double() * d["w"].double()[:, :, None]
        x = torch.where((p >= 0)[:, :, None], x, 0.0)
        v, vabs = x.sum(1), x.abs().sum(1)
    else:
        v = d["y"].double()
        vabs = v.abs()
    H = v.shape[1]
    b, babs, rel = v, vabs, torch.full_like(v[:, :1], (K + 8) * U)
    if d["gamma_post"] is not None:
        rstd = 1.0 / torch.sqrt(v.square().mean(1, keepdim=True) + EPS)
        # d(rstd) / rstd <= sum |v| |dv| / (H (mean v^2 + eps))
        rel = rel + 64 * U + K * U * (v.abs() * vabs).mean(1, keepdim=True) * rstd ** 2
        b, babs = v * rstd * d["gamma_post"].double(), vabs * rstd * d["gamma_post"].double().abs()
    gate = 1.0 if d["gate"] is None else d["gate"].double()
    r = d["residual"].double() + d["alpha"] * gate * b
    err_r = rel * (d["alpha"] * gate * babs).abs() + U * r.abs() + U * d["residual"].double().abs()
    rstd = 1.0 / torch.sqrt(r.square().mean(1, keepdim=True) + EPS)
    g = d["gamma_pre"].double()
    n = r * rstd * g
    shift = (r.abs() * err_r).mean(1, keepdim=True) * rstd ** 2
    err_n = rstd * g.abs() * err_r + (64 * U + shift) * n.abs()
    assert H == n.shape[1]
    return r, err_r, n, err_n


SHAPES = [(1, 7168), (3, 1), (5, 7), (33, 1001), (17, 256), (4, 8192), (3, 8200), (2, 16384), (2, 16383), (130, 2056)]


@pytest.mark.parametrize("T, H", SHAPES)
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_fp32_against_float64(T, H, gate):
    for post in (True, False):
        d = _inputs(T, H, gate, post, seed=T + H)
        got_r, got_h = _call(d)
        r, err_r, n, err_n = _reference(d)
        assert ((got_r.double() - r).abs() <= err_r).all()
        assert ((got_h.double() - n).abs() <= err_n).all()


@pytest.mark.parametrize("T, H, K", [(1, 256, 1), (9, 7168, 8), (40, 512, 3), (5, 768, 64), (3, 16384, 9)])
def test_reduce_fp32_against_float64(T, H, K):
    for post in (True, False):
        d = _inputs(T, H, "channel", post, seed=K, K=K)
        got_r, got_h = _call(d)
        r, err_r, n, err_n = _reference(d)
        assert ((got_r.double() - r).abs() <= err_r).all()
        assert ((got_h.double() - n).abs() <= err_n).all()
        assert torch.equal(got_r[0], d["residual"][0])      # its slots are all masked
        w1 = dict(d, w=torch.ones_like(d["w"]))
        got = _mr().moe_reduce_norm(d["rows"], d["pos"], None, d["residual"], gamma_pre=d["gamma_pre"])
        want = _mr().moe_reduce_norm(d["rows"], d["pos"], w1["w"], d["residual"], gamma_pre=d["gamma_pre"])
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_more_rows_than_a_grid_dimension_of_16_bits():
    d = _inputs(70001, 64, "token", seed=5)
    got_r, got_h = _call(d)
    r, err_r, n, err_n = _reference(d)
    assert ((got_r.double() - r).abs() <= err_r).all() and ((got_h.double() - n).abs() <= err_n).all()


def test_combine_of_rows_off_the_vector_boundary():
    """Bases off a 16-byte boundary: the same values as on it, one at a time."""
    d = _inputs(9, 512, "channel", seed=6, K=4)
    want = _call(d)
    off = dict(d)
    for k in ("rows", "residual"):
        buf = torch.empty(d[k].numel() + 1, device=DEV)
        off[k] = buf[1:].view(d[k].shape)
        off[k].copy_(d[k])
    got = _call(off)
    r, err_r, n, err_n = _reference(d)
    for g in (want, got):
        assert ((g[0].double() - r).abs() <= err_r).all() and ((g[1].double() - n).abs() <= err_n).all()


def _wide(d):
    """The same values in fp32."""
    return {k: v.float() if torch.is_tensor(v) and v.dtype.is_floating_point else v for k, v in d.items()}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("wide_residual", [False, True])
@pytest.mark.parametrize("T, H, K", [(7, 7168, 0), (6, 1001, 0), (3, 16384, 0), (11, 2048, 8), (1, 256, 2)])
def test_16_bit_is_the_fp32_path_rounded_once(dtype, wide_residual, T, H, K):
    for gate in ("none", "full", "token"):
        d = _inputs(T, H, gate, True, seed=H, dtype=dtype, K=K)
        if wide_residual:
            d["residual"] = d["residual"].float() * 1.001
        got_r, got_h = _call(d)
        want_r, want_h = _call(_wide(d))
        assert got_r.dtype == d["residual"].dtype and got_h.dtype == dtype
        assert torch.equal(got_r, want_r.to(got_r.dtype))
        assert torch.equal(got_h, want_h.to(dtype))


def _quantised(quant, h):
    """The library's own quantiser on h fp32."""
    mr = _mr()
    return {"fp8": lambda: mr.quantize_fp8_act_rows(h), "int8": lambda: mr.quantize_int8_rows(h),
            "mxfp8": lambda: mr.quantize_mx_rows(h, mr.MX_FP8),
            "mxfp4": lambda: mr.quantize_mx_rows(h, mr.MX_FP4)}[quant]()


@pytest.mark.parametrize("quant", ["fp8", "int8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("T, H, K", [(1, 7168, 0), (9, 2048, 0), (5, 16384, 0), (6, 1001, 0), (3, 96, 0), (8, 512, 4)])
def test_codes_are_the_quantisers_of_the_unrounded_h(quant, T, H, K):
    if quant.startswith("mx") and H % 32:
        pytest.skip("MX blocks of 32 do not fit")
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        d = _inputs(T, H, "none", True, seed=3, dtype=dtype, K=K)
        if K == 0:
            d["y"][-1] = 0.0
            d["residual"][-1] = 0.0                      # an all-zero row: scale 1 (E8M0 127), codes 0
        d["gamma_pre"][: H // 2] *= 2.0 ** -12           # blocks and codes near zero
        out_r, h, codes, scales = _call(d, quant=quant)
        _, wide_h = _call(_wide(d))
        want_codes, want_scales = _quantised(quant, wide_h)
        assert torch.equal(scales, want_scales)
        assert torch.equal(codes, want_codes)
        assert torch.equal(h, wide_h.to(dtype))
        plain_r, plain_h = _call(d)
        assert torch.equal(out_r, plain_r) and torch.equal(h, plain_h)


def test_first_norm_and_last_residual():
    mr = _mr()
    d = _inputs(13, 2048, "none", True, seed=1, dtype=torch.bfloat16)
    none, h = mr.moe_block_norm(None, d["residual"], gamma_pre=d["gamma_pre"])
    assert none is None
    zero_r, want = mr.moe_block_norm(torch.zeros_like(d["y"]), d["residual"], gamma_pre=d["gamma_pre"])
    assert torch.equal(zero_r, d["residual"]) and torch.equal(h, want)
    r, none = mr.moe_block_norm(d["y"], d["residual"], gamma_post=d["gamma_post"])
    assert none is None
    assert torch.equal(r, mr.moe_block_norm(d["y"], d["residual"], gamma_post=d["gamma_post"],
                                            gamma_pre=d["gamma_pre"])[0])
    # an fp32 residual stream in front of 16-bit activations
    none, h16 = mr.moe_block_norm(None, d["residual"].float(), gamma_pre=d["gamma_pre"], dtype=torch.bfloat16)
    assert torch.equal(h16, h)


def test_in_place_and_unaligned():
    mr = _mr()
    d = _inputs(21, 512, "full", True, seed=2, dtype=torch.float16)
    want = _call(d)
    y, res = d["y"].clone(), d["residual"].clone()
    got = _call(dict(d, y=y, residual=res), residual_out=res, h=y)
    assert got[0] is res and got[1] is y
    assert torch.equal(res, want[0]) and torch.equal(y, want[1])

    def shifted(t):                                        # the same values one element further on
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)
        flat[1:] = t.reshape(-1)
        return flat[1:].view(t.shape)

    e = dict(d, y=shifted(d["y"]), residual=shifted(d["residual"]))
    r, err_r, n, err_n = _reference(_wide(d))
    got_r, got_h = _call(e)
    step = torch.finfo(torch.float16).eps / 2
    assert ((got_r.double() - r).abs() <= err_r * 2 + step * r.abs() + 2.0 ** -25).all()
    assert ((got_h.double() - n).abs() <= err_n * 2 + step * n.abs() + 2.0 ** -25).all()
    with pytest.raises(mr.MoeError):
        _call(e, quant="mxfp8")


def test_rows_past_the_batch_stay():
    d = _inputs(5, 1024, seed=4, dtype=torch.bfloat16)
    big_r = torch.full((9, 1024), 7.0, dtype=torch.bfloat16, device=DEV)
    big_h, big_c = big_r.clone(), torch.full((9, 1024), 9, dtype=torch.uint8, device=DEV)
    sc = torch.full((9,), 5.0, device=DEV)
    _call(d, residual_out=big_r[2:7], h=big_h[2:7], quant="fp8", codes=big_c[2:7], scales=sc[2:7])
    for t, v in ((big_r, 7.0), (big_h, 7.0), (big_c, 9), (sc, 5.0)):
        assert (t[:2] == v).all() and (t[7:] == v).all()


def test_no_tokens():
    mr = _mr()
    r = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    g = torch.ones(256, device=DEV)
    out, h, c, s = mr.moe_block_norm(r, r, gamma_pre=g, quant="fp8")
    assert out.shape == h.shape == c.shape == (0, 256) and s.shape == (0,)


def test_other_stream_and_graph_replays():
    mr = _mr()
    d = _inputs(64, 2048, "channel", True, seed=6, dtype=torch.bfloat16, K=4)
    want = _call(d, quant="fp8")
    side = torch.cuda.Stream()
    out = [torch.empty_like(t) for t in want]
    kw = dict(residual_out=out[0], h=out[1], codes=out[2], scales=out[3], quant="fp8")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _call(d, **kw)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    args = dict(gamma_post=d["gamma_post"], gamma_pre=d["gamma_pre"], gate=d["gate"], alpha=d["alpha"], eps=EPS)
    with torch.cuda.graph(graph):
        mr.moe_reduce_norm(d["rows"], d["pos"], d["w"], d["residual"], **args, **kw)
    for i in range(4):
        d["residual"].copy_(_inputs(64, 2048, "channel", True, seed=10 + i, dtype=torch.bfloat16, K=4)["residual"])
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        want = mr.moe_reduce_norm(d["rows"], d["pos"], d["w"], d["residual"], **args, quant="fp8")
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals_of_the_binding():
    mr = _mr()
    d = _inputs(4, 256, dtype=torch.bfloat16)
    for bad in (dict(y=d["y"][:, ::2]), dict(y=d["y"].float()), dict(gamma_pre=d["gamma_pre"].half()),
                dict(gamma_pre=d["gamma_pre"][:100]), dict(gate=torch.ones(4, device=DEV)),
                dict(gate=torch.ones(4, 256, device=DEV)), dict(quant="fp4"), dict(eps=0.0),
                dict(gamma_pre=None, quant="fp8"), dict(residual=d["residual"].half()), dict(y=d["y"][:3])):
        kw = dict(y=d["y"], residual=d["residual"], gamma_pre=d["gamma_pre"])
        kw.update(bad)
        with pytest.raises(mr.MoeError):
            mr.moe_block_norm(**kw)
