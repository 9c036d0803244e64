"""GPU: the layer norm and the Linear epilogue together, as a decoder layer
uses them: a pre-norm block forward (norm -> FP8 codes -> Linear + bias +
activation -> FP8 codes -> Linear + bias + residual) and backward, eager, on
two streams, in HIP graphs and as custom ops."""

import pytest
import torch

import mlp_fp8_quant_amd as fp8
import mlp_fp8_quant_amd.torch_ops  # noqa: F401
import norm_linear_ref as ref

from gpu_util import device

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ops = torch.ops.fp8mot


def block(M, H, I, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = device()
    w1, s1 = fp8.rtn_weight((0.02 * r(I, H)).to(BF16).to(d))
    w2, s2 = fp8.rtn_weight((0.02 * r(H, I)).to(BF16).to(d))
    f = lambda t, dt: t.to(dt).to(d)  # noqa: E731
    return dict(x=f(r(M, H), BF16), g=f(1 + 0.1 * r(H), F32), b=f(0.1 * r(H), F32), w1=w1, s1=s1,
                b1=f(0.1 * r(I), BF16), w2=w2, s2=s2, b2=f(0.1 * r(H), BF16), sn=f(torch.tensor([0.012]), F32),
                sh=f(torch.tensor([0.012]), F32), dy=f(r(M, H), BF16))


def forward(t, act=ref.GELU):
    q, mean, rstd = fp8.fp8_layer_norm(t["x"], t["g"], t["b"], out_kind=fp8.OUT_FP8, sy=t["sn"], stats=True)
    h, pre = fp8.fp8_linear_act(q, t["w1"], t["sn"], t["s1"], bias=t["b1"], act=act, out_kind=fp8.OUT_FP8,
                                sy=t["sh"], pre=True)
    y = fp8.fp8_linear_act(h, t["w2"], t["sh"], t["s2"], bias=t["b2"], residual=t["x"])
    return dict(q=q, mean=mean, rstd=rstd, h=h, pre=pre, y=y)


def through_weight(dz, w, s):
    """The gradient through a frozen weight: FP8 per row against the
    transposed codes."""
    q, sq = fp8.fp8_quant_per_row(dz)
    wt = w.t().contiguous()
    return fp8.fp8_linear_rowwise(q, wt, sq, s.expand(wt.shape[0]).contiguous())


def backward(t, f, act=ref.GELU):
    dz2, db2 = fp8.fp8_linear_act_backward(t["dy"], None)
    dh = through_weight(dz2, t["w2"], t["s2"])
    dz1, db1 = fp8.fp8_linear_act_backward(dh, f["pre"], act)
    dn = through_weight(dz1, t["w1"], t["s1"])
    dx, dg, db = fp8.fp8_layer_norm_backward(dn, t["x"], t["g"], f["mean"], f["rstd"], dres=t["dy"])
    return dict(dh=dh, dz1=dz1, dn=dn, dx=dx, dg=dg, db=db, db1=db1, db2=db2)


@pytest.mark.parametrize("M", [1, 5, 70, 300])
@pytest.mark.parametrize("act", [ref.GELU, ref.SILU])
def test_block_forward_and_backward(M, act):
    # each step against the 64-bit formula on what it was given
    t = block(M, 256, 512, M)
    f = forward(t, act)
    y64, m64, r64, err = ref.norm(t["x"], t["g"], t["b"], 1e-5)
    ref.check_fp8(f["q"], y64, err, t["sn"])
    h64, z64, err, err_z = ref.linear_act(f["q"], t["w1"], t["sn"], t["s1"], t["b1"], act, None)
    ref.check_fp8(f["h"], h64, err, t["sh"])
    ref.check(f["pre"], z64, err_z)
    y64, _, err, _ = ref.linear_act(f["h"], t["w2"], t["sh"], t["s2"], t["b2"], ref.NONE, t["x"])
    ref.check(f["y"], y64, err)
    b = backward(t, f, act)
    dy = t["dy"].cpu().double()
    ref.check(b["db2"], dy.sum(0), (M + 20) * ref.U * dy.abs().sum(0))
    dz = b["dh"].cpu().double() * ref.act_slope(f["pre"].cpu().double(), act)
    e = b["dh"].cpu().double().abs() * ref.act_slope_error(f["pre"].cpu().double(), act) + dz.abs() * ref.U
    ref.check(b["dz1"], dz, e)
    ref.check(b["db1"], dz.sum(0), e.sum(0) + (M + 20) * ref.U * dz.abs().sum(0))
    dx, dw, db, ex, ew, eb = ref.norm_backward(b["dn"], t["x"], t["g"], f["mean"], f["rstd"], t["dy"])
    ref.check(b["dx"], dx, ex)
    ref.check(b["dg"], dw, ew)
    ref.check(b["db"], db, eb)


@pytest.mark.parametrize("M", [2, 130])
def test_block_gradients_point_where_the_loss_grows(M):
    # the chain's gradients against the chain of the formulas in 64 bits with
    # unquantized activations.  The chain rounds to E4M3 four times (two
    # activations, two gradients), each at most 2^-4 of a value and mostly
    # below 2^-5, so the cosine of the two gradients is 1 - O(4 * 2^-10)
    t = block(M, 256, 512, 40 + M)
    b = backward(t, forward(t))
    x, gw, gb, b1, b2, dy = (t[k].cpu().double().requires_grad_(k != "dy") for k in ("x", "g", "b", "b1", "b2", "dy"))
    w1, w2 = (ref.decode(t[w]) * t[s].cpu().double() for w, s in (("w1", "s1"), ("w2", "s2")))
    mean = x.mean(-1, keepdim=True)
    xh = (x - mean) / torch.sqrt((x - mean).square().mean(-1, keepdim=True) + 1e-5)
    z = (xh * gw + gb) @ w1.t() + b1
    y = (z * ref.phi(z)) @ w2.t() + b2 + x
    (y * dy).sum().backward()
    for name, leaf in (("dx", x), ("dg", gw), ("db", gb), ("db1", b1), ("db2", b2)):
        p, q = b[name].cpu().double().reshape(-1), leaf.grad.reshape(-1)
        cos = (p @ q / (p.norm() * q.norm())).item()
        assert cos > 1 - 4 * 2.0 ** -10, (name, cos)


def results(t):
    f = forward(t)
    return [*f.values(), *backward(t, f).values()]


def equal(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def test_two_streams_at_once():
    ta, tb = block(150, 256, 512, 1), block(70, 512, 256, 2)
    wa, wb = results(ta), results(tb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(sa):
            a = results(ta)
        with torch.cuda.stream(sb):
            b = results(tb)
        torch.cuda.synchronize()
        assert equal(a, wa) and equal(b, wb)


@pytest.mark.parametrize("M", [1, 140])
def test_captured_graphs_replay_the_eager_results(M):
    # two graphs of the block, replayed in turn with eager work between
    ts = [block(M, 256, 512, 5), block(M, 256, 512, 6)]
    want = [results(t) for t in ts]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for t in ts:
            results(t)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in ts:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(results(t))
        graphs.append(g)
    for r in range(4):
        for k in (0, 1):
            graphs[k].replay()
        noise = results(ts[r % 2])
        torch.cuda.synchronize()
        assert equal(noise, want[r % 2])
        assert equal(outs[0], want[0]) and equal(outs[1], want[1]), f"replay {r}"
    # new values in the captured input are followed
    ts[0]["x"].mul_(0.5)
    graphs[0].replay()
    fresh = results(ts[0])
    torch.cuda.synchronize()
    assert equal(outs[0], fresh) and not torch.equal(outs[0][5], want[0][5])


@pytest.mark.parametrize("M,N,K", [(16, 640, 512), (100, 1000, 528), (300, 4001, 272), (777, 2053, 272), (3000, 700, 4000),
                                   (2500, 2500, 272), (5000, 3000, 256)])
def test_captured_products(M, N, K):
    # every family of the products, with the launch that joins splits of K; one
    # graph twice in the replays, eager calls of the same shape between them
    d, g = device(), torch.Generator().manual_seed(M)
    q = lambda r: torch.randint(0, 0x60, (r, K), generator=g, dtype=torch.uint8).to(d)  # noqa: E731
    qx, qw, s = q(M), q(N), torch.tensor([0.01], device=d)
    res, dy = (torch.randn(M, N, generator=g).to(BF16).to(d) for _ in range(2))

    def run():
        y, pre = fp8.fp8_linear_act(qx, qw, s, s, act=ref.SILU, residual=res, pre=True)
        return [y, pre, *fp8.fp8_linear_act_backward(dy, pre, ref.SILU)]

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = run()
    want = run()
    for _ in range(3):
        for t in out:
            t.fill_(7.0)
        graph.replay()
        again = run()
        torch.cuda.synchronize()
        assert equal(out, want) and equal(again, want)


def test_given_workspaces():
    d = device()
    for M, N, K in ((1, 64, 16384), (3000, 700, 4096), (5, 512, 512)):
        g = torch.Generator().manual_seed(M)
        q = lambda r: torch.randint(0, 0x60, (r, K), generator=g, dtype=torch.uint8).to(d)  # noqa: E731
        qx, qw, s = q(M), q(N), torch.tensor([0.01], device=d)
        want = fp8.fp8_linear_act(qx, qw, s, s)
        ws = torch.full((max(16, fp8.fp8_linear_act_workspace(M, N, K)),), 255, dtype=torch.uint8, device=d)
        assert torch.equal(fp8.fp8_linear_act(qx, qw, s, s, workspace=ws), want)
    x = torch.randn(200, 96, device=d)
    _, mean, rstd = fp8.fp8_layer_norm(x, stats=True)
    want = fp8.fp8_layer_norm_backward(x, x, None, mean, rstd)
    nb = fp8.fp8_layer_norm_backward_workspace(200, 96)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=d)
    assert equal(fp8.fp8_layer_norm_backward(x, x, None, mean, rstd, workspace=ws), want)
    with pytest.raises(fp8.Fp8motError):
        fp8.fp8_layer_norm_backward(x, x, None, mean, rstd, workspace=ws[:nb - 16].clone())
    y = x.to(BF16)
    want = fp8.fp8_linear_act_backward(y, y, ref.SILU)
    nb = fp8.fp8_linear_act_backward_workspace(200, 96)
    ws = torch.full((nb,), 255, dtype=torch.uint8, device=d)
    assert equal(fp8.fp8_linear_act_backward(y, y, ref.SILU, workspace=ws), want)


def test_custom_ops():
    t = block(40, 256, 512, 7)
    f = forward(t)
    q, mean, rstd = ops.layer_norm(t["x"], t["g"], t["b"], 1e-5, fp8.OUT_FP8, t["sn"])
    h, pre = ops.linear_act_train(q, t["w1"], t["sn"], t["s1"], t["b1"], ref.GELU, None, fp8.OUT_FP8, t["sh"])
    y = ops.linear_act(h, t["w2"], t["sh"], t["s2"], t["b2"], 0, t["x"])
    assert equal([q, mean, rstd, h, pre, y], f.values())
    dz, db = ops.linear_act_backward(t["dy"], None)
    dx, dw, db = ops.layer_norm_backward(t["dy"], t["x"], t["g"], mean, rstd, t["dy"])
    assert equal([dx, dw, db], fp8.fp8_layer_norm_backward(t["dy"], t["x"], t["g"], mean, rstd, t["dy"]))
    for op, args in [(ops.layer_norm, (t["x"], t["g"], t["b"])),
                     (ops.linear_act, (q, t["w1"], t["sn"], t["s1"], t["b1"], ref.SILU)),
                     (ops.linear_act_train, (q, t["w1"], t["sn"], t["s1"], t["b1"], ref.SILU)),
                     (ops.linear_act_backward, (pre, pre, ref.SILU)),
                     (ops.layer_norm_backward, (t["dy"], t["x"], t["g"], mean, rstd))]:
        torch.library.opcheck(op, args, test_utils=("test_schema", "test_faketensor",
                                                    "test_aot_dispatch_dynamic"))

    def chain(x):
        q, mean, rstd = ops.layer_norm(x, t["g"], t["b"], 1e-5, fp8.OUT_FP8, t["sn"])
        h, _ = ops.linear_act_train(q, t["w1"], t["sn"], t["s1"], t["b1"], ref.GELU, None, fp8.OUT_FP8, t["sh"])
        return ops.linear_act(h, t["w2"], t["sh"], t["s2"], t["b2"], 0, x)

    assert torch.equal(torch.compile(chain, fullgraph=True, backend="aot_eager")(t["x"]), f["y"])


def test_native_front_and_python_checks_give_the_same(monkeypatch):
    # the native front of the binding against the path behind it
    from mlp_fp8_quant_amd import api

    class Nothing:
        linear_act = linear_act_backward = layer_norm = layer_norm_backward = staticmethod(lambda *a: None)

    ts = [block(3, 256, 512, 8), block(150, 256, 512, 9)]
    assert api._load_native() is api._native
    native = [results(t) for t in ts]
    monkeypatch.setattr(api, "_native", Nothing)
    assert all(equal(results(t), want) for t, want in zip(ts, native))


def test_errors_and_parameters_through_the_native_front():
    t = block(4, 256, 512, 10)
    x = t["x"]
    want = fp8.fp8_layer_norm(x, t["g"], t["b"])
    assert torch.equal(fp8.fp8_layer_norm(x, torch.nn.Parameter(t["g"]), torch.nn.Parameter(t["b"])), want)
    assert torch.equal(fp8.fp8_layer_norm(x.view(2, 2, 256), t["g"], t["b"]).view(4, 256), want)
    with pytest.raises(fp8.Fp8motError, match="ERR_INVALID_ARG"):
        fp8.fp8_layer_norm(x, eps=-1.0)
    with pytest.raises(fp8.Fp8motError, match="ERR_UNSUPPORTED"):
        fp8.fp8_layer_norm(x, out_kind=fp8.OUT_FP8)
    with pytest.raises(fp8.Fp8motError, match="ERR_INVALID_ARG"):
        fp8.fp8_linear_act_backward(x, x, act=9)
    with pytest.raises(ValueError, match="contiguous"):
        fp8.fp8_layer_norm(x.t())
    with pytest.raises(ValueError, match="bias"):
        fp8.fp8_linear_act(t["w1"], t["w1"], t["s1"], t["s1"], bias=t["b2"])
    odd = torch.empty(4 * 256 + 8, dtype=BF16, device=x.device)[1:1 + 4 * 256].view(4, 256)
    with pytest.raises(fp8.Fp8motError, match="ERR_MISALIGNED"):
        fp8.fp8_layer_norm(odd)
