"""GPU: the block-scaled products and the residual norms together, as decoder
blocks use them: a gated MLP between two residual norms forward, an MLP with its
backward pass (both gradients of every product), eager, on two streams, in HIP
graphs and as custom ops."""

import pytest
import torch

import block_norm_ref as ref
import mlp_fp8_quant_amd as fp8
import mlp_fp8_quant_amd.torch_ops  # noqa: F401

from gpu_util import device
from norm_linear_ref import SILU, act_slope

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
ops = torch.ops.fp8mot


def tensors(M, H, I, seed, gates=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = device()
    t = dict(x=r(M, H).to(BF16), dy=r(M, H).to(BF16), dr=r(M, H).to(BF16), n1=1 + 0.1 * r(H), n2=1 + 0.1 * r(H),
             post=1 + 0.1 * r(H), gate=0.5 + 0.2 * r(gates, H), b1=(0.1 * r(I)).to(BF16))
    t = {k: v.to(d) for k, v in t.items()}
    for name, n, k in (("g", I, H), ("u", I, H), ("d", H, I)):
        w = (0.05 * r(n, k)).to(BF16).to(d)
        t["q" + name], t["s" + name] = fp8.fp8_quant_block(w, tile=True)
        t["q" + name + "t"], t["s" + name + "t"] = fp8.fp8_quant_block(w, tile=True, transpose=True)
    return t


def serve(t):
    """norm -> codes -> gate and up -> SwiGLU codes -> down -> post-norm, gate, residual, norm -> codes"""
    (q, s), _ = fp8.fp8_residual_norm(t["x"], t["n1"], out_kind=fp8.OUT_FP8_BLOCK)
    g = fp8.fp8_linear_block(q, t["qg"], s, t["sg"])
    u = fp8.fp8_linear_block(q, t["qu"], s, t["su"])
    qh, sh = fp8.silu_mul_2in_block(g, u)
    h = fp8.fp8_linear_block(qh, t["qd"], sh, t["sd"])
    (q2, s2), r = fp8.fp8_residual_norm(t["x"], t["n2"], h, gate=t["gate"], post_weight=t["post"],
                                        out_kind=fp8.OUT_FP8_BLOCK)
    return dict(q=q, s=s, g=g, u=u, qh=qh, sh=sh, h=h, q2=q2, s2=s2, r=r)


def forward(t):
    n, _, rstd, _ = fp8.fp8_residual_norm(t["x"], t["n1"], stats=True)
    q, s = fp8.fp8_quant_block(n)
    u, pre = fp8.fp8_linear_block(q, t["qu"], s, t["su"], bias=t["b1"], act=SILU, pre=True)
    qu, su = fp8.fp8_quant_block(u)
    h = fp8.fp8_linear_block(qu, t["qd"], su, t["sd"])
    y, r, rstd2, post_rstd = fp8.fp8_residual_norm(t["x"], t["n2"], h, gate=t["gate"], post_weight=t["post"], alpha=0.5,
                                                   stats=True)
    return dict(n=n, rstd=rstd, u=u, pre=pre, h=h, y=y, r=r, rstd2=rstd2, post_rstd=post_rstd)


def weight_gradient(dy, x):
    """dy^T x of operands quantized along the rows that are summed over."""
    qd, sd = fp8.fp8_quant_block(dy, transpose=True)
    qx, sx = fp8.fp8_quant_block(x, transpose=True)
    return fp8.fp8_linear_block(qd, qx, sd, sx, out_kind=fp8.OUT_F32)


def through(dy, qt, st):
    q, s = fp8.fp8_quant_block(dy)
    return fp8.fp8_linear_block(q, qt, s, st)


def backward(t, f):
    dx, dh, dn2, dgate, dpost = fp8.fp8_residual_norm_backward(
        t["dy"], f["r"], t["n2"], f["rstd2"], f["h"], gate=t["gate"], post_weight=t["post"], post_rstd=f["post_rstd"],
        alpha=0.5, dr=t["dr"])
    dwd = weight_gradient(dh, f["u"])
    dz, db1 = fp8.fp8_linear_act_backward(through(dh, t["qdt"], t["sdt"]), f["pre"], SILU)
    dwu = weight_gradient(dz, f["n"])
    dn = through(dz, t["qut"], t["sut"])
    dx, _, dn1, _, _ = fp8.fp8_residual_norm_backward(dn, t["x"], t["n1"], f["rstd"], dr=dx)
    return dict(dx=dx, dn1=dn1, dwu=dwu, db1=db1, dwd=dwd, dn2=dn2, dgate=dgate, dpost=dpost, dh=dh, dz=dz, dn=dn)


def results(t):
    f = forward(t)
    return [*serve(t).values(), *f.values(), *backward(t, f).values()]


def equal(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("M,H,I", [(1, 256, 520), (5, 260, 512), (130, 384, 640), (300, 1000, 1030)])
def test_gated_block(M, H, I):
    # each step against the 64-bit formula on what it was given
    t = tensors(M, H, I, M)
    f = serve(t)
    y, *_, err, _ = ref.norm(t["x"], t["n1"], None, None, None, 1.0, 1e-6)
    ref.check_codes(f["q"], f["s"], y, err, "norm")
    for name, w in (("g", "g"), ("u", "u")):
        y, _, err, _ = ref.linear(f["q"], t["q" + w], f["s"], t["s" + w], False)
        ref.check(f[name], y, err, name)
    v, err = ref.silu_mul(f["g"], f["u"])
    ref.check_codes(f["qh"], f["sh"], v, err, "silu")
    y, _, err, _ = ref.linear(f["qh"], t["qd"], f["sh"], t["sd"], False)
    ref.check(f["h"], y, err, "down")
    y, r, _, _, err, err_r = ref.norm(t["x"], t["n2"], f["h"], t["gate"], t["post"], 1.0, 1e-6)
    ref.check(f["r"], r, err_r, "stream")
    ref.check_codes(f["q2"], f["s2"], y, err, "next norm")


@pytest.mark.parametrize("M", [2, 33, 300])
def test_backward_steps(M):
    t = tensors(M, 256, 520, M, gates=1 if M == 33 else 2)
    f = forward(t)
    b = backward(t, f)
    want = ref.norm_backward(t["dy"], f["r"], t["n2"], f["rstd2"], f["h"], t["gate"], t["post"], f["post_rstd"], 0.5,
                             t["dr"])
    for got, name in (("dh", "dhidden"), ("dn2", "dweight"), ("dgate", "dgate"), ("dpost", "dpost_weight")):
        ref.check(b[got], *want[name], name)
    for got, dy, x in (("dwd", b["dh"], f["u"]), ("dwu", b["dz"], f["n"])):
        (qd, sd), (qx, sx) = (fp8.fp8_quant_block(v, transpose=True) for v in (dy, x))
        y, _, err, _ = ref.linear(qd, qx, sd, sx, True)
        assert b[got].dtype == F32
        ref.check(b[got], y, err, got)
    q, s = fp8.fp8_quant_block(b["dz"])
    y, _, err, _ = ref.linear(q, t["qut"], s, t["sut"], False)
    ref.check(b["dn"], y, err, "dn")


@pytest.mark.parametrize("M", [32, 130])
def test_gradients_point_where_the_loss_grows(M):
    # the chain's gradients against autograd through the formulas in 64 bits with
    # unquantized activations and gradients.  A gradient here has passed at most
    # six roundings to E4M3 (activations and gradients), each at most 2^-4 of a
    # value and mostly below 2^-5: the cosine is 1 - O(6 * 2^-10)
    t = tensors(M, 256, 520, 60 + M, gates=2)
    b = backward(t, forward(t))
    leaf = {k: t[k].cpu().double().requires_grad_(True) for k in ("x", "n1", "n2", "post", "gate", "b1")}
    for w, rows, cols in (("u", 520, 256), ("d", 256, 520)):
        v = ref.decode(t["q" + w])[:, :cols] * ref.spread(t["s" + w].cpu().double(), True, rows, cols)
        leaf["w" + w] = v.requires_grad_(True)
    rms = lambda v: v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt()  # noqa: E731
    z = (rms(leaf["x"]) * leaf["n1"]) @ leaf["wu"].t() + leaf["b1"]
    h = (z * torch.sigmoid(z)) @ leaf["wd"].t()
    r = leaf["x"] + 0.5 * leaf["gate"].repeat_interleave(M // 2, 0) * rms(h) * leaf["post"]
    ((rms(r) * leaf["n2"] * t["dy"].cpu().double()).sum() + (r * t["dr"].cpu().double()).sum()).backward()
    for got, of in (("dx", "x"), ("dn1", "n1"), ("dwu", "wu"), ("db1", "b1"), ("dwd", "wd"), ("dn2", "n2"),
                    ("dgate", "gate"), ("dpost", "post")):
        p, q = b[got].cpu().double().reshape(-1), leaf[of].grad.reshape(-1)
        cos = (p @ q / (p.norm() * q.norm())).item()
        assert cos > 1 - 6 * 2.0 ** -10, (got, cos)


def test_slope_of_the_chain():
    # (the activation's slope that the chain above goes through)
    z = torch.linspace(-4, 4, 33, dtype=torch.float64)
    assert torch.allclose(act_slope(z, SILU), torch.autograd.functional.jvp(torch.nn.functional.silu, z,
                                                                             torch.ones_like(z))[1])


def test_two_streams_at_once():
    ta, tb = tensors(150, 256, 520, 1), tensors(70, 520, 256, 2)
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
    ts = [tensors(M, 256, 520, 5), tensors(M, 256, 520, 6)]
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
    ts[0]["x"].mul_(0.5)
    graphs[0].replay()
    fresh = results(ts[0])
    torch.cuda.synchronize()
    assert equal(outs[0], fresh) and not torch.equal(outs[0][9], want[0][9])


@pytest.mark.parametrize("M,N,K", [(16, 640, 512), (100, 1000, 528), (300, 4001, 272), (600, 2053, 400), (1100, 5003, 272),
                                   (1024, 3000, 2064), (510, 16380, 2064)])
@pytest.mark.parametrize("w_rows", [False, True])
def test_captured_products(M, N, K, w_rows):
    d, g = device(), torch.Generator().manual_seed(M)
    q = lambda r: torch.randint(0, 0x60, (r, K), generator=g, dtype=torch.uint8).to(d)  # noqa: E731
    sc = lambda r: (0.01 + torch.rand(r, (K + 127) // 128, generator=g)).to(d)  # noqa: E731
    args = (q(M), q(N), sc(M), sc(N if w_rows else (N + 127) // 128))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = fp8.fp8_linear_block(*args)
    want = fp8.fp8_linear_block(*args)
    for _ in range(3):
        out.fill_(7.0)
        graph.replay()
        again = fp8.fp8_linear_block(*args)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(again, want)


def test_given_workspace():
    t = tensors(400, 264, 256, 3, gates=4)
    f = forward(t)
    h = torch.randn(400, 264, device=device()).to(BF16)
    args = (t["dy"], f["r"], t["n2"], f["rstd2"], h)
    k = dict(gate=t["gate"], post_weight=t["post"], post_rstd=f["post_rstd"])
    want = fp8.fp8_residual_norm_backward(*args, **k)
    nb = fp8.fp8_residual_norm_backward_workspace(400, 264, 4)
    assert nb > 0
    ws = torch.full((nb + 64,), 255, dtype=torch.uint8, device=device())
    assert equal(fp8.fp8_residual_norm_backward(*args, **k, workspace=ws[:nb]), want) and (ws[nb:] == 255).all()
    with pytest.raises(fp8.Fp8motError, match="WORKSPACE"):
        fp8.fp8_residual_norm_backward(*args, **k, workspace=ws[:nb - 16].clone())


def test_custom_ops():
    t = tensors(40, 256, 520, 7)
    f = forward(t)
    q, s = ops.quant_block(f["n"])
    assert equal((q, s), fp8.fp8_quant_block(f["n"]))
    assert equal(ops.silu_mul_block(f["u"], f["u"]), fp8.silu_mul_2in_block(f["u"], f["u"]))
    u = ops.linear_block(q, t["qu"], s, t["su"], t["b1"], SILU)
    assert torch.equal(u, f["u"])
    y, r, rstd, post = ops.residual_norm(t["x"], f["h"], t["n2"], t["gate"], t["post"], 0.5)
    assert equal((y, r, rstd, post), (f["y"], f["r"], f["rstd2"], f["post_rstd"]))
    args = (t["dy"], r, t["n2"], rstd, f["h"], t["gate"], t["post"], post, 0.5, t["dr"])
    g = ops.residual_norm_backward(*args)
    assert equal(g[1:], [backward(t, f)[k] for k in ("dh", "dn2", "dgate", "dpost")])
    for op, a in [(ops.quant_block, (f["n"],)), (ops.quant_block, (f["n"], True, True)),
                  (ops.silu_mul_block, (f["u"], f["u"])), (ops.linear_block, (q, t["qu"], s, t["su"], t["b1"], SILU)),
                  (ops.residual_norm, (t["x"], f["h"], t["n2"])),
                  (ops.residual_norm, (t["x"], f["h"], t["n2"], t["gate"], t["post"])),
                  (ops.residual_norm_block, (t["x"], f["h"], t["n2"], t["gate"], t["post"])),
                  (ops.residual_norm_backward, args)]:
        torch.library.opcheck(op, a, test_utils=("test_schema", "test_faketensor", "test_aot_dispatch_dynamic"))

    def chain(x):
        q, s, r = ops.residual_norm_block(x, f["h"], t["n2"], t["gate"], t["post"])
        u = ops.linear_block(q, t["qu"], s, t["su"], t["b1"], SILU)
        qu, su = ops.quant_block(u)
        return ops.linear_block(qu, t["qd"], su, t["sd"], None, 0, r)

    assert torch.equal(torch.compile(chain, fullgraph=True, backend="aot_eager")(t["x"]), chain(t["x"]))


def test_native_front_and_python_checks_give_the_same(monkeypatch):
    from mlp_fp8_quant_amd import api

    ts = [tensors(3, 256, 520, 8), tensors(150, 260, 512, 9, gates=3)]
    assert api._load_native() is api._native
    native = [results(t) for t in ts]
    monkeypatch.setattr(api, "_native", api._PythonOnly)
    assert all(equal(results(t), want) for t, want in zip(ts, native))


def test_errors_through_the_native_front():
    t = tensors(4, 256, 512, 10)
    x = t["x"]
    with pytest.raises(fp8.Fp8motError, match="ERR_INVALID_ARG"):
        fp8.fp8_residual_norm(x, t["n1"], eps=-1.0)
    with pytest.raises(fp8.Fp8motError, match="ERR_UNSUPPORTED"):
        fp8.fp8_residual_norm(x, t["n1"], out_kind=fp8.OUT_FP8)
    with pytest.raises(fp8.Fp8motError, match="ERR_UNSUPPORTED"):
        fp8.fp8_linear_block(t["qg"], t["qu"], t["sg"].repeat_interleave(128, 0), t["su"], out_kind=fp8.OUT_FP8)
    with pytest.raises(ValueError, match="divide"):
        fp8.fp8_residual_norm(x, t["n1"], x, gate=torch.zeros(3, 256, device=x.device))
    with pytest.raises(ValueError, match="contiguous"):
        fp8.fp8_quant_block(x.t())
    with pytest.raises(ValueError, match="out_kind"):
        fp8.fp8_linear_block(t["qg"], t["qu"], t["sg"].repeat_interleave(128, 0), t["su"], out_kind=fp8.OUT_FP8_BLOCK)
    odd = torch.empty(4 * 256 + 8, dtype=BF16, device=x.device)[1:1 + 4 * 256].view(4, 256)
    for call in (lambda: fp8.fp8_quant_block(odd), lambda: fp8.silu_mul_2in_block(odd, x),
                 lambda: fp8.fp8_residual_norm(odd, t["n1"])):
        with pytest.raises(fp8.Fp8motError, match="ERR_MISALIGNED"):
            call()
    p = torch.nn.Parameter
    y, r = fp8.fp8_residual_norm(x, p(t["n1"]), x, gate=p(t["gate"]), post_weight=p(t["post"]))
    assert not y.requires_grad and equal((y, r), fp8.fp8_residual_norm(x, t["n1"], x, gate=t["gate"],
                                                                       post_weight=t["post"]))
