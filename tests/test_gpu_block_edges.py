"""The block's operators where they can go wrong: what must not be seen, extreme activations, graphs, streams, long
tensors, and a block's forward and backward pass put together."""

import numpy as np
import pytest
import torch

from differential_attention_03_gb300 import binding as da
from oracle import block

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from differential_attention_03_gb300 import build
    build.build()
    torch.cuda.init()


def _rnd(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, std=1.0, dtype=BF):
        return (std * torch.randn(shape, generator=g, device="cuda")).to(dtype)
    return rnd


# ----------------------------------------------------------------------------- what must not be seen
@pytest.mark.parametrize("M", [1, 5, 33, 100, 128, 130, 300, 700])
@pytest.mark.parametrize("K", [40, 72, 1000])
def test_poisoned_neighbours_are_not_seen(M, K):
    """Rows and columns around the operands hold NaN: contraction and row tails are zeros, not what lies there."""
    rnd = _rnd(M + K)
    N = 208
    wide = torch.full((M + 300, K + 64), NAN, device="cuda", dtype=BF)
    a = wide[:M, 32:32 + K]  # 64 bytes in
    a.copy_(rnd(M, K))
    pool = torch.full((N + 300, K), NAN, device="cuda", dtype=BF)
    w = pool[:N]
    w.copy_(rnd(N, K))
    clean = a.contiguous().clone(), w.clone()
    for dt in (BF, F32):
        got = da.linear(a, w, dtype=dt)
        assert torch.isfinite(got).all() and torch.equal(got, da.linear(*clean, dtype=dt))
    h = da.gated_linear(a, w)
    assert torch.isfinite(h).all() and torch.equal(h, da.gated_linear(*clean))
    wy = torch.full((M + 300, N + 64), NAN, device="cuda", dtype=BF)
    dy = wy[:M, 8:8 + N]
    dy.copy_(rnd(M, N))
    pre = rnd(M, N)
    for act in ("none", "gelu"):
        one = da.linear_backward(a, w, dy, pre=pre, act=act, bias=True)
        two = da.linear_backward(clean[0], clean[1], dy.contiguous(), pre=pre, act=act, bias=True)
        for k in one:
            assert torch.isfinite(one[k]).all() and torch.equal(one[k], two[k]), (act, k)
    da.device_status()


@pytest.mark.parametrize("M", [1, 100, 129, 300, 1000])
@pytest.mark.parametrize("N", [8, 72, 200, 456])
def test_what_lies_around_an_output_stays(M, N):
    """Outputs, stored z and gradients that end inside a tile, in the middle of a tensor of sevens: the values are those
    of the same call into tensors of its own (an fp32 output's sums go by segments, so its z is not a bf16 output's)."""
    rnd = _rnd(7 * M + N)
    K = 520  # (a short contraction, and one above 512 values)
    a, w, gu_w = rnd(M, K), rnd(N, K), rnd(2 * N, K)
    for dt in (BF, F32):
        wide = torch.full((M + 3, N + 128), 7.0, device="cuda", dtype=dt)
        pool = torch.full((M + 3, N), 7.0, device="cuda", dtype=BF)
        out = wide[1:M + 1, 64:64 + N]
        y, pre = da.linear_train(a, w, act="silu", out=out, pre=pool[:M], dtype=dt)
        alone = da.linear_train(a, w, act="silu", dtype=dt)
        assert torch.equal(out, alone[0]) and torch.equal(pre, alone[1])
        wide[1:M + 1, 64:64 + N] = 7
        assert (wide == 7).all() and (pool[M:] == 7).all()
    wide = torch.full((M + 3, N + 128), 7.0, device="cuda", dtype=BF)
    pool = torch.full((M + 3, 2 * N), 7.0, device="cuda", dtype=BF)
    out = wide[1:M + 1, 64:64 + N]
    h, gu = da.gated_linear_train(a, gu_w, out=out, gu=pool[:M])
    alone = da.gated_linear_train(a, gu_w)
    assert torch.equal(out, alone[0]) and torch.equal(gu, alone[1])
    wide[1:M + 1, 64:64 + N] = 7
    assert (wide == 7).all() and (pool[M:] == 7).all()
    dy = rnd(M, N)
    for dt in (BF, F32):
        flat = torch.full((N * K + 64,), 7.0, device="cuda", dtype=dt)
        rows = torch.full((M * K + 64,), 7.0, device="cuda", dtype=BF)
        out = {"dw": flat[:N * K].view(N, K), "da": rows[:M * K].view(M, K)}
        got = da.linear_backward(a, w, dy, out=out, dw_dtype=dt)
        want = da.linear_backward(a, w, dy, dw_dtype=dt)
        assert all(torch.equal(got[k], want[k]) for k in want)
        assert (flat[N * K:] == 7).all() and (rows[M * K:] == 7).all()
    da.device_status()


@pytest.mark.parametrize("M", [3, 60, 128, 300])
def test_a_rows_nan_stays_in_its_row(M):
    rnd = _rnd(M)
    a, w, res = rnd(M, 136), rnd(144, 136), rnd(M, 144)
    ref = da.linear(a, w, residual=res, act="silu")
    refh, refs = da.gated_linear(a, w), da.residual_norm(a, gamma_post=torch.ones(136, device="cuda"))
    refd = da.linear_backward(a, w, res, dw=False)["da"]
    a2, res2 = a.clone(), res.clone()
    a2[M // 2, 7] = NAN
    res2[0, 3] = float("inf")
    got = da.linear(a2, w, residual=res2, act="silu")
    rows = torch.arange(M, device="cuda") != M // 2
    bad = ~torch.isfinite(got)
    assert bad[M // 2].all() and int(bad.sum()) == 144 + (1 if M // 2 else 0) and (M // 2 == 0 or bool(bad[0, 3]))
    assert torch.equal(got[rows][bad[rows] == 0], ref[rows][bad[rows] == 0])
    h = da.gated_linear(a2, w)
    assert not torch.isfinite(h[M // 2]).any() and torch.equal(h[rows], refh[rows])
    y, s = da.residual_norm(a2, gamma_post=torch.ones(136, device="cuda"))
    assert torch.equal(y[rows], refs[0][rows]) and torch.equal(s[rows], refs[1][rows]) and not torch.isfinite(y[M // 2]).any()
    d2 = res.clone()
    d2[M // 2, 5] = NAN
    got = da.linear_backward(a, w, d2, dw=False)["da"]
    assert torch.equal(got[rows], refd[rows]) and not torch.isfinite(got[M // 2]).any()
    w2 = w.clone()
    w2[9, 0] = NAN  # an output feature
    got = da.linear(a, w2, residual=res, act="silu")
    cols = torch.arange(144, device="cuda") != 9
    assert torch.equal(got[:, cols], ref[:, cols]) and not torch.isfinite(got[:, 9]).any()
    da.device_status()


@pytest.mark.parametrize("D", [8, 72, 256, 264, 300, 301, 2048, 4099, 8192])
def test_norm_rows_do_not_see_each_other(D):
    """Backward: a row of infinities reaches its own gradients and the sums over rows, no other row."""
    rnd = _rnd(D)
    rows = 37
    x, s, dy, ds = rnd(rows, D), rnd(rows, D), rnd(rows, D), rnd(rows, D)
    gate = rnd(rows, D, dtype=F32)
    a = dict(gate=gate, gamma_post=rnd(D, dtype=F32), gamma=rnd(D, dtype=F32))
    ref = da.residual_norm_backward(x, s, dy, ds, **a)
    dy2 = dy.clone()
    dy2[11] = float("inf")
    got = da.residual_norm_backward(x, s, dy2, ds, **a)
    keep = torch.arange(rows, device="cuda") != 11
    for k in ("dx", "dresidual", "dgate"):
        assert torch.equal(got[k][keep], ref[k][keep]), k
    for k in ("dx", "dresidual"):
        assert not torch.isfinite(got[k][11]).any(), k
    da.device_status()


@pytest.mark.parametrize("D", [64, 1000, 2048])
def test_norm_of_zero_and_tiny_rows(D):
    """A row of zeros is zeros; with eps = 1e-5 a row of 1e-3 is far below its norm's floor; gradients stay finite."""
    x = torch.zeros(6, D, device="cuda")
    x[1] = 1e-3
    x[2, 0] = 1.0
    x[3] = 1e18  # squares of 1e36 sum up in range
    ga = torch.ones(D, device="cuda")
    y, s = da.residual_norm(x, gamma=ga)
    ref = block.residual_norm(x.cpu().numpy())[0]
    assert not y[0].any() and torch.equal(s, x)
    assert np.allclose(y.cpu().numpy(), ref, rtol=2.0 ** -17, atol=0)
    got = da.residual_norm_backward(x, s, torch.ones_like(x), None, gamma_post=ga, gamma=ga)
    assert all(torch.isfinite(t).all() for t in got.values())
    da.device_status()


# ----------------------------------------------------------------------------- activations
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_extreme_preactivations(act):
    """z from tiny to 3e38, both signs: outputs and slopes are those of the formula's limits, none is NaN."""
    z = torch.tensor([0.0, 1e-30, 1e-8, 1e-3, 0.1, 0.5, 1.0, 2.0, 3.0, 4.0, 5.0, 6.0, 9.0, 12.0, 40.0, 100.0, 1e4, 1e10, 1e19, 1e20, 3e38, 7.5, 0.02,
                      1.7])
    z = torch.cat([z, -z]).to(BF)
    N = z.numel()
    # z as a product: one token of ones against weights whose first column is z
    w = torch.zeros(N, 8, dtype=BF)
    w[:, 0] = z
    a = torch.zeros(3, 8, dtype=BF)
    a[:, 0] = 1
    Z = z.double().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        value, slope = block.activation(np.clip(Z, -1e4, 1e4), act)
    value = np.where(np.abs(Z) > 1e4, np.where(Z > 0, Z, 0.0), value)
    bound = 2.0 ** -19 * (np.minimum(np.abs(Z), 16) + np.abs(value))
    for M in (3, 300):
        out = da.linear(a[:1].expand(M, 8).contiguous().cuda(), w.cuda(), act=act, dtype=F32)
        got = out.double().cpu().numpy()
        assert np.all(np.isfinite(got))
        assert np.all(np.abs(got - value) <= bound + 1e-37), act
    dy = torch.ones(4, N, dtype=BF, device="cuda")
    got = da.linear_backward(torch.zeros(4, 8, dtype=BF, device="cuda"), w.cuda(), dy, pre=z.expand(4, N).contiguous().cuda(), act=act, da=False,
                             dw=False, bias=True)["dbias"].double().cpu().numpy()
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got / 4 - slope) <= 2.0 ** -18 * (1 + np.minimum(np.abs(Z), 16))), act
    da.device_status()


# ----------------------------------------------------------------------------- streams and graphs
def _calls(rnd, M):
    """name -> (inputs, call(inputs) -> list of outputs)."""
    K, N = 264, 520
    a, w, bias, res, pre, dy = rnd(M, K), rnd(N, K, std=K ** -0.5), rnd(N, dtype=F32), rnd(M, N), rnd(M, N), rnd(M, N)
    wg, gu, dh = rnd(2 * 136, K, std=K ** -0.5), rnd(M, 272), rnd(M, 136)
    x, st, dx, ds, gate, g1 = (rnd(M, K) for _ in range(4)), None, None, None, rnd(M, K, dtype=F32), rnd(K, dtype=F32)
    x = list(x)
    return {
        "linear": ([a, w, bias, res], lambda s, a, w, bias, res: list(da.linear_train(a, w, bias=bias, act="gelu", residual=res, stream=s))),
        "linear_f32": ([a, w, bias], lambda s, a, w, bias: [da.linear(a, w, bias=bias, dtype=F32, stream=s)]),
        "linear_backward": ([a, w, dy, pre], lambda s, a, w, dy, pre: list(da.linear_backward(a, w, dy, pre=pre, act="silu", bias=True, stream=s).values())),
        "gated": ([a, wg], lambda s, a, wg: list(da.gated_linear_train(a, wg, stream=s))),
        "gated_backward": ([a, wg, gu, dh], lambda s, a, wg, gu, dh: list(da.gated_linear_backward(a, wg, gu, dh, stream=s).values())),
        "norm": ([x[0], x[1], gate, g1], lambda s, x, r, gate, g1: list(da.residual_norm(x, r, gate=gate, gamma_post=g1, gamma=g1, stream=s))),
        "norm_backward": ([*x, gate, g1], lambda s, x, st, dy, ds, gate, g1: list(da.residual_norm_backward(
            x, st, dy, ds, gate=gate, gamma_post=g1, gamma=g1, stream=s).values())),
        "norm_backward_shared": ([*x, g1], lambda s, x, st, dy, ds, g1: list(da.residual_norm_backward(
            x, st, dy, ds, gate=g1, gamma_post=g1, gamma=g1, stream=s).values())),
    }


@pytest.mark.parametrize("M", [4, 300])
def test_graphs_replay_on_new_inputs(M):
    """Each call captured alone, two graphs of it replayed in turn on other inputs; the results are the eager call's."""
    calls, other = _calls(_rnd(M), M), _calls(_rnd(M + 1), M)
    for name, (inputs, call) in calls.items():
        graphs = []
        for source in (inputs, other[name][0]):
            mine = [t.clone() for t in source]
            stream = torch.cuda.Stream()
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                call(None, *mine)  # (first use outside of the capture)
            torch.cuda.current_stream().wait_stream(stream)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs = call(None, *mine)
            graphs.append((g, mine, outs))
        for turn in range(2):
            for k, (g, mine, outs) in enumerate(graphs):
                source = (inputs, other[name][0])[(k + turn) % 2]
                for t, src in zip(mine, source):
                    t.copy_(src)
                g.replay()
                for o, r in zip(outs, call(None, *source)):
                    assert torch.equal(o, r), (name, turn, k)
    da.device_status()


@pytest.mark.parametrize("M", [4, 300])
def test_calls_on_another_stream(M):
    """A call on a given stream: its memory is that stream's, results are the current stream's."""
    for name, (inputs, call) in _calls(_rnd(M + 7), M).items():
        ref = call(None, *inputs)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        outs = [call(side, *inputs) for _ in range(3)][-1]
        torch.cuda.current_stream().wait_stream(side)
        for o, r in zip(outs, ref):
            assert torch.equal(o, r), name
    da.device_status()


def test_two_streams_at_once():
    """The same calls on two streams at a time, workspaces of their own: both are right."""
    one, two = _calls(_rnd(50), 500), _calls(_rnd(51), 500)
    refs = {k: [call(None, *i) for i, call in (one[k], two[k])] for k in one}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = {k: [None, None] for k in one}
    for _ in range(5):
        for k in one:
            for j, (src, st) in enumerate(zip((one, two), streams)):
                got[k][j] = src[k][1](st, *src[k][0])
    torch.cuda.synchronize()
    for k in one:
        for j in range(2):
            for o, r in zip(got[k][j], refs[k][j]):
                assert torch.equal(o, r), (k, j)
    da.device_status()


def test_one_workspace_for_calls_in_a_row():
    rnd = _rnd(60)
    a, w, dy, pre = rnd(200, 264), rnd(136, 264), rnd(200, 136), rnd(200, 136)
    ws = torch.empty(max(da.linear_backward_workspace_bytes(200, 136, 264), da.residual_norm_backward_workspace_bytes(200, 264, 0)),
                     dtype=torch.uint8, device="cuda")
    for act in ("gelu", "silu"):
        ref = da.linear_backward(a, w, dy, pre=pre, act=act, bias=True)
        got = da.linear_backward(a, w, dy, pre=pre, act=act, bias=True, workspace=ws)
        for k in ref:
            assert torch.equal(ref[k], got[k]), (act, k)
    ref = da.residual_norm_backward(a, a, a, a, gamma=torch.ones(264, device="cuda"))
    got = da.residual_norm_backward(a, a, a, a, gamma=torch.ones(264, device="cuda"), workspace=ws)
    assert all(torch.equal(ref[k], got[k]) for k in ref)
    with pytest.raises(ValueError):
        da.linear_backward(a, w, dy, pre=pre, act="gelu", workspace=ws[:100])
    with pytest.raises(ValueError):
        da.linear_backward(a, w, dy, act="gelu")
    with pytest.raises(ValueError):
        da.residual_norm_backward(a, a, a, out={"dgate": ref["dx"]})


def test_results_repeat():
    """Clusters that share a contraction, split sums over rows: the same bits every time."""
    rnd = _rnd(70)
    for M, N, K in ((1, 1024, 8192), (40, 512, 8192), (128, 2048, 2048), (200, 1024, 4096), (1000, 1000, 1000)):
        a, w = rnd(M, K), rnd(N, K)
        for dt in (BF, F32):
            ref = da.linear(a, w, dtype=dt)
            for _ in range(5):
                assert torch.equal(da.linear(a, w, dtype=dt), ref), (M, N, K)
    da.device_status()


# ----------------------------------------------------------------------------- long tensors
def test_offsets_past_32_bits():
    """Outputs of more than 2^31 elements: the last rows are what a call on those rows alone gives."""
    rnd = _rnd(80)
    M, N, K = 70000, 32768, 64
    a, w = rnd(M, K), rnd(N, K)
    out = da.linear(a, w)
    assert torch.equal(out[-300:], da.linear(a[-300:].contiguous(), w)) and torch.equal(out[:300], da.linear(a[:300].contiguous(), w))
    d = da.linear_backward(a, w, out, pre=out, act="relu", dw=False)["da"]
    tail = da.linear_backward(a[-300:].contiguous(), w, out[-300:].contiguous(), pre=out[-300:].contiguous(), act="relu", dw=False)["da"]
    # (the two calls may split the contraction differently: each is within (N / 16 + 2) 2^-22 of the sum S of its terms'
    # magnitudes before it is rounded, by 2^-8 of itself at most)
    dz, t64 = out[-256:].double().clamp_min(0) * (out[-256:] > 0), tail[-256:].double()
    S = dz.abs() @ w.double().abs()
    bound = 2 * (N / 16 + 2) * 2.0 ** -22 * S * (1 + 2.0 ** -8) + 2 * 2.0 ** -8 * t64.abs()
    assert bool(((d[-256:].double() - t64).abs() <= bound).all())
    del dz, S, bound, t64
    del out, d, tail
    rows, D = 300000, 8192
    x = rnd(1, D).expand(rows, D).contiguous()
    x[-3:] = rnd(3, D)
    y, s = da.residual_norm(x, x)
    yt, st = da.residual_norm(x[-3:].contiguous(), x[-3:].contiguous())
    assert torch.equal(y[-3:], yt) and torch.equal(s[-3:], st)
    got = da.residual_norm_backward(x, s, y, None)
    assert torch.equal(got["dx"][-3:], da.residual_norm_backward(x[-3:].contiguous(), st, yt, None)["dx"])
    da.device_status()


# ----------------------------------------------------------------------------- a block put together
def _rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("B,n,D,F", [(2, 100, 256, 680), (1, 3, 256, 680), (3, 257, 512, 1368)])
def test_a_block_and_its_gradients(B, n, D, F):
    """x + attention(norm x), then gate and norms, then the gated feed-forward half with its residual; the feed-forward half's
    gradients back to the attention's output and the stream.  Stages are held to the formulas in 64 bits on the stages' own
    inputs; the gradients' path to autograd in 64 bits through all of them: at most eight roundings to bf16 lie on a path, each
    2^-8 of a value at most, so 2^-5 of the norm."""
    rnd = _rnd(B + n)
    H, d = 2, 64
    x = rnd(B, n, D)
    w_qkv, w_o = rnd(6 * H * d, D, std=D ** -0.5), rnd(D, 2 * H * d, std=(2 * H * d) ** -0.5)
    vec = [0.1 * rnd(d, dtype=F32) for _ in range(4)]
    g1, gp, g2 = (1 + 0.1 * rnd(D, dtype=F32) for _ in range(3))
    gate = 1 + 0.2 * rnd(B, D, dtype=F32)
    w_gu, w_down = rnd(2 * F, D, std=D ** -0.5), rnd(D, F, std=F ** -0.5)
    y0, s0 = da.residual_norm(x, gamma=g1)
    attn = da.layer_forward(y0, w_qkv, w_o, *vec, 0.5, H)
    y, s = da.residual_norm(attn, s0, gate=gate, scale=0.7, gamma_post=gp, gamma=g2)
    h, gu = da.gated_linear_train(y, w_gu)
    out = da.linear(h, w_down, residual=s)
    da.device_status()
    assert torch.equal(s0, x)

    def norm(t, g):
        return t / torch.sqrt((t * t).mean(-1, keepdim=True) + 1e-5) * g

    D64 = [t.double() for t in (attn, s0, gate, gp, g2, w_gu, w_down)]
    for t in D64:
        t.requires_grad_()
    a64, r64, t64, gp64, g264, wg64, wd64 = D64
    S = r64 + 0.7 * t64[:, None] * norm(a64, gp64)
    Y = norm(S, g264)
    GU = Y @ wg64.T
    Hh = torch.nn.functional.silu(GU[..., :F]) * GU[..., F:]
    O = S + Hh @ wd64.T
    for name, got, ref in (("y0", y0, norm(x.double(), g1.double())), ("s", s, S), ("y", y, Y), ("gu", gu, GU), ("h", h, Hh), ("out", out, O)):
        assert _rel(got, ref.detach()) < 2.0 ** -7, name
    dout = rnd(B, n, D)
    ref = torch.autograd.grad(O, D64, dout.double())
    down = da.linear_backward(h, w_down, dout)
    ffn = da.gated_linear_backward(y, w_gu, gu, down["da"])
    mid = da.residual_norm_backward(attn, s, ffn["dx"], dout, gate=gate, scale=0.7, gamma_post=gp, gamma=g2)
    da.device_status()
    for name, got, want in (("attention", mid["dx"], ref[0]), ("residual", mid["dresidual"], ref[1]), ("gate", mid["dgate"], ref[2]),
                            ("gamma_post", mid["dgamma_post"], ref[3]), ("gamma", mid["dgamma"], ref[4]), ("w_gu", ffn["dw"], ref[5]),
                            ("w_down", down["dw"], ref[6])):
        assert _rel(got, want) < 2.0 ** -5, (name, _rel(got, want))


def test_a_training_step_in_a_graph_beside_an_eager_one():
    """Forward and backward of the feed-forward half captured while the same tensors are in use eagerly before and after."""
    rnd = _rnd(90)
    M, D, F = 200, 256, 680
    x, w_gu, w_down, dout = rnd(M, D), rnd(2 * F, D, std=0.06), rnd(D, F, std=0.04), rnd(M, D)

    def step():
        y, s = da.residual_norm(x)
        h, gu = da.gated_linear_train(y, w_gu)
        out = da.linear(h, w_down, residual=s)
        down = da.linear_backward(h, w_down, dout)
        ffn = da.gated_linear_backward(y, w_gu, gu, down["da"])
        mid = da.residual_norm_backward(x, s, ffn["dx"], dout)
        return [out, down["dw"], ffn["dw"], mid["dx"]]
    ref = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = step()
    again = step()
    for _ in range(3):
        g.replay()
    for o, r, q in zip(outs, ref, again):
        assert torch.equal(o, r) and torch.equal(q, r)
    da.device_status()


# ----------------------------------------------------------------------------- sizes and devices that are refused
def test_sizes_past_31_bits_are_refused():
    """Expanded views: nothing of this size is allocated."""
    big = 2**32 + 8
    x, w = torch.empty(1, 8, device="cuda", dtype=BF), torch.empty(16, 8, device="cuda", dtype=BF)
    tall = x.expand(big, 8)
    for f in (lambda: da.linear(tall, w), lambda: da.linear(x, w[:1].expand(big, 8)), lambda: da.gated_linear(tall, w),
              lambda: da.linear(x[:, :1].expand(1, big), w[:, :1].expand(16, big)),
              lambda: da.linear_backward(tall, w, x), lambda: da.gated_linear_backward(tall, w, w, x),
              lambda: da.residual_norm(tall), lambda: da.residual_norm(x[:, :1].expand(1, big)),
              lambda: da.residual_norm_backward(tall, tall, tall), lambda: da.linear(tall.view(big // 8, 8, 8), w)):
        with pytest.raises(ValueError, match=r"sizes are below 2\^31"):
            f()


def test_another_device_than_the_current_one_is_refused(monkeypatch):
    x, w = torch.zeros(4, 8, device="cuda", dtype=BF), torch.zeros(16, 8, device="cuda", dtype=BF)
    stream = torch.cuda.current_stream()
    other = type("Stream", (), {"device_index": x.get_device() + 1, "cuda_stream": 0})()
    with pytest.raises(ValueError, match="the stream is on device"):
        da.linear(x, w, out=torch.empty(4, 16, device="cuda", dtype=BF), stream=other)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: x.get_device() + 1)
    for s in (None, stream):
        for f in (lambda: da.linear(x, w, stream=s), lambda: da.gated_linear(x, w, stream=s), lambda: da.residual_norm(x, stream=s),
                  lambda: da.linear_backward(x, w, x.new_zeros(4, 16), stream=s), lambda: da.residual_norm_backward(x, x, x, stream=s),
                  lambda: da.gated_linear_backward(x, w, x.new_zeros(4, 16), x, stream=s)):
            with pytest.raises(ValueError, match="the current device is"):
                f()
