"""The layer for a few tokens (moe_forward_decode, moe_forward_decode_w4)
against its definition in 64 bits, elementwise within bounds derived from the
float32 sums it makes (tests/few_rows.py)."""
import pytest
import torch

from tests import few_rows as ref

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def make(T, d, h, E, k, S=0, dtype="bf16", act="gelu", bias=True, b_g=False, b_sel=False, seed=0, group=None,
         zeros=False):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda shape, std, t=dt: (torch.randn(shape, generator=g) * std).to(t)
    n = E + S
    p = dict(x=rnd((T, d), 1.0), W_g=rnd((E, d), 0.5 / d ** 0.5), b1=rnd((n, h), 0.2) if bias else None,
             b2=rnd((n, d), 0.2) if bias else None, b_g=rnd((E,), 1.0, torch.float32) if b_g else None,
             b_sel=rnd((E,), 1.0, torch.float32) if b_sel else None, k=k, S=S, act=act, group=group)
    if group is None:
        p.update(W1=rnd((n, h, d), d ** -0.5), W2=rnd((n, d, h), h ** -0.5))
    else:
        for name, rows, cols in (("W1", h, d), ("W2", d, h)):
            p[name] = torch.randint(0, 256, (n, rows, cols // 2), generator=g, dtype=torch.uint8)
            p[name + "s"] = ((0.5 + torch.rand((n, rows, cols // group), generator=g)) * 0.2 * cols ** -0.5).to(dt)
            p[name + "z"] = (torch.randint(0, 16, (n, rows, cols // group), generator=g, dtype=torch.uint8)
                             if zeros else None)
    return p


def on_gpu(p):
    return {n: v.to(DEV) if isinstance(v, torch.Tensor) else v for n, v in p.items()}


def run(q, packed=False, workspace=None):
    import sparse_mixture_experts_28_amd as moe
    if q["group"] is not None:
        return moe.forward_decode_w4(q["x"], q["W_g"], q["W1"], q["W1s"], q["W1z"], q["b1"], q["W2"], q["W2s"],
                                     q["W2z"], q["b2"], q["k"], q["S"], q["b_g"], activation=q["act"],
                                     b_sel=q["b_sel"], workspace=workspace)
    W1, W2 = (moe.pack_weights(q["W1"]), moe.pack_weights(q["W2"])) if packed else (q["W1"], q["W2"])
    return moe.forward_decode(q["x"], q["W_g"], W1, q["b1"], W2, q["b2"], q["k"], q["S"], q["b_g"],
                              activation=q["act"], b_sel=q["b_sel"], weights_packed=packed, workspace=workspace)


def reference(p):
    f = lambda v, e: None if v is None else v[e].to(torch.float64)

    def expert(e):
        if p["group"] is None:
            return f(p["W1"], e), None, f(p["b1"], e), f(p["W2"], e), None, f(p["b2"], e)
        a, sa = ref.unpack_w4(p["W1"][e], p["W1s"][e], None if p["W1z"] is None else p["W1z"][e])
        b, sb = ref.unpack_w4(p["W2"][e], p["W2s"][e], None if p["W2z"] is None else p["W2z"][e])
        return a, sa, f(p["b1"], e), b, sb, f(p["b2"], e)
    bf = p["x"].dtype == torch.bfloat16
    return ref.layer(p["x"], p["W_g"], expert, p["W_g"].shape[0], p["k"], p["S"], p["b_g"], p["b_sel"], p["act"],
                     2.0 ** -8 if bf else 2.0 ** -24, 2.0 ** -16 if bf else 2.0 ** -24)


def check(p, r):
    torch.cuda.synchronize()
    out, idx, w, bound = reference(p)
    assert torch.equal(r.topk_idx.cpu().long(), idx)
    assert (r.topk_w.cpu().double() - w).abs().max() <= 1e-5
    ref.check(r.out, out, bound, "out")


SHAPES = [
    # T, d, h, E, k, S
    (1, 8, 8, 1, 1, 0), (1, 64, 128, 4, 2, 0), (2, 40, 24, 5, 5, 0), (7, 264, 72, 8, 2, 1), (8, 256, 512, 16, 4, 0),
    (9, 512, 256, 16, 2, 2), (16, 136, 2056, 64, 8, 0), (17, 1024, 96, 3, 1, 0), (33, 72, 520, 256, 8, 1),
    (63, 32, 128, 4, 2, 0), (64, 512, 1024, 8, 2, 8), (64, 128, 64, 256, 8, 0), (3, 4096, 520, 8, 2, 0),
    (5, 16, 8192, 8, 2, 0), (64, 24, 4104, 2, 1, 1), (17, 328, 1064, 2, 1, 1), (48, 72, 4104, 1, 1, 1),
    (49, 1032, 488, 3, 2, 0),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,h,E,k,S", SHAPES)
def test_shapes(T, d, h, E, k, S, dtype):
    p = make(T, d, h, E, k, S, dtype, act="silu" if T % 2 else "gelu", bias=T % 3 != 0, b_g=E > 4, b_sel=T > 8, seed=T)
    check(p, run(on_gpu(p)))


@pytest.mark.parametrize("T,d,h,E,k,S", [(1, 256, 256, 4, 2, 0), (13, 512, 768, 8, 2, 1), (40, 256, 1024, 16, 4, 0),
                                           (64, 512, 768, 4, 2, 1)])
def test_packed_weights_give_the_same_bits(T, d, h, E, k, S):
    p = make(T, d, h, E, k, S, seed=3)
    q = on_gpu(p)
    a, b = run(q), run(q, packed=True)
    check(p, a)
    assert torch.equal(a.out, b.out) and torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_w, b.topk_w)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,dg,hg,E,k,S", [(1, 1, 1, 1, 1, 0), (1, 5, 9, 8, 2, 0), (6, 3, 4, 4, 3, 1),
                                           (12, 7, 2, 16, 2, 0), (33, 2, 11, 64, 8, 1), (64, 4, 3, 8, 2, 0),
                                           (3, 33, 67, 4, 2, 1)])
def test_w4(T, dg, hg, E, k, S, group, zeros):
    p = make(T, dg * group, hg * group, E, k, S, act="gelu" if T % 2 else "silu", bias=E > 4, b_g=T > 6, seed=T + group,
             group=group, zeros=zeros)
    check(p, run(on_gpu(p)))


def variants():
    return [pytest.param(dict(dtype="bf16"), id="bf16"), pytest.param(dict(dtype="f32"), id="f32"),
            pytest.param(dict(dtype="bf16", group=32, zeros=True), id="w4")]


@pytest.mark.parametrize("kw", variants())
@pytest.mark.parametrize("T", [1, 11, 50])
def test_same_bits_twice_and_any_workspace(kw, T):
    """Two calls agree bit for bit, whatever the workspace holds; nothing is written past it."""
    import sparse_mixture_experts_28_amd as moe
    p = make(T, 320, 576, 16, 4, 1, seed=5, **kw)
    q = on_gpu(p)
    a = run(q)
    n = (moe.moe_workspace_bytes_decode_w4(T, 320, 576, 16, 4, 1) if kw.get("group") else
         moe.moe_workspace_bytes_decode(T, 320, 576, 16, 4, 1, moe.MOE_BF16 if kw["dtype"] == "bf16" else moe.MOE_F32))
    for fill in (0xff, 0x5a, 0):
        buf = torch.full((n + 4096,), fill, dtype=torch.uint8, device=DEV)
        b = run(q, workspace=buf[:n])
        torch.cuda.synchronize()
        assert torch.equal(a.out, b.out) and torch.equal(a.topk_idx, b.topk_idx) and torch.equal(a.topk_w, b.topk_w)
        assert bool((buf[n:] == fill).all())
    check(p, a)


@pytest.mark.parametrize("kw", variants())
def test_experts_reach_only_their_tokens(kw):
    """NaN and infinities in the weights of an expert: untaken, it changes nothing; taken, only its tokens see them."""
    p = make(20, 192, 160, 6, 1, 0, bias=False, seed=8, **kw)
    p["b_g"] = torch.tensor([0.0, 0.0, 0.0, 0.0, -1e9, 0.0])
    clean = run(on_gpu(p))
    bad = dict(p)
    names = ("W1s", "W2s") if kw.get("group") else ("W1", "W2")
    for name, v in zip(names, (float("nan"), float("inf"))):
        bad[name] = p[name].clone()
        bad[name][4] = v
    r = run(on_gpu(bad))
    assert torch.equal(clean.out, r.out)
    e = int(clean.topk_idx[0, 0])
    for name in names:
        bad[name][e] = float("nan")
    r = run(on_gpu(bad))
    hit = (r.topk_idx == e).any(1)
    assert bool(hit.any()) and not bool(hit.all())
    assert bool(r.out[hit].isnan().all())
    assert torch.equal(r.out[~hit], clean.out[~hit])


@pytest.mark.parametrize("kw", variants())
def test_nan_token_stays_alone(kw):
    p = make(18, 128, 96, 8, 2, 1, seed=9, **kw)
    clean = run(on_gpu(p))
    p["x"][5, 7] = float("nan")
    r = run(on_gpu(p))
    assert bool(r.out[5].isnan().all()) and bool(((r.topk_idx >= 0) & (r.topk_idx < 8)).all())
    keep = torch.arange(18, device=DEV) != 5
    assert torch.equal(r.out[keep], clean.out[keep]) and torch.equal(r.topk_idx[keep], clean.topk_idx[keep])


def test_ties_go_to_the_lower_expert():
    p = make(4, 64, 64, 130, 8, 0, seed=1)
    p["W_g"][:] = p["W_g"][0]
    r = run(on_gpu(p))
    assert torch.equal(r.topk_idx.cpu(), torch.arange(8, dtype=torch.int32).expand(4, 8))
    assert (r.topk_w - 0.125).abs().max() < 1e-6


def test_a_selection_bias_far_above_the_logits():
    """The weights are normalised over the chosen logits alone: an expert whose logit lies 200 below the largest is
    chosen through its bias and gets its weight without underflow."""
    p = make(3, 64, 64, 6, 2, 0, seed=2)
    p["b_g"] = torch.tensor([0.0, 0.0, 200.0, 0.0, 0.0, 0.0])
    p["b_sel"] = torch.tensor([0.0, 1000.0, 0.0, 0.0, 900.0, 0.0])
    r = run(on_gpu(p))
    check(p, r)
    assert set(r.topk_idx[0].tolist()) == {1, 4}


@pytest.mark.parametrize("kw", variants())
def test_graph_replays_and_two_streams(kw):
    """Two captured calls with workspaces of their own, replayed on two streams at once with new inputs, among eager
    calls."""
    p1, p2 = make(3, 256, 512, 8, 2, 1, seed=11, **kw), make(30, 320, 256, 8, 2, 0, seed=12, **kw)
    q = [on_gpu(p1), on_gpu(p2)]
    graphs, outs = [], []
    s = torch.cuda.Stream()
    for one in q:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run(one)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(one))
        graphs.append(g)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for seed in range(4):
        for one in q:
            one["x"].copy_(torch.randn(one["x"].shape, generator=torch.Generator().manual_seed(seed)).to(one["x"].dtype))
        eager = [run(one) for one in q]
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(side[i]):
                graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, outs):
            assert torch.equal(a.out, b.out) and torch.equal(a.topk_idx, b.topk_idx)


def test_refusals():
    import sparse_mixture_experts_28_amd as moe
    host = make(4, 64, 96, 4, 2, 1, seed=2)
    p, q = on_gpu(host), on_gpu(make(4, 64, 96, 4, 2, 1, seed=2, group=32, zeros=True))
    small = torch.zeros(256, dtype=torch.uint8, device=DEV)
    long = torch.zeros(65, 64, dtype=torch.bfloat16, device=DEV)
    odd = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)[1:]
    big = lambda t: torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype, device=DEV)[..., ::2]
    common = [dict(x=p["x"].float()), dict(x=p["x"].cpu()), dict(x=long), dict(x=long[:0]), dict(x=big(p["x"])),
              dict(W_g=p["W_g"].float()), dict(W_g=p["W_g"][:3]), dict(W_g=p["W_g"].cpu()), dict(k=0), dict(k=5),
              dict(k=(1 << 32) + 2), dict(S=0), dict(S=-1), dict(b1=p["b1"][:4]), dict(b2=p["b2"].float()),
              dict(b_g=p["b1"][0, :4]), dict(b_sel=torch.zeros(5, device=DEV)), dict(act="relu"),
              dict(workspace=small), dict(workspace=torch.zeros(1 << 20, dtype=torch.uint8)), dict(workspace=odd)]
    wide = [dict(W1=p["W1"].float()), dict(W1=p["W1"].cpu()), dict(W2=p["W2"][:4]), dict(W1=p["W1"].transpose(1, 2)),
            dict(packed=True)]
    four = [dict(W1s=q["W1s"].float()), dict(W1=q["W1"][..., ::2]), dict(W1z=q["W1z"][:4]), dict(W2s=q["W2s"][..., :1]),
            dict(W1=q["W1"].cpu()), dict(W2z=q["W2z"].to(torch.int8))]
    for base, bad in [(p, b) for b in common + wide] + [(q, b) for b in common + four]:
        kw = {n: bad[n] for n in ("packed", "workspace") if n in bad}
        with pytest.raises((ValueError, RuntimeError)):
            run(dict(base, **{n: v for n, v in bad.items() if n not in kw}), **kw)
    check(host, run(p, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)))   # and the calls before left no error


def test_as_a_server_would_use_them():
    """A prompt through the grouped layer, its continuation token by token through the few-token layer, and both again
    on 4-bit weights read back for the prompt: routing agrees, and the outputs agree within the two paths' roundings."""
    import sparse_mixture_experts_28_amd as moe
    T, d, h, E, k = 96, 256, 512, 8, 2
    p = make(T, d, h, E, k, 0, act="silu", bias=False, seed=21)
    q = on_gpu(p)
    full = moe.forward(q["x"], q["W_g"], q["W1"], None, q["W2"], None, k, activation="silu")
    scale = full.out.float().abs().max()
    for lo, hi in ((0, 1), (1, 9), (9, 64), (64, 96)):
        r = moe.forward_decode(q["x"][lo:hi], q["W_g"], q["W1"], None, q["W2"], None, k, activation="silu")
        assert torch.equal(r.topk_idx, full.topk_idx[lo:hi])
        # moe_forward rounds H and Y to bf16 and the output once more
        assert (r.out.float() - full.out[lo:hi].float()).abs().max() <= 2e-2 * scale
    W1, W2 = moe.quantize_w4(q["W1"], 64, True), moe.quantize_w4(q["W2"], 64, True)
    full4 = moe.forward(q["x"], q["W_g"], moe.dequantize_w4(*W1), None, moe.dequantize_w4(*W2), None, k,
                        activation="silu")
    scale = full4.out.float().abs().max()
    for lo, hi in ((0, 1), (1, 33), (33, 96)):
        r = moe.forward_decode_w4(q["x"][lo:hi], q["W_g"], *W1, None, *W2, None, k, activation="silu")
        assert torch.equal(r.topk_idx, full4.topk_idx[lo:hi])
        assert (r.out.float() - full4.out[lo:hi].float()).abs().max() <= 2e-2 * scale
    # the first Linear of one expert alone, as its hidden rows before the activation
    x = q["x"][:5]
    y = moe.linear_w4(x, W1[0][3], W1[1][3], W1[2][3])
    w = moe.dequantize_w4(W1[0][3], W1[1][3], W1[2][3]).float()
    assert (y.float() - x.float() @ w.t()).abs().max() <= 2e-2 * y.float().abs().max()
