"""The new calls of a block together: a training step through norm, routing, gated
experts, a shared expert with adapters, combine and the norm after, with its way back;
calls on other streams, in captured graphs, beyond 2^31 elements; and that equal calls
give equal bits."""
import pytest
import torch

import mixture_experts_layer_06_amd as moe
from test_gpu_ffn_streams import keep_busy

pytestmark = pytest.mark.gpu


def block_operands(T=48, H=64, F=32, E=6, K=2, R=4, adapters=3, seed=0):
    gen = torch.Generator().manual_seed(seed)
    mk = lambda *s, sc=1.0: torch.randn(s, generator=gen) * sc  # noqa: E731
    p = {"x": mk(T, H), "w_pre": 1 + mk(H, sc=0.1), "w_router": mk(H, E, sc=H ** -0.5),
         "w_gate": mk(E, H, F, sc=H ** -0.5), "w_up": mk(E, H, F, sc=H ** -0.5), "w_down": mk(E, F, H, sc=F ** -0.5),
         "w_shared": mk(1, H, H, sc=H ** -0.5), "a": mk(adapters, H, R, sc=H ** -0.5), "b": mk(adapters, R, H, sc=0.3),
         "w_post": 1 + mk(H, sc=0.1), "ls": 0.5 + mk(H, sc=0.1)}
    adapter = torch.randint(0, adapters + 1, (T, 1), generator=gen, dtype=torch.int32)
    return p, adapter, mk(T, H), torch.tensor([0.3, 0.05])


def forward64(p, adapter, idx, scale, counts=None):
    """The block in torch on the CPU, its selection and the loss's counts given."""
    T, E, K = p["x"].shape[0], p["w_router"].shape[1], idx.shape[1]
    h = p["x"] * torch.rsqrt(p["x"].square().mean(1, keepdim=True) + 1e-6) * p["w_pre"]
    scores = h @ p["w_router"]
    gate = torch.softmax(scores.gather(1, idx), 1)
    y = torch.zeros_like(h)
    for e in range(E):
        t, k = (idx == e).nonzero(as_tuple=True)
        z = (torch.nn.functional.silu(h[t] @ p["w_gate"][e]) * (h[t] @ p["w_up"][e])) @ p["w_down"][e]
        y = y.index_add(0, t, gate[t, k][:, None] * z)
    s = h @ p["w_shared"][0]
    delta = torch.zeros_like(s)
    for a in range(p["a"].shape[0]):
        t = (adapter[:, 0] == a).nonzero()[:, 0]
        delta = delta.index_add(0, t, scale[a] * (h[t] @ p["a"][a]) @ p["b"][a])
    y = y + s + delta
    out = 0.8 * p["x"] + p["ls"] * y * torch.rsqrt(y.square().mean(1, keepdim=True) + 1e-6) * p["w_post"]
    counts = torch.bincount(idx.reshape(-1), minlength=E).to(h.dtype)
    balance = E / (T * K) * (counts * torch.softmax(scores, 1).mean(0)).sum()
    return out, torch.stack([balance, torch.logsumexp(scores, 1).square().mean()])


def test_training_step_through_the_block():
    """Every gradient of the block in fp32 against autograd in 64 bits. A chain of about
    ten operators, sums of up to 64 values in each: 2e-5 of a gradient's norm is a
    hundred times their roundings, and far below what a wrong term would do."""
    p, adapter, dout, dloss = block_operands()
    d = {k: v.cuda() for k, v in p.items()}
    T, H = p["x"].shape
    E, K = p["w_router"].shape[1], 2
    scale = torch.tensor([2.0, 0.5, 1.0])
    n = p["a"].shape[0]
    # forward
    _, h = moe.block_norm(None, d["x"], w_pre=d["w_pre"])
    idx, gate, scores = moe.route(h, d["w_router"], K, scores=True)
    loss = moe.router_loss(scores, idx)
    plan = moe.permute(idx, E)
    hid, g, u = moe.gmm_glu(h, d["w_gate"], d["w_up"], plan["offsets"], rows=plan["perm_src"], row_div=K, save=True)
    z = moe.gmm(hid, d["w_down"], plan["offsets"])
    y = moe.combine(z, plan["perm_dst"], gate, T, K)
    one = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    s = moe.gmm(h, d["w_shared"], one)
    lp = moe.permute(adapter.cuda(), n + 1)
    lo = lp["offsets"][:n + 1]
    s, lu = moe.lora(h, d["a"], d["b"], lo, rows=lp["perm_src"], scale=scale.cuda(), base=s, out=s, u=True)
    y = y + s
    out, _ = moe.block_norm(y, d["x"], d["w_post"], gate=d["ls"], pre=False, alpha=0.8)
    # backward
    grads = moe.block_norm_bwd(None, dout.cuda(), y, None, d["w_post"], gate=d["ls"], alpha=0.8)
    dy = grads.pop("dz")
    dz, dgate = moe.combine_bwd(dy, z, plan["perm_dst"], gate)
    grads["dw_down"] = moe.gmm_wgrad(hid, dz, plan["offsets"])
    da, grads["dw_gate"], grads["dw_up"] = moe.gmm_glu_bwd(moe.gmm_dgrad(dz, d["w_down"], plan["offsets"]), g, u, h,
                                                           d["w_gate"], d["w_up"], plan["offsets"],
                                                           rows=plan["perm_src"], row_div=K)
    ones = torch.ones((T, K), device="cuda")
    dh = moe.combine(da, plan["perm_dst"], ones, T, K)
    ds = moe.router_loss_bwd(scores, idx, loss["counts"], loss["tokens"], dloss=dloss.cuda(), gate=gate, dgate=dgate)
    dh += moe.gmm_dgrad(ds, d["w_router"][None], one)
    grads["dw_router"] = moe.gmm_wgrad(h, ds, one)[0]
    grads["dw_shared"] = moe.gmm_wgrad(h, dy, one)
    dh += moe.gmm_dgrad(dy, d["w_shared"], one)
    dh, grads["da"], grads["db"] = moe.lora_bwd(dy, h, lu, d["a"], d["b"], lo, rows=lp["perm_src"], scale=scale.cuda(),
                                                base=dh, dx=dh)
    last = moe.block_norm_bwd(dh, grads.pop("dr"), None, d["x"], w_pre=d["w_pre"])
    grads["dx"], grads["dw_pre"] = last["dr"], last["dw_pre"]
    grads["dls"] = grads.pop("dgate")
    # reference
    v = {k: t.double().requires_grad_() for k, t in p.items()}
    want, want_loss = forward64(v, adapter, idx.cpu().long(), scale.double())
    ((want * dout.double()).sum() + (want_loss * dloss.double()).sum()).backward()
    near = lambda a, b: (a.detach().cpu().double() - b.detach()).norm() <= 2e-5 * b.detach().norm()  # noqa: E731
    assert near(out, want) and near(loss["loss"], want_loss)
    for k, t in v.items():
        assert near(grads.pop("d" + k), t.grad), k
    assert not grads


def serving_step(x, p, off, plan_rows, scale, K=2):
    """One decode step of a block with adapters (bf16)."""
    _, h = moe.block_norm(None, x, w_pre=p["w_pre"])
    idx, gate = moe.route(h, p["w_router"], K)
    plan = moe.permute(idx, p["w_gate"].shape[0])
    hid = moe.gmm_glu(h, p["w_gate"], p["w_up"], plan["offsets"], rows=plan["perm_src"], row_div=K)
    y = moe.combine(moe.gmm(hid, p["w_down"], plan["offsets"]), plan["perm_dst"], gate, x.shape[0], K)
    one = p["one"]
    s = moe.lora(h, p["a"], p["b"], off, rows=plan_rows, scale=scale, base=moe.gmm(h, p["w_shared"], one))
    y += s
    return moe.block_norm(y, x, p["w_post"], gate=p["ls"], w_pre=p["w_pre"])


@pytest.mark.parametrize("T", [1, 17])
def test_serving_step_in_a_graph(T):
    """A decode step, captured: replays on new tokens give the eager step's bits."""
    p, adapter, _, _ = block_operands(T=T, H=128, F=64, seed=T)
    d = {k: v.bfloat16().cuda() for k, v in p.items()}
    d["one"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    n = p["a"].shape[0]
    lp = moe.permute(adapter.cuda(), n + 1)
    args = (d, lp["offsets"][:n + 1], lp["perm_src"], torch.ones(n, device="cuda"))
    x = d["x"].clone()
    serving_step(x, *args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = serving_step(x, *args)
    for i in range(4):
        x.copy_(torch.randn((T, 128), generator=torch.Generator().manual_seed(i)))
        want = serving_step(x.clone(), *args)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def calls():
    gen = torch.Generator().manual_seed(0)
    mk = lambda *s, dt=torch.bfloat16: torch.randn(s, generator=gen).to(dt).cuda()  # noqa: E731
    T, E, K, N, H, R, e = 6000, 24, 3, 640, 512, 16, 3
    scores = mk(T, E, dt=torch.float32)
    idx = scores.topk(K, 1).indices.to(torch.int32)
    gate, dgate, dloss = torch.softmax(mk(T, K, dt=torch.float32), 1), mk(T, K, dt=torch.float32), mk(2, dt=torch.float32)
    base = moe.router_loss(scores, idx)
    dst = torch.randperm(T * K, generator=gen).to(torch.int32).cuda()
    yp, d, z, r = mk(T * K, N), mk(T, N), mk(T, N), mk(T, N, dt=torch.float32)
    w, g = mk(N), mk(N)
    x, a, b, dx = mk(T, H), mk(e, H, R), mk(e, R, N), mk(T, H)
    off = torch.tensor([0, 2000, 2100, 5900], dtype=torch.int32, device="cuda")
    rows = torch.randperm(T, generator=gen).to(torch.int32).cuda()
    u = mk(T, R, dt=torch.float32)
    norm = dict(w_post=w, gate=g, w_pre=w)
    torch.cuda.synchronize()
    return {
        "router_loss": lambda **k: tuple(moe.router_loss(scores, idx, **k).values()),
        "router_loss_bwd": lambda **k: (moe.router_loss_bwd(scores, idx, base["counts"], base["tokens"], dloss=dloss,
                                                            gate=gate, dgate=dgate, **k),),
        "combine_bwd": lambda **k: moe.combine_bwd(d, yp, dst, gate, **k),
        "block_norm": lambda **k: moe.block_norm(z, r, **norm, **k),
        "block_norm_bwd": lambda **k: tuple(moe.block_norm_bwd(d, r, z, r, **norm, **k).values()),
        "lora": lambda **k: moe.lora(x, a, b, off, rows=rows, base=d, u=True, **k),
        "lora_bwd": lambda **k: moe.lora_bwd(d, x, u, a, b, off, rows=rows, base=dx, **k),
    }


OPS = ("router_loss", "router_loss_bwd", "combine_bwd", "block_norm", "block_norm_bwd", "lora", "lora_bwd")


def covered(op, results):
    """u holds nothing in the rows of no adapter."""
    return [results[0], results[1][:5900]] if op == "lora" else list(results)


@pytest.mark.parametrize("op", OPS)
def test_same_call_same_bits(op):
    call = calls()[op]
    first = covered(op, call())
    for _ in range(3):
        for a, b in zip(first, covered(op, call())):
            assert torch.equal(a, b)


@pytest.mark.parametrize("op", OPS)
def test_results_of_another_stream_may_be_read_at_once(op):
    call = calls()[op]
    want = [t.clone() for t in covered(op, call())]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        junk = [torch.full_like(t, 1) for t in want]
    torch.cuda.synchronize()
    del junk
    hold = keep_busy(side)
    got = [t.clone() for t in covered(op, call(stream=side))]
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del hold


@pytest.mark.parametrize("op", OPS)
def test_two_streams_at_once(op):
    call = calls()[op]
    want = [t.clone() for t in covered(op, call())]
    sides = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [covered(op, call(stream=sides[i % 2])) for i in range(6)]
    torch.cuda.synchronize()
    for one in got:
        for a, b in zip(one, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("op", OPS)
def test_captured_and_replayed(op):
    """Two graphs of the same call, replayed in turn with eager calls between."""
    call = calls()[op]
    want = [t.clone() for t in covered(op, call())]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = covered(op, call())
        graphs.append((graph, out))
    for _ in range(3):
        for graph, out in graphs:
            for t in out:
                t.fill_(1)
            again = covered(op, call())
            graph.replay()
            torch.cuda.synchronize()
            for a, b, c in zip(out, want, again):
                assert torch.equal(a, b) and torch.equal(c, b)


def test_beyond_32_bits():
    """Rows whose offsets pass 2^31 elements: the last rows get what they get alone."""
    T, N = 70000, 32768
    z = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    z.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    w = torch.rand(N, device="cuda") + 0.5
    last = z[-64:].clone()
    ro, h = moe.block_norm(z, z, w, w_pre=w)
    want = moe.block_norm(last, last, w, w_pre=w)
    assert torch.equal(ro[-64:], want[0]) and torch.equal(h[-64:], want[1])
    got = moe.block_norm_bwd(h, ro, z, ro, w, w_pre=w, need_dw=False)
    part = moe.block_norm_bwd(h[-64:].clone(), ro[-64:].clone(), last, ro[-64:].clone(), w, w_pre=w, need_dw=False)
    assert torch.equal(got["dr"][-64:], part["dr"]) and torch.equal(got["dz"][-64:], part["dz"])
    del got, part, want
    a = torch.randn((1, N, 4), device="cuda").bfloat16()
    b = torch.randn((1, 4, N), device="cuda").bfloat16()
    off = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    rows = torch.arange(T - 64, T, dtype=torch.int32, device="cuda")
    out = moe.lora(z, a, b, off, rows=rows, base=h, out=h)
    one = moe.lora(last, a, b, off, base=torch.zeros_like(last))
    fresh = moe.block_norm(last, last, w, w_pre=w)[1]
    both = moe.lora(last, a, b, off, base=fresh)
    assert torch.equal(out[-64:], both) and one.any()
    dy, dg = moe.combine_bwd(z, ro, torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda"),
                             torch.ones((T, 1), device="cuda"))
    assert torch.equal(dy[0], z[-1]) and torch.equal(dy[-1], z[0])
    alone = (z[-1].double() * ro[0].double())
    assert abs(dg[-1, 0].item() - alone.sum().item()) <= N * 2.0 ** -23 * alone.abs().sum().item()
