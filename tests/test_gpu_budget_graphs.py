"""Whole prompts and the cache under a budget as programs run them: captured
into graphs, on two streams at once, over memory past 32 bits, and with the
arguments that the binding refuses."""
import numpy as np
import pytest

import kv_helpers as kh
import prompt_helpers as ph
from oracle import budget as ob
from oracle import kv as okv
from oracle import prompt as op

pytestmark = pytest.mark.gpu


def _i32(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _setup(gpu_lib, seed, lens=(150, 20000, 40), dtype="bf16", D=64, H=2, G=2, P=64, N=5, budget=96):
    """A cache of long and short sequences, prompts, nodes and new pages; and a
    step over them that gives its results in new tensors."""
    import torch
    rng = np.random.default_rng(seed)
    B, dt = len(lens), torch.bfloat16 if dtype == "bf16" else torch.float32
    c, table = kh.make_cache(rng, "e4m3", list(lens), P, H, D, extra=N, spare=B * -(-budget // P))
    used = {int(x) for b, n in enumerate(lens) for x in table[b, :-(-(n + N) // P)]}
    free = [p for p in range(c["k_pages"].shape[0]) if p not in used][:B * -(-budget // P)]
    starts = np.array([0, 130, 130, 333])
    (q, k, v), _ = ph.inputs(rng, 340, H * G, H, D, dtype)
    x = torch.from_numpy(rng.normal(size=(B, N, H * G + 2 * H, D)).astype(np.float32)).to(dt).cuda()
    qn, kn, vn = x.split((H * G, H, H), 2)
    tab, ln, pages, st = _i32(table), _i32(lens), _i32(np.reshape(free, (B, -1))), _i32(starts)
    index = _i32([[0, 2, -1, 0, 0]] * B)
    weights = torch.from_numpy(rng.random((B, H, table.shape[1] * P)).astype(np.float32)).cuda()
    dev = kh.to_device(gpu_lib, c)
    size = gpu_lib.kv_evict_workspace_size(dev, B, table.shape[1])
    assert size > 256  # rows that several workgroups share

    def step(ws):
        out, lse = gpu_lib.prompt_attention(q, k, v, st, return_lse=True)
        gathered = gpu_lib.prompt_weights(q, k, lse, st, 400)
        _, node_lse = gpu_lib.kv_attention(dev, tab, qn, ln, kn, vn, return_lse=True)
        added = torch.full_like(weights, 3.0)
        gpu_lib.kv_weights(dev, tab, qn, node_lse, ln, weights, kn, index=index, out=added)
        after = gpu_lib.kv_append(dev, tab, kn, vn, ln, index=index)
        cut = gpu_lib.kv_evict(dev, tab, after, added, pages, budget, 16, return_kept=True, workspace=ws)
        return (out, lse, gathered, node_lse, added, after) + cut + gpu_lib.kv_read(dev, cut[0], cut[1], budget)

    return step, size, (q, k, v, st)


def test_graph_of_all_calls_replayed(gpu_lib):
    """One graph of every call, replayed between eager work: each replay gives the eager bits."""
    import torch
    step, size, _ = _setup(gpu_lib, 1)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    step(ws)  # the append rounds begun blocks again; from here on the same call changes nothing
    want = [t.clone() for t in step(ws)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(ws)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(ws)
    for _ in range(4):
        for t in outs:
            t.fill_(1)
        ws.fill_(0xff)
        graph.replay()
        eager = step(torch.empty_like(ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, want))


def test_two_graphs_with_their_own_workspaces(gpu_lib):
    """Captured calls that allocate their workspaces, two graphs replayed in turn."""
    import torch
    steps = [_setup(gpu_lib, seed)[0] for seed in (2, 3)]
    want, graphs, outs = [], [], []
    for step in steps:
        step(None)
        want.append([t.clone() for t in step(None)])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(None))
        graphs.append(g)
    for _ in range(3):
        for step, g, o, w in zip(steps, graphs, outs, want):
            for t in o:
                t.fill_(1)
            g.replay()
            assert all(torch.equal(a, b) for a, b in zip(step(None), w))
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_two_streams_at_once(gpu_lib):
    """Steps in flight together on two streams, over caches and workspaces of their own."""
    import torch
    sets = [_setup(gpu_lib, seed) for seed in (4, 5)]
    steps, sizes = [s[0] for s in sets], [s[1] for s in sets]
    want, spaces = [], [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    for step, ws in zip(steps, spaces):
        step(ws)
        want.append([t.clone() for t in step(ws)])
    streams = [torch.cuda.Stream() for _ in steps]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(steps[i](spaces[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_the_same_node_twice(gpu_lib):
    """A path that names a node more than once adds it each time, in its order."""
    import torch
    rng = np.random.default_rng(6)
    lens, P, H, D, N = [90, 33], 32, 1, 64, 4
    c, table = kh.make_cache(rng, "int8", lens, P, H, D, extra=N)
    q, _, lse_in = rng.normal(size=(2, N, 2, D)), None, np.abs(rng.normal(size=(2, N, 2)) + 4).astype(np.float32)
    q = torch.from_numpy(q.astype(np.float32)).bfloat16().cuda()
    w = rng.random((2, H, table.shape[1] * P)).astype(np.float32)
    index = np.array([[1, 1, 3, 1], [2, 2, -1, 0]])
    got = gpu_lib.kv_weights(kh.to_device(gpu_lib, c), _i32(table), q, torch.from_numpy(lse_in).cuda(), _i32(lens),
                             torch.from_numpy(w).cuda(), index=_i32(index))
    want, written = ob.kv_weights(c, table, q.double().cpu().numpy(), lse_in.astype(np.float64), lens, w, D ** -0.5,
                                  None, None, index)
    x, big, mag, cnt = want
    tol = 1.01 * (ph.score_error(big, D) + 4 * ph.U * mag + (cnt + 8) * ph.U * np.abs(x)) + 1e-37
    rows = np.broadcast_to(written[:, None], w.shape)
    assert (np.abs(got.double().cpu().numpy() - x) <= tol)[rows].all()


def test_rows_past_32_bits(gpu_lib):
    """Token rows so far apart that elements and bytes pass 32 bits, and weights behind 2^31 floats."""
    import torch
    rng = np.random.default_rng(7)
    T, H, G, D, stride = 300, 1, 2, 64, 15_000_000
    big = torch.empty((T - 1) * stride + (H * G + 2 * H) * D, dtype=torch.bfloat16, device="cuda")
    (q, k, v), host = ph.inputs(rng, T, H * G, H, D, "bf16", fused=False)
    far = []
    for x, at in ((q, 0), (k, H * G * D), (v, (H * G + H) * D)):
        y = big.as_strided((T, x.shape[1], D), (stride, D, 1), at)
        y.copy_(x)
        far.append(y)
    starts = _i32([0, 3, 170, 300])
    near = gpu_lib.prompt_attention(q, k, v, starts, return_lse=True)
    got = gpu_lib.prompt_attention(*far, starts, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(got, near))
    want = op.attention(*host, [0, 3, 170, 300], D ** -0.5)
    tol, _ = ph.attention_bounds(*want, D, "bf16")
    assert (np.abs(near[0].double().cpu().numpy() - want[0]) <= tol).all()
    del want, tol
    near_w = gpu_lib.prompt_weights(q, k, near[1], starts, 200)
    capacity = 800_000_000
    far_w = gpu_lib.prompt_weights(far[0], far[1], got[1], starts, capacity)
    assert torch.equal(far_w[:, :, :200], near_w)
    for b in range(3):
        assert not far_w[b, 0, 200:].any()


def test_the_largest_capacity(gpu_lib):
    """Rows of 2^31 - 1 weights, of a sequence and of one without tokens, are cleared to their ends."""
    import torch
    rng = np.random.default_rng(11)
    (q, k, v), _ = ph.inputs(rng, 70, 2, 1, 64, "bf16")
    starts, capacity = _i32([0, 70, 70]), 2 ** 31 - 1
    _, lse = gpu_lib.prompt_attention(q, k, v, starts, return_lse=True)
    got = gpu_lib.prompt_weights(q, k, lse, starts, capacity)
    assert torch.equal(got[:, :, :90], gpu_lib.prompt_weights(q, k, lse, starts, 90))
    for b in range(2):
        for part in got[b, 0, 70:].split(1 << 29):
            assert not part.any()


def test_pools_and_weights_past_32_bits(gpu_lib):
    """Pages whose codes stand behind 2^32 bytes, and a row of weights behind
    2^31 floats: gathered, cut and read as a small cache with the same tokens."""
    import torch
    rng = np.random.default_rng(8)
    lens, P, H, D, N, budget = [300, 280], 128, 2, 256, 3, 130
    c, table = kh.make_cache(rng, "e4m3", lens, P, H, D, extra=N, spare=4)
    pages = c["k_pages"].shape[0]
    used = {int(x) for b, n in enumerate(lens) for x in table[b, :-(-(n + N) // P)]}
    new = np.array([p for p in range(pages) if p not in used][:4]).reshape(2, 2)
    small = kh.to_device(gpu_lib, c)
    lift = 70_000  # pages before them: 4.6e9 bytes
    parts = []
    for t in (small.k_pages, small.v_pages, small.k_scales, small.v_scales):
        x = torch.empty((lift + pages,) + t.shape[1:], dtype=t.dtype, device="cuda")
        x[lift:].view(torch.uint8).copy_(t.view(torch.uint8))
        parts.append(x)
    large = gpu_lib.KVCache(*parts)
    q = torch.from_numpy(rng.normal(size=(2, N, 2 * H, D)).astype(np.float32)).bfloat16().cuda()
    k = torch.from_numpy(rng.normal(size=(2, N, H, D)).astype(np.float32)).bfloat16().cuda()
    w = torch.from_numpy(rng.random((2, H, table.shape[1] * P)).astype(np.float32)).cuda()
    capacity = 600_000_000
    wide = torch.empty((2, H, capacity), dtype=torch.float32, device="cuda")
    wide[:, :, :w.shape[2]] = w
    wide[:, :, w.shape[2]:] = 9.0
    results = []
    for dev, weights, t, n in ((small, w, table, new), (large, wide, table + lift, new + lift)):
        tab = _i32(np.where(table < 0, -1, t))
        _, lse = gpu_lib.kv_attention(dev, tab, q, _i32(lens), k, torch.zeros_like(k), return_lse=True)
        gpu_lib.kv_weights(dev, tab, q, lse, _i32(lens), weights, k)
        got = gpu_lib.kv_evict(dev, tab, _i32(lens), weights, _i32(n), budget, 10, return_kept=True)
        results.append((weights[:, :, :w.shape[2]].clone(), lse, got[1], got[2][:, :, :w.shape[2]].clone(), got[3]) +
                       gpu_lib.kv_read(dev, got[0], got[1], budget))
        del got
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert (wide[1, 1, w.shape[2]:] == 9.0).all()


def test_forward_only(gpu_lib):
    """A backward pass through an attention of prompts is refused; weights carry no gradients."""
    rng = np.random.default_rng(9)
    (q, k, v), _ = ph.inputs(rng, 40, 4, 2, 64, "f32", fused=False)
    starts = _i32([0, 40])
    plain = gpu_lib.prompt_attention(q, k, v, starts)
    for t in (q, k, v):
        t.requires_grad_()
        out, lse = gpu_lib.prompt_attention(q, k, v, starts, return_lse=True)
        assert out.requires_grad and (out.detach() == plain).all()
        with pytest.raises(NotImplementedError, match="prompt_attention"):
            (out.sum() + lse.sum()).backward()
        assert not gpu_lib.prompt_weights(q, k, lse.detach(), starts, 40).requires_grad
        t.requires_grad_(False)


def test_refusals(gpu_lib):
    """Shapes, types, strides and devices that the binding names before any launch."""
    import torch
    rng = np.random.default_rng(10)
    (q, k, v), _ = ph.inputs(rng, 20, 4, 2, 64, "bf16", fused=False)
    starts, lse = _i32([0, 20]), torch.zeros(20, 4, device="cuda")
    bad = [dict(q=q[0]), dict(q=q.half()), dict(k=k[:19]), dict(k=k.float()), dict(k=k.cpu()), dict(v=v[:, :1]),
           dict(q=q[:, :3]), dict(starts=starts.long()), dict(starts=starts[:1]), dict(starts=starts.cpu()),
           dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)), dict(v=torch.stack((v, v), 1)[:, 0])]
    for kw in bad:
        a = dict(dict(q=q, k=k, v=v, starts=starts), **kw)
        with pytest.raises((ValueError, TypeError)):
            gpu_lib.prompt_attention(a["q"], a["k"], a["v"], a["starts"])
    for kw in bad[:-1] + [dict(lse=lse[:, :3]), dict(lse=lse.double()), dict(lse=lse.t().contiguous().t()), dict(capacity=0)]:
        if "v" in kw:
            continue
        a = dict(dict(q=q, k=k, starts=starts, lse=lse, capacity=20), **kw)
        with pytest.raises((ValueError, TypeError)):
            gpu_lib.prompt_weights(a["q"], a["k"], a["lse"], a["starts"], a["capacity"])
    with pytest.raises(gpu_lib.SpecVerifyError):
        gpu_lib.prompt_attention(q, k, v, starts, scale=float("nan"))

    c, table = kh.make_cache(rng, "int8", [20], 16, 2, 64)
    dev, tab, ln = kh.to_device(gpu_lib, c), _i32(table), _i32([20])
    x, s = q[None, :3].contiguous(), lse[None, :3].contiguous()
    w = torch.zeros(1, 2, table.shape[1] * 16, device="cuda")
    for kw in (dict(x=x[0]), dict(x=x[:, :, :, :32]), dict(s=s[:, :, :3]), dict(s=s.double()), dict(ln=ln.long()),
               dict(w=w[:, :, :-1]), dict(w=w.double()), dict(w=w[:, :1]), dict(w=w.clone().requires_grad_()),
               dict(index=_i32([[0]])), dict(counts=_i32([1, 1])), dict(out=w.cpu()), dict(k=x[:, :2, :2]),
               dict(k=x[:, :, :2].float())):
        a = dict(dict(x=x, s=s, ln=ln, w=w, index=None, counts=None, out=None, k=None), **kw)
        with pytest.raises((ValueError, TypeError)):
            gpu_lib.kv_weights(dev, tab, a["x"], a["s"], a["ln"], a["w"], a["k"], index=a["index"], counts=a["counts"],
                               out=a["out"])
    flat = torch.zeros(2 * w.numel(), device="cuda")
    with pytest.raises(gpu_lib.SpecVerifyError):  # a half of the other
        gpu_lib.kv_weights(dev, tab, x, s, ln, flat[:w.numel()].view(w.shape), out=flat[4:4 + w.numel()].view(w.shape))
    pages = _i32([[1]])
    for kw in (dict(budget=0), dict(budget=17), dict(recent=-1), dict(recent=17), dict(limit=15), dict(w=w[:, :, 1:]),
               dict(pages=pages.long()), dict(ln=ln.cpu())):
        a = dict(dict(ln=ln, w=w, pages=pages, budget=16, recent=4, limit=None), **kw)
        with pytest.raises((ValueError, TypeError)):
            gpu_lib.kv_evict(dev, tab, a["ln"], a["w"], a["pages"], a["budget"], a["recent"], limit=a["limit"])
    with pytest.raises(gpu_lib.SpecVerifyError):  # a workspace that is not aligned
        gpu_lib.kv_evict(dev, tab, ln, w, pages, 16, 4, workspace=torch.empty(600, dtype=torch.uint8, device="cuda")[8:])
