"""The operators of a cache under a budget as they are measured: the attention
of whole prompts, the attention weight that cached tokens gather (from a
prompt, and from the nodes that a round keeps), and the eviction of the tokens
that gathered least.

Prompts are packed: T token rows, sequence b holds rows starts[b] ..
starts[b+1]-1.  The cache: pages of P tokens; K pages [pages][Hkv][P][D], V
pages [pages][Hkv][D][P], in e4m3 (largest value 448) or int8 (127); one scale
per page and head, the smallest power of two that brings the page's largest
magnitude into the format's range.  Weights: [B][Hkv][C], the sum over queries
and over a head's query heads of e^(score - lse), by cached position.
"""
import math

import torch

own = False

_QMAX = {"e4m3": 448.0, "int8": 127.0}
_CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
_TYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases --
def listed():
    return [
        # one short prompt: launch latency
        dict(name="prompt_1x45", op="prompt", B=1, Hq=32, Hkv=8, D=128, lo=45, hi=45, dtype="bf16"),
        # the prompts of one step of a busy server, packed
        dict(name="prompt_48_ragged", op="prompt", B=48, Hq=32, Hkv=8, D=128, lo=1, hi=1500, dtype="bf16"),
        # one long document
        dict(name="prompt_1x16384", op="prompt", B=1, Hq=32, Hkv=8, D=128, lo=16384, hi=16384, dtype="bf16"),
        # a small model kept in 32 bits, one key head per query head, heads of 64
        dict(name="prompt_f32_16x600", op="prompt", B=16, Hq=16, Hkv=16, D=64, lo=3, hi=600, dtype="f32"),
        # heads of 256, few key heads
        dict(name="prompt_d256_6x2047", op="prompt", B=6, Hq=16, Hkv=2, D=256, lo=33, hi=2047, dtype="bf16"),
        # the weights that the packed prompts give their own tokens
        dict(name="sums_48_ragged", op="sums", B=48, Hq=32, Hkv=8, D=128, lo=1, hi=1500, dtype="bf16"),
        # two long prompts' weights
        dict(name="sums_2x8191", op="sums", B=2, Hq=32, Hkv=8, D=128, lo=8000, hi=8191, dtype="bf16"),
        # plain decoding of 64 requests: one token each adds its weights
        dict(name="nodes_64x1", op="nodes", B=64, N=1, Hq=32, Hkv=8, D=128, P=32, lo=301, hi=2111, fmt="e4m3",
             dtype="bf16", path=False),
        # the accepted paths of 256 trees of 32 nodes
        dict(name="nodes_path_256x32", op="nodes", B=256, N=32, Hq=32, Hkv=8, D=128, P=64, lo=97, hi=2500, fmt="int8",
             dtype="bf16", path=True),
        # four requests brought back to a small budget
        dict(name="evict_4x700", op="evict", B=4, Hkv=8, D=128, P=16, lo=400, hi=700, budget=512, recent=64,
             limit=512, fmt="e4m3"),
        # a full batch cut to a quarter of its largest length; those at the budget stay
        dict(name="evict_64x4096", op="evict", B=64, Hkv=8, D=128, P=64, lo=900, hi=4096, budget=1024, recent=128,
             limit=1024, fmt="e4m3"),
        # two very long contexts cut to a sixteenth
        dict(name="evict_long_2x131072", op="evict", B=2, Hkv=8, D=128, P=128, lo=100003, hi=131072, budget=8192,
             recent=1000, limit=8192, fmt="int8"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "sums", "nodes", "evict"])
    c = dict(op=op, Hkv=rng.choice([1, 2, 4, 8, 16]), D=rng.choice([64, 96, 128, 256]))
    row = c["Hkv"] * c["D"]
    if op in ("prompt", "sums"):
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 7, 8])
        most = 4e11 if op == "prompt" else 1e11  # scores times channels, of padded squares
        top = int(math.sqrt(most / (c["Hq"] * c["D"])))
        c["hi"] = _log_int(rng, 1, max(1, min(9000, top)))
        c["B"] = _log_int(rng, 1, max(1, min(200, int(most / (c["Hq"] * c["D"])) // c["hi"] ** 2, 40000 // c["hi"])))
        c["lo"] = rng.randint(1, c["hi"]) if rng.random() < 0.8 else 0
    elif op == "nodes":
        c.update(P=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]),
                 dtype=rng.choice(["bf16", "bf16", "f32"]), path=rng.random() < 0.6, N=_log_int(rng, 1, 64))
        c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 7, 8])
        tokens = min(600000, int(4e10 / (4.0 * c["N"] * c["Hq"] * c["D"])), int(5e8 / row))
        c["hi"] = _log_int(rng, 16, max(17, min(60000, tokens)))
        c["B"] = _log_int(rng, 1, max(1, min(256, tokens // c["hi"])))
        c["lo"] = rng.randint(0, c["hi"])
    else:
        c.update(P=rng.choice([16, 32, 64, 128]), fmt=rng.choice(["e4m3", "int8"]))
        tokens = min(250000, int(2.5e8 / row))
        c["hi"] = _log_int(rng, 16, max(17, min(60000, tokens)))
        c["B"] = _log_int(rng, 1, max(1, min(128, tokens // c["hi"])))
        c["lo"] = rng.randint(0, c["hi"])
        c["budget"] = max(1, min(c["hi"], _log_int(rng, max(1, c["hi"] // 32), c["hi"])))
        c["recent"] = rng.randint(0, c["budget"])
        c["limit"] = c["budget"] if rng.random() < 0.6 else min(c["hi"], c["budget"] + rng.randint(0, 64))
    return c


def _lengths(c):
    """Tokens per sequence: spread over [lo, hi] by the index alone."""
    span = c["hi"] - c["lo"] + 1
    return [c["lo"] + (b * 7919 + 13 * b * b + span // 2) % span for b in range(c["B"])]


def _counts(c):
    """Nodes that each sequence keeps: all N, or an accepted path of 1..8."""
    if not c["path"]:
        return [c["N"]] * c["B"]
    return [1 + (b * 5 + b // 3) % min(8, c["N"]) for b in range(c["B"])]


def work(case):
    c = case
    lens = _lengths(c)
    if c["op"] in ("prompt", "sums"):
        e, tok = 2 if c["dtype"] == "bf16" else 4, sum(lens)
        pairs = c["Hq"] * sum(x * (x + 1) / 2 for x in lens)
        if c["op"] == "prompt":
            return {"bytes": tok * c["D"] * e * 2 * (c["Hq"] + c["Hkv"]) + 4 * tok * c["Hq"], "flops": 4 * c["D"] * pairs}
        return {"bytes": tok * c["D"] * e * (c["Hq"] + c["Hkv"]) + 4 * tok * c["Hq"] + 4 * c["B"] * c["Hkv"] * c["hi"],
                "flops": 2 * c["D"] * pairs}
    if c["op"] == "nodes":
        e, cnt = 2 if c["dtype"] == "bf16" else 4, _counts(c)
        row, pages = c["Hkv"] * c["D"], sum((x + c["P"] - 1) // c["P"] for x in lens)
        nbytes = row * sum(lens) + pages * (4 + 4 * c["Hkv"]) + 8 * c["Hkv"] * sum(lens) + 4 * c["Hkv"] * sum(cnt)
        nbytes += sum(cnt) * (c["Hq"] * (c["D"] * e + 4) + row * e)
        seen = sum(n * (x + (n + 1) / 2) for x, n in zip(lens, cnt))
        return {"bytes": nbytes, "flops": 2 * c["Hq"] * c["D"] * seen}
    cut = [x for x in lens if x > c["limit"]]
    pages = len(cut) * ((c["budget"] + c["P"] - 1) // c["P"])
    # weights read, kept codes read and written, their scales, the kept positions, all weights out, the table
    nbytes = 4 * c["Hkv"] * sum(lens) + 4 * c["Hkv"] * c["D"] * c["budget"] * len(cut) + 8 * c["Hkv"] * pages
    nbytes += 4 * c["B"] * c["Hkv"] * (c["budget"] + _width(c) * c["P"]) + 8 * c["B"] * _width(c)
    return {"bytes": nbytes, "flops": 2 * c["Hkv"] * c["D"] * c["budget"] * len(cut)}


def _width(c):
    """Columns of the page table."""
    return max(1, (c["hi"] + c.get("N", 0) + c["P"] - 1) // c["P"])


# ------------------------------------------------------------- prepare --
def _pow2_scale(amax, fmt):
    """The smallest power of two s with amax <= largest * s (2^-126 at least)."""
    m, e = torch.frexp(amax)
    top, bits = (0.875, 9) if fmt == "e4m3" else (0.9921875, 7)
    k = e - bits + (m > top).int()
    k = torch.where(amax > 0, k, torch.full_like(k, -126)).clamp(-126, 127)
    return ((k.int() + 127) << 23).view(torch.float32)


def _encode(y, fmt):
    """Values in units of the scale to codes: round to nearest, ties to even."""
    y = y.clamp(-_QMAX[fmt], _QMAX[fmt])
    return y.to(torch.float8_e4m3fn) if fmt == "e4m3" else y.round().to(torch.int8)


def _tokens(g, shape, dtype, dev):
    """Keys or values: normal, with some channels several times larger."""
    x = torch.randn(shape, generator=g, device=dev)
    x *= 1.0 + 5.0 * (torch.rand(shape[-2:], generator=g, device=dev) > 0.95)
    return x.to(dtype)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    lens = _lengths(c)
    st = {"case": c}
    if c["op"] in ("prompt", "sums"):
        dtype, T = _TYPE[c["dtype"]], max(1, sum(lens))
        ends = torch.tensor([0] + lens).cumsum(0)
        st["starts"] = ends.int().to(dev)
        # one fused projection's rows: q, k and v are slices of it
        qkv = torch.empty((T, (c["Hq"] + 2 * c["Hkv"]), c["D"]), dtype=dtype, device=dev)
        qkv[:, :c["Hq"]] = torch.randn((T, c["Hq"], c["D"]), generator=g, device=dev).to(dtype)
        qkv[:, c["Hq"]:] = _tokens(g, (T, 2 * c["Hkv"], c["D"]), dtype, dev)
        st["q"], st["k"], st["v"] = qkv.split((c["Hq"], c["Hkv"], c["Hkv"]), 1)
        # where each packed row stands in [B, hi]
        st["seq"] = torch.repeat_interleave(torch.arange(c["B"]), torch.tensor(lens)).to(dev)
        st["at"] = torch.arange(sum(lens), device=dev) - st["starts"][st["seq"]]
        if c["op"] == "sums":
            st["lse"] = torch.full((T, c["Hq"]), -math.inf, device=dev)
            for b in range(c["B"]):
                for i in range(0, lens[b], 2048):
                    rows = slice(int(ends[b]) + i, int(ends[b]) + min(lens[b], i + 2048))
                    st["lse"][rows] = _lse_rows(st["q"][rows], st["k"][int(ends[b]):rows.stop], i)
        return st
    B, Hkv, D, P, fmt, N = c["B"], c["Hkv"], c["D"], c["P"], c["fmt"], c.get("N", 0)
    need, width = [(x + N + P - 1) // P for x in lens], _width(c)
    total = max(1, sum(need))
    perm = torch.randperm(total, generator=g, device=dev).int()
    ids = torch.arange(width, device=dev)
    table = torch.full((B, width), -1, dtype=torch.int32, device=dev)
    table[ids[None, :] < torch.tensor(need, device=dev)[:, None]] = perm[: sum(need)]
    st["table"], st["lengths"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    st["first"] = total
    if c["op"] == "evict":  # pages for what is kept: the pool's last ones, in any order
        new = (c["budget"] + P - 1) // P
        st["new_pages"] = (total + torch.randperm(B * new, generator=g, device=dev)).int().view(B, new)
        total += B * new
    for name in ("k", "v"):
        pages = torch.zeros((total, Hkv, P, D), dtype=_CODE[fmt], device=dev)
        scales = torch.zeros((total, Hkv), dtype=torch.float32, device=dev)
        step = max(1, (1 << 27) // (Hkv * P * D))
        for i in range(0, st["first"], step):
            n = min(step, st["first"] - i)
            x = _tokens(g, (n, P, Hkv, D), torch.float32, dev).transpose(1, 2)
            s = _pow2_scale(x.abs().amax((2, 3)), fmt)
            scales[i:i + n] = s
            pages[i:i + n] = _encode(x / s[:, :, None, None], fmt)
        if name == "v":
            pages = pages.view(torch.uint8).transpose(2, 3).contiguous().view(_CODE[fmt])
        st[name + "_pages"], st[name + "_scales"] = pages, scales
    # what positions gathered so far: few of them most of it, some exactly nothing
    C = width * P
    w = torch.rand((B, Hkv, C), generator=g, device=dev)
    w = (torch.exp(3.0 * torch.randn((B, Hkv, C), generator=g, device=dev)) * (w > 0.02)).float()
    st["weights"] = w.masked_fill(torch.arange(C, device=dev) >= st["lengths"][:, None, None], 0.0)
    if c["op"] == "nodes":
        dtype, cnt = _TYPE[c["dtype"]], torch.tensor(_counts(c), dtype=torch.int32, device=dev)
        st["q"] = torch.randn((B, N, c["Hq"], D), generator=g, device=dev).to(dtype)
        st["k"] = _tokens(g, (B, N, Hkv, D), dtype, dev)
        st["out"] = torch.zeros_like(st["weights"])
        order = torch.rand((B, N), generator=g, device=dev)
        order[:, 0] = -1.0
        keep = order.argsort(1).argsort(1) < cnt[:, None]
        idx = torch.where(keep, torch.arange(N, device=dev), N).sort(1).values
        path = torch.where(idx < N, idx, -1).int()  # increasing node indices from the root, then -1
        st["path"] = path if c["path"] else None
        lses = torch.full((B, N + 1, c["Hq"]), math.inf, device=dev)
        step = max(1, (1 << 29) // (C * Hkv * D))
        for i in range(0, B, step):
            j = slice(i, min(B, i + step))
            old, new, _ = _node_scores(st, j, path)
            old.masked_fill_((torch.arange(C, device=dev) >= st["lengths"][j, None])[:, None, None, None], -math.inf)
            lse = torch.logaddexp(torch.logsumexp(old, 4), torch.logsumexp(new, 4))  # [n, Hkv, G, M]
            lse = lse.permute(0, 3, 1, 2).reshape(lse.shape[0], -1, c["Hq"])
            at = path[j, :lse.shape[1], None].long()
            lses[j].scatter_(1, torch.where(at < 0, N, at).expand_as(lse), lse)
        st["lse"] = lses[:, :N].contiguous()
    if own:
        import speculative_sampling_verify_spec_amd as sv
        st["cache"] = sv.KVCache(st["k_pages"], st["v_pages"], st["k_scales"], st["v_scales"])
    return st


def _lse_rows(q, k, first):
    """lse of the queries at positions first .. of one sequence with keys k."""
    n, Hq, D = q.shape
    Hkv = k.shape[1]
    q = q.float().view(n, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    s = torch.matmul(q, k.float().permute(1, 2, 0)).view(Hq, n, -1) / math.sqrt(D)
    s.masked_fill_(torch.ones(s.shape[1:], dtype=torch.bool, device=q.device).triu(first + 1), -math.inf)
    return torch.logsumexp(s, 2).t()


# ----------------------------------------------------------------- run --
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    import speculative_sampling_verify_spec_amd as sv
    c = st["case"]
    if c["op"] == "prompt":
        return sv.prompt_attention(st["q"], st["k"], st["v"], st["starts"], return_lse=True)
    if c["op"] == "sums":
        return sv.prompt_weights(st["q"], st["k"], st["lse"], st["starts"], max(1, c["hi"]))
    if c["op"] == "nodes":
        return sv.kv_weights(st["cache"], st["table"], st["q"], st["lse"], st["lengths"], st["weights"], st["k"],
                             index=st["path"], out=st["out"])
    got = sv.kv_evict(st["cache"], st["table"], st["lengths"], st["weights"], st["new_pages"], c["budget"],
                      c["recent"], limit=c["limit"], return_kept=True)
    return got + _moved(st)


def _moved(st):
    """What the new pages hold: codes, which are values in units of the scales beside them."""
    return tuple(st[n][st["first"]:] for n in ("k_pages", "k_scales", "v_pages", "v_scales"))


def _run_plain(st):
    return {"prompt": _plain_prompt, "sums": _plain_sums, "nodes": _plain_nodes, "evict": _plain_evict}[st["case"]["op"]](st)


def _padded(st, name):
    """Packed rows as [B, hi, heads, D] in 32 bits, 0 behind each sequence."""
    c, x = st["case"], st[name]
    out = torch.zeros((c["B"], c["hi"]) + x.shape[1:], device="cuda")
    out[st["seq"], st["at"]] = x[: st["seq"].shape[0]].float()
    return out


def _padded_scores(st):
    """Scores [B, Hkv, G * hi, hi], -inf where a query does not see."""
    c = st["case"]
    B, L, Hkv, G, D = c["B"], c["hi"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    q = _padded(st, "q").view(B, L, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * L, D)
    s = torch.matmul(q, _padded(st, "k").permute(0, 2, 3, 1)).mul_(1.0 / math.sqrt(D))
    s.view(B, Hkv, G, L, L).masked_fill_(torch.ones((L, L), dtype=torch.bool, device="cuda").triu(1), -math.inf)
    return s


def _plain_prompt(st):
    c = st["case"]
    B, L, Hkv, G, D, T = c["B"], c["hi"], c["Hkv"], c["Hq"] // c["Hkv"], c["D"], st["q"].shape[0]
    s = _padded_scores(st)
    m = s.amax(3, keepdim=True)
    s.sub_(m).exp_()
    z = s.sum(3, keepdim=True)
    o = torch.matmul(s, _padded(st, "v").transpose(1, 2)) / z
    o = o.view(B, Hkv, G, L, D).permute(0, 3, 1, 2, 4).reshape(B, L, c["Hq"], D)
    lse = (m + torch.log(z)).view(B, Hkv, G, L).permute(0, 3, 1, 2).reshape(B, L, c["Hq"])
    out = torch.zeros((T, c["Hq"], D), dtype=_TYPE[c["dtype"]], device="cuda")
    stat = torch.full((T, c["Hq"]), -math.inf, device="cuda")
    out[: st["seq"].shape[0]] = o[st["seq"], st["at"]].to(out.dtype)
    stat[: st["seq"].shape[0]] = lse[st["seq"], st["at"]]
    return out, stat


def _plain_sums(st):
    c = st["case"]
    B, L, Hkv, G = c["B"], c["hi"], c["Hkv"], c["Hq"] // c["Hkv"]
    lse = torch.full((B, L, c["Hq"]), math.inf, device="cuda")  # rows behind a sequence weigh nothing
    lse[st["seq"], st["at"]] = st["lse"][: st["seq"].shape[0]]
    s = _padded_scores(st)
    s.sub_(lse.view(B, L, Hkv, G).permute(0, 2, 3, 1).reshape(B, Hkv, G * L, 1)).exp_()
    return s.sum(2)


def _plain_blocks(st, name, table):
    """Blocks of the table as float values [B, n, Hkv, P, D], 0 for no page."""
    pages, scales = st[name + "_pages"], st[name + "_scales"]
    ok = (table >= 0) & (table < pages.shape[0])
    t = torch.where(ok, table, 0).long()
    x = pages.view(torch.uint8)[t].view(pages.dtype).float()
    if name == "v":
        x = x.transpose(3, 4)
    return (x * scales[t][:, :, :, None, None]).masked_fill(~ok[:, :, None, None, None], 0.0)


def _node_scores(st, j, path):
    """Scores of the nodes of a path over cached tokens [n, Hkv, G, M, C] and
    over the path itself [n, Hkv, G, M, M], of the sequences j; which nodes exist."""
    c = st["case"]
    B, Hkv, G, D = j.stop - j.start, c["Hkv"], c["Hq"] // c["Hkv"], c["D"]
    M = min(c["N"], max(_counts(c)))
    p = path[j, :M].long()
    pick = lambda x: x[j].gather(1, p.clamp(min=0)[:, :, None, None].expand(-1, -1, x.shape[2], D)).float()  # noqa: E731
    q = pick(st["q"]).view(B, M, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, D) / math.sqrt(D)
    k = _plain_blocks(st, "k", st["table"][j]).transpose(1, 2).reshape(B, Hkv, -1, D)
    old = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, M, -1)
    new = torch.matmul(q, pick(st["k"]).permute(0, 2, 3, 1)).view(B, Hkv, G, M, M)
    new = new.masked_fill(torch.ones((M, M), dtype=torch.bool, device="cuda").triu(1), -math.inf)
    return old, new, p >= 0


def _plain_nodes(st):
    c = st["case"]
    B, C = c["B"], st["weights"].shape[2]
    path = torch.arange(c["N"], device="cuda").expand(B, -1) if st["path"] is None else st["path"]
    out, at = st["out"], torch.arange(C, device="cuda")
    M = min(c["N"], max(_counts(c)))
    step = max(1, (1 << 30) // (C * c["Hkv"] * max(c["D"], M * c["Hq"] // c["Hkv"])))
    for i in range(0, B, step):
        j = slice(i, min(B, i + step))
        old, new, there = _node_scores(st, j, path)
        n = there.shape[0]
        lse = st["lse"][j].gather(1, path[j, :M, None].long().clamp(min=0).expand(-1, -1, c["Hq"]))
        lse = torch.where(there[..., None], lse, math.inf).view(n, M, c["Hkv"], -1).permute(0, 2, 3, 1)[..., None]
        old = torch.exp(old.sub_(lse)).sum((2, 3))
        new = torch.exp(new - lse).sum((2, 3))
        length = st["lengths"][j, None, None]
        rel = (at - length).expand(n, c["Hkv"], C)
        x = torch.where(rel < 0, st["weights"][j] + old, new.gather(2, rel.clamp(0, M - 1)))
        out[j] = torch.where(rel < there.sum(1)[:, None, None], x, out[j])
    return out


def _plain_evict(st):
    c = st["case"]
    B, Hkv, D, P, fmt, n_keep = c["B"], c["Hkv"], c["D"], c["P"], c["fmt"], c["budget"]
    w, length = st["weights"], st["lengths"].long()
    C = w.shape[2]
    at = torch.arange(C, device="cuda")
    cut = length > c["limit"]
    gone = at >= length[:, None, None]
    key = w.masked_fill(at >= (length - c["recent"])[:, None, None], math.inf).masked_fill(gone, -math.inf)
    kept = torch.sort(key, dim=2, descending=True, stable=True).indices[..., :n_keep].sort(2).values
    kept_w = torch.nn.functional.pad(w.gather(2, kept), (0, C - n_keep))
    out_w = torch.where(cut[:, None, None], kept_w, w.masked_fill(gone, 0.0))
    kept = torch.where(cut[:, None, None], kept, -1)
    new, width = st["new_pages"], st["table"].shape[1]
    table = torch.where(cut[:, None], torch.nn.functional.pad(new, (0, width - new.shape[1]), value=-1), st["table"])
    # the kept tokens of the sequences that are cut, in pages: [n, Hkv, new pages, P]
    rows = cut.nonzero()[:, 0]
    pos = torch.nn.functional.pad(kept[rows], (0, new.shape[1] * P - n_keep), value=-1).view(len(rows), Hkv, -1, P)
    there = pos >= 0
    pos = pos.clamp(min=0)
    src = st["table"].long()[rows[:, None, None, None], pos // P].clamp(min=0)
    head, dst = torch.arange(Hkv, device="cuda")[None, :, None, None], new[rows].long()
    for name in ("k", "v"):
        pages, scales = st[name + "_pages"], st[name + "_scales"]
        raw = pages.view(torch.uint8).transpose(2, 3) if name == "v" else pages.view(torch.uint8)
        x = raw[src, head, pos % P].view(pages.dtype).float() * scales[src, head][..., None]
        x = x.masked_fill(~there[..., None], 0.0)
        s = _pow2_scale(x.abs().amax((3, 4)), fmt)                       # [n, Hkv, new pages]
        code = _encode(x / s[..., None, None], fmt).view(torch.uint8).transpose(1, 2)
        raw[dst] = torch.where(there.transpose(1, 2)[..., None], code, raw[dst])
        scales[dst] = s.transpose(1, 2)
    lengths = torch.where(cut, n_keep, length).int()
    return (table, lengths, out_w, kept.int()) + _moved(st)


# --------------------------------------------------------------- exact --
def _two_to(k):
    """2^k in 64 bits, exactly."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _decode64(pages, fmt):
    """Codes as 64-bit values, from the format's bits."""
    u = pages.view(torch.uint8).long()
    if fmt == "int8":
        return torch.where(u > 127, u - 256, u).double()
    mant, expo = (u & 7).double(), (u >> 3) & 15
    mag = torch.where(expo > 0, (8.0 + mant) * _two_to(expo - 10), mant * 2.0 ** -9)
    return torch.where(u > 127, -mag, mag)


def _round64(y, fmt):
    """The format's nearest value, ties to even, of 64-bit values."""
    if fmt == "int8":
        return torch.round(y).clamp(-127.0, 127.0)
    _, e = torch.frexp(y)  # |y| in [2^(e-1), 2^e)
    unit = _two_to((e - 1).clamp(min=-6) - 3)
    return (torch.round(y / unit) * unit).clamp(-448.0, 448.0)


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    lens = _lengths(c)
    if c["op"] in ("prompt", "sums"):
        return _exact_packed(st, lens)
    table = st["table"].cpu().tolist()

    def cached(name, b, h, n):
        """Positions 0..n-1 of one head of sequence b: [n, D]."""
        ids = torch.tensor(table[b][:(n + c["P"] - 1) // c["P"]], device="cuda", dtype=torch.long)
        x = _decode64(st[name + "_pages"].view(torch.uint8)[ids, h], c["fmt"])
        x = (x if name == "k" else x.transpose(1, 2)) * st[name + "_scales"][ids, h].double()[:, None, None]
        return x.reshape(-1, c["D"])[:n]

    if c["op"] == "nodes":
        G, counts = c["Hq"] // c["Hkv"], _counts(c)
        out = torch.zeros(st["weights"].shape, dtype=torch.float64, device="cuda")
        for b in range(c["B"]):
            n, L = counts[b], lens[b]
            p = st["path"][b, :n].long() if c["path"] else torch.arange(n, device="cuda")
            later = torch.ones((n, n), dtype=torch.bool, device="cuda").tril()  # node i sees j <= i
            for h in range(c["Hkv"]):
                k = torch.cat((cached("k", b, h, L), st["k"][b, p, h].double()))
                for hq in range(h * G, h * G + G):
                    s = (st["q"][b, p, hq].double() @ k.t().contiguous()) * c["D"] ** -0.5 - st["lse"][b, p, hq].double()[:, None]
                    e = torch.exp(s)
                    out[b, h, :L] += e[:, :L].sum(0)
                    out[b, h, L:L + n] += (e[:, L:] * later).sum(0)
            out[b, :, :L] += st["weights"][b, :, :L].double()
        return out

    B, Hkv, D, P, fmt, keep = c["B"], c["Hkv"], c["D"], c["P"], c["fmt"], c["budget"]
    C, W = st["weights"].shape[2], st["table"].shape[1]
    out_w = torch.zeros((B, Hkv, C), dtype=torch.float64, device="cuda")
    kept = torch.full((B, Hkv, keep), -1, dtype=torch.int32, device="cuda")
    out_table = [list(r) for r in table]
    dst = st["new_pages"].cpu().tolist()
    after = [keep if x > c["limit"] else x for x in lens]
    n_new = st["k_pages"].shape[0] - st["first"]
    code = {n: torch.zeros((n_new, Hkv, P, D), dtype=torch.float64, device="cuda") for n in "kv"}
    scale = {n: torch.zeros((n_new, Hkv), dtype=torch.float64, device="cuda") for n in "kv"}
    for b in range(B):
        L = lens[b]
        if L <= c["limit"]:
            out_w[b, :, :L] = st["weights"][b, :, :L].double()
            continue
        out_table[b] = dst[b] + [-1] * (W - len(dst[b]))
        old = max(0, L - c["recent"])
        for h in range(Hkv):
            w = st["weights"][b, h, :L].double()
            # rank by weight, ties by position: the number of heavier ones and of earlier equal ones
            order = torch.sort(-w[:old], stable=True).indices[:keep - (L - old)]
            at = torch.cat((torch.sort(order).values, torch.arange(old, L, device="cuda")))
            kept[b, h], out_w[b, h, :keep] = at.int(), w[at]
            for n in "kv":
                x = cached(n, b, h, L)[at]
                x = torch.cat((x, torch.zeros((-keep % P, D), dtype=torch.float64, device="cuda"))).view(-1, P, D)
                top = x.abs().amax((1, 2))
                _, e = torch.frexp(top / _QMAX[fmt])   # top <= largest * 2^e
                tight = _two_to(e - 1)
                fit = torch.where(top <= tight * _QMAX[fmt], tight, tight * 2.0)
                s = torch.where(top > 0, fit.clamp(min=2.0 ** -126), torch.full_like(fit, 2.0 ** -126))
                ids = torch.tensor(dst[b], device="cuda") - st["first"]
                code[n][ids, h], scale[n][ids, h] = _round64(x / s[:, None, None], fmt), s
    code["v"] = code["v"].transpose(2, 3).contiguous()
    if fmt == "int8":
        code = {n: x.to(torch.int8) for n, x in code.items()}
    return (torch.tensor(out_table, dtype=torch.int32, device="cuda"),
            torch.tensor(after, dtype=torch.int32, device="cuda"), out_w, kept, code["k"], scale["k"], code["v"], scale["v"])


def _exact_packed(st, lens):
    c = st["case"]
    Hq, D, G, T = c["Hq"], c["D"], c["Hq"] // c["Hkv"], st["q"].shape[0]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    sums = torch.zeros((c["B"], c["Hkv"], c["hi"]), dtype=torch.float64, device="cuda")
    first = 0
    for b, L in enumerate(lens):
        for hq in range(Hq):
            k = st["k"][first:first + L, hq // G].double()
            v = st["v"][first:first + L, hq // G].double()
            for i in range(0, L, 4096):
                n = min(4096, L - i)
                rows = slice(first + i, first + i + n)
                s = st["q"][rows, hq].double() @ k[:i + n].t().contiguous() * D ** -0.5
                s[:, i:].masked_fill_(torch.ones((n, n), dtype=torch.bool, device="cuda").triu(1), -math.inf)
                if c["op"] == "sums":
                    sums[b, hq // G, :i + n] += torch.exp(s - st["lse"][rows, hq].double()[:, None]).sum(0)
                    continue
                z = torch.logsumexp(s, 1)
                lse[rows, hq] = z
                out[rows, hq] = torch.exp(s - z[:, None]) @ v[:i + n]
        first += L
    return sums if c["op"] == "sums" else (out, lse)
