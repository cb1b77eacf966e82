"""More operators of serving over the paged latent cache, each as a case to run.

Four operators, of a step whose tokens are drafts and whose cache must not grow:

* ``window``: attention over pages in which a token sees the last ``window`` positions and the
  first ``sink`` ones;
* ``weights``: the attention weight that the rows of each page have got, over all query rows,
  added to what they had before;
* ``evict``: the pages that a request keeps, those of the most weight, and the blocks that this frees;
* ``verify``: how much of a draft the target's probabilities accept, and the token after it.

Rows are 576 wide (512 value columns, then 64), pages hold 64 rows. ``own`` false: plain torch
operations in 32 bits (64 for sums of probabilities). ``own`` true: the framework's calls.
"""
import math

import torch

own = False

DIM, NOPE, PAGE = 576, 512, 64
SCALE = 1.0 / math.sqrt(DIM)
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one request, one token, a short window: the call's latency
        {"name": "window_one", "op": "window", "dtype": "bf16", "B": 1, "T": 1, "H": 16, "ctx": 4096, "window": 512, "sink": 4, "tree": False},
        # a small draft's tree after a short, odd context
        {"name": "window_tree", "op": "window", "dtype": "bf16", "B": 3, "T": 7, "H": 16, "ctx": 1001, "window": 100, "sink": 5, "tree": True},
        # a batch of agents, three drafted tokens each, FP8 rows
        {"name": "window_step", "op": "window", "dtype": "fp8", "B": 32, "T": 4, "H": 128, "ctx": 74160, "window": 4096, "sink": 64, "tree": False},
        # a chunk of prompt of each of two requests
        {"name": "window_prompt", "op": "window", "dtype": "bf16", "B": 2, "T": 1999, "H": 16, "ctx": 8192, "window": 1024, "sink": 4, "tree": False},
        # one request, one token, a short context: the call's latency
        {"name": "weights_one", "op": "weights", "dtype": "bf16", "B": 1, "T": 1, "H": 16, "ctx": 4096},
        # what the last 16 tokens of each of four prompts looked at
        {"name": "weights_prompt", "op": "weights", "dtype": "bf16", "B": 4, "T": 16, "H": 16, "ctx": 74160},
        # a step with three drafted tokens, all heads, long contexts, FP8 rows
        {"name": "weights_step", "op": "weights", "dtype": "fp8", "B": 8, "T": 4, "H": 128, "ctx": 131072},
        # one short request
        {"name": "evict_one", "op": "evict", "B": 1, "ctx": 4096, "keep": 32},
        # requests of a million tokens, an eighth of which stays
        {"name": "evict_long", "op": "evict", "B": 16, "ctx": 1048576, "keep": 2048},
        # one request's three drafted tokens, a small vocabulary
        {"name": "verify_one", "op": "verify", "dtype": "f32", "B": 1, "T": 4, "V": 32000, "draft": True, "tree": False},
        # a batch of the same, a large vocabulary
        {"name": "verify_batch", "op": "verify", "dtype": "f32", "B": 64, "T": 4, "V": 128000, "draft": True, "tree": False},
        # drafts as trees without probabilities, an odd vocabulary
        {"name": "verify_tree", "op": "verify", "dtype": "bf16", "B": 32, "T": 16, "V": 65537, "draft": False, "tree": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = tuple(max(a, b) for a, b in zip(most.get(c["op"], (0, 0)), (w["bytes"], w["flops"])))
    while True:
        op = rng.choice(["window", "window", "weights", "weights", "evict", "verify", "verify"])
        case = {"op": op}
        if op in ("window", "weights"):
            case.update(dtype=rng.choice(["bf16", "fp8"]), H=rng.choice([8, 16, 24, 32, 64, 128]))
        if op == "window":
            kind = rng.choice(["step", "step", "tree", "prompt"])
            case.update(B=_log(rng, 1, 4 if kind == "prompt" else 64), tree=kind == "tree",
                        T=rng.choice([1, 1, 2, 3, 4]) if kind == "step" else _log(rng, 2, 32) if kind == "tree" else _log(rng, 64, 4000))
            case.update(ctx=case["T"] + _log(rng, 1, 131072), window=max(case["T"] if kind == "tree" else 1, _log(rng, 16, 8192)),
                        sink=rng.choice([0, 1, 4, 64, 130]))
        elif op == "weights":
            case.update(B=_log(rng, 1, 64), T=rng.choice([1, 1, 2, 3, 4, 16, 33]), ctx=_log(rng, 64, 131072))
        elif op == "evict":
            case.update(B=_log(rng, 1, 64), ctx=_log(rng, 64, 1048576))
            case["keep"] = _log(rng, 1, -(-case["ctx"] // PAGE))
        else:
            kind = rng.choice(["draft", "draft", "point", "tree"])
            case.update(dtype=rng.choice(["f32", "f32", "bf16"]), B=_log(rng, 1, 64), T=_log(rng, 1, 16), V=_log(rng, 100, 200000),
                        draft=kind == "draft", tree=kind == "tree")
        w = work(case)
        if op == "window" and case["B"] * case["T"] * case["H"] * _reach(case) > 2 ** 28:
            continue
        if op == "weights" and case["B"] * case["T"] * case["H"] * case["ctx"] > 2 ** 29:
            continue
        if op == "verify" and case["B"] * case["T"] * case["V"] > 2 ** 25:
            continue
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1]:
            return case


# ------------------------------------------------------------------ inputs
def _lens(case):
    """Each request's context length: ragged, the first the longest."""
    ctx, low = case["ctx"], case.get("T", 1)
    return [max(low, ctx - (617 * b) % (ctx // 4 + 1)) for b in range(case["B"])]


def _pages(case):
    return -(-case["ctx"] // PAGE)


def _row_bytes(case):
    return DIM * 2 if case["dtype"] == "bf16" else DIM + 4


def _reach(case):
    """Of how many positions the tokens of a request may see some."""
    return case["window"] + case["T"] - 1 + case["sink"]


def work(case):
    op, B, T, H = case["op"], case["B"], case.get("T", 1), case.get("H", 1)
    lens = _lens(case) if "ctx" in case else None
    if op == "window":
        rows = sum(min(n, _reach(case)) for n in lens)
        pairs = 0
        for n in lens:
            for t in range(T):
                p = n - T + t + 1
                pairs += min(p, case["window"]) + min(case["sink"], max(0, p - case["window"]))
        return {"bytes": rows * _row_bytes(case) + B * T * H * (DIM * 2 + NOPE * 2 + 4), "flops": 2 * pairs * H * (DIM + NOPE)}
    if op == "weights":  # the weights before and after of each page
        pages = sum(-(-n // PAGE) for n in lens)
        return {"bytes": sum(lens) * _row_bytes(case) + B * T * H * (DIM * 2 + 4) + 8 * pages, "flops": 2 * sum(lens) * T * H * DIM}
    if op == "evict":  # a weight and two blocks of each page, the kept pages and the freed blocks
        pages = sum(-(-n // PAGE) for n in lens)
        return {"bytes": 16 * pages, "flops": pages}
    size = 4 if case["dtype"] == "f32" else 2
    rows = B * case["V"] * (2 if case["draft"] else 1)  # one row of each request, of the target's and the draft's
    return {"bytes": rows * size + B * T * (size * 2 + 12), "flops": 2 * rows}


def _quantised(x):
    most = x.abs().amax(dim=-1, keepdim=True)
    s = most / torch.full_like(most, 448.0)  # a division, not a product with 1/448
    return (x / s).to(FP8), s.squeeze(-1)


def _tree(g, B, T, root):
    """Each node's parent (-1: none), and for each node the nodes on its way, itself among them, as bits."""
    t = torch.arange(T, device="cuda")
    parent = (torch.rand((B, T), generator=g, device="cuda") * (t + (1 - root))).long() - (1 - root)
    parent[:, 0] = -1
    reach = torch.linalg.matrix_power((parent[..., None] == t).double() + torch.eye(T, device="cuda"), T) > 0
    return parent, (reach.long() << t).sum(-1)


def _inputs(case, seed):
    """What the operators are given, as tensors on the GPU, made from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, B, T, H = case["op"], case["B"], case.get("T", 1), case.get("H", 1)
    i32 = {"dtype": torch.int32, "device": "cuda"}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    s = {"case": case}
    if op == "verify":
        V = case["V"]
        # a target that leaves a few hundred tokens a chance, and a draft near to it
        logits = 3.0 * normal(B, T, V)
        kind = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["probs"] = torch.softmax(logits, -1).to(kind)
        s["draft"] = None
        race = -torch.log(-torch.log(uniform(B, T, V).clamp(1e-12, 1 - 1e-7)))
        if case["draft"]:
            guess = logits[:, :T - 1] + 0.5 * normal(B, T - 1, V)
            s["draft"] = torch.softmax(guess, -1).to(kind)
            tokens = (guess + race[:, 1:]).argmax(-1)
        elif case["tree"]:
            parent, s["tree"] = _tree(g, B, T, 1)
            rows = logits.gather(1, parent.clamp(min=0)[:, 1:, None].expand(-1, -1, V))
            tokens = (rows + race[:, 1:]).argmax(-1)
        else:
            tokens = (2.0 * logits[:, :T - 1] + race[:, 1:]).argmax(-1)
        s["tokens"] = torch.cat([torch.zeros((B, 1), **i32), tokens.to(torch.int32)], 1)
        s["uniform"] = uniform(B, T)
        s.setdefault("tree", None)
        return s

    P = _pages(case)
    s["lens"], s["req"] = torch.tensor(_lens(case), **i32), torch.arange(B, **i32)
    last = (s["lens"] - 1).long() // PAGE
    used = torch.arange(P, device="cuda") <= last[:, None]
    s["blocks"] = n = int(used.sum())
    s["table"] = torch.full((B, P), -1, **i32)
    s["table"][used] = uniform(n).argsort().to(torch.int32)  # scattered over the pool's blocks
    if op == "evict":
        # a few pages have most of the weight, and one in eight is not resident any more
        s["table"][uniform(B, P) < 0.125] = -1
        s["weights"] = torch.exp(2.0 * normal(B, P))
        s["budget"] = torch.full((B,), case["keep"], **i32)
        return s
    s["rows"], s["scales"] = normal(n * PAGE, DIM), None
    if case["dtype"] == "bf16":
        s["rows"] = s["rows"].to(torch.bfloat16)
    else:
        s["rows"], s["scales"] = _quantised(s["rows"])
    s["q"] = normal(B, T, H, DIM).to(torch.bfloat16)
    s["tree"] = _tree(g, B, T, 0)[1] if case.get("tree") else None
    if op == "weights":
        s["before"] = torch.exp(normal(B, P))
        lse = [torch.logsumexp(_scores(s, slice(b, b + 1)), -1) for b in range(B)]
        s["lse"] = torch.cat(lse).view(B, T, H).float()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import tiered_sparse_mla_gb300 as hs
        B, T, H, op = case["B"], case.get("T", 1), case.get("H", 1), case["op"]
        i32 = {"dtype": torch.int32, "device": "cuda"}
        fp8 = op == "evict" or case["dtype"] == "fp8"
        pool = hs.Pool(dtype=hs.HS_FP8_E4M3_ROWSCALE if fp8 else hs.HS_BF16, n_gpu_blocks=s.get("blocks", 1), n_host_blocks=0,
                       max_requests=B, max_ctx=case.get("ctx", PAGE), max_topk=32)
        s["pool"] = pool
        if op == "verify":
            s["index"], s["count"], s["next"] = torch.empty((B, T), **i32), torch.empty(B, **i32), torch.empty(B, **i32)
            torch.cuda.synchronize()
            return s
        pool.set_ctx_lens(s["lens"])
        table = s["table"].cpu().numpy()
        for b in range(B):
            pool.page_map_range(b, 0, table[b], table[b] * 0 - 1)
        if op == "evict":
            P = _pages(case)
            s["kept"], s["count"] = torch.empty((B, min(P, case["keep"] + 2)), **i32), torch.empty(B, **i32)
            s["freed"] = torch.full((B, P), -1, **i32)
        else:
            pool.gpu_rows().copy_(s["rows"].view(torch.uint8))
            if fp8:
                pool.gpu_scales().copy_(s["scales"])
            s["rows"] = s["scales"] = None  # the pool has them
            if op == "window":
                s["out"] = torch.empty((B, T, H, NOPE), dtype=torch.bfloat16, device="cuda")
                s["lse"] = torch.empty((B, T, H), dtype=torch.float32, device="cuda")
                ws = hs.hs_window_workspace_bytes(pool.handle, B, T, H, case["window"], case["sink"])
            else:
                s["weights"] = torch.zeros_like(s["before"])
                ws = hs.hs_weights_workspace_bytes(pool.handle, B, T, H)
            s["workspace"] = torch.empty(max(ws, 1), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        pool = s["pool"]
        if op == "window":
            pool.page_mla_decode_window(s["q"], s["req"], s["tree"], case["window"], case["sink"], SCALE, s["out"], s["lse"],
                                        s["workspace"])
            return s["out"], s["lse"]
        if op == "weights":
            pool.page_weights(s["q"], s["lse"], s["req"], None, SCALE, s["weights"], s["before"], 0.5, s["workspace"])
            return s["weights"]
        if op == "evict":
            # the plan, which leaves the table as it is
            pool.evict_pages(s["req"], s["budget"], s["weights"], s["kept"], s["freed"], s["count"], n_first=1, n_last=2, plan=True)
            return s["kept"], s["freed"], s["count"]
        pool.verify_drafts(s["tokens"], s["probs"], s["draft"], s["tree"], s["uniform"], s["index"], s["count"], s["next"])
        return s["index"], s["count"], s["next"]
    return {"window": _window, "weights": _weights, "evict": _evict, "verify": _verify}[op](s)


def _values(s, at):
    v = s["rows"][at] if s["scales"] is None else s["rows"].view(torch.uint8)[at].view(FP8)
    return v.float() if s["scales"] is None else v.float() * s["scales"][at][..., None]


def _window(s):
    case = s["case"]
    B, T, H, W, N = case["B"], case["T"], case["H"], case["window"], case["sink"]
    draft = s["lens"].long() - T
    t = torch.arange(T, device="cuda")
    # the positions that some token may see: the first ones, then the last ones
    pos = torch.cat([torch.arange(N, device="cuda").expand(B, N),
                     draft[:, None] - W + 1 + torch.arange(W + T - 1, device="cuda")], 1)
    first = torch.arange(pos.shape[1], device="cuda") < N
    there = (pos >= 0) & (pos < s["lens"][:, None]) & (first | (pos >= N))
    if s["tree"] is None:
        at = draft[:, None] + t
        seen = pos[:, None] <= at[..., None]
    else:
        node = pos - draft[:, None]
        bits = (s["tree"][..., None] >> t) & 1
        at = draft[:, None] + bits.sum(-1) - 1
        bit = (s["tree"][..., None] >> node[:, None].clamp(0, 63)) & 1
        seen = (node[:, None] < 0) | (bit == 1)
    seen = seen & there[:, None] & (first | (pos[:, None] > (at - W)[..., None]))
    safe = pos.clamp(0, case["ctx"] - 1)
    block = s["table"].long().gather(1, safe // PAGE).clamp(min=0)
    kv = _values(s, block * PAGE + safe % PAGE)
    x = (s["q"].float().view(B, T * H, DIM) @ kv.transpose(1, 2)) * SCALE
    x = torch.where(seen.repeat_interleave(H, dim=1), x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    e = (x - top).exp()
    total = e.sum(-1, keepdim=True)
    out = (e @ kv[..., :NOPE]) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16).view(B, T, H, NOPE), (top + total.log()).view(B, T, H)


def _scores(s, b):
    """The scaled scores of the requests b (a slice) against all of their rows, -inf where unseen."""
    case = s["case"]
    T, H = case["T"], case["H"]
    table = s["table"][b].long().clamp(min=0)
    kv = _values(s, (table[..., None] * PAGE + torch.arange(PAGE, device="cuda")).view(table.shape[0], -1))
    q = s["q"][b].float().view(-1, T * H, DIM)
    x = (q @ kv.transpose(1, 2)) * SCALE
    end = s["lens"][b].long()[:, None] - T + torch.arange(T, device="cuda")
    seen = torch.arange(kv.shape[1], device="cuda") <= end[..., None]
    return torch.where(seen.repeat_interleave(H, dim=1), x, -math.inf)


def _weights(s):
    case = s["case"]
    B, T, H = case["B"], case["T"], case["H"]
    x = _scores(s, slice(None))
    e = (x - s["lse"].view(B, T * H, 1)).exp()
    got = e.sum(1).view(B, -1, PAGE).sum(-1)
    there = torch.arange(_pages(case), device="cuda") * PAGE < s["lens"][:, None]
    return torch.where(there, 0.5 * s["before"] + got, 0.0)


def _evict(s):
    case = s["case"]
    B, P = case["B"], _pages(case)
    p = torch.arange(P, device="cuda")
    n = ((s["lens"].long() + PAGE - 1) // PAGE)[:, None]
    there = (p < n) & (s["table"] >= 0)
    forced = there & ((p < 1) | (p >= n - 2))
    key = torch.where(forced, math.inf, torch.where(there, s["weights"], -math.inf))
    order = key.argsort(dim=-1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, p.expand(B, P))
    stay = there & (forced | (rank < s["budget"][:, None]))
    width = min(P, case["keep"] + 2)
    kept = torch.where(stay, p, P).sort(-1).values[:, :width]
    gone = there & ~stay
    where = torch.where(gone, p, P).sort(-1).values
    blocks = s["table"].gather(1, where.clamp(max=P - 1))
    freed = torch.where(where < P, blocks, -1)
    return torch.where(kept < P, kept, -1).to(torch.int32), freed, gone.sum(-1).to(torch.int32)


def _verify(s):
    case = s["case"]
    B, T, V = case["B"], case["T"], case["V"]
    t, b = torch.arange(T, device="cuda"), torch.arange(B, device="cuda")[:, None]
    token, u = s["tokens"].long(), s["uniform"].double()
    if s["tree"] is None:
        way = (t <= t[:, None]).expand(B, T, T)
    else:
        way = ((s["tree"][..., None] >> t) & 1) == 1
    parent = torch.where(way & (t < t[:, None]), t, -1).amax(-1)
    px = s["probs"][b, parent.clamp(min=0), token].double()
    brother = (parent[:, :, None] == parent[:, None]) & (t < t[:, None]) & (t > 0)  # [B][T][T]: an earlier child of the same node
    if s["draft"] is not None:
        qx = torch.ones_like(px)
        qx[:, 1:] = s["draft"][b, t[:-1], token[:, 1:]].double()
    else:
        # a child is a sure guess: what its refused brothers had is gone
        fresh = ~(brother & (token[:, :, None] == token[:, None])).any(-1)
        px = torch.where(fresh, px, 0.0)
        qx = 1.0 - (brother * px[:, None]).sum(-1)
    take = (u * qx < px) & (parent >= 0)
    take = take & ~(brother & take[:, None]).any(-1)
    take[:, 0] = True
    path = (take[:, None] | ~way).all(-1) & way[..., 0]
    count = path.sum(-1)
    index = torch.where(path, t, T).sort(-1).values
    end = index.gather(1, count[:, None] - 1)  # the last accepted node
    row = s["probs"].gather(1, end[..., None].expand(B, 1, V)).squeeze(1).double()
    if s["draft"] is not None:
        if T > 1:
            guess = s["draft"].gather(1, end.clamp(max=T - 2)[..., None].expand(B, 1, V)).squeeze(1).double()
            row = torch.where(end < T - 1, (row - guess).clamp(min=0.0), row)
    else:
        refused = (parent == end) & (t > 0)
        row = row.scatter_reduce(1, token, torch.where(refused, 0.0, math.inf).double(), "amin")
    sums = row.cumsum(-1)
    following = (sums <= u[:, :1] * sums[:, -1:]).sum(-1)
    return torch.where(index < T, index, -1).to(torch.int32), count.to(torch.int32), following.to(torch.int32)


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    op, B, T, H = case["op"], case["B"], case.get("T", 1), case.get("H", 1)
    lens = _lens(case) if "ctx" in case else None

    def row(b, positions):
        at = s["table"][b].long()[positions // PAGE] * PAGE + positions % PAGE
        v = s["rows"].view(torch.uint8)[at].view(s["rows"].dtype).double()
        return v if s["scales"] is None else v * s["scales"][at].double()[:, None]

    if op == "window":
        out = torch.zeros((B, T, H, NOPE), dtype=torch.float64, device="cuda")
        lse = torch.zeros((B, T, H), dtype=torch.float64, device="cuda")
        trees = s["tree"].cpu().tolist() if s["tree"] is not None else None
        for b in range(B):
            base = lens[b] - T
            for t in range(T):
                if trees is None:
                    way = list(range(base, base + t + 1))
                    here = base + t
                else:
                    way = [base + i for i in range(T) if trees[b][t] >> i & 1]
                    here = base + len(way) - 1
                first = max(0, here - case["window"] + 1)
                sinks = list(range(min(case["sink"], first, base)))
                at = torch.tensor(sinks + list(range(first, base)) + [i for i in way if i >= first], device="cuda")
                kv = row(b, at)
                x = s["q"][b, t].double() @ kv.T * SCALE
                out[b, t] = torch.softmax(x, -1) @ kv[:, :NOPE]
                lse[b, t] = torch.logsumexp(x, -1)
        return out, lse
    if op == "weights":
        got = torch.zeros(s["before"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = lens[b]
            kv = row(b, torch.arange(n, device="cuda"))
            whole = torch.zeros(-(-n // PAGE) * PAGE, dtype=torch.float64, device="cuda")
            for t in range(T):
                end = n - T + t + 1
                x = s["q"][b, t].double() @ kv[:end].T * SCALE - s["lse"][b, t].double()[:, None]
                whole[:end] += x.exp().sum(0)
            got[b, :whole.numel() // PAGE] = 0.5 * s["before"][b, :whole.numel() // PAGE].double() + whole.view(-1, PAGE).sum(1)
        return got
    if op == "evict":
        P = _pages(case)
        kept = torch.full((B, min(P, case["keep"] + 2)), -1, dtype=torch.int32, device="cuda")
        freed = torch.full((B, P), -1, dtype=torch.int32, device="cuda")
        count = torch.zeros(B, dtype=torch.int32, device="cuda")
        for b in range(B):
            n = -(-lens[b] // PAGE)
            table, weight = s["table"][b].cpu().tolist(), s["weights"][b].cpu().tolist()
            there = [p for p in range(n) if table[p] >= 0]
            must = [p for p in there if p < 1 or p >= n - 2]
            rest = sorted((p for p in there if p not in must), key=lambda p: (-weight[p], p))
            stay = sorted(must + rest[:max(0, case["keep"] - len(must))])
            gone = sorted(set(there) - set(stay))
            kept[b, :len(stay)] = torch.tensor(stay, dtype=torch.int32)
            freed[b, :len(gone)] = torch.tensor([table[p] for p in gone], dtype=torch.int32)
            count[b] = len(gone)
        return kept, freed, count
    index = torch.full((B, T), -1, dtype=torch.int32)
    count, following = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    tokens, u = s["tokens"].cpu().tolist(), s["uniform"].cpu().double().tolist()
    trees = s["tree"].cpu().tolist() if s["tree"] is not None else None
    for b in range(B):
        node, path = 0, [0]
        while True:
            p = s["probs"][b, node].double()
            if trees is None:
                children = [node + 1] if node + 1 < T else []
            else:
                above = [[i for i in range(t) if trees[b][t] >> i & 1] for t in range(T)]
                children = [t for t in range(1, T) if above[t] and above[t][-1] == node]
            left, taken, out = 1.0, None, p.clone()
            for c in children:
                x = tokens[b][c]
                if s["draft"] is not None:
                    q = s["draft"][b, c - 1].double()
                    if u[b][c] * float(q[x]) < float(p[x]):
                        taken = c
                        break
                    out = (p - q).clamp(min=0.0)
                else:
                    if u[b][c] * left < float(out[x]):
                        taken = c
                        break
                    left -= float(out[x])
                    out[x] = 0.0
            if taken is None:
                break
            node = taken
            path.append(node)
        index[b, :len(path)] = torch.tensor(path, dtype=torch.int32)
        count[b] = len(path)
        sums = out.cumsum(0)
        following[b] = int((sums <= u[b][0] * sums[-1]).sum())
    return index.cuda(), count.cuda(), following.cuda()
