"""The operators of block-sparse serving over the paged latent cache, each as a case to run.

Five operators, in the order in which a serving step uses them:

* ``append``: the latent rows of new tokens go into the cache (quantised where the pool holds
  FP8); with an index, only the accepted tokens of a draft do;
* ``means``: the mean row of a page, the cheap key that stands for its 64 tokens;
* ``select``: each query token's pages, those of the highest score (the largest product of any
  head's query with the page's mean row), the first and the last ones always among them;
* ``attend``: attention over the pages selected for each query token;
* ``tree``: attention of a tree of drafted tokens over all of a request's pages.

Rows are 576 wide (512 value columns, then 64), pages hold 64 rows. ``own`` false: plain torch
operations in 32 bits (64 next to the border of a selection). ``own`` true: the framework's calls.
"""
import math

import torch

own = False

DIM, NOPE, PAGE = 576, 512, 64
SCALE = 1.0 / math.sqrt(DIM)
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # the accepted path of each of 32 drafts of 16 tokens, at the end of an agent's first turn
        {"name": "append_accept", "op": "append", "dtype": "fp8", "B": 32, "T": 16, "ctx": 74160, "pick": True},
        # a chunk of prompt of each of eight requests
        {"name": "append_chunk", "op": "append", "dtype": "fp8", "B": 8, "T": 8192, "ctx": 16393, "pick": False},
        # the pages that a step's tokens have gone into, one per request
        {"name": "means_step", "op": "means", "dtype": "bf16", "B": 32, "ctx": 4096, "all": False},
        # every page of eight prompts, after the prefill
        {"name": "means_prompt", "op": "means", "dtype": "bf16", "B": 8, "ctx": 74160, "all": True},
        # one request, a short context: the call's latency
        {"name": "select_one", "op": "select", "B": 1, "T": 1, "H": 16, "ctx": 4096, "N": 4},
        # 16 requests with four query tokens each and a million tokens of context
        {"name": "select_long", "op": "select", "B": 16, "T": 4, "H": 128, "ctx": 1048576, "N": 32},
        # one request, few heads, few pages: the call's latency
        {"name": "attend_one", "op": "attend", "dtype": "bf16", "B": 1, "T": 1, "H": 16, "ctx": 4096, "N": 4},
        # a batch of decode steps, 2048 tokens selected for each
        {"name": "attend_batch", "op": "attend", "dtype": "bf16", "B": 32, "T": 1, "H": 128, "ctx": 131072, "N": 32},
        # four query tokens per request, each with its own pages, FP8 rows
        {"name": "attend_mtp", "op": "attend", "dtype": "fp8", "B": 16, "T": 4, "H": 128, "ctx": 1048576, "N": 32},
        # a small draft after a short, odd context
        {"name": "tree_short", "op": "tree", "dtype": "bf16", "B": 3, "T": 7, "H": 16, "ctx": 1001},
        # a few drafts over long contexts: the cache's bytes count
        {"name": "tree_long", "op": "tree", "dtype": "fp8", "B": 4, "T": 8, "H": 16, "ctx": 131072},
        # wide drafts and all heads: the matrix products count
        {"name": "tree_wide", "op": "tree", "dtype": "bf16", "B": 8, "T": 32, "H": 128, "ctx": 16384},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = tuple(max(a, b) for a, b in zip(most.get(c["op"], (0, 0)), (w["bytes"], w["flops"])))
    while True:
        op = rng.choice(["append", "means", "select", "attend", "attend", "tree", "tree"])
        case = {"op": op}
        if op != "select":
            case["dtype"] = rng.choice(["bf16", "fp8"])
        if op == "append":
            pick = rng.random() < 0.5
            case.update(B=_log(rng, 1, 64), T=_log(rng, 1, 64 if pick else 8192), pick=pick)
            case["ctx"] = case["T"] + _log(rng, 1, 100000)
        elif op == "means":
            case.update(B=_log(rng, 1, 64), ctx=_log(rng, 1, 131072), all=rng.random() < 0.5)
        elif op == "select":
            case.update(B=_log(rng, 1, 32), T=rng.choice([1, 1, 2, 3, 4]), H=rng.choice([8, 16, 24, 32, 64, 128]),
                        ctx=_log(rng, 64, 1048576), N=_log(rng, 3, 64))
        elif op == "attend":
            case.update(B=_log(rng, 1, 64), T=rng.choice([1, 1, 2, 3, 4]), H=rng.choice([8, 16, 24, 32, 64, 128]),
                        ctx=_log(rng, 64, 131072), N=_log(rng, 1, 64))
        else:
            case.update(B=_log(rng, 1, 16), T=_log(rng, 1, 64), H=rng.choice([8, 16, 24, 32, 64, 128]),
                        ctx=_log(rng, 65, 131072))
        w = work(case)
        scores = case["B"] * case.get("T", 1) * case.get("H", 1) * case["ctx"] if op == "tree" else 0
        if w["bytes"] <= most[op][0] and w["flops"] <= most[op][1] and scores <= 8 * 32 * 128 * 16384:
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


def _union(case):
    """Of how many pages a request's tokens take theirs."""
    return min(-(-min(_lens(case)) // PAGE), case["N"] + (case["T"] - 1) * (case["N"] // 4))


def work(case):
    op, B, T, H = case["op"], case["B"], case.get("T", 1), case.get("H", 1)
    if op == "append":  # every row read as BF16 and written as the pool holds it
        rows = B * T * (0.4 if case["pick"] else 1.0)
        return {"bytes": rows * (DIM * 2 + _row_bytes(case)), "flops": rows * DIM * 2}
    if op == "means":
        lens = _lens(case)
        tokens = sum(lens) if case["all"] else sum((n - 1) % PAGE + 1 for n in lens)
        pages = sum(-(-n // PAGE) for n in lens) if case["all"] else B
        return {"bytes": tokens * _row_bytes(case) + pages * DIM * 2, "flops": tokens * DIM}
    if op == "select":
        pages = sum(-(-n // PAGE) for n in _lens(case))
        return {"bytes": pages * DIM * 2 + B * T * H * DIM * 2 + B * T * case["N"] * 4, "flops": 2 * pages * T * H * DIM}
    if op == "attend":
        n = min(case["N"], _union(case)) * PAGE
        bytes_ = B * _union(case) * PAGE * _row_bytes(case)
        keys = B * n
    else:
        bytes_ = sum(_lens(case)) * _row_bytes(case)
        keys = sum(_lens(case))
    return {"bytes": bytes_ + B * T * H * (DIM * 2 + NOPE * 2 + 4), "flops": 2 * keys * T * H * (DIM + NOPE)}


def _quantised(x):
    most = x.abs().amax(dim=-1, keepdim=True)
    s = most / torch.full_like(most, 448.0)  # a division, not a product with 1/448
    return (x / s).to(FP8), s.squeeze(-1)


def _inputs(case, seed):
    """What the operators are given, as tensors on the GPU, made from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, B, T, H = case["op"], case["B"], case.get("T", 1), case.get("H", 1)
    i32 = {"dtype": torch.int32, "device": "cuda"}

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def order(*shape):
        return torch.rand(shape, generator=g, device="cuda").argsort(-1)

    s = {"case": case, "lens": torch.tensor(_lens(case), **i32), "req": torch.arange(B, **i32)}
    P = _pages(case)
    last = (s["lens"] - 1).long() // PAGE
    every = torch.arange(P, device="cuda").expand(B, P)
    if op == "append":
        used = (every >= ((s["lens"] - T).long() // PAGE)[:, None]) & (every <= last[:, None])
    elif op == "means" and not case["all"]:
        used = every == last[:, None]
    elif op == "attend":
        U, N = _union(case), min(case["N"], _union(case))
        first = every <= ((s["lens"] - T).long() // PAGE)[:, None]  # pages that every token sees some of
        key = torch.rand((B, P), generator=g, device="cuda") + 2.0 * ~first
        union = key.argsort(-1)[:, :U]
        mine = order(B, T, U)[..., :N]
        pages = union[:, None].expand(B, T, U).gather(2, mine).sort(-1).values
        s["pages"] = torch.full((B, T, case["N"]), -1, **i32)
        s["pages"][..., :N] = pages
        used = torch.zeros((B, P), dtype=torch.bool, device="cuda").scatter_(1, union, True)
    else:
        used = every <= last[:, None]
    if op == "select":
        # pages and queries share a few directions, as those of one text do
        topics = normal(24, DIM)
        mix = normal(B, P, 24) * 0.05
        s["means"] = (normal(B, P, DIM) * 0.125 + mix @ topics).to(torch.bfloat16)
        s["q"] = (normal(B, T, H, DIM) + 0.3 * (normal(B, T, H, 24) @ topics)).to(torch.bfloat16)
        return s
    n = int(used.sum())
    s["table"] = torch.full((B, P), -1, **i32)
    s["table"][used] = order(n).to(torch.int32)  # scattered over the pool's blocks
    if case["dtype"] == "bf16":
        s["rows"], s["scales"] = normal(n * PAGE, DIM).to(torch.bfloat16), None
    else:
        s["rows"], s["scales"] = _quantised(normal(n * PAGE, DIM))
    if op == "append":
        s["new"] = normal(B, T, DIM).to(torch.bfloat16)
        s["start"] = s["lens"] - T
        s["index"] = None
        if case["pick"]:  # a path down the draft, then nothing
            keep = torch.rand((B, T), generator=g, device="cuda") < 0.4
            at = torch.where(keep, torch.arange(T, device="cuda"), T).sort(-1).values
            s["index"] = torch.where(at < T, at, -1).to(torch.int32)
    elif op == "means":
        pick = used.nonzero()
        s["which"] = (pick[:, 0].to(torch.int32).contiguous(), pick[:, 1].to(torch.int32).contiguous())
        s["means"] = torch.zeros((B, P, DIM), dtype=torch.bfloat16, device="cuda")
    else:
        s["q"] = normal(B, T, H, DIM).to(torch.bfloat16)
    if op == "tree":
        # every token hangs on an earlier one, or on the context's end
        t = torch.arange(T, device="cuda")
        parent = (torch.rand((B, T, 1), generator=g, device="cuda") * (t[:, None] + 1)).long() - 1
        reach = torch.linalg.matrix_power((parent == t).double() + torch.eye(T, device="cuda"), T) > 0
        s["tree"] = (reach.long() << t).sum(-1)  # bit i of word t: token t sees token i
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import tiered_sparse_mla_gb300 as hs
        B, T, H, op = case["B"], case.get("T", 1), case.get("H", 1), case["op"]
        fp8 = case.get("dtype") == "fp8"
        n = s["rows"].shape[0] // PAGE if "rows" in s else 1
        pool = hs.Pool(dtype=hs.HS_FP8_E4M3_ROWSCALE if fp8 else hs.HS_BF16, n_gpu_blocks=n, n_host_blocks=0,
                       max_requests=B, max_ctx=case["ctx"], max_topk=32)
        pool.set_ctx_lens(s["lens"])
        if "table" in s:
            table = s["table"].cpu().numpy()
            for b in range(B):
                pool.page_map_range(b, 0, table[b], table[b] * 0 - 1)
            pool.gpu_rows().copy_(s["rows"].view(torch.uint8))
            if fp8:
                pool.gpu_scales().copy_(s["scales"])
            s["rows"] = pool.gpu_rows().view(FP8 if fp8 else torch.bfloat16)
            s["scales"] = pool.gpu_scales()
        s["pool"] = pool
        ws = 0
        if op == "select":
            s["pages"] = torch.empty((B, T, case["N"]), dtype=torch.int32, device="cuda")
            ws = hs.hs_select_workspace_bytes(pool.handle, B, T)
        elif op in ("attend", "tree"):
            s["out"] = torch.empty((B, T, H, NOPE), dtype=torch.bfloat16, device="cuda")
            s["lse"] = torch.empty((B, T, H), dtype=torch.float32, device="cuda")
            ws = (hs.hs_page_decode_workspace_bytes(B * T, 1, H, case["N"]) if op == "attend"
                  else hs.hs_page_decode_workspace_bytes(B, T, H, _pages(case)))
        s["workspace"] = torch.empty(max(ws, 1), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        pool = s["pool"]
        if op == "append":
            pool.append_rows(s["new"], s["req"], s["start"], s["index"])
            return (s["rows"], s["scales"]) if s["scales"] is not None else s["rows"]
        if op == "means":
            pool.page_means(*s["which"], s["means"])
            return s["means"]
        if op == "select":
            pool.select_pages(s["q"], s["means"], s["req"], s["pages"], n_first=1, n_last=2, workspace=s["workspace"])
            return s["pages"]
        if op == "attend":
            pool.page_mla_decode_per_token(s["q"], s["pages"], s["req"], None, SCALE, s["out"], s["lse"], s["workspace"])
        else:
            pool.page_mla_decode(s["q"], None, s["req"], s["tree"], SCALE, s["out"], s["lse"], s["workspace"])
        return s["out"], s["lse"]
    return {"append": _append, "means": _means, "select": _select, "attend": _attend, "tree": _tree}[op](s)


def _append(s):
    B, T = s["new"].shape[:2]
    k = torch.arange(T, device="cuda").expand(B, T)
    index = k if s["index"] is None else s["index"].long()
    rows = s["new"].gather(1, index.clamp(min=0)[..., None].expand(B, T, DIM))
    pos = s["start"].long()[:, None] + k
    to = s["table"].long().gather(1, pos // PAGE) * PAGE + pos % PAGE
    keep = index >= 0
    # a skipped row is written over by what its place holds already
    if s["scales"] is None:
        old = s["rows"][to]
        s["rows"][to] = torch.where(keep[..., None], rows, old)
        return s["rows"]
    codes, scale = _quantised(rows.float())
    bytes_ = s["rows"].view(torch.uint8)
    bytes_[to] = torch.where(keep[..., None], codes.view(torch.uint8), bytes_[to])
    s["scales"][to] = torch.where(keep, scale, s["scales"][to])
    return s["rows"], s["scales"]


def _values(s, at):
    v = s["rows"][at] if s["scales"] is None else s["rows"].view(torch.uint8)[at].view(FP8)
    return v.float() if s["scales"] is None else v.float() * s["scales"][at][..., None]


def _means(s):
    b, p = (x.long() for x in s["which"])
    i = torch.arange(PAGE, device="cuda")
    v = _values(s, s["table"][b, p].long()[:, None] * PAGE + i)
    live = (p[:, None] * PAGE + i) < s["lens"].long()[b][:, None]
    total = torch.where(live[..., None], v, 0.0).sum(1)
    s["means"][b, p] = (total / live.sum(1, keepdim=True)).to(torch.bfloat16)
    return s["means"]


def _select(s):
    case = s["case"]
    B, T, H, N, P = case["B"], case["T"], case["H"], case["N"], s["means"].shape[1]
    score = (s["q"].float().reshape(B, T * H, DIM) @ s["means"].float().transpose(1, 2)).view(B, T, H, P).amax(2)
    end = s["lens"].long()[:, None] - T + torch.arange(T, device="cuda") + 1  # tokens seen
    n = ((end + PAGE - 1) // PAGE)[..., None]
    p = torch.arange(P, device="cuda")
    forced = ((p < 1) | (p >= n - 2)) & (p < n)
    score = torch.where(forced, math.inf, torch.where(p < n, score, -math.inf))
    # those in question again in 64 bits, in ascending order so that ties go to the lowest
    near = score.argsort(-1, descending=True)[..., :min(P, N + 64)].sort(-1).values
    means = s["means"].gather(1, near.reshape(B, -1, 1).expand(-1, -1, DIM)).view(B, T, -1, DIM)
    fine = (s["q"].double() @ means.double().transpose(2, 3)).amax(2)
    rough = score.gather(2, near)
    fine = torch.where(rough.isinf(), rough.double(), fine)
    best, at = fine.sort(dim=-1, descending=True, stable=True)
    chosen = torch.where(best > -math.inf, near.gather(2, at), P)[..., :N].sort(-1).values
    pages = torch.full((B, T, N), -1, dtype=torch.int32, device="cuda")
    pages[..., :chosen.shape[-1]] = torch.where(chosen < P, chosen, -1)
    return pages


def _softmax_product(q, kv, seen):
    """q [L][M][576], kv [L][K][576], seen [L][M][K]: the weighted mean of the rows and ln of the weights' sum."""
    x = (q.float() @ kv.transpose(1, 2)) * SCALE
    x = torch.where(seen, x, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top.isinf(), 0.0, top)
    e = (x - top).exp()
    total = e.sum(-1, keepdim=True)
    out = (e @ kv[..., :NOPE]) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16), (top + total.log()).squeeze(-1)


def _attend(s):
    case = s["case"]
    B, T, H = case["B"], case["T"], case["H"]
    pages = s["pages"].long()
    N = pages.shape[2]
    i = torch.arange(PAGE, device="cuda")
    block = s["table"].long().gather(1, pages.clamp(min=0).view(B, -1)).view(B, T, N)
    kv = _values(s, (block.clamp(min=0)[..., None] * PAGE + i).view(B * T, N * PAGE))
    pos = torch.where(pages[..., None] >= 0, pages[..., None] * PAGE + i, 1 << 40).view(B, T, -1)
    end = s["lens"].long()[:, None] - T + torch.arange(T, device="cuda")
    seen = (pos <= end[..., None]).view(B * T, 1, -1)
    out, lse = _softmax_product(s["q"].view(B * T, H, DIM), kv, seen)
    return out.view(B, T, H, NOPE), lse.view(B, T, H)


def _tree(s):
    case = s["case"]
    B, T, H = case["B"], case["T"], case["H"]
    i = torch.arange(PAGE, device="cuda")
    table = s["table"].long().clamp(min=0)
    kv = _values(s, (table[..., None] * PAGE + i).view(B, -1))
    pos = torch.arange(kv.shape[1], device="cuda")
    node = pos - (s["lens"].long()[:, None] - T)  # [B][K]: which drafted token a row is
    bit = (s["tree"][:, :, None] >> node[:, None].clamp(0, 63)) & 1
    seen = (node[:, None] < 0) | ((node[:, None] < T) & (bit == 1))
    out, lse = _softmax_product(s["q"].view(B, T * H, DIM), kv, seen.repeat_interleave(H, dim=1))
    return out.view(B, T, H, NOPE), lse.view(B, T, H)


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    op, B, T, H = case["op"], case["B"], case.get("T", 1), case.get("H", 1)
    lens = _lens(case)

    def row(b, positions):
        at = s["table"][b].long()[positions // PAGE] * PAGE + positions % PAGE
        v = s["rows"].view(torch.uint8)[at].view(s["rows"].dtype).double()
        return at, v if s["scales"] is None else v * s["scales"][at].double()[:, None]

    if op == "append":
        rows, scales = s["rows"].float().double(), None if s["scales"] is None else s["scales"].double()
        for b in range(B):
            take = torch.arange(T, device="cuda") if s["index"] is None else s["index"][b].long()
            k = (take >= 0).nonzero().squeeze(1)
            x = s["new"][b][take[k]].double()
            at, _ = row(b, lens[b] - T + k)
            if scales is None:
                rows[at] = x
            else:
                # the scale, and each quotient, are defined as their values in 32 bits
                scale = (x.abs().max(1).values / 448).float()
                rows[at] = (x.float() / scale[:, None]).to(FP8).double()
                scales[at] = scale.double()
        return rows if scales is None else (rows, scales)
    if op == "means":
        means = torch.zeros(s["means"].shape, dtype=torch.float64, device="cuda")
        for b in range(B):
            n = lens[b]
            first = 0 if case["all"] else (n - 1) // PAGE * PAGE
            _, v = row(b, torch.arange(first, n, device="cuda"))
            whole = (n - first) // PAGE
            means[b, first // PAGE:first // PAGE + whole] = v[:whole * PAGE].view(whole, PAGE, DIM).mean(1)
            if n % PAGE:
                means[b, n // PAGE] = v[whole * PAGE:].mean(0)
        return means
    if op == "select":
        pages = torch.full((B, T, case["N"]), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            for t in range(T):
                n = -(-(lens[b] - T + t + 1) // PAGE)
                score = torch.einsum("hd,pd->hp", s["q"][b, t].double(), s["means"][b, :n].double()).max(0).values
                score[0] = score[max(0, n - 2):] = math.inf
                best = torch.argsort(score, descending=True, stable=True)[:case["N"]]
                pages[b, t, :len(best)] = best.sort().values.int()
        return pages
    out = torch.zeros((B, T, H, NOPE), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, T, H), dtype=torch.float64, device="cuda")
    for b in range(B):
        base = lens[b] - T
        if op == "tree":
            _, kv = row(b, torch.arange(lens[b], device="cuda"))
        for t in range(T):
            if op == "tree":
                mask = int(s["tree"][b, t])
                at = list(range(T))
                hidden = torch.tensor([base + i for i in at if not mask >> i & 1], dtype=torch.long, device="cuda")
                x = s["q"][b, t].double() @ kv.T * SCALE
                x[:, hidden] = -math.inf
            else:
                mine = s["pages"][b, t].long()
                at = (mine[mine >= 0][:, None] * PAGE + torch.arange(PAGE, device="cuda")).reshape(-1)
                _, kv = row(b, at[at <= base + t])
                x = s["q"][b, t].double() @ kv.T * SCALE
            out[b, t] = torch.softmax(x, -1) @ kv[:, :NOPE]
            lse[b, t] = torch.logsumexp(x, -1)
    return out, lse
