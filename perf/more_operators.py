"""The cases that the operators of a paged cache and the sampling of draft tokens are measured on.

Four calls that stand next to draft verification where the cache is cut into pages:

  plan        block tables and slot maps from the rows' lengths: pages are taken from a ring of
              free ones, and those that a row no longer needs go back
  compact     the accepted tree path's entries move up behind the history, across pages
  attention   the pass's attention over a paged cache: a prompt's chunk, single tokens, chains
              or trees of drafted tokens, with a sliding window and first tokens that stay visible
  sample      one token per row under temperature, top-k, top-p and min-p, from given uniforms:
              what a drafter does at every step

`run` is the plain form in elementary torch operations, or (own = True) the framework's call.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a verify pass of 64 rows of up to 8192 tokens, root and 5 drafts each
        dict(name="plan verify pass", op="plan", B=64, N=6, page=16, columns=512, window=0, sinks=0, lo=50, hi=8000, ragged=True),
        # a full batch of long rows whose pages behind the window are given back
        dict(name="plan long rows", op="plan", B=512, N=8, page=16, columns=2048, window=4096, sinks=4, lo=1000, hi=32000, ragged=True),
        # a small tree's path in the keys and values of one layer
        dict(name="compact one layer", op="compact", B=4, N=12, planes=2, page=16, H=8, D=128, cache="bf16", depth=4, lo=100, hi=300),
        # 32 trees of 60 nodes over the keys and values of 16 layers
        dict(name="compact trees", op="compact", B=32, N=60, planes=32, page=32, H=8, D=128, cache="e4m3", depth=6, lo=40, hi=200),
        # one sequence, one token at a time, behind a window of 1024
        dict(name="attend one token", op="attention", B=1, N=1, Hq=32, Hkv=8, D=128, q="bf16", cache="bf16", page=16, window=1024, sinks=4, lo=5000, hi=5000, tree=False, ragged=False),
        # 64 sequences of very different lengths, one token each
        dict(name="attend decode", op="attention", B=64, N=1, Hq=32, Hkv=8, D=128, q="bf16", cache="e4m3", page=16, window=4096, sinks=4, lo=300, hi=9000, tree=False, ragged=False),
        # the verify pass of 64 chains of 5 drafts
        dict(name="attend chains", op="attention", B=64, N=6, Hq=32, Hkv=8, D=128, q="bf16", cache="bf16", page=32, window=2048, sinks=16, lo=100, hi=4000, tree=False, ragged=False),
        # the verify pass of 32 draft trees of 60 nodes
        dict(name="attend trees", op="attention", B=32, N=60, Hq=32, Hkv=8, D=128, q="bf16", cache="e4m3", page=16, window=1024, sinks=4, lo=64, hi=3000, tree=True, ragged=False),
        # two prompts read in one go
        dict(name="attend prompt", op="attention", B=2, N=4096, Hq=32, Hkv=8, D=128, q="bf16", cache="bf16", page=16, window=1024, sinks=4, lo=0, hi=0, tree=False, ragged=False),
        # one sequence's next draft token: the smallest call
        dict(name="sample one row", op="sample", B=1, V=128256, dtype="bf16", top_k=50, top_p=0.9, min_p=0.0, spread=3.0),
        # the frontier of 64 draft trees, four nodes each
        dict(name="sample drafts", op="sample", B=256, V=128256, dtype="bf16", top_k=0, top_p=0.95, min_p=0.02, spread=3.0),
        # no truncation, fp32 logits of a small vocabulary: the whole law is drawn from
        dict(name="sample whole law", op="sample", B=300, V=32000, dtype="f32", top_k=0, top_p=1.0, min_p=0.0, spread=2.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "compact", "attention", "attention", "attention", "sample", "sample"])
    page = rng.choice([16, 16, 32, 64, 128])
    window = rng.choice([0, _log(rng, 1, 200), _log(rng, 200, 5000), _log(rng, 200, 5000)])
    sinks = rng.choice([0, 1, 4, 4, 16, 70]) if window else 0
    if op == "plan":
        B = _log(rng, 1, 400)
        N = rng.choice([1, 1, 2, 6, 9, 60, _log(rng, 1, max(1, 20000 // B))])
        columns = max(-(-(N + 10) // page), _log(rng, 4, 1800))
        hi = rng.randrange(0, columns * page - N + 1)
        return dict(op=op, B=B, N=N, page=page, columns=columns, window=window, sinks=sinks, lo=rng.randrange(0, hi + 1), hi=hi, ragged=rng.random() < 0.6)
    H, D = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 64, 80, 96, 128, 128, 128])
    cache = rng.choice(["e4m3", "e4m3", "bf16", "bf16", "f16"])
    if op == "compact":
        N = _log(rng, 8, 64)
        lo = rng.randrange(0, 200)
        return dict(op=op, B=_log(rng, 1, 32), N=N, planes=_log(rng, 1, 16) * 2, page=page, H=H, D=D, cache=cache, depth=rng.randrange(0, min(7, N // 2)), lo=lo, hi=lo + rng.randrange(0, 120))
    if op == "attention":
        q = cache if cache != "e4m3" else rng.choice(["bf16", "bf16", "f16"])
        kind = rng.random()
        tree = kind < 0.25
        if tree:
            B, N, G = _log(rng, 1, 32), _log(rng, 2, 60), rng.choice([1, 2, 4])
        elif kind < 0.5:  # a chunk of a prompt
            B, N, G = rng.choice([1, 1, 2, 5]), _log(rng, 30, 5000), rng.choice([1, 2, 4, 7])
        else:
            B, N, G = _log(rng, 1, 96), rng.choice([1, 1, 1, 2, 4, 5, 6, 8, 9]), rng.choice([1, 2, 4, 7, 8])
        lo = rng.choice([0, rng.randrange(0, 600), _log(rng, 300, 8000)])
        hi = lo + rng.choice([0, rng.randrange(0, 900), _log(rng, 300, 8000)])
        N = min(N, int(math.sqrt(2.2e8 / (B * H * G))))
        hi = max(0, min(hi, int(2.2e8 / (B * N * H * G)) - N, int(4e8 / (B * H * D)) - N))
        return dict(op=op, B=B, N=N, Hq=H * G, Hkv=H, D=D, q=q, cache=cache, page=page, window=window, sinks=sinks, lo=min(lo, hi), hi=hi, tree=tree, ragged=rng.random() < 0.3)
    V = _log(rng, 50, 150000)
    return dict(op=op, B=_log(rng, 1, min(256, 3e7 / V)), V=V, dtype=rng.choice(["bf16", "f32"]), top_k=rng.choice([0, 0, 1, 20, 50, 200]), top_p=rng.choice([1.0, 0.99, 0.9, 0.8, 0.3]), min_p=rng.choice([0.0, 0.0, 0.02, 0.1]), spread=rng.choice([0.5, 2.0, 3.0, 3.0]))


# --------------------------------------------------------------- the cache
def _entry(H, D, cache):
    """Bytes of one token's entry in one plane: codes and scale bytes, padded to 16."""
    return (H * D + H + 15) // 16 * 16 if cache == "e4m3" else 2 * H * D


def _pack(x, cache):
    """Cache entries of x [..., H, D] (float32): 16-bit numbers, or e4m3 codes with, per head, the smallest
    power-of-two scale 2^(byte - 127) that brings the largest magnitude to at most 448."""
    if cache != "e4m3":
        return x.to(DTYPES[cache])
    H, D = x.shape[-2:]
    bits = x.abs().amax(-1).view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_min(1)
    y = x * ((254 - byte) << 23).view(torch.float32)[..., None]
    e = torch.zeros(*x.shape[:-2], _entry(H, D, cache), dtype=torch.uint8, device=x.device)
    e[..., : H * D] = y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    e[..., H * D : H * D + H] = byte.to(torch.uint8)
    return e


def _values(entries, H, D, cache):
    """float32 values [..., H, D] of cache entries."""
    if cache != "e4m3":
        return entries.float()
    codes = entries[..., : H * D].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (H, D))
    byte = entries[..., H * D : H * D + H].int()
    return codes * torch.where(byte == 255, float("nan"), (byte << 23).view(torch.float32))[..., None]


def _lengths(n, lo, hi):
    """n lengths spread over lo..hi, in an order that is not sorted."""
    return [lo + ((7 * i + 3) % n) * (hi - lo) // max(1, n - 1) for i in range(n)]


def _counts(case):
    return [1 + (5 * b + 2) % case["N"] if case["ragged"] else case["N"] for b in range(case["B"])]


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _live(kv_len, total, columns, page, window, sinks):
    """[B, columns]: pages that hold a token of the row (total of them) that a query from kv_len on can see."""
    j = torch.arange(columns, device="cuda")
    live = j * page < total[:, None]
    if window:
        live &= ~((j * page >= sinks) & ((j + 1) * page <= kv_len[:, None] - window + 1))
    return live


def _tables(g, live, pages):
    """A block table with a page of its own, in random order, at every live place, and the pages left over."""
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    rank = torch.cumsum(live.flatten().int(), 0) - 1
    table = torch.where(live.flatten(), order[rank.clamp_min(0)], -1).view(live.shape)
    return table, order[int(live.sum()) :]


# ---------------------------------------------------------------- prepare
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "sample":
        B, V = case["B"], case["V"]
        x = case["spread"] * torch.randn(B, V, generator=g, device="cuda")
        x[:, torch.randint(0, V, (max(1, V // 6000),), generator=g, device="cuda")] += 3 * case["spread"]
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["u"] = torch.rand(B, generator=g, device="cuda")
        s["temperature"] = 0.5 + 0.7 * torch.rand(B, generator=g, device="cuda")
        s["k"] = torch.full((B,), case["top_k"], dtype=torch.int32, device="cuda") if case["top_k"] else None
        s["p"] = torch.full((B,), case["top_p"], device="cuda") if case["top_p"] < 1 else None
        s["m"] = torch.full((B,), case["min_p"], device="cuda") if case["min_p"] else None
        return s
    B, N, page = case["B"], case["N"], case["page"]
    kv_len = s["kv_len"] = _ints(_lengths(B, case["lo"], case["hi"]))
    if op == "plan":
        # where the rows stood before the last pass: up to 9 tokens back, and further on by rejected drafts
        counts = _ints(_counts(case))
        s["count"] = counts if case["ragged"] else None
        before = (kv_len - torch.randint(0, 10, (B,), generator=g, device="cuda", dtype=torch.int32)).clamp_min(0)
        over = kv_len + torch.randint(0, 4, (B,), generator=g, device="cuda", dtype=torch.int32) * (page // 2)
        had = _live(before, torch.minimum(over, torch.full_like(over, case["columns"] * page)), case["columns"], page, case["window"], case["sinks"])
        # a pool for what the rows had and what they need now
        pages = s["pages"] = sum(min(case["columns"], (n + max(N, 2 * page)) // page + 1) for n in _lengths(B, case["lo"], case["hi"])) + 37
        s["table"], left = _tables(g, had, pages)
        head = int(torch.randint(0, pages, (1,), generator=g, device="cuda"))
        s["free"] = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
        s["free"][(head + torch.arange(len(left), device="cuda")) % pages] = left
        s["ring"] = _ints([head, len(left)])
        return s
    H, D = case["H"] if op == "compact" else case["Hkv"], case["D"]
    columns = -(-(case["hi"] + N) // page) + 1
    window, sinks = (case["window"], case["sinks"]) if op == "attention" else (0, 0)
    live = _live(kv_len, kv_len + N, columns, page, window, sinks)
    pages = int(live.sum()) + 5
    s["table"], _ = _tables(g, live, pages)
    planes = case["planes"] if op == "compact" else 2
    size = torch.exp2(torch.randint(-2, 3, (planes, 1, 1, H, 1), generator=g, device="cuda").float()) if case["cache"] == "e4m3" else 1.0
    s["buffer"] = _pack(size * torch.randn(planes, pages, page, H, D, generator=g, device="cuda"), case["cache"])
    if op == "compact":
        # accepted paths of trees whose first levels are wider than the path is deep
        depth = torch.randint(0, case["depth"] + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        depth[0] = case["depth"]
        pick = torch.rand(B, N, generator=g, device="cuda").masked_fill(torch.arange(N, device="cuda") <= case["depth"], 2.0)
        nodes = pick.argsort(1)[:, : case["depth"] + 1].int().sort(1).values
        order = torch.arange(N, device="cuda")
        s["path"] = torch.full((B, N), -1, dtype=torch.int32, device="cuda")
        s["path"][:, : case["depth"]] = nodes[:, : case["depth"]]
        s["path"][order >= depth[:, None]] = -1
        s["accepted"] = depth
        return s
    s["query"] = (2.0 * torch.randn(B, N, case["Hq"], D, generator=g, device="cuda")).to(DTYPES[case["q"]])
    s["count"] = _ints(_counts(case)) if case["ragged"] else None
    # slots that no token has been written to hold whatever was there
    t = torch.arange(columns * page, device="cuda")
    total = kv_len + (s["count"] if case["ragged"] else N)
    unused = (t >= total[:, None]).view(B, columns, page) & (s["table"] >= 0)[..., None]
    row, j, k = unused.nonzero(as_tuple=True)
    s["buffer"][:, s["table"][row, j].long(), k] = 255 if case["cache"] == "e4m3" else float("nan")
    s["parent"] = None
    if case["tree"]:
        i = torch.arange(N, device="cuda")
        back = 1 + (torch.rand(B, N, generator=g, device="cuda") * i.clamp_max(10)).int()
        s["parent"] = (i - back.clamp_max(10)).clamp_min(0).int().contiguous()
        s["parent"][:, 0] = -1
    return s


# -------------------------------------------------------------------- run
def run(s):
    if own:
        import speculative_decoding_verification_32_gb300 as sv

        return {"plan": _own_plan, "compact": _own_compact, "attention": _own_attention, "sample": _own_sample}[s["op"]](sv, s)
    return {"plan": _plan, "compact": _compact, "attention": _attention, "sample": _sample}[s["op"]](s)


def _own_plan(sv, s):
    slots, status = sv.spec_page_plan(s["table"], s["free"], s["ring"], s["kv_len"], s["N"], s["page"], count=s["count"], window=s["window"], sinks=s["sinks"])
    return {"table": s["table"], "free": s["free"], "ring": s["ring"], "slots": slots, "status": status}


def _own_compact(sv, s):
    sv.spec_kv_compact_pages(s["buffer"], s["table"], s["kv_len"], s["accepted"], s["path"])
    return _held(s)


def _own_attention(sv, s):
    out, lse, _ = sv.spec_paged_attention(s["query"], s["buffer"], s["table"], s["kv_len"], count=s["count"], parent=s["parent"], window=s["window"], sinks=s["sinks"], kv_heads=s["Hkv"])
    return out, lse


def _own_sample(sv, s):
    r = sv.spec_sample(s["logits"], s["u"], s["temperature"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
    return {"token": r["token"], "prob": r["prob"]}


def _plan(s):
    B, N, page, n = s["B"], s["N"], s["page"], s["pages"]
    count = s["count"] if s["count"] is not None else torch.full((B,), N, dtype=torch.int32, device="cuda")
    total = s["kv_len"] + count
    table, columns = s["table"], s["columns"]
    live = _live(s["kv_len"], total, columns, page, s["window"], s["sinks"])
    take, give = live & (table < 0), ~live & (table >= 0)
    head, have = s["ring"][0], s["ring"][1]
    # rows are served in order as far as the free pages go
    served = torch.cumsum(take.sum(1), 0) <= have
    short = ~served & take.any(1)
    take &= served[:, None]
    taken, given = torch.cumsum(take.flatten(), 0), torch.cumsum(give.flatten(), 0)
    back = table.flatten()[give.flatten()]
    s["free"][(head + have + given[give.flatten()] - 1) % n] = back
    table.copy_(torch.where(take, s["free"][(head + taken - 1) % n].view(B, columns), torch.where(give, -1, table)))
    s["ring"].copy_(torch.stack(((head + taken[-1]) % n, have - taken[-1] + given[-1])))
    pos = s["kv_len"][:, None] + torch.arange(N, device="cuda")
    at = torch.gather(table, 1, (pos // page).clamp_max(columns - 1).long())
    used = (torch.arange(N, device="cuda") < count[:, None]) & ~short[:, None]
    slots = torch.where(used, at * page + pos % page, -1).int()
    return {"table": table, "free": s["free"], "ring": s["ring"], "slots": slots, "status": torch.where(short, 9, 0).int()}


def _held(s):
    """What the cache holds, as values: codes and scale exponents, or 16-bit numbers."""
    if s["cache"] != "e4m3":
        return {"entries": s["buffer"]}
    n = s["H"] * s["D"]
    return {"codes": s["buffer"][..., :n].view(torch.float8_e4m3fn), "exponents": s["buffer"][..., n : n + s["H"]]}


def _place(s, pos):
    """(page, token in it) of token positions pos [B, n]."""
    return torch.gather(s["table"], 1, (pos // s["page"]).long()).long(), (pos % s["page"]).long()


def _compact(s):
    k = torch.arange(s["N"], device="cuda")
    keep = k < s["accepted"][:, None]
    source = _place(s, s["kv_len"][:, None] + s["path"].clamp_min(0))
    to = _place(s, torch.where(keep, s["kv_len"][:, None] + 1 + k, 0))
    s["buffer"][:, to[0][keep], to[1][keep]] = s["buffer"][:, source[0][keep], source[1][keep]]
    return _held(s)


def _depths(parent):
    """(depth of each node [B, N], which nodes are its ancestors or itself [B, N, N])."""
    N = parent.shape[1]
    step = torch.arange(N, device="cuda") == parent[..., None]
    seen = torch.matrix_power(step.double() + torch.eye(N, device="cuda", dtype=torch.float64), N) > 0
    return seen.sum(-1) - 1, seen


def _attention(s):
    B, N, Hq, H, D = (s[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    G, T = Hq // H, s["hi"] + N
    t = torch.arange(T, device="cuda")
    page, k = _place(s, t.expand(B, T))
    count = s["count"] if s["count"] is not None else torch.full((B,), N, dtype=torch.int32, device="cuda")
    there = (page >= 0) & (t < (s["kv_len"] + count)[:, None])
    kv = _values(s["buffer"][:, page.clamp_min(0), k], H, D, s["cache"])
    key, value = torch.where(there[None, ..., None, None], kv, 0.0)
    pos = s["kv_len"][:, None] + torch.arange(N, device="cuda")
    if s["parent"] is None:
        seen = t <= pos[..., None]
    else:
        depth, up = _depths(s["parent"])
        j = t - s["kv_len"][:, None]
        tree = torch.gather(up, 2, j.clamp(0, N - 1)[:, None, :].expand(-1, N, -1))
        seen = (j < 0)[:, None, :] | ((j >= 0) & (j < N))[:, None, :] & tree
        pos = s["kv_len"][:, None] + depth
        # where a token stands: the pass's own by their depth in the tree
        t = torch.where(j < 0, t, torch.gather(pos, 1, j.clamp(0, N - 1)))[:, None, :]
    if s["window"]:
        seen &= (t < s["sinks"]) | (t > pos[..., None] - s["window"])
    used = torch.arange(N, device="cuda") < count[:, None]
    seen &= used[..., None]
    x = torch.einsum("bnhgd,bshd->bnhgs", s["query"].float().unflatten(2, (H, G)) * (1.0 / math.sqrt(D)), key)
    x.masked_fill_(~seen[:, :, None, None, :], float("-inf"))
    top = x.amax(-1, keepdim=True).clamp_min(-3e38)
    e = x.sub_(top).exp_()
    total = e.sum(-1, keepdim=True)
    out = torch.einsum("bnhgs,bshd->bnhgd", e, value) / total.clamp_min(1e-30)
    lse = torch.where(used[..., None], (top + torch.log(total)).squeeze(-1).flatten(2), float("-inf"))
    return out.flatten(2, 3).to(s["query"].dtype), lse


def _sample(s):
    x = s["logits"].double()
    V, T = s["V"], s["temperature"].double()[:, None]
    xs = torch.sort(x, 1, descending=True).values
    top = xs[:, :1]
    floor = torch.full_like(top, float("-inf"))
    if s["k"] is not None:
        k = s["k"][:, None].long()
        floor = torch.where((k >= 1) & (k < V), torch.gather(xs, 1, (k - 1).clamp(0, V - 1)), floor)
    if s["p"] is not None:
        # whole groups of equal logits, until their share of what top-k left reaches top_p
        mass = torch.cumsum(torch.where(xs >= floor, torch.exp((xs - top) / T), 0.0), 1)
        last = (mass < s["p"].double()[:, None] * mass[:, -1:]).sum(1, keepdim=True)
        floor = torch.maximum(floor, torch.gather(xs, 1, last.clamp_max(V - 1)))
    keep = x >= floor
    if s["m"] is not None:
        keep &= x - top >= T * torch.log(s["m"].double()[:, None])
    w = torch.where(keep, torch.exp((x - top) / T), 0.0)
    upto = torch.cumsum(w, 1)
    Z = upto[:, -1:]
    # the smallest token whose running sum exceeds u Z, else the last one kept
    at = (upto <= s["u"].double()[:, None] * Z).sum(1, keepdim=True)
    at = torch.minimum(at, V - 1 - (w > 0).flip(1).int().argmax(1, keepdim=True))
    return {"token": at[:, 0].int(), "prob": (torch.gather(w, 1, at) / Z)[:, 0].float()}


# ------------------------------------------------------------------- work
def _seen_pairs(n, N, window, sinks):
    """Query-key pairs of a chain of N tokens behind n, and the tokens that one of them sees."""
    if not window:
        return N * n + N * (N + 1) // 2, n + N
    # a query at p sees p + 1 tokens, without those from sinks on that lie window or more back
    pairs = sum(p + 1 - max(0, p - window + 1 - sinks) for p in range(n, n + N))
    return pairs, n + N - max(0, n - window + 1 - sinks)


def work(case):
    op = case["op"]
    if op == "sample":
        n = case["B"] * case["V"]
        return {"bytes": n * DTYPES[case["dtype"]].itemsize + 24 * case["B"], "flops": 4 * n}
    if op == "plan":
        # the table is read, the slots are written
        return {"bytes": 4 * case["B"] * (case["columns"] + case["N"] + 3), "flops": 4 * case["B"] * (case["columns"] + case["N"])}
    if op == "compact":
        moved = case["planes"] * (case["depth"] + (case["B"] - 1) * case["depth"] / 2) * _entry(case["H"], case["D"], case["cache"])
        return {"bytes": 2 * moved + 4 * case["B"] * (case["N"] + 2), "flops": 0}
    lengths, counts = _lengths(case["B"], case["lo"], case["hi"]), _counts(case)
    if case["tree"]:
        # a node sees what lies before the tree, the root's window of it, and on average half a tree's depth of nodes
        both = [(c * (_seen_pairs(n, 1, case["window"], case["sinks"])[0] + 5), _seen_pairs(n, 1, case["window"], case["sinks"])[1] + c) for n, c in zip(lengths, counts)]
    else:
        both = [_seen_pairs(n, c, case["window"], case["sinks"]) for n, c in zip(lengths, counts)]
    queries = sum(counts) * case["Hq"]
    entries = 2 * sum(t for _, t in both) * _entry(case["Hkv"], case["D"], case["cache"])
    return {"bytes": entries + queries * (4 * case["D"] + 4), "flops": 4 * sum(p for p, _ in both) * case["Hq"] * case["D"]}


# ------------------------------------------------------------------ exact
def _stored(entries, H, D, cache):
    """float64 values of cache entries [..., H, D]."""
    if cache != "e4m3":
        return entries.double()
    raw = entries[..., : H * D].long()
    exponent, fraction = (raw >> 3) & 15, (raw & 7).double()
    size = torch.where(exponent == 0, fraction * 2.0**-9, (8 + fraction) * torch.exp2(exponent.double() - 10))
    size = torch.where((raw & 127) == 127, float("nan"), size)
    x = torch.where(raw >= 128, -size, size).unflatten(-1, (H, D))
    byte = entries[..., H * D : H * D + H].double()
    return x * torch.where(byte == 255, float("nan"), torch.exp2(byte - 127))[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "sample":
        return _exact_sample(s)
    return None  # integers, and entries that are moved as they are


def _exact_attention(s):
    """Row by row and KV head by KV head: softmax over the keys that a query sees, in 64 bits."""
    B, N, Hq, H, D, W = (s[k] for k in ("B", "N", "Hq", "Hkv", "D", "window"))
    G = Hq // H
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, N, Hq), float("-inf"), dtype=torch.float64, device="cuda")
    counts = _counts(s)
    for b, n in enumerate(s["kv_len"].tolist()):
        c = counts[b]
        stands = list(range(n, n + c))
        mine = torch.ones(c, c, dtype=torch.bool).tril()
        if s["parent"] is not None:
            parents = s["parent"][b].tolist()
            mine = torch.zeros(c, c, dtype=torch.bool)
            for i in range(c):
                mine[i, i] = True
                if i:
                    mine[i] |= mine[parents[i]]
                    stands[i] = stands[parents[i]] + 1
        stands = torch.tensor(stands, device="cuda")
        seen = torch.cat((torch.ones(c, n, dtype=torch.bool, device="cuda"), mine.cuda()), 1)
        where = torch.cat((torch.arange(n, device="cuda"), stands))
        if W:
            seen &= (stands[:, None] - where < W) | (where < s["sinks"])
        used = seen.any(0).nonzero()[:, 0]  # a page that nothing sees may be gone
        seen = seen[:, used]
        place = s["table"][b, used // s["page"]].long(), used % s["page"]
        k, v = (_stored(s["buffer"][i][place], H, D, s["cache"]) for i in (0, 1))
        for h in range(H):
            q = s["query"][b, :c, h * G : (h + 1) * G].double().transpose(0, 1)
            x = (q @ k[:, h].T) / math.sqrt(D)
            x.masked_fill_(~seen, float("-inf"))
            z = torch.logsumexp(x, -1)
            out[b, :c, h * G : (h + 1) * G] = (torch.exp(x - z[..., None]) @ v[:, h]).transpose(0, 1)
            lse[b, :c, h * G : (h + 1) * G] = z.T
    return out, lse


def _exact_sample(s):
    """Row by row: the law over the distinct logits first, then its members in the order of their ids."""
    V, prob = s["V"], []
    for b in range(s["B"]):
        x, T = s["logits"][b].double(), float(s["temperature"][b])
        value, member, size = torch.unique(x, return_inverse=True, return_counts=True)
        k = int(s["k"][b]) if s["k"] is not None else 0
        above = size.flip(0).cumsum(0).flip(0)  # members of this value and the larger ones
        alive = above - size < k if 1 <= k < V else torch.ones_like(size, dtype=torch.bool)
        p = torch.exp((value - value[-1]) / T) * alive
        if s["p"] is not None:
            share = (p * size / (p * size).sum()).flip(0).cumsum(0).flip(0)
            before = torch.cat((share[1:], share.new_zeros(1)))
            alive &= before < s["p"][b].double()
        if s["m"] is not None:
            alive &= (value - value[-1]) / T >= math.log(float(s["m"][b]))
        p = torch.where(alive, p, 0.0)
        p = p / (p * size).sum()
        law = p[member]
        upto = law.cumsum(0)
        at = int(torch.searchsorted(upto, s["u"][b].double() * upto[-1], right=True))
        at = min(at, int(law.nonzero()[-1]))
        prob.append(law[at])
    return {"token": None, "prob": torch.stack(prob)}
