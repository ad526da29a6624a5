"""The cases that the cache, attention and log-probability operators are measured on.

Four calls that stand next to draft verification in a decode loop:

  append      the keys and values of newly fed tokens are rounded into the KV cache
              (8-bit codes with a power-of-two scale per token and head, or 16 bits)
  read        rows of that cache read back as dense 16- or 32-bit tensors
  attention   the verify pass's attention: the drafted tokens of every row (a chain or a
              tree) over a prefix that all rows share and over the row's own cache
  logprobs    log probability of given tokens, entropy and the top alternatives

`run` is the plain form in elementary torch operations, or (own = True) the framework's call.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one sequence decoding alone: the smallest write, where latency counts
        dict(name="append one token", op="append", B=1, N=1, S=512, H=8, D=128, src="bf16", cache="e4m3", ragged=False),
        # a verify pass of 64 rows and 5 drafts, every row at its own length, some rows with fewer drafts
        dict(name="append drafts", op="append", B=64, N=6, S=1024, H=8, D=128, src="bf16", cache="e4m3", ragged=True),
        # a prompt's keys and values written as the shared prefix
        dict(name="append prompt", op="append", B=1, N=32768, S=32768, H=8, D=128, src="bf16", cache="e4m3", ragged=False),
        # a few short rows read back
        dict(name="read short rows", op="read", B=3, T=77, H=2, D=64, cache="e4m3", out="f32", lo=0, hi=77),
        # a batch's cache read back, to be moved or to be fed to another model
        dict(name="read batch", op="read", B=32, T=2048, H=8, D=128, cache="e4m3", out="bf16", lo=200, hi=2048),
        # one sequence, one token at a time
        dict(name="attend one token", op="attention", B=1, N=1, Hq=32, Hkv=8, D=128, q="bf16", cache="bf16", P=1000, lo=150, hi=150, tree=False),
        # 64 sequences behind one prompt, one token each
        dict(name="attend decode", op="attention", B=64, N=1, Hq=32, Hkv=8, D=128, q="bf16", cache="e4m3", P=8192, lo=100, hi=2000, tree=False),
        # the verify pass of 64 chains of 5 drafts behind one prompt
        dict(name="attend chains", op="attention", B=64, N=6, Hq=32, Hkv=8, D=128, q="bf16", cache="bf16", P=8192, lo=30, hi=1000, tree=False),
        # the verify pass of 32 draft trees of 60 nodes
        dict(name="attend trees", op="attention", B=32, N=60, Hq=32, Hkv=8, D=128, q="bf16", cache="e4m3", P=4097, lo=64, hi=500, tree=True),
        # one sequence's next token (the smallest row count)
        dict(name="logprobs one row", op="logprobs", B=1, npos=1, V=128256, dtype="bf16", m=20, partial=False, masked=0.0),
        # what 64 verified chains emitted
        dict(name="logprobs emitted", op="logprobs", B=64, npos=6, V=128256, dtype="bf16", m=20, partial=True, masked=0.0),
        # a scored prompt: every position, fp32 logits
        dict(name="logprobs prompt", op="logprobs", B=1, npos=2047, V=32000, dtype="f32", m=5, partial=False, masked=0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "logprobs"])
    H = rng.choice([1, 2, 3, 4, 8])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128])
    cache = rng.choice(["e4m3", "e4m3", "bf16", "f16"])
    if op == "append":
        src = rng.choice(["bf16", "f16", "f32"])
        if rng.random() < 0.4:
            B, N = 1, _log(rng, 100, 15000 if src == "f32" else 24000)
        else:
            B, N = _log(rng, 1, 200), _log(rng, 1, 64)
        return dict(op=op, B=B, N=N, S=N + rng.randrange(1, 400), H=H, D=D, src=src, cache=cache, ragged=rng.random() < 0.5)
    if op == "read":
        B, T = _log(rng, 1, 32), _log(rng, 1, 2000)
        lo = rng.randrange(0, T + 1)
        return dict(op=op, B=B, T=T, H=H, D=D, cache=cache, out=rng.choice(["bf16", "f16", "f32"]), lo=lo, hi=rng.randrange(lo, T + 1))
    if op == "attention":
        tree = rng.random() < 0.3
        B = _log(rng, 1, 32 if tree else 96)
        N = _log(rng, 2, 60) if tree else rng.choice([1, 1, 2, 3, 4, 5, 6, 8, 9])
        q = cache if cache != "e4m3" else rng.choice(["bf16", "f16"])
        lo = rng.randrange(0, 600)
        P = rng.choice([0, _log(rng, 1, 200), _log(rng, 200, 8000), _log(rng, 200, 8000)])
        if B <= 4 and rng.random() < 0.5:  # few rows behind a long prompt
            P = _log(rng, 8000, 60000)
        Hq, hi = H * rng.choice([1, 2, 4, 4 if tree else 7]), lo + rng.randrange(0, 900)
        P = min(P, max(0, int(2.5e8 / (B * N * Hq)) - hi - N))
        return dict(op=op, B=B, N=N, Hq=Hq, Hkv=H, D=D, q=q, cache=cache, P=P, lo=lo, hi=hi, tree=tree)
    V = _log(rng, 50, 150000)
    npos = rng.choice([1, 4, 6, 9])
    B = _log(rng, 1, min(64, 5e7 / (V * npos)))
    return dict(op=op, B=B, npos=npos, V=V, dtype=rng.choice(["bf16", "f32"]), m=rng.choice([1, 5, 20, 50]), partial=rng.random() < 0.4, masked=rng.choice([0.0, 0.0, 0.3]))


# ----------------------------------------------------------- cache entries
def _entry(H, D, cache):
    """Bytes of one token's entry in one plane: codes and scale bytes, padded to 16."""
    return (H * D + H + 15) // 16 * 16 if cache == "e4m3" else 2 * H * D


def _lengths(n, lo, hi):
    """n lengths spread over lo..hi, in an order that is not sorted."""
    return [lo + ((7 * i + 3) % n) * (hi - lo) // max(1, n - 1) for i in range(n)]


def _counts(case):
    return [1 + (5 * b + 2) % case["N"] if case["ragged"] else case["N"] for b in range(case["B"])]


def _quantise(x):
    """e4m3 codes and scale bytes of x [..., D] (float32): the scale is the smallest power of two, as
    2^(byte - 127), that brings the largest magnitude to at most 448."""
    amax = x.abs().amax(-1)
    bits = amax.view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).int()).clamp_min(1)
    ok = torch.isfinite(amax)
    byte = torch.where(ok, byte, 255)
    inverse = torch.where(ok, ((254 - byte) << 23).view(torch.float32), 0.0)
    y = torch.where(ok[..., None], x * inverse[..., None], 0.0)
    return y.to(torch.float8_e4m3fn), byte.to(torch.uint8)


def _values(entries, H, D, cache):
    """float32 values [..., H, D] of cache entries."""
    if cache != "e4m3":
        return entries.float()
    codes = entries[..., : H * D].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (H, D))
    byte = entries[..., H * D : H * D + H].int()
    scale = torch.where(byte == 255, float("nan"), torch.ldexp(torch.ones((), device=entries.device), byte - 127))
    return codes * scale[..., None]


def _pack(x, cache):
    """Cache entries of x [..., H, D] (float32)."""
    if cache != "e4m3":
        return x.to(DTYPES[cache])
    H, D = x.shape[-2:]
    codes, byte = _quantise(x)
    e = torch.zeros(*x.shape[:-2], _entry(H, D, cache), dtype=torch.uint8, device=x.device)
    e[..., : H * D] = codes.view(torch.uint8).flatten(-2)
    e[..., H * D : H * D + H] = byte
    return e


def _random_cache(g, rows, slots, H, D, cache):
    """A cache [2, rows, slots, ...] of keys and values whose size differs from head to head."""
    size = torch.exp2(torch.randint(-2, 3, (2, 1, 1, H, 1), generator=g, device="cuda").float())
    x = torch.randn(2, rows, slots, H, D, generator=g, device="cuda")
    return _pack(x * size if cache == "e4m3" else x, cache)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- prepare
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "append":
        B, N, H, D, S = (case[k] for k in ("B", "N", "H", "D", "S"))
        # keys and values as one projection leaves them: side by side in one row of memory
        kv = torch.randn(B, N, 2, H, D, generator=g, device="cuda") * torch.exp(torch.randn(B, N, 2, H, 1, generator=g, device="cuda"))
        kv = kv.to(DTYPES[case["src"]])
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        if case["cache"] == "e4m3":
            s["buffer"] = torch.zeros(2, B, S, _entry(H, D, "e4m3"), dtype=torch.uint8, device="cuda")
        else:
            s["buffer"] = torch.zeros(2, B, S, H, D, dtype=DTYPES[case["cache"]], device="cuda")
        s["kv_len"] = torch.randint(0, S - N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        s["count"] = _ints(_counts(case)) if case["ragged"] else None
    elif op == "read":
        s["buffer"] = _random_cache(g, case["B"], case["T"], case["H"], case["D"], case["cache"])
        s["length"] = _ints(_lengths(case["B"], case["lo"], case["hi"]))
    elif op == "attention":
        B, N, Hq, H, D = (case[k] for k in ("B", "N", "Hq", "Hkv", "D"))
        s["query"] = (2.0 * torch.randn(B, N, Hq, D, generator=g, device="cuda")).to(DTYPES[case["q"]])
        S = case["hi"] + N + 5
        s["buffer"] = _random_cache(g, B, S, H, D, case["cache"])
        s["prefix"] = _random_cache(g, 1, case["P"], H, D, case["cache"]) if case["P"] else None
        lengths = _lengths(B, case["lo"], case["hi"])
        s["kv_len"] = _ints(lengths)
        # slots that no token has been written to hold whatever was there
        unused = torch.arange(S, device="cuda") >= s["kv_len"][:, None] + N
        s["buffer"][:, unused] = 255 if case["cache"] == "e4m3" else float("nan")
        if case["tree"]:
            i = torch.arange(N, device="cuda")
            back = 1 + (torch.rand(B, N, generator=g, device="cuda") * i.clamp_max(10)).int()
            s["parent"] = (i - back.clamp_max(10)).clamp_min(-1).int().contiguous()
            s["parent"][:, 1:].clamp_min_(0)
            s["parent"][:, 0] = -1
        else:
            s["parent"] = None
    else:
        B, n, V = case["B"], case["npos"], case["V"]
        x = 3.0 * torch.randn(B, n, V, generator=g, device="cuda")
        x[..., : max(1, V // 5000)] += 8.0
        if case["masked"]:
            x[torch.rand(B, n, V, generator=g, device="cuda") < case["masked"]] = float("-inf")
            x[..., V // 2] = 0.0
        s["logits"] = x.to(DTYPES[case["dtype"]])
        s["tokens"] = torch.randint(0, V, (B, n), generator=g, device="cuda", dtype=torch.int32)
        s["tokens"][:, 0] = x[:, 0].argmax(-1).int()
        if case["partial"]:  # a row that emitted fewer tokens than it has positions
            s["tokens"][torch.arange(n, device="cuda") >= _ints(_used(case))[:, None]] = -1
        s["temperature"] = 0.5 + torch.rand(B, generator=g, device="cuda")
    return s


def _used(case):
    return [1 + (5 * b + 2) % case["npos"] if case["partial"] else case["npos"] for b in range(case["B"])]


# -------------------------------------------------------------------- run
def run(s):
    if own:
        import speculative_decoding_verification_32_gb300 as sv

        return {"append": _own_append, "read": _own_read, "attention": _own_attention, "logprobs": _own_logprobs}[s["op"]](sv, s)
    return {"append": _append, "read": _read, "attention": _attention, "logprobs": _logprobs}[s["op"]](s)


def _written(s):
    """What the cache holds, as values: codes and scale exponents, or 16-bit numbers."""
    if s["cache"] != "e4m3":
        return {"entries": s["buffer"]}
    n = s["H"] * s["D"]
    return {"codes": s["buffer"][..., :n].view(torch.float8_e4m3fn), "exponents": s["buffer"][..., n : n + s["H"]]}


def _own_append(sv, s):
    sv.spec_kv_append(s["buffer"], s["k"], s["v"], s["kv_len"], count=s["count"])
    return _written(s)


def _own_read(sv, s):
    k, v, _ = sv.spec_kv_read(s["buffer"], s["length"], s["T"], heads=s["H"], head_dim=s["D"], dtype=DTYPES[s["out"]])
    return k, v


def _own_attention(sv, s):
    out, lse, _ = sv.spec_prefix_attention(s["query"], s["buffer"], s["kv_len"], prefix=s["prefix"], parent=s["parent"], kv_heads=s["Hkv"])
    return out, lse


def _own_logprobs(sv, s):
    r = sv.spec_token_logprobs(s["logits"], s["tokens"], s["temperature"], m=min(s["m"], s["V"]))
    return {k: r[k] for k in ("logprob", "entropy", "top_ids", "top_logprobs")}


def _append(s):
    N, S = s["N"], s["S"]
    x = _pack(torch.stack((s["k"], s["v"])).float(), s["cache"])
    i = torch.arange(N, device="cuda")
    slot = s["kv_len"][:, None] + i
    row = torch.arange(s["B"], device="cuda")[:, None].expand_as(slot)
    if s["count"] is not None:
        keep = i < s["count"][:, None]
        slot, row, x = slot[keep], row[keep], x[:, keep]
    s["buffer"][:, row, slot] = x
    return _written(s)


def _read(s):
    x = _values(s["buffer"], s["H"], s["D"], s["cache"])
    keep = torch.arange(s["T"], device="cuda") < s["length"][:, None]
    x = torch.where(keep[..., None, None], x, 0.0).to(DTYPES[s["out"]])
    return x[0], x[1]


def _visible(kv_len, N, S, parent):
    """[B, N, S]: which of a row's own slots each of its queries sees."""
    slot = torch.arange(S, device="cuda")
    if parent is None:
        last = kv_len[:, None] + torch.arange(N, device="cuda")
        return slot <= last[..., None]
    # a node's ancestors and itself: the powers of (identity + step to the parent)
    step = torch.arange(N, device="cuda") == parent[..., None]
    seen = torch.matrix_power(step.double() + torch.eye(N, device="cuda", dtype=torch.float64), N) > 0
    j = slot - kv_len[:, None]
    inside = ((j >= 0) & (j < N))[:, None, :]
    tree = torch.gather(seen, 2, j.clamp(0, N - 1)[:, None, :].expand(-1, N, -1))
    return (j < 0)[:, None, :] | (inside & tree)


def _attention(s):
    B, N, Hq, H, D = (s[k] for k in ("B", "N", "Hq", "Hkv", "D"))
    G = Hq // H
    S = s["hi"] + N
    q = s["query"].float().unflatten(2, (H, G)) * (1.0 / math.sqrt(D))
    k, v = _values(s["buffer"][:, :, :S], H, D, s["cache"])
    written = (torch.arange(S, device="cuda") < s["kv_len"][:, None] + N)[..., None, None]
    k, v = torch.where(written, k, 0.0), torch.where(written, v, 0.0)
    seen = _visible(s["kv_len"], N, S, s["parent"])
    x = torch.einsum("bnhgd,bshd->bnhgs", q, k)
    x = torch.where(seen[:, :, None, None, :], x, float("-inf"))
    if s["prefix"] is not None:
        kp, vp = _values(s["prefix"][:, 0], H, D, s["cache"])
        x = torch.cat((torch.einsum("bnhgd,phd->bnhgp", q, kp), x), -1)
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    P = s["P"]
    out = torch.einsum("bnhgs,bshd->bnhgd", e[..., P:], v)
    if P:
        out = out + torch.einsum("bnhgp,phd->bnhgd", e[..., :P], vp)
    lse = (top + torch.log(total)).squeeze(-1).flatten(2)
    return (out / total).flatten(2, 3).to(s["query"].dtype), lse


def _logprobs(s):
    x = s["logits"].float()
    V, m = s["V"], min(s["m"], s["V"])
    # order by value, equal values by the lower id: unique 64-bit keys
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long() * (1 << 32) + (V - torch.arange(V, device="cuda"))
    ids = V - (torch.topk(key, m, dim=-1).values & 0xFFFFFFFF)
    y = x / s["temperature"][:, None, None]
    y = y - y.amax(-1, keepdim=True)
    e = torch.exp(y)
    total = e.sum(-1, keepdim=True)
    lp = y - torch.log(total)
    p = e / total
    entropy = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    asked = s["tokens"] >= 0
    nan = float("nan")
    given = torch.gather(lp, 2, s["tokens"].clamp_min(0).long()[..., None]).squeeze(-1)
    return {
        "logprob": torch.where(asked, given, nan),
        "entropy": torch.where(asked, entropy, nan),
        "top_ids": torch.where(asked[..., None], ids, -1).int(),
        "top_logprobs": torch.where(asked[..., None], torch.gather(lp, 2, ids), nan),
    }


# ------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "append":
        values = 2 * sum(_counts(case)) * case["H"] * case["D"]
        entries = 2 * sum(_counts(case)) * _entry(case["H"], case["D"], case["cache"])
        return {"bytes": values * DTYPES[case["src"]].itemsize + entries, "flops": 3 * values}
    if op == "read":
        n = sum(_lengths(case["B"], case["lo"], case["hi"]))
        out = 2 * case["B"] * case["T"] * case["H"] * case["D"] * DTYPES[case["out"]].itemsize
        return {"bytes": 2 * n * _entry(case["H"], case["D"], case["cache"]) + out, "flops": 2 * n * case["H"] * case["D"]}
    if op == "attention":
        B, N = case["B"], case["N"]
        own_keys = sum(_lengths(B, case["lo"], case["hi"]))
        pairs = N * (own_keys + B * case["P"]) + B * N * (N + 1) // 2
        entries = 2 * (case["P"] + own_keys + B * N) * _entry(case["Hkv"], case["D"], case["cache"])
        return {"bytes": entries + 2 * B * N * case["Hq"] * case["D"] * 2 + 4 * B * N * case["Hq"], "flops": 4 * pairs * case["Hq"] * case["D"]}
    n = sum(_used(case))
    return {"bytes": n * case["V"] * DTYPES[case["dtype"]].itemsize + n * (12 + 8 * case["m"]), "flops": 6 * n * case["V"]}


# ------------------------------------------------------------------ exact
def _e4m3(x):
    """x (float64, at most 448 in magnitude) rounded to the e4m3 grid, ties to even."""
    _, e = torch.frexp(x)  # x = f * 2^e with f in [1/2, 1): the grid step is 2^(e - 4), at least 2^-9
    step = torch.exp2((e - 4).clamp_min(-9).double())
    return torch.round(x / step) * step


def _stored(s, entries):
    """float64 values of the cache entries a state holds."""
    H, D = (s["H"], s["D"]) if "H" in s else (s["Hkv"], s["D"])
    if s["cache"] != "e4m3":
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
    op = case["op"]
    if op == "append":
        H, D = case["H"], case["D"]
        kv = torch.stack((s["k"], s["v"])).double()
        if case["cache"] == "e4m3":
            amax = kv.abs().amax(-1, keepdim=True)
            f, e = torch.frexp(amax / 448)  # f in [1/2, 1)
            scale = torch.exp2((e - (f == 0.5).int()).double().clamp_min(-126.0))
            kv = _e4m3(kv / scale)
            to = torch.zeros(2, case["B"], case["S"], H, D, dtype=torch.float64, device="cuda")
        else:
            to = s["buffer"].double()
        counts = _counts(case)
        for b, start in enumerate(s["kv_len"].tolist()):
            to[:, b, start : start + counts[b]] = kv[:, b, : counts[b]]
        return {"codes": to.flatten(-2), "exponents": None} if case["cache"] == "e4m3" else {"entries": to}
    if op == "read":
        x = _stored(s, s["buffer"])
        for b, n in enumerate(s["length"].tolist()):
            x[:, b, n:] = 0.0
        return x[0], x[1]
    if op == "attention":
        return _exact_attention(s)
    return _exact_logprobs(s)


def _exact_attention(s):
    """Row by row: softmax over the keys that a query sees, in 64 bits."""
    B, N, H, D = (s[k] for k in ("B", "N", "Hkv", "D"))
    G = s["Hq"] // H
    out = torch.zeros(B, N, s["Hq"], D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, N, s["Hq"], dtype=torch.float64, device="cuda")
    shared = _stored(s, s["prefix"][:, 0]) if s["prefix"] is not None else None
    parents = s["parent"].tolist() if s["parent"] is not None else [[i - 1 for i in range(N)]] * B
    for b, n in enumerate(s["kv_len"].tolist()):
        mine = _stored(s, s["buffer"][:, b, : n + N])
        hidden = np.ones((N, N), dtype=bool)
        for i in range(N):
            j = i
            while j >= 0:
                hidden[i, j] = False
                j = parents[b][j]
        both = mine if shared is None else torch.cat((shared, mine), 1)
        q = s["query"][b].double().reshape(N, H, G, D).permute(1, 0, 2, 3).reshape(H, N * G, D)
        x = (q @ both[0].permute(1, 2, 0)) / math.sqrt(D)
        x = x.reshape(H, N, G, -1)
        tail = x[..., x.shape[-1] - N :]
        tail.masked_fill_(torch.from_numpy(hidden).cuda()[None, :, None, :], float("-inf"))
        total = torch.logsumexp(x, -1)
        p = torch.exp(x - total[..., None])
        o = p.reshape(H, N * G, -1) @ both[1].permute(1, 0, 2)
        out[b] = o.reshape(H, N, G, D).permute(1, 0, 2, 3).reshape(N, s["Hq"], D)
        lse[b] = total.permute(1, 0, 2).reshape(N, s["Hq"])
    return out, lse


def _exact_logprobs(s):
    B, n, V = s["logits"].shape
    m = min(s["m"], V)
    nan = float("nan")
    lp_out = torch.full((B, n), nan, dtype=torch.float64, device="cuda")
    entropy = lp_out.clone()
    tops = torch.full((B, n, m), nan, dtype=torch.float64, device="cuda")
    tokens = s["tokens"].long()
    for b in range(B):
        lp = torch.log_softmax(s["logits"][b].double() / s["temperature"][b].double(), -1)
        used = tokens[b] >= 0
        lp_out[b] = torch.where(used, lp.gather(1, tokens[b].clamp_min(0)[:, None])[:, 0], nan)
        entropy[b] = torch.where(used, -torch.nan_to_num(lp.exp() * lp, nan=0.0).sum(-1), nan)
        tops[b] = torch.where(used[:, None], torch.topk(lp, m, -1).values, nan)
    return {"logprob": lp_out, "entropy": entropy, "top_ids": None, "top_logprobs": tops}
