"""Workloads of the paged K/V cache and of draft verification.

Three operators, each as the calls a user makes of the library and as a plain form in
elementary torch operations:

* ``attend``: attention of the newest 1 to 4 tokens of every sequence over a paged K/V cache;
* ``write``, ``read`` and ``write_read``: quantising K/V rows into pages as they are written
  and reading them back as f16 rows;
* ``verify``: verification of drafted tokens against the target's probabilities from given
  random numbers.

A case is a dict of plain values. ``prepare`` makes its inputs on the GPU, ``run`` makes one
pass and ``exact`` gives the pass's outputs from the operators' definitions in 64 bits.
"""
import math
import random

import torch

own = False

FORMATS = {"f16": 0, "fp8": 1, "int4": 2}
GROUP = 32          # dims that share one scale of an int4 row
ACCEPT = 0.75       # how often one draft of prepare()'s distributions is accepted, about


def listed():
    heads = dict(n_q_heads=32, n_kv_heads=4, head_dim=128)
    rows = dict(n_kv_heads=4, head_dim=128)
    return [
        # the tiny decode configuration: one short sequence, all launch latency
        dict(name="attend 1k f16", op="attend", n_seqs=1, max_len=1024, n_queries=1, n_q_heads=8, n_kv_heads=1,
             head_dim=64, page_size=16, fmt="f16"),
        # one long sequence of the 128k layer
        dict(name="attend 126k f16", op="attend", n_seqs=1, max_len=126253, n_queries=1, page_size=64, fmt="f16", **heads),
        # one long sequence of the 256k layer with the 8-bit cache
        dict(name="attend 255k fp8", op="attend", n_seqs=1, max_len=255181, n_queries=1, page_size=64, fmt="fp8", **heads),
        # a serving batch of very different lengths, one new token each
        dict(name="attend batch fp8", op="attend", n_seqs=128, max_len=8192, n_queries=1, page_size=16, fmt="fp8", **heads),
        # a verification step of a batch: the newest token and three drafts each, 4-bit cache
        dict(name="attend drafts int4", op="attend", n_seqs=24, max_len=32768, n_queries=4, page_size=32, fmt="int4", **heads),
        # the decode step of a batch writes one token of each sequence
        dict(name="write tokens fp8", op="write", n_seqs=64, max_rows=1, max_len=2048, page_size=16, fmt="fp8", **rows),
        # the prompt of the 64k layer, written at once
        dict(name="write prompt fp8", op="write", n_seqs=1, max_rows=61789, max_len=61789, page_size=64, fmt="fp8", **rows),
        # chunks of several prompts stored in 4 bits, and what the next chunk's attention reads of them
        dict(name="write and read int4", op="write_read", n_seqs=8, max_rows=16384, max_len=16384, page_size=32, fmt="int4", **rows),
        # a stored sequence of the 128k layer taken out of the 8-bit cache
        dict(name="read 126k fp8", op="read", n_seqs=1, max_rows=126253, max_len=126253, page_size=64, fmt="fp8", **rows),
        # one sequence, drafts looked up in the text so far (they have no probabilities)
        dict(name="verify one looked up", op="verify", n_seqs=1, n_drafts=3, vocab=32000, drafter=False),
        # a serving batch with a drafting model
        dict(name="verify batch", op="verify", n_seqs=64, n_drafts=3, vocab=151936, drafter=True),
        # a large batch with long drafts and an odd vocabulary
        dict(name="verify large batch", op="verify", n_seqs=256, n_drafts=7, vocab=100003, drafter=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "write", "write_read", "read", "verify", "verify"])
    if op == "verify":
        n_seqs, n_drafts = _log(rng, 1, 256), rng.randint(1, 7)
        return dict(op=op, n_seqs=n_seqs, n_drafts=n_drafts, drafter=rng.random() < 0.7,
                    vocab=min(_log(rng, 257, 200000), 200_000_000 // (n_seqs * (n_drafts + 1))))
    n_kv_heads, head_dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    # int4 codes are looked at as the values they stand for: what is read back after the write
    fmt = rng.choice(["f16", "fp8", "fp8" if op == "write" else "int4"])
    case = dict(op=op, n_kv_heads=n_kv_heads, head_dim=head_dim, page_size=rng.choice([16, 32, 64, 128]), fmt=fmt,
                n_seqs=_log(rng, 1, 128))
    row = n_kv_heads * head_dim
    if op == "attend":
        case["n_q_heads"] = n_kv_heads * rng.randint(1, 8)
        case["n_queries"] = rng.choice([1, 1, 1, 2, 3, 4])
        # as many tokens as the longest listed sequences and batches hold
        case["max_len"] = min(_log(rng, 1, 255181), max(1, 126253 * 512 // (row * case["n_seqs"]) * 2))
    else:
        case["max_rows"] = min(_log(rng, 1, 126253), max(1, 61789 * 512 // (row * case["n_seqs"])))
        case["max_len"] = case["max_rows"] + rng.randint(0, 100)
    return case


# ------------------------------------------------------------------ inputs

def _lengths(case, most):
    """The sequences' lengths of a case: uneven, the first one the longest; among many of
    them one of no tokens and one of a single token."""
    rng = random.Random(case["n_seqs"] * 1000003 + most)
    lens = [most] + [rng.randint(most // 8, most) for _ in range(case["n_seqs"] - 1)]
    if case["n_seqs"] >= 8:
        lens[3], lens[5] = 0, 1
    return lens


def _rows_and_firsts(case):
    """(rows to write or read, position of the first of them) of every sequence."""
    rng = random.Random(case["n_seqs"] + case["max_len"])
    rows = [1] * case["n_seqs"] if case["max_rows"] == 1 else _lengths(case, case["max_rows"])
    return rows, [rng.randint(0, case["max_len"] - r) for r in rows]


def _quantise(x, fmt):
    """The codes and scales that rows x [..., D] f16 are stored as (scales None for f16)."""
    if fmt == "f16":
        return x, None
    if fmt == "fp8":   # one f32 scale a row
        amax = x.abs().amax(-1, keepdim=True).float()
        zero = amax == 0
        scale = torch.where(zero, torch.ones_like(amax), amax / 448.0)
        inv = torch.where(zero, torch.zeros_like(amax), 448.0 / amax)
        return (x.float() * inv).to(torch.float8_e4m3fn), scale.squeeze(-1)
    g = x.reshape(*x.shape[:-1], -1, GROUP).float()   # int4: one f16 scale a group
    scale = (g.abs().amax(-1) / 7.0).half()
    s = scale.float().unsqueeze(-1)
    codes = torch.where(s == 0, torch.zeros_like(g), torch.round(g * (1.0 / s))).clamp(-7, 7) + 8
    lo, hi = codes[..., :GROUP // 2].to(torch.uint8), codes[..., GROUP // 2:].to(torch.uint8)
    return (lo | (hi << 4)).reshape(*x.shape[:-1], -1), scale


def _values(codes, scales, fmt):
    """The f32 values that stored rows stand for."""
    if fmt == "f16":
        return codes.float()
    if fmt == "fp8":
        return codes.float() * scales.unsqueeze(-1)
    c = codes.reshape(*codes.shape[:-1], -1, GROUP // 2)
    c = torch.cat([c & 15, c >> 4], -1).half() - 8
    return (c * scales.unsqueeze(-1)).reshape(*codes.shape[:-1], -1).float()   # the product rounded to f16


def _paged_state(case, lens, g):
    """Pages for sequences of these lengths, in an order of their own in a pool that holds more."""
    fmt, page, heads, dim = case["fmt"], case["page_size"], case["n_kv_heads"], case["head_dim"]
    width = max(1, -(-max(lens) // page))
    used = [-(-n // page) for n in lens]
    n_pages = sum(used) + sum(used) // 16 + 8
    order = torch.randperm(n_pages, generator=g, device="cuda").int()
    table = torch.zeros(case["n_seqs"], width, dtype=torch.int32, device="cuda")
    at = torch.cumsum(torch.tensor([0] + used[:-1], device="cuda"), 0)[:, None] + torch.arange(width, device="cuda")
    held = torch.arange(width, device="cuda") < torch.tensor(used, device="cuda")[:, None]
    table[held] = order[at[held]]
    state = dict(case=case, table=table)
    for name in ("k", "v"):   # what was stored before is in the pages already
        x = torch.randn(n_pages, heads, page, dim, generator=g, device="cuda", dtype=torch.float16)
        state[name + "_pages"], state[name + "_scales"] = _quantise(x, fmt)
    state["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        import sparse_attention_decode_02_b200 as Q
        state["cache"] = Q.PagedKV(state["k_pages"], state["v_pages"], FORMATS[fmt], state["k_scales"], state["v_scales"])
    return state


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "attend":
        lens = _lengths(case, case["max_len"])
        s = _paged_state(case, lens, g)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        shape = (case["n_seqs"], case["n_queries"], case["n_q_heads"], case["head_dim"])
        s["q"] = torch.randn(shape, generator=g, device="cuda", dtype=torch.float16)
        s["out"] = torch.empty(shape, dtype=torch.float32, device="cuda")
        s["lse"] = torch.empty(shape[:3], dtype=torch.float32, device="cuda")
        if own:
            s["workspace"] = torch.empty(s["cache"].workspace_bytes(case["n_q_heads"], case["n_queries"]),
                                         dtype=torch.uint8, device="cuda")
        return s
    if case["op"] != "verify":
        rows, firsts = _rows_and_firsts(case)
        s = _paged_state(case, [f + r for f, r in zip(firsts, rows)], g)
        s["first"] = torch.tensor(firsts, dtype=torch.int32, device="cuda")
        s["row_start"] = torch.tensor([sum(rows[:i]) for i in range(len(rows) + 1)], dtype=torch.int32, device="cuda")
        shape = (sum(rows), case["n_kv_heads"], case["head_dim"])
        if case["op"] != "read":
            s["k"], s["v"] = (torch.randn(shape, generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
        if case["op"] != "write":
            s["k_out"], s["v_out"] = (torch.empty(shape, dtype=torch.float16, device="cuda") for _ in range(2))
        return s
    n, k, vocab = case["n_seqs"], case["n_drafts"], case["vocab"]
    # probabilities as peaked as a language model's, the drafter's near the target's
    logits = torch.randn(n, k + 1, vocab, generator=g, device="cuda") * 3
    s = dict(case=case, target=torch.softmax(logits, -1), draft=None)
    if case["drafter"]:
        noise = torch.randn(n, k, vocab, generator=g, device="cuda") * 0.6
        s["draft"] = torch.softmax(logits[:, :k] + noise, -1)
        drawn = torch.multinomial(s["draft"].reshape(n * k, vocab), 1, generator=g)
    else:
        drawn = torch.multinomial(torch.softmax(logits[:, :k] * 2, -1).reshape(n * k, vocab), 1, generator=g)
    s["tokens"] = drawn.reshape(n, k).int()
    s["uniforms"] = torch.rand(n, k + 1, generator=g, device="cuda")
    s["accepted"], s["next"] = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if case["op"] == "attend":
        if own:
            state["cache"].attend(state["q"], state["table"], state["lens"], state["out"], state["workspace"],
                                  lse=state["lse"], status=state["status"])
            return dict(out=state["out"], lse=state["lse"])
        return _attend(state)
    if case["op"] == "verify":
        if own:
            import sparse_attention_decode_02_b200 as Q
            Q.verify_drafts(state["target"], state["draft"], state["tokens"], state["uniforms"], state["accepted"],
                            state["next"], status=state["status"])
            return dict(accepted=state["accepted"], next=state["next"])
        return _verify(state)
    got = {}
    if case["op"] != "read":
        if own:
            state["cache"].write(state["k"], state["v"], state["table"], state["first"], state["row_start"],
                                 status=state["status"])
        else:
            _write(state)
    if case["op"] == "write":
        got = dict(k_pages=state["k_pages"], v_pages=state["v_pages"])
    if case["op"] != "read" and case["fmt"] != "f16":
        got.update(k_scales=state["k_scales"], v_scales=state["v_scales"])
    if case["op"] != "write":
        if own:
            state["cache"].read(state["k_out"], state["v_out"], state["table"], state["first"], state["row_start"],
                                status=state["status"])
        else:
            _read(state)
        got.update(k=state["k_out"], v=state["v_out"])
    return got


def _attend(s):
    case = s["case"]
    n, t, hq, dim = s["q"].shape
    hkv = case["n_kv_heads"]
    length = s["table"].shape[1] * case["page_size"]

    def rows(name):   # [n, hkv, length, dim] in 32 bits
        pages, scales = s[name + "_pages"][s["table"].long()], s[name + "_scales"]
        x = _values(pages, None if scales is None else scales[s["table"].long()], case["fmt"])
        return x.transpose(1, 2).reshape(n, hkv, length, dim)

    q = s["q"].float().reshape(n, t, hkv, hq // hkv, dim).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, dim)
    logits = torch.matmul(q, rows("k").transpose(-1, -2)) / math.sqrt(dim)
    sees = s["lens"][:, None] - t + 1 + torch.arange(t, device="cuda")               # [n, t] cells
    mask = torch.arange(length, device="cuda") < sees[..., None]                     # [n, t, length]
    mask = mask[:, None, :, None].expand(n, hkv, t, hq // hkv, length).reshape(n, hkv, -1, length)
    logits = logits.masked_fill(~mask, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, rows("v")) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (torch.log(total) + top).squeeze(-1)
    back = lambda x: x.reshape(n, hkv, t, hq // hkv, -1).permute(0, 2, 1, 3, 4).reshape(n, t, hq, -1)  # noqa: E731
    return dict(out=back(out), lse=back(lse).squeeze(-1))


def _slots(s):
    """(page, head, place in the page) of every row of a write or a read, to index pages with."""
    case = s["case"]
    row = torch.arange(s["k" if "k" in s else "k_out"].shape[0], device="cuda")
    seq = torch.searchsorted(s["row_start"].long(), row, right=True) - 1
    at = s["first"].long()[seq] + row - s["row_start"].long()[seq]
    page = s["table"].long()[seq, at // case["page_size"]]
    return page[:, None], torch.arange(case["n_kv_heads"], device="cuda")[None], (at % case["page_size"])[:, None]


def _write(s):
    at, fmt = _slots(s), s["case"]["fmt"]
    for name in ("k", "v"):
        codes, scales = _quantise(s[name], fmt)
        if fmt == "fp8":
            s[name + "_pages"].view(torch.uint8)[at] = codes.view(torch.uint8)
        else:
            s[name + "_pages"][at] = codes
        if scales is not None:
            s[name + "_scales"][at] = scales


def _read(s):
    at, fmt = _slots(s), s["case"]["fmt"]
    for name in ("k", "v"):
        scales = s[name + "_scales"]
        codes = s[name + "_pages"].view(torch.uint8)[at].view(torch.float8_e4m3fn) if fmt == "fp8" else s[name + "_pages"][at]
        s[name + "_out"].copy_(_values(codes, None if scales is None else scales[at], fmt).half())


def _verify(s):
    p, q, d, u = s["target"], s["draft"], s["tokens"].long(), s["uniforms"]
    n, k = d.shape
    pd = p[:, :k].gather(-1, d[..., None]).squeeze(-1).double()
    qd = torch.ones_like(pd) if q is None else q.gather(-1, d[..., None]).squeeze(-1).double()
    kept = torch.cumprod((u[:, :k].double() * qd < pd).long(), -1)
    accepted = kept.sum(-1)
    each, last = torch.arange(n, device="cuda"), torch.clamp(accepted, max=k - 1)
    w = p[each, accepted].double()
    if q is None:
        less = torch.zeros_like(w).scatter_(-1, d[each, last][:, None], 1.0)
        # a draft without probabilities is certain: what is left of the target is the others
        w = torch.where((accepted < k)[:, None] & (less > 0), torch.zeros_like(w), w)
    else:
        w = torch.where((accepted < k)[:, None], torch.clamp(w - q[each, last].double(), min=0.0), w)
    upto = torch.cumsum(w, -1)
    t = u[:, k].double() * upto[:, -1]
    token = (upto <= t[:, None]).sum(-1).clamp(max=w.shape[-1] - 1)
    token = torch.where(upto[:, -1] > 0, token, p[each, accepted].argmax(-1))
    return dict(accepted=accepted.int(), next=token.int())


# ------------------------------------------------------------------ what a pass cannot do without

def _row_bytes(case):
    dim = case["head_dim"]
    return {"f16": 2 * dim, "fp8": dim + 4, "int4": dim // 2 + dim // GROUP * 2}[case["fmt"]]


def work(case):
    if case["op"] == "verify":
        # the rows of the first rejected draft, or the row after the last draft
        all_kept = ACCEPT ** case["n_drafts"]
        rows = 2 - all_kept if case["drafter"] else 1
        small = case["n_seqs"] * (case["n_drafts"] * (16 if case["drafter"] else 12) + 12)
        return {"bytes": case["n_seqs"] * rows * case["vocab"] * 4 + small, "flops": 2 * case["n_seqs"] * case["vocab"]}
    if case["op"] == "attend":
        cells = sum(_lengths(case, case["max_len"]))
        heads = case["n_seqs"] * case["n_queries"] * case["n_q_heads"]
        per_seq = -(-case["max_len"] // case["page_size"]) * 4 + 4
        return {"bytes": 2 * cells * case["n_kv_heads"] * _row_bytes(case) + heads * (6 * case["head_dim"] + 4)
                + case["n_seqs"] * per_seq,
                "flops": 4 * cells * case["n_queries"] * case["n_q_heads"] * case["head_dim"]}
    rows = sum(_rows_and_firsts(case)[0])
    once = 2 * rows * case["n_kv_heads"] * (_row_bytes(case) + 2 * case["head_dim"])
    return {"bytes": once * (2 if case["op"] == "write_read" else 1) + 8 * case["n_seqs"],
            "flops": 4 * rows * case["n_kv_heads"] * case["head_dim"]}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_values(codes, scales, fmt):
    if fmt == "f16":
        return codes.double()
    if fmt == "fp8":
        return codes.double() * scales.double()[..., None]
    low = (codes % 16).double() - 8
    high = torch.div(codes, 16, rounding_mode="floor").double() - 8
    dims = codes.shape[-1] * 2
    x = torch.empty(*codes.shape[:-1], dims, dtype=torch.float64, device=codes.device)
    d = torch.arange(dims // 2, device=codes.device)
    x[..., d // 16 * 32 + d % 16] = low
    x[..., d // 16 * 32 + 16 + d % 16] = high
    # a value of this format is the product rounded to f16 (exact in 64 bits before that)
    return (x * scales.double().repeat_interleave(GROUP, -1)).half().double()


def _exact_quantise(x, fmt):
    """The values codes stand for without their scale, and the scales, of rows x f16."""
    x = x.double()
    if fmt == "f16":
        return x, None
    if fmt == "fp8":
        amax = x.abs().amax(-1, keepdim=True)
        scale = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        y = x / scale
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -20))), min=-6) - 3)
        return torch.round(y / step) * step, scale.squeeze(-1)
    g = x.unflatten(-1, (-1, GROUP))
    scale = (g.abs().amax(-1) / 7).half().double()
    unit = torch.where(scale > 0, scale, torch.ones_like(scale))[..., None]
    return (torch.round(g / unit).clamp(-7, 7) * (scale[..., None] > 0)).flatten(-2), scale


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    if case["op"] == "attend":
        return _exact_attend(s)
    fmt, page = case["fmt"], case["page_size"]
    got = {}
    rows, firsts = _rows_and_firsts(case)
    table = s["table"].tolist()
    place = [(table[i][pos // page], pos % page) for i in range(case["n_seqs"]) for pos in range(firsts[i], firsts[i] + rows[i])]
    place = torch.tensor(place, dtype=torch.long, device="cuda").reshape(-1, 2)
    for name in ("k", "v"):
        pages, scales = s[name + "_pages"], s[name + "_scales"]
        if case["op"] == "read":
            codes = pages.view(torch.uint8) if fmt == "fp8" else pages
            codes = codes.transpose(1, 2)[place[:, 0], place[:, 1]]
            codes = codes.view(torch.float8_e4m3fn) if fmt == "fp8" else codes
            got[name] = _exact_values(codes, None if scales is None else scales.transpose(1, 2)[place[:, 0], place[:, 1]], fmt)
            continue
        values, new = _exact_quantise(s[name], fmt)
        if case["op"] == "write":
            whole = pages.double()
            whole.transpose(1, 2)[place[:, 0], place[:, 1]] = values
            got[name + "_pages"] = whole
        if fmt != "f16":
            whole = scales.double()
            whole.transpose(1, 2)[place[:, 0], place[:, 1]] = new
            got[name + "_scales"] = whole
        if case["op"] == "write_read":
            if fmt == "fp8":
                values = values * new[..., None]
            elif fmt == "int4":
                values = values * new.repeat_interleave(GROUP, -1)
            got[name] = values
    return got


def _exact_attend(s):
    case, page = s["case"], s["case"]["page_size"]
    n, t, hq, dim = s["q"].shape
    group = hq // case["n_kv_heads"]
    out = torch.zeros(n, t, hq, dim, dtype=torch.float64, device="cuda")
    lse = torch.full((n, t, hq), -math.inf, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        ids = s["table"][i, : -(-length // page)].long()
        k, v = (_exact_values(s[x + "_pages"][ids], None if s[x + "_scales"] is None else s[x + "_scales"][ids], case["fmt"])
                for x in ("k", "v"))
        for u in range(t):
            cells = length - t + u + 1
            for h in range(case["n_kv_heads"] if cells > 0 else 0):
                keys, vals = k[:, h].flatten(0, 1)[:cells], v[:, h].flatten(0, 1)[:cells]
                z = s["q"][i, u, h * group:(h + 1) * group].double() @ keys.T / dim ** 0.5
                lse[i, u, h * group:(h + 1) * group] = torch.logsumexp(z, -1)
                out[i, u, h * group:(h + 1) * group] = torch.softmax(z, -1) @ vals
    return dict(out=out, lse=lse)


def _exact_verify(s):
    n, k = s["tokens"].shape
    tokens, accepted, following = s["tokens"].tolist(), [], []
    for i in range(n):
        m = 0
        while m < k:
            d = tokens[i][m]
            q = 1.0 if s["draft"] is None else float(s["draft"][i, m, d])
            if not float(s["uniforms"][i, m]) * q < float(s["target"][i, m, d]):
                break
            m += 1
        left = s["target"][i, m].double()
        if m < k and s["draft"] is not None:
            left = (left - s["draft"][i, m].double()).clamp(min=0)
        elif m < k:
            left[tokens[i][m]] = 0
        upto = left.cumsum(0)
        found = torch.nonzero(upto > float(s["uniforms"][i, k]) * upto[-1])
        accepted.append(m)
        following.append(int(found[0]) if len(found) else int(s["target"][i, m].argmax()))
    return dict(accepted=torch.tensor(accepted, dtype=torch.int32), next=torch.tensor(following, dtype=torch.int32))
