"""A serving batch's step through a block as it is measured: cases, inputs, plain forms and the framework's calls.

Four operators:

  quantize  a token's activations as 8-bit integers with one scale
  linear    product of 8-bit integers with scales for each token and each output channel
  select    routing to experts from their logits: sigmoid or softmax scores, bias, groups, top-k, weights
  shared    latent attention of new tokens of sequences that begin with the same cached prefix, each followed by
            tokens of its own, over the paged cache of perf/operators.py
"""
import math
import random

import torch

own = False

ROPE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "f32": 4}


# ---------------------------------------------------------------- cases
def _text(lens):
    return ",".join(str(v) for v in lens)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _spread(seed, n, low, high):
    r = random.Random(seed)
    return [int(round(math.exp(r.uniform(math.log(low), math.log(high))))) for _ in range(n)]


def listed():
    return [
        # one new token's hidden state before its projections: a launch's latency
        {"name": "quantize_token", "op": "quantize", "tokens": 1, "k": 6144, "dtype": "bf16"},
        # a prompt's hidden states, as the MoE layer leaves them
        {"name": "quantize_prompt", "op": "quantize", "tokens": 8191, "k": 6144, "dtype": "f32"},
        # one token's queries: the weights are read once
        {"name": "linear_token", "op": "linear", "tokens": 1, "k": 6144, "n_out": 16384, "dtype": "bf16", "bias": False},
        # a decode batch's attention outputs back to the hidden size
        {"name": "linear_batch", "op": "linear", "tokens": 61, "k": 16384, "n_out": 6144, "dtype": "fp16", "bias": False},
        # logits of a slice of a vocabulary, an odd number of them
        {"name": "linear_head", "op": "linear", "tokens": 133, "k": 6144, "n_out": 19393, "dtype": "f32", "bias": False},
        # a long prompt's queries
        {"name": "linear_prompt", "op": "linear", "tokens": 8192, "k": 6144, "n_out": 16384, "dtype": "bf16", "bias": True},
        # one new token's routing
        {"name": "select_token", "op": "select", "tokens": 1, "experts": 256, "top_k": 8, "groups": 8, "top_groups": 4,
         "softmax": False, "top2": True, "bias": True, "norm": True, "dtype": "f32"},
        # a prompt's routing
        {"name": "select_prompt", "op": "select", "tokens": 16384, "experts": 256, "top_k": 8, "groups": 8,
         "top_groups": 4, "softmax": False, "top2": True, "bias": True, "norm": True, "dtype": "f32"},
        # softmax scores of a 16-bit gate, equal logits among them; groups by their best expert
        {"name": "select_softmax", "op": "select", "tokens": 4099, "experts": 160, "top_k": 6, "groups": 8,
         "top_groups": 3, "softmax": True, "top2": False, "bias": False, "norm": False, "dtype": "bf16"},
        # a few sequences behind a common instruction, few heads
        {"name": "shared_few", "op": "shared", "prefix": 2047, "lens": _text(_spread(3, 7, 8, 200) + [0]), "n_q": 1,
         "heads": 16, "rank": 512, "dtype": "bf16", "fp8": False, "page": 16},
        # a serving batch behind a long instruction
        {"name": "shared_batch", "op": "shared", "prefix": 8192, "lens": _text(_spread(5, 64, 16, 1024)), "n_q": 1,
         "heads": 128, "rank": 512, "dtype": "fp16", "fp8": False, "page": 64},
        # speculative verify of sequences behind one long document, 8-bit cache
        {"name": "shared_verify_fp8", "op": "shared", "prefix": 32768, "lens": _text(_spread(9, 16, 16, 512)), "n_q": 4,
         "heads": 64, "rank": 512, "dtype": "bf16", "fp8": True, "page": 64},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "select", "shared", "shared"])
    if op == "quantize":
        return {"op": op, "tokens": _log(rng, 1, 8191), "k": 16 * _log(rng, 1, 384), "dtype": rng.choice(["bf16", "fp16", "f32"])}
    if op == "linear":
        k, n_out = 16 * _log(rng, 1, 1024), _log(rng, 1, 20000)
        top = 8192 * 6144 * 16384 // (k * n_out)
        return {"op": op, "tokens": _log(rng, 1, min(8192, top)), "k": k, "n_out": n_out,
                "dtype": rng.choice(["bf16", "fp16", "f32"]), "bias": rng.random() < 0.4}
    if op == "select":
        experts = rng.choice([5, 16, 60, 64, 96, 128, 160, 256, 384, 512, 1000])
        groups = rng.choice([g for g in (1, 1, 2, 3, 4, 5, 8, 16) if experts % g == 0])
        top_groups = rng.randrange(1, groups + 1)
        return {"op": op, "tokens": _log(rng, 1, 16384 * 256 // max(256, experts)), "experts": experts,
                "top_k": rng.randrange(1, min(16, experts // groups * top_groups) + 1), "groups": groups,
                "top_groups": top_groups, "softmax": rng.random() < 0.4, "top2": rng.random() < 0.6,
                "bias": rng.random() < 0.6, "norm": rng.random() < 0.6, "dtype": rng.choice(["bf16", "fp16", "f32"])}
    n, n_q, heads = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4, 7]), rng.choice([1, 5, 16, 32, 64, 128])
    own_top = _log(rng, 1, 1024)
    rows = n * n_q * heads
    top = max(64, min(32768, 4096 * 32768 // rows - own_top))
    return {"op": op, "prefix": _log(rng, 1, top), "lens": _text([rng.randrange(0, own_top + 1) for _ in range(n - 1)] + [own_top]),
            "n_q": n_q, "heads": heads, "rank": rng.choice([256, 512]), "dtype": rng.choice(["bf16", "fp16"]),
            "fp8": rng.random() < 0.5, "page": rng.choice([1, 16, 48, 64, 128])}


# ---------------------------------------------------------------- inputs
def _codes(x):
    """Rows of x as codes and scales."""
    s = x.abs().amax(-1) / 127.0
    return (x / s[:, None]).round().clamp(-127, 127).to(torch.int8), s


def _cache(case, gen, dev, lens):
    """A pool of pages with normed latents and rotated keys, and each sequence's pages out of it, in no order; the last
    of `lens` is the shared prefix."""
    dt, page, rank = DTYPES[case["dtype"]], case["page"], case["rank"]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens) - 1, max([1] + need[:-1])), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need[:-1]):
        table[b, :n] = order[at:at + n]
        at += n
    prefix_table = order[at:at + need[-1]].clone()
    if case["fp8"]:
        pages = torch.empty((n_pages, page, rank + 2 * ROPE), dtype=torch.uint8, device=dev)
        x = torch.randn((n_pages, page, rank), generator=gen, device=dev)
        s = x.abs().amax(-1) / 448.0
        pages[..., :rank] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        pages[..., rank:] = torch.randn((n_pages, page, ROPE), generator=gen, device=dev).to(dt).view(torch.uint8)
        return pages, s.reshape(-1).contiguous(), table, prefix_table
    return torch.randn((n_pages, page, rank + ROPE), generator=gen, device=dev).to(dt), None, table, prefix_table


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    st = {"case": case}
    if op == "quantize":
        n, k = case["tokens"], case["k"]
        # hidden states: tokens of different sizes, a few channels far above the others
        x = torch.randn((n, k), generator=gen, device=dev) * (0.5 + torch.rand((n, 1), generator=gen, device=dev))
        x[:, :: 97] *= 8.0
        st["x"] = x.to(dt)
        st["codes"] = torch.zeros((n, k), dtype=torch.int8, device=dev)
        st["scale"] = torch.zeros(n, dtype=torch.float32, device=dev)
    elif op == "linear":
        n, k, n_out = case["tokens"], case["k"], case["n_out"]
        st["codes"], st["scale"] = _codes(torch.randn((n, k), generator=gen, device=dev))
        st["w"], st["w_scale"] = _codes(torch.randn((n_out, k), generator=gen, device=dev) / math.sqrt(k))
        st["bias"] = torch.randn(n_out, generator=gen, device=dev) if case["bias"] else None
        st["out"] = torch.zeros((n, n_out), dtype=dt, device=dev)
    elif op == "select":
        n, e = case["tokens"], case["experts"]
        st["logits"] = (1.5 * torch.randn((n, e), generator=gen, device=dev)).to(dt)
        st["bias"] = 0.05 * torch.randn(e, generator=gen, device=dev) if case["bias"] else None
        st["idx"] = torch.zeros((n, case["top_k"]), dtype=torch.int32, device=dev)
        st["w"] = torch.zeros((n, case["top_k"]), dtype=torch.float32, device=dev)
    else:
        lens = _ints(case["lens"])
        n, h, rank = len(lens) * case["n_q"], case["heads"], case["rank"]
        st["pages"], st["kv_scale"], st["table"], st["prefix_table"] = _cache(case, gen, dev, lens + [case["prefix"]])
        st["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["max_kv"] = max(lens)
        st["scale"] = 1.0 / math.sqrt(192.0)
        st["q_lat"] = torch.randn((n, h, rank), generator=gen, device=dev).to(dt)
        st["q_pe"] = torch.randn((n, h, ROPE), generator=gen, device=dev).to(dt)
        st["out"] = torch.zeros((n, h, rank), dtype=dt, device=dev)
        st["lse"] = torch.zeros((n, h), dtype=torch.float32, device=dev)
    return st


# ---------------------------------------------------------------- plain forms
def _plain_quantize(st):
    # quotients in 64 bits: a code is the integer next to the exact quotient, borders included
    x = st["x"].double()
    st["scale"].copy_(x.abs().amax(-1) / torch.tensor(127.0, dtype=torch.float64, device=x.device))
    s = st["scale"].double()[:, None]
    st["codes"].copy_(torch.where(s > 0, x / s, 0.0).round().clamp(-127, 127))
    return {"codes": st["codes"], "scale": st["scale"]}


def _plain_linear(st):
    # 32 bits of a sum are enough for 16 of its result
    t = torch.float64 if st["out"].dtype == torch.float32 else torch.float32
    out = torch.matmul(st["codes"].to(t), st["w"].to(t).t())
    out = out * st["scale"].to(t)[:, None] * st["w_scale"].to(t)
    if st["bias"] is not None:
        out = out + st["bias"].to(t)
    return st["out"].copy_(out)


def _plain_select(st):
    # in 64 bits: neighbours in rank may differ by less than 32 hold
    c = st["case"]
    logits = st["logits"].double()
    n, e = logits.shape
    if c["softmax"]:
        p = (logits - logits.amax(-1, keepdim=True)).exp()
        score = p / p.sum(-1, keepdim=True)
    else:
        score = 1.0 / (1.0 + (-logits).exp())
    choice = score if st["bias"] is None else score + st["bias"].double()
    if c["groups"] > 1:
        members = choice.view(n, c["groups"], -1)
        best = members.sort(dim=-1, descending=True, stable=True).values
        rank = best[..., :2].sum(-1) if c["top2"] else best[..., 0]
        keep = rank.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        open_ = torch.zeros((n, c["groups"]), dtype=torch.bool, device=logits.device)
        open_.scatter_(1, keep, True)
        choice = members.masked_fill(~open_[..., None], -math.inf).view(n, e)
    idx = choice.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = score.gather(1, idx)
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True)
    st["idx"].copy_(idx)
    st["w"].copy_(w * 2.5)
    return {"idx": st["idx"], "w": st["w"]}


def _rows(st, table, positions):
    """Cached rows in 32 bits: latents and keys at `positions` [.., tokens] of the sequences whose pages `table` holds."""
    c = st["case"]
    page = c["page"]
    pid = table.gather(-1, (positions // page).clamp(max=table.shape[-1] - 1).expand(table.shape[:-1] + positions.shape[-1:])).long()
    x = st["pages"][pid, positions % page]
    if c["fp8"]:
        lat = x[..., :c["rank"]].view(torch.float8_e4m3fn).float() * st["kv_scale"][pid * page + positions % page][..., None]
        return lat, x[..., c["rank"]:].view(DTYPES[c["dtype"]]).float()
    return x[..., :c["rank"]].float(), x[..., c["rank"]:].float()


def _plain_shared(st):
    c = st["case"]
    lens, n_q, h, rank, prefix = st["kv_lens"].long(), c["n_q"], c["heads"], c["rank"], c["prefix"]
    n, dev = lens.numel(), lens.device
    q_lat, q_pe = st["q_lat"].float().view(n * n_q * h, rank), st["q_pe"].float().view(n * n_q * h, ROPE)
    # the prefix: one product for the rows of all sequences
    t = torch.arange(prefix, device=dev)
    p_lat, p_key = _rows(st, st["prefix_table"], t)
    s0 = (torch.matmul(q_lat, p_lat.t()).add_(torch.matmul(q_pe, p_key.t()))).mul_(st["scale"]).view(n, n_q * h, prefix)
    # each sequence's own tokens
    u = torch.arange(max(st["max_kv"], 1), device=dev)
    lat, key = _rows(st, st["table"], u.expand(n, -1))
    inside = (u[None, :] < lens[:, None])[..., None]
    lat, key = lat * inside, key * inside
    s1 = (torch.matmul(q_lat.view(n, n_q * h, rank), lat.transpose(1, 2))
          + torch.matmul(q_pe.view(n, n_q * h, ROPE), key.transpose(1, 2))) * st["scale"]
    # query j of a sequence sees all but the last n_q - 1 - j tokens
    limit = (prefix + lens[:, None] - n_q + 1 + torch.arange(n_q, device=dev)[None]).repeat_interleave(h, 1)[..., None]
    s0.masked_fill_(t >= limit, -math.inf)
    s1.masked_fill_(prefix + u >= limit, -math.inf)
    top = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True))
    top = torch.where(top == -math.inf, 0.0, top)
    s0, s1 = s0.sub_(top).exp_(), s1.sub_(top).exp_()
    total = s0.sum(-1, keepdim=True) + s1.sum(-1, keepdim=True)
    out = torch.matmul(s0.view(-1, prefix), p_lat).view(n, n_q * h, rank) + torch.matmul(s1, lat)
    st["out"].copy_((out / torch.where(total > 0, total, 1.0)).view_as(st["out"]))
    st["lse"].copy_((total.log() + top).view_as(st["lse"]))
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------- the framework's calls
def _own(st):
    import quantized_expert_ffn_amd as moe
    c = st["case"]
    op = c["op"]
    if op == "quantize":
        moe.coli_w8_quantize(st["x"], st["codes"], st["scale"])
        return {"codes": st["codes"], "scale": st["scale"]}
    if op == "linear":
        moe.coli_w8_linear(st["codes"], st["scale"], st["w"], st["w_scale"], st["bias"], st["out"])
        return st["out"]
    if op == "select":
        if "ws" not in st:   # a program keeps its shape and its workspace
            st["dims"] = moe.make_select_dims(
                n_experts=c["experts"], top_k=c["top_k"], n_group=c["groups"], topk_group=c["top_groups"],
                scoring=moe.COLI_SCORE_SOFTMAX if c["softmax"] else moe.COLI_SCORE_SIGMOID,
                group_score=moe.COLI_GROUP_TOP2 if c["top2"] else moe.COLI_GROUP_MAX, norm_topk_prob=c["norm"],
                routed_scaling_factor=2.5)
            st["ws"] = torch.zeros(256, dtype=torch.uint8, device="cuda")
        moe.coli_moe_select(st["dims"], st["logits"], st["bias"], st["idx"], st["w"], st["ws"])
        return {"idx": st["idx"], "w": st["w"]}
    if "ws" not in st:
        st["dims"] = moe.make_mla_dims(
            n_heads=c["heads"], rank=c["rank"], nope=128, v_dim=128, page_size=c["page"], dtype=DTYPES[c["dtype"]],
            kv_format=moe.COLI_KV_E4M3 if c["fp8"] else moe.COLI_KV_PLAIN, softmax_scale=st["scale"])
        st["ws"] = torch.zeros(moe.coli_mla_shared_workspace_bytes(st["dims"], st["kv_lens"].numel(), c["n_q"], c["prefix"],
                                                                   st["max_kv"]), dtype=torch.uint8, device="cuda")
    moe.coli_mla_decode_shared(st["dims"], st["q_lat"], st["q_pe"], st["pages"], st["kv_scale"], st["prefix_table"],
                               c["prefix"], st["table"], st["kv_lens"], st["max_kv"], st["out"], st["lse"], st["ws"])
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"quantize": _plain_quantize, "linear": _plain_linear, "select": _plain_select,
            "shared": _plain_shared}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass needs
def work(case):
    op, size = case["op"], BYTES[case["dtype"]]
    if op == "quantize":
        n, k = case["tokens"], case["k"]
        return {"bytes": n * (k * (size + 1) + 4), "flops": 3 * n * k}
    if op == "linear":
        n, k, m = case["tokens"], case["k"], case["n_out"]
        return {"bytes": (n + m) * (k + 4) + n * m * size + (4 * m if case["bias"] else 0), "flops": 2 * n * k * m}
    if op == "select":
        n, e = case["tokens"], case["experts"]
        return {"bytes": n * (e * size + 8 * case["top_k"]) + (4 * e if case["bias"] else 0), "flops": 8 * n * e}
    lens, n_q, h, rank, prefix = _ints(case["lens"]), case["n_q"], case["heads"], case["rank"], case["prefix"]
    row = rank + 2 * ROPE + 4 if case["fp8"] else 2 * (rank + ROPE)
    seen = sum(max(0, prefix + n - n_q + 1 + j) for n in lens for j in range(n_q))
    return {"bytes": (prefix + sum(lens)) * row + len(lens) * n_q * h * (2 * (2 * rank + ROPE) + 4),
            "flops": 2 * seen * h * (2 * rank + ROPE)}


# ---------------------------------------------------------------- in 64 bits
def _exact_quantize(st):
    x = st["x"].double()
    scale = x.abs().max(dim=1).values / torch.full((1,), 127.0, dtype=torch.float64, device=x.device)
    held = scale.to(torch.float32).double()   # codes are in units of the scale as it is held
    low = torch.div(x, held.where(held > 0, torch.ones_like(held))[:, None]).mul_(2.0)
    # the nearest integer of the quotient, ties to even, by way of its doubled value
    half = torch.floor(low)
    up = torch.floor((half + 1.0) / 2.0)
    tie = (half == low) & (torch.remainder(half, 2.0) == 1.0)
    codes = torch.where(tie & (torch.remainder(up, 2.0) == 1.0), up - 1.0, up)
    codes = torch.minimum(torch.maximum(codes, torch.full_like(codes, -127.0)), torch.full_like(codes, 127.0))
    return {"codes": (codes * (held > 0)[:, None]).to(torch.int8), "scale": scale}


def _exact_linear(st):
    k = st["codes"].shape[1]
    total = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    # 1024 products of codes stay below 2^24, so a sum of them in 32 bits is exact
    for a in range(0, k, 1024):
        total += st["codes"][:, a:a + 1024].float() @ st["w"][:, a:a + 1024].float().t()
    total *= st["w_scale"].double()[None, :]
    total *= st["scale"].double()[:, None]
    return total if st["bias"] is None else total.add_(st["bias"].double()[None, :])


def _exact_select(st):
    c = st["case"]
    x = st["logits"].double()
    score = torch.exp(x - torch.logsumexp(x, -1, keepdim=True)) if c["softmax"] else torch.sigmoid(x)
    choice = score + (0.0 if st["bias"] is None else st["bias"].double())
    size = c["experts"] // c["groups"]
    if c["groups"] > 1:
        rank = []
        for g in range(c["groups"]):
            members = choice[:, g * size:(g + 1) * size]
            first, at = members.max(-1)
            if c["top2"] and size > 1:
                first = first + members.scatter(1, at[:, None], -math.inf).max(-1).values
            rank.append(first)
        rank = torch.stack(rank, -1)
        # a group's place: how many stand before it
        g = torch.arange(c["groups"], device=x.device)
        before = (rank[:, None, :] > rank[:, :, None]) | ((rank[:, None, :] == rank[:, :, None]) & (g[None, None] < g[None, :, None]))
        shut = before.sum(-1) >= c["top_groups"]
        choice = choice.masked_fill(shut.repeat_interleave(size, 1), -math.inf)
    rows = torch.arange(x.shape[0], device=x.device)
    idx = torch.empty((x.shape[0], c["top_k"]), dtype=torch.int64, device=x.device)
    e = torch.arange(c["experts"], device=x.device)
    for i in range(c["top_k"]):
        top = choice.max(-1, keepdim=True).values
        at = torch.where(choice == top, e, c["experts"]).min(-1).values
        idx[:, i] = at
        choice = choice.index_put((rows, at), torch.tensor(-math.inf, dtype=torch.float64, device=x.device))
    w = score[rows[:, None], idx]
    if c["norm"]:
        w = w / w.sum(1)[:, None]
    return {"idx": idx.to(torch.int32), "w": 2.5 * w}


def _exact_shared(st):
    c = st["case"]
    page, rank, n_q, prefix = c["page"], c["rank"], c["n_q"], c["prefix"]
    if c["fp8"]:
        rows = st["pages"].view(-1, rank + 2 * ROPE)
        lat = rows[:, :rank].contiguous().view(torch.float8_e4m3fn).double() * st["kv_scale"].double()[:, None]
        key = rows[:, rank:].contiguous().view(DTYPES[c["dtype"]]).double()
    else:
        rows = st["pages"].view(-1, rank + ROPE).double()
        lat, key = rows[:, :rank], rows[:, rank:]

    def slots(pages, n):
        return (pages.long()[:, None] * page + torch.arange(page, device=pages.device)).flatten()[:n]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    before = slots(st["prefix_table"], prefix)
    for b, n in enumerate(_ints(c["lens"])):
        at = torch.cat([before, slots(st["table"][b], n)])
        x, k = lat[at], key[at]
        for j in range(n_q):
            m = prefix + n - n_q + 1 + j
            if m > 0:
                r = b * n_q + j
                s = (st["q_lat"][r].double() @ x[:m].t() + st["q_pe"][r].double() @ k[:m].t()) * st["scale"]
                lse[r] = torch.logsumexp(s, -1)
                out[r] = (s - lse[r][:, None]).exp() @ x[:m]
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return {"quantize": _exact_quantize, "linear": _exact_linear, "select": _exact_select,
            "shared": _exact_shared}[case["op"]](st)
