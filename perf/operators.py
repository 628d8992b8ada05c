"""Latent attention as it is measured: cases, inputs, plain forms and the calls of the framework's operators.

Five operators make the attention that stands before the MoE layer of a block:

  append   RMS norm of the latent, rotation of the shared key and of the queries, write into the paged cache
  project  per-head products: queries into the latent space, attention outputs out of it
  decode   attention of a few new tokens a sequence over the paged latents (absorbed form)
  expand   keys and values of every head out of the paged latents
  prefill  attention of a prompt over expanded keys and values, ragged batches, causal

The cache holds `rank` latent values and 64 rotated key values a token, in the activations' type, or as E4M3
codes with one binary32 scale a token beside rotated keys in the activations' type.
"""
import math
import random

import torch

own = False

ROPE = 64
EPS = 1e-6
THETA = 10000.0
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------- cases
def _text(lens):
    return ",".join(str(v) for v in lens)


def _ints(text):
    return [int(v) for v in text.split(",")]


def _spread(seed, n, low, high):
    r = random.Random(seed)
    return [int(round(math.exp(r.uniform(math.log(low), math.log(high))))) for _ in range(n)]


def listed():
    batch = _spread(7, 62, 16, 8192) + [8192, 0]
    verify = _spread(11, 16, 2048, 16384)
    return [
        # one decode step's append: a launch's latency
        {"name": "append_one", "op": "append", "tokens": 1, "heads": 64, "rank": 512, "dtype": "bf16", "fp8": False,
         "page": 64, "pages": 64, "norm": True, "halves": False},
        # a prompt's append into the 8-bit cache, a few padding tokens in it
        {"name": "append_prompt_fp8", "op": "append", "tokens": 8191, "heads": 64, "rank": 512, "dtype": "bf16",
         "fp8": True, "page": 64, "pages": 256, "norm": True, "halves": True},
        # absorption of one token's queries: streams the weights
        {"name": "project_one", "op": "project", "tokens": 1, "heads": 64, "n_in": 192, "n_out": 512, "dtype": "bf16"},
        # outputs of a mid-sized decode batch out of the latent space
        {"name": "project_batch", "op": "project", "tokens": 133, "heads": 128, "n_in": 512, "n_out": 128,
         "dtype": "fp16"},
        # one token early in a conversation: latency
        {"name": "decode_short", "op": "decode", "lens": "1023", "n_q": 1, "heads": 16, "rank": 512, "dtype": "bf16",
         "fp8": False, "page": 16},
        # one token of one long conversation: the work has to be split over the cache
        {"name": "decode_long", "op": "decode", "lens": "131071", "n_q": 1, "heads": 64, "rank": 512, "dtype": "bf16",
         "fp8": False, "page": 64},
        # a serving batch of uneven lengths, one slot of it empty
        {"name": "decode_batch", "op": "decode", "lens": _text(batch), "n_q": 1, "heads": 128, "rank": 512,
         "dtype": "fp16", "fp8": False, "page": 64},
        # speculative verify: four tokens a sequence, 8-bit cache
        {"name": "decode_verify_fp8", "op": "decode", "lens": _text(verify), "n_q": 4, "heads": 64, "rank": 512,
         "dtype": "bf16", "fp8": True, "page": 64},
        # a ragged batch's keys and values out of the 8-bit cache
        {"name": "expand_ragged_fp8", "op": "expand", "lens": "333,1,0,700", "heads": 64, "rank": 512, "nope": 192,
         "v": 256, "dtype": "bf16", "fp8": True, "page": 64},
        # a long prompt's keys and values
        {"name": "expand_prompt", "op": "expand", "lens": "8192", "heads": 64, "rank": 512, "nope": 192, "v": 256,
         "dtype": "bf16", "fp8": False, "page": 64},
        # short prompts of a batch, two of them behind cached prefixes
        {"name": "prefill_ragged", "op": "prefill", "q_lens": "1,77,300,513", "k_lens": "1,777,300,1500", "heads": 32,
         "nope": 128, "v": 128, "dtype": "fp16", "causal": True},
        # one long prompt
        {"name": "prefill_prompt", "op": "prefill", "q_lens": "8192", "k_lens": "8192", "heads": 64, "nope": 192,
         "v": 256, "dtype": "bf16", "causal": True},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "project", "decode", "expand", "prefill"])
    c = {"op": op, "dtype": rng.choice(["bf16", "fp16"])}
    if op == "append":
        c |= {"tokens": _log(rng, 1, 8191), "heads": rng.choice([1, 5, 16, 32, 64, 128]), "rank": rng.choice([256, 512]),
              "fp8": rng.random() < 0.5, "page": rng.choice([1, 16, 48, 64, 128]), "norm": rng.random() < 0.7,
              "halves": rng.random() < 0.5}
        c["pages"] = (c["tokens"] + rng.randrange(1, 500)) // c["page"] + 2
    elif op == "project":
        n_in, n_out = rng.choice([(128, 512), (192, 512), (512, 128), (512, 256), (128, 256), (256, 128)])
        c |= {"tokens": _log(rng, 1, 2048), "heads": rng.choice([1, 5, 16, 32, 64, 128]), "n_in": n_in, "n_out": n_out}
    elif op == "decode":
        n = _log(rng, 1, 64)
        top = _log(rng, 16, 131072 // n)
        lens = [rng.randrange(0, top + 1) for _ in range(n - 1)] + [top]
        c |= {"lens": _text(lens), "n_q": rng.choice([1, 1, 1, 2, 4, 7]), "heads": rng.choice([1, 5, 16, 32, 64, 128]),
              "rank": rng.choice([256, 512]), "fp8": rng.random() < 0.5, "page": rng.choice([1, 16, 48, 64, 128])}
    elif op == "expand":
        n = _log(rng, 1, 16)
        top = _log(rng, 1, 8192 // n)
        nope, v = rng.choice([(128, 128), (192, 256)])
        c |= {"lens": _text([rng.randrange(0, top + 1) for _ in range(n - 1)] + [top]), "nope": nope, "v": v,
              "heads": rng.choice([1, 5, 32, 64]), "rank": rng.choice([256, 512]), "fp8": rng.random() < 0.5,
              "page": rng.choice([1, 16, 48, 64, 128])}
    else:
        n = _log(rng, 1, 8)
        top = _log(rng, 1, 8192 // n)
        q_lens = [rng.randrange(0, top + 1) for _ in range(n - 1)] + [top]
        nope, v = rng.choice([(128, 128), (192, 256)])
        more = rng.random() < 0.4
        k_lens = [min(8192 // n, m + rng.randrange(0, 1024)) if more else m for m in q_lens]
        c |= {"q_lens": _text(q_lens), "k_lens": _text(k_lens), "heads": rng.choice([1, 5, 32, 64]), "nope": nope,
              "v": v, "causal": rng.random() < 0.8}
    return c


# ---------------------------------------------------------------- inputs
def _cumulative(lens, dev):
    t = torch.zeros(len(lens) + 1, dtype=torch.int32)
    t[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return t.to(dev)


def _cache(case, gen, dev, lens):
    """A pool of pages with normed latents and rotated keys, and each sequence's pages out of it, in no order."""
    dt, page, rank = DTYPES[case["dtype"]], case["page"], case["rank"]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    width = max(1, max(need))
    order = torch.randperm(n_pages, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros((len(lens), width), dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if case["fp8"]:
        pages = torch.empty((n_pages, page, rank + 2 * ROPE), dtype=torch.uint8, device=dev)
        x = torch.randn((n_pages, page, rank), generator=gen, device=dev)
        s = x.abs().amax(-1) / 448.0
        pages[..., :rank] = (x / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        pages[..., rank:] = torch.randn((n_pages, page, ROPE), generator=gen, device=dev).to(dt).view(torch.uint8)
        scale = s.reshape(-1).contiguous()
    else:
        pages = torch.randn((n_pages, page, rank + ROPE), generator=gen, device=dev).to(dt)
        scale = None
    return pages, scale, table


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op = case["op"]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev).to(dt)

    st = {"case": case, "scale": 1.0 / math.sqrt(192.0)}
    if op == "append":
        n, h, rank = case["tokens"], case["heads"], case["rank"]
        slots_all = case["pages"] * case["page"]
        st["kv_a"] = randn(n, rank + ROPE)
        st["norm_w"] = (1.0 + 0.1 * torch.randn(rank, generator=gen, device=dev)).to(dt) if case["norm"] else None
        # positions of a long conversation; slots are distinct, every 97th token is padding
        st["positions"] = (torch.arange(n, device=dev) + 100000).to(torch.int32)
        slots = torch.randperm(slots_all, generator=gen, device=dev)[:n].to(torch.int64)
        slots[96::97] = -1
        st["slots"] = slots
        st["inv_freq"] = THETA ** (-torch.arange(0, ROPE, 2, device=dev, dtype=torch.float64) / ROPE)
        q = randn(n, h, 128 + ROPE)
        st["q_pe"] = q[..., 128:]   # the rotated part of whole queries
        st["q_pe_out"] = torch.zeros((n, h, ROPE), dtype=dt, device=dev)
        if case["fp8"]:
            st["pages"] = torch.randint(0, 64, (case["pages"], case["page"], rank + 2 * ROPE), generator=gen, device=dev,
                                        dtype=torch.uint8)
            st["kv_scale"] = torch.rand(slots_all, generator=gen, device=dev)
        else:
            st["pages"] = randn(case["pages"], case["page"], rank + ROPE)
            st["kv_scale"] = None
    elif op == "project":
        n, h = case["tokens"], case["heads"]
        st["x"] = randn(n, h, case["n_in"])
        st["w"] = (torch.randn((h, case["n_out"], case["n_in"]), generator=gen, device=dev)
                   / math.sqrt(case["n_in"])).to(dt)
        st["out"] = torch.zeros((n, h, case["n_out"]), dtype=dt, device=dev)
    elif op == "decode":
        lens = _ints(case["lens"])
        n, h, rank = len(lens) * case["n_q"], case["heads"], case["rank"]
        st["pages"], st["kv_scale"], st["table"] = _cache(case, gen, dev, lens)
        st["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["max_kv"] = max(lens)
        st["q_lat"] = randn(n, h, rank)
        st["q_pe"] = randn(n, h, ROPE)
        st["out"] = torch.zeros((n, h, rank), dtype=dt, device=dev)
        st["lse"] = torch.zeros((n, h), dtype=torch.float32, device=dev)
    elif op == "expand":
        lens = _ints(case["lens"])
        n, h, wide = sum(lens), case["heads"], case["nope"] + case["v"]
        st["pages"], st["kv_scale"], st["table"] = _cache(case, gen, dev, lens)
        st["cu_k"] = _cumulative(lens, dev)
        st["w"] = (torch.randn((h, wide, case["rank"]), generator=gen, device=dev) / math.sqrt(case["rank"])).to(dt)
        st["kv"] = torch.zeros((n, h, wide), dtype=dt, device=dev)
        st["k_pe"] = torch.zeros((n, ROPE), dtype=dt, device=dev)
    else:
        q_lens, k_lens = _ints(case["q_lens"]), _ints(case["k_lens"])
        h, nope, v = case["heads"], case["nope"], case["v"]
        st["q"] = randn(sum(q_lens), h, nope + ROPE)
        kv = randn(sum(k_lens), h, nope + v)   # as the expansion leaves them
        st["k_nope"], st["v"] = kv[..., :nope], kv[..., nope:]
        st["k_pe"] = randn(sum(k_lens), ROPE)
        st["cu_q"], st["cu_k"] = _cumulative(q_lens, dev), _cumulative(k_lens, dev)
        st["max_q"], st["max_k"] = max(q_lens), max(k_lens)
        st["scale"] = 1.0 / math.sqrt(nope + ROPE)
        st["out"] = torch.zeros((sum(q_lens), h, v), dtype=dt, device=dev)
        st["lse"] = torch.zeros((sum(q_lens), h), dtype=torch.float32, device=dev)
    return st


# ---------------------------------------------------------------- plain forms
def _rotate(x, positions, inv_freq, halves):
    """x [n, ..., 64] in 32 bits; the angles in 64 (a far position times a frequency loses its fraction in 32)."""
    a = positions.double()[:, None] * inv_freq
    shape = (x.shape[0],) + (1,) * (x.dim() - 2) + (ROPE // 2,)
    c, s = a.cos().float().view(shape), a.sin().float().view(shape)
    if halves:
        a, b = x[..., :ROPE // 2], x[..., ROPE // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)


def _append_outputs(st):
    c = st["case"]
    pages = st["pages"]
    if c["fp8"]:
        return {"codes": pages[..., :c["rank"]].view(torch.float8_e4m3fn),
                "keys": pages[..., c["rank"]:].view(DTYPES[c["dtype"]]), "scale": st["kv_scale"], "q_pe": st["q_pe_out"]}
    return {"pages": pages, "q_pe": st["q_pe_out"]}


def _plain_append(st):
    c, dt = st["case"], DTYPES[st["case"]["dtype"]]
    rank = c["rank"]
    x = st["kv_a"][:, :rank].float()
    if st["norm_w"] is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * st["norm_w"].float()
    k = _rotate(st["kv_a"][:, rank:].float(), st["positions"], st["inv_freq"], c["halves"]).to(dt)
    st["q_pe_out"].copy_(_rotate(st["q_pe"].float(), st["positions"], st["inv_freq"], c["halves"]))
    used = st["slots"] >= 0
    slots = st["slots"][used]
    if c["fp8"]:
        rows = st["pages"].view(-1, rank + 2 * ROPE)
        s = x.abs().amax(-1) / 448.0
        codes = torch.where(s[:, None] > 0, x / s[:, None], 0.0).to(torch.float8_e4m3fn)
        rows[slots] = torch.cat([codes.view(torch.uint8), k.view(torch.uint8)], -1)[used]
        st["kv_scale"][slots] = s[used]
    else:
        rows = st["pages"].view(-1, rank + ROPE)
        rows[slots] = torch.cat([x.to(dt), k], -1)[used]
    return _append_outputs(st)


def _plain_project(st):
    out = torch.matmul(st["x"].float().transpose(0, 1), st["w"].float().transpose(1, 2)).transpose(0, 1)
    return st["out"].copy_(out)


def _rows(st, positions, batch):
    """Cached rows in 32 bits: latents and keys at `positions` of the sequences `batch` (tensors of one shape)."""
    c = st["case"]
    page = c["page"]
    pid = st["table"][batch, positions // page].long()
    x = st["pages"][pid, positions % page]
    if c["fp8"]:
        lat = x[..., :c["rank"]].view(torch.float8_e4m3fn).float() * st["kv_scale"][pid * page + positions % page][..., None]
        return lat, x[..., c["rank"]:].view(DTYPES[c["dtype"]]).float()
    return x[..., :c["rank"]].float(), x[..., c["rank"]:].float()


def _softmax(s, seen):
    """exp(s - max) / sum and the log of the sum; a row that sees nothing gives zeros and -inf."""
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (s - top).exp_()
    total = p.sum(-1, keepdim=True)
    lse = (total.log() + top).squeeze(-1)
    return p.div_(torch.where(total > 0, total, 1.0)), lse


def _plain_decode(st):
    c = st["case"]
    lens, n_q, h = st["kv_lens"].long(), c["n_q"], c["heads"]
    n = lens.numel()
    dev = lens.device
    t = torch.arange(max(st["max_kv"], 1), device=dev)
    lat, key = _rows(st, t[None].expand(n, -1).clamp(max=st["table"].shape[1] * c["page"] - 1), torch.arange(n, device=dev)[:, None])
    inside = t[None, :] < lens[:, None]
    lat, key = lat * inside[..., None], key * inside[..., None]
    q_lat = st["q_lat"].float().view(n, n_q * h, -1)
    q_pe = st["q_pe"].float().view(n, n_q * h, -1)
    s = (torch.matmul(q_lat, lat.transpose(1, 2)) + torch.matmul(q_pe, key.transpose(1, 2))) * st["scale"]
    limit = lens[:, None] - n_q + 1 + torch.arange(n_q, device=dev)[None]
    seen = t[None, None, :] < limit.repeat_interleave(h, 1)[..., None]
    p, lse = _softmax(s, seen)
    st["out"].copy_(torch.matmul(p, lat).view_as(st["out"]))
    st["lse"].copy_(lse.view_as(st["lse"]))
    return {"out": st["out"], "lse": st["lse"]}


def _plain_expand(st):
    n = st["kv"].shape[0]
    at = torch.arange(n, device=st["kv"].device)
    cu = st["cu_k"].long()
    b = torch.searchsorted(cu, at, right=True) - 1
    lat, key = _rows(st, at - cu[b], b)
    st["kv"].copy_(torch.matmul(lat, st["w"].float().flatten(0, 1).t()).view_as(st["kv"]))
    st["k_pe"].copy_(key)
    return {"kv": st["kv"], "k_pe": st["k_pe"]}


def _padded(x, cu, width):
    """[batch, width, ...] of a ragged [rows, ...] in 32 bits, zeros behind each length."""
    cu = cu.long()
    at = torch.arange(width, device=x.device)
    inside = at[None] < (cu[1:] - cu[:-1])[:, None]
    rows = (cu[:-1, None] + at[None]).clamp(max=x.shape[0] - 1)
    return x[rows].float() * inside.view(inside.shape + (1,) * (x.dim() - 1)), inside, rows


def _plain_prefill(st):
    cu_q, cu_k = st["cu_q"], st["cu_k"]
    q, q_in, _ = _padded(st["q"], cu_q, st["max_q"])
    k, _, _ = _padded(torch.cat([st["k_nope"], st["k_pe"][:, None].expand(-1, st["k_nope"].shape[1], -1)], -1), cu_k, max(st["max_k"], 1))
    v, k_in, _ = _padded(st["v"], cu_k, max(st["max_k"], 1))
    q, k, v = q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["scale"])
    seen = k_in[:, None, None, :]
    if st["case"]["causal"]:
        n_q, n_k = (cu_q[1:] - cu_q[:-1]).long(), (cu_k[1:] - cu_k[:-1]).long()
        i = torch.arange(st["max_q"], device=q.device)
        j = torch.arange(k.shape[2], device=q.device)
        seen = seen & (j[None, None] <= i[None, :, None] + (n_k - n_q)[:, None, None])[:, None]
    p, lse = _softmax(s, seen)
    st["out"].copy_(torch.matmul(p, v).transpose(1, 2)[q_in])
    st["lse"].copy_(lse.transpose(1, 2)[q_in])
    return {"out": st["out"], "lse": st["lse"]}


# ---------------------------------------------------------------- the framework's calls
def _own(st):
    import quantized_expert_ffn_amd as moe
    c = st["case"]
    op = c["op"]
    if op == "project":
        moe.coli_mla_project(st["x"], st["w"], st["out"])
        return st["out"]
    if "ws" not in st:   # a program keeps its shape and its workspace
        st["dims"] = moe.make_mla_dims(
            n_heads=c["heads"], rank=c.get("rank", 512), nope=c.get("nope", 128), v_dim=c.get("v", 128),
            page_size=c.get("page", 64), dtype=DTYPES[c["dtype"]],
            kv_format=moe.COLI_KV_E4M3 if c.get("fp8") else moe.COLI_KV_PLAIN,
            rope_style=moe.COLI_ROPE_HALVES if c.get("halves") else moe.COLI_ROPE_PAIRS, norm_eps=EPS,
            softmax_scale=st["scale"])
        batch = st["kv_lens"].numel() if op == "decode" else 0
        st["ws"] = torch.zeros(moe.coli_mla_workspace_bytes(st["dims"], batch, c.get("n_q", 1), st.get("max_kv", 0)),
                               dtype=torch.uint8, device="cuda")
    d, ws = st["dims"], st["ws"]
    if op == "append":
        moe.coli_mla_append(d, st["kv_a"], st["norm_w"], st["positions"], st["slots"], st["inv_freq"], st["q_pe"],
                            st["q_pe_out"], st["pages"], st["kv_scale"], ws)
        return _append_outputs(st)
    if op == "decode":
        moe.coli_mla_decode(d, st["q_lat"], st["q_pe"], st["pages"], st["kv_scale"], st["table"], st["kv_lens"],
                            st["max_kv"], st["out"], st["lse"], ws)
        return {"out": st["out"], "lse": st["lse"]}
    if op == "expand":
        moe.coli_mla_expand(d, st["pages"], st["kv_scale"], st["table"], st["cu_k"], st["w"], st["kv"], st["k_pe"], ws)
        return {"kv": st["kv"], "k_pe": st["k_pe"]}
    moe.coli_mla_prefill(d, st["q"], st["k_nope"], st["k_pe"], st["v"], st["cu_q"], st["cu_k"], st["max_q"],
                         c["causal"], st["out"], st["lse"], ws)
    return {"out": st["out"], "lse": st["lse"]}


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "project": _plain_project, "decode": _plain_decode, "expand": _plain_expand,
            "prefill": _plain_prefill}[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass needs
def _pairs(case):
    n = 0
    for a, b in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
        if not case["causal"]:
            n += a * b
        else:
            first = max(0, a - b)   # queries before the first key see nothing
            rows = a - first
            low = max(0, b - a) + 1
            n += rows * (low + low + rows - 1) // 2
    return n


def work(case):
    op, rank = case["op"], case.get("rank", 512)
    row = rank + 2 * ROPE + 4 if case.get("fp8") else 2 * (rank + ROPE)
    if op == "append":
        n, h = case["tokens"], case["heads"]
        return {"bytes": n * (2 * (rank + ROPE) + row + 4 * h * ROPE + 12) + 8 * ROPE // 2 + 2 * rank * case["norm"],
                "flops": n * (6 * rank + 3 * ROPE * (h + 1))}
    if op == "project":
        n, h, a, b = case["tokens"], case["heads"], case["n_in"], case["n_out"]
        return {"bytes": 2 * h * (a * b + n * (a + b)), "flops": 2 * n * h * a * b}
    if op == "decode":
        lens, h, n_q = _ints(case["lens"]), case["heads"], case["n_q"]
        rows = sum(max(0, n - n_q + 1 + j) for n in lens for j in range(n_q))
        return {"bytes": sum(lens) * row + len(lens) * n_q * h * (2 * (2 * rank + ROPE) + 4),
                "flops": 2 * rows * h * (2 * rank + ROPE)}
    if op == "expand":
        n, h, wide = sum(_ints(case["lens"])), case["heads"], case["nope"] + case["v"]
        return {"bytes": n * (row + 2 * ROPE + 2 * h * wide) + 2 * h * wide * rank, "flops": 2 * n * h * wide * rank}
    n_q, n_k, h = sum(_ints(case["q_lens"])), sum(_ints(case["k_lens"])), case["heads"]
    nope, v = case["nope"], case["v"]
    return {"bytes": 2 * n_q * h * (nope + ROPE + v) + 4 * n_q * h + 2 * n_k * (h * (nope + v) + ROPE),
            "flops": 2 * _pairs(case) * h * (nope + ROPE + v)}


# ---------------------------------------------------------------- in 64 bits
def _exact_rotate(x, positions, inv_freq, halves):
    """Each pair as a complex number, turned by the angle."""
    z = x.double()
    half = ROPE // 2
    z = torch.complex(z[..., :half], z[..., half:]) if halves else torch.view_as_complex(z.unflatten(-1, (half, 2)).contiguous())
    a = torch.outer(positions.double(), inv_freq.double())
    turn = torch.polar(torch.ones_like(a), a)
    z = z * (turn if z.dim() == 2 else turn[:, None])
    return torch.cat([z.real, z.imag], -1) if halves else torch.view_as_real(z).flatten(-2)


def _exact_cache(st):
    """Latents and keys of every slot, in 64 bits."""
    c = st["case"]
    if c["fp8"]:
        rows = st["pages"].view(-1, c["rank"] + 2 * ROPE)
        lat = rows[:, :c["rank"]].contiguous().view(torch.float8_e4m3fn).double() * st["kv_scale"].double()[:, None]
        return lat, rows[:, c["rank"]:].contiguous().view(DTYPES[c["dtype"]]).double()
    rows = st["pages"].view(-1, c["rank"] + ROPE).double()
    return rows[:, :c["rank"]], rows[:, c["rank"]:]


def _exact_slots(st, b, n):
    t = torch.arange(n, device=st["table"].device)
    return st["table"][b].long()[t // st["case"]["page"]] * st["case"]["page"] + t % st["case"]["page"]


def _exact_attend(s, values):
    """s [rows, keys] with -inf where a key is not seen."""
    lse = torch.logsumexp(s, -1) if s.shape[-1] else torch.full(s.shape[:-1], -math.inf, dtype=s.dtype, device=s.device)
    w = torch.where(lse[..., None] > -math.inf, (s - lse[..., None]).exp(), 0.0)
    return w @ values, lse


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "append":
        rank = case["rank"]
        x = st["kv_a"].double()
        lat = x[:, :rank]
        if case["norm"]:
            lat = lat / (lat.pow(2).sum(-1, keepdim=True) / rank + EPS).sqrt() * st["norm_w"].double()
        key = _exact_rotate(x[:, rank:], st["positions"], st["inv_freq"], case["halves"])
        q_pe = _exact_rotate(st["q_pe"], st["positions"], st["inv_freq"], case["halves"])
        keep = torch.nonzero(st["slots"] >= 0).squeeze(-1)
        slots = st["slots"][keep]
        if case["fp8"]:
            codes = st["pages"][..., :rank].contiguous().view(torch.float8_e4m3fn).double().view(-1, rank)
            keys = st["pages"][..., rank:].contiguous().view(DTYPES[case["dtype"]]).double().view(-1, ROPE)
            scale = st["kv_scale"].double()
            top = lat.abs().amax(-1) / 448.0
            q = lat / torch.where(top > 0, top, 1.0)[:, None]
            # a code holds 4 significant bits, down to steps of 2^-9
            step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
            codes[slots], keys[slots], scale[slots] = ((q / step).round() * step)[keep], key[keep], top[keep]
            shape = st["pages"].shape[:2]
            return {"codes": codes.view(*shape, rank), "keys": keys.view(*shape, ROPE), "scale": scale, "q_pe": q_pe}
        rows = st["pages"].double()
        rows.view(-1, rank + ROPE)[slots] = torch.cat([lat, key], -1)[keep]
        return {"pages": rows, "q_pe": q_pe}
    if op == "project":
        out = torch.empty((case["tokens"], case["heads"], case["n_out"]), dtype=torch.float64, device="cuda")
        for h in range(case["heads"]):
            out[:, h] = st["x"][:, h].double() @ st["w"][h].double().t()
        return out
    if op == "decode":
        lat, key = _exact_cache(st)
        out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
        lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
        n_q = case["n_q"]
        for b, n in enumerate(_ints(case["lens"])):
            at = _exact_slots(st, b, n)
            c, k = lat[at], key[at]
            for j in range(n_q):
                m = n - n_q + 1 + j
                if m > 0:
                    r = b * n_q + j
                    s = (st["q_lat"][r].double() @ c[:m].t() + st["q_pe"][r].double() @ k[:m].t()) * st["scale"]
                    out[r], lse[r] = _exact_attend(s, c[:m])
        return {"out": out, "lse": lse}
    if op == "expand":
        lat, key = _exact_cache(st)
        at = torch.cat([_exact_slots(st, b, n) for b, n in enumerate(_ints(case["lens"]))])
        kv = torch.empty(st["kv"].shape, dtype=torch.float64, device="cuda")
        for h in range(case["heads"]):
            kv[:, h] = lat[at] @ st["w"][h].double().t()
        return {"kv": kv, "k_pe": key[at]}
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for n, m in zip(_ints(case["q_lens"]), _ints(case["k_lens"])):
        if case["causal"]:
            i, j = torch.arange(n, device="cuda")[:, None], torch.arange(m, device="cuda")[None]
            hidden = j - (m - n) > i
        else:
            hidden = torch.zeros((n, m), dtype=torch.bool, device="cuda")
        for h in range(case["heads"]):
            q, pe = st["q"][q0:q0 + n, h].double(), st["k_pe"][k0:k0 + m].double()
            s = (q[:, :case["nope"]] @ st["k_nope"][k0:k0 + m, h].double().t() + q[:, case["nope"]:] @ pe.t()) * st["scale"]
            out[q0:q0 + n, h], lse[q0:q0 + n, h] = _exact_attend(s.masked_fill_(hidden, -math.inf),
                                                                 st["v"][k0:k0 + m, h].double())
        q0, k0 = q0 + n, k0 + m
    return {"out": out, "lse": lse}
