"""Cases and plain forms of the paged decode operators: the block map, the indexer's logits, and attention over the cache.

A sparse-attention step makes, for each new token (a "row"), a place in the paged cache, a score for every cached token,
the selection of the best of them, and attention over the selection. The selection is ``topk_ragged``; the three operators
here are the calls around it. Every case is one call of one of them.
"""
import math

import torch

own = False

F16, BF16, F8 = "float16", "bfloat16", "float8_e4m3fn"


def listed():
    return [
        # the map of one decode step: a new token for each of 64 requests; latency alone
        dict(name="map_decode", op="map", requests=64, ctx_lo=8192, ctx_hi=32768, new_lo=1, new_hi=1, block=64),
        # the map of a mixed step: 512 requests of which many bring a piece of their prompt; small pages
        dict(name="map_mixed", op="map", requests=512, ctx_lo=0, ctx_hi=8192, new_lo=1, new_hi=4096, block=16),
        # scores of a few short requests: latency
        dict(name="logits_small", op="logits", requests=8, next_n=1, prefill=False, len_lo=1, len_hi=4096, heads=32, dim=128, dtype=BF16, block=64),
        # scores of a decode batch over an 8-bit key cache with a scale for each token
        dict(name="logits_batch_f8", op="logits", requests=64, next_n=1, prefill=False, len_lo=8192, len_hi=32768, heads=64, dim=128, dtype=F8, block=64),
        # scores of long requests with one drafted token each: two rows read the same keys
        dict(name="logits_mtp", op="logits", requests=32, next_n=2, prefill=False, len_lo=100000, len_hi=160000, heads=64, dim=128, dtype=BF16, block=64),
        # scores of a prompt's piece: 512 rows of one request, each with a length of its own
        dict(name="logits_prefill", op="logits", requests=1, next_n=512, prefill=True, len_lo=15872, len_hi=15872, heads=64, dim=128, dtype=F16, block=64),
        # latent attention of a few short requests over 512 selected tokens: latency
        dict(name="latent_small", op="attention", requests=4, next_n=1, prefill=False, len_lo=1, len_hi=4096, heads=16, kv_heads=1, dk=576, dv=512, latent=True, topk=512, dtype=BF16, block=64),
        # latent attention of a decode batch over 2048 selected tokens, all 128 heads on this GPU
        dict(name="latent_batch", op="attention", requests=64, next_n=1, prefill=False, len_lo=8192, len_hi=32768, heads=128, kv_heads=1, dk=576, dv=512, latent=True, topk=2048, dtype=BF16, block=64),
        # long requests with a drafted token, 1024 selected tokens, the 16 heads of one GPU out of eight
        dict(name="latent_mtp", op="attention", requests=32, next_n=2, prefill=False, len_lo=100000, len_hi=160000, heads=16, kv_heads=1, dk=576, dv=512, latent=True, topk=1024, dtype=F16, block=64),
        # a prompt's piece: 1024 rows of one request, each over its own 2048 tokens
        dict(name="latent_prefill", op="attention", requests=1, next_n=1024, prefill=True, len_lo=15360, len_hi=15360, heads=64, kv_heads=1, dk=576, dv=512, latent=True, topk=2048, dtype=BF16, block=64),
        # latent attention over everything cached: a layer without selection, with a drafted token
        dict(name="latent_dense", op="attention", requests=16, next_n=2, prefill=False, len_lo=8192, len_hi=32768, heads=128, kv_heads=1, dk=576, dv=512, latent=True, topk=0, dtype=BF16, block=64),
        # grouped heads with separate keys and values over everything cached
        dict(name="grouped_dense", op="attention", requests=64, next_n=1, prefill=False, len_lo=8192, len_hi=32768, heads=32, kv_heads=4, dk=128, dv=128, latent=False, topk=0, dtype=F16, block=16),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["map", "logits", "logits", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 64, 128])
    if op == "map":
        lo = rng.choice([0, 1, 100])
        return dict(op="map", requests=_log(rng, 1, 512), ctx_lo=lo, ctx_hi=lo + _log(rng, 1, 32768), new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, 4096), block=block)
    prefill = rng.random() < 0.25
    hi = _log(rng, 64, 16384 if prefill else 160000)
    case = dict(op=op, requests=1 if prefill else _log(rng, 1, 64), next_n=_log(rng, 16, 1024 if op == "attention" else 512) if prefill else rng.choice([1, 1, 2, 3]),
                prefill=prefill, len_lo=hi if prefill else rng.choice([1, max(1, hi // 4), max(1, hi // 2)]), len_hi=hi)
    if op == "logits":
        case.update(heads=rng.choice([8, 16, 32, 64]), dim=rng.choice([64, 128]), dtype=rng.choice([F16, BF16, F8]), block=block)
    elif rng.random() < 0.65 or prefill:
        case.update(heads=rng.choice([8, 16, 32, 64, 128]), kv_heads=1, dk=576, dv=512, latent=True, topk=rng.choice([512, 1024, 2048, _log(rng, 1, 2048)]), dtype=rng.choice([F16, BF16]), block=block)
        if not prefill and rng.random() < 0.3:
            case["topk"] = 0
    else:
        kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        case.update(heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, dk=dim, dv=dim, latent=False, topk=rng.choice([0, 0, 1024]), dtype=rng.choice([F16, BF16]), block=block)
    # no dearer than the largest listed ones, in the work and in what the plain form holds
    while (lambda w: w["bytes"] > 1.5e9 or w["flops"] > 1.2e11)(work(case)) or _padded(case) > 6e9:
        case["len_hi"] = max(64, case["len_hi"] * 7 // 8)
        case["len_lo"] = case["len_hi"] if prefill else min(case["len_lo"], case["len_hi"])
        if case["requests"] > 1:
            case["requests"] = max(1, case["requests"] * 7 // 8)
        elif prefill:
            case["next_n"] = max(16, case["next_n"] * 7 // 8)
    return case


def _padded(case):
    """About the largest number of bytes that the plain form holds in one tensor."""
    rows, length = case["requests"] * case["next_n"], case["len_hi"] + (case["next_n"] if case["prefill"] else 0)
    if case["op"] == "logits":
        return 4 * rows * length * max(case["heads"], case["dim"])
    return 4 * rows * (min(case["topk"], length) if case["topk"] else length) * max(case["heads"], case["kv_heads"] * case["dk"])


def work(case):
    if case["op"] == "map":
        requests = case["requests"]
        tokens = requests * (case["new_lo"] + case["new_hi"]) / 2
        return {"bytes": 16 * tokens + 12 * requests + 4 * (requests + 1) + 8 * tokens / case["block"], "flops": 0}
    requests, next_n = case["requests"], case["next_n"]
    rows = requests * next_n
    mean = (case["len_lo"] + case["len_hi"]) / 2 + (next_n - 1) / 2
    if case["op"] == "logits":
        e = 1 if case["dtype"] == F8 else 2
        cached = requests * mean * (case["dim"] * e + (4 if e == 1 else 0))
        return {"bytes": cached + rows * (4 * mean + case["heads"] * (case["dim"] * e + 4)), "flops": 2 * rows * mean * case["heads"] * case["dim"]}
    read = min(case["topk"], mean) if case["topk"] else mean
    each = 2 * case["kv_heads"] * (case["dk"] + (0 if case["latent"] else case["dv"]))
    cached = min(rows * read, requests * mean) * each
    return {"bytes": cached + rows * (case["heads"] * (2 * (case["dk"] + case["dv"]) + 4) + 4 * case["topk"]), "flops": 2 * rows * read * case["heads"] * (case["dk"] + case["dv"])}


def _dtype(case):
    return getattr(torch, case["dtype"])


def _table(g, lengths, block, columns):
    """A block table for these lengths, its pages in a random order, and the number of pages."""
    used = (lengths + block - 1) // block
    total = int(used.sum())
    order = torch.randperm(total + 3, generator=g, device="cuda", dtype=torch.int32)
    col = torch.arange(columns, device="cuda")
    at = (torch.cumsum(used, 0) - used)[:, None] + col
    return torch.where(col < used[:, None], order[at.clamp(max=total + 2)], -1).to(torch.int32).contiguous(), total + 3


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int64)

    def normal(shape, dtype):
        if dtype == torch.float8_e4m3fn:
            return torch.randn(shape, generator=g, device="cuda", dtype=torch.float16).to(dtype)
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    state = {"case": case}
    if own:
        import sparse_attention_row_gb300 as sar
        state["decoder"] = sar.PagedDecoder(torch.cuda.current_device())
    if case["op"] == "map":
        requests, block = case["requests"], case["block"]
        context = whole(case["ctx_lo"], case["ctx_hi"], requests)
        new = whole(case["new_lo"], case["new_hi"], requests)
        columns = (case["ctx_hi"] + case["new_hi"] + block - 1) // block
        table, held = _table(g, context, block, columns)
        free = held + torch.randperm(requests * ((case["new_hi"] + block - 1) // block + 1) + 7, generator=g, device="cuda", dtype=torch.int32)
        state.update(context=context.int(), new=new.int(), table=table, free=free, taken=torch.full((1,), 5, dtype=torch.int32, device="cuda"),
                     taken_out=torch.zeros(1, dtype=torch.int32, device="cuda"), max_tokens=requests * case["new_hi"] + 1)
        return state
    requests, next_n, block, dtype = case["requests"], case["next_n"], case["block"], _dtype(case)
    rows = requests * next_n
    base = whole(case["len_lo"], case["len_hi"], requests)
    lengths = (base[:, None] + torch.arange(next_n, device="cuda")).reshape(-1)
    longest = case["len_hi"] + next_n - 1
    table, blocks = _table(g, base + next_n - 1, block, (longest + block - 1) // block)
    state.update(table=table, lengths=lengths.int(), longest=longest, row_request=torch.zeros(rows, dtype=torch.int32, device="cuda") if case["prefill"] else None)
    if case["op"] == "logits":
        state.update(q=normal((rows, case["heads"], case["dim"]), dtype), keys=normal((blocks, block, case["dim"]), dtype),
                     weights=normal((rows, case["heads"]), torch.float32) / case["heads"],
                     scales=0.5 + torch.rand((blocks, block), generator=g, device="cuda") if case["dtype"] == F8 else None,
                     out=torch.full((rows, longest), -math.inf, device="cuda"))
        return state
    state.update(q=normal((rows, case["heads"], case["dk"]), dtype), k=normal((blocks, block, case["kv_heads"], case["dk"]), dtype),
                 v=None if case["latent"] else normal((blocks, block, case["kv_heads"], case["dv"]), dtype), scale=case["dk"] ** -0.5, indices=None)
    if case["topk"]:
        state["indices"] = _selection(g, lengths, longest, case["topk"])
    return state


def _selection(g, lengths, longest, topk):
    """Distinct positions below each length, in no order, -1 past them: what the selection leaves."""
    chance = torch.rand((lengths.numel(), max(longest, topk)), generator=g, device="cuda")
    chance.masked_fill_(torch.arange(chance.shape[1], device="cuda") >= lengths[:, None], -1.0)
    value, index = torch.topk(chance, topk, dim=1, sorted=False)
    order = torch.argsort((value < 0).to(torch.int8), dim=1, stable=True)
    return torch.where(value < 0, -1, index).gather(1, order).to(torch.int32).contiguous()


def run(state):
    case = state["case"]
    if own:
        if case["op"] == "map":
            m = state["decoder"].kv_map(state["context"], state["new"], state["table"], state["free"], state["taken"], case["block"], state["max_tokens"], taken_out=state["taken_out"])
            return {"table": state["table"], "taken": state["taken_out"], "slots": m.slots, "row_lens": m.row_lens, "row_request": m.row_request, "token_start": m.token_start}
        if case["op"] == "logits":
            return state["decoder"].index_logits(state["q"], state["weights"], state["keys"], state["table"], state["lengths"], key_scales=state["scales"],
                                                 next_n=case["next_n"], row_request=state["row_request"], out=state["out"])
        out, lse = state["decoder"].attention(state["q"], state["k"], state["table"], state["lengths"], v_cache=state["v"], v_dim=case["dv"], indices=state["indices"],
                                              scale=state["scale"], next_n=case["next_n"], row_request=state["row_request"], return_lse=True)
        return {"out": out, "lse": lse}
    if case["op"] == "map":
        return _plain_map(state, case["block"])
    if case["op"] == "logits":
        return _plain_logits(state, case["next_n"])
    return _plain_attention(state, case)


def _plain_map(state, block):
    context, new, table, free = state["context"].long(), state["new"].long(), state["table"], state["free"]
    columns, tokens = table.shape[1], state["max_tokens"]
    cur = ((context + block - 1) // block).clamp(max=columns)
    need = torch.maximum(((context + new + block - 1) // block).clamp(max=columns), cur)
    first = torch.cumsum(need - cur, 0) - (need - cur) + state["taken"]
    col = torch.arange(columns, device="cuda")
    at = first[:, None] + col - cur[:, None]
    block_id = torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1)
    table = torch.where((col >= cur[:, None]) & (col < need[:, None]), block_id, table)
    ends = torch.cumsum(new, 0)
    t = torch.arange(tokens, device="cuda")
    request = torch.searchsorted(ends, t, right=True)
    real = request < context.numel()
    r = request.clamp(max=context.numel() - 1)
    pos = context[r] + t - (ends - new)[r]
    page = table[r, (pos // block).clamp(max=columns - 1)].long()
    slots = torch.where(real & (pos // block < columns) & (page >= 0), page * block + pos % block, -1)
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    return {"table": table, "taken": (state["taken"] + (need - cur).sum()).clamp(max=free.numel()).int(), "slots": slots, "row_lens": torch.where(real, pos + 1, 0).int(),
            "row_request": torch.where(real, r, -1).int(), "token_start": torch.cat([zero, ends]).int()}


def _slots(table, request, pos, block):
    """Flat cache positions of these tokens; of the first page's first token where the table has none."""
    page = table[request[:, None], (pos // block).clamp(0, table.shape[1] - 1)].long()
    return (page * block + pos % block).clamp(min=0)


def _request(state, next_n):
    rows = state["lengths"].numel()
    return state["row_request"].long() if state["row_request"] is not None else torch.arange(rows, device="cuda") // next_n


def _plain_logits(state, next_n):
    keys, lengths = state["keys"], state["lengths"]
    pos = torch.arange(state["longest"], device="cuda").expand(lengths.numel(), -1)
    slot = _slots(state["table"], _request(state, next_n), pos, keys.shape[1])
    k = keys.flatten(0, 1).to(torch.float32)[slot]
    score = torch.relu(torch.matmul(state["q"].to(torch.float32), k.transpose(1, 2)))
    total = torch.matmul(state["weights"][:, None], score)[:, 0]
    if state["scales"] is not None:
        total = total * state["scales"].flatten()[slot]
    return torch.where(pos < lengths[:, None], total, -math.inf)


def _plain_attention(state, case):
    k, lengths = state["k"], state["lengths"].long()
    if state["indices"] is not None:
        pos = state["indices"].long()
    else:
        pos = torch.arange(state["longest"], device="cuda").expand(lengths.numel(), -1)
    seen = (pos >= 0) & (pos < lengths[:, None])
    slot = _slots(state["table"], _request(state, case["next_n"]), pos.clamp(min=0), k.shape[1])
    rows, heads, dk = state["q"].shape
    kv, dv = case["kv_heads"], case["dv"]
    kk = k.flatten(0, 1)[slot].to(torch.float32)  # rows, tokens, kv heads, dk
    vv = kk[..., :dv] if state["v"] is None else state["v"].flatten(0, 1)[slot].to(torch.float32)
    q = state["q"].to(torch.float32).view(rows, kv, heads // kv, dk)
    s = torch.matmul(q, kk.permute(0, 2, 3, 1)) * state["scale"]
    s = s.masked_fill(~seen[:, None, None, :], -math.inf)
    m = s.amax(-1, keepdim=True).clamp(min=-3.0e38)  # a row that sees nothing stays finite
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, vv.transpose(1, 2)) / total.clamp(min=1e-38)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)[..., 0]
    return {"out": out.reshape(rows, heads, dv).to(state["q"].dtype), "lse": lse.reshape(rows, heads)}


def exact(case, seed):
    """The operators' definitions in 64 bits, a row at a time."""
    if case["op"] == "map":
        return None
    state = prepare(case, seed)
    table, lengths, block = state["table"].long(), state["lengths"].tolist(), case["block"]
    rows = len(lengths)
    logits = torch.full((rows, state["longest"]), -math.inf, dtype=torch.float64, device="cuda") if case["op"] == "logits" else None
    outs, lses = [], []
    for r in range(rows):
        pages = table[0 if case["prefill"] else r // case["next_n"]]
        pos = torch.arange(lengths[r], device="cuda")
        if case["op"] == "attention" and case["topk"]:
            pos = state["indices"][r].long()
            pos = pos[(pos >= 0) & (pos < lengths[r])]
        page, off = pages[pos // block], pos % block
        q = state["q"][r].double()
        if case["op"] == "logits":
            dots = q @ state["keys"][page, off].double().T
            value = (state["weights"][r].double()[:, None] * dots.clamp(min=0)).sum(0)
            logits[r, :lengths[r]] = value if state["scales"] is None else value * state["scales"][page, off].double()
            continue
        group = case["heads"] // case["kv_heads"]
        kk = state["k"][page, off].double().repeat_interleave(group, 1) if group > 1 and case["kv_heads"] > 1 else state["k"][page, off].double()
        if case["kv_heads"] == 1:
            s = (q @ kk[:, 0].T) * state["scale"]
            v = kk[:, 0, :case["dv"]] if state["v"] is None else state["v"][page, off][:, 0].double()
            lse = torch.logsumexp(s, -1)
            o = torch.exp(s - lse[:, None]) @ v
        else:
            s = torch.einsum("hd,thd->ht", q, kk) * state["scale"]
            v = state["v"][page, off].double().repeat_interleave(group, 1)
            lse = torch.logsumexp(s, -1)
            o = torch.einsum("ht,thd->hd", torch.exp(s - lse[:, None]), v)
        outs.append(o)
        lses.append(lse)
    return logits if logits is not None else {"out": torch.stack(outs), "lse": torch.stack(lses)}
