"""Cases and plain forms of further operators over a paged cache: blocks chosen by a cheap score, a prefix that requests
share, and the pages themselves.

A block is a page of the cache. ``means`` keeps the mean key of the pages that a step wrote to, ``scores`` ranks a row's
blocks by it for each key-value head (the selection from the scores is ``topk_ragged``), and ``blocks`` attends to the
tokens of the chosen ones. ``shared`` is attention over everything cached where requests begin with the same pages. ``fork``
frees the pages of some requests, gives them those of others and copies what is not full; ``compact`` moves pages to the
lowest numbers. Every case is one of these steps.
"""
import math

import torch

own = False

F16, BF16 = "float16", "bfloat16"


def listed():
    return [
        # mean keys after a decode step: one page of each request has got a token
        dict(name="means_decode", op="means", requests=64, ctx_lo=8192, ctx_hi=32768, new_lo=1, new_hi=1, kv_heads=8, dk=128, dtype=BF16, block=64),
        # mean keys after pieces of prompts of any length
        dict(name="means_prompt", op="means", requests=16, ctx_lo=0, ctx_hi=8192, new_lo=1, new_hi=8192, kv_heads=8, dk=128, dtype=F16, block=64),
        # scores of a decode batch of long requests
        dict(name="scores_decode", op="scores", requests=64, next_n=1, prefill=False, len_lo=32768, len_hi=131072, heads=64, kv_heads=8, dk=128, dtype=BF16, block=64, sinks=1, recent=2),
        # scores of a prompt's piece: 1024 rows of one request
        dict(name="scores_prompt", op="scores", requests=1, next_n=1024, prefill=True, len_lo=32768, len_hi=32768, heads=32, kv_heads=4, dk=128, dtype=F16, block=64, sinks=1, recent=2),
        # attention of a few short requests over some small blocks: latency
        dict(name="blocks_small", op="blocks", requests=4, next_n=1, prefill=False, len_lo=1, len_hi=4096, heads=16, kv_heads=2, dk=128, dv=128, latent=False, chosen=8, dtype=BF16, block=32),
        # a decode batch of long requests over 32 blocks of 64 tokens for each key-value head
        dict(name="blocks_batch", op="blocks", requests=64, next_n=1, prefill=False, len_lo=16384, len_hi=65536, heads=64, kv_heads=8, dk=128, dv=128, latent=False, chosen=32, dtype=BF16, block=64),
        # a prompt's piece: 1024 rows of one request, each over its own 16 blocks
        dict(name="blocks_prompt", op="blocks", requests=1, next_n=1024, prefill=True, len_lo=15360, len_hi=15360, heads=32, kv_heads=4, dk=128, dv=128, latent=False, chosen=16, dtype=F16, block=64),
        # a few samples of one short prompt: latency
        dict(name="shared_small", op="shared", prefixes=1, each=8, next_n=1, pre_lo=1000, pre_hi=4000, tail_lo=1, tail_hi=256, heads=32, kv_heads=8, dk=128, dv=128, latent=False, dtype=BF16, block=16),
        # a batch that shares a long document, grouped heads
        dict(name="shared_batch", op="shared", prefixes=1, each=256, next_n=1, pre_lo=32768, pre_hi=32768, tail_lo=1, tail_hi=2048, heads=32, kv_heads=8, dk=128, dv=128, latent=False, dtype=BF16, block=64),
        # two documents, latent attention with the 16 heads of one GPU out of eight, a drafted token each
        dict(name="shared_latent", op="shared", prefixes=2, each=32, next_n=2, pre_lo=12000, pre_hi=20000, tail_lo=1, tail_hi=2048, heads=16, kv_heads=1, dk=576, dv=512, latent=True, dtype=F16, block=64),
        # samples dropped and drawn anew: 32 requests with 8 children each, keys and values of two layers
        dict(name="pages_fork", op="fork", parents=32, each=8, ctx_lo=1, ctx_hi=8192, caches=4, kv_heads=4, dk=128, dtype=BF16, block=64),
        # a pool of pages with holes, of which the highest are moved down
        dict(name="pages_compact", op="compact", requests=256, ctx_lo=1, ctx_hi=1024, spare=2048, copies=1024, caches=2, kv_heads=4, dk=128, dtype=BF16, block=16),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["means", "scores", "blocks", "blocks", "shared", "shared", "fork", "compact"])
    block, dtype = rng.choice([16, 32, 64, 128]), rng.choice([F16, BF16])
    kv, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
    if op == "means":
        lo = rng.choice([0, 1, 100])
        case = dict(op=op, requests=_log(rng, 1, 64), ctx_lo=lo, ctx_hi=lo + _log(rng, 1, 32768), new_lo=rng.choice([0, 1]), new_hi=_log(rng, 1, 8192), kv_heads=kv, dk=dim, dtype=dtype, block=block)
        while work(case)["bytes"] > 1.5e8:
            case["new_hi"] = max(1, case["new_hi"] // 2)
            case["requests"] = max(1, case["requests"] * 7 // 8)
        return case
    if op == "fork":
        case = dict(op=op, parents=_log(rng, 1, 64), each=rng.choice([1, 2, 4, 7, 8]), ctx_lo=1, ctx_hi=_log(rng, 32, 8192), caches=rng.choice([1, 2, 4]), kv_heads=kv, dk=dim, dtype=dtype, block=block)
        while work(case)["bytes"] > 1.4e8 or case["parents"] * case["ctx_hi"] * kv * dim * case["caches"] > 6e8:
            case["parents"] = max(1, case["parents"] * 3 // 4)
            case["ctx_hi"] = max(32, case["ctx_hi"] * 3 // 4)
        return case
    if op == "compact":
        case = dict(op=op, requests=_log(rng, 1, 512), ctx_lo=1, ctx_hi=_log(rng, 32, 4096), spare=_log(rng, 16, 16384), copies=_log(rng, 1, 2048), caches=rng.choice([1, 2]), kv_heads=kv, dk=dim, dtype=dtype, block=block)
        while _pool(case) * block * kv * dim * case["caches"] > 4e8 or work(case)["bytes"] > 1.4e8:
            case["requests"] = max(1, case["requests"] * 3 // 4)
            case["spare"] = max(16, case["spare"] * 3 // 4)
            case["copies"] = max(1, case["copies"] * 3 // 4)
        return case
    if op == "shared":
        latent = rng.random() < 0.4
        lo, tail = _log(rng, 64, 32768), _log(rng, 1, 2048)
        case = dict(op=op, prefixes=rng.choice([1, 1, 2, 3, 8]), each=_log(rng, 1, 256), next_n=rng.choice([1, 1, 2, 3]), pre_lo=lo, pre_hi=lo + rng.choice([0, lo // 2]), tail_lo=rng.choice([0, 1]), tail_hi=tail)
        case.update(dict(heads=rng.choice([16, 32, 64, 128]), kv_heads=1, dk=576, dv=512) if latent else dict(heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, dk=dim, dv=dim))
        case.update(latent=latent, dtype=dtype, block=block)
        while (lambda w: w["bytes"] > 1.2e9 or w["flops"] > 1.4e11)(work(case)) or _padded(case) > 4e9:
            if case["each"] > 4 and rng.random() < 0.5:
                case["each"] = case["each"] * 7 // 8
            else:
                case["pre_lo"], case["pre_hi"], case["tail_hi"] = (max(1, case[x] * 7 // 8) for x in ("pre_lo", "pre_hi", "tail_hi"))
                case["tail_lo"] = min(case["tail_lo"], case["tail_hi"])
        return case
    prefill = rng.random() < 0.3
    hi = _log(rng, 64, 32768 if prefill else 131072)
    case = dict(op=op, requests=1 if prefill else _log(rng, 1, 64), next_n=_log(rng, 16, 1024) if prefill else rng.choice([1, 1, 2, 3]), prefill=prefill,
                len_lo=hi if prefill else rng.choice([1, max(1, hi // 4), max(1, hi // 2)]), len_hi=hi)
    if op == "blocks" and rng.random() < 0.2:
        case.update(heads=rng.choice([16, 64, 128]), kv_heads=1, dk=576, dv=512, latent=True)
    else:
        case.update(heads=kv * rng.choice([1, 3, 4, 8]), kv_heads=kv, dk=dim)
        if op == "blocks":
            case.update(dv=dim, latent=False)
    if op == "scores":
        case.update(sinks=rng.choice([0, 1]), recent=rng.choice([0, 1, 2]))
    else:
        case.update(chosen=_log(rng, 1, max(1, 2048 // block)))
    case.update(dtype=dtype, block=block)
    while (lambda w: w["bytes"] > 5.5e8 or w["flops"] > 2e10)(work(case)) or _padded(case) > 3e9:
        case["len_hi"] = max(64, case["len_hi"] * 7 // 8)
        case["len_lo"] = case["len_hi"] if prefill else min(case["len_lo"], case["len_hi"])
        if op == "blocks":
            case["chosen"] = max(1, case["chosen"] * 7 // 8)
        if prefill:
            case["next_n"] = max(16, case["next_n"] * 7 // 8)
        else:
            case["requests"] = max(1, case["requests"] * 7 // 8)
    return case


def _pool(case):
    """Pages of a pool that is to be compacted."""
    return case["requests"] * ((case["ctx_hi"] + case["block"] - 1) // case["block"]) + case["spare"]


def _padded(case):
    """About the largest number of bytes that the plain form holds in one tensor."""
    if case["op"] == "shared":
        rows = case["prefixes"] * case["each"] * case["next_n"]
        return 4 * max(rows * case["heads"] * case["pre_hi"], rows * (case["tail_hi"] + case["block"] + 2) * max(case["heads"], case["kv_heads"] * case["dk"]))
    rows, length = case["requests"] * case["next_n"], case["len_hi"] + case["next_n"]
    if case["op"] == "scores":
        return 4 * rows * (length // case["block"] + 1) * case["kv_heads"] * (1 if case["prefill"] else case["dk"])
    return 4 * rows * case["kv_heads"] * case["chosen"] * case["block"] * max(case["heads"] // case["kv_heads"], case["dk"])


def work(case):
    op = case["op"]
    if op == "fork":
        n = case["parents"] * case["each"]
        pages = n * (case["ctx_lo"] + case["ctx_hi"]) / 2 / case["block"]  # shared ones: freed, and given again
        page = case["block"] * case["kv_heads"] * case["dk"] * 2 * case["caches"]
        return {"bytes": 2 * n * page * (1 - 1 / case["block"]) + 24 * pages + 40 * n, "flops": 0}
    if op == "compact":
        page = case["block"] * case["kv_heads"] * case["dk"] * 2 * case["caches"]
        columns = (case["ctx_hi"] + case["block"] - 1) // case["block"]
        return {"bytes": 2 * min(case["copies"], _pool(case) // 4) * page + 8 * case["requests"] * columns + 12 * _pool(case), "flops": 0}
    each = 2 * case["kv_heads"] * case["dk"]
    if op == "means":
        new = (case["new_lo"] + case["new_hi"]) / 2
        tokens = case["requests"] * (new + min(case["block"], (case["ctx_lo"] + case["ctx_hi"]) / 2) / 2)
        pages = case["requests"] * (new / case["block"] + 0.5)
        return {"bytes": each * (tokens + pages) + 4 * pages + 8 * case["requests"], "flops": tokens * each / 2}
    rows = case["next_n"] * (case["prefixes"] * case["each"] if op == "shared" else case["requests"])
    if op == "scores":
        columns = ((case["len_lo"] + case["len_hi"]) / 2 + case["next_n"] / 2) / case["block"] + 1
        return {"bytes": case["requests"] * columns * (each + 4) + rows * (case["heads"] * case["dk"] * 2 + case["kv_heads"] * (4 * columns + 4)),
                "flops": rows * (case["heads"] * case["dk"] + 2 * case["kv_heads"] * columns * case["dk"])}
    each += 0 if case["latent"] else 2 * case["kv_heads"] * case["dv"]
    out = rows * case["heads"] * (2 * (case["dk"] + case["dv"]) + 4)
    if op == "blocks":
        mean = (case["len_lo"] + case["len_hi"]) / 2 + (case["next_n"] - 1) / 2
        read = min(case["chosen"] * case["block"], mean)
        return {"bytes": min(rows * read, case["requests"] * mean) * each + out + 4 * rows * case["kv_heads"] * case["chosen"], "flops": 2 * rows * read * case["heads"] * (case["dk"] + case["dv"])}
    prefix, tail = (case["pre_lo"] + case["pre_hi"]) / 2, (case["tail_lo"] + case["tail_hi"]) / 2
    return {"bytes": case["prefixes"] * (prefix + case["each"] * tail) * each + out, "flops": 2 * rows * (prefix + tail) * case["heads"] * (case["dk"] + case["dv"])}


def _table(g, lengths, block, columns, pool):
    """A block table for these lengths, the pool's pages in the random order in which they are handed out, and how many are."""
    used = (lengths + block - 1) // block
    order = torch.randperm(pool, generator=g, device="cuda", dtype=torch.int32)
    col = torch.arange(columns, device="cuda")
    at = (torch.cumsum(used, 0) - used)[:, None] + col
    return torch.where(col < used[:, None], order[at.clamp(max=pool - 1)], -1).to(torch.int32).contiguous(), order, used.sum()[None].int()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = getattr(torch, case["dtype"])

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g, device="cuda", dtype=torch.int64)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype)

    state, op, block, kv, dk = {"case": case}, case["op"], case["block"], case["kv_heads"], case["dk"]
    if own:
        import sparse_attention_row_gb300 as sar
        state["decoder"] = sar.PagedDecoder(torch.cuda.current_device())
    if op == "means":
        context, new = whole(case["ctx_lo"], case["ctx_hi"], case["requests"]), whole(case["new_lo"], case["new_hi"], case["requests"])
        columns = (case["ctx_hi"] + case["new_hi"] + block - 1) // block
        blocks = case["requests"] * columns
        table, _, _ = _table(g, context + new, block, columns, blocks)
        state.update(context=context.int(), new=new.int(), table=table, k=normal(blocks, block, kv, dk), means=normal(blocks, kv, dk), most=(case["new_hi"] + 2 * block - 2) // block)
        return state
    if op == "fork":
        # the last requests are children that are to be drawn anew: they hold pages of their own
        parents, n = case["parents"], case["parents"] * case["each"]
        columns = (case["ctx_hi"] + block - 1) // block
        lengths = whole(case["ctx_lo"], case["ctx_hi"], parents)
        blocks = parents * columns + 3 * n + 5
        table, free, taken = _table(g, torch.cat([lengths, whole(1, 2 * block, n).clamp(max=case["ctx_hi"])]), block, columns, blocks)
        parent = torch.randint(0, parents, (n,), generator=g, device="cuda", dtype=torch.int64)
        state.update(table=table, free=free, taken=taken, shares=torch.zeros(blocks, dtype=torch.int32, device="cuda"),
                     parent=parent.int(), child=torch.arange(parents, parents + n, device="cuda", dtype=torch.int32), kept=lengths[parent].int(), caches=normal(case["caches"], blocks, block, kv, dk))
        return state
    if op == "compact":
        blocks, columns = _pool(case), (case["ctx_hi"] + block - 1) // block
        table, free, taken = _table(g, whole(case["ctx_lo"], case["ctx_hi"], case["requests"]), block, columns, blocks)
        shares = torch.zeros(blocks, dtype=torch.int32, device="cuda").index_put((free.long(),), torch.where(torch.arange(blocks, device="cuda") < taken, whole(0, 2, blocks), 0).int())
        state.update(table=table, free=free, taken=taken, shares=shares, caches=normal(case["caches"], blocks, block, kv, dk),
                     table_out=torch.empty_like(table), free_out=torch.empty_like(free), taken_out=torch.empty(1, dtype=torch.int32, device="cuda"), shares_out=torch.empty(blocks, dtype=torch.int32, device="cuda"))
        return state
    next_n = case["next_n"]
    if op == "shared":
        prefixes, each = case["prefixes"], case["each"]
        before, tail = whole(case["pre_lo"], case["pre_hi"], prefixes), whole(case["tail_lo"], case["tail_hi"], prefixes * each)
        full = before // block  # whole pages, which are shared
        of = torch.arange(prefixes, device="cuda").repeat_interleave(each)
        base = before[of] + tail
        width = case["pre_hi"] // block
        columns = (case["pre_hi"] + case["tail_hi"] + next_n - 1) // block + 1
        # one table of the prefixes' pages and of what each request has behind them
        behind = base + next_n - 1 - (full * block)[of]
        blocks = prefixes * width + prefixes * each * ((case["tail_hi"] + next_n - 1) // block + 2)
        both, _, _ = _table(g, torch.cat([full * block, behind]), block, columns, blocks)
        col = torch.arange(columns, device="cuda")
        table = torch.where(col < full[of][:, None], both[:prefixes][of], both[prefixes:].gather(1, (col - full[of][:, None]).clamp(min=0)))
        state.update(table=table.contiguous(), prefix_table=both[:prefixes, :max(width, 1)].contiguous(), prefix_lens=before.int(), prefix_of=of.int(),
                     lengths=(base[:, None] + torch.arange(next_n, device="cuda")).reshape(-1).int(), most=case["pre_hi"] // block * block, most_tail=case["tail_hi"] + block + next_n - 1)
    else:
        base = whole(case["len_lo"], case["len_hi"], case["requests"])
        lengths = (base[:, None] + torch.arange(next_n, device="cuda")).reshape(-1)
        columns = (case["len_hi"] + next_n - 1 + block - 1) // block
        blocks = case["requests"] * columns
        table, _, _ = _table(g, base + next_n - 1, block, columns, blocks)
        state.update(table=table, lengths=lengths.int())
    rows = state["lengths"].numel()
    state["q"] = normal(rows, case["heads"], dk)
    if op == "scores":
        state.update(means=normal(blocks, kv, dk) * block ** -0.5, out=torch.full((rows, kv, columns), -math.inf, device="cuda"))
        return state
    state.update(k=normal(blocks, block, kv, dk), v=None if case["latent"] else normal(blocks, block, kv, case["dv"]), scale=dk ** -0.5)
    if op == "blocks":
        # distinct blocks of each row and head in no order, -1 behind them: what the selection leaves
        used = ((lengths + block - 1) // block)[:, None, None]
        chance = torch.rand((rows, kv, max(columns, case["chosen"])), generator=g, device="cuda")
        chance.masked_fill_(torch.arange(chance.shape[2], device="cuda") >= used, -1.0)
        value, index = torch.topk(chance, case["chosen"], dim=2)
        state["blocks"] = torch.where(value < 0, -1, index).int().contiguous()
    return state


def run(state):
    case = state["case"]
    op, block = case["op"], case["block"]
    if own:
        d = state["decoder"]
        if op == "means":
            return d.block_means(state["k"], state["table"], state["context"], state["new"], state["means"])
        if op == "scores":
            scores, lens = d.block_scores(state["q"], state["means"], state["table"], state["lengths"], block, sink_blocks=case["sinks"], recent_blocks=case["recent"], next_n=case["next_n"], out=state["out"])
            return {"scores": scores, "lens": lens}
        if op == "blocks":
            out, lse = d.block_attention(state["q"], state["k"], state["table"], state["lengths"], state["blocks"], v_cache=state["v"], v_dim=case["dv"], scale=state["scale"], next_n=case["next_n"], return_lse=True)
            return {"out": out, "lse": lse}
        if op == "shared":
            out, lse = d.shared_attention(state["q"], state["k"], state["table"], state["lengths"], state["prefix_of"], state["prefix_lens"], state["prefix_table"], v_cache=state["v"], v_dim=case["dv"],
                                          scale=state["scale"], next_n=case["next_n"], return_lse=True)
            return {"out": out, "lse": lse}
        if op == "fork":
            d.free_pages(state["child"], state["table"], state["shares"], state["free"], state["taken"])
            copies = d.fork_pages(state["parent"], state["child"], state["kept"], state["table"], state["shares"], state["free"], state["taken"], block)
            d.copy_pages(state["caches"].unbind(0), copies)
            return {"table": state["table"], "shares": state["shares"], "free": state["free"], "taken": state["taken"], "source": copies.source, "target": copies.target, "caches": state["caches"]}
        copies = d.compact_pages(state["table"], state["shares"], state["free"], state["taken"], case["copies"], table_out=state["table_out"], shares_out=state["shares_out"], free_out=state["free_out"], taken_out=state["taken_out"])
        d.copy_pages(state["caches"].unbind(0), copies)
        return {"table": state["table_out"], "shares": state["shares_out"], "free": state["free_out"], "taken": state["taken_out"], "source": copies.source, "target": copies.target, "caches": state["caches"]}
    return {"means": _plain_means, "scores": _plain_scores, "blocks": _plain_blocks, "shared": _plain_shared, "fork": _plain_fork, "compact": _plain_compact}[op](state, case)


def _plain_means(state, case):
    context, new, table, k, block = state["context"].long(), state["new"].long(), state["table"], state["k"], case["block"]
    total = context + new
    col = context[:, None] // block + torch.arange(state["most"], device="cuda")
    touched = (col * block < total[:, None]) & (new[:, None] > 0)
    page = torch.where(touched, table.gather(1, col.clamp(max=table.shape[1] - 1)).long(), 0)
    held = (total[:, None] - col * block).clamp(1, block)
    seen = torch.arange(block, device="cuda") < held[..., None]
    x = torch.where(seen[..., None, None], k[page].to(torch.float32), 0.0).sum(2) / held[..., None, None]
    wide = torch.cat([state["means"], state["means"][:1]])  # a place for what is no page
    return wide.index_put((torch.where(touched, page, k.shape[0]),), x.to(k.dtype))[:-1].contiguous()


def _request(rows, next_n):
    return torch.arange(rows, device="cuda") // next_n


def _plain_scores(state, case):
    q, means, lengths, block, kv = state["q"], state["means"], state["lengths"].long(), case["block"], case["kv_heads"]
    rows, columns = lengths.numel(), state["table"].shape[1]
    q = q.to(torch.float32).view(rows, kv, case["heads"] // kv, -1).sum(2)
    keys = means.to(torch.float32)[state["table"].long().clamp(min=0)]  # requests, columns, heads, dk
    s = torch.matmul(q.view(case["requests"], case["next_n"], kv, -1).transpose(1, 2), keys.permute(0, 2, 3, 1)).transpose(1, 2).reshape(rows, kv, columns)
    used = ((lengths + block - 1) // block)[:, None, None]
    col = torch.arange(columns, device="cuda")
    s = torch.where((col < case["sinks"]) | (col >= used - case["recent"]), math.inf, s)
    return {"scores": torch.where(col < used, s, -math.inf), "lens": used[:, 0].expand(rows, kv).int().contiguous()}


def _joined(s, v, total_dtype):
    """Softmax over the scores' last dimension and its product with the values."""
    m = s.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(s - m)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total.clamp(min=1e-38)
    return out.to(total_dtype), torch.where(total > 0, m + torch.log(total), -math.inf)[..., 0]


def _plain_blocks(state, case):
    k, lengths, block, kv, dv = state["k"], state["lengths"].long(), case["block"], case["kv_heads"], case["dv"]
    rows, heads, dk = state["q"].shape
    chosen = state["blocks"].long()
    pos = (chosen[..., None] * block + torch.arange(block, device="cuda")).flatten(2)  # rows, heads, tokens
    seen = (chosen[..., None] >= 0).expand(-1, -1, -1, block).flatten(2) & (pos < lengths[:, None, None])
    page = state["table"][_request(rows, case["next_n"])[:, None, None], chosen.clamp(min=0)].long().clamp(min=0)
    slot = (page[..., None] * block + torch.arange(block, device="cuda")).flatten(2)
    head = torch.arange(kv, device="cuda")[:, None]
    kk = k.flatten(0, 1)[slot, head].to(torch.float32)
    vv = kk[..., :dv] if state["v"] is None else state["v"].flatten(0, 1)[slot, head].to(torch.float32)
    s = torch.matmul(state["q"].to(torch.float32).view(rows, kv, heads // kv, dk), kk.transpose(2, 3)) * state["scale"]
    out, lse = _joined(s.masked_fill(~seen[:, :, None], -math.inf), vv, k.dtype)
    return {"out": out.reshape(rows, heads, dv), "lse": lse.reshape(rows, heads)}


def _plain_shared(state, case):
    k, v, table, block, kv, dv, n = state["k"], state["v"], state["table"].long(), case["block"], case["kv_heads"], case["dv"], case["prefixes"]
    q, lengths = state["q"].to(torch.float32), state["lengths"].long()
    rows, heads, dk = q.shape
    group = heads // kv
    flat_k, flat_v = k.flatten(0, 1), None if v is None else v.flatten(0, 1)
    shared = state["prefix_lens"].long() // block * block

    def scores_and_values(slot, queries):  # [..., tokens] and [..., kv, columns, dk]
        kk = flat_k[slot].to(torch.float32).transpose(-3, -2)
        vv = kk[..., :dv] if flat_v is None else flat_v[slot].to(torch.float32).transpose(-3, -2)
        return torch.matmul(queries, kk.transpose(-2, -1)) * state["scale"], vv

    # the prefixes, once for all of their rows
    pos = torch.arange(max(state["most"], 1), device="cuda")
    page = state["prefix_table"].long().clamp(min=0)[:, (pos // block).clamp(max=state["prefix_table"].shape[1] - 1)]
    first, vp = scores_and_values(page * block + pos % block, q.view(n, rows // n, kv, group, dk).transpose(1, 2).reshape(n, kv, -1, dk))
    first = first.masked_fill(pos >= shared[:, None, None, None], -math.inf)
    # what each row has behind its prefix
    request = _request(rows, case["next_n"])
    start = shared[state["prefix_of"].long()[request]]
    pos = start[:, None] + torch.arange(state["most_tail"], device="cuda")
    slot = table[request[:, None], (pos // block).clamp(max=table.shape[1] - 1)].clamp(min=0) * block + pos % block
    last, vt = scores_and_values(slot, q.view(rows, kv, group, dk))
    last = last.masked_fill((pos >= lengths[:, None])[:, None, None], -math.inf)
    m = torch.maximum(first.amax(-1).view(n, kv, rows // n, group).transpose(1, 2).reshape(rows, kv, group), last.amax(-1)).clamp(min=-3.0e38)
    p = torch.exp(first - m.view(n, rows // n, kv, group).transpose(1, 2).reshape(n, kv, -1, 1))
    out, total = torch.matmul(p, vp).view(n, kv, rows // n, group, dv).transpose(1, 2).reshape(rows, kv, group, dv), p.sum(-1).view(n, kv, rows // n, group).transpose(1, 2).reshape(rows, kv, group)
    p = torch.exp(last - m[..., None])
    out, total = out + torch.matmul(p, vt), total + p.sum(-1)
    lse = torch.where(total > 0, m + torch.log(total), -math.inf)
    return {"out": (out / total.clamp(min=1e-38)[..., None]).reshape(rows, heads, dv).to(k.dtype), "lse": lse.reshape(rows, heads)}


def _plain_fork(state, case):
    block, table, shares, free = case["block"], state["table"].long(), state["shares"].long(), state["free"].long()
    child, parent, kept, taken = state["child"].long(), state["parent"].long(), state["kept"].long(), state["taken"].long()
    blocks, n, columns = shares.numel(), child.numel(), table.shape[1]
    # the children's pages: one holder fewer each; those without any go back on the list, in the order of their first places
    page = table[child].flatten()
    at = torch.where(page >= 0, page, blocks)
    left = torch.cat([shares, shares[:1]]).index_add(0, at, torch.full_like(at, -1))
    first = torch.full((blocks + 1,), page.numel(), device="cuda").scatter_reduce(0, at, torch.arange(page.numel(), device="cuda"), "amin")
    back = (left[at] < 0) & (page >= 0) & (first[at] == torch.arange(page.numel(), device="cuda"))
    rank = torch.cumsum(back, 0) - 1
    taken = taken - back.sum()
    free = torch.cat([free, free[:1]]).index_put((torch.where(back, taken + rank, free.numel()),), page)[:-1]
    shares = left[:-1].clamp(min=0)
    # the parents' full pages, and a new page for what is left
    col = torch.arange(columns, device="cuda")
    full, rest = kept // block, kept % block > 0
    source = torch.where(rest, table[parent, (kept // block).clamp(max=columns - 1)], -1)
    rank = torch.cumsum(rest, 0) - 1
    target = torch.where(rest, free[(taken + rank).clamp(0, free.numel() - 1)], -1)
    row = torch.where(col < full[:, None], table[parent], torch.where((col == full[:, None]) & rest[:, None], target[:, None], -1))
    given = torch.where(col < full[:, None], table[parent], blocks).flatten()
    shares = torch.cat([shares, shares[:1]]).index_add(0, given, torch.ones_like(given))[:-1]
    table = table.index_put((child,), row)
    caches = state["caches"]
    # where there is nothing to copy, the list's last page, which no child gets, is copied onto itself
    caches[:, torch.where(rest, target, free[-1])] = caches[:, torch.where(rest, source, free[-1])]
    return {"table": table.int(), "shares": shares.int(), "free": free.int(), "taken": (taken + rest.sum()).int(), "source": source.int(), "target": target.int(), "caches": caches}


def _plain_compact(state, case):
    table, shares, free, copies = state["table"].long(), state["shares"], state["free"].long(), case["copies"]
    blocks = shares.numel()
    ids, taken = torch.arange(blocks, device="cuda"), state["taken"]
    live = torch.zeros(blocks + 1, dtype=torch.bool, device="cuda").index_fill(0, torch.where(table >= 0, table, blocks).flatten(), True)[:-1]
    listed = torch.arange(free.numel(), device="cuda") >= taken
    hole = torch.zeros(blocks + 1, dtype=torch.bool, device="cuda").index_fill(0, torch.where(listed, free, blocks), True)[:-1]
    low, high = torch.sort(torch.where(hole, ids, blocks)).values[:copies], torch.sort(torch.where(live, ids, -1), descending=True).values[:copies]
    moves = (low < high) & (low < blocks)
    pad = torch.full((copies - low.numel(),), -1, device="cuda")
    source, target = torch.cat([torch.where(moves, high, -1), pad]), torch.cat([torch.where(moves, low, -1), pad])
    to = torch.cat([ids, ids[:1]]).index_put((torch.where(source >= 0, source, blocks),), target)[:-1]
    table = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    new_shares = torch.zeros_like(shares).index_add(0, to, shares)
    wide = torch.cat([hole, hole[:1]])
    wide = wide.index_fill(0, torch.where(target >= 0, target, blocks), False)
    hole = wide.index_fill(0, torch.where(source >= 0, source, blocks), True)[:-1]
    holes = torch.sort(torch.where(hole, ids, blocks)).values
    free = torch.where(listed, holes[(torch.arange(free.numel(), device="cuda") - taken).clamp(0, blocks - 1)], free)
    caches = state["caches"]
    # what is no move copies a page onto itself, one that no move writes
    still = torch.where(moves[0], high[0], ids[0])
    caches[:, torch.where(target >= 0, target, still)] = caches[:, torch.where(source >= 0, source, still)]
    return {"table": table.int(), "shares": new_shares, "free": free.int(), "taken": taken, "source": source.int(), "target": target.int(), "caches": caches}


def exact(case, seed):
    """The operators' definitions in 64 bits, a request or a row at a time."""
    op, block = case["op"], case["block"]
    if op in ("fork", "compact"):
        return None
    state = prepare(case, seed)
    table = state["table"].long()
    if op == "means":
        means = state["means"].double()
        for r, (c, n) in enumerate(zip(state["context"].tolist(), state["new"].tolist())):
            if n == 0:
                continue
            lo, hi = c // block, (c + n - 1) // block
            pages = state["k"][table[r, lo:hi + 1]].double()
            means[table[r, lo:hi]] = pages[:-1].mean(1)
            means[table[r, hi]] = pages[-1, :c + n - hi * block].mean(0)
        return means
    lengths, kv = state["lengths"].tolist(), case["kv_heads"]
    rows, group = len(lengths), case["heads"] // kv
    if op == "scores":
        scores = torch.full(state["out"].shape, -math.inf, dtype=torch.float64, device="cuda")
        for r in range(rows):
            used = -(-lengths[r] // block)
            keys = state["means"][table[r // case["next_n"], :used]].double()
            scores[r, :, :used] = torch.einsum("khd,ckd->kc", state["q"][r].double().view(kv, group, -1), keys)
            scores[r, :, :min(case["sinks"], used)] = math.inf
            scores[r, :, max(0, used - case["recent"]):used] = math.inf
        return {"scores": scores, "lens": None}
    outs, lses = [], []
    every = torch.arange(max(lengths + [1]), device="cuda")
    head = torch.arange(kv, device="cuda")[:, None]
    for r in range(rows):
        pages = table[r // case["next_n"]]
        if op == "blocks":
            pos = (state["blocks"][r].long()[..., None] * block + every[:block]).flatten(1)
            seen = (pos >= 0) & (pos < lengths[r])
            pos = pos.clamp(min=0)
            at = pages[(pos // block).clamp(max=table.shape[1] - 1)].clamp(min=0), pos % block, head
        else:
            pos = every[:lengths[r]]
            seen = torch.ones((kv, lengths[r]), dtype=torch.bool, device="cuda")
            at = pages[pos // block][None], (pos % block)[None], head
        kk = state["k"][at].double()
        s = (state["q"][r].double().view(kv, group, -1) @ kk.transpose(1, 2) * state["scale"]).masked_fill(~seen[:, None], -math.inf)
        vv = kk[..., :case["dv"]] if state["v"] is None else state["v"][at].double()
        lse = torch.logsumexp(s, -1)
        p = torch.where(lse[..., None] > -math.inf, torch.exp(s - lse.clamp(min=-1e300)[..., None]), 0.0)
        outs.append((p @ vv).flatten(0, 1))
        lses.append(lse.flatten())
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}
