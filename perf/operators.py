"""Work of the paged key/value cache, as it is measured: appending new tokens
(per-head norm, rotation and scatter in one pass), attention of the new tokens
over the pages, the attention weight every cached key receives, and eviction
by that weight.

``run`` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end) or, with ``own`` set, through the framework's
entry points.  ``exact`` gives the same outputs in 64 bits, written apart.

A case holds plain values only.  Lengths are drawn from the case's own
``lens`` number, so that the work of a case is known without its inputs:
sequence b has ``past`` tokens in the cache and ``new`` ones that arrive with
the call, each uniform in its [lo, hi] range."""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def _case(name, op, dtype, batch, heads, kv_heads, head_size, page, past, new=(0, 0), lens=1, window=0, budget=0,
          recent=0, interleaved=False):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "heads": heads, "kv_heads": kv_heads,
            "head_size": head_size, "page": page, "past_lo": past[0], "past_hi": past[1], "new_lo": new[0],
            "new_hi": new[1], "lens": lens, "window": window, "budget": budget, "recent": recent,
            "interleaved": interleaved}


def listed():
    return [
        # the new rows of one decode step of a batch of 16: latency counts
        _case("append_decode_b16", "append", "bf16", 16, 32, 8, 128, 16, (1, 4095), (1, 1), lens=1),
        # four prompts of 2048 tokens entering an empty cache
        _case("append_prompt_4x2048", "append", "fp16", 4, 32, 8, 128, 64, (0, 0), (2048, 2048), lens=2),
        # one token of one short sequence: the smallest call of a chat
        _case("attend_one", "attend", "bf16", 1, 32, 8, 128, 16, (300, 300), (1, 1), lens=3),
        # one decode step of a batch of 16 of ragged lengths
        _case("attend_decode_b16", "attend", "bf16", 16, 32, 8, 128, 16, (1, 4095), (1, 1), lens=1),
        # one decode step over long contexts, eight query heads a KV head
        _case("attend_long_decode_b8", "attend", "bf16", 8, 64, 8, 128, 64, (16384, 32767), (1, 1), lens=4),
        # a few drafted tokens a sequence to be verified, head size 64
        _case("attend_verify_b32", "attend", "fp16", 32, 32, 8, 64, 32, (100, 6000), (2, 6), lens=5),
        # a chunk of 128 prompt tokens on top of ragged pasts
        _case("attend_chunk_b8", "attend", "fp16", 8, 32, 8, 128, 16, (0, 3968), (128, 128), lens=6),
        # whole prompts: the matrix products count
        _case("attend_prompt_4x2048", "attend", "fp16", 4, 32, 8, 128, 128, (0, 0), (2048, 2048), lens=2),
        # the weight of every key after a decode step (kept up while generating)
        _case("weigh_decode_b16", "weigh", "bf16", 16, 32, 8, 128, 16, (1, 4095), (1, 1), lens=1),
        # the weight of every key after a chunk of 128 prompt tokens
        _case("weigh_chunk_b8", "weigh", "fp16", 8, 32, 8, 128, 16, (0, 3968), (128, 128), lens=6),
        # one sequence cut to half its length
        _case("evict_one", "evict", "bf16", 1, 32, 8, 128, 16, (2047, 2047), lens=3, budget=1024, recent=128),
        # long contexts cut to 4096 tokens a sequence
        _case("evict_b8_to_4096", "evict", "bf16", 8, 64, 8, 128, 64, (16384, 32767), lens=4, budget=4096, recent=512),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    """One more case of the ranges the listed ones stand for."""
    while True:
        op = rng.choice(["append", "attend", "attend", "attend", "weigh", "evict"])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 6, 8])
        batch = _log_int(rng, 1, 33)
        past_hi = _log_int(rng, 1, 32767)
        past_lo = rng.randint(0, past_hi)
        new_hi = rng.choice([1, 1, _log_int(rng, 2, 8), _log_int(rng, 9, 2048)])
        new_lo = rng.choice([new_hi, rng.randint(1, new_hi)])
        window = rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]) if op in ("attend", "weigh") else 0
        budget = recent = 0
        if op == "evict":
            past_lo = max(1, past_lo)
            new_lo = new_hi = 0
            budget = rng.randint(1, past_hi)
            recent = rng.randint(0, budget)
        c = _case(None, op, rng.choice(["bf16", "fp16"]), batch, kv * group, kv, rng.choice([64, 128]),
                  rng.choice([16, 32, 64, 128]), (past_lo, past_hi), (new_lo, new_hi), lens=rng.randint(1, 1 << 30),
                  window=window, budget=budget, recent=recent, interleaved=rng.random() < 0.3)
        del c["name"]
        w = work(c)
        pool = (sum(sum(x) for x in _lengths(c)) + batch * c["page"]) * kv * c["head_size"] * 4
        if pool > 8.0e8 or w["bytes"] > 7.0e8:
            continue
        if w["flops"] > (1.3e11 if op == "attend" else 1.6e10):
            continue
        return c


# ---------------------------------------------------------------------------
# lengths, work, inputs
# ---------------------------------------------------------------------------
def _lengths(case):
    """(past, new) of every sequence."""
    rng = random.Random(case["lens"])
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(case["batch"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return past, new


def _pairs(past, new, window):
    """Visible (token, key) pairs of one sequence."""
    if window <= 0:
        return new * past + new * (new + 1) // 2
    return sum(min(past + i + 1, window) for i in range(new))


def _keys(past, new, window):
    """Keys that any new token of the sequence sees."""
    if new == 0:
        return 0
    return past + new - (max(0, past + 1 - window) if window > 0 else 0)


def work(case):
    past, new = _lengths(case)
    h, kv, d, win = case["heads"], case["kv_heads"], case["head_size"], case["window"]
    tokens = sum(new)
    pairs = sum(_pairs(p, n, win) for p, n in zip(past, new))
    keys = sum(_keys(p, n, win) for p, n in zip(past, new))
    if case["op"] == "append":
        # rows in and out, the cos and sin rows, the two norm weights
        return {"bytes": tokens * ((h + 2 * kv) * d * 4 + d * 2) + 4 * d, "flops": tokens * (h + kv) * d * 7}
    if case["op"] == "attend":
        return {"bytes": keys * kv * d * 4 + tokens * h * d * 4, "flops": 4 * d * h * pairs}
    if case["op"] == "weigh":
        # old weights are read, every key's weight in reach is written
        old = sum(_keys(p, n, win) - n for p, n in zip(past, new))
        return {"bytes": keys * kv * (d * 2 + 4) + old * kv * 4 + tokens * h * (d * 2 + 4), "flops": 2 * d * h * pairs}
    kept = sum(min(p, case["budget"]) for p in past)
    return {"bytes": sum(past) * kv * 4 + kept * kv * (d * 8 + 8), "flops": sum(past) * kv}


def _randn(gen, *shape, dtype):
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


def _tables(gen, lengths, page, spare=0):
    """A pool of pages in random order: block table [B, columns] (unused
    entries -1), its pages, and a second table of ``spare`` tokens a sequence
    on pages of its own."""
    need = [-(-n // page) for n in lengths]
    extra = [-(-min(n, spare) // page) for n in lengths] if spare else [0] * len(lengths)
    n_pages = sum(need) + sum(extra) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    tables, at = [], 0
    for counts in (need, extra):
        t = torch.full((len(lengths), max(1, max(counts))), -1, dtype=torch.int32, device="cuda")
        for b, c in enumerate(counts):
            t[b, :c] = order[at:at + c]
            at += c
        tables.append(t)
    return tables[0], tables[1], n_pages


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    past, new = _lengths(case)
    total = [p + n for p, n in zip(past, new)]
    t = DTYPES[case["dtype"]]
    h, kv, d, page = case["heads"], case["kv_heads"], case["head_size"], case["page"]
    tokens = sum(new)
    table, dst, n_pages = _tables(gen, total, page, case["budget"])
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = {"case": case, "past": past, "new": new, "total": max(total), "max_new": max(new), "table": table,
         "cu": torch.tensor(cu, dtype=torch.int32, device="cuda"),
         "seqlens": torch.tensor(past, dtype=torch.int32, device="cuda"),
         "k_pages": _randn(gen, n_pages, kv, page, d, dtype=t),
         # values of a layer with some outlying channels
         "v_pages": (torch.randn(n_pages, kv, page, d, generator=gen, device="cuda")
                     * (0.5 + torch.rand(d, generator=gen, device="cuda"))).to(t)}
    op = case["op"]
    if op == "append":
        s["query"] = _randn(gen, tokens, h * d, dtype=t)
        s["key"] = _randn(gen, tokens, kv * d, dtype=t)
        s["value"] = _randn(gen, tokens, kv * d, dtype=t)
        s["q_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(t)
        s["k_weight"] = (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(t)
        inv = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") * 2 / d)
        ang = torch.arange(max(total), dtype=torch.float64, device="cuda")[:, None] * inv
        s["cos"], s["sin"] = torch.cos(ang).to(t), torch.sin(ang).to(t)
        s["query_out"] = torch.empty_like(s["query"])
    elif op == "attend":
        s["query"] = _randn(gen, tokens, h * d, dtype=t)
        s["output"] = torch.empty_like(s["query"])
        s["lse"] = torch.empty(tokens, h, dtype=torch.float32, device="cuda")
    elif op == "weigh":
        s["query"] = _randn(gen, tokens, h * d, dtype=t)
        s["weights_in"] = torch.rand(n_pages, kv, page, generator=gen, device="cuda")
        s["weights"] = torch.zeros(n_pages, kv, page, device="cuda")
        s["lse"] = _attend(s, want_output=False)[1]
    else:
        # accumulated weights are heavy-tailed: a few keys take most of it
        s["weights"] = torch.exp(2 * torch.randn(n_pages, kv, page, generator=gen, device="cuda"))
        s["dst"] = dst
    if own:
        import shared_kv_cache_gb300 as gqa
        s["workspace"] = gqa.Workspace()
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _plain_norm_rotate(x, weight, cos, sin, interleaved):
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    half = x.shape[-1] // 2
    c, s = cos.float()[:, None], sin.float()[:, None]
    x1, x2 = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y1, y2 = x1 * c - x2 * s, x2 * c + x1 * s
    return torch.stack((y1, y2), -1).flatten(-2) if interleaved else torch.cat((y1, y2), -1)


def _append(s):
    c = s["case"]
    t, d, page = DTYPES[c["dtype"]], c["head_size"], c["page"]
    n = s["query"].shape[0]
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(c["batch"], device="cuda"), new, output_size=n)
    pos = torch.arange(n, device="cuda") - s["cu"][b] + s["seqlens"][b]
    q = _plain_norm_rotate(s["query"].view(n, -1, d), s["q_weight"], s["cos"][pos], s["sin"][pos], c["interleaved"])
    k = _plain_norm_rotate(s["key"].view(n, -1, d), s["k_weight"], s["cos"][pos], s["sin"][pos], c["interleaved"])
    where = s["table"][b, pos // page].long(), slice(None), pos % page
    s["k_pages"][where] = k.to(t)
    s["v_pages"][where] = s["value"].view(n, -1, d)
    return q.to(t).flatten(1), s["k_pages"], s["v_pages"]


def _gather(pages, table, b, length):
    """The first ``length`` rows of sequence b: [KV heads, length, ...]."""
    rows = pages[table[b, :-(-length // pages.shape[2])].long()]
    return rows.transpose(0, 1).flatten(1, 2)[:, :length]


def _scores(s, b, first):
    """Masked, scaled scores [KV heads, group, new, past + new] of one
    sequence whose tokens start at row ``first``."""
    c = s["case"]
    d, p, n = c["head_size"], s["past"][b], s["new"][b]
    k = _gather(s["k_pages"], s["table"], b, p + n).float()
    q = s["query"][first:first + n].float().view(n, c["kv_heads"], -1, d).permute(1, 2, 0, 3)
    x = torch.matmul(q, k[:, None].transpose(-1, -2)) * (1 / math.sqrt(d))
    i = torch.arange(p, p + n, device="cuda")[:, None]
    j = torch.arange(p + n, device="cuda")
    hide = j > i
    if c["window"] > 0:
        hide = hide | (j <= i - c["window"])
    return x.masked_fill_(hide, -math.inf)


def _attend(s, want_output=True):
    c = s["case"]
    t = DTYPES[c["dtype"]]
    outs, lses, first = [], [], 0
    for b, n in enumerate(s["new"]):
        x = _scores(s, b, first)
        m = x.amax(-1, keepdim=True)
        x = torch.exp_(x.sub_(m))
        total = x.sum(-1, keepdim=True)
        lses.append((m + torch.log(total)).squeeze(-1).permute(2, 0, 1).flatten(1))
        if want_output:
            v = _gather(s["v_pages"], s["table"], b, s["past"][b] + n).float()
            o = torch.matmul(x, v[:, None]) / total
            outs.append(o.permute(2, 0, 1, 3).flatten(1).to(t))
        first += n
    return torch.cat(outs) if want_output else None, torch.cat(lses)


def _weigh(s):
    page, first = s["case"]["page"], 0
    for b, n in enumerate(s["new"]):
        p, lse = s["past"][b], s["lse"][first:first + n]
        x = _scores(s, b, first)
        x = torch.exp_(x.sub_(lse.t().reshape(x.shape[0], x.shape[1], n, 1)))
        w = x.sum((1, 2))
        w[:, :p] += _gather(s["weights_in"], s["table"], b, p + n)[:, :p]
        j = torch.arange(_first_key(s, b), p + n, device="cuda")
        s["weights"][s["table"][b, j // page].long(), :, j % page] = w[:, j].t()
        first += n
    return s["weights"]


def _first_key(s, b):
    win = s["case"]["window"]
    return max(0, s["past"][b] + 1 - win) if win > 0 else 0


def _evict(s):
    c = s["case"]
    page, budget, recent = c["page"], c["budget"], c["recent"]
    kept = torch.full((c["batch"], c["kv_heads"], budget), -1, dtype=torch.int32, device="cuda")
    head = torch.arange(c["kv_heads"], device="cuda")[:, None]
    for b, n in enumerate(s["past"]):
        if n <= budget:
            idx = torch.arange(n, device="cuda").expand(c["kv_heads"], n)
        else:
            w = _gather(s["weights"], s["table"], b, n)[:, :max(0, n - recent)]
            top = torch.sort(w, dim=-1, descending=True, stable=True)[1][:, :budget - recent]
            last = torch.arange(n - recent, n, device="cuda").expand(c["kv_heads"], recent)
            idx = torch.cat((torch.sort(top, dim=-1)[0], last), -1)
        m = idx.shape[1]
        kept[b, :, :m] = idx
        j = torch.arange(m, device="cuda")
        to = s["dst"][b, j // page].long(), head, j % page
        frm = s["table"][b, idx // page].long(), head, idx % page
        for pool in (s["k_pages"], s["v_pages"], s["weights"]):
            pool[to] = pool[frm]
    return kept, torch.clamp(s["seqlens"], max=budget), s["k_pages"], s["v_pages"], s["weights"]


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _append, "attend": _attend, "weigh": _weigh, "evict": _evict}[op](s)
    import shared_kv_cache_gb300 as gqa
    if op == "append":
        q = gqa.paged_append(s["query"], s["key"], s["value"], s["k_pages"], s["v_pages"], s["table"], s["cu"],
                             s["seqlens"], s["total"], s["q_weight"], s["k_weight"], EPS, s["cos"], s["sin"],
                             query_out=s["query_out"], rotary_interleaved=int(s["case"]["interleaved"]))
        return q, s["k_pages"], s["v_pages"]
    if op == "attend":
        out = gqa.paged_attention(s["query"], s["k_pages"], s["v_pages"], s["table"], s["cu"], s["seqlens"],
                                  s["max_new"], s["total"], local_window_size=s["case"]["window"],
                                  output=s["output"], lse=s["lse"], workspace=s["workspace"])
        return out, s["lse"]
    if op == "weigh":
        return gqa.paged_key_weights(s["query"], s["lse"], s["k_pages"], s["weights"], s["table"], s["cu"],
                                     s["seqlens"], s["max_new"], s["total"], local_window_size=s["case"]["window"],
                                     weights_in=s["weights_in"], workspace=s["workspace"])
    kept, left = gqa.paged_evict(s["k_pages"], s["v_pages"], s["weights"], s["table"], s["seqlens"], s["total"],
                                 s["case"]["budget"], s["case"]["recent"], dst_block_table=s["dst"],
                                 workspace=s["workspace"])
    return kept, left, s["k_pages"], s["v_pages"], s["weights"]


# ---------------------------------------------------------------------------
# the same outputs in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op, d, page = case["op"], case["head_size"], case["page"]
    kv, group = case["kv_heads"], case["heads"] // case["kv_heads"]
    if op == "append":
        return _exact_append(s)
    if op == "evict":
        return _exact_evict(s)
    flat_k, flat_v = s["k_pages"].double(), s["v_pages"].double()
    n_rows = s["query"].shape[0]
    out = torch.zeros(n_rows, kv, group, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(n_rows, kv, group, dtype=torch.float64, device="cuda")
    weights = s["weights"].double() if op == "weigh" else None
    q_all = s["query"].double().reshape(n_rows, kv, group, d)
    row0 = 0
    for b in range(case["batch"]):
        p, n = s["past"][b], s["new"][b]
        slots = torch.arange(_first_key(s, b), p + n, device="cuda")
        pg, off = s["table"][b].long()[torch.div(slots, page, rounding_mode="floor")], slots.remainder(page)
        at = torch.arange(p, p + n, device="cuda").repeat_interleave(group)
        seen = slots[None] <= at[:, None]
        if case["window"] > 0:
            seen &= slots[None] + case["window"] > at[:, None]
        for h in range(kv):
            z = q_all[row0:row0 + n, h].reshape(n * group, d) @ flat_k[pg, h, off].T / math.sqrt(d)
            if op == "attend":
                z = torch.where(seen, z, -math.inf)
                z_max = z.max(1)[0]
                e = torch.exp(z - z_max[:, None])
                tot = e.sum(1)
                out[row0:row0 + n, h] = ((e @ flat_v[pg, h, off]) / tot[:, None]).reshape(n, group, d)
                lse[row0:row0 + n, h] = (z_max + tot.log()).reshape(n, group)
            else:
                given = s["lse"][row0:row0 + n, h * group:(h + 1) * group].double().reshape(-1, 1)
                got = torch.where(seen, torch.exp(z - given), 0.0).sum(0)
                weights[pg, h, off] = got + torch.where(slots < p, s["weights_in"][pg, h, off].double(), 0.0)
        row0 += n
    if op == "weigh":
        return weights
    return out.reshape(n_rows, -1), lse.reshape(n_rows, -1)


def _exact_append(s):
    case = s["case"]
    d, page = case["head_size"], case["page"]
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    n_rows = s["query"].shape[0]
    rows = []
    for name, weight in (("query", "q_weight"), ("key", "k_weight")):
        x = s[name].double().reshape(n_rows, -1, d)
        rows.append(x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt() * s[weight].double())
    first = 0
    turned = [torch.empty_like(r) for r in rows]
    for b in range(case["batch"]):
        p, n = s["past"][b], s["new"][b]
        turn = torch.complex(s["cos"][p:p + n].double(), s["sin"][p:p + n].double())[:, None]
        for x, y in zip(rows, turned):
            x, y = x[first:first + n], y[first:first + n]
            if case["interleaved"]:
                z = torch.complex(x[..., ::2], x[..., 1::2]) * turn
                y[..., ::2], y[..., 1::2] = z.real, z.imag
            else:
                z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * turn
                y[..., :d // 2], y[..., d // 2:] = z.real, z.imag
        for i in range(0, n, page):  # the rows of one page at most, page by page
            lo = p + i
            while lo < min(p + i + page, p + n):
                hi = min((lo // page + 1) * page, p + i + page, p + n)
                g = int(s["table"][b, lo // page])
                r = slice(first + lo - p, first + hi - p)
                o = slice(lo % page, lo % page + hi - lo)
                k_pages[g, :, o] = turned[1][r].transpose(0, 1)
                v_pages[g, :, o] = s["value"][r].double().reshape(hi - lo, -1, d).transpose(0, 1)
                lo = hi
        first += n
    return turned[0].reshape(n_rows, -1), k_pages, v_pages


def _exact_evict(s):
    case = s["case"]
    page, budget, recent, kv = case["page"], case["budget"], case["recent"], case["kv_heads"]
    pools = [s["k_pages"].double(), s["v_pages"].double(), s["weights"].double()]
    weights, table, dst = s["weights"].cpu().numpy(), s["table"].cpu().numpy(), s["dst"].cpu().numpy()
    kept = np.full((case["batch"], kv, budget), -1, np.int32)
    for b, n in enumerate(s["past"]):
        slot = np.arange(n)
        for h in range(kv):
            w = weights[table[b, slot // page], h, slot % page].astype(np.float64)
            w[max(0, n - recent):] = np.inf
            order = np.lexsort((slot, -w))[:budget]  # heaviest first, ties by the lower slot
            keep = np.sort(order)
            kept[b, h, :len(keep)] = keep
            j = np.arange(len(keep))
            to = torch.from_numpy(dst[b, j // page]).long().cuda(), h, torch.from_numpy(j % page).cuda()
            frm = (torch.from_numpy(table[b, keep // page]).long().cuda(), h, torch.from_numpy(keep % page).cuda())
            for pool in pools:
                pool[to] = pool[frm]
    left = torch.tensor([min(n, budget) for n in s["past"]], dtype=torch.int32, device="cuda")
    return torch.from_numpy(kept).cuda(), left, pools[0], pools[1], pools[2]
