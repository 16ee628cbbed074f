"""Measured cases of the operators that a server of many requests needs around the decoder's layers.

Three operators:

  plan    the indices of a step, from the requests' lengths: pages handed out and taken back, the place
          and position of every new token, the sequence that it belongs to
  lora    the requests' own low-rank adapters beside projections that share their input:
          y[t] = base[t] + s[a] * B[a] (A[a] x[t]), a the adapter of token t (none: y = base)
  sample  the next token of every row of logits: temperature, top-k, top-p, min-p, from a given random
          number, and its log-probability under the model

`own` false: elementary torch operations, in 32 bits (64 for the sums that tokens are drawn by).  `own`
true: the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one token for each of a few requests: latency
        {"name": "plan b8 decode", "op": "plan", "batch": 8, "page": 16, "max_pages": 256, "capacity": 8, "prompts": 0,
         "finished": 0, "short": False},
        # a full server: most requests at one token, some prompts in pieces, some requests over
        {"name": "plan b512 32768 tokens", "op": "plan", "batch": 512, "page": 64, "max_pages": 512, "capacity": 32768,
         "prompts": 24, "finished": 16, "short": False},
        # one request's q|k|v, 3B-shaped: latency
        {"name": "lora b1 qkv r16", "op": "lora", "tokens": 1, "k": 2048, "ns": "2048+256+256", "rank": 16, "adapters": 1,
         "loaded": 4, "idle": 0, "runs": False},
        # a decode batch in which every request has its own adapter, 14B-shaped gate|up
        {"name": "lora b64 gate|up r16", "op": "lora", "tokens": 64, "k": 5120, "ns": "13824+13824", "rank": 16,
         "adapters": 48, "loaded": 64, "idle": 9, "runs": False},
        # a wide decode batch over some popular adapters, 32B-shaped q|k|v
        {"name": "lora b256 qkv r64", "op": "lora", "tokens": 256, "k": 5120, "ns": "5120+1024+1024", "rank": 64,
         "adapters": 24, "loaded": 32, "idle": 30, "runs": False},
        # one request's long down projection, a high rank
        {"name": "lora b5 down r128", "op": "lora", "tokens": 5, "k": 27648, "ns": "5120", "rank": 128, "adapters": 5,
         "loaded": 8, "idle": 0, "runs": False},
        # prompts of several requests, 14B-shaped o
        {"name": "lora 8191 tokens o r16", "op": "lora", "tokens": 8191, "k": 5120, "ns": "5120", "rank": 16, "adapters": 5,
         "loaded": 16, "idle": 700, "runs": True},
        # prompts of several requests, 20B-shaped gate|up, a rank as adapters for hard tasks have it
        {"name": "lora 4099 gate|up r64", "op": "lora", "tokens": 4099, "k": 6144, "ns": "16384+16384", "rank": 64,
         "adapters": 3, "loaded": 8, "idle": 0, "runs": True},
        # one user's next token, the usual settings
        {"name": "sample b1 151936 k50", "op": "sample", "batch": 1, "vocab": 151936, "stride": 151936, "type": "bf16",
         "settings": "chat", "masked": 0.0},
        # a batch whose settings differ from row to row (greedy ones, unrestricted ones), an odd vocabulary
        {"name": "sample b16 50001 mixed", "op": "sample", "batch": 16, "vocab": 50001, "stride": 50001, "type": "f32",
         "settings": "mixed", "masked": 0.5},
        # a full server, the usual settings
        {"name": "sample b256 151936 chat", "op": "sample", "batch": 256, "vocab": 151936, "stride": 151936,
         "type": "bf16", "settings": "chat", "masked": 0.0},
        # samples for training or evaluation: the whole distribution, in 32 bits
        {"name": "sample b128 151936 plain", "op": "sample", "batch": 128, "vocab": 151936, "stride": 152064,
         "type": "f32", "settings": "plain", "masked": 0.0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["plan", "lora", "lora", "sample", "sample"])
    if op == "plan":
        batch = _log(rng, 1, 1024)
        prompts = rng.choice([0, 0, rng.randint(1, max(1, batch // 8))])
        finished = rng.choice([0, rng.randint(0, batch // 8)])
        return {"op": op, "batch": batch, "page": rng.choice([16, 32, 64, 128, 256]), "max_pages": rng.randint(64, 512),
                "capacity": batch + (_log(rng, 16, 31744) if prompts else rng.choice([0, 3])), "prompts": prompts,
                "finished": finished, "short": rng.random() < 0.25}
    if op == "sample":
        vocab = _log(rng, 100, 200000)
        return {"op": op, "batch": _log(rng, 1, max(1, min(512, 128 * 151936 // vocab))), "vocab": vocab,
                "stride": rng.choice([vocab, vocab, -(-vocab // 64) * 64]), "type": rng.choice(["bf16", "bf16", "f32"]),
                "settings": rng.choice(["chat", "mixed", "mixed", "plain"]), "masked": rng.choice([0.0, 0.0, 0.5])}
    k = 64 * _log(rng, 8, 432)
    ns = [rng.choice([8, 64, 1]) * _log(rng, 16, 256) for _ in range(rng.choice([1, 1, 2, 3]))]
    rank = rng.choice([8, 16, 16, 32, 64, 128])
    most = 4099 * (6144 + 4 * 16384) // (k + 2 * sum(ns))
    tokens = _log(rng, 1, max(1, min(16384, most)))
    runs = tokens > 512 or rng.random() < 0.3
    idle = rng.choice([0, tokens // 10])
    weights = 2 * rank * (len(ns) * k + sum(ns))  # of one adapter
    adapters = _log(rng, 1, max(1, min(tokens - idle, 8 if runs else 64, int(3e8) // weights)))
    return {"op": op, "tokens": tokens, "k": k, "ns": "+".join(map(str, ns)), "rank": rank, "adapters": adapters,
            "loaded": adapters + rng.choice([0, 5]), "idle": idle, "runs": runs}


def _ns(case):
    """The widths of the projections that share x."""
    return [int(n) for n in case["ns"].split("+")]


def work(case):
    op = case["op"]
    if op == "plan":
        # lengths, counts, starts; every token's place, position and sequence; an entry for every new page
        pages = case["capacity"] // case["page"] + case["prompts"]
        return {"bytes": 16 * case["batch"] + 16 * case["capacity"] + 8 * pages, "flops": 0}
    if op == "sample":
        n = case["batch"] * case["vocab"]
        return {"bytes": n * (2 if case["type"] == "bf16" else 4) + 28 * case["batch"], "flops": 3 * n}
    t, k, n, r = case["tokens"], case["k"], sum(_ns(case)), case["rank"]
    used = t - case["idle"]
    weights = case["adapters"] * r * (len(_ns(case)) * k + n)
    return {"bytes": 2 * used * k + 4 * t * n + 2 * weights + 4 * t + 4 * case["adapters"],
            "flops": 2 * used * r * (len(_ns(case)) * k + n)}


# ---------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------
def _ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    s = {"case": case}
    {"plan": _prepare_plan, "lora": _prepare_lora, "sample": _prepare_sample}[case["op"]](case, s, g, rng)
    return s


def _prepare_plan(case, s, g, rng):
    b, page, wide = case["batch"], case["page"], case["max_pages"]
    role = rng.permutation(b)
    new = np.ones(b, dtype=np.int64)
    new[role < case["finished"]] = -1
    prompt = role >= b - case["prompts"]
    room = case["capacity"] - (new > 0).sum()
    if case["prompts"]:
        share = rng.dirichlet(np.full(case["prompts"], 2.0))
        new[prompt] += np.minimum(share * room, wide * page // 2).astype(np.int64)
    # lengths of requests under way: anything up to half the table, a page's last place and first place among them
    lengths = rng.integers(1, wide * page // 2, b)
    lengths[rng.random(b) < 0.2] = page * int(rng.integers(1, max(2, wide // 2)))
    lengths[prompt] = rng.choice([0, 0, page, page + 1], case["prompts"])
    held = -(-lengths // page)
    need = np.where(new > 0, -(-(lengths + np.maximum(new, 0)) // page) - held, 0)
    # a pool with room for all; where it is short, other requests hold the rest
    pages = b * (wide // 2 + 2) + case["capacity"] // page + 64
    count = int(need.sum()) // 2 if case["short"] else pages - int(held.sum())
    order = rng.permutation(pages)
    table = np.full((b, wide), -1, dtype=np.int64)
    table[np.arange(wide)[None] < held[:, None]] = order[:held.sum()]
    ring, first = np.full(pages, -1, dtype=np.int64), int(rng.integers(0, pages))
    ring[(first + np.arange(count)) % pages] = order[pages - count:]
    t = case["capacity"]
    s |= {"lengths": _ints(lengths), "new": _ints(new), "table": _ints(table), "free": _ints(ring),
          "free_state": _ints([first, count], torch.int64), "free_out": torch.zeros(2, dtype=torch.int64, device=DEV),
          "lengths_out": torch.zeros(b, dtype=torch.int32, device=DEV),
          "starts": torch.zeros(b + 1, dtype=torch.int32, device=DEV),
          "slots": torch.zeros(t, dtype=torch.int64, device=DEV),
          "positions": torch.zeros(t, dtype=torch.int32, device=DEV),
          "sequences": torch.zeros(t, dtype=torch.int32, device=DEV)}


def _prepare_lora(case, s, g, rng):
    t, k, r, loaded = case["tokens"], case["k"], case["rank"], case["loaded"]
    used = rng.permutation(loaded)[:case["adapters"]]
    # popular adapters have more of the tokens; every used one has some
    more = t - case["idle"] - len(used)
    weight = 1.0 / np.arange(1, len(used) + 1)
    counts = 1 + np.floor(more * weight / weight.sum()).astype(np.int64)
    counts[0] += t - case["idle"] - counts.sum()
    ids = np.concatenate([np.repeat(used, counts), np.full(case["idle"], -1)])
    if not case["runs"]:
        ids = rng.permutation(ids)
    s["ids"] = _ints(ids)

    def normal(shape, scale):
        return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(torch.bfloat16)

    s["x"] = normal((t, k), 1.0)
    s["a"] = [normal((loaded, r, k), k ** -0.5) for _ in _ns(case)]
    s["b"] = [normal((loaded, n, r), r ** -0.5) for n in _ns(case)]
    s["scales"] = torch.rand(loaded, generator=g, device=DEV) * 1.5 + 0.5
    s["base"] = [normal((t, n), 1.0) for n in _ns(case)]
    s["y"] = [torch.empty_like(x) for x in s["base"]]
    if own:
        import nf4_weight_only_gb300 as nf4

        s["plan"] = nf4.lora_plan_buffer(t, loaded)
        s["workspace"] = nf4.lora_workspace(t, loaded, r, len(_ns(case)))


def _prepare_sample(case, s, g, rng):
    b, v = case["batch"], case["vocab"]
    # near normal, with a head of likely tokens as a model's logits have it
    l = torch.randn((b, case["stride"]), generator=g, device=DEV) * 2.2
    head = torch.randint(0, v, (b, 48), generator=g, device=DEV)
    l.scatter_add_(1, head, torch.rand((b, 48), generator=g, device=DEV) * 10)
    if case["masked"]:  # what a grammar or a list of banned words rules out
        out = torch.rand(l.shape, generator=g, device=DEV) < case["masked"]
        l.masked_fill_(out, float("-inf"))
    s["logits"] = l.to(torch.bfloat16 if case["type"] == "bf16" else torch.float32)
    temperature, top_k, top_p, min_p = np.ones(b), np.zeros(b, np.int64), np.ones(b), np.zeros(b)
    if case["settings"] == "chat":
        temperature[:], top_k[:], top_p[:] = rng.uniform(0.6, 1.0, b), 50, 0.95
    elif case["settings"] == "mixed":
        temperature = rng.choice([0.0, 0.5, 0.7, 1.0, 1.3], b)
        top_k = rng.choice([0, 0, 1, 20, 40, 1000, v], b)
        top_p = rng.choice([1.0, 0.5, 0.9, 0.95, 0.99], b)
        min_p = rng.choice([0.0, 0.0, 0.02, 0.1], b)
    s["temperature"], s["top_p"], s["min_p"] = (_ints(x, torch.float32) for x in (temperature, top_p, min_p))
    s["top_k"] = _ints(top_k)
    s["random"] = torch.rand(b, generator=g, device=DEV)
    s["tokens"] = torch.zeros(b, dtype=torch.int32, device=DEV)
    s["logprobs"] = torch.zeros(b, dtype=torch.float32, device=DEV)


# ---------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    return _own(op, s) if own else {"plan": _plain_plan, "lora": _plain_lora, "sample": _plain_sample}[op](s)


def _own(op, s):
    import nf4_weight_only_gb300 as nf4

    if op == "plan":
        nf4.nf4_plan_step(s["lengths"], s["new"], s["case"]["page"], s["table"], s["free"], s["free_state"], s["free_out"],
                          s["lengths_out"], s["starts"], s["slots"], s["positions"], s["sequences"])
        return _plan_out(s)
    if op == "lora":
        nf4.nf4_lora_plan(s["ids"], s["case"]["loaded"], s["plan"])
        nf4.nf4_lora(s["x"], s["plan"], s["scales"], s["a"], s["b"], s["y"], s["workspace"], bases=s["base"])
        return s["y"]
    nf4.nf4_sample(s["logits"], s["random"], s["tokens"], temperature=s["temperature"], top_k=s["top_k"],
                   top_p=s["top_p"], min_p=s["min_p"], vocab=s["case"]["vocab"], logprobs=s["logprobs"])
    return s["tokens"], s["logprobs"]


def _plan_out(s):
    return {n: s[n] for n in ("lengths_out", "table", "free", "free_out", "starts", "slots", "positions", "sequences")}


def _plain_plan(s):
    page, (b, wide), pages, t = s["case"]["page"], s["table"].shape, s["free"].shape[0], s["case"]["capacity"]
    length, new, table, ring = s["lengths"].long(), s["new"].long(), s["table"], s["free"]
    over, some = new < 0, new.clamp_min(0)
    start = torch.cumsum(some, 0) - some
    held, after = (length + page - 1) // page, (length + some + page - 1) // page
    fits = (after <= wide) & (start + some <= t)
    need = torch.where(fits & ~over, after - held, 0)
    back = torch.where(over, held, 0)
    first, count = s["free_state"][0], s["free_state"][1]
    upto, returned = torch.cumsum(need, 0), torch.cumsum(back, 0)
    served = fits & ((need == 0) | (upto <= count + returned[-1])) & ~over
    s["lengths_out"].copy_(torch.where(over, 0, torch.where(served, length + some, length)))
    s["starts"][:b] = start
    s["starts"][b:] = (start + some)[-1:]
    taken = torch.where(served, need, 0).sum()
    # what the finished sequences held goes to the ring's end, in order
    p = torch.arange(wide, device=DEV)[None]
    gone = over[:, None] & (p < held[:, None])
    at = torch.where(gone, (first + count + (returned - back)[:, None] + p) % pages, pages)
    ring = torch.cat((ring, ring[:1])).scatter(0, at.flatten(), table.flatten())[:pages]
    s["free"].copy_(ring)
    # the new pages of the served ones, in order
    fresh = served[:, None] & (p >= held[:, None]) & (p < after[:, None])
    k = (upto - need)[:, None] + p - held[:, None]
    table.copy_(torch.where(fresh, ring[(first + k) % pages], table))
    s["free_out"][0] = (first + taken) % pages
    s["free_out"][1] = count + returned[-1] - taken
    # tokens
    i = torch.arange(t, device=DEV)
    seq = (i[:, None] >= (start + some)[None]).sum(-1)
    real = seq < b
    seq = seq.clamp_max(b - 1)
    pos = length[seq] + i - start[seq]
    there = real & served[seq]
    slot = table[seq, (pos // page).clamp_max(wide - 1)].long() * page + pos % page
    s["slots"].copy_(torch.where(there, slot, -1))
    s["positions"].copy_(torch.where(real, pos, 0))
    s["sequences"].copy_(torch.where(real, seq, -1))
    return _plan_out(s)


def _plain_lora(s):
    ids, x = s["ids"], s["x"].float()
    mine = ids[:, None] == torch.arange(s["scales"].shape[0], device=DEV)[None]
    factor = torch.where(mine, s["scales"][None], 0.0)[..., None]  # [T, adapters, 1]
    # every adapter's product; the token's own is kept
    s["y"] = [_plain_adapter(x, factor, a, b, base) for a, b, base in zip(s["a"], s["b"], s["base"])]
    return s["y"]


def _plain_adapter(x, factor, a, b, base):
    h = (x @ a.flatten(0, 1).float().T).view(x.shape[0], a.shape[0], a.shape[1]) * factor
    return (base.float() + h.flatten(1) @ b.transpose(1, 2).flatten(0, 1).float()).to(torch.bfloat16)


def _plain_sample(s):
    v = s["case"]["vocab"]
    l = s["logits"][:, :v].double()
    z = l - l.amax(-1, keepdim=True)
    lse = z.exp().sum(-1).log()
    heat = s["temperature"].double()[:, None]
    w = torch.where(heat == 0, (z == 0).double(), (z / torch.where(heat == 0, 1.0, heat)).exp())
    order = torch.sort(l, dim=-1, descending=True, stable=True).indices
    ranked = w.gather(-1, order)
    rank = torch.arange(v, device=DEV)[None]
    k = s["top_k"].long()[:, None]
    keep = (rank < k) | (k <= 0)
    upto = torch.where(keep, ranked, 0.0).cumsum(-1)
    p = s["top_p"].double()[:, None]
    keep &= (torch.nn.functional.pad(upto, (1, 0))[:, :-1] < p * upto[:, -1:]) | (p >= 1)
    keep &= ranked >= s["min_p"].double()[:, None]
    keep = torch.where(heat == 0, rank == 0, keep | (rank == 0))
    w = torch.where(torch.zeros_like(keep).scatter(-1, order, keep), w, 0.0)
    upto = w.cumsum(-1)
    token = (upto <= s["random"].double()[:, None] * upto[:, -1:]).sum(-1).clamp_max(v - 1)
    s["tokens"].copy_(token)
    s["logprobs"].copy_(z.gather(-1, token[:, None])[:, 0] - lse)
    return s["tokens"], s["logprobs"]


# ---------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "plan":
        return _exact_plan(case, s)
    if case["op"] == "sample":
        return _exact_sample(case, s)
    out = []
    ids = s["ids"].tolist()
    rows = {}
    for t, a in enumerate(ids):
        rows.setdefault(a, []).append(t)
    for a, b, base in zip(s["a"], s["b"], s["base"]):
        y = base.double()
        for adapter, at in rows.items():
            if adapter < 0:
                continue
            at = torch.tensor(at, device=DEV)
            low = torch.mm(a[adapter].double(), s["x"][at].double().t())
            y[at] += torch.mm(b[adapter].double(), low).t() * float(s["scales"][adapter])
        out.append(y)
    return out


def _exact_plan(case, s):
    """One sequence after the other, as a server's program on the host would do it."""
    from collections import deque

    page, t = case["page"], case["capacity"]
    table, ring = s["table"].tolist(), s["free"].tolist()
    first, count = s["free_state"].tolist()
    pages, wide = len(ring), case["max_pages"]
    lengths, new = s["lengths"].tolist(), s["new"].tolist()
    stock = deque(ring[(first + i) % pages] for i in range(count))
    end, returned = first + count, 0
    for b, n in enumerate(new):
        if n < 0:
            for q in table[b][:math.ceil(lengths[b] / page)]:
                stock.append(q)
                ring[(end + returned) % pages] = q
                returned += 1
    out_lengths, starts, slots, positions, sequences = [], [0], [-1] * t, [0] * t, [-1] * t
    taken, empty = 0, False
    for b, n in enumerate(new):
        if n < 0:
            out_lengths.append(0)
            starts.append(starts[-1])
            continue
        grown = lengths[b] + n
        held, want = math.ceil(lengths[b] / page), math.ceil(grown / page)
        ok = want <= wide and starts[-1] + n <= t
        if ok and want > held:
            # once one sequence had to be refused for want of pages, none after it gets any
            empty = empty or want - held > len(stock)
            ok = not empty
            if ok:
                for i in range(held, want):
                    table[b][i] = stock.popleft()
                    taken += 1
        for i in range(n):
            row = starts[-1] + i
            if row < t:
                sequences[row], positions[row] = b, lengths[b] + i
                if ok:
                    slots[row] = table[b][(lengths[b] + i) // page] * page + (lengths[b] + i) % page
        out_lengths.append(grown if ok else lengths[b])
        starts.append(starts[-1] + n)
    return {"lengths_out": _ints(out_lengths), "table": _ints(table), "free": _ints(ring),
            "free_out": _ints([(first + taken) % pages, count + returned - taken], torch.int64), "starts": _ints(starts),
            "slots": _ints(slots, torch.int64), "positions": _ints(positions), "sequences": _ints(sequences)}


def _exact_sample(case, s):
    tokens, logs = [], []
    v = case["vocab"]
    for i in range(case["batch"]):
        l = s["logits"][i, :v].double()
        logs_all = torch.log_softmax(l, 0)
        heat, k = float(s["temperature"][i]), int(s["top_k"][i])
        p, least, u = float(s["top_p"][i]), float(s["min_p"][i]), float(s["random"][i])
        top = l.max()
        if heat == 0:
            token = int(torch.nonzero(l == top)[0])
        else:
            odds = torch.exp((l - top) / heat)
            there = torch.nonzero(torch.isfinite(l))[:, 0]
            ranked = there[torch.argsort(l[there], descending=True, stable=True)]
            if 0 < k < len(ranked):
                ranked = ranked[:k]
            if p < 1:
                sums = torch.cumsum(odds[ranked], 0)
                ranked = ranked[:1 + int(torch.count_nonzero(sums < p * sums[-1]))]
            ranked = ranked[odds[ranked] >= min(least, 1.0)]
            among = torch.sort(ranked).values
            sums = torch.cumsum(odds[among], 0)
            token = int(among[min(len(among) - 1, int(torch.searchsorted(sums, u * sums[-1], right=True)))])
        tokens.append(token)
        logs.append(logs_all[token])
    return _ints(tokens), torch.stack(logs)
