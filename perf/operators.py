"""The operators around a beam-search decode step, as a user calls them, and their plain forms.

Five operators, each on the paged caches and beam tables of the attention calls:

* process: the logits of every beam row through repetition / frequency / presence penalties, token
  biases, temperature and a grammar mask, with the log-sum-exp of each processed row;
* select: the best continuations of each request over all of its beams' vocabularies;
* advance: the beams' histories and cache_indirection re-ordered by the chosen parents;
* weights: the attention weight each cached prompt key received from a step's query rows;
* evict: the cached rows of highest weight moved to the front of each request's pages.

``own`` chooses between the framework's calls and elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
PAGE = 32


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one interactive request, four beams, a full-precision head over a vocabulary of odd size
        dict(name="process_b1_w4_v50257_fp32", op="process", batch=1, beam=4, vocab=50257, dtype="fp32", prompt=700,
             tokens=5, bias=16, penalties=True, temperature=True, mask_rows=0),
        # a served batch: long prompts, penalties, biases and a temperature, no grammar
        dict(name="process_b64_w30_v128000_bf16", op="process", batch=64, beam=30, vocab=128000, dtype="bf16",
             prompt=500, tokens=4, bias=32, penalties=True, temperature=True, mask_rows=0),
        # wide-beam recommendation: item codes constrained by the states of a grammar
        dict(name="process_b128_w96_v32000_fp16_mask", op="process", batch=128, beam=96, vocab=32000, dtype="fp16",
             prompt=0, tokens=3, bias=0, penalties=True, temperature=False, mask_rows=256),
        # the same three situations for the choice of the beams
        dict(name="select_b1_w4_v50257_fp32_k8", op="select", batch=1, beam=4, vocab=50257, dtype="fp32", num=8,
             mask_rows=0),
        dict(name="select_b64_w30_v128000_bf16_k60", op="select", batch=64, beam=30, vocab=128000, dtype="bf16",
             num=60, mask_rows=0),
        dict(name="select_b128_w96_v32000_bf16_k192", op="select", batch=128, beam=96, vocab=32000, dtype="bf16",
             num=192, mask_rows=0),
        # beam bookkeeping of one request and of the widest batch
        dict(name="advance_b1_w4_t3", op="advance", batch=1, beam=4, tail=3),
        dict(name="advance_b128_w96_t7", op="advance", batch=128, beam=96, tail=7),
        # an image prompt's keys, weighed by its last 32 tokens
        dict(name="weights_prefill_b4_s1024_win32_fp16", op="weights", kind="prefill", batch=4, beam=1, q_heads=32,
             kv_heads=8, dim=128, dtype="fp16", lo=1024, hi=1024, cached=0, window=32),
        # every beam of a wide step weighs its request's prompt
        dict(name="weights_decode_b128_w96_d128_bf16", op="weights", kind="decode", batch=128, beam=96, q_heads=16,
             kv_heads=8, dim=128, dtype="bf16", lo=2800, hi=3200, cached=0, window=0),
        # one long cached prompt cut to 2048 rows, and a batch of prompts cut to 1024 rows each
        dict(name="evict_b1_p10000_keep2048_fp16", op="evict", batch=1, kv_heads=8, dim=128, dtype="fp16", lo=10000,
             hi=10000, keep=2048, sinks=4, recent=64),
        dict(name="evict_b128_p3000_keep1024_bf16", op="evict", batch=128, kv_heads=8, dim=128, dtype="bf16",
             lo=2800, hi=3200, keep=1024, sinks=4, recent=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["process", "select", "advance", "weights", "evict"])
    if op in ("process", "select"):
        vocab = _log(rng, 1000, 160000)
        beam = _log(rng, 1, 96)
        batch = min(_log(rng, 1, 128), max(1, int(2e8 / (vocab * beam))))
        case = dict(op=op, batch=batch, beam=beam, vocab=vocab, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    mask_rows=rng.choice([0, 0, 7, 100]))
        if op == "process":
            case.update(prompt=rng.choice([0, _log(rng, 1, 4000)]), tokens=rng.choice([0, _log(rng, 1, 300)]),
                        bias=rng.choice([0, _log(rng, 1, 300)]), penalties=rng.random() < 0.7,
                        temperature=rng.random() < 0.5)
        else:
            case.update(num=rng.randint(1, 2 * beam))
        return case
    if op == "advance":
        return dict(op=op, batch=_log(rng, 1, 128), beam=_log(rng, 1, 300), tail=rng.randint(0, 7))
    if op == "weights":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 8])
        group = rng.choice([1, 2, 3, 4, 8])
        kind = rng.choice(["prefill", "decode"])
        beam = 1 if kind == "prefill" else _log(rng, 1, 96)
        hi = _log(rng, 20, 6000)
        batch = _log(rng, 1, 24)
        return dict(op=op, kind=kind, batch=batch, beam=beam, q_heads=kv * group, kv_heads=kv, dim=dim,
                    dtype=rng.choice(["bf16", "fp16"]), lo=max(1, hi // rng.randint(1, 4)), hi=hi,
                    cached=0 if kind == "decode" else rng.choice([0, _log(rng, 1, 500)]),
                    window=0 if kind == "decode" else rng.randint(1, 64))
    hi = _log(rng, 20, 20000)
    return dict(op=op, batch=min(_log(rng, 1, 64), max(1, 300000 // hi)), kv_heads=rng.choice([1, 2, 8]),
                dim=rng.choice([64, 128, 256]), dtype=rng.choice(["bf16", "fp16"]), lo=max(1, hi // rng.randint(1, 4)),
                hi=hi, keep=_log(rng, 1, 20000), sinks=rng.randint(0, 8), recent=rng.choice([0, rng.randint(1, 300)]))


# ---------------------------------------------------------------- what a program holds before a call

def _lengths(case, rs):
    return rs.randint(case["lo"], case["hi"] + 1, case["batch"]).astype(np.int32)


def _pages(lens, most, rs):
    """Random page ids [batch][pages of most rows] (-1 behind a request's last page) and the pages of the pool."""
    need = -(-lens // PAGE)
    wide = -(-most // PAGE)
    total = wide * len(lens) + 3
    ids = rs.permutation(total).astype(np.int32)
    table = np.full((len(lens), wide), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, total


def _step_plan(bsp, case, tail):
    """A decode plan of a step whose attention is already done: what the logits' calls take."""
    geo = bsp.geometry(2, 1, 64, PAGE, 1, "bf16")
    ws = bsp.Workspace(geo, case["batch"], case["beam"], 1)
    zero = np.zeros(case["batch"], np.int32)
    return ws, ws.plan(geo, case["batch"], case["beam"], zero, zero + tail, np.zeros((case["batch"], 1), np.int32))


def _logits(case, gen):
    rows, vocab = case["batch"] * case["beam"], case["vocab"]
    return (torch.randn((rows, vocab), generator=gen, device="cuda") * 3).to(DTYPES[case["dtype"]])


def _mask(case, gen):
    """Grammar masks: mask_rows states that allow about 3% of the tokens each, packed 32 to a word, and each
    row's state (-1 for a row without one)."""
    rows, vocab, n = case["batch"] * case["beam"], case["vocab"], case["mask_rows"]
    if not n:
        return None, None
    words = (vocab + 31) // 32
    allow = torch.rand((n, words * 32), generator=gen, device="cuda") < 0.03
    allow[:, 0] = True
    shift = torch.arange(32, device="cuda")
    bits = (allow.view(n, words, 32).to(torch.int64) << shift).sum(-1)
    index = torch.randint(-1, n, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    return torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32), index


def _ints(gen, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=gen, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rs = np.random.RandomState(seed % (1 << 31))
    s = dict(case=case)
    bsp = None
    if own:
        from beam_search_shared_gb300 import bsp
        s["bsp"] = bsp
    batch = case["batch"]
    rand = lambda lo, hi: torch.rand(batch, generator=gen, device="cuda") * (hi - lo) + lo  # noqa: E731
    if case["op"] == "process":
        rows, vocab = batch * case["beam"], case["vocab"]
        s["logits"] = _logits(case, gen)
        s["mask"], s["mask_index"] = _mask(case, gen)
        for name, n, lead in (("prompt_tokens", case["prompt"], batch), ("tokens", case["tokens"], rows)):
            s[name] = _ints(gen, 0, vocab, (lead, n)) if n else None
            s[name + "_len"] = _ints(gen, (n + 1) // 2, n + 1, (lead,)) if n else None
        s["repetition"] = rand(1.0, 1.4) if case["penalties"] else None
        s["frequency"] = rand(0.0, 0.5) if case["penalties"] else None
        s["presence"] = rand(0.0, 0.5) if case["penalties"] else None
        s["temperature"] = rand(0.5, 1.5) if case["temperature"] else None
        n = case["bias"]
        s["bias_tokens"] = _ints(gen, 0, vocab, (batch, n)) if n else None
        s["bias_values"] = torch.randn((batch, n), generator=gen, device="cuda") * 4 if n else None
        s["out"], s["lse"] = torch.empty_like(s["logits"]), torch.empty(rows, device="cuda")
        if own:
            s["ws"], s["plan"] = _step_plan(bsp, case, min(case["tokens"], bsp.MAX_TAIL))
            s["params"] = bsp.LogitsParams(
                prompt_tokens=s["prompt_tokens"], prompt_token_len=s["prompt_tokens_len"], tokens=s["tokens"],
                token_len=s["tokens_len"], repetition_penalty=s["repetition"], frequency_penalty=s["frequency"],
                presence_penalty=s["presence"], temperature=s["temperature"], bias_tokens=s["bias_tokens"],
                bias_values=s["bias_values"], mask=s["mask"], mask_index=s["mask_index"])
    elif case["op"] == "select":
        s["logits"] = _logits(case, gen)
        s["mask"], s["mask_index"] = _mask(case, gen)
        s["lse"] = torch.cat([torch.logsumexp(x.float(), -1) for x in s["logits"].split(256)])
        s["cum"] = -torch.rand((batch, case["beam"]), generator=gen, device="cuda") * 8
        shape = (batch, case["num"])
        s["scores"] = torch.empty(shape, device="cuda")
        s["parents"] = torch.empty(shape, dtype=torch.int32, device="cuda")
        s["tokens"] = torch.empty(shape, dtype=torch.int32, device="cuda")
        if own:
            s["ws"], s["plan"] = _step_plan(bsp, case, 0)
            s["select_ws"] = bsp.beam_select_workspace(batch, case["beam"], case["vocab"], case["num"])
    elif case["op"] == "advance":
        beam, tail = case["beam"], case["tail"]
        s["parents"] = _ints(gen, 0, beam, (batch, beam))
        s["new"] = _ints(gen, 0, 32000, (batch, beam))
        s["indirection"] = _ints(gen, 0, beam, (batch, beam, 16))
        s["tokens"] = _ints(gen, 0, 32000, (batch * beam, 16))
        s["indirection_out"] = torch.zeros_like(s["indirection"])
        s["tokens_out"] = torch.zeros_like(s["tokens"])
        if own:
            s["ws"], s["plan"] = _step_plan(bsp, case, tail)
    else:
        kv, dim, dt = case["kv_heads"], case["dim"], DTYPES[case["dtype"]]
        lens = _lengths(case, rs)
        cached = np.full(batch, case.get("cached", 0), np.int32)
        keys = lens + cached
        most = case["hi"] + case.get("cached", 0)
        table, total = _pages(keys, most, rs)
        pool = lambda: torch.randn((total, kv, PAGE, dim), generator=gen, device="cuda").to(dt)  # noqa: E731
        s["k_pool"] = pool()
        s["pages"] = torch.from_numpy(table).cuda()
        s["keys"] = torch.from_numpy(keys).cuda()
        if own:
            q_heads = case.get("q_heads", kv)
            geo = bsp.geometry(q_heads, kv, dim, PAGE, total, case["dtype"])
            s["ws"] = bsp.Workspace(geo, batch, max(case.get("beam", 1), int(lens.max())) if case.get(
                "kind") == "prefill" else case.get("beam", 1), table.shape[1])
            if case.get("kind") == "prefill":
                s["plan"] = bsp.plan_prefill(geo, batch, cached, lens, table, True, s["ws"])
            else:
                s["plan"] = s["ws"].plan(geo, batch, case.get("beam", 1), keys, np.zeros(batch, np.int32), table)
        if case["op"] == "weights":
            if case["kind"] == "prefill":
                rows, first = lens, np.concatenate([[0], np.cumsum(lens)[:-1]])
                seen = np.minimum(lens, case["window"])
            else:
                rows, first = np.full(batch, case["beam"]), np.arange(batch) * case["beam"]
                seen = rows
            s["q"] = torch.randn((int(rows.sum()), case["q_heads"], dim), generator=gen, device="cuda").to(dt)
            n = int(seen.max())
            i = np.arange(n)[None]
            at = (first + rows - seen)[:, None] + np.minimum(i, seen[:, None] - 1)
            limit = (keys - seen)[:, None] + i + 1 if case["kind"] == "prefill" else np.repeat(keys[:, None], n, 1)
            limit = np.where(i < seen[:, None], limit, 0)
            s["rows"] = torch.from_numpy(at).cuda()
            s["limit"] = torch.from_numpy(limit).cuda()  # keys that the row sees
            s["scale"] = dim ** -0.5
            s["lse"] = torch.zeros((s["q"].shape[0], case["q_heads"]), device="cuda")
            for b in range(batch):
                part = slice(b, b + 1)
                logit = _scores(s, part, torch.float32)
                lse = torch.logsumexp(logit, -1).view(kv, -1, n).permute(2, 0, 1).reshape(n, -1)
                real = s["limit"][b] > 0
                s["lse"][s["rows"][b][real]] = lse[real]
            s["weights"] = torch.zeros((batch, kv, most), device="cuda")
        else:
            s["v_pool"] = pool()
            # heavy-tailed, as attention gives them
            s["weights"] = torch.exp(2 * torch.randn((batch, kv, most), generator=gen, device="cuda"))
            keep = np.minimum(keys, case["keep"])
            s["keep"] = torch.from_numpy(keep).cuda()
            s["kept"] = torch.full((batch, kv, most), -1, dtype=torch.int32, device="cuda")
            s["weights_out"] = torch.zeros((batch, kv, most), device="cuda")
    return s


# ---------------------------------------------------------------- plain forms

def _allowed(mask, index, vocab):
    """[rows][vocab]: what each row's grammar state lets through."""
    word = torch.arange(vocab, device="cuda")
    state = ((mask[:, word // 32] >> (word % 32)) & 1).bool()
    return state[index.clamp(min=0).long()] | (index < 0)[:, None]


def _seen(tokens, lens, rows, vocab):
    """[rows][vocab]: how often each token occurs in the first lens of a row's list."""
    count = torch.zeros((rows, vocab), dtype=torch.int32, device="cuda")
    if tokens is not None:
        live = torch.arange(tokens.shape[1], device="cuda")[None] < lens[:, None]
        count.scatter_add_(1, tokens.long(), live.to(torch.int32))
    return count


def _process(s):
    case = s["case"]
    batch, beam, vocab = case["batch"], case["beam"], case["vocab"]
    x = s["logits"].float().view(batch, beam, vocab)
    made = _seen(s["tokens"], s["tokens_len"], batch * beam, vocab).view(batch, beam, vocab)
    if s["repetition"] is not None:
        old = _seen(s["prompt_tokens"], s["prompt_tokens_len"], batch, vocab)[:, None]
        p = s["repetition"][:, None, None]
        x = torch.where((made > 0) | (old > 0), torch.where(x > 0, x / p, x * p), x)
    if s["frequency"] is not None:
        x = x - s["frequency"][:, None, None] * made
        x = x - s["presence"][:, None, None] * (made > 0)
    if s["bias_tokens"] is not None:
        # an id that is given twice: its first value counts
        n = s["bias_tokens"].shape[1]
        first = torch.full((batch, vocab), n, dtype=torch.int64, device="cuda")
        first.scatter_reduce_(1, s["bias_tokens"].long(), torch.arange(n, device="cuda").expand(batch, n), "amin")
        value = torch.cat([s["bias_values"], torch.zeros((batch, 1), device="cuda")], 1)
        x = x + value.gather(1, first)[:, None]
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None, None]
    x = x.view(batch * beam, vocab)
    if s["mask"] is not None:
        x = torch.where(_allowed(s["mask"], s["mask_index"], vocab), x, -math.inf)
    out = x.to(s["logits"].dtype)
    y = out.float()
    top = y.amax(-1, keepdim=True)
    return out, torch.log(torch.exp(y - top).sum(-1)) + top[:, 0]


def _select(s):
    """Score: the fp32 sum of the beam's score and the fp32 difference of logit and log-sum-exp; equal scores
    go by the lower beam, then the lower token."""
    case = s["case"]
    batch, beam, vocab = case["batch"], case["beam"], case["vocab"]
    x = s["logits"].float() - s["lse"][:, None]
    x = x.view(batch, beam, vocab) + s["cum"][:, :, None]
    if s["mask"] is not None:
        x = torch.where(_allowed(s["mask"], s["mask_index"], vocab).view(x.shape), x, -math.inf)
    x = x.view(batch, beam * vocab)
    bits = x.view(torch.int32)
    rank = torch.where(bits < 0, bits ^ 0x7fffffff, bits).to(torch.int64) << 32
    rank = rank | (0xffffffff - torch.arange(beam * vocab, device="cuda"))
    at = 0xffffffff - (torch.topk(rank, case["num"]).values & 0xffffffff)
    scores = x.gather(1, at)
    none = scores == -math.inf
    return (scores, torch.where(none, -1, at // vocab).to(torch.int32),
            torch.where(none, -1, at % vocab).to(torch.int32))


def _advance(s):
    case = s["case"]
    batch, beam, tail = case["batch"], case["beam"], case["tail"]
    at = s["parents"].long()[:, :, None].expand(batch, beam, tail)
    s["indirection_out"][:, :, :tail] = s["indirection"].gather(1, at)
    s["indirection_out"][:, :, tail] = torch.arange(beam, device="cuda", dtype=torch.int32)
    old = s["tokens"].view(batch, beam, -1)
    out = s["tokens_out"].view(batch, beam, -1)
    out[:, :, :tail] = old.gather(1, at)
    out[:, :, tail] = s["new"]
    return s["indirection_out"], s["tokens_out"]


def _rows_of(pool, pages, most, dtype):
    """[batch][kv head][most][dim]: the pool's rows of each request in order."""
    x = pool[pages.clamp(min=0).long()]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :most].to(dtype)


def _scores(s, part, dtype):
    """[requests][kv head][query heads of it x rows][keys] of a slice of the batch: scaled scores, -inf where
    the row does not see the key."""
    case = s["case"]
    kv, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    limit = s["limit"][part]
    most = int(s["pages"].shape[1]) * PAGE
    q = s["q"][s["rows"][part]].to(dtype)
    q = q.unflatten(2, (kv, group)).permute(0, 2, 3, 1, 4)  # [requests][kv][group][rows][dim]
    k = _rows_of(s["k_pool"], s["pages"][part], most, dtype)
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).unflatten(2, (group, -1)) * s["scale"]
    see = torch.arange(most, device="cuda")[None, None] < limit[:, :, None]
    return x.masked_fill(~see[:, None, None], -math.inf).flatten(2, 3)


def _weigh(s, part, dtype):
    case = s["case"]
    kv = case["kv_heads"]
    lse = s["lse"][s["rows"][part]].to(dtype).unflatten(2, (kv, -1)).permute(0, 2, 3, 1).flatten(2, 3)
    return torch.exp(_scores(s, part, dtype) - lse[..., None]).sum(2)


def _weights(s):
    out = s["weights"]
    out.copy_(_weigh(s, slice(None), torch.float32)[:, :, :out.shape[2]])
    return out


def _evict(s):
    case = s["case"]
    w, batch, kv = s["weights"], case["batch"], case["kv_heads"]
    slot = torch.arange(w.shape[2], device="cuda").expand(w.shape)
    keys, keep = s["keys"][:, None, None], s["keep"][:, None, None]
    fixed = (slot < case["sinks"]) | (slot >= keys - case["recent"])
    x = torch.where(fixed, math.inf, w).masked_fill(slot >= keys, -math.inf)
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices
    live = torch.zeros(w.shape, dtype=torch.bool, device="cuda").scatter_(2, order, slot < keep)
    # the i-th evicted slot in front of keep takes the i-th kept row from behind it
    hole, mover = ~live & (slot < keep), live & (slot >= keep)
    holes = torch.sort((~hole).to(torch.int8), dim=-1, stable=True).indices
    movers = torch.sort((~mover).to(torch.int8), dim=-1, stable=True).indices
    pair = slot < hole.sum(-1, keepdim=True)
    source = slot.scatter(2, holes, torch.where(pair, movers, holes))
    kept = s["kept"]
    kept.copy_(torch.where(slot < keep, source, kept))
    out = s["weights_out"]
    out.copy_(torch.where(slot < keep, w.gather(2, source), out))
    b, h, i = hole.nonzero(as_tuple=True)
    j = source[b, h, i]
    to, of = s["pages"][b, i // PAGE].long(), s["pages"][b, j // PAGE].long()
    for_k, for_v = s["k_pool"][of, h, j % PAGE], s["v_pool"][of, h, j % PAGE]
    s["k_pool"][to, h, i % PAGE] = for_k
    s["v_pool"][to, h, i % PAGE] = for_v
    return s["k_pool"], s["v_pool"], kept, out


# ---------------------------------------------------------------- one pass

def run(s):
    case, op = s["case"], s["case"]["op"]
    if not own:
        return {"process": _process, "select": _select, "advance": _advance, "weights": _weights, "evict": _evict}[op](s)
    bsp = s["bsp"]
    if op == "process":
        bsp.process_logits(s["plan"], s["logits"], s["params"], s["out"], s["lse"])
        return s["out"], s["lse"]
    if op == "select":
        bsp.beam_select(s["plan"], s["logits"], s["lse"], s["cum"], s["scores"], s["parents"], s["tokens"],
                        s["select_ws"], mask=s["mask"], mask_index=s["mask_index"])
        return s["scores"], s["parents"], s["tokens"]
    if op == "advance":
        bsp.beam_advance(s["plan"], s["parents"], s["new"], s["indirection"], s["indirection_out"], s["tokens"],
                         s["tokens_out"])
        return s["indirection_out"], s["tokens_out"]
    if op == "weights":
        bsp.key_weights(s["plan"], s["q"], s["k_pool"], s["lse"], s["scale"], s["weights"], window=case["window"])
        return s["weights"]
    bsp.evict_prefix(s["plan"], s["weights"], s["keep"], case["sinks"], case["recent"], s["k_pool"], s["v_pool"],
                     s["kept"], weights_out=s["weights_out"])
    return s["k_pool"], s["v_pool"], s["kept"], s["weights_out"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    size = {"bf16": 2, "fp16": 2, "fp32": 4}[case.get("dtype", "bf16")]
    batch = case["batch"]
    if case["op"] in ("process", "select"):
        rows, vocab = batch * case["beam"], case["vocab"]
        # a row with a grammar state has only its allowed logits read (all sectors of them, at 3%: a third of
        # the 16-bit row, a fifth of the 32-bit one); one state index in mask_rows + 1 is none
        n = case["mask_rows"]
        read = rows * vocab * size
        if n:
            per = 32 // size
            read = read * (1 + n * (1 - 0.97 ** per)) / (n + 1)
        states = n * ((vocab + 31) // 32) * 4
        if case["op"] == "process":
            lists = 4 * (batch * case["prompt"] + rows * case["tokens"]) + 8 * batch * case["bias"]
            return {"bytes": int(read + states + rows * vocab * size + lists + 4 * rows), "flops": int(4 * read / size)}
        return {"bytes": int(read + states + 8 * rows + 12 * batch * case["num"]), "flops": int(2 * read / size)}
    if case["op"] == "advance":
        n = batch * case["beam"]
        return {"bytes": 4 * n * (4 * case["tail"] + 4), "flops": n}
    mean = (case["lo"] + case["hi"]) / 2
    keys = batch * (mean + case.get("cached", 0))
    if case["op"] == "weights":
        rows = batch * (min(case["window"], mean) if case["kind"] == "prefill" else case["beam"])
        pairs = rows / batch * keys * case["q_heads"]
        read = keys * case["kv_heads"] * case["dim"] * 2 + rows * case["q_heads"] * (case["dim"] * 2 + 4)
        return {"bytes": int(read + 4 * keys * case["kv_heads"]), "flops": int(pairs * (2 * case["dim"] + 3))}
    # evict: the weights once; per kept row its slot and weight; a row moves when it is kept (keep / keys of
    # them are) and stands behind the first keep
    keep = min(case["keep"], mean)
    fixed = min(case["sinks"] + case["recent"], keep)
    share = (keep - fixed) / max(1.0, mean - fixed)
    behind = mean - keep
    moved = share * max(0.0, behind - case["recent"]) + min(case["recent"], behind)
    per = case["kv_heads"] * batch
    return {"bytes": int(per * (4 * mean + 8 * keep + moved * 4 * case["dim"] * 2)), "flops": int(per * mean)}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, batch = case["op"], case["batch"]
    if op == "process":
        beam, vocab, dt = case["beam"], case["vocab"], s["logits"].dtype
        if batch * beam > 3000:
            return None
        outs, lses = [], []
        for r in range(batch * beam):
            b = r // beam
            x = s["logits"][r].double()
            made = s["tokens"][r, :int(s["tokens_len"][r])].long() if s["tokens"] is not None else None
            if s["repetition"] is not None:
                ids = [made] if made is not None else []
                if s["prompt_tokens"] is not None:
                    ids.append(s["prompt_tokens"][b, :int(s["prompt_tokens_len"][b])].long())
                if ids:
                    ids = torch.unique(torch.cat(ids))
                    p, old = s["repetition"][b].double(), x[ids]
                    x[ids] = torch.where(old > 0, old / p, old * p)
            if s["frequency"] is not None and made is not None:
                ids, count = torch.unique(made, return_counts=True)
                x[ids] -= s["frequency"][b].double() * count + s["presence"][b].double()
            if s["bias_tokens"] is not None:
                ids, values = s["bias_tokens"][b].cpu().numpy(), s["bias_values"][b].double().cpu().numpy()
                ids, first = np.unique(ids, return_index=True)
                x[torch.from_numpy(ids).long().cuda()] += torch.from_numpy(values[first]).cuda()
            if s["temperature"] is not None:
                x = x / s["temperature"][b].double()
            if s["mask"] is not None and int(s["mask_index"][r]) >= 0:
                words = s["mask"][int(s["mask_index"][r])]
                bit = (words[:, None] >> torch.arange(32, device="cuda")[None]) & 1
                x[bit.reshape(-1)[:vocab] == 0] = -math.inf
            if batch * beam * vocab <= 40_000_000:
                outs.append(x)
            lses.append(torch.logsumexp(x.to(dt).double(), 0))
        return (torch.stack(outs) if outs else None), torch.stack(lses)
    if op == "select":
        beam, vocab = case["beam"], case["vocab"]
        best = []
        for b in range(batch):
            rows = slice(b * beam, (b + 1) * beam)
            x = s["logits"][rows].double() - s["lse"][rows].double()[:, None] + s["cum"][b].double()[:, None]
            if s["mask"] is not None:
                for w in range(beam):
                    state = int(s["mask_index"][b * beam + w])
                    if state >= 0:
                        bit = (s["mask"][state][:, None] >> torch.arange(32, device="cuda")[None]) & 1
                        x[w, bit.reshape(-1)[:vocab] == 0] = -math.inf
            best.append(torch.topk(x.reshape(-1), case["num"]).values)
        return torch.stack(best), None, None
    if op == "weights":
        out = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
        if int(s["limit"].shape[0]) * s["limit"].shape[1] * case["q_heads"] * out.shape[2] * case["dim"] > 4e12:
            return None
        for b in range(batch):
            n = int(s["keys"][b])
            pages = s["pages"][b, :-(-n // PAGE)].long()
            k = s["k_pool"][pages].double().permute(1, 0, 2, 3).reshape(case["kv_heads"], -1, case["dim"])[:, :n]
            limit = s["limit"][b]
            rows = s["rows"][b][limit > 0]
            limit = limit[limit > 0]
            group = case["q_heads"] // case["kv_heads"]
            for h in range(case["q_heads"]):
                p = torch.exp(s["q"][rows, h].double() @ k[h // group].T * s["scale"] - s["lse"][rows, h].double()[:, None])
                p = torch.where(torch.arange(n, device="cuda")[None] < limit[:, None], p, 0.0)
                out[b, h // group, :n] += p.sum(0)
        return out
    return None
