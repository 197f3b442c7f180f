"""Cases for four serving operators over the paged cache: attention of drafted
tokens that form a tree, and attention with a sliding window and a few first
tokens that stay visible (decode over the bf16 and over the 8-bit cache, and
prefill of variable-length rows).

``own = False`` computes each operator in its plain form from elementary torch
operations in 32 bits; ``own = True`` makes the calls of this package. Shapes are
the ones this repository serves (32 query heads over 8 KV heads of 128, the
tensor-parallel shard of 8 over 1, pages of 16 tokens, rows up to 32768 keys)
and smaller and odd ones around them.

Tree: row b's drafted tokens are its last positions in the cache, and all of them
see every key in front of them; token i sees drafted token j where bit j of its
mask is set (its ancestors and itself). Window: the query at position p sees key
j <= p where j > p - window or j < sinks. Pages that hold no visible key have no
entry in the block table: a program frees them.
"""
import math

import torch

own = False

PAGE = 16
E_MIN, E_MAX = -117, 119  # exponents of the 8-bit cache's scales


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # One request verifies 8 drafts behind a short context, odd group of 5
        # query heads: launch latency.
        {"name": "tree_row_500x8", "op": "tree", "B": 1, "ctx": 500, "draft": 8, "h_kv": 8, "g": 5, "d": 128,
         "ragged": False},
        # One request with a long context and a tree of 26 drafts: the key axis
        # has to fill the machine.
        {"name": "tree_row_32768x26", "op": "tree", "B": 1, "ctx": 32768, "draft": 26, "h_kv": 8, "g": 4, "d": 128,
         "ragged": False},
        # A serving batch that speculates: rows of 1 to 16384 keys, 1 to 24 drafts.
        {"name": "tree_batch_64", "op": "tree", "B": 64, "ctx": 16384, "draft": 24, "h_kv": 8, "g": 4, "d": 128,
         "ragged": True},
        # Wide trees on a tensor-parallel shard: 61 drafts, 8 query heads over 1, heads of 64.
        {"name": "tree_wide_shard", "op": "tree", "B": 24, "ctx": 8192, "draft": 61, "h_kv": 1, "g": 8, "d": 64,
         "ragged": True},
        # One row inside a long window: launch latency.
        {"name": "decode_window_row", "op": "decode", "B": 1, "len": 20000, "window": 1024, "sinks": 4, "h_kv": 8,
         "g": 4, "d": 128, "cache": "bf16", "ragged": False},
        # A serving batch with a window of 4096: rows shorter and longer than it.
        {"name": "decode_window_batch", "op": "decode", "B": 66, "len": 16384, "window": 4096, "sinks": 4, "h_kv": 8,
         "g": 4, "d": 128, "cache": "bf16", "ragged": True},
        # One row of the 8-bit cache, a window that starts and ends inside pages.
        {"name": "decode_window_e4m3_row", "op": "decode", "B": 1, "len": 5003, "window": 777, "sinks": 1, "h_kv": 8,
         "g": 5, "d": 128, "cache": "e4m3", "ragged": False},
        # Many rows of the 8-bit cache, odd window, sinks that fill more than a page.
        {"name": "decode_window_e4m3_batch", "op": "decode", "B": 200, "len": 16384, "window": 2001, "sinks": 18,
         "h_kv": 8, "g": 4, "d": 128, "cache": "e4m3", "ragged": True},
        # Tails of short prompts, heads of 64 without sharing, a window below a page of queries.
        {"name": "prefill_window_short", "op": "prefill", "B": 5, "new": 333, "old": 100, "window": 100, "sinks": 5,
         "h_kv": 8, "g": 1, "d": 64, "ragged": True},
        # A whole prompt of 8192 tokens, window of 1024 and 4 sinks.
        {"name": "prefill_window_8192", "op": "prefill", "B": 1, "new": 8192, "old": 0, "window": 1024, "sinks": 4,
         "h_kv": 8, "g": 4, "d": 128, "ragged": False},
        # Chunks of 8 prompts over long contexts, no sinks.
        {"name": "prefill_window_chunks", "op": "prefill", "B": 8, "new": 1024, "old": 7168, "window": 4096,
         "sinks": 0, "h_kv": 8, "g": 4, "d": 128, "ragged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "decode", "decode", "prefill"])
    d = rng.choice([64, 128, 128])
    ragged = rng.random() < 0.7
    h_kv, g = rng.choice([1, 2, 5, 8]), rng.randint(1, 8)
    if op == "tree":
        B, draft = _log(rng, 1, 64), _log(rng, 1, 100)
        most = int(8e8 / (B * draft * h_kv * g))
        return {"op": op, "B": B, "ctx": _log(rng, 1, min(32768, 1000000 // B, most)), "draft": draft,
                "h_kv": h_kv, "g": g, "d": d, "ragged": ragged}
    sinks = rng.choice([0, 1, 4, 16, 33])
    if op == "decode":
        B = _log(rng, 1, 200)
        return {"op": op, "B": B, "len": _log(rng, 1, 32768), "window": _log(rng, 1, min(8192, 400000 // B)),
                "sinks": sinks, "h_kv": h_kv, "g": g, "d": d, "cache": rng.choice(["bf16", "e4m3"]),
                "ragged": ragged}
    B = _log(rng, 1, 16)
    new = _log(rng, 1, 8192 // B)
    old = rng.choice([0, _log(rng, 1, 8192 - new)])
    return {"op": op, "B": B, "new": new, "old": old, "window": _log(rng, 1, 8192), "sinks": sinks, "h_kv": h_kv,
            "g": rng.choice([1, 2, 4, 8] if h_kv < 8 else [1, 2, 4]), "d": d, "ragged": ragged}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(case, seed):
    """Keys of each row and query tokens of each row: on the host, from the case
    alone, so that every seed does the same work in another order."""
    g = torch.Generator()
    g.manual_seed(12345)
    B = case["B"]

    def up_to(n, least):
        full = torch.full((B,), n)
        return torch.randint(least, n + 1, (B,), generator=g) if case["ragged"] else full

    if case["op"] == "tree":
        new, old = up_to(case["draft"], 1), up_to(case["ctx"], 1)
    elif case["op"] == "decode":
        new, old = torch.ones(B, dtype=torch.int64), up_to(case["len"], 1) - 1
    else:
        new, old = up_to(case["new"], 1), up_to(case["old"], 0)
    order = torch.randperm(B, generator=torch.Generator().manual_seed(int(seed)))
    return (old + new)[order], new[order]


def _table(case, lens, new, seed):
    """Block table over a shuffled pool; -1 for pages without a visible key."""
    pages = torch.arange(max(1, int((lens.max() + PAGE - 1) // PAGE)))[None, :]
    live = pages * PAGE < lens[:, None]
    if case["op"] != "tree":
        first = lens - new + 1 - case["window"]  # first key of the first query's window
        live &= ((pages + 1) * PAGE > first[:, None]) | (pages * PAGE < case["sinks"])
    n = int(live.sum())
    table = torch.full(live.shape, -1, dtype=torch.int32)
    table[live] = torch.randperm(n, generator=torch.Generator().manual_seed(int(seed) + 1)).to(torch.int32)
    return table.cuda(), n


def _tree_bits(new, seed):
    """Masks of random trees, packed: draft i hangs below an earlier one or
    below the context (chains and wide levels both occur)."""
    rng = torch.Generator().manual_seed(int(seed) + 2)
    words = (int(new.max()) + 31) // 32
    out = []
    for n in new.tolist():
        u = torch.rand(n, generator=rng).tolist()
        seen = []
        for i in range(n):
            parent = max(-1, min(i - 1, int(i * math.sqrt(u[i])) - 1 + (u[i] > 0.9)))
            seen.append((seen[parent] if parent >= 0 else 0) | (1 << i))
            out.append([(seen[i] >> (32 * w)) & 0xffffffff for w in range(words)])
    bits = torch.tensor(out, dtype=torch.int64)
    return torch.where(bits >= 2 ** 31, bits - 2 ** 32, bits).to(torch.int32).cuda()


def _rows(g, shape):
    """Keys as they meet a cache: N(0,1) with a few strong channels and token
    norms that vary."""
    x = torch.randn(shape, generator=g, device="cuda")
    x[..., 1] *= 8.0
    x[..., shape[-1] // 2] *= 5.0
    return x * torch.exp2(2 * torch.rand(shape[:-1] + (1,), generator=g, device="cuda") - 1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    op, h_kv, d = case["op"], case["h_kv"], case["d"]
    h = h_kv * case["g"]
    lens, new = _lengths(case, seed)
    table, pages = _table(case, lens, new, seed)
    total = int(new.sum())
    s = {"op": op, "scale": 1.0 / math.sqrt(d), "table": table, "lens": lens.to(torch.int32).cuda(),
         "cu": torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)]).to(torch.int32).cuda(),
         "max_q": int(new.max()), "window": case.get("window"), "sinks": case.get("sinks"), "h_kv": h_kv,
         "q": torch.randn((total, h, d), generator=g, device="cuda").to(torch.bfloat16)}
    if case.get("cache") == "e4m3":
        shape = (pages, h_kv, PAGE, d)
        s["kc"], s["ks"] = _quantise(_rows(g, shape).to(torch.bfloat16))
        s["vc"], s["vs"] = _quantise(torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16))
    else:
        shape = (pages, PAGE, h_kv, d)
        s["kc"] = _rows(g, shape).to(torch.bfloat16)
        s["vc"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    if op == "tree":
        s["mask"] = _tree_bits(new, seed)
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((total, h), device="cuda")
    return s


def _quantise(x):
    """Codes and biased exponents of the rows of x."""
    x = x.float()
    m, e = torch.frexp(x.abs().amax(-1))  # a = m * 2^e, m in [0.5, 1): 448 = 0.875 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp(E_MIN, E_MAX)
    e = torch.where(m == 0, torch.full_like(e, E_MIN), e)
    codes = (x * _power(127 - e)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _power(biased):
    """2^(biased - 127) as a column of 32-bit numbers, by its bits."""
    return torch.bitwise_left_shift(biased.to(torch.int32), 23).view(torch.float32)[..., None]


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _gather(s, cache, scales, pos):
    """Rows of a cache at key positions pos [B, n], in 32 bits: [B, h_kv, n, d].
    Positions without a page read some page's rows."""
    b = torch.arange(pos.shape[0], device="cuda")[:, None]
    at = pos.clamp(min=0)
    page = s["table"][b, (at // PAGE).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0)
    if scales is None:
        return cache[page, at % PAGE].float().transpose(1, 2)
    codes = cache.view(torch.uint8)[page, :, at % PAGE].view(cache.dtype).float()
    return (codes * _power(scales[page, :, at % PAGE])).transpose(1, 2)


def _attend(q, k, v, seen):
    """q [B, h_kv, r, d], keys and values [B, h_kv, n, d], seen broadcastable to
    [B, h_kv, r, n]: outputs and log-sum-exps."""
    scores = torch.matmul(q, k.transpose(2, 3)).masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l == 0, torch.ones_like(l), l)
    lse = torch.where(l == 0, torch.full_like(l, -math.inf), m + torch.log(l))
    return o, lse[..., 0]


def _run_plain(s):
    total, h, d = s["q"].shape
    h_kv = s["h_kv"]
    lens = s["lens"].long()
    if s["op"] == "decode":
        window, sinks = s["window"], s["sinks"]
        first = torch.arange(sinks, device="cuda")[None, :].expand(total, sinks)
        last = lens[:, None] - window + torch.arange(window, device="cuda")[None, :]
        pos = torch.cat([first, last], 1)
        seen = torch.cat([first < lens[:, None], last >= sinks], 1)[:, None, None, :]
        q = s["q"].float().reshape(total, h_kv, -1, d) * s["scale"]
        o, lse = _attend(q, _gather(s, s["kc"], s.get("ks"), pos), _gather(s, s["vc"], s.get("vs"), pos), seen)
        return {"o": o.reshape(total, h, d).to(torch.bfloat16), "lse": lse.reshape(total, h)}
    # Rows side by side, each as long as the longest.
    B, n_q, n_k = len(lens), s["max_q"], s["table"].shape[1] * PAGE
    cu = s["cu"].long()
    i = torch.arange(n_q, device="cuda")[None, :]
    new = (cu[1:] - cu[:-1])[:, None]
    tok = torch.where(i < new, cu[:-1, None] + i, total)  # behind the last: a row that is dropped
    j = torch.arange(n_k, device="cuda")[None, :]
    pos = j.expand(B, n_k)
    q_pos = (lens[:, None] - new + i)[:, :, None]  # [B, n_q, 1]
    key = pos[:, None, :]
    if s["op"] == "tree":
        at = key - (lens[:, None] - new)[:, :, None]  # the draft that a key is
        words = s["mask"].shape[1]
        bits = s["mask"][tok.clamp(max=total - 1)]
        word = torch.gather(bits, 2, (at // 32).clamp(0, words - 1).expand(B, n_q, n_k))
        drawn = torch.bitwise_right_shift(word, (at % 32).to(torch.int32)) & 1
        seen = (at < 0) | ((drawn != 0) & (at < new[:, :, None]))
        del word, drawn
    else:
        seen = (key <= q_pos) & ((key > q_pos - s["window"]) | (key < s["sinks"]))
    g = h // h_kv
    o = torch.empty((total + 1, h, d), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((total + 1, h), device="cuda")
    q = torch.cat([s["q"], s["q"][:1]]).float()[tok] * s["scale"]  # [B, n_q, h, d]
    for kv in range(h_kv):
        part = slice(kv * g, kv * g + g)
        k = _gather(s, s["kc"][:, :, kv:kv + 1], None, pos)
        v = _gather(s, s["vc"][:, :, kv:kv + 1], None, pos)
        oh, lh = _attend(q[:, :, part].transpose(1, 2), k, v, seen[:, None])
        o[tok, part] = oh.transpose(1, 2).to(torch.bfloat16)
        lse[tok, part] = lh.transpose(1, 2)
    return {"o": o[:total], "lse": lse[:total]}


def _workspace(s, bytes_of):
    if "ws" not in s:  # a program keeps its scratch memory from step to step
        s["ws"] = torch.empty(bytes_of(), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _run_own(s):
    import online_softmax_attn_gb300 as attn

    total, h, d = s["q"].shape
    h_kv, B = s["h_kv"], len(s["lens"])
    if s["op"] == "tree":
        ws = _workspace(s, lambda: attn.attn_decode_tree_workspace_bytes(B, h, h_kv, d))
        o, lse = attn.attn_decode_paged_tree(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], s["mask"],
                                             s["max_q"], s["scale"], workspace=ws, o=s["o"], lse=s["lse"])
    elif s["op"] == "prefill":
        ws = _workspace(s, lambda: attn.attn_prefill_window_workspace_bytes(B, s["table"].shape[1], h_kv, d))
        o, lse = attn.attn_prefill_paged_window(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"],
                                                s["window"], s["sinks"], s["max_q"], s["scale"], workspace=ws,
                                                o=s["o"], lse=s["lse"])
    elif "ks" in s:
        ws = _workspace(s, lambda: attn.attn_decode_window_workspace_bytes(B, h, h_kv, d))
        o, lse = attn.attn_decode_paged_window_e4m3(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"],
                                                    s["lens"], s["window"], s["sinks"], s["scale"], workspace=ws,
                                                    o=s["o"], lse=s["lse"])
    else:
        ws = _workspace(s, lambda: attn.attn_decode_window_workspace_bytes(B, h, h_kv, d))
        o, lse = attn.attn_decode_paged_window(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["window"],
                                               s["sinks"], s["scale"], workspace=ws, o=s["o"], lse=s["lse"])
    return {"o": o, "lse": lse}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# Work and exact values
# ---------------------------------------------------------------------------
def work(case):
    lens, new = _lengths(case, 0)
    h_kv, d = case["h_kv"], case["d"]
    h, total = h_kv * case["g"], int(new.sum())
    if case["op"] == "tree":
        keys = int(lens.sum())
        pairs = int(((lens - new) * new).sum()) + int((new * (new + 1) // 2).sum()) // 2  # about half of a triangle
    else:
        window, sinks = case["window"], case["sinks"]
        keys = pairs = 0
        for n, m in zip(lens.tolist(), new.tolist()):
            first = max(0, n - m + 1 - window)  # first key of the first query's window
            keys += n - first + min(first, sinks)
            p = torch.arange(n - m, n)
            lo = (p + 1 - window).clamp(min=0)
            pairs += int((p + 1 - lo + lo.clamp(max=sinks)).sum())
    row = d + 1 if case.get("cache") == "e4m3" else 2 * d
    return {"bytes": 2 * keys * h_kv * row + total * h * (4 * d + 4), "flops": 4 * pairs * h * d}


def _power64(e):
    """2^e in 64 bits, by its bits (a library's power may be off in the last one)."""
    return torch.bitwise_left_shift(e.to(torch.int64) + 1023, 52).view(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    total, h, d = s["q"].shape
    h_kv, g = case["h_kv"], case["g"]
    o = torch.zeros((total, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((total, h), -math.inf, dtype=torch.float64, device="cuda")
    lens, cu = s["lens"].tolist(), s["cu"].tolist()

    def values(cache, scales, b, keys):
        """Row b's keys in 64 bits, [h_kv, n, d]."""
        pages, slots = s["table"][b].long()[keys // PAGE], keys % PAGE
        if scales is None:
            return cache[pages, slots].double().transpose(0, 1)
        x = cache.view(torch.uint8)[pages, :, slots].view(cache.dtype).double()
        return (x * _power64(scales[pages, :, slots].long() - 127)[..., None]).transpose(0, 1)

    for b, n in enumerate(lens):
        m = cu[b + 1] - cu[b]
        for i0 in range(0, m, 256):  # queries i0 .. i1 - 1 and the keys that any of them sees
            i1 = min(m, i0 + 256)
            p = torch.arange(n - m + i0, n - m + i1, device="cuda")[:, None]
            if case["op"] == "tree":
                keys = torch.arange(n, device="cuda")
                ctx = n - m
                seen = torch.ones((i1 - i0, n), dtype=torch.bool, device="cuda")
                words = s["mask"][cu[b] + i0:cu[b] + i1].long() & 0xffffffff
                for j in range(m):
                    seen[:, ctx + j] = (words[:, j // 32] >> (j % 32)) % 2 == 1
            else:
                first = max(0, n - m + i0 + 1 - case["window"])
                keys = torch.cat([torch.arange(min(first, case["sinks"]), device="cuda"),
                                  torch.arange(first, n - m + i1, device="cuda")])
                seen = (keys <= p) & ((p - keys < case["window"]) | (keys < case["sinks"]))
            k, v = values(s["kc"], s.get("ks"), b, keys), values(s["vc"], s.get("vs"), b, keys)
            q = s["q"][cu[b] + i0:cu[b] + i1].double().view(-1, h_kv, g, d)
            scores = torch.einsum("ihgd,hnd->hgin", q, k) / math.sqrt(d)
            scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
            top = scores.amax(-1, keepdim=True)
            w = torch.exp(scores - torch.where(torch.isinf(top), torch.zeros_like(top), top))
            l = w.sum(-1)
            out = torch.einsum("hgin,hnd->ihgd", w, v) / torch.where(l == 0, torch.ones_like(l), l).permute(2, 0, 1)[..., None]
            o[cu[b] + i0:cu[b] + i1] = out.reshape(-1, h, d)
            full = torch.where(l == 0, torch.full_like(l, -math.inf), top[..., 0] + torch.log(l))
            lse[cu[b] + i0:cu[b] + i1] = full.permute(2, 0, 1).reshape(-1, h)
    return {"o": o, "lse": lse}
