"""The serving operators around the paged latent cache, case by case.

Four operators of multi-head latent attention at DeepSeek-V2's widths (a
512-number latent and a 64-number RoPE key per cached token, query heads of
128 + 64 numbers, pages of 64 tokens), in the order a serving loop runs them:

  norm     RMS norm of every query head, of the latent and of the shared RoPE
           key, the position rotation, and the append of the new rows
           (mla_norm_rope)
  chunk    attention of ragged chunks of new tokens over the paged cache,
           with the absorbed query (mla_chunk_attention)
  weights  attention weight that every cached token received from a chunk's
           queries, added to what it has gathered so far (mla_attn_weights)
  evict    eviction of the cached tokens with the least gathered weight,
           survivors moved into their slots (mla_cache_evict)

``run`` computes them in elementary torch operations in 32 bits, or, where
``own`` is true, through the library.  ``exact`` computes them in 64 bits,
sequence by sequence.
"""

import math
import random

import torch

own = False

DN, DR, DC, PAGE = 128, 64, 512, 64      # head width without RoPE, RoPE width, latent, page
DQK, D = DN + DR, DC + DR
SCALE = DQK ** -0.5
BASE = 10000.0
EPS = 1e-6
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one decode step of one sequence: the smallest call of the loop
        dict(name="norm_one_token", op="norm", T=1, H=128, dtype="bf16", decode=True),
        # one decode step of a batch of 128 sequences (the batch128 workload)
        dict(name="norm_batch128", op="norm", T=128, H=128, dtype="bf16", decode=True),
        # a 4096-token prefill chunk: queries stay in their rows
        dict(name="norm_prefill_chunk", op="norm", T=4096, H=128, dtype="bf16", decode=False),
        # four speculative tokens of each of 16 sequences are verified at once
        dict(name="chunk_speculative", op="chunk", B=16, q_lo=4, q_hi=4, len_lo=4096,
             len_hi=4096, H=128),
        # prompt tails and decode tokens of a mixed batch, 16 heads per GPU
        dict(name="chunk_mixed_16_heads", op="chunk", B=13, q_lo=1, q_hi=129, len_lo=200,
             len_hi=9000, H=16),
        # prefill chunks of four sequences over long contexts
        dict(name="chunk_prefill", op="chunk", B=4, q_lo=256, q_hi=256, len_lo=16384,
             len_hi=16384, H=128),
        # the dsv2 workload's decode step: 16 sequences of 4096 tokens
        dict(name="weights_decode", op="weights", B=16, q_lo=1, q_hi=1, len_lo=4096, len_hi=4096,
             H=128),
        # ragged decode: 64 sequences with lengths over more than two decades
        dict(name="weights_ragged", op="weights", B=64, q_lo=1, q_hi=1, len_lo=129, len_hi=65537,
             H=128),
        # the last 32 queries of four prompts judge the prompt's tokens
        dict(name="weights_window", op="weights", B=4, q_lo=32, q_hi=32, len_lo=8001, len_hi=8192,
             H=128),
        # a decode step over a full budget: every sequence loses one token
        dict(name="evict_one", op="evict", B=16, len_lo=4097, len_hi=4097, drop=1, keep_pct=0,
             dtype="bf16", placed=True),
        # after ragged prompts: every sequence is cut to 30 % of its length
        dict(name="evict_ragged", op="evict", B=64, len_lo=129, len_hi=32769, drop=0, keep_pct=30,
             dtype="bf16", placed=False),
        # four contexts of 131072 tokens are halved
        dict(name="evict_long", op="evict", B=4, len_lo=131072, len_hi=131072, drop=0,
             keep_pct=50, dtype="bf16", placed=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(("norm", "chunk", "weights", "evict"))
    if op == "norm":
        H = rng.choice((8, 16, 32, 64, 128))
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        decode = rng.random() < 0.5
        T = _log_int(rng, 1, 512 if decode else 2048 if dtype == "f32" else 4096)
        return dict(op=op, T=T, H=H, dtype=dtype, decode=decode)
    if op == "evict":
        while True:
            B, hi = _log_int(rng, 1, 64), _log_int(rng, 128, 131072)
            dtype = rng.choice(("bf16", "bf16", "f32"))
            if B * hi * (2 if dtype == "f32" else 1) <= 4 * 131072:
                break
        some = rng.random() < 0.4
        return dict(op=op, B=B, len_lo=_log_int(rng, 96, hi), len_hi=hi,
                    drop=_log_int(rng, 1, 64) if some else 0,
                    keep_pct=0 if some else rng.randint(20, 95),
                    dtype=dtype, placed=rng.random() < 0.5)
    while True:
        B, H, hi = _log_int(rng, 1, 64), rng.choice((8, 16, 32, 64, 128)), _log_int(rng, 64, 65536)
        q_hi = _log_int(rng, 1, 512) if op == "chunk" else _log_int(rng, 1, 64)
        cells = B * q_hi * H * hi          # scores of the padded batch
        if (q_hi <= hi and B * hi <= 8 * 65536 and
                cells <= (4 * 256 * 128 * 16384 if op == "chunk" else 64 * 128 * 65536)):
            break
    q_lo = _log_int(rng, 1, q_hi)
    return dict(op=op, B=B, q_lo=q_lo, q_hi=q_hi, len_lo=_log_int(rng, max(q_hi, hi // 16), hi),
                len_hi=hi, H=H)


def _lengths(case):
    """Cached tokens (the chunk's among them) and chunk tokens of every sequence: the case's own,
    whatever the seed, spread over the logarithm of the range, its ends included."""
    r = random.Random("%d %d %d" % (case["B"], case["len_lo"], case["len_hi"]))
    n = case["B"]
    lens = [_log_int(r, case["len_lo"], case["len_hi"]) for _ in range(n)]
    lens[0] = case["len_hi"]
    lens[-1] = case["len_lo"] if n > 1 else lens[-1]
    if "q_lo" not in case:
        return lens, None
    qs = [_log_int(r, case["q_lo"], case["q_hi"]) for _ in range(n)]
    qs[-1] = case["q_hi"]
    return lens, [min(a, b) for a, b in zip(qs, lens)]


def _budgets(case, lens):
    if case["drop"]:
        return [max(L - case["drop"], 1) for L in lens]
    return [max(L * case["keep_pct"] // 100, 1) for L in lens]


SINK, RECENT = 4, 32      # tokens at either end of a context that are never evicted


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _type(case):
    return torch.float32 if case.get("dtype") == "f32" else torch.bfloat16


def _paged(g, lens, dtype, unused):
    """A pool of 64-token pages in random order: N(0, 1) rows for the cached tokens, `unused` in
    the slots that hold none, and the page table (-1 where a sequence has no page)."""
    pages = [-(-L // PAGE) for L in lens]
    n_pages, max_pages = sum(pages) + 1, max(pages)
    perm = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    count = torch.tensor(pages, device=DEV)
    first = torch.cumsum(count, 0) - count
    col = torch.arange(max_pages, device=DEV)
    at = (first[:, None] + col).clamp_(max=n_pages - 1)
    table = torch.where(col < count[:, None], perm[at], -1).to(torch.int32).contiguous()
    pool = torch.empty((n_pages, PAGE, D), device=DEV, dtype=dtype)
    pool.normal_(generator=g)
    if unused is not None:
        used = torch.zeros((n_pages, PAGE), dtype=torch.bool, device=DEV)
        ends = torch.tensor(lens, device=DEV)
        slot = torch.arange(max_pages * PAGE, device=DEV)
        page = table[:, slot // PAGE].long()
        live = slot < ends[:, None]
        used[page[live], (slot % PAGE).expand_as(page)[live]] = True
        pool[~used] = unused
    return pool, table


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case=dict(case))
    dt = _type(case)
    i32 = dict(dtype=torch.int32, device=DEV)
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        y = torch.empty((T, H * DQK + D), device=DEV, dtype=dt)
        y.normal_(generator=g)
        # the new tokens of max(1, T // 64) sequences, one after another behind random contexts
        n = max(1, T // 64) if not case["decode"] else T
        per = -(-T // n)
        lens = [per] * n
        pool, table = _paged(g, lens, dt, 0.0)
        tok = torch.arange(T, device=DEV)
        start = torch.randint(0, 131072 - per, (n,), generator=g, device=DEV)
        weight = lambda k: (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(dt)  # noqa: E731
        s.update(y=y, pool=pool, table=table, batch=(tok // per).to(torch.int32),
                 slot=(tok % per).to(torch.int32),
                 pos=(start[tok // per] + tok % per).to(torch.int32), w_q=weight(DQK),
                 w_c=weight(DC), w_kr=weight(DR), q=torch.zeros((T, H, DQK), device=DEV, dtype=dt),
                 qbuf=torch.zeros((T, H, D), device=DEV, dtype=dt) if case["decode"] else None)
        return s
    lens, qs = _lengths(case)
    s["max_len"] = max(lens)
    s["lens"] = torch.tensor(lens, **i32)
    if case["op"] == "evict":
        s["pool"], s["table"] = _paged(g, lens, dt, 0.0)
        n, width = case["B"], s["max_len"]
        # gathered weights span decades; one token in twenty has gathered nothing
        w = torch.exp(2.5 * torch.randn((n, width), generator=g, device=DEV))
        w[torch.rand((n, width), generator=g, device=DEV) < 0.05] = 0.0
        s["w"] = w
        s["placed"] = None
        if case["placed"]:       # earlier evictions left slots out of the order of positions
            key = torch.rand((n, width), generator=g, device=DEV)
            key.masked_fill_(torch.arange(width, device=DEV) >= s["lens"][:, None], 2.0)
            s["placed"] = (torch.argsort(key, dim=1) * 3).to(torch.int32)
        budgets = _budgets(case, lens)
        s["budget"] = torch.tensor(budgets, **i32)
        s["most_out"] = max(1, max(L - k for L, k in zip(lens, budgets)))
        s["new_w"], s["new_len"] = torch.zeros_like(w), torch.zeros(n, **i32)
        s["new_placed"] = torch.zeros((n, width), **i32)
        return s
    s["pool"], s["table"] = _paged(g, lens, dt, float("nan"))
    total, H = sum(qs), case["H"]
    s["total"], s["max_q"] = total, max(qs)
    s["cu"] = torch.tensor([0] + qs, **i32).cumsum(0).to(torch.int32)
    q = torch.empty((total, H, D), device=DEV, dtype=dt)
    s["qbuf"] = q.normal_(generator=g)
    if case["op"] == "chunk":
        s["o"] = torch.zeros((total, H, DC), device=DEV, dtype=dt)
        s["lse"] = torch.zeros((total, H), device=DEV)
    else:
        # what the attention of these queries returned: ln sum exp of L scores of variance
        # 576 / 192 is ln L + 1.5, give or take
        seq = torch.repeat_interleave(torch.arange(case["B"], device=DEV),
                                      torch.tensor(qs, device=DEV))
        s["lse"] = (torch.log(s["lens"].float())[seq][:, None] + 1.5 +
                    0.1 * torch.randn((total, H), generator=g, device=DEV))
        s["w"] = torch.exp(torch.randn((case["B"], s["max_len"]), generator=g, device=DEV))
        s["new_w"] = torch.zeros_like(s["w"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return OWN[op](s)
    return PLAIN[op](s)


def _rms(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _turn(x, pos):
    """Pairs (x_2k, x_2k+1) of the last axis turned by pos * BASE^(-2k/64); pos broadcasts over
    the axes between the first and the last."""
    k = torch.arange(0, DR, 2, device=x.device, dtype=torch.float64)
    a = (pos.double()[:, None] * BASE ** (-k / DR)).reshape(pos.shape[0], *[1] * (x.dim() - 2), -1)
    c, n = a.cos().float(), a.sin().float()
    x0, x1 = x[..., 0::2], x[..., 1::2]
    return torch.stack((x0 * c - x1 * n, x0 * n + x1 * c), -1).flatten(-2)


def _plain_norm(s):
    T, H = s["case"]["T"], s["case"]["H"]
    y = s["y"].float()
    q = _rms(y[:, :H * DQK].reshape(T, H, DQK), s["w_q"])
    q_rope = _turn(q[..., DN:], s["pos"])
    s["q"][..., :DN] = q[..., :DN].to(s["q"].dtype)
    if s["qbuf"] is None:
        s["q"][..., DN:] = q_rope.to(s["q"].dtype)
    else:
        s["qbuf"][..., DC:] = q_rope.to(s["q"].dtype)
    c = _rms(y[:, H * DQK:H * DQK + DC], s["w_c"])
    kr = _turn(_rms(y[:, H * DQK + DC:], s["w_kr"]), s["pos"])
    page = s["table"][s["batch"].long(), s["slot"].long() // PAGE].long()
    s["pool"][page, s["slot"].long() % PAGE] = torch.cat((c, kr), -1).to(s["pool"].dtype)
    return dict(q=s["q"], qbuf=s["qbuf"], pool=s["pool"])


def _scores(s):
    """Scaled scores [B, max_q, H, max_len] of the padded batch (-inf where a query does not see
    a token), the gathered rows [B, max_len, 576] and, for each query token, its place in the
    padded batch."""
    n, H, total, max_q, max_len = s["case"]["B"], s["case"]["H"], s["total"], s["max_q"], s["max_len"]
    t = torch.arange(max_len, device=DEV)
    lens = s["lens"].long()
    live = t < lens[:, None]
    page = s["table"].long()[:, t // PAGE].clamp_(min=0)
    kv = torch.where(live[..., None], s["pool"][page, t % PAGE], 0).float()
    cu = s["cu"].long()
    j = torch.arange(max_q, device=DEV)
    n_q = cu[1:] - cu[:-1]
    q = s["qbuf"][(cu[:-1, None] + j).clamp_(max=total - 1)].float()
    x = torch.matmul(q.reshape(n, max_q * H, D), kv.transpose(1, 2)).mul_(SCALE)
    x = x.view(n, max_q, H, max_len)
    seen = (t <= (lens - n_q)[:, None, None] + j[:, None]) & (j < n_q[:, None])[..., None]
    x.masked_fill_(~(seen & live[:, None])[:, :, None], -math.inf)
    tok = torch.arange(total, device=DEV)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    return x, kv, seq, tok - cu[seq]


def _plain_chunk(s):
    x, kv, seq, j = _scores(s)
    n, max_q, H, max_len = x.shape
    m = x.amax(-1, keepdim=True)
    m.masked_fill_(m == -math.inf, 0.0)
    p = x.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(n, max_q * H, max_len), kv[..., :DC]).view(n, max_q, H, DC)
    s["o"].copy_((o / z)[seq, j])
    s["lse"].copy_((m + z.log())[seq, j, :, 0])
    return dict(o=s["o"], lse=s["lse"])


def _plain_weights(s):
    x, _, seq, j = _scores(s)
    n, max_q, H, max_len = x.shape
    lse = torch.full((n, max_q, H), math.inf, device=DEV)
    lse[seq, j] = s["lse"]
    got = x.sub_(lse[..., None]).exp_().sum((1, 2))
    t = torch.arange(max_len, device=DEV)
    n_q = s["cu"][1:] - s["cu"][:-1]
    old = torch.where(t < (s["lens"] - n_q)[:, None], s["w"], 0)
    s["new_w"].copy_(torch.where(t < s["lens"][:, None], old + got, s["new_w"]))
    return s["new_w"]


def _plain_evict(s):
    n, width = s["w"].shape
    t = torch.arange(width, device=DEV)
    lens, budget = s["lens"].long()[:, None], s["budget"].long()[:, None]
    live = t < lens
    at = t.expand(n, width) if s["placed"] is None else s["placed"].long()
    end = torch.where(live, at, -1).amax(1, keepdim=True) + 1
    free = live & (at >= SINK) & (at < end - RECENT)
    order = torch.sort(torch.where(free, s["w"], math.inf), dim=1, stable=True).indices
    n_out = torch.minimum((lens - budget).clamp_(min=0), free.sum(1, keepdim=True))
    out = torch.zeros_like(live).scatter_(1, order, t < n_out) & free
    new_len = lens - n_out
    hole, mover = out & (t < new_len), live & ~out & (t >= new_len)
    # the k-th mover goes to the k-th hole; what lies past the last of either is dropped in a
    # column of its own, and a sequence's spare pairs copy its first kept slot once more
    most = s["most_out"]
    slots = lambda m: torch.zeros((n, most + 1), dtype=torch.long, device=DEV).scatter_(  # noqa: E731
        1, torch.where(m, m.cumsum(1) - 1, most), t.expand(n, width))[:, :most]
    holes, movers = slots(hole), slots(mover)
    pair = torch.arange(most, device=DEV) < hole.sum(1, keepdim=True)
    keep = t < new_len
    src = t.repeat(n, 1).scatter_(1, torch.where(pair, holes, width - 1),
                                  torch.where(pair, movers, width - 1))
    to, frm = torch.where(pair, holes, 0), torch.where(pair, movers, src[:, :1])
    page = s["table"].long().clamp(min=0)
    row = lambda x: page.gather(1, x // PAGE) * PAGE + x % PAGE           # noqa: E731
    flat = s["pool"].view(-1, D)
    flat[row(to).view(-1)] = flat[row(frm).view(-1)]
    s["new_w"].copy_(torch.where(keep, s["w"].gather(1, src), s["new_w"]))
    s["new_placed"].copy_(torch.where(keep, at.gather(1, src), s["new_placed"]))
    s["new_len"].copy_(new_len[:, 0])
    return dict(pool=s["pool"], w=s["new_w"], placed=s["new_placed"], lens=s["new_len"])


PLAIN = dict(norm=_plain_norm, chunk=_plain_chunk, weights=_plain_weights, evict=_plain_evict)


# ---------------------------------------------------------------------------
# the same passes through the library
# ---------------------------------------------------------------------------
def _lib(s):
    """The binding and this layer's dims, which a program keeps."""
    if "lib" not in s:
        from mla_latent_kv_35_b200 import binding
        c = s["case"]
        dims = binding.MLADims(c.get("H", 128), DN, DC, DR, DN, 5120, PAGE, SCALE, BASE,
                               "f32" if c.get("dtype") == "f32" else "bf16")
        s["lib"] = (binding, dims)
    return s["lib"]


def _workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.empty(max(size(), 256), dtype=torch.uint8, device=DEV)
    return s["ws"]


def _own_norm(s):
    b, d = _lib(s)
    H = d.n_heads
    b.mla_norm_rope(d, s["y"], H * DQK + D, s["w_q"], s["w_c"], s["w_kr"], EPS, s["pos"],
                    s["batch"], s["slot"], s["table"], s["table"].shape[1], s["pool"],
                    s["pool"].shape[0], s["q"], H * DQK, s["qbuf"], None, 0, s["case"]["T"])
    return dict(q=s["q"], qbuf=s["qbuf"], pool=s["pool"])


def _own_chunk(s):
    b, d = _lib(s)
    n = s["case"]["B"]
    ws = _workspace(s, lambda: b.mla_chunk_attention_workspace_size(d, n, s["total"], s["max_q"]))
    b.mla_chunk_attention(d, s["qbuf"], s["cu"], s["total"], s["max_q"], s["pool"],
                          s["pool"].shape[0], s["table"], s["table"].shape[1], s["lens"], n, ws,
                          s["o"], s["lse"])
    return dict(o=s["o"], lse=s["lse"])


def _own_weights(s):
    b, d = _lib(s)
    b.mla_attn_weights(d, s["qbuf"], s["lse"], s["cu"], s["total"], s["max_q"], s["pool"],
                       s["pool"].shape[0], s["table"], s["table"].shape[1], s["lens"],
                       s["case"]["B"], s["w"], 1.0, s["new_w"], s["max_len"])
    return s["new_w"]


def _own_evict(s):
    b, d = _lib(s)
    n = s["case"]["B"]
    ws = _workspace(s, lambda: b.mla_cache_evict_workspace_size(d, n, s["max_len"]))
    b.mla_cache_evict(d, s["pool"], s["pool"].shape[0], False, s["table"], s["table"].shape[1],
                      s["lens"], n, s["w"], s["placed"], s["max_len"], s["budget"], SINK, RECENT,
                      s["new_w"], s["new_placed"], s["new_len"], ws)
    return dict(pool=s["pool"], w=s["new_w"], placed=s["new_placed"], lens=s["new_len"])


OWN = dict(norm=_own_norm, chunk=_own_chunk, weights=_own_weights, evict=_own_evict)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    e = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        row = H * DQK + D
        return dict(bytes=2 * T * row * e + (DQK + D) * e + 16 * T, flops=6 * T * row)
    lens, qs = _lengths(case)
    pages = 4 * sum(-(-L // PAGE) for L in lens)
    if case["op"] == "evict":
        out = [L - k for L, k in zip(lens, _budgets(case, lens))]
        # weights (and positions) read and those kept written, plus the rows that move: of n_out
        # evicted slots about n_out * kept / L lie before the new end, and as many rows come in
        moved = sum(o * (L - o) / L for o, L in zip(out, lens))
        kept = sum(lens) - sum(out)
        return dict(bytes=4 * sum(lens) * (2 if case["placed"] else 1) + 8 * kept +
                    2 * moved * D * e + pages, flops=4 * sum(lens))
    H = case["H"]
    # (query, token) pairs: query j of n sees L - n + j + 1 tokens
    seen = sum(n * L - n * (n - 1) // 2 for L, n in zip(lens, qs))
    if case["op"] == "chunk":
        return dict(bytes=sum(lens) * D * 2 + sum(qs) * H * (D * 2 + DC * 2 + 4) + pages,
                    flops=2 * seen * H * (D + DC))
    return dict(bytes=sum(lens) * (D * 2 + 8) + sum(qs) * H * (D * 2 + 4) + pages,
                flops=2 * seen * H * D)


# ---------------------------------------------------------------------------
# the same values in 64 bits, from the definitions
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)

    def norm():
        T, H = case["T"], case["H"]
        f8 = torch.float64
        pos = s["pos"].to(f8)
        freq = torch.tensor([BASE ** (-2.0 * k / DR) for k in range(DR // 2)], dtype=f8, device=DEV)
        turn = torch.polar(torch.ones((), dtype=f8, device=DEV).expand(T, DR // 2),
                           pos[:, None] * freq)                       # e^{i angle}

        def rotated(x):                                               # [T, 64] pairs as numbers
            z = torch.view_as_complex(x.reshape(T, DR // 2, 2).contiguous()) * turn
            return torch.view_as_real(z).reshape(T, DR)

        def normed(x, w):
            return x / torch.sqrt((x * x).sum(1, keepdim=True) / x.shape[1] + EPS) * w.to(f8)

        q = s["q"].to(f8)
        qbuf = None if s["qbuf"] is None else s["qbuf"].to(f8)
        for h in range(H):
            x = normed(s["y"][:, h * DQK:(h + 1) * DQK].to(f8), s["w_q"])
            q[:, h, :DN] = x[:, :DN]
            if qbuf is None:
                q[:, h, DN:] = rotated(x[:, DN:])
            else:
                qbuf[:, h, DC:] = rotated(x[:, DN:])
        pool = s["pool"].to(f8)
        table, batch, slot = s["table"].cpu(), s["batch"].cpu().long(), s["slot"].cpu().long()
        page = table[batch, slot // PAGE].long().to(DEV)
        o = H * DQK
        pool[page, (slot % PAGE).to(DEV), :DC] = normed(s["y"][:, o:o + DC].to(f8), s["w_c"])
        pool[page, (slot % PAGE).to(DEV), DC:] = rotated(normed(s["y"][:, o + DC:].to(f8), s["w_kr"]))
        return dict(q=q, qbuf=qbuf, pool=pool)

    def by_sequence():
        """(sequence, first query, queries, length, cache rows in 64 bits), one after another."""
        lens, qs = _lengths(case)
        q0 = 0
        for b, (L, n) in enumerate(zip(lens, qs)):
            pages = s["table"][b, :-(-L // PAGE)].long()
            yield b, q0, n, L, s["pool"][pages].reshape(-1, D)[:L].double()
            q0 += n

    def chunk():
        H = case["H"]
        o = torch.empty((s["total"], H, DC), dtype=torch.float64, device=DEV)
        lse = torch.empty((s["total"], H), dtype=torch.float64, device=DEV)
        for b, q0, n, L, kv in by_sequence():
            for j in range(n):
                see = L - n + j + 1
                x = s["qbuf"][q0 + j].double() @ kv[:see].T * SCALE
                lse[q0 + j] = torch.logsumexp(x, 1)
                o[q0 + j] = torch.softmax(x, 1) @ kv[:see, :DC]
        return dict(o=o, lse=lse)

    def weights():
        w = s["new_w"].double()
        for b, q0, n, L, kv in by_sequence():
            got = torch.zeros(L, dtype=torch.float64, device=DEV)
            got[:L - n] = s["w"][b, :L - n]
            for j in range(n):
                see = L - n + j + 1
                x = s["qbuf"][q0 + j].double() @ kv[:see].T * SCALE
                got[:see] += (x - s["lse"][q0 + j].double()[:, None]).exp().sum(0)
            w[b, :L] = got
        return w

    def evict():
        lens, _ = _lengths(case)
        keep = _budgets(case, lens)
        pool, w, lens_out = s["pool"].clone().double(), s["new_w"].double().cpu(), []
        placed = s["new_placed"].long().cpu()
        W = s["w"].double().cpu()
        at = None if s["placed"] is None else s["placed"].long().cpu()
        for b, L in enumerate(lens):
            where = torch.arange(L) if at is None else at[b, :L]
            end = int(where.max()) + 1
            free = [t for t, p in enumerate(where.tolist()) if SINK <= p < end - RECENT]
            n_out = min(max(L - keep[b], 0), len(free))
            row = W[b, :L].tolist()
            gone = set(sorted(free, key=lambda t: (row[t], t))[:n_out])
            new = L - n_out
            hole = [t for t in sorted(gone) if t < new]
            move = [t for t in range(new, L) if t not in gone]
            src = torch.arange(new)
            src[hole] = torch.tensor(move, dtype=torch.long)
            w[b, :new], placed[b, :new] = W[b, :L][src], where[src]
            pages = s["table"][b].long().cpu()
            h, m = torch.tensor(hole, dtype=torch.long), torch.tensor(move, dtype=torch.long)
            pool[pages[h // PAGE].to(DEV), (h % PAGE).to(DEV)] = \
                s["pool"][pages[m // PAGE].to(DEV), (m % PAGE).to(DEV)].double()
            lens_out.append(new)
        return dict(pool=pool, w=w, placed=placed, lens=torch.tensor(lens_out))

    return dict(norm=norm, chunk=chunk, weights=weights, evict=evict)[case["op"]]()
