"""Cases of the prompt's side of the 8-bit cache: positions, attention of a chunk, reading back.

The cache holds each request's first 64 tokens and its newest tokens (up to
256, in a ring) in BF16, and the tokens between them in 8 bits (e4m3 or int8)
with one fp32 scale per block of 16 tokens, KV head and side (K, V).  A page
is 64 tokens of every KV head: per head 4 blocks of [K 2048 B][V 2048 B] and
then 4 (K scale, V scale) pairs.

  rope     splits the rows of a fused projection into queries, keys and values,
           normalises each query and key head (optional) and turns its channels
           by the token's position: pairs in halves or interleaved, all
           channels or the first ones, frequencies scaled for long contexts.
  prefill  T new tokens per request attend to the request's cache and causally
           to one another: a few tokens to verify, a chunk, a whole prompt.
  read     the cached tokens of a range as dense BF16 keys and values: to move
           a request to another cache or another format.

The order of use is rope, prefill, append (the chunk goes into the cache), and
at some time read.
"""
import functools
import math

import torch

own = False  # set from outside: False: plain torch, True: the package's kernels

D, PAGE, SINK, RING, BLK = 128, 64, 64, 256, 16
HEAD_BYTES = 4 * 4096 + 32
QMAX = {"e4m3": 448.0, "int8": 127.0}
TINY = 2.0 ** -100  # the smallest magnitude that a scale is made from
DEV = "cuda"


def listed():
    return [
        # five drafted tokens checked at once, a short conversation: latency
        {"name": "prefill 5 tokens 1k b1 int8", "op": "prefill", "type": "int8", "B": 1, "Hkv": 8, "G": 4, "T": 5,
         "lo": 1021, "hi": 1021},
        # the same for a batch of ragged requests: the cache is read once, so memory counts
        {"name": "prefill 5 tokens b16 e4m3", "op": "prefill", "type": "e4m3", "B": 16, "Hkv": 8, "G": 4, "T": 5,
         "lo": 8000, "hi": 32000},
        # the framework's headline shape: a 64-token chunk after 100K tokens, 32/8 heads
        {"name": "prefill chunk64 100k b1 e4m3", "op": "prefill", "type": "e4m3", "B": 1, "Hkv": 8, "G": 4, "T": 64,
         "lo": 100000, "hi": 100000},
        # odd chunks of ragged requests, 8 query heads per KV head
        {"name": "prefill chunk509 b4 g8 int8", "op": "prefill", "type": "int8", "B": 4, "Hkv": 8, "G": 8, "T": 509,
         "lo": 301, "hi": 9001},
        # a whole prompt into an empty request: causal attention alone
        {"name": "prefill prompt 8191 int8", "op": "prefill", "type": "int8", "B": 1, "Hkv": 8, "G": 4, "T": 8191,
         "lo": 0, "hi": 0},
        # a large chunk of a long prompt
        {"name": "prefill chunk2048 100k e4m3", "op": "prefill", "type": "e4m3", "B": 1, "Hkv": 8, "G": 4, "T": 2048,
         "lo": 100003, "hi": 100003},
        # one decode step: a token far into its context, heads normalised
        {"name": "rope step b1", "op": "rope", "B": 1, "Hkv": 8, "G": 4, "T": 1, "at": 100000, "layout": "half",
         "dims": 128, "scaling": "none", "norm": True},
        # a chunk of four requests, half of the channels, positions squeezed by 4
        {"name": "rope chunk64 b4 part", "op": "rope", "B": 4, "Hkv": 8, "G": 8, "T": 64, "at": 9001, "layout": "interleaved",
         "dims": 64, "scaling": "linear", "norm": False},
        # a long prompt, frequencies scaled by parts
        {"name": "rope prompt 100k yarn", "op": "rope", "B": 1, "Hkv": 8, "G": 4, "T": 100003, "at": 0, "layout": "half",
         "dims": 128, "scaling": "yarn", "norm": True},
        # a short request read whole, by heads (as the other caches import it)
        {"name": "read 1k b1 int8", "op": "read", "type": "int8", "B": 1, "Hkv": 8, "G": 4, "first": 0, "n": 1021,
         "lo": 1021, "hi": 1021, "order": "heads"},
        # a ragged batch read by tokens (as an append takes it)
        {"name": "read b32 int8 tokens", "op": "read", "type": "int8", "B": 32, "Hkv": 8, "G": 4, "first": 7, "n": 32000,
         "lo": 8000, "hi": 32000, "order": "tokens"},
        # a long request moved to another format
        {"name": "read 100k b1 e4m3", "op": "read", "type": "e4m3", "B": 1, "Hkv": 8, "G": 4, "first": 0, "n": 100000,
         "lo": 100000, "hi": 100000, "order": "heads"},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "rope", "read"])
    c = {"op": op, "Hkv": rng.choice([1, 2, 4, 8, 8]), "G": rng.choice([1, 2, 4, 8]), "B": _spread(rng, 1, 32)}
    if op == "rope":
        c.update(T=_spread(rng, 1, max(1, 100_000 * 48 // (c["B"] * c["Hkv"] * (c["G"] + 2)))), at=_spread(rng, 1, 1 << 22) - 1,
                 layout=rng.choice(["half", "interleaved"]), dims=rng.choice([16, 32, 64, 96, 112, 128, 128, 128]),
                 scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), norm=rng.random() < 0.5)
        return c
    c["type"] = rng.choice(["e4m3", "int8"])
    most = 1_000_000 // (c["B"] * c["Hkv"])  # tokens a request: no larger caches than the listed ones
    c["hi"] = _spread(rng, 1, min(100_000, most) + 1) - 1
    c["lo"] = rng.randint(0, c["hi"])
    if op == "read":
        c["hi"], c["lo"] = max(1, c["hi"]), max(1, c["lo"])
        c["first"] = rng.choice([0, 0, rng.randint(0, c["hi"] - 1)])
        c["n"] = _spread(rng, 1, c["hi"])
        c["order"] = rng.choice(["heads", "tokens"])
    else:
        pairs = 2048 * 100_000 * 32 / (c["B"] * c["Hkv"] * c["G"])  # token pairs a request: the largest listed case's
        longest = int(min(8191, pairs / (c["hi"] + 1), math.sqrt(2 * pairs), 2_000_000 // (c["B"] * c["Hkv"] * c["G"])))
        c["T"] = rng.choice([_spread(rng, 1, max(1, longest)), _spread(rng, 1, max(1, longest)), min(longest, rng.randint(1, 16))])
        c["T"] = max(1, c["T"])
    return c


def _requests(case):
    """(seq, hist) of each request before the pass: spread evenly over lo..hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    lens = [lo + (hi - lo) * b // (B - 1) if B > 1 else hi for b in range(B)]
    return [(L, BLK * -(-max(L - SINK - RING, 0) // BLK)) for L in lens]


# ------------------------------------------------------------ plain pieces
def _views(pool, Hkv):
    """(codes [pages][Hkv][4][2][2048] uint8, scales [pages][Hkv][4][2] fp32) of a pool, as views."""
    p = pool.view(-1, Hkv, HEAD_BYTES)
    codes = p[..., :4 * 4096].unflatten(-1, (4, 2, 2048))
    scales = p[..., 4 * 4096:].view(torch.float32).unflatten(-1, (4, 2))
    return codes, scales


def _values(b, kind):
    return b.view(torch.float8_e4m3fn if kind == "e4m3" else torch.int8)


def _pack(codes, side):
    """[n][16][Hkv][128] bytes in token order -> [n][Hkv][2048] as a block stores them."""
    n, _, Hkv, _ = codes.shape
    if side == 0:  # token 8r + g, channel 32c + 8q + 4s + 2h + l
        x = codes.view(n, 2, 8, Hkv, 4, 4, 2, 2, 2).permute(0, 3, 4, 2, 5, 6, 7, 1, 8)
    else:  # token 8h + 2q + l, channel 16g + 4m + 2o + r
        x = codes.view(n, 2, 4, 2, Hkv, 8, 4, 2, 2).permute(0, 4, 6, 5, 2, 7, 1, 8, 3)
    return x.reshape(n, Hkv, 2048)


def _unpack(b, side):
    """[..., 2048] stored bytes -> [..., 16, 128] in token order."""
    lead = b.shape[:-1]
    if side == 0:
        x = b.reshape(-1, 4, 8, 4, 2, 2, 2, 2).permute(0, 6, 2, 1, 3, 4, 5, 7)
    else:
        x = b.reshape(-1, 4, 8, 4, 2, 2, 2, 2).permute(0, 5, 3, 7, 2, 1, 4, 6)
    return x.reshape(*lead, 16, 128)


def _store(pool, Hkv, kind, page, sub, k, v):
    """Quantises blocks k, v [n][16][Hkv][128] into block `sub` [n] of page `page` [n]."""
    codes, scales = _views(pool, Hkv)
    for side, x in enumerate((k, v)):
        x = x.float()
        am = x.abs().amax(dim=(1, 3)).clamp_min(TINY)
        y = x * QMAX[kind] / am[:, None, :, None]
        q = y.to(torch.float8_e4m3fn) if kind == "e4m3" else torch.round(y).to(torch.int8)
        codes[page, :, sub, side] = _pack(q.view(torch.uint8), side)
        scales[page, :, sub, side] = am / QMAX[kind]


# ---------------------------------------------------------------- inputs
def _channel_sizes(g, H):
    """Keys have a few large channels and a mean, as rotary keys do."""
    size = torch.rand(H, D, device=DEV, generator=g) + 0.5
    return size * torch.where(torch.rand(H, D, device=DEV, generator=g) < 0.05, 4.0, 1.0)


def _tokens(g, n, Hkv, st):
    """n tokens' keys and values, [n][Hkv][128] BF16; one in fifty is a token that many queries look for."""
    k = torch.randn(n, Hkv, D, device=DEV, generator=g) * st["size"] + st["mean"]
    k += (torch.rand(n, 1, 1, device=DEV, generator=g) < 0.02) * st["dir"]
    v = torch.randn(n, Hkv, D, device=DEV, generator=g) * (0.2 + torch.rand(n, 1, 1, device=DEV, generator=g))
    return k.bfloat16(), v.bfloat16()


def _prepare_rope(case, g):
    B, T, Hkv, Hq = case["B"], case["T"], case["Hkv"], case["Hkv"] * case["G"]
    size = torch.rand(Hq + 2 * Hkv, D, device=DEV, generator=g) * 1.5 + 0.25
    qkv = torch.empty(B, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    for b in range(B):
        qkv[b] = torch.randn(T, Hq + 2 * Hkv, D, device=DEV, generator=g) * size
    at = torch.randint(0, 1 + case["at"] // 8, (B,), device=DEV, generator=g)
    s = {"case": case, "qkv": qkv, "positions": (case["at"] - at).int(), "gamma_q": None, "gamma_k": None, "calls": {}}
    if case["norm"]:
        for x in ("gamma_q", "gamma_k"):
            s[x] = (1 + 0.2 * torch.randn(D, device=DEV, generator=g)).bfloat16()
    for x, H in (("q", Hq), ("k", Hkv), ("v", Hkv)):
        s[x] = torch.zeros(B, T, H, D, dtype=torch.bfloat16, device=DEV)
    return s


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    if case["op"] == "rope":
        return _prepare_rope(case, g)
    B, Hkv, G, kind = case["B"], case["Hkv"], case["G"], case["type"]
    reqs = _requests(case)
    need = [-(-H // PAGE) for _, H in reqs]
    max_pages, num_pages = max(max(need), 1), sum(need) + 3
    ids = torch.randperm(num_pages, device=DEV, generator=g).int()
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    st = {"size": _channel_sizes(g, Hkv), "mean": torch.randn(Hkv, D, device=DEV, generator=g) * 0.5,
          "dir": torch.randn(Hkv, D, device=DEV, generator=g) * 0.6}
    pool = torch.zeros(num_pages * Hkv * HEAD_BYTES, dtype=torch.uint8, device=DEV)
    zeros = lambda n: torch.zeros(B, Hkv, n, D, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    win = {"sink_k": zeros(SINK), "sink_v": zeros(SINK), "ring_k": zeros(RING), "ring_v": zeros(RING)}
    for b, (L, H) in enumerate(reqs):
        n = min(L, SINK)
        if n:
            k, v = _tokens(g, n, Hkv, st)
            win["sink_k"][b, :, :n], win["sink_v"][b, :, :n] = k.transpose(0, 1), v.transpose(0, 1)
        for j in range(0, H // BLK, 2048):  # the history, 32K tokens at a time
            m = min(2048, H // BLK - j)
            k, v = _tokens(g, m * BLK, Hkv, st)
            blk = torch.arange(j, j + m, device=DEV)
            _store(pool, Hkv, kind, table[b, blk // 4].long(), blk % 4, k.view(m, BLK, Hkv, D), v.view(m, BLK, Hkv, D))
        if L - SINK > H:
            k, v = _tokens(g, L - SINK - H, Hkv, st)
            slot = torch.arange(H, L - SINK, device=DEV) % RING
            win["ring_k"][b, :, slot], win["ring_v"][b, :, slot] = k.transpose(0, 1), v.transpose(0, 1)
    lens = torch.tensor([[r[0] for r in reqs], [r[1] for r in reqs]], dtype=torch.int32, device=DEV)
    s = {"case": case, "reqs": reqs, "pages": (max_pages, num_pages), "calls": {},
         "cache": {"pool": pool, "page_table": table, **win, "seq_lens": lens[0], "hist_lens": lens[1]}}
    if case["op"] == "prefill":
        T = case["T"]
        k, v = _tokens(g, B * T, Hkv, st)
        s["k"], s["v"] = k.view(B, T, Hkv, D), v.view(B, T, Hkv, D)
        s["q"] = torch.empty(B, T, Hkv * G, D, dtype=torch.bfloat16, device=DEV)
        for b in range(B):
            q = torch.randn(T, Hkv, G, D, device=DEV, generator=g) + 0.7 * st["dir"][None, :, None]
            s["q"][b] = q.view(T, Hkv * G, D)
        s["out"] = torch.zeros_like(s["q"])
        s["lse"] = torch.zeros(B, T, Hkv * G, dtype=torch.float32, device=DEV)
    else:
        shape = (B, Hkv, case["n"], D) if case["order"] == "heads" else (B, case["n"], Hkv, D)
        for x in ("K", "V"):  # rows behind a request's end stay as they are
            s[x] = torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    return s


THETA, EPS = 1e6, 1e-6
FACTOR, TRAINED = 4.0, 32768  # of the scaled frequencies: longer by this, than these positions


# ------------------------------------------------------------------- passes
@functools.lru_cache(maxsize=None)
def _engine(device, Hq, Hkv, B, max_pages, num_pages):
    """What a program makes once for its model and its memory: the context, and the working
    memory of each stream it works on (calls that overlap cannot share that)."""
    from bit_kv_cache_int2_gb300 import oscar

    cfg = oscar.make_config(1, Hq, Hkv, max_batch=B, max_pages_per_req=max_pages, num_pages=num_pages)
    return oscar, oscar.oscar_create(cfg), functools.lru_cache(maxsize=None)(
        lambda stream: oscar.alloc_scratch_kv8(cfg, prefill=True))


@functools.lru_cache(maxsize=None)
def _rope_table(layout, dims, scaling):
    """The turning speeds of a model, made once."""
    from bit_kv_cache_int2_gb300 import oscar

    kinds = {"none": oscar.ROPE_PLAIN, "linear": oscar.ROPE_LINEAR, "ntk": oscar.ROPE_NTK, "bands": oscar.ROPE_BANDS,
             "yarn": oscar.ROPE_YARN}
    return oscar.make_rope(oscar.ROPE_HALF if layout == "half" else oscar.ROPE_INTERLEAVED, dims, THETA, kinds[scaling],
                           factor=FACTOR, trained=TRAINED)


def _bind(s, stream):
    """The operator's call with this state's buffers, made once for a stream (the current one)."""
    c = s["case"]
    if c["op"] == "rope":
        oscar, ctx, _ = _engine(s["qkv"].device.index, c["Hkv"] * c["G"], c["Hkv"], c["B"], 1, 1)
        return oscar.bind_rope(ctx, _rope_table(c["layout"], c["dims"], c["scaling"]), s["qkv"], s["positions"], c["T"], s["q"],
                               s["k"], s["v"], c["B"], gamma_q=s["gamma_q"], gamma_k=s["gamma_k"], eps=EPS)
    oscar, ctx, working = _engine(s["cache"]["pool"].device.index, c["Hkv"] * c["G"], c["Hkv"], c["B"], *s["pages"])
    kind = oscar.KV8_E4M3 if c["type"] == "e4m3" else oscar.KV8_INT8
    if c["op"] == "prefill":
        return oscar.bind_prefill_kv8(ctx, s["cache"], kind, s["q"], s["k"], s["v"], c["T"], s["out"], s["lse"],
                                      working(stream), c["B"])
    return oscar.bind_read_kv8(ctx, s["cache"], kind, c["first"], c["n"], s["K"], s["V"], c["B"],
                               order=oscar.ORDER_HEADS if c["order"] == "heads" else oscar.ORDER_TOKENS)


def run(s):
    op = s["case"]["op"]
    if own:
        stream = torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())  # current_stream() makes an object: 4 us
        if stream not in s["calls"]:
            s["calls"][stream] = _bind(s, stream)
        s["calls"][stream]()
    else:
        {"rope": _rope, "prefill": _prefill, "read": _read}[op](s)
    return {x: s[x] for x in {"rope": ("q", "k", "v"), "prefill": ("out", "lse"), "read": ("K", "V")}[op]}


def _speeds(case):
    """Radians a position of each channel pair (64 bits), and what cosine and sine are multiplied by."""
    n = case["dims"] // 2
    i = torch.arange(n, dtype=torch.float64, device=DEV)
    w = THETA ** (-2.0 * i / case["dims"])
    if case["scaling"] == "linear":
        return w / FACTOR, 1.0
    if case["scaling"] == "ntk":
        return (THETA * FACTOR ** (case["dims"] / (case["dims"] - 2))) ** (-2.0 * i / case["dims"]), 1.0
    if case["scaling"] == "bands":  # turns over the trained length: above 4 as they are, below 1 slower, a blend between
        keep = ((TRAINED * w / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return w * keep + w / FACTOR * (1 - keep), 1.0
    if case["scaling"] == "yarn":  # a ramp between the pairs that turn 32 times and once over the trained length
        at = [case["dims"] * math.log(TRAINED / (r * 2 * math.pi)) / (2 * math.log(THETA)) for r in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), n - 1)
        slow = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return w * (1 - slow) + w / FACTOR * slow, 0.1 * math.log(FACTOR) + 1.0
    return w, 1.0


def _rope(s):
    c = s["case"]
    w, size = _speeds(c)
    n, Hkv, Hq = c["dims"] // 2, c["Hkv"], c["Hkv"] * c["G"]
    heads = s["qkv"].split([Hq, Hkv, Hkv], dim=2)
    s["v"].copy_(heads[2])
    at = s["positions"].long()[:, None] + torch.arange(c["T"], device=DEV)
    a = at.double()[..., None] * w
    cos, sin = (torch.cos(a) * size).float()[:, :, None], (torch.sin(a) * size).float()[:, :, None]
    for x, out, gamma in ((heads[0], s["q"], s["gamma_q"]), (heads[1], s["k"], s["gamma_k"])):
        x = x.float()
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * gamma.float()
        if c["layout"] == "half":
            p, r, rest = x[..., :n], x[..., n:2 * n], x[..., 2 * n:]
            out.copy_(torch.cat([p * cos - r * sin, r * cos + p * sin, rest], dim=-1))
        else:
            y = x[..., :2 * n].unflatten(-1, (n, 2))
            p, r = y[..., 0], y[..., 1]
            y = torch.stack([p * cos - r * sin, r * cos + p * sin], dim=-1).flatten(-2)
            out.copy_(torch.cat([y, x[..., 2 * n:]], dim=-1))


def _cached(s, b):
    """Keys and values of request b, [Hkv][L][128] in 32 bits, in the cache's order."""
    c, cache, (L, H) = s["case"], s["cache"], s["reqs"][b]
    codes, scales = _views(cache["pool"], c["Hkv"])
    pages = cache["page_table"][b, :-(-H // PAGE)].long()
    out = []
    slot = torch.arange(H, max(L - SINK, H), device=DEV) % RING
    for side, x in enumerate("kv"):
        y = _values(_unpack(codes[pages, :, :, side], side), c["type"]).float() * scales[pages, :, :, side, None, None]
        y = y.transpose(0, 1).reshape(c["Hkv"], -1, D)[:, :H]  # [pages][Hkv][4][16][128]
        out.append(torch.cat([cache["sink_" + x][b, :, :min(L, SINK)].float(), y, cache["ring_" + x][b, :, slot].float()], dim=1))
    return out


def _prefill(s):
    c = s["case"]
    T, Hkv, G = c["T"], c["Hkv"], c["G"]
    for b, (L, _) in enumerate(s["reqs"]):
        K, V = _cached(s, b)
        K = torch.cat([K, s["k"][b].transpose(0, 1).float()], dim=1)
        V = torch.cat([V, s["v"][b].transpose(0, 1).float()], dim=1)
        q = s["q"][b].view(T, Hkv, G, D).permute(1, 2, 0, 3).float()  # [Hkv][G][T][128]
        step = max(1, (1 << 28) // (Hkv * G * (L + T)))
        for t in range(0, T, step):
            rows = torch.arange(t, min(t + step, T), device=DEV)
            z = torch.matmul(q[:, :, t:t + step], K[:, None].transpose(2, 3)) * (1.0 / math.sqrt(D))
            z = z.masked_fill(torch.arange(L + T, device=DEV) > L + rows[:, None], -math.inf)
            m = z.amax(dim=-1, keepdim=True).clamp_min(-1e30)
            p = torch.exp(z - m)
            l = p.sum(dim=-1, keepdim=True)
            o = torch.matmul(p / l, V[:, None])
            s["out"][b, t:t + step] = o.permute(2, 0, 1, 3).reshape(len(rows), Hkv * G, D)
            s["lse"][b, t:t + step] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(len(rows), Hkv * G)


def _read(s):
    c = s["case"]
    for b, (L, _) in enumerate(s["reqs"]):
        n = min(L, c["first"] + c["n"]) - c["first"]
        if n <= 0:
            continue
        for x, y in zip("KV", _cached(s, b)):
            y = y[:, c["first"]:c["first"] + n]
            if c["order"] == "heads":
                s[x][b, :, :n] = y
            else:
                s[x][b, :n] = y.transpose(0, 1)


# ------------------------------------------------------------------- figures
def work(case):
    B, Hkv, G = case["B"], case["Hkv"], case["G"]
    if case["op"] == "rope":
        heads = B * case["T"] * Hkv * (G + 2)
        return {"bytes": 4 * D * heads + 4 * B, "flops": heads * D * (3 + 4 * case["norm"])}
    by = fl = 0
    for L, H in _requests(case):
        if case["op"] == "read":
            n0, n1 = case["first"], min(L, case["first"] + case["n"])
            n = max(n1 - n0, 0)
            h = max(min(n1, SINK + H) - max(n0, SINK), 0)
            by += Hkv * (h * (2 * D + 8 / BLK) + (n - h) * 4 * D + n * 4 * D)
            fl += Hkv * h * 2 * D
        else:
            T = case["T"]
            by += Hkv * (H * (2 * D + 8 / BLK) + (L - H + T) * 4 * D) + T * Hkv * G * (4 * D + 4)
            fl += 4 * D * Hkv * G * (T * L + T * (T + 1) // 2)
    return {"bytes": int(by) + 8 * B, "flops": max(fl, 1)}


# ------------------------------------------------------- the definition, in 64 bits
def _exact_rope(s):
    c, n = s["case"], s["case"]["dims"] // 2
    w, size = _speeds(c)
    Hq, Hkv = c["Hkv"] * c["G"], c["Hkv"]
    got = {}
    for name, at, H, gamma in (("q", 0, Hq, s["gamma_q"]), ("k", Hq, Hkv, s["gamma_k"])):
        got[name] = torch.empty(c["B"], c["T"], H, D, dtype=torch.float64, device=DEV)
        first = torch.arange(n, device=DEV) * (1 if c["layout"] == "half" else 2)
        second = first + (n if c["layout"] == "half" else 1)
        for b in range(c["B"]):
            for t in range(0, c["T"], 8192):
                x = s["qkv"][b, t:t + 8192, at:at + H].double()
                if gamma is not None:
                    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.double()
                pos = s["positions"][b].double() + torch.arange(t, t + x.shape[0], device=DEV, dtype=torch.float64)
                turn = torch.polar(torch.full((x.shape[0], 1, n), size, dtype=torch.float64, device=DEV), (pos[:, None] * w)[:, None])
                z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
                x[..., first], x[..., second] = z.real, z.imag
                got[name][b, t:t + 8192] = x
    got["v"] = s["qkv"][:, :, Hq + Hkv:].double()
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s) if case["B"] * case["T"] * case["Hkv"] * (case["G"] + 2) <= 6_000_000 else None
    c, cache, kind, Hkv, G = case, s["cache"], case["type"], case["Hkv"], case["G"]
    lane = torch.arange(2048, device=DEV)
    ch, ln, by = lane // 512, lane % 512 // 16, lane % 16
    gid, tq, hi, r, lo = ln // 4, ln % 4, by // 4 % 2, by // 2 % 2, by % 2
    place = [(8 * r + gid) * D + 32 * ch + 8 * tq + 4 * (by // 8) + 2 * hi + lo,
             (8 * hi + 2 * tq + lo) * D + 16 * gid + 2 * (2 * ch + by // 8) + r]
    pages = cache["pool"].view(-1, Hkv, HEAD_BYTES)
    pos = {x: torch.arange(n, device=DEV) for x, n in (("ring", RING), ("blk", BLK))}

    def cached(b, h):
        L, H = s["reqs"][b]
        mine = pages[cache["page_table"][b, :-(-H // PAGE)].long(), h]
        raw = mine[:, :4 * 4096].reshape(-1, 2, 2048)[:H // BLK]
        sc = mine[:, 4 * 4096:].contiguous().view(torch.float32).reshape(-1, 2)[:H // BLK].double()
        out = []
        for side, x in enumerate("kv"):
            y = torch.empty(H // BLK, BLK * D, dtype=torch.float64, device=DEV)
            y[:, place[side]] = _values(raw[:, side].contiguous(), kind).double() * sc[:, side, None]
            win = cache["ring_" + x][b, h].double()[(pos["ring"] + H) % RING][:max(0, L - SINK - H)]
            out.append(torch.cat([cache["sink_" + x][b, h, :L].double(), y.view(-1, D), win]))
        return out

    if c["op"] == "read":
        got = {x: s[x].double() for x in "KV"}
        for b, (L, _) in enumerate(s["reqs"]):
            n = max(0, min(L, c["first"] + c["n"]) - c["first"])
            for h in range(Hkv):
                for x, y in zip("KV", cached(b, h)):
                    to = got[x][b, h] if c["order"] == "heads" else got[x][b, :, h]
                    to[:n] = y[c["first"]:c["first"] + n]
        return got
    if work(case)["flops"] > 4e12:
        return None
    T = c["T"]
    out = torch.empty(c["B"], T, Hkv * G, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(c["B"], T, Hkv * G, dtype=torch.float64, device=DEV)
    for b, (L, _) in enumerate(s["reqs"]):
        for h in range(Hkv):
            K, V = (torch.cat([x, s[n][b, :, h].double()]) for x, n in zip(cached(b, h), "kv"))
            step = max(1, (1 << 27) // (L + T))
            for g in range(G):
                for t in range(0, T, step):
                    q = s["q"][b, t:t + step, h * G + g].double()
                    z = q @ K.T / math.sqrt(D)
                    z += torch.full_like(z, -math.inf).triu(L + t + 1)
                    lse[b, t:t + step, h * G + g] = torch.logsumexp(z, dim=-1)
                    out[b, t:t + step, h * G + g] = torch.softmax(z, dim=-1) @ V
    return {"out": out, "lse": lse}
