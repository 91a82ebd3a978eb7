"""Cases of the 8-bit cache operators: append, decode attention, eviction.

The cache holds each request's first 64 tokens and its newest tokens (up to
256, in a ring) in BF16, and the tokens between them in 8 bits (e4m3 or int8)
with one fp32 scale per block of 16 tokens, KV head and side (K, V).  A page
is 64 tokens of every KV head: per head 4 blocks of [K 2048 B][V 2048 B] and
then 4 (K scale, V scale) pairs.

  append  T new tokens per request go to the sink and the window; whole blocks
          of 16 that the 256-token window cannot hold are quantised into the
          history.  T = 1 is a decode step, T = 64 a chunk, a long T into an
          empty request a prompt.
  decode  attention of one query token per request over all three regions;
          with `track`, the attention weight of every block is added up.
  evict   the history blocks with the smallest weights leave each head, in
          multiples of 256 tokens, and the others are packed together.

Length arithmetic is on the host (`lens`: what a scheduler knows anyway);
appending and evicting change the lengths, so those passes first set them back
(one small copy): the next pass meets the same work.
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
        # one decode step's append at 100K tokens, 8 KV heads: the window is full, so a block is quantised
        {"name": "append step b1 e4m3", "op": "append", "type": "e4m3", "B": 1, "Hkv": 8, "G": 4, "T": 1,
         "lo": 100000, "hi": 100000, "track": False},
        # the same for a batch of 32 ragged requests with weights kept for eviction
        {"name": "append step b32 int8", "op": "append", "type": "int8", "B": 32, "Hkv": 8, "G": 4, "T": 1,
         "lo": 8000, "hi": 32000, "track": True},
        # a 64-token chunk after its attention, odd lengths
        {"name": "append chunk64 b4 int8", "op": "append", "type": "int8", "B": 4, "Hkv": 8, "G": 4, "T": 64,
         "lo": 301, "hi": 9001, "track": False},
        # a whole prompt into an empty request
        {"name": "append prompt 100k e4m3", "op": "append", "type": "e4m3", "B": 1, "Hkv": 8, "G": 4, "T": 100003,
         "lo": 0, "hi": 0, "track": False},
        # latency: a short conversation, one request
        {"name": "decode 1k b1 int8", "op": "decode", "type": "int8", "B": 1, "Hkv": 8, "G": 4,
         "lo": 1021, "hi": 1021, "track": False},
        # the framework's headline shape: 100K tokens, one request, 32/8 heads
        {"name": "decode 100k b1 e4m3", "op": "decode", "type": "e4m3", "B": 1, "Hkv": 8, "G": 4,
         "lo": 100000, "hi": 100000, "track": False},
        # a serving batch of ragged lengths, weights tracked
        {"name": "decode b32 int8 track", "op": "decode", "type": "int8", "B": 32, "Hkv": 8, "G": 4,
         "lo": 8000, "hi": 32000, "track": True},
        # long requests with 8 query heads per KV head, weights tracked
        {"name": "decode 131k b8 g8 track", "op": "decode", "type": "e4m3", "B": 8, "Hkv": 8, "G": 8,
         "lo": 131071, "hi": 131071, "track": True},
        # the same length without grouped heads, few KV heads (one rank of a sharded model)
        {"name": "decode 131k b2 g1 e4m3", "op": "decode", "type": "e4m3", "B": 2, "Hkv": 2, "G": 1,
         "lo": 100003, "hi": 131071, "track": False},
        # steady state of a cache kept at a budget: 256 tokens too many in every request
        {"name": "evict step b32", "op": "evict", "type": "int8", "B": 32, "Hkv": 8, "G": 4,
         "lo": 8570, "hi": 8800, "budget": 8192},
        # a long prompt cut to a fifth
        {"name": "evict 100k to 20k b4", "op": "evict", "type": "e4m3", "B": 4, "Hkv": 8, "G": 4,
         "lo": 90000, "hi": 100000, "budget": 20000},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "evict"])
    c = {"op": op, "type": rng.choice(["e4m3", "int8"]), "Hkv": rng.choice([1, 2, 4, 8, 8]), "G": rng.choice([1, 2, 4, 8]),
         "B": _spread(rng, 1, 32)}
    most = 1_000_000 // (c["B"] * c["Hkv"])  # tokens a request: no more than the largest listed case
    if op == "append":
        if rng.random() < 0.4:
            c.update(T=_spread(rng, 2, min(100_000, most)), lo=0, hi=0)
        else:
            c.update(T=rng.choice([1, 1, 1, rng.randint(2, 300)]), hi=_spread(rng, 1, min(100_000, most)))
            c["lo"] = rng.randint(0, c["hi"])
        c["track"] = rng.random() < 0.5
    elif op == "decode":
        c["hi"] = _spread(rng, 1, min(400_000, 4 * most))
        c["lo"] = rng.randint(0, c["hi"])
        c["track"] = rng.random() < 0.5
    else:
        c["hi"] = _spread(rng, 700, min(200_000, 2 * most) + 700)
        c["lo"] = rng.randint(321, c["hi"])
        c["budget"] = rng.randint(0, c["hi"])
    return c


def _requests(case):
    """(seq, hist) of each request before the pass: spread evenly over lo..hi."""
    B, lo, hi = case["B"], case["lo"], case["hi"]
    out = []
    for b in range(B):
        L = lo + (hi - lo) * b // max(1, B - 1) if B > 1 else hi
        H = BLK * -(-max(L - SINK - RING, 0) // BLK)
        if case["op"] == "append" and case["T"] == 1 and L > SINK + RING and b % 2 == 0:
            L += -(L - SINK) % BLK  # a full window: this step quantises a block
            H = L - SINK - RING
        out.append((L, H))
    return out


def _after(case, L, H):
    """(seq, hist) after the pass."""
    if case["op"] == "append":
        L += case["T"]
        H += BLK * -(-max(L - SINK - H - RING, 0) // BLK) if L > SINK else 0
    elif case["op"] == "evict":
        out = max(H - case["budget"], 0) // RING * RING
        L, H = L - out, H - out
    return L, H


# ------------------------------------------------------------ plain pieces
def _views(pool, Hkv):
    """(codes [pages][Hkv][4][2][2048] uint8, scales [pages][Hkv][4][2] fp32) of a pool, as views."""
    p = pool.view(-1, Hkv, HEAD_BYTES)
    codes = p[..., :4 * 4096].unflatten(-1, (4, 2, 2048))
    scales = p[..., 4 * 4096:].view(torch.float32).unflatten(-1, (4, 2))
    return codes, scales


def _as_bytes(y, kind):
    """Rounds fp32 y to the 8-bit type (ties to even) and gives its bytes."""
    if kind == "e4m3":
        return y.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(y).to(torch.int8).view(torch.uint8)


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


def _quantise(x, kind):
    """x [n][16][Hkv][128] -> (bytes, the same shape, scale [n][Hkv])."""
    x = x.float()
    am = x.abs().amax(dim=(1, 3)).clamp_min(TINY)
    # x * qmax is exact (8 by 7 bits), so the one rounding before the 8-bit one is the division's: ties stay ties
    return _as_bytes(x * QMAX[kind] / am[:, None, :, None], kind), am / QMAX[kind]


def _store(pool, Hkv, kind, page, sub, k, v):
    """Quantises blocks k, v [n][16][Hkv][128] into block `sub` [n] of page `page` [n]."""
    codes, scales = _views(pool, Hkv)
    for side, x in enumerate((k, v)):
        q, s = _quantise(x, kind)
        codes[page, :, sub, side] = _pack(q, side)
        scales[page, :, sub, side] = s


def _values(b, kind):
    return b.view(torch.float8_e4m3fn if kind == "e4m3" else torch.int8)


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


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    B, Hkv, G, kind = case["B"], case["Hkv"], case["G"], case["type"]
    reqs = _requests(case)
    after = [_after(case, L, H) for L, H in reqs]
    need = [-(-max(h0, h1) // PAGE) for (_, h0), (_, h1) in zip(reqs, after)]
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
    sink_k, sink_v, ring_k, ring_v = zeros(SINK), zeros(SINK), zeros(RING), zeros(RING)
    for b, (L, H) in enumerate(reqs):
        n = min(L, SINK)
        if n:
            k, v = _tokens(g, n, Hkv, st)
            sink_k[b, :, :n], sink_v[b, :, :n] = k.transpose(0, 1), v.transpose(0, 1)
        for j in range(0, H // BLK, 2048):  # the history, 32K tokens at a time
            m = min(2048, H // BLK - j)
            k, v = _tokens(g, m * BLK, Hkv, st)
            blk = torch.arange(j, j + m, device=DEV)
            _store(pool, Hkv, kind, table[b, blk // 4].long(), blk % 4, k.view(m, BLK, Hkv, D), v.view(m, BLK, Hkv, D))
        if L - SINK > H:
            k, v = _tokens(g, L - SINK - H, Hkv, st)
            slot = torch.arange(H, L - SINK, device=DEV) % RING
            ring_k[b, :, slot], ring_v[b, :, slot] = k.transpose(0, 1), v.transpose(0, 1)
    lens0 = torch.tensor([[r[0] for r in reqs], [r[1] for r in reqs]], dtype=torch.int32, device=DEV)
    lens = lens0.clone()
    s = {"case": case, "reqs": reqs, "after": after, "pages": (max_pages, num_pages), "lens": lens, "lens0": lens0,
         "cache": {"pool": pool, "page_table": table, "sink_k": sink_k, "sink_v": sink_v, "ring_k": ring_k,
                   "ring_v": ring_v, "seq_lens": lens[0], "hist_lens": lens[1]}, "weights": None, "calls": {}}
    if case.get("track") or case["op"] == "evict":  # what earlier steps added up: few blocks carry most of it
        w = torch.rand(B, Hkv, RING // BLK + 4 * max_pages, device=DEV, generator=g)
        s["weights"] = w ** 6 * 30.0
    if case["op"] == "append":
        k, v = _tokens(g, B * case["T"], Hkv, st)
        s["k"], s["v"] = k.view(B, case["T"], Hkv, D), v.view(B, case["T"], Hkv, D)
    elif case["op"] == "decode":
        q = torch.randn(B, Hkv, G, D, device=DEV, generator=g) + 0.7 * st["dir"][None, :, None]
        s["q"] = q.view(B, Hkv * G, D).bfloat16()
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Hkv * G, dtype=torch.float32, device=DEV)
    else:
        s["weights0"] = s["weights"].clone()
    return s


DECAY = 0.98  # of the tracked weights, per step


# ------------------------------------------------------------------- passes
@functools.lru_cache(maxsize=None)
def _engine(device, Hq, Hkv, B, max_pages, num_pages):
    """What a program makes once for its model and its memory: the context, and the working
    memory of each stream it works on (calls that overlap cannot share that)."""
    from bit_kv_cache_int2_gb300 import oscar

    cfg = oscar.make_config(1, Hq, Hkv, max_batch=B, max_pages_per_req=max_pages, num_pages=num_pages)
    return oscar, oscar.oscar_create(cfg), functools.lru_cache(maxsize=None)(lambda stream: oscar.alloc_scratch_kv8(cfg))


def _bind(s, stream):
    """The operator's call with this request batch's buffers, made once for a stream (the current
    one) and called every step."""
    c = s["case"]
    oscar, ctx, working = _engine(s["lens"].device.index, c["Hkv"] * c["G"], c["Hkv"], c["B"], *s["pages"])
    kind, scratch = oscar.KV8_E4M3 if c["type"] == "e4m3" else oscar.KV8_INT8, working(stream)
    if c["op"] == "append":
        f = oscar.bind_append_kv8(ctx, s["cache"], kind, c["T"], c["B"], weights=s["weights"])
        return lambda: f(s["k"].data_ptr(), s["v"].data_ptr())
    if c["op"] == "decode":
        return oscar.bind_decode_kv8(ctx, s["cache"], kind, s["q"], s["out"], s["lse"], scratch, c["B"],
                                     weights=s["weights"], decay=DECAY)
    return oscar.bind_evict_kv8(ctx, s["cache"], s["weights"], c["budget"], scratch, c["B"])


def run(s):
    c, cache = s["case"], s["cache"]
    if c["op"] != "decode":
        s["lens"].copy_(s["lens0"])
    if c["op"] == "evict":
        s["weights"].copy_(s["weights0"])
    if own:
        stream = torch._C._cuda_getCurrentRawStream(s["lens"].device.index)  # current_stream() makes an object: 4 us
        if stream not in s["calls"]:
            s["calls"][stream] = _bind(s, stream)
        s["calls"][stream]()
    elif c["op"] == "append":
        _append(s)
    elif c["op"] == "decode":
        _decode(s)
    else:
        _evict(s)
    if c["op"] == "decode":
        return {"out": s["out"], "lse": s["lse"], "weights": _weights(s)}
    codes, scales = _views(cache["pool"], c["Hkv"])
    got = {"codes": _values(codes, c["type"]), "scales": scales, "lens": s["lens"], "weights": _weights(s)}
    if c["op"] == "append":
        got.update({x: cache[x] for x in ("sink_k", "sink_v", "ring_k", "ring_v")})
    return got


def _weights(s):
    return s["weights"] if s["weights"] is not None else None


def _grid(counts, width):
    """[B][width] truth values, the first counts[b] of row b set."""
    return torch.arange(width, device=DEV)[None] < counts[:, None]


def _append(s):
    c, cache, B, T = s["case"], s["cache"], s["case"]["B"], s["case"]["T"]
    L, H = (x.long() for x in s["lens0"])
    end = torch.tensor(s["after"], device=DEV).T
    L1, H1 = end[0], end[1]
    new = {"k": s["k"], "v": s["v"]}
    # blocks that leave the window: tokens from the ring where they are older, else from the input
    nb = max((h1 - h0) // BLK for (_, h0), (_, h1) in zip(s["reqs"], s["after"]))
    b, j = _grid((H1 - H) // BLK, nb).nonzero(as_tuple=True)
    if b.numel():
        j = H[b] // BLK + j
        pos = (SINK + BLK * j)[:, None] + torch.arange(BLK, device=DEV)
        old = pos < L[b, None]
        rows = {x: torch.where(old[..., None, None], cache["ring_" + x][b[:, None], :, (pos - SINK) % RING],
                               new[x][b[:, None], (pos - L[b, None]).clamp_min(0)]) for x in "kv"}
        _store(cache["pool"], c["Hkv"], c["type"], cache["page_table"][b, j // 4].long(), j % 4, rows["k"], rows["v"])
        if s["weights"] is not None:
            was = (j * BLK + SINK) < L[b]  # the block was (partly) in the ring and has a weight
            s["weights"][b, :, RING // BLK + j] = torch.where(was[:, None], s["weights"][b, :, j % 16], 0.0)
    # what stays goes to the sink and the ring
    pos = L[:, None] + torch.arange(T, device=DEV)
    b, t = (pos < SINK).nonzero(as_tuple=True)
    for x in "kv":
        cache["sink_" + x][b, :, pos[b, t]] = new[x][b, t]
    b, t = (pos >= SINK + H1[:, None]).nonzero(as_tuple=True)
    for x in "kv":
        cache["ring_" + x][b, :, (pos[b, t] - SINK) % RING] = new[x][b, t]
    if s["weights"] is not None:  # blocks that begin in this call have none yet
        first = ((pos - SINK) % BLK == 0) & (pos >= SINK + H1[:, None])
        b, t = first.nonzero(as_tuple=True)
        s["weights"][b, :, (pos[b, t] - SINK) % RING // BLK] = 0.0
    s["lens"].copy_(end)


def _decode(s):
    c, cache = s["case"], s["cache"]
    B, Hkv, G, kind = c["B"], c["Hkv"], c["G"], c["type"]
    L, H = (x.long() for x in s["lens"])
    codes, scales = _views(cache["pool"], Hkv)
    pt = cache["page_table"].long().clamp_min(0)
    P = pt.shape[1]
    tok = {}
    for side, x in enumerate("kv"):
        y = _values(_unpack(codes[pt, :, :, side], side), kind).float() * scales[pt, :, :, side, None, None]
        y = y.permute(0, 2, 1, 3, 4, 5).reshape(B, Hkv, P * PAGE, D)  # [B][P][Hkv][4][16][128]
        tok[x] = torch.cat([cache["sink_" + x].float(), cache["ring_" + x].float(), y], dim=2)
    slot = (torch.arange(RING, device=DEV)[None] - H[:, None]) % RING
    seen = torch.cat([_grid(L.clamp_max(SINK), SINK), slot < (L - SINK - H)[:, None], _grid(H, P * PAGE)], dim=1)
    q = s["q"].float().view(B, Hkv, G, D)
    z = torch.matmul(q, tok["k"].transpose(2, 3)) * (1.0 / math.sqrt(D))
    z = z.masked_fill(~seen[:, None, None], -math.inf)
    m = z.amax(dim=-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(z - m)
    l = p.sum(dim=-1, keepdim=True)
    p = p / l.clamp_min(1e-30)
    v = tok["v"].masked_fill(~seen[:, None, :, None], 0.0)
    s["out"].copy_(torch.matmul(p, v).view(B, Hkv * G, D))
    s["lse"].copy_(torch.where(l > 0, m + torch.log(l), -math.inf).view(B, Hkv * G))
    if s["weights"] is not None:
        w = p[..., SINK:].sum(dim=2).unflatten(-1, (-1, BLK)).sum(dim=-1)
        held = seen[:, None, SINK:].unflatten(-1, (-1, BLK)).any(dim=-1)
        s["weights"].copy_(torch.where(held, s["weights"] * DECAY + w, s["weights"]))


def _evict(s):
    c, cache, w = s["case"], s["cache"], s["weights"]
    B, Hkv, R = c["B"], c["Hkv"], RING // BLK
    H = s["lens0"][1].long()
    out = (H - c["budget"]).clamp_min(0) // RING * RING // BLK
    n = H // BLK
    idx = torch.arange(w.shape[2] - R, device=DEV)
    order = torch.sort(w[..., R:].masked_fill(idx >= n[:, None, None], math.inf), dim=-1, stable=True)[1]
    gone = torch.zeros(w[..., R:].shape, dtype=torch.bool, device=DEV)
    gone.scatter_(-1, order, (idx < out[:, None, None]).expand_as(order))
    keep = (n - out)[:, None, None]
    hole = (gone & (idx < keep)).nonzero(as_tuple=True)
    last = (~gone & (idx >= keep) & (idx < n[:, None, None])).nonzero(as_tuple=True)
    b, h = hole[0], hole[1]
    to, at = cache["page_table"][b, hole[2] // 4].long(), cache["page_table"][b, last[2] // 4].long()
    for x in _views(cache["pool"], Hkv):
        x[to, h, hole[2] % 4] = x[at, h, last[2] % 4]
    w[b, h, R + hole[2]] = w[b, h, R + last[2]]
    s["lens"].copy_(s["lens0"] - (out * BLK).int())


# ------------------------------------------------------------------- figures
def work(case):
    B, Hkv, G = case["B"], case["Hkv"], case["G"]
    by = fl = 0
    block = 2 * BLK * D + 8  # codes of K and V and their scales
    for L, H in _requests(case):
        L1, H1 = _after(case, L, H)
        if case["op"] == "append":
            T = case["T"]
            made = (H1 - H) // BLK
            from_ring = max(0, min(L - SINK, H1) - H)
            stay = T - max(0, SINK + H1 - max(L, SINK)) if L1 > SINK else T
            by += Hkv * (4 * D * (T + from_ring + max(0, stay)) + made * block)
            fl += Hkv * made * 2 * BLK * D * 4
        elif case["op"] == "decode":
            by += Hkv * (H // BLK * block + (L - H) * 4 * D) + 2 * Hkv * G * D * 2 + Hkv * G * 4
            fl += 4 * Hkv * G * D * L
            if case["track"]:
                by += 8 * Hkv * (H // BLK + min(16, -(-max(L - SINK - H, 0) // BLK)))
        else:
            n, keep = H // BLK, H1 // BLK
            moved = (n - keep) * keep / max(n, 1)  # weights in no order: as many holes among the first
            by += Hkv * (4 * n + moved * 2 * (block + 4))
            fl += Hkv * n * 32
    return {"bytes": by + 8 * B, "flops": max(fl, 1)}


# ------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c, cache, kind, Hkv, G = case, s["cache"], case["type"], case["Hkv"], case["G"]
    table, lens = cache["page_table"].tolist(), s["after"]
    pages = cache["pool"].view(-1, Hkv, HEAD_BYTES)
    w = None if s["weights"] is None else s["weights"].double()
    if c["op"] == "decode":
        lane = torch.arange(2048, device=DEV)
        ch, ln, by = lane // 512, lane % 512 // 16, lane % 16
        gid, tq, hi, r, lo = ln // 4, ln % 4, by // 4 % 2, by // 2 % 2, by % 2
        place = [(8 * r + gid) * D + 32 * ch + 8 * tq + 4 * (by // 8) + 2 * hi + lo,
                 (8 * hi + 2 * tq + lo) * D + 16 * gid + 2 * (2 * ch + by // 8) + r]
        out = torch.zeros(c["B"], Hkv, G, D, dtype=torch.float64, device=DEV)
        lse = torch.full((c["B"], Hkv, G), -math.inf, dtype=torch.float64, device=DEV)
        for b, (L, H) in enumerate(lens):
            if L == 0:
                continue
            own_pages = pages[torch.tensor(table[b][:-(-H // PAGE)], dtype=torch.long, device=DEV)]
            for h in range(Hkv):
                raw = own_pages[:, h, :4 * 4096].reshape(-1, 2, 2048)[:H // BLK]
                sc = own_pages[:, h, 4 * 4096:].contiguous().view(torch.float32).reshape(-1, 2)[:H // BLK].double()
                kv = []
                for side, x in enumerate("kv"):
                    y = torch.empty(H // BLK, BLK * D, dtype=torch.float64, device=DEV)
                    y[:, place[side]] = _values(raw[:, side].contiguous(), kind).double() * sc[:, side, None]
                    win = cache["ring_" + x][b, h].double().roll(-(H % RING), 0)[:max(0, L - SINK - H)]
                    kv.append(torch.cat([cache["sink_" + x][b, h, :L].double(), y.view(-1, D), win]))
                z = s["q"].view(c["B"], Hkv, G, D)[b, h].double() @ kv[0].T / math.sqrt(D)
                p = torch.softmax(z, dim=-1)
                out[b, h], lse[b, h] = p @ kv[1], torch.logsumexp(z, dim=-1)
                if w is not None:
                    t = p.sum(0)
                    n, at = -(-max(0, L - SINK - H) // BLK), RING // BLK
                    hist = t[SINK:SINK + H].view(-1, BLK).sum(1)
                    w[b, h, at:at + H // BLK] = w[b, h, at:at + H // BLK] * DECAY + hist
                    rest = torch.zeros(n * BLK, dtype=torch.float64, device=DEV)
                    rest[:max(0, L - SINK - H)] = t[SINK + H:]
                    slots = (torch.arange(n, device=DEV) + H // BLK) % at
                    w[b, h, slots] = w[b, h, slots] * DECAY + rest.view(n, BLK).sum(1)
        return {"out": out.view(c["B"], -1, D), "lse": lse.view(c["B"], -1), "weights": w}
    codes = pages[..., :4 * 4096].reshape(-1, Hkv, 4, 2, 2048).clone()
    scales = pages[..., 4 * 4096:].contiguous().view(torch.float32).double().reshape(-1, Hkv, 4, 2)
    if c["op"] == "evict":
        for b, ((_, H), (_, H1)) in enumerate(zip(s["reqs"], lens)):
            n, keep = H // BLK, H1 // BLK
            for h in range(Hkv):
                row = w[b, h, 16:16 + n].cpu().numpy()
                bad = set(row.argsort(kind="stable")[:n - keep].tolist())
                holes = [i for i in range(keep) if i in bad]
                ends = [i for i in range(keep, n) if i not in bad]
                if holes:
                    t = torch.tensor(table[b], device=DEV)
                    i, j = torch.tensor(holes, device=DEV), torch.tensor(ends, device=DEV)
                    codes[t[i // 4], h, i % 4] = codes[t[j // 4], h, j % 4]
                    scales[t[i // 4], h, i % 4] = scales[t[j // 4], h, j % 4]
                    w[b, h, 16 + i] = w[b, h, 16 + j]
        return {"codes": _values(codes, kind).double() if kind == "e4m3" else None, "scales": scales, "weights": w}
    got = {x: cache[x].double() for x in ("sink_k", "sink_v", "ring_k", "ring_v")}
    tok, by, g, q = (torch.arange(x, device=DEV) for x in (BLK, 16, 8, 4))
    for b, ((L, H), (L1, H1)) in enumerate(zip(s["reqs"], lens)):
        for side, x in enumerate("kv"):
            new = s[x][b].double()  # [T][Hkv][128]
            held = torch.zeros(max(0, L - SINK - H), Hkv, D, dtype=torch.float64, device=DEV)
            if L - SINK > H:
                held = got["ring_" + x][b].roll(-(H % RING), 1)[:, :L - SINK - H].transpose(0, 1)
            first = max(0, min(SINK - L, case["T"]))
            got["sink_" + x][b, :, L:L + first] = new[:first].transpose(0, 1)
            line = torch.cat([held, new[first:]])  # tokens from position 64 + H on
            for j0 in range(0, (H1 - H) // BLK, 512):
                m = min(512, (H1 - H) // BLK - j0)
                y = line[j0 * BLK:(j0 + m) * BLK].view(m, BLK, Hkv, D).transpose(1, 2)  # [m][Hkv][16][128]
                am = y.abs().amax(dim=(2, 3)).clamp_min(TINY)
                v = y * QMAX[kind] / am[..., None, None]
                if kind == "e4m3":  # steps of 2^(e - 3) in [2^e, 2^(e + 1)), of 2^-9 below 2^-6
                    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
                    code = (torch.round(v / step) * step).float().to(torch.float8_e4m3fn).view(torch.uint8)
                else:
                    code = torch.round(v).to(torch.int8).view(torch.uint8)
                chunk = torch.arange(4, device=DEV)
                if side == 0:  # byte [c][g][q][i]: token and channel of each
                    t = (8 * (by // 2 % 2) + g[:, None, None])[None]
                    ch = 32 * chunk[:, None, None, None] + 8 * q[:, None] + 4 * (by // 8) + 2 * (by // 4 % 2) + by % 2
                else:
                    t = (8 * (by // 4 % 2) + 2 * q[:, None] + by % 2)[None, None]
                    ch = 16 * g[:, None, None] + 4 * chunk[:, None, None, None] + 2 * (by // 8) + by // 2 % 2
                t, ch = (z.expand(4, 8, 4, 16).reshape(-1) for z in (t, ch))
                blk = torch.arange(j0, j0 + m, device=DEV) + H // BLK
                page = torch.tensor(table[b], device=DEV)[blk // 4]
                codes[page, :, blk % 4, side] = code[:, :, t, ch]
                scales[page, :, blk % 4, side] = am / QMAX[kind]
            stay = line[H1 - H:]
            slots = torch.arange(H1, H1 + stay.shape[0], device=DEV) % RING
            got["ring_" + x][b, :, slots] = stay.transpose(0, 1)
        if w is not None:
            lo, hi = H // BLK, -(-max(0, L - SINK) // BLK)
            fresh = w[b].clone()
            for j in range(lo, max(hi, -(-max(0, L1 - SINK) // BLK))):
                value = w[b, :, j % 16] if j < hi else torch.zeros_like(w[b, :, 0])
                fresh[:, 16 + j if j < H1 // BLK else j % 16] = value
            w[b] = fresh
    return {"codes": _values(codes, kind).double() if kind == "e4m3" else None, "scales": scales, "weights": w, **got}
