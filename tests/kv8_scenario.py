"""Shared pieces of the 8-bit-history tests: a device cache and the oracle
requests that go with it, driven in step."""
import numpy as np
import torch

from bit_kv_cache_int2_gb300 import oscar
from oracle import kv8_oracle as K8


class Pair:
    """A device cache of B requests and B oracle requests."""

    def __init__(self, kind, Hkv, G, B, pages, seed=0, max_batch=None, weights=True, dirty=True, num_pages=None):
        self.kind, self.Hkv, self.G, self.B, self.pages = kind, Hkv, G, B, pages
        mb = max_batch or B
        npg = num_pages or mb * pages
        self.cfg = oscar.make_config(1, Hkv * G, Hkv, max_batch=mb, max_pages_per_req=pages, num_pages=npg)
        self.ctx = oscar.oscar_create(self.cfg)
        self.g = torch.Generator().manual_seed(seed)
        self.cache = oscar.alloc_cache(self.cfg, kv8=True)
        if npg >= mb * pages:  # else the test hands out the pages
            ids = torch.randperm(npg, generator=self.g).int()[:mb * pages]
            self.cache["page_table"].copy_(ids.view(mb, pages))
        if dirty:  # NaN patterns wherever no token is: bf16 NaN, e4m3 NaN, fp32 NaN
            for x in ("pool", "sink_k", "sink_v", "ring_k", "ring_v"):
                self.cache[x].view(torch.uint8).fill_(0xFF)
        self.weights = oscar.alloc_weights_kv8(self.cfg) if weights else None
        self.scratch = oscar.alloc_scratch_kv8(self.cfg)
        self.scratch.fill_(0xFF)
        self.req = [K8.Request(Hkv, kind) for _ in range(B)]

    def close(self):
        torch.cuda.synchronize()
        oscar.oscar_destroy(self.ctx)

    def draw(self, T, scale=1.0, B=None):
        B = B or self.B
        amp = torch.exp2(torch.randint(-3, 4, (B, T, self.Hkv, 1), generator=self.g).float())
        k = (torch.randn(B, T, self.Hkv, 128, generator=self.g) * scale).bfloat16()
        v = (torch.randn(B, T, self.Hkv, 128, generator=self.g) * amp * scale).bfloat16()
        return k, v

    def append(self, T, kv=None, call=None, oracle=True):
        k, v = kv or self.draw(T)
        if call is None:
            oscar.oscar_append_kv8(self.ctx, self.cache, self.kind, k.cuda(), v.cuda(), T, self.B, weights=self.weights)
        else:
            call(k, v)
        if oracle:
            kn, vn = k.double().numpy(), v.double().numpy()
            for b, r in enumerate(self.req):
                for t in range(T):
                    r.append(kn[b, t], vn[b, t])

    def query(self, scale=1.0):
        return (torch.randn(self.B, self.Hkv * self.G, 128, generator=self.g) * scale).bfloat16()

    def decode(self, q, decay=1.0, weights=True):
        qd = q.cuda()
        out = torch.full_like(qd, float("nan"))
        lse = torch.full(qd.shape[:2], float("nan"), dtype=torch.float32, device="cuda")
        oscar.oscar_decode_kv8(self.ctx, self.cache, self.kind, qd, out, lse, self.scratch, self.B,
                               weights=self.weights if weights else None, decay=decay)
        return out, lse

    def host(self):
        """(codes [pages][Hkv][4][2][2048], scales [pages][Hkv][4][2]) of the pool."""
        p = self.cache["pool"].cpu().numpy().reshape(-1, self.Hkv, K8.HEAD_BYTES)
        return (p[..., :16384].reshape(-1, self.Hkv, 4, 2, 2048),
                np.ascontiguousarray(p[..., 16384:]).view(np.float32).reshape(-1, self.Hkv, 4, 2))

    def check_state(self, weight_tol=0.0):
        """The device state against the oracle's, bit for bit (weights: to a relative weight_tol)."""
        codes, scales = self.host()
        table = self.cache["page_table"].cpu().numpy()
        seq, hist = self.cache["seq_lens"].cpu().numpy(), self.cache["hist_lens"].cpu().numpy()
        w = self.weights.cpu().numpy() if self.weights is not None else None
        win = {x: self.cache[x].double().cpu().numpy() for x in ("sink_k", "sink_v", "ring_k", "ring_v")}
        for b, r in enumerate(self.req):
            assert (int(seq[b]), int(hist[b])) == (r.L, r.H), (b, int(seq[b]), int(hist[b]), r.L, r.H)
            for side, x in enumerate("kv"):
                for i, t in enumerate(r.sink):
                    np.testing.assert_array_equal(win["sink_" + x][b, :, i], t[side])
                for i, t in enumerate(r.window):
                    np.testing.assert_array_equal(win["ring_" + x][b, :, (r.H + i) % 256], t[side])
            for h in range(self.Hkv):
                for j, blk in enumerate(r.blocks[h]):
                    pg, sub = table[b, j // 4], j % 4
                    for side in (0, 1):
                        want = K8.pack(blk[2 * side], side)
                        assert np.array_equal(codes[pg, h, sub, side], want), (b, h, j, side)
                        assert np.array_equal(scales[pg, h, sub, side], blk[2 * side + 1], equal_nan=True), (b, h, j, side)
                if w is not None:
                    np.testing.assert_allclose(w[b, h, 16:16 + r.H // 16], np.asarray(r.w_hist[h], float), rtol=weight_tol, atol=weight_tol)
                    n = -(-len(r.window) // 16)
                    slots = [(r.H // 16 + i) % 16 for i in range(n)]
                    np.testing.assert_allclose(w[b, h, slots], r.w_ring[h, slots], rtol=weight_tol, atol=weight_tol)


def bounds(r, q, ps):
    """What rounding allows, per (head, query head[, channel]): (out, lse, p).

    A logit is an fp32 sum of 128 products on the tensor cores, at most 128
    roundings of 2^-23 of the sum of magnitudes, with a few more for the scale,
    the two exponentials and the sums (2^-19 relative to a weight).  History
    weights go through fp16: 2^-11 relative, 2^-25 of the largest where they are
    subnormal; window weights keep 16 bits.  The output is rounded to BF16."""
    G = q.shape[1]
    out, lse, dp = np.zeros(q.shape), np.zeros(q.shape[:2]), np.zeros((r.Hkv, G))
    for h in range(r.Hkv):
        K, V = r.tokens(h)
        mag = (np.abs(q[h]) @ np.abs(K).T).max(1) / np.sqrt(128) if len(K) else np.zeros(G)
        ds = 2.0 ** -16 * mag + 2.0 ** -19
        dp[h] = 2 * ds + 2.0 ** -19
        lse[h] = ds + 2.0 ** -19
        av = ps[h] @ np.abs(V)
        pv = (ps[h][:, :, None] * np.abs(V)[None]).max(1) if len(K) and len(K) < 4096 else np.abs(V).max(0)[None] if len(K) else 0.0
        top = ps[h].max(1)[:, None] * (np.abs(V).max() if len(V) else 0.0)
        out[h] = (2.0 ** -11 + dp[h][:, None]) * av + len(K) * 2.0 ** -25 * np.maximum(pv, top)
    return out, lse, dp


def check_decode(pair, q, out, lse, decay=None):
    """Outputs against the oracle; with decay the oracle's weights move too."""
    qn = q.double().numpy().reshape(pair.B, pair.Hkv, pair.G, 128)
    on = out.double().cpu().numpy().reshape(pair.B, pair.Hkv, pair.G, 128)
    ln = lse.double().cpu().numpy().reshape(pair.B, pair.Hkv, pair.G)
    worst = 0.0
    for b, r in enumerate(pair.req):
        ref, rl, ps = r.attend(qn[b], decay)
        if r.L == 0:
            assert (on[b] == 0).all() and np.isneginf(ln[b]).all()
            continue
        to, tl, dp = bounds(r, qn[b], ps)
        err = np.abs(on[b] - ref)
        lim = to + 2.0 ** -8 * (np.abs(ref) + to)
        assert (err <= lim).all(), (b, r.L, float((err / lim).max()))
        assert (np.abs(ln[b] - rl) <= tl + 2.0 ** -22 * np.abs(rl)).all(), (b, r.L)
        worst = max(worst, float(dp.max()))
    return worst


def dense(pair, b, h):
    """(K, V) [L][128] in float64 of a request's head from the device state itself (for long requests)."""
    L, H = int(pair.cache["seq_lens"][b]), int(pair.cache["hist_lens"][b])
    heads = pair.cache["pool"].view(-1, pair.Hkv, K8.HEAD_BYTES)[pair.cache["page_table"][b, :-(-H // 64)].long(), h]
    raw = heads[:, :16384].reshape(-1, 2, 2048)[:H // 16]
    scale = heads[:, 16384:].contiguous().view(torch.float32).view(-1, 2)[:H // 16].double()
    values = torch.from_numpy(K8.decode(np.arange(256, dtype=np.uint8), pair.kind)).cuda()
    out = []
    for side, x in enumerate("kv"):
        y = torch.empty(H // 16, 2048, dtype=torch.float64, device="cuda")
        y[:, torch.from_numpy(K8.PLACE[side]).cuda()] = values[raw[:, side].long()] * scale[:, side, None]
        win = pair.cache["ring_" + x][b, h].double().roll(-(H % 256), 0)[:max(0, L - 64 - H)]
        out.append(torch.cat([pair.cache["sink_" + x][b, h, :L].double(), y.view(-1, 128), win]))
    return out


def check_decode_dense(pair, q, out, lse, weights_before=None, decay=1.0):
    """As check_decode, from the device state: for requests too long for the oracle."""
    G = pair.G
    qd = q.cuda().double().view(pair.B, pair.Hkv, G, 128)
    od, ld = out.double().view(pair.B, pair.Hkv, G, 128), lse.double().view(pair.B, pair.Hkv, G)
    for b in range(pair.B):
        L, H = int(pair.cache["seq_lens"][b]), int(pair.cache["hist_lens"][b])
        if L == 0:
            assert bool((od[b] == 0).all()) and bool(torch.isneginf(ld[b]).all())
            continue
        for h in range(pair.Hkv):
            K, V = dense(pair, b, h)
            z = qd[b, h] @ K.T / 128 ** 0.5
            p = torch.softmax(z, 1)
            ref, rl = p @ V, torch.logsumexp(z, 1)
            ds = 2.0 ** -16 * (qd[b, h].abs() @ K.abs().T).amax(1, keepdim=True) / 128 ** 0.5 + 2.0 ** -19
            dp = 2 * ds + 2.0 ** -19
            lim = (2.0 ** -11 + dp) * (p @ V.abs()) + L * 2.0 ** -25 * p.amax(1, keepdim=True) * V.abs().max()
            lim = lim + 2.0 ** -8 * (ref.abs() + lim)
            assert bool(((od[b, h] - ref).abs() <= lim).all()), (b, h, float(((od[b, h] - ref).abs() / lim).max()))
            assert bool(((ld[b, h] - rl).abs() <= ds[:, 0] + 2.0 ** -19 + 2.0 ** -22 * rl.abs()).all()), (b, h)
            if weights_before is not None:
                t = p.sum(0)
                want = weights_before[b, h].double().clone()
                at = slice(16, 16 + H // 16)
                want[at] = want[at] * decay + t[min(L, 64):min(L, 64) + H].view(-1, 16).sum(1)
                n = -(-max(0, L - 64 - H) // 16)
                rest = torch.zeros(n * 16, dtype=torch.float64, device="cuda")
                rest[:max(0, L - 64 - H)] = t[min(L, 64) + H:]
                slots = (torch.arange(n, device="cuda") + H // 16) % 16
                want[slots] = want[slots] * decay + rest.view(n, 16).sum(1)
                got = pair.weights[b, h].double()
                held = torch.cat([slots, torch.arange(16, 16 + H // 16, device="cuda")])
                lim = float(dp.max()) * want + 2.0 ** -22 * want + 1e-12
                assert bool(((got - want).abs() <= lim)[held].all()), (b, h)
